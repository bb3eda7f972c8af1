"""The cache's oracle against cases worked by hand and against dense formulas."""
import numpy as np

import oracle
import synthetic as syn
from oracle import kv


def test_plan_worked_case():
    # pages of 16; request 0 continues inside a page, 1 starts, 2 has nothing, 3 fills its page exactly
    tables = np.full((4, 4), -1, np.int32)
    tables[0, 0], tables[3, 0] = 7, 9
    t, lens, off, slots, pos, used = kv.plan(np.array([14, 0, 0, 15]), np.array([3, 17, 0, 1]), 16,
                                             np.array([3, 1, 4, 5], np.int32), 1, tables, 22)
    assert t[0].tolist() == [7, 1, -1, -1] and t[1].tolist() == [4, 5, -1, -1] and t[3].tolist() == [9, -1, -1, -1]
    assert lens.tolist() == [17, 17, 0, 16] and off.tolist() == [0, 3, 20, 20, 21] and used == 4
    assert slots[:3].tolist() == [7 * 16 + 14, 7 * 16 + 15, 16] and slots[20] == 9 * 16 + 15 and slots[21] == -1
    assert pos[:4].tolist() == [14, 15, 16, 0]


def test_append_equals_act_quant_on_a_fresh_page():
    x = syn.normal_bf16(np.random.default_rng(0), (16, 1, 128), outlier_frac=0.01, outlier_mult=20)
    cache, scale = np.zeros((2, 1, 16, 128), np.uint8), np.zeros((2, 1), np.float32)
    c, s = kv.append(x, np.arange(16, 32), cache, scale)
    amax = np.abs(oracle.bf16_to_f32(x)).max()
    assert s[1, 0] == np.float32(amax) / np.float32(448) and s[0, 0] == 0
    got = oracle.e4m3_decode(c[1, 0]).reshape(16, 128) * s[1, 0]
    assert np.abs(got - oracle.bf16_to_f32(x).reshape(16, 128)).max() <= amax / 16


def test_append_scale_does_not_depend_on_the_steps():
    x = syn.normal_bf16(np.random.default_rng(1), (32, 2, 64))
    start = np.zeros((1, 2, 32, 64), np.uint8), np.zeros((1, 2), np.float32)
    _, whole = kv.append(x, np.arange(32), *start)
    c, s = start
    for i in range(32):
        c, s = kv.append(x[i:i + 1], np.arange(i, i + 1), c, s)
    assert np.array_equal(whole, s)


def test_attention_is_the_dense_formula():
    rng = np.random.default_rng(2)
    kc, vc = syn.random_e4m3_codes((3, 2, 16, 64), 3), syn.random_e4m3_codes((3, 2, 16, 64), 4)
    sk, sv = rng.random((3, 2)).astype(np.float32) * 0.01, rng.random((3, 2)).astype(np.float32)
    q = syn.normal_bf16(rng, (2, 4, 64))
    out, lse, _, _ = kv.attention(q, kc, sk, vc, sv, np.array([[2, 0]]), np.array([20]), np.array([0, 2]), 0.125)
    for j in range(2):
        for h in range(4):
            k = np.concatenate([oracle.e4m3_decode(kc[p, h // 2]).reshape(16, 64) * sk[p, h // 2] for p in (2, 0)])
            v = np.concatenate([oracle.e4m3_decode(vc[p, h // 2]).reshape(16, 64) * sv[p, h // 2] for p in (2, 0)])
            n = 19 + j
            s = k[:n] @ oracle.bf16_to_f32(q[j, h]).astype(np.float64) * 0.125
            e = np.exp(s - s.max())
            assert np.allclose(out[j, h], e @ v[:n] / e.sum(), rtol=1e-12)
            assert np.isclose(lse[j, h], np.log(np.exp(s).sum()), rtol=1e-12)


def test_attention_rows_with_nothing_to_see():
    kc = syn.random_e4m3_codes((1, 1, 16, 64), 5)
    one = np.ones((1, 1), np.float32)
    q = syn.normal_bf16(np.random.default_rng(3), (4, 1, 64))
    # request 0: 3 queries over 2 tokens (the first sees nothing); request 1: no tokens
    out, lse, _, _ = kv.attention(q, kc, one, kc, one, np.zeros((2, 1), np.int32), np.array([2, 0]),
                                  np.array([0, 3, 4]), 0.125)
    assert not out[0].any() and lse[0, 0] == -np.inf and not out[3].any() and lse[3, 0] == -np.inf
    assert out[1].any() and np.isfinite(lse[2, 0])


def test_append_errors_after_many_growths():
    # one token after the other, each a little larger than the last: the bounds that the header states
    n, d = 64, 64
    rng = np.random.default_rng(7)
    f = (rng.uniform(1.0, 2.0, (n, 1, d)) * np.sign(rng.standard_normal((n, 1, d)))).astype(np.float32)
    f *= (1.03 ** np.arange(n))[:, None, None].astype(np.float32)
    x = syn.to_bf16_bits(f)
    f = oracle.bf16_to_f32(x).astype(np.float64).reshape(n, d)
    for ue8m0 in (False, True):
        c, s = np.zeros((1, 1, n, d), np.uint8), np.zeros((1, 1), np.float32)
        grown, low = np.zeros(n), np.zeros(n)   # growths since a token was appended; what subnormal codes may have lost
        for i in range(n):
            was = s[0, 0]
            c, s = kv.append(x[i:i + 1], np.arange(i, i + 1), c, s, ue8m0)
            if s[0, 0] > was:
                grown[:i] += 1
                low[:i] += s[0, 0] * 2.0 ** -10
        assert grown[0] >= (2 if ue8m0 else 30)
        got = oracle.e4m3_decode(c[0, 0]).astype(np.float64).reshape(n, d) * float(s[0, 0])
        bound = np.abs(f) * (2.0 ** -4 if ue8m0 else ((1 + 2.0 ** -4) ** (grown + 1) - 1)[:, None]) + low[:, None] + s[0, 0] * 2.0 ** -10
        assert (np.abs(got - f) <= bound * (1 + 1e-6)).all()
