"""Attention over the paged 8-bit cache where a tile, a scale or a token is
unusual."""
import numpy as np
import pytest
import torch

import oracle
import synthetic as syn
from oracle import kv
from tests.helpers import host_bits
from tests.test_gpu_kv_attention import _case, _check, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import fp8_block_scaled_07_gb300 as m
    return m


# ------------------------------------------------------------------ tiles without a visible token
# the first 128 tokens left out: one page, or eight; single tokens and a few of
# them.  The four requests many times over, so that a CTA walks whole requests.
@pytest.mark.parametrize("bs", [16, 128])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [3, 2, 4, 1]])
@pytest.mark.parametrize("Hq,Hkv,dk,dv", [(8, 2, 128, 128), (1, 1, 64, 64), (16, 1, 64, 64), (6, 3, 192, 128)])
def test_first_tile_left_out(fp8, Hq, Hkv, dk, dv, bs, new):
    c = _case([400, 300, 1000, 130], new, bs, Hq, Hkv, dk, dv, seed=bs)
    c["vs"] *= np.float32(2.0 ** -6)   # V's scale far below 1: its logarithm, far below 0, is in every exponent
    tile = 128 // bs
    c["tables"][0, :tile] = -1
    c["vs"][c["tables"][1, :tile]] = 0.0
    c["tables"][2, :3 * tile] = 10 ** 6
    c["tables"][3, :tile] = -5
    want, wl, tol, eps = kv.attention(c["q"], c["kc"], c["ks"], c["vc"], c["vs"], c["tables"], c["lens"], c["offsets"], c["sm"])
    many = 240 // Hkv
    c.update(q=np.tile(c["q"], (many, 1, 1)), tables=np.tile(c["tables"], (many, 1)), lens=np.tile(c["lens"], many),
             offsets=np.concatenate([[0], np.cumsum(new * many)]).astype(np.int32))
    out, lse = _run(fp8, c, ragged=max(new) > 1)
    got = oracle.bf16_to_f32(host_bits(out)).astype(np.float64).reshape((many,) + want.shape)
    assert (np.abs(got - want) <= tol).all()
    gl = lse.cpu().numpy().astype(np.float64).reshape((many,) + wl.shape)
    assert np.isfinite(wl).all() and (np.abs(gl - wl) <= eps + 2.0 ** -18 * np.abs(wl)).all()


# holes of one tile throughout long requests that are split over the GPU: some ranges begin in one
@pytest.mark.parametrize("lens,Hkv,G,dk,dv", [([40000], 8, 1, 64, 64), ([9000, 30000], 2, 4, 128, 128)])
def test_ranges_that_begin_in_a_hole(fp8, lens, Hkv, G, dk, dv):
    c = _case(lens, [1] * len(lens), 128, Hkv * G, Hkv, dk, dv, seed=5)
    c["vs"] *= np.float32(2.0 ** -6)
    for b in range(len(lens)):
        c["tables"][b, b:-(-lens[b] // 128):3] = -1
    _check(fp8, c, ragged=False)


# ------------------------------------------------------------------ many small probabilities
# One token with weight 1 and thousands with e^-gap each, V with a common
# mean: together the small ones count.  They enter the product in multiples of
# 2^-18 of the largest, rounded either way: an error of at most that each, and
# at most half of it in the mean square, so that six standard deviations of
# the sum are 6 * 2^-19 * sqrt(sum v^2) (over sum p).  The rest of the bound:
# bf16's result, 9 significant bits of a probability, the scores' 2^-16.
@pytest.mark.parametrize("Hq,Hkv,dk,dv", [(8, 8, 64, 64), (32, 8, 128, 128), (16, 1, 128, 128)])
@pytest.mark.parametrize("flat", [True, False])
def test_many_small_probabilities(fp8, Hq, Hkv, dk, dv, flat):
    B, n, bs = 320 // Hkv, 8192, 128     # requests over the same pages: a range holds whole segments
    rng = np.random.default_rng(dk + Hq)
    P = n // bs
    kc = np.zeros((P, Hkv, bs, dk), np.uint8)
    if not flat:   # scores of a standard deviation of some 0.3
        kc[:] = oracle.e4m3_encode(rng.standard_normal(kc.shape).astype(np.float32) * 0.25).reshape(kc.shape)
    kc[0, :, 0] = oracle.e4m3_encode(np.ones(dk, np.float32))
    vc = oracle.e4m3_encode((1 + 0.25 * rng.standard_normal((P, Hkv, bs, dv))).astype(np.float32)).reshape(P, Hkv, bs, dv)
    one = np.ones((P, Hkv), np.float32)
    gaps = rng.choice([9.0, 11.0, 13.0, 13.5, 14.0], (B, Hq, 1))
    noise = rng.standard_normal((B, Hq, dk)) * (0.0 if flat else 0.3)
    q = syn.to_bf16_bits((gaps / np.sqrt(dk) + noise).astype(np.float32))
    c = dict(q=q, kc=kc, ks=one, vc=vc, vs=one, tables=np.tile(np.arange(P, dtype=np.int32), (B, 1)),
             lens=np.full(B, n, np.int32), offsets=np.arange(B + 1, dtype=np.int32), sm=dk ** -0.5)
    out, lse = _run(fp8, c, ragged=False)
    got = oracle.bf16_to_f32(host_bits(out)).astype(np.float64).reshape(B, Hq, dv)
    some = [0, B // 3, B - 1]
    kf, vf = (oracle.e4m3_decode(x).astype(np.float64).reshape(P, Hkv, bs, -1).transpose(1, 0, 2, 3).reshape(Hkv, n, -1)
              for x in (kc, vc))
    qf = oracle.bf16_to_f32(q).astype(np.float64).reshape(B, Hq, dk)
    for b in some:
        for h in range(Hq):
            k, v = kf[h * Hkv // Hq], vf[h * Hkv // Hq]
            s = k @ qf[b, h] * c["sm"]
            p = np.exp(s - s.max())
            want = p @ v / p.sum()
            tol = (np.abs(want) * 2.0 ** -8 + p @ np.abs(v) / p.sum() * (2.0 ** -9 + 2.0 ** -16) +
                   6 * 2.0 ** -19 * np.sqrt((v * v).sum(0)) / p.sum())
            assert (np.abs(got[b, h] - want) <= tol).all(), (b, h, np.abs(got[b, h] - want).max(), tol.max())
            assert abs(float(lse[b, h]) - (s.max() + np.log(p.sum()))) <= 2.0 ** -13


# ------------------------------------------------------------------ K's scale is zero, negative or lost in a product
@pytest.mark.parametrize("Hq,Hkv,dk,dv", [(8, 2, 128, 128), (4, 4, 64, 64), (3, 3, 192, 128)])
@pytest.mark.parametrize("new", [[1, 1], [2, 3], [200, 70]])
@pytest.mark.parametrize("scale,q_std", [(0.0, 1.0), (-0.0, 1.0), (-0.01, 30.0)])
def test_scales_of_k_that_are_not_positive(fp8, Hq, Hkv, dk, dv, new, scale, q_std):
    c = _case([400, 300], new, 32, Hq, Hkv, dk, dv, seed=17, q_std=q_std)
    for b, i in ((0, 1), (0, 7), (0, 12), (1, 0), (1, 8)):   # in tiles that every row sees, and in the last
        c["ks"][c["tables"][b, i]] = np.float32(scale)
    _check(fp8, c, ragged=new[0] > 1)


def test_products_of_scales_that_underflow(fp8):
    for new in ([1, 1], [200, 70]):
        c = _case([400, 300], new, 32, 8, 2, 128, 128, seed=18, q_std=0.0, sm_scale=1e-20)
        _check(fp8, c, ragged=new[0] > 1)


# ------------------------------------------------------------------ NaN in V
def _check_rows(fp8, c, T=None):
    """Every row against the oracle's answer for it alone, with the tokens that it sees and no others."""
    out, lse = _run(fp8, c)
    new = np.diff(c["offsets"])
    T = int(c["offsets"][-1])
    req = np.repeat(np.arange(len(new)), new)
    j = np.arange(T) - c["offsets"][req]
    lims = np.maximum(0, c["lens"][req] - new[req] + j + 1).astype(np.int32)
    want, wl, tol, eps = kv.attention(c["q"], c["kc"], c["ks"], c["vc"], c["vs"], c["tables"][req], lims,
                                      np.arange(T + 1), c["sm"])
    got = oracle.bf16_to_f32(host_bits(out)).astype(np.float64).reshape(want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = ~np.isnan(want)
    assert (np.abs(got - want)[fine] <= tol[fine]).all()
    gl = lse.cpu().numpy().astype(np.float64)
    live = np.isfinite(wl)
    assert np.array_equal(live, np.isfinite(gl))
    assert (np.abs(np.where(live, gl - np.where(live, wl, 0), 0))[live] <= (eps + 2.0 ** -18 * np.abs(np.where(live, wl, 0)))[live]).all()


@pytest.mark.parametrize("Hq,Hkv,dk,dv", [(8, 2, 128, 128), (4, 4, 64, 64), (3, 3, 192, 128), (16, 1, 64, 64)])
@pytest.mark.parametrize("lens,new", [([140, 9, 333], [3, 8, 2]), ([9000], [4]), ([300, 200, 129], [300, 140, 1]),
                                      ([5, 60], [9, 200]), ([700], [520])])
def test_nan_values_that_a_query_does_not_see(fp8, Hq, Hkv, dk, dv, lens, new):
    c = _case(lens, new, 16, Hq, Hkv, dk, dv, seed=21)
    rng = np.random.default_rng(22)
    for b, (n, m) in enumerate(zip(lens, new)):
        first = max(0, n - m)
        for t in {first, n - 1, (first + n) // 2, int(rng.integers(first, n)), int(rng.integers(0, n))}:
            h, d = int(rng.integers(Hkv)), int(rng.integers(dv))
            c["vc"][c["tables"][b, t // 16], h, t % 16, d] = 0x7F if t % 2 else 0xFF
    _check_rows(fp8, c)


# ------------------------------------------------------------------ fewer rows than tokens
@pytest.mark.parametrize("lens,new,T", [([300, 200], [150, 120], 200), ([300, 200], [150, 120], 120), ([40, 50], [3, 4], 5), ([700], [500], 2),
                                        ([30, 300, 60], [2, 200, 9], 140)])
def test_queries_end_inside_a_request(fp8, lens, new, T):
    c = _case(lens, new, 16, 8, 4, 128, 128, seed=23)
    want, wl, tol, eps = kv.attention(c["q"], c["kc"], c["ks"], c["vc"], c["vs"], c["tables"], c["lens"], c["offsets"], c["sm"])
    big = torch.full((T + 40, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 40, 8), 7.0, device="cuda")
    _run(fp8, {**c, "q": c["q"][:T]}, out=big[:T], lse=lse[:T])
    got = oracle.bf16_to_f32(host_bits(big[:T])).astype(np.float64).reshape(T, 8, 128)
    assert (np.abs(got - want[:T]) <= tol[:T]).all()
    assert (np.abs(lse[:T].cpu().numpy() - wl[:T]) <= eps[:T] + 2.0 ** -18 * np.abs(wl[:T])).all()
    assert (big[T:] == 7.0).all() and (lse[T:] == 7.0).all()


# ------------------------------------------------------------------ V's scale has no logarithm or no reciprocal
def test_scales_of_v_that_are_no_normal_numbers(fp8):
    for new in ([1, 1], [2, 3], [100, 70]):
        c = _case([400, 300], new, 32, 8, 2, 128, 128, seed=24)
        for (b, i), v in (((0, 1), 1e-40), ((0, 12), 3e-39), ((0, 6), np.inf), ((1, 0), np.nan), ((1, 3), -1.0), ((1, 9), 1e-45)):
            c["vs"][c["tables"][b, i]] = v
        out, lse = _run(fp8, c, ragged=new[0] > 1)
        c["vs"] = np.where((c["vs"] >= 2.0 ** -126) & np.isfinite(c["vs"]), c["vs"], 0).astype(np.float32)
        want, wl, tol, eps = kv.attention(c["q"], c["kc"], c["ks"], c["vc"], c["vs"], c["tables"], c["lens"], c["offsets"], c["sm"])
        got = oracle.bf16_to_f32(host_bits(out)).astype(np.float64).reshape(want.shape)
        assert (np.abs(got - want) <= tol).all()
        assert (np.abs(lse.cpu().numpy() - wl) <= eps + 2.0 ** -18 * np.abs(wl)).all()
