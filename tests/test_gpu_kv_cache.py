"""GPU parity of the paged 8-bit cache's plan and append: integers and codes
equal the oracle's exactly."""
import numpy as np
import pytest
import torch

import oracle
import synthetic as syn
from oracle import kv
from tests.helpers import dev_bf16, dev_e4m3, dev_f32, dev_i32, host_bits, host_f32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import fp8_block_scaled_07_gb300 as m
    return m


def _plan(fp8, past, new, bs, free, used, tables, T, **kw):
    tab = dev_i32(tables)
    lens, off, slots, pos, u = fp8.fp8_kv_plan(dev_i32(past), dev_i32(new), dev_i32(free), dev_i32([used]), tab, bs, T, **kw)
    fp8.fp8_device_status()
    return [x.cpu().numpy() for x in (tab, lens, off, slots, pos)] + [int(u.item())]


def _check_plan(fp8, past, new, bs, free, used, tables, T):
    got = _plan(fp8, past, new, bs, free, used, tables, T)
    want = kv.plan(np.asarray(past), np.asarray(new), bs, np.asarray(free, np.int32), used, tables, T)
    for name, g, w in zip(("tables", "lens", "offsets", "slots", "positions", "used"), got, want):
        assert np.array_equal(g, w), name


# one request; a ragged batch; more requests than threads, with an odd count
@pytest.mark.parametrize("B,bs,past_hi,new_hi", [(1, 16, 1, 1), (1, 128, 3000, 700), (64, 64, 4096, 1), (37, 32, 300, 40),
                                                 (513, 16, 200, 3), (4099, 64, 300, 9), (8192, 16, 20, 2)])
def test_plan(fp8, B, bs, past_hi, new_hi):
    rng = np.random.default_rng(B + bs)
    past, new = rng.integers(0, past_hi + 1, B), rng.integers(0, new_hi + 1, B)
    new[rng.random(B) < 0.2] = 0
    width = int(-(-(past + new).max() // bs)) + 1
    n_pages = int((-(-(past + new) // bs)).sum()) + 3
    pages = rng.permutation(n_pages).astype(np.int32)
    tables = np.full((B, width), -7, np.int32)
    at = 0
    for b in range(B):
        k = -(-int(past[b]) // bs)
        tables[b, :k] = pages[at:at + k]
        at += k
    free = np.concatenate([[-5, -6], pages[at:]])   # two entries are taken already
    T = int(new.sum())
    _check_plan(fp8, past, new, bs, free, 2, tables, T)
    _check_plan(fp8, past, new, bs, free, 2, tables, T + 5)              # padded rows
    if T > 3:
        _check_plan(fp8, past, new, bs, free, 2, tables, T - 3)          # fewer rows than tokens
    _check_plan(fp8, past, new, bs, free[:len(free) // 2], 2, tables, T)  # the free list runs out
    _check_plan(fp8, past, new, bs, free[:2], 2, tables, T)              # nothing free
    narrow = max(1, width // 2)
    keep = np.minimum(past, narrow * bs)
    _check_plan(fp8, keep, new, bs, free, 2, tables[:, :narrow], T)      # rows too narrow for some


def test_plan_lengths_out_of_range(fp8):
    # negative lengths count as 0; lengths and sums beyond 32 bits are refused without leaving the arrays
    past = np.array([-3, 5, 2 ** 31 - 1, 7, 0], np.int64)
    new = np.array([4, -9, 2 ** 31 - 1, 2, 2 ** 31 - 1], np.int64)
    tables = np.zeros((5, 2), np.int32)
    got = _plan(fp8, past, new, 16, np.arange(1, 4), 0, tables, 64)
    assert got[1].tolist() == [4, 5, 2 ** 31 - 1, 9, 0][:2] + [2 ** 31 - 1, 7 + 2, 0]
    assert got[3][:4].tolist() == [16, 17, 18, 19] and (got[3][4:] == -1).all()
    assert got[5] == 1


def test_plan_on_its_own_stream_unaligned_outputs(fp8):
    rng = np.random.default_rng(9)
    past, new = rng.integers(0, 50, 20), rng.integers(0, 9, 20)
    tables = np.arange(20 * 8, dtype=np.int32).reshape(20, 8)
    T, free = int(new.sum()), np.arange(200, 300, dtype=np.int32)
    slots = torch.full((T + 1,), -9, dtype=torch.int64, device="cuda")[1:]
    pos = torch.full((T + 1,), -9, dtype=torch.int32, device="cuda")[1:]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = _plan(fp8, past, new, 16, free, 0, tables, T, slots=slots, positions=pos)
    s.synchronize()
    want = kv.plan(past, new, 16, free, 0, tables, T)
    assert np.array_equal(got[3], want[3]) and np.array_equal(got[4], want[4])


def _cache(n_pages, H, bs, d, seed, ue8m0=False):
    codes = syn.random_e4m3_codes((n_pages, H, bs, d), seed)
    scale = (syn.random_pow2_scales if ue8m0 else syn.random_scales)((n_pages, H), seed + 1, lo=-9, hi=-5)
    return codes, np.asarray(scale, np.float32).reshape(n_pages, H)


def _check_append(fp8, k, v, slots, kc, ks, vc, vs, ue8m0, strided=True):
    T, H, dk = k.shape
    dv = v.shape[2]
    if strided:   # K and V side by side in one projection's rows
        both = dev_bf16(np.concatenate([k, v], axis=2))
        dk_t, dv_t = both[..., :dk], both[..., dk:]
    else:
        dk_t, dv_t = dev_bf16(k), dev_bf16(v)
    gk, gks, gv, gvs = dev_e4m3(kc), dev_f32(ks), dev_e4m3(vc), dev_f32(vs)
    sl = torch.from_numpy(np.asarray(slots, np.int64)).cuda()
    fmt = fp8.FP8_SCALE_UE8M0 if ue8m0 else fp8.FP8_SCALE_FP32
    for _ in range(2):   # a repeated call changes nothing
        fp8.fp8_kv_append(dk_t, dv_t, sl, gk, gks, gv, gvs, scale_fmt=fmt)
        fp8.fp8_device_status()
        for x, c, s, g, gs in ((k, kc, ks, gk, gks), (v, vc, vs, gv, gvs)):
            wc, ws = kv.append(x, slots, c, s, ue8m0)
            assert np.array_equal(host_f32(gs).view(np.uint32), ws.view(np.uint32)), "scales"
            assert np.array_equal(host_bits(g), wc), "codes"


def _slots(rng, past, new, bs, n_pages):
    pages = rng.permutation(n_pages)
    slots, at = [], 0
    for p, n in zip(past, new):
        first = p // bs
        count = -(-(p + n) // bs) - first
        mine = pages[at:at + count]
        at += count
        slots += [int(mine[(p + i) // bs - first]) * bs + (p + i) % bs for i in range(n)]
    return np.array(slots, np.int64)


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("H,dk,dv", [(1, 64, 64), (8, 128, 128), (3, 192, 128)])
@pytest.mark.parametrize("ue8m0", [False, True])
def test_append_ragged(fp8, bs, H, dk, dv, ue8m0):
    rng = np.random.default_rng(bs + dk + H)
    past = [0, 0, 5, bs - 1, bs, 2 * bs + 3, 1]
    new = [1, 3 * bs + 2, 1, 2, bs, 40, bs - 1]
    n_pages = 40
    slots = _slots(rng, past, new, bs, n_pages)
    T = len(slots)
    k = syn.normal_bf16(rng, (T, H, dk), outlier_frac=0.01, outlier_mult=20)
    v = syn.normal_bf16(rng, (T, H, dv))
    _check_append(fp8, k, v, slots, *_cache(n_pages, H, bs, dk, 1, ue8m0), *_cache(n_pages, H, bs, dv, 3, ue8m0), ue8m0)


# many single tokens (windows of one and of several tokens per warp), many heads
@pytest.mark.parametrize("T,H,dk,dv", [(1, 1, 64, 64), (257, 8, 128, 128), (300, 64, 192, 128)])
def test_append_single_tokens(fp8, T, H, dk, dv):
    rng = np.random.default_rng(T)
    past = rng.integers(0, 16, T).tolist()
    slots = _slots(rng, past, [1] * T, 16, T + 3)
    slots[rng.random(T) < 0.1] = -1   # tokens without a place
    k, v = syn.normal_bf16(rng, (T, H, dk)), syn.normal_bf16(rng, (T, H, dv))
    _check_append(fp8, k, v, slots, *_cache(T + 3, H, 16, dk, 5), *_cache(T + 3, H, 16, dv, 7), False, strided=False)


# long pages of few and of many values a token; more tokens than a window of one serves
@pytest.mark.parametrize("past,new,H,dk,dv,bs", [([3, 0], [140, 129], 2, 1024, 16, 128), ([0, 9, 31], [3000, 1, 64], 2, 64, 48, 64),
                                                 ([5] * 2600, [1] * 2600, 3, 64, 128, 16)])
def test_append_long(fp8, past, new, H, dk, dv, bs):
    rng = np.random.default_rng(len(new))
    n_pages = sum(-(-(p + n) // bs) - p // bs for p, n in zip(past, new)) + 2
    slots = _slots(rng, past, new, bs, n_pages)
    k, v = syn.normal_bf16(rng, (len(slots), H, dk)), syn.normal_bf16(rng, (len(slots), H, dv))
    k[7, 0, 3] = 0x7F80   # an infinity
    _check_append(fp8, k, v, slots, *_cache(n_pages, H, bs, dk, 21), *_cache(n_pages, H, bs, dv, 23), False)


def test_append_zero_blocks_extremes_and_nonfinite(fp8):
    rng = np.random.default_rng(4)
    H, d, bs = 2, 128, 16
    slots = np.concatenate([np.arange(16, 32), np.arange(32, 37), [48 + 3], [64 + 9, 64 + 10], [10 ** 12, -4]])
    T = len(slots)
    f = rng.standard_normal((T, H, d)).astype(np.float32)
    f[:16, 0] = 0                       # a block of zeros: the scale's floor
    f[0, 1, 5] = 3e38                   # the largest finite magnitudes
    f[17, 0, 7], f[18, 1, 9] = np.inf, -np.inf
    f[19, 0, 3] = np.nan
    f[21] = np.inf                      # nothing finite at all
    f[22, 1] = 1e-30                    # subnormal beside the page's scale
    x = syn.to_bf16_bits(f)
    _check_append(fp8, x, x, slots, *_cache(6, H, bs, d, 11), *_cache(6, H, bs, d, 13), False)


def test_append_keeps_to_its_slots_and_stream(fp8):
    rng = np.random.default_rng(6)
    kc, ks = _cache(8, 4, 32, 64, 17)
    x = syn.normal_bf16(rng, (50, 4, 64))
    slots = np.concatenate([np.arange(64, 96), np.arange(160, 178)])
    g, gs = dev_e4m3(kc), dev_f32(ks)
    g2, gs2 = dev_e4m3(kc), dev_f32(ks)
    t, sl = dev_bf16(x), torch.from_numpy(slots).cuda()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    fp8.fp8_kv_append(t, t, sl, g, gs, g2, gs2, stream=s)
    s.synchronize()
    want, ws = kv.append(x, slots, kc, ks)
    assert np.array_equal(host_bits(g), want) and np.array_equal(host_bits(g2), want)
    assert np.array_equal(host_f32(gs), ws)


def test_refusals(fp8):
    past = dev_i32([1, 2])
    one = dev_i32([0])
    tab = dev_i32(np.zeros((2, 2)))
    with pytest.raises(fp8.Fp8Error):
        fp8.fp8_kv_plan(past, past, one, one, tab, 24, 3)              # page size
    with pytest.raises(fp8.Fp8Error):
        fp8.fp8_kv_plan(past, past, one, one, tab, 16, 3, used_out=one)   # in place
    with pytest.raises(ValueError):
        fp8.fp8_kv_plan(past, past[:1], one, one, tab, 16, 3)
    with pytest.raises(TypeError):
        fp8.fp8_kv_plan(past.long(), past, one, one, tab, 16, 3)
    kc, ks, vc, vs = fp8.kv_cache(4, 2, 16, 64, 64)
    x = torch.zeros((3, 2, 72), dtype=torch.bfloat16, device="cuda")
    sl = torch.arange(3, device="cuda")
    with pytest.raises(ValueError):
        fp8.fp8_kv_append(x[..., :64], x[..., :64], sl[:2], kc, ks, vc, vs)
    with pytest.raises(ValueError):
        fp8.fp8_kv_append(x[..., ::2][..., :32], x[..., :64], sl, kc, ks, vc, vs)
    with pytest.raises(fp8.Fp8Error):   # rows of 68 values: not 16-byte aligned
        odd = torch.zeros((3, 2, 68), dtype=torch.bfloat16, device="cuda")
        fp8.fp8_kv_append(odd[..., :64], x[..., :64], sl, kc, ks, vc, vs)
    with pytest.raises(fp8.Fp8Error):
        fp8.fp8_kv_append(x[..., 4:68], x[..., :64], sl, kc, ks, vc, vs)
    with pytest.raises(fp8.Fp8Error):
        fp8.fp8_kv_append(x[..., :64], x[..., :64], sl, kc, ks, vc, vs, scale_fmt=3)
    with pytest.raises(TypeError):
        fp8.fp8_kv_append(x[..., :64].float(), x[..., :64], sl, kc, ks, vc, vs)


def test_append_ue8m0_under_scales_that_are_no_powers_of_two(fp8):
    # Pages written with fp32 scales, appended to in ue8m0: the page's scale stays where it is the larger, and the codes
    # are e4m3(x / s) for it.  Every bf16 mantissa over the exponents that such a page meets; page maxima of any mantissa.
    H, d, bs = 64, 128, 16
    rng = np.random.default_rng(31)
    bits = np.empty((8, H, d), np.uint16)
    bits[:] = ((np.arange(8)[:, None, None] + 116) << 7) | np.arange(128)   # 2^-11 .. 2^-4
    bits |= (rng.random(bits.shape) < 0.5).astype(np.uint16) << 15
    slots = np.concatenate([np.arange(3, 7), np.arange(16 + 9, 16 + 13)])
    kc, vc = (syn.random_e4m3_codes((2, H, bs, d), s) for s in (32, 33))
    tops = oracle.bf16_to_f32((((rng.integers(127, 140, (4, H)) << 7) | rng.integers(0, 128, (4, H))).astype(np.uint16)))
    tops = np.asarray(tops, np.float32).reshape(4, H)
    tops[:, 0] = 1104.0
    scales = tops / np.float32(448)
    x = oracle.bf16_to_f32(bits).astype(np.float32).reshape(bits.shape)
    f32 = x[:4] / scales[0][:, None]
    by_reciprocal = x[:4] * (np.float32(1) / scales[0])[:, None]
    assert (oracle.e4m3_encode(f32) != oracle.e4m3_encode(by_reciprocal)).any()   # the two ways differ here
    _check_append(fp8, bits, bits, slots, kc, scales[:2], vc, scales[2:], True)
    mixed = scales.copy()
    mixed[:, ::2] = 2.0   # powers of two beside them, in the same warp
    _check_append(fp8, bits, bits, slots, kc, mixed[:2], vc, mixed[2:], True)


def test_plan_of_no_requests(fp8):
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    lens, offsets, slots, positions, used = fp8.fp8_kv_plan(
        none, none, dev_i32([4, 5]), dev_i32([1]), none.view(0, 3), 16, 0,
        offsets=dev_i32([-7]), used_out=dev_i32([-7]), stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert offsets.tolist() == [0] and used.tolist() == [1] and not (lens.numel() or slots.numel() or positions.numel())
    with pytest.raises(fp8.Fp8Error):
        fp8.fp8_kv_plan(none, none, none, dev_i32([0]), none.view(0, 3), 16, 2)   # rows of nobody


@pytest.mark.parametrize("ue8m0", [False, True])
def test_append_token_by_token_under_growing_scales(fp8, ue8m0):
    H, d, bs, n = 3, 64, 64, 50
    rng = np.random.default_rng(41)
    x = syn.to_bf16_bits((rng.standard_normal((n, H, d)) * (1.03 ** np.arange(n))[:, None, None]).astype(np.float32))
    kc, ks, vc, vs = fp8.kv_cache(2, H, bs, d, d)
    kc.view(torch.uint8).zero_()
    vc.view(torch.uint8).zero_()
    c, s = np.zeros((2, H, bs, d), np.uint8), np.zeros((2, H), np.float32)
    t = dev_bf16(x)
    for i in range(n):
        fp8.fp8_kv_append(t[i:i + 1], t[i:i + 1], torch.tensor([bs + i], device="cuda"), kc, ks, vc, vs,
                          scale_fmt=fp8.FP8_SCALE_UE8M0 if ue8m0 else fp8.FP8_SCALE_FP32)
        c, s = kv.append(x[i:i + 1], np.array([bs + i]), c, s, ue8m0)
        assert np.array_equal(host_bits(kc), c) and np.array_equal(host_bits(vc), c), i
        assert np.array_equal(host_f32(ks), s)
    fp8.fp8_device_status()
