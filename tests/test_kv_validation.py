"""The paged cache's entry points refuse bad arguments on the host, before
anything is launched (no GPU needed)."""
import ctypes

import pytest

INVALID, UNSUPPORTED, OK = 1, 2, 0
P = 1 << 20   # an aligned address that is never followed


@pytest.fixture(scope="module")
def L():
    import fp8_block_scaled_07_gb300 as m
    return m.lib


def _call(f, order, base, **changes):
    assert set(changes) <= set(order)
    return f(*[{**base, **changes}[k] for k in order])


PLAN = dict(past=P, fresh=P, B=4, block=64, free=P, n_free=9, used=P, tables=P, width=3, lens=P, offsets=P, T=5, slots=P,
            positions=P, used_out=P + 64, stream=None)


@pytest.mark.parametrize("want,change", [
    (INVALID, dict(B=-1)), (INVALID, dict(T=-1)), (INVALID, dict(n_free=-1)), (INVALID, dict(width=0)),
    (INVALID, dict(block=24)), (INVALID, dict(block=256)), (INVALID, dict(width=1 << 30, block=16)),
    (UNSUPPORTED, dict(B=8193)), (UNSUPPORTED, dict(T=1 << 31)), (INVALID, dict(B=0)), (OK, dict(B=0, T=0)),
    (INVALID, dict(past=None)), (INVALID, dict(fresh=None)), (INVALID, dict(used=None)), (INVALID, dict(tables=None)),
    (INVALID, dict(lens=None)), (INVALID, dict(offsets=None)), (INVALID, dict(used_out=None)), (INVALID, dict(used_out=P)),
    (INVALID, dict(free=None)), (INVALID, dict(slots=None))])
def test_plan(L, want, change):
    assert _call(L.fp8_kv_plan, list(PLAN), PLAN, **change) == want


# arrays of their own for B = 4000, T = 9000, two pages free: 1 MB apart
APART = {k: (i + 1) << 20 for i, k in enumerate(("past", "fresh", "free", "used", "tables", "lens", "offsets", "slots",
                                                 "positions", "used_out"))}


@pytest.mark.parametrize("result,other,shift", [
    ("lens", "past", 0), ("lens", "fresh", 0), ("lens", "past", 4 * 3999), ("lens", "past", -4 * 3999), ("offsets", "past", 0),
    ("offsets", "fresh", -16000), ("offsets", "lens", 0), ("tables", "past", 0), ("tables", "free", -48000 + 4),
    ("slots", "fresh", 0), ("slots", "free", 4), ("positions", "past", 0), ("positions", "slots", 71996),
    ("used_out", "used", 0), ("used_out", "past", 400), ("used_out", "lens", 0), ("lens", "used", -400)])
def test_plan_refuses_results_over_other_arrays(L, result, other, shift):
    base = {**PLAN, **APART, "B": 4000, "T": 9000, "n_free": 2}
    assert _call(L.fp8_kv_plan, list(PLAN), base, **{result: base[other] + shift}) == INVALID


APPEND = dict(k=P, kts=1024, khs=128, v=P, vts=1024, vhs=128, slots=P, T=4, H=8, dk=128, dv=128, kc=P, ks=P, vc=P, vs=P,
              n_pages=7, block=64, fmt=0, stream=None)


@pytest.mark.parametrize("want,change", [
    (INVALID, dict(T=-1)), (INVALID, dict(H=0)), (INVALID, dict(dk=8)), (INVALID, dict(dv=1040)), (INVALID, dict(n_pages=-1)),
    (INVALID, dict(block=8)), (INVALID, dict(fmt=2)), (UNSUPPORTED, dict(T=1 << 31)), (UNSUPPORTED, dict(H=1 << 16)),
    (UNSUPPORTED, dict(n_pages=1 << 31)), (OK, dict(T=0, k=None)), (INVALID, dict(k=None)), (INVALID, dict(v=None)),
    (INVALID, dict(slots=None)), (INVALID, dict(kc=None)), (INVALID, dict(ks=None)), (INVALID, dict(vc=None)),
    (INVALID, dict(vs=None)), (INVALID, dict(k=P + 8)), (INVALID, dict(v=P + 2)), (INVALID, dict(kc=P + 8)),
    (INVALID, dict(vc=P + 8)), (INVALID, dict(kts=1028)), (INVALID, dict(khs=-8)), (INVALID, dict(vts=-1024)),
    (INVALID, dict(vhs=4))])
def test_append(L, want, change):
    assert _call(L.fp8_kv_append, list(APPEND), APPEND, **change) == want


ATTEND = dict(q=P, qts=1024, qhs=128, kc=P, ks=P, vc=P, vs=P, n_pages=7, block=64, tables=P, width=3, lens=P, offsets=P, B=2,
              T=4, Hq=8, Hkv=4, dk=128, dv=128, scale=0.1, out=P, lse=None, ws=P, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("want,change", [
    (INVALID, dict(T=-1)), (INVALID, dict(B=-1)), (INVALID, dict(Hq=0)), (INVALID, dict(Hkv=0)), (INVALID, dict(Hkv=3)),
    (INVALID, dict(n_pages=-1)), (INVALID, dict(block=24)), (INVALID, dict(width=0)), (INVALID, dict(offsets=None)),
    (INVALID, dict(scale=-1.0)), (INVALID, dict(scale=float("nan"))), (INVALID, dict(scale=float("inf"))),
    (UNSUPPORTED, dict(dk=96)), (UNSUPPORTED, dict(dk=64)), (UNSUPPORTED, dict(dk=192, dv=64)),
    (INVALID, dict(q=None)), (INVALID, dict(kc=None)), (INVALID, dict(ks=None)), (INVALID, dict(vc=None)),
    (INVALID, dict(vs=None)), (INVALID, dict(tables=None)), (INVALID, dict(lens=None)), (INVALID, dict(out=None)),
    (INVALID, dict(q=P + 8)), (INVALID, dict(out=P + 16)), (INVALID, dict(kc=P + 8)), (INVALID, dict(vc=P + 8)),
    (INVALID, dict(qts=1028)), (INVALID, dict(qhs=-8)), (OK, dict(T=0, q=None, out=None))])
def test_attention(L, want, change):
    assert _call(L.fp8_kv_attention, list(ATTEND), ATTEND, **change) == want


def test_attention_workspace(L):
    size = L.fp8_kv_attention_workspace_size(4, 2, 8, 4, 128, 128)
    assert size >= 1 << 14
    assert _call(L.fp8_kv_attention, list(ATTEND), ATTEND, ws_bytes=size - 1) == 5
    assert _call(L.fp8_kv_attention, list(ATTEND), ATTEND, ws=None, ws_bytes=0) == 5
    assert isinstance(ctypes.c_size_t(size).value, int)


@pytest.mark.parametrize("block,width", [(16, (1 << 27) - 1), (32, (1 << 26) - 1), (64, (1 << 25) - 1), (128, 1 << 24)])
def test_attention_counts_whole_tiles_in_31_bits(L, block, width):
    # the last tile of 128 tokens would end past 2^31 - 1
    assert _call(L.fp8_kv_attention, list(ATTEND), ATTEND, block=block, width=width) == INVALID


def test_attention_workspace_sizes_are_kept_by_what_they_depend_on():
    import fp8_block_scaled_07_gb300 as m
    seen = len(m._ws_sizes)
    m._kv_ws_size(5, 0, 8, 4, 128, 128, -1)   # (refused by the call itself)
    for T in range(1, 300):
        for B in (1, 7, T):
            assert m._kv_ws_size(T, B, 8, 4, 128, 128, -1) == m.lib.fp8_kv_attention_workspace_size(T, B, 8, 4, 128, 128)
    assert len(m._ws_sizes) - seen <= 2
    assert m._kv_ws_size(0, 3, 8, 4, 128, 128, -1) == 0
