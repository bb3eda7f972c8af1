"""Attention over the paged 8-bit cache where a tile, a scale or a token is
unusual."""
import numpy as np
import pytest
import torch

import oracle
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
