"""The attention layer on the paged cache: prompts, then single tokens, with
requests that run out of pages; each step's cache and results against the
oracle on the projections that the layer made."""
import numpy as np
import pytest
import torch

import oracle
from oracle import kv
from tests.helpers import host_bits, host_f32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from fp8_block_scaled_07_gb300 import paged_attention as m
    return m


def _np(t):
    return t.cpu().numpy()


@pytest.mark.parametrize("Hq,Hkv,dk,dv,block", [(4, 2, 64, 64, 16), (8, 2, 128, 128, 64), (2, 2, 192, 128, 32)])
def test_steps(pa, Hq, Hkv, dk, dv, block):
    import fp8_block_scaled_07_gb300 as fp8
    D, B, max_len = 256, 3, 150
    n_pages = 3 * -(-100 // block)   # request 1 runs out of them at its second step
    layer = pa.random_layer(D, Hq, Hkv, dk, dv, n_pages, block, seed=dk)
    req = pa.Requests(B, n_pages, block, max_len)
    gen = torch.Generator(device="cuda").manual_seed(1)
    want = dict(tables=_np(req.tables), lens=np.zeros(B, np.int32), used=0)
    cache = [host_bits(t) if t.dtype == torch.float8_e4m3fn else host_f32(t) for t in layer.cache]
    for new in ([70, 0, 33], [1, 300, 2], [1, 1, 1], [1, 1, 1]):
        T, single = sum(new), new == [1, 1, 1]
        x = torch.randn((T, D), device="cuda", generator=gen).bfloat16()
        plan = req.step(torch.tensor(new, dtype=torch.int32, device="cuda"), T)
        q, k, v = layer.project(x)
        out = layer.attend(x, req, plan, single)
        fp8.fp8_device_status()
        tables, lens, offsets, slots, positions, used = kv.plan(
            want["lens"], np.array(new), block, _np(req.free_pages), want["used"], want["tables"], T)
        want = dict(tables=tables, lens=lens, used=used)
        for name, got, w in (("tables", req.tables, tables), ("lens", req.lens, lens), ("offsets", plan[0], offsets),
                             ("slots", plan[1], slots), ("positions", plan[2], positions), ("used", req.used, [used])):
            assert np.array_equal(_np(got), w), name
        for i, y in ((0, k), (2, v)):
            cache[i], cache[i + 1] = kv.append(host_bits(y.contiguous()), slots, cache[i], cache[i + 1])
            assert np.array_equal(host_bits(layer.cache[i]), cache[i])
            assert np.array_equal(host_f32(layer.cache[i + 1]), cache[i + 1])
        ref, _, tol, _ = kv.attention(host_bits(q.contiguous()), *cache, tables, lens, offsets, dk ** -0.5)
        got = oracle.bf16_to_f32(host_bits(out)).astype(np.float64).reshape(ref.shape)
        assert (np.abs(got - ref) <= tol).all()
        y = layer(x, req, plan, single)   # the append again: nothing changes
        assert torch.equal(y, fp8.fp8_linear(out.flatten(1), layer.wo, layer.wo_s)[0])
    assert list(want["lens"]) == [73, 2, 37]


def test_command(pa, capsys):
    pa.main(["--layers", "2", "--requests", "3", "--prompt", "40", "--tokens", "3", "--heads", "4", "1", "--width", "256"])
    assert "3 requests, 2 layers" in capsys.readouterr().out


def test_one_token_or_one_head_of_odd_rows(pa):
    # a dimension of one has no stride to be aligned
    import fp8_block_scaled_07_gb300 as fp8
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((3, 1, 64 * 6 + 4), device="cuda", generator=gen).bfloat16()
    sl = torch.tensor([16], device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    one = torch.ones(1, **i32)

    def views(y, H):
        return [y.as_strided((1, n, 64), (388, 64, 1), a) for a, n in ((0, 2 * H), (128, H), (256, H))]
    for H in (1, 2):
        q, k, v = views(x, H)   # one token: the rows are 388 values apart
        assert q.stride(0) % 8
        res = []
        for args in ((q, k, v), (q.contiguous(), k.contiguous(), v.contiguous())):
            cache = fp8.kv_cache(2, H, 16, 64, 64)
            fp8.fp8_kv_append(args[1], args[2], sl, *cache)
            out, _ = fp8.fp8_kv_attention(args[0], *cache, one.view(1, 1), one)
            res.append((cache[0].view(torch.uint8)[1, :, 0], cache[3][1], out))
        assert all(torch.equal(a, b) for a, b in zip(*res))
    heads = torch.randn((2, 3, 68), device="cuda", generator=gen).bfloat16()[:, :1, :64]   # one head: 68 values to the next
    rows = torch.empty((2, 408), dtype=torch.bfloat16, device="cuda")
    odd = rows[:, :64].unflatten(1, (1, 64)).copy_(heads).as_strided((2, 1, 64), (408, 68, 1))
    assert odd.stride(1) % 8
    cache, want = fp8.kv_cache(1, 1, 16, 64, 64), fp8.kv_cache(1, 1, 16, 64, 64)
    slots = torch.arange(2, device="cuda")
    fp8.fp8_kv_append(odd, odd, slots, *cache)
    fp8.fp8_kv_append(heads.contiguous(), heads.contiguous(), slots, *want)
    assert torch.equal(cache[0].view(torch.uint8)[:, :, :2], want[0].view(torch.uint8)[:, :, :2])
    fp8.fp8_device_status()


def test_workspace_is_filled_on_the_calls_stream(pa):
    # A call on a stream of its own, while the current stream has long work: the workspace it gets first is zero when
    # the call uses it, though the memory held something else and a fill on the current stream would come too late.
    import fp8_block_scaled_07_gb300 as fp8
    n, d, H = 700, 128, 40
    gen = torch.Generator(device="cuda").manual_seed(3)
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = fp8.kv_cache(n // 64 + 1, H, 64, d, d)
    for codes, scale in (cache[:2], cache[2:]):
        codes.copy_(torch.randn(codes.shape, device="cuda", generator=gen).to(codes.dtype))
        scale.fill_(1.0)
    q = torch.randn((n, H, d), device="cuda", generator=gen).bfloat16()
    tables = torch.arange(n // 64 + 1, **i32).view(1, -1)
    args = (q, *cache, tables, torch.tensor([n], **i32))
    offsets, want = torch.tensor([0, n], **i32), torch.empty_like(q)
    fp8.fp8_kv_attention(*args, offsets=offsets, out=want)
    for _ in range(3):
        s = torch.cuda.Stream()
        out = torch.zeros_like(q)
        size = fp8.lib.fp8_kv_attention_workspace_size(n, 1, H, H, d, d)
        for pool in (torch.cuda.current_stream(), s):
            with torch.cuda.stream(pool):
                dirt = [torch.full((max(size, 1 << 16),), 1, dtype=torch.uint8, device="cuda") for _ in range(3)]
                del dirt
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        fp8.fp8_kv_attention(*args, offsets=offsets, out=out, stream=s)
        s.synchronize()
        assert torch.equal(out, want)
        torch.cuda.synchronize()
    fp8.fp8_device_status()
