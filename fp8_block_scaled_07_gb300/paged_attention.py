"""An attention layer on the FP8 linear and the paged 8-bit cache, as a
serving loop uses them: one plan a step for all layers, and per layer

    qkv = fp8_linear(x, wqkv);  fp8_kv_append(k, v);  fp8_kv_attention(q);  fp8_linear(., wo)

Requests and their pages live on the device: a step's host work is a handful
of launches, whatever the lengths, and nothing is read back.

    python -m fp8_block_scaled_07_gb300.paged_attention [--layers 4] [--requests 64] [--prompt 512] [--tokens 128]

runs prompts and then single tokens of random-weight layers, and prints the
time of each part.
"""
import argparse

import torch

from . import (fp8_device_status, fp8_kv_append, fp8_kv_attention, fp8_kv_plan, fp8_linear, fp8_weight_quant, kv_cache)


class Requests:
    """The requests' lengths, block tables and free pages, on the device.
    Pages are handed out and not taken back: a finished request keeps its own."""

    def __init__(self, n_requests, n_pages, block_size, max_len, device="cuda"):
        def i32(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=device)
        self.block_size = block_size
        self.tables = i32(n_requests, -(-max_len // block_size))
        self.free_pages = torch.arange(n_pages, dtype=torch.int32, device=device)
        self.lens, self.used = i32(n_requests), i32(1)
        self._lens2, self._used2 = i32(n_requests), i32(1)   # a step writes into the other pair

    def step(self, new, T):
        """Pages and slots for new [B] int32 tokens of each request, T rows in
        all.  Returns the step's (offsets, slots, positions).  A request that
        its table's width or the free pages do not cover keeps its length, and
        its rows have slot -1; the first that the free pages do not cover ends
        their handing out for the step."""
        _, offsets, slots, positions, _ = fp8_kv_plan(
            self.lens, new, self.free_pages, self.used, self.tables, self.block_size, T, lens=self._lens2,
            used_out=self._used2)
        self.lens, self._lens2 = self._lens2, self.lens
        self.used, self._used2 = self._used2, self.used
        return offsets, slots, positions


class PagedAttention:
    """One layer.  wqkv [(Hq + Hkv) dk + Hkv dv, D] and wo [D, Hq dv]: e4m3 with
    128 x 128 block scales (fp8_weight_quant), Q's heads first, then K's, then V's.
    Without a rotary embedding: its place is between project and the append, by
    the plan's positions."""

    def __init__(self, wqkv, wqkv_s, wo, wo_s, Hq, Hkv, dk, dv, n_pages, block_size):
        if wqkv.shape[0] != (Hq + Hkv) * dk + Hkv * dv or wo.shape[1] != Hq * dv:
            raise ValueError("shape mismatch")
        self.wqkv, self.wqkv_s, self.wo, self.wo_s = wqkv, wqkv_s, wo, wo_s
        self.Hq, self.Hkv, self.dk, self.dv = Hq, Hkv, dk, dv
        self.cache = kv_cache(n_pages, Hkv, block_size, dk, dv, wqkv.device)

    def project(self, x):
        """x [T, D] bf16 -> views q [T, Hq, dk], k [T, Hkv, dk], v [T, Hkv, dv] of one product."""
        qkv, _ = fp8_linear(x, self.wqkv, self.wqkv_s)
        q, k, v = qkv.split([self.Hq * self.dk, self.Hkv * self.dk, self.Hkv * self.dv], dim=1)
        return q.unflatten(1, (self.Hq, self.dk)), k.unflatten(1, (self.Hkv, self.dk)), v.unflatten(1, (self.Hkv, self.dv))

    def attend(self, x, requests, plan, single=False):
        """The heads' results [T, Hq, dv].  single: every request has one row,
        in order (the form of a decoding step, which has no offsets to follow)."""
        offsets, slots, _ = plan
        q, k, v = self.project(x)
        fp8_kv_append(k, v, slots, *self.cache)
        out, _ = fp8_kv_attention(q, *self.cache, requests.tables, requests.lens, offsets=None if single else offsets)
        return out

    def __call__(self, x, requests, plan, single=False):
        y, _ = fp8_linear(self.attend(x, requests, plan, single).flatten(1), self.wo, self.wo_s)
        return y


def random_layer(D, Hq, Hkv, dk, dv, n_pages, block_size, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def weight(n, k):
        return fp8_weight_quant(torch.randn((n, k), device="cuda", generator=gen).mul_(k ** -0.5).bfloat16())
    return PagedAttention(*weight((Hq + Hkv) * dk + Hkv * dv, D), *weight(D, Hq * dv), Hq, Hkv, dk, dv, n_pages, block_size)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--requests", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=512)
    ap.add_argument("--tokens", type=int, default=128)
    ap.add_argument("--heads", type=int, nargs=2, default=(32, 8), metavar=("HQ", "HKV"))
    ap.add_argument("--width", type=int, default=4096)
    a = ap.parse_args(argv)
    block, d, (Hq, Hkv) = 64, 128, a.heads
    n_pages = a.requests * -(-(a.prompt + a.tokens) // block)
    layers = [random_layer(a.width, Hq, Hkv, d, d, n_pages, block, i) for i in range(a.layers)]
    requests = Requests(a.requests, n_pages, block, a.prompt + a.tokens)
    gen = torch.Generator(device="cuda").manual_seed(99)
    marks = [torch.cuda.Event(enable_timing=True) for _ in range(3)]

    def step(n, single):
        x = torch.randn((a.requests * n, a.width), device="cuda", generator=gen).bfloat16()
        plan = requests.step(torch.full((a.requests,), n, dtype=torch.int32, device="cuda"), a.requests * n)
        for layer in layers:
            x = x + layer(x, requests, plan, single)
        return x
    marks[0].record()
    if a.prompt:
        step(a.prompt, False)
    marks[1].record()
    for _ in range(a.tokens):
        x = step(1, True)
    marks[2].record()
    fp8_device_status()
    assert torch.isfinite(x).all()
    print(f"{a.requests} requests, {a.layers} layers: prompts of {a.prompt} in {marks[0].elapsed_time(marks[1]):.2f} ms, "
          f"then {a.tokens} tokens at {marks[1].elapsed_time(marks[2]) / max(1, a.tokens):.3f} ms a step")


if __name__ == "__main__":
    main()
