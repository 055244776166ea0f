"""The attention entry points under HIP graph capture (GPU).

A decoding step (append of one token per sequence, attention over the cache) and a training step are captured once and
replayed; before each replay the inputs, and for decoding the lengths, change in place.  Every replay equals the same
calls made eagerly on outputs and a cache of their own, bit for bit.
"""
from __future__ import annotations

import pytest
import torch

from gpu_util import say
from input_dependent_short_amd import binding

pytestmark = pytest.mark.gpu


def _capture(calls):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    return graph


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decoding_step_replayed(dtype):
    S, Hq, Hkv, hd, page, width, base = 5, 8, 2, 64, 16, 24, 500.0
    say(f"[graph] append and decode, {dtype}")
    gen = torch.Generator(device="cuda").manual_seed(3)
    pages = torch.randperm(S * width, generator=gen, device="cuda").to(torch.int32).view(S, width)
    pool = torch.randn(2, S * width, Hkv, page, hd, generator=gen, device="cuda").to(dtype)
    rope = torch.empty(page * width, hd // 2, 2, device="cuda")
    binding.dsc_rope_table(rope, base=base)
    row = torch.randn(S, (Hq + 2 * Hkv) * hd, generator=gen, device="cuda").to(dtype)
    q, k, v = (row[:, a * hd:b * hd].unflatten(1, (b - a, hd)) for a, b in
               ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    past = torch.tensor([0, 15, 16, 200, 370], dtype=torch.int32, device="cuda")
    lens = past + 1
    n = binding.dsc_attn_decode_workspace_size(dtype, S, Hq, Hkv, hd, page, width)

    def state():
        kc, vc = pool.clone().unbind(0)
        return kc, vc, torch.empty(S, Hq, hd, dtype=dtype, device="cuda"), \
            torch.empty(S, Hq, hd, dtype=dtype, device="cuda"), \
            torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")

    def calls(kc, vc, turned, o, ws):
        binding.dsc_kv_append(k, v, kc, vc, pages, past, q=q, q_out=turned, table=rope)
        binding.dsc_attn_decode(turned, kc, vc, pages, lens, o, ws)

    held, eager = state(), state()
    graph = _capture(lambda: calls(*held))
    calls(*eager)  # the warm-up's writes
    for rep in range(4):
        if rep:
            row.copy_(torch.randn(row.shape, generator=gen, device="cuda"))
            past.add_(1)
            lens.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        calls(*eager)
        torch.cuda.synchronize()
        for name, a, b in zip(("k_cache", "v_cache", "q_out", "o"), held, eager):
            assert torch.equal(a, b), f"replay {rep}: {name} differs from the eager call"


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (64, 32)])  # few rows, and the kernels for long inputs
def test_training_step_replayed(Hq, Hkv):
    B, T, hd = 2, 333, 128
    say(f"[graph] attention and its gradients, {Hq} heads over {Hkv}")
    gen = torch.Generator(device="cuda").manual_seed(5)
    new = lambda h: torch.randn(B, T, h, hd, generator=gen, device="cuda").bfloat16()
    q, k, v, g = new(Hq), new(Hkv), new(Hkv), new(Hq)
    cu = torch.tensor([0, 1, 130, 130, 500, B * T], dtype=torch.int32, device="cuda")
    n = binding.dsc_attn_bwd_workspace_size(q.dtype, B, T, Hq, Hkv, hd)

    def state():
        return [torch.empty_like(q), torch.empty(Hq, B * T, device="cuda"), torch.empty_like(q), torch.empty_like(k),
                torch.empty_like(v), torch.empty(n, dtype=torch.uint8, device="cuda")]

    def calls(o, lse, dq, dk, dv, ws):
        binding.dsc_attn_fwd(q, k, v, o, lse, cu_seqlens=cu)
        binding.dsc_attn_bwd(q, k, v, o, lse, g, dq, dk, dv, ws, cu_seqlens=cu)

    held, eager = state(), state()
    graph = _capture(lambda: calls(*held))
    for rep in range(4):
        if rep:
            for t in (q, k, v, g):
                t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        calls(*eager)
        torch.cuda.synchronize()
        for name, a, b in zip(("o", "lse", "dq", "dk", "dv"), held, eager):
            assert torch.equal(a, b), f"replay {rep}: {name} differs from the eager call"
