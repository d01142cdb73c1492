"""One decode step of a mixture-of-experts block whose weights are all packed INT4, for the
next tokens of several requests: the shared projection (ConvRot W4A8) and each request's
low-rank adapter beside it, the router's logits (AWQ W4A16), then the experts.

    python examples/decode_block.py [--tokens 16] [--width 3840] [--inner 1280] [--experts 128]
                                    [--top 8] [--adapters 6] [--rank 16]

Weights and inputs are random.  The step is captured into a HIP graph: every buffer is
allocated once, and each launch goes to the capturing stream.  Prints the time of a step,
replayed and launched call by call.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import packed_int4_convrot_amd as ck  # noqa: E402


def packed_weight(rows, columns, zeros, g, device, experts=()):
    """Random packed codes [..., rows, columns / 2], scales and zero points [..., columns / 64, rows]."""
    p = torch.randint(0, 256, (*experts, rows, columns // 2), dtype=torch.uint8, device=device, generator=g)
    shape = (*experts, columns // 64, rows)
    s = torch.empty(shape, device=device).uniform_(0.5, 1.5, generator=g).mul_(0.25 / columns ** 0.5).bfloat16()
    z = torch.empty(shape, device=device).normal_(0, 0.01, generator=g).bfloat16() if zeros else None
    return p, s, z


class DecodeBlock:
    """Weights of the block, and the buffers of a step of T tokens."""

    def __init__(self, tokens, width, inner, experts, top, adapters, rank, device="cuda:0", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.top = top
        self.projection = packed_weight(width, width, False, g, device)
        self.router = packed_weight(experts, width, True, g, device)
        self.experts = ck.MoeExperts(*packed_weight(2 * inner, width, True, g, device, (experts,)),
                                     *packed_weight(width, inner, True, g, device, (experts,)))
        a = torch.randn((adapters, rank, width), device=device, generator=g).mul_(width ** -0.5).bfloat16()
        b = torch.randn((adapters, width, rank), device=device, generator=g).mul_(rank ** -0.5).bfloat16()
        ranks = torch.randint(1, rank + 1, (adapters,), dtype=torch.int32, device=device, generator=g)
        scaling = torch.full((adapters,), 0.5, device=device)
        self.adapters = ck.LoraAdapters(a, b, scaling, ranks)

        # A step's input, each token's adapter (-1: none) and its results.
        self.x = torch.randn((tokens, width), device=device, generator=g).bfloat16()
        self.index = torch.randint(-1, adapters, (tokens,), dtype=torch.int32, device=device, generator=g)
        self.y = torch.empty_like(self.x)
        self.logits = torch.empty((tokens, experts), dtype=torch.bfloat16, device=device)
        self.ids = torch.empty((tokens, top), dtype=torch.int32, device=device)
        self.weights = torch.empty((tokens, top), dtype=torch.float32, device=device)
        self.out = torch.empty_like(self.x)
        # One workspace serves the calls of a stream one after the other.
        need = max(ck.workspace_bytes(tokens, width, width), ck.lora_workspace_bytes(tokens, width, rank, adapters),
                   ck.moe_workspace_bytes(tokens, inner, experts, top))
        self.space = torch.empty((max(need, 1),), dtype=torch.uint8, device=device)

    def step(self):
        packed, scales, _ = self.projection
        ck.linear(self.x, 64, 8, packed, scales, True, out=self.y, workspace=self.space)
        # In place: rows without an adapter keep the projection's result.
        ck.lora_add(self.x, self.adapters, self.index, base=self.y, out=self.y, workspace=self.space)
        product = ck.w4a16_gemv if self.x.shape[0] <= 8 else ck.w4a16_gemm
        product(self.y, *self.router, out=self.logits)
        ck.moe(self.y, self.logits, self.experts, self.top, out=self.out, ids=self.ids, weights=self.weights,
               workspace=self.space)
        return self.out

    def capture(self):
        """The step as a graph (x and index may be filled anew between replays)."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph


def time_us(step, n):
    for _ in range(10):
        step()
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(n):
        step()
    torch.cuda.synchronize()
    return (time.perf_counter() - start) / n * 1e6


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("tokens", 16), ("width", 3840), ("inner", 1280), ("experts", 128), ("top", 8),
                        ("adapters", 6), ("rank", 16), ("steps", 200)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    block = DecodeBlock(a.tokens, a.width, a.inner, a.experts, a.top, a.adapters, a.rank)
    graph = block.capture()
    eager = block.step().clone()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(eager, block.out), "a replayed step differs from the calls one by one"
    print("%d tokens, width %d, %d of %d experts of inner width %d, %d adapters of rank <= %d: "
          "%.1f us a step replayed, %.1f us call by call"
          % (a.tokens, a.width, a.top, a.experts, a.inner, a.adapters, a.rank, time_us(graph.replay, a.steps),
             time_us(block.step, a.steps)))


if __name__ == "__main__":
    main()
