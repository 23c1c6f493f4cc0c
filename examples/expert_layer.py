"""One tensor-parallel block's projections with the routed operators, on one GPU.

    python examples/expert_layer.py [--tokens 64] [--graph]

The attention output of T tokens sits in R K-shards, as R ranks would hold it.
The output projection sums them, with a low-rank adapter per request beside it
(gemm_ar_lora). Its rows are then routed to experts: gemm_group_route groups the
(token, expert) entries, gemm_grouped_gated gathers the rows and applies the
gate and up projections, gemm_grouped the down projections, and
gemm_group_combine brings the experts' rows back to their tokens, weighted, on
top of the residual. Nothing waits for the host: the routing stays on the device,
so the whole block can be recorded in a CUDA graph, whatever the router picks.

Weights and activations are random; the result is compared with the same block
written in plain PyTorch in 64 bits.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from tensor_gemm_reduction_gb300 import binding as B  # noqa: E402
from tensor_gemm_reduction_gb300 import build as gbuild  # noqa: E402


class Block:
    """Weights, buffers and prepared calls of one block for up to T tokens."""

    def __init__(self, T, hidden=1024, inner=512, shards=4, experts=16, topk=4, adapters=8, rank=16, seed=0,
                 device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)
        bf = dict(dtype=torch.bfloat16, device=device)
        i32 = dict(dtype=torch.int32, device=device)

        def normal(*shape, fan_in):
            return torch.empty(*shape, **bf).normal_(0.0, fan_in ** -0.5, generator=g)

        k = hidden // shards
        self.topk, self.experts = topk, experts
        self.W_r = [normal(hidden, k, fan_in=hidden) for _ in range(shards)]
        self.A_r = [normal(adapters, rank, k, fan_in=hidden) for _ in range(shards)]
        self.Bm = normal(adapters, hidden, rank, fan_in=rank)
        self.scale = torch.full((adapters,), 0.5, device=device)
        self.router = normal(hidden, experts, fan_in=hidden)
        self.W_up = normal(experts, 2 * inner, hidden, fan_in=hidden)
        self.W_down = normal(experts, hidden, inner, fan_in=inner)
        # A step's inputs and buffers, reused step after step.
        self.X_r = [torch.zeros(T, k, **bf) for _ in range(shards)]
        self.adapter = torch.full((T,), -1, **i32)
        self.h = torch.empty(T, hidden, **bf)
        self.ids = torch.empty(T, topk, **i32)
        self.weights = torch.empty(T, topk, dtype=torch.float32, device=device)
        self.offsets = torch.empty(experts + 1, **i32)
        self.source = torch.empty(T * topk, **i32)
        self.position = torch.empty(T, topk, **i32)
        self.up = torch.empty(T * topk, inner, **bf)
        self.down = torch.empty(T * topk, hidden, **bf)
        self.y = torch.empty(T, hidden, **bf)
        self.plan = B.gemm_shard_plan_create(torch.device(device).index or 0, T * topk, max(hidden, inner),
                                             max(hidden, inner), shards)
        self.ws = B.gemm_routed_workspace_alloc(self.plan)
        B.gemm_routed_workspace_init(self.plan, self.ws)
        p, ws = self.plan, self.ws
        self.project = B.prepare_ar_lora(p, self.X_r, self.W_r, self.A_r, self.Bm, self.adapter, self.h, ws,
                                         scale=self.scale)
        self.experts_calls = [
            B.prepare_group_route(p, self.ids, experts, self.offsets, self.source, self.position),
            B.prepare_grouped_gated(p, self.h, self.W_up, self.offsets, self.up, ws, rows=self.source),
            B.prepare_grouped(p, self.up, self.W_down, self.offsets, self.down, ws),
            B.prepare_group_combine(p, self.down, self.position, self.weights, self.y, base=self.h)]

    def step(self):
        self.project()
        probs = (self.h @ self.router).float().softmax(1)
        top = probs.topk(self.topk, dim=1)
        self.ids.copy_(top.indices)
        self.weights.copy_(top.values / top.values.sum(1, keepdim=True))
        for call in self.experts_calls:
            call()
        return self.y

    def check(self):
        B.gemm_shard_check_status(self.plan, self.ws)

    def plain(self):
        """The same step in 64 bits, with the ids and weights that the step chose (a
        router's choice may turn on the rounding of h)."""
        x = torch.cat(self.X_r, 1).double()
        h = x @ torch.cat(self.W_r, 1).double().t()
        a = torch.cat(self.A_r, 2).double()
        for i in range(a.shape[0]):
            t = (self.adapter == i).nonzero()[:, 0]
            h[t] += float(self.scale[i]) * (x[t] @ a[i].t()) @ self.Bm[i].double().t()
        y = h.clone()
        for e in range(self.experts):
            t, j = (self.ids == e).nonzero(as_tuple=True)
            if t.numel():
                gate, up = (h[t] @ self.W_up[e].double().t()).chunk(2, dim=1)
                z = (gate * torch.sigmoid(gate) * up) @ self.W_down[e].double().t()
                y.index_add_(0, t, z * self.weights[t, j].double()[:, None])
        return y


def main(argv=None):
    ap = argparse.ArgumentParser(description="output projection with adapters, then routed experts")
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--graph", action="store_true", help="record the step in a CUDA graph and replay it")
    a = ap.parse_args(argv)
    gbuild.build()
    block = Block(a.tokens)
    g = torch.Generator(device="cuda:0").manual_seed(1)

    def new_inputs():
        for x in block.X_r:
            x.normal_(generator=g)
        block.adapter.copy_(torch.randint(-1, 8, (a.tokens,), generator=g, device="cuda:0"))

    new_inputs()
    block.step()
    replay = block.step
    if a.graph:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            block.step()
        replay = graph.replay
    for step in range(3):
        new_inputs()
        replay()
        block.check()
        ref = block.plain()
        err = float((block.y.double() - ref).norm() / ref.norm())
        print(f"step {step}: {a.tokens} tokens, relative error {err:.2e}")
        # five roundings to bf16 on the way (low-rank rows, h, gated, down, y), each
        # at most 2^-9 relatively
        if not err < 5 * 2.0 ** -9:
            raise SystemExit("the block is off")
    return 0


if __name__ == "__main__":
    sys.exit(main())
