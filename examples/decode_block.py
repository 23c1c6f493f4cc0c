"""One decode step of a tensor-parallel block with 8-bit projections, on one GPU.

    python examples/decode_block.py [--tokens 4] [--graph]

The attention output of T tokens sits in R K-shards, as R ranks would hold it. Each is
quantised (gemm_shard_quantize) and the output projection sums them on 8-bit operands
(gemm_ar_fp8). The residual is added and normed (gemm_shard_rms_norm); a router picks
experts for the normed rows, whose layer runs over the residual's sum
(gemm_expert_layer). A last norm leaves in 8 bits, as the next block's input projection
reads it (gemm_ag_fp8). Nothing waits for the host, so the step can be recorded in a CUDA
graph, whatever the router picks.

Weights and activations are random; every call's result is compared with plain PyTorch
in 64 bits on that call's own inputs.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from tensor_gemm_reduction_gb300 import binding as B  # noqa: E402
from tensor_gemm_reduction_gb300 import build as gbuild  # noqa: E402


def blocks(n):
    return -(-n // B.SCALE_BLOCK)


def rows_in_64_bits(q, scale):
    """What rows of e4m3 stand for (scale: column blocks x rows)."""
    return q.double() * scale.double().t().repeat_interleave(B.SCALE_BLOCK, 1)[:, :q.shape[1]]


def weights_in_64_bits(q, scale):
    """What weights of e4m3 stand for (scale: row blocks x column blocks)."""
    wide = scale.double().repeat_interleave(B.SCALE_BLOCK, 1)[:, :q.shape[1]]
    return q.double() * wide.repeat_interleave(B.SCALE_BLOCK, 0)[:q.shape[0]]


class Block:
    """Weights, buffers and prepared calls of one block for T tokens."""

    def __init__(self, T, hidden=1024, inner=512, shards=4, experts=16, topk=4, width=1536, seed=0, device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)
        bf, f32, e4 = (dict(dtype=d, device=device) for d in (torch.bfloat16, torch.float32, torch.float8_e4m3fn))

        def normal(*shape, fan_in):
            return torch.empty(*shape, **bf).normal_(0.0, fan_in ** -0.5, generator=g)

        k = hidden // shards
        self.topk, self.eps = topk, 1e-6
        self.plan = B.gemm_shard_plan_create(torch.device(device).index or 0, max(T * topk, 1), max(hidden, width),
                                             max(hidden, inner), shards)
        self.ws = B.gemm_shard_workspace_alloc(self.plan)
        B.gemm_shard_workspace_init(self.plan, self.ws)
        self.routed = B.gemm_routed_workspace_alloc(self.plan)
        B.gemm_routed_workspace_init(self.plan, self.routed)
        # 8-bit weights, quantised once.
        self.W_r = [self._quantised(normal(hidden, k, fan_in=hidden), f32, e4) for _ in range(shards)]
        self.W_in = self._quantised(normal(width, hidden, fan_in=hidden), f32, e4)
        self.gamma = [normal(hidden, fan_in=25.0) + 1 for _ in range(2)]
        self.router = normal(hidden, experts, fan_in=hidden)
        self.W_up, self.W_down = normal(experts, 2 * inner, hidden, fan_in=hidden), normal(experts, hidden, inner, fan_in=inner)
        # A step's inputs and buffers, reused step after step.
        self.X_r = [torch.zeros(T, k, **bf) for _ in range(shards)]
        self.residual = torch.zeros(T, hidden, **bf)
        self.Q_r = [torch.empty(T, k, **e4) for _ in range(shards)]
        self.S_r = [torch.empty(blocks(k), T, **f32) for _ in range(shards)]
        self.out, self.sum, self.normed, self.y = (torch.empty(T, hidden, **bf) for _ in range(4))
        self.ids = torch.empty(T, topk, dtype=torch.int32, device=device)
        self.weights = torch.empty(T, topk, **f32)
        self.Q, self.S = torch.empty(T, hidden, **e4), torch.empty(blocks(hidden), T, **f32)
        self.Z = torch.empty(T, width, **bf)
        p = self.plan
        self.project = [B.prepare_quantize(p, x, q, s) for x, q, s in zip(self.X_r, self.Q_r, self.S_r)] + [
            B.prepare_ar_fp8(p, self.Q_r, self.S_r, [w for w, _ in self.W_r], [s for _, s in self.W_r], self.out, self.ws),
            B.prepare_rms_norm(p, self.out, self.gamma[0], self.eps, residual=self.residual, sum=self.sum, Y=self.normed)]
        self.finish = [
            B.prepare_expert_layer(p, self.normed, self.ids, self.weights, self.W_up, self.W_down, self.y, self.routed,
                                   base=self.sum),
            B.prepare_rms_norm(p, self.y, self.gamma[1], self.eps, Q=self.Q, scale=self.S),
            B.prepare_ag_fp8(p, [self.Q], [self.S], *self.W_in, self.Z, self.ws)]

    def _quantised(self, w, f32, e4):
        q, s = torch.empty(w.shape, **e4), torch.empty(blocks(w.shape[0]), blocks(w.shape[1]), **f32)
        return B.gemm_shard_quantize(self.plan, w, q, s, block_rows=B.SCALE_BLOCK)

    def step(self):
        for call in self.project:
            call()
        top = (self.normed @ self.router).float().softmax(1).topk(self.topk, dim=1)
        self.ids.copy_(top.indices)
        self.weights.copy_(top.values / top.values.sum(1, keepdim=True))
        for call in self.finish:
            call()
        return self.Z

    def check(self):
        """The largest relative error of a call's result on its own inputs (2-norms)."""
        B.gemm_shard_check_status(self.plan, self.ws)
        B.gemm_shard_check_status(self.plan, self.routed)

        def off(have, want):
            return float((have.double() - want).norm() / want.norm())

        def norm(h, gamma):
            return h / torch.sqrt(h.square().mean(1, keepdim=True) + self.eps) * gamma.double()

        want = sum(rows_in_64_bits(q, s) @ weights_in_64_bits(*w).t() for q, s, w in zip(self.Q_r, self.S_r, self.W_r))
        h = self.out.double() + self.residual.double()
        y = self.sum.double()
        for e in range(self.W_up.shape[0]):
            t, j = (self.ids == e).nonzero(as_tuple=True)
            gate, up = (self.normed[t].double() @ self.W_up[e].double().t()).chunk(2, dim=1)
            z = (gate * torch.sigmoid(gate) * up) @ self.W_down[e].double().t()
            y.index_add_(0, t, z * self.weights[t, j].double()[:, None])
        z = rows_in_64_bits(self.Q, self.S) @ weights_in_64_bits(*self.W_in).t()
        rounded = max(off(self.out, want), off(self.sum, h), off(self.normed, norm(h, self.gamma[0])), off(self.y, y),
                      off(self.Z, z))
        quantised = max([off(rows_in_64_bits(q, s), x.double()) for q, s, x in zip(self.Q_r, self.S_r, self.X_r)]
                        + [off(rows_in_64_bits(self.Q, self.S), norm(self.y.double(), self.gamma[1]))])
        return rounded, quantised


def main(argv=None):
    ap = argparse.ArgumentParser(description="a decode step with 8-bit projections and an expert layer")
    ap.add_argument("--tokens", type=int, default=4)
    ap.add_argument("--graph", action="store_true", help="record the step in a CUDA graph and replay it")
    a = ap.parse_args(argv)
    gbuild.build()
    block = Block(a.tokens)
    g = torch.Generator(device="cuda:0").manual_seed(1)

    def new_inputs():
        for x in block.X_r + [block.residual]:
            x.normal_(generator=g)

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
        rounded, quantised = block.check()
        print(f"step {step}: {a.tokens} tokens, relative errors {rounded:.2e}, in 8 bits {quantised:.2e}")
        # three roundings to bf16 at most in a call, each at most 2^-8 of the value; one to
        # e4m3, at most 2^-4 (its smallest values lie far below a group's largest)
        if not (rounded < 3 * 2.0 ** -8 and quantised < 2.0 ** -4):
            raise SystemExit("the block is off")
    return 0


if __name__ == "__main__":
    sys.exit(main())
