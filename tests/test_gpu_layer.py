"""The expert layer of a few tokens against a plain 64-bit implementation: every number
of entries per expert that takes a path of its own, widths that no strip or piece
divides, dropped entries, an expert named twice, clusters, values that are not finite."""
import pytest
import torch

from tensor_gemm_reduction_gb300 import binding as B
from tensor_gemm_reduction_gb300 import build as gbuild

import routed_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def setup():
    gbuild.build()
    plan = B.gemm_shard_plan_create(0, 4096, 8192, 8192, 16)
    ws = B.gemm_routed_workspace_alloc(plan)
    B.gemm_routed_workspace_init(plan, ws)
    return plan, ws


def inputs(seed, T, topk, E, N, K, low=-1):
    g = U.gen(seed)
    ids = torch.randint(low, E, (T, topk), generator=g, device=U.DEV, dtype=torch.int32)
    return dict(X=U.normal(g, T, K), ids=ids, weights=torch.randn(T, topk, generator=g, device=U.DEV),
                W_up=U.normal(g, E, 2 * N, K, std=K ** -0.5), W_down=U.normal(g, E, K, N, std=N ** -0.5),
                base=U.normal(g, T, K))


def reference(X, ids, weights, W_up, W_down, base=None):
    """(values, bounds). Each product's fp32 sum is within SUM * sum |x w|; h is rounded to
    bf16 (ROUND) after an activation whose slope is below 1.1 and whose exponential is
    within a few 2^-22; the errors of h pass through |W_down|; the sum over entries is one
    more fp32 sum, and Y is rounded once."""
    T, topk = ids.shape
    y = torch.zeros(X.shape, dtype=torch.float64, device=X.device) if base is None else base.double()
    tol, mag = torch.zeros_like(y), y.abs()
    for e in range(W_up.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        N = W_down.shape[2]
        x, w, d = X[t].double(), W_up[e].double(), W_down[e].double()
        z, s = x @ w.t(), U.SUM * (x.abs() @ w.abs().t())
        gate, up, sg, su = z[:, :N], z[:, N:], s[:, :N], s[:, N:]
        act = gate * torch.sigmoid(gate)
        h = act * up
        dh = 1.1 * sg * up.abs() + act.abs() * su + 2.0 ** -18 * (1 + gate.abs()) * h.abs() + U.ROUND * h.abs()
        c = weights[t, j].double()[:, None]
        z = h @ d.t()
        y.index_add_(0, t, c * z)
        size = c.abs() * (h.abs() @ d.abs().t())
        more = U.ROUND * (c * z).abs() if T * topk > min(64, 8 * W_up.shape[0]) else 0.0   # rounded before they are weighted
        tol.index_add_(0, t, c.abs() * (dh @ d.abs().t()) + U.SUM * size + more)
        mag.index_add_(0, t, size)
    return y, U.ROUND * y.abs() + tol + U.SUM * mag + 1e-30


def check(setup, s, dtype=None, base=True):
    plan, ws = setup
    T, K = s["X"].shape
    full, Y = U.guarded(T, K)
    s = dict(s, base=s["base"] if base else None)
    ids = s["ids"] if dtype is None else s["ids"].to(dtype)
    B.gemm_expert_layer(plan, s["X"], ids, s["weights"], s["W_up"], s["W_down"], Y, ws, base=s["base"])
    U.close(Y, *reference(**s))
    assert U.untouched(full, T, torch.ones(T, dtype=torch.bool, device=U.DEV))
    return Y


@pytest.mark.parametrize("T,topk,E", [(1, 1, 1), (1, 8, 64), (2, 2, 3), (8, 1, 1), (9, 1, 1), (16, 8, 64), (17, 1, 1),
                                      (33, 1, 1), (33, 3, 7), (64, 1, 1), (64, 8, 256), (64, 3, 2), (64, 16, 1024), (8, 128, 5), (1, 128, 3), (64, 2, 100), (43, 3, 9), (1, 60, 8), (60, 1, 8), (16, 4, 8),
                                      (9, 7, 40), (3, 21, 100)])
@pytest.mark.parametrize("N,K", [(8, 8), (72, 200), (136, 1096), (1000, 520)])
def test_layer(setup, T, topk, E, N, K):
    """Up to hundreds of entries per expert, some dropped, some naming an expert twice."""
    check(setup, inputs(T * topk + N, T, topk, E, N, K, low=-1 if T > 1 else 0))


@pytest.mark.parametrize("T,E", [(1, 64), (16, 64), (61, 24)])
@pytest.mark.parametrize("N,K", [(896, 7168), (2048, 776)])
def test_layer_larger(setup, T, E, N, K):
    check(setup, inputs(T, T, 8, E, N, K, low=0))


@pytest.mark.parametrize("N,K", [(16, 8192), (256, 4000), (8192, 24), (4096, 512)])
def test_few_strips_or_columns_share_a_cluster(setup, N, K):
    check(setup, inputs(N, 3, 2, 4, N, K, low=0))


def test_ids_of_64_bits_and_no_base(setup):
    s = inputs(1, 7, 3, 9, 40, 264)
    a = check(setup, s)
    assert torch.equal(a, check(setup, s, dtype=torch.int64))
    check(setup, s, dtype=torch.int64, base=False)
    ids = s["ids"].long()
    ids[0, 0] = (1 << 32) + 2   # not expert 2
    check(setup, dict(s, ids=ids))


def test_every_entry_dropped(setup):
    plan, ws = setup
    s = inputs(2, 5, 2, 3, 16, 64)
    s["ids"].fill_(3)
    s["weights"].fill_(float("nan"))
    assert torch.equal(check(setup, s), s["base"])
    Y = torch.full((5, 64), 7.0, dtype=torch.bfloat16, device=U.DEV)
    B.gemm_expert_layer(plan, s["X"], s["ids"], s["weights"], s["W_up"], s["W_down"], Y, ws)
    assert not Y.any()
    none = torch.empty(0, 64, dtype=torch.bfloat16, device=U.DEV)
    B.gemm_expert_layer(plan, none, s["ids"][:0], s["weights"][:0], s["W_up"], s["W_down"], none, ws)


def test_an_expert_named_by_every_entry_of_a_token(setup):
    """Many entries of one token in one expert: a sum in their order, run after run."""
    for T in (1, 4):
        s = inputs(3, T, 96, 2, 48, 136, low=0)
        s["ids"].fill_(1)
        a = check(setup, s)
        for _ in range(3):
            assert torch.equal(a, check(setup, s))


def test_y_over_base_or_over_x(setup):
    plan, ws = setup
    s = inputs(4, 30, 4, 12, 200, 328)
    want = check(setup, s).clone()
    for name in ("base", "X"):
        c = dict(s, **{name: s[name].clone()})
        B.gemm_expert_layer(plan, c["X"], c["ids"], c["weights"], c["W_up"], c["W_down"], c[name], ws, base=c["base"])
        assert torch.equal(c[name], want)


def test_values_that_are_not_finite_stay_with_their_tokens(setup):
    """NaN in a token, infinity in an expert's weights and in a combine weight: the tokens
    that use them, and no other."""
    s = inputs(5, 40, 2, 10, 56, 72, low=0)
    s["ids"][:, 0] = torch.arange(40, device=U.DEV) % 5
    s["ids"][:, 1] = 5 + torch.arange(40, device=U.DEV) % 4   # nobody names expert 9
    want = check(setup, s).clone()
    plan, ws = setup
    s["X"][3, 5] = float("nan")
    s["W_down"][7, 11, 2] = float("inf")
    s["W_up"][9] = float("nan")
    s["weights"][20, 0] = float("inf")
    Y = torch.empty_like(want)
    B.gemm_expert_layer(plan, s["X"], s["ids"], s["weights"], s["W_up"], s["W_down"], Y, ws, base=s["base"])
    odd = torch.zeros(40, 72, dtype=torch.bool, device=U.DEV)
    odd[3] = odd[20] = True
    odd[(s["ids"][:, 1] == 7).nonzero()[:, 0], 11] = True
    assert torch.equal(Y[~odd], want[~odd]) and not Y[odd].isfinite().any()


# Entries and experts on either side of the limits up to which the two kernels run.
BOTH = pytest.mark.parametrize("T,topk,E", [(16, 4, 10), (17, 4, 10)], ids=["in two", "routed"])


@BOTH
def test_y_over_base_or_over_x_in_both_forms(setup, T, topk, E):
    plan, ws = setup
    s = inputs(14, T, topk, E, 136, 1096)
    want = check(setup, s).clone()
    for name in ("base", "X"):
        c = dict(s, **{name: s[name].clone()})
        B.gemm_expert_layer(plan, c["X"], c["ids"], c["weights"], c["W_up"], c["W_down"], c[name], ws, base=c["base"])
        assert torch.equal(c[name], want)


@BOTH
def test_values_that_are_not_finite_in_both_forms(setup, T, topk, E):
    """NaN in a token and in dropped entries' weights, infinity in an expert's weights and in
    an entry's weight: the tokens and columns that use them, and no other."""
    plan, ws = setup
    s = inputs(15, T, topk, E, 56, 200, low=0)
    s["ids"][:, 0] = torch.arange(T, device=U.DEV) % 4
    s["ids"][:, 1] = 4 + torch.arange(T, device=U.DEV) % 5   # nobody names expert 9
    s["ids"][:, 2:] = -1
    s["weights"][:, 2:] = float("nan")
    want = check(setup, dict(s, weights=s["weights"].nan_to_num())).clone()
    s["X"][3, 5] = float("nan")
    s["W_down"][7, 11, 2] = float("inf")
    s["W_up"][9] = s["W_down"][9] = float("nan")
    s["weights"][12, 0] = float("inf")
    Y = torch.empty_like(want)
    B.gemm_expert_layer(plan, s["X"], s["ids"], s["weights"], s["W_up"], s["W_down"], Y, ws, base=s["base"])
    odd = torch.zeros(T, 200, dtype=torch.bool, device=U.DEV)
    odd[3] = odd[12] = True
    odd[(s["ids"][:, 1] == 7).nonzero()[:, 0], 11] = True
    assert torch.equal(Y[~odd], want[~odd]) and not Y[odd].isfinite().any()


@BOTH
def test_every_entry_dropped_in_both_forms(setup, T, topk, E):
    s = inputs(16, T, topk, E, 64, 72)
    s["ids"].fill_(E)
    s["weights"].fill_(float("inf"))
    assert torch.equal(check(setup, s), s["base"])


@BOTH
def test_ids_written_by_the_launch_before(setup, T, topk, E):
    """Ids, weights and tokens that the kernel right before the call writes, call after call
    on the same buffers: every call uses its own."""
    plan, ws = setup
    s = [inputs(seed, T, topk, E, 64, 264) for seed in range(17, 21)]
    for c in s:
        c.update(W_up=s[0]["W_up"], W_down=s[0]["W_down"])
    want = [check(setup, c).clone() for c in s]
    buf = {k: torch.empty_like(s[0][k]) for k in ("ids", "weights", "X", "base")}
    out = [torch.empty_like(s[0]["X"]) for _ in range(40)]
    call = [B.prepare_expert_layer(plan, buf["X"], buf["ids"], buf["weights"], s[0]["W_up"], s[0]["W_down"], y, ws,
                                   base=buf["base"]) for y in out]
    for i, y in enumerate(out):
        for k in ("base", "X", "weights", "ids"):
            buf[k].copy_(s[i % 4][k])
        call[i]()
    torch.cuda.synchronize()
    for i, y in enumerate(out):
        assert torch.equal(y, want[i % 4]), i


def test_equals_the_four_routed_calls(setup):
    """The layer and route, gated, grouped, combine on the same inputs: both near the
    64-bit values, with the same experts read."""
    plan, ws = setup
    T, topk, E, N, K = 24, 4, 16, 264, 520
    s = inputs(6, T, topk, E, N, K)
    Y = check(setup, s)
    i32 = dict(dtype=torch.int32, device=U.DEV)
    offsets, source, position = torch.empty(E + 1, **i32), torch.empty(T * topk, **i32), torch.empty(T, topk, **i32)
    B.gemm_group_route(plan, s["ids"], E, offsets, source, position)
    h = torch.zeros(T * topk, N, dtype=torch.bfloat16, device=U.DEV)
    z, y = torch.zeros(T * topk, K, dtype=torch.bfloat16, device=U.DEV), torch.empty_like(Y)
    B.gemm_grouped_gated(plan, s["X"], s["W_up"], offsets, h, ws, rows=source)
    B.gemm_grouped(plan, h, s["W_down"], offsets, z, ws)
    B.gemm_group_combine(plan, z, position, s["weights"], y, base=s["base"])
    ref, bound = reference(**s)
    # the four calls round the down products to bf16 once more
    more = torch.zeros_like(ref)
    for j in range(topk):
        at = position[:, j].long()
        more += torch.where((at >= 0)[:, None], (s["weights"][:, j, None] * z[at.clamp_min(0)].float()).double().abs(), 0.0)
    U.close(y, ref, bound + U.ROUND * more)


def test_a_block_in_a_graph(setup):
    """Norm, expert layer over the residual's sum, norm in 8 bits, an 8-bit projection: as a
    decode step runs them, captured once and replayed on other inputs, beside another
    graph with a workspace of its own on another stream."""
    gbuild.build()
    T, topk, E, N, K = 12, 3, 8, 136, 272

    class Block:
        def __init__(self, seed):
            self.plan = B.gemm_shard_plan_create(0, 64, 512, 512, 2)
            self.routed = B.gemm_routed_workspace_alloc(self.plan)
            B.gemm_routed_workspace_init(self.plan, self.routed)
            self.ws = B.gemm_shard_workspace_alloc(self.plan)
            B.gemm_shard_workspace_init(self.plan, self.ws)
            self.s = inputs(seed, T, topk, E, N, K)
            g = U.gen(seed)
            bf, f32, e4 = (dict(dtype=d, device=U.DEV) for d in (torch.bfloat16, torch.float32, torch.float8_e4m3fn))
            self.res, self.gamma = U.normal(g, T, K), U.normal(g, K)
            self.sum, self.y = torch.empty(T, K, **bf), torch.empty(T, K, **bf)
            self.out, self.Q, self.S = torch.empty(T, K, **bf), torch.empty(T, K, **e4), torch.empty(3, T, **f32)
            W = U.normal(g, 40, K, std=K ** -0.5)
            self.W8, self.SW = torch.empty(40, K, **e4), torch.empty(1, 3, **f32)
            B.gemm_shard_quantize(self.plan, W, self.W8, self.SW, block_rows=128)
            self.Z = torch.empty(T, 40, **bf)
            s, p = self.s, self.plan
            self.calls = [
                B.prepare_rms_norm(p, s["X"], self.gamma, 1e-6, residual=self.res, sum=self.sum, Y=self.y),
                B.prepare_expert_layer(p, self.y, s["ids"], s["weights"], s["W_up"], s["W_down"], self.out, self.routed,
                                       base=self.sum),
                B.prepare_rms_norm(p, self.out, None, 1e-6, Q=self.Q, scale=self.S),
                B.prepare_ag_fp8(p, [self.Q], [self.S], self.W8, self.SW, self.Z, self.ws)]

        def step(self):
            for call in self.calls:
                call()

        def refill(self, seed):
            new = inputs(seed, T, topk, E, N, K)
            for name in ("X", "ids", "weights"):
                self.s[name].copy_(new[name])

    blocks = [Block(7), Block(8)]
    graphs = []
    for b in blocks:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            b.step()
        torch.cuda.current_stream().wait_stream(side)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            b.step()
    streams = [torch.cuda.Stream() for _ in blocks]
    for k in range(3):
        want = []
        for i, b in enumerate(blocks):
            b.refill(10 * k + i)
            b.step()
            torch.cuda.synchronize()
            want.append((b.out.clone(), b.Z.clone()))
            U.close(b.out, *reference(**dict(b.s, X=b.y, base=b.sum)))
            b.out.zero_()
            b.Z.zero_()
        torch.cuda.synchronize()
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for b, (out, Z) in zip(blocks, want):
            assert torch.equal(b.out, out) and torch.equal(b.Z, Z)
            B.gemm_shard_check_status(b.plan, b.ws)


@pytest.mark.parametrize("tokens,graph", [(1, False), (4, True), (37, True)])
def test_the_example_runs_a_decode_step(tokens, graph):
    import importlib.util
    import os
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_block.py")
    spec = importlib.util.spec_from_file_location("decode_block", at)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    assert mod.main(["--tokens", str(tokens)] + (["--graph"] if graph else [])) == 0
