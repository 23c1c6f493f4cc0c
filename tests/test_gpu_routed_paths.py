"""The routed projections' kernels and branches that small calls do not reach: adapters
of more than 1024 rows, adapters whose tiles are cut along k, more than sixteen token
tiles of one group or call, several weight tiles per CTA pair, combines with two vectors
per thread, and tensors of more than 2^32 elements.

The bounds are routed_util's: a sum of K products is within 2^-17 of sum |x w| for every
K here (sqrt(K) * 2^-24 < 2^-17 up to K = 16384)."""
import pytest
import torch

from tensor_gemm_reduction_gb300 import binding as B
from tensor_gemm_reduction_gb300 import build as gbuild

import routed_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def setup():
    gbuild.build()
    plan = B.gemm_shard_plan_create(0, 32768, 8192, 8192, 16)
    ws = B.gemm_routed_workspace_alloc(plan)
    B.gemm_routed_workspace_init(plan, ws)
    return plan, ws


def adapters(g, M, L, run, none):
    a = torch.randint(0, L, (-(-M // run),), generator=g, device=U.DEV, dtype=torch.int32).repeat_interleave(run)[:M]
    return a.masked_fill(torch.rand(M, generator=g, device=U.DEV) < none, -1).contiguous()


def lora(setup, M, N, K_r, L, rank, run, none=0.2, odd=()):
    """One case against the 64-bit product; `odd`: (adapter, column, place, value) of B."""
    plan, ws = setup
    g = U.gen(M + N + rank)
    K = sum(K_r)
    X_r = [U.normal(g, M, k) for k in K_r]
    W_r = [U.normal(g, N, k, std=K ** -0.5) for k in K_r]
    A_r = [U.normal(g, L, rank, k, std=K ** -0.5) for k in K_r]
    Bm = U.normal(g, L, N, rank, std=rank ** -0.5)
    for a, n, j, value in odd:
        Bm[a, n, j] = value
    adapter = adapters(g, M, L, run, none)
    if odd:
        adapter[:3] = torch.arange(min(3, M), device=U.DEV)
    scale = torch.randn(L, generator=g, device=U.DEV)
    outs = []
    for _ in range(2):
        full, Y = U.guarded(M, N)
        B.gemm_ar_lora(plan, X_r, W_r, A_r, Bm, adapter, Y, ws, scale=scale)
        outs.append(full)
        assert U.untouched(full, M, torch.ones(M, dtype=torch.bool, device=U.DEV))
    B.gemm_shard_check_status(plan, ws)
    assert torch.equal(outs[0], outs[1]), "two calls on the same inputs differ"
    ref, bound = U.lora_ref(X_r, W_r, A_r, Bm, adapter, scale)
    finite, infinite = torch.isfinite(ref), torch.isinf(ref)
    assert bool(odd) != bool(finite.all())
    assert torch.equal(torch.isnan(Y), torch.isnan(ref))
    assert torch.equal(Y[infinite].double(), ref[infinite])
    U.close(Y[finite], ref[finite], bound[finite])


ODD = [(1, 3, 0, float("inf")), (1, 150, 7, float("-inf")), (2, 40, 2, float("nan")), (0, 255, 5, float("inf"))]


@pytest.mark.parametrize("M,N,K_r,L,rank,run", [
    (1025, 264, [200], 5, 24, 1), (1100, 520, [328, 72], 9, 96, 200), (1300, 264, [136], 200, 16, 1),
    (2100, 264, [256], 7, 64, 1), (2100, 520, [72, 200], 3, 128, 300), (4200, 264, [72], 6, 40, 17),
    (2049, 200, [64] * 5, 1, 8, 1),
], ids=lambda v: str(v).replace(" ", ""))
def test_lora_of_many_rows(setup, M, N, K_r, L, rank, run):
    lora(setup, M, N, K_r, L, rank, run)


def test_lora_of_many_rows_without_an_adapter_and_with_one_each(setup):
    lora(setup, 1153, 264, [136], 4, 48, 1, none=1.0)
    lora(setup, 1153, 264, [136], 4, 48, 1, none=0.0)


def test_lora_of_many_rows_with_infinite_weights(setup):
    lora(setup, 1500, 264, [136], 4, 96, 40, odd=ODD)


@pytest.mark.parametrize("M,N,L,rank", [(40, 264, 40, 16), (100, 264, 60, 32), (100, 264, 5, 128), (200, 264, 200, 24),
                                        (256, 520, 50, 72), (300, 4096, 30, 64), (300, 4096, 100, 16),
                                        (300, 4096, 9, 128)])
@pytest.mark.parametrize("odd", [False, True], ids=["finite", "infinite"])
def test_lora_cut_along_k(setup, M, N, L, rank, odd):
    """Few tiles and a long k: pieces share the adapters' steps."""
    K_r = [6168, 1000] if M == 300 else [4160, 1000]
    lora(setup, M, N, K_r, L, rank, 1, odd=ODD if odd else ())


@pytest.mark.parametrize("counts,N,K", [
    ([1100] + [0] * 60, 264, 136),           # 64-token tiles
    ([0] * 20 + [2200], 264, 72),            # 128
    ([4500], 264, 128), ([3, 4700, 5], 520, 64),   # 256
    ([8400], 264, 72), ([8350, 1, 300], 264, 200),   # 512
], ids=lambda v: "-".join(map(str, v)) if isinstance(v, list) and len(v) < 9 else str(len(v)) if isinstance(v, list) else str(v))
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gathered"])
def test_more_than_sixteen_token_tiles(setup, counts, N, K, gated, gather):
    plan, ws = setup
    g = U.gen(sum(counts) + N)
    M, E = sum(counts), len(counts)
    T = M // 2 if gather else M
    X = U.normal(g, T, K)
    W = U.normal(g, E, 2 * N if gated else N, K, std=K ** -0.5)
    rows = torch.randint(0, T, (M,), generator=g, device=U.DEV, dtype=torch.int32) if gather else None
    full, Y = U.guarded(M, N)
    (B.gemm_grouped_gated if gated else B.gemm_grouped)(plan, X, W, U.offsets_of(counts), Y, ws, rows=rows)
    B.gemm_shard_check_status(plan, ws)
    ref, bound = U.grouped_ref(X, W, counts, rows, gated)
    U.close(Y, ref, bound)
    assert U.untouched(full, M, torch.ones(M, dtype=torch.bool, device=U.DEV))


@pytest.mark.parametrize("T,topk,H", [(701, 3, 3592), (400, 9, 6288), (5000, 1, 512)])
@pytest.mark.parametrize("base", ["none", "apart", "output"])
def test_combine_of_many_vectors(setup, T, topk, H, base):
    plan, _ = setup
    g = U.gen(T + H)
    Z = U.normal(g, T * topk, H)
    position = torch.randint(-2, T * topk + 5, (T, topk), generator=g, device=U.DEV, dtype=torch.int32)
    weights = torch.randn(T, topk, generator=g, device=U.DEV)
    dead = (position < 0) | (position >= Z.shape[0])
    weights[dead] = float("nan")
    added = U.normal(g, T, H) if base != "none" else None
    full, Y = U.guarded(T, H)
    if base == "output":
        Y.copy_(added)
    B.gemm_group_combine(plan, Z, position, weights, Y, base=Y if base == "output" else added)
    w = torch.where(dead, 0.0, weights.double())
    rows = Z.double()[position.long().clamp(0, Z.shape[0] - 1)] * w[:, :, None]
    ref = rows.sum(1) + (added.double() if added is not None else 0.0)
    U.close(Y, ref, U.ROUND * ref.abs() + U.SUM * (rows.abs().sum(1) + 1) + 1e-30)
    assert U.untouched(full, T, torch.ones(T, dtype=torch.bool, device=U.DEV))


@pytest.mark.parametrize("kind", ["grouped", "gathered", "gated", "wide", "lora few", "lora half", "lora"])
def test_waits_of_a_nanosecond(kind):
    """The shortest limit that a wait can have: the call gives its result or a status, never
    a fault, and after another init the same workspace serves the same call."""
    gbuild.build()
    g = U.gen(len(kind))
    M = {"lora few": 1, "lora half": 100, "wide": 2000}.get(kind, 700)
    N, K, L, rank = 520, 2008, 5, 16
    X, W = U.normal(g, M, K), U.normal(g, 3, 2 * N if kind == "gated" else N, K, std=K ** -0.5)
    full, Y = U.guarded(M, N)
    counts = [M // 2, 0, M - M // 2]
    A, Bm = U.normal(g, L, rank, K, std=K ** -0.5), U.normal(g, L, N, rank, std=rank ** -0.5)
    adapter = adapters(g, M, L, 1, 0.1)
    rows = torch.randint(0, M, (M,), generator=g, device=U.DEV, dtype=torch.int32) if kind == "gathered" else None
    for limit in (1, 0):   # 0: the default
        plan = B.gemm_shard_plan_create(0, 4096, 1024, 4096, 1)
        B.gemm_shard_plan_set_option(plan, B.GSR_OPT_TIMEOUT_NS, limit)
        if limit:
            ws = B.gemm_routed_workspace_alloc(plan)
        B.gemm_routed_workspace_init(plan, ws)
        if kind.startswith("lora"):
            B.gemm_ar_lora(plan, [X], [W[0]], [A], Bm, adapter, Y, ws)
        elif kind == "gated":
            B.gemm_grouped_gated(plan, X, W, U.offsets_of(counts), Y, ws)
        else:
            B.gemm_grouped(plan, X, W, U.offsets_of(counts), Y, ws, rows=rows)
        torch.cuda.synchronize()
        assert U.untouched(full, M, torch.ones(M, dtype=torch.bool, device=U.DEV))
        try:
            B.gemm_shard_check_status(plan, ws)
        except B.GsrError as e:
            assert limit and e.status == B.GSR_ERR_TIMEOUT
            continue
        ref, bound = (U.lora_ref([X], [W[0]], [A], Bm, adapter, None) if kind.startswith("lora")
                      else U.grouped_ref(X, W, counts, rows, kind == "gated"))
        U.close(Y, ref, bound)


@pytest.mark.parametrize("M,L,rank,odd", [(1, 3, 16, False), (2, 3, 16, True), (1, 3, 32, True), (40, 40, 16, True),
                                          (100, 60, 32, False), (128, 9, 128, True), (200, 200, 24, False),
                                          (256, 50, 72, True)])
@pytest.mark.parametrize("N,ctas", [(4096, 8), (4096, 2), (12008, 0)])
def test_several_weight_tiles_per_pair(M, L, rank, odd, N, ctas):
    """Few rows and more weight tiles than CTA pairs: tiles follow one another in the same
    ring, accumulators and teams."""
    gbuild.build()
    plan = B.gemm_shard_plan_create(0, 1024, 16384, 4096, 4)
    B.gemm_shard_plan_set_option(plan, B.GSR_OPT_MAX_CTAS, ctas)
    ws = B.gemm_routed_workspace_alloc(plan)
    B.gemm_routed_workspace_init(plan, ws)
    lora((plan, ws), M, N, [328, 1000], L, rank, 1, none=0.0 if M < 3 else 0.2, odd=[
        (a % (L if M > 2 else M), n, j, v) for a, n, j, v in ODD + [(1, 2050, 1, float("inf")), (0, 4090, 3, float("-inf"))]
    ] if odd else ())


# ---------------------------------------------------------------- offsets past 32 bits

def big(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16, device=U.DEV)


def test_grouped_weights_and_rows_past_32_bits(setup):
    """E x N x K and T x K above 2^32 elements: the last group's weights, the last rows."""
    plan, ws = setup
    g = U.gen(40)
    E, N, K, T = 70, 8192, 8192, 600000
    W, X = big(E, N, K), big(T, K)
    counts = [0] * E
    counts[0], counts[E - 2], counts[E - 1] = 5, 30, 3
    for e in (0, E - 2, E - 1):
        W[e].normal_(0.0, K ** -0.5, generator=g)
    rows = torch.randint(T - 100, T, (38,), generator=g, device=U.DEV, dtype=torch.int32)
    rows[::3] -= T - 100
    X[-100:].normal_(generator=g)
    X[:100].normal_(generator=g)
    for gather in (True, False):
        Y = torch.empty(38, N, dtype=torch.bfloat16, device=U.DEV)
        x = X if gather else X[-38:]
        B.gemm_grouped(plan, x, W, U.offsets_of(counts), Y, ws, rows=rows if gather else None)
        B.gemm_shard_check_status(plan, ws)
        x = x[rows.long()] if gather else x
        at = 0
        for e in (0, E - 2, E - 1):
            part, n = x[at:at + counts[e]], counts[e]
            ref, bound = U.grouped_ref(part, W[e:e + 1], [n], None, False)
            U.close(Y[at:at + n], ref, bound, f"group {e}")
            at += n


def test_combined_rows_past_32_bits(setup):
    plan, _ = setup
    g = U.gen(41)
    rows, H = 600000, 7168
    Z = big(rows, H)
    Z[-50:].normal_(generator=g)
    Z[:50].normal_(generator=g)
    for T in (7, 400):
        position = torch.randint(rows - 50, rows, (T, 2), generator=g, device=U.DEV, dtype=torch.int32)
        position[:, 1] -= rows - 50
        weights = torch.randn(T, 2, generator=g, device=U.DEV)
        Y = torch.empty(T, H, dtype=torch.bfloat16, device=U.DEV)
        B.gemm_group_combine(plan, Z, position, weights, Y)
        part = Z[position.long()].double() * weights.double()[:, :, None]
        ref = part.sum(1)
        U.close(Y, ref, U.ROUND * ref.abs() + U.SUM * (part.abs().sum(1) + 1) + 1e-30)


@pytest.mark.parametrize("M", [2, 40, 300, 1100])
def test_adapters_past_32_bits(setup, M):
    """L x N x rank and L x rank x K above 2^32 elements, adapters of both ends."""
    plan, ws = setup
    g = U.gen(42)
    L, N, K, rank = 65536, 1032, 1032, 64
    A, Bm = big(L, rank, K), big(L, N, rank)
    used = [0, 1, 40000, L - 2, L - 1]
    for a in used:
        A[a].normal_(0.0, K ** -0.5, generator=g)
        Bm[a].normal_(0.0, rank ** -0.5, generator=g)
    Bm[L - 1, 700, 5] = float("inf")
    X, W = U.normal(g, M, K), U.normal(g, N, K, std=K ** -0.5)
    adapter = torch.tensor(used, device=U.DEV)[torch.arange(M, device=U.DEV) % 5].to(torch.int32)
    adapter[M - 1] = L - 1
    Y = torch.empty(M, N, dtype=torch.bfloat16, device=U.DEV)
    B.gemm_ar_lora(plan, [X], [W], [A], Bm, adapter, Y, ws)
    B.gemm_shard_check_status(plan, ws)
    few = torch.full_like(adapter, -1)
    for i, a in enumerate(used):
        few[adapter == a] = i
    ref, bound = U.lora_ref([X], [W], [A[used]], Bm[used], few, None)
    finite, infinite = torch.isfinite(ref), torch.isinf(ref)
    assert torch.equal(Y[infinite].double(), ref[infinite]) and torch.equal(torch.isnan(Y), torch.isnan(ref))
    U.close(Y[finite], ref[finite], bound[finite])
