"""The routed projections against plain 64-bit implementations, at the sizes and
routings where they can go wrong: empty groups, groups of one row, one group
with every row, widths that no tile divides, shards of odd k, rows without an
adapter, adapters mixed row by row, values out of range, dropped entries."""
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


def status_ok(setup):
    B.gemm_shard_check_status(*setup)


# ---------------------------------------------------------------- route

@pytest.mark.parametrize("T,topk,E", [(1, 1, 1), (1, 8, 64), (33, 3, 7), (512, 8, 256), (513, 8, 1024),
                                      (1025, 4, 5), (5000, 6, 100)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_route_equals_a_stable_sort(setup, T, topk, E, dtype):
    plan, _ = setup
    ids = torch.randint(-1, E + 1, (T, topk), generator=U.gen(T), device=U.DEV).to(dtype)   # some out of range
    if dtype is torch.int64:
        ids[0, 0] = (1 << 32) + 0   # not group 0
    out = [torch.full((n,), 77, dtype=torch.int32, device=U.DEV) for n in (E + 1, T * topk)]
    pos = torch.full((T, topk), 77, dtype=torch.int32, device=U.DEV)
    B.gemm_group_route(plan, ids, E, out[0], out[1], pos)
    ref = U.route_ref(ids.cpu(), E)
    for have, want, name in zip((out[0], out[1], pos), ref, ("offsets", "source", "position")):
        assert torch.equal(have.cpu(), want), name


def test_route_of_no_tokens_and_of_dropped_ones(setup):
    plan, _ = setup
    i32 = dict(dtype=torch.int32, device=U.DEV)
    offsets = torch.full((9,), 5, **i32)
    B.gemm_group_route(plan, torch.empty(0, 2, **i32), 8, offsets, torch.empty(0, **i32), torch.empty(0, 2, **i32))
    assert not offsets.any()
    offsets.fill_(5)
    source, position = torch.full((6,), 5, **i32), torch.full((3, 2), 5, **i32)
    B.gemm_group_route(plan, torch.full((3, 2), -1, **i32), 8, offsets, source, position)
    assert not offsets.any() and (source == -1).all() and (position == -1).all()


@pytest.mark.parametrize("T,topk,E", [(32768, 8, 3), (140000, 2, 1024)])
def test_route_of_many_entries(T, topk, E):
    """The largest number of entries that stays in registers, and more than that."""
    plan = B.gemm_shard_plan_create(0, T * topk, 64, 64, 1)
    ids = torch.randint(-1, E, (T, topk), generator=U.gen(E), device=U.DEV)
    i32 = dict(dtype=torch.int32, device=U.DEV)
    offsets, source, position = torch.empty(E + 1, **i32), torch.empty(T * topk, **i32), torch.empty(T, topk, **i32)
    B.gemm_group_route(plan, ids, E, offsets, source, position)
    flat = ids.reshape(-1)
    order = torch.argsort(torch.where(flat < 0, E, flat), stable=True)
    kept = int((flat >= 0).sum())
    assert torch.equal(offsets[1:].long(), torch.bincount(flat[flat >= 0], minlength=E).cumsum(0))
    assert int(offsets[0]) == 0 and (source[kept:] == -1).all()
    assert torch.equal(source[:kept].long(), order[:kept] // topk)
    back = torch.full_like(flat, -1)
    back[order[:kept]] = torch.arange(kept, device=U.DEV)
    assert torch.equal(position.reshape(-1).long(), back)


def route_by_sorting(ids, E):
    """The route's outputs by a stable sort, ids out of range dropped."""
    flat = ids.reshape(-1).long()
    live = (flat >= 0) & (flat < E)
    order = torch.argsort(torch.where(live, flat, E), stable=True)
    kept = int(live.sum())
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.bincount(flat[live], minlength=E).cumsum(0)
    source, position = torch.full_like(flat, -1), torch.full_like(flat, -1)
    source[:kept] = order[:kept] // ids.shape[1]
    position[order[:kept]] = torch.arange(kept, device=ids.device)
    return offsets, source, position.reshape(ids.shape)


@pytest.mark.parametrize("T,topk", [(2048, 1), (683, 3), (8191, 6), (8193, 6), (65551, 1), (103, 128),
                                    (1000001, 5), (1 << 25, 1), ((1 << 25) // 3 + 7, 3)])
@pytest.mark.parametrize("E,one", [(1, False), (9, False), (1024, False), (1000, True)])
def test_route_from_few_entries_to_very_many(T, topk, E, one):
    """Numbers of entries around the changes of form, parts that end unevenly, a group of
    everything, and entries past 2^25."""
    plan = B.gemm_shard_plan_create(0, T * topk, 64, 64, 1)
    ids = torch.randint(-1, E + 1, (T, topk), generator=U.gen(E), device=U.DEV, dtype=torch.int32)
    if one:
        ids.fill_(E - 1)
    i32 = dict(dtype=torch.int32, device=U.DEV)
    have = torch.full((E + 1,), 7, **i32), torch.full((T * topk,), 7, **i32), torch.full((T, topk), 7, **i32)
    B.gemm_group_route(plan, ids, E, *have)
    for a, b, name in zip(have, route_by_sorting(ids, E), ("offsets", "source", "position")):
        assert torch.equal(a.long(), b), name


def test_routes_of_many_entries_follow_one_another(setup):
    """Calls in a row, recorded in a graph, whose ids change between replays."""
    T, topk, E = 9001, 7, 200
    plan = B.gemm_shard_plan_create(0, T * topk, 64, 64, 1)
    i32 = dict(dtype=torch.int32, device=U.DEV)
    ids = [torch.zeros(T, topk, **i32) for _ in range(3)]
    outs = [(torch.empty(E + 1, **i32), torch.empty(T * topk, **i32), torch.empty(T, topk, **i32)) for _ in ids]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        B.gemm_group_route(plan, ids[0], E, *outs[0])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids[1].copy_(ids[0] + 1)
        for x, out in zip(ids, outs):
            B.gemm_group_route(plan, x, E, *out)
        ids[2].copy_(ids[1] * 2)      # read by the next replay
    for k in range(4):
        ids[0].copy_(torch.randint(-1, E, (T, topk), generator=U.gen(k), device=U.DEV, dtype=torch.int32))
        read = [ids[0].clone(), ids[0] + 1, ids[2].clone()]
        graph.replay()
        for x, out in zip(read, outs):
            for a, b in zip(out, route_by_sorting(x, E)):
                assert torch.equal(a.long(), b)


# ---------------------------------------------------------------- grouped

GROUPS = [
    [1], [0, 1, 0], [5, 0, 3, 16, 17], [64] * 3, [65, 1, 129, 0, 63],       # narrow tiles
    [100, 128, 90], [200, 0, 60, 127],                                     # 128 tokens
    [256], [300, 257, 0, 1000], [0, 0, 700], [1500, 3],                    # 256 tokens
]


@pytest.mark.parametrize("counts", GROUPS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("N,K", [(8, 8), (264, 200), (512, 1024)])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gathered"])
def test_grouped(setup, counts, N, K, gated, gather):
    plan, ws = setup
    g = U.gen(sum(counts) + N)
    M, E = sum(counts), len(counts)
    T = max(1, M // 2) if gather else M
    X = U.normal(g, T, K)
    W = U.normal(g, E, 2 * N if gated else N, K, std=K ** -0.5)
    rows = torch.randint(0, T, (M,), generator=g, device=U.DEV, dtype=torch.int32) if gather else None
    full, Y = U.guarded(M, N)
    call = B.gemm_grouped_gated if gated else B.gemm_grouped
    call(plan, X, W, U.offsets_of(counts), Y, ws, rows=rows)
    status_ok(setup)
    ref, bound = U.grouped_ref(X, W, counts, rows, gated)
    U.close(Y, ref, bound)
    assert U.untouched(full, M, torch.ones(M, dtype=torch.bool, device=U.DEV))


@pytest.mark.parametrize("counts", [[257], [512, 1, 300], [0, 1029], [600, 528, 40]], ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gathered"])
def test_grouped_long_k(setup, counts, gated, gather):
    """Large groups and a long k: tiles of up to 512 tokens."""
    plan, ws = setup
    g = U.gen(sum(counts))
    M, E, N, K = sum(counts), len(counts), 200, 4104
    T = M // 3 if gather else M
    X = U.normal(g, T, K)
    W = U.normal(g, E, 2 * N if gated else N, K, std=K ** -0.5)
    rows = torch.randint(-1, T, (M,), generator=g, device=U.DEV, dtype=torch.int32) if gather else None
    full, Y = U.guarded(M, N)
    call = B.gemm_grouped_gated if gated else B.gemm_grouped
    call(plan, X, W, U.offsets_of(counts), Y, ws, rows=rows)
    status_ok(setup)
    ref, bound = U.grouped_ref(X, W, counts, rows, gated)
    U.close(Y, ref, bound)
    assert U.untouched(full, M, torch.ones(M, dtype=torch.bool, device=U.DEV))


@pytest.mark.parametrize("each,gather", [(12, True), (12, False), (90, True), (250, True), (250, False), (300, False)])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_whole_tiles_and_cut_ones(setup, each, gather, gated):
    """More tiles than pairs, and a k long enough that the remaining ones are cut."""
    plan, ws = setup
    N, K, counts = 1088 // (2 if gated else 1), 5160, [each] * 19 + [each - 5]
    M = sum(counts)
    g = U.gen(each)
    X = U.normal(g, M, K)
    W = U.normal(g, len(counts), 2 * N if gated else N, K, std=K ** -0.5)
    rows = torch.randint(0, M, (M,), generator=g, device=U.DEV, dtype=torch.int32) if gather else None
    full, Y = U.guarded(M, N)
    (B.gemm_grouped_gated if gated else B.gemm_grouped)(plan, X, W, U.offsets_of(counts), Y, ws, rows=rows)
    status_ok(setup)
    ref, bound = U.grouped_ref(X, W, counts, rows, gated)
    U.close(Y, ref, bound)
    assert U.untouched(full, M, torch.ones(M, dtype=torch.bool, device=U.DEV))


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_rows_of_no_group_stay(setup, gated):
    """Offsets that start past 0 and end before M: the other rows are not written."""
    plan, ws = setup
    g = U.gen(1)
    X, W = U.normal(g, 50, 128), U.normal(g, 2, 128, 128)
    N = 64 if gated else 128
    full, Y = U.guarded(50, N)
    offsets = torch.tensor([4, 20, 33], dtype=torch.int32, device=U.DEV)
    (B.gemm_grouped_gated if gated else B.gemm_grouped)(plan, X, W, offsets, Y, ws)
    status_ok(setup)
    written = torch.zeros(50, dtype=torch.bool, device=U.DEV)
    written[4:33] = True
    assert U.untouched(full, 50, written)
    ref, bound = U.grouped_ref(X[4:], W, [16, 13], None, gated)
    U.close(Y[4:33], ref, bound)


def test_offsets_out_of_range_are_clamped(setup):
    plan, ws = setup
    g = U.gen(2)
    X, W = U.normal(g, 40, 64), U.normal(g, 3, 64, 64)
    full, Y = U.guarded(40, 64)
    offsets = torch.tensor([-7, 10, 10, 900], dtype=torch.int32, device=U.DEV)
    B.gemm_grouped(plan, X, W, offsets, Y, ws)
    status_ok(setup)
    ref, bound = U.grouped_ref(X, W, [10, 0, 30], None, False)
    U.close(Y, ref, bound)
    assert U.untouched(full, 40, torch.ones(40, dtype=torch.bool, device=U.DEV))
    # decreasing offsets: empty groups
    Y.view(torch.int16).fill_(U.SENTINEL)
    B.gemm_grouped(plan, X, W, torch.tensor([30, 20, 10, 0], dtype=torch.int32, device=U.DEV), Y, ws)
    status_ok(setup)
    assert U.untouched(full, 40, torch.zeros(40, dtype=torch.bool, device=U.DEV))


def test_gathered_rows_out_of_range_are_zero(setup):
    plan, ws = setup
    g = U.gen(3)
    X, W = U.normal(g, 9, 136), U.normal(g, 2, 72, 136)
    rows = torch.tensor([0, -1, 8, 9, 1 << 30, 3, 3, -(1 << 31)], dtype=torch.int32, device=U.DEV)
    Y = torch.empty(8, 72, dtype=torch.bfloat16, device=U.DEV)
    B.gemm_grouped(plan, X, W, U.offsets_of([3, 5]), Y, ws, rows=rows)
    status_ok(setup)
    ref, bound = U.grouped_ref(X, W, [3, 5], rows, False)
    U.close(Y, ref, bound)


def test_nan_stays_in_its_row_and_group(setup):
    """A row or a weight of NaN or infinity reaches its own products only."""
    plan, ws = setup
    g = U.gen(4)
    counts = [3, 20, 1]
    X, W = U.normal(g, 24, 128), U.normal(g, 3, 136, 128)
    X[5, 7] = float("nan")
    W[2, 11, 0] = float("inf")
    Y = torch.empty(24, 136, dtype=torch.bfloat16, device=U.DEV)
    B.gemm_grouped(plan, X, W, U.offsets_of(counts), Y, ws)
    status_ok(setup)
    bad = torch.zeros(24, 136, dtype=torch.bool, device=U.DEV)
    bad[5], bad[23, 11] = True, True
    assert torch.equal(~torch.isfinite(Y), bad)
    ref, bound = U.grouped_ref(X, W, counts, None, False)
    U.close(Y[~bad], ref[~bad], bound[~bad])


def test_many_groups_and_cut_tiles(setup):
    """1024 groups of none to a few rows; and few long tiles whose k is cut."""
    plan, ws = setup
    g = U.gen(5)
    counts = torch.randint(-3, 4, (1024,), generator=g, device=U.DEV).clamp_min(0).tolist()
    X, W = U.normal(g, sum(counts), 72), U.normal(g, 1024, 40, 72, std=72 ** -0.5)
    Y = torch.empty(sum(counts), 40, dtype=torch.bfloat16, device=U.DEV)
    B.gemm_grouped(plan, X, W, U.offsets_of(counts), Y, ws)
    status_ok(setup)
    ref, bound = U.grouped_ref(X, W, counts, None, False)
    U.close(Y, ref, bound, "many groups")
    for counts in ([1, 2], [70, 0, 200], [600, 300]):
        X, W = U.normal(g, sum(counts), 4000), U.normal(g, len(counts), 520, 4000, std=4000 ** -0.5)
        outs = []
        for _ in range(2):
            Y = torch.empty(sum(counts), 520, dtype=torch.bfloat16, device=U.DEV)
            B.gemm_grouped(plan, X, W, U.offsets_of(counts), Y, ws)
            outs.append(Y)
        status_ok(setup)
        ref, bound = U.grouped_ref(X, W, counts, None, False)
        U.close(outs[0], ref, bound, f"cut tiles {counts}")
        assert torch.equal(outs[0], outs[1]), "two calls on the same inputs differ"


# ---------------------------------------------------------------- combine

@pytest.mark.parametrize("T,topk,H", [(1, 1, 8), (5, 8, 1000), (33, 3, 7168), (7, 20, 64)])
@pytest.mark.parametrize("with_base", [False, True])
def test_combine(setup, T, topk, H, with_base):
    plan, _ = setup
    g = U.gen(T + H)
    Z = U.normal(g, T * topk + 3, H)
    position = torch.randint(-2, T * topk + 5, (T, topk), generator=g, device=U.DEV, dtype=torch.int32)
    weights = torch.randn(T, topk, generator=g, device=U.DEV)
    dead = (position < 0) | (position >= Z.shape[0])
    weights[dead] = float("nan")   # of entries that add nothing
    base = U.normal(g, T, H) if with_base else None
    full, Y = U.guarded(T, H)
    B.gemm_group_combine(plan, Z, position, weights, Y, base=base)
    w = torch.where(dead, 0.0, weights.double())
    rows = Z.double()[position.long().clamp(0, Z.shape[0] - 1)] * w[:, :, None]
    ref = rows.sum(1) + (base.double() if with_base else 0.0)
    U.close(Y, ref, U.ROUND * ref.abs() + U.SUM * (rows.abs().sum(1) + 1) + 1e-30)
    assert U.untouched(full, T, torch.ones(T, dtype=torch.bool, device=U.DEV))


def test_combine_into_its_base(setup):
    plan, _ = setup
    g = U.gen(9)
    Z, Y = U.normal(g, 12, 264), U.normal(g, 4, 264)
    position = torch.randperm(12, generator=g, device=U.DEV).to(torch.int32).view(4, 3)
    weights = torch.rand(4, 3, generator=g, device=U.DEV)
    apart = torch.empty_like(Y)
    B.gemm_group_combine(plan, Z, position, weights, apart, base=Y)
    B.gemm_group_combine(plan, Z, position, weights, Y, base=Y)
    assert torch.equal(Y, apart)


# ---------------------------------------------------------------- adapters

LORA = [  # M, N, K_r, L, rank, run
    (1, 264, [8], 1, 8, 1), (1, 1024, [896, 72], 3, 16, 1), (1, 520, [304] * 16, 2, 24, 1), (2, 264, [136, 8], 3, 16, 1),
    (3, 200, [64], 2, 16, 1), (7, 512, [200, 64], 4, 32, 1),
    (64, 520, [512], 64, 16, 1), (65, 256, [128] * 4, 5, 64, 1), (128, 1000, [304, 208], 100, 24, 1),
    (129, 264, [256], 7, 128, 1), (256, 512, [136] * 3, 300, 8, 1), (257, 512, [256], 2, 48, 100),
    (600, 776, [512, 200], 40, 96, 1), (1000, 1024, [448] * 2, 3, 64, 300),
]


def adapters(g, M, L, run, none):
    a = torch.randint(0, L, (-(-M // run),), generator=g, device=U.DEV, dtype=torch.int32).repeat_interleave(run)[:M]
    return a.masked_fill(torch.rand(M, generator=g, device=U.DEV) < none, -1).contiguous()


@pytest.mark.parametrize("M,N,K_r,L,rank,run", LORA, ids=lambda v: str(v).replace(" ", ""))
@pytest.mark.parametrize("none,scaled", [(0.0, True), (0.3, True), (1.0, False), (0.0, False)])
def test_lora(setup, M, N, K_r, L, rank, run, none, scaled):
    plan, ws = setup
    g = U.gen(M + N)
    K = sum(K_r)
    X_r = [U.normal(g, M, k) for k in K_r]
    W_r = [U.normal(g, N, k, std=K ** -0.5) for k in K_r]
    A_r = [U.normal(g, L, rank, k, std=K ** -0.5) for k in K_r]
    Bm = U.normal(g, L, N, rank, std=rank ** -0.5)
    adapter = adapters(g, M, L, run, none)
    scale = torch.randn(L, generator=g, device=U.DEV) if scaled else None
    full, Y = U.guarded(M, N)
    B.gemm_ar_lora(plan, X_r, W_r, A_r, Bm, adapter, Y, ws, scale=scale)
    status_ok(setup)
    ref, bound = U.lora_ref(X_r, W_r, A_r, Bm, adapter, scale)
    U.close(Y, ref, bound)
    assert U.untouched(full, M, torch.ones(M, dtype=torch.bool, device=U.DEV))


def test_lora_ids_out_of_range_and_nan_of_others(setup):
    """Ids outside 0..L-1 have no adapter; an adapter of NaN reaches its rows alone."""
    plan, ws = setup
    g = U.gen(11)
    M, N, K, L, rank = 48, 264, 320, 6, 16
    X, W = U.normal(g, M, K), U.normal(g, N, K, std=K ** -0.5)
    A, Bm = U.normal(g, L, rank, K, std=K ** -0.5), U.normal(g, L, N, rank, std=rank ** -0.5)
    A[2], Bm[4] = float("nan"), float("inf")
    adapter = torch.randint(0, L, (M,), generator=g, device=U.DEV, dtype=torch.int32)
    adapter[:6] = torch.tensor([-1, L, 1 << 30, -(1 << 31), 0, 1], dtype=torch.int32, device=U.DEV)
    Y = torch.empty(M, N, dtype=torch.bfloat16, device=U.DEV)
    B.gemm_ar_lora(plan, [X], [W], [A], Bm, adapter, Y, ws)
    status_ok(setup)
    bad = (adapter == 2) | (adapter == 4)
    assert not torch.isfinite(Y[bad]).any()
    ref, bound = U.lora_ref([X], [W], [A], Bm, adapter, None)
    U.close(Y[~bad], ref[~bad], bound[~bad])


@pytest.mark.parametrize("M,L,run", [(2, 2, 1), (100, 3, 1), (600, 2, 40)])
def test_lora_weights_that_are_not_finite(setup, M, L, run):
    """Infinite and NaN weights of an adapter's B give what its products give, in its
    rows and their columns, and nothing in other rows of the tile."""
    plan, ws = setup
    g = U.gen(14 + M)
    N, K, rank = 264, 320, 16
    X, W = U.normal(g, M, K), U.normal(g, N, K, std=K ** -0.5)
    A, Bm = U.normal(g, L, rank, K, std=K ** -0.5), U.normal(g, L, N, rank, std=rank ** -0.5)
    Bm[1, 5, 3], Bm[1, 130, 0], Bm[1, 200, 9] = float("inf"), float("-inf"), float("nan")
    adapter = (torch.arange(M, device=U.DEV) // run % L).to(torch.int32)
    Y = torch.empty(M, N, dtype=torch.bfloat16, device=U.DEV)
    B.gemm_ar_lora(plan, [X], [W], [A], Bm, adapter, Y, ws)
    status_ok(setup)
    bad = torch.zeros(M, N, dtype=torch.bool, device=U.DEV)
    for n in (5, 130, 200):
        bad[adapter == 1, n] = True
    assert torch.equal(~torch.isfinite(Y), bad)
    assert torch.isnan(Y[adapter == 1, 200]).all() and torch.isinf(Y[adapter == 1, 5]).all()
    low = X.double() @ A[1].double().t()
    sign = torch.where(low[:, 3] > 0, 1.0, -1.0)[adapter == 1]
    assert torch.equal(torch.sign(Y[adapter == 1, 5].double()), sign)
    clean = Bm.clone()
    clean[1, [5, 130, 200]] = 0
    ref, bound = U.lora_ref([X], [W], [A], clean, adapter, None)
    U.close(Y[~bad], ref[~bad], bound[~bad])


def test_lora_without_adapters_is_the_projection(setup):
    """Rows of no adapter have the base sum alone, in the same bits as a call in
    which every adapter has a scale of 0."""
    plan, ws = setup
    g = U.gen(12)
    X, W = U.normal(g, 100, 512), U.normal(g, 512, 512, std=512 ** -0.5)
    A, Bm = U.normal(g, 4, 16, 512), U.normal(g, 4, 512, 16)
    Y, Z = (torch.empty(100, 512, dtype=torch.bfloat16, device=U.DEV) for _ in range(2))
    none = torch.full((100,), -1, dtype=torch.int32, device=U.DEV)
    B.gemm_ar_lora(plan, [X], [W], [A], Bm, none, Y, ws)
    B.gemm_ar_lora(plan, [X], [W], [A], Bm, none + 2, Z, ws, scale=torch.zeros(4, device=U.DEV))
    status_ok(setup)
    assert torch.equal(Y, Z)


# ---------------------------------------------------------------- streams, graphs

def test_calls_on_another_stream_and_in_a_graph(setup):
    plan, ws = setup
    g = U.gen(13)
    T, topk, E, H, I = 20, 2, 6, 256, 128
    X = U.normal(g, T, H)
    W1, W2 = U.normal(g, E, 2 * I, H, std=H ** -0.5), U.normal(g, E, H, I, std=I ** -0.5)
    ids = torch.randint(0, E, (T, topk), generator=g, device=U.DEV, dtype=torch.int32)
    weights = torch.rand(T, topk, generator=g, device=U.DEV)
    i32 = dict(dtype=torch.int32, device=U.DEV)
    bf = dict(dtype=torch.bfloat16, device=U.DEV)
    offsets, source, position = torch.empty(E + 1, **i32), torch.empty(T * topk, **i32), torch.empty(T, topk, **i32)
    mid, out, Y = torch.empty(T * topk, I, **bf), torch.empty(T * topk, H, **bf), torch.empty(T, H, **bf)

    def layer():
        B.gemm_group_route(plan, ids, E, offsets, source, position)
        B.gemm_grouped_gated(plan, X, W1, offsets, mid, ws, rows=source)
        B.gemm_grouped(plan, mid, W2, offsets, out, ws)
        B.gemm_group_combine(plan, out, position, weights, Y, base=X)

    layer()
    torch.cuda.synchronize()
    first = Y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Y.zero_()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        layer()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(Y, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    ids.copy_(ids.flip(0))   # a replay reads the routing anew
    X.copy_(X.flip(0))
    weights.copy_(weights.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    status_ok(setup)
    # Other rows share a tile now, but a row's sum over k has the same order.
    assert torch.equal(Y, first.flip(0))


def test_two_streams_at_once(setup):
    """Calls of two streams, each with a workspace of its own, in flight together."""
    plan, _ = setup
    g = U.gen(15)
    jobs = []
    for i, (M, N, K, L, rank) in enumerate([(128, 1024, 1024, 20, 32), (700, 520, 512, 3, 16)]):
        ws = B.gemm_routed_workspace_alloc(plan)
        B.gemm_routed_workspace_init(plan, ws)
        X, W = U.normal(g, M, K), U.normal(g, N, K, std=K ** -0.5)
        A, Bm = U.normal(g, L, rank, K, std=K ** -0.5), U.normal(g, L, N, rank, std=rank ** -0.5)
        a = adapters(g, M, L, 1, 0.1)
        We = U.normal(g, 4, N, K, std=K ** -0.5)
        off = U.offsets_of([M // 2, 0, M // 3, M - M // 2 - M // 3])
        Y, Z = (torch.empty(M, N, dtype=torch.bfloat16, device=U.DEV) for _ in range(2))
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        calls = [B.prepare_ar_lora(plan, [X], [W], [A], Bm, a, Y, ws, stream=stream),
                 B.prepare_grouped(plan, X, We, off, Z, ws, stream=stream)]
        jobs.append((calls, Y, Z, stream, ws))
    alone = []
    for calls, Y, Z, stream, ws in jobs:
        for c in calls:
            c()
        torch.cuda.synchronize()
        alone.append((Y.clone(), Z.clone()))
    for _ in range(20):
        for k in range(2):
            for calls, *_ in jobs:
                calls[k]()
    torch.cuda.synchronize()
    for (calls, Y, Z, stream, ws), (y, z) in zip(jobs, alone):
        B.gemm_shard_check_status(plan, ws)
        assert torch.equal(Y, y) and torch.equal(Z, z)


@pytest.mark.parametrize("tokens,graph", [(1, False), (33, False), (300, True)])
def test_the_example_runs_them_together(tokens, graph):
    import importlib.util
    import os
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", at)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    assert mod.main(["--tokens", str(tokens)] + (["--graph"] if graph else [])) == 0
