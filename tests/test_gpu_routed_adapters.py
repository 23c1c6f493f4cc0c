"""AR with adapters where values are not finite: infinite weights in either CTA's
half of a weight tile, infinite activations and scales at ranks that are padded,
and both together."""
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


def call(setup, X, W, A, Bm, adapter, scale=None):
    plan, ws = setup
    full, Y = U.guarded(X[0].shape[0], W[0].shape[0])
    B.gemm_ar_lora(plan, X, W, A, Bm, adapter, Y, ws, scale=scale)
    B.gemm_shard_check_status(plan, ws)
    assert U.untouched(full, Y.shape[0], torch.ones(Y.shape[0], dtype=torch.bool, device=U.DEV))
    return Y


def same_beyond_finite(Y, ref, bound):
    """NaN where the 64-bit value is NaN, the same infinity where it is infinite, and
    within the bound elsewhere."""
    finite, infinite = torch.isfinite(ref), torch.isinf(ref)
    assert torch.equal(torch.isnan(Y), torch.isnan(ref))
    assert torch.equal(Y[infinite].double(), ref[infinite])
    U.close(Y[finite], ref[finite], bound[finite])


# Columns in the first and the second half of a tile of 64 weight rows, both at its
# ends and inside, and in a last tile that is cut off.
COLUMNS = [0, 5, 31, 32, 40, 63, 130, 170, 230, 255, 256, 263]


@pytest.mark.parametrize("M,rank", [(1, 8), (1, 16), (1, 24), (1, 32), (2, 8), (2, 16), (3, 16), (2, 24), (1, 40)])
def test_infinite_weights_in_both_halves_of_a_tile(setup, M, rank):
    g = U.gen(20 + M + rank)
    N, K, L = 264, 328, 3
    X, W = U.normal(g, M, K), U.normal(g, N, K, std=K ** -0.5)
    A, Bm = U.normal(g, L, rank, K, std=K ** -0.5), U.normal(g, L, N, rank, std=rank ** -0.5)
    for i, n in enumerate(COLUMNS):
        Bm[1, n, i % rank] = (float("inf"), float("-inf"), float("nan"))[i % 3]
    scale = torch.tensor([1.5, -0.75, 2.0], device=U.DEV)
    adapter = torch.ones(M, dtype=torch.int32, device=U.DEV)
    if M > 1:
        adapter[0] = 2
    ref, bound = U.lora_ref([X], [W], [A], Bm, adapter, scale)
    same_beyond_finite(call(setup, [X], [W], [A], Bm, adapter, scale), ref, bound)


@pytest.mark.parametrize("rank", [8, 24, 40, 72, 64])
@pytest.mark.parametrize("M", [1, 2, 40, 300, 1100])
def test_infinite_activations_and_scales(setup, M, rank):
    """Ranks below their padded width. All low-rank rows are positive, so that a column
    whose weights are positive gets an infinity and not NaN."""
    g = U.gen(M + rank)
    N, K, L = 264, 136, 4
    X, W = U.normal(g, M, K).abs(), U.normal(g, N, K, std=K ** -0.5)
    A = U.normal(g, L, rank, K, std=K ** -0.5).abs()
    Bm = U.normal(g, L, N, rank, std=rank ** -0.5)
    Bm[:, ::2] = Bm[:, ::2].abs() + 2.0 ** -10
    scale = torch.tensor([0.5, float("inf"), 1.0, 0.25], device=U.DEV)
    adapter = (torch.arange(M, device=U.DEV) % (L + 1)).to(torch.int32)   # L: none
    rows = {}
    for m, a in ((0, 0), (5, 0), (M // 2, 1), (M - 2, 2), (M - 1, L)):
        if 0 <= m < M:
            rows.setdefault(m, a)
    for m, a in rows.items():
        adapter[m] = a
        if a != 1:
            X[m, 77] = float("inf")
    ref, bound = U.lora_ref([X], [W], [A], Bm, adapter, scale)
    Y = call(setup, [X], [W], [A], Bm, adapter, scale)
    assert torch.isinf(ref).any()
    same_beyond_finite(Y, ref, bound)


@pytest.mark.parametrize("M,rank", [(1, 16), (2, 16), (1, 8), (40, 16), (40, 72), (300, 24), (1100, 16)])
def test_infinite_activations_meet_infinite_weights(setup, M, rank):
    """Infinity times infinity is an infinity: columns whose infinite and finite weights
    have one sign."""
    g = U.gen(30 + M + rank)
    N, K, L = 264, 136, 3
    X, W = U.normal(g, M, K).abs(), U.normal(g, N, K, std=K ** -0.5)
    A = U.normal(g, L, rank, K, std=K ** -0.5).abs()
    Bm = U.normal(g, L, N, rank, std=rank ** -0.5).abs() + 2.0 ** -10
    Bm[:, 1::2] *= -1
    for i, n in enumerate([0, 5, 40, 63, 130, 255, 256, 263]):
        Bm[1, n, i % rank] *= float("inf")
    adapter = (torch.arange(M, device=U.DEV) % L).to(torch.int32)
    adapter[M - 1] = 1
    X[M - 1, 77] = float("inf")
    ref, bound = U.lora_ref([X], [W], [A], Bm, adapter, None)
    assert torch.isinf(ref[M - 1, [0, 5, 40, 63, 130, 255, 256, 263]]).any()
    same_beyond_finite(call(setup, [X], [W], [A], Bm, adapter), ref, bound)
