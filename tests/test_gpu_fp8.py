"""The 8-bit projections, the norm and the quantisation against plain 64-bit
implementations, at the sizes where they can go wrong: rows and columns that no tile or
block divides, shards that end inside a block, empty shards, short row shards that share
a tile, values that are not finite, one workspace over many calls, graphs, streams."""
import pytest
import torch

from tensor_gemm_reduction_gb300 import binding as B
from tensor_gemm_reduction_gb300 import build as gbuild

import fp8_util as F

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def setup():
    gbuild.build()
    plan = B.gemm_shard_plan_create(0, 32768, 32768, 32768, 16)
    ws = B.gemm_shard_workspace_alloc(plan)
    B.gemm_shard_workspace_init(plan, ws)
    return plan, ws


# ---------------------------------------------------------------- norm

@pytest.mark.parametrize("M,H", [(1, 16), (3, 136), (16, 7168), (152, 7168), (153, 7168), (300, 1000), (1000, 112),
                                 (2000, 8192), (7, 8200), (400, 16384), (5, 32768)])
@pytest.mark.parametrize("res", [False, True], ids=["x", "x+residual"])
def test_norm(setup, M, H, res):
    plan, _ = setup
    g = F.gen(M + H)
    X, gamma = F.normal(g, M, H), F.normal(g, H, std=0.3) + 1
    X[:, ::97] *= 30
    R = F.normal(g, M, H, std=4) if res else None
    bits = H % 16 == 0
    full_s, S = F.guarded(M, H)
    full_y, Y = F.guarded(M, H)
    raw_q, Q = F.guarded_flat(M * H, F.E4M3)
    raw_t, T = F.guarded_flat(F.blocks(H) * M, torch.float32)
    out8 = dict(Q=Q.view(M, H), scale=T.view(-1, M)) if bits else {}
    B.gemm_shard_rms_norm(plan, X, gamma, 1e-5, residual=R, sum=S, Y=Y, **out8)
    h, y = F.norm_ref(X, R, gamma, 1e-5)
    F.close(S, h, F.ROUND * h.abs() + 1e-30, "sum")
    F.close(Y, y, (F.ROUND + F.NORM) * y.abs() + 1e-30, "y")
    if bits:
        F.check_8_bits(out8["Q"], out8["scale"], y)
    every = torch.ones(M, dtype=torch.bool, device=F.DEV)
    assert F.untouched(full_s, M, every) and F.untouched(full_y, M, every) and F.intact(raw_q) and F.intact(raw_t)


@pytest.mark.parametrize("outs", ["sum", "y", "q", "sum q", "y q"])
def test_norm_of_some_outputs_without_gamma(setup, outs):
    plan, _ = setup
    M, H = 37, 528
    X = F.normal(F.gen(1), M, H)
    bf = dict(dtype=torch.bfloat16, device=F.DEV)
    S = torch.empty(M, H, **bf) if "sum" in outs else None
    Y = torch.empty(M, H, **bf) if "y" in outs else None
    Q = torch.empty(M, H, dtype=F.E4M3, device=F.DEV) if "q" in outs else None
    T = torch.empty(F.blocks(H), M, device=F.DEV) if "q" in outs else None
    B.gemm_shard_rms_norm(plan, X, None, 0.0, sum=S, Y=Y, Q=Q, scale=T)
    _, y = F.norm_ref(X, None, None, 0.0)
    if S is not None:
        assert torch.equal(S, X)
    if Y is not None:
        F.close(Y, y, (F.ROUND + F.NORM) * y.abs())
    if Q is not None:
        F.check_8_bits(Q, T, y)


@pytest.mark.parametrize("M,H", [(16, 7168), (1000, 7168), (3, 20000)])
def test_norm_in_place(setup, M, H):
    """sum over the residual and Y over X, or the other way around, give the same bits."""
    plan, _ = setup
    g = F.gen(2)
    X, R, gamma = F.normal(g, M, H), F.normal(g, M, H), F.normal(g, H)
    S, Y = torch.empty_like(X), torch.empty_like(X)
    B.gemm_shard_rms_norm(plan, X, gamma, 1e-6, residual=R, sum=S, Y=Y)
    for swap in (False, True):
        x, r = X.clone(), R.clone()
        B.gemm_shard_rms_norm(plan, x, gamma, 1e-6, residual=r, sum=x if swap else r, Y=r if swap else x)
        assert torch.equal(x, S if swap else Y) and torch.equal(r, Y if swap else S)


def test_norm_of_rows_that_are_not_finite(setup):
    """NaN and infinity stay in their rows; a row of zeros is zero with the least scale."""
    plan, _ = setup
    M, H = 300, 1040
    X = F.normal(F.gen(3), M, H)
    clean = X.clone()
    X[5, 7], X[6, 1039], X[299, 0] = float("nan"), float("inf"), float("-inf")
    X[9] = 0
    out = []
    for x in (X, clean):
        Y = torch.empty_like(x)
        Q, T = torch.empty(M, H, dtype=F.E4M3, device=F.DEV), torch.empty(9, M, device=F.DEV)
        B.gemm_shard_rms_norm(plan, x, None, 1e-6, Y=Y, Q=Q, scale=T)
        out.append((Y, Q.view(torch.uint8), T.t()))
    odd = [5, 6, 9, 299]
    same = [i for i in range(M) if i not in odd]
    for a, b in zip(*out):
        assert torch.equal(a[same], b[same])
    Y, Q, T = out[0]
    assert Y[5].isnan().all() and T[5].isnan().all()
    # inf * (1 / inf) is NaN, a finite value's 0
    assert Y[6, 1039].isnan() and not Y[6, :1039].any() and T[6, 8].isnan()
    assert Y[299, 0].isnan() and T[299, 0].isnan()
    assert not Y[9].any() and not Q[9].any() and (T[9] == F.TINY).all()


# ---------------------------------------------------------------- quantisation

@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 7168), (3, 144), (129, 128), (333, 1008), (4096, 896), (20000, 272)])
@pytest.mark.parametrize("block", [1, 128])
def test_quantize(setup, rows, cols, block):
    """The scales and the 8 bits are those of the documented formula in fp32, bit for bit."""
    plan, _ = setup
    g = F.gen(rows)
    X = F.normal(g, rows, cols) * torch.empty(rows, 1, device=F.DEV).normal_(0, 3, generator=g).exp_().bfloat16()
    X[rows // 2] = 0
    X[0, :16] = 1e-39   # below the least scale's range
    raw_q, Q = F.guarded_flat(rows * cols, F.E4M3)
    shape = (F.blocks(cols), rows) if block == 1 else (F.blocks(rows), F.blocks(cols))
    raw_s, S = F.guarded_flat(shape[0] * shape[1], torch.float32)
    Q, S = Q.view(rows, cols), S.view(shape)
    B.gemm_shard_quantize(plan, X, Q, S, block_rows=block)
    v = F.groups_of(X.float(), block)
    most = v.abs().amax((1, 3))
    # (By a tensor: a division by a number is a product with its rounded reciprocal.)
    scale = (most / torch.full_like(most, 448)).clamp_min(F.TINY)
    want = (v * (1 / scale)[:, None, :, None]).clamp(-448, 448).to(F.E4M3)
    want = want.view(v.shape[0] * block, v.shape[2] * 128)[:rows, :cols]
    assert torch.equal(S, scale.t() if block == 1 else scale)
    assert torch.equal(Q.view(torch.uint8), want.contiguous().view(torch.uint8))
    assert F.intact(raw_q) and F.intact(raw_s)


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_of_values_that_are_not_finite(setup, block):
    plan, _ = setup
    X = F.normal(F.gen(4), 200, 400)
    X[3, 130], X[150, 2] = float("nan"), float("-inf")
    Q = torch.empty(200, 400, dtype=F.E4M3, device=F.DEV)
    S = torch.empty((4, 200) if block == 1 else (2, 4), device=F.DEV)
    B.gemm_shard_quantize(plan, X, Q, S, block_rows=block)
    at = S[1, 3] if block == 1 else S[0, 1]
    inf = S[0, 150] if block == 1 else S[1, 0]
    assert at.isnan() and inf == float("inf") and int((~S.isfinite()).sum()) == 2
    v = F.rows_of(Q, S) if block == 1 else F.weights_of(Q, S)
    odd = torch.zeros(200, 400, dtype=torch.bool, device=F.DEV)
    if block == 1:
        odd[3, 128:256] = odd[150, :128] = True
    else:
        odd[:128, 128:256] = odd[128:, :128] = True
    assert torch.equal(v.isnan(), odd)


# ---------------------------------------------------------------- products

def ar_inputs(g, M, N, K_r):
    X = [F.bits8(g, M, k) for k in K_r]
    W = [F.bits8(g, N, k) for k in K_r]
    SX = [F.scales(g, F.blocks(k), M) for k in K_r]
    SW = [F.scales(g, F.blocks(N), F.blocks(k)) for k in K_r]
    return X, SX, W, SW


def ar_ref(X, SX, W, SW):
    return F.product_ref([F.rows_of(*a) for a in zip(X, SX)], [F.weights_of(*a) for a in zip(W, SW)])


SHARDS = [[16], [128], [400], [144, 16, 640], [896] * 3, [128, 256, 1024]]


@pytest.mark.parametrize("M", [1, 7, 9, 64, 65, 128, 129, 200, 257, 700])
@pytest.mark.parametrize("N", [8, 136, 1000])
@pytest.mark.parametrize("K_r", SHARDS, ids=lambda k: "-".join(map(str, k)))
def test_ar(setup, M, N, K_r):
    plan, ws = setup
    X, SX, W, SW = ar_inputs(F.gen(M + N + len(K_r)), M, N, K_r)
    full, Y = F.guarded(M, N)
    B.gemm_ar_fp8(plan, X, SX, W, SW, Y, ws)
    B.gemm_shard_check_status(plan, ws)
    ref, bound = ar_ref(X, SX, W, SW)
    F.close(Y, ref, bound)
    assert F.untouched(full, M, torch.ones(M, dtype=torch.bool, device=F.DEV))


@pytest.mark.parametrize("M,N,K_r", [(1, 7168, [896] * 8), (128, 7168, [896] * 8), (100, 20000, [512]), (1367, 6288, [1008] * 3),
                                     (4096, 3648, [7168]), (600, 31992, [144] * 16), (64, 264, [32768]),
                                     # weight tiles of 128, 192 and 256 rows, one or many a pair
                                     (200, 9000, [896] * 2), (300, 4000, [400, 640]), (256, 7168, [1792] * 4), (129, 5000, [1040]),
                                     (512, 7168, [896] * 3), (1000, 7168, [1008]), (2000, 4864, [272]), (2500, 9728, [640, 128])])
def test_ar_larger(setup, M, N, K_r):
    plan, ws = setup
    X, SX, W, SW = ar_inputs(F.gen(M), M, N, K_r)
    full, Y = F.guarded(M, N)
    B.gemm_ar_fp8(plan, X, SX, W, SW, Y, ws)
    B.gemm_shard_check_status(plan, ws)
    ref, bound = ar_ref(X, SX, W, SW)
    F.close(Y, ref, bound)
    assert F.untouched(full, M, torch.ones(M, dtype=torch.bool, device=F.DEV))


@pytest.mark.parametrize("M,N", [(100, 1000), (700, 1000)])
def test_ar_on_few_ctas(M, N):
    """One CTA pair walks every tile; the bits do not depend on it."""
    gbuild.build()
    X, SX, W, SW = ar_inputs(F.gen(8), M, N, [640, 144])
    out = []
    for ctas in (0, 2):
        plan = B.gemm_shard_plan_create(0, 1024, 1024, 1024, 2)
        B.gemm_shard_plan_set_option(plan, B.GSR_OPT_MAX_CTAS, ctas)
        ws = B.gemm_shard_workspace_alloc(plan)
        B.gemm_shard_workspace_init(plan, ws)
        out.append(torch.empty(M, N, dtype=torch.bfloat16, device=F.DEV))
        B.gemm_ar_fp8(plan, X, SX, W, SW, out[-1], ws)
        B.gemm_shard_check_status(plan, ws)
    ref, bound = ar_ref(X, SX, W, SW)
    F.close(out[0], ref, bound)
    F.close(out[1], ref, bound)


ROWS = [[5], [1, 0, 3], [0, 0, 7, 0], [42] * 8, [16] * 8, [17] * 8, [64, 64], [64] * 5, [100, 28, 130], [128, 256, 0, 128],
        [1, 700], [300, 5, 41, 1, 1, 90], [192] * 4, [1000, 17]]


@pytest.mark.parametrize("M_r", ROWS, ids=lambda m: "-".join(map(str, m)))
@pytest.mark.parametrize("N,K", [(8, 16), (264, 1152), (1000, 656)])
def test_ag(setup, M_r, N, K):
    plan, ws = setup
    g = F.gen(sum(M_r) + N)
    A = [F.bits8(g, m, K) for m in M_r]
    SA = [F.scales(g, F.blocks(K), m) for m in M_r]
    W, SW = F.bits8(g, N, K), F.scales(g, F.blocks(N), F.blocks(K))
    M = sum(M_r)
    full, Y = F.guarded(M, N)
    B.gemm_ag_fp8(plan, A, SA, W, SW, Y, ws)
    B.gemm_shard_check_status(plan, ws)
    x = torch.cat([F.rows_of(*a) for a in zip(A, SA)])
    ref, bound = F.product_ref([x], [F.weights_of(W, SW)])
    F.close(Y, ref, bound)
    assert F.untouched(full, M, torch.ones(M, dtype=torch.bool, device=F.DEV))


@pytest.mark.parametrize("M_r,N,K", [([42] * 8, 3648, 1792), ([100] * 16, 6288, 1024), ([33] * 16, 6288, 1024),
                                     ([1024] * 8, 6288, 640), ([40, 0, 1, 300] * 4, 5000, 1552), ([8] * 16, 7168, 896)],
                         ids=lambda v: "-".join(map(str, v)) if isinstance(v, list) else str(v))
def test_ag_larger(setup, M_r, N, K):
    test_ag(setup, M_r, N, K)


def test_products_of_no_rows(setup):
    plan, ws = setup
    g = F.gen(9)
    X, SX, W, SW = ar_inputs(g, 0, 64, [128])
    B.gemm_ar_fp8(plan, X, SX, W, SW, torch.empty(0, 64, dtype=torch.bfloat16, device=F.DEV), ws)
    B.gemm_ag_fp8(plan, X * 2, SX * 2, W[0], SW[0], torch.empty(0, 64, dtype=torch.bfloat16, device=F.DEV), ws)
    B.gemm_shard_check_status(plan, ws)


@pytest.mark.parametrize("M,N", [(40, 520), (300, 520)])
def test_values_that_are_not_finite_stay_where_they_are_used(setup, M, N):
    """NaN in an element and in a scale, infinite scales: the rows and columns that use
    them are not finite, every other keeps its bits."""
    plan, ws = setup
    X, SX, W, SW = ar_inputs(F.gen(11), M, N, [300 // 16 * 16, 256])
    base = torch.empty(M, N, dtype=torch.bfloat16, device=F.DEV)
    B.gemm_ar_fp8(plan, X, SX, W, SW, base, ws)
    X[0].view(torch.uint8)[3, 17] = 0x7F        # e4m3 NaN
    SX[1][1, 11] = float("inf")
    W[1].view(torch.uint8)[130, 200] = 0xFF
    SW[0][4, 0] = float("nan")                  # rows 512 .. of W_0
    Y = torch.empty_like(base)
    B.gemm_ar_fp8(plan, X, SX, W, SW, Y, ws)
    B.gemm_shard_check_status(plan, ws)
    odd = torch.zeros(M, N, dtype=torch.bool, device=F.DEV)
    odd[3] = odd[11] = True
    odd[:, 130] = odd[:, 512:] = True
    assert torch.equal(Y[~odd], base[~odd])
    assert not Y[odd].isfinite().any()


def test_zero_scales_give_zeros(setup):
    plan, ws = setup
    X, SX, W, SW = ar_inputs(F.gen(12), 33, 72, [272])
    Y = torch.empty(33, 72, dtype=torch.bfloat16, device=F.DEV)
    B.gemm_ar_fp8(plan, X, [SX[0] * 0], W, SW, Y, ws)
    assert not Y.any()


@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("K_r", [[1008, 1024], [48, 1040, 2000], [16] * 16], ids=lambda k: "-".join(map(str, k)))
def test_shards_whose_rows_start_inside_a_sector(setup, M, K_r):
    """Shards of K = 16 mod 32 beside aligned ones, in one call."""
    plan, ws = setup
    X, SX, W, SW = ar_inputs(F.gen(M + len(K_r)), M, 328, K_r)
    full, Y = F.guarded(M, 328)
    B.gemm_ar_fp8(plan, X, SX, W, SW, Y, ws)
    B.gemm_shard_check_status(plan, ws)
    F.close(Y, *ar_ref(X, SX, W, SW))
    assert F.untouched(full, M, torch.ones(M, dtype=torch.bool, device=F.DEV))


def test_a_row_per_shard(setup):
    """16 row shards of no or one row: boxes of eight rows, and the empty shards among them."""
    plan, ws = setup
    g = F.gen(31)
    M_r = [1, 0, 1, 1] * 4
    A, SA = [F.bits8(g, m, 272) for m in M_r], [F.scales(g, 3, m) for m in M_r]
    W, SW = F.bits8(g, 136, 272), F.scales(g, 2, 3)
    Y = torch.empty(12, 136, dtype=torch.bfloat16, device=F.DEV)
    B.gemm_ag_fp8(plan, A, SA, W, SW, Y, ws)
    B.gemm_shard_check_status(plan, ws)
    x = torch.cat([F.rows_of(*a) for a in zip(A, SA)])
    F.close(Y, *F.product_ref([x], [F.weights_of(W, SW)]))


@pytest.mark.parametrize("M", [3, 500])
def test_waits_of_a_nanosecond(M):
    """The shortest limit that a wait can have: the call gives its result or a status, never
    a fault, and after another init the same workspace serves the same call."""
    gbuild.build()
    X, SX, W, SW = ar_inputs(F.gen(13), M, 1000, [1024, 640])
    full, Y = F.guarded(M, 1000)
    for limit in (1, 0):   # 0: the default
        plan = B.gemm_shard_plan_create(0, 1024, 1024, 2048, 2)
        B.gemm_shard_plan_set_option(plan, B.GSR_OPT_TIMEOUT_NS, limit)
        if limit:
            ws = B.gemm_shard_workspace_alloc(plan)
        B.gemm_shard_workspace_init(plan, ws)
        B.gemm_ar_fp8(plan, X, SX, W, SW, Y, ws)
        torch.cuda.synchronize()
        assert F.untouched(full, M, torch.ones(M, dtype=torch.bool, device=F.DEV))
        try:
            B.gemm_shard_check_status(plan, ws)
        except B.GsrError as e:
            assert limit and e.status == B.GSR_ERR_TIMEOUT
            continue
        F.close(Y, *ar_ref(X, SX, W, SW))


# ---------------------------------------------------------------- together

class Chain:
    """AG of 8-bit rows, quantised K-shards, AR, residual and norm, 8-bit rows again."""

    def __init__(self, plan, ws, M_r, H, N, R, seed):
        g = F.gen(seed)
        M, k = sum(M_r), N // R
        e4, f32, bf = (dict(dtype=d, device=F.DEV) for d in (F.E4M3, torch.float32, torch.bfloat16))
        self.M_r, self.R, self.k = M_r, R, k
        self.X = [F.normal(g, m, H) for m in M_r]
        self.res = F.normal(g, M, H)
        self.gamma = F.normal(g, H, std=0.2) + 1
        self.W_in, self.W_out = F.normal(g, N, H, std=H ** -0.5), [F.normal(g, H, k, std=N ** -0.5) for _ in range(R)]
        self.A = [torch.empty(m, H, **e4) for m in M_r]
        self.SA = [torch.empty(F.blocks(H), m, **f32) for m in M_r]
        self.W8, self.SW8 = torch.empty(N, H, **e4), torch.empty(F.blocks(N), F.blocks(H), **f32)
        self.O8 = [torch.empty(H, k, **e4) for _ in range(R)]
        self.SO8 = [torch.empty(F.blocks(H), F.blocks(k), **f32) for _ in range(R)]
        self.Z = torch.empty(M, N, **bf)
        self.Z_r = [torch.empty(M, k, **bf) for _ in range(R)]
        self.X8 = [torch.empty(M, k, **e4) for _ in range(R)]
        self.SX8 = [torch.empty(F.blocks(k), M, **f32) for _ in range(R)]
        self.out, self.sum = torch.empty(M, H, **bf), torch.empty(M, H, **bf)
        self.Q, self.SQ, self.y = torch.empty(M, H, **e4), torch.empty(F.blocks(H), M, **f32), torch.empty(M, H, **bf)
        B.gemm_shard_quantize(plan, self.W_in, self.W8, self.SW8, block_rows=128)
        for w, q, s in zip(self.W_out, self.O8, self.SO8):
            B.gemm_shard_quantize(plan, w, q, s, block_rows=128)
        self.calls = [B.prepare_rms_norm(plan, x, self.gamma, 1e-6, Q=a, scale=s) for x, a, s in zip(self.X, self.A, self.SA) if len(x)]
        self.calls += [B.prepare_ag_fp8(plan, self.A, self.SA, self.W8, self.SW8, self.Z, ws)]
        self.tail = [B.prepare_quantize(plan, z, q, s) for z, q, s in zip(self.Z_r, self.X8, self.SX8)]
        self.tail += [B.prepare_ar_fp8(plan, self.X8, self.SX8, self.O8, self.SO8, self.out, ws),
                      B.prepare_rms_norm(plan, self.out, self.gamma, 1e-6, residual=self.res, sum=self.sum, Y=self.y,
                                         Q=self.Q, scale=self.SQ)]

    def step(self):
        for call in self.calls:
            call()
        for r, z in enumerate(self.Z_r):
            z.copy_(self.Z[:, r * self.k:(r + 1) * self.k])
        for call in self.tail:
            call()
        return self.sum, self.y, self.Q.view(torch.uint8), self.SQ

    def check(self):
        """Each call's outputs against its own inputs."""
        for x, a, s in zip(self.X, self.A, self.SA):
            if len(x):
                F.check_8_bits(a, s, F.norm_ref(x, None, self.gamma, 1e-6)[1])
        x = torch.cat([F.rows_of(*a) for a in zip(self.A, self.SA)])
        F.close(self.Z, *F.product_ref([x], [F.weights_of(self.W8, self.SW8)]))
        F.close(self.out, *ar_ref(self.X8, self.SX8, self.O8, self.SO8))
        h, y = F.norm_ref(self.out, self.res, self.gamma, 1e-6)
        F.close(self.sum, h, F.ROUND * h.abs() + 1e-30)
        F.check_8_bits(self.Q, self.SQ, y)
        # And the whole against the same chain without quantisation: an error of at most
        # 2^-4 in every element of four operands, of random signs.
        z = torch.cat([F.norm_ref(v, None, self.gamma, 1e-6)[1] for v in self.X]) @ self.W_in.double().t()
        o = z @ torch.cat(self.W_out, 1).double().t()
        assert float((self.out.double() - o).norm() / o.norm()) < 2 * 2 ** -4


@pytest.mark.parametrize("M_r", [[1, 0, 0], [5, 5, 4], [100, 300, 77]], ids=str)
def test_a_run_of_them_eager_and_in_a_graph(setup, M_r):
    plan, ws = setup
    c = Chain(plan, ws, M_r, 1040, 1056, 3, seed=sum(M_r))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    c.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.step()
    for k in range(3):
        for x in c.X + [c.res]:
            x.copy_(torch.randn(x.shape, generator=F.gen(k), device=F.DEV))
        want = [t.clone() for t in c.step()]
        for t in c.step():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((c.sum, c.y, c.Q.view(torch.uint8), c.SQ), want):
            assert torch.equal(a, b)
    c.check()
    B.gemm_shard_check_status(plan, ws)


def test_calls_on_two_streams(setup):
    """Two chains with workspaces of their own at the same time give their own bits."""
    plan, ws = setup
    ws2 = B.gemm_shard_workspace_alloc(plan)
    B.gemm_shard_workspace_init(plan, ws2)
    chains = [Chain(plan, w, m, 1040, 2112, 2, seed=i) for i, (w, m) in enumerate([(ws, [64, 30]), (ws2, [500, 200])])]
    want = [[t.clone() for t in c.step()] for c in chains]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in chains]
    for _ in range(20):
        for c, s in zip(chains, streams):
            with torch.cuda.stream(s):
                c.step()
    torch.cuda.synchronize()
    for c, w in zip(chains, want):
        for a, b in zip((c.sum, c.y, c.Q.view(torch.uint8), c.SQ), w):
            assert torch.equal(a, b)
    for w in (ws, ws2):
        B.gemm_shard_check_status(plan, w)


def test_tensors_past_2_to_the_31(setup):
    """Offsets of rows past 32 bits: the norm's and the quantisation's last rows, an
    8-bit product's last rows of Y."""
    plan = B.gemm_shard_plan_create(0, 300000, 8192, 8192, 1)
    M, H = 270000, 8192   # 2.2e9 elements
    X = torch.empty(M, H, dtype=torch.bfloat16, device=F.DEV).normal_(generator=F.gen(5))
    Y, Q = torch.empty_like(X), torch.empty(M, H, dtype=F.E4M3, device=F.DEV)
    T = torch.empty(64, M, device=F.DEV)
    B.gemm_shard_rms_norm(plan, X, None, 1e-6, Y=Y, Q=Q, scale=T)
    at = torch.tensor([0, 1, M // 2, M - 2, M - 1], device=F.DEV)
    _, y = F.norm_ref(X[at], None, None, 1e-6)
    F.close(Y[at], y, (F.ROUND + F.NORM) * y.abs())
    F.check_8_bits(Q[at], T[:, at].contiguous(), y)
    B.gemm_shard_quantize(plan, X, Q, T)
    F.check_8_bits(Q[at], T[:, at].contiguous(), X[at].double())
    del X
    ws = B.gemm_shard_workspace_alloc(plan)
    B.gemm_shard_workspace_init(plan, ws)
    W, SW = F.bits8(F.gen(6), 8192, 8192), F.scales(F.gen(6), 64, 64)
    B.gemm_ar_fp8(plan, [Q], [T], [W], [SW], Y, ws)
    B.gemm_shard_check_status(plan, ws)
    F.close(Y[at], *F.product_ref([F.rows_of(Q[at], T[:, at])], [F.weights_of(W, SW)]))


@pytest.mark.parametrize("M,H", [(20, 1040), (200, 1040), (12, 8208)])
def test_norm_of_rows_whose_squares_leave_fp32(setup, M, H):
    """Finite rows whose squares sum up past the largest number or vanish, as documented;
    the sum is theirs, and every other row keeps its bits."""
    plan, _ = setup
    X = F.normal(F.gen(41), M, H)
    clean = X.clone()
    X[7], X[8], X[9] = (X[7].float() * 2.0 ** 83).bfloat16(), (X[8].float() * 2.0 ** -85).bfloat16(), 0
    X[8][X[8] == 0] = 2.0 ** -85
    out = []
    for x in (X, clean):
        S, Y = torch.empty_like(x), torch.empty_like(x)
        Q, T = torch.empty(M, H, dtype=F.E4M3, device=F.DEV), torch.empty(F.blocks(H), M, device=F.DEV)
        B.gemm_shard_rms_norm(plan, x, None, 0.0, sum=S, Y=Y, Q=Q, scale=T)
        assert torch.equal(S, x)
        out.append((Y, Q.view(torch.uint8), T.t()))
    rows = torch.ones(M, dtype=torch.bool, device=F.DEV)
    rows[7:10] = False
    for a, b in zip(*out):
        assert torch.equal(a[rows], b[rows])
    Y, Q, T = out[0]
    assert not Y[7].any() and not (Q[7] & 0x7F).any() and (T[7] == F.TINY).all()
    assert Y[8].isinf().all() and (T[8] == float("inf")).all()
    assert Y[9].isnan().all() and T[9].isnan().all()
