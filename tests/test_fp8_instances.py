"""Every kernel instance of the 8-bit products by name of its tile, results whose bits do
not depend on the tiles or on the CTAs, and scales at the ends of fp32's range.

The bound of fp8_util on a sum (2^-17 of sum |x w|) at the K here and at K = 32768: a sum is
made of at most 128 additions within a block and one per block of 128 columns, so 128 + 256
roundings of at most 2^-24 each; of both signs, sqrt(384) * 2^-24 < 2^-19."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tensor_gemm_reduction_gb300 import binding as B
from tensor_gemm_reduction_gb300 import build as gbuild

import fp8_util as F

gpu = pytest.mark.gpu

# (form, weight rows of a tile), M, N, K_r
AR = [
    (("narrow", 32), 100, 1000, [640, 144]),
    (("narrow", 64), 1, 2440, [896] * 8),
    (("narrow", 64), 17, 3648, [400, 144]),
    (("narrow", 64), 65, 3000, [1008] * 3),
    (("narrow", 64), 128, 4800, [2048]),
    (("narrow", 96), 9, 7168, [640, 256]),
    (("narrow", 96), 120, 6288, [272]),
    (("narrow", 128), 5, 9000, [896] * 2),
    (("narrow", 128), 100, 19000, [640]),      # two tiles a pair
    (("narrow", 128), 128, 9600, [400, 16]),
    (("wide", 64), 129, 1000, [640]),
    (("wide", 64), 700, 1000, [640, 144]),
    (("wide", 128), 300, 4000, [400, 640]),
    (("wide", 192), 4096, 3648, [7168]),
    (("wide", 256), 600, 5000, [1040]),
    (("wide", 256), 2500, 9728, [640, 128]),
]
# ..., M_r, N, K
AG = [
    (("narrow", 32), [5, 0, 3, 20], 1000, 272),
    (("narrow", 64), [5, 0, 3], 3648, 1152),
    (("narrow", 64), [42, 1, 20, 1], 2504, 1024),
    (("narrow", 64), [16] * 8, 4000, 272),
    (("narrow", 96), [64, 30], 7000, 656),
    (("narrow", 128), [7, 0, 9, 1, 30], 9000, 656),
    (("wide", 128), [42] * 8, 3648, 1024),
    (("wide", 256), [100] * 16, 6288, 1024),
]


def name(case):
    return "-".join(map(str, case[0])) + "-" + "x".join(str(v) for v in case[1:]).replace(" ", "")


def test_the_cases_take_their_instances_and_every_instance_has_one():
    """As the library logs them for a device of 152 SMs, without a GPU."""
    gbuild.build()
    code = f"""
import ctypes
from tensor_gemm_reduction_gb300 import binding as B
p = B.gemm_shard_plan_create_host(152, 32768, 32768, 32768, 16)
lib, at = B.load_library(), (ctypes.c_void_p * 16)(*[0x1000] * 16)
for _, M, N, K_r in {AR!r}:
    lib.gemm_ar_fp8(p.handle, M, N, len(K_r), (ctypes.c_int64 * 16)(*K_r), at, at, at, at, 0x1000, 0x1000, 256, None)
for _, M_r, N, K in {AG!r}:
    lib.gemm_ag_fp8(p.handle, N, K, len(M_r), (ctypes.c_int64 * 16)(*M_r), at, at, 0x1000, 0x1000, 0x1000, 0x1000, 256, None)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, env={**os.environ, "GSR_LOG_CONFIG": "1"},
                       capture_output=True, text=True, check=True)
    lines = r.stderr.splitlines()
    assert len(lines) == len(AR + AG)
    for line, case in zip(lines, AR + AG):
        assert "form=%s tile_n=%d " % case[0] in line, (case, line)
    want = {("narrow", n) for n in (32, 64, 96, 128)} | {("wide", n) for n in (64, 128, 192, 256)}
    assert {c[0] for c in AR} == want


@pytest.fixture(scope="module")
def setup():
    gbuild.build()
    plan = B.gemm_shard_plan_create(0, 32768, 32768, 32768, 16)
    ws = B.gemm_shard_workspace_alloc(plan)
    B.gemm_shard_workspace_init(plan, ws)
    return plan, ws


def ar_inputs(seed, M, N, K_r):
    g = F.gen(seed)
    return ([F.bits8(g, M, k) for k in K_r], [F.scales(g, F.blocks(k), M) for k in K_r],
            [F.bits8(g, N, k) for k in K_r], [F.scales(g, F.blocks(N), F.blocks(k)) for k in K_r])


def ag_inputs(seed, M_r, N, K):
    g = F.gen(seed)
    return ([F.bits8(g, m, K) for m in M_r], [F.scales(g, F.blocks(K), m) for m in M_r], F.bits8(g, N, K),
            F.scales(g, F.blocks(N), F.blocks(K)))


def ar(setup, X, SX, W, SW):
    plan, ws = setup
    M, N = X[0].shape[0], W[0].shape[0]
    full, Y = F.guarded(M, N)
    B.gemm_ar_fp8(plan, X, SX, W, SW, Y, ws)
    B.gemm_shard_check_status(plan, ws)
    assert F.untouched(full, M, torch.ones(M, dtype=torch.bool, device=F.DEV))
    return Y


def ag(setup, A, SA, W, SW):
    plan, ws = setup
    M, N = sum(len(a) for a in A), W.shape[0]
    full, Y = F.guarded(M, N)
    B.gemm_ag_fp8(plan, A, SA, W, SW, Y, ws)
    B.gemm_shard_check_status(plan, ws)
    assert F.untouched(full, M, torch.ones(M, dtype=torch.bool, device=F.DEV))
    return Y


@gpu
@pytest.mark.parametrize("case", AR, ids=name)
def test_ar_in_every_instance(setup, case):
    _, M, N, K_r = case
    X, SX, W, SW = ar_inputs(M + N, M, N, K_r)
    F.close(ar(setup, X, SX, W, SW), *F.product_ref([F.rows_of(*a) for a in zip(X, SX)],
                                                    [F.weights_of(*a) for a in zip(W, SW)]))


@gpu
@pytest.mark.parametrize("case", AG, ids=name)
def test_ag_in_every_instance(setup, case):
    _, M_r, N, K = case
    A, SA, W, SW = ag_inputs(N, M_r, N, K)
    x = torch.cat([F.rows_of(*a) for a in zip(A, SA)])
    F.close(ag(setup, A, SA, W, SW), *F.product_ref([x], [F.weights_of(W, SW)]))


@pytest.fixture(scope="module")
def one_pair():
    """A plan whose calls run on one CTA pair, which then takes other tile widths."""
    gbuild.build()
    plan = B.gemm_shard_plan_create(0, 32768, 32768, 32768, 16)
    B.gemm_shard_plan_set_option(plan, B.GSR_OPT_MAX_CTAS, 2)
    ws = B.gemm_shard_workspace_alloc(plan)
    B.gemm_shard_workspace_init(plan, ws)
    return plan, ws


@gpu
@pytest.mark.parametrize("M,N,K_r", [(1, 600, [1040]), (100, 1000, [640, 144]), (64, 3648, [896] * 2), (120, 6288, [272]),
                                     (129, 1000, [640]), (300, 4000, [400, 640]), (700, 1000, [640, 144]),
                                     (1000, 3648, [1152])], ids=str)
def test_ar_has_the_same_bits_on_one_pair(setup, one_pair, M, N, K_r):
    s = ar_inputs(N, M, N, K_r)
    assert torch.equal(ar(setup, *s), ar(one_pair, *s))


@gpu
@pytest.mark.parametrize("M_r,N,K", [([5, 0, 3], 3648, 1152), ([7, 0, 9, 1, 30], 1000, 656), ([16] * 8, 4000, 272),
                                     ([42] * 8, 3648, 1024), ([300, 5, 41, 1, 1, 90], 1000, 656)], ids=str)
def test_ag_has_the_same_bits_on_one_pair(setup, one_pair, M_r, N, K):
    s = ag_inputs(N, M_r, N, K)
    assert torch.equal(ag(setup, *s), ag(one_pair, *s))


# ---------------------------------------------------------------- scales far from 1

# An instance of each kind of sums: narrow, wide in pairs, wide with 128 sums a thread.
FAR = pytest.mark.parametrize("M,N,K_r", [(40, 520, [272, 256]), (300, 4000, [400, 640]), (600, 5000, [1040])], ids=str)


@gpu
@FAR
def test_large_scales_beside_small_ones(setup, M, N, K_r):
    """Factors of 2^100 of one operand's scales and 2^-100 of the other's: the scales'
    products are the same numbers, so the result has the same bits."""
    X, SX, W, SW = ar_inputs(N, M, N, K_r)
    want = ar(setup, X, SX, W, SW)
    for r in range(len(K_r)):
        for b in range(SX[r].shape[0]):
            power = 100 if (r + b) % 2 else -100
            SX[r][b] *= 2.0 ** power
            SW[r][:, b] *= 2.0 ** -power
    assert torch.equal(ar(setup, X, SX, W, SW), want)


@gpu
@FAR
def test_scales_whose_product_passes_the_largest_number(setup, M, N, K_r):
    """The product of the two is an infinity, so the elements that use it are not finite,
    NaN where the block's sum is 0; the elements beside them are what they were."""
    X, SX, W, SW = ar_inputs(N, M, N, K_r)
    X[0].view(torch.uint8)[11, 128:256] = 0   # a row with a sum of 0
    SW[0][2, 1] = 2.0
    want = ar(setup, X, SX, W, SW)
    SW[0][2, 1] *= 2.0 ** 99                  # of columns 256 .. 383 of the result
    SX[0][1] *= 2.0 ** -99
    SX[0][1, 11] = SX[0][1, 13] = 2.0 ** 30
    Y = ar(setup, X, SX, W, SW)
    rows = torch.zeros(M, dtype=torch.bool, device=F.DEV)
    rows[11] = rows[13] = True
    assert Y[11, 256:384].isnan().all() and not Y[13, 256:384].isfinite().any()
    assert torch.equal(Y[~rows, 256:384], want[~rows, 256:384])
    assert Y[rows, :256].isfinite().all() and Y[rows, 384:].isfinite().all()


@gpu
@FAR
def test_scales_whose_product_has_few_bits_left(setup, M, N, K_r):
    """Products of scales below 2^-126 are fp32's subnormal numbers, below 2^-150 0: the
    result is that of these numbers. Every addition may be off by half the smallest number
    (2^-150) besides its relative error, the output by half of bf16's (2^-134)."""
    X, SX, W, SW = ar_inputs(N, M, N, K_r)
    ref, mag, blocks = 0.0, 0.0, 0
    for r, k in enumerate(K_r):
        SX[r] *= 2.0 ** -66
        SW[r] *= 2.0 ** -66
        for b in range(F.blocks(k)):
            sx, sw = SX[r][b].cpu().numpy(), SW[r][:, b].cpu().numpy()
            p = np.float32(sx)[:, None] * np.float32(sw)[None, :]
            assert p.dtype == np.float32 and (p < 2.0 ** -126).any()
            p = torch.from_numpy(p.astype(np.float64)).to(F.DEV).repeat_interleave(128, 1)[:, :N]
            x, w = X[r][:, 128 * b:128 * b + 128].double(), W[r][:, 128 * b:128 * b + 128].double()
            ref = ref + p * (x @ w.t())
            mag = mag + p * (x.abs() @ w.abs().t())
            blocks += 1
    Y = ar(setup, X, SX, W, SW)
    assert bool((ref.abs() > 2.0 ** -126).any())
    F.close(Y, ref, F.ROUND * ref.abs() + F.SUM * mag + (blocks + 1) * 2.0 ** -150 + 2.0 ** -134)
