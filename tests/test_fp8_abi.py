"""Host checks of the 8-bit projections, the norm and the quantisation, without a GPU:
refusals come before anything is launched, with a status and a message; valid arguments
reach the launch point of a host plan. Addresses are made up."""
import ctypes

import pytest
import torch

from tensor_gemm_reduction_gb300 import binding as B
from tensor_gemm_reduction_gb300 import build as gbuild

WS = 0x20000000


@pytest.fixture(scope="module")
def host():
    gbuild.build()
    return B.load_library(), B.gemm_shard_plan_create_host(152, 4096, 8192, 8192, 16)


def vp(x):
    return ctypes.c_void_p(x)


def refused(status, want, part):
    assert status == want, B.gsr_last_error_string()
    assert part in B.gsr_last_error_string()


def test_norm_refusals(host):
    lib, plan = host

    def call(plan=plan.handle, M=10, H=64, X=0x10000, residual=0, gamma=0x20000, eps=1e-6, total=0, Y=0x30000, Q=0,
             scale=0):
        return lib.gemm_shard_rms_norm(plan, M, H, vp(X), vp(residual), vp(gamma), eps, vp(total), vp(Y), vp(Q),
                                       vp(scale), None)
    for change, part in [
            (dict(plan=None), "plan"), (dict(M=-1), "M=-1"), (dict(M=4097), "max_M"), (dict(H=0), "H=0"),
            (dict(H=12), "H=12"), (dict(H=8200), "8192"), (dict(H=72, Q=0x40000, scale=0x50000), "16 for Q"),
            (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"), (dict(X=0), "X must"),
            (dict(Y=0), "no output"), (dict(Q=0x40000), "together"), (dict(scale=0x40000), "together"),
            (dict(X=0x10008), "16-byte"), (dict(residual=0x10004), "16-byte"), (dict(gamma=0x20002), "16-byte"),
            (dict(total=0x60008), "16-byte"), (dict(Y=0x30008), "16-byte"),
            (dict(Q=0x40008, scale=0x50000), "16-byte"), (dict(Q=0x40000, scale=0x50002), "4-byte")]:
        refused(call(**change), B.GSR_ERR_INVALID_VALUE, part)
    refused(call(), B.GSR_ERR_UNSUPPORTED, "arguments are valid")
    refused(call(Y=0, Q=0x40000, scale=0x50000, gamma=0, eps=0.0), B.GSR_ERR_UNSUPPORTED, "arguments are valid")
    assert call(M=0, X=0, Y=0) == B.GSR_OK
    wide = B.gemm_shard_plan_create_host(152, 64, 65536, 64, 1)
    refused(lib.gemm_shard_rms_norm(wide.handle, 1, 32776, vp(16), None, None, 0.0, None, vp(16), None, None, None),
            B.GSR_ERR_INVALID_VALUE, "32768")


def test_quantize_refusals(host):
    lib, plan = host

    def call(plan=plan.handle, rows=10, cols=64, block=1, X=0x10000, Q=0x20000, scale=0x30000):
        return lib.gemm_shard_quantize(plan, rows, cols, block, vp(X), vp(Q), vp(scale), None)
    for change, part in [
            (dict(plan=None), "plan"), (dict(block=0), "block_rows"), (dict(block=64), "block_rows"),
            (dict(rows=-1), "rows=-1"), (dict(rows=4097), "max_M"), (dict(rows=8193, block=128), "max_N"),
            (dict(cols=0), "cols=0"), (dict(cols=24), "cols=24"), (dict(cols=8208), "max_K"), (dict(X=0), "NULL"),
            (dict(Q=0), "NULL"), (dict(scale=0), "NULL"), (dict(X=0x10008), "16-byte"), (dict(Q=0x20008), "16-byte"),
            (dict(scale=0x30001), "4-byte")]:
        refused(call(**change), B.GSR_ERR_INVALID_VALUE, part)
    refused(call(), B.GSR_ERR_UNSUPPORTED, "arguments are valid")
    refused(call(rows=8192, block=128), B.GSR_ERR_UNSUPPORTED, "arguments are valid")
    assert call(rows=0, X=0, Q=0, scale=0) == B.GSR_OK


def pointers(v):
    return (ctypes.c_void_p * len(v))(*v)


def test_ar_fp8_refusals(host):
    lib, plan = host

    def call(plan=plan.handle, M=10, N=64, K_r=(128, 80), X=None, SX=None, W=None, SW=None, Y=0xb000, ws=WS, ws_bytes=256):
        R = len(K_r)
        arr = lambda v, at: pointers(v or [at + 0x1000 * r for r in range(R)])  # noqa: E731
        return lib.gemm_ar_fp8(plan, M, N, R, (ctypes.c_int64 * R)(*K_r), arr(X, 0x100000), arr(SX, 0x200000),
                               arr(W, 0x300000), arr(SW, 0x400000), vp(Y), vp(ws), ws_bytes, None)
    for change, part in [
            (dict(plan=None), "plan"), (dict(M=-1), "M must"), (dict(M=4097), "max_M"), (dict(N=12), "N must"),
            (dict(N=8200), "max_N"), (dict(K_r=(128, 60)), "K_r[1]"), (dict(K_r=(128, 88)), "multiple of 16"),
            (dict(K_r=(8192, 16)), "max_K"), (dict(X=[0, 0x1000]), "NULL"), (dict(W=[0x1000, 0x1008]), "16-byte"),
            (dict(SX=[0x1000, 0]), "SX_r[1]"), (dict(SX=[0x1002, 0x2000]), "SX_r[0]"), (dict(SW=[0x1000, 0]), "SW_r[1]"),
            (dict(SW=[0x1001, 0x2000]), "SW_r[0]"), (dict(Y=0), "Y must"), (dict(Y=0xb008), "16-byte")]:
        refused(call(**change), B.GSR_ERR_INVALID_VALUE, part)
    for change, part in [(dict(ws=0), "NULL"), (dict(ws=WS + 16), "256-byte"), (dict(ws_bytes=255), "too small")]:
        refused(call(**change), B.GSR_ERR_WORKSPACE, part)
    refused(call(), B.GSR_ERR_UNSUPPORTED, "arguments are valid")
    refused(call(M=4096, N=8192, K_r=(16,) * 16), B.GSR_ERR_UNSUPPORTED, "arguments are valid")
    assert call(M=0, X=[0, 0], SX=[0, 0], Y=0) == B.GSR_OK
    null = ctypes.POINTER(ctypes.c_void_p)()
    one = pointers([0x1000])
    refused(lib.gemm_ar_fp8(plan.handle, 1, 8, 1, (ctypes.c_int64 * 1)(16), one, null, one, one, vp(0x1000), vp(WS),
                            256, None), B.GSR_ERR_INVALID_VALUE, "SX_r and SW_r")


def test_ag_fp8_refusals(host):
    lib, plan = host

    def call(plan=plan.handle, N=64, K=144, M_r=(10, 0, 3), A=None, SA=None, W=0x300000, SW=0x400000, Y=0xb000, ws=WS,
             ws_bytes=256):
        R = len(M_r)
        arr = lambda v, at: pointers(v or [at + 0x1000 * r for r in range(R)])  # noqa: E731
        return lib.gemm_ag_fp8(plan, N, K, R, (ctypes.c_int64 * R)(*M_r), arr(A, 0x100000), arr(SA, 0x200000), vp(W),
                               vp(SW), vp(Y), vp(ws), ws_bytes, None)
    for change, part in [
            (dict(plan=None), "plan"), (dict(M_r=(1,) * 17), "R=17"), (dict(M_r=(10, -1)), "M_r[1]"),
            (dict(M_r=(4096, 1)), "max_M"), (dict(M_r=(1 << 62, 1 << 62, 1 << 62)), "max_M"),
            (dict(A=[0x1000, 0, 0]), "A_r[2]"), (dict(A=[0x1008, 0, 0x1000]), "A_r[0]"),
            (dict(SA=[0x1000, 0, 0]), "SA_r[2]"), (dict(SA=[0x1002, 0, 0x1000]), "SA_r[0]"), (dict(N=12), "N=12"),
            (dict(N=8200), "max_N"), (dict(K=24), "K=24"), (dict(K=8208), "max_K"), (dict(W=0), "W must"),
            (dict(W=0x300008), "16-byte"), (dict(SW=0), "SW 4-byte"), (dict(SW=0x400001), "SW 4-byte"),
            (dict(Y=0), "Y must"), (dict(Y=0xb008), "16-byte")]:
        refused(call(**change), B.GSR_ERR_INVALID_VALUE, part)
    for change, part in [(dict(ws=0), "NULL"), (dict(ws=WS + 16), "256-byte"), (dict(ws_bytes=255), "too small")]:
        refused(call(**change), B.GSR_ERR_WORKSPACE, part)
    refused(call(), B.GSR_ERR_UNSUPPORTED, "arguments are valid")
    refused(call(A=[0x1000, 0, 0x1000], SA=[0x1000, 0, 0x1000]), B.GSR_ERR_UNSUPPORTED, "arguments are valid")
    assert call(M_r=(0, 0), A=[0, 0], SA=[0, 0], Y=0) == B.GSR_OK


def test_binding_refuses_wrong_tensors(host):
    """Types, shapes and devices are checked before the library is called."""
    _, plan = host
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    f32, e4 = torch.float32, torch.float8_e4m3fn
    with pytest.raises(ValueError, match="X must be"):
        B.gemm_shard_rms_norm(plan, t(2, 64), None, 0.0, Y=t(2, 64))
    with pytest.raises(ValueError, match="X must be"):
        B.gemm_shard_quantize(plan, t(2, 64), t(2, 64, dtype=e4), t(1, 2, dtype=f32))
    with pytest.raises(ValueError, match="same, non-zero number"):
        B.gemm_ar_fp8(plan, [], [], [], [], t(0, 8), t(1))
    with pytest.raises(ValueError, match="W must be"):
        B.gemm_ag_fp8(plan, [t(2, 64, dtype=e4)], [t(1, 2, dtype=f32)], t(8, 64), t(1, 1, dtype=f32), t(2, 8), t(1))


def test_calls_are_logged():
    """One line per call that passes validation, with the instance it chose."""
    import os
    import subprocess
    import sys
    code = """
import ctypes
from tensor_gemm_reduction_gb300 import binding as B
p = B.gemm_shard_plan_create_host(152, 4096, 8192, 8192, 16)
arr = (ctypes.c_void_p * 1)(0x1000)
for M in (1, 128, 129):
    B.load_library().gemm_ar_fp8(p.handle, M, 7168, 1, (ctypes.c_int64 * 1)(7168), arr, arr, arr, arr, 0x1000, 0x1000, 256, None)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, env={**os.environ, "GSR_LOG_CONFIG": "1"},
                       capture_output=True, text=True, check=True)
    lines = r.stderr.splitlines()
    assert len(lines) == 3 and all("ar_fp8 N=7168 K=7168 R=1 kernel=fp8" in x for x in lines)
    assert "form=narrow tile_n=96 boxes=1x8" in lines[0] and "boxes=1x64" in lines[1] and "form=wide" in lines[2]


def test_norm_takes_every_finite_eps(host):
    lib, plan = host
    for eps in (0.0, 2.0 ** -149, 1.0, 3.2e38, 2.0 ** 128 - 2.0 ** 104):   # the last: the largest fp32
        refused(lib.gemm_shard_rms_norm(plan.handle, 1, 64, vp(0x1000), None, None, eps, None, vp(0x2000), None, None,
                                        None), B.GSR_ERR_UNSUPPORTED, "arguments are valid")
