"""Host checks of the routed projections' entry points, without a GPU: refusals
come before anything is launched, with a status and a message; valid arguments
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


BASE = dict(E=8, M=100, N=512, K=256, offsets=0x1000, T=100, X=0x10000, rows=0, W=0x20000, Y=0x30000,
            ws=WS, ws_bytes=None)


def grouped(host, gated=False, **change):
    lib, plan = host
    a = {**BASE, **change}
    size = B.gemm_routed_workspace_size(plan) if a["ws_bytes"] is None else a["ws_bytes"]
    fn = lib.gemm_grouped_gated if gated else lib.gemm_grouped
    return fn(change.get("plan", plan.handle), a["E"], a["M"], a["N"], a["K"], vp(a["offsets"]), a["T"],
              vp(a["X"]), vp(a["rows"]), vp(a["W"]), vp(a["Y"]), vp(a["ws"]), size, None)


@pytest.mark.parametrize("gated", [False, True])
def test_grouped_refusals(host, gated):
    bad = [
        (dict(plan=None), "plan"), (dict(E=0), "E=0"), (dict(E=1025), "E=1025"), (dict(M=-1), "M=-1"),
        (dict(M=4097, T=4097), "max_M"), (dict(N=0), "N=0"), (dict(N=12), "N=12"), (dict(N=8200), "max_N"),
        (dict(K=4), "K=4"), (dict(K=8200), "max_K"), (dict(T=99), "M rows"), (dict(T=0, rows=0x500), "one row"),
        (dict(offsets=0), "offsets"), (dict(offsets=0x1002), "4-byte"), (dict(rows=0x501), "4-byte"),
        (dict(W=0), "W must"), (dict(W=0x20008), "16-byte"), (dict(X=0), "X and Y"), (dict(Y=0x30004), "16-byte"),
    ]
    for change, part in bad:
        refused(grouped(host, gated, **change), B.GSR_ERR_INVALID_VALUE, part)
    for change, part in [(dict(ws=0), "NULL"), (dict(ws=WS + 64), "256-byte"), (dict(ws_bytes=4096), "too small")]:
        refused(grouped(host, gated, **change), B.GSR_ERR_WORKSPACE, part)
    refused(grouped(host, gated), B.GSR_ERR_UNSUPPORTED, "arguments are valid")
    refused(grouped(host, gated, T=7, rows=0x500), B.GSR_ERR_UNSUPPORTED, "arguments are valid")
    assert grouped(host, gated, M=0, T=0, X=0, Y=0) == B.GSR_OK


def test_route_refusals(host):
    lib, plan = host

    def call(T=10, topk=4, E=8, ids=0x1000, id_bytes=4, offsets=0x2000, source=0x3000, position=0x4000):
        return lib.gemm_group_route(plan.handle, T, topk, E, vp(ids), id_bytes, vp(offsets), vp(source),
                                    vp(position), None)
    for change, part in [
            (dict(E=0), "E=0"), (dict(E=1025), "E=1025"), (dict(topk=0), "topk"), (dict(topk=129), "topk"),
            (dict(T=-1), "T=-1"), (dict(T=1025), "max_M"), (dict(id_bytes=2), "id_bytes"), (dict(offsets=0), "offsets"),
            (dict(ids=0), "NULL"), (dict(source=0), "NULL"), (dict(position=0x4001), "aligned"),
            (dict(ids=0x1004, id_bytes=8), "aligned")]:
        refused(call(**change), B.GSR_ERR_INVALID_VALUE, part)
    refused(call(), B.GSR_ERR_UNSUPPORTED, "arguments are valid")
    refused(call(T=0, ids=0, source=0, position=0), B.GSR_ERR_UNSUPPORTED, "arguments are valid")
    assert lib.gemm_group_route(None, 1, 1, 1, None, 4, None, None, None, None) == B.GSR_ERR_INVALID_VALUE


def test_combine_refusals(host):
    lib, plan = host

    def call(T=10, topk=4, H=64, z_rows=40, Z=0x1000, position=0x2000, weights=0x3000, base=0, Y=0x4000):
        return lib.gemm_group_combine(plan.handle, T, topk, H, z_rows, vp(Z), vp(position), vp(weights), vp(base),
                                      vp(Y), None)
    for change, part in [
            (dict(topk=0), "topk"), (dict(topk=129), "topk"), (dict(T=-1), "T=-1"), (dict(T=4097), "max_M"),
            (dict(H=12), "H=12"), (dict(H=8200), "max_N"), (dict(z_rows=-1), "z_rows"), (dict(Z=0), "NULL"),
            (dict(position=0), "NULL"), (dict(weights=0), "NULL"), (dict(Y=0), "NULL"), (dict(Y=0x4008), "16-byte"),
            (dict(base=0x5004), "16-byte"), (dict(weights=0x3001), "4-byte")]:
        refused(call(**change), B.GSR_ERR_INVALID_VALUE, part)
    refused(call(), B.GSR_ERR_UNSUPPORTED, "arguments are valid")
    refused(call(Z=0, z_rows=0), B.GSR_ERR_UNSUPPORTED, "arguments are valid")
    assert call(T=0, Z=0, position=0, weights=0, Y=0) == B.GSR_OK


def test_lora_refusals(host):
    lib, plan = host
    size = B.gemm_routed_workspace_size(plan)

    def call(M=10, N=64, K_r=(64, 72), X=None, W=None, A=None, L=4, rank=16, Bm=0x9000, adapter=0xa000, scale=0,
             Y=0xb000, ws=WS, ws_bytes=size):
        R = len(K_r)
        arr = lambda v, at: (ctypes.c_void_p * R)(*(v or [at + 0x1000 * r for r in range(R)]))  # noqa: E731
        return lib.gemm_ar_lora(plan.handle, M, N, R, (ctypes.c_int64 * R)(*K_r), arr(X, 0x100000),
                                arr(W, 0x200000), L, rank, arr(A, 0x300000), vp(Bm), vp(adapter), vp(scale), vp(Y),
                                vp(ws), ws_bytes, None)
    for change, part in [
            (dict(M=-1), "M must"), (dict(M=4097), "max_M"), (dict(N=12), "N must"), (dict(K_r=(64, 60)), "K_r[1]"),
            (dict(K_r=(8192, 8)), "max_K"), (dict(X=[0, 0x1000]), "NULL"), (dict(W=[0x1000, 0x1008]), "16-byte"),
            (dict(L=0), "L=0"), (dict(L=65537), "L=65537"), (dict(rank=0), "rank=0"), (dict(rank=12), "rank=12"),
            (dict(rank=136), "rank=136"), (dict(A=[0x1000, 0]), "A_r[1]"), (dict(A=[0x1004, 0x2000]), "A_r[0]"),
            (dict(Bm=0), "B must"), (dict(Bm=0x9008), "16-byte"), (dict(adapter=0), "adapter"),
            (dict(adapter=0xa002), "4-byte"), (dict(scale=0xc001), "4-byte"), (dict(Y=0), "Y must"),
            (dict(Y=0xb008), "16-byte")]:
        refused(call(**change), B.GSR_ERR_INVALID_VALUE, part)
    for change, part in [(dict(ws=0), "NULL"), (dict(ws=WS + 16), "256-byte"), (dict(ws_bytes=size - 1), "too small")]:
        refused(call(**change), B.GSR_ERR_WORKSPACE, part)
    refused(call(), B.GSR_ERR_UNSUPPORTED, "arguments are valid")
    assert call(M=0, X=[0, 0], adapter=0, Y=0) == B.GSR_OK


def test_workspace(host):
    lib, plan = host
    assert lib.gemm_routed_workspace_size(None) == 0
    size = B.gemm_routed_workspace_size(plan)
    # two slots of 256 tokens x 256 weight rows in fp32 per pair, and the low-rank rows
    assert size >= 2 * 76 * 256 * 256 * 4 + 4096 * 128 * 2
    init = lib.gemm_routed_workspace_init
    assert init(None, vp(WS), size, None) == B.GSR_ERR_INVALID_VALUE
    refused(init(plan.handle, vp(0), size, None), B.GSR_ERR_WORKSPACE, "NULL")
    refused(init(plan.handle, vp(WS + 8), size, None), B.GSR_ERR_WORKSPACE, "256-byte")
    refused(init(plan.handle, vp(WS), size - 1, None), B.GSR_ERR_WORKSPACE, "too small")
    refused(init(plan.handle, vp(WS), size, None), B.GSR_ERR_UNSUPPORTED, "host plan")
    # a plan with more SMs than there are counters
    big = B.gemm_shard_plan_create_host(4096, 4096, 512, 512, 1)
    refused(init(big.handle, vp(WS), 1 << 40, None), B.GSR_ERR_UNSUPPORTED, "SMs")


def test_binding_refuses_wrong_tensors(host):
    """Types, shapes and devices are checked before the library is called."""
    _, plan = host
    bf, i32 = torch.bfloat16, torch.int32
    t = lambda *s, dtype=bf: torch.zeros(*s, dtype=dtype)  # noqa: E731
    cpu = dict(X=t(4, 64), W=t(2, 32, 64), offsets=t(3, dtype=i32), Y=t(4, 32))
    with pytest.raises(ValueError, match="X must be"):
        B.gemm_grouped(plan, cpu["X"], cpu["W"], cpu["offsets"], cpu["Y"], t(1))
    with pytest.raises(ValueError, match="ids must be int32 or int64"):
        B.gemm_group_route(plan, t(4, 2), 3, t(4, dtype=i32), t(8, dtype=i32), t(4, 2, dtype=i32))
    with pytest.raises(ValueError, match="Z must be"):
        B.gemm_group_combine(plan, t(4, 64), t(2, 2, dtype=i32), t(2, 2, dtype=torch.float32), t(2, 64))
    with pytest.raises(ValueError, match="same, non-zero number"):
        B.gemm_ar_lora(plan, [], [], [], t(1, 8, 8), t(0, dtype=i32), t(0, 8), t(1))
