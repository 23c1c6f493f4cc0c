"""Host checks of the expert layer, without a GPU: refusals come before anything is
launched, with a status and a message. Addresses are made up."""
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


def test_refusals(host):
    lib, plan = host
    size = B.gemm_routed_workspace_size(plan)

    def call(plan=plan.handle, T=10, topk=4, E=8, N=64, K=128, ids=0x1000, id_bytes=4, weights=0x2000, X=0x3000,
             up=0x4000, down=0x5000, base=0, Y=0x6000, ws=WS, ws_bytes=size):
        return lib.gemm_expert_layer(plan, T, topk, E, N, K, vp(ids), id_bytes, vp(weights), vp(X), vp(up), vp(down),
                                     vp(base), vp(Y), vp(ws), ws_bytes, None)
    for change, part in [
            (dict(plan=None), "plan"), (dict(E=0), "E=0"), (dict(E=1025), "E=1025"), (dict(topk=0), "topk"),
            (dict(topk=129), "topk"), (dict(T=-1), "T=-1"), (dict(T=65), "T=65"), (dict(T=64, topk=17), "1024"),
            (dict(N=0), "N=0"), (dict(N=12), "N=12"), (dict(N=8200), "max_N"), (dict(K=4), "K=4"), (dict(K=8200), "max_K"),
            (dict(id_bytes=2), "id_bytes"), (dict(ids=0), "NULL"), (dict(weights=0), "NULL"), (dict(X=0), "NULL"),
            (dict(Y=0), "NULL"), (dict(ids=0x1002), "aligned"), (dict(ids=0x1004, id_bytes=8), "aligned"),
            (dict(weights=0x2001), "aligned"), (dict(up=0), "W_up"), (dict(up=0x4008), "W_up"), (dict(down=0), "W_down"),
            (dict(X=0x3008), "16-byte"), (dict(base=0x7004), "16-byte"), (dict(Y=0x6002), "16-byte")]:
        refused(call(**change), B.GSR_ERR_INVALID_VALUE, part)
    for change, part in [(dict(ws=0), "NULL"), (dict(ws=WS + 16), "256-byte"), (dict(ws_bytes=size - 1), "too small")]:
        refused(call(**change), B.GSR_ERR_WORKSPACE, part)
    refused(call(), B.GSR_ERR_UNSUPPORTED, "arguments are valid")
    refused(call(T=64, topk=16, E=1024, N=8192, K=8192), B.GSR_ERR_UNSUPPORTED, "arguments are valid")
    assert call(T=0, ids=0, weights=0, X=0, Y=0) == B.GSR_OK
    small = B.gemm_shard_plan_create_host(152, 39, 8192, 8192, 1)
    refused(call(plan=small.handle), B.GSR_ERR_INVALID_VALUE, "max_M=39")
    # either width is an output's as well as a reduction's
    narrow = B.gemm_shard_plan_create_host(152, 64, 64, 8192, 1)
    refused(call(plan=narrow.handle), B.GSR_ERR_INVALID_VALUE, "K=128")
    short = B.gemm_shard_plan_create_host(152, 64, 8192, 56, 1)
    refused(call(plan=short.handle, K=56), B.GSR_ERR_INVALID_VALUE, "N=64")


def test_workspace_holds_the_rows_between_the_products(host):
    _, plan = host
    few = B.gemm_shard_plan_create_host(152, 1024, 8192, 8192, 16)
    wide = B.gemm_shard_plan_create_host(152, 1024, 16384, 8192, 16)
    assert B.gemm_routed_workspace_size(wide) - B.gemm_routed_workspace_size(few) == 2 * 1024 * 8192 * 2


def test_binding_refuses_wrong_tensors(host):
    _, plan = host
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    with pytest.raises(ValueError, match="X must be"):
        B.gemm_expert_layer(plan, t(2, 64), t(2, 3, dtype=torch.int32), t(2, 3, dtype=torch.float32), t(4, 16, 64),
                            t(4, 64, 8), t(2, 64), t(1))


@pytest.mark.parametrize("T", [8, 64], ids=["in two", "routed"])
def test_widths_too_large_for_the_products_are_refused_before_a_launch(host, T):
    """A matrix that the layer's own products refuse is refused by the layer, by its two
    kernels as by the routed ones, which would have written the workspace by then."""
    lib, _ = host
    side = 1 << 19
    plan = B.gemm_shard_plan_create_host(152, 4096, 2 * side, 2 * side, 1)
    size = B.gemm_routed_workspace_size(plan)

    def call(N, K):
        return lib.gemm_expert_layer(plan.handle, T, 8, 8, N, K, vp(0x1000), 4, vp(0x2000), vp(0x3000), vp(0x4000),
                                     vp(0x5000), None, vp(0x6000), vp(WS), size, None)
    for N, K in [(side, side), (2 * side, side // 8), (8, 2 * side), (2 * side, 8)]:
        grouped = [fn(plan.handle, 8, 8 * T, n, k, vp(0x1000), 8 * T, vp(0x10000), None, vp(0x20000), vp(0x30000), vp(WS),
                      size, None) for fn, n, k in ((lib.gemm_grouped_gated, N, K), (lib.gemm_grouped, K, N))]
        if N * K * 2 < 1 << 38:
            assert grouped == [B.GSR_ERR_UNSUPPORTED] * 2
            refused(call(N, K), B.GSR_ERR_UNSUPPORTED, "arguments are valid")
        else:
            assert B.GSR_ERR_INVALID_VALUE in grouped
            refused(call(N, K), B.GSR_ERR_INVALID_VALUE, "too large a matrix")
