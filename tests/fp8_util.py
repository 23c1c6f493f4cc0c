"""Inputs, 64-bit references and element bounds of the 8-bit projections' tests, on any
device.

Bounds. Rounding to bf16 is within 2^-8 of the value (half a step of 8 bits), to e4m3
within 2^-4 of it or 2^-10 (half of the smallest step). The products of e4m3 values are
exact in fp32; a sum of K of them is within 2^-17 * sum |x w| of the exact one for every
K here (errors of both signs: sqrt(K) * 2^-24 <= 2^-17 up to K = 16384), its scales and
their product included. The norm's factor comes from a sum of H squares in fp32, all
positive, whose terms meet in at most 32 + 10 + 32 additions of 2^-24 each, and its
value goes through five more roundings: within 2^-16 of itself."""
import torch

from routed_util import SENTINEL, close, guarded, untouched  # noqa: F401

ROUND, SUM, E4M3_ROUND, E4M3_LEAST = 2.0 ** -8, 2.0 ** -17, 2.0 ** -4, 2.0 ** -10
NORM = 2.0 ** -16
TINY = 2.0 ** -126
DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape, std=1.0):
    return torch.empty(*shape, dtype=torch.bfloat16, device=DEV).normal_(0.0, std, generator=g)


def blocks(n):
    return -(-n // 128)


def bits8(g, rows, cols):
    """e4m3 values of every finite kind, small ones more often."""
    x = torch.empty(rows, cols, device=DEV).normal_(0.0, 2.0, generator=g).exp_()
    sign = torch.randint(0, 2, (rows, cols), generator=g, device=DEV) * 2 - 1
    return (x * sign).clamp_(-448, 448).to(E4M3)


def scales(g, *shape):
    """Any positive factors, over three orders of magnitude, no powers of two."""
    return torch.empty(*shape, device=DEV).uniform_(-3.5, 3.5, generator=g).exp_() / 64


def rows_of(q, s):
    """What rows of e4m3 stand for, in 64 bits (s: column blocks x rows)."""
    return q.double() * s.double().t().repeat_interleave(128, 1)[:, :q.shape[1]]


def weights_of(q, s):
    """What weights stand for, in 64 bits (s: row blocks x column blocks)."""
    return q.double() * s.double().repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]


def product_ref(xs, ws):
    """(values, bounds) of sum_r x_r . w_r^T for operands in 64 bits."""
    ref = sum(x @ w.t() for x, w in zip(xs, ws))
    mag = sum(x.abs() @ w.abs().t() for x, w in zip(xs, ws))
    return ref, ROUND * ref.abs() + SUM * mag + 1e-30


def norm_ref(X, residual, gamma, eps):
    """(h, y) in 64 bits."""
    h = X.double()
    if residual is not None:
        h = h + residual.double()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    return h, y if gamma is None else y * gamma.double()


def groups_of(v, rows):
    """v padded with zeros, as (row groups, rows, column blocks, 128)."""
    n, k = -(-v.shape[0] // rows) * rows, blocks(v.shape[1]) * 128
    v = torch.nn.functional.pad(v, (0, k - v.shape[1], 0, n - v.shape[0]))
    return v.view(n // rows, rows, k // 128, 128)


def scale_ref(v, rows):
    return (groups_of(v, rows).abs().amax((1, 3)) / 448).clamp_min(TINY)


def check_8_bits(q, s, y, what=""):
    """q and s (column blocks x rows) stand for y (64 bits, itself within NORM)."""
    want = scale_ref(y, 1)
    close(s.t(), want, (NORM + SUM) * want, what + " scale")
    wide = s.double().t().repeat_interleave(128, 1)[:, :y.shape[1]]
    close(rows_of(q, s), y, E4M3_ROUND * y.abs() + E4M3_LEAST * wide + 4 * NORM * y.abs() + 1e-37, what + " q")


def guarded_flat(n, dtype):
    """n elements between sentinel bytes: (bytes, view)."""
    size = torch.empty(0, dtype=dtype).element_size()
    raw = torch.full((n * size + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    return raw, raw[256:256 + n * size].view(dtype)


def intact(raw):
    return bool((raw[:256] == 0xA5).all()) and bool((raw[-256:] == 0xA5).all())
