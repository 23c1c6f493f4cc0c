"""Inputs, 64-bit references and element bounds of the routed projections' tests.

Bounds. A bf16 result is within 2^-9 of its fp32 value, relatively: 2^-8 leaves
room for the second rounding's direction. A sum of K fp32 products is within
K * 2^-24 * sum |x w| at worst; rounding errors are not all of one sign, so
2^-17 * sum |x w| covers every K here (K <= 4096 has sqrt(K) * 2^-24 <= 2^-18)."""
import torch

ROUND = 2.0 ** -8
SUM = 2.0 ** -17
SENTINEL = 0x7FC1
DEV = "cuda:0"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape, std=1.0):
    return torch.empty(*shape, dtype=torch.bfloat16, device=DEV).normal_(0.0, std, generator=g)


def guarded(rows, cols):
    """An output between sentinel rows, filled with the sentinel itself."""
    full = torch.full((rows + 4, cols), SENTINEL, dtype=torch.int16, device=DEV)
    return full, full.view(torch.bfloat16)[2:2 + rows]


def untouched(full, rows, written):
    """Every row but those in the mask `written` still holds the sentinel."""
    keep = torch.ones(rows + 4, dtype=torch.bool, device=DEV)
    keep[2:2 + rows] = ~written
    return bool((full[keep] == SENTINEL).all())


def offsets_of(counts):
    o = torch.zeros(len(counts) + 1, dtype=torch.int32)
    o[1:] = torch.tensor(counts).cumsum(0)
    return o.to(DEV)


def close(y, ref, bound, what=""):
    err = (y.double() - ref).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} elements out of bound, first at "
        f"{bad.nonzero()[0].tolist()}, worst {float((err / bound).max()):.3g} of its bound")


def grouped_ref(X, W, counts, rows, gated):
    """(values, bounds) of the grouped product, group by group in 64 bits."""
    parts, bounds, at = [], [], 0
    for e, n in enumerate(counts):
        i = torch.arange(at, at + n, device=DEV) if rows is None else rows[at:at + n].long()
        good = (i >= 0) & (i < X.shape[0])
        x = torch.where(good[:, None], X[i.clamp(0, X.shape[0] - 1)].double(), 0.0)
        at += n
        w = W[e].double()
        z, s = x @ w.t(), SUM * (x.abs() @ w.abs().t())
        if gated:
            N = w.shape[0] // 2
            g, u, sg, su = z[:, :N], z[:, N:], s[:, :N], s[:, N:]
            act = g * torch.sigmoid(g)
            z = act * u
            # |silu'| < 1.1; the fast exponential is within a few 2^-22 of itself.
            s = 1.1 * sg * u.abs() + act.abs() * su + 2.0 ** -18 * (1 + g.abs()) * z.abs()
        parts.append(z)
        bounds.append(ROUND * z.abs() + s + 1e-30)
    return torch.cat(parts), torch.cat(bounds)


def lora_ref(X_r, W_r, A_r, B, adapter, scale):
    ref = sum(x.double() @ w.double().t() for x, w in zip(X_r, W_r))
    bound = SUM * sum(x.double().abs() @ w.double().abs().t() for x, w in zip(X_r, W_r))
    for a in range(B.shape[0]):
        t = (adapter == a).nonzero()[:, 0]
        if not t.numel():
            continue
        s = 1.0 if scale is None else float(scale[a])
        low = s * sum(x[t].double() @ A[a].double().t() for x, A in zip(X_r, A_r))
        tol = abs(s) * SUM * sum(x[t].double().abs() @ A[a].double().abs().t() for x, A in zip(X_r, A_r))
        b = B[a].double()
        ref[t] += low @ b.t()
        # the low-rank rows' own rounding to bf16 (2^-8), their sums, and this product's
        bound[t] += (ROUND * low.abs() + tol) @ b.abs().t() + SUM * (low.abs() @ b.abs().t())
    return ref, bound + ROUND * ref.abs() + 1e-30


def route_ref(ids, E):
    """The route by a plain loop over the entries (host)."""
    T, topk = ids.shape
    flat = ids.reshape(-1).tolist()
    lists = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            lists[e].append(i)
    offsets, source, position = [0], [], [-1] * len(flat)
    for rows in lists:
        for i in rows:
            position[i] = len(source)
            source.append(i // topk)
        offsets.append(len(source))
    source += [-1] * (len(flat) - len(source))
    i32 = torch.int32
    return (torch.tensor(offsets, dtype=i32), torch.tensor(source, dtype=i32),
            torch.tensor(position, dtype=i32).view(T, topk))
