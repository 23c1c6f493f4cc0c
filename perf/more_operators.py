"""The 8-bit projections, what feeds them, and the expert layer of a few tokens, as
cases that can be measured: each case is one call of one operator, on inputs made
from a seed.

  norm      h = x + residual, y = h / sqrt(mean(h^2) + eps) * gamma, with the sum, y
            in bf16, and y in 8 bits with a scale per row and 128 columns
  quantize  a matrix in 8 bits, with a scale per row and 128 columns, or per block
            of 128 x 128
  ar_fp8    Y = sum_r X_r . W_r^T, 8-bit operands with these scales
  ag_fp8    Y = concat_r(A_r) . W^T, 8-bit operands with these scales
  layer     Y[t] = base[t] + sum_j weight[t, j] * D[e] . (silu(G[e] . x_t) * (U[e] . x_t)),
            e = ids[t, j]: a layer of experts for a few tokens

8 bits: e4m3, x ~ q * scale with scale = max|x| / 448 over the group. Scales of rows
are stored by column block (blocks x rows), scales of blocks as (row blocks x column
blocks).

With `own` false an operator is computed in its plain form (elementary torch
operations in fp32, rounded once); with `own` true by the framework's call.
`exact` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

K_MODEL = 7168          # hidden size of the framework's own configurations
SHARD = 896             # one of its eight K-shards
MOST_FLOPS = 7.3e11     # of a drawn case
MOST_WEIGHTS = 64 * 3 * SHARD * K_MODEL   # elements of a drawn case's expert weights
MAX_ROWS, MAX_N, MAX_K, MAX_SHARDS = 32768, 8192, 8192, 16
EPS, LARGEST, TINY = 1e-6, 448.0, 2.0 ** -126


def listed():
    return [
        # Between two projections of a decode step of 16 sequences: latency alone.
        dict(name="norm_decode", op="norm", M=16, H=K_MODEL, residual=True),
        # The same of the largest prefill chunk of the framework's tables: bandwidth.
        dict(name="norm_prefill", op="norm", M=32768, H=K_MODEL, residual=True),
        # One rank's attention rows before an 8-bit output projection.
        dict(name="quantize_rows", op="quantize", rows=4096, cols=SHARD, block=1),
        # A projection's weights brought to 8 bits when a model is loaded.
        dict(name="quantize_weights", op="quantize", rows=6288, cols=K_MODEL, block=128),
        # The output projection of one token: a stream of 8-bit weights.
        dict(name="ar_fp8_token", op="ar_fp8", M=1, N=K_MODEL, R=8, K_r=SHARD),
        # The same of a decode step of 128 sequences.
        dict(name="ar_fp8_decode", op="ar_fp8", M=128, N=K_MODEL, R=8, K_r=SHARD),
        # An odd number of rows, a ragged width, shards that end inside a block of scales.
        dict(name="ar_fp8_ragged", op="ar_fp8", M=1367, N=6288, R=3, K_r=1008),
        # The input projection of a few tokens left over in each of eight ranks.
        dict(name="ag_fp8_small", op="ag_fp8", M=333, N=3648, R=8, K=K_MODEL),
        # The input projection of a prefill chunk: compute bound.
        dict(name="ag_fp8_prefill", op="ag_fp8", M=8192, N=6288, R=8, K=K_MODEL),
        # The experts of one token: eight experts' weights, one row each.
        dict(name="layer_token", op="layer", T=1, topk=8, E=64, N=SHARD, K=K_MODEL, skew=0.5, drop=0.0),
        # Of a decode step of 16 sequences: nearly every expert has a row or two.
        dict(name="layer_decode", op="layer", T=16, topk=8, E=64, N=SHARD, K=K_MODEL, skew=0.5, drop=0.0),
        # Of 61 sequences of a smaller model with ragged sizes, some entries dropped.
        dict(name="layer_ragged", op="layer", T=61, topk=3, E=7, N=1000, K=1832, skew=1.0, drop=0.02),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _step(rng, lo, hi, step):
    """A multiple of `step`, mostly of no higher power of two."""
    return step * _log(rng, lo // step, hi // step)


def draw(rng):
    op = rng.choice(["norm", "quantize", "ar_fp8", "ar_fp8", "ag_fp8", "ag_fp8", "layer", "layer"])
    while True:
        if op == "norm":
            c = dict(op=op, M=_log(rng, 1, 32768), H=_step(rng, 512, 7168, 16), residual=rng.random() < 0.7)
        elif op == "quantize":
            c = dict(op=op, rows=_log(rng, 1, 16384), cols=_step(rng, 512, 7168, 16), block=rng.choice([1, 128]))
        elif op == "ar_fp8":
            R = rng.choice([1, 2, 4, 8])
            c = dict(op=op, M=_log(rng, 1, 8192), N=_step(rng, 512, 7168, 8), R=R,
                     K_r=16 * max(1, _log(rng, 512, 7168) // (16 * R)))
        elif op == "ag_fp8":
            c = dict(op=op, M=_log(rng, 1, 8192), N=_step(rng, 512, 7168, 8), R=rng.choice([1, 2, 4, 8]),
                     K=_step(rng, 512, 7168, 16))
        else:
            E = rng.choice([4, 7, 8, 16, 32, 64, 100, 128])
            c = dict(op=op, T=_log(rng, 1, 64), topk=rng.randint(1, min(8, E)), E=E, N=_step(rng, 256, 2048, 8),
                     K=_step(rng, 512, 7168, 8), skew=round(rng.uniform(0.0, 1.0), 2),
                     drop=rng.choice([0.0, 0.02, 0.3]))
            if 3 * E * c["N"] * c["K"] > MOST_WEIGHTS:
                continue
        if work(c)["flops"] <= MOST_FLOPS:
            return c


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape, std=1.0):
    return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)


def _rows(g, M, K):
    """Activations: a few columns are an order of magnitude larger, as in a trained model."""
    loud = 1.0 + 15.0 * (torch.rand(K, generator=g, device="cuda") < 0.004)
    return _normal(g, M, K).mul_(loud.to(torch.bfloat16))


def _blocks(x, rows):
    """x padded with zeros to whole groups of `rows` x 128, as (.., rows, .., 128)."""
    n, k = -(-x.shape[0] // rows) * rows, -(-x.shape[1] // 128) * 128
    if (n, k) != tuple(x.shape):
        x = torch.nn.functional.pad(x, (0, k - x.shape[1], 0, n - x.shape[0]))
    return x.view(n // rows, rows, k // 128, 128)


def _to_8_bits(x, rows):
    """x in 8 bits, and the scales of its groups (groups of rows x groups of columns)."""
    b = _blocks(x.float(), rows)
    scale = (b.abs().amax(dim=(1, 3)) / LARGEST).clamp_min(TINY)
    q = (b / scale[:, None, :, None]).clamp(-LARGEST, LARGEST).to(torch.float8_e4m3fn)
    q = q.view(b.shape[0] * rows, b.shape[2] * 128)[:x.shape[0], :x.shape[1]]
    return q.contiguous(), scale


def _activations(g, M, K):
    q, scale = _to_8_bits(_rows(g, M, K), 1)
    return q, scale.t().contiguous()


def _weights(g, N, K, fan_in):
    return _to_8_bits(_normal(g, N, K, std=fan_in ** -0.5), 128)


def _popularity(c):
    p = torch.arange(1, c["E"] + 1, dtype=torch.float64) ** -c["skew"]
    return p / p.sum()


def _route_ids(c, g):
    """topk different experts for each token, some more popular than others."""
    logits = _popularity(c).log().float().cuda()
    logits = logits[torch.randperm(c["E"], generator=g, device="cuda")]
    u = torch.rand(c["T"], c["E"], generator=g, device="cuda").clamp_(1e-20, 1.0)
    ids = (logits - (-u.log()).clamp_min(1e-30).log()).topk(c["topk"], dim=1).indices.to(torch.int32)
    if c["drop"]:
        ids = ids.masked_fill(torch.rand(c["T"], c["topk"], generator=g, device="cuda") < c["drop"], -1)
    return ids


def _shard_rows(M, R):
    """M rows over R ranks, as evenly as they go."""
    return [M // R + (r < M % R) for r in range(R)]


def _inputs(c, seed):
    g, s = _gen(seed), dict(c)
    if c["op"] == "norm":
        s["X"] = _rows(g, c["M"], c["H"])
        s["res"] = _rows(g, c["M"], c["H"]).mul_(4) if c["residual"] else None
        s["gamma"] = _normal(g, c["H"], std=0.2).add_(1)
    elif c["op"] == "quantize":
        s["X"] = _rows(g, c["rows"], c["cols"]) if c["block"] == 1 else _normal(g, c["rows"], c["cols"], std=c["cols"] ** -0.5)
    elif c["op"] == "ar_fp8":
        K = c["R"] * c["K_r"]
        x = [_activations(g, c["M"], c["K_r"]) for _ in range(c["R"])]
        w = [_weights(g, c["N"], c["K_r"], K) for _ in range(c["R"])]
        s["X_r"], s["SX_r"] = [q for q, _ in x], [t for _, t in x]
        s["W_r"], s["SW_r"] = [q for q, _ in w], [t for _, t in w]
    elif c["op"] == "ag_fp8":
        a = [_activations(g, m, c["K"]) for m in _shard_rows(c["M"], c["R"])]
        s["A_r"], s["SA_r"] = [q for q, _ in a], [t for _, t in a]
        s["W"], s["SW"] = _weights(g, c["N"], c["K"], c["K"])
    else:
        s["ids"] = _route_ids(c, g)
        s["weights"] = torch.randn(c["T"], c["topk"], generator=g, device="cuda").softmax(1)
        s["X"] = _normal(g, c["T"], c["K"])
        s["base"] = _normal(g, c["T"], c["K"])
        s["up"] = _normal(g, c["E"], 2 * c["N"], c["K"], std=c["K"] ** -0.5)
        s["down"] = _normal(g, c["E"], c["K"], c["N"], std=c["N"] ** -0.5)
    return s


# ---------------------------------------------------------------- the framework's calls

_program = {}


def _plan():
    """The plan and workspaces that a program creates once."""
    from tensor_gemm_reduction_gb300 import binding as B
    if not _program:
        plan = B.gemm_shard_plan_create(0, MAX_ROWS, MAX_N, MAX_K, MAX_SHARDS)
        ws = B.gemm_shard_workspace_alloc(plan)
        B.gemm_shard_workspace_init(plan, ws)
        routed = B.gemm_routed_workspace_alloc(plan)
        B.gemm_routed_workspace_init(plan, routed)
        _program.update(plan=plan, ws=ws, routed=routed)
    return B, _program["plan"], _program["ws"], _program["routed"]


def prepare(case, seed):
    s = _inputs(case, seed)
    dev = dict(device="cuda")
    bf16, f32, e4m3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
    if s["op"] == "norm":
        M, H = s["M"], s["H"]
        s["out"] = dict(y=torch.empty(M, H, dtype=bf16, **dev), q=torch.empty(M, H, dtype=e4m3, **dev),
                        scale=torch.empty(-(-H // 128), M, dtype=f32, **dev))
        if s["residual"]:
            s["out"]["sum"] = torch.empty(M, H, dtype=bf16, **dev)
    elif s["op"] == "quantize":
        n, k = s["rows"], s["cols"]
        groups = (-(-k // 128), n) if s["block"] == 1 else (-(-n // 128), -(-k // 128))
        s["out"] = dict(q=torch.empty(n, k, dtype=e4m3, **dev), scale=torch.empty(*groups, dtype=f32, **dev))
    elif s["op"] == "layer":
        s["out"] = torch.empty(s["T"], s["K"], dtype=bf16, **dev)
    else:
        s["out"] = torch.empty(s["M"], s["N"], dtype=bf16, **dev)
    if own:   # the call on these buffers, marshalled once, as a serving loop keeps it
        B, plan, ws, routed = _plan()
        o = s["out"]
        if s["op"] == "norm":
            s["call"] = B.prepare_rms_norm(plan, s["X"], s["gamma"], EPS, residual=s["res"], sum=o.get("sum"),
                                           Y=o["y"], Q=o["q"], scale=o["scale"])
        elif s["op"] == "quantize":
            s["call"] = B.prepare_quantize(plan, s["X"], o["q"], o["scale"], block_rows=s["block"])
        elif s["op"] == "ar_fp8":
            s["call"] = B.prepare_ar_fp8(plan, s["X_r"], s["SX_r"], s["W_r"], s["SW_r"], o, ws)
        elif s["op"] == "ag_fp8":
            s["call"] = B.prepare_ag_fp8(plan, s["A_r"], s["SA_r"], s["W"], s["SW"], o, ws)
        else:
            s["call"] = B.prepare_expert_layer(plan, s["X"], s["ids"], s["weights"], s["up"], s["down"], o, routed,
                                               base=s["base"])
    return s


def run(s):
    if own:
        s["call"]()
        return s["out"]
    return globals()["_plain_" + s["op"]](s)


# ---------------------------------------------------------------- plain forms

def _plain_norm(s):
    h = s["X"].float() if s["res"] is None else s["X"].float() + s["res"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["gamma"].float()
    q, scale = _to_8_bits(y, 1)
    out = dict(y=y.to(torch.bfloat16), q=q, scale=scale.t().contiguous())
    if s["res"] is not None:
        out["sum"] = h.to(torch.bfloat16)
    return out


def _plain_quantize(s):
    q, scale = _to_8_bits(s["X"], s["block"])
    return dict(q=q, scale=scale.t().contiguous() if s["block"] == 1 else scale)


def _values(q, scale):
    """What 8-bit rows stand for; scale: (column blocks, rows)."""
    return q.float() * scale.t().repeat_interleave(128, 1)[:, :q.shape[1]]


def _block_values(q, scale):
    """What 8-bit weights stand for; scale: (row blocks, column blocks)."""
    wide = scale.repeat_interleave(128, 1)[:, :q.shape[1]]
    return q.float() * wide.repeat_interleave(128, 0)[:q.shape[0]]


def _plain_ar_fp8(s):
    x = torch.cat(list(map(_values, s["X_r"], s["SX_r"])), 1)
    w = torch.cat(list(map(_block_values, s["W_r"], s["SW_r"])), 1)
    return (x @ w.t()).to(torch.bfloat16)


def _plain_ag_fp8(s):
    a = torch.cat(list(map(_values, s["A_r"], s["SA_r"])), 0)
    return (a @ _block_values(s["W"], s["SW"]).t()).to(torch.bfloat16)


def _plain_layer(s):
    """Every expert's products for every token, weighted with zero where it was not chosen."""
    T, E, N = s["T"], s["E"], s["N"]
    z = (s["X"].float() @ s["up"].view(E * 2 * N, -1).float().t()).view(T, E, 2 * N)
    gate, up = z[:, :, :N], z[:, :, N:]
    mine = s["ids"][:, :, None] == torch.arange(E, device="cuda", dtype=torch.int32)
    h = gate / (1 + (-gate).exp()) * up * (mine * s["weights"][:, :, None]).sum(1)[:, :, None]
    down = s["down"].transpose(0, 1).reshape(-1, E * N).float()
    return (s["base"].float() + h.view(T, E * N) @ down.t()).to(torch.bfloat16)


# ---------------------------------------------------------------- exact values

def _spread(scale, rows, shape):
    """The scales of blocks of `rows` x 128 for every element, in 64 bits."""
    i = torch.arange(shape[0], device="cuda") // rows
    j = torch.arange(shape[1], device="cuda") // 128
    return scale.double()[i][:, j]


def _exact_8_bits(y, rows):
    """y over its scale, unrounded, and the scales, group by group of 128 columns."""
    n = -(-y.shape[0] // rows)
    scale = torch.empty(n, -(-y.shape[1] // 128), dtype=torch.float64, device="cuda")
    group = torch.arange(y.shape[0], device="cuda") // rows
    for j in range(scale.shape[1]):
        most = y[:, 128 * j:128 * j + 128].abs().amax(1)
        scale[:, j] = torch.zeros(n, dtype=torch.float64, device="cuda").scatter_reduce_(0, group, most, "amax")
    scale = torch.clamp_min(scale / LARGEST, TINY)
    return y / _spread(scale, rows, y.shape), scale


def exact(case, seed):
    """The definitions in 64 bits, shard by shard and expert by expert (no shared code
    but the inputs)."""
    s = _inputs(case, seed)
    if case["op"] == "norm":
        h = s["X"].double()
        if s["res"] is not None:
            h += s["res"].double()
        y = s["gamma"].double() * h / torch.sqrt(h.square().sum(1) / case["H"] + EPS)[:, None]
        q, scale = _exact_8_bits(y, 1)
        out = dict(y=y, q=q, scale=scale.t())
        if s["res"] is not None:
            out["sum"] = h
        return out
    if case["op"] == "quantize":
        q, scale = _exact_8_bits(s["X"].double(), case["block"])
        return dict(q=q, scale=scale.t() if case["block"] == 1 else scale)
    if case["op"] == "ar_fp8":
        y = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
        for x, sx, w, sw in zip(s["X_r"], s["SX_r"], s["W_r"], s["SW_r"]):
            y += torch.mm(x.double() * _spread(sx.t(), 1, x.shape), (w.double() * _spread(sw, 128, w.shape)).t())
        return y
    if case["op"] == "ag_fp8":
        w = (s["W"].double() * _spread(s["SW"], 128, s["W"].shape)).t()
        return torch.cat([torch.mm(a.double() * _spread(sa.t(), 1, a.shape), w) for a, sa in zip(s["A_r"], s["SA_r"])])
    y = s["base"].double()
    for e in range(case["E"]):
        t, j = (s["ids"] == e).nonzero(as_tuple=True)
        if t.numel():
            z = torch.mm(s["X"][t].double(), s["up"][e].double().t())
            g, u = z.chunk(2, dim=1)
            y.index_add_(0, t, torch.mm(g * torch.sigmoid(g) * u, s["down"][e].double().t()) * s["weights"][t, j].double()[:, None])
    return y


# ---------------------------------------------------------------- work

def _active(c):
    """Expected number of experts that get a row: topk different experts a token."""
    p = _popularity(c)
    lo, hi = 0.0, 1e9   # each expert is chosen with probability 1 - exp(-z p), sum = topk
    for _ in range(200):
        z = (lo * hi) ** 0.5 if lo else hi / 2
        lo, hi = (z, hi) if float((1 - (-z * p).exp()).sum()) < c["topk"] else (lo, z)
    q = (1 - (-hi * p).exp()) * (1 - c["drop"])
    return min(float((1 - (1 - q) ** c["T"]).sum()), c["T"] * c["topk"])


def work(c):
    if c["op"] == "norm":
        M, H, r = c["M"], c["H"], c["residual"]
        return dict(bytes=M * H * (2 + 2 + 1 + (4 if r else 0)) + 2 * H + 4 * M * -(-H // 128), flops=6 * M * H)
    if c["op"] == "quantize":
        n, k = c["rows"], c["cols"]
        return dict(bytes=3 * n * k + 4 * -(-n // c["block"]) * -(-k // 128), flops=2 * n * k)
    if c["op"] in ("ar_fp8", "ag_fp8"):
        M, N = c["M"], c["N"]
        K = c["R"] * c["K_r"] if c["op"] == "ar_fp8" else c["K"]
        blocks = c["R"] * -(-c["K_r"] // 128) if c["op"] == "ar_fp8" else -(-K // 128)
        return dict(bytes=(M + N) * K + 2 * M * N + 4 * blocks * (M + -(-N // 128)), flops=2 * M * N * K)
    rows, kept = c["T"] * c["topk"], c["T"] * c["topk"] * (1 - c["drop"])
    return dict(bytes=2 * (_active(c) * 3 * c["N"] * c["K"] + 3 * c["T"] * c["K"]) + 8 * rows,
                flops=2 * kept * 3 * c["N"] * c["K"])
