"""The routed projections as cases that can be measured: each case is one call
of one operator, on inputs made from a seed.

  route    expert ids of every token -> group offsets, source rows, positions
  grouped  Y[rows of group e] = X[rows of group e] . W[e]^T, ragged groups
  gated    the same with gate and up weights: Y = silu(X . Wg^T) * (X . Wu^T),
           the rows of X gathered through the route
  combine  Y[t] = base[t] + sum_j weight[t, j] * Z[position[t, j]]
  lora     Y = sum_r X_r . W_r^T + scale[a] * (sum_r X_r . A_r[a]^T) . B[a]^T,
           every row with an adapter a of its own, or none

With `own` false an operator is computed in its plain form (elementary torch
operations in fp32, rounded once); with `own` true by the framework's call.
`exact` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

K_MODEL = 7168          # hidden size of the framework's own configurations
SHARD = 896             # one of its eight K-shards
MOST_FLOPS = 8.5e11     # of a drawn case
MOST_WEIGHTS = 64 * 2 * SHARD * K_MODEL   # elements of a drawn case's expert weights
MAX_ROWS, MAX_N, MAX_K, MAX_SHARDS = 32768 * 8, 8192, 8192, 16


def listed():
    return [
        # One decode step of 16 sequences, 8 experts each: latency alone.
        dict(name="route_decode", op="route", T=16, topk=8, E=64, skew=0.5, drop=0.0),
        # The largest prefill chunk of the framework's tables, many experts.
        dict(name="route_prefill", op="route", T=32768, topk=8, E=256, skew=0.5, drop=0.02),
        # The up projections of one token: eight experts' weights, one row each.
        dict(name="gated_token", op="gated", T=1, topk=8, E=64, N=SHARD, K=K_MODEL, skew=0.5),
        # The up projections of a prefill chunk: compute bound, uneven groups.
        dict(name="gated_prefill", op="gated", T=4096, topk=8, E=64, N=SHARD, K=K_MODEL, skew=0.5),
        # The down projections of a decode step of 16 sequences: nearly every
        # expert has a row or two, so the weights are the traffic.
        dict(name="grouped_decode", op="grouped", T=16, topk=8, E=64, N=K_MODEL, K=SHARD, skew=0.5),
        # A few large groups with a ragged width and an odd number of rows.
        dict(name="grouped_ragged", op="grouped", T=1367, topk=3, E=8, N=6288, K=1000, skew=1.0),
        # The down projections of a prefill chunk.
        dict(name="grouped_prefill", op="grouped", T=4096, topk=8, E=64, N=K_MODEL, K=SHARD, skew=0.5),
        # The experts' outputs of a decode step brought back to their tokens.
        dict(name="combine_decode", op="combine", T=16, topk=8, H=K_MODEL, base=True, drop=0.0),
        # The same of a prefill chunk: bandwidth alone.
        dict(name="combine_prefill", op="combine", T=8192, topk=8, H=K_MODEL, base=False, drop=0.02),
        # The output projection of one token that uses an adapter.
        dict(name="lora_token", op="lora", M=1, N=K_MODEL, R=8, K_r=SHARD, L=64, rank=16, run=1, none=0.0),
        # A decode step of many requests, nearly each with another adapter.
        dict(name="lora_decode", op="lora", M=128, N=K_MODEL, R=8, K_r=SHARD, L=64, rank=32, run=1, none=0.1),
        # A prefill chunk of a few requests (long runs of rows with one adapter).
        dict(name="lora_prefill", op="lora", M=4096, N=K_MODEL, R=8, K_r=SHARD, L=8, rank=64, run=500, none=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _eight(rng, lo, hi):
    """A multiple of 8 (every width and reduction length is one), mostly not of 64."""
    return 8 * _log(rng, lo // 8, hi // 8)


def draw(rng):
    op = rng.choice(["route", "grouped", "grouped", "gated", "gated", "combine", "lora", "lora"])
    while True:
        E = rng.choice([4, 7, 8, 16, 32, 64, 100, 128, 256])
        topk = rng.randint(1, min(8, E))
        skew = round(rng.uniform(0.0, 1.0), 2)
        if op == "route":
            c = dict(op=op, T=_log(rng, 1, 32768), topk=topk, E=E, skew=skew, drop=rng.choice([0.0, 0.02, 0.3]))
        elif op in ("grouped", "gated"):
            lo_n, lo_k = (512, 256) if op == "grouped" else (256, 512)
            c = dict(op=op, T=_log(rng, 1, 4096), topk=topk, E=E, N=_eight(rng, lo_n, 7168),
                     K=_eight(rng, lo_k, 7168), skew=skew)
            wide = 2 * c["N"] if op == "gated" else c["N"]
            if E * wide * c["K"] > MOST_WEIGHTS:
                continue
        elif op == "combine":
            c = dict(op=op, T=_log(rng, 1, 8192), topk=topk, H=_eight(rng, 512, 7168),
                     base=rng.random() < 0.5, drop=rng.choice([0.0, 0.02, 0.3]))
        else:
            R = rng.choice([1, 2, 4, 8])
            c = dict(op=op, M=_log(rng, 1, 4096), N=_eight(rng, 512, 7168), R=R,
                     K_r=8 * max(1, _log(rng, 512, 7168) // (8 * R)), L=rng.choice([1, 4, 8, 32, 64]),
                     rank=rng.choice([8, 16, 32, 64]), run=0, none=rng.choice([0.0, 0.1, 0.5]))
            # Decode batches mix adapters row by row; prompts bring runs of rows.
            c["run"] = 1 if c["M"] <= 256 else rng.choice([50, 200, 1000])
        if work(c)["flops"] <= MOST_FLOPS:
            return c


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape, std=1.0):
    return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)


def _popularity(c):
    p = torch.arange(1, c["E"] + 1, dtype=torch.float64) ** -c["skew"]
    return p / p.sum()


def _route_ids(c, g):
    """topk different experts for each token, some more popular than others."""
    logits = _popularity(c).log().float().cuda()
    logits = logits[torch.randperm(c["E"], generator=g, device="cuda")]
    u = torch.rand(c["T"], c["E"], generator=g, device="cuda").clamp_(1e-20, 1.0)
    ids = (logits - (-u.log()).clamp_min(1e-30).log()).topk(c["topk"], dim=1).indices.to(torch.int32)
    if c.get("drop"):
        gone = torch.rand(c["T"], c["topk"], generator=g, device="cuda") < c["drop"]
        ids = ids.masked_fill(gone, -1)
    return ids


def _layout(ids, E):
    """The route of `ids` in hand already: offsets, source rows, positions."""
    flat = ids.reshape(-1).long()
    order = torch.argsort(torch.where(flat < 0, E, flat), stable=True)
    kept = int((flat >= 0).sum())
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    source = (order // ids.shape[1]).to(torch.int32)
    source[kept:] = -1
    position = torch.full_like(flat, -1, dtype=torch.int32)
    position[order[:kept]] = torch.arange(kept, dtype=torch.int32, device="cuda")
    return offsets, source, position.view(ids.shape), counts.tolist()


def _adapters(c, g):
    """Runs of about c["run"] rows with one adapter each; a share with none."""
    runs = max(1, -(-c["M"] // c["run"]))
    a = torch.randint(0, c["L"], (runs,), generator=g, device="cuda", dtype=torch.int32)
    a = a.masked_fill(torch.rand(runs, generator=g, device="cuda") < c["none"], -1)
    length = torch.full((runs,), c["run"], device="cuda")
    if c["run"] > 1:   # ragged runs: some longer, some shorter
        length = torch.randint(c["run"] // 2, 2 * c["run"], (runs,), generator=g, device="cuda")
        length[-1] += c["M"]
    return a.repeat_interleave(length)[:c["M"]].contiguous()


def _inputs(c, seed):
    g, s = _gen(seed), dict(c)
    if c["op"] == "route":
        s["ids"] = _route_ids(c, g)
    elif c["op"] in ("grouped", "gated"):
        s["offsets"], source, _, s["counts"] = _layout(_route_ids(c, g), c["E"])
        wide = 2 * c["N"] if c["op"] == "gated" else c["N"]
        s["W"] = _normal(g, c["E"], wide, c["K"], std=c["K"] ** -0.5)
        s["rows"] = source if c["op"] == "gated" else None
        s["X"] = _normal(g, c["T"] if c["op"] == "gated" else c["T"] * c["topk"], c["K"])
    elif c["op"] == "combine":
        rows = c["T"] * c["topk"]
        s["position"] = torch.randperm(rows, generator=g, device="cuda").to(torch.int32).view(c["T"], c["topk"])
        if c["drop"]:
            gone = torch.rand(c["T"], c["topk"], generator=g, device="cuda") < c["drop"]
            s["position"] = s["position"].masked_fill(gone, -1)
        s["weights"] = torch.randn(c["T"], c["topk"], generator=g, device="cuda").softmax(1)
        s["Z"] = _normal(g, rows, c["H"])
        s["base_rows"] = _normal(g, c["T"], c["H"]) if c["base"] else None
    else:
        K = c["R"] * c["K_r"]
        s["X_r"] = [_normal(g, c["M"], c["K_r"]) for _ in range(c["R"])]
        s["W_r"] = [_normal(g, c["N"], c["K_r"], std=K ** -0.5) for _ in range(c["R"])]
        s["A_r"] = [_normal(g, c["L"], c["rank"], c["K_r"], std=K ** -0.5) for _ in range(c["R"])]
        s["B"] = _normal(g, c["L"], c["N"], c["rank"], std=c["rank"] ** -0.5)
        s["adapter"] = _adapters(c, g)
        s["scale"] = 0.25 + 0.5 * torch.rand(c["L"], generator=g, device="cuda")
    return s


# ---------------------------------------------------------------- the framework's calls

_program = {}


def _plan():
    """The plan and workspace that a program creates once."""
    from tensor_gemm_reduction_gb300 import binding as B
    if not _program:
        plan = B.gemm_shard_plan_create(0, MAX_ROWS, MAX_N, MAX_K, MAX_SHARDS)
        ws = B.gemm_routed_workspace_alloc(plan)
        B.gemm_routed_workspace_init(plan, ws)
        _program.update(plan=plan, ws=ws)
    return B, _program["plan"], _program["ws"]


def prepare(case, seed):
    s = _inputs(case, seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    if s["op"] == "route":
        rows = s["T"] * s["topk"]
        s["out"] = dict(offsets=torch.empty(s["E"] + 1, **i32), source=torch.empty(rows, **i32),
                        position=torch.empty(s["T"], s["topk"], **i32))
    elif s["op"] in ("grouped", "gated"):
        s["out"] = torch.empty(s["T"] * s["topk"], s["N"], **bf16)
    elif s["op"] == "combine":
        s["out"] = torch.empty(s["T"], s["H"], **bf16)
    else:
        s["out"] = torch.empty(s["M"], s["N"], **bf16)
    if own:   # the call on these buffers, marshalled once, as a serving loop keeps it
        B, plan, ws = _plan()
        if s["op"] == "route":
            o = s["out"]
            s["call"] = B.prepare_group_route(plan, s["ids"], s["E"], o["offsets"], o["source"], o["position"])
        elif s["op"] == "grouped":
            s["call"] = B.prepare_grouped(plan, s["X"], s["W"], s["offsets"], s["out"], ws)
        elif s["op"] == "gated":
            s["call"] = B.prepare_grouped_gated(plan, s["X"], s["W"], s["offsets"], s["out"], ws, rows=s["rows"])
        elif s["op"] == "combine":
            s["call"] = B.prepare_group_combine(plan, s["Z"], s["position"], s["weights"], s["out"],
                                                base=s["base_rows"])
        else:
            s["call"] = B.prepare_ar_lora(plan, s["X_r"], s["W_r"], s["A_r"], s["B"], s["adapter"],
                                          s["out"], ws, scale=s["scale"])
    return s


def run(s):
    if own:
        s["call"]()
        return s["out"]
    return globals()["_plain_" + s["op"]](s)


# ---------------------------------------------------------------- plain forms

def _plain_route(s):
    """A stable counting sort by one-hot sums (ids of -1 belong to no group)."""
    flat = s["ids"].reshape(-1)
    hot = (torch.arange(s["E"], device="cuda", dtype=torch.int32)[:, None] == flat).to(torch.int32)
    before = hot.cumsum(1, dtype=torch.int32)
    offsets = torch.zeros(s["E"] + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = before[:, -1].cumsum(0)
    kept = flat >= 0
    start = (offsets[:-1, None] + before - 1) * hot
    position = torch.where(kept, start.sum(0, dtype=torch.int32), -1)
    token = torch.arange(flat.numel(), device="cuda", dtype=torch.int32) // s["topk"]
    source = torch.full((flat.numel() + 1,), -1, dtype=torch.int32, device="cuda")
    source[torch.where(kept, position, flat.numel()).long()] = token
    source = source[:-1]
    source = torch.where(torch.arange(flat.numel(), device="cuda") < offsets[-1], source, -1)
    return dict(offsets=offsets, source=source, position=position.view(s["ids"].shape))


def _plain_products(s):
    """One product for each group that has rows, in fp32."""
    x = s["X"] if s["rows"] is None else s["X"][s["rows"].long()]
    parts = x.split(s["counts"])
    return torch.cat([p.float() @ s["W"][e].float().t() for e, p in enumerate(parts) if p.shape[0]])


def _plain_grouped(s):
    return _plain_products(s).to(torch.bfloat16)


def _plain_gated(s):
    y = _plain_products(s)
    gate, up = y[:, :s["N"]], y[:, s["N"]:]
    return (gate / (1 + (-gate).exp()) * up).to(torch.bfloat16)


def _plain_combine(s):
    at = s["position"].long()
    rows = s["Z"][at.clamp_min(0)].float()
    w = torch.where(at >= 0, s["weights"], 0.0)
    y = (w[:, :, None] * rows).sum(1)
    if s["base_rows"] is not None:
        y = y + s["base_rows"].float()
    return y.to(torch.bfloat16)


def _plain_lora(s):
    """Every adapter's products for every row, masked to the row's own."""
    x = torch.cat(s["X_r"], 1).float()
    w = torch.cat(s["W_r"], 1).float()
    a = torch.cat(s["A_r"], 2).float()
    low = (x @ a.reshape(-1, a.shape[2]).t()).view(x.shape[0], s["L"], s["rank"])
    mine = s["adapter"][:, None] == torch.arange(s["L"], device="cuda", dtype=torch.int32)
    low = low * (mine * s["scale"])[:, :, None]
    b = s["B"].float().transpose(0, 1).reshape(s["N"], -1)
    return (x @ w.t() + low.reshape(x.shape[0], -1) @ b.t()).to(torch.bfloat16)


# ---------------------------------------------------------------- exact values

def exact(case, seed):
    """The definitions in 64 bits, row by row of the routing (no shared code but the inputs)."""
    if case["op"] == "route":
        return None
    s = _inputs(case, seed)
    if case["op"] == "combine":
        y = torch.zeros(case["T"], case["H"], dtype=torch.float64, device="cuda")
        if s["base_rows"] is not None:
            y += s["base_rows"].double()
        for j in range(case["topk"]):
            at = s["position"][:, j].long()
            t = torch.nonzero(at >= 0)[:, 0]
            y.index_add_(0, t, s["Z"][at[t]].double() * s["weights"][t, j].double()[:, None])
        return y
    if case["op"] in ("grouped", "gated"):
        y = torch.empty(case["T"] * case["topk"], case["N"], dtype=torch.float64, device="cuda")
        ends = s["offsets"].tolist()
        for e in range(case["E"]):
            lo, hi = ends[e], ends[e + 1]
            if lo == hi:
                continue
            at = torch.arange(lo, hi, device="cuda") if s["rows"] is None else s["rows"][lo:hi].long()
            z = torch.mm(s["X"][at].double(), s["W"][e].double().t())
            if case["op"] == "gated":
                z = torch.sigmoid(z[:, :case["N"]]) * z[:, :case["N"]] * z[:, case["N"]:]
            y[lo:hi] = z
        return y
    y = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
    for x, w in zip(s["X_r"], s["W_r"]):
        y += torch.mm(x.double(), w.double().t())
    for a in range(case["L"]):
        t = torch.nonzero(s["adapter"] == a)[:, 0]
        if t.numel():
            low = sum(torch.mm(x[t].double(), A[a].double().t()) for x, A in zip(s["X_r"], s["A_r"]))
            y[t] += s["scale"][a].double() * torch.mm(low, s["B"][a].double().t())
    return y


# ---------------------------------------------------------------- work

def _active(c):
    """Expected number of experts that get a row: topk different experts a token."""
    p = _popularity(c)
    lo, hi = 0.0, 1e9   # each expert is chosen with probability 1 - exp(-z p), sum = topk
    for _ in range(200):
        z = (lo * hi) ** 0.5 if lo else hi / 2
        lo, hi = (z, hi) if float((1 - (-z * p).exp()).sum()) < c["topk"] else (lo, z)
    q = 1 - (-hi * p).exp()
    return min(float((1 - (1 - q) ** c["T"]).sum()), c["T"] * c["topk"])


def work(c):
    if c["op"] == "route":
        rows = c["T"] * c["topk"]
        return dict(bytes=4 * (3 * rows + c["E"] + 1), flops=0)
    if c["op"] in ("grouped", "gated"):
        rows, wide = c["T"] * c["topk"], 2 * c["N"] if c["op"] == "gated" else c["N"]
        x_rows = c["T"] if c["op"] == "gated" else rows
        return dict(bytes=2 * (_active(c) * wide * c["K"] + x_rows * c["K"] + rows * c["N"]) + 4 * (c["E"] + 1)
                    + (4 * rows if c["op"] == "gated" else 0), flops=2 * rows * wide * c["K"])
    if c["op"] == "combine":
        rows = c["T"] * c["topk"]
        return dict(bytes=2 * c["H"] * (rows * (1 - c["drop"]) + c["T"] * (2 if c["base"] else 1)) + 8 * rows,
                    flops=2 * rows * c["H"])
    K, runs = c["R"] * c["K_r"], -(-c["M"] // c["run"])
    used = c["L"] * (1 - (1 - (1 - c["none"]) / c["L"]) ** runs)   # adapters that some row has
    with_one = c["M"] * (1 - c["none"])
    return dict(bytes=2 * (c["M"] * (K + c["N"]) + K * c["N"] + used * c["rank"] * (K + c["N"])) + 4 * (c["M"] + c["L"]),
                flops=2 * c["M"] * K * c["N"] + 2 * with_one * c["rank"] * (K + c["N"]))
