"""Linear attention with a decay for each head (prompt and single-token forms), the RMS norm around it
(residual addition, output in 8 bits with scales) and the linear layer on 8-bit operands that reads it:
the cases they are measured on, in plain torch operations and through the library's calls.

  S_t[j][i] = exp(g_t) S_{t-1}[j][i] + v_t[j] k_t[i],   o_t[j] = scale sum_i S_t[j][i] q_t[i]
  s = round(x + r),  y = s (mean s^2 + eps)^(-1/2) w,  y ~ out_q * out_scale  (e4m3, one scale a row)
  y[m][n] = x_scale[m] w_scale[n] sum_k x[m][k] w[n][k] + bias[n]
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
CHUNK = 64  # of the plain prompt form
E4M3_MAX = 448.0
TINY = 2.0 ** -126


def listed():
    return [
        # one token of one sequence: the smallest serving step, where latency counts
        {"name": "step_one", "op": "step", "batch": 1, "pool": 0, "hk": 16, "hv": 32, "dim": 128, "tiled": False,
         "dtype": "bf16", "token_decay": False, "gated": True},
        # continuous batching: 64 live sequences in a pool of 256 state slots
        {"name": "step_slots", "op": "step", "batch": 64, "pool": 256, "hk": 16, "hv": 32, "dim": 128, "tiled": True,
         "dtype": "bf16", "token_decay": True, "gated": True},
        # a large decode batch of a wide layer
        {"name": "step_batch", "op": "step", "batch": 128, "pool": 0, "hk": 16, "hv": 48, "dim": 128, "tiled": False,
         "dtype": "bf16", "token_decay": False, "gated": True},
        # one long prompt, a fixed decay for each head
        {"name": "prompt_one", "op": "prefill", "lengths": "4096", "hk": 16, "hv": 32, "dim": 128, "tiled": True,
         "dtype": "bf16", "token_decay": False, "gated": True},
        # a packed batch of ragged prompts, a decay for each token and head
        {"name": "prompt_ragged", "op": "prefill", "lengths": "8110,2965,6963,3562,4169,3929,2191,2593", "hk": 16,
         "hv": 64, "dim": 128, "tiled": False, "dtype": "bf16", "token_decay": True, "gated": False},
        # a small model in fp32: short and odd prompts, one of a single token, fp32 outputs
        {"name": "prompt_small", "op": "prefill", "lengths": "77,1,130", "hk": 2, "hv": 4, "dim": 64, "tiled": True,
         "dtype": "f32", "token_decay": True, "gated": False},
        # the norm before a layer's projection for one token
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 2048, "stride": 2048, "dtype": "bf16",
         "residual": True, "eight": True},
        # the same for a prompt of a wide model
        {"name": "norm_prompt", "op": "norm", "rows": 8192, "cols": 8192, "stride": 8192, "dtype": "bf16",
         "residual": True, "eight": True},
        # odd sizes, rows inside a wider buffer, 16-bit output
        {"name": "norm_odd", "op": "norm", "rows": 999, "cols": 2051, "stride": 2100, "dtype": "f16",
         "residual": False, "eight": False},
        # the input projection (q | k | v | z) of one token: a stream of the weights
        {"name": "linear_token", "op": "linear", "m": 1, "n": 12352, "k": 2048, "dtype": "bf16", "bias": False},
        # the same for a decode batch
        {"name": "linear_batch", "op": "linear", "m": 64, "n": 12352, "k": 2048, "dtype": "bf16", "bias": True},
        # the same for a prompt
        {"name": "linear_prompt", "op": "linear", "m": 4096, "n": 12352, "k": 2048, "dtype": "bf16", "bias": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "prefill", "norm", "linear"])
    if op in ("step", "prefill"):
        dim = rng.choice([32, 64, 96, 128, 128])
        hk = rng.choice([1, 2, 4, 8, 16])
        hv = hk * rng.choice([1, 2, 3, 4])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        heads = {"hk": hk, "hv": hv, "dim": dim, "tiled": rng.random() < 0.5, "dtype": dtype,
                 "token_decay": rng.random() < 0.5, "gated": rng.random() < 0.5}
    if op == "step":
        most = 128 * 48 * 128 * 128 // (hv * dim * dim)
        batch = _log_int(rng, 1, min(most, 512))
        pool = batch + rng.randint(1, batch + 8) if rng.random() < 0.5 and 2 * batch + 8 <= 2 * most else 0
        return {"op": "step", "batch": batch, "pool": pool, **heads}
    if op == "prefill":
        n = _log_int(rng, 1, 16)
        lengths = [_log_int(rng, 1, 4000) for _ in range(n)]
        if rng.random() < 0.3:
            lengths[rng.randrange(n)] = 0
        most = 34482 * 64 * 128 // (hv * dim)
        while sum(lengths) > most:
            lengths.pop()
        if sum(lengths) == 0:
            lengths.append(rng.randint(1, 300))
        return {"op": "prefill", "lengths": ",".join(map(str, lengths)), **heads}
    if op == "norm":
        cols = _log_int(rng, 1, 16384)
        rows = _log_int(rng, 1, max(1, 8192 * 8192 // cols // 8))
        return {"op": "norm", "rows": rows, "cols": cols, "stride": cols + rng.choice([0, 0, 8, 13]),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "residual": rng.random() < 0.5,
                "eight": rng.random() < 0.6}
    k = 16 * _log_int(rng, 1, 512)
    n = _log_int(rng, 1, 16384)
    m = _log_int(rng, 1, min(8192, 4096 * 12352 * 2048 // (n * k)))
    return {"op": "linear", "m": m, "n": n, "k": k, "dtype": rng.choice(["bf16", "bf16", "f16"]),
            "bias": rng.random() < 0.5}


def _lengths(case):
    return [int(x) for x in case["lengths"].split(",")]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    s = {"case": dict(case)}
    io = DTYPES[case["dtype"]]
    if case["op"] == "norm":
        rows, cols, stride = case["rows"], case["cols"], case["stride"]
        s["x"] = normal(rows, stride, dtype=io)[:, :cols]
        # the residual stream is wider than one layer's output, a few columns far wider
        s["residual"] = None
        if case["residual"]:
            r = normal(rows, stride, std=2.0)
            r[:, 7::512] *= 20.0
            s["residual"] = r.to(io)[:, :cols]
            s["sum"] = torch.empty((rows, cols), dtype=io, device="cuda")
        s["w"] = 1.0 + 0.2 * normal(cols)
        s["out"] = torch.empty((rows, cols), dtype=torch.float8_e4m3fn if case["eight"] else io, device="cuda")
        s["scale"] = torch.empty((rows,), device="cuda") if case["eight"] else None
        return s
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]

        def eight(rows, std):
            """Rows quantised as a user quantises them: the largest magnitude at the type's largest value."""
            t = normal(rows, k, std=std)
            sc = (t.abs().amax(dim=1) / E4M3_MAX).clamp_min(TINY)
            return (t / sc[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), sc

        s["x"], s["x_scale"] = eight(m, 1.0)
        s["w"], s["w_scale"] = eight(n, k ** -0.5)
        s["bias"] = normal(n, std=0.1) if case["bias"] else None
        s["y"] = torch.empty((m, (n + 7) // 8 * 8), dtype=io, device="cuda")[:, :n]
        return s
    hk, hv, dim = case["hk"], case["hv"], case["dim"]
    step = case["op"] == "step"
    tokens = case["batch"] if step else sum(_lengths(case))
    # q | k | v | z as the input projection leaves them, in one row for each token
    width = (2 * hk + 2 * hv) * dim
    row = normal(tokens, width)
    row[:, hk * dim:2 * hk * dim] *= dim ** -0.5
    row = row.to(io)
    s["q"], s["k"] = row[:, :hk * dim], row[:, hk * dim:2 * hk * dim]
    s["v"], s["z"] = row[:, 2 * hk * dim:(2 * hk + hv) * dim], row[:, (2 * hk + hv) * dim:]
    rate = torch.exp2(-5.0 - 5.0 * torch.arange(hv, device="cuda") / hv)  # memories of 30 to 1000 tokens
    if case["token_decay"]:
        s["g"] = -torch.nn.functional.softplus(normal(tokens, hv)) * rate * 4.0
    else:
        s["g"] = torch.log1p(-rate)
    s["norm_w"] = 1.0 + 0.2 * normal(dim)
    if step:
        slots = case["pool"] or case["batch"]
        s["slots"] = None
        if case["pool"]:
            s["slots"] = torch.randperm(slots, generator=gen, device="cuda")[:tokens].to(torch.int32)
    else:
        lengths = _lengths(case)
        slots = len(lengths)
        cu = [0]
        for n in lengths:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["lengths"] = lengths
    s["state"] = normal(slots, hv, dim, dim, std=0.1)
    # gated: the layer's 16-bit output; else the core output, fp32 for an fp32 model
    s["out"] = torch.empty((tokens, hv, dim), dtype=io, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms


def _heads(case, t, heads):
    """[tokens][heads * dim] -> [tokens][hv][dim] in fp32, each V head with the K head that it reads."""
    hv, rep = case["hv"], case["hv"] // heads
    t = t.reshape(t.shape[0], heads, case["dim"]).float()
    if rep == 1:
        return t
    h = torch.arange(hv, device=t.device)
    return t[:, h % heads if case["tiled"] else h // rep]


def _finish(case, s, o):
    """The output's gated norm, or the output itself, rounded once."""
    if case["gated"]:
        z = s["z"].reshape(o.shape).float()
        o = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS) * s["norm_w"] * z * torch.sigmoid(z)
    s["out"].copy_(o)
    return s["out"]


def _plain_step(case, s):
    q, k, v = _heads(case, s["q"], case["hk"]), _heads(case, s["k"], case["hk"]), _heads(case, s["v"], case["hv"])
    decay = torch.exp(s["g"]).expand(q.shape[0], case["hv"])
    old = s["state"] if s["slots"] is None else s["state"][s["slots"].long()]
    new = old * decay[:, :, None, None] + v[:, :, :, None] * k[:, :, None, :]
    o = (new * q[:, :, None, :]).sum(-1) * case["dim"] ** -0.5
    if s["slots"] is None:
        s["state"].copy_(new)
    else:
        s["state"][s["slots"].long()] = new
    return {"out": _finish(case, s, o), "state": s["state"]}


def _plain_prefill(case, s):
    """Chunk by chunk over padded sequences, all chunks at once: a chunk's own tokens through the masked, decayed
    products of q and k; what came before through the state at its start, a sum over the chunks before it."""
    hv, dim, n = case["hv"], case["dim"], len(s["lengths"])
    chunks = max(1, -(-max(s["lengths"]) // CHUNK))
    at = torch.arange(chunks * CHUNK, device="cuda")
    first, last = s["cu"][:-1].long(), s["cu"][1:].long()
    real = at[None, :] < (last - first)[:, None]
    src = torch.where(real, first[:, None] + at[None, :], 0)

    def padded(t):
        t = t[src] * real.reshape(*real.shape, *([1] * (t.dim() - 1)))
        return t.reshape(n, chunks, CHUNK, *t.shape[2:]).movedim(3, 1)  # [n][hv][chunk][token]...

    q, k = padded(_heads(case, s["q"], case["hk"])), padded(_heads(case, s["k"], case["hk"]))
    v = padded(_heads(case, s["v"], hv))
    g = s["g"].double().expand(s["q"].shape[0], hv)
    g = padded(g)
    run_g = g.cumsum(-1)  # sums of logarithms in 64 bits: their differences are what counts
    total = run_g[..., -1]
    mask = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril()
    decay = torch.where(mask, (run_g[..., :, None] - run_g[..., None, :]).float().exp(), 0.0)
    intra = ((q @ k.transpose(-1, -2)) * decay) @ v
    del decay
    # what each chunk adds to the state, [i][j], then the state at each chunk's start
    add = (k * (total[..., None] - run_g).float().exp()[..., None]).transpose(-1, -2) @ v
    upto = total.cumsum(-1)
    between = (upto - total)[..., :, None] - upto[..., None, :]  # decay from the end of chunk c' to the start of c
    before = torch.ones(chunks, chunks, dtype=torch.bool, device="cuda").tril(-1)
    mix = torch.where(before, between.float().exp(), 0.0)
    start = s["state"].transpose(-1, -2)  # [n][hv][i][j]
    into = (mix @ add.reshape(n, hv, chunks, dim * dim)).reshape(n, hv, chunks, dim, dim)
    into += start[:, :, None] * (upto - total).float().exp()[..., None, None]
    o = intra + (q @ into) * run_g.float().exp()[..., None]
    final = into[:, :, -1] * total[..., -1].float().exp()[..., None, None] + add[:, :, -1]
    s["state"].copy_(final.transpose(-1, -2))
    o = o.movedim(1, 3).reshape(n, chunks * CHUNK, hv, dim)
    seq = torch.searchsorted(last, torch.arange(s["q"].shape[0], device="cuda"), right=True)
    o = o[seq, torch.arange(s["q"].shape[0], device="cuda") - first[seq]] * dim ** -0.5
    return {"out": _finish(case, s, o), "state": s["state"]}


def _plain_norm(case, s):
    x = s["x"].float()
    outs = {}
    if s["residual"] is not None:
        s["sum"].copy_(x + s["residual"].float())
        outs["sum"] = s["sum"]
        x = s["sum"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["w"]
    if case["eight"]:
        s["scale"].copy_((y.abs().amax(dim=1) / E4M3_MAX).clamp_min(TINY))
        y = (y / s["scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        outs["scale"] = s["scale"]
    s["out"].copy_(y)
    outs["out"] = s["out"]
    return outs


def _plain_linear(case, s):
    y = (s["x"].float() @ s["w"].float().t()) * s["x_scale"][:, None] * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    s["y"].copy_(y)
    return s["y"]


# ------------------------------------------------------------------ the library's calls


def _own_attention(gdn, case, s):
    d = gdn.dims(case["hk"], case["hv"], case["dim"], map=gdn.GDN_MAP_TILED if case["tiled"] else gdn.GDN_MAP_GROUPED,
                 io_dtype=DTYPES[case["dtype"]], rms_eps=EPS)
    gate = {"z": s["z"], "norm_w": s["norm_w"]} if case["gated"] else {}
    if case["op"] == "step":
        gdn.gdn_decay_step(d, s["q"], s["k"], s["v"], s["g"], s["state"], out=s["out"], state_slots=s["slots"], **gate)
    else:
        gdn.gdn_decay_prefill(d, s["cu"], s["q"], s["k"], s["v"], s["g"], s["state"], out=s["out"], **gate)
    return {"out": s["out"], "state": s["state"]}


def _own_norm(gdn, case, s):
    outs = {"out": s["out"]}
    kinds = {"out_q": s["out"], "out_scale": s["scale"]} if case["eight"] else {"out": s["out"]}
    if case["eight"]:
        outs["scale"] = s["scale"]
    if s["residual"] is not None:
        kinds |= {"residual": s["residual"], "sum_out": s["sum"]}
        outs["sum"] = s["sum"]
    gdn.gdn_add_rmsnorm(s["x"], s["w"], eps=EPS, **kinds)
    return outs


def _own_linear(gdn, case, s):
    return gdn.gdn_linear_fp8(s["x"], s["x_scale"], s["w"], s["w_scale"], s["y"], bias=s["bias"])


def run(state):
    case = state["case"]
    if own:
        import gated_delta_net_causal_gb300 as gdn

        return {"step": _own_attention, "prefill": _own_attention, "norm": _own_norm,
                "linear": _own_linear}[case["op"]](gdn, case, state)
    return {"step": _plain_step, "prefill": _plain_prefill, "norm": _plain_norm,
            "linear": _plain_linear}[case["op"]](case, state)


# ------------------------------------------------------------------ floors


def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        n = case["rows"] * case["cols"]
        moved = n * es * (3 if case["residual"] else 1) + n * (1 if case["eight"] else es)
        return {"bytes": moved + 4 * case["cols"] + (4 * case["rows"] if case["eight"] else 0), "flops": 6 * n}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + m * n * es + 4 * (m + n) + (4 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    hk, hv, dim = case["hk"], case["hv"], case["dim"]
    step = case["op"] == "step"
    tokens = case["batch"] if step else sum(_lengths(case))
    states = tokens if step else sum(n > 0 for n in _lengths(case))
    acts = tokens * (2 * hk + (3 if case["gated"] else 2) * hv) * dim * es
    acts += 4 * (tokens * hv if case["token_decay"] else hv)
    return {"bytes": 8 * states * hv * dim * dim + acts, "flops": (5 if step else 4) * tokens * hv * dim * dim}


# ------------------------------------------------------------------ definitions in 64 bits


def _exact_recurrence(case, s):
    """The recurrence, token after token, for all sequences side by side."""
    hk, hv, dim = case["hk"], case["hv"], case["dim"]
    of_v = [h % hk if case["tiled"] else h * hk // hv for h in range(hv)]
    step = case["op"] == "step"
    starts = list(range(case["batch"])) if step else s["cu"].tolist()[:-1]
    lengths = [1] * case["batch"] if step else s["lengths"]
    q = s["q"].double().reshape(-1, hk, dim)
    k = s["k"].double().reshape(-1, hk, dim)
    v = s["v"].double().reshape(-1, hv, dim)
    state = s["state"].double().clone()
    rows = list(range(len(starts))) if not step or s["slots"] is None else s["slots"].tolist()
    out = torch.zeros((q.shape[0], hv, dim), dtype=torch.float64, device="cuda")
    order = sorted(range(len(starts)), key=lambda n: -lengths[n])
    live = state[[rows[n] for n in order]]
    begin = torch.tensor([starts[n] for n in order], device="cuda")
    g = s["g"].double()
    heads = torch.tensor(of_v, device="cuda")
    active = len(order)
    for t in range(max(lengths)):
        while active and lengths[order[active - 1]] <= t:
            active -= 1
        at = begin[:active] + t
        gt = g[at] if g.dim() == 2 else g[None, :]
        view = live[:active]
        view.mul_(gt.exp()[:, :, None, None])
        view.add_(torch.einsum("bhj,bhi->bhji", v[at], k[at][:, heads]))
        out[at] = torch.einsum("bhji,bhi->bhj", view, q[at][:, heads])
    out /= math.sqrt(dim)
    state[[rows[n] for n in order]] = live
    if case["gated"]:
        z = s["z"].double().reshape(out.shape)
        out = out / (out.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * s["norm_w"].double() * (z / (1 + (-z).exp()))
    return {"out": out, "state": state}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("step", "prefill"):
        return _exact_recurrence(case, s)
    if case["op"] == "linear":
        x = s["x"].double() * s["x_scale"].double()[:, None]
        w = s["w"].double() * s["w_scale"].double()[:, None]
        y = torch.einsum("mk,nk->mn", x, w)
        return y if s["bias"] is None else y + s["bias"].double()
    x = s["x"].double()
    outs = {}
    if s["residual"] is not None:
        x = x + s["residual"].double()
        outs["sum"] = x
        x = x.to(s["x"].dtype).double()
    y = x / (x.pow(2).sum(-1, keepdim=True) / case["cols"] + EPS).sqrt() * s["w"].double()
    if case["eight"]:
        outs["scale"] = (y.abs().max(dim=1).values / E4M3_MAX).clamp_min(TINY)
        y = y / outs["scale"][:, None]
    outs["out"] = y
    return outs
