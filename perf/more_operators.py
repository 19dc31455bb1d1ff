"""The softmax attention layer of a hybrid model: rotary positions (with the keys and values going into a cache), causal
attention over packed sequences (their own rows or a cache's as keys; single tokens too) and attention of a batch that
shares prefixes: the cases they are measured on, in plain torch operations and through the library's calls.

  rotary:     (y1, y2) = a (x1 cos(p f_i) - x2 sin(p f_i), x2 cos(p f_i) + x1 sin(p f_i)) for pair i at position p
  attention:  o_t = sum_s w_ts v_s, w_t = softmax over the visible s of scale q_t . k_s, lse_t = log sum_s exp(scale q_t . k_s)
              token t of a sequence of n new tokens and m keys sees its keys s <= m - n + t, and all of its prefix
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BASE = 500000.0
ORIGINAL = 8192  # length that the unscaled frequencies were made for
FACTOR = 8.0
AMPLITUDE = 0.1 * math.log(FACTOR) + 1.0  # of the ramp
LOW, HIGH = {"bands": 1.0, "ramp": 1.0}, {"bands": 4.0, "ramp": 32.0}  # turns over ORIGINAL


def listed():
    return [
        # one token of one sequence: its query rotated, its key and value put into the cache
        {"name": "rope_token", "op": "rope", "tokens": 1, "hq": 32, "hkv": 8, "dim": 128, "rotary": 128,
         "interleaved": False, "scaling": "plain", "dtype": "bf16", "cache": 512, "farthest": 8000},
        # a decode batch at far positions of a model whose heads are rotated in part
        {"name": "rope_batch", "op": "rope", "tokens": 64, "hq": 16, "hkv": 2, "dim": 128, "rotary": 32,
         "interleaved": False, "scaling": "bands", "dtype": "bf16", "cache": 4096, "farthest": 131072},
        # a prompt of a wide layer, q and k side by side in the projection's rows
        {"name": "rope_prompt", "op": "rope", "tokens": 8192, "hq": 64, "hkv": 8, "dim": 128, "rotary": 128,
         "interleaved": False, "scaling": "ramp", "dtype": "bf16", "cache": 0, "farthest": 65536},
        # neighbouring elements as pairs, odd sizes, fp32
        {"name": "rope_odd", "op": "rope", "tokens": 999, "hq": 5, "hkv": 5, "dim": 96, "rotary": 42,
         "interleaved": True, "scaling": "linear", "dtype": "f32", "cache": 0, "farthest": 1048576},
        # one long prompt
        {"name": "prompt_one", "op": "prefill", "lengths": "4096", "kept": "", "hq": 32, "hkv": 8, "dim": 128,
         "tiled": False, "dtype": "bf16", "lse": False},
        # a packed batch of ragged prompts
        {"name": "prompt_ragged", "op": "prefill", "lengths": "8110,2965,6963,3562,4169,3929,2191,2593", "kept": "",
         "hq": 32, "hkv": 4, "dim": 128, "tiled": False, "dtype": "bf16", "lse": False},
        # a small model in fp32: short and odd prompts, one of a single token
        {"name": "prompt_small", "op": "prefill", "lengths": "77,1,130", "kept": "", "hq": 4, "hkv": 2, "dim": 64,
         "tiled": True, "dtype": "f32", "lse": True},
        # the next chunks of two prompts, whose keys are in a cache
        {"name": "chunk_cached", "op": "prefill", "lengths": "512,300", "kept": "15872,801", "hq": 32, "hkv": 8,
         "dim": 64, "tiled": False, "dtype": "f16", "lse": False},
        # one token of one sequence against its cache: the smallest serving step
        {"name": "step_one", "op": "prefill", "batch": 1, "each": 1, "longest": 4000, "hq": 32, "hkv": 8, "dim": 128,
         "tiled": False, "dtype": "bf16", "lse": False},
        # a decode batch with caches of all lengths
        {"name": "step_batch", "op": "prefill", "batch": 64, "each": 1, "longest": 8192, "hq": 32, "hkv": 8,
         "dim": 128, "tiled": False, "dtype": "bf16", "lse": False},
        # a decode batch behind one long system prompt
        {"name": "shared_batch", "op": "shared", "batch": 64, "each": 1, "longest": 1024, "prefixes": "8192",
         "members": "64", "hq": 32, "hkv": 8, "dim": 128, "tiled": False, "dtype": "bf16", "lse": False},
        # two groups of sequences that check a few drafted tokens each
        {"name": "shared_groups", "op": "shared", "batch": 13, "each": 4, "longest": 777, "prefixes": "2500,333",
         "members": "8,5", "hq": 12, "hkv": 4, "dim": 96, "tiled": True, "dtype": "f16", "lse": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "prefill", "prefill", "shared"])
    dim = rng.choice([32, 64, 96, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 6, 8])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "rope":
        most = 8192 * 80 * 128 // ((hq + 2 * hkv) * dim) // (2 if dtype == "f32" else 1)
        tokens = _log_int(rng, 1, min(most, 16384))
        return {"op": "rope", "tokens": tokens, "hq": hq, "hkv": hkv, "dim": dim,
                "rotary": rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)]),
                "interleaved": rng.random() < 0.4, "scaling": rng.choice(["plain", "linear", "bands", "ramp"]),
                "dtype": dtype, "cache": tokens + rng.randint(1, 500) if rng.random() < 0.6 else 0,
                "farthest": _log_int(rng, max(2, tokens), 1 << 20)}
    case = {"op": op, "hq": hq, "hkv": hkv, "dim": dim, "tiled": rng.random() < 0.3, "dtype": dtype,
            "lse": rng.random() < 0.4}
    pairs = 80_000_000 * 32 * 128 // (hq * dim)  # visible (query, key) pairs a head: those of the ragged prompts
    if dtype == "f32":
        pairs //= 16
    if op == "shared" or rng.random() < 0.4:
        case |= {"batch": _log_int(rng, 2 if op == "shared" else 1, 64), "each": rng.choice([1, 1, 1, 2, 5, 8])}
        case["longest"] = case["each"] + _log_int(rng, 1, 8192 if op == "prefill" else 2000)
        if op == "shared":
            groups = rng.randint(1, min(3, case["batch"]))
            cuts = sorted(rng.sample(range(1, case["batch"]), groups - 1))
            members = [b - a for a, b in zip([0] + cuts, cuts + [case["batch"]])]
            case |= {"members": ",".join(map(str, members)),
                     "prefixes": ",".join(str(_log_int(rng, 1, 8192)) for _ in range(groups))}
        return case
    lengths, kept, cached = [], [], rng.random() < 0.5
    for _ in range(_log_int(rng, 1, 16)):
        n = _log_int(rng, 1, 8192)
        m = _log_int(rng, 1, 16384) if cached else 0
        if n * (m + n // 2 + 1) <= pairs and sum(lengths) + sum(kept) + n + m <= 100_000:
            pairs -= n * (m + n // 2 + 1)
            lengths.append(n)
            kept.append(m)
    if not lengths:
        lengths, kept = [rng.randint(1, 300)], [rng.randint(0, 300) if cached else 0]
    elif rng.random() < 0.3:
        lengths[rng.randrange(len(lengths))] = 0
    if sum(lengths) == 0:
        lengths[0] = 5
    return case | {"lengths": ",".join(map(str, lengths)), "kept": ",".join(map(str, kept)) if cached else ""}


def _ints(text):
    return [int(x) for x in text.split(",")] if text else []


def _sizes(case):
    """New tokens of each sequence, and the keys that it sees of its own (None: its new tokens' rows)."""
    if "batch" in case:
        n, each, longest = case["batch"], case["each"], case["longest"]
        return [each] * n, [max(each, longest * (i * 37 % n + 1) // n) for i in range(n)]
    lengths, kept = _ints(case["lengths"]), _ints(case["kept"])
    return lengths, [a + b for a, b in zip(lengths, kept)] if kept else None


def _before(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return at


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    s = {"case": dict(case)}
    io = DTYPES[case["dtype"]]
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    if case["op"] == "rope":
        tokens, pool = case["tokens"], case["cache"]
        # q | k | v as the projection leaves them, in one row for each token
        row = normal(tokens, (hq + 2 * hkv) * dim, dtype=io)
        s["q"], s["k"], s["v"] = row[:, :hq * dim], row[:, hq * dim:(hq + hkv) * dim], row[:, (hq + hkv) * dim:]
        if tokens >= 256:  # one prompt
            first = int(torch.randint(max(1, case["farthest"] - tokens), (1,), generator=gen, device="cuda"))
            s["pos"] = torch.arange(first, first + tokens, dtype=torch.int32, device="cuda")
        else:  # tokens of different sequences
            s["pos"] = torch.randint(case["farthest"], (tokens,), generator=gen, device="cuda").to(torch.int32)
        s["q_out"] = torch.empty((tokens, hq * dim), dtype=io, device="cuda")
        s["rows"] = None
        if pool:
            s["rows"] = torch.randperm(pool, generator=gen, device="cuda")[:tokens].to(torch.int32)
            s["k_out"], s["v_out"] = normal(pool, hkv * dim, dtype=io), normal(pool, hkv * dim, dtype=io)
        else:
            s["k_out"] = torch.empty((tokens, hkv * dim), dtype=io, device="cuda")
        return s
    lengths, keys = _sizes(case)
    tokens = sum(lengths)
    s["cu"] = ints(_before(lengths))
    if keys is None:
        row = normal(tokens, (hq + 2 * hkv) * dim)
        row[:, :hq * dim] *= 2.0  # scores of a standard deviation of two
        row = row.to(io)
        s["q"], s["k"], s["v"] = row[:, :hq * dim], row[:, hq * dim:(hq + hkv) * dim], row[:, (hq + hkv) * dim:]
    else:
        # a pool of rows: each sequence's keys in a stretch of its own, the stretches in some order
        s["q"] = normal(tokens, hq * dim, std=2.0, dtype=io)
        stretches = keys + _ints(case.get("prefixes", ""))
        order = torch.randperm(len(stretches), generator=gen, device="cuda").tolist()
        start, at = [0] * len(stretches), 0
        for n in order:
            start[n] = at
            at += stretches[n] + 5
        s["k"], s["v"] = normal(at, hkv * dim, dtype=io), normal(at, hkv * dim, dtype=io)
        s["kv_start"], s["kv_len"] = ints(start[:len(keys)]), ints(keys)
        if case["op"] == "shared":
            members = _ints(case["members"])
            s["groups"] = ints([n * case["each"] for n in _before(members)])
            s["prefix_start"], s["prefix_len"] = ints(start[len(keys):]), ints(stretches[len(keys):])
    s["out"] = torch.empty((tokens, hq, dim), dtype=io, device="cuda")
    s["lse"] = torch.empty((tokens, hq), device="cuda") if case["lse"] else None
    return s


# ------------------------------------------------------------------ plain forms


def _frequencies(case):
    """Radians a position for each pair, in 64 bits."""
    r = case["rotary"]
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    f = torch.exp(i * (-2.0 * math.log(BASE) / r))
    kind = case["scaling"]
    if kind == "plain":
        return f
    if kind == "linear":
        return f / FACTOR
    low, high = LOW[kind], HIGH[kind]
    if kind == "bands":  # by the turns that a pair makes over the original length
        keep = ((ORIGINAL * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
    else:  # by the pair's index, between the whole ones around these turns

        def index(turns):
            return r * math.log(ORIGINAL / (2 * math.pi * turns)) / (2 * math.log(BASE))

        first, last = max(math.floor(index(high)), 0), min(math.ceil(index(low)), r - 1)
        keep = 1 - ((i - first) / max(last - first, 0.001)).clamp(0, 1)
    return f * (keep + (1 - keep) / FACTOR)


def _plain_rope(case, s):
    r, dim = case["rotary"], case["dim"]
    angle = s["pos"].double()[:, None] * _frequencies(case)
    a = AMPLITUDE if case["scaling"] == "ramp" else 1.0
    cos, sin = (angle.cos() * a).float()[:, None], (angle.sin() * a).float()[:, None]

    def rotated(x):
        x = x.reshape(x.shape[0], -1, dim).float()
        y = x.clone()
        if case["interleaved"]:
            x1, x2, at1, at2 = x[..., 0:r:2], x[..., 1:r:2], slice(0, r, 2), slice(1, r, 2)
        else:
            x1, x2, at1, at2 = x[..., :r // 2], x[..., r // 2:r], slice(0, r // 2), slice(r // 2, r)
        y[..., at1] = x1 * cos - x2 * sin
        y[..., at2] = x2 * cos + x1 * sin
        return y.reshape(x.shape[0], -1)

    s["q_out"].copy_(rotated(s["q"]))
    if s["rows"] is None:
        s["k_out"].copy_(rotated(s["k"]))
        return {"q": s["q_out"], "k": s["k_out"]}
    at = s["rows"].long()
    s["k_out"][at] = rotated(s["k"]).to(s["k_out"].dtype)
    s["v_out"][at] = s["v"]
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _kv_head(case):
    """The key head of each query head."""
    h = torch.arange(case["hq"], device="cuda")
    return h % case["hkv"] if case["tiled"] else h // (case["hq"] // case["hkv"])


def _query_heads(case):
    """Query heads by the key head that they read, [hkv][heads of a group]."""
    return torch.argsort(_kv_head(case), stable=True).reshape(case["hkv"], -1)


def _soft(case, scores, mask, v):
    """Masked softmax of [..., queries, keys] and its product with v; the logarithm of the sums."""
    scores = scores.masked_fill(~mask, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    w = torch.exp(scores - top)
    total = w.sum(-1, keepdim=True)
    o = (w @ v) / torch.where(total > 0, total, 1.0)
    return o, (top + torch.log(total))[..., 0]


def _plain_long(case, s):
    """Sequence after sequence, their queries in pieces."""
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    lengths, keys = _sizes(case)
    first = _before(lengths)
    order = _query_heads(case)
    for n, count in enumerate(lengths):
        if count == 0:
            continue
        if keys is None:
            at, m = first[n], count
        else:
            at, m = s["kv_start"][n].long(), keys[n]
        rows = at + torch.arange(m, device="cuda")
        k = s["k"][rows].float().reshape(m, hkv, dim).permute(1, 2, 0)
        v = s["v"][rows].float().reshape(m, hkv, dim).transpose(0, 1)
        for a in range(0, count, 1024):
            b = min(a + 1024, count)
            see = m - count + b
            q = s["q"][first[n] + a:first[n] + b].float().reshape(b - a, hq, dim)
            q = q[:, order].permute(1, 2, 0, 3).reshape(hkv, -1, dim) * dim ** -0.5
            mask = torch.arange(see, device="cuda") <= (m - count + torch.arange(a, b, device="cuda"))[:, None]
            mask = mask.repeat(hq // hkv, 1)
            o, lse = _soft(case, q @ k[:, :, :see], mask, v[:, :see])
            to = slice(first[n] + a, first[n] + b)
            s["out"][to, order.flatten()] = o.reshape(hq, b - a, dim).transpose(0, 1).to(s["out"].dtype)
            if case["lse"]:
                s["lse"][to, order.flatten()] = lse.reshape(hq, b - a).t()


def _plain_batch(case, s):
    """Few tokens each: all sequences at once, over padded keys, their prefix before their own."""
    hq, hkv, dim, each = case["hq"], case["hkv"], case["dim"], case["each"]
    lengths, keys = _sizes(case)
    n = len(lengths)
    at = torch.arange(max(keys), device="cuda")
    rows = s["kv_start"].long()[:, None] + torch.minimum(at, s["kv_len"].long()[:, None] - 1)
    last = s["kv_len"].long()[:, None] - each + torch.arange(each, device="cuda")
    mask = at[None, None, :] <= last[:, :, None]
    if case["op"] == "shared":
        prefixes = _ints(case["prefixes"])
        group = torch.repeat_interleave(torch.arange(len(prefixes), device="cuda"),
                                        torch.tensor(_ints(case["members"]), device="cuda"))
        at = torch.arange(max(prefixes), device="cuda")
        length = s["prefix_len"].long()[group][:, None]
        rows = torch.cat([s["prefix_start"].long()[group][:, None] + torch.minimum(at, length - 1), rows], 1)
        mask = torch.cat([(at < length)[:, None, :].expand(n, each, -1), mask], 2)
    order = _query_heads(case)
    k = s["k"][rows].float().reshape(n, -1, hkv, dim).permute(0, 2, 3, 1)
    v = s["v"][rows].float().reshape(n, -1, hkv, dim).transpose(1, 2)
    q = s["q"].float().reshape(n, each, hq, dim)[:, :, order].permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, dim)
    mask = mask.repeat(1, hq // hkv, 1)[:, None]
    o, lse = _soft(case, q @ k * dim ** -0.5, mask, v)
    o = o.reshape(n, hq, each, dim).transpose(1, 2).reshape(n * each, hq, dim)
    s["out"][:, order.flatten()] = o.to(s["out"].dtype)
    if case["lse"]:
        s["lse"][:, order.flatten()] = lse.reshape(n, hq, each).transpose(1, 2).reshape(n * each, hq)


# ------------------------------------------------------------------ the library's calls


def _dims(gdn, case):
    return gdn.dims(case["hkv"], case["hq"], case["dim"],
                    map=gdn.GDN_MAP_TILED if case.get("tiled") else gdn.GDN_MAP_GROUPED, io_dtype=DTYPES[case["dtype"]])


def _own_rope(gdn, case, s):
    if "spec" not in s:  # a model's, made once
        kind = case["scaling"]
        s["spec"] = gdn.rope_spec(
            case["rotary"], layout=gdn.GDN_ROPE_INTERLEAVED if case["interleaved"] else gdn.GDN_ROPE_HALF, base=BASE,
            scaling={"plain": gdn.GDN_ROPE_PLAIN, "linear": gdn.GDN_ROPE_LINEAR, "bands": gdn.GDN_ROPE_BANDS,
                     "ramp": gdn.GDN_ROPE_RAMP}[kind],
            factor=FACTOR, original_length=ORIGINAL, low=LOW.get(kind, 0.0), high=HIGH.get(kind, 0.0),
            amplitude=AMPLITUDE if kind == "ramp" else 1.0)
        s["dims"] = _dims(gdn, case)
    outs = {"q": s["q_out"], "k": s["k_out"]}
    cache = {}
    if s["rows"] is not None:
        outs["v"] = s["v_out"]
        cache = {"v": s["v"], "v_out": s["v_out"], "cache_rows": s["rows"]}
    gdn.gdn_rope(s["dims"], s["spec"], s["pos"], q=s["q"], q_out=s["q_out"], k=s["k"], k_out=s["k_out"], **cache)
    return outs


def _own_attention(gdn, case, s):
    if "dims" not in s:
        s["dims"] = _dims(gdn, case)
    if case["op"] == "shared":
        gdn.gdn_attn_shared(s["dims"], s["cu"], s["q"], s["k"], s["v"], s["kv_start"], s["kv_len"], s["groups"],
                            s["prefix_start"], s["prefix_len"], s["out"], lse=s["lse"])
    else:
        gdn.gdn_attn_prefill(s["dims"], s["cu"], s["q"], s["k"], s["v"], s["out"], lse=s["lse"],
                             kv_start=s.get("kv_start"), kv_len=s.get("kv_len"))


def run(state):
    case = state["case"]
    if own:
        import gated_delta_net_causal_gb300 as gdn

        if case["op"] == "rope":
            return _own_rope(gdn, case, state)
        _own_attention(gdn, case, state)
    elif case["op"] == "rope":
        return _plain_rope(case, state)
    elif "batch" in case:
        _plain_batch(case, state)
    else:
        _plain_long(case, state)
    return {"out": state["out"], "lse": state["lse"]} if case["lse"] else {"out": state["out"]}


# ------------------------------------------------------------------ floors


def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    if case["op"] == "rope":
        tokens = case["tokens"]
        heads = hq + hkv + (hkv if case["cache"] else 0)
        return {"bytes": 2 * tokens * heads * dim * es + 4 * tokens * (2 if case["cache"] else 1),
                "flops": 3 * tokens * (hq + hkv) * case["rotary"]}
    lengths, keys = _sizes(case)
    tokens = sum(lengths)
    keys = lengths if keys is None else keys
    pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(lengths, keys))
    rows = sum(m for n, m in zip(lengths, keys) if n > 0)
    if case["op"] == "shared":
        for count, p in zip(_ints(case["members"]), _ints(case["prefixes"])):
            pairs += count * case["each"] * p
            rows += p
    return {"bytes": 2 * tokens * hq * dim * es + 2 * rows * hkv * dim * es + (4 * tokens * hq if case["lse"] else 0),
            "flops": 4 * pairs * hq * dim}


# ------------------------------------------------------------------ definitions in 64 bits


def _exact_rope(case, s):
    r, dim = case["rotary"], case["dim"]
    freqs, turns = [], 2 * math.pi / ORIGINAL
    for i in range(r // 2):
        f = BASE ** (-2.0 * i / r)
        if case["scaling"] == "linear":
            f /= FACTOR
        elif case["scaling"] == "bands":
            if f <= LOW["bands"] * turns:
                f /= FACTOR
            elif f < HIGH["bands"] * turns:
                part = (f / turns - LOW["bands"]) / (HIGH["bands"] - LOW["bands"])
                f = part * f + (1 - part) * f / FACTOR
        elif case["scaling"] == "ramp":
            a = max(math.floor(r / 2 * math.log(1 / (HIGH["ramp"] * turns), BASE)), 0)
            b = min(math.ceil(r / 2 * math.log(1 / (LOW["ramp"] * turns), BASE)), r - 1)
            part = min(max((i - a) / max(b - a, 0.001), 0.0), 1.0)
            f = (1 - part) * f + part * f / FACTOR
        freqs.append(f)
    a = AMPLITUDE if case["scaling"] == "ramp" else 1.0
    angle = torch.einsum("t,i->ti", s["pos"].double(), torch.tensor(freqs, dtype=torch.float64, device="cuda"))
    turn = torch.polar(torch.full_like(angle, a), angle)[:, None, :]

    def rotated(x):
        x = x.double().reshape(x.shape[0], -1, dim)
        part = x[..., :r]
        pairs = part.unflatten(-1, (-1, 2)) if case["interleaved"] else part.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.complex(pairs[..., 0].contiguous(), pairs[..., 1].contiguous()) * turn)
        part = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([part, x[..., r:]], -1).flatten(1)

    q, k = rotated(s["q"]), rotated(s["k"])
    if s["rows"] is None:
        return {"q": q, "k": k}
    rows = s["rows"].long()
    return {"q": q, "k": s["k_out"].double().index_copy(0, rows, k),
            "v": s["v_out"].double().index_copy(0, rows, s["v"].double())}


def _exact_attention(case, s):
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    lengths, keys = _sizes(case)
    first, total = _before(lengths), sum(lengths)
    out = torch.zeros((total, hq, dim), dtype=torch.float64, device="cuda")
    lse = torch.full((total, hq), -math.inf, dtype=torch.float64, device="cuda")
    starts = first if keys is None else s["kv_start"].tolist()
    prefix = [(0, 0)] * len(lengths)
    if case["op"] == "shared":
        prefix = [(a, p) for a, p, c in zip(s["prefix_start"].tolist(), _ints(case["prefixes"]), _ints(case["members"]))
                  for _ in range(c)]
    for n, count in enumerate(lengths):
        m = count if keys is None else keys[n]
        p0, p = prefix[n]
        for a in range(0, count, 512):
            b = min(a + 512, count)
            see = m - count + b
            rows = list(range(p0, p0 + p)) + list(range(starts[n], starts[n] + see))
            rows = torch.tensor(rows, device="cuda")
            after = torch.arange(p + see, device="cuda")[None, :] - p > torch.arange(a, b, device="cuda")[:, None] + m - count
            q = s["q"][first[n] + a:first[n] + b].double().reshape(b - a, hq, dim)
            for h in range(hq):
                kh = h % hkv if case["tiled"] else h * hkv // hq
                cols = slice(kh * dim, (kh + 1) * dim)
                x = torch.mm(q[:, h], s["k"][rows, cols].double().t()) / math.sqrt(dim)
                x[after] = -math.inf
                norm = torch.logsumexp(x, 1)
                lse[first[n] + a:first[n] + b, h] = norm
                out[first[n] + a:first[n] + b, h] = torch.mm((x - norm[:, None]).exp_(), s["v"][rows, cols].double())
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(case, s) if case["op"] == "rope" else _exact_attention(case, s)
