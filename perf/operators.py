"""The operators around the scan and its cache, as cases to measure: projections of the mixer
(matrix product with an epilogue), the gated norm, log probabilities of tokens, and the pages
and slots of a replay cache.

With `own` false, `run` computes them in their plain form, elementary torch operations in
32 bits; with `own` true it makes the framework's calls. Sizes follow the shapes of the tests
and the benchmark (H=24, 32 and 64 heads of P=64, N=128, G=1 and 8, chunk 256).
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ---- cases ----------------------------------------------------------------

def listed():
    return [
        # batch-1 decode of a 24-head layer: latency of the smallest projection
        {"name": "in_proj one token", "op": "in_proj", "M": 1, "K": 768, "H": 24, "G": 1, "P": 64,
         "N": 128, "io": "bf16", "dt": "f32"},
        # out-projection of a decode batch of 256, onto the residual stream
        {"name": "out_proj batch 256", "op": "linear", "M": 256, "K": 4096, "N": 2048,
         "io": "bf16", "out": "bf16", "act": "none", "bias": False, "residual": True},
        # in-projection of a packed prompt batch, grouped heads: the matrix-core rate counts
        {"name": "in_proj prompts", "op": "in_proj", "M": 8192, "K": 2048, "H": 64, "G": 8,
         "P": 64, "N": 128, "io": "bf16", "dt": "bf16"},
        # fp32 run of a feed-forward product with its whole epilogue, ragged in rows and columns
        {"name": "linear f32 epilogue", "op": "linear", "M": 777, "K": 1000, "N": 1537,
         "io": "f32", "out": "f32", "act": "gelu", "bias": True, "residual": True},
        # the norm of a decode batch: a launch's latency
        {"name": "gated norm batch 256", "op": "norm", "T": 256, "H": 32, "P": 64, "groups": 1,
         "io": "bf16", "before": False},
        # the norm of a packed prompt batch, grouped heads: a stream
        {"name": "gated norm prompts", "op": "norm", "T": 16384, "H": 64, "P": 64, "groups": 8,
         "io": "bf16", "before": False},
        # sampling a decode batch of 32 with 20 alternatives each, fp32 logits
        {"name": "logprobs decode", "op": "logprobs", "T": 32, "V": 50280, "io": "f32", "k": 20,
         "allowed": 1.0},
        # scoring every token of prompts
        {"name": "logprobs prompts", "op": "logprobs", "T": 4096, "V": 50280, "io": "bf16",
         "k": 5, "allowed": 1.0},
        # constrained decoding: one token in 500 allowed, the others -inf
        {"name": "logprobs masked", "op": "logprobs", "T": 512, "V": 131072, "io": "bf16", "k": 8,
         "allowed": 0.002},
        # a speculative round's page traffic: surplus pages back, pages for the drafts out
        {"name": "pages round", "op": "pages", "slots": 512, "H": 2, "G": 1, "P": 64, "N": 128,
         "Q": 256, "pt": 16, "tokens": 5, "io": "bf16", "dt": "bf16"},
        # ended sequences' slots freed, prompts forked into eight samples each
        {"name": "slots turnover", "op": "fork", "slots": 160, "sources": 16, "fan": 8, "ended": 16,
         "H": 32, "G": 1, "P": 64, "N": 128, "Q": 256, "pt": 64, "io": "bf16", "dt": "bf16"},
        # a pool squeezed after load has gone
        {"name": "pages compact", "op": "compact", "slots": 256, "H": 32, "G": 1, "P": 64, "N": 128,
         "Q": 256, "pt": 32, "io": "bf16", "dt": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ranges; sizes spread over their logarithm, mostly odd."""
    op = rng.choice(["in_proj", "linear", "linear", "norm", "logprobs", "logprobs", "pages",
                     "fork", "compact"])
    if op == "in_proj":
        H = rng.choice([8, 12, 24, 32, 48, 64])
        c = {"op": op, "K": 8 * rng.randint(32, 256), "H": H, "G": rng.choice([1, 2, 4]), "P": 64,
             "N": rng.choice([64, 128]), "io": "bf16", "dt": rng.choice(["bf16", "f32"])}
        c["M"] = _log_int(rng, 1, 8192)
    elif op == "linear":
        io = rng.choice(["bf16", "bf16", "f32"])
        c = {"op": op, "K": 8 * rng.randint(16, 512), "N": _log_int(rng, 16, 10000), "io": io,
             "out": rng.choice([io, "f32"]), "act": rng.choice(["none", "silu", "gelu", "relu2"]),
             "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}
        # at most the largest listed product, a sixteenth of it in fp32
        top = 8192 * 2048 * 10304 // (1 if io == "bf16" else 16)
        c["M"] = _log_int(rng, 1, max(1, min(8192, top // (c["K"] * c["N"]))))
    elif op == "norm":
        g = rng.choice([1, 1, 2, 4, 8])
        H = g * rng.randint(1, 64 // g)
        c = {"op": op, "H": H, "P": rng.choice([16, 32, 64, 128]) if H <= 32 else 64, "groups": g,
             "io": rng.choice(["bf16", "f32"]), "before": rng.random() < 0.3}
        c["T"] = _log_int(rng, 1, 16384 if c["io"] == "bf16" else 8192)
    elif op == "logprobs":
        V = _log_int(rng, 500, 131072)
        c = {"op": op, "V": V, "io": rng.choice(["bf16", "f32"]),
             "k": rng.choice([0, 1, rng.randint(2, 32)]),
             "allowed": rng.choice([1.0, 1.0, rng.uniform(0.001, 0.5)])}
        c["T"] = _log_int(rng, 1, min(4096, 4096 * 50280 // (V * (1 if c["io"] == "bf16" else 2))))
    else:
        Q = rng.choice([64, 128, 256])
        c = {"op": op, "H": rng.randint(1, 16), "G": 1, "P": rng.choice([32, 64]),
             "N": rng.choice([32, 64, 128]), "Q": Q, "pt": rng.choice([16, 32, 64]),
             "io": rng.choice(["bf16", "bf16", "f32"]), "dt": rng.choice(["bf16", "f32"])}
        if op == "fork":
            c.update(sources=_log_int(rng, 1, 24), fan=rng.randint(1, 8), ended=rng.randint(1, 16))
            c["slots"] = c["sources"] * (1 + c["fan"]) + c["ended"] + rng.randint(0, 9)
        else:
            c["slots"] = _log_int(rng, 8, 512)
            if op == "pages":
                c["tokens"] = rng.randint(1, 24)
    return c


# ---- inputs ---------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return torch.randn(*shape, generator=g, device=DEV).mul_(scale).to(dtype)


def _proj_cols(c):
    hp = c["H"] * c["P"]
    return hp, hp + 2 * c["G"] * c["N"], c["H"]


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    io = DT[c["io"]]
    if c["op"] in ("in_proj", "linear"):
        n = sum(_proj_cols(c)) if c["op"] == "in_proj" else c["N"]
        s["x"] = _randn(g, c["M"], c["K"], dtype=io)
        s["w"] = _randn(g, n, c["K"], dtype=io, scale=c["K"] ** -0.5)
        if c["op"] == "linear":
            s["bias"] = _randn(g, n) if c["bias"] else None
            s["residual"] = _randn(g, c["M"], n, dtype=io) if c["residual"] else None
    elif c["op"] == "norm":
        s["y"] = _randn(g, c["T"], c["H"], c["P"], dtype=io, scale=2.0)
        s["z"] = _randn(g, c["T"], c["H"], c["P"], dtype=io)
        s["w"] = _randn(g, c["H"] * c["P"], scale=0.2) + 1.0
    elif c["op"] == "logprobs":
        x = _randn(g, c["T"], c["V"], scale=3.0)
        # a few tokens stand out in each row, as a trained model's logits do
        hot = torch.randint(0, c["V"], (c["T"], 8), generator=g, device=DEV)
        x.scatter_add_(1, hot, 8.0 * torch.rand(c["T"], 8, generator=g, device=DEV))
        tok = torch.where(torch.rand(c["T"], generator=g, device=DEV) < 0.6, hot[:, 0],
                          torch.randint(0, c["V"], (c["T"],), generator=g, device=DEV))
        if c["allowed"] < 1.0:
            off = torch.rand(c["T"], c["V"], generator=g, device=DEV) >= c["allowed"]
            off.scatter_(1, tok[:, None], False)
            x.masked_fill_(off, -math.inf)
        s["logits"] = x.to(io)
        s["tokens"] = tok.to(torch.int32)
    else:
        _prepare_cache(s, c, g)
    if own:
        import exact_replay_decode_amd as erd
        s["erd"] = erd
        if "H" in c and c["op"] != "norm":
            s["shape"] = erd.Shape(c["H"], c["G"], c["P"], c["N"], c.get("Q", 256), c["io"],
                                   c["dt"])
        elif c["op"] == "norm":
            s["shape"] = erd.Shape(c["H"], c["groups"], c["P"], 128, 256, c["io"], c["io"])
        if "table" in s:
            # the cache object a serving program holds, over the arrays made above
            cache = erd.ReplayCache(s["shape"], 1, DEV, page_tokens=c["pt"], num_pages=1)
            cache.num_slots, cache.num_pages = c["slots"], s["num_pages"]
            cache.buf_pages = s["table"]
            for name in ("state", "state_bf", "buf_x", "buf_dt", "buf_B", "buf_len",
                         "boundary_pos"):
                setattr(cache, name, s[name])
            cache.work = torch.zeros(2 * c["slots"] + 34, dtype=torch.int32, device=DEV)
            s["cache"] = cache
    return s


def _prepare_cache(s, c, g):
    """A paged replay cache in the middle of a run: every slot holds a different number of
    buffered tokens, its pages scattered over the pool."""
    S, H, G, P, N, Q, pt = (c[k] for k in ("slots", "H", "G", "P", "N", "Q", "pt"))
    npp = Q // pt if Q >= pt else 1
    pt = c["pt"] = min(pt, Q)
    num_pages = S * npp + 7
    io, dt = DT[c["io"]], DT[c["dt"]]
    s["num_pages"] = num_pages
    s["state"] = _randn(g, S, H, P, N)
    s["state_bf"] = _randn(g, S, H, N // 16, P, 16, dtype=torch.bfloat16)
    s["buf_x"] = _randn(g, num_pages, pt, H, P, dtype=io)
    s["buf_dt"] = _randn(g, num_pages, pt, H, dtype=dt)
    s["buf_B"] = _randn(g, num_pages, pt, G, N, dtype=io)
    s["buf_len"] = torch.randint(0, Q, (S,), generator=g, device=DEV, dtype=torch.int32)
    s["boundary_pos"] = Q * torch.randint(0, 9, (S,), generator=g, device=DEV)
    perm = torch.randperm(num_pages, generator=g, device=DEV)[:S * npp].reshape(S, npp)
    at = torch.arange(npp, device=DEV)[None]
    held = (s["buf_len"].long()[:, None] + pt - 1) // pt
    if c["op"] == "pages":
        # some slots hold pages past their buffered tokens (their chunk ended, drafts refused)
        held = held + (torch.rand(S, 1, generator=g, device=DEV) < 0.3) * 2
        s["order"] = torch.randperm(S, generator=g, device=DEV).to(torch.int32)
        s["tokens"] = torch.full((S,), c["tokens"], dtype=torch.int32, device=DEV)
    elif c["op"] == "fork":
        n = c["sources"] * c["fan"]
        order = torch.randperm(S, generator=g, device=DEV).to(torch.int32)
        s["src"] = order[:c["sources"]].repeat_interleave(c["fan"]).contiguous()
        s["dst"] = order[c["sources"]:c["sources"] + n].contiguous()
        s["ended"] = order[c["sources"] + n:c["sources"] + n + c["ended"]].contiguous()
        held[s["dst"].long()] = 0
    s["table"] = torch.where(at < held, perm, -1).to(torch.int32)
    if c["op"] in ("fork", "compact"):
        # the table as the run left it: a pass hands out or moves pages and rewrites the table,
        # and the next pass begins from this one again
        s["before"] = s["table"].clone()


# ---- one pass -------------------------------------------------------------

def _act(v, act):
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "relu2":
        return torch.clamp(v, min=0) ** 2
    return v


def _plain_linear(s):
    c = s["case"]
    r = s["x"].float() @ s["w"].float().t()
    if c["op"] == "in_proj":
        a, b, _ = _proj_cols(c)
        io = DT[c["io"]]
        return (r[:, :a].to(io).contiguous(), r[:, a:a + b].to(io).contiguous(),
                r[:, a + b:].to(DT[c["dt"]]).contiguous())
    if s["bias"] is not None:
        r = r + s["bias"]
    r = _act(r, c["act"])
    if s["residual"] is not None:
        r = r + s["residual"].float()
    return r.to(DT[c["out"]])


def _plain_norm(s):
    c = s["case"]
    y, z = (s[k].float().reshape(c["T"], c["groups"], -1) for k in ("y", "z"))
    gate = z / (1 + torch.exp(-z))
    v = y if c["before"] else y * gate
    v = v * torch.rsqrt((v * v).mean(dim=2, keepdim=True) + EPS) * s["w"].reshape(1, c["groups"],
                                                                                  -1)
    if c["before"]:
        v = v * gate
    return v.reshape(c["T"], c["H"], c["P"]).to(DT[c["io"]])


def _sort_keys(x):
    """Whole numbers whose descending order is that of (value descending, index ascending)."""
    bits = (x + 0.0).view(torch.int32).long()
    up = torch.where(bits >= 0, bits, -(bits & 0x7fffffff))
    return up * 2 ** 20 - torch.arange(x.shape[1], device=x.device)


def _plain_logprobs(s):
    c = s["case"]
    x, tok = s["logits"].float(), s["tokens"].long()[:, None]
    m = x.max(dim=1, keepdim=True).values
    e = torch.exp(x - m)
    z = e.sum(dim=1, keepdim=True)
    log_z = torch.log(z)
    entropy = log_z - torch.where(e > 0, e * (x - m), 0.0).sum(dim=1, keepdim=True) / z
    key = _sort_keys(x)
    out = {"logprob": (x.gather(1, tok) - m - log_z)[:, 0], "entropy": entropy[:, 0],
           "rank": (key > key.gather(1, tok)).sum(dim=1).to(torch.int32)}
    if c["k"]:
        top = key.topk(c["k"], dim=1).indices
        out["top_ids"] = top.to(torch.int32)
        out["top_logprobs"] = x.gather(1, top) - m - log_z
    return out


def _used_pages(s):
    t, n = s["table"].long(), s["num_pages"]
    used = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    used[torch.where((t >= 0) & (t < n), t, n).reshape(-1)] = 1
    return used[:n]


def _plain_trim(s, slots):
    c = s["case"]
    held = (s["buf_len"][slots] + c["pt"] - 1) // c["pt"]
    at = torch.arange(s["table"].shape[1], device=DEV)[None]
    s["table"][slots] = torch.where(at < held[:, None], s["table"][slots], -1)


def _plain_reserve(s, slots, like, tokens):
    """Pages for the first buf_len[like] + tokens positions of each slot (a chunk at most):
    requests in order, lowest free pages first, all of a slot's pages or none."""
    c, rows = s["case"], s["table"][slots].long()
    n = torch.clamp(s["buf_len"][like].long() + tokens, max=c["Q"])
    at = torch.arange(rows.shape[1], device=DEV)[None]
    lack = (at < ((n + c["pt"] - 1) // c["pt"])[:, None]) & ((rows < 0) | (rows >= s["num_pages"]))
    need = lack.sum(dim=1)
    upto = need.cumsum(0)
    used = _used_pages(s)
    free = used.argsort(stable=True)
    granted = (need == 0) | (upto <= (1 - used).sum())
    rank = (upto - need)[:, None] + lack.cumsum(dim=1) - 1
    page = free[rank.clamp(0, s["num_pages"] - 1)]
    s["table"][slots] = torch.where(lack & granted[:, None], page, rows).to(torch.int32)
    return granted.to(torch.int32)


def _plain_fork(s):
    c = s["case"]
    ended, src, dst = (s[k].long() for k in ("ended", "src", "dst"))
    s["table"].copy_(s["before"])
    s["table"][ended] = -1
    for name in ("state", "state_bf", "buf_len", "boundary_pos"):
        s[name][ended] = 0
    granted = _plain_reserve(s, dst, src, 0)
    n = s["buf_len"][src]
    pos = torch.arange(c["Q"], device=DEV)[None]
    live = pos < n[:, None]
    at = lambda slots: (s["table"][slots].long()[:, pos[0] // c["pt"]] * c["pt"]  # noqa: E731
                        + pos % c["pt"])[live]
    rows_from, rows_to = at(src), at(dst)
    for name in ("buf_x", "buf_dt", "buf_B"):
        rows = s[name].view(-1, *s[name].shape[2:])
        rows[rows_to] = rows[rows_from]
    for name in ("state", "state_bf", "buf_len", "boundary_pos"):
        s[name][dst] = s[name][src]
    return granted


def _plain_compact(s):
    """Used pages at or past the used count move to the free pages below it, both in order."""
    s["table"].copy_(s["before"])
    used = _used_pages(s)
    count = used.sum()
    page = torch.arange(s["num_pages"], device=DEV)
    moves = (used > 0) & (page >= count)
    free = used.argsort(stable=True)
    to = torch.where(moves, free[(moves.cumsum(0) - 1).clamp(min=0)], page)
    source = moves.nonzero()[:, 0]
    for name in ("buf_x", "buf_dt", "buf_B"):
        s[name][to[source]] = s[name][source]
    t = s["table"].long()
    ok = (t >= 0) & (t < s["num_pages"])
    s["table"].copy_(torch.where(ok, to[t.clamp(0, s["num_pages"] - 1)], t))
    return count.to(torch.int32).reshape(1)


def _cache_outputs(s, **more):
    return {**more, **{k: s[k] for k in ("table", "state", "state_bf", "buf_x", "buf_dt", "buf_B",
                                         "buf_len", "boundary_pos")}}


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        return _own(s, c, op)
    if op in ("in_proj", "linear"):
        return _plain_linear(s)
    if op == "norm":
        return _plain_norm(s)
    if op == "logprobs":
        return _plain_logprobs(s)
    if op == "pages":
        slots = s["order"].long()
        _plain_trim(s, slots)
        granted = _plain_reserve(s, slots, slots, s["tokens"].long())
        return {"granted": granted, "table": s["table"]}
    if op == "fork":
        return _cache_outputs(s, granted=_plain_fork(s))
    return _cache_outputs(s, used=_plain_compact(s))


def _own(s, c, op):
    erd = s["erd"]
    if op == "in_proj":
        z, xBC, dt = erd.ssd_in_proj(s["shape"], s["x"], s["w"])
        return z.view(c["M"], -1), xBC, dt
    if op == "linear":
        return erd.ssd_linear(s["x"], s["w"], bias=s["bias"], activation=c["act"],
                              residual=s["residual"], out_dtype=DT[c["out"]])
    if op == "norm":
        return erd.ssd_gated_norm(s["shape"], s["y"], s["w"], z=s["z"], groups=c["groups"],
                                  eps=EPS, norm_before_gate=c["before"])
    if op == "logprobs":
        r = erd.ssd_token_logprobs(s["logits"], s["tokens"], top_k=c["k"])
        out = {"logprob": r.logprob, "entropy": r.entropy, "rank": r.rank}
        if c["k"]:
            out.update(top_ids=r.top_ids, top_logprobs=r.top_logprobs)
        return out
    shape, cache = s["shape"], s["cache"]
    if op == "pages":
        erd.ssd_replay_pages_trim(shape, cache, slot_idx=s["order"])
        granted = erd.ssd_replay_pages_reserve(shape, cache, s["tokens"], slot_idx=s["order"])
        return {"granted": granted, "table": s["table"]}
    if op == "fork":
        s["table"].copy_(s["before"])
        erd.ssd_replay_cache_free(shape, cache, slot_idx=s["ended"])
        granted = erd.ssd_replay_pages_reserve(shape, cache, 0, slot_idx=s["dst"],
                                               like_idx=s["src"])
        erd.ssd_replay_cache_copy(shape, cache, cache, s["dst"], s["src"])
        return _cache_outputs(s, granted=granted)
    s["table"].copy_(s["before"])
    return _cache_outputs(s, used=erd.ssd_replay_pages_compact(shape, cache))


# ---- what a pass cannot do without ----------------------------------------

def work(case):
    c = case
    b = {"bf16": 2, "f32": 4}
    io = b[c["io"]]
    if c["op"] in ("in_proj", "linear"):
        if c["op"] == "in_proj":
            z, xbc, d = _proj_cols(c)
            n, written = z + xbc + d, (z + xbc) * io + d * b[c["dt"]]
            extra = 0
        else:
            n, written = c["N"], c["N"] * b[c["out"]]
            extra = (4 * n if c["bias"] else 0) + (c["M"] * n * io if c["residual"] else 0)
        return {"bytes": (c["M"] + n) * c["K"] * io + c["M"] * written + extra,
                "flops": 2 * c["M"] * n * c["K"]}
    if c["op"] == "norm":
        n = c["T"] * c["H"] * c["P"]
        return {"bytes": 3 * n * io + 4 * c["H"] * c["P"], "flops": 12 * n}
    if c["op"] == "logprobs":
        n = c["T"] * c["V"]
        return {"bytes": n * io + c["T"] * (16 + 8 * c["k"]), "flops": 6 * n}
    pt = min(c["pt"], c["Q"])
    npp = c["Q"] // pt
    table = 4 * c["slots"] * npp
    row = c["H"] * c["P"] * io + c["H"] * b[c["dt"]] + c["G"] * c["N"] * io
    state = c["H"] * c["P"] * c["N"] * 6
    if c["op"] == "pages":
        return {"bytes": 2 * table + 16 * c["slots"], "flops": 0}
    if c["op"] == "fork":
        n, mean = c["sources"] * c["fan"], (c["Q"] - 1) / 2
        return {"bytes": 2 * table + c["ended"] * state + (c["sources"] + n) * (state + mean * row),
                "flops": 0}
    held = c["slots"] * sum((k + pt - 1) // pt for k in range(c["Q"])) / c["Q"]
    pages = c["slots"] * npp + 7
    return {"bytes": 2 * table + 2 * held * (1 - held / pages) * pt * row, "flops": 0}


# ---- the same in 64 bits, from the definitions ----------------------------

def _exact_act(v, act):
    if act == "silu":
        return v * torch.special.expit(v)
    if act == "gelu":
        return v * torch.special.expit(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    if act == "relu2":
        return torch.where(v > 0, v * v, torch.zeros_like(v))
    return v


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    c = case
    if c["op"] in ("in_proj", "linear"):
        v = torch.mm(s["w"].double(), s["x"].double().t().contiguous()).t()
        if c["op"] == "in_proj":
            return tuple(p.contiguous() for p in v.split(list(_proj_cols(c)), dim=1))
        if c["bias"]:
            v = v + s["bias"].double()[None]
        v = _exact_act(v, c["act"])
        return v + s["residual"].double() if c["residual"] else v.contiguous()
    if c["op"] == "norm":
        y, z, w = (s[k].double().flatten(1) if k != "w" else s[k].double() for k in "yzw")
        gate = z * torch.special.expit(z)
        v = y if c["before"] else y * gate
        rms = (v.unflatten(1, (c["groups"], -1)).square().mean(2) + EPS).sqrt()
        v = v / rms.repeat_interleave(v.shape[1] // c["groups"], dim=1) * w
        return (v * gate if c["before"] else v).reshape(c["T"], c["H"], c["P"])
    if c["op"] == "logprobs":
        x = s["logits"].double()
        lse = torch.logsumexp(x, dim=1)
        lp = x - lse[:, None]
        out = {"logprob": lp[torch.arange(c["T"], device=DEV), s["tokens"].long()],
               "entropy": -torch.special.xlogy(lp.exp(), lp.exp()).sum(1), "rank": None}
        if c["k"]:
            out["top_ids"] = None
            out["top_logprobs"] = lp.topk(c["k"], dim=1).values
        return out
    return _exact_pages(s, c)


def _exact_pages(s, c):
    """Slot by slot and page by page, on the host."""
    t, S, Q, pt = s["table"].cpu().tolist(), c["slots"], c["Q"], c["pt"]
    lens = s["buf_len"].cpu().tolist()

    def free():
        taken = {p for row in t for p in row if p >= 0}
        return [p for p in range(s["num_pages"]) if p not in taken]

    def reserve(slots, like, tokens):
        pool, got, asked = free(), [], 0
        room = len(pool)
        for b, (d, l) in enumerate(zip(slots, like)):
            n = -(-min(lens[l] + tokens, Q) // pt)
            lack = [i for i in range(n) if t[d][i] < 0]
            asked += len(lack)
            got.append(int(not lack or asked <= room))
            if got[-1]:
                for i in lack:
                    t[d][i] = pool.pop(0)
        return got

    if c["op"] == "pages":
        order = s["order"].cpu().tolist()
        for d in order:
            t[d] = [p if i * pt < lens[d] else -1 for i, p in enumerate(t[d])]
        got = reserve(order, order, c["tokens"])
        return {"granted": torch.tensor(got, dtype=torch.int32),
                "table": torch.tensor(t, dtype=torch.int32)}
    if c["op"] == "fork":
        for d in s["ended"].cpu().tolist():
            t[d] = [-1] * len(t[d])
            lens[d] = 0
            for name in ("state", "state_bf", "buf_len", "boundary_pos"):
                s[name][d].zero_()
        src, dst = s["src"].cpu().tolist(), s["dst"].cpu().tolist()
        first = {"granted": torch.tensor(reserve(dst, src, 0), dtype=torch.int32)}
        for a, d in zip(src, dst):
            for i in range(-(-lens[a] // pt)):
                rows = min(pt, lens[a] - i * pt)
                for name in ("buf_x", "buf_dt", "buf_B"):
                    s[name][t[d][i], :rows] = s[name][t[a][i], :rows]
            for name in ("state", "state_bf", "buf_len", "boundary_pos"):
                s[name][d] = s[name][a]
    else:
        pool, used = free(), sorted(p for row in t for p in row if p >= 0)
        to = dict(zip([p for p in used if p >= len(used)], pool))
        for a, d in to.items():
            for name in ("buf_x", "buf_dt", "buf_B"):
                s[name][d] = s[name][a]
        t = [[to.get(p, p) for p in row] for row in t]
        first = {"used": torch.tensor([len(used)], dtype=torch.int32)}
    s["table"] = torch.tensor(t, dtype=torch.int32, device=DEV)
    return _cache_outputs(s, **first)
