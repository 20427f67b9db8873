"""Cases of the serving operators around the gated maps of a decoder layer.

Four operators, each in its plain form (elementary torch operations in 32
bits) and as the calls a user makes of the library:

  plan       block tables and slot maps from request lengths (`paged_plan`)
  append     the rows of the qkv map split into queries and the new tokens'
             keys and values, stored in a paged cache (`cache_append`)
  attention  a chunk of new tokens of every request over the paged cache
             (`paged_attention`)
  norm       the norms after and before a block, with the block's gate and
             the residual scale (`norm_residual`)
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a small batch: every request adds one token
        dict(name="plan, 16 requests, a token each", op="plan", requests=16, page=16, cached=2000, chunk=1, every=1),
        # a large server's step: mostly single tokens, every 16th request brings a chunk of its prompt
        dict(name="plan, 4093 requests, mixed", op="plan", requests=4093, page=16, cached=4001, chunk=513, every=16),
        # the qkv map's rows of 16 decode tokens of a 13B layer (5120 wide)
        dict(name="append, 16 tokens, 40 x 128", op="append", tokens=16, q_heads=40, kv_heads=40, dim=128, page=16,
             rows="f32", cache="bf16"),
        # the qkv map's rows of a 2048-token prompt of a 6B layer (4096 wide)
        dict(name="append, 2048 tokens, 16 x 256", op="append", tokens=2048, q_heads=16, kv_heads=16, dim=256, page=64,
             rows="f32", cache="bf16"),
        # batch-1 decode of a 6B layer
        dict(name="decode, 1 token, 2048 keys, 16 x 256", op="attention", requests=1, chunk=1, keys=2048, q_heads=16,
             kv_heads=16, dim=256, page=16, cache="bf16", window=0, spare=0),
        # 16 sequences of very different lengths in one decode step of a 13B layer
        dict(name="decode, 16 requests, 8191 keys, 40 x 128", op="attention", requests=16, chunk=1, keys=8191,
             q_heads=40, kv_heads=40, dim=128, page=16, cache="bf16", window=0, spare=0),
        # one token far into a long document, grouped heads, in a cache of more than 2^31 elements
        dict(name="decode, 1 token, 260001 keys, 32/8 x 128", op="attention", requests=1, chunk=1, keys=260001,
             q_heads=32, kv_heads=8, dim=128, page=64, cache="bf16", window=0, spare=1850000),
        # a whole prompt of a 6B layer
        dict(name="prefill, 2048 tokens, 16 x 256", op="attention", requests=1, chunk=2048, keys=2048, q_heads=16,
             kv_heads=16, dim=256, page=64, cache="bf16", window=0, spare=0),
        # prompt chunks of several requests, each behind what it has cached
        dict(name="chunks, 5 requests, 509 of 8003, 32/8 x 128", op="attention", requests=5, chunk=509, keys=8003,
             q_heads=32, kv_heads=8, dim=128, page=32, cache="bf16", window=0, spare=0),
        # the float32 model of 256 channels with a sliding window
        dict(name="f32 chunks, window 128, 4 x 64", op="attention", requests=3, chunk=64, keys=600, q_heads=4,
             kv_heads=4, dim=64, page=16, cache="f32", window=128, spare=0),
        # one decode token of a 6B layer between its attention and its MLP
        dict(name="norm, 1 token, 4096", op="norm", tokens=1, width=4096, post="rms", pre="rms", gate="row", x="bf16",
             h="f32", y="f32"),
        # a prompt of a 13B layer, a gate for each of its requests
        dict(name="norm, 2049 tokens, 5120", op="norm", tokens=2049, width=5120, post="layer", pre="layer",
             gate="request", x="bf16", h="f32", y="f32"),
    ]


def _between(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(max(n, lo), hi)
    return n


def draw(rng):
    while True:
        case = _drawn(rng)
        if 3072 not in case.values():
            return case


def _drawn(rng):
    op = rng.choice(["plan", "append", "attention", "attention", "attention", "norm"])
    if op == "plan":
        return dict(op=op, requests=_between(rng, 1, 4000), page=rng.choice([16, 32, 64]), cached=_between(rng, 1, 4000),
                    chunk=_between(rng, 1, 512), every=_between(rng, 1, 16))
    if op == "append":
        kv = rng.choice([1, 2, 4, 8, 16])
        return dict(op=op, tokens=_between(rng, 1, 2048), q_heads=kv * rng.choice([1, 2, 3, 4]) if kv < 16 else 16,
                    kv_heads=kv, dim=rng.choice([64, 80, 128, 256] if kv < 16 else [64, 128, 256]),
                    page=rng.choice([16, 32, 64, 128]), rows=rng.choice(["f32", "f32", "bf16"]),
                    cache=rng.choice(["bf16", "bf16", "f32"]))
    if op == "norm":
        return dict(op=op, tokens=_between(rng, 1, 2049), width=8 * _between(rng, 16, 640) + 8 * rng.choice([0, 1]),
                    post=rng.choice(["none", "rms", "layer"]), pre=rng.choice(["rms", "layer"]),
                    gate=rng.choice(["none", "row", "request"]), x=rng.choice(["bf16", "f32"]),
                    h=rng.choice(["f32", "bf16"]), y=rng.choice(["f32", "bf16"]))
    cache = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dim = rng.choice([64, 80, 96, 128, 256] if cache == "bf16" else [32, 64, 128])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 1, 2, 3, 4, 8])
    requests = _between(rng, 1, 24)
    keys = _between(rng, 1, 16384 if cache == "bf16" else 2048)
    chunk = 1 if rng.random() < 0.4 else _between(rng, 1, 1024 if cache == "bf16" else 256)
    while requests * kv * group * chunk * keys > 3 * 10**8:
        chunk, keys, requests = (chunk + 1) // 2, max(1, keys - keys // 3), (requests + 1) // 2
    return dict(op=op, requests=requests, chunk=min(chunk, keys), keys=keys, q_heads=kv * group, kv_heads=kv, dim=dim,
                page=rng.choice([16, 32, 64, 128]), cache=cache, window=rng.choice([0, 0, 0, _between(rng, 8, 1024)]),
                spare=0)


# ------------------------------------------------------------------ inputs
def _spread(count, most):
    """`count` lengths from about an eighth of `most` up to `most`, the first of them `most` itself."""
    return [most if i == 0 else max(1, int(most * (0.125 + 0.875 * ((i * 0.6180339887) % 1.0)))) for i in range(count)]


def _lengths(case):
    """New tokens and cached tokens of each request, in an order of their own."""
    n = case["requests"]
    if case["op"] == "plan":
        fresh = [f if i % case["every"] == 0 else 1 for i, f in enumerate(_spread(n, case["chunk"]))]
        return fresh, _spread(n, case["cached"])
    fresh, total = _spread(n, case["chunk"]), _spread(n, case["keys"])
    fresh = [min(f, t) for f, t in zip(fresh, total)]
    return fresh, [t - f for f, t in zip(fresh, total)]


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    order = torch.Generator().manual_seed(int(seed))
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    s = dict(case=case)
    if case["op"] == "norm":
        T, d = case["tokens"], case["width"]
        s["h"] = normal(T, d).mul_(3.0).to(DTYPES[case["h"]])
        s["y"] = normal(T, d).mul_(0.7).to(DTYPES[case["y"]])
        s["weights"] = [1.0 + 0.1 * normal(d), 0.1 * normal(d), 1.0 + 0.1 * normal(d), 0.1 * normal(d)]
        requests = max(1, T // 400) if case["gate"] == "request" else 1
        s["gate"] = 0.3 * normal(requests, d) if case["gate"] != "none" else None
        s["which"] = (torch.arange(T, device="cuda") % requests).sort().values.int() if case["gate"] == "request" else None
        s["h_out"] = torch.empty_like(s["h"])
        s["x"] = torch.empty(T, d, dtype=DTYPES[case["x"]], device="cuda")
        return s
    page = case["page"]
    if case["op"] == "append":
        T, hq, hkv, D = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        pages = 2 * -(-T // page)
        s["rows"] = normal(T, (hq + 2 * hkv) * D).to(DTYPES[case["rows"]])
        s["K"], s["V"] = (normal(pages, hkv, page, D).to(DTYPES[case["cache"]]) for _ in range(2))
        at = torch.randperm(pages, generator=g, device="cuda")[torch.arange(T, device="cuda") // page]
        s["slots"] = at * page + torch.arange(T, device="cuda") % page
        s["Q"] = torch.empty(T, hq, D, dtype=DTYPES[case["cache"]], device="cuda")
        return s
    fresh, cached = _lengths(case)
    mixed = torch.randperm(len(fresh), generator=order).tolist()
    fresh, cached = [fresh[i] for i in mixed], [cached[i] for i in mixed]
    total = [f + c for f, c in zip(fresh, cached)]
    held = [-(-(c if case["op"] == "plan" else t) // page) for c, t in zip(cached, total)]
    wanted = [-(-t // page) for t in total]
    width, N = max(wanted), sum(fresh)
    pages = sum(wanted) + 8 + case.get("spare", 0) // page
    ids = torch.randperm(pages, generator=g, device="cuda").int()
    have = _ints(held)
    first = have.cumsum(0) - have
    col = torch.arange(width, device="cuda")
    table = ids[(first[:, None] + col).clamp(max=pages - 1)]
    s["table"] = torch.where(col < have[:, None], table, -1).int().contiguous()
    s["tokens"], s["max_q"], s["max_kv"] = N, max(fresh), max(total)
    if case["op"] == "plan":
        s["fresh"], s["cached"] = _ints(fresh), _ints(cached)
        s["free"], s["n_free"] = ids[sum(held):].contiguous(), _ints([pages - sum(held)])
        like = lambda n, dtype=torch.int32: torch.empty(n, dtype=dtype, device="cuda")  # noqa: E731
        s["plan"] = dict(q_start=like(len(fresh) + 1), kv_len=like(len(fresh)), slots=like(N, torch.int64),
                         token_req=like(N), positions=like(N), n_free=like(1), status=like(1))
        return s
    hq, hkv, D, dt = case["q_heads"], case["kv_heads"], case["dim"], DTYPES[case["cache"]]
    s["K"], s["V"] = (torch.empty(pages, hkv, page, D, dtype=dt, device="cuda").normal_(generator=g) for _ in range(2))
    s["q"] = normal(N, hq, D).mul_(2.0).to(dt)
    s["q_start"] = _ints([0] + torch.tensor(fresh).cumsum(0).tolist())
    s["kv_len"] = _ints(total)
    s["out"] = torch.empty_like(s["q"])
    s["workspace"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device="cuda")
    return s


WORKSPACE = 96 << 20  # the attention's workspace: zeroed once and kept, as a server keeps it


# ------------------------------------------------------------------ one pass
def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_plan(s):
    import gated_rank_subspace_gb300 as gsi
    p = gsi.paged_plan(s["cached"], s["fresh"], s["table"], s["free"], s["n_free"], s["case"]["page"],
                       plan=gsi.PagedPlan(**s["plan"]))
    return [p.q_start, p.kv_len, p.slots, p.token_req, p.positions, s["table"], p.n_free, p.status]


def _plain_plan(s):
    page, N, cached, fresh = s["case"]["page"], s["tokens"], s["cached"].long(), s["fresh"].long()
    dev = cached.device
    total = cached + fresh
    ends = fresh.cumsum(0)
    q_start = torch.cat([ends.new_zeros(1), ends])
    held = (cached + page - 1) // page
    need = (total + page - 1) // page - held
    before = need.cumsum(0) - need
    left = s["n_free"].long() - need.sum()
    col = torch.arange(s["table"].shape[1], device=dev)
    nth = before[:, None] + col - held[:, None]
    added = (col >= held[:, None]) & (col < (held + need)[:, None])
    popped = s["free"][(s["n_free"].long() - 1 - nth).clamp(0, s["free"].numel() - 1)]
    table = torch.where(added, popped, s["table"])
    token = torch.arange(N, device=dev)
    req = (torch.searchsorted(q_start, token, right=True) - 1).clamp(0, fresh.numel() - 1)
    pos = cached[req] + token - q_start[req]
    slots = table[req, pos // page].long() * page + pos % page
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    return [q_start.int(), total.int(), slots, req.int(), pos.int(), table, left.int(), status]


def _own_append(s):
    import gated_rank_subspace_gb300 as gsi
    cache = gsi.PagedCache(s["K"], s["V"])
    gsi.cache_append(cache, s["rows"], s["slots"], s["case"]["q_heads"], Q=s["Q"])
    return [s["Q"], s["K"], s["V"]]


def _plain_append(s):
    c = s["case"]
    hq, hkv, D, T = c["q_heads"], c["kv_heads"], c["dim"], c["tokens"]
    rows = s["rows"].float().view(T, hq + 2 * hkv, D).to(s["K"].dtype)
    at, off = s["slots"] // c["page"], s["slots"] % c["page"]
    s["K"][at, :, off] = rows[:, hq:hq + hkv]
    s["V"][at, :, off] = rows[:, hq + hkv:]
    return [rows[:, :hq].contiguous(), s["K"], s["V"]]


def _own_attention(s):
    import gated_rank_subspace_gb300 as gsi
    return gsi.paged_attention(gsi.PagedCache(s["K"], s["V"]), s["q"], s["q_start"], s["kv_len"], s["table"],
                               max_q=s["max_q"], window=s["case"]["window"], out=s["out"], workspace=s["workspace"])


def _plain_attention(s):
    c, dev = s["case"], s["q"].device
    page, hq, hkv, D, R = c["page"], c["q_heads"], c["kv_heads"], c["dim"], c["requests"]
    q_len, start = s["q_start"][1:] - s["q_start"][:-1], s["q_start"][:-1].long()
    row, key = torch.arange(s["max_q"], device=dev), torch.arange(s["max_kv"], device=dev)
    q = s["q"].float()[(start[:, None] + row).clamp(max=s["tokens"] - 1)]
    q = q.view(R, s["max_q"], hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(R, hkv, -1, D)
    at, off = s["table"].long()[:, key // page].clamp(min=0), (key % page).expand(R, -1)
    k, v = (t[at, :, off].float().transpose(1, 2) for t in (s["K"], s["V"]))
    there = key < s["kv_len"][:, None]
    v = torch.where(there[:, None, :, None], v, 0.0)
    lim = (s["kv_len"] - q_len)[:, None] + row + 1
    seen = (key < lim[..., None]) & there[:, None]
    if c["window"]:
        seen = seen & (key >= (lim - c["window"])[..., None])
    scores = (q @ k.transpose(2, 3)).view(R, hkv, hq // hkv, s["max_q"], -1) / math.sqrt(D)
    scores = torch.where(seen[:, None, None], scores, -math.inf)
    p = torch.exp(scores - scores.amax(-1, keepdim=True).clamp(min=-3e38))
    o = p.view(R, hkv, -1, s["max_kv"]) @ v
    o = o.view(R, hkv, hq // hkv, s["max_q"], D) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    token = torch.arange(s["tokens"], device=dev)
    req = torch.searchsorted(s["q_start"], token, right=True) - 1
    o = o.permute(0, 3, 1, 2, 4).reshape(R, s["max_q"], hq, D)
    return o[req, token - start[req]].to(s["q"].dtype)


def _own_norm(s):
    import gated_rank_subspace_gb300 as gsi
    c, w = s["case"], s["weights"]
    post = None if c["post"] == "none" else gsi.Norm(c["post"], w[0], w[1] if c["post"] == "layer" else None)
    pre = gsi.Norm(c["pre"], w[2], w[3] if c["pre"] == "layer" else None)
    return gsi.norm_residual(s["h"], s["y"], post=post, pre=pre, gate=s["gate"], gate_index=s["which"], alpha=0.9,
                             h_out=s["h_out"], x=s["x"])


def _plain_norm(s):
    c, w = s["case"], s["weights"]

    def norm(kind, t, weight, bias):
        if kind == "none":
            return t
        if kind == "layer":
            t = t - t.mean(-1, keepdim=True)
        t = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-5) * weight
        return t + bias if kind == "layer" else t

    y = norm(c["post"], s["y"].float(), w[0], w[1])
    if s["gate"] is not None:
        y = y * (s["gate"] if s["which"] is None else s["gate"][s["which"].long()])
    h = 0.9 * s["h"].float() + y
    return [h.to(s["h"].dtype), norm(c["pre"], h, w[2], w[3]).to(s["x"].dtype)]


_own = {"plan": _own_plan, "append": _own_append, "attention": _own_attention, "norm": _own_norm}
_plain = {"plan": _plain_plan, "append": _plain_append, "attention": _plain_attention, "norm": _plain_norm}


# ------------------------------------------------------------------ what a pass has to do
def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "norm":
        T, d = case["tokens"], case["width"]
        gates = {"none": 0, "row": 1, "request": max(1, T // 400)}[case["gate"]]
        params = {"none": 0, "rms": 1, "layer": 2}
        small = 4 * d * (gates + params[case["post"]] + params[case["pre"]]) + (4 * T if case["gate"] == "request" else 0)
        return {"bytes": T * d * (2 * size[case["h"]] + size[case["y"]] + size[case["x"]]) + small, "flops": 16 * T * d}
    if case["op"] == "append":
        values = case["tokens"] * (case["q_heads"] + 2 * case["kv_heads"]) * case["dim"]
        return {"bytes": values * (size[case["rows"]] + size[case["cache"]]) + 8 * case["tokens"], "flops": 0}
    fresh, cached = _lengths(case)
    page, R, N = case["page"], case["requests"], sum(fresh)
    if case["op"] == "plan":
        added = sum(-(-(c + f) // page) - -(-c // page) for c, f in zip(cached, fresh))
        # lengths in; starts, lengths, a slot, a request and a position for each token out; pages popped into the
        # table, and the page that each request's new tokens begin in
        return {"bytes": 4 * (5 * R + 1) + 16 * N + 8 * added, "flops": 0}
    hq, hkv, D, window = case["q_heads"], case["kv_heads"], case["dim"], case["window"]
    pairs = keys = 0
    for f, c in zip(fresh, cached):
        first = max(0, c + 1 - window) if window else 0
        keys += c + f - first
        full = min(f, max(0, window - c)) if window else f  # rows whose window has not filled yet
        pairs += full * c + full * (full + 1) // 2 + (f - full) * window
    pages = sum(-(-(c + f) // page) for c, f in zip(cached, fresh))
    return {"bytes": size[case["cache"]] * D * (2 * hkv * keys + 2 * hq * N) + 4 * (pages + 2 * R + 1),
            "flops": 4 * D * hq * pairs}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "append": _exact_append, "attention": _exact_attention, "norm": _exact_norm}[case["op"]](s)


def _exact_plan(s):
    page, free, table = s["case"]["page"], s["free"].tolist(), s["table"].tolist()
    left, starts, lens, slots, reqs, places = s["n_free"].item(), [0], [], [], [], []
    for r, (have, more) in enumerate(zip(s["cached"].tolist(), s["fresh"].tolist())):
        for place in range(have, have + more):
            if place % page == 0:
                left -= 1
                table[r][place // page] = free[left]
            slots.append(table[r][place // page] * page + place % page)
            reqs.append(r)
            places.append(place)
        starts.append(starts[-1] + more)
        lens.append(have + more)
    return [_ints(starts), _ints(lens), _ints(slots, torch.int64), _ints(reqs), _ints(places), _ints(table), _ints([left]),
            _ints([0])]


def _exact_append(s):
    T, hkv, D = s["rows"].shape[0], s["case"]["kv_heads"], s["case"]["dim"]
    K, V, rows = s["K"].double(), s["V"].double(), s["rows"].double()
    kv = hkv * D
    for t, slot in enumerate(s["slots"].tolist()):
        page, off = divmod(slot, s["case"]["page"])
        K[page, :, off] = rows[t, -2 * kv:-kv].view(hkv, D)
        V[page, :, off] = rows[t, -kv:].view(hkv, D)
    return [rows[:, :-2 * kv].reshape(T, -1, D), K, V]


def _exact_attention(s):
    c = s["case"]
    page, group, D = c["page"], c["q_heads"] // c["kv_heads"], c["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    starts, lens, table = s["q_start"].tolist(), s["kv_len"].tolist(), s["table"].tolist()
    for r, total in enumerate(lens):
        lo, hi = starts[r], starts[r + 1]
        pages = torch.tensor(table[r][:-(-total // page)], device="cuda")
        for head in range(c["kv_heads"]):
            k = s["K"][pages, head].reshape(-1, D)[:total].double()
            v = s["V"][pages, head].reshape(-1, D)[:total].double()
            for a in range(lo, hi, 256):
                b = min(a + 256, hi)
                # token t of the chunk stands at place total - (hi - t) of its sequence
                place = torch.arange(a, b, device="cuda") + total - hi
                behind = place[:, None] - torch.arange(total, device="cuda")
                hidden = behind < 0
                if c["window"]:
                    hidden = hidden | (behind >= c["window"])
                for h in range(head * group, (head + 1) * group):
                    w = s["q"][a:b, h].double() @ k.T / D**0.5
                    out[a:b, h] = torch.softmax(w.masked_fill(hidden, -math.inf), -1) @ v
    return out


def _exact_norm(s):
    c, (w0, b0, w1, b1) = s["case"], [w.double() for w in s["weights"]]
    y, h = s["y"].double(), s["h"].double()
    if c["post"] == "rms":
        y = y / (y.square().mean(1, keepdim=True) + 1e-5).sqrt() * w0
    if c["post"] == "layer":
        y = (y - y.mean(1, keepdim=True)) / (y.var(1, correction=0, keepdim=True) + 1e-5).sqrt() * w0 + b0
    if c["gate"] == "row":
        y = y * s["gate"].double()
    if c["gate"] == "request":
        y = y * s["gate"].double().index_select(0, s["which"].long())
    h = 0.9 * h + y
    if c["pre"] == "rms":
        return [h, h / (h.square().mean(1, keepdim=True) + 1e-5).sqrt() * w1]
    return [h, (h - h.mean(1, keepdim=True)) / (h.var(1, correction=0, keepdim=True) + 1e-5).sqrt() * w1 + b1]
