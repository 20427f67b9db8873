"""Cases of the serving operators for long contexts and drafted tokens.

Five operators, each in its plain form (elementary torch operations in 32
bits, in 64 where angles, long sums or comparisons need them) and as the calls
a user makes of the library:

  rotary   the rows of the qkv map split, queries and keys turned by their
           positions' angles, keys and values stored in a paged cache
           (`rotary_append`)
  weights  the attention weight that every cached key received from a step's
           tokens, added to what it has gathered (`key_weights`)
  evict    the keys of little weight leave the cache, the kept ones close the
           gaps (`cache_evict`)
  verify   drafted tokens accepted or rejected against the target's
           probabilities, one more token sampled (`verify_drafts`)
  trim     pages that requests no longer fill go back to the free ones
           (`paged_trim`)
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # batch-1 decode far into a long document, grouped heads, angles scaled for long contexts
        dict(name="rotary, 1 token at 260001, 32/8 x 128", op="rotary", tokens=1, first=260001, q_heads=32, kv_heads=8, dim=128,
             turned=128, layout="half", scaling="yarn", page=16, rows="f32", cache="bf16"),
        # a prompt of a 6B layer (4096 wide): a quarter of each head is turned, neighbouring values in pairs
        dict(name="rotary, 2048 tokens, 64 of 16 x 256", op="rotary", tokens=2048, first=0, q_heads=16, kv_heads=16, dim=256,
             turned=64, layout="pairs", scaling="none", page=64, rows="f32", cache="bf16"),
        # one decode step of 16 sequences of very different lengths, a 13B layer's heads
        dict(name="weights, 16 requests, 8191 keys, 40 x 128", op="weights", requests=16, chunk=1, keys=8191, q_heads=40,
             kv_heads=40, dim=128, page=16, cache="bf16", fresh_marks=False),
        # the last tokens of long prompts look back at all of them, before they are thinned out
        dict(name="weights, last 32 of 8003, 5 requests, 32/8 x 128", op="weights", requests=5, chunk=32, keys=8003, q_heads=32,
             kv_heads=8, dim=128, page=32, cache="bf16", fresh_marks=True),
        # every token of a 6B layer's prompt counts
        dict(name="weights, prompt of 2048, 16 x 256", op="weights", requests=1, chunk=2048, keys=2048, q_heads=16, kv_heads=16,
             dim=256, page=64, cache="bf16", fresh_marks=True),
        # the float32 model of 256 channels
        dict(name="weights, f32, 64 of 600, 4 x 64", op="weights", requests=3, chunk=64, keys=600, q_heads=4, kv_heads=4, dim=64,
             page=16, cache="f32", fresh_marks=False),
        # a decode step of 16 requests whose caches are full: every head gives up one key
        dict(name="evict, 16 requests, 1025 to 1024, 8 x 128", op="evict", requests=16, keys=1025, least=1025, budget=1024, recent=64,
             sinks=4, kv_heads=8, dim=128, page=16, cache="bf16"),
        # prompts of a 6B layer thinned out before decoding
        dict(name="evict, 5 requests, 8003 to 2048, 16 x 256", op="evict", requests=5, keys=8003, least=1000, budget=2048, recent=128,
             sinks=4, kv_heads=16, dim=256, page=64, cache="bf16"),
        # four drafted tokens of one sequence, an odd vocabulary
        dict(name="verify, 1 request, 4 drafts of 50257", op="verify", requests=1, drafts=4, vocab=50257, target="f32", draft="f32"),
        # a busy server's step with up to seven drafts a sequence
        dict(name="verify, 64 requests, 7 drafts of 100003", op="verify", requests=64, drafts=7, vocab=100003, target="f32",
             draft="f32"),
        # rejected drafts of 16 requests give their places back
        dict(name="trim, 16 requests, up to 7 places", op="trim", requests=16, page=16, keys=4001, back=7, every=0),
        # a large server's step: every 16th request has finished
        dict(name="trim, 4093 requests, some finished", op="trim", requests=4093, page=16, keys=4001, back=7, every=16),
    ]


def _between(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(n, lo), hi)


def draw(rng):
    op = rng.choice(["rotary", "weights", "weights", "evict", "evict", "verify", "trim"])
    page = rng.choice([16, 32, 64, 128])
    if op == "trim":
        return dict(op=op, requests=_between(rng, 1, 4000), page=page, keys=_between(rng, 8, 4000), back=_between(rng, 1, 8),
                    every=rng.choice([0, _between(rng, 1, 64)]))
    if op == "verify":
        requests = _between(rng, 1, 64)
        return dict(op=op, requests=requests, drafts=_between(rng, 1, 7), vocab=_between(rng, 1000, 100003),
                    target=rng.choice(["f32", "f32", "bf16"]), draft=rng.choice(["f32", "f32", "bf16", "none"]))
    cache = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dim = rng.choice([64, 80, 96, 128, 256] if cache == "bf16" else [32, 64, 128])
    kv = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 1, 2, 3, 4, 8])
    if op == "rotary":
        return dict(op=op, tokens=_between(rng, 1, 2048), first=rng.choice([0, _between(rng, 1, 10**6)]),
                    q_heads=kv * group if kv < 8 else kv, kv_heads=kv, dim=dim, turned=rng.choice([dim, dim // 2, dim // 4, 20]),
                    layout=rng.choice(["half", "pairs"]), scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]), page=page,
                    rows=rng.choice(["f32", "f32", "bf16"]), cache=cache)
    if op == "evict":
        keys = _between(rng, 2, 8003)
        budget = _between(rng, 1, keys)
        requests = min(_between(rng, 1, 24), 5 * 16 * 8003 // (kv * keys))
        return dict(op=op, requests=requests, keys=keys, least=rng.choice([keys, _between(rng, 1, keys)]), budget=budget,
                    recent=rng.choice([0, budget // 4]), sinks=rng.choice([0, min(4, budget // 4)]), kv_heads=kv, dim=dim, page=page,
                    cache=cache)
    requests = _between(rng, 1, 24)
    keys = _between(rng, 1, 16384 if cache == "bf16" else 2048)
    chunk = 1 if rng.random() < 0.4 else _between(rng, 1, 1024 if cache == "bf16" else 256)
    while requests * kv * group * chunk * keys > 6 * 10**7 // (1 if cache == "bf16" else 4):
        chunk, keys, requests = (chunk + 1) // 2, max(1, keys - keys // 3), (requests + 1) // 2
    while requests * kv * dim * keys > 6 * 10**8:
        keys -= keys // 3
    return dict(op=op, requests=requests, chunk=min(chunk, keys), keys=keys, q_heads=kv * group, kv_heads=kv, dim=dim, page=page,
                cache=cache, fresh_marks=rng.choice([False, True]))


# ------------------------------------------------------------------ inputs
def _spread(count, most, least=None):
    """`count` lengths from `least` (or about an eighth of `most`) up to `most`, the first of them `most` itself."""
    least = most / 8 if least is None else least
    return [most if i == 0 else max(1, int(least + (most - least) * ((i * 0.6180339887) % 1.0))) for i in range(count)]


def _lengths(case):
    """New tokens and keys of each request (weights), or its keys (evict, trim)."""
    if case["op"] == "weights":
        total = _spread(case["requests"], case["keys"])
        fresh = [min(f, t) for f, t in zip(_spread(case["requests"], case["chunk"]), total)]
        return fresh, total
    return _spread(case["requests"], case["keys"], case.get("least"))


def _kept(case, lengths):
    """Lengths after a step: the last `back` places and fewer are given up, every `every`-th request is done."""
    kept = [max(0, n - i % (case["back"] + 1)) for i, n in enumerate(lengths)]
    return [0 if case["every"] and i % case["every"] == 0 else n for i, n in enumerate(kept)]


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _pages(s, lengths, page, g, spare=8):
    """Block tables of pages in an order of their own; returns the pages' number and ids."""
    wanted = [-(-n // page) for n in lengths]
    pages = sum(wanted) + spare
    ids = torch.randperm(pages, generator=g, device="cuda").int()
    have = _ints(wanted)
    col = torch.arange(max(wanted), device="cuda")
    table = ids[((have.cumsum(0) - have)[:, None] + col).clamp(max=pages - 1)]
    s["table"] = torch.where(col < have[:, None], table, -1).int().contiguous()
    return pages, ids, sum(wanted)


def rates(case):
    """Radians a position of each pair of turned values, and the factor of their cosines and sines."""
    n, base, factor, context = case["turned"], 10000.0, 8.0, 8192
    plain = [base ** (-2.0 * i / n) for i in range(n // 2)]
    if case["scaling"] == "linear":  # positions divided
        return [r / factor for r in plain], 1.0
    if case["scaling"] == "ntk":  # a larger base, which leaves the first pair as it is and divides the last one
        base *= factor ** (n / (n - 2.0))
        return [base ** (-2.0 * i / n) for i in range(n // 2)], 1.0
    if case["scaling"] == "yarn":  # pairs that turn often kept, slow ones divided, a ramp between
        at = lambda turns: n * math.log(context / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        low, high = max(0, math.floor(at(32.0))), min(n - 1, math.ceil(at(1.0)))
        ramp = [min(1.0, max(0.0, (i - low) / max(high - low, 0.001))) for i in range(n // 2)]
        return [r * (1 - w) + r / factor * w for r, w in zip(plain, ramp)], 0.1 * math.log(factor) + 1.0
    if case["scaling"] == "bands":  # by the wavelength against the context
        smooth = [min(1.0, max(0.0, (context * r / (2 * math.pi) - 1.0) / (4.0 - 1.0))) for r in plain]
        return [r * w + r / factor * (1 - w) for r, w in zip(plain, smooth)], 1.0
    return plain, 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return dict(case=case, **_prepare[case["op"]](case, g))


def _prepare_rotary(case, g):
    s = {}
    T, hq, hkv, D, page = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    pages = 2 * -(-T // page)
    s["rows"] = torch.randn(T, (hq + 2 * hkv) * D, generator=g, device="cuda").to(DTYPES[case["rows"]])
    s["K"], s["V"] = (torch.randn(pages, hkv, page, D, generator=g, device="cuda").to(DTYPES[case["cache"]]) for _ in range(2))
    at = torch.randperm(pages, generator=g, device="cuda")[torch.arange(T, device="cuda") // page]
    s["slots"] = at * page + torch.arange(T, device="cuda") % page
    s["positions"] = (case["first"] + torch.arange(T, device="cuda")).int()
    per, s["scale"] = rates(case)
    s["rates"] = torch.tensor(per, dtype=torch.float64, device="cuda")
    # the handle's table: turns a position, in units of 2^-64
    whole = [round(math.ldexp(r / (2 * math.pi), 64)) % 2**64 for r in per]
    s["phases"] = torch.tensor([w - 2**64 if w >= 2**63 else w for w in whole], dtype=torch.int64, device="cuda")
    s["Q"] = torch.empty(T, hq, D, dtype=DTYPES[case["cache"]], device="cuda")
    return s


def _prepare_weights(case, g):
    s = {}
    fresh, total = _lengths(case)
    page, hq, hkv, D, dt = case["page"], case["q_heads"], case["kv_heads"], case["dim"], DTYPES[case["cache"]]
    N = sum(fresh)
    pages, _, _ = _pages(s, total, page, g)
    s["K"] = torch.empty(pages, hkv, page, D, dtype=dt, device="cuda").normal_(generator=g)
    s["q"] = torch.randn(N, hq, D, generator=g, device="cuda").mul_(2.0).to(dt)
    s["q_start"] = _ints([0] + torch.tensor(fresh).cumsum(0).tolist())
    s["kv_len"] = _ints(total)
    s["held"] = None if case["fresh_marks"] else _ints([t - f for f, t in zip(fresh, total)])
    s["offsets"] = torch.randint(0, 1000, (len(total),), generator=g, device="cuda").int()
    s["max_q"], s["max_kv"], s["tokens"], s["keys"] = max(fresh), max(total), N, sum(total)
    s["weight"] = torch.rand(pages, hkv, page, generator=g, device="cuda").mul_(4.0)
    s["place"] = torch.randint(0, 10**6, (pages, hkv, page), generator=g, device="cuda").int()
    # what the attention of this step left: the logarithm of each row's sum, in 64 bits a request at a time
    lse = torch.empty(N, hq, dtype=torch.float64, device="cuda")
    for r, (f, t) in enumerate(zip(fresh, total)):
        a = sum(fresh[:r])
        at = s["table"][r, :-(-t // page)].long()
        place = torch.arange(f, device="cuda") + t - f
        hidden = torch.arange(t, device="cuda") > place[:, None]
        for h in range(hq):
            k = s["K"][at, h // (hq // hkv)].reshape(-1, D)[:t].float()
            x = (s["q"][a:a + f, h].float() @ k.T).double() / math.sqrt(D)
            lse[a:a + f, h] = x.masked_fill_(hidden, -math.inf).logsumexp(1)
    s["lse"] = lse.float()
    s["workspace"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device="cuda")
    return s


def _prepare_evict(case, g):
    s = {}
    lengths = _lengths(case)
    page, hkv, D, dt, R = case["page"], case["kv_heads"], case["dim"], DTYPES[case["cache"]], case["requests"]
    pages, _, _ = _pages(s, lengths, page, g)
    s["K"], s["V"] = (torch.empty(pages, hkv, page, D, dtype=dt, device="cuda").normal_(generator=g) for _ in range(2))
    s["kv_len"], s["max_kv"] = _ints(lengths), max(lengths)
    s["offsets"] = torch.randint(0, 1000, (R,), generator=g, device="cuda").int()
    s["weight0"] = torch.randn(pages, hkv, page, generator=g, device="cuda").mul_(2.0).exp_()
    # a head's keys stand in an order of its own: positions of [0, keys + evicted so far), each at most once
    n = s["kv_len"].long()[:, None, None]
    key = torch.arange(s["max_kv"], device="cuda")
    order = torch.where(key < n, torch.rand(R, hkv, s["max_kv"], generator=g, device="cuda"), 2.0).argsort(-1).argsort(-1)
    place = order * (n + s["offsets"].long()[:, None, None]) // n
    s["place0"] = torch.zeros(pages, hkv, page, dtype=torch.int32, device="cuda")
    req = torch.repeat_interleave(torch.arange(R, device="cuda"), s["kv_len"].long())
    j = torch.cat([torch.arange(m, device="cuda") for m in lengths])
    s["place0"][s["table"].long()[req, j // page], :, j % page] = place[req, :, j].int()
    s["weight"], s["place"] = torch.empty_like(s["weight0"]), torch.empty_like(s["place0"])
    s["kept"], s["offsets_out"] = torch.empty_like(s["kv_len"]), torch.empty_like(s["kv_len"])
    s["workspace"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device="cuda")
    return s


WORKSPACE = 32 << 20  # zeroed once and kept, as a server keeps it


def _prepare_verify(case, g):
    s = {}
    R, V = case["requests"], case["vocab"]
    n = [case["drafts"] if i % 4 == 0 else max(0, case["drafts"] - i % 4) for i in range(R)]
    N = sum(n) + R
    s["q_start"] = _ints([0] + torch.tensor([m + 1 for m in n]).cumsum(0).tolist())
    logits = torch.randn(N, V, generator=g, device="cuda").mul_(2.5)
    s["target"] = torch.softmax(logits, -1).to(DTYPES[case["target"]])
    s["tokens"] = torch.zeros(N, dtype=torch.int32, device="cuda")
    s["draft"] = None
    if case["draft"] == "none":  # drafts looked up in the text, without probabilities: the likeliest token as a rule
        guess = torch.where(torch.rand(N, generator=g, device="cuda") < 0.7, s["target"].float().argmax(-1),
                            torch.randint(0, V, (N,), generator=g, device="cuda"))
    else:
        s["draft"] = torch.softmax(logits + 0.7 * torch.randn(N, V, generator=g, device="cuda"), -1).to(DTYPES[case["draft"]])
        guess = torch.multinomial(s["draft"].float(), 1, generator=g)[:, 0]
    s["tokens"][1:] = guess[:-1].int()  # the token behind a row is drawn from the row's probabilities
    s["uniforms"], s["samples"] = (torch.rand(m, generator=g, device="cuda") for m in (N, R))
    s["kv_len"] = torch.randint(100, 5000, (R,), generator=g, device="cuda").int()
    s["N"], s["drafts"] = N, max(n)
    s["out"] = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    s["accepted"], s["kept"] = torch.empty_like(s["kv_len"]), torch.empty_like(s["kv_len"])
    return s


def _prepare_trim(case, g):
    s = {}
    lengths = _lengths(case)
    pages, ids, used = _pages(s, lengths, case["page"], g, spare=1 + sum(lengths) // (16 * case["page"]))
    s["kv_len"], s["kept"] = _ints(lengths), _ints(_kept(case, lengths))
    s["free"] = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    s["free"][:pages - used] = ids[used:]
    s["n_free"] = _ints([pages - used])
    s["left"], s["status"] = _ints([0]), _ints([0])
    s["freed"] = sum(-(-a // case["page"]) - -(-b // case["page"]) for a, b in zip(lengths, _kept(case, lengths)))
    return s


_prepare = {"rotary": _prepare_rotary, "weights": _prepare_weights, "evict": _prepare_evict, "verify": _prepare_verify,
            "trim": _prepare_trim}


# ------------------------------------------------------------------ one pass
def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_rotary(s):
    import gated_rank_subspace_gb300 as gsi
    c = s["case"]
    turn = gsi.Rotary(c["turned"], s["phases"], c["layout"], s["scale"])
    gsi.rotary_append(gsi.PagedCache(s["K"], s["V"]), s["rows"], s["slots"], s["positions"], c["q_heads"], turn, Q=s["Q"])
    return [s["Q"], s["K"], s["V"]]


def _plain_rotary(s):
    c = s["case"]
    hq, hkv, D, T, n = c["q_heads"], c["kv_heads"], c["dim"], c["tokens"], c["turned"]
    rows = s["rows"].float().view(T, hq + 2 * hkv, D)
    angle = s["positions"].double()[:, None] * s["rates"]
    cos, sin = ((f(angle) * s["scale"]).float()[:, None] for f in (torch.cos, torch.sin))
    x = rows[:, :hq + hkv, :n]
    if c["layout"] == "half":
        a, b = x[..., :n // 2], x[..., n // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0::2], x[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    qk = torch.cat([turned, rows[:, :hq + hkv, n:]], -1).to(s["K"].dtype)
    at, off = s["slots"] // c["page"], s["slots"] % c["page"]
    s["K"][at, :, off] = qk[:, hq:]
    s["V"][at, :, off] = rows[:, hq + hkv:].to(s["K"].dtype)
    return [qk[:, :hq].contiguous(), s["K"], s["V"]]


def _own_weights(s):
    import gated_rank_subspace_gb300 as gsi
    marks = gsi.KeyMarks(s["weight"], s["place"])
    # (the keys alone are read)
    gsi.key_weights(gsi.PagedCache(s["K"], s["K"]), s["q"], s["lse"], s["q_start"], s["kv_len"], s["table"], marks, held=s["held"],
                    offsets=s["offsets"], max_q=s["max_q"], workspace=s["workspace"])
    return [s["weight"], s["place"]]


def _plain_weights(s):
    c, dev = s["case"], s["q"].device
    page, hq, hkv, D, R, M, L = c["page"], c["q_heads"], c["kv_heads"], c["dim"], c["requests"], s["max_q"], s["max_kv"]
    q_len, start = s["q_start"][1:] - s["q_start"][:-1], s["q_start"][:-1].long()
    row, key = torch.arange(M, device=dev), torch.arange(L, device=dev)
    at_row = (start[:, None] + row).clamp(max=s["tokens"] - 1)
    q = s["q"].float()[at_row].view(R, M, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(R, hkv, -1, D)
    lse = s["lse"][at_row].view(R, M, hkv, hq // hkv).permute(0, 2, 3, 1)
    at, off = s["table"].long()[:, key // page].clamp(min=0), (key % page).expand(R, -1)
    k = s["K"][at, :, off].float().transpose(1, 2)
    seen = key < ((s["kv_len"] - q_len)[:, None] + row + 1)[..., None]
    seen = seen & (row < q_len[:, None])[..., None]
    scores = (q @ k.transpose(2, 3)).view(R, hkv, hq // hkv, M, L) / math.sqrt(D)
    p = torch.exp(torch.where(seen[:, None, None], scores, -math.inf) - lse[..., None])
    given = p.sum((2, 3))
    # the keys that there are, one after the other
    lens = s["kv_len"].long()
    req = torch.repeat_interleave(torch.arange(R, device=dev), lens, output_size=s["keys"])
    j = torch.arange(s["keys"], device=dev) - (lens.cumsum(0) - lens)[req]
    pg, slot = s["table"].long()[req, j // page], j % page
    given = given[req, :, j]
    place = (j + s["offsets"].long()[req]).int()[:, None].expand(-1, hkv)
    if s["held"] is not None:
        had = (j < s["held"].long()[req])[:, None]
        given = torch.where(had, s["weight"][pg, :, slot], 0.0) + given
        place = torch.where(had, s["place"][pg, :, slot], place)
    s["weight"][pg, :, slot] = given
    s["place"][pg, :, slot] = place
    return [s["weight"], s["place"]]


def _own_evict(s):
    import gated_rank_subspace_gb300 as gsi
    c = s["case"]
    s["weight"].copy_(s["weight0"])  # what the steps before have gathered
    s["place"].copy_(s["place0"])
    gsi.cache_evict(gsi.PagedCache(s["K"], s["V"]), s["kv_len"], s["table"], gsi.KeyMarks(s["weight"], s["place"]), c["budget"],
                    recent=c["recent"], sinks=c["sinks"], offsets=s["offsets"], kept=s["kept"], offsets_out=s["offsets_out"],
                    workspace=s["workspace"])
    return [s["K"], s["V"], s["weight"], s["place"], s["kept"], s["offsets_out"]]


def _plain_evict(s):
    c, dev = s["case"], s["K"].device
    s["weight"].copy_(s["weight0"])  # what the steps before have gathered
    s["place"].copy_(s["place0"])
    page, hkv, R, B, L = c["page"], c["kv_heads"], c["requests"], c["budget"], s["max_kv"]
    n = s["kv_len"].long()
    kept = n.clamp(max=B)
    key = torch.arange(L, device=dev)
    there = (key < n[:, None])[:, None]
    at, off = s["table"].long()[:, key // page].clamp(min=0), (key % page).expand(R, -1)
    w, place = (t[at, :, off].transpose(1, 2) for t in (s["weight"], s["place"]))
    end = (n + s["offsets"].long())[:, None, None]
    w = torch.where(place < c["sinks"], 3e38, w)
    w = torch.where(place >= end - c["recent"], math.inf, w)
    w = torch.where(there, w, -1.0)  # (weights are not negative)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(2, order, key.expand(R, hkv, -1))
    stay = (rank < kept[:, None, None]) & there
    low = key < kept[:, None, None]
    # the i-th gap takes the i-th kept key behind the new length; what has no gap stays where it is
    most = min(B, max(L - B, 1))
    gaps = torch.where(low & ~stay, key, L).sort(-1).values[..., :most]
    movers = torch.where(~low & stay, key, L).sort(-1).values[..., :most]
    last = (n - 1)[:, None, None]
    dst, src = torch.where(gaps < L, gaps, last), torch.where(movers < L, movers, last)
    req, head = torch.arange(R, device=dev)[:, None, None], torch.arange(hkv, device=dev)[:, None]
    table = s["table"].long()
    to, frm = (table[req, dst // page], head, dst % page), (table[req, src // page], head, src % page)
    for t in (s["K"], s["V"], s["weight"], s["place"]):
        t[to] = t[frm]
    return [s["K"], s["V"], s["weight"], s["place"], kept.int(), (s["offsets"] + (n - kept)).int()]


def _own_verify(s):
    import gated_rank_subspace_gb300 as gsi
    gsi.verify_drafts(s["target"], s["draft"], s["tokens"], s["uniforms"], s["samples"], s["q_start"], kv_len=s["kv_len"],
                      out=s["out"], accepted=s["accepted"], kept=s["kept"])
    return [s["out"], s["accepted"], s["kept"]]


def _plain_verify(s):
    dev, M = s["tokens"].device, s["drafts"]
    start = s["q_start"][:-1].long()
    n = (s["q_start"][1:] - s["q_start"][:-1]).long() - 1
    i = torch.arange(M + 1, device=dev)
    at = (start[:, None] + i).clamp(max=s["N"] - 1)
    row, token = at[:, :M], s["tokens"].long()[at[:, 1:]]
    p = s["target"][row, token].double()
    q = s["draft"][row, token].double() if s["draft"] is not None else torch.ones_like(p)
    passed = (s["uniforms"][row].double() * q < p) & (i[:M] < n[:, None])
    accepted = passed.long().cumprod(1).sum(1)
    here = start + accepted
    rejected = accepted < n
    p = s["target"][here].double()
    if s["draft"] is not None:
        q = s["draft"][here].double()
    else:
        q = torch.zeros_like(p).scatter_(1, s["tokens"].long()[(here + 1).clamp(max=s["N"] - 1)][:, None], 1.0)
    left = torch.where(rejected[:, None], (p - q).clamp(min=0.0), p).cumsum(1)
    sampled = torch.searchsorted(left, left[:, -1:] * s["samples"].double()[:, None], right=True)
    token = torch.cat([token, sampled], 1)
    out = torch.where(i < accepted[:, None], token, torch.where(i == accepted[:, None], sampled, -1))
    req = torch.repeat_interleave(torch.arange(n.numel(), device=dev), n + 1, output_size=s["N"])
    s["out"].copy_(out[req, torch.arange(s["N"], device=dev) - start[req]])
    return [s["out"], accepted.int(), (s["kv_len"] - (n - accepted)).int()]


def _own_trim(s):
    import gated_rank_subspace_gb300 as gsi
    gsi.paged_trim(s["kv_len"], s["kept"], s["table"], s["free"], s["n_free"], s["case"]["page"], n_free_out=s["left"],
                   status=s["status"])
    return [s["free"], s["left"], s["status"]]


def _plain_trim(s):
    page, dev = s["case"]["page"], s["table"].device
    new, old = ((t.long() + page - 1) // page for t in (s["kept"], s["kv_len"]))
    back = old - new
    nth = torch.arange(s["freed"], device=dev)
    req = torch.repeat_interleave(torch.arange(back.numel(), device=dev), back, output_size=s["freed"])
    page_no = new[req] + nth - (back.cumsum(0) - back)[req]
    s["free"][s["n_free"].long() + back.sum() - 1 - nth] = s["table"][req, page_no]
    left = (s["n_free"] + back.sum()).int()
    return [s["free"], left, torch.zeros(1, dtype=torch.int32, device=dev)]


_own = {"rotary": _own_rotary, "weights": _own_weights, "evict": _own_evict, "verify": _own_verify, "trim": _own_trim}
_plain = {"rotary": _plain_rotary, "weights": _plain_weights, "evict": _plain_evict, "verify": _plain_verify, "trim": _plain_trim}


# ------------------------------------------------------------------ what a pass has to do
def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "rotary":
        T, heads = case["tokens"], case["q_heads"] + 2 * case["kv_heads"]
        values = T * heads * case["dim"]
        turned = T * (case["q_heads"] + case["kv_heads"]) * case["turned"]
        return {"bytes": values * (size[case["rows"]] + size[case["cache"]]) + 12 * T + 4 * case["turned"], "flops": 3 * turned}
    if case["op"] == "weights":
        fresh, total = _lengths(case)
        hq, hkv, D, es = case["q_heads"], case["kv_heads"], case["dim"], size[case["cache"]]
        pairs = sum(f * (t - f) + f * (f + 1) // 2 for f, t in zip(fresh, total))
        held = 0 if case["fresh_marks"] else sum(t - f for f, t in zip(fresh, total))
        new, keys, R = sum(total) - held, sum(total), case["requests"]
        marks = hkv * (8 * held + 8 * new)  # weights read and written; of new keys weight and place written
        pages = sum(-(-t // case["page"]) for t in total)
        return {"bytes": es * D * (hkv * keys + hq * sum(fresh)) + 4 * hq * sum(fresh) + marks + 4 * (pages + 4 * R + 1),
                "flops": 2 * D * hq * pairs}
    if case["op"] == "evict":
        lengths, B, hkv = _lengths(case), case["budget"], case["kv_heads"]
        moved = 0.0  # a kept key stands behind the new length as often as any: for weights in no order
        for n in lengths:
            moved += B * (n - B) / n if n > B else 0
        keys = sum(n for n in lengths if n > B)
        pages = sum(-(-n // case["page"]) for n in lengths if n > B)
        row = 2 * 2 * case["dim"] * size[case["cache"]] + 8  # K and V read and written, weight and place written
        return {"bytes": int(hkv * (8 * keys + moved * row)) + 4 * (pages + 4 * case["requests"]), "flops": 0}
    if case["op"] == "verify":
        # one row of either, where a draft is rejected or all are taken
        R, V = case["requests"], case["vocab"]
        return {"bytes": R * V * (size[case["target"]] + size.get(case["draft"], 0)) + 24 * R * (case["drafts"] + 1), "flops": 3 * R * V}
    lengths = _lengths(case)
    back = sum(-(-a // case["page"]) - -(-b // case["page"]) for a, b in zip(lengths, _kept(case, lengths)))
    return {"bytes": 8 * case["requests"] + 8 * back + 12, "flops": 0}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    return {"rotary": _exact_rotary, "weights": _exact_weights, "evict": _exact_evict, "verify": _exact_verify,
            "trim": _exact_trim}[case["op"]](prepare(case, seed))


def _exact_rotary(s):
    c = s["case"]
    hq, hkv, D, n = c["q_heads"], c["kv_heads"], c["dim"], c["turned"]
    Q, K, V = (torch.zeros(c["tokens"], hq, D, dtype=torch.float64, device="cuda"), s["K"].double(), s["V"].double())
    pair = torch.arange(n // 2, device="cuda")
    first, second = (pair, pair + n // 2) if c["layout"] == "half" else (2 * pair, 2 * pair + 1)
    page, off = s["slots"].div(c["page"], rounding_mode="floor"), s["slots"] % c["page"]
    for h in range(hq + 2 * hkv):
        x = s["rows"][:, h * D:(h + 1) * D].double()
        if h < hq + hkv:  # the pair as a complex number, times e^(i angle)
            z = torch.complex(x[:, first], x[:, second]) * torch.polar(torch.full_like(s["rates"], s["scale"])[None],
                                                                        s["positions"].double().outer(s["rates"]))
            x = x.index_copy(1, first, z.real).index_copy(1, second, z.imag)
        if h < hq:
            Q[:, h] = x
        elif h < hq + hkv:
            K[page, h - hq, off] = x
        else:
            V[page, h - hq - hkv, off] = x
    return [Q, K, V]


def _exact_weights(s):
    c = s["case"]
    page, D, group = c["page"], c["dim"], c["q_heads"] // c["kv_heads"]
    weight, places = s["weight"].double(), s["place"].clone()
    starts, lens, table, moved = s["q_start"].tolist(), s["kv_len"].tolist(), s["table"].tolist(), s["offsets"].tolist()
    held = [0] * len(lens) if s["held"] is None else s["held"].tolist()
    for r, n in enumerate(lens):
        pages = torch.tensor(table[r][:-(-n // page)], device="cuda")
        lo, hi = starts[r], starts[r + 1]
        j = torch.arange(n, device="cuda")
        for head in range(c["kv_heads"]):
            k = s["K"][pages, head].reshape(-1, D)[:n].double()
            got = torch.where(j < held[r], weight[pages, head].flatten()[:n], 0.0)
            for h in range(head * group, (head + 1) * group):
                x = k @ s["q"][lo:hi, h].double().T / D**0.5 - s["lse"][lo:hi, h].double()
                later = j[:, None] > torch.arange(lo, hi, device="cuda") - hi + n  # token t stands at place n - (hi - t)
                got = got + x.exp().masked_fill(later, 0.0).sum(1)
            all_w, all_p = weight[pages, head].flatten(), places[pages, head].flatten()
            all_w[:n] = got
            all_p[held[r]:n] = j[held[r]:].int() + moved[r]
            weight[pages, head], places[pages, head] = all_w.view(-1, page), all_p.view(-1, page)
    return [weight, places]


def _exact_evict(s):
    import numpy as np
    c = s["case"]
    page, B = c["page"], c["budget"]
    K, V = s["K"].double(), s["V"].double()
    weight, places = s["weight0"].cpu().numpy().astype(np.float64), s["place0"].cpu().numpy()
    lens, table, gone = s["kv_len"].tolist(), s["table"].cpu().numpy().astype(np.int64), s["offsets"].tolist()
    for r, n in enumerate(lens):
        if n <= B:
            continue
        j = np.arange(n)
        pg, off = table[r, j // page], j % page
        for h in range(c["kv_heads"]):
            w, at = weight[pg, h, off], places[pg, h, off]
            recent, sink = at >= n + gone[r] - c["recent"], at < c["sinks"]
            by = np.lexsort((j, -w, ~sink | recent, ~recent))  # recent ones, then the first ones, then by weight
            stay = np.zeros(n, bool)
            stay[by[:B]] = True
            dst, src = np.flatnonzero(~stay[:B]), B + np.flatnonzero(stay[B:])
            weight[pg[dst], h, off[dst]], places[pg[dst], h, off[dst]] = w[src], at[src]
            a, b, e, f = (torch.from_numpy(x).to(K.device) for x in (pg[dst], off[dst], pg[src], off[src]))
            K[a, h, b], V[a, h, b] = K[e, h, f], V[e, h, f]
    return [K, V, torch.from_numpy(weight).cuda(), torch.from_numpy(places).cuda(), _ints([min(n, B) for n in lens]),
            _ints([o + max(0, n - B) for n, o in zip(lens, gone)])]


def _exact_verify(s):
    import numpy as np
    starts, tokens, u, v = (s[k].cpu().numpy() for k in ("q_start", "tokens", "uniforms", "samples"))
    out, taken, kept = [], [], []
    for r in range(len(starts) - 1):
        a, b = int(starts[r]), int(starts[r + 1])
        t = a
        while t < b - 1:
            d = int(tokens[t + 1])
            q = 1.0 if s["draft"] is None else s["draft"][t, d].double().item()
            if not float(u[t]) * q < s["target"][t, d].double().item():
                break
            out.append(d)
            t += 1
        p = s["target"][t].double().cpu().numpy()
        if t < b - 1:
            if s["draft"] is None:
                p[int(tokens[t + 1])] = 0.0
            else:
                p = np.maximum(p - s["draft"][t].double().cpu().numpy(), 0.0)
        run = np.cumsum(p)
        out += [int(np.count_nonzero(run <= float(v[r]) * run[-1]))] + [-1] * (b - 1 - t)
        taken.append(t - a)
        kept.append(int(s["kv_len"][r]) - (b - 1 - t))
    return [_ints(out), _ints(taken), _ints(kept)]


def _exact_trim(s):
    page, free, left, table = s["case"]["page"], s["free"].tolist(), s["n_free"].item(), s["table"].tolist()
    back = [p for row, n, m in zip(table, s["kv_len"].tolist(), s["kept"].tolist()) for p in row[-(-m // page):-(-n // page)]]
    free[left:left + len(back)] = back[::-1]
    return [_ints(free), _ints([left + len(back)]), _ints([0])]
