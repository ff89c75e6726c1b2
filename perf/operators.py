"""The paged-cache operators as a program that serves requests calls them.

Four operators: the page plan of a step (block tables and slot maps from request lengths), rows written into pages,
rows read back from pages, and attention of new tokens over the pages.  Request lengths are spread evenly over their
logarithm between two ends, so what a pass has to move follows from the case alone; a seed decides their order, the
pages that hold them and every value.
"""
import math

import torch

own = False

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
TYPES = {"bf16": BF16, "e4m3": E4M3}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decoding step of a small server: what counts is how soon the plan is there
        dict(name="plan step of 16", op="plan", requests=16, page=16, shortest=1, longest=4000, new_low=1, new_high=1),
        # a step that mixes prompts, chunks of prompts and single tokens of many requests
        dict(name="plan mixed 1024", op="plan", requests=1024, page=16, shortest=1, longest=8192, new_low=1,
             new_high=2048),
        # the new tokens of 64 requests, one layer, out of a fused q/k/v projection
        dict(name="write step of 64", op="write", tokens=64, layers=1, heads=8, dim=128, page=16, rows="bf16",
             pages="bf16", fused=True),
        # a long prompt's keys and values, one layer, into an 8-bit cache
        dict(name="write prompt e4m3", op="write", tokens=32768, layers=1, heads=8, dim=128, page=128, rows="bf16",
             pages="e4m3", fused=True),
        # a short prefix of one layer taken out of its pages
        dict(name="read prefix 500", op="read", tokens=500, layers=1, heads=8, dim=128, page=16, rows="bf16",
             pages="bf16"),
        # a finished request's 36 layers gathered for the encoder
        dict(name="read 36 layers e4m3", op="read", tokens=8192, layers=36, heads=8, dim=128, page=128, rows="e4m3",
             pages="e4m3"),
        # one request decodes: the smallest attention, latency alone
        dict(name="decode one", op="attention", requests=1, shortest=1000, longest=1000, new_low=1, new_high=1,
             heads=8, group=4, dim=128, page=16, pages="bf16", lse=False, whole=False),
        # a busy decoding batch of very different lengths over an 8-bit cache
        dict(name="decode ragged 64 e4m3", op="attention", requests=64, shortest=100, longest=32768, new_low=1,
             new_high=1, heads=8, group=4, dim=128, page=16, pages="e4m3", lse=False, whole=False),
        # few requests with very long contexts: the work is split along the keys
        dict(name="decode long", op="attention", requests=4, shortest=100000, longest=131072, new_low=1, new_high=1,
             heads=8, group=8, dim=128, page=128, pages="bf16", lse=True, whole=False),
        # drafted tokens verified in one pass, wide heads, odd lengths
        dict(name="verify 5 of 32", op="attention", requests=32, shortest=99, longest=8191, new_low=5, new_high=5,
             heads=2, group=8, dim=256, page=32, pages="bf16", lse=False, whole=False),
        # whole prompts of different lengths packed one after another
        dict(name="prompts packed", op="attention", requests=6, shortest=33, longest=4096, new_low=33, new_high=4096,
             heads=8, group=4, dim=128, page=64, pages="bf16", lse=False, whole=True),
        # a chunk of a long prompt over what is cached of it
        dict(name="chunk 2048 at 32768", op="attention", requests=1, shortest=32768, longest=32768, new_low=2048,
             new_high=2048, heads=8, group=4, dim=128, page=16, pages="bf16", lse=True, whole=False),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("plan", "write", "read", "attention", "attention", "attention"))
    page = rng.choice((8, 16, 32, 64, 128, 256))
    if op == "plan":
        longest = _log(rng, 16, 8192)
        high = rng.choice((1, min(longest, _log(rng, 1, 2048))))
        return dict(op=op, requests=_log(rng, 1, 1024), page=page, shortest=_log(rng, 1, longest), longest=longest,
                    new_low=1, new_high=high)
    heads, dim = rng.choice((1, 2, 4, 8, 16)), rng.choice((64, 128, 256))
    if op != "attention":
        rows, pages = rng.choice((("bf16", "bf16"), ("e4m3", "e4m3"), ("bf16", "e4m3")))
        layers = rng.choice((1, 1, _log(rng, 2, 36)))
        tokens = _log(rng, 1, 32768)
        while layers * tokens * heads * dim > 36 * 8192 * 1024:
            tokens = tokens * 2 // 3
        case = dict(op=op, tokens=tokens, layers=layers, heads=heads, dim=dim, page=page, rows=rows, pages=pages)
        if op == "write":
            case["fused"] = rows == "bf16" and layers == 1
        return case
    group = rng.choice((1, 2, 4, 5, 7, 8, 16))
    while heads * group > 64:
        heads //= 2
    kind = rng.choice(("decode", "verify", "chunk", "prompts"))
    requests = _log(rng, 1, 128 if kind in ("decode", "verify") else 8)
    longest = _log(rng, 16, 65536 if kind == "decode" else 32768 if kind != "prompts" else 4096)
    low, high = 1, 1
    if kind == "verify":
        low, high = min(2, longest), min(longest, rng.randint(2, 9))
    elif kind == "chunk":
        high = min(longest, _log(rng, 16, 2048))
        low = _log(rng, 1, high)
    elif kind == "prompts":
        high = longest
    shortest = _log(rng, high if kind != "prompts" else 1, longest)
    if kind == "prompts":
        low = shortest
    # no dearer than the largest listed ones, and room for the padded scores of the plain form
    while (requests * longest * heads * dim > 4 * 131072 * 1024 or
           requests * high * longest * heads * group > 6 * 4096 * 4096 * 32 or
           requests * high * longest * heads * group * dim > 2048 * 32768 * 32 * 128):
        if requests > 1:
            requests = (requests + 1) // 2
        else:
            longest = max(high, longest * 2 // 3)
            shortest = min(shortest, longest)
            if longest == high:
                longest = high = max(1, high * 2 // 3)
                shortest = longest
            low = min(low, high) if kind != "prompts" else shortest
    return dict(op=op, requests=requests, shortest=shortest, longest=longest, new_low=low, new_high=high, heads=heads,
                group=group, dim=dim, page=page, pages=rng.choice(("bf16", "e4m3")), lse=rng.random() < 0.5,
                whole=kind == "prompts")


# ------------------------------------------------------------------ lengths, the same for every seed but for their order
def _spread(low, high, n):
    return [int(round(low * (high / low) ** ((i + 0.5) / n if n > 1 else 1.0))) for i in range(n)]


def _lengths(case):
    """(length, new tokens) of each request: both spread over their ranges, and paired so that neither follows the other."""
    n = case["requests"]
    lens = _spread(case["shortest"], case["longest"], n)
    if case.get("whole"):
        return [(v, v) for v in lens]
    new = _spread(case["new_low"], case["new_high"], n)
    step = next(s for s in range(max(1, int(n * 0.38)), n + 2) if math.gcd(s, n) == 1)
    return [(v, min(v, new[i * step % n])) for i, v in enumerate(lens)]


def _blocks(tokens, page):
    return -(-tokens // page)


def work(case):
    page = case["page"]
    if case["op"] == "plan":
        pairs = _lengths(case)
        tokens = sum(n for _, n in pairs)
        need = sum(_blocks(v, page) - _blocks(v - n, page) for v, n in pairs)
        touched = sum(_blocks(v, page) - (v - n) // page for v, n in pairs)
        return {"bytes": 8 * len(pairs) + 8 * need + 4 * (touched - need) + 8 * tokens + 8 * (len(pairs) + 1),
                "flops": 0}
    size = {"bf16": 2, "e4m3": 1}
    if case["op"] in ("write", "read"):
        values = 2 * case["layers"] * case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": values * (size[case["rows"]] + size[case["pages"]]) + 4 * case["tokens"], "flops": 0}
    pairs = _lengths(case)
    heads, q_heads, dim = case["heads"], case["heads"] * case["group"], case["dim"]
    tokens, cached = sum(n for _, n in pairs), sum(v for v, _ in pairs)
    keys = sum(n * (v - n) + n * (n + 1) // 2 for v, n in pairs)
    return {"bytes": 2 * cached * heads * dim * size[case["pages"]] + 4 * tokens * q_heads * dim
            + 4 * sum(_blocks(v, page) for v, _ in pairs) + (4 * tokens * q_heads if case["lse"] else 0),
            "flops": 4 * keys * q_heads * dim}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ordered(case, g):
    pairs = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    pairs = pairs[torch.randperm(len(pairs), generator=g, device="cuda")]
    return pairs[:, 0].contiguous(), pairs[:, 1].contiguous()


def _table(lens, page, ids, width):
    """Block table of these lengths over the page ids, -1 behind a request's last block."""
    need = (lens.long() + page - 1) // page
    first = need.cumsum(0) - need
    col = torch.arange(width, device="cuda")
    at = (first[:, None] + col).clamp(max=len(ids) - 1)
    return torch.where(col < need[:, None], ids[at], -1).to(torch.int32)


def _values(shape, dtype, g, sigma=None):
    """Values with a scale of their own in each channel, as keys and values have."""
    if sigma is None:
        sigma = torch.exp(0.5 * torch.randn(shape[-2:], generator=g, device="cuda"))
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1, *shape[-2:])
    step = max(1, (1 << 26) // (shape[-1] * shape[-2]))
    for i in range(0, flat.shape[0], step):
        part = flat[i:i + step]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * sigma)
    return out


def _scales(heads, g):
    return (0.5 + torch.rand(heads, generator=g, device="cuda")).contiguous()


def prepare(case, seed):
    g, page = _gen(seed), case["page"]
    s = {"case": case}
    if case["op"] == "plan":
        lens, new = _ordered(case, g)
        pairs = _lengths(case)
        held = sum(_blocks(v - n, page) for v, n in pairs)
        need = sum(_blocks(v, page) for v, _ in pairs) - held
        ids = torch.randperm(held + need + 64, generator=g, device="cuda").to(torch.int32)
        width = _blocks(case["longest"], page) + 1
        s.update(lens=lens, new=new, table=_table(lens - new, page, ids[:held], width), free=ids[held:].contiguous(),
                 tokens=sum(n for _, n in pairs))
        return s
    heads, dim, dtype = case["heads"], case["dim"], TYPES[case["pages"]]
    if case["op"] in ("write", "read"):
        tokens, layers = case["tokens"], case["layers"]
        n_pages = _blocks(tokens, page) + 32
        # the tokens of one request in order, in pages from anywhere
        ids = torch.randperm(n_pages, generator=g, device="cuda")[:_blocks(tokens, page)]
        slots = (ids[:, None] * page + torch.arange(page, device="cuda")).view(-1)[:tokens]
        s["slots"] = slots.to(torch.int32).contiguous()
        cache = _values((layers, 2, n_pages, page, heads, dim), dtype, g)
        s["k_pages"], s["v_pages"] = cache[:, 0], cache[:, 1]
        if case["rows"] != case["pages"]:
            s["k_scale"], s["v_scale"] = _scales(heads, g), _scales(heads, g)
        if case["op"] == "write":
            if case["fused"]:
                qkv = _values((layers, tokens, 6 * heads, dim), TYPES[case["rows"]], g)
                s["k"], s["v"] = qkv[:, :, 4 * heads:5 * heads], qkv[:, :, 5 * heads:]
            else:
                rows = _values((layers, 2, tokens, heads, dim), TYPES[case["rows"]], g)
                s["k"], s["v"] = rows[:, 0], rows[:, 1]
        return s
    lens, new = _ordered(case, g)
    pairs = _lengths(case)
    width = _blocks(case["longest"], page)
    used = sum(_blocks(v, page) for v, _ in pairs)
    ids = torch.randperm(used + 16, generator=g, device="cuda").to(torch.int32)
    cache = _values((2, used + 16, page, heads, dim), dtype, g)
    tokens, q_heads = sum(n for _, n in pairs), heads * case["group"]
    qkv = _values((tokens, q_heads + 2 * heads, dim), BF16, g,
                  torch.full((q_heads + 2 * heads, dim), 2.0, device="cuda"))
    starts = torch.zeros(len(pairs) + 1, dtype=torch.int32, device="cuda")
    starts[1:] = new.cumsum(0)
    s.update(lens=lens, new=new, starts=starts, table=_table(lens, page, ids, width), k_pages=cache[0],
             v_pages=cache[1], q=qkv[:, :q_heads], most=max(n for _, n in pairs), scale=dim ** -0.5)
    if case["pages"] == "e4m3":
        s["k_scale"], s["v_scale"] = _scales(heads, g), _scales(heads, g)
    return s


# ------------------------------------------------------------------ the plain forms
def _plan(s):
    page, lens, new = s["case"]["page"], s["lens"].long(), s["new"].long()
    have, want = (lens - new + page - 1) // page, (lens + page - 1) // page
    zero = torch.zeros(1, dtype=torch.long, device="cuda")
    starts = torch.cat([zero, new.cumsum(0)])
    taken = torch.cat([zero, (want - have).cumsum(0)])
    col = torch.arange(s["table"].shape[1], device="cuda")
    fresh = (col >= have[:, None]) & (col < want[:, None])
    at = (taken[:-1, None] + col - have[:, None]).clamp(0, len(s["free"]) - 1)
    table = torch.where(fresh, s["free"][at], s["table"])
    row = torch.arange(s["tokens"], device="cuda")
    of = torch.searchsorted(starts[1:], row, right=True)
    position = (lens - new)[of] + row - starts[of]
    slots = table[of, position // page] * page + position % page
    return table, slots.int(), position.int(), starts.int(), taken.int()


def _cast(x, to, scale, back):
    if x.dtype == to:
        return x
    wide = x.float()
    scale = scale[:, None]
    return (wide * scale).to(to) if back else (wide / scale).clamp(-448.0, 448.0).to(to)


def _bits(x):
    """The same bytes as integers: indexing an 8-bit float type needs them."""
    return x.view(torch.uint8) if x.dtype == E4M3 else x


def _write(s):
    at = s["slots"].long()
    for name in ("k", "v"):
        pages = s[name + "_pages"]
        rows = _cast(s[name], pages.dtype, s.get(name + "_scale"), False)
        page = pages.shape[2]
        _bits(pages)[:, at // page, at % page] = _bits(rows)
    return s["k_pages"], s["v_pages"]


def _read(s):
    at, out = s["slots"].long(), []
    for name in ("k", "v"):
        pages = s[name + "_pages"]
        page = pages.shape[2]
        rows = _bits(pages)[:, at // page, at % page].view(pages.dtype)
        out.append(_cast(rows, TYPES[s["case"]["rows"]], s.get(name + "_scale"), True))
    return tuple(out)


def _gathered(s, name):
    """[request][head][position][dim] in 32 bits."""
    pages = s[name + "_pages"]
    x = _bits(pages)[s["table"].clamp(min=0).long()].view(pages.dtype).float()
    x = x.flatten(1, 2).transpose(1, 2)
    return x * s[name + "_scale"][:, None, None] if name + "_scale" in s else x


def _attention(s):
    case = s["case"]
    group, heads = case["group"], case["heads"]
    lens, new, starts, q = s["lens"].long(), s["new"].long(), s["starts"].long(), s["q"]
    tokens, q_heads, dim = q.shape
    step = torch.arange(s["most"], device="cuda")
    rows = (starts[:-1, None] + step).clamp(max=tokens - 1)
    padded = q[rows].float().unflatten(2, (heads, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = torch.matmul(padded, _gathered(s, "k").transpose(2, 3).contiguous()) * s["scale"]
    last = (lens - new)[:, None] + step
    key = torch.arange(score.shape[3], device="cuda")
    hidden = (key > last[:, :, None]) | (key >= lens[:, None, None])
    hidden = hidden[:, None, :, None].expand(-1, 1, -1, group, -1).flatten(2, 3)
    score = score.masked_fill_(hidden, -math.inf)
    top = score.amax(3, keepdim=True)
    part = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = part.sum(3, keepdim=True)
    out = torch.matmul(part, _gathered(s, "v").contiguous()) / total.clamp(min=1e-30)
    row = torch.arange(tokens, device="cuda")
    of = torch.searchsorted(starts[1:], row, right=True)
    at = row - starts[of]
    out = out.unflatten(2, (s["most"], group))[of, :, at].reshape(tokens, q_heads, dim).to(BF16)
    if not case["lse"]:
        return out
    lse = (top + total.log()).squeeze(3).unflatten(2, (s["most"], group))[of, :, at].reshape(tokens, q_heads)
    return out, lse


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"plan": _plan, "write": _write, "read": _read, "attention": _attention}[op](s)
    from lossless_kv_cache_amd import skv
    if op == "plan":
        plan = skv.page_plan(s["lens"], s["new"], s["table"], s["free"], s["case"]["page"], s["tokens"])
        return s["table"], plan.slots, plan.positions, plan.starts, plan.taken
    if op == "write":
        skv.page_write(s["k"], s["v"], s["k_pages"], s["v_pages"], s["slots"], s.get("k_scale"), s.get("v_scale"))
        return s["k_pages"], s["v_pages"]
    if op == "read":
        return skv.page_read(s["k_pages"], s["v_pages"], s["slots"], TYPES[s["case"]["rows"]], s.get("k_scale"),
                             s.get("v_scale"))
    return skv.page_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["starts"], s["most"],
                              scale=s["scale"], k_scale=s.get("k_scale"), v_scale=s.get("v_scale"),
                              lse=s["case"]["lse"])


# ------------------------------------------------------------------ the definitions, request by request, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(s, case["page"])
    if case["op"] == "attention":
        return _exact_attention(s, case)
    out = []
    for name in ("k", "v"):
        pages, scale = s[name + "_pages"], s.get(name + "_scale")
        layers, n_pages, page, heads, dim = pages.shape
        flat = pages.reshape(layers, n_pages * page, heads, dim)
        wide = flat.double()
        for layer in range(layers):
            at = s["slots"].long()
            if case["op"] == "write":
                rows = s[name][layer].double()
                if scale is not None:
                    rows = (rows / scale.double()[None, :, None]).clamp(-448, 448).to(E4M3).double()
                wide[layer].index_copy_(0, at, rows)
        if case["op"] == "read":
            wide = wide.index_select(1, s["slots"].long())
            if scale is not None:
                wide = wide * scale.double()[None, None, :, None]
        else:
            wide = wide.view(pages.shape)
        out.append(wide)
    return tuple(out)


def _exact_plan(s, page):
    lens, new, free = s["lens"].tolist(), s["new"].tolist(), s["free"].tolist()
    table, slots, positions, starts, taken = s["table"].tolist(), [], [], [0], [0]
    for b, (length, fresh) in enumerate(zip(lens, new)):
        got = 0
        for position in range(length - fresh, length):
            block = position // page
            if position % page == 0:
                table[b][block] = free[taken[-1] + got]
                got += 1
            slots.append(table[b][block] * page + position % page)
            positions.append(position)
        starts.append(starts[-1] + fresh)
        taken.append(taken[-1] + got)
    return tuple(torch.tensor(x, dtype=torch.int32) for x in (table, slots, positions, starts, taken))


def _exact_attention(s, case):
    group, page, dim = case["group"], case["page"], case["dim"]
    lens, starts = s["lens"].tolist(), s["starts"].tolist()
    out, lse = [], []
    for b, length in enumerate(lens):
        ids = s["table"][b, :_blocks(length, page)].long()
        q = s["q"][starts[b]:starts[b + 1]].double()
        first = length - q.shape[0]
        allowed = torch.arange(length, device="cuda")[None] <= first + torch.arange(q.shape[0], device="cuda")[:, None]
        of_out, of_lse = [], []
        for h in range(case["heads"]):
            k = _bits(s["k_pages"])[ids, :, h].view(s["k_pages"].dtype).double().reshape(-1, dim)[:length]
            v = _bits(s["v_pages"])[ids, :, h].view(s["v_pages"].dtype).double().reshape(-1, dim)[:length]
            if "k_scale" in s:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for j in range(h * group, h * group + group):
                z = (q[:, j] * s["scale"]) @ k.t().contiguous()
                z = torch.where(allowed, z, -math.inf)
                of_lse.append(torch.logsumexp(z, 1))
                of_out.append(torch.exp(z - of_lse[-1][:, None]) @ v)
        out.append(torch.stack(of_out, 1))
        lse.append(torch.stack(of_lse, 1))
    out = torch.cat(out)
    return (out, torch.cat(lse)) if case["lse"] else out
