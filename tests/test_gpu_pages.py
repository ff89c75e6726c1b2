"""The paged-cache operators on the GPU against their definitions in 64 bits
(attention) or on the host (plans, rows), at the lengths, layouts and masks
where they can go wrong, alone and as a request uses them one after another.

Tolerances.  With u = 2^-24 (half a step of fp32) and h = 2^-8 (of bf16), for
a query with n keys of D values:
  a score's error is at most e_s = u (D + 16) scale sum|q||k| + 4 u |s|
    (D products and sums, the scales, the conversion to base 2), taken at its
    largest key; a probability relative to the largest is off by the factor
    exp(2 e_s) and by 4 u of the exponential itself;
  lse is off by at most e_s + (n + 32) u + 4 u |lse|;
  out rounds each probability to bf16 (h) and the result (h):
    |error| <= (h + 4 e_s + (n + 64) u) A + h |out| (1 + h),  A = sum p |v|.
"""
import math

import pytest
import torch

from workloads import gen

pytestmark = pytest.mark.gpu
U, H = 2.0 ** -24, 2.0 ** -8
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def skv():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from lossless_kv_cache_amd import skv as m
    m.lib()
    return m


def dev(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def rnd(shape, g, dtype=BF16, sigma=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)


def bits(x):
    return x.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()])


def filled(shape, dtype, nan=True):
    """Memory nobody has written: NaN in every element."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    bits(t).fill_({1: 0x7F, 2: 0x7FC1, 4: 0x7FC00001}[t.element_size()] if nan else 0)
    return t


# ------------------------------------------------------------------ plans
def plan_model(lens, new, table, free, page, tokens):
    """The plan on the host, request by request; also the flags."""
    width, flags = len(table[0]), 0
    table = [list(r) for r in table]
    slots, positions, starts, taken = [], [], [0], [0]
    for b, (n, f) in enumerate(zip(lens, new)):
        if f < 0 or n < f or n > width * page:
            flags |= 1
            n = f = 0
        have = -(-(n - f) // page)
        want = -(-n // page) if free is not None else have
        for j in range(have, want):
            e = taken[-1] + j - have
            table[b][j] = free[e] if e < len(free) else -1
            if e >= len(free):
                flags |= 8
        for pos in range(n - f, n):
            p = table[b][pos // page]
            fresh = free is not None and pos // page >= have
            if p < 0 and not (fresh and taken[-1] + pos // page - have >= len(free)):
                flags |= 2
            slots.append(p * page + pos % page if p >= 0 else -1)
            positions.append(pos)
        starts.append(starts[-1] + f)
        taken.append(taken[-1] + want - have)
    if len(slots) > tokens:
        flags |= 16
    slots = (slots + [-1] * tokens)[:tokens]
    positions = (positions + [-1] * tokens)[:tokens]
    return table, slots, positions, [min(s, tokens) for s in starts], taken, flags


def check_plan(skv, lens, new, table, free, page, tokens):
    status = dev([0])
    t = dev(table)
    p = skv.page_plan(dev(lens), dev(new), t, None if free is None else dev(free), page, tokens, status=status)
    want = plan_model(lens, new, table, free, page, tokens)
    for got, w in zip((t, p.slots, p.positions, p.starts, p.taken), want):
        assert got.tolist() == w
    assert status.item() == want[5]
    return want[5]


@pytest.mark.parametrize("page", [8, 16, 128, 1024])
@pytest.mark.parametrize("requests", [1, 3, 64, 257, 1000])
def test_plan(skv, page, requests):
    r = torch.Generator().manual_seed(page * 1000 + requests)
    longest = 3 * page + 5
    lens = torch.randint(0, longest, (requests,), generator=r).tolist()
    new = [int(torch.randint(0, n + 1, (1,), generator=r)) if b % 3 else min(n, 1) for b, n in enumerate(lens)]
    width = -(-longest // page) + 1
    held = sum(-(-(n - f) // page) for n, f in zip(lens, new))
    need = sum(-(-n // page) for n in lens) - held
    ids = torch.randperm(held + need + 3, generator=r).tolist()
    table, at = [], 0
    for n, f in zip(lens, new):
        have = -(-(n - f) // page)
        table.append(ids[at:at + have] + [-7] * (width - have))
        at += have
    free, tokens = ids[held:], sum(new)
    assert check_plan(skv, lens, new, table, free, page, tokens) == 0
    assert check_plan(skv, lens, new, table, free, page, tokens + 13) == 0          # padded
    # the whole cache of requests that have their pages
    full = plan_model(lens, new, table, free, page, tokens)[0]
    assert check_plan(skv, lens, lens, full, None, page, sum(lens)) == 0
    if need > 2:
        assert check_plan(skv, lens, new, table, free[:need - 2], page, tokens) == 8
    if tokens > 5:
        assert check_plan(skv, lens, new, table, free, page, tokens - 5) == 16


def test_plan_bad_requests(skv):
    table = [[i, i + 10, -1, -1] for i in range(5)]
    assert check_plan(skv, [20, -1, 3, 65, 33], [3, 1, 4, 1, 2], table, [50, 51, 52], 16, 8) == 1
    assert check_plan(skv, [20, 20, 20, 20, 40], [-1, 0, 4, 20, 0], table, [50, 51, 52], 16, 30) == 1
    # a table entry that names nothing, and pages whose slots would pass 2^31 - 1
    # (request 0 grows from 10 to 20 tokens, one page of 16 to two, and the list is empty: 8 as well as 2)
    assert check_plan(skv, [20, 18], [10, 2], [[-5, 3], [4, 6]], [], 16, 12) == 10
    p = skv.page_plan(dev([17]), dev([17]), dev([[0, 0]]), dev([(1 << 27) - 1, 5]), 16, 17, status=(st := dev([0])))
    assert p.slots.tolist() == [-1] * 16 + [80] and st.item() == 2
    with pytest.raises(skv.SkvError) as e:
        skv.page_check(st)
    assert e.value.status == skv.ERR_PAGES and e.value.flags == skv.PAGES_PAGE
    skv.page_check(dev([0]))
    # an empty free list that nobody needs, a request list without rows
    assert check_plan(skv, [20, 5], [0, 0], [[1, 2], [3, 4]], [], 16, 0) == 0


# ------------------------------------------------------------------ rows
def make_pool(layout, layers, pages, page, heads, dim, dtype):
    """(k, v, backing) pools, filled with NaN, in one of the layouts callers have."""
    if layout == "token":
        x = filled((layers, 2, pages, page, heads, dim), dtype)
        return x[:, 0], x[:, 1], x
    if layout == "head":
        x = filled((2, layers, pages, heads, page, dim), dtype)
        return x[0].transpose(2, 3), x[1].transpose(2, 3), x
    x = filled((layers, pages, page, 2, heads, dim + 16), dtype)          # K and V side by side, padded heads
    return x[:, :, :, 0, :, :dim], x[:, :, :, 1, :, :dim], x


@pytest.mark.parametrize("layout", ["token", "head", "pairs"])
@pytest.mark.parametrize("rows,pages", [(BF16, BF16), (E4M3, E4M3), (BF16, E4M3)])
@pytest.mark.parametrize("heads,dim,page,tokens,layers", [(8, 128, 16, 70, 1), (1, 16, 8, 1, 2), (3, 80, 32, 333, 3),
                                                          (16, 256, 64, 65, 1), (64, 1024, 8, 9, 1)])
def test_write_and_read(skv, layout, rows, pages, heads, dim, page, tokens, layers):
    g = torch.Generator(device="cuda").manual_seed(tokens)
    n = -(-tokens // page) + 5
    kp, vp, backing = make_pool(layout, layers, n, page, heads, dim, pages)
    before = backing.clone()
    qkv = rnd((layers, tokens, 2 * heads + 1, dim), g, sigma=100.0 if rows != pages else 1.0).to(rows)
    k, v = qkv[:, :, 1:heads + 1], qkv[:, :, heads + 1:]
    bits(k)[0, 0, 0, :3] = {1: dev([0x7F, 0xFE, 0x80], torch.uint8), 2: dev([0x7FC0, -128, 0x7F80], torch.int16)}[
        k.element_size()]
    slots = torch.randperm(n * page, generator=g, device="cuda")[:tokens].to(torch.int32)
    if tokens > 3:
        slots[tokens // 2] = -1
    scales = (None, None)
    if rows != pages:
        scales = tuple(0.25 + torch.rand(heads, generator=g, device="cuda") for _ in range(2))
    status = dev([0])
    skv.page_write(k, v, kp, vp, slots, *scales, status=status)
    # the same on a copy of the memory, through torch
    want = torch.empty_strided(backing.shape, backing.stride(), dtype=backing.dtype, device="cuda")
    bits(want).copy_(bits(before))
    wk, wv = (torch.as_strided(want, t.shape, t.stride(), t.storage_offset()) for t in (kp, vp))
    kept = (slots >= 0).nonzero()[:, 0]
    at = slots[kept].long()
    for w, x, s in ((wk, k, scales[0]), (wv, v, scales[1])):
        y = x[:, kept]
        if s is not None:
            y = (y.float() / s[:, None]).clamp(-448, 448)          # one correctly rounded division, then one rounding
            y = torch.where(x[:, kept].isnan(), float("nan"), y)
        bits(w)[:, at // page, at % page] = bits(y.to(pages))
    got, ref = bits(backing).clone(), bits(want)
    if rows != pages:          # a NaN's sign is nobody's
        nan = 0x7F
        got, ref = (torch.where((t & 0x7F) == nan, nan, t) for t in (got, ref))
    assert torch.equal(got, ref)
    assert status.item() == 0
    # read back: copies, and codes times scales rounded once
    rk, rv = skv.page_read(kp, vp, slots, status=status)
    assert rk.dtype is pages and rk.shape == k.shape
    for r, p in ((rk, kp), (rv, vp)):
        ref = bits(p)[:, at // page, at % page]
        assert torch.equal(bits(r)[:, kept], ref)
        assert not bits(r)[:, (slots < 0).nonzero()[:, 0]].any()
    if pages is E4M3:
        s2 = tuple(0.25 + torch.rand(heads, generator=g, device="cuda") for _ in range(2))
        out = rnd((layers, tokens, 2, heads, dim), g)
        rk, rv = skv.page_read(kp, vp, slots, BF16, *s2, out=(out[:, :, 0], out[:, :, 1]))
        for r, p, s in ((rk, kp, s2[0]), (rv, vp, s2[1])):
            codes = bits(p)[:, at // page, at % page].view(E4M3)
            ref = (codes.float() * s[:, None]).to(BF16)
            assert torch.equal(r[:, kept].isnan(), ref.isnan())
            assert torch.equal(bits(torch.nan_to_num(r[:, kept], 0.0)), bits(torch.nan_to_num(ref, 0.0)))
    assert status.item() == 0


@pytest.mark.parametrize("scale", [1.0, 0.0, -0.0, 3.0, -0.7, 1e-30, 2.0 ** -70, 2.0 ** 70, 1e38, 1e-44, 1.1754942e-38,
                                   1.9999999, 0.33333334, float("inf"), float("nan")])
def test_every_bf16_divided_by_a_scale(skv, scale):
    """All 65536 bf16 patterns into e4m3 pages: the correctly rounded quotient, rounded once more and saturated."""
    x = torch.arange(-32768, 32768, device="cuda").to(torch.int16).view(BF16).view(4096, 1, 16)
    pool = filled((2, 512, 8, 1, 16), E4M3)
    slots = torch.arange(4096, device="cuda", dtype=torch.int32)
    s = torch.full((1,), scale, device="cuda")
    skv.page_write(x, x, pool[0], pool[1], slots, s, s)
    y = x.double() / s.double()          # rounded to 32 bits below: one rounding of the exact quotient's 53 bits, which
    want = y.float()                     # lie too far from a tie of 24 for 8-bit over 24-bit numbers to be off by it
    want = torch.where(want.isnan(), want, want.clamp(-448, 448)).to(E4M3)
    got, ref = bits(pool[0]).view(-1), bits(want).view(-1)
    nan = (ref & 0x7F) == 0x7F
    assert torch.equal((got & 0x7F) == 0x7F, nan)
    assert torch.equal(got[~nan], ref[~nan]) and torch.equal(got, bits(pool[1]).view(-1))


def test_rows_skip_what_is_no_slot(skv):
    g = torch.Generator(device="cuda").manual_seed(5)
    pool = torch.zeros((2, 6, 16, 2, 64), dtype=BF16, device="cuda")
    k, v = rnd((5, 2, 64), g), rnd((5, 2, 64), g)
    status = dev([0])
    bad = dev([95, 96, -1, (1 << 31) - 1, -(1 << 31)])
    skv.page_write(k, v, pool[0], pool[1], bad, status=status)
    assert status.item() == skv.PAGES_SLOT
    assert torch.equal(pool[0].view(96, 2, 64)[95], k[0]) and torch.equal(pool[1].view(96, 2, 64)[95], v[0])
    assert not pool.view(2, 96, 2, 64)[:, :95].any()
    rk, rv = skv.page_read(pool[0], pool[1], bad, status=(st := dev([0])))
    assert st.item() == skv.PAGES_SLOT and torch.equal(rk[0], k[0]) and not rk[1:].any() and not rv[1:].any()
    # every slot twice: each 16 bytes come from one of the two rows
    two = dev([3, 3])
    skv.page_write(k[:2], v[:2], pool[0], pool[1], two)
    got = pool[0].view(96, 2, 8, 8)[3]
    a, b = k[0].view(2, 8, 8), k[1].view(2, 8, 8)
    assert ((got == a).all(-1) | (got == b).all(-1)).all()


# ------------------------------------------------------------------ attention
def batch(pairs, heads, group, dim, page, pages, g, layout="token", extra_rows=0, sigma=2.0, scales=None):
    """A batch of (len, new) requests over a NaN-filled pool whose owned tokens are random."""
    lens, new = [a for a, _ in pairs], [b for _, b in pairs]
    need = [-(-max(n, 0) // page) for n in lens]
    n_pages = sum(need) + 3
    ids = torch.randperm(n_pages, generator=g, device="cuda").tolist()
    width = max(max(need), 1)
    table, at = [], 0
    for n in need:
        table.append(ids[at:at + n] + [-1] * (width - n))
        at += n
    kp, vp, _ = make_pool(layout, 1, n_pages, page, heads, dim, pages)
    kp, vp = kp[0], vp[0]
    for b, n in enumerate(lens):
        for j in range(need[b]):
            m = min(page, n - j * page)
            for p in (kp, vp):
                bits(p)[table[b][j], :m] = bits(rnd((m, heads, dim), g, pages))
    tokens = sum(new) + extra_rows
    q = rnd((tokens, heads * group + 3, dim), g, sigma=sigma)[:, 1:1 + heads * group]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    ks, vs = scales or (None, None)
    return dict(q=q, k=kp, v=vp, table=dev(table).view(len(pairs), width), lens=dev(lens), starts=dev(starts),
                pairs=pairs, group=group, page=page, ks=ks, vs=vs)


def reference(s, scale, causal):
    """out, lse and their tolerances in 64 bits, by request and head; rows of no request are None."""
    heads, dim = s["k"].shape[2], s["k"].shape[3]
    tokens, q_heads, _ = s["q"].shape
    out = torch.zeros((tokens, q_heads, dim), dtype=torch.float64, device="cuda")
    tol_o, lse = torch.zeros_like(out), torch.full((tokens, q_heads), -math.inf, dtype=torch.float64, device="cuda")
    tol_l = torch.zeros_like(lse)
    starts = s["starts"].tolist()
    for b, (n, new) in enumerate(s["pairs"]):
        if new == 0 or n == 0:
            continue
        ids = s["table"][b, :-(-n // s["page"])].long()
        k = bits(s["k"])[ids].view(s["k"].dtype).double().flatten(0, 1)[:n]
        v = bits(s["v"])[ids].view(s["v"].dtype).double().flatten(0, 1)[:n]
        if s["ks"] is not None:
            k, v = k * s["ks"].double()[:, None], v * s["vs"].double()[:, None]
        last = torch.arange(n - new, n, device="cuda") if causal else torch.full((new,), n - 1, device="cuda")
        seen = torch.arange(n, device="cuda")[None] <= last[:, None]
        r0 = starts[b]
        for h in range(q_heads):
            kh, vh = k[:, h // s["group"]], v[:, h // s["group"]]
            qh = s["q"][r0:r0 + new, h].double()
            x = torch.where(seen, scale * (qh @ kh.t().contiguous()), -math.inf)
            mag = torch.where(seen, abs(scale) * (qh.abs() @ kh.abs().t().contiguous()), 0.0)
            e = U * (dim + 16) * mag.amax(1) + 4 * U * torch.where(seen, x.abs(), 0.0).amax(1)
            l = torch.logsumexp(x, 1)
            p = torch.where(seen, torch.exp(x - l[:, None]), 0.0)
            some = last >= 0
            a = p @ torch.nan_to_num(vh.abs(), 0.0, 0.0, 0.0)
            o = torch.stack([p[i, :m + 1] @ vh[:m + 1] if m >= 0 else torch.zeros(dim, device="cuda").double()
                             for i, m in enumerate(last.tolist())]) if not vh.isfinite().all() else p @ vh
            rows = slice(r0, r0 + new)
            out[rows, h] = torch.where(some[:, None], o, 0.0)
            lse[rows, h] = torch.where(some, l, -math.inf)
            n_u = U * (n + 64)
            tol_o[rows, h] = (H + 4 * e + n_u)[:, None] * a + H * (1 + H) * out[rows, h].abs()
            tol_l[rows, h] = e + n_u + 4 * U * torch.where(some, l.abs(), 0.0)
    return out, tol_o, lse, tol_l


def attend(skv, s, causal=True, scale=None, **kw):
    most = max([n for _, n in s["pairs"]] + [0])
    return skv.page_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["starts"], most, causal=causal,
                              scale=scale, k_scale=s["ks"], v_scale=s["vs"], lse=True, **kw)


def compare(got, want, rows):
    out, lse = (x[:rows].double() for x in got)
    o, to, l, tl = (x[:rows] for x in want)
    assert torch.equal(out.isnan(), o.isnan())
    d = torch.where(o.isnan() | (out == o), 0.0, (out - o).abs())
    ok = bool(((d <= to) | (d == 0)).all())          # (where both are NaN, so is the tolerance)
    assert ok, f"out is {(d / to).max().item():.3g} times its tolerance off"
    d = torch.where(lse == l, 0.0, (lse - l).abs())
    ok = bool((d <= tl).all())
    assert ok, f"lse is {(d / tl).max().item():.3g} times its tolerance off"


LENGTHS = {
    "one": [(1, 1)],
    "decode": [(1, 1), (17, 1), (300, 1), (64, 1), (65, 1), (128, 1), (129, 1), (2, 1)],
    "decode empty": [(0, 1), (33, 1), (0, 1), (40, 0), (0, 0)],
    "long decode": [(5000, 1), (7, 1)],
    "verify": [(200, 5), (5, 5), (67, 2), (3, 5), (1000, 3), (0, 4)],
    "chunks": [(40, 40), (100, 37), (5, 9), (0, 0), (257, 130), (1000, 33), (64, 64)],
    "prompts": [(513, 513), (1, 1), (127, 127), (130, 130)],
    "mixed": [(700, 1), (300, 300), (90, 1), (2000, 150), (31, 8)],
}


@pytest.mark.parametrize("pages", [BF16, E4M3])
@pytest.mark.parametrize("heads,group,dim,page", [(2, 4, 128, 16), (1, 1, 64, 8), (3, 5, 128, 64), (1, 16, 256, 32),
                                                  (2, 7, 64, 256), (1, 33, 128, 16), (1, 64, 64, 128)])
@pytest.mark.parametrize("kind", list(LENGTHS))
def test_attention(skv, kind, heads, group, dim, page, pages):
    g = torch.Generator(device="cuda").manual_seed(len(kind) * 100 + dim + group)
    scales = None
    if pages is E4M3:
        scales = tuple(0.5 + torch.rand(heads, generator=g, device="cuda") for _ in range(2))
    s = batch(LENGTHS[kind], heads, group, dim, page, pages, g, layout="token" if dim < 256 else "head",
              extra_rows=3, scales=scales)
    rows = s["starts"][-1].item()
    out, lse = filled(s["q"].shape, BF16), filled(s["q"].shape[:2], torch.float32)
    status = dev([0])
    for causal in (True, False):
        bits(out).fill_(0x1234)
        got = attend(skv, s, causal, out=out, status=status)
        compare(got, reference(s, dim ** -0.5, causal), rows)
        assert (bits(got[0])[rows:] == 0x1234).all(), "rows behind the last request"
    # the same call again: the same bits; without lse and with a workspace of the caller's as well
    again = attend(skv, s, False)
    assert torch.equal(bits(again[0])[:rows], bits(out)[:rows]) and torch.equal(again[1][:rows], got[1][:rows])
    assert status.item() == 0


def test_attention_layouts_and_scale(skv):
    g = torch.Generator(device="cuda").manual_seed(3)
    for layout in ("head", "pairs"):
        for pages in (BF16, E4M3):
            s = batch([(130, 70), (65, 1), (300, 2)], 2, 2, 128, 16, pages, g, layout=layout)
            for scale in (0.3, -0.05, 0.0):
                compare(attend(skv, s, scale=scale), reference(s, scale, True), 73)
    # rows with no starts: one per request, and a table with rows apart
    s = batch([(130, 1), (65, 1), (300, 1)], 2, 2, 128, 16, BF16, g)
    wide = torch.full((3, 40), -1, dtype=torch.int32, device="cuda")
    wide[:, :s["table"].shape[1]] = s["table"]
    got = skv.page_attention(s["q"], s["k"], s["v"], wide[:, :s["table"].shape[1] + 2], s["lens"], lse=True)
    compare(got, reference(s, 128 ** -0.5, True), 3)
    # an output with strides of its own
    wide_out = filled((3, 6, 256), BF16)
    got = skv.page_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], lse=True, out=wide_out[:, 1:5, 64:192])
    compare(got, reference(s, 128 ** -0.5, True), 3)
    keep = wide_out.clone()
    keep[:, 1:5, 64:192] = float("nan")
    assert keep.isnan().all()


@pytest.mark.parametrize("pages", [BF16, E4M3])
@pytest.mark.parametrize("pairs", [[(40, 40), (70, 6)], [(200, 3), (50, 2)], [(3000, 200)], [(4000, 4)]])
def test_what_a_query_does_not_see_never_reaches_it(skv, pairs, pages):
    """NaN and infinities in later tokens' keys and values: earlier queries are as if they were not there."""
    g = torch.Generator(device="cuda").manual_seed(8)
    s = batch(pairs, 2, 4, 128, 16, pages, g)
    clean = reference(s, 128 ** -0.5, True)
    rows, starts = s["starts"][-1].item(), s["starts"].tolist()
    poisoned = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for b, (n, new) in enumerate(pairs):
        for j in (n - 1, n - 2):          # the last two tokens
            page, at = s["table"][b, j // 16].item(), j % 16
            bad = [float("nan"), float("inf"), -float("inf")] if pages is BF16 else [float("nan")] * 3
            for i, x in enumerate(bad):
                s["v"][page, at, :, 5 + 40 * i] = torch.tensor(x).to(pages)
            s["k"][page, at, :, 3] = torch.tensor(float("nan")).to(pages)
        poisoned[starts[b] + new - 2:starts[b] + new] = True
    got = attend(skv, s)
    assert got[0][poisoned].isnan().all(2).all()
    for x in got:
        x[poisoned] = 0
    want = [x.clone() for x in clean]
    for x in want:
        x[:rows][poisoned] = 0
    compare(got, want, rows)


def test_values_beyond_range_propagate(skv):
    """Infinite values that a query sees: the formula's infinities and NaN."""
    g = torch.Generator(device="cuda").manual_seed(9)
    s = batch([(100, 20), (50, 1)], 2, 4, 64, 16, BF16, g)
    s["v"][s["table"][0, 0].item(), 3, :, 7] = float("inf")
    s["v"][s["table"][0, 0].item(), 4, :, 9] = float("inf")
    s["v"][s["table"][0, 1].item(), 4, :, 9] = -float("inf")
    want = reference(s, 0.125, True)
    assert want[0][:20, :, 7].isinf().all() and want[0][:20, :, 9].isnan().all()
    compare(attend(skv, s), want, 21)


@pytest.mark.parametrize("pairs", [[(100, 1)] * 4, [(100, 50)] * 4, [(3000, 40)] * 4, [(100, 2)] * 4])
def test_bad_tables_and_lengths(skv, pairs):
    """What the host cannot see is flagged and not followed; the other requests are exact."""
    g = torch.Generator(device="cuda").manual_seed(10)
    s = batch(pairs, 2, 4, 128, 16, BF16, g)
    new = pairs[0][1]
    want = reference(s, 128 ** -0.5, True)

    def go(change, flags, spared):
        t = {k: v.clone() if isinstance(v, torch.Tensor) and k in ("table", "lens", "starts") else v for k, v in s.items()}
        change(t)
        status = dev([0])
        out, lse = filled(s["q"].shape, BF16), filled(s["q"].shape[:2], torch.float32)
        bits(out).fill_(0x1234)
        got = skv.page_attention(t["q"], t["k"], t["v"], t["table"], t["lens"], t["starts"], new, lse=lse, out=out,
                                 status=status)[0]
        assert status.item() == flags
        for b in range(4):
            r = slice(b * new, b * new + new)
            if b in spared:
                assert (bits(got)[r] == 0x1234).all()
            elif b != 1:
                d = (got[r].double() - want[0][r]).abs()
                assert (d <= want[1][r]).all()

    for entry in (-1, s["k"].shape[0], (1 << 31) - 1, -(1 << 31)):
        go(lambda t: t["table"][1, 2:4].fill_(entry), skv.PAGES_PAGE, ())
    go(lambda t: t["lens"][1].fill_(-1), skv.PAGES_LENGTH, (1,))
    go(lambda t: t["lens"][1].fill_((1 << 31) - 1), skv.PAGES_LENGTH, (1,))
    go(lambda t: t["starts"][4].fill_(4 * new + 1), skv.PAGES_LENGTH, (3,))
    go(lambda t: t["starts"][0].fill_(-1), skv.PAGES_LENGTH, (0,))
    go(lambda t: t["starts"][2].fill_(new - 1), skv.PAGES_LENGTH | skv.PAGES_ROWS, (1, 2))


@pytest.mark.parametrize("pages", [BF16, E4M3])
@pytest.mark.parametrize("new", ["few", "many"])
@pytest.mark.parametrize("requests", [64, 65, 200, 257, 700])
def test_many_requests(skv, requests, new, pages):
    """More requests than a workgroup has threads: empty ones, single tokens, some longer, one of them long."""
    g = torch.Generator(device="cuda").manual_seed(21)
    r = torch.Generator().manual_seed(22)
    pairs = []
    for b in range(requests):
        n = int(torch.randint(0, 70, (1,), generator=r))
        pairs.append((n, min(n, b % 4) if new == "few" or b % 50 else n))
    pairs[requests // 2] = (2500, 7 if new == "few" else 170)
    s = batch(pairs, 2, 4, 64, 16, pages, g, extra_rows=5)
    rows, status = s["starts"][-1].item(), dev([0])
    out = filled(s["q"].shape, BF16)
    bits(out).fill_(0x1234)
    got = attend(skv, s, out=out, status=status)
    compare(got, reference(s, 0.125, True), rows)
    assert (bits(out)[rows:] == 0x1234).all() and status.item() == 0


@pytest.mark.parametrize("pages", [BF16, E4M3])
@pytest.mark.parametrize("dim,page", [(64, 8), (128, 8), (256, 8), (64, 64), (128, 32), (256, 128)])
def test_short_and_empty_requests_in_a_row(skv, dim, page, pages):
    """Workgroups that go through several requests each: ends inside a page and a tile, waves without tokens."""
    g = torch.Generator(device="cuda").manual_seed(dim + page)
    r = torch.Generator().manual_seed(dim * page)
    lens = [0, 1, 7, 8, 9, 31, 33, 64, 65, 127, 129, 130, 257, 513]
    pairs = []
    for b in range(100):
        n = lens[int(torch.randint(0, len(lens), (1,), generator=r))]
        pairs.append((n, min(n, 1 + b % 3) if b % 7 else 0))
    pairs[0], pairs[-1] = (513, 2), (1, 1)
    s = batch(pairs, 4, 8, dim, page, pages, g, layout="head" if page == 8 else "token", extra_rows=2)
    rows, status = s["starts"][-1].item(), dev([0])
    out = filled(s["q"].shape, BF16)
    bits(out).fill_(0x1234)
    got = attend(skv, s, out=out, status=status)
    compare(got, reference(s, dim ** -0.5, True), rows)
    assert (bits(out)[rows:] == 0x1234).all() and status.item() == 0


def test_no_new_tokens(skv):
    """A batch none of whose requests has a query, said and unsaid: nothing is written."""
    g = torch.Generator(device="cuda").manual_seed(16)
    s = batch([(40, 0), (0, 0), (300, 0)], 2, 4, 128, 16, BF16, g, extra_rows=70)
    for most in (0, 1, 8, 9, 70, None):
        out, lse, st = filled(s["q"].shape, BF16), filled(s["q"].shape[:2], torch.float32), dev([0])
        bits(out).fill_(0x1234)
        before = lse.clone()
        skv.page_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["starts"], most, out=out, lse=lse, status=st)
        assert (bits(out) == 0x1234).all() and torch.equal(bits(lse), bits(before)) and st.item() == 0
    # tokens of a request past the bound are not computed, and said so
    t = batch([(40, 3), (50, 2)], 2, 4, 128, 16, BF16, g)
    for most, heads in ((2, 4), (0, 4)):
        out, st = filled(t["q"].shape, BF16), dev([0])
        bits(out).fill_(0x1234)
        skv.page_attention(t["q"], t["k"], t["v"], t["table"], t["lens"], t["starts"], most, out=out, status=st)
        assert st.item() == skv.PAGES_ROWS and (bits(out)[:3] == 0x1234).all()
        assert bool((bits(out)[3:] == 0x1234).all()) == (most == 0)


def test_pool_past_four_gigabytes(skv):
    """Pages whose byte offsets pass 2^32 and element offsets 2^31."""
    g = torch.Generator(device="cuda").manual_seed(11)
    pages, page, heads, dim = 36000, 64, 8, 128          # 4.7 GB each
    pool = torch.empty((2, pages, page, heads, dim), dtype=BF16, device="cuda")
    pairs = [(200, 1), (150, 150), (64, 3)]
    ids = [pages - 1, 3, pages - 5, 33000, 32768, 16384, pages - 2, 5]
    table = dev([ids[:4], ids[4:7] + [-1], [ids[7], -1, -1, -1]])
    slots = []
    for b, (n, _) in enumerate(pairs):
        slots += [table[b, j // page].item() * page + j % page for j in range(n)]
    k, v = rnd((414, heads, dim), g), rnd((414, heads, dim), g)
    skv.page_write(k, v, pool[0], pool[1], dev(slots))
    rk, rv = skv.page_read(pool[0], pool[1], dev(slots))
    assert torch.equal(rk, k) and torch.equal(rv, v)
    small = torch.zeros((2, 8, page, heads, dim), dtype=BF16, device="cuda")
    near = dev([[0, 1, 2, 3], [4, 5, 6, -1], [7, -1, -1, -1]])
    for b in range(3):
        for j in range(4):
            if table[b, j] >= 0:
                small[:, near[b, j]] = pool[:, table[b, j]]
    q = rnd((154, 32, dim), g)
    starts = dev([0, 1, 151, 154])
    far = skv.page_attention(q, pool[0], pool[1], table, dev([200, 150, 64]), starts, 150, lse=True)
    got = skv.page_attention(q, small[0], small[1], near, dev([200, 150, 64]), starts, 150, lse=True)
    assert torch.equal(far[0], got[0]) and torch.equal(far[1], got[1])
    s = dict(q=q, k=small[0], v=small[1], table=near, starts=starts, pairs=pairs, group=4, page=page, ks=None, vs=None)
    compare(got, reference(s, dim ** -0.5, True), 154)


def test_streams_and_own_workspace(skv):
    g = torch.Generator(device="cuda").manual_seed(12)
    a = batch([(5000, 1), (300, 1)], 2, 4, 128, 16, BF16, g)
    b = batch([(3000, 200)], 2, 4, 128, 16, E4M3, g)
    want = [attend(skv, s) for s in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for st, s in zip(streams, (a, b)):
            with torch.cuda.stream(st):
                got.append(attend(skv, s))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    with pytest.raises(skv.SkvError) as e:
        attend(skv, a, work=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == skv.ERR_CAPACITY
    work = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    for s, y in ((a, want[0]), (b, want[1]), (a, want[0])):
        x = attend(skv, s, work=work)
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_binding_refusals(skv):
    g = torch.Generator(device="cuda").manual_seed(13)
    s = batch([(50, 1), (20, 1)], 2, 4, 128, 16, BF16, g)
    q, k, v, t, n = (s[x] for x in ("q", "k", "v", "table", "lens"))
    cpu = torch.zeros(2, dtype=torch.int32)
    bad = [lambda: skv.page_attention(q.half(), k, v, t, n), lambda: skv.page_attention(q[:1], k, v, t, n),
           lambda: skv.page_attention(q, k, v[:1], t, n), lambda: skv.page_attention(q, k, v, t.long(), n),
           lambda: skv.page_attention(q, k, v, t, n.long()), lambda: skv.page_attention(q, k, v, t, cpu),
           lambda: skv.page_attention(q, k, v, t[:1], n), lambda: skv.page_attention(q, k.float(), v.float(), t, n),
           lambda: skv.page_attention(q[:, :, :64], k, v, t, n),
           lambda: skv.page_attention(q, k, v, t, n, out=q[:1]),
           lambda: skv.page_attention(q, k, v, t, n, out=q[:, :1].expand(-1, 8, -1)),
           lambda: skv.page_attention(q, k, v, t, n, lse=torch.zeros((2, 7), device="cuda")),
           lambda: skv.page_attention(q, k, v, t, n, k_scale=torch.ones(3, device="cuda")),
           lambda: skv.page_attention(q, k, v, t, n, starts=dev([0, 1])),
           lambda: skv.page_attention(q, k.transpose(1, 3), v.transpose(1, 3), t, n),
           lambda: skv.page_write(q[:, :2], q[:, 2:4], k, v, dev([1])),
           lambda: skv.page_write(q[:, :2], q[:, 2:4], k[:1].expand(4, -1, -1, -1), v[:1].expand(4, -1, -1, -1), n),
           lambda: skv.page_write(q[:, :3], q[:, 3:6], k, v, n),
           lambda: skv.page_read(k, v, n, out=(q[:, :2, :64], q[:, 2:4, :64])),
           lambda: skv.page_plan(n, n, t, n.long(), 16, 2), lambda: skv.page_plan(n, n[:1], t, n, 16, 2)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(skv.SkvError):          # dims, pages and rows the library refuses
        skv.page_attention(q, k, v, t, n, k_scale=torch.ones(2, device="cuda"))


# ------------------------------------------------------------------ together
def test_a_step_captured_and_replayed(skv):
    """Plan, write and attend captured once at a padded size; each replay with other lengths, after eager work."""
    g = torch.Generator(device="cuda").manual_seed(14)
    B, page, heads, group, dim, T, W, N = 6, 16, 2, 4, 128, 24, 40, 300
    cache = skv.PageCache(skv.BF16, 1, N, page, heads, dim)
    lens, new = torch.ones(B, dtype=torch.int32, device="cuda"), torch.ones(B, dtype=torch.int32, device="cuda")
    table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
    free = torch.zeros(N, dtype=torch.int32, device="cuda")
    qkv = rnd((T, (group + 2) * heads, dim), g)
    q, k, v = qkv.split([group * heads, heads, heads], 1)
    out, lse = filled(q.shape, BF16, False), filled(q.shape[:2], torch.float32, False)

    def step():
        p = cache.plan(lens, new, table, free, T)
        cache.write(0, k, v, p.slots)
        cache.attend(0, q, table, lens, p.starts, 8, out=out, lse=lse)
        return p

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    table.fill_(-1)
    with torch.cuda.graph(graph):
        step()
    for news in ([1] * 6, [8, 1, 0, 3, 1, 1], [0] * 6, [4] * 6, [1, 8, 1, 8, 1, 5]):
        old = [int(x) for x in torch.randint(0, 500, (B,), generator=torch.Generator().manual_seed(sum(news)))]
        ids = torch.randperm(N, generator=g, device="cuda").to(torch.int32)
        table.fill_(-1)
        at = 0
        for b, o in enumerate(old):
            n = -(-o // page)
            table[b, :n] = ids[at:at + n]
            at += n
        free.zero_()
        free[:N - at] = ids[at:]
        cache.data.copy_(rnd(cache.data.shape, g))
        lens.copy_(dev(old) + dev(news))
        new.copy_(dev(news))
        qkv.copy_(rnd(qkv.shape, g))
        bits(out).fill_(0x1234)
        saved = table.clone(), cache.data.clone()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [x.clone() for x in (table, cache.data, out, lse)]
        table.copy_(saved[0])
        cache.data.copy_(saved[1])
        bits(out).fill_(0x1234)
        p = step()
        for x, y in zip((table, cache.data, out, lse), replayed):
            assert torch.equal(bits(x), bits(y))
        s = dict(q=q, k=cache.k[0], v=cache.v[0], table=table, starts=p.starts, group=group, page=page, ks=None, vs=None,
                 pairs=list(zip(lens.tolist(), news)))
        compare((out, lse), reference(s, dim ** -0.5, True), sum(news))
        assert (bits(out)[sum(news):] == 0x1234).all()
    cache.check()


@pytest.mark.parametrize("pages", [BF16, E4M3])
def test_two_graphs_of_chunks(skv, pages):
    """Attention of chunks, some in pieces, captured into two graphs that are replayed at once on two streams, with
    other lengths each time and eager work between: each replay is the eager result."""
    g = torch.Generator(device="cuda").manual_seed(23)
    sets = [batch([(3000, 60), (200, 100), (64, 40)], 2, 4, 128, 16, pages, g),
            batch([(2000, 150), (1500, 30), (31, 20)], 2, 4, 128, 32, pages, g)]
    streams, graphs, outs = [torch.cuda.Stream() for _ in sets], [], []
    for s, st in zip(sets, streams):
        attend(skv, s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            outs.append(skv.page_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["starts"], 150, lse=True))
        graphs.append(graph)
    full = [s["lens"].clone() for s in sets]
    for cut in (0, 7, 30, 1, 12, 0):
        for s, n in zip(sets, full):
            s["lens"].copy_(torch.clamp(n - cut * 3, min=1))
            s["q"].copy_(rnd(s["q"].shape, g))
        torch.cuda.synchronize()
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for s, out in zip(sets, outs):
            want = skv.page_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["starts"], 150, lse=True)
            assert torch.equal(bits(out[0]), bits(want[0])) and torch.equal(bits(out[1]), bits(want[1]))
            pairs = list(zip(s["lens"].tolist(), [n for _, n in s["pairs"]]))
            compare(out, reference(dict(s, pairs=pairs), 128 ** -0.5, True), s["starts"][-1].item())


@pytest.mark.parametrize("cid,mode", [(0, "RESIDUAL"), (2, "RESIDUAL_EXP")])
def test_a_stored_prefix_is_restored_and_attended(skv, cid, mode):
    """A request's way through the framework: its prefix found in the store, decoded into pages, its new tokens planned,
    written and attended, and at the end its cache saved into the store again, all bits kept."""
    cfg = gen.CONFIGS[cid].with_tokens(512, layers=2)
    L, heads, dim, page = 2, 8, 128, 16
    dt = skv.E4M3 if cfg.dtype == "e4m3" else skv.BF16
    tgt, prd = gen.residual_array(cfg, device="cuda")
    ct, cp = gen.residual_array(cfg, gen.CALIB, tokens=256, device="cuda")
    tabs = skv.fit_tables(dt, getattr(skv, mode), L, 2, cfg.channels, ct.cpu().numpy(), cp.cpu().numpy(), 256)
    store = skv.Store(arena_bytes=64 << 20)
    ids = list(range(512))
    store.put(tabs, tgt, prd, skv.block_hashes(ids))
    hit = store.lookup(skv.block_hashes(ids[:384] + [9] * 100))
    shared = 128 * hit.matched_blocks
    assert shared == 384

    cache = skv.PageCache(dt, L, 80, page, heads, dim)
    bits(cache.data).fill_(0)
    table = torch.full((1, 40), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(80, device="cuda").to(torch.int32)
    p = cache.plan(dev([shared]), dev([shared]), table, free, shared)
    cache.restore(store, tabs, hit.entry, prd[:, :, :shared].contiguous(), p.slots, 0, shared)
    store.release(hit.entry)
    taken = p.taken[-1].item()
    assert taken == shared // page
    # 128 new tokens: a chunk of 127, then a single one
    g = torch.Generator(device="cuda").manual_seed(15)
    at = shared
    for n in (127, 1):
        p = cache.plan(dev([at + n]), dev([n]), table, free[taken:], n)
        taken += p.taken[-1].item()
        for layer in range(L):
            k, v = (rnd((n, heads, dim), g) for _ in range(2))
            q = rnd((n, 32, dim), g)
            cache.write(layer, k, v, p.slots)
            got = cache.attend(layer, q, table, dev([at + n]), p.starts, n, lse=True)
            s = dict(q=q, k=cache.k[layer], v=cache.v[layer], table=table, starts=p.starts, group=4, page=page, ks=None,
                     vs=None, pairs=[(at + n, n)])
            compare(got, reference(s, dim ** -0.5, True), n)
            # the new rows as the cache's type holds them
            slot = p.slots.long()
            held = bits(cache.k[layer])[slot // page, slot % page]
            assert torch.equal(held, bits(k.to(cache.data.dtype)))
        at += n
    cache.check()
    # the whole cache back into the store: the restored prefix is the stored one, bit for bit
    whole = cache.plan(dev([512]), dev([512]), table, None, 512)
    entry, _ = cache.save(store, tabs, whole.slots, prd, skv.block_hashes([1] + ids[1:]))
    back = store.decode(tabs, entry, prd)
    assert torch.equal(back[:, :, :shared], tgt[:, :, :shared])
    k, v = skv.page_read(cache.k, cache.v, whole.slots)
    both = torch.stack([k, v], 1).flatten(3)
    assert torch.equal(bits(both), bits(back))
