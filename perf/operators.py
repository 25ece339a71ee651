"""Measured cases of the 8-bit key/value cache operators: the page plan, the
append that quantises new keys and values into the cache, and the attention
that reads it.

Every case is a dict of plain values.  `run` computes the operator in its
plain form (elementary torch operations in 32 bits) or, where `own` is set,
through the framework's entry points.  `exact` restates the operators in 64
bits, apart from the plain form.
"""
import math
import random

import torch

own = False

BLOCK = 16        # tokens that share one scale (per kv head)
E_MIN = -40       # smallest scale exponent: scale >= 2^-40
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one new token in each of many streams: the page bookkeeping of a token-by-token step
        dict(name="plan_tokens", op="plan", streams=256, new_lo=1, new_hi=1, old_lo=0, old_hi=9000, release=0,
             page=64, ragged=1),
        # whole latent frames (48 x 80 tokens) arrive in some streams while others end and give their pages back
        dict(name="plan_frames", op="plan", streams=24, new_lo=0, new_hi=3840, old_lo=0, old_hi=57600, release=4,
             page=64, ragged=2),
        # one token a stream written into the cache (24 heads of 128): latency
        dict(name="append_tokens", op="append", streams=32, new_lo=1, new_hi=1, old_lo=0, old_hi=1200, heads=24,
             group=1, d=128, page=64, ragged=3),
        # two 1080p latent frames (72 x 120 tokens each) of one stream: bandwidth
        dict(name="append_frames", op="append", streams=1, new_lo=17280, new_hi=17280, old_lo=8640, old_hi=8640,
             heads=24, group=1, d=128, page=64, ragged=4),
        # ragged chunks that start and end inside scale blocks; heads of 64, small pages
        dict(name="append_ragged", op="append", streams=13, new_lo=1, new_hi=701, old_lo=0, old_hi=333, heads=8,
             group=2, d=64, page=16, ragged=5),
        # the next token of one short stream: the smallest attention call
        dict(name="fwd_token", op="fwd", streams=1, new_lo=1, new_hi=1, old_lo=4100, old_hi=4100, heads=24, group=1,
             d=128, page=64, frame=0, window=0, ragged=6),
        # the next token of a few long streams (up to 30 latent frames of 48 x 80): bandwidth
        dict(name="fwd_token_long", op="fwd", streams=4, new_lo=1, new_hi=1, old_lo=57600, old_hi=115199, heads=24,
             group=1, d=128, page=64, frame=0, window=0, ragged=7),
        # a batch of very different lengths, six query heads to a kv head, small pages
        dict(name="fwd_token_shared", op="fwd", streams=48, new_lo=1, new_hi=1, old_lo=0, old_hi=12000, heads=4,
             group=6, d=128, page=16, frame=0, window=0, ragged=8),
        # a few tokens a stream under a token-causal mask, heads of 64 (draft tokens being verified)
        dict(name="fwd_few_tokens", op="fwd", streams=16, new_lo=1, new_hi=8, old_lo=100, old_hi=20000, heads=8,
             group=2, d=64, page=32, frame=1, window=0, ragged=9),
        # ragged prompts under a token-causal mask, heads of 64
        dict(name="fwd_ragged", op="fwd", streams=6, new_lo=50, new_hi=901, old_lo=0, old_hi=8000, heads=8, group=2,
             d=64, page=16, frame=1, window=0, ragged=10),
        # the next 720p latent frame (48 x 80 tokens) over ten frames: every query sees every key
        dict(name="fwd_frame_720p", op="fwd", streams=1, new_lo=3840, new_hi=3840, old_lo=34560, old_hi=34560,
             heads=24, group=1, d=128, page=64, frame=0, window=0, ragged=11),
        # two 1080p latent frames (72 x 120 tokens), frame-causal, each sees the last four frames
        dict(name="fwd_frames_1080p", op="fwd", streams=1, new_lo=17280, new_hi=17280, old_lo=34560, old_hi=34560,
             heads=24, group=1, d=128, page=128, frame=8640, window=4, ragged=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    ragged = rng.randrange(1000, 1 << 30)
    kind = rng.choice(["plan", "append", "append", "token", "token", "few", "chunk", "chunk"])
    page = rng.choice([16, 32, 64, 128])
    if kind == "plan":
        streams = _log_int(rng, 1, 1000)
        hi = _log_int(rng, 1, max(1, 90000 // streams))
        return dict(op="plan", streams=streams, new_lo=rng.choice([0, 1]), new_hi=hi, old_lo=0,
                    old_hi=_log_int(rng, 1, 30000), release=rng.randrange(0, 1 + streams // 4), page=page, ragged=ragged)
    heads, group, d = rng.choice([1, 2, 3, 4, 8, 12, 24]), rng.choice([1, 1, 2, 3, 4, 6, 8]), rng.choice([64, 128])
    case = dict(op="append" if kind == "append" else "fwd", heads=heads, group=group, d=d, page=page, ragged=ragged)
    if kind == "append":
        streams = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, max(1, 17280 * 24 * 128 // (streams * heads * d)))
        return dict(case, streams=streams, new_lo=rng.choice([0, 1]), new_hi=min(hi, 60000), old_lo=0,
                    old_hi=_log_int(rng, 1, 2000))
    if kind == "token":
        streams, new_hi, frame, window = _log_int(rng, 1, 128), 1, 0, 0
    elif kind == "few":
        streams, new_hi, frame, window = _log_int(rng, 1, 64), rng.randrange(2, 33), rng.choice([0, 1, 1, 4]), 0
    else:
        streams, new_hi = _log_int(rng, 1, 8), _log_int(rng, 40, 6000)
        frame = rng.choice([0, 1, rng.randrange(2, 2000)])
        window = rng.choice([0, 0, rng.randrange(1, 9)]) if frame > 1 else 0
    # no more than half of the largest listed work, in bytes read and in multiply-adds
    keys = min(115200, int(0.8e9 / (streams * heads * d * 2)),
               int(3.5e12 / (4.0 * streams * new_hi * heads * group * d)))
    old_hi = _log_int(rng, 1, max(2, keys))
    return dict(case, streams=streams, new_lo=1, new_hi=new_hi, old_lo=rng.choice([0, old_hi // 2]), old_hi=old_hi,
                frame=frame, window=window)


def _lengths(case):
    """(tokens held, new tokens) of every stream; new = -1: the stream ends."""
    r = random.Random(case["ragged"])
    old = [r.randint(case["old_lo"], case["old_hi"]) for _ in range(case["streams"])]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["streams"])]
    for s in r.sample(range(case["streams"]), min(case.get("release", 0), case["streams"])):
        new[s] = -1
    if max(new) < 1:
        new[0] = 1
    return old, new


def _pages(n, page):
    return -(-n // page)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _quantise_pool(gen, pages, heads, page, d):
    """A pool of pages filled with quantised normal values: e4m3 bytes and scales."""
    c = torch.empty((pages, heads, page, d), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((pages, heads, page // BLOCK), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (heads * page * d))
    for a in range(0, pages, step):
        b = min(pages, a + step)
        x = torch.randn((b - a, heads, page // BLOCK, BLOCK, d), generator=gen, device="cuda")
        # heads and blocks of different size, as a model's keys and values have
        x *= torch.exp2(2 * torch.rand((b - a, heads, page // BLOCK, 1, 1), generator=gen, device="cuda") - 1)
        e = _exponent(x.to(torch.bfloat16).float().abs().amax((-1, -2)))
        c[a:b] = (x.to(torch.bfloat16).float() * torch.exp2(-e.float())[..., None, None]).to(torch.float8_e4m3fn).view(
            b - a, heads, page, d)
        s[a:b] = torch.exp2(e.float())
    return c, s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    old, new = _lengths(case)
    page, streams = case["page"], case["streams"]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    after = [o + max(n, 0) for o, n in zip(old, new)]
    held = old if case["op"] == "plan" else after     # tokens whose pages the table lists before the call
    width = max(1, max(_pages(n, page) for n in after))
    width += width % 2
    counts = [_pages(n, page) for n in held]
    pages = sum(_pages(max(o, a), page) for o, a in zip(old, after)) + 5
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    st = dict(case=case, pages=pages, width=width)
    # block table: the streams' pages in random order, -1 where a stream has none
    cnt = ints(counts)
    first = (torch.cumsum(cnt, 0) - cnt)[:, None]
    col = torch.arange(width, device="cuda", dtype=torch.int32)[None]
    at = (first + col).clamp(max=pages - 1).long()
    st["table"] = torch.where(col < cnt[:, None], order[at], torch.full_like(at, -1, dtype=torch.int32)).contiguous()
    used, total_new = sum(counts), sum(max(n, 0) for n in new)
    if case["op"] == "plan":
        st["new"], st["lens"] = ints(new), ints(old)
        free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        free[:pages - used] = order[used:]
        st["free"], st["n_free"] = free, ints([pages - used])
        st["lens_out"], st["n_free_out"] = torch.empty_like(st["lens"]), torch.empty_like(st["n_free"])
        st["starts"] = torch.empty(streams + 1, dtype=torch.int32, device="cuda")
        st["slots"] = torch.empty(total_new + 3, dtype=torch.int32, device="cuda")
        st["result"] = torch.empty(4, dtype=torch.int32, device="cuda")
    else:
        heads, group, d = case["heads"], case["group"], case["d"]
        st["starts"] = ints([sum(new[:s]) for s in range(streams + 1)])
        st["lens"] = ints(after)
        # the new tokens' queries, keys and values: slices of one fused projection
        qkv = torch.randn((total_new, heads * (group + 2), d), generator=gen, device="cuda")
        st["qkv"] = qkv.to(torch.bfloat16)
        st["q"] = st["qkv"][:, :heads * group]
        st["k"] = st["qkv"][:, heads * group:heads * (group + 1)]
        st["v"] = st["qkv"][:, heads * (group + 1):]
        st["kc"], st["ks"] = _quantise_pool(gen, pages, heads, page, d)
        st["vc"], st["vs"] = _quantise_pool(gen, pages, heads, page, d)
        if case["op"] == "append":
            t = torch.arange(total_new, device="cuda")
            s = torch.searchsorted(st["starts"][1:].long(), t, right=True)
            pos = t - st["starts"][s] + ints(old)[s]
            st["slots"] = (st["table"][s, pos // page] * page + pos % page).to(torch.int32)
        else:
            st["o"] = torch.empty((total_new, heads * group, d), dtype=torch.bfloat16, device="cuda")
            st["lse"] = torch.empty((total_new, heads * group), dtype=torch.float32, device="cuda")
            st["max_new"] = max(new)
            st["scale"] = 1.0 / math.sqrt(d)
    if own:
        import video_dit_local_b200 as V
        st["geom"] = V.make_cache_geom(streams, case.get("heads", 1) * case.get("group", 1), case.get("heads", 1),
                                       case.get("d", 128), pages, page, width, case.get("frame", 0),
                                       case.get("window", 0))
        if case["op"] == "fwd":
            st["ws"] = torch.empty(V.vattn_cache_workspace_size(st["geom"], total_new, st["max_new"]),
                                   dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    if own:
        import video_dit_local_b200 as V
        if op == "plan":
            V.vattn_cache_plan(st["geom"], st["new"], st["lens"], st["table"], st["free"], st["n_free"],
                               st["lens_out"], st["n_free_out"], st["starts"], st["slots"], st["result"])
            return _plan_outputs(st)
        if op == "append":
            V.vattn_cache_append(st["geom"], st["k"], st["v"], st["slots"], st["kc"], st["vc"], st["ks"], st["vs"])
            return [st["kc"], st["vc"], st["ks"], st["vs"]]
        V.vattn_cache_fwd(st["geom"], st["q"], st["starts"], st["lens"], st["table"], st["kc"], st["vc"], st["ks"],
                          st["vs"], st["scale"], st["max_new"], st["o"], st["lse"], st["ws"])
        return [st["o"], st["lse"]]
    if op == "plan":
        return _plain_plan(st)
    if op == "append":
        _plain_append(st["k"], st["slots"], st["kc"], st["ks"])
        _plain_append(st["v"], st["slots"], st["vc"], st["vs"])
        return [st["kc"], st["vc"], st["ks"], st["vs"]]
    return _plain_fwd(st)


def _plan_outputs(st):
    return [st["lens_out"], st["n_free_out"], st["table"], st["free"], st["starts"], st["slots"], st["result"]]


def _plain_plan(st):
    page, lens, new, table, free = st["case"]["page"], st["lens"], st["new"], st["table"], st["free"]
    ends = new < 0
    add = torch.where(ends, 0, new)
    have = (lens + page - 1) // page
    want = torch.where(ends, 0, (lens + add + page - 1) // page)
    take = torch.where(ends, 0, want - have)
    give = torch.where(ends, have, 0)
    give0, take0 = torch.cumsum(give, 0) - give, torch.cumsum(take, 0) - take
    avail = st["n_free"] + give.sum()
    col = torch.arange(table.shape[1], device="cuda")[None]
    # pages of the streams that end go on top of the free stack, in stream order
    s, j = torch.nonzero(col < give[:, None], as_tuple=True)
    free[(st["n_free"] + give0[s] + j).long()] = table[s, j]
    # new pages come off its top, in stream order
    s, j = torch.nonzero((col >= have[:, None]) & (col < (have + take)[:, None]), as_tuple=True)
    table[s, j] = free[(avail - 1 - take0[s] - (j - have[s])).long()]
    st["starts"][0] = 0
    st["starts"][1:] = torch.cumsum(add, 0)
    st["lens_out"].copy_(torch.where(ends, 0, lens + add))
    st["n_free_out"].copy_(avail - take.sum())
    t = torch.arange(st["slots"].numel(), device="cuda")
    s = torch.searchsorted(st["starts"][1:].long(), t, right=True)
    real = s < new.numel()
    s = s.clamp(max=new.numel() - 1)
    pos = torch.where(real, t - st["starts"][s] + lens[s], 0)
    st["slots"].copy_(torch.where(real, table[s, pos // page] * page + pos % page, -1))
    st["result"].copy_(torch.stack([torch.zeros_like(avail[0]), add.sum(), st["n_free_out"][0],
                                    st["lens_out"].max()]))
    return _plan_outputs(st)


def _exponent(absmax):
    """Smallest e >= E_MIN with absmax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    m, e = torch.frexp(absmax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(absmax > 0, e, torch.full_like(e, E_MIN)).clamp(min=E_MIN)


def _plain_append(x, slots, cache, scales):
    pages, heads, page, d = cache.shape
    slots = slots.long()
    x = x.float()
    blk, off = slots // BLOCK, slots % BLOCK
    pg, sub = blk // (page // BLOCK), blk % (page // BLOCK)
    e_tok = _exponent(x.abs().amax(-1))                                              # [n, heads]
    nblk = pages * page // BLOCK
    e_new = torch.full((nblk, heads), E_MIN, dtype=e_tok.dtype, device=x.device)
    e_new.scatter_reduce_(0, blk[:, None].expand(-1, heads), e_tok, "amax")
    first = torch.full((nblk,), BLOCK, dtype=torch.int64, device=x.device)
    first.scatter_reduce_(0, blk, off, "amin")                                       # tokens the block held before
    lead = torch.nonzero(off == first[blk])[:, 0]                                    # one token for each block
    b, p, u, held = blk[lead], pg[lead], sub[lead], first[blk[lead]]
    e_old = torch.log2(scales[p, :, u]).to(e_tok.dtype)                              # [blocks, heads]
    e_blk = torch.where(held[:, None] > 0, torch.maximum(e_old, e_new[b]), e_new[b])
    e_new[b] = e_blk
    c = cache.view(pages, heads, page // BLOCK, BLOCK, d)
    was = c[p, :, u].float() * torch.exp2((e_old - e_blk).float())[:, :, None, None]
    kept = torch.arange(BLOCK, device=x.device) < held[:, None]
    c[p, :, u] = torch.where(kept[:, None, :, None], was, 0.0).to(cache.dtype)
    scales[p, :, u] = torch.exp2(e_blk.float())
    c[pg, :, sub, off] = (x * torch.exp2(-e_new[blk].float())[..., None]).to(cache.dtype)


def _bounds(case, n, length, device):
    """First and one past the last key that each of a stream's n new tokens sees."""
    p = length - n + torch.arange(n, device=device)
    if case["frame"] == 0:
        return torch.zeros_like(p), torch.full_like(p, length)
    f = torch.div(p, case["frame"], rounding_mode="floor")
    hi = torch.clamp((f + 1) * case["frame"], max=length)
    lo = torch.clamp((f - case["window"] + 1) * case["frame"], min=0) if case["window"] else torch.zeros_like(p)
    return lo, hi


def _plain_fwd(st):
    case = st["case"]
    heads, group, d, page = case["heads"], case["group"], case["d"], case["page"]
    old, new = _lengths(case)
    t0 = 0
    for s, (o, n) in enumerate(zip(old, new)):
        length = o + n
        used = st["table"][s, :_pages(length, page)].long()
        lo, hi = _bounds(case, n, length, "cuda")
        key = torch.arange(length, device="cuda")
        seen = ((key >= lo[:, None]) & (key < hi[:, None])).repeat_interleave(group, 0)
        step = max(1, min(heads, (1 << 28) // max(1, n * group * length)))
        for h in range(0, heads, step):
            e = min(heads, h + step)
            k, v = (_plain_gather(c, sc, used, h, e, length) for c, sc in ((st["kc"], st["ks"]), (st["vc"], st["vs"])))
            q = st["q"][t0:t0 + n, h * group:e * group].float().view(n, e - h, group, d)
            q = q.transpose(0, 1).reshape(e - h, n * group, d)
            x = torch.where(seen, torch.matmul(q, k.transpose(1, 2)) * st["scale"], -math.inf)
            m = x.amax(-1, keepdim=True)
            m = torch.where(m == -math.inf, 0.0, m)
            w = torch.exp(x - m)
            z = w.sum(-1, keepdim=True)
            out = torch.where(z > 0, torch.matmul(w, v) / z, 0.0)
            put = lambda y: y.view(e - h, n, group, -1).transpose(0, 1).reshape(n, (e - h) * group, -1)  # noqa: E731
            st["o"][t0:t0 + n, h * group:e * group] = put(out).to(torch.bfloat16)
            st["lse"][t0:t0 + n, h * group:e * group] = put(m + torch.log(z))[..., 0]
        t0 += n
    return [st["o"], st["lse"]]


def _plain_gather(cache, scales, used, h, e, length):
    """Dequantised rows of heads [h, e): [heads, length, d]."""
    x = cache[used, h:e].float()
    pages, heads, page, d = x.shape
    x = x.view(pages, heads, page // BLOCK, BLOCK, d) * scales[used, h:e][..., None, None]
    return x.view(pages, heads, page, d).transpose(0, 1).reshape(heads, pages * page, d)[:, :length]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    old, new = _lengths(case)
    page, streams = case["page"], case["streams"]
    if case["op"] == "plan":
        moved = sum(_pages(o, page) if n < 0 else _pages(o + n, page) - _pages(o, page) for o, n in zip(old, new))
        return {"bytes": 4 * (4 * streams + 2 * moved + sum(max(n, 0) for n in new)), "flops": 0}
    heads, group, d = case["heads"], case["group"], case["d"]
    n = sum(new)
    if case["op"] == "append":
        blocks = sum(_pages(o + m, BLOCK) - o // BLOCK for o, m in zip(old, new) if m)
        return {"bytes": n * heads * d * 6 + blocks * heads * 8 + 4 * n, "flops": 0}
    pairs, keys = 0, 0
    for o, m in zip(old, new):
        lo, hi = _bounds(case, m, o + m, "cpu")
        seen = torch.clamp(hi - lo, min=0)
        pairs += int(seen.sum())
        keys += max(0, int(hi.max()) - int(lo.min()))
    return {"bytes": keys * heads * (2 * d + 8 / BLOCK) + n * heads * group * (4 * d + 4) + 4 * keys / page,
            "flops": 4.0 * pairs * heads * group * d}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _round_e4m3(x):
    """Nearest e4m3 value (ties to even) of float64 x, |x| <= 448: steps of 2^(floor(log2|x|) - 3), 2^-9 at least."""
    _, e = torch.frexp(x.abs())
    step = torch.exp2(torch.clamp(e.double() - 4, min=-9.0))
    return torch.round(x / step) * step


def _exact_append(x, slots, cache, scales):
    n, heads, d = x.shape
    page = cache.shape[2]
    vals, sc = cache.double().cpu(), scales.double().cpu()
    x, slots = x.double().cpu(), slots.tolist()
    i = 0
    while i < n:
        b, start = slots[i] // BLOCK, slots[i] % BLOCK
        j = i
        while j < n and slots[j] // BLOCK == b:
            j += 1
        p, u = b * BLOCK // page, b * BLOCK % page // BLOCK
        rows = x[i:j].transpose(0, 1)                                                 # [heads, j - i, d]
        need = rows.abs().amax((1, 2)) / E4M3_MAX
        e = torch.ceil(torch.log2(torch.clamp(need, min=2.0 ** E_MIN)))
        e = torch.where(torch.exp2(e - 1) >= torch.clamp(need, min=2.0 ** E_MIN), e - 1, e)
        if start:
            e = torch.maximum(e, torch.log2(sc[p, :, u]))
        blk = vals[p, :, u * BLOCK:(u + 1) * BLOCK]
        blk[:, :start] = _round_e4m3(blk[:, :start] * (sc[p, :, u] / torch.exp2(e))[:, None, None])
        blk[:, start:start + j - i] = _round_e4m3(rows / torch.exp2(e)[:, None, None])
        blk[:, start + j - i:] = 0
        sc[p, :, u] = torch.exp2(e)
        i = j
    return vals, sc


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "plan":
        return None
    if case["op"] == "append":
        kv = [_exact_append(st["k"], st["slots"], st["kc"], st["ks"]),
              _exact_append(st["v"], st["slots"], st["vc"], st["vs"])]
        return [kv[0][0], kv[1][0], kv[0][1], kv[1][1]]
    heads, group, page, scale = case["heads"], case["group"], case["page"], st["scale"]
    old, new = _lengths(case)
    out, lse = st["q"].new_zeros(st["q"].shape, dtype=torch.float64), st["lse"].double()
    t0 = 0
    for s, (o, n) in enumerate(zip(old, new)):
        length = o + n
        pages = st["table"][s, :_pages(length, page)].long()
        pos = torch.arange(length, device="cuda")
        at = torch.arange(n, device="cuda") + o
        unseen = torch.zeros((n, length), dtype=torch.bool, device="cuda")
        if case["frame"]:
            # a key is seen when its frame is the query's or an earlier one, and within the window
            back = at[:, None] // case["frame"] - pos // case["frame"]
            unseen = (back < 0) | ((back >= case["window"]) if case["window"] else (back < 0))
        for h in range(heads):
            kv = []
            for c, sc in ((st["kc"], st["ks"]), (st["vc"], st["vs"])):
                rows = c[pages, h].double().view(-1, c.shape[-1])[:length]
                kv.append(rows * sc[pages, h].double().repeat_interleave(BLOCK, 1).view(-1)[:length, None])
            for g in range(group):
                x = (st["q"][t0:t0 + n, h * group + g].double() * scale) @ kv[0].T
                x.masked_fill_(unseen, -math.inf)
                z = torch.logsumexp(x, -1)
                lse[t0:t0 + n, h * group + g] = z
                out[t0:t0 + n, h * group + g] = torch.exp(x.sub_(torch.where(z == -math.inf, 0.0, z)[:, None])) @ kv[1]
        t0 += n
    return [out, lse]
