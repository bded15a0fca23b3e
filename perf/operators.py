"""Cases, plain forms and 64-bit values of the serving operators around the MoE layer:

  append   rotary positions for the new tokens' queries and keys, and their keys and values written into the paged cache
  attend   attention of each sequence's new tokens over its pages of the cache
  verify   drafted tokens accepted or replaced by the target's probabilities, from given random numbers

With `own` set, run() calls the framework; otherwise it computes the same in elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
ROPE_BASE = 10000.0


# ---------------------------------------------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # one user's next token: the latency of the smallest call
        dict(name="append one token", op="append", seqs=1, new_min=1, new=1, past_min=517, past=517, heads=32, kv_heads=8, dim=128,
             page=16, cache="bf16", rot=128, interleaved=False, axes=1),
        # drafted tokens of a full serving batch into an E4M3 cache, positions of an image prompt on three axes
        dict(name="append drafts e4m3", op="append", seqs=64, new_min=3, new=5, past_min=200, past=9000, heads=32, kv_heads=8, dim=128,
             page=32, cache="e4m3", rot=96, interleaved=True, axes=3),
        # the prompts of a few users at once (chunked prefill), ragged
        dict(name="append prompts", op="append", seqs=7, new_min=301, new=2041, past_min=0, past=700, heads=32, kv_heads=8, dim=128,
             page=16, cache="bf16", rot=128, interleaved=False, axes=1),
        # one user's next token over a short context: latency
        dict(name="attend one short", op="attend", seqs=1, new_min=1, new=1, len_min=517, len=517, heads=32, kv_heads=8, dim=128,
             page=16, cache="bf16", window=0),
        # one user over a long document
        dict(name="attend one long", op="attend", seqs=1, new_min=1, new=1, len_min=131072, len=131072, heads=32, kv_heads=8, dim=128,
             page=64, cache="bf16", window=0),
        # a serving batch of uneven lengths, one new token each
        dict(name="attend batch", op="attend", seqs=64, new_min=1, new=1, len_min=37, len=8190, heads=32, kv_heads=8, dim=128, page=16,
             cache="bf16", window=0),
        # many short chats over an E4M3 cache
        dict(name="attend chats e4m3", op="attend", seqs=256, new_min=1, new=1, len_min=1, len=2047, heads=64, kv_heads=8, dim=128,
             page=32, cache="e4m3", window=0),
        # the step that scores up to four drafted tokens a sequence
        dict(name="attend drafts", op="attend", seqs=32, new_min=2, new=5, len_min=100, len=12000, heads=32, kv_heads=8, dim=128,
             page=16, cache="bf16", window=0),
        # fp32 model with odd sizes and a sliding window
        dict(name="attend fp32 window", op="attend", seqs=13, new_min=1, new=3, len_min=1, len=5001, heads=15, kv_heads=5, dim=80,
             page=7, cache="f32", window=1023),
        # one user's four drafts: latency
        dict(name="verify one", op="verify", seqs=1, new_min=5, new=5, vocab=32000, dtype="f32"),
        # a serving batch
        dict(name="verify batch", op="verify", seqs=64, new_min=5, new=5, vocab=129280, dtype="f32"),
        # an uneven batch with an odd vocabulary
        dict(name="verify ragged", op="verify", seqs=200, new_min=1, new=9, vocab=50021, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "verify"])
    while True:
        if op == "verify":
            new = rng.randint(1, 9)
            c = dict(op=op, seqs=_log(rng, 1, 256), new_min=rng.randint(1, new), new=new, vocab=_log(rng, 1000, 131072), dtype=rng.choice(["f32", "f32", "bf16"]))
            if c["seqs"] * new * c["vocab"] <= 9e7:
                return c
            continue
        cache = rng.choice(["bf16", "bf16", "e4m3", "f32"])
        kv, group = rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        dim = rng.choice([64, 80, 96, 112, 128, 128, 128, 192, 256])
        c = dict(op=op, heads=kv * group, kv_heads=kv, dim=dim, page=rng.choice([1, 7, 16, 16, 32, 48, 64, 128]), cache=cache)
        if op == "append":
            new = _log(rng, 1, 2048)
            c.update(seqs=_log(rng, 1, 256), new_min=rng.randint(1, new), new=new, past_min=0, past=_log(rng, 1, 9000),
                     rot=2 * rng.randint(3, dim // 2), interleaved=rng.random() < 0.5, axes=rng.choice([1, 1, 3]))
            rows, slots = sum(_news(c)), sum(_news(c)) + c["seqs"] * (c["past"] / 2 + c["page"])
            if rows * (c["heads"] + 2 * kv) * dim <= 9000 * 48 * 128 and slots * kv * dim <= 1.5e8 and slots <= 600000:
                return c
        else:
            new, length = rng.choice([1, 1, 1, rng.randint(2, 8)]), _log(rng, 16, 60000)
            c.update(seqs=_log(rng, 1, 256), new_min=rng.randint(1, new), new=new, len_min=rng.randint(1, length), len=length,
                     window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]))
            if c["seqs"] * length * kv * dim <= 64 * 8190 * 8 * 128 and c["seqs"] * length * c["heads"] * new <= 9e7 and c["seqs"] * length <= 2e6:
                return c


# ---------------------------------------------------------------------------------------------------------------------------------
# inputs

def _spread(lo, hi, n):
    """n lengths from lo to hi, evenly."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]


def _news(c):
    return _spread(c["new_min"], c["new"], c["seqs"])


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _table(rs, lengths, page):
    """A block table of pages in random order over a pool with some pages to spare, and the pool's size."""
    pages = [-(-n // page) for n in lengths]
    total = sum(pages)
    pool = -(-int(sum(lengths)) // page) + len(pages) + 3  # at least total, and the same for every seed
    ids = rs.permutation(pool)[:total].astype(np.int32)
    table = np.zeros((len(lengths), max(1, max(pages))), np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = ids[at:at + n]
        at += n
    return torch.from_numpy(table).cuda(), pool


def _cache(g, c, pool):
    """Keys or values as a cache holds them (E4M3: codes, and a scale for each token and head)."""
    shape = (pool, c["page"], c["kv_heads"], c["dim"])
    if c["cache"] != "e4m3":
        return torch.empty(shape, dtype=_TYPES[c["cache"]], device="cuda").normal_(generator=g), None
    codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(shape[:3], dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (shape[1] * shape[2] * shape[3]))
    for i in range(0, pool, step):
        x = torch.empty((min(step, pool - i),) + shape[1:], dtype=torch.float32, device="cuda").normal_(generator=g)
        amax = x.abs().amax(-1)
        codes[i:i + step] = (x * (E4M3_MAX / amax)[..., None]).to(torch.float8_e4m3fn)
        scale[i:i + step] = amax / E4M3_MAX
    return codes, scale.transpose(1, 2).contiguous()  # [page][head][token]


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    order = rs.permutation(case["seqs"])
    new = np.array(_news(case), np.int64)[order]
    cu = np.zeros(case["seqs"] + 1, np.int32)
    cu[1:] = np.cumsum(new)
    T = int(cu[-1])
    s = {"case": case, "T": T, "cu": torch.from_numpy(cu).cuda()}
    make = {"append": _prepare_append, "attend": _prepare_attend, "verify": _prepare_verify}[case["op"]]
    make(s, case, rs, g, new)
    return s


def _attn_handle(s, c, **more):
    import sparse_mixture_experts_router_gb300 as moe
    kind = {"bf16": moe.MOE_BF16, "f32": moe.MOE_F32, "e4m3": moe.MOE_E4M3}[c["cache"]]
    s["cfg"] = moe.attn_config(n_seqs=c["seqs"], n_tokens=s["T"], max_new=c["new"], n_heads=c["heads"], n_kv_heads=c["kv_heads"],
                               head_dim=c["dim"], page_size=c["page"], n_pages=s["pool"], max_pages=s["table"].shape[1],
                               dtype=moe.MOE_F32 if c["cache"] == "f32" else moe.MOE_BF16, cache_dtype=kind, **more)


def _prepare_append(s, c, rs, g, new):
    T, D = s["T"], c["dim"]
    lengths = new + np.array(_spread(c["past_min"], c["past"], c["seqs"]))[rs.permutation(c["seqs"])]
    s["len"] = torch.from_numpy(lengths.astype(np.int32)).cuda()
    s["table"], s["pool"] = _table(rs, lengths, c["page"])
    wide = (c["heads"] + 2 * c["kv_heads"]) * D
    kind = torch.float32 if c["cache"] == "f32" else torch.bfloat16
    qkv = torch.empty((T, wide), dtype=kind, device="cuda").normal_(generator=g)  # the output of one projection
    s["q"], s["k"], s["v"] = (t.unflatten(1, (-1, D)) for t in qkv.split([c["heads"] * D, c["kv_heads"] * D, c["kv_heads"] * D], 1))
    s["k_cache"], s["k_scale"] = _cache(g, c, s["pool"])
    s["v_cache"], s["v_scale"] = _cache(g, c, s["pool"])
    # one axis: a token's place in its sequence; three: time, height and width of image patches behind a long text
    s["pos"] = torch.from_numpy(np.stack([rs.randint(0, 1 << 17, T), rs.randint(0, 1 << 17, T), rs.randint(0, 1 << 17, T)]).astype(np.int32)).cuda() if c["axes"] == 3 else None
    s["sections"] = _sections(c)
    s["q_out"] = torch.empty((T, c["heads"], D), dtype=kind, device="cuda")
    if own:
        import sparse_mixture_experts_router_gb300 as moe
        _attn_handle(s, c, rot_dim=c["rot"], rot_interleaved=c["interleaved"], rot_sections=s["sections"], rope_base=ROPE_BASE,
                     q_stride=wide, k_stride=wide, v_stride=wide)
        s["ws"] = moe.workspace(s["cfg"], "append")


def _sections(c):
    pairs = c["rot"] // 2
    return [pairs - 2 * (pairs // 3), pairs // 3, pairs // 3] if c["axes"] == 3 else [pairs, 0, 0]


def _prepare_attend(s, c, rs, g, new):
    lengths = np.maximum(np.array(_spread(c["len_min"], c["len"], c["seqs"]))[rs.permutation(c["seqs"])], 0)
    s["len"] = torch.from_numpy(lengths.astype(np.int32)).cuda()
    s["table"], s["pool"] = _table(rs, lengths, c["page"])
    kind = torch.float32 if c["cache"] == "f32" else torch.bfloat16
    s["q"] = (2 * torch.empty((s["T"], c["heads"], c["dim"]), dtype=torch.float32, device="cuda").normal_(generator=g)).to(kind)
    s["k_cache"], s["k_scale"] = _cache(g, c, s["pool"])
    s["v_cache"], s["v_scale"] = _cache(g, c, s["pool"])
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((s["T"], c["heads"]), dtype=torch.float32, device="cuda")
    if own:
        import sparse_mixture_experts_router_gb300 as moe
        _attn_handle(s, c, window=c["window"])
        s["ws"] = moe.workspace(s["cfg"], "attention")


def _prepare_verify(s, c, rs, g, new):
    T, V, kind = s["T"], c["vocab"], _TYPES[c["dtype"]]
    s["p"] = torch.empty((T, V), dtype=kind, device="cuda")
    s["q"] = torch.empty((T, V), dtype=kind, device="cuda")
    s["tokens"] = torch.empty(T, dtype=torch.int32, device="cuda").random_(0, V, generator=g)
    drafted = torch.empty(T, dtype=torch.int32, device="cuda")
    step = max(1, (1 << 26) // V)
    for i in range(0, T, step):  # a peaked target, and a draft model that is some way off it
        logits = torch.empty((min(step, T - i), V), device="cuda").normal_(0, 3, generator=g)
        s["p"][i:i + step] = torch.softmax(logits, 1)
        logits += torch.empty_like(logits).normal_(0, 0.6, generator=g)
        q = torch.softmax(logits, 1)
        s["q"][i:i + step] = q
        drafted[i:i + step] = (q / torch.empty_like(q).exponential_(generator=g)).argmax(1)
    first = torch.zeros(T, dtype=torch.bool, device="cuda")
    first[s["cu"][:-1].long()] = True
    s["tokens"] = torch.where(first, s["tokens"], drafted.roll(1))  # row j's draft is the input of row j + 1
    s["u"] = torch.empty(T, device="cuda").uniform_(generator=g)
    s["u_sample"] = torch.empty(c["seqs"], device="cuda").uniform_(generator=g)
    s["len"] = torch.from_numpy((new + rs.randint(0, 5000, c["seqs"])).astype(np.int32)).cuda()
    s["out"] = torch.empty(T, dtype=torch.int32, device="cuda")
    s["accepted"] = torch.empty(c["seqs"], dtype=torch.int32, device="cuda")
    s["next"] = torch.empty(c["seqs"], dtype=torch.int32, device="cuda")
    if own:
        import sparse_mixture_experts_router_gb300 as moe
        s["cfg"] = moe.verify_config(n_seqs=c["seqs"], n_tokens=T, max_new=c["new"], vocab=V,
                                     dtype=moe.MOE_F32 if c["dtype"] == "f32" else moe.MOE_BF16)
        s["ws"] = moe.workspace(s["cfg"], "verify")


# ---------------------------------------------------------------------------------------------------------------------------------
# one pass

def run(s):
    op = s["case"]["op"]
    if own:
        import sparse_mixture_experts_router_gb300 as moe
        if op == "append":
            moe.moe_rope_append(s["cfg"], s["q"], s["k"], s["v"], s["pos"], s["cu"], s["len"], s["table"], s["q_out"], s["k_cache"],
                                s["v_cache"], s["k_scale"], s["v_scale"], s["ws"])
        elif op == "attend":
            moe.moe_paged_attention(s["cfg"], s["q"], s["cu"], s["len"], s["table"], s["k_cache"], s["v_cache"], s["k_scale"],
                                    s["v_scale"], s["out"], s["lse"], s["ws"])
            return {"out": s["out"], "lse": s["lse"]}
        else:
            moe.moe_verify_drafts(s["cfg"], s["p"], s["q"], s["tokens"], s["u"], s["u_sample"], s["cu"], s["len"], s["out"],
                                  s["accepted"], s["next"], s["ws"])
            return {"tokens": s["out"], "accepted": s["accepted"], "next": s["next"]}
    elif op == "append":
        s["q_out"] = _plain_append(s)
    else:
        return (_plain_attend if op == "attend" else _plain_verify)(s)
    r = {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["k_scale"] is not None:
        r.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return r


def _rows(s):
    """Each new token's sequence and its place among that sequence's new tokens."""
    t = torch.arange(s["T"], device="cuda")
    cu = s["cu"].long()
    b = torch.searchsorted(cu[1:], t, right=True)
    return b, t - cu[b], (cu[1:] - cu[:-1])


def _plain_append(s):
    c, cu = s["case"], s["cu"]
    b, j, new = _rows(s)
    at = s["len"].long()[b] - new[b] + j
    slot, place = s["table"].long()[b, at // c["page"]], at % c["page"]
    pairs = c["rot"] // 2
    i = torch.arange(pairs, device="cuda")
    axis = (i >= s["sections"][0]).long() + (i >= s["sections"][0] + s["sections"][1]).long()
    pos = at[:, None].double() if s["pos"] is None else s["pos"].double().t()[:, axis]
    angle = pos * torch.exp(i.double() * (-2.0 / c["rot"] * math.log(ROPE_BASE)))  # far positions: 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def rotate(x):
        x = x.float()
        y = x.clone()
        lo, hi = (slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["interleaved"] else (slice(0, pairs), slice(pairs, c["rot"]))
        y[..., lo] = x[..., lo] * cos - x[..., hi] * sin
        y[..., hi] = x[..., hi] * cos + x[..., lo] * sin
        return y

    def store(cache, scale, x):
        if scale is None:
            cache[slot, place] = x.to(cache.dtype)
        else:
            amax = x.abs().amax(-1)
            inv = torch.where(amax > 0, E4M3_MAX / amax, 0.0)
            cache.view(torch.uint8)[slot, place] = (x * inv[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            scale[slot, :, place] = amax / E4M3_MAX

    store(s["k_cache"], s["k_scale"], rotate(s["k"]))
    store(s["v_cache"], s["v_scale"], s["v"].float())
    return rotate(s["q"]).to(s["q"].dtype)


def _plain_attend(s):
    c, cu, D = s["case"], s["cu"].long(), s["case"]["dim"]
    B, N, H, K = c["seqs"], c["new"], c["heads"], c["kv_heads"]
    G, L = H // K, c["len"]
    at = torch.arange(L, device="cuda")
    page, place = s["table"].long()[:, at // c["page"]], at % c["page"]
    length = s["len"].long()

    def gather(cache, scale):
        if scale is None:
            return cache[page, place].float()
        return cache.view(torch.uint8)[page, place].view(torch.float8_e4m3fn).float() * scale.transpose(1, 2)[page, place][..., None]

    row = (cu[:-1, None] + torch.arange(N, device="cuda")).clamp(max=s["T"] - 1)
    q = s["q"].float()[row].view(B, N, K, G, D).permute(0, 2, 1, 3, 4).reshape(B, K, N * G, D)
    score = torch.matmul(q, gather(s["k_cache"], s["k_scale"]).permute(0, 2, 3, 1)).view(B, K, N, G, L) * (1 / math.sqrt(D))
    pos = (length - (cu[1:] - cu[:-1]))[:, None] + torch.arange(N, device="cuda")
    seen = (at <= pos[..., None]) & (at < length[:, None, None])
    if c["window"]:
        seen &= at > pos[..., None] - c["window"]
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    w = torch.exp(score - top)
    total = w.sum(-1, keepdim=True)
    v = gather(s["v_cache"], s["v_scale"])
    v.masked_fill_((at >= length[:, None])[..., None, None], 0.0)
    o = torch.matmul(w.view(B, K, N * G, L), v.permute(0, 2, 1, 3)).view(B, K, N, G, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(B, N, H, D)
    lse = (top + total.log()).squeeze(-1).permute(0, 2, 1, 3).reshape(B, N, H)
    b, j, _ = _rows(s)
    return {"out": o[b, j].to(s["q"].dtype), "lse": lse[b, j]}


def _plain_verify(s):
    c, cu = s["case"], s["cu"].long()
    N, V, T = c["new"], c["vocab"], s["T"]
    new = cu[1:] - cu[:-1]
    j = torch.arange(max(1, N - 1), device="cuda")
    row = (cu[:-1, None] + j).clamp(max=T - 1)
    x = s["tokens"].long()[(row + 1).clamp(max=T - 1)]
    take = s["u"][row].double() * s["q"][row, x].double() < s["p"][row, x].double()  # next to a border: 64 bits
    take &= j < (new - 1)[:, None]
    a = take.long().cumprod(1).sum(1)
    last = cu[:-1] + a
    p = s["p"][last].double()
    rest = torch.where((a < new - 1)[:, None], (p - s["q"][last].double()).clamp(min=0), p)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, p)
    mass = rest.cumsum(1)
    drawn = (mass > s["u_sample"].double()[:, None] * mass[:, -1:]).to(torch.int8).argmax(1)
    b, j, _ = _rows(s)
    following = s["tokens"].roll(-1)
    out = torch.where(j < a[b], following.long(), torch.where(j == a[b], drawn[b], -1))
    return {"tokens": out.int(), "accepted": a.int(), "next": (s["len"].long() - (new - 1 - a)).int()}


# ---------------------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    c, T = case, sum(_news(case))
    if c["op"] == "verify":
        # one row of the target and, after a rejection (about a quarter of the drafts), one of the draft model
        size = 2 if c["dtype"] == "bf16" else 4
        rejected = sum(1 - 0.75 ** (n - 1) for n in _news(c))
        return {"bytes": (c["seqs"] + rejected) * c["vocab"] * size + T * 20 + c["seqs"] * 24, "flops": 3.0 * (c["seqs"] + rejected) * c["vocab"]}
    size, cached = (4, 4) if c["cache"] == "f32" else (2, 1 if c["cache"] == "e4m3" else 2)
    line = c["dim"] * cached + (4 if c["cache"] == "e4m3" else 0)  # a key or a value as the cache holds it
    if c["op"] == "append":
        read = T * (c["heads"] + 2 * c["kv_heads"]) * c["dim"] * size
        return {"bytes": read + T * (c["heads"] * c["dim"] * size + 2 * c["kv_heads"] * line) + T * (12 if c["axes"] == 3 else 4),
                "flops": 3.0 * T * (c["heads"] + c["kv_heads"]) * c["rot"]}
    lengths = _spread(c["len_min"], c["len"], c["seqs"])
    if c["window"]:
        lengths = [min(n, c["window"] + c["new"] - 1) for n in lengths]
    keys = sum(lengths)
    return {"bytes": 2.0 * keys * c["kv_heads"] * line + T * c["heads"] * (2 * c["dim"] * size + 4) + keys / c["page"] * 4,
            "flops": 4.0 * keys * c["heads"] * c["dim"] * T / c["seqs"]}


# ---------------------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "verify": _exact_verify}[case["op"]](s, case)


def _exact_append(s, c):
    cu, length, table = s["cu"].tolist(), s["len"].tolist(), s["table"].cpu().numpy()
    at = np.concatenate([np.arange(n - (e - b), n) for b, e, n in zip(cu, cu[1:], length)])
    seq = np.repeat(np.arange(c["seqs"]), np.diff(cu))
    slot, place = torch.from_numpy(table[seq, at // c["page"]].astype(np.int64)).cuda(), torch.from_numpy(at % c["page"]).cuda()
    pairs = c["rot"] // 2
    pos = np.repeat(at[:, None], pairs, 1) if s["pos"] is None else np.repeat(s["pos"].cpu().numpy(), s["sections"], 0).T
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"), torch.from_numpy(pos * ROPE_BASE ** (-np.arange(pairs) / pairs)).cuda())

    def rotated(x):
        x = x.double()
        r = x[..., :c["rot"]]
        r = r.unflatten(-1, (pairs, 2)) if c["interleaved"] else r.unflatten(-1, (2, pairs)).transpose(-1, -2)
        r = torch.view_as_real(torch.view_as_complex(r.contiguous()) * turn[:, None])
        r = r if c["interleaved"] else r.transpose(-1, -2)
        return torch.cat([r.flatten(-2), x[..., c["rot"]:]], -1)

    def stored(cache, scale, x):
        cache = cache.double()
        if scale is None:
            cache[slot, place] = x
            return cache, None
        scale, amax = scale.double(), x.abs().amax(-1)
        cache[slot, place] = torch.where(amax > 0, E4M3_MAX / amax, 0.0)[..., None] * x
        scale[slot, :, place] = amax / E4M3_MAX
        return cache, scale

    k, ks = stored(s["k_cache"], s["k_scale"], rotated(s["k"]))
    v, vs = stored(s["v_cache"], s["v_scale"], s["v"].double())
    r = {"q": rotated(s["q"]), "k_cache": k, "v_cache": v}
    return r if ks is None else dict(r, k_scale=ks, v_scale=vs)


def _exact_attend(s, c):
    cu, length, G = s["cu"].tolist(), s["len"].tolist(), c["heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for b in range(c["seqs"]):
        n, pages = length[b], s["table"][b, :-(-length[b] // c["page"])].long()

        def lines(cache, scale):
            x = cache[pages] if scale is None else cache.view(torch.uint8)[pages].view(torch.float8_e4m3fn)
            x = x.double() if scale is None else x.double() * scale[pages].double().transpose(1, 2)[..., None]
            return x.flatten(0, 1)[:n].repeat_interleave(G, 1)  # [n][heads][dim]

        k, v = lines(s["k_cache"], s["k_scale"]), lines(s["v_cache"], s["v_scale"])
        for t in range(cu[b], cu[b + 1]):
            last = n - (cu[b + 1] - t)
            first = max(0, last - c["window"] + 1) if c["window"] else 0
            if last < 0:
                continue
            score = (k[first:last + 1] * s["q"][t].double()).sum(-1) / math.sqrt(c["dim"])
            lse[t] = torch.logsumexp(score, 0)
            out[t] = (torch.exp(score - lse[t])[..., None] * v[first:last + 1]).sum(0)
    return {"out": out, "lse": lse}


def _exact_verify(s, c):
    cu, tokens, u, us = s["cu"].tolist(), s["tokens"].tolist(), s["u"].tolist(), s["u_sample"].tolist()
    out, accepted, following = [], [], []
    for b in range(c["seqs"]):
        lo, hi, got = cu[b], cu[b + 1], []
        rows, x = torch.arange(lo, hi - 1, device="cuda"), s["tokens"][lo + 1:hi].long()
        p, q = s["p"][rows, x].tolist(), s["q"][rows, x].tolist()
        while len(got) < hi - lo - 1 and u[lo + len(got)] * q[len(got)] < p[len(got)]:
            got.append(tokens[lo + len(got) + 1])
        a = len(got)
        rest = target = s["p"][lo + a].cpu().numpy().astype(np.float64) if c["dtype"] == "f32" else s["p"][lo + a].double().cpu().numpy()
        if a < hi - lo - 1:
            rest = np.maximum(target - s["q"][lo + a].double().cpu().numpy(), 0)
        mass = np.cumsum(rest if rest.sum() > 0 else target)
        got.append(int(np.searchsorted(mass, us[b] * mass[-1], side="right")))
        out += got + [-1] * (hi - lo - len(got))
        accepted.append(a)
        following.append(int(s["len"][b]) - (hi - lo - 1 - a))
    return {"tokens": np.array(out), "accepted": np.array(accepted), "next": np.array(following)}
