"""Cases, plain forms and 64-bit values of the serving operators around an E4M3 cache with page scales:

  append   rotary positions, and keys and values written into an E4M3 cache with one scale (a power of two) per page and head
  attend   attention of each sequence's new tokens over such a cache
  pages    the pages of a cache forked, freed, allocated and copied on write (step, fork, beams), compacted, or copied
  logits   penalties, biases and grammar masks on logits, temperature and softmax: what the verification of drafts reads

With `own` set, run() calls the framework; otherwise it computes the same in elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
ROPE_BASE = 10000.0
SCALE_EXP = (-110, 119)  # of a page's scale


# ---------------------------------------------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # one user's next token: the latency of the smallest call
        dict(name="append one token", op="append", seqs=1, new_min=1, new=1, past_min=517, past=517, heads=32, kv_heads=8, dim=128,
             page=16, rot=128, interleaved=False, axes=1),
        # drafted tokens of a full serving batch, positions of an image prompt on three axes
        dict(name="append drafts", op="append", seqs=64, new_min=3, new=5, past_min=200, past=9000, heads=32, kv_heads=8, dim=128,
             page=32, rot=96, interleaved=True, axes=3),
        # the prompts of a few users at once (chunked prefill), ragged
        dict(name="append prompts", op="append", seqs=7, new_min=301, new=2041, past_min=0, past=700, heads=32, kv_heads=8, dim=128,
             page=64, rot=128, interleaved=False, axes=1),
        # many short chats, one new token each
        dict(name="attend chats", op="attend", seqs=256, new_min=1, new=1, len_min=1, len=2047, heads=64, kv_heads=8, dim=128, page=32,
             window=0),
        # drafted tokens of widely shared heads: 16 to 40 rows a head group
        dict(name="attend drafts", op="attend", seqs=32, new_min=2, new=5, len_min=100, len=12000, heads=64, kv_heads=8, dim=128, page=64,
             window=0),
        # chunks of prompts behind what is cached of them
        dict(name="attend prompts", op="attend", seqs=4, new_min=200, new=1024, len_min=1500, len=4000, heads=32, kv_heads=8, dim=128,
             page=64, window=0),
        # a serving batch's step: rejected drafts given back, ended chats freed and new prompts let in, a page now and then
        dict(name="pages step", op="pages", kind="step", seqs=128, len=2000, heads=8, dim=128, page=16, cache="bf16"),
        # eight samples of each of 16 prompts
        dict(name="pages fork", op="pages", kind="fork", seqs=128, group=8, len=3001, heads=8, dim=128, page=64, cache="page"),
        # a fragmented cache moved to its low end
        dict(name="pages compact", op="pages", kind="compact", seqs=100, len=1500, pool=16384, heads=8, dim=128, page=16, cache="bf16"),
        # pages of finished prompts kept in a cache of their own, copied back: few and small
        dict(name="pages copy", op="pages", kind="copy", copies=67, pool=600, heads=5, dim=80, page=16, cache="f32"),
        # one user's next token: latency
        dict(name="logits one", op="logits", seqs=1, new_min=1, new=1, vocab=32000, history=700, biases=20, dtype="bf16", out="f32",
             masked=False),
        # a serving batch with drafted tokens, a grammar's masks and long histories
        dict(name="logits batch", op="logits", seqs=64, new_min=1, new=5, vocab=129280, history=3000, biases=100, dtype="f32", out="f32",
             masked=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "pages", "pages", "logits"])
    while True:
        if op == "logits":
            new = rng.choice([1, rng.randint(2, 8)])
            c = dict(op=op, seqs=_log(rng, 1, 256), new_min=rng.randint(1, new), new=new, vocab=_log(rng, 1000, 262144),
                     history=_log(rng, 1, 9000), biases=rng.choice([0, _log(rng, 1, 300)]), dtype=rng.choice(["f32", "bf16"]),
                     out=rng.choice(["f32", "f32", "bf16"]), masked=rng.random() < 0.5)
            if sum(_news(c)) * c["vocab"] <= 2.4e7 and c["seqs"] * c["history"] <= 400000:
                return c
            continue
        dim = rng.choice([64, 80, 96, 112, 128, 128, 128, 192, 256])
        kv, group = rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        page = rng.choice([1, 7, 16, 16, 32, 48, 64, 128])
        if op == "pages":
            kind = rng.choice(["step", "fork", "beams", "compact", "copy"])
            c = dict(op=op, kind=kind, heads=kv, dim=dim, page=page, cache=rng.choice(["bf16", "f32", "e4m3", "page", "page"]))
            if kind == "copy":
                c["copies"] = _log(rng, 1, 3000)
                c["pool"] = c["copies"] + _log(rng, 1, 2000)
                tokens = 2 * c["pool"] * page
            else:
                width = rng.randint(2, 16)
                c.update(seqs=_log(rng, 1, 256), len=_log(rng, 4, 6000))
                if kind in ("fork", "beams"):
                    c.update(seqs=width * max(1, c["seqs"] // width), group=width)
                tokens = c["seqs"] * (c["len"] + page)
                if kind == "compact":
                    c["pool"] = int(tokens / page * rng.uniform(1.1, 2.0)) + 3
                    tokens = c["pool"] * page
            if tokens * kv * dim <= 16384 * 16 * 1024 and tokens / page <= 300000:
                return c
            continue
        c = dict(op=op, heads=kv * group, kv_heads=kv, dim=dim, page=page)
        if op == "append":
            new = _log(rng, 1, 2048)
            c.update(seqs=_log(rng, 1, 256), new_min=rng.randint(1, new), new=new, past_min=0, past=_log(rng, 1, 9000),
                     rot=2 * rng.randint(3, dim // 2), interleaved=rng.random() < 0.5, axes=rng.choice([1, 1, 3]))
            rows, slots = sum(_news(c)), sum(_news(c)) + c["seqs"] * (c["past"] / 2 + c["page"])
            if rows * (c["heads"] + 2 * kv) * dim <= 9000 * 48 * 128 and slots * kv * dim <= 1.5e8 and slots <= 600000:
                return c
        else:
            new, length = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 1024)]), _log(rng, 16, 60000)
            c.update(seqs=_log(rng, 1, 256), new_min=rng.randint(1, new), new=new, len_min=rng.randint(1, length), len=length,
                     window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]))
            if c["seqs"] * length * kv * dim <= 64 * 8190 * 8 * 128 and c["seqs"] * length * c["heads"] * new <= 5e8 and c["seqs"] * length <= 2e6:
                return c


# ---------------------------------------------------------------------------------------------------------------------------------
# inputs

def _spread(lo, hi, n):
    """n lengths from lo to hi, evenly."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]


def _news(c):
    return _spread(c["new_min"], c["new"], c["seqs"])


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_F8 = torch.float8_e4m3fn


def _int(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


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
    return table, pool


def _scale_of(amax):
    """The least power of two that holds amax in E4M3, in the range of scales."""
    m, e = torch.frexp(amax / 512.0)  # amax = m 2^e 512 with m in [0.5, 1); 448 = 0.875 * 512
    e = torch.where(amax > 0, e + (m > 0.875).to(e.dtype), SCALE_EXP[0]).clamp(*SCALE_EXP)
    return (e.int() + 127 << 23).view(torch.float32)


def _cache(g, shape, kind):
    """Keys or values [pages][tokens][heads][dim] as a cache of that kind holds them, and their scales."""
    if kind in _TYPES:
        return torch.empty(shape, dtype=_TYPES[kind], device="cuda").normal_(generator=g), None
    codes = torch.empty(shape, dtype=_F8, device="cuda")
    scale = torch.empty((shape[0], shape[2]) if kind == "page" else (shape[0], shape[2], shape[1]), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (shape[1] * shape[2] * shape[3]))
    for i in range(0, shape[0], step):
        x = torch.empty((min(step, shape[0] - i),) + shape[1:], dtype=torch.float32, device="cuda").normal_(generator=g)
        # some stretches of text have larger keys than others
        x *= torch.empty((x.shape[0], 1, shape[2], 1), device="cuda").uniform_(-2, 2, generator=g).exp2_()
        if kind == "page":
            scale[i:i + step] = _scale_of(x.abs().amax((1, 3)))
            codes[i:i + step] = (x / scale[i:i + step, None, :, None]).to(_F8)
        else:
            amax = x.abs().amax(-1)
            codes[i:i + step] = (x * (E4M3_MAX / amax)[..., None]).to(_F8)
            scale[i:i + step] = (amax / E4M3_MAX).transpose(1, 2)
    return codes, scale


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "pages":
        (_prepare_copy if case["kind"] == "copy" else _prepare_pages)(s, case, rs, g)
        return s
    new = np.array(_news(case), np.int64)[rs.permutation(case["seqs"])]
    cu = np.concatenate([[0], np.cumsum(new)])
    s["T"], s["cu"] = int(cu[-1]), _int(cu)
    {"append": _prepare_append, "attend": _prepare_attend, "logits": _prepare_logits}[case["op"]](s, case, rs, g, new)
    return s


def _attn_handle(s, c, **more):
    import sparse_mixture_experts_router_gb300 as moe
    s["cfg"] = moe.attn_config(n_seqs=c["seqs"], n_tokens=s["T"], max_new=c["new"], n_heads=c["heads"], n_kv_heads=c["kv_heads"],
                               head_dim=c["dim"], page_size=c["page"], n_pages=s["pool"], max_pages=s["table"].shape[1],
                               dtype=moe.MOE_BF16, cache_dtype=moe.MOE_E4M3_PAGE, **more)


def _prepare_cache(s, c, rs, g, lengths):
    s["len"] = _int(lengths)
    table, s["pool"] = _table(rs, lengths, c["page"])
    s["table"] = _int(table)
    shape = (s["pool"], c["page"], c["kv_heads"], c["dim"])
    s["k_cache"], s["k_scale"] = _cache(g, shape, "page")
    s["v_cache"], s["v_scale"] = _cache(g, shape, "page")


def _prepare_append(s, c, rs, g, new):
    T, D = s["T"], c["dim"]
    _prepare_cache(s, c, rs, g, new + np.array(_spread(c["past_min"], c["past"], c["seqs"]))[rs.permutation(c["seqs"])])
    wide = (c["heads"] + 2 * c["kv_heads"]) * D
    qkv = torch.empty((T, wide), dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # the output of one projection
    s["q"], s["k"], s["v"] = (t.unflatten(1, (-1, D)) for t in qkv.split([c["heads"] * D, c["kv_heads"] * D, c["kv_heads"] * D], 1))
    # one axis: a token's place in its sequence; three: time, height and width of image patches behind a long text
    s["pos"] = _int(rs.randint(0, 1 << 17, (3, T))) if c["axes"] == 3 else None
    s["sections"] = _sections(c)
    s["q_out"] = torch.empty((T, c["heads"], D), dtype=torch.bfloat16, device="cuda")
    if own:
        import sparse_mixture_experts_router_gb300 as moe
        _attn_handle(s, c, rot_dim=c["rot"], rot_interleaved=c["interleaved"], rot_sections=s["sections"], rope_base=ROPE_BASE,
                     q_stride=wide, k_stride=wide, v_stride=wide)
        s["ws"] = moe.workspace(s["cfg"], "append")


def _sections(c):
    pairs = c["rot"] // 2
    return [pairs - 2 * (pairs // 3), pairs // 3, pairs // 3] if c["axes"] == 3 else [pairs, 0, 0]


def _prepare_attend(s, c, rs, g, new):
    _prepare_cache(s, c, rs, g, np.array(_spread(c["len_min"], c["len"], c["seqs"]))[rs.permutation(c["seqs"])])
    s["q"] = torch.empty((s["T"], c["heads"], c["dim"]), dtype=torch.float32, device="cuda").normal_(generator=g).bfloat16()
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((s["T"], c["heads"]), dtype=torch.float32, device="cuda")
    if own:
        import sparse_mixture_experts_router_gb300 as moe
        _attn_handle(s, c, window=c["window"])
        s["ws"] = moe.workspace(s["cfg"], "attention")


def _pages_handle(s, c):
    import sparse_mixture_experts_router_gb300 as moe
    kind = {"bf16": moe.MOE_BF16, "f32": moe.MOE_F32, "e4m3": moe.MOE_E4M3, "page": moe.MOE_E4M3_PAGE}[c["cache"]]
    s["cfg"] = moe.attn_config(n_seqs=c.get("seqs", 1), n_tokens=0, n_heads=c["heads"], n_kv_heads=c["heads"], head_dim=c["dim"],
                               page_size=c["page"], n_pages=s["pool"], max_pages=s["table"].shape[1] if "table" in s else 1,
                               dtype=moe.MOE_F32 if c["cache"] == "f32" else moe.MOE_BF16, cache_dtype=kind)
    s["ws"] = moe.workspace(s["cfg"], "pages")


def _prepare_copy(s, c, rs, g):
    s["pool"], shape = c["pool"], (c["pool"], c["page"], c["heads"], c["dim"])
    for name in ("k", "v"):
        s[name + "_cache"], s[name + "_scale"] = _cache(g, shape, c["cache"])
        s[name + "_src"], s[name + "_src_scale"] = _cache(g, shape, c["cache"])
    s["src"], s["dst"] = _int(rs.randint(0, s["pool"], c["copies"])), _int(rs.permutation(s["pool"])[:c["copies"]])
    if own:
        _pages_handle(s, c)


def _prepare_pages(s, c, rs, g):
    """Sequences over a pool, with their tables and the pages' counts, and what is to become of them."""
    B, ps, kind, L = c["seqs"], c["page"], c["kind"], c["len"]
    G = c.get("group", 1)
    lengths = np.array(_spread(max(1, L // 4), L, B))[rs.permutation(B)]
    parent = np.arange(B)
    if kind == "fork":  # the first of each group has the prompt
        lengths[np.arange(B) % G != 0] = 0
        parent = parent // G * G
        kept = lengths[parent]
        need = kept + 1
    elif kind == "beams":  # the beams of a group are as long as each other; the best go on, some more than once
        lengths = lengths[parent // G * G]
        parent = parent // G * G + rs.randint(0, G, B)
        kept = lengths[parent]
        need = kept + 1
    elif kind == "step":
        kept = np.maximum(lengths - rs.randint(0, 4, B), 0)  # rejected drafts
        need = kept + rs.randint(1, 5, B)
        ended = rs.rand(B) < 0.05
        kept[ended] = 0
        need[ended] = np.where(rs.rand(B) < 0.5, 0, rs.randint(1, L + 1, B))[ended]  # a new prompt in its place, or none
    pages = -(-lengths // ps)
    wide = -(-(2 * L + 8) // ps)
    table, at = np.full((B, wide), -1, np.int64), 0
    for b in range(B):
        first = b // G * G
        shared = pages[b] * 3 // 4 if kind == "beams" and b != first else 0  # what the beams have in common
        table[b, :shared] = table[first, :shared]
        table[b, shared:pages[b]] = np.arange(at, at + pages[b] - shared)
        at += pages[b] - shared
    s["pool"] = c["pool"] if kind == "compact" else int(sum(-(-n // ps) + 1 for n in _spread(max(1, L // 4), L, B)) * 1.1) + 2 * B + 3
    order = rs.permutation(s["pool"])
    table = np.where(table >= 0, order[table], -1)
    s["table"], s["len"] = _int(table), _int(lengths)
    s["refs"] = _int(np.bincount(table[table >= 0], minlength=s["pool"]))
    shape = (s["pool"], ps, c["heads"], c["dim"])
    s["k_cache"], s["k_scale"] = _cache(g, shape, c["cache"])
    s["v_cache"], s["v_scale"] = _cache(g, shape, c["cache"])
    s["table_out"], s["refs_out"] = torch.full_like(s["table"], -1), torch.empty_like(s["refs"])
    if kind == "compact":
        s["map"], s["live"] = torch.empty_like(s["refs"]), torch.empty(1, dtype=torch.int32, device="cuda")
    else:
        s["parent"] = None if kind == "step" else _int(parent)
        s["kept"], s["need"], s["granted"] = _int(kept), _int(need), torch.empty(B, dtype=torch.int32, device="cuda")
    if own:
        _pages_handle(s, c)


def _prepare_logits(s, c, rs, g, new):
    T, V, B = s["T"], c["vocab"], c["seqs"]
    s["logits"] = torch.empty((T, V), dtype=torch.float32, device="cuda").normal_(0, 3, generator=g).to(_TYPES[c["dtype"]])
    often = 1 / (np.arange(V) + 3.0)  # words are used unevenly
    often = np.cumsum(often / often.sum())
    words = rs.permutation(V)

    def text(n):
        return words[np.minimum(np.searchsorted(often, rs.rand(n)), V - 1)]

    lengths = np.array(_spread(c["history"] // 3, c["history"], B))[rs.permutation(B)]
    s["tokens"], s["history"] = _int(text(T)), _int(text(int(lengths.sum())))
    s["cu_history"], s["n_prompt"] = _int(np.concatenate([[0], np.cumsum(lengths)])), _int(lengths // 2)
    few = min(c["biases"], V)
    s["bias_token"] = _int(np.concatenate([np.sort(rs.choice(V, few, replace=False)) for _ in range(B)]))
    s["bias"] = torch.empty(B * few, device="cuda").normal_(0, 2, generator=g)
    s["cu_bias"] = _int(np.arange(B + 1) * few)
    f = lambda x: torch.from_numpy(np.asarray(x, np.float32)).cuda()  # noqa: E731
    s["repetition"], s["frequency"], s["presence"] = f(rs.uniform(0.9, 1.4, B)), f(rs.uniform(-0.2, 0.8, B)), f(rs.uniform(-0.2, 0.8, B))
    s["temperature"] = f(np.where(rs.rand(B) < 0.15, 0.0, rs.uniform(0.3, 1.5, B)))  # 0: the most likely token
    s["mask"] = s["mask_row"] = None
    if c["masked"]:  # a grammar allows a few tokens in one state, most of them in another; some rows have none
        masks = max(1, T // 2)
        share = torch.from_numpy(rs.choice([0.001, 0.05, 0.9], masks)).cuda()[:, None, None]
        allowed = torch.empty((masks, -(-V // 32), 32), device="cuda").uniform_(generator=g) < share
        bits = (allowed.long() << torch.arange(32, device="cuda")).sum(-1)
        s["mask"] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).int()
        s["mask_row"] = _int(rs.randint(-1, masks, T))
    s["p"] = torch.empty((T, V), dtype=_TYPES[c["out"]], device="cuda")
    if own:
        import sparse_mixture_experts_router_gb300 as moe
        kind = {"bf16": moe.MOE_BF16, "f32": moe.MOE_F32}
        s["cfg"] = moe.logits_config(n_seqs=B, n_tokens=T, max_new=c["new"], vocab=V, dtype=kind[c["dtype"]], out_dtype=kind[c["out"]],
                                     n_history=s["history"].numel(), n_bias=B * few, n_masks=0 if s["mask"] is None else s["mask"].shape[0])
        s["ws"] = moe.workspace(s["cfg"], "logits")


# ---------------------------------------------------------------------------------------------------------------------------------
# one pass

def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import sparse_mixture_experts_router_gb300 as moe
        caches = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]) if "k_cache" in s else ()
        if op == "append":
            moe.moe_rope_append(s["cfg"], s["q"], s["k"], s["v"], s["pos"], s["cu"], s["len"], s["table"], s["q_out"], *caches, s["ws"])
        elif op == "attend":
            moe.moe_paged_attention(s["cfg"], s["q"], s["cu"], s["len"], s["table"], *caches, s["out"], s["lse"], s["ws"])
            return {"out": s["out"], "lse": s["lse"]}
        elif op == "logits":
            moe.moe_logits_probs(s["cfg"], s["logits"], s["cu"], s["tokens"], s["history"], s["cu_history"], s["n_prompt"], s["repetition"],
                                 s["presence"], s["frequency"], s["bias_token"], s["bias"], s["cu_bias"], s["mask"], s["mask_row"],
                                 s["temperature"], s["p"], s["ws"])
            return {"p": s["p"]}
        elif c["kind"] == "copy":
            moe.moe_pages_copy(s["cfg"], s["src"], s["dst"], s["pool"], s["k_src"], s["v_src"], s["k_src_scale"], s["v_src_scale"], *caches,
                               s["ws"])
        elif c["kind"] == "compact":
            moe.moe_pages_compact(s["cfg"], s["len"], s["table"], s["refs"], s["table_out"], s["refs_out"], s["map"], s["live"], *caches, s["ws"])
        else:
            moe.moe_pages_update(s["cfg"], s["parent"], s["len"], s["kept"], s["need"], s["table"], s["refs"], s["table_out"], s["refs_out"],
                                 s["granted"], *caches, s["ws"])
    elif op == "append":
        s["q_out"] = _plain_append(s)
    elif op == "pages":
        {"copy": _plain_copy, "compact": _plain_compact}.get(c["kind"], _plain_update)(s)
    else:
        return (_plain_attend if op == "attend" else _plain_logits)(s)
    return {k: s[k] for k in ("q_out", "k_cache", "v_cache", "k_scale", "v_scale", "table_out", "refs_out", "granted", "map", "live")
            if s.get(k) is not None}


def _rows(s):
    """Each new token's sequence and its place among that sequence's new tokens."""
    t = torch.arange(s["T"], device="cuda")
    cu = s["cu"].long()
    b = torch.searchsorted(cu[1:], t, right=True)
    return b, t - cu[b], (cu[1:] - cu[:-1])


def _plain_append(s):
    c = s["case"]
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

    # each new token's page among those that this call writes; the pages' first new places
    starts = (j == 0) | (place == 0)
    which = torch.cumsum(starts.long(), 0) - 1
    pages = torch.zeros(s["T"], dtype=torch.long, device="cuda").index_copy_(0, which, slot)
    first = torch.full((s["T"],), c["page"], device="cuda").scatter_reduce_(0, which, place, "amin")
    used = torch.arange(s["T"], device="cuda") <= which[-1]
    pages = torch.where(used, pages, slot[0])  # what is left over repeats the first page
    first = torch.where(used, first, first[0])
    older = torch.arange(c["page"], device="cuda") < first[:, None]

    def store(cache, scale, x):
        amax = torch.zeros((s["T"], c["kv_heads"]), device="cuda").scatter_reduce_(
            0, which[:, None].expand(-1, c["kv_heads"]), x.abs().amax(-1), "amax")
        now, was = _scale_of(torch.where(used[:, None], amax, amax[:1])), scale[pages]
        now = torch.where((first > 0)[:, None], torch.maximum(now, was), now)
        step = max(1, (1 << 26) // (c["page"] * c["kv_heads"] * c["dim"]))
        for k in range(0, s["T"], step):  # the older codes of the pages whose scale has grown
            p, ratio = pages[k:k + step], (was / now)[k:k + step]
            codes = cache[p]
            grown = (older[k:k + step, :, None] & ((used[k:k + step, None] | (k == 0)) & (ratio != 1))[:, None])[..., None]
            codes = torch.where(grown, (codes.float() * ratio[:, None, :, None]).to(_F8).float(), codes.float()).to(_F8)
            cache.view(torch.uint8)[p] = codes.view(torch.uint8)
        scale[pages] = now
        cache.view(torch.uint8)[slot, place] = (x / now[which][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(_F8).view(torch.uint8)

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
        return cache.view(torch.uint8)[page, place].view(_F8).float() * scale[page][..., None]

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
    w = score.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    v = gather(s["v_cache"], s["v_scale"])
    v.masked_fill_((at >= length[:, None])[..., None, None], 0.0)
    o = torch.matmul(w.view(B, K, N * G, L), v.permute(0, 2, 1, 3)).view(B, K, N, G, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(B, N, H, D)
    lse = (top + total.log()).squeeze(-1).permute(0, 2, 1, 3).reshape(B, N, H)
    b, j, _ = _rows(s)
    return {"out": o[b, j].to(s["q"].dtype), "lse": lse[b, j]}


def _caches(s, to=("k_cache", "v_cache", "k_scale", "v_scale"), of=None):
    """Pairs of a cache's tensors, first index the page, as bytes where they are codes."""
    for a, b in zip(to, of or to):
        if s[a] is not None:
            x, y = s[a], s[b]
            yield (x.view(torch.uint8), y.view(torch.uint8)) if x.dtype == _F8 else (x, y)


def _plain_copy(s):
    for to, of in _caches(s, of=("k_src", "v_src", "k_src_scale", "v_src_scale")):
        to[s["dst"].long()] = of[s["src"].long()]


def _count(table, used, n_pages):
    """References to each page from the entries of a table that are in use."""
    at = torch.where(used, table, n_pages).flatten()
    return torch.zeros(n_pages + 1, dtype=torch.long, device="cuda").scatter_add_(0, at, torch.ones_like(at))[:n_pages]


def _ranked(chosen, n):
    """The indexes where `chosen` holds, ascending, in a list of n (the rest of it 0)."""
    at = torch.where(chosen, torch.cumsum(chosen.long(), 0) - 1, n).clamp(max=n)
    return torch.zeros(n + 1, dtype=torch.long, device="cuda").scatter_(0, at, torch.arange(chosen.numel(), device="cuda"))[:n]


def _plain_update(s):
    c, ps, n = s["case"], s["case"]["page"], s["pool"]
    table, length, kept, need = s["table"].long(), s["len"].long(), s["kept"].long(), s["need"].long()
    B, wide = table.shape
    parent = torch.arange(B, device="cuda") if s["parent"] is None else s["parent"].long()
    i = torch.arange(wide, device="cuda")
    pages = lambda t: (t + ps - 1) // ps  # noqa: E731
    new = table[parent]
    refs = s["refs"].long() - _count(table, i < pages(length)[:, None], n) + _count(new, i < pages(kept)[:, None], n)
    last = new.gather(1, (pages(kept) - 1).clamp(min=0)[:, None])[:, 0].clamp(min=0)
    cow = (need > kept) & (kept % ps > 0) & (refs[last] > 1)
    want = pages(need) - pages(kept) + cow
    upto = torch.cumsum(want, 0)
    free = _ranked(refs == 0, n)
    served = upto <= (refs == 0).sum()
    cow &= served
    begin = torch.where(cow, pages(kept) - 1, pages(kept))  # the first entry that is a new page
    fresh = (i >= begin[:, None]) & (i < pages(need)[:, None]) & served[:, None]
    rank = ((upto - want)[:, None] + i - begin[:, None]).clamp(0, n - 1)
    entry = torch.where(fresh, free[rank], new)
    valid = fresh | (i < pages(kept)[:, None])
    s["table_out"].copy_(torch.where(valid, entry, s["table_out"].long()))
    refs = refs + _count(entry, fresh, n) - _count(last[:, None], cow[:, None], n)
    s["refs_out"].copy_(refs)
    s["granted"].copy_(torch.where(served, need, kept))
    # the kept tokens of the pages that were shared; a row without one copies a page of its own to itself
    dst = entry.gather(1, (pages(kept) - 1).clamp(min=0)[:, None])[:, 0]
    some = torch.where(valid[:, 0], entry[:, 0], entry[valid[:, 0].int().argmax(), 0]).clamp(min=0)
    src, dst = torch.where(cow, last, some), torch.where(cow, dst, some)
    for x, _ in _caches(s):
        if x.dim() == 4:
            live = (torch.arange(ps, device="cuda") < (kept % ps)[:, None])[..., None, None]
        elif x.dim() == 3:
            live = (torch.arange(ps, device="cuda") < (kept % ps)[:, None])[:, None]
        else:
            live = torch.ones((B, 1), dtype=torch.bool, device="cuda")
        x[dst] = torch.where(live, x[src], x[dst])


def _plain_compact(s):
    c, ps, n = s["case"], s["case"]["page"], s["pool"]
    refs = s["refs"].long()
    live = refs > 0
    many = live.sum()
    page = torch.arange(n, device="cuda")
    hole, high = ~live & (page < many), live & (page >= many)
    holes, highs = _ranked(hole, n), _ranked(high, n)
    there = torch.where(high, holes[(torch.cumsum(high.long(), 0) - 1).clamp(min=0)], page)
    s["map"].copy_(torch.where(live, there, -1))
    came = torch.where(hole, highs[(torch.cumsum(hole.long(), 0) - 1).clamp(min=0)], page)  # the page whose tokens come here
    s["refs_out"].copy_(torch.where(page < many, refs[came], 0))
    s["live"].copy_(many)
    used = torch.arange(s["table"].shape[1], device="cuda") < ((s["len"].long() + ps - 1) // ps)[:, None]
    s["table_out"].copy_(torch.where(used, there[s["table"].long().clamp(min=0)], s["table_out"].long()))
    for x, _ in _caches(s):
        x.copy_(x[came])


def _plain_logits(s):
    c, V = s["case"], s["case"]["vocab"]
    b, j, new = _rows(s)
    x = s["logits"].float()
    # how often each token was generated, and whether it has occurred at all
    cu, h = s["cu_history"].long(), s["history"].long()
    hb = torch.searchsorted(cu[1:], torch.arange(h.numel(), device="cuda"), right=True)
    made = torch.arange(h.numel(), device="cuda") - cu[hb] >= s["n_prompt"].long()[hb]
    count = torch.zeros((c["seqs"], V), dtype=torch.int32, device="cuda").index_put_((hb, h), made.int(), accumulate=True)
    seen = torch.zeros((c["seqs"], V), dtype=torch.int32, device="cuda").index_put_((hb, h), torch.ones_like(made, dtype=torch.int32), accumulate=True)
    count, seen = count[b], seen[b]
    for k in range(c["new"]):  # the new tokens up to the row's own
        row, fed = torch.arange(s["T"], device="cuda"), s["tokens"].long()[(s["cu"].long()[b] + k).clamp(max=s["T"] - 1)]
        one = (k <= j).int()
        count.index_put_((row, fed), one, accumulate=True)
        seen.index_put_((row, fed), one, accumulate=True)
    rep, f, pr = (s[k][b][:, None] for k in ("repetition", "frequency", "presence"))
    x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - f * count.float()
    x = torch.where(count > 0, x - pr, x)
    few = c["biases"]
    if few:
        few = s["bias"].numel() // c["seqs"]
        token, value = s["bias_token"].long().view(-1, few)[b], s["bias"].view(-1, few)[b]
        x = x.scatter_add(1, token, value)
    if s["mask"] is not None:
        v = torch.arange(V, device="cuda")
        bit = (s["mask"][s["mask_row"].long().clamp(min=0)][:, v // 32] >> (v % 32).int()) & 1
        x = torch.where((bit > 0) | (s["mask_row"] < 0)[:, None], x, -math.inf)
    t = s["temperature"][b][:, None]
    top = x.amax(1, keepdim=True)
    some = top > -math.inf
    w = torch.exp((x - torch.where(some, top, 0.0)) / torch.where(t > 0, t, 1.0))
    p = torch.where(some, w / w.sum(1, keepdim=True), 0.0)
    best = torch.zeros_like(p).scatter_(1, (x == top).to(torch.int8).argmax(1, keepdim=True), some.float())
    return {"p": torch.where(t > 0, p, best).to(_TYPES[c["out"]])}


# ---------------------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "pages":
        size = {"bf16": 2, "f32": 4, "e4m3": 1, "page": 1}[c["cache"]]
        token = 2 * c["heads"] * (c["dim"] * size + (4 if c["cache"] == "e4m3" else 0))
        page = c["page"] * token + (8 * c["heads"] if c["cache"] == "page" else 0)
        if c["kind"] == "copy":
            return {"bytes": c["copies"] * (2 * page + 8), "flops": 0.0}
        lengths = _spread(max(1, c["len"] // 4), c["len"], c["seqs"])
        entries = sum(-(-n // c["page"]) for n in lengths)
        if c["kind"] == "compact":  # the live pages above the live pages' number
            moved = entries * (1 - entries / c["pool"])
            return {"bytes": moved * 2 * page + 8 * entries + 12 * c["pool"], "flops": 0.0}
        pool = int((entries + c["seqs"]) * 1.1) + 2 * c["seqs"] + 3
        copied = 0 if c["kind"] == "step" else c["seqs"] * (c["page"] - 1) / 2 * token
        return {"bytes": 2 * copied + 8 * entries + 8 * pool + 20 * c["seqs"], "flops": 0.0}
    T = sum(_news(c))
    if c["op"] == "logits":
        size = (2 if c["dtype"] == "bf16" else 4) + (2 if c["out"] == "bf16" else 4)
        masks = max(1, T // 2) * c["vocab"] / 8 if c["masked"] else 0
        return {"bytes": T * c["vocab"] * size + masks + 4 * sum(_spread(c["history"] // 3, c["history"], c["seqs"])) + c["seqs"] * 8 * c["biases"],
                "flops": 6.0 * T * c["vocab"]}
    line = c["dim"]  # a key or a value as the cache holds it
    if c["op"] == "append":
        read = T * (c["heads"] + 2 * c["kv_heads"]) * c["dim"] * 2
        return {"bytes": read + T * (c["heads"] * c["dim"] * 2 + 2 * c["kv_heads"] * line) + T * (12 if c["axes"] == 3 else 4),
                "flops": 3.0 * T * (c["heads"] + c["kv_heads"]) * c["rot"]}
    lengths, news = _spread(c["len_min"], c["len"], c["seqs"]), _news(c)
    # the places of lengths and new tokens are drawn apart: the mean sequence's pairs
    n, m = sum(lengths) / c["seqs"], T / c["seqs"]
    seen = max(1.0, n - m / 2) if n > m else n * n / 2 / m
    keys = n
    if c["window"]:
        seen, keys = min(seen, c["window"]), min(keys, c["window"] + m - 1)
    return {"bytes": c["seqs"] * keys * c["kv_heads"] * 2 * (line + 4 / c["page"]) + T * c["heads"] * (4 * c["dim"] + 4) + c["seqs"] * keys / c["page"] * 4,
            "flops": 4.0 * T * seen * c["heads"] * c["dim"]}


# ---------------------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "pages":
        return {"copy": _exact_copy, "compact": _exact_compact}.get(case["kind"], _exact_update)(s, case)
    return {"append": _exact_append, "attend": _exact_attend, "logits": _exact_logits}[case["op"]](s, case)


def _exact_append(s, c):
    cu, length, table, ps = s["cu"].tolist(), s["len"].tolist(), s["table"].cpu().numpy(), c["page"]
    at = np.concatenate([np.arange(n - (e - b), n) for b, e, n in zip(cu, cu[1:], length)])
    seq = np.repeat(np.arange(c["seqs"]), np.diff(cu))
    slot, place = table[seq, at // ps].astype(np.int64), at % ps
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

    rows = {}  # of each page that is written
    for t, p in enumerate(slot):
        rows.setdefault(int(p), []).append(t)

    def stored(cache, scale, x):
        cache, scale = cache.double(), scale.double()
        amax, new = x.abs().amax(-1).cpu().numpy(), scale.cpu().numpy()
        old = new.copy()
        for p, ts in rows.items():
            fit = np.exp2(np.clip(np.ceil(np.log2(amax[ts].max(0) / E4M3_MAX)), *SCALE_EXP))
            new[p] = fit if place[ts[0]] == 0 else np.maximum(fit, old[p])
        new, old = torch.from_numpy(new).cuda(), torch.from_numpy(old).cuda()
        pages = torch.tensor(sorted(rows), device="cuda")
        before = torch.tensor([place[rows[p][0]] for p in sorted(rows)], device="cuda")
        ratio = torch.where((torch.arange(ps, device="cuda") < before[:, None])[..., None], (old / new)[pages][:, None], 1.0)
        cache[pages] *= ratio[..., None]
        at = torch.from_numpy(slot).cuda()
        cache[at, torch.from_numpy(place).cuda()] = x / new[at][..., None]
        return cache, new

    k, ks = stored(s["k_cache"], s["k_scale"], rotated(s["k"]))
    v, vs = stored(s["v_cache"], s["v_scale"], s["v"].double())
    return {"q_out": rotated(s["q"]), "k_cache": k, "v_cache": v, "k_scale": ks, "v_scale": vs}


def _exact_attend(s, c):
    cu, length, G = s["cu"].tolist(), s["len"].tolist(), c["heads"] // c["kv_heads"]
    if sum((e - b) * n for b, e, n in zip(cu, cu[1:], length)) * c["heads"] * c["dim"] > 2e11:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for b in range(c["seqs"]):
        n, new, pages = length[b], cu[b + 1] - cu[b], s["table"][b, :-(-length[b] // c["page"])].long()

        def lines(cache, scale):
            x = cache.view(torch.uint8)[pages].view(_F8).double() * scale[pages].double()[:, None, :, None]
            return x.flatten(0, 1)[:n].transpose(0, 1)  # [head][n][dim]

        k, v = lines(s["k_cache"], s["k_scale"]), lines(s["v_cache"], s["v_scale"])
        last = n - new + torch.arange(new, device="cuda")[:, None]
        key = torch.arange(n, device="cuda")
        hide = (key > last) | (key <= last - c["window"] if c["window"] else torch.zeros_like(key > last))
        for h in range(c["kv_heads"]):
            mine = slice(h * G, (h + 1) * G)
            q = s["q"][cu[b]:cu[b + 1], mine].double().transpose(0, 1)  # [of the group][new][dim]
            score = (q @ k[h].T / math.sqrt(c["dim"])).masked_fill(hide, -math.inf)
            z = torch.logsumexp(score, 2)
            lse[cu[b]:cu[b + 1], mine] = z.T
            weight = torch.exp(score - z.clamp(min=-1e300)[..., None])
            out[cu[b]:cu[b + 1], mine] = (weight @ v[h]).transpose(0, 1)
    return {"out": out, "lse": lse}


def _moved(s, pairs, tokens=None):
    """The caches after copies of pages (from, to), each of its first tokens."""
    r = {}
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        if s[name] is None:
            continue
        x, kind = s[name], s[name].dtype
        x = (x.view(torch.uint8) if kind == _F8 else x).clone()
        for i, (a, b) in enumerate(pairs):
            n = x.shape[1] if tokens is None else tokens[i]
            if x.dim() == 4:
                x[b, :n] = x[a, :n]
            elif x.dim() == 3:
                x[b, :, :n if tokens else None] = x[a, :, :n if tokens else None]
            else:
                x[b] = x[a]
        r[name] = x.view(kind)
    return r


def _exact_copy(s, c):
    r = {}
    for name in ("k", "v"):
        for part in ("_cache", "_scale"):
            x, y = s[name + part], s[name + ("_src" if part == "_cache" else "_src_scale")]
            if x is None:
                continue
            kind = x.dtype
            x, y = (t.view(torch.uint8) if kind == _F8 else t for t in (x.clone(), y))
            for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
                x[b] = y[a]
            r[name + part] = x.view(kind)
    return r


def _exact_update(s, c):
    ps, table, refs = c["page"], s["table"].tolist(), s["refs"].tolist()
    length, kept, need = s["len"].tolist(), s["kept"].tolist(), s["need"].tolist()
    B = len(length)
    parent = list(range(B)) if s["parent"] is None else s["parent"].tolist()
    pages = lambda n: -(-n // ps)  # noqa: E731
    mine = [table[p][:pages(n)] for p, n in zip(parent, kept)]
    for b in range(B):
        for p in mine[b]:
            refs[p] += 1
        for p in table[b][:pages(length[b])]:
            refs[p] -= 1
    free = [p for p, n in enumerate(refs) if n == 0]
    out, granted, dropped, copies, tokens, taken, full = s["table_out"].tolist(), [], [], [], [], 0, False
    counts = list(refs)
    for b in range(B):
        row = mine[b]
        writes = need[b] > kept[b] and kept[b] % ps > 0 and refs[row[-1]] > 1
        want = pages(need[b]) - len(row) + writes
        full = full or taken + want > len(free)
        granted.append(kept[b] if full else need[b])
        if not full:
            got = free[taken:taken + want]
            taken += want
            for p in got:
                counts[p] = 1
            if writes:
                copies.append((row[-1], got[0]))
                tokens.append(kept[b] % ps)
                dropped.append(row[-1])
                row = row[:-1]
            row = row + got
        out[b][:len(row)] = row
    for p in dropped:
        counts[p] -= 1
    return dict(_moved(s, copies, tokens), table_out=np.array(out), refs_out=np.array(counts), granted=np.array(granted))


def _exact_compact(s, c):
    refs, ps = s["refs"].tolist(), c["page"]
    live = [p for p, n in enumerate(refs) if n]
    holes = [p for p in range(len(live)) if refs[p] == 0]
    there = {p: p for p in live}
    moves = list(zip([p for p in live if p >= len(live)], holes))
    there.update(moves)
    out, table = s["table_out"].tolist(), s["table"].tolist()
    for b, n in enumerate(s["len"].tolist()):
        for i in range(-(-n // ps)):
            out[b][i] = there[table[b][i]]
    counts = [0] * len(refs)
    for p, q in there.items():
        counts[q] = refs[p]
    return dict(_moved(s, moves), table_out=np.array(out), refs_out=np.array(counts), map=np.array([there.get(p, -1) for p in range(len(refs))]),
                live=np.array([len(live)]))


def _exact_logits(s, c):
    cu, V, T = s["cu"].tolist(), c["vocab"], s["T"]
    if T * V > 5e7:
        return None
    p = torch.zeros((T, V), dtype=torch.float64, device="cuda")
    history, begin, prompt = s["history"].cpu().numpy(), s["cu_history"].tolist(), s["n_prompt"].tolist()
    tokens, few = s["tokens"].cpu().numpy(), s["bias"].numel() // c["seqs"]
    for b in range(c["seqs"]):
        words = history[begin[b]:begin[b + 1]]
        value = {k: float(s[k][b]) for k in ("repetition", "frequency", "presence", "temperature")}
        for t in range(cu[b], cu[b + 1]):
            fed = tokens[cu[b]:t + 1]
            count = np.bincount(np.concatenate([words[prompt[b]:], fed]), minlength=V)
            seen = np.bincount(np.concatenate([words, fed]), minlength=V) > 0
            count, seen = torch.from_numpy(count).cuda(), torch.from_numpy(seen).cuda()
            x = s["logits"][t].double()
            x[seen] *= torch.where(x[seen] > 0, 1 / value["repetition"], value["repetition"])
            x -= value["frequency"] * count
            x[count > 0] -= value["presence"]
            x[s["bias_token"][b * few:(b + 1) * few].long()] += s["bias"][b * few:(b + 1) * few].double()
            if s["mask"] is not None and int(s["mask_row"][t]) >= 0:
                words_of = s["mask"][int(s["mask_row"][t])].cpu().numpy().view(np.uint32)
                bits = np.unpackbits(words_of.view(np.uint8), bitorder="little")[:V]
                x[torch.from_numpy(bits == 0).cuda()] = -math.inf
            if not bool((x > -math.inf).any()):
                continue
            if value["temperature"] == 0:
                p[t, int(torch.nonzero(x == x.max())[0])] = 1
            else:
                p[t] = torch.softmax(x / value["temperature"], 0)
    return {"p": p}
