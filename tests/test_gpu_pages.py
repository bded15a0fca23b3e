"""Pages of a cache: forked, trimmed, freed, given, copied on write (update), moved to the low end
(compact) and copied, against plain Python lists. Everything is exact."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_router_gb300 as moe

pytestmark = pytest.mark.gpu
KINDS = {"f32": (moe.MOE_F32, moe.MOE_F32, torch.float32), "bf16": (moe.MOE_BF16, moe.MOE_BF16, torch.bfloat16),
         "e4m3": (moe.MOE_BF16, moe.MOE_E4M3, torch.uint8), "page": (moe.MOE_BF16, moe.MOE_E4M3_PAGE, torch.uint8)}


def dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


class Pool:
    """Caches of random bits, in either order, and their configuration."""

    def __init__(self, n_pages, page, heads=2, dim=32, kind="bf16", order="token", pad=0, seed=0):
        self.page, self.heads, self.dim, self.kind, self.n_pages = page, heads, dim, kind, n_pages
        dtype, self.cache_dtype, t = KINDS[kind]
        g = torch.Generator().manual_seed(seed)
        self.order = order
        inner = (page, heads, dim) if order == "token" else (heads, page, dim)
        self.strides = dict(page_stride=page * heads * dim + pad, token_stride=heads * dim if order == "token" else dim,
                            head_stride=dim if order == "token" else page * dim)
        self.dtype = dtype

        def cache():
            flat = torch.randint(0, 100, (max(n_pages, 1), page * heads * dim + pad), generator=g).to(t).cuda()
            return flat, flat[:, :page * heads * dim].unflatten(1, inner)

        self.k, self.k_view = cache()
        self.v, self.v_view = cache()
        shape = {"e4m3": (n_pages, heads, page), "page": (n_pages, heads)}.get(kind)
        self.ks, self.vs = (None if shape is None else torch.rand(shape, generator=g).cuda() for _ in range(2))

    def cfg(self, n_seqs, max_pages, **kw):
        return moe.attn_config(**{**dict(n_seqs=n_seqs, n_tokens=0, n_heads=self.heads, n_kv_heads=self.heads, head_dim=self.dim,
                                         page_size=self.page, n_pages=self.n_pages, max_pages=max_pages, dtype=self.dtype,
                                         cache_dtype=self.cache_dtype), **self.strides, **kw})

    def caches(self):
        return self.k, self.v, self.ks, self.vs

    def tokens(self, x):
        """[page][token][head][dim] on the host."""
        x = x.cpu()
        return x if self.order == "token" else x.transpose(1, 2)

    def state(self):
        r = [self.tokens(self.k_view).clone(), self.tokens(self.v_view).clone()]
        return r + [None if x is None else x.cpu().clone() for x in (self.ks, self.vs)]

    def copied(self, state, pairs, of=None):
        """A state after copies (from, to, tokens)."""
        of = of or state
        of = [None if x is None else x.clone() for x in of]
        out = [None if x is None else x.clone() for x in state]
        for a, b, n in pairs:
            for x, y in zip(out[:2], of[:2]):
                x[b, :n] = y[a, :n]
            for x, y in zip(out[2:], of[2:]):
                if x is not None and x.dim() == 3:
                    x[b, :, :n] = y[a, :, :n]
                elif x is not None:
                    x[b] = y[a]
        return out


def equal(a, b):
    return all((x is None and y is None) or torch.equal(x, y) for x, y in zip(a, b))


def pages(n, page):
    return -(-n // page)


def update_lists(page, parent, length, kept, need, table, refs, out):
    """(table, refs, granted, copies) by the definition."""
    B = len(length)
    parent = list(range(B)) if parent is None else parent
    refs, out, copies, granted, drop = list(refs), [list(r) for r in out], [], [], []
    mine = [[] if p < 0 else list(table[p][:pages(k, page)]) for p, k in zip(parent, kept)]
    for b in range(B):
        for p in mine[b]:
            refs[p] += 1
        for p in table[b][:pages(length[b], page)]:
            refs[p] -= 1
    free = [p for p, n in enumerate(refs) if n == 0]
    after, asked = list(refs), 0
    for b in range(B):
        row = mine[b]
        shared = need[b] > kept[b] and kept[b] % page != 0 and refs[row[-1]] > 1
        want = pages(need[b], page) - len(row) + shared
        at, asked = asked, asked + want
        if asked > len(free):
            granted.append(kept[b])
        else:
            granted.append(need[b])
            got = free[at:asked]
            if shared:
                copies.append((row[-1], got[0], kept[b] % page))
                after[row[-1]] -= 1
                row = row[:-1]
            for p in got:
                after[p] = 1
            row = row + got
        out[b][:len(row)] = row
    return out, after, granted, copies


def random_state(rs, B, page, most, n_pages, share=0.5):
    """Sequences some of which share their first pages."""
    length = [int(rs.randint(0, most + 1)) for _ in range(B)]
    ids = list(rs.permutation(n_pages))
    width = pages(most, page) + 3
    table = np.full((B, width), -1)
    for b in range(B):
        n = pages(length[b], page)
        other = int(rs.randint(0, b)) if b and rs.rand() < share else None
        common = min(n, pages(length[other], page)) if other is not None else 0
        if other is not None and rs.rand() < 0.5 and length[other]:
            length[b], n = length[other], pages(length[other], page)  # the last page too
            common = n
        for i in range(n):
            table[b, i] = table[other, i] if i < common else ids.pop()
    refs = np.bincount(table[table >= 0], minlength=n_pages)
    return length, table, refs


def run_update(pool, parent, length, kept, need, table, refs, in_place=False):
    B, width = table.shape
    cfg = pool.cfg(B, width)
    ws = moe.workspace(cfg, "pages")
    t, r = dev(table), dev(refs)
    t_out = t if in_place else torch.full_like(t, -5)
    r_out = r if in_place else torch.full_like(r, -5)
    need_dev = dev(need)
    granted = need_dev if in_place else torch.full((B,), -5, dtype=torch.int32, device="cuda")
    moe.moe_pages_update(cfg, dev(parent), dev(length), dev(kept), need_dev, t, r, t_out, r_out, granted, *pool.caches(), ws)
    status = moe.moe_stream_status(ws)
    return status, t_out.cpu().tolist(), r_out.cpu().tolist(), granted.cpu().tolist()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("B,page,most,n_pages,order,pad", [
    (1, 1, 5, 9, "token", 0), (3, 4, 30, 40, "token", 0), (7, 16, 100, 64, "head", 0), (20, 7, 90, 300, "token", 64),
    (70, 16, 200, 1100, "head", 32), (1100, 2, 9, 5000, "token", 0),
])
def test_update_matches_the_definition(kind, B, page, most, n_pages, order, pad):
    for seed in range(3):
        rs = np.random.RandomState(seed)
        pool = Pool(n_pages, page, kind=kind, order=order, pad=pad, seed=seed)
        length, table, refs = random_state(rs, B, page, most, n_pages)
        # forks and beams; every other seed each sequence its own parent
        parent = None if seed == 1 else [int(rs.randint(-1, B)) if rs.rand() < 0.5 else b for b in range(B)]
        has = [length[b] if parent is None else 0 if parent[b] < 0 else length[parent[b]] for b in range(B)]
        kept = [n if rs.rand() < 0.6 else int(rs.randint(0, n + 1)) for n in has]
        need = [k + int(rs.choice([0, 1, 1, 3, page, 2 * page])) for k in kept]
        before = pool.state()
        in_place = parent is None
        out0 = table.tolist() if in_place else np.full_like(table, -5).tolist()
        want = update_lists(page, parent, length, kept, need, table.tolist(), refs.tolist(), out0)
        got = run_update(pool, parent, length, kept, need, table, refs, in_place)
        assert got[0] == 0 and got[1] == want[0] and got[2] == want[1] and got[3] == want[2]
        assert equal(pool.state(), pool.copied(before, want[3]))


@pytest.mark.parametrize("B,page,most,n_pages", [(1500, 16, 9, 2100), (9000, 4, 6, 11000)])
@pytest.mark.parametrize("seed", [0, 1])
def test_update_of_more_sequences_than_a_block_keeps_at_hand(B, page, most, n_pages, seed):
    """Over 1024 sequences for each block, in one block and in eight; seed 1 runs out of pages."""
    rs = np.random.RandomState(seed)
    pool = Pool(n_pages, page, heads=1, dim=16)
    length, table, refs = random_state(rs, B, page, most, n_pages)
    kept = [int(rs.randint(0, n + 1)) for n in length]
    need = [k + int(rs.choice([0, 1, page, 2 * page] if seed else [0, 1])) for k in kept]
    before = pool.state()
    want = update_lists(page, None, length, kept, need, table.tolist(), refs.tolist(), table.tolist())
    if seed:
        assert want[2] != need
    got = run_update(pool, None, length, kept, need, table, refs, True)
    assert got[0] == 0 and got[1] == want[0] and got[2] == want[1] and got[3] == want[2]
    assert equal(pool.state(), pool.copied(before, want[3]))


@pytest.mark.parametrize("forks", [False, True])
def test_updates_and_moves_of_long_tables(forks):
    """Tables of up to 400 pages over a pool of 120000, which the largest cluster works on: trimmed,
    grown by up to 300 pages, forked, and the pool compacted."""
    rs = np.random.RandomState(forks)
    B, page, most, n_pages = 250, 1, 400, 120000
    pool = Pool(n_pages, page, heads=1, dim=16)
    length, table, refs = random_state(rs, B, page, most, n_pages)
    table = np.concatenate([table, np.full((B, 300), -1)], 1)
    parent = [int(rs.randint(-1, B)) for _ in range(B)] if forks else None
    has = [length[b] if parent is None else 0 if parent[b] < 0 else length[parent[b]] for b in range(B)]
    kept = [int(rs.randint(0, n + 1)) for n in has]
    need = [k + int(rs.randint(0, 301)) for k in kept]
    before = pool.state()
    out0 = np.full_like(table, -5).tolist()
    want = update_lists(page, parent, length, kept, need, table.tolist(), refs.tolist(), out0)
    got = run_update(pool, parent, length, kept, need, table, refs)
    assert got[0] == 0 and got[1] == want[0] and got[2] == want[1] and got[3] == want[2]
    assert equal(pool.state(), pool.copied(before, want[3]))
    table, refs = np.array(got[1]), np.array(got[2])
    before = pool.state()
    want = compact_lists(page, need, table.tolist(), refs.tolist(), out0)
    assert run_compact(pool, need, table, refs, False) == (0, *want[:4])
    assert equal(pool.state(), pool.copied(before, want[4]))


@pytest.mark.parametrize("n_pages", [6, 7, 8, 9, 10, 40])
def test_update_when_the_pool_runs_out(n_pages):
    """Wants of 0, 2, 3, 0, 1 pages over a pool with few to spare: what is granted is a prefix."""
    page, kept, need = 4, [3, 4, 8, 5, 4], [4, 9, 17, 5, 5]
    table = np.full((5, 6), -1)
    table[0, 0], table[1, 0], table[2, :2], table[3, :2], table[4, 0] = 5, 0, (3, 1), (0, 2), 4
    length = kept
    refs = np.bincount(table[table >= 0], minlength=n_pages)
    pool = Pool(n_pages, page)
    want = update_lists(page, None, length, kept, need, table.tolist(), refs.tolist(), np.full_like(table, -5).tolist())
    got = run_update(pool, None, length, kept, need, table, refs)
    assert got == (0, *want[:3])


def test_eight_samples_of_a_prompt_and_back():
    """A prompt forked into eight, all but one freed again: the counts return to where they were."""
    page, n = 16, 100
    table = np.full((8, 9), -1)
    table[0, :7] = [9, 3, 20, 1, 7, 15, 0]
    refs = np.bincount(table[table >= 0], minlength=40)
    length = [n] + [0] * 7
    pool = Pool(40, page)
    before = pool.state()
    status, t, r, granted = run_update(pool, [0] * 8, length, [n] * 8, [n + 1] * 8, table, refs)
    assert status == 0 and granted == [n + 1] * 8
    assert all(row[:6] == [9, 3, 20, 1, 7, 15] for row in t) and len({row[6] for row in t}) == 8
    assert r[9] == 8 and r[0] == 0 and sum(r) == 8 * 7  # the shared partial page is given up by all
    after = pool.state()
    for row in t:
        assert torch.equal(after[0][row[6], :4], before[0][0, :4])
    status, t, r, granted = run_update(pool, None, granted, [n + 1] + [0] * 7, [n + 1] + [0] * 7, np.array(t), np.array(r))
    assert status == 0 and sum(r) == 7 and r[9] == 1 and granted == [n + 1] + [0] * 7


def test_a_page_held_by_the_caller_is_copied():
    table = np.array([[2, -1]])
    pool = Pool(4, 4)
    refs = np.array([0, 0, 2, 0])  # the caller holds page 2 as well
    status, t, r, granted = run_update(pool, None, [3], [3], [4], table, refs)
    assert (status, t[0][0], r, granted) == (0, 0, [1, 0, 1, 0], [4])
    status, t, r, granted = run_update(pool, None, [3], [2], [2], table, refs)  # nothing is written: it stays
    assert (status, t[0][0], r, granted) == (0, 2, [0, 0, 2, 0], [2])


@pytest.mark.parametrize("change", ["parent", "len", "len_high", "kept", "need", "need_high", "page", "page_low", "count"])
def test_update_records_bad_lists(change):
    parent, length, kept, need = [0, 1], [5, 3], [5, 3], [6, 4]
    table, refs = np.array([[0, 1, -1], [2, -1, -1]]), np.array([1, 1, 1, 0, 0])
    if change == "parent":
        parent[1] = 2
    elif change == "len":
        length[1] = -1
    elif change == "len_high":
        length[1] = 13
    elif change == "kept":
        kept[1] = 4
    elif change == "need":
        need[1] = 2
    elif change == "need_high":
        need[1] = 13
    elif change == "page":
        table[1, 0] = 5
    elif change == "page_low":
        table[1, 0] = -1
    else:
        refs[2], kept[1], need[1] = 0, 0, 0  # given up below 0
    status, *_ = run_update(Pool(5, 4), parent, length, kept, need, table, refs)
    assert status == moe.MOE_ERR_DEVICE_CHECK


def test_updates_without_sequences_or_pages():
    pool = Pool(5, 4)
    cfg = pool.cfg(0, 0)
    ws = moe.workspace(cfg, "pages")
    refs, out = dev([1, 0, 2, 0, 0]), dev([9] * 5)
    moe.moe_pages_update(cfg, None, None, None, None, None, refs, None, out, None, *pool.caches(), ws)
    assert moe.moe_stream_status(ws) == 0 and torch.equal(refs, out)
    cfg = Pool(0, 4).cfg(2, 0)
    ws = moe.workspace(cfg, "pages")
    zero, granted = dev([0, 0]), dev([5, 5])
    moe.moe_pages_update(cfg, None, zero, zero, zero, None, None, None, None, granted, None, None, None, None, ws)
    assert moe.moe_stream_status(ws) == 0 and granted.tolist() == [0, 0]


def test_updates_replayed_and_of_two_graphs_that_share_a_workspace():
    """Two captured updates on one workspace, replayed one after the other on their stream."""
    rs = np.random.RandomState(3)
    pool = Pool(400, 8)
    length, table, refs = random_state(rs, 12, 8, 100, 400)
    cfg = pool.cfg(12, table.shape[1])
    ws = moe.workspace(cfg, "pages")
    runs = []
    for step in (1, 9):
        need = [n + step for n in length]
        want = update_lists(8, None, length, length, need, table.tolist(), refs.tolist(), np.full_like(table, -5).tolist())
        args = [dev(length), dev(length), dev(need), dev(table), dev(refs)]
        outs = [torch.full_like(args[3], -5), torch.full_like(args[4], -5), torch.zeros_like(args[0])]
        call = lambda a=args, o=outs: moe.moe_pages_update(cfg, None, *a, *o, *pool.caches(), ws)  # noqa: E731
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        runs.append((g, outs, want))
    for _ in range(2):
        for g, outs, want in runs:
            for o in outs:
                o.fill_(-5)
            g.replay()
            torch.cuda.synchronize()
            assert [o.tolist() for o in outs] == [want[0], want[1], want[2]]


def compact_lists(page, length, table, refs, out):
    live = [p for p, n in enumerate(refs) if n > 0]
    holes = [p for p in range(len(live)) if refs[p] <= 0]
    moves = list(zip([p for p in live if p >= len(live)], holes))
    there = {**{p: p for p in live}, **dict(moves)}
    out = [list(r) for r in out]
    for b, n in enumerate(length):
        for i in range(pages(n, page)):
            out[b][i] = there[table[b][i]]
    counts = [0] * len(refs)
    for p, q in there.items():
        counts[q] = refs[p]
    return out, counts, [there.get(p, -1) for p in range(len(refs))], [len(live)], [(a, b, page) for a, b in moves]


def run_compact(pool, length, table, refs, in_place):
    B, width = table.shape
    cfg = pool.cfg(B, width)
    ws = moe.workspace(cfg, "pages")
    t, r = dev(table), dev(refs)
    t_out, r_out = (t, r) if in_place else (torch.full_like(t, -5), torch.full_like(r, -5))
    page_map, live = torch.full_like(r, -5), dev([-5])
    moe.moe_pages_compact(cfg, dev(length), t, r, t_out, r_out, page_map, live, *pool.caches(), ws)
    status = moe.moe_stream_status(ws)
    return status, t_out.cpu().tolist(), r_out.cpu().tolist(), page_map.cpu().tolist(), live.cpu().tolist()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("B,page,most,n_pages,order", [
    (1, 1, 5, 9, "token"), (4, 4, 30, 40, "head"), (20, 7, 90, 300, "token"), (90, 16, 200, 2000, "token"), (600, 2, 9, 40001, "head"),
])
def test_compact_matches_the_definition(kind, B, page, most, n_pages, order):
    for seed in range(2):
        rs = np.random.RandomState(seed)
        pool = Pool(n_pages, page, kind=kind, order=order, seed=seed, heads=1 if n_pages > 9999 else 3, dim=16)
        length, table, refs = random_state(rs, B, page, most, n_pages)
        refs[rs.permutation(n_pages)[:2]] += 1  # two pages of the caller's
        before = pool.state()
        out0 = table.tolist() if seed else np.full_like(table, -5).tolist()
        want = compact_lists(page, length, table.tolist(), refs.tolist(), out0)
        assert run_compact(pool, length, table, refs, seed == 1) == (0, *want[:4])
        assert equal(pool.state(), pool.copied(before, want[4]))


def test_compact_of_full_and_empty_pools():
    for refs in ([1] * 6, [0] * 6, [0, 0, 0, 0, 0, 1], [1, 0, 0, 0, 0, 0]):
        pool = Pool(6, 4)
        table = np.full((1, 6), -1)
        live = [p for p, n in enumerate(refs) if n]
        table[0, :len(live)] = live[::-1]
        want = compact_lists(4, [4 * len(live)], table.tolist(), refs, np.full_like(table, -5).tolist())
        assert run_compact(pool, [4 * len(live)], table, np.array(refs), False) == (0, *want[:4])


@pytest.mark.parametrize("change", ["len", "page", "free", "count"])
def test_compact_records_bad_lists(change):
    length, table, refs = [5, 3], np.array([[0, 1, -1], [4, -1, -1]]), np.array([1, 1, 0, 0, 1])
    if change == "len":
        length[0] = 13
    elif change == "page":
        table[0, 1] = 5
    elif change == "free":
        table[0, 1] = 2
    else:
        refs[3] = -1
    status, *_ = run_compact(Pool(5, 4), length, table, refs, False)
    assert status == moe.MOE_ERR_DEVICE_CHECK


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("n,page,heads,dim,order,pad", [
    (0, 4, 1, 16, "token", 0), (1, 1, 1, 16, "token", 0), (13, 7, 3, 48, "token", 0), (40, 16, 2, 64, "head", 16), (5, 200, 5, 80, "token", 0),
])
def test_copy_between_pools(kind, n, page, heads, dim, order, pad):
    a, b = (Pool(m, page, heads, dim, kind, order, pad, seed=s) for m, s in ((50, 1), (60, 2)))
    rs = np.random.RandomState(n)
    src, dst = rs.randint(0, 50, n), rs.permutation(60)[:n]
    before = b.state()
    cfg = b.cfg(1, 1)
    ws = moe.workspace(cfg, "pages")
    moe.moe_pages_copy(cfg, dev(src), dev(dst), 50, *a.caches(), *b.caches(), ws)
    assert moe.moe_stream_status(ws) == 0
    assert equal(b.state(), b.copied(before, [(int(x), int(y), page) for x, y in zip(src, dst)], a.state()))


def test_copy_leaves_out_and_records_pages_that_are_not_there():
    for src, dst in (([0, 4], [1, 2]), ([0, 1], [1, 6]), ([-1, 0], [3, 1]), ([2, 0], [-1, 1])):
        a, b = Pool(4, 4, seed=1), Pool(6, 4, seed=2)
        before = b.state()
        ws = moe.workspace(b.cfg(1, 1), "pages")
        moe.moe_pages_copy(b.cfg(1, 1), dev(src), dev(dst), 4, *a.caches(), *b.caches(), ws)
        assert moe.moe_stream_status(ws) == moe.MOE_ERR_DEVICE_CHECK
        assert equal(b.state(), b.copied(before, [(0, 1, 4)], a.state()))


def test_copies_past_32_bit_offsets():
    """A cache of more than 2^32 elements: 300000 pages of 16 x 8 x 128 bytes (4.9 GB each of K, V)."""
    n, page, heads, dim = 300000, 16, 8, 128
    cfg = moe.attn_config(n_seqs=1, n_tokens=0, n_heads=heads, n_kv_heads=heads, head_dim=dim, page_size=page, n_pages=n, max_pages=1,
                          cache_dtype=moe.MOE_E4M3_PAGE)
    k, v = (torch.zeros((n, page * heads * dim), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((n, heads), device="cuda") for _ in range(2))
    k[5], v[5], ks[5], vs[5] = 3, 4, 5.0, 6.0
    ws = moe.workspace(cfg, "pages")
    moe.moe_pages_copy(cfg, dev([5]), dev([n - 1]), n, k, v, ks, vs, k, v, ks, vs, ws)
    assert moe.moe_stream_status(ws) == 0
    assert (k[n - 1] == 3).all() and (v[n - 1] == 4).all() and (ks[n - 1] == 5).all() and (vs[n - 1] == 6).all()
    assert int(k[:5].sum()) == 0 and int(k[6:n - 1].sum(dtype=torch.long)) == 0
