"""Attention of entries that share prefixes, on the GPU against the 64-bit form of tests/cache_reference.py."""
import numpy as np
import pytest
import torch

import cache_reference as R
from test_gpu_cache import DT, check, ints, make, normal, np64, random_parents, starts, _D

pytestmark = pytest.mark.gpu


def lay_out(c, rng, g, groups, ramp=0.0):
    """Pages of the groups' sequences anywhere in the pool, values drawn per group: groups is a list of
    (shared tokens, [(tokens behind them, rows)]).  -> sequences, lengths, rows, keys and values per entry."""
    cfg, ps, dt = c.cfg, c.cfg.page_size, DT[c.cfg.dtype]
    c.pages.fill_(float("nan"))     # what no slot of an entry holds must not matter
    c.table.fill_(-1)
    c.refs.zero_()
    n = sum(len(m) for _, m in groups)
    seqs = rng.permutation(cfg.max_seq)[:n].tolist()
    perm, at, e = rng.permutation(cfg.n_pages), 0, 0
    lens, counts, kv = [], [], []

    def put(page, first, data):     # data [2][slots][hkv][hd] from slot `first` of the page on
        c.pages[int(page), cfg.n_layer - 1, :, :, first:first + data.shape[1]] = data.transpose(1, 2).cuda()

    for shared, members in groups:
        head = normal(g, (2, shared, cfg.n_head_kv, cfg.head_dim), cfg.dtype)
        if ramp:
            p = torch.arange(shared, dtype=torch.float32)
            head[0] = (head[0].float() * (1 + abs(ramp) * (p if ramp > 0 else shared - p))[:, None, None]).to(dt)
        full = shared // ps
        common = perm[at:at + full]
        at += full
        for i, p in enumerate(common):
            put(p, 0, head[:, i * ps:(i + 1) * ps])
        for tail, rows in members:
            q = seqs[e]
            own = normal(g, (2, tail + rows, cfg.n_head_kv, cfg.head_dim), cfg.dtype)
            data = torch.cat([head, own], 1)
            h = -(-data.shape[1] // ps)
            mine = np.concatenate([common, perm[at:at + h - full]])
            at += h - full
            assert at <= len(perm)
            c.table[q, :h] = ints(mine)
            c.refs.index_add_(0, ints(mine).long(), torch.ones(h, dtype=torch.int32, device="cuda"))
            c.length[q] = shared + tail
            for i in range(full, h):
                put(mine[i], 0, data[:, i * ps:(i + 1) * ps])
            lens.append(shared + tail)
            counts.append(rows)
            kv.append(np64(data))
            e += 1
    return seqs, lens, counts, kv


def prefix_case(c, rng, g, groups, mask_kind="chain", tail=2, with_lse=True, ramp=0.0, max_tree=None, plan_is=None):
    cfg = c.cfg
    hq, hd, layer = cfg.n_head, cfg.head_dim, cfg.n_layer - 1
    seqs, lens, counts, kv = lay_out(c, rng, g, groups, ramp)
    T = sum(counts) + tail
    fused = normal(g, (T, hq + 2, hd), cfg.dtype)
    q = fused.cuda()[:, 1:1 + hq]
    words = max(1, -(-max(counts + [1]) // 32))
    mask, sets, r = np.zeros((T, words), dtype=np.int32), [], 0
    for cnt in counts:
        if mask_kind == "tree":
            m = R.tree_sets(random_parents(rng, cnt, "forest"))
        elif mask_kind == "bits":
            m = rng.random((cnt, cnt)) < 0.3
            m[rng.random(cnt) < 0.4] = False
        else:
            m = np.tril(np.ones((cnt, cnt), dtype=bool))
        if mask_kind != "chain" and cnt:
            mask[r:r + cnt] = R.words_of(m, words)
        sets.append(m)
        r += cnt
    out = torch.full((T, hq + 1, hd), 5.0, dtype=DT[cfg.dtype], device="cuda")
    lse = torch.full((T, hq), 5.0, dtype=torch.float32, device="cuda") if with_lse else None
    bounds = ints(np.concatenate([[0], np.cumsum([len(m) for _, m in groups])]))
    plan = torch.full((len(seqs) + len(groups),), -9, dtype=torch.int32, device="cuda")
    work = torch.full((c.prefix_workspace(T),), 255, dtype=torch.uint8, device="cuda")    # NaN
    c.dflash_prefix_plan(bounds, plan, seqs=ints(seqs))
    full = [s // cfg.page_size * cfg.page_size if len(m) > 1 else 0 for s, m in groups]
    worth = [f if f * (len(m) - 1) >= 2048 else 0 for f, (_, m) in zip(full, groups)]
    assert plan.tolist() == [f for f, (_, m) in zip(worth, groups) for _ in m] + worth
    # (all that is common, whether worth it or not, unless the case says otherwise)
    every = [f for f, (_, m) in zip(full, groups) for _ in m] + full
    if plan_is != "as made":
        plan.copy_(ints(every if plan_is is None else plan_is(every)))
    call = dict(mask=None if mask_kind == "chain" else ints(mask), seqs=ints(seqs))
    c.dflash_prefix_attend(layer, starts(counts), max_tree or max(counts + [1]), q, out[:, :hq], bounds, plan, work, lse=lse,
                           **call)
    r, scale = 0, cfg.attn_scale or hd ** -0.5
    for n, cnt, m, (k, v) in zip(lens, counts, sets, kv):
        sees = np.concatenate([np.ones((cnt, n), dtype=bool), m], 1)
        o, ls, size, big = R.attend(np64(fused[r:r + cnt, 1:1 + hq]), k, v, sees, scale)
        tol, tol_l = R.attend_bounds(o, size, big, n + cnt, hd, cfg.dtype)
        # the two parts' weights: another exponential (2^-22, its argument of magnitude up to `big`), two
        # products and a sum
        more = 2.0 ** -22 + big * 2.0 ** -23 + 2.0 ** -22
        check(np64(out[r:r + cnt, :hq]), o, tol + 2.02 * size * more[..., None], f"length {n}, {cnt} rows")
        if with_lse:
            got, empty = np64(lse[r:r + cnt]), np.isinf(ls)
            assert (got[empty] == -np.inf).all()
            check(got[~empty], ls[~empty], (tol_l + more)[~empty], "lse")
        r += cnt
    assert (out[r:] == 5.0).all() and (out[:, hq:] == 5.0).all()
    if with_lse:
        assert (lse[r:] == 5.0).all()
    assert c.dflash_cache_read_status() == 0
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd,hq,hkv,ps", [(64, 4, 2, 16), (128, 8, 1, 64), (128, 8, 2, 128), (32, 3, 3, 32),
                                          (64, 6, 2, 256), (128, 4, 4, 16), (128, 5, 1, 32), (32, 12, 2, 64)], ids=str)
@pytest.mark.parametrize("mask_kind", ["chain", "tree", "bits"])
def test_prefix_attend(dtype, hd, hq, hkv, ps, mask_kind):
    rng = np.random.default_rng(hd + hq + ps)
    g = torch.Generator().manual_seed(hd * hq + ps)
    c = make(n_layer=2, n_head=hq, n_head_kv=hkv, head_dim=hd, page_size=ps, n_pages=260, max_seq=12, max_pages=64, dtype=dtype)
    # pages that end inside a tile, whole tiles; a group that shares nothing, one of one member, one without rows
    prefix_case(c, rng, g, [(2 * ps + 3, [(0, 1), (5, 1)])], mask_kind)
    prefix_case(c, rng, g, [(256, [(0, 3), (1, 0), (300, 17)]), (ps - 1, [(0, 2), (4, 1)]), (129, [(7, 5)]),
                            (700, [(3, 33), (0, 1), (64, 2)]), (ps, [(0, 0), (0, 0)])], mask_kind)
    prefix_case(c, rng, g, [(500, [(20, 64), (3, 65), (0, 70)])], mask_kind, with_lse=False, tail=0,
                max_tree=96 if mask_kind != "chain" else 5000)
    prefix_case(c, rng, g, [(3 * ps, [(ps, 1)] * 11)], mask_kind, tail=1)
    prefix_case(c, rng, g, [(600, [(20, 3)] * 9), (ps + 5, [(9, 4), (600, 40)]), (40, [(0, 1)])], mask_kind, plan_is="as made")


@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("bf16", 64), ("bf16", 32), ("f32", 128)])
def test_prefix_long_and_many(dtype, hd):
    """One long prefix cut over all SMs; tall tiles of many members; as many entries as a call may have."""
    rng = np.random.default_rng(9)
    g = torch.Generator().manual_seed(9)
    c = make(n_head=4, n_head_kv=1, head_dim=hd, page_size=64, n_pages=900, max_seq=100, max_pages=400, dtype=dtype)
    prefix_case(c, rng, g, [(20011, [(int(t), 1) for t in rng.integers(0, 200, 3)])])
    prefix_case(c, rng, g, [(3000, [(int(t), int(k)) for t, k in zip(rng.integers(0, 300, 90), rng.integers(1, 5, 90))])], "tree")
    prefix_case(c, rng, g, [(2000, [(5, 300), (70, 200)])])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefix_most_entries(dtype):
    rng = np.random.default_rng(10)
    g = torch.Generator().manual_seed(10)
    c = make(n_head=4, n_head_kv=1, head_dim=128, page_size=16, n_pages=4000, max_seq=1024, max_pages=12, dtype=dtype)
    sizes = [1, 2, 3, 60, 5, 9] + [7] * 105        # 815 entries, 111 groups
    groups = [(int(rng.integers(0, 70)), [(int(rng.integers(0, 20)), int(rng.integers(0, 3))) for _ in range(k)]) for k in sizes]
    prefix_case(c, rng, g, groups, "tree")
    prefix_case(c, rng, g, [(33, [(int(rng.integers(0, 20)), int(rng.integers(0, 3))) for _ in range(1023)])], "chain")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("ramp", [0.1, -0.1])
def test_prefix_scores_that_grow_along_it(dtype, hd, ramp):
    """References that move within the shared part, and differ from the entries'."""
    rng = np.random.default_rng(3)
    g = torch.Generator().manual_seed(3)
    c = make(n_head=4, n_head_kv=2, head_dim=hd, page_size=32, n_pages=100, max_seq=6, max_pages=40, dtype=dtype)
    prefix_case(c, rng, g, [(1000, [(0, 1), (40, 3), (7, 2)])], ramp=ramp)


def test_a_plan_may_share_less():
    """What the plan says is what is computed for all; slots that end no page are rounded down."""
    rng = np.random.default_rng(3)
    g = torch.Generator().manual_seed(3)
    c = make(n_head=4, n_head_kv=2, head_dim=128, page_size=32, n_pages=100, max_seq=6, max_pages=40)
    for less in (lambda v: 0, lambda v: 64, lambda v: min(v, 130)):
        prefix_case(c, rng, g, [(500, [(0, 1), (40, 3)]), (200, [(9, 9), (9, 9)])], plan_is=lambda p: [less(v) for v in p])


def test_plan_follows_forks_and_tables():
    c = make(n_layer=1, page_size=256, n_pages=80, max_seq=6, max_pages=40)
    c.dflash_cache_reserve(ints([4400]), seqs=ints([2]))
    c.dflash_cache_commit(None, ints([4400]), seqs=ints([2]))        # 17 full pages and 48 slots
    c.dflash_cache_fork(ints([2, 2]), ints([0, 5]))
    c.dflash_cache_reserve(ints([300, 300, 300]), seqs=ints([2, 0, 5]))  # the part-filled page becomes each one's own
    plan = torch.zeros(5, dtype=torch.int32, device="cuda")

    def made(bounds, seqs):
        plan.fill_(7)
        c.dflash_prefix_plan(ints(bounds), plan, seqs=ints(seqs))
        return plan.tolist()

    assert made([0, 3, 3], [2, 0, 5]) == [4352, 4352, 4352, 4352, 0]
    assert made([1, 3], [5, 2, 0, 1]) == [0, 4352, 4352, 0, 4352]    # entries outside every group
    assert made([0, 2, 3], [2, 0, 5]) == [4352, 4352, 0, 4352, 0]
    assert made([0, 4], [2, 0, 5, 1]) == [0, 0, 0, 0, 0]             # sequence 1 is empty
    assert made([0, 3, 3], [2, 2, 2]) == [4352, 4352, 4352, 4352, 0]  # (4352 of 4400: full pages)
    c.dflash_cache_trim(ints([2400]), seqs=ints([0]))
    assert made([0, 3, 3], [2, 0, 5]) == [2304, 2304, 2304, 2304, 0]
    c.table[5, 8] = c.table[5, 10]
    assert made([0, 3, 3], [2, 0, 5]) == [2048, 2048, 2048, 2048, 0]
    assert made([0, 2, 3], [2, 5, 0]) == [2048, 2048, 0, 2048, 0]
    c.table[5, 7] = c.table[5, 10]
    assert made([0, 3, 3], [2, 0, 5]) == [1792, 1792, 1792, 1792, 0]
    assert made([0, 2, 3], [2, 5, 0]) == [0, 0, 0, 0, 0]             # 1792 slots saved once: not worth it
    c.table[5, 3] = c.table[5, 10]
    assert made([0, 3, 3], [2, 0, 5]) == [0, 0, 0, 0, 0]             # 768 saved twice
    assert c.dflash_cache_read_status() == 0
    for bounds in ([0, 4, 3], [-1, 2, 3], [0, 2, 9]):
        assert made(bounds, [2, 0, 5]) == [0] * 5
        assert c.dflash_cache_read_status() == 0x8
    assert made([0, 3, 3], [2, 7, 5]) == [0] * 5                     # no such sequence: nothing is shared
    c.dflash_cache_read_status()


def test_prefix_faults():
    D = _D()
    rng = np.random.default_rng(1)
    g = torch.Generator().manual_seed(1)
    c = make(n_head=2, n_head_kv=1, head_dim=64, page_size=16, n_pages=32, max_seq=5, max_pages=6)
    seqs, lens, counts, _ = lay_out(c, rng, g, [(40, [(0, 2), (3, 2), (9, 4)])])
    q = torch.randn(8, 2, 64, device="cuda").bfloat16()
    work = torch.empty(c.prefix_workspace(8), dtype=torch.uint8, device="cuda")
    good = ints([32] * 4)

    def run(status, changed, row_start=(0, 2, 4, 8), sq=seqs, plan=good, bounds=(0, 3), max_tree=4):
        out = torch.full_like(q, 9.0)
        c.dflash_prefix_attend(0, ints(row_start), max_tree, q, out, ints(bounds), plan, work, seqs=ints(sq))
        assert c.dflash_cache_read_status() == status
        got = (out != 9.0).flatten(1).any(1).nonzero().flatten().tolist()
        assert got == changed, got

    run(0, list(range(8)))
    run(0x8, list(range(4)), max_tree=3)                               # more nodes than announced
    run(0x8, list(range(4)), row_start=(0, 2, 4, 9))                   # the group's range is none either
    run(0x40, [0, 1, 4, 5, 6, 7], sq=[seqs[0], 5, seqs[2]])
    run(0x40, [2, 3, 4, 5, 6, 7], sq=[-1, seqs[1], seqs[2]])
    run(0x8, [], plan=ints([48, 48, 64, 48]))                          # more than the lengths (40, 43, 49) have
    run(0x8, [2, 3, 4, 5, 6, 7], plan=ints([-16, 32, 32, 32]))
    run(0x8, list(range(8)), bounds=(0, 4))
    run(0x8, list(range(8)), bounds=(2, 1), plan=good)
    c.table[seqs[0], 0] = 99
    out = torch.empty_like(q)
    c.dflash_prefix_attend(0, ints([0, 2, 4, 8]), 4, q, out, ints([0, 3]), good, work, seqs=ints(seqs))
    assert c.dflash_cache_read_status() == 0x10
    with pytest.raises(D.DFlashError, match="prefix_workspace"):
        c.dflash_prefix_attend(0, ints([0, 2, 4, 8]), 4, q, out, ints([0, 3]), good, work[:-1], seqs=ints(seqs))
    with pytest.raises(D.DFlashError):
        c.dflash_prefix_attend(1, ints([0, 2, 4, 8]), 4, q, out, ints([0, 3]), good, work, seqs=ints(seqs))
    c.dflash_prefix_attend(0, ints([0, 0]), 1, q[:0], out[:0], ints([0, 1]), good[:2], work)
    assert c.dflash_cache_read_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_on_another_stream(dtype):
    """A captured plan and attention follow lengths and tables; the same bits eagerly on a side stream."""
    rng = np.random.default_rng(2)
    g = torch.Generator().manual_seed(2)
    c = make(n_head=8, n_head_kv=2, head_dim=128, page_size=32, n_pages=400, max_seq=8, max_pages=80, dtype=dtype)
    T = 8 * 5
    q = normal(g, (T, 8, 128), dtype).cuda()
    start, bounds = starts([5] * 8), ints([0, 4, 8])
    outs = [torch.zeros_like(q) for _ in range(2)]
    lses = [torch.zeros(T, 8, device="cuda") for _ in range(2)]
    plans = [torch.zeros(10, dtype=torch.int32, device="cuda") for _ in range(2)]
    works = [torch.zeros(c.prefix_workspace(T), dtype=torch.uint8, device="cuda") for _ in range(2)]
    seqs = torch.zeros(8, dtype=torch.int32, device="cuda")

    def turn(i, stream=None):
        c.dflash_prefix_plan(bounds, plans[i], seqs=seqs, stream=stream)   # (shares from 704 tokens on)
        c.dflash_prefix_attend(0, start, 5, q, outs[i], bounds, plans[i], works[i], lse=lses[i], seqs=seqs, stream=stream)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        turn(0)
    for it in range(4):
        sq, *_ = lay_out(c, rng, g, [(int(rng.integers(500, 2200)), [(int(t), 5) for t in rng.integers(0, 90, 4)]) for _ in range(2)])
        seqs.copy_(ints(sq))
        graph.replay()
        torch.cuda.synchronize()
        turn(1, stream=side)
        torch.cuda.synchronize()
        for a, b in (outs, lses, plans):
            assert torch.equal(a, b)
        assert not torch.isnan(outs[0]).any()
    assert c.dflash_cache_read_status() == 0


def test_offsets_past_32_bits():
    """Pages behind 4 GB, shared by three sequences."""
    c = make(n_layer=1, n_head=8, n_head_kv=8, head_dim=128, page_size=256, n_pages=8400, max_seq=3, max_pages=4)
    assert c.pages.numel() * 2 > 1 << 32
    g = torch.Generator().manual_seed(0)
    pages = [8399, 8398, 8300]
    kv = normal(g, (2, 600, 8, 128), "bf16")
    for i, p in enumerate(pages):
        part = kv[:, 256 * i:256 * (i + 1)]
        c.pages[p, 0, :, :, :part.shape[1]] = part.transpose(1, 2).cuda()
    for s in range(3):
        c.table[s, :3] = ints([pages[0], pages[1], pages[2]])
        c.length[s] = 599
    q, out = normal(g, (3, 8, 128), "bf16"), torch.zeros(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    plan = torch.zeros(4, dtype=torch.int32, device="cuda")
    work = torch.empty(c.prefix_workspace(3), dtype=torch.uint8, device="cuda")
    plan.fill_(512)
    c.dflash_prefix_attend(0, starts([1, 1, 1]), 1, q.cuda(), out, ints([0, 3]), plan, work)
    k, v = np64(kv)
    for s in range(3):
        o, _, size, big = R.attend(np64(q[s:s + 1]), k, v, np.ones((1, 600), bool), 128 ** -0.5)
        tol, _ = R.attend_bounds(o, size, big, 600, 128, "bf16")
        check(np64(out[s:s + 1]), o, tol + 2.02 * size * (2.0 ** -21 + big[..., None] * 2.0 ** -23), f"sequence {s}")
    assert c.dflash_cache_read_status() == 0


def test_calls_that_the_library_refuses():
    """Bad counts, null pointers and work areas return before anything is launched."""
    D = _D()
    c = make(n_head=2, n_head_kv=1, head_dim=64)
    L, h, p = D.LIB, c.h, torch.zeros(4096, device="cuda").data_ptr()
    assert p % 256 == 0

    def plan(n=1, g=1, start=p, out=p):
        return L.dflash_prefix_plan(h, n, None, g, start, out, None)

    assert plan(g=0) == plan(g=-1) == plan(start=None) == plan(out=None) == -1
    assert plan(n=-1) == plan(n=1024) == plan(n=1, g=1024) == -4

    def attend(layer=0, n=1, T=1, most=1, mask=None, words=0, g=1, start=p, pl=p, work=p, q=p, out=p + 8192, rs=p):
        return L.dflash_prefix_attend(h, layer, n, None, rs, T, most, mask, words, g, start, pl, work, q, 128, out, 128, None, None)

    assert attend(layer=1) == attend(most=0) == attend(T=-1) == attend(g=0) == attend(start=None) == attend(pl=None) == -1
    assert attend(work=None) == attend(work=p + 16) == attend(q=None) == attend(out=p + 4) == attend(rs=None) == -1
    assert attend(mask=p, words=0) == attend(mask=p, words=33) == attend(mask=p, words=1, most=33) == -1
    assert attend(n=1023, g=2) == -4 and attend(n=0, work=None) == attend(T=0, work=None) == 0
    assert L.dflash_prefix_workspace_size(h, -1, None) == -1
    assert c.dflash_cache_read_status() == 0


def test_two_handles_on_two_streams():
    """Plans and attention of two handles at the same time equal those of each alone, bit for bit."""
    rng = np.random.default_rng(7)
    g = torch.Generator().manual_seed(7)
    sides = []
    for _ in range(2):
        c = make(n_head=8, n_head_kv=2, head_dim=128, page_size=64, n_pages=120, max_seq=6, max_pages=64)
        seqs, *_ = lay_out(c, rng, g, [(2000, [(int(t), 3) for t in rng.integers(0, 300, 6)])])
        q = normal(g, (18, 8, 128), "bf16").cuda()
        sides.append(dict(c=c, q=q, seqs=ints(seqs), s=torch.cuda.Stream(), plan=torch.zeros(7, dtype=torch.int32, device="cuda"),
                          work=torch.zeros(c.prefix_workspace(18), dtype=torch.uint8, device="cuda")))
    start, bounds = starts([3] * 6), ints([0, 6])

    def turn(k, out, stream=None):
        k["c"].dflash_prefix_plan(bounds, k["plan"], seqs=k["seqs"], stream=stream)
        k["c"].dflash_prefix_attend(0, start, 3, k["q"], out, bounds, k["plan"], k["work"], seqs=k["seqs"], stream=stream)

    alone = [torch.zeros_like(k["q"]) for k in sides]
    for k, o in zip(sides, alone):
        turn(k, o)
    assert int(sides[0]["plan"].min()) > 0
    outs = [[torch.zeros_like(k["q"]) for k in sides] for _ in range(10)]
    torch.cuda.synchronize()
    for pair in outs:
        for k, o in zip(sides, pair):
            turn(k, o, stream=k["s"])
    torch.cuda.synchronize()
    for pair in outs:
        for o, want in zip(pair, alone):
            assert torch.equal(o, want)
