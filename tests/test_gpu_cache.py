"""Rotary positions, tree attention over pages, trees and cache pages on the GPU
against 64-bit and plain-Python forms (tests/cache_reference.py)."""
import numpy as np
import pytest
import torch

import cache_reference as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}   # half a step, relative


def _D():
    from block_diffusion_drafter_fc_gb300 import dflash as D
    return D


def make(n_layer=1, n_head=4, n_head_kv=2, head_dim=64, page_size=16, n_pages=64, max_seq=6, max_pages=16, **kw):
    D = _D()
    return D.PagedCache(D.CacheConfig(n_layer=n_layer, n_head=n_head, n_head_kv=n_head_kv, head_dim=head_dim,
                                      page_size=page_size, n_pages=n_pages, max_seq=max_seq, max_pages=max_pages, **kw))


def ints(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def starts(counts):
    return ints(np.concatenate([[0], np.cumsum(counts)]))


def np64(t):
    return t.detach().cpu().double().numpy()


def normal(g, shape, dtype):
    return torch.randn(*shape, generator=g).to(DT[dtype])


def check(got, want, tol, what=""):
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {err.size} off, worst {np.nanmax(err / tol)} of the bound"


# ------------------------------------------------------------------ rope

ROPES = [("half", None, {}), ("interleaved", None, {}), ("half", 0.5, {}), ("interleaved", 0.5, {}),
         ("half", -8, {}), ("interleaved", -8, {}), ("half", 0, {}),
         ("half", None, dict(rope_scaling="linear", rope_factor=4.0)),
         ("interleaved", None, dict(rope_scaling="ntk", rope_factor=8.0)),
         ("half", None, dict(rope_scaling="yarn", rope_factor=8.0, rope_orig_positions=4096)),
         ("half", -8, dict(rope_scaling="yarn", rope_factor=2.0, rope_orig_positions=32768, rope_mscale=0.75))]


def rope_setup(hd, layout, rot, kw):
    rd = hd if rot is None else int(hd * rot) if rot > 0 else hd + rot if rot < 0 else 0
    if rd == 0:
        return rd, np.zeros(0), 1.0
    f, m = R.rope_freqs(rd, scaling=kw.get("rope_scaling", "none"), factor=kw.get("rope_factor", 1.0),
                        orig=kw.get("rope_orig_positions", 0), mscale=kw.get("rope_mscale", 0.0))
    return rd, f, m


def rope_tol(size, want, dtype):
    # sin and cos: argument rounded to 2^-25 of a half turn (1e-7), sincospif within
    # 2^-23; two products and a sum in fp32: 4e-7 (|a| + |b|) m, then one rounding
    return 4e-7 * size + HALF[dtype] * np.abs(want) * 1.01


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("layout,rot,kw", ROPES, ids=str)
def test_rope(dtype, hd, layout, rot, kw):
    rd, f, m = rope_setup(hd, layout, rot, kw)
    c = make(head_dim=hd, dtype=dtype, rope_layout=layout, rotary_dim=rd, **kw)
    g = torch.Generator().manual_seed(hd + len(kw))
    for T, heads in ((1, 1), (3, 5), (37, 2), (130, 9)):
        x = normal(g, (T, heads, hd), dtype)
        pos = torch.randint(0, 3_000_000, (T,), generator=g, dtype=torch.int32)
        pos[0] = 0
        for backward in (False, True):
            out = torch.full((T, heads, hd), float("nan"), dtype=DT[dtype], device="cuda")
            c.dflash_rope(x.cuda(), pos.cuda(), out, backward=backward)
            want, size = R.rope(np64(x), pos.numpy(), layout, rd, f, m, backward)
            check(np64(out), want, rope_tol(size, want, dtype), f"{T} rows")
            np.testing.assert_array_equal(np64(out)[..., rd:], np64(x)[..., rd:])
    assert c.dflash_cache_read_status() == 0


def test_rope_many_rows_in_place_strided_and_far():
    """Several items a thread, a fused projection's rows in place, the largest position."""
    hd = 128
    c = make(head_dim=hd)
    g = torch.Generator().manual_seed(5)
    T = 2500
    fused = normal(g, (T, 48, hd), "bf16")
    pos = torch.randint(0, 200000, (T,), generator=g, dtype=torch.int32)
    pos[7], pos[8] = 2 ** 31 - 1, 1
    dev = fused.cuda()
    c.dflash_rope(dev[:, :40], pos.cuda(), dev[:, :40])
    f, m = R.rope_freqs(hd)
    want, size = R.rope(np64(fused[:, :40]), pos.numpy(), "half", hd, f, m)
    got = np64(dev[:, :40])
    near = pos.numpy() < 2 ** 30
    check(got[near], want[near], rope_tol(size, want, "bf16")[near])
    # a frequency is known to 2^-53 of itself on either side: 2^31 x 2^-53 x 2 at the last position
    check(got[7], want[7], (rope_tol(size, want, "bf16") + 2.0 ** -21 * size)[7])
    assert torch.equal(dev[:, 40:].cpu(), fused[:, 40:])
    assert c.dflash_cache_read_status() == 0


def test_rope_negative_position_skips_its_row():
    D = _D()
    c = make(head_dim=64)
    x = torch.randn(4, 2, 64).bfloat16().cuda()
    out = torch.full_like(x, 7.0)
    c.dflash_rope(x, ints([3, -1, 0, 5]), out)
    assert torch.equal(out[1], torch.full_like(out[1], 7.0)) and torch.equal(out[2], x[2])
    assert c.dflash_cache_read_status() == 2
    assert c.dflash_cache_read_status() == 0
    with pytest.raises(D.DFlashError):   # not 16-byte aligned
        c.dflash_rope(x.flatten()[4:4 + 128].view(1, 2, 64), ints([1]), x[:1])
    c.dflash_rope(x[:0], ints([]), out[:0])


@pytest.mark.parametrize("layout,rot,kw", [ROPES[0], ROPES[3], ROPES[9]], ids=str)
def test_rope_backward_against_differences(layout, rot, kw):
    """The rotation is linear: the gradient of sum(w rope(x)) is rope's backward of w, and
    the change of that sum along a direction d is <backward(w), d> without a remainder."""
    hd = 64
    rd, _, _ = rope_setup(hd, layout, rot, kw)
    c = make(head_dim=hd, dtype="f32", rope_layout=layout, rotary_dim=rd, **kw)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w, d = (torch.randn(33, 3, hd, generator=g, device="cuda") for _ in range(3))
    pos = torch.randint(0, 100000, (33,), generator=g, device="cuda", dtype=torch.int32)
    y0, y1, dx = (torch.empty_like(x) for _ in range(3))
    c.dflash_rope(x, pos, y0)
    c.dflash_rope(x + d, pos, y1)
    c.dflash_rope(w, pos, dx, backward=True)
    lhs = float((w.double() * (y1.double() - y0.double())).sum())
    rhs = float((dx.double() * ((x + d).double() - x.double())).sum())
    # three rotations, each within 4e-7 (|a| + |b|) m + 2^-24 of its values
    scale = float((w.abs().double() * (x.abs() + d.abs() + 1)).sum()) * 4
    assert abs(lhs - rhs) <= 1e-6 * scale


# ------------------------------------------------------------------ trees

def random_parents(rng, n, kind):
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "forest":
        return [int(rng.integers(-1, i)) if i else -1 for i in range(n)]
    return [int(rng.integers(0, i)) if i else -1 for i in range(n)]


@pytest.mark.parametrize("kind", ["chain", "random", "forest"])
@pytest.mark.parametrize("counts,words", [([1], 1), ([0, 5, 32, 1], 1), ([33, 64, 0], 2), ([300, 7, 129], 10),
                                          ([1024, 1000], 32)], ids=str)
def test_tree_mask(kind, counts, words):
    rng = np.random.default_rng(len(counts))
    c = make()
    trees = [random_parents(rng, n, kind) for n in counts]
    T = sum(counts) + 3                    # rows behind the last entry stay
    parents = np.full(T, -7, dtype=np.int32)
    parents[:T - 3] = np.concatenate(trees) if T > 3 else []
    mask = torch.full((T, words), 99, dtype=torch.int32, device="cuda")
    depth = torch.full((T,), 99, dtype=torch.int32, device="cuda")
    c.dflash_tree_mask(starts(counts), ints(parents), mask, depth)
    want_m, want_d = np.full((T, words), 99, dtype=np.int32), np.full(T, 99, dtype=np.int32)
    r = 0
    for t in trees:
        m = R.tree_sets(t)
        want_m[r:r + len(t)], want_d[r:r + len(t)] = R.words_of(m, words), m.sum(1) - 1 if len(t) else 0
        r += len(t)
    np.testing.assert_array_equal(mask.cpu().numpy(), want_m)
    np.testing.assert_array_equal(depth.cpu().numpy(), want_d)
    assert c.dflash_cache_read_status() == 0


def test_tree_mask_faults():
    D = _D()
    c = make()
    mask = torch.zeros(8, 1, dtype=torch.int32, device="cuda")
    c.dflash_tree_mask(starts([4, 4]), ints([-1, 0, 3, 1, -1, -2, 5, 1]), mask)   # 3, -2 and 5 are no earlier nodes
    assert c.dflash_cache_read_status() == 0x20
    assert mask.flatten().tolist() == [1, 3, 4, 11, 1, 2, 4, 10]
    mask.fill_(5)
    c.dflash_tree_mask(ints([0, 6, 3, 9]), ints([-1] * 8), mask)    # [6, 3) is no range, [3, 9) passes T
    assert c.dflash_cache_read_status() == 0x8
    assert mask.flatten().tolist() == [1, 2, 4, 8, 16, 32, 5, 5]
    big = torch.zeros(40, 1, dtype=torch.int32, device="cuda")
    c.dflash_tree_mask(starts([40]), ints([-1] * 40), big)          # more nodes than the words hold
    assert c.dflash_cache_read_status() == 0x8 and int(big.abs().sum()) == 0
    with pytest.raises(D.DFlashError):
        c.dflash_tree_mask(starts([4]), ints([-1] * 4), torch.zeros(4, 33, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("kind", ["chain", "random"])
@pytest.mark.parametrize("vocab", [1, 3, 50])
def test_tree_accept(kind, vocab):
    rng = np.random.default_rng(vocab)
    c = make()
    for counts, max_path in (([1], 1), ([5, 0, 17, 64], 6), ([200, 1, 33], 300), ([2500, 3], 2500), ([9, 9], 1)):
        trees = [random_parents(rng, n, kind) for n in counts]
        T = sum(counts)
        tok, tgt = rng.integers(0, vocab, T), rng.integers(0, vocab, T)
        path = torch.full((len(counts), max_path), 55, dtype=torch.int32, device="cuda")
        n_path = torch.full((len(counts),), 55, dtype=torch.int32, device="cuda")
        id_last = torch.full((len(counts),), 77, dtype=torch.int32, device="cuda")
        c.dflash_tree_accept(starts(counts), ints(np.concatenate(trees)), ints(tok), ints(tgt), path, n_path, id_last)
        r = 0
        for s, t in enumerate(trees):
            n = len(t)
            if n == 0:
                assert path[s].tolist() == [-1] * max_path and int(n_path[s]) == 0 and int(id_last[s]) == 77
                continue
            want, last = R.accept(t, tok[r:r + n].tolist(), tgt[r:r + n].tolist(), max_path)
            assert path[s].tolist() == want + [-1] * (max_path - len(want))
            assert int(n_path[s]) == len(want) and int(id_last[s]) == last
            r += n
    assert c.dflash_cache_read_status() == 0


def test_tree_accept_agrees_with_block_accept():
    """A chain of anchor + 15 drafts accepts what the first-mismatch scan accepts."""
    rng = np.random.default_rng(3)
    c = make()
    n = 40
    tok, tgt = rng.integers(0, 2, (n, 16)), rng.integers(0, 2, (n, 16))
    path, n_path, id_last = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((n, 16), (n,), (n,)))
    c.dflash_tree_accept(starts([16] * n), ints(np.tile(np.arange(-1, 15), n)), ints(tok.ravel()), ints(tgt.ravel()),
                         path, n_path, id_last)
    agree = tok[:, 1:] == tgt[:, :15]
    m = np.where(agree.all(1), 15, np.argmin(agree, 1))
    np.testing.assert_array_equal(n_path.cpu().numpy(), m + 1)
    np.testing.assert_array_equal(id_last.cpu().numpy(), tgt[np.arange(n), m])


# ------------------------------------------------------------------ pages

def state_equal(c, ref):
    assert c.table.cpu().tolist() == ref.table
    assert c.length.cpu().tolist() == ref.length
    assert c.refs.cpu().tolist() == ref.refs


@pytest.mark.parametrize("dtype,ps", [("bf16", 16), ("f32", 64)])
def test_pages_random_walk(dtype, ps):
    """Reserve, commit, fork, trim in random order: table, lengths, counts and every slot
    that holds a token equal a plain form's; nothing is copied that is not shared."""
    rng = np.random.default_rng(ps)
    n_seq, max_pages, n_pages = 9, 12, 40
    c = make(n_layer=3, n_head=2, n_head_kv=2, head_dim=32, page_size=ps, n_pages=n_pages, max_seq=n_seq,
             max_pages=max_pages, dtype=dtype)
    c.pages.normal_()
    ref = R.Pages(n_pages, n_seq, max_pages, ps)
    tokens = [[] for _ in range(n_seq)]     # one number per committed token, written into all of its row
    clock = 0
    shortage = 0
    for step in range(120):
        op = rng.choice(["grow", "grow", "grow", "fork", "trim", "trim"])
        k = int(rng.integers(1, n_seq + 1))
        seqs = rng.permutation(n_seq)[:k].tolist()
        if op == "grow":
            count = [int(rng.integers(0, 3 * ps)) for _ in seqs]
            before = c.pages.clone()
            c.dflash_cache_reserve(ints(count), seqs=ints(seqs))
            done = ref.reserve(seqs, count)
            assert c.dflash_cache_read_status() == (0 if done else 0x80)
            shortage += not done
            state_equal(c, ref)
            if not done:
                assert torch.equal(c.pages, before)
                continue
            for a, b, fill in ref.copies:
                before[b, ..., :fill, :] = before[a, ..., :fill, :]
            assert torch.equal(c.pages, before)
            for q, n in zip(seqs, count):        # the new tokens' rows, then a commit without a path
                for i in range(n):
                    clock += 1
                    p = len(tokens[q])
                    c.pages[ref.table[q][p // ps], ..., p % ps, :] = clock % 251
                    tokens[q].append(clock % 251)
                ref.length[q] += n
            c.dflash_cache_commit(None, ints(count), seqs=ints(seqs))
        elif op == "fork":
            full = [q for q in range(n_seq) if ref.length[q]]
            empty = [q for q in range(n_seq) if not ref.length[q] and ref.table[q][0] < 0]
            if not full or not empty:
                continue
            dst = empty[:int(rng.integers(1, len(empty) + 1))]
            src = [int(rng.choice(full)) for _ in dst]
            c.dflash_cache_fork(ints(src), ints(dst))
            ref.fork(src, dst)
            for a, b in zip(src, dst):
                tokens[b] = list(tokens[a])
        else:
            keep = [int(rng.integers(0, ref.length[q] + ps)) if rng.random() < 0.6 else 0 for q in seqs]
            c.dflash_cache_trim(ints(keep), seqs=ints(seqs))
            ref.trim(seqs, keep)
            for q, n in zip(seqs, keep):
                tokens[q] = tokens[q][:n]
        assert c.dflash_cache_read_status() == 0
        state_equal(c, ref)
        table, pages = c.table.cpu().tolist(), c.pages.float().cpu()
        for q in range(n_seq):
            for p, v in enumerate(tokens[q]):
                assert (pages[table[q][p // ps], ..., p % ps, :] == v).all()
    assert shortage
    c.dflash_cache_trim(ints([0] * n_seq))
    assert c.refs.abs().sum() == 0 and (c.table == -1).all() and c.length.abs().sum() == 0


def test_reserve_long_and_wide():
    """A prompt of thousands of pages, and a pool whose free pages lie far behind."""
    c = make(n_head_kv=1, n_head=1, head_dim=32, n_pages=20000, max_seq=1024, max_pages=16384, page_size=16)
    ref = R.Pages(20000, 1024, 16384, 16)
    for seqs, count in (([3], [16 * 9000 + 5]), ([1000, 2, 3], [16 * 5000, 1, 11]), (list(range(500, 1020)), [17] * 520),
                        ([3], [1]), ([3], [16 * 9000])):
        c.dflash_cache_reserve(ints(count), seqs=ints(seqs))
        done = ref.reserve(seqs, count)
        assert c.dflash_cache_read_status() == (0 if done else 0x80)
        if done:
            for q, n in zip(seqs, count):
                ref.length[q] += n
            c.dflash_cache_commit(None, ints(count), seqs=ints(seqs))
        state_equal(c, ref)
    assert not done


def test_reserve_refusals():
    c = make(max_seq=4, max_pages=3, page_size=16, n_pages=5)
    c.dflash_cache_reserve(ints([10, 20, 5]), seqs=ints([1, 1, 2]))          # the second 1 is not used
    assert c.dflash_cache_read_status() == 0x40
    assert c.table.cpu().tolist() == [[-1] * 3, [0, -1, -1], [1, -1, -1], [-1] * 3]
    c.dflash_cache_reserve(ints([1, -3, 4]), seqs=ints([4, 0, -1]))          # no such sequences, a negative count
    assert c.dflash_cache_read_status() == 0x48
    assert c.refs.cpu().tolist() == [1, 1, 0, 0, 0]
    c.dflash_cache_reserve(ints([1, 49]), seqs=ints([0, 3]))                 # past max_pages
    assert c.dflash_cache_read_status() == 0x80
    c.dflash_cache_reserve(ints([2 ** 31 - 1]), seqs=ints([0]))
    assert c.dflash_cache_read_status() == 0x80
    assert c.refs.cpu().tolist() == [1, 1, 0, 0, 0]
    c.dflash_cache_reserve(ints([]))
    with pytest.raises(_D().DFlashError):
        c.dflash_cache_reserve(ints([0] * 5))                                # identity entries past max_seq
    with pytest.raises(_D().DFlashError):
        c.dflash_cache_trim(ints([0] * 1025), seqs=ints([0] * 1025))


def test_reserve_skips_a_length_out_of_range():
    """One sequence with a length that is none does not keep the others from their pages."""
    c = make(max_seq=4, max_pages=3, page_size=16, n_pages=9)
    for bad in (49, 64, 2 ** 31 - 1, -1, -100):
        c.length[1] = bad
        c.dflash_cache_reserve(ints([20, 5, 1]), seqs=ints([0, 1, 2]))
        assert c.dflash_cache_read_status() == 0x8
        assert c.table.cpu().tolist() == [[0, 1, -1], [-1] * 3, [2, -1, -1], [-1] * 3]
        assert c.refs.cpu().tolist() == [1, 1, 1] + [0] * 6
        c.dflash_cache_trim(ints([0, 0]), seqs=ints([0, 2]))
    c.length[1] = 48                                      # full: no room, and none asked for
    c.dflash_cache_reserve(ints([20, 0, 1]), seqs=ints([0, 1, 2]))
    assert c.dflash_cache_read_status() == 0
    c.dflash_cache_reserve(ints([1]), seqs=ints([1]))
    assert c.dflash_cache_read_status() == 0x80


def test_fork_and_trim_refusals():
    c = make(max_seq=5, max_pages=4, page_size=16, n_pages=20)
    c.dflash_cache_reserve(ints([20, 30]))
    c.dflash_cache_commit(None, ints([20, 30]))
    # 1 is not empty; 2 twice; 3 is a source too; out of range
    c.dflash_cache_fork(ints([0, 0, 1, 3, 0, 9]), ints([1, 2, 2, 3, 7, 4]))
    assert c.dflash_cache_read_status() == 0x40
    assert c.length.cpu().tolist() == [20, 30, 20, 0, 0]
    assert c.refs.cpu().tolist()[:4] == [2, 2, 1, 1]
    c.dflash_cache_trim(ints([5, 3, -1, 0]), seqs=ints([2, 2, 1, 8]))
    assert c.dflash_cache_read_status() == 0x48
    assert c.length.cpu().tolist() == [20, 30, 5, 0, 0] and c.refs.cpu().tolist()[:4] == [2, 1, 1, 1]
    c.dflash_cache_trim(ints([1000, 1000, 1000]))                            # nothing to cut
    assert c.dflash_cache_read_status() == 0 and c.length.cpu().tolist() == [20, 30, 5, 0, 0]


@pytest.mark.parametrize("dtype,hd,ps", [("bf16", 128, 16), ("bf16", 32, 64), ("f32", 64, 32)])
def test_commit_paths(dtype, hd, ps):
    rng = np.random.default_rng(hd)
    n_seq, n_pages = 5, 60
    c = make(n_layer=2, n_head_kv=3, n_head=3, head_dim=hd, page_size=ps, n_pages=n_pages, max_seq=8, max_pages=12, dtype=dtype)
    c.pages.normal_()
    lens, counts = [0, 1, ps - 1, ps, 2 * ps + 3], [1, 70, 40, 33, 90]
    seqs = [7, 0, 3, 5, 1]
    c.table.copy_(ints(np.full((8, 12), -1)))
    perm = rng.permutation(n_pages)
    at = 0
    for q, n, k in zip(seqs, lens, counts):
        h = -(-(n + k) // ps)
        c.table[q, :h] = ints(perm[at:at + h])
        c.length[q] = n
        at += h
    c.refs[ints(perm[:at]).long()] = 1
    paths = [[0], sorted(rng.permutation(70)[:33].tolist()), list(range(40)), [5, 6, 7, 32], []]
    mp = 64
    path = np.full((n_seq, mp), -1, dtype=np.int32)
    for s, p in enumerate(paths):
        path[s, :len(p)] = p
    want, table = c.pages.clone(), c.table.cpu().tolist()
    for q, n, p in zip(seqs, lens, paths):
        for j, a in enumerate(p):
            want[table[q][(n + j) // ps], ..., (n + j) % ps, :] = want[table[q][(n + a) // ps], ..., (n + a) % ps, :]
    c.dflash_cache_commit(ints(path), ints([len(p) for p in paths]), seqs=ints(seqs))
    assert torch.equal(c.pages, want)
    assert [int(c.length[q]) for q in seqs] == [n + len(p) for n, p in zip(lens, paths)]
    assert c.dflash_cache_read_status() == 0


def test_commit_refusals():
    c = make(max_seq=4, max_pages=4, page_size=16, n_pages=10)
    c.pages.normal_()
    c.dflash_cache_reserve(ints([40, 40, 20, 0]))
    c.dflash_cache_commit(None, ints([8, 8, 8, 0]))
    before, table = c.pages.clone(), c.table.clone()

    def refuse(path, n_path, seqs, status, lengths):
        c.dflash_cache_commit(ints(path), ints(n_path), seqs=ints(seqs))
        assert c.dflash_cache_read_status() == status
        assert torch.equal(c.pages, before) and torch.equal(c.table, table)
        assert c.length.cpu().tolist() == lengths

    start = [8, 8, 8, 0]
    refuse([[3, 2]], [2], [0], 0x20, start)                # not ascending
    refuse([[-1, 2]], [2], [0], 0x20, start)
    refuse([[0, 0]], [2], [1], 0x20, start)
    refuse([[0, 30]], [2], [2], 0x10, start)               # slot 38 has no page
    refuse([[0, 2 ** 31 - 1]], [2], [2], 0x10, start)
    refuse([[0, 1]], [3], [0], 0x20, start)                # longer than the array
    refuse([[0, 1]], [-1], [0], 0x8, start)
    refuse([[0, 1], [0, 1]], [0, 2], [0, 0], 0x40, start)  # listed twice
    refuse([[0, 1]], [1], [4], 0x40, start)
    c.dflash_cache_commit(None, ints([100]), seqs=ints([0]))
    assert c.dflash_cache_read_status() == 0x8
    c.dflash_cache_commit(None, ints([25]), seqs=ints([2]))    # 8 + 25 passes the two pages
    assert c.dflash_cache_read_status() == 0x10
    c.dflash_cache_fork(ints([0]), ints([3]))
    refuse_table = c.table.clone()
    c.dflash_cache_commit(ints([[1]]), ints([1]), seqs=ints([3]))   # a shared page
    assert c.dflash_cache_read_status() == 0x10 and torch.equal(c.table, refuse_table) and torch.equal(c.pages, before)


def test_commit_without_a_path_refuses_shared_pages():
    """Slots of a page that others hold too were never written by this sequence."""
    c = make(max_seq=4, max_pages=4, page_size=16, n_pages=10)
    c.dflash_cache_reserve(ints([40]))
    c.dflash_cache_commit(None, ints([20]))
    c.dflash_cache_fork(ints([0]), ints([2]))
    for q in (0, 2):
        c.dflash_cache_commit(None, ints([1]), seqs=ints([q]))
        assert c.dflash_cache_read_status() == 0x10
    c.dflash_cache_commit(None, ints([0]), seqs=ints([2]))        # nothing to keep
    assert c.dflash_cache_read_status() == 0
    assert c.length.cpu().tolist() == [20, 0, 20, 0]
    c.dflash_cache_reserve(ints([5, 5]), seqs=ints([2, 0]))
    c.dflash_cache_commit(None, ints([5, 3]), seqs=ints([2, 0]))
    assert c.dflash_cache_read_status() == 0
    assert c.length.cpu().tolist() == [23, 0, 25, 0]


# ------------------------------------------------------------------ append

def scattered(c, rng, seqs, lens, counts, fill=None):
    """Pages of the sequences anywhere in the pool; the pool holds `fill` or noise."""
    ps = c.cfg.page_size
    if fill is None:
        c.pages.normal_()
    else:
        c.pages.fill_(fill)
    perm, at = rng.permutation(c.cfg.n_pages), 0
    c.table.fill_(-1)
    c.refs.zero_()
    for q, n, k in zip(seqs, lens, counts):
        h = -(-(n + k) // ps)
        assert at + h <= len(perm)
        c.table[q, :h] = ints(perm[at:at + h])
        c.refs[torch.as_tensor(perm[at:at + h]).cuda()] = 1
        c.length[q] = n
        at += h


@pytest.mark.parametrize("dtype,hd,ps,rot,kw", [
    ("bf16", 128, 64, None, {}), ("bf16", 64, 16, 0.5, dict(rope_layout="interleaved")), ("bf16", 32, 16, -8, {}),
    ("f32", 128, 32, None, dict(rope_layout="interleaved")), ("f32", 32, 16, 0, {}),
    ("bf16", 128, 16, None, dict(rope_scaling="yarn", rope_factor=4.0, rope_orig_positions=4096))], ids=str)
@pytest.mark.parametrize("with_q", [True, False])
def test_append(dtype, hd, ps, rot, kw, with_q):
    rng = np.random.default_rng(hd + ps)
    layout = kw.get("rope_layout", "half")
    rd, f, m = rope_setup(hd, layout, rot, kw)
    hq, hkv = 6, 2
    c = make(n_layer=3, n_head=hq, n_head_kv=hkv, head_dim=hd, page_size=ps, n_pages=200, max_seq=7, max_pages=80,
             dtype=dtype, rotary_dim=rd, **kw)
    g = torch.Generator().manual_seed(hd)
    for seqs, lens, counts, deep in (([2], [0], [1], False), ([6, 0, 3, 1], [5, 0, ps, 700], [3, 0, 1, 90], True),
                                     ([4, 5], [100, 1], [500, 333], False)):
        scattered(c, rng, seqs, lens, counts)
        T = sum(counts) + 2
        qkv = normal(g, (T, hq + 2 * hkv, hd), dtype)
        dev = qkv.cuda()
        q, k, v = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]
        trees = [random_parents(rng, n, "random") for n in counts]
        depth = np.concatenate([R.tree_sets(t).sum(1) - 1 if t else np.zeros(0, int) for t in trees] + [[9, 9]])
        before = c.pages.clone()
        q_out = torch.full((T, hq, hd), 3.0, dtype=DT[dtype], device="cuda")
        c.dflash_cache_append(1, starts(counts), k, v, depth=ints(depth) if deep else None,
                              q=q if with_q else None, q_out=q_out if with_q else None, seqs=ints(seqs))
        want, table, r = before.clone(), c.table.cpu().tolist(), 0
        got = c.pages.clone()
        for s, (qq, n, cnt) in enumerate(zip(seqs, lens, counts)):
            if not cnt:
                continue
            pos = n + (depth[r:r + cnt] if deep else np.arange(cnt))
            wk, size = R.rope(np64(qkv[r:r + cnt, hq:hq + hkv]), pos, layout, rd, f, m)
            at = torch.as_tensor([n + i for i in range(cnt)])
            page = torch.as_tensor([table[qq][i] for i in (at // ps).tolist()])
            stored = got[page.cuda(), 1, 0, :, (at % ps).cuda()]          # [cnt][hkv][hd]
            check(np64(stored), wk, rope_tol(size, wk, dtype), "keys")
            want[page.cuda(), 1, 0, :, (at % ps).cuda()] = stored
            want[page.cuda(), 1, 1, :, (at % ps).cuda()] = v[r:r + cnt]
            if with_q:
                wq, size = R.rope(np64(qkv[r:r + cnt, :hq]), pos, layout, rd, f, m)
                check(np64(q_out[r:r + cnt]), wq, rope_tol(size, wq, dtype), "queries")
            r += cnt
        assert torch.equal(got, want)                                      # and no other slot
        assert (q_out[r:] == 3.0).all()
        assert torch.equal(dev.cpu(), qkv)
        assert c.dflash_cache_read_status() == 0


def test_append_thousands_of_heads():
    """Rows of so many items that a block's numbers leave the range of its quotients."""
    hq, hkv, hd, ps, T = 4096, 512, 128, 16, 1300
    c = make(n_layer=1, n_head=hq, n_head_kv=hkv, head_dim=hd, page_size=ps, n_pages=90, max_seq=2, max_pages=90)
    rng = np.random.default_rng(1)
    scattered(c, rng, [1], [0], [T])
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn(T, hq + 2 * hkv, hd, generator=g, device="cuda", dtype=torch.bfloat16)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    q_out = torch.full((T, hq, hd), 3.0, dtype=torch.bfloat16, device="cuda")
    c.dflash_cache_append(0, starts([T]), k, v, q=q, q_out=q_out, seqs=ints([1]))
    at = torch.arange(T, device="cuda")
    page = c.table[1].long()[at // ps]
    assert torch.equal(c.pages[page, 0, 1, :, at % ps], v)
    rd, f, m = rope_setup(hd, "half", None, {})
    rows = [0, 1, 2, 3, 617, 618, T - 1]
    keys = c.pages[page, 0, 0, :, at % ps]
    for src, got in ((k, keys), (q, q_out)):
        want, size = R.rope(np64(src[rows]), np.asarray(rows), "half", rd, f, m)
        check(np64(got[rows]), want, rope_tol(size, want, "bf16"), "rows")
    assert c.dflash_cache_read_status() == 0


@pytest.mark.parametrize("dtype,hq,hkv,hd,rot,T", [
    # rows of more items than a block of one row takes in one step
    ("bf16", 64, 8, 128, None, 487), ("bf16", 64, 8, 128, None, 512), ("bf16", 64, 8, 128, None, 608),
    ("bf16", 64, 8, 128, None, 609), ("f32", 32, 8, 128, None, 406), ("f32", 32, 8, 128, None, 512),
    ("f32", 32, 8, 128, None, 608), ("bf16", 32, 8, 128, -8, 450), ("bf16", 4096, 1024, 128, None, 40),
    # either side of where a thread takes more items, a block more rows, the grid another wave
    ("bf16", 32, 8, 128, None, 810), ("bf16", 32, 8, 128, None, 811), ("bf16", 32, 8, 128, None, 1217),
    ("f32", 32, 8, 128, None, 405), ("bf16", 4, 2, 64, None, 9728), ("bf16", 4, 2, 64, None, 9729),
    ("f32", 4, 2, 32, 0.5, 9729)], ids=str)
def test_append_every_item_of_every_row(dtype, hq, hkv, hd, rot, T):
    """Nothing of a row is left out, whatever the shape of the launch."""
    ps = 64
    rd, f, m = rope_setup(hd, "half", rot, {})
    n_pages = -(-T // ps) + 1
    c = make(n_layer=1, n_head=hq, n_head_kv=hkv, head_dim=hd, page_size=ps, n_pages=n_pages, max_seq=2, max_pages=n_pages,
             dtype=dtype, rotary_dim=rd)
    c.pages.fill_(float("nan"))
    g = torch.Generator(device="cuda").manual_seed(T)
    qkv = torch.randn(T, hq + 2 * hkv, hd, generator=g, device="cuda").to(DT[dtype])
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    q_out = torch.full((T, hq, hd), float("nan"), dtype=DT[dtype], device="cuda")
    c.dflash_cache_reserve(ints([T]), seqs=ints([1]))
    c.dflash_cache_append(0, starts([T]), k, v, q=q, q_out=q_out, seqs=ints([1]))
    at = torch.arange(T, device="cuda")
    page = c.table[1].long()[at // ps]
    assert torch.equal(c.pages[page, 0, 1, :, at % ps], v)
    keys = c.pages[page, 0, 0, :, at % ps]
    assert not torch.isnan(keys).any() and not torch.isnan(q_out).any()
    rows = sorted({*range(0, T, max(1, T // 60)), T - 1})
    for src, got in ((k, keys), (q, q_out)):
        want, size = R.rope(np64(src[rows]), np.asarray(rows), "half", rd, f, m)
        check(np64(got[rows]), want, rope_tol(size, want, dtype), "rows")
    assert c.dflash_cache_read_status() == 0


def test_append_faults_write_nothing_else():
    rng = np.random.default_rng(0)
    c = make(n_layer=1, n_head=2, n_head_kv=1, head_dim=32, page_size=16, n_pages=12, max_seq=4, max_pages=3)
    kv = torch.ones(8, 1, 32, dtype=torch.bfloat16, device="cuda")

    def run(row_start, seqs, status, written, depth=None):
        c.pages.zero_()
        c.dflash_cache_append(0, ints(row_start), kv, kv, seqs=ints(seqs), depth=None if depth is None else ints(depth))
        assert c.dflash_cache_read_status() == status
        assert int((c.pages[:, 0, 1] != 0).sum()) == 32 * written

    scattered(c, rng, [0, 1, 2], [10, 20, 5], [8, 8, 8], fill=0)
    run([0, 4, 8], [0, 1], 0, 8)
    run([0, 4, 8], [0, 0], 0x40, 4)                       # listed twice
    run([0, 4, 8], [0, 4], 0x40, 4)                       # out of range
    run([0, 4, 9], [0, 1], 0x8, 4)                        # a range that passes T
    run([0, 4, 2], [0, 1], 0x8, 2)                        # not ascending: a row's range is that of its last start
    run([0, 4, 8], [0, 3], 0x10, 4)                       # sequence 3 has no pages
    run([0, 8], [2], 0x2, 7, depth=[0, 1, 2, -6, 3, 4, 5, 6])
    c.length[1] = 44                                      # 44 .. 51 passes max_pages
    run([0, 8], [1], 0x10, 0)
    c.length[1] = -5
    run([0, 8], [1], 0x8, 0)
    c.length[1] = 20
    c.table[1, 1] = 12                                    # no such page
    run([0, 8], [1], 0x10, 0)
    c.dflash_cache_fork(ints([0]), ints([3]))
    run([0, 8], [0], 0x10, 2)                             # slots 10..15 share a page, 16 and 17 do not
    run([0], [], 0, 0)


# ------------------------------------------------------------------ attention

def attend_case(c, rng, g, seqs, lens, counts, mask_kind, dtype, max_tree=None, tail=2, with_lse=True, layer=0,
                q_scale=1.0, poison=True, ramp=0.0):
    cfg = c.cfg
    ps, hd, hq = cfg.page_size, cfg.head_dim, cfg.n_head
    scattered(c, rng, seqs, lens, counts, fill=float("nan") if poison else None)
    T = sum(counts) + tail
    fused = normal(g, (T, hq + 3, hd), dtype) * q_scale
    q = fused.cuda()[:, 1:1 + hq]
    words = max(1, -(-max(counts + [1]) // 32))
    mask = np.zeros((T, words), dtype=np.int32)
    sets, r = [], 0
    table = c.table.cpu().tolist()
    kv = []
    for qq, n, cnt in zip(seqs, lens, counts):
        if mask_kind == "tree":
            m = R.tree_sets(random_parents(rng, cnt, "forest"))
        elif mask_kind == "bits":        # any bits, empty rows among them
            m = rng.random((cnt, cnt)) < 0.3
            m[rng.random(cnt) < 0.4] = False
        else:
            m = np.tril(np.ones((cnt, cnt), dtype=bool))
        if mask_kind != "chain":
            mask[r:r + cnt] = R.words_of(m, words)
        sets.append(m)
        data = normal(g, (2, n + cnt, cfg.n_head_kv, hd), dtype)
        if ramp:      # keys that grow (ramp > 0) or shrink along the sequence
            p = torch.arange(n + cnt, dtype=torch.float32)
            data[0] = (data[0].float() * (1 + abs(ramp) * (p if ramp > 0 else n + cnt - p))[:, None, None]).to(DT[dtype])
        kv.append(np64(data))
        for i in range(-(-(n + cnt) // ps)):
            part = data[:, i * ps:(i + 1) * ps].transpose(1, 2).cuda()
            c.pages[table[qq][i], layer, :, :, :part.shape[2]] = part
        r += cnt
    if mask_kind == "bits" and words * 32 > max(counts):
        # the last bit of every word too: behind the last node it means nothing
        mask |= np.int32(-2 ** 31)
        r = 0
        for i, cnt in enumerate(counts):
            sets[i] = np.unpackbits(mask[r:r + cnt].view(np.uint8), axis=1, bitorder="little")[:, :cnt].astype(bool)
            r += cnt
    out = torch.full((T, hq + 1, hd), 5.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((T, hq), 5.0, dtype=torch.float32, device="cuda") if with_lse else None
    c.dflash_tree_attend(layer, starts(counts), max_tree or max(counts + [1]), q, out[:, :hq],
                         mask=None if mask_kind == "chain" else ints(mask), lse=lse, seqs=ints(seqs))
    r = 0
    scale = cfg.attn_scale or hd ** -0.5
    for n, cnt, m, (k, v) in zip(lens, counts, sets, kv):
        sees = np.concatenate([np.ones((cnt, n), dtype=bool), m], 1)
        o, ls, size, big = R.attend(np64(fused[r:r + cnt, 1:1 + hq]), k, v, sees, scale)
        tol, tol_l = R.attend_bounds(o, size, big, n + cnt, hd, dtype)
        check(np64(out[r:r + cnt, :hq]), o, tol, f"length {n}, {cnt} rows")
        if with_lse:
            got = np64(lse[r:r + cnt])
            empty = np.isinf(ls)
            assert (got[empty] == -np.inf).all()
            check(got[~empty], ls[~empty], tol_l[~empty], "lse")
        r += cnt
    assert (out[r:] == 5.0).all() and (out[:, hq:] == 5.0).all()
    if with_lse:
        assert (lse[r:] == 5.0).all()
    assert c.dflash_cache_read_status() == 0
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd,hq,hkv,ps", [(64, 4, 2, 16), (128, 8, 1, 64), (128, 8, 2, 128), (32, 3, 3, 32),
                                          (64, 6, 2, 256), (128, 4, 4, 16)], ids=str)
@pytest.mark.parametrize("mask_kind", ["chain", "tree", "bits"])
def test_attend(dtype, hd, hq, hkv, ps, mask_kind):
    rng = np.random.default_rng(hd + hq + ps)
    g = torch.Generator().manual_seed(hd * hq + ps)
    c = make(n_layer=2, n_head=hq, n_head_kv=hkv, head_dim=hd, page_size=ps, n_pages=160, max_seq=9, max_pages=64, dtype=dtype)
    attend_case(c, rng, g, [4], [0], [1], mask_kind, dtype, layer=1)
    attend_case(c, rng, g, [8, 2, 0, 5, 1], [0, 1, 63, 64, 257], [3, 0, 1, 33, 17], mask_kind, dtype)
    attend_case(c, rng, g, [1, 3], [130, 5], [64, 65], mask_kind, dtype, with_lse=False, layer=1)
    attend_case(c, rng, g, [7, 6], [0, 300], [200, 5], mask_kind, dtype, max_tree=224 if mask_kind != "chain" else 5000, tail=0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_long_and_many(dtype):
    """Work split along the slots of one sequence, and over many short ones."""
    rng = np.random.default_rng(9)
    g = torch.Generator().manual_seed(9)
    c = make(n_head=4, n_head_kv=1, head_dim=128, page_size=64, n_pages=600, max_seq=64, max_pages=400, dtype=dtype)
    attend_case(c, rng, g, [11], [20011], [1], "chain", dtype)
    attend_case(c, rng, g, [3, 1], [15000, 77], [9, 1], "tree", dtype)
    attend_case(c, rng, g, rng.permutation(64).tolist(), rng.integers(0, 400, 64).tolist(),
                rng.integers(0, 4, 64).tolist(), "tree", dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_most_entries(dtype):
    """As many entries as a call may have, one of them with tall tiles."""
    rng = np.random.default_rng(10)
    g = torch.Generator().manual_seed(10)
    n = 1024
    c = make(n_head=4, n_head_kv=1, head_dim=128, page_size=16, n_pages=2200, max_seq=n, max_pages=8, dtype=dtype)
    counts = rng.integers(0, 4, n)
    lens = rng.integers(0, 26, n)
    counts[700], lens[700] = 70, 20
    attend_case(c, rng, g, rng.permutation(n).tolist(), lens.tolist(), counts.tolist(), "tree", dtype)


@pytest.mark.parametrize("hd,n", [(128, 52), (128, 53), (128, 1024), (64, 60)])
@pytest.mark.parametrize("mask_kind", ["tree", "chain"])
def test_attend_many_entries_of_many_chunks(hd, n, mask_kind):
    """Entry lists that leave the kernel few ring stages (3 with heads of 128 and 53 entries),
    tiles of more and of fewer than 128 rows, many chunks each."""
    rng = np.random.default_rng(n + hd)
    g = torch.Generator().manual_seed(n + hd)
    long = min(n, 60)
    counts, lens = rng.integers(0, 3, n), rng.integers(0, 40, n)
    at = rng.permutation(n)[:long]
    lens[at] = rng.integers(1500, 2700, long)
    counts[at] = rng.choice([1, 7, 20, 33, 40, 64], long)
    counts[at[0]], lens[at[0]] = 64, 6000
    counts[at[1]], lens[at[1]] = 5, 9000
    c = make(n_head=4, n_head_kv=1, head_dim=hd, page_size=64, n_pages=5000, max_seq=1024, max_pages=200)
    attend_case(c, rng, g, rng.permutation(1024)[:n].tolist(), lens.tolist(), counts.tolist(), mask_kind, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd,hq,hkv", [(128, 5, 1), (64, 40, 1), (128, 14, 2), (64, 300, 1), (32, 300, 1)], ids=str)
def test_attend_group_sizes(dtype, hd, hq, hkv):
    """Groups of query heads that no tile holds a whole number of, or that are larger than a tile."""
    rng = np.random.default_rng(hq)
    g = torch.Generator().manual_seed(hq)
    c = make(n_head=hq, n_head_kv=hkv, head_dim=hd, page_size=32, n_pages=60, max_seq=4, max_pages=16, dtype=dtype)
    attend_case(c, rng, g, [2, 0, 3], [200, 0, 31], [33, 60, 1], "tree", dtype)
    attend_case(c, rng, g, [1], [129], [52], "chain", dtype, with_lse=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_large_scores(dtype):
    """Scores far outside exp's range, of both signs, and scales of their own."""
    rng = np.random.default_rng(2)
    g = torch.Generator().manual_seed(2)
    c = make(n_head=2, n_head_kv=1, head_dim=64, page_size=16, n_pages=100, max_seq=2, max_pages=60, dtype=dtype, attn_scale=1.5)
    attend_case(c, rng, g, [0, 1], [300, 40], [20, 3], "tree", dtype, q_scale=16.0)
    c = make(n_head=2, n_head_kv=1, head_dim=64, page_size=16, n_pages=100, max_seq=2, max_pages=60, dtype=dtype, attn_scale=2.0 ** -20)
    attend_case(c, rng, g, [0, 1], [300, 40], [20, 3], "tree", dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("ramp", [0.1, -0.1])
def test_attend_scores_that_grow_along_the_sequence(dtype, hd, ramp):
    """The largest score moves by hundreds from chunk to chunk, up or down: the weights'
    reference has to follow, with what was summed before it."""
    rng = np.random.default_rng(hd)
    g = torch.Generator().manual_seed(hd)
    c = make(n_head=8, n_head_kv=2, head_dim=hd, page_size=64, n_pages=100, max_seq=4, max_pages=60, dtype=dtype)
    attend_case(c, rng, g, [0, 1, 2], [1500, 40, 700], [20, 3, 70], "tree", dtype, ramp=ramp)
    attend_case(c, rng, g, [3], [0], [300], "chain", dtype, ramp=ramp)
    attend_case(c, rng, g, [1, 0], [900, 2000], [1, 9], "tree", dtype, ramp=ramp)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("top,rows", [(56, 1), (56, 70), (64, 70)])
def test_attend_large_values(dtype, hd, top, rows):
    """Values of one sign, up to 2^56 (and, in tiles of few parts, 2^64), under scores that are
    all far above zero, as far as a reference may lag: 64 weights come to 2^59.4.  A sum that
    went on from there would reach 2^65 with the 66 halves of a chunk that a stream has here,
    and with values of 2^64 leave fp32; one that stays below 2^60 is at most 2^124, two streams
    and four parts of a tile 2^127."""
    g = torch.Generator().manual_seed(hd)
    hkv, n = 160, 8400
    c = make(n_head=hkv, n_head_kv=hkv, head_dim=hd, page_size=256, n_pages=36, max_seq=1, max_pages=36, dtype=dtype,
             attn_scale=1.0)
    scattered(c, np.random.default_rng(hd), [0], [n], [rows], fill=float("nan"))
    slots = n + rows
    key = torch.zeros(slots, hd)
    key[:, 0] = 1.0
    data = torch.stack([key, (1 + torch.rand(slots, hd, generator=g)) * 2.0 ** (top - 1)]).to(DT[dtype])
    table = c.table.cpu().tolist()
    for i in range(-(-slots // 256)):
        part = data[:, None, i * 256:(i + 1) * 256].cuda()
        c.pages[table[0][i], 0, :, :, :part.shape[2]] = part
    q = torch.zeros(rows, hkv, hd, dtype=DT[dtype])
    q[..., 0] = 37.0                                      # 53.4 in powers of two
    out, lse = torch.empty_like(q, device="cuda"), torch.empty(rows, hkv, device="cuda")
    c.dflash_tree_attend(0, starts([rows]), rows, q.cuda(), out, lse=lse)
    sees = np.concatenate([np.ones((rows, n), bool), np.tril(np.ones((rows, rows), bool))], 1)
    kv = np64(data[:, :, None])
    o, ls, size, big = R.attend(np64(q[:, :1]), kv[0], kv[1], sees, 1.0)
    tol, tol_l = R.attend_bounds(o, size, big, slots, hd, dtype)
    check(np64(out), np.broadcast_to(o, out.shape), np.broadcast_to(tol, out.shape))
    check(np64(lse), np.broadcast_to(ls, lse.shape), np.broadcast_to(tol_l, lse.shape), "lse")
    assert c.dflash_cache_read_status() == 0


def test_attend_f32_keeps_two_blocks_per_sm():
    """The same work in calls of more and more entries (all but one without rows): where the
    entries' descriptions left room for one block per SM only, a call took half as long again."""
    c = make(n_head=16, n_head_kv=8, head_dim=128, page_size=64, n_pages=1100, max_seq=4, max_pages=1024, dtype="f32")
    c.pages.normal_()
    c.table[0] = torch.arange(1024, device="cuda")
    c.length[0] = 60000
    q = torch.randn(8, 16, 128, device="cuda")
    out = torch.empty_like(q)

    def time(n):
        start, seqs = starts([8] + [0] * (n - 1)), ints([0] * n)
        ts = []
        for _ in range(12):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            c.dflash_tree_attend(0, start, 8, q, out, seqs=seqs)
            b.record()
            b.synchronize()
            ts.append(a.elapsed_time(b))
        return min(ts)

    few = time(150)
    for n in range(200, 260, 5):
        assert time(n) < 1.4 * few, n
    assert c.dflash_cache_read_status() == 0


def test_attend_faults():
    D = _D()
    rng = np.random.default_rng(1)
    c = make(n_head=2, n_head_kv=1, head_dim=64, page_size=16, n_pages=12, max_seq=4, max_pages=4)
    q = torch.randn(8, 2, 64, device="cuda").bfloat16()
    scattered(c, rng, [0, 1], [10, 20], [4, 4])

    def run(row_start, seqs, status, changed, max_tree=8):
        out = torch.full_like(q, 9.0)
        c.dflash_tree_attend(0, ints(row_start), max_tree, q, out, seqs=ints(seqs))
        assert c.dflash_cache_read_status() == status
        got = (out != 9.0).flatten(1).any(1).nonzero().flatten().tolist()
        assert got == changed

    run([0, 4, 8], [0, 1], 0, list(range(8)))
    run([0, 4, 8], [1, 1], 0, list(range(8)))             # two trees over one sequence
    run([0, 4, 9], [0, 1], 0x8, [0, 1, 2, 3])
    run([0, 4, 8], [0, 4], 0x40, [0, 1, 2, 3])
    run([0, 5, 8], [0, 1], 0x8, [5, 6, 7], max_tree=4)    # more nodes than announced
    c.length[1] = 61                                      # 61 + 4 passes max_pages
    run([0, 4, 8], [0, 1], 0x8, [0, 1, 2, 3])
    c.length[1] = -1
    run([0, 4, 8], [0, 1], 0x8, [0, 1, 2, 3])
    c.length[1] = 20
    for bad in (-1, 12, 2 ** 31 - 1):
        c.table[1, 0] = bad
        out = torch.empty_like(q)
        c.dflash_tree_attend(0, starts([4, 4]), 4, q, out, seqs=ints([0, 1]))
        assert c.dflash_cache_read_status() == 0x10
    run([0], [], 0, [])
    with pytest.raises(D.DFlashError):
        c.dflash_tree_attend(1, starts([8]), 8, q, torch.empty_like(q))
    with pytest.raises(D.DFlashError):
        c.dflash_tree_attend(0, starts([8]), 0, q, torch.empty_like(q))
    with pytest.raises(D.DFlashError):
        c.dflash_tree_attend(0, starts([8]), 33, q, torch.empty_like(q), mask=ints([[1]] * 8))


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_verification_turns_equal_a_plain_model(dtype):
    """Prompt, then turns of reserve, mask, per layer append and attend, accept and commit
    on forked sequences: every layer's attention output equals that of a plain cache of the
    accepted tokens, computed from scratch."""
    rng = np.random.default_rng(4)
    hq, hkv, hd, L, ps = 4, 2, 32, 2, 16
    c = make(n_layer=L, n_head=hq, n_head_kv=hkv, head_dim=hd, page_size=ps, n_pages=80, max_seq=4, max_pages=16, dtype=dtype)
    f, m = R.rope_freqs(hd)
    vocab = 6
    # a token's q, k, v rows by layer
    emb = normal(torch.Generator().manual_seed(1), (L, vocab, hq + 2 * hkv, hd), dtype)
    dev = emb.cuda()

    def step(seqs, tokens, trees, depths):
        counts = [len(t) for t in tokens]
        start, flat = starts(counts), torch.as_tensor(np.concatenate(tokens)).cuda()
        T = sum(counts)
        words = max(1, -(-max(counts) // 32))
        mask = torch.zeros(T, words, dtype=torch.int32, device="cuda")
        depth = torch.zeros(T, dtype=torch.int32, device="cuda")
        c.dflash_cache_reserve(ints(counts), seqs=ints(seqs))
        c.dflash_tree_mask(start, ints(np.concatenate(trees)), mask, depth)
        assert depth.cpu().tolist() == np.concatenate(depths).tolist()
        outs = []
        for layer in range(L):
            rows = dev[layer][flat]
            q_rot, out = (torch.empty(T, hq, hd, dtype=DT[dtype], device="cuda") for _ in range(2))
            c.dflash_cache_append(layer, start, rows[:, hq:hq + hkv], rows[:, hq + hkv:], depth=depth, q=rows[:, :hq],
                                  q_out=q_rot, seqs=ints(seqs))
            c.dflash_tree_attend(layer, start, max(counts), q_rot, out, mask=mask, seqs=ints(seqs))
            outs.append(np64(out))
        return outs, start

    def stored(x):     # what the pages hold: rounded once
        return np64(torch.as_tensor(x).to(DT[dtype]))

    def plain(history, tokens, tree, layer):
        e = np64(emb[layer])
        toks = np.array(history + list(tokens), dtype=int)
        sets = R.tree_sets(tree)
        pos = np.concatenate([np.arange(len(history)), len(history) + sets.sum(1) - 1]).astype(int)
        k = stored(R.rope(e[toks][:, hq:hq + hkv], pos, "half", hd, f, m)[0])
        q = stored(R.rope(e[np.array(tokens)][:, :hq], pos[len(history):], "half", hd, f, m)[0])
        sees = np.concatenate([np.ones((len(tokens), len(history)), bool), sets], 1)
        return R.attend(q, k, e[toks][:, hq + hkv:], sees, hd ** -0.5)

    def compare(outs, seqs, tokens, trees, history):
        r = 0
        for qq, t, tr in zip(seqs, tokens, trees):
            for layer in range(L):
                o, _, size, big = plain(history[qq], t, tr, layer)
                tol, _ = R.attend_bounds(o, size, big, len(history[qq]) + len(t), hd, dtype)
                # a rotated key or query may round to the other neighbour: a step of the type in one
                # operand moves a score by up to 2^-7 (2^-23) of |q| |k|, on either side
                tol = tol + size * 4 * (2 * HALF[dtype] + 1e-6) * big[..., None]
                check(outs[layer][r:r + len(t)], o, tol, f"sequence {qq}")
            r += len(t)

    history = {q: [] for q in range(4)}
    prompts = [rng.integers(0, vocab, 37).tolist(), rng.integers(0, vocab, 5).tolist()]
    chains = [[i - 1 for i in range(len(p))] for p in prompts]
    outs, _ = step([0, 2], prompts, chains, [np.arange(37), np.arange(5)])
    compare(outs, [0, 2], prompts, chains, history)
    c.dflash_cache_commit(None, ints([37, 5]), seqs=ints([0, 2]))
    history[0], history[2] = list(prompts[0]), list(prompts[1])
    c.dflash_cache_fork(ints([0, 2]), ints([1, 3]))
    history[1], history[3] = list(history[0]), list(history[2])
    for turn in range(4):
        seqs = rng.permutation(4)[:3].tolist()
        trees = [random_parents(rng, n, "random") for n in (20, 9, 41)]
        tokens = [rng.integers(0, vocab, len(t)).tolist() for t in trees]
        outs, start = step(seqs, tokens, trees, [R.tree_sets(t).sum(1) - 1 for t in trees])
        compare(outs, seqs, tokens, trees, history)
        flat_tree, flat_tok = np.concatenate(trees), np.concatenate(tokens)
        targets = rng.integers(0, vocab, len(flat_tok))
        path = torch.zeros(3, 6, dtype=torch.int32, device="cuda")
        n_path, id_last = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))
        c.dflash_tree_accept(start, ints(flat_tree), ints(flat_tok), ints(targets), path, n_path, id_last)
        c.dflash_cache_commit(path, n_path, seqs=ints(seqs))
        r = 0
        for s, (qq, t, tok) in enumerate(zip(seqs, trees, tokens)):
            want, last = R.accept(t, tok, targets[r:r + len(t)].tolist(), 6)
            assert path[s].tolist()[:len(want)] == want and int(id_last[s]) == last
            history[qq] += [tok[i] for i in want]
            r += len(t)
        assert [int(c.length[q]) for q in range(4)] == [len(history[q]) for q in range(4)]
        # reserved pages behind the accepted tokens go back
        c.dflash_cache_trim(ints([len(history[q]) for q in range(4)]))
        assert c.dflash_cache_read_status() == 0
    c.dflash_cache_trim(ints([0] * 4))
    assert int(c.refs.abs().sum()) == 0


def test_captured_turn_replays_with_new_lengths():
    """One captured graph of a turn, replayed as lengths, trees and pages change, equals the
    same calls made eagerly on a second handle, bit for bit."""
    rng = np.random.default_rng(6)
    g = torch.Generator().manual_seed(6)
    n, tree, hq, hkv, hd = 3, 24, 4, 1, 128
    T = n * tree
    rows = [torch.empty(T, hq + 2 * hkv, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    parents, tokens, targets = (torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(3))
    start, ask = starts([tree] * n), ints([tree] * n)
    seqs = ints([2, 0, 1])
    sides = []
    for _ in range(2):
        c = make(n_layer=2, n_head=hq, n_head_kv=hkv, head_dim=hd, page_size=16, n_pages=200, max_seq=3, max_pages=60)
        c.pages.zero_()
        sides.append(dict(c=c, mask=torch.zeros(T, 1, dtype=torch.int32, device="cuda"),
                          depth=torch.zeros(T, dtype=torch.int32, device="cuda"),
                          q=torch.zeros(T, hq, hd, dtype=torch.bfloat16, device="cuda"),
                          out=torch.zeros(2, T, hq, hd, dtype=torch.bfloat16, device="cuda"),
                          lse=torch.zeros(2, T, hq, device="cuda"),
                          path=torch.zeros(n, 8, dtype=torch.int32, device="cuda"),
                          n_path=torch.zeros(n, dtype=torch.int32, device="cuda"),
                          id_last=torch.zeros(n, dtype=torch.int32, device="cuda")))

    def turn(s):
        c = s["c"]
        c.dflash_cache_reserve(ask, seqs=seqs)
        c.dflash_tree_mask(start, parents, s["mask"], s["depth"])
        for layer in range(2):
            r = rows[layer]
            c.dflash_cache_append(layer, start, r[:, hq:hq + hkv], r[:, hq + hkv:], depth=s["depth"], q=r[:, :hq],
                                  q_out=s["q"], seqs=seqs)
            c.dflash_tree_attend(layer, start, tree, s["q"], s["out"][layer], mask=s["mask"], lse=s["lse"][layer], seqs=seqs)
        c.dflash_tree_accept(start, parents, tokens, targets, s["path"], s["n_path"], s["id_last"])
        c.dflash_cache_commit(s["path"], s["n_path"], seqs=seqs)

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        turn(sides[0])
    for it in range(30):
        for r in rows:
            r.copy_(normal(g, tuple(r.shape), "bf16"))
        parents.copy_(ints(np.concatenate([random_parents(rng, tree, "random") for _ in range(n)])))
        tokens.copy_(ints(rng.integers(0, 2, T)))
        targets.copy_(ints(rng.integers(0, 2, T)))
        graph.replay()
        turn(sides[1])
        a, b = sides
        for k in ("mask", "depth", "q", "out", "lse", "path", "n_path", "id_last"):
            assert torch.equal(a[k], b[k]), (it, k)
        for k in ("pages", "table", "length", "refs"):
            assert torch.equal(getattr(a["c"], k), getattr(b["c"], k)), (it, k)
    assert [s["c"].dflash_cache_read_status() for s in sides] == [0, 0]
    assert int(sides[0]["c"].length.min()) > 40


def test_other_streams_and_two_handles():
    """Calls on a stream of their own, two handles at the same time on two streams."""
    rng = np.random.default_rng(8)
    streams = [torch.cuda.Stream() for _ in range(2)]
    caches = [make(n_head=8, n_head_kv=2, head_dim=128, page_size=64, n_pages=80, max_seq=2, max_pages=64) for _ in range(2)]
    q = [torch.randn(40, 8, 128, device="cuda").bfloat16() for _ in range(2)]
    alone, both = [], []
    for c in caches:
        scattered(c, rng, [0, 1], [2000, 900], [20, 20])
    for c, x in zip(caches, q):
        out = torch.zeros_like(x)
        c.dflash_tree_attend(0, starts([20, 20]), 20, x, out)
        alone.append(out)
    start = starts([20, 20])
    torch.cuda.synchronize()
    outs = [[torch.zeros_like(x) for _ in range(20)] for x in q]
    for i in range(20):
        for k in range(2):
            caches[k].dflash_tree_attend(0, start, 20, q[k], outs[k][i], stream=streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        for o in outs[k]:
            assert torch.equal(o, alone[k])


def test_create_waits_for_what_its_memory_was_used_for():
    """A cache made on a stream of its own gets blocks that this stream freed, and that work
    in flight on it still writes: its state is that of an empty cache all the same."""
    D = _D()
    kw = dict(n_layer=1, n_head=4, n_head_kv=2, head_dim=64, page_size=16, n_pages=3000, max_seq=500, max_pages=1500)
    sizes = D.cache_workspace_size(D.make_cache_config(D.CacheConfig(**kw)))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        old = [torch.empty(n + 256, dtype=torch.uint8, device="cuda") for n in sizes]
        at = {t.data_ptr() for t in old}
        torch.cuda._sleep(200_000_000)
        for t in old:
            t.fill_(1)
        del old, t
        c = make(**kw)
    assert c.state_mem.data_ptr() in at and c.scratch.data_ptr() in at
    assert (c.table == -1).all() and not c.length.any() and not c.refs.any()
    assert c.dflash_cache_read_status() == 0


@pytest.mark.parametrize("explicit", [True, False])
def test_dropped_with_work_in_flight(explicit):
    """A cache that goes while a call on another stream than its own waits to run: its memory
    is not handed out before that call is done."""
    n = 64
    c = make(n_layer=1, n_head=4, n_head_kv=2, head_dim=64, page_size=256, n_pages=200, max_seq=2, max_pages=100)
    c.dflash_cache_reserve(ints([n]))
    start, kv = starts([n]), torch.ones(n, 2, 64, dtype=torch.bfloat16, device="cuda")
    size = c.page_mem.numel()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        if not explicit:
            c.dflash_cache_append(0, start, kv, kv)
    if explicit:
        c.dflash_cache_append(0, start, kv, kv, stream=side)
    del c
    new = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert not any(t.any() for t in new)


def test_offsets_past_32_bits():
    """Pages beyond 4 GB: append, attend and commit at the end of a large pool."""
    hd, ps = 128, 256
    n_pages = (5 << 30) // (2 * 8 * ps * hd * 2)
    c = make(n_layer=1, n_head=8, n_head_kv=8, head_dim=hd, page_size=ps, n_pages=n_pages, max_seq=2, max_pages=8)
    assert c.pages.numel() * 2 > 2 ** 32
    rng, g = np.random.default_rng(0), torch.Generator().manual_seed(0)
    c.table[1, :2] = ints([n_pages - 1, n_pages - 2])
    c.refs[n_pages - 2:] = 1
    c.length[1] = 250
    c.pages[n_pages - 2:].normal_()
    rows = normal(g, (12, 24, hd), "bf16").cuda()
    q = torch.empty(12, 8, hd, dtype=torch.bfloat16, device="cuda")
    c.dflash_cache_append(0, starts([12]), rows[:, 8:16], rows[:, 16:], q=rows[:, :8], q_out=q, seqs=ints([1]))
    out = torch.empty_like(q)
    c.dflash_tree_attend(0, starts([12]), 12, q, out, seqs=ints([1]))
    last = np64(c.pages[n_pages - 2:, 0])                  # [page][k, v][head][slot][dim]
    k, v = (np.concatenate([last[1, i], last[0, i]], 1)[:, :262].transpose(1, 0, 2) for i in (0, 1))
    sees = np.concatenate([np.ones((12, 250), bool), np.tril(np.ones((12, 12), bool))], 1)
    o, _, size, big = R.attend(np64(q), k, v, sees, hd ** -0.5)
    check(np64(out), o, R.attend_bounds(o, size, big, 262, hd, "bf16")[0])
    np.testing.assert_array_equal(v[250:262], np64(rows[:, 16:]))
    c.dflash_cache_commit(ints([[0, 7, 11]]), ints([3]), seqs=ints([1]))
    now = np64(c.pages[n_pages - 1, 0, 1, :, 250:253]).transpose(1, 0, 2)
    np.testing.assert_array_equal(now, np64(rows[[0, 7, 11], 16:]))
    assert c.dflash_cache_read_status() == 0


def test_areas_on_the_host_are_refused():
    import ctypes as C
    D = _D()
    cfg = D.make_cache_config(D.CacheConfig(n_layer=1, n_head=2, n_head_kv=1, head_dim=64, page_size=16, n_pages=4,
                                            max_seq=2, max_pages=4))
    sizes = D.cache_workspace_size(cfg)
    good = [torch.empty(n + 256, dtype=torch.uint8, device="cuda") for n in sizes]
    for bad in range(3):
        areas = list(good)
        areas[bad] = torch.empty(sizes[bad] + 256, dtype=torch.uint8)
        h = C.c_void_p()
        rc = D.LIB.dflash_cache_create(C.byref(cfg), *(D.Drafter._aligned(a) for a in areas), C.byref(h))
        assert rc != 0 and not h.value
