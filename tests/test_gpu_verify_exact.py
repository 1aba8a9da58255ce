"""Sampled verification where a few bits decide: scores of any size, and what is left after rejections."""
import numpy as np
import pytest
import torch

import verify_reference as V
from test_gpu_cache import DT, ints, make, np64, starts
from test_gpu_verify import CLOSE, exponential, padded

pytestmark = pytest.mark.gpu

def below(x, steps):
    """The f32 or bf16 number `steps` steps below x (above 0)."""
    if x.dtype == torch.float32:
        return (x.view(torch.int32) - steps).view(torch.float32)
    return (x.view(torch.int16) - steps).view(torch.bfloat16)


def check(c, trees, tokens, target, temps, uniform, noise, draft=None, rows_d=None, temps_d=None, pad=0, max_path=4, status=0):
    """One call against the reference; returns (paths, tokens behind them)."""
    counts, T = [len(t) for t in trees], sum(len(t) for t in trees)
    n = len(trees)
    path = torch.full((n, max_path), 99, dtype=torch.int32, device="cuda")
    n_path, id_last = (torch.full((n,), 99, dtype=torch.int32, device="cuda") for _ in range(2))
    kw = {}
    if draft is not None:
        kw = dict(draft=padded(draft, pad), draft_row=ints(rows_d), draft_temperature=temps_d.cuda())
    c.dflash_tree_verify(starts(counts), ints(np.concatenate(trees)), ints(tokens), padded(target, pad), uniform.cuda(),
                         padded(noise, pad), path, n_path, id_last, temperature=temps.cuda(), **kw)
    assert c.dflash_cache_read_status() == status
    t64, n64, r, close, wants = np64(target), np64(noise), 0, 0, []
    d64 = None if draft is None else np64(draft)
    for s, k in enumerate(counts):
        sl = slice(r, r + k)
        want = V.verify(trees[s], tokens[sl], t64[sl], temps[sl].tolist(), d64, None if draft is None else rows_d[sl],
                        None if draft is None else temps_d.tolist(), uniform[sl].double().numpy(), n64[s], max_path)
        got = path[s].tolist()
        if want is None:
            assert int(n_path[s]) == 0 and int(id_last[s]) == 99, (s, got)
        else:
            p, last, margin = want
            same = got == p + [-1] * (max_path - len(p)) and int(n_path[s]) == len(p) and int(id_last[s]) == last
            assert same or margin < CLOSE, (s, got, p, int(id_last[s]), last, margin)
            close += margin < CLOSE
        wants.append(want)
        r += k
    assert close <= 1 + n // 20
    return wants


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab,pad", [(7, 0), (40, 0), (40, 3), (5000, 0), (20011, 0)])
def test_rows_of_large_scores(dtype, vocab, pad):
    """Rows whose scores log2(e) x / t reach from 2^20 to just below 2^30, the largest alone, tied in one thread or
    all over the row, and in steps of a unit in the last place, where the steps are what tells tokens apart.

    With fp32 scores a reference rounds away up to 32 powers of two there: 2e-6 of a probability is left."""
    g = torch.Generator().manual_seed(vocab)
    rng = np.random.default_rng(vocab)
    c = make()
    most = 2.0 ** 30 / 1.4426951
    tops = [(1e-6, x) for x in (97.0, 101.5, 108.5, 113.0, 117.5, 120.0, 300.0, 740.0)]
    tops += [(1e-6, x) for x in 80 + 650 * rng.random(8)] + [(1.0, most * 2.0 ** -k * (0.99 - 0.4 * rng.random())) for k in range(10)]
    tops += [(0.01, -30000.0), (1e-6, -200.0), (1.0, -0.98 * most), (1.0, -3e7)]
    trees, tokens, rows, temps = [], [], [], []
    for i, (t, top) in enumerate(tops):
        for shape in range(3):
            x = (torch.tensor(top) - abs(top) * 0.01 * (1 + torch.rand(vocab, generator=g))).to(DT[dtype])
            top_v = torch.tensor([top]).to(DT[dtype])
            at = rng.permutation(vocab)[:min(vocab, 6)] if i % 2 else (rng.integers(0, max(1, vocab - 6)) + np.arange(min(vocab, 6)))
            for k, j in enumerate(at):
                if shape == 0:
                    x[j] = top_v[0] if k == 0 else x[j]
                elif shape == 1:
                    x[j] = top_v[0]
                else:
                    x[j] = below(top_v, k if top > 0 else -k)[0]
            if i % 3 == 2 and vocab > 10:
                x[(at[0] + 3 + np.arange(vocab // 3)) % vocab] = torch.finfo(DT[dtype]).min    # excluded
            trees.append([-1, 0])
            tokens += [0, int(at[rng.integers(0, 3) if shape == 1 and i % 3 < 2 else 0])]   # one that has a share
            rows += [x, x.flip(0)]
            temps += [t, t]
    target, temps = torch.stack(rows), torch.tensor(temps)
    n = len(trees)
    uniform, noise = torch.rand(2 * n, generator=g), exponential(g, n, vocab)
    tokens = np.array(tokens)
    wants = check(c, trees, tokens, target, temps, uniform, noise, pad=pad)
    assert None not in wants and len({len(w[0]) for w in wants}) == 2
    # as drafts too: tokens drawn from other rows of such scores
    rows_d = np.array([t // 2 * 2 for t in range(2 * n)])
    draft = target.clone()
    draft[0::2] = target[0::2].roll(1, 1)
    wants = check(c, trees, tokens, target, temps, uniform, noise, draft, rows_d, temps, pad=pad)
    assert None not in wants
    # the same row accepts whatever its own distribution offers
    rows_d = np.arange(2 * n)
    draft[1::2] = target[0::2]
    assert all(len(w[0]) == 2 for w in check(c, trees, tokens, target, temps, uniform * 0.999, noise, draft, rows_d, temps, pad=pad))


def left_behind(vocab, left, g):
    """A row of f32 logits whose first of all tokens holds all but `left` of the mass; tokens by falling share."""
    x = torch.randn(vocab, generator=g)
    x[int(x.argmax())] = x[x.topk(2).indices[1]] + 0.5
    e = x.double().exp()
    top = int(torch.randint(0, vocab, (1,), generator=g))
    rest = e.sum() - e[top]
    x[top] = torch.log(rest * (1 - left) / left).float()
    return x, torch.argsort(-x).tolist()


def border(r, q, up, width=2e-5):
    """A uniform number just above r / q (up: rejected) or just below."""
    return np.float32(r / q * (1 + (width if up else -width)))


@pytest.mark.parametrize("vocab,pad", [(16, 0), (16, 1), (3000, 0), (20011, 0)])
def test_after_a_nearly_certain_rejection(vocab, pad):
    """Argmax siblings: the likeliest token, which holds all but 1e-2 to 1e-4 of the mass, is rejected; then one or two
    more; the next is tested 2e-5 beside its border, and the draw from what is left follows."""
    g = torch.Generator().manual_seed(vocab)
    c = make()
    trees, tokens, rows, uniform = [], [], [], []
    for left in (1e-2, 1e-3, 1e-4):
        for more in (1, 2, 3):
            for up in (0, 1):
                x, order = left_behind(vocab, left, g)
                order = order[:1] + [order[1 + (5 * k) % 14] for k in range(more)]
                r = V.distribution(np64(x), 1.0)
                u = [0.0]
                for k, t in enumerate(order):
                    # (1 - 0.1 (1 - r): still below 1 where r is close to it)
                    u.append(border(r[t], 1, up) if k == more else np.float32(1 - 0.1 * (1 - r[t])))
                    r = np.where(np.arange(vocab) == t, 0, r)
                    r /= r.sum()
                trees.append([-1] + [0] * len(order))
                tokens += [0] + order
                rows += [x] + [torch.randn(vocab, generator=g) for _ in order]
                uniform += u
    n, T = len(trees), len(rows)
    wants = check(c, trees, np.array(tokens), torch.stack(rows), torch.ones(T), torch.tensor(np.array(uniform, dtype=np.float32)),
                  exponential(g, n, vocab), pad=pad)
    assert all(m >= CLOSE for _, _, m in wants)
    assert [len(w[0]) for w in wants] == [2, 1] * (n // 2)


@pytest.mark.parametrize("certain", [True, False])
def test_siblings_that_cover_the_support(certain):
    """Six tokens of shares that fall by a hundred each, all of them drafted: the last one is certain."""
    g = torch.Generator().manual_seed(2)
    rng = np.random.default_rng(2)
    c = make()
    trees, tokens, rows, uniform = [], [], [], []
    for k in range(24):
        x = torch.full((40,), -float("inf"))
        at = rng.permutation(40)[:6]
        x[at] = -torch.arange(6.0) * (1.0 + k % 4) + 0.1 * torch.randn(6, generator=g)
        order = at if k < 12 else at[[0, 2, 1, 4, 3, 5]]
        trees.append([-1] + [0] * 6)
        tokens += [0, *order.tolist()]
        rows += [x] + [torch.randn(40, generator=g)] * 6
        uniform += [0.0] + [0.9999] * 6
    n, T = len(trees), len(rows)
    kw = {}
    if not certain:   # of a drafter at temperature 0, and of another node's that is not: the same
        kw = dict(draft=torch.randn(T, 40, generator=g), rows_d=np.arange(T), temps_d=torch.zeros(T))
    wants = check(c, trees, np.array(tokens), torch.stack(rows), torch.ones(T), torch.tensor(uniform), exponential(g, n, 40), **kw)
    assert all(m >= CLOSE for _, _, m in wants)
    assert max(w[0][-1] for w in wants) == 6


def test_rejected_tokens_stay_out():
    """Uniform numbers of 1, outside of their range, reject every sibling: the token behind the path is still none of
    those that had no share any more when the last one was rejected."""
    g = torch.Generator().manual_seed(3)
    c = make()
    x = torch.full((1, 12), -float("inf"))
    x[0, :4] = torch.tensor([9.0, 3.0, -2.0, -9.0])
    parents, order = [-1, 0, 0, 0, 0], [0, 1, 2, 3]
    for draft in (None, torch.randn(5, 12, generator=g)):
        for order in ([0, 1, 2, 3], [3, 0, 1, 2], [2, 3, 1, 0]):
            path, n_path, last = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((1, 4), 1, 1))
            kw = {} if draft is None else dict(draft=draft.cuda(), draft_temperature=torch.zeros(5, device="cuda"))
            c.dflash_tree_verify(starts([5]), ints(parents), ints([0] + order), x.repeat(5, 1).cuda(), torch.ones(5, device="cuda"),
                                 exponential(g, 1, 12).cuda(), path, n_path, last, **kw)
            # (a share rounded to just above 1 may have been accepted)
            if int(n_path) == 1:
                assert int(last) == order[-1]
            else:
                assert int(path[0, 1]) == 4
    assert c.dflash_cache_read_status() == 0


def close_rows(vocab, spread, g, ttype="f32", dtype_d="f32"):
    """A target's row and a drafter's that differs by `spread` only, with their probabilities."""
    x = (2 * torch.randn(vocab, generator=g)).to(DT[ttype])
    y = (x.float() + spread * torch.randn(vocab, generator=g)).to(DT[dtype_d])
    return x, y, V.distribution(np64(x), 1.0), V.distribution(np64(y), 1.0)


@pytest.mark.parametrize("vocab,pad,ttype,dtype_d", [
    (40, 0, "f32", "f32"), (2000, 0, "f32", "f32"), (2000, 1, "f32", "f32"), (20011, 0, "f32", "f32"), (32768, 0, "f32", "f32"),
    (327680, 0, "f32", "f32"), (2000, 0, "bf16", "bf16"), (2000, 3, "bf16", "f32"), (9000, 0, "f32", "bf16")])
@pytest.mark.parametrize("spread", [0.05, 1e-3, 1e-4])
def test_drafters_close_to_the_target(vocab, pad, ttype, dtype_d, spread):
    """Drafts of a distribution that differs from the target's by 5e-2 to 1e-4 are rejected (a user meets that once in
    as many drafts); the draw from the rest is a race that two tokens run within 3e-5, and siblings are tested 2e-5
    beside their borders: one, or two that are both rejected."""
    g = torch.Generator().manual_seed(vocab)
    rng = np.random.default_rng(vocab)
    c = make()
    trees, tokens, rows, drafts, rows_d, uniform, noise = [], [], [], [], [], [], []
    for k in range(16):
        x, y, p, q = close_rows(vocab, spread, g, ttype, dtype_d)
        # rejected: q above p by a third of a spread
        sure = np.flatnonzero((p < q * (1 - 0.3 * spread)) & (q > 1e-6))
        order = [int(rng.choice(sure))]
        u = [0.0, np.float32(1 - 0.1 * (1 - p[order[0]] / q[order[0]]))]
        r = np.maximum(p - q, 0)
        r /= r.sum()
        if k % 4:   # a sibling of the same drafter
            ratio = r / q
            some = np.flatnonzero((ratio > 0.05) & (ratio < 0.9))
            if len(some):
                order.append(int(rng.choice(some)))
                u.append(border(r[order[1]], q[order[1]], k % 2 or k % 4 == 2))
                if k % 4 != 3 or k % 2:
                    r = np.maximum(r - q, 0)
                    r /= r.sum()
                if k % 8 > 4:   # and a third one
                    some = np.flatnonzero((r / q > 0.05) & (r / q < 0.9))
                    if len(some):
                        order.append(int(rng.choice(some)))
                        u.append(border(r[order[2]], q[order[2]], k % 3))
        e = rng.exponential(size=vocab) + 1.01
        share = np.flatnonzero(r > 1e-3 * r.max())
        a, b = rng.choice(share, 2, replace=False) if len(share) > 1 else (share[0], share[0])
        first = np.maximum(p - q, 0)
        final = r if len(order) > 1 else first / first.sum()
        e = np.where(final > 0, final * e, e)   # keys 1 / e below 1 ..
        e[a], e[b] = final[a], final[b] * (1 + 3e-5) if a != b else final[a]   # .. and two at it
        n0, T0 = len(order) + 1, len(rows)
        trees.append([-1] + [0] * len(order))
        tokens += [0] + order
        rows += [x] + [torch.randn(vocab, generator=g).to(x.dtype) for _ in order]
        rows_d += [T0] * n0
        drafts += [y] + [torch.zeros(vocab, dtype=y.dtype) for _ in order]
        uniform += u
        noise.append(torch.tensor(e).float())
    T = len(rows)
    wants = check(c, trees, np.array(tokens), torch.stack(rows), torch.ones(T), torch.tensor(np.array(uniform, dtype=np.float32)),
                  torch.stack(noise), torch.stack(drafts), np.array(rows_d), torch.ones(T), pad=pad)
    # (bf16 rows this close differ in a few tokens, by a step: their siblings have no border)
    assert {len(w[0]) for w in wants} == {1, 2} or ttype == dtype_d == "bf16"


def test_mixed_siblings_and_close_drafters():
    """A nearly certain argmax is rejected, then drawn siblings of what is left, from a drafter that knows it well:
    every step takes from what the one before left."""
    g = torch.Generator().manual_seed(11)
    rng = np.random.default_rng(11)
    c = make()
    for vocab in (24, 3000, 20011):
        trees, tokens, rows, drafts, rows_d, temps_d, uniform = [], [], [], [], [], [], []
        for k in range(16):
            left = (1e-1, 1e-2, 1e-3)[k % 3]
            x, order = left_behind(vocab, left, g)
            y = x + (0.3, 0.01)[k % 2] * torch.randn(vocab, generator=g)
            y[order[0]] = -float("inf")   # what the drafter offers beside the argmax
            p, q = V.distribution(np64(x), 1.0), V.distribution(np64(y), 1.0)
            u = [0.0, np.float32(1 - 0.1 * (1 - p[order[0]]))]
            r = np.where(np.arange(vocab) == order[0], 0, p)
            r /= r.sum()
            at, temp = [order[0]], [0.0]
            for step in range(2):
                some = np.flatnonzero((r / np.maximum(q, 1e-30) > 0.05) & (r < q * 0.995) & (q > 1e-7))
                if not len(some):
                    break
                t = int(rng.choice(some))
                at.append(t)
                temp.append(1.0)
                u.append(border(r[t], q[t], step == 0 or k % 4 < 2))
                r = np.maximum(r - q, 0)
                r /= r.sum()
            T0 = len(rows)
            trees.append([-1] + [0] * len(at))
            tokens += [0] + at
            rows += [x] + [torch.randn(vocab, generator=g) for _ in at]
            # (a row at temperature 0 means the drafted token alone; the others' row is the entry's first)
            rows_d += [T0, T0 + 1] + [T0] * (len(at) - 1)
            drafts += [y] + [torch.zeros(vocab) for _ in at]
            temps_d += [1.0, 0.0] + [1.0] * (len(at) - 1)
            uniform += u
        n, T = len(trees), len(rows)
        wants = check(c, trees, np.array(tokens), torch.stack(rows), torch.ones(T),
                      torch.tensor(np.array(uniform, dtype=np.float32)), exponential(g, n, vocab), torch.stack(drafts),
                      np.array(rows_d), torch.tensor(temps_d))
        assert max(len(w[0]) for w in wants) == 2


def test_a_star_of_a_thousand_children():
    """The most nodes of a tree, all of them children of the anchor, argmaxes and drawn ones in turn, over few tokens and
    over many: what is left is computed again and again."""
    g = torch.Generator().manual_seed(9)
    rng = np.random.default_rng(9)
    c = make()
    for vocab in (5, 6000):
        x, y = 2 * torch.randn(vocab, generator=g), 2 * torch.randn(vocab, generator=g)
        q = V.distribution(np64(y), 1.0)
        n = 1024
        tokens = rng.choice(vocab, size=n, p=q)
        uniform = torch.full((n,), 0.9995)
        temps_d = torch.ones(2)
        temps_d[1] = 0
        check(c, [[-1] + [0] * (n - 1)], tokens, x.repeat(n, 1), torch.ones(n), uniform, exponential(g, 1, vocab),
              torch.stack([y, y]), np.arange(n) % 3 // 2, temps_d)
        check(c, [[-1] + [0] * (n - 1)], np.argsort(-np64(x))[np.arange(n) % min(vocab, 700)], x.repeat(n, 1), torch.ones(n), uniform,
              exponential(g, 1, vocab))


def test_nothing_to_draw():
    """Variates that are NaN exclude their tokens: where no other is left, the entry has no result."""
    g = torch.Generator().manual_seed(1)
    c = make()
    x, y = torch.randn(3, 30, generator=g), torch.randn(3, 30, generator=g)
    p, q = V.distribution(np64(x)[0], 1.0), V.distribution(np64(y)[0], 1.0)
    t = int(np.argmax(q - p))
    noise = exponential(g, 1, 30)
    noise[0, torch.tensor(p > q)] = float("nan")
    for kw in (dict(), dict(draft=y, rows_d=np.zeros(3, dtype=np.int64), temps_d=torch.ones(3))):
        u = torch.tensor([0.0, 0.9999, 0.9999])
        wants = check(c, [[-1, 0, 0]], np.array([0, t, t]), x, torch.ones(3), u, noise, status=0x100 if kw else 0, **kw)
        assert (wants[0] is None) == bool(kw)
