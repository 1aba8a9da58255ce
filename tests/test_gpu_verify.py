"""Sampling and sampled verification on the GPU against the 64-bit forms of tests/verify_reference.py."""
import numpy as np
import pytest
import torch

import verify_reference as V
from test_gpu_cache import DT, ints, make, np64, random_parents, starts, _D

pytestmark = pytest.mark.gpu

# Tests compare numbers that fp32 weights put within 3e-7 of the formula's; a race's keys are within 4e-6
# (log2 of a variate of 2^-24 to 2^-22 of it): a decision closer than this may fall either way
CLOSE = 1e-5


def logits(g, rows, vocab, dtype, spread=2.0):
    x = torch.randn(rows, vocab, generator=g) * spread
    if vocab > 8:
        for _ in range(3):
            x.scatter_(1, torch.randint(0, vocab, (rows, 1), generator=g), 5 + 4 * torch.rand(rows, 1, generator=g))
    return x.to(DT[dtype])


def padded(x, pad):
    """The same rows, `pad` elements apart."""
    wide = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=x.dtype)
    wide[:, :x.shape[1]] = x
    return wide.cuda()[:, :x.shape[1]]


def exponential(g, *shape):
    return torch.empty(*shape).exponential_(generator=g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab,rows,pad", [(1, 3, 0), (2, 5, 0), (7, 40, 0), (33, 9, 3), (2047, 4, 0), (2048, 3, 0), (2049, 5, 0),
                                            (8192, 15, 0), (8192, 700, 8), (32001, 33, 0), (100003, 2, 5), (151936, 1, 0),
                                            (327680, 1, 0)])
def test_sample(dtype, vocab, rows, pad):
    g = torch.Generator().manual_seed(vocab + rows)
    c = make()
    x, noise = logits(g, rows, vocab, dtype), exponential(g, rows, vocab)
    temp = torch.rand(rows, generator=g) + 0.3
    temp[::3] = 0
    if rows > 2:
        temp[1], temp[2] = 2.0 ** -21, 1000.0
    x[rows // 2, :vocab // 2] = -float("inf")
    dx, dn = padded(x, pad), padded(noise, pad)
    tokens = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    c.dflash_sample(dx, dn, tokens, temperature=temp.cuda())
    got, n64, x64 = tokens.tolist(), np64(noise), np64(x)
    for r in range(rows):
        p = V.distribution(x64[r], float(temp[r]))
        i, margin = V.race(p, n64[r])
        assert got[r] == i or margin < CLOSE, (r, got[r], i, margin)
    assert sum(V.race(V.distribution(x64[r], float(temp[r])), n64[r])[1] < CLOSE for r in range(min(rows, 40))) <= 1
    again = torch.zeros_like(tokens)
    c.dflash_sample(dx, dn, again, temperature=temp.cuda())
    assert torch.equal(again, tokens)
    # without temperatures; rows picked, one of them twice with other noise
    pick = torch.randint(0, rows, (rows,), generator=g, dtype=torch.int32)
    c.dflash_sample(dx, dn, tokens, rows=pick.cuda())
    for r in range(min(rows, 60)):
        i, margin = V.race(V.distribution(x64[int(pick[r])], 1.0), n64[r])
        assert int(tokens[r]) == i or margin < CLOSE
    assert c.dflash_cache_read_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [50, 20000])
def test_sample_rows_that_are_no_distribution(dtype, vocab):
    c = make()
    g = torch.Generator().manual_seed(0)
    x, noise = logits(g, 10, vocab, dtype), exponential(g, 10, vocab)
    temp = torch.ones(10)
    inf = float("inf")
    x[1, vocab - 1] = float("nan")
    x[2] = -inf
    x[3, 7] = inf
    temp[4], temp[5], temp[6] = -1.0, float("nan"), inf
    temp[7] = 0
    x[7, 3] = float("nan")
    x[8] = torch.finfo(DT[dtype]).min          # a row masked by the type's lowest value: nothing is left
    tokens = torch.zeros(10, dtype=torch.int32, device="cuda")
    c.dflash_sample(x.cuda(), noise.cuda(), tokens, temperature=temp.cuda())
    assert c.dflash_cache_read_status() == 0x100
    assert tokens.tolist()[1:9] == [-1] * 8 and min(tokens.tolist()[0], tokens.tolist()[9]) >= 0
    # masked tokens by the lowest value, a NaN and zeros among the noise
    y = logits(g, 3, vocab, dtype)
    y[0, 5:] = torch.finfo(DT[dtype]).min
    e = exponential(g, 3, vocab)
    e[1, 0::2] = float("nan")
    e[2, 11] = 0
    c.dflash_sample(y.cuda(), e.cuda(), tokens[:3])
    for r in range(3):
        i, margin = V.race(V.distribution(np64(y)[r], 1.0), np64(e)[r])
        assert int(tokens[r]) == i or margin < CLOSE
    assert int(tokens[2]) == 11 and c.dflash_cache_read_status() == 0
    e[2, 7] = e[2, 40] = 0                     # of several variates of 0 the first one wins, whatever the logits
    y[2, 7] = -40.0
    c.dflash_sample(y.cuda(), e.cuda(), tokens[:3])
    assert int(tokens[2]) == 7
    e[2, 7], e[2, 40] = 1e-40, 1.0             # one below the least normal number counts as 0
    e[2, 11], y[2, 7] = 1.0, -400.0
    c.dflash_sample(y.cuda(), e.cuda(), tokens[:3])
    assert int(tokens[2]) == 7
    tokens.fill_(5)
    c.dflash_sample(y.cuda(), e.cuda(), tokens[:3], rows=ints([0, 3, -1]))
    assert tokens.tolist()[1:3] == [-1, -1] and c.dflash_cache_read_status() == 0x8


@pytest.mark.parametrize("pad", [0, 1])
def test_close_races_of_large_scores(pad):
    """Two tokens whose p / e differ by 1e-4 or by 3e-5, wherever they lie, whatever the scores are.

    A score's own ulp is up to 4 here; p / e is still decided by what tells the tokens apart."""
    g = torch.Generator().manual_seed(1)
    c = make()
    heats = [(1000.0, 0.1), (-30000.0, 0.5), (5e7, 1.0), (60.0, 0.6), (0.0, 1.0), (-2000.0, 0.05), (0.001, 0.001)]
    vocab, per = 40, 24
    x, e, temp = [], [], []
    for centre, t in heats:
        for k in range(per):
            row = centre + t * 4 * torch.rand(vocab, generator=g, dtype=torch.float64)
            row = row.float()
            t32 = torch.tensor(t)
            far = 1 + 3 * torch.rand(vocab, generator=g, dtype=torch.float64)
            a, b = torch.randperm(vocab if k % 2 else 8, generator=g)[:2].tolist()
            far[a], far[b] = 1, 1 + (1e-4 if k % 4 < 2 else 3e-5)
            x.append(row)
            e.append((far * torch.exp((row.double() - row.double().max()) / t32.double())).float())
            temp.append(t32)
    x, e, temp = torch.stack(x), torch.stack(e), torch.stack(temp)
    tokens = torch.zeros(len(x), dtype=torch.int32, device="cuda")
    c.dflash_sample(padded(x, pad), padded(e, pad), tokens, temperature=temp.cuda())
    want = [V.race(V.distribution(np64(x)[r], float(temp[r])), np64(e)[r]) for r in range(len(x))]
    assert min(m for _, m in want) > CLOSE
    assert tokens.tolist() == [i for i, _ in want]
    # as the draw of a verification: single nodes
    n = len(x)
    path, n_path, last = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((n, 1), n, n))
    c.dflash_tree_verify(starts([1] * n), ints([-1] * n), ints([0] * n), padded(x, pad), torch.zeros(n, device="cuda"),
                         padded(e, pad), path, n_path, last, temperature=temp.cuda())
    assert last.tolist() == [i for i, _ in want]
    assert c.dflash_cache_read_status() == 0


def test_samples_follow_the_probabilities():
    """How often each of a few tokens is drawn, against its probability: five standard deviations."""
    c = make()
    g = torch.Generator().manual_seed(3)
    n, x = 40000, torch.tensor([[0.0, 1.0, -1.0, 2.0, -float("inf"), 0.5]])
    tokens = torch.zeros(n, dtype=torch.int32, device="cuda")
    c.dflash_sample(x.cuda(), exponential(g, n, 6).cuda(), tokens, rows=torch.zeros(n, dtype=torch.int32, device="cuda"),
                    temperature=torch.full((n,), 0.8, device="cuda"))
    p = V.distribution(np64(x)[0], 0.8)
    seen = np.bincount(tokens.cpu().numpy(), minlength=6) / n
    assert (np.abs(seen - p) <= 5 * np.sqrt(p * (1 - p) / n)).all()


def tree_case(c, g, rng, counts, vocab, ttype, dtype_d, kind="random", drafts="drawn", max_path=None, pad=0, share=True,
              cold=0.0, spread_q=0.6, tail=2):
    """One call against the reference; returns how many entries had a path of each length."""
    T = sum(counts) + tail
    trees = [random_parents(rng, n, kind) for n in counts]
    parents = np.concatenate([*map(np.asarray, trees), [-1] * tail]).astype(np.int32)
    base = np.repeat(np.concatenate([[0], np.cumsum(counts)])[:-1], counts)
    target = logits(g, T, vocab, ttype)
    temp = torch.rand(T, generator=g) * 0.6 + 0.6
    temp[torch.rand(T, generator=g) < cold] = 0
    draft = (target.float() + spread_q * torch.randn(T, vocab, generator=g)).to(DT[dtype_d])
    temp_d = torch.rand(T, generator=g) * 0.6 + 0.6
    rows_d = np.concatenate([np.maximum(parents[:T - tail], 0) + base, [0] * tail]).astype(np.int32)   # siblings share a row
    if not share:
        rows_d = np.arange(T, dtype=np.int32)
    if drafts == "mixed":
        temp_d[torch.rand(T, generator=g) < 0.4] = 0
    d64 = np64(draft)
    tokens = np.zeros(T, dtype=np.int32)
    for t in range(T):
        q = V.distribution(d64[rows_d[t]], float(temp_d[rows_d[t]]))
        tokens[t] = rng.choice(vocab, p=q) if drafts != "likely" else np.argsort(-q)[t % min(3, vocab)]
    uniform = torch.rand(T, generator=g)
    noise = exponential(g, len(counts), vocab)
    max_path = max_path or max(counts + [1])
    path = torch.full((len(counts), max_path), 99, dtype=torch.int32, device="cuda")
    n_path, id_last = (torch.full((len(counts),), 99, dtype=torch.int32, device="cuda") for _ in range(2))
    given = drafts != "likely"
    c.dflash_tree_verify(starts(counts), ints(parents), ints(tokens), padded(target, pad), uniform.cuda(), padded(noise, pad), path,
                         n_path, id_last, draft=padded(draft, pad) if given else None,
                         draft_row=ints(rows_d) if given and share else None, temperature=temp.cuda(),
                         draft_temperature=temp_d.cuda() if given else None)
    t64, n64, r, close, lengths = np64(target), np64(noise), 0, 0, []
    for s, n in enumerate(counts):
        got = path[s].tolist()
        if n == 0:
            assert got == [-1] * max_path and int(n_path[s]) == 0 and int(id_last[s]) == 99
            continue
        sl = slice(r, r + n)
        want, last, margin = V.verify(trees[s], tokens[sl], t64[sl], temp[sl].tolist(), d64 if given else None, rows_d[sl],
                                      temp_d.tolist(), uniform[sl].double().numpy(), n64[s], max_path)
        same = got == want + [-1] * (max_path - len(want)) and int(n_path[s]) == len(want) and int(id_last[s]) == last
        assert same or margin < CLOSE, (s, got, want, int(id_last[s]), last, margin)
        close += margin < CLOSE
        lengths.append(len(want))
        r += n
    assert close <= 1 + len(counts) // 20
    assert c.dflash_cache_read_status() == 0
    return lengths


@pytest.mark.parametrize("ttype,dtype_d", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("vocab,pad", [(1, 0), (2, 0), (5, 0), (64, 0), (2049, 0), (5000, 8), (16400, 0)])
def test_tree_verify(ttype, dtype_d, vocab, pad):
    g = torch.Generator().manual_seed(vocab)
    rng = np.random.default_rng(vocab)
    c = make()
    tree_case(c, g, rng, [1], vocab, ttype, dtype_d, pad=pad)
    tree_case(c, g, rng, [16], vocab, ttype, dtype_d, kind="chain", share=False, pad=pad, tail=0)
    tree_case(c, g, rng, [9, 0, 33, 1, 20], vocab, ttype, dtype_d, pad=pad)
    tree_case(c, g, rng, [40] * 6, vocab, ttype, dtype_d, drafts="mixed", cold=0.1, pad=pad, spread_q=2.0)
    tree_case(c, g, rng, [16, 12, 40], vocab, ttype, dtype_d, drafts="likely", pad=pad)
    tree_case(c, g, rng, [30, 30], vocab, ttype, dtype_d, max_path=3, pad=pad, spread_q=0.1)
    tree_case(c, g, rng, [20, 20], vocab, ttype, dtype_d, kind="forest", max_path=64, pad=pad)


def test_large_calls():
    """Most nodes of a tree, hundreds of entries, the largest vocabulary."""
    g = torch.Generator().manual_seed(1)
    rng = np.random.default_rng(1)
    c = make()
    tree_case(c, g, rng, [1024, 3], 300, "f32", "f32", spread_q=0.3)
    tree_case(c, g, rng, [1024], 40, "f32", "f32", kind="chain", spread_q=0.02, share=False)
    lengths = tree_case(c, g, rng, rng.integers(0, 9, 400).tolist(), 100, "bf16", "bf16")
    assert max(lengths) > 3
    tree_case(c, g, rng, [4, 3], 327680, "f32", "f32")
    tree_case(c, g, rng, [12, 5, 9], 151936, "bf16", "bf16", spread_q=3.0)


def test_star_of_many_rejections():
    """A root with hundreds of children: one rejection after another, duplicates among the tokens."""
    g = torch.Generator().manual_seed(5)
    c = make()
    for vocab, n in ((3000, 300), (12, 200)):
        for certain in (False, True):
            parents = np.array([-1] + [0] * (n - 1), dtype=np.int32)
            target, draft = logits(g, n, vocab, "f32"), logits(g, 1, vocab, "f32")
            q = V.distribution(np64(draft)[0], 1.0)
            tokens = np.random.default_rng(vocab).choice(vocab, size=n, p=q).astype(np.int32)
            uniform = torch.rand(n, generator=g) * 0.02 + 0.98
            noise = exponential(g, 1, vocab)
            path = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
            n_path, id_last = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
            kw = {} if certain else dict(draft=draft.cuda(), draft_row=torch.zeros(n, dtype=torch.int32, device="cuda"))
            c.dflash_tree_verify(starts([n]), ints(parents), ints(tokens), target.cuda(), uniform.cuda(), noise.cuda(), path, n_path,
                                 id_last, **kw)
            want, last, margin = V.verify(parents, tokens, np64(target), [1.0] * n, None if certain else np64(draft), [0] * n, [1.0],
                                          uniform.double().numpy(), np64(noise)[0], 4)
            assert (path[0].tolist()[:len(want)] == want and int(n_path) == len(want) and int(id_last) == last) or margin < 1e-4
            assert c.dflash_cache_read_status() == 0


def test_temperature_zero_is_greedy_acceptance():
    """Equal to dflash_tree_accept with the target's argmaxes, whatever the drafts' distribution."""
    g = torch.Generator().manual_seed(8)
    rng = np.random.default_rng(8)
    c = make()
    counts, vocab = [16, 40, 7, 1], 6
    T = sum(counts)
    parents = ints(np.concatenate([random_parents(rng, n, "random") for n in counts]))
    target = logits(g, T, vocab, "bf16").cuda()
    tokens = ints(rng.integers(0, vocab, T))
    outs = [[torch.zeros(4, 9, dtype=torch.int32, device="cuda")] + [torch.zeros(4, dtype=torch.int32, device="cuda") for _ in range(2)]
            for _ in range(3)]
    zero, u, noise = torch.zeros(T, device="cuda"), torch.rand(T, generator=g).cuda(), exponential(g, 4, vocab).cuda()
    c.dflash_tree_accept(starts(counts), parents, tokens, target.float().argmax(1).to(torch.int32), *outs[0])
    c.dflash_tree_verify(starts(counts), parents, tokens, target, u, noise, *outs[1], temperature=zero)
    c.dflash_tree_verify(starts(counts), parents, tokens, target, u, noise, *outs[2], temperature=zero,
                         draft=logits(g, T, vocab, "f32").cuda())
    for o in outs[1:]:
        for a, b in zip(outs[0], o):
            assert torch.equal(a, b)


@pytest.mark.parametrize("certain", [False, True])
def test_verified_tokens_follow_the_target(certain):
    """First accepted tokens of trees of two drafted siblings: the target's distribution, five standard deviations."""
    c = make()
    g = torch.Generator().manual_seed(4)
    n, vocab, rounds = 1024, 5, 20
    x, y = torch.tensor([0.3, 1.2, -0.5, 0.9, -2.0]), torch.tensor([1.0, 0.2, 0.1, 0.4, -1.0])
    parents = ints([-1, 0, 0] * n)
    target, draft = x.repeat(3 * n, 1).cuda(), y[None].cuda()
    path = torch.zeros(n, 3, dtype=torch.int32, device="cuda")
    n_path, id_last = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2))
    seen = np.zeros(vocab)
    for _ in range(rounds):
        if certain:
            tokens = torch.randint(0, vocab, (3 * n,), generator=g, dtype=torch.int32).cuda()
            kw = {}
        else:
            tokens = torch.zeros(3 * n, dtype=torch.int32, device="cuda")
            c.dflash_sample(draft, exponential(g, 3 * n, vocab).cuda(), tokens, rows=torch.zeros_like(tokens))
            kw = dict(draft=draft, draft_row=torch.zeros_like(tokens))
        c.dflash_tree_verify(starts([3] * n), parents, tokens, target, torch.rand(3 * n, generator=g).cuda(),
                             exponential(g, n, vocab).cuda(), path, n_path, id_last, **kw)
        second = path[:, 1].long().clamp(min=0)
        first = torch.where(n_path > 1, tokens.view(n, 3).gather(1, second[:, None])[:, 0], id_last)
        seen += np.bincount(first.cpu().numpy(), minlength=vocab)
    p, total = V.distribution(x.double().numpy(), 1.0), n * rounds
    assert (np.abs(seen / total - p) <= 5 * np.sqrt(p * (1 - p) / total)).all()


def test_verify_faults():
    D = _D()
    c = make()
    g = torch.Generator().manual_seed(0)
    vocab, T = 40, 12
    target, draft, noise = logits(g, T, vocab, "f32"), logits(g, 3, vocab, "f32"), exponential(g, 3, vocab)
    parents, rows = [-1, 0, 1, 2] * 3, [0, 0, 1, 2] * 3

    def run(status, dead, start=(0, 4, 8, 12), tokens=None, target=target, draft=draft, rows=rows, temp=None, temp_d=None, u=0.0):
        path = torch.full((3, 4), 9, dtype=torch.int32, device="cuda")
        n_path, id_last = (torch.full((3,), 9, dtype=torch.int32, device="cuda") for _ in range(2))
        tokens = [5] * T if tokens is None else tokens
        c.dflash_tree_verify(ints(start), ints(parents), ints(tokens), target.cuda(), torch.full((T,), u, device="cuda"), noise.cuda(),
                             path, n_path, id_last, draft=draft.cuda(), draft_row=ints(rows),
                             temperature=None if temp is None else temp.cuda(),
                             draft_temperature=None if temp_d is None else temp_d.cuda())
        assert c.dflash_cache_read_status() == status
        for s in range(3):
            if s in dead:
                assert int(n_path[s]) == 0 and path[s].tolist() == [-1] * 4 and int(id_last[s]) == 9
            else:
                assert int(n_path[s]) > 0 and 0 <= int(id_last[s]) < vocab
        return path, n_path

    assert run(0, [])[1].tolist() == [4, 4, 4]                                  # u = 0: everything is accepted
    run(0x8, [1], start=[0, 8, 5, 12])
    run(0x8, [2], start=[0, 4, 8, 13])
    bad = target.clone()
    bad[6] = -float("inf")                                                      # entry 1's third node
    run(0x100, [1], target=bad)
    bad[6], bad[1, 2] = 0.0, float("nan")
    run(0x100, [0], target=bad)
    bad_d = draft.clone()
    bad_d[2, 3] = float("nan")                                                  # the last node's draft
    run(0x100, [0, 1, 2], draft=bad_d)
    run(0x100, [2], rows=rows[:8] + [0, 0, 3, 2])
    run(0x100, [2], rows=rows[:8] + [0, 0, -1, 2])
    temp = torch.ones(T)
    temp[9] = -1.0
    run(0x100, [2], temp=temp)
    run(0x100, [0, 1, 2], temp_d=torch.tensor([1.0, float("nan"), 1.0]))
    toks = [5] * T
    toks[5], toks[10] = vocab, -1
    assert run(0x1, [], tokens=toks)[1].tolist() == [4, 1, 2]
    # rows that the walk does not reach may hold anything
    bad = target.clone()
    bad[2:4] = float("nan")
    toks = [5] * T
    toks[2] = 7
    t0 = torch.ones(T)
    t0[1] = 0.0                                                                 # node 1 goes on to its argmax alone
    bad[1, 9] = 50.0
    assert run(0, [], target=bad, tokens=toks, temp=t0)[1].tolist()[0] == 2
    with pytest.raises(D.DFlashError):
        run(0, [], target=target[:11])
    big = torch.zeros(65537, 1)
    out = [torch.zeros(1, 1, dtype=torch.int32, device="cuda")] + [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2)]
    idx = torch.zeros(65537, dtype=torch.int32, device="cuda")
    with pytest.raises(D.DFlashError, match="too many rows"):
        c.dflash_tree_verify(ints([0, 1]), idx, idx, big.cuda(), big[:, 0].cuda(), big[:1].cuda(), *out)
    long = torch.zeros(1025, 1)
    c.dflash_tree_verify(ints([0, 1025]), idx[:1025], idx[:1025], long.cuda(), long[:, 0].cuda(), long[:1].cuda(), *out)
    assert c.dflash_cache_read_status() == 0x8 and int(out[1]) == 0
    none = torch.zeros(0, vocab, device="cuda")
    c.dflash_tree_verify(ints([0, 0]), idx[:0], idx[:0], none, none[:, 0], noise[:1].cuda(), *out)
    assert c.dflash_cache_read_status() == 0 and int(out[1]) == 0
    c.dflash_sample(none, none, idx[:0])


def test_captured_and_on_another_stream():
    """A captured draw and verification replay with new contents, bit for bit as eager calls on a side stream."""
    c = make()
    g = torch.Generator().manual_seed(6)
    rng = np.random.default_rng(6)
    n, B, vocab = 5, 16, 9001
    T = n * B
    parents = ints(np.concatenate([random_parents(rng, B, "random") for _ in range(n)]))
    start = starts([B] * n)
    target, draft = (torch.zeros(T, vocab, device="cuda") for _ in range(2))
    e1, e2, u = torch.zeros(T, vocab, device="cuda"), torch.zeros(n, vocab, device="cuda"), torch.zeros(T, device="cuda")
    outs = [[torch.zeros(n, B, dtype=torch.int32, device="cuda")] + [torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2)]
            for _ in range(2)]
    toks = [torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(2)]

    def turn(i, stream=None):
        c.dflash_sample(draft, e1, toks[i], stream=stream)
        c.dflash_tree_verify(start, parents, toks[i], target, u, e2, *outs[i], draft=draft, stream=stream)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        turn(0)
    for _ in range(5):
        target.copy_(logits(g, T, vocab, "f32"))
        draft.copy_(target + 0.5 * torch.randn(T, vocab, generator=g).cuda())
        e1.exponential_()
        e2.exponential_()
        u.uniform_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        turn(1, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(toks[0], toks[1])
        for a, b in zip(*outs):
            assert torch.equal(a, b)
    assert c.dflash_cache_read_status() == 0


def test_offsets_past_32_bits():
    """Logits behind 4 GB."""
    c = make()
    vocab, rows = 40000, 28000
    x = torch.zeros(rows, vocab, device="cuda")
    assert x.numel() * 4 > 1 << 32
    x[rows - 1, 39999] = 60.0
    x[rows - 2, 7] = 60.0
    tokens = torch.zeros(3, dtype=torch.int32, device="cuda")
    noise = torch.ones(3, vocab, device="cuda")
    noise[2, 123] = 1e-3
    c.dflash_sample(x, noise, tokens, rows=ints([rows - 1, rows - 2, 5]))
    assert tokens.tolist() == [39999, 7, 123]
    assert c.dflash_cache_read_status() == 0


def test_calls_that_the_library_refuses():
    """Bad sizes, types, strides and null pointers return before anything is launched."""
    D = _D()
    c = make()
    L, h, p = D.LIB, c.h, torch.zeros(64, device="cuda").data_ptr()

    def sample(T=2, V=8, x=p, ld=8, dt=0, n=2, rows=None, t=None, e=p, els=8, out=p):
        return L.dflash_sample(h, T, V, x, ld, dt, n, rows, t, e, els, out, None)

    assert sample(T=-1) == sample(V=0) == sample(ld=7) == sample(dt=2) == sample(dt=-1) == sample(n=1) == sample(n=-1) == -1
    assert sample(x=None) == sample(x=p + 2) == sample(x=p + 1, dt=1) == sample(e=None) == sample(els=7) == sample(out=None) == -1
    assert sample(V=327681, ld=327681, els=327681) == -2 and sample(T=(1 << 24) + 1, n=1 << 25) == -3
    assert sample(T=0, e=None, out=None) == 0

    def verify(n=1, start=p, T=2, par=p, tok=p, V=8, x=p, ld=8, dt=0, t=None, d=None, dld=8, ddt=0, nd=0, dr=None, td=None, u=p, e=p,
               els=8, path=p, mp=2, npth=p, last=p):
        return L.dflash_tree_verify(h, n, start, T, par, tok, V, x, ld, dt, t, d, dld, ddt, nd, dr, td, u, e, els, path, mp, npth,
                                    last, None)

    assert verify(T=-1) == verify(V=0) == verify(mp=0) == verify(start=None) == verify(par=None) == verify(tok=None) == -1
    assert verify(x=None) == verify(ld=7) == verify(dt=3) == verify(u=None) == verify(e=None) == verify(path=None) == -1
    assert verify(npth=None) == verify(last=None) == verify(n=2, els=7) == -1
    assert verify(nd=1) == verify(dr=p) == verify(td=p) == verify(d=p) == verify(d=p, nd=-1) == -1      # what goes with draft
    assert verify(d=p, nd=2, dld=7) == verify(d=p, nd=2, ddt=2) == -1
    assert verify(V=327681, ld=327681) == -2 and verify(n=1025) == verify(n=-1) == -4
    assert verify(T=65536, d=p, nd=1) == -3
    assert verify(n=0) == 0
    assert c.dflash_cache_read_status() == 0


def test_two_handles_on_two_streams():
    """Draws and verifications of two handles at the same time equal those of each alone."""
    g = torch.Generator().manual_seed(2)
    rng = np.random.default_rng(2)
    n, B, vocab = 7, 12, 5000
    T = n * B
    sides = []
    for _ in range(2):
        target = logits(g, T, vocab, "bf16")
        draft = target.float() + 0.5 * torch.randn(T, vocab, generator=g)
        sides.append(dict(c=make(), s=torch.cuda.Stream(), parents=ints(np.concatenate([random_parents(rng, B, "random") for _ in range(n)])),
                          target=target.cuda(), draft=draft.cuda(), e=exponential(g, T, vocab).cuda(), e2=exponential(g, n, vocab).cuda(),
                          u=torch.rand(T, generator=g).cuda()))
    start = starts([B] * n)

    def turn(k, stream=None):
        o = [torch.zeros(T, dtype=torch.int32, device="cuda"), torch.zeros(n, B, dtype=torch.int32, device="cuda"),
             torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")]
        torch.cuda.synchronize()
        return o, lambda: (k["c"].dflash_sample(k["draft"], k["e"], o[0], stream=stream),
                           k["c"].dflash_tree_verify(start, k["parents"], o[0], k["target"], k["u"], k["e2"], *o[1:], draft=k["draft"],
                                                     stream=stream))

    alone = []
    for k in sides:
        o, call = turn(k)
        call()
        alone.append(o)
    torch.cuda.synchronize()
    both = [[turn(k, k["s"]) for k in sides] for _ in range(10)]
    for pair in both:
        for _, call in pair:
            call()
    torch.cuda.synchronize()
    for pair in both:
        for (o, _), want in zip(pair, alone):
            assert all(torch.equal(a, b) for a, b in zip(o, want))
