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
