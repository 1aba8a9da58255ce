"""Norms, shared prefixes, drawing and sampled verification together, as a decoding loop uses them."""
import numpy as np
import pytest
import torch

import cache_reference as R
import norm_reference as N
import verify_reference as V
from test_gpu_cache import DT, HALF, check, ints, make, normal, np64, random_parents, starts

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sampled_turns_of_forks_equal_a_plain_model(dtype):
    """Two prompts, forked into three continuations each; turns of reserve, prefix plan, draft (sample), per layer
    norm_append and prefix_attend, tree_verify and commit: every layer's attention output and every accepted
    path equal those of a plain cache of the accepted tokens, computed from scratch in 64 bits."""
    rng = np.random.default_rng(4)
    g = torch.Generator().manual_seed(1)
    hq, hkv, hd, L, ps, vocab = 4, 2, 64, 2, 16, 12
    c = make(n_layer=L, n_head=hq, n_head_kv=hkv, head_dim=hd, page_size=ps, n_pages=160, max_seq=6, max_pages=16, dtype=dtype)
    f, m = R.rope_freqs(hd)
    emb = normal(g, (L, vocab, hq + 2 * hkv, hd), dtype)     # a token's q, k, v rows by layer
    dev = emb.cuda()
    wq, wk = ((1 + 0.3 * torch.randn(hd, generator=g)).to(DT[dtype]) for _ in range(2))
    wqd, wkd = wq.cuda(), wk.cuda()
    bounds = ints([0, 3, 6])
    history = {q: [] for q in range(6)}

    def forward(seqs, tokens, trees, groups, turn=0):
        """The layers' outputs of a tree per sequence, groups: bounds of those that share a prompt (None: plain attention)."""
        counts = [len(t) for t in tokens]
        start, flat = starts(counts), torch.as_tensor(np.concatenate(tokens)).cuda()
        T, words = sum(counts), max(1, -(-max(counts) // 32))
        mask = torch.zeros(T, words, dtype=torch.int32, device="cuda")
        depth = torch.zeros(T, dtype=torch.int32, device="cuda")
        c.dflash_cache_reserve(ints(counts), seqs=ints(seqs))
        c.dflash_tree_mask(start, ints(np.concatenate(trees)), mask, depth)
        if groups is not None:
            plan = torch.zeros(len(seqs) + groups.shape[0] - 1, dtype=torch.int32, device="cuda")
            c.dflash_prefix_plan(groups, plan, seqs=ints(seqs))
            if turn % 2:      # (these prompts are too short to be worth it: shared all the same in every other turn)
                plan.copy_(ints([32] * 3 + [48] * 3 + [32, 48]))
            work = torch.empty(c.prefix_workspace(T), dtype=torch.uint8, device="cuda")
        outs = []
        for layer in range(L):
            rows = dev[layer][flat]
            q_rot, out = (torch.empty(T, hq, hd, dtype=DT[dtype], device="cuda") for _ in range(2))
            c.dflash_norm_append(layer, start, rows[:, hq:hq + hkv], rows[:, hq + hkv:], wkd, depth=depth, q=rows[:, :hq],
                                 q_norm=wqd, q_out=q_rot, eps=EPS, seqs=ints(seqs))
            if groups is None:
                c.dflash_tree_attend(layer, start, max(counts), q_rot, out, mask=mask, seqs=ints(seqs))
            else:
                c.dflash_prefix_attend(layer, start, max(counts), q_rot, out, groups, plan, work, mask=mask, seqs=ints(seqs))
            outs.append(np64(out))
        return outs, start

    def compare(outs, seqs, tokens, trees):
        r = 0
        for q, toks, tree in zip(seqs, tokens, trees):
            sets, past = R.tree_sets(tree), history[q]
            all_tokens = np.array(past + list(toks), dtype=int)
            pos = np.concatenate([np.arange(len(past)), len(past) + sets.sum(1) - 1]).astype(int)
            sees = np.concatenate([np.ones((len(toks), len(past)), bool), sets], 1)
            for layer in range(L):
                e = np64(emb[layer])[all_tokens]
                args = (EPS, "half", hd, f, m, HALF[dtype])

                def stored(x):     # what the pages hold: rounded once
                    return np64(torch.as_tensor(x).to(DT[dtype]))

                k = stored(N.forward(e[:, hq:hq + hkv], np64(wk), pos, *args)[0])
                qq = stored(N.forward(e[len(past):, :hq], np64(wq), pos[len(past):], *args)[0])
                o, _, size, big = R.attend(qq, k, e[:, hq + hkv:], sees, hd ** -0.5)
                tol, _ = R.attend_bounds(o, size, big, len(all_tokens), hd, dtype)
                # the parts of a row (test_gpu_prefix.py); a normalised and rotated key or query may round to the
                # other neighbour: a step of the type in one operand moves a score by up to 2^-7 (2^-23) of |q| |k|, on
                # either side, and its fp32 error by 1e-5 more
                tol = tol + 2.02 * size * (2.0 ** -21 + big[..., None] * 2.0 ** -23)
                tol = tol + size * 4 * (2 * HALF[dtype] + 1e-5) * big[..., None]
                check(outs[layer][r:r + len(toks)], o, tol, f"sequence {q}, layer {layer}")
            r += len(toks)

    prompts = [rng.integers(0, vocab, 37).tolist(), rng.integers(0, vocab, 50).tolist()]
    chains = [[i - 1 for i in range(len(p))] for p in prompts]
    outs, _ = forward([0, 3], prompts, chains, None)
    compare(outs, [0, 3], prompts, chains)
    c.dflash_cache_commit(None, ints([37, 50]), seqs=ints([0, 3]))
    history[0], history[3] = list(prompts[0]), list(prompts[1])
    c.dflash_cache_fork(ints([0, 0, 3, 3]), ints([1, 2, 4, 5]))
    for q in range(6):
        history[q] = list(prompts[q // 3])
    seqs, last = list(range(6)), [int(rng.integers(0, vocab)) for _ in range(6)]
    accepted = 0
    for turn in range(4):
        trees = [random_parents(rng, n, "random") for n in (9, 1, 14, 20, 5, 11)]
        counts = [len(t) for t in trees]
        T = sum(counts)
        base = np.repeat(np.concatenate([[0], np.cumsum(counts)])[:-1], counts)
        draft_row = np.maximum(np.concatenate(trees), 0) + base
        draft, temp = 1.5 * torch.randn(T, vocab, generator=g), torch.full((T,), 0.9)
        drawn = torch.zeros(T, dtype=torch.int32, device="cuda")
        noise_d = torch.empty(T, vocab).exponential_(generator=g)
        c.dflash_sample(draft.cuda(), noise_d.cuda(), drawn, rows=ints(draft_row), temperature=temp.cuda())
        drawn = drawn.cpu().numpy()
        for t in range(T):
            i, margin = V.race(V.distribution(np64(draft)[draft_row[t]], 0.9), np64(noise_d)[t])
            assert drawn[t] == i or margin < 1e-5
        r, tokens = 0, []
        for n, q in zip(counts, seqs):
            drawn[r] = last[q]              # the anchor: the token behind the last path
            tokens.append(drawn[r:r + n].tolist())
            r += n
        outs, start = forward(seqs, tokens, trees, bounds, turn)
        compare(outs, seqs, tokens, trees)
        # (the target's logits: any function of the tokens does for the acceptance)
        target = (draft + 0.7 * torch.randn(T, vocab, generator=g)).to(DT[dtype])
        uniform, noise = torch.rand(T, generator=g), torch.empty(6, vocab).exponential_(generator=g)
        path = torch.zeros(6, 8, dtype=torch.int32, device="cuda")
        n_path, id_last = (torch.zeros(6, dtype=torch.int32, device="cuda") for _ in range(2))
        c.dflash_tree_verify(start, ints(np.concatenate(trees)), ints(np.concatenate(tokens)), target.cuda(), uniform.cuda(),
                             noise.cuda(), path, n_path, id_last, draft=draft.cuda(), draft_row=ints(draft_row), temperature=temp.cuda(),
                             draft_temperature=temp.cuda())
        c.dflash_cache_commit(path, n_path, seqs=ints(seqs))
        r = 0
        for s, (q, tree, toks) in enumerate(zip(seqs, trees, tokens)):
            n = len(toks)
            want, token, margin = V.verify(tree, toks, np64(target)[r:r + n], [0.9] * n, np64(draft), draft_row[r:r + n],
                                           [0.9] * T, uniform[r:r + n].double().numpy(), np64(noise)[s], 8)
            assert margin > 1e-5            # (of these seeds: no comparison is close)
            assert path[s].tolist()[:len(want)] == want and int(n_path[s]) == len(want) and int(id_last[s]) == token
            history[q] += [toks[i] for i in want]
            last[q] = token
            accepted += len(want) - 1
            r += n
        assert [int(c.length[q]) for q in range(6)] == [len(history[q]) for q in range(6)]
        c.dflash_cache_trim(ints([len(history[q]) for q in range(6)]))     # reserved pages go back
        assert c.dflash_cache_read_status() == 0
    assert accepted > 10
    c.dflash_cache_trim(ints([0] * 6))
    assert int(c.refs.abs().sum()) == 0
