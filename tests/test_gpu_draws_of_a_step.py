"""The drafter's step, draws from its logits where they lie and their verification, one after another on a stream."""
import numpy as np
import pytest
import torch

import gpu_harness as GH
import verify_reference as V
from block_diffusion_drafter_fc_gb300.synth import BLOCK, get_config, make_workload
from test_gpu_cache import ints, make, np64, starts
from test_gpu_verify import CLOSE, exponential

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["tiny_f32", "ragged_bf16", "small_bf16"])
def test_drafts_drawn_from_a_step(name):
    """At temperature 0 the draws are the step's own drafts; at 0.8 draws, accepted paths and the tokens behind them are
    those of the 64-bit forms over the step's logits; a captured turn replays bit for bit."""
    from block_diffusion_drafter_fc_gb300 import dflash as D
    cfg = get_config(name)
    wl = make_workload(cfg)
    dw, feats = GH.to_device(wl)
    n, vocab = cfg.n_seq, cfg.n_vocab
    dr = D.Drafter(cfg, dw, max_seq=n, max_inject=max(call[2] for call in wl.inject_calls))
    GH.prefill(dr, wl, feats)
    c = make(max_seq=max(n, 6))
    g = torch.Generator().manual_seed(3)
    id_last, n_past = wl.id_last[:n].cuda(), wl.n_past[:n].cuda()
    logits = torch.empty(n, BLOCK, vocab, device="cuda")
    drafts = torch.empty(n, BLOCK - 1, dtype=torch.int32, device="cuda")
    T = n * BLOCK
    rows = (torch.arange(n)[:, None] * BLOCK + torch.arange(1, BLOCK)).reshape(-1)   # a block's row 0 is its anchor's
    shift, noise_d = 0.5 * torch.randn(T, vocab, generator=g), exponential(g, n * (BLOCK - 1), vocab)
    uniform, noise = torch.rand(T, generator=g), exponential(g, n, vocab)
    dev = [t.cuda() for t in (shift, noise_d, uniform, noise)]
    temp, temp_d = torch.full((T,), 0.8, device="cuda"), torch.full((len(rows),), 0.8, device="cuda")
    zero, drows, start = torch.zeros_like(temp_d), ints(rows), starts([BLOCK] * n)
    parents = ints([i - 1 for i in range(BLOCK)] * n)
    argmax, drawn = (torch.full((len(rows),), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    target, tokens = torch.empty(T, vocab, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    path = torch.zeros(n, BLOCK, dtype=torch.int32, device="cuda")
    n_path, last = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2))

    def turn():
        dr.dflash_step(id_last, n_past, logits, drafts)
        flat = logits.view(T, vocab)
        c.dflash_sample(flat, dev[1], argmax, rows=drows, temperature=zero)
        c.dflash_sample(flat, dev[1], drawn, rows=drows, temperature=temp_d)
        tokens.view(n, BLOCK)[:, 1:].copy_(drawn.view(n, BLOCK - 1))
        torch.add(flat, dev[0], out=target)
        c.dflash_tree_verify(start, parents, tokens, target, dev[2], dev[3], path, n_path, last, draft=flat, temperature=temp,
                             draft_temperature=temp)

    turn()
    torch.cuda.synchronize()
    assert torch.equal(argmax.view(n, BLOCK - 1), drafts)
    t = float(temp[0])
    x = np64(logits).reshape(T, vocab)
    for k, r in enumerate(rows.tolist()):
        i, margin = V.race(V.distribution(x[r], t), np64(noise_d)[k])
        assert int(drawn[k]) == i or margin < CLOSE
    toks, y = tokens.cpu().numpy(), np64(target)
    for s in range(n):
        sl = slice(s * BLOCK, (s + 1) * BLOCK)
        want, token, margin = V.verify([i - 1 for i in range(BLOCK)], toks[sl], y[sl], [t] * BLOCK, x, np.arange(T)[sl], [t] * T,
                                       uniform[sl].double().numpy(), np64(noise)[s], BLOCK)
        same = path[s].tolist()[:len(want)] == want and int(n_path[s]) == len(want) and int(last[s]) == token
        assert same or margin < CLOSE
    first = [v.clone() for v in (logits, drawn, path, n_path, last)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        turn()
    for v in (logits, drawn, path, n_path, last):
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (logits, drawn, path, n_path, last)))
    assert c.dflash_cache_read_status() == 0 and dr.dflash_read_status() == 0
    dr.close()
