"""Norms of query and key heads with their rotation, the gradient, and the append of normalised
keys, on the GPU against 64-bit forms (tests/norm_reference.py)."""
import numpy as np
import pytest
import torch

import norm_reference as N
from test_gpu_cache import (DT, HALF, ROPES, check, ints, make, normal, np64, random_parents, rope_setup, scattered, starts,
                            _D)
import cache_reference as R

pytestmark = pytest.mark.gpu

EPS = 1e-6


def weights(g, hd, dtype):
    return (1 + 0.3 * torch.randn(hd, generator=g)).to(DT[dtype])


def adds(T, heads, others, hd, lanes):
    """Most additions a term of a weight's gradient goes through: the rows of its thread (of at least 152 blocks, shared
    by blocks of up to 256 columns), a block's threads at its place (256 over a head's lanes), 19 of up to 608
    blocks by each warp, 32 warps."""
    ny = -(-(heads + others) * lanes // 256)
    return min(T * heads, -(-T // max(1, 152 // ny)) + 256 // lanes + 19 + 32)


def lanes(hd, dtype, rd):
    """Lanes of a head: two vectors of 16 bytes each, of 8 where 16 do not hold whole pairs."""
    return hd // (8 if dtype == "f32" or rd % 16 else 16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("layout,rot,kw", ROPES, ids=str)
def test_norm_rope_and_gradient(dtype, hd, layout, rot, kw):
    rd, f, m = rope_setup(hd, layout, rot, kw)
    g = torch.Generator().manual_seed(hd + len(kw))
    for T, hq, hkv in ((1, 1, 1), (3, 6, 2), (37, 4, 4), (130, 9, 3)):
        c = make(n_head=hq, n_head_kv=hkv, head_dim=hd, dtype=dtype, rope_layout=layout, rotary_dim=rd, **kw)
        pos = torch.randint(0, 3_000_000, (T,), generator=g, dtype=torch.int32)
        x = [normal(g, (T, h, hd), dtype) * 2 for h in (hq, hkv)]
        x[0][0, 0] = 0                       # a head of zeros
        x[1][T // 2, 0, :4] = 0
        w = [weights(g, hd, dtype) for _ in x]
        dy = [normal(g, (T, h, hd), dtype) for h in (hq, hkv)]
        dev = [[t.cuda() for t in ts] for ts in (x, w, dy)]
        out = [torch.full_like(t, float("nan")) for t in dev[0]]
        c.dflash_norm_rope(pos.cuda(), q=dev[0][0], q_norm=dev[1][0], q_out=out[0], k=dev[0][1], k_norm=dev[1][1], k_out=out[1])
        dx = [torch.full_like(t, float("nan")) for t in dev[0]]
        dw = [torch.full((hd,), float("nan"), device="cuda") for _ in x]
        c.dflash_norm_rope_grad(pos.cuda(), q=dev[0][0], q_norm=dev[1][0], dq_out=dev[2][0], dq=dx[0], dq_norm=dw[0],
                                k=dev[0][1], k_norm=dev[1][1], dk_out=dev[2][1], dk=dx[1], dk_norm=dw[1])
        for i, h in enumerate((hq, hkv)):
            args = (pos.numpy(), EPS, layout, rd, f, m, HALF[dtype])
            y, tol = N.forward(np64(x[i]), np64(w[i]), *args)
            check(np64(out[i]), y, tol, f"{T} rows, part {i}")
            ex, tx, ew, tw = N.backward(np64(x[i]), np64(w[i]), np64(dy[i]), *args, adds(T, h, hq + hkv - h, hd, lanes(hd, dtype, rd)))
            check(np64(dx[i]), ex, tx, f"{T} rows, part {i}: dx")
            check(np64(dw[i]), ew, tw, f"{T} rows, part {i}: dw")
        assert c.dflash_cache_read_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [607, 609, 2500, 9731])
def test_many_rows_strided_in_place(dtype, T):
    """Several rows a block, the rows of a fused projection in place, one part alone."""
    hq, hkv, hd = 8, 2, 128
    c = make(n_head=hq, n_head_kv=hkv, head_dim=hd, dtype=dtype)
    rd, f, m = rope_setup(hd, "half", None, {})
    g = torch.Generator().manual_seed(T)
    fused, dy = normal(g, (T, hq + 2 * hkv, hd), dtype), normal(g, (T, hq + 2 * hkv, hd), dtype)
    pos = torch.randint(0, 200000, (T,), generator=g, dtype=torch.int32)
    w = [weights(g, hd, dtype) for _ in range(2)]
    wd, dev, ddev = [t.cuda() for t in w], fused.cuda(), dy.cuda()
    q, k = dev[:, :hq], dev[:, hq:hq + hkv]
    dq, dk = ddev[:, :hq], ddev[:, hq:hq + hkv]
    dw = [torch.zeros(hd, device="cuda") for _ in range(4)]
    args = (pos.numpy(), EPS, "half", rd, f, m, HALF[dtype])
    c.dflash_norm_rope_grad(pos.cuda(), k=k, k_norm=wd[1], dk_out=dk, dk=torch.empty_like(k), dk_norm=dw[2])
    c.dflash_norm_rope_grad(pos.cuda(), q=q, q_norm=wd[0], dq_out=dq, dq=torch.empty_like(q), dq_norm=dw[3])
    c.dflash_norm_rope_grad(pos.cuda(), q=q, q_norm=wd[0], dq_out=dq, dq=dq, dq_norm=dw[0], k=k, k_norm=wd[1], dk_out=dk, dk=dk,
                            dk_norm=dw[1])
    c.dflash_norm_rope(pos.cuda(), q=q, q_norm=wd[0], q_out=q)
    c.dflash_norm_rope(pos.cuda(), k=k, k_norm=wd[1], k_out=k)
    for i, (a, b, h) in enumerate(((0, hq, hq), (hq, hq + hkv, hkv))):
        y, tol = N.forward(np64(fused[:, a:b]), np64(w[i]), *args)
        check(np64(dev[:, a:b]), y, tol, f"part {i}")
        ex, tx, ew, tw = N.backward(np64(fused[:, a:b]), np64(w[i]), np64(dy[:, a:b]), *args, adds(T, h, hq + hkv - h, hd, lanes(hd, dtype, rd)))
        check(np64(ddev[:, a:b]), ex, tx, f"part {i}: dx")
        check(np64(dw[i]), ew, tw, f"part {i}: dw")
        check(np64(dw[(3, 2)[i]]), ew, tw, f"part {i} alone: dw")
    assert torch.equal(dev[:, hq + hkv:].cpu(), fused[:, hq + hkv:]) and torch.equal(ddev[:, hq + hkv:].cpu(), dy[:, hq + hkv:])
    assert c.dflash_cache_read_status() == 0


def test_gradient_against_differences():
    """The change of sum(c y) along a direction, from two forward calls, is <dx, d> + <dw, e>."""
    T, hq, hd, h = 33, 3, 64, 2.0 ** -7
    c = make(n_head=hq, n_head_kv=1, head_dim=hd, dtype="f32", rope_scaling="yarn", rope_factor=8.0, rope_orig_positions=4096)
    g = torch.Generator(device="cuda").manual_seed(2)
    x, d, cy = (torch.randn(T, hq, hd, generator=g, device="cuda") for _ in range(3))
    w = 1 + 0.3 * torch.randn(hd, generator=g, device="cuda")
    e = torch.randn(hd, generator=g, device="cuda")
    pos = torch.randint(0, 100000, (T,), generator=g, device="cuda", dtype=torch.int32)
    sides = []
    for sign in (1, -1):
        y = torch.empty_like(x)
        c.dflash_norm_rope(pos, q=x + sign * h * d, q_norm=w + sign * h * e, q_out=y)
        sides.append(y.double())
    dx, dw = torch.empty_like(x), torch.empty(hd, device="cuda")
    c.dflash_norm_rope_grad(pos, q=x, q_norm=w, dq_out=cy, dq=dx, dq_norm=dw)
    lhs = float((cy.double() * (sides[0] - sides[1])).sum()) / (2 * h)
    rhs = float((dx.double() * d.double()).sum() + (dw.double() * e.double()).sum())
    # rounding of y and of its inputs: 1e-5 of each value (|w| < 2.2, m < 1.21) over the step; third
    # derivatives of w(t) x(t) / |x(t)|, below 60 (|d| / |x|)^3 with |d| / |x| < 1.6, times h^2 / 6
    scale = float(cy.abs().double().sum())
    assert abs(lhs - rhs) <= scale * (1e-5 * 2.2 * 1.21 / (2 * h) + 60 * 1.6 ** 3 * 2.7 * h * h / 6)
    assert abs(rhs) > 0


def test_negative_position_and_no_rows():
    hd = 64
    c = make(n_head=2, n_head_kv=2, head_dim=hd, dtype="f32")
    g = torch.Generator().manual_seed(0)
    x, dy, w = normal(g, (4, 2, hd), "f32").cuda(), normal(g, (4, 2, hd), "f32").cuda(), weights(g, hd, "f32").cuda()
    out, dx, dw = torch.full_like(x, 7.0), torch.full_like(x, 7.0), torch.zeros(hd, device="cuda")
    pos = ints([3, -1, 0, 5])
    c.dflash_norm_rope(pos, q=x, q_norm=w, q_out=out)
    assert c.dflash_cache_read_status() == 2
    c.dflash_norm_rope_grad(pos, k=x, k_norm=w, dk_out=dy, dk=dx, dk_norm=dw)
    assert c.dflash_cache_read_status() == 2
    for t in (out, dx):
        assert (t[1] == 7.0).all() and not (t[[0, 2, 3]] == 7.0).any()
    keep = [0, 2, 3]
    dx2, dw2 = torch.empty_like(x[keep]), torch.zeros(hd, device="cuda")
    c.dflash_norm_rope_grad(pos[keep], k=x[keep], k_norm=w, dk_out=dy[keep], dk=dx2, dk_norm=dw2)
    assert torch.equal(dx2, dx[keep])
    # the same three rows' terms, in blocks of one row each: additions of the same numbers
    np.testing.assert_allclose(np64(dw), np64(dw2), rtol=0, atol=1e-5)
    dw.fill_(3.0)
    c.dflash_norm_rope(pos[:0], q=x[:0], q_norm=w, q_out=out[:0])
    c.dflash_norm_rope_grad(pos[:0], q=x[:0], q_norm=w, dq_out=dy[:0], dq=dx[:0], dq_norm=dw)
    assert float(dw.abs().sum()) == 0      # a sum over no rows
    assert c.dflash_cache_read_status() == 0


def test_gradient_repeats_bit_for_bit_and_in_a_graph():
    T, hq, hkv, hd = 3001, 8, 2, 128
    c = make(n_head=hq, n_head_kv=hkv, head_dim=hd)
    g = torch.Generator().manual_seed(1)
    q, k, dqo, dko = (normal(g, (T, h, hd), "bf16").cuda() for h in (hq, hkv, hq, hkv))
    wq, wk = weights(g, hd, "bf16").cuda(), weights(g, hd, "bf16").cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")

    def run(o, stream=None):
        c.dflash_norm_rope_grad(pos, q=q, q_norm=wq, dq_out=dqo, dq=o[0], dq_norm=o[1], k=k, k_norm=wk, dk_out=dko, dk=o[2],
                                dk_norm=o[3], stream=stream)

    outs = [[torch.zeros_like(q), torch.zeros(hd, device="cuda"), torch.zeros_like(k), torch.zeros(hd, device="cuda")]
            for _ in range(3)]
    run(outs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(outs[1], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(outs[2])
    graph.replay()
    for o in outs[1:]:
        for a, b in zip(outs[0], o):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,hd,ps,rot,kw", [
    ("bf16", 128, 64, None, {}), ("bf16", 64, 16, 0.5, dict(rope_layout="interleaved")), ("bf16", 32, 16, -8, {}),
    ("f32", 128, 32, None, dict(rope_layout="interleaved")), ("f32", 32, 16, 0, {}),
    ("bf16", 128, 16, None, dict(rope_scaling="yarn", rope_factor=4.0, rope_orig_positions=4096))], ids=str)
@pytest.mark.parametrize("with_q", [True, False])
def test_norm_append(dtype, hd, ps, rot, kw, with_q):
    rng = np.random.default_rng(hd + ps)
    layout = kw.get("rope_layout", "half")
    rd, f, m = rope_setup(hd, layout, rot, kw)
    hq, hkv = 6, 2
    c = make(n_layer=3, n_head=hq, n_head_kv=hkv, head_dim=hd, page_size=ps, n_pages=400, max_seq=7, max_pages=320,
             dtype=dtype, rotary_dim=rd, **kw)
    g = torch.Generator().manual_seed(hd)
    wq, wk = weights(g, hd, dtype), weights(g, hd, dtype)
    for seqs, lens, counts, deep in (([2], [0], [1], False), ([6, 0, 3, 1], [5, 0, ps, 700], [3, 0, 1, 90], True),
                                     ([4, 5], [100, 1], [3000, 333], False)):
        scattered(c, rng, seqs, lens, counts)
        T = sum(counts) + 2
        qkv = normal(g, (T, hq + 2 * hkv, hd), dtype)
        dev = qkv.cuda()
        q, k, v = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]
        trees = [random_parents(rng, n, "random") for n in counts]
        depth = np.concatenate([R.tree_sets(t).sum(1) - 1 if t else np.zeros(0, int) for t in trees] + [[9, 9]]) if deep else None
        before = c.pages.clone()
        q_out = torch.full((T, hq, hd), 3.0, dtype=DT[dtype], device="cuda")
        c.dflash_norm_append(1, starts(counts), k, v, wk.cuda(), depth=ints(depth) if deep else None, q=q if with_q else None,
                             q_norm=wq.cuda() if with_q else None, q_out=q_out if with_q else None, eps=1e-5, seqs=ints(seqs))
        want, table, r = before.clone(), c.table.cpu().tolist(), 0
        for qq, n, cnt in zip(seqs, lens, counts):
            if not cnt:
                continue
            pos = n + (depth[r:r + cnt] if deep else np.arange(cnt))
            args = (pos, 1e-5, layout, rd, f, m, HALF[dtype])
            y, tol = N.forward(np64(qkv[r:r + cnt, hq:hq + hkv]), np64(wk), *args)
            at = torch.arange(n, n + cnt)
            page = torch.as_tensor([table[qq][i] for i in (at // ps).tolist()]).cuda()
            at = (at % ps).cuda()
            stored = c.pages[page, 1, 0, :, at]
            check(np64(stored), y, tol, "keys")
            want[page, 1, 0, :, at] = stored
            want[page, 1, 1, :, at] = v[r:r + cnt]
            if with_q:
                y, tol = N.forward(np64(qkv[r:r + cnt, :hq]), np64(wq), *args)
                check(np64(q_out[r:r + cnt]), y, tol, "queries")
            r += cnt
        assert torch.equal(c.pages, want)                                  # and no other slot
        assert (q_out[r:] == 3.0).all() and torch.equal(dev.cpu(), qkv)
        assert c.dflash_cache_read_status() == 0


@pytest.mark.parametrize("n", [32, 33, 200])
def test_norm_append_of_many_entries(n):
    """Entries that a lane looks through and those that a warp does: the same rows as norm_rope's, faults reported."""
    hq, hkv, hd, ps = 4, 2, 64, 16
    rng = np.random.default_rng(n)
    c = make(n_head=hq, n_head_kv=hkv, head_dim=hd, page_size=ps, n_pages=700, max_seq=256, max_pages=6)
    counts, lens = rng.integers(0, 5, n), rng.integers(0, 40, n)
    seqs = rng.permutation(256)[:n]
    scattered(c, rng, seqs.tolist(), lens.tolist(), counts.tolist())
    seqs[n // 2] = seqs[1]                       # listed twice: the later one does nothing
    T = int(counts.sum()) + 3
    g = torch.Generator().manual_seed(n)
    x = normal(g, (T, hq + 2 * hkv, hd), "bf16").cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    wq, wk = weights(g, hd, "bf16").cuda(), weights(g, hd, "bf16").cuda()
    pos = np.full(T, -1)
    of = np.repeat(np.arange(n), counts)
    for t, s in enumerate(of):
        pos[t] = lens[s] + t - counts[:s].sum()
    dead = (of == n // 2)
    qa, qb, kb = torch.full_like(q, 3.0), torch.full_like(q, 3.0), torch.full_like(k, 3.0)
    c.pages.zero_()
    c.dflash_norm_append(0, starts(counts), k, v, wk, q=q, q_norm=wq, q_out=qa, seqs=ints(seqs))
    assert c.dflash_cache_read_status() == (0x40 if dead.any() else 0)
    pos[:len(of)][dead] = -1
    c.dflash_norm_rope(ints(pos), q=q, q_norm=wq, q_out=qb, k=k, k_norm=wk, k_out=kb)
    c.dflash_cache_read_status()
    assert torch.equal(qa, qb)
    table, want = c.table.cpu().numpy(), torch.zeros_like(c.pages)
    for t, s in enumerate(of):
        if not dead[t]:
            page, at = int(table[seqs[s], pos[t] // ps]), pos[t] % ps
            want[page, 0, 0, :, at], want[page, 0, 1, :, at] = kb[t], v[t]
    assert torch.equal(c.pages, want)


def test_norm_append_agrees_with_norm_rope_and_append():
    """The fused call's keys and queries are those of norm_rope, its faults those of the append."""
    hq, hkv, hd, ps = 8, 2, 128, 16
    c = make(n_head=hq, n_head_kv=hkv, head_dim=hd, page_size=ps, n_pages=20, max_seq=3, max_pages=6)
    rng = np.random.default_rng(0)
    scattered(c, rng, [0, 1], [10, 20], [6, 6])
    c.refs[int(c.table[1, 1])] = 2                # a page that another sequence holds too
    g = torch.Generator().manual_seed(0)
    x = normal(g, (12, hq + 2 * hkv, hd), "bf16").cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    wq, wk = weights(g, hd, "bf16").cuda(), weights(g, hd, "bf16").cuda()
    pos = ints([*range(10, 16), *range(20, 26)])
    q1, q2, k1 = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k)
    c.pages.zero_()
    c.dflash_norm_append(0, starts([6, 6]), k, v, wk, q=q, q_norm=wq, q_out=q1)
    assert c.dflash_cache_read_status() == 0x10
    c.dflash_norm_rope(pos, q=q, q_norm=wq, q_out=q2, k=k, k_norm=wk, k_out=k1)
    assert torch.equal(q1, q2)
    assert torch.equal(c.pages[int(c.table[0, 0]), 0, 0, :, 10:16].transpose(0, 1), k1[:6])
    assert float(c.pages[int(c.table[1, 1])].abs().sum()) == 0


def test_offsets_past_32_bits():
    """Rows behind 4 GB: the last ones, forward and gradient, against 64 bits."""
    hq, hkv, hd, T = 32, 8, 128, 420_001
    c = make(n_head=hq, n_head_kv=hkv, head_dim=hd)
    x = torch.zeros(T, hq + hkv, hd, dtype=torch.bfloat16, device="cuda")
    assert x.numel() * 2 > 1 << 32
    g = torch.Generator().manual_seed(0)
    rows = [0, 1, T // 2, T - 2, T - 1]
    part = normal(g, (len(rows), hq + hkv, hd), "bf16")
    x[rows] = part.cuda()
    w = weights(g, hd, "bf16")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    rd, f, m = rope_setup(hd, "half", None, {})
    args = (np.asarray(rows), EPS, "half", rd, f, m, HALF["bf16"])
    dy = normal(g, (len(rows), hkv, hd), "bf16")
    dys = torch.zeros(T, hkv, hd, dtype=torch.bfloat16, device="cuda")
    dys[rows] = dy.cuda()
    dw = torch.zeros(hd, device="cuda")
    c.dflash_norm_rope_grad(pos, k=x[:, hq:], k_norm=w.cuda(), dk_out=dys, dk=dys, dk_norm=dw)
    ex, tx, ew, tw = N.backward(np64(part[:, hq:]), np64(w), np64(dy), *args, 3000)
    check(np64(dys[rows]), ex, tx, "dx")
    check(np64(dw), ew, tw, "dw")
    c.dflash_norm_rope(pos, q=x[:, :hq], q_norm=w.cuda(), q_out=x[:, :hq], k=x[:, hq:], k_norm=w.cuda(), k_out=x[:, hq:])
    y, tol = N.forward(np64(part), np64(w), *args)
    check(np64(x[rows]), y, tol, "rows")
    assert c.dflash_cache_read_status() == 0


def test_calls_that_the_library_refuses():
    """Bad epsilons, alignments, strides and parts that are not whole return before anything is launched."""
    D = _D()
    c = make(n_head=2, n_head_kv=2, head_dim=64)
    L, h, p = D.LIB, c.h, torch.zeros(4096, device="cuda").data_ptr()

    def rope(T=1, pos=p, eps=1e-6, q=(p, 128, p, p, 128), k=(p, 128, p, p, 128)):
        return L.dflash_norm_rope(h, T, pos, eps, *q, *k, None)

    none = (None, 0, None, None, 0)
    assert rope(T=-1) == rope(pos=None) == rope(eps=0.0) == rope(eps=-1.0) == rope(eps=float("nan")) == rope(eps=float("inf")) == -1
    assert rope(q=none, k=none) == rope(q=(p, 127, p, p, 128)) == rope(q=(p + 2, 128, p, p, 128)) == rope(q=(p, 132, p, p, 128)) == -1
    assert rope(q=(p, 128, None, p, 128)) == rope(q=(p, 128, p + 2, p, 128)) == rope(k=(None, 128, p, p, 128)) == -1
    assert rope(k=(p, 128, p, None, 128)) == rope(k=(p, 128, p, p, 120)) == -1
    assert rope(T=0, q=none, k=none) == 0

    def grad(q=(p, 128, p, p, 128, p, 128, p), k=(None, 0, None, None, 0, None, 0, None), eps=1e-6):
        return L.dflash_norm_rope_grad(h, 1, p, eps, *q, *k, None)

    assert grad(eps=0.0) == grad(q=(p, 128, p, None, 128, p, 128, p)) == grad(q=(p, 128, p, p, 64, p, 128, p)) == -1
    assert grad(q=(p, 128, p, p, 128, p, 128, None)) == grad(q=(p, 128, p, p, 128, p, 128, p + 2)) == -1
    assert grad(q=(None, 0, None, None, 0, None, 0, None)) == -1

    def app(layer=0, eps=1e-6, q=(p, 128, p, p, 128), k=(p, 128, p), n=1):
        return L.dflash_norm_append(h, layer, n, None, p, 1, None, eps, *q, *k, p, 128, None)

    assert app(layer=1) == app(layer=-1) == app(eps=0.0) == app(k=(p, 128, None)) == app(k=(p, 128, p + 4)) == -1
    assert app(q=(p, 128, None, p, 128)) == app(q=(None, 0, p, None, 0)) == app(q=(p, 128, p, None, 0)) == -1
    assert app(n=1025) == -4 and app(n=0) == 0
    assert c.dflash_cache_read_status() == 0
