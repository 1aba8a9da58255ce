"""The operators of a target model's side of speculative decoding, as cases to measure.

The drafter proposes tokens; the target model verifies them as one tree over its own
cache of keys and values.  Four operators do the part of that step that is not a
projection:

  rope    rotary positions of query and key rows (forward, or the gradient), and the
          same fused with the write of the rows' keys and values into the cache pages
  attend  attention of every tree node to its sequence's pages and to its ancestors
  tree    from parent indices to ancestor masks and depths, and the greedy walk that
          accepts a path
  pages   the cache's pages: sharing them with forks of a sequence, private copies
          before a write, release, and the accepted path moved together

A cache is pages[n_pages][n_layer][k, v][n_head_kv][page_size][head_dim], a page table
int32 [max_seq][max_pages] (-1: no page), a length per sequence and a reference count per
page (0: free).  Row t of a call belongs to the sequence whose range of row_start holds it;
row i of a sequence sits in slot length + i.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# --------------------------------------------------------------------- cases

def listed():
    # geometry of the real-dimension drafter's attention: 32 query heads, 8 key/value heads of 128
    real = dict(n_head=32, n_head_kv=8, head_dim=128, page_size=64)
    return [
        # one block of 16 rows (anchor and 15 drafts), query and key heads of a fused projection
        dict(name="rope_block", kind="rope", dtype="bf16", rows=16, heads=40, head_dim=128, rotary_dim=128,
             layout="half", scaling="none", factor=1.0, far=65536, backward=False),
        # the gradient of a training batch's rotation: interleaved pairs on half of each head, stretched positions
        dict(name="rope_grad_f32", kind="rope", dtype="f32", rows=16381, heads=20, head_dim=128, rotary_dim=64,
             layout="interleaved", scaling="yarn", factor=8.0, far=1000000, backward=True),
        # a prompt chunk of one sequence: its fused q/k/v rows rotated, keys and values put into pages
        dict(name="append_prompt", kind="append", dtype="bf16", n_layer=2, n_seq=1, rows_lo=8192, rows_hi=8192,
             len_lo=4096, len_hi=4096, scaling="yarn", factor=4.0, layout="half", rotary_dim=128, **real),
        # one sequence's block verified over the drafter's own window length: the smallest call
        dict(name="attend_block", kind="attend", dtype="bf16", n_seq=1, rows_lo=16, rows_hi=16, len_lo=2048,
             len_hi=2048, tree="chain", **real),
        # continuous batching without drafts: one token of each of 32 sequences of very different lengths
        dict(name="attend_decode", kind="attend", dtype="bf16", n_seq=32, rows_lo=1, rows_hi=1, len_lo=256,
             len_hi=32767, tree="chain", **real),
        # the same batch verifying trees of different sizes
        dict(name="attend_trees", kind="attend", dtype="bf16", n_seq=32, rows_lo=17, rows_hi=64, len_lo=256,
             len_hi=8191, tree="random", **real),
        # a prompt chunk over what is in the cache already
        dict(name="attend_prompt", kind="attend", dtype="bf16", n_seq=1, rows_lo=2047, rows_hi=2047, len_lo=8192,
             len_hi=8192, tree="chain", **real),
        # 32-bit storage: trees of a few sequences
        dict(name="attend_f32", kind="attend", dtype="f32", n_seq=4, rows_lo=9, rows_hi=33, len_lo=1000,
             len_hi=4100, tree="random", **real),
        # the tree of one sequence
        dict(name="tree_one", kind="tree", n_seq=1, rows_lo=26, rows_hi=26, tree="random", vocab=8192),
        # a large batch of trees of every size
        dict(name="tree_batch", kind="tree", n_seq=256, rows_lo=1, rows_hi=128, tree="random", vocab=32768),
        # accepted paths of 32 sequences moved together in all layers of the cache
        dict(name="commit_trees", kind="commit", dtype="bf16", n_layer=32, n_seq=32, rows_lo=17, rows_hi=64,
             len_lo=100, len_hi=130, path=12, **real),
        # 8 sequences forked into 4 beams each, every beam made ready to write, the beams released by the next pass
        dict(name="fork_beams", kind="fork", dtype="bf16", n_layer=16, n_seq=8, beams=3, rows_lo=16, rows_hi=16,
             len_lo=257, len_hi=700, n_head=32, n_head_kv=8, head_dim=128, page_size=64),
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["rope", "append", "attend", "attend", "attend", "tree", "commit", "fork"])
    hd = rng.choice([32, 64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    geo = dict(n_head=hkv * rng.choice([1, 2, 4, 8]), n_head_kv=hkv, head_dim=hd, page_size=rng.choice([16, 32, 64, 128]))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    rot = dict(layout=rng.choice(["half", "interleaved"]), rotary_dim=rng.choice([hd, hd // 2, hd - 8]),
               scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=rng.choice([2.0, 4.0, 8.0]))
    if kind == "rope":
        rows = log_int(rng, 1, 16381)
        return dict(kind=kind, dtype=dtype, rows=rows, heads=rng.randint(1, 40) if rows < 8000 else rng.randint(1, 16),
                    head_dim=hd, far=log_int(rng, 1000, 2000000), backward=rng.random() < 0.5, **rot)
    if kind == "append":
        n = rng.choice([1, 1, 3, 32])
        hi = log_int(rng, 1, 8000 // n)
        lo = max(1, hi // rng.choice([1, 2, 7]))
        ln = log_int(rng, 1, 4000)
        return dict(kind=kind, dtype=dtype, n_layer=rng.choice([1, 2]), n_seq=n, rows_lo=lo, rows_hi=hi, len_lo=ln,
                    len_hi=min(8191, ln * rng.choice([1, 2])), **rot, **geo)
    if kind == "attend":
        shape = rng.choice(["decode", "trees", "prompt"])
        if shape == "decode":
            n, lo, hi, ln = rng.choice([1, 2, 7, 32, 64]), 1, 1, log_int(rng, 1, 16000)
        elif shape == "trees":
            n, hi, ln = rng.choice([1, 2, 5, 16]), log_int(rng, 2, 130), log_int(rng, 1, 8000)
            lo = max(1, hi // rng.choice([1, 2, 3]))
        else:
            n, hi, ln = 1, log_int(rng, 100, 1500), log_int(rng, 1, 6000)
            lo = hi
        if dtype == "f32":
            hi = min(hi, 200)
            lo = min(lo, hi)
            ln = min(ln, 4000)
        case = dict(kind=kind, dtype=dtype, n_seq=n, rows_lo=lo, rows_hi=hi, len_lo=ln, len_hi=ln * rng.choice([1, 2]),
                    tree="random" if shape == "trees" else "chain", **geo)
        while work(case)["bytes"] > 9e8 or work(case)["flops"] > (3e11 if dtype == "bf16" else 2e10):
            case["len_lo"], case["len_hi"] = max(1, case["len_lo"] // 2), max(1, case["len_hi"] // 2)
            case["rows_lo"], case["rows_hi"] = max(1, case["rows_lo"] * 2 // 3), max(1, case["rows_hi"] * 2 // 3)
        return case
    if kind == "tree":
        hi = log_int(rng, 1, 128)
        return dict(kind=kind, n_seq=log_int(rng, 1, 256), rows_lo=max(1, hi // rng.choice([1, 2, 5])), rows_hi=hi,
                    tree=rng.choice(["random", "chain"]), vocab=rng.choice([64, 8192, 32000]))
    if kind == "commit":
        hi = log_int(rng, 2, 64)
        ln = log_int(rng, 1, 150)
        return dict(kind=kind, dtype=dtype, n_layer=rng.choice([1, 3, 8]), n_seq=log_int(rng, 1, 32),
                    rows_lo=max(2, hi // 3), rows_hi=hi, len_lo=ln, len_hi=ln * rng.choice([1, 2]),
                    path=rng.randint(1, 16), **geo)
    ln = log_int(rng, 1, 500)
    return dict(kind="fork", dtype=dtype, n_layer=rng.choice([1, 3, 8]), n_seq=log_int(rng, 1, 16), beams=rng.randint(1, 3),
                rows_lo=1, rows_hi=rng.randint(1, 100), len_lo=ln, len_hi=ln * rng.choice([1, 2]), **geo)


def spread(case):
    """(length, rows) of every sequence: both ranges covered evenly (lengths over their logarithm), whatever the seed."""
    n = case["n_seq"]
    a, b, lo, hi = case.get("len_lo", 1), case.get("len_hi", 1), case["rows_lo"], case["rows_hi"]
    got = []
    for i in range(n):
        f = i / (n - 1) if n > 1 else 1.0
        g = (i * 7919 % n) / (n - 1) if n > 1 else 1.0
        got.append((int(round(a * (b / a) ** f)), int(round(lo + g * (hi - lo)))))
    return got


def pages_of(case):
    """(pages a sequence may hold, pages of the pool)"""
    ps = case["page_size"]
    pairs = spread(case)
    most = max(-(-(a + r) // ps) for a, r in pairs) + 1
    total = sum(-(-(a + r) // ps) for a, r in pairs)
    if case["kind"] == "fork":   # a beam's own pages: the one it copies and those of its new rows
        total += case["n_seq"] * (case["beams"] + 1) * (2 + case["rows_hi"] // ps)
    return most, total + 3


def work(case):
    kind = case["kind"]
    if kind == "rope":
        n = case["rows"] * case["heads"] * case["head_dim"]
        return {"bytes": 2 * n * SIZE[case["dtype"]] + 4 * case["rows"], "flops": 3 * case["rows"] * case["heads"] * case["rotary_dim"]}
    pairs = spread(case)
    rows = sum(r for _, r in pairs)
    if kind == "tree":
        words = -(-case["rows_hi"] // 32)
        return {"bytes": rows * 4 * (1 + words + 1 + 3) + case["n_seq"] * 4 * (3 + case["rows_hi"]), "flops": 0}
    el, hd, hq, hkv = SIZE[case["dtype"]], case["head_dim"], case["n_head"], case["n_head_kv"]
    if kind == "append":   # q, k, v in; q, k, v out
        return {"bytes": 2 * rows * (hq + 2 * hkv) * hd * el, "flops": 3 * rows * (hq + hkv) * case["rotary_dim"]}
    if kind == "attend":
        words = -(-case["rows_hi"] // 32)
        slots = sum(a + r for a, r in pairs)
        seen = sum(r * a + (r * (r + 1) // 2 if case["tree"] == "chain" else tree_pairs(r)) for a, r in pairs)
        return {"bytes": 2 * slots * hkv * hd * el + 2 * rows * hq * hd * el + rows * hq * 4 +
                (0 if case["tree"] == "chain" else 4 * rows * words), "flops": 4 * seen * hq * hd}
    token = case["n_layer"] * 2 * hkv * hd * el
    if kind == "commit":   # the anchor stays where it is, every other accepted token is read and written once
        return {"bytes": 2 * token * sum(min(case["path"], r) - 1 for _, r in pairs) + 4 * case["n_seq"] * (case["path"] + 2),
                "flops": 0}
    ps, most = case["page_size"], pages_of(case)[0]
    copied = sum((a % ps) * case["beams"] for a, _ in pairs)   # every holder of the last, part-filled page but one
    entries = sum(-(-(a + r) // ps) for a, r in pairs) * case["beams"]
    return {"bytes": 2 * token * copied + 4 * 4 * entries + 4 * most, "flops": 0}


def tree_pairs(r):
    """Expected (node, ancestor or self) pairs of a random recursive tree of r nodes: sum of harmonic numbers."""
    h, s = 0.0, 0.0
    for i in range(1, r + 1):
        h += 1.0 / i
        s += h
    return int(s)


# -------------------------------------------------------------------- inputs

def draw_trees(counts, tree, g):
    """Parents of every row (index within its own tree, -1: the root), trees one after another."""
    idx = torch.cat([torch.arange(c) for c in counts])
    if tree == "chain":
        return (idx - 1).to(torch.int32).to(DEV)
    u = torch.rand(len(idx), generator=g)
    return ((u * idx).floor().to(torch.int32) - (idx == 0).to(torch.int32)).to(DEV)


def prepare(case, seed):
    kind = case["kind"]
    host = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=TORCH[case["dtype"]])

    if kind == "rope":
        rows, heads, hd = case["rows"], case["heads"], case["head_dim"]
        s["x"] = normal(rows, heads, hd)
        s["pos"] = torch.randint(0, case["far"], (rows,), generator=g, device=DEV, dtype=torch.int32)
        s["out"] = torch.empty_like(s["x"])
        if own:
            s["cache"] = cache_of(dict(case, n_layer=1, n_head=heads, n_head_kv=heads, page_size=16), 1, 1, 1)
        return s

    pairs = spread(case)
    order = torch.randperm(len(pairs), generator=host).tolist()
    lens, counts = [pairs[i][0] for i in order], [pairs[i][1] for i in order]
    n, rows, most = case["n_seq"], sum(counts), max(counts)
    s["counts"], s["lens"], s["most"] = counts, lens, most
    s["row_start"] = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).to(DEV)
    if kind in ("tree", "attend"):
        s["parents"] = draw_trees(counts, case["tree"], host)
    words = -(-case["rows_hi"] // 32)
    if kind == "tree":
        s["tokens"] = torch.randint(0, case["vocab"], (rows,), generator=g, device=DEV, dtype=torch.int32)
        # the target agrees with one child of most nodes
        base = s["row_start"][:-1].long().repeat_interleave(torch.tensor(counts, device=DEV), output_size=rows)
        at = torch.where(s["parents"] < 0, rows, s["parents"].long() + base)
        child = torch.zeros(rows + 1, dtype=torch.int64, device=DEV)
        child.scatter_reduce_(0, at, torch.arange(rows, device=DEV), "amax")
        agree = torch.rand(rows, generator=g, device=DEV) < 0.8
        other = torch.randint(0, case["vocab"], (rows,), generator=g, device=DEV, dtype=torch.int32)
        s["targets"] = torch.where(agree & (child[:rows] > 0), s["tokens"][child[:rows]], other)
        s["mask"] = torch.empty(rows, words, dtype=torch.int32, device=DEV)
        s["depth"] = torch.empty(rows, dtype=torch.int32, device=DEV)
        s["path"] = torch.empty(n, case["rows_hi"], dtype=torch.int32, device=DEV)
        s["n_path"] = torch.empty(n, dtype=torch.int32, device=DEV)
        s["id_last"] = torch.zeros(n, dtype=torch.int32, device=DEV)
        if own:
            s["cache"] = cache_of(dict(n_layer=1, n_head=1, n_head_kv=1, head_dim=32, page_size=16, dtype="bf16"), n, 1, 1)
        return s

    ps, L, hkv, hd = case["page_size"], case.get("n_layer", 1), case["n_head_kv"], case["head_dim"]
    most_pages, n_pages = pages_of(case)
    n_all = n * (1 + case.get("beams", 0))
    held = [-(-(a + (0 if kind == "fork" else c)) // ps) for a, c in zip(lens, counts)]
    ids = torch.randperm(n_pages, generator=host)[:sum(held)].to(torch.int32)
    table = torch.full((n_all, most_pages), -1, dtype=torch.int32)
    # the sequences of the call lie anywhere in the table
    seqs = torch.randperm(n_all, generator=host)
    at = 0
    for q, h in zip(seqs[:n].tolist(), held):
        table[q, :h] = ids[at:at + h]
        at += h
    refs = torch.zeros(n_pages, dtype=torch.int32)
    refs[ids.long()] = 1
    length = torch.zeros(n_all, dtype=torch.int32)
    length[seqs[:n]] = torch.tensor(lens, dtype=torch.int32)
    if own:
        s["cache"] = c = cache_of(case, n_all, most_pages, n_pages)
        s["pages"], s["table"], s["length"], s["refs"] = c.pages, c.table, c.length, c.refs
    else:
        s["pages"] = torch.empty(n_pages, L, 2, hkv, ps, hd, dtype=TORCH[case["dtype"]], device=DEV)
        s["table"], s["length"], s["refs"] = (torch.empty_like(t, device=DEV) for t in (table, length, refs))
    s["pages"].normal_(generator=g)
    s["table"].copy_(table)
    s["length"].copy_(length)
    s["refs"].copy_(refs)
    s["start_length"] = length.to(DEV)
    s["seqs"] = seqs[:n].to(torch.int32).to(DEV)
    if kind in ("append", "attend"):
        s["layer"] = L - 1
        hq = case["n_head"]
    if kind == "append":   # one row holds q, k and v, as the fused projection leaves them
        qkv = normal(rows, hq + 2 * hkv, hd)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_out"] = torch.empty(rows, hq, hd, dtype=qkv.dtype, device=DEV)
    if kind == "attend":
        s["q"] = normal(rows, hq, hd)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(rows, hq, dtype=torch.float32, device=DEV)
        s["mask"] = None
        if case["tree"] != "chain":
            m, row, real = ancestors(s["parents"], s["row_start"], most)
            s["mask"] = flat(tree_words(m, words), row, real, rows)
    if kind == "commit":   # ascending nodes that begin with the anchor
        m = case["path"]
        path = torch.full((n, m), -1, dtype=torch.int32)
        n_path = []
        for i, c in enumerate(counts):
            k = min(m, c)
            rest = (torch.randperm(c - 1, generator=host)[:k - 1] + 1).sort().values
            path[i, :k] = torch.cat([torch.zeros(1, dtype=torch.int64), rest]).to(torch.int32)
            n_path.append(k)
        s["path"], s["n_path"] = path.to(DEV), torch.tensor(n_path, dtype=torch.int32).to(DEV)
    if kind == "fork":
        b = case["beams"]
        s["src"] = s["seqs"].repeat_interleave(b)
        s["dst"] = seqs[n:].to(torch.int32).to(DEV)
        s["every"] = torch.cat([s["seqs"], s["dst"]])
        s["none"] = torch.zeros(n * b, dtype=torch.int32, device=DEV)
        s["ask"] = torch.cat([torch.tensor(counts, dtype=torch.int32).to(DEV),
                              torch.tensor(counts, dtype=torch.int32).to(DEV).repeat_interleave(b)])
    return s


def cache_of(case, max_seq, max_pages, n_pages):
    from block_diffusion_drafter_fc_gb300.dflash import CacheConfig, PagedCache
    return PagedCache(CacheConfig(
        n_layer=case.get("n_layer", 1), n_head=case["n_head"], n_head_kv=case["n_head_kv"], head_dim=case["head_dim"],
        page_size=case["page_size"], n_pages=n_pages, max_seq=max_seq, max_pages=max_pages, dtype=case["dtype"],
        rope_layout=case.get("layout", "half"), rotary_dim=case.get("rotary_dim", case["head_dim"]),
        rope_theta=1e6, rope_scaling=case.get("scaling", "none"), rope_factor=case.get("factor", 1.0),
        rope_orig_positions=32768))


# --------------------------------------------------------------- plain forms

def inv_freq(case):
    """(angle per position of every rotated pair, in 64 bits; factor of the rotated values)"""
    rd, f, theta, orig = case["rotary_dim"], case["factor"], 1e6, 32768
    j = torch.arange(rd // 2, dtype=torch.float64, device=DEV)
    if case["scaling"] == "ntk":   # the base stretched so that the slowest pair is slowed by the factor
        theta = theta * f ** (rd / (rd - 2))
    inv = theta ** (-2 * j / rd)
    if case["scaling"] == "linear":
        return inv / f, 1.0
    if case["scaling"] != "yarn":
        return inv, 1.0
    # pairs that turn more than 32 times over the original positions keep their angle, those that turn less than
    # once are slowed by the factor, a ramp between them
    at = [rd * math.log(orig / (t * 2 * math.pi)) / (2 * math.log(theta)) for t in (32.0, 1.0)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rd - 1)
    slow = ((j - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return inv / f * slow + inv * (1 - slow), 0.1 * math.log(f) + 1.0


def rotate(x, pos, case, backward):
    """Rotated x [T][heads][head_dim]: pair (a, b) at angle t -> (a cos t - b sin t, b cos t + a sin t), or its gradient."""
    rd = case["rotary_dim"]
    inv, m = inv_freq(case)
    angle = pos.double()[:, None] * inv
    cos, sin = (angle.cos() * m).float()[:, None], (angle.sin() * m).float()[:, None]
    if backward:
        sin = -sin
    y = x.float()
    if case["layout"] == "half":
        a, b = y[..., :rd // 2], y[..., rd // 2:rd]
        z = torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., rd:]], -1)
    else:
        a, b = y[..., 0:rd:2], y[..., 1:rd:2]
        z = torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), y[..., rd:]], -1)
    return z.to(x.dtype)


def row_sequence(row_start, rows):
    return torch.searchsorted(row_start, torch.arange(rows, device=DEV, dtype=torch.int32), right=True) - 1


def ancestors(parents, row_start, most):
    """(ancestor-or-self [sequence][node][node], row of every node, whether it exists)"""
    idx = torch.arange(most, device=DEV)
    row = row_start[:-1, None] + idx
    real = row < row_start[1:, None]
    row = torch.where(real, row, 0).long()
    p = torch.where(real, parents[row], -1)
    m = (p[..., None] == idx).float() + torch.eye(most, device=DEV)
    for _ in range(max(1, (most - 1).bit_length())):   # each squaring doubles the distance that is covered
        m = ((m @ m) > 0).float()
    return m > 0, row, real


def tree_words(m, words):
    """The nodes' masks [sequence][node][node] as 32-bit words."""
    n, most = m.shape[:2]
    bits = torch.nn.functional.pad(m.long(), (0, words * 32 - most)).view(n, most, words, 32)
    w = (bits << torch.arange(32, device=DEV)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def flat(x, row, real, rows):
    """Values [sequence][node]... put into their rows."""
    out = x.new_zeros((rows + 1,) + x.shape[2:])
    out[torch.where(real, row, rows)] = x
    return out[:rows]


def attend(s):
    case = s["case"]
    hq, hkv, hd, ps = case["n_head"], case["n_head_kv"], case["head_dim"], case["page_size"]
    q, n = s["q"], case["n_seq"]
    rows, most = q.shape[0], s["most"]
    idx = torch.arange(most, device=DEV)
    row = s["row_start"][:-1, None] + idx
    real = row < s["row_start"][1:, None]
    row = torch.where(real, row, 0).long()
    length = s["length"][s["seqs"].long()].long()
    n_pages = max(-(-(a + c) // ps) for a, c in zip(s["lens"], s["counts"]))
    held = s["table"][s["seqs"].long(), :n_pages].clamp(min=0).long()
    kv = s["pages"][:, s["layer"]][held].transpose(1, 2).transpose(2, 3)       # [n][k, v][head][page][slot][dim]
    k, v = (kv[:, i].reshape(n, hkv, n_pages * ps, hd).float() for i in (0, 1))
    slot = torch.arange(n_pages * ps, device=DEV)
    node = slot - length[:, None]                                               # [n][slots]
    if s["mask"] is None:
        sees = node[:, None] <= idx[:, None]
    else:
        w = s["mask"][row]                                                      # [n][most][words]
        at = node.clamp(0, 32 * w.shape[-1] - 1)[:, None].expand(-1, most, -1)
        sees = (node[:, None] < 0) | ((w.gather(2, at // 32) >> (at % 32)) & 1).bool()
    counts = s["row_start"][1:] - s["row_start"][:-1]
    sees = sees & (node < counts[:, None])[:, None]
    qs = q[row].float().view(n, most, hkv, hq // hkv, hd).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, hd)
    sc = (qs @ k.transpose(2, 3)).view(n, hkv, hq // hkv, most, -1) * hd ** -0.5
    sc = sc.masked_fill(~sees[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    e = (sc - torch.where(top == -math.inf, 0.0, top)).exp()
    total = e.sum(-1, keepdim=True)
    o = (e.view(n, hkv, -1, e.shape[-1]) @ v).view(n, hkv, hq // hkv, most, hd) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    o, lse = o.permute(0, 3, 1, 2, 4).reshape(n, most, hq, hd), lse.permute(0, 3, 1, 2).reshape(n, most, hq)
    return flat(o.to(q.dtype), row, real, rows), flat(lse, row, real, rows)


def accept(parents, tokens, targets, row_start, most, start_id):
    m, row, real = ancestors(parents, row_start, most)
    p, tok = torch.where(real, parents[row], -2), tokens[row]
    idx = torch.arange(most, device=DEV)
    agrees = tok == targets[row].gather(1, p.clamp(min=0).long())
    # of equal children the first one is the node that the walk takes
    again = ((p[:, :, None] == p[:, None]) & (tok[:, :, None] == tok[:, None]) & (idx[None] < idx[:, None])).any(-1)
    good = ((agrees & (p >= 0) & ~again) | (idx == 0)) & real
    taken = real & ~(m & ~good[:, None]).any(-1)
    n_path = taken.sum(1).to(torch.int32)
    path = torch.where(taken, idx, most).sort(1).values
    last = torch.where(taken, idx, 0).amax(1, keepdim=True)
    id_last = torch.where(n_path > 0, targets[row].gather(1, last)[:, 0], start_id)
    return torch.where(path < most, path, -1).to(torch.int32), n_path, id_last, m, row, real


def slots_of(table, seqs, slot, ps):
    """(page, place in it) of slots [n][k] of sequences [n]"""
    return table[seqs.long()[:, None], (slot // ps)].long(), slot % ps


def reserve(s, seqs, ask):
    table, length, refs, pages = s["table"], s["length"], s["refs"], s["pages"]
    ps = s["case"]["page_size"]
    q = seqs.long()
    ln, held = length[q].long(), table[q]
    idx = torch.arange(table.shape[1], device=DEV)
    first = (ln // ps)
    inside = (idx >= first[:, None]) & (idx <= ((ln + ask - 1) // ps)[:, None]) & (ask > 0)[:, None]
    old = held.gather(1, first.clamp(max=table.shape[1] - 1)[:, None])[:, 0].long()
    part = (ln % ps != 0) & (ask > 0) & (old >= 0)
    safe = old.clamp(min=0)
    same = (old[:, None] == old) & part[:, None] & part
    earlier = same.tril(-1).sum(1)
    copies = part & (refs[safe] - earlier > 1)
    need = inside & ((held < 0) | ((idx == first[:, None]) & copies[:, None]))
    free = (refs != 0).to(torch.int32).sort(stable=True).indices
    rank = need.flatten().cumsum(0).view_as(need) - 1
    new = torch.where(need, free[rank.clamp(0, len(free) - 1)].to(torch.int32), held)
    refs.index_add_(0, safe, -copies.to(torch.int32))
    refs.index_add_(0, new.clamp(min=0).flatten().long(), need.flatten().to(torch.int32))
    table[q] = new
    # what the sequence holds of its part-filled page goes into the new one
    to = torch.where(copies, new.gather(1, first.clamp(max=table.shape[1] - 1)[:, None])[:, 0].long(), safe)
    keep = (torch.arange(ps, device=DEV) < (ln % ps)[:, None])[:, None, None, None, :, None]
    pages[to] = torch.where(keep, pages[safe], pages[to])


def run(s):
    case, kind = s["case"], s["case"]["kind"]
    if kind == "rope":
        if own:
            s["cache"].dflash_rope(s["x"], s["pos"], s["out"], backward=case["backward"])
            return s["out"]
        return rotate(s["x"], s["pos"], case, case["backward"])

    if kind == "tree":
        if own:
            c = s["cache"]
            c.dflash_tree_mask(s["row_start"], s["parents"], s["mask"], s["depth"])
            c.dflash_tree_accept(s["row_start"], s["parents"], s["tokens"], s["targets"], s["path"], s["n_path"], s["id_last"])
            return {k: s[k] for k in ("mask", "depth", "path", "n_path", "id_last")}
        path, n_path, id_last, m, row, real = accept(s["parents"], s["tokens"], s["targets"], s["row_start"], s["most"], s["id_last"])
        rows = s["parents"].shape[0]
        path = torch.nn.functional.pad(path, (0, s["path"].shape[1] - path.shape[1]), value=-1)
        return {"mask": flat(tree_words(m, s["mask"].shape[1]), row, real, rows),
                "depth": flat((m.sum(-1) - 1).to(torch.int32), row, real, rows), "path": path, "n_path": n_path,
                "id_last": id_last}

    ps = case["page_size"]
    if kind == "append":
        if own:
            s["cache"].dflash_cache_append(s["layer"], s["row_start"], s["k"], s["v"], q=s["q"], q_out=s["q_out"], seqs=s["seqs"])
            return s["q_out"], s["pages"]
        rows = s["k"].shape[0]
        of = row_sequence(s["row_start"], rows)
        slot = s["length"][s["seqs"].long()[of].long()].long() + torch.arange(rows, device=DEV) - s["row_start"][of]
        page, at = slots_of(s["table"], s["seqs"][of], slot[:, None], ps)
        s["pages"][page[:, 0], s["layer"], 0, :, at[:, 0]] = rotate(s["k"], slot, case, False)
        s["pages"][page[:, 0], s["layer"], 1, :, at[:, 0]] = s["v"]
        return rotate(s["q"], slot, case, False), s["pages"]

    if kind == "attend":
        if own:
            s["cache"].dflash_tree_attend(s["layer"], s["row_start"], s["most"], s["q"], s["out"], mask=s["mask"],
                                          lse=s["lse"], seqs=s["seqs"])
            return s["out"], s["lse"]
        return attend(s)

    if kind == "commit":
        s["length"].copy_(s["start_length"])   # the same step again
        if own:
            s["cache"].dflash_cache_commit(s["path"], s["n_path"], seqs=s["seqs"])
            return s["pages"], s["length"]
        q = s["seqs"].long()
        ln = s["length"][q].long()[:, None]
        j = torch.arange(s["path"].shape[1], device=DEV)
        there = j < s["n_path"][:, None]
        page, at = slots_of(s["table"], s["seqs"], ln + torch.where(there, s["path"], 0), ps)
        page_to, at_to = slots_of(s["table"], s["seqs"], ln + torch.where(there, j, 0), ps)
        s["pages"][page_to, :, :, :, at_to] = s["pages"][page, :, :, :, at]
        s["length"][q] += s["n_path"]
        return s["pages"], s["length"]

    if own:
        c = s["cache"]
        c.dflash_cache_trim(s["none"], seqs=s["dst"])
        c.dflash_cache_fork(s["src"], s["dst"])
        c.dflash_cache_reserve(s["ask"], seqs=s["every"])
        return s["pages"], s["table"], s["length"], s["refs"]
    table, length, refs = s["table"], s["length"], s["refs"]
    src, dst = s["src"].long(), s["dst"].long()
    idx = torch.arange(table.shape[1], device=DEV)
    gone = table[dst]                                       # release: nothing of the beams is kept
    refs.index_add_(0, gone.clamp(min=0).flatten().long(), -(gone >= 0).flatten().to(torch.int32))
    held = torch.where(idx < -(-length[src] // ps)[:, None], table[src], -1)
    table[dst] = held                                       # fork: the pages are shared
    refs.index_add_(0, held.clamp(min=0).flatten().long(), (held >= 0).flatten().to(torch.int32))
    length[dst] = length[src]
    reserve(s, s["every"], s["ask"])
    return s["pages"], table, length, refs


# ---------------------------------------------------------------- definition

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    kind = case["kind"]

    def turned(x, pos, backward=False):
        """Rotation by complex numbers: a + ib times m e^(it)."""
        rd = case["rotary_dim"]
        freq = []
        for j in range(rd // 2):
            base = 1e6
            if case["scaling"] == "ntk":
                base *= case["factor"] ** (rd / (rd - 2.0))
            f = base ** (-2.0 * j / rd)
            if case["scaling"] == "linear":
                f /= case["factor"]
            if case["scaling"] == "yarn":
                lo = max(math.floor(rd * math.log(32768 / (32 * 2 * math.pi)) / (2 * math.log(base))), 0)
                hi = min(math.ceil(rd * math.log(32768 / (2 * math.pi)) / (2 * math.log(base))), rd - 1)
                w = min(max((j - lo) / max(hi - lo, 0.001), 0.0), 1.0)
                f = w * f / case["factor"] + (1 - w) * f
            freq.append(f)
        m = 0.1 * math.log(case["factor"]) + 1 if case["scaling"] == "yarn" else 1.0
        t = pos.double()[:, None, None] * torch.tensor(freq, dtype=torch.float64, device=DEV)
        z = torch.polar(torch.full_like(t, m), -t if backward else t)
        y = x.double().clone()
        a, b = (slice(0, rd // 2), slice(rd // 2, rd)) if case["layout"] == "half" else (slice(0, rd, 2), slice(1, rd, 2))
        w = torch.complex(y[..., a], y[..., b]) * z
        y[..., a], y[..., b] = w.real, w.imag
        return y

    if kind == "rope":
        return turned(s["x"], s["pos"], case["backward"])
    if kind == "append":
        pages, ps = s["pages"].double(), case["page_size"]
        q_out = torch.empty(s["q_out"].shape, dtype=torch.float64, device=DEV)
        r0 = 0
        for q, ln, c in zip(s["seqs"].tolist(), s["lens"], s["counts"]):
            pos = torch.arange(ln, ln + c, device=DEV)
            q_out[r0:r0 + c] = turned(s["q"][r0:r0 + c], pos)
            k, v = turned(s["k"][r0:r0 + c], pos), s["v"][r0:r0 + c].double()
            for p in range(ln // ps, (ln + c - 1) // ps + 1):
                a, b = max(ln, p * ps), min(ln + c, (p + 1) * ps)
                to = pages[int(s["table"][q, p]), s["layer"]]
                to[0][:, a - p * ps:b - p * ps] = k[a - ln:b - ln].transpose(0, 1)
                to[1][:, a - p * ps:b - p * ps] = v[a - ln:b - ln].transpose(0, 1)
            r0 += c
        return q_out, pages
    if kind == "attend":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.empty(s["lse"].shape, dtype=torch.float64, device=DEV)
        hq, hkv, hd, ps = case["n_head"], case["n_head_kv"], case["head_dim"], case["page_size"]
        parents = s["parents"].tolist()
        r0 = 0
        for q, ln, c in zip(s["seqs"].tolist(), s["lens"], s["counts"]):
            sees = torch.ones(c, ln + c, dtype=torch.bool)
            tree = torch.zeros(c, c, dtype=torch.bool)
            for i in range(c):
                p = parents[r0 + i]
                if p >= 0:
                    tree[i] = tree[p]
                tree[i, i] = True
            sees[:, ln:] = tree
            sees = sees.to(DEV)
            held = s["table"][q, :-(-(ln + c) // ps)].long()
            for h in range(hq):
                kv = s["pages"][held, s["layer"], :, h // (hq // hkv)].double()
                k, v = (kv[:, i].reshape(-1, hd)[:ln + c] for i in (0, 1))
                sc = (s["q"][r0:r0 + c, h].double() @ k.T / math.sqrt(hd)).masked_fill(~sees, -math.inf)
                out[r0:r0 + c, h] = sc.softmax(-1) @ v
                lse[r0:r0 + c, h] = sc.logsumexp(-1)
            r0 += c
        return out, lse
    if kind == "commit":
        pages, length, ps = s["pages"].clone(), s["length"].clone(), case["page_size"]
        table = s["table"].tolist()
        for i, (q, ln) in enumerate(zip(s["seqs"].tolist(), s["lens"])):
            for j, node in enumerate(s["path"][i].tolist()[:int(s["n_path"][i])]):
                a, b = ln + node, ln + j
                pages[table[q][b // ps], :, :, :, b % ps] = pages[table[q][a // ps], :, :, :, a % ps]
            length[q] = ln + int(s["n_path"][i])
        return pages.double(), length
    if kind == "fork":
        pages, ps = s["pages"].clone(), case["page_size"]
        table, length, refs = s["table"].tolist(), s["length"].tolist(), s["refs"].tolist()
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            length[b] = length[a]
            for p in range(-(-length[a] // ps)):
                table[b][p] = table[a][p]
                refs[table[a][p]] += 1
        free = [p for p, r in enumerate(refs) if not r]
        for q, ask in zip(s["every"].tolist(), s["ask"].tolist()):
            for p in range(length[q] // ps, (length[q] + ask - 1) // ps + 1):
                had, fill = table[q][p], length[q] - p * ps
                if had >= 0 and not (fill > 0 and refs[had] > 1):
                    continue
                table[q][p] = free.pop(0)
                refs[table[q][p]] = 1
                if had >= 0:
                    refs[had] -= 1
                    pages[table[q][p], :, :, :, :fill] = pages[had, :, :, :, :fill]
        return pages.double(), *(torch.tensor(t, dtype=torch.int32, device=DEV) for t in (table, length, refs))
    return None
