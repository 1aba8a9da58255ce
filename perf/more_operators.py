"""Operators for sampled verification of several continuations of one prompt, as cases to measure.

A target model that normalises every head of its queries and keys, several continuations of
one prompt that share the pages of their common beginning, and drafts that are drawn from
the drafter's probabilities and verified against the target's:

  norm    norm of every query and key head with the position rotation in the same pass
          (forward, gradient, and fused with the write of keys and values into the pages)
  prefix  attention of a batch over a paged cache where groups of sequences share the pages
          of a long beginning, which is read and multiplied once for all of a group's rows
  verify  drafted tokens (chains or trees) against the target's probabilities, with given
          random numbers: the accepted path and the token behind it
  sample  one token of every row of logits, with given random numbers (what draws drafts)

Token i is drawn from weights r as the largest r_i / e_i, e_i given exponential variates
(a race of exponential clocks: i wins with probability r_i / sum r).  A drafted token x of
distribution q is accepted when u q(x) < r(x); otherwise r becomes max(r - q, 0) normalised.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6


# --------------------------------------------------------------------- cases

def listed():
    # geometry of the real-dimension drafter's attention: 32 query heads, 8 key/value heads of 128
    real = dict(n_head=32, n_head_kv=8, head_dim=128, page_size=64)
    rot = dict(rotary_dim=128, layout="half", scaling="none", factor=1.0)
    return [
        # one verified block of 16 rows, queries and keys as the fused projection leaves them
        dict(name="norm_block", kind="norm", dtype="bf16", rows=16, far=65536, backward=False, **rot, **real),
        # the gradient of a training batch: every token of 8 sequences of about 1000
        dict(name="norm_grad", kind="norm", dtype="bf16", rows=8191, far=4096, backward=True, **rot, **real),
        # a prompt chunk of one sequence put into the cache, keys and queries normalised and rotated
        dict(name="norm_append", kind="append", dtype="bf16", n_layer=2, n_seq=1, rows_lo=8192, rows_hi=8192, len_lo=4096,
             len_hi=4096, **dict(rot, scaling="yarn", factor=4.0), **real),
        # four samples of one short prompt, one token each: the smallest call, where latency counts
        dict(name="prefix_small", kind="prefix", dtype="bf16", groups=1, members=4, shared=1000, tail_lo=0, tail_hi=40,
             rows_lo=1, rows_hi=1, tree="chain", **real),
        # 32 samples of one long prompt, one token each
        dict(name="prefix_decode", kind="prefix", dtype="bf16", groups=1, members=32, shared=16384, tail_lo=1, tail_hi=700,
             rows_lo=1, rows_hi=1, tree="chain", **real),
        # four prompts of eight continuations each, trees of drafts verified in all of them
        dict(name="prefix_trees", kind="prefix", dtype="bf16", groups=4, members=8, shared=8000, tail_lo=1, tail_hi=500,
             rows_lo=9, rows_hi=33, tree="random", **real),
        # 32-bit storage: beams of one prompt
        dict(name="prefix_f32", kind="prefix", dtype="f32", groups=1, members=4, shared=4001, tail_lo=1, tail_hi=130,
             rows_lo=1, rows_hi=1, tree="chain", **real),
        # one block of one sequence whose drafts are argmaxes (no draft distribution), 16-bit logits
        dict(name="verify_one", kind="verify", dtype="bf16", n_seq=1, rows_lo=16, rows_hi=16, tree="chain", vocab=8192,
             drafts="argmax"),
        # a batch of blocks whose drafts were drawn from the drafter's logits
        dict(name="verify_chains", kind="verify", dtype="f32", n_seq=32, rows_lo=16, rows_hi=16, tree="chain", vocab=32768,
             drafts="drawn"),
        # trees of drafts, siblings drawn from one distribution, of a target with a large odd vocabulary
        dict(name="verify_trees", kind="verify", dtype="f32", n_seq=8, rows_lo=9, rows_hi=33, tree="random", vocab=100003,
             drafts="drawn"),
        # the drafts of one block
        dict(name="sample_block", kind="sample", dtype="f32", rows=15, vocab=8192),
        # the drafts of 32 blocks
        dict(name="sample_batch", kind="sample", dtype="f32", rows=480, vocab=32768),
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["norm", "append", "prefix", "prefix", "verify", "verify", "sample"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "sample":
        vocab = log_int(rng, 2, 150000)
        return dict(kind=kind, dtype=dtype, rows=log_int(rng, 1, max(2, min(2000, 15000000 // vocab))), vocab=vocab)
    if kind == "verify":
        vocab = log_int(rng, 2, 150000)
        hi = log_int(rng, 1, 64)
        return dict(kind=kind, dtype=dtype, n_seq=log_int(rng, 1, max(2, min(200, 16000000 // (vocab * hi)))),
                    rows_lo=max(1, hi // rng.choice([1, 2, 5])), rows_hi=hi, tree=rng.choice(["chain", "random"]), vocab=vocab,
                    drafts=rng.choice(["drawn", "drawn", "argmax"]))
    hd = rng.choice([32, 64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    geo = dict(n_head=hkv * rng.choice([1, 2, 4, 8]), n_head_kv=hkv, head_dim=hd, page_size=rng.choice([16, 32, 64, 128]))
    rot = dict(layout=rng.choice(["half", "interleaved"]), rotary_dim=rng.choice([hd, hd // 2, hd - 8]),
               scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=rng.choice([2.0, 4.0, 8.0]))
    if kind == "norm":
        case = dict(kind=kind, dtype=dtype, rows=log_int(rng, 1, 16381), far=log_int(rng, 1000, 2000000),
                    backward=rng.random() < 0.6, **rot, **geo)
        while work(case)["bytes"] > 1.8e8:
            case["rows"] //= 2
        return case
    if kind == "append":
        n = rng.choice([1, 1, 3, 32])
        hi = log_int(rng, 1, 4000 // n)
        ln = log_int(rng, 1, 4000)
        case = dict(kind=kind, dtype=dtype, n_layer=rng.choice([1, 2]), n_seq=n, rows_lo=max(1, hi // rng.choice([1, 2, 7])),
                    rows_hi=hi, len_lo=ln, len_hi=min(8191, ln * rng.choice([1, 2])), **rot, **geo)
        while work(case)["bytes"] > 1.8e8:
            case["rows_lo"], case["rows_hi"] = max(1, case["rows_lo"] // 2), max(1, case["rows_hi"] // 2)
        return case
    tree = rng.choice(["chain", "random"])
    hi = rng.choice([1, 1, log_int(rng, 2, 40)]) if tree == "chain" else log_int(rng, 2, 60)
    tail = log_int(rng, 1, 1000)
    case = dict(kind=kind, dtype=dtype, groups=rng.choice([1, 1, 2, 5]), members=rng.randint(1, 24), shared=log_int(rng, 1, 12000),
                tail_lo=rng.choice([0, tail // 3]), tail_hi=tail, rows_lo=max(1, hi // rng.choice([1, 2, 3])), rows_hi=hi,
                tree=tree, **geo)
    while work(case)["bytes"] > 1e8 or work(case)["flops"] > (4e10 if dtype == "bf16" else 2e9):
        case["shared"], case["members"] = max(1, case["shared"] // 2), max(1, case["members"] * 2 // 3)
        case["rows_lo"], case["rows_hi"] = max(1, case["rows_lo"] // 2), max(1, case["rows_hi"] // 2)
    return case


def even(n, lo, hi, step=7919):
    """n values that cover lo..hi evenly, in an order of their own."""
    return [int(round(lo + (i * step % n) / (n - 1) * (hi - lo))) if n > 1 else hi for i in range(n)]


def shapes(case):
    """(length, rows) of every sequence, whatever the seed."""
    if case["kind"] == "prefix":
        n = case["groups"] * case["members"]
        return [(case["shared"] + a, r) for a, r in zip(even(n, case["tail_lo"], case["tail_hi"]),
                                                        even(n, case["rows_lo"], case["rows_hi"], 104729))]
    n = case["n_seq"]
    return list(zip(even(n, case.get("len_lo", 0), case.get("len_hi", 0)), even(n, case["rows_lo"], case["rows_hi"], 104729)))


def work(case):
    kind, el = case["kind"], SIZE[case["dtype"]]
    if kind == "norm":
        n = case["rows"] * (case["n_head"] + case["n_head_kv"]) * case["head_dim"]
        return {"bytes": (3 if case["backward"] else 2) * n * el + 4 * case["rows"], "flops": (16 if case["backward"] else 8) * n}
    if kind == "sample":   # logits and variates
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (el + 4) + 8 * case["rows"], "flops": 4 * n}
    pairs = shapes(case)
    rows = sum(r for _, r in pairs)
    if kind == "verify":   # the target's logits, the drafter's, variates for one token of each sequence
        n = rows * case["vocab"]
        both = 2 if case["drafts"] == "drawn" else 1
        return {"bytes": both * n * el + 4 * case["vocab"] * case["n_seq"] + 16 * rows, "flops": 4 * both * n}
    hd, hq, hkv = case["head_dim"], case["n_head"], case["n_head_kv"]
    if kind == "append":   # q, k, v in; q, k, v out
        return {"bytes": 2 * rows * (hq + 2 * hkv) * hd * el, "flops": 8 * rows * (hq + hkv) * hd}
    full = case["shared"] // case["page_size"] * case["page_size"]   # slots that lie in shared pages
    slots = case["groups"] * full + sum(a + r - full for a, r in pairs)
    seen = sum(r * a + (r * (r + 1) // 2 if case["tree"] == "chain" else tree_pairs(r)) for a, r in pairs)
    return {"bytes": 2 * slots * hkv * hd * el + 2 * rows * hq * hd * el + 4 * rows * hq, "flops": 4 * seen * hq * hd}


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
        return (idx - 1).to(torch.int32)
    u = torch.rand(len(idx), generator=g)
    return (u * idx).floor().to(torch.int32) - (idx == 0).to(torch.int32)


def exponential(g, *shape):
    return torch.empty(*shape, device=DEV).exponential_(generator=g)


def logits_of(g, rows, vocab):
    """Logits as models give them: most tokens far below a few likely ones."""
    x = torch.randn(rows, vocab, generator=g, device=DEV) * 1.5
    for _ in range(4):
        at = torch.randint(0, vocab, (rows, 1), generator=g, device=DEV)
        x.scatter_(1, at, 6 + 5 * torch.rand(rows, 1, generator=g, device=DEV))
    return x


def prepare(case, seed):
    kind, dt = case["kind"], TORCH[case["dtype"]]
    host = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dt)

    if kind == "sample":
        rows, vocab = case["rows"], case["vocab"]
        s["logits"] = logits_of(g, rows, vocab).to(dt)
        s["temperature"] = torch.rand(rows, generator=g, device=DEV) + 0.5
        s["noise"] = exponential(g, rows, vocab)
        s["tokens"] = torch.empty(rows, dtype=torch.int32, device=DEV)
        if own:
            s["cache"] = cache_of(dict(n_head=1, n_head_kv=1, head_dim=32, page_size=16, dtype="bf16"), 1, 1, 1)
        return s
    if kind == "norm":
        rows, hq, hkv, hd = case["rows"], case["n_head"], case["n_head_kv"], case["head_dim"]
        qkv = normal(rows, hq + 2 * hkv, hd)   # one row holds q, k and v, as the fused projection leaves them
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        s["q_norm"], s["k_norm"] = ((1 + 0.2 * torch.randn(hd, generator=g, device=DEV)).to(dt) for _ in range(2))
        s["pos"] = torch.randint(0, case["far"], (rows,), generator=g, device=DEV, dtype=torch.int32)
        s["q_out"], s["k_out"] = (torch.empty(rows, h, hd, dtype=dt, device=DEV) for h in (hq, hkv))
        if case["backward"]:
            s["dq_out"], s["dk_out"] = normal(rows, hq, hd), normal(rows, hkv, hd)
            s["dq_norm"], s["dk_norm"] = (torch.empty(hd, device=DEV) for _ in range(2))
        if own:
            s["cache"] = cache_of(case, 1, 1, 1)
        return s

    pairs = shapes(case)
    n = len(pairs)
    lens, counts = [a for a, _ in pairs], [r for _, r in pairs]
    rows, most = sum(counts), max(counts)
    s["counts"], s["lens"], s["most"] = counts, lens, most
    s["row_start"] = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).to(DEV)
    if kind != "append":
        parents = draw_trees(counts, case["tree"], host)
        s["parents"] = parents.to(DEV)

    if kind == "verify":
        vocab = case["vocab"]
        s["children"] = children_of(parents.tolist(), counts).to(DEV)
        target = logits_of(g, rows, vocab)
        s["temperature"] = (torch.rand(n, generator=g, device=DEV) * 0.5 + 0.7).repeat_interleave(
            torch.tensor(counts, device=DEV), output_size=rows)   # one of each sequence, for all of its rows
        # node t's token comes from row draft_row[t], that of its parent: what the drafter thought of the place
        base = s["row_start"][:-1].long().repeat_interleave(torch.tensor(counts, device=DEV), output_size=rows)
        s["draft_row"] = (s["parents"].clamp(min=0) + base).to(torch.int32)
        draft = target + 0.6 * torch.randn(rows, vocab, generator=g, device=DEV)
        s["target"] = target.to(dt)
        if case["drafts"] == "drawn":
            s["draft"] = draft.to(dt)
            tokens = torch.empty(rows, dtype=torch.int32, device=DEV)
            for a in range(0, rows, 64):   # (a block of rows at a time: the variates are as many as the logits)
                at = s["draft_row"][a:a + 64].long()
                p = (s["draft"][at].double() / s["temperature"][at, None]).softmax(-1)
                tokens[a:a + 64] = (p / exponential(g, len(at), vocab)).argmax(-1).to(torch.int32)
        else:
            s["draft"] = s["draft_row"] = None
            # the k-th child of a node is its k-th likeliest token
            rank = (s["children"] == torch.arange(max(counts), device=DEV)[:, None, None, None]).nonzero()
            nth = torch.zeros(rows, dtype=torch.int64, device=DEV)
            nth[s["row_start"][:-1].long()[rank[:, 1]] + rank[:, 0]] = rank[:, 3]
            best = draft.topk(min(vocab, s["children"].shape[2]), -1).indices
            tokens = best[s["parents"].clamp(min=0) + base, nth % best.shape[1]].to(torch.int32)
        s["tokens"] = tokens
        s["uniform"] = torch.rand(rows, generator=g, device=DEV)
        s["noise"] = exponential(g, n, vocab)
        s["path"] = torch.empty(n, case["rows_hi"], dtype=torch.int32, device=DEV)
        s["n_path"], s["id_last"] = (torch.empty(n, dtype=torch.int32, device=DEV) for _ in range(2))
        if own:
            s["cache"] = cache_of(dict(n_head=1, n_head_kv=1, head_dim=32, page_size=16, dtype="bf16"), n, 1, 1)
        return s

    ps, L, hq, hkv, hd = case["page_size"], case.get("n_layer", 1), case["n_head"], case["n_head_kv"], case["head_dim"]
    held = [-(-(a + c) // ps) for a, c in zip(lens, counts)]
    members = case.get("members", 1)
    common = case["shared"] // ps if kind == "prefix" else 0
    n_pages = sum(held) - (n - n // members) * common + 3
    ids = torch.randperm(n_pages, generator=host).to(torch.int32)
    table = torch.full((n, max(held) + 1), -1, dtype=torch.int32)
    seqs = torch.randperm(n, generator=host)   # the sequences of the call lie anywhere in the table
    refs = torch.zeros(n_pages, dtype=torch.int32)
    at, order = 0, seqs.tolist()
    for i, (q, h) in enumerate(zip(order, held)):
        first = i // members * members
        c = common if i != first else 0
        table[q, :c] = table[order[first], :c]
        table[q, c:h] = ids[at:at + h - c]
        at += h - c
        refs.index_add_(0, table[q, :h].long(), torch.ones(h, dtype=torch.int32))
    length = torch.zeros(n, dtype=torch.int32)
    length[seqs] = torch.tensor(lens, dtype=torch.int32)
    if own:
        s["cache"] = c = cache_of(case, n, max(held) + 1, n_pages)
        s["pages"], s["table"], s["length"], s["refs"] = c.pages, c.table, c.length, c.refs
    else:
        s["pages"] = torch.empty(n_pages, L, 2, hkv, ps, hd, dtype=dt, device=DEV)
        s["table"], s["length"], s["refs"] = (torch.empty_like(t, device=DEV) for t in (table, length, refs))
    s["pages"].normal_(generator=g)
    s["table"].copy_(table)
    s["length"].copy_(length)
    s["refs"].copy_(refs)
    s["seqs"] = seqs.to(torch.int32).to(DEV)
    s["host_seqs"] = order
    s["layer"] = L - 1
    if kind == "append":
        qkv = normal(rows, hq + 2 * hkv, hd)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_norm"], s["k_norm"] = ((1 + 0.2 * torch.randn(hd, generator=g, device=DEV)).to(dt) for _ in range(2))
        s["q_out"] = torch.empty(rows, hq, hd, dtype=dt, device=DEV)
        return s
    s["q"] = normal(rows, hq, hd)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(rows, hq, dtype=torch.float32, device=DEV)
    s["group_start"] = torch.arange(0, n + 1, members, dtype=torch.int32).to(DEV)
    s["mask"] = None
    if case["tree"] != "chain":
        s["mask"] = ancestor_words(parents.tolist(), counts, -(-case["rows_hi"] // 32)).to(DEV)
    if own:
        s["plan"] = torch.empty(n + case["groups"], dtype=torch.int32, device=DEV)
        s["work"] = torch.empty(s["cache"].prefix_workspace(rows), dtype=torch.uint8, device=DEV)
    return s


def children_of(parents, counts):
    """children[sequence][node][k]: the k-th child's node index, -1 behind the last."""
    lists, r0 = [], 0
    for c in counts:
        mine = [[] for _ in range(max(counts))]
        for i in range(1, c):
            mine[parents[r0 + i]].append(i)
        lists.append(mine)
        r0 += c
    k = max(1, max(len(x) for mine in lists for x in mine))
    return torch.tensor([[x + [-1] * (k - len(x)) for x in mine] for mine in lists])


def ancestor_words(parents, counts, words):
    """Every row's ancestors and itself as 32-bit words."""
    out, r0 = [], 0
    for c in counts:
        sets = []
        for i in range(c):
            p = parents[r0 + i]
            sets.append((sets[p] if p >= 0 else 0) | 1 << i)
        for m in sets:
            w = [(m >> 32 * k) & 0xffffffff for k in range(words)]
            out.append([x - (1 << 32) if x >= 1 << 31 else x for x in w])
        r0 += c
    return torch.tensor(out, dtype=torch.int32)


def cache_of(case, max_seq, max_pages, n_pages):
    from block_diffusion_drafter_fc_gb300.dflash import CacheConfig, PagedCache
    return PagedCache(CacheConfig(
        n_layer=case.get("n_layer", 1), n_head=case["n_head"], n_head_kv=case["n_head_kv"], head_dim=case["head_dim"],
        page_size=case["page_size"], n_pages=n_pages, max_seq=max_seq, max_pages=max_pages, dtype=case["dtype"],
        rope_layout=case.get("layout", "half"), rotary_dim=case.get("rotary_dim", case["head_dim"]),
        rope_theta=1e6, rope_scaling=case.get("scaling", "none"), rope_factor=case.get("factor", 1.0),
        rope_orig_positions=32768))


# --------------------------------------------------------------- plain forms

def angles(case, pos):
    """(cos, sin) of every row's pairs, from angles in 64 bits, magnitude factor included."""
    rd, f, theta, orig, m = case["rotary_dim"], case["factor"], 1e6, 32768, 1.0
    j = torch.arange(rd // 2, dtype=torch.float64, device=DEV)
    if case["scaling"] == "ntk":   # the base stretched so that the slowest pair is slowed by the factor
        theta = theta * f ** (rd / (rd - 2))
    inv = theta ** (-2 * j / rd)
    if case["scaling"] == "linear":
        inv = inv / f
    if case["scaling"] == "yarn":
        # pairs that turn more than 32 times over the original positions keep their angle, those that turn
        # less than once are slowed by the factor, a ramp between them
        at = [rd * math.log(orig / (t * 2 * math.pi)) / (2 * math.log(theta)) for t in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rd - 1)
        slow = ((j - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        inv, m = inv / f * slow + inv * (1 - slow), 0.1 * math.log(f) + 1.0
    t = pos.double()[:, None] * inv
    return (t.cos() * m).float()[:, None], (t.sin() * m).float()[:, None]


def turn(y, cos, sin, case):
    """Pairs (a, b) of y [T][heads][head_dim] at angle t -> (a cos t - b sin t, b cos t + a sin t)."""
    rd = case["rotary_dim"]
    if case["layout"] == "half":
        a, b = y[..., :rd // 2], y[..., rd // 2:rd]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., rd:]], -1)
    a, b = y[..., 0:rd:2], y[..., 1:rd:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), y[..., rd:]], -1)


def norm_rotate(x, w, cos, sin, case):
    y = x.float()
    y = y * (y.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return turn(y * w.float(), cos, sin, case).to(x.dtype)


def norm_rotate_grad(x, w, dy, cos, sin, case):
    """(dx, dw)"""
    y = x.float()
    r = (y.square().mean(-1, keepdim=True) + EPS).rsqrt()
    n = y * r
    back = turn(dy.float(), cos, -sin, case)
    dn = back * w.float()
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    return dx.to(x.dtype), (back * n).sum((0, 1), dtype=torch.float64).float()


def attend_prefix(s):
    case = s["case"]
    hq, hkv, hd, ps = case["n_head"], case["n_head_kv"], case["head_dim"], case["page_size"]
    out, lse, r0 = [], [], 0
    for i, (q, ln, c) in enumerate(zip(s["host_seqs"], s["lens"], s["counts"])):
        slots = ln + c
        held = s["table"][q, :-(-slots // ps)].long()
        kv = s["pages"][held, s["layer"]].transpose(0, 1).transpose(1, 2)   # [k, v][head][page][slot][dim]
        k, v = (kv[j].reshape(hkv, -1, hd)[:, :slots].float() for j in (0, 1))
        node = torch.arange(c, device=DEV) if s["mask"] is None else None
        if s["mask"] is None:
            sees = node[None, :] <= node[:, None]
        else:
            j = torch.arange(c, device=DEV)
            sees = (s["mask"][r0:r0 + c][:, j // 32] >> (j % 32) & 1).bool()
        qs = s["q"][r0:r0 + c].float().view(c, hkv, hq // hkv, hd).permute(1, 2, 0, 3).reshape(hkv, -1, hd)
        sc = (qs @ k.transpose(1, 2)).view(hkv, hq // hkv, c, slots) * hd ** -0.5
        sc[..., ln:] = sc[..., ln:].masked_fill(~sees, -math.inf)
        top = sc.amax(-1, keepdim=True)
        e = (sc - top).exp()
        total = e.sum(-1, keepdim=True)
        o = (e.view(hkv, -1, slots) @ v).view(hkv, hq // hkv, c, hd) / total
        out.append(o.permute(2, 0, 1, 3).reshape(c, hq, hd))
        lse.append((top + total.log())[..., 0].permute(2, 0, 1).reshape(c, hq))
        r0 += c
    return torch.cat(out).to(s["q"].dtype), torch.cat(lse)


def probabilities(logits, temperature):
    """In 64 bits: whether a token is accepted, or wins, is decided next to a border."""
    x = logits.double() / temperature.double()[:, None]
    e = (x - x.amax(-1, keepdim=True)).exp()
    return e / e.sum(-1, keepdim=True)


def verify(s):
    n, most_path = s["path"].shape
    vocab = s["case"]["vocab"]
    start, children = s["row_start"][:-1].long(), s["children"]
    every = torch.arange(n, device=DEV)
    cur = torch.zeros(n, dtype=torch.int64, device=DEV)
    alive = torch.ones(n, dtype=torch.bool, device=DEV)
    path = torch.full((n, most_path), -1, dtype=torch.int64, device=DEV)
    path[:, 0] = 0
    final = torch.zeros(n, vocab, dtype=torch.float64, device=DEV)
    for depth in range(1, most_path + 1):
        r = probabilities(s["target"][start + cur], s["temperature"][start + cur])
        nxt = torch.full_like(cur, -1)
        if depth < most_path:
            for k in range(children.shape[2]):
                c = children[every, cur, k]
                open_ = alive & (c >= 0) & (nxt < 0)
                row = start + c.clamp(min=0)
                x = s["tokens"][row].long()[:, None]
                if s["draft"] is None:
                    q = torch.zeros_like(r).scatter_(1, x, 1.0)
                else:
                    at = s["draft_row"][row].long()
                    q = probabilities(s["draft"][at], s["temperature"][at])
                good = s["uniform"][row].double() * q.gather(1, x)[:, 0] < r.gather(1, x)[:, 0]
                nxt = torch.where(open_ & good, c, nxt)
                rest = (r - q).clamp(min=0)
                r = torch.where((open_ & ~good)[:, None], rest / rest.sum(-1, keepdim=True), r)
        ends = alive & (nxt < 0)
        final = torch.where(ends[:, None], r, final)
        alive = alive & (nxt >= 0)
        cur = torch.where(alive, nxt, cur)
        if depth < most_path:
            path[:, depth] = nxt.where(alive, -1)
    token = (final / s["noise"]).argmax(-1)
    return {"path": path.to(torch.int32), "n_path": (path >= 0).sum(1).to(torch.int32), "id_last": token.to(torch.int32)}


def row_sequence(row_start, rows):
    return torch.searchsorted(row_start, torch.arange(rows, device=DEV, dtype=torch.int32), right=True) - 1


def run(s):
    case, kind = s["case"], s["case"]["kind"]
    c = s.get("cache")
    if kind == "sample":
        if own:
            c.dflash_sample(s["logits"], s["noise"], s["tokens"], temperature=s["temperature"])
            return s["tokens"]
        p = probabilities(s["logits"], s["temperature"])
        return (p / s["noise"]).argmax(-1).to(torch.int32)

    if kind == "verify":
        if own:
            c.dflash_tree_verify(s["row_start"], s["parents"], s["tokens"], s["target"], s["uniform"], s["noise"], s["path"],
                                 s["n_path"], s["id_last"], draft=s["draft"], draft_row=s["draft_row"],
                                 temperature=s["temperature"],
                                 draft_temperature=None if s["draft"] is None else s["temperature"])
            return {k: s[k] for k in ("path", "n_path", "id_last")}
        return verify(s)

    if kind == "norm":
        if case["backward"]:
            if own:
                c.dflash_norm_rope_grad(s["pos"], q=s["q"], q_norm=s["q_norm"], dq_out=s["dq_out"], dq=s["q_out"],
                                        dq_norm=s["dq_norm"], k=s["k"], k_norm=s["k_norm"], dk_out=s["dk_out"], dk=s["k_out"],
                                        dk_norm=s["dk_norm"], eps=EPS)
                return s["q_out"], s["dq_norm"], s["k_out"], s["dk_norm"]
            cos, sin = angles(case, s["pos"])
            return (*norm_rotate_grad(s["q"], s["q_norm"], s["dq_out"], cos, sin, case),
                    *norm_rotate_grad(s["k"], s["k_norm"], s["dk_out"], cos, sin, case))
        if own:
            c.dflash_norm_rope(s["pos"], q=s["q"], q_norm=s["q_norm"], q_out=s["q_out"], k=s["k"], k_norm=s["k_norm"],
                               k_out=s["k_out"], eps=EPS)
            return s["q_out"], s["k_out"]
        cos, sin = angles(case, s["pos"])
        return norm_rotate(s["q"], s["q_norm"], cos, sin, case), norm_rotate(s["k"], s["k_norm"], cos, sin, case)

    if kind == "append":
        if own:
            c.dflash_norm_append(s["layer"], s["row_start"], s["k"], s["v"], s["k_norm"], q=s["q"], q_out=s["q_out"],
                                 q_norm=s["q_norm"], eps=EPS, seqs=s["seqs"])
            return s["q_out"], s["pages"]
        rows, ps = s["k"].shape[0], case["page_size"]
        of = row_sequence(s["row_start"], rows).long()
        q = s["seqs"].long()[of]
        slot = s["length"][q].long() + torch.arange(rows, device=DEV) - s["row_start"][of]
        page, at = s["table"][q, slot // ps].long(), slot % ps
        cos, sin = angles(case, slot)
        s["pages"][page, s["layer"], 0, :, at] = norm_rotate(s["k"], s["k_norm"], cos, sin, case)
        s["pages"][page, s["layer"], 1, :, at] = s["v"]
        return norm_rotate(s["q"], s["q_norm"], cos, sin, case), s["pages"]

    if own:
        c.dflash_prefix_plan(s["group_start"], s["plan"], seqs=s["seqs"])
        c.dflash_prefix_attend(s["layer"], s["row_start"], s["most"], s["q"], s["out"], s["group_start"], s["plan"], s["work"],
                               mask=s["mask"], lse=s["lse"], seqs=s["seqs"])
        return s["out"], s["lse"]
    return attend_prefix(s)


# ---------------------------------------------------------------- definition

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    kind = case["kind"]

    def spin(y, pos, backward=False):
        """Rotation by complex numbers: a + ib times m e^(it), in 64 bits."""
        rd, base, freq = case["rotary_dim"], 1e6, []
        if case["scaling"] == "ntk":
            base *= case["factor"] ** (rd / (rd - 2.0))
        lo = max(math.floor(rd * math.log(32768 / (64 * math.pi)) / (2 * math.log(base))), 0)
        hi = min(math.ceil(rd * math.log(32768 / (2 * math.pi)) / (2 * math.log(base))), rd - 1)
        for j in range(rd // 2):
            f = base ** (-2.0 * j / rd)
            if case["scaling"] == "linear":
                f /= case["factor"]
            if case["scaling"] == "yarn":
                w = min(max((j - lo) / max(hi - lo, 0.001), 0.0), 1.0)
                f = w * f / case["factor"] + (1 - w) * f
            freq.append(f)
        m = 0.1 * math.log(case["factor"]) + 1 if case["scaling"] == "yarn" else 1.0
        t = pos.double()[:, None, None] * torch.tensor(freq, dtype=torch.float64, device=DEV)
        z = torch.polar(torch.full_like(t, m), -t if backward else t)
        y = y.clone()
        a, b = (slice(0, rd // 2), slice(rd // 2, rd)) if case["layout"] == "half" else (slice(0, rd, 2), slice(1, rd, 2))
        w = torch.complex(y[..., a], y[..., b]) * z
        y[..., a], y[..., b] = w.real, w.imag
        return y

    def size(x):
        return torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)

    if kind == "norm":
        got = []
        for x, w, dy in ((s["q"], s["q_norm"], s.get("dq_out")), (s["k"], s["k_norm"], s.get("dk_out"))):
            x, w = x.double(), w.double()
            if not case["backward"]:
                got.append(spin(x / size(x) * w, s["pos"]))
                continue
            # y = w x / |x|_rms before the turn, so dx = (g w - x (x . g w) / (head_dim |x|^2)) / |x|
            back, z = spin(dy.double(), s["pos"], True), size(x)
            gw = back * w
            got.append((gw - x * (x * gw).sum(-1, keepdim=True) / (x.shape[-1] * z * z)) / z)
            got.append((back * x / z).sum(0).sum(0))
        return tuple(got)
    if kind == "append":
        pages, ps = s["pages"].double(), case["page_size"]
        q_out = torch.empty(s["q_out"].shape, dtype=torch.float64, device=DEV)
        r0 = 0
        for q, ln, c in zip(s["host_seqs"], s["lens"], s["counts"]):
            pos = torch.arange(ln, ln + c, device=DEV)
            x, k, v = s["q"][r0:r0 + c].double(), s["k"][r0:r0 + c].double(), s["v"][r0:r0 + c].double()
            q_out[r0:r0 + c] = spin(x / size(x) * s["q_norm"].double(), pos)
            k = spin(k / size(k) * s["k_norm"].double(), pos)
            for p in range(ln // ps, (ln + c - 1) // ps + 1):
                a, b = max(ln, p * ps), min(ln + c, (p + 1) * ps)
                to = pages[int(s["table"][q, p]), s["layer"]]
                to[0][:, a - p * ps:b - p * ps] = k[a - ln:b - ln].transpose(0, 1)
                to[1][:, a - p * ps:b - p * ps] = v[a - ln:b - ln].transpose(0, 1)
            r0 += c
        return q_out, pages
    if kind == "prefix":
        hq, hkv, hd, ps = case["n_head"], case["n_head_kv"], case["head_dim"], case["page_size"]
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.empty(s["lse"].shape, dtype=torch.float64, device=DEV)
        parents, r0 = s["parents"].tolist(), 0
        for q, ln, c in zip(s["host_seqs"], s["lens"], s["counts"]):
            tree = torch.zeros(c, c, dtype=torch.bool)
            for i in range(c):
                if parents[r0 + i] >= 0:
                    tree[i] = tree[parents[r0 + i]]
                tree[i, i] = True
            hidden = torch.cat([torch.zeros(c, ln, dtype=torch.bool), ~tree], 1).to(DEV)
            held = s["table"][q, :-(-(ln + c) // ps)].long()
            for h in range(hkv):
                kv = s["pages"][held, s["layer"], :, h].double()
                k, v = (kv[:, i].reshape(-1, hd)[:ln + c] for i in (0, 1))
                for x in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                    sc = (s["q"][r0:r0 + c, x].double() @ k.T / math.sqrt(hd)).masked_fill(hidden, -math.inf)
                    out[r0:r0 + c, x] = sc.softmax(-1) @ v
                    lse[r0:r0 + c, x] = sc.logsumexp(-1)
            r0 += c
        return out, lse
    if kind == "sample":
        x = s["logits"].double() / s["temperature"].double()[:, None]
        return torch.argmax(x - s["noise"].double().log(), -1).to(torch.int32)

    # verify: one sequence, one child at a time
    n, most_path = s["path"].shape
    path = torch.full((n, most_path), -1, dtype=torch.int32)
    n_path, id_last = (torch.zeros(n, dtype=torch.int32) for _ in range(2))
    parents, tokens, uniform, r0 = s["parents"].tolist(), s["tokens"].tolist(), s["uniform"].tolist(), 0
    for i, c in enumerate(s["counts"]):
        at = [0]
        while True:
            p = (s["target"][r0 + at[-1]].double() / s["temperature"][r0 + at[-1]].double()).softmax(0)
            found = None
            for node in range(at[-1] + 1, c if len(at) < most_path else 0):
                if parents[r0 + node] != at[-1]:
                    continue
                x = tokens[r0 + node]
                q = torch.zeros_like(p)
                if s["draft"] is None:
                    q[x] = 1.0
                else:
                    row = int(s["draft_row"][r0 + node])
                    q = (s["draft"][row].double() / s["temperature"][row].double()).softmax(0)
                if uniform[r0 + node] * float(q[x]) < float(p[x]):
                    found = node
                    break
                p = torch.relu(p - q)
                p = p / p.sum()
            if found is None:
                break
            at.append(found)
        path[i, :len(at)] = torch.tensor(at, dtype=torch.int32)
        n_path[i], id_last[i] = len(at), int(torch.argmax(p / s["noise"][i].double()))
        r0 += c
    return {"path": path.to(DEV), "n_path": n_path.to(DEV), "id_last": id_last.to(DEV)}
