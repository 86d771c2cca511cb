"""What is measured of the draft-tree operators and of what stands before and behind them: cases, plain forms, exact values.

A decoder that drafts several continuations of its sequences at once and lets the layer judge them in one pass does:

  norm     queries and keys of new tokens are normalised per head and rotated to their positions, in one pass; a
           model that is trained with such heads also needs the gradient of that (norm_grad);
  tree     every drafted token attends to its sequence's cached tokens (all, or the pools selected for it) and to its
           own ancestors in the tree of drafts;
  commit   the accepted path of each tree enters the paged cache;
  branch   sequences are forked (beams, several samples of one prompt): the branches share the trunk's full pages and
           get pages of their own to write to, and the branches of the step before give theirs back;
  compact  the used pages move to the front of the cache, so that the rest can be given up.

Definitions:

  norm     y = x * (mean(x^2) + eps)^(-1/2) * weight over each head's d channels; then the pair (x, y) of channels
           (i, i + rot/2), or (2i, 2i + 1) when interleaved, becomes (x cos a - y sin a, x sin a + y cos a) with
           a = position * freq[i].  norm_grad: the gradients of x and of the weights (summed over tokens and heads).
  tree     o[t, h] = softmax_j(scale q[t, h] . k[j]) v[j], lse[t, h] = log sum_j exp(scale q[t, h] . k[j]) over the
           keys j of node t: the cached tokens of its row (or those of the pools idx[t] and of the row's last,
           incomplete pool), its ancestors (parents[t] and so on, numbers within the row; -1: the cached end) and itself.
  commit   the d nodes from the root to node accepted[b] become tokens lens[b] .. lens[b] + d - 1 of row b: k and v in
           their pages, the keys of pools that they complete, the indexer keys of the row's last, incomplete pool
           (ktail); lens_out[b] = lens[b] + d.  accepted[b] = -1: none.
  branch   refs[page] counts the block-table entries that name a page.  Release: the old branches' entries give their
           count back.  Fork: branch i has parents[i]'s length and pages.  Reserve (room for `grow` tokens): the
           branch's last page, where it is not full and has other holders, is copied to a free one, and columns up to
           the new length get free pages: requests in order of (row, column) take the free pages in ascending order.
  compact  with U pages in use, the used pages numbered U and higher go, in order, to the free ones below U.

Layer shapes (heads, widths, k, dtypes) are those of the repository's workloads; row counts, lengths, tree and page
sizes are generic.
"""
import math
import random

import torch

own = False

BF16, FP32 = "bf16", "fp32"
EPS = 1e-6


def _case(op, name=None, **kw):
    c = {"op": op, "dtype": BF16, "batch": 1, "tokens": 4096, "ragged": False, "Hq": 16, "d": 128, "di": 64, "page": 64}
    c.update({"norm": {"rot": 128, "interleaved": False, "packed": False},
              "norm_grad": {"rot": 128, "interleaved": False, "packed": False},
              "tree": {"nodes": 16, "k": 0, "chain": False},
              "commit": {"nodes": 16, "chain": False},
              "branch": {"fan": 4, "grow": 8},
              "compact": {"fill": 0.6}}[op])
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # the drafted tokens of a serving batch: latency counts
        _case("norm", "norm_step_300", tokens=300, rot=64, packed=True),
        # a 128k training sequence, q and k slices of one projection's output
        _case("norm", "norm_train_128k", tokens=131072, packed=True),
        # its gradient, from the layer's fp32 dQ and dK
        _case("norm_grad", "norm_grad_128k", tokens=131072, packed=True),
        # the fp32 layer, a short odd sequence
        _case("norm_grad", "norm_grad_fp32_4093", dtype=FP32, tokens=4093, Hq=8, d=64, rot=16, interleaved=True),
        # one user, long context, a tree of 16 drafts
        _case("tree", "tree_b1_128k", tokens=131069),
        # a serving batch of the 32-head layer, trees of up to 61 drafts, contexts of all lengths
        _case("tree", "tree_b24_ragged_h32", batch=24, tokens=16381, ragged=True, Hq=32, nodes=61, page=128),
        # a serving batch of the sparse layer: 512 selected pools for each draft
        _case("tree", "tree_sel_b16_32k", batch=16, tokens=32767, ragged=True, nodes=24, k=512),
        # the fp32 layer, chains of drafts behind short contexts
        _case("tree", "tree_fp32_b5", dtype=FP32, batch=5, tokens=4094, ragged=True, Hq=8, d=64, nodes=7, chain=True, page=16),
        # the accepted drafts of a serving batch: latency counts
        _case("commit", "commit_b48", batch=48, tokens=30001, ragged=True),
        # many rows that accept parts of long chains
        _case("commit", "commit_b512_chains", batch=512, tokens=4094, ragged=True, nodes=128, chain=True, page=16),
        # four continuations of each of 64 sequences
        _case("branch", "branch_b64x4", batch=64, tokens=16381, ragged=True, page=128),
        # a cache of 1M tokens, 60% of its pages in use
        _case("compact", "compact_1m", batch=40, tokens=16384, ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "tree", "tree", "tree", "commit", "branch", "compact"])
    dtype = rng.choice([BF16, BF16, FP32])
    wide = 1 if dtype == BF16 else 2   # an fp32 case moves twice the bytes
    c = {"dtype": dtype, "d": rng.choice([64, 128]), "di": rng.choice([64, 128]), "page": rng.choice([4, 16, 20, 64, 64, 100, 128]),
         "Hq": rng.choice([16, 32, rng.randint(1, 32)]), "ragged": rng.random() < 0.7}
    if op in ("norm", "norm_grad"):
        c["rot"] = rng.choice([0, 16, 64, c["d"]])
        c["interleaved"] = rng.random() < 0.5
        c["packed"] = rng.random() < 0.5
        c["tokens"] = _log(rng, 1, 131072 * 16 // max(16, c["Hq"]) // wide)
    elif op == "tree":
        c["batch"], c["nodes"], c["chain"] = _log(rng, 1, 64), _log(rng, 1, 128), rng.random() < 0.3
        c["k"] = rng.choice([0, 0, 64, 512, rng.randint(1, 1024)])
        if dtype == FP32 or c["k"]:   # a drafted token is a row of its own there
            c["nodes"] = min(c["nodes"], max(1, 512 // c["batch"]))
        c["tokens"] = _log(rng, 1, 500000 // c["batch"])
        while _cost(_case(op, **c)) > 1:
            c["tokens"] = c["tokens"] * 2 // 3
    elif op == "commit":
        c["batch"], c["nodes"], c["chain"] = _log(rng, 1, 512), _log(rng, 1, 128), rng.random() < 0.3
        c["tokens"] = _log(rng, 1, 2000000 // c["batch"] // wide)
    elif op == "branch":
        c["batch"], c["fan"], c["grow"] = _log(rng, 1, 64), rng.randint(1, 8), _log(rng, 1, 128)
        c["tokens"] = _log(rng, 1, 1000000 // c["batch"] // wide)
    else:
        c["batch"], c["fill"] = _log(rng, 1, 64), rng.choice([0.2, 0.6, 0.9, 0.99])
        c["tokens"] = _log(rng, 1, 600000 // c["batch"] // wide)
    return _case(op, **c)


def _cost(c):
    """A tree's cost as a share of the largest listed one's."""
    w = work(c)
    return max(w["flops"] / 2.5e11 * (1 if c["dtype"] == BF16 and not c["k"] else 16), w["bytes"] / 1.5e9)


def _spread(n, most, ragged, idle):
    """n numbers up to `most`, the first the largest; one of 8 and more is 0 where `idle`."""
    if not ragged:
        return [most] * n
    x = [most if b == 0 else 1 + (b * 2654435761 % 2**32) * most // 2**32 for b in range(n)]
    if idle and n >= 8:
        x[n // 2] = 0
    return x


def _lens(c):
    """Cached tokens of every row; row 0 is the longest."""
    return _spread(c["batch"], c["tokens"], c["ragged"], True)


def _nodes(c):
    """Drafted tokens of every row; of 8 rows and more the last has none."""
    n = _spread(c["batch"], c["nodes"], c["ragged"], False)
    if c["ragged"] and c["batch"] >= 8:
        n[-1] = 0
    return n


def _elem(c):
    return 2 if c["dtype"] == BF16 else 4


def _page_bytes(c, tokens, tail=True):
    return (2 * tokens * c["d"] + tokens // 4 * c["di"] + (3 * c["di"] if tail else 0)) * _elem(c)


def work(c):
    e, d, di, Hq, op = _elem(c), c["d"], c["di"], c["Hq"], c["op"]
    if op == "norm":
        n = c["tokens"] * (Hq + 1)
        return {"bytes": 2 * n * d * e + 8 * d, "flops": n * (4 * d + 3 * c["rot"])}
    if op == "norm_grad":
        n = c["tokens"] * (Hq + 1)
        return {"bytes": n * d * (e + 8) + 16 * d, "flops": n * (9 * d + 3 * c["rot"])}
    if op == "compact":
        used, moved = _compact_counts(c)
        return {"bytes": 2 * moved * _page_bytes(c, c["page"]) + 8 * used, "flops": 0}
    lens = _lens(c)
    if op == "branch":
        # a branch copies the tokens of its row's last page, where that is not full
        part = [x % c["page"] for x in lens]
        tables = 4 * sum(-(-x // c["page"]) for x in lens)
        return {"bytes": c["fan"] * (sum(2 * _page_bytes(c, x) for x in part if x) + 2 * tables), "flops": 0}
    nodes = _nodes(c)
    deep = [sum(_depths(c)[b]) for b in range(c["batch"])]
    if op == "commit":
        t = sum(_depths(c)[b][_last(c, b)] if _last(c, b) >= 0 else 0 for b in range(c["batch"]))
        return {"bytes": t * (4 * d + 2 * di) * e, "flops": t * di}
    t = sum(nodes)
    if c["k"]:
        keys = sum(n * (4 * min(c["k"], x // 4) + x % 4) for x, n in zip(lens, nodes))
        read = keys
    else:
        keys = sum(n * x for x, n in zip(lens, nodes))
        read = sum(x for x, n in zip(lens, nodes) if n)
    by = 2 * (read + t) * d * e + t * Hq * (2 * d * e + 4) + 4 * c["k"] * t
    return {"bytes": by, "flops": 4 * Hq * d * (keys + sum(deep))}


# ------------------------------------------------------------------------------------------------- inputs


def _parents(c):
    """parents[b][i]: the node before node i of row b, -1 for the cached end.  The trees' shapes go with the case."""
    out = []
    for b, n in enumerate(_nodes(c)):
        r = random.Random(1000 * b + n)
        out.append([i - 1 if c["chain"] else r.randint(max(-1, i - 9), i - 1) for i in range(n)])
    return out


def _depths(c):
    """Nodes from the root to each node, itself included."""
    out = []
    for row in _parents(c):
        deep = []
        for p in row:
            deep.append(1 if p < 0 else deep[p] + 1)
        out.append(deep)
    return out


def _last(c, b):
    """The accepted node of row b: one far down the tree, for every seventh row none."""
    n = _nodes(c)[b]
    return -1 if n == 0 or b % 7 == 3 else n - 1 - b % min(n, 5)


def _compact_counts(c):
    """(pages in use, pages that move): every row's pages are dealt over a cache of which they are a share `fill`."""
    used = sum(-(-x // c["page"]) for x in _lens(c))
    where = _dealt(used, max(used, int(used / c["fill"])))
    return used, sum(p >= used for p in where)


def _dealt(used, pages):
    return random.Random(used).sample(range(pages), used)


def prepare(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = torch.bfloat16 if c["dtype"] == BF16 else torch.float32
    op, B, d, di, Hq, page = c["op"], c["batch"], c["d"], c["di"], c["Hq"], c["page"]

    def randn(*shape, dtype=dt):
        return torch.empty(shape, dtype=dtype, device=dev).normal_(generator=g)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    s = {"case": c, "scale": d ** -0.5}
    if op in ("norm", "norm_grad"):
        T = c["tokens"]
        if c["packed"]:   # the projection's output: q heads, the k head, the v head of a token behind each other
            x = randn(T, Hq + 2, d)
            s["q"], s["k"] = x[:, :Hq], x[:, Hq]
        else:
            s["q"], s["k"] = randn(T, Hq, d), randn(T, d)
        s["q_weight"], s["k_weight"] = (1 + 0.2 * randn(d, dtype=torch.float32) for _ in range(2))
        s["freq"] = s["positions"] = None
        if c["rot"]:
            s["freq"] = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
            if op == "norm" and T < 4096:   # drafted tokens: anywhere in long contexts
                s["positions"] = torch.randint(0, 1 << 20, (T,), generator=g, device=dev, dtype=torch.int32)
        if op == "norm":
            s["q_out"], s["k_out"] = torch.zeros(T, Hq, d, dtype=dt, device=dev), torch.zeros(T, d, dtype=dt, device=dev)
        else:
            s["dq_out"], s["dk_out"] = randn(T, Hq, d, dtype=torch.float32), randn(T, d, dtype=torch.float32)
            s["dq"], s["dk"] = torch.zeros_like(s["dq_out"]), torch.zeros_like(s["dk_out"])
            s["dq_weight"], s["dk_weight"] = (torch.zeros(d, device=dev) for _ in range(2))
        if own:
            import long_context_sparse_dsa_gb300 as dsa
            s["dims"] = dsa.make_dims(max(4, (T + 3) // 4 * 4), Hq, d, 8, di, 512, dtype=c["dtype"])
            s["rotation"] = dsa.make_rotation(s["freq"], interleaved=c["interleaved"]) if c["rot"] else None
            if op == "norm_grad":
                s["ws"] = torch.empty(dsa.qk_norm_bwd_workspace_bytes(s["dims"], T), dtype=torch.uint8, device=dev)
        return s

    lens = _lens(c)
    room = c["nodes"] if op == "commit" else c["grow"] if op == "branch" else 0
    cap = max(4, (max(lens) + room + 3) // 4 * 4)
    cols = -(-cap // page)
    hold = [-(-(x + (room if op == "commit" else 0)) // page) for x in lens]
    used = sum(hold)
    if op == "compact":
        pages = max(used, int(used / c["fill"]))
        order = torch.tensor(_dealt(used, pages), device=dev)
        order = order[torch.randperm(used, generator=g, device=dev)]
    else:
        # branches: up to one page for the copy and one for every page that they grow by
        pages = used + 1 + (B * c["fan"] * (2 + -(-room // page)) if op == "branch" else 0)
        order = torch.randperm(pages, generator=g, device=dev)[:used]
    table = torch.full((B, cols), -1, dtype=torch.int32, device=dev)
    table[torch.arange(cols, device=dev)[None, :] < torch.tensor(hold, device=dev)[:, None]] = order.to(torch.int32)
    s.update(lens=i32(lens), table=table, k=randn(pages, page, d), v=randn(pages, page, d),
             refs=torch.zeros(pages, dtype=torch.int32, device=dev))
    s["refs"][order] = 1
    if op != "tree":
        s["kpool"] = torch.randint(-12, 13, (pages, page // 4, di), generator=g, device=dev).to(dt)
        s["ktail"] = torch.randint(-3, 4, (pages, 3, di), generator=g, device=dev).to(dt)
    if op in ("tree", "commit"):
        nodes = _nodes(c)
        T = sum(nodes)
        s["offsets"] = i32([sum(nodes[:b]) for b in range(B + 1)])
        s["parents"] = i32([p for row in _parents(c) for p in row])
        s["new_k"], s["new_v"] = randn(T, d), randn(T, d)
    if op == "tree":
        s["q"] = randn(T, Hq, d)
        s["idx"] = None
        if c["k"]:
            # min(k, lens // 4) distinct pools for each node, ascending, then -1
            P, k = cap // 4, c["k"]
            elig = torch.tensor([x // 4 for x, n in zip(lens, nodes) for _ in range(n)], device=dev)[:, None]
            r = torch.rand(T, P, generator=g, device=dev)
            r[torch.arange(P, device=dev)[None, :] >= elig] = 2.0
            n = min(k, P)
            pick = r.topk(n, dim=1, largest=False).indices
            pick[torch.arange(n, device=dev)[None, :] >= elig] = P
            pick = pick.sort(dim=1).values
            pick[pick == P] = -1
            s["idx"] = torch.full((T, k), -1, dtype=torch.int32, device=dev)
            s["idx"][:, :n] = pick.to(torch.int32)
        s["o"], s["lse"] = torch.zeros(T, Hq, d, dtype=dt, device=dev), torch.zeros(T, Hq, device=dev)
    elif op == "commit":
        s["new_kidx"] = torch.randint(-3, 4, (T, di), generator=g, device=dev).to(dt)
        s["accepted"] = i32([_last(c, b) for b in range(B)])
        s["lens_out"] = torch.zeros(B, dtype=torch.int32, device=dev)
    elif op == "branch":
        n = B * c["fan"]
        s["from"] = torch.randint(0, B, (n,), generator=g, device=dev, dtype=torch.int32).sort().values
        s["b_table"] = torch.full((n, cols), -1, dtype=torch.int32, device=dev)   # no branches yet
        s["b_lens"], s["b_grown"] = (torch.zeros(n, dtype=torch.int32, device=dev) for _ in range(2))
        s["missing"] = torch.zeros(1, dtype=torch.int32, device=dev)
    elif op == "compact":
        s["table0"], s["refs0"] = table.clone(), s["refs"].clone()
        s["remap"] = torch.zeros(pages, dtype=torch.int32, device=dev)
        s["used"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if own:
        # the handle and the workspaces that a decoder keeps for its lifetime
        import long_context_sparse_dsa_gb300 as dsa
        dims = s["dims"] = dsa.make_dims(cap, Hq, d, 8, di, c.get("k") or 512, dtype=c["dtype"])
        s["cache"] = dsa.PagedCache(k=s["k"], v=s["v"], kpool=s.get("kpool"), ktail=s.get("ktail"))
        if op == "tree":
            s["ws"] = torch.empty(dsa.tree_workspace_bytes(dims, B, T), dtype=torch.uint8, device=dev)
        elif op in ("branch", "compact"):
            rows = s["b_lens"].numel() if op == "branch" else B
            s["ws"] = torch.empty(dsa.page_workspace_bytes(dims, s["cache"], rows), dtype=torch.uint8, device=dev)
    return s


def run(s):
    op, c = s["case"]["op"], s["case"]
    if own:
        import long_context_sparse_dsa_gb300 as dsa
        if op == "norm":
            dsa.qk_norm_rotate(s["dims"], s["q"], s["k"], s["q_out"], s["k_out"], EPS, q_weight=s["q_weight"],
                               k_weight=s["k_weight"], rotation=s["rotation"], positions=s["positions"])
        elif op == "norm_grad":
            dsa.qk_norm_rotate_bwd(s["dims"], s["q"], s["k"], s["dq_out"], s["dk_out"], s["dq"], s["dk"], EPS, s["ws"],
                                   q_weight=s["q_weight"], k_weight=s["k_weight"], dq_weight=s["dq_weight"],
                                   dk_weight=s["dk_weight"], rotation=s["rotation"], positions=s["positions"])
        elif op == "tree":
            dsa.decode_tree_attn(s["dims"], s["cache"], s["lens"], s["table"], s["offsets"],
                                 None if c["chain"] else s["parents"], s["q"], s["new_k"], s["new_v"], s["o"], s["lse"],
                                 s["ws"], idx=s["idx"])
        elif op == "commit":
            dsa.cache_commit(s["dims"], s["cache"], s["lens"], s["table"], s["offsets"], None if c["chain"] else s["parents"],
                             s["accepted"], s["new_k"], s["new_v"], s["new_kidx"], s["lens_out"])
        elif op == "branch":
            dsa.cache_release(s["dims"], s["cache"], s["refs"], s["b_grown"], s["b_table"])
            dsa.cache_fork(s["dims"], s["cache"], s["refs"], s["lens"], s["table"], s["from"], s["b_lens"], s["b_table"])
            torch.add(s["b_lens"], c["grow"], out=s["b_grown"])
            dsa.cache_reserve(s["dims"], s["cache"], s["refs"], s["b_lens"], s["b_grown"], s["b_table"], s["missing"], s["ws"])
        else:
            s["table"].copy_(s["table0"])   # the rows where they were, so that a pass has something to move
            s["refs"].copy_(s["refs0"])
            dsa.cache_compact(s["dims"], s["cache"], s["refs"], s["lens"], s["table"], s["remap"], s["used"], s["ws"])
        return _outputs(s)
    return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "tree": _plain_tree, "commit": _plain_commit,
            "branch": _plain_branch, "compact": _plain_compact}[op](s)


def _outputs(s):
    cache = ("k", "v", "kpool", "ktail")
    names = {"norm": ("q_out", "k_out"), "norm_grad": ("dq", "dk", "dq_weight", "dk_weight"), "tree": ("o", "lse"),
             "commit": cache + ("lens_out",), "branch": cache + ("refs", "b_table", "b_lens", "missing"),
             "compact": cache + ("refs", "table", "remap", "used")}[s["case"]["op"]]
    return {n: s[n] for n in names}


# ------------------------------------------------------------------------------------------------- plain forms


def _turn(s, T, dev):
    """cos and sin [T, 1, rot/2] of the angles, in 64 bits, as 32."""
    p = s["positions"] if s["positions"] is not None else torch.arange(T, device=dev)
    a = p.double()[:, None] * s["freq"]
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _rotated(y, cos, sin, interleaved):
    """y [T, H, d] fp32"""
    n = 2 * cos.shape[-1]
    a, b = (y[..., 0:n:2], y[..., 1:n:2]) if interleaved else (y[..., :n // 2], y[..., n // 2:n])
    a, b = a * cos - b * sin, a * sin + b * cos
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, y[..., n:]], -1)


def _plain_norm(s):
    c = s["case"]

    def one(x, weight):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
        return _rotated(y, *turn, c["interleaved"]) if c["rot"] else y

    turn = _turn(s, c["tokens"], s["q"].device) if c["rot"] else None
    q, k = one(s["q"], s["q_weight"]), one(s["k"][:, None], s["k_weight"])[:, 0]
    return {"q_out": q.to(s["q"].dtype), "k_out": k.to(s["k"].dtype)}


def _plain_norm_grad(s):
    c = s["case"]

    def one(x, weight, dy):
        x = x.float()
        g = _rotated(dy, turn[0], -turn[1], c["interleaved"]) if c["rot"] else dy   # turned back
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        xn = x * r
        dw = (g * xn).sum((0, 1), dtype=torch.float64).float()
        g = g * weight
        return r * (g - xn * (g * xn).mean(-1, keepdim=True)), dw

    turn = _turn(s, c["tokens"], s["q"].device) if c["rot"] else None
    dq, dqw = one(s["q"], s["q_weight"], s["dq_out"])
    dk, dkw = one(s["k"][:, None], s["k_weight"], s["dk_out"][:, None])
    return {"dq": dq, "dk": dk[:, 0], "dq_weight": dqw, "dk_weight": dkw}


def _tree_of(s):
    """Of the nodes, in one list: their row, their number in it, and their ancestors, themselves included, [T, N]."""
    c, off = s["case"], s["offsets"].long()
    dev, B, N, T = off.device, c["batch"], c["nodes"], s["parents"].numel()
    row = torch.repeat_interleave(torch.arange(B, device=dev), off.diff(), output_size=T)
    num = torch.arange(T, device=dev) - off[row]
    up = torch.zeros(B, N, N + 1, device=dev)
    up[row, num, s["parents"].long()] = 1.0           # -1: the last column, which is dropped
    up = up[:, :, :N] + torch.eye(N, device=dev)
    for _ in range(7):                                # up to 128 generations
        up = ((up @ up) > 0).float()
    return row, num, up[row, num] > 0


def _softmax(score, v):
    """score [.., h, j] with -inf where nothing is seen, v [.., j, d] -> o [.., h, d], lse [.., h]"""
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1)
    o = p @ v / torch.where(total == 0, 1.0, total)[..., None]
    return o, torch.where(total == 0, -math.inf, top[..., 0] + total.log())


def _plain_tree(s):
    c, table, lens = s["case"], s["table"].long(), s["lens"].long()
    page, dev, N, B, Hq, d = c["page"], lens.device, c["nodes"], c["batch"], c["Hq"], c["d"]
    row, num, mine = _tree_of(s)
    drafts = torch.zeros(2, B, N, d, device=dev)
    drafts[0, row, num], drafts[1, row, num] = s["new_k"].float(), s["new_v"].float()
    if s["idx"] is None:
        # by rows: all nodes and heads of a row against its tokens and its drafts
        tok = torch.arange(int(c["tokens"]), device=dev)
        where = table.gather(1, (tok // page).expand(B, -1)).clamp(min=0)
        seen = tok < lens[:, None]
        k, v = (torch.cat([s[x][where, tok % page].float().masked_fill(~seen[..., None], 0.0), y], 1)
                for x, y in (("k", drafts[0]), ("v", drafts[1])))
        q = torch.zeros(B, N, Hq, d, device=dev)
        q[row, num] = s["q"].float() * s["scale"]
        score = (q.flatten(1, 2) @ k.transpose(1, 2)).view(B, N, Hq, -1)
        allowed = torch.zeros(B, N, tok.numel() + N, dtype=torch.bool, device=dev)
        allowed[:, :, :tok.numel()] = seen[:, None]
        allowed[row, num, tok.numel():] = mine
        score.masked_fill_(~allowed[:, :, None], -math.inf)
        o, lse = _softmax(score.flatten(1, 2), v)
        o, lse = o.view(B, N, Hq, d)[row, num], lse.view(B, N, Hq)[row, num]
    else:
        # by nodes: each against the tokens selected for it and its row's drafts
        n = lens[row]
        pools = torch.cat([s["idx"].long(), torch.where(n % 4 > 0, n // 4, -1)[:, None]], 1)
        tok = (pools[:, :, None] * 4 + torch.arange(4, device=dev)).flatten(1)
        seen = torch.cat([(tok >= 0) & (tok < n[:, None]), mine], 1)
        tok = tok.clamp(min=0, max=table.shape[1] * page - 1)
        where = table[row].gather(1, tok // page).clamp(min=0)
        k, v = (torch.cat([s[x][where, tok % page].float(), y[row]], 1) for x, y in (("k", drafts[0]), ("v", drafts[1])))
        score = (s["q"].float() * s["scale"]) @ k.transpose(1, 2)
        o, lse = _softmax(score.masked_fill_(~seen[:, None], -math.inf), v)
    return {"o": o.to(s["q"].dtype), "lse": lse}


def _plain_commit(s):
    c, table, lens = s["case"], s["table"].long(), s["lens"].long()
    page, dev, B, N, di = c["page"], lens.device, c["batch"], c["nodes"], c["di"]
    row, num, mine = _tree_of(s)
    # the accepted node's ancestors, for every row; a node's place behind the cached end is its depth - 1
    path = torch.zeros(B, N, dtype=torch.bool, device=dev)
    last = s["accepted"].long()
    whose = (s["offsets"].long()[:-1] + last).clamp(min=0, max=max(0, row.numel() - 1))
    path = mine[whose] & (last >= 0)[:, None]
    new = path.sum(1)
    take = path[row, num]
    tok = take.nonzero()[:, 0]
    r = row[tok]
    pos = lens[r] + mine[tok].sum(1) - 1
    where = table[r, pos // page]
    s["k"][where, pos % page], s["v"][where, pos % page] = s["new_k"][tok], s["new_v"][tok]
    # indexer keys from the row's first open pool on: what the tail kept, then the new ones
    first = lens // 4 * 4
    seq = torch.zeros(B, (N + 3) // 4 * 4 + 4, di, device=dev)
    seq[:, :3] = s["ktail"][table.gather(1, (first // page)[:, None])[:, 0].clamp(min=0)].float()
    seq[r, pos - first[r]] = s["new_kidx"][tok].float()
    pools = seq.view(B, -1, 4, di)
    keys = (pools[:, :, 0] + pools[:, :, 1] + pools[:, :, 2] + pools[:, :, 3]).to(s["kpool"].dtype)
    done = pos % 4 == 3
    s["kpool"][where[done], pos[done] % page // 4] = keys[r[done], (pos[done] - first[r[done]]) // 4]
    after = lens + new
    open_ = pos >= (after // 4 * 4)[r]
    # kept keys of a pool that is still open stay where they are
    s["ktail"][where[open_], pos[open_] % 4] = s["new_kidx"][tok[open_]]
    s["lens_out"].copy_(after)
    return _outputs(s)


def _counted(refs, table, entries, by):
    refs.index_add_(0, table.clamp(min=0).flatten(), torch.where(entries, by, 0).flatten().to(refs.dtype))


def _plain_branch(s):
    c, refs, page, dev = s["case"], s["refs"], s["case"]["page"], s["refs"].device
    col = torch.arange(s["table"].shape[1], device=dev)
    # release
    old = s["b_table"].long()
    _counted(refs, old, col < -(-s["b_grown"].long() // page)[:, None], -1)
    # fork
    s["b_lens"].copy_(s["lens"][s["from"].long()])
    lens = s["b_lens"].long()
    held = col < -(-lens // page)[:, None]
    table = torch.where(held, s["table"][s["from"].long()].long(), -1)
    _counted(refs, table, held, 1)
    # reserve
    grown = lens + c["grow"]
    copy = (col == (lens // page)[:, None]) & held & (lens % page > 0)[:, None] & (refs[table.clamp(min=0)] > 1)
    want = copy | (~held & (col < -(-grown // page)[:, None]))
    free = torch.argsort((refs > 0).to(torch.int8), stable=True)
    place = (want.flatten().cumsum(0) - 1).view_as(want)
    got = free[place.clamp(min=0, max=free.numel() - 1)]
    _counted(refs, table, copy, -1)
    _counted(refs, got, want, 1)
    at = copy.nonzero()
    src, dst = table[at[:, 0], at[:, 1]], got[at[:, 0], at[:, 1]]
    part = (lens[at[:, 0]] % page)[:, None]
    for x, n in (("k", part), ("v", part), ("kpool", part // 4)):
        inside = (torch.arange(s[x].shape[1], device=dev) < n)[..., None]
        s[x][dst] = torch.where(inside, s[x][src], s[x][dst])
    s["ktail"][dst] = s["ktail"][src]
    s["b_table"].copy_(torch.where(want, got, table))
    s["b_grown"].copy_(grown)
    s["missing"].zero_()
    return _outputs(s)


def _plain_compact(s):
    s["table"].copy_(s["table0"])   # the rows where they were, so that a pass has something to move
    s["refs"].copy_(s["refs0"])
    refs = s["refs"]
    page = torch.arange(refs.numel(), device=refs.device)
    used = refs > 0
    n = used.sum()
    src, dst = (used & (page >= n)).nonzero()[:, 0], (~used & (page < n)).nonzero()[:, 0]
    for x in ("k", "v", "kpool", "ktail"):
        s[x][dst] = s[x][src]
    to = torch.where(used, page, -1)
    to[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    s["table"].copy_(torch.where(s["table"] >= 0, to[s["table"].clamp(min=0).long()], -1))
    s["remap"].copy_(to)
    s["used"].copy_(n.view(1))
    return _outputs(s)


# ------------------------------------------------------------------------------------------------- exact values


def _spin(z, positions, freq, interleaved, back=False):
    """z [T, H, d] in 64 bits, pairs as complex numbers, turned by exp(i a) (or back)."""
    z, h = z.clone(), freq.numel()
    i = torch.arange(h, device=z.device)
    re, im = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    a = positions.double()[:, None] * freq
    w = torch.complex(z[..., re], z[..., im]) * torch.polar(torch.ones_like(a), -a if back else a)[:, None]
    z[..., re], z[..., im] = w.real, w.imag
    return z


def _exact_norm(c, s):
    out = {}
    T = c["tokens"]
    pos = s["positions"] if s["positions"] is not None else torch.arange(T, device=s["q"].device)
    for n in ("q", "k"):
        x = s[n].double().view(T, -1, c["d"]) if n == "k" else s[n].double()
        ms = x.pow(2).sum(-1) / c["d"] + EPS
        w = s[n + "_weight"].double()
        if c["op"] == "norm":
            y = x / ms.sqrt()[..., None] * w
            if c["rot"]:
                y = _spin(y, pos, s["freq"], c["interleaved"])
            out[n + "_out"] = y.view(s[n].shape)
            continue
        dy = s["d" + n + "_out"].double().view(x.shape)
        if c["rot"]:
            dy = _spin(dy, pos, s["freq"], c["interleaved"], back=True)
        out["d" + n + "_weight"] = torch.einsum("thc,thc,th->c", dy, x, ms.rsqrt())
        dy = dy * w
        # d/dx (x m^-1/2) = m^-1/2 dy - x m^-3/2 <dy, x> / d
        dx = dy / ms.sqrt()[..., None] - x * ((dy * x).sum(-1) / c["d"] * ms.pow(-1.5))[..., None]
        out["d" + n] = dx.view(s[n].shape)
    return out


def _exact_tree(c, s):
    lens, dev, page, d = _lens(c), s["q"].device, c["page"], c["d"]
    table, offs, up = s["table"].cpu(), s["offsets"].tolist(), _parents(c)
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=dev)
    idx = None if s["idx"] is None else s["idx"].cpu()
    for b, n in enumerate(lens):
        flat = (table[b].long()[:, None] * page + torch.arange(page)).flatten()[:n]
        for i in range(len(up[b])):
            t = offs[b] + i
            line, j = [], i
            while j >= 0:
                line.append(offs[b] + j)
                j = up[b][j]
            at = flat
            if idx is not None:
                p = idx[t][idx[t] >= 0].long()
                at = flat[torch.cat([(p[:, None] * 4 + torch.arange(4)).flatten(), torch.arange(n // 4 * 4, n)])]
            if idx is not None or i == 0:
                at = at.to(dev)
                kc, vc = s["k"].view(-1, d)[at].double(), s["v"].view(-1, d)[at].double()
            line = torch.tensor(line, device=dev)
            z = s["q"][t].double() @ torch.cat([kc.T, s["new_k"][line].double().T], 1) / math.sqrt(d)
            lse[t] = torch.logsumexp(z, -1)
            p = (z - lse[t][:, None]).exp()
            o[t] = p[:, :kc.shape[0]] @ vc + p[:, kc.shape[0]:] @ s["new_v"][line].double()
    return {"o": o, "lse": lse}


def _exact_commit(c, s):
    out = {x: s[x].double() for x in ("k", "v", "kpool", "ktail")}
    page, up, offs, table = c["page"], _parents(c), s["offsets"].tolist(), s["table"].tolist()
    src, dst, keys, to, tails, tail_to = [], [], [], [], [], []
    base = s["new_k"].shape[0]
    for b, n in enumerate(_lens(c)):
        line, j = [], _last(c, b)
        while j >= 0:
            line.insert(0, offs[b] + j)
            j = up[b][j]
        if not line:
            continue
        for i, t in enumerate(line):
            src.append(t)
            dst.append(table[b][(n + i) // page] * page + (n + i) % page)
        # rows of [new_kidx; ktail]
        first = n // 4 * 4
        seq = [base + 3 * table[b][first // page] + j for j in range(n - first)] + line
        for j in range(0, len(seq) // 4 * 4, 4):
            keys.append(seq[j:j + 4])
            to.append(table[b][(first + j) // page] * (page // 4) + (first + j) % page // 4)
        for j in range(len(seq) // 4 * 4, len(seq)):
            tails.append(seq[j])
            tail_to.append(3 * table[b][(first + j) // page] + j % 4)
    dev = s["k"].device
    rows = torch.cat([s["new_kidx"].double(), s["ktail"].double().flatten(0, 1)])
    ix = lambda x: torch.tensor(x, dtype=torch.int64, device=dev)  # noqa: E731
    for x in ("k", "v"):
        out[x].view(-1, c["d"])[ix(dst)] = s["new_" + x].double()[ix(src)]
    if keys:
        out["kpool"].view(-1, c["di"])[ix(to)] = rows[ix(keys)].sum(1)
    if tails:
        out["ktail"].view(-1, c["di"])[ix(tail_to)] = rows[ix(tails)]
    out["lens_out"] = None
    return out


def _exact_branch(c, s):
    """The pages as lists, one row after the other."""
    out = {x: s[x].double() for x in ("k", "v", "kpool", "ktail")}
    lens, page, table, refs = _lens(c), c["page"], s["table"].tolist(), s["refs"].tolist()
    src = s["from"].tolist()
    for p in src:
        for j in range(-(-lens[p] // page)):
            refs[table[p][j]] += 1
    free = [p for p, n in enumerate(refs) if n == 0]
    for p in src:
        n = lens[p]
        if n % page and refs[table[p][n // page]] > 1:
            a, b = table[p][n // page], free.pop(0)
            for x, m in (("k", n % page), ("v", n % page), ("kpool", n % page // 4), ("ktail", 3)):
                out[x][b, :m] = out[x][a, :m]
        for _ in range(-(-n // page), -(-(n + c["grow"]) // page)):
            free.pop(0)
    return {**out, "refs": None, "b_table": None, "b_lens": None, "missing": None}


def _exact_compact(c, s):
    out = {x: s[x].double() for x in ("k", "v", "kpool", "ktail")}
    refs = s["refs"].tolist()
    n = sum(r > 0 for r in refs)
    a, b = [p for p in range(n, len(refs)) if refs[p]], [p for p in range(n) if not refs[p]]
    for x in out:
        out[x][b] = out[x][a]
    return {**out, "refs": None, "table": None, "remap": None, "used": None}


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    return (_exact_norm if op in ("norm", "norm_grad") else {"tree": _exact_tree, "commit": _exact_commit,
                                                             "branch": _exact_branch, "compact": _exact_compact}[op])(c, s)
