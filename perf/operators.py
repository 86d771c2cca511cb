"""What is measured of the paged decode operators: cases, plain forms, exact values.

A decoder that continues sequences with this layer keeps, for every sequence, the tokens' keys and values and
their pool keys in fixed-size pages, and for every new token does three things:

  append   writes the new tokens' k, v (k and q rotated to their positions on the way, or not at all: the layer's
           own setting) into their pages, and every pool key that the new tokens complete;
  topk     scores all complete pools of every row's sequence with the row's indexer query and keeps the k best;
  sel      attention of one query token per row over the selected pools' tokens and the row's own partial pool;
  all      attention of one query token per row over the whole cache (a dense layer, or a context short enough).

Definitions (row b holds lens[b] tokens, its query is the token at position lens[b] - 1; a pool is 4 tokens):

  append   token j of row b's n new ones has position p = lens[b] - n + j and goes to row p % page of page
           block_table[b, p // page].  With a rotation of `rot` channels, the pair (x, y) of channels
           (i, i + rot/2), or (2i, 2i + 1) when interleaved, becomes (x cos a - y sin a, x sin a + y cos a) with
           a = p * freq[i]; other channels are copied.  Pool key = the sum of the pool's 4 k_idx rows in fp32, in
           token order, rounded once.  The k_idx rows of the sequence's last, incomplete pool are kept in `ktail`.
  topk     s[b, p] = sum_h w[b, h] max(0, q_idx[b, h] . kpool[p]) for p < lens[b] // 4; the min(k, lens[b] // 4)
           best by (score descending, pool ascending), listed ascending, then -1.
  sel/all  o[b, h] = softmax_j(scale q[b, h] . k[j]) v[j], lse[b, h] = log sum_j exp(scale q[b, h] . k[j]);
           a row without keys gives o = 0 and lse = -inf.

Layer shapes (heads, widths, k, dtypes, the 10% needle tokens, the integer indexer inputs that make every fp32 score
exact) are those of the repository's workloads; sequence counts, lengths and page sizes are generic.
"""
import math

import torch

own = False

BF16, FP32 = "bf16", "fp32"


def _case(op, name=None, **kw):
    c = {"op": op, "dtype": BF16, "batch": 1, "tokens": 4096, "ragged": False, "Hq": 16, "d": 128, "Hi": 8, "di": 64,
         "k": 512, "page": 64, "rot": 0, "interleaved": False, "past": 0, "needle": 0.0, "ints": 3}
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one step of a serving batch: one new token for each of 48 sequences, half of each head rotated; latency counts
        _case("append", "append_step_b48", batch=48, tokens=30001, ragged=True, rot=64),
        # five prompts (chunks of prompts, behind 1001 cached tokens each) enter the cache in one call, no rotation
        _case("append", "append_prompts_b5", batch=5, tokens=8190, ragged=True, past=1001, page=16),
        # a whole 128k prompt, q and k rotated
        _case("append", "append_prompt_128k", batch=1, tokens=131072, past=0, rot=128, interleaved=True, page=128),
        # one user, long context: the latency of the selected keys' attention
        _case("sel", "sel_b1_128k", tokens=131071, needle=0.1),
        # an ordinary serving batch, contexts of all lengths, one idle row
        _case("sel", "sel_b96_ragged", batch=96, tokens=32765, ragged=True),
        # a full batch of the 32-head layer, the cache far larger than L2
        _case("sel", "sel_b64_h32", batch=64, tokens=65534, Hq=32, di=128),
        # the fp32 layer
        _case("sel", "sel_fp32_b16", dtype=FP32, batch=16, tokens=4093, ragged=True, Hq=8, d=64, Hi=4, k=64, page=16),
        # one user, 1M tokens, dense
        _case("all", "all_b1_1m", tokens=1048573, needle=0.1),
        # a serving batch of the 32-head layer, contexts of all lengths, one idle row
        _case("all", "all_b40_ragged_h32", batch=40, tokens=40001, ragged=True, Hq=32, page=128),
        # one user, 1M tokens, tie-heavy scores
        _case("topk", "topk_b1_1m_ties", tokens=1048576, ints=1),
        # a serving batch of long contexts of the wide indexer
        _case("topk", "topk_b32_128k", batch=32, tokens=131070, ragged=True, di=128),
        # the fp32 layer, short contexts
        _case("topk", "topk_fp32_b5", dtype=FP32, batch=5, tokens=4094, ragged=True, Hi=4, k=64, Hq=8, d=64, page=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append", "sel", "sel", "all", "all", "topk", "topk"])
    dtype = rng.choice([BF16, BF16, FP32])
    c = {"dtype": dtype, "d": rng.choice([64, 128]), "di": rng.choice([64, 128]), "page": rng.choice([4, 16, 20, 64, 64, 100, 128]),
         "ragged": rng.random() < 0.7, "Hq": rng.choice([16, 32, rng.randint(1, 32)]), "Hi": rng.choice([8, 4, rng.randint(1, 8)])}
    wide = 1 if dtype == BF16 else 2   # an fp32 case moves twice the bytes
    c["batch"] = _log(rng, 1, 128)
    if op == "append":
        c["rot"] = rng.choice([0, 16, 64, c["d"]])
        c["interleaved"] = rng.random() < 0.5
        if rng.random() < 0.5:
            c["tokens"] = _log(rng, 1, 60000 // wide)
        else:
            c["tokens"] = _log(rng, 1, 65536 // c["batch"] // wide)
            c["past"] = rng.randint(0, 4097)
    elif op == "sel":
        c["tokens"] = _log(rng, 1, min(262144, 4000000 // c["batch"]) // wide)
        c["k"] = rng.choice([64, 512, rng.randint(1, 1024)])
        c["needle"] = rng.choice([0.0, 0.1]) if dtype == BF16 else 0.0
    elif op == "all":
        c["tokens"] = _log(rng, 1, 1000000 // c["batch"] // wide // (2 if c["Hq"] > 16 else 1))
        c["needle"] = rng.choice([0.0, 0.1]) if dtype == BF16 else 0.0
    else:
        c["tokens"] = _log(rng, 1, min(1048576, 4000000 // c["batch"]) // wide)
        c["k"] = rng.choice([64, 512, rng.randint(1, 1024)])
        c["ints"] = rng.choice([1, 3])
    return _case(op, **c)


def _lens(c):
    """(lengths after the call, new tokens) of every row; row 0 is the longest, one row of a ragged batch is idle."""
    n = [c["tokens"]] * c["batch"]
    if c["ragged"]:
        n = [c["tokens"] if b == 0 else 1 + (b * 2654435761 % 2**32) * c["tokens"] // 2**32 for b in range(c["batch"])]
        if c["batch"] >= 8:
            n[c["batch"] // 2] = 0
    if c["op"] != "append":
        return n, [0] * c["batch"]
    if c["past"] == 0 and c["batch"] > 1 or c["tokens"] == 1:
        return n, [min(1, x) for x in n]             # a decode step: one token per live row
    return [x + c["past"] if x else 0 for x in n], n  # prompts, behind what is cached


def _step(c):
    """Whether an append is a decode step: one new token per row, no offsets."""
    return c["past"] == 0 and c["batch"] > 1 or c["tokens"] == 1


def _elem(c):
    return 2 if c["dtype"] == BF16 else 4


def work(c):
    lens, new = _lens(c)
    e, d, di, Hq, Hi = _elem(c), c["d"], c["di"], c["Hq"], c["Hi"]
    if c["op"] == "append":
        t = sum(new)
        by = t * (4 * d + di) * e + sum(x // 4 - (x - n) // 4 for x, n in zip(lens, new)) * di * e
        return {"bytes": by + (2 * t * Hq * d * e if c["rot"] else 0), "flops": 3 * t * c["rot"] * (Hq + 1) + t * di}
    if c["op"] == "topk":
        pools = sum(x // 4 for x in lens)
        return {"bytes": pools * di * e + c["batch"] * (Hi * di * e + 4 * Hi + 4 * c["k"]), "flops": 2 * Hi * di * pools}
    keys = sum(lens) if c["op"] == "all" else sum(4 * min(c["k"], x // 4) + x % 4 for x in lens)
    by = 2 * keys * d * e + c["batch"] * Hq * (2 * d * e + 4) + (4 * c["k"] * c["batch"] if c["op"] == "sel" else 0)
    return {"bytes": by, "flops": 4 * Hq * d * keys}


def prepare(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = torch.bfloat16 if c["dtype"] == BF16 else torch.float32
    B, d, di, Hq, Hi, page = c["batch"], c["d"], c["di"], c["Hq"], c["Hi"], c["page"]
    lens, new = _lens(c)
    cap = max(4, (max(lens) + 3) // 4 * 4)            # the longest sequence the call may hold
    cols = -(-cap // page)
    need = torch.tensor([-(-x // page) for x in lens])
    pages = int(need.sum()) + 1                       # one page of the pool stays free
    # pages in a random order; entries behind a sequence's last page are never read
    table = torch.full((B, cols), -1, dtype=torch.int32, device=dev)
    used = torch.arange(cols, device=dev)[None, :] < need.to(dev)[:, None]
    table[used] = torch.randperm(pages, generator=g, device=dev)[:int(need.sum())].to(torch.int32)

    def randn(*shape):
        out = torch.empty(shape, dtype=dt, device=dev)
        return out.normal_(generator=g)

    def ints(*shape):
        return torch.randint(-c["ints"], c["ints"] + 1, shape, generator=g, device=dev)

    s = {"case": c, "lens": torch.tensor(lens, dtype=torch.int32, device=dev), "table": table, "scale": d ** -0.5}
    op = c["op"]
    if op != "topk":
        s["k"], s["v"] = randn(pages, page, d), randn(pages, page, d)
    if op in ("append", "topk"):
        s["kpool"] = sum(ints(pages, page // 4, di) for _ in range(4)).to(dt)
    if op == "append":
        t = sum(new)
        s["ktail"] = ints(pages, 3, di).to(dt)
        s["new_k"], s["new_v"], s["new_kidx"] = randn(t, d), randn(t, d), randn(t, di)
        if _step(c) and t < B:                        # a decode step has a row for every sequence, idle ones too
            s["new_k"], s["new_v"], s["new_kidx"] = randn(B, d), randn(B, d), randn(B, di)
        s["offsets"] = None
        if not _step(c):
            s["offsets"] = torch.tensor([0] + new, dtype=torch.int32, device=dev).cumsum(0).to(torch.int32)
        if c["rot"]:
            s["freq"] = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
            s["q"] = randn(s["new_k"].shape[0], Hq, d)
            s["q_out"] = torch.zeros_like(s["q"])
    elif op == "topk":
        s["q_idx"] = ints(B, Hi, di).to(dt)
        s["w"] = (torch.randint(1, 5, (B, Hi), generator=g, device=dev) if c["ints"] == 3 else
                  torch.randint(-1, 2, (B, Hi), generator=g, device=dev)).float()
        s["idx"] = torch.zeros(B, c["k"], dtype=torch.int32, device=dev)
    else:
        s["q"] = randn(B, Hq, d)
        if c["needle"]:
            u = torch.randn(d, generator=g, device=dev)
            u = 4.0 * math.sqrt(d) * u / u.norm()
            hit = torch.rand(pages, page, generator=g, device=dev) < c["needle"]
            s["k"][hit] = (s["k"][hit].float() + u).to(dt)
            hit = torch.rand(B, generator=g, device=dev) < 0.5
            s["q"][hit] = (s["q"][hit].float() + u).to(dt)
        s["idx"] = None
        if op == "sel":
            # min(k, lens // 4) distinct pools of each row, ascending, then -1
            P, k = cap // 4, c["k"]
            elig = (s["lens"] // 4)[:, None]
            r = torch.rand(B, P, generator=g, device=dev)
            r[torch.arange(P, device=dev)[None, :] >= elig] = 2.0
            n = min(k, P)
            pick = r.topk(n, dim=1, largest=False).indices
            pick[torch.arange(n, device=dev)[None, :] >= elig] = P
            pick = pick.sort(dim=1).values
            pick[pick == P] = -1
            s["idx"] = torch.full((B, k), -1, dtype=torch.int32, device=dev)
            s["idx"][:, :n] = pick.to(torch.int32)
        s["o"] = torch.zeros(B, Hq, d, dtype=dt, device=dev)
        s["lse"] = torch.zeros(B, Hq, device=dev)
    if own:
        # the handle and the workspace that a decoder keeps for its lifetime
        import long_context_sparse_dsa_gb300 as dsa
        dims = s["dims"] = dsa.make_dims(cap, Hq, d, Hi, di, c["k"], dtype=c["dtype"])
        s["cache"] = dsa.PagedCache(k=s.get("k"), v=s.get("v"), kpool=s.get("kpool"), ktail=s.get("ktail"))
        if op == "append":
            s["rotation"] = dsa.make_rotation(s["freq"], interleaved=c["interleaved"]) if c["rot"] else None
        else:
            n = dsa.decode_workspace_bytes(dims, B)
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=dev)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        import long_context_sparse_dsa_gb300 as dsa
        if op == "append":
            dsa.cache_append(s["dims"], s["cache"], s["lens"], s["table"], s["new_k"], s["new_v"], s["new_kidx"],
                             offsets=s["offsets"], rotation=s["rotation"], q=s.get("q"), q_out=s.get("q_out"))
            return _appended(s)
        if op == "topk":
            dsa.decode_indexer_topk(s["dims"], s["cache"], s["lens"], s["table"], s["q_idx"], s["w"], s["idx"], s["ws"])
            return s["idx"]
        dsa.decode_attn(s["dims"], s["cache"], s["lens"], s["table"], s["q"], s["o"], s["lse"], s["ws"], idx=s["idx"])
        return {"o": s["o"], "lse": s["lse"]}
    if op == "append":
        return _plain_append(s)
    if op == "topk":
        return _plain_topk(s)
    return _plain_attn(s)


# ------------------------------------------------------------------------------------------------- plain forms


def _appended(s):
    out = {"k": s["k"], "v": s["v"], "kpool": s["kpool"], "ktail": s["ktail"]}
    if s["case"]["rot"]:
        out["q"] = s["q_out"]
    return out


def _rotated(x, angle, interleaved):
    """x [T, H, d], angle [T, rot/2] in 64 bits (far positions); the products in 32 bits, rounded once."""
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    n = 2 * angle.shape[1]
    y = x.float()
    a, b = (y[..., 0:n:2], y[..., 1:n:2]) if interleaved else (y[..., :n // 2], y[..., n // 2:n])
    a, b = a * cos - b * sin, a * sin + b * cos
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, y[..., n:]], -1).to(x.dtype)


def _plain_append(s):
    c, lens, table = s["case"], s["lens"].long(), s["table"].long()
    page, dev = c["page"], lens.device
    B, T = lens.numel(), s["new_k"].shape[0]
    new = s["offsets"].long().diff() if s["offsets"] is not None else torch.ones_like(lens)
    begin = s["offsets"].long()[:-1] if s["offsets"] is not None else torch.arange(B, device=dev)
    tok = torch.arange(T, device=dev)
    row = torch.repeat_interleave(torch.arange(B, device=dev), new, output_size=T)
    pos = lens[row] - new[row] + tok - begin[row]
    live = pos >= 0                                    # an idle row of a decode step appends nothing
    tok, row, pos = tok[live], row[live], pos[live]
    where = table[row, pos // page]
    k = s["new_k"][tok]
    if c["rot"]:
        angle = pos.double()[:, None] * s["freq"]
        k = _rotated(k[:, None], angle, c["interleaved"])[:, 0]
        s["q_out"][tok] = _rotated(s["q"][tok], angle, c["interleaved"])
    s["k"][where, pos % page] = k
    s["v"][where, pos % page] = s["new_v"][tok]
    # the pools that the new tokens complete: each of their 4 keys is new, or kept in the tail
    done = (pos % 4 == 3)
    last, r, w, t = pos[done], row[done], where[done], tok[done]
    key = 0
    for j in range(4):
        back = 3 - j
        fresh = s["new_kidx"][(t - back).clamp(min=0)].float()
        kept = s["ktail"][w, min(j, 2)].float()
        is_new = (last - back >= (lens - new)[r])[:, None]
        key = key + torch.where(is_new, fresh, kept)
    s["kpool"][w, (last % page) // 4] = key.to(s["kpool"].dtype)
    # and the keys of each row's last, incomplete pool are kept
    open_ = pos >= (lens[row] // 4) * 4
    s["ktail"][where[open_], pos[open_] % 4] = s["new_kidx"][tok[open_]]
    return _appended(s)


def _plain_topk(s):
    c, table = s["case"], s["table"].long()
    page, k = c["page"], c["k"]
    B, per = table.shape[0], page // 4
    kp = s["kpool"][table.clamp(min=0)].float().reshape(B, table.shape[1] * per, -1)
    score = (torch.einsum("bhi,bpi->bhp", s["q_idx"].float(), kp).clamp(min=0) * s["w"][:, :, None]).sum(1)
    P = score.shape[1]
    at = torch.arange(P, device=score.device)[None, :]
    elig = (s["lens"].long() // 4)[:, None]
    score = torch.where(at < elig, score + 0.0, -math.inf)
    n = min(k, P)
    best = score.sort(dim=1, descending=True, stable=True).indices[:, :n]
    best = torch.where(torch.arange(n, device=score.device)[None, :] < elig, best, P).sort(dim=1).values
    idx = torch.full((B, k), -1, dtype=torch.int32, device=score.device)
    idx[:, :n] = torch.where(best == P, -1, best).to(torch.int32)
    return idx


def _plain_attn(s):
    c, table, lens = s["case"], s["table"].long(), s["lens"].long()
    page, dev = c["page"], lens.device
    B = lens.numel()
    if s["idx"] is None:
        tok = torch.arange(table.shape[1] * page, device=dev)[None, :].expand(B, -1)
        seen = tok < lens[:, None]
    else:
        idx = torch.cat([s["idx"].long(), torch.where(lens % 4 > 0, lens // 4, -1)[:, None]], 1)
        tok = (idx[:, :, None] * 4 + torch.arange(4, device=dev)).flatten(1)
        seen = (tok >= 0) & (tok < lens[:, None])
    tok = tok.clamp(min=0, max=table.shape[1] * page - 1)
    where = table.gather(1, tok // page).clamp(min=0)
    k, v = (s[x][where, tok % page].float() for x in ("k", "v"))
    score = torch.einsum("bhd,bjd->bhj", s["q"].float(), k) * s["scale"]
    score = torch.where(seen[:, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1)
    v = torch.where(seen[:, :, None], v, 0.0)
    o = torch.einsum("bhj,bjd->bhd", p, v) / torch.where(total == 0, 1.0, total)[..., None]
    lse = torch.where(total == 0, -math.inf, top[..., 0] + total.log())
    return {"o": o.to(s["q"].dtype), "lse": lse}


# ------------------------------------------------------------------------------------------------- exact values


def exact(c, seed):
    if c["op"] == "topk":
        return None                                   # whole numbers: the selection has to be equal
    s = prepare(c, seed)
    lens, new = _lens(c)
    table = s["table"].cpu().tolist()
    page, d = c["page"], c["d"]
    dev = s["k"].device
    if c["op"] != "append":
        o = torch.zeros(c["batch"], c["Hq"], d, dtype=torch.float64, device=dev)
        lse = torch.full((c["batch"], c["Hq"]), -math.inf, dtype=torch.float64, device=dev)
        for b, n in enumerate(lens):
            if n == 0:
                continue
            flat = torch.tensor(table[b][:-(-n // page)], device=dev)
            flat = (flat[:, None] * page + torch.arange(page, device=dev)).flatten()[:n]
            if s["idx"] is not None:
                pools = [p for p in s["idx"][b].tolist() if p >= 0]
                keep = [4 * p + j for p in pools for j in range(4)] + list(range(n // 4 * 4, n))
                flat = flat[torch.tensor(keep, device=dev)]
            k, v = s["k"].view(-1, d)[flat].double(), s["v"].view(-1, d)[flat].double()
            z = s["q"][b].double() @ k.T / math.sqrt(d)
            lse[b] = torch.logsumexp(z, -1)
            o[b] = (z - lse[b][:, None]).exp() @ v
        return {"o": o, "lse": lse}
    out = {x: s[x].double() for x in ("k", "v", "kpool", "ktail")}
    if c["rot"]:
        out["q"] = s["q_out"].double()
    at = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        src = slice(at, at + m) if not _step(c) else slice(b, b + m)
        at += m
        if m == 0:
            continue
        pos = torch.arange(n - m, n, device=dev)
        pg = torch.tensor(table[b], device=dev)[pos // page]
        kk, vv, ki = s["new_k"][src].double(), s["new_v"][src].double(), s["new_kidx"][src].double()
        if c["rot"]:
            # pairs as complex numbers, turned by exp(i a)
            turn = torch.polar(torch.ones((), dtype=torch.float64, device=dev), pos.double()[:, None] * s["freq"])

            def spin(x):
                x, h = x.clone(), c["rot"] // 2
                i = torch.arange(h, device=dev)
                re, im = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + h)
                z = torch.complex(x[..., re], x[..., im]) * (turn if x.dim() == 2 else turn[:, None])
                x[..., re], x[..., im] = z.real, z.imag
                return x
            kk = spin(kk)
            out["q"][src] = spin(s["q"][src].double())
        out["k"][pg, pos % page] = kk
        out["v"][pg, pos % page] = vv
        # the sequence's k_idx from its first open pool on: what the tail kept, then the new ones
        first = (n - m) // 4 * 4
        kept = s["ktail"][table[b][first // page], :(n - m) - first].double()
        ki = torch.cat([kept, ki])
        full = ki.shape[0] // 4
        if full:
            pools = torch.arange(first // 4, first // 4 + full, device=dev)
            out["kpool"][torch.tensor(table[b], device=dev)[4 * pools // page], pools % (page // 4)] = \
                ki[:4 * full].view(full, 4, -1).sum(1)
        rest = ki[4 * full:]
        if rest.shape[0]:
            out["ktail"][table[b][(n - 1) // page], :rest.shape[0]] = rest
    return out
