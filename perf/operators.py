"""The serving operators (causal attention over packed prompts, and the paged
kvi8r cache with its tree attention, appends, reads, page copies and row
compaction) as cases to be measured.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, rounded once) or, with ``own`` set, through the framework's entry
points.  Codes and scales of the cache are those of the kvi8r store: rows are
rotated by the orthonormal 128-wide Hadamard matrix, given one fp16 scale
absmax / 127 and rounded to int8.
"""
import math
import random

import torch

own = False

D = 128
DEV = "cuda"


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one short prompt of a chat: the time to its first token is latency
        dict(name="prompt one 500", op="prompt", q_heads=32, kv_heads=8, seqs=1, max_q=500, max_prefix=0, causal=True, mix=0),
        # chunks of many prompts packed into one batch, each behind a prefix of its own
        dict(name="prompt packed chunks", op="prompt", q_heads=24, kv_heads=8, seqs=13, max_q=1500, max_prefix=1000, causal=True, mix=5),
        # one long document
        dict(name="prompt long 16384", op="prompt", q_heads=8, kv_heads=2, seqs=1, max_q=16384, max_prefix=0, causal=True, mix=0),
        # one new token of one sequence over a short cache: latency
        dict(name="tree one token", op="tree", q_heads=32, kv_heads=8, page_size=64, seqs=1, max_len=1024, max_nodes=1, mix=0),
        # one new token for each sequence of a batch, their lengths far apart
        dict(name="tree batch of tokens", op="tree", q_heads=32, kv_heads=8, page_size=64, seqs=33, max_len=32768, max_nodes=1, mix=7),
        # trees of up to 64 drafted tokens over long caches
        dict(name="tree drafts", op="tree", q_heads=32, kv_heads=8, page_size=64, seqs=8, max_len=16384, max_nodes=64, mix=3),
        # a decoding step's new rows, with padded entries of a captured batch
        dict(name="append tokens", op="append", kv_heads=8, page_size=64, rows=37),
        # whole prompts written into the cache and read back
        dict(name="append prompts", op="append", kv_heads=8, page_size=64, rows=65536),
        # the page in which a forked sequence goes on, copied before it is written
        dict(name="copy forked tails", op="copy", kv_heads=8, page_size=64, pages=24),
        # pages moved together so that a part of the pool falls free
        dict(name="copy pool", op="copy", kv_heads=8, page_size=64, pages=1500),
        # the accepted path of one small draft moves to its place
        dict(name="keep one draft", op="keep", kv_heads=8, page_size=64, seqs=1, max_len=1024, max_nodes=7, mix=0),
        # the same for a batch with large trees over many heads
        dict(name="keep batch", op="keep", kv_heads=32, page_size=64, seqs=48, max_len=2048, max_nodes=64, mix=2),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "tree", "tree", "append", "copy", "keep"])
    mix = rng.randrange(1, 1 << 20)
    page = rng.choice([16, 32, 64, 128])
    q_heads, kv_heads = rng.choice([(8, 8), (8, 2), (8, 1), (24, 8), (24, 4), (32, 8), (32, 32), (32, 4)])
    if op == "prompt":
        seqs = _log_int(rng, 1, 32)
        # the pairs of all heads stay below the largest listed case's
        most = int(math.sqrt(8 * 16384 ** 2 / (q_heads * seqs)) * 0.6)
        max_q = _log_int(rng, 1, most)
        prefix = rng.choice([0, 0, rng.randrange(1, most // 2 + 2)])
        return dict(op=op, q_heads=q_heads, kv_heads=kv_heads, seqs=seqs, max_q=max_q, max_prefix=prefix,
                    causal=rng.random() < 0.75, mix=mix)
    if op == "tree":
        seqs = _log_int(rng, 1, 64)
        nodes = rng.choice([1, rng.randrange(2, 65)])
        most = max(128, min(65536, (8 * 16384 * 8) // (seqs * kv_heads)))
        return dict(op=op, q_heads=q_heads, kv_heads=kv_heads, page_size=page, seqs=seqs,
                    max_len=_log_int(rng, 65, most), max_nodes=nodes, mix=mix)
    if op == "append":
        return dict(op=op, kv_heads=kv_heads, page_size=page, rows=_log_int(rng, 1, 8 * 65536 // kv_heads // 2))
    if op == "copy":
        return dict(op=op, kv_heads=kv_heads, page_size=page, pages=_log_int(rng, 1, 1500 * 8 * 64 // (kv_heads * page)))
    return dict(op=op, kv_heads=kv_heads, page_size=page, seqs=_log_int(rng, 1, 64), max_len=rng.randrange(65, 2048),
                max_nodes=rng.randrange(1, 65), mix=mix)


def _lengths(case):
    """Per sequence (new tokens or nodes, tokens in all), from the case alone."""
    r = random.Random(case["mix"])
    out = []
    for i in range(case["seqs"]):
        if case["op"] == "prompt":
            q = case["max_q"] if i == 0 else _log_int(r, max(1, case["max_q"] // 24), case["max_q"])
            p = case["max_prefix"] if i == 0 else r.randrange(0, case["max_prefix"] + 1)
            out.append((q, q + p))
        else:
            m = case["max_nodes"] if i == 0 else r.randrange(1 + case["max_nodes"] // 2, case["max_nodes"] + 1)
            n = case["max_len"] if i == 0 else _log_int(r, max(case["max_nodes"], case["max_len"] // 64), case["max_len"])
            out.append((m, n))
    return out


def work(case):
    op = case["op"]
    if op in ("append", "copy"):
        if op == "append":
            n = case["kv_heads"] * case["rows"]
            return {"bytes": 2 * 2 * n * (2 * D + D + 2), "flops": 0}
        return {"bytes": 2 * 2 * case["pages"] * case["page_size"] * case["kv_heads"] * (D + 2), "flops": 0}
    lens = _lengths(case)
    if op == "keep":
        # about a third of the nodes are kept
        return {"bytes": 2 * 2 * sum(m for m, _ in lens) // 3 * case["kv_heads"] * (D + 2) + 64, "flops": 0}
    if op == "prompt":
        pairs = sum(q * (n - q) + q * (q + 1) // 2 if case["causal"] else q * n for q, n in lens)
        rows = 2 * case["q_heads"] * sum(q for q, _ in lens) + 2 * case["kv_heads"] * sum(n for _, n in lens)
        return {"bytes": rows * 2 * D, "flops": 4 * D * case["q_heads"] * pairs}
    rows = 2 * case["q_heads"] * sum(m for m, _ in lens)
    return {"bytes": rows * 2 * D + 2 * case["kv_heads"] * sum(n for _, n in lens) * (D + 2),
            "flops": 4 * D * case["q_heads"] * sum(m * n for m, n in lens)}


# ------------------------------------------------------------------ inputs --
def _hadamard(dtype=torch.float32):
    i = torch.arange(D, device=DEV)
    x = i[:, None] & i[None, :]
    odd = torch.zeros_like(x)
    odd = odd ^ x ^ (x >> 1) ^ (x >> 2) ^ (x >> 3) ^ (x >> 4) ^ (x >> 5) ^ (x >> 6)
    return (1 - 2 * (odd & 1)).to(dtype) / math.sqrt(D)


def _quantise(x, had):
    """Rows of x [..., 128] -> (int8 codes, fp16 scales) of the kvi8r store."""
    y = x.to(had.dtype) @ had
    s = (y.abs().amax(-1) / 127).to(torch.float16)
    c = torch.where(s[..., None] > 0, y / s[..., None].to(y.dtype), torch.zeros_like(y))
    return c.round().clamp(-127, 127).to(torch.int8), s


def _dequantise(codes, scales):
    return codes.to(torch.float16) * scales[..., None]


def _normal(shape, gen, outliers=False):
    x = torch.randn(shape, generator=gen, device=DEV)
    if outliers:
        x[..., ::32] *= 20.0
    return x


def _cu(counts):
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def _pool(case, pages, gen, fill):
    h, p = case["kv_heads"], case["page_size"]
    if not fill:
        return {k: torch.zeros((pages, h, p, D), dtype=torch.int8, device=DEV) for k in ("k_codes", "v_codes")} | \
            {k: torch.zeros((pages, h, p), dtype=torch.float16, device=DEV) for k in ("k_scales", "v_scales")}
    had, pool = _hadamard(), {}
    for k in ("k", "v"):
        # keys have a few outlier channels, which the rotation spreads
        pool[k + "_codes"], pool[k + "_scales"] = _quantise(_normal((pages, h, p, D), gen, k == "k"), had)
    return pool


def _table(case, lens, gen):
    """Page 0 is left out of every table; the pages of a sequence lie anywhere."""
    p = case["page_size"]
    need = [-(-n // p) for _, n in lens]
    order = (torch.randperm(sum(need), generator=gen, device=DEV) + 1).to(torch.int32)
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, sum(need) + 1


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    s = {"case": case, "had": _hadamard()}
    if op == "prompt":
        lens = _lengths(case)
        nq, nk = sum(q for q, _ in lens), sum(n for _, n in lens)
        s["q"] = _normal((case["q_heads"], nq, D), gen).to(torch.bfloat16)
        s["k"] = _normal((case["kv_heads"], nk, D), gen).to(torch.bfloat16)
        s["v"] = _normal((case["kv_heads"], nk, D), gen).to(torch.bfloat16)
        s["cu_q"], s["cu_k"] = _cu([q for q, _ in lens]), _cu([n for _, n in lens])
        s["max_q"], s["max_k"] = max(q for q, _ in lens), max(n for _, n in lens)
        return s
    if op == "append":
        n, p = case["rows"], case["page_size"]
        pages = -(-n // p) + 1
        s |= _pool(case, pages, gen, False)
        s["k"] = _normal((case["kv_heads"], n, D), gen, True).to(torch.bfloat16)
        s["v"] = _normal((case["kv_heads"], n, D), gen).to(torch.bfloat16)
        page = (torch.randperm(pages - 1, generator=gen, device=DEV) + 1).repeat_interleave(p)[:n]
        rows = page * p + torch.arange(n, device=DEV) % p
        rows[5::8192] = -1
        s["rows"] = rows.to(torch.int32)
        return s
    if op == "copy":
        n = case["pages"]
        s |= _pool(case, 2 * n, gen, True)
        order = torch.randperm(2 * n, generator=gen, device=DEV).to(torch.int32)
        s["src"], s["dst"] = order[:n].contiguous(), order[n:].contiguous()
        return s
    lens = _lengths(case)
    s["table"], pages = _table(case, lens, gen)
    s |= _pool(case, pages, gen, True)
    s["lengths"] = torch.tensor([n for _, n in lens], dtype=torch.int32, device=DEV)
    s["cu"] = _cu([m for m, _ in lens])
    s["max_m"], s["max_k"] = max(m for m, _ in lens), max(n for _, n in lens)
    nodes = sum(m for m, _ in lens)
    at = torch.arange(nodes, device=DEV)
    first = torch.repeat_interleave(s["cu"][:-1], s["cu"].diff()).long()
    j = at - first
    u = torch.rand(nodes, generator=gen, device=DEV)
    if op == "keep":
        s["keep"] = (u < 1 / 3).to(torch.uint8)
        return s
    s["q"] = _normal((case["q_heads"], nodes, D), gen).to(torch.bfloat16)
    # the parent is one of the nodes before, mostly a late one; the first node is the root
    s["parents"] = torch.where(j > 0, (j * u.sqrt()).long().clamp(max=D), -1).to(torch.int32)
    return s


# -------------------------------------------------------------- plain form --
def _attend(q, k, v, see, scale):
    """q [n, h, rows, d], k and v [n, h, keys, d], see [n, 1, rows, keys]."""
    x = (q @ k.transpose(-1, -2)) * scale
    x = torch.where(see, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    z = e.sum(-1, keepdim=True)
    o = (e @ v) / torch.where(z == 0, 1.0, z)
    return o, (top + torch.log(z)).squeeze(-1)


def _packed(x, cu, most):
    """[h, rows, ...] packed by cu -> [n, h, most, ...] padded, and which rows are real."""
    at = torch.arange(most, device=DEV)
    real = at < cu.diff()[:, None]
    idx = (cu[:-1, None] + at).clamp(max=x.shape[1] - 1).long()
    return x[:, idx].transpose(0, 1), real


def _unpack(o, cu, rows):
    """[n, h, most, ...] -> [h, rows, ...]."""
    at = torch.arange(rows, device=DEV)
    seq = torch.searchsorted(cu, at, right=True) - 1
    return o[seq, :, at - cu[seq].long()].transpose(0, 1)


def _plain_prompt(s):
    case = s["case"]
    hq, hk = case["q_heads"], case["kv_heads"]
    g = hq // hk
    q, _ = _packed(s["q"].float(), s["cu_q"], s["max_q"])
    k, real = _packed(s["k"].float(), s["cu_k"], s["max_k"])
    v, _ = _packed(s["v"].float(), s["cu_k"], s["max_k"])
    n, mq, mk = q.shape[0], s["max_q"], s["max_k"]
    see = real[:, None, :].expand(n, mq, mk)
    if case["causal"]:
        off = (s["cu_k"].diff() - s["cu_q"].diff())[:, None, None]
        see = see & (torch.arange(mk, device=DEV) <= torch.arange(mq, device=DEV)[:, None] + off)
    see = see[:, None, None].expand(n, 1, g, mq, mk).reshape(n, 1, g * mq, mk)
    o, lse = _attend(q.reshape(n, hk, g * mq, D), k, v, see, 1 / math.sqrt(D))
    o, lse = o.reshape(n, hq, mq, D), lse.reshape(n, hq, mq)
    rows = s["q"].shape[1]
    return {"o": _unpack(o, s["cu_q"], rows).to(torch.bfloat16), "lse": _unpack(lse, s["cu_q"], rows)}


def _plain_tree(s):
    case = s["case"]
    hq, hk, p = case["q_heads"], case["kv_heads"], case["page_size"]
    g, mm, mk = hq // hk, s["max_m"], s["max_k"]
    had = s["had"]
    n = case["seqs"]
    pos = torch.arange(mk, device=DEV)
    page = s["table"].long()[:, pos // p]
    k = _dequantise(s["k_codes"][page, :, pos % p], s["k_scales"][page, :, pos % p]).float().transpose(1, 2)
    v = _dequantise(s["v_codes"][page, :, pos % p], s["v_scales"][page, :, pos % p]).float().transpose(1, 2)
    q, real = _packed((s["q"].float() @ had).to(torch.float16).float(), s["cu"], mm)
    par, _ = _packed(s["parents"][None], s["cu"], mm)
    # node j's path to its root: the powers of "itself or its parent"
    up = torch.eye(mm, device=DEV) + (par.squeeze(1)[..., None] == torch.arange(mm, device=DEV)) * real[..., None]
    path = torch.linalg.matrix_power(up, max(1, mm - 1)) > 0
    base = (s["lengths"] - s["cu"].diff()).long()
    node = pos - base[:, None]
    drafted = torch.gather(path, 2, node.clamp(0, mm - 1)[:, None, :].expand(n, mm, mk))
    see = (node < 0)[:, None] | (drafted & (pos < s["lengths"][:, None])[:, None] & (node >= 0)[:, None])
    see = see[:, None, None].expand(n, 1, g, mm, mk).reshape(n, 1, g * mm, mk)
    o, lse = _attend(q.reshape(n, hk, g * mm, D), k, v, see, 1 / math.sqrt(D))
    o, lse = (o @ had).reshape(n, hq, mm, D), lse.reshape(n, hq, mm)
    rows = s["q"].shape[1]
    return {"o": _unpack(o, s["cu"], rows).to(torch.bfloat16), "lse": _unpack(lse, s["cu"], rows)}


def _plain_append(s):
    p, had, rows = s["case"]["page_size"], s["had"], s["rows"].long()
    there = rows >= 0
    page, slot = rows.clamp(min=0) // p, rows.clamp(min=0) % p
    out = {}
    for t in ("k", "v"):
        c, z = _quantise(s[t].float(), had)
        codes, scales = s[t + "_codes"], s[t + "_scales"]
        # (a row that is left out writes what row 0, which no sequence uses, holds)
        codes[page, :, slot] = torch.where(there[:, None, None], c.transpose(0, 1), codes[0, :, 0])
        scales[page, :, slot] = torch.where(there[:, None], z.transpose(0, 1), scales[0, :, 0])
        x = _dequantise(codes[page, :, slot], scales[page, :, slot]).float() @ had
        out[t] = torch.where(there[:, None, None], x, 0.0).transpose(0, 1).to(torch.bfloat16).contiguous()
        out[t + "_scales"] = scales
    return out


def _pools(s):
    return {k: s[k] for k in ("k_codes", "v_codes", "k_scales", "v_scales")}


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for t in _pools(s).values():
        t[dst] = t[src]
    return _pools(s)


def _plain_keep(s):
    p = s["case"]["page_size"]
    keep, real = _packed(s["keep"][None].bool(), s["cu"], s["max_m"])
    keep = keep.squeeze(1) & real
    base = (s["lengths"] - s["cu"].diff()).long()[:, None]
    rank = keep.long().cumsum(1) - 1
    j = torch.arange(s["max_m"], device=DEV)
    last = s["lengths"].long()[:, None] - 1
    # place j takes the row of the j-th kept node; the places behind (and the
    # padded ones, at the sequence's last row) write their own row again
    taken = j < keep.long().sum(1, keepdim=True)
    src = torch.zeros_like(rank).scatter_add(1, torch.where(keep, rank, 0), torch.where(keep, j, 0))
    src_pos = torch.minimum(base + torch.where(taken, src, j), last)
    dst_pos = torch.minimum(base + j, last)
    table = s["table"].long()
    sp, dp = table.gather(1, src_pos // p), table.gather(1, dst_pos // p)
    for t in _pools(s).values():
        t[dp, :, dst_pos % p] = t[sp, :, src_pos % p]
    return _pools(s) | {"lengths": (base[:, 0] + keep.sum(1)).to(torch.int32)}


# --------------------------------------------------------- the framework's --
def _own(s):
    from store_h3kv_build_gb300 import binding as b

    op = s["case"]["op"]
    if op == "prompt":
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
        o = b.attend_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=s["case"]["causal"], lse=lse)
        return {"o": o, "lse": lse}
    if "store" not in s:
        s["store"] = b.PagedStore(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
    store = s["store"]
    if op == "tree":
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
        o = b.attend_tree(s["q"], store, s["table"], s["lengths"], s["cu"], s["parents"], lse=lse)
        return {"o": o, "lse": lse}
    if op == "append":
        b.paged_append(s["k"], s["v"], store, s["rows"])
        k, v = b.paged_read(store, s["rows"])
        return {"k": k, "v": v, "k_scales": store.k_scales, "v_scales": store.v_scales}
    if op == "copy":
        b.paged_copy(store, s["src"], s["dst"])
        return _pools(s)
    return _pools(s) | {"lengths": b.paged_keep(store, s["table"], s["lengths"], s["cu"], s["keep"])}


PLAIN = {"prompt": _plain_prompt, "tree": _plain_tree, "append": _plain_append, "copy": _plain_copy, "keep": _plain_keep}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------- in 64 bits --
def exact(case, seed):
    """The operators' definitions, sequence by sequence in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    had = torch.ones((1, 1), dtype=f64, device=DEV)
    for _ in range(7):
        had = torch.cat([torch.cat([had, had], 1), torch.cat([had, -had], 1)], 0)
    had = had / math.sqrt(D)
    if op in ("copy", "keep"):
        return _exact_moved(s)
    if op == "append":
        out, p = {}, case["page_size"]
        for t in ("k", "v"):
            y = s[t].to(f64) @ had
            z = (y.abs().max(dim=-1).values / 127).to(torch.float16).to(f64)
            c = torch.round(y / z.clamp(min=1e-30)[..., None]).clamp(-127, 127)
            real = (c * z[..., None]).to(torch.float16).to(f64) @ had
            gone = s["rows"] < 0
            real[:, gone] = 0
            scales = torch.zeros(s[t + "_scales"].shape, dtype=f64, device=DEV)
            flat = scales.transpose(1, 2).reshape(-1, scales.shape[1])
            flat[s["rows"][~gone].long()] = z.T[~gone]
            out[t] = real
            out[t + "_scales"] = flat.reshape(-1, p, scales.shape[1]).transpose(1, 2)
        return out
    lens = _lengths(case)
    hq, hk = case["q_heads"], case["kv_heads"]
    g = hq // hk
    o = torch.zeros(s["q"].shape, dtype=f64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=f64, device=DEV)
    q0 = k0 = 0
    for i, (m, n) in enumerate(lens):
        if op == "prompt":
            see = torch.ones((m, n), dtype=torch.bool, device=DEV)
            if case["causal"]:
                see = see.tril(n - m)
        else:
            see = torch.ones((m, n), dtype=torch.bool, device=DEV)
            rows = []
            for j, par in enumerate(s["parents"][q0:q0 + m].tolist()):
                row = list(rows[par]) if par >= 0 else [False] * m
                row[j] = True
                rows.append(row)
            see[:, n - m:] = torch.tensor(rows, device=DEV)
        for h in range(hq):
            if op == "prompt":
                q, k, v = s["q"][h, q0:q0 + m].to(f64), s["k"][h // g, k0:k0 + n].to(f64), s["v"][h // g, k0:k0 + n].to(f64)
            else:
                if h % g == 0:
                    pages = s["table"][i, :-(-n // case["page_size"])].long()
                    kv = []
                    for t in ("k", "v"):
                        c, z = s[t + "_codes"][pages, h // g].reshape(-1, D)[:n], s[t + "_scales"][pages, h // g].reshape(-1)[:n]
                        kv.append((c.to(f64) * z.to(f64)[:, None]).to(torch.float16).to(f64))
                q, (k, v) = (s["q"][h, q0:q0 + m].to(f64) @ had).to(torch.float16).to(f64), kv
            x = (q @ k.T).mul_(1 / math.sqrt(D)).masked_fill_(~see, -math.inf)
            lse[h, q0:q0 + m] = torch.logsumexp(x, -1)
            r = torch.nan_to_num(torch.softmax(x, -1)) @ v
            o[h, q0:q0 + m] = r if op == "prompt" else r @ had
        q0, k0 = q0 + m, k0 + n
    return {"o": o, "lse": lse}


def _exact_moved(s):
    """Moved rows are not computed: the scales as they come to lie, one by one."""
    out = {"k_codes": None, "v_codes": None, "lengths": None}
    for t in ("k_scales", "v_scales"):
        old = s[t].double().cpu()
        new = old.clone()
        if s["case"]["op"] == "copy":
            for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
                new[b] = old[a]
        else:
            p, cu, keep, table = s["case"]["page_size"], s["cu"].tolist(), s["keep"].tolist(), s["table"].tolist()
            for i, n in enumerate(s["lengths"].tolist()):
                base = to = n - (cu[i + 1] - cu[i])
                for j in range(cu[i + 1] - cu[i]):
                    if keep[cu[i] + j]:
                        a, b = base + j, to
                        new[table[i][b // p], :, b % p] = old[table[i][a // p], :, a % p]
                        to += 1
        out[t] = new
    if s["case"]["op"] == "copy":
        del out["lengths"]
    return out
