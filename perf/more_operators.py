"""Attention over packed sequences and over a paged cache's chunks as a benchmark sees them: cases, inputs,
plain forms, 64-bit values.

Three operators of the attention library are described here, each by the call a user makes of it
(``own`` true) and by the same arithmetic in elementary torch operations (``own`` false):

  packed_fwd  attention of sequences of different lengths that lie one after the other, without
              padding between them; query heads share key/value heads
  packed_bwd  its gradients with respect to queries, keys and values
  chunk       attention of any number of new tokens of every sequence (from one to a whole prompt)
              over a paged cache that holds them already, bf16 or e4m3 pages, with a sliding window
              and visible first tokens

Layouts: q, k and v are [tokens, heads, d] tensors: views of one fused projection ("fused"), or of
head-major arrays [heads, tokens, d] as the norm and rotation leave them ("heads"). Sequence b's tokens
are rows starts[b] to starts[b + 1] - 1. A cache is [pages, h_kv, page_size, d], and a page table
[sequences, max_pages] names each sequence's pages (-1 where it has none).
"""
import math

import torch

own = False


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a few short prompts: the smallest call, where latency is what counts
        dict(name="packed_short", op="packed_fwd", seqs=5, q_lo=3, q_hi=61, k_lo=-1, k_hi=-1, pad=0, h_q=8, h_kv=8, d=64,
             causal=True, window=-1, layout="fused"),
        # encoder self-attention of a batch of sentences, no mask inside a sentence
        dict(name="packed_sentences", op="packed_fwd", seqs=64, q_lo=21, q_hi=500, k_lo=-1, k_hi=-1, pad=64, h_q=8,
             h_kv=8, d=64, causal=False, window=-1, layout="fused"),
        # encoder-decoder attention of such a batch: other lengths on both sides
        dict(name="packed_cross", op="packed_fwd", seqs=48, q_lo=1, q_hi=257, k_lo=33, k_hi=1021, pad=0, h_q=16, h_kv=16,
             d=64, causal=False, window=-1, layout="heads"),
        # whole prompts of very different lengths, shared key heads
        dict(name="packed_prompts", op="packed_fwd", seqs=12, q_lo=129, q_hi=4099, k_lo=-1, k_hi=-1, pad=0, h_q=32,
             h_kv=8, d=128, causal=True, window=-1, layout="fused"),
        # two long training sequences, shared key heads
        dict(name="packed_long", op="packed_fwd", seqs=2, q_lo=8192, q_hi=8192, k_lo=-1, k_hi=-1, pad=0, h_q=32, h_kv=8,
             d=128, causal=True, window=-1, layout="heads"),
        # gradients of the sentences
        dict(name="packed_bwd_sentences", op="packed_bwd", seqs=64, q_lo=21, q_hi=500, k_lo=-1, k_hi=-1, pad=64, h_q=8,
             h_kv=8, d=64, causal=False, window=-1, layout="fused"),
        # gradients of packed documents with a sliding window, shared key heads
        dict(name="packed_bwd_window", op="packed_bwd", seqs=9, q_lo=5, q_hi=3301, k_lo=-1, k_hi=-1, pad=0, h_q=12,
             h_kv=4, d=64, causal=True, window=511, layout="fused"),
        # gradients of one long training sequence, shared key heads
        dict(name="packed_bwd_long", op="packed_bwd", seqs=1, q_lo=8192, q_hi=8192, k_lo=-1, k_hi=-1, pad=0, h_q=32,
             h_kv=8, d=128, causal=True, window=-1, layout="heads"),
        # the first prompt of a small model: one sequence, one partly filled page pair
        dict(name="chunk_first", op="chunk", seqs=1, singles=0, new_lo=17, new_hi=17, old_lo=0, old_hi=0, pad=0, h_q=8,
             h_kv=8, d=64, window=-1, sinks=0, cache="bf16", page=16),
        # a step of continuous batching: 40 sequences generate a token each, 6 prompts come in pieces
        dict(name="chunk_mixed", op="chunk", seqs=46, singles=40, new_lo=65, new_hi=512, old_lo=37, old_hi=4093, pad=31,
             h_q=32, h_kv=8, d=128, window=-1, sinks=0, cache="bf16", page=64),
        # a piece of one very long prompt, 8-bit cache: few rows, a long axis
        dict(name="chunk_long_e4m3", op="chunk", seqs=1, singles=0, new_lo=509, new_hi=509, old_lo=60001, old_hi=60001,
             pad=0, h_q=64, h_kv=8, d=128, window=-1, sinks=0, cache="e4m3", page=64),
        # prompts' pieces under a sliding window with visible first tokens
        dict(name="chunk_window", op="chunk", seqs=16, singles=2, new_lo=100, new_hi=1500, old_lo=0, old_hi=6007, pad=0,
             h_q=16, h_kv=4, d=64, window=1023, sinks=4, cache="bf16", page=16),
    ]


HEADS = [(8, 8), (16, 16), (12, 4), (32, 8), (5, 1), (16, 2), (6, 3), (64, 8), (7, 7), (14, 2)]
MOST = {"packed_fwd": 1.0e12, "packed_bwd": 1.2e12, "chunk": 1.0e12}  # operations, below the largest listed case's


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["packed_fwd", "packed_bwd", "chunk"])
    while True:
        h_q, h_kv = rng.choice(HEADS)
        c = dict(op=op, h_q=h_q, h_kv=h_kv, d=rng.choice([64, 128]), pad=rng.choice([0, 0, _log(rng, 1, 300)]))
        if op == "chunk":
            c["seqs"] = _log(rng, 1, 128)
            c["singles"] = rng.choice([0, 0, c["seqs"], rng.randint(0, c["seqs"])])
            c["new_hi"] = _log(rng, 1, 2048)
            c["new_lo"] = rng.randint(0 if c["seqs"] > 1 and c["new_hi"] < 64 else 1, c["new_hi"])
            c["old_hi"] = _log(rng, 1, 65536)
            c["old_lo"] = rng.randint(0, c["old_hi"])
            c["window"] = rng.choice([-1, -1, 0, _log(rng, 1, 4096)])
            c["sinks"] = 0 if c["window"] < 0 else rng.choice([0, 1, 4, 37])
            c["cache"] = rng.choice(["bf16", "bf16", "e4m3"])
            c["page"] = rng.choice([1, 8, 16, 20, 32, 64, 128, 256])
            cost = c["seqs"] * (c["old_hi"] + c["new_hi"]) * h_kv * c["d"]
            if sum(_new_tokens(c)) == 0 or cost > 2 ** 30:
                continue
        else:
            c["seqs"] = _log(rng, 1, 256)
            c["q_hi"] = _log(rng, 1, 8192)
            c["q_lo"] = rng.randint(0 if c["seqs"] > 1 else 1, c["q_hi"])
            c["k_lo"] = c["k_hi"] = -1  # as the queries'
            if rng.random() < 0.3:
                c["k_hi"] = _log(rng, 1, 8192)
                c["k_lo"] = rng.randint(0, c["k_hi"])
            c["causal"] = rng.random() < 0.6
            c["window"] = rng.choice([-1, -1, -1, 0, _log(rng, 1, 4096)])
            c["layout"] = rng.choice(["fused", "heads"]) if c["k_lo"] < 0 else "heads"
            if c["seqs"] * max(c["q_hi"], c["k_hi"]) * (h_q + h_kv) * c["d"] > 16384 * 40 * 128 * 2:
                continue
        if work(c)["flops"] <= MOST[op]:
            return c


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly: the sizes of a ragged batch."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _new_tokens(c):
    """New tokens of every sequence of a chunk call: one each for the generating ones."""
    return [1] * c["singles"] + (_spread(c["new_lo"], c["new_hi"], c["seqs"] - c["singles"])
                                 if c["seqs"] > c["singles"] else [])


def _order(count, seed):
    """The sequences' order in the batch; the sizes that belong together depend on it."""
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(count, generator=g).tolist()


def _lengths(c):
    """(queries, keys) of every sequence, the same for every seed (whose order then differs)."""
    if c["op"] == "chunk":
        new, old = _new_tokens(c), _spread(c["old_lo"], c["old_hi"], c["seqs"])
        old = [old[i] for i in _order(c["seqs"], 1)]
        return [(n, n + o) for n, o in zip(new, old)]
    q = _spread(c["q_lo"], c["q_hi"], c["seqs"])
    if c["k_lo"] < 0:
        return [(n, n) for n in q]
    k = _spread(c["k_lo"], c["k_hi"], c["seqs"])
    return list(zip(q, [k[i] for i in _order(c["seqs"], 2)]))


def _span(c, n_q, n_k, i):
    """Keys [lo, hi) that query i may use, and how many of the first tokens besides."""
    pos = n_k - n_q + i
    causal = c["op"] == "chunk" or c["causal"]
    lo, hi = 0, min(n_k, pos + 1) if causal else n_k
    if c["window"] >= 0:
        lo, hi = max(0, pos - c["window"]), min(hi, pos + c["window"] + 1)
    if hi <= lo:
        lo = hi = max(0, hi)
    more = min(c.get("sinks", 0), lo) if c["window"] >= 0 and pos >= 0 else 0
    return lo, hi, more


def _pairs(c, n_q, n_k):
    """(legal (query, key) pairs of one head, keys that some query may use)."""
    if n_q == 0 or n_k == 0:
        return 0, 0
    if c["window"] < 0:  # closed forms: these are counted often
        if c["op"] != "chunk" and not c["causal"]:
            return n_q * n_k, n_k
        m = min(n_q, n_k)  # queries before the first key see none
        return m * (n_k - m) + m * (m + 1) // 2, n_k
    pairs, low, high, first = 0, n_k, 0, 0
    for i in range(n_q):
        lo, hi, more = _span(c, n_q, n_k, i)
        pairs += hi - lo + more
        if hi > lo:
            low, high = min(low, lo), max(high, hi)
        first = max(first, more)
    return pairs, max(0, high - low) + min(first, low)


def work(c):
    """What a pass has to read and write, each once, and to compute."""
    d, h_q, h_kv = c["d"], c["h_q"], c["h_kv"]
    lens = _lengths(c)
    counted = [_pairs(c, a, b) for a, b in lens]
    pairs, keys, rows = sum(p for p, _ in counted), sum(k for _, k in counted), sum(a for a, _ in lens)
    if c["op"] == "chunk":
        per = 2 if c["cache"] == "bf16" else 1
        ids = sum(-(-k // c["page"]) for _, k in counted) + 2 * c["seqs"]
        return {"bytes": keys * h_kv * 2 * d * per + rows * h_q * (4 * d + 4) + 4 * ids, "flops": 4 * d * h_q * pairs}
    if c["op"] == "packed_fwd":
        return {"bytes": keys * h_kv * 4 * d + rows * h_q * (4 * d + 4), "flops": 4 * d * h_q * pairs}
    total = sum(b for _, b in lens)  # every key's gradient is written
    return {"bytes": (2 * keys + 2 * total) * h_kv * 2 * d + rows * h_q * (8 * d + 4), "flops": 10 * d * h_q * pairs}


# ---------------------------------------------------------------- inputs
def _normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _pages(g, lens, page):
    """A page table whose pages lie anywhere in the pool, and the number of pages of the pool."""
    need = torch.tensor([-(-x // page) for x in lens], device="cuda")
    total, width = int(need.sum()), max(1, int(need.max()))
    at = torch.arange(width, device="cuda")[None, :]
    order = torch.randperm(total + 3, generator=g, device="cuda")
    first = need.cumsum(0) - need
    table = order[(first[:, None] + at).clamp(max=total + 2)].masked_fill(at >= need[:, None], -1)
    return table.to(torch.int32), total + 3


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def _gives(layout, make, rows, h_q, h_kv, d):
    """q, k, v (or their gradients' places) as [rows, heads, d] in one of the two layouts."""
    if layout == "fused":
        x = make(rows, (h_q + 2 * h_kv) * d).view(rows, h_q + 2 * h_kv, d)
        return x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:]
    return tuple(make(h, rows, d).transpose(0, 1) for h in (h_q, h_kv, h_kv))


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d, h_q, h_kv = c["d"], c["h_q"], c["h_kv"]
    lens = _lengths(c)
    lens = [lens[i] for i in _order(c["seqs"], seed)]
    q_at, k_at = _starts(n for n, _ in lens), _starts(n for _, n in lens)
    s = {"case": c, "lens": lens, "q_at": q_at, "k_at": k_at}
    int32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    zeros = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    rows = q_at[-1] + c["pad"]  # rows behind the last sequence belong to none
    s["q_starts"] = int32(q_at)
    if c["op"] == "chunk":
        e4m3 = c["cache"] == "e4m3"
        s["page_table"], pages = _pages(g, [n for _, n in lens], c["page"])
        s["cache_lens"] = int32([n for _, n in lens])
        for x in ("k", "v"):
            s[x + "_scale"] = (0.01 + 0.004 * torch.rand(h_kv, generator=g, device="cuda")) if e4m3 else None
            y = torch.randn(pages, h_kv, c["page"], d, generator=g, device="cuda")
            s[x + "_pages"] = (y / 0.012).clamp(-448, 448).to(torch.float8_e4m3fn) if e4m3 else y.to(torch.bfloat16)
        s["q"] = _normal(g, rows, h_q, d, scale=1.5)
        s["out"], s["lse"] = zeros(rows, h_q, d), torch.zeros(rows, h_q, device="cuda")
        return s
    normal = lambda *shape: _normal(g, *shape, scale=1.2)  # noqa: E731
    if c["k_lo"] < 0:
        s["q"], s["k"], s["v"] = _gives(c["layout"], normal, rows, h_q, h_kv, d)
        s["k_starts"] = None
    else:
        s["q"] = _gives("heads", normal, rows, h_q, 0, d)[0]
        s["k"], s["v"] = _gives("heads", normal, max(1, k_at[-1]), 0, h_kv, d)[1:]
        s["k_starts"] = int32(k_at)
    s["out"], s["lse"] = zeros(rows, h_q, d), torch.zeros(rows, h_q, device="cuda")
    if c["op"] == "packed_bwd":
        _plain_packed_fwd(s)  # what the forward pass left behind
        s["dout"] = _normal(g, rows, h_q, d)
        if c["k_lo"] < 0:
            s["dq"], s["dk"], s["dv"] = _gives(c["layout"], zeros, rows, h_q, h_kv, d)
        else:
            s["dq"] = _gives("heads", zeros, rows, h_q, 0, d)[0]
            s["dk"], s["dv"] = _gives("heads", zeros, max(1, k_at[-1]), 0, h_kv, d)[1:]
    return s


# ---------------------------------------------------------------- plain forms
def _legal(c, n_q, n_k):
    """[n_q, n_k] truth values, or None where every pair is legal."""
    causal = c["op"] == "chunk" or c["causal"]
    if not causal and c["window"] < 0:
        return None
    pos = torch.arange(n_k - n_q, n_k, device="cuda")[:, None]
    key = torch.arange(n_k, device="cuda")
    legal = key <= pos if causal else torch.ones(n_q, n_k, dtype=torch.bool, device="cuda")
    if c["window"] >= 0:
        near = (key >= pos - c["window"]) & (key <= pos + c["window"])
        legal = legal & (near | (key < c.get("sinks", 0)))
    return legal


def _head_groups(h_kv, group, n_q, n_k):
    """Ranges of key/value heads whose score matrices take a gigabyte or so together."""
    step = max(1, min(h_kv, 2 ** 28 // max(1, group * n_q * n_k)))
    return [(z, min(h_kv, z + step)) for z in range(0, h_kv, step)]


def _by_kv_head(x, z0, z1, group):
    """Rows [n, h_q, d] -> float32 [z1 - z0, group * n, d], the query heads of key heads z0 to z1 - 1."""
    n, d = x.shape[0], x.shape[2]
    return x[:, z0 * group:z1 * group].float().view(n, z1 - z0, group, d).permute(1, 2, 0, 3).reshape(z1 - z0, -1, d)


def _by_token(x, n, group):
    """The way back: [heads, group * n, d] -> [n, heads * group, d]."""
    return x.view(x.shape[0], group, n, -1).permute(2, 0, 1, 3).reshape(n, x.shape[0] * group, -1)


def _attend(c, q, k, v, out, lse, n_q, n_k, group, z0, z1):
    """One sequence, key heads z0 to z1 - 1: k, v float32 [heads, n_k, d]."""
    score = torch.matmul(_by_kv_head(q, z0, z1, group), k.transpose(1, 2)).mul_(1 / math.sqrt(c["d"]))
    legal = _legal(c, n_q, n_k)
    if legal is not None:
        score.view(z1 - z0, group, n_q, n_k).masked_fill_(~legal, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top.isinf(), 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    out[:, z0 * group:z1 * group] = _by_token(o, n_q, group).to(out.dtype)
    lse[:, z0 * group:z1 * group] = _by_token(top + total.log(), n_q, group)[..., 0]


def _sequences(s):
    for (n_q, n_k), q0, k0 in zip(s["lens"], s["q_at"], s["k_at"]):
        yield n_q, n_k, slice(q0, q0 + n_q), slice(k0, k0 + n_k)


def _plain_packed_fwd(s):
    c = s["case"]
    group = c["h_q"] // c["h_kv"]
    for n_q, n_k, rows, keys in _sequences(s):
        if n_q == 0:
            continue
        if n_k == 0:
            s["out"][rows], s["lse"][rows] = 0, -math.inf
            continue
        for z0, z1 in _head_groups(c["h_kv"], group, n_q, n_k):
            k, v = (s[x][keys, z0:z1].float().transpose(0, 1) for x in ("k", "v"))
            _attend(c, s["q"][rows], k, v, s["out"][rows], s["lse"][rows], n_q, n_k, group, z0, z1)
    return {"out": s["out"], "lse": s["lse"]}


def _plain_packed_bwd(s):
    c = s["case"]
    group, scale = c["h_q"] // c["h_kv"], 1 / math.sqrt(c["d"])
    for n_q, n_k, rows, keys in _sequences(s):
        if n_q == 0 or n_k == 0:
            s["dq"][rows], s["dk"][keys], s["dv"][keys] = 0, 0, 0
            continue
        legal = _legal(c, n_q, n_k)
        for z0, z1 in _head_groups(c["h_kv"], group, n_q, n_k):
            q, o, do = (_by_kv_head(s[x][rows], z0, z1, group) for x in ("q", "out", "dout"))
            lse = _by_kv_head(s["lse"][rows][..., None], z0, z1, group)
            k, v = (s[x][keys, z0:z1].float().transpose(0, 1) for x in ("k", "v"))
            p = torch.matmul(q, k.transpose(1, 2)).mul_(scale).sub_(torch.where(lse.isinf(), 0.0, lse)).exp_()
            if legal is not None:
                p.view(z1 - z0, group, n_q, n_k).masked_fill_(~legal, 0.0)
            s["dv"][keys, z0:z1] = torch.matmul(p.transpose(1, 2), do).transpose(0, 1).to(torch.bfloat16)
            ds = torch.matmul(do, v.transpose(1, 2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
            s["dk"][keys, z0:z1] = torch.matmul(ds.transpose(1, 2), q).transpose(0, 1).to(torch.bfloat16)
            s["dq"][rows, z0 * group:z1 * group] = _by_token(torch.matmul(ds, k), n_q, group).to(torch.bfloat16)
    return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}


def _cached(pages, scale, table, n, z0, z1):
    """The first n cached rows of one sequence, key heads z0 to z1 - 1, float32 [heads, n, d]."""
    table = table[:-(-n // pages.shape[2])].long()
    if scale is None:
        x = pages[table, z0:z1].float()
    else:
        x = pages.view(torch.int8)[table, z0:z1].view(pages.dtype).float() * scale[z0:z1, None, None]
    return x.transpose(0, 1).reshape(z1 - z0, -1, pages.shape[3])[:, :n]


def _plain_chunk(s):
    c = s["case"]
    group = c["h_q"] // c["h_kv"]
    for b, (n_q, n_k, rows, _) in enumerate(_sequences(s)):
        for z0, z1 in _head_groups(c["h_kv"], group, n_q, n_k) if n_q else ():
            k, v = (_cached(s[x + "_pages"], s[x + "_scale"], s["page_table"][b], n_k, z0, z1) for x in ("k", "v"))
            _attend(c, s["q"][rows], k, v, s["out"][rows], s["lse"][rows], n_q, n_k, group, z0, z1)
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"packed_fwd": _plain_packed_fwd, "packed_bwd": _plain_packed_bwd, "chunk": _plain_chunk}[op](s)
    from transformer_scaled_dot_mha_gb300 import attn

    rows = s["q"].shape[0]
    if "workspace" not in s:
        if op == "packed_bwd":
            size = attn.attn_packed_bwd_workspace_size(rows, s["k"].shape[0], c["seqs"], c["h_q"], c["h_kv"], c["d"])
        elif op == "packed_fwd":
            size = attn.attn_packed_fwd_workspace_size(rows, c["seqs"], c["h_q"], c["h_kv"], c["d"])
        else:
            size = attn.attn_paged_chunk_workspace_size(rows, c["seqs"], c["h_q"], c["h_kv"], c["d"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    if op == "chunk":
        attn.attn_paged_chunk(s["q"], s["k_pages"], s["v_pages"], s["out"], s["q_starts"], s["page_table"],
                              s["cache_lens"], s["workspace"], lse=s["lse"], window=c["window"], sinks=c["sinks"],
                              k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"out": s["out"], "lse": s["lse"]}
    mask = attn.MASK_CAUSAL if c["causal"] else attn.MASK_NONE
    if op == "packed_fwd":
        attn.attn_packed_fwd(s["q"], s["k"], s["v"], s["out"], s["q_starts"], s["workspace"], k_starts=s["k_starts"],
                             lse=s["lse"], mask_mode=mask, window=c["window"])
        return {"out": s["out"], "lse": s["lse"]}
    attn.attn_packed_bwd(s["q"], s["k"], s["v"], s["out"], s["dout"], s["lse"], s["dq"], s["dk"], s["dv"],
                         s["q_starts"], s["workspace"], k_starts=s["k_starts"], mask_mode=mask, window=c["window"])
    return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}


# ---------------------------------------------------------------- 64-bit values
def exact(c, seed):
    """One query head after the other, from the definition, in float64."""
    if work(c)["flops"] > 1.5e12 * (1 if c["op"] == "packed_bwd" else 2):
        return None
    s = prepare(c, seed)
    d, group = c["d"], c["h_q"] // c["h_kv"]
    rows = s["q"].shape[0]
    f64 = dict(dtype=torch.float64, device="cuda")
    grads = c["op"] == "packed_bwd"
    if grads:
        got = {"d" + x: torch.zeros(s[x].shape, **f64) for x in ("q", "k", "v")}
    else:
        got = {"out": torch.zeros(rows, c["h_q"], d, **f64), "lse": torch.zeros(rows, c["h_q"], **f64)}
    for b, (n_q, n_k) in enumerate(s["lens"]):
        q0, k0 = s["q_at"][b], s["k_at"][b]
        if n_q == 0:
            continue
        if n_k == 0:
            if not grads:
                got["lse"][q0:q0 + n_q] = -math.inf
            continue
        # the first and the last + 1 key of every query, its own position's window, the first tokens
        at = n_k - n_q + torch.arange(n_q, device="cuda")
        past = c["op"] == "chunk" or c["causal"]
        hi = (at + 1).clamp(0, n_k) if past else torch.full_like(at, n_k)
        lo = torch.zeros_like(at)
        if c["window"] >= 0:
            lo = (at - c["window"]).clamp(min=0)
            hi = torch.minimum(hi, (at + c["window"] + 1).clamp(min=0))
        j = torch.arange(n_k, device="cuda")[None]
        seen = (j >= lo[:, None]) & (j < hi[:, None])
        if c["window"] >= 0 and c.get("sinks", 0) > 0:
            seen |= (j < c["sinks"]) & (j < hi[:, None])
        for z in range(c["h_kv"]):
            if c["op"] == "chunk":
                kv = []
                for x in ("k", "v"):
                    ids = s["page_table"][b, :-(-n_k // c["page"])].long()
                    y = s[x + "_pages"]
                    if c["cache"] == "e4m3":
                        y = y.view(torch.int8)[ids, z].view(y.dtype).double() * s[x + "_scale"][z].double()
                    else:
                        y = y[ids, z].double()
                    kv.append(y.reshape(-1, d)[:n_k])
                k, v = kv
            else:
                k, v = s["k"][k0:k0 + n_k, z].double(), s["v"][k0:k0 + n_k, z].double()
            for h in range(z * group, (z + 1) * group):
                x = s["q"][q0:q0 + n_q, h].double()
                a = (x @ k.T / math.sqrt(d)).masked_fill(~seen, -math.inf)
                if not grads:
                    lse = a.logsumexp(-1)
                    a = (a - torch.where(lse == -math.inf, 0.0, lse)[:, None]).exp()
                    got["lse"][q0:q0 + n_q, h] = lse
                    got["out"][q0:q0 + n_q, h] = a @ v
                    continue
                lse = s["lse"][q0:q0 + n_q, h].double()
                a = (a - torch.where(lse == -math.inf, 0.0, lse)[:, None]).exp()
                g = s["dout"][q0:q0 + n_q, h].double()
                t = a * (g @ v.T - torch.einsum("nd,nd->n", g, s["out"][q0:q0 + n_q, h].double())[:, None])
                got["dv"][k0:k0 + n_k, z] += a.T @ g
                got["dk"][k0:k0 + n_k, z] += t.T @ x / math.sqrt(d)
                got["dq"][q0:q0 + n_q, h] = t @ k / math.sqrt(d)
    return got
