"""The position and paged-cache operators as a benchmark sees them: cases, inputs, plain forms, 64-bit values.

Four operators of the attention library are described here, each by the call a user makes of it
(``own`` true) and by the same arithmetic in elementary torch operations (``own`` false):

  norm_rope      RMS norm of every query and key head and the position rotation, forward
  norm_rope_bwd  its gradients with respect to the heads and the two norm weights
  append         norm and rotation of new tokens, keys and values written into a paged cache
  decode         attention of the newest tokens over that cache (shared key/value heads,
                 sliding window with visible first tokens, bf16 or e4m3 pages)

Layouts: a fused projection holds each token's query heads, key heads and value heads side by
side, so q, k and v are strided views of it; attention reads [B, h, n, d]; a cache is
[pages, h_kv, page_size, d], and a page table [sequences, max_pages] names each sequence's pages
(-1 where it has none). The rotation table is float32 [positions, d_rot]: the cosines of the
d_rot / 2 angles, then their sines.
"""
import math

import torch

own = False

EPS = 1e-6
ROPE_BASE = 10000.0


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a short training or encoder batch: launch latency is what counts
        dict(name="norm_rope_short", op="norm_rope", B=4, n=33, h_q=8, h_kv=8, d=64, d_rot=64, style="half", norm=True),
        # a long training sequence, shared key heads: streams a third of a gigabyte
        dict(name="norm_rope_long", op="norm_rope", B=2, n=8192, h_q=32, h_kv=8, d=128, d_rot=128, style="half",
             norm=True),
        # gradients at the decoder's training length, adjacent pairs
        dict(name="norm_rope_bwd_mid", op="norm_rope_bwd", B=16, n=512, h_q=8, h_kv=8, d=64, d_rot=64, style="pairs",
             norm=True),
        # gradients of the long sequence
        dict(name="norm_rope_bwd_long", op="norm_rope_bwd", B=2, n=8192, h_q=32, h_kv=8, d=128, d_rot=128,
             style="half", norm=True),
        # one generation step of 32 sequences: a token each
        dict(name="append_step", op="append", seqs=32, tok_lo=1, tok_hi=1, pos_lo=100, pos_hi=2047, h_q=8, h_kv=8,
             d=64, d_rot=64, style="half", norm=True, cache="bf16", page=16),
        # prompts of very different lengths in one packed batch
        dict(name="append_prompts", op="append", seqs=24, tok_lo=37, tok_hi=1331, pos_lo=0, pos_hi=0, h_q=32, h_kv=8,
             d=128, d_rot=128, style="half", norm=True, cache="bf16", page=64),
        # continued prompts into an 8-bit cache, rotation of half the columns, no norm
        dict(name="append_prompts_e4m3", op="append", seqs=7, tok_lo=129, tok_hi=901, pos_lo=5, pos_hi=700, h_q=16,
             h_kv=2, d=128, d_rot=64, style="pairs", norm=False, cache="e4m3", page=32),
        # the first tokens of one sequence: the smallest call
        dict(name="decode_first", op="decode", B=1, n_q=1, h_q=8, h_kv=8, d=64, len_lo=17, len_hi=17, window=-1,
             sinks=0, cache="bf16", page=16),
        # a generation step of the base model's heads, 32 sequences
        dict(name="decode_heads", op="decode", B=32, n_q=1, h_q=8, h_kv=8, d=64, len_lo=1024, len_hi=2048, window=-1,
             sinks=0, cache="bf16", page=16),
        # shared heads over long caches
        dict(name="decode_shared", op="decode", B=16, n_q=1, h_q=32, h_kv=8, d=128, len_lo=4096, len_hi=8192,
             window=-1, sinks=0, cache="bf16", page=64),
        # few sequences, very long 8-bit caches of unequal length
        dict(name="decode_long_e4m3", op="decode", B=8, n_q=1, h_q=64, h_kv=8, d=128, len_lo=9001, len_hi=65521,
             window=-1, sinks=0, cache="e4m3", page=64),
        # four new tokens at once (a verified draft), sliding window with four visible first tokens
        dict(name="decode_window", op="decode", B=64, n_q=4, h_q=16, h_kv=4, d=64, len_lo=3, len_hi=8191, window=1023,
             sinks=4, cache="bf16", page=16),
    ]


HEADS = [(8, 8), (16, 16), (12, 4), (32, 8), (5, 1), (16, 2), (6, 3), (64, 8), (7, 7)]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "decode"])
    h_q, h_kv = rng.choice(HEADS)
    d = rng.choice([64, 128])
    if op != "decode":
        c = dict(op=op, h_q=h_q, h_kv=h_kv, d=d, d_rot=rng.choice([d, d, d // 2, 16, 48]),
                 style=rng.choice(["half", "pairs"]), norm=rng.random() < 0.75)
    if op in ("norm_rope", "norm_rope_bwd"):
        most = 16384 * 40 * 128 // ((h_q + h_kv) * d)
        tokens = _log(rng, 1, most)
        c["B"] = _log(rng, 1, min(64, tokens))
        c["n"] = max(1, min(8192, tokens // c["B"]))
        return c
    page = rng.choice([1, 8, 16, 20, 32, 64, 128, 256])
    cache = rng.choice(["bf16", "bf16", "e4m3"])
    if op == "append":
        most = 16384 * 48 * 128 // ((h_q + 2 * h_kv) * d)
        seqs = _log(rng, 1, 256)
        hi = _log(rng, 1, max(1, min(4096, most // seqs)))
        pos_hi = _log(rng, 1, 4096)
        c.update(seqs=seqs, tok_lo=rng.randint(1, hi), tok_hi=hi, pos_lo=rng.randint(0, pos_hi), pos_hi=pos_hi,
                 cache=cache, page=page)
        return c
    n_q = rng.choice([1, 1, 1, 2, 5, 16])
    most = min(8 * 37000 * 8 * 128 // (h_kv * d) // (2 if cache == "bf16" else 1),
               8 * 37000 * 64 * 128 // (h_q * n_q * d))
    B = _log(rng, 1, 128)
    hi = _log(rng, 1, max(1, min(65536, most // B)))
    window = rng.choice([-1, -1, 0, _log(rng, 1, 4096)])
    return dict(op="decode", B=B, n_q=n_q, h_q=h_q, h_kv=h_kv, d=d, len_lo=rng.randint(max(0, hi // 4), hi), len_hi=hi,
                window=window, sinks=0 if window < 0 else rng.choice([0, 1, 4, 37]), cache=cache, page=page)


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly: the sizes of a ragged batch."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _visible(c):
    """Per sequence: (keys that some query may use, legal (query, key) pairs of one head)."""
    got = []
    for length in _spread(c["len_lo"], c["len_hi"], c["B"]):
        pairs, low = 0, length
        for i in range(c["n_q"]):
            pos = length - c["n_q"] + i
            if pos < 0:
                continue
            first = 0 if c["window"] < 0 else max(0, pos - c["window"])
            pairs += pos + 1 - first + min(c["sinks"], first)
            low = min(low, first)
        got.append((length - low + min(c["sinks"], low) if pairs else 0, pairs))
    return got


def work(c):
    """What a pass has to read and write, each once, and to compute."""
    d, h_q, h_kv = c["d"], c["h_q"], c["h_kv"]
    if c["op"] == "decode":
        per = 2 if c["cache"] == "bf16" else 1
        seen = _visible(c)
        rows = c["B"] * c["n_q"] * h_q
        keys = sum(k for k, _ in seen)
        ids = sum(-(-k // c["page"]) for k, _ in seen) + c["B"]
        return {"bytes": keys * h_kv * 2 * d * per + rows * (4 * d + 4) + 4 * ids,
                "flops": 4 * d * h_q * sum(p for _, p in seen)}
    if c["op"] == "append":
        tokens = sum(_spread(c["tok_lo"], c["tok_hi"], c["seqs"]))
        starts = _spread(c["pos_lo"], c["pos_hi"], c["seqs"])
        table = min(tokens, max(starts) + c["tok_hi"]) * c["d_rot"] * 4
        per = 2 if c["cache"] == "bf16" else 1
        return {"bytes": tokens * d * (h_q * 4 + h_kv * 2 * (2 + per)) + table + 8 * tokens,
                "flops": tokens * d * (h_q + h_kv) * 8}
    tokens = c["B"] * c["n"]
    passes = 2 if c["op"] == "norm_rope" else 3
    return {"bytes": tokens * (h_q + h_kv) * d * 2 * passes + c["n"] * c["d_rot"] * 4,
            "flops": tokens * (h_q + h_kv) * d * (8 if passes == 2 else 16)}


# ---------------------------------------------------------------- inputs
def _normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def rotation_table(n_pos, d_rot):
    """float32 [n_pos, d_rot]; the angles in double, as far positions need."""
    i = torch.arange(d_rot // 2, dtype=torch.float64, device="cuda")
    angle = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * ROPE_BASE ** (-2.0 * i / d_rot)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _weights(g, s, c):
    """Norm weights near one, as trained ones are; none where the case has no norm."""
    near_one = lambda: (1 + 0.1 * torch.randn(c["d"], generator=g, device="cuda")).to(torch.bfloat16)  # noqa: E731
    s["q_weight"], s["k_weight"] = (near_one(), near_one()) if c["norm"] else (None, None)


def _pages(g, lens, page):
    """A page table whose pages lie anywhere in the pool, and the number of pages of the pool."""
    need = torch.tensor([-(-x // page) for x in lens], device="cuda")
    total, width = int(need.sum()), max(1, int(need.max()))
    at = torch.arange(width, device="cuda")[None, :]
    order = torch.randperm(total + 3, generator=g, device="cuda")
    first = need.cumsum(0) - need
    table = order[(first[:, None] + at).clamp(max=total + 2)].masked_fill(at >= need[:, None], -1)
    return table.to(torch.int32), total + 3


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d, h_q, h_kv = c["d"], c["h_q"], c["h_kv"]
    s = {"case": c}
    if c["op"] in ("norm_rope", "norm_rope_bwd"):
        B, n = c["B"], c["n"]
        qkv = _normal(g, B, n, (h_q + 2 * h_kv) * d, scale=1.7).view(B, n, h_q + 2 * h_kv, d)
        s["q"], s["k"] = qkv[:, :, :h_q], qkv[:, :, h_q:h_q + h_kv]
        s["cos_sin"] = rotation_table(n, c["d_rot"])
        _weights(g, s, c)
        if c["op"] == "norm_rope":
            s["q_out"] = torch.zeros(B, h_q, n, d, dtype=torch.bfloat16, device="cuda")
            s["k_out"] = torch.zeros(B, h_kv, n, d, dtype=torch.bfloat16, device="cuda")
        else:
            s["dq_out"], s["dk_out"] = _normal(g, B, h_q, n, d), _normal(g, B, h_kv, n, d)
            dqkv = torch.zeros_like(qkv)
            s["dq"], s["dk"] = dqkv[:, :, :h_q], dqkv[:, :, h_q:h_q + h_kv]
            s["dq_weight"] = torch.zeros(d, device="cuda") if c["norm"] else None
            s["dk_weight"] = torch.zeros(d, device="cuda") if c["norm"] else None
        return s
    count = c["seqs"] if c["op"] == "append" else c["B"]
    order = torch.randperm(count, generator=g, device="cuda").tolist()
    shuffled = lambda v: [v[i] for i in order]  # noqa: E731
    e4m3 = c["cache"] == "e4m3"
    s["k_scale"] = (0.01 + 0.004 * torch.rand(h_kv, generator=g, device="cuda")) if e4m3 else None
    s["v_scale"] = (0.01 + 0.004 * torch.rand(h_kv, generator=g, device="cuda")) if e4m3 else None

    def cache(pages):
        x = torch.randn(pages, h_kv, c["page"], d, generator=g, device="cuda")
        return (x / 0.012).clamp(-448, 448).to(torch.float8_e4m3fn) if e4m3 else x.to(torch.bfloat16)

    if c["op"] == "append":
        toks = shuffled(_spread(c["tok_lo"], c["tok_hi"], count))
        starts = shuffled(_spread(c["pos_lo"], c["pos_hi"], count))
        s["page_table"], pages = _pages(g, [a + b for a, b in zip(toks, starts)], c["page"])
        counts = torch.tensor(toks, device="cuda")
        seq = torch.repeat_interleave(torch.arange(count, device="cuda"), counts)
        within = torch.arange(len(seq), device="cuda") - (counts.cumsum(0) - counts)[seq]
        s["positions"] = (torch.tensor(starts, device="cuda")[seq] + within).to(torch.int32)
        s["seq_ids"] = seq.to(torch.int32)
        qkv = _normal(g, len(seq), (h_q + 2 * h_kv) * d, scale=1.7).view(len(seq), h_q + 2 * h_kv, d)
        s["q"], s["k"], s["v"] = qkv[:, :h_q], qkv[:, h_q:h_q + h_kv], qkv[:, h_q + h_kv:]
        s["cos_sin"] = rotation_table(int(s["positions"].max()) + 1, c["d_rot"])
        _weights(g, s, c)
        s["q_out"] = torch.zeros(len(seq), h_q, d, dtype=torch.bfloat16, device="cuda")
        s["k_pages"], s["v_pages"] = cache(pages), cache(pages)
        return s
    lens = shuffled(_spread(c["len_lo"], c["len_hi"], count))
    s["page_table"], pages = _pages(g, lens, c["page"])
    s["cache_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["k_pages"], s["v_pages"] = cache(pages), cache(pages)
    s["q"] = _normal(g, count, c["n_q"], h_q, d, scale=1.5)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(count, c["n_q"], h_q, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms
def _rotate(y, cos, sin, style, back=False):
    """Turns the pairs of the last axis' first 2 * cos.shape[-1] columns by the angles; back: by their negatives."""
    m = cos.shape[-1]
    if back:
        sin = -sin
    if style == "half":
        a, b = y[..., :m], y[..., m:2 * m]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., 2 * m:]], -1)
    a, b = y[..., 0:2 * m:2], y[..., 1:2 * m:2]
    turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, y[..., 2 * m:]], -1)


def _normed(x, weight):
    if weight is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()


def _plain_norm_rope(s):
    c, m = s["case"], s["cos_sin"].shape[1] // 2
    cos, sin = s["cos_sin"][:, None, :m], s["cos_sin"][:, None, m:]  # [n, 1, m]: the same for every head
    for x, weight, out in ((s["q"], s["q_weight"], s["q_out"]), (s["k"], s["k_weight"], s["k_out"])):
        out.copy_(_rotate(_normed(x.float(), weight), cos, sin, c["style"]).transpose(1, 2))
    return {"q": s["q_out"], "k": s["k_out"]}


def _plain_norm_rope_bwd(s):
    c, m = s["case"], s["cos_sin"].shape[1] // 2
    cos, sin = s["cos_sin"][:, None, :m], s["cos_sin"][:, None, m:]
    for x, weight, g, dx, dw in ((s["q"], s["q_weight"], s["dq_out"], s["dq"], s["dq_weight"]),
                                 (s["k"], s["k_weight"], s["dk_out"], s["dk"], s["dk_weight"])):
        gy = _rotate(g.float().transpose(1, 2), cos, sin, c["style"], back=True)
        if weight is None:
            dx.copy_(gy)
            continue
        xf = x.float()
        r = torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS)
        u = gy * weight.float()
        dx.copy_(r * (u - xf * (r * r * (u * xf).mean(-1, keepdim=True))))
        dw.copy_((gy * xf * r).sum((0, 1, 2), dtype=torch.float64))  # a long sum
    got = {"dq": s["dq"], "dk": s["dk"]}
    return {**got, "dq_weight": s["dq_weight"], "dk_weight": s["dk_weight"]} if c["norm"] else got


def _stored(x, pages, scale):
    """Float32 [tokens, h_kv, d] in the cache's type; 8-bit values saturate."""
    if scale is None:
        return x.to(pages.dtype)
    return (x / scale[:, None]).clamp(-448, 448).to(pages.dtype)


def _plain_append(s):
    c, m = s["case"], s["cos_sin"].shape[1] // 2
    rows = s["cos_sin"][s["positions"]][:, None, :]
    cos, sin = rows[..., :m], rows[..., m:]
    s["q_out"].copy_(_rotate(_normed(s["q"].float(), s["q_weight"]), cos, sin, c["style"]))
    k = _rotate(_normed(s["k"].float(), s["k_weight"]), cos, sin, c["style"])
    page = s["page_table"][s["seq_ids"], s["positions"] // c["page"]].long()
    at = (s["positions"] % c["page"]).long()
    for x, pages, scale in ((k, s["k_pages"], s["k_scale"]), (s["v"].float(), s["v_pages"], s["v_scale"])):
        pages.view(torch.int8 if scale is not None else pages.dtype)[page, :, at] = \
            _stored(x, pages, scale).view(torch.int8 if scale is not None else pages.dtype)
    return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_decode(s):
    c = s["case"]
    B, n_q, h_q, d = s["q"].shape
    h_kv, table = c["h_kv"], s["page_table"].clamp(min=0).long()
    K = table.shape[1] * c["page"]

    def gathered(pages, scale):  # [B, h_kv, K, d]
        if scale is not None:
            x = pages.view(torch.int8)[table].view(pages.dtype).float() * scale[:, None, None]
        else:
            x = pages[table].float()
        return x.permute(0, 2, 1, 3, 4).reshape(B, h_kv, K, d)

    q = s["q"].float().view(B, n_q, h_kv, h_q // h_kv, d).permute(0, 2, 1, 3, 4).reshape(B, h_kv, -1, d)
    score = torch.matmul(q, gathered(s["k_pages"], s["k_scale"]).transpose(2, 3)).mul_(1 / math.sqrt(d))
    pos = (s["cache_lens"][:, None] - n_q + torch.arange(n_q, device="cuda"))[:, :, None]
    key = torch.arange(K, device="cuda")
    legal = key <= pos
    if c["window"] >= 0:
        legal &= (key >= pos - c["window"]) | (key < c["sinks"])
    legal = legal[:, None, :, None].expand(B, 1, n_q, h_q // h_kv, K).reshape(B, 1, -1, K)
    score.masked_fill_(~legal, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top.isinf(), 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, gathered(s["v_pages"], s["v_scale"])) / torch.where(total > 0, total, 1.0)
    lse = (top + total.log())[..., 0]
    by_token = lambda x: x.view(B, h_kv, n_q, -1, *x.shape[3:]).transpose(1, 2)  # noqa: E731
    s["out"].copy_(by_token(o).reshape(B, n_q, h_q, d))
    s["lse"].copy_(by_token(lse).reshape(B, n_q, h_q))
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"norm_rope": _plain_norm_rope, "norm_rope_bwd": _plain_norm_rope_bwd, "append": _plain_append,
                "decode": _plain_decode}[op](s)
    from transformer_scaled_dot_mha_gb300 import attn

    c = s["case"]
    if op == "norm_rope":
        attn.attn_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["cos_sin"], s["q_weight"], s["k_weight"],
                            eps=EPS, interleaved=c["style"] == "pairs")
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "norm_rope_bwd":
        if "workspace" not in s:
            size = attn.attn_norm_rope_bwd_workspace_size(c["B"], c["n"], c["h_q"], c["h_kv"], c["d"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        attn.attn_norm_rope_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], s["dq"], s["dk"], s["workspace"],
                                s["cos_sin"], s["q_weight"], s["k_weight"], s["dq_weight"], s["dk_weight"], eps=EPS,
                                interleaved=c["style"] == "pairs")
        got = {"dq": s["dq"], "dk": s["dk"]}
        return {**got, "dq_weight": s["dq_weight"], "dk_weight": s["dk_weight"]} if c["norm"] else got
    if op == "append":
        attn.attn_paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["positions"], s["page_table"],
                               seq_ids=s["seq_ids"], q=s["q"], q_out=s["q_out"], cos_sin=s["cos_sin"],
                               q_weight=s["q_weight"], k_weight=s["k_weight"], k_scale=s["k_scale"],
                               v_scale=s["v_scale"], eps=EPS, interleaved=c["style"] == "pairs")
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if "workspace" not in s:
        size = attn.attn_paged_decode_workspace_size(c["B"], c["n_q"], c["h_q"], c["h_kv"], c["d"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    attn.attn_paged_decode(s["q"], s["k_pages"], s["v_pages"], s["out"], s["page_table"], s["cache_lens"],
                           s["workspace"], lse=s["lse"], window=c["window"], sinks=c["sinks"], k_scale=s["k_scale"],
                           v_scale=s["v_scale"])
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- 64-bit values
def _turn(c, z, table, sign):
    """z float64 [rows, h, d], table [rows, d_rot]: column pairs (i, j) as complex numbers times exp(sign * angle)."""
    m = c["d_rot"] // 2
    e = torch.complex(table[:, :m].double(), sign * table[:, m:].double())[:, None]
    i = torch.arange(m, device=z.device)
    first, second = (2 * i, 2 * i + 1) if c["style"] == "pairs" else (i, i + m)
    w = torch.complex(z[..., first], z[..., second]) * e
    z = z.clone()
    z[..., first], z[..., second] = w.real, w.imag
    return z


def _exact_rows(c, x, weight, table):
    x = x.double()
    if weight is not None:
        x = x / ((x ** 2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * weight.double()
    return _turn(c, x, table, 1)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm_rope":
        return {n: torch.stack([_exact_rows(c, s[n][b], s[n + "_weight"], s["cos_sin"]).transpose(0, 1)
                                for b in range(c["B"])]) for n in ("q", "k")}
    if c["op"] == "norm_rope_bwd":
        got = {}
        for n in ("q", "k"):
            dx, dw = [], 0
            for b in range(c["B"]):
                x, g = s[n][b].double(), s[f"d{n}_out"][b].double().transpose(0, 1)
                g = _turn(c, g, s["cos_sin"], -1)
                if c["norm"]:
                    w = s[n + "_weight"].double()
                    root = ((x ** 2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt()
                    unit = x / root
                    dw = dw + (g * unit).sum((0, 1))
                    g = (g * w - unit * ((g * w) * unit).sum(-1, keepdim=True) / c["d"]) / root
                dx.append(g)
            got["d" + n] = torch.stack(dx)
            if c["norm"]:
                got[f"d{n}_weight"] = dw
        return got
    if c["op"] == "append":
        table = s["cos_sin"][s["positions"].long()]
        k = _exact_rows(c, s["k"], s["k_weight"], table)
        got = {"q": _exact_rows(c, s["q"], s["q_weight"], table)}
        page = s["page_table"].long()[s["seq_ids"].long(), s["positions"].long() // c["page"]]
        for name, x, scale in (("k_pages", k, s["k_scale"]), ("v_pages", s["v"].double(), s["v_scale"])):
            full = s[name].double()
            x = x if scale is None else (x / scale.double()[:, None]).clamp(-448, 448)
            full[page, :, s["positions"].long() % c["page"]] = x
            got[name] = full
        return got
    B, n_q, h_q, d = s["q"].shape
    group = h_q // c["h_kv"]
    out, lse = torch.zeros(B, n_q, h_q, d, dtype=torch.float64, device="cuda"), torch.full(
        (B, n_q, h_q), -math.inf, dtype=torch.float64, device="cuda")
    for b, length in enumerate(s["cache_lens"].tolist()):
        if length == 0:
            continue
        pages = s["page_table"][b, :-(-length // c["page"])].long()
        kv = []
        for x, scale in ((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"])):
            y = x.view(torch.int8)[pages].view(x.dtype).double() if scale is not None else x[pages].double()
            y = y.transpose(0, 1).reshape(c["h_kv"], -1, d)[:, :length]
            kv.append(y if scale is None else y * scale.double()[:, None, None])
        for i in range(n_q):
            pos = length - n_q + i
            if pos < 0:
                continue
            keys = torch.arange(pos + 1, device="cuda")
            if c["window"] >= 0:
                keys = keys[(keys >= pos - c["window"]) | (keys < c["sinks"])]
            k, v = kv[0][:, keys], kv[1][:, keys]
            z = torch.einsum("hgd,hkd->hgk", s["q"][b, i].double().view(c["h_kv"], group, d), k) / math.sqrt(d)
            lse[b, i] = z.logsumexp(-1).reshape(h_q)
            out[b, i] = torch.einsum("hgk,hkd->hgd", z.softmax(-1), v).reshape(h_q, d)
    return {"out": out, "lse": lse}
