"""Plain float64 forms of the norm + rotation, the paged append and the paged decode step
(torch on the CPU, loops over tokens and heads), with the sizes of the terms that the
tests' tolerances are made of."""
import math

import torch

U_BF16 = 2.0 ** -8   # largest relative error of one rounding to bf16
U_F16 = 2.0 ** -11
# fp32 part of one normalised, rotated value, relative to the sum of its terms' sizes: the
# sum of squares (at most 16 + 3 additions in a row, halved by the root: 10 u), the inverse
# root (2 units in the last place: 4 u), two products, two products and an addition: 19
# roundings of u = 2^-24, below 2^-19
U_ROPE = 2.0 ** -19


def rotation_table(n_pos, d_rot, base=10000.0):
    i = torch.arange(d_rot // 2, dtype=torch.float64)
    angle = torch.arange(n_pos, dtype=torch.float64)[:, None] * base ** (-2.0 * i / max(d_rot, 1))
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def pair_columns(d_rot, interleaved):
    i = torch.arange(d_rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + d_rot // 2)


def turn(y, row, interleaved, back=False):
    """y [..., d] float64, row [d_rot]: (turned y, sizes of its terms)."""
    m = row.shape[0] // 2
    a, b = pair_columns(2 * m, interleaved)
    c, s = row[:m].double(), row[m:].double() * (-1 if back else 1)
    o, size = y.clone(), y.abs()
    o[..., a], o[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    size[..., a] = (y[..., a] * c).abs() + (y[..., b] * s).abs()
    size[..., b] = (y[..., b] * c).abs() + (y[..., a] * s).abs()
    return o, size


def norm_rope(x, weight, row, eps, interleaved):
    """One token's heads x [h, d] -> (outputs, sizes of their terms), float64."""
    y = x.double()
    if weight is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    return turn(y, row, interleaved) if row is not None else (y, y.abs())


def norm_rope_bwd(x, g, weight, row, eps, interleaved):
    """One token's heads x, g [h, d] -> (dx, sizes, dw, sizes of dw's terms), float64."""
    gy, gsize = turn(g.double(), row, interleaved, back=True) if row is not None else (g.double(), g.double().abs())
    if weight is None:
        return gy, gsize, None, None
    x, w = x.double(), weight.double()
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    u, usize = gy * w, gsize * w.abs()
    dx = r * (u - x * r ** 2 * (u * x).mean(-1, keepdim=True))
    size = r * (usize + x.abs() * r ** 2 * (usize * x.abs()).mean(-1, keepdim=True))
    return dx, size, (gy * x * r).sum(0), (gsize * x.abs() * r).sum(0)


def legal_keys(length, n_q, i, window, sinks):
    pos = length - n_q + i
    keys = torch.arange(max(pos + 1, 0))
    return keys if window < 0 else keys[(keys >= pos - window) | (keys < sinks)]


def paged_decode(q, k_pages, v_pages, table, lens, scale, window=-1, sinks=0, k_scale=None, v_scale=None):
    """-> out, lse, qbound (root of the sum of squared terms), lse_bound; float64 on the CPU.

    Weights p_j rounded with relative error u_p (bf16: 2^-8, f16: 2^-11), the output with
    2^-8: independent roundings of root mean square at most u / 2, so the error's is
    (u / 2) |out| and (u_p / 2) sqrt(sum p_j^2 v_j^2) in quadrature. Scores: d products summed in
    fp32 (relative d 2^-23 of the terms' sizes, no rounding to nearest assumed), for 8-bit
    pages entries of q moved by at most 2^-25 of the row's largest; exp2 and the sums 2^-20.
    """
    B, n_q, h_q, d = q.shape
    n_pages, h_kv, page, _ = k_pages.shape
    group = h_q // h_kv
    u_p = U_BF16 if k_scale is None else U_F16
    k_pages, v_pages = k_pages.float(), v_pages.float()  # exact
    out, lse = torch.zeros(q.shape, dtype=torch.float64), torch.full((B, n_q, h_q), -math.inf, dtype=torch.float64)
    qb, lb = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(B, n_q, h_q, dtype=torch.float64)
    for b in range(B):
        length = min(max(int(lens[b]), 0), table.shape[1] * page)
        for i in range(n_q):
            keys = legal_keys(length, n_q, i, window, sinks)
            if len(keys) == 0:
                continue
            pages = table[b].long()[keys // page]
            there = (pages >= 0) & (pages < n_pages)
            keys, pages = keys[there], pages[there]
            if len(keys) == 0:
                continue
            for h in range(h_q):
                z = h // group
                k, v = k_pages[pages, z, keys % page].double(), v_pages[pages, z, keys % page].double()
                if k_scale is not None:
                    k, v = k * k_scale[z].double(), v * v_scale[z].double()
                x = q[b, i, h].double()
                s = scale * (k @ x)
                lse[b, i, h] = torch.logsumexp(s, 0)
                p = torch.softmax(s, 0)
                out[b, i, h] = p @ v
                ds = abs(scale) * (d * 2.0 ** -23 * (k.abs() @ x.abs()) + 2.0 ** -25 * x.abs().max() * k.abs().sum(1))
                lb[b, i, h] = ds.max() + 2.0 ** -20 + 2.0 ** -22 * lse[b, i, h].abs()
                small = (2 * ds.max() + 2.0 ** -18) * (p @ v.abs())
                weights = (u_p / 2) ** 2 * (p ** 2 @ v ** 2)
                qb[b, i, h] = ((U_BF16 / 2 * out[b, i, h]) ** 2 + weights + small ** 2).sqrt()
    return out, lse, qb, lb
