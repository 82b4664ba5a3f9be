"""Plain float64 forms of attention over ragged batches (torch, one sequence after the other), with
the sizes of the terms that the tests' tolerances are made of."""
import math

import torch

from paged_reference import U_BF16


def legal_pairs(n_q, n_k, causal, window=-1, sinks=0, device="cpu"):
    """[n_q, n_k] truth values; query i stands at position n_k - n_q + i."""
    pos = torch.arange(n_k - n_q, n_k, device=device)[:, None]
    key = torch.arange(n_k, device=device)[None]
    legal = key <= pos if causal else torch.ones(n_q, n_k, dtype=torch.bool, device=device)
    if window >= 0:
        near = ((key - pos).abs() <= window) | ((key < sinks) & (key <= pos))
        legal = legal & near
    return legal


def attend(q, k, v, scale, legal):
    """One sequence: q [n_q, h_q, d], k, v [n_k, h_kv, d], legal [n_q, n_k] -> out, lse, qbound, lse_bound.

    Weights p_j rounded to bf16 (relative error at most 2^-8), the output too: independent roundings of
    root mean square at most half of that, so the error's is 2^-9 |out| and 2^-9 sqrt(sum p_j^2 v_j^2)
    in quadrature. Scores: d products summed in fp32 (relative d 2^-23 of the terms' sizes, no
    rounding to nearest assumed); exp2, its argument (fp32, up to 2^8 in size: 2^-17) and the sums 2^-17.
    """
    n_q, h_q, d = q.shape
    n_k, h_kv, _ = k.shape
    group = h_q // h_kv
    out = torch.zeros(n_q, h_q, d, dtype=torch.float64, device=q.device)
    lse = torch.full((n_q, h_q), -math.inf, dtype=torch.float64, device=q.device)
    qb, lb = torch.zeros_like(out), torch.zeros_like(lse)
    some = legal.any(1)
    if n_k == 0 or not some.any():
        return out, lse, qb, lb
    used = legal.any(0)  # what no query may see is not looked at
    k, v, legal = k[used], v[used], legal[:, used]
    for h in range(h_q):
        x, kk, vv = q[some, h].double(), k[:, h // group].double(), v[:, h // group].double()
        s = (scale * (x @ kk.T)).masked_fill(~legal[some], -math.inf)
        lse[some, h] = torch.logsumexp(s, -1)
        p = (s - lse[some, h][:, None]).exp()
        out[some, h] = o = p @ vv
        ds = scale * d * 2.0 ** -23 * (x.abs() @ kk.abs().T).masked_fill(~legal[some], 0).amax(-1)
        lb[some, h] = ds + 2.0 ** -19 + 2.0 ** -22 * lse[some, h].abs()
        small = (2 * ds + 2.0 ** -16)[:, None] * (p @ vv.abs())
        qb[some, h] = ((U_BF16 / 2 * o) ** 2 + (U_BF16 / 2) ** 2 * (p ** 2 @ vv ** 2) + small ** 2).sqrt()
    return out, lse, qb, lb


def packed(q, k, v, q_at, k_at, scale, causal, window=-1, sinks=0):
    """-> the four tensors over all rows; rows of no sequence hold 7, as the tests' outputs do before the call."""
    out = torch.full(q.shape, 7.0, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float64, device=q.device)
    qb, lb = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(len(q_at) - 1):
        r, s = slice(q_at[b], q_at[b + 1]), slice(k_at[b], k_at[b + 1])
        legal = legal_pairs(r.stop - r.start, s.stop - s.start, causal, window, sinks, q.device)
        out[r], lse[r], qb[r], lb[r] = attend(q[r], k[s], v[s], scale, legal)
    return out, lse, qb, lb


def chunk(q, q_at, k_pages, v_pages, table, lens, scale, window=-1, sinks=0, k_scale=None, v_scale=None):
    """As packed, over a paged cache; keys of pages that do not exist are illegal."""
    n_pages, h_kv, page, d = k_pages.shape
    out = torch.full(q.shape, 7.0, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float64, device=q.device)
    qb, lb = torch.zeros_like(out), torch.zeros_like(lse)
    k_pages, v_pages = k_pages.float(), v_pages.float()  # exact
    if k_scale is not None:
        k_pages, v_pages = k_pages.double() * k_scale.double()[:, None, None], v_pages.double() * v_scale.double()[:, None, None]
    for b in range(len(q_at) - 1):
        r = slice(q_at[b], q_at[b + 1])
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        key = torch.arange(n, device=q.device)
        ids = table[b].long()[key // page]
        there = (ids >= 0) & (ids < n_pages)
        legal = legal_pairs(r.stop - r.start, n, True, window, sinks, q.device) & there
        ids = ids.clamp(0, n_pages - 1)
        out[r], lse[r], qb[r], lb[r] = attend(q[r], k_pages[ids, :, key % page], v_pages[ids, :, key % page], scale, legal)
    return out, lse, qb, lb


def attend_bwd(q, k, v, out, lse, dout, scale, legal):
    """One sequence's dq, dk, dv from the definition (P from lse, D from out), each with its qbound.

    P, dS and the results are rounded to bf16: independent roundings of root mean square at most 2^-9,
    so a sum of products of theirs moves by 2^-9 sqrt(sum of squared terms), the result by 2^-9 of itself.
    Scores and dP are d products summed in fp32 (relative d 2^-23 of the terms' sizes); exp2, its argument
    and the differences dP - D: 2^-16 of |dP| + |D| (D from bf16 rows in fp32: d 2^-23 of its terms).
    """
    n_q, h_q, d = q.shape
    n_k, h_kv, _ = k.shape
    group = h_q // h_kv
    f64 = dict(dtype=torch.float64, device=q.device)
    dq, qq = torch.zeros(n_q, h_q, d, **f64), torch.zeros(n_q, h_q, d, **f64)
    dk, qk, dv, qv = (torch.zeros(n_k, h_kv, d, **f64) for _ in range(4))
    some, used = legal.any(1), legal.any(0)
    if n_k == 0 or not some.any():
        return dq, dk, dv, qq, qk, qv
    legal = legal[some][:, used]
    u2 = (U_BF16 / 2) ** 2
    small_k, small_v = torch.zeros_like(qk), torch.zeros_like(qv)
    for h in range(h_q):
        z = h // group
        x, g, o = (t[some, h].double() for t in (q, dout, out))
        kk, vv = k[used, z].double(), v[used, z].double()
        p = (scale * (x @ kk.T) - lse[some, h].double()[:, None]).exp().masked_fill(~legal, 0)
        dp, dd = g @ vv.T, (g * o).sum(-1, keepdim=True)
        ds = p * (dp - dd)
        # fp32 errors of P (relative) and of dS
        es = 2 * scale * d * 2.0 ** -23 * (x.abs() @ kk.abs().T) + 2.0 ** -16
        eds = ds.abs() * es + p * (d * 2.0 ** -22 * (g.abs() @ vv.abs().T + (g * o).abs().sum(-1, keepdim=True)))
        dq[some, h] = scale * (ds @ kk)
        dv[used, z] += p.T @ g
        dk[used, z] += scale * (ds.T @ x)
        qq[some, h] = scale ** 2 * u2 * (ds ** 2 @ kk ** 2) + (scale * (eds @ kk.abs())) ** 2
        qv[used, z] += u2 * ((p ** 2).T @ g ** 2)
        qk[used, z] += scale ** 2 * u2 * ((ds ** 2).T @ x ** 2)
        small_v[used, z] += (p * es).T @ g.abs()
        small_k[used, z] += scale * (eds.T @ x.abs())
    return (dq, dk, dv, (qq + u2 * dq ** 2).sqrt(), (qk + small_k ** 2 + u2 * dk ** 2).sqrt(),
            (qv + small_v ** 2 + u2 * dv ** 2).sqrt())


def packed_bwd(q, k, v, out, lse, dout, q_at, k_at, scale, causal, window=-1):
    """-> dq, dk, dv and their qbounds over all rows; rows of no sequence hold 7."""
    got = [torch.full(x.shape, 7.0, dtype=torch.float64, device=q.device) for x in (q, k, v)]
    bounds = [torch.zeros_like(x) for x in got]
    for b in range(len(q_at) - 1):
        r, s = slice(q_at[b], q_at[b + 1]), slice(k_at[b], k_at[b + 1])
        legal = legal_pairs(r.stop - r.start, s.stop - s.start, causal, window, 0, q.device)
        g = attend_bwd(q[r], k[s], v[s], out[r], lse[r], dout[r], scale, legal)
        for x, to, rows in zip(g, got + bounds, (r, s, s, r, s, s)):
            to[rows] = x
    return got, bounds


def check_grads(got, want, bounds):
    """Per element 6 qbound, over a tensor 2 ||qbound||: where softmax leaves one key almost all the weight, one
    rounding decides the norm, and it may be at its largest, 2^-8 of the term, twice the mean that
    qbound counts. With e_ij the roundings of dS: ||sum_i e_ij q_i||^2 summed over j is sum_ij e_ij^2 |q_i|^2
    plus products of independent roundings (zero in the mean), and e_ij^2 <= (2^-8 ds_ij)^2 = 4 (2^-9 ds_ij)^2."""
    for name, x, y, qb in zip(("dq", "dk", "dv"), got, want, bounds):
        err = (x.double() - y).abs()
        assert torch.all(err <= 6 * qb + 1e-30), f"{name}: {(err / qb.clamp_min(1e-30)).max():.2f} of qbound"
        assert err.norm() <= 2 * qb.norm() + 1e-30, f"{name}: {(err.norm() / qb.norm()):.2f} of the norm's bound"


def check(got, lse, want, want_lse, qb, lb):
    """Per element 6 qbound, over the tensor ||qbound||; each lse within its bound; NaN where the formula is."""
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.isnan(lse), torch.isnan(want_lse))
    err = torch.where(fin, got.double() - want, 0.0).abs()
    qb = torch.where(fin, qb, 0.0)
    assert torch.all(err <= 6 * qb + 1e-30), f"{(err / qb.clamp_min(1e-30)).max():.2f} of qbound"
    assert err.norm() <= qb.norm() + 1e-30
    assert torch.equal(want_lse == -math.inf, lse == -math.inf)
    ok = torch.isfinite(want_lse)
    assert torch.all((lse.double() - want_lse)[ok].abs() <= lb[ok])
