"""64-bit statements of the mixture-of-experts block's operators (norm +
quantization, routing, expert MLP) with error bounds derived from the
arithmetic, for the GPU tests. Plain torch / numpy in double precision; none of
the library's code."""

import math

import numpy as np
import torch

G = 128
E4M3_MAX = 448.0
U32 = 2.0 ** -24     # half a step of fp32, relative
U16 = 2.0 ** -8      # half a step of bf16, relative (finfo(bfloat16).eps / 2)


def e4m3_values(codes):
    return codes.view(torch.float8_e4m3fn).to(torch.float64)


def scale_values(s):
    if s.dtype == torch.float32:
        return s.double()
    return torch.exp2(s.double() - 127.0)


def dequant_rows(q, s):
    return e4m3_values(q) * scale_values(s).repeat_interleave(G, dim=-1)


def dequant_blocks(q, s):
    return e4m3_values(q) * scale_values(s).repeat_interleave(G, dim=-1).repeat_interleave(G, dim=-2)


def e4m3_step(v):
    """Distance between E4M3 values around |v| (the step of v's binade)."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    return torch.exp2(e.clamp(max=8.0) - 3.0)


def e4m3_round(v):
    step = e4m3_step(v)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def group_scale(amax, fmt):
    if fmt == "fp32":
        return amax / E4M3_MAX
    e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -140) / E4M3_MAX))
    e = torch.where(torch.exp2(e - 1) * E4M3_MAX >= amax, e - 1, e)
    e = torch.where(torch.exp2(e) * E4M3_MAX < amax, e + 1, e)
    return torch.exp2(e.clamp(-127, 127))


# -------------------------------------------------------------------- norm --
def norm_rows(x, residual, weight, eps):
    """(n, r) of bf16 rows: r exact (bf16 of the fp32 sum), n in 64 bits."""
    r = x if residual is None else (x.float() + residual.float()).to(torch.bfloat16)
    v = r.double()
    n = v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + eps)
    return (n if weight is None else n * weight.double()), r


# Relative error of the kernel's fp32 n: the sum of squares of K <= 65536 values
# runs over at most 64 chained additions per thread, 10 tree levels and one
# rounding each of the square, of the mean and of eps (< 80 steps, halved by
# the square root), then the inverse root and two products: below 2^-18.
NORM_REL = 2.0 ** -18


def check_norm(n, fmt, q, s, y=None):
    """q, s, y of the GPU against the exact n: y within half a bf16 step, the
    scales within NORM_REL, and every code's value within half an E4M3 step of
    n (relative 2^-4, or half a subnormal step 2^-10 s)."""
    M, K = n.shape
    amax = n.abs().view(M, K // G, G).amax(dim=2)
    sv = scale_values(s)
    if fmt == "fp32":
        assert bool(((sv - amax / E4M3_MAX).abs() <= amax / E4M3_MAX * 2 * NORM_REL + 2.0 ** -149).all())
    else:
        low = 2.0 ** -127
        assert bool(((sv * E4M3_MAX >= amax * (1 - 2 * NORM_REL))).all())
        assert bool(((sv / 2 * E4M3_MAX < amax * (1 + 2 * NORM_REL)) | (sv == low)).all())
    wide = sv.repeat_interleave(G, dim=1)
    err = (e4m3_values(q) * wide - n).abs()
    tol = torch.maximum(n.abs() * 2.0 ** -4, wide * 2.0 ** -10) * (1 + 2.0 ** -16) + n.abs() * 4 * NORM_REL
    assert bool((err <= tol).all()), float((err - tol).max())
    if y is not None:
        assert bool(((y.double() - n).abs() <= n.abs() * (U16 + 2 * NORM_REL) + 2.0 ** -133).all())


# ----------------------------------------------------------------- routing --
def route(logits, top_k, scoring, bias=None, n_group=1, topk_group=1, renormalize=True, scale=1.0):
    """(ids, weights in 64 bits, finite keys' order) by loops over tokens."""
    x = logits.double().cpu().numpy()
    b = None if bias is None else bias.double().cpu().numpy()
    M, E = x.shape
    ids = np.full((M, top_k), -1, np.int32)
    w = np.zeros((M, top_k))
    for m in range(M):
        live = [e for e in range(E) if x[m, e] > -math.inf and (b is None or b[e] > -math.inf)]
        sig = {e: 1.0 / (1.0 + np.exp(-x[m, e])) for e in live}
        key = {e: x[m, e] if b is None and n_group == 1 else
               (sig[e] + (0.0 if b is None else b[e])) for e in live}
        if n_group > 1:
            per = E // n_group
            score = []
            for g in range(n_group):
                two = sorted((key[e] for e in live if e // per == g), reverse=True)[:2]
                score.append(sum(two) if two else -math.inf)
            best = sorted(range(n_group), key=lambda g: (-score[g], g))[:topk_group]
            live = [e for e in live if e // per in best]
        pick = sorted(live, key=lambda e: (-key[e], e))[:top_k]
        some = [x[m, e] for e in range(E) if x[m, e] > -math.inf]
        top = max(some) if some else 0.0
        total = sum(math.exp(v - top) for v in some)
        for j, e in enumerate(pick):
            ids[m, j] = e
            w[m, j] = sig[e] if scoring == "sigmoid" else math.exp(x[m, e] - top) / total
        if renormalize:
            w[m] /= w[m].sum() + 1e-20
    return ids, w * scale


# -------------------------------------------------------------- expert MLP --
def product(a, w):
    """a . w^T and the bound of its fp32 error on the GPU: the tensor cores add
    128 products per K-block (allowed 2 roundings each) and the K-blocks are
    chained, (K / 128 + 256) roundings of the sum of magnitudes."""
    err = (a.abs() @ w.abs().T) * ((a.shape[1] // G + 256) * U32)
    return a @ w.T, err


def expert_mlp(a, wg, wd, fmt):
    """One expert on rows a: (d, bound of the error of d)."""
    I = wd.shape[1]
    gu, e_gu = product(a, wg)
    g, u, eg, eu = gu[:, :I], gu[:, I:], e_gu[:, :I], e_gu[:, I:]
    silu = g * torch.sigmoid(g)
    h = silu * u
    # silu's slope is below 1.1; fast exponential and divide: 2^-19 relative
    eh = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + h.abs() * 2.0 ** -19
    R = h.shape[0]
    amax, at = h.abs().view(R, I // G, G).max(dim=2)
    e_amax = eh.view(R, I // G, G).amax(dim=2)
    s = group_scale(amax, fmt)
    rel = (e_amax / amax.clamp(min=1e-300)).clamp(max=1.0) + 2 * U32
    one = torch.ones_like(s)
    wide, rel_w = (t.repeat_interleave(G, dim=1) for t in (torch.where(s == 0, one, s), rel))
    v = h / wide
    q = e4m3_round(v)
    # how far the quotient may be off, and with it the code: one whole step
    # where a rounding boundary is that near
    ev = eh / wide + (v.abs() * rel_w if fmt == "fp32" else 0.0)
    lo, hi = e4m3_round(v - ev), e4m3_round(v + ev)
    move = torch.maximum((hi - q).abs(), (q - lo).abs())
    eh_q = (move + (q.abs() * rel_w if fmt == "fp32" else 0.0)) * wide
    if fmt != "fp32":
        # amax within its error of a power-of-two border: the group's scale may
        # double or halve, which moves a value by up to its own half step
        near = group_scale(amax - e_amax, fmt) != group_scale(amax + e_amax, fmt)
        near = near.repeat_interleave(G, dim=1)
        eh_q = torch.where(near, eh_q + 2 * e4m3_step(v) * wide, eh_q)
    hq = q * torch.where(s == 0, torch.zeros_like(s), s).repeat_interleave(G, dim=1)
    d, ed = product(hq, wd)
    return d, ed + eh_q @ wd.abs().T


def moe(qa, sa, ids, weights, qg, sg, qd, sd, first=0):
    """(y, tolerance) of the whole layer; weights that repeat an expert add."""
    fmt = "fp32" if sa.dtype == torch.float32 else "ue8m0"
    a = dequant_rows(qa, sa)
    M, K = a.shape
    y = torch.zeros(M, K, dtype=torch.float64, device=a.device)
    err = torch.zeros_like(y)
    mag = torch.zeros_like(y)
    local = ids.long() - first
    for e in range(qg.shape[0]):
        hit = local == e
        rows = torch.nonzero(hit.any(dim=1)).view(-1)
        if rows.numel() == 0:
            continue
        d, ed = expert_mlp(a[rows], dequant_blocks(qg[e], sg[e]), dequant_blocks(qd[e], sd[e]), fmt)
        w = weights.double() * hit
        share, size = w.sum(dim=1)[rows, None], w.abs().sum(dim=1)[rows, None]
        y[rows] += share * d
        err[rows] += size * ed
        mag[rows] += size * d.abs()
    # the weighted sum: one product and one addition per choice, in any order
    # and grouping of the kernel's, on top of each d's own error
    steps = 2 * (ids.shape[1] + 8)
    tol = err + mag * steps * U32 + (y.abs() + err) * U16 + 2.0 ** -133
    return y, tol
