"""Plain definitions for the paged cache's tests: batches, the rotation, the rows' stored values
(CPU oracle) and attention in 64 bits with a bound of the rounding errors."""
import math

import numpy as np
import torch

import oracle

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
PAIRS = [("f16", "f16"), ("q8_0", "q8_0"), ("q8_0", "q4_0"), ("q4_0", "q4_0")]
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def table(rng, lens, page, spare=2, pages=None):
    """A block table of distinct shuffled pages: (int32 [n, width], pages in the pool)."""
    need = [-(-max(int(a), 0) // page) for a in lens]
    total = sum(need) + spare if pages is None else pages
    perm = rng.permutation(total).astype(np.int32)
    width = max(max(need), 1)
    t = np.full((len(lens), width), -7, np.int32)  # never read past a sequence's pages
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = perm[at:at + k]
        at += k
    return t, total


def dev(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a), dtype=dtype).cuda()


def cumulative(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def rotate(x, cos_sin, pos, rot, interleaved):
    """fp32 rotation with one rounding per operation (numpy): x [n, heads, D], pos [n]."""
    x = np.ascontiguousarray(x, np.float32)
    y = x.copy()
    c = cos_sin[pos][:, None, :rot // 2].astype(np.float32)
    s = cos_sin[pos][:, None, rot // 2:].astype(np.float32)
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., lo], x[..., hi]
    y[..., lo] = a * c - b * s
    y[..., hi] = b * c + a * s
    return y


def angles(n, rot, base=10000.0):
    a = np.arange(n, dtype=np.float64)[:, None] * base ** (-2.0 * np.arange(rot // 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], -1).astype(np.float32)


def stored(kind, rows):
    """float64 values that fp32 rows stand for once stored."""
    codes, scales = oracle.quantize(kind, np.ascontiguousarray(rows, np.float32))
    return oracle.dequantize(kind, codes, scales, rows.shape[-1])


def attend(q, k, v, scale):
    """q [n, Hq, D] (the last n positions), k, v [len, Hkv, D] float64 tensors: (out, lse, weighted
    |v|, largest sum of |q||k| per row), all float64; rows that see nothing give 0 and -inf."""
    n, hq, d = q.shape
    length, hkv = k.shape[0], k.shape[1]
    g = hq // hkv
    out = torch.zeros((n, hq, d), dtype=torch.float64, device=q.device)
    av, lse = torch.zeros_like(out), torch.full((n, hq), -math.inf, dtype=torch.float64, device=q.device)
    qk = torch.zeros((n, hq), dtype=torch.float64, device=q.device)
    if length == 0 or n == 0:
        return out, lse, av, qk
    hide = torch.arange(length, device=q.device)[None] > torch.arange(n, device=q.device)[:, None] + (length - n)
    for h in range(hkv):
        qh = q[:, h * g:(h + 1) * g].double()
        w = torch.einsum("tgd,kd->tgk", qh, k[:, h]) * scale
        w = w.masked_fill(hide[:, None], -math.inf)
        z = torch.logsumexp(w, -1)
        p = torch.where(z[..., None] == -math.inf, torch.zeros_like(w), (w - z[..., None]).exp())
        out[:, h * g:(h + 1) * g] = torch.einsum("tgk,kd->tgd", p, v[:, h])
        av[:, h * g:(h + 1) * g] = torch.einsum("tgk,kd->tgd", p, v[:, h].abs())
        lse[:, h * g:(h + 1) * g] = z
        a = torch.einsum("tgd,kd->tgk", qh.abs(), k[:, h].abs()) * abs(scale)
        qk[:, h * g:(h + 1) * g] = a.masked_fill(hide[:, None], 0.0).amax(-1)
    return out, lse, av, qk


def offset_terms(pair, q, k, v, scale, keys):
    """What the offset of 4-bit codes adds to the errors: (scores [n, Hq], outputs).

    A 4-bit value is d (c - 8), c in 0 .. 15, and a kernel may sum d c and 8 d apart and subtract: exact
    products, but the two fp32 sums are up to 15 d and 8 d times their weights while their difference can
    be 0.  With d <= max|x| / 8 over the rows, a sum of m such terms is off by at most
    (m + 1) 2^-23 (15 + 8) / 8 max|x| times the sum of the weights: m = 32 (one block) with weights |q|
    scale for the scores, m = keys with weights that sum to 1 for the outputs."""
    hq = q.shape[1]
    e = torch.zeros((q.shape[0], hq), dtype=torch.float64, device=q.device)
    if keys == 0:
        return e, 0.0
    if pair[0] == "q4_0":
        e = q.double().abs().sum(-1) * abs(scale) * float(k.abs().max()) * (23 / 8 * 33 * 2.0 ** -23)
    return e, (float(v.abs().max()) * 23 / 8 * (keys + 1) * 2.0 ** -23 if pair[1] == "q4_0" else 0.0)


def bounds(out, av, qk, dtype, keys, dim, sixteen, offset=None):
    """(bound of |out|'s error, bound of lse's) from the roundings the kernels may make.

    Scores: with `sixteen` (keys as 16-bit operands) each key value is rounded once, half a step of
    float16, 2^-11, of |q||k|; otherwise queries and keys are hi + lo pairs, 2^-20.  fp32 sums of
    `dim` products add dim 2^-23 (products and partial sums).  A score off by e changes a weight by at most 2e
    relative (numerator and denominator), e < 1.  Weights and values as 16-bit operands: 2^-11 each for 16-bit
    outputs (and one product of weight and scale, 2^-11), 2^-19 otherwise.  fp32 sums over keys:
    keys 2^-23 for numerator and denominator together.  Then half a step of the output's type.
    `offset`: offset_terms(...) of 4-bit rows."""
    e = qk * ((2.0 ** -11 if sixteen else 2.0 ** -20) + dim * 2.0 ** -23) + 2.0 ** -20
    if offset is not None:
        e = e + offset[0]
    assert float(e.max()) < 0.5, "inputs too large for the first-order bound"
    part = 3 * 2.0 ** -11 if dtype != "f32" else 2.0 ** -19
    rel = 2 * e * (1 + 2 * e) + (part + keys * 2.0 ** -23)
    tol = out.abs() * HALF_STEP[dtype] + av * rel[..., None] * (1 + HALF_STEP[dtype])
    # values below the 16-bit types' normal range are rounded absolutely
    tol = tol + (2.0 ** -25 if dtype != "f32" else 2.0 ** -60)
    if offset is not None:
        tol = tol + offset[1]
    return tol, e + keys * 2.0 ** -23 + 2.0 ** -20
