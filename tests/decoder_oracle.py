"""Plain 64-bit implementations of the decode-step operators, and the error bounds the GPU results
are held to.  Torch on the CPU, one row at a time; no code of the library.

Bounds count roundings of half a step, u(t) = torch.finfo(t).eps / 2 relative to the value."""
import math

import torch

U32 = torch.finfo(torch.float32).eps / 2
UBF = torch.finfo(torch.bfloat16).eps / 2
BIAS = 127


def unit(t):
    return torch.finfo(t).eps / 2


def power(e):
    """2^e in 64 bits for whole e."""
    return torch.bitwise_left_shift(e.long() + 1023, 52).view(torch.float64)


def round_e4m3(x):
    """x (|x| <= 448) at the nearest E4M3 value, ties to even: steps of 2^-3 of the binade, 2^-9 below 2^-6."""
    p = (x.abs().clamp(min=2.0 ** -6).view(torch.int64) >> 52) - 1023
    step = power(p - 3)
    return torch.round(x / step) * step


def quantise(x):
    """x [..., dim]: (codes as values, biased exponents).  The exponent is found by trial from below."""
    x = x.double()
    top = x.abs().amax(-1)
    e = torch.full(top.shape, -BIAS, dtype=torch.int64)
    while bool((big := top > 448.0 * power(e)).any()):
        e += big.long()
    return round_e4m3(x / power(e)[..., None]), (e + BIAS).to(torch.uint8)


def place(cache_page, table, s, p):
    return int(table[s, p // cache_page]), p % cache_page


def cached(pool, exps, page, head, row):
    """One row of the cache in 64 bits."""
    x = pool[page, head, row]
    if exps is None:
        return x.double()
    return x.view(torch.float8_e4m3fn).double() * power(exps[page, head, row].long() - BIAS)


def attention(q, k, v, k_exp, v_exp, lens, table, scale, window):
    """(out, lse, bound on out's error, bound on lse's error), 64 bits, CPU tensors.  Pages outside the
    pool count as masked, lengths past the table are cut.

    The bound.  A score is an fp32 sum of dim products (exact: 8 x 8 or 4 x 8 significant bits), so off by
    at most dim 2u32 sum|q_d k_d| however it is ordered (2u32: tensor cores may truncate); scaling it and
    taking it from the maximum round three times more at the size of the largest score.  exp2 adds 4 u32 a
    factor, and a weight is rescaled at most once a tile of 16 tokens or more.  p is rounded to bf16 or fp16
    before its product with v (UBF covers both), the sum over the tokens is off by 2u32 a term, and the
    result is rounded to bf16 once."""
    B, H, D = q.shape
    n_pages, hk, page, _ = k.shape
    out = torch.zeros(B, H, D, dtype=torch.float64)
    lse = torch.full((B, H), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(B):
        n = min(int(lens[b]), table.shape[1] * page)
        first = max(0, n - window) if window else 0
        at = [(p, r) for p, r in (place(page, table, b, j) for j in range(first, max(n, 0))) if 0 <= p < n_pages]
        if not at:
            continue
        for kv in range(hk):
            ks = torch.stack([cached(k, k_exp, p, kv, r) for p, r in at])
            vs = torch.stack([cached(v, v_exp, p, kv, r) for p, r in at])
            for h in range(kv * (H // hk), (kv + 1) * (H // hk)):
                qd = q[b, h].double()
                s = ks @ qd * scale
                lse[b, h] = torch.logsumexp(s, 0)
                p = torch.softmax(s, 0)
                out[b, h] = p @ vs
                m = len(at)
                size = (ks.abs() @ qd.abs()).max() * abs(scale)
                eps = D * 2 * U32 * size + 6 * U32 * size + 4 * U32 * (2 + m / 16)
                a = p @ vs.abs()
                tol[b, h] = UBF * out[b, h].abs() + (1 + UBF) * (UBF + 2 * eps + 2 * U32 * (m + 8)) * a
                tol_lse[b, h] = eps + 2 * U32 * m + 4 * U32 * lse[b, h].abs()
    return out, lse, tol, tol_lse


def block_norm(y, w_post, gate, alpha, residual, w_pre, eps, r_type, x_type):
    """(r', x, bound on r', bound on x) in 64 bits.  The bound: a sum of squares in the kernel runs over at
    most 32 elements a thread, 5 steps over the lanes and 16 over the warps, so 64 u32 covers it with the
    division and eps; rsqrt adds 4 u32, each product one."""
    r = residual.double()
    tol = torch.zeros_like(r)
    if y is not None:
        z = y.double()
        rel = 0.0
        if w_post is not None:
            z = z / torch.sqrt((z * z).mean(-1, keepdim=True) + eps) * w_post.double()
            rel += (32 + 4 + 2) * U32
        if gate is not None:
            z = z * gate.double()
            rel += U32
        r = r + alpha * z
        tol = (rel + 2 * U32) * (alpha * z).abs() + U32 * r.abs()
    tol_r = tol + unit(r_type) * (r.abs() + tol)
    if w_pre is None:
        return r, None, tol_r, None
    rms = torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    x = r / rms * w_pre.double()
    d_rms = torch.sqrt((tol * tol).mean(-1, keepdim=True)) / rms  # the rms moves by no more than the errors' rms
    tol_x = (tol / rms * w_pre.double().abs()) * 1.01 + x.abs() * (d_rms * 1.01 + (32 + 4 + 2) * U32)
    return r, x, tol_r, tol_x + unit(x_type) * (x.abs() + tol_x)
