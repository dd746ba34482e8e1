"""Plain 64-bit implementations of the operators that make and feed the paged cache (pages and slots, rotary
positions, rows in 4 bits), and the error bounds the GPU results are held to.  Torch on the CPU and whole numbers of
Python; no code of the library."""
import math

import torch

from tests.decoder_oracle import U32, power, unit

BIAS, LOW, HIGH, LOST = 127, -111, 119, 255
SCALES = torch.tensor([(8 + b % 8) / 8 * 2.0 ** (b // 8 - 12) for b in range(128)], dtype=torch.float64)


# ------------------------------------------------------------------------ rows in 4 bits ----

def pitch(dim):
    return (dim + 63) // 64 * 4


def quantise4(x):
    """x [..., dim] (finite): (whole numbers, scale bytes of each 16, biased exponents).  The exponent is found by trial
    from below, the scale as the first of all that is large enough."""
    x = x.double()
    top = x.abs().amax(-1)
    e = torch.full(top.shape, LOW, dtype=torch.int64)
    while bool((big := (top > 105.0 * power(e)) & (e < HIGH)).any()):
        e += big.long()
    y = (x / power(e)[..., None]).unflatten(-1, (-1, 16))
    big = y.abs().amax(-1)
    b = (7 * SCALES < big[..., None]).sum(-1).clamp(max=127)
    n = torch.round(y / SCALES[b][..., None]).clamp(-7, 7)
    return n.flatten(-2), b.to(torch.uint8), (e + BIAS).to(torch.uint8)


def values4(n, b, e):
    """Codes, scale bytes (padding or not) and exponents as values, 64 bits; NaN rows as NaN."""
    s = SCALES[b[..., : n.shape[-1] // 16].long().clamp(max=127)] * power(e.long() - BIAS)[..., None]
    v = (n.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)
    return torch.where((e == LOST)[..., None], torch.full((), math.nan, dtype=torch.float64), v)


def pack4(n):
    """Whole numbers [..., dim] as bytes [..., dim / 2]."""
    out = torch.zeros(*n.shape[:-1], n.shape[-1] // 2, dtype=torch.uint8)
    c = n.long() + 8
    for u in range(n.shape[-1] // 4):
        word = sum(c[..., 4 * u + i] << (4 * i) for i in range(4))
        word = (word << 3 | word >> 13) & 0xFFFF
        out[..., 2 * u], out[..., 2 * u + 1] = (word & 255).to(torch.uint8), (word >> 8).to(torch.uint8)
    return out


def unpack4(raw):
    n = torch.zeros(*raw.shape[:-1], raw.shape[-1] * 2, dtype=torch.float64)
    for u in range(raw.shape[-1] // 2):
        word = raw[..., 2 * u].long() | raw[..., 2 * u + 1].long() << 8
        word = (word >> 3 | word << 13) & 0xFFFF
        for i in range(4):
            n[..., 4 * u + i] = (word >> (4 * i) & 15).double() - 8
    return n


def padded(b, dim):
    return torch.cat([b, torch.zeros(*b.shape[:-1], pitch(dim) - b.shape[-1], dtype=torch.uint8)], -1)


# --------------------------------------------------------------------------------- pages ----

def plan(lens, new, table, free, n_free, page, max_tokens):
    """(seq, pos, slot, starts, lens, n_free, table, somebody refused) in whole numbers; lists in, lists out."""
    table = [list(r) for r in table]
    seq, pos, slot = [-1] * max_tokens, [-1] * max_tokens, [-1] * max_tokens
    starts, after, at, asked, refused = [], [], 0, 0, False
    top = n_free
    for b, (n, more) in enumerate(zip(lens, new)):
        n, more = max(n, 0), max(more, 0)
        starts.append(min(at, max_tokens))
        held, wanted = -(-n // page), -(-(n + more) // page)
        ok = n + more <= len(table[b]) * page and at + more <= max_tokens
        if ok:
            asked += wanted - held
            ok = wanted == held or asked <= n_free
            if ok:
                for j in range(held, wanted):
                    top -= 1
                    table[b][j] = free[top]
        refused |= not ok and more > 0
        for i in range(more):
            if at + i >= max_tokens:
                break
            seq[at + i] = b
            if ok:
                p = n + i
                pos[at + i], slot[at + i] = p, table[b][p // page] * page + p % page
        after.append(n + more if ok else n)
        at += more
    starts.append(min(at, max_tokens))
    return seq, pos, slot, starts, after, top, table, refused


def release(lens, ended, table, free, n_free, page):
    free, after = list(free), []
    for b, (n, gone) in enumerate(zip(lens, ended)):
        if gone:
            for j in range(-(-max(n, 0) // page)):
                free[n_free] = table[b][j]
                n_free += 1
        after.append(0 if gone else n)
    return after, n_free, free


# ------------------------------------------------------------------------------- rotary -----

def frequencies(rot, scaling="none", base=10000.0, factor=8.0, original=4096.0, low=1.0, high=32.0):
    """(radians a position, magnitude), pair by pair from the formulas."""
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling == "by_index":
        at = [rot * math.log(original / (2 * math.pi * r)) / (2 * math.log(base)) for r in (high, low)]
        i0, i1 = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        share = [min(max((i - i0) / max(i1 - i0, 0.001), 0), 1) for i in range(rot // 2)]
        return [x * (1 - r) + x / factor * r for x, r in zip(f, share)], 0.1 * math.log(factor) + 1
    if scaling == "by_turns":
        keep = [min(max((original * x / (2 * math.pi) - low) / (high - low), 0), 1) for x in f]
        return [x / factor * (1 - r) + x * r for x, r in zip(f, keep)], 1.0
    return f, 1.0


def turned(x, pos, freq, magnitude, interleaved, inverse=False, out=torch.float32):
    """x [T, heads, dim] turned, and the bound on the error of the result in `out`.

    The bound.  The angle: the table's frequency is off by 2^-64 of a turn (times 2^31 positions at most), the phase is
    cut to 32 bits, and what is left of it after the nearest quarter turn, below 2^29, is rounded to 24: 2^4 and two
    units more of 2^-32 of a turn.  The sine and cosine are off by one unit in the last place (2^-24 below 1), the
    magnitude and its product round twice, then a product and a fused multiply-add."""
    x = x.double()
    half = len(freq)
    a = pos.double()[:, None] * torch.tensor(freq, dtype=torch.float64)
    if inverse:
        a = -a
    c, s = (torch.cos(a) * magnitude)[:, None], (torch.sin(a) * magnitude)[:, None]
    i = torch.arange(half)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y, tol = x.clone(), torch.zeros_like(x)
    p, q = x[..., first], x[..., second]
    y[..., first], y[..., second] = p * c - q * s, q * c + p * s
    off = 18 * 2.0 ** -32 * 2 * math.pi + a.abs()[:, None] * 2.0 ** -52  # (the last: of the angle here)
    each = (p.abs() + q.abs()) * magnitude * (off + 2 * U32 + 4 * U32)
    tol[..., first] = tol[..., second] = each
    return y, tol + unit(out) * (y.abs() + tol) + (0 if out == torch.float32 else 2.0 ** -134)
