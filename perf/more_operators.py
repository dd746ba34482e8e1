"""What is measured of the operators that make and feed the paged cache on the GPU, and of the cache
in 4 bits: pages and slots of new tokens planned from the sequences' lengths, and given back; rotary
positions, alone and on the way into the cache; keys and values written, read back and attended to in
4 bits.

`listed()` gives the cases, `draw(rng)` more of the same ranges, `prepare(case, seed)` what a program has
in hand before the call, `run(state)` one pass (the plain form in elementary torch operations, or with
`own` the library's calls), `exact(case, seed)` the definition in 64 bits and `work(case)` the bytes and
operations a pass cannot do without.

The cache: pages of `page` tokens; position p of sequence s is at row p % page of page page_table[s, p //
page], and slot page * (pages' number) + row names that place.  In 4 bits a row of `dim` elements is

    value i = n_i * scale(byte of group i // 16) * 2^(exponent - 127),   n_i whole, -7 .. 7
    scale(b) = (1 + (b % 8) / 8) * 2^(b // 8 - 12),                      b in 0 .. 127

four codes c = n + 8 to 16 bits, c0 in the lowest four, and those 16 bits turned left by three.
"""
import math
import random

import torch

own = False

BIAS = 127                  # of the stored exponents
E4M3_MAX = 448.0
LOW4, HIGH4 = -111, 119     # exponents of rows in 4 bits
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------- cases ------

def listed():
    pages = dict(op="pages", page=64, ended=0, tight=False)
    rope = dict(op="rope", heads=32, dim=128, rot=128, layout="half", scaling="none", kind="bf16", far=4096)
    place = dict(op="place", heads=32, kv_heads=4, dim=128, page=64, cache="int4", src="bf16", rot=128, layout="half",
                 scaling="none")
    attn = dict(op="attn", heads=32, kv_heads=4, dim=128, page=64, window=0, lse=False)
    return [
        # a decode step's bookkeeping: one token for each of 64 users, a page for those whose last one is full
        dict(pages, name="pages-step-64", batch=64, length=4096, new=1),
        # a batch of prompts admitted at once, in small pages
        dict(pages, name="pages-prompts-192", batch=192, length=1, new=4096, page=16),
        # a large batch of which a part has ended: their pages back to the pool
        dict(pages, name="pages-ended-256", batch=256, length=16384, new=0, page=16, ended=64),
        # one user's queries and keys rotated in a decode step: the smallest call
        dict(rope, name="rope-step-1", tokens=1),
        # a 16k prompt's queries at positions far past the trained context, frequencies scaled for it
        dict(rope, name="rope-prompt-16k", tokens=16384, scaling="by_index", far=262144),
        # a decode step's queries and keys rotated, keys and values into a 4-bit cache
        dict(place, name="place-step-64-int4", batch=64, length=8192, tokens=64),
        # the same for prompts of mixed lengths into a bf16 cache, interleaved pairs over half of each head
        dict(place, name="place-prompts-16k", batch=8, length=4096, tokens=16384, cache="bf16", rot=64,
             layout="interleaved"),
        # prompts that need no rotation, into the 4-bit cache and read back for the prompt's attention
        dict(place, name="write-prompts-16k-int4", op="write", batch=8, length=4096, tokens=16384),
        # one user's next token in a sliding-window layer: all latency
        dict(attn, name="attn-int4-window-1", batch=1, length=16384, window=513),
        # one user's next token at 64k tokens: one row, a long axis to split
        dict(attn, name="attn-int4-1x64k", batch=1, length=65536),
        # a loaded server: 64 users of up to 16k tokens; the largest
        dict(attn, name="attn-int4-64x16k", batch=64, length=16384),
        # odd everything: 7 query heads a kv head, 96 wide, pages of 48, empty and one-token rows, with the
        # log-sum-exp that joins this with another part of the context
        dict(attn, name="attn-int4-odd-9", batch=9, length=3001, heads=14, kv_heads=2, dim=96, page=48, lse=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "rope", "place", "place", "write", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    scaling = rng.choice(["none", "linear", "base", "by_index", "by_turns"])
    layout = rng.choice(["half", "interleaved"])
    if op == "pages":
        batch = _log_int(rng, 1, 1024)
        new = rng.choice([0, 1, 1, _log_int(rng, 1, max(1, 400000 // batch))])
        return dict(op=op, batch=batch, length=_log_int(rng, 1, 16384), new=new, page=page,
                    ended=rng.randint(1, batch) if new == 0 else 0, tight=rng.random() < 0.3)
    if op == "rope":
        dim, heads = 8 * rng.randint(4, 32), rng.randint(1, 48)
        return dict(op=op, heads=heads, dim=dim, rot=8 * rng.randint(1, dim // 8), layout=layout, scaling=scaling,
                    kind=rng.choice(["bf16", "bf16", "fp32"]), far=_log_int(rng, 1, 1 << 22),
                    tokens=_log_int(rng, 1, min(32768, (1 << 26) // (dim * heads))))
    kv_heads = rng.randint(1, 8)
    if op == "attn":
        dim = rng.choice([64, 96, 128, 128, 160, 192, 256])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
        budget = min(1 << 19, (1 << 28) // (kv_heads * dim), (1 << 30) // (heads * dim))   # tokens of all sequences
        batch = _log_int(rng, 1, 192)
        return dict(op=op, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                    window=rng.choice([0, 0, 513, _log_int(rng, 1, 4096)]), batch=batch,
                    length=_log_int(rng, 1, min(65536, max(1, budget // batch))), lse=rng.random() < 0.3)
    cache = "int4" if op == "write" else rng.choice(["int4", "int4", "bf16", "e4m3"])
    dim = rng.choice([64, 96, 128, 128, 160, 192, 256]) if cache == "int4" else 16 * rng.randint(2, 16)
    per_token = kv_heads * dim
    batch = _log_int(rng, 1, 64)
    tokens = max(batch, _log_int(rng, 1, min(16384, (1 << 23) // per_token)))
    length = min(8192, (min(1 << 16, (1 << 25) // per_token) + tokens) // batch + 1)
    return dict(op=op, heads=kv_heads * rng.choice([1, 2, 4, 8]), kv_heads=kv_heads, dim=dim, page=page, cache=cache,
                src=rng.choice(["bf16", "bf16", "fp32"]), batch=batch, length=max(length, -(-tokens // batch)),
                tokens=tokens, rot=8 * rng.randint(1, dim // 8), layout=layout, scaling=scaling)


def _mixed(rng, n, top):
    """Lengths as in serving, short ones common, one of them `top`."""
    lens = [max(1, min(top, int(top * rng.random() ** 0.7 + 1))) for _ in range(n)]
    lens[rng.randrange(n)] = top
    return lens


def _shape(case):
    """The sequences' lengths of a case, the same for every seed, so that a case's work is one number: of
    attention's cached tokens (one as it is given, several mixed, an empty and a one-token row among them)."""
    n, top = case["batch"], case["length"]
    if n == 1:
        return [top]
    rng = random.Random("lengths of %d up to %d" % (n, top))
    lens = _mixed(rng, n, top)
    if n >= 8 and case["op"] == "attn":
        a, b = rng.sample(range(n), 2)
        lens[a], lens[b] = 0, 1
    return lens


def _written(case):
    """Sequence and position of every token a case writes: the last ones of each sequence, their counts as
    even as the token count allows (one each in a decode step)."""
    n, lens = case["batch"], _shape(case)
    seq, pos = [], []
    for s in range(n):
        each = case["tokens"] // n + (1 if s < case["tokens"] % n else 0)
        top = max(lens[s], each)
        seq += [s] * each
        pos += list(range(top - each, top))
    return seq, pos


def _row_bytes(case):
    """Bytes of one token's key and value of one kv head in the cache."""
    if case.get("cache", "int4") == "int4":
        return 2 * (case["dim"] // 2 + case["dim"] // 16 + 1)
    return 2 * (case["dim"] + 1) if case["cache"] == "e4m3" else 4 * case["dim"]


def work(case):
    size = {"bf16": 2, "fp32": 4}
    if case["op"] == "pages":
        n = case["batch"]
        if case["ended"]:
            pages = case["ended"] * case["length"] // 2 // case["page"]
            return {"bytes": 9 * n + 8 * pages, "flops": n}
        tokens = n if case["new"] == 1 else n * (case["new"] + 1) // 2
        # each new token's sequence, position and slot, each new page taken from the pool and put into the table
        return {"bytes": 16 * n + 12 * tokens + 8 * tokens // case["page"], "flops": 4 * tokens}
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * size[case["kind"]] * n * case["dim"] + 4 * case["tokens"], "flops": 3 * n * case["rot"]}
    if case["op"] == "attn":
        seen = [min(n, case["window"]) if case["window"] else n for n in _shape(case)]
        tokens, q = sum(seen), case["batch"] * case["heads"]
        return {"bytes": tokens * case["kv_heads"] * _row_bytes(case) + q * (4 * case["dim"] + (4 if case["lse"] else 0))
                + 4 * case["batch"] + 4 * sum(-(-n // case["page"]) for n in seen),
                "flops": 4 * tokens * case["heads"] * case["dim"]}
    rows, d = case["tokens"] * case["kv_heads"], case["dim"]
    n = rows * (2 * d * size[case["src"]] + _row_bytes(case)) + 8 * case["tokens"]
    if case["cache"] != "bf16":
        n += rows * (_row_bytes(case) + 4 * d)      # and read back
    if case["op"] == "write":
        return {"bytes": n, "flops": 6 * rows * d}
    q = case["tokens"] * case["heads"]
    return {"bytes": n + q * d * (size[case["src"]] + 2), "flops": 3 * (q + rows) * case["rot"] + 4 * rows * d}


# ------------------------------------------------------------------------------ inputs ------

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _gen(seed):
    g = torch.Generator(device=_device())
    g.manual_seed(seed * 1000003 + 29)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=_device())


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=_device())


def _rows_like_a_projection(g, rows, heads, dim):
    """Keys or values as a projection makes them: a spread that differs by channel, a few large channels,
    and token norms that vary."""
    x = _randn(g, rows, heads, dim)
    x *= torch.exp(0.4 * _randn(g, 1, heads, dim)) * torch.exp(0.2 * _randn(g, rows, 1, 1))
    return x


# One context of 4096 positions stretched to eight times as many, in each of the ways; pairs that turn more
# than 32 times in the original context keep their frequency, those below one turn take the stretched one
# (by index), or 4 and 1 (by turns).
_BASE, _FACTOR, _ORIGINAL = 10000.0, 8.0, 4096.0
_TURNS = {"by_index": (1.0, 32.0), "by_turns": (1.0, 4.0)}


def _frequencies(rot, scaling):
    """Radians a position of each pair (64 bits, on the GPU) and the factor on cosine and sine."""
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=_device())
    base = _BASE * _FACTOR ** (rot / (rot - 2)) if scaling == "base" and rot > 2 else _BASE
    f = torch.exp(i * (-math.log(base) / rot))
    if scaling == "linear":
        return f / _FACTOR, 1.0
    if scaling == "by_index":
        low, high = _TURNS[scaling]
        at = [rot * math.log(_ORIGINAL / (2 * math.pi * r)) / (2 * math.log(base)) for r in (high, low)]
        first, last = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((i / 2 - first) / max(last - first, 0.001)).clamp(0, 1)
        return f * (1 - ramp) + f / _FACTOR * ramp, 0.1 * math.log(_FACTOR) + 1
    if scaling == "by_turns":
        low, high = _TURNS[scaling]
        keep = ((f * (_ORIGINAL / (2 * math.pi)) - low) / (high - low)).clamp(0, 1)
        return f * keep + f / _FACTOR * (1 - keep), 1.0
    return f, 1.0


def _rope_of(st, case):
    st["freq"], st["magnitude"] = _frequencies(case["rot"], case["scaling"])
    if own:
        low, high = _TURNS.get(case["scaling"], (1.0, 4.0))
        st["rope"] = st["moe"].Rope(case["rot"], base=_BASE, interleaved=case["layout"] == "interleaved",
                                    scaling=case["scaling"], factor=_FACTOR, original=_ORIGINAL, low=low, high=high)


def _pools(g, case, n_pages):
    shape = (n_pages, case["kv_heads"], case["page"])
    pitch = -(-case["dim"] // 64) * 4
    kind = case.get("cache", "int4")
    out = {}
    for name in ("k", "v"):
        if kind == "bf16":
            out[name] = torch.zeros(shape + (case["dim"],), dtype=torch.bfloat16, device=_device())
            continue
        width = case["dim"] // 2 if kind == "int4" else case["dim"]
        out[name] = torch.zeros(shape + (width,), dtype=torch.uint8, device=_device())
        out[name + "_exp"] = torch.full(shape, BIAS, dtype=torch.uint8, device=_device())
        if kind == "int4":
            out[name + "_scale"] = torch.zeros(shape + (pitch,), dtype=torch.uint8, device=_device())
        if case["op"] != "attn":
            continue
        rows, step = shape[0] * shape[1] * shape[2], max(1, (1 << 25) // case["dim"])
        flat = [out[n].view(rows, -1) for n in (name, name + "_scale")] + [out[name + "_exp"].view(rows)]
        for at in range(0, rows, step):     # by slices: a large pool's fp32 copies would not be small
            n = min(step, rows - at)
            codes, scales, exps = _quantise4(_rows_like_a_projection(g, n, 1, case["dim"]).view(n, -1))
            flat[0][at:at + n], flat[1][at:at + n, :scales.shape[1]], flat[2][at:at + n] = _packed(codes), scales, exps
    return out


def _page_table(g, case, tops):
    """Pages handed out in no order, each sequence with room for its last position; a few belong to nobody."""
    width = max(1, max(-(-t // case["page"]) for t in tops))
    n_pages = case["batch"] * width + 3
    order = torch.randperm(n_pages, generator=g, device=_device())
    return order[: case["batch"] * width].view(case["batch"], width).int().contiguous(), n_pages


def _prepare_pages(case, st, g, seed):
    """Sequences of mixed lengths with their pages, a pool of the rest, and the new tokens of each (about one
    in eight has none where they vary).  `tight`: the pool is too small for all of them."""
    rng = random.Random("sequences of %d up to %d, %d" % (case["batch"], case["length"], case["new"]))
    n, page = case["batch"], case["page"]
    lens = [0 if rng.random() < 0.1 else x for x in _mixed(rng, n, case["length"])]
    new = [case["new"]] * n
    if case["new"] > 1:
        new = [0 if rng.random() < 0.125 else rng.randint(1, case["new"]) for _ in range(n)]
    # the same sequences for every seed, in another order: a case's sizes are its own
    rng = random.Random(seed * 7919 + 5)
    order = rng.sample(range(n), n)
    lens, new = [lens[i] for i in order], [new[i] for i in order]
    width = -(-max(a + b for a, b in zip(lens, new)) // page) + 1
    held = [-(-x // page) for x in lens]
    need = sum(-(-(a + b) // page) for a, b in zip(lens, new)) - sum(held)
    free = max(1, need // 2) if case["tight"] else need + 5
    total = sum(held) + free
    order = torch.randperm(total, generator=g, device=_device()).int()
    column = torch.arange(width, device=_device())
    at = torch.cumsum(_ints(held).long(), 0) - _ints(held).long()
    index = (at[:, None] + column).clamp(max=total - 1)
    st["table"] = torch.where(column < _ints(held)[:, None], order[index], torch.full((), -1, device=_device())).int()
    st["free"] = torch.zeros(total, dtype=torch.int32, device=_device())
    st["free"][:free] = order[sum(held):]
    st["n_free"] = _ints([free])
    st["lens"], st["new"], st["n_pages"] = _ints(lens), _ints(new), total
    # the step's tokens are padded to a fixed number, as in a captured step
    st["max_tokens"] = max(1, sum(new)) + 7
    gone = set(rng.sample(range(n), min(n, case["ended"])))
    st["ended"] = torch.tensor([b in gone for b in range(n)], device=_device())
    if own:
        m = st["moe"]
        st["ws"] = m.pages_workspace(n, _device())
        st["out"] = dict(lens_out=torch.empty_like(st["lens"]), n_free_out=torch.empty_like(st["n_free"]))
        if not case["ended"]:
            st["out"].update(starts=_ints([0] * (n + 1)),
                             **{k: _ints([0]).repeat(st["max_tokens"]) for k in ("seq", "pos", "slot")})


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    if own:
        import routed_expert_layer_fp32_gb300 as moe
        st["moe"] = moe
    if case["op"] == "pages":
        _prepare_pages(case, st, g, seed)
        return st
    if case["op"] == "rope":
        st["x"] = _randn(g, case["tokens"], case["heads"], case["dim"]).to(_TYPES[case["kind"]])
        st["pos"] = torch.randint(0, case["far"], (case["tokens"],), generator=g, device=_device()).int()
        _rope_of(st, case)
        if own:
            st["out"] = torch.empty_like(st["x"])
        return st
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "attn":
        lens = tops = _shape(case)
    else:
        seq, pos = _written(case)
        tops = [1] * case["batch"]
        for s, p in zip(seq, pos):
            tops[s] = max(tops[s], p + 1)
    st["table"], n_pages = _page_table(g, case, tops)
    st.update(_pools(g, case, n_pages))
    if case["op"] == "attn":
        # queries of a size that gives attention its usual mixture of broad and peaked rows; rows of the fused
        # projection's output, so the query rows lie (heads + 2 kv_heads) dim apart
        st["q"] = _randn(g, case["batch"], h + 2 * hk, d).bfloat16()[:, :h]
        st["lens"], st["scale"] = _ints(lens), 1.5 / math.sqrt(d)
    else:
        st["seq"], st["pos"] = _ints(seq), _ints(pos)
        new = _rows_like_a_projection(g, len(seq), h + 2 * hk, d).to(_TYPES[case["src"]])
        st["q"], st["k_new"], st["v_new"] = new[:, :h], new[:, h:h + hk], new[:, h + hk:]
        where = st["table"].long()[st["seq"].long(), st["pos"].long() // case["page"]]
        st["slot"] = (where * case["page"] + st["pos"].long() % case["page"]).int()
    if case["op"] == "place":
        _rope_of(st, case)
    if own:
        m = st["moe"]
        st["cache"] = m.KVCache(*[st.get(n) for n in ("k", "v", "k_exp", "v_exp", "k_scale", "v_scale")])
        st["ws"] = m.attn_workspace(st["cache"], h, case["batch"])
        if case["op"] == "attn":
            st["out"] = torch.empty(case["batch"], h, d, dtype=torch.bfloat16, device=_device())
            st["lse"] = torch.empty(case["batch"], h, device=_device()) if case["lse"] else None
        else:
            st["q_out"] = torch.empty(len(seq), h, d, dtype=torch.bfloat16, device=_device())
            st["k_out"], st["v_out"] = (torch.empty(len(seq), hk, d, dtype=torch.bfloat16, device=_device())
                                        for _ in range(2))
    return st


# ------------------------------------------------------------------- rows of few bits -------

def _power32(e):
    """2^e exactly, e in -126 .. 127, from its bits (pow and exp2 may be a rounding off on a GPU)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _scales(device):
    b = torch.arange(128, device=device)
    return (1 + (b % 8).float() / 8) * _power32(b // 8 - 12)


def _quantise4(x):
    """x [..., dim] fp32: whole numbers, their groups' scale bytes and the row's biased exponent: the least
    power of two that brings the row's largest magnitude to 105, then of each 16 elements the least scale that
    brings theirs to 7."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = e - 7 + (m > 105 / 128).to(e.dtype)
    e = torch.where(m == 0, torch.full_like(e, LOW4), e).clamp(LOW4, HIGH4)
    y = (x * _power32(-e)[..., None]).unflatten(-1, (-1, 16))
    scales = _scales(x.device)
    b = torch.searchsorted(7 * scales, y.abs().amax(-1).contiguous()).clamp(max=127)
    n = torch.round(y / scales[b][..., None]).clamp(-7, 7)
    return n.flatten(-2), b.to(torch.uint8), (e + BIAS).to(torch.uint8)


def _values4(n, b, e):
    unit = _scales(n.device)[b.long()] * _power32(e.int() - BIAS)[..., None]
    return (n.unflatten(-1, (-1, 16)) * unit[..., None]).flatten(-2)


def _packed(n):
    c = (n.int() + 8).unflatten(-1, (-1, 4))
    u = c[..., 0] | c[..., 1] << 4 | c[..., 2] << 8 | c[..., 3] << 12
    u = (u << 3 | u >> 13) & 0xFFFF
    return torch.stack([u & 255, u >> 8], -1).flatten(-2).to(torch.uint8)


def _unpacked(raw):
    u = raw[..., ::2].int() | raw[..., 1::2].int() << 8
    u = u >> 3 | (u & 7) << 13
    return torch.stack([u & 15, u >> 4 & 15, u >> 8 & 15, u >> 12], -1).flatten(-2).float() - 8


def _quantise8(x):
    """x [..., dim] as E4M3 codes and a biased exponent: the least power of two that brings the row's largest
    magnitude to 448."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = e - 9 + (m > 0.875).to(e.dtype)
    e = torch.where(m == 0, torch.full_like(e, -BIAS), e).clamp(min=-BIAS)
    return (x * _power32(-e)[..., None]).to(torch.float8_e4m3fn), (e + BIAS).to(torch.uint8)


# --------------------------------------------------------------------------- the passes -----

def run(st):
    case = st["case"]
    return {"pages": _run_pages, "rope": _run_rope, "place": _run_place, "write": _run_write, "attn": _run_attn}[
        case["op"]](st, case)


def _run_pages(st, case):
    if own and case["ended"]:
        return st["moe"].page_release(st["lens"], st["ended"], st["table"], st["free"], st["n_free"], case["page"],
                                      st["ws"], **st["out"]) + (st["free"],)
    if own:
        plan = st["moe"].page_plan(st["lens"], st["new"], st["table"], st["free"], st["n_free"], case["page"],
                                   st["n_pages"], st["max_tokens"], st["ws"], **st["out"])
        return tuple(plan) + (st["table"],)
    lens, table, page, free = st["lens"].long(), st["table"], case["page"], st["free"]
    room, n_free, column = table.shape[1] * page, st["n_free"].long(), torch.arange(table.shape[1], device=table.device)
    held = torch.div(lens + page - 1, page, rounding_mode="floor")
    if case["ended"]:
        back = torch.where(st["ended"], held, torch.zeros_like(held))
        at = (n_free + torch.cumsum(back, 0) - back)[:, None] + column
        mine = column < back[:, None]
        free[at[mine]] = table[mine]
        lens_out = torch.where(st["ended"], torch.zeros_like(lens), lens)
        return lens_out.int(), (n_free + back.sum()).int(), free
    new, most = st["new"].long(), st["max_tokens"]
    ends = torch.cumsum(new, 0)
    fits = (lens + new <= room) & (ends <= most)
    need = torch.where(fits, torch.div(lens + new + page - 1, page, rounding_mode="floor") - held, torch.zeros_like(held))
    upto = torch.cumsum(need, 0)
    served = fits & ((need == 0) | (upto <= n_free))
    got = torch.where(served, need, torch.zeros_like(need))
    nth = column - held[:, None]
    mine = (nth >= 0) & (nth < got[:, None])
    at = n_free - 1 - (upto - need)[:, None] - nth
    table[mine] = free[at[mine]]
    t = torch.arange(most, device=table.device)
    seq = torch.searchsorted(ends, t, right=True)
    behind = seq == len(lens)
    b = seq.clamp(max=len(lens) - 1)
    pos = lens[b] + t - (ends - new)[b]
    ok = served[b] & ~behind
    pos = torch.where(ok, pos, torch.full_like(pos, -1))
    there = pos.clamp(min=0)
    slot = table[b, torch.div(there, page, rounding_mode="floor")].long() * page + torch.remainder(there, page)
    slot = torch.where(ok, slot, torch.full_like(slot, -1))
    starts = torch.cat([torch.zeros_like(ends[:1]), ends]).clamp(max=most)
    return (torch.where(behind, torch.full_like(seq, -1), seq).int(), pos.int(), slot.int(), starts.int(),
            (lens + torch.where(served, new, torch.zeros_like(new))).int(), (n_free - got.sum()).int(), table)


def _angles(st, pos):
    """Cosine and sine of each token's pairs, fp32 from an angle in 64 bits: far positions lose it in 32."""
    a = pos.double()[:, None] * st["freq"]
    return (torch.cos(a) * st["magnitude"]).float()[:, None], (torch.sin(a) * st["magnitude"]).float()[:, None]


def _rotated(x, angles, case):
    """x [tokens, heads, dim] in fp32 with its first `rot` elements turned pair by pair."""
    c, s = angles
    x, rot = x.float(), case["rot"]
    if case["layout"] == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        return torch.cat([a * c - b * s, b * c + a * s, x[..., rot:]], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), x[..., rot:]], -1)


def _run_rope(st, case):
    if own:
        return st["moe"].rope(st["x"], st["rope"], st["pos"], out=st["out"])
    return _rotated(st["x"], _angles(st, st["pos"]), case).to(_TYPES[case["kind"]])


def _stored(st, case, name, x, pages, rows):
    """x in the cache, and what the cache then says x is."""
    if case["cache"] == "bf16":
        st[name][pages, :, rows] = x.bfloat16()
        return st[name]
    if case["cache"] == "e4m3":
        codes, exps = _quantise8(x)
        st[name][pages, :, rows], st[name + "_exp"][pages, :, rows] = codes.view(torch.uint8), exps
        # 2^(exps - 127) in two steps: the least is below the normal numbers
        return (codes.float() * _power32(exps.int() - BIAS + 1)[..., None] * 0.5).bfloat16()
    n, b, e = _quantise4(x)
    st[name][pages, :, rows], st[name + "_exp"][pages, :, rows] = _packed(n), e
    st[name + "_scale"][pages, :, rows, : b.shape[-1]] = b
    return _values4(n, b, e).bfloat16()


def _where(st):
    slot, page = st["slot"].long(), st["case"]["page"]
    return torch.div(slot, page, rounding_mode="floor"), torch.remainder(slot, page)


def _run_place(st, case):
    if own:
        q = st["moe"].rope_kv_write(st["q"], st["k_new"], st["v_new"], st["cache"], st["rope"], st["pos"], st["slot"],
                                    st["ws"], q_out=st["q_out"])
        if case["cache"] == "bf16":
            return q, st["k"], st["v"]
        return (q,) + st["moe"].kv_read(st["cache"], st["pos"], st["table"], st["ws"], seq=st["seq"], k=st["k_out"],
                                        v=st["v_out"])
    angles, where = _angles(st, st["pos"]), _where(st)
    return (_rotated(st["q"], angles, case).bfloat16(),
            _stored(st, case, "k", _rotated(st["k_new"], angles, case), *where),
            _stored(st, case, "v", st["v_new"].float(), *where))


def _run_write(st, case):
    if own:
        st["moe"].kv_write(st["k_new"], st["v_new"], st["cache"], st["pos"], st["table"], st["ws"], seq=st["seq"])
        return st["moe"].kv_read(st["cache"], st["pos"], st["table"], st["ws"], seq=st["seq"], k=st["k_out"],
                                 v=st["v_out"])
    return tuple(_stored(st, case, n, st[n + "_new"].float(), *_where(st)) for n in ("k", "v"))


def _run_attn(st, case):
    if own:
        out = st["moe"].attn_decode(st["q"], st["cache"], st["lens"], st["table"], st["ws"], scale=st["scale"],
                                    window=case["window"], out=st["out"], lse=st["lse"])
        return (out, st["lse"]) if case["lse"] else out
    b, h, hk, d = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    lens = st["lens"].long()
    room = st["table"].shape[1] * case["page"]
    if case["window"]:
        first = (lens - case["window"]).clamp(min=0)
        pos = first[:, None] + torch.arange(min(case["window"], room), device=lens.device)
    else:
        pos = torch.arange(room, device=lens.device).expand(b, room)
    seen = pos < lens[:, None]
    at = pos.clamp(max=room - 1)
    pages = torch.gather(st["table"].long(), 1, at // case["page"])
    rows = at % case["page"]
    k, v = (_values4(_unpacked(st[n][pages, :, rows]), st[n + "_scale"][pages, :, rows][..., : d // 16],
                     st[n + "_exp"][pages, :, rows]) for n in ("k", "v"))              # [b, n, hk, d] fp32
    v = torch.where(seen[:, :, None, None], v, torch.zeros((), device=v.device))
    q = st["q"].float().view(b, hk, h // hk, d)
    s = torch.einsum("bkgd,bnkd->bkgn", q, k) * st["scale"]
    s = torch.where(seen[:, None, None, :], s, torch.full((), -math.inf, device=s.device))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("bkgn,bnkd->bkgd", p, v) / torch.where(total > 0, total, torch.ones_like(total))
    out = out.reshape(b, h, d).bfloat16()
    return (out, (top + torch.log(total)).view(b, h)) if case["lse"] else out


# -------------------------------------------------------------------- the definitions -------

def exact(case, seed):
    """The definitions, in 64 bits, sequence by sequence or row by row; whole numbers have none."""
    if case["op"] == "pages":
        return None
    st = prepare(case, seed)
    return {"rope": _exact_rope, "place": _exact_place, "write": _exact_write, "attn": _exact_attn}[case["op"]](st, case)


def _power64(e):
    return torch.bitwise_left_shift(e.long() + 1023, 52).view(torch.float64)


def _turned64(x, pos, st, case):
    """Pairs as complex numbers, turned by multiplication."""
    x, half = x.double(), case["rot"] // 2
    angle = torch.outer(pos.double(), st["freq"]).unsqueeze(1)
    turn = torch.polar(torch.full_like(angle, st["magnitude"]), angle)
    first, second = (slice(0, half), slice(half, 2 * half)) if case["layout"] == "half" else (
        slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    z = torch.complex(x[..., first], x[..., second]) * turn
    out = x.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_rope(st, case):
    return _turned64(st["x"], st["pos"], st, case)


def _least_power(top, unit, low, high):
    """The least whole e in low .. high with top <= unit 2^e."""
    e = torch.ceil(torch.log2(top / unit)).clamp(low, high).long()     # -inf for a row of zeros
    # log2 may be a rounding off where top is unit times a power of two, or next to it
    e = torch.where((top > unit * _power64(e)) & (e < high), e + 1, e)
    return torch.where((top <= unit * _power64(e - 1)) & (e > low), e - 1, e)


def _rounded_e4m3(x):
    """x (64 bits, at most 448 in magnitude) at the nearest E4M3 value, ties to the even one: steps of 2^-3 of
    the value's power of two, and of 2^-9 below 2^-6."""
    power = (x.abs().clamp(min=2.0 ** -6).view(torch.int64) >> 52) - 1023
    step = _power64(power - 3)
    return torch.round(x / step) * step


def _kept64(x, kind):
    """What a cache row of x holds."""
    if kind == "bf16":
        return x
    top = x.abs().amax(-1)
    if kind == "e4m3":
        unit = _power64(_least_power(top, E4M3_MAX, -BIAS, 127))[..., None]
        return _rounded_e4m3(x / unit) * unit
    unit = _power64(_least_power(top, 105.0, LOW4, HIGH4))[..., None]
    y = (x / unit).unflatten(-1, (-1, 16))
    top = y.abs().amax(-1) / 7
    # the least of the scales that is not below top: their steps are an eighth of their power of two
    power = _power64(((top.clamp(min=2.0 ** -12).view(torch.int64) >> 52) - 1023).clamp(max=3))
    eighths = torch.ceil(top.clamp(min=2.0 ** -12) / power * 8)
    eighths = torch.where(7 * (eighths - 1) / 8 * power >= y.abs().amax(-1), eighths - 1, eighths)   # top is rounded
    s = (eighths.clamp(min=8) / 8 * power).clamp(max=15.0)[..., None]
    n = torch.round(y / s).clamp(-7, 7)
    return (n * s).flatten(-2) * unit


def _exact_place(st, case):
    q = _turned64(st["q"], st["pos"], st, case)
    return (q,) + _exact_rows(st, case, _turned64(st["k_new"], st["pos"], st, case))


def _exact_write(st, case):
    return _exact_rows(st, case, st["k_new"].double())


def _exact_rows(st, case, k):
    rows = _kept64(k, case["cache"]), _kept64(st["v_new"].double(), case["cache"])
    if case["cache"] != "bf16":
        return rows
    pools = []
    for name, x in zip(("k", "v"), rows):
        pool = st[name].double().permute(0, 2, 1, 3).reshape(-1, case["kv_heads"], case["dim"])
        pool[st["slot"].long()] = x
        pools.append(pool.view(-1, case["page"], case["kv_heads"], case["dim"]).permute(0, 2, 1, 3))
    return tuple(pools)


def _cached64(st, name, page, row):
    """The values of all kv heads at one list of (page, row): [n, kv_heads, dim] in 64 bits."""
    raw, scale, exps = (st[name + part].transpose(1, 2)[page, row] for part in ("", "_scale", "_exp"))
    unit = raw.contiguous().view(torch.int16).long() & 0xFFFF
    unit = (unit * 8192 + torch.div(unit, 8, rounding_mode="floor")) % 65536        # turned back
    n = torch.stack([torch.div(unit, 16 ** i, rounding_mode="floor") % 16 for i in range(4)], -1).flatten(-2).double() - 8
    b = scale[..., : st["case"]["dim"] // 16].long()
    s = (8 + b % 8).double() * _power64(torch.div(b, 8, rounding_mode="floor") - 15)
    return n * s.repeat_interleave(16, -1) * _power64(exps.long() - BIAS).unsqueeze(-1)


def _exact_attn(st, case):
    h, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    out = torch.zeros(case["batch"], h, d, dtype=torch.float64, device=st["q"].device)
    lse = torch.full((case["batch"], h), -math.inf, dtype=torch.float64, device=st["q"].device)
    for i, n in enumerate(_shape(case)):
        lo = max(0, n - case["window"]) if case["window"] else 0
        if n == lo:
            continue
        p = torch.arange(lo, n, device=out.device)
        where = st["table"][i].long()[torch.div(p, page, rounding_mode="floor")], torch.remainder(p, page)
        k, v = _cached64(st, "k", *where), _cached64(st, "v", *where)
        for head in range(hk):
            mine = slice(head * (h // hk), (head + 1) * (h // hk))
            logits = (st["q"][i, mine].double() @ k[:, head].T) * st["scale"]
            lse[i, mine] = torch.logsumexp(logits, 1)
            out[i, mine] = torch.softmax(logits, 1) @ v[:, head]
    return (out, lse) if case["lse"] else out
