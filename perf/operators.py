"""What is measured of the operators around the expert layer: writing keys and values into a
paged cache (as they are, or quantised), reading them back, the attention of one new token over
that cache, and the norms, gate and residual between two blocks.

`listed()` gives the cases, `draw(rng)` more of the same ranges, `prepare(case, seed)` what a
program has in hand before the call, `run(state)` one pass (the plain form in elementary torch
operations, or with `own` the library's calls), `exact(case, seed)` the definition in 64 bits and
`work(case)` the bytes and operations a pass cannot do without.

The cache: pages of `page` tokens, [n_pages, kv_heads, page, head_dim] for the keys and for the
values, bf16, or E4M3 codes with one power-of-two exponent (biased by 127, a byte) per token and
kv head.  Position p of sequence s is at row p % page of page page_table[s, p // page].
"""
import math
import random

import torch

own = False

BIAS = 127          # of the stored exponents
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------- cases ------

def listed():
    attn = dict(op="attn", heads=16, kv_heads=4, dim=128, page=16, cache="bf16", window=0, ragged=0, lse=False)
    write = dict(op="write", heads=16, kv_heads=4, dim=128, page=16, cache="bf16", src="bf16", ragged=0)
    read = dict(op="read", kv_heads=4, dim=128, page=16, cache="e4m3", dst="bf16", ragged=0)
    norm = dict(op="norm", d=2048, y="fp32", r="bf16", x="bf16", gate="none", post=True)
    return [
        # one user's next token in a sliding-window layer (513 tokens): the smallest call, all latency
        dict(attn, name="attn-window-1", batch=1, length=16384, window=513),
        # one user's next token in a full-context layer at 64k tokens: one row, a long axis to split
        dict(attn, name="attn-full-1x64k", batch=1, length=65536),
        # a small serving batch of mixed lengths over an 8-bit cache
        dict(attn, name="attn-ragged-32-e4m3", batch=32, length=4096, ragged=1, cache="e4m3"),
        # a loaded server: 64 users of up to 16k tokens, bf16 cache, larger pages; the largest
        dict(attn, name="attn-ragged-64x16k", batch=64, length=16384, ragged=2, page=64),
        # a large batch in the sliding-window layers, 8-bit cache
        dict(attn, name="attn-window-128-e4m3", batch=128, length=16384, ragged=3, window=513, cache="e4m3", page=64),
        # odd everything: 7 query heads a kv head, 80 wide, pages of 48, empty and one-token rows,
        # with the log-sum-exp that joins this with another part of the context
        dict(attn, name="attn-odd-9", batch=9, length=3001, ragged=4, heads=14, kv_heads=2, dim=80, page=48, lse=True),
        # a decode step's new keys and values, straight out of the fused projection
        dict(write, name="write-step-64", batch=64, length=1024, tokens=64),
        # prompts of mixed lengths written into an 8-bit cache, and read back for the prompt's attention
        dict(write, name="write-prompts-16k-e4m3", batch=8, length=4096, tokens=16384, ragged=5, cache="e4m3", page=64),
        # a cached prefix of one prompt read back
        dict(read, name="read-prefix-1x2k", batch=1, length=2048),
        # the cached prefixes of a batch read back
        dict(read, name="read-prefix-8x8k", batch=8, length=8192, ragged=6, page=64),
        # between two blocks of a decode step of one token: residual of the layer's fp32 output, next norm
        dict(norm, name="norm-1", tokens=1),
        # between two blocks of a 16k prompt, post-norm and a learned gate per channel
        dict(norm, name="norm-16k", tokens=16384, y="bf16", gate="channel"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "write", "read", "norm"])
    if op == "norm":
        d = 8 * rng.randint(16, 1024)
        t = _log_int(rng, 1, min(32768, 33554432 // d))
        return dict(op=op, d=d, tokens=t, y=rng.choice(["fp32", "bf16"]), r=rng.choice(["bf16", "bf16", "fp32"]),
                    x=rng.choice(["bf16", "bf16", "fp32"]), gate=rng.choice(["none", "channel", "token"]),
                    post=rng.random() < 0.7)
    dim = rng.choice([64, 80, 96, 112, 128, 128, 192, 256])
    kv_heads = rng.randint(1, 8)
    page = rng.choice([16, 32, 48, 64, 128, 256])
    cache = rng.choice(["bf16", "e4m3"])
    ragged = rng.randint(1, 1 << 20)
    per_token = kv_heads * dim
    if op == "attn":
        heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
        budget = min(1 << 18, (1 << 28) // per_token, (1 << 30) // (heads * dim))   # tokens of all sequences
        batch = _log_int(rng, 1, 192)
        length = _log_int(rng, 1, min(65536, max(1, budget // batch)))
        window = rng.choice([0, 0, 513, _log_int(rng, 1, 4096)])
        return dict(op=op, heads=heads, kv_heads=kv_heads, dim=dim, page=page, cache=cache, window=window,
                    ragged=ragged, batch=batch, length=length, lse=rng.random() < 0.3)
    budget = min(1 << 16, (1 << 25) // per_token)
    if op == "write":
        batch = _log_int(rng, 1, 64)
        tokens = max(batch, _log_int(rng, 1, min(16384, (1 << 23) // per_token)))
        length = min(8192, (budget + tokens) // batch + 1)
        return dict(op=op, heads=kv_heads * rng.choice([1, 2, 4, 8]), kv_heads=kv_heads, dim=dim, page=page,
                    cache=cache, src=rng.choice(["bf16", "bf16", "fp32"]), ragged=ragged, batch=batch,
                    length=max(length, -(-tokens // batch)), tokens=tokens)
    batch = _log_int(rng, 1, 64)
    return dict(op=op, kv_heads=kv_heads, dim=dim, page=page, cache=cache, dst=rng.choice(["bf16", "bf16", "fp32"]),
                ragged=ragged, batch=batch, length=_log_int(rng, 1, max(1, budget // batch)))


def _lens(case):
    """The sequences' lengths: all alike, or mixed (short ones common, as in serving; an empty slot
    and a first token among them once there is room)."""
    n, top = case["batch"], case["length"]
    if not case["ragged"]:
        return [top] * n
    rng = random.Random(case["ragged"])
    lens = [max(1, min(top, int(top * rng.random() ** 0.7 + 1))) for _ in range(n)]
    lens[rng.randrange(n)] = top
    if n >= 8 and case["op"] == "attn":
        a, b = rng.sample(range(n), 2)
        lens[a], lens[b] = 0, 1
    return lens


def _written(case):
    """(sequence, position) of every token a write case writes: the last ones of each sequence, their
    counts as even as the token count allows (one each in a decode step)."""
    lens, n = _lens(case), case["batch"]
    each = [case["tokens"] // n + (1 if s < case["tokens"] % n else 0) for s in range(n)]
    seq, pos = [], []
    for s in range(n):
        top = max(lens[s], each[s])
        seq += [s] * each[s]
        pos += list(range(top - each[s], top))
    return seq, pos


def _read(case):
    seq, pos = [], []
    for s, n in enumerate(_lens(case)):
        seq += [s] * n
        pos += list(range(n))
    return seq, pos


def _row_bytes(case):
    """Bytes of one token's key and value of one kv head in the cache."""
    return 2 * (case["dim"] + 1) if case["cache"] == "e4m3" else 4 * case["dim"]


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["tokens"] * case["d"]
        size = {"bf16": 2, "fp32": 4}
        gate = {"none": 0, "channel": size[case["y"]] * case["d"], "token": size[case["y"]] * n}[case["gate"]]
        return {"bytes": n * (size[case["y"]] + 2 * size[case["r"]] + size[case["x"]]) + gate
                + 4 * case["d"] * (2 if case["post"] else 1), "flops": n * (12 if case["post"] else 7)}
    if op == "attn":
        seen = [min(n, case["window"]) if case["window"] else n for n in _lens(case)]
        tokens, q = sum(seen), case["batch"] * case["heads"]
        return {"bytes": tokens * case["kv_heads"] * _row_bytes(case) + q * (4 * case["dim"] + (4 if case["lse"] else 0))
                + 4 * case["batch"] + 4 * sum(-(-n // case["page"]) for n in seen),
                "flops": 4 * tokens * case["heads"] * case["dim"]}
    if op == "write":
        rows = case["tokens"] * case["kv_heads"]
        read_back = rows * (_row_bytes(case) + 4 * case["dim"]) if case["cache"] == "e4m3" else 0
        return {"bytes": rows * (2 * case["dim"] * (2 if case["src"] == "bf16" else 4) + _row_bytes(case)) + read_back
                + 8 * case["tokens"], "flops": 4 * rows * case["dim"]}
    rows = sum(_lens(case)) * case["kv_heads"]
    return {"bytes": rows * (_row_bytes(case) + 2 * case["dim"] * (2 if case["dst"] == "bf16" else 4))
            + 8 * sum(_lens(case)), "flops": 2 * rows * case["dim"]}


# ------------------------------------------------------------------------------ inputs ------

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _gen(case, seed):
    g = torch.Generator(device=_device())
    g.manual_seed(seed * 1000003 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=_device())


def _rows_like_a_projection(g, rows, heads, dim):
    """Keys or values as a projection makes them: a spread that differs by channel, a few large
    channels, and token norms that vary."""
    x = _randn(g, rows, heads, dim)
    x *= torch.exp(0.4 * _randn(g, 1, heads, dim)) * torch.exp(0.2 * _randn(g, rows, 1, 1))
    return x


def _quantise(x):
    """x [..., dim] as E4M3 codes and a biased exponent: the smallest power of two that brings the
    row's largest magnitude to 448 at most (no rounding but that of the codes)."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = e - 9 + (m > 0.875).to(e.dtype)             # amax = m 2^e, 0.5 <= m < 1, and 448 = 0.875 * 2^9
    e = torch.where(m == 0, torch.full_like(e, -BIAS), e).clamp(min=-BIAS)
    codes = (x * _power32(-e)[..., None]).to(torch.float8_e4m3fn)
    return codes, (e + BIAS).to(torch.uint8)


def _power32(e):
    """2^e exactly, e in -126 .. 127, from its bits (pow and exp2 may be a rounding off on a GPU)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _values(codes, exps):
    # 2^(exps - 127) in two steps: the smallest is below the normal numbers
    return codes.float() * _power32(exps.int() - BIAS + 1)[..., None] * 0.5


def _pools(g, case, n_pages):
    shape = (n_pages * case["kv_heads"], case["page"], case["dim"])
    out = {}
    for name in ("k", "v"):
        x = _rows_like_a_projection(g, shape[0], shape[1], shape[2]).bfloat16()
        if case["cache"] == "e4m3":
            # by slices: a large pool's fp32 copies would not be small
            parts = [_quantise(p.float()) for p in x.split(max(1, (1 << 26) // (shape[1] * shape[2])))]
            codes = torch.cat([p[0].view(torch.uint8) for p in parts])
            out[name] = codes.view(n_pages, case["kv_heads"], case["page"], case["dim"])
            out[name + "_exp"] = torch.cat([p[1] for p in parts]).view(n_pages, case["kv_heads"], case["page"])
        else:
            out[name] = x.view(n_pages, case["kv_heads"], case["page"], case["dim"])
    return out


def _page_table(g, case, tops):
    """Pages handed out in no order, each sequence with room for its last position; a few pages
    belong to nobody."""
    width = max(1, max(-(-t // case["page"]) for t in tops))
    n_pages = case["batch"] * width + 3
    order = torch.randperm(n_pages, generator=g, device=_device())
    return order[: case["batch"] * width].view(case["batch"], width).int().contiguous(), n_pages


def prepare(case, seed):
    g, dev = _gen(case, seed), _device()
    st = {"case": case}
    if case["op"] == "norm":
        n, d = case["tokens"], case["d"]
        st["y"] = _randn(g, n, d).to(_TYPES[case["y"]])
        st["r"] = (3 * _randn(g, n, d)).to(_TYPES[case["r"]])
        st["w_pre"] = 1 + 0.1 * _randn(g, d)
        st["w_post"] = 1 + 0.1 * _randn(g, d) if case["post"] else None
        st["gate"] = {"none": lambda: None, "channel": lambda: (0.5 * _randn(g, d)).to(_TYPES[case["y"]]),
                      "token": lambda: torch.sigmoid(_randn(g, n, d)).to(_TYPES[case["y"]])}[case["gate"]]()
        st["alpha"], st["eps"] = 0.7, 1e-6
        if own:
            import routed_expert_layer_fp32_gb300 as moe
            st["moe"] = moe
            st["r_out"] = torch.empty_like(st["r"])
            st["x_out"] = torch.empty(n, d, dtype=_TYPES[case["x"]], device=dev)
        return st
    lens = _lens(case)
    if case["op"] == "write":
        seq, pos = _written(case)
        tops = [1] * case["batch"]
        for s, p in zip(seq, pos):
            tops[s] = max(tops[s], p + 1)
    elif case["op"] == "read":
        seq, pos = _read(case)
        tops = lens
    else:
        tops = lens
    st["table"], n_pages = _page_table(g, case, tops)
    st.update(_pools(g, case, n_pages))
    if case["op"] == "attn":
        # queries of a size that gives attention its usual mixture of broad and peaked rows; rows of
        # the fused projection's output, so the query rows lie (heads + 2 kv_heads) dim apart
        qkv = _randn(g, case["batch"], (case["heads"] + 2 * case["kv_heads"]) * case["dim"]).bfloat16()
        st["q"] = qkv[:, : case["heads"] * case["dim"]].view(case["batch"], case["heads"], case["dim"])
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        st["scale"] = 1.5 / math.sqrt(case["dim"])
    else:
        st["seq"] = torch.tensor(seq, dtype=torch.int32, device=dev)
        st["pos"] = torch.tensor(pos, dtype=torch.int32, device=dev)
    if case["op"] == "write":
        h, hk, d = case["heads"], case["kv_heads"], case["dim"]
        new = _rows_like_a_projection(g, len(seq), h + 2 * hk, d).to(_TYPES[case["src"]])
        st["k_new"], st["v_new"] = new[:, h:h + hk], new[:, h + hk:]
    if own:
        import routed_expert_layer_fp32_gb300 as moe
        st["moe"] = moe
        st["cache"] = moe.KVCache(st["k"], st["v"], st.get("k_exp"), st.get("v_exp"))
        st["ws"] = moe.attn_workspace(st["cache"], case.get("heads", case["kv_heads"]), case["batch"])
        if case["op"] == "attn":
            st["out"] = torch.empty(case["batch"], case["heads"], case["dim"], dtype=torch.bfloat16, device=dev)
            st["lse"] = torch.empty(case["batch"], case["heads"], device=dev) if case["lse"] else None
        elif case["op"] == "read" or case["cache"] == "e4m3":
            kind = _TYPES[case.get("dst", "bf16")]
            st["k_out"] = torch.empty(len(seq), case["kv_heads"], case["dim"], dtype=kind, device=dev)
            st["v_out"] = torch.empty_like(st["k_out"])
    return st


# --------------------------------------------------------------------------- the passes -----

def run(st):
    case = st["case"]
    return {"attn": _run_attn, "write": _run_write, "read": _run_read, "norm": _run_norm}[case["op"]](st, case)


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
    k, v = _gathered(st, "k", pages, rows), _gathered(st, "v", pages, rows)      # [b, n, hk, d] fp32
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


def _gathered(st, name, pages, rows):
    """fp32 values at (page, row) of every kv head, heads before the width."""
    if st["case"]["cache"] == "e4m3":
        return _values(st[name][pages, :, rows].view(torch.float8_e4m3fn), st[name + "_exp"][pages, :, rows])
    return st[name][pages, :, rows].float()


def _where(st):
    pages = st["table"].long()[st["seq"].long(), st["pos"].long() // st["case"]["page"]]
    return pages, st["pos"].long() % st["case"]["page"]


def _run_write(st, case):
    if own:
        st["moe"].kv_write(st["k_new"], st["v_new"], st["cache"], st["pos"], st["table"], st["ws"], seq=st["seq"])
        if case["cache"] == "bf16":
            return st["k"], st["v"]
        st["moe"].kv_read(st["cache"], st["pos"], st["table"], st["ws"], seq=st["seq"], k=st["k_out"], v=st["v_out"])
        return st["k_out"], st["v_out"], st["k_exp"], st["v_exp"]
    pages, rows = _where(st)
    for name in ("k", "v"):
        x = st[name + "_new"].float()
        if case["cache"] == "bf16":
            st[name][pages, :, rows] = x.bfloat16()
        else:
            codes, exps = _quantise(x)
            st[name][pages, :, rows] = codes.view(torch.uint8)
            st[name + "_exp"][pages, :, rows] = exps
    if case["cache"] == "bf16":
        return st["k"], st["v"]
    return (_gathered(st, "k", pages, rows).bfloat16(), _gathered(st, "v", pages, rows).bfloat16(), st["k_exp"],
            st["v_exp"])


def _run_read(st, case):
    if own:
        return st["moe"].kv_read(st["cache"], st["pos"], st["table"], st["ws"], seq=st["seq"], k=st["k_out"],
                                 v=st["v_out"])
    pages, rows = _where(st)
    kind = _TYPES[case["dst"]]
    return _gathered(st, "k", pages, rows).to(kind), _gathered(st, "v", pages, rows).to(kind)


def _run_norm(st, case):
    if own:
        return st["moe"].block_norm(st["r"], st["w_pre"], y=st["y"], w_post=st["w_post"], gate=st["gate"],
                                    alpha=st["alpha"], eps=st["eps"], residual_out=st["r_out"], out=st["x_out"])
    z = st["y"].float()
    if st["w_post"] is not None:
        z = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + st["eps"]) * st["w_post"]
    if st["gate"] is not None:
        z = z * st["gate"].float()
    r = st["r"].float() + st["alpha"] * z
    x = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + st["eps"]) * st["w_pre"]
    return r.to(_TYPES[case["r"]]), x.to(_TYPES[case["x"]])


# -------------------------------------------------------------------- the definitions -------

def exact(case, seed):
    """The definitions, in 64 bits, sequence by sequence (or row by row of the written tokens)."""
    st = prepare(case, seed)
    return {"attn": _exact_attn, "write": _exact_write, "read": _exact_read, "norm": _exact_norm}[case["op"]](st, case)


def _cached64(st, name, page, row):
    """The values of all kv heads at one list of (page, row): [n, kv_heads, dim] in 64 bits."""
    raw = st[name].permute(0, 2, 1, 3)[page, row]
    if st["case"]["cache"] == "bf16":
        return raw.double()
    e = st[name + "_exp"].permute(0, 2, 1)[page, row].long() - BIAS
    return raw.view(torch.float8_e4m3fn).double() * _power64(e).unsqueeze(-1)


def _power64(e):
    return torch.bitwise_left_shift(e.long() + 1023, 52).view(torch.float64)


def _exact_attn(st, case):
    h, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    out = torch.zeros(case["batch"], h, d, dtype=torch.float64, device=st["q"].device)
    lse = torch.full((case["batch"], h), -math.inf, dtype=torch.float64, device=st["q"].device)
    for i, n in enumerate(_lens(case)):
        lo = max(0, n - case["window"]) if case["window"] else 0
        if n == lo:
            continue
        p = torch.arange(lo, n, device=out.device)
        where = st["table"][i].long()[torch.div(p, page, rounding_mode="floor")], torch.remainder(p, page)
        k, v = _cached64(st, "k", *where), _cached64(st, "v", *where)
        for head in range(h):
            kv = head // (h // hk)
            logits = (k[:, kv] @ st["q"][i, head].double()) * st["scale"]
            lse[i, head] = torch.logsumexp(logits, 0)
            out[i, head] = torch.softmax(logits, 0) @ v[:, kv]
    return (out, lse) if case["lse"] else out


def _rounded_e4m3(x):
    """x (64 bits, at most 448 in magnitude) at the nearest E4M3 value, ties to the even one: steps of
    2^-3 of the value's power of two, and of 2^-9 below 2^-6."""
    power = (x.abs().clamp(min=2.0 ** -6).view(torch.int64) >> 52) - 1023
    step = _power64(power - 3)
    return torch.round(x / step) * step


def _exact_write(st, case):
    page = torch.stack([st["table"][s, p // case["page"]] for s, p in zip(*_written(case))]).long()
    row = st["pos"].long() % case["page"]
    outs, exps = [], []
    for name in ("k", "v"):
        x = st[name + "_new"].double()
        if case["cache"] == "bf16":
            pool = st[name].double()
            pool[page, :, row] = x
            outs.append(pool)
            continue
        top = x.abs().amax(-1)
        e = torch.ceil(torch.log2(top / E4M3_MAX)).clamp(min=-BIAS).long()     # -inf for a row of zeros
        # log2 may be a rounding off where top is 448 times a power of two, or next to it
        e = torch.where(top > E4M3_MAX * _power64(e), e + 1, e)
        e = torch.where((top <= E4M3_MAX * _power64(e - 1)) & (e > -BIAS), e - 1, e)
        unit = _power64(e)[..., None]
        outs.append(_rounded_e4m3(x / unit) * unit)
        pool = st[name + "_exp"].clone()
        pool[page, :, row] = (e + BIAS).to(torch.uint8)
        exps.append(pool)
    return tuple(outs + exps)


def _exact_read(st, case):
    page = torch.cat([st["table"][s].long().repeat_interleave(case["page"])[:n] for s, n in enumerate(_lens(case))])
    row = torch.cat([torch.arange(n, device=page.device) % case["page"] for n in _lens(case)])
    return _cached64(st, "k", page, row), _cached64(st, "v", page, row)


def _exact_norm(st, case):
    def unit(t):
        return t / torch.sqrt(torch.linalg.vector_norm(t, dim=1, keepdim=True) ** 2 / t.shape[1] + st["eps"])
    z = st["y"].double()
    if case["post"]:
        z = unit(z) * st["w_post"].double()
    if case["gate"] != "none":
        z = z * st["gate"].double()
    total = torch.add(st["r"].double(), z, alpha=st["alpha"])
    return total, unit(total) * st["w_pre"].double()
