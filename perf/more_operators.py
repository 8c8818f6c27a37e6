"""Measured cases of the microscaled (MX) cache of keys and values: rotary
positions and the quantised write in one call, the values read back, and the
attention over the cache.

The cache is pages of ``page`` tokens: codes uint8 [pages, heads, page, D / 2]
(e2m1, two a byte) or [.., D] (e4m3) and a scale byte e (2^(e - 127)) for each
block of 32 channels, [pages, heads, page, D / 32], for keys and for values.  A
row of the block table names a sequence's pages in order.

``run`` computes an operator in its plain form (elementary torch operations)
or, where ``own`` is true, with the framework's calls, on the same state.
Codes are returned as the values they stand for, so a pass of the write is
the write and the reading back of what it wrote, in both forms.  ``exact``
gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

BLOCK = 32
EMAX = {"e2m1": 2, "e4m3": 8}
LARGEST = {"e2m1": 6.0, "e4m3": 448.0}
SMALLEST_EXP = {"e2m1": 0, "e4m3": -6}  # exponent of the smallest normal value
MANTISSA = {"e2m1": 1, "e4m3": 3}
DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
# bytes of an element in the cache, its share of the scale byte among them
CACHED = {"e2m1": 0.5 + 1 / BLOCK, "e4m3": 1 + 1 / BLOCK}
BASE = 500000.0


# ------------------------------------------------------------------ the cases

def listed():
    def write(name, tokens, seqs, heads, kv_heads, dim, dtype, fmt, page, layout, rotary, start,
              smooth):
        return {"name": name, "op": "write", "tokens": tokens, "seqs": seqs, "heads": heads,
                "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "fmt": fmt, "page": page,
                "layout": layout, "rotary": rotary, "start": start, "smooth": smooth}

    def read(name, shortest, longest, seqs, kv_heads, dim, dtype, fmt, page):
        return {"name": name, "op": "read", "shortest": shortest, "longest": longest,
                "seqs": seqs, "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "fmt": fmt,
                "page": page}

    def attention(name, seqs, new_least, new_most, shortest, longest, heads, kv_heads, dim, dtype,
                  fmt, page, window=0):
        return {"name": name, "op": "attention", "seqs": seqs, "new_least": new_least,
                "new_most": new_most, "shortest": shortest, "longest": longest, "heads": heads,
                "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "fmt": fmt, "page": page,
                "window": window}

    return [
        # one token of a serving loop, far into a long context: latency
        write("write_token", 1, 1, 64, 8, 128, "bf16", "e2m1", 16, "half", 128, 100001, False),
        # a ragged batch of short prompts, full heads of a 7168-wide layer, part
        # of each head rotated, keys and queries smoothed
        write("write_ragged", 333, 7, 56, 56, 128, "f16", "e4m3", 32, "interleaved", 64, 0, True),
        # a chunk of a long prompt, rotary frequencies scaled for its length
        write("write_chunk", 16384, 1, 64, 8, 128, "bf16", "e2m1", 64, "half", 128, 98304, False),
        # one short sequence handed to a consumer of plain values
        read("read_short", 515, 515, 1, 8, 128, "f16", "e4m3", 16),
        # a batch's cache read back for a copy elsewhere, lengths far apart
        read("read_batch", 700, 16000, 12, 8, 128, "bf16", "e2m1", 64),
        # one token of one user's chat: latency
        attention("decode_chat", 1, 1, 1, 2049, 2049, 64, 8, 128, "bf16", "e2m1", 16),
        # one token of one user, a long document
        attention("decode_long", 1, 1, 1, 131079, 131079, 64, 8, 128, "bf16", "e2m1", 64),
        # a serving batch, lengths far apart
        attention("decode_batch", 64, 1, 1, 130, 32768, 64, 8, 128, "bf16", "e2m1", 32),
        # full heads of a 7168-wide layer over a cache of 8 bits
        attention("decode_heads_e4m3", 16, 1, 1, 900, 2300, 56, 56, 128, "f16", "e4m3", 16),
        # drafted tokens checked, the hidden-1024 decoder's heads
        attention("drafts", 9, 5, 5, 200, 7001, 16, 8, 128, "f16", "e2m1", 16),
        # a whole prompt
        attention("prompt", 1, 8192, 8192, 8192, 8192, 64, 8, 128, "bf16", "e2m1", 64),
        # chunks of prompts of odd lengths over cached prefixes, small heads,
        # a sliding window
        attention("chunks_window", 5, 77, 1013, 1013, 9001, 32, 4, 64, "f16", "e2m1", 32, 1024),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attention", "attention", "attention"])
    heads, kv_heads, dim = rng.choice([(64, 8, 128), (56, 56, 128), (16, 8, 128), (32, 4, 64),
                                       (8, 4, 256), (10, 2, 64), (28, 4, 128), (16, 1, 256)])
    case = {"op": op, "dim": dim, "kv_heads": kv_heads, "fmt": rng.choice(["e2m1", "e4m3"]),
            "page": rng.choice([16, 32, 64, 128])}
    row = 8 * 128
    if op == "write":
        case.update(heads=heads, dtype=rng.choice(["f16", "bf16", "f32"]),
                    layout=rng.choice(["half", "interleaved"]),
                    rotary=rng.choice([0, 32, 64, dim]), start=_log_int(rng, 1, 120000) - 1,
                    smooth=rng.random() < 0.5)
        # (as many bytes as the largest listed write at the most)
        size = SIZE[case["dtype"]]
        most = 707000000 // (dim * (2 * heads * size + 4 * kv_heads * (size + 1) + kv_heads))
        case["tokens"] = _log_int(rng, 1, min(16384, most))
        case["seqs"] = _log_int(rng, 1, min(64, case["tokens"]))
        return case
    case["seqs"] = _log_int(rng, 1, 64)
    if op == "read":
        case["dtype"] = rng.choice(["f16", "bf16", "f32"])
        most = 49152 * row // (kv_heads * dim * SIZE[case["dtype"]] // 2) // case["seqs"]
        case["longest"] = _log_int(rng, 1, most)
        case["shortest"] = _log_int(rng, 1, case["longest"])
        return case
    case.update(heads=heads, dtype=rng.choice(["f16", "bf16"]))
    case["window"] = rng.choice([0, 0, _log_int(rng, 16, 8192)])
    kind = rng.choice(["token", "token", "drafts", "prompt"])
    if kind == "prompt":
        case["seqs"] = _log_int(rng, 1, 8)
        case["new_most"] = _log_int(rng, 33, 8192 // case["seqs"])
        case["new_least"] = _log_int(rng, 1, case["new_most"])
        most = min(32768, 8192 * 4096 // case["seqs"] // case["new_most"]
                   * 64 * 128 // (heads * dim))
    else:
        case["new_most"] = 1 if kind == "token" else rng.randint(2, 9)
        case["new_least"] = 1 if kind == "token" else rng.randint(1, case["new_most"])
        most = min(131072, 393216 * row // (kv_heads * dim * 2) // case["seqs"])
    case["longest"] = max(case["new_most"], _log_int(rng, 1, max(1, most)))
    # (a sequence is at least its new tokens)
    case["shortest"] = rng.randint(min(case["new_most"], case["longest"]), case["longest"])
    return case


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly over their logarithm, the short
    and the long ones mixed (by a step that shares no factor with n)."""
    if n == 1:
        return [hi]
    v = [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]
    step = next(k for k in range(n // 2 + 1, 2 * n) if math.gcd(k, n) == 1)
    return [v[i * step % n] for i in range(n)]


def _new(case):
    """New tokens of each sequence."""
    if case["op"] == "write":
        part, n = case["seqs"], case["tokens"]
        ends = [n * (i + 1) ** 2 // part ** 2 for i in range(part)]
        return [b - a for a, b in zip([0] + ends, ends)]
    return _spread(case["new_least"], case["new_most"], case["seqs"])


def _lengths(case):
    """Tokens that each sequence has in the cache."""
    if case["op"] == "write":
        return _new(case)
    lens = _spread(case["shortest"], case["longest"], case["seqs"])
    if case["op"] == "attention":
        lens = [max(a, b) for a, b in zip(lens, _new(case))]
    return lens


def _pairs(case):
    """(query tokens x keys that they see, keys that any of them sees)."""
    pairs = keys = 0
    for n, k in zip(_new(case), _lengths(case)):
        w = case["window"]
        first = k - n + 1  # keys that the first token has before it, itself among them
        if w == 0:
            pairs += n * first + n * (n - 1) // 2
            keys += k
        else:
            pairs += sum(min(w, first + i) for i in range(n))
            keys += min(k, n - 1 + w)
    return pairs, keys


def work(case):
    dim, kv, size = case["dim"], case["kv_heads"], SIZE[case["dtype"]]
    total = sum(_lengths(case))
    if case["op"] == "attention":
        pairs, keys = _pairs(case)
        rows = sum(_new(case)) * case["heads"] * dim
        return {"bytes": 2.0 * rows * size + 2.0 * keys * kv * dim * CACHED[case["fmt"]],
                "flops": 4.0 * pairs * case["heads"] * dim}
    held = total * kv * dim
    back = 2.0 * held * (CACHED[case["fmt"]] + size)  # codes read, values written
    if case["op"] == "read":
        return {"bytes": back, "flops": 2.0 * held}
    q = total * case["heads"] * dim
    rotated = total * (case["heads"] + kv) * case["rotary"]
    return {"bytes": back + 2.0 * q * size + 2.0 * held * (size + CACHED[case["fmt"]]),
            "flops": 3.0 * rotated + 8.0 * held}


# --------------------------------------------------------------------- inputs

def _frequencies(rotary, start):
    """Rotary frequencies; for a far start interpolated by parts: the slow
    ones divided by the stretch, the fast ones kept, a ramp between."""
    half = rotary // 2
    out = []
    for i in range(half):
        f = BASE ** (-2.0 * i / rotary)
        if start >= 8192:
            turns = 8192 * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - 1.0) / (32.0 - 1.0)))
            f = f * keep + f / 16.0 * (1.0 - keep)
        out.append(f)
    return out


def _amplitude(start):
    return 0.1 * math.log(16.0) + 1.0 if start >= 8192 else 1.0


def _table(g, lens, page):
    """A block table whose pages lie in no order, and the number of pages."""
    need = [max(1, -(-n // page)) for n in lens]
    pages = sum(need)
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, pages


def _prefix(lens):
    return torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)


def _filled(g, pages, case):
    """Codes and scales of a cache that a model has written: keys with a few
    channels many times as large, values without."""
    heads, page, dim, fmt = case["kv_heads"], case["page"], case["dim"], case["fmt"]
    gain = torch.ones(heads, 1, dim, device="cuda")
    hot = torch.randperm(heads * dim, generator=g, device="cuda")[:max(1, heads * dim // 64)]
    gain.view(-1)[hot] = 4 + 8 * torch.rand(hot.numel(), generator=g, device="cuda")
    step = max(1, (1 << 25) // (heads * page * dim))
    parts = []
    for i in range(0, pages, step):
        shape = (min(step, pages - i), heads, page, dim)
        k = torch.randn(shape, generator=g, device="cuda") * gain
        v = torch.randn(shape, generator=g, device="cuda")
        parts.append(_codes(k, fmt) + _codes(v, fmt))
    return tuple(torch.cat([p[i] for p in parts]) for i in range(4)), gain


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000 + 29)
    heads, dim, page, dtype = case["kv_heads"], case["dim"], case["page"], DTYPE[case["dtype"]]
    lens, s = _lengths(case), dict(case)
    s["lens"] = lens
    s["table"], pages = _table(g, lens, page)
    s["cu"] = _prefix(lens)
    if case["op"] == "read":
        s["cache"], _ = _filled(g, pages, case)
        return s
    if case["op"] == "attention":
        s["cache"], gain = _filled(g, pages, case)
        s["new"] = _new(case)
        s["cu_q"] = _prefix(s["new"])
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        # queries a little larger than the keys' norm asks for, so that each
        # looks at some keys more than at others
        q = torch.randn(sum(s["new"]), case["heads"], dim, generator=g, device="cuda")
        group = case["heads"] // heads
        q = q / gain[:, 0].repeat_interleave(group, 0) * 2.0
        s["q"] = q.to(dtype)
        return s
    tokens, q_heads = sum(lens), case["heads"]
    # q | k | v as the layer's product leaves them: one row a token
    qkv = torch.randn(tokens, q_heads + 2 * heads, dim, generator=g, device="cuda").to(dtype)
    s["q"], s["k"], s["v"] = qkv[:, :q_heads], qkv[:, q_heads:q_heads + heads], qkv[:, q_heads + heads:]
    where = torch.cat([torch.arange(n, device="cuda") for n in lens])
    s["positions"] = where + case["start"]
    row = torch.cat([s["table"][b, torch.arange(n, device="cuda") // page] for b, n in enumerate(lens)])
    s["slots"] = row.to(torch.int64) * page + where % page
    size = dim // 2 if case["fmt"] == "e2m1" else dim
    s["cache"] = tuple(torch.zeros(pages, heads, page, n, dtype=torch.uint8, device="cuda")
                       for n in (size, dim // BLOCK) * 2)
    s["inv_freq"], s["amplitude"] = None, 1.0
    if case["rotary"]:
        s["inv_freq"] = torch.tensor(_frequencies(case["rotary"], case["start"]),
                                     dtype=torch.float64, device="cuda")
        s["amplitude"] = _amplitude(case["start"])
    s["k_mul"] = s["q_mul"] = None
    if case["smooth"]:
        # the keys' large channels divided, the queries' multiplied
        f = torch.exp(0.5 * torch.randn(heads, dim, generator=g, device="cuda"))
        s["k_mul"], s["q_mul"] = 1.0 / f, f.repeat_interleave(q_heads // heads, 0).contiguous()
    return s


# ------------------------------------------------------------ the plain forms

def _power(e):
    """2^(e - 127) of scale bytes, in fp32."""
    return ((e.to(torch.int64) + 896) << 52).view(torch.float64).to(torch.float32)


def _codes(v, fmt):
    """(codes, scale bytes) of fp32 values [..., D] in blocks of 32."""
    shape = v.shape
    v = v.reshape(-1, BLOCK)
    e = ((v.abs().amax(dim=1).view(torch.int32) >> 23) - EMAX[fmt]).clamp(min=0)
    z = v * ((254 - e) << 23).view(torch.float32).unsqueeze(1)
    # the nearest values of the format, ties to even, beyond the largest to it
    # (powers of two by their bits: every product here is exact)
    power = z.abs().clamp(min=2.0 ** SMALLEST_EXP[fmt]).view(torch.int32) & 0x7F800000
    steps = ((254 << 23) - power).view(torch.float32) * 2.0 ** MANTISSA[fmt]
    q = torch.round(z * steps) * (power.view(torch.float32) * 2.0 ** -MANTISSA[fmt])
    q = q.clamp(-LARGEST[fmt], LARGEST[fmt])
    e = e.to(torch.uint8).reshape(*shape[:-1], shape[-1] // BLOCK)
    if fmt == "e4m3":
        return q.to(torch.float8_e4m3fn).view(torch.uint8).reshape(shape), e
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=v.device)
    c = (torch.searchsorted(grid, q.abs()) + 8 * (q < 0)).to(torch.uint8)
    return (c[:, 0::2] + 16 * c[:, 1::2]).reshape(*shape[:-1], shape[-1] // 2), e


def _values(q, e, fmt):
    """The fp32 values [..., D] of codes and scale bytes."""
    if fmt == "e2m1":
        grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
        grid = torch.cat([grid, -grid])
        pairs = torch.stack([grid.repeat(16), grid.repeat_interleave(16)], dim=1)
        v = pairs[q.to(torch.int32)]
    else:
        v = q.view(torch.float8_e4m3fn).to(torch.float32)
    v = v.reshape(*e.shape, BLOCK) * _power(e).unsqueeze(-1)
    return v.reshape(*e.shape[:-1], -1)


def _sequence(s, b, which):
    """Keys (0) or values (2) of sequence b, fp32 [tokens, heads, D]."""
    pages = s["table"][b, :max(1, -(-s["lens"][b] // s["page"]))].to(torch.int64)
    v = _values(s["cache"][which][pages], s["cache"][which + 1][pages], s["fmt"])
    v = v.transpose(1, 2).reshape(-1, s["kv_heads"], s["dim"])
    return v[:s["lens"][b]]


def _read(s):
    dtype = DTYPE[s["dtype"]]
    return tuple(torch.cat([_sequence(s, b, which).to(dtype) for b in range(len(s["lens"]))])
                 for which in (0, 2))


def _rotated(s, x):
    x = x.to(torch.float32)
    r = s["rotary"]
    if r == 0:
        return x
    angle = s["positions"].to(torch.float64).unsqueeze(1) * s["inv_freq"]
    c = (torch.cos(angle) * s["amplitude"]).to(torch.float32).unsqueeze(1)
    d = (torch.sin(angle) * s["amplitude"]).to(torch.float32).unsqueeze(1)
    if s["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * c - b * d, b * c + a * d], dim=-1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * c - b * d, b * c + a * d], dim=-1).flatten(-2)
    return torch.cat([y, x[..., r:]], dim=-1)


def _write(s):
    q, k = _rotated(s, s["q"]), _rotated(s, s["k"])
    if s["smooth"]:
        q, k = q * s["q_mul"], k * s["k_mul"]
    page, at = s["slots"] // s["page"], s["slots"] % s["page"]
    new = _codes(k, s["fmt"]) + _codes(s["v"].to(torch.float32), s["fmt"])
    for held, rows in zip(s["cache"], new):
        held[page, :, at] = rows
    return (q.to(DTYPE[s["dtype"]]),) + _read(s)


def _attention(s):
    dtype, heads, kv, dim = DTYPE[s["dtype"]], s["heads"], s["kv_heads"], s["dim"]
    group, out, at = heads // kv, [], 0
    for b, (n, length) in enumerate(zip(s["new"], s["lens"])):
        k, v = _sequence(s, b, 0), _sequence(s, b, 2)
        q = s["q"][at:at + n].to(torch.float32)
        at += n
        y = torch.empty(n, heads, dim, device=q.device)
        # (so many tokens at a time that the scores stay within 2 GB)
        step = max(1, (1 << 29) // (group * length))
        for i in range(0, n, step):
            m = min(step, n - i)
            last = length - n + i + torch.arange(m, device=q.device).unsqueeze(1)
            j = torch.arange(length, device=q.device).unsqueeze(0)
            hidden = j > last
            if s["window"]:
                hidden = hidden | (j <= last - s["window"])
            for h in range(kv):
                rows = q[i:i + m, h * group:(h + 1) * group].transpose(0, 1).reshape(-1, dim)
                score = torch.matmul(rows, k[:, h].t().contiguous()) * dim ** -0.5
                score = score.view(group, m, length).masked_fill_(hidden, -math.inf)
                p = torch.exp(score - score.amax(dim=2, keepdim=True))
                o = torch.matmul(p.view(-1, length), v[:, h].contiguous()).view(group, m, dim)
                o = o / p.sum(dim=2, keepdim=True)
                y[i:i + m, h * group:(h + 1) * group] = o.transpose(0, 1)
        out.append(y.to(dtype))
    return torch.cat(out)


def run(state):
    if own:
        return _run_own(state)
    return {"write": _write, "read": _read, "attention": _attention}[state["op"]](state)


def _run_own(s):
    import w8a8_post_quantization_amd as sq

    fmt = sq.SQ_MX_E2M1 if s["fmt"] == "e2m1" else sq.SQ_MX_E4M3
    if s["op"] == "attention":
        one = s["new_most"] == 1
        return sq.attention_kv_mx(s["q"], s["cache"], s["table"], s["seq_lens"],
                                  None if one else s["cu_q"], fmt=fmt, max_q=s["new_most"],
                                  window=s["window"])
    total = sum(s["lens"])
    if s["op"] == "read":
        return sq.dequantize_kv_mx(s["cache"], s["table"], s["cu"], total, fmt=fmt,
                                   out_dtype=DTYPE[s["dtype"]])
    layout = sq.SQ_ROPE_HALF if s["layout"] == "half" else sq.SQ_ROPE_INTERLEAVED
    q = sq.rope_quantize_kv_mx(s["q"], s["k"], s["v"], s["slots"], s["cache"], fmt=fmt,
                               positions=s["positions"], inv_freq=s["inv_freq"],
                               amplitude=s["amplitude"], layout=layout, q_mul=s["q_mul"],
                               k_mul=s["k_mul"])
    k, v = sq.dequantize_kv_mx(s["cache"], s["table"], s["cu"], total, fmt=fmt,
                               out_dtype=DTYPE[s["dtype"]])
    return q, k, v


# -------------------------------------------------------- the values, 64 bits

def _fl(v):
    """A 64-bit result rounded to fp32, where the definition rounds."""
    return v.to(torch.float32).to(torch.float64)


def _two_to(e):
    """2^e in fp64, by its bits (a library power may be off by a rounding)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _grid(fmt, device):
    if fmt == "e2m1":
        v = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    else:
        v = [m * 2.0 ** -9 for m in range(8)]
        v += [(8 + m) * 2.0 ** (x - 10) for x in range(1, 16) for m in range(8)][:-1]
    return torch.tensor(v, dtype=torch.float64, device=device)


def _exact_blocks(v, fmt):
    """The values that fp32-valued rows have once quantised, by frexp and the
    midpoints of the format's values."""
    grid = _grid(fmt, v.device)
    mid = (grid[1:] + grid[:-1]) / 2
    out = torch.empty_like(v)
    step = max(1, (1 << 24) // v[0].numel())
    for i in range(0, v.shape[0], step):
        part = v[i:i + step].reshape(-1, BLOCK)
        top = part.abs().amax(dim=1, keepdim=True)
        p = torch.frexp(top).exponent  # largest in [2^(p - 1), 2^p)
        e = torch.where(top > 0, p - 1 - EMAX[fmt], torch.full_like(p, -127)).clamp(min=-127)
        z = (part * _two_to(-e)).abs()
        below = torch.bucketize(z, mid, right=False)  # midpoints under z
        through = torch.bucketize(z, mid, right=True)  # midpoints up to z
        pick = torch.where((below != through) & (through % 2 == 0), through, below)
        out[i:i + step] = (grid[pick] * torch.sign(part) * _two_to(e)).view_as(out[i:i + step])
    return out


def _exact_codes(q, e, fmt):
    """fp64 values of one head's codes and scale bytes [tokens, ..]."""
    grid = _grid(fmt, q.device)
    if fmt == "e2m1":
        c = torch.stack([q & 15, q >> 4], dim=-1).flatten(-2).to(torch.int64)
        v = grid[c & 7] * (1 - 2 * (c >> 3))
    else:
        c = q.to(torch.int64)
        v = grid[c & 127] * (1 - 2 * (c >> 7))
    return v * _two_to(e.to(torch.int64) - 127).repeat_interleave(BLOCK, dim=-1)


def _exact_head(s, b, h, which):
    n = torch.arange(s["lens"][b], device="cuda")
    page = s["table"][b].to(torch.int64)[n // s["page"]]
    at = n % s["page"]
    return _exact_codes(s["cache"][which][page, h, at], s["cache"][which + 1][page, h, at], s["fmt"])


def _exact_attention(s, case):
    heads, kv, dim = case["heads"], case["kv_heads"], case["dim"]
    group = heads // kv
    y = torch.zeros(sum(s["new"]), heads, dim, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, length) in enumerate(zip(s["new"], s["lens"])):
        for h in range(kv):
            k, v = _exact_head(s, b, h, 0), _exact_head(s, b, h, 2)
            step = max(1, (1 << 27) // length)
            for head in range(h * group, (h + 1) * group):
                for i in range(0, n, step):
                    rows = s["q"][at + i:at + min(n, i + step), head].to(torch.float64)
                    pos = torch.arange(i, i + rows.shape[0], device="cuda") + (length - n)
                    gap = pos.unsqueeze(1) - torch.arange(length, device="cuda").unsqueeze(0)
                    seen = gap >= 0
                    if case["window"]:
                        seen = seen & (gap < case["window"])
                    score = torch.where(seen, rows @ k.t() / math.sqrt(dim), -math.inf)
                    y[at + i:at + i + rows.shape[0], head] = torch.softmax(score, dim=1) @ v
        at += n
    return y


def _exact_rotated(s, case, x):
    x, r = x.to(torch.float64), case["rotary"]
    if r == 0:
        return x
    angle = torch.outer(s["positions"].to(torch.float64), s["inv_freq"])
    c = _fl(torch.cos(angle) * s["amplitude"])[:, None, :]
    d = _fl(torch.sin(angle) * s["amplitude"])[:, None, :]
    i = torch.arange(r // 2, device=x.device)
    one, two = (i, i + r // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
    y = x.clone()
    y[..., one] = _fl(_fl(x[..., one] * c) - _fl(x[..., two] * d))
    y[..., two] = _fl(_fl(x[..., two] * c) + _fl(x[..., one] * d))
    return y


def exact(case, seed):
    # (64-bit products of the largest draws would take minutes)
    if case["op"] == "attention" and work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(s, case)
    if case["op"] == "read":
        return tuple(torch.cat([torch.stack([_exact_head(s, b, h, which)
                                             for h in range(case["kv_heads"])], dim=1)
                                for b in range(case["seqs"])]) for which in (0, 2))
    q, k = _exact_rotated(s, case, s["q"]), _exact_rotated(s, case, s["k"])
    if case["smooth"]:
        q, k = _fl(q * s["q_mul"].to(torch.float64)), _fl(k * s["k_mul"].to(torch.float64))
    return (q, _exact_blocks(k, case["fmt"]),
            _exact_blocks(s["v"].to(torch.float64), case["fmt"]))
