"""The microscaled cache of keys and values on the GPU against plain 64-bit
forms: rotary positions and the quantized write, reading back (both to the
bit), and the attention within its derived bound."""
import numpy as np
import pytest

import w8a8_post_quantization_amd as sq
from tests import kv_reference as ref
from tests import mx_reference as mx
from tests.gpu_util import assert_bits_equal, dev, host, log, to_bf16_bits

pytestmark = pytest.mark.gpu

FMTS = {"e2m1": mx.E2M1, "e4m3": mx.E4M3}


def to_dt(x, dt):
    """float values as an array of the type (bfloat16 as its bits)."""
    x = np.asarray(x, np.float32)
    if dt == "bf16":
        return to_bf16_bits(x)
    return x.astype({"f32": np.float32, "f16": np.float16}[dt])


def torch_dt(torch, dt):
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dt]


def on_gpu(torch, arrays):
    return tuple(dev(a, torch) for a in arrays)


# ------------------------------------------------------- rotary and the write

WRITES = [
    # tokens, q heads, heads, dim, page, dt, fmt, interleaved, rotary, smooth
    (1, 8, 1, 128, 16, "bf16", "e2m1", False, 128, False),
    (1, 16, 16, 64, 32, "f32", "e4m3", True, 64, True),
    (3, 10, 2, 64, 16, "f16", "e2m1", False, 32, True),
    (5, 7, 7, 256, 64, "bf16", "e4m3", True, 256, False),
    (37, 12, 3, 128, 16, "f32", "e2m1", False, 48, True),
    (37, 4, 4, 256, 128, "f16", "e2m1", True, 16, False),
    (64, 5, 5, 64, 16, "bf16", "e2m1", False, 0, True),
    (130, 2, 1, 128, 32, "f16", "e4m3", False, 128, True),
    (4100, 1, 1, 64, 1024, "bf16", "e4m3", False, 64, False),
]


@pytest.mark.parametrize("case", WRITES, ids=lambda c: "-".join(map(str, c)))
def test_write_matches_the_definition(case):
    import torch

    T, q_heads, heads, dim, page, dt, fmt, inter, rotary, smooth = case
    log(f"write {case}")
    rng = np.random.default_rng(T * 131 + dim + rotary)
    f = FMTS[fmt]
    pages = -(-T // page) + 3
    lens = [pages * page]
    cache = ref.Cache(rng, lens, heads, page, dim, f, spare=0)
    # rows of a wider product, keys with large channels, a few special values
    x = rng.standard_normal((T, q_heads + 2 * heads + 1, dim)).astype(np.float32)
    x[:, :, :: max(1, dim // 8)] *= 30
    x[0, q_heads, :32] = 0.0
    x[T // 2, -2, 5] = 3e4
    x = to_dt(x, dt)
    positions = rng.integers(0, 1 << 20, T)
    positions[-1] = (1 << 31) + 12345
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    if T > 2:
        slots[1], slots[2] = -1, pages * page  # neither is written
    inv_freq, amplitude = (None, 1.0) if rotary == 0 else sq.rope_frequencies(
        rotary, 10000.0, "yarn", 16.0, 4096, device="cpu")
    q_mul = np.exp(rng.standard_normal((q_heads, dim))).astype(np.float32) if smooth else None
    k_mul = np.exp(rng.standard_normal((heads, dim))).astype(np.float32) if smooth else None

    xt = dev(x, torch)
    held = on_gpu(torch, cache.arrays())
    g = lambda a: None if a is None else dev(a, torch)  # noqa: E731
    y = sq.rope_quantize_kv_mx(
        xt[:, :q_heads], xt[:, q_heads:q_heads + heads], xt[:, q_heads + heads:-1], dev(slots, torch),
        held, fmt=f, positions=dev(positions, torch),
        inv_freq=None if inv_freq is None else inv_freq.cuda(), amplitude=amplitude,
        layout=sq.SQ_ROPE_INTERLEAVED if inter else sq.SQ_ROPE_HALF, q_mul=g(q_mul), k_mul=g(k_mul))
    torch.cuda.synchronize()

    x32 = mx.to_f32(x)
    q, k, v = x32[:, :q_heads], x32[:, q_heads:q_heads + heads], x32[:, q_heads + heads:-1]
    if rotary:
        q = ref.rotated(q, positions, inv_freq.numpy(), amplitude, inter)
        k = ref.rotated(k, positions, inv_freq.numpy(), amplitude, inter)
    if smooth:
        q, k = q * q_mul, k * k_mul
    assert_bits_equal(host(y, torch), to_dt(q, dt), "q")
    kept = (slots >= 0) & (slots < pages * page)
    p, at = slots[kept] // page, slots[kept] % page
    want = [a.copy() for a in cache.arrays()]
    for i, rows in ((0, k), (2, v)):
        want[i][p, :, at], want[i + 1][p, :, at] = ref.quantized(rows[kept], f)
    for got, w, name in zip(held, want, ("kq", "ks", "vq", "vs")):
        assert_bits_equal(host(got, torch), w, name)


def test_write_without_queries_and_of_infinities():
    import torch

    log("write of keys and values alone, with an infinity and a NaN")
    rng = np.random.default_rng(5)
    cache = ref.Cache(rng, [32], 2, 16, 64, mx.E2M1)
    kv = rng.standard_normal((2, 20, 2, 64)).astype(np.float32)
    kv[0, 3, 1, 40], kv[1, 7, 0, 2] = np.inf, np.nan
    slots = cache.slots(0)[5:25]
    held = on_gpu(torch, cache.arrays())
    kt, vt = dev(kv[0], torch), dev(kv[1], torch)
    assert sq.rope_quantize_kv_mx(None, kt, vt, dev(slots, torch), held) is None
    torch.cuda.synchronize()
    want = [a.copy() for a in cache.arrays()]
    p, at = slots // 16, slots % 16
    for i in (0, 1):
        want[2 * i][p, :, at], want[2 * i + 1][p, :, at] = ref.quantized(kv[i], mx.E2M1)
    for got, w, name in zip(held, want, ("kq", "ks", "vq", "vs")):
        assert_bits_equal(host(got, torch), w, name)
    assert host(held[1], torch)[p[3], 1, at[3], 1] == 255 and host(held[3], torch)[p[7], 0, at[7], 0] == 255


# ---------------------------------------------------------------- reading back

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim,heads,page", [(64, 3, 16), (128, 1, 64), (256, 2, 32)])
def test_read_matches_the_values(dt, fmt, dim, heads, page):
    import torch

    log(f"read {dt} {fmt} {dim} {heads} {page}")
    rng = np.random.default_rng(dim + heads)
    lens = [0, 1, page, 0, 2 * page + 3, 5, 0]
    cache = ref.Cache(rng, lens, heads, page, dim, FMTS[fmt])
    cu = np.cumsum([0] + lens).astype(np.int32)
    total = int(cu[-1]) + 6
    out = tuple(torch.full((total, heads, dim), 7.0, dtype=torch_dt(torch, dt), device="cuda") for _ in range(2))
    held = on_gpu(torch, cache.arrays())
    got = sq.dequantize_kv_mx(held, dev(cache.table, torch), dev(cu, torch), total, fmt=FMTS[fmt], out=out)
    assert got[0] is out[0] and got[1] is out[1]
    torch.cuda.synchronize()
    for which in (0, 1):
        want = np.full((total, heads, dim), 7.0)
        for b in range(len(lens)):
            want[cu[b]:cu[b + 1]] = cache.read(b)[which]
        assert_bits_equal(host(got[which], torch), to_dt(want, dt), "kv"[which])


@pytest.mark.parametrize("fmt", FMTS)
def test_read_of_every_code_and_scale(fmt):
    import torch

    log(f"every code and scale, {fmt}")
    n = 16 if fmt == "e2m1" else 256
    codes = np.arange(256, dtype=np.uint8)[:n]
    skip = np.zeros(n, bool) if fmt == "e2m1" else (codes & 127) == 127
    codes = np.where(skip, 0, codes)
    row = np.tile(codes, 256 // n)  # every code in a head of 256 channels
    if fmt == "e2m1":
        row = row[0::2] | row[1::2] << 4
    q = np.broadcast_to(row, (1, 1, 256, len(row))).copy()
    e = np.broadcast_to(np.arange(256, dtype=np.uint8)[None, None, :, None], (1, 1, 256, 8)).copy()
    held = on_gpu(torch, (q, e, q, e))
    table, cu = dev(np.zeros((1, 1), np.int32), torch), dev(np.array([0, 256], np.int32), torch)
    want = ref.values(q[0, 0], e[0, 0], FMTS[fmt])[:, None, :]
    for dt in ("f32", "f16", "bf16"):
        k, v = sq.dequantize_kv_mx(held, table, cu, 256, fmt=FMTS[fmt], out_dtype=torch_dt(torch, dt))
        torch.cuda.synchronize()
        for t in (k, v):
            # (values, since a NaN has many bit patterns; the reference's fp32
            # holds each value of the formats)
            got = t.float().cpu().numpy()
            with np.errstate(over="ignore"):
                w = mx.to_f32(to_dt(want, dt))
            nan = np.isnan(want)
            assert np.array_equal(np.isnan(got), nan), dt
            assert np.array_equal(got[~nan], w[~nan]) and np.array_equal(
                np.signbit(got[~nan]), np.signbit(w[~nan])), dt


def test_read_of_pages_that_are_none():
    import torch

    log("pages that are not in the cache read as NaN")
    rng = np.random.default_rng(9)
    cache = ref.Cache(rng, [40, 20], 2, 16, 64, mx.E4M3, width=3)
    cache.table[0, 1] = cache.pages  # tokens 16 .. 31 of the first
    cu = np.array([0, 60, 80], np.int32)  # the first: 60 tokens of a table of 48
    k, v = sq.dequantize_kv_mx(on_gpu(torch, cache.arrays()), dev(cache.table, torch), dev(cu, torch), 80,
                               fmt=mx.E4M3, out_dtype=torch.float32)
    torch.cuda.synchronize()
    k = host(k, torch)
    nan = np.isnan(k).all(axis=(1, 2))
    assert nan[16:32].all() and nan[48:60].all() and not nan[:16].any() and not nan[60:].any()
    cache.table[0, 1] = 0
    assert_bits_equal(k[60:], cache.read(1)[0].astype(np.float32), "the sequence beside it")


# ------------------------------------------------------------------- attention

def run_attention(case, mark=None):
    """One call against the reference; `mark` changes cache and queries."""
    import torch

    lens, new, q_heads, heads, dim, page, dt, fmt, causal, window = case
    log(f"attention {case}")
    rng = np.random.default_rng(sum(lens) * 7 + dim + q_heads)
    cache = ref.Cache(rng, lens, heads, page, dim, FMTS[fmt])
    T = sum(new) + 2  # two rows behind the last sequence
    q = to_dt(rng.standard_normal((T, q_heads, dim)) * 1.5, dt)
    if mark is not None:
        mark(cache, q)
    pad = np.full((T, q_heads + 3, dim), np.nan, np.float32)
    wide = dev(to_dt(pad, dt), torch)  # rows of a wider product
    wide[:, 1:1 + q_heads] = dev(q, torch)
    qt = wide[:, 1:1 + q_heads]
    cu = dev(np.cumsum([0] + list(new)).astype(np.int32), torch)
    out = torch.full((T, q_heads, dim), 3.0, dtype=qt.dtype, device="cuda")
    args = (qt, on_gpu(torch, cache.arrays()), dev(cache.table, torch),
            dev(np.array(lens, np.int32), torch), cu)
    y = sq.attention_kv_mx(*args, fmt=FMTS[fmt], max_q=max(max(new), 1), causal=causal, window=window,
                           out=out)
    torch.cuda.synchronize()
    again = sq.attention_kv_mx(*args, fmt=FMTS[fmt], max_q=max(max(new), 1), causal=causal,
                               window=window, out=torch.full_like(out, 3.0))
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), again.view(torch.int16)), "the same call, other bits"
    got = y.float().cpu().numpy().astype(np.float64)
    assert (got[T - 2:] == 3.0).all(), "rows behind the last sequence"
    q64, at = mx.to_f32(q).astype(np.float64), 0
    worst = 0.0
    for b, n in enumerate(new):
        k, v = cache.read(b)
        want, tol = ref.attention(q64[at:at + n], k, v, dt, dim ** -0.5, causal, window)
        g = got[at:at + n]
        bad = ~np.isfinite(want)
        assert np.array_equal(np.isfinite(g), ~bad), (b, "finite where the reference is")
        if (~bad).any():
            err = np.abs(g - want)[~bad]
            assert (err <= tol[~bad]).all(), (b, (err / np.maximum(tol[~bad], 1e-30)).max())
            worst = max(worst, (err / np.maximum(tol[~bad], 1e-30)).max())
        at += n
    print(f"  largest error {worst:.2f} of its bound")


TOKENS = [
    # lengths, new tokens, q heads, heads, dim, page, dt, fmt, causal, window
    ((1,), (1,), 1, 1, 128, 16, "bf16", "e2m1", True, 0),
    ((2, 31, 0, 33, 17), (1, 1, 1, 1, 1), 8, 1, 128, 16, "bf16", "e2m1", True, 0),
    ((129, 128, 127, 640), (1, 1, 1, 1), 16, 2, 64, 32, "f16", "e2m1", True, 0),
    ((2049,), (1,), 8, 8, 128, 16, "f16", "e4m3", True, 0),
    ((700, 33), (1, 1), 4, 2, 256, 64, "bf16", "e4m3", True, 0),
    ((700, 33), (1, 1), 12, 2, 256, 64, "f16", "e2m1", True, 0),
    ((1500, 3, 260), (1, 1, 1), 12, 4, 64, 16, "bf16", "e4m3", True, 100),
    ((6001,), (1,), 8, 1, 128, 128, "bf16", "e2m1", True, 0),
    # G = 32: two column groups; G = 48: the tile kernel with split keys
    ((333, 90), (1, 1), 32, 1, 128, 16, "bf16", "e2m1", True, 0),
    ((1333, 90, 0), (1, 1, 1), 48, 1, 64, 32, "f16", "e2m1", True, 0),
    ((1333, 90, 2), (1, 1, 1), 71, 1, 64, 32, "bf16", "e4m3", True, 37),
]
DRAFTS = [
    ((5, 300, 64), (5, 3, 4), 4, 2, 128, 16, "bf16", "e2m1", True, 0),
    ((900, 17, 1), (4, 4, 1), 8, 1, 128, 16, "f16", "e4m3", True, 0),       # 32 rows
    ((900, 200), (2, 7), 8, 2, 64, 32, "f16", "e2m1", True, 50),
    ((130, 4), (3, 6), 4, 4, 256, 16, "bf16", "e2m1", True, 0),             # more queries than keys
    ((130, 40), (3, 5), 4, 2, 256, 16, "f16", "e4m3", False, 0),
    ((130, 40, 0), (3, 5, 2), 4, 2, 128, 16, "bf16", "e2m1", False, 20),
    ((61, 61), (0, 3), 2, 2, 64, 16, "bf16", "e2m1", True, 0),              # one without queries
]
PROMPTS = [
    ((33,), (33,), 2, 2, 128, 16, "bf16", "e2m1", True, 0),
    ((64, 65), (64, 65), 8, 2, 128, 32, "f16", "e2m1", True, 0),
    ((300, 131, 20), (100, 131, 1), 4, 1, 64, 16, "f16", "e4m3", True, 0),  # one of a single token
    ((300, 77), (40, 77), 4, 2, 256, 64, "bf16", "e2m1", True, 0),
    ((200, 50), (60, 50), 4, 2, 256, 16, "f16", "e4m3", True, 33),
    ((700, 300), (130, 70), 6, 2, 64, 16, "bf16", "e2m1", True, 64),
    ((150, 40), (90, 64), 4, 1, 128, 16, "f16", "e2m1", False, 0),          # not causal
    ((20, 150), (90, 150), 3, 1, 128, 16, "bf16", "e4m3", True, 0),         # more queries than keys
    ((0, 150), (90, 40), 3, 1, 128, 16, "bf16", "e2m1", True, 0),           # no keys at all
    ((1200,), (300,), 4, 2, 128, 64, "bf16", "e4m3", True, 0),
    ((257,), (257,), 1, 1, 64, 32, "bf16", "e4m3", True, 0),
]


@pytest.mark.parametrize("case", TOKENS + DRAFTS + PROMPTS, ids=lambda c: "-".join(map(str, c)))
def test_attention_matches_the_definition(case):
    run_attention(case)


@pytest.mark.parametrize("case", [
    ((300, 40), (4, 3), 4, 2, 128, 16, "bf16", "e2m1", True, 0),
    ((300, 40), (4, 3), 4, 2, 256, 16, "f16", "e4m3", True, 12),
    ((300, 40), (1, 1), 4, 2, 64, 16, "f16", "e2m1", True, 9),
    ((300, 140), (100, 90), 4, 2, 128, 16, "bf16", "e2m1", True, 0),
    ((300, 140), (100, 90), 4, 2, 64, 16, "f16", "e4m3", True, 50),
    ((300, 140), (100, 90), 2, 1, 256, 16, "bf16", "e4m3", True, 0),
], ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("which", ["key", "value"])
def test_a_nan_reaches_only_the_queries_that_see_it(case, which):
    """NaN blocks in the last token, in one among the queries' own, and before
    the window."""
    def mark(cache, q):
        scales = cache.ks if which == "key" else cache.vs
        for b, t in ((0, cache.lens[0] - 1), (0, 1 if case[-1] else cache.lens[0] - 2),
                     (1, cache.lens[1] - 2)):
            p, at = cache.where(b)
            scales[p[t], 0, at[t], 1] = 255
    run_attention(case, mark)


def test_values_beyond_fp16_reach_only_the_queries_that_see_them():
    """In fp16 a value of 4 2^15 is infinite: queries before it are finite."""
    def mark(cache, q):
        p, at = cache.where(0)
        cache.vs[p[-1], 0, at[-1], 0] = 127 + 15
        cache.vq[p[-1], 0, at[-1], :8] = 0x66  # 4, 4
    for case in (((60,), (4,), 2, 1, 128, 16, "f16", "e2m1", True, 0),
                 ((60,), (50,), 2, 1, 128, 16, "f16", "e2m1", True, 0)):
        import torch

        lens, new, q_heads, heads, dim, page = case[:6]
        log(f"infinite values {case}")
        rng = np.random.default_rng(3)
        cache = ref.Cache(rng, lens, heads, page, dim, mx.E2M1)
        mark(cache, None)
        q = dev(to_dt(rng.standard_normal((new[0], q_heads, dim)), "f16"), torch)
        y = sq.attention_kv_mx(q, on_gpu(torch, cache.arrays()), dev(cache.table, torch),
                               dev(np.array(lens, np.int32), torch),
                               dev(np.array([0, new[0]], np.int32), torch), max_q=new[0])
        torch.cuda.synchronize()
        y = host(y, torch)
        assert np.isfinite(y[:-1]).all()
        assert np.isposinf(y[-1, :, :16]).all() and np.isfinite(y[-1, :, 32:]).all()


def test_pages_that_are_none_and_lengths_past_the_table():
    import torch

    log("bad pages and lengths in attention")
    rng = np.random.default_rng(11)
    for n in (1, 40):
        lens = [60, 60, 60, 60]
        cache = ref.Cache(rng, lens, 2, 16, 64, mx.E2M1, width=4)
        cache.table[1, 1] = cache.pages
        q = dev(to_dt(rng.standard_normal((4 * n, 4, 64)), "bf16"), torch)
        cu = dev(np.arange(5, dtype=np.int32) * n, torch)
        y = sq.attention_kv_mx(q, on_gpu(torch, cache.arrays()), dev(cache.table, torch),
                               dev(np.array([60, 60, 65, -3], np.int32), torch), cu, max_q=n)
        torch.cuda.synchronize()
        y = y.float().cpu().numpy().reshape(4, n, 4, 64)
        assert np.isfinite(y[0]).all() and np.isnan(y[2]).all() and (y[3] == 0).all()
        p = 60 - n + np.arange(n)
        assert np.isnan(y[1][p >= 16]).all() and np.isfinite(y[1][p < 16]).all()


def test_attention_of_many_sequences_and_defaults():
    """More sequences than threads of a block, and the calls' defaults: no
    cu_q, no max_q."""
    import torch

    log("600 sequences")
    rng = np.random.default_rng(12)
    lens = [int(x) for x in rng.integers(0, 200, 600)]
    cache = ref.Cache(rng, lens, 1, 16, 64, mx.E4M3)
    q = to_dt(rng.standard_normal((600, 2, 64)), "f16")
    held, table = on_gpu(torch, cache.arrays()), dev(cache.table, torch)
    n = dev(np.array(lens, np.int32), torch)
    y = sq.attention_kv_mx(dev(q, torch), held, table, n, fmt=mx.E4M3)
    torch.cuda.synchronize()
    got = y.float().cpu().numpy()
    for b in range(600):
        k, v = cache.read(b)
        want, tol = ref.attention(mx.to_f32(q[b:b + 1]).astype(np.float64), k, v, "f16", 0.125)
        assert (np.abs(got[b] - want[0]) <= tol[0]).all(), b
    # without max_q any number of queries is expected
    cu = dev(np.arange(601, dtype=np.int32), torch)
    z = sq.attention_kv_mx(dev(q, torch), held, table, n, cu, fmt=mx.E4M3)
    torch.cuda.synchronize()
    assert np.abs(z.float().cpu().numpy() - got).max() <= 2.0 ** -9


def test_queries_past_max_q_do_no_harm():
    """A sequence with more queries than max_q says: its rows may stay, the
    others' are right."""
    import torch

    log("max_q too small")
    rng = np.random.default_rng(13)
    lens = [50, 70]
    cache = ref.Cache(rng, lens, 1, 16, 128, mx.E2M1)
    q = to_dt(rng.standard_normal((41, 1, 128)), "bf16")
    y = sq.attention_kv_mx(dev(q, torch), on_gpu(torch, cache.arrays()), dev(cache.table, torch),
                           dev(np.array(lens, np.int32), torch), dev(np.array([0, 40, 41], np.int32), torch),
                           max_q=1)
    torch.cuda.synchronize()
    k, v = cache.read(1)
    want, tol = ref.attention(mx.to_f32(q[40:]).astype(np.float64), k, v, "bf16", 128 ** -0.5)
    assert (np.abs(y[40:].float().cpu().numpy() - want) <= tol).all()
