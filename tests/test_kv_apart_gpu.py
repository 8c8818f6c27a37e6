"""Values that are infinite or NaN, or of a block that may hold such, in keys
that only some of a tile's rows see, where other tiles follow: the attention of
many queries sets them apart from tile to tile.  NaN, both infinities and
finite values are compared each for themselves."""
import numpy as np
import pytest

import w8a8_post_quantization_amd as sq
from tests import kv_reference as ref
from tests import mx_reference as mx
from tests.gpu_util import dev, log
from tests.test_kv_gpu import FMTS, on_gpu, to_dt

pytestmark = pytest.mark.gpu

# From here on a value is infinite in the type: half a step past its largest.
INFINITE = {"f16": 65520.0, "bf16": (2.0 - 2.0 ** -8) * 2.0 ** 127}


def put_value(cache, b, token, head, channel, what, dt):
    """Value `channel` of a token becomes `what`, the others of its block
    (e2m1) or none (e4m3) 0.  "large": finite, though its block's scale is one
    at which values may be infinite in fp16."""
    p, at = cache.where(b)
    p, at = p[token], at[token]
    block, code = channel // 32, cache.vq[p, head, at]
    if cache.fmt == mx.E4M3:
        if what == "nan":
            code[channel] = 0x7f
            return
        # 2^8 2^15 and 2^7 2^8 in fp16 (scales from 2^8 on are suspect)
        code[32 * block:32 * block + 32] = 0
        code[channel] = {"inf": 0x78, "-inf": 0xf8, "large": 0x70}[what]
        e = {"f16": {"large": 135}, "bf16": {}}[dt].get(what, 142 if dt == "f16" else 254)
    else:
        code[16 * block:16 * block + 16] = 0
        nibble = {"inf": 7, "-inf": 15, "large": 2, "nan": 7}[what]
        code[channel // 2] = nibble << 4 * (channel & 1)
        # 6 2^15 and 2^14 in fp16, 6 2^126 in bf16
        e = 255 if what == "nan" else 141 if what == "large" else 142 if dt == "f16" else 253
    cache.vs[p, head, at, block] = e


def check(lens, new, q_heads, heads, dim, page, dt, fmt, causal, window, marks, seed=0):
    """marks: (sequence, token, head, channel, what).  The same call twice gives
    the same bits."""
    import torch

    rng = np.random.default_rng(seed)
    cache = ref.Cache(rng, lens, heads, page, dim, FMTS[fmt])
    for b, token, head, channel, what in marks:
        put_value(cache, b, token, head, channel, what, dt)
    q = to_dt(rng.standard_normal((sum(new), q_heads, dim)), dt)
    held, table = on_gpu(torch, cache.arrays()), dev(cache.table, torch)
    args = (dev(q, torch), held, table, dev(np.array(lens, np.int32), torch),
            dev(np.cumsum([0] + list(new)).astype(np.int32), torch))
    call = lambda: sq.attention_kv_mx(*args, fmt=FMTS[fmt], max_q=max(new), causal=causal, window=window)  # noqa: E731
    y = call()
    again = [call() for _ in range(3)]
    torch.cuda.synchronize()
    for z in again:
        assert torch.equal(y.view(torch.int16), z.view(torch.int16)), "the same call, other bits"
    got, q64, at = y.double().cpu().numpy(), mx.to_f32(q).astype(np.float64), 0
    reached = 0
    for b, n in enumerate(new):
        k, v = cache.read(b)
        v = np.where(np.abs(v) >= INFINITE[dt], np.copysign(np.inf, v), v)
        with np.errstate(invalid="ignore"):
            want, tol = ref.attention(q64[at:at + n], k, v, dt, dim ** -0.5, causal, window)
        g = got[at:at + n]
        for name, kind in (("NaN", np.isnan), ("+inf", np.isposinf), ("-inf", np.isneginf)):
            assert np.array_equal(kind(g), kind(want)), (b, name, np.argwhere(kind(g) != kind(want))[:5])
        fine = np.isfinite(want)
        err = np.abs(g[fine] - want[fine])
        assert (err <= tol[fine]).all(), (b, (err / np.maximum(tol[fine], 1e-30)).max())
        reached += (~fine).sum()
        at += n
    return reached


def whats(fmt, dt):
    # ("large" in fp16 alone: in bf16 the largest values times a weight past 1
    # leave fp32, whatever holds them)
    return ("nan", "inf", "-inf") + (("large",) if dt == "f16" else ())


# One sequence of 480 keys (up to 512 are not split over blocks), its block's
# tiles 64 keys, or 128 for 128 channels and more than 128 rows.
MANY = [
    # new, q heads, heads, dim, page, dt, fmt, window
    (150, 1, 1, 128, 16, "f16", "e2m1", 120),   # eight waves: tiles from 128, 256, 384, all masked
    (150, 2, 2, 128, 32, "bf16", "e4m3", 120),
    (256, 1, 1, 128, 16, "bf16", "e2m1", 0),    # the diagonal over three tiles
    (256, 1, 1, 128, 16, "f16", "e4m3", 0),
    (100, 1, 1, 128, 16, "f16", "e2m1", 90),    # four waves
    (128, 1, 1, 128, 16, "bf16", "e4m3", 0),
    (128, 2, 2, 64, 16, "f16", "e2m1", 70),
    (128, 1, 1, 64, 64, "bf16", "e4m3", 0),
    (90, 2, 1, 64, 16, "f16", "e4m3", 64),
    (128, 1, 1, 256, 16, "f16", "e2m1", 70),
    (128, 2, 2, 256, 16, "bf16", "e4m3", 0),
    (70, 2, 1, 256, 64, "f16", "e4m3", 50),
]


@pytest.mark.parametrize("place", ["first unit", "last unit", "every unit"])
@pytest.mark.parametrize("case", MANY, ids=lambda c: "-".join(map(str, c)))
def test_values_set_apart_in_tile_after_tile(case, place):
    """A key of each tile that rows see and others do not, in the tile's first
    or last 32 keys or all of them, each in a channel of its own."""
    new, q_heads, heads, dim, page, dt, fmt, window = case
    log(f"set apart {case} {place}")
    tile = 128 if dim == 128 and new * q_heads // heads > 128 else 64
    n = 480
    first = max(0, n - new + 1 - window) if window else 0
    kinds, marks, at = whats(fmt, dt), [], 0
    for t in range(first // tile * tile, n, tile):
        units = {"first unit": [0], "last unit": [tile // 32 - 1], "every unit": range(tile // 32)}[place]
        for u in units:
            for key in (t + 32 * u + 3, t + 32 * u + 22, t + 32 * u + 31):
                if first <= key < n:
                    # (channels in 32 apart: a mark clears its block)
                    marks.append((0, key, at % heads, (at * 32 + at * 5 % 32) % dim, kinds[at % len(kinds)]))
                    at += 1
    reached = check((n,), (new,), q_heads, heads, dim, page, dt, fmt, True, window, marks)
    assert reached > 0


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_a_value_of_the_first_windowed_tile_before_many_others(dim, fmt):
    """The last keys of the first tile of a window, with tiles behind it that
    all rows see in full, in blocks of their own or not."""
    for lens, new, window in (((480,), (140,), 330), ((3000, 900), (140, 60), 800)):
        log(f"first tile {dim} {fmt} {lens}")
        marks = []
        for b, (n, m) in enumerate(zip(lens, new)):
            first = n - m + 1 - window
            # (the window's first tiles and those that its rows leave)
            for j, key in enumerate(range(max(first, 0) | 31, n - m, 32)):
                if key < first + m + 128:
                    marks.append((b, key, 0, (j * 37) % dim, whats(fmt, "f16")[j % 4]))
        assert marks
        assert check(lens, new, 1, 1, dim, 16, "f16", fmt, True, window, marks) > 0


@pytest.mark.parametrize("i", range(24))
def test_random_values_set_apart(i):
    rng = np.random.default_rng(5000 + i)
    dim, fmt, dt = (64, 128, 256)[i % 3], ("e2m1", "e4m3")[i // 3 % 2], ("f16", "bf16")[i // 6 % 2]
    heads = int(rng.integers(1, 3))
    group = int(rng.integers(1, 4))
    seqs = int(rng.integers(1, 4))
    new = [int(rng.integers(1, 300)) for _ in range(seqs)]
    lens = [n + int(rng.integers(0, 400)) for n in new]
    window = int(rng.integers(1, 250)) if rng.random() < 0.6 else 0
    marks = []
    for b, n in enumerate(lens):
        for _ in range(int(rng.integers(1, 20))):
            marks.append((b, int(rng.integers(n)), int(rng.integers(heads)), int(rng.integers(dim)),
                          whats(fmt, dt)[int(rng.integers(len(whats(fmt, dt))))]))
    log(f"random {i} {lens} {new} {group} {heads} {dim} {window}")
    check(tuple(lens), tuple(new), heads * group, heads, dim, 16, dt, fmt, True, window, marks, i)
