"""The attention's softmax weights at the ends of their range: weights far below
the largest, which fp16 holds with few bits or not at all."""
import numpy as np
import pytest

import w8a8_post_quantization_amd as sq
from tests import kv_reference as ref
from tests import mx_reference as mx
from tests.gpu_util import dev, log
from tests.test_kv_gpu import FMTS, on_gpu, to_dt

pytestmark = pytest.mark.gpu


def attend(cache, q, dt, seqs, scale, window=0):
    """q [T, heads, D] over the cache's one sequence, `seqs` times in a call:
    float64 y of each."""
    import torch

    T = q.shape[0]
    y = sq.attention_kv_mx(dev(np.tile(q, (seqs, 1, 1)), torch), on_gpu(torch, cache.arrays()),
                           dev(np.repeat(cache.table, seqs, 0), torch),
                           dev(np.full(seqs, cache.lens[0], np.int32), torch),
                           dev(np.arange(seqs + 1, dtype=np.int32) * T, torch), fmt=cache.fmt, max_q=T, scale=scale,
                           window=window)
    torch.cuda.synchronize()
    return y.double().cpu().numpy().reshape(seqs, *q.shape)


@pytest.mark.parametrize("spread", [0.0, 0.4])
@pytest.mark.parametrize("nats", [14.0, 16.0, 18.0])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,seqs", [(1, 512), (3, 256), (40, 4), (150, 2)])
@pytest.mark.parametrize("fmt,dim", [("e2m1", 128), ("e4m3", 64)])
def test_small_weights_add_up(fmt, dim, T, seqs, dt, nats, spread):
    """A first key whose score is 14 to 18 nats above some 3500 others, and whose
    value is 0: the output is the others' alone.

    The bound is that of ref.attention but for fp16's smallest step.  There a
    weight is rounded by 2^-25 at the most where it is below 2^-14, and the
    sequence's largest weight is 2^7 at least, so a key adds 2^-32 |v| and not
    2^-25 |v| to the error."""
    log(f"small weights {fmt} {dim} {T} {seqs} {dt} {nats} {spread}")
    rng = np.random.default_rng(61)
    n, scale = 3500, dim ** -0.5
    d = np.sign(rng.standard_normal(dim)).astype(np.float32)
    size = nats / (2.0 * dim * scale)  # the first key is 2 d
    q = to_dt(np.broadcast_to(d * np.float32(size), (T, 1, dim)), dt)
    k = (spread * rng.standard_normal((n, 1, dim))).astype(np.float32)
    k[0, 0] = 2.0 * d
    v = (64.0 + 32.0 * rng.random((n, 1, dim))).astype(np.float32)
    v[0] = 0.0
    cache = ref.Cache(rng, [n], 1, 64, dim, FMTS[fmt], k=[k], v=[v])
    keys, values = cache.read(0)
    want, tol = ref.attention(mx.to_f32(q).astype(np.float64), keys, values, dt, scale)
    if dt == "f16":
        seen = np.cumsum(np.abs(values), axis=0)[n - T:]  # [T, 1, D]: of each query's keys
        tol = tol - (2.0 ** -25 - 2.0 ** -32) * seen
    got = attend(cache, q, dt, seqs, scale)
    err = np.abs(got - want)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-42, -1e-42])
@pytest.mark.parametrize("T", [1, 5, 70, 150])
@pytest.mark.parametrize("fmt,dim", [("e2m1", 128), ("e4m3", 64), ("e2m1", 256)])
def test_scales_of_zero_against_infinite_scores(fmt, dim, T, scale):
    """A key of -2^17 is infinite in fp16.  Times a scale of 0 its score is NaN,
    and so are the queries that see it, whichever kernel takes them; times the
    least scales above and below 0 it is an infinity of its sign, whose weight
    is 0 or, of +inf, NaN.  All others' scores are 0, or as good as."""
    log(f"scale {scale} {fmt} {dim} {T}")
    rng = np.random.default_rng(62)
    n, at = 200, 190 - T // 2  # (about half of several queries see it)
    q = to_dt(1.0 + rng.random((T, 2, dim)), "f16")
    k, v = (rng.standard_normal((n, 2, dim)).astype(np.float32) for _ in range(2))
    k[at, 0, :32] = 0.0
    k[at, 0, 3] = -2.0 ** 17
    cache = ref.Cache(rng, [n], 2, 16, dim, FMTS[fmt], k=[k], v=[v])
    got = attend(cache, q, "f16", 1, scale)[0]
    _, values = cache.read(0)
    u = ref.HALF_STEP["f16"]
    for i in range(T):
        for h in range(2):
            keys = np.arange(n - T + i + 1)
            meets = h == 0 and at in keys
            if meets and (scale <= 0):  # (-0.0 <= 0: 0 inf is NaN; a negative scale makes it +inf)
                assert np.isnan(got[i, h]).all(), (i, h)
                continue
            if meets:
                keys = keys[keys != at]
            # equal weights, exact in the type: sums in fp32, the output rounded
            want, a = values[keys, h].mean(axis=0), np.abs(values[keys, h]).mean(axis=0)
            tol = (n + 64) * 2.0 ** -23 * a + u * np.abs(want) + 2.0 ** -25
            assert (np.abs(got[i, h] - want) <= tol).all(), (i, h)


# a scale that is 1 as a power of two, once log2(e) is multiplied in fp32
LN2 = float(np.float32(0.6931471824645996))


@pytest.mark.parametrize("rise", [1, 2, 40, 128])
@pytest.mark.parametrize("T,seqs,n", [(1, 300, 600), (5, 100, 600), (60, 1, 300), (150, 1, 400)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt,dim", [("e4m3", 128), ("e4m3", 64), ("e4m3", 256)])
def test_scores_a_step_of_fp32_apart(fmt, dim, dt, T, seqs, n, rise):
    """Scores of 2^27 + 16 i (powers of two), i rising by 1 every `rise` keys:
    neighbours in fp32, whose weights differ by 2^16.  Sums are exact."""
    log(f"a step apart {fmt} {dim} {dt} {T} {seqs} {rise}")
    assert np.float32(LN2) * np.float32(1.44269504088896341) == np.float32(1.0)
    rng = np.random.default_rng(64)
    q, k = np.zeros((T, 1, dim)), np.zeros((n, 1, dim), np.float32)
    half = dim // 2
    q[..., :half], k[..., :half] = 2.0 ** 11, 2.0 ** 16 / half  # 2^27
    i = np.minimum(np.arange(n) // rise, 200)
    # 16 i from two channels of a block of their own, by the fifteens and the rest
    q[..., half], q[..., half + 1] = 16.0 * 15, 16.0
    k[:, 0, half], k[:, 0, half + 1] = i // 15, i % 15
    q = to_dt(q, dt)
    v = rng.standard_normal((n, 1, dim)).astype(np.float32)
    cache = ref.Cache(rng, [n], 1, 16, dim, FMTS[fmt], k=[k], v=[v])
    keys, values = cache.read(0)
    assert np.array_equal(keys, k)  # (the format holds them)
    got, u, least = attend(cache, q, dt, seqs, LN2), ref.HALF_STEP[dt], 2.0 ** -25 if dt == "f16" else 0.0
    for t in range(T):
        m = n - T + t + 1
        w = np.exp2(16.0 * (i[:m] - i[:m].max()))
        w /= w.sum()
        want, a = w @ values[:m, 0], w @ np.abs(values[:m, 0])
        tol = (u + (n + 64) * 2.0 ** -23) * a * (1 + u) + u * np.abs(want) + least
        tol = tol + least * np.abs(values[:m, 0]).sum(axis=0)
        err = np.abs(got[:, t, 0] - want)
        assert (err <= tol).all(), (t, (err / tol).max())


@pytest.mark.parametrize("order", ["random", "rising", "falling"])
@pytest.mark.parametrize("exponent", [20, 24, 27, 28, 31, 40, 90])
@pytest.mark.parametrize("T,seqs,n", [(1, 300, 600), (5, 100, 600), (60, 1, 300), (150, 1, 400), (60, 1, 3000)])
@pytest.mark.parametrize("fmt,dim,dt", [("e4m3", 128, "f16"), ("e4m3", 64, "bf16"), ("e4m3", 256, "f16"),
                                        ("e4m3", 128, "bf16")])
def test_scores_of_any_size(fmt, dim, dt, T, seqs, n, exponent, order):
    """Keys of 8/8 .. 14/8 along one direction, scores of up to 14/8 2^exponent
    of either sign; every third query is 2^-18 of the others, its scores
    moderate where theirs are largest.

    All products and sums are exact in fp32.  Scores past 2^12 are equal or a
    fourteenth apart, where the lesser's weight is 0 in fp32: such rows are means of
    the keys with the largest, off by the roundings of equal weights.  Others'
    scores are off by three roundings, 2^-21.  The bound's other terms are those of
    ref.attention."""
    log(f"large scores {fmt} {dim} {dt} {T} {seqs} {exponent} {order} {n}")
    rng = np.random.default_rng(63)
    step = rng.integers(8, 15, n)
    step = {"random": step, "rising": np.sort(step), "falling": np.sort(step)[::-1]}[order]
    d = np.sign(rng.standard_normal(dim)).astype(np.float32)
    k = (step[:, None, None] / 8.0 * d).astype(np.float32)
    v = rng.standard_normal((n, 1, dim)).astype(np.float32)
    size = np.where(np.arange(T) % 3 == 1, 2.0 ** -14, 16.0)[:, None, None] * np.array([1.0, -1.0])[None, :, None]
    q = to_dt(size * d, dt)
    cache = ref.Cache(rng, [n], 1, 16, dim, FMTS[fmt], k=[k], v=[v])
    keys, values = cache.read(0)
    assert np.array_equal(keys, k)  # (the format holds them)
    scale = 2.0 ** exponent / (16.0 * dim)
    got, want, tol = attend(cache, q, dt, seqs, scale), np.zeros((T, 2, dim)), np.zeros((T, 2, dim))
    u, least = ref.HALF_STEP[dt], 2.0 ** -25 if dt == "f16" else 0.0
    for i in range(T):
        see = slice(0, n - T + i + 1)
        for h in range(2):
            s = (keys[see, 0] @ mx.to_f32(q[i, h]).astype(np.float64)) * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            a, top = w @ np.abs(values[see, 0]), np.abs(s).max()
            off = 0.0 if top > 4096 else np.expm1(2 * 3 * 2.0 ** -23 * top)
            want[i, h] = w @ values[see, 0]
            tol[i, h] = (u + off + (n + 64) * 2.0 ** -23) * a * (1 + u) + u * np.abs(want[i, h])
            tol[i, h] += least + least * np.abs(values[see, 0]).sum(axis=0)
    err = np.abs(got - want)
    assert (err <= tol).all(), (err / tol).max()
