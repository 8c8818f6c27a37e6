"""The microscaled cache's entry points without a GPU: what they export and
refuse on the host, the rotary frequencies, and the reference forms that the
GPU tests compare with."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import w8a8_post_quantization_amd as sq
from tests import kv_reference as ref
from tests import mx_reference as mx

OK, NULL, SHAPE, DTYPE, ALIGN, ARG, WORKSPACE, UNSUP, HIP = range(9)
FAKE = 0x100000  # aligned, not null; never read on these paths

built = pytest.mark.skipif(not os.path.exists(sq.LIB_PATH), reason="libsq.so not built")


def cache(**kw):
    a = dict(kq=FAKE, ks=FAKE, vq=FAKE, vs=FAKE, pages=4, heads=2, page=16, dim=128, fmt=0)
    a.update(kw)
    return sq._KvCache(*a.values())


def strides(a, b):
    return (ctypes.c_int64 * 2)(a, b)


@built
def test_exports():
    L = sq.lib()
    declared = sq.header_functions(sq.KV_HEADER)
    assert declared == ["sq_attention_kv_mx", "sq_attention_kv_mx_workspace", "sq_dequantize_kv_mx",
                        "sq_rope_quantize_kv_mx"]
    for name in declared:
        assert hasattr(L, name) and name in sq.SIGNATURES, name


BAD_CACHES = [(dict(fmt=2), ARG), (dict(dim=48), SHAPE), (dict(dim=96), UNSUP), (dict(dim=0), SHAPE),
              (dict(page=8), SHAPE), (dict(page=48), SHAPE), (dict(page=1 << 21), SHAPE),
              (dict(pages=0), SHAPE), (dict(heads=0), SHAPE), (dict(heads=65536), SHAPE),
              (dict(pages=1 << 30), UNSUP), (dict(kq=None), NULL), (dict(vs=None), NULL),
              (dict(vq=FAKE + 8), ALIGN), (dict(ks=FAKE + 2), ALIGN)]


@built
def test_write_refuses():
    L = sq.lib()

    def call(c=None, **kw):
        a = dict(q=FAKE, qs=strides(1024, 128), k=FAKE, ks=strides(1024, 128), v=FAKE, vs=strides(1024, 128),
                 dt=sq.SQ_F16, T=4, q_heads=8, pos=FAKE, freq=FAKE, rotary=64, amp=1.0, layout=0, qm=None,
                 km=None, slots=FAKE, cache=c or cache(), out=FAKE)
        a.update(kw)
        return L.sq_rope_quantize_kv_mx(*a.values(), None)

    for kw, status in BAD_CACHES:
        assert call(cache(**kw)) == status, kw
    for kw, status in [(dict(dt=3), DTYPE), (dict(layout=2), ARG), (dict(amp=math.nan), ARG),
                       (dict(T=-1), SHAPE), (dict(rotary=24), SHAPE), (dict(rotary=144), SHAPE),
                       (dict(q_heads=0), SHAPE), (dict(T=(1 << 24) + 1), UNSUP), (dict(k=None), NULL),
                       (dict(v=None), NULL), (dict(ks=None), NULL), (dict(out=None), NULL),
                       (dict(slots=None), NULL), (dict(pos=None), NULL), (dict(freq=None), NULL),
                       (dict(q=FAKE + 8), ALIGN), (dict(qs=strides(1028, 128)), ALIGN),
                       (dict(ks=strides(1024, 100)), ALIGN), (dict(dt=sq.SQ_F32, vs=strides(1026, 128)), ALIGN),
                       (dict(vs=strides(-1024, 128)), SHAPE), (dict(vs=strides(1 << 40, 128)), UNSUP),
                       (dict(out=FAKE + 8), ALIGN), (dict(qm=FAKE + 4), ALIGN), (dict(km=FAKE + 4), ALIGN),
                       (dict(slots=FAKE + 4), ALIGN), (dict(pos=FAKE + 4), ALIGN)]:
        assert call(**kw) == status, kw
    assert call(T=0, k=None, v=None, q=None, slots=None) == OK
    assert call(cache=None) == NULL


@built
def test_read_refuses():
    L = sq.lib()

    def call(c=None, **kw):
        a = dict(cache=c or cache(), table=FAKE, B=2, width=3, cu=FAKE, total=9, k=FAKE, v=FAKE, dt=sq.SQ_BF16)
        a.update(kw)
        return L.sq_dequantize_kv_mx(*a.values(), None)

    for kw, status in BAD_CACHES:
        assert call(cache(**kw)) == status, kw
    for kw, status in [(dict(dt=7), DTYPE), (dict(B=-1), SHAPE), (dict(width=-1), SHAPE), (dict(total=-1), SHAPE),
                       (dict(B=(1 << 24) + 1), UNSUP), (dict(total=(1 << 24) + 1), UNSUP),
                       (dict(width=1 << 28), UNSUP), (dict(cu=None), NULL), (dict(k=None), NULL),
                       (dict(v=None), NULL), (dict(table=None), NULL), (dict(k=FAKE + 4), ALIGN),
                       (dict(table=FAKE + 2), ALIGN), (dict(cu=FAKE + 2), ALIGN), (dict(cache=None), NULL)]:
        assert call(**kw) == status, kw
    assert call(total=0, k=None, v=None) == OK
    assert call(B=0, table=None, cu=None) == OK


@built
def test_attention_refuses():
    L = sq.lib()

    def call(c=None, **kw):
        a = dict(q=FAKE, qs=strides(1024, 128), dt=sq.SQ_F16, T=4, q_heads=8, cache=c or cache(), table=FAKE,
                 B=4, width=3, lens=FAKE, cu=None, max_q=1, scale=0.1, causal=1, window=0, y=FAKE, ws=FAKE,
                 size=1 << 40)
        a.update(kw)
        return L.sq_attention_kv_mx(*a.values(), None)

    for kw, status in BAD_CACHES:
        assert call(cache(**kw)) == status, kw
    for kw, status in [(dict(dt=sq.SQ_F32), DTYPE), (dict(T=-1), SHAPE), (dict(q_heads=7), SHAPE),
                       (dict(q_heads=0), SHAPE), (dict(T=5), SHAPE), (dict(max_q=0), SHAPE),
                       (dict(max_q=-1), SHAPE), (dict(width=1 << 28), UNSUP),
                       (dict(T=1 << 25, B=1 << 25), UNSUP),
                       (dict(q_heads=65536), UNSUP), (dict(T=1 << 20, q_heads=1024, cu=FAKE), UNSUP),
                       (dict(B=(1 << 21) + 1, T=(1 << 21) + 1), UNSUP), (dict(width=(1 << 26) + 1), UNSUP),
                       (dict(scale=math.inf), ARG), (dict(window=-1), ARG), (dict(q=None), NULL),
                       (dict(qs=None), NULL), (dict(lens=None), NULL), (dict(y=None), NULL),
                       (dict(table=None), NULL), (dict(ws=None), WORKSPACE), (dict(size=64), WORKSPACE),
                       (dict(ws=FAKE + 8), ALIGN), (dict(q=FAKE + 2), ALIGN), (dict(y=FAKE + 8), ALIGN),
                       (dict(qs=strides(1024, 4)), ALIGN), (dict(lens=FAKE + 2), ALIGN), (dict(cu=FAKE + 1), ALIGN),
                       (dict(cache=None), NULL)]:
        assert call(**kw) == status, kw
    assert call(T=0, B=0, q=None, y=None, ws=None) == OK
    assert call(B=0, cu=FAKE) == OK
    assert call(cache(heads=65535), width=1 << 24, q_heads=65535) == UNSUP


@built
def test_outputs_that_are_one_refuse():
    """Keys and values that would be written over one another."""
    L = sq.lib()
    s = strides(1024, 128)
    for kw in (dict(), dict(vq=FAKE + 64), dict(vs=FAKE + 64)):
        assert L.sq_rope_quantize_kv_mx(None, None, FAKE, s, FAKE, s, sq.SQ_F16, 4, 0, None, None, 0, 1.0, 0, None,
                                        None, FAKE, cache(**kw), None, None) == ARG, kw
    assert L.sq_dequantize_kv_mx(cache(), FAKE, 2, 3, FAKE, 9, FAKE, FAKE, sq.SQ_BF16, None) == ARG


# Operands at addresses of their own, never read: (name, address, bytes).
def _apart(sizes):
    at, out = 1 << 32, {}
    for name, n in sizes.items():
        out[name] = (at, n)
        at += (n + 4095) // 4096 * 4096 + 4096
    return out


def _meeting(places, first, second):
    """Addresses of `second` that share some bytes with `first`: its last bytes
    on the first's first, its first on the first's last, and inside."""
    at, n = places[first]
    m = places[second][1]
    return [at - (m - 16) // 16 * 16, at + (n - 16) // 16 * 16, at]


def _assert_pairs_refuse(call, places, outputs):
    pairs = 0
    for out in outputs:
        for name in places:
            if name == out:
                continue
            for at in _meeting(places, out, name):
                moved = {k: p for k, (p, _) in places.items()}
                moved[name] = at
                assert call(moved) == ARG, (out, name, at - places[out][0])
                pairs += 1
    return pairs


CACHE_BYTES = dict(kq=4 * 2 * 16 * 64, ks=4 * 2 * 16 * 4, vq=4 * 2 * 16 * 64, vs=4 * 2 * 16 * 4)


def _cache_at(p):
    return cache(kq=p["kq"], ks=p["ks"], vq=p["vq"], vs=p["vs"])


@built
def test_outputs_of_a_write_that_meet_refuse():
    """The rotated queries and the four arrays of the cache, in part over one
    another or over what a write reads."""
    L = sq.lib()
    T = 40  # (queries, keys and values as thirds of rows of 12 heads of 128, 2 bytes each)
    rows = (T - 1) * 12 * 128 * 2
    places = _apart(dict(q=rows + 8 * 256, k=rows + 2 * 256, v=rows + 2 * 256, pos=8 * T, freq=8 * 32, qm=4 * 8 * 128,
                         km=4 * 2 * 128, slots=8 * T, out=T * 8 * 256, **CACHE_BYTES))
    s = strides(12 * 128, 128)

    def call(p):
        return L.sq_rope_quantize_kv_mx(p["q"], s, p["k"], s, p["v"], s, sq.SQ_F16, T, 8, p["pos"], p["freq"], 64, 1.0,
                                        0, p["qm"], p["km"], p["slots"], _cache_at(p), p["out"], None)

    assert _assert_pairs_refuse(call, places, ["out", "kq", "ks", "vq", "vs"]) == 5 * 12 * 3


@built
def test_outputs_of_a_read_that_meet_refuse():
    L = sq.lib()
    places = _apart(dict(table=4 * 6, cu=4 * 3, k=9 * 2 * 256, v=9 * 2 * 256, **CACHE_BYTES))

    def call(p):
        return L.sq_dequantize_kv_mx(_cache_at(p), p["table"], 2, 3, p["cu"], 9, p["k"], p["v"], sq.SQ_BF16, None)

    assert _assert_pairs_refuse(call, places, ["k", "v"]) == 2 * 7 * 3


@built
def test_outputs_of_an_attention_that_meet_refuse():
    """Its output and workspace; queries as rows of a wider product, and as
    heads far apart."""
    L = sq.lib()
    T, B, width = 40, 2, 3
    need = L.sq_attention_kv_mx_workspace(T, 8, cache(), B, width, 9)
    assert need > 0
    for token, head in ((12 * 128, 128), (128, 64 * 128)):
        q = (T - 1) * token * 2 + 7 * head * 2 + 256
        places = _apart(dict(q=q, table=4 * B * width, lens=4 * B, cu=4 * (B + 1), y=T * 8 * 256, ws=need,
                             **CACHE_BYTES))

        def call(p):
            return L.sq_attention_kv_mx(p["q"], strides(token, head), sq.SQ_BF16, T, 8, _cache_at(p), p["table"], B,
                                        width, p["lens"], p["cu"], 9, 0.1, 1, 0, p["y"], p["ws"], need, None)

        assert _assert_pairs_refuse(call, places, ["y", "ws"]) == 2 * 9 * 3


@built
def test_workspace_sizes():
    """Enough for the parts of the blocks, whatever the lengths: it depends on
    shapes alone, and refused shapes need none."""
    L = sq.lib()
    size = lambda T, h, B, w, q, **kw: L.sq_attention_kv_mx_workspace(T, h, cache(**kw), B, w, q)  # noqa: E731
    one = size(1, 16, 1, 4096, 1)
    assert 0 < one <= 40 << 20
    assert size(1, 16, 1, 4096, 9) == one  # (one query is there)
    assert size(64, 16, 64, 4096, 1) == one
    assert size(7, 15, 7, 8, 1) == 0 and size(7, 16, 7, 8, 1, dim=96) == 0 and size(0, 16, 7, 8, 1) == 0
    # 48 heads share a key's head: tiles, and none of them split where they are many
    assert size(4096, 96, 4096, 64, 1) == 0 < size(40, 96, 40, 64, 1)
    # a prompt whose keys are split keeps its rows' parts for every split
    assert size(64, 16, 1, 4096, 64) >= 64 * 16 * 130 * 4 * 2


def test_binding_refuses_host_tensors_and_bad_shapes():
    c = sq.new_kv_cache_mx(2, 2, 16, 64, device="cpu")
    assert [tuple(t.shape) for t in c] == [(2, 2, 16, 32), (2, 2, 16, 2)] * 2
    assert sq.new_kv_cache_mx(2, 2, 16, 64, sq.SQ_MX_E4M3, device="cpu")[0].shape[3] == 64
    with pytest.raises(ValueError):
        sq.new_kv_cache_mx(2, 2, 16, 40, device="cpu")
    k = torch.zeros(3, 2, 64)
    i = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        sq.rope_quantize_kv_mx(None, k, k, i, c)
    with pytest.raises(ValueError, match="GPU"):
        sq.dequantize_kv_mx(c, i.to(torch.int32), i, 3)
    with pytest.raises(ValueError, match="GPU"):
        sq.attention_kv_mx(k.half(), c, i.to(torch.int32), i)


def test_rope_frequencies():
    f, a = sq.rope_frequencies(64, 10000.0, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,) and a == 1.0
    assert f[0] == 1.0 and abs(f[16].item() - 0.01) < 1e-16
    g, a = sq.rope_frequencies(64, 10000.0, "linear", 4.0, device="cpu")
    assert torch.equal(g * 4, f) and a == 1.0
    g, _ = sq.rope_frequencies(64, 10000.0, "ntk", 8.0, device="cpu")
    assert g[0] == 1.0 and abs((f[-1] / g[-1]).item() - 8) < 1e-9  # the slowest: divided by 8
    g, a = sq.rope_frequencies(64, 10000.0, "yarn", 8.0, 4096, device="cpu")
    ratio = (f / g).numpy()
    turns = 4096 * f.numpy() / (2 * math.pi)
    assert abs(a - (0.1 * math.log(8) + 1)) < 1e-15
    assert np.allclose(ratio[turns >= 32], 1) and np.allclose(ratio[turns <= 1], 8)
    assert (np.diff(ratio) >= -1e-12).all() and ratio.min() >= 1 - 1e-12 and ratio.max() <= 8 + 1e-12
    for bad in (dict(rotary=7), dict(rotary=64, scaling="other"), dict(rotary=64, scaling="yarn", factor=2.0),
                dict(rotary=64, base=0.0), dict(rotary=64, scaling="linear", factor=0.5)):
        with pytest.raises(ValueError):
            sq.rope_frequencies(**bad, device="cpu")


def test_reference_rotation_keeps_lengths_and_differences():
    """The rotation keeps a pair's length, and scores depend on the positions'
    difference alone."""
    rng = np.random.default_rng(1)
    f, _ = sq.rope_frequencies(64, device="cpu")
    x = rng.standard_normal((2, 1, 64)).astype(np.float32)
    for inter in (False, True):
        a = ref.rotated(np.repeat(x[:1], 3, 0), np.array([0, 5, 905]), f.numpy(), 1.0, inter)
        b = ref.rotated(np.repeat(x[1:], 3, 0), np.array([7, 12, 912]), f.numpy(), 1.0, inter)
        assert np.array_equal(a[0], x[0])
        # 64 channels, each off by two fp32 roundings of numbers below 8
        assert np.abs(np.linalg.norm(a, axis=2) - np.linalg.norm(x[0])).max() < 64 * 2.0 ** -21
        s = (a.astype(np.float64) * b).sum(axis=2)
        assert np.abs(s - s[0]).max() < 64 * 2.0 ** -18


def test_reference_attention_of_plain_cases():
    rng = np.random.default_rng(2)
    v = rng.standard_normal((5, 1, 64))
    k = np.zeros((5, 1, 64))
    q = rng.standard_normal((2, 2, 64))
    y, tol = ref.attention(q, k, v, "bf16", 0.125)
    assert np.allclose(y[1], v.mean(axis=0)) and np.allclose(y[0], v[:4].mean(axis=0)) and (tol > 0).all()
    y, _ = ref.attention(q, k, v, "bf16", 0.125, True, 2)
    assert np.allclose(y[1], v[3:].mean(axis=0))
    y, tol = ref.attention(np.concatenate([q] * 4), k[:3], v[:3], "f16", 0.125)
    assert (y[:5] == 0).all() and (tol[:5] == 0).all() and np.allclose(y[5], v[:1])
    v[4] = np.nan
    y, _ = ref.attention(q, k, v, "bf16", 0.125)
    assert np.isfinite(y[0]).all() and np.isnan(y[1]).all()


def test_reference_cache_holds_nan_where_no_token_is():
    rng = np.random.default_rng(3)
    c = ref.Cache(rng, [17, 0, 5], 2, 16, 64, mx.E2M1)
    assert (c.ks == 255).any() and np.isfinite(c.read(0)[0]).all() and c.read(1)[0].shape == (0, 2, 64)
    assert len(np.unique(np.concatenate([c.slots(b) for b in range(3)]))) == 22
