"""The microscaled cache's calls as a program makes them: one after another
from the norm to the output product, in captured graphs, on other streams, with
bounds watched, over caches past 4 GiB; and random shapes of every kernel."""
import numpy as np
import pytest

import w8a8_post_quantization_amd as sq
from tests import kv_reference as ref
from tests import mx_reference as mx
from tests.gpu_util import assert_bits_equal, dev, host, log
from tests.test_kv_gpu import on_gpu, run_attention, to_dt

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------- random shapes

def _random_case(i):
    rng = np.random.default_rng(1000 + i)
    dim = (64, 128, 256)[i % 3]
    fmt, dt = ("e2m1", "e4m3")[i // 3 % 2], ("bf16", "f16")[i // 6 % 2]
    heads = int(rng.integers(1, 4))
    # rows of an item: one, few, up to 16, 17 .. 32, and many
    kind = i % 5
    group = int(rng.integers(1, (2, 9, 17, 33, 7)[kind]))
    seqs = int(rng.integers(1, 7))
    most = (1, 3, 1, 1, 90)[kind]
    new = [int(rng.integers(0, most + 1)) for _ in range(seqs)]
    new[-1] = most
    lens = [int(np.exp(rng.uniform(0, np.log(900)))) for _ in range(seqs)]
    window = int(rng.integers(1, 300)) if rng.random() < 0.4 else 0
    return (tuple(lens), tuple(new), heads * group, heads, dim, (16, 32, 64, 256)[int(rng.integers(4))], dt, fmt,
            bool(rng.random() < 0.8), window)


@pytest.mark.parametrize("i", range(60))
def test_random_attention(i):
    run_attention(_random_case(i))


# ------------------------------------------------------- scores of every kind

def _one(q, k, v, dt, scale=None, causal=True, window=0, fmt=mx.E2M1, page=16):
    """q [T, heads, D], k and v [n, kv, D] of one sequence: kernel, reference."""
    import torch

    rng = np.random.default_rng(0)
    T, heads, dim = q.shape
    cache = ref.Cache(rng, [len(k)], k.shape[1], page, dim, fmt, k=[k], v=[v])
    q = to_dt(q, dt)
    y = sq.attention_kv_mx(dev(q, torch), on_gpu(torch, cache.arrays()), dev(cache.table, torch),
                           dev(np.array([len(k)], np.int32), torch), dev(np.array([0, T], np.int32), torch),
                           fmt=fmt, max_q=T, scale=scale, causal=causal, window=window)
    torch.cuda.synchronize()
    want, tol = ref.attention(mx.to_f32(q).astype(np.float64), *cache.read(0), dt,
                              dim ** -0.5 if scale is None else scale, causal, window)
    return y.float().cpu().numpy().astype(np.float64), want, tol


@pytest.mark.parametrize("T", [1, 5, 70])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_maxima_that_creep_and_leap(T, dim):
    """Scores that grow by less than the rescaling's slack from tile to tile,
    by much more, and that fall: each key along one direction, its size a
    function of its place."""
    rng = np.random.default_rng(21)
    n = 700
    d = np.sign(rng.standard_normal(dim)).astype(np.float32)
    q = np.broadcast_to(d, (T, 2, dim)) * np.float32(0.5)
    v = rng.standard_normal((n, 1, dim)).astype(np.float32)
    for name, size in (("creep", np.arange(n) / 40), ("leap", (np.arange(n) // 100) ** 2 / 2.0),
                       ("fall", 20 - np.arange(n) / 30), ("saw", np.arange(n) % 90 / 6.0)):
        log(f"{name} {T} {dim}")
        k = (size[:, None, None] * d * 2 / dim ** 0.5).astype(np.float32)
        y, want, tol = _one(q, k, v, "bf16")
        assert (np.abs(y - want) <= tol).all(), (name, (np.abs(y - want) / tol).max())


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("scale", [0.3, -0.2, 0.0])
def test_scales_of_any_sign(T, scale):
    log(f"scale {scale} {T}")
    rng = np.random.default_rng(22)
    q, k, v = (rng.standard_normal(s).astype(np.float32) for s in ((T, 4, 128), (200, 2, 128), (200, 2, 128)))
    for dt in ("bf16", "f16"):
        y, want, tol = _one(q, k, v, dt, scale=scale)
        assert (np.abs(y - want) <= tol).all(), (np.abs(y - want) / tol).max()


@pytest.mark.parametrize("T", [1, 50])
def test_queries_that_are_not_finite_stay_alone(T):
    rng = np.random.default_rng(23)
    q, k, v = (rng.standard_normal(s).astype(np.float32) for s in ((T, 4, 128), (300, 2, 128), (300, 2, 128)))
    q[T - 1, 1, 5] = np.nan
    y, want, tol = _one(q, k, v, "bf16")
    assert np.isnan(y[T - 1, 1]).all()
    rest = np.ones(y.shape, bool)
    rest[T - 1, 1] = False
    assert (np.abs(y - want)[rest] <= tol[rest]).all()


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("T,n", [(1, 1), (1, 40), (1, 5000), (3, 200), (70, 90), (70, 5000), (70, 30)])
def test_scores_of_minus_infinity(T, n, dim, fmt):
    """Keys of -2^17 are infinite in fp16, their scores -inf: a query that sees
    no others has a softmax of 0 / 0 and gets NaN, one that sees a finite key
    too has all its weight there, one that sees no key gets 0."""
    log(f"scores of -inf {T} {n} {dim} {fmt}")
    rng = np.random.default_rng(26)
    q = np.ones((T, 4, dim), np.float32)
    k, v = (rng.standard_normal((n, 2, dim)).astype(np.float32) for _ in range(2))
    k[:, :, 0], k[:, :, 1:32] = -2.0 ** 17, 0.0
    f = {"e2m1": mx.E2M1, "e4m3": mx.E4M3}[fmt]
    y, _, _ = _one(q, k, v, "f16", fmt=f)
    blind = max(T - n, 0)  # queries before the first key
    assert (y[:blind] == 0).all()
    assert np.isnan(y[blind:]).all()
    k[n - 1, :, 0] = 0.0
    y, _, _ = _one(q, k, v, "f16", fmt=f)
    assert (y[:blind] == 0).all()
    assert np.isnan(y[blind:T - 1]).all()
    last = ref.values(*ref.quantized(v[n - 1:], f), f)[0]  # (at most 8 bits, in fp16's range: exact)
    assert (y[T - 1] == np.repeat(last, 2, axis=0)).all()


@pytest.mark.parametrize("new", [(1, 1), (4, 3), (100, 90)])
@pytest.mark.parametrize("which", ["key", "value"])
@pytest.mark.parametrize("code", [0x7f, 0xff])
def test_codes_that_are_nan(new, which, code):
    """e4m3 codes of NaN, in the last token and among the queries' own."""
    def mark(cache, q):
        held = cache.kq if which == "key" else cache.vq
        for b, t in ((0, cache.lens[0] - 1), (1, cache.lens[1] - 2)):
            p, at = cache.where(b)
            held[p[t], 0, at[t], 37] = code
    run_attention(((300, 140), new, 4, 2, 64, 16, "f16", "e4m3", True, 0), mark)


@pytest.mark.parametrize("new", [(1, 1, 1), (3, 5, 1), (90, 1, 77)])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_pages_that_sequences_share(new, fmt):
    """Sequences with the same first pages, one of them twice in a row."""
    def mark(cache, q):
        cache.table[1, :6] = cache.table[0, :6]
        cache.table[2, :4] = cache.table[0, 2]
    run_attention(((300, 140, 200), new, 4, 2, 128, 16, "bf16", fmt, True, 0), mark)


@pytest.mark.parametrize("T", [1, 3, 60])
def test_windows_of_one_and_beyond_the_length(T):
    rng = np.random.default_rng(24)
    q, k, v = (rng.standard_normal(s).astype(np.float32) for s in ((T, 2, 64), (150, 2, 64), (150, 2, 64)))
    for window in (1, 16, 17, 149, 150, 151, 1 << 40):
        log(f"window {window} {T}")
        y, want, tol = _one(q, k, v, "f16", window=window)
        assert (np.abs(y - want) <= tol).all(), window


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("T,n", [(1, 1), (5, 1), (5, 150), (60, 1), (60, 0), (60, 150)])
@pytest.mark.parametrize("causal", [True, False])
def test_the_largest_windows(T, n, dim, causal):
    """Windows up to 2^63 - 1 hide nothing, with more queries than keys too."""
    rng = np.random.default_rng(27)
    q, k, v = (rng.standard_normal(s).astype(np.float32) for s in ((T, 2, dim), (n, 2, dim), (n, 2, dim)))
    plain, want, tol = _one(q, k, v, "bf16", causal=causal)
    assert (np.abs(plain - want) <= tol).all()
    for window in (1 << 30, (1 << 30) + 1, 1 << 62, (1 << 63) - 1):
        log(f"window {window} {T} {n} {dim} {causal}")
        y, _, _ = _one(q, k, v, "bf16", causal=causal, window=window)
        assert (y == plain).all(), window


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_keys_and_values_near_the_types_smallest(T, fmt):
    """Keys of 2^-126 and 2^-124 in bf16 against queries of 2^126, keys and values of 2^-16
    in fp16: what the codes stand for is subnormal in the type, and held."""
    f = {"e2m1": mx.E2M1, "e4m3": mx.E4M3}[fmt]
    for dt, key, value, query in (("bf16", -126 if f == mx.E2M1 else -124, 0, 126), ("f16", -16, -16, 12)):
        log(f"small keys {dt} {T} {fmt}")
        rng = np.random.default_rng(28)
        q = np.ldexp(rng.uniform(-1, 1, (T, 4, 128)), query).astype(np.float32)
        k = np.ldexp(rng.standard_normal((300, 2, 128)), key).astype(np.float32)
        v = np.ldexp(rng.standard_normal((300, 2, 128)), value).astype(np.float32)
        if f == mx.E4M3:  # (whole multiples of 1/32 of the size: in the type to the bit)
            k = np.ldexp(np.rint(np.ldexp(k, 5 - key)), key - 5).astype(np.float32)
            v = np.ldexp(np.rint(np.ldexp(v, 5 - value)), value - 5).astype(np.float32)
        y, want, tol = _one(q, k, v, dt, scale=2.0 ** (-key - query - 3), fmt=f)
        assert (np.abs(y - want) <= tol).all(), (dt, (np.abs(y - want) / tol).max())


def test_heads_with_any_strides():
    """Queries laid out [heads, tokens, channels], keys from a wider row."""
    import torch

    log("strides")
    rng = np.random.default_rng(25)
    cache = ref.Cache(rng, [90, 60], 2, 32, 64, mx.E4M3)
    args = (dev(cache.table, torch), dev(np.array([90, 60], np.int32), torch),
            dev(np.array([0, 40, 45], np.int32), torch))
    held = on_gpu(torch, cache.arrays())
    q = torch.randn(45, 6, 64, device="cuda", dtype=torch.float16)
    want = sq.attention_kv_mx(q, held, *args, fmt=mx.E4M3)
    got = sq.attention_kv_mx(q.transpose(0, 1).contiguous().transpose(0, 1), held, *args, fmt=mx.E4M3)
    k = torch.randn(45, 2, 64, device="cuda", dtype=torch.float16)
    slots = torch.arange(45, device="cuda")
    f, _ = sq.rope_frequencies(32)
    a = sq.new_kv_cache_mx(4, 2, 16, 64)
    b = sq.new_kv_cache_mx(4, 2, 16, 64)
    p = torch.arange(45, device="cuda") * 1000
    turn = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    y = sq.rope_quantize_kv_mx(q, k, k + 1, slots, a, positions=p, inv_freq=f)
    z = sq.rope_quantize_kv_mx(turn(q), turn(k), turn(k + 1), slots, b, positions=p, inv_freq=f)
    torch.cuda.synchronize()
    assert torch.equal(want, got) and torch.equal(y, z)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


# ------------------------------------------------------ one call after another

def _layer(torch, tokens, hidden, q_heads, heads, dim, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    n = (q_heads + 2 * heads) * dim
    return dict(x=r(tokens, hidden).to(torch.bfloat16), gamma=1 + 0.1 * r(hidden),
                qkv=sq.smooth_weights_mxfp4(r(n, hidden) / hidden ** 0.5),
                o=sq.smooth_weights_mxfp4(r(hidden, q_heads * dim) / (q_heads * dim) ** 0.5))


def _step(w, x, q_heads, heads, dim, cache, slots, positions, table, lens, cu, max_q, f):
    """Norm -> MX -> q|k|v product -> rotary and write -> attention -> MX ->
    output product, every step a call of the library."""
    import torch

    xq, xs = sq.norm_quantize_act_mx(x, w["gamma"], norm=sq.SQ_NORM_RMS, fmt=sq.SQ_MX_E4M3)
    qkv = sq.gemm_mxfp4(xq, xs, *w["qkv"], sq.SQ_MX_E4M3, out_dtype=torch.bfloat16)
    qkv = qkv.view(x.shape[0], q_heads + 2 * heads, dim)
    q = sq.rope_quantize_kv_mx(qkv[:, :q_heads], qkv[:, q_heads:q_heads + heads], qkv[:, q_heads + heads:],
                               slots, cache, positions=positions, inv_freq=f)
    y = sq.attention_kv_mx(q, cache, table, lens, cu, max_q=max_q)
    yq, ys = sq.quantize_act_mx(y.view(x.shape[0], -1), fmt=sq.SQ_MX_E4M3)
    return q, y, sq.gemm_mxfp4(yq, ys, *w["o"], sq.SQ_MX_E4M3, out_dtype=torch.bfloat16)


def test_a_layer_from_norm_to_output():
    """Two prompts, then three tokens of each by single steps: the attention of
    each call against 64 bits on the queries and cache that it saw, and the
    queries of each single step against those of the whole sequences in one
    call."""
    import torch

    log("a layer's calls in a row")
    hidden, q_heads, heads, dim, page = 512, 8, 2, 128, 16
    lens, more = [37, 70], 3
    total = [n + more for n in lens]
    w = _layer(torch, sum(total), hidden, q_heads, heads, dim, 31)
    f, _ = sq.rope_frequencies(dim)
    pages = [-(-n // page) for n in total]
    table = torch.full((2, max(pages)), -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(sum(pages)).to(torch.int32).cuda()
    table[0, :pages[0]], table[1, :pages[1]] = order[:pages[0]], order[pages[0]:]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731

    def place(b, t):
        return table[b, t // page].to(torch.int64) * page + t % page

    def call(cache, spans):
        """spans: (first token, end) of each sequence, x in the order of tokens."""
        rows = torch.cat([torch.arange(a, e, device="cuda") + sum(total[:b]) for b, (a, e) in enumerate(spans)])
        t = [torch.arange(a, e, device="cuda") for a, e in spans]
        slots = torch.cat([place(b, i) for b, i in enumerate(t)])
        new = [e - a for a, e in spans]
        out = _step(w, w["x"][rows], q_heads, heads, dim, cache, slots, torch.cat(t), table,
                    i32([e for _, e in spans]), i32(np.cumsum([0] + new).tolist()), max(new), f)
        torch.cuda.synchronize()
        return out

    def check(cache, q, y, spans):
        k, v = sq.dequantize_kv_mx(cache, table, i32(np.cumsum([0] + [e for _, e in spans]).tolist()),
                                   sum(e for _, e in spans), out_dtype=torch.float32)
        torch.cuda.synchronize()
        k, v, at, kt = host(k, torch), host(v, torch), 0, 0
        for a, e in spans:
            want, tol = ref.attention(q[at:at + e - a].double().cpu().numpy(), k[kt:kt + e].astype(np.float64),
                                      v[kt:kt + e].astype(np.float64), "bf16", dim ** -0.5)
            assert (np.abs(y[at:at + e - a].double().cpu().numpy() - want) <= tol).all()
            at, kt = at + e - a, kt + e

    steps = sq.new_kv_cache_mx(sum(pages), heads, page, dim)
    spans = [(0, n) for n in lens]
    q, y, _ = call(steps, spans)
    check(steps, q, y, spans)
    tails = []
    for i in range(more):
        spans = [(n + i, n + i + 1) for n in lens]
        q, y, z = call(steps, spans)
        check(steps, q, y, spans)
        tails.append((q, y, z))
    whole = sq.new_kv_cache_mx(sum(pages), heads, page, dim)
    spans = [(0, n) for n in total]
    q, y, z = call(whole, spans)
    check(whole, q, y, spans)
    # the same queries: the products' sums differ in their order (512 terms: far
    # below a step of bf16), so their outputs are equal or neighbours (2^-7 of
    # the value), and a rotated pair differs by 2^-7 of both, rounded again
    for i in range(more):
        for b in range(2):
            one, all_ = tails[i][0][b].float(), q[sum(total[:b]) + lens[b] + i].float()
            assert (one - all_).norm() <= 2.0 ** -6 * all_.norm(), (i, b)


def test_captured_steps_replay():
    """Write and attention of a decode step in two graphs that take turns, each
    with a pool of its own; lengths, slots and positions change between the
    replays, eager work runs in between."""
    import torch

    log("graphs")
    rng = np.random.default_rng(41)
    lens = [40, 300, 7]
    cache = ref.Cache(rng, [n + 40 for n in lens], 2, 16, 128, mx.E2M1)
    table, f = dev(cache.table, torch), sq.rope_frequencies(64)[0]
    held = on_gpu(torch, cache.arrays())
    eager = tuple(t.clone() for t in held)
    qkv = torch.randn(3, 12, 128, device="cuda", dtype=torch.bfloat16)
    state = dict(slots=torch.zeros(3, dtype=torch.int64, device="cuda"),
                 pos=torch.zeros(3, dtype=torch.int64, device="cuda"),
                 n=torch.zeros(3, dtype=torch.int32, device="cuda"))

    def step(c):
        q = sq.rope_quantize_kv_mx(qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], state["slots"], c,
                                   positions=state["pos"], inv_freq=f)
        y = sq.attention_kv_mx(q, c, table, state["n"])
        k, v = sq.dequantize_kv_mx(c, table[:1], torch.cat([state["n"][:1] * 0, state["n"][:1]]), 80)
        return y, k, v

    def move(i):
        state["n"].copy_(torch.tensor([n + i + 1 for n in lens], dtype=torch.int32))
        state["pos"].copy_(torch.tensor([n + i for n in lens]))
        state["slots"].copy_(torch.tensor([int(cache.slots(b)[n + i]) for b, n in enumerate(lens)]))
        qkv.normal_()

    move(0)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step(held)  # (the library and the allocator, once)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(held)
        graphs.append((g, out))
    for i in range(12):
        move(i)
        g, out = graphs[i % 2]
        g.replay()
        want = step(eager)
        torch.randn(1 << 16, device="cuda").sum()
        torch.cuda.synchronize()
        assert torch.equal(out[0].view(torch.int16), want[0].view(torch.int16)), i
        n = lens[0] + i + 1
        for a, b in zip(out[1:], want[1:]):
            assert torch.equal(a[:n].view(torch.int16), b[:n].view(torch.int16)), i
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), i


def test_prompts_in_a_graph():
    """The tile kernel with its keys split, and both kernels together."""
    import torch

    log("prompts in a graph")
    rng = np.random.default_rng(42)
    lens, new = [900, 400, 130], [60, 1, 50]
    cache = ref.Cache(rng, lens, 2, 16, 64, mx.E4M3)
    held, table = on_gpu(torch, cache.arrays()), dev(cache.table, torch)
    q = torch.randn(111, 6, 64, device="cuda", dtype=torch.float16)
    n, cu = dev(np.array(lens, np.int32), torch), dev(np.cumsum([0] + new).astype(np.int32), torch)
    call = lambda: sq.attention_kv_mx(q, held, table, n, cu, fmt=mx.E4M3, max_q=60)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for i in range(4):
        q.normal_()
        n.copy_(torch.tensor([k - i for k in lens], dtype=torch.int32))
        g.replay()
        want = call()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)), i


def test_calls_at_once_on_two_streams():
    """Two calls that run at the same time have workspaces of their own, and new
    outputs belong to the stream that writes them."""
    import torch

    from tests.test_mx_streams_gpu import _pool_of

    log("two streams")
    rng = np.random.default_rng(43)
    cases = []
    for b in range(2):
        cache = ref.Cache(rng, [3000 + 500 * b], 2, 16, 128, mx.E2M1)
        cases.append((torch.randn(1, 8, 128, device="cuda", dtype=torch.bfloat16), on_gpu(torch, cache.arrays()),
                      dev(cache.table, torch), dev(np.array(cache.lens, np.int32), torch)))
    want = [sq.attention_kv_mx(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        got = [sq.attention_kv_mx(*c, stream=s) for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    s = streams[0]
    q, held, table, n = cases[0]
    slots = torch.arange(1, device="cuda")
    made = {
        "attention_kv_mx": lambda st: (sq.attention_kv_mx(q, held, table, n, stream=st),),
        "rope_quantize_kv_mx": lambda st: (sq.rope_quantize_kv_mx(q, q[:, :2], q[:, 2:4], slots, held, stream=st),),
        "dequantize_kv_mx": lambda st: sq.dequantize_kv_mx(held, table, dev(np.array([0, 5], np.int32), torch), 5,
                                                           stream=st),
    }
    torch.cuda.synchronize()
    for name, call in made.items():
        mine, others = call(None), call(s)
        torch.cuda.synchronize()
        for t, u in zip(mine, others):
            assert _pool_of(torch, u) == s.cuda_stream, name
            assert _pool_of(torch, t) == torch.cuda.current_stream().cuda_stream, name
            assert torch.equal(t.view(torch.int16), u.view(torch.int16)), name


# ---------------------------------------------------------- bounds and offsets

@pytest.mark.parametrize("lens,new,q_heads,dim", [((700, 40), (1, 1), 8, 128), ((700, 40), (30, 2), 8, 64),
                                                  ((700, 40), (30, 2), 8, 256)])
def test_nothing_outside_outputs_and_workspace(lens, new, q_heads, dim):
    import torch

    log(f"guards {lens} {new} {dim}")
    rng = np.random.default_rng(51)
    cache = ref.Cache(rng, lens, 2, 16, dim, mx.E2M1)
    held, table = on_gpu(torch, cache.arrays()), dev(cache.table, torch)
    T = sum(new)
    need = sq.attention_kv_mx_workspace(T, q_heads, held, len(lens), table.shape[1], max(new))
    work = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    whole = torch.full((T + 2, q_heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.randn(T, q_heads, dim, device="cuda", dtype=torch.bfloat16)
    cu = dev(np.cumsum([0] + list(new)).astype(np.int32), torch)
    n = dev(np.array(lens, np.int32), torch)
    y = sq.attention_kv_mx(q, held, table, n, cu, max_q=max(new), out=whole[1:-1], workspace=work[:need])
    want = sq.attention_kv_mx(q, held, table, n, cu, max_q=max(new))
    torch.cuda.synchronize()
    assert (whole[0] == 7).all() and (whole[-1] == 7).all() and (work[need:] == 0xA5).all()
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))
    for t, a in zip(held, cache.arrays()):
        assert_bits_equal(host(t, torch), a, "the cache")
    with pytest.raises(sq.SQError):
        sq.attention_kv_mx(q, held, table, n, cu, max_q=max(new), workspace=work[:need - 16])


def test_a_cache_past_four_gib():
    """Pages whose codes begin past 2^32 bytes: written, read and attended."""
    import torch

    log("a cache of 4.8 GiB a side")
    heads, dim, page, pages = 64, 256, 32, 9500  # 16 KB a token, 5e9 bytes of e4m3 codes
    kq, vq = (torch.empty(pages, heads, page, dim, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty(pages, heads, page, dim // 32, dtype=torch.uint8, device="cuda") for _ in range(2))
    cache = (kq, ks, vq, vs)
    assert kq.numel() > 1 << 32
    n = 70
    ids = [pages - 1, 5, pages - 2]
    rng = np.random.default_rng(52)
    k, v = (rng.standard_normal((n, heads, dim)).astype(np.float32) for _ in range(2))
    t = np.arange(n)
    slots = np.array(ids)[t // page] * page + t % page
    sq.rope_quantize_kv_mx(None, dev(k, torch), dev(v, torch), dev(slots, torch), cache, fmt=mx.E4M3)
    table, cu = dev(np.array([ids], np.int32), torch), dev(np.array([0, n], np.int32), torch)
    gk, gv = sq.dequantize_kv_mx(cache, table, cu, n, fmt=mx.E4M3, out_dtype=torch.float32)
    torch.cuda.synchronize()
    want = [ref.values(*ref.quantized(x, mx.E4M3), mx.E4M3) for x in (k, v)]
    assert_bits_equal(host(gk, torch), want[0].astype(np.float32), "k")
    assert_bits_equal(host(gv, torch), want[1].astype(np.float32), "v")
    for T in (1, 20):
        q = to_dt(rng.standard_normal((T, heads, dim)), "bf16")
        y = sq.attention_kv_mx(dev(q, torch), cache, table, dev(np.array([n], np.int32), torch),
                               dev(np.array([0, T], np.int32), torch), fmt=mx.E4M3, max_q=T)
        torch.cuda.synchronize()
        w, tol = ref.attention(mx.to_f32(q).astype(np.float64), *want, "bf16", dim ** -0.5)
        assert (np.abs(y.float().cpu().numpy() - w) <= tol).all()


def test_many_queries_of_many_heads_without_workspace():
    """More than 32 heads share a key head: tiles alone, and so many that their
    keys are not split: no workspace is needed."""
    import torch

    log("48 heads a key head, 1200 sequences")
    rng = np.random.default_rng(53)
    lens = [int(x) for x in rng.integers(0, 40, 1200)]
    cache = ref.Cache(rng, lens, 1, 16, 64, mx.E2M1)
    q = to_dt(rng.standard_normal((1200, 48, 64)), "bf16")
    held, table = on_gpu(torch, cache.arrays()), dev(cache.table, torch)
    assert sq.attention_kv_mx_workspace(1200, 48, held, 1200, table.shape[1], 1) == 0
    y = sq.attention_kv_mx(dev(q, torch), held, table, dev(np.array(lens, np.int32), torch))
    torch.cuda.synchronize()
    got = y.float().cpu().numpy()
    for b in range(0, 1200, 7):
        want, tol = ref.attention(mx.to_f32(q[b:b + 1]).astype(np.float64), *cache.read(b), "bf16", 0.125)
        assert (np.abs(got[b] - want[0]) <= tol[0]).all(), b


def test_the_binding_refuses():
    import torch

    c = sq.new_kv_cache_mx(4, 2, 16, 64)
    q = torch.zeros(3, 4, 64, device="cuda", dtype=torch.float16)
    k = q[:, :2]
    i64 = torch.zeros(3, dtype=torch.int64, device="cuda")
    table = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    n = torch.ones(3, dtype=torch.int32, device="cuda")
    f, _ = sq.rope_frequencies(64)
    write = lambda **kw: sq.rope_quantize_kv_mx(**{**dict(q=q, k=k, v=k, slots=i64, cache=c), **kw})  # noqa: E731
    att = lambda **kw: sq.attention_kv_mx(**{**dict(q=q, cache=c, table=table, seq_lens=n), **kw})  # noqa: E731
    read = lambda **kw: sq.dequantize_kv_mx(**{**dict(cache=c, table=table, cu=torch.zeros(4, dtype=torch.int32,
                                                      device="cuda"), total=3), **kw})  # noqa: E731
    write(), att(), read()
    bad_cache = (c[0], c[1][:, :1].contiguous(), c[2], c[3])
    for call, kw in [
        (write, dict(cache=bad_cache)), (write, dict(cache=(c[0].to(torch.int8),) + c[1:])),
        (write, dict(fmt=sq.SQ_MX_E4M3)), (write, dict(fmt=7)), (write, dict(v=k.float())),
        (write, dict(k=q)), (write, dict(slots=None)), (write, dict(slots=i64[:2])),
        (write, dict(slots=i64.to(torch.int32))), (write, dict(inv_freq=f)),
        (write, dict(inv_freq=f.float(), positions=i64)), (write, dict(inv_freq=f[:9], positions=i64)),
        (write, dict(q=q[:2])), (write, dict(q=q.float())), (write, dict(q=q, out=q)),
        (write, dict(q=None, out=q)), (write, dict(q_mul=torch.ones(64, device="cuda"))),
        (write, dict(k_mul=torch.ones(2, 64, device="cuda", dtype=torch.float16))),
        (write, dict(k=k.cpu())), (write, dict(k=q[:, :2, ::2])),
        (att, dict(cache=bad_cache)), (att, dict(q=q.float())), (att, dict(q=q[:, :3])), (att, dict(q=q[:, :0])),
        (att, dict(q=q[:2])), (att, dict(seq_lens=n[:2])), (att, dict(seq_lens=None)), (att, dict(table=table[0])),
        (att, dict(table=table.to(torch.int64))), (att, dict(cu_q=n)), (att, dict(window=-1)), (att, dict(out=q)),
        (att, dict(out=q[:2])), (att, dict(cu_q=torch.zeros(4, dtype=torch.int32, device="cuda"), max_q=0)),
        (att, dict(workspace=torch.zeros(9, device="cuda"))),
        (read, dict(cu=n)), (read, dict(cu=None)), (read, dict(total=-1)), (read, dict(out_dtype=torch.int8)),
        (read, dict(out=(q, q))), (read, dict(table=table.cpu())),
    ]:
        with pytest.raises(ValueError):
            call(**kw)
    odd = torch.zeros(3, 2 * 64 + 4, device="cuda", dtype=torch.float16)[:, :128].view(3, 2, 64)
    with pytest.raises(sq.SQError):  # rows that are not whole 16-byte vectors
        write(q=None, k=odd)
    with pytest.raises(sq.SQError):
        att(scale=float("inf"))
    # no tokens, no sequences: nothing to do
    assert write(q=q[:0], k=k[:0], v=k[:0], slots=i64[:0]).shape == (0, 4, 64)
    assert att(q=q[:0], table=table[:0], seq_lens=n[:0]).shape == (0, 4, 64)
    assert read(total=0)[0].shape == (0, 2, 64)


def test_the_binding_refuses_outputs_that_are_one():
    import torch

    c = sq.new_kv_cache_mx(4, 2, 16, 64)
    k = torch.zeros(3, 2, 64, device="cuda", dtype=torch.float16)
    with pytest.raises(sq.SQError):
        sq.rope_quantize_kv_mx(None, k, k, torch.arange(3, device="cuda"), (c[0], c[1], c[0], c[1]))
    with pytest.raises(sq.SQError):
        sq.dequantize_kv_mx(c, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                            torch.tensor([0, 3], dtype=torch.int32, device="cuda"), 3, out=(k, k))


def test_outputs_inside_inputs_refuse_and_neighbours_do_not():
    """Outputs that begin inside the queries, or lie in part over one another,
    are refused; ones that end where an input begins, or lie in the gap between
    two heads' queries, are not."""
    import torch

    log("outputs beside and inside inputs")
    T, heads, dim, n = 6, 2, 64, 6 * 2 * 64
    c = sq.new_kv_cache_mx(4, heads, 16, dim)
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    lens, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([20], [0, T]))
    k = torch.randn(20, heads, dim, device="cuda", dtype=torch.float16)
    sq.rope_quantize_kv_mx(None, k, k, torch.arange(20, device="cuda"), c)
    buf = torch.randn(4 * n, device="cuda", dtype=torch.float16)
    rows = lambda at: buf[at:at + n].view(T, heads, dim)  # noqa: E731
    att = lambda q, **kw: sq.attention_kv_mx(q, c, table, lens, cu, max_q=T, **kw)  # noqa: E731
    write = lambda q, **kw: sq.rope_quantize_kv_mx(q, k[:T], k[:T], torch.full((T,), -1, device="cuda"), c, **kw)  # noqa: E731
    q = rows(n)
    want, turned = att(q.clone()), write(q.clone())
    for at in (n - 8, n + 8, 2 * n - 8, 8):
        for call in (att, write):
            with pytest.raises(sq.SQError):
                call(q, out=rows(at))
        with pytest.raises(sq.SQError):
            sq.dequantize_kv_mx(c, table, cu, T, out=(rows(n), rows(at)))
    saved = q.clone()
    for at in (0, 2 * n):
        for call, w in ((att, want), (write, turned)):
            y = call(q, out=rows(at))
            torch.cuda.synchronize()
            assert torch.equal(y, w) and torch.equal(q, saved)
    # head 0's queries, room for an output, head 1's
    far = torch.as_strided(buf, (T, heads, dim), (dim, T * dim + n, 1), 0)
    far.copy_(saved)
    for call, w in ((att, want), (write, turned)):
        y = call(far, out=rows(T * dim))
        torch.cuda.synchronize()
        assert torch.equal(y, w) and torch.equal(far, saved)
        for at in (T * dim - 8, T * dim + 8):
            with pytest.raises(sq.SQError):
                call(far, out=rows(at))


def test_whole_numbers_past_64_bits():
    """A window or a number of queries past 64 bits is as good as none, a
    rotary layout of that kind is no layout."""
    import torch

    log("numbers past 64 bits")
    rng = np.random.default_rng(71)
    cache = ref.Cache(rng, [90, 70], 2, 16, 64, mx.E2M1)
    held, table = on_gpu(torch, cache.arrays()), dev(cache.table, torch)
    q = torch.randn(45, 4, 64, device="cuda", dtype=torch.bfloat16)
    n, cu = dev(np.array([90, 70], np.int32), torch), dev(np.array([0, 40, 45], np.int32), torch)
    call = lambda **kw: sq.attention_kv_mx(q, held, table, n, cu, out=torch.full_like(q, 3.0), **kw)  # noqa: E731
    want, most, need = call(max_q=40), call(), sq.attention_kv_mx_workspace(45, 4, held, 2, table.shape[1], 45)
    for big in ((1 << 64) + 1, 1 << 64, (1 << 63) + 1, 1 << 80):
        y, z = call(max_q=40, window=big), call(max_q=big)
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), want.view(torch.int16)), big
        assert torch.equal(z.view(torch.int16), most.view(torch.int16)), big
        assert sq.attention_kv_mx_workspace(45, 4, held, 2, table.shape[1], big) == need
        with pytest.raises(sq.SQError):
            sq.rope_quantize_kv_mx(q, q[:, :2], q[:, 2:], torch.full((45,), -1, device="cuda"), held, layout=big)
    for small in (-1, -(1 << 64) + 1, -(1 << 80)):
        for kw in (dict(window=small), dict(max_q=small)):
            with pytest.raises(ValueError):
                call(**kw)
        assert sq.attention_kv_mx_workspace(45, 4, held, 2, table.shape[1], small) == 0
