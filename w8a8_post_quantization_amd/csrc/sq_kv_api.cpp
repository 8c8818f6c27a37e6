// C ABI of the microscaled cache of keys and values (include/sq_kv.h):
// argument validation on the host, then kernel launches on the caller's stream.
#include "../../include/sq_kv.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "sq_kv_launch.h"

namespace {

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline size_t esize(int dt) { return dt == SQ_F32 ? 4 : 2; }
inline bool valid_dt(int dt) { return dt == SQ_F32 || dt == SQ_F16 || dt == SQ_BF16; }
inline hipStream_t st(void *s) { return reinterpret_cast<hipStream_t>(s); }
int finish() { return hipGetLastError() == hipSuccess ? SQ_OK : SQ_ERR_HIP; }

constexpr int64_t kMaxTokens = 1 << 24, kMaxHeads = 65535, kMaxSlots = 0x7fffffff,
                  kMaxKeys = 1 << 30;

inline bool power_of_two(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }

// The cache's own members, and the kernels' form of it.
int check_cache(const sq_kv_cache *c, sq::KvCache &out) {
    if (!c) return SQ_ERR_NULL;
    if (c->fmt != SQ_MX_E2M1 && c->fmt != SQ_MX_E4M3) return SQ_ERR_ARG;
    if (c->dim <= 0 || c->dim % 32) return SQ_ERR_SHAPE;
    if (c->dim != 64 && c->dim != 128 && c->dim != 256) return SQ_ERR_UNSUPPORTED;
    if (!power_of_two(c->page) || c->page < 16 || c->page > 1 << 20) return SQ_ERR_SHAPE;
    if (c->pages < 1 || c->heads < 1 || c->heads > kMaxHeads) return SQ_ERR_SHAPE;
    if (c->pages > kMaxSlots / c->page) return SQ_ERR_UNSUPPORTED;
    out.pages = c->pages;
    out.heads = (int)c->heads;
    out.page_log = __builtin_ctzll((unsigned long long)c->page);
    out.dim = (int)c->dim;
    out.fmt = c->fmt;
    out.kq = c->kq;
    out.ks = c->ks;
    out.vq = c->vq;
    out.vs = c->vs;
    return SQ_OK;
}

int check_arrays(const sq_kv_cache *c) {
    if (!c->kq || !c->ks || !c->vq || !c->vs) return SQ_ERR_NULL;
    if (!aligned(c->kq, 16) || !aligned(c->vq, 16) || !aligned(c->ks, 4) || !aligned(c->vs, 4)) return SQ_ERR_ALIGN;
    return SQ_OK;
}

// Rows of whole 16-byte vectors.
int check_rows(const void *x, const int64_t stride[2], int dt) {
    if (!x || !stride) return SQ_ERR_NULL;
    if (stride[0] < 0 || stride[1] < 0) return SQ_ERR_SHAPE;
    const int64_t n = 16 / (int64_t)esize(dt);
    if (!aligned(x, 16) || stride[0] % n || stride[1] % n) return SQ_ERR_ALIGN;
    // (a token's offset, in bytes, stays within 63 bits)
    if (stride[0] > (int64_t)1 << 36 || stride[1] > (int64_t)1 << 36) return SQ_ERR_UNSUPPORTED;
    return SQ_OK;
}

// What the shapes of an attention call have to be.
int check_attention(int64_t T, int64_t q_heads, const sq::KvCache &c, int64_t B, int64_t width, int64_t max_q) {
    if (T < 0 || B < 0 || width < 0 || max_q < 0 || q_heads < 1) return SQ_ERR_SHAPE;
    if (q_heads % c.heads) return SQ_ERR_SHAPE;
    if (q_heads > kMaxHeads || T > kMaxTokens || B > kMaxTokens) return SQ_ERR_UNSUPPORTED;
    // (grids of fewer than 2^32 threads; keys, and tiles of keys of a sequence's
    // heads, counted in 31 bits)
    if (T * q_heads > (int64_t)1 << 29 || B * c.heads > (int64_t)1 << 22) return SQ_ERR_UNSUPPORTED;
    if (width > kMaxKeys >> c.page_log) return SQ_ERR_UNSUPPORTED;
    if (((width << c.page_log) >> 7) * c.heads > kMaxKeys) return SQ_ERR_UNSUPPORTED;
    return SQ_OK;
}

// The bytes of a dense operand.
struct Span {
    int64_t at, n;
};
inline Span span(const void *p, int64_t n) { return {(int64_t)(uintptr_t)p, p ? n : 0}; }
inline bool meet(const Span &a, const Span &b) { return a.n && b.n && a.at < b.at + b.n && b.at < a.at + a.n; }

// Whether an output meets any of these, or one of [T, heads] strided rows of n
// bytes.  Rows are looked at a head at a time where the output lies between the
// first's beginning and the last's end: it may lie between rows.
template <int N>
bool meet_any(const Span &out, const Span (&in)[N]) {
    for (const Span &s : in)
        if (meet(out, s)) return true;
    return false;
}
bool meet_rows(const Span &out, const void *x, const int64_t stride[2], int dt, int64_t T, int64_t heads, int64_t n) {
    const int64_t at = (int64_t)(uintptr_t)x, token = stride[0] * (int64_t)esize(dt), head = stride[1] * (int64_t)esize(dt);
    if (!meet(out, {at, (T - 1) * token + (heads - 1) * head + n})) return false;
    for (int64_t h = 0; h < heads; ++h) {
        const int64_t first = at + h * head;
        // the first token whose row ends behind the output's beginning
        const int64_t short_of = out.at - n - first;
        const int64_t t = short_of < 0 ? 0 : token ? short_of / token + 1 : T;
        if (t < T && first + t * token < out.at + out.n) return true;
    }
    return false;
}

// The bytes of the cache's arrays, keys first.
struct CacheSpans {
    Span kq, ks, vq, vs;
};
CacheSpans cache_spans(const sq_kv_cache *c) {
    const int64_t rows = c->pages * c->page * c->heads, codes = c->fmt == SQ_MX_E2M1 ? c->dim / 2 : c->dim;
    return {span(c->kq, rows * codes), span(c->ks, rows * (c->dim / 32)), span(c->vq, rows * codes),
            span(c->vs, rows * (c->dim / 32))};
}

// No sequence has more queries than there are.
int64_t most_queries(int64_t max_q, int64_t T) { return max_q < T ? max_q : T; }

}  // namespace

extern "C" {

int sq_rope_quantize_kv_mx(const void *q, const int64_t q_stride[2], const void *k,
                           const int64_t k_stride[2], const void *v, const int64_t v_stride[2],
                           int dt, int64_t T, int64_t q_heads, const int64_t *positions,
                           const double *inv_freq, int64_t rotary, double amplitude, int layout,
                           const float *q_mul, const float *k_mul, const int64_t *slots,
                           const sq_kv_cache *cache, void *q_out, void *stream) {
    if (!valid_dt(dt)) return SQ_ERR_DTYPE;
    sq::RopeWrite a = {};
    if (const int e = check_cache(cache, a.cache)) return e;
    if (layout != SQ_ROPE_HALF && layout != SQ_ROPE_INTERLEAVED) return SQ_ERR_ARG;
    if (rotary && !std::isfinite(amplitude)) return SQ_ERR_ARG;
    if (T < 0 || rotary < 0 || rotary > cache->dim || rotary % 16) return SQ_ERR_SHAPE;
    if (q && (q_heads < 1 || q_heads > kMaxHeads)) return SQ_ERR_SHAPE;
    if (T > kMaxTokens) return SQ_ERR_UNSUPPORTED;
    if (T == 0) return SQ_OK;
    if (const int e = check_arrays(cache)) return e;
    if (const int e = check_rows(k, k_stride, dt)) return e;
    if (const int e = check_rows(v, v_stride, dt)) return e;
    if (q) {
        if (const int e = check_rows(q, q_stride, dt)) return e;
        if (!q_out) return SQ_ERR_NULL;
        if (!aligned(q_out, 16) || !aligned(q_mul, 16)) return SQ_ERR_ALIGN;
    }
    if (!slots || (rotary && (!positions || !inv_freq))) return SQ_ERR_NULL;
    if (!aligned(slots, 8) || !aligned(k_mul, 16) || !aligned(positions, 8) || !aligned(inv_freq, 8))
        return SQ_ERR_ALIGN;
    // Nothing that the call writes lies over what it reads or over one another.
    const CacheSpans c = cache_spans(cache);
    const int64_t row = cache->dim * (int64_t)esize(dt);
    const Span out = span(q ? q_out : nullptr, T * q_heads * row);
    const Span written[5] = {c.kq, c.ks, c.vq, c.vs, out};
    const Span read[5] = {span(slots, T * 8), span(rotary ? positions : nullptr, T * 8),
                          span(rotary ? inv_freq : nullptr, rotary / 2 * 8),
                          span(q ? q_mul : nullptr, q_heads * cache->dim * 4),
                          span(k_mul, cache->heads * cache->dim * 4)};
    for (int i = 0; i < 5; ++i) {
        if (!written[i].n) continue;
        for (int j = 0; j < i; ++j)
            if (meet(written[i], written[j])) return SQ_ERR_ARG;
        if (meet_any(written[i], read) || meet_rows(written[i], k, k_stride, dt, T, cache->heads, row) ||
            meet_rows(written[i], v, v_stride, dt, T, cache->heads, row) ||
            (q && meet_rows(written[i], q, q_stride, dt, T, q_heads, row)))
            return SQ_ERR_ARG;
    }
    a.q = q;
    a.k = k;
    a.v = v;
    if (q) {
        a.q_st = q_stride[0];
        a.q_sh = q_stride[1];
        a.q_heads = (int)q_heads;
        a.q_mul = q_mul;
        a.q_out = q_out;
    }
    a.k_st = k_stride[0];
    a.k_sh = k_stride[1];
    a.v_st = v_stride[0];
    a.v_sh = v_stride[1];
    a.T = T;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.rotary = (int)rotary;
    a.layout = layout;
    a.amplitude = amplitude;
    a.k_mul = k_mul;
    a.slots = slots;
    sq::launch_rope_write(a, dt, st(stream));
    return finish();
}

int sq_dequantize_kv_mx(const sq_kv_cache *cache, const int32_t *table, int64_t B, int64_t width,
                        const int32_t *cu, int64_t total, void *k, void *v, int dt, void *stream) {
    if (!valid_dt(dt)) return SQ_ERR_DTYPE;
    sq::KvRead a = {};
    if (const int e = check_cache(cache, a.cache)) return e;
    if (B < 0 || width < 0 || total < 0) return SQ_ERR_SHAPE;
    if (B > kMaxTokens || width > kMaxSlots >> a.cache.page_log || total > kMaxTokens) return SQ_ERR_UNSUPPORTED;
    if (B == 0 || total == 0) return SQ_OK;
    if (const int e = check_arrays(cache)) return e;
    if (!cu || !k || !v || (width && !table)) return SQ_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(table, 4) || !aligned(cu, 4)) return SQ_ERR_ALIGN;
    const CacheSpans c = cache_spans(cache);
    const int64_t dense = total * cache->heads * cache->dim * (int64_t)esize(dt);
    const Span out_k = span(k, dense), out_v = span(v, dense);
    const Span read[6] = {c.kq, c.ks, c.vq, c.vs, span(table, B * width * 4), span(cu, (B + 1) * 4)};
    if (meet(out_k, out_v) || meet_any(out_k, read) || meet_any(out_v, read)) return SQ_ERR_ARG;
    a.table = table;
    a.width = width;
    a.cu = cu;
    a.B = (int)B;
    a.total = total;
    a.k = k;
    a.v = v;
    sq::launch_kv_read(a, dt, st(stream));
    return finish();
}

size_t sq_attention_kv_mx_workspace(int64_t T, int64_t q_heads, const sq_kv_cache *cache,
                                    int64_t B, int64_t width, int64_t max_q) {
    sq::KvCache c;
    if (check_cache(cache, c) || check_attention(T, q_heads, c, B, width, max_q)) return 0;
    if (T == 0 || B == 0) return 0;
    return sq::kv_attention_workspace(T, (int)q_heads, c.heads, c.dim, c.fmt, (int)B, width << c.page_log,
                                      most_queries(max_q, T));
}

int sq_attention_kv_mx(const void *q, const int64_t q_stride[2], int dt, int64_t T,
                       int64_t q_heads, const sq_kv_cache *cache, const int32_t *table, int64_t B,
                       int64_t width, const int32_t *seq_lens, const int32_t *cu_q, int64_t max_q,
                       float scale, int causal, int64_t window, void *y, void *workspace,
                       size_t workspace_bytes, void *stream) {
    if (dt != SQ_F16 && dt != SQ_BF16) return SQ_ERR_DTYPE;
    sq::KvAttention a = {};
    if (const int e = check_cache(cache, a.cache)) return e;
    if (const int e = check_attention(T, q_heads, a.cache, B, width, max_q)) return e;
    if (!std::isfinite(scale)) return SQ_ERR_ARG;
    if (window < 0) return SQ_ERR_ARG;
    if (!cu_q && T != B) return SQ_ERR_SHAPE;
    if (T == 0 || B == 0) return SQ_OK;
    if (max_q < 1) return SQ_ERR_SHAPE;
    if (const int e = check_arrays(cache)) return e;
    if (const int e = check_rows(q, q_stride, dt)) return e;
    if (!seq_lens || !y || (width && !table)) return SQ_ERR_NULL;
    if (!aligned(y, 16) || !aligned(table, 4) || !aligned(seq_lens, 4) || !aligned(cu_q, 4)) return SQ_ERR_ALIGN;
    const int64_t most = cu_q ? most_queries(max_q, T) : 1;
    const size_t need = sq::kv_attention_workspace(T, (int)q_heads, a.cache.heads, a.cache.dim, a.cache.fmt, (int)B,
                                                   width << a.cache.page_log, most);
    if (need && (!workspace || workspace_bytes < need)) return SQ_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return SQ_ERR_ALIGN;
    const CacheSpans c = cache_spans(cache);
    const int64_t row = cache->dim * (int64_t)esize(dt);
    const Span out = span(y, T * q_heads * row), work = span(workspace, (int64_t)need);
    const Span read[7] = {c.kq, c.ks, c.vq, c.vs, span(table, B * width * 4), span(seq_lens, B * 4),
                          span(cu_q, (B + 1) * 4)};
    if (meet(out, work) || meet_any(out, read) || meet_any(work, read) ||
        meet_rows(out, q, q_stride, dt, T, q_heads, row) || (need && meet_rows(work, q, q_stride, dt, T, q_heads, row)))
        return SQ_ERR_ARG;
    a.q = q;
    a.q_st = q_stride[0];
    a.q_sh = q_stride[1];
    a.y = y;
    a.table = table;
    a.width = width;
    a.seq_lens = seq_lens;
    a.cu_q = cu_q;
    a.T = T;
    a.B = (int)B;
    a.q_heads = (int)q_heads;
    a.group = (int)(q_heads / a.cache.heads);
    a.scale = scale;
    a.causal = causal != 0;
    // (no sequence has as many keys: kernels count places less the window in 64 bits)
    a.window = window > kMaxKeys ? 0 : window;
    a.work = workspace;
    sq::launch_kv_attention(a, most, dt, st(stream));
    return finish();
}

}  // extern "C"
