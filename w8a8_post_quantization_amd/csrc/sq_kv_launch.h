// Internal launchers behind include/sq_kv.h.  Arguments arrive validated; each
// launcher only enqueues kernels on `stream`.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sq {

// The cache as the kernels take it (fmt 0 e2m1, 1 e4m3).
struct KvCache {
    uint8_t *kq, *ks, *vq, *vs;
    int64_t pages;
    int heads, page_log, dim, fmt;
};

struct RopeWrite {
    const void *q, *k, *v;  // q NULL: q_heads = 0
    int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh;  // strides in elements: token, head
    int64_t T;
    int q_heads;
    const int64_t *positions;
    const double *inv_freq;
    int rotary, layout;
    double amplitude;
    const float *q_mul, *k_mul;
    const int64_t *slots;
    KvCache cache;
    void *q_out;
};
void launch_rope_write(const RopeWrite &a, int dt, hipStream_t stream);

struct KvRead {
    KvCache cache;
    const int32_t *table;
    int64_t width;
    const int32_t *cu;
    int B;
    int64_t total;
    void *k, *v;
};
void launch_kv_read(const KvRead &a, int dt, hipStream_t stream);

struct KvAttention {
    const void *q;
    int64_t q_st, q_sh;
    void *y;
    KvCache cache;
    const int32_t *table;
    int64_t width;
    const int32_t *seq_lens;
    const int32_t *cu_q;  // or NULL: one query a sequence
    int64_t T;
    int B, q_heads, group;  // group = q_heads / cache.heads
    float scale;
    int causal;
    int64_t window;  // 0: none
    void *work;
};
size_t kv_attention_workspace(int64_t T, int q_heads, int heads, int dim, int fmt, int B, int64_t keys,
                              int64_t max_q);
// The tile kernel: sequences of rows_min rows and more, 4 or 8 waves a block,
// the keys in so many splits (their parts, where there are several, in `parts`).
void launch_kv_tiles(const KvAttention &a, int dt, int waves, int rows_min, int splits, float *parts,
                     hipStream_t stream);
void launch_kv_attention(const KvAttention &a, int64_t max_q, int dt, hipStream_t stream);

}  // namespace sq
