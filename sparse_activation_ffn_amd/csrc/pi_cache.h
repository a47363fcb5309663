// pi_cache.h -- the paged key/value cache as its kernels see it, and the checks
// of the descriptors that its entry points share.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pi.h"
#include "pi_device.h"
#include "pi_launch.h"

namespace pi {

// One layer of a cache.  Offsets are 64-bit throughout: a cache of 288 GB has
// more elements than 32 bits count.
struct CacheLayer {
    uint8_t* k;
    uint8_t* v;
    int pages, kv_heads, page_size, page_shift, head_dim;
};

// A batch of sequences (pi_seq_batch).
struct Batch {
    const int* q_start;
    const int* kv_len;
    const int* table;
    int n_seqs, n_tokens, table_stride;
};

inline int log2i(int v) { return 31 - __builtin_clz((unsigned)v); }
inline int dtype_size(int dt) { return dt == PI_F32 ? 4 : 2; }

inline int64_t layer_bytes(const pi_kv_cache* c) {
    return (int64_t)c->pages * c->kv_heads * c->page_size * c->head_dim * dtype_size(c->dtype);
}

inline CacheLayer cache_layer(const pi_kv_cache* c, int layer) {
    const int64_t off = layer * layer_bytes(c);
    return CacheLayer{(uint8_t*)c->k + off, (uint8_t*)c->v + off, c->pages, c->kv_heads, c->page_size,
                      log2i(c->page_size), c->head_dim};
}

inline Batch seq_batch(const pi_seq_batch* b) {
    return Batch{b->q_start, b->kv_len, b->table, b->n_seqs, b->n_tokens, b->table_stride};
}

// ---- argument checks ------------------------------------------------------------
inline bool page_size_ok(int ps) { return ps >= 8 && ps <= PI_MAX_PAGE_SIZE && (ps & (ps - 1)) == 0; }

inline pi_status check_cache(const pi_kv_cache* c) {
    CHECK(c, PI_ERR_ARG, "NULL cache");
    CHECK(c->dtype == PI_F32 || c->dtype == PI_F16, PI_ERR_DTYPE, "cache: dtype must be PI_F32 or PI_F16");
    CHECK(c->layers >= 1 && c->kv_heads >= 1 && c->kv_heads <= 65535, PI_ERR_SHAPE,
          "cache: layers >= 1 and kv_heads in 1..65535");
    CHECK(c->pages >= 1 && c->pages <= (1 << 24), PI_ERR_SHAPE, "cache: pages must be in 1..2^24");
    CHECK(page_size_ok(c->page_size), PI_ERR_SHAPE, "cache: page_size must be a power of two in 8..%d",
          (int)PI_MAX_PAGE_SIZE);
    CHECK(c->head_dim >= 8 && c->head_dim <= PI_MAX_HEAD_DIM && c->head_dim % 8 == 0, PI_ERR_SHAPE,
          "cache: head_dim must be a multiple of 8 in 8..%d", (int)PI_MAX_HEAD_DIM);
    CHECK(c->k && c->v, PI_ERR_ARG, "cache: k and v are required");
    CHECK(aligned(c->k, 16) && aligned(c->v, 16), PI_ERR_ALIGN, "cache: k and v must be 16-byte aligned");
    return PI_OK;
}

inline pi_status check_layer(const pi_kv_cache* c, int layer) {
    TRY(check_cache(c));
    CHECK(layer >= 0 && layer < c->layers, PI_ERR_SHAPE, "layer %d of a cache of %d", layer, c->layers);
    return PI_OK;
}

inline pi_status check_batch(const pi_seq_batch* b) {
    CHECK(b, PI_ERR_ARG, "NULL batch");
    CHECK(b->n_seqs >= 0 && b->n_seqs <= 65535, PI_ERR_SHAPE, "batch: n_seqs must be in 0..65535");
    CHECK(b->n_tokens >= 0 && b->n_tokens <= (1 << 23), PI_ERR_SHAPE, "batch: n_tokens must be in 0..2^23");
    CHECK(b->max_new >= 0 && b->max_len >= 0, PI_ERR_SHAPE, "batch: max_new and max_len must be >= 0");
    if (b->n_seqs == 0 || b->n_tokens == 0) return PI_OK;
    CHECK(b->table_stride >= 1, PI_ERR_SHAPE, "batch: table_stride must be >= 1");
    CHECK(b->q_start && b->kv_len && b->table, PI_ERR_ARG, "batch: q_start, kv_len and table are required");
    CHECK(aligned(b->q_start, 4) && aligned(b->kv_len, 4) && aligned(b->table, 4), PI_ERR_ALIGN,
          "batch: q_start, kv_len and table must be 4-byte aligned");
    return PI_OK;
}

inline pi_status check_rows(const pi_rows* r, const char* name, int dtype) {
    const int size = dtype_size(dtype);
    CHECK(r && r->data, PI_ERR_ARG, "%s is required", name);
    CHECK(aligned(r->data, 16), PI_ERR_ALIGN, "%s must be 16-byte aligned", name);
    CHECK(r->token_stride >= 0 && r->head_stride >= 0 && r->token_stride < ((int64_t)1 << 40) &&
              r->head_stride < ((int64_t)1 << 40),
          PI_ERR_SHAPE, "%s: strides must be in 0..2^40", name);
    CHECK(r->token_stride * size % 16 == 0 && r->head_stride * size % 16 == 0, PI_ERR_ALIGN,
          "%s: strides must be multiples of 16 bytes", name);
    return PI_OK;
}

// ---- device ---------------------------------------------------------------------

// tokens that a table row can hold, and 2^30 at most: sums of two lengths stay in 32 bits
__device__ __forceinline__ int64_t longest(int table_stride, int page_shift) {
    return min((int64_t)table_stride << page_shift, (int64_t)1 << 30);
}

// the length of sequence s, inside what its table can hold
__device__ __forceinline__ int clamped_len(const Batch& b, const int page_shift, int s) {
    const int64_t cap = longest(b.table_stride, page_shift);
    const int len = b.kv_len[s];
    return len < 0 ? 0 : len > cap ? (int)cap : len;
}

// rows t0 <= t < t1 of sequence s, inside the batch's rows whatever the first rows are; t1 - t0 is in 0..n_tokens (the
// difference of two first rows as they are need not fit 32 bits)
__device__ __forceinline__ void seq_rows(const Batch& b, int s, int& t0, int& t1) {
    t0 = min(max(b.q_start[s], 0), b.n_tokens);
    t1 = max(min(b.q_start[s + 1], b.n_tokens), t0);
}

// the sequence of row t: the number of sequences that end at or before t; found
// by the whole wave (all 64 lanes call it with the same t).  n_seqs if none.
__device__ __forceinline__ int seq_of_row(const Batch& b, int t) {
    const int lane = threadIdx.x % WAVE;
    int s = 0;
    for (int i = 0; i < b.n_seqs; i += WAVE) {
        const bool before = i + lane < b.n_seqs && b.q_start[i + lane + 1] <= t;
        s += __popcll(__ballot(before));
    }
    return s;
}

}  // namespace pi
