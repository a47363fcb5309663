// pi_attn.hip -- attention of new tokens over the paged cache.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "pi.h"
#include "pi_attn.h"
#include "pi_launch.h"

using namespace pi;

namespace {

constexpr int MAXD_PER_LANE = PI_MAX_HEAD_DIM / WAVE;

// One wave per row and query head: a lane scores one key of 64, then owns every
// 64th element of the output.
template <int DT>
__global__ __launch_bounds__(WAVE) void k_attn(AttnArgs a) {
    typedef typename ElemT<DT>::T T;
    __shared__ float q[PI_MAX_HEAD_DIM], ps[WAVE];
    __shared__ int64_t at[WAVE];
    const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x;
    const int s = seq_of_row(a.b, t);
    if (s >= a.b.n_seqs || a.b.q_start[s] > t) return;
    const int d = a.c.head_dim, kvh = h / a.group;
    const int len = clamped_len(a.b, a.c.page_shift, s);
    const int pos = len - (a.b.q_start[s + 1] - t);
    int lo = a.first ? max(a.first[t], 0) : 0, hi = pos + 1;
    if (a.window > 0 && pos - a.window + 1 > lo) lo = pos - a.window + 1;
    if (a.prefix) hi = max(hi, a.prefix[s]);
    hi = min(hi, len);
    const T* qr = (const T*)a.q + t * a.q_ts + h * a.q_hs;
    for (int e = lane; e < d; e += WAVE) q[e] = (float)qr[e] * a.scale;
    __syncthreads();
    const float slope = a.slopes ? a.slopes[h] : 0.0f;
    float m = -INFINITY, l = 0.0f, acc[MAXD_PER_LANE] = {};
    for (int j0 = lo; j0 < hi; j0 += WAVE) {
        const int j = j0 + lane;
        float x = -INFINITY;
        at[lane] = -1;
        if (j < hi) {
            const int page = a.b.table[(int64_t)s * a.b.table_stride + (j >> a.c.page_shift)];
            if (page >= 0 && page < a.c.pages) {
                const int64_t row = ((int64_t)page * a.c.kv_heads + kvh) * a.c.page_size + (j & (a.c.page_size - 1));
                at[lane] = row;
                const T* k = (const T*)a.c.k + row * d;
                x = 0.0f;
                for (int e = 0; e < d; ++e) x = fmaf(q[e], (float)k[e], x);
                if (a.cap > 0.0f) x = a.cap * tanhf(x / a.cap);
                x -= slope * (float)abs(pos - j);
            }
        }
        float mx = x;
        for (int o = WAVE / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o, WAVE));
        mx = fmaxf(mx, m);
        const float ref = mx == -INFINITY ? 0.0f : mx;
        const float p = at[lane] >= 0 ? expf(x - ref) : 0.0f;
        const float alpha = expf(m - ref);
        m = mx;
        l = l * alpha + wave_sum(p);
        ps[lane] = p;
        __syncthreads();
        for (int e = 0; e < MAXD_PER_LANE; ++e) acc[e] *= alpha;
        for (int i = 0; i < min(WAVE, hi - j0); ++i) {
            if (at[i] < 0) continue;
            const T* v = (const T*)a.c.v + at[i] * d;
            for (int e = 0; e < MAXD_PER_LANE; ++e)
                if (lane + e * WAVE < d) acc[e] = fmaf(ps[i], (float)v[lane + e * WAVE], acc[e]);
        }
        __syncthreads();
    }
    T* o = (T*)a.out + t * a.o_ts + h * a.o_hs;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    for (int e = 0; e < MAXD_PER_LANE; ++e)
        if (lane + e * WAVE < d) o[lane + e * WAVE] = (T)(acc[e] * inv);
    if (a.lse && lane == 0) a.lse[(int64_t)t * a.q_heads + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// Which kernel a call runs, how the keys are split, and the workspace for it.
struct Plan {
    bool few;                  // at most 16 rows per sequence and key head
    int rows, chunk, splits;
    size_t part, ml, n, bytes; // offsets in the workspace, its size
};

Plan plan_attention(const pi_kv_cache* c, const pi_seq_batch* b, int q_heads) {
    Plan p{};
    const int64_t rows = (int64_t)std::min(b->max_new, b->n_tokens) * (q_heads / c->kv_heads);
    p.few = rows <= FEW_ROWS;
    p.rows = (int)std::min<int64_t>(rows, FEW_ROWS);
    p.splits = 1;
    p.chunk = 1 << 30;
    if (p.few) {
        const int64_t alone = std::max<int64_t>(1, (int64_t)b->n_seqs * c->kv_heads);
        const int64_t want = std::max<int64_t>(1, 2048 / alone);
        const int64_t chunk = std::max<int64_t>(256, ((int64_t)b->max_len + want - 1) / want);
        p.chunk = (int)std::min<int64_t>((chunk + 127) / 128 * 128, 1 << 30);
        p.splits = std::max(1, (int)(((int64_t)b->max_len + p.chunk - 1) / p.chunk));
    }
    p.part = 0;
    const size_t slots = p.splits > 1 ? (size_t)b->n_seqs * c->kv_heads * p.splits * p.rows : 0;
    p.ml = align256(slots * c->head_dim * 4);
    p.n = p.ml + align256(slots * 8);
    p.bytes = p.n + align256(std::max<size_t>((size_t)b->n_seqs * 4, 4));
    return p;
}

template <int DT, int DP, bool FULL>
pi_status launch_few(const AttnArgs& a, hipStream_t s) {
    auto kern = k_attn_few<DT, DP, FULL>;
    TRY(allow_lds(kern, few_lds<DP>()));
    TRY(launch(PI_K_ATTN, kern, dim3(a.splits, a.c.kv_heads, a.b.n_seqs), dim3(WAVE * FEW_WAVES), few_lds<DP>(), s, a));
    if (a.splits == 1) return PI_OK;
    const int pieces = a.rows * (a.c.head_dim / 4);
    return launch(PI_K_ATTN_JOIN, k_attn_join<DT>, dim3((pieces + WAVE - 1) / WAVE, a.c.kv_heads, a.b.n_seqs), dim3(WAVE),
                  0, s, a);
}

template <int DT>
pi_status attend(const AttnArgs& a, const Plan& p, int q_heads, hipStream_t s) {
    const int d = a.c.head_dim;
    if (p.few) {
        if (d == 64) return launch_few<DT, 64, true>(a, s);
        if (d < 64) return launch_few<DT, 64, false>(a, s);
        if (d == 128) return launch_few<DT, 128, true>(a, s);
        if (d < 128) return launch_few<DT, 128, false>(a, s);
        if (d == 256) return launch_few<DT, 256, true>(a, s);
        return launch_few<DT, 256, false>(a, s);
    }
    return launch(PI_K_ATTN, k_attn<DT>, dim3(a.b.n_tokens, q_heads), dim3(WAVE), 0, s, a);
}

pi_status check_q_heads(const pi_kv_cache* c, int q_heads) {
    CHECK(q_heads >= 1 && q_heads <= 65535 && q_heads % c->kv_heads == 0, PI_ERR_SHAPE,
          "q_heads (%d) must be a multiple of kv_heads (%d) and at most 65535", q_heads, c->kv_heads);
    return PI_OK;
}

}  // namespace

extern "C" {

size_t pi_attention_workspace_bytes(const pi_kv_cache* cache, const pi_seq_batch* batch, int32_t q_heads) {
    if (check_cache(cache) != PI_OK || check_batch(batch) != PI_OK || check_q_heads(cache, q_heads) != PI_OK) return 0;
    return plan_attention(cache, batch, q_heads).bytes;
}

pi_status pi_paged_attention(const pi_kv_cache* cache, int32_t layer, const pi_seq_batch* batch,
                             const pi_score_rule* rule, int32_t q_heads, const pi_rows* q, const pi_rows* out,
                             float* lse, void* ws, size_t ws_bytes, void* stream) {
    TRY(check_layer(cache, layer));
    TRY(check_batch(batch));
    TRY(check_q_heads(cache, q_heads));
    CHECK(rule, PI_ERR_ARG, "NULL rule");
    CHECK(std::isfinite(rule->scale) && std::isfinite(rule->cap) && rule->cap >= 0.0f && rule->window >= 0,
          PI_ERR_ARG, "rule: scale must be finite, cap and window >= 0");
    CHECK(aligned(rule->slopes, 4) && aligned(rule->prefix, 4) && aligned(rule->first, 4) && aligned(lse, 4),
          PI_ERR_ALIGN, "slopes, prefix, first and lse must be 4-byte aligned");
    if (batch->n_seqs == 0 || batch->n_tokens == 0) return PI_OK;
    TRY(check_rows(q, "q", cache->dtype));
    TRY(check_rows(out, "out", cache->dtype));
    const Plan p = plan_attention(cache, batch, q_heads);
    CHECK(ws, PI_ERR_WORKSPACE, "workspace is NULL");
    CHECK(aligned(ws, 256), PI_ERR_ALIGN, "workspace must be 256-byte aligned");
    CHECK(ws_bytes >= p.bytes, PI_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, p.bytes);
    if (batch->max_new == 0) return PI_OK;
    AttnArgs a{};
    a.c = cache_layer(cache, layer);
    a.b = seq_batch(batch);
    a.q = (const uint8_t*)q->data;
    a.out = (uint8_t*)out->data;
    a.lse = lse;
    a.q_ts = q->token_stride;
    a.q_hs = q->head_stride;
    a.o_ts = out->token_stride;
    a.o_hs = out->head_stride;
    a.q_heads = q_heads;
    a.group = q_heads / cache->kv_heads;
    a.scale = rule->scale;
    a.cap = rule->cap;
    a.window = rule->window;
    a.slopes = rule->slopes;
    a.prefix = rule->prefix;
    a.first = rule->first;
    a.rows = p.rows;
    a.chunk = p.chunk;
    a.splits = p.splits;
    a.part = (float*)((uint8_t*)ws + p.part);
    a.part_ml = (float2*)((uint8_t*)ws + p.ml);
    a.part_n = (int*)((uint8_t*)ws + p.n);
    hipStream_t s = (hipStream_t)stream;
    return cache->dtype == PI_F32 ? attend<F32>(a, p, q_heads, s) : attend<F16>(a, p, q_heads, s);
}

}  // extern "C"
