// pi_attn.hip -- attention of new tokens over the paged cache.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "pi.h"
#include "pi_attn.h"
#include "pi_launch.h"

using namespace pi;

namespace {

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// Which kernel a call runs, how the keys are split, and the workspace for it.
struct Plan {
    bool few;                  // at most 16 rows per sequence and key head
    int64_t tiles, most_rows;
    int rows, chunk, splits;
    size_t part, ml, n, bytes; // offsets in the workspace, its size
};

constexpr int64_t MAX_ITEMS = 1 << 23;   // workgroups of a launch: 2^31 threads

// Keys per split so that about `want` workgroups have work when every sequence is max_len long (`alone`: without
// splits); none smaller than `least` keys.
void split_keys(Plan& p, int64_t alone, int64_t want, int64_t least, int max_len) {
    const int64_t n = std::max<int64_t>(1, want / std::max<int64_t>(1, alone));
    const int64_t chunk = std::max<int64_t>(least, ((int64_t)max_len + n - 1) / n);
    p.chunk = (int)std::min<int64_t>((chunk + 127) / 128 * 128, 1 << 30);
    p.splits = std::max(1, (int)(((int64_t)max_len + p.chunk - 1) / p.chunk));
}

// rule NULL: a plan for the rule that needs most
Plan plan_attention(const pi_kv_cache* c, const pi_seq_batch* b, int q_heads, const pi_score_rule* rule) {
    Plan p{};
    // keys that the rows of one sequence span (a prefix longer than the window leaves the rest to the last split)
    const int span = rule && rule->window > 0 ? (int)std::min<int64_t>(b->max_len, (int64_t)rule->window + b->max_new) : b->max_len;
    const int group = q_heads / c->kv_heads;
    p.most_rows = (int64_t)std::min(b->max_new, b->n_tokens) * group;
    p.few = p.most_rows <= FEW_ROWS;
    if (p.few) {
        p.tiles = b->n_seqs;
        p.rows = (int)p.most_rows;
        // The chip holds 512 workgroups.  One or two sequences are about alike, so two rounds do (one of 131072 tokens
        // with 8 key heads: 89 us for 1024 workgroups, 97 for 2048, 105 for 3072); the lengths of many differ, and smaller
        // pieces even them out.  Keys of 300 to 8191, 8 key heads of 128 f16, us for 1024, 2048 and 3072 workgroups:
        //   4 sequences 19.3 19.4 19.3    5: 22.6 20.4 20.4    8: 26.8 29.0 28.9    16: 42.6 43.4 41.3
        //   17: 49.0 48.6 43.7            32: 74.8 71.8 67.3   48: 131.7 103.9 94.8
        // so both steps lie where the choice matters least.  What they cost if the lengths are alike after all (8000 keys
        // each): 8 sequences 50.8 58.2 58.1, 16: 89.2 99.3 101.9, 48: 245 263 269.  The lengths are on the device.
        const int64_t want = b->n_seqs <= 4 ? 1024 : b->n_seqs <= 16 ? 2048 : 3072, alone = p.tiles * c->kv_heads;
        // A workgroup takes 3 to 4 us before its first key, the join 4: one piece up to 128 KB of keys (500 keys of 128
        // f16: 10.5 us against 12.3 in two), and the more workgroups there are, the longer the pieces (1000 keys,
        // 512 workgroups: 43 us, in pieces of 256 53; 64 workgroups 14.6 and 12.5).
        const bool small = (int64_t)span * c->head_dim * dtype_size(c->dtype) <= 128 << 10;
        const int least = small ? std::max(span, 1) : alone <= 128 ? 256 : alone <= 256 ? 512 : 1024;
        split_keys(p, alone, want, least, span);
    } else {
        p.rows = MANY_ROWS;
        p.tiles = std::min((int64_t)b->n_tokens * group / MANY_ROWS + b->n_seqs,
                           b->n_seqs * ((p.most_rows + MANY_ROWS - 1) / MANY_ROWS));
        // One sequence: its tiles are about alike.  f16: 128 rows over 1000 keys take 17.5 us in pieces of 256 keys, 24
        // in pieces of 512; over 131072 keys 120 us for 512 workgroups, 142 for 1024.  A step of an f32 tile takes four
        // times as long, so smaller pieces pay: 64 rows over 500 keys 26 us in pieces of 128, 35 of 256, 50 unsplit;
        // over 16000 keys 80 us for 1024 workgroups, 85 for 512.
        // Several: the tiles of the longest would be left alone at the end, so they are split further, but not under
        // 2048 keys where there are enough without (8 sequences of 100 to 8000 tokens, 1024 to 1 of them new: 180 us for
        // 512 workgroups, 113 for 2048, 174 for 4096; all 8 of 8000: 531 us against 555).
        const bool f32 = c->dtype == PI_F32, several = !f32 && b->n_seqs > 1;
        const int64_t alone = p.tiles * c->kv_heads;
        split_keys(p, alone, f32 ? 1024 : several ? 2048 : 512, f32 ? 128 : several && alone >= 512 ? 2048 : 256, span);
    }
    // (a shorter span never takes more workspace)
    if (rule) p.splits = std::min(p.splits, plan_attention(c, b, q_heads, nullptr).splits);
    p.part = 0;
    const size_t slots = p.splits > 1 ? (size_t)p.tiles * c->kv_heads * p.splits * p.rows : 0;
    p.ml = align256(slots * c->head_dim * 4);
    p.n = p.ml + align256(slots * 8);
    p.bytes = p.n + align256(std::max<size_t>((size_t)p.tiles * 4, 4));
    return p;
}

template <int DT, int GROUPS>
pi_status launch_join_by(const AttnArgs& a, hipStream_t s) {
    const int pieces = a.rows * (a.c.head_dim / 4), per = 256 / GROUPS;
    return launch(PI_K_ATTN_JOIN, k_attn_join<DT, GROUPS>, dim3((pieces + per - 1) / per, a.c.kv_heads, a.tiles), dim3(256), 0,
                  s, a);
}

template <int DT>
pi_status launch_join(const AttnArgs& a, hipStream_t s) {
    if (a.splits == 1) return PI_OK;
    // one thread's loads of many splits would wait for each other
    return a.splits <= 4    ? launch_join_by<DT, 1>(a, s)
           : a.splits <= 24 ? launch_join_by<DT, 4>(a, s)
                            : launch_join_by<DT, 16>(a, s);
}

template <int DT, int DP, bool FULL>
pi_status launch_few(const AttnArgs& a, hipStream_t s) {
    auto kern = k_attn_few<DT, DP, FULL>;
    TRY(allow_lds(kern, few_lds<DP>()));
    TRY(launch(PI_K_ATTN, kern, dim3(a.c.kv_heads, a.splits, a.b.n_seqs), dim3(WAVE * FEW_WAVES), few_lds<DP>(), s, a));
    return launch_join<DT>(a, s);
}

template <int DT, int DP, bool FULL, bool RULES>
pi_status launch_many(const AttnArgs& a, hipStream_t s) {
    auto kern = k_attn_many<DT, DP, FULL, RULES>;
    TRY(allow_lds(kern, many_lds<DT, DP>()));
    const int grid = (a.tiles * a.c.kv_heads * a.splits + XCDS - 1) / XCDS * XCDS;
    TRY(launch(PI_K_ATTN, kern, dim3(grid), dim3(WAVE * MANY_WAVES), many_lds<DT, DP>(), s, a));
    return launch_join<DT>(a, s);
}

template <int DT, int DP, bool FULL>
pi_status attend(const AttnArgs& a, const Plan& p, hipStream_t s) {
    if (p.few) return launch_few<DT, DP, FULL>(a, s);
    if (a.cap > 0.0f || a.slopes || a.scale == 0.0f) return launch_many<DT, DP, FULL, true>(a, s);
    return launch_many<DT, DP, FULL, false>(a, s);
}

template <int DT>
pi_status attend_dim(const AttnArgs& a, const Plan& p, hipStream_t s) {
    const int d = a.c.head_dim;
    if (d == 64) return attend<DT, 64, true>(a, p, s);
    if (d < 64) return attend<DT, 64, false>(a, p, s);
    if (d == 128) return attend<DT, 128, true>(a, p, s);
    if (d < 128) return attend<DT, 128, false>(a, p, s);
    if (d == 256) return attend<DT, 256, true>(a, p, s);
    return attend<DT, 256, false>(a, p, s);
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
    return plan_attention(cache, batch, q_heads, nullptr).bytes;
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
    const Plan p = plan_attention(cache, batch, q_heads, rule);
    CHECK(ws, PI_ERR_WORKSPACE, "workspace is NULL");
    CHECK(aligned(ws, 256), PI_ERR_ALIGN, "workspace must be 256-byte aligned");
    CHECK(ws_bytes >= p.bytes, PI_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, p.bytes);
    if (batch->max_new == 0) return PI_OK;
    CHECK(p.tiles * cache->kv_heads * p.splits <= MAX_ITEMS, PI_ERR_SHAPE, "too many rows for one call");
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
    a.tiles = (int)p.tiles;
    a.rows = p.rows;
    a.most_rows = p.most_rows;
    a.chunk = p.chunk;
    a.splits = p.splits;
    a.part = (float*)((uint8_t*)ws + p.part);
    a.part_ml = (float2*)((uint8_t*)ws + p.ml);
    a.part_n = (int*)((uint8_t*)ws + p.n);
    hipStream_t s = (hipStream_t)stream;
    return cache->dtype == PI_F32 ? attend_dim<F32>(a, p, s) : attend_dim<F16>(a, p, s);
}

}  // extern "C"
