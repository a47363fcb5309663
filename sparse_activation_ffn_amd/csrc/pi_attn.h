// pi_attn.h -- kernels of the attention over the paged cache.
//
// For a row (token t, query head h) that sees the keys lo <= j < hi:
//   out = sum_j w_j V[j] / sum_j w_j,   w_j = exp(score_j - m),   lse = m + ln sum_j w_j
// formed in one pass over the keys: the weights are taken against a running
// reference m, and when a score passes it the sums so far are scaled by
// 2^(m_old - m_new).  Scores are kept in units of log2 e, so a weight is one exp2.
// m only has to be near the largest score, not equal to it: it moves when a score
// passes it by more than SLACK (8), which is rare after the first keys.  The f16
// weights for the matrix cores are carried 2^LIFT (64) times too large, so at
// most 2^14, and small ones stay clear of f16's subnormals (they lose bits below
// 2^-20 of the largest one).  f32 weights are at most 2^8: values of any size up to
// 2^120 divided by the number of keys are summed without overflow.
#pragma once
#include <algorithm>
#include <type_traits>

#include "pi_cache.h"

namespace pi {

// on a lambda: part of the kernel, whatever its size
#define INLINE __attribute__((always_inline))

typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

constexpr float LOG2E = 1.44269504088896340736f;
constexpr float LN2 = 0.69314718055994530942f;
constexpr float SLACK = 8.0f;
template <int DT> constexpr float LIFT = DT == F16 ? 6.0f : 0.0f;
constexpr int XCDS = 8;               // dies with an L2 each; workgroups go round them

struct AttnArgs {
    CacheLayer c;
    Batch b;
    const uint8_t* q;
    uint8_t* out;
    float* lse;
    int64_t q_ts, q_hs, o_ts, o_hs;   // strides in elements
    int q_heads, group;               // group: query heads per key head
    float scale, cap;
    int window;
    const float* slopes;
    const int* prefix;
    const int* first;
    // split of the keys
    int chunk, splits;                // keys per split, most splits of a sequence
    int tiles;                        // row tiles of the call (few rows: one per sequence)
    int rows;                         // rows of a tile
    int64_t most_rows;                // rows of a sequence and key head that are computed
    float* part;                      // [tiles][kv_heads][splits][rows][head_dim], when splits > 1
    float2* part_ml;                  // [tiles][kv_heads][splits][rows]: reference, sum
    int* part_n;                      // [tiles]: splits that hold something
};

// keys that row t at position pos of sequence s sees: 0 <= lo <= hi <= len (lo == hi: none), whatever the bounds given
__device__ __forceinline__ void visible(const AttnArgs& a, int t, int pos, int s, int len, int& lo, int& hi) {
    hi = pos + 1;
    if (a.prefix) hi = max(hi, a.prefix[s]);
    hi = max(min(hi, len), 0);
    lo = a.first ? max(a.first[t], 0) : 0;
    if (a.window > 0 && pos >= a.window) lo = max(lo, pos - a.window + 1);
    lo = min(lo, hi);
}

// weight of a sum taken against reference m, seen from reference top (-inf: nothing was summed)
__device__ __forceinline__ float weight_of(float m, float top) {
    return m == -INFINITY ? 0.0f : m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top);
}

// Adds a part (sum of weights pl, sums of values po) times its weight f.  A weight of 0 is multiplied too: a NaN score leaves
// the reference as it is (-inf where a part has no other), so only the sums tell of it.
__device__ __forceinline__ void add_part(float f, float pl, f4 po, float& l, f4& o) {
    l += f * pl;
    o += f * po;
}

template <int DT>
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? -INFINITY : (m - LIFT<DT> + __builtin_amdgcn_logf(l)) * LN2;
}

// Capped scores are cap tanh(x), x = scale q.k / cap.  f32 caches: tanhf.  f16 caches: for |x| <= 3/4 x times a quartic in
// x^2 (its coefficients are those of the least largest relative error, 6.1e-7, found by weighted least squares; 7.0e-7 with
// the roundings of f32), else
// 1 - 2 / (e^2x + 1), which is within 2^-22 and so within 1e-6 of the value there, but not for small x.
constexpr float TANH_SMALL = 0.75f;

constexpr float TANH_C[5] = {0.99999943f, -0.33328252f, 0.13258983f, -0.05005630f, 0.01292963f};
__device__ __forceinline__ float odd_poly(float x, float c1, float c3, float c5, float c7, float c9) {
    const float u = x * x;
    return x * fmaf(u, fmaf(u, fmaf(u, fmaf(u, c9, c7), c5), c3), c1);
}

template <int DT>
__device__ __forceinline__ float tanh_of(float x) {
    if (DT == F32) return tanhf(x);
    const float big = fmaf(-2.0f, __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(x * (2.0f * LOG2E)) + 1.0f), 1.0f);
    return fabsf(x) <= TANH_SMALL ? odd_poly(x, TANH_C[0], TANH_C[1], TANH_C[2], TANH_C[3], TANH_C[4]) : big;
}

// scale / cap, cap log2 e, scale log2 e and slope log2 e, kept finite so that a product q.k or a distance of 0 stays 0
__device__ __forceinline__ float kept_finite(float f) { return f != f ? f : fmaxf(-3e38f, fminf(f, 3e38f)); }
__device__ __forceinline__ float cap_rate(float scale, float cap) { return kept_finite(scale / cap); }
__device__ __forceinline__ float cap_unit(float cap) { return fminf(cap, 2e38f) * LOG2E; }

template <int DT> struct ElemT;
template <> struct ElemT<F32> { typedef float T; typedef f4 V4; };
template <> struct ElemT<F16> { typedef _Float16 T; typedef h4 V4; };

// elements e..e+3 of a row's output from its sums (reference m, sum of weights l)
template <int DT>
__device__ __forceinline__ void store_row(const AttnArgs& a, int t, int head, int e, f4 o, float m, float l) {
    typedef typename ElemT<DT>::T T;
    typedef typename ElemT<DT>::V4 V4;
    const bool none = l == 0.0f;                  // (o may hold infinities and NaN of keys with scores of -inf)
    const float inv = 1.0f / l;
    V4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = none ? (T)0.0f : (T)(o[i] * inv);
    *reinterpret_cast<V4*>((T*)a.out + t * a.o_ts + head * a.o_hs + e) = v;
    if (e == 0 && a.lse) a.lse[(int64_t)t * a.q_heads + head] = lse_of<DT>(m, l);
}

// ---- few rows: single tokens, and up to 16 rows per key head ------------------------
//
// Bound by reading the cache, so everything else serves the loads: a workgroup
// takes one sequence, one key head (all its query heads share each load) and a
// chunk of the keys; its four waves take every fourth step of 32 (f32: 16) keys.
// K and V go from memory to registers in 16-byte pieces, straight in the layouts
// of the matrix instructions, with the next step's loads issued as soon as a
// register is free; there is no barrier and no LDS traffic until the waves' sums
// are joined at the end.
//   S^T = K Q^T:   16 keys x 16 rows; lane (g = lane / 16, m = lane % 16) loads key m's
//                  elements of group g, and gets the scores of row m with keys 4g .. 4g+3
//   O^T = V^T P^T: the weights a lane has just formed are its B operand as they
//                  are, if its group's part of the sum over keys is these same keys; the A
//                  operand is then V of these keys, element m of each tile, and a tile is
//                  every 8th element of the head: f16 transposes 8 x 8 blocks in
//                  registers (32 permutes per step), f32 needs nothing.
// Measured (f16, 64 query and 8 key heads of 128): 48 sequences of 300 to 8191 tokens 91 us, 5.2 TB/s of K and V; two
// of 100001 and 131072 tokens 155 us, 6.1 TB/s (the plain read stream reaches 5.4); the counters show 1.02 times the
// bytes of K and V.  One sequence of 511, 16 heads of 64: 8.5 us, three memory latencies before the first key.

template <int DT, int DP> struct Few;

template <int DP> struct Few<F16, DP> {
    static constexpr int STEP = 32;                // keys per step
    static constexpr int EV = 8;                   // elements per 16 bytes
    static constexpr int VW = DP >= 128 ? 8 : 4;   // V elements per lane and load
};
template <int DP> struct Few<F32, DP> {
    static constexpr int STEP = 16;
    static constexpr int EV = 4;
    static constexpr int VW = 4;
};

constexpr int FEW_WAVES = 4;
constexpr int FEW_ROWS = 16;

// The LDS of the join: per wave 16 rows of DP sums, then reference and sum per row
template <int DP> constexpr size_t few_lds() { return FEW_WAVES * FEW_ROWS * (DP + 4 + 2) * sizeof(float); }

// split sp of `splits` covers [base + sp chunk, base + (sp + 1) chunk) of the keys, the last one all
// that is left; returns the number of splits that have keys (at least 1)
__device__ __forceinline__ int active_splits(const AttnArgs& a, int base, int end) {
    return min((max(end - base, 1) - 1) / a.chunk + 1, a.splits);
}

__device__ __forceinline__ unsigned nonfinite_h2(unsigned w) {
    // an f16 with all exponent bits set carries into its sign bit
    return ((w & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
}

// Split sp of rows r0 and on (16 at most are there) of sequence s and key head kvh, by the whole workgroup;
// `flat` is the tile's place in the workspace.
template <int DT, int DP, bool FULL>
__device__ __forceinline__ void few_rows(const AttnArgs& a, int s, int r0, int kvh, int sp, int flat, float* lds) {
    typedef Few<DT, DP> F;
    constexpr int STEP = F::STEP, U = STEP / 16, EV = F::EV, VW = F::VW;
    constexpr int NK = DP / (4 * EV);              // 16-byte pieces of a key per lane
    constexpr int NV = DP / (16 * VW);             // pieces of a value row per lane
    constexpr int ES = 16 / EV;                    // bytes per element

    const int lane = threadIdx.x % WAVE, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int m = lane % 16, g = lane / 16;
    const int d = FULL ? DP : a.c.head_dim;
    const int ps = a.c.page_size, shift = a.c.page_shift;

    int t0, t1;
    seq_rows(a.b, s, t0, t1);
    const int len = clamped_len(a.b, shift, s), q_end = a.b.q_start[s + 1];
    const int n_rows = (int)min(min((int64_t)(t1 - t0) * a.group, a.most_rows) - r0, (int64_t)FEW_ROWS);
    if (n_rows <= 0) return;

    // this lane's row, and the keys it sees; lanes without a row see whatever the others do
    const int tok = t0 + (r0 + m) / a.group, head = kvh * a.group + (r0 + m) % a.group;
    const bool row = m < n_rows;
    int lo = 0, hi = 0x7fffffff, pos = 0;
    if (row) {
        pos = len - (q_end - tok);
        visible(a, tok, pos, s, len, lo, hi);
    }
    int start = row && lo < hi ? lo : 0x7fffffff, end = row && lo < hi ? hi : 0;
    int lo_max = row ? lo : 0, hi_min = hi;
#pragma unroll
    for (int o = 1; o < 16; o *= 2) {
        start = min(start, __shfl_xor(start, o, WAVE));
        end = max(end, __shfl_xor(end, o, WAVE));
        lo_max = max(lo_max, __shfl_xor(lo_max, o, WAVE));
        hi_min = min(hi_min, __shfl_xor(hi_min, o, WAVE));
    }
    start = __builtin_amdgcn_readfirstlane(start) & ~(STEP - 1);
    end = __builtin_amdgcn_readfirstlane(end);
    lo_max = __builtin_amdgcn_readfirstlane(lo_max);
    hi_min = __builtin_amdgcn_readfirstlane(hi_min);
    if (end == 0) start = 0;
    const int n_split = active_splits(a, start, end);
    if (sp >= n_split) return;
    if (a.splits > 1 && sp == 0 && kvh == 0 && threadIdx.x == 0) a.part_n[flat] = n_split;
    const int from = start + sp * a.chunk;
    const int to = sp == n_split - 1 ? end : from + a.chunk;

    // queries: B operand, row m, the same elements of group g as the keys
    u4 q[NK];
#pragma unroll
    for (int c = 0; c < NK; ++c) {
        const int e = (c * 4 + g) * EV;
        q[c] = u4{0, 0, 0, 0};
        if (row && (FULL || e < d)) q[c] = ld16(a.q + (tok * a.q_ts + head * a.q_hs + e) * ES);
    }
    const float slope = a.slopes && row ? kept_finite(a.slopes[head] * LOG2E) : 0.0f;
    const float scale = a.cap > 0.0f ? cap_rate(a.scale, a.cap) : kept_finite(a.scale * LOG2E);

    const int* table = a.b.table + (int64_t)s * a.b.table_stride;
    const int last_page = (len - 1) >> shift;
    const int64_t page_bytes = (int64_t)a.c.kv_heads * ps * d * ES;
    const int head_off = kvh * ps;                 // rows before this head in a page

    // the pages of a step: 8 keys lie in one page at least, so one number per 8 keys
    struct Pages { int p[2 * U]; };
    auto fetch = [&](int j) {
        Pages r;
#pragma unroll
        for (int i = 0; i < 2 * U; ++i) r.p[i] = table[min((j + 8 * i) >> shift, last_page)];
        return r;
    };
    // byte offset of key j of step u (`second`: in the step's second 8 keys, whose page may be another); a page that is
    // none reads page 0, masked
    auto row_at = [&](const Pages& r, int u, bool second, int j) {
        const int p0 = r.p[2 * u], p1 = r.p[2 * u + 1];
        int p = second ? p1 : p0;
        p = (unsigned)p < (unsigned)a.c.pages ? p : 0;
        return p * page_bytes + (int64_t)(head_off + (j & (ps - 1))) * d * ES;
    };
    u4 kr[U][NK];
    auto load_k = [&](int j, const Pages& r) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint8_t* p = a.c.k + row_at(r, u, m >= 8, j + 16 * u + m) + g * 16;
#pragma unroll
            for (int c = 0; c < NK; ++c) {
                kr[u][c] = u4{0, 0, 0, 0};
                if (FULL || (c * 4 + g) * EV < d) kr[u][c] = ld16_stream(p + c * 64);
            }
        }
    };
    typedef typename std::conditional<VW * ES == 16, u4, u2>::type vraw;
    vraw vr[U][4][NV];
    auto load_v = [&](int j, const Pages& r) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint8_t* p = a.c.v + row_at(r, u, g >= 2, j + 16 * u + 4 * g) + m * VW * ES;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    vr[u][i][n] = vraw{};
                    if (FULL || (n * 16 + m) * VW < d)
                        vr[u][i][n] = __builtin_nontemporal_load((const vraw*)(p + (int64_t)i * d * ES + n * 16 * VW * ES));
                }
        }
    };

    f4 acc[NV][VW];
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int c = 0; c < VW; ++c) acc[n][c] = f4{0, 0, 0, 0};
    float ref = -INFINITY, sum = 0.0f;

    const int hop = FEW_WAVES * STEP;
    int j = from + wave * STEP;
    Pages pg{}, pg_next{};
    if (j < to) {
        pg = fetch(j);
        load_k(j, pg);
        load_v(j, pg);
        pg_next = fetch(j + hop);
    }
    for (; j < to; j += hop) {
        // scores
        f4 sc[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            sc[u] = f4{0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < NK; ++c) {
                if constexpr (DT == F16) {
                    sc[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, kr[u][c]),
                                                                   __builtin_bit_cast(h8, q[c]), sc[u], 0, 0, 0);
                } else {
                    const f4 kk = __builtin_bit_cast(f4, kr[u][c]), qq = __builtin_bit_cast(f4, q[c]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[u] = __builtin_amdgcn_mfma_f32_16x16x4f32(kk[e], qq[e], sc[u], 0, 0, 0);
                }
            }
        }
        const bool more = j + hop < to;
        if (more) load_k(j + hop, pg_next);

        bool ok[2 * U], whole = j >= lo_max && j + STEP <= hi_min && j + STEP <= to;
#pragma unroll
        for (int i = 0; i < 2 * U; ++i) {
            ok[i] = (unsigned)pg.p[i] < (unsigned)a.c.pages;
            whole = whole && ok[i];
        }
        float x[U][4], top = -INFINITY;
        bool sees[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = j + 16 * u + 4 * g + i;
                float v = sc[u][i] * scale;
                if (a.cap > 0.0f) v = cap_unit(a.cap) * tanh_of<DT>(v);
                if (a.slopes) v -= slope * (float)abs(pos - key);
                sees[u][i] = true;
                if (!whole) {
                    sees[u][i] = key >= lo && key < hi && key < to && (g >= 2 ? ok[2 * u + 1] : ok[2 * u]);
                    if (!sees[u][i]) v = -INFINITY;
                }
                x[u][i] = v;
                top = fmaxf(top, v);
            }
        if (__any(top > ref + SLACK)) {
            top = fmaxf(top, __shfl_xor(top, 16, WAVE));
            top = fmaxf(top, __shfl_xor(top, 32, WAVE));
            const float now = fmaxf(ref, top), f = weight_of(ref, now);
            ref = now;
            sum *= f;
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
                for (int c = 0; c < VW; ++c) acc[n][c] *= f;
        }
        const float off = LIFT<DT> - (ref == -INFINITY ? 0.0f : ref);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[u][i] = __builtin_amdgcn_exp2f(x[u][i] + off);
                sum += x[u][i];
            }

        if constexpr (DT == F16) {
            h8 p;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) p[4 * u + i] = (_Float16)x[u][i];
            constexpr int W = VW / 2;                  // dwords per value piece
            // Where some row does not see every key of the step, an infinity or NaN in V would reach it through
            // 0 * V: such elements are taken out, and added to the rows that do see them.
            unsigned odd = 0;
            if (!whole) {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int n = 0; n < NV; ++n)
#pragma unroll
                            for (int w = 0; w < W; ++w) odd |= nonfinite_h2(vr[u][i][n][w]);
            }
            const bool special = __any(odd != 0);
            h8 seen;
#pragma unroll
            for (int e = 0; e < 8; ++e) seen[e] = sees[e / 4][e % 4] ? (_Float16)1.0f : (_Float16)0.0f;
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    unsigned e0[4], e1[4];             // elements 2w and 2w+1 of the 8 keys
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const unsigned lo2 = vr[k / 2][2 * (k % 2)][n][w], hi2 = vr[k / 2][2 * (k % 2) + 1][n][w];
                        e0[k] = __builtin_amdgcn_perm(hi2, lo2, 0x05040100u);
                        e1[k] = __builtin_amdgcn_perm(hi2, lo2, 0x07060302u);
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        u4 bits = half ? u4{e1[0], e1[1], e1[2], e1[3]} : u4{e0[0], e0[1], e0[2], e0[3]};
                        f4& o = acc[n][2 * w + half];
                        if (special) {
                            h8 v = __builtin_bit_cast(h8, bits), pinf, ninf, nan;
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float f = (float)v[e];
                                pinf[e] = f == INFINITY ? (_Float16)1.0f : (_Float16)0.0f;
                                ninf[e] = f == -INFINITY ? (_Float16)1.0f : (_Float16)0.0f;
                                nan[e] = f != f ? (_Float16)1.0f : (_Float16)0.0f;
                                v[e] = f - f == 0.0f ? v[e] : (_Float16)0.0f;
                            }
                            bits = __builtin_bit_cast(u4, v);
                            const f4 z = f4{0, 0, 0, 0};
                            const f4 np = __builtin_amdgcn_mfma_f32_16x16x32_f16(pinf, seen, z, 0, 0, 0);
                            const f4 nn = __builtin_amdgcn_mfma_f32_16x16x32_f16(ninf, seen, z, 0, 0, 0);
                            const f4 nq = __builtin_amdgcn_mfma_f32_16x16x32_f16(nan, seen, z, 0, 0, 0);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (np[i] > 0.0f) o[i] += INFINITY;
                                if (nn[i] > 0.0f) o[i] -= INFINITY;
                                if (nq[i] > 0.0f) o[i] = NAN;
                            }
                        }
                        o = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, bits), p, o, 0, 0, 0);
                    }
                }
        } else {
            unsigned odd = 0;
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int n = 0; n < NV; ++n)
#pragma unroll
                        for (int w = 0; w < 4; ++w) odd |= (vr[0][i][n][w] & 0x7f800000u) == 0x7f800000u;
            }
            const bool special = __any(odd != 0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    f4 v = __builtin_bit_cast(f4, vr[0][i][n]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (special) {
                            const float seen = sees[0][i] ? 1.0f : 0.0f;
                            const f4 z = f4{0, 0, 0, 0};
                            const f4 np = __builtin_amdgcn_mfma_f32_16x16x4f32(v[c] == INFINITY ? 1.0f : 0.0f, seen, z, 0, 0, 0);
                            const f4 nn = __builtin_amdgcn_mfma_f32_16x16x4f32(v[c] == -INFINITY ? 1.0f : 0.0f, seen, z, 0, 0, 0);
                            const f4 nq = __builtin_amdgcn_mfma_f32_16x16x4f32(v[c] != v[c] ? 1.0f : 0.0f, seen, z, 0, 0, 0);
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                if (np[r] > 0.0f) acc[n][c][r] += INFINITY;
                                if (nn[r] > 0.0f) acc[n][c][r] -= INFINITY;
                                if (nq[r] > 0.0f) acc[n][c][r] = NAN;
                            }
                            v[c] = v[c] - v[c] == 0.0f ? v[c] : 0.0f;
                        }
                        acc[n][c] = __builtin_amdgcn_mfma_f32_16x16x4f32(v[c], x[0][i], acc[n][c], 0, 0, 0);
                    }
                }
        }
        if (more) {
            load_v(j + hop, pg_next);
            pg = pg_next;
            pg_next = fetch(j + 2 * hop);
        }
    }

    // join of the waves: lane (m, g) holds row m, elements VW (16 n + 4 g + i) + c
    sum += __shfl_xor(sum, 16, WAVE);
    sum += __shfl_xor(sum, 32, WAVE);
    constexpr int LD = DP + 4;
    float* o_lds = lds;
    float* ml = lds + FEW_WAVES * FEW_ROWS * LD;
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < VW; c += 4) {
                const f4 v = f4{acc[n][c][i], acc[n][c + 1][i], acc[n][c + 2][i], acc[n][c + 3][i]};
                *reinterpret_cast<f4*>(o_lds + (wave * FEW_ROWS + m) * LD + VW * (16 * n + 4 * g + i) + c) = v;
            }
    if (g == 0) {
        ml[(wave * FEW_ROWS + m) * 2] = ref;
        ml[(wave * FEW_ROWS + m) * 2 + 1] = sum;
    }
    __syncthreads();
    const int pieces = d / 4;
    for (int i = threadIdx.x; i < n_rows * pieces; i += WAVE * FEW_WAVES) {
        const int r = i / pieces, e = (i - r * pieces) * 4;
        float mw[FEW_WAVES], all = -INFINITY, l = 0.0f;
#pragma unroll
        for (int w = 0; w < FEW_WAVES; ++w) {
            mw[w] = ml[(w * FEW_ROWS + r) * 2];
            all = fmaxf(all, mw[w]);
        }
        f4 o = f4{0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < FEW_WAVES; ++w) {
            const float f = weight_of(mw[w], all);
            add_part(f, ml[(w * FEW_ROWS + r) * 2 + 1], *reinterpret_cast<const f4*>(o_lds + (w * FEW_ROWS + r) * LD + e), l, o);
        }
        if (n_split > 1) {
            const int64_t at = (((int64_t)flat * a.c.kv_heads + kvh) * a.splits + sp) * a.rows + r;
            *reinterpret_cast<f4*>(a.part + at * d + e) = o;
            if (e == 0) a.part_ml[at] = make_float2(all, l);
        } else {
            store_row<DT>(a, t0 + (r0 + r) / a.group, kvh * a.group + (r0 + r) % a.group, e, o, all, l);
        }
    }
}

template <int DT, int DP, bool FULL>
__global__ __launch_bounds__(WAVE * FEW_WAVES, DP == 64 ? 3 : DP == 128 ? 2 : 1) void k_attn_few(AttnArgs a) {
    extern __shared__ float lds[];
    // Workgroups go round the XCDs.  Heads vary fastest, and the order of the splits turns with the sequence:
    // short sequences have no late splits, and the XCD that got only those would be idle (48 sequences of
    // 300 to 8191 tokens, 8 splits: 179 us with splits fastest, 101 us with 5 splits).
    few_rows<DT, DP, FULL>(a, blockIdx.z, 0, blockIdx.x, (blockIdx.y + blockIdx.z) % a.splits, blockIdx.z, lds);
}

// ---- many rows: chunks of new tokens -----------------------------------------------
//
// Bound by the matrix cores, so the loads serve them: a workgroup takes MANY_ROWS
// rows (row r of a sequence and key head: token r / group, so all query heads of
// a key head share its keys) and walks over the keys in tiles of TILE.  The tile
// after the current one is on its way from memory to LDS meanwhile (two buffers,
// loads that write LDS directly).  Each wave owns 32 rows:
//   S^T = K Q^T (32 keys x 32 rows per instruction): the queries stay in
//   registers; lane (m = lane % 32, h = lane / 32) gets the scores of row m with the
//   keys 8b + 4h + i of a block of 32, i < 4;
//   O^T = V^T P^T: these weights are the B operand as they lie, if the sum over
//   the keys is taken in that order; the A operand is V read from LDS
//   transposed (f16) or as it lies (f32: elements c, c + DP / 32, ... make a tile).
// Two workgroups per CU hide each other's waits (a form with two groups of waves half a tile apart, 256 rows, was as
// fast within 4% and slower under 8192 keys; three buffers, loads two tiles ahead and 8 waves gained nothing).
// Measured (f16): 2048 tokens over 10001 keys, 56 heads of 128: 600 to 630 us, 840 to 875 TFLOP/s, where the library's
// 8192^3 product makes 1097; both run at the power limit (1.6 to 1.9 and 1.45 GHz of 2.4), so what counts is work,
// not waiting.  The counters show 1.05 times the bytes of Q, K and V: the row tiles of a head share them in L2.
// LDS rows are DP elements without padding; the 16-byte pieces of row r are
// permuted by an exclusive or with a function of r, chosen so that the rows that
// one instruction reads lie in different banks.

typedef float f16v __attribute__((ext_vector_type(16)));
typedef short s4v __attribute__((ext_vector_type(4)));

constexpr int MANY_WAVES = 4;
constexpr int MANY_ROWS = 32 * MANY_WAVES;

template <int DT, int DP> struct Many {
    static constexpr int TILE = DT == F16 && DP <= 128 ? 64 : 32;   // keys per tile
    static constexpr int ES = DT == F16 ? 2 : 4;
    static constexpr int ROW = DP * ES;                             // bytes of an LDS row
    static constexpr int BYTES = TILE * ROW;
};

// K and V, two buffers each (f32 tiles of few rows: their join)
template <int DT, int DP> constexpr size_t many_lds() {
    return std::max(4 * (size_t)Many<DT, DP>::BYTES, DT == F32 ? few_lds<DP>() : 0);
}

// piece c of row r of a K tile: 16 rows in a row at the same c read 16 different pieces of 256 bytes
template <int ROW>
__device__ __forceinline__ int k_piece(int r, int c) {
    return c ^ (ROW >= 256 ? r & 15 : (r >> 1) & 7);
}
// of a V tile, f16: 4 rows at 4 pieces each (a transposed read) are 16 different pieces of 256 bytes;
// f32: a read takes whole rows, two of them 4 apart
template <int DT, int ROW>
__device__ __forceinline__ int v_piece(int r, int c) {
    if (DT == F32) return c;
    return c ^ (ROW >= 256 ? (r & 3) << 2 : ((r >> 1) & 1) << 2);
}

__device__ __forceinline__ void load_to_lds(const uint8_t* from, uint8_t* to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                     (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

// an address that is the same in all lanes, in scalar registers
__device__ __forceinline__ const uint8_t* scalar(const uint8_t* p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint64_t lo = (unsigned)__builtin_amdgcn_readfirstlane((int)v), hi = (unsigned)__builtin_amdgcn_readfirstlane((int)(v >> 32));
    return reinterpret_cast<const uint8_t*>(hi << 32 | lo);
}

// all loads of this wave have arrived (vmcnt 0, the other counters as they are)
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0f70); }

// The sequence and first row of row tile `flat` when sequences have tiles of `tile`
// rows, at most `most` rows each; false past the last one.  The whole wave calls it.
__device__ __forceinline__ bool tile_at(const AttnArgs& a, int flat, int tile, int64_t most, int& s, int& r0) {
    const int lane = threadIdx.x % WAVE;
    int before = 0;
    for (int base = 0; base < a.b.n_seqs; base += WAVE) {
        int n = 0;
        if (base + lane < a.b.n_seqs) {
            int t0, t1;
            seq_rows(a.b, base + lane, t0, t1);
            n = (int)((min((int64_t)(t1 - t0) * a.group, most) + tile - 1) / tile);
        }
        const int incl = wave_incl_scan(n);
        const uint64_t past = __ballot(before + incl > flat);
        if (past) {
            const int at = __builtin_ctzll(past);
            s = base + at;
            r0 = (flat - before - (__shfl(incl, at, WAVE) - __shfl(n, at, WAVE))) * tile;
            return true;
        }
        before += __shfl(incl, WAVE - 1, WAVE);
    }
    return false;
}

__device__ __forceinline__ bool finite(float f) { return f - f == 0.0f; }

template <int DT>
__device__ __forceinline__ bool nonfinite(u4 w) {
    if (DT == F16) return (nonfinite_h2(w.x) | nonfinite_h2(w.y) | nonfinite_h2(w.z) | nonfinite_h2(w.w)) != 0;
    return !(finite(bits_f(w.x)) && finite(bits_f(w.y)) && finite(bits_f(w.z)) && finite(bits_f(w.w)));
}

// infinities and NaN replaced by 0
template <int DT>
__device__ __forceinline__ u4 only_finite(u4 w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (DT == F16) {
            const unsigned odd = nonfinite_h2(w[i]);
            w[i] &= ~((odd >> 15) * 0xffffu);      // both carries: 0x80000000 and 0x8000
        } else {
            w[i] = finite(bits_f(w[i])) ? w[i] : 0u;
        }
    }
    return w;
}

// The infinities and NaN in V of keys k0 <= k < k1 of a tile with a page (ok), added to the rows that see them:
// each lane's row sees lo <= k < hi.
template <int DT, int DP>
__device__ __forceinline__ void add_nonfinite(f16v* acc, const uint8_t* vt, int lane, int k0, int k1, int lo, int hi,
                                              uint64_t ok) {
    constexpr int ROW = Many<DT, DP>::ROW, ND = DP / 32;
    for (int k = k0; k < k1; ++k) {
        if (!((ok >> k) & 1)) continue;
        bool odd = false;
        for (int i = lane; i < ROW / 4; i += WAVE) {
            const unsigned w = *reinterpret_cast<const unsigned*>(vt + k * ROW + i * 4);
            odd |= DT == F16 ? nonfinite_h2(w) != 0 : !finite(bits_f(w));
        }
        if (!__any(odd)) continue;
        const bool sees = k >= lo && k < hi;
        const int h = lane / 32;
#pragma unroll
        for (int t = 0; t < ND; ++t)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {      // acc[t][i .. i + 3]: see the end of k_attn_many
                float f[4];
                if constexpr (DT == F16) {
                    const int piece = v_piece<DT, ROW>(k, 4 * t + i / 4);
                    const u2 w = *reinterpret_cast<const u2*>(vt + k * ROW + piece * 16 + 8 * h);
                    f[0] = half_lo(w.x), f[1] = half_hi(w.x), f[2] = half_lo(w.y), f[3] = half_hi(w.y);
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        f[c] = reinterpret_cast<const float*>(vt + k * ROW)[ND * (2 * i + 4 * h + c) + t];
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[t][i + c] += sees && !finite(f[c]) ? f[c] : 0.0f;
            }
    }
}

// RULES: scores may be capped or biased (else they are scale * q.k alone)
template <int DT, int DP, bool FULL, bool RULES>
__global__ __launch_bounds__(WAVE * MANY_WAVES, DP == 64 ? 3 : DP == 128 ? 2 : 1) void k_attn_many(AttnArgs a) {
    typedef Many<DT, DP> M;
    constexpr int TILE = M::TILE, ES = M::ES, ROW = M::ROW, KB = TILE / 32;
    constexpr int EV = 16 / ES, NC = ROW / 16;     // elements per piece, pieces per row
    constexpr int NK = NC / 2;                     // pieces of a key per lane
    constexpr int ND = DP / 32;                    // tiles of 32 elements of the output
    constexpr int RPI = 1024 / ROW;                // rows per load instruction
    constexpr int LOADS = TILE / RPI / MANY_WAVES; // load instructions per wave, K and V each
    extern __shared__ __align__(1024) uint8_t smem[];

    // Work item: splits fastest, then row tiles, last (longest) first, then heads.  Workgroups go round the XCDs; with eight key heads or
    // more each XCD takes a run of items, so that those that share keys share an L2 (with fewer heads a run would
    // hold long or short tiles only).
    const int total = a.tiles * a.c.kv_heads * a.splits, per = gridDim.x / XCDS;
    const int item = a.c.kv_heads >= XCDS ? (blockIdx.x % XCDS) * per + blockIdx.x / XCDS : blockIdx.x;
    if (item >= total) return;
    const int sp = item % a.splits, rest = item / a.splits;
    const int flat = a.tiles - 1 - rest % a.tiles, kvh = rest / a.tiles;
    int s, r0;
    if (!tile_at(a, flat, MANY_ROWS, a.most_rows, s, r0)) return;
    s = __builtin_amdgcn_readfirstlane(s);
    r0 = __builtin_amdgcn_readfirstlane(r0);

    const int lane = threadIdx.x % WAVE, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int m = lane % 32, h = lane / 32;
    const int d = FULL ? DP : a.c.head_dim;
    const int ps = a.c.page_size, shift = a.c.page_shift;
    int t0, t1;
    seq_rows(a.b, s, t0, t1);
    const int len = clamped_len(a.b, shift, s), q_end = a.b.q_start[s + 1];
    const int n_rows = (int)min(min((int64_t)(t1 - t0) * a.group, a.most_rows) - r0, (int64_t)MANY_ROWS);

    // In an f32 tile of so few rows three waves would have none and one all the matrix products: the waves share the
    // keys instead (512 tokens over 3000 and 48 single ones over 300 to 6000, 16 heads of 64: 593 us without, 340 with;
    // 1 to 160 tokens over 200 to 1500: 33 and 28).  f16 tiles wait for memory either way (157 and 171).
    if constexpr (DT == F32) {
        if (n_rows <= FEW_ROWS) {
            few_rows<DT, DP, FULL>(a, s, r0, kvh, sp, flat, reinterpret_cast<float*>(smem));
            return;
        }
    }

    const int my = wave * 32 + m;
    const bool row = my < n_rows;
    const int tok = t0 + (r0 + my) / a.group, head = kvh * a.group + (r0 + my) % a.group;
    int lo = 0, hi = 0, pos = 0;
    if (row) {
        pos = len - (q_end - tok);
        visible(a, tok, pos, s, len, lo, hi);
    }
    // keys that some row of the wave sees, keys that all of them see; then the workgroup's
    int w_lo = lo < hi ? lo : 0x7fffffff, w_hi = lo < hi ? hi : 0, in_lo = row ? lo : 0, in_hi = row ? hi : 0x7fffffff;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        w_lo = min(w_lo, __shfl_xor(w_lo, o, WAVE));
        w_hi = max(w_hi, __shfl_xor(w_hi, o, WAVE));
        in_lo = max(in_lo, __shfl_xor(in_lo, o, WAVE));
        in_hi = min(in_hi, __shfl_xor(in_hi, o, WAVE));
    }
    w_lo = __builtin_amdgcn_readfirstlane(w_lo);
    w_hi = __builtin_amdgcn_readfirstlane(w_hi);
    in_lo = __builtin_amdgcn_readfirstlane(in_lo);
    in_hi = __builtin_amdgcn_readfirstlane(in_hi);
    int* scratch = reinterpret_cast<int*>(smem);
    if (lane == 0) {
        scratch[wave] = w_lo;
        scratch[MANY_WAVES + wave] = w_hi;
        scratch[2 * MANY_WAVES + wave] = in_lo;
        scratch[3 * MANY_WAVES + wave] = in_hi;
    }
    __syncthreads();
    int start = 0x7fffffff, end = 0, all_lo = 0, all_hi = 0x7fffffff;
#pragma unroll
    for (int w = 0; w < MANY_WAVES; ++w) {
        start = min(start, scratch[w]);
        end = max(end, scratch[MANY_WAVES + w]);
        all_lo = max(all_lo, scratch[2 * MANY_WAVES + w]);
        all_hi = min(all_hi, scratch[3 * MANY_WAVES + w]);
    }
    all_lo = __builtin_amdgcn_readfirstlane(all_lo);
    all_hi = __builtin_amdgcn_readfirstlane(all_hi);
    __syncthreads();
    start = __builtin_amdgcn_readfirstlane(end > 0 ? start & ~(TILE - 1) : 0);
    end = __builtin_amdgcn_readfirstlane(end);
    const int n_split = active_splits(a, start, end);
    if (sp >= n_split) return;
    if (a.splits > 1 && sp == 0 && kvh == 0 && threadIdx.x == 0) a.part_n[flat] = n_split;
    const int from = start + sp * a.chunk;
    const int to = sp == n_split - 1 ? end : from + a.chunk;

    // queries: B operand, row m, pieces 2c + h.  A negative scale goes into their sign.
    u4 q[NK];
    const unsigned flip = a.scale < 0.0f ? (DT == F16 ? 0x80008000u : 0x80000000u) : 0u;
#pragma unroll
    for (int c = 0; c < NK; ++c) {
        const int e = (2 * c + h) * EV;
        q[c] = u4{0, 0, 0, 0};
        if (row && (FULL || e < d)) q[c] = ld16(a.q + (tok * a.q_ts + head * a.q_hs + e) * ES);
        q[c] ^= flip;
    }
    const float abs_scale = fabsf(a.scale);
    const float scale = RULES && a.cap > 0.0f ? cap_rate(abs_scale, a.cap) : kept_finite(abs_scale * LOG2E);
    const float slope = RULES && a.slopes && row ? kept_finite(a.slopes[head] * LOG2E) : 0.0f;

    const int* table = a.b.table + (int64_t)s * a.b.table_stride;
    const int last_page = max(len - 1, 0) >> shift;
    const int64_t page_bytes = (int64_t)a.c.kv_heads * ps * d * ES;
    const int head_off = kvh * ps;

    // pieces past the head's last element are zero, and no load writes them
    if (!FULL) {
        for (int i = threadIdx.x; i < 4 * M::BYTES / 16; i += WAVE * MANY_WAVES)
            reinterpret_cast<u4*>(smem)[i] = u4{0, 0, 0, 0};
        __syncthreads();
    }
    auto page_of = [&](int j) INLINE { return table[min((j + lane) >> shift, last_page)]; };
    // what a lane loads of a row: the piece that belongs where its 16 bytes go in LDS
    unsigned k_off[LOADS], v_off[LOADS];
    bool k_ok[LOADS], v_ok[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int r = lane / NC, row_in_tile = (wave * LOADS + i) * RPI + r;
        const int kc = k_piece<ROW>(row_in_tile, lane % NC), vc = v_piece<DT, ROW>(row_in_tile, lane % NC);
        k_off[i] = r * d * ES + kc * 16;
        v_off[i] = r * d * ES + vc * 16;
        k_ok[i] = kc * EV < d;
        v_ok[i] = vc * EV < d;
    }
    // Keys j .. j + TILE - 1 of K or V into a buffer; `page` holds the page of key j + lane.  The rows of one
    // instruction lie in one page, one after the other: a scalar address and fixed lane offsets.
    static_assert(RPI <= 8, "a page holds 8 rows or more");
    auto load_tile = [&](const uint8_t* base, int j, int page, const unsigned (&off)[LOADS], const bool (&has)[LOADS],
                         uint8_t* __restrict__ to_lds) INLINE {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int first = (wave * LOADS + i) * RPI;
            const int id = __builtin_amdgcn_readlane(page, first);
            const int p = (unsigned)id < (unsigned)a.c.pages ? id : 0;
            const uint8_t* at = scalar(base + (p * page_bytes + (int64_t)(head_off + ((j + first) & (ps - 1))) * d * ES));
            unsigned lane_off = off[i];
            asm volatile("" : "+v"(lane_off));     // (else it is kept as 64 bits, and the address is formed in vector registers)
            if (FULL || has[i]) load_to_lds(at + lane_off, to_lds + first * ROW);
        }
    };

    f16v acc[ND];
#pragma unroll
    for (int t = 0; t < ND; ++t) acc[t] = f16v{};
    float ref = -INFINITY, sum = 0.0f;

    // byte offsets of this lane's reads in a buffer, before c and t are put in
    const int k_base = m * ROW + k_piece<ROW>(m, h) * 16;
    const int v_row = 4 * h + lane % 16 / 4, v_elem = 16 * (lane / 16 % 2) + 4 * (lane % 4);
    const int v_base = v_row * ROW + v_piece<DT, ROW>(v_row, v_elem / 8) * 16 + v_elem % 8 * 2;

    // scores are kept in units of `unit` / log2 e: times scale, or as the tanh of a cap alone
    const float unit = !RULES ? scale : a.cap > 0.0f && !a.slopes ? cap_unit(a.cap) : 1.0f;
    int page = 0, page_next = 0;

    const bool in_range = DT == F16 && scale >= 1e-4f && scale <= 1e3f;
    const float s2 = scale * scale, c1 = TANH_C[0] * scale, c3 = TANH_C[1] * scale * s2;
    const float c5 = TANH_C[2] * scale * s2 * s2, c7 = TANH_C[3] * scale * s2 * s2 * s2;
    const float c9 = TANH_C[4] * scale * s2 * s2 * s2 * s2;
    // cap and bias of the scores of tile j; score r of block k belongs to key j + 32 k + 8 (r / 4) + 4 h + r % 4
    auto by_rule = [&](f16v (&sc)[KB], int j) INLINE {
        if (!RULES) return;
        if (a.cap > 0.0f) {
            // A cap is there for the few scores that come near it: a wave whose tile has none past 3/4 of it forms six
            // operations per score, the factor scale / cap in the coefficients (while these stay in range), and no
            // transcendental one, which takes four times as long.  Mixed prompts, 112 row tiles of 8 key heads: 25.6 us,
            // with the exponential form alone 27.4; 35 where every tile has scores past it (both forms for each score).
            float most = 0.0f;
            if (in_range) {
#pragma unroll
                for (int k = 0; k < KB; ++k)
#pragma unroll
                    for (int r = 0; r < 16; ++r) most = fmaxf(most, fabsf(sc[k][r]));
            }
            if (in_range && !__any(most * scale > TANH_SMALL)) {
#pragma unroll
                for (int k = 0; k < KB; ++k)
#pragma unroll
                    for (int r = 0; r < 16; ++r) sc[k][r] = odd_poly(sc[k][r], c1, c3, c5, c7, c9);
            } else {
#pragma unroll
                for (int k = 0; k < KB; ++k)
#pragma unroll
                    for (int r = 0; r < 16; ++r) sc[k][r] = tanh_of<DT>(sc[k][r] * scale);
            }
        } else {
#pragma unroll
            for (int k = 0; k < KB; ++k) sc[k] *= scale;
        }
        if (a.slopes) {
            const float away = (float)(pos - j - 4 * h), first = a.cap > 0.0f ? cap_unit(a.cap) : 1.0f;
#pragma unroll
            for (int k = 0; k < KB; ++k)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    sc[k][r] = fmaf(-slope, fabsf(away - (float)(32 * k + 8 * (r / 4) + r % 4)), sc[k][r] * first);
        }
    };
    // moves the reference when a score passes it by too much
    auto raise = [&](const f16v (&sc)[KB]) INLINE {
        float top = sc[0][0];
#pragma unroll
        for (int k = 0; k < KB; ++k)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, sc[k][r]);
        top *= unit;
        if (__any(top > ref + SLACK)) {
            top = fmaxf(top, __shfl_xor(top, 32, WAVE));
            // (nothing is summed while ref is -inf but infinities, which no factor may turn into NaN)
            const float now = fmaxf(ref, top), w = ref == -INFINITY ? 1.0f : weight_of(ref, now);
            // of sums of f16 values a factor of 0 leaves 10^-37, which is less than 10^-18; f32 ones may be any size and
            // become 0
            const float f = fmaxf(w, 1e-37f);
            ref = now;
            sum *= f;
            if (DT == F16 || !__any(w < f)) {
#pragma unroll
                for (int t = 0; t < ND; ++t) acc[t] *= f;
            } else {
#pragma unroll
                for (int t = 0; t < ND; ++t)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[t][i] = w > 0.0f ? w * acc[t][i] : finite(acc[t][i]) ? 0.0f : acc[t][i];
            }
        }
    };
    // one tile: its keys and values lie at cur, the next tile's go to next
    auto step = [&](int j, uint8_t* __restrict__ cur, uint8_t* __restrict__ next) INLINE {
        wait_loads();
        __syncthreads();                           // tile j is there, and every wave is done with the other buffer
        const uint64_t ok = __ballot((unsigned)page < (unsigned)a.c.pages);
        if (j + TILE < to) {
            load_tile(a.c.k, j + TILE, page_next, k_off, k_ok, next);
            load_tile(a.c.v, j + TILE, page_next, v_off, v_ok, next + M::BYTES);
            page = page_next;
            page_next = page_of(j + 2 * TILE);
        }
        constexpr uint64_t ALL = TILE == 64 ? ~0ull : (1ull << (TILE % 64)) - 1;
        const bool pages = (ok & ALL) == ALL, idle = j >= w_hi || j + TILE <= w_lo;
        if (!(j >= all_lo && j + TILE <= all_hi && j + TILE <= to && pages)) {
            // Where some row does not see every key, an infinity or NaN in V would reach it through 0 * V: such
            // elements go to the rows that see them one by one, and become 0 for the product.
            u4* vt = reinterpret_cast<u4*>(cur + M::BYTES);
            bool odd = false;
            for (int i = threadIdx.x; i < M::BYTES / 16; i += WAVE * MANY_WAVES) odd |= nonfinite<DT>(vt[i]);
            if (__syncthreads_or(odd)) {
                if (!idle)
                    add_nonfinite<DT, DP>(acc, cur + M::BYTES, lane, max(w_lo - j, 0), min(min(w_hi, to) - j, TILE), lo - j,
                                          hi - j, ok);
                __syncthreads();
                for (int i = threadIdx.x; i < M::BYTES / 16; i += WAVE * MANY_WAVES) vt[i] = only_finite<DT>(vt[i]);
                __syncthreads();
            }
        }
        if (idle) return;                          // no row of this wave sees these keys

        // (opaque here, so that the addresses made of them are not kept in registers)
        int kb0 = k_base, vb0 = v_base;
        asm volatile("" : "+v"(kb0), "+v"(vb0));
        u4 kk[NK][KB];
#pragma unroll
        for (int c = 0; c < NK; ++c)
#pragma unroll
            for (int k = 0; k < KB; ++k)           // piece 2c + h of row 32 k + m: the permutation leaves an
                kk[c][k] = *reinterpret_cast<const u4*>(cur + ((kb0 ^ (c * 32)) + k * 32 * ROW));      // exclusive or with 2c
        f16v sc[KB];
#pragma unroll
        for (int k = 0; k < KB; ++k) sc[k] = f16v{};
#pragma unroll
        for (int c = 0; c < NK; ++c) {
#pragma unroll
            for (int k = 0; k < KB; ++k) {
                if constexpr (DT == F16) {
                    sc[k] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, kk[c][k]), __builtin_bit_cast(h8, q[c]),
                                                                   sc[k], 0, 0, 0);
                } else {
                    const f4 kf = __builtin_bit_cast(f4, kk[c][k]), qf = __builtin_bit_cast(f4, q[c]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[k] = __builtin_amdgcn_mfma_f32_32x32x2f32(kf[e], qf[e], sc[k], 0, 0, 0);
                }
            }
        }
        const bool whole = j >= in_lo && j + TILE <= in_hi && j + TILE <= to && pages;
        by_rule(sc, j);
        if (!whole) {
            // seen: lo <= key < min(hi, to), as one unsigned comparison relative to this lane's first key
            const int at = lo - j - 4 * h;
            const unsigned many = max(min(hi, to) - lo, 0);
#pragma unroll
            for (int k = 0; k < KB; ++k)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    sc[k][r] = (unsigned)(32 * k + 8 * (r / 4) + r % 4 - at) < many ? sc[k][r] : -INFINITY;
            if (!pages) {                          // a page that is none hides its 8 keys or more
#pragma unroll
                for (int k = 0; k < KB; ++k)
#pragma unroll
                    for (int r = 0; r < 16; r += 4)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sc[k][r + i] = (ok >> (32 * k + 2 * r)) & 1 ? sc[k][r + i] : -INFINITY;
            }
        }
        raise(sc);
        const float off = LIFT<DT> - (ref == -INFINITY ? 0.0f : ref);
        float part = 0.0f;
        if constexpr (DT == F16) {
            // V^T: elements 32 t + m of the keys 16 n + {4 h + i, 8 + 4 h + i} (rows 16 n + 4 h .. + 3, then 8
            // further on, where the permutation is the same)
            h8 v[ND][2 * KB];
#pragma unroll
            for (int n = 0; n < 2 * KB; ++n)
#pragma unroll
                for (int t = 0; t < ND; ++t) {
                    const uint8_t* p0 = cur + ((vb0 ^ (t * 64)) + M::BYTES + n * 16 * ROW);
                    const s4v x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4v*)p0);
                    const s4v y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4v*)(p0 + 8 * ROW));
                    v[t][n] = __builtin_bit_cast(h8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
                }
            h8 p[2 * KB];
#pragma unroll
            for (int n = 0; n < 2 * KB; ++n)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float w = __builtin_amdgcn_exp2f(fmaf(sc[n / 2][8 * (n % 2) + e], unit, off));
                    part += w;
                    p[n][e] = (_Float16)w;
                }
#pragma unroll
            for (int n = 0; n < 2 * KB; ++n)
#pragma unroll
                for (int t = 0; t < ND; ++t) acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v[t][n], p[n], acc[t], 0, 0, 0);
        } else {
            // V: elements ND m .. ND m + ND - 1 of key 32 k + 8 (r / 4) + 4 h + r % 4
            typedef float vrow __attribute__((ext_vector_type(ND)));
            auto v_at = [&](int k, int r) {
                return *reinterpret_cast<const vrow*>(cur + M::BYTES + (32 * k + 8 * (r / 4) + 4 * h + r % 4) * ROW + m * ND * 4);
            };
#pragma unroll
            for (int k = 0; k < KB; ++k)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const vrow v = v_at(k, r);
                    const float w = __builtin_amdgcn_exp2f(fmaf(sc[k][r], unit, off));
                    part += w;
#pragma unroll
                    for (int t = 0; t < ND; ++t) acc[t] = __builtin_amdgcn_mfma_f32_32x32x2f32(v[t], w, acc[t], 0, 0, 0);
                }
        }
        sum += part;
    };
    if (from < to) {
        page = page_of(from);
        load_tile(a.c.k, from, page, k_off, k_ok, smem);
        load_tile(a.c.v, from, page, v_off, v_ok, smem + M::BYTES);
        page_next = page_of(from + TILE);
    }
    for (int j = from; j < to; j += 2 * TILE) {
        step(j, smem, smem + 2 * M::BYTES);
        if (j + TILE < to) step(j + TILE, smem + 2 * M::BYTES, smem);
    }

    sum += __shfl_xor(sum, 32, WAVE);
    if (!row) return;
    // acc[t][i]: element 32 t + 8 (i / 4) + 4 h + i % 4 (f16), ND (8 (i / 4) + 4 h + i % 4) + t (f32)
    const int64_t at = (((int64_t)flat * a.c.kv_heads + kvh) * a.splits + sp) * a.rows + my;
    auto put = [&](int e, f4 o) {
        if (!FULL && e >= d) return;
        if (n_split > 1) *reinterpret_cast<f4*>(a.part + at * d + e) = o;
        else store_row<DT>(a, tok, head, e, o, ref, sum);
    };
    if (n_split > 1 && h == 0) a.part_ml[at] = make_float2(ref, sum);
    if constexpr (DT == F16) {
#pragma unroll
        for (int t = 0; t < ND; ++t)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                put(32 * t + 8 * (i / 4) + 4 * h, f4{acc[t][i], acc[t][i + 1], acc[t][i + 2], acc[t][i + 3]});
    } else {
        float flat_out[16 * ND];
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int t = 0; t < ND; ++t) flat_out[i * ND + t] = acc[t][i];
#pragma unroll
        for (int i = 0; i < 16; i += 4)
#pragma unroll
            for (int x = 0; x < 4 * ND; x += 4)
                put(ND * (8 * (i / 4) + 4 * h) + x, f4{flat_out[i * ND + x], flat_out[i * ND + x + 1],
                                                       flat_out[i * ND + x + 2], flat_out[i * ND + x + 3]});
    }
}

// Join of a row's splits: four elements per thread, GROUPS threads for the same ones, each with every
// GROUPS-th split; the order of the sums is fixed.  Bound by its latencies: 4 us for two splits, 6.5 us for 64 (one
// thread for all of 128 splits: 41 us).
template <int DT, int GROUPS>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
    constexpr int PIECES = 256 / GROUPS;
    __shared__ f4 po[256];
    __shared__ float2 pml[256];
    const int flat = blockIdx.z, kvh = blockIdx.y, d = a.c.head_dim, pieces = d / 4;
    const int n = min(a.part_n[flat], a.splits);
    if (n <= 1) return;                           // written by the only one
    int s = flat, r0 = 0;
    if (a.rows > FEW_ROWS && !tile_at(a, flat, a.rows, a.most_rows, s, r0)) return;
    int t0, t1;
    seq_rows(a.b, s, t0, t1);
    const int g = threadIdx.x / PIECES;
    const int i = blockIdx.x * PIECES + threadIdx.x % PIECES, r = i / pieces, e = (i - r * pieces) * 4;
    const bool row = r < min(min((int64_t)(t1 - t0) * a.group, a.most_rows) - r0, (int64_t)a.rows);
    const int64_t at = ((int64_t)flat * a.c.kv_heads + kvh) * a.splits * a.rows + r;
    float top = -INFINITY, l = 0.0f;
    f4 o = f4{0, 0, 0, 0};
    // (a split that saw nothing holds no more than zeros)
    auto add = [&](float2 ml, f4 v) INLINE { add_part(weight_of(ml.x, top), ml.y, v, l, o); };
    if (row) {
#pragma unroll 4
        for (int k = g; k < n; k += GROUPS) top = fmaxf(top, a.part_ml[at + (int64_t)k * a.rows].x);
#pragma unroll 4
        for (int k = g; k < n; k += GROUPS)
            add(a.part_ml[at + (int64_t)k * a.rows], *reinterpret_cast<const f4*>(a.part + (at + (int64_t)k * a.rows) * d + e));
    }
    if (GROUPS > 1) {
        po[threadIdx.x] = o;
        pml[threadIdx.x] = make_float2(top, l);
        __syncthreads();
        if (g > 0) return;
#pragma unroll
        for (int k = 1; k < GROUPS; ++k) top = fmaxf(top, pml[threadIdx.x + k * PIECES].x);
        const float2 first = make_float2(pml[threadIdx.x].x, l);
        const f4 v = o;
        l = 0.0f;
        o = f4{0, 0, 0, 0};
        add(first, v);
#pragma unroll
        for (int k = 1; k < GROUPS; ++k) add(pml[threadIdx.x + k * PIECES], po[threadIdx.x + k * PIECES]);
    }
    if (row) store_row<DT>(a, t0 + (r0 + r) / a.group, kvh * a.group + (r0 + r) % a.group, e, o, top, l);
}

}  // namespace pi
