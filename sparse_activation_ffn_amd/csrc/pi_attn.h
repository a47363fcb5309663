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
// 2^-20 of the largest one).
#pragma once
#include <type_traits>

#include "pi_cache.h"

namespace pi {

typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

constexpr float LOG2E = 1.44269504088896340736f;
constexpr float LN2 = 0.69314718055994530942f;
constexpr float SLACK = 8.0f;
constexpr float LIFT = 6.0f;

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
    int rows;                         // rows per sequence and key head that the workspace holds
    float* part;                      // [n_seqs][kv_heads][splits][rows][head_dim], when splits > 1
    float2* part_ml;                  // [n_seqs][kv_heads][splits][rows]: reference, sum
    int* part_n;                      // [n_seqs]: splits that hold something
};

// keys that row t at position pos of sequence s sees
__device__ __forceinline__ void visible(const AttnArgs& a, int t, int pos, int s, int len, int& lo, int& hi) {
    lo = a.first ? max(a.first[t], 0) : 0;
    if (a.window > 0) lo = max(lo, pos - a.window + 1);
    hi = pos + 1;
    if (a.prefix) hi = max(hi, a.prefix[s]);
    hi = min(hi, len);
}

// weight of a sum taken against reference m, seen from reference top (-inf: nothing was summed)
__device__ __forceinline__ float weight_of(float m, float top) {
    return m == -INFINITY ? 0.0f : m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top);
}

__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? -INFINITY : (m - LIFT + __builtin_amdgcn_logf(l)) * LN2;
}

template <int DT> struct ElemT;
template <> struct ElemT<F32> { typedef float T; typedef f4 V4; };
template <> struct ElemT<F16> { typedef _Float16 T; typedef h4 V4; };

// elements e..e+3 of a row's output from its sums (reference m, sum of weights l)
template <int DT>
__device__ __forceinline__ void store_row(const AttnArgs& a, int t, int head, int e, f4 o, float m, float l) {
    typedef typename ElemT<DT>::T T;
    typedef typename ElemT<DT>::V4 V4;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    V4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (T)(o[i] * inv);
    *reinterpret_cast<V4*>((T*)a.out + t * a.o_ts + head * a.o_hs + e) = v;
    if (e == 0 && a.lse) a.lse[(int64_t)t * a.q_heads + head] = lse_of(m, l);
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

template <int DT, int DP, bool FULL>
__global__ __launch_bounds__(WAVE * FEW_WAVES, DP == 64 ? 3 : DP == 128 ? 2 : 1) void k_attn_few(AttnArgs a) {
    typedef Few<DT, DP> F;
    constexpr int STEP = F::STEP, U = STEP / 16, EV = F::EV, VW = F::VW;
    constexpr int NK = DP / (4 * EV);              // 16-byte pieces of a key per lane
    constexpr int NV = DP / (16 * VW);             // pieces of a value row per lane
    constexpr int ES = 16 / EV;                    // bytes per element
    extern __shared__ float lds[];

    const int s = blockIdx.z, kvh = blockIdx.y, sp = blockIdx.x;
    const int lane = threadIdx.x % WAVE, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int m = lane % 16, g = lane / 16;
    const int d = FULL ? DP : a.c.head_dim;
    const int ps = a.c.page_size, shift = a.c.page_shift;

    const int t0 = max(a.b.q_start[s], 0), t1 = min(a.b.q_start[s + 1], a.b.n_tokens);
    const int len = clamped_len(a.b, shift, s), q_end = a.b.q_start[s + 1];
    const int n_rows = min((t1 - t0) * a.group, a.rows);
    if (n_rows <= 0) return;

    // this lane's row, and the keys it sees; lanes without a row see whatever the others do
    const int tok = t0 + m / a.group, head = kvh * a.group + m % a.group;
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
    if (a.splits > 1 && sp == 0 && kvh == 0 && threadIdx.x == 0) a.part_n[s] = n_split;
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
    const float slope = a.slopes && row ? a.slopes[head] * LOG2E : 0.0f;
    const float scale = a.cap > 0.0f ? a.scale / a.cap : a.scale * LOG2E;

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
    // byte offset of key j + i (i in the 8 keys `eight` of the step); a page that is none reads page 0, masked
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
                if (a.cap > 0.0f) v = a.cap * LOG2E * tanhf(v);
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
        const float off = LIFT - (ref == -INFINITY ? 0.0f : ref);
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
            if (f == 0.0f) continue;
            l += f * ml[(w * FEW_ROWS + r) * 2 + 1];
            o += f * *reinterpret_cast<const f4*>(o_lds + (w * FEW_ROWS + r) * LD + e);
        }
        if (n_split > 1) {
            const int64_t at = (((int64_t)s * a.c.kv_heads + kvh) * a.splits + sp) * a.rows + r;
            *reinterpret_cast<f4*>(a.part + at * d + e) = o;
            if (e == 0) a.part_ml[at] = make_float2(all, l);
        } else {
            store_row<DT>(a, t0 + r / a.group, kvh * a.group + r % a.group, e, o, all, l);
        }
    }
}

// Join of a row's splits, in their order: four elements per thread.
template <int DT>
__global__ __launch_bounds__(WAVE) void k_attn_join(AttnArgs a) {
    const int s = blockIdx.z, kvh = blockIdx.y, d = a.c.head_dim, pieces = d / 4;
    const int t0 = max(a.b.q_start[s], 0), t1 = min(a.b.q_start[s + 1], a.b.n_tokens);
    const int i = blockIdx.x * WAVE + threadIdx.x, r = i / pieces, e = (i - r * pieces) * 4;
    if (r >= min((t1 - t0) * a.group, a.rows)) return;
    const int n = min(a.part_n[s], a.splits);
    if (n <= 1) return;                           // written by the only one
    const int64_t at = ((int64_t)s * a.c.kv_heads + kvh) * a.splits * a.rows + r;
    float top = -INFINITY, l = 0.0f;
#pragma unroll 8
    for (int k = 0; k < n; ++k) top = fmaxf(top, a.part_ml[at + (int64_t)k * a.rows].x);
    f4 o = f4{0, 0, 0, 0};
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
        const float2 ml = a.part_ml[at + (int64_t)k * a.rows];
        const f4 v = *reinterpret_cast<const f4*>(a.part + (at + (int64_t)k * a.rows) * d + e);
        const float f = weight_of(ml.x, top);
        l += f == 0.0f ? 0.0f : f * ml.y;
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] += f == 0.0f ? 0.0f : f * v[c];
    }
    store_row<DT>(a, t0 + r / a.group, kvh * a.group + r % a.group, e, o, top, l);
}

}  // namespace pi
