// pi_sample.hip -- a token from each row of logits.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "pi.h"
#include "pi_cache.h"
#include "pi_launch.h"
#include "pi_mx.h"

using namespace pi;

namespace {

constexpr int ST = 512;                  // threads of a workgroup
constexpr int EACH = 8;                  // logits of a thread and step
constexpr int BINS = 2048;               // of a row's histogram
constexpr int LIST = 4096;               // tokens in the bins that a rule's border lies in
constexpr int BLOCK = ST * EACH;         // logits of a workgroup and step: sums are kept for each
constexpr int MOST_BLOCKS = 256;         // of a row: 2^20 logits

typedef unsigned long long u64;
constexpr int FRACTION = 43;             // weights are integers of 2^-43: 2^20 of them sum below 2^63

struct SampleArgs {
    const uint8_t* logits;
    int64_t stride;                      // in elements
    const float* temperature;
    const int* top_k;
    const float* top_p;
    const float* min_p;
    const float* u;
    int* token;
    float* prob;
    int* kept;
    int rows, vocab;
    int chunks, chunk, blocks;           // workgroups of a row, logits of one (a multiple of BLOCK); blocks of a row
    uint8_t* ws;
    int64_t row_bytes;                   // of ws
};

// What the workgroups of a row leave for each other (offsets in the row's part of the workspace).
struct Top {
    unsigned most, least;                // largest and smallest key of a chunk (0: none)
    int at, count;                       // lowest index of the largest; tokens that may be kept
};
struct RowState {
    u64 mass_lo, p_before;               // weights before k_bin and before the lowest bin of top-p's border
    int k_bin, k_before;
    unsigned listed;                     // tokens in the list
};
constexpr int64_t WS_STATE = 0;
constexpr int64_t WS_TOPS = 256;                                   // Top [chunks]
constexpr int64_t WS_MASS = WS_TOPS + MOST_BLOCKS * 16;            // u64 [BINS]
constexpr int64_t WS_COUNT = WS_MASS + BINS * 8;                   // unsigned [BINS]
constexpr int64_t WS_BLOCK_MASS = WS_COUNT + BINS * 4;             // u64 [blocks]
constexpr int64_t WS_BLOCK_KEPT = WS_BLOCK_MASS + MOST_BLOCKS * 8; // unsigned [blocks]
constexpr int64_t WS_LIST = WS_BLOCK_KEPT + MOST_BLOCKS * 4;       // u64 [LIST]: key above the index's complement
constexpr int64_t WS_ROW = WS_LIST + LIST * 8;

// A logit as an unsigned integer in the same order; 0 for -inf and NaN, which are never kept.  -0 and 0 are equal.
__device__ __forceinline__ unsigned order_key(float l) {
    const unsigned b = __builtin_bit_cast(unsigned, l + 0.0f);
    return l > -INFINITY ? (b >> 31 ? ~b : b | 0x80000000u) : 0u;
}
__device__ __forceinline__ float key_logit(unsigned key) {
    return __builtin_bit_cast(float, key >> 31 ? key & 0x7fffffffu : ~key);
}

// exp for z <= 0 by a table of 2^(j/32) (Tang, ACM TOMS 15(2), 1989): z = (32 m + j) ln 2 / 32 + r with |r| <= ln 2 / 64, exp(z)
// = 2^m 2^(j/32) exp(r), exp(r) by its series to r^5 (the next term is 2^-49).  Weights are needed to 2^-44; the library's
// function takes three times the operations, and a row's distribution hundreds of thousands of them.
__constant__ double EXP2_32[32] = {
    0x1.0000000000000p+0, 0x1.059b0d3158574p+0, 0x1.0b5586cf9890fp+0, 0x1.11301d0125b51p+0,
    0x1.172b83c7d517bp+0, 0x1.1d4873168b9aap+0, 0x1.2387a6e756238p+0, 0x1.29e9df51fdee1p+0,
    0x1.306fe0a31b715p+0, 0x1.371a7373aa9cbp+0, 0x1.3dea64c123422p+0, 0x1.44e086061892dp+0,
    0x1.4bfdad5362a27p+0, 0x1.5342b569d4f82p+0, 0x1.5ab07dd485429p+0, 0x1.6247eb03a5585p+0,
    0x1.6a09e667f3bcdp+0, 0x1.71f75e8ec5f74p+0, 0x1.7a11473eb0187p+0, 0x1.82589994cce13p+0,
    0x1.8ace5422aa0dbp+0, 0x1.93737b0cdc5e5p+0, 0x1.9c49182a3f090p+0, 0x1.a5503b23e255dp+0,
    0x1.ae89f995ad3adp+0, 0x1.b7f76f2fb5e47p+0, 0x1.c199bdd85529cp+0, 0x1.cb720dcef9069p+0,
    0x1.d5818dcfba487p+0, 0x1.dfc97337b9b5fp+0, 0x1.ea4afa2a490dap+0, 0x1.f50765b6e4540p+0};

constexpr double LN2 = 0.693147180559945309417;

struct Exp {
    const double* table;                 // in LDS
    // the whole workgroup calls it, a barrier follows before the first use
    static __device__ void fill(double* lds) {
        if (threadIdx.x < 32) lds[threadIdx.x] = EXP2_32[threadIdx.x];
    }
    __device__ __forceinline__ double operator()(double z) const {
        if (z < -110.0) return 0.0;      // (below the least float32, which min-p may be)
        // the nearest integer by the addition of 1.5 2^52, in whose lowest bits it then is
        const double t = fma(z, 32 / LN2, 0x1.8p52), n = t - 0x1.8p52;
        const int i = (int)(unsigned)__builtin_bit_cast(uint64_t, t);
        const double r = fma(n, -LN2 / 32, z);     // (ln 2's own rounding: |z| 2^-54, below 2^-47)
        double p = fma(r, 1.0 / 120, 1.0 / 24);
        p = fma(r, p, 1.0 / 6);
        p = fma(r, p, 0.5);
        p = fma(r, p, 1.0);
        p = fma(r, p, 1.0);
        // times 2^(i / 32): the product is in 1 .. 2 and the result no smaller than 2^-159
        return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, table[i & 31] * p) + ((uint64_t)(int64_t)(i >> 5) << 52));
    }
};

// What the rules of a row come to.
struct Rule {
    double inv_t, min_p, top_p;          // min_p 0 and top_p 1: none
    float top;                           // the largest logit
    int top_k;                           // 0: none
    bool greedy;

    const double* table;                 // of Exp

    // exp((l - max) / T) of a logit that may be kept
    __device__ __forceinline__ double weight(float l) const {
        return l == top ? 1.0 : top == INFINITY ? 0.0 : Exp{table}(((double)l - (double)top) * inv_t);
    }
};

// the nearest integer to w 2^43, w in 0 .. 1: the lowest bits of its sum with 2^52
__device__ __forceinline__ uint64_t fixed(double w) {
    return __builtin_bit_cast(uint64_t, fma(w, (double)(1ull << FRACTION), 0x1p52)) & ((1ull << 52) - 1);
}

// (table: 32 numbers in LDS, filled here; a barrier follows)
__device__ __forceinline__ Rule rule_of(const SampleArgs& a, int row, double* table) {
    Rule r;
    Exp::fill(table);
    r.table = table;
    const float t = a.temperature ? a.temperature[row] : 1.0f;
    r.greedy = !(t > 0.0f);
    r.inv_t = r.greedy ? 1.0 : 1.0 / (double)t;
    r.top_k = a.top_k ? max(a.top_k[row], 0) : 0;
    const float p = a.top_p ? a.top_p[row] : 1.0f, m = a.min_p ? a.min_p[row] : 0.0f;
    r.top_p = p < 1.0f ? (double)p : 1.0;
    r.min_p = m > 0.0f ? fmin((double)m, 1.0) : 0.0;
    return r;
}

template <int DT>
__device__ __forceinline__ float logit(const uint8_t* row, int i) {
    return DT == F16 ? (float)reinterpret_cast<const _Float16*>(row)[i] : reinterpret_cast<const float*>(row)[i];
}

// The lane's value from the one that CTRL selects, 0 where there is none or the row is outside ROW_MASK (a shuffle through LDS
// takes ten times as long, and these sums wait for each other).
template <int CTRL, int ROW_MASK = 0xf>
__device__ __forceinline__ unsigned moved(unsigned v) {
    return (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROW_MASK, 0xf, false);
}
template <int CTRL, int ROW_MASK = 0xf>
__device__ __forceinline__ u64 moved(u64 v) {
    return (u64)moved<CTRL, ROW_MASK>((unsigned)(v >> 32)) << 32 | moved<CTRL, ROW_MASK>((unsigned)v);
}
// sum over lanes 0 .. this one
__device__ __forceinline__ u64 wave_scan(u64 v) {
    v += moved<DPP_ROW_SHR1>(v);
    v += moved<DPP_ROW_SHR1 + 1>(v);
    v += moved<DPP_ROW_SHR1 + 3>(v);
    v += moved<DPP_ROW_SHR1 + 7>(v);
    v += moved<DPP_ROW_BCAST15, 0xA>(v);
    v += moved<DPP_ROW_BCAST31, 0xC>(v);
    return v;
}
__device__ __forceinline__ u64 last_lane(u64 v) {
    return (u64)(unsigned)__builtin_amdgcn_readlane((int)(v >> 32), WAVE - 1) << 32 |
           (unsigned)__builtin_amdgcn_readlane((int)(unsigned)v, WAVE - 1);
}
__device__ __forceinline__ u64 wave_sum(u64 v) { return last_lane(wave_scan(v)); }
__device__ __forceinline__ unsigned wave_max(unsigned v) {
    v = max(v, moved<DPP_ROW_SHR1>(v));
    v = max(v, moved<DPP_ROW_SHR1 + 1>(v));
    v = max(v, moved<DPP_ROW_SHR1 + 3>(v));
    v = max(v, moved<DPP_ROW_SHR1 + 7>(v));
    v = max(v, moved<DPP_ROW_BCAST15, 0xA>(v));
    v = max(v, moved<DPP_ROW_BCAST31, 0xC>(v));
    return (unsigned)__builtin_amdgcn_readlane((int)v, WAVE - 1);
}

// Sums of a value over the threads before this one, and over all.
__device__ __forceinline__ u64 before_and_total(u64 v, u64* lds, u64& total) {
    const u64 incl = wave_scan(v);
    __syncthreads();
    if (threadIdx.x % WAVE == WAVE - 1) lds[threadIdx.x / WAVE] = incl;
    __syncthreads();
    u64 base = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < ST / WAVE; ++w) {
        const u64 sum = lds[w];
        if (w < (int)threadIdx.x / WAVE) base += sum;
        total += sum;
    }
    return base + incl - v;
}

// A row by one workgroup, whatever it holds: the border of the kept set, in the order of the keys, is found digit by digit (8
// bits, from the top), top-k by counts, top-p by sums of weights.  mass has room for 256.
template <int DT>
__device__ void whole_row(const SampleArgs& a, int row, const Rule& rule, u64* mass, u64* scan) {
    __shared__ unsigned s_key;
    __shared__ u64 s_before;
    const int tid = threadIdx.x;
    const uint8_t* l = a.logits + row * a.stride * (DT == F16 ? 2 : 4);

    // kept: keys above `key`, and of those equal to it the first `ties` by index
    unsigned key = 1;
    int64_t ties = a.vocab;
    for (int by_mass = 0; by_mass < 2; ++by_mass) {
        if (by_mass ? rule.top_p >= 1.0 : rule.top_k == 0) continue;
        // what lies above the digits found so far, and what is looked for: the last token with less than `want` before it
        u64 before = 0, want = by_mass ? 0 : (u64)rule.top_k;
        unsigned found = 0;
        bool all = false;
        const unsigned floor_key = key;
        const int64_t floor_ties = ties;
        for (int shift = 24; shift >= 0 && !all; shift -= 8) {
            for (int b = tid; b < 256; b += ST) mass[b] = 0;
            __syncthreads();
            for (int i = tid; i < a.vocab; i += ST) {
                const float x = logit<DT>(l, i);
                const unsigned k = order_key(x);
                if (k < floor_key || (shift < 24 && (k >> (shift + 8)) != (found >> (shift + 8)))) continue;
                // (tokens at the floor weigh alike; as many as it keeps are added below)
                if (by_mass && k == floor_key && floor_ties < a.vocab) continue;
                atomicAdd(&mass[k >> shift & 255], by_mass ? (u64)fixed(rule.weight(x)) : 1ull);
            }
            __syncthreads();
            if (tid == 0) {
                if (by_mass && floor_ties < a.vocab && (shift == 24 || floor_key >> (shift + 8) == found >> (shift + 8)))
                    mass[floor_key >> shift & 255] += floor_ties * fixed(rule.weight(key_logit(floor_key)));
                if (by_mass && shift == 24) {
                    u64 total = 0;
                    for (int b = 0; b < 256; ++b) total += mass[b];
                    const double p = ceil(rule.top_p * (double)total);
                    want = p > 1.0 ? (u64)p : 1;
                    scan[0] = want;
                }
                int b = 255;
                u64 sum = before;
                for (; b > 0 && sum + mass[b] < want; --b) sum += mass[b];
                s_before = sum;
                // fewer than `want` in all
                s_key = sum + mass[b] < want ? 0xffffffffu : (unsigned)b;
            }
            __syncthreads();
            if (by_mass && shift == 24) want = scan[0];
            if (s_key == 0xffffffffu) all = true;
            else found |= s_key << shift;
            before = s_before;
            __syncthreads();
        }
        if (all) continue;
        if (by_mass) {
            const u64 each = fixed(rule.weight(key_logit(found)));
            ties = each ? (int64_t)((want - before + each - 1) / each) : 1;
            if (found == floor_key) ties = min(ties, floor_ties);
        } else {
            ties = (int64_t)(want - before);
        }
        key = found;
    }

    // every thread a piece of the row, in order
    const int piece = (a.vocab + ST - 1) / ST, lo = min(tid * piece, a.vocab), hi = min(lo + piece, a.vocab);
    int equal = 0;
    for (int i = lo; i < hi; ++i) equal += order_key(logit<DT>(l, i)) == key;
    u64 total;
    const int64_t equal_before = (int64_t)before_and_total(equal, scan, total);
    u64 sum = 0, n = 0;
    int64_t rank = equal_before;
    for (int i = lo; i < hi; ++i) {
        const float x = logit<DT>(l, i);
        const unsigned k = order_key(x);
        if (k < key || (k == key && rank++ >= ties)) continue;
        const double w = rule.weight(x);
        if (w >= rule.min_p) sum += fixed(w), ++n;
    }
    const u64 before = before_and_total(sum, scan, total);
    u64 all_kept;
    before_and_total(n, scan, all_kept);
    const float u = a.u[row];
    u64 target = u > 0.0f ? (u64)((double)u * (double)total) : 0;
    if (u >= 1.0f || target >= total) target = total - 1;
    if (tid == 0 && a.kept) a.kept[row] = (int)all_kept;
    if (target < before || target >= before + sum) return;
    rank = equal_before;
    u64 run = before;
    for (int i = lo; i < hi; ++i) {
        const float x = logit<DT>(l, i);
        const unsigned k = order_key(x);
        if (k < key || (k == key && rank++ >= ties)) continue;
        const double w = rule.weight(x);
        if (w < rule.min_p) continue;
        run += fixed(w);
        if (run > target) {
            a.token[row] = i;
            if (a.prob) a.prob[row] = (float)((double)fixed(w) / (double)total);
            return;
        }
    }
}

// ---- a row by many workgroups --------------------------------------------------------
//
// The logits' bytes would take a microsecond or two (64 rows of 151003 in f16: 3.9); what there is to do is to keep a row's
// pieces busy at the same time, and to read them few times.  Four launches, a workgroup to each chunk of a row but in the
// last; us for 64 x 151003 f16 with rules of every kind, for 48 x 50007 float32 with top-p and for 1 x 128000 with top-k:
//   k_sample_top     the largest and smallest logit of the chunk                                              9.8   5.8   3.7
//   k_sample_count   with the row's largest known: the chunk's part of a histogram of the distance to it
//                    (counts for top-k, sums of weights for top-p); without either rule the sum of its
//                    weights                                                                                 19.5  11.9   5.9
//   k_sample_list    from the histogram the bins in which the border of top-k and of top-p can lie: sums
//                    over the tokens above them, and a list of the tokens in them (left out where no row
//                    has either rule)                                                                        18.7  14.2   6.9
//   k_sample_pick    a workgroup to each row: sorts the list, finds the border and the token                 13.7  10.9   8.1
// The whole call: 60.8, 40.8 and 24.1 us.  A dependent launch costs some 4 us here; what is left are the chains of sums in
// each, weights in 64 bits and additions to LDS, not bytes.  (A row's last workgroup doing the pick in the launch before
// needs fences between the dies, which write back and drop whole caches: 26 us in place of 13 for one row, 108 for 64.)
// Sums are integers, so that neither their order nor that of the list matters.  A row whose border bins hold more than
// LIST tokens (equal logits, or a border far below the others) is done by k_sample_pick alone, from the start: 0.5 to
// 0.9 ms for 128000 logits, equal ones or normal ones of a tenth of the temperature beside one of -1e30.

// 8 logits from i on; those past the row's end are -inf
template <int DT>
__device__ __forceinline__ void load_logits(const uint8_t* row, int i, int vocab, float* v) {
    if (i + EACH <= vocab) {
        if constexpr (DT == F16) {
            h8 t;
            __builtin_memcpy(&t, row + (int64_t)i * 2, 16);
#pragma unroll
            for (int e = 0; e < EACH; ++e) v[e] = (float)t[e];
        } else {
            f4 t[2];
            __builtin_memcpy(t, row + (int64_t)i * 4, 32);
#pragma unroll
            for (int e = 0; e < EACH; ++e) v[e] = t[e / 4][e % 4];
        }
    } else {
#pragma unroll
        for (int e = 0; e < EACH; ++e) v[e] = i + e < vocab ? logit<DT>(row, i + e) : -INFINITY;
    }
}

template <int DT>
__global__ __launch_bounds__(ST) void k_sample_top(SampleArgs a) {
    __shared__ unsigned s_most[ST / WAVE], s_least[ST / WAVE], s_at[ST / WAVE];
    __shared__ int s_count[ST / WAVE];
    const int row = blockIdx.y, tid = threadIdx.x, wave = tid / WAVE;
    const uint8_t* l = a.logits + row * a.stride * (DT == F16 ? 2 : 4);
    uint8_t* ws = a.ws + row * a.row_bytes;
    // what the later launches add to
    for (int b = blockIdx.x * ST + tid; b < BINS; b += gridDim.x * ST) {
        reinterpret_cast<u64*>(ws + WS_MASS)[b] = 0;
        reinterpret_cast<unsigned*>(ws + WS_COUNT)[b] = 0;
    }
    if (blockIdx.x == 0 && tid == 0) reinterpret_cast<RowState*>(ws + WS_STATE)->listed = 0;

    // the smallest key as the largest of the complements
    unsigned most = 0, low = 0, at = 0;
    int count = 0;
    const int from = blockIdx.x * a.chunk, to = min(from + a.chunk, a.vocab);
    for (int i = from + tid * EACH; i < to; i += ST * EACH) {
        float v[EACH];
        load_logits<DT>(l, i, a.vocab, v);
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const unsigned key = order_key(v[e]);
            if (key > most) most = key, at = i + e;
            low = max(low, key ? ~key : 0u);
            count += key != 0;
        }
    }
    const unsigned top = wave_max(most);
    // the lowest index of the largest (a thread has met its own lowest first)
    const unsigned first = ~wave_max(most == top ? ~at : 0u);
    low = wave_max(low);
    count = (int)wave_sum((u64)count);
    if (tid % WAVE == 0) s_most[wave] = top, s_at[wave] = first, s_least[wave] = low, s_count[wave] = count;
    __syncthreads();
    if (tid) return;
    Top t{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < ST / WAVE; ++w) {
        if (s_most[w] > t.most || (s_most[w] == t.most && (int)s_at[w] < t.at)) t.most = s_most[w], t.at = (int)s_at[w];
        t.least = max(t.least, s_least[w]);
        t.count += s_count[w];
    }
    t.least = ~t.least;
    reinterpret_cast<Top*>(ws + WS_TOPS)[blockIdx.x] = t;
}

// The row's largest and smallest key, the largest's lowest index, and the tokens that may be kept, from its chunks'.
__device__ __forceinline__ Top row_top(const SampleArgs& a, const uint8_t* ws, Top* s_top) {
    if (threadIdx.x < WAVE) {
        Top t{0, ~0u, 0, 0};
        for (int c = threadIdx.x; c < a.chunks; c += WAVE) {
            const Top o = reinterpret_cast<const Top*>(ws + WS_TOPS)[c];
            if (o.most > t.most) t.most = o.most, t.at = o.at;
            t.least = min(t.least, o.least);
            t.count += o.count;
        }
        const unsigned top = wave_max(t.most);
        t.at = (int)~wave_max(t.most == top ? ~(unsigned)t.at : 0u);
        t.least = ~wave_max(~t.least);
        t.count = (int)wave_sum((u64)t.count);
        t.most = top;
        if (threadIdx.x == 0) *s_top = t;
    }
    __syncthreads();
    return *s_top;
}

// Bin of a logit: its distance to the largest, in steps that cover the tokens with a weight (40 temperatures) or, for top-k,
// at least 64; everything farther in the last one.
struct Binning {
    float top, scale;
    __device__ Binning(const Rule& r, const Top& t) : top(r.top) {
        const float range = top - key_logit(t.least), span = (float)(40.0 / r.inv_t);
        const float most = fminf(fminf(range, r.top_k ? fmaxf(span, 64.0f) : span), 3e38f);
        scale = most > 0.0f ? (float)(BINS - 1) / most : 0.0f;
        if (!(scale < INFINITY)) scale = 3e38f;
    }
    __device__ __forceinline__ int of(float l) const {
        if (l == top) return 0;
        return (int)fminf((top - l) * scale, (float)(BINS - 1));
    }
};

// adds what the workgroup's threads have to a block's sum of weights and count
__device__ __forceinline__ void add_block(u64 sum, unsigned n, u64* mass, unsigned* count) {
    if (!__any(n != 0)) return;
    sum = wave_sum(sum);
    n = (unsigned)wave_sum((u64)n);
    if (threadIdx.x % WAVE == 0) atomicAdd(mass, sum), atomicAdd(count, n);
}

// the sums of this workgroup's blocks to the workspace
__device__ __forceinline__ void store_blocks(const SampleArgs& a, uint8_t* ws, const u64* mass, const unsigned* count) {
    const int first = blockIdx.x * (a.chunk / BLOCK);
    for (int b = threadIdx.x; b < a.chunk / BLOCK && first + b < a.blocks; b += ST) {
        reinterpret_cast<u64*>(ws + WS_BLOCK_MASS)[first + b] = mass[b];
        reinterpret_cast<unsigned*>(ws + WS_BLOCK_KEPT)[first + b] = count[b];
    }
}

template <int DT>
__global__ __launch_bounds__(ST) void k_sample_count(SampleArgs a) {
    __shared__ u64 s_mass[BINS];
    __shared__ unsigned s_count[BINS];
    __shared__ Top s_top;
    const int row = blockIdx.y, tid = threadIdx.x;
    const uint8_t* l = a.logits + row * a.stride * (DT == F16 ? 2 : 4);
    uint8_t* ws = a.ws + row * a.row_bytes;
    __shared__ double s_exp[32];
    Rule rule = rule_of(a, row, s_exp);
    const Top t = row_top(a, ws, &s_top);
    if (t.most == 0 || rule.greedy) return;
    rule.top = key_logit(t.most);
    if (rule.top_k >= t.count) rule.top_k = 0;
    const bool by_count = rule.top_k != 0, by_mass = rule.top_p < 1.0;
    const int from = blockIdx.x * a.chunk, to = min(from + a.chunk, a.vocab);
    if (!by_count && !by_mass) {
        for (int b = tid; b < MOST_BLOCKS; b += ST) s_mass[b] = 0, s_count[b] = 0;
        __syncthreads();
        for (int base = from, b = 0; base < to; base += BLOCK, ++b) {
            u64 sum = 0;
            unsigned n = 0;
            float v[EACH];
            load_logits<DT>(l, base + tid * EACH, a.vocab, v);
#pragma unroll
            for (int e = 0; e < EACH; ++e) {
                if (!order_key(v[e])) continue;
                const double w = rule.weight(v[e]);
                if (w >= rule.min_p) sum += fixed(w), ++n;
            }
            add_block(sum, n, &s_mass[b], &s_count[b]);
        }
        __syncthreads();
        store_blocks(a, ws, s_mass, s_count);
        return;
    }
    const Binning bin(rule, t);
    for (int b = tid; b < BINS; b += ST) s_mass[b] = 0, s_count[b] = 0;
    __syncthreads();
    for (int i = from + tid * EACH; i < to; i += ST * EACH) {
        float v[EACH];
        load_logits<DT>(l, i, a.vocab, v);
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            if (!order_key(v[e])) continue;
            const int b = bin.of(v[e]);
            if (by_count) atomicAdd(&s_count[b], 1u);
            if (by_mass) {
                const u64 w = fixed(rule.weight(v[e]));
                if (w) atomicAdd(&s_mass[b], w);
            }
        }
    }
    __syncthreads();
    for (int b = tid; b < BINS; b += ST) {
        if (s_count[b]) atomicAdd(reinterpret_cast<unsigned*>(ws + WS_COUNT) + b, s_count[b]);
        if (s_mass[b]) atomicAdd(reinterpret_cast<u64*>(ws + WS_MASS) + b, s_mass[b]);
    }
}

// the lowest bin with which the running sum reaches `want`; BINS if none does.  before: the sum of this thread's bins'
// predecessors; own: its BINS / ST bins' values
__device__ __forceinline__ void find_bin(u64 want, u64 before, const u64* own, int* s_bin) {
    u64 sum = before;
#pragma unroll
    for (int e = 0; e < BINS / ST; ++e) {
        if (sum < want && sum + own[e] >= want) *s_bin = threadIdx.x * (BINS / ST) + e;
        sum += own[e];
    }
}

template <int DT>
__global__ __launch_bounds__(ST) void k_sample_list(SampleArgs a) {
    __shared__ u64 s_list[LIST];
    __shared__ unsigned s_listed, s_first;
    __shared__ u64 scan[ST / WAVE];
    __shared__ u64 s_mass[MOST_BLOCKS];
    __shared__ unsigned s_kept[MOST_BLOCKS];
    __shared__ Top s_top;
    __shared__ int s_bin[3];
    __shared__ u64 s_at[4];
    const int row = blockIdx.y, tid = threadIdx.x;
    const uint8_t* l = a.logits + row * a.stride * (DT == F16 ? 2 : 4);
    uint8_t* ws = a.ws + row * a.row_bytes;
    RowState* state = reinterpret_cast<RowState*>(ws + WS_STATE);
    __shared__ double s_exp[32];
    Rule rule = rule_of(a, row, s_exp);
    if (rule.greedy || (rule.top_k == 0 && rule.top_p >= 1.0)) return;
    const Top t = row_top(a, ws, &s_top);
    rule.top = key_logit(t.most);
    if (rule.top_k >= t.count) rule.top_k = 0;
    const bool by_count = rule.top_k != 0, by_mass = rule.top_p < 1.0;
    if (t.most == 0 || !(by_count || by_mass)) return;
    const Binning bin(rule, t);

    // Bins: k_bin holds the border of top-k; the sum that top-p is a part of lies between those without and with it, so the
    // border of top-p lies in p_lo .. p_hi.
    int k_bin = BINS, p_lo = BINS, p_hi = BINS;
    u64 k_before = 0, mass_lo = 0, p_before = 0;      // tokens before k_bin, weights before it and before p_lo
    u64 n[BINS / ST], m[BINS / ST], own_n = 0, own_m = 0, all_n, all_m;
#pragma unroll
    for (int e = 0; e < BINS / ST; ++e) {
        n[e] = reinterpret_cast<const unsigned*>(ws + WS_COUNT)[tid * (BINS / ST) + e];
        m[e] = reinterpret_cast<const u64*>(ws + WS_MASS)[tid * (BINS / ST) + e];
        own_n += n[e], own_m += m[e];
    }
    const u64 before_n = before_and_total(own_n, scan, all_n), before_m = before_and_total(own_m, scan, all_m);
    if (tid < 3) s_bin[tid] = BINS;
    __syncthreads();
    if (by_count) find_bin((u64)rule.top_k, before_n, n, &s_bin[0]);
    __syncthreads();
    k_bin = s_bin[0];
    if (tid == 0) s_at[0] = s_at[2] = 0, s_at[1] = s_at[3] = all_m;
    __syncthreads();
    if (k_bin < BINS && k_bin / (BINS / ST) == tid) {
        u64 c = before_n, w = before_m;
        for (int e = 0; e < k_bin % (BINS / ST); ++e) c += n[e], w += m[e];
        s_at[0] = c, s_at[1] = w, s_at[3] = w + m[k_bin % (BINS / ST)];
    }
    __syncthreads();
    k_before = s_at[0], mass_lo = s_at[1];
    if (by_mass) {
        const double lo = ceil(rule.top_p * (double)mass_lo), hi = ceil(rule.top_p * (double)s_at[3]);
        find_bin(lo > 1.0 ? (u64)lo : 1, before_m, m, &s_bin[1]);
        find_bin(hi > 1.0 ? (u64)hi : 1, before_m, m, &s_bin[2]);
        __syncthreads();
        p_lo = s_bin[1], p_hi = s_bin[2];
        if (p_lo < BINS && p_lo / (BINS / ST) == tid) {
            u64 w = before_m;
            for (int e = 0; e < p_lo % (BINS / ST); ++e) w += m[e];
            s_at[2] = w;
        }
        __syncthreads();
        p_before = s_at[2];
    }
    if (blockIdx.x == 0 && tid == 0) state->mass_lo = mass_lo, state->p_before = p_before, state->k_bin = k_bin, state->k_before = (int)k_before;
    const int border = by_mass ? p_lo : k_bin;           // bins before it are kept for certain

    for (int b = tid; b < MOST_BLOCKS; b += ST) s_mass[b] = 0, s_kept[b] = 0;
    if (tid == 0) s_listed = 0;
    __syncthreads();
    const int from = blockIdx.x * a.chunk, to = min(from + a.chunk, a.vocab);
    for (int base = from, block = 0; base < to; base += BLOCK, ++block) {
        u64 sum = 0;
        unsigned n = 0, in_list = 0;               // (a bit for each)
        float v[EACH];
        load_logits<DT>(l, base + tid * EACH, a.vocab, v);
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            if (!order_key(v[e])) continue;
            const int b = bin.of(v[e]);
            if (b < border) {
                const double w = rule.weight(v[e]);
                if (w >= rule.min_p) sum += fixed(w), ++n;
            } else if (b == k_bin || (by_mass && b <= p_hi)) {
                in_list |= 1u << e;
            }
        }
        if (__any(in_list != 0)) {
            const int mine = __popc(in_list), incl = wave_incl_scan(mine);
            unsigned at = 0;
            if (tid % WAVE == WAVE - 1) at = atomicAdd(&s_listed, (unsigned)incl);
            at = __shfl(at, WAVE - 1) + incl - mine;
#pragma unroll
            for (int e = 0; e < EACH; ++e) {
                if (!(in_list >> e & 1)) continue;
                if (at < LIST) s_list[at] = (u64)order_key(v[e]) << 32 | ~(unsigned)(base + tid * EACH + e);
                ++at;
            }
        }
        add_block(sum, n, &s_mass[block], &s_kept[block]);
    }
    __syncthreads();
    store_blocks(a, ws, s_mass, s_kept);
    // one addition to the row's count for all of the workgroup's tokens: each waits for the one before (with one for every
    // wave and step 48 rows of 50007 took 16 us here)
    if (s_listed == 0) return;
    if (tid == 0) s_first = atomicAdd(&state->listed, s_listed);
    __syncthreads();
    for (unsigned i = tid; i < s_listed && s_first + i < LIST; i += ST) reinterpret_cast<u64*>(ws + WS_LIST)[s_first + i] = s_list[i];
}

// The token of a row: a workgroup each.
template <int DT>
__global__ __launch_bounds__(ST) void k_sample_pick(SampleArgs a) {
    __shared__ u64 s_list[LIST];
    __shared__ u64 scan[ST / WAVE];
    __shared__ u64 s_mass[MOST_BLOCKS];
    __shared__ unsigned s_kept[MOST_BLOCKS];
    __shared__ Top s_top;
    __shared__ u64 s_sum;
    __shared__ unsigned s_n;
    const int row = blockIdx.x, tid = threadIdx.x;
    const uint8_t* l = a.logits + row * a.stride * (DT == F16 ? 2 : 4);
    const uint8_t* ws = a.ws + row * a.row_bytes;
    const RowState state = *reinterpret_cast<const RowState*>(ws + WS_STATE);
    __shared__ double s_exp[32];
    Rule rule = rule_of(a, row, s_exp);
    const Top t = row_top(a, ws, &s_top);
    if (t.most == 0 || rule.greedy) {
        if (tid == 0) {
            a.token[row] = t.most ? t.at : -1;
            if (a.prob) a.prob[row] = t.most ? 1.0f : 0.0f;
            if (a.kept) a.kept[row] = t.most ? 1 : 0;
        }
        return;
    }
    rule.top = key_logit(t.most);
    if (rule.top_k >= t.count) rule.top_k = 0;
    const bool by_count = rule.top_k != 0, by_mass = rule.top_p < 1.0;
    const Binning bin(rule, t);
    const int k_bin = state.k_bin;
    const u64 k_before = (u64)state.k_before, mass_lo = state.mass_lo, p_before = state.p_before;
    const unsigned listed = by_count || by_mass ? state.listed : 0;
    if (listed > LIST) {
        whole_row<DT>(a, row, rule, s_list, scan);
        return;
    }
    for (int b = tid; b < a.blocks; b += ST) {
        s_mass[b] = reinterpret_cast<const u64*>(ws + WS_BLOCK_MASS)[b];
        s_kept[b] = reinterpret_cast<const unsigned*>(ws + WS_BLOCK_KEPT)[b];
    }
    // the list, largest first: short ones by counting the larger ones of each, long ones by a bitonic network
    int size = WAVE;
    while (size < (int)listed) size *= 2;
    for (int i = tid; i < size; i += ST)
        s_list[i] = i < (int)listed ? reinterpret_cast<const u64*>(ws + WS_LIST)[i] : 0ull;
    __syncthreads();
    if (listed <= ST) {
        const u64 mine = tid < (int)listed ? s_list[tid] : 0;
        int rank = 0;
#pragma unroll 8
        for (int i = 0; i < (int)listed; ++i) rank += s_list[i] > mine;
        __syncthreads();
        if (tid < (int)listed) s_list[rank] = mine;
        __syncthreads();
    } else {
        for (int run = 2; run <= size; run *= 2)
            for (int step = run / 2; step > 0; step /= 2) {
                for (int i = tid; i < size / 2; i += ST) {
                    const int x = 2 * i - (i & (step - 1)), y = x + step;
                    const u64 p = s_list[x], q = s_list[y];
                    if ((p < q) == ((x & run) == 0)) s_list[x] = q, s_list[y] = p;
                }
                __syncthreads();
            }
    }

    // How many of the list are kept: a prefix.  Its tokens of k_bin are the last; top-k keeps top_k - k_before of them.
    unsigned last_key = 1, last_at = 0xffffffffu;        // the last token kept
    if (listed) {
        constexpr int PER = LIST / ST;
        u64 w[PER], own = 0, own_k = 0, all, in_k;
        int of_k = 0;
        const int per = (size + ST - 1) / ST;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int i = tid * per + e;
            w[e] = 0;
            if (e < per && i < (int)listed) {
                const float x = key_logit((unsigned)(s_list[i] >> 32));
                w[e] = fixed(rule.weight(x));
                of_k += by_count && bin.of(x) == k_bin;
            }
        }
        // tokens of the list before those of k_bin, and how many of the list top-k leaves
        u64 n_k;
        before_and_total((u64)of_k, scan, n_k);
        const int begin_k = (int)listed - (int)n_k;
        const int by_k = by_count ? begin_k + (int)((u64)rule.top_k - k_before) : (int)listed;
        int keep = by_k;
        if (by_mass) {
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const int i = tid * per + e;
                if (e >= per || i >= by_k) w[e] = 0;
                own += w[e];
                if (i >= begin_k) own_k += w[e];
            }
            before_and_total(own_k, scan, in_k);
            const u64 before = p_before + before_and_total(own, scan, all);
            const double p = ceil(rule.top_p * (double)(mass_lo + in_k));
            const u64 want = p > 1.0 ? (u64)p : 1;
            // (past p_hi there are tokens that the list leaves out, but the sum has reached `want` before)
            u64 run = before;
            int n = 0;
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const int i = tid * per + e;
                if (e < per && i < by_k && run < want) ++n;
                run += w[e];
            }
            u64 total_n;
            before_and_total((u64)n, scan, total_n);
            keep = (int)total_n;
        }
        const u64 last = s_list[max(keep, 1) - 1];
        last_key = (unsigned)(last >> 32), last_at = ~(unsigned)last;
        for (int i = tid; i < keep; i += ST) {
            const double x = rule.weight(key_logit((unsigned)(s_list[i] >> 32)));
            const int b = (int)(~(unsigned)s_list[i]) / BLOCK;
            if (x >= rule.min_p) atomicAdd(&s_mass[b], fixed(x)), atomicAdd(&s_kept[b], 1u);
        }
        __syncthreads();
    } else {
        __syncthreads();
    }

    // the block that the random number falls into
    u64 total, kept;
    const u64 mine = tid < a.blocks ? s_mass[tid] : 0;
    const u64 before = before_and_total(mine, scan, total);
    before_and_total(tid < a.blocks ? (u64)s_kept[tid] : 0ull, scan, kept);
    const float u = a.u[row];
    u64 target = u > 0.0f ? (u64)((double)u * (double)total) : 0;
    if (u >= 1.0f || target >= total) target = total - 1;
    if (tid == 0 && a.kept) a.kept[row] = (int)kept;
    if (before <= target && target < before + mine) s_n = tid, s_sum = before;
    __syncthreads();
    // and the token in it: every thread has a run of eight
    const int from = (int)s_n * BLOCK + tid * EACH;
    float v[EACH];
    load_logits<DT>(l, from, a.vocab, v);
    u64 w[EACH], sum = 0, in_block;
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        const unsigned key = order_key(v[e]);
        w[e] = 0;
        if (key > last_key || (key == last_key && (unsigned)(from + e) <= last_at)) {
            const double x = rule.weight(v[e]);
            w[e] = x >= rule.min_p ? fixed(x) : 0;
        }
        sum += w[e];
    }
    u64 at = s_sum + before_and_total(sum, scan, in_block);
    if (target < at || target >= at + sum) return;
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        if (target >= at && target < at + w[e]) {
            a.token[row] = from + e;
            if (a.prob) a.prob[row] = (float)((double)w[e] / (double)total);
        }
        at += w[e];
    }
}

size_t sample_bytes(int rows, int) { return (size_t)rows * WS_ROW; }

// Chunks of a row so that some 512 workgroups have work, of 4096 logits at least.
void chunks_of(SampleArgs& a) {
    const int want = std::max(1, 512 / a.rows);
    a.chunk = std::max(1, (int)(((int64_t)a.vocab + (int64_t)want * BLOCK - 1) / ((int64_t)want * BLOCK))) * BLOCK;
    a.chunks = (a.vocab + a.chunk - 1) / a.chunk;
    a.blocks = (a.vocab + BLOCK - 1) / BLOCK;
}

template <int DT>
pi_status sample(const SampleArgs& a, hipStream_t s) {
    const dim3 grid(a.chunks, a.rows), block(ST);
    TRY(launch(PI_K_SAMPLE, k_sample_top<DT>, grid, block, 0, s, a));
    TRY(launch(PI_K_SAMPLE, k_sample_count<DT>, grid, block, 0, s, a));
    if (a.top_k || a.top_p) TRY(launch(PI_K_SAMPLE, k_sample_list<DT>, grid, block, 0, s, a));
    return launch(PI_K_SAMPLE, k_sample_pick<DT>, dim3(a.rows), block, 0, s, a);
}

}  // namespace

extern "C" {

size_t pi_sample_workspace_bytes(int32_t rows, int32_t vocab) {
    if (rows < 0 || rows > 65535 || vocab < 1 || vocab > (1 << 20)) return 0;
    return sample_bytes(rows, vocab);
}

pi_status pi_sample(const void* logits, int32_t rows, int32_t vocab, int64_t row_stride, int32_t dtype,
                    const pi_sample_rule* rule, const float* u, int32_t* token, float* prob, int32_t* kept, void* ws,
                    size_t ws_bytes, void* stream) {
    CHECK(rule, PI_ERR_ARG, "NULL rule");
    CHECK(rows >= 0 && rows <= 65535 && vocab >= 1 && vocab <= (1 << 20), PI_ERR_SHAPE,
          "sample: rows must be in 0..65535 and vocab in 1..2^20");
    TRY(check_elem_dtype(dtype, "logits"));
    if (rows == 0) return PI_OK;
    CHECK(logits && u && token, PI_ERR_ARG, "sample: logits, u and token are required");
    CHECK(aligned(logits, dtype_size(dtype)), PI_ERR_ALIGN, "logits must be aligned to its elements");
    CHECK(row_stride >= 0 && row_stride < ((int64_t)1 << 40), PI_ERR_SHAPE, "logits: row_stride must be in 0..2^40");
    CHECK(aligned(u, 4) && aligned(token, 4) && aligned(prob, 4) && aligned(kept, 4) && aligned(rule->temperature, 4) &&
              aligned(rule->top_k, 4) && aligned(rule->top_p, 4) && aligned(rule->min_p, 4),
          PI_ERR_ALIGN, "sample: lists must be 4-byte aligned");
    CHECK(ws && ws_bytes >= sample_bytes(rows, vocab), PI_ERR_WORKSPACE, "sample: workspace of %zu bytes, %zu needed", ws_bytes,
          sample_bytes(rows, vocab));
    CHECK(aligned(ws, 256), PI_ERR_ALIGN, "sample: workspace must be 256-byte aligned");
    const int64_t list = (int64_t)rows * 4, span = ((rows - 1) * row_stride + vocab) * dtype_size(dtype);
    const void* outs[] = {token, prob, kept};
    const void* ins[] = {u, rule->temperature, rule->top_k, rule->top_p, rule->min_p};
    for (int i = 0; i < 3; ++i) {
        bool free = apart(outs[i], list, logits, span) && apart(outs[i], list, ws, sample_bytes(rows, vocab)) &&
                    apart(outs[i], list, outs[(i + 1) % 3], list);
        for (const void* in : ins) free = free && apart(outs[i], list, in, list);
        CHECK(free, PI_ERR_ARG, "sample: token, prob and kept may overlap neither each other nor what the call reads");
    }
    SampleArgs a{(const uint8_t*)logits, row_stride, rule->temperature, rule->top_k, rule->top_p, rule->min_p, u, token, prob,
                 kept, rows, vocab, 0, 0, 0, (uint8_t*)ws, WS_ROW};
    chunks_of(a);
    return dtype == PI_F16 ? sample<F16>(a, (hipStream_t)stream) : sample<F32>(a, (hipStream_t)stream);
}

}  // extern "C"
