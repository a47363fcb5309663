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

// exp for z <= 0 by a table of 2^(j/128) (Tang, ACM TOMS 15(2), 1989): z = (128 m + j) ln 2 / 128 + r with |r| <= ln 2 / 256,
// exp(z) = 2^m 2^(j/128) exp(r), exp(r) by its series to r^4 (the next term is 2^-49).  Weights are needed to 2^-44; the
// library's function takes three times the operations, and a row's distribution hundreds of thousands of them.
constexpr double LN2 = 0.693147180559945309417;
constexpr int EXPS = 128;

// the table, by the whole workgroup; a barrier follows before the first use
__device__ __forceinline__ void fill_exps(double* lds) {
    if (threadIdx.x < EXPS) lds[threadIdx.x] = exp2((double)threadIdx.x / EXPS);
}
__device__ __forceinline__ double exp_by(const double* table, double z) {
    z = fmax(z, -110.0);                 // (below the least float32, which min-p may be)
    // the nearest integer by the addition of 1.5 2^52, in whose lowest bits it then is
    const double t = fma(z, EXPS / LN2, 0x1.8p52), n = t - 0x1.8p52;
    const int i = (int)(unsigned)__builtin_bit_cast(uint64_t, t);
    const double r = fma(n, -LN2 / EXPS, z);           // (ln 2's own rounding: |z| 2^-54, below 2^-47)
    double p = fma(r, 1.0 / 24, 1.0 / 6);
    p = fma(r, p, 0.5);
    p = fma(r, p, 1.0);
    p = fma(r, p, 1.0);
    // times 2^(i / 128): the product is in 1 .. 2 and the result no smaller than 2^-159
    const uint64_t b = __builtin_bit_cast(uint64_t, table[i & (EXPS - 1)] * p);
    return __builtin_bit_cast(double, (uint64_t)((unsigned)(b >> 32) + ((unsigned)(i >> 7) << 20)) << 32 | (unsigned)b);
}

// What the rules of a row come to.
struct Rule {
    double inv_t, min_p, top_p;          // min_p 0 and top_p 1: none
    float top;                           // the largest logit
    int top_k;                           // 0: none
    bool greedy;                         // the first token alone is kept

    const double* table;                 // of exp_by

    // exp((l - max) / T) of a logit that may be kept
    __device__ __forceinline__ double weight(float l) const {
        if (top == INFINITY) return l == top ? 1.0 : 0.0;
        return exp_by(table, ((double)l - (double)top) * inv_t);
    }
};

// the nearest integer to w 2^43, w in 0 .. 1: the lowest bits of its sum with 2^52
__device__ __forceinline__ uint64_t fixed(double w) {
    return __builtin_bit_cast(uint64_t, fma(w, (double)(1ull << FRACTION), 0x1p52)) & ((1ull << 52) - 1);
}

// (table: EXPS numbers in LDS, filled here; a barrier follows)
__device__ __forceinline__ Rule rule_of(const SampleArgs& a, int row, double* table) {
    Rule r;
    fill_exps(table);
    r.table = table;
    const float t = a.temperature ? a.temperature[row] : 1.0f;
    const float p = a.top_p ? a.top_p[row] : 1.0f, m = a.min_p ? a.min_p[row] : 0.0f;
    r.greedy = !(t > 0.0f) || m > 1.0f;  // (no weight reaches a min-p above 1)
    r.inv_t = r.greedy ? 1.0 : 1.0 / (double)t;
    r.top_k = a.top_k ? max(a.top_k[row], 0) : 0;
    r.top_p = p < 1.0f ? (double)p : 1.0;
    r.min_p = m > 0.0f ? (double)m : 0.0;
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

// The same of two values, between the same two barriers (lds: 2 ST / WAVE).
__device__ __forceinline__ void before_and_total(u64 v, u64 v2, u64* lds, u64& before, u64& before2, u64& total, u64& total2) {
    const u64 incl = wave_scan(v), incl2 = wave_scan(v2);
    __syncthreads();
    if (threadIdx.x % WAVE == WAVE - 1) lds[threadIdx.x / WAVE] = incl, lds[ST / WAVE + threadIdx.x / WAVE] = incl2;
    __syncthreads();
    total = total2 = 0;
    before = incl - v, before2 = incl2 - v2;
#pragma unroll
    for (int w = 0; w < ST / WAVE; ++w) {
        const u64 sum = lds[w], sum2 = lds[ST / WAVE + w];
        if (w < (int)threadIdx.x / WAVE) before += sum, before2 += sum2;
        total += sum, total2 += sum2;
    }
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
//   k_sample_top     the largest and smallest logit of the chunk                                              8.2   5.7   3.6
//   k_sample_count   with the row's largest known: the chunk's part of a histogram of the distance to it
//                    (counts for top-k, sums of weights for top-p); without either rule the sum of its
//                    weights                                                                                 17.5   9.7   5.2
//   k_sample_list    from the histogram the bins in which the border of top-k and of top-p can lie: sums
//                    over the tokens above them, and a list of the tokens in them (left out where no row
//                    has either rule)                                                                        17.8  13.2   5.8
//   k_sample_pick    a workgroup to each row: sorts the list, finds the border and the token                 12.7   9.8   7.3
// The whole call: 55.3, 36.4 and 21.5 us.  A dependent launch costs some 4 us here; what is left are the chains of sums in
// each and weights in 64 bits (6 of k_sample_count's 17.5), neither bytes nor atomics.  (A row's last workgroup doing the pick
// in the launch before needs fences between the dies, which write back and drop whole caches: 26 us in place of 13 for one
// row, 108 for 64.)  Short rows take one launch, k_sample_row.
// Sums are integers, so that neither their order nor that of the list matters.  A row whose border bins hold more than
// LIST tokens (equal logits, or a border far below the others) is done by k_sample_pick alone, from the start: 0.5 to
// 0.9 ms for 128000 logits, equal ones or normal ones of a tenth of the temperature beside one of -1e30.

// 8 logits from i on, as they are stored; those past the row's end are -inf
template <int DT>
struct Logits {
    u4 v[DT == F16 ? 1 : 2];
    __device__ __forceinline__ void load(const uint8_t* row, int i, int vocab) {
        if (i + EACH <= vocab) {
            __builtin_memcpy(v, row + (int64_t)i * (DT == F16 ? 2 : 4), sizeof(v));
        } else if constexpr (DT == F16) {
            h8 t;
#pragma unroll
            for (int e = 0; e < EACH; ++e) t[e] = i + e < vocab ? reinterpret_cast<const _Float16*>(row)[i + e] : (_Float16)-INFINITY;
            v[0] = __builtin_bit_cast(u4, t);
        } else {
#pragma unroll
            for (int e = 0; e < EACH; ++e) v[e / 4][e % 4] = __builtin_bit_cast(unsigned, i + e < vocab ? logit<DT>(row, i + e) : -INFINITY);
        }
    }
    __device__ __forceinline__ float operator[](int e) const {
        if constexpr (DT == F32) return bits_f(v[e / 4][e % 4]);
        return e % 2 ? half_hi(v[0][e / 2]) : half_lo(v[0][e / 2]);
    }
};

// A workgroup's logits, BLOCK by BLOCK: STEPS of them are loaded at once, the first before all else that a kernel does, and
// the next while these are worked on (one after the other each took 2 us: 64 x 151003, five to a chunk).
template <int DT>
struct Chunk {
    static constexpr int STEPS = DT == F16 ? 4 : 2;      // (registers for two workgroups on a unit)
    const uint8_t* row;
    int from, to, vocab;
    Logits<DT> next[STEPS];
    __device__ __forceinline__ Chunk(const SampleArgs& a)
        : row(a.logits + blockIdx.y * a.stride * (DT == F16 ? 2 : 4)), from(blockIdx.x * a.chunk),
          to(min(from + a.chunk, a.vocab)), vocab(a.vocab) {}
    __device__ __forceinline__ void load(int base) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            if (base + s * BLOCK < to) next[s].load(row, base + s * BLOCK + threadIdx.x * EACH, vocab);
    }
    // f(logits, index of the thread's first, number of the block in the chunk)
    template <class F>
    __device__ __forceinline__ void each(F f) {
#pragma unroll 1
        for (int base = from, block = 0; base < to; base += STEPS * BLOCK, block += STEPS) {
            Logits<DT> now[STEPS];
#pragma unroll
            for (int s = 0; s < STEPS; ++s) now[s] = next[s];
            load(base + STEPS * BLOCK);
#pragma unroll
            for (int s = 0; s < STEPS; ++s)
                if (base + s * BLOCK < to) f(now[s], base + s * BLOCK + (int)threadIdx.x * EACH, block + s);
        }
    }
};

template <int DT, bool ALONE>
__device__ __forceinline__ void top_stage(const SampleArgs& a) {
    __shared__ unsigned s_most[ST / WAVE], s_least[ST / WAVE], s_at[ST / WAVE];
    __shared__ int s_count[ST / WAVE];
    const int row = blockIdx.y, tid = threadIdx.x, wave = tid / WAVE;
    Chunk<DT> chunk(a);
    chunk.load(chunk.from);
    uint8_t* ws = a.ws + row * a.row_bytes;
    // what the later launches add to
    if constexpr (!ALONE) {
        for (int b = blockIdx.x * ST + tid; b < BINS; b += gridDim.x * ST) {
            reinterpret_cast<u64*>(ws + WS_MASS)[b] = 0;
            reinterpret_cast<unsigned*>(ws + WS_COUNT)[b] = 0;
        }
    }
    if (blockIdx.x == 0 && tid == 0) reinterpret_cast<RowState*>(ws + WS_STATE)->listed = 0;

    // the largest, smallest and number of those that may be kept; `best` holds the largest first
    float most = -INFINITY, least = INFINITY;
    int count = 0, best_at = 0;                // (count: of the whole wave)
    Logits<DT> best{};
    chunk.each([&](const Logits<DT>& v, int i, int) __attribute__((always_inline)) {
        float m = -INFINITY;
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const bool may = v[e] > -INFINITY;
            count += __popcll(__ballot(may));
            m = fmaxf(m, v[e]);                // (the other one of a NaN)
            least = fminf(least, may ? v[e] : INFINITY);
        }
        if (m > most) most = m, best = v, best_at = i;
    });
    unsigned at = 0;
#pragma unroll
    for (int e = EACH - 1; e >= 0; --e)
        if (best[e] == most) at = best_at + e;
    const unsigned key = order_key(most);
    unsigned low = least < INFINITY ? ~order_key(least) : 0u;
    const unsigned top = wave_max(key);
    // the lowest index of the largest (a thread has met its own lowest first)
    const unsigned first = ~wave_max(key == top ? ~at : 0u);
    // the smallest as the largest of the complements
    low = wave_max(low);
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

// The row's largest and smallest key, the largest's lowest index, and the tokens that may be kept, from its chunks' (by each
// wave for itself; first: what load_top gave).
__device__ __forceinline__ Top load_top(const SampleArgs& a, const uint8_t* ws, int c) {
    return c < a.chunks ? reinterpret_cast<const Top*>(ws + WS_TOPS)[c] : Top{0, ~0u, 0, 0};
}
__device__ __forceinline__ Top row_top(const SampleArgs& a, const uint8_t* ws, Top first) {
    Top t = first;
    for (int c = threadIdx.x % WAVE + WAVE; c < a.chunks; c += WAVE) {
        const Top o = load_top(a, ws, c);
        if (o.most > t.most) t.most = o.most, t.at = o.at;
        t.least = min(t.least, o.least);
        t.count += o.count;
    }
    const unsigned top = wave_max(t.most);
    t.at = (int)~wave_max(t.most == top ? ~(unsigned)t.at : 0u);
    t.least = ~wave_max(~t.least);
    t.count = (int)wave_sum((u64)t.count);
    t.most = top;
    return t;
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

// adds what the wave's threads have to a block's sum of weights and count
__device__ __forceinline__ void add_block(u64 sum, unsigned n, u64* mass, unsigned* count) {
    if (n == 0) return;
    sum = wave_sum(sum);
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

template <int DT, bool ALONE>
__device__ __forceinline__ void count_stage(const SampleArgs& a) {
    __shared__ u64 s_mass[BINS];
    __shared__ unsigned s_count[BINS];
    __shared__ double s_exp[EXPS];
    const int row = blockIdx.y, tid = threadIdx.x;
    uint8_t* ws = a.ws + row * a.row_bytes;
    const Top first = load_top(a, ws, tid % WAVE);
    Chunk<DT> chunk(a);
    chunk.load(chunk.from);
    Rule rule = rule_of(a, row, s_exp);
    for (int b = tid; b < BINS; b += ST) s_mass[b] = 0, s_count[b] = 0;
    const Top t = row_top(a, ws, first);
    if (t.most == 0 || rule.greedy) return;
    rule.top = key_logit(t.most);
    if (rule.top_k >= t.count) rule.top_k = 0;
    const bool by_count = rule.top_k != 0, by_mass = rule.top_p < 1.0;
    __syncthreads();
    if (!by_count && !by_mass) {
        chunk.each([&](const Logits<DT>& v, int, int block) __attribute__((always_inline)) {
            u64 sum = 0;
            unsigned n = 0;
#pragma unroll
            for (int e = 0; e < EACH; ++e) {
                const double w = rule.weight(v[e]);
                const bool keep = v[e] > -INFINITY && w >= rule.min_p;
                sum += keep ? fixed(w) : 0;
                n += __popcll(__ballot(keep));
            }
            add_block(sum, n, &s_mass[block], &s_count[block]);
        });
        __syncthreads();
        store_blocks(a, ws, s_mass, s_count);
        return;
    }
    const Binning bin(rule, t);
    chunk.each([&](const Logits<DT>& v, int, int) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            if (!(v[e] > -INFINITY)) continue;
            const int b = bin.of(v[e]);
            if (by_count) atomicAdd(&s_count[b], 1u);
            if (by_mass) {
                const u64 w = fixed(rule.weight(v[e]));
                if (w) atomicAdd(&s_mass[b], w);
            }
        }
    });
    __syncthreads();
    for (int b = tid; b < BINS; b += ST) {
        if constexpr (ALONE) {
            reinterpret_cast<unsigned*>(ws + WS_COUNT)[b] = s_count[b];
            reinterpret_cast<u64*>(ws + WS_MASS)[b] = s_mass[b];
        } else {
            if (s_count[b]) atomicAdd(reinterpret_cast<unsigned*>(ws + WS_COUNT) + b, s_count[b]);
            if (s_mass[b]) atomicAdd(reinterpret_cast<u64*>(ws + WS_MASS) + b, s_mass[b]);
        }
    }
}

constexpr int OWN = BINS / ST;           // bins of a thread

template <int DT, bool ALONE>
__device__ __forceinline__ void list_stage(const SampleArgs& a) {
    __shared__ u64 s_list[LIST];
    __shared__ unsigned s_listed, s_first;
    __shared__ u64 scan[2 * ST / WAVE];
    __shared__ u64 s_mass[MOST_BLOCKS];
    __shared__ unsigned s_kept[MOST_BLOCKS];
    __shared__ int s_bin[3];
    __shared__ u64 s_at[4];
    __shared__ double s_exp[EXPS];
    const int row = blockIdx.y, tid = threadIdx.x;
    uint8_t* ws = a.ws + row * a.row_bytes;
    RowState* state = reinterpret_cast<RowState*>(ws + WS_STATE);
    const Top first = load_top(a, ws, tid % WAVE);
    u64 n[OWN], m[OWN], own_n = 0, own_m = 0, all_n, all_m;
#pragma unroll
    for (int e = 0; e < OWN; ++e) {
        n[e] = reinterpret_cast<const unsigned*>(ws + WS_COUNT)[tid * OWN + e];
        m[e] = reinterpret_cast<const u64*>(ws + WS_MASS)[tid * OWN + e];
    }
    Chunk<DT> chunk(a);
    chunk.load(chunk.from);
    Rule rule = rule_of(a, row, s_exp);
    if (rule.greedy || (rule.top_k == 0 && rule.top_p >= 1.0)) return;
    const Top t = row_top(a, ws, first);
    rule.top = key_logit(t.most);
    if (rule.top_k >= t.count) rule.top_k = 0;
    const bool by_count = rule.top_k != 0, by_mass = rule.top_p < 1.0;
    if (t.most == 0 || !(by_count || by_mass)) return;
    const Binning bin(rule, t);

    // Bins: k_bin holds the border of top-k; the sum that top-p is a part of lies between those without and with it, so the
    // border of top-p lies in p_lo .. p_hi.  s_bin: these three; s_at: tokens before k_bin, weights before it, with it, and
    // before p_lo.
#pragma unroll
    for (int e = 0; e < OWN; ++e) own_n += n[e], own_m += m[e];
    u64 before_n, before_m;
    if (tid < 3) s_bin[tid] = BINS;
    if (tid == 0) s_listed = 0;
    for (int b = tid; b < MOST_BLOCKS; b += ST) s_mass[b] = 0, s_kept[b] = 0;
    before_and_total(own_n, own_m, scan, before_n, before_m, all_n, all_m);
    // the lowest bin with which a sum reaches `want`; f(weights and tokens before it, with it)
    auto find_bin = [&](u64 want, bool tokens, int which, auto f) __attribute__((always_inline)) {
        u64 c = before_n, w = before_m;
#pragma unroll
        for (int e = 0; e < OWN; ++e) {
            const u64 sum = tokens ? c : w, with = sum + (tokens ? n[e] : m[e]);
            if (sum < want && with >= want) s_bin[which] = tid * OWN + e, f(c, w, w + m[e]);
            c += n[e], w += m[e];
        }
    };
    u64 k_before = 0, mass_lo = all_m, mass_hi = all_m;
    int k_bin = BINS;
    if (by_count) {
        find_bin((u64)rule.top_k, true, 0, [&](u64 c, u64 w, u64 with) { s_at[0] = c, s_at[1] = w, s_at[2] = with; });
        __syncthreads();
        k_bin = s_bin[0];                                // (found: there are more tokens than top_k)
        k_before = s_at[0], mass_lo = s_at[1], mass_hi = s_at[2];
    }
    int p_lo = BINS, p_hi = BINS;
    u64 p_before = 0;
    if (by_mass) {
        const double lo = ceil(rule.top_p * (double)mass_lo), hi = ceil(rule.top_p * (double)mass_hi);
        find_bin(lo > 1.0 ? (u64)lo : 1, false, 1, [&](u64, u64 w, u64) { s_at[3] = w; });
        find_bin(hi > 1.0 ? (u64)hi : 1, false, 2, [&](u64, u64, u64) {});
        __syncthreads();
        p_lo = s_bin[1], p_hi = s_bin[2];
        p_before = p_lo < BINS ? s_at[3] : 0;
    }
    if (blockIdx.x == 0 && tid == 0) state->mass_lo = mass_lo, state->p_before = p_before, state->k_bin = k_bin, state->k_before = (int)k_before;
    const int border = by_mass ? p_lo : k_bin;           // bins before it are kept for certain

    chunk.each([&](const Logits<DT>& v, int i, int block) __attribute__((always_inline)) {
        u64 sum = 0;
        unsigned kept = 0, in_list = 0;            // (a bit for each)
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const bool may = v[e] > -INFINITY;
            const int b = bin.of(v[e]);
            bool keep = may && b < border;
            if (__any(keep)) {
                const double w = rule.weight(v[e]);
                keep = keep && w >= rule.min_p;
                sum += keep ? fixed(w) : 0;
                kept += __popcll(__ballot(keep));
            }
            if (may && b >= border && (b == k_bin || (by_mass && b <= p_hi))) in_list |= 1u << e;
        }
        if (__any(in_list != 0)) {
            const int mine = __popc(in_list), incl = wave_incl_scan(mine);
            unsigned at = 0;
            if (tid % WAVE == WAVE - 1) at = atomicAdd(&s_listed, (unsigned)incl);
            at = __shfl(at, WAVE - 1) + incl - mine;
#pragma unroll
            for (int e = 0; e < EACH; ++e) {
                if (!(in_list >> e & 1)) continue;
                if (at < LIST) s_list[at] = (u64)order_key(v[e]) << 32 | ~(unsigned)(i + e);
                ++at;
            }
        }
        add_block(sum, kept, &s_mass[block], &s_kept[block]);
    });
    __syncthreads();
    store_blocks(a, ws, s_mass, s_kept);
    // one addition to the row's count for all of the workgroup's tokens: each waits for the one before (with one for every
    // wave and step 48 rows of 50007 took 16 us here)
    if (s_listed == 0) return;
    if (tid == 0) {
        if constexpr (ALONE)
            s_first = 0, state->listed = s_listed;
        else
            s_first = atomicAdd(&state->listed, s_listed);
    }
    __syncthreads();
    for (unsigned i = tid; i < s_listed && s_first + i < LIST; i += ST) reinterpret_cast<u64*>(ws + WS_LIST)[s_first + i] = s_list[i];
}

// The token of a row: a workgroup each.
template <int DT>
__device__ __forceinline__ void pick_stage(const SampleArgs& a, int row) {
    __shared__ __align__(16) u64 s_list[LIST];
    __shared__ u64 scan[2 * ST / WAVE];
    __shared__ u64 s_mass[MOST_BLOCKS];
    __shared__ unsigned s_kept[MOST_BLOCKS];
    __shared__ u64 s_sum;
    __shared__ unsigned s_n;
    __shared__ double s_exp[EXPS];
    const int tid = threadIdx.x;
    const uint8_t* l = a.logits + row * a.stride * (DT == F16 ? 2 : 4);
    const uint8_t* ws = a.ws + row * a.row_bytes;
    const Top first = load_top(a, ws, tid % WAVE);
    const RowState state = *reinterpret_cast<const RowState*>(ws + WS_STATE);
    // (whatever there is of it)
    const u64 in_list = reinterpret_cast<const u64*>(ws + WS_LIST)[tid];
    if (tid < a.blocks) {
        s_mass[tid] = reinterpret_cast<const u64*>(ws + WS_BLOCK_MASS)[tid];
        s_kept[tid] = reinterpret_cast<const unsigned*>(ws + WS_BLOCK_KEPT)[tid];
    }
    Rule rule = rule_of(a, row, s_exp);
    const Top t = row_top(a, ws, first);
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
        __syncthreads();
        whole_row<DT>(a, row, rule, s_list, scan);
        return;
    }
    // the list, largest first: short ones by counting the larger ones of each, long ones by a bitonic network
    int size = WAVE;
    while (size < (int)listed) size *= 2;
    for (int i = tid; i < size; i += ST)
        s_list[i] = i >= (int)listed ? 0ull : i < ST ? in_list : reinterpret_cast<const u64*>(ws + WS_LIST)[i];
    __syncthreads();
    if (listed <= ST) {
        const u64 mine = tid < (int)listed ? s_list[tid] : 0;
        int rank = 0;
        // (past the list are zeros)
#pragma unroll 4
        for (int i = 0; i < (int)listed; i += 2) {
            const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&s_list[i]);
            rank += (o.x > mine) + (o.y > mine);
        }
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
            u64 before, before_k;
            before_and_total(own, own_k, scan, before, before_k, all, in_k);
            before += p_before;
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
    u64 total, kept, before, kept_before;
    const u64 mine = tid < a.blocks ? s_mass[tid] : 0;
    before_and_total(mine, tid < a.blocks ? (u64)s_kept[tid] : 0ull, scan, before, kept_before, total, kept);
    const float u = a.u[row];
    u64 target = u > 0.0f ? (u64)((double)u * (double)total) : 0;
    if (u >= 1.0f || target >= total) target = total - 1;
    if (tid == 0 && a.kept) a.kept[row] = (int)kept;
    if (before <= target && target < before + mine) s_n = tid, s_sum = before;
    __syncthreads();
    // and the token in it: every thread has a run of eight
    const int from = (int)s_n * BLOCK + tid * EACH;
    Logits<DT> v;
    v.load(l, from, a.vocab);
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

template <int DT>
__global__ __launch_bounds__(ST) void k_sample_top(SampleArgs a) { top_stage<DT, false>(a); }
template <int DT>
__global__ __launch_bounds__(ST) void k_sample_count(SampleArgs a) { count_stage<DT, false>(a); }
template <int DT>
__global__ __launch_bounds__(ST) void k_sample_list(SampleArgs a) { list_stage<DT, false>(a); }
template <int DT>
__global__ __launch_bounds__(ST) void k_sample_pick(SampleArgs a) { pick_stage<DT>(a, blockIdx.x); }

// All of it for a row of one chunk, by one workgroup: what the stages leave for each other has one writer.
template <int DT>
__global__ __launch_bounds__(ST) void k_sample_row(SampleArgs a) {
    top_stage<DT, true>(a);
    __syncthreads();
    count_stage<DT, true>(a);
    __syncthreads();
    if (a.top_k || a.top_p) list_stage<DT, true>(a);
    __syncthreads();
    pick_stage<DT>(a, blockIdx.y);
}

size_t sample_bytes(int rows, int) { return (size_t)rows * WS_ROW; }

// Short rows go by one workgroup each, as long as each has a unit of its own (its LDS leaves room for one): launches saved
// against chunks side by side.  us with top-k and with top-p, float32, one launch and four:
//   1 x 1000  15.7 17.2, 19.6 21.3    1 x 8192    15.9 20.8, 18.2 21.3     1 x 16384    19.3 27.1, 18.1 21.3
//   64 x 8192 17.4 21.7, 21.3 24.8    256 x 8192  18.3 23.1, 28.2 33.9     1000 x 8192  68.3 86.7, 52.9 69.1
bool row_alone(const SampleArgs& a) { return a.vocab <= 8192 && a.rows <= 256; }

// Chunks of a row so that some 512 workgroups have work, of 4096 logits at least.
void chunks_of(SampleArgs& a) {
    const int want = row_alone(a) ? 1 : std::max(1, 512 / a.rows);
    a.chunk = std::max(1, (int)(((int64_t)a.vocab + (int64_t)want * BLOCK - 1) / ((int64_t)want * BLOCK))) * BLOCK;
    a.chunks = (a.vocab + a.chunk - 1) / a.chunk;
    a.blocks = (a.vocab + BLOCK - 1) / BLOCK;
}

template <int DT>
pi_status sample(const SampleArgs& a, hipStream_t s) {
    const dim3 grid(a.chunks, a.rows), block(ST);
    if (row_alone(a)) return launch(PI_K_SAMPLE, k_sample_row<DT>, grid, block, 0, s, a);
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
    bool free = apart(ws, sample_bytes(rows, vocab), logits, span);
    for (const void* in : ins) free = free && apart(ws, sample_bytes(rows, vocab), in, list);
    CHECK(free, PI_ERR_ARG, "sample: the workspace overlaps what the call reads");
    SampleArgs a{(const uint8_t*)logits, row_stride, rule->temperature, rule->top_k, rule->top_p, rule->min_p, u, token, prob,
                 kept, rows, vocab, 0, 0, 0, (uint8_t*)ws, WS_ROW};
    chunks_of(a);
    return dtype == PI_F16 ? sample<F16>(a, (hipStream_t)stream) : sample<F32>(a, (hipStream_t)stream);
}

}  // extern "C"
