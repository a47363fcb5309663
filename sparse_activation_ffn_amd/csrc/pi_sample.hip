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

constexpr int ST = 1024;                 // threads of a row's workgroup
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
};

// A logit as an unsigned integer in the same order; 0 for -inf and NaN, which are never kept.  -0 and 0 are equal.
__device__ __forceinline__ unsigned order_key(float l) {
    const unsigned b = __builtin_bit_cast(unsigned, l + 0.0f);
    return l > -INFINITY ? (b >> 31 ? ~b : b | 0x80000000u) : 0u;
}
__device__ __forceinline__ float key_logit(unsigned key) {
    return __builtin_bit_cast(float, key >> 31 ? key & 0x7fffffffu : ~key);
}

// What the rules of a row come to.
struct Rule {
    double inv_t, min_p, top_p;          // min_p 0 and top_p 1: none
    float top;                           // the largest logit
    int top_k;                           // 0: none
    bool greedy;

    // exp((l - max) / T) of a logit that may be kept
    __device__ __forceinline__ double weight(float l) const {
        return l == top ? 1.0 : top == INFINITY ? 0.0 : exp(((double)l - (double)top) * inv_t);
    }
};

__device__ __forceinline__ uint64_t fixed(double w) { return (uint64_t)(w * (double)(1ull << FRACTION) + 0.5); }

__device__ __forceinline__ Rule rule_of(const SampleArgs& a, int row) {
    Rule r;
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

// Sums of a value over the threads before this one, and over all.
template <typename T>
__device__ T before_and_total(T v, T* lds, T& total) {
    T incl = v;
#pragma unroll
    for (int o = 1; o < WAVE; o *= 2) {
        const T up = __shfl_up(incl, o);
        if ((int)(threadIdx.x % WAVE) >= o) incl += up;
    }
    __syncthreads();
    if (threadIdx.x % WAVE == WAVE - 1) lds[threadIdx.x / WAVE] = incl;
    __syncthreads();
    T base = 0;
    total = 0;
    for (int w = 0; w < ST / WAVE; ++w) {
        if (w < (int)threadIdx.x / WAVE) base += lds[w];
        total += lds[w];
    }
    return base + incl - v;
}

// One workgroup per row.  The border of the kept set, in the order of the keys, is found digit by digit (8 bits, from
// the top): top-k by counts, top-p by sums of weights.
template <int DT>
__global__ __launch_bounds__(ST) void k_sample(SampleArgs a) {
    typedef unsigned long long u64;
    __shared__ u64 mass[256];
    __shared__ int count[256];
    __shared__ u64 scan[ST / WAVE];
    __shared__ unsigned best;
    __shared__ int first;
    __shared__ unsigned s_key;
    __shared__ u64 s_before;
    const int row = blockIdx.x, tid = threadIdx.x;
    const uint8_t* l = a.logits + row * a.stride * (DT == F16 ? 2 : 4);
    Rule rule = rule_of(a, row);

    if (tid == 0) best = 0, first = a.vocab;
    __syncthreads();
    unsigned mine = 0;
    int at = a.vocab;
    for (int i = tid; i < a.vocab; i += ST) {
        const unsigned key = order_key(logit<DT>(l, i));
        if (key > mine) mine = key, at = i;
    }
    atomicMax(&best, mine);
    __syncthreads();
    if (mine == best && mine) atomicMin(&first, at);
    __syncthreads();
    if (best == 0 || rule.greedy) {
        if (tid == 0) {
            a.token[row] = best ? first : -1;
            if (a.prob) a.prob[row] = best ? 1.0f : 0.0f;
            if (a.kept) a.kept[row] = best ? 1 : 0;
        }
        return;
    }
    rule.top = key_logit(best);

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
            for (int b = tid; b < 256; b += ST) mass[b] = 0, count[b] = 0;
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
    const int64_t equal_before = (int64_t)before_and_total<u64>(equal, scan, total);
    u64 sum = 0, n = 0;
    int64_t rank = equal_before;
    for (int i = lo; i < hi; ++i) {
        const float x = logit<DT>(l, i);
        const unsigned k = order_key(x);
        if (k < key || (k == key && rank++ >= ties)) continue;
        const double w = rule.weight(x);
        if (w >= rule.min_p) sum += fixed(w), ++n;
    }
    const u64 before = before_and_total<u64>(sum, scan, total);
    u64 all_kept;
    before_and_total<u64>(n, scan, all_kept);
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

size_t sample_bytes(int, int) { return 256; }

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
    SampleArgs a{(const uint8_t*)logits, row_stride, rule->temperature, rule->top_k, rule->top_p, rule->min_p, u, token, prob,
                 kept, rows, vocab};
    hipStream_t s = (hipStream_t)stream;
    return dtype == PI_F16 ? launch(PI_K_SAMPLE, k_sample<F16>, dim3(rows), dim3(ST), 0, s, a)
                           : launch(PI_K_SAMPLE, k_sample<F32>, dim3(rows), dim3(ST), 0, s, a);
}

}  // extern "C"
