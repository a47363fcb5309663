// pi_norm.hip -- the residual's addition with a root-mean-square norm, and
// microscaled quantisation and its inverse.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "pi.h"
#include "pi_cache.h"
#include "pi_launch.h"
#include "pi_mx.h"

using namespace pi;

namespace {

constexpr int NT = 256;        // threads of a workgroup
constexpr int NONE = -1;       // no delta, no weight, no microscaled output

struct NormArgs {
    const uint8_t* x;
    const uint8_t* delta;
    uint8_t* sum;
    uint8_t* y;
    uint8_t* codes;
    uint8_t* scales;
    const uint8_t* weight;
    int64_t x_ts, x_hs, d_ts, d_hs, s_ts, s_hs, y_ts, y_hs;   // strides in bytes
    double eps;
    int rows, heads, d;
    int ddtype, wdtype, format;                               // or NONE
};

// ---- the norm ----------------------------------------------------------------------
//
// s = x + delta; y = s w / sqrt(mean(s^2) + eps).  Every input and output byte moves once, some ten operations an
// element: the HBM rate bounds it, a launch and two dependent latencies where there are few rows.  So a row stays in
// registers between the sum of its squares and its outputs: 8 elements (a 16-byte load of f16) per thread and chunk, a
// row on 8 to 64 lanes of a wave (heads) or on a workgroup.  The squares are summed in 64 bits: exact products of
// f16, and no overflow for float32.  us: 4099 tokens of 64 heads of 128 in f16, 27.9 (4.8 TB/s); 8191 rows of 8192 in f16
// with an f16 delta, to their sum and MXFP8, 91 (5.2 TB/s); one row of 7168 with a float32 delta, 3.4.

template <int CTRL>
__device__ __forceinline__ double add_dpp(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const unsigned lo = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)b, CTRL, 0xf, 0xf, false);
    const unsigned hi = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)(b >> 32), CTRL, 0xf, 0xf, false);
    return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// the sum over LANES consecutive lanes, in every one of them
template <int LANES>
__device__ __forceinline__ double lanes_sum(double v) {
    v = add_dpp<DPP_QUAD_1032>(v);
    v = add_dpp<DPP_QUAD_2301>(v);
    v = add_dpp<DPP_ROW_HALF_MIRROR>(v);
    if constexpr (LANES >= 16) v = add_dpp<DPP_ROW_MIRROR>(v);
    if constexpr (LANES >= 32) v += __shfl_xor(v, 16);
    if constexpr (LANES >= 64) v += __shfl_xor(v, 32);
    return v;
}

// the sum over a workgroup of N threads
template <int N>
__device__ __forceinline__ double workgroup_sum(double v, double* lds) {
    v = lanes_sum<64>(v);
    if (threadIdx.x % WAVE == 0) lds[threadIdx.x / WAVE] = v;
    __syncthreads();
    double sum = lds[0];
#pragma unroll
    for (int i = 1; i < N / WAVE; ++i) sum += lds[i];
    return sum;
}

template <int XT>
__device__ __forceinline__ float rounded(float v) {
    return XT == F16 ? (float)(_Float16)v : v;
}

__device__ __forceinline__ float element(const uint8_t* p, int dtype, int i) {
    return dtype == F16 ? (float)reinterpret_cast<const _Float16*>(p)[i] : reinterpret_cast<const float*>(p)[i];
}

// y of one element.  f16 times f16 is exact in float32, so with r as a sum of two floats one rounding is left; the other
// forms go through 64 bits.  ODD: the float32 next to y whose last bit is 1, unless y is one: rounded on to fewer bits, it
// gives what y itself would.  That costs twice the operations, so it is for values that may lie half between two codes,
// where the nearest float32 has 19 bits of zeros at its end (which at this distance from y is one in 2^19).
struct Scale {
    double r;
    float hi, lo;
    __device__ explicit Scale(double mean_eps) {
        // the instruction's 24 bits or so, doubled twice
        r = __builtin_amdgcn_rsq(mean_eps);
        if (mean_eps > 0.0 && mean_eps < (double)INFINITY) {
            r = r * fma(-0.5 * mean_eps * r, r, 1.5);
            r = r * fma(-0.5 * mean_eps * r, r, 1.5);
        }
        hi = (float)r, lo = (float)(r - (double)hi);
    }
    template <bool EXACT, bool ODD>
    __device__ __forceinline__ float of(float s, float w) const {
        float y, rest;
        if constexpr (EXACT) {
            const float t = s * w;
            const float low = fabsf(t) < INFINITY ? t * lo : 0.0f;   // (an infinite weight meets lo of either sign)
            y = fmaf(t, hi, low);
            rest = ODD ? fmaf(t, hi, -y) + low : 0.0f;
        } else {
            const double v = (double)s * r * (double)w;
            y = (float)v;
            // (its sign alone: next to a subnormal y the difference is below float32's smallest number)
            const double more = ODD ? v - (double)y : 0.0;
            rest = more < 0.0 ? -1.0f : more > 0.0 ? 1.0f : 0.0f;
        }
        if (ODD && fabsf(y) < INFINITY && rest != 0.0f) {
            unsigned b = __builtin_bit_cast(unsigned, y);
            if ((rest < 0.0f) != (b >> 31 != 0)) --b;      // (towards 0; a y of 0 has the sign of the rest)
            y = __builtin_bit_cast(float, b | 1u);
        }
        return y;
    }
};

__device__ __forceinline__ bool may_be_tie(float y) { return (__builtin_bit_cast(unsigned, y) & 0x7ffffu) == 0; }

// 8 elements as they are stored: float32 takes two pieces of 16 bytes
template <int DT>
struct Raw8 {
    u4 v[DT == F16 ? 1 : 2];
    __device__ __forceinline__ void load(const uint8_t* p) {
        v[0] = ld16(p);
        if constexpr (DT == F32) v[1] = ld16(p + 16);
    }
    __device__ __forceinline__ float get(int e) const {
        if constexpr (DT == F32) return bits_f(v[e / 4][e % 4]);
        return e % 2 ? half_hi(v[0][e / 2]) : half_lo(v[0][e / 2]);
    }
    __device__ __forceinline__ void set(const float* f) { store8<DT, true>(v, f); }
};

// TPR threads to a row, C chunks of 8 elements to a thread, the sum kept as it is stored.  d % 8 == 0 and every row 16-byte
// aligned.  FORMAT: of the microscaled output, or NONE.
template <int XT, int TPR, int C, int FORMAT>
__global__ __launch_bounds__(std::max(NT, TPR)) void k_rms_norm(NormArgs a) {
    constexpr int PER = std::max(NT / TPR, 1);           // rows of a workgroup
    __shared__ double lds[std::max(NT, TPR) / WAVE];
    const int t = threadIdx.x % TPR;
    const int row = blockIdx.x * PER + threadIdx.x / TPR;
    if (PER > 1 && row >= a.rows) return;                // (whole groups of lanes that work together)
    const int token = a.heads == 1 ? row : row / a.heads, head = row - token * a.heads;
    constexpr int ES = XT == F16 ? 2 : 4;
    const uint8_t* x = a.x + token * a.x_ts + head * a.x_hs;
    const uint8_t* delta = a.delta + token * a.d_ts + head * a.d_hs;
    auto load_weight = [&](int at, float* w) __attribute__((always_inline)) {
        if (a.wdtype == F16)
            load8<F16, true>(a.weight + (int64_t)at * 2, w);
        else if (a.wdtype == F32)
            load8<F32, true>(a.weight + (int64_t)at * 4, w);
        else
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = 1.0f;
    };
    Raw8<XT> s[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = (c * TPR + t) * 8;
        if (at < a.d)
            s[c].load(x + (int64_t)at * ES);
        else
            s[c] = Raw8<XT>{};
    }
    // (asked for before the sum, which is a barrier away, where there are registers for it)
    float w[8];
    if (C == 1 && t * 8 < a.d) load_weight(t * 8, w);
    if (a.ddtype != NONE) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = (c * TPR + t) * 8;
            if (at < a.d) {
                float v[8];
                if (a.ddtype == F16)
                    load8<F16, true>(delta + (int64_t)at * 2, v);
                else
                    load8<F32, true>(delta + (int64_t)at * 4, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += s[c].get(e);
                s[c].set(v);
            }
        }
    }
    double squares = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) squares = fma((double)s[c].get(e), (double)s[c].get(e), squares);
    double total;
    if constexpr (TPR <= WAVE)
        total = lanes_sum<TPR>(squares);
    else
        total = workgroup_sum<TPR>(squares, lds);
    // (opaque, so that the elements are kept as they are stored and not as the float32 of the squares)
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < (XT == F16 ? 1 : 2); ++i) asm volatile("" : "+v"(s[c].v[i]));
    const Scale scale(total / a.d + a.eps);
    uint8_t* sum = a.sum + token * a.s_ts + head * a.s_hs;
    uint8_t* y = a.y + token * a.y_ts + head * a.y_hs;
    const bool exact = XT == F16 && a.wdtype != F32;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = (c * TPR + t) * 8;
        if (at >= a.d) continue;
        if (a.sum) {
            reinterpret_cast<u4*>(sum + (int64_t)at * ES)[0] = s[c].v[0];
            if constexpr (XT == F32) reinterpret_cast<u4*>(sum + (int64_t)at * ES)[1] = s[c].v[1];
        }
        if (C > 1) load_weight(at, w);
        float v[8];
        bool tie = false;
        if (exact) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = scale.of<true, false>(s[c].get(e), w[e]);
        } else {
            // (the last bit of a subnormal is 2^-149 wherever it lies, so that fewer zeros end a tie's; f16 times f16 has none)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = scale.of<false, false>(s[c].get(e), w[e]);
                tie |= fabsf(v[e]) < 0x1p-126f;
            }
        }
        if (a.y) store8<XT, true>(y + (int64_t)at * ES, v);
        if constexpr (FORMAT != NONE) {
#pragma unroll
            for (int e = 0; e < 8; ++e) tie |= may_be_tie(v[e]);
            if (__any(tie)) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = exact ? scale.of<true, true>(s[c].get(e), w[e]) : scale.of<false, true>(s[c].get(e), w[e]);
            }
            store_block<FORMAT>(v, (int64_t)row * a.d + at, a.codes, a.scales);
        }
    }
}

// Any size and alignment: a workgroup per row, an element per thread and step, the row read again from the caches.
template <int XT>
__global__ __launch_bounds__(NT) void k_rms_norm_any(NormArgs a) {
    typedef typename std::conditional<XT == F16, _Float16, float>::type T;
    __shared__ double lds[NT / WAVE];
    const int row = blockIdx.x;
    const int token = row / a.heads, head = row - token * a.heads;
    const T* x = reinterpret_cast<const T*>(a.x + token * a.x_ts + head * a.x_hs);
    const uint8_t* delta = a.delta + token * a.d_ts + head * a.d_hs;
    T* sum = reinterpret_cast<T*>(a.sum + token * a.s_ts + head * a.s_hs);
    T* y = reinterpret_cast<T*>(a.y + token * a.y_ts + head * a.y_hs);
    double squares = 0.0;
    for (int i = threadIdx.x; i < a.d; i += NT) {
        float s = (float)x[i];
        if (a.ddtype != NONE) s = rounded<XT>(s + element(delta, a.ddtype, i));
        if (a.sum) sum[i] = (T)s;
        squares = fma((double)s, (double)s, squares);
    }
    const Scale scale(workgroup_sum<NT>(squares, lds) / a.d + a.eps);
    for (int i = threadIdx.x; i < a.d; i += NT) {
        // (a sum may have replaced x or delta; this thread wrote it)
        float s = a.sum ? (float)sum[i] : (float)x[i];
        if (!a.sum && a.ddtype != NONE) s = rounded<XT>(s + element(delta, a.ddtype, i));
        const float w = a.wdtype == NONE ? 1.0f : element(a.weight, a.wdtype, i);
        const float v = scale.of<false, false>(s, w);
        if (a.y) y[i] = (T)v;
        if (a.format != NONE) {
            // d % 32 == 0: 32 lanes hold a block
            const float odd = scale.of<false, true>(s, w);
            unsigned top = magnitude_bits(odd);
#pragma unroll
            for (int m = 1; m < 32; m *= 2) top = max(top, (unsigned)__shfl_xor((int)top, m));
            const int64_t in_all = (int64_t)row * a.d + i;
            const float v8[8] = {odd, 0, 0, 0, 0, 0, 0, 0};
            int e;
            if (a.format == PI_MXFP8) {
                e = block_exponent<PI_MXFP8>(top);
                a.codes[in_all] = (uint8_t)mx_codes<PI_MXFP8>(v8, e).x;
            } else {
                e = block_exponent<PI_MXFP4>(top);
                const unsigned c = mx_codes<PI_MXFP4>(v8, e).x & 15u, next = __shfl_xor((int)c, 1);
                if (i % 2 == 0) a.codes[in_all / 2] = (uint8_t)(c | next << 4);
            }
            if (i % 32 == 0) a.scales[in_all / 32] = scale_byte(top, e);
        }
    }
}

// ---- microscaled quantisation ----------------------------------------------------------
//
// Bytes alone bound both directions.  A thread takes 8 elements, a quad of lanes a block; 2^log lanes a row, so that
// short rows fill a wave.  One piece of a row to a thread, in as many workgroups as that takes: two, four and eight rows of a
// thread in flight at once took 1, 5 and 9 us longer (10240 x 8192 f16 to MXFP4: 39.7 us, 5.3 TB/s, back 43.2; on other
// data every time, one after the other, both take 97, 4.4 TB/s, with one row or four).
struct ConvertArgs {
    const uint8_t* x;
    uint8_t* out;
    uint8_t* codes;
    uint8_t* scales;
    int64_t stride;            // of x or out, in bytes
    int rows, cols, log;
};

template <int XT, int FMT, bool VEC>
__global__ __launch_bounds__(NT) void k_mx_quantize(ConvertArgs a) {
    constexpr int ES = XT == F16 ? 2 : 4;
    const int at = ((int)blockIdx.y << a.log | (int)(threadIdx.x & ((1u << a.log) - 1))) * 8;
    if (at >= a.cols) return;
    const int per = NT >> a.log;
    for (int row = blockIdx.x * per + (threadIdx.x >> a.log); row < a.rows; row += gridDim.x * per) {
        float v[8];
        load8<XT, VEC>(a.x + (int64_t)row * a.stride + (int64_t)at * ES, v);
        store_block<FMT>(v, (int64_t)row * a.cols + at, a.codes, a.scales);
    }
}

template <int XT, int FMT, bool VEC>
__global__ __launch_bounds__(NT) void k_mx_dequantize(ConvertArgs a) {
    constexpr int ES = XT == F16 ? 2 : 4;
    const int at = ((int)blockIdx.y << a.log | (int)(threadIdx.x & ((1u << a.log) - 1))) * 8;
    if (at >= a.cols) return;
    const int per = NT >> a.log;
    for (int row = blockIdx.x * per + (threadIdx.x >> a.log); row < a.rows; row += gridDim.x * per) {
        const int64_t in_all = (int64_t)row * a.cols + at;
        u2 c;
        if constexpr (FMT == PI_MXFP8)
            c = *reinterpret_cast<const u2*>(a.codes + in_all);
        else
            c.x = *reinterpret_cast<const unsigned*>(a.codes + in_all / 2);
        const int scale = a.scales[in_all / 32];
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (FMT == PI_MXFP8) {
                const auto p = e % 2 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)c[e / 2], true)
                                     : __builtin_amdgcn_cvt_pk_f32_fp8((int)c[e / 2], false);
                v[2 * e] = p[0], v[2 * e + 1] = p[1];
            } else {
                const auto p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x >> (8 * e), 1.0f, 0);
                v[2 * e] = p[0], v[2 * e + 1] = p[1];
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = scale == 255 ? __builtin_nanf("") : __builtin_ldexpf(v[e], scale - 127);
        store8<XT, VEC>(a.out + (int64_t)row * a.stride + (int64_t)at * ES, v);
    }
}

template <bool QUANTIZE, int XT, int FMT, bool VEC>
pi_status launch_convert(const ConvertArgs& a, hipStream_t s) {
    const int per = NT >> a.log;
    const dim3 grid(std::min((a.rows + per - 1) / per, 1 << 16), ((a.cols / 8) + (1 << a.log) - 1) >> a.log);
    if constexpr (QUANTIZE)
        return launch(PI_K_MX_CONVERT, k_mx_quantize<XT, FMT, VEC>, grid, dim3(NT), 0, s, a);
    else
        return launch(PI_K_MX_CONVERT, k_mx_dequantize<XT, FMT, VEC>, grid, dim3(NT), 0, s, a);
}

template <bool QUANTIZE>
pi_status convert(const void* data, int64_t stride, int dtype, const pi_mx* mx, hipStream_t s) {
    const int size = dtype_size(dtype);
    ConvertArgs a{};
    a.x = (const uint8_t*)data;
    a.out = QUANTIZE ? nullptr : (uint8_t*)const_cast<void*>(data);
    a.codes = (uint8_t*)mx->codes, a.scales = mx->scales;
    a.stride = stride * size;
    a.rows = mx->rows, a.cols = mx->cols;
    a.log = 2;
    while (a.log < 8 && (1 << a.log) < mx->cols / 8) ++a.log;
    const bool vec = aligned(data, 16) && (mx->rows == 1 || a.stride % 16 == 0);
    const bool f16 = dtype == PI_F16, fp8 = mx->format == PI_MXFP8;
#define GO(XT, FMT) (vec ? launch_convert<QUANTIZE, XT, FMT, true>(a, s) : launch_convert<QUANTIZE, XT, FMT, false>(a, s))
    return f16 ? (fp8 ? GO(F16, PI_MXFP8) : GO(F16, PI_MXFP4)) : (fp8 ? GO(F32, PI_MXFP8) : GO(F32, PI_MXFP4));
#undef GO
}

pi_status check_matrix(const void* data, int64_t stride, int dtype, const pi_mx* mx, const char* name, bool out) {
    TRY(check_mx(mx, "mx"));
    TRY(check_elem_dtype(dtype, name));
    if (mx->rows == 0) return PI_OK;
    CHECK(data, PI_ERR_ARG, "%s is required", name);
    CHECK(aligned(data, dtype_size(dtype)), PI_ERR_ALIGN, "%s must be aligned to its elements", name);
    CHECK(stride >= (out && mx->rows > 1 ? mx->cols : 0) && stride < ((int64_t)1 << 40), PI_ERR_SHAPE,
          "%s: row_stride must be in %s..2^40", name, out ? "cols" : "0");
    CHECK(apart(data, ((mx->rows - 1) * stride + mx->cols) * dtype_size(dtype), mx), PI_ERR_ARG, "%s and mx overlap", name);
    return PI_OK;
}

// ---- the norm's entry point ---------------------------------------------------------

template <int XT, int TPR, int C>
pi_status launch_norm(const NormArgs& a, hipStream_t s) {
    constexpr int PER = std::max(NT / TPR, 1);
    const dim3 grid((a.rows + PER - 1) / PER), block(std::max(NT, TPR));
    if (a.format == PI_MXFP8) return launch(PI_K_NORM, k_rms_norm<XT, TPR, C, PI_MXFP8>, grid, block, 0, s, a);
    if (a.format == PI_MXFP4) return launch(PI_K_NORM, k_rms_norm<XT, TPR, C, PI_MXFP4>, grid, block, 0, s, a);
    return launch(PI_K_NORM, k_rms_norm<XT, TPR, C, NONE>, grid, block, 0, s, a);
}

// Threads of a row: one chunk each up to 8192 elements.  8192 elements on 1024 threads, and four chunks each on 256, us of
// f16 with an f16 delta, a sum, and MXFP8 or y: 1024 rows 14.4 and 14.0, 15.6 and 13.2; 8191 rows 95.6 and 94.8, 90.6 and
// 102.5; one row's kernel 4.2, 6.3.
template <int XT>
pi_status norm_by_size(const NormArgs& a, bool vec, hipStream_t s) {
    if (!vec || a.d > 8 * 2048) return launch(PI_K_NORM, k_rms_norm_any<XT>, dim3(a.rows), dim3(NT), 0, s, a);
    if (a.d <= 64) return launch_norm<XT, 8, 1>(a, s);
    if (a.d <= 128) return launch_norm<XT, 16, 1>(a, s);
    if (a.d <= 256) return launch_norm<XT, 32, 1>(a, s);
    if (a.d <= 512) return launch_norm<XT, 64, 1>(a, s);
    if (a.d <= 2048) return launch_norm<XT, 256, 1>(a, s);
    if (a.d <= 4096) return launch_norm<XT, 512, 1>(a, s);
    if (a.d <= 8192) return launch_norm<XT, 1024, 1>(a, s);
    return launch_norm<XT, 1024, 2>(a, s);
}

// Whether rows at i * s1 + j * s2 (i < n1, j < n2; s1, s2 >= len) share memory, each `len` long.  Two rows' places differ by
// k * s1 + l * s2; for every k the one l that can bring that inside a row is looked at.
bool rows_collide(int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t len) {
    if (n1 > n2) std::swap(n1, n2), std::swap(s1, s2);
    if (n1 == 1 || s2 >= (n1 - 1) * s1 + len || s1 >= (n2 - 1) * s2 + len) return false;
    for (int64_t k = 1; k < n1; ++k) {
        const int64_t l = std::min(k * s1 / s2, n2 - 1), past = k * s1 - l * s2;
        if (past < len || (l + 1 < n2 && s2 - past < len)) return true;
    }
    return false;
}

// An operand's rows, in bytes.
struct Place {
    int64_t at, ts, hs, len;
    Place(const pi_rows* r, int dtype, int d, int tokens, int heads)
        : at((int64_t)(uintptr_t)r->data), ts(tokens > 1 ? r->token_stride * dtype_size(dtype) : 0),
          hs(heads > 1 ? r->head_stride * dtype_size(dtype) : 0), len((int64_t)d * dtype_size(dtype)) {}
};

// Whether rows of two operands may share memory.  Where both have the same strides, rows that lie between each other are told
// from rows that meet: as above, for every k the l's that can bring two rows together.  Where the strides of the heads alone
// differ, so are the heads of every token of one that lie between those of the other.
bool rows_may_meet(const Place& p, const Place& q, int64_t tokens, int64_t heads) {
    const int64_t size_p = (heads - 1) * p.hs + p.len, size_q = (heads - 1) * q.hs + q.len;   // of a token
    if (p.at + (tokens - 1) * p.ts + size_p <= q.at || q.at + (tokens - 1) * q.ts + size_q <= p.at) return false;
    if (p.ts != q.ts) return true;
    const int64_t apart = q.at - p.at;
    if (p.hs != q.hs) {
        if (p.ts == 0) return true;
        const int64_t in_token = (apart % p.ts + p.ts) % p.ts;
        return in_token < size_p || in_token + size_q > p.ts;
    }
    int64_t n1 = tokens, s1 = p.ts, n2 = heads, s2 = p.hs;
    if (n1 > n2) std::swap(n1, n2), std::swap(s1, s2);
    for (int64_t k = 1 - n1; k < n1; ++k) {
        const int64_t from = apart + k * s1;
        // the lowest l for which q's row ends past p's beginning
        int64_t l = 1 - n2;
        if (s2 > 0) {
            const int64_t past = -q.len - from;                              // l s2 > past
            l = std::max(l, past >= 0 ? past / s2 + 1 : -((-past - 1) / s2));
        }
        if (l < n2 && from + l * s2 < p.len && from + l * s2 > -q.len) return true;
    }
    return false;
}

// rows of an operand, and whether all of them are 16-byte aligned
pi_status check_norm_rows(const pi_rows* r, const char* name, int dtype, int d, int tokens, int heads, bool out, bool& vec) {
    const int size = dtype_size(dtype);
    CHECK(r->data, PI_ERR_ARG, "%s is required", name);
    CHECK(aligned(r->data, size), PI_ERR_ALIGN, "%s must be aligned to its elements", name);
    CHECK(r->token_stride >= 0 && r->head_stride >= 0 && r->token_stride < ((int64_t)1 << 40) &&
              r->head_stride < ((int64_t)1 << 40),
          PI_ERR_SHAPE, "%s: strides must be in 0..2^40", name);
    CHECK((tokens - 1) * r->token_stride + (heads - 1) * r->head_stride < (int64_t)1 << 56, PI_ERR_SHAPE,
          "%s: rows past what addresses reach", name);
    CHECK(!out || ((tokens == 1 || r->token_stride >= d) && (heads == 1 || r->head_stride >= d)), PI_ERR_SHAPE,
          "%s: rows that are written may not overlap", name);
    vec = vec && aligned(r->data, 16) && (tokens == 1 || r->token_stride * size % 16 == 0) &&
          (heads == 1 || r->head_stride * size % 16 == 0);
    return PI_OK;
}

// an output takes an input's place with the same rows, of the same type; it may not overlap an operand in another way
pi_status check_in_place(const pi_rows* out, const char* name, int dtype, const pi_rows* in, const char* in_name, int in_dtype, int d,
                         int tokens, int heads) {
    if (!out || !in) return PI_OK;
    if (out->data == in->data) {
        CHECK(dtype == in_dtype && (tokens == 1 || out->token_stride == in->token_stride) &&
                  (heads == 1 || out->head_stride == in->head_stride),
              PI_ERR_ARG, "norm: %s takes the place of %s with other rows or another type", name, in_name);
        return PI_OK;
    }
    CHECK(!rows_may_meet(Place(out, dtype, d, tokens, heads), Place(in, in_dtype, d, tokens, heads), tokens, heads), PI_ERR_ARG,
          "norm: %s overlaps %s", name, in_name);
    return PI_OK;
}

// a matrix in a microscaled format takes no input's or output's place
pi_status check_apart(const pi_rows* r, const char* name, int dtype, const pi_mx* mx, int d, int tokens, int heads) {
    if (!r || !mx) return PI_OK;
    const int64_t last = (tokens - 1) * r->token_stride + (heads - 1) * r->head_stride;
    CHECK(apart(r->data, (last + d) * dtype_size(dtype), mx), PI_ERR_ARG, "norm: %s and mx overlap", name);
    return PI_OK;
}

}  // namespace

extern "C" {

pi_status pi_rms_norm(const pi_norm* norm, int32_t tokens, int32_t heads, int32_t dtype, const pi_rows* x, int32_t ddtype,
                      const pi_rows* delta, const pi_rows* sum, const pi_rows* y, const pi_mx* mx, void* stream) {
    CHECK(norm, PI_ERR_ARG, "NULL norm");
    CHECK(norm->d >= 1 && norm->d <= (1 << 20), PI_ERR_SHAPE, "norm: d must be in 1..2^20");
    CHECK(norm->eps >= 0.0f && std::isfinite(norm->eps), PI_ERR_ARG, "norm: eps must be finite and not negative");
    CHECK(tokens >= 0 && heads >= 1 && (int64_t)tokens * heads <= (1 << 23), PI_ERR_SHAPE,
          "norm: heads must be >= 1 and tokens * heads in 0..2^23");
    // (a workgroup to a row: a launch holds fewer than 2^32 threads)
    CHECK(norm->d <= 2048 || (int64_t)tokens * heads <= (1 << 21), PI_ERR_SHAPE, "norm: tokens * heads must be in 0..2^21 for d > 2048");
    TRY(check_elem_dtype(dtype, "norm"));
    const int d = norm->d;
    bool vec = d % 8 == 0;
    if (norm->weight) {
        TRY(check_elem_dtype(norm->wdtype, "norm: weight"));
        CHECK(aligned(norm->weight, dtype_size(norm->wdtype)), PI_ERR_ALIGN, "norm: weight must be aligned to its elements");
        vec = vec && aligned(norm->weight, 16);
    }
    CHECK(sum || y || mx, PI_ERR_ARG, "norm: one of sum, y and mx is required");
    CHECK(delta || !sum, PI_ERR_ARG, "norm: sum without delta");
    if (delta) TRY(check_elem_dtype(ddtype, "norm: delta"));
    if (mx) {
        TRY(check_mx(mx, "mx"));
        CHECK(d % 32 == 0, PI_ERR_SHAPE, "norm: d must be a multiple of 32 for mx");
        CHECK(mx->rows == tokens && mx->cols == (int64_t)heads * d, PI_ERR_SHAPE, "norm: mx must be [tokens][heads * d]");
    }
    if (tokens == 0) return PI_OK;
    CHECK(x, PI_ERR_ARG, "x is required");
    NormArgs a{};
    const int size = dtype_size(dtype);
    TRY(check_norm_rows(x, "x", dtype, d, tokens, heads, false, vec));
    a.x = (const uint8_t*)x->data, a.x_ts = x->token_stride * size, a.x_hs = x->head_stride * size;
    a.ddtype = a.wdtype = a.format = NONE;
    if (delta) {
        TRY(check_norm_rows(delta, "delta", ddtype, d, tokens, heads, false, vec));
        a.ddtype = ddtype;
        a.delta = (const uint8_t*)delta->data;
        a.d_ts = delta->token_stride * dtype_size(ddtype), a.d_hs = delta->head_stride * dtype_size(ddtype);
    }
    if (sum) {
        TRY(check_norm_rows(sum, "sum", dtype, d, tokens, heads, true, vec));
        a.sum = (uint8_t*)sum->data, a.s_ts = sum->token_stride * size, a.s_hs = sum->head_stride * size;
    }
    if (y) {
        TRY(check_norm_rows(y, "y", dtype, d, tokens, heads, true, vec));
        a.y = (uint8_t*)y->data, a.y_ts = y->token_stride * size, a.y_hs = y->head_stride * size;
        CHECK(!sum || sum->data != y->data, PI_ERR_ARG, "norm: sum and y must differ");
    }
    for (const pi_rows* out : {sum, y}) {
        const char* name = out == sum ? "sum" : "y";
        TRY(check_in_place(out, name, dtype, x, "x", dtype, d, tokens, heads));
        TRY(check_in_place(out, name, dtype, delta, "delta", ddtype, d, tokens, heads));
        TRY(check_apart(out, name, dtype, mx, d, tokens, heads));
        CHECK(!out || !rows_collide(tokens, out->token_stride, heads, out->head_stride, d), PI_ERR_SHAPE,
              "norm: %s has rows that overlap", name);
    }
    TRY(check_in_place(sum, "sum", dtype, y, "y", dtype, d, tokens, heads));   // (not in one place: see above)
    if (mx) TRY(check_written(mx, "mx"));
    TRY(check_apart(x, "x", dtype, mx, d, tokens, heads));
    TRY(check_apart(delta, "delta", ddtype, mx, d, tokens, heads));
    if (norm->weight) {
        const int64_t bytes = (int64_t)d * dtype_size(norm->wdtype);
        // (a weight between two rows of an output is refused as well)
        for (const pi_rows* out : {sum, y}) {
            if (!out) continue;
            const Place p(out, dtype, d, tokens, heads);
            CHECK(apart(out->data, (tokens - 1) * p.ts + (heads - 1) * p.hs + p.len, norm->weight, bytes), PI_ERR_ARG,
                  "norm: %s overlaps the weight", out == sum ? "sum" : "y");
        }
        CHECK(!mx || apart(norm->weight, bytes, mx), PI_ERR_ARG, "norm: mx overlaps the weight");
    }
    if (mx) a.format = mx->format, a.codes = (uint8_t*)mx->codes, a.scales = mx->scales;
    if (norm->weight) a.wdtype = norm->wdtype, a.weight = (const uint8_t*)norm->weight;
    a.eps = norm->eps;
    a.rows = tokens * heads, a.heads = heads, a.d = d;
    return dtype == PI_F16 ? norm_by_size<F16>(a, vec, (hipStream_t)stream) : norm_by_size<F32>(a, vec, (hipStream_t)stream);
}

pi_status pi_mx_quantize(const void* x, int64_t row_stride, int32_t dtype, const pi_mx* mx, void* stream) {
    TRY(check_matrix(x, row_stride, dtype, mx, "x", false));
    TRY(check_written(mx, "mx"));
    return mx->rows == 0 ? PI_OK : convert<true>(x, row_stride, dtype, mx, (hipStream_t)stream);
}

pi_status pi_mx_dequantize(const pi_mx* mx, void* out, int64_t row_stride, int32_t dtype, void* stream) {
    TRY(check_matrix(out, row_stride, dtype, mx, "out", true));
    return mx->rows == 0 ? PI_OK : convert<false>(out, row_stride, dtype, mx, (hipStream_t)stream);
}

}  // extern "C"
