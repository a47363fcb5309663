// pi_mx.hip -- product of two microscaled matrices.
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

typedef int i8v __attribute__((ext_vector_type(8)));

struct ProductArgs {
    const uint8_t* a;
    const uint8_t* a_scales;
    const uint8_t* w;
    const uint8_t* w_scales;
    const float* bias;
    uint8_t* out;
    int64_t out_stride;          // in elements
    int m, n, k;
};

// How a product is formed:
//   FP4     both sides MXFP4: the scaled matrix instruction of 16 x 16 x 128, whose products are exact
//   FP8     a MXFP8: the same instruction.  It cuts the products of eight neighbouring elements 2^-13 below the largest
//           of them, which leaves outputs off by 2e-5 of their size (measured; activations with outliers): a tenth of
//           f16's own rounding, so it is taken for f16 outputs alone
//   FP8_F32 a MXFP8, float32 outputs: both sides turned to bfloat16 with their scales, which is exact down to 2^-126,
//           and the instruction of 16 x 16 x 32, half as fast
enum { M_FP4 = 0, M_FP8 = 1, M_FP8_F32 = 2 };

// A fragment: row l % 16 of 16 rows, a part of 128 elements in each lane; g = l / 16.
//   MXFP4, and MXFP8 of M_FP8_F32: elements 32 g .. 32 g + 31 (a block)
//   MXFP8 of M_FP8: elements 16 g .. 16 g + 15 and 64 + 16 g .. 64 + 16 g + 15, the instruction's own order
// The scale of lane l is block g's in every form.  Result: column l % 16 (of the second operand), rows 4 g .. 4 g + 3.
template <bool WIDE>
struct Frag {
    u4 v[WIDE ? 2 : 1];
};

// byte of a row of codes at which chunk c of lane group g begins, for 128 elements
template <int MODE, bool WIDE>
__device__ __forceinline__ int chunk_at(int g, int c) {
    if constexpr (!WIDE) return 16 * g;
    if constexpr (MODE == M_FP8) return 16 * g + 64 * c;
    return 32 * g + 16 * c;
}

// 128 elements from step `k` on; those past K are zero
template <int MODE, bool WIDE>
__device__ __forceinline__ Frag<WIDE> load_frag(const uint8_t* row, int k, int K, int g) {
    Frag<WIDE> f;
    constexpr int PER = WIDE ? 1 : 2;       // elements of a byte
#pragma unroll
    for (int c = 0; c < (WIDE ? 2 : 1); ++c) {
        const int at = k / PER + chunk_at<MODE, WIDE>(g, c);
        f.v[c] = at * PER < K ? ld16(row + at) : u4{0u, 0u, 0u, 0u};
    }
    return f;
}

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));

template <bool WIDE>
__device__ __forceinline__ i8v regs(const Frag<WIDE>& f) {
    const u4 hi = WIDE ? f.v[WIDE ? 1 : 0] : u4{0u, 0u, 0u, 0u};
    return i8v{(int)f.v[0].x, (int)f.v[0].y, (int)f.v[0].z, (int)f.v[0].w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// the i-th 8 elements of a lane in bfloat16, scaled (byte 0 of scale; 255 gives NaN)
__device__ __forceinline__ bf8 wide_bf16(const Frag<true>& f, int i, int scale) {
    const float s = bits_f((unsigned)(scale & 255) << 23);
    const unsigned lo = f.v[i / 2][2 * (i % 2)], hi = f.v[i / 2][2 * (i % 2) + 1];
    const bf2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true);
    const bf2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true);
    return bf8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ bf8 wide_bf16(const Frag<false>& f, int i, int scale) {
    const float s = bits_f((unsigned)(scale & 255) << 23);
    const unsigned v = f.v[0][i];
    const bf2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, s, 1);
    const bf2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, s, 2), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, s, 3);
    return bf8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// sum += the products of 128 elements: 16 rows of w by 16 rows of a
template <int MODE>
__device__ __forceinline__ f4 step(const Frag<false>& w, int w_scale, const Frag<MODE != M_FP4>& a, int a_scale, f4 sum) {
    if constexpr (MODE == M_FP8_F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wide_bf16(w, i, w_scale), wide_bf16(a, i, a_scale), sum, 0, 0, 0);
        return sum;
    } else {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(regs(w), regs(a), sum, 4, MODE == M_FP4 ? 4 : 0, 0, w_scale, 0,
                                                                a_scale);
    }
}

constexpr int WAVES = 4;

// 16 rows of w by 16 of a for each workgroup, the steps of 128 dealt to its waves.
template <int MODE, int DT>
__global__ __launch_bounds__(WAVE * WAVES) void k_mx_product(ProductArgs p) {
    __shared__ f4 parts[WAVES][WAVE];
    constexpr bool WIDE = MODE != M_FP4;
    const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE, g = lane / 16;
    const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16;
    const int64_t n = min(n0 + lane % 16, p.n - 1), m = min(m0 + lane % 16, p.m - 1);
    const uint8_t* w = p.w + n * (p.k / 2);
    const uint8_t* a = p.a + m * (WIDE ? p.k : p.k / 2);
    const uint8_t* ws = p.w_scales + n * (p.k / 32);
    const uint8_t* as = p.a_scales + m * (p.k / 32);
    f4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k = wave * 128; k < p.k; k += WAVES * 128) {
        const bool in = k + 32 * g < p.k;
        sum = step<MODE>(load_frag<MODE, false>(w, k, p.k, g), in ? ws[k / 32 + g] : 127, load_frag<MODE, WIDE>(a, k, p.k, g),
                         in ? as[k / 32 + g] : 127, sum);
    }
    // (a matrix instruction takes every lane: it may not sink below a branch)
    asm volatile("" : "+v"(sum));
    parts[wave][lane] = sum;
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int i = 1; i < WAVES; ++i) sum += parts[i][lane];
    const int row = m0 + lane % 16;
    if (row >= p.m) return;
    typedef typename std::conditional<DT == F16, _Float16, float>::type T;
    T* out = reinterpret_cast<T*>(p.out) + row * p.out_stride;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int col = n0 + 4 * g + i;
        if (col < p.n) out[col] = (T)(sum[i] + (p.bias ? p.bias[col] : 0.0f));
    }
}

}  // namespace

extern "C" {

size_t pi_mx_product_workspace_bytes(int32_t m, int32_t n, int32_t k) { return 0; }

pi_status pi_mx_product(const pi_mx* a, const pi_mx* w, const float* bias, void* out, int64_t out_stride, int32_t dtype,
                        void* ws, size_t ws_bytes, void* stream) {
    TRY(check_mx(a, "a"));
    TRY(check_mx(w, "w"));
    CHECK(w->format == PI_MXFP4, PI_ERR_DTYPE, "w must be PI_MXFP4");
    CHECK(a->cols == w->cols, PI_ERR_SHAPE, "a and w must have the same cols");
    TRY(check_elem_dtype(dtype, "out"));
    if (a->rows == 0 || w->rows == 0) return PI_OK;
    CHECK(out, PI_ERR_ARG, "out is required");
    CHECK(aligned(out, dtype_size(dtype)), PI_ERR_ALIGN, "out must be aligned to its elements");
    CHECK(!bias || aligned(bias, 4), PI_ERR_ALIGN, "bias must be 4-byte aligned");
    CHECK((a->rows == 1 || out_stride >= w->rows) && out_stride >= 0 && out_stride < ((int64_t)1 << 40), PI_ERR_SHAPE,
          "out: out_stride must be in w->rows..2^40");
    ProductArgs p{(const uint8_t*)a->codes, a->scales, (const uint8_t*)w->codes, w->scales, bias, (uint8_t*)out, out_stride,
                  a->rows, w->rows, a->cols};
    hipStream_t s = (hipStream_t)stream;
    const dim3 grid((p.n + 15) / 16, (p.m + 15) / 16), block(WAVE * WAVES);
#define GO(MODE, DT) launch(PI_K_MX_PRODUCT, k_mx_product<MODE, DT>, grid, block, 0, s, p)
    if (a->format == PI_MXFP8) return dtype == PI_F16 ? GO(M_FP8, F16) : GO(M_FP8_F32, F32);
    return dtype == PI_F16 ? GO(M_FP4, F16) : GO(M_FP4, F32);
#undef GO
}

}  // extern "C"
