// pi_mx.h -- microscaled formats: how a block of 32 elements is quantised, and the
// checks of the descriptors that the entry points share.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "pi.h"
#include "pi_device.h"
#include "pi_launch.h"

namespace pi {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));

inline int64_t mx_row_bytes(int format, int64_t cols) { return format == PI_MXFP4 ? cols / 2 : cols; }

inline pi_status check_mx(const pi_mx* m, const char* name) {
    CHECK(m, PI_ERR_ARG, "%s is required", name);
    CHECK(m->format == PI_MXFP8 || m->format == PI_MXFP4, PI_ERR_DTYPE, "%s: format must be PI_MXFP8 or PI_MXFP4", name);
    CHECK(m->rows >= 0 && m->rows <= (1 << 24), PI_ERR_SHAPE, "%s: rows must be in 0..2^24", name);
    CHECK(m->cols >= 32 && m->cols <= (1 << 20) && m->cols % 32 == 0, PI_ERR_SHAPE,
          "%s: cols must be a multiple of 32 in 32..2^20", name);
    if (m->rows == 0) return PI_OK;
    CHECK(m->codes && m->scales, PI_ERR_ARG, "%s: codes and scales are required", name);
    CHECK(aligned(m->codes, 16) && aligned(m->scales, 16), PI_ERR_ALIGN, "%s: codes and scales must be 16-byte aligned", name);
    return PI_OK;
}

// Whether spans of bytes lie apart (one that is NULL does)
inline bool apart(const void* a, int64_t bytes_a, const void* b, int64_t bytes_b) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return !a || !b || x + (uint64_t)bytes_a <= y || y + (uint64_t)bytes_b <= x;
}

inline bool apart(const void* p, int64_t bytes, const pi_mx* m) {
    return apart(p, bytes, m->codes, m->rows * mx_row_bytes(m->format, m->cols)) &&
           apart(p, bytes, m->scales, (int64_t)m->rows * (m->cols / 32));
}

// codes and scales of a matrix that is written
inline pi_status check_written(const pi_mx* m, const char* name) {
    CHECK(apart(m->codes, m->rows * mx_row_bytes(m->format, m->cols), m->scales, (int64_t)m->rows * (m->cols / 32)), PI_ERR_ARG,
          "%s: codes and scales overlap", name);
    return PI_OK;
}

inline pi_status check_elem_dtype(int dtype, const char* name) {
    CHECK(dtype == PI_F32 || dtype == PI_F16, PI_ERR_DTYPE, "%s: dtype must be PI_F32 or PI_F16", name);
    return PI_OK;
}

// ---- device: 8 elements of one thread -------------------------------------------

// 8 consecutive elements as float32.  VEC: p is 16-byte aligned.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void* p, float* v) {
    if constexpr (DT == F32) {
        if constexpr (VEC) {
            const f4 a = reinterpret_cast<const f4*>(p)[0], b = reinterpret_cast<const f4*>(p)[1];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = a[e], v[e + 4] = b[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = reinterpret_cast<const float*>(p)[e];
        }
    } else {
        if constexpr (VEC) {
            const h8 a = *reinterpret_cast<const h8*>(p);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (float)a[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (float)reinterpret_cast<const _Float16*>(p)[e];
        }
    }
}

// 8 consecutive elements, each rounded once
template <int DT, bool VEC>
__device__ __forceinline__ void store8(void* p, const float* v) {
    if constexpr (DT == F32) {
        if constexpr (VEC) {
            reinterpret_cast<f4*>(p)[0] = f4{v[0], v[1], v[2], v[3]};
            reinterpret_cast<f4*>(p)[1] = f4{v[4], v[5], v[6], v[7]};
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) reinterpret_cast<float*>(p)[e] = v[e];
        }
    } else {
        if constexpr (VEC) {
            h8 a;
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] = (_Float16)v[e];
            *reinterpret_cast<h8*>(p) = a;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) reinterpret_cast<_Float16*>(p)[e] = (_Float16)v[e];
        }
    }
}

// ---- device: quantisation --------------------------------------------------------

__device__ __forceinline__ unsigned magnitude_bits(float v) { return __builtin_bit_cast(unsigned, v) & 0x7fffffffu; }

// The exponent e of a block's scale 2^e from the bits of its largest magnitude (as integers, magnitudes compare like
// the floats, infinities and NaN above them): floor(log2) less the format's largest exponent, at least -127.
template <int FMT>
__device__ __forceinline__ int block_exponent(unsigned top) {
    const int e = (int)(top >> 23) - 127 - (FMT == PI_MXFP8 ? 8 : 2);   // (a subnormal's is below -127 anyway)
    return e < -127 ? -127 : e;
}

__device__ __forceinline__ uint8_t scale_byte(unsigned top, int e) {
    return top >= 0x7f800000u ? 255 : (uint8_t)(e + 127);
}

// Codes of 8 elements, first in the lowest bits: 8 bytes (MXFP8) or 4 in .x (MXFP4).  x / 2^e is exact in float32
// where its rounding matters; the conversions round to nearest, ties to even (measured over every f16 value).
template <int FMT>
__device__ __forceinline__ u2 mx_codes(const float* v, int e) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = __builtin_ldexpf(v[i], -e);
    if constexpr (FMT == PI_MXFP8) {
        // (the conversion makes NaN of what is past the largest value)
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = fminf(fmaxf(t[i], -448.0f), 448.0f);
        int a = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
        a = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], a, true);
        int b = __builtin_amdgcn_cvt_pk_fp8_f32(t[4], t[5], 0, false);
        b = __builtin_amdgcn_cvt_pk_fp8_f32(t[6], t[7], b, true);
        return u2{(unsigned)a, (unsigned)b};
    } else {
        unsigned a = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, t[0], t[1], 1.0f, 0);
        a = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(a, t[2], t[3], 1.0f, 1);
        a = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(a, t[4], t[5], 1.0f, 2);
        a = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(a, t[6], t[7], 1.0f, 3);
        return u2{a, 0u};
    }
}

// Quantises the 8 elements of each of the 4 lanes of a quad, which hold a block together, and stores codes and scale:
// `at` the index of the thread's first element in the whole matrix.  All 4 lanes are here.
template <int FMT>
__device__ __forceinline__ void store_block(const float* v, int64_t at, uint8_t* codes, uint8_t* scales) {
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, magnitude_bits(v[i]));
    top = max(top, (unsigned)__builtin_amdgcn_update_dpp(0, (int)top, DPP_QUAD_1032, 0xf, 0xf, false));
    top = max(top, (unsigned)__builtin_amdgcn_update_dpp(0, (int)top, DPP_QUAD_2301, 0xf, 0xf, false));
    const int e = block_exponent<FMT>(top);
    const u2 c = mx_codes<FMT>(v, e);
    if constexpr (FMT == PI_MXFP8)
        *reinterpret_cast<u2*>(codes + at) = c;
    else
        *reinterpret_cast<unsigned*>(codes + at / 2) = c.x;
    if (threadIdx.x % 4 == 0) scales[at / 32] = scale_byte(top, e);
}

}  // namespace pi
