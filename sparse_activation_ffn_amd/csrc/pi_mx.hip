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

constexpr int XCDS = 8;

struct ProductArgs {
    const uint8_t* a;
    const uint8_t* a_scales;
    const uint8_t* w;
    const uint8_t* w_scales;
    const float* bias;
    uint8_t* out;
    int64_t out_stride;          // in elements
    int m, n, k;
    int splits;                  // of K; each split's sums go to part [splits][m][n] if there are several
    float* part;
    bool vec;                    // four outputs of a row, from a multiple of four on, are aligned to their size
};

// How a product is formed:
//   FP4     both sides MXFP4: the scaled matrix instruction of 16 x 16 x 128, whose products are exact
//   FP8     a MXFP8: the same instruction.  It cuts the products of eight neighbouring elements 2^-13 below the largest
//           of them, which leaves outputs off by 2e-5 of their size (measured; activations with outliers): a tenth of
//           f16's own rounding, so it is taken for f16 outputs alone
//   FP8_F32 a MXFP8, float32 outputs: both sides turned to bfloat16 with their scales, which is exact from 2^-126 to below
//           2^128 (what float32 holds, and so what is quantised from it), and the instruction of 16 x 16 x 32, half as fast
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
__host__ __device__ constexpr __forceinline__ int chunk_at(int g, int c) {
    if constexpr (!WIDE) return 16 * g;
    if constexpr (MODE == M_FP8) return 16 * g + 64 * c;
    return 32 * g + 16 * c;
}

// 128 elements from `k` on, at `off` of a base that is the same in all lanes.  FULL: all of them are there; else lanes whose
// elements are past K read the row's first bytes, and clear_tail clears what they got.
template <int MODE, bool WIDE, bool FULL>
__device__ __forceinline__ Frag<WIDE> load_frag(const uint8_t* base, unsigned off, int k, int K, int g) {
    Frag<WIDE> f;
    constexpr int PER = WIDE ? 1 : 2;       // elements of a byte
#pragma unroll
    for (int c = 0; c < (WIDE ? 2 : 1); ++c) {
        const int at = k / PER + chunk_at<MODE, WIDE>(g, c);
        f.v[c] = ld16(base + (off + (unsigned)(FULL || at * PER < K ? at : 0)));
    }
    return f;
}

template <int MODE, bool WIDE>
__device__ __forceinline__ void clear_tail(Frag<WIDE>& f, int& scale, int k, int K, int g) {
    constexpr int PER = WIDE ? 1 : 2;
#pragma unroll
    for (int c = 0; c < (WIDE ? 2 : 1); ++c)
        if (k + chunk_at<MODE, WIDE>(g, c) * PER >= K) f.v[c] = u4{0u, 0u, 0u, 0u};
    if (k + 32 * g >= K) scale = 127;
}

// the scale of block g of the 128 elements from k on
__device__ __forceinline__ int load_scale(const uint8_t* base, unsigned off, int k, int K, int g) {
    return base[off + (k + 32 * g < K ? k / 32 + g : 0)];
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

// sum[i][j] += the products of 128 elements: 16 rows of a (i) by 16 rows of w (j).  Scales are in byte 0.
template <int MODE, int MT, int NT>
__device__ __forceinline__ void steps_of(const Frag<false> (&w)[NT], const int (&ws)[NT], const Frag<MODE != M_FP4> (&a)[MT],
                                         const int (&as)[MT], f4 (&sum)[MT][NT]) {
    if constexpr (MODE == M_FP8_F32) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            bf8 wv[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) wv[j] = wide_bf16(w[j], c, ws[j]);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const bf8 av = wide_bf16(a[i], c, as[i]);
#pragma unroll
                for (int j = 0; j < NT; ++j) sum[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[j], av, sum[i][j], 0, 0, 0);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                sum[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(regs(w[j]), regs(a[i]), sum[i][j], 4,
                                                                             MODE == M_FP4 ? 4 : 0, 0, ws[j], 0, as[i]);
    }
}

// sum + bias, rounded once, at row i and column j of the output
template <int DT>
__device__ __forceinline__ void store_out(const ProductArgs& p, int i, int j, float sum) {
    typedef typename std::conditional<DT == F16, _Float16, float>::type T;
    reinterpret_cast<T*>(p.out)[i * p.out_stride + j] = (T)(sum + (p.bias ? p.bias[j] : 0.0f));
}

constexpr int LONG = 512;        // elements whose scales come in one load

// The elements past the last whole 512: fragments straight from memory, in steps of 128.
template <int MODE>
__device__ __forceinline__ void tail_steps(const ProductArgs& p, const uint8_t* w, const uint8_t* ws, const uint8_t* a,
                                           const uint8_t* as, unsigned w_row, unsigned a_row, int g, f4 (&sum)[1][1]) {
    constexpr bool WIDE = MODE != M_FP4;
    const int wb = p.k / 2, ab = WIDE ? p.k : p.k / 2, sb = p.k / 32;
    for (int k = p.k / LONG * LONG; k < p.k; k += 128) {
        Frag<false> wf[1] = {load_frag<MODE, false, false>(w, w_row * wb, k, p.k, g)};
        Frag<WIDE> af[1] = {load_frag<MODE, WIDE, false>(a, a_row * ab, k, p.k, g)};
        int wsc[1] = {load_scale(ws, w_row * sb, k, p.k, g)}, asc[1] = {load_scale(as, a_row * sb, k, p.k, g)};
        if (k + 128 > p.k) {
            clear_tail<MODE, false>(wf[0], wsc[0], k, p.k, g);
            clear_tail<MODE, WIDE>(af[0], asc[0], k, p.k, g);
        }
        steps_of<MODE, 1, 1>(wf, wsc, af, asc, sum);
    }
}

// the same of four columns, from a multiple of four on
template <int DT>
__device__ __forceinline__ void store_out4(const ProductArgs& p, int i, int j, f4 sum) {
    if (j + 4 > p.n || !p.vec) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e < p.n) store_out<DT>(p, i, j + e, sum[e]);
        return;
    }
    if (p.bias) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += p.bias[j + e];
    }
    if constexpr (DT == F16) {
        typedef _Float16 h4 __attribute__((ext_vector_type(4)));
        *reinterpret_cast<h4*>(p.out + (i * p.out_stride + j) * 2) =
            h4{(_Float16)sum[0], (_Float16)sum[1], (_Float16)sum[2], (_Float16)sum[3]};
    } else {
        *reinterpret_cast<f4*>(p.out + (i * p.out_stride + j) * 4) = sum;
    }
}

// ---- few rows of a -----------------------------------------------------------------
//
// The weights' bytes bound it: every one is read once, by one wave, from memory into the registers of the matrix
// instruction, no LDS and no barrier on the way.  A workgroup takes 16 rows of w and 16 of a; its KW waves share out K in
// pieces of 512 elements and join their sums in LDS in a fixed order.  A piece is what is loaded at once, so that both
// halves of a 128-byte line are asked for together and a row's scales in one load: in pieces of 128 the lines had left the
// 32 KB of the first-level cache before their other half was asked for (1 x 10240 x 8192: 18.4 us, 14.5 so).  A load
// of 16 rows takes the path to memory some 64 cycles whatever it brings, which is why tiles through LDS are faster where
// there are enough of them; 1 x 4096 x 8192 takes 7.0 us with the launch.
constexpr int STEPS = LONG / 128;
template <int MODE>
struct Piece {
    Frag<false> w[STEPS][1];
    Frag<MODE != M_FP4> a[STEPS][1];
    unsigned ws[STEPS], as[STEPS];          // 4 scales each
};

template <int MODE, int DT, int KW>
__global__ __launch_bounds__(WAVE * KW) void k_mx_few(ProductArgs p) {
    __shared__ f4 parts[KW][WAVE];
    constexpr bool WIDE = MODE != M_FP4;
    const int lane = threadIdx.x % WAVE, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE), g = lane / 16;
    const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16;
    const int wb = p.k / 2, ab = WIDE ? p.k : p.k / 2, sb = p.k / 32;   // bytes of a row
    const uint8_t* w = p.w + (int64_t)n0 * wb;
    const uint8_t* a = p.a + (int64_t)m0 * ab;
    const uint8_t* ws = p.w_scales + (int64_t)n0 * sb;
    const uint8_t* as = p.a_scales + (int64_t)m0 * sb;
    const unsigned w_row = min(lane % 16, p.n - 1 - n0), a_row = min(lane % 16, p.m - 1 - m0);
    const int pieces = p.k / LONG, each = (pieces + KW - 1) / KW;
    const int from = min(wave * each, pieces), to = min(from + each, pieces);

    auto load = [&](Piece<MODE>& s, int at) __attribute__((always_inline)) {
        const int k = at * LONG;
#pragma unroll
        for (int t = 0; t < STEPS; ++t) s.w[t][0] = load_frag<MODE, false, true>(w, w_row * wb, k + 128 * t, p.k, g);
        __builtin_memcpy(s.ws, ws + (w_row * sb + k / 32), sizeof(s.ws));     // (at any alignment)
#pragma unroll
        for (int t = 0; t < STEPS; ++t) s.a[t][0] = load_frag<MODE, WIDE, true>(a, a_row * ab, k + 128 * t, p.k, g);
        __builtin_memcpy(s.as, as + (a_row * sb + k / 32), sizeof(s.as));
    };
    f4 sum[1][1] = {{f4{0.0f, 0.0f, 0.0f, 0.0f}}};
    auto compute = [&](const Piece<MODE>& s) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < STEPS; ++t) {
            const int wsc[1] = {(int)(s.ws[t] >> (8 * g))}, asc[1] = {(int)(s.as[t] >> (8 * g))};
            steps_of<MODE, 1, 1>(s.w[t], wsc, s.a[t], asc, sum);
        }
    };
    if (from < to) {
        Piece<MODE> x, y;
        load(x, from);
        int at = from;
        for (; at + 2 < to; at += 2) {
            load(y, at + 1);
            compute(x);
            load(x, at + 2);
            compute(y);
        }
        if (at + 1 < to) {
            load(y, at + 1);
            compute(x);
            compute(y);
        } else {
            compute(x);
        }
    }
    if (wave == KW - 1) tail_steps<MODE>(p, w, ws, a, as, w_row, a_row, g, sum);
    // (a matrix instruction takes every lane: it may not sink below a branch)
    asm volatile("" : "+v"(sum[0][0]));
    parts[wave][lane] = sum[0][0];
    __syncthreads();
    for (int e = threadIdx.x; e < 256; e += WAVE * KW) {
        const int row = e / 16, col = e % 16, m = m0 + row, n = n0 + col;
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < KW; ++i) v += parts[i][col / 4 * 16 + row][col % 4];
        if (m < p.m && n < p.n) store_out<DT>(p, m, n, v);
    }
}

template <int MODE, int DT, int KW>
pi_status launch_few(const ProductArgs& p, hipStream_t s) {
    const dim3 grid((p.n + 15) / 16, (p.m + 15) / 16), block(WAVE * KW);
    return launch(PI_K_MX_PRODUCT, k_mx_few<MODE, DT, KW>, grid, block, 0, s, p);
}

// ---- many rows of a ----------------------------------------------------------------
//
// Tiles of BM rows of a by BN rows of w through LDS, in a ring of stages of KS elements: while one is multiplied, the RING - 1
// after it come in by direct loads, which are waited for by count.  A row's 16-byte pieces are permuted by the row, so that the
// 16 rows that a fragment read takes at one piece lie in 16 different pieces of 256 bytes.  Scales come 512 elements at a time,
// by direct loads where K is a multiple of 512, else through registers.  The matrix cores bound large products, bytes and the
// depth of the ring small ones.  us (TFLOP/s), 4096 x 10240 x 8192: MXFP8 to f16 276 (2490), to float32 488 (1410: half the
// rate, and both sides turned to bfloat16 by every wave that reads them), MXFP4 224 (3060: there the waves wait 45% of their
// cycles, for the next stage above all, and LDS is busy for a third).
__device__ __forceinline__ void load_to_lds(const uint8_t* from, uint8_t* to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                     (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

// piece c of row r of a tile with rows of RB bytes
template <int RB>
__device__ __forceinline__ int piece_of(int r, int c) {
    return c ^ (RB >= 256 ? r & 15 : RB == 128 ? (r >> 1) & 7 : (r >> 2) & 3);
}

// all but the last N loads of this wave have arrived (the other counters as they are)
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N < 64, "a 6-bit counter");
    __builtin_amdgcn_s_waitcnt((N & 15) | 0x0f70 | (N >> 4) << 14);
}

template <int MODE, int MT, int NT, int WM, int WN, int KS, int RING>
struct Tile {
    static constexpr bool WIDE = MODE != M_FP4;
    static constexpr int BM = 16 * MT * WM, BN = 16 * NT * WN, WAVES = WM * WN;
    static constexpr int RA = WIDE ? KS : KS / 2, RW = KS / 2;                    // bytes of a row in a stage
    static constexpr int A_BYTES = BM * RA, W_BYTES = BN * RW, STAGE = A_BYTES + W_BYTES;
    static constexpr int NA = A_BYTES / 1024, NW = W_BYTES / 1024;                // load instructions of a stage
    static constexpr int LA = (NA + WAVES - 1) / WAVES, LW = (NW + WAVES - 1) / WAVES; // of a wave: all have as many, so
                                                                                  // that all count alike (some load a piece again)
    static constexpr int SCALES = (BM + BN + WAVE - 1) / WAVE * WAVE * 16;          // whole loads
    static constexpr int LDS = RING * STAGE + 2 * SCALES;
    static_assert(NA * 1024 == A_BYTES && NW * 1024 == W_BYTES, "whole loads");
};

template <int MODE, int DT, int MT, int NT, int WM, int WN, int KS, int RING, bool ALIGNED>
__global__ __launch_bounds__(WAVE * WM * WN, 2) void k_mx_many(ProductArgs p) {
    typedef Tile<MODE, MT, NT, WM, WN, KS, RING> T;
    constexpr bool WIDE = T::WIDE;
    constexpr int BM = T::BM, BN = T::BN, THREADS = WAVE * T::WAVES, SPT = (BM + BN + THREADS - 1) / THREADS;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int lane = threadIdx.x % WAVE, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE), g = lane / 16;

    // Workgroups go round the 8 XCDs: each XCD takes a run of tiles, eight rows of tiles at a time, so that what its
    // workgroups read at one time fits its 4 MB of cache.
    const int tiles_m = (p.m + BM - 1) / BM, tiles_n = (p.n + BN - 1) / BN, total = tiles_m * tiles_n;
    const int per = (int)(gridDim.x / XCDS), tile = (int)(blockIdx.x % XCDS) * per + (int)(blockIdx.x / XCDS);
    if (tile >= total) return;
    const int band = tile / (8 * tiles_n), high = min(8, tiles_m - band * 8), in_band = tile - band * 8 * tiles_n;
    const int m0 = (band * 8 + in_band % high) * BM, n0 = in_band / high * BN;

    const int wb = p.k / 2, ab = WIDE ? p.k : p.k / 2, sb = p.k / 32;
    const uint8_t* w = p.w + (int64_t)n0 * wb;
    const uint8_t* a = p.a + (int64_t)m0 * ab;
    const uint8_t* ws = p.w_scales + (int64_t)n0 * sb;
    const uint8_t* as = p.a_scales + (int64_t)m0 * sb;

    // what this lane loads of a stage: the piece that belongs where its 16 bytes go
    unsigned a_off[T::LA], w_off[T::LW];
#pragma unroll
    for (int i = 0; i < T::LA; ++i) {
        const int row = min(wave * T::LA + i, T::NA - 1) * (1024 / T::RA) + lane / (T::RA / 16);
        a_off[i] = (unsigned)min(row, p.m - 1 - m0) * ab + piece_of<T::RA>(row, lane % (T::RA / 16)) * 16;
    }
#pragma unroll
    for (int i = 0; i < T::LW; ++i) {
        const int row = min(wave * T::LW + i, T::NW - 1) * (1024 / T::RW) + lane / (T::RW / 16);
        w_off[i] = (unsigned)min(row, p.n - 1 - n0) * wb + piece_of<T::RW>(row, lane % (T::RW / 16)) * 16;
    }
    // (of a last stage that is cut, lanes whose pieces are past the row's end read its first ones again: all waves have to
    // have as many loads in flight; clear_stage clears what they got)
    auto load_stage = [&](int k, uint8_t* __restrict__ to) __attribute__((always_inline)) {
        const int ak = k / (WIDE ? 1 : 2), wk = k / 2;
        if (!ALIGNED && k + KS > p.k) {
#pragma unroll
            for (int i = 0; i < T::LA; ++i) {
                const int q = min(wave * T::LA + i, T::NA - 1), row = q * (1024 / T::RA) + lane / (T::RA / 16);
                const int at = ak + piece_of<T::RA>(row, lane % (T::RA / 16)) * 16;
                load_to_lds(a + ((unsigned)min(row, p.m - 1 - m0) * ab + (at < ab ? at : 0)), to + q * 1024);
            }
#pragma unroll
            for (int i = 0; i < T::LW; ++i) {
                const int q = min(wave * T::LW + i, T::NW - 1), row = q * (1024 / T::RW) + lane / (T::RW / 16);
                const int at = wk + piece_of<T::RW>(row, lane % (T::RW / 16)) * 16;
                load_to_lds(w + ((unsigned)min(row, p.n - 1 - n0) * wb + (at < wb ? at : 0)), to + T::A_BYTES + q * 1024);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < T::LA; ++i) load_to_lds(a + ak + a_off[i], to + min(wave * T::LA + i, T::NA - 1) * 1024);
#pragma unroll
        for (int i = 0; i < T::LW; ++i) load_to_lds(w + wk + w_off[i], to + T::A_BYTES + min(wave * T::LW + i, T::NW - 1) * 1024);
    };
    auto clear_stage = [&](int k, uint8_t* stage) __attribute__((always_inline)) {
        for (int i = threadIdx.x; i < (T::A_BYTES + T::W_BYTES) / 16; i += THREADS) {
            const bool of_a = i < T::A_BYTES / 16;
            const int at = of_a ? i : i - T::A_BYTES / 16, row = at / (of_a ? T::RA / 16 : T::RW / 16);
            const int piece = of_a ? piece_of<T::RA>(row, at % (T::RA / 16)) : piece_of<T::RW>(row, at % (T::RW / 16));
            if ((of_a ? k / (WIDE ? 1 : 2) : k / 2) + piece * 16 >= (of_a ? ab : wb))
                reinterpret_cast<u4*>(stage)[i] = u4{0u, 0u, 0u, 0u};
        }
    };
    // Scales of 512 elements of every row, rows of a first: by direct loads where every row's are 16-byte aligned (ALIGNED),
    // else through registers, and put_scales waits for all loads.
    u4 sc[SPT];
    uint8_t* const scales = smem + RING * T::STAGE;
    auto row_scales = [&](int r, int k) __attribute__((always_inline)) {
        return r < BM ? as + ((unsigned)min(r, p.m - 1 - m0) * sb + k / 32)
                      : ws + ((unsigned)min(r - BM, p.n - 1 - n0) * sb + k / 32);
    };
    auto fetch_scales = [&](int k, uint8_t* __restrict__ to) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < SPT; ++i) {
            const int r0 = (wave + i * T::WAVES) * WAVE;
            if ((BM + BN) % THREADS != 0 && r0 >= BM + BN) continue;
            const int r = min(r0 + lane, BM + BN - 1);
            if constexpr (ALIGNED) {
                // (a last piece of fewer rows than lanes writes past them, into what SCALES holds for it)
                load_to_lds(row_scales(r, k), to + r0 * 16);
            } else if (k + LONG <= p.k) {
                __builtin_memcpy(&sc[i], row_scales(r, k), 16);
            } else {
                const uint8_t* from = row_scales(r, k);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sc[i][e] = 0x7f7f7f7fu;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (k + (4 * e + c) * 32 < p.k) sc[i][e] = (sc[i][e] & ~(255u << (8 * c))) | (unsigned)from[4 * e + c] << (8 * c);
                }
            }
        }
    };
    auto put_scales = [&](int half) __attribute__((always_inline)) {
        if constexpr (ALIGNED) return;
#pragma unroll
        for (int i = 0; i < SPT; ++i) {
            const int r = (wave + i * T::WAVES) * WAVE + lane;
            if (r < BM + BN) *reinterpret_cast<u4*>(scales + half * T::SCALES + r * 16) = sc[i];
        }
    };

    const int wm = wave / WN * (16 * MT), wn = wave % WN * (16 * NT);   // this wave's rows in the tile
    f4 sum[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) sum[i][j] = f4{0.0f, 0.0f, 0.0f, 0.0f};

    // Byte offsets of this lane's reads in a buffer.  Rows 16 apart are permuted alike, and the piece of a later step or half
    // differs in its bits alone: an exclusive or.
    const int r16 = lane % 16;
    const int a_base = (wm + r16) * T::RA + piece_of<T::RA>(r16, chunk_at<MODE, WIDE>(g, 0) / 16) * 16;
    const int w_base = T::A_BYTES + (wn + r16) * T::RW + piece_of<T::RW>(r16, g) * 16;
    const int as_base = (wm + r16) * 16, ws_base = (BM + wn + r16) * 16, shift = 8 * g;
    constexpr int OTHER = chunk_at<MODE, WIDE>(0, WIDE ? 1 : 0);
    auto compute = [&](const uint8_t* __restrict__ cur, const uint8_t* __restrict__ scl, int part) __attribute__((always_inline)) {
        int ab0 = a_base, wb0 = w_base, sa0 = as_base, sw0 = ws_base;
        asm volatile("" : "+v"(ab0), "+v"(wb0), "+v"(sa0), "+v"(sw0));   // (else the addresses made of them are kept)
#pragma unroll
        for (int t = 0; t < KS / 128; ++t) {
            Frag<false> wf[NT];
            int wsc[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                wf[j].v[0] = *reinterpret_cast<const u4*>(cur + (wb0 ^ (64 * t)) + j * 16 * T::RW);
                wsc[j] = *reinterpret_cast<const int*>(scl + sw0 + j * 256 + 4 * (part + t)) >> shift;
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                Frag<WIDE> af[1];
                int asc[1];
                af[0].v[0] = *reinterpret_cast<const u4*>(cur + (ab0 ^ ((WIDE ? 128 : 64) * t)) + i * 16 * T::RA);
                if constexpr (WIDE)
                    af[0].v[1] = *reinterpret_cast<const u4*>(cur + (ab0 ^ (128 * t) ^ OTHER) + i * 16 * T::RA);
                asc[0] = *reinterpret_cast<const int*>(scl + sa0 + i * 256 + 4 * (part + t)) >> shift;
                steps_of<MODE, 1, NT>(wf, wsc, af, asc, reinterpret_cast<f4(&)[1][NT]>(sum[i]));
            }
        }
    };

    // Stage i is multiplied while the RING - 1 stages after it come in.  The loads have one place in the loop, and the buffers
    // are told apart there: else the compiler would wait for all of them before it reads any.
    const int longs = (p.k + LONG - 1) / LONG, each = (longs + p.splits - 1) / p.splits, first = min((int)blockIdx.y * each, longs);
    const int stages = (min(min(first + each, longs) * LONG, p.k) - min(first * LONG, p.k) + KS - 1) / KS;
    constexpr int PER = LONG / KS, LOADS = T::LA + T::LW;
    static_assert(RING - 2 <= PER, "scales are older than the loads that a wait leaves out");
    // (scales of the next 512 elements come into the other half of their buffer, which nothing reads at that time)
    auto stage = [&](int i, const uint8_t* __restrict__ cur, uint8_t* __restrict__ next, const uint8_t* __restrict__ scl,
                     uint8_t* __restrict__ scl_next) __attribute__((always_inline)) {
        if (i >= 0) {
            if (stages - 1 - i >= RING - 2)
                wait_loads<(RING - 2) * LOADS>();
            else
                wait_loads<0>();
            __syncthreads();                       // stage i is there, and every wave is done with the buffer of stage i - 1
            if (!ALIGNED && first * LONG + (i + 1) * KS > p.k) {
                clear_stage(first * LONG + i * KS, const_cast<uint8_t*>(cur));
                __syncthreads();
            }
        }
        const int at = i + RING - 1, half = i / PER & 1, part = i % PER, more = i < 0 ? i + RING - 1 : i + PER;
        const bool fetch = (i < 0 ? i == 1 - RING : part == 0) && more < stages;
        if (fetch) fetch_scales(first * LONG + more * KS, scl_next);
        if (at < stages) load_stage(first * LONG + at * KS, next);
        if (!ALIGNED && fetch && i < 0) put_scales(0);
        if (i < 0) return;
        compute(cur, scl, part * (KS / 128));
        if (part == PER - 1 && i + 1 < stages) put_scales(half ^ 1);
    };
    int cur = 0, next = 0;
#pragma unroll 1
    for (int i = 1 - RING; i < stages; ++i) {
        const int half = i < 0 ? 1 : i / PER & 1;
        stage(i, smem + cur, smem + next, scales + half * T::SCALES, scales + (half ^ 1) * T::SCALES);
        next = next == (RING - 1) * T::STAGE ? 0 : next + T::STAGE;
        if (i >= 0) cur = cur == (RING - 1) * T::STAGE ? 0 : cur + T::STAGE;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) asm volatile("" : "+v"(sum[i][j]));
    const bool direct = p.splits > 1 ? p.n % 4 == 0 : p.vec;
    float* part = p.splits > 1 ? p.part + (int64_t)blockIdx.y * p.m * p.n : nullptr;
    if (direct) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int row = m0 + wm + 16 * i + lane % 16;
            if (row >= p.m) continue;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int col = n0 + wn + 16 * j + 4 * g;
                if (col >= p.n) continue;
                if (part)
                    *reinterpret_cast<f4*>(part + (int64_t)row * p.n + col) = sum[i][j];
                else
                    store_out4<DT>(p, row, col, sum[i][j]);
            }
        }
        return;
    }
    // Outputs whose rows are not aligned go through LDS, so that a store takes a run of a row (3952 x 6755 x 224, float32: 91
    // us with the four outputs of a lane one by one).
    constexpr int ROW = NT * 16 + 4;
    static_assert(T::WAVES * 16 * ROW * 4 <= T::LDS, "a piece of every wave");
    float* mine = reinterpret_cast<float*>(smem) + wave * 16 * ROW;
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < MT; ++i) {
#pragma unroll
        for (int k = 0; k < MT; ++k)
            if (k == i) {
#pragma unroll
                for (int j = 0; j < NT; ++j) *reinterpret_cast<f4*>(mine + r16 * ROW + 16 * j + 4 * g) = sum[k][j];
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");    // (written and read by this wave alone)
        constexpr int AT_ONCE = 4;         // (reads that do not wait for each other's stores)
#pragma unroll 1
        for (int e0 = lane; e0 < 16 * NT * 16; e0 += AT_ONCE * WAVE) {
            float v[AT_ONCE];
#pragma unroll
            for (int u = 0; u < AT_ONCE; ++u) {
                const int e = e0 + u * WAVE;
                v[u] = mine[e / (NT * 16) * ROW + e % (NT * 16)];
            }
#pragma unroll
            for (int u = 0; u < AT_ONCE; ++u) {
                const int e = e0 + u * WAVE, row = m0 + wm + 16 * i + e / (NT * 16), col = n0 + wn + e % (NT * 16);
                if (row >= p.m || col >= p.n) continue;
                if (part)
                    part[(int64_t)row * p.n + col] = v[u];
                else
                    store_out<DT>(p, row, col, v[u]);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// the splits' sums, in their order
template <int DT>
__global__ __launch_bounds__(256) void k_mx_join(ProductArgs p) {
    const int col = blockIdx.x * 256 + threadIdx.x;
    if (col >= p.n) return;
    for (int row = blockIdx.y; row < p.m; row += gridDim.y) {
        const int64_t at = (int64_t)row * p.n + col, next = (int64_t)p.m * p.n;
        float sum = p.part[at];
        for (int i = 1; i < p.splits; ++i) sum += p.part[at + i * next];
        store_out<DT>(p, row, col, sum);
    }
}

template <int MODE, int DT, int MT, int NT, int WM, int WN, int KS, int RING>
pi_status launch_many(const ProductArgs& p, hipStream_t s) {
    typedef Tile<MODE, MT, NT, WM, WN, KS, RING> T;
    const int64_t total = (int64_t)((p.m + T::BM - 1) / T::BM) * ((p.n + T::BN - 1) / T::BN);
    const dim3 grid((total + XCDS - 1) / XCDS * XCDS, p.splits), block(WAVE * WM * WN);
    if (p.k % LONG == 0) {
        auto kern = k_mx_many<MODE, DT, MT, NT, WM, WN, KS, RING, true>;
        TRY(allow_lds(kern, T::LDS));
        TRY(launch(PI_K_MX_PRODUCT, kern, grid, block, T::LDS, s, p));
    } else {
        auto kern = k_mx_many<MODE, DT, MT, NT, WM, WN, KS, RING, false>;
        TRY(allow_lds(kern, T::LDS));
        TRY(launch(PI_K_MX_PRODUCT, kern, grid, block, T::LDS, s, p));
    }
    if (p.splits == 1) return PI_OK;
    return launch(PI_K_MX_JOIN, k_mx_join<DT>, dim3((p.n + 255) / 256, std::min(p.m, 65535)), dim3(256), 0, s, p);
}

// Which form a product takes.  The chip holds one or two workgroups per unit; forms whose tiles are fewer split K so that
// each of the 256 units has one, in pieces of 1024 elements at least, and join (a launch of 4 us).  us of MXFP8 to f16, MXFP8
// to float32 and MXFP4 to f16, weights from memory, by splits (* what the rule takes):
//                       1               2               3               4               6
//   32 x 7168 x 8192    18.8 26.3 16.7  14.0 18.0 13.2* 15.3 17.1 14.4  14.7 16.7 13.8  17.2 19.8 15.1
//   48 x 7168 x 8192    28.7 43.2 24.0  19.7 27.3 17.8  17.3 23.0 15.6  15.2 18.8 14.2* 21.7 27.1 17.8
//   64 x 10240 x 8192   29.7 43.9 25.5  21.8 29.1 19.8  19.8 25.5 18.4* 26.3 33.4 22.3  26.7 31.5 23.0
//   128 x 10240 x 8192  51.0 78.2 37.6  34.7 48.5 27.5  30.3 40.7 25.2* 32.8 42.6 28.9  32.7 40.3 30.3
enum Form { WAVES_SHARE_K, TILE_16, TILE_32, TILE_64, TILE_128, TILE_WIDE };
struct ProductPlan {
    Form form;
    int splits;
};

ProductPlan plan_product(int64_t m, int64_t n, int64_t k) {
    const Form form = m <= 16 ? TILE_16 : m <= 32 ? TILE_32 : m <= 64 ? TILE_64 : TILE_128;
    const int64_t rows = form == TILE_128 ? 128 : 64, cols = form <= TILE_32 ? 64 : 128;
    const int64_t tiles = (m + rows - 1) / rows * ((n + cols - 1) / cols);
    // Tiles of 128 x 256 take four fifths of the time of two of 128 x 128, where there are enough.  us of 128 x 128 and of
    // 128 x 256, MXFP8 to f16, to float32, MXFP4: 512 x 8192 x 8192, 128 of them: 54 81 37, 75 127 66; 1024 x 8192 x 8192, 256:
    // 75 120 52, 77 129 68; 1100 x 8192 x 8192, 288: 111 177 77, 98 183 79; 4096 x 10240 x 8192: 336 566 234, 278 496 228.
    if (form == TILE_128 && (m + 127) / 128 * ((n + 255) / 256) > 256) return {TILE_WIDE, 1};
    const int64_t most = std::max<int64_t>(1, std::min(256 / tiles, k / (2 * LONG)));
    // (Every split takes as many pieces of 512, so that fewer of them may do: 5 for 16 pieces are 4 with four each.  One that
    // is left without any adds zeros that the join has to read: 256 x 1408 x 12288, 11 and 8 splits, 21.5 and 20.0 us.)
    const int64_t pieces = (k + LONG - 1) / LONG, each = (pieces + most - 1) / most, splits = (pieces + each - 1) / each;
    // Sixteen rows or fewer: one wave per 16 rows of w and eighth of K where tiles of 64 rows of w are too few, without a
    // join.  us of waves and of tiles, MXFP8 to f16, to float32, MXFP4 (K = 8192): 1 x 1024 5.9 6.1 5.8, 11.5 15.7 11.7; 1 x 4096
    // 7.0 7.5 6.1, 11.3 15.8 12.1; 1 x 8192, 128 tiles: 11.5 12.6 9.9, 11.7 16.2 12.9; 1 x 10240 14.6 16.7 14.5, 12.4 16.4 13.6.
    // (The border is MXFP8 to f16's, whose use is the widest; the other two could go to some 150 tiles.)
    if (form == TILE_16) return {tiles < 128 ? WAVES_SHARE_K : TILE_16, 1};
    return {form, (int)splits};
}

size_t product_bytes(int64_t m, int64_t n, const ProductPlan& p) {
    return p.splits > 1 ? ((size_t)p.splits * m * n * 4 + 255) / 256 * 256 : 0;
}

template <int MODE, int DT>
pi_status product(const ProductArgs& p, Form form, hipStream_t s) {
    constexpr bool FP4 = MODE == M_FP4;
    switch (form) {
        case WAVES_SHARE_K: return launch_few<MODE, DT, 8>(p, s);
        case TILE_16: return launch_many<MODE, DT, 1, 1, 1, 4, 512, 3>(p, s);
        case TILE_32: return launch_many<MODE, DT, 2, 1, 1, 4, 256, 4>(p, s);
        case TILE_64: return launch_many<MODE, DT, 2, 2, 2, 4, 256, 3>(p, s);
        case TILE_128: return launch_many<MODE, DT, 4, 4, 2, 2, FP4 ? 256 : 128, FP4 ? 2 : 3>(p, s);
        default:
            // (MXFP4, 4096 x 10240 x 8192, one run: 235 us, with 128 x 128 x 256 242, with 256 x 128 x 128 240)
            if constexpr (MODE == M_FP8_F32)
                return launch_many<MODE, DT, 8, 4, 1, 4, 128, 2>(p, s);
            else
                return launch_many<MODE, DT, 4, 8, 2, 2, 128, 2>(p, s);
    }
}

}  // namespace

extern "C" {

size_t pi_mx_product_workspace_bytes(int32_t m, int32_t n, int32_t k) {
    if (m < 0 || m > (1 << 24) || n < 0 || n > (1 << 24) || k < 32 || k > (1 << 20) || k % 32) return 0;
    if (m == 0 || n == 0) return 0;
    // (a form or a row of tiles that ends below m may split more)
    size_t need = product_bytes(m, n, plan_product(m, n, k));
    for (int64_t at : {32, 64}) need = at < m ? std::max(need, product_bytes(at, n, plan_product(at, n, k))) : need;
    for (int64_t at = 128; at < m && at <= 128 * 256; at += 128) need = std::max(need, product_bytes(at, n, plan_product(at, n, k)));
    return need;
}

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
    CHECK(((int64_t)a->rows + 127) / 128 * (((int64_t)w->rows + 127) / 128) <= 1 << 23, PI_ERR_SHAPE,
          "more than 2^23 tiles of 128 x 128");
    const ProductPlan plan = plan_product(a->rows, w->rows, a->cols);
    const size_t need = product_bytes(a->rows, w->rows, plan);
    if (need) {
        CHECK(ws, PI_ERR_WORKSPACE, "workspace is NULL");
        CHECK(aligned(ws, 256), PI_ERR_ALIGN, "workspace must be 256-byte aligned");
        CHECK(ws_bytes >= need, PI_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
    }
    const int size = dtype_size(dtype);
    const int64_t span = ((a->rows - 1) * out_stride + w->rows) * size;
    CHECK(apart(out, span, a) && apart(out, span, w) && apart(out, span, bias, (int64_t)w->rows * 4) &&
              apart(out, span, need ? ws : nullptr, need),
          PI_ERR_ARG, "out overlaps what the call reads");
    CHECK(!need || (apart(ws, need, a) && apart(ws, need, w) && apart(ws, need, bias, (int64_t)w->rows * 4)), PI_ERR_ARG,
          "the workspace overlaps what the call reads");
    const bool vec = aligned(out, 4 * size) && (a->rows == 1 || out_stride % 4 == 0);
    ProductArgs p{(const uint8_t*)a->codes, a->scales, (const uint8_t*)w->codes, w->scales, bias, (uint8_t*)out, out_stride,
                  a->rows, w->rows, a->cols, plan.splits, (float*)ws, vec};
    hipStream_t s = (hipStream_t)stream;
    const Form f = plan.form;
    if (a->format == PI_MXFP8) return dtype == PI_F16 ? product<M_FP8, F16>(p, f, s) : product<M_FP8_F32, F32>(p, f, s);
    return dtype == PI_F16 ? product<M_FP4, F16>(p, f, s) : product<M_FP4, F32>(p, f, s);
}

}  // extern "C"
