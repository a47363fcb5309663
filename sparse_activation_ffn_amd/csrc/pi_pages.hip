// pi_pages.hip -- what writes the paged cache and keeps its pages: rotary
// positions with the append of new keys and values, and the pages' bookkeeping
// (extend, fork, free, compact, copy).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "pi.h"
#include "pi_cache.h"
#include "pi_launch.h"

using namespace pi;

namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// ---- rotary positions and append ---------------------------------------------------
//
// Per token: (q_heads + kv_heads) heads turned and kv_heads value heads copied,
// 16 bytes per thread and step.  Every byte is read and written once, so the
// HBM rate bounds it (a launch, for single tokens).  The angles of a token are
// the same for all its heads: a workgroup takes one token (and a slice of its
// heads), forms each angle's sin and cos once and keeps them in LDS.
// Measured: 8192 tokens, 128 query and 8 key heads of 64 f16: 60 us, 5.0 TB/s (a
// copy of 2 GB: 4.9); 64 tokens, 64 and 8 heads of 128: 3.6 us.
constexpr int RT = 256;

struct RopeArgs {
    CacheLayer c;
    Batch b;
    const double* turns;
    const int* positions;
    const uint8_t* q;
    uint8_t* q_out;
    const uint8_t* k;
    const uint8_t* v;
    int64_t q_ts, q_hs, o_ts, o_hs, k_ts, k_hs, v_ts, v_hs;   // strides in elements
    int q_heads, rotary, layout;
    float magnitude;
};

template <int DT> struct Elem;
template <> struct Elem<F32> {
    typedef float T;
    typedef f4 V;                                 // 16 bytes
    static constexpr int N = 4;
};
template <> struct Elem<F16> {
    typedef _Float16 T;
    typedef h8 V;
    static constexpr int N = 8;
};

// How a head is cut into units of one thread:
//   PAIRS     a unit is one 16-byte chunk (its pairs lie inside it)
//   HALVES    rotary/2 a multiple of the chunk: a unit is a chunk of the first
//             half with its partner in the second, or a chunk past the rotary part
//   HALVES_1  any other rotary: a unit is up to N pairs, or up to N elements
//             past the rotary part, element by element
enum { U_PAIRS = 0, U_HALVES = 1, U_HALVES_1 = 2 };

template <int DT, int MODE>
__device__ __forceinline__ int head_units(int d, int rotary) {
    constexpr int N = Elem<DT>::N;
    if (MODE == U_PAIRS) return d / N;
    if (MODE == U_HALVES) return d / N - rotary / 2 / N;
    return (rotary / 2 + N - 1) / N + (d - rotary + N - 1) / N;
}

template <int DT, int MODE>
__device__ __forceinline__ void turn_unit(const typename Elem<DT>::T* x, typename Elem<DT>::T* y, int u, int d,
                                          int rotary, const float2* cs) {
    typedef typename Elem<DT>::T T;
    typedef typename Elem<DT>::V V;
    constexpr int N = Elem<DT>::N;
    if constexpr (MODE == U_PAIRS) {
        V a = *reinterpret_cast<const V*>(x + u * N);
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const int i = (u * N + e) / 2;
            if (2 * i < rotary) {
                const float2 t = cs[i];
                const float x0 = a[e], x1 = a[e + 1];
                a[e] = (T)(x0 * t.x - x1 * t.y);
                a[e + 1] = (T)(x1 * t.x + x0 * t.y);
            }
        }
        *reinterpret_cast<V*>(y + u * N) = a;
    } else if constexpr (MODE == U_HALVES) {
        const int half = rotary / 2, pairs = half / N;
        if (u < pairs) {
            V a = *reinterpret_cast<const V*>(x + u * N);
            V b = *reinterpret_cast<const V*>(x + half + u * N);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float2 t = cs[u * N + e];
                const float x0 = a[e], x1 = b[e];
                a[e] = (T)(x0 * t.x - x1 * t.y);
                b[e] = (T)(x1 * t.x + x0 * t.y);
            }
            *reinterpret_cast<V*>(y + u * N) = a;
            *reinterpret_cast<V*>(y + half + u * N) = b;
        } else {
            const int at = (u + pairs) * N;
            *reinterpret_cast<V*>(y + at) = *reinterpret_cast<const V*>(x + at);
        }
    } else {
        const int half = rotary / 2, pairs = (half + N - 1) / N;
        if (u < pairs) {
            for (int i = u * N; i < half && i < u * N + N; ++i) {
                const float2 t = cs[i];
                const float x0 = x[i], x1 = x[half + i];
                y[i] = (T)(x0 * t.x - x1 * t.y);
                y[half + i] = (T)(x1 * t.x + x0 * t.y);
            }
        } else {
            const int at = rotary + (u - pairs) * N;
            for (int i = at; i < d && i < at + N; ++i) y[i] = x[i];
        }
    }
}

template <int DT, int MODE>
__global__ __launch_bounds__(RT) void k_rope_append(RopeArgs a) {
    typedef typename Elem<DT>::T T;
    typedef typename Elem<DT>::V V;
    constexpr int N = Elem<DT>::N;
    __shared__ float2 cs[PI_MAX_HEAD_DIM / 2];
    const int t = blockIdx.x;
    const int s = seq_of_row(a.b, t);
    // a row of no sequence (s need not hold t: the first rows may not ascend, and pos has to stay under the length)
    if (s >= a.b.n_seqs || a.b.q_start[s] > t || a.b.q_start[s + 1] <= t) return;
    // where the token lies in the cache (a length past the table is clamped as for reading)
    const int pos = clamped_len(a.b, a.c.page_shift, s) - (a.b.q_start[s + 1] - t);
    const int turn = a.positions ? a.positions[t] : pos;
    const int half = a.rotary / 2, d = a.c.head_dim;
    if ((int)threadIdx.x < half) {
        const double full = a.turns[threadIdx.x] * (double)turn;
        float sn, cn;
        sincospif((float)(2.0 * (full - rint(full))), &sn, &cn);
        cs[threadIdx.x] = make_float2(cn * a.magnitude, sn * a.magnitude);
    }
    __syncthreads();

    int64_t slot = -1;                                        // row of head 0 in the pages
    if (pos >= 0) {
        const int page = a.b.table[(int64_t)s * a.b.table_stride + (pos >> a.c.page_shift)];
        if (page >= 0 && page < a.c.pages)
            slot = (int64_t)page * a.c.kv_heads * a.c.page_size + (pos & (a.c.page_size - 1));
    }
    const int units = head_units<DT, MODE>(d, a.rotary), chunks = d / N;
    const int n_q = a.q ? a.q_heads * units : 0, n_k = a.c.kv_heads * units;
    const int n_all = n_q + n_k + a.c.kv_heads * chunks;
    const T* q = (const T*)a.q + t * a.q_ts;
    T* q_out = (T*)a.q_out + t * a.o_ts;
    const T* k = (const T*)a.k + t * a.k_ts;
    const T* v = (const T*)a.v + t * a.v_ts;
    T* kc = (T*)a.c.k;
    T* vc = (T*)a.c.v;
    for (int i = blockIdx.y * RT + threadIdx.x; i < n_all; i += RT * gridDim.y) {
        if (i < n_q) {
            const int h = i / units, u = i - h * units;
            turn_unit<DT, MODE>(q + h * a.q_hs, q_out + h * a.o_hs, u, d, a.rotary, cs);
        } else if (slot >= 0) {
            if (i < n_q + n_k) {
                const int h = (i - n_q) / units, u = i - n_q - h * units;
                turn_unit<DT, MODE>(k + h * a.k_hs, kc + (slot + (int64_t)h * a.c.page_size) * d, u, d, a.rotary, cs);
            } else {
                const int h = (i - n_q - n_k) / chunks, u = i - n_q - n_k - h * chunks;
                *reinterpret_cast<V*>(vc + (slot + (int64_t)h * a.c.page_size) * d + u * N) =
                    *reinterpret_cast<const V*>(v + h * a.v_hs + u * N);
            }
        }
    }
}

template <int DT>
pi_status launch_rope(const RopeArgs& a, hipStream_t s) {
    constexpr int N = Elem<DT>::N;
    const int d = a.c.head_dim, chunks = d / N;
    // a token's heads over several workgroups where the tokens alone do not fill the chip
    const int64_t work = (int64_t)(a.q_heads + 2 * a.c.kv_heads) * chunks;
    const int most = (int)((work + RT - 1) / RT);
    const int want = (1024 + a.b.n_tokens - 1) / a.b.n_tokens;
    const dim3 grid(a.b.n_tokens, std::max(1, std::min({most, want, 65535})));
    const int mode = a.layout == PI_ROPE_PAIRS ? U_PAIRS : a.rotary / 2 % N == 0 ? U_HALVES : U_HALVES_1;
    if (mode == U_PAIRS) return launch(PI_K_ROPE_APPEND, k_rope_append<DT, U_PAIRS>, grid, dim3(RT), 0, s, a);
    if (mode == U_HALVES) return launch(PI_K_ROPE_APPEND, k_rope_append<DT, U_HALVES>, grid, dim3(RT), 0, s, a);
    return launch(PI_K_ROPE_APPEND, k_rope_append<DT, U_HALVES_1>, grid, dim3(RT), 0, s, a);
}

// ---- page bookkeeping ------------------------------------------------------------------

constexpr int PT = 1024;      // threads of the planning kernels (one workgroup)
constexpr int PER = 8;        // pages per thread and step of a scan over the counts

// Exclusive prefix sum over the PT threads of a workgroup; `total` is the sum.
__device__ __forceinline__ int block_excl_scan(int v, int* lds, int& total) {
    const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE;
    const int incl = wave_incl_scan(v);
    __syncthreads();                                          // lds is free again
    if (lane == WAVE - 1) lds[wave] = incl;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < PT / WAVE; ++w) {
        const int x = lds[w];
        before += w < wave ? x : 0;
        all += x;
    }
    total = all;
    return before + incl - v;
}

// The same for 64-bit values (needs, whose sums pass 32 bits).
__device__ __forceinline__ int64_t block_excl_scan64(int64_t v, int64_t* lds, int64_t& total) {
    const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE;
    int64_t incl = v;
#pragma unroll
    for (int o = 1; o < WAVE; o *= 2) {
        const int64_t x = __shfl_up(incl, o, WAVE);
        if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == WAVE - 1) lds[wave] = incl;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < PT / WAVE; ++w) {
        const int64_t x = lds[w];
        before += w < wave ? x : 0;
        all += x;
    }
    total = all;
    return before + incl - v;
}

// refs of the PER pages from p on (1 past the end: not free)
__device__ __forceinline__ void load_refs(const int* refs, int pages, int p, int r[PER]) {
    if (p + PER <= pages && reinterpret_cast<uintptr_t>(refs) % 16 == 0) {   // p is a multiple of PER
#pragma unroll
        for (int e = 0; e < PER; e += 4) {
            const u4 w = *reinterpret_cast<const u4*>(refs + p + e);
            r[e] = w.x, r[e + 1] = w.y, r[e + 2] = w.z, r[e + 3] = w.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < PER; ++e) r[e] = p + e < pages ? refs[p + e] : 1;
    }
}

// Needs, grants and page numbers of a call of pi_pages_extend, one workgroup: a
// scan over the sequences' needs, then over the counts for the lowest free
// pages, which ends as soon as enough are found; then the tables' entries.
// One workgroup because every step needs the sums of the one before; bound by
// its chain of loads (list, length, table, count): 6 to 7.5 us for 128 to 205
// sequences in pools of 10007 to 16384 pages.
__global__ __launch_bounds__(PT) void k_pages_extend(pi_page_state st, const int* seqs, const int* add, int n,
                                                     int* granted, int* copies, int* start, int* free_ids) {
    __shared__ int lds[PT / WAVE];
    __shared__ int64_t lds64[PT / WAVE];
    const int shift = 31 - __builtin_clz((unsigned)st.page_size), tid = threadIdx.x;
    // 1. needs: start[i] = sum of the needs before i, -1 where the sequence does not fit
    int64_t need_all = 0;
    for (int base = 0; base < n; base += PT) {
        const int i = base + tid;
        int need = 0, last = -1;
        bool fits = false;
        if (i < n) {
            const int s = seqs[i], a = add[i];
            if (s >= 0 && s < st.max_seqs && a >= 0) {
                const int64_t len = st.lens[s], cap = longest(st.table_stride, shift);
                if (len >= 0 && len + a <= cap) {
                    fits = true;
                    const int have = (int)((len + st.page_size - 1) >> shift);
                    const int want = (int)((len + a + st.page_size - 1) >> shift);
                    if (a > 0 && (len & (st.page_size - 1))) {
                        const int p = st.table[(int64_t)s * st.table_stride + have - 1];
                        if (p >= 0 && p < st.pages && st.refs[p] > 1) last = p;
                    }
                    need = want - have + (last >= 0);
                }
            }
        }
        int64_t total;
        const int64_t before = block_excl_scan64(need, lds64, total);
        if (i < n) {
            // a running total past the pool grants nothing more: it may stop growing there
            start[i] = fits ? (int)min(need_all + before, (int64_t)st.pages + 1) : -1;
            granted[i] = need;                                // until step 3
            copies[i] = last;
        }
        need_all = min(need_all + total, (int64_t)st.pages + 1);
    }
    // 2. the lowest free pages, as many as are needed
    int found = 0;
    for (int base = 0; base < st.pages && found < need_all; base += PT * PER) {
        int r[PER], mine = 0, total;
        const int p = base + tid * PER;
        load_refs(st.refs, st.pages, p, r);
#pragma unroll
        for (int e = 0; e < PER; ++e) mine += r[e] == 0;
        int at = found + block_excl_scan(mine, lds, total);
#pragma unroll
        for (int e = 0; e < PER; ++e)
            if (r[e] == 0) free_ids[at++] = p + e;
        found += total;
    }
    __threadfence_block();
    __syncthreads();
    // 3. grants and table entries: a thread per sequence, and the whole wave for one that takes many pages
    constexpr int FEW = 4;
    const int lane = tid % WAVE;
    for (int base = 0; base < n; base += PT) {
        const int i = base + tid;
        int s = 0, from = 0, begin = 0, need = 0;
        bool ok = false;
        if (i < n) {
            from = start[i];
            need = granted[i];
            const int last = copies[i];
            ok = from >= 0 && (int64_t)from + need <= found;
            int fresh = -1;
            if (ok) {
                s = seqs[i];
                const int len = st.lens[s];
                begin = (int)(((int64_t)len + st.page_size - 1) >> shift) - (last >= 0);
                st.lens[s] = len + add[i];
                if (last >= 0) {
                    atomicSub(&st.refs[last], 1);
                    fresh = free_ids[from];
                }
            }
            granted[i] = ok;
            copies[i] = ok ? last : -1;
            copies[n + i] = fresh;
        }
        int* row = st.table + (int64_t)s * st.table_stride;
        auto take = [&](int* row, int begin, int from, int e) {
            const int p = free_ids[from + e];
            // (a sequence named twice may have any length by now)
            if ((unsigned)(begin + e) < (unsigned)st.table_stride) row[begin + e] = p;
            st.refs[p] = 1;
        };
        if (ok && need <= FEW)
            for (int e = 0; e < need; ++e) take(row, begin, from, e);
        for (uint64_t many = __ballot(ok && need > FEW); many; many &= many - 1) {
            const int k = __builtin_ctzll(many);
            int* r = st.table + (int64_t)__shfl(s, k, WAVE) * st.table_stride;
            const int b0 = __shfl(begin, k, WAVE), f0 = __shfl(from, k, WAVE), m = __shfl(need, k, WAVE);
            for (int e = lane; e < m; e += WAVE) take(r, b0, f0, e);
        }
    }
}

// Page copies: pair i (src, dst) of every layer, k and v.  A page of one layer is
// one contiguous block; a workgroup takes pieces of it of COPY_BYTES.  Bound by
// HBM: 47 MB read and written in 8.4 us, 420 MB in 87 us (4.8 TB/s).
constexpr int CT = 256;
constexpr int COPY_BYTES = CT * 16 * 4;

struct CopyArgs {
    uint8_t* k;
    uint8_t* v;
    const int* src;
    const int* dst;
    const int* count;        // device count of pairs, or NULL: n
    int n, layers, pages;
    int64_t page_bytes;
};

__device__ void copy_pages(const CopyArgs& a, int block, int blocks) {
    const int n = a.count ? min(*a.count, a.n) : a.n;
    const int pieces = (int)((a.page_bytes + COPY_BYTES - 1) / COPY_BYTES);
    const int64_t per_pair = (int64_t)a.layers * 2 * pieces;
    for (int64_t i = block; i < n * per_pair; i += blocks) {
        const int pair = (int)(i / per_pair), rest = (int)(i - pair * per_pair);
        const int s = a.src[pair], d = a.dst[pair];
        if (s < 0 || s >= a.pages || d < 0 || d >= a.pages || s == d) continue;
        const int piece = rest % pieces, lk = rest / pieces;
        uint8_t* base = lk & 1 ? a.v : a.k;
        const int64_t layer = (int64_t)(lk >> 1) * a.pages, off = (int64_t)piece * COPY_BYTES;
        const u4* from = (const u4*)(base + (layer + s) * a.page_bytes + off);
        u4* to = (u4*)(base + (layer + d) * a.page_bytes + off);
        const int n16 = (int)(min((int64_t)COPY_BYTES, a.page_bytes - off) / 16);
        u4 x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if ((int)threadIdx.x + e * CT < n16) x[e] = from[threadIdx.x + e * CT];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if ((int)threadIdx.x + e * CT < n16) to[threadIdx.x + e * CT] = x[e];
    }
}

__global__ __launch_bounds__(CT) void k_page_copy(CopyArgs a) { copy_pages(a, blockIdx.x, gridDim.x); }

// Fork, first kernel: what every src was, into the workspace; its pages gain a name.
__global__ __launch_bounds__(CT) void k_fork_read(pi_page_state st, const int* src, const int* dst, int* rows,
                                                  int* lens) {
    const int i = blockIdx.x, s = src[i], d = dst[i];
    const bool ok = s >= 0 && s < st.max_seqs && d >= 0 && d < st.max_seqs;
    if (threadIdx.x == 0) lens[i] = ok ? st.lens[s] : 0;
    if (!ok) return;
    for (int e = threadIdx.x; e < st.table_stride; e += CT) {
        const int p = st.table[(int64_t)s * st.table_stride + e];
        rows[(int64_t)i * st.table_stride + e] = p;
        if (p >= 0 && p < st.pages) atomicAdd(&st.refs[p], 1);
    }
}

// Second: dst's old pages lose one, and its row becomes src's.
__global__ __launch_bounds__(CT) void k_fork_write(pi_page_state st, const int* src, const int* dst, const int* rows,
                                                   const int* lens) {
    const int i = blockIdx.x, s = src[i], d = dst[i];
    if (s < 0 || s >= st.max_seqs || d < 0 || d >= st.max_seqs) return;
    if (threadIdx.x == 0) st.lens[d] = lens[i];
    for (int e = threadIdx.x; e < st.table_stride; e += CT) {
        int* at = &st.table[(int64_t)d * st.table_stride + e];
        const int p = *at;
        if (p >= 0 && p < st.pages) atomicSub(&st.refs[p], 1);
        *at = rows[(int64_t)i * st.table_stride + e];
    }
}

__global__ __launch_bounds__(CT) void k_pages_free(pi_page_state st, const int* seqs) {
    const int s = seqs[blockIdx.x];
    if (s < 0 || s >= st.max_seqs) return;
    if (threadIdx.x == 0) st.lens[s] = 0;
    for (int e = threadIdx.x; e < st.table_stride; e += CT) {
        int* at = &st.table[(int64_t)s * st.table_stride + e];
        const int p = *at;
        if (p >= 0 && p < st.pages) atomicSub(&st.refs[p], 1);
        *at = -1;
    }
}

// Plan of a compaction, one workgroup: the number of pages in use, the free ids
// below it (dst) and the pages in use from it on (src), both ascending; the
// counts follow at once, the tables and the pages in k_pages_move.
__global__ __launch_bounds__(PT) void k_compact_plan(pi_page_state st, int* moved, int* count, int* src, int* dst) {
    __shared__ int lds[PT / WAVE];
    const int tid = threadIdx.x;
    int live = 0;
    for (int base = 0; base < st.pages; base += PT * PER) {
        int r[PER];
        load_refs(st.refs, st.pages, base + tid * PER, r);
#pragma unroll
        for (int e = 0; e < PER; ++e) live += base + tid * PER + e < st.pages && r[e] > 0;
    }
    int total;
    block_excl_scan(live, lds, total);
    live = total;
    int holes = 0, movers = 0;
    for (int base = 0; base < st.pages; base += PT * PER) {
        int r[PER], h = 0, m = 0;
        const int p = base + tid * PER;
        load_refs(st.refs, st.pages, p, r);
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            h += p + e < live && r[e] <= 0;
            m += p + e >= live && p + e < st.pages && r[e] > 0;
        }
        int th, tm;
        int ah = holes + block_excl_scan(h, lds, th), am = movers + block_excl_scan(m, lds, tm);
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            if (p + e >= st.pages) break;
            if (r[e] <= 0 && p + e < live) dst[ah++] = p + e;
            if (r[e] > 0 && p + e >= live) src[am++] = p + e;
            moved[p + e] = r[e] > 0 ? p + e : -1;
        }
        holes += th;
        movers += tm;
    }
    __threadfence_block();
    __syncthreads();
    // as many holes below `live` as pages in use above it
    for (int i = tid; i < movers; i += PT) {
        const int a = src[i], b = dst[i];
        moved[a] = b;
        st.refs[b] = st.refs[a];
        st.refs[a] = 0;
    }
    if (tid == 0) *count = movers;
}

// The tables' entries (the first `remap` workgroups) and the pages themselves.
__global__ __launch_bounds__(CT) void k_pages_move(pi_page_state st, const int* moved, CopyArgs a, int remap) {
    if ((int)blockIdx.x < remap) {
        const int64_t all = (int64_t)st.max_seqs * st.table_stride;
        for (int64_t e = (int64_t)blockIdx.x * CT + threadIdx.x; e < all; e += (int64_t)remap * CT) {
            const int p = st.table[e];
            if (p >= 0 && p < st.pages) st.table[e] = moved[p];
        }
    } else if (a.k) {
        copy_pages(a, blockIdx.x - remap, gridDim.x - remap);
    }
}

pi_status check_state(const pi_page_state* st) {
    CHECK(st, PI_ERR_ARG, "NULL page state");
    CHECK(st->pages >= 1 && st->pages <= (1 << 24), PI_ERR_SHAPE, "state: pages must be in 1..2^24");
    CHECK(st->max_seqs >= 1 && st->max_seqs <= (1 << 20) && st->table_stride >= 1 && st->table_stride <= (1 << 24),
          PI_ERR_SHAPE, "state: max_seqs must be in 1..2^20 and table_stride in 1..2^24");
    CHECK(page_size_ok(st->page_size), PI_ERR_SHAPE, "state: page_size must be a power of two in 8..%d",
          (int)PI_MAX_PAGE_SIZE);
    CHECK(st->refs && st->table && st->lens, PI_ERR_ARG, "state: refs, table and lens are required");
    CHECK(aligned(st->refs, 4) && aligned(st->table, 4) && aligned(st->lens, 4), PI_ERR_ALIGN,
          "state: refs, table and lens must be 4-byte aligned");
    return PI_OK;
}

pi_status check_state_cache(const pi_page_state* st, const pi_kv_cache* c) {
    TRY(check_cache(c));
    CHECK(c->pages == st->pages && c->page_size == st->page_size, PI_ERR_SHAPE,
          "cache (%d pages of %d) and page state (%d pages of %d) differ", c->pages, c->page_size, st->pages,
          st->page_size);
    return PI_OK;
}

pi_status check_list(const pi_page_state* st, int n, const void* a, const void* b) {
    CHECK(n >= 0 && n <= st->max_seqs, PI_ERR_SHAPE, "n must be in 0..max_seqs");
    CHECK(n == 0 || (a && b), PI_ERR_ARG, "lists are required");
    CHECK(aligned(a, 4) && aligned(b, 4), PI_ERR_ALIGN, "lists must be 4-byte aligned");
    return PI_OK;
}

pi_status check_pages_ws(const pi_page_state* st, int n, const void* ws, size_t bytes) {
    const size_t need = pi_pages_workspace_bytes(st, n);
    CHECK(ws, PI_ERR_WORKSPACE, "workspace is NULL");
    CHECK(aligned(ws, 256), PI_ERR_ALIGN, "workspace must be 256-byte aligned");
    CHECK(bytes >= need, PI_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", bytes, need);
    return PI_OK;
}

CopyArgs copy_args(const pi_kv_cache* c, const int* src, const int* dst, const int* count, int n) {
    CopyArgs a{};
    a.src = src;
    a.dst = dst;
    a.count = count;
    a.n = n;
    if (!c) return a;
    a.k = (uint8_t*)c->k;
    a.v = (uint8_t*)c->v;
    a.layers = c->layers;
    a.pages = c->pages;
    a.page_bytes = layer_bytes(c) / c->pages;
    return a;
}

// workgroups for up to n pairs: at most eight per compute unit, each looping
int copy_grid(const CopyArgs& a) {
    const int64_t pieces = (a.page_bytes + COPY_BYTES - 1) / COPY_BYTES;
    return (int)std::min<int64_t>(2048, std::max<int64_t>(1, (int64_t)a.n * a.layers * 2 * pieces));
}

}  // namespace

extern "C" {

pi_status pi_rope_turns(int32_t rotary_dim, double base, int32_t scaling, double factor, double low, double high,
                        double context, double* turns) {
    CHECK(rotary_dim >= 0 && rotary_dim <= PI_MAX_HEAD_DIM && rotary_dim % 2 == 0, PI_ERR_SHAPE,
          "rotary_dim must be even and in 0..%d", (int)PI_MAX_HEAD_DIM);
    CHECK(scaling >= PI_SCALE_NONE && scaling <= PI_SCALE_BANDS, PI_ERR_ARG, "unknown scaling");
    CHECK(base > 1.0 && std::isfinite(base), PI_ERR_ARG, "base must be finite and > 1");
    CHECK(scaling == PI_SCALE_NONE || (factor >= 1.0 && std::isfinite(factor)), PI_ERR_ARG,
          "factor must be finite and >= 1");
    CHECK(scaling != PI_SCALE_BANDS || (low < high && std::isfinite(low) && std::isfinite(high) && context > 0.0 &&
                                        std::isfinite(context)),
          PI_ERR_ARG, "bands need low < high and a positive context");
    CHECK(rotary_dim == 0 || turns, PI_ERR_ARG, "turns is required");
    const double tau = 6.283185307179586476925286766559;
    if (scaling == PI_SCALE_BASE && rotary_dim > 2) base *= std::pow(factor, (double)rotary_dim / (rotary_dim - 2));
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rotary_dim);
        if (scaling == PI_SCALE_LINEAR) {
            f /= factor;
        } else if (scaling == PI_SCALE_BANDS) {
            const double w = std::min(1.0, std::max(0.0, (context * f / tau - low) / (high - low)));
            f = w * f + (1.0 - w) * f / factor;
        }
        turns[i] = f / tau;
    }
    return PI_OK;
}

pi_status pi_rope_append(const pi_kv_cache* cache, int32_t layer, const pi_seq_batch* batch, const pi_rope* rope,
                         const int32_t* positions, int32_t q_heads, const pi_rows* q, const pi_rows* q_out,
                         const pi_rows* k, const pi_rows* v, void* stream) {
    TRY(check_layer(cache, layer));
    TRY(check_batch(batch));
    CHECK(rope, PI_ERR_ARG, "NULL rope");
    CHECK(rope->rotary_dim >= 0 && rope->rotary_dim <= cache->head_dim && rope->rotary_dim % 2 == 0, PI_ERR_SHAPE,
          "rope: rotary_dim must be even and in 0..head_dim");
    CHECK(rope->layout == PI_ROPE_HALVES || rope->layout == PI_ROPE_PAIRS, PI_ERR_ARG, "rope: unknown layout");
    CHECK(rope->rotary_dim == 0 || rope->turns, PI_ERR_ARG, "rope: turns is required");
    CHECK(aligned(rope->turns, 8) && aligned(positions, 4), PI_ERR_ALIGN,
          "rope: turns must be 8-byte, positions 4-byte aligned");
    const bool with_q = (q && q->data) || (q_out && q_out->data);
    CHECK(q_heads >= 0 && q_heads <= 65535 && (q_heads >= 1 || !with_q), PI_ERR_SHAPE, "q_heads must be in 1..65535");
    if (batch->n_seqs == 0 || batch->n_tokens == 0) return PI_OK;
    if (with_q) {
        TRY(check_rows(q, "q", cache->dtype));
        TRY(check_rows(q_out, "q_out", cache->dtype));
    }
    TRY(check_rows(k, "k", cache->dtype));
    TRY(check_rows(v, "v", cache->dtype));
    RopeArgs a{};
    a.c = cache_layer(cache, layer);
    a.b = seq_batch(batch);
    a.turns = rope->turns;
    a.positions = positions;
    if (with_q) {
        a.q = (const uint8_t*)q->data;
        a.q_out = (uint8_t*)q_out->data;
        a.q_ts = q->token_stride;
        a.q_hs = q->head_stride;
        a.o_ts = q_out->token_stride;
        a.o_hs = q_out->head_stride;
        a.q_heads = q_heads;
    }
    a.k = (const uint8_t*)k->data;
    a.v = (const uint8_t*)v->data;
    a.k_ts = k->token_stride;
    a.k_hs = k->head_stride;
    a.v_ts = v->token_stride;
    a.v_hs = v->head_stride;
    a.rotary = rope->rotary_dim;
    a.layout = rope->layout;
    a.magnitude = rope->magnitude;
    return cache->dtype == PI_F32 ? launch_rope<F32>(a, (hipStream_t)stream) : launch_rope<F16>(a, (hipStream_t)stream);
}

size_t pi_pages_workspace_bytes(const pi_page_state* st, int32_t n) {
    if (!st || st->pages < 1 || st->pages > (1 << 24) || st->max_seqs < 1 || st->max_seqs > (1 << 20) ||
        st->table_stride < 1 || st->table_stride > (1 << 24) || n < 0 || n > st->max_seqs)
        return 0;
    const size_t pages = align256((size_t)st->pages * 4), list = align256((size_t)n * 4);
    const size_t extend = list + pages;                                  // starts, free pages
    const size_t fork = list + (size_t)n * st->table_stride * 4;         // lengths, rows
    const size_t compact = 256 + 2 * pages;                              // count, from, to
    return std::max({extend, align256(fork), compact});
}

pi_status pi_pages_extend(const pi_page_state* st, const pi_kv_cache* cache, const int32_t* seqs, const int32_t* add,
                          int32_t n, int32_t* granted, int32_t* copies, void* ws, size_t ws_bytes, void* stream) {
    TRY(check_state(st));
    if (cache) TRY(check_state_cache(st, cache));
    TRY(check_list(st, n, seqs, add));
    TRY(check_list(st, n, granted, copies));
    TRY(check_pages_ws(st, n, ws, ws_bytes));
    if (n == 0) return PI_OK;
    hipStream_t s = (hipStream_t)stream;
    int* start = (int*)ws;
    int* free_ids = (int*)((uint8_t*)ws + align256((size_t)n * 4));
    TRY(launch(PI_K_PAGES, k_pages_extend, dim3(1), dim3(PT), 0, s, *st, seqs, add, (int)n, granted, copies, start,
               free_ids));
    if (!cache) return PI_OK;
    const CopyArgs a = copy_args(cache, copies, copies + n, nullptr, n);
    return launch(PI_K_PAGE_COPY, k_page_copy, dim3(copy_grid(a)), dim3(CT), 0, s, a);
}

pi_status pi_pages_fork(const pi_page_state* st, const int32_t* src, const int32_t* dst, int32_t n, void* ws,
                        size_t ws_bytes, void* stream) {
    TRY(check_state(st));
    TRY(check_list(st, n, src, dst));
    TRY(check_pages_ws(st, n, ws, ws_bytes));
    if (n == 0) return PI_OK;
    hipStream_t s = (hipStream_t)stream;
    int* lens = (int*)ws;
    int* rows = (int*)((uint8_t*)ws + align256((size_t)n * 4));
    TRY(launch(PI_K_PAGES, k_fork_read, dim3(n), dim3(CT), 0, s, *st, src, dst, rows, lens));
    return launch(PI_K_PAGES, k_fork_write, dim3(n), dim3(CT), 0, s, *st, src, dst, (const int*)rows,
                  (const int*)lens);
}

pi_status pi_pages_free(const pi_page_state* st, const int32_t* seqs, int32_t n, void* stream) {
    TRY(check_state(st));
    TRY(check_list(st, n, seqs, seqs));
    if (n == 0) return PI_OK;
    return launch(PI_K_PAGES, k_pages_free, dim3(n), dim3(CT), 0, (hipStream_t)stream, *st, seqs);
}

pi_status pi_pages_compact(const pi_page_state* st, const pi_kv_cache* cache, int32_t* moved, void* ws,
                           size_t ws_bytes, void* stream) {
    TRY(check_state(st));
    if (cache) TRY(check_state_cache(st, cache));
    CHECK(moved, PI_ERR_ARG, "moved is required");
    CHECK(aligned(moved, 4), PI_ERR_ALIGN, "moved must be 4-byte aligned");
    TRY(check_pages_ws(st, 0, ws, ws_bytes));
    hipStream_t s = (hipStream_t)stream;
    int* count = (int*)ws;
    int* src = (int*)((uint8_t*)ws + 256);
    int* dst = (int*)((uint8_t*)ws + 256 + align256((size_t)st->pages * 4));
    TRY(launch(PI_K_PAGES, k_compact_plan, dim3(1), dim3(PT), 0, s, *st, moved, count, src, dst));
    const CopyArgs a = copy_args(cache, src, dst, count, st->pages / 2);
    const int64_t entries = (int64_t)st->max_seqs * st->table_stride;
    const int remap = (int)std::min<int64_t>(256, (entries + CT - 1) / CT);
    return launch(PI_K_PAGE_COPY, k_pages_move, dim3(remap + (cache ? copy_grid(a) : 0)), dim3(CT), 0, s, *st,
                  (const int*)moved, a, remap);
}

pi_status pi_pages_copy(const pi_kv_cache* cache, const int32_t* src, const int32_t* dst, int32_t n, void* stream) {
    TRY(check_cache(cache));
    CHECK(n >= 0, PI_ERR_SHAPE, "n must be >= 0");
    if (n == 0) return PI_OK;
    CHECK(src && dst, PI_ERR_ARG, "src and dst are required");
    CHECK(aligned(src, 4) && aligned(dst, 4), PI_ERR_ALIGN, "src and dst must be 4-byte aligned");
    const CopyArgs a = copy_args(cache, src, dst, nullptr, n);
    return launch(PI_K_PAGE_COPY, k_page_copy, dim3(copy_grid(a)), dim3(CT), 0, (hipStream_t)stream, a);
}

}  // extern "C"
