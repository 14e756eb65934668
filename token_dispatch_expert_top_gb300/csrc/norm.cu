// norm.cu -- root-mean-square norm with the residual's addition, and its gradient:
//   s = x + residual (rounded to x's type, the residual stream),  r = 1 / sqrt(mean(s^2) + eps)
//   y = s r w,  and its MXFP8 copy by the layer's own block rule
//   gradient, with h = s r and g = dy w:  dx = dsum + r (g - h mean(g h)),  dw = sum over rows of dy h
// Everything between loads and stores is FP32; y, s and dx are rounded once.  Both are bound by HBM: a row is
// read once, its sum formed, and the row written, with a rows-long queue of copies ahead of the sums.
//   8192 x 7168 BF16, residual, MXFP8 copy   82 us (6.4 TB/s)      gradient, 16384 x 7168 BF16, dsum  149 us (6.3 TB/s)
//   8192 x 7161 BF16, residual               76 us (6.2 TB/s)      gradient, 8192 x 7161 BF16, dsum   100 us (4.7 TB/s)
//   8192 x 7168 BF16                         41 us (5.7 TB/s)      gradient, 16384 x 7168 BF16        126 us (5.6 TB/s)
//   131072 x 128 BF16                        12 us (5.4 TB/s)      gradient, 8192 x 7168 FP32, dsum   141 us (6.7 TB/s)
//   4096 x 16384 BF16, residual             108 us (5.0 TB/s)      gradient, 4096 x 16384 BF16, dsum  145 us (3.7 TB/s)
//
// Three ways, by the rows: through shared memory (below: up to 8192 columns, up to 65536 where rows are
// aligned); in registers, up to 8192 or 16384 columns, what the first does not take (matrices other than BF16 whose
// rows begin at different elements of eight, few rows that begin anywhere, MXFP8 copies of such rows); all others, read
// twice.  The latter two deal a row in chunks of 256 columns per warp: aligned, lane l has columns 8l .. 8l+7; otherwise
// columns l, l+32, ..., so that the lanes touch neighbouring elements.  Always a block of 32 columns (one MXFP8
// scale) lies within a warp.
#include <float.h>

#include "kernels.cuh"
#include "pieces.cuh"
#include "vec_io.cuh"

namespace moe {
namespace {

// A row whose mean square and eps overflow FP32 is summed again with its elements at this scale (and eps at its
// square); elements up to FP32's largest then square to at most 2^96.
constexpr float kDown = 0x1p-80f;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the threads of a row: one warp, or the whole block (`part`: 32 floats of its shared
// memory that no earlier sum still reads).  Every thread gets the same bits.
template <bool WARP_ROW>
__device__ __forceinline__ float row_sum(float v, float* part) {
    v = warp_sum(v);
    if constexpr (WARP_ROW) return v;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    if (lane == 0) part[warp] = v;
    __syncthreads();
    return warp_sum(lane < warps ? part[lane] : 0.f);
}

// This lane's elements of the 256 columns from c0 on: VEC, columns 8 lane + i; otherwise columns lane + 32 i.
template <typename T, bool VEC>
__device__ __forceinline__ void load_chunk(const T* row, int64_t c0, int64_t cols, int lane, float (&v)[8]) {
    if constexpr (VEC) {
        const int64_t c = c0 + lane * 8;
        if (c < cols) {
            load8<T, true>(row + c, 8, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t c = c0 + i * 32 + lane;
            v[i] = c < cols ? to_f32<T>(row[c]) : 0.f;
        }
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_chunk(T* row, int64_t c0, int64_t cols, int lane, const float (&v)[8]) {
    if constexpr (VEC) {
        const int64_t c = c0 + lane * 8;
        if (c < cols) store8<T, true>(row + c, 8, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t c = c0 + i * 32 + lane;
            if (c < cols) row[c] = from_f32<T>(v[i]);
        }
    }
}

// The weights of a chunk in either type; without any, ones.
template <bool VEC>
__device__ __forceinline__ void load_weight(const void* w, int w_dtype, int64_t c0, int64_t cols, int lane,
                                            float (&v)[8]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 1.f;
    } else if (w_dtype == MOE_F32) {
        load_chunk<float, VEC>((const float*)w, c0, cols, lane, v);
    } else {
        load_chunk<uint16_t, VEC>((const uint16_t*)w, c0, cols, lane, v);
    }
}

// The MXFP8 codes of the eight columns from c on, and their block's scale (four lanes have a block).
__device__ __forceinline__ void store_mx8(uint8_t* codes, uint8_t* scales, int64_t c, bool in, int lane,
                                          const float (&v)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if (!in) return;
    const int s = mx_scale_exponent(m);
    const float inv = mx_inv_scale(s);
    uint2 q;
    q.x = cvt_e4m3x2(v[0] * inv, v[1] * inv) | (uint32_t)cvt_e4m3x2(v[2] * inv, v[3] * inv) << 16;
    q.y = cvt_e4m3x2(v[4] * inv, v[5] * inv) | (uint32_t)cvt_e4m3x2(v[6] * inv, v[7] * inv) << 16;
    *reinterpret_cast<uint2*>(codes + c) = q;
    if (lane % 4 == 0) scales[c / 32] = (uint8_t)(s + 127);
}

// The MXFP8 codes and scales of a chunk of a row of the output, as it is rounded.
template <bool VEC>
__device__ __forceinline__ void store_mx_chunk(uint8_t* codes, uint8_t* scales, int64_t c0, int64_t cols, int lane,
                                               const float (&v)[8]) {
    if constexpr (VEC) {
        store_mx8(codes, scales, c0 + lane * 8, c0 + lane * 8 < cols, lane, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (c0 + i * 32 >= cols) break;                 // rows are whole blocks
            // a NaN has no part in the block's maximum
            const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fabsf(v[i]), 0.f)));
            const int s = mx_scale_exponent(__uint_as_float(m));
            codes[c0 + i * 32 + lane] = (uint8_t)cvt_e4m3x2(v[i] * mx_inv_scale(s), 0.f);
            if (lane == 0) scales[c0 / 32 + i] = (uint8_t)(s + 127);
        }
    }
}

// As the type rounds it, again in FP32.
template <typename T>
__device__ __forceinline__ void round_to(float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32<T>(from_f32<T>(v[i]));
}

// ------------------------------------------------------------- rows through shared memory
// Persistent blocks whose threads each own P pieces of E columns of a row, up to 8192; a row
// belongs to a team of warps (or, where fewer lanes suffice, several rows to a warp).  E is 16 bytes of
// the widest type, so that lanes touch whole neighbouring sectors.  Every thread copies its own pieces of
// the rows to come into its own places of shared memory (cp.async), STAGES rows ahead, so that no thread
// waits for another's copy and loads do not pause for a row's sum.
// ODD: rows that begin anywhere, as those of an odd number of columns do, but in all matrices at the same
// element of E.  Pieces then begin `shift` columns before the row, at the aligned place; its first and
// last piece are masked.  A thread's rows are a multiple of E apart, so that its shift is the same for
// all of them and its weights and sums stay in registers.
// SHIFTED: BF16 rows that begin so in what is written, and anywhere else in what is read: a thread copies the two
// aligned pieces that hold its own, and shifts it out of them (8091 x 7168 in rows of 7169: 65 us, by single elements
// 100; gradient with dsum 186, 230; 139423 x 416 66 and 87, gradient 181 and 282.  Words of four bytes, one more than
// the piece has, in place of the second piece: 68 and 198, 74 and 185).
// WIDE: aligned rows of more columns, by a cluster of two to eight blocks, `share` columns each, which write
// their sums into each other's shared memory; bound by the cluster's barrier (read twice by one block, which
// needs none, 16384 columns took 165 us and their gradient 299).
enum RowKind { kGroups, kOdd, kShifted, kWide };
constexpr int kRingCols = 8192, kMostBlocks = 8;
struct RowTeams {
    int team_warps, lanes;      // lanes: 32 with more than one warp to a row
    int cluster, share;         // kWide: blocks of a row and columns of a block
    int blocks;                 // that walk the rows; those behind them have a job of their own
};

struct RowPlace {
    int lane, warp, team;
    uint32_t at, width;         // this thread's number in its row's team, threads of a row
    uint32_t base, sub, step;   // first row of the warp's, this lane's row among them, stride
    uint32_t rank;              // kWide: of this block in its cluster
};

template <RowKind KIND>
__device__ __forceinline__ RowPlace row_place(const RowTeams& t) {
    RowPlace p;
    if constexpr (KIND == kWide) {                          // a block is one team
        p.lane = threadIdx.x % 32, p.warp = threadIdx.x / 32, p.team = 0, p.sub = 0;
        p.at = threadIdx.x, p.width = blockDim.x;
        p.base = blockIdx.x / t.cluster, p.step = t.blocks / t.cluster;
        p.rank = cluster_ctarank();
        return p;
    }
    p.rank = 0;
    p.lane = threadIdx.x % 32, p.warp = threadIdx.x / 32;
    p.team = p.warp / t.team_warps;
    const int rows = 32 / t.lanes, teams = blockDim.x / 32 / t.team_warps;
    p.sub = p.lane / t.lanes;
    p.at = (p.warp - p.team * t.team_warps) * t.lanes + p.lane % t.lanes;
    p.width = t.team_warps * t.lanes;
    p.base = (blockIdx.x * teams + p.team) * rows;
    p.step = t.blocks * teams * rows;
    return p;
}

// Sum over a row's threads; `turn` alternates between calls, and part[2][32] is the block's.  At most
// 15 teams of several warps: each has a barrier of its own, number team + 1.
template <RowKind KIND>
__device__ __forceinline__ float team_sum(float v, const RowTeams& t, const RowPlace& p, float (*part)[32], int turn) {
    if (t.team_warps == 1) {
        if (t.lanes == 32) v += __shfl_xor_sync(0xffffffffu, v, 16);
        if (t.lanes >= 16) v += __shfl_xor_sync(0xffffffffu, v, 8);
#pragma unroll
        for (int o = 4; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);    // eight lanes at least
        return v;
    }
    v = warp_sum(v);
    if (p.lane == 0) part[turn & 1][p.warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(p.team + 1), "r"(t.team_warps * 32) : "memory");
    if constexpr (KIND == kWide) {
        __shared__ float blocks[2][kMostBlocks];
        if (p.warp == 0) {
            v = warp_sum(p.lane < t.team_warps ? part[turn & 1][p.lane] : 0.f);
            if (p.lane < t.cluster) st_cluster_f32(&blocks[turn & 1][p.rank], p.lane, v);
        }
        cluster_sync();
        v = blocks[turn & 1][0];
        for (int i = 1; i < t.cluster; ++i) v += blocks[turn & 1][i];
        return v;
    }
    return warp_sum(p.lane < t.team_warps ? part[turn & 1][p.team * t.team_warps + p.lane] : 0.f);
}

// A thread's places in the ring: `stage` bytes from one row to the next; piece number u of a row's
// tensors lies `unit` bytes behind the one before it (16 bytes a thread, whatever the piece's size).
struct Ring {
    uint32_t at, stage, unit;   // at: this thread's first place, a shared-memory address
};
__device__ __forceinline__ Ring ring_place(uint4* ring, int units) {
    return {smem_u32(ring) + threadIdx.x * 16, units * blockDim.x * 16, blockDim.x * 16};
}
// `bytes` of the piece, zeros behind them.
template <typename T, int E>
__device__ __forceinline__ void ring_copy(const Ring& g, uint32_t offset, int u, const void* src, uint32_t bytes) {
    constexpr uint32_t kBytes = E * sizeof(T);
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(g.at + offset + u * g.unit), "l"(src),
                     "r"(bytes)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(g.at + offset + u * g.unit), "l"(src),
                     "r"(bytes)
                     : "memory");
}
// A piece that may begin before the matrix: its elements from `first` to `last`, one by one, to shared memory.
template <typename T, int E>
__device__ __noinline__ void ring_patch(uint32_t at, const T* src, int first, int last) {
    Piece<T, E> r;
#pragma unroll
    for (int i = 0; i < Piece<T, E>::kWords; ++i) r.w[i] = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        if (i < first || i >= last) continue;
        if constexpr (sizeof(T) == 2) r.w[i / 2] |= (uint32_t)src[i] << (16 * (i % 2));
        else r.w[i] = __float_as_uint(src[i]);
    }
#pragma unroll
    for (int i = 0; i < Piece<T, E>::kWords; ++i)
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + 4 * i), "r"(r.w[i]) : "memory");
}
template <typename T, int E>
__device__ __forceinline__ Piece<T, E> ring_read(const Ring& g, uint32_t offset, int u) {
    Piece<T, E> r;
    const uint32_t at = g.at + offset + u * g.unit;
    if constexpr (Piece<T, E>::kWords == 4)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                     : "r"(at) : "memory");
    else
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "r"(at) : "memory");
    return r;
}

// Columns c .. c + E - 1 of a row, of which first .. last - 1 are in it.
struct Span {
    int c, first, last;
};
template <bool ODD, int E>
__device__ __forceinline__ Span span_at(int c, int cols) {
    if (!ODD) return {c, 0, c < cols ? E : 0};
    return {c, c < 0 ? -c : 0, cols - c < E ? cols - c : E};
}
template <bool ODD, int E>
__device__ __forceinline__ bool whole(const Span& s) {
    return ODD ? s.first == 0 && s.last == E : s.last > 0;
}
// Fetches a piece of row r, or zeros.  What lies before a row is the end of the row before it; only for
// the first E rows the aligned place may lie before the matrix, and ring_patch brings those pieces.
template <bool ODD, int E>
__device__ __forceinline__ bool patched(const Span& s, uint32_t r) {
    return ODD && s.first > 0 && r < E;
}
template <bool ODD, typename T, int E>
__device__ __forceinline__ void ring_fetch(const Ring& g, uint32_t offset, int u, const uint8_t* src, const Span& s,
                                           uint32_t r, bool live) {
    if (patched<ODD, E>(s, r)) return;
    ring_copy<T, E>(g, offset, u, src, live && s.last > 0 ? (ODD ? s.last : E) * (uint32_t)sizeof(T) : 0);
}
// What lies before the row is not its own.
template <bool ODD, typename T, int E>
__device__ __forceinline__ Piece<T, E> ring_take(const Ring& g, uint32_t offset, int u, const Span& s) {
    Piece<T, E> r = ring_read<T, E>(g, offset, u);
    if (ODD && s.first > 0) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if constexpr (sizeof(T) == 2) r.w[i / 2] &= i < s.first ? (i % 2 ? 0xFFFFu : 0xFFFF0000u) : 0xFFFFFFFFu;
            else r.w[i] = i < s.first ? 0u : r.w[i];
        }
    }
    return r;
}

// SHIFTED (BF16): the two aligned pieces that hold a piece lie in two places of the ring, one unit apart; it
// begins `skip` elements behind the first one's beginning.
__device__ __forceinline__ int pieces_skip(const uint8_t* src) { return (int)((uintptr_t)src >> 1 & 7); }
// Fetches a piece of row r, from 8 on, or zeros.  It may begin up to 14 elements before the row: in the matrix,
// whose rows are two elements apart or more.
__device__ __forceinline__ void pieces_fetch(const Ring& g, uint32_t offset, int u, const uint8_t* src, const Span& s,
                                             int skip, uint32_t r, bool live) {
    if (r < 8) return;
    const int last = live && s.last > s.first ? s.last + skip : 0;   // up to the row's last element
    const uint8_t* low = (const uint8_t*)((uintptr_t)src & ~(uintptr_t)15);
    ring_copy<uint16_t, 8>(g, offset, u, low, 2 * min(last, 8));
    ring_copy<uint16_t, 8>(g, offset, u + 1, low + 16, 2 * max(last - 8, 0));
}
// The same of the first rows, element by element.
__device__ __noinline__ void pieces_first(uint32_t at, uint32_t unit, const uint8_t* src, Span s, int skip, bool live) {
    for (int k = 0; k < 16; ++k) {
        const int i = k - skip;
        const uint16_t x = live && i >= s.first && i < s.last ? ((const uint16_t*)src)[i] : 0;
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + (k < 8 ? 0 : unit) + 2 * (k % 8)), "h"(x) : "memory");
    }
}
__device__ __forceinline__ Piece<uint16_t, 8> pieces_take(const Ring& g, uint32_t offset, int u, const Span& s,
                                                          int skip) {
    const Piece<uint16_t, 8> low = ring_read<uint16_t, 8>(g, offset, u), high = ring_read<uint16_t, 8>(g, offset, u + 1);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = low.w[i], w[4 + i] = high.w[i];
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = skip & 4 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = skip & 2 ? w[i + 1] : w[i];
    Piece<uint16_t, 8> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.w[i] = __funnelshift_r(w[i], w[i + 1], 16 * (skip & 1));
        if (s.first > 0)
            r.w[i] &= (2 * i < s.first ? 0u : 0xFFFFu) | (2 * i + 1 < s.first ? 0u : 0xFFFF0000u);
    }
    return r;
}

template <RowKind KIND, typename T, int E>
__device__ __forceinline__ Piece<T, E> taken(const Ring& g, uint32_t offset, int u, const Span& s, int skip) {
    if constexpr (KIND == kShifted) return pieces_take(g, offset, u, s, skip);
    else return ring_take<KIND == kOdd, T, E>(g, offset, u, s);
}

template <bool ODD, typename T, int E>
__device__ __forceinline__ void store_span(uint8_t* place, const Span& s, const Piece<T, E>& r) {
    T* to = (T*)place;
    if (whole<ODD, E>(s)) {
        store_piece<T, E>(to, r);
    } else if (ODD) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (i < s.first || i >= s.last) continue;
            if constexpr (sizeof(T) == 2) to[i] = (uint16_t)(r.w[i / 2] >> (16 * (i % 2)));
            else to[i] = __uint_as_float(r.w[i]);
        }
    }
}
// Its weights; ones without any.
template <int E>
__device__ __forceinline__ void load_weights(const void* w, int w_dtype, const Span& s, F2* v) {
    float f[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        f[i] = 1.f;
        if (w && i >= s.first && i < s.last)
            f[i] = w_dtype == MOE_F32 ? ((const float*)w)[s.c + i] : bf16_to_f32(((const uint16_t*)w)[s.c + i]);
    }
#pragma unroll
    for (int i = 0; i < E / 2; ++i) v[i] = f2(f[2 * i], f[2 * i + 1]);
}

// MXFP8 codes of a piece as the output type holds it, and its block's scale (32 / E lanes have a
// block); NaN has no part in the block's maximum.
template <typename T, int E>
__device__ __forceinline__ void store_mx_piece(uint8_t* codes, uint8_t* scale, bool in, const Piece<T, E>& r) {
    F2 v[E / 2];
    to_pairs(r, v);
    float f[E], amax;
    if constexpr (sizeof(T) == 2) {
        uint32_t m = r.w[0] & 0x7FFF7FFFu;
#pragma unroll
        for (int i = 1; i < E / 2; ++i) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(r.w[i] & 0x7FFF7FFFu));
#pragma unroll
        for (int o = 1; o < 32 / E; o *= 2) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, m, o);
            asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(other));
        }
        amax = fmaxf(fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u)), 0.f);
    } else {
        amax = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) amax = fmaxf(amax, fabsf(__uint_as_float(r.w[i])));
#pragma unroll
        for (int o = 1; o < 32 / E; o *= 2) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    }
    if (!in) return;
    const int s = mx_scale_exponent(amax);
    const float inv = mx_inv_scale(s);
    const F2 by = f2(inv, inv);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) f2_split(f2_mul(v[i], by), f[2 * i], f[2 * i + 1]);
    uint32_t q[E / 4];
#pragma unroll
    for (int i = 0; i < E / 4; ++i)
        q[i] = cvt_e4m3x2(f[4 * i], f[4 * i + 1]) | (uint32_t)cvt_e4m3x2(f[4 * i + 2], f[4 * i + 3]) << 16;
    if constexpr (E == 8) *reinterpret_cast<uint2*>(codes) = make_uint2(q[0], q[1]);
    else *reinterpret_cast<uint32_t*>(codes) = q[0];
    if (threadIdx.x % (32 / E) == 0) *scale = (uint8_t)(s + 127);
}

__device__ __forceinline__ float pair_sum(F2 v) {
    float a, b;
    f2_split(v, a, b);
    return a + b;
}

// 1 / sqrt(x) for x from 1e-30 up, 0 for infinity: the approximate root and one Newton step.
__device__ __forceinline__ float inv_root(float x) {
    const float r = rsqrtf(x);
    const float better = fmaf(0.5f * r, fmaf(-x * r, r, 1.f), r);
    return r == 0.f ? 0.f : better;
}

// Row r of a matrix whose rows are `stride` bytes apart.
__device__ __forceinline__ const uint8_t* row_at(const uint8_t* p, uint32_t r, uint32_t stride) {
    return p + (uint64_t)r * stride;
}
__device__ __forceinline__ uint8_t* row_at(uint8_t* p, uint32_t r, uint32_t stride) { return p + (uint64_t)r * stride; }

struct RowStrides {
    uint32_t in[3], out[2];     // bytes
    uint32_t shift, turn;       // ODD: columns that row 0 begins behind an aligned place, and how many more per row
};

// RES: with a residual.  (Asked for again at run time: without that the compiler's order of the instructions costs
// such rows up to 3%.)
template <typename T, typename TO, RowKind KIND, bool RES, int STAGES>
__global__ void __launch_bounds__(1024)
    rms_norm_ring_kernel(const __grid_constant__ RmsNormCall a, const __grid_constant__ RowStrides ld, RowTeams t) {
    extern __shared__ uint4 ring_memory[];
    __shared__ float part[2][32];
    constexpr int E = sizeof(T) == 4 || sizeof(TO) == 4 ? 4 : 8, H = E / 2, P = 8 / E;
    constexpr bool ODD = KIND == kOdd || KIND == kShifted, SHIFTED = KIND == kShifted;
    constexpr int U = SHIFTED ? 2 : 1;                      // places of a piece
    if constexpr (KIND == kWide) cluster_sync();            // every block of it is there to be written to
    grid_dependency_wait();
    const RowPlace p = row_place<KIND>(t);
    const bool residual = RES && a.residual != nullptr;
    const Ring ring = ring_place(ring_memory, residual ? 2 * P * U : P * U);
    const uint32_t rows = (uint32_t)a.rows, cols = (uint32_t)a.cols, end = STAGES * ring.stage;
    const uint32_t shift = ODD ? (ld.shift + (p.base + p.sub) * ld.turn) % E : 0;
    // this block's columns
    const uint32_t from = KIND == kWide ? p.rank * t.share : 0, to = KIND == kWide ? min(cols, from + t.share) : cols;
    Span at[P];
#pragma unroll
    for (int k = 0; k < P; ++k) at[k] = span_at<ODD, E>((int)(from + (p.at + k * p.width) * E - shift), (int)to);
    const uint32_t next = p.width * E;                      // columns from one piece to the next
    const uint8_t* x = (const uint8_t*)((const T*)a.x + at[0].c);
    const uint8_t* res = (const uint8_t*)((const T*)a.residual + at[0].c);
    uint8_t *sum_out = (uint8_t*)((T*)a.sum + at[0].c), *out = (uint8_t*)((TO*)a.out + at[0].c);
    const int x_skip = pieces_skip(row_at(x, p.base + p.sub, ld.in[0]));   // SHIFTED, where P is 1
    const int res_skip = pieces_skip(row_at(res, p.base + p.sub, ld.in[1]));
    uint32_t far = p.base, put = 0;                         // the rows fetched next
    auto fetch = [&]() {
        if (far < rows) {
            const uint32_t r = far + p.sub;
            const uint8_t *xr = row_at(x, r, ld.in[0]), *rr = row_at(res, r, ld.in[1]);
#pragma unroll
            for (int k = 0; k < P; ++k) {
                if constexpr (SHIFTED) {
                    pieces_fetch(ring, put, 0, xr, at[0], x_skip, r, r < rows);
                    if (residual) pieces_fetch(ring, put, 2, rr, at[0], res_skip, r, r < rows);
                    continue;
                }
                ring_fetch<ODD, T, E>(ring, put, k, xr + k * next * sizeof(T), at[k], r, r < rows);
                if (residual) ring_fetch<ODD, T, E>(ring, put, P + k, rr + k * next * sizeof(T), at[k], r, r < rows);
            }
        }
        cp_async_commit();
        far += p.step;
        put = put + ring.stage == end ? 0 : put + ring.stage;
    };
#pragma unroll
    for (int k = 0; k < STAGES; ++k) fetch();
    if constexpr (SHIFTED) {
        if (const uint32_t r = p.base + p.sub; r < 8) {
            pieces_first(ring.at, ring.unit, row_at(x, r, ld.in[0]), at[0], x_skip, r < rows);
            if (residual)
                pieces_first(ring.at + 2 * ring.unit, ring.unit, row_at(res, r, ld.in[1]), at[0], res_skip, r < rows);
        }
    } else if (const uint32_t r = p.base + p.sub; patched<ODD, E>(at[0], r)) {
        const int last = r < rows ? at[0].last : 0;
        ring_patch<T, E>(ring.at, (const T*)row_at(x, r, ld.in[0]), at[0].first, last);
        if (residual) ring_patch<T, E>(ring.at + P * ring.unit, (const T*)row_at(res, r, ld.in[1]), at[0].first, last);
    }

    F2 w[P][H];
#pragma unroll
    for (int k = 0; k < P; ++k) load_weights<E>(a.weight, a.w_dtype, at[k], w[k]);
    // 1 / cols and what its rounding leaves: the mean of every row would be off the same way
    const float inv_cols = 1.f / (float)a.cols, inv_rest = fmaf(-inv_cols, (float)a.cols, 1.f) * inv_cols;
    const bool keeper = a.rstd && p.at == 0 && p.rank == 0;
    uint32_t r = p.base + p.sub, get = 0;
    int turn = 0;
    for (uint32_t base = p.base; base < rows; base += p.step) {
        const bool live = r < rows;
        cp_async_wait<STAGES - 1>();
        F2 v[P][H], squares = f2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < P; ++k) {
            Piece<T, E> s = taken<KIND, T, E>(ring, get, k * U, at[k], x_skip);
            if (residual) {
                s = add_pieces<T, E>(s, taken<KIND, T, E>(ring, get, (P + k) * U, at[k], res_skip));
                if (live) store_span<ODD, T, E>(row_at(sum_out, r, ld.out[0]) + k * next * sizeof(T), at[k], s);
            }
            to_pairs(s, v[k]);
#pragma unroll
            for (int i = 0; i < H; ++i) squares = f2_fma(v[k][i], v[k][i], squares);
        }
        get = get + ring.stage == end ? 0 : get + ring.stage;
        float sum = team_sum<KIND>(pair_sum(squares), t, p, part, turn++);
        fetch();
        auto mean_square = [&](float sum, float eps) {
            return fmaf(sum, inv_cols, fmaf(fminf(sum, FLT_MAX), inv_rest, eps));
        };
        float mean = mean_square(sum, a.eps), down = 1.f;
        if (__any_sync(0xffffffffu, mean == INFINITY)) {    // the whole team, or other rows of the warp
            const F2 by = f2(kDown, kDown);
            squares = f2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < P; ++k)
#pragma unroll
                for (int i = 0; i < H; ++i) squares = f2_fma(f2_mul(v[k][i], by), f2_mul(v[k][i], by), squares);
            sum = team_sum<KIND>(pair_sum(squares), t, p, part, turn++);
            if (mean == INFINITY) {
                down = inv_root(mean_square(sum, a.eps * kDown * kDown));
                // at most 2^92 with an element; in one factor a subnormal number
#pragma unroll
                for (int k = 0; k < P; ++k)
#pragma unroll
                    for (int i = 0; i < H; ++i) v[k][i] = f2_mul(f2_mul(v[k][i], f2(down, down)), by);
                down *= kDown, mean = 1.f;
            }
        }
        const float rstd = inv_root(mean);
        if (keeper && live) a.rstd[r] = rstd * down;
        const F2 by = f2(rstd, rstd);
#pragma unroll
        for (int k = 0; k < P; ++k) {
#pragma unroll
            for (int i = 0; i < H; ++i) v[k][i] = f2_mul(f2_mul(v[k][i], by), w[k][i]);
            const Piece<TO, E> y = from_pairs<TO, E>(v[k]);
            if (a.out && live) store_span<ODD, TO, E>(row_at(out, r, ld.out[1]) + k * next * sizeof(TO), at[k], y);
            if (KIND != kOdd && a.codes)                      // SHIFTED: only where `out` is aligned
                store_mx_piece<TO, E>(row_at(a.codes, r, cols) + at[k].c, row_at(a.scales, r, cols / 32) + at[k].c / 32,
                                      live && at[k].last > 0, y);
        }
        r += p.step;
    }
}

// Rows of other types than BF16 whose matrices begin at different elements, few rows that begin anywhere, and MXFP8
// copies of rows that are not aligned: one row by one warp (WARP_ROW, four rows to a block) or by a block, its
// elements in registers, up to CHUNKS chunks per warp.  Bound by the instructions of single-element accesses: 4045 x
// 7168 FP32 in rows of 7169 48 us (aligned 39), BF16 of twice as many rows 100 (65 through shared memory).
template <typename T, int CHUNKS, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? 128 : CHUNKS == 4 ? 512 : 1024)
    rms_norm_kernel(const __grid_constant__ RmsNormCall a) {
    __shared__ float part[2][32];
    grid_dependency_wait();
    const int lane = threadIdx.x % 32, warps = WARP_ROW ? 1 : blockDim.x / 32;
    const int warp = WARP_ROW ? 0 : threadIdx.x / 32;
    const int64_t r = WARP_ROW ? (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.x;
    if (r >= a.rows) return;
    float v[CHUNKS][8];
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < CHUNKS; ++j)
        load_chunk<T, false>((const T*)a.x + r * a.ld_x, (int64_t)(j * warps + warp) * 256, a.cols, lane, v[j]);
    if (a.residual) {
        float q[CHUNKS][8];
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j)
            load_chunk<T, false>((const T*)a.residual + r * a.ld_res, (int64_t)(j * warps + warp) * 256, a.cols, lane,
                                 q[j]);
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] += q[j][i];
            round_to<T>(v[j]);
            store_chunk<T, false>((T*)a.sum + r * a.ld_sum, (int64_t)(j * warps + warp) * 256, a.cols, lane, v[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < CHUNKS; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(v[j][i], v[j][i], sum);
    sum = row_sum<WARP_ROW>(sum, part[0]);
    float down = 1.f, mean = sum / (float)a.cols + a.eps;
    if (isinf(mean)) {
        down = kDown, sum = 0.f;
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(v[j][i] * kDown, v[j][i] * kDown, sum);
        mean = row_sum<WARP_ROW>(sum, part[1]) / (float)a.cols + a.eps * kDown * kDown;
    }
    float rstd = inv_root(mean);
    if (a.rstd && warp == 0 && lane == 0) a.rstd[r] = rstd * down;
    if (down != 1.f) {                                      // one after the other, as above
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * rstd * kDown;
        rstd = 1.f;
    }
#pragma unroll
    for (int j = 0; j < CHUNKS; ++j) {
        const int64_t c0 = (int64_t)(j * warps + warp) * 256;
        if (c0 >= a.cols) break;
        float w[8];
        load_weight<false>(a.weight, a.w_dtype, c0, a.cols, lane, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * rstd * w[i];
        if (a.out_dtype == MOE_F32) {
            if (a.out) store_chunk<float, false>((float*)a.out + r * a.ld_out, c0, a.cols, lane, v[j]);
        } else {
            round_to<uint16_t>(v[j]);
            if (a.out) store_chunk<uint16_t, false>((uint16_t*)a.out + r * a.ld_out, c0, a.cols, lane, v[j]);
        }
        if (a.codes)
            store_mx_chunk<false>(a.codes + r * a.cols, a.scales + r * (a.cols / 32), c0, a.cols, lane, v[j]);
    }
}

// Rows of any length, by a block of 1024 threads: the row is read twice, the second time what the
// first pass left (the sum, or x), mostly in L2 by then.  1024 x 65544 BF16 with a residual 151 us
// (3.6 TB/s), 4096 x 16385 185 (2.9 TB/s; single-element accesses).
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) rms_norm_long_kernel(const __grid_constant__ RmsNormCall a) {
    __shared__ float part[2][32];
    grid_dependency_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t r = blockIdx.x;
    const T* x = (const T*)a.x + r * a.ld_x;
    const T* s = a.residual ? (const T*)a.sum + r * a.ld_sum : x;
    float sum = 0.f;
    for (int64_t c0 = warp * 256; c0 < a.cols; c0 += 32 * 256) {
        float v[8], q[8];
        load_chunk<T, VEC>(x, c0, a.cols, lane, v);
        if (a.residual) {
            load_chunk<T, VEC>((const T*)a.residual + r * a.ld_res, c0, a.cols, lane, q);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += q[i];
            round_to<T>(v);
            store_chunk<T, VEC>((T*)a.sum + r * a.ld_sum, c0, a.cols, lane, v);
        }
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t = fmaf(v[i], v[i], t);
        sum += t;
    }
    sum = row_sum<false>(sum, part[0]);
    float down = 1.f, mean = sum / (float)a.cols + a.eps;
    if (isinf(mean)) {
        down = kDown, sum = 0.f;
        for (int64_t c0 = warp * 256; c0 < a.cols; c0 += 32 * 256) {
            float v[8];
            load_chunk<T, VEC>(s, c0, a.cols, lane, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(v[i] * kDown, v[i] * kDown, sum);
        }
        mean = row_sum<false>(sum, part[1]) / (float)a.cols + a.eps * kDown * kDown;
    }
    const float rstd = inv_root(mean);
    if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd * down;
    for (int64_t c0 = warp * 256; c0 < a.cols; c0 += 32 * 256) {
        float v[8], w[8];
        load_chunk<T, VEC>(s, c0, a.cols, lane, v);
        load_weight<VEC>(a.weight, a.w_dtype, c0, a.cols, lane, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * rstd * down * w[i];
        if (a.out_dtype == MOE_F32) {
            if (a.out) store_chunk<float, VEC>((float*)a.out + r * a.ld_out, c0, a.cols, lane, v);
        } else {
            round_to<uint16_t>(v);
            if (a.out) store_chunk<uint16_t, VEC>((uint16_t*)a.out + r * a.ld_out, c0, a.cols, lane, v);
        }
        if (a.codes) store_mx_chunk<VEC>(a.codes + r * a.cols, a.scales + r * (a.cols / 32), c0, a.cols, lane, v);
    }
}

// Threads of a block and its teams for rows of `cols` columns; blocks for `rows` of them.
struct RowGrid {
    RowTeams teams;
    int threads;
    int64_t blocks;
    bool one_row;               // at most one row (of each warp's) to a team
};
inline RowGrid row_grid(int64_t rows, int64_t cols, int columns, int64_t most_blocks) {
    RowGrid g{};
    g.teams.cluster = 1;
    const int threads = (int)((cols + columns - 1) / columns);   // that a row needs
    g.teams.team_warps = (threads + 31) / 32;
    g.teams.lanes = 32;
    while (g.teams.lanes > 8 && g.teams.lanes / 2 >= threads) g.teams.lanes /= 2;
    int teams = 32 / g.teams.team_warps;
    if (g.teams.team_warps > 1 && teams > 15) teams = 15;
    const int64_t per = 32 / g.teams.lanes;
    // few rows: on as many SMs as there are
    while (teams > 1 && (rows + per * teams - 1) / (per * teams) < most_blocks) teams = (teams + 1) / 2;
    g.threads = teams * g.teams.team_warps * 32;
    g.blocks = (rows + per * teams - 1) / (per * teams);
    g.one_row = g.blocks <= most_blocks;
    // a multiple of eight: a thread's rows then begin at the same element of eight (152 SMs are one)
    if (!g.one_row) g.blocks = most_blocks >= 8 ? most_blocks / 8 * 8 : most_blocks;
    g.teams.blocks = (int)g.blocks;
    return g;
}

// Launches a kernel on a ring of `stages` rows of `stage` bytes.  Where every team has one row only, one stage
// is all it touches; up to 48 KB with the kernel's own arrays need no attribute, whose call costs the host
// about a microsecond.  It asks for the most that any call has, so that calls of several host threads
// ask for the same.
constexpr int kRingMost = 192 * 1024;   // 1024 threads, two stages of six 16-byte pieces
template <typename... Params, typename... Args>
cudaError_t launch_ring(void (*k)(Params...), const RowGrid& g, size_t stage, int stages, cudaStream_t stream,
                        const Args&... args) {
    const size_t smem = g.one_row ? stage : stage * stages;
    if (smem > 47 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingMost);
        if (e != cudaSuccess) return e;
    }
    return launch_after(k, g.blocks, g.threads, smem, g.teams.cluster, stream, args..., g.teams);
}

// Clusters for rows of more than kRingCols columns: as many as fit the GPU at a time.
template <typename... Params>
RowGrid wide_grid(void (*k)(Params...), int64_t rows, int64_t cols, size_t stage_of_thread, int stages, cudaError_t& e) {
    RowGrid g{};
    g.teams.lanes = 32;
    g.teams.cluster = (int)((cols + kRingCols - 1) / kRingCols);
    g.teams.share = (int)((cols + g.teams.cluster - 1) / g.teams.cluster + 31) / 32 * 32;
    g.threads = (g.teams.share / 8 + 31) / 32 * 32;
    g.teams.team_warps = g.threads / 32;
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingMost);
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)g.teams.cluster, at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)g.teams.cluster), cfg.blockDim = dim3((unsigned)g.threads);
    cfg.dynamicSmemBytes = stage_of_thread * g.threads * stages, cfg.attrs = &at, cfg.numAttrs = 1;
    int most = 0;
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&most, k, &cfg);
    if (e == cudaSuccess && most < 1) e = cudaErrorInvalidConfiguration;
    g.one_row = rows <= most;
    g.blocks = (g.one_row ? rows : most) * g.teams.cluster;
    g.teams.blocks = (int)g.blocks;
    return g;
}

// The matrices of a call as these kernels see them: row strides in bytes, and the element of E that rows begin
// at, which has to be the same in all of them.
struct RowCheck {
    int E;
    bool ok = true, odd = false, any = false;
    uint32_t shift = 0, turn = 0;
    uint32_t stride(const void* p, int64_t ld, size_t size) {
        if (!p) return 0;
        const uint32_t begin = (uint32_t)((uintptr_t)p / size % E), more = (uint32_t)(ld % E);
        if (any && (begin != shift || more != turn)) ok = false;
        any = true, shift = begin, turn = more;
        odd = odd || begin || more;
        if (ld > 0x3fffffff) ok = false;
        return (uint32_t)(ld * size);
    }
    bool takes(int64_t cols) const { return ok && cols + (odd || cols % 8 ? E - 1 : 0) <= kRingCols; }
    bool takes_wide(int64_t cols) const { return ok && !odd && cols % 8 == 0 && cols <= kMostBlocks * kRingCols; }
};

// So few rows that begin anywhere are quicker in registers, a block to each: 400 x 1409 BF16 2.6 us (2.9 through
// shared memory), 777 rows 4.5 (4.1); FP32 1600 x 1409 5.4 (5.7), 3200 rows 9.2 (8.5).  The gradient goes by the same
// rule, which is too low for it: 400 rows 5.9 us (6.5), 777 rows, which go through shared memory, 7.0 (8.8); FP32
// 1600 rows 9.7 (11.9), 3200 rows 19.9 (17.2).
template <int E>
bool few_rows(int64_t rows, int64_t cols) {
    return rows * cols < (E == 8 ? 1 << 20 : 5 << 19);
}

template <typename T, typename TO>
bool launch_rms_norm_ring(const RmsNormCall& c, cudaStream_t stream, cudaError_t& e) {
    constexpr int E = sizeof(T) == 4 || sizeof(TO) == 4 ? 4 : 8, P = 8 / E;
    RowCheck check{E};
    RowStrides ld{};
    ld.in[0] = check.stride(c.x, c.ld_x, sizeof(T)), ld.in[1] = check.stride(c.residual, c.ld_res, sizeof(T));
    ld.out[0] = check.stride(c.sum, c.ld_sum, sizeof(T)), ld.out[1] = check.stride(c.out, c.ld_out, sizeof(TO));
    ld.shift = check.shift, ld.turn = check.turn;
    const bool odd = check.odd || c.cols % E;
    if (c.codes && (uintptr_t)c.codes % 8) return false;
    if (!check.ok || (c.codes && odd)) {
        if constexpr (P == 1) {                             // by what is written
            RowCheck x{E}, residual{E}, written{E};
            x.stride(c.x, c.ld_x, sizeof(T)), residual.stride(c.residual, c.ld_res, sizeof(T));
            written.stride(c.sum, c.ld_sum, sizeof(T)), written.stride(c.out, c.ld_out, sizeof(TO));
            const RowGrid g = row_grid(c.rows, c.cols + E - 1, 8, c.num_sms);
            if (few_rows<E>(c.rows, c.cols) || !x.ok || !residual.ok || !written.ok || c.cols < 2 ||
                c.cols + E - 1 > kRingCols || (c.codes && written.odd) || (!g.one_row && g.blocks % 8))
                return false;
            ld.shift = written.shift, ld.turn = written.turn;
            const size_t stage = (size_t)g.threads * 32 * (c.residual ? 2 : 1);
            e = c.residual ? launch_ring(rms_norm_ring_kernel<T, TO, kShifted, true, 2>, g, stage, 2, stream, c, ld)
                           : launch_ring(rms_norm_ring_kernel<T, TO, kShifted, false, 4>, g, stage, 4, stream, c, ld);
            return true;
        }
        return false;
    }
    if (c.cols > kRingCols && check.takes_wide(c.cols)) {
        const size_t stage = 16 * P * (c.residual ? 2 : 1);
        auto go = [&](auto k) {
            const RowGrid g = wide_grid(k, c.rows, c.cols, stage, 2, e);
            if (e == cudaSuccess) e = launch_ring(k, g, stage * g.threads, 2, stream, c, ld);
        };
        if (c.residual) go(rms_norm_ring_kernel<T, TO, kWide, true, 2>);
        else go(rms_norm_ring_kernel<T, TO, kWide, false, 2>);
        return true;
    }
    if (!check.takes(c.cols)) return false;
    const RowGrid g = row_grid(c.rows, c.cols + (odd ? E - 1 : 0), 8, c.num_sms);
    if (odd && ((!g.one_row && g.blocks % 8) || few_rows<E>(c.rows, c.cols))) return false;
    const size_t stage = (size_t)g.threads * 16 * P * (c.residual ? 2 : 1);
    // The rows ahead: as many as 64 KB in flight hold, but two at least, and four at most; more take memory time
    // from the writes.  BF16 with a residual and codes: 8192 x 7168 83 us with two rows, 93 with three or four;
    // 13942 x 4160 92 with two, 82 with three.  Without a residual 8192 x 7168 46 with two, 42 with three or four; FP32
    // 7211 x 4160 46 with two, 40 with three; where a warp has several rows and writes codes too, 453125 x 128
    // 47 with two, 51 with four.
    const size_t row = (size_t)g.threads * 8 * sizeof(T) * (c.residual ? 2 : 1), most = 64 * 1024;
#define MOE_RING(RES, STAGES)                                                                                     \
    (odd ? launch_ring(rms_norm_ring_kernel<T, TO, kOdd, RES, STAGES>, g, stage, STAGES, stream, c, ld)            \
         : launch_ring(rms_norm_ring_kernel<T, TO, kGroups, RES, STAGES>, g, stage, STAGES, stream, c, ld))
    if (c.residual) e = 3 * row <= most ? MOE_RING(true, 3) : MOE_RING(true, 2);
    else if (sizeof(T) == 4) e = 3 * row <= most ? MOE_RING(false, 3) : MOE_RING(false, 2);
    else e = g.teams.team_warps == 1 && c.codes ? MOE_RING(false, 2) : MOE_RING(false, sizeof(T) == 2 ? 4 : 2);
#undef MOE_RING
    return true;
}

// Rows that the ring does not take, by the registers that hold them.
template <typename T>
cudaError_t launch_rms_norm_odd(const RmsNormCall& c, cudaStream_t stream) {
    const int64_t chunks = (c.cols + 255) / 256;
    if (chunks <= 2) {
        const int64_t blocks = (c.rows + 3) / 4;
        return chunks == 1 ? launch_after(rms_norm_kernel<T, 1, true>, blocks, 128, 0, 1, stream, c)
                           : launch_after(rms_norm_kernel<T, 2, true>, blocks, 128, 0, 1, stream, c);
    }
    if (chunks > 64) return launch_after(rms_norm_long_kernel<T, false>, c.rows, 1024, 0, 1, stream, c);
    // few rows: the most threads; many: the most loads in flight per thread
    const int per = c.rows >= 4 * c.num_sms ? 4 : chunks <= 32 ? 1 : 2;
    const int threads = (int)((chunks + per - 1) / per) * 32;
    return per == 1   ? launch_after(rms_norm_kernel<T, 1, false>, c.rows, threads, 0, 1, stream, c)
           : per == 2 ? launch_after(rms_norm_kernel<T, 2, false>, c.rows, threads, 0, 1, stream, c)
                      : launch_after(rms_norm_kernel<T, 4, false>, c.rows, threads, 0, 1, stream, c);
}

template <typename T>
cudaError_t launch_rms_norm_rows(const RmsNormCall& c, bool vec, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    if (c.out_dtype == MOE_F32 ? launch_rms_norm_ring<T, float>(c, stream, e)
                               : launch_rms_norm_ring<T, uint16_t>(c, stream, e))
        return e;
    if (!vec) return launch_rms_norm_odd<T>(c, stream);
    return launch_after(rms_norm_long_kernel<T, true>, c.rows, 1024, 0, 1, stream, c);
}

// ------------------------------------------------------------------ gradient
constexpr int kGradStages = 2, kFewParts = 304;

// Rows of other types than BF16 whose matrices begin at different elements, and few rows that begin anywhere:
// blocks walk the rows; each keeps the weight gradient of its rows in registers and leaves it in row blockIdx.x
// of `part`.  A row belongs to a warp (WARP_ROW) or to the block.
template <typename T, typename TG, int CHUNKS, bool WARP_ROW>
__global__ void __launch_bounds__(512, CHUNKS == 1 ? 2 : 1)
    rms_norm_grad_kernel(const __grid_constant__ RmsNormGradCall a) {
    __shared__ float part[2][32];
    extern __shared__ float joint[];                        // WARP_ROW: [warps][CHUNKS * 256]
    grid_dependency_wait();
    const int lane = threadIdx.x % 32, all = blockDim.x / 32, warps = WARP_ROW ? 1 : all;
    const int warp = WARP_ROW ? 0 : threadIdx.x / 32;
    const int64_t first = WARP_ROW ? (int64_t)blockIdx.x * all + threadIdx.x / 32 : blockIdx.x;
    const int64_t step = (int64_t)gridDim.x * (WARP_ROW ? all : 1);
    float w[CHUNKS][8], dw[CHUNKS][8];
#pragma unroll
    for (int j = 0; j < CHUNKS; ++j) {
        load_weight<false>(a.weight, a.w_dtype, (int64_t)(j * warps + warp) * 256, a.cols, lane, w[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
    }
    const float inv_cols = 1.f / (float)a.cols;
    int turn = 0;
    for (int64_t r = first; r < a.rows; r += step, ++turn) {
        float h[CHUNKS][8], g[CHUNKS][8], d[CHUNKS][8] = {};
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j) {
            const int64_t c0 = (int64_t)(j * warps + warp) * 256;
            load_chunk<T, false>((const T*)a.s + r * a.ld_s, c0, a.cols, lane, h[j]);
            load_chunk<TG, false>((const TG*)a.dout + r * a.ld_dout, c0, a.cols, lane, g[j]);
            if (a.dsum) load_chunk<T, false>((const T*)a.dsum + r * a.ld_dsum, c0, a.cols, lane, d[j]);
        }
        const float rstd = a.rstd[r];
        float c = 0.f;
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[j][i] *= rstd;
                dw[j][i] = fmaf(g[j][i], h[j][i], dw[j][i]);
                g[j][i] *= w[j][i];
                c = fmaf(g[j][i], h[j][i], c);
            }
        c = row_sum<WARP_ROW>(c, part[turn & 1]) * inv_cols;
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j) {
            const int64_t c0 = (int64_t)(j * warps + warp) * 256;
            if (c0 >= a.cols) break;
#pragma unroll
            for (int i = 0; i < 8; ++i) d[j][i] = fmaf(rstd, fmaf(-h[j][i], c, g[j][i]), d[j][i]);
            store_chunk<T, false>((T*)a.dx + r * a.ld_dx, c0, a.cols, lane, d[j]);
        }
    }
    if (!a.dweight) return;
    float* mine = a.part + (int64_t)blockIdx.x * a.cols;
    if constexpr (WARP_ROW) {
        float* row = joint + threadIdx.x / 32 * (CHUNKS * 256);
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) row[j * 256 + i * 32 + lane] = dw[j][i];
        __syncthreads();
        for (int64_t c = threadIdx.x; c < a.cols; c += blockDim.x) {
            float t = 0.f;
            for (int k = 0; k < all; ++k) t += joint[k * (CHUNKS * 256) + c];
            mine[c] = t;
        }
    } else {
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t c = (int64_t)(j * warps + warp) * 256 + i * 32 + lane;
                if (c < a.cols) mine[c] = dw[j][i];
            }
    }
}

// The weight gradient of 32 q columns by one block, for rows that its warps read in one round of kDirectRows
// each: beside the blocks that walk the rows in the same launch, it reads them again (from L2) and needs
// neither partial sums nor a kernel to join them (64 x 7168 BF16: 3.7 us, 8.4 with those; a second round costs
// more than they do: 256 rows 10.9 against 9.7).
constexpr int kDirectRows = 4, kDirectColumns = 4;

template <typename T, typename TG>
__device__ __noinline__ void weight_grad_block(const RmsNormGradCall& a, const RowStrides& ld, int block, int q,
                                               float* sums) {
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const uint32_t rows = (uint32_t)a.rows, cols = (uint32_t)a.cols, c = block * 32 * q + lane;
    float dw[kDirectColumns] = {};
    float x[kDirectRows][kDirectColumns], g[kDirectRows][kDirectColumns], rstd[kDirectRows];
#pragma unroll
    for (int u = 0; u < kDirectRows; ++u) {
        const uint32_t r = warp + u * warps;
        rstd[u] = r < rows ? a.rstd[r] : 0.f;
#pragma unroll
        for (int j = 0; j < kDirectColumns; ++j) {
            const bool in = j < q && c + 32 * j < cols && r < rows;
            x[u][j] = in ? to_f32<T>(((const T*)row_at((const uint8_t*)a.s, r, ld.in[0]))[c + 32 * j]) : 0.f;
            g[u][j] = in ? to_f32<TG>(((const TG*)row_at((const uint8_t*)a.dout, r, ld.in[1]))[c + 32 * j]) : 0.f;
        }
    }
#pragma unroll
    for (int u = 0; u < kDirectRows; ++u)
#pragma unroll
        for (int j = 0; j < kDirectColumns; ++j) dw[j] = fmaf(g[u][j], x[u][j] * rstd[u], dw[j]);
#pragma unroll
    for (int j = 0; j < kDirectColumns; ++j) sums[(j * warps + warp) * 32 + lane] = dw[j];
    __syncthreads();
    for (uint32_t j = warp; j < (uint32_t)q; j += warps) {  // the warps' sums in order
        if (c + 32 * j >= cols) continue;
        float t = 0.f;
        for (uint32_t k = 0; k < warps; ++k) t += sums[(j * warps + k) * 32 + lane];
        a.dweight[c + 32 * j] = a.accumulate ? a.dweight[c + 32 * j] + t : t;
    }
}

// Those blocks in a launch of their own, ahead of the rows that are written over.
template <typename T, typename TG>
__global__ void __launch_bounds__(1024)
    rms_norm_weight_grad_kernel(const __grid_constant__ RmsNormGradCall a, const __grid_constant__ RowStrides ld,
                                int direct) {
    extern __shared__ float warp_sums[];
    grid_dependency_wait();
    weight_grad_block<T, TG>(a, ld, blockIdx.x, direct, warp_sums);
}

// The same through shared memory, as rms_norm_ring_kernel (DSUM as RES there; without it rows of 7161 BF16 columns
// take 8% less): dx, and the weight gradient of the block's
// rows, which its threads keep in registers, added over its teams at the end (or left to blocks of its own).
template <typename T, typename TG, RowKind KIND, bool DSUM>
__global__ void __launch_bounds__(1024)
    rms_norm_grad_ring_kernel(const __grid_constant__ RmsNormGradCall a, const __grid_constant__ RowStrides ld,
                              int direct, RowTeams t) {
    extern __shared__ uint4 ring_memory[];
    __shared__ float part[2][32];
    constexpr int E = sizeof(T) == 4 || sizeof(TG) == 4 ? 4 : 8, H = E / 2, P = 8 / E, STAGES = kGradStages;
    constexpr bool ODD = KIND == kOdd || KIND == kShifted, SHIFTED = KIND == kShifted;
    constexpr int U = SHIFTED ? 2 : 1;                      // places of a piece
    if constexpr (KIND == kWide) cluster_sync();            // every block of it is there to be written to
    grid_dependency_wait();
    if (KIND != kWide && blockIdx.x >= t.blocks) {          // direct: groups of 32 columns to a block
        weight_grad_block<T, TG>(a, ld, blockIdx.x - t.blocks, direct, reinterpret_cast<float*>(ring_memory));
        return;
    }
    const RowPlace p = row_place<KIND>(t);
    const bool with_sum = DSUM && a.dsum != nullptr;
    const Ring ring = ring_place(ring_memory, with_sum ? 3 * P * U : 2 * P * U);
    const uint32_t rows = (uint32_t)a.rows, cols = (uint32_t)a.cols, end = STAGES * ring.stage;
    const uint32_t shift = ODD ? (ld.shift + (p.base + p.sub) * ld.turn) % E : 0;
    // this block's columns
    const uint32_t from = KIND == kWide ? p.rank * t.share : 0, to = KIND == kWide ? min(cols, from + t.share) : cols;
    Span at[P];
#pragma unroll
    for (int k = 0; k < P; ++k) at[k] = span_at<ODD, E>((int)(from + (p.at + k * p.width) * E - shift), (int)to);
    const uint32_t next = p.width * E;                      // columns from one piece to the next
    const uint8_t *s = (const uint8_t*)((const T*)a.s + at[0].c), *dout = (const uint8_t*)((const TG*)a.dout + at[0].c);
    const uint8_t* dsum = (const uint8_t*)((const T*)a.dsum + at[0].c);
    uint8_t* dx = (uint8_t*)((T*)a.dx + at[0].c);
    const int s_skip = pieces_skip(row_at(s, p.base + p.sub, ld.in[0]));   // SHIFTED, where P is 1
    const int g_skip = pieces_skip(row_at(dout, p.base + p.sub, ld.in[1]));
    const int u_skip = pieces_skip(row_at(dsum, p.base + p.sub, ld.in[2]));
    uint32_t far = p.base, put = 0;                         // the rows fetched next
    auto fetch = [&]() {
        if (far < rows) {
            const uint32_t r = far + p.sub;
            const uint8_t *sr = row_at(s, r, ld.in[0]), *gr = row_at(dout, r, ld.in[1]), *ur = row_at(dsum, r, ld.in[2]);
#pragma unroll
            for (int k = 0; k < P; ++k) {
                if constexpr (SHIFTED) {
                    pieces_fetch(ring, put, 0, sr, at[0], s_skip, r, r < rows);
                    pieces_fetch(ring, put, 2, gr, at[0], g_skip, r, r < rows);
                    if (with_sum) pieces_fetch(ring, put, 4, ur, at[0], u_skip, r, r < rows);
                    continue;
                }
                ring_fetch<ODD, T, E>(ring, put, k, sr + k * next * sizeof(T), at[k], r, r < rows);
                ring_fetch<ODD, TG, E>(ring, put, P + k, gr + k * next * sizeof(TG), at[k], r, r < rows);
                if (with_sum) ring_fetch<ODD, T, E>(ring, put, 2 * P + k, ur + k * next * sizeof(T), at[k], r, r < rows);
            }
        }
        cp_async_commit();
        far += p.step;
        put = put + ring.stage == end ? 0 : put + ring.stage;
    };
#pragma unroll
    for (int k = 0; k < STAGES; ++k) fetch();
    if constexpr (SHIFTED) {
        if (const uint32_t r = p.base + p.sub; r < 8) {
            pieces_first(ring.at, ring.unit, row_at(s, r, ld.in[0]), at[0], s_skip, r < rows);
            pieces_first(ring.at + 2 * ring.unit, ring.unit, row_at(dout, r, ld.in[1]), at[0], g_skip, r < rows);
            if (with_sum)
                pieces_first(ring.at + 4 * ring.unit, ring.unit, row_at(dsum, r, ld.in[2]), at[0], u_skip, r < rows);
        }
    } else if (const uint32_t r = p.base + p.sub; patched<ODD, E>(at[0], r)) {
        const int last = r < rows ? at[0].last : 0;
        ring_patch<T, E>(ring.at, (const T*)row_at(s, r, ld.in[0]), at[0].first, last);
        ring_patch<TG, E>(ring.at + P * ring.unit, (const TG*)row_at(dout, r, ld.in[1]), at[0].first, last);
        if (with_sum)
            ring_patch<T, E>(ring.at + 2 * P * ring.unit, (const T*)row_at(dsum, r, ld.in[2]), at[0].first, last);
    }

    F2 w[P][H], dw[P][H];
#pragma unroll
    for (int k = 0; k < P; ++k) {
        load_weights<E>(a.weight, a.w_dtype, at[k], w[k]);
#pragma unroll
        for (int i = 0; i < H; ++i) dw[k][i] = f2(0.f, 0.f);
    }
    const float inv_cols = 1.f / (float)a.cols;
    uint32_t r = p.base + p.sub, get = 0;
    float next_rstd = r < rows ? a.rstd[r] : 0.f;
    int turn = 0;
    for (uint32_t base = p.base; base < rows; base += p.step) {
        const bool live = r < rows;
        const float rstd = next_rstd;
        next_rstd = r + p.step < rows ? a.rstd[r + p.step] : 0.f;
        cp_async_wait<STAGES - 1>();
        F2 h[P][H], g[P][H], c2 = f2(0.f, 0.f);
        const F2 by = f2(rstd, rstd);
#pragma unroll
        for (int k = 0; k < P; ++k) {
            to_pairs(taken<KIND, T, E>(ring, get, k * U, at[k], s_skip), h[k]);
            to_pairs(taken<KIND, TG, E>(ring, get, (P + k) * U, at[k], g_skip), g[k]);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                h[k][i] = f2_mul(h[k][i], by);
                dw[k][i] = f2_fma(g[k][i], h[k][i], dw[k][i]);
                g[k][i] = f2_mul(g[k][i], w[k][i]);
                c2 = f2_fma(g[k][i], h[k][i], c2);
            }
        }
        const float mean = -inv_cols * team_sum<KIND>(pair_sum(c2), t, p, part, turn++);
        const F2 minus = f2(mean, mean);
#pragma unroll
        for (int k = 0; k < P; ++k) {
#pragma unroll
            for (int i = 0; i < H; ++i) g[k][i] = f2_mul(by, f2_fma(h[k][i], minus, g[k][i]));
            if (with_sum) {
                to_pairs(taken<KIND, T, E>(ring, get, (2 * P + k) * U, at[k], u_skip), h[k]);
#pragma unroll
                for (int i = 0; i < H; ++i) g[k][i] = f2_add(g[k][i], h[k][i]);
            }
            if (live)
                store_span<ODD, T, E>(row_at(dx, r, ld.out[0]) + k * next * sizeof(T), at[k], from_pairs<T, E>(g[k]));
        }
        get = get + ring.stage == end ? 0 : get + ring.stage;
        fetch();
        r += p.step;
    }
    if (!a.dweight || direct) return;
    cp_async_wait<0>();
    __syncthreads();
    float* joint = reinterpret_cast<float*>(ring_memory);   // [threads][P * E]
#pragma unroll
    for (int k = 0; k < P; ++k)
#pragma unroll
        for (int i = 0; i < H; ++i) {
            float* to = joint + (threadIdx.x * P + k) * E + 2 * i;
            f2_split(dw[k][i], to[0], to[1]);
        }
    __syncthreads();
    const uint32_t per = 32 / t.lanes, teams = blockDim.x / 32 / t.team_warps;
    const uint32_t share = KIND == kWide ? blockIdx.x / t.cluster : blockIdx.x;   // of the rows
    for (uint32_t col = from + threadIdx.x; col < to; col += blockDim.x) {
        float sum = 0.f;
        for (uint32_t j = 0; j < teams * per; ++j) {    // the threads that have the column, row by row of the block
            const uint32_t row = blockIdx.x * teams * per + j;
            const uint32_t place = col - from + (ODD ? (ld.shift + row * ld.turn) % E : 0);
            const uint32_t piece = place / E, k = piece / p.width, thread = piece - k * p.width;
            sum += joint[((j / per * t.team_warps * 32 + j % per * t.lanes + thread) * P + k) * E + place % E];
        }
        a.part[(int64_t)share * a.cols + col] = sum;
    }
}

// Rows that the ring does not take and registers do not hold: the row is read twice by its block, and the
// weight gradient is summed by a kernel of its own.  4096 x 16385 BF16 with dsum 266 us, 8000 x 8193 301 (single-element
// accesses, three passes); aligned, 1024 x 65544 198 us (2.7 TB/s).
template <typename T, typename TG, bool VEC>
__global__ void __launch_bounds__(1024) rms_norm_grad_long_kernel(const __grid_constant__ RmsNormGradCall a) {
    __shared__ float part[32];
    grid_dependency_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t r = blockIdx.x;
    const T* s = (const T*)a.s + r * a.ld_s;
    const TG* dout = (const TG*)a.dout + r * a.ld_dout;
    const float rstd = a.rstd[r];
    float c = 0.f;
    for (int64_t c0 = warp * 256; c0 < a.cols; c0 += 32 * 256) {
        float h[8], g[8], w[8], t = 0.f;
        load_chunk<T, VEC>(s, c0, a.cols, lane, h);
        load_chunk<TG, VEC>(dout, c0, a.cols, lane, g);
        load_weight<VEC>(a.weight, a.w_dtype, c0, a.cols, lane, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) t = fmaf(g[i] * w[i], h[i] * rstd, t);
        c += t;
    }
    c = row_sum<false>(c, part) / (float)a.cols;
    for (int64_t c0 = warp * 256; c0 < a.cols; c0 += 32 * 256) {
        float h[8], g[8], w[8], d[8];
        load_chunk<T, VEC>(s, c0, a.cols, lane, h);
        load_chunk<TG, VEC>(dout, c0, a.cols, lane, g);
        load_weight<VEC>(a.weight, a.w_dtype, c0, a.cols, lane, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = 0.f;
        if (a.dsum) load_chunk<T, VEC>((const T*)a.dsum + r * a.ld_dsum, c0, a.cols, lane, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = fmaf(rstd, fmaf(-h[i] * rstd, c, g[i] * w[i]), d[i]);
        store_chunk<T, VEC>((T*)a.dx + r * a.ld_dx, c0, a.cols, lane, d);
    }
}

// The weight gradient's partial sums for such rows, before dx may be written over dout: one warp
// per 256 columns, blockIdx.y-th of gridDim.y shares of the rows.
template <typename T, typename TG, bool VEC>
__global__ void __launch_bounds__(128) rms_norm_dw_long_kernel(const __grid_constant__ RmsNormGradCall a,
                                                               int shares, int64_t chunk_blocks) {
    grid_dependency_wait();
    const int lane = threadIdx.x % 32;
    const int64_t share = blockIdx.x / chunk_blocks, block = blockIdx.x - share * chunk_blocks;
    const int64_t c0 = (block * 4 + threadIdx.x / 32) * 256;
    if (c0 >= a.cols) return;
    float dw[8] = {};
    for (int64_t r = share; r < a.rows; r += shares) {
        float h[8], g[8];
        load_chunk<T, VEC>((const T*)a.s + r * a.ld_s, c0, a.cols, lane, h);
        load_chunk<TG, VEC>((const TG*)a.dout + r * a.ld_dout, c0, a.cols, lane, g);
        const float rstd = a.rstd[r];
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[i] = fmaf(g[i], h[i] * rstd, dw[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t c = c0 + (VEC ? lane * 8 + i : i * 32 + lane);
        if (c < a.cols) a.part[share * a.cols + c] = dw[i];
    }
}

// dweight (+)= the sum of `rows` partial rows, in the same order every time: warp k adds rows k, k + 32, ...,
// then the warps' sums are added in pairs (one after another they are 32 roundings deep: 777 x 1409 FP32 was 1.31e-7 off
// 64-bit arithmetic, so it is 1.00e-7, as a plain FP32 sum).
__global__ void __launch_bounds__(1024) rms_norm_dw_join_kernel(const float* part, int64_t rows, int64_t cols,
                                                                float* dweight, int accumulate) {
    __shared__ float sums[32][33];
    grid_dependency_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float t = 0.f;
    if (c < cols)
        for (int64_t r = warp; r < rows; r += 32) t += part[r * cols + c];
    sums[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && c < cols) {
        float v[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = sums[k][lane];
#pragma unroll
        for (int n = 16; n; n /= 2)
#pragma unroll
            for (int k = 0; k < n; ++k) v[k] += v[k + n];
        dweight[c] = accumulate ? dweight[c] + v[0] : v[0];
    }
}

template <typename T, typename TG>
bool launch_grad_ring(const RmsNormGradCall& c, cudaStream_t stream, int64_t& parts, bool& joined, cudaError_t& e) {
    constexpr int E = sizeof(T) == 4 || sizeof(TG) == 4 ? 4 : 8, P = 8 / E;
    RowCheck check{E};
    RowStrides ld{};
    ld.in[0] = check.stride(c.s, c.ld_s, sizeof(T)), ld.in[1] = check.stride(c.dout, c.ld_dout, sizeof(TG));
    ld.in[2] = check.stride(c.dsum, c.ld_dsum, sizeof(T)), ld.out[0] = check.stride(c.dx, c.ld_dx, sizeof(T));
    ld.shift = check.shift, ld.turn = check.turn;
    const bool shifted = !check.ok && P == 1, odd = shifted || check.odd || c.cols % E;
    if (shifted) {                                          // by what is written
        RowCheck s{E}, dout{E}, dsum{E}, written{E};
        s.stride(c.s, c.ld_s, sizeof(T)), dout.stride(c.dout, c.ld_dout, sizeof(TG));
        dsum.stride(c.dsum, c.ld_dsum, sizeof(T)), written.stride(c.dx, c.ld_dx, sizeof(T));
        if (!s.ok || !dout.ok || !dsum.ok || !written.ok || c.cols < 2 || c.cols + E - 1 > kRingCols) return false;
        ld.shift = written.shift, ld.turn = written.turn;
    }
    if (c.cols > kRingCols && check.takes_wide(c.cols)) {
        const size_t stage = 16 * P * (c.dsum ? 3 : 2);
        auto go = [&](auto k) {
            const RowGrid g = wide_grid(k, c.rows, c.cols, stage, kGradStages, e);
            parts = g.blocks / g.teams.cluster;
            if (parts > kNormParts) e = cudaErrorInvalidConfiguration;
            if (e == cudaSuccess) e = launch_ring(k, g, stage * g.threads, kGradStages, stream, c, ld, 0);
        };
        if (c.dsum) go(rms_norm_grad_ring_kernel<T, TG, kWide, true>);
        else go(rms_norm_grad_ring_kernel<T, TG, kWide, false>);
        return true;
    }
    if (!shifted && !check.takes(c.cols)) return false;
    RowGrid g = row_grid(c.rows, c.cols + (odd ? E - 1 : 0), 8, c.num_sms < kFewParts ? c.num_sms : kFewParts);
    const bool directly = c.dweight && c.rows <= kDirectRows * (g.threads / 32);
    if (odd && ((!g.one_row && g.blocks % 8) || (few_rows<E>(c.rows, c.cols) && !directly))) return false;
    size_t stage = (size_t)g.threads * 16 * P * (c.dsum ? 3 : 2) * (shifted ? 2 : 1);
    parts = g.blocks;
    int direct = 0;
    if (directly) {
        const int64_t groups = (c.cols + 31) / 32;
        direct = groups <= 64 ? 1 : groups <= 128 ? 2 : kDirectColumns;
        const int64_t blocks = (groups + direct - 1) / direct;
        const size_t sums = (size_t)g.threads * kDirectColumns * sizeof(float);
        joined = true;
        if (c.dx == c.s || c.dx == c.dout) {                // gone before it is read again
            e = launch_after(rms_norm_weight_grad_kernel<T, TG>, blocks, g.threads, sums, 1, stream, c, ld, direct);
            if (e != cudaSuccess) return true;
        } else {
            g.blocks += blocks;
            if (stage < sums) stage = sums;
        }
    }
    auto go = [&](auto k) { e = launch_ring(k, g, stage, kGradStages, stream, c, ld, direct); };
    if constexpr (P == 1) {
        if (shifted) {
            c.dsum ? go(rms_norm_grad_ring_kernel<T, TG, kShifted, true>)
                   : go(rms_norm_grad_ring_kernel<T, TG, kShifted, false>);
            return true;
        }
    }
    if (odd && c.dsum) go(rms_norm_grad_ring_kernel<T, TG, kOdd, true>);
    else if (odd) go(rms_norm_grad_ring_kernel<T, TG, kOdd, false>);
    else if (c.dsum) go(rms_norm_grad_ring_kernel<T, TG, kGroups, true>);
    else go(rms_norm_grad_ring_kernel<T, TG, kGroups, false>);
    return true;
}

// Shares of the rows for rms_norm_dw_long_kernel: 32 rows one after another, as far as kNormParts shares allow
// (in 16 shares whatever the rows, FP32 sums were 8192 additions deep at 131072 of them, and too few blocks read:
// 8000 x 8193 BF16 with dsum 761 us, 301 so).
int64_t long_parts(int64_t rows) {
    int64_t parts = (rows + 31) / 32;
    if (parts < 16) parts = rows < 16 ? rows : 16;
    return parts < kNormParts ? parts : kNormParts;
}

template <typename T, typename TG>
cudaError_t launch_grad_rows(const RmsNormGradCall& c, bool vec, cudaStream_t stream) {
    const int64_t chunks = (c.cols + 255) / 256;
    int64_t parts = 0;
    bool joined = false;
    cudaError_t e = cudaSuccess;
    if (c.rows > 0 && launch_grad_ring<T, TG>(c, stream, parts, joined, e)) {
    } else if (c.rows > 0 && !vec && chunks <= 2) {
        const int warps = c.rows >= 16 * kFewParts ? 16 : 4;   // 226562 x 128 FP32 with dsum 77 us with 16
        const int64_t blocks = (c.rows + warps - 1) / warps;
        parts = blocks < kFewParts ? blocks : kFewParts;
        const size_t joint = (size_t)warps * chunks * 1024;
        e = chunks == 1 ? launch_after(rms_norm_grad_kernel<T, TG, 1, true>, parts, warps * 32, joint, 1, stream, c)
                        : launch_after(rms_norm_grad_kernel<T, TG, 2, true>, parts, warps * 32, joint, 1, stream, c);
    } else if (c.rows > 0 && !vec && chunks <= 32) {
        // two blocks per SM, or four of up to 256 threads (20596 x 1408 FP32 with dsum 134 us with two, 90 with four)
        const int64_t most = chunks <= 8 && c.rows >= 16 * kFewParts ? kNormParts : kFewParts;
        parts = c.rows < most ? c.rows : most;
        const int per = chunks <= 16 ? 1 : 2;
        const int threads = (int)((chunks + per - 1) / per) * 32;
        e = per == 1 ? launch_after(rms_norm_grad_kernel<T, TG, 1, false>, parts, threads, 0, 1, stream, c)
                     : launch_after(rms_norm_grad_kernel<T, TG, 2, false>, parts, threads, 0, 1, stream, c);
    } else if (c.rows > 0) {
        if (c.dweight) {
            parts = long_parts(c.rows);
            const int64_t blocks = (chunks + 3) / 4;
            auto go = [&](auto k) { e = launch_after(k, parts * blocks, 128, 0, 1, stream, c, (int)parts, blocks); };
            vec ? go(rms_norm_dw_long_kernel<T, TG, true>) : go(rms_norm_dw_long_kernel<T, TG, false>);
        }
        if (e == cudaSuccess)
            e = vec ? launch_after(rms_norm_grad_long_kernel<T, TG, true>, c.rows, 1024, 0, 1, stream, c)
                    : launch_after(rms_norm_grad_long_kernel<T, TG, false>, c.rows, 1024, 0, 1, stream, c);
    }
    if (e != cudaSuccess || !c.dweight || joined) return e;
    return launch_after(rms_norm_dw_join_kernel, (c.cols + 31) / 32, 1024, 0, 1, stream, (const float*)c.part, parts,
                        c.cols, c.dweight, c.accumulate);
}

}  // namespace

cudaError_t launch_rms_norm(const RmsNormCall& c, cudaStream_t stream) {
    const bool vec = rows_in_groups(c.x, c.cols, c.ld_x, c.dtype) &&
                     (!c.residual || (rows_in_groups(c.residual, c.cols, c.ld_res, c.dtype) &&
                                      rows_in_groups(c.sum, c.cols, c.ld_sum, c.dtype))) &&
                     (!c.out || rows_in_groups(c.out, c.cols, c.ld_out, c.out_dtype)) &&
                     (!c.weight || rows_in_groups(c.weight, c.cols, c.cols, c.w_dtype)) &&
                     (!c.codes || (uintptr_t)c.codes % 8 == 0);
    return c.dtype == MOE_F32 ? launch_rms_norm_rows<float>(c, vec, stream)
                              : launch_rms_norm_rows<uint16_t>(c, vec, stream);
}

cudaError_t launch_rms_norm_backward(const RmsNormGradCall& c, cudaStream_t stream) {
    const bool vec = rows_in_groups(c.s, c.cols, c.ld_s, c.dtype) &&
                     rows_in_groups(c.dout, c.cols, c.ld_dout, c.dout_dtype) &&
                     rows_in_groups(c.dx, c.cols, c.ld_dx, c.dtype) &&
                     (!c.dsum || rows_in_groups(c.dsum, c.cols, c.ld_dsum, c.dtype)) &&
                     (!c.weight || rows_in_groups(c.weight, c.cols, c.cols, c.w_dtype));
    if (c.dtype == MOE_F32)
        return c.dout_dtype == MOE_F32 ? launch_grad_rows<float, float>(c, vec, stream)
                                       : launch_grad_rows<float, uint16_t>(c, vec, stream);
    return c.dout_dtype == MOE_F32 ? launch_grad_rows<uint16_t, float>(c, vec, stream)
                                   : launch_grad_rows<uint16_t, uint16_t>(c, vec, stream);
}

}  // namespace moe
