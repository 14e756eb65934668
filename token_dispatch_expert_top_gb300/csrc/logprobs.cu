// logprobs.cu -- log probabilities of given tokens over rows of logits, with the
// distribution's entropy and the most likely alternatives, and the gradient.
// With c = scale (1 / temperature), m = max_j x_j, S = sum_j exp(c (x_j - m)), l = ln S:
//   logp_j  = c (x_j - m) - l
//   entropy = l - (1/S) sum_j c (x_j - m) exp(c (x_j - m))
//   d x_j   = c [ g_logp (1[j = t] - p_j) - g_entropy p_j (logp_j + entropy) ]
// A logit of -inf is masked out: it adds nothing to any sum and gets no gradient.  A row
// that is masked throughout has logp -inf, entropy 0 and no gradient.  The row's maximum is
// subtracted before the scale is applied, so logits down to the type's lowest value keep
// their meaning (a row of nothing else is uniform).  All sums are FP32.
#include <float.h>

#include "kernels.cuh"
#include "vec_io.cuh"

namespace moe {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two FP32 values in one 64-bit register: one instruction adds or multiplies both.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void f2_split(F2 x, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v));
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// Running sums of a row relative to its largest logit so far, m: with y = (x - m) c2,
// c2 = scale log2 e, s = sum 2^y, t = sum y 2^y.  Logits are raised to kFloor first: a masked
// logit then adds 0 to both sums.  Good for rows whose maximum lies inside (-2^59, 2^59) and
// scales in [2^-20, 2^20]; the careful sums below take the others.
constexpr float kFloor = -0x1p60f, kFastMax = 0x1p59f;
constexpr uint32_t kFloorBf16x2 = 0xDD80DD80u;
inline bool fast_scale(float scale) { return scale >= 0x1p-20f && scale <= 0x1p20f; }
struct RowSums {
    float m, s, t;
    __device__ void init() {
        m = kFloor;
        s = t = 0.f;
    }
    __device__ void raise(float m2, float c2) {
        const float d = (m - m2) * c2, f = exp2_approx(d);
        t = f * fmaf(d, s, t);
        s *= f;
        m = m2;
    }
    __device__ void merge(RowSums o, float c2) {
        if (o.m > m) raise(o.m, c2);
        else o.raise(m, c2);
        s += o.s;
        t += o.t;
    }
};

// The same for any row and scale: s = sum exp(c d), t = sum d exp(c d),
// d = x - m.  m starts at the lowest finite value, so masked logits give d = -inf, exp 0.
struct CarefulSums {
    float m, s, t;
    __device__ void init() {
        m = -FLT_MAX;
        s = t = 0.f;
    }
    __device__ void raise(float m2, float c2) {
        const float d = m - m2, f = exp2_approx(d * c2);
        t = f > 0.f ? f * fmaf(d, s, t) : 0.f;       // f = 0 may meet d = -inf
        s *= f;
        m = m2;
    }
    __device__ void add(float x, float c2) {
        if (x > m) raise(x, c2);
        const float d = x - m, e = exp2_approx(d * c2);
        s += e;
        t = fmaf(e, fmaxf(d, -FLT_MAX), t);          // a masked logit's 0 * -inf is 0
    }
    __device__ void merge(CarefulSums o, float c2) {
        if (o.m > m) raise(o.m, c2);
        else o.raise(m, c2);
        s += o.s;
        t += o.t;
    }
};

// A row as 16-byte vectors of its own alignment: vector v holds the elements
// v*VEC - mis .. v*VEC - mis + VEC - 1; the first and the last may be partial.  (A row has at
// most 2^22 elements.)
template <typename T>
struct RowView {
    static constexpr int VEC = 16 / sizeof(T);
    const T* p;
    int V, mis, nvec;
    __device__ RowView(const T* row, int V_) : p(row), V(V_) {
        mis = (int)(((uintptr_t)row / sizeof(T)) % VEC);
        nvec = (V + mis + VEC - 1) / VEC;
    }
    __device__ int first(int v) const { return v * VEC - mis; }
    __device__ bool whole(int v) const { return first(v) >= 0 && first(v) + VEC <= V; }
    // the vector's elements; fill past the row
    __device__ uint4 load(int v, float fill) const {
        const int j = first(v);
        if (whole(v)) return ld_v4(p + j);
        T e[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) e[i] = j + i >= 0 && j + i < V ? p[j + i] : from_f32<T>(fill);
        uint4 q;
        if constexpr (sizeof(T) == 2)
            q = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16, e[4] | (uint32_t)e[5] << 16,
                           e[6] | (uint32_t)e[7] << 16);
        else
            q = make_uint4(__float_as_uint(e[0]), __float_as_uint(e[1]), __float_as_uint(e[2]), __float_as_uint(e[3]));
        return q;
    }
    __device__ static void unpack(const uint4& q, float (&x)[VEC]) {
        if constexpr (sizeof(T) == 2) {
            unpack_bf16x8(q, x);
        } else {
            x[0] = __uint_as_float(q.x), x[1] = __uint_as_float(q.y), x[2] = __uint_as_float(q.z),
            x[3] = __uint_as_float(q.w);
        }
    }
};

// ------------------------------------------------------------------------ top list
// A logit as an unsigned integer of the same order (0 is below every number); -0 and +0
// are equal.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return x != x ? 0u : (b & 0x80000000u ? ~b : b | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return o == 0u ? __uint_as_float(0x7FC00000u) : __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

// An entry as one number: the larger one is the better one.
__device__ __forceinline__ uint64_t pack_entry(uint32_t key, uint32_t idx) { return (uint64_t)key << 32 | (uint32_t)~idx; }

// A warp's list of entries (key, idx), best first (key descending, then idx ascending), entry
// i in lane i; empty entries are (0, kNone).
constexpr uint32_t kNone = 0xFFFFFFFFu;
struct WarpList {
    uint32_t key, idx;
    __device__ void init() { key = 0u, idx = kNone; }
    __device__ static bool beats(uint32_t k, uint32_t j, uint32_t k2, uint32_t j2) {
        return k > k2 || (k == k2 && j < j2);
    }
    // Compares with the entry `stride` lanes away and keeps the better one where `first`.
    __device__ void exchange(int stride, bool first) {
        const uint32_t k = __shfl_xor_sync(0xffffffffu, key, stride), j = __shfl_xor_sync(0xffffffffu, idx, stride);
        if (beats(k, j, key, idx) == first && (k != key || j != idx)) key = k, idx = j;
    }
    // Bitonic sort of any 32 entries.
    __device__ void sort() {
        const int lane = threadIdx.x % 32;
#pragma unroll
        for (int size = 2; size <= 32; size *= 2)
#pragma unroll
            for (int stride = size / 2; stride; stride /= 2)
                exchange(stride, ((lane & stride) == 0) == ((lane & size) == 0));
    }
    // The best 32 of this list and another sorted one, whose entry 31 - lane is (k, j).
    __device__ void merge_reversed(uint32_t k, uint32_t j) {
        const int lane = threadIdx.x % 32;
        if (beats(k, j, key, idx)) key = k, idx = j;
#pragma unroll
        for (int stride = 16; stride; stride /= 2) exchange(stride, (lane & stride) == 0);
    }
};

constexpr int kLpMaxWarps = 8;
constexpr int kLpUnroll = 4;                    // vectors a lane holds at once
constexpr int kLpChunk = 32 * kLpUnroll;        // vectors a warp reads at once: one chunk
constexpr int kLpMaxCluster = 8;
constexpr int kLpAside = 512;                   // vectors set aside during the pass
constexpr int kLpRanked = 256;                  // logits whose places are found by comparing all of them
static_assert(kLpMaxCluster * kMaxTop <= kLpRanked, "the CTAs' lists are ranked together");

struct LogprobArgs {
    const void* logits;
    int V;
    int64_t ld;
    float scale;
    int careful;                                // the scale is outside the fast sums' range
    const void* targets;
    float *logp, *entropy, *stats;
    int n_top;
    int32_t* top_idx;
    float* top_logp;
    WsHeader* ws;
};

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Raises both halves to kFloor; NaN stays NaN.
__device__ __forceinline__ uint32_t floor_bf16x2(uint32_t a) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(kFloorBf16x2));
    return r;
}
__device__ __forceinline__ float floor_f32(float a) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(kFloor));
    return r;
}

// A float in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ float ld_cluster_f32(const void* p, uint32_t rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint64_t ld_cluster_u64(const void* p, uint32_t rank) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
    return v;
}

// Largest logit of a vector (NaN ignored).
template <typename T>
__device__ __forceinline__ float vector_max(const uint4& q) {
    if constexpr (sizeof(T) == 2) {
        const uint32_t none = 0xFF80FF80u;      // -inf, -inf
        const uint32_t h = max_bf16x2(max_bf16x2(max_bf16x2(q.x, q.y), max_bf16x2(q.z, q.w)), none);
        return fmaxf(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u));
    } else {
        return fmaxf(fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)),
                           fmaxf(__uint_as_float(q.z), __uint_as_float(q.w))), -INFINITY);
    }
}
template <typename T>
__device__ __forceinline__ float lane_max(const uint4 (&q)[kLpUnroll]) {
    float m = vector_max<T>(q[0]);
#pragma unroll
    for (int u = 1; u < kLpUnroll; ++u) m = fmaxf(m, vector_max<T>(q[u]));
    return m;
}

// Adds 2^y and y 2^y of the lane's vectors.
template <typename T>
__device__ __forceinline__ void add_vectors(const uint4 (&q)[kLpUnroll], float c2, RowSums& sums) {
    const F2 c = f2(c2, c2), r = f2(-sums.m, -sums.m);
    F2 s[2] = {f2(sums.s, 0.f), f2(0.f, 0.f)}, t[2] = {f2(sums.t, 0.f), f2(0.f, 0.f)};
#pragma unroll
    for (int u = 0; u < kLpUnroll; ++u) {
        const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
        constexpr int P = sizeof(T) == 2 ? 4 : 2;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            F2 x;
            if constexpr (sizeof(T) == 2) {
                const uint32_t h = floor_bf16x2(w[p]);
                x = f2(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u));
            } else {
                x = f2(floor_f32(__uint_as_float(w[2 * p])), floor_f32(__uint_as_float(w[2 * p + 1])));
            }
            const F2 y = f2_mul(f2_add(x, r), c);
            float y0, y1;
            f2_split(y, y0, y1);
            const F2 e = f2(exp2_approx(y0), exp2_approx(y1));
            s[p & 1] = f2_add(s[p & 1], e);
            t[p & 1] = f2_fma(e, y, t[p & 1]);
        }
    }
    float a, b;
    f2_split(f2_add(s[0], s[1]), a, b);
    sums.s = a + b;
    f2_split(f2_add(t[0], t[1]), a, b);
    sums.t = a + b;
}

// One cluster of CTAs per row (each takes a contiguous share of the row's chunks), one pass
// over the row: 8192 x 127901 BF16 in 305 us (6.9 TB/s), with the top 8 in 334 us.  The pass is
// bound by HBM: up to 8 loads of 16 bytes per lane are in flight, 32 warps an SM, and per BF16
// logit about 7 instructions are issued, one of them the exponential.  With the top list it
// is the latency of each row's end that shows, which the other rows in flight do not hide.
// For the top list the pass sets aside, from registers, the vectors with a logit that reaches a
// bound which rises as it goes; about a hundred for n = 8, of which some 3 n logits reach the
// last bound and are ranked.  Masked logits are never set aside; they fill the list's end by
// index.  (Reading the best chunks again afterwards cost a trip to DRAM per row, as the rows
// in flight do not fit L2: 369 against 345 us for 8192 x 127901 BF16 and n = 8.)  Where
// the logits' order or ties make too many, a way whose work does not depend on the logits is
// taken: the n best logits lie in the n best chunks (what a warp reads at once) by (maximum,
// position), as a chunk below those has n chunks before it, each with a logit that beats all
// of its own; likewise in the n best vectors of these, which are 8 n (FP32: 4 n) logits.
template <typename T, typename Id, bool TOP>
__global__ void __launch_bounds__(kLpMaxWarps * 32, 4) logprobs_kernel(const __grid_constant__ LogprobArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];          // the chunks read ahead; later chunk_max
    __shared__ RowSums warp_sums[kLpMaxWarps], cta_sums;
    __shared__ CarefulSums warp_careful[kLpMaxWarps], cta_careful;
    __shared__ uint32_t vote[kLpMaxWarps], sel[32];
    __shared__ uint32_t list_key[kLpMaxWarps][32], list_idx[kLpMaxWarps][32];
    __shared__ uint4 aside[kLpAside];
    __shared__ int aside_v[kLpAside];
    __shared__ uint64_t few[kLpRanked], cta_list[32];
    __shared__ int found, ranked;
    constexpr int VEC = RowView<T>::VEC;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const uint32_t rank = cluster_ctarank(), ctas = cluster_nctarank();
    const int64_t r = blockIdx.x / ctas;
    const RowView<T> row((const T*)a.logits + r * a.ld, a.V);
    const int row_chunks = (row.nvec + kLpChunk - 1) / kLpChunk;
    const int share = (row_chunks + (int)ctas - 1) / (int)ctas;
    const int g_first = (int)rank * share;
    const int chunks = max(0, min(share, row_chunks - g_first));     // this CTA's
    const float c2 = a.scale * kLog2e;
    auto sync_cluster = [&]() {
        __syncwarp();                                        // the barrier wants whole warps
        cluster_sync();
    };
    auto load_chunk = [&](int g, uint4 (&q)[kLpUnroll]) {
        const int v0 = (g_first + g) * kLpChunk;
        const T* p = row.p + row.first(v0) + lane * VEC;
        if (row.whole(v0) && row.whole(v0 + kLpChunk - 1)) {         // the same for the whole warp
#pragma unroll
            for (int u = 0; u < kLpUnroll; ++u) q[u] = ld_v4(p + u * 32 * VEC);
        } else {
            const uint32_t none = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;      // -inf
#pragma unroll
            for (int u = 0; u < kLpUnroll; ++u) {
                const int v = v0 + u * 32 + lane;
                q[u] = v < row.nvec ? row.load(v, -INFINITY) : make_uint4(none, none, none, none);
            }
        }
    };
    // BF16 rows (twice the arithmetic per byte): the pass copies each warp's next chunk to shared
    // memory while it works on this one: 335 against 345 us for 8192 x 127901 and n = 8.  FP32 rows
    // were up to 20% slower so.  Every lane copies and takes its own vectors: no barrier.
    constexpr bool kAhead = sizeof(T) == 2;
    uint4* ring = reinterpret_cast<uint4*>(smem) + warp * kLpUnroll * 32 + lane;
    auto prefetch = [&](int g) {
        const int v0 = (g_first + g) * kLpChunk;
        if (g < chunks && row.whole(v0) && row.whole(v0 + kLpChunk - 1)) {
            const T* p = row.p + row.first(v0) + lane * VEC;
#pragma unroll
            for (int u = 0; u < kLpUnroll; ++u) cp_async_16(ring + u * 32, p + u * 32 * VEC);
        }
    };
    auto take_chunk = [&](int g, uint4 (&q)[kLpUnroll]) {
        const int v0 = (g_first + g) * kLpChunk;
        if (kAhead && row.whole(v0) && row.whole(v0 + kLpChunk - 1)) {
            cp_async_wait_all();
#pragma unroll
            for (int u = 0; u < kLpUnroll; ++u) q[u] = ring[u * 32];
        } else {
            load_chunk(g, q);
        }
    };

    // For the top list each of the first `voters` warps publishes its j-th best lane maximum so
    // far, voters * j >= n: the lowest of them is a bound that n logits reach.  (A warp with a
    // single chunk that does not fill its lanes stands aside if others can.)
    const int n = a.n_top;
    int voters = min(warps, chunks);
    if (voters > 1 && chunks <= warps && (g_first + chunks - 1) * kLpChunk + 31 >= row.nvec) --voters;
    float lane_top = -INFINITY;
    auto publish = [&]() {
        if (warp >= voters) {
            if (lane == 0) vote[warp] = 0xFFFFFFFFu;
            return;
        }
        uint32_t key = (g_first + warp) * kLpChunk + lane < row.nvec ? order_of(lane_top) : 0u;
        uint32_t nth = 0u;
        for (int i = 0; i < n; i += voters) {
            nth = __reduce_max_sync(0xffffffffu, key);
            if (lane == __ffs(__ballot_sync(0xffffffffu, key == nth)) - 1) key = 0u;
        }
        if (lane == 0) vote[warp] = nth;
    };
    auto lowest_vote = [&]() {
        return __reduce_min_sync(0xffffffffu, lane < voters ? *(volatile uint32_t*)&vote[lane] : 0xFFFFFFFFu);
    };
    if (TOP && threadIdx.x == 0) found = 0, ranked = 0;
    int round = 0;
    bool all = true;                                         // no bound yet
    float bound = -INFINITY;
    RowSums sums;
    sums.init();
    if (kAhead) prefetch(warp);
    for (int g = warp; g < chunks; g += warps, ++round) {
        uint4 q[kLpUnroll];
        take_chunk(g, q);
        if (kAhead) prefetch(g + warps);
        float mx[kLpUnroll], top;
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u) {
            mx[u] = vector_max<T>(q[u]);
            top = u ? fmaxf(top, mx[u]) : mx[u];
        }
        if constexpr (TOP) {
            lane_top = fmaxf(lane_top, top);
            // a new bound in rounds 0, 1, 2, 4, 8, ...; for long lists in 3, 6, 12, ... too
            if ((round & (round - 1)) == 0 || (n > 8 && round == 3 * (round & -round))) {
                publish();
                if (round == 0) __syncthreads();
                else __syncwarp();
                const uint32_t lowest = lowest_vote();
                all = lowest == 0u;
                bound = value_of(lowest);
            }
            if (__any_sync(0xffffffffu, all || top >= bound)) {
#pragma unroll
                for (int u = 0; u < kLpUnroll; ++u) {
                    const int v = (g_first + g) * kLpChunk + u * 32 + lane;
                    if (v < row.nvec && mx[u] > -INFINITY && (all || mx[u] >= bound)) {
                        const int at = atomicAdd(&found, 1);
                        if (at < kLpAside) aside[at] = q[u], aside_v[at] = v;
                    }
                }
            }
        }
        if (top > sums.m) sums.raise(top, c2);
        add_vectors<T>(q, c2, sums);
    }
    if constexpr (TOP) {
        publish();                                           // read after the next barrier
        if (round == 0) __syncthreads();                     // a warp without chunks: the others' first round
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        RowSums other;
        other.m = __shfl_xor_sync(0xffffffffu, sums.m, o);
        other.s = __shfl_xor_sync(0xffffffffu, sums.s, o);
        other.t = __shfl_xor_sync(0xffffffffu, sums.t, o);
        sums.merge(other, c2);
    }
    if (lane == 0) warp_sums[warp] = sums;
    __syncthreads();
    sums.init();
    if (lane < warps) sums = warp_sums[lane];
    for (int o = kLpMaxWarps / 2; o; o >>= 1) {
        RowSums other;
        other.m = __shfl_xor_sync(0xffffffffu, sums.m, o);
        other.s = __shfl_xor_sync(0xffffffffu, sums.s, o);
        other.t = __shfl_xor_sync(0xffffffffu, sums.t, o);
        sums.merge(other, c2);
    }
    // lane 0's, so that every thread holds the same bits
    sums.m = __shfl_sync(0xffffffffu, sums.m, 0);
    sums.s = __shfl_sync(0xffffffffu, sums.s, 0);
    sums.t = __shfl_sync(0xffffffffu, sums.t, 0);
    if (ctas > 1) {
        if (threadIdx.x == 0) cta_sums = sums;
        sync_cluster();
        sums.init();
        for (uint32_t k = 0; k < ctas; ++k) {
            RowSums o;
            o.m = ld_cluster_f32(&cta_sums.m, k), o.s = ld_cluster_f32(&cta_sums.s, k);
            o.t = ld_cluster_f32(&cta_sums.t, k);
            sums.merge(o, c2);
        }
    }
    float m = sums.m, ls, entropy;
    if (a.careful || !(fabsf(m) < kFastMax)) {
        // the same in every CTA of the cluster
        CarefulSums cs;
        cs.init();
        for (int g = warp; g < chunks; g += warps) {
            uint4 q[kLpUnroll];
            load_chunk(g, q);
#pragma unroll
            for (int u = 0; u < kLpUnroll; ++u) {
                float x[VEC];
                RowView<T>::unpack(q[u], x);
#pragma unroll
                for (int i = 0; i < VEC; ++i) cs.add(x[i], c2);
            }
        }
        for (int o = 16; o; o >>= 1) {
            CarefulSums other;
            other.m = __shfl_xor_sync(0xffffffffu, cs.m, o);
            other.s = __shfl_xor_sync(0xffffffffu, cs.s, o);
            other.t = __shfl_xor_sync(0xffffffffu, cs.t, o);
            cs.merge(other, c2);
        }
        if (lane == 0) warp_careful[warp] = cs;
        __syncthreads();
        cs = warp_careful[0];
        for (int w = 1; w < warps; ++w) cs.merge(warp_careful[w], c2);
        if (ctas > 1) {
            if (threadIdx.x == 0) cta_careful = cs;
            sync_cluster();
            cs.init();
            for (uint32_t k = 0; k < ctas; ++k) {
                CarefulSums o;
                o.m = ld_cluster_f32(&cta_careful.m, k), o.s = ld_cluster_f32(&cta_careful.s, k);
                o.t = ld_cluster_f32(&cta_careful.t, k);
                cs.merge(o, c2);
            }
        }
        m = cs.m;
        ls = cs.s == 0.f ? -INFINITY : logf(cs.s);                   // 0: masked throughout
        entropy = cs.s == 0.f ? 0.f : ls - a.scale * (cs.t / cs.s);
    } else {
        const float l2 = log2f(sums.s);
        ls = kLn2 * l2;
        entropy = kLn2 * (l2 - sums.t / sums.s);
    }
    if (entropy < 0.f) entropy = 0.f;                                // by rounding; NaN stays
    const bool empty = ls == -INFINITY;
    auto logp_of = [&](float x) { return empty || x == -INFINITY ? -INFINITY : (x - m) * a.scale - ls; };
    if (rank == 0 && threadIdx.x == 0) {
        if (a.targets) {
            const Id t = ((const Id*)a.targets)[r];
            float lp = 0.f;
            if (t >= 0 && (int64_t)t < a.V) lp = logp_of(to_f32<T>(row.p[t]));
            else if (t >= 0) set_status(a.ws, MOE_ERR_DEVICE_CHECK);
            a.logp[r] = lp;
        }
        if (a.entropy) a.entropy[r] = entropy;
        if (a.stats) {
            a.stats[2 * r] = m;
            a.stats[2 * r + 1] = ls;
        }
    }
    if constexpr (!TOP) {
        if (ctas > 1) sync_cluster();                                // remote sums have been read
        return;
    }

    // Lists of the first `lists` warps -> one list in warp 0.  Every warp calls it; a warp's
    // place in list_key is written once per call, before the barrier of its level.
    auto merge_lists = [&](WarpList& list, int lists) {
        for (int step = 1; step < lists; step *= 2) {
            if (warp % (2 * step) == step && warp < lists) {
                list_key[warp][lane] = list.key;
                list_idx[warp][lane] = list.idx;
            }
            __syncthreads();
            if (warp % (2 * step) == 0 && warp + step < lists)
                list.merge_reversed(list_key[warp + step][31 - lane], list_idx[warp + step][31 - lane]);
        }
    };
    // adds an entry per lane to the warp's list, unless none of them beats its n-th
    auto take = [&](WarpList& list, uint32_t key, uint32_t idx) {
        const uint32_t last_key = __shfl_sync(0xffffffffu, list.key, a.n_top - 1);
        const uint32_t last_idx = __shfl_sync(0xffffffffu, list.idx, a.n_top - 1);
        if (!__any_sync(0xffffffffu, WarpList::beats(key, idx, last_key, last_idx))) return;
        WarpList next;
        next.key = key, next.idx = idx;
        next.sort();
        list.merge_reversed(__shfl_sync(0xffffffffu, next.key, 31 - lane),
                            __shfl_sync(0xffffffffu, next.idx, 31 - lane));
    };
    auto write_top = [&](int i, uint32_t key, uint32_t idx) {
        a.top_idx[r * n + i] = (int32_t)idx;
        a.top_logp[r * n + i] = logp_of(value_of(key));
    };
    // place i of the CTA's own list
    auto put = [&](int i, uint32_t key, uint32_t idx) {
        if (ctas > 1) cta_list[i] = pack_entry(key, idx);
        else write_top(i, key, idx);
    };
    bool general = true;
    if (found <= kLpAside) {
        // of the vectors set aside the logits that reach the last bound, and their places by
        // comparing all of them
        const uint32_t lowest = lowest_vote(), masked = order_of(-INFINITY);
        const float last = value_of(lowest);
        for (int i = threadIdx.x; i < found * VEC; i += blockDim.x) {
            const float x = to_f32<T>(reinterpret_cast<const T*>(aside)[i]);
            const int j = row.first(aside_v[i / VEC]) + i % VEC;
            if (j < 0 || j >= a.V || !(x > -INFINITY) || !(lowest == 0u || x >= last)) continue;
            const int at = atomicAdd(&ranked, 1);
            if (at < kLpRanked) few[at] = pack_entry(order_of(x), (uint32_t)j);
        }
        __syncthreads();
        const int j0 = max(0, row.first(g_first * kLpChunk));        // this CTA's first logit
        const int need = min(n, chunks ? min(a.V, row.first((g_first + chunks) * kLpChunk)) - j0 : 0);
        // Fewer unmasked logits than places (they have all been set aside then): masked ones
        // follow, the lowest indices, which are among the first `need`.
        unsigned rest = 0u;
        if (ranked < need && lowest <= masked)
            rest = __ballot_sync(0xffffffffu, lane < need && to_f32<T>(row.p[j0 + lane]) == -INFINITY);
        if (ranked <= kLpRanked && ranked + __popc(rest) >= need) {
            general = false;
            for (int i = threadIdx.x; i < ranked; i += blockDim.x) {
                const uint64_t own = few[i];
                int place = 0;
                for (int o = 0; o < ranked; ++o) place += few[o] > own;
                if (place < n) put(place, (uint32_t)(own >> 32), ~(uint32_t)own);
            }
            if (warp == 0) {
                const int place = ranked + __popc(rest & ((1u << lane) - 1u));
                if (rest >> lane & 1 && place < need) put(place, masked, (uint32_t)(j0 + lane));
                if (lane >= need && lane < n) put(lane, 0u, kNone);
            }
        }
    }
    if (general) {
        // The general way, whose work does not depend on the logits: the n best chunks ...
        uint32_t* chunk_max = reinterpret_cast<uint32_t*>(smem);     // order_of the maximum, at least 1
        for (int g = warp; g < chunks; g += warps) {
            uint4 q[kLpUnroll];
            load_chunk(g, q);
            const uint32_t o = __reduce_max_sync(0xffffffffu, max(order_of(lane_max<T>(q)), 1u));
            if (lane == 0) chunk_max[g] = o;
        }
        __syncthreads();
        WarpList list;
        list.init();
        for (int g = warp * 32; g < chunks; g += warps * 32)
            take(list, g + lane < chunks ? chunk_max[g + lane] : 0u, g + lane < chunks ? g + lane : kNone);
        merge_lists(list, min(warps, (chunks + 31) / 32));
        if (warp == 0) sel[lane] = list.idx;
        __syncthreads();
        // ... the n best vectors of those ...
        list.init();
        const int picked = min(n, chunks) * kLpUnroll;
        for (int i = warp; i < picked; i += warps) {
            const int v = (g_first + (int)sel[i / kLpUnroll]) * kLpChunk + i % kLpUnroll * 32 + lane;
            uint32_t key = 0u;
            if (v < row.nvec) {
                float x[VEC];
                RowView<T>::unpack(row.load(v, -INFINITY), x);
                float mx = x[0];
#pragma unroll
                for (int e = 1; e < VEC; ++e) mx = fmaxf(mx, x[e]);
                key = max(order_of(mx), 1u);
            }
            take(list, key, v < row.nvec ? (uint32_t)v : kNone);
        }
        __syncthreads();                                     // sel has been read
        merge_lists(list, min(warps, picked));
        if (warp == 0) sel[lane] = list.idx;
        __syncthreads();
        // ... and the n best logits of those
        list.init();
        for (int i = warp * 32 + lane; i - lane < n * VEC; i += warps * 32) {
            uint32_t key = 0u, idx = kNone;
            if (i < n * VEC && sel[i / VEC] != kNone) {
                const int j = row.first((int)sel[i / VEC]) + i % VEC;
                if (j >= 0 && j < a.V) key = order_of(to_f32<T>(row.p[j])), idx = (uint32_t)j;
            }
            take(list, key, idx);
        }
        merge_lists(list, min(warps, (n * VEC + 31) / 32));
        if (warp == 0 && lane < n) put(lane, list.key, list.idx);
    }
    if (ctas > 1) {
        // the CTAs' lists, n entries each, by comparing all of them
        sync_cluster();
        if (rank == 0) {
            const int all = n * (int)ctas;                   // <= kLpRanked
            for (int i = threadIdx.x; i < all; i += blockDim.x)
                few[i] = ld_cluster_u64(&cta_list[i % n], i / n);
            __syncthreads();
            for (int i = threadIdx.x; i < all; i += blockDim.x) {
                const uint64_t own = few[i];
                int place = 0;
                for (int o = 0; o < all; ++o) place += few[o] > own;
                if (place < n && own != pack_entry(0u, kNone)) write_top(place, (uint32_t)(own >> 32), ~(uint32_t)own);
            }
        }
        sync_cluster();                                      // remote lists and sums have been read
    }
}

template <typename T, bool TOP>
static auto pick_logprobs(int id_bytes) -> void (*)(LogprobArgs) {
    return id_bytes == 8 ? logprobs_kernel<T, int64_t, TOP> : logprobs_kernel<T, int32_t, TOP>;
}

cudaError_t launch_token_logprobs(const LogprobCall& c, cudaStream_t stream) {
    if (c.T == 0) return cudaSuccess;
    LogprobArgs a{c.logits, (int)c.V, c.ld, c.scale, !fast_scale(c.scale), c.targets, c.logp,
                  c.entropy, c.stats, c.n_top, c.top_idx, c.top_logp, c.ws};
    const int64_t vec = 16 / (int64_t)dtype_bytes(c.dtype);
    const int64_t chunks = (c.V + 2 * vec - 2) / (vec * kLpChunk) + 1;         // at most, at any alignment
    // Eight warps per row, in a cluster of CTAs while these fill at most 13/16 of the places (not
    // every place takes a cluster; 128000 FP32, n = 5: 64 rows take 14.4 us in 256 CTAs and 16.4
    // in 512, 150 rows 25 us in 300 CTAs and 32 in 600).  Many rows: four warps, so that twice
    // as many rows are in flight and one row's end hides behind more others (8192 x 127901
    // BF16, n = 8: 345 against 372 us), unless that leaves the last wave of CTAs much emptier
    // (1300 rows: 80 against 74 us).
    const int64_t eights = 4 * (int64_t)c.num_sms, fours = 2 * eights;       // CTAs resident at once
    const int64_t waves8 = (c.T + eights - 1) / eights, waves4 = (c.T + fours - 1) / fours;
    const int most = c.T > eights && 2 * waves4 * 4 <= waves8 * 5 ? 4 : kLpMaxWarps;
    int warps = 1, ctas = 1;
    while (warps < most && warps < chunks) warps *= 2;
    while (ctas < kLpMaxCluster && chunks > (int64_t)warps * ctas && c.T * ctas * 2 <= eights * 13 / 16) ctas *= 2;
    const size_t ahead = c.dtype == MOE_F32 ? 0 : (size_t)warps * kLpChunk * sizeof(uint4);
    const size_t maxima = c.n_top ? sizeof(uint32_t) * (size_t)((chunks + ctas - 1) / ctas) : 0;
    const size_t smem = ahead > maxima ? ahead : maxima;
    void (*k)(LogprobArgs) =
        c.n_top ? (c.dtype == MOE_F32 ? pick_logprobs<float, true>(c.id_bytes) : pick_logprobs<uint16_t, true>(c.id_bytes))
                : (c.dtype == MOE_F32 ? pick_logprobs<float, false>(c.id_bytes)
                                      : pick_logprobs<uint16_t, false>(c.id_bytes));
    cudaLaunchConfig_t cfg{};
    if (c.T * ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    cfg.gridDim = dim3((unsigned)(c.T * ctas));
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = ctas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = ctas > 1;
    return cudaLaunchKernelEx(&cfg, k, a);
}

// ------------------------------------------------------------------------ gradient
// d x_j = p_j (g1 + g2 lp_j) + 1[j = t] scale g_logp with g2 = -scale g_entropy and
// g1 = -scale (g_logp + g_entropy entropy).  dlogits may be the logits' own buffer: a thread
// reads its elements before it writes them.  The kernel moves each logit in and its
// gradient out once, HBM-bound: 4096 x 128000 BF16 in 294 us (7.1 TB/s, part of the logits still in
// L2).  That leaves about 20 instructions per BF16 logit: whole blocks of a row away from its
// ends and its target take a path without checks (with them it issued 21 and took 365 us).
struct LogprobGradArgs {
    const void* logits;
    int64_t T;
    int V;
    int64_t ld;
    float scale;
    int careful;              // the scale is outside the fast path's range
    const void* targets;
    const float *stats, *entropy, *g_logp, *g_entropy;
    void* dlogits;
    int64_t ld_d;
    int blocks_per_row;
    WsHeader* ws;
};
constexpr int kGradThreads = 128, kGradUnroll = 4;
constexpr int kGradVectors = kGradThreads * kGradUnroll;

struct GradRow {
    float m, scale, ls, g1, g2;
};
// 2^y as the square of 2^(y/2): probabilities below FP32's normal numbers keep their bits, at
// the price of one multiplication (the factor they meet may be large).
__device__ __forceinline__ F2 grad_pair(F2 x, const GradRow& g) {
    const F2 lp = f2_fma(f2_add(x, f2(-g.m, -g.m)), f2(g.scale, g.scale), f2(-g.ls, -g.ls));
    float y0, y1;
    f2_split(f2_mul(lp, f2(0.5f * kLog2e, 0.5f * kLog2e)), y0, y1);
    const F2 e = f2(exp2_approx(y0), exp2_approx(y1));
    return f2_mul(f2_mul(e, e), f2_fma(lp, f2(g.g2, g.g2), f2(g.g1, g.g1)));
}
// The same for any logit: a masked one, whose 0 * -inf is 0 here, and any row.
__device__ __forceinline__ float grad_one(float x, const GradRow& g) {
    float lp = (x - g.m) * g.scale - g.ls;
    if (lp < -1e4f) lp = -1e4f;                                      // NaN stays
    const float e = exp2_approx(lp * (0.5f * kLog2e));
    return e * e * fmaf(lp, g.g2, g.g1);
}

template <typename T, typename Id, bool VECTOR>
__global__ void __launch_bounds__(kGradThreads) logprobs_grad_kernel(const __grid_constant__ LogprobGradArgs a) {
    constexpr int VEC = RowView<T>::VEC;
    // the last rows first: they are the ones a forward pass has left in L2 (0.5% faster)
    const int64_t r = a.T - 1 - blockIdx.x / (unsigned)a.blocks_per_row;
    const int v0 = (int)(blockIdx.x % (unsigned)a.blocks_per_row) * kGradVectors;
    const T* in = (const T*)a.logits + r * a.ld;
    T* out = (T*)a.dlogits + r * a.ld_d;
    // logits and gradient rows of the same alignment: vectors of that alignment, their loads
    // before the row's numbers are waited for
    const RowView<T> row(in, a.V);
    const bool inside = VECTOR && row.whole(v0) && row.whole(v0 + kGradVectors - 1);
    const T* p = in + row.first(v0) + (int)threadIdx.x * VEC;
    uint4 q[kGradUnroll];
    if (inside) {
#pragma unroll
        for (int u = 0; u < kGradUnroll; ++u) q[u] = ld_v4(p + u * (kGradThreads * VEC));
    }
    GradRow g;
    g.m = a.stats[2 * r];
    g.ls = a.stats[2 * r + 1];
    g.scale = a.scale;
    int t = -1;
    float gl = 0.f, ge = 0.f, h = 0.f;
    if (a.g_logp) {
        const Id target = ((const Id*)a.targets)[r];
        gl = a.g_logp[r] * a.scale;
        if (target >= 0 && (int64_t)target < a.V) t = (int)target;
        else gl = 0.f;
        if ((int64_t)target >= a.V && v0 == 0 && threadIdx.x == 0) set_status(a.ws, MOE_ERR_DEVICE_CHECK);
    }
    if (a.g_entropy) ge = a.g_entropy[r] * a.scale, h = a.entropy[r];
    const bool empty = g.ls == -INFINITY;                            // masked throughout: no gradient
    g.g2 = -ge;
    g.g1 = -fmaf(ge, h, gl);
    const bool special = empty || a.careful || !(fabsf(g.m) < kFastMax) || fabsf(ge) > 1e6f ||
                         (t >= row.first(v0) && t < row.first(v0 + kGradVectors));
    if (inside && !special) {
        T* o = out + row.first(v0) + (int)threadIdx.x * VEC;
#pragma unroll
        for (int u = 0; u < kGradUnroll; ++u) {
            const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
            uint32_t d[4];
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t f = floor_bf16x2(w[i]);
                    float d0, d1;
                    f2_split(grad_pair(f2(__uint_as_float(f << 16), __uint_as_float(f & 0xFFFF0000u)), g), d0, d1);
                    d[i] = pack_bf16x2(d0, d1);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    float d0, d1;
                    f2_split(grad_pair(f2(floor_f32(__uint_as_float(w[i])), floor_f32(__uint_as_float(w[i + 1]))), g),
                             d0, d1);
                    d[i] = __float_as_uint(d0), d[i + 1] = __float_as_uint(d1);
                }
            }
            st_v4(o + u * (kGradThreads * VEC), make_uint4(d[0], d[1], d[2], d[3]));
        }
        return;
    }
    // element by element, neighbouring lanes on neighbouring elements, eight loads at a time
    const int first = VECTOR ? row.first(v0) : v0 * VEC;
    const int j1 = min(a.V, first + kGradVectors * VEC);
    constexpr int E = 8;
    for (int j0 = max(first, 0) + (int)threadIdx.x; j0 < j1; j0 += E * kGradThreads) {
        T x[E];
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (j0 + i * kGradThreads < j1) x[i] = in[j0 + i * kGradThreads];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int j = j0 + i * kGradThreads;
            if (j >= j1) continue;
            float d = grad_one(to_f32<T>(x[i]), g);
            if (j == t && to_f32<T>(x[i]) != -INFINITY) d += gl;     // a masked target has no part
            out[j] = from_f32<T>(empty ? 0.f : d);
        }
    }
}

template <typename T, typename Id>
static cudaError_t launch_grad_t(LogprobGradArgs& a, cudaStream_t stream) {
    constexpr int64_t VEC = 16 / sizeof(T);
    const bool vec = (((uintptr_t)a.logits - (uintptr_t)a.dlogits) & 15) == 0 &&
                     ((a.ld - a.ld_d) * (int64_t)sizeof(T)) % 16 == 0;
    a.blocks_per_row = (int)(((a.V + 2 * VEC - 2) / VEC + kGradVectors - 1) / kGradVectors);
    const int64_t grid = a.T * a.blocks_per_row;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    auto* k = vec ? logprobs_grad_kernel<T, Id, true> : logprobs_grad_kernel<T, Id, false>;
    k<<<(unsigned)grid, kGradThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_token_logprobs_backward(const LogprobGradCall& c, cudaStream_t stream) {
    if (c.T == 0) return cudaSuccess;
    LogprobGradArgs a{c.logits, c.T, (int)c.V, c.ld, c.scale, !fast_scale(c.scale), c.targets, c.stats, c.entropy, c.g_logp, c.g_entropy,
                      c.dlogits, c.ld_d, 0, c.ws};
    if (c.dtype == MOE_F32)
        return c.id_bytes == 8 ? launch_grad_t<float, int64_t>(a, stream) : launch_grad_t<float, int32_t>(a, stream);
    return c.id_bytes == 8 ? launch_grad_t<uint16_t, int64_t>(a, stream) : launch_grad_t<uint16_t, int32_t>(a, stream);
}

}  // namespace moe
