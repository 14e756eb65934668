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

// c (x - m), 0 or below, for any two logits and scale: the difference may pass FP32's range where c
// brings it back (their halves' does not).
__device__ __forceinline__ float scaled_difference(float x, float m, float scale) {
    const float d = x - m;
    return d == -INFINITY && x != -INFINITY ? 2.f * ((0.5f * x - 0.5f * m) * scale) : d * scale;
}

// The same for any row and scale: s = sum e^z, t = sum z e^z, z = c (x - m).  (The scale comes
// before log2 e: the two's product may pass FP32's range.)  m starts at the lowest finite value, so
// masked logits give z = -inf, e^z = 0.
struct CarefulSums {
    float m, s, t;
    __device__ void init() {
        m = -FLT_MAX;
        s = t = 0.f;
    }
    __device__ void raise(float m2, float scale) {
        const float z = scaled_difference(m, m2, scale), f = exp2_approx(z * kLog2e);
        t = f > 0.f ? f * fmaf(z, s, t) : 0.f;       // f = 0 may meet z = -inf
        s *= f;
        m = m2;
    }
    __device__ void add(float x, float scale) {
        if (x > m) raise(x, scale);
        const float z = scaled_difference(x, m, scale), e = exp2_approx(z * kLog2e);
        s += e;
        t = fmaf(e, fmaxf(z, -FLT_MAX), t);          // a masked logit's 0 * -inf is 0
    }
    __device__ void merge(CarefulSums o, float scale) {
        if (o.m > m) raise(o.m, scale);
        else o.raise(m, scale);
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
constexpr int kLpKept = 512;                    // groups of a CTA whose lanes' maxima are kept (32 KB)
constexpr int kLpAhead = 2;                      // chunks read ahead
constexpr int kLpRanked = 256;                  // logits whose places are found by comparing all of them
// dynamic shared memory at most: the CTAs' lists, BF16 chunks read ahead, and the kept maxima
constexpr int kLpLists = kLpMaxCluster * kMaxTop * 8;
constexpr int kLpMaxSmem = kLpLists + kLpAhead * kLpMaxWarps * kLpChunk * 16 + kLpKept * 64;
static_assert(kLpMaxSmem >= kLpLists + 4 * (kMaxLogprobVocab / (4 * kLpChunk) + 2), "the general way's chunk maxima fit, too");

struct LogprobArgs {
    const void* logits;
    int V;
    int64_t ld;
    float scale;
    int careful;                                // the scale is outside the fast sums' range
    int keep;                                   // shared memory holds the lanes' maxima of the chunks
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
__device__ __forceinline__ void st_cluster_f32(void* p, uint32_t rank, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(smem_u32(p), rank)), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u64(void* p, uint32_t rank, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_shared(smem_u32(p), rank)), "l"(v) : "memory");
}
// Halves of a barrier that only says that the cluster's CTAs have started.
__device__ __forceinline__ void cluster_started_arrive() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_started_wait() {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// Largest logit of one vector, or of a lane's vectors (NaN where all are; otherwise ignored).
template <typename T>
__device__ __forceinline__ float vector_max(const uint4& q) {
    if constexpr (sizeof(T) == 2) {
        const uint32_t h = max_bf16x2(max_bf16x2(q.x, q.y), max_bf16x2(q.z, q.w));
        return fmaxf(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u));
    } else {
        return fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)),
                     fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
    }
}
template <typename T>
__device__ __forceinline__ float lane_max(const uint4 (&q)[kLpUnroll]) {
    static_assert(kLpUnroll == 4, "");
    if constexpr (sizeof(T) == 2) {
        uint4 h;
        h.x = max_bf16x2(max_bf16x2(q[0].x, q[1].x), max_bf16x2(q[2].x, q[3].x));
        h.y = max_bf16x2(max_bf16x2(q[0].y, q[1].y), max_bf16x2(q[2].y, q[3].y));
        h.z = max_bf16x2(max_bf16x2(q[0].z, q[1].z), max_bf16x2(q[2].z, q[3].z));
        h.w = max_bf16x2(max_bf16x2(q[0].w, q[1].w), max_bf16x2(q[2].w, q[3].w));
        return vector_max<T>(h);
    } else {
        return fmaxf(fmaxf(vector_max<T>(q[0]), vector_max<T>(q[1])), fmaxf(vector_max<T>(q[2]), vector_max<T>(q[3])));
    }
}

// A lane's running sums, RowSums' as four partial ones each.
struct LaneSums {
    float m;
    F2 s[2], t[2];
    __device__ void init() {
        m = kFloor;
        s[0] = s[1] = t[0] = t[1] = f2(0.f, 0.f);
    }
    __device__ void raise(float m2, float c2) {
        const float d = (m - m2) * c2, f = exp2_approx(d);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            t[i] = f2_mul(f2(f, f), f2_fma(f2(d, d), s[i], t[i]));
            s[i] = f2_mul(f2(f, f), s[i]);
        }
        m = m2;
    }
    // Adds 2^y and y 2^y of the lane's vectors.
    template <typename T>
    __device__ void add(const uint4 (&q)[kLpUnroll], float c2) {
        const F2 c = f2(c2, c2), r = f2(-m, -m);
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
    }
    __device__ RowSums total() const {
        RowSums o;
        float a, b;
        o.m = m;
        f2_split(f2_add(s[0], s[1]), a, b);
        o.s = a + b;
        f2_split(f2_add(t[0], t[1]), a, b);
        o.t = a + b;
        return o;
    }
};

// One cluster of CTAs per row (each takes a contiguous share of the row's chunks), one pass
// over the row: 8192 x 127901 BF16 in 286 us (7.3 TB/s), with the top 8 in 312 us; 4096 x 128000
// FP32 in 286 and 304 us.  The pass is bound by HBM: 8 copies of 16 bytes per lane are in flight, 32 warps an SM, and per BF16
// logit about 7 instructions are issued, one of them the exponential.  With the top list it
// is the latency of each row's end that shows, which the other rows in flight do not hide.
// For the top list the pass only keeps the lanes' maxima of one or two chunks (a chunk is what
// a warp reads at once), in 16 bits.  Afterwards they give a bound that the n best logits reach
// and tell which lanes' shares of chunks hold such logits, some 3 n; these are read again, all
// at once, and their logits that reach the bound are ranked.  (Noting logits during the pass,
// against a bound that rises, cost 12200 warp instructions a row of 128000; this costs 7100
// beside the pass's 29100.)  In a cluster the warps write their sums, and the CTAs their lists,
// into the shared memory of those that want them, so that a row ends with one barrier of the
// cluster: one row of 128000 FP32, n = 20, takes 8.6 us, 64 of 50001 BF16, n = 5, 8.3.  Masked logits
// never count; they fill the list's end by index.  Where the logits' order or ties leave too
// many, a way whose work does not depend on the logits is taken: the n best logits lie in the
// n best chunks by (maximum, position), as a chunk below those has n chunks before it, each
// with a logit that beats all of its own; likewise in the n best vectors of these, which are
// 8 n (FP32: 4 n) logits.
template <typename T, typename Id, bool TOP, bool CLUSTER>
__global__ void __launch_bounds__(kLpMaxWarps * 32, 4) logprobs_kernel(const __grid_constant__ LogprobArgs a) {
    // lists; the chunks read ahead; later chunk_max.  (Copies to shared memory that are not aligned
    // to its lines of 128 bytes fetch their sectors twice: 340 instead of 326 us.)
    extern __shared__ __align__(128) uint8_t dynamic_smem[];
    __shared__ RowSums warp_sums[kLpMaxWarps * kLpMaxCluster];
    __shared__ CarefulSums warp_careful[kLpMaxWarps], cta_careful;
    __shared__ uint32_t vote[kLpMaxWarps], sel[32];
    __shared__ uint32_t list_key[kLpMaxWarps][32], list_idx[kLpMaxWarps][32];
    __shared__ uint32_t again[kLpRanked];
    __shared__ uint64_t few[kLpRanked];
    __shared__ int reached, ranked;
    constexpr int VEC = RowView<T>::VEC;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const uint32_t rank = CLUSTER ? cluster_ctarank() : 0, ctas = CLUSTER ? cluster_nctarank() : 1;
    const int64_t r = blockIdx.x / ctas;
    if (CLUSTER) cluster_started_arrive();
    grid_dependency_wait();
    uint64_t* lists = reinterpret_cast<uint64_t*>(dynamic_smem);     // the CTAs', n entries each, in the first
    uint8_t* smem = dynamic_smem + (TOP ? ctas * kMaxTop * sizeof(uint64_t) : 0);
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
    // this CTA's chunks of whole vectors: all but the row's first and last, at most
    const int whole_from = g_first == 0 && !row.whole(0) ? 1 : 0;
    const int whole_to = row.whole((g_first + chunks) * kLpChunk - 1) ? chunks : chunks - 1;
    const T* lane_row = row.p + row.first(g_first * kLpChunk) + lane * VEC;
    auto load_partial = [&](int g, uint4 (&q)[kLpUnroll]) {
        const uint32_t none = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;      // -inf
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u) {
            const int v = (g_first + g) * kLpChunk + u * 32 + lane;
            q[u] = v < row.nvec ? row.load(v, -INFINITY) : make_uint4(none, none, none, none);
        }
    };
    auto whole = [&](int g) { return g >= whole_from && g < whole_to; };       // the same for the whole warp
    auto load_chunk = [&](int g, uint4 (&q)[kLpUnroll]) {
        if (!whole(g)) return load_partial(g, q);
        const T* p = lane_row + g * (kLpChunk * VEC);
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u) q[u] = ld_v4(p + u * 32 * VEC);
    };
    // The pass copies each warp's next two chunks to shared memory while it works on one; every
    // lane copies and takes its own vectors: no barrier.  With n = 8, 4096 x 128000 FP32 take 301
    // us so and 319 with plain loads, 700 rows 60 and 67; one chunk ahead is enough for neither
    // type (8192 x 127901 BF16: 323 against 312 us).
    uint4* ring = reinterpret_cast<uint4*>(smem) + warp * kLpAhead * kLpChunk + lane;
    auto prefetch = [&](int g, int slot) {
        if (whole(g)) {
            const T* p = lane_row + g * (kLpChunk * VEC);
#pragma unroll
            for (int u = 0; u < kLpUnroll; ++u) cp_async_16(ring + slot * kLpChunk + u * 32, p + u * 32 * VEC);
        }
        cp_async_commit();
    };
    auto take_chunk = [&](int g, int slot, uint4 (&q)[kLpUnroll]) {
        if (!whole(g)) {
            load_partial(g, q);
        } else {
            cp_async_wait<kLpAhead - 1>();
#pragma unroll
            for (int u = 0; u < kLpUnroll; ++u) q[u] = ring[slot * kLpChunk + u * 32];
        }
    };

    // For the top list: the upper half of the lanes' maxima of every kGroup chunks of a warp: of
    // every two, which leaves the copies more shared memory (8192 rows: 4 us less), or in a
    // cluster of every one, as then less is read again (64 x 50001 BF16: 0.7 us less).
    const int n = a.n_top;
    constexpr int kGroup = CLUSTER ? 1 : 2;
    uint16_t* kept = reinterpret_cast<uint16_t*>(smem + kLpAhead * warps * kLpChunk * sizeof(uint4));
    const bool keep = a.keep;                                // room for them, in every CTA of the launch
    float lane_top = -INFINITY, group_top = -INFINITY;
    int round = 0, slot = 0;
    if (TOP && threadIdx.x == 0) reached = ranked = 0;
    LaneSums lane_sums;
    lane_sums.init();
    const bool first = rank == 0 && threadIdx.x == 0;
    Id target = (Id)-1;
    T target_logit = 0;
    if (first && a.targets) target = ((const Id*)a.targets)[r];
#pragma unroll
    for (int d = 0; d < kLpAhead; ++d) prefetch(warp + d * warps, d);
    for (int g = warp; g < chunks; g += warps) {
        uint4 q[kLpUnroll];
        take_chunk(g, slot, q);
        prefetch(g + kLpAhead * warps, slot);
        slot = slot + 1 == kLpAhead ? 0 : slot + 1;
        const float top = lane_max<T>(q);
        if constexpr (TOP) {
            lane_top = fmaxf(lane_top, top);
            group_top = kGroup > 1 && round % kGroup ? fmaxf(group_top, top) : top;
            if (keep) kept[(round / kGroup * warps + warp) * 32 + lane] = (uint16_t)(__float_as_uint(group_top) >> 16);
            ++round;
        }
        if (top > lane_sums.m) lane_sums.raise(top, c2);
        lane_sums.template add<T>(q, c2);
    }
    if (target >= 0 && (int64_t)target < a.V) target_logit = row.p[target];
    RowSums sums = lane_sums.total();
    // Each of the first `voters` warps casts its j-th best lane maximum, voters * j >= n: the lowest
    // of these votes is a bound that n logits reach.  (A warp with a single chunk that does not
    // fill its lanes stands aside if others can vote.)
    int voters = min(warps, chunks);
    if (voters > 1 && chunks <= warps && (g_first + chunks - 1) * kLpChunk + 31 >= row.nvec) --voters;
    if (TOP && warp < voters) {
        uint32_t key = (g_first + warp) * kLpChunk + lane < row.nvec ? order_of(lane_top) : 0u;
        uint32_t nth = 0u;
        for (int i = 0; i < n; i += voters) {
            nth = __reduce_max_sync(0xffffffffu, key);
            if (lane == __ffs(__ballot_sync(0xffffffffu, key == nth)) - 1) key = 0u;
        }
        if (lane == 0) vote[warp] = nth;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        RowSums other;
        other.m = __shfl_xor_sync(0xffffffffu, sums.m, o);
        other.s = __shfl_xor_sync(0xffffffffu, sums.s, o);
        other.t = __shfl_xor_sync(0xffffffffu, sums.t, o);
        sums.merge(other, c2);
    }
    if (CLUSTER) {
        // every CTA of the cluster gets every warp's sums
        __syncwarp();
        cluster_started_wait();
        if (lane < (int)ctas) {
            RowSums* p = &warp_sums[rank * warps + warp];
            st_cluster_f32(&p->m, lane, sums.m);
            st_cluster_f32(&p->s, lane, sums.s);
            st_cluster_f32(&p->t, lane, sums.t);
        }
        if (TOP) __syncthreads();
    } else {
        if (lane == 0) warp_sums[warp] = sums;
        __syncthreads();
    }
    if constexpr (TOP) {
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
        // place i of the CTA's list
        auto put = [&](int i, uint64_t entry) {
            if (CLUSTER) st_cluster_u64(&lists[rank * n + i], 0, entry);
            else lists[i] = entry;
        };
        bool general = true;
        if (keep) {
            // the lanes' shares of chunks that reach the bound; their logits that do; and these ones'
            // places, by comparing all of them
            const uint32_t lowest = __reduce_min_sync(0xffffffffu, lane < voters ? vote[lane] : 0xFFFFFFFFu);
            const uint32_t masked = order_of(-INFINITY);
            const float last = value_of(lowest);
            const float last_half = __uint_as_float(__float_as_uint(last) & 0xFFFF0000u);
            for (int c = warp, k = warp; c < chunks; c += kGroup * warps, k += warps) {
                const float top = __uint_as_float((uint32_t)kept[k * 32 + lane] << 16);
                if (top > -INFINITY && (lowest == 0u || top >= last_half)) {
                    const int at = atomicAdd(&reached, 1);
                    if (at < kLpRanked) again[at] = (uint32_t)(c * 32 + lane);
                }
            }
            __syncthreads();
            for (int i = threadIdx.x; i < min(reached, kLpRanked) * (kGroup * kLpUnroll); i += blockDim.x) {
                const uint32_t share = again[i / (kGroup * kLpUnroll)];
                const int g = (int)(share / 32) + i / kLpUnroll % kGroup * warps;
                const int v = (g_first + g) * kLpChunk + i % kLpUnroll * 32 + (int)(share % 32);
                if (g >= chunks || v >= row.nvec) continue;
                const int j0 = row.first(v);
                unsigned hits = 0u;
                auto test = [&](int e, float x) {
                    if (x > -INFINITY && (lowest == 0u || x >= last)) hits |= 1u << e;
                };
                if (row.whole(v)) {
                    float x[VEC];
                    RowView<T>::unpack(ld_v4(row.p + j0), x);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) test(e, x[e]);
                } else {
#pragma unroll 1
                    for (int e = 0; e < VEC; ++e)
                        if (j0 + e >= 0 && j0 + e < a.V) test(e, to_f32<T>(row.p[j0 + e]));
                }
                for (; hits; hits &= hits - 1u) {
                    const int jj = j0 + __ffs(hits) - 1, at = atomicAdd(&ranked, 1);
                    if (at < kLpRanked) few[at] = pack_entry(order_of(to_f32<T>(row.p[jj])), (uint32_t)jj);
                }
            }
            __syncthreads();
            const int j0 = max(0, row.first(g_first * kLpChunk));        // this CTA's first logit
            const int need = min(n, chunks ? min(a.V, row.first((g_first + chunks) * kLpChunk)) - j0 : 0);
            // Fewer unmasked logits than places (they have all been set aside then): masked ones
            // follow, the lowest indices, which are among the first `need`.
            unsigned rest = 0u;
            if (ranked < need && lowest <= masked)
                rest = __ballot_sync(0xffffffffu, lane < need && to_f32<T>(row.p[j0 + lane]) == -INFINITY);
            if (reached <= kLpRanked && ranked <= kLpRanked && ranked + __popc(rest) >= need) {
                general = false;
                // four lanes compare an entry
                for (int i0 = warp * 8; i0 < ranked; i0 += warps * 8) {
                    const int i = i0 + lane / 4;
                    const uint64_t own = i < ranked ? few[i] : ~(uint64_t)0;
                    int place = 0;
                    for (int o = lane % 4; o < ranked; o += 4) place += few[o] > own;
                    place += __shfl_xor_sync(0xffffffffu, place, 1);
                    place += __shfl_xor_sync(0xffffffffu, place, 2);
                    if (lane % 4 == 0 && i < ranked && place < n) put(place, own);
                }
                if (warp == 0) {
                    const int place = ranked + __popc(rest & ((1u << lane) - 1u));
                    if (rest >> lane & 1 && place < need) put(place, pack_entry(masked, (uint32_t)(j0 + lane)));
                    if (lane >= need && lane < n) put(lane, pack_entry(0u, kNone));
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
            if (warp == 0 && lane < n) put(lane, pack_entry(list.key, list.idx));
        }
    }
    // the sums of the row's warps, the same bits in every thread of the cluster
    if (CLUSTER) {
        sync_cluster();
        sums.init();
        for (int i = lane; i < warps * (int)ctas; i += 32) sums.merge(warp_sums[i], c2);
#pragma unroll 1
        for (int o = 16; o >= kLpMaxWarps; o >>= 1) {
            RowSums other;
            other.m = __shfl_xor_sync(0xffffffffu, sums.m, o);
            other.s = __shfl_xor_sync(0xffffffffu, sums.s, o);
            other.t = __shfl_xor_sync(0xffffffffu, sums.t, o);
            sums.merge(other, c2);
        }
    } else {
        if (TOP) __syncthreads();
        sums.init();
        if (lane < warps) sums = warp_sums[lane];
    }
    for (int o = kLpMaxWarps / 2; o; o >>= 1) {
        RowSums other;
        other.m = __shfl_xor_sync(0xffffffffu, sums.m, o);
        other.s = __shfl_xor_sync(0xffffffffu, sums.s, o);
        other.t = __shfl_xor_sync(0xffffffffu, sums.t, o);
        sums.merge(other, c2);
    }
    sums.m = __shfl_sync(0xffffffffu, sums.m, 0);
    sums.s = __shfl_sync(0xffffffffu, sums.s, 0);
    sums.t = __shfl_sync(0xffffffffu, sums.t, 0);
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
                for (int i = 0; i < VEC; ++i) cs.add(x[i], a.scale);
            }
        }
        for (int o = 16; o; o >>= 1) {
            CarefulSums other;
            other.m = __shfl_xor_sync(0xffffffffu, cs.m, o);
            other.s = __shfl_xor_sync(0xffffffffu, cs.s, o);
            other.t = __shfl_xor_sync(0xffffffffu, cs.t, o);
            cs.merge(other, a.scale);
        }
        if (lane == 0) warp_careful[warp] = cs;
        __syncthreads();
        cs = warp_careful[0];
        for (int w = 1; w < warps; ++w) cs.merge(warp_careful[w], a.scale);
        if (CLUSTER) {
            if (threadIdx.x == 0) cta_careful = cs;
            sync_cluster();
            cs.init();
            for (uint32_t k = 0; k < ctas; ++k) {
                CarefulSums o;
                o.m = ld_cluster_f32(&cta_careful.m, k), o.s = ld_cluster_f32(&cta_careful.s, k);
                o.t = ld_cluster_f32(&cta_careful.t, k);
                cs.merge(o, a.scale);
            }
            sync_cluster();                                          // remote sums have been read
        }
        m = cs.m;
        ls = cs.s == 0.f ? -INFINITY : logf(cs.s);                   // 0: masked throughout
        entropy = cs.s == 0.f ? 0.f : ls - cs.t / cs.s;
    } else {
        const float l2 = log2f(sums.s);
        ls = kLn2 * l2;
        entropy = kLn2 * (l2 - sums.t / sums.s);
    }
    if (entropy < 0.f) entropy = 0.f;                                // by rounding; NaN stays
    const bool empty = ls == -INFINITY;
    // (-inf for a masked logit, but NaN where the row's sum is)
    auto logp_of = [&](float x) { return empty ? -INFINITY : scaled_difference(x, m, a.scale) - ls; };
    if (first) {
        if (a.targets) {
            float lp = 0.f;
            if (target >= 0 && (int64_t)target < a.V) lp = logp_of(to_f32<T>(target_logit));
            else if (target >= 0) set_status(a.ws, MOE_ERR_DEVICE_CHECK);
            a.logp[r] = lp;
        }
        if (a.entropy) a.entropy[r] = entropy;
        if (a.stats) {
            a.stats[2 * r] = m;
            a.stats[2 * r + 1] = ls;
        }
    }
    if constexpr (TOP) {
        auto write_top = [&](int i, uint64_t entry) {
            const uint32_t key = (uint32_t)(entry >> 32);
            a.top_idx[r * n + i] = (int32_t)~(uint32_t)entry;
            a.top_logp[r * n + i] = logp_of(value_of(key));
        };
        if (!CLUSTER) {
            if (threadIdx.x < n) write_top(threadIdx.x, lists[threadIdx.x]);
        } else if (rank == 0) {
            // an entry's place is the number of entries above it in every list, each in order
            for (int i = threadIdx.x; i < n * (int)ctas; i += blockDim.x) {
                const uint64_t own = lists[i];
                int above[kLpMaxCluster] = {}, place = 0;
#pragma unroll 1
                for (int step = kMaxTop; step; step /= 2) {
#pragma unroll
                    for (int l = 0; l < kLpMaxCluster; ++l) {
                        const int at = above[l] + step - 1;
                        if (l < (int)ctas && at < n && lists[l * n + at] > own) above[l] += step;
                    }
                }
#pragma unroll
                for (int l = 0; l < kLpMaxCluster; ++l) place += above[l];
                if (place < n && own != pack_entry(0u, kNone)) write_top(place, own);
            }
        }
    }
}

template <typename T, bool TOP, bool CLUSTER>
static auto pick_logprobs(int id_bytes) -> void (*)(LogprobArgs) {
    return id_bytes == 8 ? logprobs_kernel<T, int64_t, TOP, CLUSTER> : logprobs_kernel<T, int32_t, TOP, CLUSTER>;
}
template <typename T>
static auto pick_logprobs(bool top, bool cluster, int id_bytes) -> void (*)(LogprobArgs) {
    return top ? (cluster ? pick_logprobs<T, true, true>(id_bytes) : pick_logprobs<T, true, false>(id_bytes))
               : (cluster ? pick_logprobs<T, false, true>(id_bytes) : pick_logprobs<T, false, false>(id_bytes));
}

cudaError_t launch_token_logprobs(const LogprobCall& c, cudaStream_t stream) {
    if (c.T == 0) return cudaSuccess;
    LogprobArgs a{c.logits, (int)c.V, c.ld, c.scale, !fast_scale(c.scale), 0, c.targets, c.logp,
                  c.entropy, c.stats, c.n_top, c.top_idx, c.top_logp, c.ws};
    const int64_t vec = 16 / (int64_t)dtype_bytes(c.dtype);
    const int64_t chunks = (c.V + 2 * vec - 2) / (vec * kLpChunk) + 1;         // at most, at any alignment
    // Eight warps per row, in a cluster of CTAs while these fill at most 13/16 of the places (not
    // every place takes a cluster; 128000 FP32, n = 5: 76 rows take 14.4 us in 304 CTAs and 16.5
    // in 608, 150 rows 21 us in 300 CTAs and 25 in 600).  Somewhat more rows than places: four
    // warps, which all fit at once (128000 FP32, n = 8: 700 rows take 60 us so and 78 in two
    // waves of eight warps, but 1216 rows 123 and 104).
    const int64_t eights = 4 * (int64_t)c.num_sms;                             // CTAs resident at once
    const int most = c.T > eights && c.T <= eights * 5 / 4 ? 4 : kLpMaxWarps;
    int warps = 1, ctas = 1;
    while (warps < most && warps < chunks) warps *= 2;
    while (ctas < kLpMaxCluster && chunks > (int64_t)warps * ctas && c.T * ctas * 2 <= eights * 13 / 16) ctas *= 2;
    const size_t ahead = (size_t)kLpAhead * warps * kLpChunk * sizeof(uint4);
    const size_t share = c.n_top ? (size_t)((chunks + ctas - 1) / ctas) : 0;
    const size_t per = (size_t)(ctas > 1 ? 1 : 2) * warps;
    const size_t groups = (share + per - 1) / per * warps;           // of chunks c, c + warps, ...
    a.keep = c.n_top && groups <= kLpKept;
    const size_t kept = ahead + (a.keep ? 64 * groups : 0), maxima = sizeof(uint32_t) * share;
    const size_t smem = (c.n_top ? ctas * kMaxTop * sizeof(uint64_t) : 0) + (kept > maxima ? kept : maxima);
    void (*k)(LogprobArgs) = c.dtype == MOE_F32 ? pick_logprobs<float>(c.n_top > 0, ctas > 1, c.id_bytes)
                                               : pick_logprobs<uint16_t>(c.n_top > 0, ctas > 1, c.id_bytes);
    cudaError_t err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kLpMaxSmem);
    if (err != cudaSuccess) return err;
    return launch_after(k, c.T * ctas, 32 * warps, smem, ctas, stream, a);
}

// ------------------------------------------------------------------------ gradient
// d x_j = p_j (g1 + g2 lp_j) + 1[j = t] scale g_logp with g2 = -scale g_entropy and
// g1 = -scale (g_logp + g_entropy entropy).  dlogits may be the logits' own buffer: a thread
// reads its elements before it writes them.  The kernel moves each logit in and its
// gradient out once, HBM-bound: 4096 x 128000 BF16 in 297 us (7.1 TB/s, part of the logits still in
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
    float lp = scaled_difference(x, g.m, g.scale) - g.ls;
    if (lp < -1e4f) lp = -1e4f;                                      // NaN stays
    const float e = exp2_approx(lp * (0.5f * kLog2e));
    return e * e * fmaf(lp, g.g2, g.g1);
}

template <typename T, typename Id, bool VECTOR>
__global__ void __launch_bounds__(kGradThreads) logprobs_grad_kernel(const __grid_constant__ LogprobGradArgs a) {
    constexpr int VEC = RowView<T>::VEC;
    grid_dependency_wait();
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
    // scales outside the fast path's range come last: what they meet may be 0, and then the result is
    const float before = a.careful ? 1.f : a.scale, after = a.careful ? a.scale : 1.f;
    if (a.g_logp) {
        const Id target = ((const Id*)a.targets)[r];
        gl = a.g_logp[r] * before;
        if (target >= 0 && (int64_t)target < a.V) t = (int)target;
        else gl = 0.f;
        if ((int64_t)target >= a.V && v0 == 0 && threadIdx.x == 0) set_status(a.ws, MOE_ERR_DEVICE_CHECK);
    }
    if (a.g_entropy) ge = a.g_entropy[r] * before, h = a.entropy[r];
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
            out[j] = from_f32<T>(empty ? 0.f : d * after);
        }
    }
}

template <typename T, typename Id>
static cudaError_t launch_grad_t(LogprobGradArgs& a, cudaStream_t stream) {
    constexpr int64_t VEC = 16 / sizeof(T);
    const bool vec = (((uintptr_t)a.logits - (uintptr_t)a.dlogits) & 15) == 0 &&
                     ((a.ld - a.ld_d) * (int64_t)sizeof(T)) % 16 == 0;
    a.blocks_per_row = (int)(((a.V + 2 * VEC - 2) / VEC + kGradVectors - 1) / kGradVectors);
    auto* k = vec ? logprobs_grad_kernel<T, Id, true> : logprobs_grad_kernel<T, Id, false>;
    return launch_after(k, a.T * a.blocks_per_row, kGradThreads, 0, 1, stream, a);
}

cudaError_t launch_token_logprobs_backward(const LogprobGradCall& c, cudaStream_t stream) {
    if (c.T == 0) return cudaSuccess;
    LogprobGradArgs a{c.logits, c.T, (int)c.V, c.ld, c.scale, !fast_scale(c.scale), c.targets, c.stats,
                      c.entropy, c.g_logp, c.g_entropy, c.dlogits, c.ld_d, 0, c.ws};
    if (c.dtype == MOE_F32)
        return c.id_bytes == 8 ? launch_grad_t<float, int64_t>(a, stream) : launch_grad_t<float, int32_t>(a, stream);
    return c.id_bytes == 8 ? launch_grad_t<uint16_t, int64_t>(a, stream) : launch_grad_t<uint16_t, int32_t>(a, stream);
}

}  // namespace moe
