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

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The same with subnormal results: the gradient multiplies small probabilities by what may
// be large.
__device__ __forceinline__ float exp2_full(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Running maximum, sum and first moment of a row's exponentials, relative to m:
// s = sum exp(c d), t = sum d exp(c d), d = x - m.  m starts at the lowest finite value,
// so masked logits give d = -inf, exp 0.
struct RowSums {
    float m, s, t;
    __device__ void init() {
        m = -FLT_MAX;
        s = t = 0.f;
    }
    // moves the reference point up to m2 >= m
    __device__ void raise(float m2, float c2) {
        const float d = m - m2, f = exp2_approx(d * c2);
        t = f > 0.f ? f * fmaf(d, s, t) : 0.f;       // f = 0 may meet d = -inf
        s *= f;
        m = m2;
    }
    __device__ void add(float x, float c2) {
        const float d = x - m, e = exp2_approx(d * c2);
        s += e;
        t = fmaf(e, fmaxf(d, -FLT_MAX), t);          // a masked logit's 0 * -inf is 0
    }
    __device__ void merge(RowSums o, float c2) {
        if (o.m > m) raise(o.m, c2);
        else o.raise(m, c2);
        s += o.s;
        t += o.t;
    }
};

// A row as 16-byte vectors of its own alignment: vector v holds the elements
// v*VEC - mis .. v*VEC - mis + VEC - 1; the first and the last may be partial.
template <typename T>
struct RowView {
    static constexpr int VEC = 16 / sizeof(T);
    const T* p;
    int64_t V;
    int mis;
    int nvec;
    __device__ RowView(const T* row, int64_t V_) : p(row), V(V_) {
        mis = (int)(((uintptr_t)row / sizeof(T)) % VEC);
        nvec = (int)((V + mis + VEC - 1) / VEC);
    }
    __device__ int64_t first(int v) const { return (int64_t)v * VEC - mis; }
    __device__ bool whole(int v) const { return v >= (mis ? 1 : 0) && first(v) + VEC <= V; }
    // the vector's elements; fill past the row
    __device__ uint4 load(int v, float fill) const {
        const int64_t j = first(v);
        if (whole(v)) return ld_nc_v4(p + j);
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

// The best entry over the warp by (key descending, index ascending); every lane gets it.
__device__ __forceinline__ void warp_best(uint32_t key, uint32_t idx, uint32_t* best_key, uint32_t* best_idx) {
    *best_key = __reduce_max_sync(0xffffffffu, key);
    *best_idx = __reduce_min_sync(0xffffffffu, key == *best_key ? idx : 0xFFFFFFFFu);
}

// A warp's sorted list, entry i in lane i.  Inserts (k, j) if it beats entry n-1.
struct WarpList {
    uint32_t key, idx;
    __device__ void init() { key = 0, idx = 0xFFFFFFFFu; }
    __device__ static bool beats(uint32_t k, uint32_t j, uint32_t k2, uint32_t j2) {
        return k > k2 || (k == k2 && j < j2);
    }
    __device__ void insert(uint32_t k, uint32_t j) {
        const int lane = threadIdx.x % 32;
        const unsigned after = __ballot_sync(0xffffffffu, beats(k, j, key, idx));   // entries that move down
        const uint32_t up_key = __shfl_up_sync(0xffffffffu, key, 1), up_idx = __shfl_up_sync(0xffffffffu, idx, 1);
        if (after >> lane & 1) {
            const bool here = lane == __ffs(after) - 1;
            key = here ? k : up_key;
            idx = here ? j : up_idx;
        }
    }
};

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32;
constexpr int kLpUnroll = 4;

struct LogprobArgs {
    const void* logits;
    int64_t V, ld;
    float scale;
    const void* targets;
    float *logp, *entropy, *stats;
    int n_top;
    int32_t* top_idx;
    float* top_logp;
    WsHeader* ws;
};

// One CTA per row, one pass over it.  For the top list the pass only keeps the maximum of
// each chunk of 32 vectors (what a warp reads at once).  The n best logits lie in the n best
// chunks by (maximum, position): a chunk below those has n chunks before it, each with a
// logit that beats all of its own.  So n chunks are read again, from L2, whatever the
// logits are.
template <typename T, typename Id>
__global__ void __launch_bounds__(kLpThreads, 4) logprobs_kernel(const __grid_constant__ LogprobArgs a) {
    extern __shared__ uint32_t chunk_max[];                  // order_of the chunk's maximum; 0: taken
    __shared__ RowSums warp_sums[kLpWarps];
    __shared__ uint32_t sel[kMaxTop];
    __shared__ uint32_t list_key[kLpWarps][kMaxTop], list_idx[kLpWarps][kMaxTop];
    constexpr int VEC = RowView<T>::VEC;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t r = blockIdx.x;
    const RowView<T> row((const T*)a.logits + r * a.ld, a.V);
    const int chunks = (row.nvec + 31) / 32;
    const float c2 = a.scale * kLog2e;
    RowSums sums;
    sums.init();
    for (int g0 = warp; g0 < chunks; g0 += kLpWarps * kLpUnroll) {
        uint4 q[kLpUnroll];
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u) {
            const int v = (g0 + u * kLpWarps) * 32 + lane;
            const uint32_t none = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;      // -inf
            q[u] = v < row.nvec ? row.load(v, -INFINITY) : make_uint4(none, none, none, none);
        }
        float x[kLpUnroll][VEC], top = -INFINITY;
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u) {
            RowView<T>::unpack(q[u], x[u]);
            float mx = x[u][0];
#pragma unroll
            for (int i = 1; i < VEC; ++i) mx = fmaxf(mx, x[u][i]);
            top = fmaxf(top, mx);
            if (a.n_top) {
                const uint32_t o = __reduce_max_sync(0xffffffffu, max(order_of(mx), 1u));
                if (lane == 0 && g0 + u * kLpWarps < chunks) chunk_max[g0 + u * kLpWarps] = o;
            }
        }
        if (top > sums.m) sums.raise(top, c2);
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u)
#pragma unroll
            for (int i = 0; i < VEC; ++i) sums.add(x[u][i], c2);
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
    sums = warp_sums[0];
    for (int w = 1; w < kLpWarps; ++w) sums.merge(warp_sums[w], c2);
    const bool empty = sums.s == 0.f;
    const float ls = empty ? -INFINITY : logf(sums.s);
    auto logp_of = [&](float x) { return empty || x == -INFINITY ? -INFINITY : (x - sums.m) * a.scale - ls; };
    if (threadIdx.x == 0) {
        if (a.targets) {
            const Id t = ((const Id*)a.targets)[r];
            float lp = 0.f;
            if (t >= 0 && (int64_t)t < a.V) lp = logp_of(to_f32<T>(row.p[t]));
            else if (t >= 0) set_status(a.ws, MOE_ERR_DEVICE_CHECK);
            a.logp[r] = lp;
        }
        if (a.entropy) a.entropy[r] = empty ? 0.f : ls - a.scale * (sums.t / sums.s);
        if (a.stats) {
            a.stats[2 * r] = sums.m;
            a.stats[2 * r + 1] = ls;
        }
    }
    if (!a.n_top) return;

    // the n best chunks, by one warp: each lane watches every 32nd chunk
    if (warp == 0) {
        uint32_t best = 0, at = 0xFFFFFFFFu;
        auto rescan = [&]() {
            best = 0, at = 0xFFFFFFFFu;
            for (int g = lane; g < chunks; g += 32)
                if (chunk_max[g] > best) best = chunk_max[g], at = g;
        };
        rescan();
        for (int i = 0; i < a.n_top; ++i) {
            uint32_t k, g;
            warp_best(best, at, &k, &g);
            if (lane == 0) sel[i] = g;                       // 0xFFFFFFFF: fewer than n chunks
            if (g == 0xFFFFFFFFu) continue;
            if (g % 32 == (uint32_t)lane) {
                chunk_max[g] = 0;
                rescan();
            }
        }
    }
    __syncthreads();
    // each warp lists the best of its share of those chunks
    WarpList list;
    list.init();
    for (int i = warp; i < a.n_top; i += kLpWarps) {
        if (sel[i] == 0xFFFFFFFFu) break;
        const int v = (int)sel[i] * 32 + lane;
        float x[VEC];
        const bool in = v < row.nvec;
        RowView<T>::unpack(in ? row.load(v, 0.f) : make_uint4(0, 0, 0, 0), x);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int64_t j = in ? row.first(v) + e : -1;
            const uint32_t key = order_of(x[e]);
            const bool real = j >= 0 && j < a.V;
            const uint32_t last_key = __shfl_sync(0xffffffffu, list.key, a.n_top - 1);
            const uint32_t last_idx = __shfl_sync(0xffffffffu, list.idx, a.n_top - 1);
            unsigned todo = __ballot_sync(0xffffffffu, real && WarpList::beats(key, (uint32_t)j, last_key, last_idx));
            while (todo) {
                const int src = __ffs(todo) - 1;
                todo &= todo - 1;
                list.insert(__shfl_sync(0xffffffffu, key, src), (uint32_t)__shfl_sync(0xffffffffu, (uint32_t)j, src));
            }
        }
    }
    if (lane < a.n_top) {
        list_key[warp][lane] = list.key;
        list_idx[warp][lane] = list.idx;
    }
    __syncthreads();
    // merge the lists: lane w holds warp w's next entry
    if (warp == 0) {
        int at = 0;
        uint32_t k = lane < kLpWarps ? list_key[lane][0] : 0, j = lane < kLpWarps ? list_idx[lane][0] : 0xFFFFFFFFu;
        for (int i = 0; i < a.n_top; ++i) {
            uint32_t bk, bj;
            warp_best(k, j, &bk, &bj);
            if (lane == 0) {
                a.top_idx[r * a.n_top + i] = (int32_t)bj;
                a.top_logp[r * a.n_top + i] = logp_of(value_of(bk));
            }
            if (j == bj && lane < kLpWarps) {
                ++at;
                k = at < a.n_top ? list_key[lane][at] : 0;
                j = at < a.n_top ? list_idx[lane][at] : 0xFFFFFFFFu;
            }
        }
    }
}

cudaError_t launch_token_logprobs(const LogprobCall& c, cudaStream_t stream) {
    if (c.T == 0) return cudaSuccess;
    LogprobArgs a{c.logits, c.V, c.ld, c.scale, c.targets, c.logp, c.entropy, c.stats, c.n_top, c.top_idx, c.top_logp,
                  c.ws};
    const int vec = 16 / (int)dtype_bytes(c.dtype);
    const size_t smem = c.n_top ? sizeof(uint32_t) * (size_t)((c.V + vec) / (32 * vec) + 1) : 0;
    void (*k)(LogprobArgs) =
        c.dtype == MOE_F32 ? (c.id_bytes == 8 ? logprobs_kernel<float, int64_t> : logprobs_kernel<float, int32_t>)
                           : (c.id_bytes == 8 ? logprobs_kernel<uint16_t, int64_t> : logprobs_kernel<uint16_t, int32_t>);
    cudaError_t err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    k<<<(unsigned)c.T, kLpThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

// ------------------------------------------------------------------------ gradient
// One thread per vector of a row, blockIdx.y strides over the rows.  dlogits may be the
// logits' own buffer: a thread reads its elements before it writes them.
struct LogprobGradArgs {
    const void* logits;
    int64_t T, V, ld;
    float scale;
    const void* targets;
    const float *stats, *entropy, *g_logp, *g_entropy;
    void* dlogits;
    int64_t ld_d;
    WsHeader* ws;
};

template <typename T, typename Id, bool VECTOR>
__global__ void __launch_bounds__(256) logprobs_grad_kernel(const __grid_constant__ LogprobGradArgs a) {
    const int64_t groups = (a.V + 7) / 8;
    for (int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; b < a.T * groups;
         b += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = b / groups, j = (b % groups) * 8;
        const int n = (int)(a.V - j < 8 ? a.V - j : 8);
        const float m = a.stats[2 * r], ls = a.stats[2 * r + 1];
        const bool empty = ls == -INFINITY;
        float gl = 0.f, ge = 0.f, h = 0.f;
        int64_t t = -1;
        if (a.g_logp) {
            t = (int64_t)((const Id*)a.targets)[r];
            if (t >= a.V) {
                if (j == 0) set_status(a.ws, MOE_ERR_DEVICE_CHECK);
                t = -1;
            }
            if (t >= 0) gl = a.g_logp[r] * a.scale;
        }
        if (a.g_entropy) ge = a.g_entropy[r] * a.scale, h = a.entropy[r];
        float x[8];
        load8<T, VECTOR>((const T*)a.logits + r * a.ld + j, n, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool off = empty || x[i] == -INFINITY;
            const float lp = (x[i] - m) * a.scale - ls;
            const float p = exp2_full(lp * kLog2e);
            const float d = -p * fmaf(ge, fmaxf(lp, -1e4f) + h, gl) + (j + i == t ? gl : 0.f);
            x[i] = off ? 0.f : d;
        }
        store8<T, VECTOR>((T*)a.dlogits + r * a.ld_d + j, n, x);
    }
}

template <typename T, typename Id>
static cudaError_t launch_grad_t(const LogprobGradArgs& a, bool vec, int num_sms, cudaStream_t stream) {
    const int64_t total = a.T * ((a.V + 7) / 8);
    int64_t grid = (total + 255) / 256;
    if (grid > (int64_t)num_sms * 8) grid = (int64_t)num_sms * 8;
    auto* k = vec ? logprobs_grad_kernel<T, Id, true> : logprobs_grad_kernel<T, Id, false>;
    k<<<(unsigned)grid, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_token_logprobs_backward(const LogprobGradCall& c, cudaStream_t stream) {
    if (c.T == 0) return cudaSuccess;
    LogprobGradArgs a{c.logits, c.T, c.V, c.ld, c.scale, c.targets, c.stats, c.entropy, c.g_logp, c.g_entropy,
                      c.dlogits, c.ld_d, c.ws};
    const bool vec = rows_in_groups(c.logits, c.V, c.ld, c.dtype) && rows_in_groups(c.dlogits, c.V, c.ld_d, c.dtype);
    if (c.dtype == MOE_F32)
        return c.id_bytes == 8 ? launch_grad_t<float, int64_t>(a, vec, c.num_sms, stream)
                               : launch_grad_t<float, int32_t>(a, vec, c.num_sms, stream);
    return c.id_bytes == 8 ? launch_grad_t<uint16_t, int64_t>(a, vec, c.num_sms, stream)
                           : launch_grad_t<uint16_t, int32_t>(a, vec, c.num_sms, stream);
}

}  // namespace moe
