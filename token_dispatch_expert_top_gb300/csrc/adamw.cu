// adamw.cu -- the AdamW step over many tensors, with moments in FP32 or in 8 bits, and the global
// norm of their gradients with the factor that clips it.
//
// A launch takes the list (pointers, sizes, types) as its argument: no table in device memory to
// keep up to date, and a captured graph holds its own copy.  Every tensor is cut into pieces, whose numbers
// say which tensor a block works on.
#include <float.h>
#include <math.h>

#include <type_traits>

#include "kernels.cuh"
#include "philox.cuh"
#include "pieces.cuh"
#include "vec_io.cuh"

namespace moe {
namespace {

// A kernel's arguments may hold 32764 bytes; a short list takes the small form.
constexpr int kFewTensors = 16, kManyTensors = 384;

// Which tensor of a launch's list a piece is of: first[k] is the first piece of tensor k (the largest
// number behind the last one).  Two rounds of independent comparisons: a bisection's nine rounds would
// each wait for a constant-cache miss on an SM that has not seen the list yet.
template <int CAP>
struct PieceMap {
    static constexpr int kRow = CAP < 16 ? CAP : 16, kRows = CAP / kRow;
    uint32_t row[kRows];        // first[16 k]
    uint32_t first[CAP];
    uint32_t pieces;

    PieceMap() {
        for (uint32_t& f : first) f = 0xFFFFFFFFu;
    }
    void finish(uint32_t all) {
        pieces = all;
        for (int i = 0; i < kRows; ++i) row[i] = first[i * kRow];
    }
    __device__ __forceinline__ int find(uint32_t piece) const {
        int r = 0, k = 0;
#pragma unroll
        for (int i = 1; i < kRows; ++i) r += row[i] <= piece;
#pragma unroll
        for (int i = 1; i < kRow; ++i) k += first[r * kRow + i] <= piece;
        return r * kRow + k;
    }
};

// ------------------------------------------------------------------ global norm
// Elements from the first 16-byte aligned one on, and how many lie before it.
struct GradEntry {
    const void* grad;
    int64_t n;
};
template <int CAP>
struct GradArgs {
    GradEntry e[CAP];
    PieceMap<CAP> map;
    uint32_t f32[(CAP + 31) / 32];   // bit per tensor
    uint8_t head[CAP];
    int onto;                   // add to the partial sums (a list in several launches)
    float* part;                // null: one block, which leaves the results
    float max_norm;
    float *norm, *factor;
};

// Four 16-byte loads a thread.
template <typename T>
constexpr int kGradPiece = 64 / sizeof(T);

template <typename T, int THREADS>
__device__ __forceinline__ float squares(const T* g, int64_t at, int64_t n) {
    constexpr int E = 16 / sizeof(T);
    uint4 q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t i = at + (int64_t)(k * THREADS + threadIdx.x) * E;
        if (i + E <= n) {
            q[k] = ld_v4(g + i);
        } else {
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < E; ++j) {
                if (i + j >= n) continue;
                if constexpr (sizeof(T) == 2) w[j / 2] |= (uint32_t)g[i + j] << (16 * (j % 2));
                else w[j] = __float_as_uint(g[i + j]);
            }
            q[k] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    F2 t = f2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const Piece<T, E> r{{q[k].x, q[k].y, q[k].z, q[k].w}};
        F2 v[E / 2];
        to_pairs(r, v);
#pragma unroll
        for (int j = 0; j < E / 2; ++j) t = f2_fma(v[j], v[j], t);
    }
    float a, b;
    f2_split(t, a, b);
    return a + b;
}

// Piece number `piece` of a tensor, and with the first one the elements before the aligned ones.
template <typename T, int THREADS>
__device__ __forceinline__ float piece_squares(const GradEntry& e, int head, uint32_t piece) {
    const T* g = (const T*)e.grad;
    float t = squares<T, THREADS>(g, (int64_t)piece * (THREADS * kGradPiece<T>), e.n);
    if (piece == 0 && (int)threadIdx.x < head) {
        const float v = to_f32<T>(g[(int)threadIdx.x - head]);
        t = fmaf(v, v, t);
    }
    return t;
}

// In FP32: the additions of FP64 took longer than all the rest of a small list.
__device__ __forceinline__ float block_sum(float v, float* sums) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = v;
    __syncthreads();
    v = threadIdx.x % 32 < blockDim.x / 32 ? sums[threadIdx.x % 32] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ void leave_norm(float sum, float max_norm, float* norm, float* factor) {
    const float r = __fsqrt_rn(sum);
    if (norm) *norm = r;
    if (factor) *factor = isfinite(r) ? fminf(1.f, max_norm / (r + 1e-6f)) : __int_as_float(0x7fc00000);
}

constexpr int kNormThreads = 256, kOneBlock = 1024;   // kOneBlock: a list that one block takes by itself

inline int64_t grad_pieces(const moe_adamw_tensor_t& t, int threads) {
    static_assert(kGradPiece<float> == 16 && kGradPiece<uint16_t> == 32, "powers of two");
    // (a division takes the host longer than all else that it does for a tensor)
    const int shift = (threads == kOneBlock ? 10 : 8) + (t.grad_dtype == MOE_F32 ? 4 : 5);
    return (t.n + (1ll << shift) - 1) >> shift;
}

template <int CAP, int THREADS>
__global__ void __launch_bounds__(THREADS) grad_norm_kernel(const __grid_constant__ GradArgs<CAP> a) {
    __shared__ float sums[32];
    grid_dependency_wait();
    float t = 0.f;
    for (uint32_t piece = blockIdx.x; piece < a.map.pieces; piece += gridDim.x) {
        const int k = a.map.find(piece);
        const uint32_t mine = piece - a.map.first[k];
        t += a.f32[k / 32] >> (k % 32) & 1 ? piece_squares<float, THREADS>(a.e[k], a.head[k], mine)
                                           : piece_squares<uint16_t, THREADS>(a.e[k], a.head[k], mine);
    }
    t = block_sum(t, sums);
    if (threadIdx.x) return;
    if (!a.part) leave_norm(t, a.max_norm, a.norm, a.factor);
    else a.part[blockIdx.x] = a.onto ? a.part[blockIdx.x] + t : t;
}

__global__ void __launch_bounds__(1024) grad_norm_join_kernel(const float* part, int parts, float max_norm,
                                                              float* norm, float* factor) {
    __shared__ float sums[32];
    grid_dependency_wait();
    float v = 0.f;
    for (int i = threadIdx.x; i < parts; i += 1024) v += part[i];
    v = block_sum(v, sums);
    if (threadIdx.x == 0) leave_norm(v, max_norm, norm, factor);
}

template <int CAP, int THREADS>
cudaError_t launch_grad_norm_list(const moe_adamw_tensor_t* t, int count, GradArgs<CAP>& a, int blocks,
                                  cudaStream_t stream) {
    for (uint32_t& f : a.f32) f = 0;
    uint32_t pieces = 0;
    int k = 0;
    for (int i = 0; i < count; ++i) {
        if (t[i].n == 0) continue;
        const size_t size = dtype_bytes(t[i].grad_dtype);
        int64_t head = (16 - (uintptr_t)t[i].grad % 16) % 16 / size;
        if (head > t[i].n) head = t[i].n;
        a.e[k].grad = (const uint8_t*)t[i].grad + head * size;
        a.e[k].n = t[i].n - head;
        a.head[k] = (uint8_t)head;
        a.map.first[k] = pieces;
        a.f32[k / 32] |= (uint32_t)(t[i].grad_dtype == MOE_F32) << (k % 32);
        pieces += (uint32_t)grad_pieces(t[i], THREADS);   // of all n: at least one
        ++k;
    }
    a.map.finish(pieces);
    return launch_after(grad_norm_kernel<CAP, THREADS>, blocks, THREADS, 0, 1, stream, a);
}

// ------------------------------------------------------------------ AdamW
// A list takes a launch for each kind of tensor that it has.
enum Kind { kF32Moments, kEightBf16, kEightF32 };   // moments in FP32; in 8 bits with BF16 or FP32 weights
inline Kind kind_of(const moe_adamw_tensor_t& t) {
    return t.state_dtype == MOE_F32 ? kF32Moments : t.param_dtype == MOE_F32 ? kEightF32 : kEightBf16;
}
constexpr int kStepThreads = 256, kEightThreads = 128;
// Moments in 8 bits: neighbouring blocks take the groups of a stretch in turn, so that what is read and written
// at a time lies together (352M BF16 weights, 32 groups to a block: 664 us where each has groups of its
// own in a row, 577 in turns of 4 to 256).
constexpr int kTurns = 16;
template <Kind KIND>
constexpr int kThreads = KIND == kF32Moments ? kStepThreads : kEightThreads;

struct StepEntry {
    void* param;
    void* copy;
    const void* grad;
    void* m;
    void* v;
    uint8_t* m_scales;
    uint8_t* v_scales;
    int64_t n;
    float weight_decay;
    uint16_t number;            // place in the list, from number0 on
    uint8_t param_f32, grad_f32, vec, pad[3];
};
struct StepScalars {
    float lr, beta1, beta2, one_minus_beta1, one_minus_beta2, eps;
    float log_beta1, log_beta2;            // of the bias corrections, where the step is read on the device
    float inv_bias1, inv_root_bias2;       // 1 / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
    uint32_t step;                         // low word
    const float *device_lr, *grad_scale;
    const int64_t* device_step;
    PhiloxKeys keys;
};
template <int CAP>
struct StepArgs {
    StepEntry e[CAP];
    PieceMap<CAP> map;
    uint32_t number0;           // list place of number 0
    int groups;                 // that a block has at most (moments in 8 bits)
    StepScalars s;
};

// One update's numbers, the same for all elements of a tensor; false: nothing changes.
struct Update {
    float f, beta1, beta2, c1, c2, decay, inv_root, eps;
    uint32_t step;
};
__device__ __forceinline__ bool make_update(const StepScalars& s, float weight_decay, Update& u) {
    u.f = s.grad_scale ? *s.grad_scale : 1.f;
    const float lr = s.device_lr ? *s.device_lr : s.lr;
    u.step = s.step;
    float inv_bias1 = s.inv_bias1;
    u.inv_root = s.inv_root_bias2;
    if (s.device_step) {
        const int64_t t = *s.device_step;
        if (t < 1) return false;
        u.step = (uint32_t)t;
        inv_bias1 = 1.f / -expm1f((float)t * s.log_beta1);
        u.inv_root = 1.f / sqrtf(-expm1f((float)t * s.log_beta2));
    }
    u.beta1 = s.beta1, u.beta2 = s.beta2, u.c1 = s.one_minus_beta1, u.c2 = s.one_minus_beta2;
    // -lr / (1 - beta1^t) / (root inv_root + eps), its numerator in the denominator's terms (one multiplication an
    // element less: 352M BF16 weights 577 us, 585 with it).  At FP32's ends: no rate, no step; and what has no
    // moments has no step at any rate.
    const float size = -lr * inv_bias1, by = size == 0.f ? INFINITY : 1.f / size;
    u.inv_root = copysignf(fminf(fabsf(u.inv_root * by), FLT_MAX), by);
    u.eps = copysignf(fminf(fmaxf(fabsf(s.eps * by), FLT_MIN), FLT_MAX), by);
    u.decay = -lr * weight_decay;
    if (u.decay == 0.f) u.decay = 0x1p-149f;                // nothing beside any weight; an infinite one stays
    return isfinite(u.f);
}

// New moments of pairs.  In the form m + (1 - beta) (g - m) what beta and the difference are rounded by
// weighs 1 - beta only, so that little but the last rounding is left; it needs beta >= 1/2 (below that
// the difference would cancel).  EIGHT: m is rounded towards zero, since its code goes up if m reaches a border:
// rounded to nearest, what lies less than half a last place below reaches it too (of 2.1G codes of m 1722 fell
// otherwise than in 64 bits, 1170 so; of v 950 and 345).
template <int PAIRS, bool EIGHT>
__device__ __forceinline__ void new_moments(const Update& u, const F2* g, F2* m, F2* v) {
    const F2 c1 = f2(u.c1, u.c1), c2 = f2(u.c2, u.c2);
    F2 h[PAIRS];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) h[i] = f2_mul(g[i], f2(u.f, u.f));
    if (fminf(u.beta1, u.beta2) >= 0.5f) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            const F2 d = f2_sub(h[i], m[i]);
            m[i] = EIGHT ? f2_fma_rz(c1, d, m[i]) : f2_fma(c1, d, m[i]);
            v[i] = f2_fma(c2, f2_sub(f2_mul(h[i], h[i]), v[i]), v[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            const F2 d = f2_mul(c1, h[i]), beta1 = f2(u.beta1, u.beta1);
            m[i] = EIGHT ? f2_fma_rz(beta1, m[i], d) : f2_fma(beta1, m[i], d);
            v[i] = f2_fma(f2(u.beta2, u.beta2), v[i], f2_mul(f2_mul(c2, h[i]), h[i]));
        }
    }
}

// New weights of two elements; root: sqrt(v).  The reciprocal is approximate: it moves the subtracted
// step by 2^-22 of itself, far below the weight's own rounding.  The decay is part of what is subtracted, and the
// weight is rounded once: 1 - lr weight_decay as a factor has FP32's grid below 1, which at lr weight_decay = 1e-7
// takes 19% too much of every weight alike, and at 2e-8 nothing.
__device__ __forceinline__ F2 stepped(const Update& u, F2 p, F2 m, F2 root) {
    float a, b;
    f2_split(f2_fma(root, f2(u.inv_root, u.inv_root), f2(u.eps, u.eps)), a, b);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
    return f2_add(p, f2_fma(m, f2(a, b), f2_mul(p, f2(u.decay, u.decay))));
}

// Elements at .. at + 7 (`n` in the tensor), in one or two 16-byte accesses where all are there and VEC.
template <typename T, bool VEC>
__device__ __forceinline__ Piece<T, 8> load_eight(const T* p, int64_t at, int64_t n) {
    Piece<T, 8> r;
    if (VEC && at + 8 <= n) {
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k) {
            const uint4 q = ld_v4((const uint8_t*)(p + at) + 16 * k);
            r.w[4 * k] = q.x, r.w[4 * k + 1] = q.y, r.w[4 * k + 2] = q.z, r.w[4 * k + 3] = q.w;
        }
        return r;
    }
#pragma unroll
    for (int i = 0; i < Piece<T, 8>::kWords; ++i) r.w[i] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (at + i >= n) continue;
        if constexpr (sizeof(T) == 2) r.w[i / 2] |= (uint32_t)p[at + i] << (16 * (i % 2));
        else r.w[i] = __float_as_uint(p[at + i]);
    }
    return r;
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_eight(T* p, int64_t at, int64_t n, const F2 (&v)[4]) {
    const Piece<T, 8> r = from_pairs<T, 8>(v);
    if (VEC && at + 8 <= n) {
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k)
            st_v4((uint8_t*)(p + at) + 16 * k, make_uint4(r.w[4 * k], r.w[4 * k + 1], r.w[4 * k + 2], r.w[4 * k + 3]));
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (at + i >= n) continue;
        if constexpr (sizeof(T) == 2) p[at + i] = (uint16_t)(r.w[i / 2] >> (16 * (i % 2)));
        else p[at + i] = __uint_as_float(r.w[i]);
    }
}

// ---- moments in FP32: HBM-bound
// Where a tensor does not move in groups, a thread has every kStepThreads-th element, so that lanes touch
// neighbouring ones.
template <typename T>
__device__ __forceinline__ void load_strided(const T* p, int64_t at, int64_t n, F2 (&v)[4]) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = at + i * kStepThreads < n ? to_f32<T>(p[at + i * kStepThreads]) : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2(f[2 * i], f[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ void store_strided(T* p, int64_t at, int64_t n, const F2 (&v)[4]) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_split(v[i], f[2 * i], f[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (at + i * kStepThreads < n) p[at + i * kStepThreads] = from_f32<T>(f[i]);
}

__device__ __forceinline__ F2 roots_approx(F2 v) {
    float a, b;
    f2_split(v, a, b);
    asm("sqrt.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("sqrt.approx.ftz.f32 %0, %0;" : "+f"(b));
    return f2(a, b);
}

template <typename TP, typename TG, bool VEC>
__device__ __forceinline__ void step_group(const StepEntry& e, const StepScalars& s, int64_t group) {
    const int64_t at = group * (kStepThreads * 8) + (VEC ? threadIdx.x * 8 : threadIdx.x), n = e.n;
    F2 p[4], g[4], m[4], v[4];
    if constexpr (VEC) {
        const auto rp = load_eight<TP, true>((const TP*)e.param, at, n);
        const auto rg = load_eight<TG, true>((const TG*)e.grad, at, n);
        const auto rm = load_eight<float, true>((const float*)e.m, at, n);
        const auto rv = load_eight<float, true>((const float*)e.v, at, n);
        to_pairs(rp, p), to_pairs(rg, g), to_pairs(rm, m), to_pairs(rv, v);
    } else {
        load_strided((const TP*)e.param, at, n, p);
        load_strided((const TG*)e.grad, at, n, g);
        load_strided((const float*)e.m, at, n, m);
        load_strided((const float*)e.v, at, n, v);
    }
    Update u;
    if (!make_update(s, e.weight_decay, u)) return;
    new_moments<4, false>(u, g, m, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = stepped(u, p[i], m[i], roots_approx(v[i]));
    if constexpr (VEC) {
        store_eight<float, true>((float*)e.m, at, n, m);
        store_eight<float, true>((float*)e.v, at, n, v);
        store_eight<TP, true>((TP*)e.param, at, n, p);
        if (e.copy) store_eight<uint16_t, true>((uint16_t*)e.copy, at, n, p);
    } else {
        store_strided((float*)e.m, at, n, m);
        store_strided((float*)e.v, at, n, v);
        store_strided((TP*)e.param, at, n, p);
        if (e.copy) store_strided((uint16_t*)e.copy, at, n, p);
    }
}

// ---- moments in 8 bits: E4M3 codes and a UE8M0 scale per 32 elements (four lanes of eight)
// Bound by instructions: 48 an element, where 10 bytes move in the time of 44.
__device__ __forceinline__ float scale_value(uint32_t byte) {     // 2^(byte - 127)
    return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

__device__ __forceinline__ void decode8(uint2 q, uint32_t scale, F2 (&v)[4]) {
    const float s = scale_value(scale);
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        asm("{\n\t.reg .b16 lo, hi;\n\t.reg .b32 h;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 h, lo;\n\t"
            "mov.b32 {lo, hi}, h;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
            : "=f"(a), "=f"(b)
            : "r"(i % 2 ? w[i / 2] >> 16 : w[i / 2]));
        v[i] = f2_mul(f2(a, b), f2(s, s));
    }
}

// The least power of two that keeps amax at or below 448 = 1.75 * 2^8: its byte.
__device__ __forceinline__ uint32_t state_scale(uint32_t amax_bits) {
    const uint32_t e = (amax_bits + 0x1FFFFFu) >> 23;
    return e > 8 ? e - 8 : 0;
}

// Codes of eight values under a scale, rounded up or down by 16 bits each.  x / scale, times 2^-120,
// has E4M3's exponent (bias 7) in FP32's exponent field, with E4M3's subnormal numbers where FP32's
// are: the sign and bits 20 to 26 are the code, and what lies below them is the distance to it from the code
// below, to which the random bits are added.  The second moment takes the neighbour's bits.  For values
// up to kPlainMost, all finite.
constexpr uint32_t kPlainMost = 0x46E00000u;                // 448 * 2^6: scales up to 2^6
template <bool POSITIVE>
__device__ __forceinline__ uint2 encode8(const F2 (&x)[4], uint32_t scale, const uint32_t (&bits)[4]) {
    const float by = __uint_as_float((134 - scale) << 23);  // 2^(7 - scale) = 2^(127 - scale) 2^-120
    uint32_t t[8], w[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float f[2];
        f2_split(f2_mul(x[i], f2(by, by)), f[0], f[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t b = __float_as_uint(f[k]);
            // the code in the upper byte: bits 20 to 26, and their distance, times 16
            t[2 * i + k] = b * 16 + __byte_perm(bits[i], 0, k == POSITIVE ? 0x4104 : 0x4324);
            if (!POSITIVE) t[2 * i + k] = (t[2 * i + k] & 0x7FFFFFFFu) | (b & 0x80000000u);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        w[i] = __byte_perm(__byte_perm(t[4 * i], t[4 * i + 1], 0x73), __byte_perm(t[4 * i + 2], t[4 * i + 3], 0x73), 0x5410);
        if (POSITIVE && ((w[i] - 0x01010101u) & ~w[i] & 0x80808080u)) {     // a zero among them (below 0x80 all)
#pragma unroll
            for (int k = 0; k < 4; ++k) {                   // at least the first code for what is not zero
                float f[2];
                f2_split(x[2 * i + k / 2], f[0], f[1]);
                if (!(w[i] >> (8 * k) & 0xFF) && f[k % 2] != 0.f) w[i] |= 1u << (8 * k);
            }
        }
    }
    return make_uint2(w[0], w[1]);
}

// The same for any values.
__device__ __noinline__ uint2 encode8_any(F2 x0, F2 x1, F2 x2, F2 x3, uint32_t scale, uint4 bits, bool positive) {
    const F2 x[4] = {x0, x1, x2, x3};
    const uint32_t word[4] = {bits.x, bits.y, bits.z, bits.w};
    // 2^(7 - scale), which is below FP32's normal numbers from 134 on, in two factors
    const float one = __uint_as_float(scale > 133 ? (254 - scale) << 23 : (134 - scale) << 23);
    const float two = scale > 133 ? 0x1p-120f : 1.f;
    uint32_t half[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float f[2];
        f2_split(x[i], f[0], f[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t chance = k == positive ? word[i] & 0xFFFF : word[i] >> 16;
            uint32_t sum = __float_as_uint(f[k] * one * two) + chance * 16;
            if (positive) sum = max(sum, min(__float_as_uint(f[k]), 0x00100000u));
            // now exact in E4M3; 0 x makes it a NaN where x is not finite
            f[k] = fmaf(__uint_as_float(sum & 0xFFF00000u), 0x1p120f, f[k] * 0.f);
        }
        half[i] = cvt_e4m3x2(f[0], f[1]);
    }
    return make_uint2(half[0] | half[1] << 16, half[2] | half[3] << 16);
}

// Largest magnitude of a block, as its bits: of its numbers, or of all values, NaN above any number.
template <bool NUMBERS>
__device__ __forceinline__ uint32_t block_max(const F2 (&x)[4]) {
    float f[8], m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_split(x[i], f[2 * i], f[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        if constexpr (NUMBERS) asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(f[i]), "f"(f[i + 1]));
        else asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(f[i]), "f"(f[i + 1]));
    }
    uint32_t top = __float_as_uint(m);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    return max(top, __shfl_xor_sync(0xffffffffu, top, 2));
}

// sqrt(v): v times its approximate inverse root, and one Newton step, rounded towards zero as m is.  Below FP32's normal numbers the
// inverse root is infinite; limited to 1e19 it leaves 0 for 0, and at most 1e-19 for what is not.
__device__ __forceinline__ F2 roots(F2 v) {
    float a, b, x, y;
    f2_split(v, x, y);
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(x));
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(y));
    const F2 r = f2(fminf(a, 1e19f), fminf(b, 1e19f));
    const F2 root = f2_mul(v, r);
    return f2_fma_rz(f2_mul(root, f2(-0.5f, -0.5f)), f2_fma(root, r, f2(-1.f, -1.f)), root);
}

template <bool VEC>
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int64_t at, int64_t n) {
    if (VEC && at + 8 <= n) return *reinterpret_cast<const uint2*>(p + at);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (at + i < n) w[i / 4] |= (uint32_t)p[at + i] << (8 * (i % 4));
    return make_uint2(w[0], w[1]);
}
template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t at, int64_t n, uint2 q) {
    if (VEC && at + 8 <= n) {
        *reinterpret_cast<uint2*>(p + at) = q;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (at + i < n) p[at + i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i % 4)));
}

// The update of a group of eight: codes and scales in, new ones out; p, g as pairs.
__device__ __forceinline__ void update_eight(const Update& u, const StepScalars& s, uint32_t number, int64_t at,
                                             F2 (&p)[4], const F2 (&g)[4], uint2& qm, uint2& qv, uint32_t& sm,
                                             uint32_t& sv) {
    F2 m[4], root[4];
    decode8(qm, sm, m);
    decode8(qv, sv, root);
#pragma unroll
    for (int i = 0; i < 4; ++i) root[i] = f2_mul(root[i], root[i]);
    new_moments<4, true>(u, g, m, root);
#pragma unroll
    for (int i = 0; i < 4; ++i) root[i] = roots(root[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = stepped(u, p[i], m[i], root[i]);
    uint32_t bits[4] = {(uint32_t)(at / 8), (uint32_t)((uint64_t)at >> 35), u.step, number};
    philox_10(bits, s.keys);
    const uint32_t top_m = block_max<false>(m), top_v = block_max<false>(root);
    if (__any_sync(0xffffffffu, max(top_m, top_v) > kPlainMost)) {
        const uint4 all = make_uint4(bits[0], bits[1], bits[2], bits[3]);
        sm = state_scale(block_max<true>(m)), sv = state_scale(block_max<true>(root));
        qm = encode8_any(m[0], m[1], m[2], m[3], sm, all, false);
        qv = encode8_any(root[0], root[1], root[2], root[3], sv, all, true);
        return;
    }
    sm = state_scale(top_m), sv = state_scale(top_v);
    qm = encode8<false>(m, sm, bits);
    qv = encode8<true>(root, sv, bits);
}

// One group of a tensor that does not move in whole groups, or its last one.
template <typename TP, typename TG, bool VEC>
__device__ __noinline__ void step_edge_eight(const StepEntry& e, const StepScalars& s, uint32_t number, int64_t at) {
    const int64_t n = e.n;
    Update u;
    if (!make_update(s, e.weight_decay, u)) return;
    F2 p[4], g[4];
    to_pairs(load_eight<TP, VEC>((const TP*)e.param, at, n), p);
    to_pairs(load_eight<TG, VEC>((const TG*)e.grad, at, n), g);
    uint2 qm = load_codes<VEC>((const uint8_t*)e.m, at, n), qv = load_codes<VEC>((const uint8_t*)e.v, at, n);
    uint32_t sm = at < n ? e.m_scales[at / 32] : 0, sv = at < n ? e.v_scales[at / 32] : 0;
    update_eight(u, s, number, at, p, g, qm, qv, sm, sv);
    if (at >= n) return;
    store_eight<TP, VEC>((TP*)e.param, at, n, p);
    if (e.copy) store_eight<uint16_t, VEC>((uint16_t*)e.copy, at, n, p);
    store_codes<VEC>((uint8_t*)e.m, at, n, qm);
    store_codes<VEC>((uint8_t*)e.v, at, n, qv);
    if (threadIdx.x % 4 == 0) e.m_scales[at / 32] = (uint8_t)sm, e.v_scales[at / 32] = (uint8_t)sv;
}

// `groups` groups of 1024 elements, every kTurns-th from `first` on.
template <typename TP, typename TG>
__device__ __forceinline__ void step_groups_eight(const StepEntry& e, const StepScalars& s, uint32_t number,
                                                  int64_t first, int groups) {
    constexpr int kGroup = kEightThreads * 8;
    constexpr int kStep = kTurns * kGroup;
    int64_t at = first * kGroup + threadIdx.x * 8;
    const int64_t left = e.vec ? (e.n / kGroup - first + kTurns - 1) / kTurns : 0;
    const int whole = left < groups ? (left > 0 ? (int)left : 0) : groups;
    uint8_t *pp = (uint8_t*)e.param + at * sizeof(TP), *pm = (uint8_t*)e.m + at, *pv = (uint8_t*)e.v + at;
    uint8_t *pms = e.m_scales + at / 32, *pvs = e.v_scales + at / 32, *pc = e.copy ? (uint8_t*)e.copy + at * 2 : nullptr;
    const uint8_t* pg = (const uint8_t*)e.grad + at * sizeof(TG);
    // the next group's loads ahead of this one's arithmetic
    Piece<TP, 8> next_p{};
    Piece<TG, 8> next_g{};
    uint2 next_m{}, next_v{};
    uint32_t next_sm = 0, next_sv = 0;
    auto fetch = [&]() {
        next_p = load_eight<TP, true>((const TP*)pp, 0, 8);
        next_g = load_eight<TG, true>((const TG*)pg, 0, 8);
        next_m = *(const uint2*)pm, next_v = *(const uint2*)pv;
        next_sm = *pms, next_sv = *pvs;
    };
    if (whole) fetch();
    Update u;
    if (!make_update(s, e.weight_decay, u)) return;
    for (int k = 0; k < whole; ++k) {
        F2 p[4], g[4];
        to_pairs(next_p, p);
        to_pairs(next_g, g);
        uint2 qm = next_m, qv = next_v;
        uint32_t sm = next_sm, sv = next_sv;
        pp += kStep * sizeof(TP), pg += kStep * sizeof(TG), pm += kStep, pv += kStep;
        pms += kStep / 32, pvs += kStep / 32;
        if (k + 1 < whole) fetch();
        update_eight(u, s, number, at, p, g, qm, qv, sm, sv);
        store_eight<TP, true>((TP*)(pp - kStep * sizeof(TP)), 0, 8, p);
        if (pc) {
            store_eight<uint16_t, true>((uint16_t*)pc, 0, 8, p);
            pc += kStep * 2;
        }
        *(uint2*)(pm - kStep) = qm;
        *(uint2*)(pv - kStep) = qv;
        if (threadIdx.x % 4 == 0) pms[-kStep / 32] = (uint8_t)sm, pvs[-kStep / 32] = (uint8_t)sv;
        at += kStep;
    }
    for (int k = whole; k < groups; ++k, at += kStep) {
        if (e.vec) step_edge_eight<TP, TG, true>(e, s, number, at);
        else step_edge_eight<TP, TG, false>(e, s, number, at);
    }
}

// 8-bit moments, 352M weights with 128 threads to a block: BF16 weights 577 us with seven blocks per SM (72
// registers), 4% more with six (80), 6% with eight (64, spills); FP32 weights and their copies 835 with six, 3% more
// with five or seven.
template <int CAP, Kind KIND>
__global__ void __launch_bounds__(kThreads<KIND>, KIND == kF32Moments ? 4 : KIND == kEightF32 ? 6 : 7)
    adamw_kernel(const __grid_constant__ StepArgs<CAP> a) {
    grid_dependency_wait();
    const int k = a.map.find(blockIdx.x);
    const StepEntry& e = a.e[k];
    const uint32_t block = blockIdx.x - a.map.first[k];
    if constexpr (KIND == kF32Moments) {
#define MOE_STEP(TP, TG) (e.vec ? step_group<TP, TG, true>(e, a.s, block) : step_group<TP, TG, false>(e, a.s, block))
        if (e.param_f32) e.grad_f32 ? MOE_STEP(float, float) : MOE_STEP(float, uint16_t);
        else e.grad_f32 ? MOE_STEP(uint16_t, float) : MOE_STEP(uint16_t, uint16_t);
#undef MOE_STEP
    } else {
        using TP = std::conditional_t<KIND == kEightF32, float, uint16_t>;
        const int64_t all = (e.n + kEightThreads * 8 - 1) / (kEightThreads * 8);
        const int64_t first = (int64_t)(block / kTurns) * (kTurns * a.groups) + block % kTurns;
        const int64_t left = (all - first + kTurns - 1) / kTurns;
        const int groups = left < a.groups ? (int)left : a.groups;
        if (groups <= 0) return;
        const uint32_t number = a.number0 + e.number;
        if (e.grad_f32) step_groups_eight<TP, float>(e, a.s, number, first, groups);
        else step_groups_eight<TP, uint16_t>(e, a.s, number, first, groups);
    }
}

bool groups_at(const void* p, int dtype) { return (uintptr_t)p % (dtype == MOE_MXFP8 ? 8 : 16) == 0; }

// The tensors t[first], ..., t[first + count - 1] that are of one kind.
template <int CAP, Kind KIND>
cudaError_t launch_adamw_list(const moe_adamw_tensor_t* t, int first, int count, const StepScalars& s, int num_sms,
                              cudaStream_t stream) {
    constexpr int64_t kGroup = kThreads<KIND> * 8;
    StepArgs<CAP> a;
    a.number0 = (uint32_t)first, a.s = s, a.groups = 1;
    if (KIND != kF32Moments) {
        // several groups to a block spread its search and scalars, where that leaves enough blocks (352M BF16
        // weights: 2% more with eight)
        int64_t all = 0;
        for (int i = 0; i < count; ++i) all += kind_of(t[first + i]) == KIND ? t[first + i].n / kGroup : 0;
        if (all >= (int64_t)num_sms * 64) a.groups = 8;
        if (all >= (int64_t)num_sms * 1024) a.groups = 32;
    }
    uint32_t blocks = 0;
    int k = 0;
    for (int i = 0; i < count; ++i) {
        const moe_adamw_tensor_t& x = t[first + i];
        if (x.n == 0 || kind_of(x) != KIND) continue;
        StepEntry& e = a.e[k];
        e.param = x.param, e.copy = x.copy, e.grad = x.grad, e.m = x.m, e.v = x.v;
        e.m_scales = x.m_scales, e.v_scales = x.v_scales;
        e.n = x.n;
        e.weight_decay = x.weight_decay;
        e.number = (uint16_t)i;
        e.param_f32 = x.param_dtype == MOE_F32;
        e.grad_f32 = x.grad_dtype == MOE_F32;
        e.vec = groups_at(x.param, x.param_dtype) && groups_at(x.grad, x.grad_dtype) && groups_at(x.m, x.state_dtype) &&
                groups_at(x.v, x.state_dtype) && groups_at(x.copy, MOE_BF16);
        a.map.first[k++] = blocks;
        const uint32_t turns = a.groups == 1 ? 1 : kTurns;  // whole stretches; blocks past the tensor's end have nothing
        const uint32_t stretch = a.groups * turns;
        blocks += (uint32_t)(((x.n + kGroup - 1) / kGroup + stretch - 1) / stretch) * turns;
    }
    if (!k) return cudaSuccess;
    a.map.finish(blocks);
    return launch_after(adamw_kernel<CAP, KIND>, blocks, kThreads<KIND>, 0, 1, stream, a);
}

// Runs f(first, count, pieces) over the list in as few launches as its capacity and the number of
// pieces of a grid allow.
template <typename P, typename F>
cudaError_t in_launches(const moe_adamw_tensor_t* t, int count, P pieces_of, F f) {
    cudaError_t e = cudaSuccess;
    for (int at = 0; at < count && e == cudaSuccess;) {
        int64_t pieces = 0;
        int k = 0;
        while (at + k < count && k < kManyTensors) {
            const int64_t more = pieces_of(t[at + k]);
            if (k && pieces + more > 0x7fffffffLL) break;
            pieces += more;
            ++k;
        }
        e = f(at, k, pieces);
        at += k;
    }
    return e;
}

}  // namespace

cudaError_t launch_grad_norm(const moe_adamw_tensor_t* t, int count, float max_norm, float* part, float* norm,
                             float* factor, cudaStream_t stream) {
    int64_t all = 0, most = 0;
    for (int i = 0; i < count; ++i) all += grad_pieces(t[i], kOneBlock);
    if (count <= kManyTensors && all <= 4) {
        GradArgs<kFewTensors> few;
        few.onto = 0, few.part = nullptr, few.max_norm = max_norm, few.norm = norm, few.factor = factor;
        if (count <= kFewTensors) return launch_grad_norm_list<kFewTensors, kOneBlock>(t, count, few, 1, stream);
        GradArgs<kManyTensors> many;
        many.onto = 0, many.part = nullptr, many.max_norm = max_norm, many.norm = norm, many.factor = factor;
        return launch_grad_norm_list<kManyTensors, kOneBlock>(t, count, many, 1, stream);
    }
    auto pieces_of = [](const moe_adamw_tensor_t& x) { return grad_pieces(x, kNormThreads); };
    in_launches(t, count, pieces_of, [&](int, int, int64_t pieces) {
        most = pieces > most ? pieces : most;
        return cudaSuccess;
    });
    const int parts = most < kGradNormParts ? (int)most : kGradNormParts;
    cudaError_t e = cudaSuccess;
    if (parts > 0)
        e = in_launches(t, count, pieces_of, [&](int at, int k, int64_t) {
            if (k <= kFewTensors) {
                GradArgs<kFewTensors> a;
                a.onto = at > 0, a.part = part;
                return launch_grad_norm_list<kFewTensors, kNormThreads>(t + at, k, a, parts, stream);
            }
            GradArgs<kManyTensors> a;
            a.onto = at > 0, a.part = part;
            return launch_grad_norm_list<kManyTensors, kNormThreads>(t + at, k, a, parts, stream);
        });
    if (e != cudaSuccess) return e;
    return launch_after(grad_norm_join_kernel, 1, 1024, 0, 1, stream, (const float*)part, parts, max_norm, norm, factor);
}

cudaError_t launch_adamw(const moe_adamw_tensor_t* t, int count, const moe_adamw_t& p, int num_sms,
                         cudaStream_t stream) {
    StepScalars s{};
    s.lr = (float)p.lr, s.eps = (float)p.eps;
    s.beta1 = (float)p.beta1, s.beta2 = (float)p.beta2;
    s.one_minus_beta1 = (float)(1.0 - p.beta1), s.one_minus_beta2 = (float)(1.0 - p.beta2);
    s.device_lr = p.device_lr, s.grad_scale = p.grad_scale, s.device_step = p.device_step;
    if (p.device_step) {
        s.log_beta1 = (float)log(p.beta1), s.log_beta2 = (float)log(p.beta2);
    } else {
        const double n = (double)p.step;
        s.inv_bias1 = (float)(1.0 / -expm1(n * log(p.beta1)));
        s.inv_root_bias2 = (float)(1.0 / sqrt(-expm1(n * log(p.beta2))));
        s.step = (uint32_t)p.step;
    }
    s.keys = philox_keys(p.seed);
    auto groups_of = [](const moe_adamw_tensor_t& x) { return (x.n + kStepThreads * 8 - 1) / (kStepThreads * 8); };
    return in_launches(t, count, groups_of, [&](int at, int k, int64_t) {
        const bool few = k <= kFewTensors;
        cudaError_t e = few ? launch_adamw_list<kFewTensors, kF32Moments>(t, at, k, s, num_sms, stream)
                            : launch_adamw_list<kManyTensors, kF32Moments>(t, at, k, s, num_sms, stream);
        if (e == cudaSuccess)
            e = few ? launch_adamw_list<kFewTensors, kEightBf16>(t, at, k, s, num_sms, stream)
                    : launch_adamw_list<kManyTensors, kEightBf16>(t, at, k, s, num_sms, stream);
        if (e == cudaSuccess)
            e = few ? launch_adamw_list<kFewTensors, kEightF32>(t, at, k, s, num_sms, stream)
                    : launch_adamw_list<kManyTensors, kEightF32>(t, at, k, s, num_sms, stream);
        return e;
    });
}

}  // namespace moe
