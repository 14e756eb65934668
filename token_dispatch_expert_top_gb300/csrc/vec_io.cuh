// vec_io.cuh -- shared by the operators around the layer (embedding.cu, logprobs.cu,
// dropout.cu): a few instructions, and groups of eight consecutive FP32 or BF16 elements as
// FP32 registers, the unit in which they move rows.  VECTOR: the group is 16-byte aligned and
// whole (one 16-byte access for BF16, two for FP32); otherwise element by element, `n` of the
// eight.
#pragma once

#include "common.cuh"

namespace moe {

// ------------------------------------------------- launches that overlap their predecessor
// Waits until the kernel before this one in the stream has finished and its writes are
// visible (for kernels launched with programmatic stream serialization; otherwise at once).
// Such a kernel's inputs may still be written while its blocks are resident, so none of them is
// declared `const __restrict__`: that would promise that they are constant for the kernel's whole
// life, and allow loads that are not coherent or that begin before this wait.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets such a kernel's blocks start, up to their wait, as soon as every block of this one has
// come here.
__device__ __forceinline__ void grid_dependents_launch() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// CTAs of this cluster (1 without one).
__device__ __forceinline__ uint32_t cluster_nctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// ------------------------------------------------------------------------ rows
// Asynchronous 16-byte copy global -> shared (both addresses 16-byte aligned); the end of a
// group of them, and the wait for all of this thread's groups but the last KEEP.
__device__ __forceinline__ void cp_async_16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int KEEP>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(KEEP) : "memory");
}

// Element types by moe_dtype_t; BF16 travels as its 16 bits.
template <typename T>
__device__ __forceinline__ float to_f32(T v) {
    if constexpr (sizeof(T) == 2) return bf16_to_f32(v);
    else return v;
}
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
    if constexpr (sizeof(T) == 2) return f32_to_bf16_rn(v);
    else return v;
}

__device__ __forceinline__ void unpack_bf16x8(const uint4& q, float* v) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        v[2 * p] = __uint_as_float(w[p] << 16);
        v[2 * p + 1] = __uint_as_float(w[p] & 0xFFFF0000u);
    }
}

// 16-byte load through the coherent path: an operator may write the buffer it reads (each
// thread its own elements, after reading them).  Without a hint: keeping L1 out of it was
// slower for every streaming kernel here (the embedding by 9%, the gradient of the log
// probabilities by 4%).
__device__ __forceinline__ uint4 ld_v4(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <typename T, bool VECTOR>
__device__ __forceinline__ void load8(const T* p, int n, float* v) {
    if constexpr (VECTOR && sizeof(T) == 2) {
        unpack_bf16x8(ld_v4(p), v);
    } else if constexpr (VECTOR) {
        const uint4 a = ld_v4(p), b = ld_v4(p + 4);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32<T>(p[i]) : 0.f;
    }
}

template <typename T, bool VECTOR>
__device__ __forceinline__ void store8(T* p, int n, const float* v) {
    if constexpr (VECTOR && sizeof(T) == 2) {
        st_v4(p, make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                            pack_bf16x2(v[6], v[7])));
    } else if constexpr (VECTOR) {
#pragma unroll
        for (int i = 0; i < 8; i += 4)
            st_v4(p + i, make_uint4(__float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]),
                                    __float_as_uint(v[i + 3])));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = from_f32<T>(v[i]);
    }
}

// Launches a kernel that waits on the device for the one before it in the stream
// (grid_dependency_wait, first of all), so that its launch overlaps that one's end.  In a
// stream of calls this saves 2 to 3 us of the lookup of 8192 x 7168 BF16 rows (of 33 us), 2 of the
// dropout of 4001 x 1409 FP32 (of 12), 1.6 of the log probabilities of 64 x 50001 BF16 (of 10) and 5
// of those of 4096 x 128000 with their gradient (of 453).  cluster: CTAs per cluster.
template <typename... Params, typename... Args>
inline cudaError_t launch_after(void (*k)(Params...), int64_t blocks, int threads, size_t smem, int cluster,
                                cudaStream_t stream, const Args&... args) {
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k, args...);
}

inline size_t dtype_bytes(int dtype) { return dtype == MOE_F32 ? 4 : 2; }

// Whether rows of `cols` elements, `ld` apart, split into whole 16-byte aligned groups of
// eight.
inline bool rows_in_groups(const void* base, int64_t cols, int64_t ld, int dtype) {
    return cols % 8 == 0 && ((uintptr_t)base & 15) == 0 && (ld * (int64_t)dtype_bytes(dtype)) % 16 == 0;
}

}  // namespace moe
