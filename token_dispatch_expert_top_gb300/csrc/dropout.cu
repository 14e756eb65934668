// dropout.cu -- dropout from a counter-based generator, with the residual add:
//   out = residual + keep(r, c) * x * 65536 / (65536 - thr),   thr = round(65536 p)
// keep is a pure function of (seed, offset, r, c), so the mask is never stored and the
// gradient is the same call on dout.  The generator is Philox4x32-10 (Salmon, Moraes,
// Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3", SC 2011): one counter gives
// 128 bits, cut into 16 bits for each of eight consecutive columns.  Sixteen bits make
// the rate exact to 1/65536 and need a quarter of the multiplies of 32; the kept values
// are scaled by the rate the bits really have, so the mean is kept exactly.
#include "kernels.cuh"
#include "vec_io.cuh"

namespace moe {

// Ten rounds on the counter (x0, x1, x2, x3) under the key (k0, k1).
__device__ __forceinline__ void philox_10(uint32_t (&x)[4], uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = (uint64_t)x[0] * 0xD2511F53u, b = (uint64_t)x[2] * 0xCD9E8D57u;
        x[0] = (uint32_t)(b >> 32) ^ x[1] ^ k0;
        x[1] = (uint32_t)b;
        x[2] = (uint32_t)(a >> 32) ^ x[3] ^ k1;
        x[3] = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
}

// One thread per group of eight columns of a row (one counter); VECTOR as in vec_io.cuh.
// The residual and x may each be `out` itself: a thread reads its own elements before it
// writes them.
template <typename T, bool VECTOR>
__global__ void __launch_bounds__(256) dropout_kernel(const T* x, int64_t ld_x, const T* residual, int64_t ld_res,
                                                      int64_t rows, int64_t cols, uint32_t thr, float keep_scale,
                                                      uint64_t seed, uint64_t offset, T* out, int64_t ld_out) {
    const int64_t blocks = (cols + 7) / 8;
    const int64_t total = rows * blocks;
    for (int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; b < total;
         b += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = b / blocks, c = (b % blocks) * 8;
        const int n = (int)(cols - c < 8 ? cols - c : 8);
        float v[8], y[8];
        load8<T, VECTOR>(x + r * ld_x + c, n, v);
        if (residual) load8<T, VECTOR>(residual + r * ld_res + c, n, y);
        uint32_t w[4] = {(uint32_t)b, (uint32_t)(b >> 32), (uint32_t)offset, (uint32_t)(offset >> 32)};
        philox_10(w, (uint32_t)seed, (uint32_t)(seed >> 32));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t bits = i % 2 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu;
            const float base = residual ? y[i] : 0.f;
            y[i] = bits >= thr ? fmaf(v[i], keep_scale, base) : base;
        }
        store8<T, VECTOR>(out + r * ld_out + c, n, y);
    }
}

template <typename T>
static cudaError_t launch_dropout_t(const void* x, int64_t ld_x, const void* residual, int64_t ld_res, int64_t rows,
                                    int64_t cols, bool vec, uint32_t thr, float keep_scale, uint64_t seed,
                                    uint64_t offset, void* out, int64_t ld_out, int num_sms, cudaStream_t stream) {
    const int64_t total = rows * ((cols + 7) / 8);
    int64_t grid = (total + 255) / 256;
    if (grid > (int64_t)num_sms * 8) grid = (int64_t)num_sms * 8;
    auto* k = vec ? dropout_kernel<T, true> : dropout_kernel<T, false>;
    k<<<(unsigned)grid, 256, 0, stream>>>((const T*)x, ld_x, (const T*)residual, ld_res, rows, cols, thr, keep_scale,
                                          seed, offset, (T*)out, ld_out);
    return cudaGetLastError();
}

cudaError_t launch_dropout(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld_x, const void* residual,
                           int64_t ld_res, uint32_t thr, uint64_t seed, uint64_t offset, void* out, int64_t ld_out,
                           int num_sms, cudaStream_t stream) {
    if (rows == 0 || cols == 0) return cudaSuccess;
    const float keep_scale = thr < 65536u ? (float)(65536.0 / (65536.0 - thr)) : 0.f;
    const bool vec = rows_in_groups(x, cols, ld_x, dtype) && rows_in_groups(out, cols, ld_out, dtype) &&
                     (!residual || rows_in_groups(residual, cols, ld_res, dtype));
    return dtype == MOE_F32 ? launch_dropout_t<float>(x, ld_x, residual, ld_res, rows, cols, vec, thr, keep_scale,
                                                      seed, offset, out, ld_out, num_sms, stream)
                            : launch_dropout_t<uint16_t>(x, ld_x, residual, ld_res, rows, cols, vec, thr, keep_scale,
                                                         seed, offset, out, ld_out, num_sms, stream);
}

}  // namespace moe
