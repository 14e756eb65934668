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

struct DropoutArgs {
    const void *x, *residual;
    void* out;
    int64_t ld_x, ld_res, ld_out;
    int64_t rows, cols;
    int64_t groups;             // per row: ceil(cols / 8)
    uint32_t thr_high;          // thr << 16
    int drop_all;               // thr = 65536
    float keep_scale;
    uint64_t offset;
    uint32_t key[10][2];        // the rounds' keys: seed + round * Weyl constants
};

// The generator's ten rounds on the counter (b, offset): one wide multiplication and one
// three-way exclusive or per word, the keys from the kernel's arguments.
__device__ __forceinline__ void philox_10(uint64_t b, const DropoutArgs& a, uint32_t (&x)[4]) {
    x[0] = (uint32_t)b, x[1] = (uint32_t)(b >> 32), x[2] = (uint32_t)a.offset, x[3] = (uint32_t)(a.offset >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p = (uint64_t)x[0] * 0xD2511F53u, q = (uint64_t)x[2] * 0xCD9E8D57u;
        x[0] = (uint32_t)(q >> 32) ^ x[1] ^ a.key[i][0];
        x[1] = (uint32_t)q;
        x[2] = (uint32_t)(p >> 32) ^ x[3] ^ a.key[i][1];
        x[3] = (uint32_t)p;
    }
}
// Whether element i of the counter's eight is kept: its 16 bits, moved to the top of a word
// (what lies below them does not matter), against thr there.
__device__ __forceinline__ bool kept(const uint32_t (&w)[4], int i, const DropoutArgs& a) {
    return (i % 2 ? w[i / 2] : w[i / 2] << 16) >= a.thr_high;
}

// The residual and x may each be `out` itself: every thread reads its own elements before it
// writes them.
// Aligned rows: one thread per group of eight columns (one counter), 16-byte accesses.  Each
// thread does one group and ends: blocks that write in address order keep the DRAM writes
// together (zeroing 3.7 GB: 7.8 TB/s so, 6.6 TB/s by a grid that strides over the data).
// HBM-bound: 16384 x 7168 BF16 with a residual in 102 us (6.9 TB/s), 60% of the issue slots
// taken, most of them by the generator's multiplications.
constexpr int kDropThreads = 128;
template <typename T>
__global__ void __launch_bounds__(kDropThreads) dropout_groups_kernel(const __grid_constant__ DropoutArgs a) {
    grid_dependency_wait();
    const uint64_t b = (uint64_t)blockIdx.x * kDropThreads + threadIdx.x;
    uint64_t r = 0;
    if (a.rows == 1) {
        if (b >= (uint64_t)a.groups) return;
    } else {
        r = b >> 32 || a.groups >> 32 ? b / (uint64_t)a.groups : (uint32_t)b / (uint32_t)a.groups;
        if (r >= (uint64_t)a.rows) return;
    }
    const int64_t c = (int64_t)(b - r * a.groups) * 8;
    float v[8], y[8];
    load8<T, true>((const T*)a.x + r * a.ld_x + c, 8, v);
    if (a.residual) load8<T, true>((const T*)a.residual + r * a.ld_res + c, 8, y);
    if (!a.residual) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = 0.f;
    }
    uint32_t w[4];
    philox_10(b, a, w);
    if (!a.drop_all) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (kept(w, i, a)) y[i] = fmaf(v[i], a.keep_scale, y[i]);
    }
    store8<T, true>((T*)a.out + r * a.ld_out + c, 8, y);
}

// Any alignment: one warp per 256 columns of a row.  Lane l draws the counter of columns
// 8l .. 8l+7, but reads and writes every 32nd column, so that the lanes touch neighbouring
// elements; the decisions travel by shuffles.  4001 x 1409 FP32 in 10.3 us (4.4 TB/s), and 9.4 us
// against 6.9 for 1408 columns in groups, the same rows again and again: 71% of the issue slots are
// taken, by twice the groups' instructions per element (single-element accesses, their bounds and
// the shuffles).  Blocks of 64 to 512 threads made no difference.
template <typename T>
__global__ void __launch_bounds__(256) dropout_columns_kernel(const __grid_constant__ DropoutArgs a, int64_t chunks) {
    grid_dependency_wait();
    const int lane = threadIdx.x % 32;
    const int64_t item = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    const int64_t r = item / chunks;
    if (r >= a.rows) return;
    const int64_t c0 = (item - r * chunks) * 256;
    const T* x = (const T*)a.x + r * a.ld_x + c0 + lane;
    const T* res = (const T*)a.residual + r * a.ld_res + c0 + lane;
    T* out = (T*)a.out + r * a.ld_out + c0 + lane;
    float v[8], y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool in = c0 + i * 32 + lane < a.cols;
        v[i] = in ? to_f32<T>(x[i * 32]) : 0.f;
        y[i] = in && a.residual ? to_f32<T>(res[i * 32]) : 0.f;
    }
    uint32_t w[4], mine = 0;                    // bit i: element i of this lane's counter is kept
    philox_10((uint64_t)(r * a.groups + c0 / 8 + lane), a, w);
    if (!a.drop_all) {
#pragma unroll
        for (int i = 0; i < 8; ++i) mine |= (uint32_t)kept(w, i, a) << i;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t keep = __shfl_sync(0xffffffffu, mine, 4 * i + lane / 8);
        if (keep >> (lane % 8) & 1) y[i] = fmaf(v[i], a.keep_scale, y[i]);
        if (c0 + i * 32 + lane < a.cols) out[i * 32] = from_f32<T>(y[i]);
    }
}

cudaError_t launch_dropout(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld_x, const void* residual,
                           int64_t ld_res, uint32_t thr, uint64_t seed, uint64_t offset, void* out, int64_t ld_out,
                           cudaStream_t stream) {
    if (rows == 0 || cols == 0) return cudaSuccess;
    const bool vec = rows_in_groups(x, cols, ld_x, dtype) && rows_in_groups(out, cols, ld_out, dtype) &&
                     (!residual || rows_in_groups(residual, cols, ld_res, dtype));
    if (vec && ld_x == cols && ld_out == cols && (!residual || ld_res == cols) && rows <= (1ll << 60) / cols) {
        cols *= rows;                           // one long row has the same counters
        rows = 1;
    }
    DropoutArgs a{};
    a.x = x, a.residual = residual, a.out = out;
    a.ld_x = ld_x, a.ld_res = ld_res, a.ld_out = ld_out;
    a.rows = rows, a.cols = cols, a.groups = (cols + 7) / 8;
    a.thr_high = thr << 16;
    a.drop_all = thr >= 65536u;
    a.keep_scale = a.drop_all ? 0.f : (float)(65536.0 / (65536.0 - thr));
    a.offset = offset;
    for (uint32_t i = 0; i < 10; ++i) {
        a.key[i][0] = (uint32_t)seed + i * 0x9E3779B9u;
        a.key[i][1] = (uint32_t)(seed >> 32) + i * 0xBB67AE85u;
    }
    if (rows > (1ll << 60) / a.groups) return cudaErrorInvalidValue;
    if (vec)
        return launch_after(dtype == MOE_F32 ? dropout_groups_kernel<float> : dropout_groups_kernel<uint16_t>,
                            (rows * a.groups + kDropThreads - 1) / kDropThreads, kDropThreads, 0, 1, stream, a);
    const int64_t chunks = (cols + 255) / 256;
    return launch_after(dtype == MOE_F32 ? dropout_columns_kernel<float> : dropout_columns_kernel<uint16_t>,
                        (rows * chunks + 7) / 8, 256, 0, 1, stream, a, chunks);
}

}  // namespace moe
