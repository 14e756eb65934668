// embedding.cu -- token embedding with scaling, and the gradient of its table.
//   forward:  out[n] = scale * table[ids[n]]
//   gradient: dtable[v] (+)= scale * sum_{n : ids[n] = v} dout[n]
// A negative id is "no token": a zero row, no gradient.  An id of V or more does the same
// and records MOE_ERR_DEVICE_CHECK.
//
// The gradient sorts the tokens by id without a comparison sort and without atomics on
// values, so it is deterministic:
//   1. embed_order_kernel: each CTA owns a range of ids, reads all N ids (they stay in L2),
//      counts its own and how many live ids lie below its range, and places its tokens in
//      ascending token order -- no exchange between CTAs.  Rows no token names are set to
//      zero here (unless the caller accumulates).
//   2. embed_segment_kernel: the sorted list is cut into ranges of Q tokens whatever the
//      ids, so a frequent token cannot unbalance it; a run of equal ids inside a range is
//      summed in FP32 in token order and written, a run that crosses a range's end leaves
//      an FP32 partial row.
//   3. embed_join_kernel: adds the partial rows of each run that crossed, in order.
#include "kernels.cuh"
#include "vec_io.cuh"

namespace moe {

// ids[n] as an int: -1 for "no token" or out of range (*bad set for the latter).
template <typename Id>
__device__ __forceinline__ int live_id(Id id, int64_t V, bool* bad) {
    if (id < 0) return -1;
    if ((int64_t)id >= V) {
        *bad = true;
        return -1;
    }
    return (int)id;
}

// ------------------------------------------------------------------------ forward
// One thread per group of eight columns of an output row, four groups a round with
// their loads issued first.
template <typename Id, typename In, typename Out, bool VECTOR>
__global__ void __launch_bounds__(256) embedding_kernel(const Id* __restrict__ ids, int64_t N,
                                                        const In* __restrict__ table, int64_t V, int64_t H,
                                                        int64_t ld_table, float scale, Out* __restrict__ out,
                                                        int64_t ld_out, WsHeader* ws) {
    constexpr int U = 4;
    const int64_t groups = (H + 7) / 8;
    const int64_t total = N * groups;
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t g0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; g0 < total; g0 += U * step) {
        float v[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t g = g0 + u * step;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
            if (g >= total) continue;
            const int64_t n = g / groups, c = (g % groups) * 8;
            bool bad = false;
            const int id = live_id(ids[n], V, &bad);
            if (bad && c == 0) set_status(ws, MOE_ERR_DEVICE_CHECK);
            if (id >= 0) load8<In, VECTOR>(table + id * ld_table + c, (int)(H - c < 8 ? H - c : 8), v[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t g = g0 + u * step;
            if (g >= total) continue;
            const int64_t n = g / groups, c = (g % groups) * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] *= scale;
            store8<Out, VECTOR>(out + n * ld_out + c, (int)(H - c < 8 ? H - c : 8), v[u]);
        }
    }
}

template <typename Id, typename In, typename Out>
static cudaError_t launch_embedding_t(const void* ids, int64_t N, const void* table, int64_t V, int64_t H,
                                      int64_t ld_table, float scale, void* out, int64_t ld_out, bool vec,
                                      int num_sms, WsHeader* ws, cudaStream_t stream) {
    const int64_t total = N * ((H + 7) / 8);
    int64_t grid = (total + 255) / 256;
    if (grid > (int64_t)num_sms * 8) grid = (int64_t)num_sms * 8;
    auto* k = vec ? embedding_kernel<Id, In, Out, true> : embedding_kernel<Id, In, Out, false>;
    k<<<(unsigned)grid, 256, 0, stream>>>((const Id*)ids, N, (const In*)table, V, H, ld_table, scale, (Out*)out,
                                          ld_out, ws);
    return cudaGetLastError();
}

template <typename Id>
static cudaError_t launch_embedding_id(const void* ids, int64_t N, const void* table, int table_dtype, int64_t V,
                                       int64_t H, int64_t ld_table, float scale, void* out, int out_dtype,
                                       int64_t ld_out, int num_sms, WsHeader* ws, cudaStream_t stream) {
    const bool vec = rows_in_groups(table, H, ld_table, table_dtype) && rows_in_groups(out, H, ld_out, out_dtype);
    if (table_dtype == MOE_F32)
        return out_dtype == MOE_F32
                   ? launch_embedding_t<Id, float, float>(ids, N, table, V, H, ld_table, scale, out, ld_out, vec,
                                                          num_sms, ws, stream)
                   : launch_embedding_t<Id, float, uint16_t>(ids, N, table, V, H, ld_table, scale, out, ld_out, vec,
                                                             num_sms, ws, stream);
    return out_dtype == MOE_F32
               ? launch_embedding_t<Id, uint16_t, float>(ids, N, table, V, H, ld_table, scale, out, ld_out, vec,
                                                         num_sms, ws, stream)
               : launch_embedding_t<Id, uint16_t, uint16_t>(ids, N, table, V, H, ld_table, scale, out, ld_out, vec,
                                                            num_sms, ws, stream);
}

cudaError_t launch_embedding(const void* ids, int id_bytes, int64_t N, const void* table, int table_dtype, int64_t V,
                             int64_t H, int64_t ld_table, float scale, void* out, int out_dtype, int64_t ld_out,
                             int num_sms, WsHeader* ws, cudaStream_t stream) {
    if (N == 0) return cudaSuccess;
    return id_bytes == 8 ? launch_embedding_id<int64_t>(ids, N, table, table_dtype, V, H, ld_table, scale, out,
                                                        out_dtype, ld_out, num_sms, ws, stream)
                         : launch_embedding_id<int32_t>(ids, N, table, table_dtype, V, H, ld_table, scale, out,
                                                        out_dtype, ld_out, num_sms, ws, stream);
}

// ------------------------------------------------------------------------ order
constexpr int kOrderThreads = 512;
constexpr int kOrderTile = kOrderThreads;     // ids placed per round

// Exclusive prefix sum over the CTA's threads; *total is the sum.  All threads call it.
__device__ __forceinline__ int block_scan_exclusive(int v, int* warp_sums, int* total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    __syncthreads();                          // earlier reads of warp_sums are done
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < warps; ++w) {
        const int s = warp_sums[w];
        if (w < warp) before += s;
        all += s;
    }
    *total = all;
    return before + incl - v;
}

// CTA b places the tokens whose ids lie in [b * range, (b + 1) * range): order[i] is the
// token at place i of the list sorted by (id, token), key[i] its id.  cursor: `range` ints of
// shared memory.
template <typename Id, typename Grad, bool VECTOR>
__global__ void __launch_bounds__(kOrderThreads)
    embed_order_kernel(const Id* __restrict__ ids, int N, int64_t V, int range, int32_t* __restrict__ order,
                       int32_t* __restrict__ key, int32_t* __restrict__ n_live, Grad* __restrict__ dtable, int64_t H,
                       int64_t ld, int fill, WsHeader* ws) {
    extern __shared__ int cursor[];
    __shared__ int warp_sums[kOrderThreads / 32];
    __shared__ int list_row[kOrderTile], list_pos[kOrderTile];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int64_t v0 = (int64_t)blockIdx.x * range;
    const int rows = (int)(V - v0 < range ? V - v0 : range);
    for (int i = tid; i < rows; i += kOrderThreads) cursor[i] = 0;
    __syncthreads();
    // count this range's tokens by id, and the live tokens below the range
    int below = 0, live = 0;
    bool bad = false;
    for (int n = tid; n < N; n += kOrderThreads) {
        const int id = live_id(ids[n], V, &bad);
        if (id < 0) continue;
        ++live;
        if (id < v0) ++below;
        else if (id < v0 + rows) atomicAdd(&cursor[id - (int)v0], 1);
    }
    if (bad && blockIdx.x == 0) set_status(ws, MOE_ERR_DEVICE_CHECK);
    int base, all_live;
    block_scan_exclusive(below, warp_sums, &base);
    block_scan_exclusive(live, warp_sums, &all_live);
    if (blockIdx.x == 0 && tid == 0) *n_live = all_live;
    // counts -> first places
    __syncthreads();
    int run = base;
    for (int i0 = 0; i0 < rows; i0 += kOrderThreads) {
        const int i = i0 + tid;
        const int c = i < rows ? cursor[i] : 0;
        int total;
        const int ex = block_scan_exclusive(c, warp_sums, &total);
        if (i < rows) cursor[i] = run + ex;
        run += total;
    }
    __syncthreads();
    // place, tile by tile in token order: the tile's own tokens are listed in order, then
    // one warp gives each its id's next place
    if (run > base) {
        for (int n0 = 0; n0 < N; n0 += kOrderTile) {
            const int n = n0 + tid;
            bool b2 = false;
            const int id = n < N ? live_id(ids[n], V, &b2) : -1;
            const bool mine = id >= v0 && id < v0 + rows;
            int total;
            const int at = block_scan_exclusive(mine ? 1 : 0, warp_sums, &total);
            if (mine) {
                list_row[at] = id - (int)v0;
                list_pos[at] = n;
            }
            __syncthreads();
            if (warp == 0) {
                for (int i0 = 0; i0 < total; i0 += 32) {
                    const int i = i0 + lane;
                    const int row = i < total ? list_row[i] : -1 - lane;
                    const unsigned same = __match_any_sync(0xffffffffu, row);
                    if (row >= 0) {
                        const int place = cursor[row] + __popc(same & ((1u << lane) - 1u));
                        order[place] = list_pos[i];
                        key[place] = (int)v0 + row;
                    }
                    __syncwarp();
                    if (row >= 0 && lane == 31 - __clz(same)) cursor[row] += __popc(same);
                    __syncwarp();
                }
            }
            // the next round's scan begins with a barrier before the list is written again
        }
    }
    if (!fill) return;
    __syncthreads();
    // cursor[i] is now the first place after row i: equal neighbours mean no token
    const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int i = warp; i < rows; i += kOrderThreads / 32) {
        if (cursor[i] != (i ? cursor[i - 1] : base)) continue;
        Grad* dst = dtable + (v0 + i) * ld;
        for (int64_t c = lane * 8; c < H; c += 256)
            store8<Grad, VECTOR>(dst + c, (int)(H - c < 8 ? H - c : 8), zero);
    }
}

// ------------------------------------------------------------------------ sums
// Writes scale * sum (+ the row's old value) of the columns c .. c+7 of row v.
template <typename Grad, bool VECTOR>
__device__ __forceinline__ void write_row(Grad* dtable, int64_t ld, int v, int64_t c, int n, const float* sum,
                                          float scale, int accumulate) {
    float o[8];
    Grad* dst = dtable + v * ld + c;
    if (accumulate) {
        load8<Grad, VECTOR>(dst, n, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = fmaf(sum[i], scale, o[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = sum[i] * scale;
    }
    store8<Grad, VECTOR>(dst, n, o);
}

// FP32 partial rows: two per range, [0] a run that began before the range, [1] a run that
// goes on after it.  Rows are Hp columns (H rounded up to 8), 32-byte aligned.
__device__ __forceinline__ float* partial_row(float* part, int range, int which, int64_t Hp) {
    return part + ((int64_t)range * 2 + which) * Hp;
}

// One warp per (range of kEmbedRange places, 256 columns).
template <typename In, typename Grad, bool VEC_IN, bool VEC_OUT>
__global__ void __launch_bounds__(128)
    embed_segment_kernel(const int32_t* __restrict__ order, const int32_t* __restrict__ key,
                         const int32_t* __restrict__ n_live, const In* __restrict__ dout, int64_t ld_dout, int64_t H,
                         float scale, Grad* dtable, int64_t ld, int accumulate, float* __restrict__ part,
                         int ranges, int chunks) {
    const int lane = threadIdx.x % 32;
    const int64_t item = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    if (item >= (int64_t)ranges * chunks) return;
    const int range = (int)(item / chunks);
    const int64_t c = (item % chunks) * 256 + lane * 8;
    const int live = *n_live;
    const int p0 = range * kEmbedRange;
    if (p0 >= live) return;
    const int cnt = min(kEmbedRange, live - p0);
    const int my_key = lane < cnt ? key[p0 + lane] : -1;
    const int my_pos = lane < cnt ? order[p0 + lane] : 0;
    const int before = p0 ? key[p0 - 1] : -1;
    const int after = p0 + cnt < live ? key[p0 + cnt] : -1;
    const int n = c < H ? (int)(H - c < 8 ? H - c : 8) : 0;
    const int64_t Hp = (H + 7) / 8 * 8;
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    bool from_before = __shfl_sync(0xffffffffu, my_key, 0) == before;
    constexpr int U = 8;
    for (int i0 = 0; i0 < cnt; i0 += U) {
        float v[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t pos = __shfl_sync(0xffffffffu, my_pos, (i0 + u) & 31);
            if (i0 + u < cnt && n > 0) load8<In, VEC_IN>(dout + pos * ld_dout + c, n, v[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u;
            const int k = __shfl_sync(0xffffffffu, my_key, i & 31);
            const int k_next = i + 1 < cnt ? __shfl_sync(0xffffffffu, my_key, (i + 1) & 31) : after;
            if (i < cnt) {
                if (n > 0)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[j] += v[u][j];
                if (k != k_next || i + 1 == cnt) {
                    if (n > 0) {
                        if (from_before) store8<float, true>(partial_row(part, range, 0, Hp) + c, 8, sum);
                        else if (k == k_next) store8<float, true>(partial_row(part, range, 1, Hp) + c, 8, sum);
                        else write_row<Grad, VEC_OUT>(dtable, ld, k, c, n, sum, scale, accumulate);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[j] = 0.f;
                    from_before = false;
                }
            }
        }
    }
}

// One warp per (range, 256 columns): if the range's last run begins in it and goes on, the
// run's partial rows are added in order and written.
template <typename Grad, bool VEC_OUT>
__global__ void __launch_bounds__(128)
    embed_join_kernel(const int32_t* __restrict__ key, const int32_t* __restrict__ n_live, int64_t H, float scale,
                      Grad* dtable, int64_t ld, int accumulate, float* part, int ranges, int chunks) {
    const int lane = threadIdx.x % 32;
    const int64_t item = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    if (item >= (int64_t)ranges * chunks) return;
    const int range = (int)(item / chunks);
    const int live = *n_live;
    const int p0 = range * kEmbedRange, p1 = p0 + kEmbedRange;
    if (p1 >= live) return;                                       // nothing follows this range
    const int k = key[p1 - 1];
    if (key[p1] != k) return;                                     // the last run ends here
    if (key[p0] == k && p0 > 0 && key[p0 - 1] == k) return;       // it began in an earlier range
    const int64_t c = (item % chunks) * 256 + lane * 8;
    if (c >= H) return;
    const int64_t Hp = (H + 7) / 8 * 8;
    float sum[8], v[8];
    load8<float, true>(partial_row(part, range, 1, Hp) + c, 8, sum);
    for (int r = range + 1;; ++r) {
        load8<float, true>(partial_row(part, r, 0, Hp) + c, 8, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += v[j];
        const int end = (r + 1) * kEmbedRange;
        if (end >= live || key[end] != k) break;                  // equal ids are neighbours
    }
    write_row<Grad, VEC_OUT>(dtable, ld, k, c, (int)(H - c < 8 ? H - c : 8), sum, scale, accumulate);
}

// ------------------------------------------------------------------------ host side
template <typename Id, typename Grad>
static cudaError_t launch_order_t(const EmbedBackward& c, bool vec, cudaStream_t stream) {
    int64_t grid = c.num_sms;
    if (grid > c.V) grid = c.V;
    const int64_t widest = 8192;                                  // ids per CTA: 32 KB of counters
    if ((c.V + grid - 1) / grid > widest) grid = (c.V + widest - 1) / widest;
    const int range = (int)((c.V + grid - 1) / grid);
    grid = (c.V + range - 1) / range;
    auto* k = vec ? embed_order_kernel<Id, Grad, true> : embed_order_kernel<Id, Grad, false>;
    k<<<(unsigned)grid, kOrderThreads, (size_t)range * sizeof(int), stream>>>(
        (const Id*)c.ids, (int)c.N, c.V, range, c.order, c.key, c.n_live, (Grad*)c.dtable, c.H, c.ld_dtable,
        !c.accumulate, c.ws);
    return cudaGetLastError();
}

template <typename In, typename Grad>
static cudaError_t launch_sums_t(const EmbedBackward& c, bool vec_out, cudaStream_t stream) {
    const bool vec_in = rows_in_groups(c.dout, c.H, c.ld_dout, c.dout_dtype);
    const int ranges = embed_ranges(c.N);
    const int64_t chunks = (c.H + 255) / 256;
    const int64_t blocks = (ranges * chunks + 3) / 4;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    auto* k = vec_in ? (vec_out ? embed_segment_kernel<In, Grad, true, true> : embed_segment_kernel<In, Grad, true, false>)
                     : (vec_out ? embed_segment_kernel<In, Grad, false, true> : embed_segment_kernel<In, Grad, false, false>);
    k<<<(unsigned)blocks, 128, 0, stream>>>(c.order, c.key, c.n_live, (const In*)c.dout, c.ld_dout, c.H, c.scale,
                                            (Grad*)c.dtable, c.ld_dtable, c.accumulate, c.part, ranges, (int)chunks);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess || ranges == 1) return err;            // one range: no run crosses
    auto* j = vec_out ? embed_join_kernel<Grad, true> : embed_join_kernel<Grad, false>;
    j<<<(unsigned)blocks, 128, 0, stream>>>(c.key, c.n_live, c.H, c.scale, (Grad*)c.dtable, c.ld_dtable, c.accumulate,
                                            c.part, ranges, (int)chunks);
    return cudaGetLastError();
}

cudaError_t launch_embedding_backward(const EmbedBackward& c, cudaStream_t stream) {
    const bool vec_out = rows_in_groups(c.dtable, c.H, c.ld_dtable, c.dtable_dtype);
    const bool f32 = c.dtable_dtype == MOE_F32;
    cudaError_t err = c.id_bytes == 8
                          ? (f32 ? launch_order_t<int64_t, float>(c, vec_out, stream)
                                 : launch_order_t<int64_t, uint16_t>(c, vec_out, stream))
                          : (f32 ? launch_order_t<int32_t, float>(c, vec_out, stream)
                                 : launch_order_t<int32_t, uint16_t>(c, vec_out, stream));
    if (err != cudaSuccess || c.N == 0) return err;
    if (c.dout_dtype == MOE_F32)
        return f32 ? launch_sums_t<float, float>(c, vec_out, stream) : launch_sums_t<float, uint16_t>(c, vec_out, stream);
    return f32 ? launch_sums_t<uint16_t, float>(c, vec_out, stream)
               : launch_sums_t<uint16_t, uint16_t>(c, vec_out, stream);
}

}  // namespace moe
