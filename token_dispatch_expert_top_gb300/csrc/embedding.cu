// embedding.cu -- token embedding with scaling, and the gradient of its table.
//   forward:  out[n] = scale * table[ids[n]]
//   gradient: dtable[v] (+)= scale * sum_{n : ids[n] = v} dout[n]
// A negative id is "no token": a zero row, no gradient.  An id of V or more does the same
// and records MOE_ERR_DEVICE_CHECK.
//
// The gradient uses no atomics on values, so it is deterministic.  For few tokens
// embed_few_kernel finds and sums every run in one launch.  For more, the tokens are sorted by
// id without a comparison sort:
//   1. embed_order_kernel: each CTA owns a range of ids, reads all N ids (they stay in L2),
//      counts its own and how many live ids lie below its range, and places its tokens in
//      ascending token order -- no exchange between CTAs.
//   2. embed_segment_kernel: the sorted list is cut into ranges of 4 to 32 tokens whatever the
//      ids, so a frequent token cannot unbalance it; a run of equal ids inside a range is
//      summed in FP32 in token order and written, a run that crosses a range's end leaves
//      an FP32 partial row.  (Before it embed_fill_kernel sets the rows no token names to
//      zero, unless the caller accumulates.)
//   3. embed_join_kernel: adds the partial rows of each run that crossed, in an order that
//      its length alone sets.
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
// Eight columns of a row in a lane's registers.  VECTOR: eight neighbours, by 16-byte
// accesses; otherwise every 32nd column, so that the warp's lanes touch neighbouring elements
// whatever the alignment.  Both cover the warp's 256 columns from c0.
template <typename T, bool VECTOR>
__device__ __forceinline__ void load_cols(const T* row, int64_t c0, int lane, int64_t H, float* v) {
    if constexpr (VECTOR) {
        if (c0 + lane * 8 < H) load8<T, true>(row + c0 + lane * 8, 8, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c0 + i * 32 + lane < H ? to_f32<T>(row[c0 + i * 32 + lane]) : 0.f;
    }
}
template <typename T, bool VECTOR>
__device__ __forceinline__ void store_cols(T* row, int64_t c0, int lane, int64_t H, const float* v) {
    if constexpr (VECTOR) {
        if (c0 + lane * 8 < H) store8<T, true>(row + c0 + lane * 8, 8, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c0 + i * 32 + lane < H) row[c0 + i * 32 + lane] = from_f32<T>(v[i]);
    }
}

// The same eight columns as they lie in memory, converted when they are used: half the
// registers for BF16 rows in flight.
template <typename T, bool VECTOR>
struct RawCols {
    static constexpr bool kPacked = VECTOR && sizeof(T) == 2;
    uint4 q;
    float v[kPacked ? 1 : 8];
    __device__ void load(const T* row, int64_t c0, int lane, int64_t H) {
        if constexpr (kPacked) {
            if (c0 + lane * 8 < H) q = ld_v4(row + c0 + lane * 8);
        } else {
            load_cols<T, VECTOR>(row, c0, lane, H, v);
        }
    }
    __device__ void add_to(float* sum) const {
        if constexpr (kPacked) {
            float x[8];
            unpack_bf16x8(q, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += x[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += v[j];
        }
    }
};

// A memory-bound copy with a scale.  Short rows (aligned, at most 128 columns): 2^lane_bits
// lanes per row, each one group of eight columns.  Otherwise one warp per 256 * U columns of
// a row; its loads are all issued before the first store.  8192 rows of 7168 BF16 in 29.9 us
// (7.7 TB/s, some of it L2's); a single row is bound by the launch.
constexpr int kEmbedUnroll = 4;
template <typename Id, typename In, typename Out, bool VECTOR>
__global__ void __launch_bounds__(256) embedding_kernel(const Id* ids, int64_t N, const In* table, int64_t V,
                                                        int64_t H, int64_t ld_table, float scale, Out* out,
                                                        int64_t ld_out, int chunks, int lane_bits, WsHeader* ws) {
    grid_dependency_wait();
    const int lane = threadIdx.x % 32;
    const uint64_t item = (uint64_t)blockIdx.x * 8 + threadIdx.x / 32;
    if (lane_bits < 5) {
        const int64_t n = (int64_t)(item << (5 - lane_bits)) + (lane >> lane_bits);
        const int64_t c = (lane & ((1 << lane_bits) - 1)) * 8;
        if (n >= N || c >= H) return;
        bool bad = false;
        const int id = live_id(ids[n], V, &bad);
        if (bad && c == 0) set_status(ws, MOE_ERR_DEVICE_CHECK);
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (id >= 0) load8<In, true>(table + id * ld_table + c, 8, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= scale;
        store8<Out, true>(out + n * ld_out + c, 8, v);
        return;
    }
    const int64_t n = item >> 32 ? (int64_t)(item / (uint32_t)chunks) : (int64_t)((uint32_t)item / (uint32_t)chunks);
    if (n >= N) return;
    const int64_t c0 = (int64_t)(item - (uint64_t)n * chunks) * (256 * kEmbedUnroll);
    bool bad = false;
    const int id = live_id(ids[n], V, &bad);
    if (bad && lane == 0 && c0 == 0) set_status(ws, MOE_ERR_DEVICE_CHECK);
    float v[kEmbedUnroll][8];
#pragma unroll
    for (int u = 0; u < kEmbedUnroll; ++u) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
        if (id >= 0) load_cols<In, VECTOR>(table + id * ld_table, c0 + u * 256, lane, H, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kEmbedUnroll; ++u) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] *= scale;
        store_cols<Out, VECTOR>(out + n * ld_out, c0 + u * 256, lane, H, v[u]);
    }
}

template <typename Id, typename In, typename Out>
static cudaError_t launch_embedding_t(const void* ids, int64_t N, const void* table, int64_t V, int64_t H,
                                      int64_t ld_table, float scale, void* out, int64_t ld_out, bool vec,
                                      WsHeader* ws, cudaStream_t stream) {
    int lane_bits = 5;
    if (vec && H <= 128)
        for (lane_bits = 0; (8 << lane_bits) < H;) ++lane_bits;
    const int64_t chunks = lane_bits < 5 ? 1 : (H + 256 * kEmbedUnroll - 1) / (256 * kEmbedUnroll);
    const int64_t items = lane_bits < 5 ? (N + (32 >> lane_bits) - 1) >> (5 - lane_bits) : N * chunks;
    const int64_t grid = (items + 7) / 8;
    auto* k = vec ? embedding_kernel<Id, In, Out, true> : embedding_kernel<Id, In, Out, false>;
    return launch_after(k, grid, 256, 0, 1, stream, (const Id*)ids, N, (const In*)table, V, H, ld_table, scale,
                        (Out*)out, ld_out, (int)chunks, lane_bits, ws);
}

template <typename Id>
static cudaError_t launch_embedding_id(const void* ids, int64_t N, const void* table, int table_dtype, int64_t V,
                                       int64_t H, int64_t ld_table, float scale, void* out, int out_dtype,
                                       int64_t ld_out, WsHeader* ws, cudaStream_t stream) {
    const bool vec = rows_in_groups(table, H, ld_table, table_dtype) && rows_in_groups(out, H, ld_out, out_dtype);
    if (table_dtype == MOE_F32)
        return out_dtype == MOE_F32
                   ? launch_embedding_t<Id, float, float>(ids, N, table, V, H, ld_table, scale, out, ld_out, vec,
                                                          ws, stream)
                   : launch_embedding_t<Id, float, uint16_t>(ids, N, table, V, H, ld_table, scale, out, ld_out, vec,
                                                             ws, stream);
    return out_dtype == MOE_F32
               ? launch_embedding_t<Id, uint16_t, float>(ids, N, table, V, H, ld_table, scale, out, ld_out, vec,
                                                         ws, stream)
               : launch_embedding_t<Id, uint16_t, uint16_t>(ids, N, table, V, H, ld_table, scale, out, ld_out, vec,
                                                            ws, stream);
}

cudaError_t launch_embedding(const void* ids, int id_bytes, int64_t N, const void* table, int table_dtype, int64_t V,
                             int64_t H, int64_t ld_table, float scale, void* out, int out_dtype, int64_t ld_out,
                             WsHeader* ws, cudaStream_t stream) {
    if (N == 0) return cudaSuccess;
    return id_bytes == 8 ? launch_embedding_id<int64_t>(ids, N, table, table_dtype, V, H, ld_table, scale, out,
                                                        out_dtype, ld_out, ws, stream)
                         : launch_embedding_id<int32_t>(ids, N, table, table_dtype, V, H, ld_table, scale, out,
                                                        out_dtype, ld_out, ws, stream);
}

// ------------------------------------------------------------------------ order
constexpr int kOrderThreads = 1024;
constexpr int kOrderIds = 4;                  // ids a thread reads per sweep of the CTA
constexpr int kOrderList = 4096;              // own tokens kept in shared memory

// Exclusive prefix sum over the CTA's threads; *total is the sum.  All threads call it.
__device__ __forceinline__ int block_scan_exclusive(int v, int* warp_sums, int* total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    __syncthreads();                          // earlier reads of warp_sums are done
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int s = warp_sums[lane];                  // kOrderThreads / 32 = 32 warps
    int before = lane < warp ? s : 0;
    before = __reduce_add_sync(0xffffffffu, before);
    *total = __reduce_add_sync(0xffffffffu, s);
    return before + incl - v;
}

// Gives the CTA's own tokens list_row / list_pos [0, n), which are in token order, their places
// in the sorted list; cursor[row] is the row's next place.  All threads call it.
//   Short lists: one warp, 32 tokens at a time.  Long ones (a frequent token): kPlaceWarps
// warps count their shares' tokens by row, the counts are summed up over the warps, and
// every token's place is its row's, its warp's and its own rank.
constexpr int kPlaceWarps = 8, kPlaceShare = kOrderList / kPlaceWarps, kPlaceSerial = 512;
__device__ __forceinline__ void place_list(int* list_row, const int* list_pos, int n, int* cursor, uint16_t* counts,
                                           int rows, int v0, int32_t* order, int32_t* key) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if (n <= kPlaceSerial) {
        if (warp == 0) {
            for (int i0 = 0; i0 < n; i0 += 32) {
                const int i = i0 + lane;
                const int row = i < n ? list_row[i] : -1 - lane;
                const unsigned same = __match_any_sync(0xffffffffu, row);
                if (row >= 0) {
                    const int place = cursor[row] + __popc(same & ((1u << lane) - 1u));
                    order[place] = list_pos[i];
                    key[place] = v0 + row;
                }
                __syncwarp();
                if (row >= 0 && lane == 31 - __clz(same)) cursor[row] += __popc(same);
                __syncwarp();
            }
        }
        __syncthreads();
        return;
    }
    for (int i = threadIdx.x; i < kPlaceWarps * rows; i += blockDim.x) counts[i] = 0;
    __syncthreads();
    if (warp < kPlaceWarps) {
        uint16_t* mine = counts + warp * rows;
        const int end = min(n, (warp + 1) * kPlaceShare);
        for (int i0 = warp * kPlaceShare; i0 < end; i0 += 32) {
            const int i = i0 + lane;
            const int row = i < end ? list_row[i] : -1 - lane;
            const unsigned same = __match_any_sync(0xffffffffu, row);
            if (row >= 0) list_row[i] = row | (mine[row] + __popc(same & ((1u << lane) - 1u))) << 16;
            __syncwarp();
            if (row >= 0 && lane == 31 - __clz(same)) mine[row] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    for (int row = threadIdx.x; row < rows; row += blockDim.x) {
        int sum = 0;
        for (int w = 0; w < kPlaceWarps; ++w) {
            const int c = counts[w * rows + row];
            counts[w * rows + row] = (uint16_t)sum;
            sum += c;
        }
        counts[kPlaceWarps * rows + row] = (uint16_t)sum;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int row = list_row[i] & 0xFFFF, rank = list_row[i] >> 16;
        const int place = cursor[row] + counts[i / kPlaceShare * rows + row] + rank;
        order[place] = list_pos[i];
        key[place] = v0 + row;
    }
    __syncthreads();
    for (int row = threadIdx.x; row < rows; row += blockDim.x) cursor[row] += counts[kPlaceWarps * rows + row];
    __syncthreads();
}
constexpr int kOrderRange = 2048;             // ids of a CTA at most
static_assert(kOrderRange <= 1 << 16 && kOrderList <= 1 << 15, "rows and ranks are packed into a word");
// Dynamic shared memory of embed_order_kernel: the list, `range` next places and the counts.
inline size_t order_smem(int range) {
    return sizeof(int) * (2 * (size_t)kOrderList + range) + sizeof(uint16_t) * (size_t)(kPlaceWarps + 1) * range;
}

// Sets one row to zero, thread `t` of `threads`: 16-byte stores, single elements at the ends of
// an unaligned row.
template <typename Grad>
__device__ __forceinline__ void zero_row(Grad* row, int64_t H, int t, int threads) {
    constexpr int VEC = 16 / sizeof(Grad);
    int64_t head = (VEC - (int64_t)((uintptr_t)row / sizeof(Grad) % VEC)) % VEC;
    if (head > H) head = H;
    const int vectors = (int)((H - head) / VEC);
    Grad* body = row + head;
#pragma unroll 4
    for (int i = t; i < vectors; i += threads) st_v4(body + (int64_t)i * VEC, make_uint4(0u, 0u, 0u, 0u));
    if (t < head) row[t] = Grad(0);
    if (t < H - head - (int64_t)vectors * VEC) body[(int64_t)vectors * VEC + t] = Grad(0);
}

// CTA b places the tokens whose ids lie in [b * range, (b + 1) * range): order[i] is the
// token at place i of the list sorted by (id, token), key[i] its id; bit v of `present` says
// that a token names v.  range is a multiple of 32.
//   One sweep over the ids counts the CTA's own tokens by id, counts the live tokens below
// its range (where its part of the list begins) and lists its own tokens in order; if the
// list overflows, a second sweep places them piece by piece.
//   A small table is set to zero meanwhile by the CTAs from fill_from on, which saves the
// launch of embed_fill_kernel; the rows that tokens name are written over by the sums.
template <typename Id, typename Grad>
__global__ void __launch_bounds__(kOrderThreads)
    embed_order_kernel(const Id* ids, int N, int64_t V, int range, int32_t* order, int32_t* key, int32_t* n_live,
                       uint32_t* present, int fill_from, Grad* dtable, int64_t H, int64_t ld, WsHeader* ws) {
    grid_dependents_launch();
    grid_dependency_wait();
    if ((int)blockIdx.x >= fill_from) {
        const int64_t warps = (int64_t)(gridDim.x - fill_from) * (kOrderThreads / 32);
        for (int64_t v = (int64_t)(blockIdx.x - fill_from) * (kOrderThreads / 32) + threadIdx.x / 32; v < V; v += warps)
            zero_row(dtable + v * ld, H, threadIdx.x % 32, 32);
        return;
    }
    extern __shared__ int smem[];
    __shared__ int warp_sums[kOrderThreads / 32];
    int *list_row = smem, *list_pos = list_row + kOrderList, *cursor = list_pos + kOrderList;
    uint16_t* counts = reinterpret_cast<uint16_t*>(cursor + range);
    constexpr int kSweep = kOrderThreads * kOrderIds;
    static_assert(kSweep <= kOrderList, "a sweep's own tokens fit the list");
    const int tid = threadIdx.x, lane = tid % 32;
    const int v0 = (int)((int64_t)blockIdx.x * range);
    const int rows = (int)(V - v0 < range ? V - v0 : range);
    for (int i = tid; i < rows; i += kOrderThreads) cursor[i] = 0;
    // ids[n0 + kOrderIds * tid ..], -1 past the end
    auto read_ids = [&](int n0, int (&id)[kOrderIds], bool* bad) {
#pragma unroll
        for (int i = 0; i < kOrderIds; ++i) {
            const int n = n0 + tid * kOrderIds + i;
            id[i] = n < N ? live_id(ids[n], V, bad) : -1;
        }
    };
    __syncthreads();
    int below = 0, live = 0, listed = 0;
    bool bad = false;
    int next[kOrderIds];
    read_ids(0, next, &bad);
    for (int n0 = 0; n0 < N; n0 += kSweep) {
        int id[kOrderIds], mine = 0;
#pragma unroll
        for (int i = 0; i < kOrderIds; ++i) id[i] = next[i];
        if (n0 + kSweep < N) read_ids(n0 + kSweep, next, &bad);
#pragma unroll
        for (int i = 0; i < kOrderIds; ++i) {
            live += id[i] >= 0;
            below += id[i] >= 0 && id[i] < v0;
            if (id[i] >= v0 && id[i] < v0 + rows) {
                ++mine;
                atomicAdd(&cursor[id[i] - v0], 1);
            }
        }
        int total;
        int at = listed + block_scan_exclusive(mine, warp_sums, &total);
        if (listed + total <= kOrderList) {
#pragma unroll
            for (int i = 0; i < kOrderIds; ++i)
                if (id[i] >= v0 && id[i] < v0 + rows) {
                    list_row[at] = id[i] - v0;
                    list_pos[at++] = n0 + tid * kOrderIds + i;
                }
        }
        listed += total;
    }
    if (bad && blockIdx.x == 0) set_status(ws, MOE_ERR_DEVICE_CHECK);
    int base, all_live;
    block_scan_exclusive(below, warp_sums, &base);
    block_scan_exclusive(live, warp_sums, &all_live);
    if (blockIdx.x == 0 && tid == 0) n_live[0] = all_live, n_live[1] = n_live[2] = 0;
    // counts -> first places, and the rows' presence
    __syncthreads();
    int run = base;
    for (int i0 = 0; i0 < rows; i0 += kOrderThreads) {
        const int i = i0 + tid;
        const int c = i < rows ? cursor[i] : 0;
        const unsigned bits = __ballot_sync(0xffffffffu, c > 0);
        if (lane == 0 && i < rows) present[((int64_t)v0 + i) / 32] = bits;
        int total;
        const int ex = block_scan_exclusive(c, warp_sums, &total);
        if (i < rows) cursor[i] = run + ex;
        run += total;
    }
    __syncthreads();
    if (listed <= kOrderList) {
        place_list(list_row, list_pos, listed, cursor, counts, rows, v0, order, key);
        return;
    }
    for (int n0 = 0; n0 < N; n0 += kSweep) {
        int id[kOrderIds], mine = 0;
        read_ids(n0, id, &bad);
#pragma unroll
        for (int i = 0; i < kOrderIds; ++i) mine += id[i] >= v0 && id[i] < v0 + rows;
        int total;
        int at = block_scan_exclusive(mine, warp_sums, &total);
#pragma unroll
        for (int i = 0; i < kOrderIds; ++i)
            if (id[i] >= v0 && id[i] < v0 + rows) {
                list_row[at] = id[i] - v0;
                list_pos[at++] = n0 + tid * kOrderIds + i;
            }
        __syncthreads();
        place_list(list_row, list_pos, total, cursor, counts, rows, v0, order, key);
    }
}

// ------------------------------------------------------------------------ sums
// Writes scale * sum (+ the row's old value) of the warp's 256 columns of row v.
template <typename Grad, bool VECTOR>
__device__ __forceinline__ void write_row(Grad* dtable, int64_t ld, int v, int64_t c0, int lane, int64_t H,
                                          const float* sum, float scale, int accumulate) {
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    Grad* row = dtable + v * ld;
    if (accumulate) load_cols<Grad, VECTOR>(row, c0, lane, H, o);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = accumulate ? fmaf(sum[i], scale, o[i]) : sum[i] * scale;
    store_cols<Grad, VECTOR>(row, c0, lane, H, o);
}

struct EmbedSumArgs {
    const int32_t* order;
    const int32_t* key;
    int32_t* n_live;          // [0] tokens with an id, [1] short and [2] long runs that cross ranges
    int4* crossing;           // [ranges] (first range, partial rows, id, -): short runs from the front, long
                              // ones from the back
    const void* dout;
    int64_t ld_dout, H;
    float scale;
    void* dtable;
    int64_t ld;
    int accumulate;
    float* part;
    int places;               // sorted tokens per range
    int ranges, chunks;
};

constexpr int kSumWarps = 4;

// FP32 partial rows: two per range, [0] a run that began before the range, [1] a run that
// goes on after it.  A row is a.chunks blocks of 256 columns; a lane's eight columns of a
// block lie together, whichever they are, so every lane moves two whole 16-byte groups.
__device__ __forceinline__ float* partial_cols(const EmbedSumArgs& a, int64_t range, int which, int64_t c0) {
    return a.part + (range * 2 + which) * a.chunks * 256 + c0 + threadIdx.x % 32 * 8;
}
constexpr int kFillThreads = 256;
constexpr int kFillBytes = 16384;             // about what one CTA fills

// Sets the rows without a token to zero: long rows one per CTA, short ones (at most half of
// kFillBytes) one per warp, fill_rows per CTA.  Many short CTAs in address order rather than a
// few that stride over the table: 7.8 against 6.6 TB/s on 3.7 GB, as the DRAM sees one moving
// front of writes.  A kernel of its own, because it needs every thread an SM can hold to cover
// the look at `present`.
template <typename Grad>
__global__ void __launch_bounds__(kFillThreads)
    embed_fill_kernel(const uint32_t* present, int64_t V, int64_t H, Grad* dtable, int64_t ld, int fill_rows) {
    grid_dependency_wait();
    if (fill_rows == 1) {
        const uint32_t v = blockIdx.x;
        if (!(present[v / 32] >> (v % 32) & 1)) zero_row(dtable + (int64_t)v * ld, H, threadIdx.x, kFillThreads);
        return;
    }
    const int64_t v0 = (int64_t)blockIdx.x * fill_rows;
    for (int i = threadIdx.x / 32; i < fill_rows && v0 + i < V; i += kFillThreads / 32) {
        const int64_t v = v0 + i;
        if (!(present[v / 32] >> (v % 32) & 1)) zero_row(dtable + v * ld, H, threadIdx.x % 32, 32);
    }
}

template <typename Grad>
static cudaError_t launch_fill_t(const EmbedBackward& c, cudaStream_t stream) {
    const int64_t row_bytes = c.H * (int64_t)sizeof(Grad);
    const int fill_rows = row_bytes > kFillBytes / 2 ? 1 : (int)(kFillBytes / row_bytes);
    const int64_t blocks = (c.V + fill_rows - 1) / fill_rows;
    return launch_after(embed_fill_kernel<Grad>, blocks, kFillThreads, 0, 1, stream, (const uint32_t*)c.present, c.V,
                        c.H, (Grad*)c.dtable, c.ld_dtable, fill_rows);
}

// Lists the run of id k that begins in `range` and goes on: how many partial rows it has (its
// own and one per range after it), short runs and long ones apart, each in any order.
constexpr int kShortRun = 12;
__device__ __forceinline__ void list_crossing(const EmbedSumArgs& a, int range, int k, int live) {
    const int lane = threadIdx.x % 32;
    // equal ids are neighbours: the run covers the next ranges as long as they begin with it;
    // the first that does not, among the next 32 or, 32 looks at a time, all others
    int lo = range + 1, hi = a.ranges;
    for (int step = 1; lo < hi; step = (hi - lo + 31) / 32) {
        const int64_t r = lo + (int64_t)lane * step;
        const bool in = r < hi && r * a.places < live && a.key[r * a.places] == k;
        const int n = __popc(__ballot_sync(0xffffffffu, in));
        if (n < 32) hi = min((int64_t)hi, lo + (int64_t)n * step);
        if (n == 0) break;
        lo += (n - 1) * step + 1;
    }
    const int rows = lo - range;
    if (lane == 0) {
        const int at = rows <= kShortRun ? atomicAdd(a.n_live + 1, 1) : a.ranges - 1 - atomicAdd(a.n_live + 2, 1);
        a.crossing[at] = make_int4(range, rows, k, 0);
    }
}

// One warp per (range of places, 256 columns), bound by the latency of the rows' loads, eight
// (FP32: four) of which a lane has in flight.  16384 tokens of 7168 BF16 columns into FP32: 69 us
// beside 445 us for the zero rows of a 3.7 GB table; ordering takes 12 us and the join 7.5.
// Accumulating onto that table: 114 us, as the rows' old values are read, and 136 us in all.  The
// ordering's time grows with N, as every CTA reads all ids (131072 tokens: 114 us, and 154 us if they
// share one id, which one CTA places), and so does the join's for one id (133 us).
template <typename In, typename Grad, bool VECTOR>
__global__ void __launch_bounds__(kSumWarps * 32) embed_segment_kernel(const __grid_constant__ EmbedSumArgs a) {
    grid_dependency_wait();
    const int lane = threadIdx.x % 32;
    const int64_t item = (int64_t)blockIdx.x * kSumWarps + threadIdx.x / 32;
    if (item >= (int64_t)a.ranges * a.chunks) return;
    const int range = (int)(item / a.chunks);
    const int64_t c0 = (item - (int64_t)range * a.chunks) * 256;
    const int live = *a.n_live;
    const int p0 = range * a.places;
    if (p0 >= live) return;
    const int cnt = min(a.places, live - p0);
    const int my_key = lane < cnt ? a.key[p0 + lane] : -1;
    const int my_pos = lane < cnt ? a.order[p0 + lane] : 0;
    const int before = p0 ? a.key[p0 - 1] : -1;
    const int after = p0 + cnt < live ? a.key[p0 + cnt] : -1;
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    bool from_before = __shfl_sync(0xffffffffu, my_key, 0) == before;
    constexpr int U = RawCols<In, VECTOR>::kPacked ? 8 : 4;
    for (int i0 = 0; i0 < cnt; i0 += U) {
        RawCols<In, VECTOR> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t pos = __shfl_sync(0xffffffffu, my_pos, (i0 + u) & 31);
            if (i0 + u < cnt) v[u].load((const In*)a.dout + pos * a.ld_dout, c0, lane, a.H);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u;
            const int k = __shfl_sync(0xffffffffu, my_key, i & 31);
            const int k_in = __shfl_sync(0xffffffffu, my_key, (i + 1) & 31);
            if (i < cnt) {
                const int k_next = i + 1 < cnt ? k_in : after;
                v[u].add_to(sum);
                if (k != k_next || i + 1 == cnt) {
                    if (from_before)
                        store8<float, true>(partial_cols(a, range, 0, c0), 8, sum);
                    else if (k == k_next) {
                        store8<float, true>(partial_cols(a, range, 1, c0), 8, sum);
                        if (c0 == 0) list_crossing(a, range, k, live);
                    } else
                        write_row<Grad, VECTOR>((Grad*)a.dtable, a.ld, k, c0, lane, a.H, sum, a.scale, a.accumulate);
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[j] = 0.f;
                    from_before = false;
                }
            }
        }
    }
}

// Adds up partial rows [first, last) of a run that begins in `range`, in order: row 0 is
// [range][1], row i is [range + i][0].
__device__ __forceinline__ void add_partials(const EmbedSumArgs& a, int range, int first, int last, int64_t c0,
                                             float (&sum)[8]) {
    constexpr int U = 6;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] = 0.f;
#pragma unroll 1
    for (int i0 = first; i0 < last; i0 += U) {
        float v[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u < last) load8<float, true>(partial_cols(a, range + i0 + u, i0 + u == 0, c0), 8, v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u < last) {
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] += v[u][j];
            }
    }
}

// The runs that cross ranges.  Long ones first: kJoinCols * 256 columns of one per CTA, the
// partial rows cut into kJoinParts parts, one warp each, whose sums are added in order.
// Short ones: one warp per 256 columns.  (A run's sum does not depend on the lists' order.)
constexpr int kJoinCols = 2, kJoinParts = 4, kJoinCtas = 3, kJoinWarps = kJoinCols * kJoinParts;
template <typename Grad, bool VECTOR>
__global__ void __launch_bounds__(kJoinWarps * 32, kJoinCtas) embed_join_kernel(const __grid_constant__ EmbedSumArgs a) {
    __shared__ float sums[kJoinParts - 1][kJoinCols][8][32];
    grid_dependency_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, col = warp % kJoinCols, part = warp / kJoinCols;
    const uint32_t groups = (uint32_t)(a.chunks + kJoinCols - 1) / kJoinCols, chunks = (uint32_t)a.chunks;
    const uint32_t longs = (uint32_t)a.n_live[2] * groups, shorts = (uint32_t)a.n_live[1] * chunks;   // < 2^31
    float sum[8];
    for (uint32_t item = blockIdx.x; item < longs; item += gridDim.x) {
        const int4 run = a.crossing[a.ranges - 1 - (int)(item / groups)];
        const int64_t c0 = (int64_t)(item % groups * kJoinCols + col) * 256;
        if (c0 < a.H) {
            add_partials(a, run.x, (int)((int64_t)run.y * part / kJoinParts),
                         (int)((int64_t)run.y * (part + 1) / kJoinParts), c0, sum);
            if (part > 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) sums[part - 1][col][j][lane] = sum[j];
            }
        }
        __syncthreads();
        if (part == 0 && c0 < a.H) {
#pragma unroll
            for (int p = 0; p < kJoinParts - 1; ++p)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] += sums[p][col][j][lane];
            write_row<Grad, VECTOR>((Grad*)a.dtable, a.ld, run.z, c0, lane, a.H, sum, a.scale, a.accumulate);
        }
        __syncthreads();
    }
    // (from the last CTA down: the first ones may have had a long run)
    for (uint32_t item = (gridDim.x - 1 - blockIdx.x) * kJoinWarps + warp; item < shorts; item += gridDim.x * kJoinWarps) {
        const int4 run = a.crossing[item / chunks];
        const int64_t c0 = (int64_t)(item % chunks) * 256;
        add_partials(a, run.x, 0, run.y, c0, sum);
        write_row<Grad, VECTOR>((Grad*)a.dtable, a.ld, run.z, c0, lane, a.H, sum, a.scale, a.accumulate);
    }
}

// ------------------------------------------------------------------------ few tokens
// The gradient in one launch, for at most kFewTokens tokens.  A CTA per token and slice of 2048
// columns marks the tokens that share its id, and so knows the run and its own rank in it; the
// run's CTAs divide the slice's columns among them in groups of eight, at least four, and those
// that get none leave.  So every token's row is read once, a frequent id keeps as many CTAs busy
// as it has tokens, and nothing is exchanged between CTAs.  In a CTA, 2^bits neighbouring lanes
// hold a row's groups and the others the run's next rows; their FP32 sums are added in
// pairs.  The first `zero_ctas` CTAs set the rows that no token names to zero, `zero_rows` each.
//   777 rows of 1409 FP32 columns into 5003: 9.9 us; the odd rows, which move by single elements,
// cost 1.4 of them (9.0 us against 7.6 for 1408 columns, the same rows again and again).  With
// nothing else in the stream to overlap 11.0 us against 17.2 by sorting, and 12.9 with three or
// five CTAs to an SM; one id for all of 1000 rows of 2048: 9.7 against 19.7.  Every CTA reads all
// ids, so the work grows with N^2: at 2000 tokens it took 27.2 us against 18.8.
//   Bound by latency: of 17 cycles between a warp's instructions 5 are waits for memory and 39% of
// the issue slots are taken; the rest is barriers and the chain from ids to rows to stores.
constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32;
constexpr int kFewTokens = 1024, kFewSweeps = kFewTokens / kFewThreads;
constexpr int kFewCols = kFewThreads * 8;
constexpr int kFewZeroRows = 4096;
constexpr int kFewGroups = 4;                 // groups a CTA takes at least: whole sectors of a row
static_assert(kFewTokens == 32 * 32, "a lane looks at one word of marks");

struct EmbedFewArgs {
    const void* ids;
    int N;
    int64_t V;
    const void* dout;
    int64_t ld_dout, H;
    float scale;
    void* dtable;
    int64_t ld;
    int accumulate;
    int slices, zero_ctas, zero_rows;
    WsHeader* ws;
};

template <typename Id, typename In, typename Grad, bool VECTOR>
__global__ void __launch_bounds__(kFewThreads, 4) embed_few_kernel(const __grid_constant__ EmbedFewArgs a) {
    __shared__ uint32_t words[kFewZeroRows / 32];
    __shared__ uint16_t list[kFewTokens];
    __shared__ float sums[8][kFewThreads];
    grid_dependency_wait();
    const Id* ids = (const Id*)a.ids;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    bool bad = false;
    if ((int)blockIdx.x < a.zero_ctas) {
        const int64_t v0 = (int64_t)blockIdx.x * a.zero_rows;
        const int rows = (int)(a.V - v0 < a.zero_rows ? a.V - v0 : a.zero_rows);
        for (int i = tid; i < (rows + 31) / 32; i += kFewThreads) words[i] = 0u;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kFewSweeps; ++k) {
            const int n = k * kFewThreads + tid;
            const int64_t v = (n < a.N ? live_id(ids[n], a.V, &bad) : -1) - v0;
            if (v >= 0 && v < rows) atomicOr(&words[v / 32], 1u << v % 32);
        }
        __syncthreads();
        for (int i = warp; i < rows; i += kFewWarps)
            if (!(words[i / 32] >> (i % 32) & 1)) zero_row((Grad*)a.dtable + (v0 + i) * a.ld, a.H, lane, 32);
        return;
    }
    const int item = (int)blockIdx.x - a.zero_ctas, n = item / a.slices, slice = item - n * a.slices;
    const int own = live_id(ids[n], a.V, &bad);
    if (bad && slice == 0 && tid == 0) set_status(a.ws, MOE_ERR_DEVICE_CHECK);
    if (own < 0) return;
    // the run's tokens; `list` gets them in order
    bool same[kFewSweeps], others = false;
#pragma unroll
    for (int k = 0; k < kFewSweeps; ++k) {
        const int i = k * kFewThreads + tid;
        same[k] = i < a.N && ids[i] == (Id)own;
        others |= same[k] && i != n;
    }
#pragma unroll
    for (int k = 0; k < kFewSweeps; ++k) {
        const uint32_t w = __ballot_sync(0xffffffffu, same[k]);
        if (lane == 0) words[k * kFewWarps + warp] = w;
    }
    const bool alone = !__syncthreads_or(others);
    int before = 0, total = 1, rank = 0;      // marks before the lane's word
    if (!alone) {
        const int c = __popc(words[lane]);
        int incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        before = incl - c;
        total = __shfl_sync(0xffffffffu, incl, 31);
        rank = __shfl_sync(0xffffffffu, before, n / 32) + __popc(words[n / 32] & ((1u << n % 32) - 1u));
    }
    const int64_t c0 = (int64_t)slice * kFewCols;
    const int groups = (int)((min((int64_t)kFewCols, a.H - c0) + 7) / 8);
    const int share = max((groups + total - 1) / total, kFewGroups);
    const int first = rank * share, last = min(groups, first + share);
    if (first >= groups) return;              // the same for the whole CTA
    if (!alone) {
#pragma unroll
        for (int k = 0; k < kFewSweeps; ++k) {
            const int i = k * kFewWarps + warp;
            const int at = __shfl_sync(0xffffffffu, before, i) + __popc(words[i] & ((1u << lane) - 1u));
            if (same[k]) list[at] = (uint16_t)(k * kFewThreads + tid);
        }
        __syncthreads();
    }
    int bits = 2;
    while (1 << bits < share) ++bits;
    const int width = 1 << bits, g = tid & (width - 1), r = tid >> bits, step = kFewThreads >> bits;
    // VECTOR: eight neighbouring columns, otherwise every width-th
    const int64_t begin = c0 + first * 8 + (VECTOR ? g * 8 : g), end = min(a.H, c0 + last * 8);
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    auto load = [&](int i, float (&v)[8]) {
        const In* row = (const In*)a.dout + (alone ? n : list[i]) * a.ld_dout;
        if constexpr (VECTOR) {
            if (begin < end) load8<In, true>(row + begin, 8, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = begin + j * width < end ? to_f32<In>(row[begin + j * width]) : 0.f;
        }
    };
    constexpr int U = 4;
    int i0 = r;
    for (; i0 + (U - 1) * step < total; i0 += U * step) {
        float v[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) load(i0 + u * step, v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += v[u][j];
    }
#pragma unroll 1
    for (; i0 < total; i0 += step) {
        float v[8];
        load(i0, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += v[j];
    }
    for (int half = alone ? 0 : step / 2; half; half /= 2) {
        if (r >= half && r < 2 * half) {
#pragma unroll
            for (int j = 0; j < 8; ++j) sums[j][tid] = sum[j];
        }
        __syncthreads();
        if (r < half) {
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += sums[j][tid + half * width];
        }
    }
    if (r > 0 || begin >= end) return;
    Grad* row = (Grad*)a.dtable + own * a.ld;
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (a.accumulate) {
        if constexpr (VECTOR) {
            load8<Grad, true>(row + begin, 8, o);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (begin + j * width < end) o[j] = to_f32<Grad>(row[begin + j * width]);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = a.accumulate ? fmaf(sum[j], a.scale, o[j]) : sum[j] * a.scale;
    if constexpr (VECTOR) {
        store8<Grad, true>(row + begin, 8, o);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (begin + j * width < end) row[begin + j * width] = from_f32<Grad>(o[j]);
    }
}

// ------------------------------------------------------------------------ host side
template <typename Id, typename In, typename Grad>
static cudaError_t launch_few_t(const EmbedBackward& c, cudaStream_t stream) {
    const bool vec = rows_in_groups(c.dout, c.H, c.ld_dout, c.dout_dtype) &&
                     rows_in_groups(c.dtable, c.H, c.ld_dtable, c.dtable_dtype);
    EmbedFewArgs a{};
    a.ids = c.ids;
    a.N = (int)c.N;
    a.V = c.V;
    a.dout = c.dout;
    a.ld_dout = c.ld_dout;
    a.H = c.H;
    a.scale = c.scale;
    a.dtable = c.dtable;
    a.ld = c.ld_dtable;
    a.accumulate = c.accumulate;
    a.slices = (int)((c.H + kFewCols - 1) / kFewCols);
    a.ws = c.ws;
    if (!c.accumulate) {
        // two CTAs per SM
        const int64_t rows = (c.V + 2 * c.num_sms - 1) / (2 * c.num_sms);
        a.zero_rows = (int)(rows < kFewZeroRows ? rows : kFewZeroRows);
        a.zero_ctas = (int)((c.V + a.zero_rows - 1) / a.zero_rows);
    }
    const int64_t blocks = a.zero_ctas + c.N * a.slices;
    if (blocks == 0) return cudaSuccess;
    auto* k = vec ? embed_few_kernel<Id, In, Grad, true> : embed_few_kernel<Id, In, Grad, false>;
    return launch_after(k, blocks, kFewThreads, 0, 1, stream, a);
}
template <typename Id>
static cudaError_t launch_few_id(const EmbedBackward& c, cudaStream_t stream) {
    if (c.dout_dtype == MOE_F32)
        return c.dtable_dtype == MOE_F32 ? launch_few_t<Id, float, float>(c, stream)
                                         : launch_few_t<Id, float, uint16_t>(c, stream);
    return c.dtable_dtype == MOE_F32 ? launch_few_t<Id, uint16_t, float>(c, stream)
                                     : launch_few_t<Id, uint16_t, uint16_t>(c, stream);
}

template <typename Id, typename Grad>
static cudaError_t launch_order_t(const EmbedBackward& c, bool fill, cudaStream_t stream) {
    // one CTA per SM, ranges of whole words of `present`
    int64_t range = (c.V + c.num_sms - 1) / c.num_sms;
    range = (range + 31) / 32 * 32;
    if (range > kOrderRange) range = kOrderRange;
    const int64_t grid = (c.V + range - 1) / range;
    cudaError_t err = cudaFuncSetAttribute(embed_order_kernel<Id, Grad>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)order_smem(kOrderRange));
    if (err != cudaSuccess) return err;
    const int64_t fill_ctas = !fill ? 0 : (c.V + 31) / 32 < 2 * c.num_sms ? (c.V + 31) / 32 : 2 * c.num_sms;
    return launch_after(embed_order_kernel<Id, Grad>, grid + fill_ctas, kOrderThreads, order_smem((int)range), 1,
                        stream, (const Id*)c.ids, (int)c.N, c.V, (int)range, c.order, c.key, c.n_live, c.present,
                        (int)grid, (Grad*)c.dtable, c.H, c.ld_dtable, c.ws);
}

template <typename In, typename Grad>
static cudaError_t launch_sums_t(const EmbedBackward& c, cudaStream_t stream) {
    const bool vec = rows_in_groups(c.dout, c.H, c.ld_dout, c.dout_dtype) &&
                     rows_in_groups(c.dtable, c.H, c.ld_dtable, c.dtable_dtype);
    EmbedSumArgs a{};
    a.order = c.order;
    a.key = c.key;
    a.n_live = c.n_live;
    a.crossing = c.crossing;
    a.dout = c.dout;
    a.ld_dout = c.ld_dout;
    a.H = c.H;
    a.scale = c.scale;
    a.dtable = c.dtable;
    a.ld = c.ld_dtable;
    a.accumulate = c.accumulate;
    a.part = c.part;
    a.places = embed_places(c.N, c.H);
    a.ranges = embed_ranges(c.N, c.H);
    a.chunks = (int)((c.H + 255) / 256);
    const int64_t blocks = ((int64_t)a.ranges * a.chunks + kSumWarps - 1) / kSumWarps;
    if ((int64_t)a.ranges * a.chunks > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (blocks == 0) return cudaSuccess;
    auto* k = vec ? embed_segment_kernel<In, Grad, true> : embed_segment_kernel<In, Grad, false>;
    cudaError_t err = launch_after(k, blocks, kSumWarps * 32, 0, 1, stream, a);
    if (err != cudaSuccess || a.ranges <= 1) return err;          // one range: no run crosses
    auto* j = vec ? embed_join_kernel<Grad, true> : embed_join_kernel<Grad, false>;
    const int64_t most = (int64_t)(a.ranges - 1) * ((a.chunks + kJoinCols - 1) / kJoinCols);   // items
    return launch_after(j, most < kJoinCtas * c.num_sms ? most : kJoinCtas * c.num_sms, kJoinWarps * 32, 0, 1, stream, a);
}

// Tables and token rows (written twice then) of at most so many bytes are zeroed beside the
// ordering: 41.7 against 45.7 us for 125 MB and 16 MB, 76.5 against 81.3 for 250 MB and 65 MB.
// Larger ones gain more from embed_fill_kernel's order of writes, and lose more by writing
// twice, than the launch costs.
constexpr int64_t kSmallTable = 256ll << 20, kSmallRows = 64ll << 20;

cudaError_t launch_embedding_backward(const EmbedBackward& c, cudaStream_t stream) {
    const bool f32 = c.dtable_dtype == MOE_F32;
    const int64_t row_bytes = c.H * (f32 ? 4 : 2);
    const bool small = c.V * row_bytes <= kSmallTable && c.N * row_bytes <= kSmallRows;
    // (a large table is set to zero by embed_fill_kernel's writes in address order)
    if (c.N <= kFewTokens && (small || c.accumulate))
        return c.id_bytes == 8 ? launch_few_id<int64_t>(c, stream) : launch_few_id<int32_t>(c, stream);
    const bool fill_now = small && !c.accumulate;
    cudaError_t err = c.id_bytes == 8 ? (f32 ? launch_order_t<int64_t, float>(c, fill_now, stream)
                                             : launch_order_t<int64_t, uint16_t>(c, fill_now, stream))
                                      : (f32 ? launch_order_t<int32_t, float>(c, fill_now, stream)
                                             : launch_order_t<int32_t, uint16_t>(c, fill_now, stream));
    if (err == cudaSuccess && !small && !c.accumulate)
        err = f32 ? launch_fill_t<float>(c, stream) : launch_fill_t<uint16_t>(c, stream);
    if (err != cudaSuccess) return err;
    if (c.dout_dtype == MOE_F32)
        return c.dtable_dtype == MOE_F32 ? launch_sums_t<float, float>(c, stream)
                                         : launch_sums_t<float, uint16_t>(c, stream);
    return c.dtable_dtype == MOE_F32 ? launch_sums_t<uint16_t, float>(c, stream)
                                     : launch_sums_t<uint16_t, uint16_t>(c, stream);
}

}  // namespace moe
