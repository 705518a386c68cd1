// The paged key/value cache of the serving step: block tables and slot maps
// from request lengths (thd_kv_block_tables), and the write of new rows into
// their slots (thd_kv_write).
//
// Block tables.  With n, m the cached and new tokens of a request and bs the
// page size: held = ceil(n / bs) pages are in its table, a growing request
// needs ceil((n + m) / bs) - held more, an ended one gives its held back.
// Three prefix sums over the requests say everything: cu (rows), back (pages
// given back) and off (pages wanted).  Then every output is a flat loop whose
// element finds its request by bisection:
//   pushed page y:  free[n_free + y]       = table[b][y - back[b]]
//   popped page x:  table[b][held + x - off[b]] = free[top - 1 - x]
//   packed row t:   pos = n + t - cu[b], page = pos / bs; a page below held is
//                   in the table, another one is popped page
//                   off[b] + page - held, read from the stack itself so that
//                   rows need not wait for the table.
// Latency bound: a few KB to a MB move.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/thd_attn.h"
#include "tma_map.h"

namespace {

constexpr int kTabThreads = 1024;
constexpr int kMaxReq = 8192;  // four int32 arrays of the requests in shared memory
constexpr int32_t kRefused = static_cast<int32_t>(0x80000000u);  // flag on a refused request's length

struct TabParams {
    const int32_t* seq_lens;
    const int32_t* new_lens;
    int32_t* table;
    int32_t* free_blocks;
    const int32_t* free_count;
    const int32_t* first_pos;
    int32_t* seq_out;
    int32_t* free_out;
    int32_t* cu_out;
    int32_t* slots;
    int32_t* positions;
    int32_t* refused;
    int64_t capacity, n_rows;
    int n_req, block, max_blocks;
};

// Exclusive prefix sum of one value per thread over the block, and the total.
__device__ int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int64_t s = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    total = warp_sums[31];
    return x - v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

// Largest value over the block (values >= 0).
__device__ int64_t block_max(int64_t v, int64_t* warp_vals) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const int64_t y = __shfl_xor_sync(0xffffffffu, v, o);
        v = y > v ? y : v;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) warp_vals[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
    for (int w = 0; w < kTabThreads / 32; ++w) v = warp_vals[w] > v ? warp_vals[w] : v;
    return v;
}

// Last b in [0, n) with a[b] <= x (a is non-decreasing and a[0] <= x).
__device__ __forceinline__ int find_request(const int32_t* a, int n, int32_t x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kTabThreads) thd_kv_block_tables_kernel(const TabParams p) {
    extern __shared__ int32_t arrays[];
    int32_t* cu = arrays;               // first packed row
    int32_t* back = cu + p.n_req;       // first pushed page
    int32_t* off = back + p.n_req;      // first popped page
    int32_t* seq = off + p.n_req;       // cached tokens
    __shared__ int64_t warp_sums[32];
    const int tid = threadIdx.x;
    const int per = (p.n_req + kTabThreads - 1) / kTabThreads;  // consecutive requests of a thread
    const int b0 = min(p.n_req, tid * per), b1 = min(p.n_req, b0 + per);
    const int64_t bs = p.block;
    const int n_free = static_cast<int>(min(static_cast<int64_t>(max(*p.free_count, 0)), p.capacity));

    int64_t add = 0, give = 0;
    for (int b = b0; b < b1; ++b) {
        const int n = p.seq_lens[b], m = p.new_lens[b];
        if (n >= 0 && m >= 0) add += m;
        if (n >= 0 && m < 0) give += min((n + bs - 1) / bs, static_cast<int64_t>(p.max_blocks));
    }
    int64_t rows, pushed;
    add = block_scan(add, warp_sums, rows);
    give = block_scan(give, warp_sums, pushed);
    const int64_t top = min(n_free + pushed, p.capacity);
    constexpr int64_t kMax = 0x7fffffff;
    // Pages wanted; a request refused for its width or rows wants none.
    int64_t want = 0;
    {
        int64_t r = add, g = give;
        for (int b = b0; b < b1; ++b) {
            const int n = p.seq_lens[b], m = p.new_lens[b];
            cu[b] = static_cast<int32_t>(min(r, kMax));
            back[b] = static_cast<int32_t>(min(g, kMax));
            seq[b] = n;
            if (n >= 0 && m >= 0) {
                r += m;
                const int64_t total = (static_cast<int64_t>(n) + m + bs - 1) / bs;
                if (m > 0 && total <= p.max_blocks && r <= p.n_rows) want += total - (n + bs - 1) / bs;
            } else if (n >= 0) {
                g += min((n + bs - 1) / bs, static_cast<int64_t>(p.max_blocks));
            }
        }
    }
    int64_t wanted;
    int64_t o = block_scan(want, warp_sums, wanted);
    int64_t taken = 0;
    int n_refused = 0;
    {
        int64_t r = add;
        for (int b = b0; b < b1; ++b) {
            const int n = p.seq_lens[b], m = p.new_lens[b];
            off[b] = static_cast<int32_t>(min(o, kMax));
            if (n < 0 || m <= 0) continue;
            r += m;
            const int64_t total = (static_cast<int64_t>(n) + m + bs - 1) / bs;
            bool no = total > p.max_blocks || r > p.n_rows;
            if (!no) {
                const int64_t need = total - (n + bs - 1) / bs;
                no = need > 0 && o + need > top;
                if (!no && need > 0) taken = o + need;
                o += need;
            }
            if (no) {
                ++n_refused;
                seq[b] = n | kRefused;
            }
        }
    }
    int64_t all_refused;
    block_scan(n_refused, warp_sums, all_refused);
    taken = block_max(taken, warp_sums);

    // Pages of ended requests onto the stack (a page below max_blocks of a
    // row, so the row's own entries).
    const int64_t n_push = min(pushed, p.capacity - n_free);
    for (int64_t y = tid; y < n_push; y += kTabThreads) {
        const int b = find_request(back, p.n_req, static_cast<int32_t>(y));
        p.free_blocks[n_free + y] = p.table[static_cast<int64_t>(b) * p.max_blocks + (y - back[b])];
    }
    __syncthreads();

    if (tid == 0) {
        *p.free_out = static_cast<int32_t>(top - taken);
        *p.refused = static_cast<int32_t>(all_refused);
        p.cu_out[p.n_req] = static_cast<int32_t>(min(rows, kMax));
    }
    for (int b = b0; b < b1; ++b) {
        const int n = p.seq_lens[b], m = p.new_lens[b];
        p.cu_out[b] = cu[b];
        p.seq_out[b] = n < 0 || m < 0 ? -1 : (m > 0 && seq[b] < 0) ? n : n + m;
    }
    for (int64_t x = tid; x < taken; x += kTabThreads) {
        const int b = find_request(off, p.n_req, static_cast<int32_t>(x));
        const int64_t held = (seq[b] + bs - 1) / bs;
        p.table[static_cast<int64_t>(b) * p.max_blocks + held + (x - off[b])] = p.free_blocks[top - 1 - x];
    }
    const int first = p.first_pos != nullptr ? *p.first_pos : 0;
    for (int64_t t = tid; t < p.n_rows; t += kTabThreads) {
        int slot = -1, position = 0;
        if (t < rows) {
            const int b = find_request(cu, p.n_req, static_cast<int32_t>(t));
            const int n = seq[b] & ~kRefused;
            const int64_t far = static_cast<int64_t>(n) + (t - cu[b]);  // (a refused request may pass 2^31)
            position = static_cast<int>(min(first + far, kMax));
            if (seq[b] >= 0) {
                const int at = static_cast<int>(far);
                const int held = static_cast<int>((n + bs - 1) / bs), page = at / p.block;
                const int32_t id = page < held ? p.table[static_cast<int64_t>(b) * p.max_blocks + page]
                                               : p.free_blocks[top - 1 - (off[b] + page - held)];
                if (id >= 0 && id < kMax / bs) slot = id * p.block + at % p.block;
            }
        }
        p.slots[t] = slot;
        p.positions[t] = position;
    }
}

// One thread per 16 bytes of a key and the same 16 bytes of a value.
struct WriteParams {
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    const int32_t* slots;
    __nv_bfloat16* kc;
    __nv_bfloat16* vc;
    int64_t k_row, v_row, n_rows, n_slots, block_stride, token_stride, head_stride;
    int Hkv, D, block;
};

__global__ void __launch_bounds__(256) thd_kv_write_kernel(const WriteParams p) {
    const int per_head = p.D / 8, per_row = p.Hkv * per_head;
    const int64_t total = p.n_rows * per_row;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t r = i / per_row;
        const int c = static_cast<int>(i - r * per_row), h = c / per_head, d = (c - h * per_head) * 8;
        const int slot = p.slots[r];
        if (slot < 0 || slot >= p.n_slots) continue;
        const int64_t to = static_cast<int64_t>(slot / p.block) * p.block_stride +
                           static_cast<int64_t>(slot % p.block) * p.token_stride + h * p.head_stride + d;
        *reinterpret_cast<uint4*>(p.kc + to) = *reinterpret_cast<const uint4*>(p.k + r * p.k_row + h * p.D + d);
        *reinterpret_cast<uint4*>(p.vc + to) = *reinterpret_cast<const uint4*>(p.v + r * p.v_row + h * p.D + d);
    }
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

extern "C" int thd_kv_block_tables(const int32_t* seq_lens, const int32_t* new_lens, int n_req,
                                   int block_size, int32_t* block_tables, int max_blocks,
                                   int32_t* free_blocks, int64_t free_capacity,
                                   const int32_t* free_count, const int32_t* first_position_or_null,
                                   int64_t n_rows, int32_t* seq_lens_out, int32_t* free_count_out,
                                   int32_t* cu_new, int32_t* slots, int32_t* positions,
                                   int32_t* refused, void* stream_ptr) {
    constexpr int64_t kMax = 0x7fffffff;
    if (n_req < 0 || block_size < 1 || max_blocks < 1 || free_capacity < 0 || free_capacity > kMax ||
        n_rows < 0 || n_rows > kMax || static_cast<int64_t>(max_blocks) * block_size > kMax)
        return THD_ERR_INVALID_ARG;
    if (n_req > kMaxReq) return THD_ERR_UNSUPPORTED;
    if (n_req == 0) return THD_OK;
    const void* needed[] = {seq_lens, new_lens, block_tables, free_count, seq_lens_out,
                            free_count_out, cu_new, refused};
    for (const void* q : needed)
        if (q == nullptr || !aligned4(q)) return THD_ERR_INVALID_ARG;
    if ((free_capacity > 0 && free_blocks == nullptr) || (n_rows > 0 && (!slots || !positions)) ||
        !aligned4(free_blocks) || !aligned4(slots) || !aligned4(positions) ||
        !aligned4(first_position_or_null))
        return THD_ERR_INVALID_ARG;
    TabParams p{seq_lens, new_lens, block_tables, free_blocks, free_count, first_position_or_null,
                seq_lens_out, free_count_out, cu_new, slots, positions, refused,
                free_capacity, n_rows, n_req, block_size, max_blocks};
    const int smem = 16 * n_req;
    if (smem > 40000 &&
        cudaFuncSetAttribute(thd_kv_block_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             16 * kMaxReq) != cudaSuccess)
        return THD_ERR_CUDA;
    thd_kv_block_tables_kernel<<<1, kTabThreads, smem, static_cast<cudaStream_t>(stream_ptr)>>>(p);
    return cudaGetLastError() == cudaSuccess ? THD_OK : THD_ERR_CUDA;
}

extern "C" int thd_kv_write(const void* k, const void* v, int64_t k_row_stride, int64_t v_row_stride,
                            const int32_t* slots, int64_t n_rows, int Hkv, int D, void* k_cache,
                            void* v_cache, int64_t num_blocks, int block_size, int64_t block_stride,
                            int64_t token_stride, int64_t head_stride, void* stream_ptr) {
    if (n_rows < 0 || Hkv <= 0 || num_blocks < 0 || block_size < 1 || num_blocks > 0x7fffffffll / block_size)
        return THD_ERR_INVALID_ARG;
    if (D != 64 && D != 128 && D != 256) return THD_ERR_UNSUPPORTED;
    if (n_rows == 0 || num_blocks == 0) return THD_OK;
    if (!k || !v || !slots || !k_cache || !v_cache) return THD_ERR_INVALID_ARG;
    if (!thd::aligned16(k) || !thd::aligned16(v) || !thd::aligned16(k_cache) || !thd::aligned16(v_cache) ||
        !aligned4(slots))
        return THD_ERR_INVALID_ARG;
    const int64_t row = static_cast<int64_t>(Hkv) * D;
    if (k_row_stride < row || v_row_stride < row || (k_row_stride | v_row_stride) % 8 != 0)
        return THD_ERR_INVALID_ARG;
    if (block_stride < 0 || token_stride < D || head_stride < D ||
        (block_stride | token_stride | head_stride) % 8 != 0)
        return THD_ERR_INVALID_ARG;
    WriteParams p{static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), slots,
                  static_cast<__nv_bfloat16*>(k_cache), static_cast<__nv_bfloat16*>(v_cache),
                  k_row_stride, v_row_stride, n_rows, num_blocks * block_size, block_stride,
                  token_stride, head_stride, Hkv, D, block_size};
    const int64_t threads = n_rows * (row / 8);
    const int64_t blocks = (threads + 255) / 256;
    thd_kv_write_kernel<<<static_cast<unsigned>(blocks < 148 * 64 ? blocks : 148 * 64), 256, 0,
                          static_cast<cudaStream_t>(stream_ptr)>>>(p);
    return cudaGetLastError() == cudaSuccess ? THD_OK : THD_ERR_CUDA;
}
