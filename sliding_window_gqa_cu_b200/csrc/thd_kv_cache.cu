// The paged key/value cache of the serving step: block tables and slot maps
// from request lengths (thd_kv_block_tables), and the write of new rows into
// their slots (thd_kv_write).
//
// Block tables.  With n, m the cached and new tokens of a request and bs the
// page size: held = ceil(n / bs) pages are in its table, a growing request
// needs ceil((n + m) / bs) - held more, an ended one gives its held back.
// Prefix sums over the requests say everything: cu (rows), back (pages given
// back) and off (pages wanted).  Then every output is a flat loop whose element
// finds its request by bisection:
//   pushed page y:  free[n_free + y]       = table[b][y - back[b]]
//   popped page x:  table[b][held + x - off[b]] = stack(top - 1 - x)
//   packed row t:   pos = n + t - cu[b], page = pos / bs; a page below held is
//                   in the table, another one is popped page
//                   off[b] + page - held
// where stack(i) is free[i] below n_free and pushed page i - n_free above, read
// from the ended request's own row.  So no output depends on another one, and the
// work is shared by CTAs that each compute the sums for themselves.  Only where the
// lengths are updated in place must all have read them before one writes: there
// the CTAs are a cluster, with a barrier between the two.
//
// Latency bound: a few KB to a MB move.  A step of 256 requests is one CTA, whose
// time is loads, three barriers and the stores one after the other; for more each
// CTA gets about 4,096 rows, or 64 requests' pages, so that every loop below is
// gone through about once.  4,096 mixed requests and 131,072 rows: one CTA 228 us a
// pass, a cluster of eight 37 us, 64 CTAs 20 us (what the call takes).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/thd_attn.h"
#include "sm100_ptx.cuh"
#include "tma_map.h"

namespace {

constexpr int kTabThreads = 1024;
constexpr int kMaxReq = 8192;  // four int32 arrays of the requests in shared memory
constexpr int32_t kRefused = static_cast<int32_t>(0x80000000u);  // flag on a refused request's length
// CTAs that share the rows of a larger step: at most, and in a cluster.
constexpr int kTabCtas = 64, kTabCluster = 8;

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
    bool cluster;
};

// Exclusive prefix sums of one value per thread over the block, and the total.
// `sums` (32 values) is used by one call only, so one barrier is enough.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sums, int64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int64_t s = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    total = __shfl_sync(0xffffffffu, s, 31);
    const int64_t before = __shfl_sync(0xffffffffu, s, (warp + 31) & 31);
    return x - v + (warp > 0 ? before : 0);
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

// PER consecutive requests per thread.
template <int PER>
__global__ void __launch_bounds__(kTabThreads) thd_kv_block_tables_kernel(const TabParams p) {
    extern __shared__ int32_t arrays[];
    int32_t* cu = arrays;               // first packed row
    int32_t* back = cu + p.n_req;       // first pushed page
    int32_t* off = back + p.n_req;      // first popped page
    int32_t* seq = off + p.n_req;       // cached tokens
    __shared__ int64_t sums[4][32];
    const int tid = threadIdx.x;
    const int64_t bs = p.block;
    const int ctas = gridDim.x, me = blockIdx.x;
    constexpr int64_t kMax = 0x7fffffff;

    int n[PER], m[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = tid * PER + i;
        n[i] = b < p.n_req ? p.seq_lens[b] : -1;
        m[i] = b < p.n_req ? p.new_lens[b] : 0;
    }
    const int n_free = static_cast<int>(min(static_cast<int64_t>(max(*p.free_count, 0)), p.capacity));
    const int first = p.first_pos != nullptr ? *p.first_pos : 0;
    auto pages = [&](int64_t tokens) { return (tokens + bs - 1) / bs; };
    int64_t held[PER], total[PER];  // pages of n and of n + m tokens
    int64_t add = 0, give = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        held[i] = n[i] > 0 ? (n[i] - 1) / p.block + 1 : 0;
        total[i] = held[i];
        if (n[i] >= 0 && m[i] > 0) {
            add += m[i];
            total[i] = pages(static_cast<int64_t>(n[i]) + m[i]);
        }
        if (n[i] >= 0 && m[i] < 0) give += min(held[i], static_cast<int64_t>(p.max_blocks));
    }
    int64_t rows, pushed;
    add = block_scan(add, sums[0], rows);
    give = block_scan(give, sums[1], pushed);
    const int64_t top = min(n_free + pushed, p.capacity);
    // Pages wanted; a request refused for its width or rows wants none.
    int64_t want = 0;
    uint32_t narrow = 0;
    {
        int64_t r = add, g = give;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int b = tid * PER + i;
            if (b >= p.n_req) break;
            cu[b] = static_cast<int32_t>(min(r, kMax));
            back[b] = static_cast<int32_t>(min(g, kMax));
            if (n[i] >= 0 && m[i] >= 0) {
                r += m[i];
                if (m[i] > 0 && (total[i] > p.max_blocks || r > p.n_rows)) narrow |= 1u << i;
                else want += total[i] - held[i];
            } else if (n[i] >= 0) {
                g += min(held[i], static_cast<int64_t>(p.max_blocks));
            }
        }
    }
    int64_t wanted;
    int64_t o = block_scan(want, sums[2], wanted);
    int taken = 0;  // (at most the capacity)
    int n_refused = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = tid * PER + i;
        if (b >= p.n_req) break;
        off[b] = static_cast<int32_t>(min(o, kMax));
        bool no = (narrow >> i & 1u) != 0;
        if (!no && n[i] >= 0 && m[i] > 0) {
            const int64_t need = total[i] - held[i];
            no = need > 0 && o + need > top;
            if (!no && need > 0) taken = static_cast<int>(o + need);
            o += need;
        }
        n_refused += no;
        seq[b] = no ? n[i] | kRefused : n[i];
        m[i] = no ? 0 : m[i];
    }
    taken = __reduce_max_sync(0xffffffffu, taken);
    n_refused = __reduce_add_sync(0xffffffffu, n_refused);
    if ((tid & 31) == 0) sums[3][tid >> 5] = static_cast<int64_t>(n_refused) << 32 | static_cast<uint32_t>(taken);
    // (In a cluster every CTA has read the lengths and the count then.)
    __syncthreads();
    if (p.cluster) thd::cluster_sync();
    {
        const int64_t v = sums[3][tid & 31];
        taken = __reduce_max_sync(0xffffffffu, static_cast<int>(v & 0xffffffff));
        n_refused = __reduce_add_sync(0xffffffffu, static_cast<int>(v >> 32));
    }

    // The page at stack place i.
    auto stack = [&](int64_t i) -> int32_t {
        if (i < n_free) return p.free_blocks[i];
        const int32_t y = static_cast<int32_t>(i - n_free);
        const int b = find_request(back, p.n_req, y);
        return p.table[static_cast<int64_t>(b) * p.max_blocks + (y - back[b])];
    };
    if (me == 0) {
        if (tid == 0) {
            *p.free_out = static_cast<int32_t>(top - taken);
            *p.refused = n_refused;
            p.cu_out[p.n_req] = static_cast<int32_t>(min(rows, kMax));
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int b = tid * PER + i;
            if (b >= p.n_req) break;
            p.cu_out[b] = cu[b];
            p.seq_out[b] = n[i] < 0 || m[i] < 0 ? -1 : n[i] + m[i];
        }
    }
    const int64_t at = static_cast<int64_t>(me) * kTabThreads + tid, step = static_cast<int64_t>(ctas) * kTabThreads;
    // Pages of ended requests onto the stack (below max_blocks of a row, so the
    // row's own entries).
    const int64_t n_push = min(pushed, p.capacity - n_free);
    for (int64_t y = at; y < n_push; y += step) p.free_blocks[n_free + y] = stack(n_free + y);
    // New pages into the tables.
    for (int64_t x = at; x < taken; x += step) {
        const int b = find_request(off, p.n_req, static_cast<int32_t>(x));
        const int held_b = seq[b] > 0 ? (seq[b] - 1) / p.block + 1 : 0;
        p.table[static_cast<int64_t>(b) * p.max_blocks + held_b + (x - off[b])] = stack(top - 1 - x);
    }
    // Four packed rows at a time: the first one's request by bisection, the
    // others' by walking on.
    const bool vec = ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.positions)) & 15u) == 0;
    for (int64_t t0 = at * 4; t0 < p.n_rows; t0 += step * 4) {
        int slot[4], position[4];
        int b = t0 < rows ? find_request(cu, p.n_req, static_cast<int32_t>(t0)) : 0;
        int last_page = -1;
        int32_t id = -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t t = t0 + i;
            slot[i] = -1;
            position[i] = 0;
            if (t >= rows) continue;
            while (b + 1 < p.n_req && cu[b + 1] <= t) {
                ++b;
                last_page = -1;
            }
            const int have = seq[b] & ~kRefused;
            const int64_t far = static_cast<int64_t>(have) + (t - cu[b]);  // (a refused request may pass 2^31)
            position[i] = static_cast<int>(min(first + far, kMax));
            if (seq[b] >= 0) {
                const int pos = static_cast<int>(far), page = pos / p.block;
                if (page != last_page) {
                    const int held_b = have > 0 ? (have - 1) / p.block + 1 : 0;
                    id = page < held_b ? p.table[static_cast<int64_t>(b) * p.max_blocks + page]
                                       : stack(top - 1 - (off[b] + page - held_b));
                    last_page = page;
                }
                if (id >= 0 && id < kMax / bs) slot[i] = id * p.block + (pos - page * p.block);
            }
        }
        if (vec && t0 + 3 < p.n_rows) {
            *reinterpret_cast<int4*>(p.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            *reinterpret_cast<int4*>(p.positions + t0) = make_int4(position[0], position[1], position[2], position[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t0 + i < p.n_rows) {
                    p.slots[t0 + i] = slot[i];
                    p.positions[t0 + i] = position[i];
                }
        }
    }
}

// One thread per 16 bytes of a key and the same 16 bytes of a value.  Bound by
// memory: every byte is read once (so its line leaves L2 first) and written once.
// 65,536 rows of 8 heads x 128 (504 MB): 82 us, 6.1 TB/s, 94 % of a copy's rate
// (loads that stay in L2 86 us; two or four rows a thread 83 to 92 us).
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
        const uint4 k = __ldcs(reinterpret_cast<const uint4*>(p.k + r * p.k_row + h * p.D + d));
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p.v + r * p.v_row + h * p.D + d));
        *reinterpret_cast<uint4*>(p.kc + to) = k;
        *reinterpret_cast<uint4*>(p.vc + to) = v;
    }
}

template <int PER>
int launch_tables(const TabParams& p, int ctas, cudaStream_t stream) {
    const int smem = 16 * p.n_req;
    if (smem > 40000 && cudaFuncSetAttribute(thd_kv_block_tables_kernel<PER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             16 * kMaxReq) != cudaSuccess)
        return THD_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kTabThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = ctas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = p.cluster ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, thd_kv_block_tables_kernel<PER>, p) == cudaSuccess ? THD_OK : THD_ERR_CUDA;
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
                free_capacity, n_rows, n_req, block_size, max_blocks, false};
    int ctas = static_cast<int>(std::clamp<int64_t>(std::max<int64_t>(n_rows / 4096, n_req / 64), 1, kTabCtas));
    if (n_req <= 256 && n_rows <= 4096) ctas = 1;
    const bool in_place = seq_lens_out == seq_lens || seq_lens_out == new_lens || free_count_out == free_count;
    if (in_place) ctas = std::min(ctas, kTabCluster);
    p.cluster = ctas > 1 && in_place;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    const int per = (n_req + kTabThreads - 1) / kTabThreads;
    if (per == 1) return launch_tables<1>(p, ctas, stream);
    if (per == 2) return launch_tables<2>(p, ctas, stream);
    if (per <= 4) return launch_tables<4>(p, ctas, stream);
    return launch_tables<8>(p, ctas, stream);
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
