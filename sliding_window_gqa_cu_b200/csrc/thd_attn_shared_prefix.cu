// Attention of a step's new tokens over a shared prefix and each request's
// own pages of a paged cache (thd_attn_shared_prefix).  The pages print no
// serving form of MuseMagiPlan.attention / FlintMagiPlan.attention
// ("muse_spark.magi_cp", "flint.magi"): masks, GQA mapping, sinks and the
// log-sum-exp are those of the packed forward, over the sequence [prefix; own]
// of every request.
//
// Three launches, overlapped by programmatic dependent launch:
//   thd_sp_prefix_kernel  the shared prefix, once for all rows (tensor cores)
//   thd_sp_paged_kernel   each request's own pages (bound by memory); it runs
//                         on the SMs that the prefix kernel leaves
//   thd_sp_merge_kernel   adds the parts and the sinks, divides, writes
// With few rows on a short prefix the paged kernel takes that as well and the first
// launch falls away.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <numeric>
#include <type_traits>
#include <unordered_map>

#include "../../include/thd_attn.h"
#include "thd_sp_paged_kernel.cuh"
#include "thd_sp_prefix_kernel.cuh"
#include "tma_map.h"

namespace {

using thd::SpParams;

// Status word of the waits (a device symbol, so that a call allocates nothing
// and can be captured); one per device.
__device__ int g_sp_status;

// Adds up the parts of every row in a fixed order.  A CTA takes 8 consecutive rows
// of a kv head, a warp 16 columns of their parts of the prefix or of their own
// pages, a thread four columns of a row.  The parts are a few MB in L2 and the
// kernel is bound by the latency of its loads (plan, then places, then parts): 16
// threads find the rows' places for all, and four parts are loaded at a time.
// (Nothing branches on a part's maximum: the compiler would move the loads behind
// the branch, one latency after the other.)
template <int D>
__global__ void __launch_bounds__(512) thd_sp_merge_kernel(const SpParams p, const int* status) {
    constexpr int NT = thd::PrefixConfig<D>::NT;
    constexpr int BATCH = 4;
    constexpr int WARPS = D < 128 ? D / 16 : 8;  // of a run
    // A run of parts, of the prefix or of the request's pages: the home place,
    // then the own places of the following workers.
    struct Run {
        const float* home;  // of the row, column 0
        const float2* home_ml;
        const float* cont;
        const float2* cont_ml;
        int64_t part_step, ml_step;
        int n, home_rows, cont_rows, vacant;
    };
    __shared__ Run runs[2][8];
    __shared__ float own_part[WARPS][6][32];
    const int groups = (p.rows + 7) / 8;
    const int h = blockIdx.x / groups, row0 = (blockIdx.x - h * groups) * 8;
    const bool quads = p.pre_lanes > 0;  // the prefix's parts are the prefix kernel's
    thd::wait_for_previous_grid();
    // After a stall the places of the parts may not have been written: leave the rows.
    if (*reinterpret_cast<const volatile int*>(status) != 0) return;
    if (threadIdx.x < 16) {
        const int which = threadIdx.x >> 3, r = min(row0 + static_cast<int>(threadIdx.x & 7), p.rows - 1);
        const int b = r / p.RB, rr = r - b * p.RB;
        const int64_t bh = static_cast<int64_t>(b) * p.Hkv + h;
        const int pre_item = r / p.pg_rows * p.Hkv + h;
        const int n = thd::sp_own_len(p, b);
        thd::SpPlan plan{0, 0, 0, 0};
        long long begin = 0;  // (means nothing for an item without keys)
        if (p.any_keys) {
            plan = *p.plan;
            if (which == 1) begin = p.own_desc[bh * p.pg_units + rr / p.pg_rows];
            else if (p.pg_prefix > 0) begin = p.pgp_desc[pre_item];
            if (!quads && p.pg_prefix == 0) plan.pre_tiles = 0;
        }
        Run u;
        u.n = 0;
        u.home = u.cont = nullptr;
        u.home_ml = u.cont_ml = nullptr;
        u.part_step = u.ml_step = 0;
        u.home_rows = u.cont_rows = 0;
        u.vacant = n < 0 ? 1 : 0;
        long long units = plan.pg_units, x = begin + thd::kItemUnits;
        int lanes = plan.pg_lanes, count = plan.pre_tiles, step = 1, member = 0, tile_rows = p.pg_rows;
        if (which == 0 && quads) {
            const int tile = r >> 7, group = tile / NT, q = tile - group * NT, row = r & 127;
            const int len = plan.pre_tiles + thd::kItemTiles;
            units = static_cast<long long>((p.pre_groups + p.pre_width - 1) / p.pre_width) * p.Hkv * len;
            lanes = plan.pre_lanes;
            x = (static_cast<long long>(group / p.pre_width) * p.Hkv + h) * len + thd::kItemTiles;
            step = p.pre_width;
            member = group % p.pre_width;
            tile_rows = NT * 128;
            const int64_t at = (static_cast<int64_t>(h) * p.pre_groups + group) * NT + q;
            u.home = p.pre_home + at * (128 * D) + row * 4;
            u.home_ml = p.pre_home_ml + at * 128 + row;
            u.cont = p.pre_cont + static_cast<int64_t>(q) * (128 * D) + row * 4;
            u.cont_ml = p.pre_cont_ml + q * 128 + row;
            u.home_rows = u.cont_rows = 128;
        } else if (which == 0) {
            const int row = r % p.pg_rows;
            u.home_rows = u.cont_rows = p.pg_rows;
            u.home = p.pgp_home + static_cast<int64_t>(pre_item) * p.pg_rows * D + row * 4;
            u.home_ml = p.pgp_home_ml + static_cast<int64_t>(pre_item) * p.pg_rows + row;
            u.cont = p.pg_cont + row * 4;
            u.cont_ml = p.pg_cont_ml + row;
        } else {
            const int row = rr % p.pg_rows;
            count = thd::sp_own_slices(p, n);
            u.home_rows = p.RB;
            u.cont_rows = p.pg_rows;
            u.home = p.own_home + bh * p.RB * D + rr * 4;
            u.home_ml = p.own_home_ml + bh * p.RB + rr;
            u.cont = p.pg_cont + row * 4;
            u.cont_ml = p.pg_cont_ml + row;
        }
        if (count > 0) {
            const int first = thd::lane_of(units, lanes, x), last = thd::lane_of(units, lanes, x + count - 1);
            u.n = last - first + 1;
            u.part_step = static_cast<int64_t>(step) * tile_rows * D;
            u.ml_step = static_cast<int64_t>(step) * tile_rows;
            // (places of workers first + 1, .. follow: part 0 is the home place)
            const int64_t at = (static_cast<int64_t>(first) * step + member) * tile_rows;
            u.cont += at * D;
            u.cont_ml += at;
        }
        runs[which][threadIdx.x & 7] = u;
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, r = row0 + (lane & 7), warp = threadIdx.x >> 5;
    const int which = warp / WARPS;
    const int c4 = (blockIdx.y * WARPS + warp % WARPS) * 4 + (lane >> 3);
    float m = -INFINITY, l = 0.0f;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    {
        const Run u = runs[which][lane & 7];
        const float* part = u.home + c4 * 4 * u.home_rows;
        const float2* ml_at = u.home_ml;
        const float* cont = u.cont + c4 * 4 * u.cont_rows + u.part_step;
        const float2* cont_ml = u.cont_ml + u.ml_step;
        const int n = u.n;
#pragma unroll 1
        for (int c0 = 0; c0 < n; c0 += BATCH) {
            float2 ml[BATCH];
            float4 o[BATCH];
#pragma unroll
            for (int c = 0; c < BATCH; ++c) {
                ml[c] = __ldcg(ml_at);
                o[c] = __ldcg(reinterpret_cast<const float4*>(part));
                if (c0 + c >= n) ml[c].x = -INFINITY;  // (the last part again)
                if (c0 + c + 1 < n) {
                    part = cont;
                    ml_at = cont_ml;
                    cont += u.part_step;
                    cont_ml += u.ml_step;
                }
            }
            float top = m;
#pragma unroll
            for (int c = 0; c < BATCH; ++c) top = fmaxf(top, ml[c].x);
            const float base = top == -INFINITY ? 0.0f : top;
            const float a = exp2f(m - base);
            m = top;
            l *= a;
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[k] *= a;
#pragma unroll
            for (int c = 0; c < BATCH; ++c) {
                const float x = exp2f(ml[c].x - base);
                const bool there = x > 0.0f;  // (a part with nothing in it may never have been written)
                l = fmaf(there ? ml[c].y : 0.0f, x, l);
                acc[0] = fmaf(there ? o[c].x : 0.0f, x, acc[0]);
                acc[1] = fmaf(there ? o[c].y : 0.0f, x, acc[1]);
                acc[2] = fmaf(there ? o[c].z : 0.0f, x, acc[2]);
                acc[3] = fmaf(there ? o[c].w : 0.0f, x, acc[3]);
            }
        }
    }
    if (which == 1) {
        float(&at)[6][32] = own_part[warp - WARPS];
#pragma unroll
        for (int k = 0; k < 4; ++k) at[k][lane] = acc[k];
        at[4][lane] = m;
        at[5][lane] = l;
    }
    __syncthreads();
    if (which == 1 || r >= p.rows || runs[0][lane & 7].vacant) return;
    const int t = r / p.G, head = h * p.G + (r - t * p.G);
    const float sink = p.sinks != nullptr ? p.sinks[head] * 1.4426950408889634f : -INFINITY;
    const float(&own)[6][32] = own_part[warp];
    const float top = fmaxf(fmaxf(m, own[4][lane]), sink);
    const float base = top == -INFINITY ? 0.0f : top;
    const float x = exp2f(m - base), y = exp2f(own[4][lane] - base);
    const float sum = l * x + own[5][lane] * y + exp2f(sink - base);
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = (acc[k] * x + own[k][lane] * y) * inv;
    const int64_t orow = static_cast<int64_t>(t) * p.Hq + head;
    *reinterpret_cast<uint2*>(p.out + orow * D + c4 * 4) =
        make_uint2(thd::pack_bf16x2(acc[0], acc[1]), thd::pack_bf16x2(acc[2], acc[3]));
    if (p.lse != nullptr && c4 == 0)
        p.lse[orow] = sum > 0.0f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

constexpr int kMaxUnits = 4096;
constexpr int kPagedCtas = 3 * thd::kSpLanes;  // three fit an SM
// Up to this many rows of a kv head the blocks may lie any distance apart (the paged
// kernel takes the prefix where the prefix kernel's map cannot).
constexpr int kAnyPlacesRows = 32;

// Whether the paged kernel takes a prefix (of at most `tokens`, what its table
// holds: the length itself lies on the device) too, once per row tile: it is done with
// few keys before another launch has started.  Paged against prefix kernel, whole
// calls with 100 own tokens, us:
//   8 kv heads of 128  16 rows 4,096 keys 26 and 27, 8,192 32 and 32; 32 rows 4,096 27 and
//                      28, 8,192 37 and 33; 64 rows 1,024 22 and 26, 4,096 32 and 29; 256 rows
//                      1,024 30 and 29
//   8 kv heads of 64   the same to within 5 %
//   2 kv heads of 128  fewer SMs share the work of a long prefix: 8 rows 4,096 keys 9 %
//                      slower, 16,384 15 %; 64 rows 4,096 keys 6 % faster, 256 rows
//                      1,024 14 %
// so 2^18 rows times keys is within 20 % either way of where the two meet.  Tiles of more
// rows are bound by products and those of 256 columns have slower slices (8 rows of 256
// columns: 2,048 keys 7 to 11 % slower, 4,096 30 %).  One tile of 8 rows leaves the prefix
// kernel little to share (8 kv heads of 128: 5 to 18 % faster up to 32,768 keys).
bool prefix_by_pages(int tiles, int tile_rows, int64_t tokens, int D) {
    if (tile_rows == 8 && D <= 128) return tiles == 1 || tokens * tiles * tile_rows <= 1 << 18;
    return tokens <= 2048 && tokens * tiles * tile_rows <= 1 << 18;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// The split of the work and the places in the workspace, from the sizes alone.
struct Layout {
    int rows, RB, pg_rows, pg_units, pg_prefix, pre_groups, pre_width, pre_lanes;
    size_t own_home, own_home_ml, own_desc, pg_cont, pg_cont_ml, plan;
    size_t pgp_home, pgp_home_ml, pgp_desc;                   // paged prefix
    size_t pre_home, pre_home_ml, pre_cont, pre_cont_ml;      // prefix kernel
    size_t bytes;
};

Layout make_layout(int n_req, int n_q, int Hq, int Hkv, int D) {
    Layout y{};
    y.RB = n_q * (Hq / Hkv);
    y.rows = n_req * y.RB;
    y.pg_rows = y.RB <= 8 ? 8 : y.RB <= 16 ? 16 : y.RB <= 32 || D == 256 ? 32 : 64;
    y.pg_units = (y.RB + y.pg_rows - 1) / y.pg_rows;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += align256(bytes);
        return here;
    };
    const size_t all = static_cast<size_t>(y.rows) * Hkv;
    y.plan = take(sizeof(thd::SpPlan));
    y.own_home = take(all * D * 4);
    y.own_home_ml = take(all * 8);
    y.own_desc = take(static_cast<size_t>(n_req) * Hkv * y.pg_units * 8);
    // Workers of a CTA x rows of a tile: 32 rows (8 a warp) or 64.
    const int warp_rows = y.pg_rows == 8 || D == 256 ? 8 : 16;
    y.pg_cont = take(static_cast<size_t>(kPagedCtas) * 4 * warp_rows * D * 4);
    y.pg_cont_ml = take(static_cast<size_t>(kPagedCtas) * 4 * warp_rows * 8);
    // The prefix's parts, of the paged kernel or in the same place of the prefix kernel.
    const size_t shared = at;
    y.pg_prefix = (y.rows + y.pg_rows - 1) / y.pg_rows;
    const size_t tiles = static_cast<size_t>(y.pg_prefix) * Hkv;
    y.pgp_home = take(tiles * y.pg_rows * D * 4);
    y.pgp_home_ml = take(tiles * y.pg_rows * 8);
    y.pgp_desc = take(tiles * 8);
    const size_t end = at;
    at = shared;
    const int tile = D == 256 ? 128 : 256;  // rows of a group
    y.pre_groups = (y.rows + tile - 1) / tile;
    // Groups in step: as many as keep the CTAs busy (idle ones and empty
    // places of the last bundle cost their share, reading K and V for fewer
    // groups at once about 0.15 / width).
    double best = -1.0;
    for (int w = 1; w <= std::min(y.pre_groups, 8); ++w) {
        const int bundles = (y.pre_groups + w - 1) / w, lanes = thd::kSpLanes / w;
        const double busy = static_cast<double>(y.pre_groups) / (bundles * w) * (lanes * w) / thd::kSpLanes;
        const double score = busy / (1.0 + 0.15 / w);
        if (score > best) {
            best = score;
            y.pre_width = w;
            y.pre_lanes = lanes;
        }
    }
    const size_t padded = static_cast<size_t>(y.pre_groups) * tile;
    y.pre_home = take(padded * Hkv * D * 4);
    y.pre_home_ml = take(padded * Hkv * 8);
    y.pre_cont = take(static_cast<size_t>(thd::kSpLanes) * tile * D * 4);
    y.pre_cont_ml = take(static_cast<size_t>(thd::kSpLanes) * tile * 8);
    at = std::max(at, end);
    y.bytes = at;
    return y;
}

// The kernels' shared memory, once per device.
template <class K>
bool allow_smem(K kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return false;
    if (done.load(std::memory_order_relaxed) >> dev & 1) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    // All of the SM's shared memory, so that both kernels' CTAs fit it together.
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
        cudaSuccess)
        return false;
    done.fetch_or(1ull << dev, std::memory_order_relaxed);
    return true;
}

// Launch that may begin when every CTA of the kernel before it has allowed it.
template <class... P, class... A>
bool launch_early(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, bool early, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

template <int D>
bool launch_prefix(const SpParams& p, const CUtensorMap& mk, const CUtensorMap& mv, int* status, cudaStream_t stream) {
    using C = thd::PrefixConfig<D>;
    static std::atomic<uint64_t> done{0};
    return allow_smem(thd::thd_sp_prefix_kernel<C>, C::SMEM_BYTES, done) &&
           launch_early(thd::thd_sp_prefix_kernel<C>, dim3(p.pre_lanes * p.pre_width), C::THREADS, C::SMEM_BYTES, stream,
                        false, mk, mv, p, status);
}

template <int D, int NR, int WR>
bool launch_paged(const SpParams& p, int* status, bool early, cudaStream_t stream) {
    using C = thd::PagedConfig<D, NR, WR>;
    static std::atomic<uint64_t> done{0};
    return allow_smem(thd::thd_sp_paged_kernel<C>, C::SMEM_BYTES, done) &&
           launch_early(thd::thd_sp_paged_kernel<C>, dim3(p.pg_ctas), C::THREADS, C::SMEM_BYTES, stream, early,
                        p, status);
}

struct Maps {
    CUtensorMap k, v;
};

template <int D>
int launch_all(SpParams p, const Maps& maps, cudaStream_t stream) {
    void* status = nullptr;
    if (cudaGetSymbolAddress(&status, g_sp_status) != cudaSuccess) return THD_ERR_CUDA;
    int* st = static_cast<int*>(status);
    bool early = false;
    p.pg_slice = p.pg_rows == 8 || D == 256 ? thd::PagedConfig<D, 1, 1>::KS : thd::PagedConfig<D, 2, 1>::KS;
    if (p.any_keys) {
        if (p.pre_lanes > 0) {
            if (!launch_prefix<D>(p, maps.k, maps.v, st, stream)) return THD_ERR_CUDA;
            early = true;
        }
        // No more CTAs than there can be slices (tables may be longer than what is used).
        const int64_t slices = (static_cast<int64_t>(p.max_blocks) * p.pg_units * p.n_req +
                                static_cast<int64_t>(p.prefix_blocks) * p.pg_prefix) * (p.block / 16) * p.Hkv;
        p.pg_ctas = static_cast<int>(std::clamp<int64_t>(slices, 1, kPagedCtas));
        bool ok;
        if (p.pg_rows == 8) ok = launch_paged<D, 1, 1>(p, st, early, stream);
        else if constexpr (D == 256)
            ok = p.pg_rows == 16 ? launch_paged<D, 1, 2>(p, st, early, stream)
                                 : launch_paged<D, 1, 4>(p, st, early, stream);
        else
            ok = p.pg_rows == 16   ? launch_paged<D, 2, 1>(p, st, early, stream)
                 : p.pg_rows == 32 ? launch_paged<D, 2, 2>(p, st, early, stream)
                                   : launch_paged<D, 2, 4>(p, st, early, stream);
        if (!ok) return THD_ERR_CUDA;
        early = true;
    }
    const int64_t ctas = static_cast<int64_t>(p.Hkv) * ((p.rows + 7) / 8);
    if (!launch_early(thd_sp_merge_kernel<D>, dim3(static_cast<unsigned>(ctas), D > 128 ? D / 128 : 1),
                      D < 128 ? 4 * D : 512, 0, stream, early,
                      static_cast<const SpParams&>(p), static_cast<const int*>(st)))
        return THD_ERR_CUDA;
    return THD_OK;
}

}  // namespace

extern "C" size_t thd_attn_shared_prefix_workspace_bytes(int n_req, int n_q, int Hq, int Hkv, int D) {
    if (n_req <= 0 || n_q <= 0 || Hkv <= 0 || Hq <= 0 || Hq % Hkv != 0 || D <= 0) return 0;
    if (D != 64 && D != 128 && D != 256) return 0;
    const int64_t G = Hq / Hkv;
    if (G > 128 || n_req * ((n_q + 128 / G - 1) / (128 / G)) > kMaxUnits) return 0;
    return make_layout(n_req, n_q, Hq, Hkv, D).bytes;
}

extern "C" int thd_attn_shared_prefix(const void* q, const void* k_cache, const void* v_cache,
                                      int64_t num_blocks, int block_size, int64_t block_stride,
                                      int64_t token_stride, int64_t head_stride,
                                      const int32_t* prefix_table_or_null, int prefix_blocks,
                                      const int32_t* prefix_len_or_null, const int32_t* block_tables,
                                      int max_blocks, const int32_t* kv_lens, int n_req, int n_q, int Hq,
                                      int Hkv, int D, int window, float scale, const float* sinks_or_null,
                                      void* out, float* lse, void* workspace, size_t workspace_bytes,
                                      void* stream_ptr) {
    constexpr int64_t kMax = 0x7fffffff;
    if (n_req < 0 || n_q < 1 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || window < 0 || num_blocks < 0 ||
        prefix_blocks < 0 || max_blocks < 0)
        return THD_ERR_INVALID_ARG;
    if (!(std::isfinite(scale) && scale > 0.0f)) return THD_ERR_INVALID_ARG;
    if (D != 64 && D != 128 && D != 256) return THD_ERR_UNSUPPORTED;
    const int G = Hq / Hkv;
    if (G > 128) return THD_ERR_UNSUPPORTED;
    if (block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128 && block_size != 256)
        return THD_ERR_UNSUPPORTED;
    const int64_t tokens_per_tile = 128 / G;
    if (n_req * ((n_q + tokens_per_tile - 1) / tokens_per_tile) > kMaxUnits) return THD_ERR_UNSUPPORTED;
    if (num_blocks > kMax / block_size ||
        (static_cast<int64_t>(prefix_blocks) + max_blocks) * block_size > kMax)
        return THD_ERR_INVALID_ARG;
    if ((prefix_table_or_null == nullptr) != (prefix_len_or_null == nullptr)) return THD_ERR_INVALID_ARG;
    if (prefix_table_or_null == nullptr) prefix_blocks = 0;
    if (n_req == 0) return THD_OK;
    if (!q || !kv_lens || !out || !workspace || (max_blocks > 0 && !block_tables) ||
        (num_blocks > 0 && (!k_cache || !v_cache)))
        return THD_ERR_INVALID_ARG;
    if (!thd::aligned16(q) || !thd::aligned16(k_cache) || !thd::aligned16(v_cache) || !thd::aligned16(out) ||
        !thd::aligned16(workspace) || !aligned4(prefix_table_or_null) || !aligned4(prefix_len_or_null) ||
        !aligned4(block_tables) || !aligned4(kv_lens) || !aligned4(sinks_or_null) || !aligned4(lse))
        return THD_ERR_INVALID_ARG;
    if (block_stride < 0 || token_stride < D || head_stride < D ||
        (block_stride | token_stride | head_stride) % 8 != 0)
        return THD_ERR_INVALID_ARG;
    if (workspace_bytes < thd_attn_shared_prefix_workspace_bytes(n_req, n_q, Hq, Hkv, D))
        return THD_ERR_INVALID_ARG;
    SpParams p{};
    // Without blocks there are no keys: the merge alone writes the rows.
    const bool any_keys = num_blocks > 0 && prefix_blocks + static_cast<int64_t>(max_blocks) > 0;
    if (!any_keys) prefix_blocks = max_blocks = 0;
    const bool prefix = prefix_blocks > 0;
    const Layout y = make_layout(n_req, n_q, Hq, Hkv, D);
    // The prefix kernel's map counts places in units of the strides' divisor.
    const int64_t bs = num_blocks > 1 ? block_stride : 0, hs = Hkv > 1 ? head_stride : 0;
    const int64_t g = std::max<int64_t>(std::gcd(bs, hs), 8);
    const int64_t places = any_keys ? (num_blocks - 1) * (bs / g) + (Hkv - 1) * (hs / g) + 1 : 0;
    if (prefix && places > kMax && y.rows > kAnyPlacesRows) return THD_ERR_UNSUPPORTED;
    const bool by_pages = places > kMax || prefix_by_pages(y.pg_prefix, y.pg_rows, static_cast<int64_t>(prefix_blocks) * block_size, D);
    char* ws = static_cast<char*>(workspace);
    auto f = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    auto f2 = [&](size_t at) { return reinterpret_cast<float2*>(ws + at); };
    auto i8 = [&](size_t at) { return reinterpret_cast<long long*>(ws + at); };
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.kc = static_cast<const __nv_bfloat16*>(k_cache);
    p.vc = static_cast<const __nv_bfloat16*>(v_cache);
    p.block_stride = block_stride;
    p.token_stride = token_stride;
    p.head_stride = head_stride;
    p.any_keys = any_keys ? 1 : 0;
    p.prefix_table = prefix ? prefix_table_or_null : nullptr;
    p.prefix_len = prefix ? prefix_len_or_null : nullptr;
    p.tables = block_tables;
    p.kv_lens = kv_lens;
    p.sinks = sinks_or_null;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.num_blocks = static_cast<int>(num_blocks);
    p.block = block_size;
    while (1 << p.block_shift < block_size) ++p.block_shift;
    p.prefix_blocks = prefix_blocks;
    p.max_blocks = max_blocks;
    p.n_req = n_req;
    p.n_q = n_q;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = G;
    // A window as long as all tables hides nothing.
    p.window = window >= (static_cast<int64_t>(prefix_blocks) + max_blocks) * block_size ? 0 : window;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.RB = y.RB;
    p.rows = y.rows;
    p.box_rows = std::min(block_size, 128);
    p.pre_groups = y.pre_groups;
    p.pre_width = y.pre_width;
    p.pre_lanes = prefix && !by_pages ? y.pre_lanes : 0;
    p.pre_home = f(y.pre_home);
    p.pre_home_ml = f2(y.pre_home_ml);
    p.pre_cont = f(y.pre_cont);
    p.pre_cont_ml = f2(y.pre_cont_ml);
    p.plan = reinterpret_cast<thd::SpPlan*>(ws + y.plan);
    p.pg_rows = y.pg_rows;
    p.pg_units = y.pg_units;
    p.pg_prefix = prefix && by_pages ? y.pg_prefix : 0;
    p.own_home = f(y.own_home);
    p.own_home_ml = f2(y.own_home_ml);
    p.own_desc = i8(y.own_desc);
    p.pgp_home = f(y.pgp_home);
    p.pgp_home_ml = f2(y.pgp_home_ml);
    p.pgp_desc = i8(y.pgp_desc);
    p.pg_cont = f(y.pg_cont);
    p.pg_cont_ml = f2(y.pg_cont_ml);
    Maps maps{};
    if (any_keys && p.pre_lanes > 0) {
        p.places = static_cast<int>(places);
        p.place_block = static_cast<int>(bs / g);
        p.place_head = static_cast<int>(hs / g);
        auto map = [&](CUtensorMap* m, const void* base) {
            return thd::make_paged_map(m, base, block_size, D, token_stride, g, places, p.box_rows, std::min(D, 128) / 64);
        };
        if (!map(&maps.k, k_cache) || !map(&maps.v, v_cache)) return THD_ERR_INVALID_ARG;
    }
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    switch (D) {
        case 64: return launch_all<64>(p, maps, stream);
        case 128: return launch_all<128>(p, maps, stream);
        default: return launch_all<256>(p, maps, stream);
    }
}

// Stalls found so far on a device, and how many of them each stream has been told of.
// One word is enough for the kernels, but whoever reads it first must not take the
// report away from the other streams, whose calls wrote nothing either.
struct SpReports {
    uint64_t stalls = 0;
    int last = THD_OK;
    std::unordered_map<void*, uint64_t> told;
};
static std::mutex g_sp_reports_mu;
static SpReports g_sp_reports[64];

extern "C" int thd_attn_shared_prefix_get_error(void* stream_ptr) {
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream_ptr)) != cudaSuccess) return THD_ERR_CUDA;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return THD_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_sp_reports_mu);
    SpReports& r = g_sp_reports[dev];
    int s = 0;
    if (cudaMemcpyFromSymbol(&s, g_sp_status, sizeof(int)) != cudaSuccess) return THD_ERR_CUDA;
    if (s != 0) {
        // The word stays until every call that it stops has ended: a merge that found it
        // taken back would add up parts that were never written.
        const int zero = 0;
        if (cudaDeviceSynchronize() != cudaSuccess ||
            cudaMemcpyToSymbol(g_sp_status, &zero, sizeof(int)) != cudaSuccess)
            return THD_ERR_CUDA;
        ++r.stalls;
        r.last = s;
    }
    if (r.stalls == 0) return THD_OK;
    try {
        uint64_t& told = r.told[stream_ptr];
        if (told == r.stalls) return THD_OK;
        told = r.stalls;
    } catch (...) {  // no host memory: the stream is told again next time
    }
    return r.last;
}

#if THD_DEBUG
// Debug build: sets the status word, as a stalled kernel would (no kernel has to stall
// for the tests of what follows a stall).
extern "C" int thd_attn_shared_prefix_set_status(int status) {
    return cudaMemcpyToSymbol(g_sp_status, &status, sizeof(int)) == cudaSuccess ? THD_OK : THD_ERR_CUDA;
}
#endif
