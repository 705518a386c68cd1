// Attention of a step's new tokens over a shared prefix and each request's
// own pages of a paged cache (thd_attn_shared_prefix).  The pages print no
// serving form of MuseMagiPlan.attention / FlintMagiPlan.attention
// ("muse_spark.magi_cp", "flint.magi"): masks, GQA mapping, sinks and the
// log-sum-exp are those of the packed forward, over the sequence [prefix; own]
// of every request.
//
// Three launches, overlapped by programmatic dependent launch:
//   thd_sp_prefix_kernel  the shared prefix, once for all rows (tensor cores)
//   thd_sp_paged_kernel   each request's own pages (bound by memory); it starts
//                         while the prefix kernel runs and shares its SMs
//   thd_sp_merge_kernel   adds the parts and the sinks, divides, writes
// With few rows in all (one row tile of the paged kernel) that kernel takes the
// prefix as well and the first launch falls away.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/thd_attn.h"
#include "thd_sp_paged_kernel.cuh"
#include "thd_sp_prefix_kernel.cuh"
#include "tma_map.h"

namespace {

using thd::SpParams;

// Status word of the waits (a device symbol, so that a call allocates nothing
// and can be captured); one per device.
__device__ int g_sp_status;

// Adds up the parts of every row in a fixed order.  A warp takes 8 consecutive
// rows of a kv head x 64 columns; a thread one row and four groups of four
// columns.  Reads the parts once (a few MB): a small fraction of the step.
template <int D>
__global__ void __launch_bounds__(256) thd_sp_merge_kernel(const SpParams p) {
    constexpr int NT = thd::PrefixConfig<D>::NT;
    constexpr int KT = thd::PagedConfig<D, 1>::KT;
    const int lane = threadIdx.x & 31;
    const int groups = (p.rows + 7) / 8;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int h = static_cast<int>(w / groups);
    const int r = static_cast<int>(w - static_cast<int64_t>(h) * groups) * 8 + (lane & 7);
    const int c4 = blockIdx.y * 16 + (lane >> 3);
    thd::wait_for_previous_grid();
    if (h >= p.Hkv || r >= p.rows) return;
    const int b = r / p.RB, rr = r - b * p.RB;
    const int n = thd::sp_own_len(p, b);
    if (n < 0) return;

    // Up to two sources (the prefix and the request's pages), each a home place
    // and the own places of CTAs first, first + step, ... < end.
    struct Source {
        const float* home;
        const float2* home_ml;
        const float* cont;
        const float2* cont_ml;
        int64_t cont_tile;
        int rows, row, cont_row, cont_rows, first, end, step;
    } src[2];
    int n_src = 0;
    const int pre_tiles = p.pre_lanes > 0 || p.pg_prefix > 0 ? p.pre_plan[1] : 0;
    if (pre_tiles > 0 && p.pre_lanes > 0) {
        const int tile = r >> 7, group = tile / NT;
        const long long units = static_cast<long long>((p.pre_groups + p.pre_width - 1) / p.pre_width) * p.Hkv * pre_tiles;
        const int lanes = static_cast<int>(min(units, static_cast<long long>(p.pre_lanes)));
        const long long x = (static_cast<long long>(group / p.pre_width) * p.Hkv + h) * pre_tiles;
        const int member = group % p.pre_width, q = tile - group * NT;
        const int64_t at = (static_cast<int64_t>(h) * p.pre_groups + group) * NT + q;
        src[n_src++] = Source{p.pre_home + at * (128 * D), p.pre_home_ml + at * 128,
                              p.pre_cont + static_cast<int64_t>(q) * (128 * D), p.pre_cont_ml + q * 128,
                              static_cast<int64_t>(NT) * 128, 128, r & 127, r & 127, 128,
                              (thd::lane_of(units, lanes, x) + 1) * p.pre_width + member,
                              thd::lane_of(units, lanes, x + pre_tiles - 1) * p.pre_width + member + 1, p.pre_width};
    } else if (pre_tiles > 0) {
        const int item = r / p.pg_rows * p.Hkv + h, row = r % p.pg_rows;
        const int2 d = p.pgp_desc[item];
        src[n_src++] = Source{p.pgp_home + static_cast<int64_t>(item) * p.pg_rows * D,
                              p.pgp_home_ml + static_cast<int64_t>(item) * p.pg_rows, p.pg_cont, p.pg_cont_ml,
                              p.pg_rows, p.pg_rows, row, row, p.pg_rows, d.x + 1, d.y + 1, 1};
    }
    if (thd::sp_own_tiles<KT>(p, n) > 0) {
        const int64_t bh = static_cast<int64_t>(b) * p.Hkv + h;
        const int2 d = p.own_desc[bh * p.pg_units + rr / p.pg_rows];
        src[n_src++] = Source{p.own_home + bh * p.RB * D, p.own_home_ml + bh * p.RB, p.pg_cont, p.pg_cont_ml,
                              p.pg_rows, p.RB, rr, rr % p.pg_rows, p.pg_rows, d.x + 1, d.y + 1, 1};
    }
    const int g = r % p.G, head = h * p.G + g;
    const int64_t t = r / p.G;
    float m = -INFINITY;
    const float sink = p.sinks != nullptr ? p.sinks[head] * 1.4426950408889634f : -INFINITY;
    m = sink;
    for (int i = 0; i < n_src; ++i) {
        const Source& s = src[i];
        m = fmaxf(m, s.home_ml[s.row].x);
#pragma unroll 4
        for (int c = s.first; c < s.end; c += s.step) m = fmaxf(m, s.cont_ml[c * s.cont_tile + s.cont_row].x);
    }
    float l = sink == -INFINITY ? 0.0f : exp2f(sink - m);
    float4 acc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float* part, int rows, int row, float2 ml) {
        if (ml.x == -INFINITY) return;  // (nothing was stored)
        const float a = exp2f(ml.x - m);
        l = fmaf(ml.y, a, l);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 o = *reinterpret_cast<const float4*>(part + (static_cast<int64_t>(c4 + 4 * k) * rows + row) * 4);
            acc[k].x = fmaf(o.x, a, acc[k].x);
            acc[k].y = fmaf(o.y, a, acc[k].y);
            acc[k].z = fmaf(o.z, a, acc[k].z);
            acc[k].w = fmaf(o.w, a, acc[k].w);
        }
    };
    for (int i = 0; i < n_src; ++i) {
        const Source& s = src[i];
        add(s.home, s.rows, s.row, s.home_ml[s.row]);
#pragma unroll 2
        for (int c = s.first; c < s.end; c += s.step)
            add(s.cont + c * s.cont_tile * D, s.cont_rows, s.cont_row, s.cont_ml[c * s.cont_tile + s.cont_row]);
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    __nv_bfloat16* o = p.out + (t * p.Hq + head) * D;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint2*>(o + (c4 + 4 * k) * 4) = make_uint2(thd::pack_bf16x2(acc[k].x * inv, acc[k].y * inv),
                                                                    thd::pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
    if (p.lse != nullptr && blockIdx.y == 0 && lane < 8)
        p.lse[t * p.Hq + head] = l > 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

constexpr int kMaxUnits = 4096;
constexpr int kPagedCtas = 3 * thd::kSpLanes;  // three fit an SM
// The paged kernel takes the prefix too when all rows of a kv head fit one row
// tile of two 16-row groups.
constexpr int kPagedPrefixRows = 32;

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
    const bool small = y.rows <= kPagedPrefixRows;
    const int want = small ? y.rows : y.RB;
    y.pg_rows = want <= 16 ? 16 : want <= 32 || D == 256 ? 32 : 64;
    y.pg_units = (y.RB + y.pg_rows - 1) / y.pg_rows;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += align256(bytes);
        return here;
    };
    const size_t all = static_cast<size_t>(y.rows) * Hkv;
    y.plan = take(8);
    y.own_home = take(all * D * 4);
    y.own_home_ml = take(all * 8);
    y.own_desc = take(static_cast<size_t>(n_req) * Hkv * y.pg_units * 8);
    y.pg_cont = take(static_cast<size_t>(kPagedCtas) * y.pg_rows * D * 4);
    y.pg_cont_ml = take(static_cast<size_t>(kPagedCtas) * y.pg_rows * 8);
    if (small) {
        y.pg_prefix = 1;
        y.pgp_home = take(static_cast<size_t>(Hkv) * y.pg_rows * D * 4);
        y.pgp_home_ml = take(static_cast<size_t>(Hkv) * y.pg_rows * 8);
        y.pgp_desc = take(static_cast<size_t>(Hkv) * 8);
    } else {
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
    }
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

template <int D, int WR>
bool launch_paged(const SpParams& p, const CUtensorMap& mk, const CUtensorMap& mv, int* status, bool early,
                  cudaStream_t stream) {
    using C = thd::PagedConfig<D, WR>;
    static std::atomic<uint64_t> done{0};
    return allow_smem(thd::thd_sp_paged_kernel<C>, C::SMEM_BYTES, done) &&
           launch_early(thd::thd_sp_paged_kernel<C>, dim3(p.pg_ctas), C::THREADS, C::SMEM_BYTES, stream, early, mk, mv, p,
                        status);
}

struct Maps {
    CUtensorMap pre_k, pre_v, pg_k, pg_v;
};

template <int D>
int launch_all(SpParams p, const Maps& maps, bool any_keys, cudaStream_t stream) {
    void* status = nullptr;
    if (cudaGetSymbolAddress(&status, g_sp_status) != cudaSuccess) return THD_ERR_CUDA;
    int* st = static_cast<int*>(status);
    bool early = false;
    if (any_keys) {
        if (p.pre_lanes > 0) {
            if (!launch_prefix<D>(p, maps.pre_k, maps.pre_v, st, stream)) return THD_ERR_CUDA;
            early = true;
        }
        constexpr int KT = 32;  // (the least of the variants' tiles)
        const int64_t own = (static_cast<int64_t>(p.max_blocks) * p.block + KT - 1) / KT * p.pg_units * p.n_req;
        const int64_t pre = (static_cast<int64_t>(p.prefix_blocks) * p.block + KT - 1) / KT * p.pg_prefix;
        p.pg_ctas = static_cast<int>(std::clamp<int64_t>((own + pre) * p.Hkv, 1, kPagedCtas));
        bool ok;
        if (p.pg_rows == 16) ok = launch_paged<D, 1>(p, maps.pg_k, maps.pg_v, st, early, stream);
        else if (p.pg_rows == 32) ok = launch_paged<D, 2>(p, maps.pg_k, maps.pg_v, st, early, stream);
        else if constexpr (D != 256) ok = launch_paged<D, 4>(p, maps.pg_k, maps.pg_v, st, early, stream);
        else ok = false;
        if (!ok) return THD_ERR_CUDA;
        early = true;
    }
    const int64_t warps = static_cast<int64_t>(p.Hkv) * ((p.rows + 7) / 8);
    if (!launch_early(thd_sp_merge_kernel<D>, dim3(static_cast<unsigned>((warps + 7) / 8), D / 64), 256, 0, stream, early, p))
        return THD_ERR_CUDA;
    return THD_OK;
}

}  // namespace

extern "C" size_t thd_attn_shared_prefix_workspace_bytes(int n_req, int n_q, int Hq, int Hkv, int D) {
    if (n_req <= 0 || n_q <= 0 || Hkv <= 0 || Hq <= 0 || Hq % Hkv != 0 || D <= 0) return 0;
    if (D != 64 && D != 128 && D != 256) return 0;
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
    char* ws = static_cast<char*>(workspace);
    auto f = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    auto f2 = [&](size_t at) { return reinterpret_cast<float2*>(ws + at); };
    auto i2 = [&](size_t at) { return reinterpret_cast<int2*>(ws + at); };
    p.q = static_cast<const __nv_bfloat16*>(q);
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
    p.pre_lanes = prefix ? y.pre_lanes : 0;
    p.pre_home = f(y.pre_home);
    p.pre_home_ml = f2(y.pre_home_ml);
    p.pre_cont = f(y.pre_cont);
    p.pre_cont_ml = f2(y.pre_cont_ml);
    p.pre_plan = reinterpret_cast<int*>(ws + y.plan);
    p.pg_rows = y.pg_rows;
    p.pg_units = y.pg_units;
    p.pg_prefix = prefix ? y.pg_prefix : 0;
    p.own_home = f(y.own_home);
    p.own_home_ml = f2(y.own_home_ml);
    p.own_desc = i2(y.own_desc);
    p.pgp_home = f(y.pgp_home);
    p.pgp_home_ml = f2(y.pgp_home_ml);
    p.pgp_desc = i2(y.pgp_desc);
    p.pg_cont = f(y.pg_cont);
    p.pg_cont_ml = f2(y.pg_cont_ml);
    // Maps with the boxes of the prefix kernel (a page, 128 tokens at most) and
    // of the paged kernel (a page's part of a slice).
    Maps maps{};
    const int slice = std::min(block_size, y.pg_rows == 16 ? 16 : 32);
    auto map = [&](CUtensorMap* m, const void* base, int box) {
        return thd::make_paged_map(m, base, num_blocks, block_size, Hkv, D, block_stride, token_stride, head_stride, box);
    };
    if (any_keys && (!map(&maps.pg_k, k_cache, slice) || !map(&maps.pg_v, v_cache, slice)))
        return THD_ERR_INVALID_ARG;
    if (any_keys && p.pre_lanes > 0 &&
        (!map(&maps.pre_k, k_cache, p.box_rows) || !map(&maps.pre_v, v_cache, p.box_rows)))
        return THD_ERR_INVALID_ARG;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    switch (D) {
        case 64: return launch_all<64>(p, maps, any_keys, stream);
        case 128: return launch_all<128>(p, maps, any_keys, stream);
        default: return launch_all<256>(p, maps, any_keys, stream);
    }
}

extern "C" int thd_attn_shared_prefix_get_error(void* stream_ptr) {
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream_ptr)) != cudaSuccess) return THD_ERR_CUDA;
    int s = 0;
    if (cudaMemcpyFromSymbol(&s, g_sp_status, sizeof(int)) != cudaSuccess) return THD_ERR_CUDA;
    const int zero = 0;
    if (s != 0 && cudaMemcpyToSymbol(g_sp_status, &zero, sizeof(int)) != cudaSuccess) return THD_ERR_CUDA;
    return s;
}
