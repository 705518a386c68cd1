// Attention of a step's new tokens over a shared prefix and each request's
// own pages of a paged cache (thd_attn_shared_prefix).  The pages print no
// serving form of MuseMagiPlan.attention / FlintMagiPlan.attention
// ("muse_spark.magi_cp", "flint.magi"): masks, GQA mapping, sinks and the
// log-sum-exp are those of the packed forward, over the sequence [prefix; own]
// of every request.
//
// One warp per (token, query head): a lane holds D / 32 columns; the keys are
// taken one by one with a running maximum and sum in fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/thd_attn.h"
#include "tma_map.h"

namespace {

struct SpParams {
    const __nv_bfloat16* q;
    const __nv_bfloat16* kc;
    const __nv_bfloat16* vc;
    const int32_t* prefix_table;
    const int32_t* prefix_len;
    const int32_t* tables;
    const int32_t* kv_lens;
    const float* sinks;
    __nv_bfloat16* out;
    float* lse;
    int64_t num_blocks, block_stride, token_stride, head_stride;
    int block, prefix_blocks, max_blocks, n_req, n_q, Hq, G, window;
    float scale_log2;
};

template <int D>
__global__ void __launch_bounds__(256) thd_attn_shared_prefix_kernel(const SpParams p) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (row >= static_cast<int64_t>(p.n_req) * p.n_q * p.Hq) return;
    const int h = static_cast<int>(row % p.Hq);
    const int64_t tok = row / p.Hq;
    const int b = static_cast<int>(tok / p.n_q), i = static_cast<int>(tok % p.n_q);
    if (p.kv_lens[b] < 0) return;
    const int P = p.prefix_len ? min(max(*p.prefix_len, 0), p.prefix_blocks * p.block) : 0;
    const int n = min(p.kv_lens[b], p.max_blocks * p.block);
    const int pos = P + n - p.n_q + i;
    const int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    float q[E], acc[E];
    const __nv_bfloat16* qrow = p.q + row * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = __bfloat162float(qrow[e]) * p.scale_log2;
        acc[e] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    if (p.sinks) {
        m = p.sinks[h] * 1.4426950408889634f;
        l = m == -INFINITY ? 0.0f : 1.0f;
    }
    for (int j = lo; j <= pos; ++j) {
        const int32_t page = j < P ? p.prefix_table[j / p.block]
                                   : p.tables[static_cast<int64_t>(b) * p.max_blocks + (j - P) / p.block];
        if (page < 0 || page >= p.num_blocks) continue;
        const int in_page = (j < P ? j : j - P) % p.block;
        const int64_t at = page * p.block_stride + in_page * p.token_stride + (h / p.G) * p.head_stride + lane * E;
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], __bfloat162float(p.kc[at + e]), s);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (s > m) {
            const float a = exp2f(m - s);
            l *= a;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] *= a;
            m = s;
        }
        const float w = exp2f(s - m);
        l += w;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(w, __bfloat162float(p.vc[at + e]), acc[e]);
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) p.out[row * D + lane * E + e] = __float2bfloat16_rn(acc[e] * inv);
    if (p.lse && lane == 0) p.lse[row] = l > 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

constexpr int kMaxUnits = 4096;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

extern "C" size_t thd_attn_shared_prefix_workspace_bytes(int n_req, int n_q, int Hq, int Hkv, int D) {
    if (n_req <= 0 || n_q <= 0 || Hkv <= 0 || Hq <= 0 || Hq % Hkv != 0 || D <= 0) return 0;
    return 16;
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
    SpParams p{static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k_cache),
               static_cast<const __nv_bfloat16*>(v_cache), prefix_table_or_null, prefix_len_or_null,
               block_tables, kv_lens, sinks_or_null, static_cast<__nv_bfloat16*>(out), lse,
               num_blocks, block_stride, token_stride, head_stride, block_size, prefix_blocks, max_blocks,
               n_req, n_q, Hq, G, window, scale * 1.4426950408889634f};
    const int64_t rows = static_cast<int64_t>(n_req) * n_q * Hq;
    const unsigned grid = static_cast<unsigned>((rows + 7) / 8);
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    switch (D) {
        case 64: thd_attn_shared_prefix_kernel<64><<<grid, 256, 0, stream>>>(p); break;
        case 128: thd_attn_shared_prefix_kernel<128><<<grid, 256, 0, stream>>>(p); break;
        default: thd_attn_shared_prefix_kernel<256><<<grid, 256, 0, stream>>>(p); break;
    }
    return cudaGetLastError() == cudaSuccess ? THD_OK : THD_ERR_CUDA;
}

extern "C" int thd_attn_shared_prefix_get_error(void* stream_ptr) {
    return cudaStreamSynchronize(static_cast<cudaStream_t>(stream_ptr)) == cudaSuccess ? THD_OK : THD_ERR_CUDA;
}
