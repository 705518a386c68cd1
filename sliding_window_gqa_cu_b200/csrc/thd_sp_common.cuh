// What the kernels of thd_attn_shared_prefix share: the parameters, the split
// of the work over the grid, and the layout of partial results.
//
// Rows.  The query rows of one kv head are numbered r = token * G + g (token
// over the whole batch, g the query head inside the group), so a request has
// RB = n_q * G consecutive rows and a tile of rows may cut anywhere.
//
// Work.  A unit is one tile of keys of one item (a row tile of one kv head).
// A kernel's units are numbered item by item and cut into as many equal
// consecutive ranges as it has lanes (a CTA, or a group of CTAs in step), so
// every lane gets the same number whatever the lengths.  An item counts a few
// units more, before its keys, for what it costs to start and end it.  What a lane does of
// one item is a piece.  Its unnormalised output, running maximum (in units of
// log2) and sum go to the item's home place if the piece holds the item's first
// tile, else to the CTA's own place (only a lane's first piece can begin inside
// an item); the merge kernel adds them up in a fixed order.
//
// A partial tile is stored as [D / 4][rows][4] fp32 with (maximum, sum) per row
// beside it: threads that hold neighbouring rows then write, and the merge kernel
// reads, whole lines.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sp_lanes.h"

namespace thd {

constexpr int kSpLanes = 148;  // CTAs of the prefix kernel (one per SM)
// What starting and ending an item costs, in units: key tiles of the prefix
// kernel, slices of the paged kernel.
constexpr int kItemTiles = 4;
constexpr int kItemUnits = 1;

// What the kernels derived from the lengths, for the merge kernel.
struct SpPlan {
    long long pg_units;
    int pg_lanes;
    int pre_tiles;  // key tiles (paged kernel: slices) of the prefix
    int pre_lanes;
};

struct SpParams {
    const __nv_bfloat16* q;
    const __nv_bfloat16* kc;
    const __nv_bfloat16* vc;
    int64_t block_stride, token_stride, head_stride;  // of the caches, in elements
    const int32_t* prefix_table;
    const int32_t* prefix_len;
    const int32_t* tables;
    const int32_t* kv_lens;
    const float* sinks;
    __nv_bfloat16* out;
    float* lse;
    int num_blocks, block, block_shift, prefix_blocks, max_blocks;
    int n_req, n_q, Hq, Hkv, G, window;
    float scale_log2;
    int any_keys;  // there are blocks and tables
    int RB;        // rows of a request and kv head
    int rows;      // rows of a kv head
    int box_rows;  // tokens of one TMA box of the prefix kernel
    int places, place_block, place_head;  // extent and steps of its map's place coordinate
    // prefix kernel
    int pre_groups;  // row groups of a kv head
    int pre_width;   // CTAs of a lane (row groups in step)
    int pre_lanes;
    float* pre_home;
    float2* pre_home_ml;
    float* pre_cont;
    float2* pre_cont_ml;
    // paged kernel
    int pg_rows;        // rows of its row tile
    int pg_units;       // row tiles of a request
    int pg_prefix;      // row tiles of the prefix that it takes (0: none)
    int pg_ctas;
    int pg_slice;       // keys of a slice (16 or 32)
    float* own_home;
    float2* own_home_ml;
    long long* own_desc;  // first unit of an item
    float* pgp_home;
    float2* pgp_home_ml;
    long long* pgp_desc;
    float* pg_cont;
    float2* pg_cont_ml;
    SpPlan* plan;
};

// 16 bytes into shared memory, zeros if !there.
__device__ __forceinline__ void load16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// Lanes that the prefix kernel's units are cut over at most: three units each (a part costs
// the traffic of two to four tiles).
__device__ __forceinline__ int sp_prefix_lanes(const SpParams& p, long long units) {
    return static_cast<int>(min((units + 2) / 3, static_cast<long long>(p.pre_lanes)));
}

__device__ __forceinline__ int sp_prefix_len(const SpParams& p) {
    if (p.prefix_len == nullptr) return 0;
    return min(max(*p.prefix_len, 0), p.prefix_blocks * p.block);
}

// Own tokens of request b (what its table holds at most); negative: vacant.
__device__ __forceinline__ int sp_own_len(const SpParams& p, int b) {
    return min(p.kv_lens[b], p.max_blocks * p.block);
}

// First key of the sequence [prefix; own] that a query at position pos sees.
__device__ __forceinline__ int sp_first_key(const SpParams& p, int pos) {
    return p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
}

// First own key that some query of a request of n own tokens sees (the
// windows of its consecutive queries overlap, so all keys behind it are seen).
__device__ __forceinline__ int sp_first_own(const SpParams& p, int n) {
    const int t = n - p.n_q + 1;
    return p.window > 0 && t > p.window ? t - p.window : 0;
}

// Slices of KS own keys that the queries of a request of n own tokens see.
template <int KS>
__device__ __forceinline__ int sp_own_slices(const SpParams& p, int n) {
    return n > 0 ? (n - 1) / KS + 1 - sp_first_own(p, n) / KS : 0;
}

__device__ __forceinline__ int sp_own_slices(const SpParams& p, int n) {
    return p.pg_slice == 32 ? sp_own_slices<32>(p, n) : sp_own_slices<16>(p, n);
}

// What the paged kernel spends on a request of n own tokens, in keys of a kv head and
// row tile that an SM reads meanwhile.  Starting and ending an item is latency that
// other items hide once there is enough to read: an item of one key takes as long as
// 64 keys of a long one, from some 100 keys on there is nothing to see of it.  Counting
// keys alone gave the first tokens after a long prefix a few SMs, as if they cost
// nothing: one token a request, 8 kv heads of 128, 64 requests after 4,096 tokens
// 135 us against 37, 256 after 16,384 268 against 182.
__device__ __forceinline__ float sp_own_cost(const SpParams& p, int n) {
    if (n <= 0) return 0.0f;
    const float sliced = static_cast<float>(sp_own_slices(p, n)) * p.pg_slice;
    return fmaxf(static_cast<float>(n - sp_first_own(p, n)), 48.0f + 0.5f * sliced);
}

// Units of the prefix kernel for n_tiles key tiles.
__device__ __forceinline__ long long sp_prefix_units(const SpParams& p, int n_tiles) {
    if (n_tiles <= 0) return 0;
    return static_cast<long long>((p.pre_groups + p.pre_width - 1) / p.pre_width) * p.Hkv * (n_tiles + kItemTiles);
}

struct SpSplit {
    int lanes;  // of the prefix kernel that work
    int free;   // SMs that it leaves to the paged kernel
};

// How the two kernels share the SMs: the prefix kernel is bound by its chain of
// products and softmax, the paged kernel by memory, which half of the SMs can
// keep busy, so both run side by side and the choice that ends the later one
// soonest is taken.  The prefix takes kStart + tile * units / lanes; the requests'
// own keys kStartPaged + their cost (sp_own_cost) at an SM's rate each, kMemRate at
// most (ns, and bytes a ns, as measured; row tiles of 32 and more are bound by their
// products, about 0.57 TFLOP/s an SM, and read an item's keys once each).  Every
// thread has its own candidates; the best of the warp wins.  64 requests on 8,191
// tokens 92 us one after the other, 75 side by side, 256 on 32,768 474 and 400 (both
// before the power cap, under which the latter is 462); both kernels' CTAs on
// the same SM 96 and 638 (the softmax warps lose more by waiting for issue slots and
// loads than memory gains).  One rate for all row tiles: 64 requests of 16 rows,
// 32,000 + 50..200 tokens, 272 against 165; one of 64 rows, 65,536 + 2,048, 446
// against 96.  With few SMs for the own pages they read, at D = 64, 128 and 256, 61 to
// 66, 73 to 92 and 59 to 77 bytes a ns each (8 rows), 54, 38 to 42 and 31 to 37 (16
// rows); a tile takes 1,850, 2,130 and 1,800 to 2,100 ns.  44 at D = 256 is between that
// and 50, where requests of 200 tokens got too few SMs (256 on 65,536: 490 us, with 44
// 268); 36 would be as fast there and costs the prefix with a window 2 us in 56.
template <int D>
__device__ __forceinline__ SpSplit sp_split(const SpParams& p, long long units, float own_cost) {
    constexpr float kMemRate = 6000.0f, kStart = 10000.0f, kStartPaged = 12000.0f;
    constexpr float kSmRate = D == 64 ? 60.0f : 76.0f, kSmRows = 570.0f;
    constexpr float kSmRate16 = D == 64 ? 55.0f : D == 128 ? 50.0f : 44.0f;
    constexpr float kTile = D == 64 ? 1600.0f : 2300.0f;
    const float bytes = own_cost * p.Hkv * p.pg_units * (D * 4);
    const float sm_rate = p.pg_rows <= 8 ? kSmRate : p.pg_rows <= 16 ? kSmRate16 : kSmRows / p.pg_rows;
    const int most = units > 0 ? sp_prefix_lanes(p, units) : 0;
    float best = INFINITY;
    int lanes = most;
    for (int l = 1 + static_cast<int>(threadIdx.x & 31); l <= most; l += 32) {
        const float prefix = kStart + kTile * (static_cast<float>(units) / l);
        const float rate = fminf(kMemRate, (kSpLanes - l * p.pre_width) * sm_rate);
        const float time = bytes > 0.0f ? fmaxf(prefix, kStartPaged + bytes / rate) : prefix;
        if (time <= best) {
            best = time;
            lanes = l;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, best, o);
        const int l = __shfl_xor_sync(0xffffffffu, lanes, o);
        if (other < best || (other == best && l > lanes)) {
            best = other;
            lanes = l;
        }
    }
    return SpSplit{lanes, kSpLanes - lanes * p.pre_width};
}

}  // namespace thd
