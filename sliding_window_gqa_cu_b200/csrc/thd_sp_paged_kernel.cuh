// Each request's own pages (and a prefix that few rows share): few query rows
// against many keys, so every K and V element is used once per pass and the
// kernel is bound by reading them.
//
// A CTA takes row tiles of 16 WR rows.  The products are mma.sync m16n8k16 on
// purpose: a tile of 64 keys x D = 128 x 16 rows takes some 64 instructions per
// warp, far less than the 32 KB it reads take to arrive, and the scores stay in
// registers (a tcgen05 tile would be 128 rows high, 1/8 to 1/16 used, and send
// the scores through TMEM).
//
// Work split: (request, kv head, row tile) items, a unit is a tile of KT keys;
// all units of the batch are numbered and cut into equal ranges, one per CTA, so
// long and short requests balance whatever the lengths.
//
// Four warps, WR row groups x WK key groups x WC column groups of the output.
// Every key group walks its own slices of the tiles through its own ring of
// slots (a K or V slice each); its first warp issues the TMA loads, the next
// slice into a slot as soon as the slot has been read.  For 16 rows a key group
// is one warp, so warps never wait for each other inside a piece and nearly the
// whole ring (48 KB per CTA, three CTAs per SM or one beside the prefix kernel)
// is in flight at any time.
#pragma once

#include "thd_attn_kernel.cuh"
#include "thd_sp_common.cuh"

namespace thd {

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// c += A B for 16 x 8 x 16, bf16 in, fp32 accumulate.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D_, int WR_>
struct PagedConfig {
    static constexpr int D = D_;
    static constexpr int WR = WR_;                  // 16-row groups of a row tile
    static constexpr int WC = D == 256 ? 2 : 1;     // column groups of the output
    static constexpr int WK = 4 / (WR * WC);        // key groups
    static constexpr int KS = WR == 1 ? 16 : 32;    // keys of a slice
    static constexpr int KT = KS * WK;              // keys of a tile
    static constexpr int GROUP = WR * WC;           // warps of a key group
    static constexpr int ROWS = 16 * WR;
    static constexpr int DW = D / WC;               // output columns of a warp
    static constexpr int CHUNK_BYTES = KS * 128;
    static constexpr int SLOT_BYTES = KS * D * 2;
    static constexpr int RING_BYTES = D == 256 ? 65536 : 49152;
    static constexpr int NSLOT = RING_BYTES / WK / SLOT_BYTES;  // of a key group
    static constexpr int THREADS = 128;
    // CTAs on an SM: 128 registers a thread, so that one CTA also fits beside
    // the prefix kernel (12 warp places of 128 registers).
    static constexpr int RESIDENT = 4;

    static constexpr int Q_BYTES = ROWS * D * 2;
    // The key groups' results are added through shared memory CB columns at a
    // time, over the Q rows (no longer needed then).
    static constexpr int CB = DW < 128 / WR / WC ? DW : 128 / WR / WC;
    static constexpr int COMB_BYTES = WK > 1 ? ROWS * WC * CB * 4 : 0;
    static constexpr int SMEM_Q = RING_BYTES;
    static constexpr int SMEM_ML = SMEM_Q + (Q_BYTES > COMB_BYTES ? Q_BYTES : COMB_BYTES);  // float2 [WK][ROWS]
    static constexpr int SMEM_BAR = SMEM_ML + WK * ROWS * 8;
    static constexpr int B_FULL = 0, B_EMPTY = WK * NSLOT, B_TEAM = 2 * WK * NSLOT, NUM_BARS = B_TEAM + 1;
    static constexpr int SMEM_START = SMEM_BAR + NUM_BARS * 8;  // int64 [8]
    static constexpr int SMEM_MASK = SMEM_START + 64;           // uint32 [WK][NSLOT]: 16-key parts in pages of the cache
    static constexpr int SMEM_ABORT = SMEM_MASK + WK * NSLOT * 4;
    static constexpr int SMEM_BYTES = SMEM_ABORT + 4;
    static_assert(WK >= 1 && NSLOT >= 3, "K and V of a slice and the next K");
};

struct PagedPiece {
    const int32_t* table;
    int table_len;
    int kt, n;           // first tile of the sequence and how many
    int base;            // position of the sequence's key 0
    int first, end;      // keys that some row sees: [first, end)
    int row0, rows;      // rows of the tile
    int h;
    bool home;
    int last_cta;        // (home pieces) the CTA that ends the item
    float* part;         // [D / 4][part_rows][4]
    float2* ml;
    int2* desc;
    int part_rows;
};

template <class C>
struct PagedWalk {
    long long x, x1, units, pre_units;
    long long rem;       // unit inside request b's own units
    int b, lanes;
    int P, pre_first_tile, pre_tiles, pre_first;
    int cache_b, cache_n;  // own lengths of requests [cache_b, cache_b + 32), one per thread

    __device__ __forceinline__ bool next(const SpParams& p, PagedPiece& pc) {
        if (x >= x1) return false;
        long long item_begin;
        int at, tiles;
        if (x < pre_units) {
            const int item = static_cast<int>(x / pre_tiles);
            item_begin = static_cast<long long>(item) * pre_tiles;
            at = static_cast<int>(x - item_begin);
            tiles = pre_tiles;
            const int rt = item / p.Hkv;
            pc.h = item - rt * p.Hkv;
            pc.table = p.prefix_table;
            pc.table_len = p.prefix_blocks;
            pc.base = 0;
            pc.first = pre_first;
            pc.end = P;
            pc.row0 = rt * C::ROWS;
            pc.rows = min(C::ROWS, p.rows - pc.row0);
            pc.kt = pre_first_tile + at;
            pc.part = p.pgp_home + static_cast<int64_t>(item) * (C::ROWS * C::D);
            pc.ml = p.pgp_home_ml + static_cast<int64_t>(item) * C::ROWS;
            pc.part_rows = C::ROWS;
            pc.desc = p.pgp_desc + item;
        } else {
            const int lane = threadIdx.x & 31;
            const int per = p.pg_units * p.Hkv;
            int n, t;
            while (true) {  // the next request with keys
                if (b < cache_b || b >= cache_b + 32) {
                    cache_b = b;
                    cache_n = b + lane < p.n_req ? sp_own_len(p, b + lane) : -1;
                }
                const uint32_t live = __ballot_sync(0xffffffffu, cache_n > 0 && cache_b + lane >= b);
                if (live == 0) {
                    if (cache_b + 32 >= p.n_req) return false;
                    b = cache_b + 32;
                    continue;
                }
                b = cache_b + __ffs(live) - 1;
                n = __shfl_sync(0xffffffffu, cache_n, b - cache_b);
                t = sp_own_tiles<C::KT>(p, n);
                if (rem < static_cast<long long>(t) * per) break;
                rem -= static_cast<long long>(t) * per;
                ++b;
            }
            tiles = t;
            const int hu = static_cast<int>(rem / tiles);
            at = static_cast<int>(rem - static_cast<long long>(hu) * tiles);
            item_begin = x - at;
            pc.h = hu / p.pg_units;
            const int u = hu - pc.h * p.pg_units;
            pc.table = p.tables + static_cast<int64_t>(b) * p.max_blocks;
            pc.table_len = p.max_blocks;
            pc.base = P;
            pc.first = sp_first_own(p, n);
            pc.end = n;
            pc.row0 = b * p.RB + u * C::ROWS;
            pc.rows = min(C::ROWS, p.RB - u * C::ROWS);
            pc.kt = pc.first / C::KT + at;
            const int64_t bh = static_cast<int64_t>(b) * p.Hkv + pc.h;
            pc.part = p.own_home + bh * p.RB * C::D + u * C::ROWS * 4;
            pc.ml = p.own_home_ml + bh * p.RB + u * C::ROWS;
            pc.part_rows = p.RB;
            pc.desc = p.own_desc + bh * p.pg_units + u;
        }
        pc.n = static_cast<int>(min(static_cast<long long>(tiles - at), x1 - x));
        pc.home = at == 0;
        pc.last_cta = lane_of(units, lanes, item_begin + tiles - 1);
        if (!pc.home) {
            pc.part = p.pg_cont + static_cast<int64_t>(blockIdx.x) * (C::ROWS * C::D);
            pc.ml = p.pg_cont_ml + static_cast<int64_t>(blockIdx.x) * C::ROWS;
            pc.part_rows = C::ROWS;
        }
        if (x >= pre_units) rem += pc.n;
        x += pc.n;
        return true;
    }
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::RESIDENT)
thd_sp_paged_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                    const SpParams p, int* status) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_addr(smem);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    launch_dependents();

    auto bar = [&](int idx) -> uint32_t { return sbase + C::SMEM_BAR + 8u * idx; };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::SMEM_ABORT);
    long long* start = reinterpret_cast<long long*>(smem + C::SMEM_START);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::WK * C::NSLOT; ++s) {
            mbar_init(bar(C::B_FULL + s), 1);
            mbar_init(bar(C::B_EMPTY + s), C::GROUP);
        }
        mbar_init(bar(C::B_TEAM), 4);
        int bad = *reinterpret_cast<volatile int*>(status) != 0 ? 1 : 0;
        if ((sbase & 1023u) != 0) {  // the swizzled tiles need it
            atomicCAS(status, 0, kStatusBadItem);
            bad = 1;
        }
        *abort_flag = bad;
        fence_barrier_init();
    }

    // Own units of the batch: every thread counts the tiles of a run of requests
    // and, where the prefix goes here, its least own length.
    PagedWalk<C> walk;
    {
        const int P = sp_prefix_len(p);
        const int per = (p.n_req + C::THREADS - 1) / C::THREADS;
        const int b0 = min(p.n_req, static_cast<int>(threadIdx.x) * per), b1 = min(p.n_req, b0 + per);
        int least = 0x7fffffff;
        long long tiles = 0;
        for (int b = b0; b < b1; ++b) {
            const int n = sp_own_len(p, b);
            tiles += sp_own_tiles<C::KT>(p, n);
            if (n >= 0) least = min(least, n);
        }
        long long incl = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        least = __reduce_min_sync(0xffffffffu, least);
        // start[0 .. 4]: tiles of the warps; least own lengths in the Q area
        int* least_of = reinterpret_cast<int*>(smem + C::SMEM_Q);
        if (lane == 31) start[warp] = incl;
        if (lane == 0) least_of[warp] = least;
        __syncthreads();
        long long before = 0, total = 0;
        for (int w = 0; w < C::THREADS / 32; ++w) {
            if (w < warp) before += start[w];
            total += start[w];
            least = min(least, least_of[w]);
        }
        __syncthreads();
        const int unit = p.pg_units * p.Hkv;
        const int lo = least == 0x7fffffff ? P : sp_first_key(p, P + least - p.n_q);
        walk.P = P;
        walk.pre_first = lo;
        walk.pre_first_tile = lo / C::KT;
        walk.pre_tiles = lo < P && p.pg_prefix > 0 ? (P - 1) / C::KT + 1 - walk.pre_first_tile : 0;
        walk.pre_units = static_cast<long long>(p.pg_prefix) * p.Hkv * walk.pre_tiles;
        walk.units = walk.pre_units + total * unit;
        walk.lanes = static_cast<int>(min(walk.units, static_cast<long long>(p.pg_ctas)));
        const int c = blockIdx.x;
        walk.x = c < walk.lanes ? lane_begin(walk.units, walk.lanes, c) : 0;
        walk.x1 = c < walk.lanes ? lane_begin(walk.units, walk.lanes, c + 1) : 0;
        walk.cache_b = -64;
        walk.cache_n = -1;
        // Where the range begins among the own units.
        const long long want = max(walk.x, walk.pre_units) - walk.pre_units;
        const long long mine = (before + incl - tiles) * unit;
        if (tiles > 0 && want >= mine && want < mine + tiles * unit) {
            long long at = want - mine;
            int b = b0;
            for (; b < b1; ++b) {
                const long long t = static_cast<long long>(sp_own_tiles<C::KT>(p, sp_own_len(p, b))) * unit;
                if (at < t) break;
                at -= t;
            }
            start[0] = b;
            start[1] = at;
        }
        __syncthreads();
        walk.b = static_cast<int>(start[0]);
        walk.rem = start[1];
        if (total == 0) walk.b = p.n_req;
        if (blockIdx.x == 0 && threadIdx.x == 0 && p.pg_prefix > 0) {
            p.pre_plan[0] = walk.pre_first_tile;
            p.pre_plan[1] = walk.pre_tiles;
        }
    }
    const bool skip = *abort_flag != 0;
    PagedPiece pc;

    const int wr = warp % C::WR, wc = (warp / C::WR) % C::WC, wk = warp / C::GROUP;
    const bool leader = warp % C::GROUP == 0;  // issues the key group's loads
    if (leader && lane == 0) {
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
    }
    {
        const int mi = lane >> 3, m8 = lane & 7;
        const int qr = lane >> 2, qc = (lane & 3) * 2;  // this thread's row (and row + 8) and column pair
        const uint32_t q_s = sbase + C::SMEM_Q;
        float2* ml_s = reinterpret_cast<float2*>(smem + C::SMEM_ML);
        float* comb = reinterpret_cast<float*>(smem + C::SMEM_Q) + (wr * C::WC + wc) * (16 * C::CB);
        const float sl2 = p.scale_log2;
        const uint32_t ring = sbase + wk * (C::NSLOT * C::SLOT_BYTES);
        const int full0 = C::B_FULL + wk * C::NSLOT, empty0 = C::B_EMPTY + wk * C::NSLOT;
        volatile uint32_t* const masks = reinterpret_cast<volatile uint32_t*>(smem + C::SMEM_MASK) + wk * C::NSLOT;
        int pos = 0, issued = 0, team = 0;  // ring positions read and loaded
        bool ok = !skip;
        // All four computing warps (bounded, so that an abort cannot hang it).
        auto team_sync = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_TEAM));
            ok = warp_wait(bar(C::B_TEAM), team & 1, abort_flag, status);
            ++team;
        };
        while (ok && walk.next(p, pc)) {
            if (pc.home && threadIdx.x == 0) *pc.desc = make_int2(blockIdx.x, pc.last_cta);
            const int pos0 = pos;
            // Loads of this key group: position 2 i is K, 2 i + 1 V of its slice i.
            const int end_pos = pos + 2 * pc.n;
            int slice = 0;              // of the next load
            int page0 = 0, page1 = 0;   // thread t: pages of slice (slice & ~31) + t, first and second 16 keys
            auto load_next = [&]() {
                if (!leader || issued >= end_pos) return;
                const int slot = issued % C::NSLOT;
                const bool v = ((issued ^ pos0) & 1) != 0;
                if (C::GROUP > 1 && issued >= C::NSLOT) {
                    ok = warp_wait(bar(empty0 + slot), (issued / C::NSLOT - 1) & 1, abort_flag, status);
                    if (!ok) return;
                }
                if (!v && (slice & 31) == 0) {
                    const int key = (pc.kt + slice + lane) * C::KT + wk * C::KS;
                    auto page_of = [&](int k) -> int {  // one past the cache if there is none
                        const int idx = k >> p.block_shift;
                        int id = -1;
                        if (slice + lane < pc.n && idx < pc.table_len) id = pc.table[idx];
                        return id >= 0 && id < p.num_blocks ? id : p.num_blocks;
                    };
                    page0 = page_of(key);
                    if (C::KS == 32) page1 = p.block == 16 ? page_of(key + 16) : page0;
                }
                const int id0 = __shfl_sync(0xffffffffu, page0, slice & 31);
                const int id1 = C::KS == 32 ? __shfl_sync(0xffffffffu, page1, slice & 31) : id0;
                if (lane == 0) {
                    const int row = ((pc.kt + slice) * C::KT + wk * C::KS) & (p.block - 1);
                    masks[slot] = (id0 < p.num_blocks ? 1u : 0u) | (id1 < p.num_blocks ? 2u : 0u);
                    mbar_arrive_expect_tx(bar(full0 + slot), C::SLOT_BYTES);
                    const uint32_t dst = ring + slot * C::SLOT_BYTES;
                    const CUtensorMap* map = v ? &tmap_v : &tmap_k;
#pragma unroll
                    for (int c = 0; c < C::D / 64; ++c) {
                        tma_load_4d(dst + c * C::CHUNK_BYTES, map, bar(full0 + slot), c * 64, pc.h, row, id0);
                        if (C::KS == 32 && p.block == 16)
                            tma_load_4d(dst + c * C::CHUNK_BYTES + 2048, map, bar(full0 + slot), c * 64, pc.h, row, id1);
                    }
                }
                ++issued;
                if (v) ++slice;
            };
            for (int i = 0; i < C::NSLOT && ok; ++i) load_next();
            if (!ok) break;
            // Q rows into shared memory, 16-byte pieces swizzled by the row.
            {
                constexpr int PER = C::D / 8;
                for (int i = threadIdx.x; i < C::ROWS * PER; i += C::THREADS) {
                    const int rr = i / PER, c = i % PER;
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (rr < pc.rows) {
                        const int r = pc.row0 + rr, t = r / p.G;
                        v = *reinterpret_cast<const uint4*>(
                            p.q + (static_cast<int64_t>(t) * p.Hq + pc.h * p.G + (r - t * p.G)) * C::D + c * 8);
                    }
                    st_shared_v4(q_s + rr * (C::D * 2) + ((c ^ (rr & 7)) << 4), v.x, v.y, v.z, v.w);
                }
            }
            // Keys of the sequence that this thread's two rows see: [lo, hi].
            int lo[2], hi[2];
            bool any = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rr = wr * 16 + qr + 8 * e;
                lo[e] = pc.first;  // (unused rows: all)
                hi[e] = pc.end - 1;
                if (rr < pc.rows) {
                    const int r = pc.row0 + rr, b = r / p.RB;
                    const int n = sp_own_len(p, b);
                    if (n >= 0) {
                        const int at = walk.P + n - p.n_q + (r - b * p.RB) / p.G;
                        lo[e] = max(pc.first, sp_first_key(p, at) - pc.base);
                        hi[e] = min(pc.end - 1, at - pc.base);
                    }
                    any = true;
                }
            }
            const bool rows_here = __any_sync(0xffffffffu, any);
            const int all_lo = __reduce_max_sync(0xffffffffu, max(lo[0], lo[1]));
            const int all_hi = __reduce_min_sync(0xffffffffu, min(hi[0], hi[1]));
            team_sync();
            if (!ok) break;

            float acc[C::DW / 8][4];
#pragma unroll
            for (int i = 0; i < C::DW / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][e] = 0.0f;
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

            for (int j = 0; j < pc.n; ++j) {
                const int ks = pos % C::NSLOT;
                const uint32_t k_s = ring + ks * C::SLOT_BYTES;
                const int key = (pc.kt + j) * C::KT + wk * C::KS;  // first key of the slice
                ok = warp_wait(bar(full0 + ks), (pos / C::NSLOT) & 1, abort_flag, status);
                if (!ok) break;
                const uint32_t parts = masks[ks];  // 16-key parts whose page exists
                uint32_t pa[C::KS / 16][4];
                bool edge = false;
                if (rows_here) {
                    float s[C::KS / 8][4];
#pragma unroll
                    for (int i = 0; i < C::KS / 8; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[i][e] = 0.0f;
                    const uint32_t qa = q_s + (wr * 16 + (mi & 1) * 8 + m8) * (C::D * 2);
                    const uint32_t ka = k_s + ((mi >> 1) * 8 + m8) * 128;
#pragma unroll
                    for (int kk = 0; kk < C::D / 16; ++kk) {
                        uint32_t a[4];
                        ldsm4(qa + (((kk * 2 + (mi >> 1)) ^ m8) << 4), a);
#pragma unroll
                        for (int i = 0; i < C::KS / 16; ++i) {
                            uint32_t b[4];
                            ldsm4(ka + (kk >> 2) * C::CHUNK_BYTES + i * 16 * 128 +
                                      ((((kk & 3) * 2 + (mi & 1)) ^ m8) << 4), b);
                            mma16816(s[2 * i], a, b[0], b[1]);
                            mma16816(s[2 * i + 1], a, b[2], b[3]);
                        }
                    }
                    edge = key < all_lo || key + C::KS - 1 > all_hi || parts != 3u;
                    if (edge) {
#pragma unroll
                        for (int i = 0; i < C::KS / 8; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int at = key + i * 8 + qc + (e & 1);
                                if (at < lo[e >> 1] || at > hi[e >> 1] || !((parts >> (i >> 1)) & 1u)) s[i][e] = -INFINITY;
                            }
                    }
                    // Running maximum and sum of the two rows (a quad holds a row).
                    float alpha[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float t = fmaxf(s[0][2 * e], s[0][2 * e + 1]);
#pragma unroll
                        for (int i = 1; i < C::KS / 8; ++i) t = max3f(t, s[i][2 * e], s[i][2 * e + 1]);
                        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2)) * sl2;
                        const float now = fmaxf(m[e], t);
                        const float neg = now == -INFINITY ? 0.0f : -now;
                        alpha[e] = now == m[e] ? 1.0f : ex2_approx(m[e] - now);
                        m[e] = now;
                        float sum = 0.0f;
#pragma unroll
                        for (int i = 0; i < C::KS / 8; ++i) {
                            const float p0 = ex2_approx(fmaf(s[i][2 * e], sl2, neg));
                            const float p1 = ex2_approx(fmaf(s[i][2 * e + 1], sl2, neg));
                            sum += p0 + p1;
                            pa[i >> 1][(i & 1) * 2 + e] = pack_bf16x2(p0, p1);
                        }
                        l[e] = l[e] * alpha[e] + sum;  // (of this thread's columns)
                    }
                    if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
                        for (int i = 0; i < C::DW / 8; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[i][e] *= alpha[e >> 1];
                    }
                }
                // The K slot has been read: the next load goes there.
                __syncwarp();
                if (C::GROUP > 1 && lane == 0) mbar_arrive(bar(empty0 + ks));
                ++pos;
                load_next();
                if (!ok) break;
                const int vs = pos % C::NSLOT;
                ok = warp_wait(bar(full0 + vs), (pos / C::NSLOT) & 1, abort_flag, status);
                if (!ok) break;
                if (rows_here) {
                    const uint32_t va = ring + vs * C::SLOT_BYTES + ((mi & 1) * 8 + m8) * 128 +
                                        wc * (C::DW / 64) * C::CHUNK_BYTES;
#pragma unroll
                    for (int i = 0; i < C::KS / 16; ++i) {
                        // Keys that no row sees may hold anything, and 0 * NaN would stay NaN.
                        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
                        if (edge) {
                            const int at = key + i * 16 + qc;
                            auto seen = [&](int k) { return k >= pc.first && k < pc.end; };
                            keep0 = (seen(at) ? 0xffffu : 0u) | (seen(at + 1) ? 0xffff0000u : 0u);
                            keep1 = (seen(at + 8) ? 0xffffu : 0u) | (seen(at + 9) ? 0xffff0000u : 0u);
                        }
#pragma unroll
                        for (int d = 0; d < C::DW / 16; ++d) {
                            uint32_t b[4];
                            ldsm4_trans(va + (d >> 2) * C::CHUNK_BYTES + i * 16 * 128 +
                                            ((((d & 3) * 2 + (mi >> 1)) ^ m8) << 4), b);
                            b[0] &= keep0;
                            b[1] &= keep1;
                            b[2] &= keep0;
                            b[3] &= keep1;
                            mma16816(acc[2 * d], pa[i], b[0], b[1]);
                            mma16816(acc[2 * d + 1], pa[i], b[2], b[3]);
                        }
                    }
                }
                __syncwarp();
                if (C::GROUP > 1 && lane == 0) mbar_arrive(bar(empty0 + vs));
                ++pos;
                load_next();
                if (!ok) break;
            }
            if (!ok) break;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            }
            if constexpr (C::WK > 1) {
                // Bring the key groups to one maximum and add them up, the last first.
                if (wc == 0 && (lane & 3) == 0)
#pragma unroll
                    for (int e = 0; e < 2; ++e) ml_s[wk * C::ROWS + wr * 16 + qr + 8 * e] = make_float2(m[e], l[e]);
                team_sync();
                if (!ok) break;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = -INFINITY;
#pragma unroll
                    for (int g = 0; g < C::WK; ++g) top = fmaxf(top, ml_s[g * C::ROWS + wr * 16 + qr + 8 * e].x);
                    float sum = 0.0f;
#pragma unroll
                    for (int g = 0; g < C::WK; ++g) {
                        const float2 v = ml_s[g * C::ROWS + wr * 16 + qr + 8 * e];
                        sum += v.x == -INFINITY ? 0.0f : v.y * ex2_approx(v.x - top);
                    }
                    const float a = m[e] == -INFINITY ? 0.0f : ex2_approx(m[e] - top);
#pragma unroll
                    for (int i = 0; i < C::DW / 8; ++i) {
                        acc[i][2 * e] *= a;
                        acc[i][2 * e + 1] *= a;
                    }
                    m[e] = top;
                    l[e] = sum;
                }
#pragma unroll
                for (int c0 = 0; c0 < C::DW; c0 += C::CB) {
#pragma unroll
                    for (int g = C::WK - 1; g >= 0; --g) {
                        if (wk == g) {
#pragma unroll
                            for (int i = 0; i < C::CB / 8; ++i) {
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    // [CB / 4][16][4] fp32
                                    float2* at = reinterpret_cast<float2*>(
                                        comb + ((i * 2 + (qc >> 2)) * 16 + qr + 8 * e) * 4 + (qc & 3));
                                    float* mine = &acc[c0 / 8 + i][2 * e];
                                    if (g < C::WK - 1) {
                                        const float2 o = *at;
                                        mine[0] += o.x;
                                        mine[1] += o.y;
                                    }
                                    if (g > 0) *at = make_float2(mine[0], mine[1]);
                                }
                            }
                        }
                        team_sync();
                        if (!ok) break;
                    }
                    if (!ok) break;
                }
                if (!ok) break;
            }
            if (wk == 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int rr = wr * 16 + qr + 8 * e;
                    if (rr < pc.rows) {
#pragma unroll
                        for (int i = 0; i < C::DW / 8; ++i) {
                            const int col = wc * C::DW + i * 8 + qc;
                            *reinterpret_cast<float2*>(pc.part + (static_cast<int64_t>(col >> 2) * pc.part_rows + rr) * 4 +
                                                       (col & 3)) = make_float2(acc[i][2 * e], acc[i][2 * e + 1]);
                        }
                        if (wc == 0 && (lane & 3) == 0) pc.ml[rr] = make_float2(m[e], l[e]);
                    }
                }
            }
            if constexpr (C::WK == 1) team_sync();  // Q may be overwritten
        }
        // After an abort let the loads in flight land before the CTA ends.
        if (!ok && leader && lane == 0)
            for (int i = pos; i < issued; ++i) drain_wait(bar(full0 + i % C::NSLOT), (i / C::NSLOT) & 1);
    }

    __syncthreads();
    // The prefix kernel before this grid may still run: one CTA stays until it
    // has ended, so that this grid's end means both.
    if (blockIdx.x == 0) wait_for_previous_grid();
}

}  // namespace thd
