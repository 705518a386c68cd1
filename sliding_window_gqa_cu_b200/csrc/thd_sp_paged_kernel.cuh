// Each request's own pages (and a prefix that few rows share): few query rows
// against many keys, so every K and V element is used once per pass and the
// kernel is bound by reading them.
//
// The products are mma.sync m16n8k16 with the keys as the 16 rows and 8 query
// rows as the 8 columns: S^T = K Q^T and O^T = V^T P^T, so that 8 query rows (a
// group of 8 heads) leave no lane of the product idle, Q^T, the scores and O^T
// stay in registers, and 32 keys of head dim 128 take some 250 instructions per
// warp while their 16 KB take longer to arrive.  With 8 query rows a tcgen05 tile
// would send the scores through TMEM for products that are not what bounds this; from
// 32 rows on, with the keys as its 128 rows and the query rows as its columns, it would
// be full, and these tiles are bound by mma.sync (below): not built.
//
// P goes into its product as a bf16 number and a second one for what that rounding
// lost (2^-17 is left): up to 16 rows the products are not what bounds the kernel, and a
// single rounding would add as much error as that of the output.  Row tiles of 32 and 64
// pay for it (three products a slice instead of two) and keep it for that error's sake.
//
// A worker is WR warps of 8 NR rows each, which share a ring of slots (a K or V
// slice of KS keys each) and refill a slot as soon as it has been read.  Workers
// never wait for each other.  16 KB a warp, 64 KB a CTA are in flight, three
// CTAs on an SM.  The loads are cp.async: a page
// of 16 tokens is too small a box for TMA, which took 75 to 85 ns per box and SM
// here (24 to 27 GB/s of the SM's share of 44).
//
// Without a prefix, 16 requests of 4,096 tokens, 8 kv heads of 128: 60 us for 4 or 8
// rows a request, 65 for 16 (4.5 and 4.1 TB/s); 32 rows are bound by the products, 118
// us, 64 rows 214 (72 and 80 TFLOP/s).
//
// Work split: (request, kv head, row tile) items; a unit is a slice, and an item
// counts kItemUnits more for its start and end.  The units of the batch are cut
// into equal ranges, one per worker, so long and short requests balance
// whatever the lengths.
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

// The same for data that is read once: L2 gives it up first, before the prefix's
// keys and the parts that the merge kernel reads.
__device__ __forceinline__ uint64_t read_once_policy() {
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    return policy;
}
__device__ __forceinline__ void load16_once(uint32_t dst, const void* src, bool there, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::128B [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src),
                 "r"(there ? 16 : 0), "l"(policy) : "memory");
}

// Arrives on the barrier when this thread's loads so far have landed.
__device__ __forceinline__ void loads_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Transposes the 8 x 8 matrix of 16-bit elements that the warp holds.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// What the packed bf16 pair lost of p0 (low half) and p1, as a bf16 pair.
__device__ __forceinline__ uint32_t rounding_error(uint32_t packed, float p0, float p1) {
    return pack_bf16x2(p0 - __uint_as_float(packed << 16), p1 - __uint_as_float(packed & 0xffff0000u));
}

// c += A B for 16 x 8 x 16, bf16 in, fp32 accumulate.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D_, int NR_, int WR_>
struct PagedConfig {
    static constexpr int D = D_;
    static constexpr int NR = NR_;                      // 8-row groups of a warp
    static constexpr int WR = WR_;                      // warps of a worker
    static constexpr int WORKERS = 4 / WR;              // of a CTA
    static constexpr int ROWS = 8 * NR * WR;            // rows of a row tile
    static constexpr int KS = D * NR <= 128 ? 32 : 16;  // keys of a slice (what the registers hold)
    static constexpr int ROW_BYTES = D * 2;
    static constexpr int SLOT_BYTES = KS * D * 2;
    static constexpr int RING_BYTES = 65536;
    static constexpr int NSLOT = RING_BYTES / 4 * WR / SLOT_BYTES;
    static constexpr int THREADS = 128;
    static constexpr int RESIDENT = 3;  // CTAs on an SM

    static constexpr int SMEM_BAR = RING_BYTES;
    static constexpr int B_FULL = 0, B_EMPTY = WORKERS * NSLOT, NUM_BARS = 2 * WORKERS * NSLOT;
    static constexpr int SMEM_START = SMEM_BAR + NUM_BARS * 8;  // int64 [16]
    static constexpr int SMEM_ABORT = SMEM_START + 128;
    static constexpr int SMEM_BYTES = SMEM_ABORT + 4;
    static_assert(NSLOT >= 2, "K and V of a slice");
};

struct PagedPiece {
    const int32_t* table;
    int table_len;
    int slice, n;        // first slice of the sequence and how many
    int base;            // position of the sequence's key 0
    int first, end;      // keys that some row sees: [first, end)
    int row0, rows;      // rows of the tile
    int h;
    float* part;         // [D / 4][part_rows][4]
    float2* ml;
    int part_rows;
};

template <class C>
struct PagedWalk {
    long long x, x1, pre_units;
    long long rem;       // unit inside request b's own units
    int b, worker;
    int P, pre_first_slice, pre_slices, pre_first;
    int cache_b, cache_n;  // own lengths of requests [cache_b, cache_b + 32), one per thread

    __device__ __forceinline__ bool next(const SpParams& p, PagedPiece& pc) {
        while (x < x1) {
            long long item_begin;
            long long* desc;
            int at, slices;
            if (x < pre_units) {
                const int item = static_cast<int>(x <= 0x7fffffff ? static_cast<int>(x) / (pre_slices + kItemUnits)
                                                                   : x / (pre_slices + kItemUnits));
                item_begin = static_cast<long long>(item) * (pre_slices + kItemUnits);
                at = static_cast<int>(x - item_begin);
                slices = pre_slices;
                const int rt = item / p.Hkv;
                pc.h = item - rt * p.Hkv;
                pc.table = p.prefix_table;
                pc.table_len = p.prefix_blocks;
                pc.base = 0;
                pc.first = pre_first;
                pc.end = P;
                pc.row0 = rt * C::ROWS;
                pc.rows = min(C::ROWS, p.rows - pc.row0);
                pc.slice = pre_first_slice;
                pc.part = p.pgp_home + static_cast<int64_t>(item) * (C::ROWS * C::D);
                pc.ml = p.pgp_home_ml + static_cast<int64_t>(item) * C::ROWS;
                pc.part_rows = C::ROWS;
                desc = p.pgp_desc + item;
            } else {
                const int lane = threadIdx.x & 31;
                const int per = p.pg_units * p.Hkv;
                int n;
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
                    slices = sp_own_slices<C::KS>(p, n);
                    const long long mine = static_cast<long long>(slices + kItemUnits) * per;
                    if (rem < mine) break;
                    rem -= mine;
                    ++b;
                }
                const int len = slices + kItemUnits;
                const int hu = rem <= 0x7fffffff ? static_cast<int>(rem) / len : static_cast<int>(rem / len);
                at = static_cast<int>(rem - static_cast<long long>(hu) * len);
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
                pc.slice = pc.first / C::KS;
                const int64_t bh = static_cast<int64_t>(b) * p.Hkv + pc.h;
                pc.part = p.own_home + bh * p.RB * C::D + u * C::ROWS * 4;
                pc.ml = p.own_home_ml + bh * p.RB + u * C::ROWS;
                pc.part_rows = p.RB;
                desc = p.own_desc + bh * p.pg_units + u;
            }
            const int len = slices + kItemUnits;
            const int cnt = static_cast<int>(min(static_cast<long long>(len - at), x1 - x));
            const int s0 = max(at - kItemUnits, 0), s1 = at + cnt - kItemUnits;
            if (x >= pre_units) rem += cnt;
            x += cnt;
            if (s1 <= s0) continue;  // only the item's start
            pc.slice += s0;
            pc.n = s1 - s0;
            if (s0 > 0) {
                pc.part = p.pg_cont + static_cast<int64_t>(worker) * (C::ROWS * C::D);
                pc.ml = p.pg_cont_ml + static_cast<int64_t>(worker) * C::ROWS;
                pc.part_rows = C::ROWS;
            } else {
                *desc = item_begin;  // (every thread the same)
            }
            return true;
        }
        return false;
    }
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::RESIDENT)
thd_sp_paged_kernel(const SpParams p, int* status) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_addr(smem);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    launch_dependents();

    auto bar = [&](int idx) -> uint32_t { return sbase + C::SMEM_BAR + 8u * idx; };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::SMEM_ABORT);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::WORKERS * C::NSLOT; ++s) {
            mbar_init(bar(C::B_FULL + s), 32 * C::WR);
            mbar_init(bar(C::B_EMPTY + s), C::WR);
        }
        *abort_flag = *reinterpret_cast<volatile int*>(status) != 0 ? 1 : 0;
        fence_barrier_init();
    }

    // Units of the batch: every thread counts the slices of a run of requests
    // and, where the prefix goes here, its least own length.
    PagedWalk<C> walk;
    {
        long long* start = reinterpret_cast<long long*>(smem + C::SMEM_START);  // [4] units, [4] least, [4][2] starts
        const int P = sp_prefix_len(p);
        const int unit = p.pg_units * p.Hkv;
        const int per = (p.n_req + C::THREADS - 1) / C::THREADS;
        const int b0 = min(p.n_req, static_cast<int>(threadIdx.x) * per), b1 = min(p.n_req, b0 + per);
        auto units_of = [&](int n) -> long long {
            return n > 0 ? static_cast<long long>(sp_own_slices<C::KS>(p, n) + kItemUnits) * unit : 0;
        };
        int least = 0x7fffffff, longest = 0;  // own length; slices of an item
        float cost = 0.0f;
        long long mine = 0;
        for (int b = b0; b < b1; ++b) {
            const int n = sp_own_len(p, b);
            mine += units_of(n);
            if (n >= 0) least = min(least, n);
            if (n <= 0) continue;
            longest = max(longest, sp_own_slices<C::KS>(p, n));
            cost += sp_own_cost(p, n);
        }
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        least = __reduce_min_sync(0xffffffffu, least);
        longest = __reduce_max_sync(0xffffffffu, longest);
        float* cost_of = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) cost += __shfl_xor_sync(0xffffffffu, cost, o);
        if (lane == 31) start[warp] = incl;
        if (lane == 0) cost_of[warp] = cost;
        if (lane == 0) start[4 + warp] = static_cast<long long>(longest) << 32 | least;
        __syncthreads();
        long long before = incl - mine, total = 0;
        cost = cost_of[0] + cost_of[1] + cost_of[2] + cost_of[3];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w < warp) before += start[w];
            total += start[w];
            least = min(least, static_cast<int>(start[4 + w] & 0x7fffffff));
            longest = max(longest, static_cast<int>(start[4 + w] >> 32));
        }
        const int lo = least == 0x7fffffff ? P : sp_first_key(p, P + least - p.n_q);
        walk.P = P;
        walk.pre_first = lo;
        walk.pre_first_slice = lo / C::KS;
        walk.pre_slices = lo < P && p.pg_prefix > 0 ? (P - 1) / C::KS + 1 - walk.pre_first_slice : 0;
        walk.pre_units = walk.pre_slices > 0
                             ? static_cast<long long>(p.pg_prefix) * p.Hkv * (walk.pre_slices + kItemUnits) : 0;
        const long long units = walk.pre_units + total;
        // Units that a worker gets at least.  A part more costs its traffic (written
        // and read, 2 ROWS / KS slices' worth) and, for the item with most parts, time in
        // the merge kernel: some 0.15 us a part against 0.7 us a slice here, so the time
        // of u units and longest / u parts is least near the root of longest / 5.
        longest = max(longest, walk.pre_slices);
        const int least_units = max(max(4, 2 * C::ROWS / C::KS), static_cast<int>(sqrtf(0.2f * longest)));
        // One wave of CTAs on the SMs that the prefix kernel leaves.
        int ctas = p.pg_ctas;
        if (p.pre_lanes > 0 && lo < P)
            ctas = min(ctas, C::RESIDENT * max(1, sp_split<C::D>(p, sp_prefix_units(p, (P - 1) / 128 + 1 - lo / 128), cost).free));
        const int lanes = static_cast<int>(min((units + least_units - 1) / least_units,
                                               static_cast<long long>(ctas) * C::WORKERS));
        // Where each worker's range begins among the own units.
#pragma unroll
        for (int i = 0; i < C::WORKERS; ++i) {
            const int w = blockIdx.x * C::WORKERS + i;
            if (w >= lanes) break;
            const long long want = max(lane_begin(units, lanes, w), walk.pre_units) - walk.pre_units;
            if (want >= before && want < before + mine) {
                long long at = want - before;
                int b = b0;
                for (; b < b1; ++b) {
                    const long long t = units_of(sp_own_len(p, b));
                    if (at < t) break;
                    at -= t;
                }
                start[8 + 2 * i] = b;
                start[9 + 2 * i] = at;
            }
        }
        __syncthreads();
        walk.worker = blockIdx.x * C::WORKERS + warp / C::WR;
        walk.x = walk.worker < lanes ? lane_begin(units, lanes, walk.worker) : 0;
        walk.x1 = walk.worker < lanes ? lane_begin(units, lanes, walk.worker + 1) : 0;
        walk.b = total > 0 ? static_cast<int>(start[8 + 2 * (warp / C::WR)]) : p.n_req;
        walk.rem = start[9 + 2 * (warp / C::WR)];
        walk.cache_b = -64;
        walk.cache_n = -1;
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            if (p.pg_prefix > 0) p.plan->pre_tiles = walk.pre_slices;
            p.plan->pg_units = units;
            p.plan->pg_lanes = lanes;
        }
    }

    {
        const int wr = warp % C::WR, wk = warp / C::WR;
        const int mi = lane >> 3, m8 = lane & 7;
        const int r8 = lane >> 2, c2 = (lane & 3) * 2;
        const float sl2 = p.scale_log2;
        constexpr float kTau = 8.0f;  // rescale only when a maximum grows by more than 2^8
        const uint32_t ring = sbase + wk * (C::NSLOT * C::SLOT_BYTES);
        const int full0 = C::B_FULL + wk * C::NSLOT, empty0 = C::B_EMPTY + wk * C::NSLOT;
        const uint64_t once = read_once_policy();
        int pos = 0, issued = 0;  // ring positions read and loaded
        bool ok = *abort_flag == 0;
        PagedPiece pc;
        while (ok && walk.next(p, pc)) {
            const int pos0 = pos;
            // Loads: position 2 i is K, 2 i + 1 V of the piece's slice i.
            const int end_pos = pos + 2 * pc.n;
            int slice = 0;             // of the next load
            int page0 = 0, page1 = 0;  // thread t: pages of slice (slice & ~31) + t, first and second 16 keys
            uint32_t there = 0;        // bit 2 (issued slices) + part: its page exists (the last 16 slices)
            const int64_t head = static_cast<int64_t>(pc.h) * p.head_stride + (lane % (C::D / 8)) * 8;
            auto load_next = [&]() {
                if (issued >= end_pos) return;
                const int slot = issued % C::NSLOT;
                const bool v = ((issued ^ pos0) & 1) != 0;
                if (C::WR > 1 && issued >= C::NSLOT) {
                    ok = warp_wait(bar(empty0 + slot), (issued / C::NSLOT - 1) & 1, abort_flag, status);
                    if (!ok) return;
                }
                if (!v && (slice & 31) == 0) {
                    auto page_of = [&](int k) -> int {  // -1 if there is none
                        const int idx = k >> p.block_shift;
                        int id = -1;
                        if (slice + lane < pc.n && idx < pc.table_len) id = pc.table[idx];
                        return id < p.num_blocks ? id : -1;
                    };
                    const int key = (pc.slice + slice + lane) * C::KS;
                    page0 = page_of(key);
                    if (C::KS == 32) page1 = p.block == 16 ? page_of(key + 16) : page0;
                }
                const int id0 = __shfl_sync(0xffffffffu, page0, slice & 31);
                const int id1 = C::KS == 32 ? __shfl_sync(0xffffffffu, page1, slice & 31) : id0;
                // A warp loads its share of the slice's rows, 16 bytes a thread.
                constexpr int LANES = C::D / 8;               // threads of a row
                constexpr int STEP = 32 / LANES * C::WR;      // rows of the worker at a time
                const int row = lane / LANES + wr * (32 / LANES);
                const int in_page = (((pc.slice + slice) * C::KS) & (p.block - 1)) + row;
                const __nv_bfloat16* cache = v ? p.vc : p.kc;
                const uint32_t dst = ring + slot * C::SLOT_BYTES + row * C::ROW_BYTES;
                const int64_t step = static_cast<int64_t>(STEP) * p.token_stride;
#pragma unroll
                for (int part = 0; part < C::KS / 16; ++part) {
                    const int id = part == 0 ? id0 : id1;
                    const __nv_bfloat16* src = cache;
                    if (id >= 0)
                        src += static_cast<int64_t>(id) * p.block_stride +
                               static_cast<int64_t>(in_page + (part == 1 && p.block != 16 ? 16 : 0)) * p.token_stride + head;
#pragma unroll
                    for (int i = 0; i < 16 / STEP; ++i) {
                        const int rr = part * 16 + i * STEP;  // + row: the row in the slice
                        load16_once(dst + rr * C::ROW_BYTES + (((lane % LANES) ^ ((rr + row) & 7)) << 4),
                                    src + (id >= 0 ? i * step : 0), id >= 0, once);
                    }
                }
                loads_arrive(bar(full0 + slot));
                if (!v) there = there << 2 | (id0 >= 0 ? 1u : 0u) | (id1 >= 0 ? 2u : 0u);
                ++issued;
                if (v) ++slice;
            };
            for (int i = 0; i < C::NSLOT && ok; ++i) load_next();
            if (!ok) break;

            // Q^T as the second operand: columns are this warp's rows.
            uint32_t qf[C::NR][C::D / 16][2];
#pragma unroll
            for (int t = 0; t < C::NR; ++t) {
                const int rr = (wr * C::NR + t) * 8 + r8;
                const bool here = rr < pc.rows;
                const int r = pc.row0 + (here ? rr : 0), tok = r / p.G;
                const uint32_t* src = reinterpret_cast<const uint32_t*>(
                    p.q + (static_cast<int64_t>(tok) * p.Hq + pc.h * p.G + (r - tok * p.G)) * C::D + c2);
#pragma unroll
                for (int kk = 0; kk < C::D / 16; ++kk) {
                    qf[t][kk][0] = here ? src[kk * 8] : 0u;
                    qf[t][kk][1] = here ? src[kk * 8 + 4] : 0u;
                }
            }
            // Keys of the sequence that this thread's rows c2, c2 + 1 of each group see.
            int lo[C::NR][2], hi[C::NR][2];
            int all_lo = 0, all_hi = 0x7fffffff;
#pragma unroll
            for (int t = 0; t < C::NR; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int rr = (wr * C::NR + t) * 8 + c2 + e;
                    lo[t][e] = pc.first;  // (unused rows: all)
                    hi[t][e] = pc.end - 1;
                    if (rr < pc.rows) {
                        const int r = pc.row0 + rr, b = r / p.RB;
                        const int n = sp_own_len(p, b);
                        if (n >= 0) {
                            const int at = walk.P + n - p.n_q + (r - b * p.RB) / p.G;
                            lo[t][e] = max(pc.first, sp_first_key(p, at) - pc.base);
                            hi[t][e] = min(pc.end - 1, at - pc.base);
                        }
                    }
                    all_lo = max(all_lo, lo[t][e]);
                    all_hi = min(all_hi, hi[t][e]);
                }
            all_lo = __reduce_max_sync(0xffffffffu, all_lo);
            all_hi = __reduce_min_sync(0xffffffffu, all_hi);
            const bool rows_here = wr * C::NR * 8 < pc.rows;

            float acc[C::D / 16][C::NR][4];
#pragma unroll
            for (int i = 0; i < C::D / 16; ++i)
#pragma unroll
                for (int t = 0; t < C::NR; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][t][e] = 0.0f;
            float m[C::NR][2], l[C::NR][2];  // maximum of the row; sum of this thread's keys
#pragma unroll
            for (int t = 0; t < C::NR; ++t) {
                m[t][0] = m[t][1] = -INFINITY;
                l[t][0] = l[t][1] = 0.0f;
            }

            for (int j = 0; j < pc.n; ++j) {
                const int ks = pos % C::NSLOT;
                const int key = (pc.slice + j) * C::KS;  // first key of the slice
                ok = warp_wait(bar(full0 + ks), (pos / C::NSLOT) & 1, abort_flag, status);
                if (!ok) break;
                uint32_t pf[C::KS / 16][C::NR][2], pl[C::KS / 16][C::NR][2];  // P^T, its rounding errors
                bool edge = false;
                if (rows_here) {
                    // 16-key parts whose page exists
                    const uint32_t parts = there >> (2 * ((issued - pos - 1) >> 1)) & 3u;
                    float s[C::KS / 16][C::NR][4];
#pragma unroll
                    for (int i = 0; i < C::KS / 16; ++i)
#pragma unroll
                        for (int t = 0; t < C::NR; ++t)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[i][t][e] = 0.0f;
                    const uint32_t ka = ring + ks * C::SLOT_BYTES + ((mi & 1) * 8 + m8) * C::ROW_BYTES;
#pragma unroll
                    for (int kk = 0; kk < C::D / 16; ++kk)
#pragma unroll
                        for (int i = 0; i < C::KS / 16; ++i) {
                            uint32_t a[4];
                            ldsm4(ka + i * 16 * C::ROW_BYTES + (((kk * 2 + (mi >> 1)) ^ m8) << 4), a);
#pragma unroll
                            for (int t = 0; t < C::NR; ++t) mma16816(s[i][t], a, qf[t][kk][0], qf[t][kk][1]);
                        }
                    edge = key < all_lo || key + C::KS - 1 > all_hi || parts != 3u;
                    if (edge) {
#pragma unroll
                        for (int i = 0; i < C::KS / 16; ++i)
#pragma unroll
                            for (int t = 0; t < C::NR; ++t)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const int at = key + i * 16 + r8 + (e >> 1) * 8;
                                    if (at < lo[t][e & 1] || at > hi[t][e & 1] || !((parts >> i) & 1u)) s[i][t][e] = -INFINITY;
                                }
                    }
                    // The maxima are only brought up to date when some key lies above one by
                    // more than 2^8 (the scores' range; p <= 2^8 then): rare after the start.
                    float top[C::NR][2];
                    bool grows = false;
#pragma unroll
                    for (int t = 0; t < C::NR; ++t)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x = fmaxf(s[0][t][e], s[0][t][e + 2]);
#pragma unroll
                            for (int i = 1; i < C::KS / 16; ++i) x = max3f(x, s[i][t][e], s[i][t][e + 2]);
                            top[t][e] = x * sl2;
                            grows |= top[t][e] > m[t][e] + kTau;
                        }
                    if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                        for (int t = 0; t < C::NR; ++t)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float x = top[t][e];
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                                const float now = fmaxf(m[t][e], x);
                                const float a = now == m[t][e] ? 1.0f : ex2_approx(m[t][e] - now);
                                m[t][e] = now;
                                l[t][e] *= a;
#pragma unroll
                                for (int i = 0; i < C::D / 16; ++i) {
                                    acc[i][t][e] *= a;
                                    acc[i][t][e + 2] *= a;
                                }
                            }
                    }
#pragma unroll
                    for (int t = 0; t < C::NR; ++t) {
                        const float neg0 = m[t][0] == -INFINITY ? 0.0f : -m[t][0];
                        const float neg1 = m[t][1] == -INFINITY ? 0.0f : -m[t][1];
#pragma unroll
                        for (int i = 0; i < C::KS / 16; ++i) {
                            const float p0 = ex2_approx(fmaf(s[i][t][0], sl2, neg0));
                            const float p1 = ex2_approx(fmaf(s[i][t][1], sl2, neg1));
                            const float p2 = ex2_approx(fmaf(s[i][t][2], sl2, neg0));
                            const float p3 = ex2_approx(fmaf(s[i][t][3], sl2, neg1));
                            l[t][0] += p0 + p2;
                            l[t][1] += p1 + p3;
                            const uint32_t a = pack_bf16x2(p0, p1), b = pack_bf16x2(p2, p3);
                            pf[i][t][0] = transpose8(a);
                            pf[i][t][1] = transpose8(b);
                            pl[i][t][0] = transpose8(rounding_error(a, p0, p1));
                            pl[i][t][1] = transpose8(rounding_error(b, p2, p3));
                        }
                    }
                }
                // The K slot has been read: the next load goes there.
                __syncwarp();
                if (C::WR > 1 && lane == 0) mbar_arrive(bar(empty0 + ks));
                ++pos;
                load_next();
                if (!ok) break;
                const int vs = pos % C::NSLOT;
                ok = warp_wait(bar(full0 + vs), (pos / C::NSLOT) & 1, abort_flag, status);
                if (!ok) break;
                if (rows_here) {
                    const uint32_t va = ring + vs * C::SLOT_BYTES + ((mi >> 1) * 8 + m8) * C::ROW_BYTES;
                    auto pv = [&](auto masked) {
#pragma unroll
                        for (int i = 0; i < C::KS / 16; ++i) {
                            // Keys that no row sees may hold anything, and 0 * NaN would stay NaN.
                            uint32_t keep0 = 0, keep1 = 0;
                            if (masked) {
                                const int at = key + i * 16 + c2;
                                auto seen = [&](int k) { return k >= pc.first && k < pc.end; };
                                keep0 = (seen(at) ? 0xffffu : 0u) | (seen(at + 1) ? 0xffff0000u : 0u);
                                keep1 = (seen(at + 8) ? 0xffffu : 0u) | (seen(at + 9) ? 0xffff0000u : 0u);
                            }
#pragma unroll
                            for (int d = 0; d < C::D / 16; ++d) {
                                uint32_t a[4];
                                ldsm4_trans(va + i * 16 * C::ROW_BYTES + (((d * 2 + (mi & 1)) ^ m8) << 4), a);
                                if (masked) {
                                    a[0] &= keep0;
                                    a[1] &= keep0;
                                    a[2] &= keep1;
                                    a[3] &= keep1;
                                }
#pragma unroll
                                for (int t = 0; t < C::NR; ++t) {
                                    mma16816(acc[d][t], a, pf[i][t][0], pf[i][t][1]);
                                    mma16816(acc[d][t], a, pl[i][t][0], pl[i][t][1]);
                                }
                            }
                        }
                    };
                    if (edge) pv(std::true_type{});
                    else pv(std::false_type{});
                }
                __syncwarp();
                if (C::WR > 1 && lane == 0) mbar_arrive(bar(empty0 + vs));
                ++pos;
                load_next();
                if (!ok) break;
            }
            if (!ok) break;
#pragma unroll
            for (int t = 0; t < C::NR; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = l[t][e];
                    x += __shfl_xor_sync(0xffffffffu, x, 4);
                    x += __shfl_xor_sync(0xffffffffu, x, 8);
                    x += __shfl_xor_sync(0xffffffffu, x, 16);
                    const int rr = (wr * C::NR + t) * 8 + c2 + e;
                    if (rr < pc.rows) {
#pragma unroll
                        for (int i = 0; i < C::D / 16; ++i) {
                            const int64_t q4 = i * 4 + (r8 >> 2);
                            pc.part[(q4 * pc.part_rows + rr) * 4 + (r8 & 3)] = acc[i][t][e];
                            pc.part[((q4 + 2) * pc.part_rows + rr) * 4 + (r8 & 3)] = acc[i][t][e + 2];
                        }
                        if (r8 == 0) pc.ml[rr] = make_float2(m[t][e], x);
                    }
                }
        }
        // After an abort let the loads in flight land before the CTA ends.
        asm volatile("cp.async.wait_all;" ::: "memory");
    }

    __syncthreads();
    // The prefix kernel before this grid may still run: one CTA stays until it
    // has ended, so that this grid's end means both.
    if (blockIdx.x == 0) wait_for_previous_grid();
}

}  // namespace thd
