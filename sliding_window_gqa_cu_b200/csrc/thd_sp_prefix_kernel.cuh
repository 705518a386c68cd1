// The shared prefix on the tensor cores: every query row of the batch against
// the pages of the prefix, each key tile read once for NT * 128 rows.
//
// With P prefix keys and R = tokens * G rows per kv head this is two matrix
// products of 2 R P D operations each per kv head around a softmax, so with
// many rows the tensor core bounds it (a 128 x 128 tile at D = 128: 2 * 512
// cycles) next to the exponential unit (16 a cycle: 1024 cycles a tile).
// NT = 2 row tiles per CTA (D <= 128) take turns: while one tile's scores are
// in the softmax the tensor core works on the other's.  At D = 256 the two
// accumulators would fill TMEM, so one row tile with two score buffers does
// the same, and two threads share a row.
//
// Work split: groups of NT * 128 rows; `pre_width` groups of a kv head walk the
// same keys in step (one CTA each, so that K and V come from L2 for all but the
// first), and the sequence (bundle of groups, kv head, key tile) is cut into
// equal ranges, one per lane of CTAs.  How many lanes work is decided from the
// lengths (sp_split): the CTAs beyond leave their SMs to the paged kernel.
//
// Warps: 8 softmax warps (a thread a row; D = 256: two), a TMA producer for K and
// one for V, an MMA issuer for each row tile.  A TMA box holds a page's tokens
// (128 at most) x all columns of a slot: [tokens / 8][column chunk][8 tokens][64
// columns], whose groups of 8 tokens have one stride over the pages of a tile, as
// the matrix descriptors need it.
#pragma once

#include "sp_ring.h"
#include "thd_attn_kernel.cuh"
#include "thd_sp_common.cuh"

namespace thd {

template <int D_>
struct PrefixConfig {
    static constexpr int D = D_;
    static constexpr int NT = D == 256 ? 1 : 2;   // row tiles of a CTA
    static constexpr int NSB = D == 256 ? 2 : 1;  // score buffers of a row tile
    static constexpr int BN = 128;                // keys of a tile
    static constexpr int SC = D < 128 ? D : 128;  // columns of a ring slot
    static constexpr int SUB = D / SC;            // slots of a K or V tile
    static constexpr int CH = SC / 64;            // 128-byte chunks of a slot row
    static constexpr int NSLOT = D == 64 ? 10 : 5;
    static constexpr int HALVES = D == 256 ? 2 : 1;  // threads that share a row's softmax
    static constexpr int COLS = BN / HALVES;         // keys of a tile that a thread takes,
    static constexpr int CK = COLS / 2;              // in two chunks of this many
    static constexpr int Q_CHUNK_BYTES = 128 * 128;    // one chunk of a Q tile
    static constexpr int GROUP_BYTES = CH * 1024;      // 8 keys of a slot, chunk by chunk
    static constexpr int SLOT_BYTES = BN * SC * 2;
    static constexpr int Q_TILE_BYTES = 128 * D * 2;
    static constexpr int SOFTMAX_WARPS = 4 * NT * HALVES;
    static constexpr int K_WARP = SOFTMAX_WARPS;
    static constexpr int V_WARP = SOFTMAX_WARPS + 1;
    static constexpr int MMA_WARP = SOFTMAX_WARPS + 2;
    static constexpr int THREADS = (SOFTMAX_WARPS + 2 + NT) * 32;
    static constexpr int TMEM_O = NT * NSB * BN;
    static_assert(TMEM_O + NT * D <= 512, "TMEM budget exceeded");

    static constexpr int B_Q_FULL = 0;                        // [NT]
    static constexpr int B_SLOT_FULL = B_Q_FULL + NT;
    static constexpr int B_SLOT_EMPTY = B_SLOT_FULL + NSLOT;
    static constexpr int B_S_FULL = B_SLOT_EMPTY + NSLOT;     // [NT][NSB]
    static constexpr int B_P_FULL = B_S_FULL + NT * NSB;      // [NT][2]: P of 64 keys written, O rescaled
    static constexpr int B_O_FULL = B_P_FULL + 2 * NT;        // [NT]
    static constexpr int B_TURN = B_O_FULL + NT;              // [NT]
    static constexpr int B_DRAIN = B_TURN + NT;
    static constexpr int NUM_BARS = B_DRAIN + 1;

    static constexpr int SMEM_SLOTS = NT * Q_TILE_BYTES;
    static constexpr int SMEM_BAR = SMEM_SLOTS + NSLOT * SLOT_BYTES;
    static constexpr int SMEM_MIN = SMEM_BAR + NUM_BARS * 8;  // [2][16]: least own length, cost of the own keys of a warp's requests
    static constexpr int SMEM_XCH = SMEM_MIN + 32 * 4;          // float [NSB][NT][2][128]: maxima (sums) of two threads of a row
    static constexpr int SMEM_TMEM_SLOT = SMEM_XCH + (HALVES > 1 ? NSB * NT * 2 * 128 * 4 : 0);
    static constexpr int SMEM_ABORT = SMEM_TMEM_SLOT + 4;
    static constexpr int SMEM_BYTES = SMEM_ABORT + 4;
    static_assert(SMEM_BYTES <= 232448 && NSLOT >= 2 * SUB, "shared memory budget");
};

// One CTA's share of one item.
struct PrefixPiece {
    int h, row0, tiles;       // kv head, first row, active row tiles
    int kt, n;                // first key tile and how many
    int lo;                   // first key that some row sees
    bool home;                // holds the item's first tile
    int group;                // row group
};

// Walks the pieces of a CTA; called by whole warps, which all get the same.
template <class C>
struct PrefixWalk {
    long long x, x1;
    int member, first_tile, n_tiles, prefix;

    __device__ __forceinline__ bool next(const SpParams& p, PrefixPiece& pc) {
        while (x < x1) {
            const int len = n_tiles + kItemTiles;
            const int item = x <= 0x7fffffff ? static_cast<int>(x) / len : static_cast<int>(x / len);
            const int at = static_cast<int>(x - static_cast<long long>(item) * len);
            const int cnt = static_cast<int>(min(static_cast<long long>(len - at), x1 - x));
            const int t0 = max(at - kItemTiles, 0), t1 = at + cnt - kItemTiles;
            x += cnt;
            pc.h = item % p.Hkv;
            pc.group = item / p.Hkv * p.pre_width + member;
            if (pc.group >= p.pre_groups || t1 <= t0) continue;
            pc.row0 = pc.group * (C::NT * 128);
            const int left = p.rows - pc.row0;
            pc.tiles = C::NT == 2 && left > 128 ? 2 : 1;
            pc.home = t0 == 0;
            int lo = 0;
            if (p.window > 0) {
                // least own length of the group's requests
                const int last = min(left, C::NT * 128) - 1;
                const int b0 = pc.row0 / p.RB, b1 = (pc.row0 + last) / p.RB;
                int n = 0x7fffffff;
                for (int b = b0 + static_cast<int>(threadIdx.x & 31); b <= b1; b += 32) {
                    const int len = sp_own_len(p, b);
                    if (len >= 0) n = min(n, len);
                }
                n = __reduce_min_sync(0xffffffffu, n);
                lo = n == 0x7fffffff ? prefix : sp_first_key(p, prefix + n - p.n_q);
            }
            pc.lo = lo;
            const int k0 = max(first_tile + t0, lo / C::BN);
            pc.kt = k0;
            pc.n = max(0, first_tile + t1 - k0);
            if (lo >= prefix) pc.n = 0;
            return true;
        }
        return false;
    }
};

// Wait of a whole warp, every thread polling: the shortest way if the phase is
// over already.
__device__ __forceinline__ bool warp_poll(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return warp_wait(bar, parity, abort_flag, status);
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
thd_sp_prefix_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                     const SpParams p, int* status) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_addr(smem);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    launch_dependents();

    auto bar = [&](int idx) -> uint32_t { return sbase + C::SMEM_BAR + 8u * idx; };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::SMEM_ABORT);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::SMEM_TMEM_SLOT);
    int* warp_min = reinterpret_cast<int*>(smem + C::SMEM_MIN);
    float* warp_cost = reinterpret_cast<float*>(warp_min + 16);

    if (threadIdx.x == 0) {
        for (int q = 0; q < C::NT; ++q) {
            mbar_init(bar(C::B_Q_FULL + q), 4 * C::HALVES);
            mbar_init(bar(C::B_P_FULL + 2 * q), 4);
            mbar_init(bar(C::B_P_FULL + 2 * q + 1), 4);
            mbar_init(bar(C::B_O_FULL + q), 1);
        }
        for (int s = 0; s < C::NSLOT; ++s) {
            mbar_init(bar(C::B_SLOT_FULL + s), 1);
            mbar_init(bar(C::B_SLOT_EMPTY + s), C::NT);
        }
        for (int i = 0; i < C::NT * C::NSB; ++i) mbar_init(bar(C::B_S_FULL + i), 1);
        for (int q = 0; q < C::NT; ++q) mbar_init(bar(C::B_TURN + q), 1);
        mbar_init(bar(C::B_DRAIN), C::NT);
        int bad = *reinterpret_cast<volatile int*>(status) != 0 ? 1 : 0;
        if ((sbase & 1023u) != 0) {  // the swizzled tiles need it
            atomicCAS(status, 0, kStatusBadItem);
            bad = 1;
        }
        *abort_flag = bad;
        fence_barrier_init();
    }
    if (threadIdx.x == 32) {
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
    }
    // Least own length (for the first key that any row sees) and what all own keys cost.
    const int P = sp_prefix_len(p);
    {
        int n = 0x7fffffff;
        float cost = 0.0f;
        for (int b = threadIdx.x; b < p.n_req; b += C::THREADS) {
            const int len = sp_own_len(p, b);
            if (len < 0) continue;
            n = min(n, len);
            cost += sp_own_cost(p, len);
        }
        n = __reduce_min_sync(0xffffffffu, n);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) cost += __shfl_xor_sync(0xffffffffu, cost, o);
        if (lane == 0) {
            warp_min[warp] = n;
            warp_cost[warp] = cost;
        }
    }
    __syncthreads();
    PrefixWalk<C> walk;
    {
        int n = 0x7fffffff;
        float cost = 0.0f;
        for (int w = 0; w < C::THREADS / 32; ++w) {
            n = min(n, warp_min[w]);
            cost += warp_cost[w];
        }
        const int lo = n == 0x7fffffff ? P : sp_first_key(p, P + n - p.n_q);
        walk.first_tile = lo / C::BN;
        walk.n_tiles = lo < P ? (P - 1) / C::BN + 1 - walk.first_tile : 0;
        walk.prefix = P;
        walk.member = blockIdx.x % p.pre_width;
        const int my_lane = blockIdx.x / p.pre_width;
        const long long units = sp_prefix_units(p, walk.n_tiles);
        const int lanes = sp_split<C::D>(p, units, cost).lanes;
        walk.x = lanes > 0 ? lane_begin(units, lanes, my_lane) : 0;
        walk.x1 = lanes > 0 ? lane_begin(units, lanes, my_lane + 1) : 0;
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            p.plan->pre_tiles = walk.n_tiles;
            p.plan->pre_lanes = lanes;
        }
        if (my_lane >= lanes) return;  // its SM is the paged kernel's
    }
    if (warp == C::MMA_WARP) {
        tmem_alloc(smem_addr(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const bool skip = *abort_flag != 0;
    PrefixPiece pc;

    if (warp == C::K_WARP || warp == C::V_WARP) {
        // ----------------------------------------------- TMA producers (K, V)
        if (!skip) {
            const bool is_v = warp == C::V_WARP;
            const CUtensorMap* map = is_v ? &tmap_v : &tmap_k;
            const int boxes = C::BN / p.box_rows;  // of a slot, one lane each
            const int box = lane < boxes ? lane : 0;
            int pos = 0;        // ring position
            uint32_t mine = 0;  // bit i: this warp loaded position pos - 1 - i
            bool ok = true;
            // Place of this lane's box of key tile kt (behind the cache if it has no page).
            auto place_of = [&](int kt, int h) -> int {
                const int idx = (kt * C::BN + box * p.box_rows) >> p.block_shift;
                int id = -1;
                if (idx < p.prefix_blocks) id = p.prefix_table[idx];
                return id >= 0 && id < p.num_blocks ? id * p.place_block + h * p.place_head : p.places;
            };
            while (ok && walk.next(p, pc)) {
                if (pc.n == 0) continue;
                int next = place_of(pc.kt, pc.h);
                int j = 0;  // this warp's next tile
                ok = ring_piece<C::NSB>(pc.n, [&](bool v) {
                    const bool load = v == is_v;
                    if (!load) mine <<= C::SUB;
                    const int place = next;
                    if (load && j + 1 < pc.n) next = place_of(pc.kt + j + 1, pc.h);
                    const int eight = (((pc.kt + j) * C::BN + box * p.box_rows) & (p.block - 1)) >> 3;
                    if (load) ++j;
                    return ring_tile(
                        load, C::SUB, C::NSLOT, pos,
                        [&](int slot, int parity) {
                            return warp_wait(bar(C::B_SLOT_EMPTY + slot), parity, abort_flag, status);
                        },
                        [&](int s, int slot) {
                            if (lane == 0) mbar_arrive_expect_tx(bar(C::B_SLOT_FULL + slot), C::SLOT_BYTES);
                            __syncwarp();
                            if (lane < boxes)
                                tma_load_5d(sbase + C::SMEM_SLOTS + slot * C::SLOT_BYTES + box * (p.box_rows / 8) * C::GROUP_BYTES,
                                            map, bar(C::B_SLOT_FULL + slot), 0, 0, s * C::CH, eight, place);
                            mine = mine << 1 | 1u;
                        });
                });
            }
            if (!ok && lane == 0)  // let the loads in flight land before the CTA ends
                for (int i = 0; i < C::NSLOT && i < pos; ++i)
                    if (mine >> i & 1)
                        drain_wait(bar(C::B_SLOT_FULL + (pos - 1 - i) % C::NSLOT), ((pos - 1 - i) / C::NSLOT) & 1);
        }
        __syncwarp();
    } else if (warp >= C::MMA_WARP && warp < C::MMA_WARP + C::NT) {
        // ------------------------------------------ MMA issuers, one a row tile
        // Issuing is what one warp for both row tiles spends its time on: 32 instructions
        // (about 52 cycles each), six waits (some 200) and four commits, 4,000 cycles a
        // pair of tiles, where the products need 2,048.  One warp a tile: 256 requests on
        // 32,768 tokens 256 -> 250 us, 64 on 8,191 38 -> 33 us for this kernel.
        if (!skip) {
            const int q = warp - C::MMA_WARP;
            const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
            constexpr uint32_t idesc_qk = idesc_bf16_f32(128, C::BN, false);
            constexpr uint32_t idesc_pv = idesc_bf16_f32(128, C::SC, true);
            const uint64_t dq0 = smem_desc_sw128(sbase, 16, 1024);
            const uint64_t dk0 = smem_desc_sw128(sbase + C::SMEM_SLOTS, 16, C::GROUP_BYTES);
            const uint64_t dv0 = smem_desc_sw128(sbase + C::SMEM_SLOTS, 1024, C::GROUP_BYTES);
            // Part s of S = Q K^T: head-dim columns [s SC, (s + 1) SC).
            auto issue_qk = [&](int b, int s, int slot) {
                const uint32_t d_tmem = tmem_base + (q * C::NSB + b) * C::BN;
                const uint64_t dq = dq0 + ((q * C::Q_TILE_BYTES + s * C::CH * C::Q_CHUNK_BYTES) >> 4);
                const uint64_t dk = dk0 + ((slot * C::SLOT_BYTES) >> 4);
                if (!elect_one()) return;
#pragma unroll
                for (int kk = 0; kk < C::SC / 16; ++kk) {
                    const uint32_t qo = ((kk >> 2) * C::Q_CHUNK_BYTES + (kk & 3) * 32) >> 4;
                    const uint32_t ko = ((kk >> 2) * 1024 + (kk & 3) * 32) >> 4;
                    mma_bf16_ss(d_tmem, dq + qo, dk + ko, idesc_qk, s > 0 || kk > 0 ? 1u : 0u);
                }
            };
            // Part s of O += P V (columns [s SC, ..)) over keys [64 half, 64 half + 64),
            // whose P lies in the first half of every CK score columns.
            auto issue_pv = [&](int b, int s, int slot, int half, bool acc) {
                const uint32_t d_tmem = tmem_base + C::TMEM_O + q * C::D + s * C::SC;
                const uint32_t p_tmem = tmem_base + (q * C::NSB + b) * C::BN + half * 64;
                const uint64_t dv = dv0 + ((slot * C::SLOT_BYTES + half * 8 * C::GROUP_BYTES) >> 4);
                if (!elect_one()) return;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_bf16_ts(d_tmem, p_tmem + kk * 16 / C::CK * C::CK + kk * 16 % C::CK / 2,
                                dv + ((kk * 2 * C::GROUP_BYTES) >> 4), idesc_pv, acc || kk > 0 ? 1u : 0u);
            };
            auto commit = [&](int idx) {
                if (elect_one()) mma_commit(bar(idx));
            };
            int pos = 0, pieces = 0, done = 0, turns = 0;
            bool ok = true;
            auto wait = [&](int idx, uint32_t parity) -> bool {
                return warp_poll(bar(idx), parity, abort_flag, status);
            };
            auto wait_slot = [&](int at) -> bool {
                return wait(C::B_SLOT_FULL + at % C::NSLOT, (at / C::NSLOT) & 1);
            };
            while (walk.next(p, pc)) {
                if (pc.n == 0 || !ok) continue;
                const int n = pc.n;
                if (q >= pc.tiles) {
                    // No rows in this tile: its share of the slots' releases only.
                    for (int i = 0; i < 2 * n * C::SUB && ok; ++i, ++pos) {
                        ok = wait_slot(pos);
                        if (ok && lane == 0) mbar_arrive(bar(C::B_SLOT_EMPTY + pos % C::NSLOT));
                    }
                    continue;
                }
                ok = wait(C::B_Q_FULL + q, pieces & 1);
                // K tile of step jj at ring position `pos`: one part per slot
                auto qk = [&](int jj) {
                    for (int s = 0; s < C::SUB && ok; ++s, ++pos) {
                        ok = wait_slot(pos);
                        if (!ok) return;
                        tc_fence_after();
                        issue_qk((done + jj) % C::NSB, s, pos % C::NSLOT);
                        if (s == C::SUB - 1) commit(C::B_S_FULL + q * C::NSB + (done + jj) % C::NSB);
                        commit(C::B_SLOT_EMPTY + pos % C::NSLOT);
                    }
                };
                for (int jj = 0; jj < C::NSB && jj < n && ok; ++jj) qk(jj);
                if (C::NT == 2 && pc.tiles == 2) {
                    // The row tiles take turns: PV(j) and QK(j + 1) of one go out as one run
                    // while the other is in its softmax.  (Without turns both tiles drift into
                    // step, all softmax and then all products: 4,500 cycles a pair of tiles.)
                    for (int j = 0; j < n && ok; ++j) {
                        const bool more = j + 1 < n;
                        // (what is long there is waited for first)
                        ok = wait_slot(pos) && (!more || wait_slot(pos + 1)) && wait(C::B_P_FULL + 2 * q + 1, (done + j) & 1);
                        if (!ok) break;
                        tc_fence_after();
                        issue_pv(0, 0, pos % C::NSLOT, 1, j > 0);
                        ok = wait(C::B_P_FULL + 2 * q, (done + j) & 1) && wait(C::B_TURN + q, (turns & 1) ^ (q == 0 ? 1 : 0));
                        if (!ok) break;
                        tc_fence_after();
                        issue_pv(0, 0, pos % C::NSLOT, 0, true);
                        if (more) {
                            issue_qk(0, 0, (pos + 1) % C::NSLOT);
                            commit(C::B_S_FULL + q);
                        } else {
                            commit(C::B_O_FULL + q);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(C::B_TURN + 1 - q));
                        ++turns;
                        commit(C::B_SLOT_EMPTY + pos % C::NSLOT);
                        if (more) commit(C::B_SLOT_EMPTY + (pos + 1) % C::NSLOT);
                        pos += more ? 2 : 1;
                    }
                    ++pieces;
                    done += n;
                    continue;
                }
                for (int j = 0; j < n && ok; ++j) {
                    const bool more = j + C::NSB < n;
                    const int b = (done + j) % C::NSB;
                    // PV(j); with one score buffer S(j + 1) ready also says that O holds it.
                    for (int s = 0; s < C::SUB && ok; ++s, ++pos) {
                        ok = wait_slot(pos);
                        // (with one thread a row its second chunk is published first)
                        for (int i = 0; i < 2 && ok; ++i) {
                            const int half = C::HALVES == 1 ? 1 - i : i;
                            if (s == 0) ok = wait(C::B_P_FULL + 2 * q + half, (done + j) & 1);
                            if (!ok) break;
                            tc_fence_after();
                            issue_pv(b, s, pos % C::NSLOT, half, j > 0 || i > 0);
                        }
                        if (!ok) break;
                        if (s == C::SUB - 1 && (C::NSB == 2 || !more)) commit(C::B_O_FULL + q);
                        commit(C::B_SLOT_EMPTY + pos % C::NSLOT);
                    }
                    if (ok && more) qk(j + C::NSB);
                }
                ++pieces;
                done += n;
            }
            if (elect_one()) mma_commit(bar(C::B_DRAIN));
            if (lane == 0) drain_wait(bar(C::B_DRAIN), 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        const int q = warp / (4 * C::HALVES), half = (warp >> 2) % C::HALVES;
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        // This warp's share of O and, in a score buffer, of S and P.
        constexpr int O_COLS = C::D / C::HALVES;
        const uint32_t o_tmem = lane_base + C::TMEM_O + q * C::D + half * O_COLS;
        const uint32_t s_tmem0 = lane_base + q * C::NSB * C::BN + half * C::COLS;
        float* xch = reinterpret_cast<float*>(smem + C::SMEM_XCH) + q * 256 + row;
        const uint32_t pair_bar = 1 + q * 4 + (warp & 3);  // of the two warps that share rows
        const float sl2 = p.scale_log2;
        constexpr float kTau = 8.0f;  // rescale O only when the maximum grows by more than 2^8
        int pos = 0, pieces = 0, done = 0, turn = 0;
        bool ok = !skip;
        // The two threads of a row swap a value.  (With one score buffer S(j + 1) is only
        // ready when both have published P(j), so the place is free again; with two
        // they take turns.)  A warp that gives up still arrives (below), and its
        // partner sees the flag before it could wait again.
        auto swap = [&](float v) -> float {
            float* at = xch + turn % C::NSB * (C::NT * 256);
            ++turn;
            at[half * 128] = v;
            if (*abort_flag != 0) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) return v;
            asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
            return at[(1 - half) * 128];
        };
        // Q rows of a piece into shared memory, 128-byte swizzled: every warp of a row
        // tile its share.
        auto load_q = [&](const PrefixPiece& c) {
            constexpr int PER = C::D / 8;  // 16-byte pieces of a row
            constexpr int SHARE = 32 / C::HALVES;
            const int l_first = warp % (4 * C::HALVES) * SHARE, r_first = c.row0 + q * 128 + l_first;
            int64_t off = 0;  // thread t: row r_first + t
            const int mine = min(r_first + lane % SHARE, p.rows - 1), t = mine / p.G;
            off = (static_cast<int64_t>(t) * p.Hq + c.h * p.G + (mine - t * p.G)) * C::D;
#pragma unroll
            for (int i = 0; i < SHARE * PER / 32; ++i) {
                const int rr = (i * 32 + lane) / PER, piece = (i * 32 + lane) % PER, lr = l_first + rr;
                const int64_t at = __shfl_sync(0xffffffffu, off, rr);
                const uint32_t dst = sbase + q * C::Q_TILE_BYTES + (piece >> 3) * C::Q_CHUNK_BYTES + lr * 128 +
                                     (((piece & 7) ^ (lr & 7)) << 4);
                load16(dst, p.q + at + piece * 8, r_first + rr < p.rows);
            }
        };
        // The page of 16-key group `lane` of this warp's share of tile kt.
        const int page_of_lane = (half * C::COLS + lane % (C::COLS / 16) * 16) >> p.block_shift;
        constexpr uint32_t kAllPages = (1u << (C::COLS / 16)) - 1;
        auto load_id = [&](int kt) -> int {
            const int idx = ((kt * C::BN) >> p.block_shift) + page_of_lane;
            return idx < p.prefix_blocks ? p.prefix_table[idx] : -1;
        };

        bool more = ok && walk.next(p, pc);
        bool q_loading = false;  // pc's Q is on its way
        while (ok && more) {
            const int base_pos = pos;
            pos += 2 * C::SUB * pc.n;
            if (q >= pc.tiles) {
                more = walk.next(p, pc);
                continue;
            }
            if (pc.n > 0 && !q_loading) load_q(pc);
            q_loading = false;
            const int r = pc.row0 + q * 128 + row;
            int jlo = pc.lo, jhi = P - 1;  // keys of the prefix that the row sees (unused rows: all)
            if (r < p.rows) {
                const int b = r / p.RB;
                const int n_own = sp_own_len(p, b);
                if (n_own >= 0) {
                    const int at = P + n_own - p.n_q + (r - b * p.RB) / p.G;
                    jlo = sp_first_key(p, at);
                    jhi = min(at, P - 1);
                }
            }
            float m_ref = -INFINITY, l = 0.0f;
            float* home;
            float2* ml;
            if (pc.home) {
                const int64_t tile = (static_cast<int64_t>(pc.h) * p.pre_groups + pc.group) * C::NT + q;
                home = p.pre_home + tile * (128 * C::D);
                ml = p.pre_home_ml + tile * 128;
            } else {
                const int64_t tile = static_cast<int64_t>(blockIdx.x) * C::NT + q;
                home = p.pre_cont + tile * (128 * C::D);
                ml = p.pre_cont_ml + tile * 128;
            }
            PrefixPiece next = pc;
            const int n = pc.n;
            if (n > 0) {
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_Q_FULL + q));
                int id = load_id(pc.kt);
                for (int j = 0; j < n; ++j) {
                    const int t = done + j;
                    const int b = t % C::NSB;
                    const int key0 = (pc.kt + j) * C::BN + half * C::COLS;  // this warp's first key
                    const uint32_t pages = __ballot_sync(0xffffffffu, id >= 0 && id < p.num_blocks) & kAllPages;
                    if (j + 1 < n) id = load_id(pc.kt + j + 1);
                    ok = warp_wait(bar(C::B_S_FULL + q * C::NSB + b), (t / C::NSB) & 1, abort_flag, status);
                    if (!ok) break;
                    tc_fence_after();
                    if (j == n - 1) {
                        // All products with this Q are done: the next piece's may come.
                        more = walk.next(p, next);
                        if (more && next.n > 0 && q < next.tiles) {
                            load_q(next);
                            q_loading = true;
                        }
                    }
                    const uint32_t s_tmem = s_tmem0 + b * C::BN;
                    const bool all = __all_sync(0xffffffffu, key0 >= jlo && key0 + C::COLS - 1 <= jhi) && pages == kAllPages;
                    // Scores of columns [c0, c0 + CK); hidden ones become -inf.
                    float sv[C::CK];
                    auto load = [&](int c0) {
                        uint32_t raw[C::CK];
#pragma unroll
                        for (int c = 0; c < C::CK; c += 32) tmem_ld32(s_tmem + c0 + c, *reinterpret_cast<uint32_t(*)[32]>(&raw[c]));
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < C::CK; c += 32) reg_fence32(*reinterpret_cast<uint32_t(*)[32]>(&raw[c]));
#pragma unroll
                        for (int c = 0; c < C::CK; ++c) sv[c] = __uint_as_float(raw[c]);
                        if (!all) {
                            const int at = key0 + c0;
#pragma unroll
                            for (int c = 0; c < C::CK; ++c)
                                if (at + c < jlo || at + c > jhi || !((pages >> ((c0 + c) >> 4)) & 1u)) sv[c] = -INFINITY;
                        }
                    };
                    auto largest = [&]() -> float {
                        float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
                        for (int c = 4; c < C::CK; c += 2) mx[(c >> 1) & 3] = max3f(mx[(c >> 1) & 3], sv[c], sv[c + 1]);
                        return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    };
                    load(0);
                    float m_tile = largest();
                    load(C::CK);
                    m_tile = fmaxf(m_tile, largest()) * sl2;
                    if constexpr (C::HALVES > 1) {
                        m_tile = fmaxf(m_tile, swap(m_tile));
                        if (!ok) break;
                    }

                    float alpha = 1.0f;
                    bool rescale = false;
                    if (j == 0) {
                        m_ref = m_tile;
                    } else if (m_tile > m_ref + kTau) {
                        alpha = ex2_approx(m_ref - m_tile);
                        m_ref = m_tile;
                        rescale = true;
                    }
                    l *= alpha;
                    const float neg_m = m_ref == -INFINITY ? 0.0f : -m_ref;
                    // O has to hold PV(j - 1) before it is rescaled and before P(j) is
                    // published.  With one score buffer S(j) ready says so.
                    if (C::NSB == 2 && j > 0) {
                        ok = warp_wait(bar(C::B_O_FULL + q), (t - 1) & 1, abort_flag, status);
                        if (!ok) break;
                        tc_fence_after();
                    }
                    // Values of keys that no row of the group sees may be anything: zero
                    // them, as 0 * NaN would stay NaN.  (Whatever held V(j)'s slots before
                    // has been consumed by now, so their phase is this one's.)
                    if (key0 < pc.lo || key0 + C::COLS - 1 >= P) {  // (up to 2^31 - 1)
                        const int v_tiles = min(n, C::NSB + j) + j;  // K and V tiles before V(j)
#pragma unroll 1
                        for (int s = 0; s < C::SUB && ok; ++s) {
                            const int at = base_pos + C::SUB * v_tiles + s;
                            ok = warp_wait(bar(C::B_SLOT_FULL + at % C::NSLOT), (at / C::NSLOT) & 1, abort_flag, status);
                            if (!ok) break;
                            // (every warp all keys of its share, so that none waits for another)
#pragma unroll 1
                            for (int k = lane; k < C::COLS; k += 32) {
                                if (key0 + k >= pc.lo && key0 + k < P) continue;
                                const int kr = half * C::COLS + k;
                                const uint32_t dst = sbase + C::SMEM_SLOTS + (at % C::NSLOT) * C::SLOT_BYTES +
                                                     (kr >> 3) * C::GROUP_BYTES + (kr & 7) * 128;
#pragma unroll
                                for (int c = 0; c < C::CH; ++c)
#pragma unroll
                                    for (int u = 0; u < 8; ++u) st_shared_v4(dst + c * 1024 + u * 16, 0, 0, 0, 0);
                            }
                        }
                        if (!ok) break;
                        fence_proxy_async_smem();
                    }
                    if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
                        for (int c = 0; c < O_COLS / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(o_tmem + c * 32, o);
                            tmem_wait_ld();
                            reg_fence32(o);
#pragma unroll
                            for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * alpha);
                            tmem_st32(o_tmem + c * 32, o);
                        }
                        tmem_wait_st();
                    }
                    const float2 sl2x2 = make_float2(sl2, sl2);
                    const float2 negm2 = make_float2(neg_m, neg_m);
                    float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
                    // P (rounded to bf16 once: another product for what that loses, as in the
                    // paged kernel, would add half of the products, which bound this one)
                    // of CK keys over the first half of their score columns: the second chunk
                    // is still in registers, the first is read again (holding both would
                    // spill).
                    auto publish = [&](int i) {
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(C::B_P_FULL + 2 * q + i));
                    };
                    exp_and_store_p<0, C::CK / 32, C::CK, 0>(sv, sl2x2, negm2, s_tmem + C::CK, acc0, acc1);
                    if constexpr (C::HALVES == 1) publish(1);
                    load(0);
                    exp_and_store_p<0, C::CK / 32, C::CK, 0>(sv, sl2x2, negm2, s_tmem, acc0, acc1);
                    publish(half);
                    l += (acc0.x + acc0.y) + (acc1.x + acc1.y);
                }
                if (ok)
                    ok = warp_wait(bar(C::B_O_FULL + q), C::NSB == 1 ? pieces & 1 : (done + n - 1) & 1, abort_flag, status);
                if (!ok) break;
                if constexpr (C::HALVES > 1) {
                    l += swap(l);
                    if (!ok) break;
                }
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < O_COLS / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(o_tmem + c * 32, o);
                    tmem_wait_ld();
                    reg_fence32(o);
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        *reinterpret_cast<uint4*>(home + ((half * (O_COLS / 4) + c * 8 + u) * 128 + row) * 4) =
                            make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
                }
                ++pieces;
                done += n;
            } else {
                more = walk.next(p, next);
            }
            if (half == 0) ml[row] = make_float2(m_ref, l);
            pc = next;
        }
        if (C::HALVES > 1 && !ok) asm volatile("bar.arrive %0, 64;" ::"r"(pair_bar) : "memory");
        asm volatile("cp.async.wait_all;" ::: "memory");
    }

    tc_fence_before();
    __syncthreads();
    if (warp == C::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

}  // namespace thd
