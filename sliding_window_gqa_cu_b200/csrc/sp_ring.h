// The order in which the K and V tiles of the shared prefix go through their ring of
// slots, and what a producer waits for.  Plain C++, for the device and for the host's
// tests.
#pragma once

#ifdef __CUDACC__
#define SP_RING_FN __host__ __device__ __forceinline__
#else
#define SP_RING_FN inline
#endif

namespace thd {

// A piece of n key tiles with NSB score buffers: K tiles ahead, then V(0), K(NSB),
// V(1), ...  `tile(is_v)` returns whether to go on.
template <int NSB, class Tile>
SP_RING_FN bool ring_piece(int n, Tile tile) {
    for (int i = 0; i < NSB && i < n; ++i)
        if (!tile(false)) return false;
    for (int i = 0; i < n; ++i) {
        if (!tile(true)) return false;
        if (i + NSB < n && !tile(false)) return false;
    }
    return true;
}

// The `sub` slots of one tile at ring position `pos`, by a producer that loads the
// tile (mine) or goes past it.  wait(slot, parity) waits for the slot's release, load(s,
// slot) fills it.  A producer waits for the slots that it fills and for no others: of
// another's slot it may come too late, after the other has filled it and the consumers
// have released it again, and the parity that it looks for is then that of a release
// which comes only after tiles of its own.  Of its own slots it cannot be ahead by two
// releases either, because its tiles are never more than `nslot` positions apart (at the
// start of a piece with NSB = 2: 5) and the consumers go in order.
template <class Wait, class Load>
SP_RING_FN bool ring_tile(bool mine, int sub, int nslot, int& pos, Wait wait, Load load) {
    for (int s = 0; s < sub; ++s, ++pos) {
        if (!mine) continue;
        const int slot = pos % nslot;
        if (!wait(slot, ((pos / nslot) & 1) ^ 1)) return false;
        load(s, slot);
    }
    return true;
}

}  // namespace thd

#undef SP_RING_FN
