"""The ring of K and V slots of the shared prefix (csrc/sp_ring.h), compiled for the
host: one thread a producer and one a consumer, barriers with phases as the GPU's
(a wait only sees the parity), and delays anywhere.  No slot may be filled before
all consumers have released it, every tile arrives in order, and nobody waits for ever."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <thread>
#include <vector>
#include "sp_ring.h"

using Clock = std::chrono::steady_clock;
struct Barrier {                        // completes a phase every `count` arrivals
    std::atomic<int> phase{0}, arrived{0};
    int count = 1;
    void arrive() { if (arrived.fetch_add(1) + 1 == count) { arrived = 0; phase.fetch_add(1); } }
    bool done(int parity) const { return (phase.load() & 1) != parity; }
};

template <int NSB>
int run(int nslot, int sub, int consumers, unsigned seed, int late) {
    std::mt19937 rng(seed);
    std::vector<int> pieces;
    for (int i = 0; i < 12; ++i) pieces.push_back(rng() % 5 == 0 ? 0 : 1 + rng() % 7);
    std::vector<Barrier> full(nslot), empty(nslot);
    for (auto& e : empty) e.count = consumers;
    std::vector<std::atomic<int>> held(nslot);      // tile number of the slot's contents, 0: released
    std::vector<std::atomic<int>> readers(nslot);   // consumers that have read it
    for (int i = 0; i < nslot; ++i) held[i] = readers[i] = 0;
    std::atomic<int> bad{0};
    auto wait = [&](Barrier& b, int parity) {
        const auto t0 = Clock::now();
        while (!b.done(parity)) {
            if (bad) return false;
            if (Clock::now() - t0 > std::chrono::seconds(20)) { bad = 1; return false; }
            std::this_thread::yield();
        }
        return true;
    };
    auto pause = [&](std::mt19937& r, int who) {     // the late one often waits long, the others briefly
        const int odds = who == late ? 3 : 40;
        if (r() % odds == 0) std::this_thread::sleep_for(std::chrono::microseconds(who == late ? 400 : 30));
    };
    auto producer = [&](bool is_v) {
        std::mt19937 r(seed * 7 + is_v);
        int pos = 0;
        for (int n : pieces)
            if (!thd::ring_piece<NSB>(n, [&](bool v) {
                    pause(r, is_v);
                    return thd::ring_tile(v == is_v, sub, nslot, pos,
                        [&](int slot, int parity) { return wait(empty[slot], parity); },
                        [&](int s, int slot) {
                            if (held[slot].exchange(pos + 1) != 0) bad = 2;      // still in use
                            full[slot].arrive();
                        });
                })) return;
    };
    auto consumer = [&](int me) {
        std::mt19937 r(seed * 13 + me);
        int pos = 0;
        for (int n : pieces)
            for (int i = 0; i < 2 * n * sub; ++i, ++pos) {
                const int slot = pos % nslot;
                if (!wait(full[slot], (pos / nslot) & 1)) return;
                if (held[slot] != pos + 1) bad = 3;                               // another tile
                pause(r, 2 + me);
                if (readers[slot].fetch_add(1) + 1 == consumers) { readers[slot] = 0; held[slot] = 0; }
                empty[slot].arrive();
            }
    };
    std::vector<std::thread> t;
    t.emplace_back(producer, false);
    t.emplace_back(producer, true);
    for (int c = 0; c < consumers; ++c) t.emplace_back(consumer, c);
    for (auto& x : t) x.join();
    return bad;
}

int main(int argc, char** argv) {
    const int nsb = atoi(argv[1]), nslot = atoi(argv[2]), sub = atoi(argv[3]), consumers = atoi(argv[4]);
    for (unsigned seed = 1; seed <= 24; ++seed)
        for (int late = 0; late < 2; ++late) {
            const int bad = nsb == 2 ? run<2>(nslot, sub, consumers, seed, late) : run<1>(nslot, sub, consumers, seed, late);
            if (bad) {
                printf("%s (seed %u, late %s)\n", bad == 1 ? "a wait that does not end" : bad == 2 ? "a slot filled while in use"
                       : "a tile out of order", seed, late ? "V" : "K");
                return 1;
            }
        }
    return 0;
}
"""


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    (d / "ring.cpp").write_text(SOURCE)
    exe = d / "ring"
    subprocess.run(["g++", "-O1", "-std=c++17", "-pthread", "-I", os.path.join(ROOT, "sliding_window_gqa_cu_b200", "csrc"),
                    "-o", str(exe), str(d / "ring.cpp")], check=True)
    return exe


@pytest.mark.parametrize("nsb,nslot,sub,consumers", [(1, 10, 1, 2), (1, 5, 1, 2), (2, 5, 2, 1)],
                         ids=["head dim 64", "head dim 128", "head dim 256"])
def test_ring_of_the_prefix(ring, nsb, nslot, sub, consumers):
    r = subprocess.run([str(ring), str(nsb), str(nslot), str(sub), str(consumers)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
