// How many blocks share a sequence's verification (host only).
#pragma once

#include <algorithm>

// `wide`: how many clusters of sixteen blocks the device runs at a time (it need not run any: eight is what all do).
//
// Eight where the vocabulary gives each thread some work (1 / 2 / 4 / 8 blocks, 8 sequences of 5 x 32000: 46 / 34 / 23 / 19 us,
// of 5 x 8000 27 / 23 / 23 / 22), fewer where that would take more than two rounds of blocks for short sweeps (64 sequences of
// 5 x 32000 48 / 36 / 31 / 46 us, of 5 x 8000 28 / 24 / 25 / 43, but of 9 x 151936 335 / 185 / 120 / 85).  Sixteen where a
// few sequences have long sweeps: 8 / 16 blocks, 4 sequences of 5 x 102400 27.3 / 25.4, 12 26.6 / 28.9, 16 28.9 / 37.3; of
// 5 x 262144 36.6 / 28.9, 44.1 / 38.0, 47.6 / 45.1, 18 55.6 / 56.5; trees of 17 x 151936 bf16 under an automaton, 1 / 8 / 16 /
// 24 of them: 13.9 / 34.0 / 31.0 / 34.8 against 12.5 / 25.8 / 25.3 / 31.9.
inline int fa_verify_blocks(int B, int V, int wide) {
    if (wide > 0 && V >= 98304 && B <= std::min(16, V / 8192)) return 16;
    int cluster = 8;
    while (cluster > 1 && (V < 2048 * cluster || (V < 65536 && B * cluster > 2 * 152))) cluster /= 2;
    return cluster;
}
