// How many blocks share a sequence's verification (host only).
#pragma once

#include <algorithm>

// `wide`: how many clusters of sixteen blocks the device runs at a time (it need not run any: eight is what all do).
//
// Eight where the vocabulary gives each thread some work (1 / 2 / 4 / 8 blocks, 8 sequences of 5 x 32000: 46 / 34 / 23 / 19 us,
// of 5 x 8000 27 / 23 / 23 / 22), fewer where that would take more than two rounds of blocks for short sweeps (64 sequences of
// 5 x 32000 48 / 36 / 31 / 46 us, of 5 x 8000 28 / 24 / 25 / 43, but of 9 x 151936 335 / 185 / 120 / 85).
//
// Sixteen where few sequences have long sweeps: a token costs more with a draft's row, with live bits, and 16-bit ones more a
// byte.  8 / 16 blocks, chains of 5 (7 under the automaton) or trees of 17, in us:
//   with an automaton: 8 bf16 chains with a draft, V 65536 34.8 / 36.8, 98304 53.4 / 43.9, 151936 46.4 / 37.0; 8 fp32 trees
//     98304 22.6 / 20.5, 151936 37.0 / 30.8; 8 bf16 trees 65536 26.6 / 26.7, 98304 24.6 / 24.6, 151936 37.0 / 28.8
//   bf16 with a draft, 8 chains: 65536 26.7 / 29.5, 98304 35.0 / 32.9, 151936 36.9 / 32.9
//   fp32 with a draft, 10 chains: 98304 28.8 / 31.7, 114688 30.7 / 30.6, 131072 34.8 / 32.9, 262144 45.1 / 41.2
//   fp32 without, 10 chains: 98304 20.6 / 20.5, 131072 18.6 / 18.4, 262144 16.4 / 14.5
//   bf16 without, 10 chains: 98304 20.7 / 22.7, 131072 18.5 / 20.5, 151936 18.5 / 16.5, 262144 22.7 / 20.6
// Few are those that run at a time, 14 here: of fp32 chains with a draft, V 131072, 14 take 34.9 / 32.8, 15 34.9 / 41.9, 16 41.2 /
// 41.8.  Under an automaton paths end early and over a large vocabulary two more pay: 16 bf16 trees of 131072 26.7 / 26.6, of
// 151936 36.9 / 30.8, 15 and 16 fp32 ones of 151936 38.9 / 41.1 and 32.8 / 30.9, 16 chains with a draft of 131072 41.0 / 39.2 and
// 45.0 / 39.0, of 262144 80.0 / 63.7 and 101 / 78; 24 bf16 trees of 131072 30.8 / 37.0, of 262144 41.1 / 41.2.
inline int fa_verify_blocks(int B, int V, int element_bytes, bool draft, bool automaton, int wide) {
    const int from = automaton ? 98304 : element_bytes == 4 ? (draft ? 122880 : 131072) : draft ? 98304 : 147456;
    if (wide > 0 && V >= from && B <= wide + (automaton && V >= 131072 ? 2 : 0)) return 16;
    int cluster = 8;
    while (cluster > 1 && (V < 2048 * cluster || (V < 65536 && B * cluster > 2 * 152))) cluster /= 2;
    return cluster;
}
