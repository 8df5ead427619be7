// Host check of the number of blocks that share a sequence's verification (fa_verify_blocks in csrc/fa_verify_blocks.cuh, the function
// fa_verify calls): reads lines "B V element_bytes draft automaton wide", prints the number for each.
#include <cstdio>

#include "../constrained_decoding_diffusion_gb300/csrc/fa_verify_blocks.cuh"

int main() {
    int B, V, bytes, draft, automaton, wide;
    while (scanf("%d %d %d %d %d %d", &B, &V, &bytes, &draft, &automaton, &wide) == 6)
        printf("%d\n", fa_verify_blocks(B, V, bytes, draft != 0, automaton != 0, wide));
    return 0;
}
