// Host check of the number of blocks that share a sequence's verification (fa_verify_blocks in csrc/fa_verify_blocks.cuh, the function
// fa_verify calls): reads lines "B V wide", prints the number for each.
#include <cstdio>

#include "../constrained_decoding_diffusion_gb300/csrc/fa_verify_blocks.cuh"

int main() {
    int B, V, wide;
    while (scanf("%d %d %d", &B, &V, &wide) == 3) printf("%d\n", fa_verify_blocks(B, V, wide));
    return 0;
}
