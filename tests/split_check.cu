// Host-side check of the K-split rule, compiled and run by tests/test_split_rule.py:
// prints slices_of for "tiles blocks sms" lines. No device code runs.
#include <stdio.h>

#include "../sparse_moe_transformer_gemm_b200/csrc/block_tile.cuh"

int main() {
    long tiles;
    int blocks, sms;
    while (scanf("%ld %d %d", &tiles, &blocks, &sms) == 3)
        printf("%d\n", moe::block::slices_of(tiles, blocks, sms));
    return 0;
}
