// Host-side check of the register hand-over's condition, compiled and run by
// tests/test_register_split.py: prints split_fits for the splits and launch register
// counts given as "few many groups regs" lines. No device code runs.
#include <cuda_runtime.h>
#include <stdio.h>

#include "../sparse_moe_transformer_gemm_b200/csrc/tc.cuh"

int main() {
    moe::tc::RegSplit s;
    int regs;
    while (scanf("%d %d %d %d", &s.few, &s.many, &s.groups, &regs) == 4)
        printf("%d\n", (int)moe::tc::split_fits(s, regs));
    return 0;
}
