// block_gemm.cu -- FP8 (e4m3) matrix products with an fp32 scale per block of
// 128, dense or grouped by row offsets, and the SwiGLU gate_up form whose
// result is quantised again: which kernel takes a call, and the host parts.
//
//   out[m, n] = sum_b sx[m, b] sw[n / 128, b] sum_{c in block b} xq[m, c] wq[n, c]
//   gate_up:  h = SiLU(g) u in fp32, hq / sh its quantisation per 128 features
//
// The kernels let the tensor core sum one block of 128 columns at a time into TMEM
// and add it, scaled, to fp32 registers. They differ in what the MMA's rows are:
// weight rows with up to 128 tokens as its columns, on pairs of SMs (block_few.cu);
// tokens with 256 weight rows as its columns, on pairs (block_many.cu); or weight
// rows on single SMs that share the columns of K (block_split.cu), for one product
// that is too small to give every pair a tile.
#include "block_tile.cuh"

namespace moe {
namespace block {

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault,
                                                &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
    }();
    return fn;
}

}  // namespace

bool make_byte_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols,
                   uint32_t box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {cols};
    cuuint32_t box[2] = {(cuuint32_t)BK, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_token_byte_maps(TokenMaps* tm, const void* base, uint64_t rows, uint64_t cols,
                          int boxes) {
    for (int lg = 0; lg < boxes; ++lg)
        if (!make_byte_map(&tm->m[lg], base, rows, cols, NBOX << lg)) return false;
    return true;
}

cudaError_t allow_smem(const void* kernel, int smem, std::atomic<uint64_t>& done,
                       const tc::RegSplit& split) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    cudaFuncAttributes attr;
    err = cudaFuncGetAttributes(&attr, kernel);
    if (err != cudaSuccess) return err;
    if (!tc::split_fits(split, attr.numRegs)) return cudaErrorLaunchOutOfResources;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return err;
}

int sm_pairs() {
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return (n > 1 ? n : 148) / 2;
}

namespace {

// The weight rows in the MMA's M up to so many rows a group on average: most groups
// then have one tile of at most 128 tokens, so that each weight is read once.
// Measured, Hy3 experts, both kernels' layer: 85 rows 726 us against 1041, 125
// rows 1126 against 1130, 171 rows 1618 against 1172. One product whose rows are
// known: up to the 128 of a tile.
constexpr long kFewRows = 112;
bool few(const BlockGemm& p) {
    return (long)p.M <= kFewRows * p.G || (!p.offsets && p.M <= 128);
}

}  // namespace
}  // namespace block

cudaError_t launch_block_gemm(const BlockGemm& p, cudaStream_t s) {
    if (block::splits(p)) return block::launch_split(p, s);
    return block::few(p) ? block::launch_few(p, false, s) : block::launch_many(p, false, s);
}
cudaError_t launch_block_gate_up(const BlockGemm& p, cudaStream_t s) {
    return block::few(p) ? block::launch_few(p, true, s) : block::launch_many(p, true, s);
}

}  // namespace moe
