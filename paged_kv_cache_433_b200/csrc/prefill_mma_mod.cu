// Compiled warp-MMA instances of the multi-token query with modified scores
// and masks (the shapes that the tcgen05 kernel does not take).
#include "decode_launch.cuh"

namespace kvp {

cudaError_t launch_prefill_mod(const DecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int dtype, int DH,
                               int P, dim3 grid, cudaStream_t st) {
    return dtype == KV_DTYPE_BF16 ? launch_prefill_dt<KV_DTYPE_BF16, true>(p, tk, tv, DH, P, grid, st)
                                  : launch_prefill_dt<KV_DTYPE_F16, true>(p, tk, tv, DH, P, grid, st);
}

}  // namespace kvp
