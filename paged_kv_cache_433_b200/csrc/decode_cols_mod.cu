// Compiled heads-as-columns decode instances with modified scores and masks.
#include "decode_cols.cuh"

namespace kvp {

cudaError_t launch_cols_mod(const DecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int dtype, int DH, int P,
                            dim3 grid, cudaStream_t st) {
    return dtype == KV_DTYPE_BF16 ? launch_cols_dt<KV_DTYPE_BF16, KV_DTYPE_BF16, true>(p, tk, tv, DH, P, grid, st)
                                  : launch_cols_dt<KV_DTYPE_F16, KV_DTYPE_F16, true>(p, tk, tv, DH, P, grid, st);
}

}  // namespace kvp
