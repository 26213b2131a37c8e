// Compiled heads-as-columns decode instances for int8 K/V (q in bf16 or fp16).
#include "decode_cols.cuh"

namespace kvp {

cudaError_t launch_cols_int8(const DecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int q_dtype, int DH,
                             int P, dim3 grid, cudaStream_t st) {
    return q_dtype == KV_DTYPE_BF16 ? launch_cols_dt<KV_DTYPE_INT8, KV_DTYPE_BF16, false>(p, tk, tv, DH, P, grid, st)
                                    : launch_cols_dt<KV_DTYPE_INT8, KV_DTYPE_F16, false>(p, tk, tv, DH, P, grid, st);
}

}  // namespace kvp
