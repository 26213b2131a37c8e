// Compiled instances of the tcgen05 multi-token query kernel with modified
// scores and masks (Dh = 128; bf16 and fp16 K/V; page size 16 and 32).
#include "prefill_mod_tc.cuh"

namespace kvp {

cudaError_t launch_prefill_tc_mod(const DecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int dtype, int P,
                                  dim3 grid, cudaStream_t st) {
    if (dtype == KV_DTYPE_BF16)
        return P == 16 ? launch_prefill_mod_tc_inst<KV_DTYPE_BF16, 16>(p, tk, tv, grid, st)
                       : launch_prefill_mod_tc_inst<KV_DTYPE_BF16, 32>(p, tk, tv, grid, st);
    return P == 16 ? launch_prefill_mod_tc_inst<KV_DTYPE_F16, 16>(p, tk, tv, grid, st)
                   : launch_prefill_mod_tc_inst<KV_DTYPE_F16, 32>(p, tk, tv, grid, st);
}

}  // namespace kvp
