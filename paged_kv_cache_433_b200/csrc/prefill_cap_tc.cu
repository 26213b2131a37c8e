// Compiled instances of the tcgen05 multi-token query kernel for capped scores (bf16, Dh = 128; page size 16 and 32).
#include "prefill_cap_tc.cuh"

namespace kvp {

cudaError_t launch_prefill_cap_tc(const DecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int P, int n_tiles,
                                  cudaStream_t st) {
    return P == 16 ? launch_prefill_cap_tc_inst<16>(p, tk, tv, n_tiles, st)
                   : launch_prefill_cap_tc_inst<32>(p, tk, tv, n_tiles, st);
}

}  // namespace kvp
