// The wide attention kernel of rows that each read their own entries (sv_attend_wide.cuh).

#include "sv_attend_wide.cuh"

namespace sv {

int launch_attend_wide(const AttendParams& P, bool f16, const CUtensorMap& k, const CUtensorMap& v,
                       const CUtensorMap& q, int q_tokens, int grid, cudaStream_t st) {
  return f16 ? launch_type<true, false>(P, k, v, q, q_tokens, grid, st) : launch_type<false, false>(P, k, v, q, q_tokens, grid, st);
}

}  // namespace sv
