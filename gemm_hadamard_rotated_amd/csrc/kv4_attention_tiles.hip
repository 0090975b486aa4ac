// Attention over a cache of 4-bit numbers for many rows (attn_many_rows.h).
#include "attn_many_rows.h"

namespace pq1 {

hipError_t launch_kv4_many_rows(const AttnPlan& plan, const AttnWindowArgs& a, int dtype, int out_dtype,
                                void* workspace, hipStream_t s) {
  return launch_types<kFourBit>(plan, a, dtype, out_dtype, workspace, s);
}

}  // namespace pq1
