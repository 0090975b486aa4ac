// Attention over a cache of 4-bit numbers (pq1_kv4_attention): few rows, the join
// of a call's parts, and the choice between few rows and many.
#include "attn_few_rows.h"

namespace pq1 {

hipError_t launch_kv4_attention(const AttnPlan& plan, const AttnWindowArgs& a, int dtype, int out_dtype,
                                void* workspace, hipStream_t s) {
  const hipError_t e = plan.many
                           ? launch_kv4_many_rows(plan, a, dtype, out_dtype, workspace, s)
                           : launch_few_rows<kFourBit>(plan, a, dtype, out_dtype, workspace, s);
  if (e != hipSuccess || !plan.joined) return e;
  return join_parts<true>(plan, a, out_dtype, workspace, s);
}

}  // namespace pq1
