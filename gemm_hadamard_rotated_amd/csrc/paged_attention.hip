// Attention of new tokens over a paged key/value cache (pq1_paged_attention): few
// rows (attn_few_rows.h), and the choice between those and many.
#include "attn_few_rows.h"

namespace pq1 {

hipError_t launch_attention(const AttnPlan& plan, const AttnArgs& a, int dtype, int out_dtype,
                            void* workspace, hipStream_t s) {
  const hipError_t e = plan.many
                           ? launch_many_rows(plan, a, dtype, out_dtype, workspace, s)
                           : launch_few_rows<kTwoByte>(plan, a, dtype, out_dtype, workspace, s);
  if (e != hipSuccess || plan.nsplit == 1) return e;
  return join_parts<false>(plan, a, out_dtype, workspace, s);
}

}  // namespace pq1
