// Attention in windows whose first keys stay visible, for many rows
// (attn_many_rows.h).
#include "attn_many_rows.h"

namespace pq1 {

hipError_t launch_sinks_many_rows(const AttnPlan& plan, const AttnWindowArgs& a, int dtype, int out_dtype,
                                  void* workspace, hipStream_t s) {
  return launch_types<kTwoByteSinks>(plan, a, dtype, out_dtype, workspace, s);
}

}  // namespace pq1
