// Attention in windows whose first keys stay visible, for many rows
// (attn_many_rows.h).
//
// Prompts of 500 to 6000 tokens in a window of 1024 with 16 first keys, 6 query heads to
// each of 4 cache heads, D = 256: 403 to 412 us, 809 to 827 TFLOP/s of what rows see.  A tile of 43
// tokens walks over 34 key tiles, of which 6 are edges (masks 1 % of the time, taking
// invisible values out of V 4 %); the rest of what keeps it from the 990 of long chunks
// is a workgroup's beginning and end, which nothing overlaps with one workgroup to a CU,
// and the last of 5.6 rounds of workgroups.  The barrier after taking values out moved
// past the scores: 427 us for 429, but 889 for 885 where windows hold all keys.
#include "attn_many_rows.h"

namespace pq1 {

hipError_t launch_sinks_many_rows(const AttnPlan& plan, const AttnWindowArgs& a, int dtype, int out_dtype,
                                  void* workspace, hipStream_t s) {
  return launch_types<kTwoByteSinks>(plan, a, dtype, out_dtype, workspace, s);
}

}  // namespace pq1
