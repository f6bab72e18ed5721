// attention_d128.hip — attention_kernel.h for heads of 128 channels (a file each, so
// that they compile side by side).
#include "attention_kernel.h"

namespace w4a4 {

void launch_attention_128(const AttentionArgs& a, const AttentionPlan& plan, bool pair, hipStream_t st) {
  launch_head_dim<128>(a, plan, pair, st);
}

}  // namespace w4a4
