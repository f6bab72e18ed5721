// attention_d64.hip — attention_kernel.h for heads of 64 channels (a file each, so
// that they compile side by side).
#include "attention_kernel.h"

namespace w4a4 {

void launch_attention_64(const AttentionArgs& a, const AttentionCut& c, int front, int slot0, int slots, bool pair,
                         hipStream_t st) {
  launch_head_dim<64>(a, c, front, slot0, slots, pair, st);
}

}  // namespace w4a4
