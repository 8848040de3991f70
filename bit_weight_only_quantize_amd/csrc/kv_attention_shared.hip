// Attention over the 4-bit cache for a prefix that the requests of a batch share: its
// keys are read once for the query rows of all of them.

#include "kv_attention.h"

namespace awq {

hipError_t attn_launch_shared(const KvAttn &p, int D, XType xt, const KvAttnPlan &pl, hipStream_t st) {
  return attn_launch<kShared>(p, 1, D, xt, pl, st);
}

}  // namespace awq
