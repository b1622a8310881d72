// attn.cu -- attention of packed prompts (attn_prompt) and of drafted token
// trees over a paged cache (attn_tree): launches of attn_kernel.cuh.
#include "attn_kernel.cuh"

namespace mxg {

cudaError_t launch_attn_prompt(const AttnParams &p, int sm_count, cudaStream_t stream) {
  return p.D == 64 ? launch_t<64, kPrompt>(p, sm_count, stream) : launch_t<128, kPrompt>(p, sm_count, stream);
}
cudaError_t launch_attn_tree(const AttnParams &tree, int sm_count, cudaStream_t stream) {
  AttnParams p = tree;
  p.slots = kJoinFloats;
  const cudaError_t e = p.D == 64 ? launch_t<64, kTree>(p, sm_count, stream) : launch_t<128, kTree>(p, sm_count, stream);
  if (e != cudaSuccess) return e;
  return p.D == 64 ? launch_join<64, kTree>(p, sm_count, stream) : launch_join<128, kTree>(p, sm_count, stream);
}
size_t attn_tree_ws_bytes(int D, int sm_count) {
  const long long f = D == 64 ? Cfg<64, kTree>::kSlotFloats : Cfg<128, kTree>::kSlotFloats;
  return (size_t)(kJoinFloats + 2 * f * (sm_count < kMaxCtas ? sm_count : kMaxCtas)) * sizeof(float);
}

}  // namespace mxg
