// Single-token attention over a paged cache: bf16 instantiations.
#include "decode.cuh"

namespace zyfa {
zyfa_status_t decode_bf16(decode::DecodeArgs& a, int D_qk, int nsm, int dev, uint8_t* ws, cudaStream_t stream) {
  return D_qk == 64    ? decode::launch<false, 64, 64>(a, nsm, dev, ws, stream)
         : D_qk == 128 ? decode::launch<false, 128, 128>(a, nsm, dev, ws, stream)
                       : decode::launch<false, 192, 128>(a, nsm, dev, ws, stream);
}
int decode_launches_bf16(decode::DecodeArgs& a, int D_qk, int nsm) {
  return D_qk == 64    ? decode::launches<false, 64, 64>(a, nsm)
         : D_qk == 128 ? decode::launches<false, 128, 128>(a, nsm)
                       : decode::launches<false, 192, 128>(a, nsm);
}
}  // namespace zyfa
