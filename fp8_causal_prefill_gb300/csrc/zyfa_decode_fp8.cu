// Single-token attention over a paged cache: e4m3 instantiations.
#include "decode.cuh"

namespace zyfa {
zyfa_status_t decode_fp8(decode::DecodeArgs& a, int D_qk, int nsm, int dev, uint8_t* ws, cudaStream_t stream) {
  return D_qk == 64    ? decode::launch<true, 64, 64>(a, nsm, dev, ws, stream)
         : D_qk == 128 ? decode::launch<true, 128, 128>(a, nsm, dev, ws, stream)
                       : decode::launch<true, 192, 128>(a, nsm, dev, ws, stream);
}
int decode_launches_fp8(decode::DecodeArgs& a, int D_qk, int nsm) {
  return D_qk == 64    ? decode::launches<true, 64, 64>(a, nsm)
         : D_qk == 128 ? decode::launches<true, 128, 128>(a, nsm)
                       : decode::launches<true, 192, 128>(a, nsm);
}
}  // namespace zyfa
