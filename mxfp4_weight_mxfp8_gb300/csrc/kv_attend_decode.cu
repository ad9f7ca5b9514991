// The decode form of a request's attention (kv_attend_decode.cuh).
#include "kv_attend_decode.cuh"

namespace moe {

cudaError_t launch_kv_attend_decode(const AttendArgs& a, const AttendMaps& maps, int tile, int shift, int sms, cudaStream_t stream) {
  return launch_decode<kWhole>(a, maps, tile, shift, sms, stream);
}

int kv_attend_decode_ctas(int head_dim, int tile, int sms) { return decode_ctas(head_dim, tile, sms); }

}  // namespace moe
