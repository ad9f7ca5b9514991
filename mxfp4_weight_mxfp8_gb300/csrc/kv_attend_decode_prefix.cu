// The decode form of attention over a shared prefix (kv_attend_decode.cuh).
#include "kv_attend_decode.cuh"

namespace moe {

cudaError_t launch_kv_attend_decode_prefix(const AttendArgs& a, const AttendMaps& maps, int tile, int shift, int sms, cudaStream_t stream) {
  return launch_decode<kPrefix>(a, maps, tile, shift, sms, stream);
}

}  // namespace moe
