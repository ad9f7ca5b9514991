// The many-row form of attention over a shared prefix (kv_attend_rows.cuh).
#include "kv_attend_rows.cuh"

namespace moe {

cudaError_t launch_kv_attend_rows_prefix(const AttendArgs& a, const AttendMaps& maps, int shift, int sms, cudaStream_t stream) {
  return launch_rows<kPrefix>(a, maps, shift, sms, stream);
}

}  // namespace moe
