// The many-row form of attention over what follows a shared prefix (kv_attend_rows.cuh).
#include "kv_attend_rows.cuh"

namespace moe {

cudaError_t launch_kv_attend_rows_suffix(const AttendArgs& a, const AttendMaps& maps, int shift, int sms, cudaStream_t stream) {
  return launch_rows<kSuffix>(a, maps, shift, sms, stream);
}

}  // namespace moe
