// The many-row form of a request's attention (kv_attend_rows.cuh).
#include "kv_attend_rows.cuh"

namespace moe {

cudaError_t launch_kv_attend_rows(const AttendArgs& a, const AttendMaps& maps, int shift, int sms, cudaStream_t stream) {
  return launch_rows<kWhole>(a, maps, shift, sms, stream);
}

int kv_attend_rows_ctas(int sms) { return rows_ctas(sms); }

}  // namespace moe
