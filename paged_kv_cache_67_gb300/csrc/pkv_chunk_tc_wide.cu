// pkv_chunk_tc_wide.cu -- the tcgen05 chunk attention's instances for head_dim
// 192 and 256 (pkv_chunk_tc.cuh has the kernel, pkv_chunk_tc.cu its callers).
#include "pkv_chunk_tc.cuh"

namespace pkv {

pkv_status launch_chunk_tc_wide(const CtArgs &a, pkv_dtype dt, const CUtensorMap &mq, const CUtensorMap &mk,
                                const CUtensorMap &mv, int sms, cudaStream_t stream) {
  switch (a.c.D) {
    case 192: return launch_ct_dt<192>(a, dt, mq, mk, mv, sms, stream);
    case 256: return launch_ct_dt<256>(a, dt, mq, mk, mv, sms, stream);
  }
  return PKV_ERR_UNSUPPORTED;
}

}  // namespace pkv
