// pkv_quant_decode_int4.cu -- the tensor-core decode's instances for int4 codes.
#include "pkv_quant_decode_mma.cuh"

namespace pkv {

pkv_status launch_quant_mma_int4(const QuantDecodeArgs &a, bool split, pkv_dtype dt, cudaStream_t stream) {
  return launch_qm_f<kInt4>(a, split, dt, stream);
}

}  // namespace pkv
