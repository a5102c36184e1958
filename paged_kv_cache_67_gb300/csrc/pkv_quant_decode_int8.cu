// pkv_quant_decode_int8.cu -- the tensor-core decode's instances for int8 codes.
#include "pkv_quant_decode_mma.cuh"

namespace pkv {

pkv_status launch_quant_mma_int8(const QuantDecodeArgs &a, bool split, pkv_dtype dt, cudaStream_t stream) {
  return launch_qm_f<kInt8>(a, split, dt, stream);
}

}  // namespace pkv
