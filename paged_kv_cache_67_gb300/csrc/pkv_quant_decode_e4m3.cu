// pkv_quant_decode_e4m3.cu -- the tensor-core decode's instances for e4m3 codes.
#include "pkv_quant_decode_mma.cuh"

namespace pkv {

pkv_status launch_quant_mma_e4m3(const QuantDecodeArgs &a, bool split, pkv_dtype dt, cudaStream_t stream) {
  return launch_qm_f<kE4m3>(a, split, dt, stream);
}

}  // namespace pkv
