// pkv_chunk_simt_f16.cu -- the CUDA-core chunk attention's fp16 instances
// (pkv_chunk_simt.cuh has the kernel; a file per type, so that they compile
// side by side).
#include "pkv_chunk_simt.cuh"

namespace pkv {

pkv_status launch_chunk_simt_f16(const ChunkArgs &a, int rows, cudaStream_t stream) {
  return launch_cs_dt<__half>(a, rows, stream);
}

}  // namespace pkv
