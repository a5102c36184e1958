// pkv_chunk_simt_bf16.cu -- the CUDA-core chunk attention's bf16 instances
// (pkv_chunk_simt.cuh has the kernel; a file per type, so that they compile
// side by side).
#include "pkv_chunk_simt.cuh"

namespace pkv {

pkv_status launch_chunk_simt_bf16(const ChunkArgs &a, int rows, cudaStream_t stream) {
  return launch_cs_dt<__nv_bfloat16>(a, rows, stream);
}

}  // namespace pkv
