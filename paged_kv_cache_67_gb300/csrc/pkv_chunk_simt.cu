// pkv_chunk_simt.cu -- the CUDA-core chunk attention's fp32 instances and its
// entry (pkv_chunk_simt.cuh has the kernel).
#include "pkv_chunk_simt.cuh"

namespace pkv {

pkv_status launch_chunk_simt_bf16(const ChunkArgs &a, int rows, cudaStream_t stream);
pkv_status launch_chunk_simt_f16(const ChunkArgs &a, int rows, cudaStream_t stream);

// rows: packed rows per CTA, 4, 16 or (head_dim up to 256) 64.
pkv_status launch_chunk_simt(const ChunkArgs &a, int rows, pkv_dtype dt, cudaStream_t stream) {
  switch (dt) {
    case PKV_F32: return launch_cs_dt<float>(a, rows, stream);
    case PKV_BF16: return launch_chunk_simt_bf16(a, rows, stream);
    case PKV_F16: return launch_chunk_simt_f16(a, rows, stream);
  }
  return PKV_ERR_INVALID_ARG;
}

}  // namespace pkv
