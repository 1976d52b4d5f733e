// Chunk attention over K in fp8 (chunk_kernel.cuh).
#include "chunk_kernel.cuh"

namespace memra {

cudaError_t launch_chunk_fp8(int D, int vf, const ChunkParams &p, cudaStream_t st) {
  return launch_chunk_formats<MEMRA_KV_FP8_E4M3>(D, vf, p, st);
}

}  // namespace memra
