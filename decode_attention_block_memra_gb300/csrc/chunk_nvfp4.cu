// Chunk attention over K in NVFP4 (chunk_kernel.cuh).
#include "chunk_kernel.cuh"

namespace memra {

cudaError_t launch_chunk_nvfp4(int D, int vf, const ChunkParams &p, cudaStream_t st) {
  return launch_chunk_formats<MEMRA_KV_NVFP4>(D, vf, p, st);
}

}  // namespace memra
