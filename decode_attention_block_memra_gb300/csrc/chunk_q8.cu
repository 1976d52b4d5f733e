// Chunk attention over K in q8_0 (chunk_kernel.cuh).
#include "chunk_kernel.cuh"

namespace memra {

cudaError_t launch_chunk_q8(int D, int vf, const ChunkParams &p, cudaStream_t st) {
  return launch_chunk_formats<MEMRA_KV_Q8_0>(D, vf, p, st);
}

}  // namespace memra
