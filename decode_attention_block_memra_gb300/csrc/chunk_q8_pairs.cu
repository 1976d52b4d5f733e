// Chunk attention over K in q8_0 as exact pairs (chunk_kernel.cuh).
#include "chunk_kernel.cuh"

namespace memra {

cudaError_t launch_chunk_q8_pairs(int D, int vf, const ChunkParams &p, cudaStream_t st) {
  return launch_chunk_formats<MEMRA_KV_Q8_0, true>(D, vf, p, st);
}

}  // namespace memra
