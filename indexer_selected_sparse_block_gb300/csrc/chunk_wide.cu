// chunk_wide.cu -- the attention kernel with 512 value dims of chunks.
#include "chunk_wide.cuh"

namespace sfa {
namespace chunk {

int launch_wide(const Params &p, int dkq, int64_t n_cells, cudaStream_t st) {
    return launch_wide_any<false>(p, dkq, n_cells, st);
}

}  // namespace chunk
}  // namespace sfa
