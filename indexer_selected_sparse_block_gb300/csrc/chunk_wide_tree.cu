// chunk_wide_tree.cu -- the attention kernel with 512 value dims of drafted trees.
#include "chunk_wide.cuh"

namespace sfa {
namespace chunk {

int launch_wide_tree(const Params &p, int dkq, int64_t n_cells, cudaStream_t st) {
    return launch_wide_any<true>(p, dkq, n_cells, st);
}

}  // namespace chunk
}  // namespace sfa
