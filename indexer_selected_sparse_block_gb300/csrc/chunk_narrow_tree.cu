// chunk_narrow_tree.cu -- the attention kernel with 128- and 64-wide heads of drafted trees.
#include "chunk_narrow.cuh"

namespace sfa {
namespace chunk {

int launch_narrow_tree(const Params &p, int d, int64_t n_cells, cudaStream_t st) {
    return launch_narrow_any<true>(p, d, n_cells, st);
}

}  // namespace chunk
}  // namespace sfa
