// paged_chunks_tree.cu -- the chunk kernel over the nodes of trees.
#include "paged_chunks.cuh"

namespace ea {

cudaError_t launch_cache_chunks_tree(const PgAttn &p, const PgPlan &pl, const PgMaps &maps, const PgWork &w, bool early,
                                     cudaStream_t st) {
    return launch_chunks<true>(p, pl, maps, w, early, st);
}

}  // namespace ea
