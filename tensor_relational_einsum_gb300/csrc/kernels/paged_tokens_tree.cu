// paged_tokens_tree.cu -- the token kernel over the nodes of trees.
#include "paged_tokens.cuh"

namespace ea {

cudaError_t launch_cache_tokens_tree(const PgAttn &p, const PgPlan &pl, const PgWork &w, bool early, cudaStream_t st) {
    return launch_tokens<true>(p, pl, w, early, st);
}

}  // namespace ea
