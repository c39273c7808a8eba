// kvq_tree_16.cu -- the tree attention kernel (kvq_tree.cuh) for caches of 16
// bits.  One unit a width: a kernel then holds the code of one width only,
// which its instruction fetch notices (one node over 4-bit tokens: 141 -> 124 us).
#include "kvq_tree.cuh"

namespace kvq {
template cudaError_t launch_tree_bits<16>(const TreePlan& p, cudaStream_t s);
}  // namespace kvq
