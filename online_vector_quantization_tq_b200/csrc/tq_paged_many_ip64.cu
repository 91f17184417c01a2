// Paged attention of many rows: head dimension 64, inner-product keys.
#include "tq_paged_tiles.cuh"

namespace tq {
template tq_status paged_tiles_launch<64, true>(const PagedParams &, int, int, cudaStream_t);
}  // namespace tq
