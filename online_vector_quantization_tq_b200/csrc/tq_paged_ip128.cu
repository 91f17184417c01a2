// Paged attention of few rows: head dimension 128, inner-product keys.
#include "tq_paged_rows.cuh"

namespace tq {
template tq_status paged_rows_launch<128, true>(const PagedParams &, int, int, cudaStream_t);
}  // namespace tq
