// Paged attention of few rows: head dimension 64, TurboQuant-MSE keys.
#include "tq_paged_rows.cuh"

namespace tq {
template tq_status paged_rows_launch<64, false>(const PagedParams &, int, int, cudaStream_t);
}  // namespace tq
