// The decode-step kernel of tq_paged_attend at d = 64 (paged_rows.cuh).
#include "paged_rows.cuh"

namespace tq {
tq_status paged_rows_launch_64(const PagedAttendParams& p, int kb, int vb, bool alg2, int ctas, cudaStream_t st) {
  return launch_row_keys<64>(p, kb, vb, alg2, ctas, st);
}
}  // namespace tq
