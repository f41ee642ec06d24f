// The decode-step kernel of tq_paged_attend at d = 128 (paged_rows.cuh).
#include "paged_rows.cuh"

namespace tq {
tq_status paged_rows_launch_128(const PagedAttendParams& p, int kb, int vb, bool alg2, int ctas, cudaStream_t st) {
  return launch_row_keys<128>(p, kb, vb, alg2, ctas, st);
}
}  // namespace tq
