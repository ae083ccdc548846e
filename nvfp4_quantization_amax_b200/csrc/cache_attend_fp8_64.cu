// Tensor-core attention over fp8 pages, head size 64 (cache_attend_tc.cuh).
#include "cache_attend_tc.cuh"

namespace mxq {
namespace attend {

int tc_fp8_64(const Args& a, int dt, int nb, int64_t units, int* grid, cudaStream_t st) {
  switch (nb) {
    case 1: return launch_tc_dt<MXQ_FMT_FP8, 64, 1>(a, dt, units, grid, st);
    default: return launch_tc_dt<MXQ_FMT_FP8, 64, 2>(a, dt, units, grid, st);
  }
}

}  // namespace attend

MXQ_DEFINE_CHECK_READER(check_record_attend_fp8_64)

}  // namespace mxq
