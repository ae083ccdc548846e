// Tensor-core attention over mxfp4 and nvfp4 pages (cache_attend_tc.cuh).
#include "cache_attend_tc.cuh"

namespace mxq {
namespace attend {

int tc_mxfp4(const Args& a, int dt, int64_t units, int* grid, cudaStream_t st) {
  if (a.c.dim == 64) return launch_tc_dt<MXQ_FMT_MXFP4, 64, 2>(a, dt, units, grid, st);
  if (a.c.dim == 128) return launch_tc_dt<MXQ_FMT_MXFP4, 128, 4>(a, dt, units, grid, st);
  return launch_tc_dt<MXQ_FMT_MXFP4, 256, 8>(a, dt, units, grid, st);
}

int tc_nvfp4(const Args& a, int dt, int64_t units, int* grid, cudaStream_t st) {
  if (a.c.dim == 64) return launch_tc_dt<MXQ_FMT_NVFP4, 64, 4>(a, dt, units, grid, st);
  if (a.c.dim == 128) return launch_tc_dt<MXQ_FMT_NVFP4, 128, 8>(a, dt, units, grid, st);
  return launch_tc_dt<MXQ_FMT_NVFP4, 256, 16>(a, dt, units, grid, st);
}

}  // namespace attend

MXQ_DEFINE_CHECK_READER(check_record_attend_fp4)

}  // namespace mxq
