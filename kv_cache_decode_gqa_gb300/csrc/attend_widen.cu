// The kernels of attend_tc.cuh over fp8 and MXFP4 caches, whose rows are
// widened to f16.
#include "attend_tc.cuh"

namespace kvd {

cudaError_t launch_attend_widen(const TcParams &tp, bool one, cudaStream_t s) {
  if (tp.p.dtype == DT_MXFP4)
    return one ? launch_attend_t<DT_MXFP4, 128, 1>(tp, s)
               : launch_attend_t<DT_MXFP4, 128, 2>(tp, s);
  if (tp.p.dk == 64) return launch_attend_t<DT_FP8, 64, 2>(tp, s);
  return one ? launch_attend_t<DT_FP8, 128, 1>(tp, s)
             : launch_attend_t<DT_FP8, 128, 2>(tp, s);
}

}  // namespace kvd
