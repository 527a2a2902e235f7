// Low-rank adapters, forward (adapters.h).
#include "adapters.h"

namespace moe {

hipError_t launch_adapters_forward(const AdapterArgs& A, bool y_f32, int cus, hipStream_t s, const KTime& kt) {
  return y_f32 ? adapters_rows_any<false, true>(A, cus, s, kt.start, kt.stop)
               : adapters_rows_any<false, false>(A, cus, s, kt.start, kt.stop);
}

}  // namespace moe
