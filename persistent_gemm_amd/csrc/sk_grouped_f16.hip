// The products grouped by expert (sk_grouped.h) of fp16 rows.
#include "sk_grouped.h"

namespace sk {
hipError_t launch_grouped_f16(const GroupedGemm& g, int kind, int cus, hipStream_t s) {
  return launch_grouped_of<Fp16>(g, kind, cus, s);
}
}  // namespace sk
