// The products grouped by expert (sk_grouped.h) of bf16 rows.
#include "sk_grouped.h"

namespace sk {
hipError_t launch_grouped_bf16(const GroupedGemm& g, int kind, int cus, hipStream_t s) {
  return launch_grouped_of<Bf16>(g, kind, cus, s);
}
}  // namespace sk
