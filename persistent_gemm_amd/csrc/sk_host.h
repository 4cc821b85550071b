// Host-side helpers of sk_api.cpp that the block-scaled and norm entry points (sk_api_block.cpp) share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <mutex>

#include "../../include/sk_gemm.h"

namespace sk {
namespace host {

// The current device, which must be a gfx950, and the compute units kernels on `stream` may use.
sk_status device_for(hipStream_t stream, int* dev, int* cus);
// SK_ERR_UNSUPPORTED while the stream is being captured: the calls that use the library's scratch.
sk_status refuse_capture(hipStream_t stream);
// The scratch of (device, stream) that one call's kernels share, grown to `bytes`.  It is the call's own while it keeps
// *hold, to be kept until its last launch: other host threads' calls on the stream, and the release of its scratch, wait.
using Hold = std::unique_lock<std::recursive_mutex>;
sk_status scratch(int dev, hipStream_t stream, size_t bytes, Hold* hold, uint8_t** out);
// Whether [a, a + na) and [b, b + nb) share a byte; absent (NULL) ranges share none.
bool overlaps(const void* a, int64_t na, const void* b, int64_t nb);

}  // namespace host
}  // namespace sk
