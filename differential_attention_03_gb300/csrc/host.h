// What the C entry points of the library share on the host: the thread's
// error message, the device status word, the launch counter and the TMA
// descriptor encoder.  Defined in api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "diffattn.h"

namespace da {
namespace host {

// Records the message of a non-OK status on this thread and returns the status.
diffattn_status error(diffattn_status s, const char* msg);
// Clears the message and returns DIFFATTN_OK.
diffattn_status success();
// Device address of the status word on the current device.
diffattn_status status_address(int** out);
// SMs of the current device (0 if unknown).
int sms();
// Adds `k` to diffattn_launch_count().
void count_launches(int k);

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
diffattn_status encoder(EncodeTiled* fn);

}  // namespace host
}  // namespace da
