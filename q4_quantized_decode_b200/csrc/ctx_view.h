// What the library's other sources see of a handle.
#pragma once

#include <cuda_runtime.h>

#include "../../include/q4gemv.h"

namespace q4 {

struct CtxView {
    int device, sms;
    bool fail_launch;     // fault injection: launches fail
    int* err;             // device error word
    float* attn_ws;       // pieces of units that several CTAs share, and their counts;
                          // the segments' states of the linear attention
    size_t attn_ws_bytes;
    int* attn_cnt;
};

// Device setup of the token-mixing kernels: shared-memory limits, and the
// bytes of attn_ws and attn_cnt on a device of `sms` SMs.
cudaError_t mix_setup();
void mix_workspace(int sms, size_t* ws_bytes, size_t* cnt_bytes);

CtxView ctx_view(q4gemv_t h);
// Sets the handle's error text and returns `status`.
int ctx_fail(q4gemv_t h, int status, const char* text);

}  // namespace q4
