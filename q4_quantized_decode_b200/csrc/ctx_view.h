// What the library's other sources see of a handle.
#pragma once

#include "../../include/q4gemv.h"

namespace q4 {

struct CtxView {
    int device, sms;
    bool fail_launch;     // fault injection: launches fail
    int* err;             // device error word
};

CtxView ctx_view(q4gemv_t h);
// Sets the handle's error text and returns `status`.
int ctx_fail(q4gemv_t h, int status, const char* text);

}  // namespace q4
