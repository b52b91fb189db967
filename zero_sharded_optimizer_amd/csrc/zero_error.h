// The calling thread's error message, shared by the ABI's translation units.
#pragma once

#include "zero_adam.h"

namespace zerror {

// Sets the message that zero_last_error() returns and passes `st` through.
zero_status fail(zero_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears it.
zero_status ok();

}  // namespace zerror
