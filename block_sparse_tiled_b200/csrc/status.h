// Error reporting shared by the library's translation units.
#pragma once
#include "vsa.h"

namespace vsa {

// Sets the calling thread's error message (vsa_last_error) and returns `s`.  Never throws.
__attribute__((visibility("hidden"))) vsa_status set_error(vsa_status s, const char* format, ...) noexcept
    __attribute__((format(printf, 2, 3)));

}  // namespace vsa
