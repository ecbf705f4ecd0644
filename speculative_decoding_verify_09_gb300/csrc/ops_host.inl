// Host helpers shared by the operators' C entries (defined in api.cu): the
// thread-local error text behind sv_last_error().
#pragma once

#include <stdint.h>

#include "spec_verify.h"

namespace sv {

// Records the message of a failed call and returns its status.
sv_status record_error(sv_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));

// SMs of the current device (0 if it cannot be asked).
int device_sms();

inline bool is_aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace sv
