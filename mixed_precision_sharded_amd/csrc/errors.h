// The calling thread's last error (adamw_last_error), kept in api.cpp and set
// by every entry point.
#pragma once

namespace mps {

// Records the message and returns `code`.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

// Clears the message and returns MPS_OK.
int ok();

}  // namespace mps
