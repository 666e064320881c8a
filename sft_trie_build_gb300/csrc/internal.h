// Internal helpers shared by the translation units of libstp.so.
#pragma once

#include <cstdarg>
#include <cstdint>

#include "stp.h"

namespace stp {

// Records a printf-style message as the thread's last error and returns `code`.
stp_status fail(stp_status code, const char* fmt, ...);

// Clears the thread's last error.
void clear_error();

// Validates an attention descriptor (records the reason and returns its code).
stp_status check_desc(const stp_attn_desc* d);

// Validates the window and the number of visible first tokens of windowed attention.
stp_status check_window(int32_t window, int32_t n_sink);

// Positions lie below 2^30: a window of that size hides nothing.
inline int32_t clip_window(int32_t window) { return window < (1 << 30) ? window : (1 << 30); }

}  // namespace stp
