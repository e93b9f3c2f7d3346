// Host-side services of the library's entry points: the thread's error
// message and the check of the current device.
#pragma once

namespace tg {

void set_error(const char* fmt, ...) __attribute__((format(printf, 1, 2)));
void clear_error();
// Strides above this (elements) are refused: no memory holds two such rows, and
// their products stay far inside 64 bits below it.
constexpr long long MOST_STRIDE = 1LL << 40;
// The launch grid's limit: threads in all fit 32 bits.
inline bool grid_fits(double workgroups, int threads) { return workgroups * threads <= 4294967295.0; }

// TGEMM_OK if the current device is a gfx950, else a TGEMM_E_* code (message set)
int current_device_ok();

}  // namespace tg
