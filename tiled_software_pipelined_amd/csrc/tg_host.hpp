// Host-side services of the library's entry points: the thread's error
// message and the check of the current device.
#pragma once

namespace tg {

void set_error(const char* fmt, ...) __attribute__((format(printf, 1, 2)));
void clear_error();
// TGEMM_OK if the current device is a gfx950, else a TGEMM_E_* code (message set)
int current_device_ok();

}  // namespace tg
