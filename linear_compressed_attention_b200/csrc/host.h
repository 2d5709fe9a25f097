// Host state shared by the library's translation units (not part of the C ABI).
#pragma once

namespace edit {

// Adds one to the calling thread's edit_attn_kernel_launches().
void count_launch();
// SM count of the current device (148 when none is visible).
int device_sms();

}  // namespace edit
