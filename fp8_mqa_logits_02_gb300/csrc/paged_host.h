// What the library's two host files know of each other.
#pragma once

#include <cstdint>

namespace fp8mqa {

// The limit of one on-device wait (fp8_mqa_logits_set_wait_limit_ns).
uint64_t wait_limit_ns();

// Reads and clears the paged kernels' status word on device `dev` into *flags, after the caller
// has synchronized; false if a read failed.  Allocates nothing.
bool paged_take_status(int dev, int32_t* flags);

}  // namespace fp8mqa
