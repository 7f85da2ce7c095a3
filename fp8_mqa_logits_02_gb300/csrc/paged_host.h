// What the library's two host files know of each other.
#pragma once

#include <cuda.h>

#include <cstdint>

namespace fp8mqa {

// The limit of one on-device wait (fp8_mqa_logits_set_wait_limit_ns).
uint64_t wait_limit_ns();

// A tensor map of `rows` rows of 128 bytes, `pitch` bytes apart, in boxes of `box` rows under the
// 128-byte swizzle; false if the driver does not take it.
bool encode_rows128(CUtensorMap* map, const void* base, uint64_t rows, uint64_t pitch, uint32_t box);

// Reads and clears the paged kernels' status word on device `dev` into *flags, after the caller
// has synchronized; false if a read failed.  Allocates nothing.
bool paged_take_status(int dev, int32_t* flags);

}  // namespace fp8mqa
