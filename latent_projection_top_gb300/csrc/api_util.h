// What the C ABI's translation units share: the per-thread error message and
// the driver's tensor-map encoder.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "route.h"

namespace route {

// Sets the calling thread's message (route_last_error) and returns `st`.
route_status api_fail(route_status st, const char *fmt, ...);

// 2-D map of a 16-bit operand with rows of `inner` values, `ld` values
// apart, read in boxes of box_inner x box_outer with 128-byte swizzle; zeros
// outside.  `ptr` is 16-byte aligned and ld a multiple of 8.
route_status api_encode_operand(CUtensorMap *m, const void *ptr, bool fp16, uint64_t inner,
                                uint64_t outer, uint64_t ld, uint32_t box_inner,
                                uint32_t box_outer, const char *what);

// The same of `count` such matrices, `step` values apart (a multiple of 8), in
// boxes of one of them.
route_status api_encode_operands(CUtensorMap *m, const void *ptr, bool fp16, uint64_t inner, uint64_t outer,
                                 uint64_t count, uint64_t ld, uint64_t step, uint32_t box_inner,
                                 uint32_t box_outer, const char *what);

}  // namespace route
