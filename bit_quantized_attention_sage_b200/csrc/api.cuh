// api.cuh -- what the C ABI's source files share.
#pragma once

#include <cuda.h>

#include <cstdint>

namespace sage {

// The current device's status word pair after its one-time set-up (null: the
// set-up failed).
int* api_status_word();
// Budget of a bounded device wait, SM clock cycles.
long long api_wait_budget();
// TMA map over uint8 [tiles][rows][D], boxes of box_rows rows, D-byte swizzle.
bool api_tile_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t tiles, uint32_t D,
                  uint32_t box_rows);

}  // namespace sage
