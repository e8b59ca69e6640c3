// fp8_stage.hpp -- where the bytes of a tile's stage come from, for the product in 8 bits: plain arithmetic, for device and host.
#pragma once

#include <stdint.h>

namespace lora {

constexpr int kFp8Block = 128;  // columns of a scale and of a stage, and rows of a weight's scale

// The column, from the stage's first, of the 16 codes that slot `slot` of the tile's row r holds.
constexpr uint32_t stage_chunk(uint32_t r, uint32_t slot) { return (slot ^ ((r >> 1) & 7)) * 16; }

// The same where the stage begins at column k0 of rows of k codes: codes at
// or past k are not there, and the row's first of the stage stand in for them,
// to be zeroed once they have landed.  A transfer's checked offset carries its
// row and this column but not k0, which goes in beside it and may not count
// into the check; no column past k may hang on that.
constexpr uint32_t stage_column(uint32_t chunk, uint32_t k0, uint32_t k) { return k0 + chunk < k ? chunk : 0; }

}  // namespace lora
