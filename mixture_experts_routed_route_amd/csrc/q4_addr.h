// Where the lanes of a wave read a strip of 16 rows of 4-bit weights: offsets from
// the strip's first row, in a buffer whose descriptor ends with the strip's last byte.
// Plain constant expressions, so that a host program can walk over them.
//
// A load gets its place in two parts: v, a lane's own, which the descriptor's range is
// checked against word by word (words behind the end read as zeros, without an access),
// and s, the same for all lanes, which no check need count. So s is only used where a
// load stays inside its own row whatever s is; a load that may pass its row's end
// carries the whole place in v.
#pragma once

#include <cstdint>

namespace moe {

struct LoadAt { uint32_t v, s; };

// a lane's offset past every descriptor's end, also with a place in a row added
constexpr uint32_t kPastEnd = 0x80000000u;

// Codes: lane l has piece l & 3 (32 codes, 16 bytes) of row l >> 2 of a block; rb bytes
// a row, a multiple of 16. Short last blocks (not whole) have pieces behind the row.
constexpr uint32_t codes_start(uint32_t lane, uint32_t rb) { return (lane >> 2) * rb + (lane & 3) * 16u; }
constexpr LoadAt codes_at(uint32_t start, int kb, bool whole) {
  return whole ? LoadAt{start, (uint32_t)kb * 64u} : LoadAt{start + (uint32_t)kb * 64u, 0u};
}

// Parameters of one block: lane l < 16 has row l's, `per` bytes (8, or 16 for groups of
// 32 with a bias); pb bytes a row.
constexpr uint32_t params_start(uint32_t lane, uint32_t pb) { return lane < 16 ? lane * pb : kPastEnd; }
constexpr LoadAt params_at(uint32_t start, int kb, uint32_t per, bool whole) {
  return whole ? LoadAt{start, (uint32_t)kb * per} : LoadAt{start + (uint32_t)kb * per, 0u};
}

// Parameters of a run of blocks, 64 bytes a row: lane 4 r + q has 16 bytes of row r. A
// run starts at any block and so may pass the row's end, as may two blocks of 8 bytes
// asked for at once, the second behind the row.
constexpr uint32_t run_start(uint32_t lane, uint32_t pb) { return (lane >> 2) * pb + (lane & 3) * 16u; }
constexpr LoadAt run_at(uint32_t start, int kb, uint32_t per) {
  return {start + (uint32_t)kb * per, 0u};
}

}  // namespace moe
