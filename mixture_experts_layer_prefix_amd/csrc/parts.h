// Reads of a part of a buffer (a slab or a pair of slabs of K) through a buffer
// address, at a scalar offset that all lanes share and an offset of the lane's.
#pragma once
#include <stdint.h>

namespace moe {

// The scalar offset of part i of `parts` at byte `at` of n.  It never passes the
// length, which part i < parts must see to with `at`; from the last part on it is
// the length.  Then lanes read what lies before the end and zeros from there on,
// whether the address check takes the sum of both offsets or compares the lane's
// with what the scalar one leaves of the length: past the length it would leave
// less than none, which an unsigned difference takes for almost 4 GB.
constexpr uint32_t part_at(int i, int parts, uint32_t at, uint32_t n) { return i < parts ? at : n; }

}  // namespace moe
