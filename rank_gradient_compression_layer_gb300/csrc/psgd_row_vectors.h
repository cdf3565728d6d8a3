// Rows of any width, one behind the other, in vectors of eight values that start
// at multiples of eight of the row-major order: which vectors a row lies in, and
// which of them end behind the tensor.
#pragma once

#include <stdint.h>

namespace psgd {

// Where a row starts in its first vector.
constexpr int first_offset(int64_t row, int width) { return (int)(row * width & 7); }

// Vectors of a row that starts at value `off` of its first one.
constexpr int vectors_of(int off, int width) { return (off + width + 7) / 8; }

// The first row whose last vector ends behind the last of `rows` rows: row r does
// where it reaches past the whole vectors' n values, (r + 1) width > n.  Of rows of
// eight values or more that is the last row at most, of shorter ones as many as share
// the tensor's last vector.
constexpr int64_t first_ragged(int64_t rows, int width) { return rows * width / 8 * 8 / width; }

}  // namespace psgd
