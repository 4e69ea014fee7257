// Where the keys of a 16-key group lie, as plain C++ that host and device
// compile alike.
//
// Keys are read in shares of ROWS (8 or 16) whose first key g is a multiple
// of ROWS; with pages of whole 16-key groups a group lies in one page, so a
// share's rows stand at row * stride from its first one.  Keys outside the
// span [lo, hi) that the rows of a workgroup see must not be read: such a row
// is read at the nearest key inside.
#pragma once

namespace nvfp4 {

constexpr int kGroupKeys = 16;

// The share that is read for the one at `key`: the last one of the span for
// those past it (hi > 0).
template <int ROWS>
constexpr int group_at(int hi, int key) {
  return key < ((hi - 1) & ~(ROWS - 1)) ? key : (hi - 1) & ~(ROWS - 1);
}

// First and last row, counted from key g, that may be read: g is at most 15
// below lo and below hi.  Both lie in 0 .. 15 however far lo and hi are, so
// that their products with a token stride below 2^26 bytes stay below 2^30.
struct RowBounds {
  int first, end;
};
constexpr RowBounds rows_seen(int lo, int hi, int g) {
  return {lo > g ? lo - g : 0, hi - g < kGroupKeys ? hi - 1 - g : kGroupKeys - 1};
}

// Bytes from key g to the one that is read for row r: the bounds are taken
// times the stride, so that a caller's several rows need no multiplication of
// their own.
struct ByteBounds {
  int first, end;
};
constexpr ByteBounds bytes_seen(RowBounds b, int stride) {
  return {b.first * stride, b.end * stride};
}
constexpr int byte_of(int row_bytes, ByteBounds b) {
  const int at = row_bytes > b.first ? row_bytes : b.first;
  return at < b.end ? at : b.end;
}

}  // namespace nvfp4
