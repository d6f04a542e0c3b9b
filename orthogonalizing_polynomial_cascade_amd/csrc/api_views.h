// Argument checks of the training operators' entry points: element types, pitches and shared memory.
#pragma once

#include <hip/hip_runtime.h>

#include <initializer_list>

#include "../../include/anvil.h"
#include "api_common.h"

namespace anvil {

constexpr int64_t kMaxRows = int64_t(1) << 31;
// columns of one row: tile offsets of 256 rows stay within 32 bits
constexpr int64_t kMaxWidth = int64_t(1) << 22;
constexpr int64_t kMaxPitch = int64_t(1) << 22;

inline int elem_bytes(int dtype) { return dtype == ANVIL_F32 ? 4 : 2; }
inline bool elem_known(int dtype) {
  return dtype == ANVIL_F32 || dtype == ANVIL_BF16 || dtype == ANVIL_F16;
}

// A caller buffer of `rows` rows of `width` bytes, `pitch` bytes apart (null: not given).
struct View {
  const void* p;
  int64_t rows, width, pitch;
  bool written;
};

inline View dense(const void* p, size_t bytes, bool written) {
  return {p, 1, static_cast<int64_t>(bytes), static_cast<int64_t>(bytes), written};
}

// Whether two views share a byte.  Views whose spans cross but whose rows lie side by side at the
// same pitch (two column ranges of one buffer) do not.
inline bool shares(const View& a, const View& b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  const size_t na = static_cast<size_t>((a.rows - 1) * a.pitch + a.width);
  const size_t nb = static_cast<size_t>((b.rows - 1) * b.pitch + b.width);
  if (!overlap(a.p, na, b.p, nb)) return false;
  if (a.pitch != b.pitch || a.rows < 2 || b.rows < 2) return true;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const int64_t pitch = a.pitch;
  const int64_t shift = y >= x ? static_cast<int64_t>((y - x) % pitch)
                               : (pitch - static_cast<int64_t>((x - y) % pitch)) % pitch;
  return !(shift >= a.width && shift + b.width <= pitch);
}

// ANVIL_ERR_ALIAS if an output shares memory with anything else.
inline int check_views(std::initializer_list<View> views) {
  for (auto i = views.begin(); i != views.end(); ++i)
    for (auto j = i + 1; j != views.end(); ++j)
      if ((i->written || j->written) && shares(*i, *j)) return ANVIL_ERR_ALIAS;
  return ANVIL_OK;
}

// A pitch in elements: at least the row, within bounds.  A single row has none: its is taken as the
// row's width, whatever the caller's value (the last token of a long sequence has the sequence's).
inline bool take_pitch(const void* p, int64_t* ld, int64_t width, int64_t rows) {
  if (rows <= 1) *ld = width;
  return !p || (*ld >= width && *ld <= kMaxPitch);
}

}  // namespace anvil
