// Which calls' tensors share bytes, from their addresses, sizes and strides (host).
#pragma once

#include <algorithm>
#include <cstdint>

namespace bsq {

// n[0] times n[1] pieces of `width` bytes, `step` bytes apart (steps of at least 0; that of a single piece does not matter).  Without an address
// or without pieces it is empty.
struct HostRegion {
  const void* at;
  int64_t width;
  int64_t n[2], step[2];

  bool empty() const { return !at || width <= 0 || n[0] <= 0 || n[1] <= 0; }
  int64_t apart(int level) const { return n[level] > 1 ? step[level] : 0; }
  // Bytes from the first to the last; nothing is as large as the most that it says.
  int64_t extent() const {
    const __int128 e = static_cast<__int128>(n[0] - 1) * apart(0) + static_cast<__int128>(n[1] - 1) * apart(1) + width;
    return e < (int64_t(1) << 61) ? static_cast<int64_t>(e) : int64_t(1) << 61;
  }
};
inline HostRegion host_region(const void* at, int64_t width) { return {at, width, {1, 1}, {0, 0}}; }

// Whether low < d + i step < high for an i from `first` to `last` (step >= 0).
inline bool multiple_between(int64_t d, int64_t step, int64_t first, int64_t last, int64_t low, int64_t high) {
  if (step == 0 || first == last) return low < d + first * step && d + first * step < high;
  const int64_t past = low + 1 - d, least = past > 0 ? (past + step - 1) / step : -(-past / step);  // the first that is above low
  const int64_t i = std::max(first, least);
  return i <= last && d + i * step < high;
}

// Whether two of them share bytes.  Exact where the steps of the pieces that both have several of are equal; regions of other steps count as
// sharing where their extents do (on the inner level: the extents of one outer piece).
inline bool regions_overlap(const HostRegion& a, const HostRegion& b) {
  if (a.empty() || b.empty()) return false;
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.at) - reinterpret_cast<uintptr_t>(a.at));
  const int64_t ea = a.extent(), eb = b.extent(), most = int64_t(1) << 61;
  if (d >= ea || -d >= eb) return false;
  if (ea == most || eb == most) return true;
  if (a.n[0] > 1 && b.n[0] > 1 && a.step[0] != b.step[0]) return true;
  const int64_t outer = std::max(a.apart(0), b.apart(0)), inner = std::max(a.apart(1), b.apart(1));
  const int64_t first = 1 - a.n[0], last = b.n[0] - 1;  // b's outer pieces less a's
  // one outer piece as a whole: enough where a token's heads lie side by side
  const int64_t wa = a.apart(1) * (a.n[1] - 1) + a.width, wb = b.apart(1) * (b.n[1] - 1) + b.width;
  if (!multiple_between(d, outer, first, last, -wb, wa)) return false;
  if (a.n[1] > 1 && b.n[1] > 1 && a.step[1] != b.step[1]) return true;
  for (int64_t k = 1 - a.n[1]; k < b.n[1]; ++k)
    if (multiple_between(d + k * inner, outer, first, last, -b.width, a.width)) return true;
  return false;
}

// Whether pieces of one share bytes.
inline bool region_overlaps_itself(const HostRegion& a) {
  if (a.empty()) return false;
  const int64_t outer = a.apart(0), inner = a.apart(1);
  if ((a.n[0] > 1 && outer < a.width) || (a.n[1] > 1 && inner < a.width)) return true;
  if (a.extent() == int64_t(1) << 61) return false;
  if (a.n[0] == 1 || a.n[1] == 1 || (a.n[1] - 1) * inner + a.width <= outer || (a.n[0] - 1) * outer + a.width <= inner) return false;
  for (int64_t k = 1; k < a.n[1]; ++k)
    if (multiple_between(k * inner, outer, 1 - a.n[0], a.n[0] - 1, -a.width, a.width)) return true;
  return false;
}

}  // namespace bsq
