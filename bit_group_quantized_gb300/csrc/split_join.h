// split_join.h — which parts of a cut unit kv4_split.cu joins together, and
// where their CTAs count their arrivals. Plain C++, so that the host can check
// the arithmetic as the kernel runs it.
#pragma once

#include "host_device.h"

namespace bgq {

// The CTA whose share of the list, [total * c / ctas, total * (c + 1) / ctas), holds a place.
BGQ_HOST_DEVICE int split_cta(long long place, long long ctas, long long total) {
  return (int)(((place + 1) * ctas - 1) / total);
}

// Many and large parts are joined by eights first, each eight by its own last CTA: one SM alone reads half a MB too
// slowly (76 parts of 16 columns of 256: 49 us for the call with one join, 40 with two; 38 parts of 4 columns of
// 128: 44.5 with one, 46.9 with two).
constexpr int kJoinGroup = 8;
BGQ_HOST_DEVICE bool split_two_levels(int parts, int columns, int head_dim) { return parts * columns * head_dim > 1 << 17; }

// The parts first, first + step, ... (n of them) of the unit that CTAs c0 .. c1 share, joined by the last of their CTAs to count
// at `counter` (-1: one part, with nobody to wait for).
struct SplitJoin {
  int first, step, n, counter;
};
// CTA `cta`'s eight. Its counter is that of its first CTA: of the eights of two parts or more none begins at c1, where the next
// unit may begin its own first eight.
BGQ_HOST_DEVICE SplitJoin split_eight(int c0, int c1, int cta, int grid) {
  const int first = (cta - c0) / kJoinGroup * kJoinGroup, left = c1 - c0 + 1 - first;
  const int n = left < kJoinGroup ? left : kJoinGroup;
  return SplitJoin{first, 1, n, n > 1 ? grid + c0 + first : -1};
}
// All parts, or all eights. One unit at most begins in CTA c0 and does not end there.
BGQ_HOST_DEVICE SplitJoin split_all(int c0, int c1, bool eights) {
  const int parts = c1 - c0 + 1;
  return eights ? SplitJoin{0, kJoinGroup, (parts + kJoinGroup - 1) / kJoinGroup, c0} : SplitJoin{0, 1, parts, c0};
}

}  // namespace bgq
