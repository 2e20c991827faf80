// Launches of the serial walks, by whichever way suits the batch.
#pragma once

#include "scan_rows.hpp"
#include "scan_split.hpp"

namespace rs {

namespace {

template <typename T, int DK, typename Ops, bool KEEP>
hipError_t launch_scan(const DeltaArgs& a, const Kept& kept, hipStream_t s) {
  Walk walk;
  const hipError_t e = choose_walk<T>(a, &walk);
  if (e != hipSuccess) return e;
  if constexpr (sizeof(T) == 2) {
    if (walk == Walk::kRows128) return launch_scan_rows<T, DK, 2, Ops, KEEP>(a, kept, s);
  }
  if (walk == Walk::kSplit) return launch_scan_split<T, DK, Ops, KEEP>(a, kept, s);
  return launch_scan_rows<T, DK, 1, Ops, KEEP>(a, kept, s);
}

template <typename T, int DK, typename Ops>
hipError_t launch_reverse(const DeltaArgs& a, const Kept& kept, hipStream_t s) {
  Walk walk;
  const hipError_t e = choose_walk<T>(a, &walk);
  if (e != hipSuccess) return e;
  // (128 rows at a time would take more LDS than there is beside T^T and P^T in three parts, twice)
  if (walk == Walk::kSplit) return launch_reverse_split<T, DK, Ops>(a, kept, s);
  return launch_reverse_rows<T, DK, 1, Ops>(a, kept, s);
}

}  // namespace

}  // namespace rs
