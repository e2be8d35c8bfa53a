// Limits of a launch's grid, and the most (expert, block of slots) items there can be.  Host
// code, without HIP.
#pragma once

namespace w4a16 {
namespace {

// A launch of 256 threads a workgroup has at most this many (2^32 threads).
constexpr long kMaxBlocks = (1L << 24) - 8;

// The most items there can be: every expert with a slot adds at most one
// partly filled block.
inline long max_items(long R, long E, long B) {
  const long active = R < E ? R : E;
  return (R + (B - 1) * active) / B;
}

}  // namespace
}  // namespace w4a16
