// Products of fp32 values in three bf16 parts each, largest first.
#pragma once

namespace mps {
namespace {

// Parts that are multiplied: those whose product can reach 2^-16 of the largest
// (the others are at most 2^-24 of it each), the smallest first: the sums of
// the small ones then round at their own size, and fp32 logits are half as far
// off as with the largest first.  Behind the last pair, where a walk over their
// stages looks ahead, the last one.
constexpr int kPairs = 6;
constexpr int held(int pair) { return pair < kPairs ? pair : kPairs - 1; }
constexpr int part_a(int pair) { return (0x001012 >> (4 * held(pair))) & 0xf; }
constexpr int part_b(int pair) { return (0x010210 >> (4 * held(pair))) & 0xf; }

}  // namespace
}  // namespace mps
