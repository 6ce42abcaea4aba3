// Rings, converting groups and tensor memory of the 4-bit tensor-core kernel
// (int4_mma.cu) for each token tile.  Plain C++, so that a host program can
// print the numbers and walk the roles' barriers with them.
#pragma once

namespace lq {

constexpr int kMaxRing = 8, kMaxA = 4;
constexpr int kWeightTile = 128 * 64;   // bytes of a 128-row, 128-wide block of codes

// NT <= 64: two CTAs per SM, one accumulator, the converting warps also run
// the epilogue (the other CTA computes meanwhile, and the next launch fits
// beside this one).  Larger tiles: one CTA per SM and eight epilogue warps; at
// 128 tokens two accumulators, at 256 one, which with four converted blocks
// fills the tensor memory.
template <int NT>
struct MmaShape {
  static constexpr int kTokenTile = NT * 256;                    // bytes of NT tokens x 128 k
  static constexpr int kStage = kWeightTile + kTokenTile;
  static constexpr bool kTwo = NT <= 64;
  // converting groups of four warps, group g takes blocks g, g + kGroups, ...; one keeps up with the
  // MMAs of 256 tokens, and 14 warps have 128 registers a thread (18 have 96), so that the epilogue's 64
  // words of packed columns spill 92 to 120 bytes only
  static constexpr int kGroups = NT == 256 ? 1 : 2;
  // converted weight blocks in tensor memory.  128 tokens: with four, a ring of five slots does not meet
  // the condition below; three and five, or four and a ring of four: [24576, 4096] at 128 tokens 32.2 / 35.0 us,
  // [5120, 25600] at 100 35.2 / 39.0, 8008 rows of 128 experts [1536, 2048] 88 / 98, [2048, 768] 62.4 / 64.2.
  static constexpr int kA = NT <= 128 ? 3 : 4;
  static constexpr int kD = NT == 128 ? 2 : 1;                   // accumulators
  static constexpr int kCols = kTwo ? 256 : 512;                 // tensor-memory columns
  static constexpr int kFit = (kTwo ? 100 : 217) * 1024 / kStage;
  static constexpr int kRing = kFit < kMaxRing ? kFit : kMaxRing;
  static constexpr int kSmem = kRing * kStage + 1024;
  static constexpr int kConvWarps = 4 * kGroups;
  static constexpr int kWarps = 2 + kConvWarps + (kTwo ? 0 : 8);
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kEpiFirst = kTwo ? 2 : 2 + kConvWarps;    // first of the eight epilogue warps
  static_assert(kA * 64 + kD * NT <= kCols, "tensor memory");
  static_assert(!kTwo || kD == 1, "the converting warps' epilogue knows one accumulator");
  // A barrier tells the phases apart by their parity only, so a group that
  // waits for block j in ring slot j % kRing has to know that block j - kRing
  // of the same slot has arrived; else the wait may end one phase early, before
  // j's copies.  It knows when that block was its own (kRing a multiple of
  // kGroups), or when the MMAs that its previous block waited for, those up to
  // block j - kGroups - kA, include it.  The same for the converted blocks: for
  // block j a group waits for the MMAs of j - kA, and its previous block waited
  // for those of j - kGroups - kA, which have to include j - 2 kA.
  static_assert(kRing % kGroups == 0 || kGroups + kA <= kRing, "a ring slot's phases are told apart by parity");
  static_assert(kGroups <= kA, "a converted block's phases are told apart by parity");
};

}  // namespace lq
