// Shared memory of the wide kernel (k_shared_wide): its barriers, and the ring of
// stages that K and V tiles come into, K of tile t as fill 2 t and V as 2 t + 1.
#pragma once

#include "shared_plan.cuh"

namespace bpkv {
namespace shared {
namespace wide {

constexpr int kTile = kWideTile;
constexpr int kSoftmaxWarps = 8;                 // four a stream, a thread per row
constexpr int kRing16 = 32 * 1024;               // bytes of a stage: 128 rows of bf16
constexpr int kRing8 = 16 * 1024;                // 128 rows of codes
// Not 10: a wait for a fill reads one bit of the stage's phase, so the fill
// before must be known to have landed when it begins.  A stream's scale warp
// waits for V of tile t (fill 2 t + 1) once the softmax of its tile t - 4 is done.
// That says that K and V of t - 4 have landed, and all fills up to K of t - 5, but
// not V of t - 5, the other stream's: fill 2 t - 9.
constexpr int kMaxStages = 9;

template <int BITS>
struct Scales {};

template <>
struct Scales<8> {
  float qf[2][2][kTile];  // scales of the rows of q, by segment parity and stream
  __align__(16) float tok[2][2][3][kTile];  // by stream, twice: 2^ek log2(e)/sqrt(D), ev, 2^-ev of a tile's tokens
};

template <int BITS>
struct Smem {
  Scales<BITS> sc;
  WidePlan plan;
  uint32_t tmem;
  uint32_t abort;
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t s_full[2], p_ready[2], o_done[2];
  uint64_t q_full, q_empty, done;
  uint64_t sc_go[2], sc_full[2][2], sc_empty[2][2];
  uint64_t p_half[2], fin;
  float2 ml[2][kTile];  // each row's maximum and sum, where both streams hold the rows
};

// Smem, then 1024-byte aligned the rows of q, then the ring.
template <int BITS>
struct Shape {
  static constexpr int kQ = kTile * kD * 2;                       // one stream's rows of q (16 bits, or two 8-bit pieces)
  static constexpr int kStage = BITS == 16 ? kRing16 : kRing8;    // K or V tile
  static constexpr int kExps = BITS == 16 ? 0 : 2 * kTile;        // exponent bytes that come with V
  static constexpr int kSmemMax = 227 * 1024;
  static constexpr int kBase = (sizeof(Smem<BITS>) + 1023) / 1024 * 1024 + 1024;
  static constexpr int stages(bool dual) {
    const int n = (kSmemMax - kBase - (dual ? 2 : 1) * kQ) / (kStage + kExps);
    return n < kMaxStages ? n : kMaxStages;
  }
  static int bytes(bool dual) { return kBase + (dual ? 2 : 1) * kQ + stages(dual) * (kStage + kExps); }
};

static_assert(Shape<16>::stages(true) >= 4 && Shape<8>::stages(true) >= 8, "two tiles of K and V at least");
static_assert(Shape<8>::stages(true) <= 9 && Shape<8>::stages(false) <= 9,
              "the fill before V of tile t is V of t - 4 or K of t - 4, which the scale warp knows of");

}  // namespace wide
}  // namespace shared
}  // namespace bpkv
