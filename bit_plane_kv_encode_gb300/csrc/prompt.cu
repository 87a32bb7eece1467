// Attention of several new tokens of each sequence at once, on the 5th-generation
// tensor cores: causal over packed prompts or over the rows of a cache that they
// end (bpkv_prompt_attend), or as a tree of drafted tokens over a cache
// (bpkv_tree_attend, bpkv_tree_attend8).  The plan is in prompt_plan.cuh; calls of few
// tokens are streamed instead (prompt_few.cu, few_ctas below).
//
// For every query row, o = sum_x softmax_x(q . k_x / sqrt(D)) v_x over the keys x
// that its token sees, with a running maximum and sum: one pass over the keys.
//
// A segment (a CTA's part of a unit).  One thread loads K and V tiles by TMA into a
// ring of stages; one walks the segments and loads their rows of q; one thread a stream
// issues its products; and two groups of four warps do the softmax, a thread per query
// row: S = Q K^T (128 x 128 x 128) into tensor memory, p = exp2(S - m) written back over
// S as the A operand of O += P V, with O in tensor memory too.  p is rounded to bf16
// there (2^-8), since a product's operands have one type and V is bf16; S, m, O and the
// sum of the unrounded p are float32.  The groups are two streams that take turns at the
// tensor cores: each has 128 rows of its own over every tile, or both hold the same rows
// and take every other tile.  m only follows the maximum when that has risen by a factor
// of 2^kLazy, so O is seldom rescaled.  Only tiles that some row sees a part of are
// masked, by a bit for each key.
//
// What bounds it: the chain of a stream, in cycles (timed inside the kernel when 8191 tokens
// took 390 us): S 700 (both its operands come from shared memory, whose whole bandwidth it
// takes), 300 until the softmax sees it, 600 to the maximum, 600 and 400 to the two halves of
// P, 400 to the end of O: 3000 for two streams' tiles, of which the products are 2048.  And
// the power limit: a call of 400 us runs at 2.0 GHz, calls back to back at 1.8.  Between
// segments 6500 cycles: the last O, 256 rows through the load-store unit (4000, whatever way
// they were turned), the next S.  Less of it, in us, 8191 tokens 369 and 16 packed prompts 602:
// without any softmax 320 and 507, without the exponentials 343 and 566, without most of the
// maximum 358 and 583, without the stores of O 357 and 567.
// Measured on a GB300, 8 x 4 heads: 8191 tokens 365 us, 1.50 PFLOP/s (392 in a long
// run); 16383 tokens 1.32 ms, 1.67 PFLOP/s; 16 packed prompts of 251 to 4001 tokens 600
// us, 1.28; up to 512 tokens of four sequences behind up to 32256 rows 294 us, 1.51 (28 more
// where each run reads the rows when it comes to them); trees of 32 nodes of 16 sequences
// of up to 8192 rows 53 us, 5.2 TB/s.
//
// 8-bit rows.  A group of four more warps turns the tiles of codes, as they come,
// into tiles of bf16: a code times its power of two is exactly a bf16 number, so
// that products, softmax and results are those of bf16 rows of the same values.  A
// tile of K is turned in some 1400 cycles, and there is room for three tiles of bf16
// only, which bounds them: 1000 tokens behind 100000 rows 1.23 ms, 1.34 PFLOP/s;
// trees of 64 nodes of 4 sequences of up to 131071 rows 219 us, 1.26 PFLOP/s.
#include "prompt_plan.cuh"
#include "rows8_core.cuh"
#include "tc.cuh"

namespace bpkv {

int64_t prompt_units(int64_t tokens, int64_t n_seq, int64_t n_heads, int64_t group);

namespace prompt {

template <int BITS>
cudaError_t launch_few_tokens(const FewArgs& a, int ctas, cudaStream_t st);

namespace {

using namespace tc;
using shared::ex2;
using shared::kLogScale;

constexpr uint32_t kTmemCols = 512;              // S of both streams, then O of both
// How far the maximum may pass m before O is rescaled, in powers of two.  Weights are
// numbers with an exponent, and lose nothing above 1; sums of 2^30 of them times values of
// 2^80 stay below 2^126.  With 8 / 12 / 16 / 1000, in us: 8191 tokens 372 / 370 / 367 / 367,
// 16 packed prompts 610 / 604 / 603 / 603, 1000 behind 100000 8-bit rows 1244 / 1234 / 1229 / 1228.
constexpr float kLazy = 16.f;
constexpr int kQ = kTile * kD * 2;               // bytes of a stream's rows of q
constexpr int kStage = kTile * kD * 2;           // of a K or V tile
constexpr int kCodes = kTile * kD;               // of a tile of codes
constexpr int kCodeStage = kCodes + kTile;       // with its exponent bytes

template <int BITS>
struct Shape {
  static constexpr int kThreads = BITS == 16 ? 384 : 512;
  static constexpr int kStages = BITS == 16 ? 4 : 3;       // K of tile t as fill 2 t, V as 2 t + 1
  static constexpr int kCodeStages = BITS == 16 ? 0 : 3;   // of codes, in the same order
  static constexpr int kReaders = 3 + 8 + (BITS == 16 ? 0 : 4);  // of segments: loads, products, the other warps
};
constexpr int kSegments = 2;  // that are known at once

template <int BITS>
struct Smem {
  Plan plan;
  Segment seg[kSegments];
  Cut cut;  // of the last segment
  uint32_t tmem;
  uint32_t abort;
  uint64_t full[4], empty[4];
  uint64_t code_full[3], code_empty[3];
  uint64_t s_full[2], p_half[2], p_ready[2], o_done[2];
  uint64_t turn[2];
  uint64_t seg_full[kSegments], seg_empty[kSegments];
  uint64_t q_full, q_empty, done, fin;
  float2 ml[2][kTile];  // each row's maximum and sum, where both streams hold the rows
};

template <int BITS>
constexpr int kBase = (sizeof(Smem<BITS>) + 1023) / 1024 * 1024 + 1024;
template <int BITS>
constexpr int kSmem = kBase<BITS> + 2 * kQ + Shape<BITS>::kStages * kStage + Shape<BITS>::kCodeStages * kCodeStage;
static_assert(kSmem<16> <= 227 * 1024 && kSmem<8> <= 227 * 1024, "shared memory of a CTA");

// Bytes of a cache's keys and values from which runs go side by side (prompt_plan.cuh):
// about what L2 holds.  With / without, in us, 8 x 4 heads, bf16 rows: 512 tokens behind
// 16000 rows (66 MB) 98 / 97, 32000 (131 MB) 175 / 186, 64000 326 / 372; 128 behind 8000
// 30.3 / 30.3, 64000 99 / 110; 256 of 4 sequences of 4000 (66 MB) 66.7 / 68.2, 8000 105 / 110,
// 16000 182 / 202; 512 of 8 of 3000 (98 MB) 150 / 150; 8-bit rows: 512 of 8 of 3000 (49 MB)
// 181 / 177, behind 64000 (131 MB) 401 / 400, 1000 behind 100000 1229 / 1227, in a long run
// 1233 / 1275.
constexpr int64_t kBesideBytes = 112 << 20;

struct Maps {
  CUtensorMap q, k, v;
};

// Waits for the phase of the given parity to complete.  Gives up (false) after some
// seconds, raising *abort, or once another wait of the CTA has.  Short: it stands in
// many places, and instructions that are not in the cache cost more than the wait.  The
// SM's own clock bounds it: reading the global timer takes longer than most waits.
constexpr int64_t kWaitCycles = 4000000000;
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort) {
  if (mbar_try(bar, parity)) return true;
  const int64_t t0 = clock64();
#pragma unroll 1
  for (uint32_t i = 0; i < kMbarRounds; ++i) {
    if (mbar_try(bar, parity)) return true;
    if (*abort || clock64() - t0 > kWaitCycles) break;
  }
  *abort = 1;
  return false;
}

// The same for what is not urgent: the others keep the issue slots.  tiles: of what is waited
// for.  Two streams' tile is some 3000 cycles, of 8-bit rows 3500, and a segment may have
// millions: with 1.2 million, 150 million rows, it is longer than kWaitCycles.  So 2^16 tiles
// have that, 17 times what they take.  That something is stuck is known sooner, from the waits
// of those who compute, which are for a tile.
template <int NS>
__device__ __forceinline__ bool doze(uint32_t bar, uint32_t parity, volatile uint32_t* abort, int tiles) {
  const int64_t end = clock64() + ((tiles >> 16) + 1) * kWaitCycles;
#pragma unroll 1
  for (uint32_t i = 0; i < 0xffffffffu; ++i) {
    if (mbar_try(bar, parity)) return true;
    if (*abort || clock64() > end) break;
    __nanosleep(NS);
  }
  *abort = 1;
  return false;
}

// The same without the hardware's suspension of a waiting thread: where a hundred cycles count.
__device__ __forceinline__ bool spin(uint32_t bar, uint32_t parity, volatile uint32_t* abort) {
  const int64_t t0 = clock64();
#pragma unroll 1
  for (uint32_t i = 0; i < kMbarRounds; ++i) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (done) return true;
    if ((i & 63u) == 63u && (*abort || clock64() - t0 > kWaitCycles)) break;
  }
  *abort = 1;
  return false;
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Where the keys of a KV head of a sequence begin, as a tile's coordinates.
struct Place {
  int row, plane;
};
__device__ __forceinline__ Place place_of(const Args& a, const Plan& p, const Segment& g) {
  if (a.rows == kCache) return {0, g.seq * a.n_heads + g.h};
  if (a.rows == kToken) return {p.start[g.seq], g.h};
  return {p.start[g.seq] * a.n_heads + g.h * g.t, 0};
}

// The keys of the tile at key0 that a row sees, a bit each.
struct Sees {
  uint32_t w[4];
};
__device__ __forceinline__ uint32_t ones_below(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; }
__device__ __forceinline__ Sees sees_below(int n) {
  return {{ones_below(n), ones_below(n - 32), ones_below(n - 64), ones_below(n - 96)}};
}
// the rows before the tree, which begins at `at` within the tile, and its own as the mask says
__device__ __forceinline__ Sees sees_tree(int at, uint64_t mask) {
  Sees s = sees_below(at);
  uint64_t lo = 0, hi = 0;
  if (at >= 64) {
    if (at < kTile) hi = mask << (at - 64);
  } else if (at > 0) {
    lo = mask << at;
    hi = mask >> (64 - at);
  } else if (at > -64) {
    lo = mask >> -at;
  }
  s.w[0] |= (uint32_t)lo;
  s.w[1] |= (uint32_t)(lo >> 32);
  s.w[2] |= (uint32_t)hi;
  s.w[3] |= (uint32_t)(hi >> 32);
  return s;
}

// 64 logits of a row to weights in bf16, and their sum (of the weights unrounded).
__device__ __forceinline__ void weights(const float* x, float m, uint32_t* w, F2& sum) {
  const float base = m == -INFINITY ? 0.f : m * kLogScale;
  const F2 base2(-base, -base), unit2(kLogScale, kLogScale);
  F2 ls[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    float p0, p1;
    fma2(F2(x[2 * i], x[2 * i + 1]), unit2, base2).get(p0, p1);
    p0 = ex2(p0);
    p1 = ex2(p1);
    ls[i & 1] = add2(ls[i & 1], F2(p0, p1));
    w[i] = bf16x2(p0, p1);
  }
  sum = add2(ls[0], ls[1]);
}

__device__ __forceinline__ void load_half(uint32_t ts, float* x) {
  tmem_ld32(ts, reinterpret_cast<uint32_t*>(x));
  tmem_ld32(ts + 32, reinterpret_cast<uint32_t*>(x) + 32);
}

// Hides what a row does not see of 64 keys; the largest of the rest.
__device__ __forceinline__ float look(float* x, bool masked, uint32_t see0, uint32_t see1) {
  if (masked) {
#pragma unroll
    for (int k = 0; k < 64; ++k)
      if (!(((k < 32 ? see0 : see1) >> (k % 32)) & 1u)) x[k] = -INFINITY;
  }
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int k = 0; k < 64; k += 2) mx[(k / 2) & 3] = max3(mx[(k / 2) & 3], x[k], x[k + 1]);
  return max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
}

// One tile of one query row: S from tensor memory to weights over it, m and l of the
// row so far, and O when m moves.  The first 64 keys' weights are announced on `half`.
__device__ __forceinline__ void softmax_step(uint32_t ts, uint32_t to, bool masked, const Sees& sees, bool first,
                                             uint32_t half, float& m, float& l) {
  float x[64], y[64];
  load_half(ts, x);
  load_half(ts + 64, y);
  wait_ld();
  float top = look(x, masked, sees.w[0], sees.w[1]);
  top = fmaxf(top, look(y, masked, sees.w[2], sees.w[3]));
  const bool up = top > m + kLazy / kLogScale;
  if (first) {
    m = top;
  } else if (__any_sync(0xffffffffu, up)) {
    // S of this step is complete, so O of the stream's step before it is too
    const float f = up ? ex2((m - top) * kLogScale) : 1.f;
    l *= f;
    if (up) m = top;
#pragma unroll 1
    for (int k = 0; k < kD; k += 32) {  // (16 at a time: 1.5% slower over all)
      uint32_t o[32];
      tmem_ld32(to + k, o);
      wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
      tmem_st16(to + k, o);
      tmem_st16(to + k + 16, o + 16);
    }
  }
  uint32_t w[32];
  F2 sum, rest;
  weights(x, m, w, sum);
  tmem_st16(ts, w);
  tmem_st16(ts + 16, w + 16);
  wait_st();
  fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(half);
  weights(y, m, w, rest);
  tmem_st16(ts + 32, w);
  tmem_st16(ts + 48, w + 16);
  float l0, l1;
  add2(sum, rest).get(l0, l1);
  l += l0 + l1;
}

__device__ __forceinline__ uint64_t normal_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// 32 bytes of a row; at an address that is only a multiple of 16 in two stores.
__device__ __forceinline__ void store32(unsigned char* p, const uint32_t* w, bool aligned) {
  if (aligned) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(p + 16) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Two codes to bf16, times `f` each.  A code's magnitude moved to where a bf16 number
// has its own is 2^-120 of it; the sign comes from the byte above, a copy of it.
template <int PAIR>
__device__ __forceinline__ uint32_t bf16_codes(uint32_t w, uint32_t f) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(w), "n"(PAIR ? 0xb3a2 : 0x9180));
  const uint32_t bits = (r << 4) & 0x87f087f0u;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(bits), "r"(f));
  return r;
}
__device__ __forceinline__ uint32_t times(uint32_t x, uint32_t f) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(f));
  return r;
}
// a power of two twice
__device__ __forceinline__ uint32_t twice2(int e) { return (uint32_t)(e + 127) << 7 | (uint32_t)(e + 127) << 23; }

template <int BITS>
__global__ void __launch_bounds__(Shape<BITS>::kThreads, 1) k_prompt(const __grid_constant__ Args a,
                                                                     const __grid_constant__ Maps maps) {
  extern __shared__ __align__(1024) unsigned char raw[];
  Smem<BITS>& sm = *reinterpret_cast<Smem<BITS>*>(raw);
  unsigned char* q_smem = raw + ((smem_u32(raw) + sizeof(Smem<BITS>) + 1023) / 1024 * 1024 - smem_u32(raw));
  constexpr int kStages = Shape<BITS>::kStages, kCodeStages = Shape<BITS>::kCodeStages;
  unsigned char* ring = q_smem + 2 * kQ;
  unsigned char* codes = ring + kStages * kStage;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile uint32_t* abort = &sm.abort;

  if (tid == 0) {
    sm.abort = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&sm.full[i]), BITS == 16 ? 1 : 4);
      mbar_init(smem_u32(&sm.empty[i]), 2);
    }
    for (int i = 0; i < kCodeStages; ++i) {
      mbar_init(smem_u32(&sm.code_full[i]), 1);
      mbar_init(smem_u32(&sm.code_empty[i]), 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sm.s_full[s]), 1);
      mbar_init(smem_u32(&sm.p_half[s]), 4);
      mbar_init(smem_u32(&sm.p_ready[s]), 4);
      mbar_init(smem_u32(&sm.o_done[s]), 1);
      mbar_init(smem_u32(&sm.turn[s]), 1);
    }
    for (int i = 0; i < kSegments; ++i) {
      mbar_init(smem_u32(&sm.seg_full[i]), 1);
      mbar_init(smem_u32(&sm.seg_empty[i]), Shape<BITS>::kReaders);
    }
    mbar_init(smem_u32(&sm.q_full), 1);
    mbar_init(smem_u32(&sm.q_empty), 2);
    mbar_init(smem_u32(&sm.done), 2);
    mbar_init(smem_u32(&sm.fin), kSoftmaxWarps);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_shared();
  }
  if (warp == 2) tmem_alloc(smem_u32(&sm.tmem), kTmemCols);
  if (warp == 3 && lane < 3) prefetch_map(lane == 0 ? &maps.q : lane == 1 ? &maps.k : &maps.v);
  fence_before();
  pdl_enter();
  make_plan(a, sm.plan);  // ends with a barrier of the CTA
  fence_after();
  const uint32_t tmem = sm.tmem;
  // Segments come from one thread, each role takes them in order: its n-th, until
  // `end_segment`, which gives its place back.  By one thread, or by all of a warp.
  uint32_t seg_no = 0;
  Segment g;
  auto next = [&](bool& ok) {
    const uint32_t i = seg_no % kSegments;
    ok = ok && wait(smem_u32(&sm.seg_full[i]), (seg_no / kSegments) & 1, abort);
    if (ok) g = sm.seg[i];
    return ok && g.tiles > 0;
  };
  auto end_segment = [&] { mbar_arrive(smem_u32(&sm.seg_empty[seg_no++ % kSegments])); };

  if (warp < 4) {
    // registers: 128 x 96 + 256 x 200 of the launch's 384 x 168; 8-bit rows:
    // 128 x 48 + 256 x 184 + 128 x 96 of 512 x 128
    regs_fewer<BITS == 16 ? 96 : 48>();
    if (warp == 0) {
      if (elect_one()) {
        // ---- loads: K then V of every tile
        constexpr int kRing = BITS == 16 ? kStages : kCodeStages;
        uint64_t* full = BITS == 16 ? sm.full : sm.code_full;
        uint64_t* empty = BITS == 16 ? sm.empty : sm.code_empty;
        uint32_t stage = 0, phase = 0, issued = 0;
        // keys that only one unit reads go through L2 before anything else
        const uint64_t policy = a.once ? shared::evict_first_policy() : normal_policy();
        bool ok = true;
        while (next(ok)) {
          const Place at = place_of(a, sm.plan, g);
#pragma unroll 1
          for (int t = g.tile0; ok && t < g.tile0 + g.tiles; ++t) {
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              ok = ok && wait(smem_u32(&empty[stage]), phase ^ 1, abort);
              if (!ok) break;
              const uint32_t bar = smem_u32(&full[stage]);
              const CUtensorMap* m = kv ? &maps.v : &maps.k;
              if constexpr (BITS == 16) {
                mbar_expect_tx(bar, kStage);
                tma_load_4d(smem_u32(ring + stage * kStage), m, bar, 0, at.row + t * kTile, 0, at.plane, policy);
              } else {
                const uint32_t dst = smem_u32(codes + stage * kCodeStage);
                mbar_expect_tx(bar, kCodeStage);
                tma_load_3d(dst, m, bar, 0, t * kTile, at.plane, policy);
                bulk_load(dst + kCodes, a.exps[kv] + (int64_t)at.plane * a.cap + t * kTile, kTile, bar);
              }
              ++issued;
              if (++stage == (uint32_t)kRing) stage = 0, phase ^= 1;
            }
          }
          end_segment();
        }
        // the copies in flight must land before the CTA's shared memory is given up
        uint32_t never = 0;
#pragma unroll 1
        for (uint32_t k = issued > (uint32_t)kRing ? issued - kRing : 0; k < issued; ++k)
          wait(smem_u32(&full[k % kRing]), (k / kRing) & 1, &never);
      }
    } else if (warp == 1 || warp == 3) {
      if (elect_one()) {
        // ---- products of stream s, in its own thread: S of a step is issued right
        // behind O of the step before, whose P it takes the place of, so that the tensor
        // cores work while the other stream's softmax runs.  (One thread for both
        // streams spent more cycles on its waits than on the products.)
        const int s = warp >> 1;
        constexpr uint32_t kDescS = mma_desc(1, 1, 0, kTile, kTile);
        constexpr uint32_t kDescO = mma_desc(1, 1, 1, kTile, kD);
        const uint32_t d_s = tmem + s * kTile, d_o = tmem + 2 * kTile + s * kD;
        uint32_t p_phase = 0, tile_no = 0, turns = 0;
        bool ok = true;
        // Streams of their own rows take turns, a turn being the rest of O and the next S:
        // left alone they fall into step, and neither's products hide the other's softmax.
        auto begin_turn = [&] {
          ok = ok && spin(smem_u32(&sm.turn[s]), (turns & 1) ^ (s ? 0 : 1), abort);
          ++turns;
          return ok;
        };
        auto end_turn = [&] { mbar_arrive(smem_u32(&sm.turn[s ^ 1])); };
        // Every fill of the ring is waited for by both threads, and released by both: a
        // wait reads one bit of the stage's phase, which must not run ahead of it.
        auto await = [&](uint32_t use) {
          ok = ok && wait(smem_u32(&sm.full[use % kStages]), (use / kStages) & 1, abort);
          return ok;
        };
        auto skip = [&](uint32_t use) {  // of the other stream's tile
          if (await(use)) mbar_arrive(smem_u32(&sm.empty[use % kStages]));
        };
        auto release = [&](uint32_t use) { mma_commit(smem_u32(&sm.empty[use % kStages])); };
        while (next(ok)) {
          ok = wait(smem_u32(&sm.q_full), seg_no & 1, abort);
          if (!ok) break;
          const bool dual = g.dual;
          const int tiles = g.tiles;
          const uint32_t qb = smem_desc(smem_u32(q_smem + (dual ? s : 0) * kQ), 16);
          const int step = dual ? 1 : 2, t0 = dual ? 0 : s;
          if (t0 >= tiles) mbar_arrive(smem_u32(&sm.q_empty));
          if (!dual && s) {
            skip(2 * tile_no);
            skip(2 * tile_no + 1);
          }
          // S of tile t, and what the barriers wait for: it, the rows of q, the stage
          auto scores = [&](int t) {
            const uint32_t use = 2 * (tile_no + t);
            const uint32_t kb = smem_desc(smem_u32(ring + use % kStages * kStage), 16);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t o = ((k / 4) * (kTile * 128) + (k % 4) * 32) >> 4;
              mma16_ss(d_s, qb + o, kb + o, kDescS, k > 0);
            }
            mma_commit(smem_u32(&sm.s_full[s]));
            if (t + step >= tiles) mma_commit(smem_u32(&sm.q_empty));
          };
          if (t0 < tiles && await(2 * (tile_no + t0)) && (!dual || begin_turn())) {
            fence_after();
            scores(t0);
            release(2 * (tile_no + t0));
            if (dual) end_turn();
          }
#pragma unroll 1
          for (int t = t0; ok && t < tiles; t += step) {
            const uint32_t use = 2 * (tile_no + t);
            const bool more = t + step < tiles, other = !dual && t + 1 < tiles;
            if (!await(use + 1)) break;
            if (other) skip(use + 2);
            const uint32_t vb = smem_desc(smem_u32(ring + (use + 1) % kStages * kStage), kTile * 128);
            ok = ok && spin(smem_u32(&sm.p_half[s]), p_phase, abort);
            if (!ok) break;
            fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k) mma16_ts(d_o, d_s + k * 8, vb + (k * 16 * 128 >> 4), kDescO, (t > t0) | (k > 0));
            // a tile that comes from memory is not waited for before V of this one is given back
            if (dual) {
              if (more) await(use + 2);
              begin_turn();
            }
            ok = ok && spin(smem_u32(&sm.p_ready[s]), p_phase, abort);
            if (!ok) break;
            p_phase ^= 1;
            fence_after();
#pragma unroll
            for (int k = 4; k < 8; ++k) mma16_ts(d_o, d_s + k * 8, vb + (k * 16 * 128 >> 4), kDescO, 1);
            if (!more) mma_commit(smem_u32(&sm.o_done[s]));
            if (!dual) release(use + 1);
            if (other) skip(use + 3);
            if (more && (dual || await(use + 4))) scores(t + step);
            if (dual) {
              end_turn();
              release(use + 1);
            }
            if (more) release(use + 2 * step);
          }
          tile_no += tiles;
          end_segment();
        }
        // every product is complete before tensor memory is given up
        uint32_t never = 0;
        mma_commit(smem_u32(&sm.done));
        wait(smem_u32(&sm.done), 0, &never);
      }
    } else if (warp == 2) {
      if (elect_one()) {
        // ---- the segments, and the loads of their rows of q, once the products have read the last one's
        const uint32_t bytes = 128 * a.group * a.run, bar = smem_u32(&sm.q_full);
        const uint64_t policy = shared::evict_first_policy();
        Walk walk(sm.plan, a);
        uint32_t loads = 0;
        int last = 0;  // tiles of the segment before
        bool ok = true;
        for (;; ++seg_no) {
          const uint32_t i = seg_no % kSegments;
          g = walk.next();
          const uint32_t old = smem_u32(&sm.seg_empty[i]), parity = ((seg_no / kSegments) & 1) ^ 1;
          // that it sleeps costs 8-bit rows 1% (chunk 1241 / 1228) and gives bf16 rows as much (8191 tokens 368 / 373)
          ok = BITS == 16 ? doze<100>(old, parity, abort, 0) : wait(old, parity, abort);
          if (!ok) break;
          sm.seg[i] = g;
          mbar_arrive(smem_u32(&sm.seg_full[i]));
          if (g.tiles == 0) break;
          if (seg_no > 0) ok = doze<100>(smem_u32(&sm.q_empty), (seg_no - 1) & 1, abort, last);
          if (!ok) break;
          const int n = g.dual ? 2 : 1;
          mbar_expect_tx(bar, 2 * n * bytes);
#pragma unroll 1
          for (int s = 0; s < n; ++s)
            for (int half = 0; half < 2; ++half)  // 64 channels each
              tma_load_3d(smem_u32(q_smem + s * kQ + half * (kTile * 128)), &maps.q, bar, half * 64, g.h * a.group,
                          g.token + s * a.run, policy);
          ++loads;
          last = g.tiles;
        }
        uint32_t never = 0;  // as above
        if (loads > 0) wait(bar, (loads - 1) & 1, &never);
      }
    }
  } else if (warp < 4 + kSoftmaxWarps) {
    // ---- softmax of stream s, a thread per row
    regs_more<BITS == 16 ? 200 : 184>();
    const int s = (warp - 4) >> 2, w4 = warp & 3, row = w4 * 32 + lane;
    const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
    const uint32_t ts = tmem + lanes + s * kTile, to = tmem + lanes + 2 * kTile + s * kD;
    const int tok = row * a.group_inv >> 16;  // of the stream's
    uint32_t tile_no = 0, s_phase = 0, o_phase = 0, fin_phase = 0;
    if (row == 0 && s == 0) sm.cut = {};
    bool ok = true;
    while (__all_sync(0xffffffffu, next(ok))) {
      // read where it lies: in registers it costs spills (8191 tokens 392 / 376 us)
      const Segment& g = sm.seg[seg_no % kSegments];
      const int steps = g.steps_of(s), first_tok = g.dual ? s * a.run : 0;
      const bool there = tok < a.run && first_tok + tok < g.tokens;  // a row of the unit
      // keys before this row's end; rows that are not there are not masked
      const int own = g.first + first_tok + tok;
      const int end = there ? g.off + own + 1 : 0x7fffffff;
      uint64_t mask = 0;
      if (a.tree && there)
        mask = a.tree[(int64_t)g.seq * a.t + own] & (a.t >= 64 ? ~0ull : (1ull << a.t) - 1);
      const int keys = g.off + g.t;
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int j = 0; j < steps; ++j) {
        const int t = g.tile_of(s, j), key0 = t * kTile;
        ok = wait(smem_u32(&sm.s_full[s]), s_phase, abort);
        if (BITS == 16 && keys < key0 + kTile) {
          // rows of V past the last key may hold anything: zeros, so that 0 x does not
          // become NaN (of two streams both write them, each before its own product)
          const uint32_t use = 2 * (tile_no + t - g.tile0) + 1, stage = use % kStages;
          ok = ok && wait(smem_u32(&sm.full[stage]), (use / kStages) & 1, abort);
          if (ok) {
            const int valid = max(0, keys - key0);
#pragma unroll 1
            for (int x = row; x < (kTile - valid) * 16; x += kTile) {
              const int v = valid + x / 16, c = x % 16;
              *reinterpret_cast<uint4*>(ring + stage * kStage + (c / 8) * (kTile * 128) + v * 128 + (c % 8) * 16) =
                  make_uint4(0, 0, 0, 0);
            }
            fence_async_shared();
            __syncwarp();  // the first half's announcement is for these too
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        s_phase ^= 1;
        fence_after();
        bool masked;
        Sees sees;
        if (a.tree) {
          masked = g.off < key0 + kTile;
          if (masked) sees = there ? sees_tree(g.off - key0, mask) : sees_below(kTile);
        } else {
          masked = __any_sync(0xffffffffu, end < key0 + kTile);
          if (masked) sees = sees_below(end - key0);
        }
        softmax_step(ts, to, masked, sees, j == 0, smem_u32(&sm.p_half[s]), m, l);
        wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.p_ready[s]));
      }
      if (!ok) break;
      tile_no += g.tiles;
      // what the segment's end takes of it; the walk to the next one hides behind the last O
      const bool dual = g.dual, whole = g.whole, both = !dual && g.steps_of(1) > 0;
      const int rows = min(a.run, g.tokens - first_tok) * a.group, token = g.token + first_tok, h = g.h, slot = g.slot();
      if (row == 0 && s == 0) sm.cut = {g.token, g.h, g.tokens, g.pieces, 1 << sm.plan.beside};  // of the last segment
      const bool writes = (dual || both || s == 0) && w4 * 32 < rows;
      const int c0 = both ? s * 64 : 0, c1 = both ? c0 + 64 : kD;
      const int64_t at = (int64_t)slot * a.slot_rows + (dual ? s * kTile : 0) + w4 * 32;
      // this thread's row, from channel c0 on
      const int x = there ? tok : 0;
      unsigned char* dst =
          whole ? reinterpret_cast<unsigned char*>(
                      a.out + ((((int64_t)token + x) * a.n_heads + h) * a.group + row - x * a.group) * kD + c0)
                : reinterpret_cast<unsigned char*>(a.part_o + (at + lane) * kD + c0);
      const bool aligned = !whole || (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
      __syncwarp();
      if (lane == 0) end_segment();
      else ++seg_no;
      if (steps > 0) {
        ok = __all_sync(0xffffffffu, wait(smem_u32(&sm.o_done[s]), o_phase, abort));
        if (!ok) break;
        o_phase ^= 1;
      }
      m *= kLogScale;
      float f0 = 1.f, f1 = 0.f;
      auto meet = [&] {  // of all softmax warps
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.fin));
        ok = __all_sync(0xffffffffu, wait(smem_u32(&sm.fin), fin_phase, abort));
        fin_phase ^= 1;
        return ok;
      };
      if (both) {  // streams that hold the same rows join them, each half of the channels
        sm.ml[s][row] = make_float2(m, l);
        if (!meet()) break;
        const float2 a0 = sm.ml[0][row], a1 = sm.ml[1][row];
        m = fmaxf(a0.x, a1.x);
        f0 = a0.y == 0.f ? 0.f : ex2(a0.x - m);
        f1 = a1.y == 0.f ? 0.f : ex2(a1.x - m);
        l = f0 * a0.y + f1 * a1.y;
      }
      fence_after();
      if (writes) {
        const uint32_t o0 = (dual ? to : tmem + lanes + 2 * kTile) + c0;
        if (whole) {
          const float inv = l == 0.f ? 0.f : __frcp_rn(l);  // a sum that is NaN stays one
          f0 *= inv;
          f1 *= inv;
        } else if (row < rows && c0 == 0) {
          a.part_ml[at + lane] = make_float2(m, l);
        }
        uint32_t o[32];
        tmem_ld32(o0, o);
#pragma unroll 1
        for (int k = 0; k < c1 - c0; k += 32) {
          wait_ld();
          if (both) {
            uint32_t v[32];
            tmem_ld32(o0 + kD + k, v);
            wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = __float_as_uint(fmaf(__uint_as_float(o[i]), f0, __uint_as_float(v[i]) * f1));
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f0);
          }
          if (whole) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = bf16x2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
            if (k + 32 < c1 - c0) tmem_ld32(o0 + k + 32, o);  // comes while this part leaves
            if (row < rows) {
              store32(dst + k * 2, w, aligned);
              store32(dst + k * 2 + 32, w + 8, aligned);
            }
          } else {
            if (row < rows) {
#pragma unroll
              for (int i = 0; i < 4; ++i) store32(dst + k * 4 + 32 * i, o + 8 * i, true);
            }
            if (k + 32 < c1 - c0) tmem_ld32(o0 + k + 32, o);
          }
        }
      }
      fence_before();
      // O and the rows' maxima are read before the next segment's take their place
      if (both && !meet()) break;
    }
    if (a.split && s == 0 && row == 0) a.cuts[blockIdx.x] = sm.cut;
  } else if constexpr (BITS == 8) {
    // ---- codes to bf16, all four warps each tile
    regs_fewer<96>();
    // A thread a row, in chunks of 16 codes in such an order that eight neighbouring
    // threads' loads, and their stores, meet in no bank.
    const int r = tid - 384, r7 = r & 7;
    const uint32_t src0 = r * 128 + (r7 << 4);
    const uint32_t dst0 = r * 128 + ((r7 & 4) << 12) + (((2 * (r7 & 3)) ^ r7) << 4);
    uint32_t n = 0;
    bool ok = true;
    while (__all_sync(0xffffffffu, next(ok))) {
      const int keys = g.off + g.t;
#pragma unroll 1
      for (int t = g.tile0; ok && t < g.tile0 + g.tiles; ++t) {
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++n) {
          const uint32_t from = n % kCodeStages, to = n % kStages;
          ok = __all_sync(0xffffffffu, wait(smem_u32(&sm.code_full[from]), (n / kCodeStages) & 1, abort));
          if (!ok) break;
          const unsigned char* src = codes + from * kCodeStage;
          unsigned char* dst = ring + to * kStage;
          const bool there = r < keys - t * kTile;
          const int e = min(max((int)src[kCodes + r] - kExpBias, kExpMin), kExpMax);
          // 2^(e + 120), as far as bf16 has it; the rest below.  Rows past the last key
          // may hold anything: zeros, so that 0 x does not become NaN
          const uint32_t f = twice2(min(e, 7) + 120);
          uint4 x[8], y[16];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] = *reinterpret_cast<const uint4*>(src + (src0 ^ (i << 4)));
            if (!there) x[i] = make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            y[2 * i] = make_uint4(bf16_codes<0>(x[i].x, f), bf16_codes<1>(x[i].x, f), bf16_codes<0>(x[i].y, f),
                                  bf16_codes<1>(x[i].y, f));
            y[2 * i + 1] = make_uint4(bf16_codes<0>(x[i].z, f), bf16_codes<1>(x[i].z, f), bf16_codes<0>(x[i].w, f),
                                      bf16_codes<1>(x[i].w, f));
          }
          if (__any_sync(0xffffffffu, e > 7)) {
            const uint32_t f2 = twice2(max(e - 7, 0));
#pragma unroll
            for (int i = 0; i < 16; ++i)
              y[i] = make_uint4(times(y[i].x, f2), times(y[i].y, f2), times(y[i].z, f2), times(y[i].w, f2));
          }
          if (lane == 0) mbar_arrive(smem_u32(&sm.code_empty[from]));
          // only the stores wait for the stage
          ok = __all_sync(0xffffffffu, wait(smem_u32(&sm.empty[to]), ((n / kStages) & 1) ^ 1, abort));
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t at = dst0 ^ ((i & 4) << 12) ^ ((i & 3) << 5);
            *reinterpret_cast<uint4*>(dst + at) = y[2 * i];
            *reinterpret_cast<uint4*>(dst + (at ^ 16)) = y[2 * i + 1];
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.full[to]));
        }
      }
      __syncwarp();
      if (lane == 0) end_segment();
      else ++seg_no;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (tid == 0 && sm.abort) set_status(a.status, BPKV_DEV_TIMEOUT);
  if (warp == 2) tmem_dealloc(tmem, kTmemCols);
}

// The rows of units that were cut: out = sum_pieces 2^(m - M) o / sum_pieces 2^(m - M) l,
// a warp a row, four pieces at a time.
constexpr int kJoinWarps = 8;
constexpr int kJoinDeep = 4;

__global__ void __launch_bounds__(kJoinWarps * 32) k_prompt_join(const __grid_constant__ Args a) {
  pdl_enter();
  const Cut cut = a.cuts[blockIdx.x];
  const int lane = threadIdx.x & 31, r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
  if (cut.pieces > 0 && r < cut.tokens * a.group) {
    const int x = r * a.group_inv >> 16, s = x >= a.run;
    const int64_t in = r + s * (kTile - a.run * a.group);
    float M = -INFINITY, L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < cut.pieces; k0 += kJoinDeep) {
      float2 ml[kJoinDeep];
      float4 o[kJoinDeep];
      float top = M;
#pragma unroll
      for (int i = 0; i < kJoinDeep; ++i) {
        const int k = k0 + i;
        ml[i] = make_float2(-INFINITY, 0.f);
        o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < cut.pieces) {
          const int64_t at = (int64_t)(2 * (blockIdx.x + k * cut.step) + (k == 0)) * a.slot_rows + in;
          ml[i] = a.part_ml[at];
          o[i] = reinterpret_cast<const float4*>(a.part_o + at * kD)[lane];
        }
        if (ml[i].y != 0.f) top = fmaxf(top, fmaxf(ml[i].x, -3e38f));  // a sum that is NaN stays one
      }
      if (top == -INFINITY) continue;
      const float f = ex2(M - top);
      M = top;
      L *= f;
      O = make_float4(O.x * f, O.y * f, O.z * f, O.w * f);
#pragma unroll
      for (int i = 0; i < kJoinDeep; ++i) {
        if (ml[i].y == 0.f) continue;
        const float w = ex2(fmaxf(ml[i].x, -3e38f) - M);
        L = fmaf(w, ml[i].y, L);
        O.x = fmaf(w, o[i].x, O.x);
        O.y = fmaf(w, o[i].y, O.y);
        O.z = fmaf(w, o[i].z, O.z);
        O.w = fmaf(w, o[i].w, O.w);
      }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    uint16_t* dst = a.out + (((cut.token + x) * a.n_heads + cut.h) * a.group + (r - x * a.group)) * kD;
    *reinterpret_cast<uint2*>(dst + lane * 4) = make_uint2(bf16x2(O.x * inv, O.y * inv), bf16x2(O.z * inv, O.w * inv));
  }
}

// ---- host side

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return f;
}

bool encode(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dim,
            const cuuint64_t* stride, const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  const EncodeTiled f = encode_tiled();
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return f && f(m, type, rank, const_cast<void*>(base), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of q [tokens][heads][D], `ld` elements from one token to the next: boxes of
// `run` tokens with the `group` heads of a KV head, 64 channels.
bool map_q(CUtensorMap* m, const void* q, int64_t tokens, int64_t heads, int64_t ld, int group, int run) {
  const cuuint64_t dim[3] = {kD, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t stride[2] = {kD * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)run};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q, dim, stride, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Rows of bf16, `ld` elements apart, in `planes` planes: tiles of 128 rows in two halves of 64 channels.
bool map_rows(CUtensorMap* m, const void* rows, int64_t n, int64_t ld, int64_t planes, int64_t plane_ld) {
  const cuuint64_t dim[4] = {64, (cuuint64_t)n, 2, (cuuint64_t)planes};
  const cuuint64_t stride[3] = {(cuuint64_t)ld * 2, 128, (cuuint64_t)plane_ld * 2};
  const cuuint32_t box[4] = {64, kTile, 2, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, rows, dim, stride, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool map_codes(CUtensorMap* m, const void* rows, int64_t cap, int64_t planes) {
  const cuuint64_t dim[3] = {kD, (cuuint64_t)cap, (cuuint64_t)planes};
  const cuuint64_t stride[2] = {kD, (cuuint64_t)cap * kD};
  const cuuint32_t box[3] = {kD, kTile, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, rows, dim, stride, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct Space {
  size_t starts, cuts, ml, o, total;
  int slot_rows;
};

Space space(int64_t tokens, int64_t group) {
  Space s;
  // of the tokens of a unit at most, a stream's 128 rows, or both streams'
  s.slot_rows = tokens <= kTile / group ? kTile : kRows;
  size_t off = 256;  // status word
  s.starts = off;  // of the call's sequences, where the streaming half hands it over
  off = up256(off + (kMaxSeq + 1) * sizeof(int64_t));
  s.cuts = off;
  off = up256(off + kSms * sizeof(Cut));
  s.ml = off;
  off = up256(off + (size_t)2 * kSms * s.slot_rows * sizeof(float2));
  s.o = off;
  off = up256(off + (size_t)2 * kSms * s.slot_rows * kD * sizeof(float));
  s.total = off;
  return s;
}

// tokens: of a sequence at most; keys: that a unit has at most, as the host knows it
template <int BITS>
cudaError_t launch(Args& a, const Maps& maps, int64_t longest, int64_t keys, void* ws, cudaStream_t st) {
  const Space sp = space(longest, a.group);
  unsigned char* w = static_cast<unsigned char*>(ws);
  a.run = kTile / a.group;
  a.group_inv = ((1u << 16) + a.group - 1) / a.group;
  a.cuts = reinterpret_cast<Cut*>(w + sp.cuts);
  a.part_ml = reinterpret_cast<float2*>(w + sp.ml);
  a.part_o = reinterpret_cast<float*>(w + sp.o);
  a.slot_rows = sp.slot_rows;
  a.once = longest <= 2 * a.run;
  a.status = static_cast<int32_t*>(ws);
  const int64_t units = prompt_units(a.tokens, a.n_seq, a.n_heads, a.group);
  const int64_t tiles = max64(1, (keys + kTile - 1) / kTile);
  a.split = tiles > 4;
  a.beside = a.rows == kCache && !a.once && (int64_t)a.n_seq * a.n_heads * keys * (kD * BITS / 4) >= kBesideBytes;
  const int ctas = (int)max64(1, min64(kSms, a.split ? units * (tiles + 1) / 2 : units));
  static std::atomic<uint64_t> done;
  cudaError_t e = shared::allow_smem(k_prompt<BITS>, kSmem<BITS>, done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k_prompt<BITS>, dim3(ctas), dim3(Shape<BITS>::kThreads), (size_t)kSmem<BITS>, st, a, maps);
  if (e != cudaSuccess || !a.split) return e;
  return launch_pdl(k_prompt_join, dim3(ctas, a.slot_rows / kJoinWarps), dim3(kJoinWarps * 32), 0, st, a);
}

}  // namespace

}  // namespace prompt

using namespace prompt;

int64_t prompt_units(int64_t tokens, int64_t n_seq, int64_t n_heads, int64_t group) {
  return n_heads * (tokens / (2 * (kTile / group)) + min64(n_seq, tokens));
}

// Whether what the units count (with `keys` keys each at most) stays below 2^31.
bool prompt_in_range(int64_t tokens, int64_t n_seq, int64_t n_heads, int64_t group, int64_t keys) {
  return prompt_units(tokens, n_seq, n_heads, group) <= (((int64_t)1 << 31) - 1) / (keys / kTile + 1 + kOver);
}

size_t prompt_bytes(int64_t tokens, int64_t group) { return space(tokens, group).total; }

// The rows of a cache of either kind.
struct PromptRows {
  const void* k;
  const void* v;
  const uint8_t* kexp;
  const uint8_t* vexp;
  const int64_t* len;
  int64_t cap, n_max;
};

namespace {

template <int BITS>
cudaError_t over_cache(Args& a, Maps& maps, const PromptRows& c, int64_t longest, void* ws, cudaStream_t st) {
  const int64_t planes = (int64_t)a.n_seq * a.n_heads;
  a.rows = kCache;
  a.len = c.len;
  a.cap = c.cap;
  a.exps[0] = c.kexp;
  a.exps[1] = c.vexp;
  const bool ok = BITS == 16 ? map_rows(&maps.k, c.k, c.cap, kD, planes, c.cap * kD) &&
                                   map_rows(&maps.v, c.v, c.cap, kD, planes, c.cap * kD)
                             : map_codes(&maps.k, c.k, c.cap, planes) && map_codes(&maps.v, c.v, c.cap, planes);
  if (!ok) return cudaErrorInvalidValue;
  return launch<BITS>(a, maps, longest, c.n_max, ws, st);
}

PromptRows rows_of(const bpkv_cache& c) {
  return {c.k_rows, c.v_rows, nullptr, nullptr, c.seq_len, c.cap_tokens, c.n_max};
}
PromptRows rows_of(const bpkv_rows8& c) { return {c.k8, c.v8, c.kexp, c.vexp, c.seq_len, c.cap_tokens, c.n_max}; }

}  // namespace

// Tokens of a call of bpkv_prompt_attend that may be streamed: a row's mask has 64 bits.
constexpr int64_t kFewTokens = 64;

// CTAs of a cluster that streams each of n units (16 rows at most of a sequence and KV
// head), 0: the tensor cores take the call.  As many CTAs as leave all units resident at
// once (clusters of 8 find room for 12 at least).  rows: of a sequence and KV head at
// most; again: the units of a sequence are several, which read its keys each; wide: units
// of the tensor cores.
//
// Streamed / tensor cores, in us, trees of t nodes of 4 heads for each of 8 KV heads, bf16
// rows (8-bit rows in brackets).  Up to 16 rows the keys are read once either way:
//   1 sequence, t = 1, 300 keys 5.6 / 9.3 (6.2 / 10.4), 4000 7.5 / 12.3 (7.5 / 14.0), 64000
//   43 / 44 (40 / 48); 16 sequences of 4000 40 / 45 (23 / 52); 64 of 4000 148 / 160 (91 / 176);
//   t = 4: 1 of 4000 10.7 / 12.6 (10.5 / 14.1), of 16000 20.7 / 17.5 (19.5 / 21.2), of 64000
//   60 / 44 (55 / 49); 4 of 64000 152 / 153 (102 / 161); 64 of 1000 57 / 51 (51 / 69), of 4000
//   165 / 163 (121 / 176).
// More rows read them again, from L2, for every 16:
//   t = 8: 1 of 1000 9.1 / 11.0 (9.0 / 12.6), of 4000 13.9 / 12.8 (13.6 / 14.4), of 16000
//   33 / 18 (31 / 21); 4 of 1000 11.1 / 12.9 (11.0 / 15.0), of 4000 20.9 / 18.4 (19.8 / 22.2);
//   16 of 300 16.2 / 10.8 (17.2 / 11.7); t = 16: 1 of 4000 14.1 / 13.8 (13.6 / 15.4); 4 of 1000
//   13.3 / 13.5 (12.9 / 15.4), of 4000 33 / 20 (31 / 22.5).
// Prompts over their own keys: 1 token 3.9 / 7.2, 17 5.7 / 7.3, 64 6.2 / 9.3, 32 of 1
//   token 8.0 / 13.0; of 32 heads in groups of 1, 64 tokens 7.0 / 7.5.
int few_ctas(int bits, int64_t n, int64_t wide, int rows, bool again, int64_t keys) {
  // no wider than there are tiles for, below 600 keys not as wide: the barriers cost what it saves
  const int ctas = keys <= 128 ? 1 : n <= 12 ? (keys < 600 ? 4 : 8) : n <= 32 ? 4 : n <= 72 ? 2 : 1;
  // of few keys a unit takes some 4.5 us of its SM streamed, and 3.5, behind 5.5 once, on the tensor cores
  if (keys <= kFewTokens) return n <= kSms * 3 / 4 * (1 + (wide + kSms - 1) / kSms) ? ctas : 0;
  if (again) return n <= kSms && keys <= (bits == 16 ? 1000 : 2000) * ctas ? ctas : 0;
  // 64 to 96 CTAs with two products for each load of a tile
  if (bits == 16 && rows > 8 && ctas == 8 && keys > 12000) return 0;
  return ctas;
}

// few_ctas takes a call's tokens for spread over its sequences; one may have them all, and its
// rows, 16 at a time, are then streamed again and again by CTAs that each read all keys.  Whether
// that would cost more than a look at the lengths on the device and a launch of both halves.  Us
// without / with it, where one sequence has all tokens, and where each has one; 8 x 4 heads, bf16
// rows (8-bit rows in brackets):
//   64 of 64 sequences of 16000: 118 / 40 and 592 / 600 (109 / 41, 385 / 393), of 100000: 659 / 93
//   and 3618 / 3600 (601 / 105, 2295 / 2285); 16 of 16 of 16000: 111 / 24 and 149 / 157 (101 / 26,
//   101 / 106).  Of fewer keys there is less to gain: 64 of 64 of 4000: 41, one sequence alone on
//   the tensor cores 21 (39, 22), of 2000: 28, 19 (27, 19).
// Where n_max is far above the lengths it costs 6 us, of 64 sequences 12 (16 of one token each, of
// 300 rows: 7.8 / 14.2; 64 25 / 37).
// The groups that are then busy, of all KV heads, take turns on the SMs.
static bool one_may_have_them(int64_t H, int64_t rows, int64_t per, int ctas, int64_t keys) {
  const int64_t busy = H * ((rows + per - 1) / per);
  return rows > per && keys * ((busy + kSms - 1) / kSms) > 4000 * ctas;
}

static void few_rows(FewArgs& f, const PromptRows& r, int64_t step) {
  f.len = r.len;
  f.rows[0][0] = r.k;
  f.rows[0][1] = r.v;
  f.exps[0][0] = r.kexp;
  f.exps[0][1] = r.vexp;
  f.cap = r.cap;
  f.step[0] = f.step[1] = step;
  f.where = kCache;
}

cudaError_t launch_prompt(const bpkv_prompt_args& p, void* ws, cudaStream_t st) {
  Args a = {};
  Maps maps;
  a.q_start = p.q_start;
  a.out = p.out;
  a.tokens = p.n_tokens;
  a.n_seq = p.n_seq;
  a.n_heads = p.n_kv_heads;
  a.group = p.group;
  const int64_t H = p.n_kv_heads, T = p.n_tokens;
  const bool by_token = p.ld_k != 0;
  if (T <= kFewTokens) {
    // groups of rows at most: one more for every sequence that has tokens
    const int64_t per = T * p.group <= 8 ? 8 : 16, some = min64(p.n_seq, T);
    const int groups = (int)(T * p.group / per + some);
    FewArgs f = {p.q_start, nullptr, nullptr, p.q, p.out, {{p.k, p.v}}, {{nullptr, nullptr}}, 0, p.ld_q,
                 {kD * 2, kD * 2}, (int32_t)T, p.n_seq, p.n_kv_heads, p.group, 0, by_token ? kToken : kSeq, groups, (int32_t)per};
    if (by_token) f.step[0] = p.ld_k * 2, f.step[1] = p.ld_v * 2;
    if (p.cache) few_rows(f, rows_of(*p.cache), kD * 2);
    if (p.rows8) few_rows(f, rows_of(*p.rows8), kD);
    const int64_t keys = p.cache ? p.cache->n_max : p.rows8 ? p.rows8->n_max : T;
    const bool again = 2 * groups > 3 * some;
    const int ctas = few_ctas(p.rows8 ? 8 : 16, H * groups, prompt_units(T, p.n_seq, H, p.group), (int)(T * p.group), again, keys);
    if (ctas) {
      const bool either = f.len && !again && one_may_have_them(H, T * p.group, per, ctas, keys);
      if (either) f.starts = reinterpret_cast<int64_t*>(static_cast<unsigned char*>(ws) + space(T, p.group).starts);
      const cudaError_t e = p.rows8 ? launch_few_tokens<8>(f, ctas, st) : launch_few_tokens<16>(f, ctas, st);
      if (e != cudaSuccess || !either) return e;
      a.q_start = f.starts;
    }
  }
  if (!map_q(&maps.q, p.q, T, H * p.group, p.ld_q, p.group, kTile / p.group)) return cudaErrorInvalidValue;
  if (p.cache) return over_cache<16>(a, maps, rows_of(*p.cache), T, ws, st);
  if (p.rows8) return over_cache<8>(a, maps, rows_of(*p.rows8), T, ws, st);
  a.rows = by_token ? kToken : kSeq;
  const bool ok = by_token ? map_rows(&maps.k, p.k, T, p.ld_k, H, kD) && map_rows(&maps.v, p.v, T, p.ld_v, H, kD)
                           : map_rows(&maps.k, p.k, T * H, kD, 1, T * H * kD) &&
                                 map_rows(&maps.v, p.v, T * H, kD, 1, T * H * kD);
  if (!ok) return cudaErrorInvalidValue;
  return launch<16>(a, maps, T, T, ws, st);
}

template <typename C>
static cudaError_t tree(const C& c, int32_t t, const uint64_t* mask, const uint16_t* q, uint16_t* out, void* ws,
                        cudaStream_t st) {
  constexpr int BITS = sizeof(C) == sizeof(bpkv_cache) ? 16 : 8;
  const PromptRows r = rows_of(c);
  const int32_t per = t * c.group <= 8 ? 8 : 16, groups = (t * c.group + per - 1) / per;
  const int ctas = few_ctas(BITS, (int64_t)c.n_seq * c.n_kv_heads * groups,
                            prompt_units((int64_t)c.n_seq * t, c.n_seq, c.n_kv_heads, c.group), t * c.group, groups > 1, c.n_max);
  if (ctas) {
    FewArgs a = {nullptr, nullptr, mask, q, out, {{nullptr, nullptr}}, {{nullptr, nullptr}}, 0, (int64_t)c.n_kv_heads * c.group * kD,
                 {0, 0}, c.n_seq * t, c.n_seq, c.n_kv_heads, c.group, t, kCache, groups, per};
    few_rows(a, r, BITS == 16 ? kD * 2 : kD);
    return launch_few_tokens<BITS>(a, ctas, st);
  }
  Args a = {};
  Maps maps;
  a.tree = mask;
  a.out = out;
  a.n_seq = c.n_seq;
  a.n_heads = c.n_kv_heads;
  a.group = c.group;
  a.t = t;
  a.tokens = (int64_t)c.n_seq * t;
  const int64_t heads = (int64_t)c.n_kv_heads * c.group;
  if (!map_q(&maps.q, q, a.tokens, heads, heads * kD, c.group, kTile / c.group)) return cudaErrorInvalidValue;
  return over_cache<BITS>(a, maps, r, t, ws, st);
}
static_assert(sizeof(bpkv_cache) != sizeof(bpkv_rows8), "which of the two a template has");

cudaError_t launch_tree(const bpkv_cache& c, int32_t t, const uint64_t* mask, const uint16_t* q, uint16_t* out, void* ws,
                        cudaStream_t st) {
  return tree(c, t, mask, q, out, ws, st);
}
cudaError_t launch_tree8(const bpkv_rows8& c, int32_t t, const uint64_t* mask, const uint16_t* q, uint16_t* out, void* ws,
                         cudaStream_t st) {
  return tree(c, t, mask, q, out, ws, st);
}

}  // namespace bpkv
