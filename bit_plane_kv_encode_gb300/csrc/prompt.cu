// Attention of several new tokens of each sequence at once, on the 5th-generation
// tensor cores: causal over packed prompts or over the rows of a cache that they
// end (bpkv_prompt_attend), or as a tree of drafted tokens over a cache
// (bpkv_tree_attend, bpkv_tree_attend8).  The plan is in prompt_plan.cuh.
//
// For every query row, o = sum_x softmax_x(q . k_x / sqrt(D)) v_x over the keys x
// that its token sees, with a running maximum and sum: one pass over the keys.
//
// A segment (a CTA's part of a unit).  One thread loads K and V tiles by TMA into a
// ring of stages, one loads the rows of q, one issues the products, and two groups
// of four warps do the softmax, a thread per query row: S = Q K^T (128 x 128 x 128)
// into tensor memory, p = exp2(S - m) written back over S as the A operand of
// O += P V, with O in tensor memory too.  p is rounded to bf16 there (2^-8), since a
// product's operands have one type and V is bf16; S, m, O and the sum of the
// unrounded p are float32.  The groups are two streams that take turns at the tensor
// cores: each has 128 rows of its own over every tile, or both hold the same rows and
// take every other tile.  m only follows the maximum when that has risen by a factor
// of 2^kLazy, so O is seldom rescaled.  Only tiles that some row sees a part of are
// masked, by a bit for each key.
//
// 8-bit rows.  A group of four more warps turns the tiles of codes, as they come,
// into tiles of bf16: a code times its power of two is exactly a bf16 number, so
// that products, softmax and results are those of bf16 rows of the same values.
#include "prompt_plan.cuh"
#include "rows8_core.cuh"
#include "tc.cuh"

namespace bpkv {
namespace prompt {

namespace {

using namespace tc;

constexpr uint32_t kTmemCols = 512;              // S of both streams, then O of both
constexpr float kLogScale = 0.08838834764831845f * 1.4426950408889634f;  // log2(e) / sqrt(D)
constexpr float kLazy = 8.f;                     // how far the maximum may pass m before O is rescaled, in powers of two
constexpr int kQ = kTile * kD * 2;               // bytes of a stream's rows of q
constexpr int kStage = kTile * kD * 2;           // of a K or V tile
constexpr int kCodes = kTile * kD;               // of a tile of codes
constexpr int kCodeStage = kCodes + kTile;       // with its exponent bytes

template <int BITS>
struct Shape {
  static constexpr int kThreads = BITS == 16 ? 384 : 512;
  static constexpr int kStages = BITS == 16 ? 4 : 3;       // K of tile t as fill 2 t, V as 2 t + 1
  static constexpr int kCodeStages = BITS == 16 ? 0 : 3;   // of codes, in the same order
};

template <int BITS>
struct Smem {
  Plan plan;
  Walk walk[Shape<BITS>::kThreads / 32];
  uint32_t tmem;
  uint32_t abort;
  uint64_t full[4], empty[4];
  uint64_t code_full[3], code_empty[3];
  uint64_t s_full[2], p_half[2], p_ready[2], o_done[2];
  uint64_t q_full, q_empty, done, fin;
  float2 ml[2][kTile];  // each row's maximum and sum, where both streams hold the rows
};

template <int BITS>
constexpr int kBase = (sizeof(Smem<BITS>) + 1023) / 1024 * 1024 + 1024;
template <int BITS>
constexpr int kSmem = kBase<BITS> + 2 * kQ + Shape<BITS>::kStages * kStage + Shape<BITS>::kCodeStages * kCodeStage;
static_assert(kSmem<16> <= 227 * 1024 && kSmem<8> <= 227 * 1024, "shared memory of a CTA");

struct Maps {
  CUtensorMap q, k, v;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 16 bytes of row r, chunk c of a 128-byte-row tile in the 128-byte swizzle
__device__ __forceinline__ uint32_t swz(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

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

// One tile of one query row: S from tensor memory to weights over it, m and l of the
// row so far, and O when m moves.  The first 64 keys' weights are announced on `half`.
__device__ __forceinline__ void softmax_step(uint32_t ts, uint32_t to, bool masked, const Sees& sees, bool first,
                                             uint32_t half, float& m, float& l) {
  float x[kTile];
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int k = 0; k < 64; k += 32) tmem_ld32(ts + k, reinterpret_cast<uint32_t*>(x) + k);
  wait_ld();
#pragma unroll
  for (int k = 64; k < 128; k += 32) tmem_ld32(ts + k, reinterpret_cast<uint32_t*>(x) + k);  // while the first is looked at
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    if (part) wait_ld();
    if (masked) {
#pragma unroll
      for (int k = part * 64; k < part * 64 + 64; ++k)
        if (!((sees.w[k / 32] >> (k % 32)) & 1u)) x[k] = -INFINITY;
    }
#pragma unroll
    for (int k = part * 64; k < part * 64 + 64; k += 2) mx[(k / 2) & 3] = max3(mx[(k / 2) & 3], x[k], x[k + 1]);
  }
  const float top = max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
  if (first) {
    m = top;
  } else {
    const bool up = top > m + kLazy / kLogScale;
    if (__any_sync(0xffffffffu, up)) {
      // S of this step is complete, so O of the stream's step before it is too
      const float f = up ? ex2((m - top) * kLogScale) : 1.f;
      l *= f;
      if (up) m = top;
#pragma unroll 1
      for (int k = 0; k < kD; k += 16) {
        uint32_t o[16];
        tmem_ld16(to + k, o);
        wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        tmem_st16(to + k, o);
      }
    }
  }
  const float base = m == -INFINITY ? 0.f : m * kLogScale;
  const F2 base2(-base, -base), unit2(kLogScale, kLogScale);
  F2 ls[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
#pragma unroll
  for (int k = 0; k < kTile; k += 32) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float p0, p1;
      fma2(F2(x[k + 2 * i], x[k + 2 * i + 1]), unit2, base2).get(p0, p1);
      p0 = ex2(p0);
      p1 = ex2(p1);
      ls[i & 1] = add2(ls[i & 1], F2(p0, p1));
      w[i] = bf16x2(p0, p1);
    }
    tmem_st16(ts + k / 2, w);
    if (k == 32) {
      wait_st();
      fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(half);
    }
  }
  float l0, l1;
  add2(ls[0], ls[1]).get(l0, l1);
  l += l0 + l1;
}

// Sixteen words of this warp's rows, a row a lane, to sixteen bytes of four
// neighbouring rows a lane: lane q of four ends with the rows' q-th four words.
__device__ __forceinline__ void quads(uint32_t (&r)[16]) {
  const int q = threadIdx.x & 3;
#pragma unroll
  for (int u = 0; u < 4; u += 2)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t y = __shfl_xor_sync(0xffffffffu, q & 1 ? r[4 * u + i] : r[4 * u + 4 + i], 1);
      if (q & 1) r[4 * u + i] = y;
      else r[4 * u + 4 + i] = y;
    }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t y = __shfl_xor_sync(0xffffffffu, q & 2 ? r[i] : r[8 + i], 2);
    if (q & 2) r[i] = y;
    else r[8 + i] = y;
  }
}

// Four codes as two pairs of bf16, times 2^(e + 120) each (exact): the code's bits
// moved to a bf16 number's are 2^-120 of its value.
__device__ __forceinline__ uint32_t bf16_codes(uint32_t spread, uint32_t f0, uint32_t f1) {
  // spread: a code in the upper byte of each half
  const uint32_t bits = ((spread >> 4) & 0x07f007f0u) | (spread & 0x80008000u);
  uint32_t r;
  asm("{\n .reg .b32 t;\n mul.rn.bf16x2 t, %1, %2;\n mul.rn.bf16x2 %0, t, %3;\n}" : "=r"(r) : "r"(bits), "r"(f0), "r"(f1));
  return r;
}

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
      mbar_init(smem_u32(&sm.empty[i]), 1);
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
    }
    mbar_init(smem_u32(&sm.q_full), 1);
    mbar_init(smem_u32(&sm.q_empty), 1);
    mbar_init(smem_u32(&sm.done), 1);
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
  Walk& walk = sm.walk[warp];
  const Segment& g = walk.g;
  if (lane == 0) walk.begin(sm.plan);
  __syncwarp();
  auto next = [&] { return walk.next(sm.plan, a); };  // by one thread of the warp
  auto next_all = [&] {                               // by all of it
    __syncwarp();
    const bool more = __shfl_sync(0xffffffffu, lane == 0 && next(), 0);
    __syncwarp();
    return more;
  };

  if (warp < 4) {
    // registers: 128 x 80 + 256 x 208 of the launch's 384 x 168; 8-bit rows:
    // 256 x 48 + 256 x 208 of 512 x 128
    regs_fewer<BITS == 16 ? 80 : 48>();
    if (warp == 0) {
      if (elect_one()) {
        // ---- loads: K then V of every tile
        constexpr int kRing = BITS == 16 ? kStages : kCodeStages;
        uint64_t* full = BITS == 16 ? sm.full : sm.code_full;
        uint64_t* empty = BITS == 16 ? sm.empty : sm.code_empty;
        uint32_t stage = 0, phase = 0, issued = 0;
        const uint64_t policy = shared::evict_first_policy();
        bool ok = true;
        while (ok && next()) {
          const Place at = place_of(a, sm.plan, g);
          for (int t = g.tile0; ok && t < g.tile0 + g.tiles; ++t) {
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              ok = ok && mbar_wait(smem_u32(&empty[stage]), phase ^ 1, abort);
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
        }
        if (!ok) {  // the copies in flight must land before the CTA's shared memory is given up
          uint32_t never = 0;
          for (uint32_t k = issued > (uint32_t)kRing ? issued - kRing : 0; k < issued; ++k)
            mbar_wait(smem_u32(&full[k % kRing]), (k / kRing) & 1, &never);
        }
      }
    } else if (warp == 1) {
      if (elect_one()) {
        // ---- products.  Steps follow one another through all segments; a step's S is
        // issued before O of the step before, which is another stream's, so that the
        // tensor cores work while that one's softmax runs (of the same stream, O comes
        // first: S takes the place of P).  Products run in the order issued.
        constexpr uint32_t kDescS = mma_desc(1, 1, 0, kTile, kTile);
        constexpr uint32_t kDescO = mma_desc(1, 1, 1, kTile, kD);
        uint32_t seg = 0, p_phase = 0, tile_no = 0;
        bool ok = true;
        // the O that is still to be issued
        bool pend = false, p_dual = false, p_last = false, p_acc = false;
        int p_s = 0;
        uint32_t p_use = 0;
        auto flush = [&] {
          pend = false;
          const int s = p_s;
          const uint32_t st = p_use % kStages;
          const uint32_t pp = (p_phase >> s) & 1;
          p_phase ^= 1u << s;
          ok = (p_dual && s) || mbar_wait(smem_u32(&sm.full[st]), (p_use / kStages) & 1, abort);
          ok = ok && mbar_wait(smem_u32(&sm.p_half[s]), pp, abort);
          if (!ok) return;
          fence_after();
          const uint32_t vb = smem_desc(smem_u32(ring + st * kStage), kTile * 128);
          const uint32_t p = tmem + s * kTile, d = tmem + 2 * kTile + s * kD;
#pragma unroll
          for (int k = 0; k < 4; ++k) mma16_ts(d, p + k * 8, vb + (k * 16 * 128 >> 4), kDescO, p_acc | (k > 0));
          ok = mbar_wait(smem_u32(&sm.p_ready[s]), pp, abort);
          if (!ok) return;
          fence_after();
#pragma unroll
          for (int k = 4; k < 8; ++k) mma16_ts(d, p + k * 8, vb + (k * 16 * 128 >> 4), kDescO, 1);
          if (!p_dual || s) mma_commit(smem_u32(&sm.empty[st]));
          if (p_last) mma_commit(smem_u32(&sm.o_done[s]));
        };
        while (ok && next()) {
          // a segment's last O does not wait for the next one's rows of q
          if (pend && !mbar_try(smem_u32(&sm.q_full), seg & 1)) flush();
          ok = ok && mbar_wait(smem_u32(&sm.q_full), seg & 1, abort);
          if (!ok) break;
          const int steps = g.steps();
          for (int i = 0; ok && i < steps; ++i) {
            const int s = i & 1;
            const uint32_t use = 2 * (tile_no + (g.dual ? i >> 1 : i)), st = use % kStages;
            if (pend && p_s == s) flush();
            if (!g.dual || s == 0) ok = ok && mbar_wait(smem_u32(&sm.full[st]), (use / kStages) & 1, abort);
            if (!ok) break;
            fence_after();
            const uint32_t kb = smem_desc(smem_u32(ring + st * kStage), 16);
            const uint32_t qb = smem_desc(smem_u32(q_smem + (g.dual ? s : 0) * kQ), 16);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t o = ((k / 4) * (kTile * 128) + (k % 4) * 32) >> 4;
              mma16_ss(tmem + s * kTile, qb + o, kb + o, kDescS, k > 0);
            }
            mma_commit(smem_u32(&sm.s_full[s]));
            if (!g.dual || s) mma_commit(smem_u32(&sm.empty[st]));
            if (i == steps - 1) mma_commit(smem_u32(&sm.q_empty));
            if (pend) flush();
            pend = true;
            p_dual = g.dual;
            p_last = i + 2 >= steps;
            p_acc = i >= 2;
            p_s = s;
            p_use = use + 1;
          }
          tile_no += g.tiles;
          ++seg;
        }
        if (ok && pend) flush();
        // every product is complete before tensor memory is given up
        uint32_t never = 0;
        mma_commit(smem_u32(&sm.done));
        mbar_wait(smem_u32(&sm.done), 0, &never);
      }
    } else if (warp == 2) {
      if (elect_one()) {
        // ---- loads: the rows of q of every segment, once the products have read the last one's
        const uint32_t bytes = 128 * a.group * a.run, bar = smem_u32(&sm.q_full);
        const uint64_t policy = shared::evict_first_policy();
        uint32_t seg = 0;
        bool ok = true;
        while (ok && next()) {
          if (seg > 0) ok = mbar_wait(smem_u32(&sm.q_empty), (seg - 1) & 1, abort);
          if (!ok) break;
          const int n = g.dual ? 2 : 1;
          mbar_expect_tx(bar, 2 * n * bytes);
          for (int s = 0; s < n; ++s)
            for (int half = 0; half < 2; ++half)  // 64 channels each
              tma_load_3d(smem_u32(q_smem + s * kQ + half * (kTile * 128)), &maps.q, bar, half * 64, g.h * a.group,
                          g.token + s * a.run, policy);
          ++seg;
        }
        uint32_t never = 0;  // the last ones' landing is nobody's to wait for when another role gave up
        if (seg > 0) mbar_wait(bar, (seg - 1) & 1, &never);
      }
    }
  } else if (warp < 4 + kSoftmaxWarps) {
    // ---- softmax of stream s, a thread per row
    regs_more<208>();
    const int s = (warp - 4) >> 2, w4 = warp & 3, row = w4 * 32 + lane;
    const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
    const uint32_t ts = tmem + lanes + s * kTile, to = tmem + lanes + 2 * kTile + s * kD;
    const int tok = row * a.group_inv >> 16;  // of the stream's
    uint32_t tile_no = 0, s_phase = 0, o_phase = 0, fin_phase = 0;
    Cut cut = {};
    bool ok = true;
    while (ok && next_all()) {
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
      for (int j = 0; j < steps; ++j) {
        const int t = g.tile_of(s, j), key0 = t * kTile;
        ok = mbar_wait(smem_u32(&sm.s_full[s]), s_phase, abort);
        if (BITS == 16 && keys < key0 + kTile && (!g.dual || s == 0)) {
          // rows of V past the last key may hold anything: zeros, so that 0 x does not become NaN
          const uint32_t use = 2 * (tile_no + t - g.tile0) + 1, stage = use % kStages;
          ok = ok && mbar_wait(smem_u32(&sm.full[stage]), (use / kStages) & 1, abort);
          if (ok) {
            const int valid = max(0, keys - key0);
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
      if (steps > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.o_done[s]), o_phase, abort));
        if (!ok) break;
        o_phase ^= 1;
      }
      m *= kLogScale;
      float f0 = 1.f, f1 = 0.f;
      auto meet = [&] {  // of all softmax warps
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.fin));
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.fin), fin_phase, abort));
        fin_phase ^= 1;
        return ok;
      };
      const bool both = !g.dual && g.steps_of(1) > 0;
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
      if (g.dual || both || s == 0) {
        const int c0 = both ? s * 64 : 0, c1 = both ? c0 + 64 : kD;
        const uint32_t o0 = g.dual ? to : tmem + lanes + 2 * kTile;
        if (g.whole) {
          const float inv = l == 0.f ? 0.f : 1.f / l;  // a sum that is NaN stays one
          f0 *= inv;
          f1 *= inv;
        }
        auto load = [&](int k, uint32_t* o) {  // 16 channels of this thread's row
          tmem_ld16(o0 + k, o);
          if (both) {
            uint32_t v[16];
            tmem_ld16(o0 + kD + k, v);
            wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[i] = __float_as_uint(fmaf(__uint_as_float(o[i]), f0, __uint_as_float(v[i]) * f1));
          } else {
            wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f0);
          }
        };
        const int q = lane & 3;
        const int rows = min(a.run, g.tokens - first_tok) * a.group;
        if (g.whole) {
          uint16_t* dst[4];  // the four rows that the lane stores
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = row - q + i, x = r * a.group_inv >> 16;
            dst[i] = a.out + ((((int64_t)g.token + first_tok + x) * a.n_heads + g.h) * a.group + (r - x * a.group)) * kD + q * 8;
            if (r >= rows) dst[i] = nullptr;
          }
#pragma unroll 1
          for (int k = c0; k < c1; k += 32) {
            uint32_t o[32], w[16];
            load(k, o);
            load(k + 16, o + 16);
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = bf16x2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
            quads(w);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (dst[i])
                *reinterpret_cast<uint4*>(dst[i] + k) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          }
        } else {
          const int64_t at = (int64_t)g.slot() * a.slot_rows + (g.dual ? s * kTile : 0) + row;
          float* po = a.part_o + (at - q) * kD + q * 4;
#pragma unroll 1
          for (int k = c0; k < c1; k += 16) {
            uint32_t o[16];
            load(k, o);
            quads(o);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (row - q + i < rows)
                *reinterpret_cast<uint4*>(po + i * kD + k) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
          if (row < rows && c0 == 0) a.part_ml[at] = make_float2(m, l);
        }
      }
      cut = {g.token, g.h, g.tokens, g.pieces, 0};  // of the last segment
      fence_before();
      // O and the rows' maxima are read before the next segment's take their place
      if (both && !meet()) break;
    }
    if (a.split && s == 0 && row == 0) a.cuts[blockIdx.x] = cut;
  } else if constexpr (BITS == 8) {
    // ---- codes to bf16, all four warps each tile
    regs_fewer<48>();
    const int t128 = tid - 384, c = t128 & 7;
    uint32_t n = 0;
    bool ok = true;
    while (ok && next_all()) {
      const int keys = g.off + g.t;
      for (int t = g.tile0; ok && t < g.tile0 + g.tiles; ++t) {
        for (int kv = 0; kv < 2; ++kv, ++n) {
          const uint32_t from = n % kCodeStages, to = n % kStages;
          ok = mbar_wait(smem_u32(&sm.code_full[from]), (n / kCodeStages) & 1, abort) &&
               mbar_wait(smem_u32(&sm.empty[to]), ((n / kStages) & 1) ^ 1, abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const unsigned char* src = codes + from * kCodeStage;
          // of 16 codes, a row's c-th, as two 16-byte chunks; the upper half of a row
          // stores its odd chunk first, so that eight lanes' stores meet in no bank
          unsigned char* dst = ring + to * kStage + (c >> 2) * (kTile * 128);
          const int k0 = (c & 3) * 2 + (c >> 2), k1 = k0 ^ 1;
          const int valid = keys - t * kTile;
#pragma unroll 2
          for (int i = 0; i < 8; ++i) {
            const int r = i * 16 + (t128 >> 3);
            uint4 x = *reinterpret_cast<const uint4*>(src + r * 128 + c * 16);
            if (kv && r >= valid) x = make_uint4(0, 0, 0, 0);  // may hold anything: zeros, so that 0 x does not become NaN
            const int e = min(max((int)src[kCodes + r] - kExpBias, kExpMin), kExpMax);
            // 2^(e + 120) passes bf16's range: 2^60, then the rest
            const uint32_t f0 = (uint32_t)(60 + 127) << 7, f1 = (uint32_t)(e + 60 + 127) << 7;
            const uint32_t m0 = f0 | f0 << 16, m1 = f1 | f1 << 16;
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            uint32_t y[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              y[2 * k] = bf16_codes(__byte_perm(w[k], 0, 0x1404), m0, m1);
              y[2 * k + 1] = bf16_codes(__byte_perm(w[k], 0, 0x3424), m0, m1);
            }
            const bool odd = c >> 2;
            *reinterpret_cast<uint4*>(dst + swz(r, k0)) =
                odd ? make_uint4(y[4], y[5], y[6], y[7]) : make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(dst + swz(r, k1)) =
                odd ? make_uint4(y[0], y[1], y[2], y[3]) : make_uint4(y[4], y[5], y[6], y[7]);
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&sm.full[to]));
            mbar_arrive(smem_u32(&sm.code_empty[from]));
          }
        }
      }
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (tid == 0 && sm.abort) set_status(a.status, BPKV_DEV_TIMEOUT);
  if (warp == 2) tmem_dealloc(tmem, kTmemCols);
}

// The rows of units that were cut: out = sum_pieces 2^(m - M) o / sum_pieces 2^(m - M) l,
// a warp a row, eight pieces at a time.
constexpr int kJoinWarps = 8;
constexpr int kJoinDeep = 8;

__global__ void __launch_bounds__(kJoinWarps * 32) k_prompt_join(const __grid_constant__ Args a) {
  pdl_enter();
  const Cut cut = a.cuts[blockIdx.x];
  const int lane = threadIdx.x & 31, rows = cut.tokens * a.group;
  if (cut.pieces == 0) return;
  for (int r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5); r < rows; r += gridDim.y * kJoinWarps) {
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
          const int64_t at = (int64_t)(2 * (blockIdx.x + k) + (k == 0)) * a.slot_rows + in;
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
  size_t cuts, ml, o, total;
  int slot_rows;
};

Space space(int64_t tokens, int64_t group) {
  Space s;
  // of the tokens of a unit at most, a stream's 128 rows, or both streams'
  s.slot_rows = tokens <= kTile / group ? kTile : kRows;
  size_t off = 256;  // status word
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
  a.status = static_cast<int32_t*>(ws);
  // units and their tiles at most
  const int64_t units = a.n_heads * (a.tokens / (2 * a.run) + min64(a.n_seq, a.tokens));
  const int64_t tiles = max64(1, (keys + kTile - 1) / kTile);
  a.split = tiles > 4;
  const int ctas = (int)max64(1, min64(kSms, a.split ? units * (tiles + 1) / 2 : units));
  static std::atomic<uint64_t> done;
  cudaError_t e = shared::allow_smem(k_prompt<BITS>, kSmem<BITS>, done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k_prompt<BITS>, dim3(ctas), dim3(Shape<BITS>::kThreads), (size_t)kSmem<BITS>, st, a, maps);
  if (e != cudaSuccess || !a.split) return e;
  return launch_pdl(k_prompt_join, dim3(ctas, 4), dim3(kJoinWarps * 32), 0, st, a);
}

}  // namespace

}  // namespace prompt

using namespace prompt;

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
  if (!map_q(&maps.q, p.q, T, H * p.group, p.ld_q, p.group, kTile / p.group)) return cudaErrorInvalidValue;
  if (p.cache) return over_cache<16>(a, maps, rows_of(*p.cache), T, ws, st);
  if (p.rows8) return over_cache<8>(a, maps, rows_of(*p.rows8), T, ws, st);
  const bool by_token = p.ld_k != 0;
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
  constexpr int BITS = sizeof(C) == sizeof(bpkv_cache) ? 16 : 8;
  return over_cache<BITS>(a, maps, rows_of(c), t, ws, st);
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
