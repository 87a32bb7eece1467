// Attention of many query rows over a shared prefix, on the 5th-generation
// tensor cores (the wide half of bpkv_shared_attend over bf16 rows and
// bpkv_shared_attend8 over 8-bit rows; the plan is in shared_plan.cuh).
//
// A segment.  One thread loads K and V tiles by TMA into a ring of shared
// memory stages, one thread issues the products, and two groups of four warps
// do the softmax, a thread per query row: S = Q K^T (128 x 128 x 128) into
// tensor memory, p = exp2(S - m) written back over S as the A operand of
// O += P V, with O in tensor memory too.  p is rounded to bf16 there (2^-8),
// since a product's operands have one type and V is bf16; S, m, O and the sum of
// the unrounded p are float32.  The groups are two streams that take
// turns at the tensor cores: with more than 128 rows each has its own 128 rows
// and both take every tile; with fewer both hold the same rows and each takes
// every other tile.  Rows that fill half or a quarter of the 128 are held twice
// or four times (the instruction takes 128), each copy's threads weighing their
// share of the tile's tokens; the copies are joined when the segment ends.  m
// only follows the maximum when that has risen by a factor of 2^kLazy, so O is
// seldom rescaled.
//
// What bounds it: with 256 rows the chain S -> softmax (about 1650 cycles) -> O,
// of which two streams hide half: the tensor cores are busy 65% of the time.
// Measured on a GB300 with 128 sequences of 8 x 4 heads over one prefix of
// 131072 tokens: 195 us for this kernel, 1.41 PFLOP/s; with 32 over 32768 tokens
// 25 us, 5.4 TB/s.  8-bit rows, 16 sequences of 4 x 8 heads over two prefixes of
// 131071 tokens: 72 us, 3.7 TB/s, bound by the softmax with its scales.
//
// 8-bit rows.  The products take the codes as they lie.  q becomes two e4m3
// pieces of 4 bits under a power-of-two scale of its row, which is all of a
// bf16 number above 2^-9 of the row's largest.  K's scales multiply S; V's
// scales join the exponent, a = S 2^ek + ev, so that p' = p 2^ev is what the
// product needs and p = p' 2^-ev is what the sum needs.  p' becomes two e5m2
// pieces, together good to 2^-6 (0.25% in the mean square) over the range of a
// half.
#include "rows8_core.cuh"
#include "shared_plan.cuh"
#include "shared_ring.cuh"
#include "tc.cuh"

namespace bpkv {
namespace shared {

template <int BITS>
cudaError_t launch_few(const Args& a, int64_t whole, int64_t own_max, bool wait_first, uint16_t* out, cudaStream_t st);
int few_tile(int bits);
int unit_split(int64_t units, int64_t tokens);

namespace {

using namespace tc;
using namespace wide;

constexpr int kThreads = 128 + 32 * kSoftmaxWarps;
constexpr uint32_t kTmemCols = 512;              // S of both streams, then O of both
constexpr float kLogScale = 0.08838834764831845f * 1.4426950408889634f;  // log2(e) / sqrt(D)

// How far the maximum may pass m before O is rescaled, and where exp2's
// results sit: bf16 P has float32's range; e5m2 pieces lie in 2^-16 .. 1.75 2^15.
template <int BITS>
struct Range {
  static constexpr float kLazy = BITS == 16 ? 8.f : 4.f;
  static constexpr float kShift = BITS == 16 ? 0.f : 11.f;
};

struct Maps {
  CUtensorMap m[2];  // K, V
};

// One CTA's part of a unit.
struct Segment {
  int32_t index;  // prefix
  int32_t h;      // KV head
  int32_t rows;   // query rows of the unit
  int32_t row0;   // its first among the prefix's
  bool dual;      // both streams take every tile
  int64_t unit;
  int64_t tile0;  // first tile
  int32_t tiles;
  int64_t tokens;  // of the whole unit
  __device__ int steps() const { return dual ? 2 * tiles : tiles; }
  __device__ int steps_of(int s) const { return dual ? tiles : (tiles + 1 - s) / 2; }
  __device__ int tile_of(int s, int j) const { return dual ? j : 2 * j + s; }
  __device__ int rows_of(int s) const { return dual ? (s ? rows - kTile : kTile) : rows; }
  __device__ int copies() const { return dual ? 1 : copies_of(rows); }
  // tokens of the segment's tile t that exist
  __device__ int valid(int t) const { return (int)min64(kTile, tokens - (tile0 + t) * kTile); }
};

// Walks the segments of one CTA; every role of the CTA walks alike.
struct Walk {
  const WidePlan& p;
  const Args& a;
  int64_t pos, end;
  int item;
  __device__ Walk(const WidePlan& plan, const Args& args) : p(plan), a(args) {
    const Share share(p.wide[p.n_pre] * a.n_heads, a.wide_ctas);
    pos = end = 0;
    item = 0;
    if ((int64_t)blockIdx.x >= share.n) return;
    pos = share.lo(blockIdx.x);
    end = share.lo(blockIdx.x + 1);
    int lo = 0, hi = p.n_pre - 1;  // the last item that begins at or before pos
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (p.wide[mid] * a.n_heads <= pos) lo = mid;
      else hi = mid - 1;
    }
    item = lo;
  }
  __device__ bool next(Segment& s) {
    if (pos >= end) return false;
    while (p.wide[item + 1] * a.n_heads <= pos) ++item;
    const int64_t tiles = p.wide[item + 1] - p.wide[item];
    const int64_t off = pos - p.wide[item] * a.n_heads;
    s.h = (int)quot(off, tiles);
    s.tile0 = off - s.h * tiles;
    s.tiles = (int)min64(tiles - s.tile0, end - pos);
    s.index = p.it_p[item];
    s.row0 = (item - p.item0[s.index]) * kPair;
    s.rows = pre_rows(a, p, item);
    s.tokens = p.tok[s.index];
    s.unit = (int64_t)item * a.n_heads + s.h;
    s.dual = s.rows > kTile;
    pos += s.tiles;
    return true;
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes of row r, chunk c of a 128-byte-row tile in the 128-byte swizzle
__device__ __forceinline__ uint32_t swz(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// The rows of q of one stream into shared memory, by n threads (t): all rows'
// copies are issued, then awaited.  For 8-bit products a row's sixteen lanes
// turn what they copied, in place, into two e4m3 pieces under a power of two:
// x 2^-e with the row's largest magnitude in 128 .. 256, hi to 4 bits, lo the 4
// (with its sign) below.
template <int BITS>
__device__ __forceinline__ void load_q(const Args& a, const WidePlan& p, const Segment& g, int s, int t, int n,
                                       unsigned char* dst, float* qf) {
  const int l16 = t & 15, rows = g.rows_of(s), span = kTile / g.copies();
  const uint32_t base = g.row0 + (g.dual ? s * kTile : 0), first = p.first[g.index], group = a.group;
  unsigned char* half = dst + (l16 / 8) * (kTile * 128);
  const uint16_t* q = a.q + (int64_t)g.h * a.group * kD + l16 * 8;
  const uint32_t seq_step = a.n_heads * a.group * kD;
#pragma unroll 4
  for (int r = t / 16; r < kTile; r += n / 16) {
    const uint32_t of = r & (span - 1);
    if ((int)of < rows) {
      const uint32_t x = base + of, i = x * a.group_inv >> 16, seq = p.order[first + i];
      cp_async16(half + (BITS == 16 ? swz(r, l16 & 7) : (uint32_t)(r * 128 + (l16 & 7) * 16)),
                 q + (uint64_t)seq * seq_step + (x - i * group) * kD);
    }
  }
  cp_async_commit();
  cp_async_wait_all();
  if constexpr (BITS == 8) {
#pragma unroll 1
    for (int r = t / 16; r < kTile; r += n / 16) {
      const uint4 w = *reinterpret_cast<const uint4*>(half + r * 128 + (l16 & 7) * 16);
      uint32_t m = abs_max(w);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
      m = max(m & 0xffffu, m >> 16);
      const int e = max(-100, (int)(m >> 7) - 127 - 7);
      const float f = exp2i(-e);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x0 = __uint_as_float(ww[i] << 16) * f, x1 = __uint_as_float(ww[i] & 0xffff0000u) * f;
        hi[i] = e4m3x2(x0, x1);
        const float2 y = __half22float2(half2_of_e4m3x2((uint16_t)hi[i]));
        lo[i] = e4m3x2(x0 - y.x, x1 - y.y);
      }
      __syncwarp();  // the row's lanes have read it
      if ((r & (span - 1)) < rows) {
        const uint32_t at = swz(r, l16 >> 1) + (l16 & 1) * 8;
        *reinterpret_cast<uint2*>(dst + at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
        *reinterpret_cast<uint2*>(dst + kTile * 128 + at) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
        if (l16 == 0) qf[r] = exp2i(e);
      }
    }
  }
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, float* x) {
#pragma unroll
  for (int k = 0; k < N; k += 32) tmem_ld32(addr + k, reinterpret_cast<uint32_t*>(x) + k);
}

// One tile of one query row: S from tensor memory, this thread's COLS columns
// (the copy-th) to weights over it, zeros to the other copies'; m and l of the
// row's columns so far, and O when m moves.  With one copy the first 64 tokens'
// weights are announced on `half` as soon as they are there.
template <int BITS, int COLS>
__device__ __forceinline__ void softmax_step(uint32_t ts, uint32_t to, int copy, int valid, bool first, float qf,
                                             const float* scales, uint32_t half, float& m, float& l) {
  const int c0 = copy * COLS;
  float x[COLS];
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  constexpr int kParts = COLS > 64 ? 2 : 1, kPer = COLS / kParts;
  tmem_ld<kPer>(ts + c0, x);
  wait_ld();
  if constexpr (kParts == 2) tmem_ld<kPer>(ts + kPer, x + kPer);  // comes while the first part is looked at
#pragma unroll
  for (int part = 0; part < kParts; ++part) {
    if (part) wait_ld();
    if constexpr (BITS == 8) {
      const F2 q2(qf, qf);
#pragma unroll
      for (int k = part * kPer; k < (part + 1) * kPer; k += 4) {
        const float4 kf = *reinterpret_cast<const float4*>(scales + c0 + k);
        const float4 ev = *reinterpret_cast<const float4*>(scales + kTile + c0 + k);
        fma2(mul2(F2(x[k], x[k + 1]), F2(kf.x, kf.y)), q2, F2(ev.x, ev.y)).get(x[k], x[k + 1]);
        fma2(mul2(F2(x[k + 2], x[k + 3]), F2(kf.z, kf.w)), q2, F2(ev.z, ev.w)).get(x[k + 2], x[k + 3]);
      }
    }
    if (valid < c0 + COLS) {
#pragma unroll
      for (int k = part * kPer; k < (part + 1) * kPer; ++k)
        if (c0 + k >= valid) x[k] = -INFINITY;
    }
#pragma unroll
    for (int k = part * kPer; k < (part + 1) * kPer; k += 2) mx[(k / 2) & 3] = max3(mx[(k / 2) & 3], x[k], x[k + 1]);
  }
  const float top = max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
  constexpr float kUnit = BITS == 16 ? kLogScale : 1.f;  // x times this is in powers of two
  if (first) {
    m = top;
  } else {
    const bool up = top > lazy_top<BITS>(m, Range<BITS>::kLazy / kUnit);
    if (__any_sync(0xffffffffu, up)) {
      // S of this step is complete, so O of the stream's step before it is too
      const float f = up ? ex2((m - top) * kUnit) : 1.f;
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
  const float base = m == -INFINITY ? 0.f : shifted<BITS>(m, kUnit, Range<BITS>::kShift);
  const F2 base2(-base, -base), unit2(kUnit, kUnit);
  F2 ls[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
#pragma unroll
  for (int k = 0; k < COLS; k += 32) {
    float p[32];
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const F2 v(x[k + i], x[k + i + 1]);
      const F2 e = BITS == 16 ? fma2(v, unit2, base2) : add2(v, base2);
      e.get(p[i], p[i + 1]);
      p[i] = ex2(p[i]);
      p[i + 1] = ex2(p[i + 1]);
    }
    if constexpr (BITS == 16) {
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        ls[i & 1] = add2(ls[i & 1], F2(p[2 * i], p[2 * i + 1]));
        const __nv_bfloat162 h = __floats2bfloat162_rn(p[2 * i], p[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      tmem_st16(ts + (c0 + k) / 2, w);
    } else {
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 iv = *reinterpret_cast<const float4*>(scales + 2 * kTile + c0 + k + i * 4);
        ls[0] = fma2(F2(p[4 * i], p[4 * i + 1]), F2(iv.x, iv.y), ls[0]);
        ls[1] = fma2(F2(p[4 * i + 2], p[4 * i + 3]), F2(iv.z, iv.w), ls[1]);
        // the upper byte of a half is the e5m2 number below it: adding half a
        // step first rounds (p is positive, the rest has a sign)
        uint32_t h[2], r[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const __half2 v = __floats2half2_rn(p[4 * i + 2 * c], p[4 * i + 2 * c + 1]);
          h[c] = (*reinterpret_cast<const uint32_t*>(&v) + 0x00800080u) & 0xff00ff00u;
          const __half2 d = __hsub2(v, *reinterpret_cast<const __half2*>(&h[c]));
          r[c] = *reinterpret_cast<const uint32_t*>(&d) + 0x00800080u;
        }
        hi[i] = __byte_perm(h[0], h[1], 0x7531);
        lo[i] = __byte_perm(r[0], r[1], 0x7531);
      }
      tmem_st8(ts + (c0 + k) / 4, hi);
      tmem_st8(ts + 32 + (c0 + k) / 4, lo);
    }
    if (COLS > 64 && k == 32) {
      wait_st();
      fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(half);
    }
  }
  if constexpr (COLS < kTile) {
    const uint32_t zero[16] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k)  // 32 columns each
      if (k * 32 / COLS != copy) {
        if constexpr (BITS == 16) {
          tmem_st16(ts + k * 16, zero);
        } else {
          tmem_st8(ts + k * 8, zero);
          tmem_st8(ts + 32 + k * 8, zero);
        }
      }
  }
  float l0, l1;
  add2(ls[0], ls[1]).get(l0, l1);
  l += l0 + l1;
}

// Sixteen columns of this warp's rows, a row a lane, to sixteen bytes of four
// neighbouring rows a lane: lane q of four ends with the rows' q-th four columns.
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

template <int BITS>
__global__ void __launch_bounds__(kThreads, 1) k_shared_wide(const __grid_constant__ Args a,
                                                             const __grid_constant__ Maps maps) {
  extern __shared__ __align__(1024) unsigned char raw[];
  Smem<BITS>& sm = *reinterpret_cast<Smem<BITS>*>(raw);
  unsigned char* q_smem = raw + ((smem_u32(raw) + sizeof(Smem<BITS>) + 1023) / 1024 * 1024 - smem_u32(raw));
  using S = Shape<BITS>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_stage = a.stages;
  const bool any_dual = a.n_seq * a.group > kTile;
  unsigned char* ring = q_smem + (any_dual ? 2 : 1) * S::kQ;
  unsigned char* ring_exps = ring + n_stage * S::kStage;  // [stage][K bytes, V bytes]
  volatile uint32_t* abort = &sm.abort;

  if (tid == 0) {
    sm.abort = 0;
    for (int i = 0; i < n_stage; ++i) {
      mbar_init(smem_u32(&sm.full[i]), 1);
      mbar_init(smem_u32(&sm.empty[i]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sm.s_full[s]), 1);
      mbar_init(smem_u32(&sm.p_half[s]), 4);
      mbar_init(smem_u32(&sm.p_ready[s]), 4);
      mbar_init(smem_u32(&sm.o_done[s]), 1);
      mbar_init(smem_u32(&sm.sc_go[s]), 4);
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_u32(&sm.sc_full[s][b]), 1);
        mbar_init(smem_u32(&sm.sc_empty[s][b]), 4);
      }
    }
    mbar_init(smem_u32(&sm.q_full), kSoftmaxWarps);
    mbar_init(smem_u32(&sm.q_empty), 1);
    mbar_init(smem_u32(&sm.fin), kSoftmaxWarps);
    mbar_init(smem_u32(&sm.done), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_shared();
  }
  if (warp == 2) tmem_alloc(smem_u32(&sm.tmem), kTmemCols);
  if (warp == 3 && lane < 2) prefetch_map(&maps.m[lane]);
  fence_before();
  // the streaming kernel may start once this one has seen all earlier work complete
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  make_plan(a, sm.plan, kTile);  // ends with a barrier of the CTA
  fence_after();
  const uint32_t tmem = sm.tmem;
  Walk walk(sm.plan, a);
  Segment g;

  if (a.finish && (warp == 2 || warp == 3)) {
    const int64_t n = (int64_t)a.n_seq * a.n_heads * a.group;
    for (int64_t r = blockIdx.x + (int64_t)gridDim.x * (tid - 64); r < n; r += (int64_t)gridDim.x * 64)
      a.parts[r] = parts_of(a, sm.plan, r);
  }
  if (warp < 4) {
    // registers: 128 x 80 + 256 x 208 of the launch's 384 x 168
    regs_fewer<80>();
    if (warp == 0) {
      if (elect_one()) {
        // ---- loads: K then V of every tile
        uint32_t stage = 0, phase = 0, issued = 0;
        const uint64_t policy = evict_first_policy();
        bool ok = true;
        while (ok && walk.next(g)) {
          const int64_t base = (int64_t)g.index * a.n_heads + g.h;
          for (int t = 0; ok && t < g.tiles; ++t) {
            const int64_t tok = (g.tile0 + t) * kTile;
  #pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              ok = ok && mbar_wait(smem_u32(&sm.empty[stage]), phase ^ 1, abort);
              if (!ok) break;
              const uint32_t bar = smem_u32(&sm.full[stage]);
              const uint32_t dst = smem_u32(ring + stage * S::kStage);
              mbar_expect_tx(bar, S::kStage + (kv ? S::kExps : 0));
              if constexpr (BITS == 16) {
                tma_load_4d(dst, &maps.m[kv], bar, 0, (int)tok, 0, (int)base, policy);
              } else {
                tma_load_3d(dst, &maps.m[kv], bar, 0, (int)tok, (int)base, policy);
                if (kv) {
                  const uint32_t e = smem_u32(ring_exps + stage * S::kExps);
                  bulk_load(e, a.exps[0][0] + base * a.pcap + tok, kTile, bar);
                  bulk_load(e + kTile, a.exps[0][1] + base * a.pcap + tok, kTile, bar);
                }
              }
              ++issued;
              if (++stage == (uint32_t)n_stage) stage = 0, phase ^= 1;
            }
          }
        }
        if (!ok) {  // the copies in flight must land before the CTA's shared memory is given up
          uint32_t never = 0;
          for (uint32_t k = issued > (uint32_t)n_stage ? issued - n_stage : 0; k < issued; ++k)
            mbar_wait(smem_u32(&sm.full[k % n_stage]), (k / n_stage) & 1, &never);
        }
      }
    } else if (warp == 1) {
      if (elect_one()) {
        // ---- products.  Step i of a segment is stream i & 1; S of step i is
        // issued before O of step i - 1, so the tensor cores work while the
        // other stream's softmax runs.  Products run in the order issued: S(i)
        // overwrites P(i - 2) only after O(i - 2) has read it.
        constexpr uint32_t kDescS = BITS == 16 ? mma_desc(1, 1, 0, kTile, kTile) : mma_desc(0, 0, 0, kTile, kTile);
        constexpr uint32_t kDescO = BITS == 16 ? mma_desc(1, 1, 1, kTile, kD) : mma_desc(1, 0, 1, kTile, kD);
        uint32_t seg = 0, p_phase = 0;
        bool ok = true;
        uint32_t k_st = 0, k_ph = 0, v_st = 1, v_ph = 0;
        auto skip = [&](uint32_t& st, uint32_t& ph) {  // two stages on
          st += 2;
          if (st >= (uint32_t)n_stage) st -= n_stage, ph ^= 1;
        };
        while (ok && walk.next(g)) {
          ok = mbar_wait(smem_u32(&sm.q_full), seg & 1, abort);
          if (!ok) break;
          const int steps = g.steps();
          for (int i = 0; ok && i <= steps; ++i) {
            if (i < steps) {
              const int s = i & 1;
              const uint32_t st = k_st;
              if (!g.dual || s == 0) {
                ok = mbar_wait(smem_u32(&sm.full[st]), k_ph, abort);
                if (!ok) break;
              }
              fence_after();
              const uint32_t kb = smem_desc(smem_u32(ring + st * S::kStage), 16);
              const uint32_t qb = smem_desc(smem_u32(q_smem + (g.dual ? s : 0) * S::kQ), 16);
              const uint32_t d = tmem + s * kTile;
              if constexpr (BITS == 16) {
  #pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const uint32_t o = ((k / 4) * (kTile * 128) + (k % 4) * 32) >> 4;
                  mma16_ss(d, qb + o, kb + o, kDescS, k > 0);
                }
              } else {
  #pragma unroll
                for (int k = 0; k < 8; ++k)  // both pieces of q against the same codes
                  mma8_ss(d, qb + (((k / 4) * (kTile * 128) + (k % 4) * 32) >> 4), kb + ((k % 4) * 32 >> 4), kDescS, k > 0);
              }
              mma_commit(smem_u32(&sm.s_full[s]));
              if (!g.dual || s) {
                mma_commit(smem_u32(&sm.empty[st]));
                skip(k_st, k_ph);
              }
              if (i == steps - 1) mma_commit(smem_u32(&sm.q_empty));
            }
            if (i > 0) {
              const int j = i - 1, s = j & 1;
              const uint32_t st = v_st;
              const uint32_t pp = (p_phase >> s) & 1;
              p_phase ^= 1u << s;
              ok = (g.dual && s) || mbar_wait(smem_u32(&sm.full[st]), v_ph, abort);
              ok = ok && mbar_wait(smem_u32(&sm.p_half[s]), pp, abort);
              if (!ok) break;
              fence_after();
              const uint32_t vb = smem_desc(smem_u32(ring + st * S::kStage), BITS == 16 ? kTile * 128 : 16);
              const uint32_t p = tmem + s * kTile, d = tmem + 2 * kTile + s * kD;
              const uint32_t acc = j >= 2;
  #pragma unroll
              for (int h = 0; h < 2; ++h) {  // 64 tokens each
                if (h) {
                  ok = mbar_wait(smem_u32(&sm.p_ready[s]), pp, abort);
                  if (!ok) break;
                  fence_after();
                }
  #pragma unroll
                for (int i = 0; i < 4; ++i) {
                  if (BITS == 16) {
                    const int k = h * 4 + i;
                    mma16_ts(d, p + k * 8, vb + (k * 16 * 128 >> 4), kDescO, acc | (h | i));
                  } else {  // two products of the high pieces, two of the low
                    const int k = h * 2 + (i & 1);
                    mma8_ts(d, p + (i >> 1) * 32 + k * 8, vb + (k * 32 * 128 >> 4), kDescO, acc | (h | i));
                  }
                }
              }
              if (!ok) break;
              if (!g.dual || s) {
                mma_commit(smem_u32(&sm.empty[st]));
                skip(v_st, v_ph);
              }
              if (j + 2 >= steps) mma_commit(smem_u32(&sm.o_done[s]));
            }
          }
          ++seg;
        }
        // every product is complete before tensor memory is given up
        uint32_t never = 0;
        mma_commit(smem_u32(&sm.done));
        mbar_wait(smem_u32(&sm.done), 0, &never);
      }
    } else {
      if constexpr (BITS == 8) {
        // ---- warp 2 + s: the scales of stream s's tiles as floats.  It begins a
        // segment when the stream does, and in it keeps at most two of the stream's
        // tiles ahead of the softmax (sc_empty): further ahead, a stage's phase bit
        // could be that of an earlier fill (kMaxStages).
        const int s = warp - 2;
        uint32_t tile_no = 0, n = 0, go = 0;
        bool ok = true;
        while (ok && walk.next(g)) {
          const int steps = g.steps_of(s);
          if (steps > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.sc_go[s]), go, abort));
            if (!ok) break;
            go ^= 1;
          }
          for (int j = 0; j < steps; ++j, ++n) {
            const int t = g.tile_of(s, j), b = n & 1;
            const uint32_t use = 2 * (tile_no + t) + 1, st = use % n_stage;
            ok = mbar_wait(smem_u32(&sm.sc_empty[s][b]), ((n >> 1) & 1) ^ 1, abort) &&
                 mbar_wait(smem_u32(&sm.full[st]), (use / n_stage) & 1, abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t* e = reinterpret_cast<const uint32_t*>(ring_exps + st * S::kExps);
            const uint32_t ke = e[lane], ve = e[kTile / 4 + lane];
            const int valid = g.valid(t) - lane * 4;
            float kf[4], ev[4], iv[4];
  #pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int k = min(max((int)((ke >> (8 * i)) & 0xff) - kExpBias, kExpMin), kExpMax);
              const int v = min(max((int)((ve >> (8 * i)) & 0xff) - kExpBias, kExpMin), kExpMax);
              kf[i] = i < valid ? exp2i(k) * kLogScale : 0.f;
              ev[i] = i < valid ? (float)v : 0.f;
              iv[i] = i < valid ? exp2i(-v) : 0.f;
            }
            *reinterpret_cast<float4*>(&sm.sc.tok[s][b][0][lane * 4]) = make_float4(kf[0], kf[1], kf[2], kf[3]);
            *reinterpret_cast<float4*>(&sm.sc.tok[s][b][1][lane * 4]) = make_float4(ev[0], ev[1], ev[2], ev[3]);
            *reinterpret_cast<float4*>(&sm.sc.tok[s][b][2][lane * 4]) = make_float4(iv[0], iv[1], iv[2], iv[3]);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.sc_full[s][b]));
          }
          tile_no += g.tiles;
        }
      }
    }
  } else {
    // ---- softmax of stream s, a thread per row
    regs_more<208>();
    const int s = (warp - 4) >> 2, w4 = warp & 3, row = w4 * 32 + lane;
    const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
    const uint32_t ts = tmem + lanes + s * kTile, to = tmem + lanes + 2 * kTile + s * kD;
    uint32_t tile_no = 0, seg = 0, s_phase = 0, o_phase = 0, fin_phase = 0, n = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
      if (seg > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.q_empty), (seg - 1) & 1, abort));
        if (!ok) break;
      }
      float* qfs = nullptr;
      if constexpr (BITS == 8) qfs = sm.sc.qf[seg & 1][g.dual ? s : 0];
      load_q<BITS>(a, sm.plan, g, s, g.dual ? row : tid - 128, g.dual ? 128 : 256, q_smem + (g.dual ? s : 0) * S::kQ, qfs);
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.q_full));
      // also keeps a stream without a tile here from arriving for the next segment early
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.q_full), seg & 1, abort));
      if (!ok) break;
      const float qf = BITS == 8 ? qfs[row] : 1.f;
      const int rows = g.rows_of(s), steps = g.steps_of(s), copies = g.copies();
      const int r = row & (kTile / copies - 1), copy = row / (kTile / copies);  // this thread's row of the unit
      if (BITS == 8 && steps > 0 && lane == 0) mbar_arrive(smem_u32(&sm.sc_go[s]));
      const bool active = r - lane < rows;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < steps; ++j, ++n) {
        const int t = g.tile_of(s, j), valid = g.valid(t), b = n & 1;
        ok = mbar_wait(smem_u32(&sm.s_full[s]), s_phase, abort);
        if (BITS == 8) ok = ok && mbar_wait(smem_u32(&sm.sc_full[s][b]), (n >> 1) & 1, abort);
        if (valid < kTile && (!g.dual || s == 0)) {
          // rows of V past the last token may hold anything: zeros, so that 0 x does not become NaN
          const uint32_t use = 2 * (tile_no + t) + 1, stage = use % n_stage;
          ok = ok && mbar_wait(smem_u32(&sm.full[stage]), (use / n_stage) & 1, abort);
          if (ok) {
            constexpr int kChunks = BITS == 16 ? 16 : 8;  // 16-byte pieces of a row
            for (int x = row; x < (kTile - valid) * kChunks; x += kTile) {
              const int v = valid + x / kChunks, c = x % kChunks;
              *reinterpret_cast<uint4*>(ring + stage * S::kStage + (c / 8) * (kTile * 128) + v * 128 + (c % 8) * 16) =
                  make_uint4(0, 0, 0, 0);
            }
            fence_async_shared();
            __syncwarp();  // the first half's announcement is for these too
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        s_phase ^= 1;
        const bool whole = copies == 1 && active;
        if (active) {
          fence_after();
          const float* scales = nullptr;
          if constexpr (BITS == 8) scales = sm.sc.tok[s][b][0];
          const uint32_t half = smem_u32(&sm.p_half[s]);
          if (copies == 1) softmax_step<BITS, 128>(ts, to, 0, valid, j == 0, qf, scales, half, m, l);
          else if (copies == 2) softmax_step<BITS, 64>(ts, to, copy, valid, j == 0, qf, scales, half, m, l);
          else softmax_step<BITS, 32>(ts, to, copy, valid, j == 0, qf, scales, half, m, l);
          wait_st();
          fence_before();
        }
        __syncwarp();
        if (lane == 0) {
          if (!whole) mbar_arrive(smem_u32(&sm.p_half[s]));
          mbar_arrive(smem_u32(&sm.p_ready[s]));
          if (BITS == 8) mbar_arrive(smem_u32(&sm.sc_empty[s][b]));
        }
      }
      if (!ok) break;
      if (steps > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.o_done[s]), o_phase, abort));
        if (!ok) break;
        o_phase ^= 1;
      }
      m *= BITS == 16 ? kLogScale : 1.f;
      // Streams that hold the same rows join them, each half of the channels, and
      // so do a row's copies: the upper half of the copies through shared memory
      // (the rows of q, which are read), then of four the second.
      float f0 = 1.f, f1 = 0.f;
      auto meet = [&] {  // of all softmax warps
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.fin));
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.fin), fin_phase, abort));
        fin_phase ^= 1;
        return ok;
      };
      if (!g.dual) {
        sm.ml[s][row] = make_float2(m, l);
        if (!meet()) break;
        m = -INFINITY;
        for (int c = r; c < kTile; c += kTile / copies) m = fmaxf(m, fmaxf(sm.ml[0][c].x, sm.ml[1][c].x));
        l = 0.f;
        for (int c = r; c < kTile; c += kTile / copies) {
          const float2 a0 = sm.ml[0][c], a1 = sm.ml[1][c];
          const float g0 = a0.y == 0.f ? 0.f : ex2(a0.x - m), g1 = a1.y == 0.f ? 0.f : ex2(a1.x - m);
          if (c == row) f0 = g0, f1 = g1;
          l += g0 * a0.y + g1 * a1.y;
        }
      }
      fence_after();
      const int c0 = g.dual ? 0 : s * 64, c1 = g.dual ? kD : c0 + 64;
      const uint32_t o0 = g.dual ? to : tmem + lanes + 2 * kTile;
      const bool both = !g.dual && g.steps_of(1) > 0;
      auto own = [&](int k, uint32_t (&o)[16]) {  // 16 channels of this thread's row
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
          if (copies > 1) {
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f0);
          }
        }
      };
      // 16 bytes of a slot, one of 64 rows of this stream's channels
      auto slot = [&](int x, int k, int i) {
        return reinterpret_cast<float4*>(q_smem + s * (kTile * kD) + x * 256 + (((((k - c0) >> 2) + i) ^ (x & 15)) << 4));
      };
      auto put = [&](int x, int k, const uint32_t (&o)[16]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *slot(x, k, i) = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                       __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
      };
      auto add = [&](int x, int k, uint32_t (&o)[16]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = *slot(x, k, i);
          o[4 * i] = __float_as_uint(__uint_as_float(o[4 * i]) + v.x);
          o[4 * i + 1] = __float_as_uint(__uint_as_float(o[4 * i + 1]) + v.y);
          o[4 * i + 2] = __float_as_uint(__uint_as_float(o[4 * i + 2]) + v.z);
          o[4 * i + 3] = __float_as_uint(__uint_as_float(o[4 * i + 3]) + v.w);
        }
      };
      uint32_t o[16];
      if (copies > 1) {
        if (active && copy >= copies / 2) {
#pragma unroll 1
          for (int k = c0; k < c1; k += 16) {
            own(k, o);
            put(row - kTile / 2, k, o);
          }
        }
        if (!meet()) break;
        if (copies == 4) {
          if (active && copy == 1) {
#pragma unroll 1
            for (int k = c0; k < c1; k += 16) {
              own(k, o);
              add(row, k, o);
              put(row, k, o);
            }
          }
          if (!meet()) break;
        }
      }
      if (active && copy == 0) {
        const int64_t at = wide_row(g.unit, blockIdx.x) + (g.dual ? s * kTile : 0) + row;
        const int q = lane & 3;
        float* po = a.part_o + (at - q) * kD + q * 4;
#pragma unroll 1
        for (int k = c0; k < c1; k += 16) {
          own(k, o);
          if (copies > 1) add(row, k, o);
          if (copies == 4) add(row + 32, k, o);
          quads(o);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (r - q + i < rows)
              *reinterpret_cast<uint4*>(po + i * kD + k) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
        if ((g.dual || s == 0) && r < rows) a.part_ml[at] = make_float2(m, l);
      }
      fence_before();
      if (copies > 1 && !meet()) break;  // the slots are read before the next rows of q come
      tile_no += g.tiles;
      ++seg;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (tid == 0 && sm.abort) set_status(a.status, BPKV_DEV_TIMEOUT);
  if (warp == 2) tmem_dealloc(tmem, kTmemCols);
}

// ---- host side

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Most prefix units that n_seq sequences can make.
int64_t units(int64_t n_seq, int64_t n_prefix, int64_t group, int log) {
  return n_prefix ? min64(n_prefix, n_seq) + (n_seq * group >> log) : 0;
}

struct Space {
  size_t parts, ml, o, total;
  int64_t few0, own0;  // first partial rows of the kinds
};

Space space(int64_t n_seq, int64_t n_prefix, int64_t n_heads, int64_t group) {
  Space s;
  // a segment is unit u's part in worker w, slot u + w of its kind
  const int64_t wide =
      n_prefix && n_seq * group > kFew ? (units(n_seq, n_prefix, group, kPairLog) * n_heads + kSms) * kPair : 0;
  const int64_t few = n_prefix ? (units(n_seq, n_prefix, group, kFewLog) * n_heads + kSms * kFewWarps) * kFew : 0;
  const int64_t own = (n_seq * n_heads + kSms * kFewWarps) * group;
  s.few0 = wide;
  s.own0 = wide + few;
  size_t off = 256;  // status word
  s.parts = off;
  off = up256(off + n_seq * n_heads * group * sizeof(Parts));
  s.ml = off;
  off = up256(off + (wide + few + own) * sizeof(float2));
  s.o = off;
  off = up256(off + (wide + few + own) * kD * sizeof(float));
  s.total = off;
  return s;
}

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

// Rows [units][cap][D] as tiles of 128 rows in 128-byte swizzled rows.
template <int BITS>
bool make_map(CUtensorMap* m, const void* rows, int64_t units, int64_t cap) {
  const EncodeTiled f = encode_tiled();
  if (!f) return false;
  const cuuint32_t one[4] = {1, 1, 1, 1};
  if constexpr (BITS == 16) {  // two halves of 64 channels
    const cuuint64_t dim[4] = {64, (cuuint64_t)cap, 2, (cuuint64_t)units};
    const cuuint64_t stride[3] = {kD * 2, 128, (cuuint64_t)cap * kD * 2};
    const cuuint32_t box[4] = {64, kTile, 2, 1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(rows), dim, stride, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  const cuuint64_t dim[3] = {kD, (cuuint64_t)cap, (cuuint64_t)units};
  const cuuint64_t stride[2] = {kD, (cuuint64_t)cap * kD};
  const cuuint32_t box[3] = {kD, kTile, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(rows), dim, stride, box, one,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Short calls are one launch of k_shared_unit, by the tokens of a prefix and a
// sequence together and of a sequence alone (as the host knows them; a long one
// among short ones would be waited for) for each CTA of a unit, and the rows of
// prefixes that all units together read.  One call / planned, in us, 8 x 4 heads,
// bf16 rows (8-bit rows in brackets).
//   Own rows only: 1 sequence of up to 500 tokens 4.7 / 7.5, 4000 6.4 / 13.9,
//   32000 20 / 26 (20 / 21); 8 of 4000 13.1 / 15.0 (11.7 / 13.0), of 8000 22.6 /
//   23.6 (19.5 / 17.0); 32 of 500 6.6 / 12.0, of 2000 21 / 24 (18 / 18).
//   Over a prefix: 1 over 300 4.5 / 9.2, over 4000 6.6 / 16.4, over 32000 22 / 30;
//   8 over 8000 18.7 / 25.5 (19.5 / 21.2), over 16000 32 / 29; 32 over 900 10.4 /
//   18.4, over 2000 17.8 / 24.0; 96 over 300 15.3 / 19.3, over 900 (691200 rows)
//   27.6 / 27.5.
// A sequence of many units has half the bound: with one of 2000 tokens among 31
// of 500 a call takes 19.2 / 17.7 (of 100 15.3 / 17.6, all of 2000 35 / 40; 8-bit
// rows, of 100, 12.8 / 17.1).
constexpr int64_t kWholeTokens = 2048, kWholeMany = 1024, kWholeRows = 600000;

// Behind the wide kernel, sequences that are short enough for k_shared_unit take
// it too and join the prefix's partials there, which saves the streaming kernel's
// plan and the join's launch.  This / streamed and joined, in us, 8 x 4 heads,
// bf16 rows (8-bit rows in brackets): 32 sequences of up to 1000 tokens over
// 32768 39.3 / 49.7; over 20000 8 of 2000 31 / 38 (33 / 38), 18 of 4000 45 / 52
// (43 / 52), 8 of 8000 53 / 50 (54 / 47); 96 of 1000 72 / 81 (98 / 109), of 2000
// 91 / 106 (107 / 123).  The bounds are as long as a long sequence among short
// ones may be waited for; of many units a CTA has fewer warps.
constexpr int64_t kFinishTokens = 4096, kFinishMany = 2048;

// Prefixes are streamed by units of 16 rows, from L2 again for each, and the wide
// kernel is left out, while that reads at most this many bytes.  Streamed / wide,
// in us: 40 sequences of 2 x 4 heads over five prefixes of up to 3000 tokens (31
// MB) 16.3 / 23.3 (8-bit 16.2 / 27.5); 96 of 8 x 1 over two of 1500 (38 MB) 22.8 /
// 20.3 (22.0 / 23.9); 20 of 8 x 4 over 2500 (51 MB) 24.0 / 15.4 (21.0 / 19.7); 17
// of 1 x 4 over 20000 (51 MB) 24.5 / 18.3 (24.3 / 22.0); 80 of 8 x 4 over 1000 in
// 8 bits (41 MB) 24.6 / 28.5.
template <int BITS>
constexpr int64_t kStreamBytes = BITS == 16 ? 40000000 : 50000000;

// One side's rows: K and V (with their exponents for 8-bit rows).
struct Side {
  const void* rows[2];
  const uint8_t* exps[2];
  const int64_t* len;
  int64_t cap, n_max;
  int32_t n;
};

template <int BITS>
cudaError_t launch(const Side* prefix, const Side& own, const int32_t* prefix_of, int32_t n_heads, int32_t group,
                   const uint16_t* q, uint16_t* out, void* ws, cudaStream_t st) {
  const Space sp = space(own.n, prefix ? prefix->n : 0, n_heads, group);
  unsigned char* w = static_cast<unsigned char*>(ws);
  const Side* sides[2] = {prefix ? prefix : &own, &own};
  Args a = {};
  for (int i = 0; i < 2; ++i)
    for (int kv = 0; kv < 2; ++kv) {
      a.rows[i][kv] = sides[i]->rows[kv];
      a.exps[i][kv] = sides[i]->exps[kv];
    }
  a.prefix_of = prefix_of;
  a.plen = prefix ? prefix->len : nullptr;
  a.len = own.len;
  a.pcap = prefix ? prefix->cap : 0;
  a.cap = own.cap;
  a.n_prefix = prefix ? prefix->n : 0;
  a.n_seq = own.n;
  a.n_heads = n_heads;
  a.group = group;
  a.group_inv = ((1u << 16) + group - 1) / group;
  a.q = q;
  a.parts = reinterpret_cast<Parts*>(w + sp.parts);
  a.part_ml = reinterpret_cast<float2*>(w + sp.ml);
  a.part_o = reinterpret_cast<float*>(w + sp.o);
  a.few0 = sp.few0;
  a.own0 = sp.own0;
  a.status = static_cast<int32_t*>(ws);
  const int64_t pn = prefix ? prefix->n : 0, pmax = prefix ? prefix->n_max : 0;
  const int64_t again =
      max64(min64(pn, own.n), (own.n * group + kFew - 1) / kFew) * n_heads * pmax * (BITS == 16 ? 4 * kD : 2 * kD);
  const int64_t total = own.n_max + pmax;
  const int64_t n_own = (int64_t)own.n * n_heads;
  const int split = unit_split(n_own, total);
  const bool whole = total <= (split > 1 ? 2 : 1) * split * kWholeTokens &&
                     own.n_max <= (n_own > kSms ? kWholeMany : (split > 2 ? 2 : 1) * split * kWholeTokens) &&
                     n_own * pmax <= kWholeRows;
  const bool has_wide = !whole && prefix && own.n * group > kFew && again > kStreamBytes<BITS>;
  a.unit_log = has_wide ? kPairLog : kFewLog;
  a.finish = has_wide && own.n_max <= (n_own > kSms ? kFinishMany : kFinishTokens);
  a.few_rows = a.finish ? 0 : kFew;
  // no more CTAs than tiles, as far as the host knows (longer sequences than
  // it knows of only find fewer CTAs)
  const int64_t n_units = units(own.n, pn, group, a.unit_log), tok = few_tile(BITS);
  const int64_t wide = has_wide ? n_heads * n_units * ((pmax + kTile - 1) / kTile) : 0;
  const int64_t few = n_heads * ((own.n_max + tok - 1) / tok * own.n + n_units * ((pmax + tok - 1) / tok));
  a.wide_ctas = (int32_t)max64(1, min64(kSms, wide));
  a.few_workers = (int32_t)max64(1, min64(kSms, few)) * kFewWarps;
  if (has_wide) {
    Maps maps;
    for (int kv = 0; kv < 2; ++kv)
      if (!make_map<BITS>(&maps.m[kv], prefix->rows[kv], (int64_t)prefix->n * n_heads, prefix->cap))
        return cudaErrorInvalidValue;
    const bool dual = own.n * group > kTile;
    a.stages = Shape<BITS>::stages(dual);
    static std::atomic<uint64_t> done;
    cudaError_t e = allow_smem(k_shared_wide<BITS>, Shape<BITS>::kSmemMax, done);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k_shared_wide<BITS>, dim3(a.wide_ctas), dim3(kThreads), (size_t)Shape<BITS>::bytes(dual), st, a, maps);
    if (e != cudaSuccess) return e;
  }
  return launch_few<BITS>(a, whole ? total : -1, own.n_max, !has_wide, out, st);
}

}  // namespace

}  // namespace shared

using namespace shared;

size_t shared_bytes(int64_t n_seq, int64_t n_prefix, int64_t n_heads, int64_t group) {
  return space(n_seq, n_prefix, n_heads, group).total;
}

cudaError_t launch_shared(const bpkv_cache* p, const int32_t* prefix_of, const bpkv_cache& c, const uint16_t* q,
                          uint16_t* out, void* ws, cudaStream_t st) {
  Side side[2];
  const bpkv_cache* cs[2] = {p, &c};
  for (int i = 0; i < 2; ++i)
    if (cs[i])
      side[i] = {{cs[i]->k_rows, cs[i]->v_rows}, {nullptr, nullptr}, cs[i]->seq_len, cs[i]->cap_tokens, cs[i]->n_max,
                 cs[i]->n_seq};
  return launch<16>(p ? &side[0] : nullptr, side[1], prefix_of, c.n_kv_heads, c.group, q, out, ws, st);
}

cudaError_t launch_shared8(const bpkv_rows8* p, const int32_t* prefix_of, const bpkv_rows8& c, const uint16_t* q,
                           uint16_t* out, void* ws, cudaStream_t st) {
  Side side[2];
  const bpkv_rows8* cs[2] = {p, &c};
  for (int i = 0; i < 2; ++i)
    if (cs[i])
      side[i] = {{cs[i]->k8, cs[i]->v8}, {cs[i]->kexp, cs[i]->vexp}, cs[i]->seq_len, cs[i]->cap_tokens, cs[i]->n_max,
                 cs[i]->n_seq};
  return launch<8>(p ? &side[0] : nullptr, side[1], prefix_of, c.n_kv_heads, c.group, q, out, ws, st);
}

}  // namespace bpkv
