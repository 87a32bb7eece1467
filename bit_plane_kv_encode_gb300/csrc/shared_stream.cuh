// What a warp does that streams its own tiles of K and V rows under few query rows:
// its ring of copies, the products, the softmax (shared_few.cu says why so).
//
// A walk W says which tiles: tok (tokens of a tile), t, valid(), more(), next(), row0,
// side, a (Args with rows[side][K, V] and exps), q_of(r), the address of query row r,
// where a row does not see all of the last rows (kMasked), base, the first of those, and
// mask_of(r), a bit for each, and where rows do not lie one behind the other (kStrided)
// first[K, V], the bytes before them, and a.step[K, V], from one to the next.
#pragma once

#include "rows8_core.cuh"
#include "shared_plan.cuh"

namespace bpkv {
namespace shared {
namespace few {

constexpr int kStages = 3;
constexpr int kStage = 8192;  // K rows then V rows

template <int BITS>
struct Shape {
  static constexpr int kTok = BITS == 16 ? 16 : 32;       // tokens of a stage
  static constexpr int kSub = kTok / 16;                  // 16-token blocks of a stage
  static constexpr int kRow = kD * BITS / 8;              // bytes of a row
  static constexpr int kExps = BITS == 16 ? 0 : 2 * kTok; // exponent bytes
  static constexpr int kRing = kFewWarps * kStages * (kStage + kExps);
  static constexpr float kLazy = BITS == 16 ? 8.f : 4.f;  // rise of the maximum before O is rescaled
  static constexpr float kShift = BITS == 16 ? 0.f : 11.f;  // p' below 2^15: a half
};

__device__ __forceinline__ void cp16_zero(uint32_t dst, const void* src, bool there, uint64_t policy) {
  const int n = there ? 16 : 0;
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(n),
               "l"(policy)
               : "memory");
}
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
template <int BITS>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, const uint32_t* b) {
  if constexpr (BITS == 16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
template <int BITS>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  if constexpr (BITS == 16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}
__device__ __forceinline__ uint32_t halves(uint32_t codes) {
  const __half2 h = half2_of_e4m3x2((uint16_t)codes);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Issue the copies of the walk's tile into a stage.
template <int BITS, typename W>
__device__ __forceinline__ void load_tile(const W& w, uint32_t stage, uint32_t exps, uint64_t policy) {
  using S = Shape<BITS>;
  const int lane = threadIdx.x & 31, valid = w.valid();
  const int64_t row = w.row0 + (int64_t)w.t * S::kTok;
  constexpr int kChunks = S::kRow / 16;  // 16-byte pieces of a row
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const unsigned char* src = static_cast<const unsigned char*>(w.a.rows[w.side][kv]);
    if constexpr (W::kStrided) src += w.first[kv] + (int64_t)w.t * S::kTok * w.a.step[kv];
    else src += row * S::kRow;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int x = i * 32 + lane, tok = x / kChunks, c = x % kChunks;
      const unsigned char* from = src + x * 16;
      if constexpr (W::kStrided) from = src + tok * w.a.step[kv] + c * 16;
      cp16_zero(stage + kv * (kStage / 2) + tok * S::kRow + ((c ^ (tok & 7)) << 4), from, tok < valid, policy);
    }
    if (BITS == 8 && lane < 2) cp16_zero(exps + kv * S::kTok + lane * 16, w.a.exps[w.side][kv] + row + lane * 16, true, policy);
  }
}

// q of the unit as the 8-side operand of S^T, rows lane / 4 (+ 8), for 8-bit
// rows as halves under a power-of-two scale of the row.
template <int BITS, int NB, typename W>
__device__ __forceinline__ void load_q(const W& w, int rows, uint32_t (*qb)[8][2], float (*qf)[2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int r = nb * 8 + g;
    const uint16_t* q = r < rows ? w.q_of(r) : nullptr;
    if constexpr (BITS == 16) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        qb[nb][k][0] = q ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 2 * c) : 0u;
        qb[nb][k][1] = q ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 8 + 2 * c) : 0u;
      }
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint2 v = q ? *reinterpret_cast<const uint2*>(q + 16 * k + 4 * c) : make_uint2(0u, 0u);
        qb[nb][k][0] = v.x;
        qb[nb][k][1] = v.y;
        m = __vmaxu2(m, __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu));
      }
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
      m = max(m & 0xffffu, m >> 16);
      const int e = max(-100, (int)(m >> 7) - 127 - 7);  // the largest within 128 .. 256
      const float f = exp2i(-e);
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          qb[nb][k][i] = pack<8>(__uint_as_float(qb[nb][k][i] << 16) * f, __uint_as_float(qb[nb][k][i] & 0xffff0000u) * f);
      const float s = exp2i(e);  // of row g; this thread's sums are of rows 2 c, 2 c + 1
      qf[nb][0] = __shfl_sync(0xffffffffu, s, 8 * c);
      qf[nb][1] = __shfl_sync(0xffffffffu, s, 8 * c + 4);
    }
  }
}

// What a warp has of its unit's rows: this thread's of O^T (channels g, g + 8 of
// each 16 for bf16 rows, 2 g, 2 g + 1 for 8-bit ones; rows 2 c, 2 c + 1), m in
// units of the logits, l of this thread's tokens.
template <int NB>
struct State {
  float o[NB][8][4], m[NB][2], l[NB][2];
};

// The warp's tiles from `cur` on; the copies of those before `ahead` are already
// under way.  end(unit, state, rows) after each unit.
template <int BITS, int NB, typename W, typename R, typename E>
__device__ __forceinline__ void stream(W& cur, W& ahead, uint32_t ring, const unsigned char* exps,
                                       uint64_t policy, R&& rows_of, E&& end) {
  using S = Shape<BITS>;
  const int lane = threadIdx.x & 31, g = lane >> 2;
  constexpr float kUnit = BITS == 16 ? kLogScale : 1.f;  // logits times this are in powers of two
  uint32_t qb[NB][8][2];
  float qf[NB][2];
  [[maybe_unused]] uint64_t mask[NB][2];
  State<NB> state;
  auto& o = state.o;
  auto& m = state.m;
  auto& l = state.l;
  int rows = 0;
  bool fresh = true;
  int st = 0;
  while (cur.more()) {
    if (fresh) {
      rows = rows_of(cur);
      load_q<BITS, NB>(cur, rows, qb, qf);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        m[nb][0] = m[nb][1] = -INFINITY;
        l[nb][0] = l[nb][1] = 0.f;
        if constexpr (W::kMasked) {
#pragma unroll
          for (int i = 0; i < 2; ++i) mask[nb][i] = cur.mask_of(min(nb * 8 + 2 * (lane & 3) + i, rows - 1));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[nb][j][i] = 0.f;
      }
    }
    cp_wait<kStages - 2>();
    __syncwarp();  // everyone's copies of this stage have landed, and the stage before is read
    {
      const int into = st == 0 ? kStages - 1 : st - 1;
      if (ahead.more()) {
        load_tile<BITS>(ahead, ring + into * kStage, smem_u32(exps) + into * S::kExps, policy);
        ahead.next();
      }
      cp_async_commit();
    }
    const uint32_t ks = ring + st * kStage, vs = ks + kStage / 2;
    const bool two = NB > 1 && rows > 8;
    const int valid = cur.valid();
    float x[S::kSub][NB][4];
    float iv[S::kSub][2];
    // ---- S^T of the stage's tokens: this thread has tokens g, g + 8 of each block, rows 2 c, 2 c + 1
#pragma unroll
    for (int b = 0; b < S::kSub; ++b) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[b][nb][i] = 0.f;
      const int tok = b * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
      for (int k = 0; k < 8; k += BITS == 16 ? 1 : 2) {
        uint32_t r[4];
        if constexpr (BITS == 16) {
          ldm4(r, ks + tok * S::kRow + (((2 * k + (lane >> 4)) ^ (tok & 7)) << 4));
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            if (nb == 0 || two) mma<16>(x[b][nb], r, qb[nb][k]);
        } else {
          ldm4(r, ks + tok * S::kRow + (((k + (lane >> 4)) ^ (tok & 7)) << 4));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t f[4] = {halves(r[2 * i]), halves(r[2 * i + 1]), halves(r[2 * i] >> 16),
                                   halves(r[2 * i + 1] >> 16)};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              if (nb == 0 || two) mma<8>(x[b][nb], f, qb[nb][k + i]);
          }
        }
      }
      if constexpr (BITS == 8) {
        const unsigned char* e = exps + st * S::kExps + b * 16 + g;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int ke = min(max((int)e[8 * i] - kExpBias, kExpMin), kExpMax);
          const int ve = min(max((int)e[S::kTok + 8 * i] - kExpBias, kExpMin), kExpMax);
          const float kf = exp2i(ke) * kLogScale, ev = (float)ve;
          iv[b][i] = exp2i(-ve);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            x[b][nb][2 * i] = fmaf(x[b][nb][2 * i] * kf, qf[nb][0], ev);
            x[b][nb][2 * i + 1] = fmaf(x[b][nb][2 * i + 1] * kf, qf[nb][1], ev);
          }
        }
      }
      if constexpr (W::kMasked) {
        const int64_t in = cur.t * (int64_t)S::kTok + S::kTok - cur.base;  // rows of the masked ones before the tile's end
        if (in > 0) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int64_t j = in - S::kTok + b * 16 + g + 8 * i;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int k = 0; k < 2; ++k)
                if (j >= 0 && (j > 63 || !((mask[nb][k] >> j) & 1))) x[b][nb][2 * i + k] = -INFINITY;
          }
        }
      }
      if (valid < S::kTok) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (b * 16 + g + 8 * i >= valid) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) x[b][nb][2 * i] = x[b][nb][2 * i + 1] = -INFINITY;
          }
      }
    }
    // ---- m follows the maximum when that has risen far enough
    float top[NB][2];
    bool up = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[nb][i] = fmaxf(x[0][nb][i], x[0][nb][2 + i]);
#pragma unroll
        for (int b = 1; b < S::kSub; ++b) top[nb][i] = fmaxf(top[nb][i], fmaxf(x[b][nb][i], x[b][nb][2 + i]));
        up |= top[nb][i] > lazy_top<BITS>(m[nb][i], S::kLazy / kUnit);
      }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float t = top[nb][i];
#pragma unroll
          for (int s = 4; s < 32; s <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, s));
          if (t > m[nb][i]) {
            const float f = ex2((m[nb][i] - t) * kUnit);
            m[nb][i] = t;
            l[nb][i] *= f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              o[nb][j][i] *= f;
              o[nb][j][2 + i] *= f;
            }
          }
        }
    }
    float base[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        base[nb][i] = m[nb][i] == -INFINITY ? 0.f : shifted<BITS>(m[nb][i], kUnit, S::kShift);
    // ---- P^T, and O^T += V^T P^T
#pragma unroll
    for (int b = 0; b < S::kSub; ++b) {
      uint32_t pb[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[i] = ex2(fmaf(x[b][nb][i], kUnit, -base[nb][i & 1]));
          l[nb][i & 1] = BITS == 16 ? l[nb][i & 1] + p[i] : fmaf(p[i], iv[b][i >> 1], l[nb][i & 1]);
        }
        pb[nb][0] = transpose8(pack<BITS>(p[0], p[1]));
        pb[nb][1] = transpose8(pack<BITS>(p[2], p[3]));
      }
      if constexpr (BITS == 16) {
        const int tok = b * 16 + (lane & 7) + (lane >> 4) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t r[4];
          ldm4t(r, vs + tok * S::kRow + (((2 * j + ((lane >> 3) & 1)) ^ (tok & 7)) << 4));
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            if (nb == 0 || two) mma<16>(o[nb][j], r, pb[nb]);
        }
      } else {
        const int tok = b * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          uint32_t r[4];
          ldm4t(r, vs + tok * S::kRow + (((j + (lane >> 4)) ^ (tok & 7)) << 4));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // of two neighbouring channels: the even ones are rows 0 .. 7 of the product, the odd ones 8 .. 15
            const uint32_t f[4] = {halves(__byte_perm(r[2 * i], 0, 0x4420)), halves(__byte_perm(r[2 * i], 0, 0x4431)),
                                   halves(__byte_perm(r[2 * i + 1], 0, 0x4420)),
                                   halves(__byte_perm(r[2 * i + 1], 0, 0x4431))};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              if (nb == 0 || two) mma<8>(o[nb][j + i], f, pb[nb]);
          }
        }
      }
    }
    st = st == kStages - 1 ? 0 : st + 1;
    const W was = cur;
    fresh = cur.next();
    if (fresh || !cur.more()) end(was, state, rows);
  }
  cp_wait<0>();
}

// This warp's sum of the l of row 2 c + i.
template <int NB>
__device__ __forceinline__ float row_sum(const State<NB>& st, int nb, int i) {
  float s = st.l[nb][i];
#pragma unroll
  for (int k = 4; k < 32; k <<= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
  return s;
}

// The thread's part of row 2 c + i of O^T to the row at p.
template <int BITS, int NB>
__device__ __forceinline__ void put_row(const State<NB>& st, int nb, int i, float* p) {
  const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (BITS == 16) {
      p[16 * j + g] = st.o[nb][j][i];
      p[16 * j + 8 + g] = st.o[nb][j][2 + i];
    } else {
      *reinterpret_cast<float2*>(p + 16 * j + 2 * g) = make_float2(st.o[nb][j][i], st.o[nb][j][2 + i]);
    }
  }
}

// Start the first copies of a warp's tiles.
template <int BITS, typename W>
__device__ __forceinline__ void prime(W& ahead, uint32_t ring, const unsigned char* exps, uint64_t policy) {
  for (int i = 0; i < kStages - 1; ++i) {
    if (ahead.more()) {
      load_tile<BITS>(ahead, ring + i * kStage, smem_u32(exps) + i * Shape<BITS>::kExps, policy);
      ahead.next();
    }
    cp_async_commit();
  }
}

}  // namespace few
}  // namespace shared
}  // namespace bpkv
