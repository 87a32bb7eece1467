// Projected heads to cache rows: RMS norm of query and key heads, position
// rotation and layout in one pass (bpkv_qkv_rope).
//
// A head is read once, in 16-byte pieces, and written once; what bounds the
// kernel after the bytes is instructions, so a thread takes 16 channels: eight
// lanes hold a head, and both channels of a rotated pair are the thread's own
// (halves: channels 8 l .. and rot/2 + 8 l .., for rot/2 a multiple of 8; other
// rot read the partner a second time).  The mean square is three shuffles.  A
// CTA takes up to eight tokens at once, a turn; cosines and sines are worked out
// once for all of a token's heads into shared memory, in the order in which the
// lanes read them as 16-byte pieces without bank conflicts, and each thread's
// next loads are issued before a head is worked on.  The grid has a CTA for each
// turn up to 4864 of them; only longer prompts give a CTA a second one.
//
// Angles: the position times the frequency in turns, as 64-bit fixed point
// whose wrap-around drops whole turns.  Only the frequency is rounded, down to
// 2^-64 of a turn from a 64-bit 2^64 / (2 pi) that is cut off too: a position p
// is off by less than |p| (1 + frequency) 2^-64 turns (2^-44 at a million, 2^-23
// at 2^40).  The top 32 bits are the angle within half a turn to 2^-31, which a
// float holds to 2^-24.
//
// Measured on a GB300 (G = 4, H = 8, normed, rotated by halves, bf16 queries):
// a prompt of 8191 tokens (201 MB) 38.0 us, 5.3 TB/s, 74% of the issue slots in
// use; with sixteen lanes a head and partners by shuffle it took 72.0 us, with
// the 8-bit rows chosen at run time instead of by an instantiation 39.9.  One
// token 2.9 us, one of each of 32 sequences into 8-bit rows 3.1 us (latency);
// 3 x 1365 tokens of H = 2, G = 7, float queries, 64 channels rotated in pairs
// (52 MB) 12.5 us, 4.2 TB/s.
#include "rows8_core.cuh"

namespace bpkv {

constexpr int kQkvThreads = 192;
constexpr int kQkvLanes = 8;                             // of a head
constexpr int kQkvHeads = kQkvThreads / kQkvLanes;       // heads a CTA holds at once
constexpr int kQkvTokens = 8;                            // tokens of a CTA's turn at most

struct QkvArgs {
  const uint16_t* qkv;
  int64_t ld;
  const int64_t* pos;
  const float* inv_freq;
  const float* q_weight;
  const float* k_weight;
  void* q_out;
  uint16_t* k_out;
  uint16_t* v_out;
  Rows8Out c;  // k8 NULL: no 8-bit cache
  int32_t* status;
  float eps;
  int32_t n_seq, n_heads, group, t_new, rot;
  int32_t pairs, q_bf16;
  int32_t bump;           // positions are the cache's lengths: 0 no, 1 a launch of its own raises them, 2 the token's CTA
  int32_t toks;           // tokens of a CTA's turn
  int32_t heads_per_cta;  // of each token
};

// Turns per position of a frequency in radians, modulo one, in 2^-64 turns:
// the frequency's 24-bit mantissa times 2^64 / (2 pi), shifted by its exponent;
// below the exact number by less than 1 + frequency.
__device__ __forceinline__ uint64_t turns64(float inv_freq) {
  const uint32_t b = __float_as_uint(inv_freq);
  const int e = (int)((b >> 23) & 0xff);
  const uint64_t m = (b & 0x7fffffu) | (e ? 0x800000u : 0u);
  const int shift = 150 - (e ? e : 1);  // inv_freq = m 2^-shift
  constexpr uint64_t k = 0x28be60db9391054aull;  // 2^64 / (2 pi)
  const uint64_t lo = m * k, hi = __umul64hi(m, k);
  const uint64_t t = shift <= 0    ? (shift > -64 ? lo << -shift : 0)
                     : shift < 64  ? (lo >> shift) | (hi << (64 - shift))
                     : shift < 128 ? hi >> (shift - 64)
                                   : 0;
  return b >> 31 ? 0 - t : t;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// A token of the CTA's turn.
struct QkvToken {
  int64_t tok;    // among all; -1: none
  int64_t row;    // first row in k_out / v_out, for head 0
  int64_t row8;   // first row in the 8-bit cache, for head 0; -1: not written
};

enum { kRotPairs, kRotHalves, kRotAny };

// Angle f of a token in its table: lane l's eight angles are 8 l .., two to a
// piece {cos, cos', sin, sin'}.
__device__ __forceinline__ int angle_at(int f) { return (((f & 7) >> 1) * 8 + (f >> 3)) * 4 + (f & 1); }

__device__ __forceinline__ void unpack8(const uint4& w, float* y) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = __uint_as_float(x[i] << 16);
    y[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
  }
}

template <int ROT, bool ROWS8>
__global__ void __launch_bounds__(kQkvThreads, 5) k_qkv_rope(const __grid_constant__ QkvArgs a) {
  pdl_enter();
  __shared__ __align__(16) float4 s_tab[2][kQkvTokens][32];
  __shared__ __align__(16) float4 s_w[2][2][16];  // [query, key][first, second four][eight channels]
  __shared__ QkvToken s_tok[2][kQkvTokens];
  const int tid = threadIdx.x, l8 = tid & 7;
  const int half = a.rot / 2;
  // this thread's two runs of eight channels
  int ca, cb;
  if (ROT == kRotHalves && l8 < half / 8) {
    ca = l8;
    cb = l8 + half / 8;
  } else {
    ca = 2 * l8;  // halves: the runs behind the rotated ones
    cb = ca + 1;
  }
  const bool norm_q = a.q_weight != nullptr, norm_k = a.k_weight != nullptr;
  const int n_q = a.n_heads * a.group, heads = n_q + 2 * a.n_heads;
  const int head0 = blockIdx.y * a.heads_per_cta, n_here = min(heads - head0, a.heads_per_cta);
  const int64_t tokens = (int64_t)a.n_seq * a.t_new, turns_n = (tokens + a.toks - 1) / a.toks;
  const bool small = tokens < (1ll << 31);
  const int j0 = (tid / kQkvLanes) / n_here, h0 = (tid / kQkvLanes) % n_here;  // the first of this thread's heads
  const int dj = kQkvHeads / n_here, dh = kQkvHeads % n_here;                  // and from one to the next
  if (tid < kD) {
    float* w = reinterpret_cast<float*>(&s_w[0][(tid & 7) >> 2][tid >> 3]) + (tid & 3);
    if (norm_q) w[0] = a.q_weight[tid];
    if (norm_k) w[kD] = a.k_weight[tid];
  }
  uint64_t step = 0;
  if (tid < 64 * 3 && (tid & 63) < half) step = turns64(a.inv_freq[tid & 63]);
  int buf = 0;
  for (int64_t turn = blockIdx.x; turn < turns_n; turn += gridDim.x, buf ^= 1) {
    const int64_t tok0 = turn * a.toks;
    const int n_tok = (int)min64(a.toks, tokens - tok0);
    auto load = [&](int j, int h, uint4& wa, uint4& wb) {
      if (j < n_tok) {
        const uint16_t* x = a.qkv + (tok0 + j) * a.ld + (head0 + h) * kD;
        wa = __ldcs(reinterpret_cast<const uint4*>(x + ca * 8));
        wb = __ldcs(reinterpret_cast<const uint4*>(x + cb * 8));
      }
    };
    int j = j0, h = h0;
    uint4 wa = make_uint4(0, 0, 0, 0), wb = wa;
    load(j, h, wa, wb);
    // the table of the turn before last is no longer read: a barrier lies between
    for (int i = tid >> 6; i < n_tok; i += kQkvThreads / 64) {
      const int64_t tok = tok0 + i;
      const int64_t s = small ? (int64_t)((uint32_t)tok / (uint32_t)a.t_new) : tok / a.t_new;
      const int64_t t = tok - s * a.t_new, p0 = a.pos[s];
      if ((tid & 63) < half) {
        const uint64_t ph = (uint64_t)(p0 + t) * step;
        const float u = (float)(int32_t)(ph >> 32) * 4.6566128730773926e-10f;  // half turns: 2^-31
        float sn, cs;
        sincospif(u, &sn, &cs);
        float* e = reinterpret_cast<float*>(s_tab[buf][i]) + angle_at(tid & 63);
        e[0] = cs;
        e[2] = sn;
      }
      if ((tid & 63) == 0) {
        const bool fits = ROWS8 && rows8_fits(p0, a.t_new, a.c.cap);
        s_tok[buf][i] = {tok, s * a.n_heads * a.t_new + t, fits ? s * a.n_heads * a.c.cap + p0 + t : -1};
        if (ROWS8 && t == 0 && head0 == 0) {
          if (!fits)
            set_status(a.status, BPKV_DEV_OVERFLOW);
          else if (!a.bump)
            a.c.seq_len[s] = p0 + a.t_new;
        }
      }
    }
    __syncthreads();
    if (ROWS8 && a.bump == 2 && tid < n_tok) {  // one token a sequence, and this CTA alone has read its length
      const QkvToken& tk = s_tok[buf][tid];
      if (tk.row8 >= 0) a.c.seq_len[tk.tok] = tk.row8 - tk.tok * a.n_heads * a.c.cap + 1;
    }
    // as many rounds as the warp's first head has: the shuffles are the warp's
    const int items = n_tok * n_here;
#pragma unroll 1
    for (int item = (tid & ~31) / kQkvLanes; item < items; item += kQkvHeads) {
      const bool there = j < n_tok;
      int jn = j + dj, hn = h + dh;
      if (hn >= n_here) hn -= n_here, ++jn;
      uint4 na = make_uint4(0, 0, 0, 0), nb = na;
      load(jn, hn, na, nb);
      const int head = head0 + h, jt = there ? j : 0;
      const int kind = head < n_q ? 0 : head < n_q + a.n_heads ? 1 : 2;  // query, key, value
      float y[16];
      unpack8(wa, y);
      unpack8(wb, y + 8);
      const bool norm = kind == 0 ? norm_q : kind == 1 && norm_k;
      float r = 1.f;
      if (norm) {
        float ss[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 16; ++i) ss[i & 1] = fmaf(y[i], y[i], ss[i & 1]);
        ss[0] += ss[1];
        const uint32_t mask = 0xffu << (tid & 24);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) ss[0] += __shfl_xor_sync(mask, ss[0], o);
        r = rsqrtf(ss[0] * (1.f / kD) + a.eps);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 w = s_w[kind][i & 1][i < 2 ? ca : cb];
          y[4 * i] *= r * w.x;
          y[4 * i + 1] *= r * w.y;
          y[4 * i + 2] *= r * w.z;
          y[4 * i + 3] *= r * w.w;
        }
      }
      const float4* tab = s_tab[buf][jt];
      if constexpr (ROT == kRotPairs) {
        if (kind < 2 && 16 * l8 < a.rot) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 e = tab[i * 8 + l8];
            if (16 * l8 + 4 * i < a.rot) {
              const float p = y[4 * i], q = y[4 * i + 1];
              y[4 * i] = fmaf(-q, e.z, p * e.x);
              y[4 * i + 1] = fmaf(p, e.z, q * e.x);
            }
            if (16 * l8 + 4 * i + 2 < a.rot) {
              const float p = y[4 * i + 2], q = y[4 * i + 3];
              y[4 * i + 2] = fmaf(-q, e.w, p * e.y);
              y[4 * i + 3] = fmaf(p, e.w, q * e.y);
            }
          }
        }
      } else if constexpr (ROT == kRotHalves) {
        if (kind < 2 && l8 < half / 8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 e = tab[i * 8 + l8];
            const float p0 = y[2 * i], p1 = y[2 * i + 1], q0 = y[8 + 2 * i], q1 = y[9 + 2 * i];
            y[2 * i] = fmaf(-q0, e.z, p0 * e.x);
            y[2 * i + 1] = fmaf(-q1, e.w, p1 * e.y);
            y[8 + 2 * i] = fmaf(p0, e.z, q0 * e.x);
            y[9 + 2 * i] = fmaf(p1, e.w, q1 * e.y);
          }
        }
      } else if (there && kind < 2) {
        const uint16_t* x = a.qkv + (tok0 + j) * a.ld + head * kD;
        const float* w = reinterpret_cast<const float*>(s_w[kind]);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int c = 16 * l8 + i;
          if (c < a.rot) {
            const bool first = c < half;
            const int pc = first ? c + half : c - half;
            float o = bf16_bits_to_float(x[pc]);
            if (norm) o *= r * w[((pc & 7) >> 2) * 64 + (pc >> 3) * 4 + (pc & 3)];
            const float* e = reinterpret_cast<const float*>(tab) + angle_at(first ? c : pc);
            y[i] = first ? fmaf(-o, e[2], y[i] * e[0]) : fmaf(o, e[2], y[i] * e[0]);
          }
        }
      }
      if (kind < 2) {
        wa = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
        wb = make_uint4(pack_bf16(y[8], y[9]), pack_bf16(y[10], y[11]), pack_bf16(y[12], y[13]), pack_bf16(y[14], y[15]));
      }
      const QkvToken& tk = s_tok[buf][jt];
      if (there && kind == 0) {
        const int64_t o = (tk.tok * n_q + head) * kD;
        if (a.q_bf16) {
          uint16_t* q = static_cast<uint16_t*>(a.q_out) + o;
          *reinterpret_cast<uint4*>(q + ca * 8) = wa;
          *reinterpret_cast<uint4*>(q + cb * 8) = wb;
        } else {
          float4* q = reinterpret_cast<float4*>(static_cast<float*>(a.q_out) + o);
          q[2 * ca] = make_float4(y[0], y[1], y[2], y[3]);
          q[2 * ca + 1] = make_float4(y[4], y[5], y[6], y[7]);
          q[2 * cb] = make_float4(y[8], y[9], y[10], y[11]);
          q[2 * cb + 1] = make_float4(y[12], y[13], y[14], y[15]);
        }
      } else if (there) {
        const int hk = head - n_q - (kind == 1 ? 0 : a.n_heads);
        uint16_t* rows = kind == 1 ? a.k_out : a.v_out;
        if (rows) {
          rows += (tk.row + (int64_t)hk * a.t_new) * kD;
          *reinterpret_cast<uint4*>(rows + ca * 8) = wa;
          *reinterpret_cast<uint4*>(rows + cb * 8) = wb;
        }
        if (ROWS8 && tk.row8 >= 0) {
          const int64_t row = tk.row8 + (int64_t)hk * a.c.cap;
          uint32_t m = __vmaxu2(abs_max(wa), abs_max(wb));
          const uint32_t mask = 0xffu << (tid & 24);
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(mask, m, o));
          const int e = rows8_exponent(max(m & 0xffffu, m >> 16));
          uint8_t* codes = (kind == 1 ? a.c.k8 : a.c.v8) + row * kD;
          *reinterpret_cast<uint2*>(codes + ca * 8) = row_codes(wa, e);
          *reinterpret_cast<uint2*>(codes + cb * 8) = row_codes(wb, e);
          if (l8 == 0) (kind == 1 ? a.c.kexp : a.c.vexp)[row] = (uint8_t)(e + kExpBias);
        }
      }
      wa = na;
      wb = nb;
      j = jn;
      h = hn;
    }
  }
}

template <bool ROWS8>
void (*pick(int kind))(QkvArgs) {
  return kind == kRotPairs    ? k_qkv_rope<kRotPairs, ROWS8>
         : kind == kRotHalves ? k_qkv_rope<kRotHalves, ROWS8>
                              : k_qkv_rope<kRotAny, ROWS8>;
}

cudaError_t launch_rows8_bump(const bpkv_rows8& c, int32_t t_new, cudaStream_t st);

cudaError_t launch_qkv_rope(const bpkv_qkv_args& q, cudaStream_t st) {
  QkvArgs a = {};
  a.qkv = q.qkv;
  a.ld = q.ld;
  a.inv_freq = q.inv_freq;
  a.q_weight = q.q_weight;
  a.k_weight = q.k_weight;
  a.q_out = q.q_out;
  a.k_out = q.k_out;
  a.v_out = q.v_out;
  a.status = q.status;
  a.eps = q.eps;
  a.n_seq = q.n_seq;
  a.n_heads = q.n_kv_heads;
  a.group = q.group;
  a.t_new = q.t_new;
  a.rot = q.rot_dim;
  a.pairs = (q.flags & BPKV_QKV_PAIRS) != 0;
  a.q_bf16 = (q.flags & BPKV_QKV_Q_BF16) != 0;
  a.pos = q.pos;
  if (q.rows8) {
    const bpkv_rows8& c = *q.rows8;
    a.c = {c.k8, c.v8, c.kexp, c.vexp, c.seq_len, c.cap_tokens};
    a.bump = q.pos == nullptr || q.pos == c.seq_len;
    if (a.bump) a.pos = c.seq_len;
  }
  const int heads = (q.group + 2) * q.n_kv_heads;
  const int64_t tokens = (int64_t)q.n_seq * q.t_new;
  // few tokens: their heads go to CTAs 24 at a time, so that they run side by
  // side; many: a CTA takes all heads of up to eight tokens for each barrier,
  // while that leaves every SM some CTAs
  a.heads_per_cta = tokens * heads <= (int64_t)152 * 8 * kQkvHeads ? kQkvHeads : heads;
  // a decode step into the 8-bit cache: the token's CTA can raise the length
  // when it is the only one to read it, which saves the second launch.  48 heads,
  // 1 / 32 / 512 sequences, in a graph: 3.4 / 3.8 / 6.1 us instead of 3.6 / 3.8 /
  // 7.4, outside 3.5 / 3.9 / 6.3 instead of 4.6 / 4.6 / 8.0; with 96 heads, four
  // rounds of one CTA, 4.8 instead of 3.6.
  if (a.bump && q.t_new == 1 && (heads <= 2 * kQkvHeads || a.heads_per_cta == heads)) {
    a.bump = 2;
    a.heads_per_cta = heads;
  }
  if (a.heads_per_cta > heads) a.heads_per_cta = heads;
  a.toks = kQkvTokens;
  while (a.toks > 1 && (a.toks * a.heads_per_cta > 8 * kQkvHeads || tokens / a.toks < 152 * 8)) a.toks /= 2;
  const dim3 grid((unsigned)min64((tokens + a.toks - 1) / a.toks, 152 * 32),
                  (heads + a.heads_per_cta - 1) / a.heads_per_cta);
  const int kind = a.pairs ? kRotPairs : a.rot % 16 == 0 ? kRotHalves : kRotAny;
  const cudaError_t e = launch_pdl(q.rows8 ? pick<true>(kind) : pick<false>(kind), grid, dim3(kQkvThreads), 0, st, a);
  if (e != cudaSuccess || a.bump != 1) return e;
  return launch_rows8_bump(*q.rows8, q.t_new, st);
}

}  // namespace bpkv
