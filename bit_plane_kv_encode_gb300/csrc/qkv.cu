// Projected heads to cache rows: RMS norm of query and key heads, position
// rotation and layout in one pass (bpkv_qkv_rope).
//
// Bound by bytes: a head is read once, in 16-byte pieces, and written once.
// Sixteen lanes hold a head, eight channels each, so the mean square is four
// shuffles and both channels of a rotated pair sit in the group: in the same
// lane (neighbouring pairs), in lane l +- rot/16 (halves, rot/2 a multiple of
// 8), or are read a second time (other rot).  A CTA takes 48 heads at a time,
// of one token or of several that have few heads; each thread issues the loads
// of its three before the tokens' cosines and sines are worked out, once for
// all of a token's heads, in shared memory.
//
// Angles: the position times the frequency in turns, as 64-bit fixed point
// whose wrap-around drops whole turns, is exact however far the position; the
// top 32 bits are the angle within half a turn to 2^-32.
#include "rows8_core.cuh"

namespace bpkv {

constexpr int kQkvThreads = 256;
constexpr int kQkvGroups = kQkvThreads / 16;
constexpr int kQkvPer = 3;                         // heads of a thread
constexpr int kQkvHeads = kQkvGroups * kQkvPer;    // heads a CTA holds at once
constexpr int kQkvTokens = 16;                     // tokens it holds at most

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
  int32_t pairs, q_bf16, bump;
  int32_t toks;  // tokens of a CTA's turn
};

// Turns per position of a frequency in radians, modulo one, in 2^-64 turns.
__device__ __forceinline__ uint64_t turns64(float inv_freq) {
  const double t = (double)inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  const double f = t - floor(t);
  return f < 1.0 ? __double2ull_rd(f * 18446744073709551616.0) : 0ull;
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
  int64_t pos;
};

enum { kRotPairs, kRotHalves, kRotAny };

template <int ROT>
__global__ void __launch_bounds__(kQkvThreads, 4) k_qkv_rope(const __grid_constant__ QkvArgs a) {
  pdl_enter();
  __shared__ __align__(16) float2 s_cs[kQkvTokens][kD / 2];
  __shared__ __align__(16) float s_w[2][kD];
  __shared__ uint64_t s_turns[kD / 2];
  __shared__ QkvToken s_tok[kQkvTokens];
  const int tid = threadIdx.x, l16 = tid & 15, grp = tid >> 4, c0 = l16 * 8;
  const int half = a.rot / 2;
  const bool norm_q = a.q_weight != nullptr, norm_k = a.k_weight != nullptr;
  const int n_q = a.n_heads * a.group, heads = n_q + 2 * a.n_heads;
  const int head0 = blockIdx.y * kQkvHeads, n_here = min(heads - head0, kQkvHeads);  // of each token
  const int64_t tokens = (int64_t)a.n_seq * a.t_new, turns_n = (tokens + a.toks - 1) / a.toks;
  if (tid < kD) {
    if (norm_q) s_w[0][tid] = a.q_weight[tid];
    if (norm_k) s_w[1][tid] = a.k_weight[tid];
  }
  if (tid < half) s_turns[tid] = turns64(a.inv_freq[tid]);
  for (int64_t turn = blockIdx.x; turn < turns_n; turn += gridDim.x) {
    const int64_t tok0 = turn * a.toks;
    const int n_items = (int)min64(a.toks, tokens - tok0) * n_here;
    uint4 w[kQkvPer];
#pragma unroll
    for (int k = 0; k < kQkvPer; ++k) {
      const int item = k * kQkvGroups + grp;
      w[k] = make_uint4(0, 0, 0, 0);
      if (item < n_items) {
        const int j = a.toks > 1 ? item / n_here : 0;
        w[k] = *reinterpret_cast<const uint4*>(a.qkv + (tok0 + j) * a.ld + (int64_t)(head0 + item - j * n_here) * kD + c0);
      }
    }
    if (tid < a.toks && tok0 + tid < tokens) {
      const int64_t tok = tok0 + tid;
      const int64_t s = tokens < (1ll << 31) ? (int64_t)((uint32_t)tok / (uint32_t)a.t_new) : tok / a.t_new;
      const int64_t t = tok - s * a.t_new, p0 = a.pos[s];
      const bool fits = a.c.k8 && rows8_fits(p0, a.t_new, a.c.cap);
      s_tok[tid] = {tok, s * a.n_heads * a.t_new + t, fits ? s * a.n_heads * a.c.cap + p0 + t : -1, p0 + t};
      if (a.c.k8 && t == 0 && head0 == 0) {
        if (!fits)
          set_status(a.status, BPKV_DEV_OVERFLOW);
        else if (!a.bump)
          a.c.seq_len[s] = p0 + a.t_new;
      }
    }
    __syncthreads();
    for (int i = tid; i < a.toks * 64; i += kQkvThreads) {
      const int j = i >> 6, f = i & 63;
      if (f < half && tok0 + j < tokens) {
        const uint64_t ph = (uint64_t)s_tok[j].pos * s_turns[f];
        const float u = (float)(int32_t)(ph >> 32) * 4.6566128730773926e-10f;  // half turns: 2^-31
        float sn, cs;
        sincospif(u, &sn, &cs);
        s_cs[j][f] = make_float2(cs, sn);
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kQkvPer; ++k) {
      if (k * kQkvGroups >= n_items) break;
      const int item = k * kQkvGroups + grp;
      const bool there = item < n_items;
      const int j = there && a.toks > 1 ? item / n_here : 0;
      const int head = head0 + (there ? item - j * n_here : 0);
      const QkvToken& tk = s_tok[j];
      const int kind = head < n_q ? 0 : head < n_q + a.n_heads ? 1 : 2;  // query, key, value
      float y[8] = {__uint_as_float(w[k].x << 16), __uint_as_float(w[k].x & 0xffff0000u),
                    __uint_as_float(w[k].y << 16), __uint_as_float(w[k].y & 0xffff0000u),
                    __uint_as_float(w[k].z << 16), __uint_as_float(w[k].z & 0xffff0000u),
                    __uint_as_float(w[k].w << 16), __uint_as_float(w[k].w & 0xffff0000u)};
      if (__any_sync(0xffffffffu, kind < 2)) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const bool norm = kind == 0 ? norm_q : kind == 1 && norm_k;
        const float* wt = s_w[kind & 1];
        const float r = rsqrtf(ss * (1.f / kD) + a.eps);
        if (norm) {
          const float4 w0 = *reinterpret_cast<const float4*>(wt + c0), w1 = *reinterpret_cast<const float4*>(wt + c0 + 4);
          y[0] *= r * w0.x;
          y[1] *= r * w0.y;
          y[2] *= r * w0.z;
          y[3] *= r * w0.w;
          y[4] *= r * w1.x;
          y[5] *= r * w1.y;
          y[6] *= r * w1.z;
          y[7] *= r * w1.w;
        }
        const float2* cs = s_cs[j];
        if constexpr (ROT == kRotPairs) {
          if (kind < 2) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              if (c0 + i < a.rot) {
                const float2 v = cs[(c0 + i) / 2];
                const float p = y[i], q = y[i + 1];
                y[i] = p * v.x - q * v.y;
                y[i + 1] = q * v.x + p * v.y;
              }
            }
          }
        } else if constexpr (ROT == kRotHalves) {
          // the partner channels are the same eight of lane l +- half / 8
          const int d = half / 8;
          const bool first = l16 < d, in = kind < 2 && l16 < 2 * d;
          const int src = first ? l16 + d : l16 < 2 * d ? l16 - d : l16;
          const float4* v4 = reinterpret_cast<const float4*>(cs + (in ? (first ? c0 : c0 - half) : 0));
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float o0 = __shfl_sync(0xffffffffu, y[i], src, 16), o1 = __shfl_sync(0xffffffffu, y[i + 1], src, 16);
            if (in) {
              const float4 v = v4[i / 2];
              y[i] = y[i] * v.x + (first ? -o0 : o0) * v.y;
              y[i + 1] = y[i + 1] * v.z + (first ? -o1 : o1) * v.w;
            }
          }
        } else if (kind < 2) {
          const uint16_t* x = a.qkv + tk.tok * a.ld + (int64_t)head * kD;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int c = c0 + i;
            if (c < a.rot) {
              const bool first = c < half;
              const int pc = first ? c + half : c - half;
              float o = bf16_bits_to_float(x[pc]);
              if (norm) o *= r * wt[pc];
              const float2 v = cs[first ? c : pc];
              y[i] = y[i] * v.x + (first ? -o : o) * v.y;
            }
          }
        }
        if (kind < 2)
          w[k] = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
      }
      const int h = kind == 0 ? 0 : kind == 1 ? head - n_q : head - n_q - a.n_heads;
      if (there && kind == 0) {
        const int64_t o = (tk.tok * n_q + head) * kD + c0;
        if (a.q_bf16) {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.q_out) + o) = w[k];
        } else {
          float4* q = reinterpret_cast<float4*>(static_cast<float*>(a.q_out) + o);
          q[0] = make_float4(y[0], y[1], y[2], y[3]);
          q[1] = make_float4(y[4], y[5], y[6], y[7]);
        }
      } else if (there) {
        uint16_t* rows = kind == 1 ? a.k_out : a.v_out;
        if (rows) *reinterpret_cast<uint4*>(rows + (tk.row + (int64_t)h * a.t_new) * kD + c0) = w[k];
      }
      if (a.c.k8 && __any_sync(0xffffffffu, kind > 0))
        store_row8(w[k], kind == 1 ? a.c.k8 : a.c.v8, kind == 1 ? a.c.kexp : a.c.vexp, tk.row8 + (int64_t)h * a.c.cap,
                   l16, tk.row8 >= 0 && there && kind > 0);
    }
    __syncthreads();
  }
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
  // as many whole tokens as a CTA's 48 heads hold, but enough CTAs for all SMs
  int toks = heads >= kQkvHeads ? 1 : kQkvHeads / heads;
  while (toks > 1 && tokens / toks < 152) toks /= 2;
  a.toks = toks > kQkvTokens ? kQkvTokens : toks;
  const dim3 grid((unsigned)min64((tokens + a.toks - 1) / a.toks, 152 * 16), (heads + kQkvHeads - 1) / kQkvHeads);
  const auto kernel = a.pairs ? k_qkv_rope<kRotPairs> : a.rot % 16 == 0 ? k_qkv_rope<kRotHalves> : k_qkv_rope<kRotAny>;
  const cudaError_t e = launch_pdl(kernel, grid, dim3(kQkvThreads), 0, st, a);
  if (e != cudaSuccess || !a.bump) return e;
  return launch_rows8_bump(*q.rows8, q.t_new, st);
}

}  // namespace bpkv
