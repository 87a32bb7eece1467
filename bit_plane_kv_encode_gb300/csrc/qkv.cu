// Projected heads to cache rows: RMS norm of query and key heads, position
// rotation and layout in one pass (bpkv_qkv_rope).
//
// Sixteen lanes hold a head, eight channels each, so the mean square is four
// shuffles and both channels of a rotated pair sit in the group: in the same
// lane (neighbouring pairs), in lane l +- rot/16 (halves, rot/2 a multiple of
// 8), or are read a second time (other rot).  The token's cosines and sines
// are computed once per CTA and token in shared memory.
//
// Angles: the position times the frequency in turns, as 64-bit fixed point
// whose wrap-around drops whole turns, is exact however far the position; the
// top 32 bits are the angle within half a turn to 2^-32.
#include "rows8_core.cuh"

namespace bpkv {

constexpr int kQkvThreads = 256;
constexpr int kQkvHeads = kQkvThreads / 16;  // heads a CTA holds at once

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
  int32_t heads_per_cta;
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

__global__ void __launch_bounds__(kQkvThreads) k_qkv_rope(QkvArgs a) {
  pdl_enter();
  __shared__ float2 s_cs[kD / 2];
  __shared__ float s_w[2][kD];
  const int tid = threadIdx.x, l16 = tid & 15;
  const int half = a.rot / 2;
  const bool norm_q = a.q_weight != nullptr, norm_k = a.k_weight != nullptr;
  if (tid < kD) {
    if (norm_q) s_w[0][tid] = a.q_weight[tid];
    if (norm_k) s_w[1][tid] = a.k_weight[tid];
  }
  const uint64_t turns = tid < half ? turns64(a.inv_freq[tid]) : 0;
  const int n_q = a.n_heads * a.group, heads = n_q + 2 * a.n_heads;
  const int head0 = blockIdx.y * a.heads_per_cta;
  const int head1 = min(head0 + a.heads_per_cta, heads);
  const int64_t tokens = (int64_t)a.n_seq * a.t_new;
  for (int64_t tok = blockIdx.x; tok < tokens; tok += gridDim.x) {
    const int64_t s = tok / a.t_new, t = tok % a.t_new;
    const int64_t p0 = a.pos[s];
    if (tid < half) {
      const uint64_t ph = (uint64_t)(p0 + t) * turns;
      const float u = (float)(int32_t)(ph >> 32) * 4.6566128730773926e-10f;  // half turns: 2^-31
      sincospif(u, &s_cs[tid].y, &s_cs[tid].x);
    }
    const bool fits = a.c.k8 && rows8_fits(p0, a.t_new, a.c.cap);
    if (a.c.k8 && tid == 0 && t == 0 && head0 == 0) {
      if (!fits)
        set_status(a.status, BPKV_DEV_OVERFLOW);
      else if (!a.bump)
        a.c.seq_len[s] = p0 + a.t_new;
    }
    __syncthreads();
    for (int hb = head0; hb < head1; hb += kQkvHeads) {
      const int head = hb + tid / 16;
      const bool there = head < head1;
      const uint16_t* x = a.qkv + tok * a.ld + (int64_t)(there ? head : head0) * kD;
      uint4 w = *reinterpret_cast<const uint4*>(x + l16 * 8);
      const int kind = head < n_q ? 0 : head < n_q + a.n_heads ? 1 : 2;  // query, key, value
      float y[8] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                    __uint_as_float(w.y & 0xffff0000u), __uint_as_float(w.z << 16), __uint_as_float(w.z & 0xffff0000u),
                    __uint_as_float(w.w << 16), __uint_as_float(w.w & 0xffff0000u)};
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const bool norm = kind == 0 ? norm_q : kind == 1 && norm_k;
      const float* wt = s_w[kind & 1];
      const float r = rsqrtf(ss * (1.f / kD) + a.eps);
      if (norm) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = y[i] * r * wt[l16 * 8 + i];
      }
      const int c0 = l16 * 8;
      if (a.pairs) {
        if (kind < 2) {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            if (c0 + i < a.rot) {
              const float2 cs = s_cs[(c0 + i) / 2];
              const float p = y[i], q = y[i + 1];
              y[i] = p * cs.x - q * cs.y;
              y[i + 1] = q * cs.x + p * cs.y;
            }
          }
        }
      } else if (half % 8 == 0) {
        // the partner channels are the same eight of lane l +- half / 8
        const int d = half / 8;
        const bool first = l16 < d;
        const int src = first ? l16 + d : l16 < 2 * d ? l16 - d : l16;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float o = __shfl_sync(0xffffffffu, y[i], src, 16);
          if (kind < 2 && c0 < a.rot) {
            const float2 cs = s_cs[first ? c0 + i : c0 + i - half];
            y[i] = first ? y[i] * cs.x - o * cs.y : y[i] * cs.x + o * cs.y;
          }
        }
      } else if (kind < 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = c0 + i;
          if (c < a.rot) {
            const bool first = c < half;
            const int pc = first ? c + half : c - half;
            float o = bf16_bits_to_float(x[pc]);
            if (norm) o = o * r * wt[pc];
            const float2 cs = s_cs[first ? c : pc];
            y[i] = first ? y[i] * cs.x - o * cs.y : y[i] * cs.x + o * cs.y;
          }
        }
      }
      if (kind < 2)
        w = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
      if (there && kind == 0) {
        const int64_t o = (tok * n_q + head) * kD + c0;
        if (a.q_bf16) {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.q_out) + o) = w;
        } else {
          float4* q = reinterpret_cast<float4*>(static_cast<float*>(a.q_out) + o);
          q[0] = make_float4(y[0], y[1], y[2], y[3]);
          q[1] = make_float4(y[4], y[5], y[6], y[7]);
        }
      } else if (there) {
        const int h = kind == 1 ? head - n_q : head - n_q - a.n_heads;
        uint16_t* rows = kind == 1 ? a.k_out : a.v_out;
        if (rows) *reinterpret_cast<uint4*>(rows + ((s * a.n_heads + h) * a.t_new + t) * kD + c0) = w;
      }
      if (a.c.k8) {
        const int h = kind == 1 ? head - n_q : head - n_q - a.n_heads;
        store_row8(w, kind == 1 ? a.c.k8 : a.c.v8, kind == 1 ? a.c.kexp : a.c.vexp,
                   (s * a.n_heads + h) * a.c.cap + p0 + t, l16, fits && there && kind > 0);
      }
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
  const int chunks = (heads + kQkvHeads - 1) / kQkvHeads;
  // few tokens: one CTA for every 16 heads of a token, so that the heads run
  // side by side; many: one CTA takes all heads of a token
  const bool split = tokens * chunks <= 152 * 4;
  a.heads_per_cta = split ? kQkvHeads : heads;
  const int64_t gx = min64(tokens, 152 * 8);
  const cudaError_t e =
      launch_pdl(k_qkv_rope, dim3((unsigned)gx, split ? chunks : 1), dim3(kQkvThreads), 0, st, a);
  if (e != cudaSuccess || !a.bump) return e;
  return launch_rows8_bump(*q.rows8, q.t_new, st);
}

}  // namespace bpkv
