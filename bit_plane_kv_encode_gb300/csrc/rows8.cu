// Rows of a KV cache quantised to 8 bits as they are written, and read back.
//
// Bound by bytes.  Sixteen lanes take a row of K and the same row of V, eight
// channels each (16 bytes of bf16, 8 of codes); with many rows each group
// takes four, its loads issued together, so that enough bytes are in flight.
// The rows' exponent bytes of a CTA meet in shared memory and leave as runs of
// neighbouring bytes.
//
// Measured on a GB300: 32768 tokens of 8 KV heads quantised (202 MB) in 30.6 us,
// 6.6 TB/s; 4 x 8191 tokens read back (202 MB) in 32.6 us, 6.2 TB/s.  With one
// row a group and an exponent byte stored at a time: 36.6 and 36.5 us.  One
// token of 32 sequences: 2.1 us, latency.
#include "rows8_core.cuh"

namespace bpkv {

constexpr int kR8Threads = 256;
constexpr int kR8Groups = kR8Threads / 16;
constexpr int kR8Many = 4;  // rows of a group when there are many

// Rows per group: four once that still leaves every SM four CTAs; below, a call
// is a few microseconds of latency, which more CTAs of less work keep short.
bool many_rows(int64_t rows) { return rows >= (int64_t)152 * 4 * kR8Groups * kR8Many; }

// r = u n + t, in 32 bits where that is enough.
__device__ __forceinline__ void split(int64_t r, int32_t n, int64_t& u, int64_t& t) {
  u = r < (1ll << 32) ? (int64_t)((uint32_t)r / (uint32_t)n) : r / n;
  t = r - u * n;
}

struct AppendArgs {
  Rows8Out c;
  const uint16_t* k_new;
  const uint16_t* v_new;
  const int64_t* start;
  int32_t* status;
  int32_t n_seq, n_heads, t_new;
  int32_t per;   // rows of a CTA
  int32_t bump;  // the lengths are raised by a launch of their own
};

template <int R>
__global__ void __launch_bounds__(kR8Threads) k_rows8_append(const __grid_constant__ AppendArgs a) {
  pdl_enter();
  __shared__ uint8_t s_exp[2][kR8Groups * R];
  __shared__ int64_t s_dst[kR8Groups * R];  // -1: not written
  const int tid = threadIdx.x, l16 = tid & 15, grp = tid >> 4;
  const int64_t rows = (int64_t)a.n_seq * a.n_heads * a.t_new, r0 = (int64_t)blockIdx.x * a.per;
  const int64_t end = min64(rows, r0 + a.per);
  uint4 w[R][2];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t r = r0 + i * kR8Groups + grp;
    w[i][0] = w[i][1] = make_uint4(0, 0, 0, 0);
    if (r < end) {
      w[i][0] = __ldcs(reinterpret_cast<const uint4*>(a.k_new + r * kD + l16 * 8));
      w[i][1] = __ldcs(reinterpret_cast<const uint4*>(a.v_new + r * kD + l16 * 8));
    }
  }
  int64_t s = 0, len = -1;  // of the thread that has a sequence's first row: its new length
  if (tid < kR8Groups * R) {
    const int64_t r = r0 + tid;
    int64_t dst = -1;
    if (r < end) {
      int64_t unit, t, h;
      split(r, a.t_new, unit, t);
      split(unit, a.n_heads, s, h);
      const int64_t p = a.start[s];
      if (rows8_fits(p, a.t_new, a.c.cap)) dst = unit * a.c.cap + p + t;
      if (t == 0 && h == 0) {
        if (dst < 0)
          set_status(a.status, BPKV_DEV_OVERFLOW);
        else if (!a.bump)
          len = p + a.t_new;
      }
    }
    s_dst[tid] = dst;
  }
  __syncthreads();
  if (len >= 0) a.c.seq_len[s] = len;  // the CTA has read the old one
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t dst = s_dst[i * kR8Groups + grp];
    const int ke = row_exponent(w[i][0]), ve = row_exponent(w[i][1]);
    if (l16 == 0) {
      s_exp[0][i * kR8Groups + grp] = (uint8_t)(ke + kExpBias);
      s_exp[1][i * kR8Groups + grp] = (uint8_t)(ve + kExpBias);
    }
    if (dst >= 0) {
      *reinterpret_cast<uint2*>(a.c.k8 + dst * kD + l16 * 8) = row_codes(w[i][0], ke);
      *reinterpret_cast<uint2*>(a.c.v8 + dst * kD + l16 * 8) = row_codes(w[i][1], ve);
    }
  }
  __syncthreads();
  if (tid < 2 * kR8Groups * R) {
    const int kv = tid / (kR8Groups * R), x = tid % (kR8Groups * R);
    if (s_dst[x] >= 0) (kv ? a.c.vexp : a.c.kexp)[s_dst[x]] = s_exp[kv][x];
  }
}

// Lengths after an append at the lengths themselves, once every CTA has read them.
__global__ void k_rows8_bump(int64_t* seq_len, int n_seq, int32_t t_new, int64_t cap) {
  pdl_enter();
  const int s = blockIdx.x * blockDim.x + threadIdx.x;
  if (s < n_seq && rows8_fits(seq_len[s], t_new, cap)) seq_len[s] += t_new;
}

cudaError_t launch_rows8_bump(const bpkv_rows8& c, int32_t t_new, cudaStream_t st) {
  return launch_pdl(k_rows8_bump, dim3((c.n_seq + 127) / 128), dim3(128), 0, st, c.seq_len, (int)c.n_seq, t_new,
                    c.cap_tokens);
}

cudaError_t launch_rows8_append(const bpkv_rows8& c, const uint16_t* k_new, const uint16_t* v_new, int32_t t_new,
                                const int64_t* start, int32_t* status, cudaStream_t st) {
  const bool at_len = start == nullptr || start == c.seq_len;
  const int64_t rows = (int64_t)c.n_seq * c.n_kv_heads * t_new, of_seq = (int64_t)c.n_kv_heads * t_new;
  // Lengths that are also the starts may change only when all have read them.
  // A decode step's rows of a sequence fit one CTA, which then raises the length
  // itself (32 sequences of 8 heads: 1.9 us a call in a graph, 3.8 outside,
  // instead of 2.6 and 5.4); for more rows a second launch does.
  const bool whole = at_len && of_seq <= kR8Groups * kR8Many, bump = at_len && !whole;
  const bool many = whole ? of_seq > kR8Groups : many_rows(rows);
  const int per = whole ? (int)of_seq : kR8Groups * (many ? kR8Many : 1);
  AppendArgs a{{c.k8, c.v8, c.kexp, c.vexp, c.seq_len, c.cap_tokens}, k_new, v_new, at_len ? c.seq_len : start, status,
               c.n_seq, c.n_kv_heads, t_new, per, bump ? 1 : 0};
  const cudaError_t e = launch_pdl(many ? k_rows8_append<kR8Many> : k_rows8_append<1>,
                                   dim3((unsigned)((rows + per - 1) / per)), dim3(kR8Threads), 0, st, a);
  if (e != cudaSuccess || !bump) return e;
  return launch_rows8_bump(c, t_new, st);
}

struct AcceptArgs {
  Rows8Out c;
  const uint16_t* k_new;
  const uint16_t* v_new;
  const int64_t* start;
  const int32_t* path;   // NULL: token j itself
  const int32_t* count;
  int32_t* status;
  int32_t n_seq, n_heads, t;
  int32_t bump;  // the lengths are set by a launch of their own
};

__device__ __forceinline__ bool accept_fits(int64_t start, int32_t count, int32_t t, int64_t cap) {
  return count >= 0 && count <= t && rows8_fits(start, count, cap);
}

// As k_rows8_append, but of a sequence's t tokens only the first count rows are
// there, and each goes by way of the path: one more dependent load before the
// row's own.  A thread a row finds out where it comes from and goes.
template <int R>
__global__ void __launch_bounds__(kR8Threads) k_rows8_accept(const __grid_constant__ AcceptArgs a) {
  pdl_enter();
  __shared__ uint8_t s_exp[2][kR8Groups * R];
  __shared__ int64_t s_from[kR8Groups * R], s_dst[kR8Groups * R];  // -1: not written
  const int tid = threadIdx.x, l16 = tid & 15, grp = tid >> 4;
  const int64_t rows = (int64_t)a.n_seq * a.n_heads * a.t, r0 = (int64_t)blockIdx.x * (kR8Groups * R);
  bool mine = false;
  if (tid < kR8Groups * R) {
    const int64_t r = r0 + tid;
    int64_t from = -1, dst = -1;
    if (r < rows) {
      int64_t unit, j, s, h;
      split(r, a.t, unit, j);
      split(unit, a.n_heads, s, h);
      const int64_t p = a.start[s];
      const int32_t n = a.count[s];
      const int32_t node = a.path ? a.path[s * a.t + j] : (int32_t)j;
      const bool fits = accept_fits(p, n, a.t, a.c.cap);
      if (fits && j < n) {
        mine = true;
        from = unit * a.t + min(max(node, 0), a.t - 1);
        dst = unit * a.c.cap + p + j;
        if (h == 0 && (node < 0 || node >= a.t)) set_status(a.status, BPKV_DEV_OVERFLOW);
      }
      if (h == 0 && j == 0) {
        if (!fits) set_status(a.status, BPKV_DEV_OVERFLOW);
        else if (!a.bump) a.c.seq_len[s] = p + n;
      }
    }
    s_from[tid] = from;
    s_dst[tid] = dst;
  }
  if (!__syncthreads_or(mine)) return;  // padding
  uint4 w[R][2];
  int64_t dst[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t from = s_from[i * kR8Groups + grp];
    dst[i] = s_dst[i * kR8Groups + grp];
    w[i][0] = w[i][1] = make_uint4(0, 0, 0, 0);
    if (from >= 0) {
      w[i][0] = __ldg(reinterpret_cast<const uint4*>(a.k_new + from * kD + l16 * 8));
      w[i][1] = __ldg(reinterpret_cast<const uint4*>(a.v_new + from * kD + l16 * 8));
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int ke = row_exponent(w[i][0]), ve = row_exponent(w[i][1]);
    if (l16 == 0) {
      s_exp[0][i * kR8Groups + grp] = (uint8_t)(ke + kExpBias);
      s_exp[1][i * kR8Groups + grp] = (uint8_t)(ve + kExpBias);
    }
    if (dst[i] >= 0) {
      *reinterpret_cast<uint2*>(a.c.k8 + dst[i] * kD + l16 * 8) = row_codes(w[i][0], ke);
      *reinterpret_cast<uint2*>(a.c.v8 + dst[i] * kD + l16 * 8) = row_codes(w[i][1], ve);
    }
  }
  __syncthreads();
  if (tid < 2 * kR8Groups * R) {
    const int kv = tid / (kR8Groups * R), x = tid % (kR8Groups * R);
    if (s_dst[x] >= 0) (kv ? a.c.vexp : a.c.kexp)[s_dst[x]] = s_exp[kv][x];
  }
}

// Lengths that are also the starts, once every CTA has read them.
__global__ void k_rows8_accept_len(const __grid_constant__ AcceptArgs a) {
  pdl_enter();
  const int s = blockIdx.x * blockDim.x + threadIdx.x;
  if (s < a.n_seq && accept_fits(a.c.seq_len[s], a.count[s], a.t, a.c.cap)) a.c.seq_len[s] += a.count[s];
}

cudaError_t launch_rows8_accept(const bpkv_rows8& c, const uint16_t* k_new, const uint16_t* v_new, int32_t t,
                                const int64_t* start, const int32_t* path, const int32_t* count, int32_t* status,
                                cudaStream_t st) {
  const int64_t rows = (int64_t)c.n_seq * c.n_kv_heads * t;
  const bool many = many_rows(rows), bump = start == c.seq_len;
  const int per = kR8Groups * (many ? kR8Many : 1);
  const AcceptArgs a{{c.k8, c.v8, c.kexp, c.vexp, c.seq_len, c.cap_tokens}, k_new, v_new, start, path, count, status,
                     c.n_seq, c.n_kv_heads, t, bump ? 1 : 0};
  const cudaError_t e = launch_pdl(many ? k_rows8_accept<kR8Many> : k_rows8_accept<1>,
                                   dim3((unsigned)((rows + per - 1) / per)), dim3(kR8Threads), 0, st, a);
  if (e != cudaSuccess || !bump) return e;
  return launch_pdl(k_rows8_accept_len, dim3((c.n_seq + 127) / 128), dim3(128), 0, st, a);
}

struct ReadArgs {
  const uint8_t* codes[2];
  const uint8_t* exps[2];
  uint16_t* out[2];
  const int64_t* seq_len;
  int64_t cap, t0;
  int32_t n_seq, n_heads, n;
};

__device__ __forceinline__ uint32_t bf16x2_of(uint16_t codes, float s) {
  const float2 f = __half22float2(half2_of_e4m3x2(codes));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
  return *reinterpret_cast<const uint32_t*>(&b);
}

template <int R>
__global__ void __launch_bounds__(kR8Threads) k_rows8_read(const __grid_constant__ ReadArgs a) {
  pdl_enter();
  const int l16 = threadIdx.x & 15;
  const int64_t rows = (int64_t)a.n_seq * a.n_heads * a.n;
  const int64_t r0 = (int64_t)blockIdx.x * (kR8Groups * R) + threadIdx.x / 16;
  uint2 c[R][2];
  int e[R][2];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t r = r0 + i * kR8Groups;
    c[i][0] = c[i][1] = make_uint2(0, 0);
    e[i][0] = e[i][1] = 0;
    if (r < rows) {
      int64_t unit, t, s, h;
      split(r, a.n, unit, t);
      split(unit, a.n_heads, s, h);
      if (a.t0 + t < min64(a.seq_len[s], a.cap)) {
        const int64_t row = unit * a.cap + a.t0 + t;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
          if (a.out[kv]) {
            c[i][kv] = __ldcs(reinterpret_cast<const uint2*>(a.codes[kv] + row * kD + l16 * 8));
            e[i][kv] = a.exps[kv][row];
          }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t r = r0 + i * kR8Groups;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
      if (r < rows && a.out[kv]) {
        const float f = exp2i(min(max(e[i][kv] - kExpBias, kExpMin), kExpMax));
        const uint2 x = c[i][kv];
        *reinterpret_cast<uint4*>(a.out[kv] + r * kD + l16 * 8) = make_uint4(
            bf16x2_of(x.x & 0xffffu, f), bf16x2_of(x.x >> 16, f), bf16x2_of(x.y & 0xffffu, f), bf16x2_of(x.y >> 16, f));
      }
  }
}

cudaError_t launch_rows8_read(const bpkv_rows8& c, int64_t t0, int32_t n, uint16_t* k_out, uint16_t* v_out,
                              cudaStream_t st) {
  ReadArgs a{{c.k8, c.v8}, {c.kexp, c.vexp}, {k_out, v_out}, c.seq_len, c.cap_tokens, t0, c.n_seq, c.n_kv_heads, n};
  const int64_t rows = (int64_t)c.n_seq * c.n_kv_heads * n;
  const int per = kR8Groups * (many_rows(rows) ? kR8Many : 1);
  return launch_pdl(many_rows(rows) ? k_rows8_read<kR8Many> : k_rows8_read<1>, dim3((unsigned)((rows + per - 1) / per)),
                    dim3(kR8Threads), 0, st, a);
}

}  // namespace bpkv
