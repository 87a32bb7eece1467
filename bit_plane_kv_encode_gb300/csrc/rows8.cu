// Rows of a KV cache quantised to 8 bits as they are written, and read back.
#include "rows8_core.cuh"

namespace bpkv {

constexpr int kR8Threads = 256;
constexpr int kR8Rows = kR8Threads / 16;  // rows a CTA holds at once

struct AppendArgs {
  Rows8Out c;
  const uint16_t* k_new;
  const uint16_t* v_new;
  const int64_t* start;
  int32_t* status;
  int32_t n_seq, n_heads, t_new, bump;
};

__global__ void __launch_bounds__(kR8Threads) k_rows8_append(AppendArgs a) {
  pdl_enter();
  const int l16 = threadIdx.x & 15;
  const int64_t rows = (int64_t)a.n_seq * a.n_heads * a.t_new;
  const int64_t r = (int64_t)blockIdx.x * kR8Rows + threadIdx.x / 16;
  const bool there = r < rows;
  uint4 kw = make_uint4(0, 0, 0, 0), vw = kw;
  int64_t dst = 0;
  bool store = false;
  if (there) {
    const int64_t unit = r / a.t_new, t = r % a.t_new;
    const int64_t s = unit / a.n_heads;
    const int64_t p = a.start[s];
    store = rows8_fits(p, a.t_new, a.c.cap);
    dst = unit * a.c.cap + p + t;
    if (store) {
      kw = *reinterpret_cast<const uint4*>(a.k_new + r * kD + l16 * 8);
      vw = *reinterpret_cast<const uint4*>(a.v_new + r * kD + l16 * 8);
    }
    if (t == 0 && unit % a.n_heads == 0 && l16 == 0) {
      if (!store)
        set_status(a.status, BPKV_DEV_OVERFLOW);
      else if (!a.bump)
        a.c.seq_len[s] = p + a.t_new;
    }
  }
  store_row8(kw, a.c.k8, a.c.kexp, dst, l16, store);
  store_row8(vw, a.c.v8, a.c.vexp, dst, l16, store);
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
  const bool bump = start == nullptr || start == c.seq_len;
  AppendArgs a{{c.k8, c.v8, c.kexp, c.vexp, c.seq_len, c.cap_tokens}, k_new, v_new, bump ? c.seq_len : start, status,
               c.n_seq, c.n_kv_heads, t_new, bump ? 1 : 0};
  const int64_t rows = (int64_t)c.n_seq * c.n_kv_heads * t_new;
  const cudaError_t e =
      launch_pdl(k_rows8_append, dim3((unsigned)((rows + kR8Rows - 1) / kR8Rows)), dim3(kR8Threads), 0, st, a);
  if (e != cudaSuccess || !bump) return e;
  return launch_rows8_bump(c, t_new, st);
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

__global__ void __launch_bounds__(kR8Threads) k_rows8_read(ReadArgs a) {
  pdl_enter();
  const int l16 = threadIdx.x & 15;
  const int64_t rows = (int64_t)a.n_seq * a.n_heads * a.n;
  const int64_t r = (int64_t)blockIdx.x * kR8Rows + threadIdx.x / 16;
  if (r >= rows) return;
  const int64_t unit = r / a.n, x = a.t0 + r % a.n;
  const bool there = x < min64(a.seq_len[unit / a.n_heads], a.cap);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!a.out[i]) continue;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (there) {
      const int64_t row = unit * a.cap + x;
      const uint2 c = *reinterpret_cast<const uint2*>(a.codes[i] + row * kD + l16 * 8);
      const int e = min(max((int)a.exps[i][row] - kExpBias, kExpMin), kExpMax);
      const float s = exp2i(e);
      w = make_uint4(bf16x2_of(c.x & 0xffffu, s), bf16x2_of(c.x >> 16, s), bf16x2_of(c.y & 0xffffu, s),
                     bf16x2_of(c.y >> 16, s));
    }
    *reinterpret_cast<uint4*>(a.out[i] + r * kD + l16 * 8) = w;
  }
}

cudaError_t launch_rows8_read(const bpkv_rows8& c, int64_t t0, int32_t n, uint16_t* k_out, uint16_t* v_out,
                              cudaStream_t st) {
  ReadArgs a{{c.k8, c.v8}, {c.kexp, c.vexp}, {k_out, v_out}, c.seq_len, c.cap_tokens, t0, c.n_seq, c.n_kv_heads, n};
  const int64_t rows = (int64_t)c.n_seq * c.n_kv_heads * n;
  return launch_pdl(k_rows8_read, dim3((unsigned)((rows + kR8Rows - 1) / kR8Rows)), dim3(kR8Threads), 0, st, a);
}

}  // namespace bpkv
