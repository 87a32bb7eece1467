// How the shared-prefix attention's work is laid out: units, tiles, the cut of
// the tiles over workers, and where the partial results go.
//
// A unit is a set of query rows that attend over the same KV rows: the query
// heads of all sequences of one prefix, 256 at a time (16 where the prefixes are
// short), for each KV head; and for each sequence and KV head its own rows with
// its G query heads.  Units of more than kFew rows belong to the tensor-core
// kernel (k_shared_wide, tiles of kWideTile tokens, a CTA per worker), the
// others to the streaming kernel (k_shared_few, a warp per worker).  Each
// kernel's tiles form one list, cut into equal stretches, one per worker; a
// worker's part of a unit is a segment and leaves its rows' (m, l, o).  Lengths
// are read on the device, so the cut fits ragged batches; every CTA works the
// same plan out for itself.
//
// Where all sequences' own rows are short, there is no streaming kernel behind
// the wide one (Args::finish): the wide kernel takes every prefix unit, also
// those of at most kFew rows, and k_shared_unit each sequence's own rows.  Short
// sequences and prefixes need no plan at all (k_shared_unit alone).
#pragma once

#include <atomic>

#include "common.cuh"

namespace bpkv {
namespace shared {

// Lets a kernel use `bytes` of shared memory, once for each device; `done` is
// the kernel's own.
template <typename K>
inline cudaError_t allow_smem(K* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// L2 policy of rows that are streamed once: they go before anything else, so
// that a cache larger than L2 does not push out what the next kernels read (the
// partial results, and the kernels' own instructions).
__device__ __forceinline__ uint64_t evict_first_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}

constexpr float kLogScale = 0.08838834764831845f * 1.4426950408889634f;  // log2(e) / sqrt(D)

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr int kWideTile = 128;       // tokens of a wide tile, rows of a stream
constexpr int kPair = 2 * kWideTile; // rows of a wide unit at most
constexpr int kPairLog = 8;
constexpr int kFew = 16;             // rows a streaming unit has at most
constexpr int kFewLog = 4;
constexpr int kMaxSeq = BPKV_SHARED_MAX_SEQ;
constexpr int kSms = 152;
constexpr int kFewWarps = 8;         // per CTA of the streaming kernel

// A query row's partials, as rows of the partial buffers: of pre_n segments of
// its prefix, then of own_n segments of its own rows.
struct Parts {
  int64_t pre, own;   // first
  int32_t pre_n, own_n;
  int32_t pre_step;   // rows from one segment to the next
  int32_t pad;
};
static_assert(sizeof(Parts) == 32, "two 16-byte loads");

struct Args {
  const int32_t* prefix_of;
  const int64_t* plen;  // NULL: no prefixes
  const int64_t* len;
  int64_t pcap, cap;
  int32_t n_prefix, n_seq, n_heads, group;
  uint32_t group_inv;  // 2^16 / group rounded up: x group_inv >> 16 is x / group for every row x of a prefix
  const uint16_t* q;
  const void* rows[2][2];     // [prefix, own][K, V]
  const uint8_t* exps[2][2];  // scale exponents of 8-bit rows
  Parts* parts;               // [N][H][G]
  float* part_o;              // [rows][D]
  float2* part_ml;            // [rows] maximum (log2 domain) and sum
  int64_t few0, own0;         // first rows of the streaming kernel's prefix units and own units
  int32_t* status;
  int32_t wide_ctas, few_workers;
  int32_t unit_log;           // rows of a prefix unit: kPairLog, or kFewLog without the wide kernel
  int32_t stages;             // of the wide kernel's ring
  int32_t few_rows;           // rows of the largest prefix unit that is streamed: kFew, or 0
  int32_t finish;             // k_shared_unit joins: the wide kernel writes the table of partials
};

// Prefix items there can be with units of 2^log rows: one more for every full unit.
constexpr int max_pre(int log) { return kMaxSeq + (kMaxSeq * BPKV_MAX_GROUP >> log); }

// What every CTA works out; the wide kernel needs no streaming tiles.
template <int MAX_PRE, bool STREAM>
struct Plan {
  static constexpr bool kStream = STREAM;
  int64_t wide[MAX_PRE + 1];  // wide tiles before each prefix item, for one KV head
  // streaming tiles before each prefix item, then before each sequence
  int64_t few[STREAM ? MAX_PRE + kMaxSeq + 1 : 1];
  uint16_t order[kMaxSeq];     // sequences by prefix
  uint16_t rank[kMaxSeq];      // each sequence's place among its prefix's
  int16_t pof[kMaxSeq];        // prefix of each sequence, -1: none
  uint16_t cnt[kMaxSeq];       // sequences of each prefix
  uint16_t first[kMaxSeq];     // where they begin in order
  uint16_t item0[kMaxSeq];     // first item of each prefix
  int32_t tok[kMaxSeq];        // its tokens
  int32_t own[STREAM ? kMaxSeq : 1];  // tokens of each sequence's own
  uint16_t it_p[MAX_PRE];      // prefix of each prefix item
  int32_t n_pre;               // prefix items
};

using WidePlan = Plan<max_pre(kPairLog), false>;
using FewPlan = Plan<max_pre(kFewLog), true>;

// a / b of numbers that are not negative; in 32 bits where they fit, which they
// nearly always do: a 64-bit division is some 100 dependent instructions.
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

__device__ __forceinline__ int64_t tokens_of(int64_t n, int64_t cap) { return max64(0, min64(n, cap)); }

// Exclusive sums of n values in place, the total behind them; one warp.
__device__ __forceinline__ void warp_sums(int64_t* v, int n) {
  const int lane = threadIdx.x & 31;
  int64_t sum = 0;
  for (int b = 0; b < n; b += 32) {
    const int64_t t = b + lane < n ? v[b + lane] : 0;
    int64_t c = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c += u;
    }
    if (b + lane < n) v[b + lane] = sum + c - t;
    sum += __shfl_sync(0xffffffffu, c, 31);
  }
  if (lane == 0) v[n] = sum;
}

static_assert(kMaxSeq * BPKV_MAX_GROUP * (BPKV_MAX_GROUP - 1) < 1 << 16, "x / group by group_inv");

template <typename P>
__device__ __forceinline__ int pre_rows(const Args& a, const P& p, int item) {
  const int x = p.it_p[item];
  return min(1 << a.unit_log, p.cnt[x] * a.group - ((item - p.item0[x]) << a.unit_log));
}

// All threads of the CTA (at least 256); ends with a barrier.  The lengths are
// loaded at once; a single prefix, the usual case, needs no search for who has
// which.
template <typename Q>
__device__ __forceinline__ void make_plan(const Args& a, Q& p, int few_tile) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31;
  const int P = a.plen ? a.n_prefix : 0, N = a.n_seq;
  constexpr int kPer = kMaxSeq / 256;
  int64_t own[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = tid + k * nt;
    own[k] = Q::kStream && i < N ? tokens_of(a.len[i], a.cap) : 0;
  }
  if (P == 0) {
    for (int i = tid; i < N; i += nt) p.pof[i] = -1;
    if (tid == 0) p.n_pre = 0;
  } else {
    for (int x = tid; x < P; x += nt) {
      p.cnt[x] = 0;
      p.tok[x] = (int32_t)tokens_of(a.plen[x], a.pcap);
    }
    for (int i = tid; i < N; i += nt) {
      const int x = a.prefix_of ? a.prefix_of[i] : 0;
      p.pof[i] = (int16_t)(x >= 0 && x < P ? x : -1);
      if (!a.prefix_of) p.rank[i] = (uint16_t)i;
    }
    __syncthreads();
    if (a.prefix_of) {
      for (int i = tid; i < N; i += nt) {
        const int x = p.pof[i];
        int rank = 0, cnt = 0;
        for (int j = 0; j < N; ++j) {
          const bool same = p.pof[j] == x;
          cnt += same;
          rank += same && j < i;
        }
        if (x >= 0) p.cnt[x] = (uint16_t)cnt;
        p.rank[i] = (uint16_t)rank;
      }
      __syncthreads();
    }
    if (tid < 32) {
      int at = 0, item = 0;
      for (int b = 0; b < P; b += 32) {
        const int x = b + lane;
        const int c = x >= P ? 0 : a.prefix_of ? p.cnt[x] : x == 0 ? N : 0;
        const int it = x < P && p.tok[x] > 0 ? (c * a.group + (1 << a.unit_log) - 1) >> a.unit_log : 0;
        int sc = c, si = it;
        if (P > 1) {
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, sc, o), w = __shfl_up_sync(0xffffffffu, si, o);
            if (lane >= o) {
              sc += u;
              si += w;
            }
          }
        }
        if (x < P) {
          p.cnt[x] = (uint16_t)c;
          p.first[x] = (uint16_t)(at + sc - c);
          p.item0[x] = (uint16_t)(item + si - it);
          for (int k = 0; k < it; ++k) p.it_p[item + si - it + k] = (uint16_t)x;
        }
        const int last = P > 1 ? 31 : 0;
        at += __shfl_sync(0xffffffffu, sc, last);
        item += __shfl_sync(0xffffffffu, si, last);
      }
      if (lane == 0) p.n_pre = item;
    }
  }
  __syncthreads();
  const int n_pre = p.n_pre;
  for (int i = tid; i < n_pre; i += nt) {
    const int64_t n = p.tok[p.it_p[i]];
    const bool wide = pre_rows(a, p, i) > a.few_rows;
    p.wide[i] = wide ? (n + kWideTile - 1) / kWideTile : 0;
    if constexpr (Q::kStream) p.few[i] = wide ? 0 : (n + few_tile - 1) / few_tile;
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = tid + k * nt;
    if (i < N) {
      if constexpr (Q::kStream) p.own[i] = (int32_t)own[k];
      if constexpr (Q::kStream) p.few[n_pre + i] = (own[k] + few_tile - 1) / few_tile;
      const int x = p.pof[i];
      if (x >= 0) p.order[p.first[x] + p.rank[i]] = (uint16_t)i;
    }
  }
  __syncthreads();
  if (tid < 32) warp_sums(p.wide, n_pre);
  if constexpr (Q::kStream)
    if (tid >= 32 && tid < 64) warp_sums(p.few, n_pre + N);
  __syncthreads();
}

// Worker w of n takes tiles [w T / n, (w + 1) T / n) of a list of T.
struct Share {
  int64_t total;
  int64_t n;  // workers that take part: no more than tiles
  __device__ Share(int64_t t, int64_t workers) : total(t), n(min64(t, workers)) {}
  __device__ int64_t lo(int64_t w) const { return quot(w * total, n); }
  __device__ int64_t owner(int64_t tile) const { return quot((tile + 1) * n - 1, total); }
};

// Copies of a wide unit's rows among the 128 of a stream.  With 64 rows or
// fewer the copies' softmax threads share the tile's tokens, so that all four
// warps work; each copy has its own m, l and o until the segment's end.
__device__ __forceinline__ int copies_of(int rows) { return rows <= kWideTile / 4 ? 4 : rows <= kWideTile / 2 ? 2 : 1; }

// What a logit may reach before m follows it, and what is taken from the logits
// (times unit) before exp2.  8-bit rows' weights have the range of a half: both
// are rounded so that x <= lazy_top(m) never makes more than 2^(lazy + shift),
// also where the logits' last bit is worth more than the shift.  bf16 weights
// have float32's range.
template <int BITS>
__device__ __forceinline__ float lazy_top(float m, float lazy) {
  return BITS == 8 ? __fadd_rd(m, lazy) : m + lazy;
}
template <int BITS>
__device__ __forceinline__ float shifted(float m, float unit, float shift) {
  return BITS == 8 ? __fadd_ru(m, -shift) : fmaf(m, unit, -shift);
}

// Partial rows of segment (unit, worker): the segments in order have ascending
// unit + worker, each its own.
__device__ __forceinline__ int64_t wide_row(int64_t unit, int64_t cta) { return (unit + cta) * kPair; }
__device__ __forceinline__ int64_t few_row(const Args& a, int64_t unit, int64_t worker) {
  return a.few0 + (unit + worker) * kFew;
}
__device__ __forceinline__ int64_t own_row(const Args& a, int64_t unit, int64_t worker) {
  return a.own0 + (unit + worker) * a.group;
}

// Where the partials of query row r = (sequence, KV head, head of the group) will be.
template <typename P>
__device__ __forceinline__ Parts parts_of(const Args& a, const P& p, int64_t r) {
  const Share wide(p.wide[p.n_pre] * a.n_heads, a.wide_ctas);
  const Share few(P::kStream ? p.few[p.n_pre + a.n_seq] * a.n_heads : 0, a.few_workers);
  const int64_t u = quot(r, a.group);
  const int g = (int)(r - u * a.group), i = (int)quot(u, a.n_heads), h = (int)(u - (int64_t)i * a.n_heads);
  Parts q = {};
  const int x = p.pof[i];
  const int row = x >= 0 ? p.rank[i] * a.group + g : 0, item = x >= 0 ? p.item0[x] + (row >> a.unit_log) : 0;
  if (x >= 0 && item < p.n_pre && p.it_p[item] == x) {  // a prefix of length 0 has no items
    const int in = row & ((1 << a.unit_log) - 1), rows = pre_rows(a, p, item);
    const bool is_wide = !P::kStream || rows > a.few_rows;
    const Share& share = is_wide ? wide : few;
    const int64_t* sums = is_wide ? p.wide : p.few;
    const int64_t tiles = sums[item + 1] - sums[item], at = sums[item] * a.n_heads + h * tiles;
    const int64_t w0 = share.owner(at), unit = (int64_t)item * a.n_heads + h;
    q.pre_n = (int)(share.owner(at + tiles - 1) - w0) + 1;
    if (is_wide) {
      q.pre = wide_row(unit, w0) + in;
      q.pre_step = kPair;
    } else {
      q.pre = few_row(a, unit, w0) + in;
      q.pre_step = kFew;
    }
  }
  if constexpr (P::kStream) {
    const int own = p.n_pre + i;
    const int64_t tiles = p.few[own + 1] - p.few[own], at = p.few[own] * a.n_heads + h * tiles;
    if (tiles > 0) {
      const int64_t w0 = few.owner(at);
      q.own_n = (int)(few.owner(at + tiles - 1) - w0) + 1;
      q.own = own_row(a, u, w0) + g;
    }
  }
  return q;
}

}  // namespace shared
}  // namespace bpkv
