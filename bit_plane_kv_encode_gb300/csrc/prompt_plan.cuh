// How the attention of several new tokens a sequence (bpkv_prompt_attend,
// bpkv_tree_attend, bpkv_tree_attend8) is laid out: units, tiles, the cut of the
// tiles over CTAs, and the shared memory of its kernel.
//
// A unit is a run of a sequence's new tokens with the G query heads of one KV
// head, at most two streams of 128 rows (token by token, head by head, whole
// tokens only: 2 floor(128 / G) tokens), over the keys that its last token sees,
// in tiles of 128.  The units in order (sequence, KV head, run) form one list;
// a unit counts its tiles and kOver more for its start and end.  The list is cut
// into equal stretches, one per CTA; a unit that a cut goes through leaves partial
// rows (m, l, o) in two slots a CTA has, one for a unit that began before it and
// one for a unit that goes on behind it, and k_prompt_join joins them in order.
// Where units are short they are not cut: each counts one.
//
// Long rows of a cache, more than L2 holds, are read again by each run of a
// sequence.  There 2, 4 or 8 runs go side by side, as one unit of the list as long as
// the last of them: as many CTAs take the same stretch, a run each, and come by the same
// tiles at the same time.  As many as lose 1/32 at most to runs that are missing, which
// the lengths tell.
//
// Lengths are read on the device; every CTA works the cut out for itself.
#pragma once

#include "shared_plan.cuh"

namespace bpkv {
namespace prompt {

constexpr int kTile = 128;      // keys of a tile, rows of a stream
constexpr int kRows = 256;      // rows of a unit at most
constexpr int kMaxSeq = BPKV_SHARED_MAX_SEQ;
constexpr int kSms = 152;
constexpr int kSoftmaxWarps = 8;
// What a unit's start and end cost, in tiles: its rows of q, the first S and the
// last O, that nothing of its own overlaps.  With 1 / 2 / 3 / 5, in us: 8191 tokens
// 391 / 367 / 369 / 374, packed prompts 655 / 603 / 616 / 643, trees of 16 sequences
// 58.2 / 55.2 / 54.9 / 55.7.
constexpr int kOver = 2;

constexpr int kBeside = 3;

enum Rows : int32_t { kToken, kSeq, kCache };  // where keys and values lie

// What the CTA that a cut unit begins in leaves for the join.
struct Cut {
  int64_t token;   // first token of the unit in q
  int32_t h;       // KV head
  int32_t tokens;
  int32_t pieces;  // 0: this CTA's last unit is whole
  int32_t step;    // from the CTA of one piece to that of the next
};

struct Args {
  const int64_t* q_start;  // NULL: sequence i has the tokens i t .. (i + 1) t - 1
  const int64_t* len;      // rows of each sequence of a cache; NULL: the keys are those of the new tokens
  const uint64_t* tree;    // NULL: causal
  uint16_t* out;
  const uint8_t* exps[2];  // scale exponents of 8-bit rows
  int64_t cap, tokens;     // rows a sequence of the cache can have; tokens of q
  int32_t n_seq, n_heads, group, t;
  int32_t rows;            // Rows
  int32_t run;             // tokens of a stream: 128 / G
  uint32_t group_inv;      // 2^16 / group rounded up: x group_inv >> 16 is x / group for x below 256
  int32_t split;           // units may be cut
  int32_t beside;          // runs may go side by side
  int32_t once;            // a sequence's tokens are one unit of a KV head
  int32_t slot_rows;       // rows of a slot of partial rows
  float* part_o;           // [slots][slot_rows][D]
  float2* part_ml;         // [slots][slot_rows] maximum (log2 domain) and sum
  Cut* cuts;               // [CTAs]
  int32_t* status;
};

// What the streaming kernel of few new tokens takes (prompt_few.cu).
struct FewArgs {
  const int64_t* q_start;     // NULL: t tokens of each sequence
  const int64_t* len;         // NULL: the keys are those of the new tokens
  const uint64_t* tree;       // NULL: a chain
  const uint16_t* q;
  uint16_t* out;
  const void* rows[1][2];     // K, V
  const uint8_t* exps[1][2];  // scale exponents of 8-bit rows
  int64_t cap, ld_q;
  int64_t step[2];            // bytes from one row to the next
  int32_t tokens;             // of q
  int32_t n_seq, n_heads, group, t;
  int32_t where;              // Rows
  int32_t groups, per;        // a tree's query rows, per (8 or 16) at a time; groups: of a sequence, or of all
  int64_t* starts;            // NULL, or where the tensor cores' half behind this one finds q_start (prompt_few.cu)
};

// Counts are below 2^31: the host makes sure.
struct Plan {
  int32_t cum[kMaxSeq + 1];   // what the sequences before count together
  int32_t start[kMaxSeq + 1]; // a sequence's first token in q
  int32_t n[kMaxSeq];         // its new tokens
  int32_t off[kMaxSeq];       // keys before the first of them (negative: that many of them have none)
  // where this CTA's stretch begins
  int32_t seq, h, run;
  int32_t at, left;           // within that unit, and the stretch's length
  int32_t per;                // a stretch's length (the last ones may be shorter)
  int32_t beside;             // 2^beside runs go side by side: this CTA takes one of each
  int32_t total[kBeside + 1]; // what all count, by beside
};

// Runs of a sequence, keys and tiles of its run b.
__device__ __forceinline__ int runs_of(const Args& a, int t) { return (t + 2 * a.run - 1) / (2 * a.run); }
__device__ __forceinline__ int tiles_of(const Args& a, int t, int off, int b) {
  const int last = a.tree ? t : min(t, (b + 1) * 2 * a.run);
  return max(1, (off + last + kTile - 1) >> 7);
}
__device__ __forceinline__ int count_of(const Args& a, int tiles) { return a.split ? tiles + kOver : 1; }

// Sum of x of this lane and those below.
__device__ __forceinline__ int below(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += u;
  }
  return x;
}

// All threads of the CTA; ends with a barrier.
__device__ __forceinline__ void make_plan(const Args& a, Plan& p) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, N = a.n_seq;
#pragma unroll 1
  for (int i = tid; i <= N; i += nt) {
    p.start[i] = a.q_start ? (int32_t)max64(0, min64(a.q_start[i], a.tokens)) : i * a.t;
    if (i < N) p.off[i] = a.len ? (int32_t)shared::tokens_of(a.len[i], a.cap) : 0;
  }
  __syncthreads();
  if (a.q_start && warp == 0) {  // one that lies before the last one's counts as that: no two sequences share a token
    int top = 0;
#pragma unroll 1
    for (int b = 0; b <= N; b += 32) {
      int x = b + lane <= N ? p.start[b + lane] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x = max(x, u);
      }
      x = max(x, top);
      if (b + lane <= N) p.start[b + lane] = x;
      top = __shfl_sync(0xffffffffu, x, 31);
    }
  }
  if (tid <= kBeside) p.total[tid] = 0;
  __syncthreads();
  int beside = 0;
  if (a.beside) {
#pragma unroll 1
    for (int i = warp; i < N; i += nt / 32) {
      const int t = p.start[i + 1] - p.start[i], runs = runs_of(a, t);
      int sum[kBeside + 1] = {};
#pragma unroll 1
      for (int b = lane; b < runs; b += 32) {
        const int n = count_of(a, tiles_of(a, t, p.off[i] - t, b));
#pragma unroll
        for (int k = 0; k <= kBeside; ++k)
          if (b == runs - 1 || (~b & ((1 << k) - 1)) == 0) sum[k] += n;
      }
#pragma unroll
      for (int k = 0; k <= kBeside; ++k) {
        sum[k] = __reduce_add_sync(0xffffffffu, sum[k]);
        if (lane == 0) atomicAdd(&p.total[k], sum[k] * a.n_heads);
      }
    }
    __syncthreads();
    const uint32_t per = (uint32_t)(p.total[0] + gridDim.x - 1) / gridDim.x;
#pragma unroll 1
    for (int k = kBeside; k > 0 && beside == 0; --k) {
      const uint32_t groups = gridDim.x >> k;
      if (groups > 0 && (p.total[k] + groups - 1) / groups <= per + per / 32) beside = k;
    }
  }
#pragma unroll 1
  for (int i = warp; i < N; i += nt / 32) {
    const int t = p.start[i + 1] - p.start[i], off = a.len ? p.off[i] - t : 0;
    const int units = (runs_of(a, t) + (1 << beside) - 1) >> beside;
    int sum = 0;
#pragma unroll 1
    for (int b = lane; b < units; b += 32) sum += count_of(a, tiles_of(a, t, off, ((b + 1) << beside) - 1));
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0) {
      p.n[i] = t;
      p.off[i] = off;
      p.cum[i] = sum * a.n_heads;
    }
  }
  __syncthreads();
  if (warp == 0) {
    int total = 0;
#pragma unroll 1
    for (int b = 0; b < N; b += 32) {
      const int t = b + lane < N ? p.cum[b + lane] : 0, c = below(t, lane);
      if (b + lane < N) p.cum[b + lane] = total + c - t;
      total += __shfl_sync(0xffffffffu, c, 31);
    }
    if (lane == 0) p.cum[N] = total;
    __syncwarp();
    const int groups = gridDim.x >> beside, group = blockIdx.x >> beside;
    const int per = (uint32_t)(total + groups - 1) / groups;
    const int lo = group < groups ? min((int64_t)group * per, (int64_t)total) : total;
    int at = 0, seq = 0, h = 0, b = 0;
    if (lo < total) {
      int x = 0, y = N - 1;  // the last sequence that begins at or before lo: empty ones end where they begin
#pragma unroll 1
      while (x < y) {
        const int mid = (x + y + 1) / 2;
        if (p.cum[mid] <= lo) x = mid;
        else y = mid - 1;
      }
      seq = x;
      const int head = (uint32_t)(p.cum[seq + 1] - p.cum[seq]) / a.n_heads;
      h = (uint32_t)(lo - p.cum[seq]) / head;
      at = lo - p.cum[seq] - h * head;
      const int t = p.n[seq], off = p.off[seq];
#pragma unroll 1
      for (;; b += 32) {  // 32 units at a time
        const int n = count_of(a, tiles_of(a, t, off, ((b + lane + 1) << beside) - 1)), sum = below(n, lane);
        const uint32_t in = __ballot_sync(0xffffffffu, at < sum);
        if (in) {
          const int k = __ffs(in) - 1;
          at -= __shfl_sync(0xffffffffu, sum - n, k);
          b += k;
          break;
        }
        at -= __shfl_sync(0xffffffffu, sum, 31);
      }
    }
    if (lane == 0) {
      p.seq = seq;
      p.h = h;
      p.run = (b << beside) + (blockIdx.x & ((1 << beside) - 1));
      p.at = at;
      p.left = min(per, total - lo);
      p.per = per;
      p.beside = beside;
    }
  }
  __syncthreads();
}

// One CTA's part of a unit.
struct Segment {
  int32_t seq, h;
  int32_t token;    // the unit's first in q
  int32_t first;    // and in its sequence
  int32_t tokens;   // of the unit
  bool dual;        // two streams of rows, each over every tile; else one that both hold, every other tile each
  int32_t tile0, tiles;
  bool whole;       // all of the unit's tiles
  int32_t pieces;   // of a unit that begins here and goes on, else 0
  int32_t t, off;   // of the sequence
  __device__ int steps_of(int s) const { return dual ? tiles : (tiles + 1 - s) / 2; }
  __device__ int tile_of(int s, int j) const { return tile0 + (dual ? j : 2 * j + s); }
  // the segment's slot of partial rows
  __device__ int slot() const { return 2 * blockIdx.x + (tile0 == 0); }
};

// Walks the segments of one CTA: one thread, which leaves them for the others.
struct Walk {
  const Plan& p;
  const Args& a;
  int32_t at, left, seq, h, run;
  __device__ Walk(const Plan& plan, const Args& args)
      : p(plan), a(args), at(p.at), left(p.left), seq(p.seq), h(p.h), run(p.run) {}
  // The next one; without tiles behind the last.
  __device__ Segment next() {
    Segment s = {};
#pragma unroll 1
    while (left > 0) {
#pragma unroll 1
      while (p.n[seq] == 0) ++seq;  // what is left lies in a sequence further on
      const int t = p.n[seq], off = p.off[seq];
      // of the last of the runs side by side, and its own: none where that is missing
      const int beside = p.beside, last = run | ((1 << beside) - 1);
      const int count = count_of(a, tiles_of(a, t, off, last));
      const int n = run * 2 * a.run < t ? tiles_of(a, t, off, run) : 0;
      const int take = min(left, count - at), done = p.left - left;
      s.seq = seq;
      s.h = h;
      s.t = t;
      s.off = off;
      s.first = run * 2 * a.run;
      s.token = p.start[seq] + s.first;
      s.tokens = min(t - s.first, 2 * a.run);
      s.dual = s.tokens > a.run;
      s.pieces = 0;
      s.tile0 = 0;
      s.tiles = n;
      if (a.split) {
        s.tile0 = min(at, n);
        s.tiles = min(at + take, n) - s.tile0;
      }
      s.whole = s.tiles == n;
      if (!s.whole && s.tile0 == 0) {
        s.pieces = (uint32_t)(done + n - 1) / p.per + 1;  // up to the CTA that has the unit's last tile
      }
      left -= take;
      at += take;
      if (at == count) {
        at = 0;
        if ((last + 1) * 2 * a.run < t) {
          run += 1 << beside;
        } else {
          run &= (1 << beside) - 1;
          if (++h == a.n_heads) h = 0, ++seq;
        }
      }
      if (s.tiles > 0) return s;
    }
    s.tiles = 0;
    return s;
  }
};

}  // namespace prompt
}  // namespace bpkv
