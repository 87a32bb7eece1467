// Attention of few query rows over long rows of KV: each sequence's G heads
// over its own rows, and units of at most 16 query rows over a prefix (the
// streaming half of bpkv_shared_attend / bpkv_shared_attend8; the plan is in
// shared_plan.cuh, which kernel takes what in shared.cu's launch).
//
// Bound by the bytes of K and V, so every warp is a worker with its own ring of
// asynchronous copies (three stages of 8 KB: 16 tokens of bf16, 32 of codes)
// that runs ahead across the borders of units, and nothing in the CTA waits for
// anything else.  Products are S^T = K Q^T and O^T = V^T P^T, so that the 16
// side of the warp-level matrix instruction holds tokens or channels and the 8
// side the query rows: no part of a product is padding for G = 8, and P^T is
// S^T's own registers through one 8 x 8 transpose.  P^T enters its product as
// bf16 (2^-8), the type of V; its sum takes it unrounded, in float32.  The 5th-generation tensor
// instructions take 128 rows at least, and the units here change every few
// tiles: there a switch of unit cost 2.5 us, more than the tiles between two.
//
// 8-bit rows: a code is exactly a half, so codes become halves in registers;
// channels are taken in the order the bytes come in (the same for K and q).
// K's scales multiply S, V's join the exponent as in the wide kernel: p' = p
// 2^ev is the weight in the product, p = p' 2^-ev the term of the sum.  p' is a
// half here, 2^-11 of rounding: the product is of halves anyway.
//
// Measured on a GB300: 32 sequences of 8 x 4 heads over 8-bit rows of their own,
// up to 16384 tokens (542 MB): 85.5 us with the join, 6.3 TB/s.
#include <cooperative_groups.h>

#include "shared_stream.cuh"

namespace bpkv {
namespace shared {

namespace {

using namespace few;

constexpr int kThreads = kFewWarps * 32;
template <int BITS>
constexpr int kSmem = Shape<BITS>::kRing + (int)sizeof(FewPlan);

// One worker's way through its tiles.
struct Walk {
  static constexpr bool kMasked = false, kStrided = false;
  const FewPlan& p;
  const Args& a;
  int tok;
  int64_t pos, end;
  int item, h;
  int32_t n;
  int64_t t, tiles, row0, unit;
  int side;  // 0: a prefix, 1: own rows
  int index;
  __device__ __forceinline__ Walk(const FewPlan& plan, const Args& args, int worker, int tile) : p(plan), a(args), tok(tile) {
    const int items = p.n_pre + a.n_seq;
    const Share share(p.few[items] * a.n_heads, a.few_workers);
    pos = end = 0;
    if (worker >= share.n) return;
    pos = share.lo(worker);
    end = share.lo(worker + 1);
    int lo = 0, hi = items - 1;  // the last item that begins at or before pos
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (p.few[mid] * a.n_heads <= pos) lo = mid;
      else hi = mid - 1;
    }
    item = lo;
    const int64_t off = pos - p.few[item] * a.n_heads;
    tiles = p.few[item + 1] - p.few[item];
    h = (int)quot(off, tiles);
    t = off - h * tiles;
    set();
  }
  __device__ __forceinline__ void set() {
    side = item < p.n_pre ? 0 : 1;
    index = side ? item - p.n_pre : p.it_p[item];
    const int64_t u = (int64_t)index * a.n_heads + h;
    unit = side ? u : (int64_t)item * a.n_heads + h;
    row0 = u * (side ? a.cap : a.pcap);
    n = side ? p.own[index] : p.tok[index];
  }
  __device__ __forceinline__ bool more() const { return pos < end; }
  // one tile on; true when that is another unit's
  __device__ __forceinline__ bool next() {
    ++pos;
    if (++t < tiles) return false;
    t = 0;
    if (++h == a.n_heads) {
      h = 0;
      if (pos < end) {
        do ++item;
        while (p.few[item + 1] == p.few[item]);
        tiles = p.few[item + 1] - p.few[item];
      }
    }
    if (pos < end) set();
    return true;
  }
  __device__ __forceinline__ int valid() const { return (int)min64(tok, n - t * tok); }
  __device__ __forceinline__ const uint16_t* q_of(int r) const {
    int seq = index, head = r;
    if (side == 0) {
      const int x = ((item - p.item0[index]) << a.unit_log) + r;
      seq = p.order[p.first[index] + x / a.group];
      head = x % a.group;
    }
    return a.q + (((int64_t)seq * a.n_heads + h) * a.group + head) * kD;
  }
};

namespace cg = cooperative_groups;
constexpr int kMaxCluster = 8;
enum { kAlone, kCluster, kFinish };  // what a CTA of k_shared_unit joins besides its own warps

// A warp's way through all rows of one sequence and KV head that a CTA or a
// cluster of them takes whole, the prefix's and then its own: every step-th
// tile, step the warps of all.
struct UnitWalk {
  static constexpr bool kMasked = false, kStrided = false;
  const Args& a;
  int tok, index, h, side, x, step, tiles, pre_tiles, t, n, n_pre, n_own;
  int64_t row0, own_row0, pre_row0;
  __device__ __forceinline__ UnitWalk(const Args& args, int tile, uint32_t unit, int first, int stride)
      : a(args), tok(tile), x(first), step(stride) {
    index = (int)(unit / (uint32_t)a.n_heads);
    h = (int)(unit - (uint32_t)index * a.n_heads);
    own_row0 = unit * a.cap;
    n_pre = 0;
    n_own = (int)tokens_of(a.len[index], a.cap);
    pre_row0 = 0;
    if (a.plen) {
      const int p = a.prefix_of ? a.prefix_of[index] : 0;
      if (p >= 0 && p < a.n_prefix) {
        n_pre = (int)tokens_of(a.plen[p], a.pcap);
        pre_row0 = ((int64_t)p * a.n_heads + h) * a.pcap;
      }
    }
    pre_tiles = (n_pre + tok - 1) / tok;
    tiles = pre_tiles + (n_own + tok - 1) / tok;
    set();
  }
  __device__ __forceinline__ void set() {
    side = x < pre_tiles ? 0 : 1;
    t = side ? x - pre_tiles : x;
    n = side ? n_own : n_pre;
    row0 = side ? own_row0 : pre_row0;
  }
  __device__ __forceinline__ bool more() const { return x < tiles; }
  __device__ __forceinline__ bool next() {
    x += step;
    set();
    return false;
  }
  __device__ __forceinline__ int valid() const { return min(tok, n - t * tok); }
  __device__ __forceinline__ const uint16_t* q_of(int r) const {
    return a.q + (((int64_t)index * a.n_heads + h) * a.group + r) * kD;
  }
};

template <int BITS, int NB>
__global__ void __launch_bounds__(kThreads, 1) k_shared_few(const __grid_constant__ Args a, int32_t wait_first) {
  extern __shared__ __align__(1024) unsigned char smem[];
  using S = Shape<BITS>;
  constexpr float kUnit = BITS == 16 ? kLogScale : 1.f;
  FewPlan& plan = *reinterpret_cast<FewPlan*>(smem + S::kRing);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  // Behind the wide kernel of the same call, which starts this one only after
  // its own wait, what that wait covered is complete: only the end waits.  Both
  // kernels want an SM's whole shared memory, so no two of their CTAs share one;
  // this one's begin where the wide kernel has no CTA, or its CTA has ended.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (wait_first) asm volatile("griddepcontrol.wait;" ::: "memory");
  make_plan(a, plan, S::kTok);
  const int worker = warp * gridDim.x + blockIdx.x;
  const uint32_t ring = smem_u32(smem) + warp * kStages * kStage;
  const unsigned char* exps = smem + kFewWarps * kStages * kStage + warp * kStages * S::kExps;
  Walk ahead(plan, a, worker, S::kTok), cur = ahead;
  const uint64_t policy = evict_first_policy();
  prime<BITS>(ahead, ring, exps, policy);
  // the join's table, while the first copies come
  {
    const int64_t n = (int64_t)a.n_seq * a.n_heads * a.group;
    for (int64_t r = blockIdx.x + (int64_t)gridDim.x * tid; r < n; r += (int64_t)gridDim.x * kThreads)
      a.parts[r] = parts_of(a, plan, r);
  }
  stream<BITS, NB>(
      cur, ahead, ring, exps, policy, [&](const Walk& w) { return w.side ? a.group : pre_rows(a, plan, w.item); },
      [&](const Walk& w, const State<NB>& st, int rows) {  // the segment's partial rows
        const int64_t at = w.side ? own_row(a, w.unit, worker) : few_row(a, w.unit, worker);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = nb * 8 + 2 * c + i;
            const float s = row_sum(st, nb, i);
            if (r < rows) {
              put_row<BITS>(st, nb, i, a.part_o + (at + r) * kD);
              if (g == 0) a.part_ml[at + r] = make_float2(st.m[nb][i] * kUnit, s);
            }
          }
      });
  // the join follows this kernel: it must find the wide kernel complete too
  if (!wait_first) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A lane's four channels of a row, and the row's maximum and sum.
struct Joined {
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
};

constexpr int kJoinDeep = 8;  // parts in flight

// Every step-th of a row's n parts from the first-th on, by one warp, each
// part's (m, l) and o loaded together, under a running maximum.
__device__ __forceinline__ void join_parts(const Args& a, const Parts& q, int n, int first, int step, int lane, Joined& j) {
  for (int k0 = first; k0 < n; k0 += step * kJoinDeep) {
    float2 ml[kJoinDeep];
    float4 o[kJoinDeep];
#pragma unroll
    for (int i = 0; i < kJoinDeep; ++i) {
      const int k = k0 + i * step;
      ml[i] = make_float2(-INFINITY, 0.f);
      if (k < n) {
        const int64_t row =
            k < q.pre_n ? q.pre + (int64_t)k * q.pre_step : q.own + (int64_t)(k - q.pre_n) * a.group;
        ml[i] = a.part_ml[row];
        o[i] = reinterpret_cast<const float4*>(a.part_o + row * kD)[lane];
      }
    }
    float top = j.m;
#pragma unroll
    for (int i = 0; i < kJoinDeep; ++i) {
      if (ml[i].y != 0.f) ml[i].x = fmaxf(ml[i].x, -3e38f);  // a sum that is NaN stays one
      top = fmaxf(top, ml[i].y != 0.f ? ml[i].x : -INFINITY);
    }
    if (top == -INFINITY) continue;
    const float f = ex2(j.m - top);
    j.m = top;
    j.l *= f;
    j.o.x *= f;
    j.o.y *= f;
    j.o.z *= f;
    j.o.w *= f;
#pragma unroll
    for (int i = 0; i < kJoinDeep; ++i) {
      if (ml[i].y == 0.f) continue;  // no tokens: o was not written
      const float w = ex2(ml[i].x - j.m);
      j.l = fmaf(w, ml[i].y, j.l);
      j.o.x = fmaf(w, o[i].x, j.o.x);
      j.o.y = fmaf(w, o[i].y, j.o.y);
      j.o.z = fmaf(w, o[i].z, j.o.z);
      j.o.w = fmaf(w, o[i].w, j.o.w);
    }
  }
}

// Short sequences and prefixes: a CTA takes all rows of one sequence and KV head,
// its warps join in shared memory, and neither plan nor partials nor join are
// needed; a prefix is read again for every sequence, from L2.  One
// sequence of 8 x 4 heads and 500 bf16 tokens takes 4.8 us: the launch, four
// rounds of loads and products of each warp, and the join, all latency.  Few
// units are dealt to a cluster of CTAs each (kCluster), which join through
// distributed shared memory: over 32000 tokens (131 MB) 22 us, 6 TB/s.  Behind
// the wide kernel (kFinish) a CTA streams its sequence's own rows and joins them
// with the prefix's partials, a warp or several for each row.
template <int BITS, int W, int JOIN>
__global__ void __launch_bounds__(W * 32, kFewWarps / W) k_shared_unit(const __grid_constant__ Args a, uint16_t* out) {
  extern __shared__ __align__(1024) unsigned char smem[];
  using S = Shape<BITS>;
  constexpr float kUnit = BITS == 16 ? kLogScale : 1.f;
  __shared__ float2 s_ml[W][8];
  uint32_t ctas = 1, rank = 0;
  if constexpr (JOIN == kCluster) {
    ctas = cg::this_cluster().num_blocks();
    rank = cg::this_cluster().block_rank();
  }
  const uint32_t unit = blockIdx.x / ctas;
  // kCluster: the CTA's o, (m, l) of each row; kFinish: a warp's of a prefix's partials
  __shared__ __align__(16) float2 s_part[JOIN != kAlone ? 8 : 1][kD / 2];
  __shared__ float2 s_part_ml[8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  if constexpr (JOIN == kFinish) {
    // behind the wide kernel of the same call, which has waited for what came before it
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  } else {
    pdl_enter();
  }
  const uint32_t ring = smem_u32(smem) + warp * kStages * kStage;
  const unsigned char* exps = smem + W * kStages * kStage + warp * kStages * S::kExps;
  UnitWalk ahead(a, S::kTok, unit, rank * W + warp, ctas * W), cur = ahead;
  const uint64_t policy = evict_first_policy();
  prime<BITS>(ahead, ring, exps, policy);
  if (tid < W * 8) s_ml[tid / 8][tid % 8] = make_float2(-INFINITY, 0.f);
  __syncthreads();
  float* rows_o = reinterpret_cast<float*>(smem + warp * kStages * kStage);  // the warp's ring, once it is read
  stream<BITS, 1>(
      cur, ahead, ring, exps, policy, [&](const UnitWalk&) { return a.group; },
      [&](const UnitWalk&, const State<1>& st, int rows) {
        cp_wait<0>();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float s = row_sum(st, 0, i);
          if (2 * c + i < rows) {
            put_row<BITS>(st, 0, i, rows_o + (2 * c + i) * kD);
            if (g == 0) s_ml[warp][2 * c + i] = make_float2(st.m[0][i] * kUnit, s);
          }
        }
      });
  const int split = JOIN == kFinish && a.group <= W / 2 ? W / a.group : 1;  // warps of a row's partials
  if constexpr (JOIN == kFinish) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int t = warp; t < a.group * split; t += W) {
      const int r = t % a.group;
      const Parts q = a.parts[(int64_t)unit * a.group + r];
      Joined j;
      join_parts(a, q, q.pre_n, t / a.group, split, lane, j);
      *reinterpret_cast<float4*>(&s_part[t][lane * 2]) = j.o;
      if (lane == 0) s_part_ml[t] = make_float2(j.m, j.l);
    }
  }
  __syncthreads();
  for (int x = tid; x < a.group * (kD / 2); x += W * 32) {
    const int r = x / (kD / 2), d = x % (kD / 2) * 2;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) M = fmaxf(M, s_ml[w][r].y == 0.f ? -INFINITY : fmaxf(s_ml[w][r].x, -3e38f));
    if constexpr (JOIN == kFinish)
      for (int t = r; t < a.group * split; t += a.group) M = fmaxf(M, s_part_ml[t].x);
    float L = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 ml = s_ml[w][r];
      if (ml.y == 0.f) continue;  // no tile: o was not written
      const float f = ex2(fmaxf(ml.x, -3e38f) - M);
      const float2 v = *reinterpret_cast<const float2*>(smem + w * kStages * kStage + (r * kD + d) * sizeof(float));
      L = fmaf(f, ml.y, L);
      o0 = fmaf(f, v.x, o0);
      o1 = fmaf(f, v.y, o1);
    }
    if constexpr (JOIN == kFinish) {
      for (int t = r; t < a.group * split; t += a.group) {
        const float2 ml = s_part_ml[t], v = s_part[t][d / 2];
        if (ml.y == 0.f) continue;
        const float f = ex2(ml.x - M);
        L = fmaf(f, ml.y, L);
        o0 = fmaf(f, v.x, o0);
        o1 = fmaf(f, v.y, o1);
      }
    }
    if constexpr (JOIN == kCluster) {
      s_part[r][d / 2] = make_float2(o0, o1);
      if (d == 0) s_part_ml[r] = make_float2(M, L);
    } else {
      const float s = L == 0.f ? 0.f : 1.f / L;
      *reinterpret_cast<uint32_t*>(out + ((int64_t)unit * a.group + r) * kD + d) = pack<16>(o0 * s, o1 * s);
    }
  }
  if constexpr (JOIN == kCluster) {
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    for (int x = rank * (W * 32) + tid; x < a.group * (kD / 2); x += ctas * W * 32) {
      const int r = x / (kD / 2), d = x % (kD / 2) * 2;
      float2 ml[kMaxCluster], v[kMaxCluster];
      float M = -INFINITY, L = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i) {
        ml[i] = make_float2(-INFINITY, 0.f);
        if (i < ctas) {
          ml[i] = *cl.map_shared_rank(&s_part_ml[r], i);
          v[i] = *cl.map_shared_rank(&s_part[r][d / 2], i);
        }
        M = fmaxf(M, ml[i].x);
      }
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i) {
        if (ml[i].y == 0.f) continue;
        const float f = ex2(ml[i].x - M);
        L = fmaf(f, ml[i].y, L);
        o0 = fmaf(f, v[i].x, o0);
        o1 = fmaf(f, v[i].y, o1);
      }
      const float s = L == 0.f ? 0.f : 1.f / L;
      *reinterpret_cast<uint32_t*>(out + ((int64_t)unit * a.group + r) * kD + d) = pack<16>(o0 * s, o1 * s);
    }
    cl.sync();  // no CTA leaves while another reads its shared memory
  }
}

// ---- join: out = sum_parts 2^(m - M) o / sum_parts 2^(m - M) l
//
// W warps a row; each takes every W-th part, with its own running maximum, so
// that a part's (m, l) and o are loaded together: two round trips in all, the
// table's and the parts'.  Many rows have few parts each and take one warp,
// few rows have many and take eight.  About 5 us behind its kernels, latency.

constexpr int kJoinWarps = 8;

template <int W>
__global__ void __launch_bounds__(kJoinWarps * 32) k_shared_join(const __grid_constant__ Args a, uint16_t* out) {
  pdl_enter();
  __shared__ float4 s_o[kJoinWarps][kD / 4];
  __shared__ float2 s_ml[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part0 = warp % W;
  const int64_t rows = (int64_t)a.n_seq * a.n_heads * a.group;
  const int64_t r = (int64_t)blockIdx.x * (kJoinWarps / W) + warp / W;
  Joined j;
  if (r < rows) {
    const Parts q = a.parts[r];
    join_parts(a, q, q.pre_n + q.own_n, part0, W, lane, j);
  }
  float L = j.l;
  float4 O = j.o;
  if constexpr (W > 1) {
    s_o[warp][lane] = O;
    if (lane == 0) s_ml[warp] = make_float2(j.m, L);
    __syncthreads();
    if (part0 != 0) return;
    float top = j.m;
#pragma unroll
    for (int w = 1; w < W; ++w) top = fmaxf(top, s_ml[warp + w].x);
    const float f = top == -INFINITY ? 0.f : ex2(j.m - top);
    L *= f;
    O = make_float4(O.x * f, O.y * f, O.z * f, O.w * f);
#pragma unroll
    for (int w = 1; w < W; ++w) {
      const float2 ml = s_ml[warp + w];
      const float g = ml.y == 0.f ? 0.f : ex2(ml.x - top);
      const float4 v = s_o[warp + w][lane];
      L = fmaf(g, ml.y, L);
      O.x = fmaf(g, v.x, O.x);
      O.y = fmaf(g, v.y, O.y);
      O.z = fmaf(g, v.z, O.z);
      O.w = fmaf(g, v.w, O.w);
    }
  }
  if (r < rows) {
    const float s = L == 0.f ? 0.f : 1.f / L;
    *reinterpret_cast<uint2*>(out + r * kD + lane * 4) =
        make_uint2(pack<16>(O.x * s, O.y * s), pack<16>(O.z * s, O.w * s));
  }
}

template <int BITS, int NB>
cudaError_t go(const Args& a, int ctas, bool wait_first, cudaStream_t st) {
  static std::atomic<uint64_t> done;
  const cudaError_t e = allow_smem(k_shared_few<BITS, NB>, kSmem<BITS>, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_shared_few<BITS, NB>, dim3(ctas), dim3(kThreads), (size_t)kSmem<BITS>, st, a,
                    (int32_t)wait_first);
}

}  // namespace

int unit_split(int64_t units, int64_t tokens);

// Warps of a CTA that takes a unit whole: 8 while every unit has an SM to
// itself (32 x 8 units of up to 500 tokens would take 8.3 us instead of 6.6),
// else 4, and 2 for many short units (128 x 8 of up to 100: 7.8 us instead of
// 10.9; of up to 1000: 40.4 instead of 37.9).
constexpr int64_t kShortUnit = 512;

template <int BITS, int W, int JOIN = kAlone>
cudaError_t go_unit(const Args& a, cudaStream_t st, uint16_t* out, int ctas = 1) {
  constexpr int kSmem = Shape<BITS>::kRing / kFewWarps * W;
  static std::atomic<uint64_t> done;
  const auto kernel = k_shared_unit<BITS, W, JOIN>;
  const cudaError_t e = allow_smem(kernel, kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)a.n_seq * a.n_heads * ctas));
  cfg.blockDim = dim3(W * 32);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)ctas, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = JOIN == kCluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, out);
}

// whole: tokens of a unit at most, for CTAs that take units whole; else -1, for
// the streaming kernel and the join, or for k_shared_unit behind the wide kernel
// (a.finish).  own_max: tokens of a sequence at most.  wait_first: no wide kernel
// came before.
template <int BITS>
cudaError_t launch_few(const Args& a, int64_t whole, int64_t own_max, bool wait_first, uint16_t* out, cudaStream_t st) {
  if (whole >= 0) {
    const int64_t units = (int64_t)a.n_seq * a.n_heads;
    const int split = unit_split(units, whole);
    if (split > 1) return go_unit<BITS, 8, kCluster>(a, st, out, split);
    if (units <= kSms) return go_unit<BITS, 8>(a, st, out);
    if (units > 4 * kSms && whole <= kShortUnit) return go_unit<BITS, 2>(a, st, out);
    return go_unit<BITS, 4>(a, st, out);
  }
  if (a.finish) {
    Args own = a;
    own.plen = nullptr;
    const int64_t units = (int64_t)a.n_seq * a.n_heads;
    if (units <= kSms) return go_unit<BITS, 8, kFinish>(own, st, out);
    if (units > 4 * kSms && own_max <= kShortUnit) return go_unit<BITS, 2, kFinish>(own, st, out);
    return go_unit<BITS, 4, kFinish>(own, st, out);
  }
  const int ctas = a.few_workers / kFewWarps;
  const cudaError_t e = a.plen ? go<BITS, 2>(a, ctas, wait_first, st) : go<BITS, 1>(a, ctas, wait_first, st);
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)a.n_seq * a.n_heads * a.group;
  const int warps = rows <= 152 * 4 ? 8 : rows <= 152 * 16 ? 2 : 1;
  const auto join = warps == 8 ? k_shared_join<8> : warps == 2 ? k_shared_join<2> : k_shared_join<1>;
  return launch_pdl(join, dim3((unsigned)((rows * warps + kJoinWarps - 1) / kJoinWarps)), dim3(kJoinWarps * 32), 0, st, a,
                    out);
}

template cudaError_t launch_few<16>(const Args&, int64_t, int64_t, bool, uint16_t*, cudaStream_t);
template cudaError_t launch_few<8>(const Args&, int64_t, int64_t, bool, uint16_t*, cudaStream_t);

// CTAs that share a unit (k_shared_unit): as many as leave all units resident at
// once, clusters of 8 finding room for 12 at least.  In us for one / two / four /
// eight CTAs, bf16 rows of 8 x 4 heads: 1 sequence of up to 500 tokens 4.8 / 4.8 /
// 4.6 / 4.8, 1000 6.5 / 5.9 / 5.2 / 4.8, 2000 9.9 / 8.0 / 6.1 / 5.4, 4000 16.8 /
// 12.9 / 8.0 / 6.4; below 600 tokens the cluster's barriers cost what they save.
int unit_split(int64_t units, int64_t tokens) {
  if (tokens < 600) return 1;
  return units <= 12 ? 8 : units <= 32 ? 4 : units <= 72 ? 2 : 1;
}

int few_tile(int bits) { return bits == 16 ? Shape<16>::kTok : Shape<8>::kTok; }

}  // namespace shared
}  // namespace bpkv
