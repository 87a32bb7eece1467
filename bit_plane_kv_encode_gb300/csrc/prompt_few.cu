// Few new tokens, in a tree or not: the streaming half of bpkv_tree_attend,
// bpkv_tree_attend8 and bpkv_prompt_attend (which call takes which half in prompt.cu).
//
// A cluster of CTAs takes up to 16 query rows of a sequence and KV head over all of
// its rows of the cache; every warp streams its own tiles (shared_stream.cuh), the
// warps join in shared memory, the CTAs through distributed shared memory.  One
// launch, no plan, no partials in memory: the tensor-core kernel's start, its wait for
// the first tiles and its join cost more than such a call's work.  A tree's rows are
// taken 16 at a time, each time over all keys, from L2 again.
//
// Of prompts behind long rows of a cache the host does not know whether each sequence has
// its few rows or one has them all.  There this half looks, and leaves the call to the
// tensor cores, which are launched behind it in any case, where rows would be read again.
//
// Measured on a GB300: one new token of a sequence of 4000 bf16 rows, 8 x 4 heads, 7.5 us,
// latency; of 64000 (262 MB) 43 us, 6.1 TB/s; 64 sequences of 4000 in 8 bits (528 MB) 91 us,
// 5.8 TB/s.  Weights enter their product as bf16 (2^-8), for 8-bit rows as halves (2^-11).
#include <cooperative_groups.h>

#include "prompt_plan.cuh"
#include "shared_stream.cuh"

namespace bpkv {
namespace prompt {

namespace {

namespace cg = cooperative_groups;
using namespace shared::few;
using shared::ex2;
using shared::kLogScale;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;

// A warp's way through the rows of one unit: every step-th tile, step the warps of all its CTAs.
// EITHER: it also finds out whether the call is for the tensor cores.
template <bool EITHER>
struct FewWalk {
  static constexpr bool kMasked = true, kStrided = true;
  static constexpr int side = 0;
  const FewArgs& a;
  int tok, index, h, row0_q, step, tiles, t, n, count, start;
  int64_t row0, base, first[2];
  bool theirs;
  __device__ __forceinline__ FewWalk(const FewArgs& args, int tile, uint32_t unit, int begin, int stride)
      : a(args), tok(tile), t(begin), step(stride) {
    const uint32_t head = unit / (uint32_t)a.groups;
    uint32_t group = unit - head * a.groups;
    if (a.q_start) {  // heads, then the groups of all sequences
      h = (int)head;
      find(group);
    } else {
      index = (int)(head / (uint32_t)a.n_heads);
      h = (int)(head - (uint32_t)index * a.n_heads);
      count = a.t;
      start = index * a.t;
    }
    row0_q = (int)group * a.per;
    n = a.len ? (int)shared::tokens_of(a.len[index], a.cap) : count;
    base = n - count;
    tiles = rows() > 0 ? (n + tok - 1) / tok : 0;
    row0 = a.where == kCache ? ((int64_t)index * a.n_heads + h) * a.cap
           : a.where == kSeq ? (int64_t)start * a.n_heads + (int64_t)h * count
                             : start;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) first[kv] = row0 * a.step[kv] + (a.where == kToken ? h * (kD * 2) : 0);
  }
  // The sequence that a group of rows belongs to, and its place there; none: no tokens.
  // Starts as prompt_plan.cuh takes them: within the tokens, none before the last.
  // It is for the tensor cores where the groups would read half as many rows again as there are:
  // the host's rule (few_ctas' `again`), but by the tokens and rows that each sequence has.
  __device__ __forceinline__ void find(uint32_t& group) {
    const int lane = threadIdx.x & 31;
    int top = 0, before = 0;
    [[maybe_unused]] int64_t more = 0;
    [[maybe_unused]] uint32_t found = 0xffffffffu;
    index = count = start = 0;
#pragma unroll 1
    for (int b = 0; b < a.n_seq; b += 32) {
      const int i = min(b + lane, a.n_seq - 1);
      int lo = b + lane < a.n_seq ? (int)max64(0, min64(a.q_start[i], a.tokens)) : 0;
      const int next = (int)max64(0, min64(a.q_start[i + 1], a.tokens));
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, lo, o);
        if (lane >= o) lo = max(lo, u);
      }
      lo = max(lo, top);
      const int hi = max(lo, next), mine = b + lane < a.n_seq ? hi - lo : 0;
      const int groups = (mine * a.group + a.per - 1) / a.per;
      if constexpr (EITHER)
        if (mine > 0) more += shared::tokens_of(a.len[i], a.cap) * (2 * groups - 3);
      int sum = groups;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += u;
      }
      const uint32_t in = __ballot_sync(0xffffffffu, (int)group < before + sum);
      if (in && (!EITHER || found == 0xffffffffu)) {
        const int k = __ffs(in) - 1;
        index = b + k;
        count = __shfl_sync(0xffffffffu, mine, k);
        start = __shfl_sync(0xffffffffu, lo, k);
        found = group - before - __shfl_sync(0xffffffffu, sum - groups, k);
        if constexpr (!EITHER) {
          group = found;
          return;
        }
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
      top = __shfl_sync(0xffffffffu, hi, 31);
    }
    group = 0;
    if constexpr (EITHER) {
      if (found != 0xffffffffu) group = found;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) more += __shfl_xor_sync(0xffffffffu, more, o);
      theirs = more > 0;
    }
  }
  __device__ __forceinline__ bool more() const { return t < tiles; }
  __device__ __forceinline__ bool next() {
    t += step;
    return false;
  }
  __device__ __forceinline__ int valid() const { return min(tok, n - t * tok); }
  __device__ __forceinline__ int rows() const { return min(a.per, count * a.group - row0_q); }
  // token and head of the group of row r
  __device__ __forceinline__ void place(int r, int& node, int& head) const {
    node = (row0_q + r) / a.group;
    head = row0_q + r - node * a.group;
  }
  __device__ __forceinline__ const uint16_t* q_of(int r) const {
    int node, head;
    place(r, node, head);
    return a.q + (int64_t)(start + node) * a.ld_q + (h * a.group + head) * kD;
  }
  __device__ __forceinline__ uint16_t* out_of(int r) const {
    int node, head;
    place(r, node, head);
    return a.out + (((int64_t)(start + node) * a.n_heads + h) * a.group + head) * kD;
  }
  __device__ __forceinline__ uint64_t mask_of(int r) const {
    const int node = (row0_q + r) / a.group;
    if (!a.tree) return (2ull << node) - 1;
    return a.tree[(int64_t)index * a.t + node] & (a.t >= 64 ? ~0ull : (1ull << a.t) - 1);
  }
};

template <int BITS, int NB, bool CLUSTER, bool EITHER>
__global__ void __launch_bounds__(kThreads, 1) k_few_unit(const __grid_constant__ FewArgs a) {
  extern __shared__ __align__(1024) unsigned char smem[];
  using S = Shape<BITS>;
  constexpr float kUnit = BITS == 16 ? kLogScale : 1.f;
  constexpr int kR = 8 * NB;
  __shared__ float2 s_ml[kWarps][kR];
  // the CTA's o, and (m, l) of each row, for the other CTAs
  __shared__ __align__(16) float2 s_part[CLUSTER ? kR : 1][kD / 2];
  __shared__ float2 s_part_ml[kR];
  uint32_t ctas = 1, rank = 0;
  if constexpr (CLUSTER) {
    ctas = cg::this_cluster().num_blocks();
    rank = cg::this_cluster().block_rank();
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  pdl_enter();
  const uint32_t ring = smem_u32(smem) + warp * kStages * kStage;
  const unsigned char* exps = smem + kWarps * kStages * kStage + warp * kStages * S::kExps;
  using Walk = FewWalk<EITHER>;
  Walk ahead(a, S::kTok, blockIdx.x / ctas, rank * kWarps + warp, ctas * kWarps), cur = ahead;
  const uint64_t policy = shared::evict_first_policy();
  if constexpr (EITHER) {  // this half takes the call, or the one behind it, which finds no tokens else
    if (blockIdx.x == 0)
      for (int i = tid; i <= a.n_seq; i += kThreads) a.starts[i] = cur.theirs ? a.q_start[i] : 0;
    if (cur.theirs) return;  // all CTAs
  }
  prime<BITS>(ahead, ring, exps, policy);
  const int rows = cur.rows();
  if (rows <= 0) return;  // of no sequence: the whole cluster
  const Walk unit = cur;
  for (int i = tid; i < kWarps * kR; i += kThreads) s_ml[i / kR][i % kR] = make_float2(-INFINITY, 0.f);
  __syncthreads();
  float* rows_o = reinterpret_cast<float*>(smem + warp * kStages * kStage);  // the warp's ring, once it is read
  stream<BITS, NB>(
      cur, ahead, ring, exps, policy, [&](const Walk&) { return rows; },
      [&](const Walk&, const State<NB>& st, int) {
        cp_wait<0>();
        __syncwarp();
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = nb * 8 + 2 * c + i;
            const float s = row_sum(st, nb, i);
            if (r < rows) {
              put_row<BITS>(st, nb, i, rows_o + r * kD);
              if (g == 0) s_ml[warp][r] = make_float2(st.m[nb][i] * kUnit, s);
            }
          }
      });
  __syncthreads();
  for (int x = tid; x < rows * (kD / 2); x += kThreads) {
    const int r = x / (kD / 2), d = x % (kD / 2) * 2;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_ml[w][r].y == 0.f ? -INFINITY : fmaxf(s_ml[w][r].x, -3e38f));
    float L = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = s_ml[w][r];
      if (ml.y == 0.f) continue;  // no tile: o was not written
      const float f = ex2(fmaxf(ml.x, -3e38f) - M);
      const float2 v = *reinterpret_cast<const float2*>(smem + w * kStages * kStage + (r * kD + d) * sizeof(float));
      L = fmaf(f, ml.y, L);
      o0 = fmaf(f, v.x, o0);
      o1 = fmaf(f, v.y, o1);
    }
    if constexpr (CLUSTER) {
      s_part[r][d / 2] = make_float2(o0, o1);
      if (d == 0) s_part_ml[r] = make_float2(M, L);
    } else {
      const float s = L == 0.f ? 0.f : 1.f / L;
      *reinterpret_cast<uint32_t*>(unit.out_of(r) + d) = pack<16>(o0 * s, o1 * s);
    }
  }
  if constexpr (CLUSTER) {
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    for (int x = rank * kThreads + tid; x < rows * (kD / 2); x += ctas * kThreads) {
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
      *reinterpret_cast<uint32_t*>(unit.out_of(r) + d) = pack<16>(o0 * s, o1 * s);
    }
    cl.sync();  // no CTA leaves while another reads its shared memory
  }
}

template <int BITS, int NB, bool CLUSTER, bool EITHER = false>
cudaError_t go(const FewArgs& a, int ctas, cudaStream_t st) {
  constexpr int kSmem = Shape<BITS>::kRing;
  static std::atomic<uint64_t> done;
  const auto kernel = k_few_unit<BITS, NB, CLUSTER, EITHER>;
  const cudaError_t e = shared::allow_smem(kernel, kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.q_start ? 1 : (int64_t)a.n_seq) * a.n_heads * a.groups * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)ctas, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = CLUSTER ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

// ctas: of a unit's cluster
template <int BITS>
cudaError_t launch_few_tokens(const FewArgs& a, int ctas, cudaStream_t st) {
  if (a.starts) return ctas > 1 ? go<BITS, 2, true, true>(a, ctas, st) : go<BITS, 2, false, true>(a, 1, st);
  if (a.per == 8) return ctas > 1 ? go<BITS, 1, true>(a, ctas, st) : go<BITS, 1, false>(a, 1, st);
  return ctas > 1 ? go<BITS, 2, true>(a, ctas, st) : go<BITS, 2, false>(a, 1, st);
}
template cudaError_t launch_few_tokens<16>(const FewArgs&, int, cudaStream_t);
template cudaError_t launch_few_tokens<8>(const FewArgs&, int, cudaStream_t);

}  // namespace prompt
}  // namespace bpkv
