// Trees of few drafted tokens, or single new ones: the streaming half of
// bpkv_tree_attend and bpkv_tree_attend8 (which call takes which half in
// prompt.cu's launch).
//
// A cluster of CTAs takes up to 16 query rows of a sequence and KV head over all of
// its rows of the cache; every warp streams its own tiles (shared_stream.cuh), the
// warps join in shared memory, the CTAs through distributed shared memory.  One
// launch, no plan, no partials in memory: the tensor-core kernel's start, its wait for
// the first tiles and its join cost more than such a call's work.  A tree's rows are
// taken 16 at a time, each time over all keys, from L2 again.
//
// Measured on a GB300: one new token of a sequence of 4000 bf16 rows, 8 x 4 heads, 6.8 us,
// latency; of 64000 (262 MB) 42 us, 6.3 TB/s; 64 sequences of 4000 in 8 bits (528 MB) 88 us,
// 6.0 TB/s.  Weights enter their product as bf16 (2^-8), for 8-bit rows as halves (2^-11).
#include <cooperative_groups.h>

#include "prompt_plan.cuh"
#include "shared_stream.cuh"

namespace bpkv {
namespace prompt {

namespace {

namespace cg = cooperative_groups;
using namespace shared::few;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A warp's way through the rows of one unit: every step-th tile, step the warps of all its CTAs.
struct TreeWalk {
  static constexpr bool kMasked = true;
  static constexpr int side = 0;
  const FewArgs& a;
  int tok, index, h, row0_q, x, step, tiles, t, n;
  int64_t row0, base;
  __device__ __forceinline__ TreeWalk(const FewArgs& args, int tile, uint32_t unit, int first, int stride)
      : a(args), tok(tile), t(first), step(stride) {
    const uint32_t head = unit / (uint32_t)a.groups;
    row0_q = (int)(unit - head * a.groups) * a.per;
    index = (int)(head / (uint32_t)a.n_heads);
    h = (int)(head - (uint32_t)index * a.n_heads);
    row0 = head * a.cap;
    n = (int)shared::tokens_of(a.len[index], a.cap);
    base = n - a.t;
    tiles = (n + tok - 1) / tok;
  }
  __device__ __forceinline__ bool more() const { return t < tiles; }
  __device__ __forceinline__ bool next() {
    t += step;
    return false;
  }
  __device__ __forceinline__ int valid() const { return min(tok, n - t * tok); }
  __device__ __forceinline__ int rows() const { return min(a.per, a.t * a.group - row0_q); }
  // element of q and out where row r begins
  __device__ __forceinline__ int64_t at(int r) const {
    const int node = (row0_q + r) / a.group, head = row0_q + r - node * a.group;
    return ((((int64_t)index * a.t + node) * a.n_heads + h) * a.group + head) * kD;
  }
  __device__ __forceinline__ const uint16_t* q_of(int r) const { return a.q + at(r); }
  __device__ __forceinline__ uint64_t mask_of(int r) const {
    const int node = (row0_q + r) / a.group;
    if (!a.tree) return (2ull << node) - 1;
    return a.tree[(int64_t)index * a.t + node] & (a.t >= 64 ? ~0ull : (1ull << a.t) - 1);
  }
};

template <int BITS, int NB, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 1) k_tree_unit(const __grid_constant__ FewArgs a) {
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
  TreeWalk ahead(a, S::kTok, blockIdx.x / ctas, rank * kWarps + warp, ctas * kWarps), cur = ahead;
  const uint64_t policy = shared::evict_first_policy();
  prime<BITS>(ahead, ring, exps, policy);
  const int rows = cur.rows();
  const TreeWalk unit = cur;
  for (int i = tid; i < kWarps * kR; i += kThreads) s_ml[i / kR][i % kR] = make_float2(-INFINITY, 0.f);
  __syncthreads();
  float* rows_o = reinterpret_cast<float*>(smem + warp * kStages * kStage);  // the warp's ring, once it is read
  stream<BITS, NB>(
      cur, ahead, ring, exps, policy, [&](const TreeWalk&) { return rows; },
      [&](const TreeWalk&, const State<NB>& st, int) {
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
      *reinterpret_cast<uint32_t*>(a.out + unit.at(r) + d) = pack<16>(o0 * s, o1 * s);
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
      *reinterpret_cast<uint32_t*>(a.out + unit.at(r) + d) = pack<16>(o0 * s, o1 * s);
    }
    cl.sync();  // no CTA leaves while another reads its shared memory
  }
}

template <int BITS, int NB, bool CLUSTER>
cudaError_t go(const FewArgs& a, int ctas, cudaStream_t st) {
  constexpr int kSmem = Shape<BITS>::kRing;
  static std::atomic<uint64_t> done;
  const auto kernel = k_tree_unit<BITS, NB, CLUSTER>;
  const cudaError_t e = shared::allow_smem(kernel, kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)a.n_seq * a.n_heads * a.groups * ctas));
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
cudaError_t launch_tree_few(const FewArgs& a, int ctas, cudaStream_t st) {
  if (a.per == 8) return ctas > 1 ? go<BITS, 1, true>(a, ctas, st) : go<BITS, 1, false>(a, 1, st);
  return ctas > 1 ? go<BITS, 2, true>(a, ctas, st) : go<BITS, 2, false>(a, 1, st);
}
template cudaError_t launch_tree_few<16>(const FewArgs&, int, cudaStream_t);
template cudaError_t launch_tree_few<8>(const FewArgs&, int, cudaStream_t);

}  // namespace prompt
}  // namespace bpkv
