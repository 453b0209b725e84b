// Eviction from the 4-bit paged cache by accumulated attention weight.
//
// Of the n cached tokens of a sequence, each key/value head keeps its last `recent` ones and, of those
// before, the ones with the largest weights (ties: the first), `keep` in all, in their order; all of
// them where n <= keep. They become tokens 0, 1, .. of the pages that another table names, so pages
// that sequences share stay as they are, and nothing is read that this call writes.
//
// Codes and scales of a token stand for themselves, so moving is copying: bound by the bytes of
// the kept tokens (2 * 9/8 dim each, and their weights) and, ahead of that, by the latency of the selection.
//   * k_evict_select: a cluster of CTAs a (sequence, head), each with a piece of the tokens. The
//     smallest weight kept is found in four passes of eight bits over order-preserving integers, each CTA's
//     counts read by the others through distributed shared memory; then every CTA knows how many it
//     keeps and writes their places. No atomics across CTAs: the result does not depend on their order.
//   * k_evict_move: 16 bytes a lane, four tokens in flight.
#include "kv4.cuh"

#include <cooperative_groups.h>

namespace cg = cooperative_groups;

namespace jepa {

namespace {

constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int BINS = 256;

// Weights as integers in the same order: NaN the least, -0 as 0.
__device__ __forceinline__ uint32_t ordered(float x) {
  if (x != x) return 0;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct EvictArgs {
  const int* kv_len;
  const float* mass;
  int keep, recent;
  int* len_out;
  float* mass_out;
  int* places;       // workspace: [batch][heads][keep] kept tokens in order
};

__device__ __forceinline__ int cached_length(const PageView& c, const int* kv_len, int s, int* err_flag) {
  const int n = __ldg(kv_len + s), most = c.max_pages << c.page_log2;
  if (n < 0 || n > most) {
    if (err_flag) atomicOr(err_flag, DEV_ERR_INDEX);
    return n < 0 ? 0 : most;
  }
  return n;
}

// Sum over the CTA of two counts packed in 64 bits, and what lies ahead of this thread.
__device__ __forceinline__ unsigned long long scan(unsigned long long x, unsigned long long* sm,
                                                   unsigned long long& before) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned long long incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();                       // the last scan's sums have been read
  if (lane == 31) sm[warp] = incl;
  __syncthreads();
  unsigned long long ahead = 0, total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) ahead += sm[w];
    total += sm[w];
  }
  before = ahead + incl - x;
  return total;
}

__global__ void __launch_bounds__(THREADS) k_evict_select(Kv4View c, EvictArgs a, int out_reach, int* err_flag) {
  __shared__ int hist[2][BINS];
  __shared__ int counts_all[BINS];       // of the whole cluster
  __shared__ unsigned long long sums[WARPS], piece_counts;
  __shared__ int found[2];               // bin, tokens above it
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), size = (int)cluster.num_blocks();
  const int item = blockIdx.x / size, s = item / c.heads, head = item - s * c.heads;
  const int n = cached_length(c, a.kv_len, s, head == 0 && rank == 0 && threadIdx.x == 0 ? err_flag : nullptr);
  const int kept = min(n, a.keep);
  const float* mass = a.mass + (long long)item * ((long long)c.max_pages << c.page_log2);
  int* const places = a.places + (long long)item * a.keep;
  float* const mass_out = a.mass_out ? a.mass_out + (long long)item * out_reach : nullptr;
  if (head == 0 && rank == 0 && threadIdx.x == 0) a.len_out[s] = kept;
  if (mass_out)                          // nothing behind the kept tokens
    for (int i = kept + rank * THREADS + threadIdx.x; i < out_reach; i += size * THREADS) mass_out[i] = 0.f;
  if (kept == n) {                       // nothing to choose (the same for the whole cluster)
    for (int i = rank * THREADS + threadIdx.x; i < n; i += size * THREADS) {
      places[i] = i;
      if (mass_out) mass_out[i] = mass[i];
    }
    return;
  }
  // n > keep >= recent
  const int old = n - a.recent, want = a.keep - a.recent;
  for (int i = rank * THREADS + threadIdx.x; i < a.recent; i += size * THREADS) {
    places[want + i] = old + i;
    if (mass_out) mass_out[want + i] = mass[old + i];
  }
  if (want == 0) return;
  const int each = (old + size - 1) / size;
  const int begin = min(old, rank * each), end = min(old, begin + each);
  // ---- the smallest weight kept: digit by digit from the top ----
  uint32_t prefix = 0;                   // its digits so far
  int need = want;                       // tokens still to be taken from those with this prefix
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    int* const mine = hist[pass & 1];    // the other one may still be read
    for (int b = threadIdx.x; b < BINS; b += THREADS) mine[b] = 0;
    __syncthreads();
    for (int i = begin + threadIdx.x; i < end; i += THREADS) {
      const uint32_t u = ordered(__ldg(mass + i));
      if (pass == 0 || (u >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(mine + ((u >> shift) & 255), 1);
    }
    cluster.sync();
    if (threadIdx.x < BINS) {
      int all = 0;
      for (int r = 0; r < size; ++r) all += cluster.map_shared_rank(mine, r)[threadIdx.x];
      counts_all[threadIdx.x] = all;
    }
    __syncthreads();
    if (threadIdx.x < 32) {              // eight bins a lane, from the top
      const int lane = threadIdx.x, top = BINS - 1 - 8 * lane;
      int own = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) own += counts_all[top - k];
      int incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      int above = incl - own;
      if (above < need && need <= incl) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int in = counts_all[top - k];
          if (above < need && need <= above + in) {
            found[0] = top - k;
            found[1] = above;
          }
          above += in;
        }
      }
    }
    __syncthreads();
    prefix |= (uint32_t)found[0] << shift;
    need -= found[1];
  }
  // ---- where the kept ones go: all above the prefix, and the first `need` equal to it ----
  unsigned long long counts = 0, before;
  for (int i = begin + threadIdx.x; i < end; i += THREADS) {
    const uint32_t u = ordered(__ldg(mass + i));
    counts += u > prefix ? 1ull << 32 : u == prefix ? 1ull : 0ull;
  }
  counts = scan(counts, sums, before);
  if (threadIdx.x == 0) piece_counts = counts;
  cluster.sync();
  unsigned int above = 0, equal = 0;     // of the pieces ahead
  for (int r = 0; r < rank; ++r) {
    const unsigned long long x = *cluster.map_shared_rank(&piece_counts, r);
    above += (unsigned int)(x >> 32);
    equal += (unsigned int)x;
  }
  cluster.sync();                        // every CTA's counts have been read before it ends
  for (int i0 = begin; i0 < end; i0 += THREADS) {
    const int i = i0 + threadIdx.x;
    const float x = i < end ? __ldg(mass + i) : 0.f;
    const uint32_t u = ordered(x);
    const bool gt = i < end && u > prefix, eq = i < end && u == prefix;
    const unsigned long long all = scan(gt ? 1ull << 32 : eq ? 1ull : 0ull, sums, before);
    const unsigned int g = above + (unsigned int)(before >> 32), e = equal + (unsigned int)before;
    if (gt || (eq && e < (unsigned int)need)) {
      const unsigned int to = g + min(e, (unsigned int)need);
      places[to] = i;
      if (mass_out) mass_out[to] = x;
    }
    above += (unsigned int)(all >> 32);
    equal += (unsigned int)all;
  }
}

// A warp takes RPW kept tokens of a head at a time, AHEAD times.
template <int D>
__global__ void __launch_bounds__(256) k_evict_move(Kv4View c, Kv4View to, const int* kv_len, int keep,
                                                    const int* places, int* err_flag) {
  constexpr int LPT = D / 16, RPW = 32 / LPT, AHEAD = 4;   // lanes a token, half of them K's, half V's
  constexpr int KB = D / 2, SB = D / 16;
  const int s = blockIdx.z, head = blockIdx.y, lane = threadIdx.x & 31;
  const int n = min(cached_length(c, kv_len, s, nullptr), keep);
  const int first = (blockIdx.x * (256 / 32) + (threadIdx.x >> 5)) * (RPW * AHEAD) + lane / LPT;
  if (first - lane / LPT >= n) return;
  const int part = lane % LPT;
  const bool is_v = part >= LPT / 2;
  const int chunk = part % (LPT / 2);
  const int* from = places + ((long long)s * c.heads + head) * keep;
  const uint8_t *codes = is_v ? c.v : c.k, *scales = is_v ? c.v_scale : c.k_scale;
  uint8_t *codes_to = is_v ? to.v : to.k, *scales_to = is_v ? to.v_scale : to.k_scale;
  uint4 x[AHEAD];
  uint2 sc[AHEAD];
  long long row_to[AHEAD];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) {
    const int i = first + k * RPW;
    row_to[k] = -1;
    if (i >= n) continue;
    const int j = __ldg(from + i);
    const int pg = kv8_page_at(c.table, c.max_pages, c.num_pages, c.page_log2, s, j);
    const int pt = kv8_page_at(to.table, to.max_pages, to.num_pages, to.page_log2, s, i);
    if (pg < 0 || pt < 0) {
      if (part == 0) atomicOr(err_flag, DEV_ERR_INDEX);
      continue;
    }
    const long long row = (((long long)pg * c.heads + head) << c.page_log2) + (j & (c.page - 1));
    row_to[k] = (((long long)pt * c.heads + head) << to.page_log2) + (i & (to.page - 1));
    x[k] = *reinterpret_cast<const uint4*>(codes + row * KB + 16 * chunk);
    if (chunk == 0) {
      if (D == 128)
        sc[k] = *reinterpret_cast<const uint2*>(scales + row * SB);
      else
        sc[k].x = *reinterpret_cast<const uint32_t*>(scales + row * SB);
    }
  }
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) {
    if (row_to[k] < 0) continue;
    *reinterpret_cast<uint4*>(codes_to + row_to[k] * KB + 16 * chunk) = x[k];
    if (chunk == 0) {
      if (D == 128)
        *reinterpret_cast<uint2*>(scales_to + row_to[k] * SB) = sc[k];
      else
        *reinterpret_cast<uint32_t*>(scales_to + row_to[k] * SB) = sc[k].x;
    }
  }
}

}  // namespace

size_t kv4_evict_workspace(const PageView& c, int keep) {
  return (size_t)c.batch * c.heads * keep * sizeof(int);
}

cudaError_t kv4_evict(const Kv4View& c, const int* kv_len, const float* mass, int keep, int recent,
                      const Kv4View& to, int* len_out, float* mass_out, void* workspace,
                      int* err_flag, int num_sms, cudaStream_t s) {
  const long long items = (long long)c.batch * c.heads;
  EvictArgs a{kv_len, mass, keep, recent, len_out, mass_out, (int*)workspace};
  // CTAs a (sequence, head): pieces of a few thousand tokens, up to the portable cluster size
  const long long reach = (long long)c.max_pages << c.page_log2;
  int size = 1;
  while (size < 8 && reach > 2048LL * size && items * size < 2LL * num_sms) size *= 2;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = size;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * size));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, k_evict_select, c, a, to.max_pages << to.page_log2, err_flag);
  if (e != cudaSuccess) return e;
  const int most = (int)(reach < keep ? reach : keep);
  const int per = 8 * (32 / (c.dim / 16)) * 4;             // tokens a CTA moves
  const dim3 grid((most + per - 1) / per, c.heads, c.batch);
  if (c.dim == 64)
    k_evict_move<64><<<grid, 256, 0, s>>>(c, to, kv_len, keep, a.places, err_flag);
  else
    k_evict_move<128><<<grid, 256, 0, s>>>(c, to, kv_len, keep, a.places, err_flag);
  return cudaGetLastError();
}

}  // namespace jepa
