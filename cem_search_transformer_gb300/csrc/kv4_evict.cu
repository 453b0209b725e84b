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
//   * k_evict_move: 16 bytes a lane, two tokens in flight.
// Measured: 8 heads of 128 of six sequences of 34648 to 70001 tokens back to 8192: selection 27 us (issue 57%: the six
// looks at each weight), moving 31 (130 MB read for 57: a token's 8 bytes of scales cost a 32-byte sector each), the
// read-back that follows 43. Slower: moving by the clusters that chose (16% of the whole), digits of eleven bits (the
// clusters' counts then are eight times the traffic between SMs: 43%).
#include "kv4.cuh"

#include <cooperative_groups.h>

namespace cg = cooperative_groups;

namespace jepa {

namespace {

constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int BINS = 256;
constexpr int MAX_CLUSTER = 8;           // the portable size

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
  const int n = kv_len[s], most = c.max_pages << c.page_log2;
  if (n < 0 || n > most) {
    if (err_flag) atomicOr(err_flag, DEV_ERR_INDEX);
    return n < 0 ? 0 : most;
  }
  return n;
}

__device__ __forceinline__ float unordered(uint32_t u) {
  if (u == 0) return __int_as_float(0x7fc00000);
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

constexpr int HELD = 11008;              // weights of a CTA's piece that stay in shared memory (43 KB)

__global__ void __launch_bounds__(THREADS) k_evict_select(Kv4View c, EvictArgs a, int out_reach, int* err_flag) {
  __shared__ uint32_t held[HELD];
  __shared__ int hist[2][BINS];
  __shared__ int counts_all[BINS];       // of the whole cluster
  __shared__ uint2 warp_counts[WARPS], piece_counts;   // above the border, equal to it
  __shared__ int found[2];               // bin, tokens above it
  asm volatile("griddepcontrol.launch_dependents;");   // k_evict_move may be set up meanwhile
  asm volatile("griddepcontrol.wait;" ::: "memory");   // what the kernel before writes is there
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), size = (int)cluster.num_blocks();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
  // a warp's piece of the tokens: its lanes take every 32nd, as integers in the order of the weights
  const int pieces = size * WARPS, each = ((old + pieces - 1) / pieces + 31) & ~31;
  const int begin = min((long long)old, (long long)(rank * WARPS + warp) * each), end = min(old, begin + each);
  const int first = warp * each;         // of its piece among the CTA's
  // f(i, weight) for the lane's tokens: those that are held, then those that are not
  static_assert(HELD % 32 == 0, "a warp's turns are held or not as a whole");
  const int held_end = min(end, begin + max(0, HELD - first));
  const uint32_t* const mine_held = held + (first - begin);
  auto each_token = [&](auto f) {
    int i = begin + lane;
#pragma unroll 4
    for (; i < held_end; i += 32) f(i, mine_held[i]);
    for (; i < end; i += 32) f(i, ordered(load_late(mass + i)));
  };
  for (int b = threadIdx.x; b < BINS; b += THREADS) hist[0][b] = 0;
  __syncthreads();
  // ---- the smallest weight kept: digit by digit from the top ----
  constexpr int AHEAD = 8;
  for (int i0 = begin; i0 < end; i0 += 32 * AHEAD) {
    float x[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int i = i0 + 32 * k + lane;
      x[k] = i < end ? load_late(mass + i) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int i = i0 + 32 * k + lane, at = first + i - begin;
      const uint32_t u = ordered(x[k]);
      if (i < end && at < HELD) held[at] = u;
      // weights share few exponents: one addition for the lanes that have the same
      const uint32_t bin = i < end ? u >> 24 : BINS;
      const uint32_t same = __match_any_sync(0xffffffffu, bin);
      if (bin < BINS && lane == __ffs((int)same) - 1) atomicAdd(&hist[0][bin], __popc(same));
    }
  }
  uint32_t prefix = 0;                   // the border's digits so far
  int need = want;                       // tokens still to be taken from those with this prefix
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    int* const mine = hist[pass & 1];    // the other one may still be read
    if (pass > 0) {
      for (int b = threadIdx.x; b < BINS; b += THREADS) mine[b] = 0;
      __syncthreads();
      each_token([&](int, uint32_t u) {
        if ((u >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(mine + ((u >> shift) & 255), 1);
      });
    }
    cluster.sync();
    if (threadIdx.x < BINS) {
      int all = 0;
#pragma unroll
      for (int r = 0; r < MAX_CLUSTER; ++r)          // side by side: a microsecond each
        if (r < size) all += cluster.map_shared_rank(mine, r)[threadIdx.x];
      counts_all[threadIdx.x] = all;
    }
    __syncthreads();
    if (warp == 0) {                     // eight bins a lane, from the top
      const int top = BINS - 1 - 8 * lane;
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
  // ---- where the kept ones go: all above the border, and the first `need` equal to it ----
  uint32_t above = 0, equal = 0;
  each_token([&](int, uint32_t u) {
    above += u > prefix;
    equal += u == prefix;
  });
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) warp_counts[warp] = make_uint2(above, equal);
  __syncthreads();
  above = equal = 0;                     // of the warps ahead
  uint2 total = make_uint2(0, 0);
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const uint2 x = warp_counts[w];
    if (w < warp) {
      above += x.x;
      equal += x.y;
    }
    total.x += x.x;
    total.y += x.y;
  }
  if (threadIdx.x == 0) piece_counts = total;
  cluster.sync();
#pragma unroll
  for (int r = 0; r < MAX_CLUSTER; ++r)
    if (r < rank) {
      const uint2 x = *cluster.map_shared_rank(&piece_counts, r);
      above += x.x;
      equal += x.y;
    }
  cluster.sync();                        // every CTA's counts have been read before it ends
  const uint32_t below = (1u << lane) - 1, last = (uint32_t)need;
  auto place = [&](int i, uint32_t u) {
    const bool gt = i < end && u > prefix, eq = i < end && u == prefix;
    const uint32_t gts = __ballot_sync(0xffffffffu, gt), eqs = __ballot_sync(0xffffffffu, eq);
    const uint32_t e = equal + __popc(eqs & below);
    if (gt || (eq && e < last)) {
      const uint32_t to = above + __popc(gts & below) + min(e, last);
      places[to] = i;
      if (mass_out) mass_out[to] = unordered(u);
    }
    above += __popc(gts);
    equal += __popc(eqs);
  };
  int i0 = begin;
#pragma unroll 2
  for (; i0 < held_end; i0 += 32) place(i0 + lane, i0 + lane < end ? mine_held[i0 + lane] : 0u);
  for (; i0 < end; i0 += 32) place(i0 + lane, i0 + lane < end ? ordered(load_late(mass + i0 + lane)) : 0u);
}

// A warp takes RPW kept tokens of a head at a time, AHEAD times.
template <int D>
__global__ void __launch_bounds__(256) k_evict_move(Kv4View c, Kv4View to, const int* kv_len, int keep,
                                                    const int* places, int* err_flag) {
  constexpr int LPT = D / 16, RPW = 32 / LPT, AHEAD = 2;   // lanes a token, half of them K's, half V's
  constexpr int KB = D / 2, SB = D / 16;
  asm volatile("griddepcontrol.wait;" ::: "memory");       // the places are there
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
    const int j = from[i];
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
  // CTAs a (sequence, head): pieces of two thousand tokens or more, up to the portable cluster size, while the machine has
  // room. Six sequences of up to 70001 tokens and 8 heads, with the read-back: one CTA 249 us, two 170, four 129,
  // eight 102; eight of up to 2001 and 16 heads (128 items): one 19, two 21, four 28, eight 43.
  const long long reach = (long long)c.max_pages << c.page_log2;
  int size = 1;
  while (size < MAX_CLUSTER && reach > 2048LL * size && items * size < 2LL * num_sms) size *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * size));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, k_evict_select, c, a, to.max_pages << to.page_log2, err_flag);
  if (e != cudaSuccess) return e;
  const int most = (int)(reach < keep ? reach : keep);
  const int per = 8 * (32 / (c.dim / 16)) * 2;             // tokens a CTA moves
  cfg.attrs = attr + 1;                  // no clusters
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((most + per - 1) / per, c.heads, c.batch);
  cfg.blockDim = dim3(256);
  return cudaLaunchKernelEx(&cfg, c.dim == 64 ? k_evict_move<64> : k_evict_move<128>, c, to, kv_len, keep,
                            (const int*)a.places, err_flag);
}

}  // namespace jepa
