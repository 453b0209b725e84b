// Attention of whole packed prompts on the sm_103a tensor cores (tcgen05 + TMEM + TMA), grouped
// heads, head dim 64 or 128.
//
//   o[i] = sum_{j < lim(i)} softmax_j(scale q[i] . k[j]) v[j],   lim(i) = min(nk, (p / F + 1) F),
//   p = i + nk - nq: the query's position among the keys; F = 1 is causal, F = T block-causal over
//   frames of T tokens (the predictor's mask), F >= nk without a mask.
//
// A CTA takes 256 query rows of one sequence and key/value head, two tiles of 128. A row is a
// (token, head of the group) pair, token-major, so that a group's heads share the tile of keys
// and short prompts still fill the rows; groups that do not divide 128 leave a few rows unused.
// Warps:
//   0-3, 4-7  softmax of tile 0 and 1, a row a thread: read S from TMEM, running maximum and sum,
//             P (bf16) over S, rescale O in TMEM when the maximum moved by more than 2^8, and at
//             the end normalise and store;
//   8         MMA issuer: S_w = Q_w K^T, O_w += P_w V (P from TMEM, V MN-major from its TMA tile).
//             The two tiles alternate, so that one tile's products run under the other's softmax;
//   9         TMA producer: the Q tiles, then K_0, V_0, K_1, V_1, ... through one ring;
//   10, 11    nothing (registers are handed over by warpgroups of four).
// A barrier on S_w of key tile j also says that O_w += P_w V of tile j - 1 is complete: tensor-core
// operations of one thread complete in order, and the commit follows both.
// What lies behind a sequence's last key in its last tile is another sequence's (or nothing), and
// a masked probability of 0 times an infinity or NaN there is NaN. So in tiles where some row's
// limit ends, the softmax warps zero V rows past the sequence and any non-finite value before
// they hand over P; the (rare) latter are added to the rows that see them in the epilogue.
// All waits are bounded.
#include "kv8.cuh"
#include "tc_common.cuh"

namespace jepa {

namespace {

using namespace tc;

constexpr int TQ = 128;            // rows of a query tile (MMA M)
constexpr int TK = 128;            // keys of a tile
constexpr int P_THREADS = 384;
// Registers a thread after setmaxnreg. The block launches with 168 each (384 threads); the two
// softmax warpgroups draw what the third returns: 256 * 208 + 128 * 88 = 384 * 168.
constexpr int REGS_SOFTMAX = 208, REGS_OTHER = 88;
static_assert(256 * REGS_SOFTMAX + 128 * REGS_OTHER == P_THREADS * 168, "register split");
constexpr uint32_t P_TMEM = 512;
constexpr int BLK = TQ * 128;      // bytes of 128 rows x 64 bf16 (one swizzled block)

template <int D>
struct PShape {
  static constexpr int NB = D / 64;                 // 64-column blocks
  static constexpr int TILE = NB * BLK;             // bytes of a Q, K or V tile
  static constexpr int STAGES = D == 128 ? 4 : 6;
  static constexpr int OFF_RING = 2 * TILE;
  static constexpr int OFF_BAR = OFF_RING + STAGES * TILE;
  // q_full, kv_full[STAGES], kv_empty[STAGES], s_full[2], p_full[2], o_full[2], teardown
  static constexpr int NUM_BARS = 1 + 2 * STAGES + 6 + 1;
  static constexpr int SMEM = OFF_BAR + NUM_BARS * 8 + 64 + 1024;
};

struct PArgs {
  bf16* out;
  float* lse;
  const bf16* v;
  long long v_stride;
  const int *cu_q, *cu_k;
  int tokens_q, tokens_k, batch, q_heads, kv_heads, group, per_tile, frame;
  float scale_log2;
};

// What a CTA works on.
struct Item {
  int valid;
  int head;            // key / value head
  int q0, nq, k0, nk;  // the sequence's first packed row and length
  int t0;              // first token of tile 0 within the sequence
};

__device__ __forceinline__ float p_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float p_max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// Bounded wait as mbar_wait of the other kernels, without a call: the register split of
// setmaxnreg does not go together with one.
__device__ __forceinline__ bool p_wait(uint32_t bar, uint32_t parity, volatile int* abort_smem,
                                       int* err_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = globaltimer();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 0) {
      if (*abort_smem) return false;
      if (globaltimer() - t0 > WAIT_LIMIT_NS) {
        *abort_smem = 1;
        atomicOr(err_flag, DEV_ERR_TIMEOUT);
        return false;
      }
    }
  }
}
// MN-major operand of two 64-wide blocks: the leading byte offset is the distance between them.
__device__ __forceinline__ uint64_t desc_mn_blocks(uint32_t saddr) {
  return (desc_sw128_mn(saddr) & ~((uint64_t)0x3fff << 16)) | ((uint64_t)(BLK >> 4) << 16);
}

// Keys that token i of a sequence sees.
__device__ __forceinline__ int limit_of(const Item& it, int i, int frame) {
  const int p = i + it.nk - it.nq;
  if (p < 0) return 0;
  const long long lim = ((long long)(p / frame) + 1) * frame;
  return lim < it.nk ? (int)lim : it.nk;
}

// The `index`-th 256-row item; sequences in order, within one the last rows (most keys) first.
__device__ __forceinline__ void find_item(const PArgs& a, long long index, Item& it, int* err_flag) {
  const int lane = threadIdx.x & 31, span = 2 * a.per_tile;
  long long base = 0;
  it.valid = 0;
  for (int s0 = 0; s0 < a.batch; s0 += 32) {
    const int s = s0 + lane;
    int q0 = 0, nq = 0, k0 = 0, nk = 0;
    if (s < a.batch) {
      q0 = __ldg(a.cu_q + s);
      k0 = __ldg(a.cu_k + s);
      const int q1 = __ldg(a.cu_q + s + 1), k1 = __ldg(a.cu_k + s + 1);
      if (q0 < 0 || q1 < q0 || q1 > a.tokens_q || k0 < 0 || k1 < k0 || k1 > a.tokens_k) {
        atomicOr(err_flag, DEV_ERR_INDEX);   // offsets outside the buffers: sequence skipped
      } else {
        nq = q1 - q0;
        nk = k1 - k0;
      }
    }
    const int tiles = (nq + span - 1) / span;
    long long incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const uint32_t beyond = __ballot_sync(0xffffffffu, base + incl * a.kv_heads > index);
    if (beyond) {
      const int src = __ffs((int)beyond) - 1;
      const int n = __shfl_sync(0xffffffffu, tiles, src);
      const long long first = base + (__shfl_sync(0xffffffffu, incl, src) - n) * a.kv_heads;
      const long long in = index - first;
      it.valid = 1;
      it.head = (int)(in % a.kv_heads);
      it.t0 = (n - 1 - (int)(in / a.kv_heads)) * span;
      it.q0 = __shfl_sync(0xffffffffu, q0, src);
      it.nq = __shfl_sync(0xffffffffu, nq, src);
      it.k0 = __shfl_sync(0xffffffffu, k0, src);
      it.nk = __shfl_sync(0xffffffffu, nk, src);
      return;
    }
    base += __shfl_sync(0xffffffffu, incl, 31) * a.kv_heads;
  }
}

template <int D>
__global__ void __launch_bounds__(P_THREADS, 1)
    k_attention_packed(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const PArgs a, int* err_flag) {
  using S = PShape<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t sb = smem_u32(smem);
  const uint32_t q_full = sb + S::OFF_BAR;
  auto kv_full = [&](int s) { return q_full + 8u * (1 + s); };
  auto kv_empty = [&](int s) { return q_full + 8u * (1 + S::STAGES + s); };
  const uint32_t s_full0 = q_full + 8u * (1 + 2 * S::STAGES);
  auto s_full = [&](int w) { return s_full0 + 8u * w; };
  auto p_full = [&](int w) { return s_full0 + 16 + 8u * w; };
  auto o_full = [&](int w) { return s_full0 + 32 + 8u * w; };
  const uint32_t teardown = s_full0 + 48;
  uint8_t* tail = smem + S::OFF_BAR + S::NUM_BARS * 8;
  uint32_t* tmem_slot = (uint32_t*)tail;
  volatile int* abort_flag = (volatile int*)(tail + 4);
  volatile int* dirty = (volatile int*)(tail + 8);   // a non-finite V was taken out of a tile
  Item* item_slot = (Item*)(tail + 16);
  static_assert(sizeof(Item) <= 48, "the item fits behind the barriers");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 9) {
    Item it;
    find_item(a, blockIdx.x, it, err_flag);
    if (lane == 0) *item_slot = it;
  }
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(kv_full(s), 1);
      mbar_init(kv_empty(s), 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(s_full(w), 1);
      mbar_init(p_full(w), 4);
      mbar_init(o_full(w), 1);
    }
    mbar_init(teardown, 1);
    *abort_flag = 0;
    *dirty = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  __syncthreads();
  const Item it = *item_slot;
  if (!it.valid) return;
  if (warp == 8) tmem_alloc(smem_u32(tmem_slot), P_TMEM);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto tS = [&](int w) { return tmem + 128u * w; };
  auto tO = [&](int w) { return tmem + 256u + 128u * w; };

  // key tiles of each query tile (0: it has no rows, or none that sees a key)
  const int span = a.per_tile;
  int nt[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int first = it.t0 + w * span, last = min(it.nq, first + span) - 1;
    nt[w] = first < it.nq ? (limit_of(it, last, a.frame) + TK - 1) / TK : 0;
  }
  const int n_tiles = max(nt[0], nt[1]);
  // the first key tile in which some row's limit ends
  const int first_edge = limit_of(it, it.t0, a.frame) / TK;

  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
  if (warp == 9) {
    if (lane == 0) {
      // ---------------- TMA producer ----------------
      const int box = a.per_tile * a.group * 128;
      if (n_tiles > 0) {
        mbar_expect_tx(q_full, (uint32_t)(S::NB * box * ((nt[0] > 0) + (nt[1] > 0))));
        for (int w = 0; w < 2; ++w)
          if (nt[w] > 0)
            for (int b = 0; b < S::NB; ++b)
              tma_load_3d(sb + w * S::TILE + b * BLK, &tmQ, 64 * b, it.head * a.group,
                          it.q0 + it.t0 + w * span, q_full);
      }
      for (int n = 0; n < 2 * n_tiles; ++n) {
        const int st = n % S::STAGES;
        if (n >= S::STAGES &&
            !p_wait(kv_empty(st), ((n / S::STAGES) - 1) & 1, abort_flag, err_flag))
          break;
        const uint32_t dst = sb + S::OFF_RING + st * S::TILE;
        mbar_expect_tx(kv_full(st), S::TILE);
        for (int b = 0; b < S::NB; ++b)
          tma_load_3d(dst + b * BLK, (n & 1) ? &tmV : &tmK, 64 * b, it.head, it.k0 + (n >> 1) * TK,
                      kv_full(st));
      }
      if (*abort_flag) {
        // give copies still in flight into this CTA's shared memory time to land
        const unsigned long long t0 = globaltimer();
        while (globaltimer() - t0 < 2000000ull) {
        }
      }
    }
  } else if (warp == 8) {
    if (lane == 0 && n_tiles > 0) {
      // ---------------- MMA issuer ----------------
      constexpr uint32_t idS = idesc_bf16(TQ, TK, false);
      constexpr uint32_t idO = idesc_bf16(TQ, D, true);
      auto slot = [&](int n) { return sb + S::OFF_RING + (n % S::STAGES) * S::TILE; };
      auto landed = [&](int n) {
        return p_wait(kv_full(n % S::STAGES), (n / S::STAGES) & 1, abort_flag, err_flag);
      };
      auto scores = [&](int w, int j) {
        const uint64_t qd = desc_sw128(sb + w * S::TILE), kd = desc_sw128(slot(2 * j));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t at = (uint64_t)((kk >> 2) * (BLK >> 4) + 2 * (kk & 3));
          mma_bf16_ss(tS(w), qd + at, kd + at, idS, kk > 0);
        }
        mma_commit(s_full(w));
      };
      auto product = [&](int w, int j) {
        const uint64_t vd = D == 128 ? desc_mn_blocks(slot(2 * j + 1)) : desc_sw128_mn(slot(2 * j + 1));
#pragma unroll
        for (int kk = 0; kk < TK / 16; ++kk)
          mma_bf16_ts(tO(w), tS(w) + 8u * kk, vd + (uint64_t)(kk * (2048 >> 4)), idO,
                      (j > 0) || (kk > 0));
        if (j + 1 == nt[w]) mma_commit(o_full(w));
      };
      bool ok = p_wait(q_full, 0, abort_flag, err_flag) && landed(0);
      if (ok) {
        tc_fence_after();
        if (nt[0] > 0) scores(0, 0);
        if (nt[1] > 0) scores(1, 0);
        mma_commit(kv_empty(0));
      }
      for (int j = 0; j < n_tiles && ok; ++j) {
        ok = landed(2 * j + 1);
        for (int w = 0; w < 2 && ok; ++w) {
          if (j < nt[w]) {
            ok = p_wait(p_full(w), j & 1, abort_flag, err_flag);
            if (!ok) break;
            tc_fence_after();
            product(w, j);
          }
          if (w == 1) mma_commit(kv_empty((2 * j + 1) % S::STAGES));
          if (j + 1 < n_tiles && w == 0) ok = landed(2 * j + 2);
          if (ok && j + 1 < nt[w]) {
            tc_fence_after();
            scores(w, j + 1);
          }
          if (w == 1 && j + 1 < n_tiles) mma_commit(kv_empty((2 * j + 2) % S::STAGES));
        }
      }
      mma_commit(teardown);
      const unsigned long long t0 = globaltimer();
      while (!mbar_try_wait(teardown, 0) && globaltimer() - t0 < WAIT_LIMIT_NS) {
      }
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
    // ---------------- softmax (thread = row) ----------------
    const int w = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const int tok = it.t0 + w * span + row / a.group;       // within the sequence
    const bool mine = row < span * a.group && tok < it.nq;
    const int lim = mine ? limit_of(it, tok, a.frame) : 0x7fffffff;
    const int lim_min = __reduce_min_sync(0xffffffffu, lim);
    const bool active = __any_sync(0xffffffffu, mine);
    const uint32_t tSw = tS(w) + lane_off, tOw = tO(w) + lane_off;
    const float scale_log2 = a.scale_log2;
    // a warp goes on, or gives up, as one: what follows a wait are warp-wide instructions
    auto all_wait = [&](uint32_t bar, uint32_t parity) {
      return __all_sync(0xffffffffu, p_wait(bar, parity, abort_flag, err_flag)) != 0;
    };
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < nt[w]; ++j) {
      if (!all_wait(s_full(w), j & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (active) {
        uint32_t r[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32_async(tSw + 32 * q, r[q]);
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_wait(r[q]);
        if ((j + 1) * TK > lim_min) {
          const int left = lim - j * TK;
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (32 * q + c >= left) r[q][c] = __float_as_uint(-INFINITY);
        }
        float part[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const uint32_t* x = &r[q >> 2][8 * (q & 3)];
          part[q] = p_max3(p_max3(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2])),
                           p_max3(__uint_as_float(x[3]), __uint_as_float(x[4]), __uint_as_float(x[5])),
                           fmaxf(__uint_as_float(x[6]), __uint_as_float(x[7])));
        }
        const float cmax =
            fmaxf(p_max3(p_max3(part[0], part[1], part[2]), p_max3(part[3], part[4], part[5]),
                         p_max3(part[6], part[7], part[8])),
                  p_max3(p_max3(part[9], part[10], part[11]), p_max3(part[12], part[13], part[14]),
                         part[15]));
        // the exponent's reference moves only when the maximum grew by more than 2^8: the same
        // reference scales O and the sum, so the result is unchanged
        const bool bump = cmax > m && (m == -INFINITY || (cmax - m) * scale_log2 > 8.0f);
        const float mnew = bump ? cmax : m;
        const float alpha = bump ? p_ex2((m - mnew) * scale_log2) : 1.f;
        const float ms = mnew == -INFINITY ? 0.f : mnew * scale_log2;
        m = mnew;
        if (j > 0 && __any_sync(0xffffffffu, bump)) {
          // O holds the product of tile j - 1 and before (see the head of the file)
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            uint32_t ov[32];
            tmem_ld32_async(tOw + 32 * q, ov);
            tmem_wait(ov);
#pragma unroll
            for (int c = 0; c < 32; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * alpha);
            tmem_st32(tOw + 32 * q, ov);
          }
        }
        const unsigned long long sc2 = f2_pack(scale_log2, scale_log2), nms2 = f2_pack(-ms, -ms);
        unsigned long long sum2[2] = {0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const uint32_t* x = &r[2 * h + (c >> 4)][2 * (c & 15)];
            const float2 e = f2_unpack(
                f2_fma(f2_pack(__uint_as_float(x[0]), __uint_as_float(x[1])), sc2, nms2));
            const float p0 = p_ex2(e.x), p1 = p_ex2(e.y);
            sum2[c & 1] = f2_add(sum2[c & 1], f2_pack(p0, p1));
            const __nv_bfloat162 b = __floats2bfloat162_rn(p0, p1);
            pk[c] = *reinterpret_cast<const uint32_t*>(&b);
          }
          tmem_st32(tSw + 32 * h, pk);
        }
        const float2 sm = f2_unpack(f2_add(sum2[0], sum2[1]));
        l = l * alpha + (sm.x + sm.y);
        tmem_st_wait();
      }
      if (j >= first_edge && w == (j < nt[0] ? 0 : 1)) {
        // this tile's V is about to be used for the first time: thread = key
        const int n = 2 * j + 1;
        if (!all_wait(kv_full(n % S::STAGES), (n / S::STAGES) & 1)) {
          ok = false;
          break;
        }
        uint8_t* v_row = smem + S::OFF_RING + (n % S::STAGES) * S::TILE + row * 128;
        const bool behind = j * TK + row >= it.nk;
        uint32_t odd = 0;
        if (!behind) {
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            const uint4 x = *reinterpret_cast<const uint4*>(v_row + (c >> 3) * BLK + 16 * ((c & 7) ^ (row & 7)));
            odd |= ((x.x & 0x7f807f80u) + 0x00800080u) | ((x.y & 0x7f807f80u) + 0x00800080u) |
                   ((x.z & 0x7f807f80u) + 0x00800080u) | ((x.w & 0x7f807f80u) + 0x00800080u);
          }
          odd &= 0x80008000u;
        }
        if (behind || odd) {
          if (odd) *dirty = 1;
          for (int c = 0; c < D / 8; ++c) {
            uint4* at = reinterpret_cast<uint4*>(v_row + (c >> 3) * BLK + 16 * ((c & 7) ^ (row & 7)));
            uint32_t x[4] = {0, 0, 0, 0};
            if (!behind) {
              const uint4 y = *at;
              x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if ((x[i] & 0x7f80u) == 0x7f80u) x[i] &= 0xffff0000u;
                if ((x[i] & 0x7f800000u) == 0x7f800000u) x[i] &= 0x0000ffffu;
              }
            }
            *at = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(w));
    }
    if (ok && active) {
      const long long at = ((long long)(it.q0 + tok) * a.q_heads + it.head * a.group + row % a.group);
      const bool any = nt[w] > 0;
      if (any) {
        ok = all_wait(o_full(w), 0);
        tc_fence_after();
      }
      if (ok) {
        const bool empty = l == 0.f;
        const float inv = empty ? 0.f : 1.f / l;
        const bool fix = any && *dirty != 0;
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t ov[32];
          if (any) {
            tmem_ld32_async(tOw + 32 * q, ov);
            tmem_wait(ov);
          }
#pragma unroll
          for (int c = 0; c < 32; ++c)
            ov[c] = __float_as_uint(empty ? 0.f : __uint_as_float(ov[c]) * inv);
          if (fix && mine) {
            for (int key = first_edge * TK; key < lim; ++key) {
              const bf16* vr = a.v + (long long)(it.k0 + key) * a.v_stride + (long long)it.head * D + 32 * q;
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                const float x = __bfloat162float(vr[c]);
                if (!(fabsf(x) < INFINITY)) ov[c] = __float_as_uint(__uint_as_float(ov[c]) + x);
              }
            }
          }
          if (mine) {
            bf16* to = a.out + at * D + 32 * q;
#pragma unroll
            for (int c = 0; c < 32; c += 8) {
              uint32_t u[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(ov[c + 2 * i]),
                                                               __uint_as_float(ov[c + 2 * i + 1]));
                u[i] = *reinterpret_cast<const uint32_t*>(&b);
              }
              *reinterpret_cast<uint4*>(to + c) = make_uint4(u[0], u[1], u[2], u[3]);
            }
          }
        }
        if (mine && a.lse)
          a.lse[at] = empty ? -INFINITY
                            : ((m == -INFINITY ? 0.f : m * scale_log2) + log2f(l)) * 0.69314718055994531f;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    __syncwarp();
    tmem_dealloc(tmem, P_TMEM);
  }
}

// bf16 [tokens][heads][dim] (row stride `stride` elements) in boxes of `box_tokens` tokens x
// `box_heads` heads x 64 columns, 128-byte swizzle.
bool make_map_heads(CUtensorMap* m, const void* ptr, int tokens, int heads, int dim,
                    long long stride, int box_tokens, int box_heads) {
  PFN_encodeTiled enc = get_encode();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)stride * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_packed(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                          const PArgs& a, int* err_flag, cudaStream_t s) {
  using S = PShape<D>;
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t e = set_max_dynamic_smem((const void*)k_attention_packed<D>, S::SMEM, attr_done);
  if (e != cudaSuccess) return e;
  // lengths are on the device: an upper bound of the items, surplus CTAs return at once
  const long long items = ((long long)a.tokens_q / (2 * a.per_tile) + a.batch) * a.kv_heads;
  if (items > 0x7fffffffLL) return cudaErrorInvalidValue;
  k_attention_packed<D><<<(unsigned)items, P_THREADS, S::SMEM, s>>>(mq, mk, mv, a, err_flag);
  return cudaGetLastError();
}

}  // namespace

cudaError_t attention_packed(const bf16* q, long long q_stride, const bf16* k, long long k_stride,
                             const bf16* v, long long v_stride, int tokens_q, int tokens_k,
                             int batch, int q_heads, int kv_heads, int dim, const int* cu_q,
                             const int* cu_k, float scale, int frame, bf16* out, float* lse,
                             int* err_flag, int num_sms, cudaStream_t s) {
  (void)num_sms;
  PArgs a;
  a.out = out;
  a.lse = lse;
  a.v = v;
  a.v_stride = v_stride;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.tokens_q = tokens_q;
  a.tokens_k = tokens_k;
  a.batch = batch;
  a.q_heads = q_heads;
  a.kv_heads = kv_heads;
  a.group = q_heads / kv_heads;
  a.per_tile = TQ / a.group;
  a.frame = frame;
  a.scale_log2 = scale * 1.4426950408889634f;
  CUtensorMap mq, mk, mv;
  if (!make_map_heads(&mq, q, tokens_q, q_heads, dim, q_stride, a.per_tile, a.group) ||
      !make_map_heads(&mk, k, tokens_k, kv_heads, dim, k_stride, TK, 1) ||
      !make_map_heads(&mv, v, tokens_k, kv_heads, dim, v_stride, TK, 1))
    return cudaErrorInvalidValue;
  if (dim == 64) return launch_packed<64>(mq, mk, mv, a, err_flag, s);
  if (dim == 128) return launch_packed<128>(mq, mk, mv, a, err_flag, s);
  return cudaErrorInvalidValue;
}

}  // namespace jepa
