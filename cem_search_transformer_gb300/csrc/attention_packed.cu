// Attention of whole packed prompts on the sm_103a tensor cores (tcgen05 + TMEM + TMA), grouped
// heads, head dim 64 or 128.
//
//   o[i] = sum_{j < lim(i)} softmax_j(scale q[i] . k[j]) v[j],   lim(i) = min(nk, (p / F + 1) F),
//   p = i + nk - nq: the query's position among the keys; F = 1 is causal, F = T block-causal over
//   frames of T tokens (the predictor's mask), F >= nk without a mask.
//
// A CTA takes 256 query rows of one sequence and key/value head, two tiles of 128 (or the last 128
// of two heads). A row is a (token, head of the group) pair, token-major, so that a group's heads
// share the tile of keys and short prompts still fill the rows; groups that do not divide 128
// leave a few rows unused.
// Warps:
//   0-3, 4-7  softmax of tile 0 and 1, a row a thread: read S from TMEM, running maximum and sum,
//             P (bf16) over the read scores, rescale O in TMEM when the maximum moved by more than
//             2^8, and at the end normalise and store;
//   8, 9      MMA issuers of tile 0 and 1: S_w = Q_w K^T, O_w += P_w V (P from TMEM, V MN-major from
//             its TMA tile). One warp for both spent its time on issuing: an MMA of 64 columns takes
//             32 cycles, its issue 40 to 60;
//   10        scheduler and TMA producer: the next item, its Q tiles, then K_0, K_1, V_0, K_2, V_1, ...
//             through one ring that runs on across items;
//   11        cleaning of V (below).
// The grid has a CTA for every item there can be, the heaviest of a sequence first. A running CTA
// takes over items whose CTA has not begun (cluster launch control), so that loads and scores of
// the next item run under the present one's last products and read-out, and SMs that finish early
// take more.
// Key tiles are 64 wide and each query tile has two score buffers, so that the scores of tile j + 1
// are there when the softmax is done with tile j: with one buffer of 128 keys a tile waited about
// 1200 cycles for its P V and the next scores after 2200 of softmax (D = 128). The price is 64-key
// scores MMAs, which read Q from shared memory twice as often.
// What bounds it. D = 128: the tensor cores and the power limit (one prompt of 10007 tokens, 32
// query heads over 8: 506 us, 1.63 PFLOP/s). D = 64: the chain of a step, scores -> softmax -> P,
// about 1500 cycles for both tiles, two softmax warps a scheduler with a serial chain each. No pipe is
// half full: the exponentials take 512 of those cycles (32 a cycle and SM, 24% by the counters; half
// of them left out takes 6% off), issue 44%, tensor 25%. And an item's 2000 to 3000 cycles between
// two loops, of which half is hidden
// (32 prompts of 774 tokens, 16 heads, frames of 258: 118 us, of which 22 for the last six rows of
// each, a tile of their own, two heads at a time; 125 a head at a time, and with its keys shared
// out over both tiles 124, and 2% more elsewhere).
// What lies behind a sequence's last key in its last tile is another sequence's (or nothing), and
// a masked probability of 0 times an infinity or NaN there is NaN. So in tiles where some row's
// limit ends, a warp zeroes V rows past the sequence and any non-finite value before the product
// reads them; the (rare) latter are added to the rows that see them in the read-out.
// P is rounded to bf16 (half a step 2^-8) because both operands of the product have one type, and V in
// f16 would lose bf16's range; its sum is that of the unrounded ones, fp32. Against 64 bits the
// output is off by 0.0023 (relative, all rows) where fp32 weights and one rounding give 0.0017.
// All waits are bounded, by what moves and not by the clock alone: an item of 2^27 keys lasts 1.6 s
// (twice that for a pair of heads), and adding non-finite values of as many keys 19 s.
#include "kv8.cuh"
#include "tc_common.cuh"
#include "wait_clock.h"

namespace jepa {

namespace {

using namespace tc;

constexpr int TQ = 128;            // rows of a query tile (MMA M)
constexpr int P_THREADS = 384;     // 8 warps of softmax, then two issuers, producer, cleaning
constexpr int W_MMA = 8, W_TMA = 10;   // issuers: W_MMA and the next; cleaning: the last
// Registers a thread after setmaxnreg. The block launches with 168 each; the softmax warpgroups
// draw what the last one returns.
constexpr int REGS_SOFTMAX = 192, REGS_OTHER = 120;
static_assert(256 * REGS_SOFTMAX + 128 * REGS_OTHER == P_THREADS * 168, "register split");
constexpr uint32_t P_TMEM = 512;
// Items for each SM from which on a sequence's last rows, where they fill one query tile at most, are
// taken for two heads at a time, a tile each with its own keys: the two chains run side by side (512
// sequences of six tokens 105 against 155 us). With few items the heads are better on SMs of their
// own (four sequences of 774 tokens, 16 heads: 29 us, 32 in pairs).
constexpr int PAIRS_FROM = 4;
constexpr int BLK = TQ * 128;      // bytes of 128 rows x 64 bf16 (one swizzled block of Q)

template <int D>
struct PShape {
  static constexpr int TK = 64;                     // keys of a tile
  static constexpr int NBUF = 2;                    // score buffers of a query tile
  static constexpr int TM = TK * NBUF + D;          // its columns of TMEM: scores, then output
  static constexpr int NB = D / 64;                 // 64-column blocks
  static constexpr int KBLK = TK * 128;             // bytes of one block of K or V
  static constexpr int QTILE = NB * BLK, TILE = NB * KBLK;   // bytes of a Q tile, of K or V
  static constexpr int STAGES = D == 64 ? 8 : 4;    // of the ring: V_j and K_{j + NBUF}
  static constexpr int OFF_RING = 2 * QTILE;
  static constexpr int OFF_OUT = OFF_RING + STAGES * 2 * TILE;   // read-out: 2 x 32 rows x 64 B a warp
  static constexpr int OFF_BAR = OFF_OUT + 8 * 4096;
  // kv_full[STAGES], kv_empty[STAGES], edge_full[STAGES], q_full[2], q_empty[2], s_full[2][NBUF],
  // p_full[2][NBUF], pv[2][NBUF], item_full[2], item_empty[2], next, teardown
  static constexpr int NUM_BARS = 3 * STAGES + 10 + 6 * NBUF;
  static constexpr int OFF_TAIL = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_ROWS = OFF_TAIL + 176;   // (token, place among its heads) of a tile's rows
  static constexpr int SMEM = OFF_ROWS + TQ * 8 + 1024;
  static_assert(SMEM <= 232448, "shared memory of a CTA");
  static_assert(NBUF == 2, "two score buffers in turn");
  static_assert(2 * TM <= (int)P_TMEM && TK % 32 == 0 && KBLK % 1024 == 0, "tiles");
};

struct PArgs {
  bf16* out;
  float* lse;
  const bf16* v;
  long long v_stride;
  const int *cu_q, *cu_k;
  int tokens_q, tokens_k, batch, q_heads, kv_heads, group, per_tile, frame;
  int pairs;                      // 1: items of a single query tile take two heads
  unsigned long long frame_inv;   // floor(2^63 / frame) + 1
  float scale_log2;
};

// What a CTA works on next.
struct Item {
  int valid;           // 0: nothing is left
  int head;            // key / value head
  int q0, nq, k0, nk;  // the sequence's first packed row and length
  int t0;              // first token of tile 0 within the sequence
  int nt[2];           // key tiles of each query tile (0: no rows, or none that sees a key)
  int first_edge;      // the first key tile in which some row's limit ends; where dirty, the first in
                       // which V is not finite (the cleaning warp moves it)
  int dirty;           // 0, or one past the last tile out of which a non-finite V was taken
  int pair;            // both tiles hold the sequence's last rows, of this head and the next
};
// Where the search for an item goes on: items come in ascending order as a rule.
struct Cursor {
  int s0;
  long long base, total;   // total: all items, once a search has come to the end
};

__device__ __forceinline__ float p_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float p_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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
// setmaxnreg does not go together with one. The cleaning warp waits as long as there are items, and so
// stands watch: its waits give up where nothing MOVED for one to two limits (no tile was loaded, no key
// read again in the read-out: counted behind the abort flag), and take all others along. The others'
// limit lies beyond the longest item or read-out of two tiles: the rule's code in the softmax too took
// 5% (one prompt of 10007 tokens 531 us, 505), in all but softmax and issuers 1% of the frames' case.
constexpr unsigned long long STEP_LIMIT_NS = 20 * WAIT_LIMIT_NS;
template <bool MOVED = false>
__device__ __forceinline__ bool p_wait(uint32_t bar, uint32_t parity, volatile int* abort_smem,
                                       int* err_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  WaitClock clock(globaltimer());
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 0) {
      if (*abort_smem) return false;
      const unsigned long long now = globaltimer();
      if (clock.due(now, MOVED ? WAIT_LIMIT_NS : STEP_LIMIT_NS) &&
          (!MOVED || clock.stuck(now, (unsigned)(abort_smem[1] + abort_smem[2])))) {
        *abort_smem = 1;
        atomicOr(err_flag, DEV_ERR_TIMEOUT);
        return false;
      }
    }
  }
}
// 32 lanes x 16 columns TMEM store (thread i -> lane i).
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ float max32(const uint32_t (&r)[32]) {
  float part[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t* x = &r[8 * q];
    part[q] = p_max3(p_max3(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2])),
                     p_max3(__uint_as_float(x[3]), __uint_as_float(x[4]), __uint_as_float(x[5])),
                     fmaxf(__uint_as_float(x[6]), __uint_as_float(x[7])));
  }
  return fmaxf(p_max3(part[0], part[1], part[2]), part[3]);
}
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(yes));
  return yes != 0;
}
// MN-major operand of two 64-wide blocks `apart` bytes from each other: the leading byte offset.
__device__ __forceinline__ uint64_t desc_mn_blocks(uint32_t saddr, uint32_t apart) {
  return (desc_sw128_mn(saddr) & ~((uint64_t)0x3fff << 16)) | ((uint64_t)(apart >> 4) << 16);
}


// MMAs and commits of a whole warp, of which the elected lane's counts: the predicate is inside, so
// that the code around stays convergent and its addresses in uniform registers.
__device__ __forceinline__ void w_mma_ss(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc, uint32_t leader) {
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\t" "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(ad), "l"(bd), "r"(idesc), "r"(acc), "r"(leader));
}
__device__ __forceinline__ void w_mma_ts(uint32_t d, uint32_t at, uint64_t bd, uint32_t idesc, uint32_t acc, uint32_t leader) {
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\t" "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(at), "l"(bd), "r"(idesc), "r"(acc), "r"(leader));
}
__device__ __forceinline__ void w_commit(uint32_t bar, uint32_t leader) {
  asm volatile("{\n\t.reg .pred q;\n\t" "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(leader) : "memory");
}
// Keys that token i of a sequence sees. floor(p / frame) for 0 <= p < 2^31 as the high half of
// 2 p * frame_inv: the product exceeds 2^64 p / frame by less than 2 p <= 2^32, too little to
// reach the next multiple (a division's latency was a third of an item's start).
__device__ __forceinline__ int limit_of(const Item& it, int i, const PArgs& a) {
  const int p = i + it.nk - it.nq;
  if (p < 0) return 0;
  const long long f = (long long)__umul64hi(2ull * (unsigned)p, a.frame_inv);
  const long long lim = (f + 1) * a.frame;
  return lim < it.nk ? (int)lim : it.nk;
}

// The `index`-th 256-row item; sequences in order, within one the last rows (most keys) first, of
// which a pair of heads may be one item.
template <int TK>
__device__ __forceinline__ void find_item(const PArgs& a, long long index, Cursor& cur, Item& it,
                                          int* err_flag) {
  const int lane = threadIdx.x & 31, span = 2 * a.per_tile;
  it.valid = 0;
  it.dirty = 0;
  if (index >= cur.total) return;
  if (index < cur.base) cur = Cursor{0, 0, cur.total};   // not in order after all
  long long base = cur.base;
  for (int s0 = cur.s0; s0 < a.batch; s0 += 32) {
    const int s = s0 + lane;
    int q0 = 0, nq = 0, k0 = 0, nk = 0;
    if (s < a.batch) {
      q0 = __ldg(a.cu_q + s);
      k0 = __ldg(a.cu_k + s);
      const int q1 = __ldg(a.cu_q + s + 1), k1 = __ldg(a.cu_k + s + 1);
      if (!(kv8_span_ok(q0, q1, a.tokens_q) & kv8_span_ok(k0, k1, a.tokens_k))) {
        atomicOr(err_flag, DEV_ERR_INDEX);   // offsets outside the buffers: sequence skipped
      } else {
        nq = q1 - q0;
        nk = k1 - k0;
      }
    }
    const int tiles = (nq + span - 1) / span;
    const bool lone = a.pairs && tiles > 0 && nq - (tiles - 1) * span <= a.per_tile;
    const long long mine = (long long)tiles * a.kv_heads - (lone ? a.kv_heads >> 1 : 0);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const uint32_t beyond = __ballot_sync(0xffffffffu, base + incl > index);
    if (beyond) {
      const int src = __ffs((int)beyond) - 1;
      const int n = __shfl_sync(0xffffffffu, tiles, src);
      const bool pairs = __shfl_sync(0xffffffffu, (int)lone, src) != 0;
      const unsigned in = (unsigned)__shfl_sync(0xffffffffu, (int)(index - base - (incl - mine)), src);
      const unsigned heads = a.kv_heads, wide = pairs ? (heads + 1) >> 1 : heads;
      int row = 0;
      if (in < wide) {
        it.head = (int)(pairs ? 2 * in : in);
      } else {
        row = 1 + (int)((in - wide) / heads);
        it.head = (int)((in - wide) % heads);
      }
      it.valid = 1;
      it.pair = pairs && row == 0 && it.head + 1 < a.kv_heads;
      it.t0 = (n - 1 - row) * span;
      it.q0 = __shfl_sync(0xffffffffu, q0, src);
      it.nq = __shfl_sync(0xffffffffu, nq, src);
      it.k0 = __shfl_sync(0xffffffffu, k0, src);
      it.nk = __shfl_sync(0xffffffffu, nk, src);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int t = it.t0 + w * a.per_tile, last = min(it.nq, t + a.per_tile) - 1;
        it.nt[w] = t < it.nq ? (limit_of(it, last, a) + TK - 1) / TK : 0;
      }
      if (it.pair) it.nt[1] = it.nt[0];
      it.first_edge = limit_of(it, it.t0, a) / TK;
      cur.s0 = s0;
      cur.base = base;
      return;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  cur.total = base;
}

// Reports bad offsets among the sequences of a place of the grid, 256 at a time, by THREADS threads.
// Searches look at all sequences as long as one of them runs to the end, which may be none where
// there are more sequences than queries: every place then has an item. (One query among 65535
// sequences 31 us, 10 unchecked; among 1024 the same 10.)
template <int THREADS>
__device__ __forceinline__ void report_offsets(const PArgs& a, int place, int thread, int* err_flag) {
  bool ok = true;
#pragma unroll 4
  for (long long s0 = place * 256LL; s0 < a.batch; s0 += gridDim.x * 256LL)
#pragma unroll
    for (int k = thread; k < 256; k += THREADS) {
      const int s = (int)min(s0 + k, a.batch - 1LL);
      ok &= kv8_span_ok(__ldg(a.cu_q + s), __ldg(a.cu_q + s + 1), a.tokens_q) &
            kv8_span_ok(__ldg(a.cu_k + s), __ldg(a.cu_k + s + 1), a.tokens_k);
    }
  if (!ok) atomicOr(err_flag, DEV_ERR_INDEX);
}

// Asks for the next CTA of the grid that has not begun to run to be given to this one instead (16
// bytes at `dst`, announced at `bar`); clc_index reads the answer: its index, or -1 for none.
__device__ __forceinline__ void clc_request(uint32_t dst, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
      ::"r"(dst), "r"(bar)
      : "memory");
}
__device__ __forceinline__ int clc_index(uint32_t src) {
  int x;
  asm volatile(
      "{\n\t.reg .b128 answer;\n\t.reg .pred given;\n\t.reg .b32 y, z;\n\t"
      "ld.shared.b128 answer, [%1];\n\t"
      "mov.b32 %0, -1;\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 given, answer;\n\t"
      "@given clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, _}, answer;\n\t"
      "}"
      : "=r"(x)
      : "r"(src)
      : "memory");
  return x;
}

template <int D>
__global__ void __launch_bounds__(P_THREADS, 1)
    k_attention_packed(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const PArgs a, int* err_flag) {
  using S = PShape<D>;
  constexpr int TK = S::TK, KBLK = S::KBLK;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t sb = smem_u32(smem);
  const uint32_t bars = sb + S::OFF_BAR;
  auto kv_full = [&](int s) { return bars + 8u * s; };
  auto kv_empty = [&](int s) { return bars + 8u * (S::STAGES + s); };
  auto edge_full = [&](int s) { return bars + 8u * (2 * S::STAGES + s); };
  const uint32_t rest = bars + 24u * S::STAGES;
  auto q_full = [&](int w) { return rest + 8u * w; };
  auto q_empty = [&](int w) { return rest + 16 + 8u * w; };
  // of query tile w and score buffer b
  auto s_full = [&](int w, int b) { return rest + 32 + 8u * (S::NBUF * w + b); };
  auto p_full = [&](int w, int b) { return rest + 32 + 8u * (S::NBUF * (2 + w) + b); };
  auto pv_done = [&](int w, int b) { return rest + 32 + 8u * (S::NBUF * (4 + w) + b); };
  const uint32_t rest2 = rest + 32 + 48u * S::NBUF;
  auto item_full = [&](int b) { return rest2 + 8u * b; };
  auto item_empty = [&](int b) { return rest2 + 16 + 8u * b; };
  const uint32_t next_full = rest2 + 32, teardown = rest2 + 40;
  uint8_t* tail = smem + ((S::OFF_TAIL + 15) & ~15);
  Item* items = (Item*)tail;                              // two slots
  const uint32_t next_slot = smem_u32(tail + 2 * sizeof(Item));   // 16 bytes, 16-byte aligned
  uint32_t* tmem_slot = (uint32_t*)(tail + 2 * sizeof(Item) + 16);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  volatile int* tiles_loaded = abort_flag + 1;
  int* const keys_read = (int*)(tmem_slot + 3);
  static_assert(2 * sizeof(Item) + 16 + 16 + 15 <= 160 && sizeof(Item) % 16 == 0, "tail");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int span = a.per_tile;
  int2* const tile_rows = (int2*)(smem + S::OFF_ROWS);
  if (threadIdx.x < TQ) {
    const int t = threadIdx.x / a.group;
    tile_rows[threadIdx.x] = make_int2(t < span ? t : 0x7fffffff, t * a.q_heads + (threadIdx.x - t * a.group));
  }
  Cursor cursor{0, 0, 0x7fffffffffffffffLL};
  if (warp == W_TMA) {
    Item it;
    find_item<S::TK>(a, blockIdx.x, cursor, it, err_flag);
    if (lane == 0) items[0] = it;
  } else if (warp < W_MMA && a.tokens_q < a.batch) {
    report_offsets<256>(a, blockIdx.x, threadIdx.x, err_flag);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(kv_full(s), 2);    // the producer twice, or once it and once the cleaning warp
      mbar_init(kv_empty(s), 2);   // both issuers
      mbar_init(edge_full(s), 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(q_full(w), 1);
      mbar_init(q_empty(w), 1);
      for (int b = 0; b < S::NBUF; ++b) {
        mbar_init(s_full(w, b), 1);
        mbar_init(p_full(w, b), 4);
        mbar_init(pv_done(w, b), 1);
      }
      mbar_init(item_full(w), 1);
      mbar_init(item_empty(w), 11);   // all warps but the producer
    }
    mbar_init(next_full, 1);
    mbar_init(teardown, 2);
    *abort_flag = 0;
    *tiles_loaded = 0;
    *keys_read = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  __syncthreads();
  if (warp == W_MMA) tmem_alloc(smem_u32(tmem_slot), P_TMEM);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  auto tS = [&](int w, int b) { return tmem + (uint32_t)(S::TM * w + TK * b); };
  auto tO = [&](int w) { return tmem + (uint32_t)(S::TM * w + TK * S::NBUF); };
  if (warp >= W_MMA) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
    if (warp == W_TMA) {
      // ---------------- scheduler and TMA producer ----------------
      const int box = a.per_tile * a.group * 128;
      int n = 0, qn[2] = {0, 0};   // tiles through the ring, items that loaded Q_w
      uint32_t answers = 0;
      bool asked = false;
      auto ask = [&]() {           // for another CTA's item
        asked = true;
        if (lane == 0) {
          fence_proxy_async_smem();   // the slot's last answer has been read
          mbar_expect_tx(next_full, 16);
          clc_request(next_slot, next_full);
        }
      };
      bool ok = true;
      for (int i = 0; ok; ++i) {
        Item it;
        it.valid = 0;
        if (i == 0) it = items[0];
        // the grid may be larger than what there is to do: CTAs without an item are taken out of it
        // here, which is faster than letting each begin (4 of 1024 sequences not empty: 66 us, 1130)
        while (!it.valid) {
          if (!asked) ask();
          ok = __all_sync(0xffffffffu, p_wait(next_full, answers & 1, abort_flag, err_flag));
          if (!ok) break;
          ++answers;
          asked = false;
          const int index = clc_index(next_slot);
          __syncwarp();
          if (index < 0) break;
          if (a.tokens_q < a.batch) report_offsets<32>(a, index, lane, err_flag);
          find_item<S::TK>(a, index, cursor, it, err_flag);
        }
        if (!ok) break;
        if (i >= 2) {
          ok = __all_sync(0xffffffffu, p_wait(item_empty(i & 1), ((i >> 1) - 1) & 1, abort_flag, err_flag));
          if (!ok) break;
        }
        if (lane == 0) items[i & 1] = it;
        __syncwarp();
        if (lane == 0) mbar_arrive(item_full(i & 1));
        if (!it.valid) break;
        ask();
        if (lane == 0) {
          const int pair = it.pair, n_tiles = max(it.nt[0], it.nt[1]) << pair;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (!ok || it.nt[w] == 0) continue;
            ok = qn[w] == 0 || p_wait(q_empty(w), (qn[w] - 1) & 1, abort_flag, err_flag);
            if (!ok) continue;
            ++qn[w];
            mbar_expect_tx(q_full(w), (uint32_t)(S::NB * box));
            for (int b = 0; b < S::NB; ++b)
              tma_load_3d(sb + w * S::QTILE + b * BLK, &tmQ, 64 * b, (it.head + (pair & w)) * a.group,
                          it.q0 + it.t0 + (pair ? 0 : w * span), q_full(w));
          }
          // K_0 and K_1 in a stage of their own each, then V_j beside K_{j + 2}: what the issuers
          // take in one step, behind one barrier. A pair's heads take turns: i is its key tile i / 2
          auto load = [&](int i_v, int i_k) {
            const int j_v = i_v >> pair, j_k = i_k >> pair;
            const int head = it.head + (pair & i_k);              // i_v is i_k - 2 or none
            const int st = n % S::STAGES;
            ok = ok && (n < S::STAGES ||
                        p_wait(kv_empty(st), ((n / S::STAGES) - 1) & 1, abort_flag, err_flag));
            if (!ok) return;
            ++n;
            *tiles_loaded = n;
            const uint32_t dst = sb + S::OFF_RING + st * 2 * S::TILE;
            // V tiles with an edge land at the cleaning warp, which passes them on to the issuers
            const bool has_k = i_k < n_tiles, has_v = i_v >= 0, edge = has_v && j_v >= it.first_edge;
            const uint32_t bytes = (has_k ? S::TILE : 0) + (has_v && !edge ? S::TILE : 0);
            if (edge) mbar_expect_tx(edge_full(st), S::TILE);
            if (bytes)
              mbar_expect_tx(kv_full(st), bytes);
            else
              mbar_arrive(kv_full(st));
            if (!edge) mbar_arrive(kv_full(st));
            for (int b = 0; b < S::NB; ++b) {
              if (has_v)
                tma_load_3d(dst + b * KBLK, &tmV, 64 * b, head, it.k0 + j_v * TK,
                            edge ? edge_full(st) : kv_full(st));
              if (has_k)
                tma_load_3d(dst + S::TILE + b * KBLK, &tmK, 64 * b, head, it.k0 + j_k * TK, kv_full(st));
            }
          };
          for (int j = 0; j < min(S::NBUF, n_tiles); ++j) load(-1, j);
          for (int j = 0; j < n_tiles && ok; ++j) load(j, j + S::NBUF);
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (*abort_flag && lane == 0) {
        // give copies still in flight into this CTA's shared memory time to land
        const unsigned long long t0 = globaltimer();
        while (globaltimer() - t0 < 2000000ull) {
        }
      }
    } else if (warp < W_TMA) {
      // ---------------- MMA issuers, one for each query tile ----------------
      // The whole warp walks the loop, so that addresses and descriptors stay in uniform registers;
      // one lane's MMAs count. Each issuer's order of S and P V is that of its tile's chain.
      constexpr uint32_t idS = idesc_bf16(TQ, TK, false);
      constexpr uint32_t idO = idesc_bf16(TQ, D, true);
      auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, p_wait(bar, parity, abort_flag, err_flag)) != 0;
      };
      const int w = __shfl_sync(0xffffffffu, warp - W_MMA, 0);
      const uint32_t leader = elect_one();
      const uint64_t q_desc = desc_sw128(sb + w * S::QTILE);
      const uint64_t ring_k = desc_sw128(sb + S::OFF_RING + S::TILE);
      const uint64_t ring_v = D == 128 ? desc_mn_blocks(sb + S::OFF_RING, KBLK)
                                       : desc_sw128_mn(sb + S::OFF_RING);
      constexpr uint64_t STEP = 2 * S::TILE >> 4;     // of a stage, in descriptor units
      int ks = 0, k_phase = 0;       // ring stage and lap of the next tile
      auto advance = [&]() {
        if (++ks == S::STAGES) {
          ks = 0;
          k_phase ^= 1;
        }
      };
      int buf = 0;                   // score buffer and lap of the next key tile
      uint32_t lap = 0;
      uint32_t q_phase = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        ok = wait(item_full(i & 1), (i >> 1) & 1);
        if (!ok) break;
        const volatile Item* slot = &items[i & 1];
        const int valid = __shfl_sync(0xffffffffu, slot->valid, 0);
        const int nt = __shfl_sync(0xffffffffu, slot->nt[w], 0);
        const int pair = __shfl_sync(0xffffffffu, slot->pair, 0);
        const int n_tiles = __shfl_sync(0xffffffffu, max(slot->nt[0], slot->nt[1]), 0) << pair;
        if (lane == 0) mbar_arrive(item_empty(i & 1));
        __syncwarp();
        if (!valid) break;
        auto scores = [&](int j, int b) {
          const uint64_t kd = ring_k + ks * STEP;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            w_mma_ss(tS(w, b), q_desc + (uint64_t)((kk >> 2) * (BLK >> 4) + 2 * (kk & 3)),
                     kd + (uint64_t)((kk >> 2) * (KBLK >> 4) + 2 * (kk & 3)), idS, kk > 0, leader);
          w_commit(s_full(w, b), leader);
          if (j + 1 == nt) w_commit(q_empty(w), leader);
        };
        // the first scores, then P V of tile j and the scores of tile j + 2 in turn. Of a pair this
        // tile's are every other one, and its next scores, in the other buffer, come first
        int b0 = buf;
        for (int i2 = 0; i2 < min(S::NBUF, n_tiles) && ok; ++i2) {
          ok = wait(kv_full(ks), k_phase);
          if (ok && i2 == 0 && nt > 0) {
            ok = wait(q_full(w), q_phase);
            q_phase ^= 1;
          }
          if (!ok) break;
          tc_fence_after();
          if (pair ? i2 == w : i2 < nt) {
            scores(i2 >> pair, b0);
            b0 ^= 1;
          }
          w_commit(kv_empty(ks), leader);
          advance();
        }
        for (int i2 = 0; i2 < n_tiles && ok; ++i2) {
          const int b = buf, j = i2 >> pair;
          ok = wait(kv_full(ks), k_phase);
          if (ok && (pair ? (i2 & 1) == w : j < nt)) {
            if (pair && j + 1 < nt) {
              tc_fence_after();
              scores(j + 1, b ^ 1);
            }
            ok = wait(p_full(w, b), lap);
            if (!ok) break;
            tc_fence_after();
            const uint64_t vd = ring_v + ks * STEP;
#pragma unroll
            for (int kk = 0; kk < TK / 16; ++kk)
              w_mma_ts(tO(w), tS(w, b) + 8u * kk, vd + (uint64_t)(kk * (2048 >> 4)), idO,
                       (j > 0) || (kk > 0), leader);
            w_commit(pv_done(w, b), leader);
            if (!pair && j + 2 < nt) scores(j + 2, b);
            if (++buf == S::NBUF) {
              buf = 0;
              lap ^= 1;
            }
          }
          w_commit(kv_empty(ks), leader);
          advance();
        }
      }
      w_commit(teardown, leader);
      const unsigned long long t0 = globaltimer();
      while (!mbar_try_wait(teardown, 0) && globaltimer() - t0 < WAIT_LIMIT_NS) {
      }
    } else {
      // ---------------- cleaning of V in tiles where some row's limit ends ----------------
      int n0 = 0;
      uint32_t phase = 0;            // a bit for each stage
      bool ok = true;
      for (int i = 0; ok; ++i) {
        ok = __all_sync(0xffffffffu, p_wait<true>(item_full(i & 1), (i >> 1) & 1, abort_flag, err_flag));
        if (!ok) break;
        const Item it = items[i & 1];
        if (!it.valid) break;
        const int n_tiles = max(it.nt[0], it.nt[1]) << it.pair;
        bool found = false;
        for (int i2 = it.first_edge << it.pair; i2 < n_tiles && ok; ++i2) {
          const int j = i2 >> it.pair, st = (n0 + min(S::NBUF, n_tiles) + i2) % S::STAGES;
          ok = __all_sync(0xffffffffu, p_wait<true>(edge_full(st), (phase >> st) & 1, abort_flag, err_flag));
          if (!ok) break;
          phase ^= 1u << st;
          bool any = false;
#pragma unroll 1
          for (int row = lane; row < TK; row += 32) {   // thread = key
            uint8_t* v_row = smem + S::OFF_RING + st * 2 * S::TILE + row * 128;
            const bool behind = j * TK + row >= it.nk;
            uint32_t odd = 0;
            if (!behind) {
#pragma unroll 8
              for (int c = 0; c < D / 8; ++c) {
                const uint4 x = *reinterpret_cast<const uint4*>(v_row + (c >> 3) * KBLK + 16 * ((c & 7) ^ (row & 7)));
                odd |= ((x.x & 0x7f807f80u) + 0x00800080u) | ((x.y & 0x7f807f80u) + 0x00800080u) |
                       ((x.z & 0x7f807f80u) + 0x00800080u) | ((x.w & 0x7f807f80u) + 0x00800080u);
              }
              odd &= 0x80008000u;
            }
            if (behind || odd) {
              any = any || odd;
#pragma unroll 1
              for (int c = 0; c < D / 8; ++c) {
                uint4* at = reinterpret_cast<uint4*>(v_row + (c >> 3) * KBLK + 16 * ((c & 7) ^ (row & 7)));
                uint32_t x[4] = {0, 0, 0, 0};
                if (!behind) {
                  const uint4 y = *at;
                  x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    if ((x[k] & 0x7f80u) == 0x7f80u) x[k] &= 0xffff0000u;
                    if ((x[k] & 0x7f800000u) == 0x7f800000u) x[k] &= 0x0000ffffu;
                  }
                }
                *at = make_uint4(x[0], x[1], x[2], x[3]);
              }
            }
          }
          if (__any_sync(0xffffffffu, any)) {
            volatile Item* slot = &items[i & 1];
            if (lane == 0) {
              if (!found) slot->first_edge = j;
              slot->dirty = j + 1;
            }
            found = true;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(kv_full(st));
        }
        n0 += min(S::NBUF, n_tiles) + n_tiles;
        __syncwarp();
        if (lane == 0) mbar_arrive(item_empty(i & 1));
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
    // ---------------- softmax: thread = row ----------------
    const int w = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tOw = tO(w) + lane_off;
    const float scale_log2 = a.scale_log2;
    const int row_tok = row / a.group, row_head = row % a.group;
    uint8_t* const stage = smem + S::OFF_OUT + warp * 4096;
    // a warp goes on, or gives up, as one: what follows a wait are warp-wide instructions
    auto all_wait = [&](uint32_t bar, uint32_t parity) {
      return __all_sync(0xffffffffu, p_wait(bar, parity, abort_flag, err_flag)) != 0;
    };
    int buf = 0;           // score buffer and lap of the next key tile
    uint32_t lap = 0;
    // what the row does next: read ahead, while the last product of the item before it runs (the
    // producer hands an item over without waiting for the read-out of the one before)
    struct Ahead {
      bool valid, mine, active;
      int ntw, lim, lim_min;
    } next;
    auto look = [&](int i) {
      if (!all_wait(item_full(i & 1), (i >> 1) & 1)) return false;
      const Item it = items[i & 1];
      next.valid = it.valid;
      next.ntw = ((const volatile Item*)items)[i & 1].nt[w];
      const int tok = it.t0 + (it.pair ? 0 : w * span) + row_tok;   // within the sequence
      next.mine = row_tok < span && tok < it.nq;
      next.lim = next.mine ? limit_of(it, tok, a) : 0x7fffffff;
      next.lim_min = __reduce_min_sync(0xffffffffu, next.lim);
      next.active = __any_sync(0xffffffffu, next.mine);
      return true;
    };
    bool ok = look(0);
    for (int i = 0; ok; ++i) {
      if (!next.valid) break;
      const volatile Item* slot = &items[i & 1];
      const int ntw = next.ntw, lim = next.lim, lim_min = next.lim_min;
      const bool mine = next.mine, active = next.active;
      // scores of 32 keys from key0 on, those past the row's limit to -inf
      auto hide = [&](uint32_t (&r)[32], int key0) {
        if (key0 + 32 <= lim_min) return;                       // seen by all rows of the warp
        const int left = lim - key0;
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (c >= left) r[c] = __float_as_uint(-INFINITY);
      };
      float m = -INFINITY, l = 0.f;
      auto scores_of = [&](int b) { return tS(w, b) + lane_off; };
      auto ready = [&](int b, uint32_t phase) {
        const bool there = all_wait(s_full(w, b), phase);
        tc_fence_after();
        return there;
      };
      auto step_on = [&](int& b, uint32_t& phase) {
        if (++b == S::NBUF) {
          b = 0;
          phase ^= 1;
        }
      };
      int last_buf = 0;                  // of the tile before
      uint32_t last_lap = 0;
      auto tile = [&](int j) {
        const int b = buf;
        if (!ready(b, lap)) return false;
        uint32_t r[TK / 32][32];
#pragma unroll
        for (int q = 0; q < TK / 32; ++q) tmem_ld32_async(scores_of(b) + 32 * q, r[q]);
#pragma unroll
        for (int q = 0; q < TK / 32; ++q) tmem_wait(r[q]);
        float cmax = -INFINITY;
#pragma unroll
        for (int q = 0; q < TK / 32; ++q) {
          hide(r[q], j * TK + 32 * q);
          cmax = fmaxf(cmax, max32(r[q]));
        }
        // the exponent's reference moves only when the maximum grew by more than 2^8: the same
        // reference scales O and the sum, so the result is unchanged
        const bool bump = cmax > m && (m == -INFINITY || (cmax - m) * scale_log2 > 8.0f);
        if (__any_sync(0xffffffffu, bump)) {
          const float mnew = bump ? cmax : m;
          const float alpha = bump ? p_ex2((m - mnew) * scale_log2) : 1.f;
          m = mnew;
          l *= alpha;
          if (j > 0) {
            // the last product must be complete (those before it are: the issuer began this
            // tile's scores after them)
            if (!all_wait(pv_done(w, last_buf), last_lap)) return false;
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              uint32_t ov[32];
              tmem_ld32_async(tOw + 32 * q, ov);
              tmem_wait(ov);
#pragma unroll
              for (int c = 0; c < 32; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * alpha);
              tmem_st32(tOw + 32 * q, ov);
            }
          }
        }
        const float ms = m == -INFINITY ? 0.f : m * scale_log2;
        const unsigned long long sc2 = f2_pack(scale_log2, scale_log2), nms2 = f2_pack(-ms, -ms);
        unsigned long long sum2[2] = {0, 0};
        // P over the first columns of the scores, two keys a column
#pragma unroll
        for (int q = 0; q < TK / 32; ++q) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float2 e = f2_unpack(f2_fma(
                f2_pack(__uint_as_float(r[q][2 * c]), __uint_as_float(r[q][2 * c + 1])), sc2, nms2));
            const float p0 = p_ex2(e.x), p1 = p_ex2(e.y);
            sum2[c & 1] = f2_add(sum2[c & 1], f2_pack(p0, p1));
            const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
            pk[c] = *reinterpret_cast<const uint32_t*>(&h);
          }
          tmem_st16(scores_of(b) + 16 * q, pk);
        }
        const float2 sm = f2_unpack(f2_add(sum2[0], sum2[1]));
        l += sm.x + sm.y;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(w, b));
        last_buf = b;
        last_lap = lap;
        step_on(buf, lap);
        return true;
      };
      if (active) {
        for (int j = 0; j < ntw && ok; ++j) ok = tile(j);
      } else {
        for (int j = 0; j < ntw && ok; ++j) {   // none of the warp's rows is in use
          ok = ready(buf, lap);
          tc_fence_before();
          __syncwarp();
          if (lane == 0 && ok) mbar_arrive(p_full(w, buf));
          last_buf = buf;
          last_lap = lap;
          step_on(buf, lap);
        }
      }
      ok = ok && look(i + 1);
      if (!ok) break;
      if (ntw > 0) {
        ok = all_wait(pv_done(w, last_buf), last_lap);
        if (!ok) break;
        tc_fence_after();
      }
      if (active) {
        // the item is read again here: its fields need not live through the loop above
        const int pair = slot->pair, q0 = slot->q0, t0 = slot->t0 + (pair ? 0 : w * span);
        const int left = slot->nq - t0, head = slot->head + (pair & w);
        const bool empty = l == 0.f;
        const float inv = empty ? 0.f : p_rcp(l);                // 1 ulp, ahead of bf16
        const bool fix = ntw > 0 && slot->dirty != 0;
        // this lane stores 16 bytes of row 8 g + lane / 4 at a time: an offset each (-1: not a row)
        long long to[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int2 at = tile_rows[quarter * 32 + 8 * g + (lane >> 2)];
          to[g] = at.x < left ? ((long long)(q0 + t0) * a.q_heads + head * a.group + at.y) * D : -1;
        }
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          const int col = 32 * q;
          uint8_t* const buffer = stage + (q & 1) * 2048;   // two: one barrier a pass is enough
          uint32_t ov[32];
          if (ntw > 0) {
            tmem_ld32_async(tOw + 32 * q, ov);
            tmem_wait(ov);
          }
#pragma unroll
          for (int c = 0; c < 32; ++c)
            ov[c] = __float_as_uint(empty ? 0.f : __uint_as_float(ov[c]) * inv);
          if (fix) {
            // lane = column: a key's 32 in one load, 16 keys in flight. The keys up to the least limit,
            // added to the rows that have it, then on to the next limit
            const int last = mine ? min(lim, slot->dirty * TK) : 0;
            const bf16* column = a.v + (long long)slot->k0 * a.v_stride + (long long)head * D + col + lane;
            float odd = 0.f;             // sum of the column's values so far that are not finite
            for (int key = slot->first_edge * TK;;) {
              const int next = __reduce_min_sync(0xffffffffu, last > key ? last : 0x7fffffff);
              if (next == 0x7fffffff) break;
#pragma unroll 1
              for (; key + 16 <= next; key += 16) {
                float x[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) x[k] = __bfloat162float(column[(long long)(key + k) * a.v_stride]);
#pragma unroll
                for (int k = 0; k < 16; ++k) odd += fabsf(x[k]) < INFINITY ? 0.f : x[k];
                if ((key & 0x3ff0) == 0 && lane == 0) atomicAdd(keys_read, 1);
              }
#pragma unroll 1
              for (; key < next; ++key) {
                const float x = __bfloat162float(column[(long long)key * a.v_stride]);
                odd += fabsf(x) < INFINITY ? 0.f : x;
              }
              const uint32_t columns = __ballot_sync(0xffffffffu, odd != 0.f);
              if (columns == 0) continue;
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                const float x = __shfl_sync(0xffffffffu, odd, c);
                if (last == next && (columns >> c & 1)) ov[c] = __float_as_uint(__uint_as_float(ov[c]) + x);
              }
            }
          }
          // 32 columns at a time through shared memory: a row's 64 bytes then leave by four lanes
          // together
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(ov[8 * c + 2 * k]),
                                                             __uint_as_float(ov[8 * c + 2 * k + 1]));
              u[k] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(buffer + lane * 64 + 16 * (c ^ ((lane >> 1) & 3))) =
                make_uint4(u[0], u[1], u[2], u[3]);
          }
          __syncwarp();
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int rr = 8 * g + (lane >> 2), chunk = lane & 3;
            const uint4 x = *reinterpret_cast<const uint4*>(buffer + rr * 64 + 16 * (chunk ^ ((rr >> 1) & 3)));
            if (to[g] >= 0) *reinterpret_cast<uint4*>(a.out + to[g] + col + 8 * chunk) = x;
          }
        }
        if (mine && a.lse)
          a.lse[(long long)(q0 + t0 + row_tok) * a.q_heads + head * a.group + row_head] =
              empty ? -INFINITY
                    : ((m == -INFINITY ? 0.f : m * scale_log2) + log2f(l)) * 0.69314718055994531f;
      }
      // O is read out: the next item's first hand-over of P tells the issuer so
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(item_empty(i & 1));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
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
                          PArgs a, int* err_flag, int num_sms, cudaStream_t s) {
  using S = PShape<D>;
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t e = set_max_dynamic_smem((const void*)k_attention_packed<D>, S::SMEM, attr_done);
  if (e != cudaSuccess) return e;
  // lengths are on the device: an upper bound of the items
  const int sequences = a.batch < a.tokens_q ? a.batch : a.tokens_q;   // that are not empty
  const long long items = ((long long)a.tokens_q / (2 * a.per_tile) + sequences) * a.kv_heads;
  a.pairs = items >= PAIRS_FROM * num_sms;
  if (items > (1LL << 28)) return cudaErrorInvalidValue;   // taking them out may last a second
  k_attention_packed<D><<<(unsigned)items, P_THREADS, S::SMEM, s>>>(mq, mk, mv, a, err_flag);
  return cudaGetLastError();
}

}  // namespace

cudaError_t attention_packed(const bf16* q, long long q_stride, const bf16* k, long long k_stride,
                             const bf16* v, long long v_stride, int tokens_q, int tokens_k,
                             int batch, int q_heads, int kv_heads, int dim, const int* cu_q,
                             const int* cu_k, float scale, int frame, bf16* out, float* lse,
                             int* err_flag, int num_sms, cudaStream_t s) {
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
  a.pairs = 0;
  a.frame_inv = (1ull << 63) / (unsigned)frame + 1;
  a.scale_log2 = scale * 1.4426950408889634f;
  constexpr int box_keys = PShape<64>::TK;
  static_assert(box_keys == PShape<128>::TK, "one box for both");
  CUtensorMap mq, mk, mv;
  if (!make_map_heads(&mq, q, tokens_q, q_heads, dim, q_stride, a.per_tile, a.group) ||
      !make_map_heads(&mk, k, tokens_k, kv_heads, dim, k_stride, box_keys, 1) ||
      !make_map_heads(&mv, v, tokens_k, kv_heads, dim, v_stride, box_keys, 1))
    return cudaErrorInvalidValue;
  if (dim == 64) return launch_packed<64>(mq, mk, mv, a, err_flag, num_sms, s);
  if (dim == 128) return launch_packed<128>(mq, mk, mv, a, err_flag, num_sms, s);
  return cudaErrorInvalidValue;
}

}  // namespace jepa
