// Attention of a few new tokens per sequence over the 8-bit paged cache.
//
//   o[r] = sum_j softmax_j(scale q[r] . K[j]) V[j],  K[j] = ks[page] * code, V[j] = vs[page] * code
//
// for the rows r = (new token, head of the group) that share a key/value head. Bound by the HBM
// bytes of the codes (2 kv_heads * dim a cached token), so the codes go from shared memory
// straight into mma.sync fragments: e4m3 -> f16 is exact, 64 conversions a warp's 16 keys.
//   * The products are transposed, S^T = K Q^T and O^T = V^T P^T: codes are the 16-row operand and
//     query rows the 8-wide one, so that up to 8 rows (one new token, groups up to 8) cost 8 + 8
//     MMAs a 16-key step; 9 to 16 rows take two 8-wide tiles over the same converted codes. With
//     the query rows as the 16-row operand one row cost as much as 16, and issue, not HBM, was the
//     bound (two sequences of 100001 to 130001 tokens, 64 query heads over 8: 129 us).
//   * Work: items (sequence, head, tile of rows), each cut into units of 4 warps * KS keys.
//     All units of the call in one line are shared out evenly over the CTAs, so ragged lengths
//     and few long sequences fill the machine alike; an item that crosses CTAs leaves partial
//     (max, sum, output) rows in the workspace, which k_combine joins in a fixed order. Where all
//     sequences are short, items stay whole.
//   * A warp owns KS keys of each unit and its own ring of NST stages filled with cp.async
//     (zero-filled past the sequence's end, so stale codes there never meet the tensor cores).
//   * q is scaled per row by a power of two into f16's range; the exact scores are fp32. The
//     probabilities enter the second product as f16 (2^-12 relative, finer than bf16's 2^-9).
//   * Scores are exponentiated against a reference that moves only when the maximum grows by
//     more than 2^8, so that most steps leave the accumulators alone.
//   * Fragment layouts. A lane (g = lane / 4, t = lane % 4) takes bytes [t D/4, (t+1) D/4) of keys
//     g and g + 8 for K Q^T, and bytes [g D/8, (g+1) D/8) of keys 2t, 2t+1, 2t+8, 2t+9 for V^T P^T:
//     the order of the summed index is free, and so is the naming of output rows. Both are wide
//     loads without bank conflicts under the XOR swizzle (dim 64: two-way for V), and a lane ends
//     with D/8 consecutive outputs of two query rows.
// Measured, inputs behind L2: those two sequences 86 us (5.7 TB/s), 32 sequences of 100 to 8000
// tokens 57 us (4.9 TB/s), 256 of 776 tokens with 16 heads of 64 and two queries 87 us (4.7 TB/s),
// one of 517 tokens 10 us (latency). What is left of the copy rate is the start, the shares' uneven
// ends and the joining, 12 us of the first; heads of 64 are bound by issue: the load stream's state
// (keys left, the table's row, the head) is kept from step to step, a division for the head in
// each step took 5% there.
#include "decode_line.cuh"

namespace jepa {

namespace {

template <int D, int NR>
struct Shape {
  static constexpr int ROWS = 8 * NR;              // query rows of an item
  // cp.async stages of a warp and CTAs a SM. Narrow heads: four CTAs with two stages hide more of
  // a step's latency than three with three (256 candidates of 776 tokens: 6% less);
  // heads of 128 the other way round (two long sequences: 7% less). Two row tiles of 128
  // columns need 244 registers a thread and 82 KB, so two CTAs (32 sequences of up to 8000
  // tokens, 16 rows: 85 us; a quarter more with three CTAs of two stages, which spill).
  static constexpr int NST = D == 64 && NR == 1 ? 2 : 3;
  static constexpr int CTAS = D == 64 ? (NR == 1 ? 4 : 3) : (NR == 1 ? 3 : 2);
  static constexpr int KS = 2048 / D;              // keys a warp takes in a step
  static constexpr int GROUPS = KS / 16;           // 16-key groups of P V
  static constexpr int UNIT = WARPS * KS;          // keys of a unit
  static constexpr int KW = D / 16;                // 32-bit words of a key a lane takes
  static constexpr int VN = D / 8;                 // values of a V row a lane takes
  static constexpr int MT = D / 16;                // output tiles of 16 columns
  static constexpr int STAGE = 2 * KS * D;         // K and V codes
  static constexpr int OUT_LD = OUT_ROW<D>;
  static constexpr int OFF_SCALE = WARPS * NST * STAGE;
  static constexpr int OFF_OUT = OFF_SCALE + WARPS * NST * 16;
  static constexpr int SMEM = OFF_OUT + WARPS * ROWS * OUT_LD * 4;
  static_assert(CTAS <= MAX_CTAS_PER_SM && CTAS * (SMEM + 2048) <= 228 * 1024, "CTAs of a SM");
  static_assert(COMBINE_SMEM<D> * CTAS * MAX_SMS <= 48 * 1024, "what a launch may have without an attribute");
};

__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t w) {   // low 16 bits of w
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(h) : "r"(w));
  return h;
}
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2_hi(uint32_t w) {   // high 16 bits of w
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
      : "=r"(h) : "r"(w));
  return h;
}
__device__ __forceinline__ float sane_scale(float s) {
  return s >= KV8_SCALE_MIN ? fminf(s, KV8_SCALE_MAX) : KV8_SCALE_MIN;
}
// any e4m3 NaN (0x7f, 0xff) among the four codes of w
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

template <int D, int NR>
__global__ void __launch_bounds__(THREADS, (Shape<D, NR>::CTAS))
    k_attention_kv8(Kv8View c, Args a, int whole, int* err_flag) {
  using S = Shape<D, NR>;
  constexpr int ROWS = S::ROWS, NST = S::NST;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sm_m[WARPS][ROWS], sm_l[WARPS][ROWS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;");   // k_combine may be set up meanwhile
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * (NST * S::STAGE);
  const uint8_t* ring_ptr = smem + warp * (NST * S::STAGE);
  const uint32_t ring_sc =
      (uint32_t)__cvta_generic_to_shared(smem) + S::OFF_SCALE + warp * (NST * 16);
  const float* ring_sc_ptr = reinterpret_cast<const float*>(smem + S::OFF_SCALE) + warp * NST * 4;
  float* const sm_o = reinterpret_cast<float*>(smem + S::OFF_OUT);

  int* const flag0 = blockIdx.x == 0 ? err_flag : nullptr;
  long long u_begin, u_end, total = 0;
  int workers = 0;
  if (whole) {
    // items in equal numbers, a place each
    const long long items = (long long)c.batch * c.heads * a.tiles;
    u_begin = kv8_share(items, gridDim.x, blockIdx.x);
    u_end = kv8_share(items, gridDim.x, blockIdx.x + 1);
    if (flag0 && warp == 0) total_places(c, a, S::UNIT, flag0);   // reports lengths out of range
  } else {
    total = total_places(c, a, S::UNIT, flag0);
    workers = workers_of(total, gridDim.x);
    if ((int)blockIdx.x >= workers) {
      if (threadIdx.x == 0) a.split[blockIdx.x] = make_int4(0, 0, 0, 0);
      write_empty<D>(c, a);
      return;
    }
    u_begin = kv8_share(total, workers, blockIdx.x);
    u_end = kv8_share(total, workers, blockIdx.x + 1);
  }
  int4 begun = make_int4(0, 0, 0, 0);
  const int rows = a.q_tokens * a.group;
  // ---- loading: the warp's steps of all segments in one stream, NST - 1 ahead of their use ----
  constexpr int CPR = D / 16;                  // 16-byte chunks of a row
  constexpr int RPI = 32 / CPR;                // rows a warp copies in one instruction
  const int chunk = lane % CPR, sub = lane / CPR;
  Cursor load_cur{0, 0, 0, 0};
  Segment ld;
  int ld_left = 0, ld_stage = 0;               // steps left of the segment
  bool ld_more = plan<S::UNIT, ROWS>(c, a, whole, u_begin, u_end, load_cur, ld);
  // a lane's place in a 16-key group of codes, in global and (swizzled) in shared memory
  const uint32_t lane_from = sub * D + 16 * chunk;
  uint32_t lane_to[16 / RPI];
#pragma unroll
  for (int q = 0; q < 16 / RPI; ++q) {
    const int row = q * RPI + sub;
    lane_to[q] = ring + row * D + 16 * (D == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3));
  }
  const uint32_t block_bytes = (uint32_t)c.page * D, slot_mask = c.page - 1;
  int pg_next[S::GROUPS];                      // pages of the step that is issued next
  int ld_key = 0;                              // first key of that step
  const int* ld_pages = nullptr;               // the sequence's row of the table
  auto begin_segment = [&]() {
    ld_key = ld.k0 * S::UNIT + warp * S::KS;
    ld_pages = c.table + (long long)ld.s * c.max_pages;
    ld_left = ld.k1 - ld.k0;
  };
  if (ld_more) begin_segment();
  auto fetch_pages = [&]() {
    const int key = ld_key;
    const int* at = ld_pages;
#pragma unroll
    for (int p = 0; p < S::GROUPS; ++p)
      pg_next[p] = ld_more && key + 16 * p < ld.len ? __ldg(at + ((key + 16 * p) >> c.page_log2)) : -1;
  };
  auto issue = [&]() {                         // the next step of the stream into the next stage
    const int key0 = ld_key;
    if (ld_more && key0 < ld.len) {
      const uint32_t st = ld_stage * S::STAGE;
      bool whole_step = key0 + S::KS <= ld.len;
      uint32_t block[S::GROUPS];               // num_pages * heads is below 2^31
#pragma unroll
      for (int p = 0; p < S::GROUPS; ++p) {
        const bool there = (uint32_t)pg_next[p] < (uint32_t)c.num_pages;
        if (!there && key0 + 16 * p < ld.len && lane == 0) atomicOr(err_flag, DEV_ERR_INDEX);
        whole_step = whole_step && there;
        block[p] = (there ? (uint32_t)pg_next[p] : 0u) * (uint32_t)c.heads + (uint32_t)ld.head;
      }
#pragma unroll
      for (int p = 0; p < S::GROUPS; ++p) {
        const uint64_t from = (uint64_t)block[p] * block_bytes +
                              (((uint32_t)(key0 + 16 * p) & slot_mask) * D + lane_from);
        const uint8_t *fk = c.k + from, *fv = c.v + from;
        if (whole_step) {
#pragma unroll
          for (int q = 0; q < 16 / RPI; ++q) {
            cp16(lane_to[q] + st + 16 * p * D, fk + q * RPI * D, 16);
            cp16(lane_to[q] + st + 16 * p * D + S::KS * D, fv + q * RPI * D, 16);
          }
        } else {                               // keys past the end, or without a page, are zeros
          const int keys = (uint32_t)pg_next[p] < (uint32_t)c.num_pages ? ld.len - (key0 + 16 * p) : 0;
#pragma unroll
          for (int q = 0; q < 16 / RPI; ++q) {
            const uint32_t bytes = q * RPI + sub < keys ? 16 : 0;
            cp16(lane_to[q] + st + 16 * p * D, fk + q * RPI * D, bytes);
            cp16(lane_to[q] + st + 16 * p * D + S::KS * D, fv + q * RPI * D, bytes);
          }
        }
      }
      if (lane < 2 * S::GROUPS) {              // k, v scale of each group
        const int p = lane >> 1;
        const bool there =
            (uint32_t)(S::GROUPS == 1 || p == 0 ? pg_next[0] : pg_next[S::GROUPS - 1]) < (uint32_t)c.num_pages;
        cp4(ring_sc + ld_stage * 16 + lane * 4,
            ((lane & 1) ? c.v_scale : c.k_scale) + (p == 0 ? block[0] : block[S::GROUPS - 1]),
            there ? 4 : 0);
      }
    }
    cp_commit();
    ld_stage = ld_stage + 1 == NST ? 0 : ld_stage + 1;
    ld_key += S::UNIT;
    if (ld_more && --ld_left == 0) {
      ld_more = plan<S::UNIT, ROWS>(c, a, whole, ld.next, u_end, load_cur, ld);
      begin_segment();
    }
    fetch_pages();
  };
  fetch_pages();
#pragma unroll 1
  for (int i = 0; i < NST - 1; ++i) issue();

  int stage = 0;
  Cursor cur{0, 0, 0, 0};
  Segment sg;
  sg.next = u_begin;
  while (plan<S::UNIT, ROWS>(c, a, whole, sg.next, u_end, cur, sg)) {
    const int s = sg.s, len = sg.len;
    const int head = sg.head, r0 = sg.r0;
    Queries<D, NR> qr;
    qr.load(a, s, head, r0, rows, len);
    auto& qf = qr.qf;
    auto& qs = qr.qs;
    auto& lim = qr.lim;
    auto& lim_g = qr.lim_g;
    const int lim_min = qr.lim_min;

    float o[NR][S::MT][4];
    float m[NR][2], l[NR][2];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      m[nr][0] = m[nr][1] = -INFINITY;
      l[nr][0] = l[nr][1] = 0.f;
#pragma unroll
      for (int i = 0; i < S::MT; ++i) o[nr][i][0] = o[nr][i][1] = o[nr][i][2] = o[nr][i][3] = 0.f;
    }
    float vs_cur = 0.f;    // outputs are o * vs_cur; 0 before the first key

    for (int k = sg.k0; k < sg.k1; ++k) {
      cp_wait<NST - 2>();
      __syncwarp();
      issue();                         // into the stage that the step before this one has read
      const int key0 = k * S::UNIT + warp * S::KS;
      const uint8_t* kb = ring_ptr + stage * S::STAGE;
      const uint8_t* vb = kb + S::KS * D;
      const float* scales = ring_sc_ptr + stage * 4;
      stage = stage + 1 == NST ? 0 : stage + 1;
      if (key0 >= len) continue;

      // scores of keys g, g + 8 (c0 c1, c2 c3) and query rows 2t, 2t + 1
      float sc[S::GROUPS][NR][4];
#pragma unroll
      for (int p = 0; p < S::GROUPS; ++p) {
        uint32_t w[2][S::KW];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = 16 * p + 8 * h + g;
#pragma unroll
          for (int i4 = 0; i4 < S::KW / 4; ++i4) {
            const int ch = t * (S::KW / 4) + i4;
            const int sw = D == 128 ? ch ^ (row & 7) : ch ^ ((row >> 1) & 3);
            const uint4 x = *reinterpret_cast<const uint4*>(kb + row * D + 16 * sw);
            w[h][4 * i4] = x.x; w[h][4 * i4 + 1] = x.y; w[h][4 * i4 + 2] = x.z; w[h][4 * i4 + 3] = x.w;
          }
        }
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) sc[p][nr][0] = sc[p][nr][1] = sc[p][nr][2] = sc[p][nr][3] = 0.f;
#pragma unroll
        for (int q = 0; q < S::KW; ++q) {
          const uint32_t a0 = f16x2_of_e4m3x2(w[0][q]), a1 = f16x2_of_e4m3x2(w[1][q]);
          const uint32_t a2 = f16x2_of_e4m3x2_hi(w[0][q]), a3 = f16x2_of_e4m3x2_hi(w[1][q]);
#pragma unroll
          for (int nr = 0; nr < NR; ++nr)
            mma_f16(sc[p][nr], a0, a1, a2, a3, qf[nr][q][0], qf[nr][q][1]);
        }
      }
      const bool edge = key0 + S::KS > lim_min;   // some row does not see some key (warp-uniform)
      bool move = false;
      float top[NR][2];
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
        for (int p = 0; p < S::GROUPS; ++p) {
          const float ks = sane_scale(scales[2 * p]);
          const float f0 = qs[nr][0] * ks, f1 = qs[nr][1] * ks;
          sc[p][nr][0] *= f0; sc[p][nr][1] *= f1; sc[p][nr][2] *= f0; sc[p][nr][3] *= f1;
        }
        if (edge) {
#pragma unroll
          for (int p = 0; p < S::GROUPS; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key0 + 16 * p + 8 * (e >> 1) + g >= lim[nr][e & 1]) sc[p][nr][e] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(sc[0][nr][e], sc[0][nr][2 + e]);
#pragma unroll
          for (int p = 1; p < S::GROUPS; ++p) x = fmaxf(x, fmaxf(sc[p][nr][e], sc[p][nr][2 + e]));
          top[nr][e] = x;
          move = move || x > m[nr][e] + P_SLACK || (m[nr][e] == -INFINITY && x > -INFINITY);
        }
      }
      if (__any_sync(0xffffffffu, move)) {
        // the maxima over all keys of the step; the reference moves where it has to
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = top[nr][e];
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            const float mn = fmaxf(m[nr][e], x);
            const float al = mn == -INFINITY ? 1.f : ex2f(m[nr][e] - mn);
            m[nr][e] = mn;
            l[nr][e] *= al;
#pragma unroll
            for (int d = 0; d < S::MT; ++d) {
              o[nr][d][e] *= al;
              o[nr][d][2 + e] *= al;
            }
          }
      }
#pragma unroll
      for (int p = 0; p < S::GROUPS; ++p) {
        const float vs = sane_scale(scales[2 * p + 1]);
        float ratio = 1.f;
        if (vs != vs_cur) {
          ratio = vs_cur > 0.f ? vs / vs_cur : 2.f;
          if (!(ratio >= 0x1p-6f && ratio <= 1.f)) {
            // larger than the accumulators' unit, or far below it: move them (by 2^80 at most)
            const float f = vs_cur / vs;
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
              for (int d = 0; d < S::MT; ++d) {
                o[nr][d][0] *= f; o[nr][d][1] *= f; o[nr][d][2] *= f; o[nr][d][3] *= f;
              }
            vs_cur = vs;
            ratio = 1.f;
          }
        }
        uint32_t b[NR][2];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          float pr[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float mr = m[nr][e & 1];
            pr[e] = ex2f(sc[p][nr][e] - (mr == -INFINITY ? 0.f : mr - P_SHIFT));
            l[nr][e & 1] += pr[e];
          }
          if (ratio != 1.f) {
#pragma unroll
            for (int e = 0; e < 4; ++e) pr[e] *= ratio;
          }
          b[nr][0] = transposed(pack_f16(pr[0], pr[1]));
          b[nr][1] = transposed(pack_f16(pr[2], pr[3]));
        }
        // V rows 2t, 2t + 1, 2t + 8, 2t + 9 of the group, D/8 values each
        uint32_t w[4][S::VN / 4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = 16 * p + 2 * t + (k & 1) + 8 * (k >> 1);
          if (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(vb + row * D + 16 * (g ^ (row & 7)));
            w[k][0] = x.x; w[k][1] = x.y; w[k][S::VN / 4 - 2] = x.z; w[k][S::VN / 4 - 1] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(
                vb + row * D + 16 * ((g >> 1) ^ ((row >> 1) & 3)) + 8 * (g & 1));
            w[k][0] = x.x; w[k][1] = x.y;
          }
        }
        // A NaN in V reaches only rows that see its key: a product with a masked probability of
        // 0 would spread it. Rows can differ in what they see only at the causal edge.
        bool bad = false;
        if (edge) {
          uint32_t any = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int q = 0; q < S::VN / 4; ++q) any |= nan_codes(w[k][q]);
          bad = __any_sync(0xffffffffu, any != 0);
        }
        if (!bad) {
#pragma unroll
          for (int q = 0; q < S::VN / 4; ++q)
#pragma unroll
            for (int hb = 0; hb < 2; ++hb) {
              const uint32_t x = __byte_perm(w[0][q], w[1][q], hb ? 0x7362 : 0x5140);
              const uint32_t y = __byte_perm(w[2][q], w[3][q], hb ? 0x7362 : 0x5140);
              const uint32_t a0 = f16x2_of_e4m3x2(x), a1 = f16x2_of_e4m3x2_hi(x);
              const uint32_t a2 = f16x2_of_e4m3x2(y), a3 = f16x2_of_e4m3x2_hi(y);
#pragma unroll
              for (int nr = 0; nr < NR; ++nr)
                mma_f16(o[nr][2 * q + hb], a0, a1, a2, a3, b[nr][0], b[nr][1]);
            }
        } else {
          // second product: 1 where V is NaN, times 1 where a row sees the key
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) {
            uint32_t see[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int key = key0 + 16 * p + 8 * h + 2 * t;
              see[h] = pack_f16(key < lim_g[nr] ? 1.f : 0.f, key + 1 < lim_g[nr] ? 1.f : 0.f);
            }
#pragma unroll
            for (int q = 0; q < S::VN / 4; ++q)
#pragma unroll
              for (int hb = 0; hb < 2; ++hb) {
                uint32_t av[4], an[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {     // a0, a1: keys 2t..; a2, a3: keys 2t + 8..
                  const uint32_t sel = 0x40u + 0x11u * (2 * hb + (k & 1));
                  const uint32_t codes = __byte_perm(w[2 * (k >> 1)][q], w[2 * (k >> 1) + 1][q], sel) & 0xffffu;
                  const uint32_t nan = (nan_codes(codes) & 0x8080u) >> 7;   // 1 per NaN code
                  av[k] = f16x2_of_e4m3x2(codes & ~(nan * 0xffu));
                  an[k] = ((nan & 1u) ? 0x3c00u : 0u) | ((nan & 0x100u) ? 0x3c000000u : 0u);
                }
                float hit[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16(o[nr][2 * q + hb], av[0], av[1], av[2], av[3], b[nr][0], b[nr][1]);
                mma_f16(hit, an[0], an[1], an[2], an[3], see[0], see[1]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (hit[e] > 0.f) o[nr][2 * q + hb][e] = __int_as_float(0x7fc00000);
              }
          }
        }
      }
    }
    // ---- join the four warps ----
    __syncthreads();   // the joining before this one has been read
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[nr][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        const int row = 8 * nr + 2 * t + e;
        if (g == 0) {
          // from here on m is the exponent's reference; -inf only where no key was seen (scores
          // that are all NaN leave the maximum at -inf, but a NaN sum)
          sm_m[warp][row] = m[nr][e] != -INFINITY ? m[nr][e] - P_SHIFT : x == 0.f ? -INFINITY : 0.f;
          sm_l[warp][row] = x;
        }
        float* to = sm_o + (warp * ROWS + row) * S::OUT_LD + g * S::VN;
#pragma unroll
        for (int d = 0; d < S::MT; d += 2)   // tile d: columns 2d and 2d + 1 of the lane's
          *reinterpret_cast<float4*>(to + 2 * d) =
              make_float4(o[nr][d][e] * vs_cur, o[nr][d][2 + e] * vs_cur, o[nr][d + 1][e] * vs_cur,
                          o[nr][d + 1][2 + e] * vs_cur);
      }
    __syncthreads();
    join_warps<D, NR>(a, sg, rows, total, workers, sm_o, sm_m, sm_l, begun);
  }
  cp_wait<0>();
  if (whole) return;
  if (threadIdx.x == 0) a.split[blockIdx.x] = begun;
  write_empty<D>(c, a);
}

template <int D, int NR>
cudaError_t launch(const Kv8View& c, Args a, int* err_flag, int num_sms, cudaStream_t s) {
  using S = Shape<D, NR>;
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = set_max_dynamic_smem((const void*)k_attention_kv8<D, NR>, S::SMEM, attr_done);
  if (e != cudaSuccess) return e;
  a.tiles = (a.q_tokens * a.group + S::ROWS - 1) / S::ROWS;
  const long long max_len = (long long)c.max_pages << c.page_log2;
  const long long max_units = (max_len + S::UNIT - 1) / S::UNIT;
  const long long slots = (long long)(num_sms < MAX_SMS ? num_sms : MAX_SMS) * S::CTAS;
  const long long items = (long long)c.batch * c.heads * a.tiles;
  const int whole = max_units <= WHOLE_UNITS;
  // every SM's slots, or the work there can be if that is less
  const long long work = whole ? items : max_units > slots ? slots : items * max_units;
  const int grid = (int)(work < slots ? work : slots);
  k_attention_kv8<D, NR><<<grid, THREADS, S::SMEM, s>>>(c, a, whole, err_flag);
  if ((e = cudaGetLastError()) != cudaSuccess || whole) return e;
  return launch_combine<D, NR>(a, grid, s);
}

}  // namespace

size_t attention_kv8_workspace(int dim, int num_sms) {
  return notes_bytes(num_sms) + (size_t)num_sms * MAX_CTAS_PER_SM * 2 * 16 * (dim + 2) * sizeof(float);
}

cudaError_t attention_kv8(const Kv8View& c, const bf16* q, int q_tokens, int q_heads,
                          const int* kv_len, float scale, int causal, bf16* out, float* lse,
                          void* workspace, int* err_flag, int num_sms, cudaStream_t s) {
  Args a;
  a.q = q;
  a.kv_len = kv_len;
  a.out = out;
  a.lse = lse;
  a.split = (int4*)workspace;
  a.part = (float*)((uint8_t*)workspace + notes_bytes(num_sms));
  a.scale_log2 = scale * 1.4426950408889634f;
  a.q_tokens = q_tokens;
  a.q_heads = q_heads;
  a.group = q_heads / c.heads;
  a.tiles = 0;
  a.causal = causal;
  const bool narrow = q_tokens * a.group <= 8;
  if (c.dim == 64)
    return narrow ? launch<64, 1>(c, a, err_flag, num_sms, s) : launch<64, 2>(c, a, err_flag, num_sms, s);
  if (c.dim == 128)
    return narrow ? launch<128, 1>(c, a, err_flag, num_sms, s) : launch<128, 2>(c, a, err_flag, num_sms, s);
  return cudaErrorInvalidValue;
}

}  // namespace jepa
