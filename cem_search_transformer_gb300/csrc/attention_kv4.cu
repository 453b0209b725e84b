// Attention of a few new tokens per sequence over the 4-bit paged cache, and the weights that the
// cached tokens receive.
//
//   o[r] = sum_j w[r][j] V[j],  w[r][j] = softmax_j(scale q[r] . K[j]),  K, V = code * scale * unit
//   mass_out[j] = decay * mass[j] + sum_r w[r][j]
//
// for the rows r = (new token, head of the group) that share a key/value head. It cannot do without the HBM
// bytes of codes and scales (9/8 kv_heads * dim a cached token); what bounds it is issue (below). Line of work, joining, transposed
// products and the softmax are those of the attention over the 8-bit cache (attention_kv8.cu). What
// four bits change:
//   * Codes to fragments: e2m1 -> f16 two codes an instruction, then one packed product with the
//     block's e4m3 scale as f16: six significant bits, so exact. Four registers of a fragment of K are four
//     conversions and four products.
//   * A lane (g = lane / 4, t = lane % 4) takes elements [t D/4, (t+1) D/4) of keys g and g + 8 for K Q^T:
//     two blocks (dim 128) or one. For V^T P^T it takes elements [g D/8, (g+1) D/8), one block or half of one, of
//     keys 2t, 2t+1, 2t+8, 2t+9; the halves of their bytes are put together first (two keys of one
//     element in a byte), so that a conversion gives a register of the fragment.
//   * No scale varies within what a warp accumulates, as pages' scales do in 8 bits: the units
//     of a head multiply the scores and the outputs once.
//   * Queries and probabilities are f16, which is what the matrix instruction takes beside exact keys and values. A query
//     loses nothing (eight bits, scaled by its row); a probability's half step of 2^-11 is an eighth of the output's, and
//     the output's error against 64 bits grows by 0.5 to 1%. A weight is not rounded to f16: it is the fp32 exponential of
//     score - lse, where lse has been to natural units and back (errors of up to 2.3e-7 of it; 7e-8 without).
//   * The weights need the rows' sums, so their keys are read and multiplied a second time, by the same kernel
//     without values, once for each tile of query rows (64 rows of 32 sequences of 4000 tokens: 111 us; a tile's
//     queries loaded anew in each step instead 228). Holding the scores of short items in shared memory instead gained 1 to 7 us of 110
//     (256 candidates of 776 tokens) and cost every other call half a microsecond.
// Measured, inputs behind L2: two sequences of 100001 to 130001 tokens, 64 query heads over 8 of 128, 62 us
// (4.5 TB/s; the kernel alone 57, 0.73 of the copy rate); 32 of 100 to 8000 tokens 40 us; 16 of 4000 to 30000
// with weights 109 us, of which the weights' pass is 41; 256 of 776 tokens with 16 heads of 64, two queries and weights 107;
// one of 517 tokens 8 us (latency). Bound by issue: 64 conversions and 64 products a 16-key group of 128 columns
// share the SM's dispatch (a loop of the two alone issues 0.73 a cycle, this kernel 0.58 to 0.64), and no single part
// that is left out of it (copies, products, exponentials, scales) makes it more than an eighth faster.
#include "decode_line.cuh"

#include "kv4.cuh"

namespace jepa {

namespace {

// What a kernel does: attention with an item's keys shared by the four warps of a CTA, attention with an
// item a warp, or the weights (a place of the line a warp).
enum Kind { BY_CTA, BY_WARP, WEIGHTS };

template <int D, int NR, int KIND>
struct Shape {
  static constexpr int ROWS = 8 * NR;              // query rows of an item
  // Keys a warp takes in a step, cp.async stages of a warp and CTAs a SM. Heads of 64: steps of 64 keys in two
  // stages 76 us (256 of 776 tokens), of 32 in three 78; four groups side by side hide more of each other's
  // latency than turns of two (12% more). Heads of 128: three CTAs with three stages 57 us (the two long sequences),
  // four with two 59.
  static constexpr int KS = D == 64 && NR == 1 ? 64 : 32;
  static constexpr int NST = D == 64 && NR == 1 ? 2 : 3;
  static constexpr int CTAS = (D == 64 ? 4 : 3) - (NR == 2);
  static constexpr int GROUPS = KS / 16;           // 16-key groups
  static constexpr int SHARERS = KIND == BY_CTA ? WARPS : 1;   // warps that share an item's keys
  static constexpr int UNIT = SHARERS * KS;        // keys of a unit
  static constexpr int KB = D / 2, SB = D / 16;    // bytes of a key's codes, and of its scales
  static constexpr int KW = D / 32;                // 32-bit words of a key a lane takes
  static constexpr int VW = D / 64;                // 32-bit words of a V row a lane takes
  static constexpr int KINDS = KIND == WEIGHTS ? 1 : 2;        // K, or K and V
  static constexpr int OFF_V = KS * KB, OFF_SC = KINDS * KS * KB;   // of a stage: K, V codes, K, V scales
  static constexpr int STAGE = OFF_SC + KINDS * KS * SB;
  static constexpr int OUT_LD = OUT_ROW<D>;
  static constexpr int OFF_OUT = WARPS * NST * STAGE;
  static constexpr int SMEM = OFF_OUT + (KIND == BY_CTA ? WARPS * ROWS * OUT_LD * 4 : 0);
  static_assert(2 * KS * SB / 16 <= 32, "a step's scales are a chunk a lane at most");
  static_assert(CTAS <= MAX_CTAS_PER_SM && CTAS * (SMEM + 2048) <= 228 * 1024, "CTAs of a SM");
  static_assert(COMBINE_SMEM<D> * CTAS * MAX_SMS <= 48 * 1024, "what a launch may have without an attribute");
};

// Byte of 16-byte chunk `chunk` of key `row` among a stage's codes. Lines of 128 bytes hold 2 keys (dim
// 128) or 4; the XOR spreads the rows 2t, t = 0..3, that a load of V takes over the banks.
template <int D>
__device__ __forceinline__ uint32_t code_at(int row, int chunk) {
  if (D == 128) return (row >> 1) * 128 + 16 * (((row & 1) * 4 + chunk) ^ (((row >> 1) & 3) << 1));
  return (row >> 2) * 128 + 16 * (((row & 3) * 2 + chunk) ^ (((row >> 2) & 1) << 1));
}

// x[i] of an array in registers.
template <class T, int N>
__device__ __forceinline__ T pick(const T (&x)[N], int i) {
  T y = x[0];
#pragma unroll
  for (int k = 1; k < N; ++k)
    if (i == k) y = x[k];
  return y;
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&y);
}

// Fragments of a 16-key group of K (keys g and g + 8 of this lane): words w[h][i] with the scales
// sc[h][b], both halves alike.
template <int D, int NR>
__device__ __forceinline__ void scores_of(const uint32_t (&w)[2][D / 32], const uint32_t (&sc)[2][D / 64],
                                          const uint32_t (&qf)[NR][D / 16][2], float (&s)[NR][4]) {
#pragma unroll
  for (int nr = 0; nr < NR; ++nr) s[nr][0] = s[nr][1] = s[nr][2] = s[nr][3] = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const uint32_t s0 = sc[0][i / 2], s1 = sc[1][i / 2];
    const uint32_t a0 = mul2(f16x2_of_e2m1x2<0>(w[0][i]), s0), a1 = mul2(f16x2_of_e2m1x2<0>(w[1][i]), s1);
    const uint32_t a2 = mul2(f16x2_of_e2m1x2<1>(w[0][i]), s0), a3 = mul2(f16x2_of_e2m1x2<1>(w[1][i]), s1);
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) mma_f16(s[nr], a0, a1, a2, a3, qf[nr][2 * i][0], qf[nr][2 * i][1]);
    const uint32_t b0 = mul2(f16x2_of_e2m1x2<2>(w[0][i]), s0), b1 = mul2(f16x2_of_e2m1x2<2>(w[1][i]), s1);
    const uint32_t b2 = mul2(f16x2_of_e2m1x2<3>(w[0][i]), s0), b3 = mul2(f16x2_of_e2m1x2<3>(w[1][i]), s1);
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
      mma_f16(s[nr], b0, b1, b2, b3, qf[nr][2 * i + 1][0], qf[nr][2 * i + 1][1]);
  }
}

// A lane's D / 64 scales of one key, each in both halves of a register, from their bytes.
template <int D>
__device__ __forceinline__ void key_scales(uint32_t bytes, uint32_t (&sc)[D / 64]) {
  const uint32_t x = f16x2_of_e4m3_pair(bytes);
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tmov.b32 %0, {lo, lo};\n\t}" : "=r"(sc[0]) : "r"(x));
  if (D == 128)
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tmov.b32 %0, {hi, hi};\n\t}" : "=r"(sc[D / 64 - 1]) : "r"(x));
}

// Scores are raw products times qs, and masked ones -inf before that: qs stays positive and finite.
template <int D, int NR>
__device__ __forceinline__ void scale_queries(Queries<D, NR>& qr, float unit) {
#pragma unroll
  for (int nr = 0; nr < NR; ++nr)
#pragma unroll
    for (int e = 0; e < 2; ++e) qr.qs[nr][e] = fminf(fmaxf(qr.qs[nr][e] * unit, 0x1p-126f), 0x1.fffffep127f);
}

template <int D, int NR, int KIND>
__global__ void __launch_bounds__(THREADS, (Shape<D, NR, KIND>::CTAS))
    k_attention_kv4(Kv4View c, Args a, MassArgs ma, int whole, int* err_flag) {
  using S = Shape<D, NR, KIND>;
  constexpr int ROWS = S::ROWS, NST = S::NST;
  [[maybe_unused]] constexpr int MT = D / 16;          // output tiles of 16 columns
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // worker of the line: the CTA, or the warp
  const int worker = KIND == BY_CTA ? blockIdx.x : blockIdx.x * WARPS + warp;
  const int first_key = KIND == BY_CTA ? warp * S::KS : 0;      // of this warp in a unit
  asm volatile("griddepcontrol.launch_dependents;");   // what comes next may be set up meanwhile
  asm volatile("griddepcontrol.wait;" ::: "memory");   // what the call before writes is there
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * (NST * S::STAGE);
  const uint8_t* ring_ptr = smem + warp * (NST * S::STAGE);

  int* const flag0 = KIND != WEIGHTS && blockIdx.x == 0 ? err_flag : nullptr;
  const int most = KIND == BY_CTA ? gridDim.x : gridDim.x * WARPS;
  long long u_begin, u_end, total = 0;
  int workers = most;
  if (whole) {
    // items in equal numbers, a place each
    const long long items = (long long)c.batch * c.heads * a.tiles;
    u_begin = kv8_share(items, most, worker);
    u_end = kv8_share(items, most, worker + 1);
    if (flag0 && warp == 0) total_places(c, a, S::UNIT, flag0);   // reports lengths out of range
  } else {
    total = total_places(c, a, S::UNIT, flag0);
    workers = workers_of(total, most);
    if (worker >= workers) {
      if (KIND == BY_CTA) {
        if (threadIdx.x == 0) a.split[blockIdx.x] = make_int4(0, 0, 0, 0);
        write_empty<D>(c, a);
      }
      return;
    }
    u_begin = kv8_share(total, workers, worker);
    u_end = kv8_share(total, workers, worker + 1);
  }
  [[maybe_unused]] int4 begun = make_int4(0, 0, 0, 0);
  const int rows = a.q_tokens * a.group;
  // ---- loading: the warp's steps of all segments in one stream, NST - 1 ahead of their use ----
  constexpr int CPR = S::KB / 16;              // 16-byte chunks of a key's codes
  constexpr int RPI = 32 / CPR;                // keys a warp copies in one instruction
  constexpr int SPG = D / 16;                  // 16-byte chunks of a group's scales (16 keys)
  constexpr int KPC = 16 / S::SB;              // keys of such a chunk
  const int chunk = lane % CPR, sub = lane / CPR;
  Cursor load_cur{0, 0, 0, 0};
  Segment ld;
  // row tiles of an item of the weights: its keys are gone through once for each
  [[maybe_unused]] const int tiles = KIND == WEIGHTS ? (rows + ROWS - 1) / ROWS : 1;
  [[maybe_unused]] int ld_tile = 0;
  int ld_left = 0, ld_stage = 0;               // steps left of the segment
  bool ld_more = plan<S::UNIT, ROWS>(c, a, whole, u_begin, u_end, load_cur, ld);
  uint32_t lane_to[16 / RPI];                  // of a lane's chunks of a 16-key group
#pragma unroll
  for (int q = 0; q < 16 / RPI; ++q) lane_to[q] = ring + code_at<D>(q * RPI + sub, chunk);
  const uint32_t lane_from = sub * S::KB + 16 * chunk;
  // scales of a step: lane -> (K or V, group, chunk of the group)
  const int sc_chunk = lane % SPG, sc_group = lane / SPG % S::GROUPS, sc_v = lane / SPG / S::GROUPS;
  const uint32_t sc_to = ring + S::OFF_SC + lane * 16;
  const uint32_t slot_mask = c.page - 1;
  int pg_next[S::GROUPS];                      // pages of the step that is issued next
  int ld_key = 0;                              // first key of that step
  const int* ld_pages = nullptr;               // the sequence's row of the table
  auto begin_segment = [&]() {
    ld_key = ld.k0 * S::UNIT + first_key;
    ld_pages = c.table + (long long)ld.s * c.max_pages;
    ld_left = ld.k1 - ld.k0;
  };
  if (ld_more) begin_segment();
  auto fetch_pages = [&]() {
    const int key = ld_key;
    const int* at = ld_pages;
#pragma unroll
    for (int p = 0; p < S::GROUPS; ++p)
      pg_next[p] = ld_more && key + 16 * p < ld.len ? at[(key + 16 * p) >> c.page_log2] : -1;
  };
  auto issue = [&]() {                         // the next step of the stream into the next stage
    const int key0 = ld_key;
    if (ld_more && key0 < ld.len) {
      const uint32_t st = ld_stage * S::STAGE;
      uint64_t row[S::GROUPS];                 // of the group's first key among all blocks' keys
      bool inside = key0 + S::KS <= ld.len;
#pragma unroll
      for (int p = 0; p < S::GROUPS; ++p) {
        const bool there = (uint32_t)pg_next[p] < (uint32_t)c.num_pages;
        inside = inside && there;
        const uint32_t block = (there ? (uint32_t)pg_next[p] : 0u) * (uint32_t)c.heads + (uint32_t)ld.head;
        row[p] = ((uint64_t)block << c.page_log2) + ((uint32_t)(key0 + 16 * p) & slot_mask);
      }
      const uint8_t* const scales = (sc_v ? c.v_scale : c.k_scale) + 16 * sc_chunk;
      if (inside) {
#pragma unroll
        for (int p = 0; p < S::GROUPS; ++p) {
          const uint64_t from = row[p] * S::KB + lane_from;
          const uint8_t *fk = c.k + from, *fv = c.v + from;
#pragma unroll
          for (int q = 0; q < 16 / RPI; ++q) {
            cp16(lane_to[q] + st + 16 * p * S::KB, fk + q * RPI * S::KB, 16);
            if (S::KINDS == 2) cp16(lane_to[q] + st + 16 * p * S::KB + S::OFF_V, fv + q * RPI * S::KB, 16);
          }
        }
        if (lane < S::KINDS * S::GROUPS * SPG)
          cp16(sc_to + st, scales + pick(row, sc_group) * S::SB, 16);
      } else {                                 // keys past the end, or without a page, are zeros
        int keys[S::GROUPS];
#pragma unroll
        for (int p = 0; p < S::GROUPS; ++p) {
          const bool there = (uint32_t)pg_next[p] < (uint32_t)c.num_pages;
          const int left = ld.len - (key0 + 16 * p);
          if (!there && left > 0 && lane == 0) atomicOr(err_flag, DEV_ERR_INDEX);
          keys[p] = there ? max(0, min(16, left)) : 0;
          const uint64_t from = row[p] * S::KB + lane_from;
          const uint8_t *fk = c.k + from, *fv = c.v + from;
#pragma unroll
          for (int q = 0; q < 16 / RPI; ++q) {
            const uint32_t bytes = q * RPI + sub < keys[p] ? 16 : 0;
            cp16(lane_to[q] + st + 16 * p * S::KB, fk + q * RPI * S::KB, bytes);
            if (S::KINDS == 2) cp16(lane_to[q] + st + 16 * p * S::KB + S::OFF_V, fv + q * RPI * S::KB, bytes);
          }
        }
        if (lane < S::KINDS * S::GROUPS * SPG) {
          const int n = pick(keys, sc_group) - sc_chunk * KPC;
          cp16(sc_to + st, scales + pick(row, sc_group) * S::SB, max(0, min(KPC, n)) * S::SB);
        }
      }
    }
    cp_commit();
    ld_stage = ld_stage + 1 == NST ? 0 : ld_stage + 1;
    ld_key += S::UNIT;
    if (ld_more && --ld_left == 0) {
      if (KIND != WEIGHTS || ++ld_tile == tiles) {
        ld_more = plan<S::UNIT, ROWS>(c, a, whole, ld.next, u_end, load_cur, ld);
        ld_tile = 0;
      }
      begin_segment();                         // of the next, or again for the next tile of rows
    }
    fetch_pages();
  };
  fetch_pages();
#pragma unroll 1
  for (int i = 0; i < NST - 1; ++i) issue();

  // where a lane reads in a stage: key g; V row 2t (row 2t + 1 lies in the same line); their scales. Eight
  // keys further on is a fixed distance on.
  const uint32_t at_k = D == 128 ? code_at<D>(g, t) : code_at<D>(g, t >> 1) + 8 * (t & 1);
  const uint32_t at_v = S::OFF_V + (D == 128 ? code_at<D>(2 * t, g >> 1) + 8 * (g & 1) : code_at<D>(2 * t, g >> 2) + 4 * (g & 3));
  const uint32_t at_v1 = S::OFF_V + (D == 128 ? code_at<D>(2 * t + 1, g >> 1) + 8 * (g & 1) : code_at<D>(2 * t + 1, g >> 2) + 4 * (g & 3));
  const uint32_t at_ks = S::OFF_SC + g * S::SB + (D == 128 ? 2 * t : t);
  const uint32_t at_vs = S::OFF_SC + S::KS * S::SB + 2 * t * S::SB + (D == 128 ? g : g >> 1);
  // scores of a stage's 16-key group p: keys g, g + 8 (c0 c1, c2 c3) and query rows 2t, 2t + 1
  auto scores = [&](const uint8_t* kb, int p, const Queries<D, NR>& qr, float (&x)[NR][4]) {
    uint32_t w[2][S::KW], f[2][S::VW];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = 16 * p + 8 * h;
      if (D == 128) {
        const uint4 y = *reinterpret_cast<const uint4*>(kb + at_k + row * S::KB);
        w[h][0] = y.x; w[h][1] = y.y; w[h][S::KW - 2] = y.z; w[h][S::KW - 1] = y.w;
        key_scales<D>(*reinterpret_cast<const uint16_t*>(kb + at_ks + row * S::SB), f[h]);
      } else {
        const uint2 y = *reinterpret_cast<const uint2*>(kb + at_k + row * S::KB);
        w[h][0] = y.x; w[h][1] = y.y;
        key_scales<D>(kb[at_ks + row * S::SB], f[h]);
      }
    }
    scores_of<D, NR>(w, f, qr.qf, x);
  };
  int stage = 0;
  Cursor cur{0, 0, 0, 0};
  Segment sg;
  sg.next = u_begin;
  while (plan<S::UNIT, ROWS>(c, a, whole, sg.next, u_end, cur, sg)) {
    const int s = sg.s, len = sg.len;
    const int head = sg.head, r0 = sg.r0;
    Queries<D, NR> qr;
    const float k_unit = kv4_unit(c.k_unit, head);
    if constexpr (KIND == WEIGHTS) {
      const long long at = ((long long)s * c.heads + head) * ((long long)c.max_pages << c.page_log2);
      float norm[NR][2];                       // lse in base 2 of rows 2t, 2t + 1
      bool full = false;                       // no row of the tile lies behind the last
      auto load_rows = [&](int first) {
        qr.load(a, s, head, first, rows, len);
        scale_queries(qr, k_unit);
        full = first + ROWS <= rows;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = first + 8 * nr + 2 * t + e;
            norm[nr][e] = r < rows ? a.lse[row_at(a, s, head, r)] * 1.4426950408889634f : 0.f;
            if (r >= rows) qr.lim[nr][e] = 0;  // no weight
          }
      };
      for (int tile = 0; tile < tiles; ++tile) {
        load_rows(tile * ROWS);
        // what a key has so far: from the call's input, then from the tiles before, by the same lane
        const float* const before = tile ? ma.out : ma.mass;
        const float decay = tile ? 1.f : ma.decay;
        for (int k = sg.k0; k < sg.k1; ++k) {
          const int key0 = k * S::UNIT;
          // This lane writes keys (16 p + 8 h + g) of its share of the pairs (p, h): with four groups p = t, with
          // two p = t / 2 and h = t % 2. What they had is loaded ahead of its use.
          constexpr int OWN = S::GROUPS / 2;
          float old[OWN];
#pragma unroll
          for (int j = 0; j < OWN; ++j) {
            const int key = key0 + (OWN == 2 ? 16 * t + 8 * j : 8 * t) + g;
            old[j] = before && key < len ? before[at + key] : 0.f;
          }
          cp_wait<NST - 2>();
          __syncwarp();
          issue();
          const uint8_t* kb = ring_ptr + stage * S::STAGE;
          stage = stage + 1 == NST ? 0 : stage + 1;
          float sum[S::GROUPS][2];
#pragma unroll
          for (int p = 0; p < S::GROUPS; ++p) sum[p][0] = sum[p][1] = 0.f;
          const bool inside = full && key0 + S::KS <= qr.lim_min;   // every row sees every key (warp-uniform)
#pragma unroll
          for (int p = 0; p < S::GROUPS; ++p) {
            float x[NR][4];
            scores(kb, p, qr, x);
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float y = ex2f(fmaf(x[nr][e], qr.qs[nr][e & 1], -norm[nr][e & 1]));
                if (inside || key0 + 16 * p + 8 * (e >> 1) + g < qr.lim[nr][e & 1]) sum[p][e >> 1] += y;
              }
          }
          // sums over the four lanes t of a key, each of which ends with its share: half of the values go
          // to the lane 2 away and half of what is left to the neighbour
          float half[S::GROUPS];                 // pairs (p, h) in order, those of this lane's half
#pragma unroll
          for (int i = 0; i < S::GROUPS; ++i) {
            const float lo = sum[i / 2][i & 1], hi = sum[(S::GROUPS + i) / 2][i & 1];
            half[i] = ((t & 2) ? hi : lo) + __shfl_xor_sync(0xffffffffu, (t & 2) ? lo : hi, 2);
          }
#pragma unroll
          for (int j = 0; j < OWN; ++j) {
            const float lo = half[j], hi = half[OWN + j];
            const float x = ((t & 1) ? hi : lo) + __shfl_xor_sync(0xffffffffu, (t & 1) ? lo : hi, 1);
            const int key = key0 + (OWN == 2 ? 16 * t + 8 * j : 8 * t) + g;
            if (key < len) ma.out[at + key] = before ? fmaf(decay, old[j], x) : x;
          }
        }
      }
    } else {
      qr.load(a, s, head, r0, rows, len);
      scale_queries(qr, k_unit);
      float o[NR][MT][4];
      float m[NR][2], ref[NR][2], l[NR][2];        // ref: m - P_SHIFT, 0 before the first key
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        m[nr][0] = m[nr][1] = -INFINITY;
        ref[nr][0] = ref[nr][1] = 0.f;
        l[nr][0] = l[nr][1] = 0.f;
#pragma unroll
        for (int i = 0; i < MT; ++i) o[nr][i][0] = o[nr][i][1] = o[nr][i][2] = o[nr][i][3] = 0.f;
      }

      for (int k = sg.k0; k < sg.k1; ++k) {
        cp_wait<NST - 2>();
        __syncwarp();
        issue();                         // into the stage that the step before this one has read
        const int key0 = k * S::UNIT + first_key;
        const uint8_t* kb = ring_ptr + stage * S::STAGE;
        stage = stage + 1 == NST ? 0 : stage + 1;
        if (key0 >= len) continue;

        float sc[S::GROUPS][NR][4];
#pragma unroll
        for (int p = 0; p < S::GROUPS; ++p) scores(kb, p, qr, sc[p]);
        const bool edge = key0 + S::KS > qr.lim_min;   // some row does not see some key (warp-uniform)
        bool move = false;
        float top[NR][2];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          if (edge) {
#pragma unroll
            for (int p = 0; p < S::GROUPS; ++p)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (key0 + 16 * p + 8 * (e >> 1) + g >= qr.lim[nr][e & 1]) sc[p][nr][e] = -INFINITY;
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(sc[0][nr][e], sc[0][nr][2 + e]);
#pragma unroll
            for (int p = 1; p < S::GROUPS; ++p) x = fmaxf(x, fmaxf(sc[p][nr][e], sc[p][nr][2 + e]));
            top[nr][e] = x * qr.qs[nr][e];
            move = move || top[nr][e] > m[nr][e] + P_SLACK;   // a first score is larger than -inf
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
              ref[nr][e] = mn == -INFINITY ? 0.f : mn - P_SHIFT;
              l[nr][e] *= al;
#pragma unroll
              for (int d = 0; d < MT; ++d) {
                o[nr][d][e] *= al;
                o[nr][d][2 + e] *= al;
              }
            }
        }
#pragma unroll
        for (int p = 0; p < S::GROUPS; ++p) {
          uint32_t b[NR][2];
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) {
            float pr[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              pr[e] = ex2f(fmaf(sc[p][nr][e], qr.qs[nr][e & 1], -ref[nr][e & 1]));
              l[nr][e & 1] += pr[e];
            }
            b[nr][0] = transposed(pack_f16(pr[0], pr[1]));
            b[nr][1] = transposed(pack_f16(pr[2], pr[3]));
          }
          // V rows 2t, 2t + 1, 2t + 8, 2t + 9 of the group, D/8 values each, and their scales
          uint32_t w[4][S::VW], vs[4];
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {
            const int row = 16 * p + 8 * (k4 >> 1);
            const uint8_t* from = kb + ((k4 & 1) ? at_v1 : at_v) + row * S::KB;
            if (D == 128) {
              const uint2 x = *reinterpret_cast<const uint2*>(from);
              w[k4][0] = x.x; w[k4][S::VW - 1] = x.y;
            } else {
              w[k4][0] = *reinterpret_cast<const uint32_t*>(from);
            }
            vs[k4] = kb[at_vs + (row + (k4 & 1)) * S::SB];
          }
          // A block that reads as NaN reaches only rows that see its key: a product with a masked
          // probability of 0 would spread it. Rows can differ in what they see only at the causal edge.
          uint32_t nan = 0;                      // bit k4: this lane's block of key k4 is NaN
          if (edge) {
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4)
              if ((vs[k4] & 0x7fu) == 0x7fu) {
                nan |= 1u << k4;
                vs[k4] = 0;
              }
          }
          const uint32_t sa = f16x2_of_e4m3_pair(vs[0] | (vs[1] << 8)), sb = f16x2_of_e4m3_pair(vs[2] | (vs[3] << 8));
#pragma unroll
          for (int q = 0; q < S::VW; ++q) {
            // bytes (even element of the first key, of the second), and the odd elements
            const uint32_t x0 = (w[0][q] & 0x0f0f0f0fu) | ((w[1][q] << 4) & 0xf0f0f0f0u);
            const uint32_t x1 = ((w[0][q] >> 4) & 0x0f0f0f0fu) | (w[1][q] & 0xf0f0f0f0u);
            const uint32_t y0 = (w[2][q] & 0x0f0f0f0fu) | ((w[3][q] << 4) & 0xf0f0f0f0u);
            const uint32_t y1 = ((w[2][q] >> 4) & 0x0f0f0f0fu) | (w[3][q] & 0xf0f0f0f0u);
            auto tile = [&](int d, uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3) {
              const uint32_t a0 = mul2(c0, sa), a1 = mul2(c1, sa), a2 = mul2(c2, sb), a3 = mul2(c3, sb);
#pragma unroll
              for (int nr = 0; nr < NR; ++nr) mma_f16(o[nr][d], a0, a1, a2, a3, b[nr][0], b[nr][1]);
            };
            tile(4 * q, f16x2_of_e2m1x2<0>(x0), f16x2_of_e2m1x2<0>(x1), f16x2_of_e2m1x2<0>(y0), f16x2_of_e2m1x2<0>(y1));
            tile(4 * q + 1, f16x2_of_e2m1x2<1>(x0), f16x2_of_e2m1x2<1>(x1), f16x2_of_e2m1x2<1>(y0), f16x2_of_e2m1x2<1>(y1));
            tile(4 * q + 2, f16x2_of_e2m1x2<2>(x0), f16x2_of_e2m1x2<2>(x1), f16x2_of_e2m1x2<2>(y0), f16x2_of_e2m1x2<2>(y1));
            tile(4 * q + 3, f16x2_of_e2m1x2<3>(x0), f16x2_of_e2m1x2<3>(x1), f16x2_of_e2m1x2<3>(y0), f16x2_of_e2m1x2<3>(y1));
          }
          if (edge && __any_sync(0xffffffffu, nan != 0)) {
            // how many NaN blocks of a lane's elements each row sees
            const uint32_t n0 = ((nan & 1u) ? 0x3c00u : 0u) | ((nan & 2u) ? 0x3c000000u : 0u);
            const uint32_t n1 = ((nan & 4u) ? 0x3c00u : 0u) | ((nan & 8u) ? 0x3c000000u : 0u);
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
              uint32_t see[2];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int key = key0 + 16 * p + 8 * h + 2 * t;
                see[h] = pack_f16(key < qr.lim_g[nr] ? 1.f : 0.f, key + 1 < qr.lim_g[nr] ? 1.f : 0.f);
              }
              float hit[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(hit, n0, n0, n1, n1, see[0], see[1]);
#pragma unroll
              for (int d = 0; d < MT; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (hit[e] > 0.f) o[nr][d][e] = __int_as_float(0x7fc00000);
            }
          }
        }
      }
      const float unit = kv4_unit(c.v_unit, head);
      if constexpr (KIND == BY_WARP) {
        // ---- the warp has all of the item ----
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = l[nr][e];
            x += __shfl_xor_sync(0xffffffffu, x, 4);
            x += __shfl_xor_sync(0xffffffffu, x, 8);
            x += __shfl_xor_sync(0xffffffffu, x, 16);
            const int r = r0 + 8 * nr + 2 * t + e;
            if (r >= rows) continue;
            const bool none = m[nr][e] == -INFINITY && x == 0.f;   // no key was seen (scores of NaN: a NaN sum)
            const float f = none ? 0.f : unit / x;
            const long long at = row_at(a, s, head, r);
            uint32_t w[MT];
#pragma unroll
            for (int d = 0; d < MT; ++d) {
              const __nv_bfloat162 y = __floats2bfloat162_rn(o[nr][d][e] * f, o[nr][d][2 + e] * f);
              w[d] = *reinterpret_cast<const uint32_t*>(&y);
            }
            uint4* to = reinterpret_cast<uint4*>(a.out + at * D + g * (D / 8));
#pragma unroll
            for (int d = 0; d < MT; d += 4) to[d / 4] = make_uint4(w[d], w[d + 1], w[d + 2], w[d + 3]);
            if (a.lse && g == 0) a.lse[at] = none ? -INFINITY : (ref[nr][e] + log2f(x)) * 0.69314718055994531f;
          }
      } else {
        // ---- join the four warps ----
        __shared__ float sm_m[WARPS][ROWS], sm_l[WARPS][ROWS];
        float* const sm_o = reinterpret_cast<float*>(smem + S::OFF_OUT);
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
            float* to = sm_o + (warp * ROWS + row) * S::OUT_LD + g * (D / 8);
#pragma unroll
            for (int d = 0; d < MT; d += 2)   // tile d: columns 2d and 2d + 1 of the lane's
              *reinterpret_cast<float4*>(to + 2 * d) =
                  make_float4(o[nr][d][e] * unit, o[nr][d][2 + e] * unit, o[nr][d + 1][e] * unit,
                              o[nr][d + 1][2 + e] * unit);
          }
        __syncthreads();
        join_warps<D, NR>(a, sg, rows, total, workers, sm_o, sm_m, sm_l, begun);
      }
    }
  }
  cp_wait<0>();
  if (KIND == BY_CTA && !whole) {
    if (threadIdx.x == 0) a.split[blockIdx.x] = begun;
    write_empty<D>(c, a);
  }
}

template <int D, int NR, int KIND>
cudaError_t start(const Kv4View& c, const Args& a, const MassArgs& w, int grid, int whole,
                  int* err_flag, cudaStream_t s) {
  using S = Shape<D, NR, KIND>;
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t e = set_max_dynamic_smem((const void*)k_attention_kv4<D, NR, KIND>, S::SMEM, attr_done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;   // every path waits for the kernel before
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = S::SMEM;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_attention_kv4<D, NR, KIND>, c, a, w, whole, err_flag);
}

// CTAs of a launch whose workers are `sharers` a CTA: every SM's slots, or the work there can be if that is less.
int grid_of(long long work, long long slots, int sharers) {
  const long long need = (work + sharers - 1) / sharers;
  return (int)(need < slots ? need : slots);
}

template <int D, int NR>
cudaError_t launch(const Kv4View& c, Args a, const MassArgs* w, int* err_flag, int num_sms, cudaStream_t s) {
  using S = Shape<D, NR, BY_CTA>;
  a.tiles = (a.q_tokens * a.group + S::ROWS - 1) / S::ROWS;
  const long long max_len = (long long)c.max_pages << c.page_log2;
  const long long max_units = (max_len + S::UNIT - 1) / S::UNIT;
  const long long slots = (long long)(num_sms < MAX_SMS ? num_sms : MAX_SMS) * S::CTAS;
  const long long items = (long long)c.batch * c.heads * a.tiles;
  const int whole = max_units <= WHOLE_UNITS;
  // Short items a warp each, without barriers and joining, where their rounds fill the warps to four fifths: 4096 items of 776
  // keys (84% of the rounds) 110 us with the weights, shared by four warps each 157.
  const long long warps = slots * WARPS, rounds = (items + warps - 1) / warps;
  cudaError_t e;
  if (whole && 5 * items >= 4 * rounds * warps) {
    e = start<D, NR, BY_WARP>(c, a, MassArgs{}, grid_of(items, slots, WARPS), 1, err_flag, s);
  } else {
    const int grid = whole ? grid_of(items, slots, 1) : grid_of(max_units > slots ? slots : items * max_units, slots, 1);
    e = start<D, NR, BY_CTA>(c, a, MassArgs{}, grid, whole, err_flag, s);
    if (e == cudaSuccess && !whole) e = launch_combine<D, NR>(a, grid, s);
  }
  if (e != cudaSuccess || !w) return e;
  // The second pass over the keys: items are (sequence, head), each key belongs to one lane, which sums over all
  // query rows. No atomics: the order is fixed.
  a.tiles = 1;
  const long long steps = (max_len + S::KS - 1) / S::KS, all = (long long)c.batch * c.heads;
  const long long work = steps > slots * WARPS ? slots * WARPS : all * steps;
  return start<D, NR, WEIGHTS>(c, a, *w, grid_of(work, slots, WARPS), 0, err_flag, s);
}

}  // namespace

size_t attention_kv4_workspace(int dim, int num_sms) {
  return notes_bytes(num_sms) + (size_t)num_sms * MAX_CTAS_PER_SM * 2 * 16 * (dim + 2) * sizeof(float);
}

cudaError_t attention_kv4(const Kv4View& c, const bf16* q, int q_tokens, int q_heads,
                          const int* kv_len, float scale, int causal, bf16* out, float* lse,
                          const MassArgs* mass, void* workspace, int* err_flag, int num_sms,
                          cudaStream_t s) {
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
  // Up to 8 rows in one 8-wide tile: two long sequences with 8 rows 62 us, in the shape for 16 rows 79. A shape for 32 rows
  // (heads of 64) took 110 us for 64 rows of 64 sequences of 2000 tokens against 119, but 15 against 12 for one of 1000.
  const bool narrow = q_tokens * a.group <= 8;
  if (c.dim == 64)
    return narrow ? launch<64, 1>(c, a, mass, err_flag, num_sms, s) : launch<64, 2>(c, a, mass, err_flag, num_sms, s);
  if (c.dim == 128)
    return narrow ? launch<128, 1>(c, a, mass, err_flag, num_sms, s) : launch<128, 2>(c, a, mass, err_flag, num_sms, s);
  return cudaErrorInvalidValue;
}

}  // namespace jepa
