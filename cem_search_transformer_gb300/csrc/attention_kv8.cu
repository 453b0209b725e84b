// Attention of a few new tokens per sequence over the 8-bit paged cache.
//
//   o[r] = sum_j softmax_j(scale q[r] . K[j]) V[j],  K[j] = ks[page] * code, V[j] = vs[page] * code
//
// for the rows r = (new token, head of the group) that share a key/value head. Bound by the HBM
// bytes of the codes (2 kv_heads * dim a cached token), so the codes go from shared memory
// straight into mma.sync fragments: e4m3 -> f16 is exact, 64 conversions a 16-key step, and 16
// rows cost the same as one.
//   * Work: items (sequence, head, tile of 16 rows), each cut into units of 4 warps * KS keys.
//     All units of the call in one line are shared out evenly over the CTAs, so ragged lengths
//     and few long sequences fill the machine alike; an item that crosses CTAs leaves partial
//     (max, sum, output) rows in the workspace, which k_combine joins in a fixed order.
//   * A warp owns KS keys of each unit and its own ring of NST stages filled with cp.async
//     (zero-filled past the sequence's end, so stale codes there never meet the tensor cores).
//   * q is scaled per row by a power of two into f16's range; the exact scores are fp32. The
//     probabilities enter the second product as f16 (2^-12 relative, finer than bf16's 2^-9).
//   * Scores are exponentiated against a reference that moves only when the maximum grows by
//     more than 2^8, so that most steps leave the accumulators alone.
//   * Fragment layouts. A lane (g = lane / 4, t = lane % 4) takes bytes [t D/4, (t+1) D/4) of key
//     g for Q K^T, and bytes [g D/8, (g+1) D/8) of keys 2t, 2t+1, 2t+8, 2t+9 for P V: the order
//     of the summed index is free, and so is the naming of output columns. Both are wide loads
//     without bank conflicts under the XOR swizzle (dim 64: two-way for V), and a lane ends with
//     D/4 consecutive outputs of two rows.
#include "kv8.cuh"

#include <cuda_fp16.h>

namespace jepa {

namespace {

constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int NST = 4;              // cp.async stages of a warp
constexpr int ROWS = 16;            // query rows of an item
constexpr int CTAS_PER_SM = 3;
constexpr int MIN_UNITS = 2;        // units a CTA takes at least

// Probabilities are 2^(s - m + P_SHIFT) for the running reference m, which trails the maximum by
// P_SLACK at most: up to 2^15 as f16, so that the many small weights of a long context keep
// their bits (f16 ends at 2^-24, here 2^-31 of the largest).
constexpr float P_SHIFT = 7.f, P_SLACK = 8.f;

template <int D>
struct Shape {
  static constexpr int KS = 2048 / D;              // keys a warp takes in a step
  static constexpr int GROUPS = KS / 16;           // 16-key groups of P V
  static constexpr int UNIT = WARPS * KS;          // keys of a unit
  static constexpr int NT = KS / 8;                // score tiles (8 keys)
  static constexpr int KW = D / 16;                // 32-bit words of a key a lane takes
  static constexpr int VN = D / 8;                 // output tiles = values of a V row a lane takes
  static constexpr int STAGE = 2 * KS * D;         // K and V codes
  static constexpr int OFF_SCALE = WARPS * NST * STAGE;
  static constexpr int SMEM = OFF_SCALE + WARPS * NST * 16;
  static constexpr int OUT_LD = D + 4;             // fp32 row of a partial in shared memory
};

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
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
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float sane_scale(float s) {
  return s >= KV8_SCALE_MIN ? fminf(s, KV8_SCALE_MAX) : KV8_SCALE_MIN;
}
// any e4m3 NaN (0x7f, 0xff) among the four codes of w
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

struct Args {
  const bf16* q;
  const int* kv_len;
  bf16* out;
  float* lse;
  float* part;       // workspace: [CTA][2][ROWS][D + 2]
  float scale_log2;
  int q_tokens, q_heads, group, tiles, causal;
};

// Cached length of sequence s, clamped to what the table can name.
__device__ __forceinline__ int length_of(const Kv8View& c, const Args& a, int s, int* err_flag) {
  const int n = __ldg(a.kv_len + s), most = c.max_pages << c.page_log2;
  if (n < 0 || n > most) {
    if (err_flag) atomicOr(err_flag, DEV_ERR_INDEX);
    return n < 0 ? 0 : most;
  }
  return n;
}

__device__ __forceinline__ int units_of(int len, int unit) {
  return len > 0 ? (len + unit - 1) / unit : 1;   // an empty sequence has its (zero) rows written
}

// The line of units: sequence by sequence, each with heads * tiles items of units_of(len) units.
// Totals by one warp (every warp of the CTA computes the same).
__device__ __forceinline__ long long total_units(const Kv8View& c, const Args& a, int unit,
                                                 int* err_flag) {
  const int lane = threadIdx.x & 31;
  long long n = 0;
  for (int s = lane; s < c.batch; s += 32) n += units_of(length_of(c, a, s, err_flag), unit);
#pragma unroll
  for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n * c.heads * a.tiles;
}

// Position in the line: sequence s whose items begin at unit `base`, of `n` units each.
struct Cursor {
  int s, n, len;
  long long base;
};
__device__ __forceinline__ void seek(const Kv8View& c, const Args& a, int unit, long long u,
                                     Cursor& at) {
  const int lane = threadIdx.x & 31;
  const long long per = (long long)c.heads * a.tiles;
  long long base = at.base;
  for (int s0 = at.s; s0 < c.batch; s0 += 32) {
    const int s = s0 + lane;
    const int len = s < c.batch ? length_of(c, a, s, nullptr) : 0;
    const int n = s < c.batch ? units_of(len, unit) : 0;
    long long incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const uint32_t beyond = __ballot_sync(0xffffffffu, base + incl * per > u);
    if (beyond) {
      const int src = __ffs((int)beyond) - 1;
      at.s = s0 + src;
      at.n = __shfl_sync(0xffffffffu, n, src);
      at.len = __shfl_sync(0xffffffffu, len, src);
      at.base = base + (__shfl_sync(0xffffffffu, incl, src) - at.n) * per;
      return;
    }
    base += __shfl_sync(0xffffffffu, incl, 31) * per;
  }
  at.s = c.batch;
}

// CTAs that take part: each has MIN_UNITS units at least.
__device__ __forceinline__ int workers_of(long long total, int grid) {
  const long long w = (total + MIN_UNITS - 1) / MIN_UNITS;
  return w < grid ? (int)w : grid;
}

template <int D>
__device__ __forceinline__ float* part_of(const Args& a, int cta, int which) {
  return a.part + ((long long)cta * 2 + which) * (ROWS * (D + 2));
}

template <int D>
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM)
    k_attention_kv8(Kv8View c, Args a, int* err_flag) {
  using S = Shape<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sm_m[WARPS][ROWS], sm_l[WARPS][ROWS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * (NST * S::STAGE);
  const uint8_t* ring_ptr = smem + warp * (NST * S::STAGE);
  const uint32_t ring_sc =
      (uint32_t)__cvta_generic_to_shared(smem) + S::OFF_SCALE + warp * (NST * 16);
  const float* ring_sc_ptr = reinterpret_cast<const float*>(smem + S::OFF_SCALE) + warp * NST * 4;

  const long long total = total_units(c, a, S::UNIT, blockIdx.x == 0 ? err_flag : nullptr);
  const int workers = workers_of(total, gridDim.x);
  if ((int)blockIdx.x >= workers) return;
  const long long u_begin = kv8_share(total, workers, blockIdx.x);
  const long long u_end = kv8_share(total, workers, blockIdx.x + 1);
  Cursor cur{0, 0, 0, 0};
  const int rows = a.q_tokens * a.group;

  for (long long u = u_begin; u < u_end;) {
    seek(c, a, S::UNIT, u, cur);
    const long long in = u - cur.base;
    const int item = (int)(in / cur.n), k0 = (int)(in % cur.n);
    const int k1 = (int)min((long long)cur.n, k0 + (u_end - u));   // units [k0, k1) of the item
    const int head = item / a.tiles, r0 = (item % a.tiles) * ROWS;
    const int s = cur.s, len = cur.len;
    const long long table0 = (long long)s * c.max_pages;

    // ---- the warp's share of the keys: steps k0 .. k1 - 1, KS keys each ----
    const int steps = k1 - k0;
    auto key_of = [&](int i) { return (k0 + i) * S::UNIT + warp * S::KS; };
    // page of the 16-key group `grp` of step i (-1: none, or out of range)
    auto page_of = [&](int i, int grp) {
      const int key = key_of(i) + 16 * grp;
      if (i >= steps || key >= len) return -1;
      return __ldg(c.table + table0 + (key >> c.page_log2));
    };
    int pg_next[S::GROUPS];
    auto fetch_pages = [&](int i) {
#pragma unroll
      for (int p = 0; p < S::GROUPS; ++p) pg_next[p] = page_of(i, p);
    };
    auto issue = [&](int i) {   // step i into stage i % NST; pg_next holds its pages
      const uint32_t st = ring + (i % NST) * S::STAGE;
      const int key0 = key_of(i);
      if (i < steps && key0 < len) {
        constexpr int CPR = D / 16;                // 16-byte chunks of a row
        constexpr int RPI = 32 / CPR;              // rows a warp copies in one instruction
        const int chunk = lane % CPR, sub = lane / CPR;
#pragma unroll
        for (int q = 0; q < S::KS / RPI; ++q) {
          const int row = q * RPI + sub, key = key0 + row;
          const int grp = (q * RPI) / 16;          // RPI divides 16
          int pg = pg_next[grp];
          const bool there = pg >= 0 && pg < c.num_pages && key < len;
          if (!there) pg = 0;
          const long long from =
              (((long long)pg * c.heads + head) * c.page + (key & (c.page - 1))) * D + 16 * chunk;
          const int sw = D == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3);
          const uint32_t to = st + row * D + 16 * sw;
          cp16(to, c.k + from, there ? 16 : 0);
          cp16(to + S::KS * D, c.v + from, there ? 16 : 0);
        }
        if (lane < 2 * S::GROUPS) {
          int pg = S::GROUPS == 1 || lane < 2 ? pg_next[0] : pg_next[S::GROUPS - 1];
          const bool named = key0 + 16 * (lane >> 1) < len;
          const bool there = pg >= 0 && pg < c.num_pages && named;
          if (!there && named) atomicOr(err_flag, DEV_ERR_INDEX);
          if (!there) pg = 0;
          cp4(ring_sc + (i % NST) * 16 + lane * 4,
              ((lane & 1) ? c.v_scale : c.k_scale) + (long long)pg * c.heads + head,
              there ? 4 : 0);
        }
      }
      cp_commit();
    };
    fetch_pages(0);
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) {
      issue(i);
      fetch_pages(i + 1);
    }

    // ---- queries: rows g and g + 8 of the tile as f16, times 2^-e so that |q| < 2^15 ----
    uint32_t qf[S::KW][4];
    float qs[2];        // 2^e * softmax scale * log2(e)
    int lim[2];         // keys a row sees
    int lim_min = len;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int r = r0 + g + 8 * hf;
      const bool valid = r < rows;
      const int tok = valid ? r / a.group : 0, hd = head * a.group + (valid ? r % a.group : 0);
      const bf16* src = a.q + (((long long)s * a.q_tokens + tok) * a.q_heads + hd) * D + t * (D / 4);
      uint32_t w[D / 8];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 x = valid ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0, 0, 0, 0);
        w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
      }
      uint32_t top = 0;   // largest |q| as bits (bf16 magnitudes compare as integers)
#pragma unroll
      for (int i = 0; i < D / 8; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // exponent e with |q| 2^-e < 2^15; a row of zeros, infinities or NaN keeps a harmless one
      int e = (int)(top >> 7) - 127 - 14;
      e = max(-126, min(e, 113));
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
      qs[hf] = __uint_as_float((uint32_t)(127 + e) << 23) * a.scale_log2;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const float lo = __uint_as_float(w[i] << 16) * down;
        const float hi = __uint_as_float(w[i] & 0xffff0000u) * down;
        qf[i >> 1][(i & 1) * 2 + hf] = pack_f16(lo, hi);
      }
      lim[hf] = len;
      if (a.causal && valid) lim[hf] = max(0, len - a.q_tokens + tok + 1);
      lim_min = min(lim_min, lim[hf]);
    }
    lim_min = __reduce_min_sync(0xffffffffu, lim_min);

    float o[S::VN][4];
#pragma unroll
    for (int i = 0; i < S::VN; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float vs_cur = 1.f;   // outputs are o * vs_cur
    bool first_scale = true;

    for (int i = 0; i < steps; ++i) {
      cp_wait<NST - 2>();
      __syncwarp();
      issue(i + NST - 1);
      fetch_pages(i + NST);
      const int key0 = key_of(i);
      if (key0 >= len) continue;
      const uint8_t* kb = ring_ptr + (i % NST) * S::STAGE;
      const uint8_t* vb = kb + S::KS * D;
      const float* scales = ring_sc_ptr + (i % NST) * 4;

      // scores
      float sc[S::NT][4];
#pragma unroll
      for (int j = 0; j < S::NT; ++j) {
        sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
        const int row = 8 * j + g;
        uint32_t w[S::KW];
#pragma unroll
        for (int i4 = 0; i4 < S::KW / 4; ++i4) {
          const int chunk = t * (S::KW / 4) + i4;
          const int sw = D == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3);
          const uint4 x = *reinterpret_cast<const uint4*>(kb + row * D + 16 * sw);
          w[4 * i4] = x.x; w[4 * i4 + 1] = x.y; w[4 * i4 + 2] = x.z; w[4 * i4 + 3] = x.w;
        }
#pragma unroll
        for (int q = 0; q < S::KW; ++q)
          mma_f16(sc[j], qf[q][0], qf[q][1], qf[q][2], qf[q][3], f16x2_of_e4m3x2(w[q]),
                  f16x2_of_e4m3x2_hi(w[q]));
      }
      const bool edge = key0 + S::KS > lim_min;   // some row does not see some key (warp-uniform)
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < S::NT; ++j) {
        const float ks = sane_scale(scales[2 * (j >> 1)]);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = sc[j][2 * hf + e] * (qs[hf] * ks);
            if (edge && key0 + 8 * j + 2 * t + e >= lim[hf]) x = -INFINITY;
            sc[j][2 * hf + e] = x;
            top[hf] = fmaxf(top[hf], x);
          }
      }
      bool move = false;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        top[hf] = fmaxf(top[hf], __shfl_xor_sync(0xffffffffu, top[hf], 1));
        top[hf] = fmaxf(top[hf], __shfl_xor_sync(0xffffffffu, top[hf], 2));
        move = move || top[hf] > m[hf] + P_SLACK || (m[hf] == -INFINITY && top[hf] > -INFINITY);
      }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float mn = fmaxf(m[hf], top[hf]);
          const float al = mn == -INFINITY ? 1.f : ex2f(m[hf] - mn);
          m[hf] = mn;
          l[hf] *= al;
#pragma unroll
          for (int d = 0; d < S::VN; ++d) {
            o[d][2 * hf] *= al;
            o[d][2 * hf + 1] *= al;
          }
        }
      }
      const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0] - P_SHIFT,
                            m[1] == -INFINITY ? 0.f : m[1] - P_SHIFT};
#pragma unroll
      for (int p = 0; p < S::GROUPS; ++p) {
        const float vs = sane_scale(scales[2 * p + 1]);
        if (first_scale) {
          vs_cur = vs;
          first_scale = false;
        }
        float ratio = vs / vs_cur;
        if (!(ratio >= 0x1p-6f && ratio <= 1.f)) {
          // larger than the accumulators' unit, or far below it: move them (by 2^80 at most)
          const float f = vs_cur / vs;
#pragma unroll
          for (int d = 0; d < S::VN; ++d) {
            o[d][0] *= f; o[d][1] *= f; o[d][2] *= f; o[d][3] *= f;
          }
          vs_cur = vs;
          ratio = 1.f;
        }
        float pr[2][4];   // [tile of the group][c index]
#pragma unroll
        for (int jj = 0; jj < 2; ++jj)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = ex2f(sc[2 * p + jj][e] - ref[e >> 1]);
            l[e >> 1] += x;
            pr[jj][e] = x * ratio;
          }
        const uint32_t a0 = pack_f16(pr[0][0], pr[0][1]), a1 = pack_f16(pr[0][2], pr[0][3]);
        const uint32_t a2 = pack_f16(pr[1][0], pr[1][1]), a3 = pack_f16(pr[1][2], pr[1][3]);
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
              mma_f16(o[4 * q + 2 * hb], a0, a1, a2, a3, f16x2_of_e4m3x2(x), f16x2_of_e4m3x2(y));
              mma_f16(o[4 * q + 2 * hb + 1], a0, a1, a2, a3, f16x2_of_e4m3x2_hi(x),
                      f16x2_of_e4m3x2_hi(y));
            }
        } else {
          // second product: 1 where a row sees a key, times 1 where V is NaN
          uint32_t see[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int hf = k & 1, key = key0 + 16 * p + 8 * (k >> 1) + 2 * t;
            see[k] = pack_f16(key < lim[hf] ? 1.f : 0.f, key + 1 < lim[hf] ? 1.f : 0.f);
          }
#pragma unroll
          for (int q = 0; q < S::VN / 4; ++q)
#pragma unroll
            for (int hb = 0; hb < 4; ++hb) {
              const uint32_t sel = hb == 0 ? 0x40 : hb == 1 ? 0x51 : hb == 2 ? 0x62 : 0x73;
              uint32_t b[2], n[2];
#pragma unroll
              for (int h2 = 0; h2 < 2; ++h2) {
                const uint32_t codes = __byte_perm(w[2 * h2][q], w[2 * h2 + 1][q], sel) & 0xffffu;
                const uint32_t nan = (nan_codes(codes) & 0x8080u) >> 7;   // 1 per NaN code
                b[h2] = f16x2_of_e4m3x2(codes & ~(nan * 0xffu));
                n[h2] = ((nan & 1u) ? 0x3c00u : 0u) | ((nan & 0x100u) ? 0x3c000000u : 0u);
              }
              float hit[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(o[4 * q + hb], a0, a1, a2, a3, b[0], b[1]);
              mma_f16(hit, see[0], see[1], see[2], see[3], n[0], n[1]);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (hit[e] > 0.f) o[4 * q + hb][e] = __int_as_float(0x7fc00000);
            }
        }
      }
    }
    cp_wait<0>();

    // ---- join the four warps ----
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 1);
      l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 2);
      // from here on m is the exponent's reference; -inf only where no key was seen (scores
      // that are all NaN leave the maximum at -inf, but a NaN sum)
      m[hf] = m[hf] != -INFINITY ? m[hf] - P_SHIFT : l[hf] == 0.f ? -INFINITY : 0.f;
      if (t == 0) {
        sm_m[warp][g + 8 * hf] = m[hf];
        sm_l[warp][g + 8 * hf] = l[hf];
      }
    }
    __syncthreads();   // all warps are done with their rings: they hold the outputs now
    float* sm_o = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) mx = fmaxf(mx, sm_m[w][g + 8 * hf]);
      const float f = (m[hf] == -INFINITY ? 0.f : ex2f(m[hf] - mx)) * vs_cur;
      float* to = sm_o + (warp * ROWS + g + 8 * hf) * S::OUT_LD + t * (D / 4);
      // o[d] columns 2t, 2t + 1 are values (2t) VN + d and (2t + 1) VN + d
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int d = 0; d < S::VN; d += 4) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (m[hf] != -INFINITY)
            x = make_float4(o[d][2 * hf + e] * f, o[d + 1][2 * hf + e] * f, o[d + 2][2 * hf + e] * f,
                            o[d + 3][2 * hf + e] * f);
          *reinterpret_cast<float4*>(to + e * S::VN + d) = x;
        }
    }
    __syncthreads();
    {
      constexpr int TPR = THREADS / ROWS;    // threads a row
      constexpr int CPT = D / TPR;           // columns a thread
      const int row = threadIdx.x / TPR, c0 = (threadIdx.x % TPR) * CPT;
      float mx = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) mx = fmaxf(mx, sm_m[w][row]);
#pragma unroll
      for (int w = 0; w < WARPS; ++w)
        sum += sm_m[w][row] == -INFINITY ? 0.f : sm_l[w][row] * ex2f(sm_m[w][row] - mx);
      float acc[CPT];
#pragma unroll
      for (int i = 0; i < CPT; i += 4) {
        float4 x = *reinterpret_cast<const float4*>(sm_o + row * S::OUT_LD + c0 + i);
#pragma unroll
        for (int w = 1; w < WARPS; ++w) {
          const float4 y =
              *reinterpret_cast<const float4*>(sm_o + (w * ROWS + row) * S::OUT_LD + c0 + i);
          x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
        }
        acc[i] = x.x; acc[i + 1] = x.y; acc[i + 2] = x.z; acc[i + 3] = x.w;
      }
      const int r = r0 + row;
      if (k0 == 0 && k1 == cur.n) {
        if (r < rows) {
          const int tok = r / a.group, hd = head * a.group + r % a.group;
          const long long at = ((long long)s * a.q_tokens + tok) * a.q_heads + hd;
          const float inv = mx == -INFINITY ? 0.f : 1.f / sum;
          uint32_t w[CPT / 2];
#pragma unroll
          for (int i = 0; i < CPT / 2; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(mx == -INFINITY ? 0.f : acc[2 * i] * inv,
                                                           mx == -INFINITY ? 0.f : acc[2 * i + 1] * inv);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
          }
#pragma unroll
          for (int i = 0; i < CPT / 8; ++i)
            *reinterpret_cast<uint4*>(a.out + at * D + c0 + 8 * i) =
                make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          if (a.lse && c0 == 0)
            a.lse[at] = mx == -INFINITY ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994531f;
        }
      } else {
        // part 1 begins in this CTA and goes on in the next; part 0 began in an earlier one
        float* to = part_of<D>(a, blockIdx.x, k0 == 0 ? 1 : 0);
#pragma unroll
        for (int i = 0; i < CPT; i += 2)
          *reinterpret_cast<float2*>(to + row * D + c0 + i) = make_float2(acc[i], acc[i + 1]);
        if (c0 == 0) {
          to[ROWS * D + row] = mx;
          to[ROWS * D + ROWS + row] = sum;
        }
      }
    }
    __syncthreads();   // before the rings are filled again
    u += k1 - k0;
  }
}

// Joins the items that were split: the CTA in whose share such an item begins reads its parts in
// order. One thread per (row, 4 columns).
template <int D>
__global__ void __launch_bounds__(ROWS * D / 4) k_combine(Kv8View c, Args a, int grid_main) {
  using S = Shape<D>;
  const long long total = total_units(c, a, S::UNIT, nullptr);
  const int workers = workers_of(total, grid_main);
  const int w0 = blockIdx.x;
  if (w0 >= workers) return;
  const long long u_begin = kv8_share(total, workers, w0), u_end = kv8_share(total, workers, w0 + 1);
  Cursor cur{0, 0, 0, 0};
  seek(c, a, S::UNIT, u_end - 1, cur);
  const long long in = u_end - 1 - cur.base;
  const int item = (int)(in / cur.n);
  const long long i_begin = cur.base + (long long)item * cur.n, i_end = i_begin + cur.n;
  if (i_begin < u_begin || i_end <= u_end) return;   // begins earlier, or ends here
  const int w1 = kv8_worker_of(total, workers, i_end - 1);
  const int row = threadIdx.x / (D / 4), c0 = (threadIdx.x % (D / 4)) * 4;
  const int head = item / a.tiles, r = (item % a.tiles) * ROWS + row;
  if (r >= a.q_tokens * a.group) return;
  float mx = -INFINITY;
  for (int w = w0; w <= w1; ++w) mx = fmaxf(mx, part_of<D>(a, w, w == w0)[ROWS * D + row]);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  if (mx != -INFINITY) {
    for (int w = w0; w <= w1; ++w) {
      const float* p = part_of<D>(a, w, w == w0);
      const float pm = p[ROWS * D + row];
      if (pm == -INFINITY) continue;
      const float f = ex2f(pm - mx);
      const float2 x = *reinterpret_cast<const float2*>(p + row * D + c0);
      const float2 y = *reinterpret_cast<const float2*>(p + row * D + c0 + 2);
      sum = fmaf(p[ROWS * D + ROWS + row], f, sum);
      acc.x = fmaf(x.x, f, acc.x); acc.y = fmaf(x.y, f, acc.y);
      acc.z = fmaf(y.x, f, acc.z); acc.w = fmaf(y.y, f, acc.w);
    }
  }
  const int tok = r / a.group, hd = head * a.group + r % a.group;
  const long long at = ((long long)cur.s * a.q_tokens + tok) * a.q_heads + hd;
  const float inv = mx == -INFINITY ? 0.f : 1.f / sum;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  uint2 o2;
  o2.x = *reinterpret_cast<const uint32_t*>(&lo);
  o2.y = *reinterpret_cast<const uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(a.out + at * D + c0) = o2;
  if (a.lse && c0 == 0)
    a.lse[at] = mx == -INFINITY ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994531f;
}

int tiles_of(int q_tokens, int group) { return (q_tokens * group + ROWS - 1) / ROWS; }

// CTAs of a call: every SM's slots, or the units there can be if they are fewer.
int grid_of(int tiles, int heads, int batch, long long max_units, int num_sms) {
  const long long slots = (long long)num_sms * CTAS_PER_SM;
  const long long most = max_units > slots ? slots : max_units * heads * tiles * batch;
  return (int)(most < slots ? (most < 1 ? 1 : most) : slots);
}

template <int D>
cudaError_t launch(const Kv8View& c, const Args& a, int* err_flag, int num_sms, cudaStream_t s) {
  using S = Shape<D>;
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = set_max_dynamic_smem((const void*)k_attention_kv8<D>, S::SMEM, attr_done);
  if (e != cudaSuccess) return e;
  const long long max_len = (long long)c.max_pages << c.page_log2;
  const int grid = grid_of(a.tiles, c.heads, c.batch, (max_len + S::UNIT - 1) / S::UNIT, num_sms);
  k_attention_kv8<D><<<grid, THREADS, S::SMEM, s>>>(c, a, err_flag);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (max_len > S::UNIT) {   // otherwise every item is one unit and none is split
    k_combine<D><<<grid, ROWS * D / 4, 0, s>>>(c, a, grid);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace

size_t attention_kv8_workspace(int dim, int num_sms) {
  return (size_t)num_sms * CTAS_PER_SM * 2 * ROWS * (dim + 2) * sizeof(float);
}

cudaError_t attention_kv8(const Kv8View& c, const bf16* q, int q_tokens, int q_heads,
                          const int* kv_len, float scale, int causal, bf16* out, float* lse,
                          void* workspace, int* err_flag, int num_sms, cudaStream_t s) {
  Args a;
  a.q = q;
  a.kv_len = kv_len;
  a.out = out;
  a.lse = lse;
  a.part = (float*)workspace;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.q_tokens = q_tokens;
  a.q_heads = q_heads;
  a.group = q_heads / c.heads;
  a.tiles = tiles_of(q_tokens, a.group);
  a.causal = causal;
  if (c.dim == 64) return launch<64>(c, a, err_flag, num_sms, s);
  if (c.dim == 128) return launch<128>(c, a, err_flag, num_sms, s);
  return cudaErrorInvalidValue;
}

}  // namespace jepa
