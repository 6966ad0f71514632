// Products with 4-bit weights and group scales, grouped by expert, and the
// quantizer of their layout: codes 0..15, two to a byte along k, the lower
// input in the low half; w[i][j] = (code - 8) * scale[j / group][i].
#include "w4.cuh"

#include "api_common.cuh"

#include <cfloat>
#include <cstring>

#include "tc_common.cuh"

namespace moe {

namespace {

__device__ __forceinline__ float silu_f(float u) { return u / (1.0f + __expf(-u)); }

// ---------------------------------------------------------------- quantizer

// One warp per row and 256 inputs: a lane holds 8 consecutive inputs, group / 8
// lanes a group. 32 experts of 2048 x 7168: 780 us of bf16, 760 of fp32, 4.3
// and 2.3 times what their bytes take; the loads by element and the 2-byte
// stores of the scales, a row of outputs apart, are what is left.
template <typename T>
__global__ void __launch_bounds__(256) quantize_w4_kernel(const T* w, int64_t rows, int n, int k,
                                                          int group, uint8_t* q,
                                                          __nv_bfloat16* scales) {
  grid_dependency();
  const int kc = ceil_div(k, 256);
  const int64_t unit = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  if (unit >= rows * kc) return;
  const int lane = threadIdx.x % 32;
  const int64_t row = unit / kc;
  const int j = (int)(unit % kc) * 256 + lane * 8;
  float v[8];
  float m = 0.f;
  bool bad = false;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    v[u] = j < k ? to_f32(w[row * k + j + u]) : 0.f;
    m = fmaxf(m, fabsf(v[u]));
    bad |= !(fabsf(v[u]) <= FLT_MAX);
  }
  uint32_t badm = bad;
  for (int o = 1; o < group / 8; o <<= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    badm |= __shfl_xor_sync(0xffffffffu, badm, o);
  }
  __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(m, 7.0f));
  float s = __bfloat162float(sb);
  if (s == 0.f) {
    sb = __float2bfloat16_rn(1.0f);
    s = 1.0f;
  }
  if (badm) {
    s = __int_as_float(0x7fc00000);
    sb = __float2bfloat16_rn(s);
  }
  uint32_t c = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    int i = badm ? 0 : __float2int_rn(fminf(fmaxf(__fdiv_rn(v[u], s), -8.f), 7.f));
    c |= (uint32_t)(i + 8) << (4 * u);
  }
  if (j < k) {
    *reinterpret_cast<uint32_t*>(q + (row * k + j) / 2) = c;
    if (j % group == 0) {
      const int64_t e = row / n, i = row % n;
      scales[(e * (k / group) + j / group) * n + i] = sb;
    }
  }
}

// ---------------------------------------------------------------- products
//
// A CTA takes a tile of 128 weight rows (SWIGLU: 64 rows of w1 over the same
// 64 of w3) and up to TOK of their expert's token rows. A producer warp keeps
// STAGES stages of 256 inputs in flight: the codes by TMA (128 bytes a row,
// 128-byte swizzle), their scales by TMA, the token rows by TMA gathers of
// four rows. Each of four warps multiplies 32 of the weight rows over all
// inputs: it turns codes into bf16 in registers and feeds them to mma.sync
// m16n8k16 as its A side, the token rows as its B side. The weights' bytes
// bound these calls, and the tensor work of a few columns is far below either
// tensor path's rate, so what decides is the way from bytes to operands:
// registers here, where a tcgen05 operand would take the widened weights
// through shared or tensor memory first (with x as 8-bit digits on the integer
// tensor path: 442 instead of 423 us for the call below). Warps own whole rows, so a tile ends
// without a sum over warps or a barrier; in a SWIGLU tile the MMA's rows g and
// g + 8 are the same feature of w1 and of w3, and a thread holds both sums.
//
// Measured: 128 tokens' down-projection (1024 rows, 256 experts of 7168 x
// 2048, groups of 128) 417-423 us, 4.6 TB/s of codes, scales and rows, and 470
// in a loop that the power cap slows; the copies alone run at 6.4 TB/s, the
// arithmetic alone takes 393 us (28 of 72 million instructions turn codes into
// bf16, 20 move data). Issue slots are 60 % full: three multiplying warps a
// scheduler do not cover the way from a word's load through its conversion to
// its MMA. One token's up-projection 36 us and down-projection 21 us: launch,
// the offsets and a first round of loads, then 3.4 and 2.9 TB/s.
//
// The k order within 32 inputs (16 bytes of codes) is the codes' own: quad
// lane t holds the word of inputs 8t..8t+7; (word >> 4s) & 0x000f000f are the
// codes of inputs 8t+s and 8t+s+4, and or-ing 0x4300 makes them bf16 128 +
// code (the mantissa's unit is 1 there), minus 136 the weight's integer, both
// exact: the conversion through a float's exponent and mantissa bits that Kim,
// Henry, Fahim and Hassan Awadalla describe for fp16 ("Who Says Elephants Can't
// Run", 2022). The token rows' operand takes the same pairs.

using namespace tc;

constexpr int KS = 256;                  // inputs per stage
constexpr int WR = 128;                  // weight rows per tile
constexpr int W_BYTES = WR * KS / 2;     // 16 KB of codes
constexpr int NUM_THREADS = 160;
constexpr int MAX_E = 1024;

// TOK = 8 NT token rows a tile; a stage's scales are [KS / group][128] bf16.
// DEEP: a launch whose tiles are at most two per SM keeps more stages in
// flight instead of a third tile (256 tiles of one token's up-projection 37
// against 42 us; 448 tiles of its down-projection 23.0 against 22.5, 14336 of a
// decode batch's 451 against 417). Groups of 32, whose stages are larger, keep
// four: with five only one block fits an SM, and the second tiles wait (the
// same up-projection 49.3 against 37.7 us, 41.5 without the deep form).
template <int NT, bool G32, bool DEEP> struct W4Cfg {
  static constexpr int TOK = 8 * NT;
  static constexpr int X_BYTES = TOK * KS * 2;  // 4 slices of [TOK][64]
  static constexpr int S_BYTES = WR * (KS / (G32 ? 32 : 64)) * 2;
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES + S_BYTES;
  static constexpr int CTAS = NT == 1 && !DEEP ? 3 : 2;  // per SM
  static constexpr int STAGES = DEEP ? (G32 ? 4 : 5) : NT == 2 ? 4 : 3;
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + 256 + (MAX_E + 1) * 4;
  // an SM has 228 KB; each block takes 1 KB beside its own
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "CTAS blocks per SM");
};

struct W4Tma {
  CUtensorMap q1[2], q3[2];  // codes {k / 2, n, E}
  CUtensorMap s1[2], s3[2];  // scales {n, k / group, E}
  CUtensorMap x[2];          // token rows, gathered
};

// What the multiplying warps need to know of a tile; rows < 0: no more tiles.
struct W4Tile {
  int64_t row0;  // first row of the expert order (kind 0) or of x (kind 1)
  int kind, e, f0, rows;
};

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ float lds_bf16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return __uint_as_float((uint32_t)v << 16);
}

// Codes s and s + 4 of a word as the bf16 pair of their integers code - 8.
template <int s> __device__ __forceinline__ uint32_t pair_of(uint32_t q) {
  uint32_t v;  // ((q >> 4 s) & 0x000f000f) | 0x43004300 in one logic operation
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(v) : "r"(q >> (4 * s)), "r"(0x000f000fu), "r"(0x43004300u));
  const uint32_t b = 0x43084308u;  // 136, 136
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&d);
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same with a zero accumulator
__device__ __forceinline__ void mma16816_0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// One stage of a warp: acc += scale * (codes - 8) x over its two blocks of 16
// weight rows, 256 inputs and NT blocks of 8 tokens. wrow: this lane's first
// row; second block +wblk, rows 8..15 of a block +w8 (bytes; scales half of
// an element each: sc, sblk, s8). GPC: chunks of 32 inputs per scale.
template <int NT, int TOK, int GPC>
__device__ __forceinline__ void stage_mma(float (&acc)[2][TOK / 8][4], uint32_t wrow, uint32_t wblk,
                                          uint32_t w8, uint32_t x, uint32_t sc, uint32_t sblk,
                                          uint32_t s8, uint32_t sgrp, int gr, int t) {
  const int tok = (gr >> 1) | ((gr & 1) << 2);  // token of column gr: conflict-free reads
#pragma unroll
  for (int c0 = 0; c0 < 8; c0 += GPC) {  // one group of inputs
    float p[2][NT][4];
#pragma unroll
    for (int c = c0; c < c0 + GPC; ++c) {
      uint32_t b[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 v = lds128(x + (c >> 1) * (TOK * 128) + (n * 8 + tok) * 128 +
                               ((((c & 1) * 4 + t) ^ tok) << 4));
        b[n][0] = __byte_perm(v.x, v.z, 0x5410);
        b[n][1] = __byte_perm(v.x, v.z, 0x7632);
        b[n][2] = __byte_perm(v.y, v.w, 0x5410);
        b[n][3] = __byte_perm(v.y, v.w, 0x7632);
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint32_t a = wrow + m * wblk + ((c ^ gr) << 4);
        const uint32_t q0 = lds32(a), q1 = lds32(a + w8);
        const uint32_t lo[4] = {pair_of<0>(q0), pair_of<0>(q1), pair_of<1>(q0), pair_of<1>(q1)};
        const uint32_t hi[4] = {pair_of<2>(q0), pair_of<2>(q1), pair_of<3>(q0), pair_of<3>(q1)};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (c == c0) mma16816_0(p[m][n], lo, b[n][0], b[n][1]);
          else mma16816(p[m][n], lo, b[n][0], b[n][1]);
          mma16816(p[m][n], hi, b[n][2], b[n][3]);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint32_t sa = sc + m * sblk + c0 / GPC * sgrp;
      const float s0 = lds_bf16(sa), s1 = lds_bf16(sa + s8);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        acc[m][n][0] = fmaf(s0, p[m][n][0], acc[m][n][0]);
        acc[m][n][1] = fmaf(s0, p[m][n][1], acc[m][n][1]);
        acc[m][n][2] = fmaf(s1, p[m][n][2], acc[m][n][2]);
        acc[m][n][3] = fmaf(s1, p[m][n][3], acc[m][n][3]);
      }
    }
  }
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

template <bool SWIGLU, int NT, int GPC, bool DEEP>
__global__ void __launch_bounds__(NUM_THREADS, W4Cfg<NT, GPC == 1, DEEP>::CTAS)
    w4_kernel(const __grid_constant__ W4Args g, const __grid_constant__ W4Tma m) {
  using C = W4Cfg<NT, GPC == 1, DEEP>;
  constexpr int TOK = C::TOK, STAGES = C::STAGES;
  constexpr int FW = SWIGLU ? WR / 2 : WR;  // features per tile
  constexpr int NG = 8 / GPC;               // scales per row and stage
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(tiles + STAGES * C::STAGE_BYTES);
  uint64_t* empty = full + STAGES;
  W4Tile* info = reinterpret_cast<W4Tile*>(empty + STAGES);  // [STAGES]: the tile a stage begins
  volatile int* abort_flag = reinterpret_cast<volatile int*>(info + STAGES);
  int32_t* P = reinterpret_cast<int32_t*>(tiles + STAGES * C::STAGE_BYTES + 256);
  uint64_t* hang = reinterpret_cast<uint64_t*>(tiles + STAGES * C::STAGE_BYTES + 248);  // (see W4Args::stall)
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int E = g.E;

  if (warp == 1 && lane < (g.t_shared > 0 ? 2 : 1)) {
    prefetch_map(&m.q1[lane]);
    prefetch_map(&m.s1[lane]);
    prefetch_map(&m.x[lane]);
    if (SWIGLU) {
      prefetch_map(&m.q3[lane]);
      prefetch_map(&m.s3[lane]);
    }
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 4); }
    mbar_init(hang, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // token tiles per expert, by all threads (their loads side by side: one
  // warp's turns through 256 experts took 4 us of a 20 us call)
  bool bad = false;
#pragma unroll 4
  for (int e = threadIdx.x; e < E; e += NUM_THREADS) {
    const Span sp = expert_span(g.offsets, e, g.rows);
    bad |= sp.bad;
    P[e] = (int)(((int64_t)sp.count + TOK - 1) / TOK);
  }
  if (bad && blockIdx.x == 0) set_error(g.err, ERRBIT_BAD_INDEX);
  __syncthreads();

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    // the tiles' exclusive prefix over the experts
    const int per = (E + 31) / 32;
    int64_t lsum = 0;
    for (int u = 0; u < per; ++u) {
      const int e = lane * per + u;
      if (e < E) lsum += P[e];
    }
    int64_t incl = lsum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t p = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += p;
    }
    // more tiles than the rows can fill: bad offsets whose ranges overlap
    // (reported above), and a sum that may pass an int: none then
    const bool over = __shfl_sync(0xffffffffu, incl, 31) > g.rows / TOK + E;
    int run = (int)(incl - lsum);
    for (int u = 0; u < per; ++u) {
      const int e = lane * per + u;
      if (e < E) {
        const int c = P[e];
        P[e] = run;
        run += c;
      }
    }
    if (lane == 31) P[E] = over ? 0 : (int)incl;
    __syncwarp();
    const int nt0 = (g.n[0] + FW - 1) / FW, nt1 = (g.n[1] + FW - 1) / FW;
    const int mt_sh = (int)((g.t_shared + TOK - 1) / TOK);
    const int routed = nt0 * P[E], total = routed + nt1 * mt_sh;
    int s = 0, issued = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int i = blockIdx.x; ok; i += gridDim.x) {
      W4Tile t;
      t.rows = -1;
      if (i < routed) {
        const int q = i / nt0;
        int lo = 0, hi = E;  // the e with P[e] <= q < P[e + 1]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (P[mid] <= q) lo = mid; else hi = mid;
        }
        const int mt = P[lo + 1] - P[lo];
        const int l = i - nt0 * P[lo];
        const Span sp = expert_span(g.offsets, lo, g.rows);
        t.kind = 0;
        t.e = lo;
        t.f0 = l / mt * FW;
        t.row0 = (int64_t)sp.b + (l % mt) * TOK;
        t.rows = min(TOK, sp.count - (l % mt) * TOK);
      } else if (i < total) {
        const int l = i - routed;
        t.kind = 1;
        t.e = 0;
        t.f0 = l / mt_sh * FW;
        t.row0 = (int64_t)(l % mt_sh) * TOK;
        t.rows = (int)min((int64_t)TOK, g.t_shared - t.row0);
      }
      const bool end = t.rows < 0;
      const int ks = end ? 1 : (g.k[t.kind] + KS - 1) / KS;
      const int nx = (t.rows + 3) >> 2;  // gathers of four rows per slice
      // this lane's gathers: slice lane % 4, rows 4 (lane / 4) ..; a row past
      // the tile or out of x takes the out-of-range row (zeros)
      int r[4];
      if (!end) {
        const int oob = (int)(t.kind == 0 ? g.x_rows : g.t_shared);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int v = (lane >> 2) * 4 + j;
          r[j] = oob;
          if (v < t.rows) {
            r[j] = (int)(t.row0 + v);
            if (t.kind == 0 && g.src != nullptr) {
              r[j] = g.src[t.row0 + v];
              if (r[j] < 0 || r[j] >= oob) {
                r[j] = oob;
                set_error(g.err, ERRBIT_BAD_INDEX);
              }
            }
          }
        }
      }
      const uint32_t tx = W_BYTES + (uint32_t)(WR * NG * 2) + (uint32_t)(nx * 4 * KS * 2);
      for (int kb = 0; kb < ks; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], ph ^ 1, abort_flag, g.err))) { ok = false; break; }
        uint8_t* sw = tiles + s * C::STAGE_BYTES;
        uint8_t* sx = sw + W_BYTES;
        uint8_t* ss = sx + C::X_BYTES;
        if (lane == 0 && kb == 0) info[s] = t;
        if (end) {
          if (lane == 0) mbar_arrive(&full[s]);
          break;
        }
        if (lane == 0) {
          mbar_expect_tx(&full[s], tx);
          tma_load_3d(sw, &m.q1[t.kind], &full[s], kb * (KS / 2), t.f0, t.e);
          tma_load_3d(ss, &m.s1[t.kind], &full[s], t.f0, kb * NG, t.e);
          if (SWIGLU) {
            tma_load_3d(sw + W_BYTES / 2, &m.q3[t.kind], &full[s], kb * (KS / 2), t.f0, t.e);
            tma_load_3d(ss + FW * NG * 2, &m.s3[t.kind], &full[s], t.f0, kb * NG, t.e);
          }
        }
        __syncwarp();
        if (lane < 4 * nx)
          tma_gather4(sx + (lane & 3) * (TOK * 128) + (lane >> 2) * 512, &m.x[t.kind], &full[s],
                      kb * KS + (lane & 3) * 64, r[0], r[1], r[2], r[3]);
        ++issued;
        if (++s == STAGES) { s = 0; ph ^= 1; }
      }
      if (end) break;
    }
    // The next kernel may start once every CTA has asked for its last copies;
    // any earlier, and CTAs of a next call of this kernel would fill the SMs
    // unevenly while this one's still run (one token's up-projection: 50
    // instead of 39 us a call).
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // after a wait that ran out, in any warp: no copy may still be under way
    __syncthreads();
    if (*abort_flag && lane == 0)
      for (int j = 0; j < STAGES; ++j) {
        const int n = issued / STAGES + (j < issued % STAGES ? 1 : 0);
        if (n > 0) mbar_drain(&full[j], (uint32_t)((n - 1) & 1));
      }
    return;
  }

  // ------------------------------------------------------------------ multiply
  const int w = warp - 1, gr = lane >> 2, t4 = lane & 3;
  // a lane's rows: plain 32w + 16m + g and + 8; SWIGLU feature 16w + 8m + g of
  // w1 and, 64 rows on, of w3
  const int row = (SWIGLU ? 16 : 32) * w + gr;
  constexpr uint32_t WBLK = (SWIGLU ? 8 : 16) * 128, W8 = (SWIGLU ? 64 : 8) * 128;
  constexpr uint32_t SBLK = (SWIGLU ? 8 : 16) * 2, S8 = SWIGLU ? FW * NG * 2 : 8 * 2;
  const uint32_t base = smem_u32(tiles);
  const uint32_t o_w = (uint32_t)(row * 128 + t4 * 4);
  const uint32_t o_s = (uint32_t)(W_BYTES + C::X_BYTES + row * 2);
  int s = 0;
  uint32_t ph = 0;
  bool ok = true;
  if (g.stall && blockIdx.x == 0 && w == 0) ok = __all_sync(0xffffffffu, mbar_wait(hang, 0, abort_flag, g.err));
  while (ok) {
    ok = __all_sync(0xffffffffu, mbar_wait(&full[s], ph, abort_flag, g.err));
    if (!ok) break;
    const W4Tile t = info[s];
    if (t.rows < 0) break;
    const int ks = (g.k[t.kind] + KS - 1) / KS;
    float acc[2][NT][4];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[a][n][q] = 0.f;
    for (int kb = 0; kb < ks; ++kb) {
      if (kb > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&full[s], ph, abort_flag, g.err));
        if (!ok) break;
      }
      const uint32_t st = base + s * C::STAGE_BYTES;
      if (NT == 1 || t.rows <= 8)
        stage_mma<1, TOK, GPC>(acc, st + o_w, WBLK, W8, st + W_BYTES, st + o_s, SBLK, S8, FW * 2, gr, t4);
      else if (NT == 2 || t.rows <= 16)
        stage_mma<(NT < 2 ? NT : 2), TOK, GPC>(acc, st + o_w, WBLK, W8, st + W_BYTES, st + o_s, SBLK, S8,
                                               FW * 2, gr, t4);
      else
        stage_mma<NT, TOK, GPC>(acc, st + o_w, WBLK, W8, st + W_BYTES, st + o_s, SBLK, S8, FW * 2, gr, t4);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      if (++s == STAGES) { s = 0; ph ^= 1; }
    }
    if (!ok) break;
    // column 2t of a block is token t, column 2t + 1 token t + 4
    const int n_out = g.n[t.kind];
    __nv_bfloat16* out = g.out[t.kind] + t.row0 * n_out;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const int f = t.f0 + row + a * (SWIGLU ? 8 : 16);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = n * 8 + t4 + 4 * h;
          if (c >= t.rows) continue;
          __nv_bfloat16* o = out + (int64_t)c * n_out + f;
          if (SWIGLU) {
            if (f < n_out) *o = __float2bfloat16_rn(silu_f(acc[a][n][h]) * acc[a][n][2 + h]);
          } else {
            if (f < n_out) *o = __float2bfloat16_rn(acc[a][n][h]);
            if (f + 8 < n_out) o[8] = __float2bfloat16_rn(acc[a][n][2 + h]);
          }
        }
    }
  }
  __syncthreads();  // (the producer's)
}

}  // namespace

cudaError_t launch_quantize_w4(bool bf16, const void* w, int64_t E, int n, int k, int group,
                               uint8_t* q, __nv_bfloat16* scales, cudaStream_t st) {
  const int64_t rows = E * n, units = rows * ceil_div(k, 256);
  const int64_t ctas = ceil_div<int64_t>(units, 8);
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)ctas), block(256);
  if (bf16)
    return launch_pdl(true, quantize_w4_kernel<__nv_bfloat16>, grid, block, 0, st,
                      static_cast<const __nv_bfloat16*>(w), rows, n, k, group, q, scales);
  return launch_pdl(true, quantize_w4_kernel<float>, grid, block, 0, st, static_cast<const float*>(w), rows, n,
                    k, group, q, scales);
}

namespace {

bool map_u8_3d(CUtensorMap* m, const void* p, int64_t E, int64_t n, int64_t cols, uint32_t box_n) {
  auto fn = tc::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)n, (cuuint64_t)E};
  cuuint64_t strides[2] = {(cuuint64_t)cols, (cuuint64_t)(n * cols)};
  cuuint32_t box[3] = {KS / 2, box_n, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(p), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool map_scales(CUtensorMap* m, const void* p, int64_t E, int64_t groups, int64_t n, uint32_t box_n,
                uint32_t box_g) {
  auto fn = tc::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)n, (cuuint64_t)groups, (cuuint64_t)E};
  cuuint64_t strides[2] = {(cuuint64_t)(n * 2), (cuuint64_t)(n * groups * 2)};
  cuuint32_t box[3] = {box_n, box_g, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool SWIGLU, int NT, int GPC, bool DEEP>
cudaError_t launch_w4_kernel(const W4Args& g, const W4Tma& m, int64_t bound, int num_sms, cudaStream_t st) {
  using C = W4Cfg<NT, GPC == 1, DEEP>;
  static std::atomic<uint64_t> allowed{0};
  // Groups of 32: blocks of at most one tile per SM ask for more than half of
  // its shared memory, so that no two share an SM while others idle (128 tiles
  // of 64 outputs, 7168 inputs: 25.4 against 29.2 us a call, back to back).
  constexpr bool SPREAD = DEEP && GPC == 1;
  constexpr size_t ALONE = 116 * 1024;
  const size_t smem = SPREAD && bound <= num_sms ? ALONE : C::SMEM;
  cudaError_t e = allow_smem(w4_kernel<SWIGLU, NT, GPC, DEEP>, (int)(SPREAD ? ALONE : C::SMEM), &allowed);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)C::CTAS * num_sms;
  return launch_pdl(true, w4_kernel<SWIGLU, NT, GPC, DEEP>, dim3((unsigned)(bound < most ? bound : most)),
                    dim3(NUM_THREADS), smem, st, g, m);
}

template <bool SWIGLU, int NT, bool DEEP>
cudaError_t launch_w4_group(const W4Args& g, const W4Tma& m, int64_t bound, int num_sms, cudaStream_t st) {
  if (g.group == 32) return launch_w4_kernel<SWIGLU, NT, 1, DEEP>(g, m, bound, num_sms, st);
  if (g.group == 64) return launch_w4_kernel<SWIGLU, NT, 2, DEEP>(g, m, bound, num_sms, st);
  return launch_w4_kernel<SWIGLU, NT, 4, DEEP>(g, m, bound, num_sms, st);
}

template <bool SWIGLU>
cudaError_t launch_w4_tokens(const W4Args& g, const W4Tma& m, int64_t bound, int num_sms, cudaStream_t st) {
  // Token rows per tile, by the rows an expert has on average, experts without
  // rows counted (the host does not know the counts) and the shared MLP's rows
  // not: more rows share their weights' way to operands, fewer leave less
  // padding and more stages. Measured at one shape:
  // Down-projection of 256 experts of 7168 x 2048 with 8 / 16 / 32, uniform
  // routing: 417 / 440 / 451 us at 4 rows, 450 / 464 / 477 at 5, 493 / 485 /
  // 496 at 6, 700 / 573 / 577 at 10, 811 / 659 / 620 at 12. Skewed routing
  // (Zipf 0.6, 1.2) wants more rows sooner, 8 / 16: 331 / 348 and 260 / 254 at
  // 2, 439 / 440 and 405 / 395 at 4, 483 / 475 and 454 / 426 at 5.
  const int64_t avg = g.rows / g.E;
  if (avg > 10) return launch_w4_group<SWIGLU, 4, false>(g, m, bound, num_sms, st);
  if (avg > 4) return launch_w4_group<SWIGLU, 2, false>(g, m, bound, num_sms, st);
  if (bound <= 2 * (int64_t)num_sms) return launch_w4_group<SWIGLU, 1, true>(g, m, bound, num_sms, st);
  return launch_w4_group<SWIGLU, 1, false>(g, m, bound, num_sms, st);
}

}  // namespace

cudaError_t launch_w4(bool swiglu, const W4Args& g, int num_sms, cudaStream_t st) {
  W4Tma m;
  memset(&m, 0, sizeof(m));
  const uint32_t fw = swiglu ? WR / 2 : WR;
  int64_t bound = 0;
  for (int kind = 0; kind < 2; ++kind) {
    const int64_t rows = kind == 0 ? g.rows : g.t_shared, E = kind == 0 ? g.E : 1;
    if (rows == 0) continue;
    const int n = g.n[kind], k = g.k[kind];
    if (!tc::map_gather(&m.x[kind], g.x[kind], (uint64_t)(kind == 0 ? g.x_rows : rows), (uint64_t)k) ||
        !map_u8_3d(&m.q1[kind], g.q1[kind], E, n, k / 2, fw) ||
        !map_scales(&m.s1[kind], g.s1[kind], E, k / g.group, n, fw, KS / g.group))
      return cudaErrorInvalidValue;
    if (swiglu && (!map_u8_3d(&m.q3[kind], g.q3[kind], E, n, k / 2, fw) ||
                   !map_scales(&m.s3[kind], g.s3[kind], E, k / g.group, n, fw, KS / g.group)))
      return cudaErrorInvalidValue;
    bound += (int64_t)ceil_div(n, (int)fw) * (rows / 8 + (rows > E ? E : rows));
  }
  if (bound == 0) return cudaSuccess;
  return swiglu ? launch_w4_tokens<true>(g, m, bound, num_sms, st)
                : launch_w4_tokens<false>(g, m, bound, num_sms, st);
}

}  // namespace moe
