// Products with 4-bit weights and group scales, grouped by expert, and the
// quantizer of their layout: codes 0..15, two to a byte along k, the lower
// input in the low half; w[i][j] = (code - 8) * scale[j / group][i].
#include "w4.cuh"

#include <cstring>

#include "tc_common.cuh"

namespace moe {

namespace {

__device__ __forceinline__ float silu_f(float u) { return u / (1.0f + __expf(-u)); }

// ---------------------------------------------------------------- quantizer

// One warp per row i and 32 * CPT inputs: a lane holds 8 consecutive inputs,
// group / 8 lanes a group.
template <typename T>
__global__ void __launch_bounds__(256) quantize_w4_kernel(const T* w, int64_t rows, int n, int k,
                                                          int group, uint8_t* q,
                                                          __nv_bfloat16* scales) {
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
    bad |= !(fabsf(v[u]) <= 3.4e38f);
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
// 64 of w3) and up to 16 of their expert's token rows. A producer warp keeps
// STAGES stages of 256 inputs in flight: the codes by TMA (128 bytes a row,
// 128-byte swizzle), their scales by TMA, the token rows by TMA gathers of
// four rows. Eight warps multiply: warp (mi, ki) takes 64 weight rows and 64
// of the stage's inputs, turns codes into bf16 in registers and feeds them to
// mma.sync m16n8k16 as its A side, the token rows as its B side, and sums the
// four ki at the end of the tile. The weights' bytes bound these calls, and
// the tensor work of a few columns is far below either tensor path's rate, so
// what decides is the way from bytes to operands: registers here, where a
// tcgen05 operand would take the widened weights through shared or tensor
// memory first.
//
// The k order within 32 inputs (16 bytes of codes) is the codes' own: quad
// lane t holds the word of inputs 8t..8t+7; (word >> 4s) & 0x000f000f are the
// codes of inputs 8t+s and 8t+s+4, and or-ing 0x4300 makes them bf16 128 +
// code (the mantissa's unit is 1 there), minus 136 the weight's integer, both
// exact. The token rows' operand takes the same pairs.

using namespace tc;

constexpr int KS = 256;                  // inputs per stage
constexpr int WR = 128;                  // weight rows per tile
constexpr int TOK = 16;                  // token rows per tile
constexpr int W_BYTES = WR * KS / 2;     // 16 KB of codes
constexpr int X_BYTES = TOK * KS * 2;    // 8 KB of token rows: 4 slices of [16][64]
constexpr int S_BYTES = WR * (KS / 32) * 2;  // 2 KB of scales (group 32)
constexpr int STAGE_BYTES = W_BYTES + X_BYTES + S_BYTES;
constexpr int STAGES = 3;
constexpr int RED_BYTES = 8 * 64 * 8 * 4;    // [warp][64 rows][8 tokens] fp32
constexpr int NUM_THREADS = 288;
constexpr int MAX_E = 1024;
constexpr size_t SMEM_BYTES = 1024 + (size_t)STAGES * STAGE_BYTES + RED_BYTES + 128 + (MAX_E + 1) * 4;

struct W4Tma {
  CUtensorMap q1[2], q3[2];  // codes {k / 2, n, E}
  CUtensorMap s1[2], s3[2];  // scales {n, k / group, E}
  CUtensorMap x[2];          // token rows, gathered
};

struct W4Tile {
  int kind, e, f0;
  int64_t row0;  // first row of the expert order (kind 0) or of x (kind 1)
  int rows;
};

struct W4Sched {
  const int32_t* P;  // smem: token-tile prefix over experts
  int E, nt0, nt1, mt_sh, routed, total;
  int fw;            // features per tile
};

__device__ __forceinline__ W4Tile decode(const W4Sched& S, const W4Args& g, int i) {
  W4Tile t;
  if (i < S.routed) {
    const int q = i / S.nt0;
    int lo = 0, hi = S.E;  // the e with P[e] <= q < P[e + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (S.P[mid] <= q) lo = mid; else hi = mid;
    }
    const int mt = S.P[lo + 1] - S.P[lo];
    const int l = i - S.nt0 * S.P[lo];
    const Span sp = expert_span(g.offsets, lo, g.rows);
    t.kind = 0;
    t.e = lo;
    t.f0 = l / mt * S.fw;
    t.row0 = (int64_t)sp.b + (l % mt) * TOK;
    t.rows = min(TOK, sp.count - (l % mt) * TOK);
  } else {
    const int l = i - S.routed;
    t.kind = 1;
    t.e = 0;
    t.f0 = l / S.mt_sh * S.fw;
    t.row0 = (int64_t)(l % S.mt_sh) * TOK;
    t.rows = (int)min((int64_t)TOK, g.t_shared - t.row0);
  }
  return t;
}

// Named barrier 1 over the eight multiplying warps that ORs a flag across them.
__device__ __forceinline__ bool sync_any(bool flag) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)flag)
      : "memory");
  return r != 0;
}

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
  uint32_t v = ((q >> (4 * s)) & 0x000f000fu) | 0x43004300u;
  const uint32_t b = 0x43084308u;  // 136, 136
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&d);
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One stage for warp (mi, ki): acc += scale * (codes - 8) x, over its 64
// weight rows, its 64 inputs and NT blocks of 8 tokens.
template <int NT, bool G32>
__device__ __forceinline__ void stage_mma(float (&acc)[4][TOK / 8][4], uint32_t wrow, uint32_t xs,
                                          uint32_t sc, uint32_t sc_step, int ki, int gr, int t) {
  const int tok = (gr >> 1) | ((gr & 1) << 2);  // token of column gr: conflict-free reads
  uint32_t b[NT][2][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint4 v = lds128(xs + (n * 8 + tok) * 128 + (((c * 4 + t) ^ tok) << 4));
      b[n][c][0] = __byte_perm(v.x, v.z, 0x5410);
      b[n][c][1] = __byte_perm(v.x, v.z, 0x7632);
      b[n][c][2] = __byte_perm(v.y, v.w, 0x5410);
      b[n][c][3] = __byte_perm(v.y, v.w, 0x7632);
    }
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    float p[NT][4];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (c == 0 || G32) {
#pragma unroll
        for (int n = 0; n < NT; ++n) p[n][0] = p[n][1] = p[n][2] = p[n][3] = 0.f;
      }
      const uint32_t a = wrow + m * 16 * 128 + (((ki * 2 + c) ^ gr) << 4);
      const uint32_t q0 = lds32(a), q1 = lds32(a + 8 * 128);
      const uint32_t l0 = pair_of<0>(q0), l1 = pair_of<0>(q1), l2 = pair_of<1>(q0), l3 = pair_of<1>(q1);
      const uint32_t h0 = pair_of<2>(q0), h1 = pair_of<2>(q1), h2 = pair_of<3>(q0), h3 = pair_of<3>(q1);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma16816(p[n], l0, l1, l2, l3, b[n][c][0], b[n][c][1]);
        mma16816(p[n], h0, h1, h2, h3, b[n][c][2], b[n][c][3]);
      }
      if (c == 1 || G32) {
        const uint32_t sa = sc + m * 32 + (G32 ? c * sc_step : 0u);
        const float s0 = lds_bf16(sa), s1 = lds_bf16(sa + 16);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[m][n][0] = fmaf(s0, p[n][0], acc[m][n][0]);
          acc[m][n][1] = fmaf(s0, p[n][1], acc[m][n][1]);
          acc[m][n][2] = fmaf(s1, p[n][2], acc[m][n][2]);
          acc[m][n][3] = fmaf(s1, p[n][3], acc[m][n][3]);
        }
      }
    }
  }
}

template <bool SWIGLU, bool G32>
__global__ void __launch_bounds__(NUM_THREADS, 2)
    w4_kernel(const __grid_constant__ W4Args g, const __grid_constant__ W4Tma m) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  float* red = reinterpret_cast<float*>(tiles + STAGES * STAGE_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(tiles + STAGES * STAGE_BYTES + RED_BYTES);
  uint64_t* empty = full + STAGES;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + STAGES);
  int32_t* P = reinterpret_cast<int32_t*>(tiles + STAGES * STAGE_BYTES + RED_BYTES + 128);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int E = g.E;

  if (warp == 0) {
    if (lane == 0) {
      for (int s = 0; s < STAGES; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 8); }
      *abort_flag = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    const int per = (E + 31) / 32;
    int lsum = 0;
    bool bad = false;
    for (int u = 0; u < per; ++u) {
      const int e = lane * per + u;
      if (e < E) {
        const Span sp = expert_span(g.offsets, e, g.rows);
        bad |= sp.bad;
        P[e] = (int)(((int64_t)sp.count + TOK - 1) / TOK);
        lsum += P[e];
      }
    }
    if (bad && blockIdx.x == 0) set_error(g.err, ERRBIT_BAD_INDEX);
    int incl = lsum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int p = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += p;
    }
    int run = incl - lsum;
    for (int u = 0; u < per; ++u) {
      const int e = lane * per + u;
      if (e < E) {
        const int c = P[e];
        P[e] = run;
        run += c;
      }
    }
    if (lane == 31) P[E] = incl;
  }
  __syncthreads();

  W4Sched S;
  S.P = P;
  S.E = E;
  S.fw = SWIGLU ? WR / 2 : WR;
  S.nt0 = (g.n[0] + S.fw - 1) / S.fw;
  S.nt1 = g.t_shared > 0 ? (g.n[1] + S.fw - 1) / S.fw : 0;
  S.mt_sh = (int)((g.t_shared + TOK - 1) / TOK);
  S.routed = S.nt0 * P[E];
  S.total = S.routed + S.nt1 * S.mt_sh;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    int s = 0, issued = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int i = blockIdx.x; ok && i < S.total; i += gridDim.x) {
      const W4Tile t = decode(S, g, i);
      const int ks = (g.k[t.kind] + KS - 1) / KS;
      const int nx = (t.rows + 3) >> 2;  // gathers of four rows per slice
      // this lane's gather: slice lane % 4, rows 4 (lane / 4) ..; a row past
      // the tile or out of x takes the out-of-range row (zeros)
      const int oob = (int)(t.kind == 0 ? g.x_rows : g.t_shared);
      int r[4];
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
      const uint32_t tx = W_BYTES + (uint32_t)(WR * (KS / g.group) * 2) + (uint32_t)(nx * 4 * KS * 2);
      for (int kb = 0; kb < ks; ++kb) {
        int w = 1;
        if (lane == 0) w = mbar_wait(&empty[s], ph ^ 1, abort_flag, g.err) ? 1 : 0;
        if (!__shfl_sync(0xffffffffu, w, 0)) { ok = false; break; }
        uint8_t* sw = tiles + s * STAGE_BYTES;
        uint8_t* sx = sw + W_BYTES;
        uint8_t* ss = sx + X_BYTES;
        const int kg = kb * (KS / g.group);
        if (lane == 0) {
          mbar_expect_tx(&full[s], tx);
          tma_load_3d(sw, &m.q1[t.kind], &full[s], kb * (KS / 2), t.f0, t.e);
          tma_load_3d(ss, &m.s1[t.kind], &full[s], t.f0, kg, t.e);
          if (SWIGLU) {
            tma_load_3d(sw + W_BYTES / 2, &m.q3[t.kind], &full[s], kb * (KS / 2), t.f0, t.e);
            tma_load_3d(ss + (WR / 2) * (KS / g.group) * 2, &m.s3[t.kind], &full[s], t.f0, kg, t.e);
          }
        }
        __syncwarp();
        if (lane < 4 * nx)
          tma_gather4(sx + (lane & 3) * (TOK * 128) + (lane >> 2) * 512, &m.x[t.kind], &full[s],
                      kb * KS + (lane & 3) * 64, r[0], r[1], r[2], r[3]);
        ++issued;
        if (++s == STAGES) { s = 0; ph ^= 1; }
      }
    }
    if (!ok && lane == 0)
      for (int j = 0; j < STAGES; ++j) {
        const int n = issued / STAGES + (j < issued % STAGES ? 1 : 0);
        if (n > 0) mbar_drain(&full[j], (uint32_t)((n - 1) & 1));
      }
    return;
  }

  // ------------------------------------------------------------------ multiply
  const int cw = warp - 1, mi = cw >> 2, ki = cw & 3;
  const int gr = lane >> 2, t4 = lane & 3;
  const int ng = KS / g.group;
  // byte offsets within a stage: this lane's weight row, its slice of the
  // token rows, its scale
  const uint32_t base = smem_u32(tiles);
  const uint32_t o_w = (uint32_t)((mi * 64 + gr) * 128 + t4 * 4);
  const uint32_t o_x = (uint32_t)(W_BYTES + ki * (TOK * 128));
  const int sgrp = ki * 64 / g.group;  // group of the warp's first input
  const uint32_t s_row = SWIGLU ? 64 * 2 : WR * 2;  // bytes per group of scales
  const uint32_t o_s = (uint32_t)(W_BYTES + X_BYTES) + sgrp * s_row +
                       (SWIGLU ? mi * ng * s_row : mi * 64 * 2) + gr * 2;
  const int tid = threadIdx.x - 32;
  int s = 0;
  uint32_t ph = 0;
  for (int i = blockIdx.x; i < S.total; i += gridDim.x) {
    const W4Tile t = decode(S, g, i);
    const int ks = (g.k[t.kind] + KS - 1) / KS;
    const bool two = t.rows > 8;
    float acc[4][TOK / 8][4];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int n = 0; n < TOK / 8; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[a][n][q] = 0.f;
    int ok = 1;
    for (int kb = 0; kb < ks; ++kb) {
      if (lane == 0) ok = mbar_wait(&full[s], ph, abort_flag, g.err) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      const uint32_t st = base + s * STAGE_BYTES;
      if (two)
        stage_mma<2, G32>(acc, st + o_w, st + o_x, st + o_s, s_row, ki, gr, t4);
      else
        stage_mma<1, G32>(acc, st + o_w, st + o_x, st + o_s, s_row, ki, gr, t4);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      if (++s == STAGES) { s = 0; ph ^= 1; }
    }
    // the four ki of each row, eight tokens at a time, in a fixed order
    const int n_out = g.n[t.kind];
    __nv_bfloat16* out = g.out[t.kind];
    bool stop = false;
#pragma unroll
    for (int n = 0; n < TOK / 8; ++n) {
      if (n * 8 >= t.rows) break;
      if (sync_any(!ok)) { stop = true; break; }
      float* w = red + cw * (64 * 8);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        float* q = w + (a * 16 + gr) * 8 + t4;
        q[0] = acc[a][n][0];
        q[4] = acc[a][n][1];
        q[64] = acc[a][n][2];
        q[68] = acc[a][n][3];
      }
      if (sync_any(!ok)) { stop = true; break; }
      auto sum = [&](int row, int c) {  // weight row of the tile, token
        const float* q = red + (row >> 6) * (4 * 64 * 8) + (row & 63) * 8 + c;
        return ((q[0] + q[64 * 8]) + q[2 * 64 * 8]) + q[3 * 64 * 8];
      };
      if (SWIGLU) {
        const int f = tid & 63;
        if (t.f0 + f < n_out)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int c = (tid >> 6) * 2 + u;
            if (n * 8 + c < t.rows)
              out[(t.row0 + n * 8 + c) * n_out + t.f0 + f] =
                  __float2bfloat16_rn(silu_f(sum(f, c)) * sum(64 + f, c));
          }
      } else {
        const int f = tid & 127;
        if (t.f0 + f < n_out)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int c = (tid >> 7) * 4 + u;
            if (n * 8 + c < t.rows)
              out[(t.row0 + n * 8 + c) * n_out + t.f0 + f] = __float2bfloat16_rn(sum(f, c));
          }
      }
    }
    if (stop) break;
  }
}

}  // namespace

cudaError_t launch_quantize_w4(bool bf16, const void* w, int64_t E, int n, int k, int group,
                               uint8_t* q, __nv_bfloat16* scales, cudaStream_t st) {
  const int64_t rows = E * n, units = rows * ceil_div(k, 256);
  const int64_t ctas = ceil_div<int64_t>(units, 8);
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  if (bf16)
    quantize_w4_kernel<<<(unsigned)ctas, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(w), rows, n,
                                                       k, group, q, scales);
  else
    quantize_w4_kernel<<<(unsigned)ctas, 256, 0, st>>>(static_cast<const float*>(w), rows, n, k,
                                                       group, q, scales);
  return cudaGetLastError();
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

template <bool SWIGLU, bool G32>
cudaError_t launch_w4_kernel(const W4Args& g, const W4Tma& m, int ctas, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(w4_kernel<SWIGLU, G32>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
  if (e != cudaSuccess) return e;
  w4_kernel<SWIGLU, G32><<<ctas, NUM_THREADS, SMEM_BYTES, st>>>(g, m);
  return cudaGetLastError();
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
    bound += (int64_t)ceil_div(n, (int)fw) * (rows / TOK + (kind == 0 && rows > E ? E : rows));
  }
  if (bound == 0) return cudaSuccess;
  const int ctas = (int)(bound < 2 * num_sms ? bound : 2 * num_sms);
  if (swiglu)
    return g.group == 32 ? launch_w4_kernel<true, true>(g, m, ctas, st)
                         : launch_w4_kernel<true, false>(g, m, ctas, st);
  return g.group == 32 ? launch_w4_kernel<false, true>(g, m, ctas, st)
                       : launch_w4_kernel<false, false>(g, m, ctas, st);
}

}  // namespace moe
