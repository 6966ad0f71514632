// Products with 4-bit weights and group scales, grouped by expert, and the
// quantizer of their layout: codes 0..15, two to a byte along k, the lower
// input in the low half; w[i][j] = (code - 8) * scale[j / group][i].
#include "w4.cuh"

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

constexpr int WROWS = 4;  // rows a warp carries through one reading of its weights

// sum over 8 inputs of (code - 8) x
__device__ __forceinline__ float dot8(uint32_t c, const uint4& xv) {
  const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
  float s = 0.f;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    s = fmaf((float)((int)((c >> (8 * u)) & 15u) - 8), __uint_as_float(xw[u] << 16), s);
    s = fmaf((float)((int)((c >> (8 * u + 4)) & 15u) - 8), __uint_as_float(xw[u] & 0xffff0000u), s);
  }
  return s;
}

// A warp per output of an expert: lanes along k, 8 inputs each; the expert's
// rows in runs of WROWS.
template <bool SWIGLU>
__global__ void __launch_bounds__(256) w4_kernel(const W4Args g) {
  const int kind = blockIdx.y < (unsigned)g.E ? 0 : 1;
  const int e = kind == 0 ? blockIdx.y : 0;
  const int n = g.n[kind], k = g.k[kind];
  const int i = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x % 32;
  int64_t row0 = 0, count = g.t_shared;
  if (kind == 0) {
    const Span sp = expert_span(g.offsets, e, g.rows);
    if (sp.bad && threadIdx.x == 0 && blockIdx.x == 0) set_error(g.err, ERRBIT_BAD_INDEX);
    row0 = sp.b;
    count = sp.count;
  }
  if (i >= n) return;
  const uint8_t* q1 = g.q1[kind] + ((int64_t)e * n + i) * (k / 2);
  const uint8_t* q3 = SWIGLU ? g.q3[kind] + ((int64_t)e * n + i) * (k / 2) : nullptr;
  const __nv_bfloat16* s1 = g.s1[kind] + (int64_t)e * (k / g.group) * n + i;
  const __nv_bfloat16* s3 = SWIGLU ? g.s3[kind] + (int64_t)e * (k / g.group) * n + i : nullptr;
  for (int64_t r0 = 0; r0 < count; r0 += WROWS) {
    const __nv_bfloat16* xr[WROWS];
    float a[WROWS], b[WROWS];
#pragma unroll
    for (int u = 0; u < WROWS; ++u) {
      a[u] = b[u] = 0.f;
      xr[u] = nullptr;
      if (r0 + u < count) {
        int64_t t = row0 + r0 + u;
        if (kind == 0 && g.src != nullptr) {
          t = g.src[t];
          if (t < 0 || t >= g.x_rows) {
            if (lane == 0 && i == 0) set_error(g.err, ERRBIT_BAD_INDEX);
            t = -1;
          }
        }
        if (t >= 0) xr[u] = g.x[kind] + t * k;
      }
    }
    for (int j = lane * 8; j < k; j += 256) {
      const uint32_t c1 = *reinterpret_cast<const uint32_t*>(q1 + j / 2);
      const float w1 = __bfloat162float(s1[(int64_t)(j / g.group) * n]);
      const uint32_t c3 = SWIGLU ? *reinterpret_cast<const uint32_t*>(q3 + j / 2) : 0;
      const float w3 = SWIGLU ? __bfloat162float(s3[(int64_t)(j / g.group) * n]) : 0.f;
#pragma unroll
      for (int u = 0; u < WROWS; ++u) {
        if (xr[u] == nullptr) continue;
        const uint4 xv = *reinterpret_cast<const uint4*>(xr[u] + j);
        a[u] = fmaf(w1, dot8(c1, xv), a[u]);
        if (SWIGLU) b[u] = fmaf(w3, dot8(c3, xv), b[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < WROWS; ++u) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        a[u] += __shfl_xor_sync(0xffffffffu, a[u], o);
        if (SWIGLU) b[u] += __shfl_xor_sync(0xffffffffu, b[u], o);
      }
      if (lane == 0 && r0 + u < count)
        g.out[kind][(row0 + r0 + u) * n + i] = __float2bfloat16_rn(SWIGLU ? silu_f(a[u]) * b[u] : a[u]);
    }
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

cudaError_t launch_w4(bool swiglu, const W4Args& g, cudaStream_t st) {
  const int n = g.t_shared > 0 && g.n[1] > g.n[0] ? g.n[1] : g.n[0];
  const dim3 grid((unsigned)ceil_div(n, 8), (unsigned)(g.E + (g.t_shared > 0 ? 1 : 0)));
  if (swiglu) w4_kernel<true><<<grid, 256, 0, st>>>(g);
  else w4_kernel<false><<<grid, 256, 0, st>>>(g);
  return cudaGetLastError();
}

}  // namespace moe
