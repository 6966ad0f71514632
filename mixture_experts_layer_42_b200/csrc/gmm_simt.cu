// Grouped products by expert on the CUDA cores (fp32 FMA): the fp32 calls of
// moe_grouped_matmul, _dx and _dw (tensor cores have no full-precision fp32
// product), and a cross-check of the tensor-core kernel for bf16.
//
// One kernel for the three products. Out tile [i][j], reduced over t:
//   FWD  i row of the expert, j output, t input:  A x[row][t],  B w[e][j][t]
//   DX   i row, j input, t output:                A dy[row][t], B w[e][t][j]
//   DW   i output, j input, t row:                A dy[t][i],   B x[t][j]
#include "gmm.cuh"

namespace moe {

namespace {

constexpr int GM = 128, GN = 128, GK = 16, GPAD = 4;

// Four consecutive elements as fp32 (8- or 16-byte aligned by the shapes' rule).
template <typename T> __device__ __forceinline__ float4 load4(const T* p);
template <> __device__ __forceinline__ float4 load4<float>(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <> __device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                     __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
}

// A 128 x 16 operand slice in registers, then in shared memory as S[t][i].
// ALONG_T: t is contiguous in memory (element (i, t) at p[i * ld + t]), else i
// is (p[t * ld + i]). Out-of-range elements read as zeros.
template <typename T, bool ALONG_T>
struct Slice {
  float4 v[2];
  __device__ __forceinline__ void load(const T* p, int64_t ld, int i0, int ni, int t0, int64_t nt) {
    const int tid = threadIdx.x;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = ALONG_T ? tid / 4 + 64 * u : (tid % 32) * 4;
      const int t = ALONG_T ? (tid % 4) * 4 : tid / 32 + 8 * u;
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + i < ni && t0 + t < nt)
        v[u] = load4<T>(p + (ALONG_T ? (int64_t)(i0 + i) * ld + t0 + t : (int64_t)(t0 + t) * ld + i0 + i));
    }
  }
  __device__ __forceinline__ void store(float (*S)[GM + GPAD]) const {
    const int tid = threadIdx.x;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (ALONG_T) {
        const int i = tid / 4 + 64 * u, t = (tid % 4) * 4;
        S[t + 0][i] = v[u].x;
        S[t + 1][i] = v[u].y;
        S[t + 2][i] = v[u].z;
        S[t + 3][i] = v[u].w;
      } else {
        *reinterpret_cast<float4*>(&S[tid / 32 + 8 * u][(tid % 32) * 4]) = v[u];
      }
    }
  }
};

template <typename T, typename TO, int MODE>
__global__ void __launch_bounds__(256, 2) gmm_simt_kernel(const GmmArgs g) {
  __shared__ __align__(16) float As[2][GK][GM + GPAD];
  __shared__ __align__(16) float Bs[2][GK][GN + GPAD];
  __shared__ int s_e, s_m;
  const int tid = threadIdx.x;

  // this CTA's expert and, for FWD and DX, its m-tile among the expert's rows
  const int NJ = MODE == GMM_FWD ? g.n : g.k;
  const int nj = ceil_div(NJ, GN);  // column tiles, fastest over the CTAs
  int e, i0 = 0, jt;
  if (MODE == GMM_DW) {
    const int per = nj * ceil_div(g.n, GM);
    e = blockIdx.x / per;
    i0 = blockIdx.x % per / nj * GM;
    jt = blockIdx.x % nj;
    if (tid == 0 && blockIdx.x % per == 0 && expert_span(g.offsets, e, g.rows).bad)
      set_error(g.err, ERRBIT_BAD_INDEX);
  } else {
    __shared__ int wsum[8];
    const int lane = tid % 32, warp = tid / 32;
    if (tid == 0) s_e = -1;
    int loc[4], lsum = 0;
    bool bad = false;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int x = tid * 4 + u;
      loc[u] = 0;
      if (x < g.E) {
        const Span s = expert_span(g.offsets, x, g.rows);
        bad |= s.bad;
        loc[u] = ceil_div(s.count, GM);
      }
      lsum += loc[u];
    }
    if (bad && blockIdx.x == 0) set_error(g.err, ERRBIT_BAD_INDEX);
    int incl = lsum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int p = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += p;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int run = incl - lsum;
    for (int w = 0; w < warp; ++w) run += wsum[w];
    const int mi = blockIdx.x / nj;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (mi >= run && mi < run + loc[u]) {
        s_e = tid * 4 + u;
        s_m = mi - run;
      }
      run += loc[u];
    }
    __syncthreads();
    e = s_e;
    if (e < 0) return;
    i0 = s_m * GM;
    jt = blockIdx.x % nj;
  }
  const Span sp = expert_span(g.offsets, e, g.rows);
  const int j0 = jt * GN;
  const int NI = MODE == GMM_DW ? g.n : sp.count;
  const int64_t NT = MODE == GMM_FWD ? g.k : MODE == GMM_DX ? g.n : sp.count;

  const T* A = static_cast<const T*>(g.a) + (int64_t)sp.b * (MODE == GMM_FWD ? g.k : g.n);
  const T* B = static_cast<const T*>(g.b) +
               (MODE == GMM_DW ? (int64_t)sp.b * g.k : (int64_t)e * g.n * g.k);
  const int64_t lda = MODE == GMM_FWD ? g.k : g.n;
  const int64_t ldb = g.k;

  const int tm = tid / 16, tn = tid % 16;
  float acc[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;

  Slice<T, MODE != GMM_DW> sa;
  Slice<T, MODE == GMM_FWD> sb;
  const int nk = (int)ceil_div<int64_t>(NT, GK);
  if (nk > 0) {
    sa.load(A, lda, i0, NI, 0, NT);
    sb.load(B, ldb, j0, NJ, 0, NT);
    sa.store(As[0]);
    sb.store(Bs[0]);
    __syncthreads();
  }
  for (int kb = 0; kb < nk; ++kb) {
    const int cur = kb & 1;
    if (kb + 1 < nk) {
      sa.load(A, lda, i0, NI, (kb + 1) * GK, NT);
      sb.load(B, ldb, j0, NJ, (kb + 1) * GK, NT);
    }
#pragma unroll
    for (int t = 0; t < GK; ++t) {
      float a[8], b[8];
      *reinterpret_cast<float4*>(a) = *reinterpret_cast<const float4*>(&As[cur][t][tm * 4]);
      *reinterpret_cast<float4*>(a + 4) = *reinterpret_cast<const float4*>(&As[cur][t][64 + tm * 4]);
      *reinterpret_cast<float4*>(b) = *reinterpret_cast<const float4*>(&Bs[cur][t][tn * 4]);
      *reinterpret_cast<float4*>(b + 4) = *reinterpret_cast<const float4*>(&Bs[cur][t][64 + tn * 4]);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    if (kb + 1 < nk) {
      sa.store(As[cur ^ 1]);
      sb.store(Bs[cur ^ 1]);
      __syncthreads();
    }
  }

  // rows i and columns j of the tile, four columns at a time (NJ is a
  // multiple of 4)
  TO* out = static_cast<TO*>(g.out);
  const bool acc_in = MODE == GMM_DW && g.accumulate;
  if (acc_in && sp.count == 0) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int ii = i0 + (i / 4) * 64 + tm * 4 + i % 4;
    if (ii >= NI) continue;
    const int64_t row = MODE == GMM_DW ? (int64_t)e * g.n + ii : (int64_t)sp.b + ii;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = j0 + h * 64 + tn * 4;
      if (j >= NJ) continue;
      TO* o = out + row * NJ + j;
      float4 v = make_float4(acc[i][4 * h], acc[i][4 * h + 1], acc[i][4 * h + 2], acc[i][4 * h + 3]);
      if (acc_in) {
        const float4 old = load4<TO>(o);
        v = make_float4(old.x + v.x, old.y + v.y, old.z + v.z, old.w + v.w);
      }
      if (sizeof(TO) == 4) {
        *reinterpret_cast<float4*>(o) = v;
      } else {
        const __nv_bfloat162 p0 = __floats2bfloat162_rn(v.x, v.y), p1 = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&p0),
                                                  *reinterpret_cast<const uint32_t*>(&p1));
      }
    }
  }
}

template <typename T, typename TO, int MODE>
cudaError_t launch(const GmmArgs& g, cudaStream_t st) {
  // FWD and DX: at most rows / GM full m-tiles and one partial per expert
  const int64_t it = MODE == GMM_DW ? (int64_t)g.E * ceil_div(g.n, GM) : g.rows / GM + g.E;
  const int64_t ctas = it * ceil_div(MODE == GMM_FWD ? g.n : g.k, GN);
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  gmm_simt_kernel<T, TO, MODE><<<(unsigned)ctas, 256, 0, st>>>(g);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_mode(int mode, const GmmArgs& g, cudaStream_t st) {
  if (mode == GMM_FWD) return launch<T, T, GMM_FWD>(g, st);
  if (mode == GMM_DX) return launch<T, T, GMM_DX>(g, st);
  if (g.out_f32) return launch<T, float, GMM_DW>(g, st);
  return launch<T, T, GMM_DW>(g, st);
}

}  // namespace

cudaError_t launch_gmm_simt(int mode, bool bf16, const GmmArgs& g, cudaStream_t st) {
  return bf16 ? launch_mode<__nv_bfloat16>(mode, g, st) : launch_mode<float>(mode, g, st);
}

}  // namespace moe
