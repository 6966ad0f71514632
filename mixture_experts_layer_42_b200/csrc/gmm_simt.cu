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

constexpr int GTHREADS = 64;

// A tile of M x N by 64 threads, each 4 RM rows x 4 CN columns, in slices of
// K of the reduction. What bounds large calls is the fma pipe, and next to it
// shared memory's reads: 16 x 8 a thread needs 6 reads of 16 bytes for 64
// packed fmas (8 x 8 needs 4 for 32, and shared memory bounds it: 590 us of
// the odd fp32 input gradient's sizes against 540). Calls whose large tiles
// would not fill the GPU take small ones, whose K is deep because latency
// counts (19 -> 6 us for the tiny layer's up-projection).
struct Large { static constexpr int M = 64, N = 128, K = 8, RM = 4, CN = 2, CTAS = 4; };
struct Small { static constexpr int M = 16, N = 64, K = 32, RM = 1, CN = 1, CTAS = 4; };

// An operand slice of W x K in registers, then in shared memory by t: S[t][i].
// ALONG_T: t is contiguous in memory (element (i, t) at p[i * ld + t]), else i
// is (p[t * ld + i]). Out-of-range elements read as zeros.
template <typename T, bool ALONG_T, int W, int K>
struct Slice {
  static constexpr int LD = W + 4;
  static constexpr int NV = W * K / 4 / GTHREADS;  // float4s a thread carries
  float4 v[NV];
  static constexpr int TPT = GTHREADS / K;         // threads per t (not ALONG_T)
  __device__ __forceinline__ static int at_i(int u) {
    return ALONG_T ? (threadIdx.x + GTHREADS * u) % W : (threadIdx.x % TPT + TPT * u) * 4;
  }
  __device__ __forceinline__ static int at_t(int u) {
    return ALONG_T ? (threadIdx.x + GTHREADS * u) / W * 4 : threadIdx.x / TPT;
  }
  __device__ __forceinline__ void load(const T* p, int64_t ld, int i0, int ni, int t0, int64_t nt) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int i = i0 + at_i(u), t = t0 + at_t(u);
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < ni && t < nt) v[u] = load4<T>(p + (ALONG_T ? (int64_t)i * ld + t : (int64_t)t * ld + i));
    }
  }
  __device__ __forceinline__ void store(float (*S)[LD]) const {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int i = at_i(u), t = at_t(u);
      if (ALONG_T) {
        S[t + 0][i] = v[u].x;
        S[t + 1][i] = v[u].y;
        S[t + 2][i] = v[u].z;
        S[t + 3][i] = v[u].w;
      } else {
        *reinterpret_cast<float4*>(&S[t][i]) = v[u];
      }
    }
  }
};

// (d0, d1) += (a0 b0, a1 b1): two fp32 fmas in one instruction.
__device__ __forceinline__ void fma2(uint64_t& d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}

__device__ __forceinline__ uint64_t twice(float a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(a));
  return r;
}

// This CTA's expert and, for FWD and DX, its tile among the expert's rows:
// the row tiles of all experts, in order, are blockIdx.x / nj.
template <int GM>
__device__ __forceinline__ bool find_tile(const GmmArgs& g, int mi, int* e_out, int* m_out) {
  __shared__ int s_e, s_m, wsum[GTHREADS / 32];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int per = ceil_div(g.E, GTHREADS);
  if (tid == 0) s_e = -1;
  int lsum = 0;
  bool bad = false;
#pragma unroll 4
  for (int u = 0; u < per; ++u) {
    const int x = tid * per + u;
    if (x < g.E) {
      const Span s = expert_span(g.offsets, x, g.rows);
      bad |= s.bad;
      lsum += ceil_div(s.count, GM);
    }
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
  if (mi >= run && mi < run + lsum)
    for (int u = 0; u < per; ++u) {
      const int x = tid * per + u;
      const int n = x < g.E ? ceil_div(expert_span(g.offsets, x, g.rows).count, GM) : 0;
      if (mi >= run && mi < run + n) {
        s_e = x;
        s_m = mi - run;
      }
      run += n;
    }
  __syncthreads();
  *e_out = s_e;
  *m_out = s_m;
  return s_e >= 0;
}

// A slice's products: a thread's 4 RMV rows by 4 CN columns.
template <typename C, int RMV, int LDA, int LDB>
__device__ __forceinline__ void multiply(uint64_t (&acc)[4 * C::RM][2 * C::CN], const float (*As)[LDA],
                                         const float (*Bs)[LDB], int tm, int tn) {
  constexpr int NTN = C::N / (4 * C::CN), NTM = GTHREADS / NTN;
#pragma unroll 8
  for (int t = 0; t < C::K; ++t) {
    float a[4 * C::RM];
    ulonglong2 b[C::CN];  // pairs of columns
#pragma unroll
    for (int h = 0; h < RMV; ++h)
      *reinterpret_cast<float4*>(a + 4 * h) = *reinterpret_cast<const float4*>(&As[t][4 * NTM * h + 4 * tm]);
#pragma unroll
    for (int h = 0; h < C::CN; ++h)
      b[h] = *reinterpret_cast<const ulonglong2*>(&Bs[t][4 * NTN * h + 4 * tn]);
#pragma unroll
    for (int i = 0; i < 4 * RMV; ++i) {
      const uint64_t ai = twice(a[i]);
#pragma unroll
      for (int h = 0; h < C::CN; ++h) {
        fma2(acc[i][2 * h], ai, b[h].x);
        fma2(acc[i][2 * h + 1], ai, b[h].y);
      }
    }
  }
}

template <typename T, typename TO, int MODE, typename C>
__global__ void __launch_bounds__(GTHREADS, C::CTAS) gmm_simt_kernel(const GmmArgs g) {
  constexpr int GM = C::M, GN = C::N, GK = C::K;
  constexpr int NTN = GN / (4 * C::CN), NTM = GTHREADS / NTN;  // threads over columns, rows
  static_assert(NTM * 4 * C::RM == GM, "threads cover the tile");
  using SA = Slice<T, MODE != GMM_DW, GM, GK>;
  using SB = Slice<T, MODE == GMM_FWD, GN, GK>;
  __shared__ __align__(16) float As[2][GK][SA::LD];
  __shared__ __align__(16) float Bs[2][GK][SB::LD];
  grid_dependency();
  const int tid = threadIdx.x;
  const int NJ = MODE == GMM_FWD ? g.n : g.k;
  const int nj = ceil_div(NJ, GN);  // column tiles, fastest over the CTAs
  int e, i0;
  const int jt = blockIdx.x % nj;
  if (MODE == GMM_DW) {
    const int per = nj * ceil_div(g.n, GM);
    e = blockIdx.x / per;
    i0 = blockIdx.x % per / nj * GM;
    if (tid == 0 && blockIdx.x % per == 0 && expert_span(g.offsets, e, g.rows).bad)
      set_error(g.err, ERRBIT_BAD_INDEX);
  } else {
    int m;
    if (!find_tile<GM>(g, blockIdx.x / nj, &e, &m)) return;
    i0 = m * GM;
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

  // a thread's rows 4 NTM h + 4 tm .., its columns 4 NTN h + 4 tn ..
  const int tm = tid / NTN, tn = tid % NTN;
  uint64_t acc[4 * C::RM][2 * C::CN];
#pragma unroll
  for (int i = 0; i < 4 * C::RM; ++i)
#pragma unroll
    for (int j = 0; j < 2 * C::CN; ++j) acc[i][j] = 0;

  // a tile of at most half its rows multiplies no others
  const bool half = MODE != GMM_DW && C::RM > 1 && NI - i0 <= GM / 2;
  SA sa;
  SB sb;
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
    if (half) multiply<C, C::RM / 2>(acc, As[cur], Bs[cur], tm, tn);
    else multiply<C, C::RM>(acc, As[cur], Bs[cur], tm, tn);
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
  for (int i = 0; i < 4 * C::RM; ++i) {
    const int ii = i0 + (i / 4) * 4 * NTM + tm * 4 + i % 4;
    if (ii >= NI) continue;
    const int64_t row = MODE == GMM_DW ? (int64_t)e * g.n + ii : (int64_t)sp.b + ii;
#pragma unroll
    for (int h = 0; h < C::CN; ++h) {
      const int j = j0 + h * 4 * NTN + tn * 4;
      if (j >= NJ) continue;
      TO* o = out + row * NJ + j;
      const float* f = reinterpret_cast<const float*>(&acc[i][2 * h]);
      float4 v = make_float4(f[0], f[1], f[2], f[3]);
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

// CTAs of a launch. FWD and DX: at most rows / M full row tiles and one partial
// per expert.
template <typename C>
int64_t ctas_of(int mode, const GmmArgs& g) {
  const int64_t it = mode == GMM_DW ? (int64_t)g.E * ceil_div(g.n, C::M)
                                    : g.rows / C::M + (g.rows < g.E ? g.rows : g.E);
  return it * ceil_div(mode == GMM_FWD ? g.n : g.k, C::N);
}

template <typename T, typename TO, int MODE>
cudaError_t launch(const GmmArgs& g, int num_sms, cudaStream_t st) {
  const bool small = ctas_of<Large>(MODE, g) <= num_sms;
  const int64_t ctas = small ? ctas_of<Small>(MODE, g) : ctas_of<Large>(MODE, g);
  if (ctas == 0) return cudaSuccess;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)ctas), block(GTHREADS);
  return small ? launch_pdl(true, gmm_simt_kernel<T, TO, MODE, Small>, grid, block, 0, st, g)
               : launch_pdl(true, gmm_simt_kernel<T, TO, MODE, Large>, grid, block, 0, st, g);
}

template <typename T>
cudaError_t launch_mode(int mode, const GmmArgs& g, int num_sms, cudaStream_t st) {
  if (mode == GMM_FWD) return launch<T, T, GMM_FWD>(g, num_sms, st);
  if (mode == GMM_DX) return launch<T, T, GMM_DX>(g, num_sms, st);
  if (g.out_f32) return launch<T, float, GMM_DW>(g, num_sms, st);
  return launch<T, T, GMM_DW>(g, num_sms, st);
}

}  // namespace

cudaError_t launch_gmm_simt(int mode, bool bf16, const GmmArgs& g, int num_sms, cudaStream_t st) {
  return bf16 ? launch_mode<__nv_bfloat16>(mode, g, num_sms, st) : launch_mode<float>(mode, g, num_sms, st);
}

}  // namespace moe
