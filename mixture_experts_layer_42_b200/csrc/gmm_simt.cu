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

// A tile of M x N by 64 threads, each R rows x Q columns, in slices of K of the
// reduction, CTAS blocks per SM. What bounds large calls is the fma pipe, with
// few warps to hide its latency, and the last wave of tiles. 4084 skewed rows
// of 16 experts of 1032 x 2052: dx 415 us, dw 374 us (46 of the pipe's 74 TF),
// the product 556 us; tiles of 64 x 128 with 16 x 8 a thread (two warps a
// scheduler) and transposed slices took 442, 398 and 760 us. More blocks an SM
// spill (the product with 5: 997 us). Calls of few such tiles take small ones,
// whose K is deep because latency counts (19 -> 5 us for the tiny layer's
// up-projection).
struct Large { static constexpr int M = 64, N = 64, K = 16, R = 8, Q = 8, CTAS = 5, CTAS_FWD = 4; };
struct Small { static constexpr int M = 16, N = 64, K = 32, R = 4, Q = 4, CTAS = 4, CTAS_FWD = 4; };

// An operand's slice of W x K in shared memory, as it lies in memory: ALONG_T
// (t is contiguous, element (i, t) at p[i * ld + t]) by i, S[i][t], else (p[t *
// ld + i]) by t, S[t][i]. Out-of-range elements read as zeros. fp32 is copied
// asynchronously, bf16 widened through registers.
template <typename T, bool ALONG_T, int W, int K>
struct Slice {
  static constexpr bool ASYNC = sizeof(T) == 4;
  static constexpr int ROWS = ALONG_T ? W : K, LEN = ALONG_T ? K : W;
  static constexpr int LD = LEN + 4;               // no bank twice among 8 rows
  static constexpr int NV = W * K / 4 / GTHREADS;  // float4s of a thread
  using Tile = float[ROWS][LD];
  float4 v[ASYNC ? 1 : NV];
  // float4 u of this thread: its row and column of the slice
  __device__ __forceinline__ static int row(int u) { return (threadIdx.x + GTHREADS * u) / (LEN / 4); }
  __device__ __forceinline__ static int col(int u) { return (threadIdx.x + GTHREADS * u) % (LEN / 4) * 4; }
  // its address, or null out of range
  __device__ __forceinline__ static const T* at(int u, const T* p, int64_t ld, int i0, int ni, int t0,
                                                int64_t nt) {
    const int i = i0 + (ALONG_T ? row(u) : col(u)), t = t0 + (ALONG_T ? col(u) : row(u));
    return i < ni && t < nt ? p + (ALONG_T ? (int64_t)i * ld + t : (int64_t)t * ld + i) : nullptr;
  }
  __device__ __forceinline__ void load(const T* p, int64_t ld, int i0, int ni, int t0, int64_t nt) {
    if (ASYNC) return;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const T* q = at(u, p, ld, i0, ni, t0, nt);
      v[u] = q ? load4<T>(q) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __device__ __forceinline__ void store(Tile& S) const {
    if (ASYNC) return;
#pragma unroll
    for (int u = 0; u < NV; ++u) *reinterpret_cast<float4*>(&S[row(u)][col(u)]) = v[u];
  }
  __device__ __forceinline__ static void copy(Tile& S, const T* p, int64_t ld, int i0, int ni, int t0, int64_t nt) {
    if (!ASYNC) return;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const T* q = at(u, p, ld, i0, ni, t0, nt);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                       (uint32_t)__cvta_generic_to_shared(&S[row(u)][col(u)])),
                   "l"(q ? q : p), "r"(q ? 16 : 0)
                   : "memory");
    }
  }
};

// Which row (column) of the tile a thread's q-th is, of NT threads side by
// side: of a slice by i every NT-th (8 threads' 16-byte reads then meet no bank
// twice), of one by t four neighbours in one read.
template <bool ALONG_T, int NT> __device__ __forceinline__ int owned(int q, int thread) {
  return ALONG_T ? thread + NT * q : q / 4 * 4 * NT + thread * 4 + q % 4;
}

// (d0, d1) += (a0 b0, a1 b1): two fp32 fmas in one instruction.
__device__ __forceinline__ void fma2(uint64_t& d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
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

__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}

// A slice's products: RV of a thread's R rows by its Q columns. Two fmas an
// instruction: where both operands lie by i, those of two t (a sum of the even
// t and one of the odd; no operand moves), else those of two columns.
template <int MODE, typename C, int RV, typename SA, typename SB, int NACC>
__device__ __forceinline__ void multiply(uint64_t (&acc)[C::R][NACC], const typename SA::Tile& As,
                                         const typename SB::Tile& Bs, int tm, int tn) {
  constexpr int NTN = C::N / C::Q, NTM = GTHREADS / NTN;
#pragma unroll
  for (int t = 0; t < C::K; t += 4) {
    float4 a[RV];  // MODE != DW: rows, four t
    if (MODE != GMM_DW)
#pragma unroll
      for (int q = 0; q < RV; ++q)
        a[q] = *reinterpret_cast<const float4*>(&As[owned<true, NTM>(q, tm)][t]);
    if (MODE == GMM_FWD) {
#pragma unroll
      for (int j = 0; j < C::Q; ++j) {
        const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(&Bs[owned<true, NTN>(j, tn)][t]);
#pragma unroll
        for (int q = 0; q < RV; ++q) {
          fma2(acc[q][j], pair(a[q].x, a[q].y), b.x);
          fma2(acc[q][j], pair(a[q].z, a[q].w), b.y);
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        ulonglong2 b[C::Q / 4];
#pragma unroll
        for (int h = 0; h < C::Q / 4; ++h)
          b[h] = *reinterpret_cast<const ulonglong2*>(&Bs[t + v][owned<false, NTN>(4 * h, tn)]);
        float4 d[RV / 4];  // DW: rows of this t
        if (MODE == GMM_DW)
#pragma unroll
          for (int h = 0; h < RV / 4; ++h)
            d[h] = *reinterpret_cast<const float4*>(&As[t + v][owned<false, NTM>(4 * h, tm)]);
#pragma unroll
        for (int q = 0; q < RV; ++q) {
          const float x = MODE == GMM_DW ? reinterpret_cast<const float*>(&d[q / 4])[q % 4]
                                         : reinterpret_cast<const float*>(&a[q])[v];
          const uint64_t xx = pair(x, x);
#pragma unroll
          for (int h = 0; h < C::Q / 4; ++h) {
            fma2(acc[q][2 * h], xx, b[h].x);
            fma2(acc[q][2 * h + 1], xx, b[h].y);
          }
        }
      }
    }
  }
}

template <typename T, typename TO, int MODE, typename C>
__global__ void __launch_bounds__(GTHREADS, MODE == GMM_FWD ? C::CTAS_FWD : C::CTAS)
    gmm_simt_kernel(const GmmArgs g) {
  constexpr int GM = C::M, GN = C::N, GK = C::K;
  constexpr int NTN = GN / C::Q, NTM = GTHREADS / NTN;  // threads over columns, rows
  static_assert(NTM * C::R == GM, "threads cover the tile");
  using SA = Slice<T, MODE != GMM_DW, GM, GK>;
  using SB = Slice<T, MODE == GMM_FWD, GN, GK>;
  constexpr int NS = 3;  // slices in shared memory
  __shared__ __align__(16) typename SA::Tile As[NS];
  __shared__ __align__(16) typename SB::Tile Bs[NS];
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

  const int tm = tid / NTN, tn = tid % NTN;
  constexpr int NACC = MODE == GMM_FWD ? C::Q : C::Q / 2;
  uint64_t acc[C::R][NACC];
#pragma unroll
  for (int q = 0; q < C::R; ++q)
#pragma unroll
    for (int j = 0; j < NACC; ++j) acc[q][j] = 0;

  // a tile of at most half its rows multiplies no others
  const bool half = C::R > 4 && NI - i0 <= GM / 2;
  // Slice kb is multiplied after a barrier that follows its arrival. By then
  // the copies of slice kb + 2 are asked for (into the place of slice kb - 1,
  // which the barrier says is done with) and the loads of slice kb + 1, which
  // is stored after the products.
  SA sa;
  SB sb;
  const int nk = (int)ceil_div<int64_t>(NT, GK);
  sa.load(A, lda, i0, NI, 0, NT);
  sb.load(B, ldb, j0, NJ, 0, NT);
#pragma unroll
  for (int p = 0; p < NS - 1; ++p) {
    SA::copy(As[p], A, lda, i0, NI, p * GK, NT);
    SB::copy(Bs[p], B, ldb, j0, NJ, p * GK, NT);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  sa.store(As[0]);
  sb.store(Bs[0]);
  int cur = 0;
  for (int kb = 0; kb < nk; ++kb) {
    asm volatile("cp.async.wait_group %0;" ::"n"(NS - 2) : "memory");
    __syncthreads();
    const int nxt = cur + 1 == NS ? 0 : cur + 1, far = cur == 0 ? NS - 1 : cur - 1;
    const int t1 = (kb + 1) * GK;
    SA::copy(As[far], A, lda, i0, NI, t1 + GK, NT);
    SB::copy(Bs[far], B, ldb, j0, NJ, t1 + GK, NT);
    asm volatile("cp.async.commit_group;" ::: "memory");
    sa.load(A, lda, i0, NI, t1, NT);
    sb.load(B, ldb, j0, NJ, t1, NT);
    if (half) multiply<MODE, C, (C::R > 4 ? C::R / 2 : C::R), SA, SB>(acc, As[cur], Bs[cur], tm, tn);
    else multiply<MODE, C, C::R, SA, SB>(acc, As[cur], Bs[cur], tm, tn);
    sa.store(As[nxt]);
    sb.store(Bs[nxt]);
    cur = nxt;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");

  TO* out = static_cast<TO*>(g.out);
  const bool acc_in = MODE == GMM_DW && g.accumulate;
  if (acc_in && sp.count == 0) return;
#pragma unroll
  for (int q = 0; q < C::R; ++q) {
    const int i = i0 + owned<MODE != GMM_DW, NTM>(q, tm);
    if (i >= NI) continue;
    TO* o = out + (MODE == GMM_DW ? (int64_t)e * g.n + i : (int64_t)sp.b + i) * NJ;
    const float* f = reinterpret_cast<const float*>(acc[q]);
    if (MODE == GMM_FWD) {
#pragma unroll
      for (int c = 0; c < C::Q; ++c) {
        const int j = j0 + owned<true, NTN>(c, tn);
        if (j < NJ) o[j] = from_f32<TO>(f[2 * c] + f[2 * c + 1]);
      }
    } else {
      // four columns at a time (NJ is a multiple of 4)
#pragma unroll
      for (int h = 0; h < C::Q / 4; ++h) {
        const int j = j0 + owned<false, NTN>(4 * h, tn);
        if (j >= NJ) continue;
        float4 v = make_float4(f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]);
        if (acc_in) {
          const float4 old = load4<TO>(o + j);
          v = make_float4(old.x + v.x, old.y + v.y, old.z + v.z, old.w + v.w);
        }
        if (sizeof(TO) == 4) {
          *reinterpret_cast<float4*>(o + j) = v;
        } else {
          const __nv_bfloat162 p0 = __floats2bfloat162_rn(v.x, v.y), p1 = __floats2bfloat162_rn(v.z, v.w);
          *reinterpret_cast<uint2*>(o + j) = make_uint2(*reinterpret_cast<const uint32_t*>(&p0),
                                                        *reinterpret_cast<const uint32_t*>(&p1));
        }
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
  // Small tiles fill the GPU sooner; large ones read shared memory less. Small
  // against large, us, by the large tiles: products and dx 288: 71 / 104 and
  // 74 / 95; 640: 70 / 75 and 73 / 82; 768 (few rows an expert): 87 / 116;
  // 1343: 542 / 556; 2176: 862 / 803; 2607 (dx): 533 / 415. dw, whose count is
  // exact: 256: 15.4 / 15.6; 512: 15.9 / 14.3; 2048: 35 / 20.
  const bool small = ctas_of<Large>(MODE, g) <= (int64_t)num_sms * (MODE == GMM_DW ? 2 : 8);
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
