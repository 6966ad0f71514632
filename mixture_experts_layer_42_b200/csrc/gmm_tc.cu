// Grouped products by expert on the tensor cores (bf16): moe_grouped_matmul
// and its gradients, one persistent kernel on CTA pairs.
//
//   FWD  y[r]  = W_e x[r]      M = outputs of W_e, N = rows, reduced over inputs
//   DX   dx[r] = W_e^T dy[r]   M = inputs of W_e,  N = rows, reduced over outputs
//   DW   dW_e  = sum dy x^T    M = outputs, N = inputs, reduced over e's rows
//
// The features are the MMA's M side (256 over a pair, cta_group::2) and the
// token rows its N side, whose width follows the tile's rows in steps of 32:
// an expert's last rows cost what they are, where 128- or 256-row tiles would
// pad them, and a decode batch's few rows need no form of their own. A tile
// has one or two halves of up to 256 N columns, each in one of the two TMEM
// accumulators: two halves read their weights' tile once for up to 512 rows.
//
// Shared-memory tiles are 128-byte-swizzled, 64 deep in the reduction.
// K-major operands (x, dy and w in FWD; dy in DX): rows of 64 reduction
// elements. MN-major operands (w in DX, dy and x in DW): 64 reduction rows of
// 64 features each, 8 KB a box; the matrix descriptor's leading offset steps
// over the boxes (64 features), its stride over 8 reduction rows.
//
// Stages of the shared-memory ring are as large as their tile's operands, so
// that the same 192 KB hold 10 stages of a decode tile and 4 of a tile of 512
// rows: what covers the memory's latency is bytes in flight.
//
// Per CTA, 352 threads: warp 0 the TMA producer, warp 1 of the pair's leader
// the MMA issuer, warps 2-9 the epilogue (two warps on each 32 TMEM lanes, in
// turn over the columns), warp 10 the scheduler, which works the tiles out
// ahead of the others. Rows leave through a warp's own shared memory (the
// accumulator holds features by rows), dw straight from registers. Rows of a
// tile past its expert's end are other rows of the matrix (their columns are
// not stored); only DW, which sums over rows, reads through per-expert maps
// that end at the expert's last row.
//
// What bounds it, and what it measured (V3 sizes, 256 experts of 2048 x 7168,
// cold; the memory's copy rate is 6.5 TB/s): 1024 rows read at 7.2 TB/s (1022
// us); 65536 rows 1700-1840 us and skewed 2120-2340 us, dw of 24576 rows of 64
// experts of 1408 x 2048 149-165 us and of 16384 rows of 32 of 2048 x 7168 in
// fp32 530-580 us, each at 10-11 TB/s between L2 and the SMs, dw's stores
// counted, and 0.85-1.15 PFLOP/s. A loop of seconds is bound by the 1 kW power
// cap (65536 rows: 2050-2250 us at 1.1-1.2 GHz). dw tiles of 256 x 512, whose
// write-out nothing overlaps for want of a second accumulator, took 233 and
// 653 us; a panel of dy kept over a row of tiles 190 and 757. Every wait is
// bounded (1 s, in DW and 4 us for each 64 rows of the call); on expiry the
// kernel raises the error word's timeout bit, drains its copies and returns.
#include "api_common.cuh"
#include "gmm.cuh"
#include "tc_common.cuh"

#include <cstring>

namespace moe {

namespace {

using namespace tc;

constexpr int BK = 64;                    // reduction depth of a stage (128 bytes)
constexpr int FM = 128;                   // features per CTA; a pair holds 256
constexpr int MAXN = 256;                 // N columns of one half
constexpr int TILE = FM * BK * 2;         // 16 KB: an operand tile of a stage
constexpr int NUM_THREADS = 352;
constexpr uint32_t TMEM_COLS = 512;
constexpr int MAX_E = 1024;
constexpr int NBOX = 9;                   // row boxes of 8, 16, 32, 48, ... 128 rows
constexpr int SLOTS = 12;                 // stages in flight, at most
constexpr int TQ = 4;                     // tiles the scheduler works out ahead
// DW: what a step of 64 rows adds to the waits' limit. The epilogue waits for
// a tile's whole reduction, and the scheduler's queue for the epilogue: all rows
// of an expert, up to 2^30. A step takes 0.1-0.8 us.
constexpr uint64_t STEP_LIMIT_NS = 4000;
// DW: steps summed in tensor memory, 768 rows. The tensor cores truncate every
// addition into their fp32 sums, which costs 1.1e-9 of the result a row: of
// 8192 random rows 9.1e-6, of 2^20 1.2e-3, and of 2^20 positive ones 9e-3.
// Longer reductions add such parts up in registers, where fp32 additions round:
// 7e-7 at any length (65536 rows of 8 experts of 2048 x 2048: 410 instead of
// 395 us; parts of 512 rows 417).
constexpr int PART = 12;

template <int MODE> struct Cfg {
  static constexpr int HALVES = MODE == GMM_DW ? 1 : 2;
  static constexpr int RING = MODE == GMM_DW ? 6 * 2 * TILE : 192 * 1024;
  // staging of an epilogue warp: 32 rows x 32 features in bf16
  static constexpr int STG = MODE == GMM_DW ? 0 : 2048;
  // experts' first rows and counts, and (FWD, DX) the prefixes of their tiles
  static constexpr int TABLE = (MODE == GMM_DW ? 2 : 3) * (MAX_E + 1) * 4;
  static constexpr size_t SMEM = 1024 + RING + 8 * STG + 512 + TABLE;
};

struct TcGmm {
  CUtensorMap tmA;          // FWD, DX: the weights
  CUtensorMap tmB[NBOX];    // FWD, DX: the rows, boxes of 8, 16, 32, 48, ... 128 rows
  const CUtensorMap* maps;  // DW: [2, E] maps of dy and of x ending at each expert's last row
  void* out;
  const int32_t* offsets;
  int64_t rows;
  int E, n, k;
  int out_f32, accumulate;
  int nw;                   // DW: inputs per tile
  int wide;                 // MN-major A by one box of 128 features (rows of whole 64s)
  int stall;                // test hook: CTA 0's MMA thread lets a wait run out
  uint64_t wait_ns;         // limit of each wait
  uint32_t* err;
};

// M features (over both CTAs of the pair), N columns and reduction depth.
struct Tile {
  int e;       // expert; -1: no more tiles
  int f0;      // first of the pair's 256 features
  int c0;      // first N column: row of the matrix (FWD, DX) or input (DW)
  int cols;    // valid N columns
  int halves;
  int nh;      // N columns of each half (a multiple of 32; the last may hold fewer valid)
  int depth;   // reduction elements
  int r0;      // DW: the expert's first row
};

struct Sched {
  const int32_t* off;  // smem: first row and number of rows of each expert
  const int32_t* cnt;
  const int32_t* P;    // smem: token-tile prefixes over experts [E + 1] (FWD, DX)
  int E, nf, nc, nw, total, n, k;
};

__device__ __forceinline__ int round32(int v) { return (v + 31) & ~31; }
__device__ __forceinline__ int tile_rows(int count, int mt) { return round32((count + mt - 1) / mt); }

// Tile i of the launch, expert by expert: its feature blocks, and the tiles
// that share a block's weights (FWD, DX: expert e's rows in mt tiles of
// tile_rows each) side by side. The experts' own order stands: the tiles of
// experts with many rows and of those with few in even turns, so that the MMAs
// of the one kind would run beside the other's bytes, took 1814 instead of
// 1518 us of 32768 skewed rows (Zipf 1.2 over 256 experts of 2048 x 7168).
template <int MODE>
__device__ __forceinline__ Tile decode(const Sched& S, int i) {
  Tile t;
  if (MODE == GMM_DW) {
    const int per = S.nf * S.nc;
    t.e = i / per;
    const int l = i % per;
    t.f0 = l / S.nc * (2 * FM);
    t.c0 = l % S.nc * S.nw;
    t.cols = min(S.nw, S.k - t.c0);
    t.halves = 1;
    t.nh = round32(t.cols);
    t.depth = S.cnt[t.e];
    t.r0 = S.off[t.e];
  } else {
    const int32_t* P = S.P;
    const int q = i / S.nf;
    int lo = 0, hi = S.E;  // the e with P[e] <= q < P[e + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (P[mid] <= q) lo = mid; else hi = mid;
    }
    t.e = lo;
    const int mt = P[lo + 1] - P[lo];
    const int l = i - S.nf * P[lo];
    t.f0 = l / mt * (2 * FM);
    const int c = S.cnt[lo], per = tile_rows(c, mt), m = l % mt;
    t.c0 = S.off[lo] + m * per;
    t.cols = min(per, c - m * per);
    t.halves = t.cols > MAXN ? 2 : 1;
    t.nh = t.halves == 2 ? round32((t.cols + 1) / 2) : round32(t.cols);
    t.depth = MODE == GMM_FWD ? S.k : S.n;
    t.r0 = 0;
  }
  return t;
}
// N columns of half h: all but a last half's missing steps of 32
__device__ __forceinline__ int half_n(const Tile& t, int h) {
  return h == t.halves - 1 ? round32(t.cols - h * t.nh) : t.nh;
}

// Matrix descriptors: the upper word is the same for both majors (128-byte
// swizzle, 8-row groups 1024 bytes apart), the lower holds the address / 16
// and the leading offset (MN-major: 8 KB boxes of 64 features; unused for
// K-major). A step of 16 in the reduction is 32 bytes of a K-major tile and
// 2048 bytes of an MN-major one.
constexpr uint32_t DESC_HI = (1024 >> 4) | (1u << 14) | (2u << 29);
template <bool MN> __device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) {
  return (saddr >> 4) | (MN ? (8192u >> 4) << 16 : 1u << 16);
}
template <bool MN> constexpr uint32_t K16 = MN ? 2048 >> 4 : 32 >> 4;

__device__ __forceinline__ void mma_pair_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(DESC_HI)
      : "memory");
}

// The MMAs of a stage: a0, b0, b1 its operands' lower descriptor words.
template <bool A_MN, bool B_MN, bool TWO>
__device__ __forceinline__ void mma_stage(uint32_t d0, uint32_t d1, uint32_t a0, uint32_t b0, uint32_t b1,
                                          uint32_t id0, uint32_t id1, uint32_t accumulate) {
#pragma unroll
  for (uint32_t kk = 0; kk < BK / 16; ++kk) {
    mma_pair_lo(d0, a0 + kk * K16<A_MN>, b0 + kk * K16<B_MN>, id0, kk == 0 ? accumulate : 1u);
    if (TWO) mma_pair_lo(d1, a0 + kk * K16<A_MN>, b1 + kk * K16<B_MN>, id1, kk == 0 ? accumulate : 1u);
  }
}

// Lane 0's values, for the compiler to hold in uniform registers.
__device__ __forceinline__ Tile uniform(Tile t) {
  t.e = __shfl_sync(0xffffffffu, t.e, 0);
  t.f0 = __shfl_sync(0xffffffffu, t.f0, 0);
  t.c0 = __shfl_sync(0xffffffffu, t.c0, 0);
  t.cols = __shfl_sync(0xffffffffu, t.cols, 0);
  t.halves = __shfl_sync(0xffffffffu, t.halves, 0);
  t.nh = __shfl_sync(0xffffffffu, t.nh, 0);
  t.depth = __shfl_sync(0xffffffffu, t.depth, 0);
  t.r0 = __shfl_sync(0xffffffffu, t.r0, 0);
  return t;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// A wait by the whole warp; all lanes agree on its outcome.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t* err,
                                         uint64_t limit) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, err, limit));
}

// A role's place in the scheduler's queue of tiles. next() reads a tile for
// the whole warp; false on an abort or when there are no more.
struct TileQueue {
  uint32_t q = 0, ph = 0;
  __device__ __forceinline__ bool next(Tile& t, const Tile* tq, uint64_t* qfull, uint64_t* qempty, int lane,
                                       volatile int* abort_flag, uint32_t* err, uint64_t limit) {
    if (!wait_all(&qfull[q], ph, abort_flag, err, limit)) return false;
    t = uniform(tq[q]);
    if (lane == 0) mbar_arrive(&qempty[q]);
    if (++q == TQ) { q = 0; ph ^= 1; }
    return t.e >= 0;
  }
};

// FWD, DX: which box brings the valid rows among a CTA's n / 2 columns of a
// half (-1: there are none), and its rows. What a box leaves of the columns
// holds an earlier stage's rows; results of such columns are not stored. Rows
// that are not needed are not read: a decode batch's 28 tiles of an expert
// all read its few rows, and 32 rows a stage instead of 8 cost the V3
// down-projection 18 % of its time.
__device__ __forceinline__ int row_box(int cols, int n, int rank) {
  const int need = min(cols - rank * (n / 2), n / 2);
  return need <= 0 ? -1 : need <= 8 ? 0 : (need + 15) >> 4;
}
__device__ __forceinline__ int box_rows(int box) { return box < 0 ? 0 : box == 0 ? 8 : 16 * box; }

// Stage of a tile: A, then the halves of B; the ring's position after it.
template <int MODE> __device__ __forceinline__ uint32_t stage_bytes(const Tile& t) {
  if (MODE == GMM_DW) return TILE + (t.nh > MAXN / 2 ? TILE : TILE / 2);  // boxes of 64 inputs
  const uint32_t n = (uint32_t)(half_n(t, 0) + (t.halves == 2 ? half_n(t, 1) : 0));
  return (TILE + n * BK + 1023) & ~1023u;
}

// Position in the ring of stages: its slot (barriers) and phase, and its byte
// offset. The same sequence in every role of both CTAs.
template <int MODE> struct Ring {
  uint32_t slot = 0, ph = 0, pos = 0, pad = 0;
  // where a stage of b bytes goes: at pos, or at the ring's start if it would
  // straddle the end
  __device__ __forceinline__ uint32_t place(uint32_t b) {
    pad = 0;
    if (pos + b > (uint32_t)Cfg<MODE>::RING) {
      pad = Cfg<MODE>::RING - pos;
      pos = 0;
    }
    return pos;
  }
  __device__ __forceinline__ void advance(uint32_t b) {
    pos += b;
    if (++slot == SLOTS) { slot = 0; ph ^= 1; }
  }
};

// The producer's account of the stages not yet known to be consumed, all in
// registers: the oldest run of equal-sized stages and the newest (a tile's
// stages are of one size), and where the oldest begins, as an offset into the
// ring and as a running count of the bytes given out (differences only).
template <int MODE> struct Outstanding {
  uint32_t old_n = 0, old_sz = 0, new_n = 0, new_sz = 0;
  uint32_t pos = 0, v = 0, vpos = 0;  // the oldest's offset and count; the next's count
  uint32_t slot = 0, ph = 0;          // the oldest's barrier
  __device__ __forceinline__ bool retire(uint64_t* empty, volatile int* abort_flag, uint32_t* err,
                                         uint64_t limit) {
    if (!wait_all(&empty[slot], ph, abort_flag, err, limit)) return false;
    if (++slot == SLOTS) { slot = 0; ph ^= 1; }
    pos += old_sz;
    v += old_sz;
    if (--old_n == 0) {
      old_n = new_n;
      old_sz = new_sz;
      new_n = 0;
    }
    if (pos + old_sz > (uint32_t)Cfg<MODE>::RING) {  // the next began at the ring's start
      v += Cfg<MODE>::RING - pos;
      pos = 0;
    }
    return true;
  }
  // before a tile of stages of sz bytes: two runs at most
  __device__ __forceinline__ bool begin(uint32_t sz, uint64_t* empty, volatile int* abort_flag, uint32_t* err,
                                        uint64_t limit) {
    while (new_n > 0 && new_sz != sz)
      if (!retire(empty, abort_flag, err, limit)) return false;
    return true;
  }
  // until `bytes` more (padding included) and a slot are free
  __device__ __forceinline__ bool make_room(uint32_t bytes, uint64_t* empty, volatile int* abort_flag,
                                            uint32_t* err, uint64_t limit) {
    while (old_n > 0 && (old_n + new_n == SLOTS || vpos + bytes - v > (uint32_t)Cfg<MODE>::RING))
      if (!retire(empty, abort_flag, err, limit)) return false;
    return true;
  }
  __device__ __forceinline__ void push(uint32_t sz, uint32_t at, uint32_t pad) {
    if (old_n == 0) {
      old_sz = sz;
      pos = at;
      v = vpos + pad;
    }
    if (new_n == 0 && old_sz == sz) {
      ++old_n;
    } else {
      new_sz = sz;
      ++new_n;
    }
    vpos += pad + sz;
  }
};

// Arrive on the leader's barrier that an accumulator's columns have been read.
// Relaxed: what it orders is the TMEM reads (tcgen05.wait::ld has completed
// them, tcgen05.fence::before_thread_sync precedes it); a release would also
// wait until L2 has taken the result's stores, ~3300 cycles a tile.
__device__ __forceinline__ void arrive_read(uint32_t remote_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote_bar) : "memory");
}

// 16 TMEM lanes x 32 columns: thread T gets of lanes T / 4 (r[4i], r[4i + 1])
// and T / 4 + 8 (r[4i + 2], r[4i + 3]) the columns 8i + 2 (T % 4) and the next.
__device__ __forceinline__ void tmem_ld16x32(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// A 32 x 32 block of dw (outputs x inputs) lies in a warp's registers as
// tmem_ld16x32 leaves its lanes 0-15 and 16-31; nr x nc of it are valid. Four
// threads hold 8 neighbouring inputs of a row, thread t of them 2t and 2t + 1.

__device__ __forceinline__ float2 pair_at(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 pair_at(const __nv_bfloat16* p) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
}

// Brings into L2 what this warp will add of a tile of dw, while it is multiplied:
// the accumulating 24576 rows of 64 experts of 1408 x 2048 492 instead of 591 us.
template <typename T>
__device__ __forceinline__ void prefetch_old(const TcGmm& g, const Tile& t, int fw, int cg, int lane) {
  if (fw + lane >= g.n) return;
  const T* row = static_cast<const T*>(g.out) + ((int64_t)t.e * g.n + fw + lane) * g.k + t.c0;
  for (int c = cg * 32; c < t.cols; c += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + c));
}

// Adds what dw holds, all of it asked for at once (the same call 591 instead of
// 721 us with a row of the block asked for, added and stored before the next;
// 16384 rows of 32 of 2048 x 7168 in fp32 982 instead of 2420).
template <typename T>
__device__ __forceinline__ void add_old(float (&r)[2][16], const T* out, int64_t ld, int nr, int nc, int lane) {
  float2 o[4][4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const int row = h * 8 + (lane >> 2);
    const T* p = out + (int64_t)row * ld + (lane & 3) * 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[h][i] = row < nr && 8 * i < nc ? pair_at(p + 8 * i) : make_float2(0.f, 0.f);
  }
#pragma unroll
  for (int h = 0; h < 4; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[h >> 1][4 * i + (h & 1) * 2] += o[h][i].x;
      r[h >> 1][4 * i + (h & 1) * 2 + 1] += o[h][i].y;
    }
  __syncwarp();  // read before other lanes' stores
}

// Writes it: 32 bytes of fp32 by four threads; for bf16 the rounded pairs of
// two blocks of 8 are exchanged between them, so that four threads write 32
// bytes of bf16 too (16-byte pieces of L2's sectors cost the softmax layer's
// gradient a tenth; exchanging fp32, twice the shuffles, took 172 instead of
// 137 us of 26 rows' 5744 x 7160 of 6 experts).
__device__ __forceinline__ void store_dw(const float (&r)[2][16], float* out, int64_t ld, int nr, int nc, int lane) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const int row = h * 8 + (lane >> 2);
    float* p = out + (int64_t)row * ld + (lane & 3) * 2;
    if (row < nr)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (8 * i < nc)
          *reinterpret_cast<float2*>(p + 8 * i) =
              make_float2(r[h >> 1][4 * i + (h & 1) * 2], r[h >> 1][4 * i + (h & 1) * 2 + 1]);
  }
}
__device__ __forceinline__ void store_dw(const float (&r)[2][16], __nv_bfloat16* out, int64_t ld, int nr, int nc,
                                         int lane) {
  const int t = lane & 3;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const int row = h * 8 + (lane >> 2);
    uint32_t w[4];  // this thread's pair of each block of 8
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p =
          __floats2bfloat162_rn(r[h >> 1][4 * i + (h & 1) * 2], r[h >> 1][4 * i + (h & 1) * 2 + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    // threads 0 and 1 take block 2u, threads 2 and 3 block 2u + 1: inputs
    // 4 (t & 1) .. + 3
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t own = (t & 2) ? w[2 * u + 1] : w[2 * u];
      const uint32_t o = __shfl_xor_sync(0xffffffffu, (t & 2) ? w[2 * u] : w[2 * u + 1], 2);
      const uint32_t lo = (t & 2) ? o : own, hi = (t & 2) ? own : o;  // pairs t & 1 and 2 + (t & 1)
      const uint32_t x = __shfl_xor_sync(0xffffffffu, (t & 1) ? lo : hi, 1);
      const int c = 16 * u + (t >> 1) * 8 + (t & 1) * 4;
      if (row < nr && c < nc)
        *reinterpret_cast<uint2*>(out + (int64_t)row * ld + c) = (t & 1) ? make_uint2(x, hi) : make_uint2(lo, x);
    }
  }
}

// Into dw, from output fw and the tile's input c on.
template <typename T>
__device__ __forceinline__ void put_dw(const TcGmm& g, float (&v)[2][16], const Tile& t, int fw, int c, int lane) {
  T* out = static_cast<T*>(g.out) + ((int64_t)t.e * g.n + fw) * g.k + t.c0 + c;
  const int nr = g.n - fw, nc = t.cols - c;
  // (two write-outs: one, with the addition before it where asked for, cost the
  // tiles without it 1.5 %)
  if (g.accumulate) {
    add_old(v, out, g.k, nr, nc, lane);
    store_dw(v, out, g.k, nr, nc, lane);
    asm volatile("" ::: "memory");
  } else {
    store_dw(v, out, g.k, nr, nc, lane);
  }
}

// mbar_wait without a call.
__device__ __forceinline__ bool wait_inline(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t* err,
                                            uint64_t limit) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t n = 1; !mbar_try_wait_sleep(bar, parity); ++n) {
    if ((n & 63) != 0) continue;
    if (*abort_flag) return false;
    if (globaltimer() - t0 > limit) {
      *abort_flag = 1;
      set_error(err, ERRBIT_TIMEOUT);
      return false;
    }
  }
  return true;
}

// 32 TMEM lanes (a thread's own) x 8 columns, and the inverse.
__device__ __forceinline__ void tmem_ld32x8(uint32_t taddr, float (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32x8(uint32_t taddr, const float (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
               : "memory");
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NUM_THREADS, 1)
    gmm_tc_kernel(const __grid_constant__ TcGmm g) {
  using C = Cfg<MODE>;
  constexpr bool A_MN = MODE != GMM_FWD, B_MN = MODE == GMM_DW;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* stage_out = tiles + C::RING;
  uint64_t* full = reinterpret_cast<uint64_t*>(stage_out + 8 * C::STG);
  uint64_t* empty = full + SLOTS;
  uint64_t* tfull = empty + SLOTS;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* qfull = drain + 1;
  uint64_t* qempty = qfull + TQ;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(qempty + TQ);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Tile* tq = reinterpret_cast<Tile*>(tmem_slot + 4);  // [TQ]
  int32_t* cnt = reinterpret_cast<int32_t*>(stage_out + 8 * C::STG + 512);
  int32_t* off = cnt + MAX_E + 1;
  int32_t* P = off + MAX_E + 1;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int E = g.E;
  const int NF = MODE == GMM_DX ? g.k : g.n;  // features: M extent
  const int nf = (NF + 2 * FM - 1) / (2 * FM);

  if (warp == 0) {
    if (lane == 0) {
      for (int s = 0; s < SLOTS; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
      // tempty: one arrive per epilogue warp of both CTAs (used on the leader)
      for (int a = 0; a < 2; ++a) { mbar_init(&tfull[a], 1); mbar_init(&tempty[a], 16); }
      mbar_init(drain, 1);
      // read by the epilogue warps, the producer and the leader's MMA issuer
      for (int q = 0; q < TQ; ++q) { mbar_init(&qfull[q], 1); mbar_init(&qempty[q], leader ? 10 : 9); }
      *abort_flag = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
  } else if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(TMEM_COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  if (MODE != GMM_DW) {
    // zeros for the columns that no box brings (see row_box)
    for (uint32_t i = threadIdx.x; i < C::RING / 16; i += NUM_THREADS)
      reinterpret_cast<uint4*>(tiles)[i] = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  grid_dependency();
  bool bad = false;
#pragma unroll 4
  for (int e = threadIdx.x; e < E; e += NUM_THREADS) {
    const Span sp = expert_span(g.offsets, e, g.rows);
    bad |= sp.bad;
    cnt[e] = sp.count;
    off[e] = sp.b;
  }
  if (bad && blockIdx.x == 0) set_error(g.err, ERRBIT_BAD_INDEX);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // barriers of both CTAs initialised before any cross-CTA use
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer (both CTAs)
    // The whole warp runs the loop on warp-uniform values and one lane issues:
    // the copies' operands then come from uniform registers. No shared memory
    // is read per stage (a load would queue behind the copies, ~230 cycles).
    const bool el = elect_one();
    Ring<MODE> R;
    Outstanding<MODE> Q;
    uint32_t issued = 0;
    int last_e = -1;
    bool ok = true;
    TileQueue T;
    Tile t;
    while (ok && T.next(t, tq, qfull, qempty, lane, abort_flag, g.err, g.wait_ns)) {
      const int kb_n = (t.depth + BK - 1) / BK;
      if (kb_n == 0) continue;
      const uint32_t sz = stage_bytes<MODE>(t);
      const int f = t.f0 + (int)rank * FM;
      // this CTA's N columns of each half: [c0 + h nh + rank n/2, + n/2)
      const int n0 = half_n(t, 0), n1 = t.halves == 2 ? half_n(t, 1) : 0;
      const int cb0 = t.c0 + (int)rank * (n0 / 2), cb1 = t.c0 + t.nh + (int)rank * (n1 / 2);
      const CUtensorMap *ma = &g.tmA, *mb0 = g.maps + E + t.e, *mb1 = nullptr;
      uint32_t tx = 2u * TILE;
      bool ld0 = true, ld1 = false;
      if (MODE == GMM_DW) {
        ma = g.maps + t.e;
        if (t.e != last_e) {
          tmap_acquire(ma);
          tmap_acquire(mb0);
          last_e = t.e;
        }
        tx += t.nh > MAXN / 2 ? 2u * TILE : (uint32_t)TILE;
      } else {
        const int c0 = min(t.cols, t.nh), c1 = t.cols - c0;  // valid columns of the halves
        const int x0 = row_box(c0, n0, rank), x1 = t.halves == 2 ? row_box(c1, n1, rank) : -1;
        ld0 = x0 >= 0;
        ld1 = x1 >= 0;
        mb0 = &g.tmB[max(x0, 0)];
        mb1 = &g.tmB[max(x1, 0)];
        int rows = box_rows(row_box(c0, n0, 0)) + box_rows(row_box(c0, n0, 1));
        if (t.halves == 2) rows += box_rows(row_box(c1, n1, 0)) + box_rows(row_box(c1, n1, 1));
        tx += (uint32_t)rows * (BK * 2);
      }
      ok = Q.begin(sz, empty, abort_flag, g.err, g.wait_ns);
      for (int kb = 0; ok && kb < kb_n; ++kb) {
        const uint32_t at = R.place(sz);
        if (!Q.make_room(R.pad + sz, empty, abort_flag, g.err, g.wait_ns)) { ok = false; break; }
        Q.push(sz, at, R.pad);
        if (el) {
          uint8_t* sa = tiles + at;
          uint8_t* sb = sa + TILE;
          const uint32_t fb = mapa(smem_u32(&full[R.slot]), 0);
          if (leader) mbar_expect_tx(&full[R.slot], tx);
          const int kk = kb * BK;
          if (MODE == GMM_FWD) {
            tma2_load_3d(sa, ma, fb, kk, f, t.e);
          } else if (MODE == GMM_DX) {
            if (g.wide) {
              tma2_load_4d(sa, ma, fb, 0, kk, f / 64, t.e);
            } else {
              tma2_load_3d(sa, ma, fb, f, kk, t.e);
              tma2_load_3d(sa + TILE / 2, ma, fb, f + 64, kk, t.e);
            }
          } else {
            const int c = t.c0 + (int)rank * (t.nh / 2);
            if (g.wide) {
              tma2_load_4d(sa, ma, fb, 0, t.r0 + kk, f / 64, 0);
            } else {
              tma2_load_2d(sa, ma, fb, f, t.r0 + kk);
              tma2_load_2d(sa + TILE / 2, ma, fb, f + 64, t.r0 + kk);
            }
            tma2_load_2d(sb, mb0, fb, c, t.r0 + kk);
            if (t.nh > MAXN / 2) tma2_load_2d(sb + TILE / 2, mb0, fb, c + 64, t.r0 + kk);
          }
          if (MODE != GMM_DW) {
            if (ld0) tma2_load_2d(sb, mb0, fb, kk, cb0);
            if (ld1) tma2_load_2d(sb + n0 * BK, mb1, fb, kk, cb1);
          }
        }
        ++issued;
        R.advance(sz);
      }
    }
    if (*abort_flag && leader && el)
      for (uint32_t j = 0; j < SLOTS; ++j) {
        const uint32_t n = issued / SLOTS + (j < issued % SLOTS ? 1 : 0);
        if (n > 0) mbar_drain(&full[j], (n - 1) & 1);
      }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (leader)
    if (leader) {
      const bool el = elect_one();
      Ring<MODE> R;
      const uint32_t tiles0 = smem_u32(tiles);
      uint32_t hb = 0;  // halves so far; half i uses accumulator i & 1
      bool ok = true;
      if (g.stall && blockIdx.x == 0) ok = wait_all(drain, 0, abort_flag, g.err, g.wait_ns);
      TileQueue T;
      Tile t;
      while (ok && T.next(t, tq, qfull, qempty, lane, abort_flag, g.err, g.wait_ns)) {
        const int kb_n = (t.depth + BK - 1) / BK;
        if (kb_n == 0) continue;
        const uint32_t sz = stage_bytes<MODE>(t), b1 = (uint32_t)half_n(t, 0) * BK;
        constexpr uint32_t MAJ = (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
        const uint32_t id0 = idesc_bf16(2 * FM, half_n(t, 0)) | MAJ;
        const uint32_t id1 = t.halves == 2 ? idesc_bf16(2 * FM, half_n(t, 1)) | MAJ : 0u;
        const uint32_t d0 = tmem_base + (hb & 1) * MAXN, d1 = tmem_base + (~hb & 1) * MAXN;
        if (!wait_all(&tempty[hb & 1], ((hb >> 1) & 1) ^ 1, abort_flag, g.err, g.wait_ns)) break;
        if (t.halves == 2 && !wait_all(&tempty[~hb & 1], (((hb + 1) >> 1) & 1) ^ 1, abort_flag, g.err, g.wait_ns))
          break;
        tc_fence_after();
        uint32_t dp = d0;  // DW: the part's accumulator
        bool sum = false;  // added to what it holds
        for (int kb = 0; kb < kb_n; ++kb) {
          if (MODE == GMM_DW && kb > 0 && kb % PART == 0) {  // the next part, in the other one
            if (el) commit_pair(&tfull[hb & 1]);
            ++hb;
            dp = tmem_base + (hb & 1) * MAXN;
            sum = false;
            if (!wait_all(&tempty[hb & 1], ((hb >> 1) & 1) ^ 1, abort_flag, g.err, g.wait_ns)) { ok = false; break; }
            tc_fence_after();
          }
          const uint32_t st = tiles0 + R.place(sz);
          if (!wait_all(&full[R.slot], R.ph, abort_flag, g.err, g.wait_ns)) { ok = false; break; }
          tc_fence_after();
          if (el) {
            const uint32_t al = desc_lo<A_MN>(st), bl = desc_lo<B_MN>(st + TILE);
            if (C::HALVES == 2 && t.halves == 2)
              mma_stage<A_MN, B_MN, true>(d0, d1, al, bl, bl + (b1 >> 4), id0, id1, sum);
            else
              mma_stage<A_MN, B_MN, false>(dp, 0, al, bl, 0, id0, 0, sum);
            commit_pair(&empty[R.slot]);
          }
          sum = true;
          R.advance(sz);
        }
        if (!ok) break;
        if (el) {
          commit_pair(&tfull[hb & 1]);
          if (t.halves == 2) commit_pair(&tfull[~hb & 1]);
        }
        hb += t.halves;
      }
      if (el) {
        commit_pair(drain);
        mbar_drain(drain, 0);
      }
      __syncwarp();
    }
  } else if (warp == 10) {
    // ---------------------------------------------------------------- scheduler (both CTAs)
    int64_t rows = 0;  // of all experts
    if (MODE != GMM_DW) {
      const int per = (E + 31) / 32;
      int maxc = 0;
      int64_t wide = 0;             // rows of experts with more than a half's
      int tl[5] = {0, 0, 0, 0, 0};  // tiles at a cap of 512, 256, 128, 64, 32 rows
      for (int u = 0; u < per; ++u) {
        const int e = lane * per + u;
        if (e < E) {
          maxc = max(maxc, cnt[e]);
          rows += cnt[e];
          if (cnt[e] > MAXN) wide += cnt[e];
#pragma unroll
          for (int c = 0; c < 5; ++c) tl[c] += (int)(((int64_t)cnt[e] + (512 >> c) - 1) >> (9 - c));
        }
      }
      // The rows a tile may hold, by the time it takes in units of a row or
      // feature in a step of 64 of the reduction (0.86 ns: the traffic from L2
      // that the pairs share): (256 + rows) steps and 700 a tile. The write-out
      // is 14 a row and 200 a tile beside the next tile's MMAs, or 16 a row after its own where
      // a tile of two halves holds both accumulators. A small call also waits
      // for its last tile. Against 512 rows always: 8192 rows of 8 experts of
      // 1024 x 2048 34 instead of 50 us, 16384 of 8 of 4096 x 512 66 instead of
      // 87, 300 of one 2048 x 2048 17 instead of 21; against 256 always: 65536
      // of 256 of 2048 x 7168 1814 instead of 2010.
      const int steps = ((MODE == GMM_FWD ? g.k : g.n) + BK - 1) / BK;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        maxc = max(maxc, __shfl_xor_sync(0xffffffffu, maxc, o));
        rows += __shfl_xor_sync(0xffffffffu, rows, o);
        wide += __shfl_xor_sync(0xffffffffu, wide, o);
#pragma unroll
        for (int c = 0; c < 5; ++c) tl[c] += __shfl_xor_sync(0xffffffffu, tl[c], o);
      }
      int cap = 512;
      int64_t best = INT64_MAX;
#pragma unroll
      for (int c = 0; c < 5; ++c) {
        const int m = min(512 >> c, round32(maxc));
        const int64_t most = (int64_t)(256 + m) * steps + 16 * m;
        int64_t all = ((int64_t)tl[c] * 256 + rows) * steps + (int64_t)tl[c] * 700;
        if (c == 0) all += 16 * wide;
        all = max(all, 14 * rows + (int64_t)tl[c] * 200) * nf / npairs;
        const int64_t cost = tl[c] * (int64_t)nf <= npairs ? most : all + most;
        if (cost < best) { best = cost; cap = 512 >> c; }
      }
      int sum = 0;  // token tiles of this lane's experts
      for (int u = 0; u < per; ++u) {
        const int e = lane * per + u;
        if (e < E) sum += (int)(((int64_t)cnt[e] + cap - 1) / cap);
      }
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int p = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += p;
      }
      if (lane == 31) P[E] = incl;
      int run = incl - sum;
      for (int u = 0; u < per; ++u) {
        const int e = lane * per + u;
        if (e < E) {
          P[e] = run;
          run += (int)(((int64_t)cnt[e] + cap - 1) / cap);
        }
      }
    }
    __syncwarp();
    Sched S;
    S.off = off;
    S.cnt = cnt;
    S.P = P;
    S.E = E;
    S.nf = nf;
    S.nw = g.nw;
    S.nc = (g.k + g.nw - 1) / g.nw;
    S.n = g.n;
    S.k = g.k;
    // more rows than there are: bad offsets whose ranges overlap (reported
    // above), and a sum of tiles that may pass an int: none then
    S.total = MODE == GMM_DW ? E * nf * S.nc : rows > g.rows ? 0 : nf * P[E];
    uint32_t q = 0, ph = 0;
    for (int i = pair;; i += npairs) {
      Tile t;
      t.e = -1;
      if (i < S.total) t = decode<MODE>(S, i);
      if (!wait_all(&qempty[q], ph ^ 1, abort_flag, g.err, g.wait_ns)) break;
      if (lane == 0) {
        tq[q] = t;
        mbar_arrive(&qfull[q]);
      }
      if (t.e < 0) break;
      if (++q == TQ) { q = 0; ph ^= 1; }
    }
  } else {
    // ---------------------------------------------------------------- epilogue (both CTAs)
    const int quad = warp & 3, cg = (warp - 2) >> 2;  // TMEM lanes, turn over the columns
    const uint32_t free_bar[2] = {mapa(smem_u32(&tempty[0]), 0), mapa(smem_u32(&tempty[1]), 0)};
    uint8_t* stg = stage_out + (warp - 2) * C::STG;
    uint32_t hb = 0;
    int ok = 1;
    TileQueue T;
    Tile t;
    while (ok && T.next(t, tq, qfull, qempty, lane, abort_flag, g.err, g.wait_ns)) {
      const int fw = t.f0 + (int)rank * FM + quad * 32;  // this warp's first feature
      const bool zero = t.depth == 0;  // DW of an expert without rows
      if (zero && g.accumulate) continue;
      if (MODE == GMM_DW && g.accumulate) {
        if (g.out_f32) prefetch_old<float>(g, t, fw, cg, lane);
        else prefetch_old<__nv_bfloat16>(g, t, fw, cg, lane);
      }
      const bool parts = MODE == GMM_DW && t.depth > PART * BK;
      if (parts) {
        // the parts' sums are added up in registers, and the whole is left in
        // the last part's accumulator, from where it is written out as any
        // tile (a write-out of its own, from the registers, cost the tiles of
        // one part 3 %)
        constexpr int NB = MODE == GMM_DW ? MAXN / 64 : 1;  // this warp's blocks of 32 inputs
        float sum[NB * 4][8];
#pragma unroll
        for (int b = 0; b < NB * 4; ++b)
#pragma unroll
          for (int j = 0; j < 8; ++j) sum[b][j] = 0.f;
        for (int d = t.depth;; d -= PART * BK) {
          // (no call here: around one, not all of the sums could stay in registers)
          if (lane == 0) ok = wait_inline(&tfull[hb & 1], (hb >> 1) & 1, abort_flag, g.err, g.wait_ns) ? 1 : 0;
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          tc_fence_after();
          const uint32_t ta = tmem_base + ((uint32_t)(quad * 32) << 16) + (hb & 1) * MAXN + cg * 32;
#pragma unroll
          for (int b = 0; b < NB * 4; ++b) {
            if (cg * 32 + b / 4 * 64 >= t.cols) break;
            const uint32_t at = ta + b / 4 * 64 + b % 4 * 8;
            float r[8];
            tmem_ld32x8(at, r);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[b][j] += r[j];
            if (d <= PART * BK) tmem_st32x8(at, sum[b]);
          }
          if (d <= PART * BK) break;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_read(free_bar[hb & 1]);
          ++hb;
        }
        if (!ok) break;
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      }
      for (int h = 0; h < t.halves; ++h) {
        if (!zero && !parts) {
          if (lane == 0) ok = mbar_wait(&tfull[hb & 1], (hb >> 1) & 1, abort_flag, g.err, g.wait_ns) ? 1 : 0;
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          tc_fence_after();
        }
        const uint32_t tb = tmem_base + ((uint32_t)(quad * 32) << 16) + (hb & 1) * MAXN;
        const int nv = min(t.cols - h * t.nh, t.nh);  // valid columns of this half
        const int cb = t.c0 + h * t.nh;
#pragma unroll 1
        for (int c = cg * 32; c < nv; c += 64) {
          __syncwarp();  // (the staging's last reads)
          if (MODE == GMM_DW) {
            uint32_t r[2][16];
            float v[2][16];
            if (!zero) {
              tmem_ld16x32(tb + c, r[0]);
              tmem_ld16x32(tb + (16u << 16) + c, r[1]);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                v[0][j] = __uint_as_float(r[0][j]);
                v[1][j] = __uint_as_float(r[1][j]);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j) v[0][j] = v[1][j] = 0.f;
            }
            if (g.out_f32) put_dw<float>(g, v, t, fw, c, lane);
            else put_dw<__nv_bfloat16>(g, v, t, fw, c, lane);
          } else {
            // lane = feature, 32 rows: through shared memory to 64-byte
            // pieces of the rows
            uint32_t r[32];
            tmem_ld16(tb + c, *reinterpret_cast<uint32_t(*)[16]>(r));
            tmem_ld16(tb + c + 16, *reinterpret_cast<uint32_t(*)[16]>(r + 16));
            tmem_wait_ld();
            __nv_bfloat16* blk = reinterpret_cast<__nv_bfloat16*>(stg);
#pragma unroll
            for (int j = 0; j < 32; ++j) blk[j * 32 + lane] = __float2bfloat16_rn(__uint_as_float(r[j]));
            __syncwarp();
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(g.out);
            const int fp = fw + (lane & 3) * 8;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int q = j * 8 + (lane >> 2);
              if (c + q < nv && fp < NF)
                *reinterpret_cast<uint4*>(out + (int64_t)(cb + c + q) * NF + fp) =
                    *reinterpret_cast<const uint4*>(blk + q * 32 + (lane & 3) * 8);
            }
          }
        }
        if (!zero) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_read(free_bar[hb & 1]);
          ++hb;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no remote arrive or MMA into this CTA is still pending
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(TMEM_COLS));
  }
}

// DW: each expert's copies of the maps of dy and x, ending at its last row,
// so that a stage that reaches past it reads zeros: one warp a map.
struct EndMapArgs {
  CUtensorMap base[2];
  CUtensorMap* maps;
};

__global__ void __launch_bounds__(256) gmm_end_maps_kernel(const __grid_constant__ EndMapArgs a,
                                                           const int32_t* offsets, int64_t rows, int E) {
  __shared__ __align__(128) CUtensorMap sm[8];
  grid_dependency();
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int e = blockIdx.x * 8 + w;
  if (e >= E) return;  // whole warps
  reinterpret_cast<uint32_t*>(&sm[w])[lane] =
      reinterpret_cast<const uint32_t*>(&a.base[blockIdx.y])[lane];
  __syncwarp();
  if (lane == 0) {
    const Span s = expert_span(offsets, e, rows);
    const int end = s.b + s.count;
    asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(
                     smem_u32(&sm[w])),
                 "r"(end > 0 ? end : 1)
                 : "memory");
  }
  __syncwarp();
  asm volatile(
      "tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned [%0], "
      "[%1], 128;" ::"l"(a.maps + (int64_t)blockIdx.y * E + e),
      "r"(smem_u32(&sm[w]))
      : "memory");
}

// bf16 maps with 128-byte swizzle: a row matrix [rows, cols] in boxes of 64
// columns x box rows, and stacked matrices [E, n, k] in boxes of 64 inputs x
// box outputs.
bool map_rows(CUtensorMap* m, const void* p, int64_t rows, int cols, uint32_t box) {
  return tc::map_2d(m, p, (uint64_t)rows, (uint64_t)cols, box);
}

// Stacked matrices [E, rows, cols], cols a multiple of 64, as {64, rows, cols
// / 64, E}: a box of 64 rows x 128 columns is two 8 KB MN-major boxes in one
// copy.
bool map_chunks(CUtensorMap* m, const void* p, int64_t E, int64_t rows, int64_t cols) {
  auto fn = tc::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {64, (cuuint64_t)rows, (cuuint64_t)(cols / 64), (cuuint64_t)E};
  cuuint64_t strides[3] = {(cuuint64_t)cols * 2, 128, (cuuint64_t)(rows * cols * 2)};
  cuuint32_t box[4] = {64, BK, FM / 64, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE>
cudaError_t launch(const GmmArgs& a, void* maps, int num_sms, cudaStream_t st) {
  using C = Cfg<MODE>;
  TcGmm g;
  memset(&g, 0, sizeof(g));
  if (MODE == GMM_DW) {
    if (a.rows > 0) {
      EndMapArgs m;
      m.maps = static_cast<CUtensorMap*>(maps);
      g.wide = a.n % 64 == 0;
      if (!(g.wide ? map_chunks(&m.base[0], a.a, 1, a.rows, a.n) : map_rows(&m.base[0], a.a, a.rows, a.n, BK)) ||
          !map_rows(&m.base[1], a.b, a.rows, a.k, BK))
        return cudaErrorInvalidValue;
      const cudaError_t e = launch_pdl(true, gmm_end_maps_kernel, dim3((unsigned)ceil_div(a.E, 8), 2), dim3(256),
                                       0, st, m, a.offsets, a.rows, a.E);
      if (e != cudaSuccess) return e;
    }
    g.maps = static_cast<const CUtensorMap*>(maps);
  } else {
    if (a.rows == 0) return cudaSuccess;
    g.wide = MODE == GMM_DX && a.k % 64 == 0;
    if (!(g.wide ? map_chunks(&g.tmA, a.b, a.E, a.n, a.k)
                 : tc::map_3d(&g.tmA, a.b, (uint64_t)a.E, (uint64_t)a.n, (uint64_t)a.k,
                              MODE == GMM_FWD ? FM : BK)))
      return cudaErrorInvalidValue;
    for (int i = 0; i < NBOX; ++i)
      if (!map_rows(&g.tmB[i], a.a, a.rows, MODE == GMM_FWD ? a.k : a.n, i == 0 ? 8 : 16 * i))
        return cudaErrorInvalidValue;
  }
  g.out = a.out;
  g.offsets = a.offsets;
  g.rows = a.rows;
  g.E = a.E;
  g.n = a.n;
  g.k = a.k;
  g.out_f32 = a.out_f32;
  g.accumulate = a.accumulate;
  g.stall = pipeline_stall() == STALL_EXPERTS_UP ? 1 : 0;
  g.wait_ns = WAIT_LIMIT_NS;
  if (MODE == GMM_DW) g.wait_ns += (uint64_t)ceil_div<int64_t>(a.rows, BK) * STEP_LIMIT_NS;
  g.err = a.err;
  // upper bound on the tiles (the count depends on the device's offsets)
  const int64_t nf = ceil_div(MODE == GMM_DX ? a.k : a.n, 2 * FM);
  // DW: the inputs of a tile, 256 unless narrower tiles leave fewer pairs
  // without work in the last turn, in the scheduler's units (8192 rows of 16
  // experts of 1000 x 1000: 32 instead of 37 us; 4096 of 8 of 512 x 512: 10.0
  // instead of 11.5)
  g.nw = MAXN;
  if (MODE == GMM_DW) {
    const int64_t steps = ceil_div<int64_t>(ceil_div<int64_t>(a.rows, a.E), BK);
    int64_t best = INT64_MAX;
    for (int nw = MAXN; nw >= 64; nw /= 2) {
      const int64_t turns = ceil_div<int64_t>(nf * ceil_div(a.k, nw) * a.E, num_sms / 2);
      const int64_t tile = (256 + nw) * steps + 700, out = 14 * nw + 200;
      const int64_t cost = turns * (tile > out ? tile : out);
      if (cost < best) {
        best = cost;
        g.nw = nw;
      }
    }
  }
  const int64_t bound = MODE == GMM_DW ? nf * ceil_div(a.k, g.nw) * a.E : nf * (a.rows / 32 + a.E);
  const int pairs = (int)(bound < num_sms / 2 ? bound : num_sms / 2);
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(gmm_tc_kernel<MODE>, (int)C::SMEM, &allowed);
  if (e != cudaSuccess) return e;
  return launch_pdl(true, gmm_tc_kernel<MODE>, dim3(2 * pairs), dim3(NUM_THREADS), C::SMEM, st, g);
}

}  // namespace

cudaError_t launch_gmm_tc(int mode, const GmmArgs& g, void* maps, int num_sms, cudaStream_t st) {
  if (mode == GMM_FWD) return launch<GMM_FWD>(g, maps, num_sms, st);
  if (mode == GMM_DX) return launch<GMM_DX>(g, maps, num_sms, st);
  return launch<GMM_DW>(g, maps, num_sms, st);
}

}  // namespace moe
