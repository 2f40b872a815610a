// Ragged e4m3 products of the routed experts with a power-of-two scale for
// each 128 elements of K (rows) and each 128 x 128 block (weights):
//   out[r, n] = sum_b 2^(ea[r, b] + ew[n / 128, b]) sum_{k in b} a[r, k] w[n, k].
// The tensor cores apply the scales themselves (kind::mxf8f6f4, one E8M0 byte
// for 32 elements of K: a block's byte serves its four K steps), so the sum
// over all of K stays in one fp32 TMEM accumulator.
//
// One persistent, warp-specialised kernel; a tile is 128 rows of one expert (256
// on a CTA pair) x 256 columns (SiTU: 128 gate and the 128 matching up columns), K in blocks of
// 128 (one 128-byte swizzle row):
//   warp 0      TMA producer: A rows and two 128-row B boxes per K block,
//   warp 1      MMA issuer and TMEM allocator,
//   warps 4-19  epilogue, four per 32-row quarter, sharing its columns,
//   warps 20-23 the scale words of four K blocks at a time, written to TMEM.
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "experts_fp8.h"
#include "kernels.h"
#include "launch.h"
#include "quantize.cuh"
#include "tc_ptx.cuh"

namespace lmoe {
namespace {

using namespace tc;

constexpr int BM = 128, SUB = 128, BK = 128;
constexpr int A_BYTES = BM * BK, SUB_BYTES = SUB * BK;
// Heights of the boxes of A: a CTA loads the smallest that holds its rows of a
// tile.  The rows of shared memory behind a small box start as zeros: the
// MMAs multiply all 128, and on a decode step that many empty rows of leftover
// data drew the GPU to its power cap (K3 width, 64 tokens: 645 us, 580 with
// zeros).  On pairs each CTA has its own box: K3 width, 8192 tokens evenly
// spread (146 rows an expert) 1437 -> 1405 us.
constexpr int BOX8 = 8, BOX32 = 32;
constexpr int SF_STAGES = 4;              // scale stages, each four K blocks
constexpr int SF_COLS = 16;               // TMEM columns of a scale stage (4 + 8 used)
constexpr int TMEM_COLS = 512, SF_COL0 = 256;
static_assert(SF_COL0 + SF_STAGES * SF_COLS <= TMEM_COLS, "TMEM");
constexpr int EPI_WARP0 = 4, EPI_WARPS = 16, SCALE_WARP0 = EPI_WARP0 + EPI_WARPS, SCALE_WARPS = 4;
constexpr int THREADS = 32 * (SCALE_WARP0 + SCALE_WARPS);
// The 768 threads start with 80 registers each; the 16 epilogue warps hold 64
// accumulators a thread and take what the other 8 give up (512 x 96 + 256 x 48
// = 768 x 80).  Shared memory leaves almost no L1, so a spilled register is read
// back from L2: the roles are cut to spill little (SiTU 20 bytes, the plain forms none).
constexpr int REGS_EPI = 96, REGS_OTHER = 48;
enum Out { OUT_BF16 = 0, OUT_F32 = 1, OUT_SITU = 2 };

// CG = 1: a CTA computes a 128-row tile and loads both B boxes of a K block.
// CG = 2: a CTA pair (cluster of 2) computes a 256-row tile; each CTA loads its
//   own 128 rows of A, one of the two B boxes and its own scale words, and the
//   leader (rank 0) issues the MMAs of both.
template <int CG>
struct Cfg {
  static constexpr int STAGE_BYTES = A_BYTES + (CG == 1 ? 2 : 1) * SUB_BYTES;
  static constexpr int STAGES = CG == 1 ? 4 : 6;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024;
};

struct Params {
  CUtensorMap tmA, tmA32, tmA8, tmB0, tmB1;
  const uint32_t* a_words;               // [words, rows]
  const uint32_t *w_words, *w_up_words;  // [R, w_blocks, words]
  int rows, words, w_blocks, kb, n_tiles, n_out;
  int bn;                                // output columns of a tile (SiTU: hidden units)
  const int4* tiles;                     // nullptr: one expert,
  const int32_t* offsets;                // with its two bounds here, or every row
  const int32_t* n_mtiles;
  void* out;
  uint8_t* out_scales;
  int32_t* status;
  float beta1, beta2;
  int wide_rows;                         // rows of out are 32-byte aligned
};

// This CTA (or its pair): which of the tiles it takes, and its rank in the pair.
struct Unit {
  int first, step, rank;
  int lo, hi;  // without a tile list: the only expert's rows
};
// A tile, or a CTA's share of its rows: [m0, m0 + rows) of expert e, column tile n.
struct Tile {
  int e, m0, rows, n;
};
template <int CG>
__device__ __forceinline__ int total_tiles(const Params& p, const Unit& u) {
  return (p.tiles != nullptr ? *p.n_mtiles : (u.hi - u.lo + BM * CG - 1) / (BM * CG)) * p.n_tiles;
}
template <int CG>
__device__ __forceinline__ Tile decode_tile(const Params& p, const Unit& u, int t) {
  const int mt = t / p.n_tiles, n = t - mt * p.n_tiles;
  if (p.tiles == nullptr) {
    const int m0 = u.lo + mt * BM * CG;
    return {0, m0, min(BM * CG, u.hi - m0), n};
  }
  const int4 e = p.tiles[mt];
  return {e.x, e.y, e.z, n};
}
// Tile t, which a role asks for one tile ahead so that its load is over when
// the tile's turn comes (each role waiting for it in turn cost some 1000 cycles
// a tile); any tile behind the last.
template <int CG>
__device__ __forceinline__ Tile tile_ahead(const Params& p, const Unit& u, int t, int total) {
  return t < total ? decode_tile<CG>(p, u, t) : Tile{0, 0, 0, 0};
}
template <int CG>
__device__ __forceinline__ Tile own_rows(const Tile& t, int rank) {
  if (CG == 1) return t;
  return {t.e, t.m0 + BM * rank, min(BM, max(0, t.rows - BM * rank)), t.n};
}
// Whether a plain tile of a single CTA has a second 128-column half (a pair's
// second box may lie outside W: it loads zeros).
template <int OUT, int CG>
__device__ __forceinline__ bool two_subs(const Params& p, const Tile& tl) {
  return OUT == OUT_SITU || CG == 2 || (p.bn > SUB && tl.n * p.bn + SUB < p.n_out);
}

struct Sync {
  uint64_t full[6], empty[6], sfull[SF_STAGES], sempty[SF_STAGES], tfull, tempty, drain, quarter[4];
  float amax[2 * 4 * 128];  // SiTU: maxima by tile parity, warp of the quarter, row
  uint32_t tmem;
  volatile int abort_flag;
};
static_assert(Cfg<1>::SMEM_BYTES + sizeof(Sync) <= 232448 &&
                  Cfg<2>::SMEM_BYTES + sizeof(Sync) <= 232448, "shared memory");

// Before the second CTA of a pair exits: waits for the last arrival of the MMA
// issuer's commits on each barrier of a ring that was left at (stage, phase).  A
// commit arrives in both CTAs, ordered by no cluster barrier: a block that left
// first could have it land in the shared memory of the next block there.  (The
// leader waits for its last commit itself.  A barrier that was never used counts
// as done.)
template <int N>
__device__ __forceinline__ void last_arrivals(uint64_t* ring, int stage, uint32_t phase, Sync& s,
                                              int32_t* status) {
#pragma unroll 1
  for (int i = 0; i < N; ++i)
    if (!mbar_wait(smem_u32(&ring[i]), i < stage ? phase : phase ^ 1u, &s.abort_flag, status)) return;
}

// Rows of the box of A that a CTA loads for the rows it has.
__device__ __forceinline__ int box_rows(int rows) {
  return rows > BOX32 ? BM : rows > BOX8 ? BOX32 : BOX8;
}

template <int OUT, int CG>
__device__ void produce(const Params& p, uint32_t ring, Sync& s, Unit u) {
  using C = Cfg<CG>;
  int stage = 0;
  uint32_t phase = 0, issued = 0, issued_phase = 0;
  bool ok = true;
  const int total = total_tiles<CG>(p, u);
  const uint32_t full0 = smem_u32(s.full), lead0 = CG == 1 ? full0 : map_to_rank(full0, 0);
  Tile next = tile_ahead<CG>(p, u, u.first, total);
  for (int t = u.first; ok && t < total; t += u.step) {
    const Tile tl = next;
    next = tile_ahead<CG>(p, u, t + u.step, total);
    const bool two = two_subs<OUT, CG>(p, tl);
    const int box = box_rows(tl.rows - BM * u.rank);
    const CUtensorMap* map_a = box == BM ? &p.tmA : box == BOX32 ? &p.tmA32 : &p.tmA8;
    // a pair's second CTA loads no A when it has no rows (its accumulator is not stored)
    const bool load_a = u.rank == 0 || tl.rows > BM;
    // of the whole tile; the leader's barrier counts both CTAs' boxes
    const int a_rows = box_rows(tl.rows) + (CG == 2 && tl.rows > BM ? box_rows(tl.rows - BM) : 0);
    const uint32_t bytes = a_rows * BK + (two ? 2 : 1) * SUB_BYTES;
    // this CTA's boxes of W: gate and up, or two neighbouring boxes; of a pair, each CTA one
    const int row0 = tl.n * p.bn;
    const int row1 = OUT == OUT_SITU ? row0 : row0 + SUB;
    const CUtensorMap* map1 = OUT == OUT_SITU ? &p.tmB1 : &p.tmB0;
    const CUtensorMap* map_b = u.rank == 0 ? &p.tmB0 : map1;
    const int row_b = u.rank == 0 ? row0 : row1;
    for (int kb = 0; kb < p.kb; ++kb) {
      if (!mbar_wait(smem_u32(&s.empty[stage]), phase ^ 1u, &s.abort_flag, p.status)) {
        ok = false;
        break;
      }
      const uint32_t dst = ring + stage * C::STAGE_BYTES, bar = lead0 + 8 * stage;
      if (u.rank == 0) mbar_expect_tx(full0 + 8 * stage, bytes);
      if (load_a) tma_load_2d<CG>(dst, map_a, bar, kb * BK, tl.m0 + BM * u.rank);
      tma_load_3d<CG>(dst + A_BYTES, map_b, bar, kb * BK, row_b, tl.e);
      if (CG == 1 && two) tma_load_3d<CG>(dst + A_BYTES + SUB_BYTES, map1, bar, kb * BK, row1, tl.e);
      issued |= 1u << stage;
      issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
  if (CG == 2 && ok && u.rank != 0) {
    last_arrivals<C::STAGES>(s.empty, stage, phase, s, p.status);
    mbar_wait(smem_u32(&s.drain), 0, &s.abort_flag, p.status);
  }
  // every load issued has landed before the block exits (a pair's loads land on
  // the leader's barriers).
  if (u.rank == 0)
    for (int i = 0; i < C::STAGES; ++i)
      if (issued & (1u << i)) {
        volatile int no_abort = 0;
        mbar_wait(full0 + 8 * i, (issued_phase >> i) & 1u, &no_abort, p.status);
      }
}

// Scale words of four K blocks of a tile: of 128 rows of A, four per lane (rows
// lane + 32 j), and of the two weight blocks.
struct ScaleRows {
  int row[4];   // rows of A, -1: none (its product is not stored)
  int64_t at;   // first word of the weight block (SiTU: in both matrices)
  int second;   // words from there to the second block's
};
struct ScaleWords {
  uint32_t a[4], b0, b1;
};
template <int OUT, int CG>
__device__ __forceinline__ ScaleRows scale_rows(const Params& p, const Tile& tl) {
  const int lane = threadIdx.x & 31;
  const int nb0 = tl.n * p.bn / SUB;
  ScaleRows r{{-1, -1, -1, -1}, ((int64_t)tl.e * p.w_blocks + nb0) * p.words,
              nb0 + 1 < p.w_blocks ? p.words : 0};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = lane + 32 * j;
    if (i < tl.rows) r.row[j] = tl.m0 + i;
  }
  return r;
}
template <int OUT>
__device__ __forceinline__ ScaleWords scale_words(const Params& p, const ScaleRows& r, int q) {
  ScaleWords w{{0, 0, 0, 0}, 0, 0};
  const uint32_t* a = p.a_words + (int64_t)q * p.rows;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (r.row[j] >= 0) w.a[j] = a[r.row[j]];
  w.b0 = p.w_words[r.at + q];
  w.b1 = OUT == OUT_SITU ? p.w_up_words[r.at + q] : p.w_words[r.at + r.second + q];
  return w;
}
// Scale warp w writes the words to TMEM lanes 32 w ...: columns 0-3 the words of
// rows 0-31, 32-63, 64-95 and 96-127 of A, 4-7 and 8-11 those of the two weight
// blocks (one word for their 128 rows), the same in each quarter, as the
// block-scaled MMA reads them.  Words and tiles are loaded one step ahead.
template <int OUT, int CG>
__device__ void feed_scales(const Params& p, uint32_t tmem, Sync& s, Unit u) {
  const int lane = threadIdx.x & 31;
  const int total = total_tiles<CG>(p, u);
  const uint32_t full0 = CG == 1 ? smem_u32(s.sfull) : map_to_rank(smem_u32(s.sfull), 0);
  const uint32_t sf0 = tmem + SF_COL0 + ((threadIdx.x & 96) << 16);
  int stage = 0;
  uint32_t phase = 0;
  Tile tn = own_rows<CG>(tile_ahead<CG>(p, u, u.first + u.step, total), u.rank);
  ScaleRows rows = scale_rows<OUT, CG>(p, own_rows<CG>(tile_ahead<CG>(p, u, u.first, total), u.rank));
  ScaleWords next = scale_words<OUT>(p, rows, 0);
  for (int t = u.first; t < total; t += u.step) {
    const ScaleRows rows1 = scale_rows<OUT, CG>(p, tn);
    tn = own_rows<CG>(tile_ahead<CG>(p, u, t + 2 * u.step, total), u.rank);
    for (int q = 0; q < p.words; ++q) {
      const ScaleWords w = next;
      if (q + 1 == p.words) rows = rows1;
      next = scale_words<OUT>(p, rows, q + 1 < p.words ? q + 1 : 0);
      if (!warp_wait(smem_u32(&s.sempty[stage]), phase ^ 1u, &s.abort_flag, p.status)) return;
      fence_after();
      const uint32_t v[16] = {w.a[0], w.a[1], w.a[2], w.a[3], w.b0, w.b0, w.b0, w.b0,
                              w.b1,   w.b1,   w.b1,   w.b1,   0,    0,    0,    0};
      st16(sf0 + stage * SF_COLS, v);
      fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 1) mbar_arrive(full0 + 8 * stage);
        else mbar_arrive_remote(full0 + 8 * stage);
      }
      if (++stage == SF_STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
  if (CG == 2 && u.rank != 0) last_arrivals<SF_STAGES>(s.sempty, stage, phase, s, p.status);
}

// The whole warp walks the tiles, so that addresses and descriptors stay in
// uniform registers, and one elected lane issues (a single lane walking alone
// took about 700 cycles a K block to issue what the tensor cores do in 512).
template <int OUT, int CG>
__device__ void issue_mmas(const Params& p, uint32_t ring, uint32_t tmem, Sync& s, Unit u) {
  using C = Cfg<CG>;
  constexpr bool PAIR = CG == 2;
  int stage = 0, sstage = 0;
  uint32_t phase = 0, sphase = 0, tphase = 0;
  bool ok = true;
  const int total = total_tiles<CG>(p, u);
  Tile next = tile_ahead<CG>(p, u, u.first, total);
  for (int t = u.first; ok && t < total; t += u.step) {
    const bool two = two_subs<OUT, CG>(p, next);
    next = tile_ahead<CG>(p, u, t + u.step, total);
    const uint32_t idesc = instr_desc_mxf8<CG>(two ? 2 * SUB : SUB);
    if (!warp_wait<PAIR>(smem_u32(&s.tempty), tphase ^ 1u, &s.abort_flag, p.status)) break;
    tphase ^= 1u;
    fence_after();
    for (int kb = 0; kb < p.kb; ++kb) {
      const uint32_t sfa = tmem + SF_COL0 + sstage * SF_COLS, sfb = sfa + 4;
      if ((kb & 3) == 0) {
        if (!warp_wait<PAIR>(smem_u32(&s.sfull[sstage]), sphase, &s.abort_flag, p.status)) {
          ok = false;
          break;
        }
        fence_after();
      }
      if (!warp_wait<PAIR>(smem_u32(&s.full[stage]), phase, &s.abort_flag, p.status)) {
        ok = false;
        break;
      }
      fence_after();
      const uint64_t a = desc_sw128(ring + stage * C::STAGE_BYTES), b = a + (A_BYTES >> 4);
      const uint32_t id = idesc | sf_id_bits(kb & 3);
      const bool last = kb == p.kb - 1;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < BK / 32; ++k)
          mma_mxf8<CG>(tmem, a + 2 * k, b + 2 * k, id, sfa, sfb, (kb > 0 || k > 0) ? 1u : 0u);
        commit<CG>(smem_u32(&s.empty[stage]));
        if ((kb & 3) == 3 || last) commit<CG>(smem_u32(&s.sempty[sstage]));
        if (last) commit<CG>(smem_u32(&s.tfull));
      }
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
      if ((kb & 3) == 3 || last) {
        if (++sstage == SF_STAGES) {
          sstage = 0;
          sphase ^= 1u;
        }
      }
    }
  }
  if (elect_one()) commit<CG>(smem_u32(&s.drain));  // all MMAs are complete before TMEM is freed
  volatile int no_abort = 0;
  mbar_wait(smem_u32(&s.drain), 0, &no_abort, p.status);
}

// Stores 32 bytes of this lane's row at dst, the first `bytes` of them (a
// multiple of 16): a whole sector in one instruction where rows are 32-byte
// aligned (wide).  Each lane writes its own row: a transpose through shared
// memory, for longer runs per instruction, took longer than it saved.
__device__ __forceinline__ void store32(char* dst, const uint32_t (&w)[8], int bytes, bool wide) {
  if (wide && bytes >= 32) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    if (bytes >= 16) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    if (bytes >= 32) *reinterpret_cast<uint4*>(dst + 16) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// ------------------------------------------------------------- hidden units
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two fp32 values in one register pair, for the packed instructions: half the
// issue slots of the polynomials below.
typedef uint64_t f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 both(float a) { return pack2(a, a); }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// tanh(x) / x as polynomials in u = x^2, fitted by least squares with the
// weights moved towards the largest relative error: relative error in 32 bits
// at most 4.2 * 2^-24 for |x| <= kGateX, 1.9 * 2^-24 for |x| <= kUpX.
constexpr float kGateX = 1.5f, kUpX = 0.5f;
__device__ __forceinline__ f32x2 gate_poly(f32x2 u) {
  f32x2 p = both(2.553440027e-05f);
  p = fma2(p, u, both(-3.205151297e-04f));
  p = fma2(p, u, both(1.872322173e-03f));
  p = fma2(p, u, both(-7.067439146e-03f));
  p = fma2(p, u, both(2.066442743e-02f));
  p = fma2(p, u, both(-5.348970741e-02f));
  p = fma2(p, u, both(1.332349330e-01f));
  p = fma2(p, u, both(-3.333253562e-01f));
  return fma2(p, u, both(9.999998808e-01f));
}
__device__ __forceinline__ f32x2 up_poly(f32x2 u) {
  f32x2 p = both(1.713500172e-02f);
  p = fma2(p, u, both(-5.298607424e-02f));
  p = fma2(p, u, both(1.332477927e-01f));
  p = fma2(p, u, both(-3.333306909e-01f));
  return fma2(p, u, both(1.0f));
}
// Two SiTU-GLU hidden units beta1 tanh(a / beta1) sigmoid(a) beta2 tanh(c / beta2),
// in place of a, off by at most 25 * 2^-24 of their value for any a and c: a hidden
// unit is rounded to e4m3 next, and a coarser value would fall on the other side
// of a rounding border more often.  Near zero, tanh(x) = x P(x^2): no cancellation,
// and beta tanh(a / beta) = a P.  Beyond (|x| > kGateX, kUpX), tanh(x) =
// (1 - t) / (1 + t) with t = e^(-2 |x|), its denominator shared with the
// sigmoid's.  e^-a = 2^-y, y = a log2 e rounded: off by 2^-24 for each unit of
// |a|, so beyond kNearA times 1 + r ln 2, r the rest of the exponent.  (For every
// unit that took the mid layer's gate and up products from 270 to 281 us and moved
// no hidden unit across a border.)  Past kFarA the sigmoid takes |a| = kFarA: it is
// 1, or under 2^-126 and 0.  WIDE: some unit of the warp is beyond a bound; the
// others get the bits that they get without.
constexpr float kLog2e = 1.44269502f, kLog2eRest = 1.92596299e-8f, kLn2 = 0.693147181f;
constexpr float kNearA = 5.5f, kFarA = 200.0f;
template <bool WIDE>
__device__ __forceinline__ void situ_units(float& a0, float& a1, float c0, float c1, float b1,
                                           float b2, float i1, float i2) {
  const f32x2 a = pack2(a0, a1), c = pack2(c0, c1);
  const f32x2 x1 = mul2(a, both(i1)), x2 = mul2(c, both(i2));
  f32x2 n1 = mul2(a, gate_poly(mul2(x1, x1))), n2 = mul2(c, up_poly(mul2(x2, x2)));
  float d0 = 1.0f + ex2(-kLog2e * a0), d1 = 1.0f + ex2(-kLog2e * a1);
  if (WIDE) {
    float n[2][2], d[2] = {d0, d1};
    unpack2(n1, n[0][0], n[0][1]);
    unpack2(n2, n[1][0], n[1][1]);
    const float av[2] = {a0, a1}, cv[2] = {c0, c1};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float xa = fabsf(av[i] * i1), xc = fabsf(cv[i] * i2);
      const float t1 = ex2(-2.0f * kLog2e * xa), t2 = ex2(-2.0f * kLog2e * xc);
      if (fabsf(av[i]) > kNearA) {
        const float s = copysignf(fminf(fabsf(av[i]), kFarA), av[i]), y = s * kLog2e;
        const float r = fmaf(s, -kLog2eRest, fmaf(s, -kLog2e, y));
        d[i] = fmaf(ex2(-y), fmaf(r, kLn2, 1.0f), 1.0f);
      }
      if (xa > kGateX) {
        n[0][i] = copysignf(b1 - b1 * t1, av[i]);
        d[i] *= 1.0f + t1;
      }
      if (xc > kUpX) {
        n[1][i] = copysignf(b2 - b2 * t2, cv[i]);
        d[i] *= 1.0f + t2;
      }
    }
    n1 = pack2(n[0][0], n[0][1]);
    n2 = pack2(n[1][0], n[1][1]);
    d0 = d[0];
    d1 = d[1];
  }
  unpack2(mul2(mul2(n1, n2), pack2(rcp(d0), rcp(d1))), a0, a1);
}

// A tile's hidden units of this warp: 32 rows x 32 units, quantised with the
// maximum over the row's 128.
__device__ __forceinline__ void finish_situ(const Params& p, const Tile& tl, float (&v)[64], int rows,
                                            int quarter, int part, float* amax,
                                            uint32_t phase, Sync& s, bool& ok) {
  const int lane = threadIdx.x & 31;
  amax += phase * 512 + 32 * quarter + lane;  // of this row: [part * 128]
  float m = 0.0f;
  if (rows > 0) {
    float ma = 0.0f, mc = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      ma = fmaxf(ma, fabsf(v[i]));
      mc = fmaxf(mc, fabsf(v[32 + i]));
    }
    const float i1 = 1.0f / p.beta1, i2 = 1.0f / p.beta2;
    if (__any_sync(0xffffffffu, ma * i1 > kGateX || mc * i2 > kUpX || ma > kNearA)) {
#pragma unroll
      for (int i = 0; i < 32; i += 2)
        situ_units<true>(v[i], v[i + 1], v[32 + i], v[33 + i], p.beta1, p.beta2, i1, i2);
    } else {
#pragma unroll
      for (int i = 0; i < 32; i += 2)
        situ_units<false>(v[i], v[i + 1], v[32 + i], v[33 + i], p.beta1, p.beta2, i1, i2);
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) m = fmaxf(m, fabsf(v[i]));  // finite, or NaN: left out
  }
  amax[128 * part] = m;
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(&s.quarter[quarter]));
  ok = warp_wait(smem_u32(&s.quarter[quarter]), phase, &s.abort_flag, p.status);
  if (!ok || rows <= 0) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, amax[128 * i]);
  const int e = scale_exponent(m);
  const float inv = pow2_f(-e);
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i] = pack_e4m3_finite(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv,
                            v[4 * i + 3] * inv);
  if (lane >= rows) return;
  const int64_t row = tl.m0 + 32 * quarter + lane;
  const int col = tl.n * SUB + 32 * part;
  store32(static_cast<char*>(p.out) + row * p.n_out + col, w, p.n_out - col, p.wide_rows);
  if (part == 0)
    p.out_scales[((int64_t)(tl.n >> 2) * p.rows + row) * 4 + (tl.n & 3)] = (uint8_t)(e + 127);
}

// A plain tile's 32 rows x 64 columns of this warp.
template <int OUT>
__device__ __forceinline__ void finish_store(const Params& p, const Tile& tl, const float (&v)[64],
                                             int rows, int quarter, int part) {
  constexpr int ES = OUT == OUT_F32 ? 4 : 2, CB = 32 / ES;  // columns of 32 bytes
  const int lane = threadIdx.x & 31, col0 = tl.n * p.bn + 64 * part;
  if (lane >= rows || 64 * part >= p.bn) return;
  char* row = static_cast<char*>(p.out) + ((int64_t)(tl.m0 + 32 * quarter + lane) * p.n_out + col0) * ES;
#pragma unroll
  for (int b = 0; b < 64 / CB; ++b) {
    const float* f = v + b * CB;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = OUT == OUT_F32 ? __float_as_uint(f[i]) : bf16x2(f[2 * i], f[2 * i + 1]);
    store32(row + b * 32, w, (p.n_out - col0 - b * CB) * ES, p.wide_rows);
  }
}

template <int OUT, int CG>
__device__ void epilogue(const Params& p, uint32_t tmem, Sync& s, Unit u) {
  const int lane = threadIdx.x & 31, ew = (threadIdx.x >> 5) - EPI_WARP0;
  const int quarter = ew & 3, part = ew >> 2;  // TMEM lanes 32 (warp mod 4) ..., columns
  const uint32_t ta = tmem + ((uint32_t)(32 * quarter) << 16);
  // the leader's MMA thread waits for the epilogues of both CTAs
  const uint32_t tempty = CG == 1 ? smem_u32(&s.tempty) : map_to_rank(smem_u32(&s.tempty), 0);
  uint32_t phase = 0;
  const int total = total_tiles<CG>(p, u);
  Tile next = tile_ahead<CG>(p, u, u.first, total);
  for (int t = u.first; t < total; t += u.step) {
    const Tile tl = own_rows<CG>(next, u.rank);
    next = tile_ahead<CG>(p, u, t + u.step, total);
    const int rows = min(32, tl.rows - 32 * quarter);
    if (!warp_wait(smem_u32(&s.tfull), phase, &s.abort_flag, p.status)) return;
    fence_after();
    float v[64];
    if (rows > 0) {  // SiTU: 32 gate and the matching 32 up columns
      ld32(ta + (OUT == OUT_SITU ? 32 : 64) * part, v);
      ld32(ta + (OUT == OUT_SITU ? SUB + 32 * part : 64 * part + 32), v + 32);
      ld_wait();
    }
    // the accumulator is in registers: the next tile's MMAs may start
    fence_before();
    __syncwarp();
    if (lane == 0) {
      if (CG == 1) mbar_arrive(tempty);
      else mbar_arrive_remote(tempty);
    }
    if constexpr (OUT == OUT_SITU) {
      bool ok;
      finish_situ(p, tl, v, rows, quarter, part, s.amax, phase, s, ok);
      if (!ok) return;
    } else {
      finish_store<OUT>(p, tl, v, rows, quarter, part);
    }
    phase ^= 1u;
  }
}

template <int OUT, int CG>
__global__ void __launch_bounds__(THREADS, 1)
    experts_fp8_kernel(const __grid_constant__ Params p) {
  using C = Cfg<CG>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Sync s;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5;
  Unit u = CG == 1 ? Unit{(int)blockIdx.x, (int)gridDim.x, 0, 0, p.rows}
                   : Unit{(int)(blockIdx.x >> 1), (int)(gridDim.x >> 1), (int)cluster_rank(), 0, p.rows};
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < SF_STAGES; ++i) {
      mbar_init(smem_u32(&s.sfull[i]), CG * SCALE_WARPS);
      mbar_init(smem_u32(&s.sempty[i]), 1);
    }
    mbar_init(smem_u32(&s.tfull), 1);
    mbar_init(smem_u32(&s.tempty), CG * EPI_WARPS);
    mbar_init(smem_u32(&s.drain), 1);
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&s.quarter[i]), EPI_WARPS / 4);
    s.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<CG>(smem_u32(&s.tmem), TMEM_COLS);
  for (int i = 0; i < C::STAGES; ++i)
    for (int b = threadIdx.x * 16; b < A_BYTES; b += THREADS * 16)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(ring + i * C::STAGE_BYTES + b), "r"(0)
                   : "memory");
  fence_async_smem();  // before TMA writes there, and the MMAs read
  fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();  // both CTAs' barriers exist before any remote arrive
  fence_after();
  const uint32_t tmem = s.tmem;
  // everything above overlaps the previous kernel; inputs are read only below
  pdl_trigger();
  pdl_wait();
  if (p.offsets != nullptr) {  // clamped, as a tile list would be
    u.lo = min(max(p.offsets[0], 0), p.rows);
    u.hi = min(max(p.offsets[1], u.lo), p.rows);
  }

  if (warp < EPI_WARP0) {
    regs_dec<REGS_OTHER>();
    if (warp == 0) {
      if ((threadIdx.x & 31) == 0) produce<OUT, CG>(p, ring, s, u);
    } else if (warp == 1) {
      if (u.rank == 0) issue_mmas<OUT, CG>(p, ring, tmem, s, u);
    }
  } else if (warp < SCALE_WARP0) {
    regs_inc<REGS_EPI>();
    epilogue<OUT, CG>(p, tmem, s, u);
  } else {
    regs_dec<REGS_OTHER>();
    feed_scales<OUT, CG>(p, tmem, s, u);
  }

  fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();  // neither CTA frees TMEM or exits while its pair still works
  fence_after();
  if (warp == 1) tmem_free<CG>(tmem, TMEM_COLS);
}

// ------------------------------------------------------------ host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::mutex mu;
  static EncodeTiledFn fn = nullptr;
  std::lock_guard<std::mutex> lk(mu);
  if (fn == nullptr) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  }
  return fn;
}

// Bytes [dim2][dim1][dim0] (dim0 contiguous) with a box of 128 x rows (x 1),
// 128-byte swizzle, zeros outside the tensor.
bool make_map(CUtensorMap* m, const void* base, uint64_t dim0, uint64_t dim1, uint64_t dim2,
              uint32_t box_rows, uint32_t rank) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {dim0, dim1, dim2};
  cuuint64_t strides[2] = {dim0, dim0 * dim1};
  cuuint32_t box[3] = {(cuuint32_t)BK, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// SM count of the current device, and whether a kernel's shared-memory limit
// has been raised there.
constexpr int kMaxDevices = 64;
std::mutex g_mu;
struct Device {
  int sms;
};

template <int OUT, int CG>
cudaError_t launch(const Params& p, int64_t max_tiles, cudaStream_t st) {
  using C = Cfg<CG>;
  static Device devs[kMaxDevices];
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    Device& d = devs[dev];
    if (d.sms == 0) {
      e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
      if (e != cudaSuccess) return e;
      e = cudaFuncSetAttribute(experts_fp8_kernel<OUT, CG>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
      if (e != cudaSuccess) return e;
      d.sms = sms;
    }
    sms = d.sms;
  }
  const int units = (int)std::min<int64_t>(max_tiles * p.n_tiles, sms / CG);
  if (units <= 0) return cudaSuccess;
  count_launch();
  return launch_pdl(experts_fp8_kernel<OUT, CG>, dim3(CG * units), dim3(THREADS),
                    (size_t)C::SMEM_BYTES, st, CG, p);
}
template <int OUT>
cudaError_t launch(const Params& p, bool pairs, int64_t max_tiles, cudaStream_t st) {
  return pairs ? launch<OUT, 2>(p, max_tiles, st) : launch<OUT, 1>(p, max_tiles, st);
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8Gemm& g, int32_t* status, cudaStream_t st) {
  if (g.rows == 0) return cudaSuccess;
  Params p{};
  bool ok = make_map(&p.tmA, g.a, g.n_in, g.rows, 1, BM, 2) &&
            make_map(&p.tmA32, g.a, g.n_in, g.rows, 1, BOX32, 2) &&
            make_map(&p.tmA8, g.a, g.n_in, g.rows, 1, BOX8, 2) &&
            make_map(&p.tmB0, g.w, g.n_in, g.n_out, g.R, SUB, 3) &&
            (!g.situ || make_map(&p.tmB1, g.w_up, g.n_in, g.n_out, g.R, SUB, 3));
  if (!ok) return cudaErrorInvalidValue;
  p.a_words = reinterpret_cast<const uint32_t*>(g.a_scales);
  p.w_words = reinterpret_cast<const uint32_t*>(g.w_scales);
  p.w_up_words = reinterpret_cast<const uint32_t*>(g.w_up_scales);
  p.rows = (int)g.rows;
  p.words = q_words(g.n_in);
  p.w_blocks = q_blocks(g.n_out);
  p.kb = q_blocks(g.n_in);
  p.n_out = g.n_out;
  p.tiles = g.tiles;
  p.offsets = g.tiles == nullptr ? g.offsets : nullptr;
  p.n_mtiles = g.n_mtiles;
  p.out = g.out;
  p.out_scales = g.out_scales;
  p.status = status;
  const int64_t row_bytes = (int64_t)g.n_out * (g.situ ? 1 : g.out_f32 ? 4 : 2);
  p.wide_rows = row_bytes % 32 == 0 && reinterpret_cast<uintptr_t>(g.out) % 32 == 0;
  p.beta1 = g.beta1;
  p.beta2 = g.beta2;
  const int tile_m = g.pairs ? 2 * BM : BM;
  const int64_t max_tiles = g.tiles != nullptr ? g.max_tiles : (g.rows + tile_m - 1) / tile_m;
  // Plain tiles are 128 columns wide where those of 256 would leave half of the
  // SMs idle (1000 rows x 784 -> 392: 9.2 us in 16 tiles, 6.4 in 32).
  const int64_t row_tiles = std::min<int64_t>(g.rows, (g.rows + tile_m - 1) / tile_m + g.R - 1);
  const int64_t wide_tiles = row_tiles * ((g.n_out + 2 * SUB - 1) / (2 * SUB));
  p.bn = g.situ || (!g.pairs && wide_tiles <= 74) ? SUB : 2 * SUB;
  p.n_tiles = (g.n_out + p.bn - 1) / p.bn;
  if (g.situ) return launch<OUT_SITU>(p, g.pairs, max_tiles, st);
  return g.out_f32 ? launch<OUT_F32>(p, g.pairs, max_tiles, st)
                   : launch<OUT_BF16>(p, g.pairs, max_tiles, st);
}

}  // namespace lmoe
