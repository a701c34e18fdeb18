// Grouped products of microscaled 4-bit rows with 4-bit expert weights, on the
// block-scaled tensor cores (tcgen05.mma kind::mxf4; the format is in
// mx4.cuh). Over the segments of the dispatch's offsets, for each row p of
// segment e:
//   product   out[p, n] = sum_b 2^(sa[p,b] + sw[e,n,b] - 254) sum_{i<32} a w
//   gate_up   h[p, n] = silu(product with the gate row n) * (... up row n),
//             bf16, or rounded to bf16 and then quantised to 4 bits
//
// The MMA multiplies 64 values of K at a time by their two scale bytes per row
// and accumulates in fp32; nothing is dequantised.
//
// What bounds it. Few rows: streaming the experts' weights from HBM once (gate_up
// of 16 tokens, 256 experts, H 7168, I 2048: 1.6 GB in 242 us, 6.6 TB/s). Many
// rows: shared memory, which takes the operands from L2 and gives them to the
// tensor cores (at N 192 and 256 values of K, 28 KB in and some 40 KB out a
// step of 384 MMA clocks, 128 bytes a clock), and the power limit (gate_up of 8192
// tokens, 64 experts, H 4096, I 2048: 416 us, 4.0 PFLOP/s, at 1.6 GHz in launches
// with pauses; 469 us, 3.5 PFLOP/s, at 1.3 GHz in calls back to back for seconds).
//
// Design (a CTA on each SM, persistent, warp-specialised, 480 threads):
//   warp 0      TMA producer, 256 values of K a step: the tile's rows of A (one
//               box of 128, or for a short tile as many of 32 as it has), and
//               64 rows of W per unit of the tile; for gate_up 32 gate rows per
//               unit and then the 32 up rows of the same features.
//   warp 1      MMA issuer: up to four MMAs a step. Two accumulators.
//   warp 2      copies each step's scales from shared memory to TMEM, into the
//               columns of the step's stage.
//   warps 3-6   scale producers: the tensor core wants the four scale bytes of
//               a row's 128 values as one word, row r at lane r % 32 and column
//               r / 32. A lane loads 16 scale bytes (512 values) of its rows r,
//               r+32, ... from their plain row-major places and stores the
//               transposed words, so neither rows nor weights need a layout of
//               their own and a segment may start at any row.
//   warps 7-14  epilogue: TMEM to registers, SwiGLU / rounding / quantisation
//               of a lane's own row, stores by TMA from a staging buffer.
// A tile is 128 rows by 1..3 units, which every CTA picks from the number of
// row tiles, known to the device only (choose_units); the ring's stages follow.
// For large segments two CTAs share a tile of 256 rows by 3 units: each loads
// its own rows of A and half of W's, and the leader's threads issue the MMAs
// and scale copies of both (use_pairs says when); the second CTA's warp 1 tells the
// leader of its scales (forward_scales), its warp 2 idles.
//
// Waits are bounded as in gemm_tc.cu.
#include <cuda.h>

#include <mutex>

#include "kernels.h"
#include "mx4.cuh"
#include "tc_ptx.cuh"
#include "tiles.cuh"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace stm {
namespace {

using namespace tc;

constexpr int BM = 128;
constexpr int BK = 256;              // values per step: 128 data bytes, one swizzle row
constexpr int UNIT = 64;             // B rows per unit
constexpr int MAX_UNITS = 3;
constexpr int A_BYTES = BM * BK / 2;
constexpr int A_BOX_ROWS = 32;       // rows of the small A box (a short tile loads only those it needs)
constexpr int UNIT_BYTES = UNIT * BK / 2;
// Scales: a row's 16-byte vector covers 512 values of K, two steps.
constexpr int SF_ATOM_BYTES = 512;   // scale words of 128 rows for 128 values of K; a vector has four
constexpr int MAX_STAGES = 8;
constexpr int ACC_COLS = MAX_UNITS * UNIT;         // TMEM columns of one accumulator
constexpr int SF_COL = 2 * ACC_COLS;               // the stages' scale columns follow: two atoms of A, two of B
constexpr int SFB_COL = 2 * 4;
constexpr int TMEM_COLS = 512;
constexpr int SF_WARPS = 4;
constexpr int SF_WARP0 = 3;
constexpr int EPI_WARP0 = SF_WARP0 + SF_WARPS;
constexpr int GTHREADS = 32 * (EPI_WARP0 + 8);
constexpr int STAGING_BYTES = 32 * 128;            // per epilogue warp

// A CTA of a pair holds its own rows of A and half of B.
__host__ __device__ constexpr int stage_bytes(int units, bool pair) {
  return A_BYTES + units * UNIT_BYTES / (pair ? 2 : 1);
}
constexpr int RING_BYTES = 4 * stage_bytes(3, false);
__host__ __device__ constexpr int ring_stages(int units, bool pair) {
  return RING_BYTES / stage_bytes(units, pair) < MAX_STAGES ? RING_BYTES / stage_bytes(units, pair) : MAX_STAGES;
}
__host__ __device__ constexpr int sfb_blocks(int units) { return (units * UNIT + 127) / 128; }
__host__ __device__ constexpr int sf_cols(int units) { return SFB_COL + 2 * 4 * sfb_blocks(units); }
static_assert(SF_COL + ring_stages(1, false) * sf_cols(1) <= TMEM_COLS, "accumulators and scales fit TMEM");
static_assert(SF_COL + ring_stages(2, false) * sf_cols(2) <= TMEM_COLS, "accumulators and scales fit TMEM");
static_assert(SF_COL + ring_stages(3, false) * sf_cols(3) <= TMEM_COLS, "accumulators and scales fit TMEM");
static_assert(SF_COL + ring_stages(3, true) * sf_cols(3) <= TMEM_COLS, "accumulators and scales fit TMEM");
__host__ __device__ constexpr int sf_stage_bytes(int units) { return 4 * (1 + sfb_blocks(units)) * SF_ATOM_BYTES; }
constexpr int SF_RING_BYTES = SF_WARPS * sf_stage_bytes(MAX_UNITS);
// Scale stages: one for each scale warp; of a pair, whose second CTA tells of a
// stage by way of another thread, as many as fit behind its operand ring.
__host__ __device__ constexpr int sf_ring_at(bool pair) {
  return pair ? ring_stages(MAX_UNITS, true) * stage_bytes(MAX_UNITS, true) : RING_BYTES;
}
__host__ __device__ constexpr int sf_stages(bool pair) {
  return pair ? (RING_BYTES + SF_RING_BYTES - sf_ring_at(true)) / sf_stage_bytes(MAX_UNITS) : SF_WARPS;
}
constexpr int MAX_SF_STAGES = sf_stages(true);
static_assert(MAX_SF_STAGES >= SF_WARPS && sf_ring_at(true) % 1024 == 0, "a pair's scale stages");

enum { OUT_BF16 = 0, OUT_F32 = 1, SWIGLU_BF16 = 2, SWIGLU_MX4 = 3 };
constexpr bool is_swiglu(int mode) { return mode >= SWIGLU_BF16; }

struct Maps {
  CUtensorMap a_box, a_tile;  // A in boxes of 32 rows, and of 128
  CUtensorMap b[MAX_UNITS];   // W in boxes of 1..3 units; a pair's first: of half a tile's rows
  CUtensorMap out;            // out in a warp's staged boxes
};

struct Args {
  const int32_t* offsets;
  int32_t E;
  int64_t rows_total;
  int32_t N;         // output columns (gate_up: I)
  int32_t n_units;   // 64-row units of B per expert
  int32_t k_steps;
  int32_t K;
  const uint8_t* a_scale;
  const uint8_t* b_scale;
  int32_t pitch;     // scale bytes per row of K values
  int64_t b_rows;    // B rows per expert
  void* out;         // bf16 / fp32 [rows, N], or data bytes [rows, N/2]
  uint8_t* out_scale;
  int32_t out_pitch;
  int32_t* err;
};

struct __align__(8) Ctl {
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  uint64_t sfull[MAX_SF_STAGES];
  uint64_t sempty[MAX_SF_STAGES];
  uint64_t sready[MAX_SF_STAGES];  // of a pair's second CTA: its own stage is written
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;   // every MMA is done, and every copy of scales
  uint64_t cdrain;
  uint32_t tmem_base;
  int abort;
  int units;
  int off[kMaxExperts + 1];
  int pre[kMaxExperts + 1];
};

static_assert(RING_BYTES % 1024 == 0 && SF_RING_BYTES % 1024 == 0 && STAGING_BYTES % 1024 == 0, "swizzled buffers");
constexpr size_t kSmemBytes = 1024 + (size_t)RING_BYTES + SF_RING_BYTES + 8 * STAGING_BYTES + sizeof(Ctl);
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");

// Instruction descriptor, kind::mxf4: A and B e2m1 (bits 7-9, 10-12 = 1), K
// major, N>>3 in bits 17-22, scales ue8m0 (bit 23), M>>4 in 24-28; which half
// of the scale words (0, or 2 for the second 64 values) in bits 4-5 for B and
// 29-30 for A.
__device__ __forceinline__ uint32_t make_idesc_mxf4(int M, int N, uint32_t half) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24) |
         (half << 4) | (half << 29);
}

// The three issuing threads (TMA, MMA, scale copies) each run one loop a step,
// which has to stay below the step's 384 MMA clocks: they keep shared-memory
// addresses as 32-bit words that a step advances, and descriptors as their low
// words; the first two test the next step's barrier before the present step's
// work (a wait takes about 100 clocks even when its phase is long complete). With
// pointers, indices and whole descriptors gate_up of 8192 tokens took 412 us, so
// 406.

// High words of the descriptors: an operand (128-byte swizzle, 8-row groups
// 1024 bytes apart, see sw128_desc), and a scale atom for tcgen05.cp (32 rows of
// 16 bytes, no swizzle, 8-row groups 128 bytes apart). The low word is the
// address / 16, with 1 in the leading offset.
#define MX4_DESC_HIGH "0x40004040"
#define MX4_SF_DESC_HIGH "0x00004008"
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr) { return saddr >> 4 | 1u << 16; }

// Of a pair, both CTAs copy from their own shared memory to their own TMEM.
template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t desc) {
  if constexpr (PAIR)
    asm volatile("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, " MX4_SF_DESC_HIGH "};\n\t"
                 "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n\t}\n" ::"r"(taddr), "r"(desc) : "memory");
  else
    asm volatile("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, " MX4_SF_DESC_HIGH "};\n\t"
                 "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}\n" ::"r"(taddr), "r"(desc) : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void umma_mxf4(uint32_t d, uint32_t adesc, uint32_t bdesc, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, " MX4_DESC_HIGH "};\n\tmov.b64 db, {%2, " MX4_DESC_HIGH "};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "r"(adesc), "r"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, " MX4_DESC_HIGH "};\n\tmov.b64 db, {%2, " MX4_DESC_HIGH "};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "r"(adesc), "r"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Arrive on the barrier at `bar`, a pair's in both CTAs, once the work that this
// thread has issued so far is done; commit_here: on this CTA's only.
template <bool PAIR>
__device__ __forceinline__ void commit_here(uint32_t bar) {
  if constexpr (PAIR)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)0x3)
        : "memory");
  else
    commit_here<false>(bar);
}

// TMA loads to dst that complete on `bar` (of a pair, the leader's).
template <bool PAIR>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
        "[%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                        int c3) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, "
        "%6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// Whether a phase is complete.
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// The same acquiring at cluster scope.
__device__ __forceinline__ bool bar_test_cluster(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// mbar_wait by address.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, int* abort, int32_t* err, int site) {
  return mbar_wait(static_cast<uint64_t*>(__cvta_shared_to_generic(bar)), parity, abort, err, site);
}

// A ring of stages as a thread steps through it: offset of the stage's barrier,
// and the phase.
struct Ring {
  uint32_t bar, phase;
  __device__ __forceinline__ Ring next(uint32_t bar_bytes) const {
    const bool wrap = bar + 8 == bar_bytes;
    return {wrap ? 0u : bar + 8u, phase ^ (wrap ? 1u : 0u)};
  }
};

__device__ __forceinline__ void fence_to_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// One lane of a converged warp. The tensor-core and TMA instructions take
// their operands from uniform registers. In a loop that a lane chosen by number
// runs (`if (lane == 0)`) each of them took about 100 clocks, 1050 for a step;
// a lane chosen by elect.sync issues a step in 180.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// mbar_wait of a whole warp, which stays converged.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* abort, int32_t* err, int site) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err, site));
}

// Units per tile: the fewest rounds of tiles over the grid, each weighed by the
// operand bytes of its tiles (8 KB a unit and step, 4 KB for each 32 rows of A
// that the average tile has). Few row tiles take narrow tiles, so that every
// SM streams weights; many take wide ones, which re-read A least.
// Called by a whole warp: a lane weighs one choice.
__device__ __forceinline__ int choose_units(int row_tiles, int rows, int n_units, int grid) {
  const int u = MAX_UNITS - min((int)(threadIdx.x & 31), MAX_UNITS - 1);
  const int boxes = row_tiles > 0 ? min(4, (rows / row_tiles + 31) / 32) : 1;
  const uint32_t tiles = (uint32_t)row_tiles * ((uint32_t)(n_units + u - 1) / u);
  const uint32_t cost = (tiles + grid - 1) / (uint32_t)grid * (2 * u + max(1, boxes));
  // the least cost, and of equal ones the most units
  const uint32_t least = __reduce_min_sync(0xffffffffu, cost);
  return MAX_UNITS - (__ffs(__ballot_sync(0xffffffffu, cost == least)) - 1);
}

struct Tile {
  int e, row0, row_end, unit0;
};

// The tile's place (of a pair's, this CTA's 128 rows, which may lie past the
// segment); e is the expert of an earlier tile of the same CTA (row
// tiles come in rising order).
template <bool PAIR>
__device__ __forceinline__ Tile decode(const Ctl* ctl, int E, int units, int n_tiles, int tile, int e, int rank) {
  Tile t;
  const int mt = tile / n_tiles;
  t.unit0 = (tile - mt * n_tiles) * units;
  if (ctl->pre[e + 1] <= mt) {  // pre[lo] <= mt < pre[hi]
    int lo = e + 1, hi = E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (ctl->pre[mid] <= mt) lo = mid;
      else hi = mid;
    }
    e = lo;
  }
  t.e = e;
  t.row0 = ctl->off[e] + (mt - ctl->pre[e]) * (PAIR ? 2 * BM : BM) + rank * BM;
  t.row_end = ctl->off[e + 1];
  return t;
}

// silu(g) = g / (1 + 2^u), u = -g log2 e. u / 2 is carried in two parts (its
// rounding would grow with |g|), t and low, and 2^u is the square of 2^t times
// 1 + 2 low ln 2 (low is below 2^-17, its square out of reach). All of the
// denominator is taken times 2^-64, so that neither it nor its reciprocal leaves
// the normal numbers before silu itself does: for g in [-131, 3e38] off by at
// most 2^-20 of the value (2^-21 from the squared ex2.approx, the rest from
// rcp.approx and three products) and, where 1 / (1 + 2^u) is below 2^-126, by
// 2^-150 |g|. Below -131, where silu is less than 2^-180, the reciprocal is 0,
// and so is the result; for -inf it is NaN as in the quotient. (Division and expf
// cost a slow path on zeros and tiny values, which the rows past a segment hold:
// 60 thousand clocks a tile.)
__device__ __forceinline__ float silu(float g) {
  constexpr float kHalfLog2e = 0.5f * 1.4426950408889634f;
  constexpr float kHalfLog2eLow = (float)(0.5 * 1.4426950408889634074 - (double)kHalfLog2e);
  constexpr float kTiny = 0x1p-64f;
  const float x = -fminf(fmaxf(g, -133.f), 88.f);
  const float t = x * kHalfLog2e;
  const float low = fmaf(x, kHalfLog2eLow, fmaf(x, kHalfLog2e, -t));
  const float scale = fmaf(low, 2.f * 0.6931471805599453f * kTiny, kTiny);  // 2^-64 (2^low)^2
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(e * scale, e, kTiny)));
  return g * (r * kTiny);
}

// A warp stages boxes of its 32 rows by BYTES (64 or 128) of a row and stores
// them by TMA, or where the tile has fewer rows by plain stores. The 16-byte
// piece c of row r is at c ^ (r & 7), or c ^ (r / 2 & 3): the TMA swizzles of
// these widths, and neither lanes that write their own row nor lanes that read
// along rows meet in a bank. (Stores straight from the lanes' rows, 32 lines an
// instruction, bound the product's epilogue; plain stores of staged rows held
// their warp for about 900 clocks a box.)
template <int BYTES>
__device__ __forceinline__ int staged(int r, int c) {
  return r * BYTES + 16 * (BYTES == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3));
}

template <int BYTES>
__device__ __forceinline__ void store_box(const uint8_t* stage, const CUtensorMap* map, int col, int row, uint8_t* out,
                                          int64_t row_bytes, int nrows, int bytes, int lane) {
  if (nrows >= 32) {
    fence_to_async();
    __syncwarp();
    if (lane == 0) tma_store_2d(map, stage, col, row);
  } else {
    __syncwarp();
    constexpr int kPerRow = BYTES / 16;
    const int c = lane % kPerRow;
#pragma unroll
    for (int i = 0; i < kPerRow; ++i) {
      const int r = i * (32 / kPerRow) + lane / kPerRow;
      if (r < nrows && c * 16 < bytes)
        *reinterpret_cast<uint4*>(out + r * row_bytes + c * 16) =
            *reinterpret_cast<const uint4*>(stage + staged<BYTES>(r, c));
    }
    __syncwarp();
  }
  if (lane == 0) bulk_commit();  // a box is a group, an empty one where it went out by plain stores
}

// The buffers of all but the last N boxes may be written again.
template <int N>
__device__ __forceinline__ void box_free(int lane) {
  if (lane == 0) bulk_wait_read<N>();
  __syncwarp();
}

// A pair's leader issues the copies of both CTAs' scale words. Those of the second
// CTA are ordered before its copies by this thread of the second CTA: it waits for
// the storing warp's arrive (CTA scope), and one release at cluster scope, about
// 1500 clocks, tells the leader of every stage that is ready by then; a stage takes
// 768. (gate_up of 8192 tokens: a release a stage by the storing warps 762 us, by
// this thread 505, by two threads 424; several stages a release 416, as without
// any release. The product of the same sizes: 231, and 225 where the storing warps
// told the leader themselves without one.)
__device__ __forceinline__ void forward_scales(Ctl* ctl, int64_t vectors, int32_t* err) {
  constexpr int kStages = sf_stages(true);
  const uint32_t sready = smem_u32(ctl->sready), sfull = mapa_shared(smem_u32(ctl->sfull), 0);
  Ring at{0, 0};
  for (int64_t v = 0; v < vectors;) {
    if (!bar_wait(sready + at.bar, at.phase, &ctl->abort, err, 11)) break;
    Ring told = at;
    int n = 0;
    do {
      ++n;
      ++v;
      at = at.next(8 * kStages);
    } while (n < kStages && v < vectors && bar_test(sready + at.bar, at.phase));
    fence_cluster();
    for (; n > 0; --n) {
      mbar_arrive_remote_relaxed(sfull + told.bar);
      told = told.next(8 * kStages);
    }
  }
}

template <int MODE, bool PAIR>
__device__ __forceinline__ void mx4_gemm(const Maps& maps, const Args& args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int SF_STAGES = sf_stages(PAIR);
  uint8_t* sf_base = base + sf_ring_at(PAIR);
  uint8_t* staging = base + RING_BYTES + SF_RING_BYTES;
  Ctl* ctl = reinterpret_cast<Ctl*>(staging + 8 * STAGING_BYTES);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = PAIR ? (int)cluster_ctarank() : 0;
  const bool leader = rank == 0;
  // a worker is a CTA, or a pair
  const int worker = PAIR ? blockIdx.x >> 1 : blockIdx.x, workers = PAIR ? gridDim.x >> 1 : gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < MAX_STAGES; ++s) {
      mbar_init(&ctl->full[s], 2);  // the TMA producer and the scale copier
      mbar_init(&ctl->empty[s], 1);
    }
    for (int s = 0; s < SF_STAGES; ++s) {
      mbar_init(&ctl->sfull[s], PAIR ? 2 : 1);  // a scale warp, and of a pair the second CTA's forwarder
      mbar_init(&ctl->sempty[s], 1);
      if constexpr (PAIR) mbar_init(&ctl->sready[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&ctl->tfull[a], 1);
      mbar_init(&ctl->tempty[a], PAIR ? 8 : 4);  // the accumulator's epilogue warps
    }
    mbar_init(&ctl->drain, 1);
    mbar_init(&ctl->cdrain, 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == SF_WARP0) {
    warp_build_tile_table(args.offsets, args.E, 0, PAIR ? 2 * BM : BM, ctl->off, ctl->pre, args.rows_total, args.err);
    __syncwarp();
    if constexpr (!PAIR) {
      const int row_tiles = ctl->pre[args.E];
      const int rows = row_tiles > 0 ? ctl->off[args.E] - ctl->off[0] : 0;
      const int units = choose_units(row_tiles, rows, args.n_units, workers);
      if (lane == 0) ctl->units = units;
    }
  }
  if (warp == 1) {
    if constexpr (PAIR) tmem_alloc2(&ctl->tmem_base, TMEM_COLS);
    else tmem_alloc(&ctl->tmem_base, TMEM_COLS);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();  // the peer's barriers exist before any remote arrive
  tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;
  const int units = PAIR ? MAX_UNITS : ctl->units;
  const int n_tiles = (args.n_units + units - 1) / units;
  const int total = ctl->pre[args.E] * n_tiles;
  const int blocks = sfb_blocks(units);
  // 512-value vectors of scales over this worker's tiles
  const int64_t vectors = total > worker ? (int64_t)((total - worker - 1) / workers + 1) * ((args.k_steps + 1) / 2) : 0;

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (elect_one()) {
      const int stages = ring_stages(units, PAIR), sbytes = stage_bytes(units, PAIR);
      const uint32_t ring = smem_u32(base), full = smem_u32(ctl->full), empty = smem_u32(ctl->empty);
      const uint32_t load_bar = PAIR ? mapa_shared(full, 0) : full;  // the leader's barriers count a pair's bytes
      uint32_t dst = ring;
      Ring at{0, 0};
      int steps = 0, e = 0;
      bool ok = true, seen = false;
      const CUtensorMap* tmB = &maps.b[PAIR ? 0 : units - 1];
      for (int tile = worker; ok && tile < total; tile += workers) {
        const Tile t = decode<PAIR>(ctl, args.E, units, n_tiles, tile, e, rank);
        e = t.e;
        // boxes of A that the rows from row0 on fill
        auto boxes_from = [&](int row0) {
          return max(0, min(BM / A_BOX_ROWS, (t.row_end - row0 + A_BOX_ROWS - 1) / A_BOX_ROWS));
        };
        constexpr uint32_t box_bytes = A_BYTES * A_BOX_ROWS / BM;
        const int boxes = boxes_from(t.row0);
        const bool whole = boxes == BM / A_BOX_ROWS;
        const uint32_t bytes = (boxes + (PAIR ? boxes_from(t.row0 + BM) : 0)) * box_bytes + units * UNIT_BYTES;
        // W's rows of the tile; a pair loads half each, in gate_up the leader the gate rows and its peer the up rows
        const int n0 = t.unit0 * (is_swiglu(MODE) ? UNIT / 2 : UNIT) +
                       (PAIR && !is_swiglu(MODE) ? rank * (MAX_UNITS * UNIT / 2) : 0);
        const int half = PAIR && is_swiglu(MODE) ? rank : 0;
        for (int kb = 0; kb < args.k_steps * (BK / 2); kb += BK / 2) {
          if (!seen && !bar_wait(empty + at.bar, at.phase ^ 1u, &ctl->abort, args.err, 1)) {
            ok = false;
            break;
          }
          const Ring next = at.next(8 * stages);
          seen = bar_test(empty + next.bar, next.phase ^ 1u);
          if (!PAIR || leader) bar_expect(full + at.bar, bytes);
          load_4d<PAIR>(dst + A_BYTES, tmB, load_bar + at.bar, kb, n0, half, e);
          if (whole) {
            load_2d<PAIR>(dst, &maps.a_tile, load_bar + at.bar, kb, t.row0);
          } else {
            for (int i = 0; i < boxes; ++i)
              load_2d<PAIR>(dst + i * box_bytes, &maps.a_box, load_bar + at.bar, kb, t.row0 + A_BOX_ROWS * i);
          }
          dst = next.bar == 0 ? ring : dst + sbytes;
          at = next;
          ++steps;
        }
      }
      // Every copy has landed before the CTA may exit (a pair's leader counts
      // both CTAs' bytes, and the CTAs exit together).
      if (!PAIR || leader)
        for (int s = max(0, steps - stages); s < steps; ++s)
          mbar_wait(&ctl->full[s % stages], (uint32_t)(s / stages) & 1u, &ctl->abort, args.err, 6, true);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (leader && elect_one()) {
      const int stages = ring_stages(units, PAIR);
      const uint32_t desc_step = stage_bytes(units, PAIR) / 16, sf_step = sf_cols(units), sfb_step = 4 * blocks;
      const uint32_t full = smem_u32(ctl->full), empty = smem_u32(ctl->empty);
      const uint32_t desc0 = desc_low(smem_u32(base)), sf0 = tmem_base + SF_COL;
      constexpr int M = PAIR ? 2 * BM : BM;
      const uint32_t idesc0 = make_idesc_mxf4(M, units * UNIT, 0), idesc2 = make_idesc_mxf4(M, units * UNIT, 2);
      const int k_tail = args.K - (args.k_steps - 1) * BK;  // values of the last step
      uint32_t adesc = desc0, sfa = sf0, acc_phase = 0;
      Ring at{0, 0};
      int acc = 0;
      bool ok = true, seen = false;
      for (int tile = worker; ok && tile < total; tile += workers) {
        if (!mbar_wait(&ctl->tempty[acc], acc_phase ^ 1u, &ctl->abort, args.err, 2)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * ACC_COLS);
        uint32_t accumulate = 0;
        for (int kt = args.k_steps; kt > 0; --kt) {
          if (!seen && !bar_wait(full + at.bar, at.phase, &ctl->abort, args.err, 3)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const Ring next = at.next(8 * stages);
          seen = bar_test(full + next.bar, next.phase);
          const uint32_t bdesc = adesc + A_BYTES / 16, sfb = sfa + SFB_COL;
          const int left = kt == 1 ? k_tail : BK;
          umma_mxf4<PAIR>(d_tmem, adesc, bdesc, idesc0, sfa, sfb, accumulate);
          if (left > 64) umma_mxf4<PAIR>(d_tmem, adesc + 2, bdesc + 2, idesc2, sfa, sfb, 1u);
          if (left > 128) umma_mxf4<PAIR>(d_tmem, adesc + 4, bdesc + 4, idesc0, sfa + 4, sfb + sfb_step, 1u);
          if (left > 192) umma_mxf4<PAIR>(d_tmem, adesc + 6, bdesc + 6, idesc2, sfa + 4, sfb + sfb_step, 1u);
          commit<PAIR>(empty + at.bar);
          accumulate = 1;
          adesc = next.bar == 0 ? desc0 : adesc + desc_step;
          sfa = next.bar == 0 ? sf0 : sfa + sf_step;
          at = next;
        }
        if (!ok) break;
        commit<PAIR>(smem_u32(&ctl->tfull[acc]));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      commit<PAIR>(smem_u32(&ctl->drain));
      mbar_wait(&ctl->drain, 0, &ctl->abort, args.err, 7, true);
    }
    if (PAIR && !leader && elect_one()) forward_scales(ctl, vectors, args.err);
    __syncwarp();
  } else if (warp == 2) {
    // ---------------- scales from shared memory to TMEM ----------------
    // A thread of its own: twelve copies for every two steps took a third of the
    // MMA issuer's time. Every stage of the operands has its columns, so that a
    // step's copies complete its full barrier like its operands.
    if (leader && elect_one()) {
      const int stages = ring_stages(units, PAIR);
      const uint32_t desc_step = sf_stage_bytes(units) / 16, sf_step = sf_cols(units);
      const uint32_t full = smem_u32(ctl->full), empty = smem_u32(ctl->empty);
      const uint32_t sfull = smem_u32(ctl->sfull), sempty = smem_u32(ctl->sempty);
      const uint32_t desc0 = desc_low(smem_u32(sf_base)), sf0 = tmem_base + SF_COL;
      constexpr uint32_t kAtom = SF_ATOM_BYTES / 16;
      uint32_t desc = desc0, sfa = sf0;
      Ring at{0, 0}, sf{0, 0};
      bool ok = true;
      for (int tile = worker; ok && tile < total; tile += workers) {
        for (int kt = 0; kt < args.k_steps; ++kt) {
          ok = bar_wait(empty + at.bar, at.phase ^ 1u, &ctl->abort, args.err, 9) &&
               ((kt & 1) || (bar_wait(sfull + sf.bar, sf.phase, &ctl->abort, args.err, 10) &&
                             (!PAIR || bar_test_cluster(sfull + sf.bar, sf.phase))));
          if (!ok) break;
          tc_fence_after();
          // the step's two atoms of A, and of B after A's four
          const uint32_t sfb = sfa + SFB_COL, da = desc + (kt & 1) * 2 * kAtom;
          const uint32_t db = desc + (4 + (kt & 1) * 2 * blocks) * kAtom;
          copy_scales<PAIR>(sfa, da);
          copy_scales<PAIR>(sfa + 4, da + kAtom);
          copy_scales<PAIR>(sfb, db);
          copy_scales<PAIR>(sfb + 4, db + kAtom);
          if (blocks == 2) {
            copy_scales<PAIR>(sfb + 8, db + 2 * kAtom);
            copy_scales<PAIR>(sfb + 12, db + 3 * kAtom);
          }
          commit_here<PAIR>(full + at.bar);
          at = at.next(8 * stages);
          sfa = at.bar == 0 ? sf0 : sfa + sf_step;
          if ((kt & 1) || kt + 1 == args.k_steps) {
            commit<PAIR>(sempty + sf.bar);
            sf = sf.next(8 * SF_STAGES);
            desc = sf.bar == 0 ? desc0 : desc + desc_step;
          }
        }
      }
      commit<PAIR>(smem_u32(&ctl->cdrain));
      mbar_wait(&ctl->cdrain, 0, &ctl->abort, args.err, 7, true);
    }
    __syncwarp();
  } else if (warp < EPI_WARP0) {
    // ---------------- scale producers ----------------
    // The warps take the 512-value vectors of the CTA's tiles in turn, so that the
    // loads of several are in flight.
    constexpr int kA = BM / 32, kB = MAX_UNITS * UNIT / 32;  // rows of a lane
    const int n_vec = (args.k_steps + 1) / 2;
    int tile = worker, stage = warp - SF_WARP0, kv = stage, e = 0;
    uint32_t phase = 0;
    const uint4 *src_a[kA], *src_b[kB];  // this lane's rows' scales, nullptr for a row that the tile lacks
    for (bool set_up = true;;) {
      for (; kv >= n_vec; kv -= n_vec) {
        tile += workers;
        set_up = true;
      }
      if (tile >= total) break;
      if (set_up) {
        set_up = false;
        const Tile t = decode<PAIR>(ctl, args.E, units, n_tiles, tile, e, rank);
        e = t.e;
#pragma unroll
        for (int c = 0; c < kA; ++c) {
          const int row = t.row0 + 32 * c + lane;
          src_a[c] = row < t.row_end ? reinterpret_cast<const uint4*>(args.a_scale + (int64_t)row * args.pitch)
                                     : nullptr;
        }
        const uint8_t* w = args.b_scale + (int64_t)e * args.b_rows * args.pitch;
#pragma unroll
        for (int c = 0; c < kB; ++c) {
          // gate_up: the tile's gate rows, 32 a unit, then its up rows
          const int up = is_swiglu(MODE) && c >= units ? 1 : 0;
          const int n = is_swiglu(MODE) ? (t.unit0 + c - up * units) * 32 + lane : t.unit0 * UNIT + 32 * c + lane;
          const int64_t row = (int64_t)up * args.N + n;
          src_b[c] = c < 2 * units && n < args.N ? reinterpret_cast<const uint4*>(w + row * args.pitch) : nullptr;
        }
      }
      uint4 va[kA], vb[kB];
#pragma unroll
      for (int c = 0; c < kA; ++c) va[c] = src_a[c] ? __ldg(src_a[c] + kv) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int c = 0; c < kB; ++c) vb[c] = src_b[c] ? __ldg(src_b[c] + kv) : make_uint4(0, 0, 0, 0);
      if (!warp_wait(&ctl->sempty[stage], phase ^ 1u, &ctl->abort, args.err, 5)) break;
      uint8_t* const stage_base = sf_base + stage * sf_stage_bytes(units) + lane * 16;
#pragma unroll
      for (int atom = 0; atom < 4; ++atom) {
        // bytes past K / 32 are the caller's padding and count as zeros: the last MMA may take in one
        const int valid = args.K / mx4::kBlock - kv * 16 - atom * 4;
        const uint32_t mask = valid >= 4 ? 0xffffffffu : valid <= 0 ? 0u : (1u << (8 * valid)) - 1u;
        auto word = [&](const uint4& v) {
          return mask & (atom == 0 ? v.x : atom == 1 ? v.y : atom == 2 ? v.z : v.w);
        };
        *reinterpret_cast<uint4*>(stage_base + atom * SF_ATOM_BYTES) =
            make_uint4(word(va[0]), word(va[1]), word(va[2]), word(va[3]));
        const uint4 lo = make_uint4(word(vb[0]), word(vb[1]), word(vb[2]), word(vb[3]));
        uint8_t* dst_b = stage_base + 4 * SF_ATOM_BYTES;
        if (blocks == 2) {
          *reinterpret_cast<uint4*>(dst_b + 2 * atom * SF_ATOM_BYTES) = lo;
          *reinterpret_cast<uint4*>(dst_b + (2 * atom + 1) * SF_ATOM_BYTES) =
              make_uint4(word(vb[4]), word(vb[5]), 0u, 0u);
        } else {
          *reinterpret_cast<uint4*>(dst_b + atom * SF_ATOM_BYTES) = lo;
        }
      }
      fence_to_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(PAIR && !leader ? &ctl->sready[stage] : &ctl->sfull[stage]);
      }
      kv += SF_WARPS;
      stage += SF_WARPS;
      if (stage >= SF_STAGES) {
        stage -= SF_STAGES;
        phase ^= 1u;
      }
    }
    __syncwarp();
  } else {
    // ---------------- epilogue: four warps take the first accumulator's tiles, four the second's ----------------
    const int quarter = warp & 3;  // TMEM lanes this warp may access
    const int acc = (warp - EPI_WARP0) >> 2;
    const uint32_t tbase = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * ACC_COLS);
    auto release = [&] {  // the warp has read the accumulator
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_remote(mapa_shared(smem_u32(&ctl->tempty[acc]), 0));
        else mbar_arrive(&ctl->tempty[acc]);
      }
    };
    uint8_t* stg = staging + (warp - EPI_WARP0) * STAGING_BYTES;
    uint32_t acc_phase = 0;
    int e = 0;
    [[maybe_unused]] int other = 0;
    for (int tile = worker + acc * workers; tile < total; tile += 2 * workers) {
      const Tile t = decode<PAIR>(ctl, args.E, units, n_tiles, tile, e, rank);
      e = t.e;
      const int row_w0 = t.row0 + quarter * 32;
      const int nrows = t.row_end - row_w0;
      if (!warp_wait(&ctl->tfull[acc], acc_phase, &ctl->abort, args.err, 4)) break;
      acc_phase ^= 1u;
      tc_fence_after();
      if (nrows > 0) {
        if constexpr (is_swiglu(MODE)) {
          const int count = min(units, args.n_units - t.unit0);
#pragma unroll 1
          for (int j = 0; j < count; ++j) {
            uint32_t g[32], u[32];
            tmem_ld32(tbase + j * 32, g);
            tmem_ld32(tbase + (units + j) * 32, u);
            tmem_ld_wait_regs(g);
            tmem_ld_wait_regs(u);
            if (j + 1 == count) release();  // the tile's last read
            const int n0 = (t.unit0 + j) * 32;  // N is a multiple of 32: the block lies inside
            uint32_t h[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              h[i] = pack_bf16x2(silu(__uint_as_float(g[2 * i])) * __uint_as_float(u[2 * i]),
                                 silu(__uint_as_float(g[2 * i + 1])) * __uint_as_float(u[2 * i + 1]));
            if constexpr (MODE == SWIGLU_BF16) {
              uint8_t* box = stg + other;  // two buffers in turn
              other ^= 32 * 64;
              box_free<1>(lane);
#pragma unroll
              for (int c = 0; c < 4; ++c)
                *reinterpret_cast<uint4*>(box + staged<64>(lane, c)) =
                    make_uint4(h[4 * c], h[4 * c + 1], h[4 * c + 2], h[4 * c + 3]);
              store_box<64>(box, &maps.out, n0, row_w0,
                            reinterpret_cast<uint8_t*>(args.out) + ((int64_t)row_w0 * args.N + n0) * 2,
                            (int64_t)args.N * 2, nrows, 64, lane);
            } else {
              // the lane's own row: 32 values, one scale
              uint32_t m = 0;
#pragma unroll
              for (int i = 0; i < 16; ++i) m = max(m, max((h[i] << 16) & 0x7fffffffu, h[i] & 0x7fff0000u));
              const uint32_t b = mx4::scale_byte(m);
              const float inv = mx4::inverse_scale(b);
              uint32_t code[4];
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                float f[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  f[2 * i] = __uint_as_float(h[4 * c + i] << 16) * inv;
                  f[2 * i + 1] = __uint_as_float(h[4 * c + i] & 0xffff0000u) * inv;
                }
                code[c] = b == mx4::kScaleNaN ? 0u : mx4::pack8(f);
              }
              if (lane < nrows) {
                const int64_t row = row_w0 + lane;
                *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(args.out) + (row * args.N + n0) / 2) =
                    make_uint4(code[0], code[1], code[2], code[3]);
                uint8_t* s = args.out_scale + row * args.out_pitch;
                s[n0 / 32] = (uint8_t)b;
                if (n0 + 32 == args.N)  // the row's last block also writes the padding
                  for (int i = args.N / 32; i < args.out_pitch; ++i) s[i] = 0;
              }
            }
          }
        } else {
          const int n0 = t.unit0 * UNIT;
          const int count = min(units * UNIT, args.N - n0);
          constexpr int kCols = MODE == OUT_BF16 ? 64 : 32;  // 128 bytes of a row
          constexpr int es = MODE == OUT_BF16 ? 2 : 4;
#pragma unroll 1
          for (int c0 = 0; c0 < count; c0 += kCols) {
            uint32_t v[32];
            if constexpr (MODE == OUT_BF16) {
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                uint32_t d[32];
                tmem_ld32(tbase + c0 + half * 32, d);
                tmem_ld_wait_regs(d);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  v[half * 16 + i] = pack_bf16x2(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1]));
              }
            } else {
              tmem_ld32(tbase + c0, v);
              tmem_ld_wait_regs(v);
            }
            if (c0 + kCols >= count) release();  // the tile's last read
            box_free<0>(lane);
#pragma unroll
            for (int c = 0; c < 8; ++c)
              *reinterpret_cast<uint4*>(stg + staged<128>(lane, c)) =
                  make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
            store_box<128>(stg, &maps.out, n0 + c0, row_w0,
                           reinterpret_cast<uint8_t*>(args.out) + ((int64_t)row_w0 * args.N + n0 + c0) * es,
                           (int64_t)args.N * es, nrows, min(128, (count - c0) * es), lane);
          }
        }
      } else {
        release();
      }
    }
    if constexpr (MODE != SWIGLU_MX4) box_free<0>(lane);
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) {
    // The leader's last commits arrive in the second CTA too. (It waits for them here, where they are due, and not
    // from its start on: a wait is shorter than a large product.)
    if (!leader && warp == 1) {
      if (lane == 0) {
        mbar_wait(&ctl->drain, 0, &ctl->abort, args.err, 7, true);
        mbar_wait(&ctl->cdrain, 0, &ctl->abort, args.err, 7, true);
      }
      __syncwarp();
    }
    cluster_sync_all();  // no remote arrive or pair MMA still targets either CTA
  }
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    if constexpr (PAIR) tmem_dealloc2(tmem_base, TMEM_COLS);
    else tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

template <int MODE>
__global__ void __launch_bounds__(GTHREADS, 1) mx4_gemm_kernel(const __grid_constant__ Maps maps, const Args args) {
  mx4_gemm<MODE, false>(maps, args);
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(GTHREADS, 1)
    mx4_pair_gemm_kernel(const __grid_constant__ Maps maps, const Args args) {
  mx4_gemm<MODE, true>(maps, args);
}

template <int MODE, bool PAIR>
cudaError_t launch(int64_t rows, int64_t E, int64_t N, int64_t K, const void* a_data, const void* a_scale,
                   const int32_t* offsets, const void* w_data, const void* w_scale, void* out, void* out_scale,
                   int32_t* err, cudaStream_t s) {
  static std::once_flag once[kSmemAttrDevices];  // one set per kernel instance
  static cudaError_t attr[kSmemAttrDevices];
  void (*const kernel_fn)(Maps, Args) = PAIR ? mx4_pair_gemm_kernel<MODE> : mx4_gemm_kernel<MODE>;
  const void* kernel = reinterpret_cast<const void*>(kernel_fn);
  const cudaError_t e = set_max_dynamic_smem_once(kernel, (int)kSmemBytes, once, attr);
  if (e != cudaSuccess) return e;
  if (!get_encode()) return cudaErrorNotSupported;
  Maps maps;
  for (int i = 0; i < (rows > BM - A_BOX_ROWS ? 2 : 1); ++i) {  // fewer rows never fill the tile's box
    const uint64_t dims[2] = {(uint64_t)K / 2, (uint64_t)rows};
    const uint64_t strides[1] = {(uint64_t)K / 2};
    const uint32_t box[2] = {BK / 2, (uint32_t)(i == 0 ? A_BOX_ROWS : BM)};
    if (!make_tensor_map(i == 0 ? &maps.a_box : &maps.a_tile, CU_TENSOR_MAP_DATA_TYPE_UINT8,
                         CU_TENSOR_MAP_SWIZZLE_128B, a_data, 2, dims, strides, box))
      return cudaErrorInvalidValue;
  }
  for (int u = 1; u <= (PAIR ? 1 : MAX_UNITS); ++u) {
    // W [E][halves][N][K/2]: gate_up's two halves, or one
    const uint64_t halves = is_swiglu(MODE) ? 2 : 1;
    const uint64_t dims[4] = {(uint64_t)K / 2, (uint64_t)N, halves, (uint64_t)E};
    const uint64_t strides[3] = {(uint64_t)K / 2, (uint64_t)N * K / 2, halves * (uint64_t)N * K / 2};
    const uint32_t box[4] = {BK / 2, PAIR ? MAX_UNITS * UNIT / 2u : (uint32_t)(u * UNIT / halves),
                             PAIR ? 1u : (uint32_t)halves, 1};
    if (!make_tensor_map(&maps.b[u - 1], CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, w_data, 4, dims,
                         strides, box))
      return cudaErrorInvalidValue;
  }
  if (MODE != SWIGLU_MX4) {
    const uint64_t es = MODE == OUT_F32 ? 4 : 2;
    const uint64_t dims[2] = {(uint64_t)N, (uint64_t)rows};
    const uint64_t strides[1] = {(uint64_t)N * es};
    const uint32_t box[2] = {MODE == OUT_BF16 ? 64u : 32u, 32};
    if (!make_tensor_map(&maps.out,
                         MODE == OUT_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                         MODE == SWIGLU_BF16 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, out, 2, dims,
                         strides, box))
      return cudaErrorInvalidValue;
  }
  Args a{};
  a.offsets = offsets;
  a.E = (int32_t)E;
  a.rows_total = rows;
  a.N = (int32_t)N;
  a.n_units = (int32_t)ceil_div(N, is_swiglu(MODE) ? UNIT / 2 : UNIT);
  a.k_steps = (int32_t)ceil_div(K, BK);
  a.K = (int32_t)K;
  a.a_scale = static_cast<const uint8_t*>(a_scale);
  a.b_scale = static_cast<const uint8_t*>(w_scale);
  a.pitch = (int32_t)mx4::scale_pitch(K);
  a.b_rows = N * (is_swiglu(MODE) ? 2 : 1);
  a.out = out;
  a.out_scale = static_cast<uint8_t*>(out_scale);
  a.out_pitch = (int32_t)mx4::scale_pitch(N);
  a.err = err;
  // tiles of one unit, or of a pair
  const int64_t most = PAIR ? (rows / (2 * BM) + std::min<int64_t>(rows, E)) * ceil_div(a.n_units, MAX_UNITS)
                            : (rows / BM + std::min<int64_t>(rows, E)) * a.n_units;
  const int workers = (int)std::max<int64_t>(1, std::min<int64_t>(num_sms() / (PAIR ? 2 : 1), most));
  kernel_fn<<<workers * (PAIR ? 2 : 1), GTHREADS, kSmemBytes, s>>>(maps, a);
  return cudaGetLastError();
}

// Pairs halve the traffic of W but fill 256-row tiles: they pay from about 512
// rows an expert on (us, one CTA / pairs, unequal segments of 384, 512, 768 and
// 1024 rows in the mean: product of 64 experts, N 4096, K 2048 135 / 138, 169 / 167,
// 236 / 230, 304 / 292; of 128 experts, N 2048, K 768 70 / 73, 87 / 88, 123 / 122,
// 159 / 157; gate_up of 64 experts, H 4096, I 2048 253 / 251, 318 / 304, 443 / 416,
// 565 / 526), and lose with few steps a pair (gate_up of 16 experts, H 1024, I 512
// at 768: 17.9 / 20.7).
bool use_pairs(int64_t rows, int64_t E, int64_t n_units, int64_t k_steps) {
  return rows >= 512 * E && rows / (2 * BM) * ceil_div(n_units, MAX_UNITS) * k_steps >= 64 * (num_sms() / 2);
}

template <int MODE>
cudaError_t launch_product(int64_t rows, int64_t E, int64_t N, int64_t K, const void* a_data, const void* a_scale,
                           const int32_t* offsets, const void* w_data, const void* w_scale, void* out, void* out_scale,
                           int32_t* err, cudaStream_t s) {
  const bool pairs = use_pairs(rows, E, ceil_div(N, is_swiglu(MODE) ? UNIT / 2 : UNIT), ceil_div(K, BK));
  return pairs ? launch<MODE, true>(rows, E, N, K, a_data, a_scale, offsets, w_data, w_scale, out, out_scale, err, s)
               : launch<MODE, false>(rows, E, N, K, a_data, a_scale, offsets, w_data, w_scale, out, out_scale, err, s);
}

bool ok_ptr(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// rows, E, N, K of a product; rows and tiles are counted in 32 bits, and the last
// tile of a segment that ends at the last row reaches up to 2 * BM - 1 rows past it.
// K: the second accumulator's epilogue waits for two whole tiles, and a wait gives
// up after 2e9 clocks; a step of 256 that streams its operands from HBM takes some
// 1300, so the 2^20 steps of two tiles of 2^27 stay below it.
constexpr int64_t kMaxK = int64_t(1) << 27;
moe_status check_sizes(int64_t rows, int64_t E, int64_t N, int64_t K, int64_t n_multiple) {
  const int64_t lim = int64_t(1) << 31;
  if (rows < 0 || rows >= lim - 2 * BM || E < 1 || E > kMaxExperts || N < 1 || N >= lim / 4 || K < 1 || K >= kMaxK)
    return MOE_ERR_INVALID_ARGUMENT;
  if (K % mx4::kBlock != 0 || N % n_multiple != 0) return MOE_ERR_INVALID_ARGUMENT;
  if ((rows / BM + E) * ceil_div(N, 32) >= lim - 4096) return MOE_ERR_INVALID_ARGUMENT;  // a round of tiles beyond
  return MOE_OK;
}

bool ok_ws(const void* ws) { return (reinterpret_cast<uintptr_t>(ws) & 15u) == 0; }

}  // namespace
}  // namespace stm

using namespace stm;

MOE_API moe_status moe_mx4_grouped_matmul(int64_t rows, int64_t E, int64_t N, int64_t K, int32_t out_dtype,
                                          const void* a_data, const void* a_scale, const int32_t* offsets,
                                          const void* w_data, const void* w_scale, void* out, void* ws,
                                          moe_stream_t stream) {
  const moe_status st = check_sizes(rows, E, N, K, 8);
  if (st != MOE_OK) return st;
  if (out_dtype != MOE_DTYPE_F32 && out_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARGUMENT;
  if (rows == 0) return MOE_OK;
  if (!ok_ptr(a_data) || !ok_ptr(a_scale) || !ok_ptr(offsets) || !ok_ptr(w_data) || !ok_ptr(w_scale) || !ok_ptr(out) ||
      !ok_ws(ws))
    return MOE_ERR_INVALID_ARGUMENT;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int32_t* err = static_cast<int32_t*>(ws);
  const cudaError_t e =
      out_dtype == MOE_DTYPE_F32
          ? launch_product<OUT_F32>(rows, E, N, K, a_data, a_scale, offsets, w_data, w_scale, out, nullptr, err, s)
          : launch_product<OUT_BF16>(rows, E, N, K, a_data, a_scale, offsets, w_data, w_scale, out, nullptr, err, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

MOE_API moe_status moe_mx4_grouped_gate_up(int64_t rows, int64_t E, int64_t I, int64_t H, const void* a_data,
                                           const void* a_scale, const int32_t* offsets, const void* w_data,
                                           const void* w_scale, void* h, void* h_scale, void* ws,
                                           moe_stream_t stream) {
  const moe_status st = check_sizes(rows, E, I, H, 32);
  if (st != MOE_OK) return st;
  if (rows == 0) return MOE_OK;
  if (!ok_ptr(a_data) || !ok_ptr(a_scale) || !ok_ptr(offsets) || !ok_ptr(w_data) || !ok_ptr(w_scale) || !ok_ptr(h) ||
      !ok_ws(h_scale) || !ok_ws(ws))
    return MOE_ERR_INVALID_ARGUMENT;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int32_t* err = static_cast<int32_t*>(ws);
  const cudaError_t e =
      h_scale == nullptr
          ? launch_product<SWIGLU_BF16>(rows, E, I, H, a_data, a_scale, offsets, w_data, w_scale, h, nullptr, err, s)
          : launch_product<SWIGLU_MX4>(rows, E, I, H, a_data, a_scale, offsets, w_data, w_scale, h, h_scale, err, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
