// Products of 4-bit rows and 4-bit weights on the block-scaled tensor cores (tcgen05 kind::mxf4nvf4 and
// kind::mxf4, TMEM, TMA): the expert FFN's grouped GEMMs and the product of two matrices.
//
//   mode 0  H = quantise(silu(A W_gate^T) * (A W_up^T)), codes and block scales, from the fp32 product
//   mode 1  yd (bf16) = (A W_down^T) * row_weight
//   mode 2  y (bf16 or fp32) = A B^T, one group
//
// A and B are e2m1 codes, two a byte, row-major along K, with a scale byte for 16 (NVFP4, e4m3) or 32
// (MXFP4, e8m0) elements; the tensor core multiplies codes and scales itself and accumulates in fp32, so
// nothing is expanded: a K block of 256 elements is one 128-byte swizzled row of shared memory. The fp32
// product is rounded once, to the output; H is quantised from it without a bf16 step between.
//
//   * tiles of 128 rows x 256 columns (mode 0: 128 gate and the 128 matching up columns), persistent,
//     one CTA per SM: a 4-stage ring of 48 KB for the codes (TMA), a 2-slot ring of 12 KB for the scales.
//   * scales: `tcgen05.mma` reads them from TMEM, where row r of a 128-row operand has its 4 scale bytes
//     of a step in lane r % 32 of column r / 32, repeated in the four lane quarters; `tcgen05.cp
//     .32x128b.warpx4` copies 512 bytes of shared memory [32 lanes][4 columns][4 bytes] there. The scales
//     stay row-major in HBM (the layout of the quantised weights, a plain copy of a checkpoint): six
//     warps load 32-byte sectors of the rows, one or two at once, and store them transposed, a 16-byte line
//     per step. (16 bytes a row from each of four warps: 307 us where sectors took 208, 8192 x 14336 x 4096
//     NVFP4.)
//   * TMEM: two accumulators of 256 columns do not leave room for the scales, so they share 48: columns
//     [0, 256) and [208, 464), scales in [464, 512). The epilogue reads the shared columns of a tile
//     first and hands them over; the next tile's MMAs then run beside the rest of the epilogue. (Two
//     whole accumulators of 192 columns do without that wait, but a K block takes as long for fewer
//     columns: 207 us where this took 189.)
//   * few tiles: of 64 columns each (mode 0: 32 + 32), in a ring of 8 stages of 24 KB, so that more SMs load the
//     weights. (A cluster of 2 - 8 CTAs that shares a tile's K and adds its sums through distributed shared memory
//     gained only past K = 4096, and cost 2 us otherwise: 1 x 4096 x 14336 25 -> 16 us, 1 x 7168 x 2048 7.2 -> 9.1.)
//   * eight epilogue warps, two per TMEM lane quarter; in mode 0 a lane holds whole quantisation blocks
//     of its row, so H is quantised in registers.
//   * a tile of at most 96 rows loads only the 32-row boxes that hold rows (a few rows an expert: the
//     weights are the traffic); the rest of the tile keeps stale codes, whose products are not stored.
//
// What bounds it (GB300, 2.07 GHz). Few rows a group: HBM; the experts of a 256-token step, 226 of 256 active, h
// 7168, I 2048: 0.82 - 0.83 ms, 6.8 TB/s (a copy: 6.8). Many rows: 8192 x 14336 x 4096 185 us out of HBM and 175 - 178
// out of L2 (NVFP4, 5.2 and 5.5 PFLOP/s), 169 and 162 - 165 us (MXFP4); fp32 output 227 and 214 us out of L2. The
// comparisons of variants, here and below, are with inputs in L2. A K block takes 512 cycles of MMA and about 600 with
// the scales' copies in the same queue, but 700 - 1000 while an epilogue stores: an SM sends L2 one request a cycle, 384
// of a K block for the codes, 96 for the scales, and 2048 a tile for its output. A short K feels the last most: 16384 x
// 7168 x 2048 107 us out of HBM, 104 out of L2 (NVFP4, 4.6 PFLOP/s). Without the stores the two NVFP4 products would take
// 166 and 91 us, without half of B's codes 177 and 112 when they took 190 and 116. The wait at a tile boundary hides
// behind those requests (a first K block in two halves, the one without shared columns before the wait: no change). CTA
// pairs (tcgen05.mma.cta_group::2, 256 x 256 and 256 x 192) halve the codes' requests, but each cta_group::2 scale copy
// holds the queue for about 40 cycles instead of 11: 225 - 265 us. A single token: launch, set-up and 8 K blocks in a
// row, 6.2 us for 7168 x 2048; a long K is walked alone by each of the few CTAs, 20 us for 4096 x 14336 (56 blocks).
// Ragged sizes: 1000 x 4096 x 2048 takes 8.0 us (NVFP4; MXFP4 7.6), with 4101 columns, whose rows are stored element by
// element, 10.6; with K 2080, whose rows of scales are no whole 16 bytes and are loaded byte by byte, 18.5 (11.1); with
// both 21.1 (14.1).
#include <cuda.h>

#include <algorithm>

#include "common.cuh"
#include "fp4_impl.cuh"
#include "gemm_a4_host.h"
#include "gemm_common.cuh"
#include "kernels.h"

namespace moe {
namespace a4 {

constexpr int BM = 128;
constexpr int BN = 256;        // columns of a wide tile
constexpr int BN_NARROW = 64;  // of a narrow one
constexpr int BK = 256;        // elements of a K block: 128 bytes of codes
constexpr int A_BYTES = BM * BK / 2;
template <int NB>
constexpr int kBBytes = NB * BK / 2;
template <int NB>
constexpr int kStageBytes = A_BYTES + kBBytes<NB>;
constexpr int RING_BYTES = 4 * kStageBytes<BN>;
template <int NB>
constexpr int kStages = RING_BYTES / kStageBytes<NB>;  // 4 or 8
constexpr int MAX_STAGES = kStages<BN_NARROW>;
constexpr int SLOTS = 2;                 // ring of scales
constexpr int SLOT_WORDS = 8;            // 4-byte words of scales of a row in a slot: a 32-byte sector
constexpr int SLOT_BYTES = SLOT_WORDS * (BM + BN) * 4;
constexpr int SCALE_WARP0 = 2;
constexpr int SCALE_WARPS = 6;           // 3 blocks of 128 rows (A, two of B) x 2 slots
constexpr int EPI_WARP0 = SCALE_WARP0 + SCALE_WARPS;
template <int FMT>
constexpr int kWords = BK / fp4::kBlock<FMT> / 4;  // words of a row's K block
template <int FMT>
constexpr int kSlotBlocks = SLOT_WORDS / kWords<FMT>;  // K blocks of a slot
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
constexpr int ACC1 = 208;    // column of the second accumulator
constexpr int SFA_COL = 464;
constexpr int SFB_COL = 480;

constexpr int SMEM_BYTES = RING_BYTES + SLOTS * SLOT_BYTES + 1024;

struct Args {
  const int32_t* offsets;
  const int32_t* slot_expert;
  int E, shared, R, T, K, N, n_tiles, mode, I, f32;
  int a_rows, b_rows;
  const uint8_t* a_scales;
  const uint8_t* b_scales;
  const uint8_t* bs_scales;
  const float* a_g;
  const float* b_g;
  const float* bs_g;
  int64_t ldo;
  int aligned;  // output rows start on 16 bytes
  int scales32;  // all scales' addresses are on 32 bytes
  void* out;
  uint8_t* out_scales;
  const float* out_g;
  const float* row_weight;
  int* status;
  long long wait_limit;
};

struct Shared {
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  uint64_t sfull[SLOTS];
  uint64_t sempty[SLOTS];
  uint64_t tfull[2];
  uint64_t tfree;
  uint64_t mma_done;
  uint32_t tmem_slot;
  volatile int abort_flag;
  grp::Table tb;
};

using grp::wait_or_abort;

// where a launch without a status word records a wait that gave up (moe_matmul_fp4_status)
__device__ int default_status;

// One lane of a converged warp, the same one on every call.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, e;\n\t}"
      : "=r"(p));
  return p;
}

// The instructions of the MMA thread are issued by one lane (`one`) of a warp that walks its loop together: their
// operands are then computed once for the warp, in uniform registers. In a branch that one lane had taken alone,
// each operand went through vector registers first.

// D (+)= A * B^T with block scales in TMEM; K = 64 elements. a, b: the low words of the operands' descriptors.
template <int FMT>
__device__ __forceinline__ void umma_fp4(uint32_t one, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
  // high word: stride 1024 bytes between groups of 8 rows, version 1, 128-byte swizzle (sw128_kmajor_desc)
  constexpr uint32_t kHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
  if (FMT == fp4::kNv)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "mov.b64 da, {%1, %8};\n\tmov.b64 db, {%2, %8};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], da, db, %3, [%4], [%5], p;\n\t}" ::"r"(
            d),
        "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(one), "r"(kHigh)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "mov.b64 da, {%1, %8};\n\tmov.b64 db, {%2, %8};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(one), "r"(kHigh)
        : "memory");
}
__device__ __forceinline__ uint32_t operand_desc(uint32_t saddr) { return saddr >> 4 | 1u << 16; }

// 512 bytes of scales [32][16] (no swizzle, groups of 8 lines 128 bytes apart) from shared memory to 4 TMEM columns,
// once for each lane quarter.
__device__ __forceinline__ void copy_scales(uint32_t one, uint32_t taddr, uint32_t desc) {
  constexpr uint32_t kHigh = (128u >> 4) | 1u << 14;
  asm volatile(
      "{\n\t.reg .pred q;\n\t.reg .b64 ds;\n\t"
      "setp.ne.b32 q, %2, 0;\n\tmov.b64 ds, {%1, %3};\n\t"
      "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], ds;\n\t}" ::"r"(taddr),
      "r"(desc), "r"(one), "r"(kHigh)
      : "memory");
}
__device__ __forceinline__ uint32_t scales_desc(uint32_t saddr) { return saddr >> 4 | (128u >> 4) << 16; }

__device__ __forceinline__ void commit(uint32_t one, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(one)
      : "memory");
}

// Instruction descriptor: e2m1 operands, both K-major, fp32 accumulators; scales e4m3 (NVFP4) or e8m0.
template <int FMT>
__host__ __device__ constexpr uint32_t idesc_fp4(int M, int N) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (FMT == fp4::kNv ? 0u : 1u << 23) |
         ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 32 scale bytes of a row at p, of which the row has `left` (more, fewer or none): the rest are 0. `whole`: rows are
// whole 32-byte sectors; with VEC alone they are whole 16-byte halves.
template <bool VEC>
__device__ __forceinline__ void load_scales(uint32_t (&w)[8], const uint8_t* p, int left, bool whole) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 0;
  if constexpr (VEC) {
    if (whole) {
      if (left > 0)
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
      return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (left <= 16 * h) continue;
      const uint4 v = reinterpret_cast<const uint4*>(p)[h];
      w[4 * h] = v.x, w[4 * h + 1] = v.y, w[4 * h + 2] = v.z, w[4 * h + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < left) w[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
  }
}

// The scales' copies and the MMAs of one K block: codes at a (A) and b (B), scales of its words at sf. Copies and
// MMAs of one thread run in order: the copies wait for the MMAs that read the columns they write.
template <int FMT, int NB>
__device__ __forceinline__ void issue_k_block(uint32_t one, uint32_t tmem, uint32_t d, uint32_t a, uint32_t b, uint32_t sf,
                                              bool first) {
  constexpr uint32_t IDESC = idesc_fp4<FMT>(BM, NB);
  const uint32_t da = operand_desc(a), db = operand_desc(b), ds = scales_desc(sf);
#pragma unroll
  for (int i = 0; i < kWords<FMT>; ++i) {
    copy_scales(one, tmem + SFA_COL + 4 * i, ds + 96 * i);
    copy_scales(one, tmem + SFB_COL + 8 * i, ds + 96 * i + 32);
    if (NB > 128) copy_scales(one, tmem + SFB_COL + 8 * i + 4, ds + 96 * i + 64);
  }
#pragma unroll
  for (int kk = 0; kk < BK / 64; ++kk) {
    const int w = FMT == fp4::kNv ? kk : kk / 2;               // word of the scales
    const uint32_t id = FMT == fp4::kNv ? 0u : 2u * (kk & 1);  // bytes of it: all four, or a half
    umma_fp4<FMT>(one, d, da + 2 * kk, db + 2 * kk, IDESC | id << 4 | id << 29, tmem + SFA_COL + 4 * w,
                  tmem + SFB_COL + 8 * w, !(first && kk == 0));
  }
}

// Scale producers: six warps, two for each 128-row block (A, the first and the second of B). A lane stores a 16-byte
// line for each word of a slot, of rows l, l + 32, l + 64 and l + 96.
//
// NVFP4: both warps of a block fill every slot, 16 of its lines each. Even lanes load a slot's sector of their rows
// and odd lanes the next slot's, so that a row is asked for once in two slots (8192 x 14336 x 4096: 178 us; with a
// sector at a time, as below, 191).
// MXFP4, with half as many scales: each warp of a block has a slot of its own and loads a sector of all rows for it
// (8192 x 14336 x 4096 and 16384 x 7168 x 2048: 165 and 97 us; two sectors at once, which is a tile's whole row in the
// second, 166 and 100). Rows that are loaded byte by byte go the first way, for fewer rows an instruction.
//
// The next loads are issued once the last sector is stored, a slot's use ahead of the first wait for room. No warp
// waits for a slot more than a phase ahead, which a parity could not tell. Tiles first, first + step, ...
template <int FMT, bool VEC>
constexpr int kPiece = FMT == fp4::kNv || !VEC ? 2 : 1;  // sectors of a row loaded at once, and warps that fill a slot's block
template <int FMT, bool VEC, bool SWIGLU, int NB>
__device__ __forceinline__ void scale_producer(const Args& args, const grp::Table& tb, int warp, int lane, uint32_t slots,
                                               int first, int step, uint64_t* sempty, uint64_t* sfull,
                                               volatile int* abort_flag, int* status) {
  constexpr int PIECE = kPiece<FMT, VEC>;
  static_assert(SLOTS == 2 && SCALE_WARPS == 6 && SLOT_WORDS == 8, "two warps a block, a sector a slot");
  const int G = args.E + args.shared;
  const int total = tb.gtile[G] * args.n_tiles;
  const int kblocks = (args.K + BK - 1) / BK;
  const int block = (warp - SCALE_WARP0) >> 1, member = (warp - SCALE_WARP0) & 1;
  if (NB <= 128 && block == 2) return;
  const int line = PIECE == 1 ? lane : 16 * member + lane / 2, q = PIECE == 1 ? 0 : lane % 2;
  const int pitch = args.K / fp4::kBlock<FMT>;
  const bool whole = pitch % 32 == 0 && args.scales32;
  const int per_tile = (kblocks + kSlotBlocks<FMT> - 1) / kSlotBlocks<FMT>;
  const uint32_t dst = slots + (uint32_t)(block * 512 + 16 * line);
  int fill = 0;  // fill number i of this CTA is slot i % 2
  for (int tile = first; tile < total; tile += step) {
    const grp::Tile t = grp::decode(tb, G, args.n_tiles, tile, BM);
    const bool routed = t.g < args.E;
    const int64_t z = routed ? (args.slot_expert ? args.slot_expert[t.g] : t.g) : 0;
    const int n0 = SWIGLU ? t.n_tile * (NB / 2) : t.n_tile * NB;
    const int n1 = SWIGLU ? args.I + n0 : n0 + NB / 2;
    const int r0 = block == 0 ? t.a_row : block == 1 ? n0 : n1;
    const int rows = block == 0 ? args.a_rows : args.b_rows;
    const uint8_t* base = block == 0 ? args.a_scales
                      : (routed ? args.b_scales : args.bs_scales) + z * args.b_rows * (int64_t)pitch;
    const uint8_t* p[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // a narrow tile has two rows of B a line; the other words hold them again, and are not used
      const int r = NB == 64 && block == 1 ? (j & 1 ? n1 : n0) : r0 + 32 * j;
      // rows past the end take the last one's scales: they are not stored
      p[j] = base + min(r + line, rows - 1) * (int64_t)pitch + 32 * q;
    }
    for (int f = 0; f < per_tile; f += PIECE) {
      if (PIECE == 1 && (fill & 1) != member) {
        ++fill;
        continue;
      }
      uint32_t v[4][8];
#pragma unroll
      for (int j = 0; j < 4; ++j) load_scales<VEC>(v[j], p[j] + 32 * f, pitch - 32 * (f + q), whole);
#pragma unroll
      for (int o = 0; o < PIECE; ++o) {
        if (f + o >= per_tile) break;
        const int slot = fill & 1;
        const int got = wait_or_abort(&sempty[slot], (uint32_t)(fill >> 1 & 1) ^ 1, abort_flag, status, args.wait_limit);
        if (!__all_sync(0xffffffffu, got)) return;
        ++fill;
        if (q == o) {
#pragma unroll
          for (int w = 0; w < 8; ++w)
            sts128(dst + slot * SLOT_BYTES + 1536 * w, v[0][w], v[1][w], v[2][w], v[3][w]);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfull[slot]);
      }
    }
  }
}

// H of a row quantised and stored: 16 bytes of codes and the scale bytes of their blocks.
template <int FMT>
__device__ __forceinline__ void store_codes(const Args& args, int64_t row, int col, const float (&h)[32],
                                            const fp4::Scale& hg) {
  uint32_t q[4], sc = 0;
  constexpr int kBlk = fp4::kBlock<FMT>;
#pragma unroll
  for (int b = 0; b < 32 / kBlk; ++b) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kBlk; ++j) m = max(m, fp4::abs_bits(h[kBlk * b + j]));
    float by;
    sc |= fp4::block_scale<FMT>(m, hg, by) << (8 * b);
#pragma unroll
    for (int j = 0; j < kBlk / 8; ++j) q[kBlk / 8 * b + j] = fp4::codes8<FMT>(h + kBlk * b + 8 * j, by, m);
  }
  *reinterpret_cast<uint4*>(static_cast<uint8_t*>(args.out) + (row * args.ldo + col) / 2) =
      make_uint4(q[0], q[1], q[2], q[3]);
  uint8_t* so = args.out_scales + (row * args.ldo + col) / kBlk;
  if (FMT == fp4::kNv)
    *reinterpret_cast<uint16_t*>(so) = (uint16_t)sc;
  else
    *so = (uint8_t)sc;
}

// rows of scales that are whole 16-byte pieces are loaded as such, others byte by byte
inline bool scales_vec(const GemmA4Desc& d) {
  return d.K / (d.format == fp4::kNv ? fp4::kBlock<fp4::kNv> : fp4::kBlock<fp4::kMx>) % 16 == 0;
}

// One 128-byte run (64 bf16 or 32 fp32 columns) of each of a warp's 32 rows to the output: lane = row, w = its run. A
// lane that stored its own row would touch 32 lines an instruction, and the stores would hold up the scales' way
// through the same unit. So four lanes exchange their rows' 32-byte quarters first, and an instruction stores 8
// whole lines. `out`: the run of the first row; rows are 16-byte aligned; `rows` of them exist.
template <bool WIDE>
__device__ __forceinline__ void store_lines(char* out, int64_t pitch, int lane, uint32_t (&w)[32], int rows) {
  // after the step over lanes that differ in bit b, words 8 p .. hold quarter (p with that bit the lane's) of the row
  // with that bit p's
#pragma unroll
  for (int b = 1; b < 4; b *= 2) {
    const bool up = lane & b;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if ((i >> 3) & b) continue;
      const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[i] : w[i + 8 * b], b);
      if (up)
        w[i] = got;
      else
        w[i + 8 * b] = got;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = (lane & ~3) + j;
    if (r >= rows) continue;
    char* o = out + r * pitch + 32 * (lane & 3);
    if (WIDE) {
      st_global_v8(o, w + 8 * j);
    } else {
      reinterpret_cast<uint4*>(o)[0] = make_uint4(w[8 * j], w[8 * j + 1], w[8 * j + 2], w[8 * j + 3]);
      reinterpret_cast<uint4*>(o)[1] = make_uint4(w[8 * j + 4], w[8 * j + 5], w[8 * j + 6], w[8 * j + 7]);
    }
  }
}

// The same for rows of any alignment, and runs of which `n` bytes exist: exchanged over all 32 lanes and stored
// element by element, one line an instruction.
__device__ __forceinline__ void store_elements(char* out, int64_t pitch, int lane, uint32_t (&w)[32], int rows, int n,
                                               bool f32) {
#pragma unroll
  for (int b = 16; b > 0; b /= 2) {
    const bool up = lane & b;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (i & b) continue;
      const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[i] : w[i + b], b);
      if (up)
        w[i] = got;
      else
        w[i + b] = got;
    }
  }
  const int at = 4 * lane;
#pragma unroll
  for (int r = 0; r < 32; ++r) {
    if (r >= rows) continue;
    char* o = out + r * pitch + at;
    if (f32) {
      if (at < n) *reinterpret_cast<uint32_t*>(o) = w[r];
    } else {
      if (at < n) reinterpret_cast<uint16_t*>(o)[0] = (uint16_t)w[r];
      if (at + 2 < n) reinterpret_cast<uint16_t*>(o)[1] = (uint16_t)(w[r] >> 16);
    }
  }
}

// What a kernel writes: H in 4 bits; bf16 rows that start on 32 bytes and have whole runs; any rows. A kernel for each:
// in one for all three the epilogue's registers spilled.
enum { kCodes, kLines, kAny };

template <int FMT, bool VEC, int OUT, int NB>
__global__ void __launch_bounds__(THREADS, 1)
    gemm_a4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA32,
                   const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmBs, const Args args) {
  constexpr int STAGES = kStages<NB>, B_BYTES = kBBytes<NB>, STAGE_BYTES = kStageBytes<NB>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared s;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // the same in all lanes, and known to be: the roles' addresses and counters stay in uniform registers
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int G = args.E + args.shared;
  int* status = args.status ? args.status : &default_status;

  if (warp == 0) {
    grp::build_table(s.tb, args.offsets, args.E, args.shared, args.R, args.T, BM, lane);
    if (lane == 0) {
      for (int i = 0; i < STAGES; ++i) {
        mbar_init(&s.full[i], 1);
        mbar_init(&s.empty[i], 1);
      }
      for (int i = 0; i < SLOTS; ++i) {
        mbar_init(&s.sfull[i], (NB > 128 ? 3 : 2) * kPiece<FMT, VEC>);
        mbar_init(&s.sempty[i], 1);
      }
      mbar_init(&s.tfull[0], 1);
      mbar_init(&s.tfull[1], 1);
      mbar_init(&s.tfree, EPI_WARPS);
      mbar_init(&s.mma_done, 1);
      s.abort_flag = 0;
      fence_mbar_init();
      tma_prefetch_desc(&tmA);
      tma_prefetch_desc(&tmA32);
      tma_prefetch_desc(&tmB);
      tma_prefetch_desc(&tmBs);
    }
  }
  if (warp == 1) {
    tmem_alloc(&s.tmem_slot, 512);
    tmem_relinquish();
  }
  // the kernel behind this one in the stream may set itself up now; this one waits here for the one before it
  // (launch_gemm_a4 says which), after its own set-up, which reads offsets that were there before that one began
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = s.tmem_slot;
  const int total = s.tb.gtile[G] * args.n_tiles;
  const int kblocks = (args.K + BK - 1) / BK;
  const uint32_t slots = smem_u32(smem) + RING_BYTES;

  if (warp == 0 && lane == 0) {
    // ---------------- TMA producer
    int stage = 0;
    uint32_t phase = 0;
    long long issued = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      const grp::Tile t = grp::decode(s.tb, G, args.n_tiles, tile, BM);
      const CUtensorMap* mb = t.g < args.E ? &tmB : &tmBs;
      const int z = t.g < args.E ? (args.slot_expert ? args.slot_expert[t.g] : t.g) : 0;
      const int n0 = OUT == kCodes ? t.n_tile * (NB / 2) : t.n_tile * NB;
      const int n1 = OUT == kCodes ? args.I + n0 : n0 + NB / 2;
      const int boxes = (t.rows + 31) / 32;
      const uint32_t a_bytes = boxes == 4 ? A_BYTES : boxes * (A_BYTES / 4);
      for (int kb = 0; kb < kblocks; ++kb) {
        if (!wait_or_abort(&s.empty[stage], phase ^ 1, &s.abort_flag, status, args.wait_limit)) {
          ok = false;
          break;
        }
        uint8_t* a = smem + stage * STAGE_BYTES;
        uint8_t* b = a + A_BYTES;
        mbar_arrive_expect_tx(&s.full[stage], a_bytes + B_BYTES);
        if (boxes == 4)
          tma_load_2d(a, &tmA, &s.full[stage], kb * (BK / 2), t.a_row);
        else
          for (int i = 0; i < boxes; ++i)
            tma_load_2d(a + i * (A_BYTES / 4), &tmA32, &s.full[stage], kb * (BK / 2), t.a_row + 32 * i);
        tma_load_3d(b, mb, &s.full[stage], kb * (BK / 2), n0, z);
        if (OUT == kCodes) tma_load_3d(b + B_BYTES / 2, mb, &s.full[stage], kb * (BK / 2), n1, z);
        ++issued;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    const long long first = issued > STAGES ? issued - STAGES : 0;
    for (long long i = first; i < issued; ++i)
      grp::drain_wait(&s.full[i % STAGES], (uint32_t)((i / STAGES) & 1), args.wait_limit);
  } else if (warp == 1) {
    // ---------------- MMA issuer: the whole warp walks the loop, one lane issues
    const uint32_t leader = elect_one();
    int stage = 0, slot = 0, n = 0;  // n: tiles of this CTA so far
    uint32_t phase = 0, sphase = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x, ++n) {
      // the columns shared with the tile before have been read (and all of the tile before that one)
      if (n > 0 && !__all_sync(0xffffffffu, wait_or_abort(&s.tfree, (uint32_t)(n - 1) & 1, &s.abort_flag, status,
                                                          args.wait_limit)))
        break;
      const uint32_t d = tmem_base + (n & 1 ? ACC1 : 0);
      for (int kb = 0; kb < kblocks; ++kb) {
        const int in_slot = kb % kSlotBlocks<FMT>;
        if (!__all_sync(0xffffffffu,
                        (in_slot > 0 || wait_or_abort(&s.sfull[slot], sphase, &s.abort_flag, status, args.wait_limit)) &&
                            wait_or_abort(&s.full[stage], phase, &s.abort_flag, status, args.wait_limit))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a = smem_u32(smem) + stage * STAGE_BYTES;
        const uint32_t b = a + A_BYTES;
        const uint32_t sf = slots + slot * SLOT_BYTES + in_slot * kWords<FMT> * 3 * 512;
        const bool slot_done = in_slot == kSlotBlocks<FMT> - 1 || kb + 1 == kblocks;
        issue_k_block<FMT, NB>(leader, tmem_base, d, a, b, sf, kb == 0);
        if (slot_done) commit(leader, &s.sempty[slot]);
        commit(leader, &s.empty[stage]);
        if (kb + 1 == kblocks) commit(leader, &s.tfull[n & 1]);
        if (slot_done && ++slot == SLOTS) {
          slot = 0;
          sphase ^= 1;
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (leader) {
      umma_commit(&s.mma_done);
      grp::drain_wait(&s.mma_done, 0, args.wait_limit);
    }
    __syncwarp();
  } else if (warp >= SCALE_WARP0 && warp < EPI_WARP0) {
    scale_producer<FMT, VEC, OUT == kCodes, NB>(args, s.tb, warp, lane, slots, blockIdx.x, gridDim.x, s.sempty, s.sfull,
                                                &s.abort_flag, status);
  } else if (warp >= EPI_WARP0) {
    // ---------------- epilogue
    const int quarter = warp & 3, half = (warp - EPI_WARP0) >> 2;
    const int r = quarter * 32 + lane;
    const uint32_t tq = tmem_base + ((uint32_t)(quarter * 32) << 16);
    const float ag = args.a_g ? *args.a_g : 1.0f;
    const fp4::Scale hg(OUT == kCodes ? args.out_g : nullptr);
    const bool f32 = OUT == kAny && args.f32;
    const int chunks = NB / (f32 ? 32 : 64);  // 32 columns of H, runs of 64 bf16 or 32 fp32 columns
    int n = 0;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x, ++n) {
      const grp::Tile t = grp::decode(s.tb, G, args.n_tiles, tile, BM);
      const bool routed = t.g < args.E;
      const bool valid = r < t.rows;
      const int64_t row = (int64_t)t.a_row + r;
      const float* bg = routed ? args.b_g : args.bs_g;
      float scale = bg ? ag * bg[routed ? (args.slot_expert ? args.slot_expert[t.g] : t.g) : 0] : ag;
      if (args.mode == 1 && valid && routed) scale *= args.row_weight[row];
      const int got = wait_or_abort(&s.tfull[n & 1], (uint32_t)(n >> 1) & 1, &s.abort_flag, status, args.wait_limit);
      if (__any_sync(0xffffffffu, !got)) break;
      __syncwarp();
      tc_fence_after();
      const uint32_t tacc = tq + (n & 1 ? ACC1 : 0);
      const bool any = quarter * 32 < t.rows;  // this quarter has rows
      // Positions in the order that frees the shared columns first (the last 48 of the first accumulator, the first
      // 48 of the second), alternate ones for the two warps of a quarter: the shared columns lie in the first position
      // (of 64 columns) or the first two (of 32). A warp that reads none of them still says here that it is done
      // with the tile before.
      if (half >= chunks) {  // a narrow tile has nothing for this warp
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.tfree);
      }
      for (int i = half; i < chunks; i += 2) {
        const int at = n & 1 ? i : chunks - 1 - i;
        uint32_t w[32], u[32];  // 64 columns; codes: gate and up; fp32 rows: 32
        if (any) {
          tmem_ld32(tacc + (f32 || OUT == kCodes ? 32 : 64) * at, w);
          if (!f32) tmem_ld32(tacc + (OUT == kCodes ? NB / 2 + 32 * at : 64 * at + 32), u);
          tmem_ld_wait_regs(w);
          if (!f32) tmem_ld_wait_regs(u);
        }
        if (i < 2) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.tfree);
        }
        if (!any) continue;
        if (OUT == kCodes) {
          float h[32];
#pragma unroll
          for (int j = 0; j < 32; ++j)
            h[j] = grp::silu(__uint_as_float(w[j]) * scale) * (__uint_as_float(u[j]) * scale);
          if (valid) store_codes<FMT>(args, row, t.n_tile * (NB / 2) + 32 * at, h, hg);
          continue;
        }
        if (f32) {
#pragma unroll
          for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(__uint_as_float(w[j]) * scale);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            w[j] = pack_bf16x2(__uint_as_float(w[2 * j]) * scale, __uint_as_float(w[2 * j + 1]) * scale);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            w[16 + j] = pack_bf16x2(__uint_as_float(u[2 * j]) * scale, __uint_as_float(u[2 * j + 1]) * scale);
        }
        const int col = t.n_tile * NB + (f32 ? 32 : 64) * at, elem = f32 ? 4 : 2;
        char* out = static_cast<char*>(args.out) + (((int64_t)t.a_row + quarter * 32) * args.ldo + col) * elem;
        // rows, and bytes of the 128-byte run, that exist (N may be close to 2^31: not in bytes)
        const int rows = t.rows - quarter * 32, run = min(args.N - col, 128 / elem) * elem;
        if (OUT == kLines) {
          if (run > 0) store_lines<true>(out, args.ldo * elem, lane, w, rows);
        } else if (args.aligned && run == 128) {
          store_lines<false>(out, args.ldo * elem, lane, w, rows);
        } else if (run > 0) {
          store_elements(out, args.ldo * elem, lane, w, rows, run, f32);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

}  // namespace a4

cudaError_t gemm_a4_default_status(int** word) {
  static PerDevice<int*> addr;
  return per_device<int*>(
      addr,
      [](int*& p) {
        void* v = nullptr;
        const cudaError_t r = cudaGetSymbolAddress(&v, a4::default_status);
        p = static_cast<int*>(v);
        return r;
      },
      word);
}

// bytes (32, 16 or fewer: 0) that every output row is aligned to
int row_alignment(const GemmA4Desc& d) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(d.out) | (uintptr_t)(d.ldo * (d.f32 ? 4 : 2));
  return at % 32 == 0 ? 32 : at % 16 == 0 ? 16 : 0;
}

a4::Args gemm_a4_args(const GemmA4Desc& d, int columns) {
  a4::Args a;
  a.offsets = d.offsets;
  a.slot_expert = d.slot_expert;
  a.E = d.E;
  a.shared = d.B_shared != nullptr;
  a.R = d.R;
  a.T = d.T;
  a.K = d.K;
  a.N = d.N;
  a.mode = d.mode;
  a.I = d.I;
  a.f32 = d.f32;
  a.n_tiles = d.mode == 0 ? d.I / (columns / 2) : (int)cdiv(d.N, columns);
  a.a_rows = (int)d.a_rows;
  a.b_rows = (int)d.b_rows;
  a.a_scales = static_cast<const uint8_t*>(d.As);
  a.b_scales = static_cast<const uint8_t*>(d.Bs);
  a.bs_scales = static_cast<const uint8_t*>(d.Bs_shared);
  a.a_g = d.Ag;
  a.b_g = d.Bg;
  a.bs_g = d.Bg_shared;
  a.scales32 = ((reinterpret_cast<uintptr_t>(d.As) | reinterpret_cast<uintptr_t>(d.Bs) |
                 reinterpret_cast<uintptr_t>(d.Bs_shared)) & 31) == 0;
  a.ldo = d.ldo;
  a.aligned = row_alignment(d) >= 16;
  a.out = d.out;
  a.out_scales = static_cast<uint8_t*>(d.out_scales);
  a.out_g = d.out_g;
  a.row_weight = d.row_weight;
  a.status = d.status;
  a.wait_limit = a4::wait_limit(cdiv(d.K, a4::BK));
  return a;
}

cudaError_t launch_gemm_a4(const GemmA4Desc& d, cudaStream_t stream, std::string* err) {
  cudaError_t e = tma_encoder_ready();
  if (e != cudaSuccess) {
    *err = "cuTensorMapEncodeTiled is not available from the driver";
    return e;
  }
  using namespace a4;
  using Kernel = decltype(&gemm_a4_kernel<fp4::kNv, true, kCodes, BN>);
  // [narrow][format][scales in 16-byte pieces][output]
#define MOE_A4_OUTPUTS(FMT, VEC, NB) \
  {gemm_a4_kernel<FMT, VEC, kCodes, NB>, gemm_a4_kernel<FMT, VEC, kLines, NB>, gemm_a4_kernel<FMT, VEC, kAny, NB>}
#define MOE_A4_FORMATS(NB)                                                      \
  {{MOE_A4_OUTPUTS(fp4::kNv, false, NB), MOE_A4_OUTPUTS(fp4::kNv, true, NB)},   \
   {MOE_A4_OUTPUTS(fp4::kMx, false, NB), MOE_A4_OUTPUTS(fp4::kMx, true, NB)}}
  static const Kernel kernels[2][2][2][3] = {MOE_A4_FORMATS(BN), MOE_A4_FORMATS(BN_NARROW)};
#undef MOE_A4_FORMATS
#undef MOE_A4_OUTPUTS
  // the dynamic shared-memory opt-in is a per-device function attribute
  static PerDevice<bool> attr;
  bool attr_set = false;
  e = per_device<bool>(
      attr,
      [](bool& v) {
        cudaError_t r = cudaSuccess;
        const Kernel* all = &kernels[0][0][0][0];
        for (size_t i = 0; i < sizeof(kernels) / sizeof(Kernel) && r == cudaSuccess; ++i)
          r = cudaFuncSetAttribute(all[i], cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
        v = r == cudaSuccess;
        return r;
      },
      &attr_set);
  if (e != cudaSuccess) {
    *err = "cudaFuncSetAttribute failed";
    return e;
  }
  const int64_t rows = d.offsets ? (int64_t)d.R + (d.B_shared ? d.T : 0) : d.T;
  const int64_t groups = d.offsets ? std::min<int64_t>(d.E + (d.B_shared ? 1 : 0), rows) : 1;
  const int64_t row_tiles = row_tiles_at_most(rows, groups, BM);
  // Narrow tiles where all of them run at once. NVFP4, narrow and wide: 128 x 7168 x 2048, 28 wide tiles: 5.7 us and
  // 7.4; 256 x 4096 x 7168, 32: 10.7 and 15.2; 256 x 4864 x 4096, 38: 7.7 and 10.3; 64 rows on 8 experts, h 512, I 256:
  // 8.7 and 10.8. 128 x 14336 x 4096, 56: 12.9 and 11.8.
  const int64_t wide_tiles = row_tiles * (d.mode == 0 ? d.I / (BN / 2) : cdiv(d.N, BN));
  const bool narrow = narrow_tiles(wide_tiles, BN / BN_NARROW, num_sms());
  const int columns = narrow ? BN_NARROW : BN;
  const Args args = gemm_a4_args(d, columns);
  CUtensorMap tA, tA32, tB, tBs;
  const int b_box = d.mode == 0 ? columns / 2 : columns;
  const CUtensorMapDataType U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  // an encode costs a small call about a microsecond: a map that no tile uses is a copy of another
  bool ok = tma_encode_2d(&tA32, d.A, U8, 1, d.a_rows, d.K / 2, a4::BM / 4) &&
            tma_encode_3d(&tB, d.B, U8, 1, d.n_experts, d.b_rows, d.K / 2, b_box);
  tA = tA32;
  tBs = tB;
  if (d.a_rows > a4::BM - 32) ok = ok && tma_encode_2d(&tA, d.A, U8, 1, d.a_rows, d.K / 2, a4::BM);
  if (d.B_shared) ok = ok && tma_encode_3d(&tBs, d.B_shared, U8, 1, 1, d.b_rows, d.K / 2, b_box);
  if (!ok) {
    *err = "cuTensorMapEncodeTiled rejected a 4-bit GEMM operand";
    return cudaErrorInvalidValue;
  }
  const int out = d.mode == 0 ? kCodes : !d.f32 && d.N % 64 == 0 && row_alignment(d) == 32 ? kLines : kAny;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(num_sms(), row_tiles * args.n_tiles));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = d.after_gemm ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kernels[narrow][d.format == fp4::kNv ? 0 : 1][scales_vec(d)][out], tA, tA32, tB, tBs, args);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
