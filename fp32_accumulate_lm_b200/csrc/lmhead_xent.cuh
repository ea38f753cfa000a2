// Softmax cross entropy over the LM head's vocabulary with its gradient, no logits kept.
//
//   z[r, v] = alpha * (sum_k h[r, k] * W[v, k] + bias[v])                 fp32
//   lse_r   = log sum_v exp z[r, v],   loss_r = lse_r - z[r, t_r] + z_loss * lse_r^2
//   d[r, v] = a_r * exp(z[r, v] - lse_r) - b_r * [v == t_r]               fp32, rounded to 16 bits
//   dH      = scale * d @ W,   dW = scale * d^T @ h,   dbias = scale * sum_r d[r, v]
//
// with a_r = 1 + 2 z_loss lse_r and b_r = 1 where every row has the same upstream gradient g (then
// scale = alpha * g / rows that count), or both times g_r where each row has its own (scale =
// alpha). So with one upstream gradient the target's entry of a row is p - 1, and g itself is never
// rounded to 16 bits. A power of two 2^k, the same for the whole call, joins a_r and b_r and leaves
// again with `scale`, so that the largest factor lies in [2^13, 2^14): 2^15, the most an entry can
// reach, stays below fp16's 65504, and softmax values of 1e-8 keep all their bits in the rows of the
// largest factor. In a row whose factor is 2^-j of that, values below 2^(j - 27) are fp16's
// subnormals, each off by up to 2^-38 of the largest factor; that is below what fp16 can return of
// such a gradient unless the largest weight is far above 1. bf16 takes the same path; there the
// power of two changes no bit.
//
// Why d is rounded to the operands' 16-bit type: it is the operand of two tensor-core products
// whose other operand has that type (one MMA never mixes types). Each rounding is off by at most
// half a step (2^-8 relative in bf16, 2^-11 in fp16), independently from entry to entry; the sums
// over the vocabulary and over the rows are fp32, and the gradients leave in that type anyway. The
// error of an entry that is most of its row's d does not average out in that row of dH. The target's
// is one in every row, and is mended in fp32 (xent_finish_kernel). A wrong entry that a row is sure
// of is another, and is not: such rows of dH are off by 1.10 to 1.15 times what rounding them alone
// gives (256 rows sure of a wrong entry by 0.58 to 0.86, bf16; 1.5 times at worst), and the rows of
// dW that are no row's target by 1.13 times (512 rows, 8192 entries). dbias, no operand's product,
// is summed from d in fp32.
//
// Four products of 2 rows V H operations each: the logits for the loss, the logits again for the
// gradient (they are not kept), and the two gradients. The vocabulary is taken in pieces: the
// d of a piece ([rows, Vc], at most about 128 MB, two buffers) is written by the product that
// makes it and read by the two that follow. Each launch takes the tiles of three products, the
// two gradient products of piece c and the logits of piece c + 1, so the device drains once a
// piece and not three times.
//
// All products are one kernel, xent_gemm_kernel: C[M, N] = A[M, K] B[N, K]^T, operands by TMA in
// boxes of 128-byte-swizzled rows, fp32 accumulators in TMEM (two, so that the epilogue of a tile
// runs under the MMAs of the next). An operand whose K runs along its rows in memory is a K-major
// tile of 8-row atoms; one whose K runs down the columns (h and d in dW = d^T h, W in dH = d W) is
// read as an MN-major tile, 64 entries of M or N by 8 of K an atom. So nothing is ever transposed in
// memory. A TMEM lane holds a row of the tile: a thread has 128 logits of one row in turn, and the
// softmax statistics need no exchange between lanes.
//
// Rows whose target is ignored are taken out first (xent_pack_kernel): the rows that count are
// copied side by side, and every product runs over those alone. Masked rows cost no tensor time,
// and what they hold (NaN of padding) never meets a product. The number of rows that count is known
// on the device only; the tile walk reads it there.
//
// Roles: warp 0 TMA, warp 1 MMA, warps 2-9 epilogue (and 10-17, where each accumulator has its own),
// the last warp tile scheduler (cluster launch control, in launch order). Results are the same on
// every run: no split's order varies, an element of dH is added to once a launch, and the only
// atomics are minima of row numbers.
#pragma once

#include "lmhead_bf16.cuh"

namespace lmh {

constexpr int kXN = 256;                  // accumulator columns (MMA N)
constexpr int kXBlock = 64 * 64 * 2;      // bytes of 64 K rows of 64 entries of M or N
constexpr int kXEpiWarps = 8;             // epilogue warps of an accumulator
constexpr int kXInfoSlots = 2;            // tile slots of the scheduler warp
constexpr int kXAskAhead = 12;            // K steps before a tile's end at which the next is taken
constexpr int kXStoreBox = 32 * 32 * 2;   // an epilogue warp's store box: 32 rows of 32 elements
constexpr int kXMaxProblems = 3;
constexpr int kXChunk = 128;              // vocab entries per (max, sum) pair of a row
constexpr uint32_t kXTmemCols = 2 * kXN;
constexpr int32_t kXNoRow = 0x7fffffff;

// The shapes of a tile: 128 x 256 on a lone CTA, 256 x 256 on a CTA pair, and the big ones. A big
// tile is two accumulators of 256 x 256 on a CTA pair, side by side
// along N where the product is `wide` (256 x 512) and along M elsewhere (512 x 256): a K step then
// brings 48 KB into a CTA's shared memory for 1024 clocks of MMAs, and not 32 KB for 512. Under the
// power cap the loads are what the tensor time is lost to: the weight product ran at 1190 TFLOP/s
// with its loads and at 1750 with none (its MMAs on whatever lay there).
enum : int { kXLone = 0, kXPair = 1, kXBig = 2 };

template <int kShape>
struct XentTile {
  static constexpr bool kPair = kShape != kXLone;
  static constexpr bool kBig = kShape == kXBig;
  static constexpr int kM = kPair ? 256 : 128;                // MMA rows
  static constexpr int kRows = 128;                           // A rows in one CTA, per accumulator
  static constexpr int kBRows = kPair ? kXN / 2 : kXN;        // B rows in one CTA, per accumulator
  static constexpr int kABytes = kRows * 64 * 2;
  static constexpr int kBBytes = kBRows * 64 * 2;
  static constexpr int kStageBytes = kABytes + kBBytes + (kBig ? kABytes : 0);  // (A and B alike)
  static constexpr int kStages = kShape == kXPair ? 6 : 4;    // 192 KB each way
  // A big tile's accumulators have 8 epilogue warps each: TMEM is full, so the tensor pipe waits
  // for whichever is read out last (with 8 warps for both in turn, the logits of 4096 x 1024 x
  // 50304 took 371 us and not 356). So have those of lone CTAs, whose tiles of few K steps are bound
  // by the epilogue: the loads and stores of two tiles overlap (the weight gradient of 96 x 2048 x
  // 151936: 324 us with 8 warps in all, 304 so). Pairs have 8 for the tiles in turn: 16
  // cost the loss of 4096 x 2048 x 151936 0 to 1.5 % and won 0 to 2 % for gradients of 300 to 1000 rows.
  static constexpr bool kOwnWarps = kShape != kXPair;
  static constexpr int kEpiWarps = kOwnWarps ? 2 * kXEpiWarps : kXEpiWarps;
  static constexpr int kThreads = 64 + 32 * kEpiWarps + 32;
  static constexpr size_t kSmem =
      1024 + (size_t)kStages * kStageBytes + kEpiWarps * kXStoreBox + 512;
  // tile height and width of a product
  __host__ __device__ static constexpr int rows(int wide) { return kBig && !wide ? 2 * kM : kM; }
  __host__ __device__ static constexpr int cols(int wide) { return kBig && wide ? 2 * kXN : kXN; }
};

enum : int32_t {
  kXentStats = 0,    // (max, sum) per row and 128 vocab entries, the target left out
  kXentDlogits = 1,  // d, 16 bits, [rows, ld] of one vocab piece
  kXentDweight = 2,  // dW rows, 16 bits, optionally added to what is there
  kXentDhidden = 3,  // fp32 partial sums of dH, one buffer per split of K
};

// Tensor maps of one launch, those of loads with 128-byte swizzle. A K-major operand is a 2-D matrix
// in boxes of 64 columns by all rows of a CTA's tile (128 of A, kBRows of B). An MN-major one comes as
// a 3-D view [columns / 64][rows][64], a box being 64 rows of every 64-column block of the CTA's
// tile. One box a stage and operand either way: with 64 x 64 boxes, two to four of them, the same
// loads fed the tensor cores at 1150 TFLOP/s and not at 1325 (4096 x 4096 x 128256 logits under
// the power cap). The view of hidden and W has the whole blocks of H only; a tile at the edge of H
// takes its columns as 64 x 64 boxes of the 2-D matrix, as many as it needs.
enum : int32_t {
  kMapHidden = 0,    // [rows, H], K-major
  kMapHiddenMn = 1,  // [rows, H], MN-major
  kMapW = 2,         // [V, H], K-major
  kMapWMn = 3,       // [V, H], MN-major
  kMapD = 4,         // the two d buffers [rows_pad, piece], K-major
  kMapDMn = 6,       // the same, MN-major
  kMapDStore = 8,    // the same in boxes of 32 rows of 32 columns, 64-byte swizzle (stores)
  kMapDw = 10,       // dW [V, H] in the same boxes (stores)
  kMapDh = 11,       // the fp32 sums of dH [splits * rows_pad, H], boxes of 32 rows of 16 columns
  kMapHiddenEdge = 12,  // hidden and W in boxes of 64 x 64
  kMapWEdge = 13,
  kMapCount = 14,
};
struct XentMaps {
  CUtensorMap m[kMapCount];
};

struct XentProblem {
  int32_t kind;
  int32_t a_map, b_map, out_map;
  int32_t b_edge;         // an MN-major B's map for tiles at the edge of H
  int32_t a_mn, b_mn;     // 1: the operand is MN-major (its K runs down the rows of its matrix)
  int32_t m_rows;         // 1: M is the number of rows that count (else m_len)
  int32_t k_rows;         // 1: K is the number of rows that count (else k_len)
  int32_t m_len, n_len, k_len;
  int32_t b_off;          // first row of B's matrix (a piece of W starts at vocab entry b_off)
  int32_t b_k;            // 1: b_off is along K (dH: the piece's rows of W are B's K)
  int32_t splits;         // of K
  int32_t group;          // M tiles walked together
  int32_t wide;           // big tiles: 256 x 512 (else 512 x 256)
  int32_t out_off;        // first output row (dW: the piece's first vocab entry)
  int32_t add;            // dW: add to what is there; dH: add to the partial sums
};

struct XentParams {
  int32_t n_problems;
  XentProblem prob[kXMaxProblems];
  int32_t rows;               // rows of hidden (the number that count when n_rows is null)
  const int32_t* n_rows;      // device: how many rows count, or null
  int32_t H;
  int32_t rows_pad;           // rows of one split's sums of dH
  int32_t a_rows;             // rows of a K-major A box (fewer than a CTA's 128: few rows in all)
  float alpha;
  const uint16_t* bias;       // [V] or null
  const int32_t* targets;     // [rows that count]
  float2* partials;           // stats: [2 * ceil(V / 256)][rows]
  const float4* row_info;     // dlogits: (lse * log2(e), a, d at the target, target as int bits)
  const float* scale;         // device: [1] = the factor of the gradients
  float* bias_part;           // dlogits: [rows_pad / 32][piece] column sums of d in fp32, or null
  int32_t piece;              // entries of a full piece (the pitch of bias_part)
  int32_t* first;             // [V]: the first row whose target is this entry (kXNoRow: none)
  float* side;                // [rows that count][H]: dW's row of that target before its rounding
  uint16_t* d_weight;         // dW as memory, for add
  WaitCfg wait;
};

// ------------------------------------------------------------------ small wrappers

__device__ __forceinline__ void tmem_ld_32x32b_x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// The TMEM loads issued so far have arrived; `r`, the last of them, is used behind this only.
__device__ __forceinline__ void tmem_ld_wait_x32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// Pairs of fp32 values in one instruction (each half rounds as the scalar instruction does).
__device__ __forceinline__ uint64_t pair_f32(float lo, float hi) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
  return p;
}
__device__ __forceinline__ void unpair_f32(uint64_t p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A word of another CTA's shared memory in the cluster, at the address of `p` in this one's.
__device__ __forceinline__ int32_t cluster_load(const void* p, uint32_t rank) {
  uint32_t remote;
  int32_t v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}
__device__ __forceinline__ float cluster_load_f32(const float* p, uint32_t rank) {
  return __int_as_float(cluster_load(p, rank));
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// One K step of 64 (four K = 16 MMAs, M rows across the pair for a pair) from a converged warp, one
// elected lane issuing; the operands advance by their own steps, in 16-byte units. Only the first
// MMA may start a fresh accumulator.
template <bool kPair>
__device__ __forceinline__ void mma4_f16_steps_elect(uint32_t d_tmem, uint64_t a, uint64_t b,
                                                     uint64_t a_step, uint64_t b_step,
                                                     uint32_t idesc, uint32_t accumulate) {
  if constexpr (kPair) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "add.s64 a1, %1, %5;\n\tadd.s64 a2, a1, %5;\n\tadd.s64 a3, a2, %5;\n\t"
        "add.s64 b1, %2, %6;\n\tadd.s64 b2, b1, %6;\n\tadd.s64 b3, b2, %6;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a1, b1, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a2, b2, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "l"(a_step), "l"(b_step)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "add.s64 a1, %1, %5;\n\tadd.s64 a2, a1, %5;\n\tadd.s64 a3, a2, %5;\n\t"
        "add.s64 b1, %2, %6;\n\tadd.s64 b2, b1, %6;\n\tadd.s64 b3, b2, %6;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "l"(a_step), "l"(b_step)
        : "memory");
  }
}

// Shared-memory descriptor of an MN-major tile in 64 x 64 blocks: each block is 64 K rows of 128
// bytes (64 entries of M or N, 128-byte swizzle), 8 K rows make an atom of 1024 bytes (the stride
// offset), the next 64 entries of M or N are the next block (the leading offset).
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw128(uint32_t smem_addr) {
  const uint64_t start = (smem_addr & 0x3FFFFu) >> 4;
  const uint64_t lbo = (uint32_t)kXBlock >> 4;
  const uint64_t sbo = 1024u >> 4;
  return start | (lbo << 16) | (sbo << 32) | (1ull << 46) | (2ull << 61);
}

// As tma_load_2d_pair, from a 3-D view.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map,
                                                 uint32_t bar, int32_t x, int32_t y, int32_t z,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(pair_leader_addr(bar)), "r"(x), "r"(y), "r"(z),
      "l"(policy)
      : "memory");
}

template <bool kPair>
__device__ __forceinline__ void xent_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                             int32_t col, int32_t row, uint64_t policy) {
  if constexpr (kPair)
    tma_load_2d_pair(dst, map, bar, tma_x((int64_t)col * 2, 2), row, policy);
  else
    tma_load_2d(dst, map, bar, tma_x((int64_t)col * 2, 2), row, policy);
}
// `col` is a multiple of 64: the block is its own coordinate.
template <bool kPair>
__device__ __forceinline__ void xent_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                             int32_t col, int32_t row, uint64_t policy) {
  if constexpr (kPair)
    tma_load_3d_pair(dst, map, bar, 0, row, col / 64, policy);
  else
    tma_load_3d(dst, map, bar, 0, row, col / 64, policy);
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int32_t x,
                                             int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y)
               : "memory");
}
// The same, added in fp32 to what is there.
__device__ __forceinline__ void tma_add_2d_f32(const CUtensorMap* map, uint32_t src, int32_t x,
                                               int32_t y) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], "
      "[%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// The shared memory of this thread's bulk stores has been read.
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

template <bool kF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (kF16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <bool kF16>
__device__ __forceinline__ float unpack16(uint32_t bits16) {
  if constexpr (kF16) return __half2float(__ushort_as_half((unsigned short)bits16));
  return __uint_as_float(bits16 << 16);
}

// ------------------------------------------------------------------ the tile walk

struct XentTileAt {
  int32_t prob;           // -1: no tile (the walk's tail when rows were taken out)
  int32_t m0, n0;         // first row and column of the tile
  int32_t k0, k_steps;    // first 64-wide K step and their number (may be 0)
  int32_t split;
};

__device__ __forceinline__ int32_t ceil_div(int32_t a, int32_t b) { return (a + b - 1) / b; }

// Half the columns of a tile, a multiple of 64 (lone: 32): what either CTA of a pair loads of B, and
// what either half of the epilogue's warps takes. All of them but at the edge of H, where the tile
// is as narrow as what is left, since its MMAs cost by the column (both gradients of 700 x 1032 x
// 32771, with 8 columns in a row's fifth tile: 202 us, with whole tiles 207; 1000 x 896 x 65536: 350
// and 357). Vocab entries are many, and their last tile stays whole.
template <int kShape>
__device__ __forceinline__ int32_t xent_share(const XentProblem& q, int32_t n0) {
  using T = XentTile<kShape>;
  const int32_t all = T::cols(q.wide) / 2, unit = T::kPair ? 64 : 32;
  if (q.kind < kXentDweight) return all;
  return min(all, ceil_div(q.n_len - n0, 2 * unit) * unit);
}
// The part of it that is accumulator h's. (A big wide tile's accumulators share its columns.)
template <int kShape>
__device__ __forceinline__ int32_t xent_share_of(const XentProblem& q, int32_t share, int h) {
  return XentTile<kShape>::kBig && q.wide ? min(max(share - h * kXChunk, 0), kXChunk) : share;
}

// The launch's tiles: the problems one after another, each split by split, M tiles in groups of the
// problem's own number, N-major within a group. What does not depend on the tile is worked out once:
// a tile's coordinates cost three 32-bit divisions.
template <int kShape>
struct XentWalk {
  int32_t mt[kXMaxProblems], nt[kXMaxProblems], ks[kXMaxProblems];

  __device__ __forceinline__ XentWalk(const XentParams& p, int32_t n_rows) {
#pragma unroll
    for (int i = 0; i < kXMaxProblems; ++i) {
      const XentProblem& q = p.prob[i];
      const bool used = i < p.n_problems;
      mt[i] = used ? ceil_div(q.m_rows ? n_rows : q.m_len, XentTile<kShape>::rows(q.wide)) : 0;
      nt[i] = used ? ceil_div(q.n_len, XentTile<kShape>::cols(q.wide)) : 0;
      ks[i] = used ? ceil_div(q.k_rows ? n_rows : q.k_len, kBK) : 0;
    }
  }

  __device__ __forceinline__ XentTileAt at(const XentParams& p, int32_t t) const {
    XentTileAt c;
    c.prob = -1;
    c.m0 = c.n0 = c.k0 = c.k_steps = c.split = 0;
#pragma unroll
    for (int i = 0; i < kXMaxProblems; ++i) {
      const uint32_t per = (uint32_t)(mt[i] * nt[i]);
      const int32_t splits = p.prob[i].splits;
      if (c.prob < 0 && t >= 0) {
        if (t < (int32_t)per * splits) {
          const uint32_t split = splits == 1 ? 0u : (uint32_t)t / per;
          const uint32_t u = (uint32_t)t - split * per;
          const int32_t group = p.prob[i].group, wide = p.prob[i].wide;
          const uint32_t group_tiles = (uint32_t)(group * nt[i]);
          const uint32_t g = u / group_tiles;
          const uint32_t local = u - g * group_tiles;
          const uint32_t gm = (uint32_t)min(group, mt[i] - (int32_t)g * group);
          const uint32_t n = local / gm;
          c.prob = i;
          c.m0 = ((int32_t)g * group + (int32_t)(local - n * gm)) * XentTile<kShape>::rows(wide);
          c.n0 = (int32_t)n * XentTile<kShape>::cols(wide);
          c.split = (int32_t)split;
          // (at most 2^24 steps by 32 splits)
          c.k0 = splits == 1 ? 0 : (int32_t)((uint32_t)ks[i] * split / (uint32_t)splits);
          c.k_steps = (splits == 1 ? ks[i]
                                   : (int32_t)((uint32_t)ks[i] * (split + 1) / (uint32_t)splits)) -
                      c.k0;
        }
        t -= (int32_t)per * splits;
      }
    }
    return c;
  }
};

// The tiles of a CTA as its scheduler warp announces them to the other roles. That warp asks for
// tiles by cluster launch control, takes the answers and works out the coordinates: done by the MMA
// warp itself, between two tiles, this took 1000 clocks a tile in which nothing was issued. It asks
// when the producer says that it nears the end of its tile and no sooner: a unit that holds tiles
// it has not begun leaves other units idle at the launch's end.
struct XentInfo {
  uint32_t slot0, full0, empty0, want;
};

__device__ __forceinline__ bool xent_announce(const XentInfo& f, int j, const XentTileAt& c,
                                              bool last, const WaitCfg& w,
                                              volatile int* abort_flag) {
  const int k = j % kXInfoSlots;
  if (!wait_bounded(f.empty0 + 8 * k, ((uint32_t)(j / kXInfoSlots) & 1u) ^ 1u, w, abort_flag,
                    kSleepHintNs))
    return false;
  if ((threadIdx.x & 31) == 0) {
    st_shared_v4(f.slot0 + 32 * k, last ? 0xfffffffeu : (uint32_t)c.prob, (uint32_t)c.m0,
                 (uint32_t)c.n0, (uint32_t)c.k0);
    st_shared_v4(f.slot0 + 32 * k + 16, (uint32_t)c.k_steps, (uint32_t)c.split, 0u, 0u);
    mbar_arrive(f.full0 + 8 * k);
  }
  __syncwarp();
  return true;
}

// Tile j, by a whole warp. prob is -1 where there is nothing to do and -2 behind the last tile.
__device__ __forceinline__ bool xent_read(const XentInfo& f, int j, XentTileAt& c,
                                          const WaitCfg& w, volatile int* abort_flag,
                                          uint32_t sleep_ns = 0) {
  const int k = j % kXInfoSlots;
  if (!wait_bounded(f.full0 + 8 * k, (uint32_t)(j / kXInfoSlots) & 1u, w, abort_flag, sleep_ns))
    return false;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(c.prob), "=r"(c.m0), "=r"(c.n0), "=r"(c.k0)
               : "r"(f.slot0 + 32 * k)
               : "memory");
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
               : "=r"(c.k_steps), "=r"(c.split)
               : "r"(f.slot0 + 32 * k + 16)
               : "memory");
  // the same in every lane, and the compiler may know it
  c.prob = __shfl_sync(0xffffffffu, c.prob, 0);
  c.k_steps = __shfl_sync(0xffffffffu, c.k_steps, 0);
  __syncwarp();  // every lane has read the slot
  if ((threadIdx.x & 31) == 0) mbar_arrive(f.empty0 + 8 * k);
  __syncwarp();
  return true;
}

// ------------------------------------------------------------------ epilogues
// Each is called by one warp with its 32 rows of the tile (row = its lane's) and its 128 columns
// from `col`; `tacc` addresses the first of them in TMEM; `zero` says that K was empty and the
// accumulator was never written. Columns come 32 at a time. The two softmax epilogues work in units
// of log 2 (z * log2(e), one multiply for alpha and the change of base) on pairs of values: at
// 1024-wide hidden rows a tile's MMAs take about 8000 clocks and 128 x 256 exponentials 2000 of the
// SM's special-function unit, but one instruction at a time (some 18 an entry) the epilogue took
// 15000 and held the tensor pipe up.

__device__ __forceinline__ void xent_acc_load(uint32_t tacc, bool zero, uint32_t (&r)[32]) {
  __syncwarp();  // the lanes may come from rows of their own; the TMEM load is the warp's
  if (zero) {
#pragma unroll
    for (int j = 0; j < 32; ++j) r[j] = 0u;
  } else {
    tmem_ld_32x32b_x32(tacc, r);
  }
}

// Calls step(c, r) for the column groups c = 0, 32, 64, 96 that begin before `cols`. (One group at a
// time: the two warps that share a scheduler cover each other's TMEM loads, and a second buffer of
// 32 registers spilled.)
template <typename Step>
__device__ __forceinline__ void xent_columns(uint32_t tacc, bool zero, int32_t cols, Step step) {
#pragma unroll 1
  for (int c = 0; c < kXChunk && c < cols; c += 32) {
    uint32_t r[32];
    xent_acc_load(tacc + (uint32_t)c, zero, r);
    tmem_ld_wait_x32(r);
    step(c, r);
  }
}

// Lane's own column of 32: the bias of vocab entry v0 + lane (0 past the end), times `factor`.
template <bool kF16>
__device__ __forceinline__ float xent_bias(const XentParams& p, int32_t v0, int32_t v_end,
                                           float factor) {
  const int32_t v = v0 + (int)(threadIdx.x & 31);
  return v < v_end ? unpack16<kF16>(p.bias[v]) * factor : 0.0f;
}

// x[j] = acc[j] * factor + shift (+ bias * factor), in pairs.
template <bool kF16>
__device__ __forceinline__ void xent_scaled(const XentParams& p, uint32_t (&r)[32], float factor,
                                            float shift, int32_t v0, int32_t v_end) {
  const uint64_t f2 = pair_f32(factor, factor), s2 = pair_f32(shift, shift);
  if (p.bias == nullptr) {
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      float lo, hi;
      unpair_f32(fma2(pair_f32(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), f2, s2), lo, hi);
      r[j] = __float_as_uint(lo);
      r[j + 1] = __float_as_uint(hi);
    }
  } else {
    const float b = xent_bias<kF16>(p, v0, v_end, factor);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const uint64_t b2 = pair_f32(__shfl_sync(0xffffffffu, b, j), __shfl_sync(0xffffffffu, b, j + 1));
      float lo, hi;
      unpair_f32(fma2(pair_f32(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), f2, add2(b2, s2)),
                 lo, hi);
      r[j] = __float_as_uint(lo);
      r[j + 1] = __float_as_uint(hi);
    }
  }
}

// (max, sum of 2^(x - max)) of this thread's row over its 128 vocab entries, x = z * log2(e), the
// target left out: its logit is taken exactly later (see xent_target_logit). Per 32 entries: their
// maximum first, one rescaling of the running sum, then the terms. Entries past V and the target
// count as -inf; -inf alone gives (-inf, 0). A NaN logit reaches the sum through its own term;
// +inf gives inf - inf there, NaN as well.
template <bool kF16>
__device__ __forceinline__ void xent_epi_stats(const XentParams& p, const XentProblem& q,
                                               uint32_t tacc, bool zero, int32_t row, bool row_ok,
                                               int32_t t, int32_t col) {
  const int32_t V = q.n_len;
  float m = -INFINITY, s = 0.0f;
  xent_columns(tacc, zero, V - col, [&](int c, uint32_t(&r)[32]) {
    const int32_t v0 = col + c;
    xent_scaled<kF16>(p, r, p.alpha * kLog2e, 0.0f, v0, V);
    if (v0 + 32 > V || __any_sync(0xffffffffu, t >= v0 && t < v0 + 32)) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (v0 + j >= V || v0 + j == t) r[j] = __float_as_uint(-INFINITY);
    }
    float nm = m, m1 = -INFINITY;
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      nm = max3(nm, __uint_as_float(r[j]), __uint_as_float(r[j + 1]));
      m1 = max3(m1, __uint_as_float(r[j + 2]), __uint_as_float(r[j + 3]));
    }
    nm = fmaxf(nm, m1);
    const float ref = nm == -INFINITY ? 0.0f : nm;
    const uint64_t neg = pair_f32(-ref, -ref);
    uint64_t s0 = pair_f32(0.0f, 0.0f), s1 = s0;
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      float a0, a1, b0, b1;
      unpair_f32(add2(pair_f32(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), neg), a0, a1);
      unpair_f32(add2(pair_f32(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3])), neg), b0, b1);
      s0 = add2(s0, pair_f32(exp2_approx(a0), exp2_approx(a1)));
      s1 = add2(s1, pair_f32(exp2_approx(b0), exp2_approx(b1)));
    }
    float lo, hi;
    unpair_f32(add2(s0, s1), lo, hi);
    s = s * exp2_approx(m - ref) + (lo + hi);
    m = nm;
  });
  if (row_ok && col < V)
    __stcs(p.partials + (int64_t)(col / kXChunk) * p.rows + row, make_float2(m, s));
}

// The 32 columns of one store box, as 16-bit values in this warp's staging buffer: 32 rows of 64
// bytes, with TMA's 64-byte swizzle (the 16-byte pieces of a row are permuted by its row pair).
struct XentStage {
  uint32_t buf;  // 1024-byte aligned
  __device__ __forceinline__ void put(const uint32_t (&w)[16]) const {
    const uint32_t row = threadIdx.x & 31;
    if (row == 0) bulk_wait_read();
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j)
      st_shared_v4(buf + row * 64u + (((uint32_t)j ^ ((row >> 1) & 3u)) << 4), w[4 * j],
                   w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  }
  __device__ __forceinline__ void store(const CUtensorMap* map, int32_t x, int32_t y) const {
    fence_async_smem();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      tma_store_2d(map, buf, tma_x((int64_t)x * 2, 2), y);
      bulk_commit();
    }
  }
};

template <bool kF16>
__device__ __forceinline__ void xent_pack32(const uint32_t (&r)[32], uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j)
    w[j] = pack16<kF16>(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
}

// The sums of 32 columns over the warp's 32 rows, a lane holding its row: lane c gets column c's.
// Each step halves the columns that a lane holds and adds the other lane's half, so a column is a
// tree of the rows, always the same one. `r` is used up.
__device__ __forceinline__ float xent_column_sums(uint32_t (&r)[32]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool upper = (threadIdx.x & o) != 0;
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const float a = __uint_as_float(r[j]), b = __uint_as_float(r[j + o]);
      const float other = __shfl_xor_sync(0xffffffffu, upper ? a : b, o);
      r[j] = __float_as_uint((upper ? b : a) + other);
    }
  }
  return __uint_as_float(r[0]);
}

// d of this thread's row over its 128 vocab entries of the piece, 16 bits, into the piece's buffer.
// Rows that do not count and entries past V are written as 0: the products that read d take whole
// 64-wide steps. (Rows behind the last such step are not written.) The target's entry comes ready
// with the row's factors.
template <bool kF16>
__device__ __forceinline__ void xent_epi_dlogits(const XentParams& p, const XentProblem& q,
                                                 const XentMaps& maps, const XentStage& st,
                                                 uint32_t tacc, bool zero, int32_t row0,
                                                 int32_t row, int32_t n_rows, const float4& info,
                                                 int32_t col) {
  const bool row_ok = row < n_rows;
  if (row0 >= (n_rows + kBK - 1) / kBK * kBK) return;  // the whole warp
  const int lane = threadIdx.x & 31;
  const int32_t V = q.b_off + q.n_len;  // the end of the piece as vocab ids
  const int32_t t = __float_as_int(info.w);
  const uint64_t a2 = pair_f32(info.y, info.y);
  const bool all_ok = __all_sync(0xffffffffu, row_ok);
  // (whole boxes of 64 columns: what lies past the piece's end is 0)
  const int32_t cols = min(kXChunk, (q.n_len - col + 63) / 64 * 64);
  xent_columns(tacc, zero, cols, [&](int c, uint32_t(&r)[32]) {
    const int32_t v0 = q.b_off + col + c;
    xent_scaled<kF16>(p, r, p.alpha * kLog2e, -info.x, v0, V);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      float lo, hi;
      unpair_f32(mul2(pair_f32(exp2_approx(__uint_as_float(r[j])),
                               exp2_approx(__uint_as_float(r[j + 1]))), a2), lo, hi);
      r[j] = __float_as_uint(lo);
      r[j + 1] = __float_as_uint(hi);
    }
    if (__any_sync(0xffffffffu, t >= v0 && t < v0 + 32)) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (v0 + j == t) r[j] = __float_as_uint(info.z);
      // (a minimum does not depend on the order)
      if (t >= v0 && t < v0 + 32 && t < V) atomicMin(p.first + t, row);
    }
    if (!all_ok || v0 + 32 > V) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (!row_ok || v0 + j >= V) r[j] = 0u;
    }
    uint32_t w[16];
    xent_pack32<kF16>(r, w);
    st.put(w);
    st.store(&maps.m[q.out_map], col + c, row0);
    if (p.bias_part != nullptr)  // of d in fp32: dbias needs no operand of a product
      p.bias_part[(int64_t)(row0 / 32) * p.piece + col + c + lane] = xent_column_sums(r);
  });
}

// dW of this thread's vocab entry: the sum times `scale`, added in fp32 to what is there if asked
// for, rounded once. A row that is some row's target also goes to that row's place in `side`
// as it is, for xent_finish_kernel to round again with what d lost at the target.
template <bool kF16>
__device__ __forceinline__ void xent_epi_dweight(const XentParams& p, const XentProblem& q,
                                                 const XentMaps& maps, const XentStage& st,
                                                 uint32_t tacc, bool zero, int32_t first,
                                                 int32_t row0, int32_t row, int32_t col,
                                                 int32_t cols) {
  const float scale = zero ? 0.0f : p.scale[1];  // (no row counts: 0, whatever the scale is)
  const bool add_row = q.add && row < q.m_len;
  const int64_t at = (int64_t)(q.out_off + row) * p.H;
  xent_columns(tacc, zero, min(cols, p.H - col), [&](int c, uint32_t(&r)[32]) {
    const int32_t x = col + c;
#pragma unroll
    for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * scale);
    if (add_row) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (x + 8 * j < p.H) {  // H is a multiple of 8
          const uint4 old = *reinterpret_cast<const uint4*>(p.d_weight + at + x + 8 * j);
          const uint32_t o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = 8 * j + 2 * i;
            r[e] = __float_as_uint(__uint_as_float(r[e]) + unpack16<kF16>(o[i] & 0xffffu));
            r[e + 1] = __float_as_uint(__uint_as_float(r[e + 1]) + unpack16<kF16>(o[i] >> 16));
          }
        }
      }
    }
    if (first != kXNoRow) {
      uint4* side = reinterpret_cast<uint4*>(p.side + (int64_t)first * p.H + x);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (x + 4 * j < p.H)
          __stcs(side + j, make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]));
    }
    uint32_t w[16];
    xent_pack32<kF16>(r, w);
    st.put(w);
    // a box that starts past the piece's rows belongs to the next piece or to nothing
    if (row0 < q.m_len) st.store(&maps.m[q.out_map], x, q.out_off + row0);
  });
}

// fp32 sums of dH over this piece's (and split's) vocab entries, added to the earlier pieces' by
// TMA: one addition an element and piece, in the order of the launches. (Read, added and written
// by the threads, 16 bytes a lane of 32 rows at a time, a tile's epilogue took 80000 clocks, more
// than the MMAs of 1024-wide pieces.) Rows that do not count are written too, and never read.
__device__ __forceinline__ void xent_epi_dhidden(const XentParams& p, const XentProblem& q,
                                                 const XentMaps& maps, const XentStage& st,
                                                 uint32_t tacc, bool zero, int32_t split,
                                                 int32_t row0, int32_t n_rows, int32_t col,
                                                 int32_t cols) {
  if (row0 >= n_rows) return;  // the whole warp
  const CUtensorMap* map = &maps.m[kMapDh];
  const int32_t y = split * p.rows_pad + row0;
  xent_columns(tacc, zero, min(cols, p.H - col), [&](int c, uint32_t(&r)[32]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (col + c + 16 * k >= p.H) break;
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j] = r[16 * k + j];
      st.put(w);
      fence_async_smem();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) {
        if (q.add)
          tma_add_2d_f32(map, st.buf, col + c + 16 * k, y);
        else
          tma_store_2d(map, st.buf, col + c + 16 * k, y);
        bulk_commit();
      }
    }
  });
}

// ------------------------------------------------------------------ the kernel

template <int kShape, bool kF16>
__global__ void __launch_bounds__(XentTile<kShape>::kThreads, 1)
    xent_gemm_kernel(const __grid_constant__ XentMaps maps, const __grid_constant__ XentParams p) {
  using T = XentTile<kShape>;
  constexpr bool kPair = T::kPair, kBig = T::kBig;
  extern __shared__ uint8_t smem_raw[];
  if (threadIdx.x == 0) pdl_trigger();
  uint8_t* smem = align_up_1024(smem_raw);
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  constexpr int S = T::kStages;
  const uint32_t rank = kPair ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;

  uint8_t* staging = smem + (size_t)S * T::kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + T::kEpiWarps * kXStoreBox);
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = smem_u32(bars + S);
  const uint32_t tfull0 = smem_u32(bars + 2 * S);
  const uint32_t tempty0 = smem_u32(bars + 2 * S + 2);
  const uint32_t done_bar = smem_u32(bars + 2 * S + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // (2 * S is even, so the 16-byte answer and tile slots are aligned)
  const ClcRing clc{smem_u32(bars + 2 * S + 6), smem_u32(bars + 2 * S + 14),
                    smem_u32(bars + 2 * S + 18)};
  const XentInfo info_ring{smem_u32(bars + 2 * S + 22), smem_u32(bars + 2 * S + 30),
                           smem_u32(bars + 2 * S + 32), smem_u32(bars + 2 * S + 34)};

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int k = 0; k < kClcSlots; ++k) {
      mbar_init(clc.full0 + 8 * k, 1);
      mbar_init(clc.empty0 + 8 * k, kPair ? 2 : 1);  // read by the scheduler warps
    }
    for (int k = 0; k < kXInfoSlots; ++k) {
      mbar_init(info_ring.full0 + 8 * k, 1);
      // read by the producer, the epilogue warps and, in a pair's leader alone, the MMA warp
      mbar_init(info_ring.empty0 + 8 * k, 1 + T::kEpiWarps + (leader ? 1 : 0));
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull0 + 8 * a, 1);
      mbar_init(tempty0 + 8 * a, (kPair ? 2 : 1) * 32 * kXEpiWarps);
    }
    mbar_init(info_ring.want, 1);
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(smem_u32(tmem_slot), kXTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), kXTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before_sync();
  if constexpr (kPair) {
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  tc_fence_after_sync();
  pdl_wait();
  const uint32_t tmem_base = *tmem_slot;
  const int32_t n_rows = p.n_rows != nullptr ? *p.n_rows : p.rows;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    const uint64_t pol = l2_policy_evict_normal();
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;
    bool ok = true;
    for (int j = 0; ok; ++j) {
      XentTileAt tc;
      if (!xent_read(info_ring, j, tc, p.wait, abort_flag)) {
        fail(kRoleProducer, abort_flag);
        break;
      }
      if (tc.prob == -2) break;
      const int32_t ask_at = tc.prob < 0 ? 0 : max(0, tc.k_steps - kXAskAhead);
      if (tc.prob < 0 || tc.k_steps == 0) {
        if (lane == 0) mbar_arrive(info_ring.want);
        __syncwarp();
        continue;
      }
      const XentProblem& q = p.prob[tc.prob];
      const CUtensorMap* ma = &maps.m[q.a_map];
      const bool edge = q.b_mn && tc.n0 + T::cols(q.wide) > q.n_len;
      const CUtensorMap* mb = &maps.m[edge ? q.b_edge : q.b_map];
      // this CTA's part of the tile: its half of the rows of A and of B in a pair
      const int32_t m0 = tc.m0 + (kPair ? (int32_t)rank * (T::rows(q.wide) / 2) : 0);
      const int32_t share = xent_share<kShape>(q, tc.n0);
      const int32_t n0 = tc.n0 + (kPair ? (int32_t)rank * share : 0) + (q.b_k ? 0 : q.b_off);
      const uint32_t a_bytes = (kBig && !q.wide ? 2u : 1u) * T::kABytes;
      // A K-major A box brings a_rows rows only; what lies below them in the tile is other rows' of
      // the accumulator, and nobody reads those.
      const int b_blocks = (kPair ? share : 2 * share) / 64;
      const uint32_t tx = (kPair ? 2u : 1u) * (a_bytes + (uint32_t)(b_blocks * kXBlock)) -
                          (kPair || q.a_mn ? 0u : (uint32_t)(128 - p.a_rows) * 128u);
      for (int ks = 0; ks < tc.k_steps; ++ks) {
        if (!wait_bounded(empty0 + 8 * stage, phase ^ 1u, p.wait, abort_flag)) {
          fail(kRoleProducer, abort_flag);
          ok = false;
          break;
        }
        if (lane == 0 && ks == ask_at) mbar_arrive(info_ring.want);
        if (lane == 0 && !p.wait.starve_loads) {
          const uint32_t full = full0 + 8 * stage;
          const uint32_t sa = smem_u32(smem + (size_t)stage * T::kStageBytes);
          const uint32_t sb = sa + a_bytes;
          const int32_t k = (tc.k0 + ks) * kBK;
          const int32_t kb = k + (q.b_k ? q.b_off : 0);
          if (leader) mbar_arrive_expect_tx(full, tx);
          if (q.a_mn)
            xent_load_3d<kPair>(sa, ma, full, m0, k, pol);
          else
            xent_load_2d<kPair>(sa, ma, full, k, m0, pol);
          if (!q.b_mn) {
            xent_load_2d<kPair>(sb, mb, full, kb, n0, pol);
          } else if (!edge) {
            xent_load_3d<kPair>(sb, mb, full, n0, kb, pol);
          } else {
            for (int i = 0; i < b_blocks; ++i)
              xent_load_2d<kPair>(sb + i * kXBlock, mb, full, n0 + 64 * i, kb, pol);
          }
        }
        __syncwarp();
        ++issued;
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // Drain, as in the fp32 head: loads land (or, for a pair, the stages they filled are
    // released) before the CTA may exit.
    if (!p.wait.starve_loads) {
      const int outstanding = issued < S ? issued : S;
      for (int i = 0; i < outstanding; ++i) {
        if (--stage < 0) {
          stage = S - 1;
          phase ^= 1u;
        }
        if (!wait_bounded((kPair ? empty0 : full0) + 8 * stage, phase, p.wait, nullptr)) {
          fail(kRoleDrain, abort_flag);
          break;
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    int stage = 0;
    uint32_t phase = 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = leader;
    for (int j = 0; ok; ++j) {
      XentTileAt tc;
      if (!xent_read(info_ring, j, tc, p.wait, abort_flag)) {
        fail(kRoleMma, abort_flag);
        break;
      }
      if (tc.prob == -2) break;
      if (tc.prob < 0) continue;
      const XentProblem& q = p.prob[tc.prob];
      const int32_t share = xent_share<kShape>(q, tc.n0);
      const uint32_t layout = ((uint32_t)q.a_mn << 15) | ((uint32_t)q.b_mn << 16);
      const uint32_t idesc[2] = {
          layout | idesc_f16kind_f32(T::kM, 2 * xent_share_of<kShape>(q, share, 0), !kF16),
          layout | idesc_f16kind_f32(T::kM, 2 * xent_share_of<kShape>(q, share, 1), !kF16)};
      const bool empty = xent_share_of<kShape>(q, share, 1) == 0;  // (a big tile's second)
      // one K = 16 step further along: 32 bytes in a K-major tile, 16 rows in an MN-major one
      const uint64_t a_step = q.a_mn ? (16 * 128) >> 4 : 32 >> 4;
      const uint64_t b_step = q.b_mn ? (16 * 128) >> 4 : 32 >> 4;
      // accumulator h of the tile: of a big one both, else the one whose turn it is
      auto acquire = [&](int h) {
        if (!wait_bounded(tempty0 + 8 * h, acc_phase ^ 1u, p.wait, abort_flag)) return false;
        tc_fence_after_sync();
        return true;
      };
      auto filled = [&](int st, uint32_t ph) {
        if (!wait_bounded(full0 + 8 * st, ph, p.wait, abort_flag)) return false;
        tc_fence_after_sync();
        return true;
      };
      auto multiply = [&](int st, int h, bool more) {
        if (kBig && h == 1 && empty) return;
        const uint32_t sa = smem_u32(smem + (size_t)st * T::kStageBytes);
        const uint32_t sb = sa + (kBig && !q.wide ? 2u : 1u) * T::kABytes;
        // the second accumulator's part of the operand that a big tile has two of
        const uint32_t oa = kBig && !q.wide ? (uint32_t)h * T::kABytes : 0u;
        const uint32_t ob = kBig && q.wide ? (uint32_t)h * T::kBBytes : 0u;
        const uint64_t ad = q.a_mn ? sdesc_mnmajor_sw128(sa + oa) : sdesc_kmajor_sw128(sa + oa);
        const uint64_t bd = q.b_mn ? sdesc_mnmajor_sw128(sb + ob) : sdesc_kmajor_sw128(sb + ob);
        mma4_f16_steps_elect<kPair>(tmem_base + (uint32_t)(h * kXN), ad, bd, a_step, b_step,
                                    idesc[kBig ? h : 0], more);
      };
      auto release = [&](uint32_t bar) {
        if constexpr (kPair)
          mma_commit_pair_elect(bar, 0x3);
        else
          mma_commit_elect(bar);
        __syncwarp();
      };
      if constexpr (!kBig) {
        if (!acquire(acc)) {
          fail(kRoleMma, abort_flag);
          break;
        }
        for (int ks = 0; ks < tc.k_steps; ++ks) {
          if (!filled(stage, phase)) {
            ok = false;
            break;
          }
          multiply(stage, acc, ks != 0);
          release(empty0 + 8 * stage);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) {
          fail(kRoleMma, abort_flag);
          break;
        }
        release(tfull0 + 8 * acc);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      } else {
        // Both accumulators of a big tile fill TMEM, so the epilogue of one runs under the MMAs of
        // the other: the tile's first and last S steps go through all S stages for the first
        // accumulator, then again for the second.
        for (int ks = 0; ok && ks < tc.k_steps;) {
          const int left = tc.k_steps - ks;
          const int n = ks == 0 || left <= S ? min(S, left) : 1;
          int st = stage;
          uint32_t ph = phase;
          if (ks == 0) ok = acquire(0);
          for (int i = 0; ok && i < n; ++i) {
            ok = filled(st, ph);
            if (!ok) break;
            multiply(st, 0, ks + i != 0);
            if (++st == S) {
              st = 0;
              ph ^= 1u;
            }
          }
          if (ok && n == left) release(tfull0);
          if (ok && ks == 0) ok = acquire(1);
          for (int i = 0; ok && i < n; ++i) {
            multiply(stage, 1, ks + i != 0);
            release(empty0 + 8 * stage);
            if (++stage == S) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (ok && n == left) release(tfull0 + 8);
          ks += n;
        }
        if (ok && tc.k_steps == 0) {
          ok = acquire(0) && acquire(1);
          if (ok) {
            release(tfull0);
            release(tfull0 + 8);
          }
        }
        if (!ok) {
          fail(kRoleMma, abort_flag);
          break;
        }
        acc_phase ^= 1u;
      }
    }
    if (leader) {
      if constexpr (kPair)
        mma_commit_pair_elect(done_bar, 0x1);
      else
        mma_commit_elect(done_bar);
      __syncwarp();
      if (!wait_bounded(done_bar, 0, p.wait, nullptr)) fail(kRoleDrain, abort_flag);
    }
  } else if (warp == 2 + T::kEpiWarps) {
    // ---------------------------------------------------------------- scheduler
    const XentWalk<kShape> walk(p, n_rows);
    int tile = (int)blockIdx.x >> (kPair ? 1 : 0);
    bool ok = true;
    int asked = 0;
    for (int j = 0;; ++j) {
      if (!xent_announce(info_ring, j, walk.at(p, tile), tile < 0, p.wait, abort_flag)) {
        fail(kRoleProducer, abort_flag);
        break;
      }
      if (tile < 0) break;
      if (leader) {
        if (!wait_bounded(info_ring.want, (uint32_t)j & 1u, p.wait, abort_flag, kSleepHintNs) ||
            !clc_ask<kPair>(clc, j + 1, p.wait, abort_flag)) {
          fail(kRoleProducer, abort_flag);
          break;
        }
        asked = j + 1;
      }
      tile = clc_take<kPair>(clc, j + 1, p.wait, abort_flag, ok);
      if (!ok) {
        fail(kRoleProducer, abort_flag);
        break;
      }
    }
    // An answer asked for but not read (an error path) must still land before the CTA exits.
    if (leader && asked > 0) {
      const int slot = (asked - 1) % kClcSlots;
      const uint32_t ph = (uint32_t)((asked - 1) / kClcSlots) & 1u;
      if (!wait_bounded(clc.full0 + 8 * slot, ph, p.wait, nullptr)) fail(kRoleDrain, abort_flag);
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int quarter = warp & 3;      // TMEM lanes this warp may access
    const int own = (warp - 2) / kXEpiWarps;    // its accumulator (kOwnWarps)
    const int half = ((warp - 2) >> 2) & 1;     // which half of the accumulator's columns
    const XentStage st{smem_u32(staging + (warp - 2) * kXStoreBox)};
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int j = 0;; ++j) {
      XentTileAt tc;
      if (!xent_read(info_ring, j, tc, p.wait, abort_flag, kSleepHintNs)) {
        fail(kRoleEpilogue, abort_flag);
        break;
      }
      if (tc.prob == -2) break;
      if (tc.prob < 0) continue;
      const XentProblem& q = p.prob[tc.prob];
      // the tile's accumulator (a big tile has both), and this warp's
      const int h = kBig ? own : acc;
      const uint32_t tile_phase = acc_phase;
      if (!kBig) acc ^= 1;
      if (kBig || acc == 0) acc_phase ^= 1u;
      if (T::kOwnWarps && h != own) continue;
      // The rows and columns of its part of the accumulator. A big tile's accumulators are the
      // halves of each CTA's A rows, or of its B rows: 128 columns of either CTA's.
      const int32_t share = xent_share<kShape>(q, tc.n0);
      const int32_t cols = xent_share_of<kShape>(q, share, h);
      int32_t row0 = tc.m0 + quarter * 32, col = tc.n0 + half * share;
      if (kPair) row0 += (int32_t)rank * (T::rows(q.wide) / 2);
      if (kBig && q.wide) col += h * kXChunk;
      if (kBig && !q.wide) row0 += h * T::kRows;
      const int32_t row = row0 + lane;
      // what the row needs besides the sums, on its way during the wait
      int32_t target = -1, first = kXNoRow;
      float4 info = make_float4(0.0f, 0.0f, 0.0f, __int_as_float(-1));
      if (!kBig && q.kind == kXentStats && row < n_rows) target = p.targets[row];
      if (q.kind == kXentDlogits && row < n_rows) info = p.row_info[row];
      if (q.kind == kXentDweight && row < q.m_len) first = p.first[q.out_off + row];
      if (!wait_bounded(tfull0 + 8 * h, tile_phase, p.wait, abort_flag, kSleepHintNs)) {
        fail(kRoleEpilogue, abort_flag);
        break;
      }
      tc_fence_after_sync();
      const bool zero = tc.k_steps == 0;
      const uint32_t tacc = tmem_base + ((uint32_t)(quarter * 32) << 16) +
                            (uint32_t)(h * kXN + half * cols);
      if (q.kind == kXentStats) {
        if constexpr (!kBig)  // (big tiles are refused for the loss on the host)
          xent_epi_stats<kF16>(p, q, tacc, zero, row, row < n_rows, target, col);
      } else if (q.kind == kXentDlogits) {
        xent_epi_dlogits<kF16>(p, q, maps, st, tacc, zero, row0, row, n_rows, info, col);
      } else if (q.kind == kXentDweight) {
        xent_epi_dweight<kF16>(p, q, maps, st, tacc, zero, first, row0, row, col, cols);
      } else {
        xent_epi_dhidden(p, q, maps, st, tacc, zero, tc.split, row0, n_rows, col, cols);
      }
      tc_fence_before_sync();
      if constexpr (kPair)
        mbar_arrive_remote(tempty0 + 8 * h, 0);
      else
        mbar_arrive(tempty0 + 8 * h);
    }
    if (lane == 0) bulk_wait_all();  // the stores have left this CTA's shared memory and landed
    __syncwarp();
  }

  tc_fence_before_sync();
  if constexpr (kPair) {
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after_sync();
    if constexpr (kPair)
      tmem_dealloc_pair(tmem_base, kXTmemCols);
    else
      tmem_dealloc(tmem_base, kXTmemCols);
  }
}

// ------------------------------------------------------------------ rows that count

// The rows whose target is not `ignore`, side by side: packed hidden rows, their targets, the
// packed place of every row (-1: ignored), the row of every packed place, and their number. Each
// block places `block_rows` (at most 32) rows: it counts the rows that count before its own and in
// all (the targets are a few KB that sit in L2; a scan over blocks would be a launch of its own),
// then copies. The packed rows up to the next multiple of 64 are cleared: the weight gradient's
// product takes rows 64 at a time. A packed row begins on a 128-byte line, with zeros before it: TMA is
// slower on boxes of 128-byte rows that do not (4096 x 1000 x 50304, gradient: 1225 us, with the
// rows 2000 bytes apart 1370; loss: 415 and 474).
constexpr int kPackRows = 32, kPackThreads = 256;
__global__ void __launch_bounds__(kPackThreads)
    xent_pack_kernel(const uint4* hidden, const int32_t* targets,
                     int32_t rows, int32_t block_rows, int32_t row_vecs, int32_t packed_vecs,
                     int32_t ignore, uint4* packed,
                     int32_t* packed_targets, int32_t* place, int32_t* row_of, int32_t* n_rows) {
  __shared__ int32_t s_before[kPackThreads / 32], s_all[kPackThreads / 32];
  __shared__ int32_t s_place[kPackRows];
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t r0 = (int32_t)blockIdx.x * block_rows;
  int32_t before = 0, all = 0;
  for (int32_t r = threadIdx.x; r < rows; r += kPackThreads) {
    const int32_t counts = targets[r] != ignore;
    all += counts;
    if (r < r0) before += counts;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  all = __reduce_add_sync(0xffffffffu, all);
  if (lane == 0) {
    s_before[warp] = before;
    s_all[warp] = all;
  }
  __syncthreads();
  before = all = 0;
#pragma unroll
  for (int w = 0; w < kPackThreads / 32; ++w) {
    before += s_before[w];
    all += s_all[w];
  }
  if (warp == 0) {
    const int32_t r = r0 + lane;
    const bool mine = lane < block_rows && r < rows;
    const int32_t t = mine ? targets[r] : ignore;
    const bool counts = t != ignore;
    const uint32_t mask = __ballot_sync(0xffffffffu, counts);
    const int32_t at = before + __popc(mask & ((1u << lane) - 1u));
    s_place[lane] = counts ? at : -1;
    if (mine) place[r] = counts ? at : -1;
    if (counts) {
      row_of[at] = r;
      packed_targets[at] = t;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *n_rows = all;
  __syncthreads();
  for (int i = warp; i < block_rows; i += kPackThreads / 32) {
    const int32_t at = s_place[i];
    if (at < 0) continue;
    const uint4* src = hidden + (int64_t)(r0 + i) * row_vecs;
    uint4* dst = packed + (int64_t)at * packed_vecs;
#pragma unroll 4
    for (int32_t x = lane; x < row_vecs; x += 32) dst[x] = load_cs(src + x);
    if (row_vecs + lane < packed_vecs) dst[row_vecs + lane] = make_uint4(0u, 0u, 0u, 0u);
  }
  const int32_t end = (all + kBK - 1) / kBK * kBK;
  for (int32_t r = all + (int32_t)blockIdx.x; r < end; r += (int32_t)gridDim.x)
    for (int32_t x = threadIdx.x; x < packed_vecs; x += kPackThreads)
      packed[(int64_t)r * packed_vecs + x] = make_uint4(0u, 0u, 0u, 0u);
}

// ------------------------------------------------------------------ the target's logit

// z of one row's target, summed here in fp32 and not taken from the tensor cores: their fp32
// accumulator drops low bits at each of its H / 16 steps and comes out about 1e-6 of z low at
// H = 1024 (twice that at 2048), always towards zero, so the error would not average out over the
// rows of a mean. The loss is a difference against this one logit; for the others the same loss is
// a factor of 1 + 1e-6 z in the softmax. Called by a whole warp, the result in every lane.
template <bool kF16>
__device__ __forceinline__ float xent_target_logit(const uint4* h,
                                                   const uint4* w, int32_t row_vecs,
                                                   const uint16_t* bias, int32_t t, float alpha) {
  float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 4
  for (int32_t x = (int)(threadIdx.x & 31); x < row_vecs; x += 32) {
    const uint4 a = h[x], b = w[x];
    const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s0 = fmaf(unpack16<kF16>(u[i] & 0xffffu), unpack16<kF16>(v[i] & 0xffffu), s0);
      s1 = fmaf(unpack16<kF16>(u[i] >> 16), unpack16<kF16>(v[i] >> 16), s1);
    }
  }
  float s = s0 + s1;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return alpha * (bias != nullptr ? s + unpack16<kF16>(bias[t]) : s);
}

// ------------------------------------------------------------------ the loss from the statistics

// Folds each row's (max, sum) pairs in a fixed order, joins the target's term and writes lse and the
// row's loss. The chunks are taken as 128 segments of consecutive ones, each folded in order, then
// the segments in order, a warp a row. A block serves kRows rows, 8 or 32, and as many lanes read the
// pairs of its rows of a chunk: 8 make four times the blocks, for few rows; 32 read 256 bytes at a
// place and not 64, for many (8192 rows of 151936 entries: 62 us with 8 a block). The order, and so
// every bit, is the same. With x = z * log2(e) and the
// others' (m, s):
//   lse - z_t = log1p(s * 2^(m - x_t))                        where the target leads,
//             = (m - x_t + log2(s + 2^(x_t - m))) / log2(e)   elsewhere,
// so the loss of a row that is almost sure of its target keeps its bits. Ignored rows get 0 and 0 (they
// have no place among the packed rows; where rows were not packed, their target is `ignore`);
// a target outside [0, V) makes the row's loss NaN, and its lse is that of all entries. Where the
// launch is a single cluster (at most 64 rows), its first block also adds the rows up in order
// (`total`), which saves the next launch.
__device__ __forceinline__ void xent_merge(float& m, float& s, float m2, float s2) {
  // NaN sums (a NaN or +inf logit) survive: exp of a NaN difference is NaN, and so is NaN * 0
  const float nm = fmaxf(m, m2);
  const float ref = nm == -INFINITY ? 0.0f : nm;
  s = s * exp2f(m - ref) + s2 * exp2f(m2 - ref);
  m = nm;
}
constexpr int kFoldFew = 8, kFoldMany = 32, kFoldSegs = 128, kFoldCluster = 8;
template <int kRows, bool kF16>
__global__ void __launch_bounds__(1024)
    xent_fold_kernel(const float2* partials, int32_t n_chunks, int32_t pitch,
                     int32_t rows, int32_t V, const int32_t* place,
                     const int32_t* targets, const uint4* hidden,
                     const uint4* W, int32_t row_vecs,
                     const uint16_t* bias, float alpha, float z_loss,
                     float* row_loss, float* lse_out, int32_t ignoring, int32_t ignore,
                     int32_t mean, float* total) {
  constexpr int kOwn = kFoldSegs * kRows / 1024;  // segments of a lane
  __shared__ float2 seg[kFoldSegs][kRows + 1];
  __shared__ float s_loss[kRows];
  __shared__ int32_t s_counts[kRows];
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t r0 = (int32_t)blockIdx.x * kRows;
  {
    const int row = lane % kRows, part = (int)threadIdx.x / kRows;
    const int32_t r = r0 + row;
    const int32_t at = r >= rows ? -1 : place != nullptr ? place[r] : r;
    const int per_seg = (n_chunks + kFoldSegs - 1) / kFoldSegs;
#pragma unroll 1
    for (int k = part * kOwn; k < (part + 1) * kOwn; ++k) {
      const int c0 = k * per_seg, c1 = at >= 0 ? min(n_chunks, c0 + per_seg) : c0;
      float m = -INFINITY, s = 0.0f;
      for (int c = c0; c < c1; c += 8) {
        float2 q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          q[i] = c + i < c1 ? load_cs(partials + (int64_t)(c + i) * pitch + at)
                            : make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) xent_merge(m, s, q[i].x, q[i].y);
      }
      seg[k][row] = make_float2(m, s);
    }
  }
  // the row's own warp: the target's logit, then the segments
  const int32_t r = r0 + warp;
  const bool mine = warp < kRows && r < rows;  // the whole warp
  const int32_t t = mine ? targets[r] : -1;
  const bool counts = mine && !(ignoring && t == ignore);
  const bool held = counts && t >= 0 && t < V;
  float zt = 0.0f;
  if (held)
    zt = xent_target_logit<kF16>(hidden + (int64_t)r * row_vecs, W + (int64_t)t * row_vecs,
                                 row_vecs, bias, t, alpha);
  __syncthreads();
  float loss = 0.0f, lse = 0.0f;
  if (counts) {
    float m = -INFINITY, s = 0.0f;
#pragma unroll
    for (int i = 0; i < kFoldSegs / 32; ++i) {
      const float2 q = seg[lane * (kFoldSegs / 32) + i][warp];
      xent_merge(m, s, q.x, q.y);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float m2 = __shfl_down_sync(0xffffffffu, m, o), s2 = __shfl_down_sync(0xffffffffu, s, o);
      xent_merge(m, s, m2, s2);  // (lanes past the end fold others' parts; lane 0 is used)
    }
    m = __shfl_sync(0xffffffffu, m, 0);
    s = __shfl_sync(0xffffffffu, s, 0);
    if (held) {
      const float xt = zt * kLog2e;
      if (zt == INFINITY) {  // inf - inf, as for +inf elsewhere in the row
        loss = lse = __int_as_float(0x7fc00000);
      } else if (xt >= m) {
        loss = log1pf(s * exp2f(m - xt));
        lse = zt + loss;
      } else {
        const float l = log2f(s + exp2f(xt - m));
        lse = (m + l) * kLn2;
        // (a target near the lowest fp32 value, taken out by its bias: x_t is past it)
        loss = xt > -INFINITY ? (m - xt + l) * kLn2 : lse - zt;
      }
    } else {
      lse = (m + log2f(s)) * kLn2;
      loss = __int_as_float(0x7fc00000);
    }
    if (z_loss != 0.0f) loss += z_loss * lse * lse;
  }
  if (mine && lane == 0) {
    lse_out[r] = lse;
    row_loss[r] = loss;
  }
  if (total == nullptr) return;
  if (warp < kRows && lane == 0) {
    s_loss[warp] = loss;
    s_counts[warp] = counts;
  }
  cluster_sync_all();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    float sum = 0.0f;
    int32_t n = 0;
    for (uint32_t c = 0; c < gridDim.x; ++c) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        sum += cluster_load_f32(&s_loss[i], c);
        n += cluster_load(&s_counts[i], c);
      }
    }
    *total = mean ? sum / (float)max(n, 1) : sum;
  }
  cluster_sync_all();  // (the other blocks' sums have been read)
}

// The rows' losses added in a fixed order (each of 1024 threads every 1024th row, then a tree),
// and divided by the number of rows that count (at least 1) for the mean.
__global__ void __launch_bounds__(1024)
    xent_reduce_kernel(const float* row_loss, const int32_t* targets,
                       int32_t rows, int32_t ignoring, int32_t ignore, int32_t mean, float* loss) {
  __shared__ float part[32];
  __shared__ int32_t count[32];
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float s = 0.0f;
  int32_t n = 0;
  for (int32_t r = threadIdx.x; r < rows; r += 1024) {
    s += row_loss[r];
    n += !(ignoring && targets[r] == ignore);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) {
    part[warp] = s;
    count[warp] = n;
  }
  __syncthreads();
  if (warp > 0) return;
  s = part[lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  n = __reduce_add_sync(0xffffffffu, count[lane]);
  if (lane == 0) *loss = mean ? s / (float)max(n, 1) : s;
}

// ------------------------------------------------------------------ factors of the gradient

// (lse * log2(e), a, d at the target, target) of every row that counts, and scale[1] = the factor
// of the gradients (see the top of this file). The target's entry of d, a p - b, is taken from the
// target's exact logit as b (p - 1) + (a - b) p with p - 1 = expm1(z_t - lse), so that a row
// almost sure of its target keeps its small gradient. What its rounding to 16 bits takes away goes
// to lost[i]: it is the largest entry of most rows, so its error is the same throughout a row of
// dH, and, where few rows have that target, of dW (xent_finish_kernel puts it back). Also clears
// the table of the targets' first rows. The power of two needs the largest factor of
// all rows first: each block finds it by itself (a few KB that sit in L2), then takes rows 32 at a
// time, a warp a row. A target outside [0, V) makes its row NaN.
constexpr int kRowsBlock = 32;
template <bool kF16>
__global__ void __launch_bounds__(1024)
    xent_rows_kernel(const float* lse, const int32_t* targets,
                     const int32_t* row_of, int32_t rows,
                     const int32_t* n_rows, int32_t V,
                     const uint4* hidden, const uint4* W,
                     int32_t row_vecs, const uint16_t* bias,
                     const float* grad, int32_t per_row, int32_t mean, float z_loss,
                     float alpha, float4* row_info, float* lost, float* scale, int32_t* first) {
  __shared__ float part[32];
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();
  for (int32_t v = (int32_t)blockIdx.x * 1024 + (int32_t)threadIdx.x; v < V;
       v += (int32_t)gridDim.x * 1024)
    first[v] = kXNoRow;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t n = n_rows != nullptr ? *n_rows : rows;
  float top = 1.0f;
  if (per_row || z_loss != 0.0f) {
    top = 0.0f;
    for (int32_t i = threadIdx.x; i < n; i += 1024) {
      const int32_t r = row_of != nullptr ? row_of[i] : i;
      const float b = per_row ? fabsf(grad[r]) : 1.0f;
      const float a = fabsf(b * (1.0f + 2.0f * z_loss * lse[r]));
      if (a < INFINITY) top = fmaxf(top, a);  // (false for NaN)
      if (b < INFINITY) top = fmaxf(top, b);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) part[warp] = top;
    __syncthreads();
    top = part[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  // (2^k and 2^-k stay normal numbers: top may be any fp32 value)
  const int k = top > 0.0f ? min(126, 13 - ilogbf(top)) : 0;
  const float up = ldexpf(1.0f, k), down = ldexpf(1.0f, -k);
  for (int32_t i = (int32_t)blockIdx.x * kRowsBlock + warp; i < n;
       i += (int32_t)gridDim.x * kRowsBlock) {
    const int32_t r = row_of != nullptr ? row_of[i] : i;
    const int32_t t = targets[r];
    const float l = lse[r];
    const float b = (per_row ? grad[r] : 1.0f) * up;
    float a = z_loss != 0.0f ? b * (1.0f + 2.0f * z_loss * l) : b;
    float at_target = __int_as_float(0x7fc00000);
    if (t >= 0 && t < V) {  // the whole warp
      const float z = xent_target_logit<kF16>(hidden + (int64_t)r * row_vecs,
                                              W + (int64_t)t * row_vecs, row_vecs, bias, t, alpha);
      const float e = expm1f(z - l);
      at_target = b * e;
      if (z_loss != 0.0f) at_target += b * (2.0f * z_loss * l) * (e + 1.0f);
    } else {
      a = at_target;
    }
    if (lane == 0) {
      row_info[i] = make_float4(l * kLog2e, a, at_target, __int_as_float(t));
      lost[i] = at_target - unpack16<kF16>(pack16<kF16>(at_target, 0.0f) & 0xffffu);
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    float f = alpha;
    if (!per_row) f *= mean ? *grad / (float)max(n, 1) : *grad;
    scale[0] = up;
    scale[1] = f * down;
  }
}

// The launch that ends the gradient. Its first `hidden_blocks` blocks write dH from its partial
// sums: the splits in order, plus what the target's entry of d lost in its rounding times the
// target's row of W, times the factor, rounded once; ignored rows 0. A thread takes 8 entries of a
// row. The other blocks write the rows of dW that are some row's target once more, from the fp32
// values that the product left in `side`: a block takes 2048 columns of the target of one row that
// counts, if no earlier row has the same target, and adds what d lost there, for all rows of that
// target in order. With it dH, and dW at the targets, are as far off as their own rounding where the
// target is most of its row's d; without, by half as much again (96 weighted rows: 0.0026 and not
// 0.0017 of dH). The rows of one target are added one after another, a memory latency each: a target
// of very many rows costs more time than it need.
struct XentFinishParams {
  int32_t rows, H, V;
  const int32_t* n_rows;
  const int32_t* place;
  const int32_t* targets;         // [rows]
  const int32_t* packed_targets;  // [rows that count]
  const float* lost;
  const float* scale;
  // dH
  int32_t hidden_blocks;
  int32_t splits;
  int64_t split_len;
  const float* partial;
  const uint4* W;
  uint4* d_hidden;
  // dW
  int32_t slices;                 // blocks a row
  const int32_t* first;
  const float* side;
  const uint4* hidden;            // the rows that count
  int32_t hidden_vecs;            // from one to the next
  uint4* d_weight;
};
constexpr int kFinishThreads = 256, kFinishScan = 16;

template <bool kF16>
__device__ __forceinline__ void xent_fma8(float (&s)[8], float e, const uint4& q) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    s[2 * j] = fmaf(e, unpack16<kF16>(w[j] & 0xffffu), s[2 * j]);
    s[2 * j + 1] = fmaf(e, unpack16<kF16>(w[j] >> 16), s[2 * j + 1]);
  }
}

__device__ __forceinline__ void xent_add8(float (&s)[8], const float4* src) {
  const float4 u = load_cs(src), v = load_cs(src + 1);
  s[0] += u.x;
  s[1] += u.y;
  s[2] += u.z;
  s[3] += u.w;
  s[4] += v.x;
  s[5] += v.y;
  s[6] += v.z;
  s[7] += v.w;
}

template <bool kF16>
__device__ __forceinline__ uint4 xent_pack8(const float (&s)[8]) {
  return make_uint4(pack16<kF16>(s[0], s[1]), pack16<kF16>(s[2], s[3]), pack16<kF16>(s[4], s[5]),
                    pack16<kF16>(s[6], s[7]));
}

template <bool kF16>
__device__ __forceinline__ void xent_finish_hidden(const XentFinishParams& p) {
  const int32_t row_vecs = p.H / 8;
  const int64_t i = (int64_t)blockIdx.x * kFinishThreads + threadIdx.x;
  if (i >= (int64_t)p.rows * row_vecs) return;
  const int32_t r = (int32_t)(i / row_vecs), x = (int32_t)(i - (int64_t)r * row_vecs);
  const int32_t at = p.place != nullptr ? p.place[r] : r;
  uint4 out = make_uint4(0u, 0u, 0u, 0u);
  if (at >= 0) {
    const float f = p.scale[1];
    float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    const float4* src =
        reinterpret_cast<const float4*>(p.partial) + ((int64_t)at * row_vecs + x) * 2;
#pragma unroll 8
    for (int32_t k = 0; k < p.splits; ++k) xent_add8(s, src + k * (p.split_len / 4));
    const int32_t t = p.targets[r];
    if (t >= 0 && t < p.V)  // (elsewhere the row is NaN already)
      xent_fma8<kF16>(s, p.lost[at], p.W[(int64_t)t * row_vecs + x]);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] *= f;
    out = xent_pack8<kF16>(s);
  }
  p.d_hidden[i] = out;
}

template <bool kF16>
__device__ __forceinline__ void xent_finish_weight(const XentFinishParams& p) {
  __shared__ uint32_t s_hits[kFinishScan * kFinishThreads / 32];
  const int32_t b = (int32_t)blockIdx.x - p.hidden_blocks;
  const int32_t i = b / p.slices, slice = b - i * p.slices;
  const int32_t n = p.n_rows != nullptr ? *p.n_rows : p.rows;
  if (i >= n) return;
  const int32_t t = p.packed_targets[i];
  if (t < 0 || t >= p.V || p.first[t] != i) return;  // (the same for the whole block)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t row_vecs = p.H / 8;
  const int32_t x = slice * kFinishThreads + (int)threadIdx.x;
  const bool mine = x < row_vecs;
  const float f = p.scale[1];
  float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (mine)
    xent_add8(s, reinterpret_cast<const float4*>(p.side) + ((int64_t)i * row_vecs + x) * 2);
  // the rows with this target, 4096 at a time (none is before row i)
  for (int32_t r0 = i & ~31; r0 < n; r0 += kFinishScan * kFinishThreads) {
    bool hit[kFinishScan];
#pragma unroll
    for (int k = 0; k < kFinishScan; ++k) {
      const int32_t r = r0 + (k * (kFinishThreads / 32) + warp) * 32 + lane;
      hit[k] = r < n && p.packed_targets[r] == t;
    }
#pragma unroll
    for (int k = 0; k < kFinishScan; ++k) {
      const uint32_t bits = __ballot_sync(0xffffffffu, hit[k]);
      if (lane == 0) s_hits[k * (kFinishThreads / 32) + warp] = bits;
    }
    __syncthreads();
    for (int w0 = 0; w0 < kFinishScan * kFinishThreads / 32; w0 += 32) {
      const uint32_t my = s_hits[w0 + lane];
      for (uint32_t words = __ballot_sync(0xffffffffu, my != 0); words != 0; words &= words - 1) {
        const int w = __ffs((int)words) - 1;
        for (uint32_t bits = __shfl_sync(0xffffffffu, my, w); bits != 0; bits &= bits - 1) {
          const int32_t r = r0 + (w0 + w) * 32 + __ffs((int)bits) - 1;
          const float e = p.lost[r] * f;
          if (mine) xent_fma8<kF16>(s, e, p.hidden[(int64_t)r * p.hidden_vecs + x]);
        }
      }
    }
    __syncthreads();
  }
  if (mine) p.d_weight[(int64_t)t * row_vecs + x] = xent_pack8<kF16>(s);
}

template <bool kF16>
__global__ void __launch_bounds__(kFinishThreads)
    xent_finish_kernel(const XentFinishParams p) {
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();
  if ((int32_t)blockIdx.x < p.hidden_blocks)
    xent_finish_hidden<kF16>(p);
  else
    xent_finish_weight<kF16>(p);
}

// dbias of a piece: the column sums of d in fp32 that the product which made d left for each 32
// rows, added up (read again from d itself, 134 MB a piece of 4096 rows, this took 18 us a piece). A
// block takes 64 columns, 8 threads each: every 8th block of 32 rows, then the eight in order.
constexpr int kBiasCols = 64, kBiasParts = 8;
template <bool kF16>
__global__ void __launch_bounds__(kBiasCols* kBiasParts)
    xent_bias_kernel(const float* part, int32_t pitch, int32_t cols, int32_t rows,
                     const int32_t* n_rows, const float* scale, int32_t add,
                     uint16_t* d_bias) {
  __shared__ float s_part[kBiasParts][kBiasCols];
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();
  const int32_t n = n_rows != nullptr ? *n_rows : rows;
  const int col = (int)threadIdx.x % kBiasCols, k = (int)threadIdx.x / kBiasCols;
  const int32_t c = (int32_t)blockIdx.x * kBiasCols + col;
  float s = 0.0f;
  // (a 64-column box of d is whole wherever one of its columns is)
#pragma unroll 8
  for (int32_t b = k; b < (n + 31) / 32; b += kBiasParts) s += part[(int64_t)b * pitch + c];
  s_part[k][col] = s;
  __syncthreads();
  if (k > 0 || c >= cols) return;
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < kBiasParts; ++i) t += s_part[i][col];
  t = n > 0 ? t * scale[1] : 0.0f;
  uint16_t* at = d_bias + c;
  if (add) t += unpack16<kF16>(*at);
  *at = (uint16_t)(pack16<kF16>(t, 0.0f) & 0xffffu);
}

}  // namespace lmh
