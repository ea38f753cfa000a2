// Softmax cross entropy over the LM head's vocabulary with its gradient, no logits kept.
//
//   z[r, v] = alpha * (sum_k h[r, k] * W[v, k] + bias[v])                 fp32
//   lse_r   = log sum_v exp z[r, v],   loss_r = lse_r - z[r, t_r] + z_loss * lse_r^2
//   d[r, v] = a_r * exp(z[r, v] - lse_r) - b_r * [v == t_r]               fp32, rounded to 16 bits
//   dH      = scale * d @ W,   dW = scale * d^T @ h,   dbias = scale * sum_r d[r, v]
//
// with a_r = 1 + 2 z_loss lse_r and b_r = 1 where every row has the same upstream gradient g (then
// scale = alpha * g / rows that count), or both times g_r where each row has its own (scale =
// alpha). So with one upstream gradient the target's entry of a row is p - 1, which bf16 holds to
// 2^-9 of a number near 1, and g itself is never rounded to 16 bits. A power of two 2^k joins a_r
// and b_r and leaves again with `scale`, so that the largest factor lies in [2^13, 2^14): fp16 has
// 2^-28 of the largest entry as its smallest normal number then (softmax values of 1e-8 keep all
// their bits), and 2^15, the most an entry can reach, stays below its 65504. bf16 takes the same
// path; there the power of two changes no bit.
//
// Why d is rounded to the operands' 16-bit type: it is the operand of two tensor-core products
// whose other operand has that type (one MMA never mixes types). Each rounding is off by at most
// half a step (2^-9 relative in bf16, 2^-12 in fp16), independently from entry to entry; the sums
// over the vocabulary and over the rows are fp32, and the gradients leave in that type anyway.
//
// Four products of 2 rows V H operations each: the logits for the loss, the logits again for the
// gradient (they are not kept), and the two gradients. The vocabulary is taken in pieces: the
// d of a piece ([rows, Vc], at most about 128 MB, two buffers) is written by the product that
// makes it and read by the two that follow. Each launch takes the tiles of three products, the
// two gradient products of piece c and the logits of piece c + 1, so the device drains once a
// piece and not three times.
//
// All products are one kernel, xent_gemm_kernel: C[M, N] = A[M, K] B[N, K]^T in tiles of 256 x 256
// on CTA pairs (128 x 256 on lone CTAs), operands by TMA as 64 x 64 boxes of 128-byte-swizzled
// rows, fp32 accumulators in TMEM (two of 256 columns, so that the epilogue of a tile runs under
// the MMAs of the next). An operand whose K runs along its rows in memory is a K-major tile of
// 8-row atoms; one whose K runs down the columns (h and d in dW = d^T h, W in dH = d W) is the same
// boxes read as an MN-major tile: 64 entries of M or N by 8 of K per atom. So nothing is ever
// transposed in memory. A TMEM lane holds a row of the tile: a thread has 128 logits of one row in
// turn, and the softmax statistics need no exchange between lanes.
//
// Rows whose target is ignored are taken out first (xent_pack_kernel): the rows that count are
// copied side by side, and every product runs over those alone. Masked rows cost no tensor time,
// and what they hold (NaN of padding) never meets a product. The number of rows that count is known
// on the device only; the tile walk reads it there.
//
// Roles as in the fp32 head: warp 0 TMA, warp 1 MMA, warps 2-9 epilogue; tiles by cluster launch
// control in launch order. No atomics on data and no split whose order varies: results are the
// same on every run.
#pragma once

#include "lmhead_bf16.cuh"

namespace lmh {

constexpr int kXN = 256;                  // tile columns (MMA N)
constexpr int kXBox = 64 * 64 * 2;        // bytes of one TMA box: 64 rows of 64 16-bit elements
constexpr int kXEpiWarps = 8;
constexpr int kXThreads = 64 + 32 * kXEpiWarps;
constexpr int kXStoreBox = 32 * 64 * 2;   // an epilogue warp's store box: 32 rows of 64 elements
constexpr int kXMaxProblems = 3;
constexpr int kXChunk = 128;              // vocab entries per (max, sum) pair of a row
constexpr uint32_t kXTmemCols = 2 * kXN;

template <bool kPair>
struct XentTile {
  static constexpr int kM = kPair ? 256 : 128;                // tile rows
  static constexpr int kBRows = kPair ? kXN / 2 : kXN;        // B rows in one CTA's shared memory
  static constexpr int kABytes = 128 * 64 * 2;
  static constexpr int kBBytes = kBRows * 64 * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = kPair ? 6 : 4;               // 192 KB either way
  static constexpr size_t kSmem =
      1024 + (size_t)kStages * kStageBytes + kXEpiWarps * kXStoreBox + 512;
};

enum : int32_t {
  kXentStats = 0,    // (max, sum of exp(z - max)) per row and 128 vocab entries, the target's logit
  kXentDlogits = 1,  // d, 16 bits, [rows, ld] of one vocab piece
  kXentDweight = 2,  // dW rows, 16 bits, optionally added to what is there
  kXentDhidden = 3,  // fp32 partial sums of dH, one buffer per split of K
};

// Tensor maps of one launch, all of them 2-D with 128-byte swizzle.
enum : int32_t {
  kMapHidden = 0,  // [rows, H], boxes of 64 rows
  kMapW = 1,       // [V, H], boxes of 64 rows
  kMapD0 = 2,      // d buffers [rows_pad, ld], boxes of 64 rows (loads)
  kMapD1 = 3,
  kMapD0Store = 4,  // the same with boxes of 32 rows (stores)
  kMapD1Store = 5,
  kMapDw = 6,      // dW [V, H], boxes of 32 rows (stores)
  kMapCount = 7,
};
struct XentMaps {
  CUtensorMap m[kMapCount];
};

struct XentProblem {
  int32_t kind;
  int32_t a_map, b_map, out_map;
  int32_t a_mn, b_mn;     // 1: the operand's K runs down the rows of its matrix
  int32_t m_rows;         // 1: M is the number of rows that count (else m_len)
  int32_t k_rows;         // 1: K is the number of rows that count (else k_len)
  int32_t m_len, n_len, k_len;
  int32_t a_off, b_off;   // first row of the operand's matrix (a piece of W starts at vocab b_off)
  int32_t b_k;            // 1: b_off is along K (dH: the piece's rows of W are B's K)
  int32_t splits;         // of K
  int32_t out_off;        // first output row (dW: the piece's first vocab entry)
  int32_t add;            // dW: add to what is there; dH: add to the partial sums
};

struct XentParams {
  int32_t n_problems;
  XentProblem prob[kXMaxProblems];
  int32_t rows;               // rows of hidden (the number that count when n_rows is null)
  const int32_t* n_rows;      // device: how many rows count, or null
  int32_t H;
  int32_t rows_pad;           // row pitch of the dH partial buffers
  int32_t group;              // M tiles walked together (their rows stay in L2)
  float alpha;
  const uint16_t* bias;       // [V] or null
  const int32_t* targets;     // [rows that count]
  float2* partials;           // stats: [2 * ceil(V / 256)][rows]
  float* target_z;            // stats: [rows that count]
  const float4* row_info;     // dlogits: (lse, a, b, target as int bits) of each row that counts
  const float* scale;         // device: [1] = the factor of the gradients
  uint16_t* d_weight;         // dW as memory, for add
  float* dh_partial;          // [splits][rows_pad][H]
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

// As mma_bf16_ss_elect for a CTA pair (issued by the even CTA only).
__device__ __forceinline__ void mma_bf16_ss_pair_elect(uint32_t d_tmem, uint64_t a_desc,
                                                       uint64_t b_desc, uint32_t idesc,
                                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Shared-memory descriptor of an MN-major tile in 64 x 64 boxes: each box is 64 K rows of 128
// bytes (64 entries of M or N, 128-byte swizzle), 8 K rows make an atom of 1024 bytes (the stride
// offset), the next 64 entries of M or N are the next box (the leading offset).
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw128(uint32_t smem_addr) {
  const uint64_t start = (smem_addr & 0x3FFFFu) >> 4;
  const uint64_t lbo = (uint32_t)kXBox >> 4;
  const uint64_t sbo = 1024u >> 4;
  return start | (lbo << 16) | (sbo << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int32_t x,
                                             int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
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

// Tile t of the launch: the problems one after another, each split by split, M tiles in groups
// walked N-major (a wave of tiles is then about as high as wide, and its operands fit L2).
template <int kM>
__device__ __forceinline__ XentTileAt xent_tile(const XentParams& p, int32_t n_rows, int32_t t) {
  XentTileAt c;
  c.prob = -1;
  c.m0 = c.n0 = c.k0 = c.k_steps = c.split = 0;
#pragma unroll
  for (int i = 0; i < kXMaxProblems; ++i) {
    if (i >= p.n_problems) break;
    const XentProblem& q = p.prob[i];
    const int32_t mt = ceil_div(q.m_rows ? n_rows : q.m_len, kM);
    const int32_t nt = ceil_div(q.n_len, kXN);
    const int32_t per = mt * nt, count = per * q.splits;
    if (t < count) {
      const int32_t split = t / per;
      const int32_t u = t - split * per;
      const int32_t g = u / (p.group * nt);
      const int32_t local = u - g * p.group * nt;
      const int32_t gm = min(p.group, mt - g * p.group);
      const int32_t n = local / gm;
      c.prob = i;
      c.m0 = (g * p.group + (local - n * gm)) * kM;
      c.n0 = n * kXN;
      c.split = split;
      const int32_t ks = ceil_div(q.k_rows ? n_rows : q.k_len, kBK);
      c.k0 = (int32_t)((int64_t)ks * split / q.splits);
      c.k_steps = (int32_t)((int64_t)ks * (split + 1) / q.splits) - c.k0;
      return c;
    }
    t -= count;
  }
  return c;
}

// ------------------------------------------------------------------ epilogues
// Each is called by one warp with its 32 rows of the tile (row = its lane's) and its 128 columns
// from `col`; `tacc` addresses the first of them in TMEM; `zero` says that K was empty and the
// accumulator was never written.

__device__ __forceinline__ void xent_acc32(uint32_t tacc, bool zero, uint32_t (&r)[32]) {
  __syncwarp();  // the lanes may come from rows of their own; the TMEM load is the warp's
  if (zero) {
#pragma unroll
    for (int j = 0; j < 32; ++j) r[j] = 0u;
  } else {
    tmem_ld_32x32b_x32(tacc, r);
    tmem_ld_wait();
  }
}

// Lane's own column of 32: the bias of vocab entry v0 + lane (0 past the end or without a bias).
template <bool kF16>
__device__ __forceinline__ float xent_bias(const XentParams& p, int32_t v0, int32_t v_end) {
  const int32_t v = v0 + (int)(threadIdx.x & 31);
  return p.bias != nullptr && v < v_end ? unpack16<kF16>(p.bias[v]) : 0.0f;
}

__device__ __forceinline__ float xent_logit(const XentParams& p, uint32_t acc, float bias_lane,
                                            int j) {
  const float a = __uint_as_float(acc);
  return p.bias == nullptr
             ? __fmul_rn(p.alpha, a)
             : __fmul_rn(p.alpha, __fadd_rn(a, __shfl_sync(0xffffffffu, bias_lane, j)));
}

// (max, sum of exp(z - max)) of this thread's row over its 128 vocab entries, and the target's
// logit if it is one of them. Per 32 entries: their maximum first, one rescaling of the running
// sum, then the terms. Entries past V count as -inf; a row of -inf alone gives (-inf, 0).
template <bool kF16>
__device__ __forceinline__ void xent_epi_stats(const XentParams& p, const XentProblem& q,
                                               uint32_t tacc, bool zero, int32_t row, bool row_ok,
                                               int32_t col) {
  const int32_t V = q.n_len;
  const int32_t t = row_ok ? p.targets[row] : -1;
  float m = -INFINITY, s = 0.0f;
#pragma unroll 1
  for (int c = 0; c < kXChunk && col + c < V; c += 32) {
    uint32_t r[32];
    xent_acc32(tacc + (uint32_t)c, zero, r);
    const int32_t v0 = col + c;
    const float b = xent_bias<kF16>(p, v0, V);
    float cm = -INFINITY;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      float z = xent_logit(p, r[j], b, j);
      if (v0 + j >= V) z = -INFINITY;
      r[j] = __float_as_uint(z);
      cm = fmaxf(cm, z);
    }
    if (__any_sync(0xffffffffu, t >= v0 && t < v0 + 32)) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (v0 + j == t && t < V) p.target_z[row] = __uint_as_float(r[j]);
    }
    const float nm = fmaxf(m, cm);
    const float ref = nm == -INFINITY ? 0.0f : nm;
    // a NaN logit reaches the sum through its own term; +inf gives inf - inf there, NaN as well
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      s0 += __expf(__uint_as_float(r[j]) - ref);
      s1 += __expf(__uint_as_float(r[j + 1]) - ref);
    }
    s = s * __expf(m - ref) + (s0 + s1);
    m = nm;
  }
  if (row_ok && col < V)
    __stcs(p.partials + (int64_t)(col / kXChunk) * p.rows + row, make_float2(m, s));
}

// The 64 columns of one store box, as 16-bit values in this warp's swizzled staging buffer.
struct XentStage {
  uint32_t buf;  // 32 rows of 128 bytes, 1024-byte aligned
  __device__ __forceinline__ void begin() const {
    if ((threadIdx.x & 31) == 0) bulk_wait_read();
    __syncwarp();
  }
  // 32 columns: four 16-byte pieces, `half` 0 or 1 of the box
  __device__ __forceinline__ void put(int half, const uint32_t (&w)[16]) const {
    const uint32_t row = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      st_shared_v4(buf + row * 128u + (((uint32_t)(half * 4 + j) ^ (row & 7u)) << 4), w[4 * j],
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

// d of this thread's row over its 128 vocab entries of the piece, 16 bits, into the piece's buffer.
// Rows that do not count and entries past V are written as 0: the products that read d take whole
// 64-wide steps.
template <bool kF16>
__device__ __forceinline__ void xent_epi_dlogits(const XentParams& p, const XentProblem& q,
                                                 const XentMaps& maps, const XentStage& st,
                                                 uint32_t tacc, bool zero, int32_t row0,
                                                 int32_t row, bool row_ok, int32_t col) {
  const int32_t V = q.b_off + q.n_len;  // the end of the piece as vocab ids
  float4 info = make_float4(0.0f, 0.0f, 0.0f, __int_as_float(-1));
  if (row_ok) info = p.row_info[row];
  const int32_t t = __float_as_int(info.w);
#pragma unroll 1
  for (int c = 0; c < kXChunk && col + c < q.n_len; c += 64) {
    st.begin();
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      uint32_t r[32], w[16];
      xent_acc32(tacc + (uint32_t)(c + 32 * h), zero, r);
      const int32_t v0 = q.b_off + col + c + 32 * h;
      const float b = xent_bias<kF16>(p, v0, V);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float z = xent_logit(p, r[j], b, j);
        const float d = info.y * __expf(z - info.x);
        r[j] = row_ok && v0 + j < V ? __float_as_uint(d) : 0u;
      }
      if (__any_sync(0xffffffffu, t >= v0 && t < v0 + 32)) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (v0 + j == t) r[j] = __float_as_uint(__uint_as_float(r[j]) - info.z);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j)
        w[j] = pack16<kF16>(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
      st.put(h, w);
    }
    st.store(&maps.m[q.out_map], col + c, row0);
  }
}

// dW of this thread's vocab entry: the sum times `scale`, added in fp32 to what is there if asked
// for, rounded once.
template <bool kF16>
__device__ __forceinline__ void xent_epi_dweight(const XentParams& p, const XentProblem& q,
                                                 const XentMaps& maps, const XentStage& st,
                                                 uint32_t tacc, bool zero, int32_t row0,
                                                 int32_t row, int32_t col) {
  const float scale = p.scale[1];
  const bool row_ok = row < q.m_len;
  const int64_t at = (int64_t)(q.out_off + row) * p.H;
#pragma unroll 1
  for (int c = 0; c < kXChunk && col + c < p.H; c += 64) {
    st.begin();
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      uint32_t r[32], w[16];
      const int32_t x = col + c + 32 * h;
      xent_acc32(tacc + (uint32_t)(c + 32 * h), zero, r);
#pragma unroll
      for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * scale);
      // nothing to add where no row counts: 0 times a scale that may be NaN stays 0
      if (zero) {
#pragma unroll
        for (int j = 0; j < 32; ++j) r[j] = 0u;
      }
      if (q.add && row_ok) {
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
#pragma unroll
      for (int j = 0; j < 16; ++j)
        w[j] = pack16<kF16>(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
      st.put(h, w);
    }
    // a box that starts past the piece's rows belongs to the next piece or to nothing
    if (row0 < q.m_len) st.store(&maps.m[q.out_map], col + c, q.out_off + row0);
  }
}

// fp32 sums of dH over this piece's (and split's) vocab entries, added to the earlier pieces'.
__device__ __forceinline__ void xent_epi_dhidden(const XentParams& p, const XentProblem& q,
                                                 uint32_t tacc, bool zero, int32_t split,
                                                 int32_t row, bool row_ok, int32_t col) {
  float* dst = p.dh_partial + ((int64_t)split * p.rows_pad + row) * p.H;
#pragma unroll 1
  for (int c = 0; c < kXChunk && col + c < p.H; c += 32) {
    uint32_t r[32];
    xent_acc32(tacc + (uint32_t)c, zero, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int32_t x = col + c + 4 * j;
      if (row_ok && x < p.H) {
        float4 v = make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                               __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3]));
        float4* a = reinterpret_cast<float4*>(dst + x);
        if (q.add) {
          const float4 o = *a;
          v.x += o.x;
          v.y += o.y;
          v.z += o.z;
          v.w += o.w;
        }
        *a = v;
      }
    }
  }
}

// ------------------------------------------------------------------ the kernel

template <bool kPair, bool kF16>
__global__ void __launch_bounds__(kXThreads, 1)
    xent_gemm_kernel(const __grid_constant__ XentMaps maps, const __grid_constant__ XentParams p) {
  using T = XentTile<kPair>;
  extern __shared__ uint8_t smem_raw[];
  if (threadIdx.x == 0) pdl_trigger();
  uint8_t* smem = align_up_1024(smem_raw);
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  constexpr int S = T::kStages;
  const uint32_t rank = kPair ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;

  uint8_t* staging = smem + (size_t)S * T::kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + kXEpiWarps * kXStoreBox);
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = smem_u32(bars + S);
  const uint32_t tfull0 = smem_u32(bars + 2 * S);
  const uint32_t tempty0 = smem_u32(bars + 2 * S + 2);
  const uint32_t done_bar = smem_u32(bars + 2 * S + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // (2 * S is even, so the 16-byte answer slots are aligned)
  const ClcRing clc{smem_u32(bars + 2 * S + 6), smem_u32(bars + 2 * S + 14),
                    smem_u32(bars + 2 * S + 18)};
  constexpr uint32_t kReaders = (kPair ? 2u : 1u) * (1u + kXEpiWarps) + 1u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int k = 0; k < kClcSlots; ++k) {
      mbar_init(clc.full0 + 8 * k, 1);
      mbar_init(clc.empty0 + 8 * k, kReaders);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull0 + 8 * a, 1);
      mbar_init(tempty0 + 8 * a, (kPair ? 2 : 1) * 32 * kXEpiWarps);
    }
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
  const int first_tile = (int)blockIdx.x >> (kPair ? 1 : 0);

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    const uint64_t pol = l2_policy_evict_normal();
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;
    bool ok = true;
    int asked = 0;
    int tile = first_tile;
    for (int j = 0; ok && tile >= 0; ++j) {
      if (leader) {
        if (!clc_ask<kPair>(clc, j + 1, p.wait, abort_flag)) {
          fail(kRoleProducer, abort_flag);
          break;
        }
        asked = j + 1;
      }
      const XentTileAt tc = xent_tile<T::kM>(p, n_rows, tile);
      if (tc.prob >= 0) {
        const XentProblem& q = p.prob[tc.prob];
        const CUtensorMap* ma = &maps.m[q.a_map];
        const CUtensorMap* mb = &maps.m[q.b_map];
        // this CTA's part of the tile: 128 rows of A, kBRows of B
        const int32_t m0 = tc.m0 + (kPair ? (int32_t)rank * 128 : 0) + q.a_off;
        const int32_t n0 = tc.n0 + (kPair ? (int32_t)rank * T::kBRows : 0) + (q.b_k ? 0 : q.b_off);
        for (int ks = 0; ks < tc.k_steps; ++ks) {
          if (!wait_bounded(empty0 + 8 * stage, phase ^ 1u, p.wait, abort_flag)) {
            fail(kRoleProducer, abort_flag);
            ok = false;
            break;
          }
          if (lane == 0 && !p.wait.starve_loads) {
            const uint32_t full = full0 + 8 * stage;
            const uint32_t sa = smem_u32(smem + (size_t)stage * T::kStageBytes);
            const uint32_t sb = sa + T::kABytes;
            const int32_t k = (tc.k0 + ks) * kBK;
            const int32_t kb = k + (q.b_k ? q.b_off : 0);
            if (leader) mbar_arrive_expect_tx(full, (kPair ? 2u : 1u) * T::kStageBytes);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int32_t mn = m0 + 64 * i;
              const int32_t x = q.a_mn ? mn : k, y = q.a_mn ? k : mn;
              if constexpr (kPair)
                tma_load_2d_pair(sa + i * kXBox, ma, full, tma_x((int64_t)x * 2, 2), y, pol);
              else
                tma_load_2d(sa + i * kXBox, ma, full, tma_x((int64_t)x * 2, 2), y, pol);
            }
#pragma unroll
            for (int i = 0; i < T::kBRows / 64; ++i) {
              const int32_t mn = n0 + 64 * i;
              const int32_t x = q.b_mn ? mn : kb, y = q.b_mn ? kb : mn;
              if constexpr (kPair)
                tma_load_2d_pair(sb + i * kXBox, mb, full, tma_x((int64_t)x * 2, 2), y, pol);
              else
                tma_load_2d(sb + i * kXBox, mb, full, tma_x((int64_t)x * 2, 2), y, pol);
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
      if (!ok) break;
      tile = clc_take<kPair>(clc, j + 1, p.wait, abort_flag, ok);
      if (!ok) fail(kRoleProducer, abort_flag);
    }
    // An answer asked for but not read (an error path) must still land before the CTA exits.
    if (leader && asked > 0) {
      const int slot = (asked - 1) % kClcSlots;
      const uint32_t ph = (uint32_t)((asked - 1) / kClcSlots) & 1u;
      if (!wait_bounded(clc.full0 + 8 * slot, ph, p.wait, nullptr)) fail(kRoleDrain, abort_flag);
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
    const uint32_t idesc0 = idesc_f16kind_f32(T::kM, kXN, !kF16);
    int stage = 0;
    uint32_t phase = 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    int tile = leader ? first_tile : -1;
    for (int tj = 0; ok && tile >= 0; ++tj) {
      const XentTileAt tc = xent_tile<T::kM>(p, n_rows, tile);
      if (tc.prob >= 0) {
        const XentProblem& q = p.prob[tc.prob];
        const uint32_t idesc = idesc0 | ((uint32_t)q.a_mn << 15) | ((uint32_t)q.b_mn << 16);
        // one K = 16 step further along: 32 bytes in a K-major tile, 16 rows in an MN-major one
        const uint64_t a_step = q.a_mn ? (16 * 128) >> 4 : 32 >> 4;
        const uint64_t b_step = q.b_mn ? (16 * 128) >> 4 : 32 >> 4;
        if (!wait_bounded(tempty0 + 8 * acc, acc_phase ^ 1u, p.wait, abort_flag)) {
          fail(kRoleMma, abort_flag);
          break;
        }
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * kXN);
        for (int ks = 0; ks < tc.k_steps; ++ks) {
          if (!wait_bounded(full0 + 8 * stage, phase, p.wait, abort_flag)) {
            fail(kRoleMma, abort_flag);
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t sa = smem_u32(smem + (size_t)stage * T::kStageBytes);
          const uint32_t sb = sa + T::kABytes;
          uint64_t ad = q.a_mn ? sdesc_mnmajor_sw128(sa) : sdesc_kmajor_sw128(sa);
          uint64_t bd = q.b_mn ? sdesc_mnmajor_sw128(sb) : sdesc_kmajor_sw128(sb);
#pragma unroll
          for (int i = 0; i < kBK / kUK; ++i) {
            if constexpr (kPair)
              mma_bf16_ss_pair_elect(d_tmem, ad, bd, idesc, (ks | i) != 0);
            else
              mma_bf16_ss_elect(d_tmem, ad, bd, idesc, (ks | i) != 0);
            ad += a_step;
            bd += b_step;
          }
          if constexpr (kPair)
            mma_commit_pair_elect(empty0 + 8 * stage, 0x3);
          else
            mma_commit_elect(empty0 + 8 * stage);
          __syncwarp();
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if constexpr (kPair)
          mma_commit_pair_elect(tfull0 + 8 * acc, 0x3);
        else
          mma_commit_elect(tfull0 + 8 * acc);
        __syncwarp();
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      tile = clc_take<kPair>(clc, tj + 1, p.wait, abort_flag, ok);
      if (!ok) fail(kRoleMma, abort_flag);
    }
    if (leader) {
      if constexpr (kPair)
        mma_commit_pair_elect(done_bar, 0x1);
      else
        mma_commit_elect(done_bar);
      __syncwarp();
      if (!wait_bounded(done_bar, 0, p.wait, nullptr)) fail(kRoleDrain, abort_flag);
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int quarter = warp & 3;      // TMEM lanes this warp may access
    const int half = (warp - 2) >> 2;  // which 128 of the tile's columns
    const XentStage st{smem_u32(staging + (warp - 2) * kXStoreBox)};
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    int tile = first_tile;
    for (int tj = 0; ok && tile >= 0; ++tj) {
      const XentTileAt tc = xent_tile<T::kM>(p, n_rows, tile);
      if (tc.prob >= 0) {
        const XentProblem& q = p.prob[tc.prob];
        if (!wait_bounded(tfull0 + 8 * acc, acc_phase, p.wait, abort_flag, kSleepHintNs)) {
          fail(kRoleEpilogue, abort_flag);
          break;
        }
        tc_fence_after_sync();
        const int32_t row0 = tc.m0 + (kPair ? (int32_t)rank * 128 : 0) + quarter * 32;
        const int32_t row = row0 + lane;
        const int32_t col = tc.n0 + half * kXChunk;
        const bool zero = tc.k_steps == 0;
        const uint32_t tacc = tmem_base + ((uint32_t)(quarter * 32) << 16) +
                              (uint32_t)(acc * kXN + half * kXChunk);
        if (q.kind == kXentStats)
          xent_epi_stats<kF16>(p, q, tacc, zero, row, row < n_rows, col);
        else if (q.kind == kXentDlogits)
          xent_epi_dlogits<kF16>(p, q, maps, st, tacc, zero, row0, row, row < n_rows, col);
        else if (q.kind == kXentDweight)
          xent_epi_dweight<kF16>(p, q, maps, st, tacc, zero, row0, row, col);
        else
          xent_epi_dhidden(p, q, tacc, zero, tc.split, row, row < n_rows, col);
        tc_fence_before_sync();
        if constexpr (kPair)
          mbar_arrive_remote(tempty0 + 8 * acc, 0);
        else
          mbar_arrive(tempty0 + 8 * acc);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      tile = clc_take<kPair>(clc, tj + 1, p.wait, abort_flag, ok);
      if (!ok) fail(kRoleEpilogue, abort_flag);
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
// block places 32 rows: it counts the rows that count before its own and in all (the targets are
// a few KB that sit in L2; a scan over blocks would be a launch of its own), then copies. The
// packed rows up to the next multiple of 64 are cleared: the weight gradient's product takes rows
// 64 at a time.
constexpr int kPackRows = 32, kPackThreads = 256;
__global__ void __launch_bounds__(kPackThreads)
    xent_pack_kernel(const uint4* __restrict__ hidden, const int32_t* __restrict__ targets,
                     int32_t rows, int32_t row_vecs, int32_t ignore, uint4* packed,
                     int32_t* packed_targets, int32_t* place, int32_t* row_of, int32_t* n_rows) {
  __shared__ int32_t s_before[kPackThreads / 32], s_all[kPackThreads / 32];
  __shared__ int32_t s_place[kPackRows];
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t r0 = (int32_t)blockIdx.x * kPackRows;
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
    const int32_t t = r < rows ? targets[r] : ignore;
    const bool counts = t != ignore;
    const uint32_t mask = __ballot_sync(0xffffffffu, counts);
    const int32_t at = before + __popc(mask & ((1u << lane) - 1u));
    s_place[lane] = counts ? at : -1;
    if (r < rows) place[r] = counts ? at : -1;
    if (counts) {
      row_of[at] = r;
      packed_targets[at] = t;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *n_rows = all;
  __syncthreads();
  for (int i = warp; i < kPackRows; i += kPackThreads / 32) {
    const int32_t at = s_place[i];
    if (at < 0) continue;
    const uint4* src = hidden + (int64_t)(r0 + i) * row_vecs;
    uint4* dst = packed + (int64_t)at * row_vecs;
    for (int32_t x = lane; x < row_vecs; x += 32) dst[x] = src[x];
  }
  const int32_t end = (all + kBK - 1) / kBK * kBK;
  for (int32_t r = all + (int32_t)blockIdx.x; r < end; r += (int32_t)gridDim.x)
    for (int32_t x = threadIdx.x; x < row_vecs; x += kPackThreads)
      packed[(int64_t)r * row_vecs + x] = make_uint4(0u, 0u, 0u, 0u);
}

// ------------------------------------------------------------------ the loss from the statistics

// Folds each row's (max, sum) pairs in a fixed order (32 segments of consecutive pairs, then the
// segments) into lse and the row's loss. A block of 32 warps serves 32 rows, lane i row i, so the
// reads of the pair arrays are 256 bytes wide. Ignored rows get 0 and 0; a target outside [0, V)
// makes the row's loss NaN.
__device__ __forceinline__ void xent_merge(float& m, float& s, float m2, float s2) {
  // NaN sums (a NaN or +inf logit) survive both branches: exp of a NaN difference is NaN
  const float nm = fmaxf(m, m2);
  const float ref = nm == -INFINITY ? 0.0f : nm;
  s = s * __expf(m - ref) + s2 * __expf(m2 - ref);
  m = nm;
}
constexpr int kFoldRows = 32;
__global__ void __launch_bounds__(1024)
    xent_fold_kernel(const float2* __restrict__ partials, int32_t n_chunks, int32_t pitch,
                     int32_t rows, int32_t V, const int32_t* __restrict__ place,
                     const int32_t* __restrict__ targets, const float* __restrict__ target_z,
                     float z_loss, float* row_loss, float* lse_out) {
  __shared__ float2 seg[32][kFoldRows + 1];
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t r = (int32_t)blockIdx.x * kFoldRows + lane;
  const int32_t at = r >= rows ? -1 : place != nullptr ? place[r] : r;
  const int per_seg = (n_chunks + 31) / 32;
  const int c0 = warp * per_seg, c1 = min(n_chunks, c0 + per_seg);
  float m = -INFINITY, s = 0.0f;
  if (at >= 0) {
    int c = c0;
    for (; c + 8 <= c1; c += 8) {
      float2 q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = __ldcs(partials + (int64_t)(c + i) * pitch + at);
#pragma unroll
      for (int i = 0; i < 8; ++i) xent_merge(m, s, q[i].x, q[i].y);
    }
    for (; c < c1; ++c) {
      const float2 q = __ldcs(partials + (int64_t)c * pitch + at);
      xent_merge(m, s, q.x, q.y);
    }
  }
  seg[warp][lane] = make_float2(m, s);
  __syncthreads();
  if (warp != 0 || r >= rows) return;
  if (at < 0) {
    row_loss[r] = 0.0f;
    lse_out[r] = 0.0f;
    return;
  }
  m = -INFINITY;
  s = 0.0f;
  for (int w = 0; w < 32; ++w) xent_merge(m, s, seg[w][lane].x, seg[w][lane].y);
  const float lse = m + logf(s);
  const int32_t t = targets[at];
  const float nll = t >= 0 && t < V ? lse - target_z[at] : __int_as_float(0x7fc00000);
  lse_out[r] = lse;
  row_loss[r] = z_loss != 0.0f ? nll + z_loss * lse * lse : nll;
}

// The rows' losses added in a fixed order (each of 1024 threads every 1024th row, then a tree),
// and divided by the number of rows that count (at least 1) for the mean.
__global__ void __launch_bounds__(1024)
    xent_reduce_kernel(const float* __restrict__ row_loss, int32_t rows,
                       const int32_t* __restrict__ n_rows, int32_t mean, float* loss) {
  __shared__ float part[32];
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();
  float s = 0.0f;
  for (int32_t r = threadIdx.x; r < rows; r += 1024) s += row_loss[r];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  s = part[threadIdx.x];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (threadIdx.x == 0) {
    const int32_t n = n_rows != nullptr ? *n_rows : rows;
    *loss = mean ? s / (float)max(n, 1) : s;
  }
}

// ------------------------------------------------------------------ factors of the gradient

// (lse, a, b, target) of every row that counts, and scale[1] = the factor of the gradients (see the
// top of this file). One block: the power of two needs the largest factor of all rows first, and
// the rows are a few thousand numbers. A target outside [0, V) makes its row NaN.
__global__ void __launch_bounds__(1024)
    xent_rows_kernel(const float* __restrict__ lse, const int32_t* __restrict__ targets,
                     const int32_t* __restrict__ row_of, int32_t rows,
                     const int32_t* __restrict__ n_rows, int32_t V,
                     const float* __restrict__ grad, int32_t per_row, int32_t mean, float z_loss,
                     float alpha, float4* row_info, float* scale) {
  __shared__ float part[32];
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();
  const int32_t n = n_rows != nullptr ? *n_rows : rows;
  auto factors = [&](int32_t i, float& l, float& a, float& b) {
    const int32_t r = row_of != nullptr ? row_of[i] : i;
    l = lse[r];
    b = per_row ? grad[r] : 1.0f;
    a = z_loss != 0.0f ? b * (1.0f + 2.0f * z_loss * l) : b;
  };
  float top = 0.0f;
  for (int32_t i = threadIdx.x; i < n; i += 1024) {
    float l, a, b;
    factors(i, l, a, b);
    if (fabsf(a) < INFINITY) top = fmaxf(top, fabsf(a));  // (false for NaN)
    if (fabsf(b) < INFINITY) top = fmaxf(top, fabsf(b));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
  __syncthreads();
  top = part[threadIdx.x & 31];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int k = top > 0.0f ? min(100, max(-100, 13 - ilogbf(top))) : 0;
  const float up = ldexpf(1.0f, k), down = ldexpf(1.0f, -k);
  for (int32_t i = threadIdx.x; i < n; i += 1024) {
    float l, a, b;
    factors(i, l, a, b);
    const int32_t t = targets[i];
    if (t < 0 || t >= V) a = b = __int_as_float(0x7fc00000);
    row_info[i] = make_float4(l, a * up, b * up, __int_as_float(t));
  }
  if (threadIdx.x == 0) {
    float f = alpha;
    if (!per_row) f *= mean ? *grad / (float)max(n, 1) : *grad;
    scale[0] = up;
    scale[1] = f * down;
  }
}

// dH from its partial sums: the splits in order, times the factor, rounded once; ignored rows 0.
// A thread takes 8 entries of a row.
constexpr int kFinishThreads = 256;
template <bool kF16>
__global__ void __launch_bounds__(kFinishThreads)
    xent_finish_hidden_kernel(const float* __restrict__ partial, int32_t splits, int64_t split_len,
                              int32_t rows, int32_t H, const int32_t* __restrict__ place,
                              const float* __restrict__ scale, uint4* d_hidden) {
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();
  const int64_t i = (int64_t)blockIdx.x * kFinishThreads + threadIdx.x;
  const int32_t vecs = H / 8;
  if (i >= (int64_t)rows * vecs) return;
  const int32_t r = (int32_t)(i / vecs), x = (int32_t)(i - (int64_t)r * vecs) * 8;
  const int32_t at = place != nullptr ? place[r] : r;
  uint4 out = make_uint4(0u, 0u, 0u, 0u);
  if (at >= 0) {
    const float f = scale[1];
    float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    const float* src = partial + (int64_t)at * H + x;
    for (int32_t k = 0; k < splits; ++k) {
      const float4 u = __ldcs(reinterpret_cast<const float4*>(src + k * split_len));
      const float4 v = __ldcs(reinterpret_cast<const float4*>(src + k * split_len) + 1);
      s[0] += u.x;
      s[1] += u.y;
      s[2] += u.z;
      s[3] += u.w;
      s[4] += v.x;
      s[5] += v.y;
      s[6] += v.z;
      s[7] += v.w;
    }
    out.x = pack16<kF16>(s[0] * f, s[1] * f);
    out.y = pack16<kF16>(s[2] * f, s[3] * f);
    out.z = pack16<kF16>(s[4] * f, s[5] * f);
    out.w = pack16<kF16>(s[6] * f, s[7] * f);
  }
  d_hidden[i] = out;
}

// dbias of a piece: the columns of d summed over the rows that count, in fp32. A block takes 64
// columns: 8 threads of 8 columns by 32 row lanes (each every 32nd row), then the lanes in order.
constexpr int kBiasCols = 64;
template <bool kF16>
__global__ void __launch_bounds__(256)
    xent_bias_kernel(const uint16_t* __restrict__ d, int32_t ld, int32_t cols, int32_t rows,
                     const int32_t* __restrict__ n_rows, const float* __restrict__ scale,
                     int32_t add, uint16_t* d_bias) {
  __shared__ float part[32][kBiasCols + 1];
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();
  const int32_t n = n_rows != nullptr ? *n_rows : rows;
  const int32_t cg = threadIdx.x & 7, rl = threadIdx.x >> 3;
  const int32_t c0 = (int32_t)blockIdx.x * kBiasCols;
  float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  // (a 64-column panel of d is whole in the buffer wherever one of its columns is)
  const uint16_t* src = d + c0 + cg * 8;
#pragma unroll 8
  for (int32_t r = rl; r < n; r += 32) {
    const uint4 q = *reinterpret_cast<const uint4*>(src + (int64_t)r * ld);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[2 * i] += unpack16<kF16>(w[i] & 0xffffu);
      s[2 * i + 1] += unpack16<kF16>(w[i] >> 16);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) part[rl][cg * 8 + i] = s[i];
  __syncthreads();
  if (threadIdx.x < kBiasCols && c0 + (int32_t)threadIdx.x < cols) {
    float t = 0.0f;
    for (int i = 0; i < 32; ++i) t += part[i][threadIdx.x];
    t = n > 0 ? t * scale[1] : 0.0f;
    uint16_t* at = d_bias + c0 + threadIdx.x;
    if (add) t += unpack16<kF16>(*at);
    *at = (uint16_t)(pack16<kF16>(t, 0.0f) & 0xffffu);
  }
}

}  // namespace lmh
