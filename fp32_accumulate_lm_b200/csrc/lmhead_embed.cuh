// Token embedding and its gradient.
//
//   out[t] = scale * W[id_t]                                    (0 for an id outside the table)
//   dW[v]  = scale * sum over {t : id_t = v} of d_out[t]        (in order of t, fp32)
//
// The forward pass is a gather: T rows of H read and written once, bound by memory.
//
// The gradient is bound by memory as well: d_out is read once, and dW is written whole (or, when it
// accumulates, only the rows that occur are read and written). Adding rows with atomics would make
// the sums' order change from run to run, and would need an fp32 table; so the tokens are sorted by
// id, stably, and each row's tokens are summed in order by one thread per four columns:
//   1. embed_sort_kernel: one cluster of 8 CTAs sorts (id, position) by a least-significant-digit
//      radix sort of 9 bits a pass, its passes separated by cluster barriers, in one launch. The
//      sort is a few KB a pass and bound by latency, so the launch's other CTAs write zeros to the
//      table's first rows in the meantime: as many bytes as fit in about its time.
//   2. embed_sum_kernel: blocks take `tile` sorted entries by 512 columns. A run (the entries of one
//      id) inside a tile is summed and written; the parts of a run that crosses tiles go to fp32
//      partial rows. So one id that fills the batch is summed by as many blocks as any other batch.
//      The launch's other blocks write the rest of the zeros, to rows that the sort's bitmap says
//      have no token, beside the sums and not before them.
//   3. embed_join_kernel: adds each crossing run's partial rows, in order, and writes its row.
#pragma once

#include "lmhead_xent.cuh"

namespace lmh {

// ------------------------------------------------------------------ forward

// A warp takes 128 16-byte pieces (1024 elements) of one token's row, four per lane, all of them
// loaded before the first is stored.
constexpr int kEmbedVecs = 128, kEmbedThreads = 256;
template <bool kF16>
__global__ void __launch_bounds__(kEmbedThreads)
    embed_kernel(const int32_t* ids, int64_t tokens, int32_t v_begin, int32_t V,
                 const uint4* W, int32_t row_vecs, int32_t pieces, float scale,
                 uint4* out) {
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();
  const int64_t w = (int64_t)blockIdx.x * (kEmbedThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = w / pieces;
  if (t >= tokens) return;
  const int32_t x0 = (int32_t)(w - t * pieces) * kEmbedVecs + (int)(threadIdx.x & 31);
  const int64_t v = (int64_t)ids[t] - v_begin;
  const bool held = v >= 0 && v < V;
  const uint4* src = W + (held ? v : 0) * row_vecs;
  uint4 q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int32_t x = x0 + 32 * i;
    q[i] = held && x < row_vecs ? src[x] : make_uint4(0u, 0u, 0u, 0u);
  }
  uint4* dst = out + t * row_vecs;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int32_t x = x0 + 32 * i;
    uint32_t u[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
    if (held) {  // (an absent row stays 0 whatever the scale)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        u[j] = pack16<kF16>(unpack16<kF16>(u[j] & 0xffffu) * scale,
                            unpack16<kF16>(u[j] >> 16) * scale);
    }
    if (x < row_vecs) dst[x] = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// ------------------------------------------------------------------ sort by id

constexpr int kSortCtas = 8;         // one portable cluster
constexpr int kSortThreads = 1024;
constexpr int kSortBits = 9;         // digits of at most 9 bits: two passes up to 262143 ids
constexpr int kSortDigits = 1 << kSortBits;
constexpr int kSortMaxPasses = 4;    // 2^30 ids and the mark for none

constexpr int kSortItems = 8;        // entries a thread holds at once

struct EmbedSortParams {
  const int32_t* ids;
  int32_t tokens, v_begin, V;
  int32_t passes, bits;       // digits of `bits` bits; passes * bits hold V, the mark of an absent id
  int32_t* keys[2];           // [tokens] each; the last pass writes keys[(passes - 1) & 1]
  int32_t* pos[2];
  uint4* zero;                // dW's first rows as 16-byte pieces, or null
  int64_t zero_vecs;
  uint32_t* seen;             // [(V + 31) / 32] bits of the rows with a token, or null
};

// Cluster 0 sorts; the other clusters, if any, write zeros. keys are id - v_begin, or V for an id
// outside the table, so those sort behind all others. Each CTA owns an eighth of the entries of a
// pass, and takes them up to 8192 at a time, each warp a consecutive part: an entry's place is its
// digit's start (from the counts of all CTAs, read out of their shared memory), plus the entries of
// that digit before it in the CTA's earlier turns, in earlier warps (a count for each warp and
// digit), and in its own warp (32 at a time, by __match_any_sync). Where a CTA's entries fit one
// turn, at most 65536 tokens in all, the counts come out of the ranking and the entries are read
// once a pass; else they are counted first. Entries written in one pass are read in the next past
// the L1 (ld.cg). A first form, 1024 entries a turn with a scan of the 32 warps' counts each time,
// took 35 us for 16384 tokens and 130 us for 65536.
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const EmbedSortParams p) {
  __shared__ __align__(16) uint16_t s_warp[32][kSortDigits];
  __shared__ int32_t s_count[kSortDigits];
  __shared__ int32_t s_base[kSortDigits];
  __shared__ int32_t s_scan[kSortDigits / 32];
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (blockIdx.x >= kSortCtas) {
    const int64_t stride = (int64_t)(gridDim.x - kSortCtas) * kSortThreads;
    for (int64_t i = (int64_t)(blockIdx.x - kSortCtas) * kSortThreads + tid; i < p.zero_vecs;
         i += stride)
      p.zero[i] = make_uint4(0u, 0u, 0u, 0u);
    return;  // (whole clusters: nobody waits for these CTAs)
  }
  const int cta = (int)blockIdx.x;
  const int32_t per = ((p.tokens + kSortCtas - 1) / kSortCtas + 31) / 32 * 32;
  const int32_t begin = min(p.tokens, cta * per), end = min(p.tokens, begin + per);
  // entries a thread takes in a turn: no more than spread a CTA's entries over its threads
  const int32_t items = min(kSortItems, (per + kSortThreads - 1) / kSortThreads);
  const int32_t turn = items * kSortThreads;
  const bool single = per <= turn;
  const uint32_t mask = (1u << p.bits) - 1u;
  if (p.seen != nullptr)  // set behind the first cluster barrier
    for (int32_t i = cta * kSortThreads + tid; i < (p.V + 31) / 32; i += kSortCtas * kSortThreads)
      p.seen[i] = 0u;

  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits;
    const int32_t* keys = pass & 1 ? p.keys[0] : p.keys[1];
    const int32_t* pos = pass & 1 ? p.pos[0] : p.pos[1];
    int32_t* to_keys = pass & 1 ? p.keys[1] : p.keys[0];
    int32_t* to_pos = pass & 1 ? p.pos[1] : p.pos[0];
    auto key_at = [&](int32_t i) {
      if (pass > 0) return load_cg(keys + i);
      const int64_t v = (int64_t)p.ids[i] - p.v_begin;
      return v >= 0 && v < p.V ? (int32_t)v : p.V;
    };
    int32_t key[kSortItems], from[kSortItems];
    uint16_t rank[kSortItems];
    // this thread's entries of the turn at i0, and each one's rank among its digit's in the warp
    auto load = [&](int32_t i0) {
#pragma unroll
      for (int k = 0; k < kSortItems; ++k) {
        const int32_t i = i0 + warp * (items * 32) + k * 32 + lane;
        const bool mine = k < items && i < end;
        key[k] = mine ? key_at(i) : -1;
        from[k] = !mine ? 0 : pass > 0 ? load_cg(pos + i) : i;
      }
    };
    auto place = [&]() {
      uint4* clear = reinterpret_cast<uint4*>(&s_warp[warp][0]);
#pragma unroll
      for (int j = 0; j < (int)sizeof(s_warp[0]) / (16 * 32); ++j)
        clear[j * 32 + lane] = make_uint4(0u, 0u, 0u, 0u);
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kSortItems; ++k) {
        if (k >= items) break;  // (the same for all)
        const uint32_t digit = key[k] >= 0 ? ((uint32_t)key[k] >> shift) & mask : 0xffffffffu;
        const uint32_t peers = __match_any_sync(0xffffffffu, digit);
        const int32_t before = __popc(peers & ((1u << lane) - 1u));
        const int32_t first = key[k] >= 0 ? s_warp[warp][digit] : 0;
        rank[k] = (uint16_t)(first + before);
        __syncwarp();
        if (key[k] >= 0 && before == 0) s_warp[warp][digit] = (uint16_t)(first + __popc(peers));
        __syncwarp();
      }
    };
    // digit `tid`: each warp's first place among the turn's entries of the digit; their number
    auto scan_warps = [&]() {
      int32_t at = 0;
#pragma unroll 8
      for (int w = 0; w < 32; ++w) {
        const int32_t n = s_warp[w][tid];
        s_warp[w][tid] = (uint16_t)at;
        at += n;
      }
      return at;
    };
    auto scatter = [&](const int32_t* start) {
#pragma unroll
      for (int k = 0; k < kSortItems; ++k) {
        if (key[k] < 0) continue;
        const uint32_t digit = ((uint32_t)key[k] >> shift) & mask;
        const int32_t at = start[digit] + s_warp[warp][digit] + rank[k];
        __stcg(to_keys + at, key[k]);
        __stcg(to_pos + at, from[k]);
        if (pass == 0 && p.seen != nullptr && key[k] < p.V)
          atomicOr(p.seen + (key[k] >> 5), 1u << (key[k] & 31));
      }
    };
    if (single) {
      load(begin);
      place();
      __syncthreads();
      if (tid < kSortDigits) s_count[tid] = scan_warps();
    } else {
      if (tid < kSortDigits) s_count[tid] = 0;
      __syncthreads();
      for (int32_t i = begin + tid; i < end; i += kSortThreads)
        atomicAdd(&s_count[((uint32_t)key_at(i) >> shift) & mask], 1);
    }
    cluster_sync_all();
    // digit `tid`: entries of it in all CTAs, in the CTAs before this one, and of smaller digits
    int32_t all = 0, before = 0;
    if (tid < kSortDigits) {
#pragma unroll
      for (int c = 0; c < kSortCtas; ++c) {
        const int32_t n = cluster_load(&s_count[tid], (uint32_t)c);
        all += n;
        if (c < cta) before += n;
      }
    }
    int32_t upto = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t n = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += n;
    }
    if (tid < kSortDigits && lane == 31) s_scan[warp] = upto;
    __syncthreads();
    if (tid < kSortDigits) {
      int32_t start = upto - all + before;
      for (int w = 0; w < warp; ++w) start += s_scan[w];
      s_base[tid] = start;
    }
    __syncthreads();
    if (single) {
      scatter(s_base);
    } else {
      for (int32_t i0 = begin; i0 < end; i0 += turn) {
        load(i0);
        place();
        __syncthreads();
        int32_t n = 0;
        if (tid < kSortDigits) n = scan_warps();
        __syncthreads();
        scatter(s_base);
        __syncthreads();
        if (tid < kSortDigits) s_base[tid] += n;
      }
    }
    // the entries are placed, and no CTA reads this one's counts any more
    cluster_sync_all();
  }
}

// ------------------------------------------------------------------ sums over runs

struct EmbedSumParams {
  const int32_t* keys;   // sorted; V marks the entries without a row, behind all others
  const int32_t* pos;
  int32_t tokens, V, H;
  int32_t tile;          // sorted entries a block takes
  const uint16_t* d_out;
  float scale;
  int32_t add;
  uint16_t* d_weight;
  float* part;           // [tiles][2][H]: a run that began earlier, a run that goes on
  int32_t sum_blocks;    // tiles times slices of 512 columns; blocks behind them write zeros
  int32_t slices;
  const uint32_t* seen;  // bits of the rows with a token
  int32_t zero_from;     // first row to write zeros to
  int32_t zero_rows;     // rows a block
};

constexpr int kSumThreads = 128, kSumCols = 4 * kSumThreads, kSumTileMax = 1024, kSumBatch = 8;
constexpr int kSumTileMin = 8, kZeroVecs = 4096;  // 64 KB of zeros a block

// Zeros to this block's rows, but for those with a token.
__device__ __forceinline__ void embed_zero_rows(const EmbedSumParams& p, int32_t block) {
  const int32_t r0 = p.zero_from + block * p.zero_rows;
  const int32_t n = min(p.zero_rows, p.V - r0);
  const int32_t row_vecs = p.H / 8;
  uint4* dst = reinterpret_cast<uint4*>(p.d_weight) + (int64_t)r0 * row_vecs;
  for (int32_t i = threadIdx.x; i < n * row_vecs; i += kSumThreads) {
    const int32_t r = r0 + i / row_vecs;
    if (!((p.seen[r >> 5] >> (r & 31)) & 1u)) dst[i] = make_uint4(0u, 0u, 0u, 0u);
  }
}

template <bool kF16>
__device__ __forceinline__ void embed_add4(float (&a)[4], uint2 q) {
  a[0] += unpack16<kF16>(q.x & 0xffffu);
  a[1] += unpack16<kF16>(q.x >> 16);
  a[2] += unpack16<kF16>(q.y & 0xffffu);
  a[3] += unpack16<kF16>(q.y >> 16);
}

__device__ __forceinline__ uint2* embed_row(const EmbedSumParams& p, int32_t v, int32_t x) {
  return reinterpret_cast<uint2*>(p.d_weight + (int64_t)v * p.H + x);
}

// Row v's four columns: the sum times the scale, plus `old` where it accumulates, rounded once.
template <bool kF16>
__device__ __forceinline__ void embed_write(const EmbedSumParams& p, int32_t v, int32_t x,
                                            float (&a)[4], uint2 old) {
#pragma unroll
  for (int j = 0; j < 4; ++j) a[j] *= p.scale;
  if (p.add) embed_add4<kF16>(a, old);
  *embed_row(p, v, x) = make_uint2(pack16<kF16>(a[0], a[1]), pack16<kF16>(a[2], a[3]));
}

template <bool kF16>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const EmbedSumParams p) {
  __shared__ int32_t s_key[kSumTileMax + 1], s_pos[kSumTileMax];
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();
  if ((int32_t)blockIdx.x >= p.sum_blocks) {
    embed_zero_rows(p, (int32_t)blockIdx.x - p.sum_blocks);
    return;
  }
  const int32_t tile = (int32_t)blockIdx.x / p.slices;
  const int32_t e0 = tile * p.tile;
  const int32_t n_all = min(p.tile, p.tokens - e0);
  for (int i = threadIdx.x; i < n_all; i += kSumThreads) {
    s_key[i] = p.keys[e0 + i];
    s_pos[i] = p.pos[e0 + i];
  }
  if (threadIdx.x == 0) s_key[n_all] = e0 + n_all < p.tokens ? p.keys[e0 + n_all] : -1;
  const int32_t earlier = e0 > 0 ? p.keys[e0 - 1] : -1;
  __syncthreads();
  const int32_t x = ((int32_t)blockIdx.x - tile * p.slices) * kSumCols + (int)threadIdx.x * 4;
  if (x >= p.H) return;
  bool began_earlier = earlier == s_key[0];
  float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  float* part = p.part + (int64_t)tile * 2 * p.H + x;
  const uint16_t* src = p.d_out + x;
  bool open = false;
  for (int e = 0; e < n_all && s_key[e] < p.V; e += kSumBatch) {
    uint2 q[kSumBatch], old[kSumBatch];
#pragma unroll
    for (int i = 0; i < kSumBatch; ++i) {
      const int k = e + i;
      const bool used = k < n_all && s_key[k] < p.V;
      q[i] = used ? load_cs(reinterpret_cast<const uint2*>(src + (int64_t)s_pos[k] * p.H))
                  : make_uint2(0u, 0u);
      // what the row of a run that ends here holds, on its way with the rest
      old[i] = p.add && used && s_key[k + 1] != s_key[k] ? *embed_row(p, s_key[k], x)
                                                         : make_uint2(0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kSumBatch; ++i) {
      const int k = e + i;
      if (k >= n_all || s_key[k] >= p.V) break;
      embed_add4<kF16>(a, q[i]);
      open = true;
      if (s_key[k + 1] == s_key[k]) continue;
      // the run ends here
      if (began_earlier)
        *reinterpret_cast<float4*>(part) = make_float4(a[0], a[1], a[2], a[3]);
      else
        embed_write<kF16>(p, s_key[k], x, a, old[i]);
      began_earlier = false;
      open = false;
      a[0] = a[1] = a[2] = a[3] = 0.0f;
    }
  }
  // a run that goes on in the next tile: the first half if it also began earlier
  if (open)
    *reinterpret_cast<float4*>(part + (began_earlier ? 0 : p.H)) =
        make_float4(a[0], a[1], a[2], a[3]);
}

// A block looks at the end of one tile: if a run begins in the tile and goes on behind it, its parts
// are the tile's second partial row and the first of each later tile up to the run's end. Four
// groups of threads add a quarter of the later parts each, in order, and the quarters are added in
// order.
constexpr int kJoinGroups = 4;
template <bool kF16>
__global__ void __launch_bounds__(kJoinGroups* kSumThreads)
    embed_join_kernel(const EmbedSumParams p) {
  __shared__ int32_t s_last;
  __shared__ float4 s_part[kJoinGroups - 1][kSumThreads];
  if (threadIdx.x == 0) {
    pdl_trigger();
    s_last = 0x7fffffff;
  }
  pdl_wait();
  const int32_t tiles = (p.tokens + p.tile - 1) / p.tile;
  const int32_t i = (int32_t)blockIdx.x;
  const int32_t next = (i + 1) * p.tile;
  if (next >= p.tokens) return;
  const int32_t key = p.keys[next];
  if (key >= p.V || p.keys[next - 1] != key) return;
  if (i > 0 && p.keys[i * p.tile] == key && p.keys[i * p.tile - 1] == key) return;
  __syncthreads();
  // the last tile that the run reaches: the first whose successor begins with another key
  for (int32_t j0 = i + 1; j0 < tiles; j0 += (int)blockDim.x) {
    const int32_t j = j0 + (int)threadIdx.x;
    const bool ends = j < tiles && ((int64_t)(j + 1) * p.tile >= p.tokens ||
                                    p.keys[(j + 1) * p.tile] != key);
    if (ends) atomicMin(&s_last, j);
    if (__syncthreads_or(ends)) break;
  }
  const int32_t last = s_last;  // (the last tile of all ends every run)
  const int group = (int)threadIdx.x / kSumThreads, col = (int)threadIdx.x % kSumThreads;
  const int32_t x = (int32_t)blockIdx.y * kSumCols + col * 4;
  float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const float* src = p.part + x;
  if (x < p.H) {
    if (group == 0) {
      const float4 q = *reinterpret_cast<const float4*>(src + ((int64_t)i * 2 + 1) * p.H);
      a[0] = q.x;
      a[1] = q.y;
      a[2] = q.z;
      a[3] = q.w;
    }
    const int32_t n = last - i;  // later parts
    const int32_t j0 = i + 1 + (int32_t)((int64_t)n * group / kJoinGroups);
    const int32_t j1 = i + 1 + (int32_t)((int64_t)n * (group + 1) / kJoinGroups);
#pragma unroll 8
    for (int32_t j = j0; j < j1; ++j) {
      const float4 q = load_cs(reinterpret_cast<const float4*>(src + (int64_t)j * 2 * p.H));
      a[0] += q.x;
      a[1] += q.y;
      a[2] += q.z;
      a[3] += q.w;
    }
    if (group > 0) s_part[group - 1][col] = make_float4(a[0], a[1], a[2], a[3]);
  }
  __syncthreads();
  if (group > 0 || x >= p.H) return;
#pragma unroll
  for (int g = 0; g < kJoinGroups - 1; ++g) {
    const float4 q = s_part[g][col];
    a[0] += q.x;
    a[1] += q.y;
    a[2] += q.z;
    a[3] += q.w;
  }
  embed_write<kF16>(p, key, x, a, p.add ? *embed_row(p, key, x) : make_uint2(0u, 0u));
}

}  // namespace lmh
