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
//      sort is a few KB a pass and bound by latency, so the other CTAs of the launch write the
//      table's zeros in the meantime, which is most of the bytes.
//   2. embed_sum_kernel: blocks take `tile` sorted entries by 512 columns. A run (the entries of one
//      id) inside a tile is summed and written; the parts of a run that crosses tiles go to fp32
//      partial rows. So one id that fills the batch is summed by as many blocks as any other batch.
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
    embed_kernel(const int32_t* __restrict__ ids, int64_t tokens, int32_t v_begin, int32_t V,
                 const uint4* __restrict__ W, int32_t row_vecs, int32_t pieces, float scale,
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
    q[i] = held && x < row_vecs ? __ldg(src + x) : make_uint4(0u, 0u, 0u, 0u);
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

struct EmbedSortParams {
  const int32_t* ids;
  int32_t tokens, v_begin, V;
  int32_t passes, bits;       // digits of `bits` bits; passes * bits hold V, the mark of an absent id
  int32_t* keys[2];           // [tokens] each; the last pass writes keys[(passes - 1) & 1]
  int32_t* pos[2];
  int32_t* hist;              // [passes][kSortCtas][kSortDigits]
  uint4* zero;                // dW as 16-byte pieces, or null
  int64_t zero_vecs;
};

// Cluster 0 sorts; the other clusters, if any, write zeros. keys are id - v_begin, or V for an id
// outside the table, so those sort behind all others. Each CTA owns an eighth of the entries of a
// pass: it counts its digits, learns the other CTAs' counts, and places its entries 1024 at a time:
// an entry's place is its digit's start, plus the entries of that digit before it in the CTA's
// earlier tiles, in earlier warps (a count for each warp and digit), and in earlier lanes
// (__match_any_sync). Entries written in one pass are read in the next past the L1 (ld.cg).
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const EmbedSortParams p) {
  __shared__ uint16_t s_warp[32][kSortDigits];
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
  const uint32_t mask = (1u << p.bits) - 1u;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits;
    const int32_t* keys = p.keys[(pass + 1) & 1];
    const int32_t* pos = p.pos[(pass + 1) & 1];
    int32_t* to_keys = p.keys[pass & 1];
    int32_t* to_pos = p.pos[pass & 1];
    auto key_at = [&](int32_t i) {
      if (pass > 0) return __ldcg(keys + i);
      const int64_t v = (int64_t)p.ids[i] - p.v_begin;
      return v >= 0 && v < p.V ? (int32_t)v : p.V;
    };
    if (tid < kSortDigits) s_count[tid] = 0;
    __syncthreads();
    for (int32_t i = begin + tid; i < end; i += kSortThreads)
      atomicAdd(&s_count[((uint32_t)key_at(i) >> shift) & mask], 1);
    __syncthreads();
    int32_t* hist = p.hist + pass * kSortCtas * kSortDigits;
    if (tid < kSortDigits) __stcg(hist + cta * kSortDigits + tid, s_count[tid]);
    cluster_sync_all();
    // digit `tid`: entries of it in all CTAs, in the CTAs before this one, and of smaller digits
    int32_t all = 0, before = 0;
    if (tid < kSortDigits) {
#pragma unroll
      for (int c = 0; c < kSortCtas; ++c) {
        const int32_t n = __ldcg(hist + c * kSortDigits + tid);
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
    for (int32_t i0 = begin; i0 < end; i0 += kSortThreads) {
      uint4* clear = reinterpret_cast<uint4*>(&s_warp[0][0]);
      for (int j = tid; j < (int)sizeof(s_warp) / 16; j += kSortThreads)
        clear[j] = make_uint4(0u, 0u, 0u, 0u);
      __syncthreads();
      const int32_t i = i0 + tid;
      const bool mine = i < end;
      const int32_t key = mine ? key_at(i) : 0;
      const int32_t from = !mine ? 0 : pass > 0 ? __ldcg(pos + i) : i;
      const uint32_t digit = mine ? ((uint32_t)key >> shift) & mask : 0xffffffffu;
      const uint32_t peers = __match_any_sync(0xffffffffu, digit);
      const int32_t rank = __popc(peers & ((1u << lane) - 1u));
      if (mine && rank == 0) s_warp[warp][digit] = (uint16_t)__popc(peers);
      __syncthreads();
      // per digit: each warp's first place, and the start of the next tile's
      if (tid < kSortDigits) {
        int32_t at = 0;
#pragma unroll 8
        for (int w = 0; w < 32; ++w) {
          const int32_t n = s_warp[w][tid];
          s_warp[w][tid] = (uint16_t)at;
          at += n;
        }
        s_count[tid] = s_base[tid];
        s_base[tid] += at;
      }
      __syncthreads();
      if (mine) {
        const int32_t at = s_count[digit] + s_warp[warp][digit] + rank;
        __stcg(to_keys + at, key);
        __stcg(to_pos + at, from);
      }
      __syncthreads();
    }
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
};

constexpr int kSumThreads = 128, kSumCols = 4 * kSumThreads, kSumTileMax = 1024, kSumBatch = 8;

template <bool kF16>
__device__ __forceinline__ void embed_add4(float (&a)[4], uint2 q) {
  a[0] += unpack16<kF16>(q.x & 0xffffu);
  a[1] += unpack16<kF16>(q.x >> 16);
  a[2] += unpack16<kF16>(q.y & 0xffffu);
  a[3] += unpack16<kF16>(q.y >> 16);
}

template <bool kF16>
__device__ __forceinline__ void embed_write(const EmbedSumParams& p, int32_t v, int32_t x,
                                            float (&a)[4]) {
  uint2* at = reinterpret_cast<uint2*>(p.d_weight + (int64_t)v * p.H + x);
#pragma unroll
  for (int j = 0; j < 4; ++j) a[j] *= p.scale;
  if (p.add) embed_add4<kF16>(a, *at);
  *at = make_uint2(pack16<kF16>(a[0], a[1]), pack16<kF16>(a[2], a[3]));
}

template <bool kF16>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const EmbedSumParams p) {
  __shared__ int32_t s_key[kSumTileMax + 1], s_pos[kSumTileMax];
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();
  const int32_t e0 = (int32_t)blockIdx.x * p.tile;
  const int32_t n_all = min(p.tile, p.tokens - e0);
  for (int i = threadIdx.x; i < n_all; i += kSumThreads) {
    s_key[i] = p.keys[e0 + i];
    s_pos[i] = p.pos[e0 + i];
  }
  if (threadIdx.x == 0) s_key[n_all] = e0 + n_all < p.tokens ? p.keys[e0 + n_all] : -1;
  const int32_t earlier = e0 > 0 ? p.keys[e0 - 1] : -1;
  __syncthreads();
  const int32_t x = (int32_t)blockIdx.y * kSumCols + (int)threadIdx.x * 4;
  if (x >= p.H) return;
  bool began_earlier = earlier == s_key[0];
  float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  float* part = p.part + (int64_t)blockIdx.x * 2 * p.H + x;
  const uint16_t* src = p.d_out + x;
  bool open = false;
  for (int e = 0; e < n_all && s_key[e] < p.V; e += kSumBatch) {
    uint2 q[kSumBatch];
#pragma unroll
    for (int i = 0; i < kSumBatch; ++i) {
      const int k = e + i;
      q[i] = k < n_all && s_key[k] < p.V
                 ? __ldcs(reinterpret_cast<const uint2*>(src + (int64_t)s_pos[k] * p.H))
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
        embed_write<kF16>(p, s_key[k], x, a);
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
// are the tile's second partial row and the first of each later tile up to the run's end.
template <bool kF16>
__global__ void __launch_bounds__(kSumThreads) embed_join_kernel(const EmbedSumParams p) {
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();
  const int32_t tiles = (p.tokens + p.tile - 1) / p.tile;
  const int32_t i = (int32_t)blockIdx.x;
  const int32_t next = (i + 1) * p.tile;
  if (next >= p.tokens) return;
  const int32_t key = p.keys[next];
  if (key >= p.V || p.keys[next - 1] != key) return;
  if (i > 0 && p.keys[i * p.tile] == key && p.keys[i * p.tile - 1] == key) return;
  // the last tile that the run reaches: the first whose successor begins with another key
  __shared__ int32_t s_last;
  if (threadIdx.x == 0) s_last = tiles - 1;
  __syncthreads();
  for (int32_t j0 = i + 1; j0 < tiles; j0 += kSumThreads) {
    const int32_t j = j0 + (int)threadIdx.x;
    const bool ends = j < tiles && ((int64_t)(j + 1) * p.tile >= p.tokens ||
                                    p.keys[(j + 1) * p.tile] != key);
    if (ends) atomicMin(&s_last, j);
    if (__syncthreads_or(ends)) break;
  }
  const int32_t last = s_last;
  const int32_t x = (int32_t)blockIdx.y * kSumCols + (int)threadIdx.x * 4;
  if (x >= p.H) return;
  const float* src = p.part + x;
  const float4 first = *reinterpret_cast<const float4*>(src + ((int64_t)i * 2 + 1) * p.H);
  float a[4] = {first.x, first.y, first.z, first.w};
#pragma unroll 8
  for (int32_t j = i + 1; j <= last; ++j) {
    const float4 q = __ldcs(reinterpret_cast<const float4*>(src + (int64_t)j * 2 * p.H));
    a[0] += q.x;
    a[1] += q.y;
    a[2] += q.z;
    a[3] += q.w;
  }
  embed_write<kF16>(p, key, x, a);
}

}  // namespace lmh
