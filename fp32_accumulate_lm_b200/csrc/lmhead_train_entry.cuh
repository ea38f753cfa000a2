// Host side of the training entry points (declared in include/lmhead.h): argument checks, the
// division of the work, the workspaces and the launches. Included at the end of lmhead.cu, whose
// helpers (device set-up, tensor maps, launches) it uses.
#pragma once

namespace {

constexpr int64_t kTrainMax = (int64_t)1 << 30;  // sizes below this leave room for rounding up

int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

// Hands out 256-byte aligned parts of a workspace; with a null base it only counts.
struct Carver {
  uint8_t* base;
  int64_t used = 0;
  explicit Carver(void* b) : base(reinterpret_cast<uint8_t*>(b)) {}
  template <typename T>
  T* take(int64_t count) {
    T* p = base != nullptr ? reinterpret_cast<T*>(base + used) : nullptr;
    used += round_up(count * (int64_t)sizeof(T), 256);
    return p;
  }
};

struct Region {
  const void* p;
  int64_t bytes;
};

// LMHEAD_ERR_ALIAS if an output overlaps another output or an input (null regions are skipped).
int check_overlap(const Region* in, int n_in, const Region* out, int n_out) {
  for (int i = 0; i < n_out; ++i) {
    if (out[i].p == nullptr || out[i].bytes == 0) continue;
    for (int j = 0; j < n_in; ++j)
      if (in[j].p != nullptr && in[j].bytes > 0 &&
          overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes))
        return LMHEAD_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (out[j].p != nullptr && out[j].bytes > 0 &&
          overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
        return LMHEAD_ERR_ALIAS;
  }
  return LMHEAD_OK;
}

// ---------------------------------------------------------------- cross entropy

// The rows that count, side by side (only where a target can be ignored).
struct XentPack {
  uint4* hidden = nullptr;
  int32_t *targets = nullptr, *place = nullptr, *row_of = nullptr, *n_rows = nullptr;
};

// Entries from one packed row to the next.
int64_t packed_cols(int64_t H) { return round_up(H, 64); }

XentPack carve_pack(Carver& c, int64_t rows, int64_t H, bool ignoring) {
  XentPack k;
  if (!ignoring) return k;
  k.hidden = c.take<uint4>(round_up(rows, lmh::kBK) * (packed_cols(H) / 8));
  k.targets = c.take<int32_t>(rows);
  k.place = c.take<int32_t>(rows);
  k.row_of = c.take<int32_t>(rows);
  k.n_rows = c.take<int32_t>(1);
  return k;
}

struct XentForward {
  XentPack pack;
  float2* partials;
  float* row_loss;
};

int64_t xent_chunks(int64_t V) { return (V + lmh::kXChunk - 1) / lmh::kXChunk; }

// Ignored rows are taken out of the loss's product where that saves a tile; what they hold meets no
// other row there. (The gradient always takes them out.)
bool xent_loss_packs(int64_t rows, bool ignoring) { return ignoring && rows > 128; }

XentForward carve_forward(Carver& c, int64_t rows, int64_t H, int64_t V, bool ignoring) {
  XentForward f;
  f.pack = carve_pack(c, rows, H, xent_loss_packs(rows, ignoring));
  f.partials = c.take<float2>(xent_chunks(V) * rows);
  f.row_loss = c.take<float>(rows);
  return f;
}

// The vocabulary in pieces of `piece` entries (a multiple of the tile width): d of a piece, 16 bits
// a row and entry, takes about 128 MB, near what L2 holds, but a piece has at least 4096 entries,
// so that its products fill the device at any number of rows. Pieces of equal length.
// `splits` is the most that dH's K (a piece) is split into, for which there are buffers.
struct XentPieces {
  int64_t rows_pad, piece;
  int32_t n_pieces, splits;
};

// How many parts dH's K (a piece) is split into, at 512 entries a part or more; each has an fp32
// buffer of its own, and they are added in order at the end. For dH alone its tiles are as many as
// a B200 has units (148 SMs, 74 pairs: constants, since the workspace's size is asked for without a
// device), and no more, as a second round costs a whole tile's time (96 x 2048 x
// 151936: 259 us with 18 splits of 8 tiles on 148 SMs, 287 with 19). Beside dW they leave units to
// dW's tiles, so that the one reads W while the other writes: 2/5 of the units for lone CTAs, where
// memory bounds both (both gradients of 8 x 1024 x 50304: 108 us with 14 splits, 127 with 32; of 32
// x 1024 x 32768: 74 and 100), and 2/3 for pairs (1000 x 1024 x 32768: 205 us with 3, 209 with 4;
// with 2, as much as with 4).
int32_t xent_splits(const XentPieces& x, int64_t rows, int64_t H, bool beside) {
  const bool pair = rows > 128;
  const int64_t units = pair ? (beside ? 49 : 74) : (beside ? 59 : 148);
  const int64_t tiles = (pair ? x.rows_pad / 256 : 1) * ((H + lmh::kXN - 1) / lmh::kXN);
  int64_t s = units / tiles;
  const int64_t by_k = x.piece / 512;
  if (s > by_k) s = by_k;
  if (s > 32) s = 32;
  return (int32_t)(s < 1 ? 1 : s);
}

XentPieces xent_pieces(int64_t rows, int64_t H, int64_t V) {
  XentPieces x;
  x.rows_pad = round_up(rows, 256);
  const int64_t v_pad = round_up(V, lmh::kXN);
  int64_t most = ((int64_t)128 << 20) / (2 * x.rows_pad) / lmh::kXN * lmh::kXN;
  if (most < 4096) most = 4096;
  x.n_pieces = (int32_t)((v_pad + most - 1) / most);
  x.piece = round_up((v_pad + x.n_pieces - 1) / x.n_pieces, lmh::kXN);
  x.n_pieces = (int32_t)((V + x.piece - 1) / x.piece);
  x.splits = xent_splits(x, rows, H, false);
  return x;
}

struct XentBackward {
  XentPack pack;
  float4* row_info;
  float *lost, *scale;
  int32_t* first;
  float *side, *bias_part[2];
  uint16_t* d[2];
  float* dh_partial;
};

XentBackward carve_backward(Carver& c, const XentPieces& x, int64_t rows, int64_t H, int64_t V,
                            bool ignoring) {
  XentBackward b;
  b.pack = carve_pack(c, rows, H, ignoring);
  b.row_info = c.take<float4>(rows);
  b.lost = c.take<float>(rows);
  b.scale = c.take<float>(2);
  b.first = c.take<int32_t>(V);
  b.side = c.take<float>(rows * H);
  b.d[0] = c.take<uint16_t>(x.rows_pad * x.piece);
  for (int i = 0; i < 2; ++i) b.bias_part[i] = c.take<float>(x.rows_pad / 32 * x.piece);
  b.d[1] = x.n_pieces > 1 ? c.take<uint16_t>(x.rows_pad * x.piece) : b.d[0];
  b.dh_partial = c.take<float>((int64_t)x.splits * x.rows_pad * H);
  return b;
}

int check_xent_args(const void* hidden, int dtype, int64_t rows, int64_t H, const void* W,
                    int64_t V, const void* bias, int64_t ignore_index, int reduction) {
  const int st = check_f32_head_args(hidden, dtype, rows, H, W, V, bias);
  if (st != LMHEAD_OK) return st;
  if (rows >= kTrainMax || H >= kTrainMax || V >= kTrainMax) return LMHEAD_ERR_SHAPE;
  if (ignore_index != LMHEAD_IGNORE_NONE &&
      (ignore_index < INT32_MIN || ignore_index > INT32_MAX))
    return LMHEAD_ERR_SHAPE;
  if (reduction != LMHEAD_REDUCE_NONE && reduction != LMHEAD_REDUCE_SUM &&
      reduction != LMHEAD_REDUCE_MEAN)
    return LMHEAD_ERR_SHAPE;
  return LMHEAD_OK;
}

int launch_pack(const XentPack& k, const void* hidden, const int32_t* targets, int64_t rows,
                int64_t H, int64_t ignore_index, lmhead_stream_t stream) {
  // a row a warp, so that few rows are copied by many blocks; for many rows 32 a block, since each
  // block reads all targets
  const int32_t block_rows = rows <= 8192 ? lmh::kPackThreads / 32 : lmh::kPackRows;
  const unsigned blocks = (unsigned)((rows + block_rows - 1) / block_rows);
  return launch_head(lmh::xent_pack_kernel, blocks, lmh::kPackThreads, 0, stream, 1u,
                     reinterpret_cast<const uint4*>(hidden), targets, (int32_t)rows, block_rows,
                     (int32_t)(H / 8), (int32_t)(packed_cols(H) / 8), (int32_t)ignore_index,
                     k.hidden, k.targets, k.place, k.row_of, k.n_rows);
}

// A matrix of 16-bit elements in boxes of 64 columns by `box_rows` rows.
int encode_xent(CUtensorMap* map, const void* base, int64_t cols, int64_t rows,
                uint32_t box_rows) {
  return encode_rows(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, base, cols * 2, rows, 128, box_rows,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// A matrix that is stored to, in the epilogues' boxes of 32 rows of 32 columns.
int encode_xent_store(CUtensorMap* map, const void* base, int64_t cols, int64_t rows) {
  return encode_rows(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, base, cols * 2, rows, 64, 32,
                     CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// The same matrix (cols a multiple of 64) seen as [cols / 64][rows][64], in boxes of 64 rows of
// `blocks` column blocks.
int encode_xent_mn(CUtensorMap* map, const void* base, int64_t cols, int64_t rows,
                   uint32_t blocks) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return LMHEAD_ERR_LAUNCH;
  const int esize = LMHEAD_TMA_WIDE ? 4 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)(128 / esize), (cuuint64_t)rows, (cuuint64_t)(cols / 64)};
  const cuuint64_t strides[2] = {(cuuint64_t)(cols * 2), 128};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / esize), 64, blocks};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r =
      enc(map, LMHEAD_TMA_WIDE ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3,
          const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? LMHEAD_OK : LMHEAD_ERR_LAUNCH;
}

// How a call's products are tiled, and with it the boxes of the tensor maps.
struct XentShape {
  int shape;
  int64_t rows;
  // rows of an operand in one CTA's tile: A of the wide products; A of the weight product; B of the
  // wide products; B of the weight product
  // (A: no more than there are, in whole swizzle atoms of 8. TMA is slow on rows past the matrix's
  // end: one row in boxes of 128 took 335 us at 2048 x 151936, in boxes of 64 189 us, where 96 rows
  // take 128 us.)
  uint32_t wide_a() const {
    return shape == lmh::kXLone && rows < 128 ? (uint32_t)round_up(rows, 8) : 128;
  }
  uint32_t tall_a() const { return shape == lmh::kXBig ? 256 : 128; }
  uint32_t wide_b() const { return shape == lmh::kXPair ? 128 : 256; }
  uint32_t tall_b() const { return shape == lmh::kXLone ? 256 : 128; }
};

// CTA pairs for more than 128 rows. With at most 128 rows, half of a pair's 256-row tile would be
// empty and the call is bound by reading W; lone CTAs of 128 rows spend half the tensor time.
// Big tiles for the gradient of 2^28 logits or more: there they are 3 to 8 % faster (4096 rows x
// 4096 x 151936: 11.89 ms against 12.71; 2048 x 2048: 3.17 against 3.26), with half as many logits 1
// to 2 % slower on average (the waves of larger tiles fill the device worse, and a tile's epilogue is
// in part exposed). The loss alone keeps pairs: its products have no output to write, and big tiles
// measured 1 % faster at the largest sizes and up to 15 % slower elsewhere.
XentShape xent_shape(const DeviceInfo& dev, int64_t rows, int64_t V, bool gradient) {
  if (rows <= 128 || dev.pair_clusters <= 0 || g_no_cta_pairs.load(std::memory_order_relaxed))
    return {lmh::kXLone, rows};
  return {gradient && rows * V >= (int64_t)1 << 28 ? lmh::kXBig : lmh::kXPair, rows};
}

// Whether a shape's kernel has the epilogues of a launch's products. Big tiles have none for the
// loss's statistics: its warps would leave their accumulators, and the loss, unwritten.
bool xent_shape_serves(int shape, const lmh::XentParams& p) {
  for (int i = 0; i < p.n_problems; ++i)
    if (shape == lmh::kXBig && p.prob[i].kind == lmh::kXentStats) return false;
  return true;
}

template <int kShape>
int64_t xent_tiles(const lmh::XentParams& p) {
  using T = lmh::XentTile<kShape>;
  int64_t tiles = 0;
  for (int i = 0; i < p.n_problems; ++i) {
    const lmh::XentProblem& q = p.prob[i];
    const int64_t m = q.m_rows ? p.rows : q.m_len, tm = T::rows(q.wide), tn = T::cols(q.wide);
    tiles += ((m + tm - 1) / tm) * ((q.n_len + tn - 1) / tn) * q.splits;
  }
  return tiles;
}

template <int kShape>
int launch_xent_shape(const DeviceInfo& dev, bool fp16, const lmh::XentMaps& maps,
                      const lmh::XentParams& p, lmhead_stream_t stream) {
  using T = lmh::XentTile<kShape>;
  if (!xent_shape_serves(kShape, p)) return LMHEAD_ERR_SHAPE;
  const int64_t ctas = xent_tiles<kShape>(p) * (T::kPair ? 2 : 1);
  if (ctas > kInt32Max || (int64_t)T::kSmem > dev.smem_optin) return LMHEAD_ERR_SHAPE;
  return launch_head(
      fp16 ? lmh::xent_gemm_kernel<kShape, true> : lmh::xent_gemm_kernel<kShape, false>,
      (unsigned)ctas, T::kThreads, T::kSmem, stream, T::kPair ? 2u : 1u, maps, p);
}

int launch_xent_gemm(const DeviceInfo& dev, bool fp16, XentShape s, const lmh::XentMaps& maps,
                     const lmh::XentParams& p, lmhead_stream_t stream) {
  return s.shape == lmh::kXBig    ? launch_xent_shape<lmh::kXBig>(dev, fp16, maps, p, stream)
         : s.shape == lmh::kXPair ? launch_xent_shape<lmh::kXPair>(dev, fp16, maps, p, stream)
                                  : launch_xent_shape<lmh::kXLone>(dev, fp16, maps, p, stream);
}

lmh::XentProblem xent_problem(int kind, int a_map, int b_map, int64_t n_len, int64_t k_len) {
  lmh::XentProblem q = {};
  q.kind = kind;
  q.a_map = a_map;
  q.b_map = b_map;
  q.n_len = (int32_t)n_len;
  q.k_len = (int32_t)k_len;
  q.splits = 1;
  // M tiles walked together. The logits take 16, the rows' operands of a batch of 4096 staying in
  // L2 while W streams by (4096 x 4096 x 128256: 3.34 ms, one at a time 3.96); the weight product
  // one, d streaming by (3.39 ms, 16 at a time 3.57); dH's is the same within 1 % from 1 to 8.
  q.group = kind == lmh::kXentDweight ? 1 : kind == lmh::kXentDhidden ? 4 : 16;
  q.wide = kind != lmh::kXentDweight;
  return q;
}

int run_xent_forward(const void* hidden, int dtype, int64_t rows, int64_t H, const void* W,
                     int64_t V, float alpha, const void* bias, const int32_t* targets,
                     int64_t ignore_index, float z_loss, int reduction, float* loss, float* lse,
                     const XentForward& f, lmhead_stream_t stream) {
  DeviceInfo dev;
  int st = current_device(&dev);
  if (st != LMHEAD_OK) return st;
  const bool ignoring = ignore_index != LMHEAD_IGNORE_NONE;
  const bool packing = xent_loss_packs(rows, ignoring);
  const bool fp16 = dtype == LMHEAD_DTYPE_F16;
  const XentPack& k = f.pack;
  if (packing) {
    st = launch_pack(k, hidden, targets, rows, H, ignore_index, stream);
    if (st != LMHEAD_OK) return st;
  }
  const XentShape shape = xent_shape(dev, rows, V, false);
  lmh::XentMaps maps = {};
  st = encode_xent(&maps.m[lmh::kMapHidden], packing ? k.hidden : hidden,
                   packing ? packed_cols(H) : H, packing ? round_up(rows, lmh::kBK) : rows,
                   shape.wide_a());
  if (st != LMHEAD_OK) return st;
  st = encode_xent(&maps.m[lmh::kMapW], W, H, V, shape.wide_b());
  if (st != LMHEAD_OK) return st;

  lmh::XentParams p = {};
  p.n_problems = 1;
  p.prob[0] = xent_problem(lmh::kXentStats, lmh::kMapHidden, lmh::kMapW, V, H);
  p.prob[0].m_rows = 1;
  p.rows = (int32_t)rows;
  p.a_rows = (int32_t)shape.wide_a();
  p.n_rows = k.n_rows;
  p.H = (int32_t)H;
  p.alpha = alpha;
  p.bias = reinterpret_cast<const uint16_t*>(bias);
  p.targets = packing ? k.targets : targets;
  p.partials = f.partials;
  p.wait = wait_cfg();
  st = launch_xent_gemm(dev, fp16, shape, maps, p, stream);
  if (st != LMHEAD_OK) return st;

  const bool each = reduction == LMHEAD_REDUCE_NONE, mean = reduction == LMHEAD_REDUCE_MEAN;
  const bool few = rows < 2048;
  const int64_t fold_rows = few ? lmh::kFoldFew : lmh::kFoldMany;
  const unsigned folds = (unsigned)((rows + fold_rows - 1) / fold_rows);
  const bool one_cluster = !each && folds <= (unsigned)lmh::kFoldCluster;
  float* row_loss = each ? loss : f.row_loss;
  auto fold = few ? (fp16 ? lmh::xent_fold_kernel<lmh::kFoldFew, true>
                          : lmh::xent_fold_kernel<lmh::kFoldFew, false>)
                  : (fp16 ? lmh::xent_fold_kernel<lmh::kFoldMany, true>
                          : lmh::xent_fold_kernel<lmh::kFoldMany, false>);
  st = launch_head(fold, folds, 1024, 0, stream, one_cluster ? folds : 1u,
                   (const float2*)f.partials, (int32_t)xent_chunks(V), (int32_t)rows,
                   (int32_t)rows, (int32_t)V, (const int32_t*)k.place, targets,
                   reinterpret_cast<const uint4*>(hidden), reinterpret_cast<const uint4*>(W),
                   (int32_t)(H / 8), p.bias, alpha, z_loss, row_loss, lse,
                   (int32_t)ignoring, (int32_t)ignore_index, (int32_t)mean,
                   one_cluster ? loss : nullptr);
  if (st != LMHEAD_OK || each || one_cluster) return st;
  return launch_head(lmh::xent_reduce_kernel, 1, 1024, 0, stream, 1u, (const float*)row_loss,
                     targets, (int32_t)rows, (int32_t)ignoring, (int32_t)ignore_index,
                     (int32_t)mean, loss);
}

int run_xent_backward(const void* hidden, int dtype, int64_t rows, int64_t H, const void* W,
                      int64_t V, float alpha, const void* bias, const int32_t* targets,
                      int64_t ignore_index, float z_loss, int reduction, const float* lse,
                      const float* grad_loss, void* d_hidden, void* d_W, void* d_bias,
                      int accumulate, const XentPieces& x, const XentBackward& b,
                      lmhead_stream_t stream) {
  DeviceInfo dev;
  int st = current_device(&dev);
  if (st != LMHEAD_OK) return st;
  const bool ignoring = ignore_index != LMHEAD_IGNORE_NONE;
  const bool fp16 = dtype == LMHEAD_DTYPE_F16;
  const XentShape shape = xent_shape(dev, rows, V, true);
  const int32_t splits = xent_splits(x, rows, H, d_W != nullptr);
  const XentPack& k = b.pack;
  if (ignoring) {
    st = launch_pack(k, hidden, targets, rows, H, ignore_index, stream);
    if (st != LMHEAD_OK) return st;
  }
  // 32 rows a block, and 4096 entries of the table that it clears
  int64_t row_blocks = (rows + lmh::kRowsBlock - 1) / lmh::kRowsBlock;
  if (row_blocks < (V + 4095) / 4096) row_blocks = (V + 4095) / 4096;
  if (row_blocks > 2 * dev.num_sms) row_blocks = 2 * dev.num_sms;
  st = launch_head(fp16 ? lmh::xent_rows_kernel<true> : lmh::xent_rows_kernel<false>,
                   (unsigned)row_blocks, 1024, 0, stream, 1u, lse, targets,
                   (const int32_t*)k.row_of, (int32_t)rows, (const int32_t*)k.n_rows, (int32_t)V,
                   reinterpret_cast<const uint4*>(hidden), reinterpret_cast<const uint4*>(W),
                   (int32_t)(H / 8), reinterpret_cast<const uint16_t*>(bias), grad_loss,
                   (int32_t)(reduction == LMHEAD_REDUCE_NONE),
                   (int32_t)(reduction == LMHEAD_REDUCE_MEAN), z_loss, alpha, b.row_info, b.lost, b.scale, b.first);
  if (st != LMHEAD_OK) return st;

  const void* h = ignoring ? k.hidden : hidden;
  const int64_t h_cols = ignoring ? packed_cols(H) : H;
  const int64_t h_rows = ignoring ? round_up(rows, lmh::kBK) : rows;
  lmh::XentMaps maps = {};
  st = encode_xent(&maps.m[lmh::kMapHidden], h, h_cols, h_rows, shape.wide_a());
  if (st == LMHEAD_OK) st = encode_xent(&maps.m[lmh::kMapW], W, H, V, shape.wide_b());
  // hidden and W as B's MN-major operand (below 64 columns every tile is an edge)
  if (st == LMHEAD_OK) st = encode_xent(&maps.m[lmh::kMapHiddenEdge], h, h_cols, h_rows, 64);
  if (st == LMHEAD_OK) st = encode_xent(&maps.m[lmh::kMapWEdge], W, H, V, 64);
  if (st == LMHEAD_OK && H >= 64)
    st = encode_xent_mn(&maps.m[lmh::kMapHiddenMn], h, h_cols, h_rows, shape.tall_b() / 64);
  if (st == LMHEAD_OK && H >= 64)
    st = encode_xent_mn(&maps.m[lmh::kMapWMn], W, H, V, shape.wide_b() / 64);
  for (int i = 0; i < (x.n_pieces > 1 ? 2 : 1) && st == LMHEAD_OK; ++i) {
    st = encode_xent(&maps.m[lmh::kMapD + i], b.d[i], x.piece, x.rows_pad, shape.wide_a());
    if (st == LMHEAD_OK)
      st = encode_xent_mn(&maps.m[lmh::kMapDMn + i], b.d[i], x.piece, x.rows_pad, shape.tall_a() / 64);
    if (st == LMHEAD_OK)
      st = encode_xent_store(&maps.m[lmh::kMapDStore + i], b.d[i], x.piece, x.rows_pad);
  }
  if (st == LMHEAD_OK && d_hidden != nullptr)
    st = encode_2d(&maps.m[lmh::kMapDh], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, b.dh_partial, H,
                   (int64_t)splits * x.rows_pad, 16, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  if (st == LMHEAD_OK && d_W != nullptr) st = encode_xent_store(&maps.m[lmh::kMapDw], d_W, H, V);
  if (st != LMHEAD_OK) return st;

  lmh::XentParams p = {};
  p.rows = (int32_t)rows;
  p.a_rows = (int32_t)shape.wide_a();
  p.n_rows = k.n_rows;
  p.H = (int32_t)H;
  p.rows_pad = (int32_t)x.rows_pad;
  p.alpha = alpha;
  p.bias = reinterpret_cast<const uint16_t*>(bias);
  p.targets = ignoring ? k.targets : targets;
  p.first = b.first;
  p.side = b.side;
  p.row_info = b.row_info;
  p.scale = b.scale;
  p.d_weight = reinterpret_cast<uint16_t*>(d_W);
  p.wait = wait_cfg();

  auto start = [&](int c) { return (int64_t)c * x.piece; };
  auto length = [&](int c) { return V - start(c) < x.piece ? V - start(c) : x.piece; };
  auto logits_of = [&](int c) {
    lmh::XentProblem q =
        xent_problem(lmh::kXentDlogits, lmh::kMapHidden, lmh::kMapW, length(c), H);
    q.m_rows = 1;
    q.b_off = (int32_t)start(c);
    q.out_map = lmh::kMapDStore + (c & 1);
    return q;
  };
  p.piece = (int32_t)x.piece;
  p.bias_part = d_bias != nullptr ? b.bias_part[0] : nullptr;
  p.n_problems = 1;
  p.prob[0] = logits_of(0);
  st = launch_xent_gemm(dev, fp16, shape, maps, p, stream);
  for (int c = 0; c < x.n_pieces && st == LMHEAD_OK; ++c) {
    if (d_bias != nullptr) {
      const unsigned blocks = (unsigned)((length(c) + lmh::kBiasCols - 1) / lmh::kBiasCols);
      st = launch_head(fp16 ? lmh::xent_bias_kernel<true> : lmh::xent_bias_kernel<false>, blocks,
                       lmh::kBiasCols * lmh::kBiasParts, 0, stream, 1u,
                       (const float*)b.bias_part[c & 1], (int32_t)x.piece,
                       (int32_t)length(c), (int32_t)rows, (const int32_t*)k.n_rows,
                       (const float*)b.scale, (int32_t)(accumulate != 0),
                       reinterpret_cast<uint16_t*>(d_bias) + start(c));
      if (st != LMHEAD_OK) return st;
    }
    if (d_bias != nullptr) p.bias_part = b.bias_part[(c + 1) & 1];
    p.n_problems = 0;
    if (d_hidden != nullptr) {  // the longest tiles first
      lmh::XentProblem q = xent_problem(lmh::kXentDhidden, lmh::kMapD + (c & 1),
                                         lmh::kMapWMn, H, length(c));
      q.m_rows = 1;
      q.b_mn = 1;
      q.b_edge = lmh::kMapWEdge;
      q.b_off = (int32_t)start(c);
      q.b_k = 1;
      q.splits = splits;
      q.add = c > 0;
      p.prob[p.n_problems++] = q;
    }
    if (d_W != nullptr) {
      lmh::XentProblem q = xent_problem(lmh::kXentDweight, lmh::kMapDMn + (c & 1),
                                         lmh::kMapHiddenMn, H, 0);
      q.m_len = (int32_t)length(c);
      q.k_rows = 1;
      q.a_mn = q.b_mn = 1;
      q.b_edge = lmh::kMapHiddenEdge;
      q.out_off = (int32_t)start(c);
      q.out_map = lmh::kMapDw;
      q.add = accumulate != 0;
      p.prob[p.n_problems++] = q;
    }
    if (c + 1 < x.n_pieces) p.prob[p.n_problems++] = logits_of(c + 1);
    if (p.n_problems > 0) st = launch_xent_gemm(dev, fp16, shape, maps, p, stream);
  }
  if (st != LMHEAD_OK) return st;
  lmh::XentFinishParams f = {};
  f.rows = (int32_t)rows;
  f.H = (int32_t)H;
  f.V = (int32_t)V;
  f.n_rows = k.n_rows;
  f.place = k.place;
  f.targets = targets;
  f.packed_targets = p.targets;
  f.lost = b.lost;
  f.scale = b.scale;
  f.splits = splits;
  f.split_len = x.rows_pad * H;
  f.partial = b.dh_partial;
  f.W = reinterpret_cast<const uint4*>(W);
  f.d_hidden = reinterpret_cast<uint4*>(d_hidden);
  f.first = b.first;
  f.side = b.side;
  f.hidden = reinterpret_cast<const uint4*>(h);
  f.hidden_vecs = (int32_t)(h_cols / 8);
  f.d_weight = reinterpret_cast<uint4*>(d_W);
  const int64_t hidden_blocks =
      d_hidden == nullptr ? 0 : (rows * (H / 8) + lmh::kFinishThreads - 1) / lmh::kFinishThreads;
  const int64_t slices = (H / 8 + lmh::kFinishThreads - 1) / lmh::kFinishThreads;
  const int64_t weight_blocks = d_W == nullptr ? 0 : rows * slices;
  if (hidden_blocks + weight_blocks == 0) return LMHEAD_OK;  // d_bias alone
  if (hidden_blocks + weight_blocks > kInt32Max) return LMHEAD_ERR_SHAPE;
  f.hidden_blocks = (int32_t)hidden_blocks;
  f.slices = (int32_t)slices;
  return launch_head(fp16 ? lmh::xent_finish_kernel<true> : lmh::xent_finish_kernel<false>,
                     (unsigned)(hidden_blocks + weight_blocks), lmh::kFinishThreads, 0, stream, 1u,
                     f);
}

int cleared(int st) {
  if (st != LMHEAD_OK) (void)cudaGetLastError();  // leave no stale error for the next call
  return st;
}

// Zeros in `bytes` bytes of device memory, on the stream.
int write_zeros(void* p, int64_t bytes, lmhead_stream_t stream) {
  if (p == nullptr || bytes == 0) return LMHEAD_OK;
  return cudaMemsetAsync(p, 0, (size_t)bytes, (cudaStream_t)stream) == cudaSuccess
             ? LMHEAD_OK
             : LMHEAD_ERR_LAUNCH;
}

bool xent_sizes_ok(int64_t rows, int64_t H, int64_t V) {
  return rows > 0 && H > 0 && V > 0 && rows < kTrainMax && H < kTrainMax && V < kTrainMax;
}

// ---------------------------------------------------------------- embedding

struct EmbedPlan {
  int32_t passes, bits;  // of the sort
  int32_t tile, tiles;   // sorted entries per block of the sums
};

// Digits of equal width, as few passes as 9 bits a digit allow, that hold every id and the mark V.
// The sums take at least 8 entries a block, and as many as leave 4096 blocks (two waves; 16384
// tokens of 4096 columns: the sums 197 us in tiles of 16 and of 64, but the join, a block for each
// tile and slice of columns, 21 us against 9; few tokens still make many blocks: 1025 tokens of 264
// columns take 15 us in tiles of 64, 5 in tiles of 8) and 1024 tiles, so that a run through all
// tokens is joined from at most 1024 parts (up to a million tokens: tiles end at 1024 entries).
EmbedPlan embed_plan(int64_t tokens, int64_t V, int64_t H) {
  EmbedPlan e;
  int bits = 1;
  while (((int64_t)1 << bits) <= V) ++bits;
  e.passes = (bits + lmh::kSortBits - 1) / lmh::kSortBits;
  e.bits = (bits + e.passes - 1) / e.passes;
  e.tile = lmh::kSumTileMin;
  const int64_t slices = (H + lmh::kSumCols - 1) / lmh::kSumCols;
  const int64_t tiles = slices < 4 ? 1024 : slices < 4096 ? 4096 / slices : 1;
  while (e.tile < lmh::kSumTileMax && (int64_t)e.tile * tiles < tokens) e.tile *= 2;
  e.tiles = (int32_t)((tokens + e.tile - 1) / e.tile);
  return e;
}

struct EmbedScratch {
  int32_t *keys[2], *pos[2];
  uint32_t* seen;
  float* part;
};

EmbedScratch carve_embed(Carver& c, const EmbedPlan& e, int64_t tokens, int64_t V, int64_t H) {
  EmbedScratch s;
  for (int i = 0; i < 2; ++i) {
    s.keys[i] = c.take<int32_t>(tokens);
    s.pos[i] = c.take<int32_t>(tokens);
  }
  s.seen = c.take<uint32_t>((V + 31) / 32);
  s.part = c.take<float>((int64_t)e.tiles * 2 * H);
  return s;
}

// The sizes and the table's place in the vocabulary; token ids are int32.
int check_embed_sizes(int dtype, int64_t tokens, int64_t V, int64_t v_begin, int64_t H) {
  if (dtype != LMHEAD_DTYPE_BF16 && dtype != LMHEAD_DTYPE_F16) return LMHEAD_ERR_SHAPE;
  if (tokens < 0 || V <= 0 || H <= 0) return LMHEAD_ERR_SHAPE;
  if (H % 8 != 0) return LMHEAD_ERR_ALIGN;
  if (tokens >= kTrainMax || V >= kTrainMax || H >= kTrainMax) return LMHEAD_ERR_SHAPE;
  if (v_begin < 0 || v_begin > kInt32Max || V > (int64_t)kInt32Max + 1 - v_begin)
    return LMHEAD_ERR_SHAPE;
  return LMHEAD_OK;
}

int run_embed_grad(const DeviceInfo& dev, const void* d_out, int dtype, const int32_t* ids,
                   int64_t tokens, int64_t V, int64_t v_begin, int64_t H, float scale, void* d_W,
                   int accumulate, const EmbedPlan& e, const EmbedScratch& s,
                   lmhead_stream_t stream) {
  lmh::EmbedSortParams q = {};
  q.ids = ids;
  q.tokens = (int32_t)tokens;
  q.v_begin = (int32_t)v_begin;
  q.V = (int32_t)V;
  q.passes = e.passes;
  q.bits = e.bits;
  for (int i = 0; i < 2; ++i) {
    q.keys[i] = s.keys[i];
    q.pos[i] = s.pos[i];
  }
  // the rows that the sort's launch clears: about what the device writes while the sort runs
  const int64_t row_bytes = H * 2;
  int64_t head = accumulate ? 0 : (((int64_t)24 << 20) + 2048 * tokens) / row_bytes;
  if (head > V) head = V;
  const int64_t rest = accumulate ? 0 : V - head;
  unsigned clusters = 1;
  if (head > 0) {
    q.zero = reinterpret_cast<uint4*>(d_W);
    q.zero_vecs = head * (H / 8);
    // two CTAs of 1024 threads an SM, or as many as the rows have work for
    int64_t fill = (q.zero_vecs + 4 * lmh::kSortThreads - 1) / (4 * lmh::kSortThreads);
    if (fill > 2 * dev.num_sms) fill = 2 * dev.num_sms;
    clusters += (unsigned)((fill + lmh::kSortCtas - 1) / lmh::kSortCtas);
  }
  if (rest > 0) q.seen = s.seen;
  int st = launch_head(lmh::embed_sort_kernel, clusters * lmh::kSortCtas, lmh::kSortThreads, 0,
                       stream, lmh::kSortCtas, q);
  if (st != LMHEAD_OK) return st;
  const bool fp16 = dtype == LMHEAD_DTYPE_F16;
  lmh::EmbedSumParams p = {};
  p.keys = s.keys[(e.passes - 1) & 1];
  p.pos = s.pos[(e.passes - 1) & 1];
  p.tokens = (int32_t)tokens;
  p.V = (int32_t)V;
  p.H = (int32_t)H;
  p.tile = e.tile;
  p.d_out = reinterpret_cast<const uint16_t*>(d_out);
  p.scale = scale;
  p.add = accumulate != 0;
  p.d_weight = reinterpret_cast<uint16_t*>(d_W);
  p.part = s.part;
  p.slices = (int32_t)((H + lmh::kSumCols - 1) / lmh::kSumCols);
  p.seen = s.seen;
  p.zero_from = (int32_t)head;
  p.zero_rows = (int32_t)(lmh::kZeroVecs / (H / 8) > 1 ? lmh::kZeroVecs / (H / 8) : 1);
  const int64_t sums = (int64_t)e.tiles * p.slices;
  const int64_t zeros = (rest + p.zero_rows - 1) / p.zero_rows;
  if (sums + zeros > kInt32Max) return LMHEAD_ERR_SHAPE;
  p.sum_blocks = (int32_t)sums;
  st = launch_head(fp16 ? lmh::embed_sum_kernel<true> : lmh::embed_sum_kernel<false>,
                   (unsigned)(sums + zeros), lmh::kSumThreads, 0, stream, 1u, p);
  if (st != LMHEAD_OK || e.tiles == 1) return st;
  return launch_head(fp16 ? lmh::embed_join_kernel<true> : lmh::embed_join_kernel<false>,
                     dim3((unsigned)(e.tiles - 1), (unsigned)p.slices),
                     lmh::kJoinGroups * lmh::kSumThreads, 0, stream, 1u, p);
}

}  // namespace

extern "C" {

#if LMHEAD_TEST_HOOKS
// For the tests: the rule above for a launch with a product of `kind`. (No knob: it sets nothing.)
int lmhead_debug_xent_shape_serves(int shape, int kind) {
  lmh::XentParams p = {};
  p.n_problems = 2;  // a product that every shape serves, then the one in question
  p.prob[0].kind = lmh::kXentDweight;
  p.prob[1].kind = kind;
  return xent_shape_serves(shape, p) ? 1 : 0;
}
#endif

size_t lmhead_cross_entropy_workspace_bytes(int64_t rows, int64_t H, int64_t V,
                                            int64_t ignore_index) {
  if (!xent_sizes_ok(rows, H, V)) return 0;
  Carver c(nullptr);
  carve_forward(c, rows, H, V, ignore_index != LMHEAD_IGNORE_NONE);
  return (size_t)c.used;
}

size_t lmhead_cross_entropy_grad_workspace_bytes(int64_t rows, int64_t H, int64_t V,
                                                 int64_t ignore_index) {
  if (!xent_sizes_ok(rows, H, V)) return 0;
  Carver c(nullptr);
  carve_backward(c, xent_pieces(rows, H, V), rows, H, V, ignore_index != LMHEAD_IGNORE_NONE);
  return (size_t)c.used;
}

int lmhead_cross_entropy_f32(const void* hidden, int dtype, int64_t rows, int64_t H,
                             const void* W, int64_t V, float alpha, const void* bias,
                             const int32_t* targets, int64_t ignore_index, float z_loss,
                             int reduction, float* loss, float* lse, void* workspace,
                             size_t workspace_bytes, lmhead_stream_t stream) {
  int st = check_xent_args(hidden, dtype, rows, H, W, V, bias, ignore_index, reduction);
  if (st != LMHEAD_OK) return st;
  if (rows == 0) {
    if (reduction == LMHEAD_REDUCE_NONE) return LMHEAD_OK;
    if (loss == nullptr) return LMHEAD_ERR_NULL;
    if (!aligned(loss, 4)) return LMHEAD_ERR_ALIGN;
    DeviceInfo dev;
    st = current_device(&dev);
    return st != LMHEAD_OK ? st : cleared(write_zeros(loss, 4, stream));
  }
  if (targets == nullptr || loss == nullptr || lse == nullptr || workspace == nullptr)
    return LMHEAD_ERR_NULL;
  if (!aligned(targets, 4) || !aligned(loss, 4) || !aligned(lse, 4) || !aligned(workspace, 256))
    return LMHEAD_ERR_ALIGN;
  if (workspace_bytes < lmhead_cross_entropy_workspace_bytes(rows, H, V, ignore_index))
    return LMHEAD_ERR_SHAPE;
  const Region in[4] = {
      {hidden, rows * H * 2}, {W, V * H * 2}, {bias, V * 2}, {targets, rows * 4}};
  const Region out[3] = {{loss, reduction == LMHEAD_REDUCE_NONE ? rows * 4 : 4},
                         {lse, rows * 4},
                         {workspace, (int64_t)workspace_bytes}};
  st = check_overlap(in, 4, out, 3);
  if (st != LMHEAD_OK) return st;
  Carver c(workspace);
  const XentForward f = carve_forward(c, rows, H, V, ignore_index != LMHEAD_IGNORE_NONE);
  return cleared(run_xent_forward(hidden, dtype, rows, H, W, V, alpha, bias, targets, ignore_index,
                                  z_loss, reduction, loss, lse, f, stream));
}

int lmhead_cross_entropy_grad(const void* hidden, int dtype, int64_t rows, int64_t H,
                              const void* W, int64_t V, float alpha, const void* bias,
                              const int32_t* targets, int64_t ignore_index, float z_loss,
                              int reduction, const float* lse, const float* grad_loss,
                              void* d_hidden, void* d_W, void* d_bias, int accumulate,
                              void* workspace, size_t workspace_bytes, lmhead_stream_t stream) {
  int st = check_xent_args(hidden, dtype, rows, H, W, V, bias, ignore_index, reduction);
  if (st != LMHEAD_OK) return st;
  if (d_hidden == nullptr && d_W == nullptr && d_bias == nullptr && rows > 0)
    return LMHEAD_ERR_NULL;
  if ((d_hidden != nullptr && !aligned(d_hidden, 16)) || (d_W != nullptr && !aligned(d_W, 16)) ||
      (d_bias != nullptr && !aligned(d_bias, 2)))
    return LMHEAD_ERR_ALIGN;
  if (rows == 0) {
    if (accumulate) return LMHEAD_OK;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st == LMHEAD_OK) st = write_zeros(d_W, V * H * 2, stream);
    if (st == LMHEAD_OK) st = write_zeros(d_bias, V * 2, stream);
    return cleared(st);
  }
  if (targets == nullptr || lse == nullptr || grad_loss == nullptr || workspace == nullptr)
    return LMHEAD_ERR_NULL;
  if (!aligned(targets, 4) || !aligned(lse, 4) || !aligned(grad_loss, 4) ||
      !aligned(workspace, 256))
    return LMHEAD_ERR_ALIGN;
  if (workspace_bytes < lmhead_cross_entropy_grad_workspace_bytes(rows, H, V, ignore_index))
    return LMHEAD_ERR_SHAPE;
  const Region in[6] = {{hidden, rows * H * 2},
                        {W, V * H * 2},
                        {bias, V * 2},
                        {targets, rows * 4},
                        {lse, rows * 4},
                        {grad_loss, reduction == LMHEAD_REDUCE_NONE ? rows * 4 : 4}};
  const Region out[4] = {{d_hidden, rows * H * 2},
                         {d_W, V * H * 2},
                         {d_bias, V * 2},
                         {workspace, (int64_t)workspace_bytes}};
  st = check_overlap(in, 6, out, 4);
  if (st != LMHEAD_OK) return st;
  const XentPieces x = xent_pieces(rows, H, V);
  Carver c(workspace);
  const XentBackward b = carve_backward(c, x, rows, H, V, ignore_index != LMHEAD_IGNORE_NONE);
  return cleared(run_xent_backward(hidden, dtype, rows, H, W, V, alpha, bias, targets, ignore_index,
                                   z_loss, reduction, lse, grad_loss, d_hidden, d_W, d_bias,
                                   accumulate, x, b, stream));
}

int lmhead_embedding(const int32_t* ids, int64_t tokens, const void* W, int dtype, int64_t V,
                     int64_t v_begin, int64_t H, float scale, void* out, lmhead_stream_t stream) {
  int st = check_embed_sizes(dtype, tokens, V, v_begin, H);
  if (st != LMHEAD_OK || tokens == 0) return st;
  if (ids == nullptr || W == nullptr || out == nullptr) return LMHEAD_ERR_NULL;
  if (!aligned(ids, 4) || !aligned(W, 16) || !aligned(out, 16)) return LMHEAD_ERR_ALIGN;
  const Region in[2] = {{ids, tokens * 4}, {W, V * H * 2}};
  const Region o[1] = {{out, tokens * H * 2}};
  st = check_overlap(in, 2, o, 1);
  if (st != LMHEAD_OK) return st;
  const int64_t pieces = (H / 8 + lmh::kEmbedVecs - 1) / lmh::kEmbedVecs;
  const int64_t blocks =
      (tokens * pieces + lmh::kEmbedThreads / 32 - 1) / (lmh::kEmbedThreads / 32);
  if (blocks > kInt32Max) return LMHEAD_ERR_SHAPE;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != LMHEAD_OK) return st;
  return cleared(launch_head(
      dtype == LMHEAD_DTYPE_F16 ? lmh::embed_kernel<true> : lmh::embed_kernel<false>,
      (unsigned)blocks, lmh::kEmbedThreads, 0, stream, 1u, ids, tokens, (int32_t)v_begin,
      (int32_t)V, reinterpret_cast<const uint4*>(W), (int32_t)(H / 8), (int32_t)pieces, scale,
      reinterpret_cast<uint4*>(out)));
}

size_t lmhead_embedding_grad_workspace_bytes(int64_t tokens, int64_t V, int64_t H) {
  if (tokens <= 0 || V <= 0 || H <= 0 || tokens >= kTrainMax || V >= kTrainMax || H >= kTrainMax)
    return 0;
  Carver c(nullptr);
  carve_embed(c, embed_plan(tokens, V, H), tokens, V, H);
  return (size_t)c.used;
}

int lmhead_embedding_grad(const void* d_out, int dtype, const int32_t* ids, int64_t tokens,
                          int64_t V, int64_t v_begin, int64_t H, float scale, void* d_W,
                          int accumulate, void* workspace, size_t workspace_bytes,
                          lmhead_stream_t stream) {
  int st = check_embed_sizes(dtype, tokens, V, v_begin, H);
  if (st != LMHEAD_OK) return st;
  if (d_W == nullptr) return LMHEAD_ERR_NULL;
  if (!aligned(d_W, 16)) return LMHEAD_ERR_ALIGN;
  if (tokens == 0 && accumulate) return LMHEAD_OK;
  DeviceInfo dev;
  if (tokens == 0) {
    st = current_device(&dev);
    return st != LMHEAD_OK ? st : cleared(write_zeros(d_W, V * H * 2, stream));
  }
  if (d_out == nullptr || ids == nullptr || workspace == nullptr) return LMHEAD_ERR_NULL;
  if (!aligned(d_out, 16) || !aligned(ids, 4) || !aligned(workspace, 256)) return LMHEAD_ERR_ALIGN;
  if (workspace_bytes < lmhead_embedding_grad_workspace_bytes(tokens, V, H))
    return LMHEAD_ERR_SHAPE;
  const Region in[2] = {{d_out, tokens * H * 2}, {ids, tokens * 4}};
  const Region out[2] = {{d_W, V * H * 2}, {workspace, (int64_t)workspace_bytes}};
  st = check_overlap(in, 2, out, 2);
  if (st != LMHEAD_OK) return st;
  if ((H + lmh::kSumCols - 1) / lmh::kSumCols > 65535) return LMHEAD_ERR_SHAPE;  // grid rows
  st = current_device(&dev);
  if (st != LMHEAD_OK) return st;
  const EmbedPlan e = embed_plan(tokens, V, H);
  Carver c(workspace);
  const EmbedScratch s = carve_embed(c, e, tokens, V, H);
  return cleared(run_embed_grad(dev, d_out, dtype, ids, tokens, V, v_begin, H, scale, d_W,
                                accumulate, e, s, stream));
}

}  // extern "C"
