// cache_capi.cu -- entry points of the paged key/value cache: argument validation, launch shapes.
// (A translation unit of its own, compiled beside fp8q_capi.cu.)
#include "host_launch.cuh"
#include "cache_kernels.cuh"
#include "paged_attention_kernels.cuh"

using namespace fp8q_host;

namespace fp8q_host {

fp8q_status take_cache_device_error(unsigned int* bits) {
  const unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(bits, fp8q::g_device_error, sizeof *bits);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpyFromSymbol(g_device_error)");
  e = cudaMemcpyToSymbol(fp8q::g_device_error, &zero, sizeof zero);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpyToSymbol(g_device_error)");
  return FP8Q_OK;
}

}  // namespace fp8q_host

namespace {

constexpr int64_t kMaxHeads = 4096, kMaxLd = int64_t(1) << 40, kMaxTokens = int64_t(1) << 40;

// Rows of `width` bytes at a stride of `ld` bytes.
struct Strided {
  const void* p;
  int64_t rows, ld, width;
};

bool same(const Strided& a, const Strided& b) {
  return a.p == b.p && a.rows == b.rows && a.width == b.width && (a.rows <= 1 || a.ld == b.ld);
}

// Whether two arrays of rows share a byte. Rows at one stride (column slices of a packed array) are
// compared column by column; at different strides the arrays' extents count.
bool overlap(const Strided& a, const Strided& b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0) return false;
  const Range ra{a.p, size_t((a.rows - 1) * a.ld + a.width)};
  const Range rb{b.p, size_t((b.rows - 1) * b.ld + b.width)};
  if (!fp8q_host::overlap(ra, rb)) return false;
  if (a.ld != b.ld) return true;
  const int64_t d = int64_t(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
  const int64_t m = ((d % a.ld) + a.ld) % a.ld;  // where b's columns begin in a's rows
  return m < a.width || m + b.width > a.ld;
}

Strided flat(const void* p, int64_t bytes) { return Strided{p, bytes > 0 ? 1 : 0, bytes, bytes}; }

fp8q_status check_cache_shape(const fp8q_paged_cache& c) {
  if (c.type != FP8Q_INT8 && c.type != FP8Q_E4M3 && c.type != FP8Q_BF16) return FP8Q_ERR_VALUE;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return FP8Q_ERR_SHAPE;
  if (c.heads < 1 || c.heads > kMaxHeads || c.page_size < 16 || c.page_size > 1024 ||
      c.page_size % 16 != 0 || c.pages < 0 || c.pages > INT32_MAX ||
      c.pages * c.page_size >= (int64_t(1) << 47))
    return FP8Q_ERR_SHAPE;
  const int64_t page = c.heads * c.page_size * c.head_dim;
  for (int64_t s : {c.k_stride, c.v_stride})
    if (s < page || s % 16 != 0 || s > kMaxLd / 16) return FP8Q_ERR_SHAPE;
  if (c.type != FP8Q_BF16)
    for (int64_t s : {c.k_scale_stride, c.v_scale_stride})
      if (s < c.heads * c.page_size || s % 4 != 0 || s > kMaxLd / 16) return FP8Q_ERR_SHAPE;
  return FP8Q_OK;
}

fp8q_status check_cache_pointers(const fp8q_paged_cache& c) {
  const bool scaled = c.type != FP8Q_BF16;
  if (c.pages == 0) return FP8Q_OK;
  if (!c.k || !c.v || (scaled && (!c.k_scale || !c.v_scale))) return FP8Q_ERR_NULL;
  if (!aligned16(c.k) || !aligned16(c.v) || !aligned16(c.k_scale) || !aligned16(c.v_scale))
    return FP8Q_ERR_ALIGN;
  return FP8Q_OK;
}

fp8q::CacheView view(const fp8q_paged_cache& c) {
  const int64_t size = c.type == FP8Q_BF16 ? 2 : 1;
  fp8q::CacheView v{};
  v.k = static_cast<uint8_t*>(c.k);
  v.v = static_cast<uint8_t*>(c.v);
  v.k_scale = c.k_scale;
  v.v_scale = c.v_scale;
  v.k_stride = c.k_stride * size;
  v.v_stride = c.v_stride * size;
  v.ks_stride = c.k_scale_stride;
  v.vs_stride = c.v_scale_stride;
  v.pages = c.pages;
  v.page_magic = UINT64_MAX / uint64_t(c.page_size) + 1;  // ceil(2^64 / page_size)
  v.page_size = int(c.page_size);
  v.heads = int(c.heads);
  return v;
}

// The cache's four arrays as rows of pages.
struct CacheRows {
  Strided a[4];
  int n;
};
CacheRows cache_rows(const fp8q_paged_cache& c) {
  const int64_t size = c.type == FP8Q_BF16 ? 2 : 1, rows = c.heads * c.page_size;
  CacheRows r;
  r.n = c.type == FP8Q_BF16 ? 2 : 4;
  r.a[0] = Strided{c.k, c.pages, c.k_stride * size, rows * c.head_dim * size};
  r.a[1] = Strided{c.v, c.pages, c.v_stride * size, rows * c.head_dim * size};
  r.a[2] = Strided{c.k_scale, c.pages, c.k_scale_stride * 4, rows * 4};
  r.a[3] = Strided{c.v_scale, c.pages, c.v_scale_stride * 4, rows * 4};
  return r;
}

fp8q_status check_rotary(const fp8q_rotary* r, int64_t tokens, int64_t head_dim) {
  if (!r) return FP8Q_OK;
  if (r->pairs < 1 || r->pairs > head_dim / 2 || r->axes < 1) return FP8Q_ERR_SHAPE;
  if (!r->interleaved && r->pairs != head_dim / 2 && r->pairs % 8 != 0) return FP8Q_ERR_SHAPE;
  if (r->axes > 1 && (r->position_stride < tokens || r->position_stride > kMaxLd))
    return FP8Q_ERR_SHAPE;
  if (r->position_bytes != 4 && r->position_bytes != 8) return FP8Q_ERR_VALUE;
  return FP8Q_OK;
}

fp8q_status check_rotary_pointers(const fp8q_rotary* r) {
  if (!r) return FP8Q_OK;
  if (!r->inv_freq || !r->positions) return FP8Q_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(r->inv_freq) & 7) != 0 || !aligned4(r->axis) ||
      (reinterpret_cast<uintptr_t>(r->positions) & uintptr_t(r->position_bytes - 1)) != 0)
    return FP8Q_ERR_ALIGN;
  return FP8Q_OK;
}

bool fine_rows(int64_t ld, int64_t heads, int64_t head_dim) {
  return ld >= heads * head_dim && ld % 8 == 0 && ld <= kMaxLd / 16;
}

template <int D, int ROPE, bool CACHE, int TYPE>
fp8q_status launch_heads(fp8q::HeadsParams p, const DeviceInfo& dev, cudaStream_t stream) {
  auto* fn = fp8q::heads_kernel<D, ROPE, CACHE, TYPE>;
  constexpr int kWarps = fp8q::kHeadsThreads / 32, HPW = 32 / (D / 16);
  int bps = 0;
  const fp8q_status st = blocks_per_sm(reinterpret_cast<const void*>(fn), fp8q::kHeadsThreads, 0, &bps);
  if (st != FP8Q_OK) return st;
  const int64_t resident = int64_t(dev.sms) * std::max(bps, 1);
  const int steps = (p.q_heads + HPW - 1) / HPW + (CACHE ? 2 : 1) * ((p.kv_heads + HPW - 1) / HPW);
  // Tokens a group, by the rounds of groups and a round's length: a warp's steps and about one step's
  // time for the barrier (8192 tokens of 48 + 8 heads: 49.9 us with three, 45.5 with one, 62 with none).
  p.group_tokens = 1;
  int64_t best = INT64_MAX;
  const int most = std::min(fp8q::kHeadsTokens, 2 * fp8q::kHeadsAngles * fp8q::kHeadsThreads / D);
  for (int t = 1; t <= most; t *= 2) {
    const int64_t rounds = ((p.tokens + t - 1) / t + resident - 1) / resident;
    const int64_t cost = rounds * ((steps * t + kWarps - 1) / kWarps + 1);
    if (cost < best) best = cost, p.group_tokens = t;
  }
  // With few tokens, as many CTAs a token as have a step for each warp.
  p.parts = int(std::max<int64_t>(
      1, std::min<int64_t>((steps + kWarps - 1) / kWarps, resident / std::min(p.tokens, resident))));
  const int64_t groups = (p.tokens + p.group_tokens - 1) / p.group_tokens;
  const int64_t grid = std::min<int64_t>(groups, std::max<int64_t>(resident / p.parts, 1)) * p.parts;
  return launch(fn, dim3(unsigned(grid)), dim3(fp8q::kHeadsThreads), 0, stream, p);
}

template <int D, int ROPE>
fp8q_status launch_heads_type(const fp8q::HeadsParams& p, int type, const DeviceInfo& dev,
                              cudaStream_t stream) {
  switch (type) {
    case FP8Q_INT8: return launch_heads<D, ROPE, true, fp8q::kCacheInt8>(p, dev, stream);
    case FP8Q_E4M3: return launch_heads<D, ROPE, true, fp8q::kCacheE4m3>(p, dev, stream);
    case FP8Q_BF16: return launch_heads<D, ROPE, true, fp8q::kCacheBf16>(p, dev, stream);
    default: return launch_heads<D, ROPE, false, fp8q::kCacheBf16>(p, dev, stream);
  }
}

template <int D>
fp8q_status launch_heads_rope(const fp8q::HeadsParams& p, const fp8q_rotary* r, int type,
                              const DeviceInfo& dev, cudaStream_t stream) {
  if (!r) return launch_heads_type<D, fp8q::kRopeNone>(p, type, dev, stream);
  if (r->interleaved) return launch_heads_type<D, fp8q::kRopePairs>(p, type, dev, stream);
  return launch_heads_type<D, fp8q::kRopeHalves>(p, type, dev, stream);
}

// type: of the cache, -1 without one.
fp8q_status launch_heads_any(fp8q::HeadsParams& p, const fp8q_rotary* r, int64_t head_dim, int type,
                             const DeviceInfo& dev, cudaStream_t stream) {
  if (r) {
    p.rope.inv_freq = r->inv_freq;
    p.rope.axis = r->axis;
    p.rope.positions = r->positions;
    p.rope.stride = r->position_stride;
    p.rope.axes = r->axes;
    p.rope.pairs = r->pairs;
    p.rope.wide = r->position_bytes == 8;
  }
  switch (head_dim) {
    case 64: return launch_heads_rope<64>(p, r, type, dev, stream);
    case 128: return launch_heads_rope<128>(p, r, type, dev, stream);
    default: return launch_heads_rope<256>(p, r, type, dev, stream);
  }
}

// ------------------------------------------------------------------------------------------

template <int TYPE, int D>
fp8q_status launch_read(const fp8q::ReadParams& p, cudaStream_t stream) {
  const int64_t grid = (p.rows + fp8q::kReadRows - 1) / fp8q::kReadRows;
  if (grid > INT32_MAX) return FP8Q_ERR_SHAPE;
  return launch(fp8q::cache_read_kernel<D, TYPE>, dim3(unsigned(grid)), dim3(fp8q::kReadThreads), 0,
                stream, p);
}

template <int TYPE>
fp8q_status launch_read_dim(const fp8q::ReadParams& p, int64_t head_dim, cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_read<TYPE, 64>(p, stream);
    case 128: return launch_read<TYPE, 128>(p, stream);
    default: return launch_read<TYPE, 256>(p, stream);
  }
}

// ------------------------------------------------------------------------------------------

// Columns (query heads) of a block: 16 where a group has more than eight and the sums of both
// fit the registers.
int attn_columns(int64_t group, int64_t head_dim) { return group > 8 && head_dim <= 128 ? 2 : 1; }

struct AttnShape {
  int nt, blocks, warps, grid, ctas, segments;
  bool join;  // sequences may be long enough for several CTAs
};

AttnShape attn_shape(const fp8q_paged_cache& c, int64_t batch, int64_t q_heads, int64_t width,
                     int sms) {
  AttnShape s;
  const int64_t group = q_heads / c.heads;
  s.nt = attn_columns(group, c.head_dim);
  s.blocks = int((group + 8 * s.nt - 1) / (8 * s.nt));
  const int64_t most = width * (c.page_size / 16);  // tiles of a sequence
  const int64_t segments = batch * c.heads * s.blocks;
  s.warps = fp8q::attn_warps(c.type, int(c.head_dim), s.nt);
  s.segments = int(segments);
  s.grid = int(std::min<int64_t>(sms * fp8q::attn_ctas(c.type, int(c.head_dim), s.nt), segments * std::max<int64_t>(most, 1)));
  // (as many tiles a warp as kMuchWork at least, if every sequence fills its table)
  const bool much = segments * most >= int64_t(fp8q::kMuchWork) * s.grid * s.warps;
  s.ctas = s.grid * (much && 2 * segments >= s.grid && (s.nt == 1 || c.type == FP8Q_BF16) ? 2 : 1);
  s.join = most > s.warps;  // (AttnSplit: by tile only then)
  return s;
}

fp8q_status check_attention(const fp8q_paged_cache& c, int64_t batch, int64_t q_heads,
                            int64_t width) {
  const fp8q_status st = check_cache_shape(c);
  if (st != FP8Q_OK) return st;
  if (batch < 0 || batch > (1 << 20) || q_heads < 1 || q_heads > kMaxHeads * 64 ||
      q_heads % c.heads != 0 || batch * q_heads > INT32_MAX || width < 0 ||
      width * c.page_size >= (int64_t(1) << 30) ||
      // (tiles of a sequence over all heads, of all sequences, with what the split adds to each; of all
      // over all, so that a warp's share stays below 2^31 where 512 warps are resident)
      (width * (c.page_size / 16) + fp8q::kAttnExtra) * std::max(q_heads, batch) > INT32_MAX ||
      (width * (c.page_size / 16) + fp8q::kAttnExtra) * batch * q_heads > (int64_t(1) << 40))
    return FP8Q_ERR_SHAPE;
  return FP8Q_OK;
}

// A slot for each warp and two for each CTA (AttnParams::part_o, part_ml).
int64_t workspace_slots(const AttnShape& s) { return int64_t(s.ctas) * (s.warps + 2); }
int64_t workspace_bytes_of(const AttnShape& s, int64_t head_dim) {
  return s.join ? (workspace_slots(s) * head_dim + int64_t(2) * s.ctas * 2) * 8 * s.nt * 4 : 0;
}

fp8q::FastDiv fast_div_by(int64_t d) { return fp8q::FastDiv{d == 1 ? 0 : UINT64_MAX / uint64_t(d) + 1}; }

// Tensor map of a cache's pages: lines of 128 bytes at least, boxes of 16 tokens by 128 bytes.
template <typename L>
fp8q_status tile_map(CUtensorMap* map, uint8_t* pages, int64_t page_bytes, const fp8q::CacheView& c) {
  EncodeTiled fn = nullptr;
  const fp8q_status st = encode_tiled(&fn);
  if (st != FP8Q_OK) return st;
  const cuuint64_t lines = cuuint64_t(c.heads) * c.page_size * L::kLines / 16;
  const cuuint64_t dims[3] = {cuuint64_t(L::kLine), lines, cuuint64_t(std::max<int64_t>(c.pages, 1))};
  const cuuint64_t strides[2] = {cuuint64_t(L::kLine), cuuint64_t(page_bytes)};
  const cuuint32_t box[3] = {128, cuuint32_t(L::kLines), 1};
  const cuuint32_t steps[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, pages, dims, strides, box, steps,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return cuda_fail(cudaErrorInvalidValue, "cuTensorMapEncodeTiled", r);
  return FP8Q_OK;
}

template <int TYPE, int D, int NT>
fp8q_status launch_attention(const fp8q::AttnParams& p, const AttnShape& s, cudaStream_t stream) {
  using L = fp8q::AttnLayout<TYPE, D, NT>;
  static_assert(L::kStages >= 2 && L::kStages <= 16 && L::kBytes <= L::kMost, "a ring fits its SM's share");
  static_assert(L::kItems % (2 * fp8q::kJoinItems) == 0, "whole CTAs of the join");
  auto* fn = fp8q::paged_attention_kernel<TYPE, D, NT>;
  int bps = 0;
  fp8q_status st = blocks_per_sm(reinterpret_cast<const void*>(fn), L::kWarps * 32, L::kBytes, &bps);
  if (st != FP8Q_OK) return st;
  if (bps <= 0) return cuda_fail(cudaErrorInvalidConfiguration, "occupancy", (long long)L::kBytes);
  CUtensorMap map_k, map_v;
  // (without pages nothing is read, but a map wants an address)
  uint8_t* none = reinterpret_cast<uint8_t*>(const_cast<uint16_t*>(p.q));
  st = tile_map<L>(&map_k, p.cache.pages > 0 ? p.cache.k : none, p.cache.k_stride, p.cache);
  if (st != FP8Q_OK) return st;
  st = tile_map<L>(&map_v, p.cache.pages > 0 ? p.cache.v : none, p.cache.v_stride, p.cache);
  if (st != FP8Q_OK) return st;
  st = launch(fn, dim3(unsigned(s.ctas)), dim3(L::kWarps * 32), size_t(L::kBytes), stream, p, map_k,
              map_v);
  if (st != FP8Q_OK || !s.join) return st;
  // Two parts of a piece a CTA of the join where there would be more than kJoinMany CTAs an SM.
  constexpr int kGroups = L::kItems / fp8q::kJoinItems;
  const int segments = std::min(p.segments, p.ctas);
  if (segments * kGroups > fp8q::kJoinMany * (p.grid / L::kCtas))
    return launch(fp8q::attn_join_kernel<TYPE, D, NT, 2>, dim3(unsigned(segments), kGroups / 2),
                  dim3(fp8q::kJoinWarps * 32), 0, stream, p);
  return launch(fp8q::attn_join_kernel<TYPE, D, NT, 1>, dim3(unsigned(segments), kGroups),
                dim3(fp8q::kJoinWarps * 32), 0, stream, p);
}

template <int TYPE>
fp8q_status launch_attention_dim(const fp8q::AttnParams& p, const AttnShape& s, int64_t head_dim,
                                 cudaStream_t stream) {
  switch (head_dim) {
    case 64:
      return s.nt == 2 ? launch_attention<TYPE, 64, 2>(p, s, stream)
                       : launch_attention<TYPE, 64, 1>(p, s, stream);
    case 128:
      return s.nt == 2 ? launch_attention<TYPE, 128, 2>(p, s, stream)
                       : launch_attention<TYPE, 128, 1>(p, s, stream);
    default: return launch_attention<TYPE, 256, 1>(p, s, stream);
  }
}

}  // namespace

extern "C" {

fp8q_status fp8q_qk_norm_rope(void* q_out, int64_t q_out_ld, void* k_out, int64_t k_out_ld,
                              const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                              const void* q_weight, const void* k_weight, float eps,
                              const fp8q_rotary* rotary, int64_t tokens, int64_t q_heads,
                              int64_t kv_heads, int64_t head_dim, cudaStream_t stream) {
  if (tokens < 0 || tokens > kMaxTokens || q_heads < 1 || kv_heads < 1 || q_heads > kMaxHeads ||
      kv_heads > kMaxHeads || (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return FP8Q_ERR_SHAPE;
  if (!fine_rows(q_ld, q_heads, head_dim) || !fine_rows(q_out_ld, q_heads, head_dim) ||
      !fine_rows(k_ld, kv_heads, head_dim) || !fine_rows(k_out_ld, kv_heads, head_dim))
    return FP8Q_ERR_SHAPE;
  fp8q_status st = check_rotary(rotary, tokens, head_dim);
  if (st != FP8Q_OK) return st;
  if ((q_weight || k_weight) && !(eps > 0.0f && std::isfinite(eps))) return FP8Q_ERR_VALUE;
  if (tokens == 0) return FP8Q_OK;
  if (!q_out || !k_out || !q || !k) return FP8Q_ERR_NULL;
  st = check_rotary_pointers(rotary);
  if (st != FP8Q_OK) return st;
  for (const void* p : {static_cast<const void*>(q_out), static_cast<const void*>(k_out), q, k,
                        q_weight, k_weight})
    if (!aligned16(p)) return FP8Q_ERR_ALIGN;
  const int64_t qw = q_heads * head_dim * 2, kw = kv_heads * head_dim * 2;
  const Strided qo{q_out, tokens, q_out_ld * 2, qw}, ko{k_out, tokens, k_out_ld * 2, kw};
  const Strided qi{q, tokens, q_ld * 2, qw}, ki{k, tokens, k_ld * 2, kw};
  if (overlap(qo, ko)) return FP8Q_ERR_ALIAS;
  if ((overlap(qo, qi) && !same(qo, qi)) || overlap(qo, ki)) return FP8Q_ERR_ALIAS;
  if ((overlap(ko, ki) && !same(ko, ki)) || overlap(ko, qi)) return FP8Q_ERR_ALIAS;
  for (const Strided& o : {qo, ko}) {
    if (overlap(o, flat(q_weight, head_dim * 2)) || overlap(o, flat(k_weight, head_dim * 2)))
      return FP8Q_ERR_ALIAS;
    if (rotary && (overlap(o, flat(rotary->inv_freq, int64_t(rotary->pairs) * 8)) ||
                   overlap(o, flat(rotary->axis, int64_t(rotary->pairs) * 4)) ||
                   overlap(o, Strided{rotary->positions, rotary->axes,
                                      rotary->position_stride * rotary->position_bytes,
                                      tokens * rotary->position_bytes})))
      return FP8Q_ERR_ALIAS;
  }
  const DeviceInfo* dev = nullptr;
  st = current_device(&dev);
  if (st != FP8Q_OK) return st;
  fp8q::HeadsParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.q_ld = q_ld;
  p.k_ld = k_ld;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_out = static_cast<uint16_t*>(k_out);
  p.q_out_ld = q_out_ld;
  p.k_out_ld = k_out_ld;
  p.q_weight = static_cast<const uint16_t*>(q_weight);
  p.k_weight = static_cast<const uint16_t*>(k_weight);
  p.tokens = tokens;
  p.q_heads = int(q_heads);
  p.kv_heads = int(kv_heads);
  p.eps = eps;
  return launch_heads_any(p, rotary, head_dim, -1, *dev, stream);
}

fp8q_status fp8q_cache_write(const fp8q_paged_cache* cache, const int64_t* slots, void* q_out,
                             int64_t q_out_ld, const void* q, int64_t q_ld, const void* k,
                             int64_t k_ld, const void* v, int64_t v_ld, const void* q_weight,
                             const void* k_weight, float eps, const fp8q_rotary* rotary,
                             int64_t tokens, int64_t q_heads, cudaStream_t stream) {
  if (!cache) return FP8Q_ERR_NULL;
  fp8q_status st = check_cache_shape(*cache);
  if (st != FP8Q_OK) return st;
  const int64_t head_dim = cache->head_dim, kv_heads = cache->heads;
  if (tokens < 0 || tokens > kMaxTokens || q_heads < 0 || q_heads > kMaxHeads) return FP8Q_ERR_SHAPE;
  if (!fine_rows(k_ld, kv_heads, head_dim) || !fine_rows(v_ld, kv_heads, head_dim) ||
      (q_heads > 0 && (!fine_rows(q_ld, q_heads, head_dim) || !fine_rows(q_out_ld, q_heads, head_dim))))
    return FP8Q_ERR_SHAPE;
  st = check_rotary(rotary, tokens, head_dim);
  if (st != FP8Q_OK) return st;
  if ((q_weight || k_weight) && !(eps > 0.0f && std::isfinite(eps))) return FP8Q_ERR_VALUE;
  if (tokens == 0) return FP8Q_OK;
  if (!k || !v || !slots || (q_heads > 0 && (!q || !q_out))) return FP8Q_ERR_NULL;
  st = check_cache_pointers(*cache);
  if (st != FP8Q_OK) return st;
  st = check_rotary_pointers(rotary);
  if (st != FP8Q_OK) return st;
  if (q_heads == 0) q = q_out = nullptr;
  for (const void* p : {static_cast<const void*>(q_out), q, k, v, q_weight, k_weight})
    if (!aligned16(p)) return FP8Q_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(slots) & 7) != 0) return FP8Q_ERR_ALIGN;
  const int64_t qw = q_heads * head_dim * 2, kw = kv_heads * head_dim * 2;
  const Strided qo{q_out, tokens, q_out_ld * 2, qw}, qi{q, tokens, q_ld * 2, qw};
  const CacheRows rows = cache_rows(*cache);
  Strided outs[5];
  int n = 0;
  outs[n++] = qo;
  for (int i = 0; i < rows.n; ++i) outs[n++] = rows.a[i];
  const Strided ins[] = {
      qi, Strided{k, tokens, k_ld * 2, kw}, Strided{v, tokens, v_ld * 2, kw},
      flat(slots, tokens * 8), flat(q_weight, head_dim * 2), flat(k_weight, head_dim * 2),
      rotary ? flat(rotary->inv_freq, int64_t(rotary->pairs) * 8) : flat(nullptr, 0),
      rotary ? flat(rotary->axis, int64_t(rotary->pairs) * 4) : flat(nullptr, 0),
      rotary ? Strided{rotary->positions, rotary->axes,
                       rotary->position_stride * rotary->position_bytes,
                       tokens * rotary->position_bytes}
             : flat(nullptr, 0)};
  for (int i = 0; i < n; ++i) {
    for (int j = i + 1; j < n; ++j)
      if (overlap(outs[i], outs[j])) return FP8Q_ERR_ALIAS;
    for (const Strided& in : ins)
      if (overlap(outs[i], in) && !(i == 0 && &in == &ins[0] && same(qo, qi))) return FP8Q_ERR_ALIAS;
  }
  const DeviceInfo* dev = nullptr;
  st = current_device(&dev);
  if (st != FP8Q_OK) return st;
  fp8q::HeadsParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_ld = q_ld;
  p.k_ld = k_ld;
  p.v_ld = v_ld;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.q_out_ld = q_out_ld;
  p.q_weight = static_cast<const uint16_t*>(q_weight);
  p.k_weight = static_cast<const uint16_t*>(k_weight);
  p.slots = slots;
  p.cache = view(*cache);
  p.tokens = tokens;
  p.q_heads = int(q_heads);
  p.kv_heads = int(kv_heads);
  p.eps = eps;
  return launch_heads_any(p, rotary, head_dim, cache->type, *dev, stream);
}

fp8q_status fp8q_cache_read(void* k_out, void* v_out, const fp8q_paged_cache* cache,
                            const int32_t* page_table, int64_t table_ld, int64_t width,
                            const int64_t* offsets, int64_t batch, int64_t rows,
                            cudaStream_t stream) {
  if (!cache) return FP8Q_ERR_NULL;
  fp8q_status st = check_cache_shape(*cache);
  if (st != FP8Q_OK) return st;
  if (rows < 0 || rows > kMaxTokens || batch < 0 || batch > INT32_MAX - 1 || width < 0 ||
      width > INT32_MAX || (batch > 1 && table_ld < width) || table_ld > kMaxLd)
    return FP8Q_ERR_SHAPE;
  if (rows == 0 || batch == 0) return FP8Q_OK;
  if (!k_out || !v_out || !offsets || (width > 0 && !page_table)) return FP8Q_ERR_NULL;
  st = check_cache_pointers(*cache);
  if (st != FP8Q_OK) return st;
  if (!aligned16(k_out) || !aligned16(v_out) || !aligned4(page_table) ||
      (reinterpret_cast<uintptr_t>(offsets) & 7) != 0)
    return FP8Q_ERR_ALIGN;
  const int64_t bytes = rows * cache->heads * cache->head_dim * 2;
  const Strided ko = flat(k_out, bytes), vo = flat(v_out, bytes);
  const CacheRows cr = cache_rows(*cache);
  if (overlap(ko, vo)) return FP8Q_ERR_ALIAS;
  for (const Strided& o : {ko, vo}) {
    for (int i = 0; i < cr.n; ++i)
      if (overlap(o, cr.a[i])) return FP8Q_ERR_ALIAS;
    if (overlap(o, Strided{page_table, batch, table_ld * 4, width * 4}) ||
        overlap(o, flat(offsets, (batch + 1) * 8)))
      return FP8Q_ERR_ALIAS;
  }
  const DeviceInfo* dev = nullptr;
  st = current_device(&dev);
  if (st != FP8Q_OK) return st;
  fp8q::ReadParams p{};
  p.cache = view(*cache);
  p.table = page_table;
  p.table_ld = table_ld;
  p.offsets = offsets;
  p.k = static_cast<uint16_t*>(k_out);
  p.v = static_cast<uint16_t*>(v_out);
  p.rows = rows;
  p.batch = int(batch);
  p.width = int(width);
  switch (cache->type) {
    case FP8Q_INT8: return launch_read_dim<fp8q::kCacheInt8>(p, cache->head_dim, stream);
    case FP8Q_E4M3: return launch_read_dim<fp8q::kCacheE4m3>(p, cache->head_dim, stream);
    default: return launch_read_dim<fp8q::kCacheBf16>(p, cache->head_dim, stream);
  }
}

int64_t fp8q_paged_attention_workspace(const fp8q_paged_cache* cache, int64_t batch,
                                       int64_t q_heads, int64_t width) {
  if (!cache || check_attention(*cache, batch, q_heads, width) != FP8Q_OK) return -1;
  const DeviceInfo* dev = nullptr;
  if (current_device(&dev) != FP8Q_OK) return -1;
  return workspace_bytes_of(attn_shape(*cache, batch, q_heads, width, dev->sms), cache->head_dim);
}

fp8q_status fp8q_paged_attention(void* out, float* lse, const void* q, int64_t q_ld,
                                 const fp8q_paged_cache* cache, const int32_t* page_table,
                                 int64_t table_ld, int64_t width, const int32_t* lengths,
                                 int64_t batch, int64_t q_heads, float scale, int64_t window,
                                 void* workspace, int64_t workspace_bytes, cudaStream_t stream) {
  if (!cache) return FP8Q_ERR_NULL;
  fp8q_status st = check_attention(*cache, batch, q_heads, width);
  if (st != FP8Q_OK) return st;
  if (!fine_rows(q_ld, q_heads, cache->head_dim) || (batch > 1 && table_ld < width) ||
      table_ld > kMaxLd)
    return FP8Q_ERR_SHAPE;
  const float scale_log2 = scale * 1.4426950408889634f;  // logits in log2 units
  if (!std::isfinite(scale_log2) || window < 0) return FP8Q_ERR_VALUE;
  if (batch == 0) return FP8Q_OK;
  if (!out || !q || !lengths || (width > 0 && !page_table)) return FP8Q_ERR_NULL;
  st = check_cache_pointers(*cache);
  if (st != FP8Q_OK) return st;
  if (!aligned16(out) || !aligned16(q) || !aligned4(lse) || !aligned4(page_table) ||
      !aligned4(lengths) || !aligned16(workspace))
    return FP8Q_ERR_ALIGN;
  const Strided o = flat(out, batch * q_heads * cache->head_dim * 2), l = flat(lse, batch * q_heads * 4);
  const Strided w = flat(workspace, workspace_bytes);
  const CacheRows cr = cache_rows(*cache);
  if (overlap(o, l) || overlap(o, w) || overlap(l, w)) return FP8Q_ERR_ALIAS;
  for (const Strided& x : {o, l, w}) {
    for (int i = 0; i < cr.n; ++i)
      if (overlap(x, cr.a[i])) return FP8Q_ERR_ALIAS;
    if (overlap(x, Strided{q, batch, q_ld * 2, q_heads * cache->head_dim * 2}) ||
        overlap(x, Strided{page_table, batch, table_ld * 4, width * 4}) ||
        overlap(x, flat(lengths, batch * 4)))
      return FP8Q_ERR_ALIAS;
  }
  const DeviceInfo* dev = nullptr;
  st = current_device(&dev);
  if (st != FP8Q_OK) return st;
  const AttnShape s = attn_shape(*cache, batch, q_heads, width, dev->sms);
  const int64_t need = workspace_bytes_of(s, cache->head_dim);
  if (need > 0 && !workspace) return FP8Q_ERR_NULL;
  if (workspace_bytes < need) return FP8Q_ERR_SHAPE;
  fp8q::AttnParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.q_ld = q_ld;
  p.cache = view(*cache);
  p.table = page_table;
  p.table_ld = table_ld;
  p.lengths = lengths;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = p.part_o ? reinterpret_cast<float2*>(p.part_o + workspace_slots(s) * 8 * s.nt * cache->head_dim)
                       : nullptr;
  p.batch = int(batch);
  p.width = cache->pages > 0 ? int(width) : 0;  // no page to read: no tokens
  p.window = int(std::min<int64_t>(window, INT32_MAX));
  p.q_heads = int(q_heads);
  p.group = int(q_heads / cache->heads);
  p.blocks = s.blocks;
  p.grid = s.grid;
  p.ctas = s.ctas;
  p.segments = s.segments;
  p.heads = int(cache->heads) * s.blocks;
  p.warp_rounds = int((int64_t(s.segments) + int64_t(s.grid) * s.warps - 1) / (int64_t(s.grid) * s.warps));
  p.by_warps = fast_div_by(int64_t(s.grid) * s.warps);
  p.by_heads = fast_div_by(p.heads);
  p.by_blocks = fast_div_by(p.blocks);
  p.scale_log2 = scale_log2;
  p.page_tiles = int(cache->page_size / 16);
  p.tile_magic = uint32_t(((int64_t(1) << 32) + p.page_tiles - 1) / p.page_tiles);
  switch (cache->type) {
    case FP8Q_INT8: return launch_attention_dim<fp8q::kCacheInt8>(p, s, cache->head_dim, stream);
    case FP8Q_E4M3: return launch_attention_dim<fp8q::kCacheE4m3>(p, s, cache->head_dim, stream);
    default: return launch_attention_dim<fp8q::kCacheBf16>(p, s, cache->head_dim, stream);
  }
}

}  // extern "C"
