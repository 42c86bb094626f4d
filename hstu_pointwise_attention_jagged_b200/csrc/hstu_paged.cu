// hstu_paged.cu — host side of the calls declared in include/hstu_paged.h: argument checks, launch
// shapes and tensor maps.  Nothing synchronises; nothing falls back to another path.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <utility>

#include "host_state.h"
#include "hstu_paged.h"
#include "paged_cache.cuh"
#include "paged_rows_sm100.cuh"
#include "paged_schedule.cuh"
#include "rotary_sm100.cuh"

namespace hstu {
namespace {

bool head_size_ok(int32_t d) { return d == 32 || d == 64 || d == 128; }

// Extents that no memory has are refused before anything is computed from them, and so are more users than a plan
// can number with their blocks, or a block's threads step over, in 32 bits.
constexpr int64_t kMaxElements = 1ll << 46;
constexpr int32_t kMaxUsers = 1 << 30;

// A token tensor's row stride: at least the packed row, a multiple of 16 bytes.
hstu_status_t check_ld(int64_t ld, int64_t width, int64_t rows) {
  if (ld < width) return HSTU_ERR_INVALID_ARGUMENT;
  return ld % 8 == 0 && ld <= kMaxElements / rows ? HSTU_OK : HSTU_ERR_UNSUPPORTED;
}

// Whether two row blocks of `width` elements share an element.  Blocks of one wide matrix (equal
// strides) interleave without touching: their columns are compared.
bool rows_overlap(const void* a, int64_t a_ld, const void* b, int64_t b_ld, int64_t rows, int64_t width) {
  if (!overlaps(a, static_cast<size_t>((rows - 1) * a_ld + width) * 2, b,
                static_cast<size_t>((rows - 1) * b_ld + width) * 2))
    return false;
  if (a_ld != b_ld) return true;
  int64_t off = (reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a)) / 2 % a_ld;
  if (off < 0) off += a_ld;
  return off < width || a_ld - off < width;
}

// An output that is its own input (same rows, same stride) is written by the thread that read it.
bool clashes(const void* out, int64_t out_ld, const void* in, int64_t in_ld, bool own, int64_t rows, int64_t width) {
  if (own && out == in && out_ld == in_ld) return false;
  return rows_overlap(out, out_ld, in, in_ld, rows, width);
}

hstu_status_t check_rotation(const hstu_rotation_t* r, int32_t d, int64_t rows, bool need_positions) {
  if (!r || r->pairs < 1 || r->axes < 1 || r->axes > HSTU_MAX_AXES) return HSTU_ERR_INVALID_ARGUMENT;
  if (2 * static_cast<int64_t>(r->pairs) > d) return HSTU_ERR_INVALID_ARGUMENT;
  int64_t sum = 0;
  for (int a = 0; a < r->axes; ++a) {
    if (r->sections[a] < 0) return HSTU_ERR_INVALID_ARGUMENT;
    sum += r->sections[a];
  }
  if (sum != r->pairs) return HSTU_ERR_INVALID_ARGUMENT;
  if (r->pairs % 8 != 0) return HSTU_ERR_UNSUPPORTED;
  if (rows == 0) return HSTU_OK;
  if (!r->freqs || (!r->positions && (need_positions || r->axes > 1))) return HSTU_ERR_INVALID_ARGUMENT;
  if (r->positions && r->axes > 1 && r->positions_ld < rows) return HSTU_ERR_INVALID_ARGUMENT;
  if ((reinterpret_cast<uintptr_t>(r->freqs) & 7u) || (reinterpret_cast<uintptr_t>(r->positions) & 3u))
    return HSTU_ERR_UNSUPPORTED;
  return HSTU_OK;
}

hstu_status_t check_cache(const hstu_paged_cache_t* c, int32_t d) {
  if (!c || !c->k || !c->v || c->num_pages < 1 || c->table_width < 0 || c->table_ld < c->table_width)
    return HSTU_ERR_INVALID_ARGUMENT;
  if (c->table_width > 0 && !c->page_table) return HSTU_ERR_INVALID_ARGUMENT;
  if (c->page_size < 8 || c->page_size > 1024 || (c->page_size & (c->page_size - 1))) return HSTU_ERR_UNSUPPORTED;
  const int64_t strides[3] = {c->page_stride, c->row_stride, c->head_stride};
  for (int64_t s : strides) {
    if (s < d) return HSTU_ERR_INVALID_ARGUMENT;
    if (s % 8 != 0 || s > (1ll << 38)) return HSTU_ERR_UNSUPPORTED;  // tensor-map strides are < 2^40 bytes
  }
  if (c->page_stride > kMaxElements / c->num_pages) return HSTU_ERR_UNSUPPORTED;
  if (!aligned16(c->k) || !aligned16(c->v) || (reinterpret_cast<uintptr_t>(c->page_table) & 3u))
    return HSTU_ERR_UNSUPPORTED;
  return HSTU_OK;
}

// Bytes from the first to past the last element of K (and of V).
size_t cache_bytes(const hstu_paged_cache_t& c, int32_t H, int32_t d) {
  return static_cast<size_t>((c.num_pages - 1) * c.page_stride + (c.page_size - 1) * c.row_stride +
                             static_cast<int64_t>(H - 1) * c.head_stride + d) * 2;
}

// The dimensions of K (and of V) beside the columns, by increasing stride; a dimension of one entry has no stride.
struct CacheAxes {
  int64_t n[3], stride[3];
};

CacheAxes cache_axes(const hstu_paged_cache_t& c, int32_t H) {
  CacheAxes a = {{c.num_pages, c.page_size, H}, {c.page_stride, c.row_stride, c.head_stride}};
  for (int i = 0; i < 3; ++i)
    if (a.n[i] == 1) a.stride[i] = 0;
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (a.stride[j] > a.stride[j + 1]) {
        std::swap(a.stride[j], a.stride[j + 1]);
        std::swap(a.n[j], a.n[j + 1]);
      }
  return a;
}

// Whether rows of K can share elements: every stride has to step over all that the smaller ones reach.
bool rows_share(const CacheAxes& a, int32_t d) {
  int64_t extent = d;
  for (int i = 0; i < 3; ++i) {
    if (a.n[i] == 1) continue;
    if (a.stride[i] < extent) return true;
    extent += (a.n[i] - 1) * a.stride[i];
  }
  return false;
}

// Whether two caches of this form, `delta` elements apart, share an element.  With rows that share none, the
// steps along an axis that bring `delta` within the reach of the smaller strides are the two next to
// delta / stride.
bool caches_meet(const CacheAxes& a, int32_t d, int64_t delta, int i = 2) {
  if (i < 0) return -d < delta && delta < d;
  if (a.n[i] == 1) return caches_meet(a, d, delta, i - 1);
  int64_t step = delta / a.stride[i];
  if (step * a.stride[i] > delta) --step;
  for (int k = 0; k < 2; ++k, ++step)
    if (-a.n[i] < step && step < a.n[i] && caches_meet(a, d, delta - step * a.stride[i], i - 1)) return true;
  return false;
}

PagedView view_of(const hstu_paged_cache_t& c) {
  PagedView v;
  v.k = static_cast<__nv_bfloat16*>(c.k);
  v.v = static_cast<__nv_bfloat16*>(c.v);
  v.page_stride = c.page_stride;
  v.row_stride = c.row_stride;
  v.head_stride = c.head_stride;
  v.num_pages = c.num_pages;
  v.page_shift = __builtin_ctz(static_cast<unsigned>(c.page_size));
  v.table = c.page_table;
  v.table_width = c.table_width;
  v.table_ld = c.table_ld;
  return v;
}

void add_tensor(RotArgs& a, const void* src, int64_t ld, void* dst, int64_t dst_ld, RotTarget target, bool rotated) {
  RotTensor& t = a.t[a.tensors++];
  t.src = static_cast<const __nv_bfloat16*>(src);
  t.src_ld = ld;
  t.dst = static_cast<__nv_bfloat16*>(dst);
  t.dst_ld = dst_ld;
  t.target = target;
  t.rotated = rotated;
}

void set_rotation(RotArgs& a, const hstu_rotation_t* r, bool inverse) {
  if (!r) return;
  a.freqs = r->freqs;
  a.positions = r->positions;
  a.positions_ld = r->positions_ld;
  a.pairs = r->pairs;
  a.axes = r->axes;
  int32_t end = 0;
  for (int i = 0; i + 1 < r->axes; ++i) a.section_end[i] = end += r->sections[i];
  a.interleaved = r->interleaved != 0;
  a.sign = inverse ? -1.0f : 1.0f;
}

// Programmatic dependents of the previous kernel in the stream: a launch's set-up overlaps that kernel's
// tail, and the kernel waits for it (griddepcontrol.wait) before touching global memory.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), int64_t grid, int threads, int smem, int cluster,
                             cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Shape of the rotation's blocks: as many rows side by side as have a thread for each unit, and
// kRotBatch x kRotPasses units for each thread; fewer rows where that would leave SMs without a block (a
// call for a few rows is bound by the latency of one block).
hstu_status_t launch_rotary(RotArgs& a, int32_t d, bool paged, const DeviceState& st, cudaStream_t stream) {
  a.head_shift = d == 128 ? 3 : (d == 64 ? 2 : 1);
  const int64_t units = static_cast<int64_t>(a.tensors) * a.H << a.head_shift;
  if (units > INT_MAX / 2) return HSTU_ERR_UNSUPPORTED;
  const int spread = a.rows / (2 * st.num_sms) > 1 ? a.rows / (2 * st.num_sms) : 1;
  auto at_most = [](int64_t x, int64_t y) { return static_cast<int32_t>(x < y ? x : y); };
  a.row_units = static_cast<int32_t>(units);
  a.side_rows = units < kRotThreads ? at_most(kRotThreads / units, kRotSideRows) : 1;
  a.side_rows = at_most(a.side_rows, spread);
  a.block_rows = at_most(a.side_rows * kRotBatch * kRotPasses, spread);
  int threads = at_most((a.side_rows * units + 31) / 32 * 32, kRotThreads);
  if (threads < 64) threads = 64;  // the angles and the look-ups: at least one thread a pair, and one a row
  static_assert(kRotMaxPairs <= 64 && kRotMaxRows <= 64, "threads of the smallest block");
  const int64_t grid = (static_cast<int64_t>(a.rows) + a.block_rows - 1) / a.block_rows;
  const int smem = a.block_rows * a.pairs * 8;
  const cudaError_t e = paged ? launch_dependent(rotary_kernel<true>, grid, threads, smem, 0, stream, a)
                              : launch_dependent(rotary_kernel<false>, grid, threads, smem, 0, stream, a);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

// Sets a kernel up once for each device.
constexpr int kMaxDevices = 64;

template <typename F>
cudaError_t once_per_device(std::once_flag (&once)[kMaxDevices], cudaError_t (&result)[kMaxDevices], F&& f) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [&] { result[dev] = f(); });
  return result[dev];
}

// How the few-rows kernels would take a call.
struct RowsShape {
  bool clustered;  // clusters of `cluster` CTAs (else equal runs)
  int cluster;
  bool few;        // the few-rows kernels are the ones to take it
};

// Clusters as large as keeps every CTA resident at once and busy with two tiles, if that leaves each CTA a
// short stretch of tiles: then one launch does it all.  A long stretch takes the equal runs, which ragged
// lengths cannot unbalance.  (us, clusters against runs, d = 128, one row a user: 64 users x 4 heads of 700
// rows, 11 tiles a CTA, 17.6 against 23.4; 16 x 4 of 3000, 12 tiles, 19.9 against 23.1; 64 x 4 of ragged
// histories up to 4096, 65 tiles, 57 against 40; 1 x 4 of 32000, 32 tiles, 27.7 against 18.8.)
//
// More than 16 rows a user come here while the call is short.  Every block of 16 rows reads all keys again,
// but the tcgen05 kernel has its plan, its fill and tiles of 128 rows to pay for.  (us, here against there:
// 4 users x 4 heads of 100 rows over 1000, d = 128, 13.1 against 18.0; 1 x 4 of 256 over 2000, 13.7 against
// 24.9; 16 x 4 of 80 over 300, 14.5 against 13.6; 64 x 4 of 24 over 300, 17.6 against 21.0.)  The limits were set at
// d = 128; they count tiles of 16 KB, so in keys they grow with 1 / d.
RowsShape rows_shape(const RowsArgs& a, int keys, int num_sms) {
  const int64_t items = static_cast<int64_t>(a.B) * a.H * a.blocks;
  const int64_t tiles = a.max_kv / keys + 1;  // of an item, at most
  RowsShape s;
  s.cluster = 1;
  while (s.cluster < kRowsMaxSplit && 2 * s.cluster * items <= 2 * num_sms && 4 * s.cluster <= tiles) s.cluster *= 2;
  const int64_t stretch = (tiles + s.cluster - 1) / s.cluster;
  s.clustered = stretch <= kRowsClusterTiles || a.B > kRunUsers || items * tiles > INT_MAX;
  s.few = a.blocks == 1;
  if (a.blocks > 1) {
    s.few = stretch <= kRowsClusterTiles && items * tiles <= 2 * num_sms * kRowsBlocksTiles;
    s.clustered = true;
  }
  return s;
}

// A few rows a user; R: rows of an item at most.
template <int D, int R>
hstu_status_t launch_rows(const RowsArgs& a, const DeviceState& st, cudaStream_t stream) {
  using Cfg = RowsCfg<D>;
  static std::once_flag once[kMaxDevices];
  static cudaError_t ready[kMaxDevices];
  cudaError_t e = once_per_device(once, ready, [] {
    cudaError_t r = cudaFuncSetAttribute(paged_rows_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmemBytes);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(paged_rows_kernel<D, R>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (r == cudaSuccess)
      r = cudaFuncSetAttribute(paged_rows_run_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmemBytes);
    return r;
  });
  if (e != cudaSuccess) return HSTU_ERR_CUDA;
  const RowsShape shape = rows_shape(a, Cfg::kKeys, st.num_sms);
  const int64_t items = static_cast<int64_t>(a.B) * a.H * a.blocks;
  if (shape.clustered) {
    if (items * shape.cluster > INT_MAX) return HSTU_ERR_UNSUPPORTED;
    e = launch_dependent(paged_rows_kernel<D, R>, items * shape.cluster, kRowsThreads, Cfg::kSmemBytes, shape.cluster, stream,
                         a);
    return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
  }
  const int runs = 2 * st.num_sms;
  const size_t parts_bytes = (static_cast<size_t>(items) * sizeof(int2) + 255) / 256 * 256;
  void* buf = nullptr;
  if (cudaMallocFromPoolAsync(&buf, parts_bytes + static_cast<size_t>(2 * runs) * kRowsBlock * D * 4, st.pool, stream) !=
      cudaSuccess)
    return HSTU_ERR_CUDA;
  RunsArgs r;
  r.rows = a;
  r.parts = static_cast<int2*>(buf);
  r.sums = reinterpret_cast<float*>(static_cast<uint8_t*>(buf) + parts_bytes);
  e = launch_dependent(paged_rows_run_kernel<D, R>, runs, kRowsThreads, Cfg::kSmemBytes, 0, stream, r);
  if (e == cudaSuccess) e = launch_dependent(paged_rows_sum_kernel<D>, items, kSumThreads, 0, 0, stream, r);
  if (cudaFreeAsync(buf, stream) != cudaSuccess && e == cudaSuccess) return HSTU_ERR_CUDA;
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

size_t pad256(size_t n) { return (n + 255) / 256 * 256; }

// 4-D map of the pool: columns, rows of a page, heads, pages; the box is one page's rows, at most a tile's.
bool encode_pool(CUtensorMap* map, const void* base, const hstu_paged_cache_t& c, int32_t H, int32_t d) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(c.num_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.row_stride) * 2, static_cast<cuuint64_t>(c.head_stride) * 2,
                                 static_cast<cuuint64_t>(c.page_stride) * 2};
  const cuuint32_t box[4] = {d >= 64 ? 64u : 32u,
                             static_cast<cuuint32_t>(c.page_size < kTileRows ? c.page_size : kTileRows), 1u, 1u};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  const CUtensorMapSwizzle swz = d >= 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  return tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_q(CUtensorMap* map, const void* base, int64_t rows, int64_t width, int64_t ld, int32_t d) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {d >= 64 ? 64u : 32u, static_cast<cuuint32_t>(kTileRows)};
  const cuuint32_t estr[2] = {1u, 1u};
  const CUtensorMapSwizzle swz = d >= 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  return tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pieces the plan may cut items into.  It cuts none in batches of too many users or blocks (each user's last
// block may be a short one, so there are at least total_new / 128), nor where the longest item is too short; an
// item becomes at most one piece for each kMinPieceTiles of its tiles, and kMaxCuts.
int64_t most_cut_pieces(const RowsArgs& a, int64_t items, int ctas) {
  const int64_t blocks = (static_cast<int64_t>(a.total_new) + kItemRows - 1) / kItemRows;
  if (a.B > kCachedUsers || blocks > kCachedBlocks || blocks > kMaxRounds * ctas / a.H) return 0;
  const int longest = cost_bound(a.max_kv) / kMinPieceTiles;
  const int each = longest < kMaxCuts ? longest : kMaxCuts;
  if (each < 2) return 0;
  const int64_t most = static_cast<int64_t>(kMaxCutRounds) * ctas;
  return items < most / each ? items * each : most;
}

// Many rows a user: the plan, then the tcgen05 kernel, over one buffer from the library's pool.
template <int D>
hstu_status_t launch_many(const RowsArgs& a, const hstu_paged_cache_t& cache, float alpha, uint64_t wait_limit_ns,
                          DeviceState& st, cudaStream_t stream) {
  static std::once_flag once[kMaxDevices];
  static cudaError_t ready[kMaxDevices];
  cudaError_t e = once_per_device(once, ready, [] {
    return cudaFuncSetAttribute(hstu_fwd_kernel<D, false, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                FwdCfg<D>::kSmemBytes);
  });
  if (e != cudaSuccess || !tensor_map_encoder()) return HSTU_ERR_CUDA;
  const int ctas = st.num_sms;
  const int64_t capacity = static_cast<int64_t>(a.H) * (a.total_new / kItemRows + a.B);
  if (capacity > INT_MAX / 2) return HSTU_ERR_UNSUPPORTED;
  const int64_t width = static_cast<int64_t>(a.H) * D;
  CUtensorMap tq, tk, tv;
  if (!encode_q(&tq, a.q, a.total_new, width, a.q_ld, D) || !encode_pool(&tk, cache.k, cache, a.H, D) ||
      !encode_pool(&tv, cache.v, cache, a.H, D))
    return HSTU_ERR_CUDA;
  // header | block_start | done | pieces | partials
  const int64_t max_cut = most_cut_pieces(a, capacity, ctas);
  const size_t o_block = 256, o_done = o_block + pad256((static_cast<size_t>(a.B) + 1) * 4),
               o_pieces = o_done + pad256(4 * max_cut * 4),
               o_partials = o_pieces + pad256((capacity + max_cut) * sizeof(PagedPiece)),
               bytes = o_partials + static_cast<size_t>(max_cut) * kTileRows * D * 4;
  void* buf = nullptr;
  if (cudaMallocFromPoolAsync(&buf, bytes, st.pool, stream) != cudaSuccess) return HSTU_ERR_CUDA;
  uint8_t* at = static_cast<uint8_t*>(buf);
  PagedSchedArgs s;
  s.cache = a.cache;
  s.q_offsets = a.q_offsets;
  s.kv_len = a.kv_len;
  s.num_targets = a.num_targets;
  s.B = a.B;
  s.H = a.H;
  s.total_new = a.total_new;
  s.max_new = a.max_new;
  s.max_kv = a.max_kv;
  s.wave_rows = plan_wave_rows(a.H);
  s.num_ctas = ctas;
  s.max_cut = static_cast<int32_t>(max_cut);
  s.plan.header = reinterpret_cast<int32_t*>(at);
  s.plan.block_start = reinterpret_cast<int32_t*>(at + o_block);
  s.plan.done = reinterpret_cast<int32_t*>(at + o_done);
  s.plan.pieces = reinterpret_cast<PagedPiece*>(at + o_pieces);
  s.err = a.err;
  FwdParams p;
  std::memset(&p, 0, sizeof(p));
  p.work_counter = s.plan.header;
  p.out = a.out;
  p.out_ld = a.out_ld;
  p.H = a.H;
  p.half_alpha = 0.5f * alpha;
  p.inv_n = a.inv_n;
  p.err = a.err;
  p.wait_limit_ns = wait_limit_ns;
  p.paged.cache = a.cache;
  p.paged.plan = s.plan;
  p.paged.partials = reinterpret_cast<float4*>(at + o_partials);
  e = launch_dependent(paged_schedule_kernel, 1, kSchedThreads, 0, 0, stream, s);
  if (e == cudaSuccess)
    e = launch_dependent(hstu_fwd_kernel<D, false, true>, ctas, kPagedThreads, FwdCfg<D>::kSmemBytes, 0, stream, tq, tk, tv, p);
  if (cudaFreeAsync(buf, stream) != cudaSuccess && e == cudaSuccess) return HSTU_ERR_CUDA;
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

// hstu_paged_attn_fwd; with limit_ns, its self-check: the tcgen05 kernel with that limit on every wait.
hstu_status_t run_paged_attn(const void* q, int64_t q_ld, const hstu_paged_cache_t* cache, const int32_t* q_offsets,
                             const int32_t* kv_len, const int32_t* num_targets, int32_t B, int32_t H, int32_t d,
                             int32_t total_new, int32_t max_new, int32_t max_kv, float alpha, float N, void* out,
                             int64_t out_ld, void* stream, uint64_t limit_ns) {
  if (B < 0 || H < 1 || total_new < 0 || max_new < 0 || max_kv < 0) return HSTU_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(alpha) || !std::isfinite(N) || !(N > 0.0f)) return HSTU_ERR_INVALID_ARGUMENT;
  if (!head_size_ok(d) || static_cast<int64_t>(H) * d > INT_MAX / 4 || max_kv > INT_MAX - 4096 || B > kMaxUsers)
    return HSTU_ERR_UNSUPPORTED;
  hstu_status_t s = check_cache(cache, d);
  if (s != HSTU_OK || total_new == 0) return s;
  if (B == 0) return HSTU_ERR_INVALID_ARGUMENT;  // rows of no user
  if (!q || !q_offsets || !kv_len || !out) return HSTU_ERR_INVALID_ARGUMENT;
  const int64_t width = static_cast<int64_t>(H) * d;
  for (int64_t ld : {q_ld, out_ld})
    if ((s = check_ld(ld, width, total_new)) != HSTU_OK) return s;
  if (!aligned16(q) || !aligned16(out)) return HSTU_ERR_UNSUPPORTED;
  const size_t pool = cache_bytes(*cache, H, d), out_bytes = static_cast<size_t>((total_new - 1) * out_ld + width) * 2;
  if (overlaps(cache->k, pool, out, out_bytes) || overlaps(cache->v, pool, out, out_bytes) ||
      rows_overlap(out, out_ld, q, q_ld, total_new, width))
    return HSTU_ERR_INVALID_ARGUMENT;
  DeviceState* st = device_state();
  if (!st) return HSTU_ERR_CUDA;
  RowsArgs a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_ld = q_ld;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.out_ld = out_ld;
  a.cache = view_of(*cache);
  a.q_offsets = q_offsets;
  a.kv_len = kv_len;
  a.num_targets = num_targets;
  a.B = B;
  a.H = H;
  a.total_new = total_new;
  a.max_kv = max_kv;
  a.half_alpha = 0.5f * alpha;
  a.inv_n = 1.0f / N;
  a.err = st->err_word;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int32_t most = max_new < total_new ? max_new : total_new;
  a.blocks = most > kRowsBlock ? (most + kRowsBlock - 1) / kRowsBlock : 1;
  a.max_new = most;
  if (limit_ns || !rows_shape(a, 64 * 128 / d, st->num_sms).few) {
    const uint64_t limit = limit_ns ? limit_ns : kWaitLimitNs;
    return d == 128 ? launch_many<128>(a, *cache, alpha, limit, *st, cs)
                    : (d == 64 ? launch_many<64>(a, *cache, alpha, limit, *st, cs)
                               : launch_many<32>(a, *cache, alpha, limit, *st, cs));
  }
  if (most <= 8)
    return d == 128 ? launch_rows<128, 8>(a, *st, cs)
                    : (d == 64 ? launch_rows<64, 8>(a, *st, cs) : launch_rows<32, 8>(a, *st, cs));
  return d == 128 ? launch_rows<128, 16>(a, *st, cs)
                  : (d == 64 ? launch_rows<64, 16>(a, *st, cs) : launch_rows<32, 16>(a, *st, cs));
}

}  // namespace
}  // namespace hstu

extern "C" {

hstu_status_t hstu_rotary(const void* q, int64_t q_ld, const void* k, int64_t k_ld, const hstu_rotation_t* rotation,
                          int32_t inverse, int32_t H, int32_t d, int32_t rows, void* q_out, int64_t q_out_ld,
                          void* k_out, int64_t k_out_ld, void* stream) {
  using namespace hstu;
  if (H < 1 || rows < 0 || (inverse != 0 && inverse != 1)) return HSTU_ERR_INVALID_ARGUMENT;
  if (!head_size_ok(d) || static_cast<int64_t>(H) * d > INT_MAX / 4) return HSTU_ERR_UNSUPPORTED;
  hstu_status_t s = check_rotation(rotation, d, rows, true);
  if (s != HSTU_OK || rows == 0) return s;
  if (!q || !q_out || (k == nullptr) != (k_out == nullptr)) return HSTU_ERR_INVALID_ARGUMENT;
  const int64_t width = static_cast<int64_t>(H) * d;
  const int64_t lds[4] = {q_ld, q_out_ld, k ? k_ld : width, k ? k_out_ld : width};
  for (int64_t ld : lds)
    if ((s = check_ld(ld, width, rows)) != HSTU_OK) return s;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out)) return HSTU_ERR_UNSUPPORTED;
  if (clashes(q_out, q_out_ld, q, q_ld, true, rows, width)) return HSTU_ERR_INVALID_ARGUMENT;
  if (k && (clashes(k_out, k_out_ld, k, k_ld, true, rows, width) ||
            clashes(q_out, q_out_ld, k, k_ld, false, rows, width) ||
            clashes(k_out, k_out_ld, q, q_ld, false, rows, width) ||
            clashes(k_out, k_out_ld, q_out, q_out_ld, false, rows, width)))
    return HSTU_ERR_INVALID_ARGUMENT;
  DeviceState* st = device_state();
  if (!st) return HSTU_ERR_CUDA;
  RotArgs a;
  std::memset(&a, 0, sizeof(a));
  a.rows = rows;
  a.H = H;
  add_tensor(a, q, q_ld, q_out, q_out_ld, kToRows, true);
  if (k) add_tensor(a, k, k_ld, k_out, k_out_ld, kToRows, true);
  set_rotation(a, rotation, inverse != 0);
  return launch_rotary(a, d, false, *st, static_cast<cudaStream_t>(stream));
}

hstu_status_t hstu_paged_append(const void* q, int64_t q_ld, const void* k, int64_t k_ld, const void* v, int64_t v_ld,
                                const hstu_rotation_t* rotation, const hstu_paged_cache_t* cache,
                                const int32_t* q_offsets, const int32_t* kv_len, int32_t B, int32_t H, int32_t d,
                                int32_t total_new, void* q_out, int64_t q_out_ld, void* stream) {
  using namespace hstu;
  if (B < 0 || H < 1 || total_new < 0) return HSTU_ERR_INVALID_ARGUMENT;
  if (!head_size_ok(d) || static_cast<int64_t>(H) * d > INT_MAX / 4 || B > kMaxUsers) return HSTU_ERR_UNSUPPORTED;
  hstu_status_t s = check_cache(cache, d);
  if (s == HSTU_OK && rotation) s = check_rotation(rotation, d, total_new, false);
  if (s != HSTU_OK || total_new == 0) return s;
  if (B == 0) return HSTU_ERR_INVALID_ARGUMENT;  // rows of no user
  if (!k || !v || !q_offsets || !kv_len) return HSTU_ERR_INVALID_ARGUMENT;
  if ((q == nullptr) != (q_out == nullptr) || (q && !rotation)) return HSTU_ERR_INVALID_ARGUMENT;
  const int64_t width = static_cast<int64_t>(H) * d;
  const int64_t lds[4] = {k_ld, v_ld, q ? q_ld : width, q ? q_out_ld : width};
  for (int64_t ld : lds)
    if ((s = check_ld(ld, width, total_new)) != HSTU_OK) return s;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out)) return HSTU_ERR_UNSUPPORTED;
  // The cache overlaps no token tensor, and no element of it is written for two places.
  const size_t pool = cache_bytes(*cache, H, d);
  const void* tokens[4] = {k, v, q, q_out};
  for (int i = 0; i < (q ? 4 : 2); ++i) {
    const size_t n = static_cast<size_t>((total_new - 1) * lds[i] + width) * 2;
    if (overlaps(cache->k, pool, tokens[i], n) || overlaps(cache->v, pool, tokens[i], n))
      return HSTU_ERR_INVALID_ARGUMENT;
  }
  const CacheAxes axes = cache_axes(*cache, H);
  if (rows_share(axes, d) ||
      caches_meet(axes, d, (reinterpret_cast<intptr_t>(cache->v) - reinterpret_cast<intptr_t>(cache->k)) / 2))
    return HSTU_ERR_INVALID_ARGUMENT;
  if (q && (clashes(q_out, q_out_ld, q, q_ld, true, total_new, width) ||
            clashes(q_out, q_out_ld, k, k_ld, false, total_new, width) ||
            clashes(q_out, q_out_ld, v, v_ld, false, total_new, width)))
    return HSTU_ERR_INVALID_ARGUMENT;
  DeviceState* st = device_state();
  if (!st) return HSTU_ERR_CUDA;
  RotArgs a;
  std::memset(&a, 0, sizeof(a));
  a.rows = total_new;
  a.H = H;
  if (q) add_tensor(a, q, q_ld, q_out, q_out_ld, kToRows, true);
  add_tensor(a, k, k_ld, nullptr, 0, kToCacheK, rotation != nullptr);
  add_tensor(a, v, v_ld, nullptr, 0, kToCacheV, false);
  set_rotation(a, rotation, false);
  a.cache = view_of(*cache);
  a.q_offsets = q_offsets;
  a.kv_len = kv_len;
  a.B = B;
  a.err = st->err_word;
  return launch_rotary(a, d, true, *st, static_cast<cudaStream_t>(stream));
}

hstu_status_t hstu_paged_attn_fwd(const void* q, int64_t q_ld, const hstu_paged_cache_t* cache, const int32_t* q_offsets,
                                  const int32_t* kv_len, const int32_t* num_targets, int32_t B, int32_t H, int32_t d,
                                  int32_t total_new, int32_t max_new, int32_t max_kv, float alpha, float N, void* out,
                                  int64_t out_ld, void* stream) {
  return hstu::run_paged_attn(q, q_ld, cache, q_offsets, kv_len, num_targets, B, H, d, total_new, max_new, max_kv, alpha,
                              N, out, out_ld, stream, 0);
}

hstu_status_t hstu_paged_selfcheck_fwd_timeout(const void* q, int64_t q_ld, const hstu_paged_cache_t* cache,
                                               const int32_t* q_offsets, const int32_t* kv_len,
                                               const int32_t* num_targets, int32_t B, int32_t H, int32_t d,
                                               int32_t total_new, int32_t max_new, int32_t max_kv, float alpha, float N,
                                               void* out, int64_t out_ld, uint64_t limit_ns, void* stream) {
  if (limit_ns == 0 || limit_ns > 1000000000ull) return HSTU_ERR_INVALID_ARGUMENT;
  return hstu::run_paged_attn(q, q_ld, cache, q_offsets, kv_len, num_targets, B, H, d, total_new, max_new, max_kv, alpha,
                              N, out, out_ld, stream, limit_ns);
}

}  // extern "C"
