// C ABI of the attention library: argument checks, TMA tensor-map encoding and
// kernel launches on the caller's stream. No device memory is allocated here.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <unordered_map>
#include <vector>

#include <cudaTypedefs.h>

#include "common.cuh"
#include "fa_gb300.h"

namespace {

thread_local char g_last_cuda_error[256] = "no error";

int launch_error(cudaError_t e) {
  std::snprintf(g_last_cuda_error, sizeof(g_last_cuda_error), "%s: %s", cudaGetErrorName(e),
                cudaGetErrorString(e));
  return FA_ERR_LAUNCH;
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Tensor maps are cached per (address, type, extents, strides, box, swizzle):
// a call with the same buffers reuses the encoded map. The cache is shared by
// all threads (behind a mutex) and emptied when it reaches kMapCacheSize.
struct MapKey {
  uintptr_t ptr;
  int dtype, swizzle;
  uint64_t dims[3], strides[2];
  uint32_t box[3];
  bool operator==(const MapKey& o) const {
    return ptr == o.ptr && dtype == o.dtype && swizzle == o.swizzle &&
           std::memcmp(dims, o.dims, sizeof(dims)) == 0 && std::memcmp(strides, o.strides, sizeof(strides)) == 0 &&
           std::memcmp(box, o.box, sizeof(box)) == 0;
  }
};
struct MapKeyHash {
  size_t operator()(const MapKey& k) const {
    uint64_t h = k.ptr * 0x9E3779B97F4A7C15ull;
    auto mix = [&h](uint64_t v) { h = (h ^ v) * 0x100000001B3ull; };
    mix(static_cast<uint64_t>(k.dtype));
    mix(static_cast<uint64_t>(k.swizzle));
    for (uint64_t d : k.dims) mix(d);
    for (uint64_t st : k.strides) mix(st);
    for (uint32_t b : k.box) mix(b);
    return static_cast<size_t>(h);
  }
};
constexpr size_t kMapCacheSize = 512;

bool encode_3d(CUtensorMap* m, CUtensorMapDataType dtype, const void* ptr, const uint64_t dims[3],
               const uint64_t strides[2], const uint32_t box[3], CUtensorMapSwizzle swizzle) {
  static std::mutex mu;
  static std::unordered_map<MapKey, CUtensorMap, MapKeyHash> cache;
  MapKey key{reinterpret_cast<uintptr_t>(ptr), static_cast<int>(dtype), static_cast<int>(swizzle), {}, {}, {}};
  for (int i = 0; i < 3; ++i) {
    key.dims[i] = dims[i];
    key.box[i] = box[i];
  }
  key.strides[0] = strides[0];
  key.strides[1] = strides[1];
  {
    std::lock_guard<std::mutex> lk(mu);
    auto it = cache.find(key);
    if (it != cache.end()) {
      *m = it->second;
      return true;
    }
  }
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  // The encoder is a driver call: a host thread that has made no CUDA runtime
  // call yet has no current context, and the encode then fails. Binding the
  // current device's primary context first (cudaSetDevice does since CUDA 12)
  // makes the library callable from any host thread.
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) return false;
  cuuint64_t d[3] = {dims[0], dims[1], dims[2]};
  cuuint64_t st[2] = {strides[0], strides[1]};
  cuuint32_t bx[3] = {box[0], box[1], box[2]};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, dtype, 3, const_cast<void*>(ptr), d, st, bx, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return false;
  std::lock_guard<std::mutex> lk(mu);
  if (cache.size() >= kMapCacheSize) cache.clear();
  cache.emplace(key, *m);
  return true;
}

// 3-D map over a [BH, N, D] bf16 tensor: box = 64 columns (128 B, the swizzle
// width) x box_rows rows x 1 slice (rows past N read as zero).
bool encode_bhnd(CUtensorMap* m, const void* ptr, int BH, int N, int D, int box_rows) {
  const uint64_t dims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(N), static_cast<uint64_t>(BH)};
  const uint64_t strides[2] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(N) * D * 2};
  const uint32_t box[3] = {64, static_cast<uint32_t>(box_rows), 1};
  return encode_3d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, ptr, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// 3-D map over a packed [total, H, D] bf16 tensor: box = 64 columns x 1 head x
// box_rows tokens (rows past `total` read as zero).
bool encode_thd(CUtensorMap* m, const void* ptr, int H, int total, int D, int box_rows) {
  const uint64_t dims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(H), static_cast<uint64_t>(total)};
  const uint64_t strides[2] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(H) * D * 2};
  const uint32_t box[3] = {64, 1, static_cast<uint32_t>(box_rows)};
  return encode_3d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, ptr, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// The same for a grouped Q tile: box = 64 columns x P heads x tok tokens (in
// shared memory row token * P + head).
bool encode_thd_group(CUtensorMap* m, const void* ptr, int H, int total, int D, fa::QTile t) {
  const uint64_t dims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(H), static_cast<uint64_t>(total)};
  const uint64_t strides[2] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(H) * D * 2};
  const uint32_t box[3] = {64, static_cast<uint32_t>(t.P), static_cast<uint32_t>(t.tok)};
  return encode_3d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, ptr, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Heads packed into one Q tile for groups of G heads: the largest divisor P of
// G that leaves at most 4 of the tile's 128 rows unused (128 / P whole tokens;
// a P of 24 or 48 would waste 8 or 32 rows in every tile of a long prompt).
fa::QTile q_tile(int G) {
  int P = std::min(G, 128);
  while (G % P != 0 || 128 / P * P < 124) --P;  // P = 1 always fits
  return fa::QTile{P, 128 / P};
}

// 3-D map over an 8-bit tensor [dim2][dim1][dim0] (dim0 contiguous, row
// pitch stride1 bytes, slice pitch stride2 bytes); box = 128 x 128 x 1 with a
// 128-byte swizzle (one 128-byte row per box row).
bool encode_u8(CUtensorMap* m, const void* ptr, long long dim0, long long dim1, long long dim2, long long stride1,
               long long stride2) {
  const uint64_t dims[3] = {static_cast<uint64_t>(dim0), static_cast<uint64_t>(dim1), static_cast<uint64_t>(dim2)};
  const uint64_t strides[2] = {static_cast<uint64_t>(stride1), static_cast<uint64_t>(stride2)};
  const uint32_t box[3] = {128, 128, 1};
  return encode_3d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, ptr, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Check mode: copy cu_seqlens to the host and validate them (`spare`: rows of
// no sequence may follow the last one).
int check_cu_seqlens(const int* cu, int batch, int total, int max_len, cudaStream_t stream, bool spare = false);

bool check_mode() {
  static int mode = -1;
  if (mode < 0) {
    const char* e = std::getenv("FA_CHECK");
    mode = (e != nullptr && e[0] != '\0' && e[0] != '0') ? 1 : 0;
  }
  return mode == 1;
}

int check_shape(int B, int H, int N, int d, float scale) {
  if (B < 1 || H < 1 || N < 1) return FA_ERR_INVALID;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  const long long elems = static_cast<long long>(B) * H * N * d;
  if (elems > (1LL << 40) || static_cast<long long>(B) * H > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Check mode: copy kv_lens to the host and validate them.
int check_kv_lens(const int* kv_lens, int B, int N, cudaStream_t stream) {
  if (kv_lens == nullptr || !check_mode()) return FA_OK;
  std::vector<int> h(B);
  cudaError_t e = cudaMemcpyAsync(h.data(), kv_lens, sizeof(int) * B, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return launch_error(e);
  for (int b = 0; b < B; ++b)
    if (h[b] < 0 || h[b] > N) return FA_ERR_INVALID;
  return FA_OK;
}

int check_cu_seqlens(const int* cu, int batch, int total, int max_len, cudaStream_t stream, bool spare) {
  if (!check_mode()) return FA_OK;
  std::vector<int> h(batch + 1);
  cudaError_t e = cudaMemcpyAsync(h.data(), cu, sizeof(int) * (batch + 1), cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return launch_error(e);
  if (h[0] != 0 || (spare ? h[batch] > total : h[batch] != total)) return FA_ERR_INVALID;
  for (int b = 0; b < batch; ++b)
    if (h[b + 1] < h[b] || h[b + 1] - h[b] > max_len) return FA_ERR_INVALID;
  return FA_OK;
}

fa::AttnShape make_shape(int B, int H, int N, int d, float scale, int causal) {
  fa::AttnShape s;
  s.B = B;
  s.H = H;
  s.N = N;
  s.D = d;
  s.Nk = N;
  s.Hk = H;
  s.causal = causal ? 1 : 0;
  s.scale = scale;
  s.scale_log2 = scale * fa::kLog2e;
  return s;
}

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// How a decoding step splits each sequence's keys over CTAs: about 1024 CTAs
// in all (several waves on the GPU), chunks of whole 64-key tiles. Computed
// from the shapes alone, so the workspace size does not depend on the device.
struct DecodePlan {
  int nsplit, chunk;
};
DecodePlan decode_plan(int B, int H, int max_seq_len) {
  const long long bh = static_cast<long long>(B) * H;
  const long long tiles = (static_cast<long long>(max_seq_len) + 63) / 64;
  long long ns = (1024 + bh - 1) / bh;
  if (ns > tiles) ns = tiles;
  if (ns < 1) ns = 1;
  long long chunk = ((max_seq_len + ns - 1) / ns + 63) / 64 * 64;
  if (chunk < 64) chunk = 64;
  const long long n = (max_seq_len + chunk - 1) / chunk;
  return DecodePlan{static_cast<int>(n < 1 ? 1 : n), static_cast<int>(chunk)};
}

// Check mode: copy seq_lens and the block table to the host and validate them.
int check_decode_tables(const int* seq_lens, const int* table, int B, int max_blocks, int block_size,
                        int num_blocks, int max_seq_len, cudaStream_t stream) {
  if (!check_mode()) return FA_OK;
  std::vector<int> lens(B), tab(static_cast<size_t>(B) * max_blocks);
  cudaError_t e = cudaMemcpyAsync(lens.data(), seq_lens, sizeof(int) * B, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(tab.data(), table, sizeof(int) * tab.size(), cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return launch_error(e);
  for (int b = 0; b < B; ++b) {
    if (lens[b] < 0 || lens[b] > max_seq_len) return FA_ERR_INVALID;
    for (int p = 0; p < (lens[b] + block_size - 1) / block_size; ++p) {
      const int x = tab[static_cast<size_t>(b) * max_blocks + p];
      if (x < 0 || x >= num_blocks) return FA_ERR_INVALID;
    }
  }
  return FA_OK;
}

// How the shared-prefix step splits its keys over CTAs, from the shapes alone
// (the workspace size depends on it). `base` items (rows x key heads) of
// `tiles` 64-key tiles: as many splits as bring the item count to `target`,
// each of whole tiles.
void split_keys(long long base, long long len, long long target, int* chunk, int* splits) {
  const long long tiles = std::max<long long>((len + 63) / 64, 1);
  long long ns = std::min(std::max<long long>(target / std::max<long long>(base, 1), 1), tiles);
  const long long per = (tiles + ns - 1) / ns;
  *chunk = static_cast<int>(per * 64);
  *splits = static_cast<int>((tiles + per - 1) / per);
}
void shared_plan(fa::SharedArgs* a) {
  const int G = a->H / a->Hk;
  const long long group_rows = static_cast<long long>(a->max_group) * G;
  a->seq_blocks = (G + 63) / 64;
  // Items of about 4 us to start and end and 0.7 us per tile, on each of 152 SMs
  // two at a time (d 128) or four (d 64): prefixes cut into about 152 or 304
  // items, sequences into about 608 (their lengths differ). Measured at d 64 on
  // 40 sequences of up to 700 tokens behind six prefixes of up to 4000: 17.6 us
  // with 304 prefix items, 22.5 with 152, 21.3 with 608 (two per SM with six
  // stages: 19.6 with 152, 21.4 with 304); 64 sequences of 4096 own tokens, 32/8
  // heads: 88 us, 94.6 two per SM; own parts in 1216 items 1 to 5 us slower.
  split_keys(static_cast<long long>(a->B) * a->Hk * a->seq_blocks, a->max_seq_len, 608, &a->seq_chunk,
             &a->seq_splits);
  // More than one 16-row block of the streaming kernel: 128-row tiles. Measured
  // on prefixes of 2000 / 8000 / 32000 tokens, 8 key heads, d = 128: 24 rows
  // 15.4 / 18.6 / 37.3 us in tiles, 14.0 / 21.6 / 50.9 streamed; 16 rows 15.3 /
  // 17.7 / 35.7 in tiles, 12.3 / 15.8 / 33.0 streamed; 64 rows 18.1 / 22.5 /
  // 40.9 in tiles, 20.8 / 34.5 / 87.7 streamed.
  a->prefix_tiles = group_rows > 16;
  if (!a->prefix_tiles) {
    split_keys(static_cast<long long>(a->P) * a->Hk, a->max_prefix_len, a->D == 64 ? 304 : 152,
               &a->prefix_chunk, &a->prefix_splits);
    return;
  }
  // 128-row tiles, two per CTA and one CTA per SM: the number of splits whose
  // waves take the least time, a CTA costing its 128-key blocks and about
  // three more to start and to write its part.
  const fa::QTile qt = q_tile(G);
  const int pairs = (a->max_group + 2 * qt.tok - 1) / (2 * qt.tok);
  const long long base = static_cast<long long>(a->P) * (a->H / qt.P) * pairs;
  const long long blocks = (static_cast<long long>(a->max_prefix_len) + 127) / 128;
  long long best = -1;
  for (long long ns = 1; ns <= std::min<long long>(blocks, 152); ++ns) {
    const long long per = (blocks + ns - 1) / ns, n = (blocks + per - 1) / per;
    const long long cost = (base * n + 151) / 152 * (per + 3);
    if (best >= 0 && cost >= best) continue;
    best = cost;
    a->prefix_chunk = static_cast<int>(per * 128);
    a->prefix_splits = static_cast<int>(n);
  }
}

// Check mode: the tables and lengths of a shared-prefix step on the host.
int check_shared_tables(const fa::SharedArgs& a, cudaStream_t stream) {
  if (!check_mode()) return FA_OK;
  std::vector<int> cu(a.P + 1);
  cudaError_t e = cudaMemcpyAsync(cu.data(), a.cu_seqs, sizeof(int) * cu.size(), cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return launch_error(e);
  if (cu[0] < 0 || cu[a.P] > a.B) return FA_ERR_INVALID;
  for (int p = 0; p < a.P; ++p)
    if (cu[p + 1] < cu[p] || cu[p + 1] - cu[p] > a.max_group) return FA_ERR_INVALID;
  const int st = check_decode_tables(a.prefix_lens, a.prefix_table, a.P, a.max_prefix_blocks, a.block_size,
                                     a.num_blocks, a.max_prefix_len, stream);
  if (st != FA_OK) return st;
  return check_decode_tables(a.seq_lens, a.block_table, a.B, a.max_blocks, a.block_size, a.num_blocks, a.max_seq_len,
                             stream);
}

// Test hooks, read from the environment on every call: FA_TEST_WAIT_LIMIT_NS
// bounds each device wait (default 2 s), FA_TEST_DROP_LOADS=1 makes the TMA
// producers issue no loads so that the dependent waits run out. Used by the
// tests of the timeout path; the device values change only when these
// variables change.
int apply_test_hooks(cudaStream_t stream) {
  static std::mutex mu;
  static unsigned long long applied_limit = 2000000000ull;
  static int applied_drop = 0;
  const char* el = std::getenv("FA_TEST_WAIT_LIMIT_NS");
  const char* ed = std::getenv("FA_TEST_DROP_LOADS");
  unsigned long long limit = 2000000000ull;
  if (el != nullptr && el[0] != '\0') {
    const unsigned long long v = std::strtoull(el, nullptr, 10);
    if (v > 0) limit = v;
  }
  const int drop = (ed != nullptr && ed[0] == '1') ? 1 : 0;
  std::lock_guard<std::mutex> lk(mu);
  if (limit == applied_limit && drop == applied_drop) return FA_OK;
  cudaError_t e = fa::set_fwd_test_hooks(limit, drop, stream);
  if (e == cudaSuccess) e = fa::set_bwd_test_hooks(limit, drop, stream);
  if (e == cudaSuccess) e = fa::set_decode_test_hooks(limit, drop, stream);
  if (e == cudaSuccess) e = fa::set_fp8_test_hooks(limit, drop, stream);
  if (e == cudaSuccess) e = fa::set_fwd_gqa_test_hooks(limit, drop, stream);
  if (e == cudaSuccess) e = fa::set_bwd_gqa_test_hooks(limit, drop, stream);
  if (e == cudaSuccess) e = fa::set_decode_shared_test_hooks(limit, drop, stream);
  if (e == cudaSuccess) e = fa::set_decode_prefix_test_hooks(limit, drop, stream);
  if (e != cudaSuccess) return launch_error(e);
  applied_limit = limit;
  applied_drop = drop;
  return FA_OK;
}

// Kernel timing: pairs of CUDA events per kernel kind, filled call by call.
// 0 forward, 1 backward pre-pass, 2 backward main, 3 dQ conversion, 4 paged
// decode, 5 decode split merge, 6 FP8 forward.
constexpr int kKinds = 7;
struct Timing {
  bool on = false;
  int cap = 0;
  std::vector<cudaEvent_t> start[kKinds], stop[kKinds];
  int used[kKinds] = {0, 0, 0, 0, 0, 0, 0};
};
Timing g_timing;
std::mutex g_timing_mu;

// Event slots for the next call's kernels (first = kind of its first kernel).
bool next_marks(fa::LaunchMarks* m, int first, int count) {
  std::lock_guard<std::mutex> lk(g_timing_mu);
  if (!g_timing.on) return false;
  for (int i = 0; i < count; ++i)
    if (g_timing.used[first + i] >= g_timing.cap) return false;
  for (int i = 0; i < count; ++i) {
    const int k = first + i, u = g_timing.used[k]++;
    m->start[i] = g_timing.start[k][u];
    m->stop[i] = g_timing.stop[k][u];
  }
  return true;
}

}  // namespace

extern "C" {

const char* fa_status_string(int status) {
  switch (status) {
    case FA_OK: return "FA_OK";
    case FA_ERR_INVALID: return "FA_ERR_INVALID: invalid argument";
    case FA_ERR_UNSUPPORTED: return "FA_ERR_UNSUPPORTED: unsupported head dim, alignment or size";
    case FA_ERR_LAUNCH: return "FA_ERR_LAUNCH: CUDA error";
    case FA_ERR_TIMEOUT: return "FA_ERR_TIMEOUT: a device wait ran out";
    case FA_ERR_WORKSPACE: return "FA_ERR_WORKSPACE: workspace missing or too small";
    case FA_ERR_SCRATCH_LIMIT:
      return "FA_ERR_SCRATCH_LIMIT: problem needs more than the fixed scratch of fa_bwd_noalloc";
    default: return "unknown fa_status";
  }
}

const char* fa_last_cuda_error(void) { return g_last_cuda_error; }

int fa_check_status(void* stream) {
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return launch_error(e);
  const int words[] = {fa::take_fwd_status(), fa::take_bwd_status(),     fa::take_decode_status(),
                       fa::take_fp8_status(), fa::take_fwd_gqa_status(), fa::take_bwd_gqa_status(),
                       fa::take_decode_shared_status(), fa::take_decode_prefix_status()};
  bool late = false;
  for (int w : words) {
    if (w == FA_ERR_LAUNCH) return launch_error(cudaGetLastError());
    late = late || w != 0;
  }
  if (late) return FA_ERR_TIMEOUT;
  return FA_OK;
}

int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N, int d,
           float scale, int causal, const int* kv_lens, void* stream) {
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID;
  int st = check_shape(B, H, N, d, scale);
  if (st != FA_OK) return st;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return FA_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = check_kv_lens(kv_lens, B, N, s);
  if (st != FA_OK) return st;
  st = apply_test_hooks(s);
  if (st != FA_OK) return st;
  const int BH = B * H;
  CUtensorMap tq, tk, tv;
  if (!encode_bhnd(&tq, q, BH, N, d, 128) || !encode_bhnd(&tk, k, BH, N, d, 128) ||
      !encode_bhnd(&tv, v, BH, N, d, 128))
    return launch_error(cudaErrorInvalidValue);
  fa::FwdArgs a;
  a.s = make_shape(B, H, N, d, scale, causal);
  a.pk = fa::Packing{0, nullptr, nullptr, 0, 0};
  a.kv_lens = kv_lens;
  a.o = o;
  a.lse = lse;
  fa::LaunchMarks marks;
  const bool timed = next_marks(&marks, 0, 1);
  cudaError_t e = fa::launch_fwd(tq, tk, tv, a, s, timed ? &marks : nullptr);
  if (e != cudaSuccess) return launch_error(e);
  if (check_mode()) return fa_check_status(stream);
  return FA_OK;
}

int fa_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse, const int* cu_seqlens_q,
                  const int* cu_seqlens_k, int batch, int H, int d, int total_q, int total_k, int max_seqlen_q,
                  int max_seqlen_k, float scale, int causal, void* stream) {
  if (!q || !k || !v || !o || !lse || !cu_seqlens_q || !cu_seqlens_k) return FA_ERR_INVALID;
  if (total_q < 1 || total_k < 1 || max_seqlen_q < 1 || max_seqlen_k < 1) return FA_ERR_INVALID;
  if (max_seqlen_q > total_q || max_seqlen_k > total_k) return FA_ERR_INVALID;
  int st = check_shape(batch, H, max_seqlen_q, d, scale);
  if (st != FA_OK) return st;
  if (static_cast<long long>(total_q) * H * d > (1LL << 40) || static_cast<long long>(total_k) * H * d > (1LL << 40))
    return FA_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return FA_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = check_cu_seqlens(cu_seqlens_q, batch, total_q, max_seqlen_q, s);
  if (st == FA_OK) st = check_cu_seqlens(cu_seqlens_k, batch, total_k, max_seqlen_k, s);
  if (st != FA_OK) return st;
  st = apply_test_hooks(s);
  if (st != FA_OK) return st;
  CUtensorMap tq, tk, tv;
  if (!encode_thd(&tq, q, H, total_q, d, 128) || !encode_thd(&tk, k, H, total_k, d, 128) ||
      !encode_thd(&tv, v, H, total_k, d, 128))
    return launch_error(cudaErrorInvalidValue);
  fa::FwdArgs a;
  a.s = make_shape(batch, H, max_seqlen_q, d, scale, causal);
  a.pk = fa::Packing{1, cu_seqlens_q, cu_seqlens_k, total_q, total_k};
  a.kv_lens = nullptr;
  a.o = o;
  a.lse = lse;
  fa::LaunchMarks marks;
  const bool timed = next_marks(&marks, 0, 1);
  cudaError_t e = fa::launch_fwd(tq, tk, tv, a, s, timed ? &marks : nullptr);
  if (e != cudaSuccess) return launch_error(e);
  if (check_mode()) return fa_check_status(stream);
  return FA_OK;
}

// Argument checks that the grouped-head packed entry points share.
static int check_gqa(int batch, int H, int H_kv, int d, int total_q, int total_k, int max_seqlen_q, int max_seqlen_k,
                     float scale) {
  if (total_q < 1 || total_k < 1 || max_seqlen_q < 1 || max_seqlen_k < 1) return FA_ERR_INVALID;
  if (max_seqlen_q > total_q || max_seqlen_k > total_k) return FA_ERR_INVALID;
  if (H_kv < 1 || H < 1 || H % H_kv != 0) return FA_ERR_INVALID;
  const int st = check_shape(batch, H, max_seqlen_q, d, scale);
  if (st != FA_OK) return st;
  if (static_cast<long long>(total_q) * H * d > (1LL << 40) || static_cast<long long>(total_k) * H_kv * d > (1LL << 40))
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

int fa_fwd_varlen_gqa(const void* q, const void* k, const void* v, void* o, float* lse, const int* cu_seqlens_q,
                      const int* cu_seqlens_k, int batch, int H, int H_kv, int d, int total_q, int total_k,
                      int max_seqlen_q, int max_seqlen_k, float scale, int causal, void* stream) {
  if (!q || !k || !v || !o || !lse || !cu_seqlens_q || !cu_seqlens_k) return FA_ERR_INVALID;
  int st = check_gqa(batch, H, H_kv, d, total_q, total_k, max_seqlen_q, max_seqlen_k, scale);
  if (st != FA_OK) return st;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return FA_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = check_cu_seqlens(cu_seqlens_q, batch, total_q, max_seqlen_q, s, true);
  if (st == FA_OK) st = check_cu_seqlens(cu_seqlens_k, batch, total_k, max_seqlen_k, s, true);
  if (st != FA_OK) return st;
  st = apply_test_hooks(s);
  if (st != FA_OK) return st;
  fa::FwdGroupedArgs a;
  a.qt = q_tile(H / H_kv);
  CUtensorMap tq, tk, tv;
  if (!encode_thd_group(&tq, q, H, total_q, d, a.qt) || !encode_thd(&tk, k, H_kv, total_k, d, 128) ||
      !encode_thd(&tv, v, H_kv, total_k, d, 128))
    return launch_error(cudaErrorInvalidValue);
  a.s = make_shape(batch, H, max_seqlen_q, d, scale, causal);
  a.s.Nk = max_seqlen_k;
  a.s.Hk = H_kv;
  a.pk = fa::Packing{1, cu_seqlens_q, cu_seqlens_k, total_q, total_k};
  a.kv_lens = nullptr;
  a.o = o;
  a.lse = lse;
  fa::LaunchMarks marks;
  const bool timed = next_marks(&marks, 0, 1);
  cudaError_t e = fa::launch_fwd_gqa(tq, tk, tv, a, s, timed ? &marks : nullptr);
  if (e != cudaSuccess) return launch_error(e);
  if (check_mode()) return fa_check_status(stream);
  return FA_OK;
}

size_t fa_bwd_workspace_size(int B, int H, int N, int d) {
  if (check_shape(B, H, N, d, 1.f) != FA_OK) return 0;
  // Rows are padded per head to whole 128-row blocks.
  const size_t rows = static_cast<size_t>(B) * H * ((static_cast<size_t>(N) + 127) / 128 * 128);
  return align_up(rows * 4, 256) * 2 + align_up(rows * d * 4, 256) + align_up(rows / 128 * 4, 256) + 256;
}

// Carves the workspace: delta, -LSE*log2(e), the dQ accumulator, then the
// per-block counters and the ticket of the deterministic order.
static void carve_workspace(fa::BwdArgs* a, void* workspace, size_t rows, int d) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t vec = align_up(rows * 4, 256), acc = align_up(rows * d * 4, 256);
  a->delta = reinterpret_cast<float*>(ws);
  a->lse2 = reinterpret_cast<float*>(ws + vec);
  a->dq_acc = reinterpret_cast<float*>(ws + 2 * vec);
  a->dq_turn = reinterpret_cast<uint32_t*>(ws + 2 * vec + acc);
  a->ticket = reinterpret_cast<uint32_t*>(ws + 2 * vec + acc + align_up(rows / 128 * 4, 256));
}

static int bwd_fixed(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                     void* dq, void* dk, void* dv, int B, int H, int N, int d, float scale, int causal,
                     const int* kv_lens, void* workspace, size_t workspace_bytes, void* stream, int det) {
  if (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv) return FA_ERR_INVALID;
  int st = check_shape(B, H, N, d, scale);
  if (st != FA_OK) return st;
  const void* ptrs[] = {q, k, v, o, lse, dO, dq, dk, dv};
  for (const void* p : ptrs)
    if (!aligned16(p)) return FA_ERR_UNSUPPORTED;
  const size_t need = fa_bwd_workspace_size(B, H, N, d);
  if (workspace == nullptr || workspace_bytes < need || !aligned16(workspace)) return FA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = check_kv_lens(kv_lens, B, N, s);
  if (st != FA_OK) return st;
  st = apply_test_hooks(s);
  if (st != FA_OK) return st;
  const int BH = B * H;
  CUtensorMap tq, tk, tv, tdo;
  if (!encode_bhnd(&tq, q, BH, N, d, 128) || !encode_bhnd(&tk, k, BH, N, d, 128) ||
      !encode_bhnd(&tv, v, BH, N, d, 128) || !encode_bhnd(&tdo, dO, BH, N, d, 128))
    return launch_error(cudaErrorInvalidValue);
  const size_t rows = static_cast<size_t>(BH) * ((static_cast<size_t>(N) + 127) / 128 * 128);
  fa::BwdArgs a;
  a.s = make_shape(B, H, N, d, scale, causal);
  a.pk = fa::Packing{0, nullptr, nullptr, 0, 0};
  a.kv_lens = kv_lens;
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.dO = dO;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  carve_workspace(&a, workspace, rows, d);
  a.deterministic = det;
  fa::LaunchMarks marks;
  const bool timed = next_marks(&marks, 1, 3);
  cudaError_t e = fa::launch_bwd(tq, tk, tv, tdo, a, s, timed ? &marks : nullptr);
  if (e != cudaSuccess) return launch_error(e);
  if (check_mode()) return fa_check_status(stream);
  return FA_OK;
}

int fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
           void* dq, void* dk, void* dv, int B, int H, int N, int d, float scale, int causal,
           const int* kv_lens, void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_fixed(q, k, v, o, lse, dO, dq, dk, dv, B, H, N, d, scale, causal, kv_lens, workspace,
                   workspace_bytes, stream, 0);
}

int fa_bwd_deterministic(const void* q, const void* k, const void* v, const void* o, const float* lse,
                         const void* dO, void* dq, void* dk, void* dv, int B, int H, int N, int d, float scale,
                         int causal, const int* kv_lens, void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_fixed(q, k, v, o, lse, dO, dq, dk, dv, B, H, N, d, scale, causal, kv_lens, workspace,
                   workspace_bytes, stream, 1);
}

int fa_timing_end(void) {
  std::lock_guard<std::mutex> lk(g_timing_mu);
  for (int k = 0; k < kKinds; ++k) {
    for (cudaEvent_t ev : g_timing.start[k]) cudaEventDestroy(ev);
    for (cudaEvent_t ev : g_timing.stop[k]) cudaEventDestroy(ev);
    g_timing.start[k].clear();
    g_timing.stop[k].clear();
    g_timing.used[k] = 0;
  }
  g_timing.on = false;
  g_timing.cap = 0;
  return FA_OK;
}

int fa_timing_begin(int max_calls) {
  if (max_calls < 1 || max_calls > (1 << 20)) return FA_ERR_INVALID;
  fa_timing_end();
  std::lock_guard<std::mutex> lk(g_timing_mu);
  for (int k = 0; k < kKinds; ++k) {
    g_timing.start[k].assign(max_calls, nullptr);
    g_timing.stop[k].assign(max_calls, nullptr);
    for (int i = 0; i < max_calls; ++i) {
      cudaError_t e = cudaEventCreate(&g_timing.start[k][i]);
      if (e == cudaSuccess) e = cudaEventCreate(&g_timing.stop[k][i]);
      if (e != cudaSuccess) return launch_error(e);
    }
  }
  g_timing.cap = max_calls;
  g_timing.on = true;
  return FA_OK;
}

int fa_timing_read(int kind, double* total_ms, int* count) {
  if (kind < 0 || kind >= kKinds || total_ms == nullptr || count == nullptr) return FA_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_timing_mu);
  double tot = 0.0;
  const int n = g_timing.used[kind];
  for (int i = 0; i < n; ++i) {
    cudaError_t e = cudaEventSynchronize(g_timing.stop[kind][i]);
    float ms = 0.f;
    if (e == cudaSuccess) e = cudaEventElapsedTime(&ms, g_timing.start[kind][i], g_timing.stop[kind][i]);
    if (e != cudaSuccess) return launch_error(e);
    tot += ms;
  }
  *total_ms = tot;
  *count = n;
  return FA_OK;
}

// Backward without any device allocation: the workspace is the library's
// fixed static scratch (see fa_bwd_noalloc in the header).
int fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                   void* dq, void* dk, void* dv, int B, int H, int N, int d, float scale, int causal,
                   const int* kv_lens, void* stream) {
  const int st = check_shape(B, H, N, d, scale);
  if (st != FA_OK) return st;
  if (fa_bwd_workspace_size(B, H, N, d) > FA_NOALLOC_SCRATCH_BYTES) return FA_ERR_SCRATCH_LIMIT;
  void* scratch = nullptr;
  size_t bytes = 0;
  const cudaError_t e = fa::noalloc_scratch(&scratch, &bytes);
  if (e != cudaSuccess) return launch_error(e);
  return fa_bwd(q, k, v, o, lse, dO, dq, dk, dv, B, H, N, d, scale, causal, kv_lens, scratch, bytes, stream);
}

static int bwd_varlen(const void* q, const void* k, const void* v, const void* o, const float* lse,
                      const void* dO, void* dq, void* dk, void* dv, const int* cu_seqlens_q,
                      const int* cu_seqlens_k, int batch, int H, int d, int total_q, int total_k, int max_seqlen_q,
                      int max_seqlen_k, float scale, int causal, void* workspace, size_t workspace_bytes,
                      void* stream, int det) {
  if (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv || !cu_seqlens_q || !cu_seqlens_k)
    return FA_ERR_INVALID;
  if (total_q < 1 || total_k < 1 || max_seqlen_q < 1 || max_seqlen_k < 1) return FA_ERR_INVALID;
  if (max_seqlen_q > total_q || max_seqlen_k > total_k) return FA_ERR_INVALID;
  int st = check_shape(batch, H, max_seqlen_q, d, scale);
  if (st != FA_OK) return st;
  if (static_cast<long long>(total_q) * H * d > (1LL << 40) || static_cast<long long>(total_k) * H * d > (1LL << 40))
    return FA_ERR_UNSUPPORTED;
  const void* ptrs[] = {q, k, v, o, lse, dO, dq, dk, dv};
  for (const void* p : ptrs)
    if (!aligned16(p)) return FA_ERR_UNSUPPORTED;
  const size_t need = fa_bwd_workspace_size(batch, H, max_seqlen_q, d);
  if (workspace == nullptr || workspace_bytes < need || !aligned16(workspace)) return FA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = check_cu_seqlens(cu_seqlens_q, batch, total_q, max_seqlen_q, s);
  if (st == FA_OK) st = check_cu_seqlens(cu_seqlens_k, batch, total_k, max_seqlen_k, s);
  if (st != FA_OK) return st;
  st = apply_test_hooks(s);
  if (st != FA_OK) return st;
  CUtensorMap tq, tk, tv, tdo;
  if (!encode_thd(&tq, q, H, total_q, d, 128) || !encode_thd(&tk, k, H, total_k, d, 128) ||
      !encode_thd(&tv, v, H, total_k, d, 128) || !encode_thd(&tdo, dO, H, total_q, d, 128))
    return launch_error(cudaErrorInvalidValue);
  const size_t rows = static_cast<size_t>(batch) * H * ((static_cast<size_t>(max_seqlen_q) + 127) / 128 * 128);
  fa::BwdArgs a;
  a.s = make_shape(batch, H, max_seqlen_q, d, scale, causal);
  a.s.Nk = max_seqlen_k;
  a.pk = fa::Packing{1, cu_seqlens_q, cu_seqlens_k, total_q, total_k};
  a.kv_lens = nullptr;
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.dO = dO;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  carve_workspace(&a, workspace, rows, d);
  a.deterministic = det;
  fa::LaunchMarks marks;
  const bool timed = next_marks(&marks, 1, 3);
  cudaError_t e = fa::launch_bwd(tq, tk, tv, tdo, a, s, timed ? &marks : nullptr);
  if (e != cudaSuccess) return launch_error(e);
  if (check_mode()) return fa_check_status(stream);
  return FA_OK;
}

int fa_bwd_varlen(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                  void* dq, void* dk, void* dv, const int* cu_seqlens_q, const int* cu_seqlens_k, int batch, int H,
                  int d, int total_q, int total_k, int max_seqlen_q, int max_seqlen_k, float scale, int causal,
                  void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_varlen(q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, batch, H, d, total_q, total_k,
                    max_seqlen_q, max_seqlen_k, scale, causal, workspace, workspace_bytes, stream, 0);
}

int fa_bwd_varlen_deterministic(const void* q, const void* k, const void* v, const void* o, const float* lse,
                                const void* dO, void* dq, void* dk, void* dv, const int* cu_seqlens_q,
                                const int* cu_seqlens_k, int batch, int H, int d, int total_q, int total_k,
                                int max_seqlen_q, int max_seqlen_k, float scale, int causal, void* workspace,
                                size_t workspace_bytes, void* stream) {
  return bwd_varlen(q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, batch, H, d, total_q, total_k,
                    max_seqlen_q, max_seqlen_k, scale, causal, workspace, workspace_bytes, stream, 1);
}

static int bwd_varlen_gqa(const void* q, const void* k, const void* v, const void* o, const float* lse,
                          const void* dO, void* dq, void* dk, void* dv, const int* cu_seqlens_q,
                          const int* cu_seqlens_k, int batch, int H, int H_kv, int d, int total_q, int total_k,
                          int max_seqlen_q, int max_seqlen_k, float scale, int causal, void* workspace,
                          size_t workspace_bytes, void* stream, int det) {
  if (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv || !cu_seqlens_q || !cu_seqlens_k)
    return FA_ERR_INVALID;
  int st = check_gqa(batch, H, H_kv, d, total_q, total_k, max_seqlen_q, max_seqlen_k, scale);
  if (st != FA_OK) return st;
  const void* ptrs[] = {q, k, v, o, lse, dO, dq, dk, dv};
  for (const void* p : ptrs)
    if (!aligned16(p)) return FA_ERR_UNSUPPORTED;
  const size_t need = fa_bwd_workspace_size(batch, H, max_seqlen_q, d);
  if (workspace == nullptr || workspace_bytes < need || !aligned16(workspace)) return FA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = check_cu_seqlens(cu_seqlens_q, batch, total_q, max_seqlen_q, s, true);
  if (st == FA_OK) st = check_cu_seqlens(cu_seqlens_k, batch, total_k, max_seqlen_k, s, true);
  if (st != FA_OK) return st;
  st = apply_test_hooks(s);
  if (st != FA_OK) return st;
  CUtensorMap tq, tk, tv, tdo;
  if (!encode_thd(&tq, q, H, total_q, d, 128) || !encode_thd(&tk, k, H_kv, total_k, d, 128) ||
      !encode_thd(&tv, v, H_kv, total_k, d, 128) || !encode_thd(&tdo, dO, H, total_q, d, 128))
    return launch_error(cudaErrorInvalidValue);
  const size_t rows = static_cast<size_t>(batch) * H * ((static_cast<size_t>(max_seqlen_q) + 127) / 128 * 128);
  fa::BwdArgs a;
  a.s = make_shape(batch, H, max_seqlen_q, d, scale, causal);
  a.s.Nk = max_seqlen_k;
  a.s.Hk = H_kv;
  a.pk = fa::Packing{1, cu_seqlens_q, cu_seqlens_k, total_q, total_k};
  a.kv_lens = nullptr;
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.dO = dO;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  carve_workspace(&a, workspace, rows, d);
  a.deterministic = det;
  fa::LaunchMarks marks;
  const bool timed = next_marks(&marks, 1, 3);
  cudaError_t e = fa::launch_bwd_gqa(tq, tk, tv, tdo, a, s, timed ? &marks : nullptr);
  if (e != cudaSuccess) return launch_error(e);
  if (check_mode()) return fa_check_status(stream);
  return FA_OK;
}

int fa_bwd_varlen_gqa(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                      void* dq, void* dk, void* dv, const int* cu_seqlens_q, const int* cu_seqlens_k, int batch,
                      int H, int H_kv, int d, int total_q, int total_k, int max_seqlen_q, int max_seqlen_k,
                      float scale, int causal, void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_varlen_gqa(q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, batch, H, H_kv, d, total_q,
                        total_k, max_seqlen_q, max_seqlen_k, scale, causal, workspace, workspace_bytes, stream, 0);
}

int fa_bwd_varlen_gqa_deterministic(const void* q, const void* k, const void* v, const void* o, const float* lse,
                                    const void* dO, void* dq, void* dk, void* dv, const int* cu_seqlens_q,
                                    const int* cu_seqlens_k, int batch, int H, int H_kv, int d, int total_q,
                                    int total_k, int max_seqlen_q, int max_seqlen_k, float scale, int causal,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_varlen_gqa(q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, batch, H, H_kv, d, total_q,
                        total_k, max_seqlen_q, max_seqlen_k, scale, causal, workspace, workspace_bytes, stream, 1);
}

size_t fa_decode_workspace_size(int B, int H, int d, int max_seq_len) {
  if (check_shape(B, H, max_seq_len, d, 1.f) != FA_OK) return 0;
  const DecodePlan pl = decode_plan(B, H, max_seq_len);
  const size_t parts = static_cast<size_t>(B) * H * pl.nsplit;
  return align_up(parts * d * 4, 256) + align_up(parts * 2 * 4, 256);
}

int fa_decode_paged(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                    const int* block_table, const int* seq_lens, int B, int H, int d, int num_blocks,
                    int block_size, int max_blocks_per_seq, int max_seq_len, float scale, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!q || !k_cache || !v_cache || !o || !lse || !block_table || !seq_lens) return FA_ERR_INVALID;
  if (num_blocks < 1 || max_blocks_per_seq < 1 || block_size < 1) return FA_ERR_INVALID;
  int st = check_shape(B, H, max_seq_len, d, scale);
  if (st != FA_OK) return st;
  if (block_size % 64 != 0) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_seq_len) > static_cast<long long>(max_blocks_per_seq) * block_size)
    return FA_ERR_INVALID;
  if (static_cast<long long>(num_blocks) * block_size > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  const void* ptrs[] = {q, k_cache, v_cache, o};
  for (const void* p : ptrs)
    if (!aligned16(p)) return FA_ERR_UNSUPPORTED;
  const DecodePlan pl = decode_plan(B, H, max_seq_len);
  const size_t need = fa_decode_workspace_size(B, H, d, max_seq_len);
  if (pl.nsplit > 1 && (workspace == nullptr || workspace_bytes < need || !aligned16(workspace)))
    return FA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = check_decode_tables(seq_lens, block_table, B, max_blocks_per_seq, block_size, num_blocks, max_seq_len, s);
  if (st != FA_OK) return st;
  st = apply_test_hooks(s);
  if (st != FA_OK) return st;
  CUtensorMap tk, tv;
  const int rows = num_blocks * block_size;
  if (!encode_thd(&tk, k_cache, H, rows, d, 64) || !encode_thd(&tv, v_cache, H, rows, d, 64))
    return launch_error(cudaErrorInvalidValue);
  fa::DecodeArgs a;
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.B = B;
  a.H = H;
  a.D = d;
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  a.max_blocks = max_blocks_per_seq;
  a.max_seq_len = max_seq_len;
  a.chunk = pl.chunk;
  a.nsplit = pl.nsplit;
  a.scale_log2 = scale * fa::kLog2e;
  const size_t parts = static_cast<size_t>(B) * H * pl.nsplit;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.part_o = pl.nsplit > 1 ? reinterpret_cast<float*>(ws) : nullptr;
  a.part_ml = pl.nsplit > 1 ? reinterpret_cast<float*>(ws + align_up(parts * d * 4, 256)) : nullptr;
  fa::LaunchMarks marks;
  const bool timed = next_marks(&marks, 4, pl.nsplit > 1 ? 2 : 1);
  cudaError_t e = fa::launch_decode(tk, tv, a, s, timed ? &marks : nullptr);
  if (e != cudaSuccess) return launch_error(e);
  if (check_mode()) return fa_check_status(stream);
  return FA_OK;
}

// Sizes of a shared-prefix step, checked, and its plan.
static int shared_sizes(fa::SharedArgs* a, int n_prefix, int B, int H, int H_kv, int d, int max_group,
                        int max_prefix_len, int max_seq_len, float scale) {
  if (n_prefix < 1 || max_group < 1 || H < 1 || H_kv < 1 || H % H_kv != 0) return FA_ERR_INVALID;
  if (max_group > B) return FA_ERR_INVALID;
  int st = check_shape(B, H, max_prefix_len, d, scale);
  if (st == FA_OK) st = check_shape(B, H, max_seq_len, d, scale);
  if (st == FA_OK) st = check_shape(n_prefix, H, 1, d, scale);
  if (st != FA_OK) return st;
  *a = fa::SharedArgs{};
  a->P = n_prefix;
  a->B = B;
  a->H = H;
  a->Hk = H_kv;
  a->D = d;
  a->max_group = max_group;
  a->max_prefix_len = max_prefix_len;
  a->max_seq_len = max_seq_len;
  a->scale_log2 = scale * fa::kLog2e;
  shared_plan(a);
  return FA_OK;
}

// Bytes of the partial O, then of the partial sums, of a plan.
static size_t shared_part_bytes(const fa::SharedArgs& a, size_t* o_bytes) {
  const size_t parts = static_cast<size_t>(a.B) * a.H * (a.prefix_splits + a.seq_splits);
  *o_bytes = align_up(parts * a.D * 4, 256);
  return *o_bytes + align_up(parts * 4, 256);
}

size_t fa_decode_shared_prefix_workspace_size(int n_prefix, int B, int H, int H_kv, int d, int max_group,
                                              int max_prefix_len, int max_seq_len) {
  fa::SharedArgs a;
  if (shared_sizes(&a, n_prefix, B, H, H_kv, d, max_group, max_prefix_len, max_seq_len, 1.f) != FA_OK) return 0;
  size_t o_bytes;
  return shared_part_bytes(a, &o_bytes);
}

int fa_decode_shared_prefix(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                            const int* prefix_table, const int* prefix_lens, const int* cu_prefix_seqs,
                            const int* block_table, const int* seq_lens, int n_prefix, int B, int H, int H_kv, int d,
                            int num_blocks, int block_size, int max_prefix_blocks, int max_blocks_per_seq,
                            int max_group, int max_prefix_len, int max_seq_len, float scale, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (!q || !k_cache || !v_cache || !o || !lse || !prefix_table || !prefix_lens || !cu_prefix_seqs || !block_table ||
      !seq_lens)
    return FA_ERR_INVALID;
  if (num_blocks < 1 || block_size < 1 || max_prefix_blocks < 1 || max_blocks_per_seq < 1) return FA_ERR_INVALID;
  fa::SharedArgs a;
  int st = shared_sizes(&a, n_prefix, B, H, H_kv, d, max_group, max_prefix_len, max_seq_len, scale);
  if (st != FA_OK) return st;
  if (block_size % 64 != 0) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_prefix_len) > static_cast<long long>(max_prefix_blocks) * block_size ||
      static_cast<long long>(max_seq_len) > static_cast<long long>(max_blocks_per_seq) * block_size)
    return FA_ERR_INVALID;
  if (static_cast<long long>(num_blocks) * block_size > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  const void* ptrs[] = {q, k_cache, v_cache, o};
  for (const void* p : ptrs)
    if (!aligned16(p)) return FA_ERR_UNSUPPORTED;
  size_t o_bytes;
  if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < shared_part_bytes(a, &o_bytes))
    return FA_ERR_WORKSPACE;
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.prefix_table = prefix_table;
  a.prefix_lens = prefix_lens;
  a.cu_seqs = cu_prefix_seqs;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  a.max_prefix_blocks = max_prefix_blocks;
  a.max_blocks = max_blocks_per_seq;
  a.part_o = static_cast<float*>(workspace);
  a.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + o_bytes);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = check_shared_tables(a, s);
  if (st != FA_OK) return st;
  st = apply_test_hooks(s);
  if (st != FA_OK) return st;
  CUtensorMap tk, tv;
  const int rows = num_blocks * block_size;
  if (!encode_thd(&tk, k_cache, H_kv, rows, d, 64) || !encode_thd(&tv, v_cache, H_kv, rows, d, 64))
    return launch_error(cudaErrorInvalidValue);
  fa::LaunchMarks marks;
  const bool timed = next_marks(&marks, 4, 2);
  if (a.prefix_tiles) {
    const fa::QTile qt = q_tile(H / H_kv);
    CUtensorMap tq;
    if (!encode_thd_group(&tq, q, H, B, d, qt)) return launch_error(cudaErrorInvalidValue);
    fa::LaunchMarks pm;
    const bool ptimed = next_marks(&pm, 0, 1);
    const cudaError_t pe = fa::launch_decode_prefix(tq, tk, tv, a, qt, s, ptimed ? &pm : nullptr);
    if (pe != cudaSuccess) return launch_error(pe);
  }
  cudaError_t e = fa::launch_decode_shared(tk, tv, a, s, timed ? &marks : nullptr);
  if (e != cudaSuccess) return launch_error(e);
  if (check_mode()) return fa_check_status(stream);
  return FA_OK;
}

int fa_quantize_fp8(const void* x, void* out, float* block_scale, int B, int H, int N, int d, int transpose,
                    void* stream) {
  if (!x || !out || !block_scale) return FA_ERR_INVALID;
  int st = check_shape(B, H, N, d, 1.f);
  if (st != FA_OK) return st;
  if (!aligned16(x) || !aligned16(out)) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * H > 65535) return FA_ERR_UNSUPPORTED;  // grid.y
  fa::QuantArgs a;
  a.x = x;
  a.out = static_cast<uint8_t*>(out);
  a.scale = block_scale;
  a.BH = B * H;
  a.N = N;
  a.D = d;
  a.Np = (N + 127) / 128 * 128;
  a.transpose = transpose ? 1 : 0;
  cudaError_t e = fa::launch_quantize_fp8(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return launch_error(e);
  if (check_mode()) return fa_check_status(stream);
  return FA_OK;
}

int fa_fwd_fp8(const void* q8, const void* k8, const void* v8t, const float* q_scale, const float* k_scale,
               const float* v_scale, void* o, float* lse, int B, int H, int N, int d, float scale, int causal,
               const int* kv_lens, void* stream) {
  if (!q8 || !k8 || !v8t || !q_scale || !k_scale || !v_scale || !o || !lse) return FA_ERR_INVALID;
  int st = check_shape(B, H, N, d, scale);
  if (st != FA_OK) return st;
  if (d != 128) return FA_ERR_UNSUPPORTED;
  const void* ptrs[] = {q8, k8, v8t, o};
  for (const void* p : ptrs)
    if (!aligned16(p)) return FA_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = check_kv_lens(kv_lens, B, N, s);
  if (st != FA_OK) return st;
  st = apply_test_hooks(s);
  if (st != FA_OK) return st;
  const long long BH = static_cast<long long>(B) * H;
  const long long Np = (static_cast<long long>(N) + 127) / 128 * 128;
  CUtensorMap tq, tk, tv;
  if (!encode_u8(&tq, q8, d, N, BH, d, static_cast<long long>(N) * d) ||
      !encode_u8(&tk, k8, d, N, BH, d, static_cast<long long>(N) * d) ||
      !encode_u8(&tv, v8t, Np, d, BH, Np, Np * d))
    return launch_error(cudaErrorInvalidValue);
  fa::Fp8FwdArgs a;
  a.s = make_shape(B, H, N, d, scale, causal);
  a.kv_lens = kv_lens;
  a.q_scale = q_scale;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.nb = static_cast<int>(Np / 128);
  a.o = o;
  a.lse = lse;
  fa::LaunchMarks marks;
  const bool timed = next_marks(&marks, 6, 1);
  cudaError_t e = fa::launch_fwd_fp8(tq, tk, tv, a, s, timed ? &marks : nullptr);
  if (e != cudaSuccess) return launch_error(e);
  if (check_mode()) return fa_check_status(stream);
  return FA_OK;
}

// Argument checks and arguments that both directions of the norm + rotation share.
static int norm_rope_args(fa::NormRopeArgs* a, const void* q, const void* k, const void* q_weight,
                          const void* k_weight, const float* cos, const float* sin, const int* positions, int T, int H,
                          int H_kv, int d, int rot, int max_pos, long long q_stride, long long k_stride, float eps,
                          int interleaved) {
  if (!q || !k || !q_weight || !k_weight || !positions) return FA_ERR_INVALID;
  if (rot != 0 && (!cos || !sin)) return FA_ERR_INVALID;  // without a rotation the tables are empty and not read
  if (H_kv < 1 || max_pos < 1 || rot < 0 || rot > d) return FA_ERR_INVALID;
  if (!std::isfinite(eps) || eps < 0.f) return FA_ERR_INVALID;
  int st = check_shape(T, H, 1, d, 1.f);
  if (st == FA_OK) st = check_shape(T, H_kv, 1, d, 1.f);
  if (st != FA_OK) return st;
  if (q_stride < static_cast<long long>(H) * d || k_stride < static_cast<long long>(H_kv) * d) return FA_ERR_INVALID;
  if (rot % 16 != 0 || q_stride % 8 != 0 || k_stride % 8 != 0) return FA_ERR_UNSUPPORTED;
  if (q_stride > (1LL << 40) / T || k_stride > (1LL << 40) / T) return FA_ERR_UNSUPPORTED;
  const void* ptrs[] = {q, k, q_weight, k_weight};
  for (const void* p : ptrs)
    if (!aligned16(p)) return FA_ERR_UNSUPPORTED;
  if (rot != 0 && (!aligned16(cos) || !aligned16(sin))) return FA_ERR_UNSUPPORTED;
  *a = fa::NormRopeArgs{};
  a->q = q;
  a->k = k;
  a->wq = q_weight;
  a->wk = k_weight;
  a->cos = cos;
  a->sin = sin;
  a->positions = positions;
  a->T = T;
  a->H = H;
  a->Hk = H_kv;
  a->D = d;
  a->rot = rot;
  a->max_pos = max_pos;
  a->q_stride = q_stride;
  a->k_stride = k_stride;
  a->eps = eps;
  a->interleaved = interleaved ? 1 : 0;
  return FA_OK;
}

// Check mode: copy the positions to the host and validate them.
static int check_positions(const int* positions, int T, int max_pos, cudaStream_t stream) {
  if (!check_mode()) return FA_OK;
  std::vector<int> h(T);
  cudaError_t e = cudaMemcpyAsync(h.data(), positions, sizeof(int) * T, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return launch_error(e);
  for (int p : h)
    if (p < 0 || p >= max_pos) return FA_ERR_INVALID;
  return FA_OK;
}

int fa_qk_norm_rope(const void* q, const void* k, const void* q_weight, const void* k_weight, const float* cos,
                    const float* sin, const int* positions, void* q_out, void* k_out, int T, int H, int H_kv, int d,
                    int rot, int max_pos, long long q_stride, long long k_stride, float eps, int interleaved,
                    void* stream) {
  fa::NormRopeArgs a;
  if (!q_out || !k_out) return FA_ERR_INVALID;
  int st = norm_rope_args(&a, q, k, q_weight, k_weight, cos, sin, positions, T, H, H_kv, d, rot, max_pos, q_stride,
                          k_stride, eps, interleaved);
  if (st != FA_OK) return st;
  if (!aligned16(q_out) || !aligned16(k_out)) return FA_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = check_positions(positions, T, max_pos, s);
  if (st != FA_OK) return st;
  a.yq = q_out;
  a.yk = k_out;
  cudaError_t e = fa::launch_norm_rope(a, s);
  if (e != cudaSuccess) return launch_error(e);
  if (check_mode()) return fa_check_status(stream);
  return FA_OK;
}

size_t fa_qk_norm_rope_bwd_workspace_size(int T, int H, int H_kv, int d) {
  if (check_shape(T, H, 1, d, 1.f) != FA_OK || check_shape(T, H_kv, 1, d, 1.f) != FA_OK) return 0;
  return static_cast<size_t>(fa::kNormRopeMaxCtas) * 2 * d * sizeof(float);
}

int fa_qk_norm_rope_bwd(const void* q, const void* k, const void* q_weight, const void* k_weight, const float* cos,
                        const float* sin, const int* positions, const void* dq_out, const void* dk_out, void* dq,
                        void* dk, float* dq_weight, float* dk_weight, int T, int H, int H_kv, int d, int rot,
                        int max_pos, long long q_stride, long long k_stride, long long dq_stride,
                        long long dk_stride, float eps, int interleaved, void* workspace, size_t workspace_bytes,
                        void* stream) {
  fa::NormRopeArgs a;
  if (!dq_out || !dk_out || !dq || !dk || !dq_weight || !dk_weight) return FA_ERR_INVALID;
  int st = norm_rope_args(&a, q, k, q_weight, k_weight, cos, sin, positions, T, H, H_kv, d, rot, max_pos, q_stride,
                          k_stride, eps, interleaved);
  if (st != FA_OK) return st;
  if (dq_stride < static_cast<long long>(H) * d || dk_stride < static_cast<long long>(H_kv) * d) return FA_ERR_INVALID;
  if (dq_stride % 8 != 0 || dk_stride % 8 != 0) return FA_ERR_UNSUPPORTED;
  if (dq_stride > (1LL << 40) / T || dk_stride > (1LL << 40) / T) return FA_ERR_UNSUPPORTED;
  const void* ptrs[] = {dq_out, dk_out, dq, dk};
  for (const void* p : ptrs)
    if (!aligned16(p)) return FA_ERR_UNSUPPORTED;
  if (workspace == nullptr || !aligned16(workspace) ||
      workspace_bytes < fa_qk_norm_rope_bwd_workspace_size(T, H, H_kv, d))
    return FA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = check_positions(positions, T, max_pos, s);
  if (st != FA_OK) return st;
  a.gq = dq_out;
  a.gk = dk_out;
  a.yq = dq;
  a.yk = dk;
  a.dwq = dq_weight;
  a.dwk = dk_weight;
  a.dq_stride = dq_stride;
  a.dk_stride = dk_stride;
  a.part = static_cast<float*>(workspace);
  cudaError_t e = fa::launch_norm_rope_bwd(a, s);
  if (e != cudaSuccess) return launch_error(e);
  if (check_mode()) return fa_check_status(stream);
  return FA_OK;
}

}  // extern "C"
