// Writing a paged KV cache and reading it back: new tokens appended with the
// position rotation on the way, to a cache of bf16 (the one fa_decode_paged and
// fa_decode_shared_prefix read) or to one held in 4 bits, and the 4-bit cache
// gathered into packed keys and values.
//
// Rotation, per row of d elements and pair (a, b) of its first rot ones:
//   (a, b) -> (a c - b s, b c + a s),
// every product and sum rounded to fp32 by itself (no fma), then to bf16: both
// caches start from the same bf16 row, and the codes below depend on nothing
// but that row.
//
// 4 bits: 64 consecutive elements share s = bf16((max - min) / 15) and z = min
// (exact: the elements are bf16) and stand for z + s code, with code the
// nearest integer to (x - z) / s, ties to even, in 0..15. The quotient is not
// computed: with k = rint((x - z) * (1 / s)), off by at most one, the remainder
// (x - z) - k s is exact in one fma (k s has 12 bits) and says which side of
// the border between two codes x lies on.
#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace fa {

namespace {

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t swap_halves(uint32_t w) { return __funnelshift_l(w, w, 16); }
__device__ __forceinline__ void words(const uint4& v, uint32_t (&w)[4]) {
  w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
}

// NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Cosines and signed sines of a lane's eight elements (from element e0 on) at a
// token's position, and the lane that holds their partners.
template <bool INTER>
struct Turn {
  bool on;      // this lane's elements are rotated
  int partner;  // lane of the warp (its own when interleaved)
  float c[8], s[8];
  __device__ __forceinline__ void load(const KvAppendArgs& a, long long token, int e0, int lane, bool wanted) {
    on = wanted && e0 < a.rot;
    partner = lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
    if (!on) return;
    const int half = a.rot / 2;
    const int pos = min(max(a.positions[token], 0), a.max_pos - 1);
    const long long row = static_cast<long long>(pos) * half;
    if constexpr (INTER) {
      const float4 c4 = *reinterpret_cast<const float4*>(a.cos + row + e0 / 2);
      const float4 s4 = *reinterpret_cast<const float4*>(a.sin + row + e0 / 2);
      const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = cc[i / 2], s[i] = (i & 1) ? ss[i / 2] : -ss[i / 2];
    } else {
      const bool second = e0 >= half;
      const long long at = row + (second ? e0 - half : e0);
      partner = second ? lane - half / 8 : lane + half / 8;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 c4 = *reinterpret_cast<const float4*>(a.cos + at + 4 * h);
        const float4 s4 = *reinterpret_cast<const float4*>(a.sin + at + 4 * h);
        const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) c[4 * h + i] = cc[i], s[4 * h + i] = second ? ss[i] : -ss[i];
      }
    }
  }
  // The row's packed words w, turned and rounded. Every lane of the warp calls
  // it; what is not rotated comes back bit for bit.
  __device__ __forceinline__ void apply(uint32_t (&w)[4]) const {
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = INTER ? swap_halves(w[i]) : __shfl_sync(0xffffffffu, w[i], partner);
    if (!on) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = pack_bf16x2(
          __fadd_rn(__fmul_rn(lo_f(w[i]), c[2 * i]), __fmul_rn(lo_f(p[i]), s[2 * i])),
          __fadd_rn(__fmul_rn(hi_f(w[i]), c[2 * i + 1]), __fmul_rn(hi_f(p[i]), s[2 * i + 1])));
  }
};

// The eight codes (element i in bits 4 i) of a lane's packed words, and the
// packed (s, z) of its group, which eight neighbouring lanes hold.
__device__ __forceinline__ uint32_t quantise(const uint32_t (&w)[4], uint32_t& sz) {
  float lo = min_nan(lo_f(w[0]), hi_f(w[0])), hi = max_nan(lo_f(w[0]), hi_f(w[0]));
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    lo = min_nan(lo, min_nan(lo_f(w[i]), hi_f(w[i])));
    hi = max_nan(hi, max_nan(lo_f(w[i]), hi_f(w[i])));
  }
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, off));
  }
  // (max - min) / 15 to bf16: the fp32 quotient in between rounds no other way
  // than the exact one would, whose bf16 ties are fp32 numbers times 15.
  uint32_t sb = pack_bf16x2(__fdiv_rn(__fsub_rn(hi, lo), 15.f), 0.f) & 0xFFFFu;
  float s = __uint_as_float(sb << 16);
  if (s < 0x1p-126f) s = 0.f, sb = 0u;  // 1 / s stays finite
  if (!(s <= 0x1.fep127f)) {            // a NaN, an infinity or a range past fp32: all of the group reads as NaN
    sz = 0x7FFF7FFFu;
    return 0u;
  }
  sz = sb | (__float_as_uint(lo) & 0xFFFF0000u);
  const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
  uint32_t codes = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = (i & 1) ? hi_f(w[i / 2]) : lo_f(w[i / 2]);
    const float t = __fsub_rn(x, lo);
    float k = rintf(t * inv);
    const float r = fmaf(-k, s, t), r2 = r + r;
    const bool odd = (static_cast<int>(k) & 1) != 0;
    if (r2 > s || (odd && r2 == s)) k += 1.f;
    if (r2 < -s || (odd && r2 == -s)) k -= 1.f;
    codes |= static_cast<uint32_t>(min(max(static_cast<int>(k), 0), 15)) << (4 * i);
  }
  return s > 0.f ? codes : 0u;
}

// Section and rows of a unit of the append: `n` consecutive heads of one token
// of q (0), k (1) or v (2).
struct AppendUnit {
  long long token;
  int section, head, n;
};
__device__ __forceinline__ AppendUnit append_unit(const KvAppendArgs& a, long long u) {
  const int per = a.q_slices + 2 * a.k_slices;
  AppendUnit t;
  t.token = u / per;
  int x = static_cast<int>(u - t.token * per);
  t.section = x < a.q_slices ? 0 : (x < a.q_slices + a.k_slices ? 1 : 2);
  if (t.section > 0) x -= a.q_slices + (t.section - 1) * a.k_slices;
  t.head = x * a.rows;
  t.n = min(a.rows, (t.section == 0 ? a.H : a.Hk) - t.head);
  return t;
}

}  // namespace

// d/8 lanes own a row, 16 bytes each; a group of lanes takes one unit.
template <int D, bool INTER, bool Q4>
__global__ void __launch_bounds__(256) fa_kv_append_kernel(const KvAppendArgs a) {
  constexpr int LPR = D / 8, GROUPS = 256 / LPR;
  const int lane = threadIdx.x & 31, l = threadIdx.x % LPR;
  const long long n_units = a.T * (a.q_slices + 2 * a.k_slices);
  const long long u = static_cast<long long>(blockIdx.x) * GROUPS + threadIdx.x / LPR;
  const AppendUnit t = append_unit(a, u < n_units ? u : 0);
  const int slot = t.section == 0 ? 0 : a.slots[t.token];
  // Slots outside the pool (negative ones mark padding) are not written.
  const bool live = u < n_units && (t.section == 0 || (slot >= 0 && slot < a.num_blocks * a.block_size));
  Turn<INTER> turn;
  turn.load(a, t.token, l * 8, lane, live && t.section < 2);
  const uint16_t* src = static_cast<const uint16_t*>(t.section == 0 ? a.q : (t.section == 1 ? a.k : a.v)) +
                        t.token * (t.section == 0 ? a.q_stride : (t.section == 1 ? a.k_stride : a.v_stride)) +
                        static_cast<long long>(t.head) * D + l * 8;
  for (int i = 0; i < a.rows; ++i) {
    const bool on = live && i < t.n;
    uint32_t w[4];
    words(on ? *reinterpret_cast<const uint4*>(src + static_cast<long long>(i) * D) : make_uint4(0u, 0u, 0u, 0u), w);
    turn.apply(w);
    const int head = t.head + i;
    if (!Q4 || t.section == 0) {
      uint16_t* dst = static_cast<uint16_t*>(t.section == 0 ? a.q_out : (t.section == 1 ? a.k_cache : a.v_cache)) +
                      ((t.section == 0 ? t.token * a.H : static_cast<long long>(slot) * a.Hk) + head) * D + l * 8;
      if (on) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if constexpr (Q4) {
      uint32_t sz;
      const uint32_t codes = quantise(w, sz);
      if (on && t.section > 0) {
        const int block = slot / a.block_size;
        const long long row =
            (static_cast<long long>(block) * a.Hk + head) * a.block_size + (slot - block * a.block_size);
        (static_cast<uint32_t*>(t.section == 1 ? a.k_cache : a.v_cache))[row * LPR + l] = codes;
        if ((l & 7) == 0) (static_cast<uint32_t*>(t.section == 1 ? a.k_scales : a.v_scales))[row * (D / 64) + l / 8] = sz;
      }
    }
  }
}

// Rows of the 4-bit cache as bf16, z + s code rounded once: a group of d/8
// lanes takes up to `rows` heads of one packed row of K or V.
template <int D>
__global__ void __launch_bounds__(256) fa_kv_gather_q4_kernel(const KvGatherArgs a) {
  constexpr int LPR = D / 8, GROUPS = 256 / LPR;
  const int l = threadIdx.x % LPR;
  const long long u = static_cast<long long>(blockIdx.x) * GROUPS + threadIdx.x / LPR;
  const long long row = u / (2 * a.slices);
  if (row >= a.total) return;
  const int x = static_cast<int>(u - row * (2 * a.slices));
  const bool is_v = x >= a.slices;
  const int head = (is_v ? x - a.slices : x) * a.rows;
  // The sequence of the row: the last b with cu[b] <= row.
  int lo = 0, hi = a.batch + 1;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (a.cu[mid] <= row) lo = mid + 1;
    else hi = mid;
  }
  const int b = lo - 1;
  if (b < 0 || b >= a.batch) return;  // a row of no sequence: left as it is
  const long long pos = row - a.cu[b] + (a.starts == nullptr ? 0 : a.starts[b]);
  const long long page = pos / a.block_size;
  int phys = -1;
  if (pos >= 0 && page < a.max_blocks) phys = a.block_table[static_cast<long long>(b) * a.max_blocks + page];
  const bool held = phys >= 0 && phys < a.num_blocks;  // others read as zeros
  const int off = static_cast<int>(pos - page * a.block_size);
  const uint32_t* codes = static_cast<const uint32_t*>(is_v ? a.v_codes : a.k_codes);
  const uint32_t* scales = static_cast<const uint32_t*>(is_v ? a.v_scales : a.k_scales);
  uint16_t* out = static_cast<uint16_t*>(is_v ? a.v : a.k) + row * a.Hk * D + l * 8;
  for (int h = head; h < min(head + a.rows, a.Hk); ++h) {
    const long long at = (static_cast<long long>(phys) * a.Hk + h) * a.block_size + off;
    const uint32_t c = held ? codes[at * LPR + l] : 0u, sz = held ? scales[at * (D / 64) + l / 8] : 0u;
    const float s = lo_f(sz), z = hi_f(sz);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = pack_bf16x2(fmaf(static_cast<float>((c >> (8 * i)) & 15u), s, z),
                         fmaf(static_cast<float>((c >> (8 * i + 4)) & 15u), s, z));
    *reinterpret_cast<uint4*>(out + static_cast<long long>(h) * D) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int D, bool Q4>
static cudaError_t launch_append_t(KvAppendArgs a, cudaStream_t stream) {
  constexpr int kGroups = 256 / (D / 8);
  a.rows = a.T * (a.H + 2 * a.Hk) >= 152 * 64 ? 4 : 1;
  a.q_slices = (a.H + a.rows - 1) / a.rows;
  a.k_slices = (a.Hk + a.rows - 1) / a.rows;
  const long long grid = (a.T * (a.q_slices + 2 * a.k_slices) + kGroups - 1) / kGroups;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  auto kern = a.interleaved ? fa_kv_append_kernel<D, true, Q4> : fa_kv_append_kernel<D, false, Q4>;
  kern<<<static_cast<unsigned>(grid), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream) {
  if (a.k_scales != nullptr) return a.D == 64 ? launch_append_t<64, true>(a, stream) : launch_append_t<128, true>(a, stream);
  return a.D == 64 ? launch_append_t<64, false>(a, stream) : launch_append_t<128, false>(a, stream);
}

cudaError_t launch_kv_gather_q4(const KvGatherArgs& args, cudaStream_t stream) {
  KvGatherArgs a = args;
  a.rows = std::min(a.Hk, 4);
  a.slices = (a.Hk + a.rows - 1) / a.rows;
  const int groups = 256 / (a.D / 8);
  const long long grid = (static_cast<long long>(a.total) * 2 * a.slices + groups - 1) / groups;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (a.D == 64) fa_kv_gather_q4_kernel<64><<<static_cast<unsigned>(grid), 256, 0, stream>>>(a);
  else fa_kv_gather_q4_kernel<128><<<static_cast<unsigned>(grid), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
