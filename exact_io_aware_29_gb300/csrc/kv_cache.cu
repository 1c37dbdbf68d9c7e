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
// nearest integer to (x - z) / s, ties to even, in 0..15. No quotient is
// rounded: a product with a reciprocal that is a little too small gives a
// candidate that is right or one too low, and a remainder that fp32 holds
// exactly says which.
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

// The larger and the smaller of each pair of bf16, NaN where either is.
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min_nan2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Cosines and signed sines of a lane's eight elements (from element e0 on) at a
// token's position, and the lane that holds their partners.
template <bool INTER>
struct Turn {
  bool on;      // this lane's elements are rotated
  int partner;  // lane of the warp (its own when interleaved)
  uint64_t c[4], s[4];  // pairs
  __device__ __forceinline__ void load(const KvAppendArgs& a, long long token, int e0, int lane, bool wanted) {
    on = wanted && e0 < a.rot;
    partner = lane;
    if (!on) return;
    const int half = a.rot / 2;
    const int pos = min(max(a.positions[token], 0), a.max_pos - 1);
    const long long row = static_cast<long long>(pos) * half;
    if constexpr (INTER) {
      const float4 c4 = *reinterpret_cast<const float4*>(a.cos + row + e0 / 2);
      const float4 s4 = *reinterpret_cast<const float4*>(a.sin + row + e0 / 2);
      const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = f2_pack(cc[i], cc[i]), s[i] = f2_pack(-ss[i], ss[i]);
    } else {
      const bool second = e0 >= half;
      const long long at = row + (second ? e0 - half : e0);
      partner = second ? lane - half / 8 : lane + half / 8;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 c4 = *reinterpret_cast<const float4*>(a.cos + at + 4 * h);
        const float4 s4 = *reinterpret_cast<const float4*>(a.sin + at + 4 * h);
        const float sign = second ? 1.f : -1.f;
        c[2 * h] = f2_pack(c4.x, c4.y), c[2 * h + 1] = f2_pack(c4.z, c4.w);
        s[2 * h] = f2_pack(sign * s4.x, sign * s4.y), s[2 * h + 1] = f2_pack(sign * s4.z, sign * s4.w);
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
    for (int i = 0; i < 4; ++i) {
      // (Packed products with scalar sums: a packed product and sum are contracted into one rounding.)
      float x0, x1, y0, y1;
      f2_unpack(f2_mul(f2_pack(lo_f(w[i]), hi_f(w[i])), c[i]), x0, x1);
      f2_unpack(f2_mul(f2_pack(lo_f(p[i]), hi_f(p[i])), s[i]), y0, y1);
      w[i] = pack_bf16x2(__fadd_rn(x0, y0), __fadd_rn(x1, y1));
    }
  }
};

// The eight codes (element i in bits 4 i) of a lane's packed words, and the
// packed (s, z) of its group, which eight neighbouring lanes hold.
__device__ __forceinline__ uint32_t quantise(const uint32_t (&w)[4], uint32_t& sz) {
  uint32_t lo2 = min_nan2(min_nan2(w[0], w[1]), min_nan2(w[2], w[3]));
  uint32_t hi2 = max_nan2(max_nan2(w[0], w[1]), max_nan2(w[2], w[3]));
  lo2 = min_nan2(lo2, swap_halves(lo2));
  hi2 = max_nan2(hi2, swap_halves(hi2));
  uint32_t ends = (lo2 & 0xFFFFu) | (hi2 & 0xFFFF0000u);  // minimum and maximum
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) {
    const uint32_t x = __shfl_xor_sync(0xffffffffu, ends, off);
    ends = (min_nan2(ends, x) & 0xFFFFu) | (max_nan2(ends, x) & 0xFFFF0000u);
  }
  const float lo = lo_f(ends), hi = hi_f(ends);
  // s: the bf16 number below the product, or the next one if the range is over
  // 15 times their midpoint (13 bits: exact), or just that and the lower one odd.
  const float range = __fsub_rn(hi, lo);
  uint32_t sb = __float_as_uint(range * (1.f / 15.f)) >> 16;
  const float border = 15.f * __uint_as_float(sb << 16 | 0x8000u);
  if (range > border || (range == border && (sb & 1u))) ++sb;
  if (sb < 0x80u) sb = 0u;         // below 2^-126, whose reciprocal is not finite
  const bool bad = sb >= 0x7F80u;  // a NaN, an infinity or a range past fp32: all of the group reads as NaN
  sz = bad ? 0x7FFF7FFFu : (sb | ends << 16);
  const float s = __uint_as_float(sb << 16);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  inv *= 1.f - 0x1p-21f;  // 2^-23 off at most: now between (1 - 2^-20) / s and 1 / s
  const int half = __float_as_int(0.5f * s);
  const float magic = 12582912.f;  // 1.5 2^23: sums with it are integers, in their low bits
  const uint64_t lo2f = f2_pack(lo, lo), inv2 = f2_pack(inv, inv), magic2 = f2_pack(magic, magic);
  const uint64_t minus = f2_pack(-s, -s);
  uint32_t codes = 0u - 0x4B400000u * 0x11111111u;  // the bits of 1.5 2^23 in each term, taken out
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t t = f2_sub(f2_pack(lo_f(w[i]), hi_f(w[i])), lo2f);
    const uint64_t kf = f2_fma(t, inv2, magic2);
    const uint64_t r = f2_fma(f2_sub(kf, magic2), minus, t);
    float k[2], rest[2];
    f2_unpack(kf, k[0], k[1]);
    f2_unpack(r, rest[0], rest[1]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      // One more if the remainder is over s / 2, or just that and k odd. (t <= 15 s (1 + 2^-8): codes stay below 16.)
      int c = __float_as_int(k[e]);
      if (rest[e] > __int_as_float(half - (c & 1))) ++c;
      codes += static_cast<uint32_t>(c) << (4 * (2 * i + e));
    }
  }
  return sb != 0u && !bad ? codes : 0u;
}

}  // namespace

// d/8 lanes own a row, 16 bytes each; a group of lanes takes up to R
// consecutive heads of one token, all read before the first is written. The CTAs
// of q, k and v take turns (`ratio` of q, one of k, one of v): those that
// quantise are bound by their instructions, the others by HBM.
// Registers: 48, or 64 with eight rows, into which the forms that quantise do not
// quite fit (8 to 24 bytes spilled). A CTA less per SM, which spills nothing, is
// slower: 16384 tokens, 16 + 4 heads, 40.5 us instead of 37.3 at d 128, 22.8
// instead of 21.2 at d 64.
template <int D, bool INTER, bool Q4, int R>
__global__ void __launch_bounds__(256, R == 8 ? 4 : 5) fa_kv_append_kernel(const KvAppendArgs a) {
  constexpr int LPR = D / 8, GROUPS = 256 / LPR;
  // Launched programmatically: nothing of the stream's is read or written before
  // this. (What follows is not let in early: CTAs that only wait would take room.
  // 512 tokens, 16 + 4 heads, written in 4 bits and read back: 6.2 us if it is,
  // 5.9 as it stands; 16384 tokens, 32 + 8 heads: 80.4 either way.)
  griddep_wait();
  const int lane = threadIdx.x & 31, l = threadIdx.x % LPR;
  int section = 0, cta = blockIdx.x;
  if (cta < a.k_ctas * (a.ratio + 2)) {
    const int turn = cta / (a.ratio + 2), at = cta - turn * (a.ratio + 2);
    section = max(at - a.ratio + 1, 0);
    cta = section == 0 ? turn * a.ratio + at : turn;
  } else {
    cta -= 2 * a.k_ctas;  // the rest of q's
  }
  const int slices = section == 0 ? a.q_slices : a.k_slices, heads = section == 0 ? a.H : a.Hk;
  const long long u = static_cast<long long>(cta) * GROUPS + threadIdx.x / LPR;
  long long token;
  int head0;
  if (a.T * slices <= 0x7fffffffLL) {  // a 64-bit division would take half as long as a row
    const unsigned t = static_cast<unsigned>(u) / static_cast<unsigned>(slices);
    token = t;
    head0 = (static_cast<unsigned>(u) - t * slices) * R;
  } else {
    token = u / slices;
    head0 = static_cast<int>(u - token * slices) * R;
  }
  token = min(token, a.T - 1);
  const int slot = section == 0 ? 0 : a.slots[token];
  // Slots outside the pool (negative ones mark padding) are not written.
  const bool live = u < a.T * slices && (section == 0 || (slot >= 0 && slot < a.num_blocks * a.block_size));
  const int n = live ? min(R, heads - head0) : 0;
  const uint16_t* src = static_cast<const uint16_t*>(section == 0 ? a.q : (section == 1 ? a.k : a.v)) +
                        token * (section == 0 ? a.q_stride : (section == 1 ? a.k_stride : a.v_stride)) +
                        static_cast<long long>(head0) * D + l * 8;
  uint4 x[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    x[i] = i < n ? *reinterpret_cast<const uint4*>(src + i * D) : make_uint4(0u, 0u, 0u, 0u);
  Turn<INTER> turn;
  if (section < 2) turn.load(a, token, l * 8, lane, live);
  const int block = slot / a.block_size;
  // First head's row of the output, in rows of d elements.
  const long long row =
      section == 0 ? token * a.H + head0
      : Q4         ? (static_cast<long long>(block) * a.Hk + head0) * a.block_size + slot - block * a.block_size
                   : static_cast<long long>(slot) * a.Hk + head0;
  void* out = section == 0 ? a.q_out : (section == 1 ? a.k_cache : a.v_cache);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    uint32_t w[4];
    words(x[i], w);
    if (section < 2) turn.apply(w);
    if (!Q4 || section == 0) {
      if (i < n)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + (row + i) * D + l * 8) =
            make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      uint32_t sz;
      const uint32_t codes = quantise(w, sz);
      const long long at = row + static_cast<long long>(i) * a.block_size;
      if (i < n) {
        static_cast<uint32_t*>(out)[at * LPR + l] = codes;
        if ((l & 7) == 0) static_cast<uint32_t*>(section == 1 ? a.k_scales : a.v_scales)[at * (D / 64) + l / 8] = sz;
      }
    }
  }
}

// The number of entries of cu[0 .. n) that are <= row (cu ascends), by all lanes
// of a warp: 32 entries a turn.
__device__ __forceinline__ int count_upto(const int* cu, int n, int row, int lane) {
  int lo = 0, hi = n;
  for (;;) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const int c = __popc(__ballot_sync(0xffffffffu, at < hi && cu[min(at, n - 1)] <= row));
    if (step <= 1) return lo + c;
    hi = min(hi, lo + c * step);
    lo = c > 0 ? lo + (c - 1) * step + 1 : lo;
    if (lo >= hi) return lo;
  }
}

// Rows of the 4-bit cache as bf16, z + s code rounded once (fma.rn.bf16x2: the
// codes are exact, 128 + code being the bits of a nibble under 128's exponent).
// A CTA takes `tokens` packed rows: its warps look up where they lie, then
// groups of d/8 lanes take a token's K or V each, four heads at a time.
// (110000 tokens of 8 heads, d 128: 75.4 us with 8 rows a CTA, 77.4 with 4, 78.2
// with 16, 81.8 with 32; eight heads at a time 77.8.)
constexpr int kGatherTokens = 8;
template <int D>
__global__ void __launch_bounds__(256) fa_kv_gather_q4_kernel(const KvGatherArgs a) {
  constexpr int LPR = D / 8, GROUPS = 256 / LPR, R = 4;
  __shared__ long long place[kGatherTokens];  // row of head 0 in the cache; -1: reads as zeros; -2: of no sequence
  griddep_wait();  // as above
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = threadIdx.x % LPR;
  const int row0 = blockIdx.x * a.tokens, count = min(a.tokens, a.total - row0);
  for (int t = warp; t < count; t += 8) {
    const int row = row0 + t, b = count_upto(a.cu, a.batch + 1, row, lane) - 1;
    if (lane > 0) continue;
    long long at = -2;
    if (b >= 0 && b < a.batch) {
      const long long pos = static_cast<long long>(row) - a.cu[b] + (a.starts == nullptr ? 0 : a.starts[b]);
      at = -1;
      if (pos >= 0 && pos < static_cast<long long>(a.max_blocks) * a.block_size) {
        const int page = static_cast<int>(static_cast<unsigned long long>(pos) / static_cast<unsigned>(a.block_size));
        const int phys = a.block_table[static_cast<long long>(b) * a.max_blocks + page];
        if (phys >= 0 && phys < a.num_blocks)
          at = static_cast<long long>(phys) * a.Hk * a.block_size + (pos - static_cast<long long>(page) * a.block_size);
      }
    }
    place[t] = at;
  }
  __syncthreads();
  for (int u = threadIdx.x / LPR; u < 2 * count; u += GROUPS) {
    const int t = u >> 1;
    const bool is_v = u & 1;
    const long long at = place[t];
    if (at < -1) continue;
    const uint32_t* codes = static_cast<const uint32_t*>(is_v ? a.v_codes : a.k_codes) + at * LPR + l;
    const uint32_t* scales = static_cast<const uint32_t*>(is_v ? a.v_scales : a.k_scales) + at * (D / 64) + l / 8;
    uint16_t* out = static_cast<uint16_t*>(is_v ? a.v : a.k) + static_cast<long long>(row0 + t) * a.Hk * D + l * 8;
    for (int h0 = 0; h0 < a.Hk; h0 += R) {
      uint32_t c[R], sz[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const bool on = at >= 0 && h0 + i < a.Hk;
        const long long h = static_cast<long long>(h0 + i) * a.block_size;
        c[i] = on ? codes[h * LPR] : 0u;
        sz[i] = on ? scales[h * (D / 64)] : 0u;
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (h0 + i >= a.Hk) break;
        const uint32_t s2 = __byte_perm(sz[i], 0u, 0x1010), z2 = __byte_perm(sz[i], 0u, 0x3232);
        uint32_t p[4];  // elements k and k + 4
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t v = ((c[i] >> (4 * k)) & 0x000F000Fu) | 0x43004300u;
          asm("{\n\t.reg .b32 x;\n\tadd.rn.bf16x2 x, %1, %4;\n\tfma.rn.bf16x2 %0, x, %2, %3;\n\t}"
              : "=r"(p[k])
              : "r"(v), "r"(s2), "r"(z2), "r"(0xC300C300u));
        }
        *reinterpret_cast<uint4*>(out + static_cast<long long>(h0 + i) * D) =
            make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                       __byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632));
      }
    }
  }
}

template <int D, bool Q4, int R>
static cudaError_t launch_append_r(KvAppendArgs a, cudaStream_t stream) {
  constexpr int kGroups = 256 / (D / 8);
  a.q_slices = std::max((a.H + R - 1) / R, 1);
  a.k_slices = (a.Hk + R - 1) / R;
  auto ctas = [&](long long units) { return (units + kGroups - 1) / kGroups; };
  const long long q = a.H > 0 ? ctas(a.T * a.q_slices) : 0, k = ctas(a.T * a.k_slices);
  if (q + 2 * k > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  a.k_ctas = static_cast<int>(k);
  a.ratio = static_cast<int>(q / k);
  auto kern = a.interleaved ? fa_kv_append_kernel<D, true, Q4, R> : fa_kv_append_kernel<D, false, Q4, R>;
  return launch_maybe_pdl(kern, dim3(static_cast<unsigned>(q + 2 * k)), dim3(256), 0, stream, true, a);
}

template <int D, bool Q4>
static cudaError_t launch_append_t(const KvAppendArgs& a, cudaStream_t stream) {
  // Four rows to a group of lanes once that leaves two CTAs for every SM, and
  // eight of those that are quantised where there are many. (16384 tokens, d 128,
  // with one, two, four and eight rows: 32 + 8 heads 111, 78, 61 and 61 us in
  // bf16; written in 4 bits and read back, 138, 115, 82 and 78 us, 16 + 4 heads
  // 73, 61, 46 and 50; 512 tokens of those 5.9, 5.8, 6.7 and 6.8.)
  const long long lanes = a.T * (a.H + 2 * a.Hk) * (D / 8);
  if constexpr (Q4 && D == 128) {
    if (a.Hk >= 8 && lanes >= 152LL * 4 * 256 * 8) return launch_append_r<D, Q4, 8>(a, stream);
  }
  return lanes >= 152LL * 2 * 256 * 4 ? launch_append_r<D, Q4, 4>(a, stream) : launch_append_r<D, Q4, 1>(a, stream);
}

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream) {
  if (a.k_scales != nullptr)
    return a.D == 64 ? launch_append_t<64, true>(a, stream) : launch_append_t<128, true>(a, stream);
  return a.D == 64 ? launch_append_t<64, false>(a, stream) : launch_append_t<128, false>(a, stream);
}

cudaError_t launch_kv_gather_q4(const KvGatherArgs& args, cudaStream_t stream) {
  KvGatherArgs a = args;
  a.tokens = std::min(std::max(a.total / (152 * 4), 1), kGatherTokens);
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(a.total) + a.tokens - 1) / a.tokens);
  return launch_maybe_pdl(a.D == 64 ? fa_kv_gather_q4_kernel<64> : fa_kv_gather_q4_kernel<128>, dim3(grid), dim3(256),
                          0, stream, true, a);
}

}  // namespace fa
