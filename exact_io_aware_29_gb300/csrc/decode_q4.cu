// Decoding steps over a paged KV cache held in 4 bits, with grouped heads: the
// n_new newest queries of each sequence attend to its cached keys (bottom-right
// causal: query i of n_new sees the keys c <= L - n_new + i). 64 consecutive
// elements of a key or value row stand for z + s code (kv_cache.cu), so with
// the codes as integers
//   q . k = sum over groups g of  s_g sum_{e in g} q_e code_e + z_g sum_{e in g} q_e,
//   O     = sum over keys of  (p s_g) code_e + p z_g,  over sum p:
// the products run on the codes and scales stay outside of them, in fp32.
//
// A key and head is 2 (d/2 + d/16) bytes against 4 d flops per row, a row being
// one (query, head) of the key head. The products run on mma.sync with the
// codes as the A operand (16 keys, or 16 dimensions of V transposed) and eight
// rows as n: up to eight heads of a key head pad nothing, and the operand is
// made in registers from the words as they lie in the cache (tcgen05 would take
// them through shared or tensor memory). Both products are f16: a nibble in the
// low bits of an f16 is code 2^-24 (a subnormal, exact), four bits further up
// code 2^-20, so one AND makes two codes.
//   Q K^T: the row of q is scaled to [2^14, 2^15) by a power of two, so that its
//   f16 is exact (below 2^-29 of the row's largest: rounded at 2^-40 of it).
//   P V: p s is scaled by a power of two of the row and group, such that the
//   largest so far is at most 2^15 and was 2^9 or more when the power was
//   chosen: rounded to f16, 2^-12 of a term (an eighth of what the rounding of
//   O to bf16 costs), at terms down to 2^-23 of the largest.
// The logic pipe, not the tensor cores, stands nearest to HBM: about 125
// instructions on it for 16 keys, of 200 that HBM leaves time for (d 128).
//
// A persistent grid shares the 128-key tiles of all sequences and key heads out
// evenly, in order, whatever their lengths: a CTA takes a run of tiles, whole
// items (row block, key head) and the ends of two. One warp streams the tiles
// through a ring with bulk copies (a block's keys of one head lie together:
// codes, then scales, in up to 8 pieces), the others compute on 16 keys each.
// Softmax statistics and sums are fp32. A cut item's parts are joined in the
// order of the keys by a second kernel.
#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace fa {

template <int D, int NT>
struct Q4Cfg {
  static constexpr int TK = kQ4Tile;               // keys per tile
  static constexpr int NG = D / 64;                // groups of a row
  static constexpr int ROWS = 8 * NT;              // rows of an item
  static constexpr int CODE_BYTES = TK * D / 2;
  static constexpr int SCALE_BYTES = TK * NG * 4;
  static constexpr int OFF_KS = CODE_BYTES, OFF_VC = OFF_KS + SCALE_BYTES, OFF_VS = OFF_VC + CODE_BYTES;
  static constexpr int STAGE_BYTES = 2 * (CODE_BYTES + SCALE_BYTES);
  static constexpr int CWARPS = 4;                 // consumer warps
  static constexpr int THREADS = (CWARPS + 1) * 32;
  static constexpr int CTAS = (D == 64 ? 4 : 3) - (NT - 1);  // per SM
  static constexpr int STAGES = D == 64 ? 5 : 2 + NT;
  static constexpr int RED_STRIDE = D + 4;         // floats of a row in the join of the warps
  static constexpr int OFF_RED = STAGES * STAGE_BYTES;
  static constexpr int OFF_ML = OFF_RED + CWARPS * ROWS * RED_STRIDE * 4;
  static constexpr int OFF_BAR = OFF_ML + CWARPS * ROWS * 2 * 4;
  static constexpr int OFF_SCAN = OFF_BAR + 2 * STAGES * 8;
  static constexpr int SMEM_BYTES = OFF_SCAN + STAGES * 4 + 4 + (CWARPS + 1) * 4 + 16;
  static_assert(SMEM_BYTES * CTAS <= 227 * 1024 - (CTAS - 1) * 1024, "fits in an SM");
};

namespace {

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit elements, two neighbours of a row to a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
__device__ __forceinline__ int exponent(float x) { return static_cast<int>((__float_as_uint(x) >> 23) & 255u) - 127; }
// max(a, b), NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

constexpr float kNoLogit = -1e30f;  // the maximum before the first key; below every finite logit

__device__ __forceinline__ int q4_len(const Q4DecodeArgs& a, int b) {
  return min(max(a.seq_lens[b], 0), a.max_seq_len);
}
__device__ __forceinline__ int q4_tiles(int L) { return (L + kQ4Tile - 1) / kQ4Tile; }
// First tile of CTA c's share of `total`.
__device__ __forceinline__ int q4_share(int c, int total, int ctas) {
  return static_cast<int>(static_cast<long long>(c) * total / ctas);
}

// A CTA's way along its run of tiles [x, end): item by item.
struct Q4Walk {
  int b, item, tile, left;  // sequence, (key head, row block) of it, first tile in it, tiles of the run from here on
  int L, n;                 // length, tiles and
  int here;                 // tiles of the run in this item
  __device__ __forceinline__ void enter(const Q4DecodeArgs& a) {
    L = q4_len(a, b);
    n = q4_tiles(L);
    here = min(n - tile, left);
  }
  __device__ __forceinline__ bool next(const Q4DecodeArgs& a) {  // false at the end of the run
    left -= here;
    if (left <= 0) return false;
    tile = 0;
    if (++item < a.Hk * a.row_blocks) {
      here = min(n, left);
      return true;
    }
    item = 0;
    do ++b; while (q4_len(a, b) == 0);  // tiles are left, so there is one
    enter(a);
    return true;
  }
};

// Row r of row block `blk` of (b, kvh) as the flattened row (b * n_new + query) * H + head.
__device__ __forceinline__ long long q4_row(const Q4DecodeArgs& a, int b, int kvh, int row) {
  const int G = a.H / a.Hk;
  return (static_cast<long long>(b) * a.n_new + row / G) * a.H + kvh * G + row % G;
}

// What a lane holds of the queries: lane (r, c) = (lane / 4, lane % 4).
template <int D, int NT>
struct Q4Rows {
  static constexpr int NG = D / 64;
  uint32_t q[NT][NG][4][2];  // B fragments of row 8 j + r, k-step t of group g
  float qs[NT][2];           // of rows 8 j + 2 c + {0, 1}: what a product of codes is multiplied by
  float sum[NT][NG][2];      // scale log2e times the sum of the row's group
};

template <int D, int NT>
__device__ __forceinline__ void q4_load_rows(const Q4DecodeArgs& a, int b, int kvh, int row0, int rows, int lane,
                                             Q4Rows<D, NT>& R) {
  constexpr int NG = D / 64;
  const int r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const bool on = j * 8 + r < rows;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                      (on ? q4_row(a, b, kvh, row0 + j * 8 + r) : 0LL) * D);
    uint32_t w[NG][8];  // elements 64 g + 16 c + {0 .. 15}
    float mx = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint4 x = on ? src[g * 8 + c * 2] : make_uint4(0u, 0u, 0u, 0u);
      const uint4 y = on ? src[g * 8 + c * 2 + 1] : make_uint4(0u, 0u, 0u, 0u);
      w[g][0] = x.x, w[g][1] = x.y, w[g][2] = x.z, w[g][3] = x.w;
      w[g][4] = y.x, w[g][5] = y.y, w[g][6] = y.z, w[g][7] = y.w;
#pragma unroll
      for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fmaxf(fabsf(lo_f(w[g][i])), fabsf(hi_f(w[g][i]))));
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // 2^shift q is below 2^15; 2^shift and 2^(24 - shift) are fp32 numbers.
    const int shift = min(max(14 - exponent(mx), -100), 100);
    const float up = pow2(shift);
    float s[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      s[g] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s[g] += lo_f(w[g][i]) + hi_f(w[g][i]);
      s[g] += __shfl_xor_sync(0xffffffffu, s[g], 1);
      s[g] += __shfl_xor_sync(0xffffffffu, s[g], 2);
      s[g] *= a.scale_log2;
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // word 2 c + h of the codes: elements 8 h + {0 .. 7}
        const uint32_t* x = &w[g][4 * h];
        // Nibbles (0, 4), (1, 5) 16-fold, (2, 6), (3, 7) 16-fold.
        R.q[j][g][2 * h][0] = pack_f16x2(lo_f(x[0]) * up, lo_f(x[2]) * up);
        R.q[j][g][2 * h][1] = pack_f16x2(hi_f(x[0]) * (up * 0.0625f), hi_f(x[2]) * (up * 0.0625f));
        R.q[j][g][2 * h + 1][0] = pack_f16x2(lo_f(x[1]) * up, lo_f(x[3]) * up);
        R.q[j][g][2 * h + 1][1] = pack_f16x2(hi_f(x[1]) * (up * 0.0625f), hi_f(x[3]) * (up * 0.0625f));
      }
    }
    const float down = a.scale_log2 * pow2(24 - shift);
    // To the lanes of the C fragments' columns: row 8 j + 2 c + i comes from lane (2 c + i, .).
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      R.qs[j][i] = __shfl_sync(0xffffffffu, down, (2 * c + i) * 4);
#pragma unroll
      for (int g = 0; g < NG; ++g) R.sum[j][g][i] = __shfl_sync(0xffffffffu, s[g], (2 * c + i) * 4);
    }
  }
}

// Running softmax of a lane's columns (rows 8 j + 2 c + {0, 1}): maximum and
// powers are the same in all lanes of a column, the sums are the lane's own.
template <int D, int NT>
struct Q4State {
  static constexpr int NG = D / 64;
  float o[NT][NG][4][4];  // C fragments: dimensions 64 g + 8 r + 2 t (c0 c1) and, 16-fold, the next one (c2 c3)
  float m[NT][2], l[NT][2], z[NT][NG][2];
  float up[NT][NG][2];    // the power of two that p s is multiplied by
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[j][i] = kNoLogit, l[j][i] = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) z[j][g][i] = 0.f, up[j][g][i] = 0x1p120f;
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
#pragma unroll
        for (int t = 0; t < 4; ++t) o[j][g][t][0] = o[j][g][t][1] = o[j][g][t][2] = o[j][g][t][3] = 0.f;
      }
    }
  }
};

// The largest of a column over its lanes.
__device__ __forceinline__ float column_max(float x) {
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

// 16 keys of a tile from key k0 of it on. MASKED: some of them may be hidden
// from some rows (row x sees the tile's keys below open + (row0 + x) / G - row0 / G),
// or past the sequence (`left` keys of the tile are in it), or in a block that
// is not in the pool (held = false: they read as zeros).
template <int D, int NT, bool MASKED>
__device__ __forceinline__ void q4_slice(const uint8_t* st, int k0, int lane, bool held, int left, int open, int row0,
                                         int G, const Q4Rows<D, NT>& R, Q4State<D, NT>& S) {
  using C = Q4Cfg<D, NT>;
  constexpr int NG = D / 64;
  const int r = lane >> 2, c = lane & 3;
  // Row i of the A operand of Q K^T, and k index i of P V, is key (i >> 1) + 4 (i & 1)
  // of its eight: the lanes of a load then meet two banks' worth of rows, not one.
  const int ka = k0 + (r >> 1) + 4 * (r & 1);
  float sc[NT][2][2];  // [key ka + 8 h][row i]
  float vs[NG][2], vz[NG][2];
  {
    float ks[NG][2], kz[NG][2], acc[NT][NG][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t* pk = reinterpret_cast<const uint32_t*>(st + C::OFF_KS) + (ka + 8 * h) * NG;
      const uint32_t* pv = reinterpret_cast<const uint32_t*>(st + C::OFF_VS) + (ka + 8 * h) * NG;
      const bool on = !MASKED || (held && ka + 8 * h < left);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t k = on ? pk[g] : 0u, v = on ? pv[g] : 0u;
        ks[g][h] = lo_f(k), kz[g][h] = hi_f(k);
        vs[g][h] = lo_f(v), vz[g][h] = hi_f(v);
      }
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint2 x = *reinterpret_cast<const uint2*>(st + ka * (D / 2) + g * 32 + c * 8);
      const uint2 y = *reinterpret_cast<const uint2*>(st + (ka + 8) * (D / 2) + g * 32 + c * 8);
      const uint32_t wx[4] = {x.x, x.x >> 8, x.y, x.y >> 8}, wy[4] = {y.x, y.x >> 8, y.y, y.y >> 8};
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j][g][0] = acc[j][g][1] = acc[j][g][2] = acc[j][g][3] = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
          mma_f16(acc[j][g], wx[t] & 0x000F000Fu, wy[t] & 0x000F000Fu, wx[t] & 0x00F000F0u, wy[t] & 0x00F000F0u,
                  R.q[j][g][t][0], R.q[j][g][t][1]);
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = acc[j][0][2 * h + i] * ks[0][h], y = kz[0][h] * R.sum[j][0][i];
#pragma unroll
          for (int g = 1; g < NG; ++g) {
            x = fmaf(acc[j][g][2 * h + i], ks[g][h], x);
            y = fmaf(kz[g][h], R.sum[j][g][i], y);
          }
          sc[j][h][i] = fmaf(x, R.qs[j][i], y);
        }
      }
    }
  }
  bool seen[NT][2][2], higher = false;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        seen[j][h][i] =
            !MASKED || (ka + 8 * h < left && ka + 8 * h < open + (row0 + j * 8 + 2 * c + i) / G - row0 / G);
        if (!seen[j][h][i]) sc[j][h][i] = -INFINITY;
      }
      // The maximum follows once a logit is 2^3 times above it: p up to 8 costs
      // fp32 nothing, and most slices pass.
      higher = higher || fmaxf(sc[j][0][i], sc[j][1][i]) > S.m[j][i] + 3.f;
    }
  }
  if (__any_sync(0xffffffffu, higher)) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float mn = column_max(fmaxf(fmaxf(sc[j][0][i], sc[j][1][i]), S.m[j][i]));
        const float alpha = ex2(S.m[j][i] - mn);
        S.m[j][i] = mn;
        S.l[j][i] *= alpha;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          S.z[j][g][i] *= alpha;
#pragma unroll
          for (int t = 0; t < 4; ++t) S.o[j][g][t][i] *= alpha, S.o[j][g][t][2 + i] *= alpha;
        }
      }
    }
  }
  float ps[NT][NG][2][2];  // [group][key][row]: p s
  bool over = false;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float p[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        p[h] = ex2(sc[j][h][i] - S.m[j][i]);
        S.l[j][i] += p[h];
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ps[j][g][h][i] = seen[j][h][i] ? p[h] * vs[g][h] : 0.f;  // a hidden key's scale may be NaN
          S.z[j][g][i] = fmaf(p[h], seen[j][h][i] ? vz[g][h] : 0.f, S.z[j][g][i]);
        }
        over = over || fmaxf(ps[j][g][0][i], ps[j][g][1][i]) * S.up[j][g][i] > 0x1p15f;
      }
    }
  }
  if (__any_sync(0xffffffffu, over)) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float mx = column_max(fmaxf(ps[j][g][0][i], ps[j][g][1][i]));
          if (mx * S.up[j][g][i] > 0x1p15f) {  // (the same in all lanes of the column)
            const float up = pow2(min(9 - exponent(mx), 120)), f = up / S.up[j][g][i];
            S.up[j][g][i] = up;
#pragma unroll
            for (int t = 0; t < 4; ++t) S.o[j][g][t][i] *= f, S.o[j][g][t][2 + i] *= f;
          }
        }
      }
    }
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    uint32_t bp[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        bp[j][h] = transpose8(pack_f16x2(ps[j][g][h][0] * S.up[j][g][0], ps[j][g][h][1] * S.up[j][g][1]));
    }
    // Word r of the group of keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9 (as k indices).
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = *reinterpret_cast<const uint32_t*>(st + C::OFF_VC + (k0 + c + 4 * (i & 1) + 8 * (i >> 1)) * (D / 2) +
                                                g * 32 + r * 4);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      // Byte t of both keys of a pair: dimensions 8 r + 2 t (rows 0 .. 7) and 8 r + 2 t + 1 (rows 8 .. 15).
      const uint32_t x = __byte_perm(w[0], w[1], t | t << 4 | (4 + t) << 8 | (4 + t) << 12);
      const uint32_t y = __byte_perm(w[2], w[3], t | t << 4 | (4 + t) << 8 | (4 + t) << 12);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        mma_f16(S.o[j][g][t], x & 0x000F000Fu, x & 0x00F000F0u, y & 0x000F000Fu, y & 0x00F000F0u, bp[j][0], bp[j][1]);
    }
  }
}

}  // namespace

template <int D, int NT>
__global__ void __launch_bounds__(Q4Cfg<D, NT>::THREADS, Q4Cfg<D, NT>::CTAS) fa_decode_q4_kernel(const Q4DecodeArgs a) {
  using C = Q4Cfg<D, NT>;
  constexpr int NG = C::NG;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::STAGES;
  uint32_t* held_bits = reinterpret_cast<uint32_t*>(smem + C::OFF_SCAN);  // per stage: slices whose block is in the pool
  volatile int* abort_flag = reinterpret_cast<volatile int*>(held_bits + C::STAGES);
  int* warp_sum = reinterpret_cast<int*>(held_bits + C::STAGES + 1);
  int* found = warp_sum + C::CWARPS + 1;  // sequence of the CTA's first tile, tiles of those before it
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    griddep_launch_dependents();
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], C::CWARPS);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  // The tiles of all sequences, and the sequence that this CTA's run starts in:
  // each thread adds up a stretch of sequences, then their sums are scanned.
  const int items = a.Hk * a.row_blocks;  // of a sequence
  const int stretch = (a.B + C::THREADS - 1) / C::THREADS;
  const int b0 = min(static_cast<int>(threadIdx.x) * stretch, a.B), b1 = min(b0 + stretch, a.B);
  int own = 0;
  for (int b = b0; b < b1; ++b) own += q4_tiles(q4_len(a, b));
  int upto = own;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += x;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  int total = 0, before = upto - own;
#pragma unroll
  for (int w = 0; w <= C::CWARPS; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  total *= items;
  const int cta = blockIdx.x, ctas = min(static_cast<int>(gridDim.x), total);  // one tile each at least
  const int start = cta < ctas ? q4_share(cta, total, ctas) : 0, end = cta < ctas ? q4_share(cta + 1, total, ctas) : 0;
  if (start < end && start / items >= before && start / items < before + own) {
    int b = b0, x = before;
    for (int n; x + (n = q4_tiles(q4_len(a, b))) <= start / items; ++b) x += n;
    found[0] = b, found[1] = x;
  }
  __syncthreads();
  Q4Walk w;
  w.left = end - start;
  if (w.left > 0) {
    w.b = found[0];
    const int rem = start - found[1] * items;
    const int n = q4_tiles(q4_len(a, w.b));
    w.item = rem / n;
    w.tile = rem - w.item * n;
    w.enter(a);
  }

  if (warp == C::CWARPS) {
    // ----------------------------------------------------------- copy warp
    if (lane == 0) {
      // For the kernel that joins: whether this CTA is the second one of a cut item.
      int4 cut = make_int4(-1, 0, 0, 0);
      if (w.left > 0 && w.tile > 0) {
        const int first = start - w.tile, prev = q4_share(cta - 1, total, ctas);
        if (prev <= first)
          cut = make_int4(w.b, w.item, prev == first ? 0 : 1,
                          static_cast<int>((static_cast<long long>(first + w.n) * ctas - 1) / total));
      }
      a.cuts[cta] = cut;
    }
    if (w.left <= 0 || g_test_drop_loads) return;
    // Lane (piece, array): one copy of `piece` keys of the codes or scales of K or V.
    const int p = lane >> 2, arr = lane & 3;
    const int row_bytes = (arr & 1) ? NG * 4 : D / 2;
    const uint8_t* base = arr == 0 ? a.k_codes : (arr == 1 ? a.k_scales : (arr == 2 ? a.v_codes : a.v_scales));
    const int dst0 = (arr == 0 ? 0 : (arr == 1 ? C::OFF_KS : (arr == 2 ? C::OFF_VC : C::OFF_VS))) +
                     p * a.piece * row_bytes;
    int issued = 0;
    bool ok = true;
    do {
      const int kvh = w.item / a.row_blocks;
      for (int t = 0; t < w.here && ok; ++t, ++issued) {
        const int s = issued % C::STAGES;
        const int key = (w.tile + t) * C::TK + p * a.piece;
        const bool mine = p * a.piece < C::TK && key < w.L;
        int phys = -1, block = 0;
        if (mine) {
          block = key / a.block_size;
          phys = a.block_table[static_cast<long long>(w.b) * a.max_blocks + block];
        }
        const bool held = mine && phys >= 0 && phys < a.num_blocks;
        const uint32_t lanes = __ballot_sync(0xffffffffu, held && arr == 0);
        if (issued >= C::STAGES &&
            !__all_sync(0xffffffffu, mbar_wait(&empty[s], (issued / C::STAGES - 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          uint32_t bits = 0u;  // of 16-key slices
          for (int i = 0; i < C::TK / 16; ++i) bits |= ((lanes >> (i * 16 / a.piece * 4)) & 1u) << i;
          held_bits[s] = bits;
          mbar_arrive_expect_tx(&full[s], __popc(lanes) * a.piece * 2 * (D / 2 + NG * 4));
        }
        __syncwarp();
        if (held) {
          const long long row = (static_cast<long long>(phys) * a.Hk + kvh) * a.block_size + (key - block * a.block_size);
          bulk_load(smem + s * C::STAGE_BYTES + dst0, base + row * row_bytes, a.piece * row_bytes, &full[s]);
        }
      }
    } while (ok && w.next(a));
    // Do not leave with copies in flight (matters only after an abort, when
    // the consumers stopped waiting; every issued copy lands).
    if (lane == 0)
      for (int t = max(0, issued - C::STAGES); t < issued; ++t)
        mbar_wait_drain(&full[t % C::STAGES], (t / C::STAGES) & 1);
    return;
  }

  // -------------------------------------------------------- consumer warps
  const int r = lane >> 2, c = lane & 3;
  const int G = a.H / a.Hk;
  float* red_o = reinterpret_cast<float*>(smem + C::OFF_RED);  // [warp][ROWS][RED_STRIDE]
  float* red_ml = reinterpret_cast<float*>(smem + C::OFF_ML);  // [warp][ROWS][2]
  int taken = 0;
  bool ok = true, first_item = true;
  if (w.left > 0) do {
    const int kvh = w.item / a.row_blocks, row0 = (w.item - kvh * a.row_blocks) * C::ROWS;
    const int rows = min(a.n_new * G - row0, C::ROWS);
    Q4Rows<D, NT> R;
    q4_load_rows<D, NT>(a, w.b, kvh, row0, rows, lane, R);
    Q4State<D, NT> S;
    S.clear();
    const int open = w.L - a.n_new + 1 + row0 / G;  // keys from here on are hidden from some row
    for (int t = 0; t < w.here; ++t, ++taken) {
      const int s = taken % C::STAGES;
      ok = __all_sync(0xffffffffu, mbar_wait(&full[s], (taken / C::STAGES) & 1, abort_flag));
      if (!ok) break;
      const uint8_t* st = smem + s * C::STAGE_BYTES;
      const int first = (w.tile + t) * C::TK, left = w.L - first;
      const uint32_t held = held_bits[s];
#pragma unroll 1
      for (int k0 = warp * 16; k0 < min(C::TK, left); k0 += C::CWARPS * 16) {
        const bool on = (held >> (k0 / 16)) & 1u;
        if (on && k0 + 16 <= min(open - first, left)) q4_slice<D, NT, false>(st, k0, lane, true, left, 0, 0, 1, R, S);
        else q4_slice<D, NT, true>(st, k0, lane, on, left, open - first, row0, G, R, S);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          S.l[j][i] += __shfl_xor_sync(0xffffffffu, S.l[j][i], off);
#pragma unroll
          for (int g = 0; g < NG; ++g) S.z[j][g][i] += __shfl_xor_sync(0xffffffffu, S.z[j][g][i], off);
        }
      }
    }
    // Join the warps, once all of them have read what they joined last.
    named_bar_sync(1, C::CWARPS * 32);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = warp * C::ROWS + j * 8 + 2 * c + i;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float f = 1.f / S.up[j][g][i];
          const float f0 = f * 0x1p24f, f1 = f * 0x1p20f;
#pragma unroll
          for (int t = 0; t < 4; ++t)
            *reinterpret_cast<float2*>(&red_o[row * C::RED_STRIDE + g * 64 + r * 8 + t * 2]) =
                make_float2(fmaf(S.o[j][g][t][i], f0, S.z[j][g][i]), fmaf(S.o[j][g][t][2 + i], f1, S.z[j][g][i]));
        }
        if (r == 0) *reinterpret_cast<float2*>(&red_ml[row * 2]) = make_float2(S.m[j][i], S.l[j][i]);
      }
    }
    named_bar_sync(1, C::CWARPS * 32);
    const bool whole = w.here == w.n;
    const int slot = 2 * cta + (first_item ? 0 : 1);
    for (int x = threadIdx.x / (D / 4); x < rows; x += C::CWARPS * 32 / (D / 4)) {
      const int col = threadIdx.x % (D / 4) * 4;
      float M = kNoLogit;
#pragma unroll
      for (int v = 0; v < C::CWARPS; ++v) M = fmaxf(M, red_ml[(v * C::ROWS + x) * 2]);
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int v = 0; v < C::CWARPS; ++v) {
        const float2 ml = *reinterpret_cast<const float2*>(&red_ml[(v * C::ROWS + x) * 2]);
        const float f = ex2(ml.x - M);
        const float4 y = *reinterpret_cast<const float4*>(&red_o[(v * C::ROWS + x) * C::RED_STRIDE + col]);
        sum = fmaf(ml.y, f, sum);
        acc.x = fmaf(y.x, f, acc.x), acc.y = fmaf(y.y, f, acc.y);
        acc.z = fmaf(y.z, f, acc.z), acc.w = fmaf(y.w, f, acc.w);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const float lse2 = sum == 0.f ? -INFINITY : M + log2f(sum);
      if (whole) {
        const long long row = q4_row(a, w.b, kvh, row0 + x);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + row * D + col) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (col == 0) a.lse[row] = lse2 * kLn2;
      } else {
        const size_t at = static_cast<size_t>(slot) * C::ROWS + x;
        *reinterpret_cast<float4*>(a.part_o + at * D + col) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (col == 0) a.part_lse[at] = lse2;
      }
    }
    first_item = false;
  } while (ok && w.next(a));
  // Sequences without keys have no tiles: every CTA writes its share of their rows.
  for (int b = cta; b < a.B; b += gridDim.x) {
    if (q4_len(a, b) > 0) continue;
    const long long row = static_cast<long long>(b) * a.n_new * a.H;
    const int n = a.n_new * a.H;
    for (int x = threadIdx.x; x < n * (D / 8); x += C::CWARPS * 32)
      reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + row * D)[x] = make_uint4(0u, 0u, 0u, 0u);
    for (int x = threadIdx.x; x < n; x += C::CWARPS * 32) a.lse[row + x] = -INFINITY;
  }
}

// Joins the parts of cut items: CTA (x, y) takes row y of the item whose second
// part is grid CTA x's first one. O = sum of 2^(lse_i - M) O_i over the sum of
// the weights, in the order of the keys: the warps every fourth part, then
// their sums.
template <int D>
__global__ void __launch_bounds__(128) fa_decode_q4_join_kernel(const Q4DecodeArgs a) {
  constexpr int CPL = D / 32;  // columns per lane
  __shared__ float red[4][D + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  const int4 cut = a.cuts[blockIdx.x];
  if (cut.x < 0) return;
  const int kvh = cut.y / a.row_blocks, row = (cut.y - kvh * a.row_blocks) * a.rows_per + blockIdx.y;
  if (row >= a.n_new * (a.H / a.Hk)) return;
  const int c0 = blockIdx.x - 1, n = cut.w - c0 + 1;
  auto part = [&](int i) {
    return static_cast<size_t>(2 * (c0 + i) + (i == 0 ? cut.z : 0)) * a.rows_per + blockIdx.y;
  };
  float M = -INFINITY;
  for (int i = lane; i < n; i += 32) M = max_nan(M, a.part_lse[part(i)]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, off));
  float sum = 0.f, acc[CPL];
#pragma unroll
  for (int k = 0; k < CPL; ++k) acc[k] = 0.f;
  if (M != -INFINITY) {
#pragma unroll 4
    for (int i = warp; i < n; i += 4) {
      const float f = ex2(a.part_lse[part(i)] - M);
      const float* src = a.part_o + part(i) * D + lane * CPL;
      sum += f;
#pragma unroll
      for (int k = 0; k < CPL; ++k) acc[k] = fmaf(f, src[k], acc[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < CPL; ++k) red[warp][lane * CPL + k] = acc[k];
  if (lane == 0) red[warp][D] = sum;
  __syncthreads();
  if (warp > 0) return;
  sum = red[0][D];
#pragma unroll
  for (int v = 1; v < 4; ++v) {
    sum += red[v][D];
#pragma unroll
    for (int k = 0; k < CPL; ++k) acc[k] += red[v][lane * CPL + k];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const long long at = q4_row(a, cut.x, kvh, row);
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + at * D + lane * CPL);
#pragma unroll
  for (int k = 0; k < CPL; k += 2) out[k / 2] = pack_bf16x2(acc[k] * inv, acc[k + 1] * inv);
  if (lane == 0) a.lse[at] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
}

template <int D, int NT>
static cudaError_t launch_q4_t(const Q4DecodeArgs& a, cudaStream_t stream, const LaunchMarks* marks) {
  using C = Q4Cfg<D, NT>;
  static_assert(C::CTAS * 152 <= kQ4MaxCtas, "the workspace holds the parts of every CTA");
  auto kern = fa_decode_q4_kernel<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const int grid = std::min(a.most_tiles, C::CTAS * 152);
  mark(marks, true, 0, stream);
  kern<<<grid, C::THREADS, C::SMEM_BYTES, stream>>>(a);
  e = cudaGetLastError();
  mark(marks, false, 0, stream);
  if (e != cudaSuccess) return e;
  mark(marks, true, 1, stream);
  e = launch_maybe_pdl(fa_decode_q4_join_kernel<D>, dim3(grid, C::ROWS), dim3(128), 0, stream, marks == nullptr, a);
  mark(marks, false, 1, stream);
  return e;
}

cudaError_t launch_decode_q4(const Q4DecodeArgs& a, cudaStream_t stream, const LaunchMarks* m) {
  if (a.rows_per == 8) return a.D == 64 ? launch_q4_t<64, 1>(a, stream, m) : launch_q4_t<128, 1>(a, stream, m);
  return a.D == 64 ? launch_q4_t<64, 2>(a, stream, m) : launch_q4_t<128, 2>(a, stream, m);
}

cudaError_t set_decode_q4_test_hooks(unsigned long long wait_limit_ns, int drop_loads, cudaStream_t stream) {
  return set_test_hooks_here(wait_limit_ns, drop_loads, stream);
}

int take_decode_q4_status() { return take_status_here(); }

}  // namespace fa
