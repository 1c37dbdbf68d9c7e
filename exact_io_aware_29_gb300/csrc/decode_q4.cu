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
//   f16 is exact (below 2^-27 of the row's largest: rounded at 2^-35 of it).
//   P V: p s is scaled by a power of two of the row and group, such that the
//   largest so far, each at its present weight, lies in [2^9, 2^15): rounded to
//   f16, 2^-11 of a term (an eighth of what the rounding of O to bf16 costs), at
//   terms down to 2^-23 of the largest (and 2^-134). It is a choice for speed:
//   as the sum of two f16 numbers, 64 sequences of 1024 to 8192 tokens, 32/8
//   heads, d 128, take 65.1 us instead of 59.5, with four drafts each 113 instead
//   of 96, and O is off by 1.67e-3 instead of 1.74e-3 (its rounding to bf16 alone:
//   1.665e-3).
// The logic pipe, not the tensor cores, stands nearest to HBM: about 125
// instructions on it for 16 keys, of 205 that HBM leaves time for (d 128).
//
// A persistent grid shares the 128-key tiles of all sequences and key heads out
// evenly, in order, whatever their lengths: a CTA takes a run of tiles, whole
// items (row block, key head) and the ends of two. Each of its four warps works
// on 32 keys of every tile (two independent halves hide each other's latencies),
// which it copies ahead itself into a ring of its own (cp.async, 16 bytes a
// lane; what is not there is filled with zeros), so that warps meet only where
// an item ends.
// Softmax statistics and sums are fp32. A cut item's parts are joined in the
// order of the keys by a second kernel.
// A step of few, short sequences goes another way, its time being a sum of
// latencies: a cluster of up to eight CTAs shares an item's tiles and joins its
// parts through their shared memory.
// 64 sequences of 1024 to 8192 tokens, 32/8 heads, d 128: 59.5 us, 5.6 TB/s (the
// copies alone 59); one of 131072: 32.7 us, 4.6 TB/s. About 8 of them are spent
// before the first tile and after the last.
#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace fa {

template <int D, int NT>
struct Q4Cfg {
  static constexpr int NG = D / 64;                // groups of a row
  static constexpr int ROWS = 8 * NT;              // rows of an item
  static constexpr int KEYS = 32;                  // a warp's keys of a tile
  static constexpr int HALVES = KEYS / 16;
  static constexpr int WARPS = kQ4Tile / KEYS;
  static constexpr int THREADS = WARPS * 32;
  // Per SM; registers at most 168, 128 at d 64 with NT = 1, 255 at d 128 with NT = 2.
  static constexpr int CTAS = q4_ctas(D, ROWS);
  // A stage of a warp's ring: codes of K and V, scales of K and V.
  static constexpr int CODE_BYTES = KEYS * D / 2, SCALE_BYTES = KEYS * NG * 4;
  static constexpr int OFF_VC = CODE_BYTES, OFF_KS = 2 * CODE_BYTES, OFF_VS = OFF_KS + SCALE_BYTES;
  static constexpr int STAGE_BYTES = 2 * (CODE_BYTES + SCALE_BYTES);
  static constexpr int STAGES = D == 64 ? 4 : 2 + NT;
  static constexpr int RED_STRIDE = D + 4;         // floats of a row in the join of the warps
  static constexpr int OFF_RED = WARPS * STAGES * STAGE_BYTES;
  static constexpr int OFF_ML = OFF_RED + WARPS * ROWS * RED_STRIDE * 4;
  static constexpr int OFF_SCAN = OFF_ML + WARPS * ROWS * 2 * 4;
  static constexpr int SMEM_BYTES = OFF_SCAN + WARPS * 8 + 8;
  static_assert((SMEM_BYTES + 1024) * CTAS <= 228 * 1024, "fits in an SM");
};

namespace {

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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
__device__ __forceinline__ float pow2_or_0(int e) { return e < -126 ? 0.f : pow2(e); }
__device__ __forceinline__ float inverse_pow2(float x) { return __uint_as_float(0x7F000000u - __float_as_uint(x)); }
__device__ __forceinline__ int exponent(float x) { return static_cast<int>((__float_as_uint(x) >> 23) & 255u) - 127; }
// Two fp32 numbers for the instructions that work on pairs of them.
__device__ __forceinline__ uint64_t pair(const float (&x)[2]) { return f2_pack(x[0], x[1]); }
__device__ __forceinline__ uint64_t both(float x) { return f2_pack(x, x); }
// max(a, b), NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 16 bytes global -> shared, asynchronously; zeros if !on.
__device__ __forceinline__ void cp_async16(uint32_t dst, const uint8_t* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
// The larger of each pair of f16 (NaN only where both are).
__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

constexpr float kNoLogit = -3.402823466e38f;  // the maximum before the first key; no finite logit is below it

__device__ __forceinline__ int q4_len(const Q4DecodeArgs& a, int b) {
  return min(max(a.seq_lens[b], 0), a.max_seq_len);
}
__device__ __forceinline__ int q4_tiles(int L) {  // (L may be 2^31 - 1)
  return static_cast<int>((static_cast<unsigned>(L) + kQ4Tile - 1) / kQ4Tile);
}
// How `total` units of work are shared out over `ctas` CTAs: runs of `per` or
// per + 1, the longer ones first. A unit is a tile; an item may count as some
// units more (its head), in front of its tiles.
struct Q4Shares {
  int per, longer;
  __device__ __forceinline__ Q4Shares(int total, int ctas) : per(total / ctas), longer(total % ctas) {}
  __device__ __forceinline__ int start(int c) const { return c * per + min(c, longer); }
  __device__ __forceinline__ int of(int unit) const {  // the CTA that has it
    const int x = longer * (per + 1);
    return unit < x ? unit / (per + 1) : longer + (unit - x) / per;
  }
};

// A CTA's way along its run, item by item.
struct Q4Walk {
  int b, item, tile, left;  // sequence, (key head, row block) of it, first tile in it, units of the run from there on
  int L, n;                 // length, tiles and
  int here;                 // tiles of the run in this item
  __device__ __forceinline__ void enter(const Q4DecodeArgs& a) {
    L = q4_len(a, b);
    n = q4_tiles(L);
    here = min(n - tile, left);
  }
  __device__ __forceinline__ bool next(const Q4DecodeArgs& a, int head) {  // false at the end of the run
    left -= here + head;
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

// The first of the two columns (rows of the queries) whose logits lane (., c)
// works on. With up to four rows the columns from 4 on are empty, and the lanes
// that have them take the first ones' logits of the stage's other 16 keys.
template <bool FEW>
__device__ __forceinline__ int column(int c) {
  return FEW ? 2 * (c & 1) : 2 * c;
}

// What a lane holds of the queries: lane (r, c) = (lane / 4, lane % 4).
template <int D, int NT>
struct Q4Rows {
  static constexpr int NG = D / 64;
  uint32_t q[NT][NG][4][2];  // B fragments of row 8 j + r, k-step t of group g
  float qs[NT][2];           // of rows 8 j + column + {0, 1}: what a product of codes is multiplied by
  float sum[NT][NG][2];      // scale log2e times the sum of the row's group
};

// The queries as they lie in memory: elements 64 g + 16 c + {0 .. 15} of row 8 j + r.
template <int D, int NT>
struct Q4Raw {
  uint4 x[NT][D / 64][2];
  __device__ __forceinline__ void read(const Q4DecodeArgs& a, int b, int kvh, int row0, int rows, int lane) {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const bool on = j * 8 + r < rows;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                        (on ? q4_row(a, b, kvh, row0 + j * 8 + r) : 0LL) * D);
#pragma unroll
      for (int g = 0; g < D / 64; ++g) {
#pragma unroll
        for (int h = 0; h < 2; ++h) x[j][g][h] = on ? src[g * 8 + c * 2 + h] : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
};

template <int D, int NT, bool FEW>
__device__ __forceinline__ void q4_rows(const Q4DecodeArgs& a, const Q4Raw<D, NT>& raw, int lane, Q4Rows<D, NT>& R) {
  constexpr int NG = D / 64;
  const int c = lane & 3;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    uint32_t w[NG][8];
    float mx = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 x = raw.x[j][g][h];
        w[g][4 * h] = x.x, w[g][4 * h + 1] = x.y, w[g][4 * h + 2] = x.z, w[g][4 * h + 3] = x.w;
      }
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
    // To the lanes of the C fragments' columns: row 8 j + x comes from lane (x, .).
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int x = column<FEW>(c) + i;
      R.qs[j][i] = __shfl_sync(0xffffffffu, down, x * 4);
#pragma unroll
      for (int g = 0; g < NG; ++g) R.sum[j][g][i] = __shfl_sync(0xffffffffu, s[g], x * 4);
    }
  }
}

// Running softmax of a lane's columns (rows 8 j + column + {0, 1}): maximum and
// powers are the same in all lanes of a column, the sums are the lane's own.
template <int D, int NT>
struct Q4State {
  static constexpr int NG = D / 64;
  float o[NT][NG][4][4];  // C fragments: dimensions 64 g + 8 r + 2 t (c0 c1) and, 16-fold, the next one (c2 c3)
  float m[NT][2], l[NT][2], z[NT][NG][2];
  float up[NT][NG][2];    // the power of two, 2^-119 to 2^120, that p s is multiplied by
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
template <bool FEW>
__device__ __forceinline__ float column_max(float x) {
#pragma unroll
  for (int off = FEW ? 2 : 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

// The keys of a stage. MASKED: some of them may be hidden from some rows (row x
// sees the keys below open + (row0 + x) / G - row0 / G) or past the sequence
// (`left` of them are in it).
template <int D, int NT, bool FEW, bool MASKED>
__device__ __forceinline__ void q4_step(const uint8_t* st, int lane, int left, int open, int row0, int G,
                                        const Q4Rows<D, NT>& R, Q4State<D, NT>& S) {
  using C = Q4Cfg<D, NT>;
  constexpr int NG = D / 64, KH = FEW ? 2 : 2 * C::HALVES;  // logits of keys kl + 8 h of a lane, h < KH
  const int r = lane >> 2, c = lane & 3;
  // Row i of the A operand of Q K^T, and k index i of P V, is key (i >> 1) + 4 (i & 1)
  // of its eight: the lanes of a load then meet two banks' worth of rows, not one.
  const int ka = (r >> 1) + 4 * (r & 1), kl = FEW ? ka + 8 * (c & 2) : ka;
  float sc[NT][KH][2];  // [key kl + 8 h][row i]
  uint32_t vsz[NG][KH];
  float acc[C::HALVES][NT][NG][4];
  {
    uint2 x[C::HALVES][NG], y[C::HALVES][NG];
#pragma unroll
    for (int s = 0; s < C::HALVES; ++s) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        x[s][g] = *reinterpret_cast<const uint2*>(st + (ka + 16 * s) * (D / 2) + g * 32 + c * 8);
        y[s][g] = *reinterpret_cast<const uint2*>(st + (ka + 16 * s + 8) * (D / 2) + g * 32 + c * 8);
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[s][j][g][0] = acc[s][j][g][1] = acc[s][j][g][2] = acc[s][j][g][3] = 0.f;
      }
    }
    // Products that do not wait for one another in a row.
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int s = 0; s < C::HALVES; ++s) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const uint32_t wx = (t < 2 ? x[s][g].x : x[s][g].y) >> (8 * (t & 1));
          const uint32_t wy = (t < 2 ? y[s][g].x : y[s][g].y) >> (8 * (t & 1));
#pragma unroll
          for (int j = 0; j < NT; ++j)
            mma_f16(acc[s][j][g], wx & 0x000F000Fu, wy & 0x000F000Fu, wx & 0x00F000F0u, wy & 0x00F000F0u,
                    R.q[j][g][t][0], R.q[j][g][t][1]);
        }
      }
    }
  }
  if constexpr (FEW) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float other = __shfl_xor_sync(0xffffffffu, acc[1][0][g][i], 2);
        acc[0][0][g][i] = (c & 2) ? other : acc[0][0][g][i];
      }
    }
  }
#pragma unroll
  for (int h = 0; h < KH; ++h) {
    const int s = h / 2, e = h % 2;
    const uint32_t* pk = reinterpret_cast<const uint32_t*>(st + C::OFF_KS) + (kl + 8 * h) * NG;
    const uint32_t* pv = reinterpret_cast<const uint32_t*>(st + C::OFF_VS) + (kl + 8 * h) * NG;
    uint32_t ksz[NG];
    if constexpr (NG == 2) {
      const uint2 k = *reinterpret_cast<const uint2*>(pk), v = *reinterpret_cast<const uint2*>(pv);
      ksz[0] = k.x, ksz[1] = k.y, vsz[0][h] = v.x, vsz[1][h] = v.y;
    } else {
      ksz[0] = *pk, vsz[0][h] = *pv;
    }
    if (MASKED && kl + 8 * h >= left) {
#pragma unroll
      for (int g = 0; g < NG; ++g) ksz[g] = vsz[g][h] = 0u;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      uint64_t x = f2_mul(f2_pack(acc[s][j][0][2 * e], acc[s][j][0][2 * e + 1]), both(lo_f(ksz[0])));
      uint64_t y = f2_mul(both(hi_f(ksz[0])), pair(R.sum[j][0]));
#pragma unroll
      for (int g = 1; g < NG; ++g) {
        x = f2_fma(f2_pack(acc[s][j][g][2 * e], acc[s][j][g][2 * e + 1]), both(lo_f(ksz[g])), x);
        y = f2_fma(both(hi_f(ksz[g])), pair(R.sum[j][g]), y);
      }
      f2_unpack(f2_fma(x, pair(R.qs[j]), y), sc[j][h][0], sc[j][h][1]);
    }
  }
  bool seen[NT][KH][2];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int h = 0; h < KH; ++h) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        seen[j][h][i] =
            !MASKED || (kl + 8 * h < left && kl + 8 * h < open + (row0 + j * 8 + column<FEW>(c) + i) / G - row0 / G);
        if (!seen[j][h][i]) sc[j][h][i] = -INFINITY;
      }
    }
  }
  // p and, in f16, p s times its power of two. The maximum (rounded up to an
  // integer) follows a logit that is more than 2^3 times above it (p up to 8 costs
  // fp32 nothing), and the power rises by what the weights of the keys so far fall
  // then, exactly: it looks back at no term that has lost its weight, and the sums
  // in it stay as they are. The power follows a p s of 2^15 or more down: most steps
  // change neither.
  float p[NT][KH][2];
  uint32_t ph[NT][NG][KH];
  auto weigh = [&]() {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int h = 0; h < KH; ++h) {
        float x0, x1;
        f2_unpack(f2_sub(pair(sc[j][h]), pair(S.m[j])), x0, x1);
        p[j][h][0] = ex2(x0), p[j][h][1] = ex2(x1);
#pragma unroll
        for (int g = 0; g < NG; ++g) {  // (a hidden key's scale may be NaN)
          f2_unpack(f2_mul(pair(p[j][h]), both(lo_f(vsz[g][h]))), x0, x1);
          f2_unpack(f2_mul(f2_pack(seen[j][h][0] ? x0 : 0.f, seen[j][h][1] ? x1 : 0.f), pair(S.up[j][g])), x0, x1);
          ph[j][g][h] = pack_f16x2(x0, x1);
        }
      }
    }
  };
  weigh();
  float most = 0.f;
  uint32_t most_h = 0u;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int h = 0; h < KH; ++h) {
      most = max3f(most, p[j][h][0], p[j][h][1]);
#pragma unroll
      for (int g = 0; g < NG; ++g) most_h = max_f16x2(most_h, ph[j][g][h]);
    }
  }
  if (__any_sync(0xffffffffu, most > 8.f || ((most_h + 0x08000800u) & 0x80008000u) != 0u)) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mn = S.m[j][i];
#pragma unroll
        for (int h = 0; h < KH; ++h) mn = fmaxf(mn, sc[j][h][i]);
        mn = ceilf(column_max<FEW>(mn));
        // The weights of the keys so far fall by 2^fall (below 2^-126: to nothing).
        const int fall = -static_cast<int>(fmaxf(S.m[j][i] - mn, -252.f));
        const float alpha = pow2_or_0(-fall);
        S.m[j][i] = mn;
        S.l[j][i] *= alpha;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          S.z[j][g][i] *= alpha;
          float mx = 0.f;
#pragma unroll
          for (int h = 0; h < KH; ++h)
            if (seen[j][h][i]) mx = fmaxf(mx, ex2(sc[j][h][i] - mn) * lo_f(vsz[g][h]));
          mx = column_max<FEW>(mx);
          const int was = exponent(S.up[j][g][i]);
          int now = min(was + fall, 120);
          if (mx * pow2(now) >= 0x1p15f) now = min(9 - exponent(mx), 120);  // (the same in all lanes of the column)
          S.up[j][g][i] = pow2(now);
          const float f = pow2_or_0(now - was - fall);
#pragma unroll
          for (int t = 0; t < 4; ++t) S.o[j][g][t][i] *= f, S.o[j][g][t][2 + i] *= f;
        }
      }
    }
    weigh();
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int h = 0; h < KH; ++h) {
      f2_unpack(f2_add(pair(S.l[j]), pair(p[j][h])), S.l[j][0], S.l[j][1]);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float z = hi_f(vsz[g][h]);
        f2_unpack(f2_fma(pair(p[j][h]), f2_pack(seen[j][h][0] ? z : 0.f, seen[j][h][1] ? z : 0.f), pair(S.z[j][g])),
                  S.z[j][g][0], S.z[j][g][1]);
      }
    }
  }
#pragma unroll
  for (int s = 0; s < C::HALVES; ++s) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      uint32_t bp[NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // (FEW: each half's own P stands in the first four columns, the other's in the empty ones.)
          const uint32_t x = ph[j][g][FEW ? e : 2 * s + e];
          bp[j][e] = transpose8(FEW && s == 1 ? __shfl_xor_sync(0xffffffffu, x, 2) : x);
        }
      }
      // Word r of the group of keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9 (as k indices).
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = *reinterpret_cast<const uint32_t*>(
            st + C::OFF_VC + (16 * s + c + 4 * (i & 1) + 8 * (i >> 1)) * (D / 2) + g * 32 + r * 4);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        // Byte t of both keys of a pair: dimensions 8 r + 2 t (rows 0 .. 7) and 8 r + 2 t + 1 (rows 8 .. 15).
        const uint32_t x = __byte_perm(w[0], w[1], t | t << 4 | (4 + t) << 8 | (4 + t) << 12);
        const uint32_t y = __byte_perm(w[2], w[3], t | t << 4 | (4 + t) << 8 | (4 + t) << 12);
#pragma unroll
        for (int j = 0; j < NT; ++j)
          mma_f16(S.o[j][g][t], x & 0x000F000Fu, x & 0x00F000F0u, y & 0x000F000Fu, y & 0x00F000F0u, bp[j][0],
                  bp[j][1]);
      }
    }
  }
}

// A warp's copies: its keys of the CTA's tiles, in order, across items. Lane i
// holds where the 16 keys of the i-th half from tile `base` on lie; in a copy
// the warp's lower half takes the first 16 keys of the stage, the upper one the
// other 16.
template <int D, int NT>
struct Q4Copies {
  using C = Q4Cfg<D, NT>;
  Q4Walk w;
  int head;
  int at, base, upto;  // the next tile of the item to copy; the tiles whose places the lanes hold
  long long row;       // this lane's: (block, key head, slot) of the first key; -1: nowhere
  bool more;
  const uint8_t *kc, *vc, *sc;  // the cache, at this lane's 16 bytes
  uint32_t dst;                 // and the ring
  __device__ __forceinline__ void begin(const Q4DecodeArgs& a, const Q4Walk& first, int h, uint32_t ring, int warp,
                                        int lane) {
    w = first;
    head = h;
    more = true;
    at = w.tile;
    const int i = lane & 15, half = lane >> 4;
    kc = a.k_codes + i * 16;
    vc = a.v_codes + i * 16;
    constexpr int SL = 16 * C::NG * 4 / 16;  // lanes of 16 keys' scales of K, then of V
    sc = (i < SL ? a.k_scales : a.v_scales) + i % SL * 16;
    dst = ring + half * (C::CODE_BYTES / 2) + i * 16;
    look(a, warp, lane);
  }
  __device__ __forceinline__ void look(const Q4DecodeArgs& a, int warp, int lane) {
    base = at;
    upto = min(at + 32 / C::HALVES, w.tile + w.here);
    const int tile = at + lane / C::HALVES;
    const int key = tile < upto ? tile * kQ4Tile + warp * C::KEYS + lane % C::HALVES * 16 : w.L;
    row = -1;
    if (key < w.L) {
      const int block = key / a.block_size;
      const int phys = a.block_table[static_cast<long long>(w.b) * a.max_blocks + block];
      if (phys >= 0 && phys < a.num_blocks)
        row = (static_cast<long long>(phys) * a.Hk + w.item / a.row_blocks) * a.block_size + key - block * a.block_size;
    }
  }
  // The next tile's keys into stage s (an empty group past the end).
  __device__ __forceinline__ void copy(const Q4DecodeArgs& a, int s, int warp, int lane) {
    if (more && at == upto) {
      if (at == w.tile + w.here) {
        more = w.next(a, head);
        at = w.tile;
      }
      if (more) look(a, warp, lane);
    }
    if (more) {
      const long long from = __shfl_sync(0xffffffffu, row, (at - base) * C::HALVES + (lane >> 4));
      const bool on = from >= 0;
      const long long f = on ? from * (D / 2) : 0;
      const uint32_t d = dst + s * C::STAGE_BYTES;
      constexpr int N = C::CODE_BYTES / 2 / 256;
#pragma unroll
      for (int i = 0; i < N; ++i) cp_async16(d + i * 256, kc + f + i * 256, on);
#pragma unroll
      for (int i = 0; i < N; ++i) cp_async16(d + C::OFF_VC + i * 256, vc + f + i * 256, on);
      constexpr int SL = 16 * C::NG * 4 / 16;
      const int i = lane & 15, half = lane >> 4;
      // (The scales take an eighth of the codes' bytes.)
      if (i < 2 * SL)
        cp_async16(d - half * (C::CODE_BYTES / 2) - i * 16 + (i < SL ? C::OFF_KS : C::OFF_VS) + half * (SL * 16) +
                       i % SL * 16,
                   sc + (f >> 3), on);
      ++at;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
};

}  // namespace

// Where a CTA's run begins, and what it needs to say where its last item ends.
struct Q4Start {
  Q4Walk w;
  int head, run_end;
  Q4Shares shares;
};
template <int D, int NT>
__device__ __forceinline__ Q4Start q4_start(const Q4DecodeArgs& a, uint8_t* smem, int warp, int lane) {
  using C = Q4Cfg<D, NT>;
  long long* warp_sum = reinterpret_cast<long long*>(smem + C::OFF_SCAN);
  int* found = reinterpret_cast<int*>(warp_sum + C::WARPS);  // sequence of the first tile, units of those before it
  // The tiles of all sequences (and, in the upper half, how many have any), and
  // the sequence that this CTA's run starts in: each thread adds up a stretch of
  // sequences, then their sums are scanned.
  const int items = a.Hk * a.row_blocks;  // of a sequence
  const int stretch = (a.B + C::THREADS - 1) / C::THREADS;
  const int b0 = min(static_cast<int>(threadIdx.x) * stretch, a.B), b1 = min(b0 + stretch, a.B);
  long long own = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = q4_tiles(q4_len(a, b));
    own += n > 0 ? n + (1LL << 32) : 0;
  }
  long long upto = own;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += x;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  long long all = 0, before = upto - own;
#pragma unroll
  for (int v = 0; v < C::WARPS; ++v) {
    if (v < warp) before += warp_sum[v];
    all += warp_sum[v];
  }
  // An item costs about three tiles' time besides its tiles (its queries, the
  // first steps' maxima, the join of the warps), six with 9 to 16 rows: 64
  // sequences of up to 8192 tokens 59.5 us, 70 if it is left out, and 96 with four
  // drafts each, 104 if it counts as three. Where runs are short, what counts is
  // the longest of them: only tiles then.
  const int tiles = static_cast<int>(all) * items;
  const int cta = blockIdx.x, ctas = min(static_cast<int>(gridDim.x), tiles);  // one tile each at least
  const int head = tiles >= 8 * ctas ? q4_head(C::ROWS) : 0;
  const Q4Shares shares(tiles + head * static_cast<int>(all >> 32) * items, max(ctas, 1));
  auto units = [&](long long sum) { return (static_cast<int>(sum) + head * static_cast<int>(sum >> 32)) * items; };
  const int start = shares.start(cta);
  if (cta < ctas && start >= units(before) && start < units(before + own)) {
    int b = b0, x = units(before);
    for (;; ++b) {
      const int n = q4_tiles(q4_len(a, b)), u = n > 0 ? (n + head) * items : 0;
      if (x + u > start) break;
      x += u;
    }
    found[0] = b, found[1] = x;
  }
  __syncthreads();
  Q4Start at{Q4Walk{}, head, shares.start(cta + 1), shares};
  if (cta < ctas) {
    Q4Walk& w = at.w;
    w.b = found[0];
    const int rem = start - found[1], u = q4_tiles(q4_len(a, w.b)) + head;
    w.item = rem / u;
    const int into = rem - w.item * u;  // units of the item in front of the run
    w.tile = max(into - head, 0);
    w.left = at.run_end - start - max(head - into, 0);
    w.enter(a);
  }
  return at;
}
// The same for an item shared by a cluster: its tiles in equal runs.
template <int D, int NT>
__device__ __forceinline__ Q4Start q4_start_spread(const Q4DecodeArgs& a) {
  Q4Start at{Q4Walk{}, 0, 0, Q4Shares(0, 1)};
  const int items = a.Hk * a.row_blocks, id = blockIdx.x / a.spread, rank = blockIdx.x - id * a.spread;
  Q4Walk& w = at.w;
  w.b = id / items;
  w.item = id - w.b * items;
  const int n = q4_tiles(q4_len(a, w.b));
  w.tile = rank * n / a.spread;
  w.left = (rank + 1) * n / a.spread - w.tile;
  w.enter(a);
  return at;
}

template <int D, int NT, bool FEW, bool SPREAD>
__global__ void __launch_bounds__(Q4Cfg<D, NT>::THREADS, Q4Cfg<D, NT>::CTAS) fa_decode_q4_kernel(const Q4DecodeArgs a) {
  using C = Q4Cfg<D, NT>;
  constexpr int NG = C::NG;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!SPREAD && threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();  // launched programmatically: nothing of the stream's is read before
  const int items = a.Hk * a.row_blocks, cta = blockIdx.x, G = a.H / a.Hk;
  Q4Start at = SPREAD ? q4_start_spread<D, NT>(a) : q4_start<D, NT>(a, smem, warp, lane);
  Q4Walk& w = at.w;
  const int head = at.head;
  int kvh, row0, rows;
  auto item = [&]() {
    kvh = w.item / a.row_blocks;
    row0 = (w.item - kvh * a.row_blocks) * C::ROWS;
    rows = min(a.n_new * G - row0, C::ROWS);
  };
  // For the kernel that joins: the item that begins in this run and does not end
  // in it, by CTA (there is one at most) or by item.
  if (!SPREAD && threadIdx.x == 0 && !a.cuts_by_item) a.cuts[cta] = make_int4(-1, 0, 0, 0);
  // A cluster's parts: this CTA's, [ROWS][RED_STRIDE], a row's maximum and sum
  // behind its columns.
  float* share = reinterpret_cast<float*>(smem);

  if (w.left > 0) {
    const uint8_t* ring = smem + warp * (C::STAGES * C::STAGE_BYTES);
    Q4Copies<D, NT> copies;
    copies.begin(a, w, head, smem_u32(ring), warp, lane);
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s) copies.copy(a, s, warp, lane);
    const int r = lane >> 2, c = lane & 3;
    float* red_o = reinterpret_cast<float*>(smem + C::OFF_RED);  // [warp][ROWS][RED_STRIDE]
    float* red_ml = reinterpret_cast<float*>(smem + C::OFF_ML);  // [warp][ROWS][2]
    int stage = 0;
    bool first_item = true;
    do {
      item();
      Q4Raw<D, NT> raw;
      raw.read(a, w.b, kvh, row0, rows, lane);
      if (!SPREAD && threadIdx.x == 0 && w.tile == 0 && (a.cuts_by_item || w.here < w.n))
        a.cuts[a.cuts_by_item ? w.b * items + w.item : cta] =
            w.here < w.n ? make_int4(w.b, w.item, 2 * cta + (first_item ? 0 : 1),
                                     at.shares.of(at.run_end - w.left + w.n - 1))
                         : make_int4(-1, 0, 0, 0);
      Q4Rows<D, NT> R;
      q4_rows<D, NT, FEW>(a, raw, lane, R);
      Q4State<D, NT> S;
      S.clear();
      // Of the tile's keys of this warp: those in the sequence, and those that every row sees.
      int left = w.L - w.tile * kQ4Tile - warp * C::KEYS;
      int open = left - a.n_new + 1 + row0 / G;
      for (int t = 0; t < w.here; ++t) {
        asm volatile("cp.async.wait_group %0;" ::"n"(C::STAGES - 2) : "memory");
        __syncwarp();  // every lane's copies have landed, and the stage that is filled next has been read
        copies.copy(a, stage == 0 ? C::STAGES - 1 : stage - 1, warp, lane);
        const uint8_t* st = ring + stage * C::STAGE_BYTES;
        stage = stage == C::STAGES - 1 ? 0 : stage + 1;
        if (open >= C::KEYS) q4_step<D, NT, FEW, false>(st, lane, 0, 0, 0, 1, R, S);
        else if (left > 0) q4_step<D, NT, FEW, true>(st, lane, left, open, row0, G, R, S);
        left -= kQ4Tile, open -= kQ4Tile;
      }
#pragma unroll
      for (int off = FEW ? 2 : 4; off < 32; off <<= 1) {
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
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = warp * C::ROWS + j * 8 + 2 * c + i;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const float f = inverse_pow2(S.up[j][g][i]);
#pragma unroll
            for (int t = 0; t < 4; ++t)
              *reinterpret_cast<float2*>(&red_o[row * C::RED_STRIDE + g * 64 + r * 8 + t * 2]) =
                  make_float2(fmaf(S.o[j][g][t][i] * 0x1p24f, f, S.z[j][g][i]),
                              fmaf(S.o[j][g][t][2 + i] * 0x1p20f, f, S.z[j][g][i]));
          }
          if (r == 0) *reinterpret_cast<float2*>(&red_ml[row * 2]) = make_float2(S.m[j][i], S.l[j][i]);
        }
      }
      __syncthreads();
      const bool whole = w.here == w.n;
      const int slot = 2 * cta + (first_item ? 0 : 1);
      for (int x = threadIdx.x / (D / 4); x < rows; x += C::THREADS / (D / 4)) {
        const int col = threadIdx.x % (D / 4) * 4;
        float M = kNoLogit;
#pragma unroll
        for (int v = 0; v < C::WARPS; ++v) M = fmaxf(M, red_ml[(v * C::ROWS + x) * 2]);
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int v = 0; v < C::WARPS; ++v) {
          const float2 ml = *reinterpret_cast<const float2*>(&red_ml[(v * C::ROWS + x) * 2]);
          const float f = ex2(ml.x - M);
          const float4 y = *reinterpret_cast<const float4*>(&red_o[(v * C::ROWS + x) * C::RED_STRIDE + col]);
          sum = fmaf(ml.y, f, sum);
          acc.x = fmaf(y.x, f, acc.x), acc.y = fmaf(y.y, f, acc.y);
          acc.z = fmaf(y.z, f, acc.z), acc.w = fmaf(y.w, f, acc.w);
        }
        if constexpr (SPREAD) {  // (the rings have been read)
          *reinterpret_cast<float4*>(&share[x * C::RED_STRIDE + col]) = acc;
          if (col == 0) *reinterpret_cast<float2*>(&share[x * C::RED_STRIDE + D]) = make_float2(M, sum);
          continue;
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
    } while (w.next(a, head));
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  if constexpr (SPREAD) {
    // The cluster's parts, in the order of the keys: four columns of a row a
    // thread, spread over all CTAs. A CTA without tiles has a sum of zero.
    item();
    if (w.here == 0) {
      for (int x = threadIdx.x; x < rows; x += C::THREADS)
        *reinterpret_cast<float2*>(&share[x * C::RED_STRIDE + D]) = make_float2(kNoLogit, 0.f);
    }
    cluster_sync();
    for (int e = threadIdx.x * a.spread + cta % a.spread; e < rows * (D / 4); e += C::THREADS * a.spread) {
      const int x = e / (D / 4), col = e % (D / 4) * 4;
      const uint32_t row = smem_u32(&share[x * C::RED_STRIDE]);
      float4 ml[kQ4Cluster], y[kQ4Cluster];
#pragma unroll
      for (int v = 0; v < kQ4Cluster; ++v) {
        ml[v].y = 0.f;
        if (v >= a.spread) continue;
        const uint32_t from = map_to_rank(row, v);
        ml[v] = ld_cluster_f4(from + D * 4);  // maximum, sum, nothing
        y[v] = ld_cluster_f4(from + col * 4);
      }
      float M = kNoLogit, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int v = 0; v < kQ4Cluster; ++v)
        if (v < a.spread) M = fmaxf(M, ml[v].x);
#pragma unroll
      for (int v = 0; v < kQ4Cluster; ++v) {
        if (ml[v].y == 0.f) continue;
        const float f = ex2(ml[v].x - M);
        sum = fmaf(ml[v].y, f, sum);
        acc.x = fmaf(y[v].x, f, acc.x), acc.y = fmaf(y[v].y, f, acc.y);
        acc.z = fmaf(y[v].z, f, acc.z), acc.w = fmaf(y[v].w, f, acc.w);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const long long to = q4_row(a, w.b, kvh, row0 + x);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + to * D + col) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      if (col == 0) a.lse[to] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
    }
    cluster_sync();  // no CTA's shared memory goes before it has been read
    return;
  }
  // Sequences without keys have no tiles: every CTA writes its share of their rows.
  for (int b = cta; b < a.B; b += gridDim.x) {
    if (q4_len(a, b) > 0) continue;
    const long long row = static_cast<long long>(b) * a.n_new * a.H;
    const int n = a.n_new * a.H;
    for (long long x = threadIdx.x; x < static_cast<long long>(n) * (D / 8); x += C::THREADS)
      reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + row * D)[x] = make_uint4(0u, 0u, 0u, 0u);
    for (int x = threadIdx.x; x < n; x += C::THREADS) a.lse[row + x] = -INFINITY;
    for (int x = threadIdx.x; a.cuts_by_item && x < items; x += C::THREADS)
      a.cuts[b * items + x] = make_int4(-1, 0, 0, 0);
  }
}

// Joins the parts of cut items: CTA (x, y) rows of the x-th cut. O = sum of
// 2^(lse_i - M) O_i over the sum of the weights, in a fixed order: a row's SUBS
// warps take every SUBS-th part, then the first adds up theirs. A warp's first
// eight parts are read along with the sums, so that with 8 SUBS parts there are
// two reads to wait for.
template <int D, int SUBS>
__global__ void __launch_bounds__(512, 2) fa_decode_q4_join_kernel(const Q4DecodeArgs a) {
  constexpr int CPL = D / 32, AHEAD = 8;  // columns per lane
  __shared__ float red[SUBS > 1 ? 16 : 1][D + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % SUBS;
  const int x = blockIdx.y * (blockDim.x / (32 * SUBS)) + warp / SUBS;
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  const int4 cut = a.cuts[blockIdx.x];
  if (cut.x < 0) return;
  const int kvh = cut.y / a.row_blocks, row0 = (cut.y - kvh * a.row_blocks) * a.rows_per;
  const bool on = x < min(a.n_new * (a.H / a.Hk) - row0, a.rows_per);
  const int n = on ? cut.w - cut.z / 2 + 1 : 0;
  auto part = [&](int i) { return static_cast<size_t>(i == 0 ? cut.z : cut.z / 2 * 2 + 2 * i) * a.rows_per + x; };
  struct Part {
    float lse, y[CPL];
  };
  auto read = [&](int i) {
    Part p;
    p.lse = a.part_lse[part(i)];
    const float* src = a.part_o + part(i) * D + lane * CPL;
    if constexpr (CPL == 4) {
      const float4 v = *reinterpret_cast<const float4*>(src);
      p.y[0] = v.x, p.y[1] = v.y, p.y[2] = v.z, p.y[3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(src);
      p.y[0] = v.x, p.y[1] = v.y;
    }
    return p;
  };
  Part first[AHEAD];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k)
    if (sub + k * SUBS < n) first[k] = read(sub + k * SUBS);
  float M = -INFINITY, sum = 0.f, acc[CPL];
  for (int i = lane; i < n; i += 32) M = max_nan(M, a.part_lse[part(i)]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, off));
#pragma unroll
  for (int k = 0; k < CPL; ++k) acc[k] = 0.f;
  auto add = [&](const Part& p) {
    const float f = ex2(p.lse - M);
    sum += f;
#pragma unroll
    for (int k = 0; k < CPL; ++k) acc[k] = fmaf(f, p.y[k], acc[k]);
  };
  if (M != -INFINITY) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (sub + k * SUBS < n) add(first[k]);
#pragma unroll 4
    for (int i = sub + AHEAD * SUBS; i < n; i += SUBS) add(read(i));
  }
  if constexpr (SUBS > 1) {
#pragma unroll
    for (int k = 0; k < CPL; ++k) red[warp][lane * CPL + k] = acc[k];
    if (lane == 0) red[warp][D] = sum;
    __syncthreads();
  }
  if (!on || sub > 0) return;
#pragma unroll
  for (int v = 1; v < SUBS; ++v) {
    sum += red[warp + v][D];
#pragma unroll
    for (int k = 0; k < CPL; ++k) acc[k] += red[warp + v][lane * CPL + k];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const long long at = q4_row(a, cut.x, kvh, row0 + x);
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + at * D + lane * CPL);
#pragma unroll
  for (int k = 0; k < CPL; k += 2) out[k / 2] = pack_bf16x2(acc[k] * inv, acc[k + 1] * inv);
  if (lane == 0) a.lse[at] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
}

template <int D, int NT, bool FEW>
static cudaError_t launch_q4_t(const Q4DecodeArgs& a, cudaStream_t stream, const LaunchMarks* marks) {
  using C = Q4Cfg<D, NT>;
  static_assert(C::CTAS * 152 <= kQ4MaxCtas, "the workspace holds every CTA's parts");
  auto kern = a.spread ? fa_decode_q4_kernel<D, NT, FEW, true> : fa_decode_q4_kernel<D, NT, FEW, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const int items = a.B * a.Hk * a.row_blocks;
  const int grid = a.spread ? items * a.spread : std::min(a.most_tiles, C::CTAS * 152);
  mark(marks, true, 0, stream);
  e = launch_cluster_maybe_pdl(kern, dim3(grid), dim3(C::THREADS), C::SMEM_BYTES, stream, marks == nullptr,
                               std::max(a.spread, 1), a);
  mark(marks, false, 0, stream);
  if (e != cudaSuccess || a.spread) return e;
  mark(marks, true, 1, stream);
  if (a.cuts_by_item) {
    const unsigned rows = std::min(a.n_new * (a.H / a.Hk), C::ROWS);
    e = launch_maybe_pdl(fa_decode_q4_join_kernel<D, 8>, dim3(items, (rows + 1) / 2), dim3(512), 0, stream,
                         marks == nullptr, a);
  } else {
    e = launch_maybe_pdl(fa_decode_q4_join_kernel<D, 1>, dim3(grid), dim3(32 * C::ROWS), 0, stream, marks == nullptr,
                         a);
  }
  mark(marks, false, 1, stream);
  return e;
}

template <int D>
static cudaError_t launch_q4_d(const Q4DecodeArgs& a, cudaStream_t stream, const LaunchMarks* m) {
  if (a.rows_per > 8) return launch_q4_t<D, 2, false>(a, stream, m);
  return a.n_new * (a.H / a.Hk) > 4 ? launch_q4_t<D, 1, false>(a, stream, m) : launch_q4_t<D, 1, true>(a, stream, m);
}

cudaError_t launch_decode_q4(const Q4DecodeArgs& a, cudaStream_t stream, const LaunchMarks* m) {
  return a.D == 64 ? launch_q4_d<64>(a, stream, m) : launch_q4_d<128>(a, stream, m);
}

}  // namespace fa
