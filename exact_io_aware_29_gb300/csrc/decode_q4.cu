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
// made in registers from the words as they lie in the cache, two instructions
// for two codes (tcgen05 would take them through shared or tensor memory).
//   Q K^T: f16. A nibble in the low bits of an f16 is code 2^-24 (a subnormal,
//   exact), four bits further up code 2^-20: one AND for two codes. The row of
//   q is scaled to [2^14, 2^15) by a power of two, so that its f16 is exact
//   (smaller than 2^-29 of the row's largest: rounded at 2^-40 of it).
//   P V: bf16. A nibble under the exponent of 128 is 128 + code; p (z - 128 s)
//   in place of p z takes the 128 out again. p s as the sum of two bf16 numbers
//   (relative error 2^-17).
// One warp streams 128-key tiles through a ring with bulk copies (a block's
// keys of one head lie together: codes, then scales, in up to 8 pieces), four
// warps compute on 16 keys at a time. Softmax statistics and sums are fp32.
// Every item (rows, key range) writes a normalised partial O and the log2 of
// its sum; a second kernel joins them in a fixed order.
#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace fa {

template <int D>
struct Q4Cfg {
  static constexpr int TK = 128;                   // keys per tile
  static constexpr int NG = D / 64;                // groups of a row
  static constexpr int CODE_BYTES = TK * D / 2;
  static constexpr int SCALE_BYTES = TK * NG * 4;
  static constexpr int OFF_KS = CODE_BYTES, OFF_VC = OFF_KS + SCALE_BYTES, OFF_VS = OFF_VC + CODE_BYTES;
  static constexpr int STAGE_BYTES = 2 * (CODE_BYTES + SCALE_BYTES);
  static constexpr int STAGES = 4;
  static constexpr int CWARPS = 4;                 // consumer warps
  static constexpr int THREADS = (CWARPS + 1) * 32;
  static constexpr int OFF_BAR = STAGES * STAGE_BYTES;
  static constexpr int SMEM_BYTES = OFF_BAR + 2 * STAGES * 8 + STAGES * 4 + 16;
  static_assert(CWARPS * 16 * (D + 2) * 4 <= OFF_BAR, "the join of the warps fits in the stages");
};

namespace {

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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
// max(a, b), NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The work of one CTA: rows row0 .. row0 + rows - 1 of sequence b and key head
// kvh (row = query * G + head of the group), keys [c0, c1).
struct Q4Item {
  int b, kvh, row0, rows, c0, c1, L, split;
};
__device__ __forceinline__ bool q4_item(const Q4DecodeArgs& a, int id, Q4Item& it) {
  it.split = id % a.nsplit;
  int x = id / a.nsplit;
  const int blk = x % a.row_blocks;
  x /= a.row_blocks;
  it.kvh = x % a.Hk;
  it.b = x / a.Hk;
  it.row0 = blk * a.rows_per;
  it.rows = min(a.n_new * (a.H / a.Hk) - it.row0, a.rows_per);
  it.L = min(max(a.seq_lens[it.b], 0), a.max_seq_len);
  it.c0 = it.split * a.chunk;
  it.c1 = min(it.L, it.c0 + a.chunk);
  return it.c1 > it.c0;
}

// Row r of the item as the flattened row (b * n_new + query) * H + head.
__device__ __forceinline__ long long q4_row(const Q4DecodeArgs& a, const Q4Item& it, int r) {
  const int G = a.H / a.Hk, row = it.row0 + r;
  return (static_cast<long long>(it.b) * a.n_new + row / G) * a.H + it.kvh * G + row % G;
}

// What a lane holds of the queries: lane (r, c) = (lane / 4, lane % 4).
template <int D, int NT>
struct Q4Rows {
  static constexpr int NG = D / 64;
  uint32_t q[NT][NG][4][2];  // B fragments of row 8 j + r, k-step t of group g
  float qs[NT][2];           // of rows 8 j + 2 c + {0, 1}: what a product of codes is multiplied by
  float sum[NT][NG][2];      // scale log2e times the sum of the row's group
  int last[NT][2];           // keys c < last are visible
};

template <int D, int NT>
__device__ __forceinline__ void q4_load_rows(const Q4DecodeArgs& a, const Q4Item& it, int lane, Q4Rows<D, NT>& R) {
  constexpr int NG = D / 64;
  const int r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const bool on = j * 8 + r < it.rows;
    const uint4* src =
        reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (on ? q4_row(a, it, j * 8 + r) : 0LL) * D);
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
    // 2^shift q is at most 2^15; 2^shift and 2^(24 - shift) are fp32 numbers.
    const int e = static_cast<int>(__float_as_uint(mx) >> 23) - 127;
    const int shift = min(max(14 - e, -100), 100);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
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
      for (int h = 0; h < 2; ++h) {  // words 2 c + h of the codes: elements {0 .. 7} + 8 h
        const uint32_t* x = &w[g][4 * h];
        // Nibbles (0, 4), (1, 5) 16-fold, (2, 6), (3, 7) 16-fold.
        R.q[j][g][2 * h][0] = pack_f16x2(lo_f(x[0]) * up, lo_f(x[2]) * up);
        R.q[j][g][2 * h][1] = pack_f16x2(hi_f(x[0]) * (up * 0.0625f), hi_f(x[2]) * (up * 0.0625f));
        R.q[j][g][2 * h + 1][0] = pack_f16x2(lo_f(x[1]) * up, lo_f(x[3]) * up);
        R.q[j][g][2 * h + 1][1] = pack_f16x2(hi_f(x[1]) * (up * 0.0625f), hi_f(x[3]) * (up * 0.0625f));
      }
    }
    const float down = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + 24 - shift) << 23);
    // To the lanes of the C fragments' columns: row 8 j + 2 c + i comes from lane (2 c + i, .).
    const int G = a.H / a.Hk;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      R.qs[j][i] = __shfl_sync(0xffffffffu, down, (2 * c + i) * 4);
#pragma unroll
      for (int g = 0; g < NG; ++g) R.sum[j][g][i] = __shfl_sync(0xffffffffu, s[g], (2 * c + i) * 4);
      R.last[j][i] = it.L - a.n_new + 1 + (it.row0 + j * 8 + 2 * c + i) / G;
    }
  }
}

// Running softmax of a lane's columns (rows 8 j + 2 c + {0, 1}): the maximum is
// the same in all lanes of a column, the sums are the lane's own.
template <int D, int NT>
struct Q4State {
  static constexpr int NG = D / 64;
  float o[NT][NG][4][4];  // C fragments: dimensions 64 g + 8 r + 2 t + {0, 1} (c0 c1, c2 c3)
  float m[NT][2], l[NT][2], z[NT][NG][2];
};

// 16 keys of a tile from key k0 of it on; `left`: keys of the range from the
// tile's first on. MASKED: some of them may be hidden from some rows, or past
// the range; `first` is the tile's first key. held: the keys' block is in the
// pool (others read as zeros).
template <int D, int NT, bool MASKED>
__device__ __forceinline__ void q4_slice(const uint8_t* st, int k0, int lane, bool held, int first, int left,
                                         const Q4Rows<D, NT>& R, Q4State<D, NT>& S) {
  using C = Q4Cfg<D>;
  constexpr int NG = D / 64;
  const int r = lane >> 2, c = lane & 3;
  // Row i of the A operand of Q K^T, and k index i of P V, is key (i >> 1) + 4 (i & 1)
  // of its eight: the lanes of a load then meet two banks' worth of rows, not one.
  const int ka = k0 + (r >> 1) + 4 * (r & 1);
  float sc[NT][2][2];  // [key ka + 8 h][row i]
  float vs[NG][2], vz[NG][2];
  {
    uint32_t ksz[2][NG], vsz[2][NG];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t* pk = reinterpret_cast<const uint32_t*>(st + C::OFF_KS) + (ka + 8 * h) * NG;
      const uint32_t* pv = reinterpret_cast<const uint32_t*>(st + C::OFF_VS) + (ka + 8 * h) * NG;
      const bool on = held && (!MASKED || ka + 8 * h < left);
#pragma unroll
      for (int g = 0; g < NG; ++g) ksz[h][g] = on ? pk[g] : 0u, vsz[h][g] = on ? pv[g] : 0u;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) sc[j][0][0] = sc[j][0][1] = sc[j][1][0] = sc[j][1][1] = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint2 x = *reinterpret_cast<const uint2*>(st + ka * (D / 2) + g * 32 + c * 8);
      const uint2 y = *reinterpret_cast<const uint2*>(st + (ka + 8) * (D / 2) + g * 32 + c * 8);
      const uint32_t wx[4] = {x.x, x.x >> 8, x.y, x.y >> 8}, wy[4] = {y.x, y.x >> 8, y.y, y.y >> 8};
      float acc[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
          mma_f16(acc[j], wx[t] & 0x000F000Fu, wy[t] & 0x000F000Fu, wx[t] & 0x00F000F0u, wy[t] & 0x00F000F0u,
                  R.q[j][g][t][0], R.q[j][g][t][1]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float s = lo_f(ksz[h][g]), z = hi_f(ksz[h][g]);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            sc[j][h][i] = fmaf(acc[j][2 * h + i] * R.qs[j][i], s, fmaf(z, R.sum[j][g][i], sc[j][h][i]));
        }
        vs[g][h] = lo_f(vsz[h][g]);
        vz[g][h] = fmaf(-128.f, vs[g][h], hi_f(vsz[h][g]));
      }
    }
  }
  bool seen[NT][2][2];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        seen[j][h][i] = !MASKED || (ka + 8 * h < left && first + ka + 8 * h < R.last[j][i]);
        if (!seen[j][h][i]) sc[j][h][i] = -INFINITY;
      }
      // The maximum follows once a logit is 2^8 times above it: sums of up to
      // 2^8 terms' worth more cost fp32 nothing, and most slices pass.
      const float mx = fmaxf(sc[j][0][i], sc[j][1][i]);
      if (__any_sync(0xffffffffu, mx > S.m[j][i] + 8.f)) {
        float mn = fmaxf(mx, S.m[j][i]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
        const float alpha = mn == -INFINITY ? 1.f : ex2(S.m[j][i] - mn);
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
  // P, times the groups' scales, as B operands.
  uint32_t bh[NT][NG][2], bl[NT][NG][2];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    float neg[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) neg[i] = S.m[j][i] == -INFINITY ? 0.f : -S.m[j][i];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float p[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        p[i] = ex2(sc[j][h][i] + neg[i]);
        S.l[j][i] += p[i];
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          x[i] = seen[j][h][i] ? p[i] * vs[g][h] : 0.f;  // a hidden key's scale may be NaN
          S.z[j][g][i] = fmaf(p[i], seen[j][h][i] ? vz[g][h] : 0.f, S.z[j][g][i]);
        }
        const uint32_t hi = pack_bf16x2(x[0], x[1]);
        bh[j][g][h] = transpose8(hi);
        bl[j][g][h] = transpose8(pack_bf16x2(x[0] - lo_f(hi), x[1] - hi_f(hi)));
      }
    }
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    // Word r of the group of keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9 (as k indices).
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = *reinterpret_cast<const uint32_t*>(st + C::OFF_VC + (k0 + c + 4 * (i & 1) + 8 * (i >> 1)) * (D / 2) +
                                                g * 32 + r * 4);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      // Nibbles 2 t (dimensions 8 r + 2 t: rows 0 .. 7) and 2 t + 1 (rows 8 .. 15) of both keys of a pair.
      const uint32_t sel = t < 2 ? 0x5410u : 0x7632u;
      const uint32_t p0 = __byte_perm(w[0], w[1], sel) >> (8 * (t & 1));
      const uint32_t p1 = __byte_perm(w[2], w[3], sel) >> (8 * (t & 1));
      const uint32_t a0 = (p0 & 0x000F000Fu) | 0x43004300u, a1 = ((p0 >> 4) & 0x000F000Fu) | 0x43004300u;
      const uint32_t a2 = (p1 & 0x000F000Fu) | 0x43004300u, a3 = ((p1 >> 4) & 0x000F000Fu) | 0x43004300u;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        mma_bf16(S.o[j][g][t], a0, a1, a2, a3, bh[j][g][0], bh[j][g][1]);
        mma_bf16(S.o[j][g][t], a0, a1, a2, a3, bl[j][g][0], bl[j][g][1]);
      }
    }
  }
}

}  // namespace

template <int D, int NT>
__global__ void __launch_bounds__(Q4Cfg<D>::THREADS) fa_decode_q4_kernel(const Q4DecodeArgs a) {
  using C = Q4Cfg<D>;
  constexpr int NG = C::NG;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::STAGES;
  uint32_t* held_bits = reinterpret_cast<uint32_t*>(empty + C::STAGES);  // per stage: slices whose block is in the pool
  volatile int* abort_flag = reinterpret_cast<volatile int*>(held_bits + C::STAGES);

  if (threadIdx.x == 0) griddep_launch_dependents();
  Q4Item it;
  if (!q4_item(a, blockIdx.x, it)) return;  // the whole CTA
  const int ntiles = (it.c1 - it.c0 + C::TK - 1) / C::TK;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], C::CWARPS);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();

  if (warp == C::CWARPS) {
    // ----------------------------------------------------------- copy warp
    // Lane (piece, array): one copy of `piece` keys of the codes or scales of K or V.
    if (g_test_drop_loads) return;
    const int p = lane >> 2, arr = lane & 3;
    const int row_bytes = (arr & 1) ? NG * 4 : D / 2;
    const uint8_t* base = arr == 0 ? a.k_codes : (arr == 1 ? a.k_scales : (arr == 2 ? a.v_codes : a.v_scales));
    const int dst0 = (arr == 0 ? 0 : (arr == 1 ? C::OFF_KS : (arr == 2 ? C::OFF_VC : C::OFF_VS))) +
                     p * a.piece * row_bytes;
    int issued = 0;
    for (int t = 0; t < ntiles; ++t) {
      const int s = t % C::STAGES;
      const int key = it.c0 + t * C::TK + p * a.piece;
      const bool mine = p * a.piece < C::TK && key < it.c1;
      int phys = -1, block = 0;
      if (mine) {
        block = key / a.block_size;
        phys = a.block_table[static_cast<long long>(it.b) * a.max_blocks + block];
      }
      const bool held = mine && phys >= 0 && phys < a.num_blocks;
      const uint32_t lanes = __ballot_sync(0xffffffffu, held && arr == 0);
      if (t >= C::STAGES &&
          !__all_sync(0xffffffffu, mbar_wait(&empty[s], (t / C::STAGES - 1) & 1, abort_flag)))
        break;
      if (lane == 0) {
        uint32_t bits = 0u;  // of 16-key slices
        for (int i = 0; i < C::TK / 16; ++i) bits |= ((lanes >> (i * 16 / a.piece * 4)) & 1u) << i;
        held_bits[s] = bits;
        mbar_arrive_expect_tx(&full[s], __popc(lanes) * a.piece * 2 * (D / 2 + NG * 4));
      }
      __syncwarp();
      if (held) {
        const long long row = (static_cast<long long>(phys) * a.Hk + it.kvh) * a.block_size + (key - block * a.block_size);
        bulk_load(smem + s * C::STAGE_BYTES + dst0, base + row * row_bytes, a.piece * row_bytes, &full[s]);
      }
      ++issued;
    }
    // Do not leave with copies in flight (matters only after an abort, when
    // the consumers stopped waiting; every issued copy lands).
    if (lane == 0)
      for (int t = max(0, issued - C::STAGES); t < issued; ++t)
        mbar_wait_drain(&full[t % C::STAGES], (t / C::STAGES) & 1);
    return;
  }

  // -------------------------------------------------------- consumer warps
  Q4Rows<D, NT> R;
  q4_load_rows<D, NT>(a, it, lane, R);
  Q4State<D, NT> S;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      S.m[j][i] = -INFINITY, S.l[j][i] = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) S.z[j][g][i] = 0.f;
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int t = 0; t < 4; ++t) S.o[j][g][t][0] = S.o[j][g][t][1] = S.o[j][g][t][2] = S.o[j][g][t][3] = 0.f;
    }
  }
  // Keys from here on are hidden from some row.
  const int open = it.L - a.n_new + 1 + it.row0 / (a.H / a.Hk);
  for (int t = 0; t < ntiles; ++t) {
    const int s = t % C::STAGES;
    if (!__all_sync(0xffffffffu, mbar_wait(&full[s], (t / C::STAGES) & 1, abort_flag))) break;
    const uint8_t* st = smem + s * C::STAGE_BYTES;
    const int first = it.c0 + t * C::TK, left = it.c1 - first;
    const uint32_t held = held_bits[s];
    for (int k0 = warp * 16; k0 < min(C::TK, left); k0 += C::CWARPS * 16) {
      const bool h = (held >> (k0 / 16)) & 1u;
      if (k0 + 16 > left || first + k0 + 16 > open) q4_slice<D, NT, true>(st, k0, lane, h, first, left, R, S);
      else q4_slice<D, NT, false>(st, k0, lane, h, first, left, R, S);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
  }
  const int r = lane >> 2, c = lane & 3;
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
  // Join the warps: every consumer is past its last tile, so the stage memory
  // (all copies landed) is free for the partial results.
  named_bar_sync(1, C::CWARPS * 32);
  constexpr int ROWS = 8 * NT;
  float* red_o = reinterpret_cast<float*>(smem);      // [warp][ROWS][D]
  float* red_ml = red_o + C::CWARPS * ROWS * D;       // [warp][ROWS][2]
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = warp * ROWS + j * 8 + 2 * c + i;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
          *reinterpret_cast<float2*>(&red_o[row * D + g * 64 + r * 8 + t * 2]) =
              make_float2(S.o[j][g][t][i] + S.z[j][g][i], S.o[j][g][t][2 + i] + S.z[j][g][i]);
      }
      if (r == 0) {
        red_ml[row * 2] = S.m[j][i];
        red_ml[row * 2 + 1] = S.l[j][i];
      }
    }
  }
  named_bar_sync(1, C::CWARPS * 32);
  for (int x = threadIdx.x / (D / 4); x < it.rows; x += C::CWARPS * 32 / (D / 4)) {
    const int col = threadIdx.x % (D / 4) * 4;
    float M = -INFINITY;
    for (int w = 0; w < C::CWARPS; ++w) M = fmaxf(M, red_ml[(w * ROWS + x) * 2]);
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < C::CWARPS; ++w) {
      const float mw = red_ml[(w * ROWS + x) * 2], lw = red_ml[(w * ROWS + x) * 2 + 1];
      if (lw == 0.f) continue;  // no keys (NaN logits alone leave mw at -inf, too, but make lw NaN)
      const float f = ex2(mw - M);
      const float4 v = *reinterpret_cast<const float4*>(&red_o[(w * ROWS + x) * D + col]);
      sum = fmaf(lw, f, sum);
      acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y);
      acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const float lse2 = sum == 0.f ? -INFINITY : M + log2f(sum);
    const size_t row = static_cast<size_t>(q4_row(a, it, x)), at = row * a.nsplit + it.split;
    *reinterpret_cast<float4*>(a.part_o + at * D + col) =
        make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (col == 0) a.part_lse[at] = lse2;
  }
}

// Joins the parts of a row: O = sum of 2^(lse_i - M) O_i over the sum of the
// weights, in the order of the keys. One CTA per row, its warps every fourth
// part, then their sums.
template <int D>
__global__ void __launch_bounds__(128) fa_decode_q4_join_kernel(const Q4DecodeArgs a) {
  constexpr int CPL = D / 32;  // columns per lane
  __shared__ float red[4][D + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int L = min(max(a.seq_lens[blockIdx.x / (a.n_new * a.H)], 0), a.max_seq_len);
  const int n = (L + a.chunk - 1) / a.chunk;
  const size_t at0 = static_cast<size_t>(blockIdx.x) * a.nsplit;
  griddep_wait();
  float M = -INFINITY;
  for (int i = lane; i < n; i += 32) M = max_nan(M, a.part_lse[at0 + i]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, off));
  float sum = 0.f, acc[CPL];
#pragma unroll
  for (int k = 0; k < CPL; ++k) acc[k] = 0.f;
  for (int i = warp; i < n && M != -INFINITY; i += 4) {
    const float w = ex2(a.part_lse[at0 + i] - M);
    const float* src = a.part_o + (at0 + i) * D + lane * CPL;
    sum += w;
#pragma unroll
    for (int k = 0; k < CPL; ++k) acc[k] = fmaf(w, src[k], acc[k]);
  }
#pragma unroll
  for (int k = 0; k < CPL; ++k) red[warp][lane * CPL + k] = acc[k];
  if (lane == 0) red[warp][D] = sum;
  __syncthreads();
  if (warp > 0) return;
  sum = red[0][D];
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    sum += red[w][D];
#pragma unroll
    for (int k = 0; k < CPL; ++k) acc[k] += red[w][lane * CPL + k];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + static_cast<size_t>(blockIdx.x) * D +
                                              lane * CPL);
#pragma unroll
  for (int k = 0; k < CPL; k += 2) out[k / 2] = pack_bf16x2(acc[k] * inv, acc[k + 1] * inv);
  if (lane == 0) a.lse[blockIdx.x] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
}

template <int D, int NT>
static cudaError_t launch_q4_t(const Q4DecodeArgs& a, cudaStream_t stream, const LaunchMarks* marks) {
  using C = Q4Cfg<D>;
  auto kern = fa_decode_q4_kernel<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const long long items = static_cast<long long>(a.B) * a.Hk * a.row_blocks * a.nsplit;
  const long long rows = static_cast<long long>(a.B) * a.n_new * a.H;
  if (items > 0x7fffffffLL || rows > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  mark(marks, true, 0, stream);
  kern<<<static_cast<unsigned>(items), C::THREADS, C::SMEM_BYTES, stream>>>(a);
  e = cudaGetLastError();
  mark(marks, false, 0, stream);
  if (e != cudaSuccess) return e;
  mark(marks, true, 1, stream);
  e = launch_maybe_pdl(fa_decode_q4_join_kernel<D>, dim3(static_cast<unsigned>(rows)), dim3(128), 0, stream,
                       marks == nullptr, a);
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
