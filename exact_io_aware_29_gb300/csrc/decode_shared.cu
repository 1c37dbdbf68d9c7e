// One decoding step for a batch whose sequences share long prefixes, over a
// paged KV cache with grouped heads: the query of (sequence b, head h) attends
// to the tokens of b's prefix and to b's own tokens, which follow them:
//   O = softmax(scale q [K_prefix; K_own]^T) [V_prefix; V_own].
// The softmax of the two parts is joined by its running maximum and sum
// ("FlashAttention算法详解", §Online Softmax: merging two states), so the
// prefix is computed once per key head for all rows that share it (rows =
// sequences x G heads of the group), each own part once per sequence.
//
// A prefix with more than 16 rows is a dense product (decode_prefix.cu). The
// rest is streamed here: a work item is (rows, key head, key range), the up to
// 16 rows (sequence, head) of one prefix or up to 64 heads of one sequence on
// its own tokens. Reading K and V is the bound (4 d bytes per key against 4 d
// flops per key and row), so one warp streams 64-key tiles through a ring with
// TMA (a page is a multiple of 64 tokens: no tile crosses one) while four warps
// compute on 16-row blocks with mma.sync: at up to 16 rows the padded products
// need about a quarter of that unit's rate at HBM speed (64 sequences of 4096
// own tokens, 32/8 heads, d 128: 165 us, 6.5 TB/s). With more than one 16-row
// block the warps share the blocks out and each takes more keys of the tile.
//   S = Q K^T (bf16, fp32 sums), p = 2^(scale log2e S - m), O += p V with p
//   as the sum of two bf16 numbers (hi = bf16(p), lo = bf16(p - hi): relative
//   error 2^-17), so P costs no more accuracy than the fp32 sums around it.
// Every item writes a normalised partial O and the log2 of its sum; a second
// kernel joins the parts of each row in a fixed order (deterministic). Only a
// sum of exactly zero (no keys) is left out of a join: a NaN logit makes its
// part's sum NaN and the row's O and LSE with it, however its keys are split.
#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace fa {

template <int D>
struct SharedCfg {
  static constexpr int TK = 64;                       // keys per tile (TMA box height)
  static constexpr int BOXES = D / 64;                // 64-column boxes per row
  static constexpr int BOX_BYTES = TK * 128;          // 64 rows x 64 bf16, 128B-swizzled
  static constexpr int TILE_BYTES = BOXES * BOX_BYTES;
  static constexpr int STAGE_BYTES = 2 * TILE_BYTES;  // K tile, then V tile
  static constexpr int STAGES = 3;                    // two CTAs per SM with 96 KB each, four with 48 (d 64)
  static constexpr int CTAS = D == 128 ? 2 : 4;       // per SM (the registers allow no more at d 128)
  static constexpr int CWARPS = 4;                    // consumer warps
  static constexpr int ROWS = 16 * CWARPS;            // most rows of an item
  static constexpr int THREADS = (CWARPS + 1) * 32;
  static constexpr int OFF_BAR = STAGES * STAGE_BYTES;
  static constexpr int SMEM_BYTES = OFF_BAR + 2 * STAGES * 8 + 16 + 1024;  // + alignment slack
  static_assert(CWARPS * 16 * (D + 2) * 4 <= OFF_BAR, "merge buffer fits in the stages");
};

namespace {

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c (16 x 8, fp32) += a (16 x 16, bf16) b (16 x 8, bf16).
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte unit u (8 columns) of tile row r.
__device__ __forceinline__ uint32_t unit_off(int r, int u) {
  return static_cast<uint32_t>((u >> 3) * (64 * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4));
}

// p0, p1 as packed bf16 pairs hi + lo.
__device__ __forceinline__ void split_bf16(float p0, float p1, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(p0, p1);
  lo = pack_bf16x2(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xFFFF0000u));
}

// max(a, b), NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

}  // namespace

// What one CTA works on.
struct SharedItem {
  int seq0, rows, row0;    // rows row0 .. row0 + rows - 1 of the sequences from seq0 on (row = sequence * G + head)
  int kvh, c0, c1;         // key head, key range
  int slot;                // partial index of every row
  const int* table;        // pages of the keys
  int phys;                // block id of the first page
};

// False if item `id` has nothing to do. What it reads (offsets, length, first
// block id) it reads in one go: a short item's time is made of such latencies.
template <int D>
__device__ __forceinline__ bool shared_item(const SharedArgs& a, int id, SharedItem& it) {
  using C = SharedCfg<D>;
  const int G = a.H / a.Hk;
  const int n_prefix_items = a.prefix_tiles ? 0 : a.P * a.Hk * a.prefix_splits;
  if (id < n_prefix_items) {
    const int split = id % a.prefix_splits;
    int x = id / a.prefix_splits;
    it.kvh = x % a.Hk;
    const int p = x / a.Hk;
    int n;
    it.c0 = split * a.prefix_chunk;
    it.table = a.prefix_table + static_cast<size_t>(p) * a.max_prefix_blocks;
    it.phys = it.table[it.c0 / a.block_size];  // c0 < max_prefix_len: inside the row
    const int L = min(max(a.prefix_lens[p], 0), a.max_prefix_len);
    prefix_seqs(a, p, it.seq0, n);
    it.row0 = 0;
    it.rows = min(n * G, 16);  // max_group * G <= 16 here
    it.c1 = min(L, it.c0 + a.prefix_chunk);
    it.slot = split;
  } else {
    id -= n_prefix_items;
    const int split = id % a.seq_splits;
    int x = id / a.seq_splits;
    const int blk = x % a.seq_blocks;
    x /= a.seq_blocks;
    it.kvh = x % a.Hk;
    it.seq0 = x / a.Hk;
    it.row0 = blk * C::ROWS;
    it.rows = min(G - it.row0, C::ROWS);
    it.c0 = split * a.seq_chunk;
    it.table = a.block_table + static_cast<size_t>(it.seq0) * a.max_blocks;
    it.phys = it.table[it.c0 / a.block_size];
    const int L = min(max(a.seq_lens[it.seq0], 0), a.max_seq_len);
    it.c1 = min(L, it.c0 + a.seq_chunk);
    it.slot = a.prefix_splits + split;
  }
  return it.rows > 0 && it.c1 > it.c0;
}

template <int D>
__global__ void __launch_bounds__(SharedCfg<D>::THREADS, SharedCfg<D>::CTAS)
    fa_decode_shared_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                            const SharedArgs a) {
  using C = SharedCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::STAGES;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + C::STAGES);

  if (threadIdx.x == 0) griddep_launch_dependents();
  // With the prefix part in a kernel of its own before this one (launched
  // programmatically, so that the two overlap), this grid must not end before
  // that one: the kernel that joins the parts waits for this grid only. Its
  // last CTA sees to that.
  const bool waits = a.prefix_tiles && blockIdx.x == gridDim.x - 1 && threadIdx.x == 0;
  SharedItem it;
  if (!shared_item<D>(a, blockIdx.x, it)) {  // the whole CTA
    if (waits) griddep_wait();
    return;
  }
  const int ntiles = (it.c1 - it.c0 + C::TK - 1) / C::TK;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Tile t into its stage, from block `phys` (the page of key c0 + 64 t).
  // Out-of-range block ids read as zeros (TMA fills outside the pool).
  auto issue = [&](int t, int phys) {
    const int key = it.c0 + t * C::TK, s = t % C::STAGES;
    const int row = (phys < 0 || phys >= a.num_blocks) ? -C::TK : phys * a.block_size + key % a.block_size;
    uint8_t* st = smem + s * C::STAGE_BYTES;
    mbar_arrive_expect_tx(&full[s], C::STAGE_BYTES);
#pragma unroll
    for (int c = 0; c < C::BOXES; ++c) {
      tma_load_3d(st + c * C::BOX_BYTES, &tmK, &full[s], c * 64, it.kvh, row);
      tma_load_3d(st + C::TILE_BYTES + c * C::BOX_BYTES, &tmV, &full[s], c * 64, it.kvh, row);
    }
  };
  // nb 16-row blocks (1, 2 or 4): consumer warp w works on block w % nb and on
  // every (4 / nb)-th 16-key part of a tile from part w / nb on.
  const int G = a.H / a.Hk;
  const int nb = it.rows <= 16 ? 1 : (it.rows <= 32 ? 2 : 4);
  const int blk = warp % nb, part0 = warp / nb, step = C::CWARPS / nb;
  // Flattened query row (b * H + h) of the block's row r, or -1.
  auto q_index = [&](int r) {
    const int row = it.row0 + r;
    return r < it.rows ? static_cast<long long>(it.seq0 + row / G) * a.H + it.kvh * G + row % G : -1LL;
  };
  const int gr = lane >> 2, gc = (lane & 3) * 2;  // this lane's rows gr, gr + 8 and columns gc, gc + 1
  uint32_t qf[D / 16][4];
  if (warp == C::CWARPS) {
    if (lane == 0) {
      for (int s = 0; s < C::STAGES; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&empty[s], C::CWARPS);
      }
      *abort_flag = 0;
      fence_mbar_init();
      if (!g_test_drop_loads) issue(0, it.phys);  // the first copy overlaps the rest of the set-up
    }
  } else {
    const long long r0 = q_index(blk * 16 + gr), r1 = q_index(blk * 16 + gr + 8);
    const uint16_t* q = static_cast<const uint16_t*>(a.q);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const int c = kk * 16 + gc;
      qf[kk][0] = r0 < 0 ? 0u : *reinterpret_cast<const uint32_t*>(q + r0 * D + c);
      qf[kk][1] = r1 < 0 ? 0u : *reinterpret_cast<const uint32_t*>(q + r1 * D + c);
      qf[kk][2] = r0 < 0 ? 0u : *reinterpret_cast<const uint32_t*>(q + r0 * D + c + 8);
      qf[kk][3] = r1 < 0 ? 0u : *reinterpret_cast<const uint32_t*>(q + r1 * D + c + 8);
    }
  }
  __syncthreads();

  if (warp == C::CWARPS) {
    // ------------------------------------------------------------ TMA warp
    if (lane == 0 && !g_test_drop_loads) {
      int issued = 1;
      for (int t = 1; t < ntiles; ++t) {
        const int phys = it.table[(it.c0 + t * C::TK) / a.block_size];
        if (t >= C::STAGES && !mbar_wait(&empty[t % C::STAGES], (t / C::STAGES - 1) & 1, abort_flag)) break;
        issue(t, phys);
        ++issued;
      }
      // Do not leave with copies in flight (matters only after an abort, when
      // the consumers stopped waiting; every issued copy lands).
      for (int t = max(0, issued - C::STAGES); t < issued; ++t)
        mbar_wait_drain(&full[t % C::STAGES], (t / C::STAGES) & 1);
    }
    return;
  }

  // -------------------------------------------------------- consumer warps
  float o[D / 8][4];
#pragma unroll
  for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  // ldmatrix rows and 16-byte units of this lane: K as [key][dim] (two key
  // halves of a part, two units), V transposed (two key halves, two units).
  const int krow = (lane & 7) + ((lane >> 4) << 3), kunit = (lane >> 3) & 1;
  const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vunit = lane >> 4;
  for (int t = 0; t < ntiles; ++t) {
    const int s = t % C::STAGES;
    if (!__all_sync(0xffffffffu, mbar_wait(&full[s], (t / C::STAGES) & 1, abort_flag))) break;
    uint8_t* st = smem + s * C::STAGE_BYTES;
    const uint32_t kt = smem_u32(st), vt = kt + C::TILE_BYTES;
    const int left = it.c1 - (it.c0 + t * C::TK);  // keys of the range from the tile's first on
    for (int part = part0; part < C::TK / 16 && part * 16 < left; part += step) {
      const int k0 = part * 16;
      float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t b[4];
        ldsm4(kt + unit_off(k0 + krow, kk * 2 + kunit), b);
        mma16816(sc[0], qf[kk], b[0], b[1]);
        mma16816(sc[1], qf[kk], b[2], b[3]);
      }
      if (k0 + 16 > left) {
        // Keys past the range: their V rows are zeroed (their P is 0, but what
        // the page holds there may be NaN), their logits are -inf.
        for (int e = lane; e < (k0 + 16 - left) * (D / 8); e += 32) {
          const int r = left + e / (D / 8), u = e % (D / 8);
          *reinterpret_cast<uint4*>(st + C::TILE_BYTES + unit_off(r, u)) = make_uint4(0u, 0u, 0u, 0u);
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (k0 + h * 8 + gc + (i & 1) >= left) sc[h][i] = -INFINITY;
        }
      }
      // Online softmax of rows gr (i = 0) and gr + 8 (i = 1), logits in base 2.
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = fmaxf(fmaxf(sc[0][2 * i], sc[0][2 * i + 1]), fmaxf(sc[1][2 * i], sc[1][2 * i + 1])) * a.scale_log2;
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        if (__any_sync(0xffffffffu, mx > m[i])) {
          const float mn = fmaxf(m[i], mx);
          const float alpha = mn == -INFINITY ? 1.f : ex2(m[i] - mn);
          m[i] = mn;
          l[i] *= alpha;
#pragma unroll
          for (int j = 0; j < D / 8; ++j) o[j][2 * i] *= alpha, o[j][2 * i + 1] *= alpha;
        }
        const float neg = m[i] == -INFINITY ? 0.f : -m[i];
        float p[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          p[k] = ex2(fmaf(sc[k >> 1][2 * i + (k & 1)], a.scale_log2, neg));
          l[i] += p[k];
        }
        split_bf16(p[0], p[1], hi[i], lo[i]);
        split_bf16(p[2], p[3], hi[2 + i], lo[2 + i]);
      }
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        uint32_t b[4];
        ldsm4_t(vt + unit_off(k0 + vrow, j * 2 + vunit), b);
        mma16816(o[2 * j], hi, b[0], b[1]);
        mma16816(o[2 * j], lo, b[0], b[1]);
        mma16816(o[2 * j + 1], hi, b[2], b[3]);
        mma16816(o[2 * j + 1], lo, b[2], b[3]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
  }
  // Join the warps of each block: every consumer is past its last tile, so the
  // stage memory (all copies landed) is free for the partial results.
  named_bar_sync(1, C::CWARPS * 32);
  float* red_o = reinterpret_cast<float*>(smem);       // [warp][16][D]
  float* red_ml = red_o + C::CWARPS * 16 * D;          // [warp][16][2]
#pragma unroll
  for (int j = 0; j < D / 8; ++j) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<float2*>(&red_o[(warp * 16 + gr + 8 * i) * D + j * 8 + gc]) =
          make_float2(o[j][2 * i], o[j][2 * i + 1]);
  }
  if ((lane & 3) == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      red_ml[(warp * 16 + gr + 8 * i) * 2] = m[i];
      red_ml[(warp * 16 + gr + 8 * i) * 2 + 1] = l[i];
    }
  }
  named_bar_sync(1, C::CWARPS * 32);
  const int nparts = a.prefix_splits + a.seq_splits;
  for (int r = threadIdx.x / (D / 4); r < it.rows; r += C::CWARPS * 32 / (D / 4)) {
    const int c = threadIdx.x % (D / 4) * 4, b = r >> 4;
    float M = -INFINITY;
    for (int w = b; w < C::CWARPS; w += nb) M = fmaxf(M, red_ml[(w * 16 + (r & 15)) * 2]);
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = b; w < C::CWARPS; w += nb) {
      const float mw = red_ml[(w * 16 + (r & 15)) * 2], lw = red_ml[(w * 16 + (r & 15)) * 2 + 1];
      if (lw == 0.f) continue;  // no keys (NaN logits alone leave mw at -inf, too, but make lw NaN)
      const float f = ex2(mw - M);
      const float4 x = *reinterpret_cast<const float4*>(&red_o[(w * 16 + (r & 15)) * D + c]);
      sum = fmaf(lw, f, sum);
      acc.x = fmaf(x.x, f, acc.x), acc.y = fmaf(x.y, f, acc.y);
      acc.z = fmaf(x.z, f, acc.z), acc.w = fmaf(x.w, f, acc.w);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const size_t at = static_cast<size_t>(q_index(r)) * nparts + it.slot;
    *reinterpret_cast<float4*>(a.part_o + at * D + c) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (c == 0) a.part_lse[at] = sum == 0.f ? -INFINITY : M + log2f(sum);
  }
  if (waits) griddep_wait();
}

// Joins the parts of each row (sequence, head), prefix splits before own
// splits: O = sum of 2^(lse_i - M) O_i over the sum of the weights. One CTA
// per row: its four warps take every fourth part, then sum theirs in shared
// memory. How many parts there are follows from the lengths and is worked out
// before the wait for the kernels that write them (this one is launched
// programmatically); after it there are two dependent reads, the sums and the
// parts. (One warp per row, part after part: 14 us for 64 rows of 20 parts.)
template <int D>
__global__ void __launch_bounds__(128) fa_decode_shared_join_kernel(const SharedArgs a) {
  constexpr int CPL = D / 32;  // columns per lane
  __shared__ float red[4][D + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x / a.H;
  // The prefix of sequence b: the last p with cu_seqs[p] <= b.
  int lo = 0, hi = a.P;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (a.cu_seqs[mid] <= b) lo = mid + 1;
    else hi = mid;
  }
  int Lp = 0;
  if (lo > 0) {
    int first, n;
    prefix_seqs(a, lo - 1, first, n);
    if (b >= first && b < first + n) Lp = min(max(a.prefix_lens[lo - 1], 0), a.max_prefix_len);
  }
  const int L = min(max(a.seq_lens[b], 0), a.max_seq_len);
  const int np = (Lp + a.prefix_chunk - 1) / a.prefix_chunk;
  const int n = np + (L + a.seq_chunk - 1) / a.seq_chunk;
  const size_t at0 = static_cast<size_t>(blockIdx.x) * (a.prefix_splits + a.seq_splits);
  auto part = [&](int i) { return at0 + (i < np ? i : a.prefix_splits + i - np); };
  griddep_wait();
  float M = -INFINITY;
  for (int i = lane; i < n; i += 32) M = max_nan(M, a.part_lse[part(i)]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, off));
  float sum = 0.f, acc[CPL];
#pragma unroll
  for (int k = 0; k < CPL; ++k) acc[k] = 0.f;
  for (int i0 = 0; i0 < n && M != -INFINITY; i0 += 128) {
    // This warp's parts i0 + warp + 4 j, j < 32: lane j holds the weight of the j-th.
    const int mine = i0 + warp + 4 * lane;
    const float w = mine < n ? ex2(a.part_lse[part(mine)] - M) : 0.f;
    const int count = min(32, (n - i0 - warp + 3) / 4);
#pragma unroll 8
    for (int j = 0; j < count; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const float* src = a.part_o + part(i0 + warp + 4 * j) * D + lane * CPL;
      sum += wj;
      if constexpr (CPL == 4) {
        const float4 x = *reinterpret_cast<const float4*>(src);
        acc[0] = fmaf(wj, x.x, acc[0]), acc[1] = fmaf(wj, x.y, acc[1]);
        acc[2] = fmaf(wj, x.z, acc[2]), acc[3] = fmaf(wj, x.w, acc[3]);
      } else {
        const float2 x = *reinterpret_cast<const float2*>(src);
        acc[0] = fmaf(wj, x.x, acc[0]), acc[1] = fmaf(wj, x.y, acc[1]);
      }
    }
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
  uint16_t* row = static_cast<uint16_t*>(a.o) + static_cast<size_t>(blockIdx.x) * D;
  uint32_t* out = reinterpret_cast<uint32_t*>(row + lane * CPL);
#pragma unroll
  for (int k = 0; k < CPL; k += 2) out[k / 2] = pack_bf16x2(acc[k] * inv, acc[k + 1] * inv);
  if (lane == 0) a.lse[blockIdx.x] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
}

template <int D>
static cudaError_t launch_shared_t(const CUtensorMap& tk, const CUtensorMap& tv, const SharedArgs& args,
                                   cudaStream_t stream, const LaunchMarks* marks) {
  using C = SharedCfg<D>;
  SharedArgs a = args;
  auto kern = fa_decode_shared_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const long long items = (a.prefix_tiles ? 0 : static_cast<long long>(a.P) * a.Hk * a.prefix_splits) +
                          static_cast<long long>(a.B) * a.Hk * a.seq_blocks * a.seq_splits;
  const long long rows = static_cast<long long>(a.B) * a.H;
  if (items > 0x7fffffffLL || rows > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  mark(marks, true, 0, stream);
  e = launch_maybe_pdl(kern, dim3(static_cast<unsigned>(items)), dim3(C::THREADS), C::SMEM_BYTES, stream,
                       a.prefix_tiles && marks == nullptr, tk, tv, a);
  mark(marks, false, 0, stream);
  if (e != cudaSuccess) return e;
  mark(marks, true, 1, stream);
  e = launch_maybe_pdl(fa_decode_shared_join_kernel<D>, dim3(static_cast<unsigned>(rows)), dim3(128), 0,
                       stream, marks == nullptr, a);
  mark(marks, false, 1, stream);
  return e;
}

cudaError_t launch_decode_shared(const CUtensorMap& tk, const CUtensorMap& tv, const SharedArgs& a,
                                 cudaStream_t stream, const LaunchMarks* m) {
  return a.D == 64 ? launch_shared_t<64>(tk, tv, a, stream, m) : launch_shared_t<128>(tk, tv, a, stream, m);
}

cudaError_t set_decode_shared_test_hooks(unsigned long long wait_limit_ns, int drop_loads, cudaStream_t stream) {
  return set_test_hooks_here(wait_limit_ns, drop_loads, stream);
}

int take_decode_shared_status() { return take_status_here(); }

}  // namespace fa
