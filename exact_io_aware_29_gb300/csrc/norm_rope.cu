// Per-head RMS norm of queries and keys with the position rotation, forward
// and backward: what turns the projections' output into the q and k that the
// attention entry points take.
//
// Forward, per row x of d elements (one head of one token) with weight w:
//   r = rsqrt(mean(x^2) + eps),  u = r x o w,
//   y = u with each rotated pair (a, b) replaced by (a c - b s, b c + a s),
// pairs (i, i + rot/2) or, interleaved, (2i, 2i+1); c and s from the tables at
// the token's position. Written per element: y_e = r (x_e w_e c_e + x_e' w_e' s'_e)
// with e' the other member of the pair and s' = -s for a, +s for b (c = 1,
// s' = 0 past rot).
// Backward, with g = dL/dy: du_e = g_e c_e - g_e' s'_e (the rotation
// transposed), n = r x, dw = sum over rows of du o n, dn = du o w,
// dx = r (dn - n mean(dn o n)).
//
// Everything is computed in fp32 and rounded once. HBM is the bound: each row
// is read once and written once (16384 tokens, 32 + 8 heads, d 128: forward
// 55 us, 6.2 TB/s; backward 81 us, 6.3 TB/s). d/8 lanes own a row, 16 bytes each; the sums
// over a row and the exchange of half-apart pairs are shuffles (of the packed
// bf16 words: four a row, the norm and weight of the partner being known); the
// table entries times the weight stay in registers for all rows of a group.
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

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// 16 bytes global -> this thread's shared memory, asynchronously; zeros if !on.
__device__ __forceinline__ void cp_async16(uint4* dst, const uint16_t* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr int kNormRopeSlots = 4;  // batches of the backward's copies

// Where a lane's eight elements sit in the rotation: the lane holding their
// partners (its own when interleaved or past rot), and c and s' of each.
template <int LPR, bool INTER>
struct Rotation {
  int partner;  // lane of the warp
  float c[8], s[8];
  __device__ __forceinline__ void load(const NormRopeArgs& a, long long token, int lane) {
    const int l = lane % LPR, e0 = l * 8, half = a.rot / 2;
    int pos = a.positions[token];
    pos = min(max(pos, 0), a.max_pos - 1);
    partner = lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
    if (e0 >= a.rot) return;
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
  // The partners of the eight elements whose packed words are w.
  __device__ __forceinline__ void partners(const uint32_t (&w)[4], uint32_t (&p)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = INTER ? swap_halves(w[i]) : __shfl_sync(0xffffffffu, w[i], partner);
  }
};

// Unit u of the work: `rows` consecutive heads of one token, of q (the first
// nq units) or of k.
struct Unit {
  long long token;
  int head, n;
  bool is_k;
};
__device__ __forceinline__ Unit unit_of(const NormRopeArgs& a, long long u) {
  Unit t;
  const long long nq = a.T * a.q_slices;
  t.is_k = u >= nq;
  const int slices = t.is_k ? a.k_slices : a.q_slices, heads = t.is_k ? a.Hk : a.H;
  const long long v = t.is_k ? u - nq : u;
  t.token = v / slices;
  t.head = static_cast<int>(v - t.token * slices) * a.rows;
  t.n = min(a.rows, heads - t.head);
  return t;
}

}  // namespace

// A group's way through its units of one phase (0: q, 1: k), every n_groups-th
// from its own on, with the rows it will need copied ahead: NS tensors (x; x
// and the gradient), batches of B rows, SLOTS - 1 of them ahead and across
// units, into shared memory that only the copying lane reads (cp.async; no
// barrier). ring: [SLOTS][NS B][256] by thread.
template <int D, int B, int NS>
struct RowStream {
  static constexpr int LPR = D / 8, GROUPS = 256 / LPR, SLOTS = kNormRopeSlots;
  const NormRopeArgs& a;
  uint4* ring;
  const uint16_t* base[NS];
  long long tok_stride[NS];
  long long un, end, stride, nq, n_units;
  Unit tn;
  int phase, rows, i1 = 0, ahead = 0, slot = 0;
  __device__ __forceinline__ RowStream(const NormRopeArgs& args, uint4* r, int ph, long long u0)
      : a(args), ring(r), un(u0), phase(ph) {
    nq = a.T * a.q_slices;
    n_units = a.T * (a.q_slices + a.k_slices);
    end = phase == 0 ? nq : n_units;
    stride = static_cast<long long>(gridDim.x) * GROUPS;
    rows = min(a.rows, phase == 0 ? a.H : a.Hk);  // of a unit, at most
    base[0] = static_cast<const uint16_t*>(phase ? a.k : a.q);
    tok_stride[0] = phase ? a.k_stride : a.q_stride;
    if (NS == 2) {
      base[NS - 1] = static_cast<const uint16_t*>(phase ? a.gk : a.gq);
      tok_stride[NS - 1] = static_cast<long long>(phase ? a.Hk : a.H) * D;
    }
    if (un < end) tn = unit_at(un);
#pragma unroll
    for (int i = 0; i < SLOTS - 1; ++i) copy_next();
  }
  // This group's unit of the CTA's step at u0: none (n = 0) in a step that
  // straddles the phases if the unit belongs to the other one.
  __device__ __forceinline__ Unit unit_at(long long u0) const {
    const long long u = u0 + threadIdx.x / LPR;
    const bool live = u < n_units && (u >= nq) == (phase == 1);
    Unit t = unit_of(a, live ? u : (phase == 1 ? nq : 0));
    if (!live) t.n = 0;
    return t;
  }
  __device__ __forceinline__ void copy_next() {
    if (un < end) {
      uint4* dst = ring + ahead * (NS * B * 256) + threadIdx.x;
#pragma unroll
      for (int k = 0; k < NS; ++k) {
        const uint16_t* src = base[k] + tn.token * tok_stride[k] + static_cast<long long>(tn.head) * D +
                              threadIdx.x % LPR * 8;
#pragma unroll
        for (int i = 0; i < B; ++i) {
          const bool on = i1 + i < tn.n;  // a row that is not there reads as zeros
          cp_async16(dst + (k * B + i) * 256, src + (on ? static_cast<long long>(i1 + i) * D : 0), on);
        }
      }
      i1 += B;
      if (i1 >= rows) {
        i1 = 0;
        un += stride;
        if (un < end) tn = unit_at(un);
      }
    }
    cp_async_commit();  // an empty group at the end keeps the count
    ahead = (ahead + 1) % SLOTS;
  }
  // The next batch, copied three steps ago, and the copy of another one into
  // the slot that was read in the step before.
  __device__ __forceinline__ void take(uint4 (&x)[NS][B]) {
    cp_async_wait<SLOTS - 2>();
    const uint4* src = ring + slot * (NS * B * 256) + threadIdx.x;
    slot = (slot + 1) % SLOTS;
#pragma unroll
    for (int k = 0; k < NS; ++k) {
#pragma unroll
      for (int i = 0; i < B; ++i) x[k][i] = src[(k * B + i) * 256];
    }
    copy_next();
  }
};

// Forward: a persistent grid, four CTAs per SM, q units before k units (a step
// whose groups straddle the two is made in both, each group idle in the other
// one).
template <int D, bool INTER, int B>
__global__ void __launch_bounds__(256, 4) fa_norm_rope_kernel(const NormRopeArgs a) {
  constexpr int LPR = D / 8, GROUPS = 256 / LPR;
  extern __shared__ uint4 ring[];
  const int lane = threadIdx.x & 31, l = lane % LPR;
  long long u0 = static_cast<long long>(blockIdx.x) * GROUPS;
#pragma unroll
  for (int phase = 0; phase < 2; ++phase) {
    RowStream<D, B, 1> rs(a, ring, phase, u0);
    while (u0 < rs.end) {
      const Unit t = rs.unit_at(u0);
      uint16_t* dst =
          static_cast<uint16_t*>(phase ? a.yk : a.yq) + (t.token * (phase ? a.Hk : a.H) + t.head) * D + l * 8;
      Rotation<LPR, INTER> rot;
      rot.load(a, t.token, lane);
      {
        uint32_t w[4], wp[4];
        words(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(phase ? a.wk : a.wq) + l * 8), w);
        rot.partners(w, wp);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          rot.c[2 * i] *= lo_f(w[i]), rot.c[2 * i + 1] *= hi_f(w[i]);
          rot.s[2 * i] *= lo_f(wp[i]), rot.s[2 * i + 1] *= hi_f(wp[i]);
        }
      }
      for (int i0 = 0; i0 < rs.rows; i0 += B) {
        uint4 x[1][B];
        rs.take(x);
#pragma unroll
        for (int i = 0; i < B; ++i) {
          uint32_t w[4], p[4], y[4];
          words(x[0][i], w);
          rot.partners(w, p);
          float ss = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) ss = fmaf(lo_f(w[k]), lo_f(w[k]), fmaf(hi_f(w[k]), hi_f(w[k]), ss));
          const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + a.eps);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float y0 = r * fmaf(lo_f(w[k]), rot.c[2 * k], lo_f(p[k]) * rot.s[2 * k]);
            const float y1 = r * fmaf(hi_f(w[k]), rot.c[2 * k + 1], hi_f(p[k]) * rot.s[2 * k + 1]);
            y[k] = pack_bf16x2(y0, y1);
          }
          if (i0 + i < t.n)
            *reinterpret_cast<uint4*>(dst + static_cast<long long>(i0 + i) * D) = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
      if (phase == 0 && u0 + GROUPS > rs.nq) break;  // the straddling step again, for its k units
      u0 += rs.stride;
    }
    cp_async_wait<0>();
  }
}

// Backward: a persistent grid, each group of lanes taking every n_groups-th
// unit, the q units before the k units, so that the weight gradients stay in
// registers; they are summed over the CTA's groups in shared memory, written as
// one partial row per CTA and added up in CTA order by the second kernel (a
// fixed order: the same bits on every run).
// The registers admit two CTAs per SM, whose loads of one batch of rows are
// 32 KB in flight: too few for HBM (16384 tokens, 32 + 8 heads, d 128: 105 us).
// With RowStream's copies three batches ahead it is 81 us.
template <int D, bool INTER, int B>
__global__ void __launch_bounds__(256, 2) fa_norm_rope_bwd_kernel(const NormRopeArgs a) {
  constexpr int LPR = D / 8;
  constexpr int GROUPS = 256 / LPR;
  extern __shared__ uint4 ring[];
  float (*red)[2 * D] = reinterpret_cast<float (*)[2 * D]>(ring);  // [GROUPS][2 D], once the ring is done with
  const int lane = threadIdx.x & 31, l = lane % LPR, grp = threadIdx.x / LPR;
  long long u0 = static_cast<long long>(blockIdx.x) * GROUPS;  // the CTA's first group: a uniform trip count
  float dw[2][8];
#pragma unroll
  for (int phase = 0; phase < 2; ++phase) {
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[phase][i] = 0.f;
    RowStream<D, B, 2> rs(a, ring, phase, u0);
    uint32_t w[4];
    words(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(phase ? a.wk : a.wq) + l * 8), w);
    while (u0 < rs.end) {
      const Unit t = rs.unit_at(u0);
      uint16_t* dst = static_cast<uint16_t*>(phase ? a.yk : a.yq) + t.token * (phase ? a.dk_stride : a.dq_stride) +
                      static_cast<long long>(t.head) * D + l * 8;
      Rotation<LPR, INTER> rot;
      rot.load(a, t.token, lane);
      for (int i0 = 0; i0 < rs.rows; i0 += B) {
        uint4 xg[2][B];
        rs.take(xg);
#pragma unroll
        for (int i = 0; i < B; ++i) {
          uint32_t xw[4], gw[4], gp[4];
          words(xg[0][i], xw);
          words(xg[1][i], gw);
          rot.partners(gw, gp);
          float du[8], ss = 0.f, dot = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            ss = fmaf(lo_f(xw[k]), lo_f(xw[k]), fmaf(hi_f(xw[k]), hi_f(xw[k]), ss));
            du[2 * k] = fmaf(lo_f(gw[k]), rot.c[2 * k], -lo_f(gp[k]) * rot.s[2 * k]);
            du[2 * k + 1] = fmaf(hi_f(gw[k]), rot.c[2 * k + 1], -hi_f(gp[k]) * rot.s[2 * k + 1]);
            dot = fmaf(du[2 * k] * lo_f(w[k]), lo_f(xw[k]), fmaf(du[2 * k + 1] * hi_f(w[k]), hi_f(xw[k]), dot));
          }
          ss = row_sum<LPR>(ss);
          dot = row_sum<LPR>(dot);
          const float r = rsqrtf(ss * (1.f / D) + a.eps);
          const bool on = i0 + i < t.n;
          const float rw = on ? r : 0.f;              // rows that are not there add nothing to dw
          const float m = dot * (1.f / D) * r * r;  // mean(dn o n) / r * r: dx = r (dn - x m)
          uint32_t y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float x0 = lo_f(xw[k]), x1 = hi_f(xw[k]);
            dw[phase][2 * k] = fmaf(du[2 * k], x0 * rw, dw[phase][2 * k]);
            dw[phase][2 * k + 1] = fmaf(du[2 * k + 1], x1 * rw, dw[phase][2 * k + 1]);
            y[k] = pack_bf16x2(r * fmaf(-x0, m, du[2 * k] * lo_f(w[k])), r * fmaf(-x1, m, du[2 * k + 1] * hi_f(w[k])));
          }
          if (on)
            *reinterpret_cast<uint4*>(dst + static_cast<long long>(i0 + i) * D) = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
      if (phase == 0 && u0 + GROUPS > rs.nq) break;  // the straddling step again, for its k units
      u0 += rs.stride;
    }
    cp_async_wait<0>();
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    red[grp][l * 8 + i] = dw[0][i];
    red[grp][D + l * 8 + i] = dw[1][i];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * D; c += 256) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) s += red[k][c];
    a.part[static_cast<long long>(blockIdx.x) * (2 * D) + c] = s;
  }
  griddep_launch_dependents();
}

// dw of q and k (columns 0..D-1 and D..2D-1 of the partial rows): 32 columns a
// CTA, every 32nd partial row to a thread, then the 32 threads of a column.
template <int D>
__global__ void __launch_bounds__(1024) fa_norm_rope_dw_kernel(const NormRopeArgs a, int n_part) {
  __shared__ float red[32][33];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), lane = threadIdx.x >> 5;
  griddep_wait();
  float s = 0.f;
#pragma unroll 4
  for (int p = lane; p < n_part; p += 32) s += a.part[static_cast<long long>(p) * (2 * D) + col];
  red[lane][threadIdx.x & 31] = s;
  __syncthreads();
  if (lane == 0) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) s += red[k][threadIdx.x];
    (col < D ? a.dwq : a.dwk)[col < D ? col : col - D] = s;
  }
}

// Rows (heads) per unit: `most` for long calls, where a group's set-up
// (position, table entries, weights: about as many bytes as four rows) is paid
// per unit; fewer while the units' lanes are fewer than `lanes`.
static void set_units(NormRopeArgs* a, int most, long long lanes) {
  auto slices = [](int heads, int rows) { return (heads + rows - 1) / rows; };
  int rows = most;
  while (rows > 1 && a->T * (slices(a->H, rows) + slices(a->Hk, rows)) * (a->D / 8) < lanes) rows /= 2;
  a->rows = rows;
  a->q_slices = slices(a->H, rows);
  a->k_slices = slices(a->Hk, rows);
}

template <int D, bool INTER>
static cudaError_t launch_fwd_rows(NormRopeArgs a, cudaStream_t stream) {
  // Half of the persistent grid's lanes. Measured on 16384 tokens of 32 + 8
  // heads: 55.3 us with up to 8 rows, 61.0 with 16 (the last q units leave lanes
  // idle); one unit per group, not persistent: 58.7.
  set_units(&a, 8, 152LL * 1024);
  constexpr int kGroups = 256 / (D / 8);
  const long long units = a.T * (a.q_slices + a.k_slices);
  const int grid = static_cast<int>(std::min<long long>((units + kGroups - 1) / kGroups, 152 * 4));
  const int b = a.rows >= 2 ? 2 : 1;
  auto kern = b == 2 ? fa_norm_rope_kernel<D, INTER, 2> : fa_norm_rope_kernel<D, INTER, 1>;
  kern<<<grid, 256, kNormRopeSlots * b * 256 * 16, stream>>>(a);
  return cudaGetLastError();
}

template <int D, bool INTER>
static cudaError_t launch_bwd_rows(NormRopeArgs a, cudaStream_t stream) {
  // Half of the persistent grid's lanes. Measured on 16384 tokens of 32 + 8 heads: 81 us
  // with up to 16 rows, 85 with up to 8.
  set_units(&a, 16, kNormRopeMaxCtas * 128LL);
  constexpr int kGroups = 256 / (D / 8);
  const long long units = a.T * (a.q_slices + a.k_slices);
  const int grid = static_cast<int>(std::min<long long>((units + kGroups - 1) / kGroups, kNormRopeMaxCtas));
  auto kern = a.rows >= 2 ? fa_norm_rope_bwd_kernel<D, INTER, 2> : fa_norm_rope_bwd_kernel<D, INTER, 1>;
  const int smem = kNormRopeSlots * 2 * (a.rows >= 2 ? 2 : 1) * 256 * 16;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<grid, 256, smem, stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_maybe_pdl(fa_norm_rope_dw_kernel<D>, dim3(2 * D / 32), dim3(1024), 0, stream, true, a, grid);
}

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
  if (a.D == 64)
    return a.interleaved ? launch_fwd_rows<64, true>(a, stream) : launch_fwd_rows<64, false>(a, stream);
  return a.interleaved ? launch_fwd_rows<128, true>(a, stream) : launch_fwd_rows<128, false>(a, stream);
}

cudaError_t launch_norm_rope_bwd(const NormRopeArgs& a, cudaStream_t stream) {
  if (a.D == 64)
    return a.interleaved ? launch_bwd_rows<64, true>(a, stream) : launch_bwd_rows<64, false>(a, stream);
  return a.interleaved ? launch_bwd_rows<128, true>(a, stream) : launch_bwd_rows<128, false>(a, stream);
}

}  // namespace fa
