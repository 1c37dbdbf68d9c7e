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
// is read once and written once. d/8 lanes own a row, 16 bytes each; the sums
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

__device__ __forceinline__ void words(const uint4& v, uint32_t (&w)[4]) { w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w; }

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

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

// One unit per group of d/8 lanes; rows in batches of B so that B loads are in
// flight per lane.
template <int D, bool INTER, int B>
__global__ void __launch_bounds__(256) fa_norm_rope_kernel(const NormRopeArgs a) {
  constexpr int LPR = D / 8;
  const int lane = threadIdx.x & 31, l = lane % LPR;
  const long long u = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / LPR;
  // Groups past the last unit stay for the shuffles of their warp with no rows.
  const bool live = u < a.T * (a.q_slices + a.k_slices);
  Unit t = unit_of(a, live ? u : 0);
  if (!live) t.n = 0;
  const uint16_t* src = static_cast<const uint16_t*>(t.is_k ? a.k : a.q) +
                        t.token * (t.is_k ? a.k_stride : a.q_stride) + static_cast<long long>(t.head) * D + l * 8;
  uint16_t* dst = static_cast<uint16_t*>(t.is_k ? a.yk : a.yq) +
                  (t.token * (t.is_k ? a.Hk : a.H) + t.head) * D + l * 8;
  uint4 x[B];
  auto load = [&](int i0) {
#pragma unroll
    for (int i = 0; i < B; ++i)
      x[i] = i0 + i < t.n ? *reinterpret_cast<const uint4*>(src + static_cast<long long>(i0 + i) * D)
                          : make_uint4(0u, 0u, 0u, 0u);
  };
  load(0);
  Rotation<LPR, INTER> rot;
  rot.load(a, t.token, lane);
  {
    uint32_t w[4], wp[4];
    words(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(t.is_k ? a.wk : a.wq) + l * 8), w);
    rot.partners(w, wp);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rot.c[2 * i] *= lo_f(w[i]), rot.c[2 * i + 1] *= hi_f(w[i]);
      rot.s[2 * i] *= lo_f(wp[i]), rot.s[2 * i + 1] *= hi_f(wp[i]);
    }
  }
  for (int i0 = 0; i0 < a.rows; i0 += B) {
    if (i0 > 0) load(i0);
#pragma unroll
    for (int i = 0; i < B; ++i) {
      uint32_t w[4], p[4], y[4];
      words(x[i], w);
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
}

// Backward: a persistent grid, each group of lanes taking every n_groups-th
// unit, the q units before the k units, so that the weight gradients of both
// stay in registers; they are summed over the CTA's groups in shared memory,
// written as one partial row per CTA and added up in CTA order by the second
// kernel (a fixed order: the same bits on every run).
template <int D, bool INTER, int B>
__global__ void __launch_bounds__(256) fa_norm_rope_bwd_kernel(const NormRopeArgs a) {
  constexpr int LPR = D / 8;
  constexpr int GROUPS = 256 / LPR;
  __shared__ float red[GROUPS][2 * D];
  const int lane = threadIdx.x & 31, l = lane % LPR, grp = threadIdx.x / LPR;
  const long long n_units = a.T * (a.q_slices + a.k_slices), nq = a.T * a.q_slices;
  const long long stride = static_cast<long long>(gridDim.x) * GROUPS;
  float dw[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0.f;
  long long u0 = static_cast<long long>(blockIdx.x) * GROUPS;  // the CTA's first group: a uniform trip count
#pragma unroll
  for (int phase = 0; phase < 2; ++phase) {
    // Phase 0 takes the q units, phase 1 the k units; a step whose groups
    // straddle the two is made in both, each group idle in the other one.
    for (; u0 < (phase == 0 ? nq : n_units); u0 += stride) {
      const long long u = u0 + grp;
      const bool live = u < n_units && (u >= nq) == (phase == 1);
      Unit t = unit_of(a, live ? u : (phase == 1 ? nq : 0));
      if (!live) t.n = 0;
      const long long in = t.token * (phase ? a.k_stride : a.q_stride) + static_cast<long long>(t.head) * D + l * 8;
      const long long gin = (t.token * (phase ? a.Hk : a.H) + t.head) * D + l * 8;
      const long long out = t.token * (phase ? a.dk_stride : a.dq_stride) + static_cast<long long>(t.head) * D + l * 8;
      const uint16_t* xs = static_cast<const uint16_t*>(phase ? a.k : a.q) + in;
      const uint16_t* gs = static_cast<const uint16_t*>(phase ? a.gk : a.gq) + gin;
      uint16_t* dst = static_cast<uint16_t*>(phase ? a.yk : a.yq) + out;
      uint4 x[B], g[B];
      auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < B; ++i) {
          const bool on = i0 + i < t.n;
          x[i] = on ? *reinterpret_cast<const uint4*>(xs + static_cast<long long>(i0 + i) * D) : make_uint4(0u, 0u, 0u, 0u);
          g[i] = on ? *reinterpret_cast<const uint4*>(gs + static_cast<long long>(i0 + i) * D) : make_uint4(0u, 0u, 0u, 0u);
        }
      };
      load(0);
      Rotation<LPR, INTER> rot;
      rot.load(a, t.token, lane);
      uint32_t w[4];
      words(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(phase ? a.wk : a.wq) + l * 8), w);
      for (int i0 = 0; i0 < a.rows; i0 += B) {
        if (i0 > 0) load(i0);
#pragma unroll
        for (int i = 0; i < B; ++i) {
          uint32_t xw[4], gw[4], gp[4];
          words(x[i], xw);
          words(g[i], gw);
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
          if (on) *reinterpret_cast<uint4*>(dst + static_cast<long long>(i0 + i) * D) = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
      if (phase == 0 && u0 + GROUPS > nq) break;  // the straddling step again, for its k units
    }
  }
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

// Rows (heads) per unit: as many as a token has for long calls, where a
// group's set-up (position, table entries, weights: about as many bytes as
// four rows) is paid per unit; fewer while that leaves lanes of the GPU idle.
static int rows_per_unit(const NormRopeArgs& a, int batch) {
  constexpr long long kLanes = 152LL * 2048;
  int rows = 8;
  while (rows > batch && a.T * ((a.H + rows - 1) / rows + (a.Hk + rows - 1) / rows) * (a.D / 8) < 2 * kLanes) rows /= 2;
  return rows;
}

static void set_units(NormRopeArgs* a, int batch) {
  a->rows = rows_per_unit(*a, batch);
  a->q_slices = (a->H + a->rows - 1) / a->rows;
  a->k_slices = (a->Hk + a->rows - 1) / a->rows;
}

template <int D, bool INTER>
static cudaError_t launch_fwd_rows(NormRopeArgs a, cudaStream_t stream) {
  set_units(&a, 1);
  const long long blocks = (a.T * (a.q_slices + a.k_slices) * (D / 8) + 255) / 256;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (a.rows >= 4)
    fa_norm_rope_kernel<D, INTER, 4><<<grid, 256, 0, stream>>>(a);
  else
    fa_norm_rope_kernel<D, INTER, 1><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int D, bool INTER>
static cudaError_t launch_bwd_rows(NormRopeArgs a, cudaStream_t stream) {
  set_units(&a, 1);
  constexpr int kGroups = 256 / (D / 8);
  const long long units = a.T * (a.q_slices + a.k_slices);
  const int grid = static_cast<int>(std::min<long long>((units + kGroups - 1) / kGroups, kNormRopeMaxCtas));
  if (a.rows >= 2)
    fa_norm_rope_bwd_kernel<D, INTER, 2><<<grid, 256, 0, stream>>>(a);
  else
    fa_norm_rope_bwd_kernel<D, INTER, 1><<<grid, 256, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
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
