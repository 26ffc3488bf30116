// Decayed linear attention: the state recurrence without the delta term,
//
//   S_t = alpha_t S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t,   alpha_t = exp(g_t)
//
// with q and k used as given (no normalisation), states [Hv, dv, dk] as the gated
// delta rule's, and g either one log-decay per token and value head or one fixed
// per value head (token stride 0).
#pragma once

#include "common.cuh"
#include "decode.cuh"

namespace gdn {
namespace lin {

// ---------------------------------------------------------------- decode ---
// One token per sequence, the state updated in place. As in the delta rule's
// decode every state row is read and written once: with the old row S_i,
//
//   S'_i = alpha S_i + v_i k,    o_i = alpha (S_i . q) + v_i (k . q)
//
// and the step is bound by the bytes of the state. Layout and rows per warp are
// the delta rule's (DecodeShape), but 8 bf16 rows per warp (131 sequences x 32 heads: 49.3
// us a step against 53.4 with 16 and 56.5 with 4; keeping them packed until their turn
// 53.4). CTAs are numbered along the state in memory: with the heads as the grid's fast
// dimension, neighbours 64 KB apart, the fp32 step at 64 sequences x 32 heads took 50.7 us
// instead of 43.2. Warps per CTA (2 to 8) and fp32 rows per warp (2 to 16) make no
// difference then.
constexpr int kDecodeWarps = 4;

template <int DK, typename TS>
struct LinearDecodeShape {
  static constexpr int kRowsPerSlot = DecodeShape<DK, TS>::kRowsPerSlot;
  static constexpr int kRows = sizeof(TS) == 4 ? 4 : 8;
  static constexpr int kSlots = kRows / kRowsPerSlot > 0 ? kRows / kRowsPerSlot : 1;
  static constexpr int kRowsPerWarp = kRowsPerSlot * kSlots;
  static constexpr int kRowsPerCta = kRowsPerWarp * kDecodeWarps;
};

// grid: B * Hv * parts, parts = ceil(dv / rows per CTA)
template <typename TIO, int DK, typename TS>
__global__ void __launch_bounds__(kDecodeWarps * 32)
decode_kernel(const TIO* __restrict__ q, const TIO* __restrict__ k, const TIO* __restrict__ v,
              const float* __restrict__ g, int g_stride, TS* __restrict__ state, int Hqk, int Hv, int dv, int parts,
              float scale, TIO* __restrict__ o) {
  using Sh = LinearDecodeShape<DK, TS>;
  constexpr int E = DecodeShape<DK, TS>::kElems;
  constexpr int LPR = DecodeShape<DK, TS>::kLanesPerRow;
  const int bh = blockIdx.x / parts, part = blockIdx.x - bh * parts;   // bh = b * Hv + h
  const int b = bh / Hv, h = bh - b * Hv;
  const int hq = h / (Hv / Hqk);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LPR;                // 16-byte chunk within the row
  const int slot_row = lane / LPR;           // row within a slot

  // the state rows first: their latency covers everything else
  const int row0 = (part * kDecodeWarps + warp) * Sh::kRowsPerWarp + slot_row;
  TS* S = state + (size_t)bh * dv * DK;
  float s[Sh::kSlots][E], vv[Sh::kSlots];
#pragma unroll
  for (int j = 0; j < Sh::kSlots; ++j) {
    const int r = row0 + j * Sh::kRowsPerSlot;
    if (r < dv) {
      StateChunk<TS>::load(S + (size_t)r * DK + E * sub, s[j]);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) s[j][e] = 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < Sh::kSlots; ++j) {
    const int r = row0 + j * Sh::kRowsPerSlot;
    vv[j] = r < dv ? to_f32(v[(size_t)bh * dv + r]) : 0.f;
  }
  const float alpha = expf(g[(size_t)b * g_stride + h]);

  const size_t qk_off = ((size_t)b * Hqk + hq) * DK + E * sub;
  float kf[E], qf[E];
  load_vec<E>(k + qk_off, kf);
  load_vec<E>(q + qk_off, qf);
  float kq = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qf[e] *= scale;
    kq = fmaf(kf[e], qf[e], kq);
  }
  kq = group_sum<LPR>(kq);

#pragma unroll
  for (int j = 0; j < Sh::kSlots; ++j) {
    float sq = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) sq = fmaf(s[j][e], qf[e], sq);
    sq = group_sum<LPR>(sq);
    const int r = row0 + j * Sh::kRowsPerSlot;
    if (r < dv) {
      float ns[E];
#pragma unroll
      for (int e = 0; e < E; ++e) ns[e] = fmaf(alpha, s[j][e], vv[j] * kf[e]);
      StateChunk<TS>::store(S + (size_t)r * DK + E * sub, ns);
      if (sub == 0) o[(size_t)bh * dv + r] = from_f32<TIO>(fmaf(alpha, sq, vv[j] * kq));
    }
  }
}

// --------------------------------------------------------------- prefill ---
// The recurrence token by token in fp32, for fp32 inputs (the tensor cores' products
// would round them). A state row is spread over 4 lanes (columns 4 (sub + 4 i) .. + 3), 8
// rows a warp, and stays in registers; a block of 16 tokens' q, k and v is staged in
// shared memory, where the 8 row groups of a warp read the same q and k words. Issue
// bound: three operations a state element and token, two in the first pass.
//
// Over time. Heads and rows alone give few warps, each with one long chain, so sequences
// are cut into segments of `seg` tokens, all worked on at once, in three launches: each
// segment's state from zero (kOut = false), the states that enter the segments (and the
// final ones) as the running combination of those, and the outputs from them.
//
// Precision. exp(g_t) rounded once is off by up to 2^-24, always the same way where the
// decay is fixed, which a thousand tokens add up to 6e-5. So the decays that are carried
// far are exact: across segments exp of the sum of g in fp64, and inside one the state
// is corrected after every block of 16 tokens by exp of the block's sum over the product
// of the rounded decays.
constexpr int kScanTokens = 16;   // tokens staged at a time
constexpr int kScanRows = 32;     // state rows per CTA: 4 warps of 8
constexpr int kScanThreads = 128;

struct ScanParams {
  const float* g;
  const float* state_in;
  const int32_t* cu_seqlens;
  float* state_out;
  float* states;       // [segments][Hv][dv][dk]: each segment's own state, then the one that enters it
  float* decays;       // [segments][Hv]
  int g_stride, n_seqs, total_T, Hqk, Hv, dv, seg;
  int segments;        // that the workspace has room for
  float scale;
};

// Segment `item` of the packed sequences (one at least for each): its sequence, number in
// it, their count and its tokens; false behind the last. By a whole warp.
struct Segment {
  int n, j, J, t0, len;
};
__device__ __forceinline__ bool find_segment(const ScanParams& p, int item, Segment& it) {
  const int lane = threadIdx.x & 31;
  for (int n = 0, base = 0; n < p.n_seqs; n += 32) {
    int a = 0, len = 0, J = 0;
    if (n + lane < p.n_seqs) {
      // a cu_seqlens that breaks its rules never makes a token outside [0, total_T) read
      a = min(max(p.cu_seqlens[n + lane], 0), p.total_T);
      len = max(min(max(p.cu_seqlens[n + lane + 1], 0), p.total_T) - a, 0);
      J = max(1, (len + p.seg - 1) / p.seg);
    }
    int incl = J;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += x;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, base + incl > item);
    if (hit) {
      const int src = __ffs(hit) - 1;
      it.n = n + src;
      it.J = __shfl_sync(0xffffffffu, J, src);
      it.j = item - base - __shfl_sync(0xffffffffu, incl - J, src);
      it.t0 = __shfl_sync(0xffffffffu, a, src) + it.j * p.seg;
      it.len = min(p.seg, __shfl_sync(0xffffffffu, len, src) - it.j * p.seg);
      return true;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// grid: (segments at most, Hv, ceil(dv / kScanRows))
template <typename TIO, int DK, bool kOut>
__global__ void __launch_bounds__(kScanThreads)
scan_kernel(const TIO* __restrict__ q, const TIO* __restrict__ k, const TIO* __restrict__ v, TIO* __restrict__ o,
            const ScanParams p) {
  constexpr int E = DK / 4;                  // columns per lane
  __shared__ __align__(16) float qs[kOut ? kScanTokens : 1][DK];
  __shared__ __align__(16) float ks[kScanTokens][DK];
  __shared__ float vs[kScanTokens][kScanRows];   // v, replaced by o
  __shared__ float as[kScanTokens];
  __shared__ float fix;
  const int h = blockIdx.y, hq = h / (p.Hv / p.Hqk), dv = p.dv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sub = lane & 3, rl = warp * 8 + (lane >> 2);
  const int i0 = blockIdx.z * kScanRows, row = i0 + rl;
  Segment it;
  if (!find_segment(p, blockIdx.x, it)) return;
  if (!kOut && it.J == 1) return;            // nothing to combine

  const size_t slot = (((size_t)blockIdx.x * p.Hv + h) * dv + row) * DK + 4 * sub;
  const size_t srow = (((size_t)it.n * p.Hv + h) * dv + row) * DK + 4 * sub;
  const float* from = !kOut ? nullptr : it.J > 1 ? p.states + slot : p.state_in ? p.state_in + srow : nullptr;
  float s[E];
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    const float4 x = from && row < dv ? *reinterpret_cast<const float4*>(from + 16 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
    s[4 * i] = x.x; s[4 * i + 1] = x.y; s[4 * i + 2] = x.z; s[4 * i + 3] = x.w;
  }

  double sum = 0.0;                          // of the segment's g (warp 0)
  for (int c0 = 0; c0 < it.len; c0 += kScanTokens) {
    const int L = min(kScanTokens, it.len - c0), t0 = it.t0 + c0;
    for (int e = tid; e < L * (DK / 4); e += kScanThreads) {
      const int t = e / (DK / 4), j = 4 * (e - t * (DK / 4));
      const size_t at = ((size_t)(t0 + t) * p.Hqk + hq) * DK + j;
      if constexpr (kOut) {
        float4 x = load4(q + at);
        x.x *= p.scale; x.y *= p.scale; x.z *= p.scale; x.w *= p.scale;
        *reinterpret_cast<float4*>(&qs[t][j]) = x;
      }
      *reinterpret_cast<float4*>(&ks[t][j]) = load4(k + at);
    }
    for (int e = tid; e < L * kScanRows; e += kScanThreads) {
      const int t = e / kScanRows, i = e - t * kScanRows;
      vs[t][i] = i0 + i < dv ? to_f32(v[((size_t)(t0 + t) * p.Hv + h) * dv + i0 + i]) : 0.f;
    }
    if (warp == 0) {
      const float g = lane < L ? p.g[(size_t)(t0 + lane) * p.g_stride + h] : 0.f;
      const float a = expf(g);
      if (lane < L) as[lane] = a;
      double gs = g, prod = lane < L ? (double)a : 1.0;
#pragma unroll
      for (int off = kScanTokens / 2; off > 0; off >>= 1) {
        gs += __shfl_xor_sync(0xffffffffu, gs, off);
        prod *= __shfl_xor_sync(0xffffffffu, prod, off);
      }
      sum += gs;
      if (lane == 0) fix = prod > 1e-30 ? (float)(exp(gs) / prod) : 1.f;   // (below, nothing is left to correct)
    }
    __syncthreads();
    for (int t = 0; t < L; ++t) {
      const float a = as[t], vi = vs[t][rl];
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const float4 kk = *reinterpret_cast<const float4*>(&ks[t][4 * (sub + 4 * i)]);
        s[4 * i] = fmaf(a, s[4 * i], vi * kk.x);
        s[4 * i + 1] = fmaf(a, s[4 * i + 1], vi * kk.y);
        s[4 * i + 2] = fmaf(a, s[4 * i + 2], vi * kk.z);
        s[4 * i + 3] = fmaf(a, s[4 * i + 3], vi * kk.w);
        if constexpr (kOut) {
          const float4 qq = *reinterpret_cast<const float4*>(&qs[t][4 * (sub + 4 * i)]);
          acc[0] = fmaf(s[4 * i], qq.x, acc[0]);
          acc[1] = fmaf(s[4 * i + 1], qq.y, acc[1]);
          acc[2] = fmaf(s[4 * i + 2], qq.z, acc[2]);
          acc[3] = fmaf(s[4 * i + 3], qq.w, acc[3]);
        }
      }
      if constexpr (kOut) {
        const float r = group_sum<4>((acc[0] + acc[1]) + (acc[2] + acc[3]));
        if (sub == 0) vs[t][rl] = r;         // only this row's lanes read v_t[row], and they have
      }
    }
    const float f = fix;
#pragma unroll
    for (int i = 0; i < E; ++i) s[i] *= f;
    __syncthreads();
    if constexpr (kOut) {
      for (int e = tid; e < L * kScanRows; e += kScanThreads) {
        const int t = e / kScanRows, i = e - t * kScanRows;
        if (i0 + i < dv) o[((size_t)(t0 + t) * p.Hv + h) * dv + i0 + i] = from_f32<TIO>(vs[t][i]);
      }
      __syncthreads();
    }
  }
  float* to = !kOut ? p.states + slot : it.J == 1 ? p.state_out + srow : nullptr;
  if (to && row < dv) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i)
      *reinterpret_cast<float4*>(to + 16 * i) = make_float4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
  }
  if (!kOut && i0 == 0 && tid == 0) p.decays[(size_t)blockIdx.x * p.Hv + h] = (float)exp(sum);
}

// The states that enter the segments, in place of the segments' own, and the final ones.
// grid: (ceil(dv dk / 1024), Hv, n_seqs); 256 threads of 4 values. Bound by the bytes of the
// states; four segments' loads are in flight at a time.
__global__ void __launch_bounds__(256)
combine_kernel(const ScanParams p, int per_state) {
  const int h = blockIdx.y, n = blockIdx.z, at = (blockIdx.x * 256 + threadIdx.x) * 4, lane = threadIdx.x & 31;
  // the sequence's first segment: those of the sequences before it
  long long first = 0;
  int J = 0;
  for (int m = 0; m <= n; m += 32) {
    int x = 0;
    if (m + lane <= n) {
      const int a = min(max(p.cu_seqlens[m + lane], 0), p.total_T);
      const int len = max(min(max(p.cu_seqlens[m + lane + 1], 0), p.total_T) - a, 0);
      x = max(1, (len + p.seg - 1) / p.seg);
      if (m + lane == n) J = x;
    }
    first += __reduce_add_sync(0xffffffffu, x);
  }
  J = __reduce_max_sync(0xffffffffu, J);
  first -= J;
  if (J == 1 || at >= per_state) return;
  if (first + J > p.segments) return;   // (sequences that overlap, which no valid cu_seqlens makes)
  const size_t own = ((size_t)n * p.Hv + h) * per_state + at, step = (size_t)p.Hv * per_state;
  float* slot = p.states + ((size_t)first * p.Hv + h) * per_state + at;
  const float* decay = p.decays + (size_t)first * p.Hv + h;
  float4 s = p.state_in ? *reinterpret_cast<const float4*>(p.state_in + own) : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = 0; j < J; j += 4) {
    float4 x[4];
    float a[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (j + u < J) {
        x[u] = *reinterpret_cast<const float4*>(slot + (j + u) * step);
        a[u] = decay[(size_t)(j + u) * p.Hv];
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (j + u < J) {
        *reinterpret_cast<float4*>(slot + (j + u) * step) = s;
        s.x = fmaf(a[u], s.x, x[u].x);
        s.y = fmaf(a[u], s.y, x[u].y);
        s.z = fmaf(a[u], s.z, x[u].z);
        s.w = fmaf(a[u], s.w, x[u].w);
      }
    }
  }
  *reinterpret_cast<float4*>(p.state_out + own) = s;
}

}  // namespace lin
}  // namespace gdn
