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
// the delta rule's (DecodeShape).
template <typename TIO, int DK, typename TS>
__global__ void __launch_bounds__(DecodeShape<DK, TS>::kWarps * 32)
decode_kernel(const TIO* __restrict__ q, const TIO* __restrict__ k, const TIO* __restrict__ v,
              const float* __restrict__ g, int g_stride, TS* __restrict__ state, int Hqk, int Hv, int dv,
              float scale, TIO* __restrict__ o) {
  using Sh = DecodeShape<DK, TS>;
  constexpr int E = Sh::kElems;
  constexpr int LPR = Sh::kLanesPerRow;
  const int bh = blockIdx.x;                 // b * Hv + h
  const int b = bh / Hv, h = bh - b * Hv;
  const int hq = h / (Hv / Hqk);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LPR;                // 16-byte chunk within the row
  const int slot_row = lane / LPR;           // row within a slot

  // the state rows first: their latency covers everything else
  const int row0 = blockIdx.y * Sh::kRowsPerCta + warp * Sh::kRowsPerWarp + slot_row;
  TS* S = state + (size_t)bh * dv * DK;
  float s[Sh::kSlots][E];
  float vv[Sh::kSlots];
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
// The recurrence token by token in fp32. A state row is spread over 4 lanes
// (columns 4 (sub + 4 i) .. + 3), 8 rows a warp, and stays in registers for the
// whole sequence; a block of tokens' q, k and v is staged in shared memory as
// fp32, where the 8 row groups of a warp read the same q and k words.
constexpr int kScanTokens = 32;   // tokens staged at a time
constexpr int kScanRows = 32;     // state rows per CTA: 4 warps of 8
constexpr int kScanThreads = 128;

// grid: (ceil(dv / kScanRows), Hv, n_seqs)
template <typename TIO, int DK>
__global__ void __launch_bounds__(kScanThreads)
scan_kernel(const TIO* __restrict__ q, const TIO* __restrict__ k, const TIO* __restrict__ v,
            const float* __restrict__ g, int g_stride, const float* state_in,
            const int32_t* __restrict__ cu_seqlens, int Hqk, int Hv, int dv, float scale,
            TIO* __restrict__ o, float* state_out, long long total_T) {
  constexpr int E = DK / 4;                  // columns per lane
  __shared__ __align__(16) float qs[kScanTokens][DK];
  __shared__ __align__(16) float ks[kScanTokens][DK];
  __shared__ float vs[kScanTokens][kScanRows];   // v, replaced by o
  __shared__ float as[kScanTokens];
  const int h = blockIdx.y, n = blockIdx.z, hq = h / (Hv / Hqk);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sub = lane & 3, rl = warp * 8 + (lane >> 2);
  const int i0 = blockIdx.x * kScanRows, row = i0 + rl;

  // a cu_seqlens that breaks its rules never makes a token outside [0, total_T) read
  long long t_begin = cu_seqlens[n], t_end = cu_seqlens[n + 1];
  if (t_end > total_T) t_end = total_T;
  if (t_begin < 0) t_begin = 0;
  if (t_begin > t_end) t_begin = t_end;

  const size_t srow = (((size_t)n * Hv + h) * dv + row) * DK + 4 * sub;
  float s[E];
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    const float4 x = state_in && row < dv ? *reinterpret_cast<const float4*>(state_in + srow + 16 * i)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
    s[4 * i] = x.x; s[4 * i + 1] = x.y; s[4 * i + 2] = x.z; s[4 * i + 3] = x.w;
  }

  for (long long c0 = t_begin; c0 < t_end; c0 += kScanTokens) {
    const int L = (int)min((long long)kScanTokens, t_end - c0);
    for (int e = tid; e < L * (DK / 4); e += kScanThreads) {
      const int t = e / (DK / 4), j = 4 * (e - t * (DK / 4));
      const size_t at = ((size_t)(c0 + t) * Hqk + hq) * DK + j;
      float4 x = load4(q + at);
      x.x *= scale; x.y *= scale; x.z *= scale; x.w *= scale;
      *reinterpret_cast<float4*>(&qs[t][j]) = x;
      *reinterpret_cast<float4*>(&ks[t][j]) = load4(k + at);
    }
    for (int e = tid; e < L * kScanRows; e += kScanThreads) {
      const int t = e / kScanRows, i = e - t * kScanRows;
      vs[t][i] = i0 + i < dv ? to_f32(v[((size_t)(c0 + t) * Hv + h) * dv + i0 + i]) : 0.f;
    }
    if (tid < L) as[tid] = expf(g[(size_t)(c0 + tid) * g_stride + h]);
    __syncthreads();
    for (int t = 0; t < L; ++t) {
      const float a = as[t], vi = vs[t][rl];
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const float4 kk = *reinterpret_cast<const float4*>(&ks[t][4 * (sub + 4 * i)]);
        const float4 qq = *reinterpret_cast<const float4*>(&qs[t][4 * (sub + 4 * i)]);
        s[4 * i] = fmaf(a, s[4 * i], vi * kk.x);
        s[4 * i + 1] = fmaf(a, s[4 * i + 1], vi * kk.y);
        s[4 * i + 2] = fmaf(a, s[4 * i + 2], vi * kk.z);
        s[4 * i + 3] = fmaf(a, s[4 * i + 3], vi * kk.w);
        acc[0] = fmaf(s[4 * i], qq.x, acc[0]);
        acc[1] = fmaf(s[4 * i + 1], qq.y, acc[1]);
        acc[2] = fmaf(s[4 * i + 2], qq.z, acc[2]);
        acc[3] = fmaf(s[4 * i + 3], qq.w, acc[3]);
      }
      const float r = group_sum<4>((acc[0] + acc[1]) + (acc[2] + acc[3]));
      if (sub == 0) vs[t][rl] = r;           // only this row's lanes read v_t[row], and they have
    }
    __syncthreads();
    for (int e = tid; e < L * kScanRows; e += kScanThreads) {
      const int t = e / kScanRows, i = e - t * kScanRows;
      if (i0 + i < dv) o[((size_t)(c0 + t) * Hv + h) * dv + i0 + i] = from_f32<TIO>(vs[t][i]);
    }
    __syncthreads();
  }
  if (row < dv) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i)
      *reinterpret_cast<float4*>(state_out + srow + 16 * i) =
          make_float4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
  }
}

}  // namespace lin
}  // namespace gdn
