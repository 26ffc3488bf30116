// Decayed linear attention: the state recurrence without the delta term,
//
//   S_t = alpha_t S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t,   alpha_t = exp(g_t)
//
// with q and k used as given (no normalisation), states [Hv, dv, dk] as the gated
// delta rule's, and g either one log-decay per token and value head or one fixed
// per value head (token stride 0).
#pragma once

#include <type_traits>

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
// rows a warp, and stays in registers; blocks of 16 tokens' q, k and v are staged in
// shared memory, one ahead, where the 8 row groups of a warp read the same q and k words.
// Those reads are what bounds it, before the arithmetic (three operations a state element
// and token where o is made, one in the first pass), so a lane holds two rows where d_v
// has them: one 4096-token sequence of 16 heads of 128 takes 307 us, 32 packed heads of
// 16 x 300 tokens 430 us; with one row a lane and no stage ahead 477 and 1218. (Exact decays
// cost the case of two sequences of 500 to 2000 tokens, 16 heads of 64, 3 us of 88.)
//
// Over time. Heads and rows alone give few warps, each with one long chain, so sequences
// are cut into segments of `seg` tokens, all worked on at once, in three launches: each
// segment's state from zero (kOut = false), the states that enter the segments (and the
// final ones) as the running combination of those, and the outputs from them.
//
// Precision. exp(g_t) rounded once is off by up to 2^-24, always the same way where the
// decay is fixed, which a thousand tokens add up to 6e-5. So decays are sums of g in fp64:
// in the first pass a token enters with the weight it has at the end of its block of 16
// tokens, and the state decays a block at a time; where o is made the decay of a block's last
// token is exp of the block's sum over the product of the other rounded decays. What rounding
// such a factor to fp32 loses goes into the next block's, so that the product of any number
// of them is off by 2^-23 at most, and a segment's decay is held in two floats. A factor is
// applied in the fma that adds a token: alone, s (1 - 2^-24) would always round the same way,
// by a whole step. What is left is the rounding of the state itself, at random: 2^-25 sqrt(T)
// relative.
constexpr int kScanTokens = 16;   // tokens staged at a time
constexpr int kScanThreads = 128;
// State rows per lane, and of a CTA of 4 warps.
__host__ __device__ constexpr int scan_rows_per_lane(int dv) { return dv >= 64 ? 2 : 1; }
__host__ __device__ constexpr int scan_rows(int dv) { return 32 * scan_rows_per_lane(dv); }

// 16 bytes to shared memory, of which the first `bytes` are read and the others zeros.
__device__ __forceinline__ void copy16_async(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_all;" ::: "memory"); }

struct ScanParams {
  const float* g;
  const float* state_in;
  const int32_t* cu_seqlens;
  float* state_out;
  float* states;       // [segments][Hv][dv][dk]: each segment's own state, then the one that enters it
  float2* decays;      // [segments][Hv]: exp of the segment's sum of g, in two parts
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

// grid: (segments at most, Hv, ceil(dv / (32 kR)))
template <int DK, int kR, bool kOut>
__global__ void __launch_bounds__(kScanThreads)
scan_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v, float* __restrict__ o,
            const ScanParams p) {
  constexpr int E = DK / 4;                  // columns per lane
  constexpr int kScanRows = 32 * kR;
  // two stages: the next one's tokens arrive while this one's are worked on
  __shared__ __align__(16) float qs[2][kOut ? kScanTokens : 1][DK];
  __shared__ __align__(16) float ks[2][kScanTokens][DK];
  __shared__ __align__(16) float vs[2][kScanTokens][kScanRows];   // v, replaced by o
  __shared__ float as[2][kScanTokens];       // kOut: exp(g); else the weight of a token in the state behind the stage
  __shared__ float stage[2];                 // !kOut: the stage's decay
  const int h = blockIdx.y, hq = h / (p.Hv / p.Hqk), dv = p.dv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sub = lane & 3, rl = warp * 8 + (lane >> 2);
  const int i0 = blockIdx.z * kScanRows, row = i0 + rl;
  Segment it;
  if (!find_segment(p, blockIdx.x, it)) return;
  if (!GDN_CHECK(it.n < p.n_seqs && it.j >= 0 && it.j < it.J && it.t0 >= 0 && it.len >= 0 && it.t0 + it.len <= p.total_T &&
                 (int)blockIdx.x < p.segments))
    return;
  if (!kOut && it.J == 1) return;            // nothing to combine

  // row 32 u further on: u * 32 * DK words
  const size_t slot = (((size_t)blockIdx.x * p.Hv + h) * dv + row) * DK + 4 * sub;
  const size_t srow = (((size_t)it.n * p.Hv + h) * dv + row) * DK + 4 * sub;
  const float* from = !kOut ? nullptr : it.J > 1 ? p.states + slot : p.state_in ? p.state_in + srow : nullptr;
  float s[kR][E];
#pragma unroll
  for (int u = 0; u < kR; ++u) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      const float4 x = from && row + 32 * u < dv ? *reinterpret_cast<const float4*>(from + 32 * u * DK + 16 * i)
                                                 : make_float4(0.f, 0.f, 0.f, 0.f);
      s[u][4 * i] = x.x; s[u][4 * i + 1] = x.y; s[u][4 * i + 2] = x.z; s[u][4 * i + 3] = x.w;
    }
  }

  double sum = 0.0;                          // of the segment's g (warp 0)
  double rest = 1.0;                         // what the last factor lost in rounding (warp 0)
  auto fetch = [&](int c0) {
    const int L = min(kScanTokens, it.len - c0), t0 = it.t0 + c0, b = (c0 / kScanTokens) & 1;
    for (int e = tid; e < L * (DK / 4); e += kScanThreads) {
      const int t = e / (DK / 4), j = 4 * (e - t * (DK / 4));
      const size_t at = ((size_t)(t0 + t) * p.Hqk + hq) * DK + j;
      if constexpr (kOut) copy16_async(&qs[b][t][j], q + at, 16);
      copy16_async(&ks[b][t][j], k + at, 16);
    }
    for (int e = tid; e < L * (kScanRows / 4); e += kScanThreads) {
      const int t = e / (kScanRows / 4), i = 4 * (e - t * (kScanRows / 4));
      const bool in = i0 + i < dv;           // (zeros behind the last row)
      copy16_async(&vs[b][t][i], v + ((size_t)(t0 + t) * p.Hv + h) * dv + (in ? i0 + i : 0), in ? 16 : 0);
    }
  };
  // by warp 0
  auto gate = [&](int c0) {
    return lane < min(kScanTokens, it.len - c0) ? p.g[(size_t)(it.t0 + c0 + lane) * p.g_stride + h] : 0.f;
  };
  auto decays = [&](int c0, float g) {
    const int b = (c0 / kScanTokens) & 1;
    if constexpr (kOut) {
      const bool last = lane == min(kScanTokens, it.len - c0) - 1;
      const float a = expf(g);               // (1 behind the last token)
      double gs = g, prod = last ? 1.0 : a;
#pragma unroll
      for (int off = kScanTokens / 2; off > 0; off >>= 1) {
        gs += __shfl_xor_sync(0xffffffffu, gs, off);
        prod *= __shfl_xor_sync(0xffffffffu, prod, off);
      }
      const double want = rest * exp(gs) / prod;
      float got = (float)want;
      if (got > 1e-30f && got < 1e30f && prod > 1e-30) {
        rest = want / got;
      } else {                               // (nothing is left to correct)
        got = a;
        rest = 1.0;
      }
      if (lane < kScanTokens) as[b][lane] = last ? got : a;
    } else {
      double after = g;                      // the sum of g from this token to the stage's end, then from the next one
#pragma unroll
      for (int off = 1; off < kScanTokens; off <<= 1) {
        const double x = __shfl_down_sync(0xffffffffu, after, off);
        if (lane + off < kScanTokens) after += x;
      }
      const double all = __shfl_sync(0xffffffffu, after, 0), next = __shfl_down_sync(0xffffffffu, after, 1);
      double want = exp(lane == kScanTokens ? all : lane + 1 < kScanTokens ? next : 0.0);
      if (lane == kScanTokens) want *= rest;
      const float w = (float)want;
      rest = w > 1e-30f && w < 1e30f ? want / w : 1.0;
      if (lane < kScanTokens) as[b][lane] = w;
      if (lane == kScanTokens) stage[b] = w;
      sum += all;
    }
  };
  if (it.len > 0) {
    fetch(0);
    if (warp == 0) decays(0, gate(0));
  }
  for (int c0 = 0; c0 < it.len; c0 += kScanTokens) {
    const int L = min(kScanTokens, it.len - c0), t0 = it.t0 + c0, b = (c0 / kScanTokens) & 1;
    const bool more = c0 + kScanTokens < it.len;
    wait_copies();
    __syncthreads();                         // this stage is there, and the one before has been left
    float g_next = 0.f;
    if (more) {
      fetch(c0 + kScanTokens);
      if (warp == 0) g_next = gate(c0 + kScanTokens);
    }
    auto token = [&](int t, auto first) {    // first: the one that takes the stage's decay
      const float a = as[b][t];
      [[maybe_unused]] const float f = kOut ? 0.f : stage[b];
      float vi[kR], acc[kR][4];
#pragma unroll
      for (int u = 0; u < kR; ++u) {
        vi[u] = vs[b][t][rl + 32 * u];
        if constexpr (!kOut) vi[u] *= a;
        acc[u][0] = acc[u][1] = acc[u][2] = acc[u][3] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const float4 kk = *reinterpret_cast<const float4*>(&ks[b][t][4 * (sub + 4 * i)]);
        [[maybe_unused]] float4 qq;
        if constexpr (kOut) qq = *reinterpret_cast<const float4*>(&qs[b][t][4 * (sub + 4 * i)]);
#pragma unroll
        for (int u = 0; u < kR; ++u) {
          float* x = s[u] + 4 * i;
          if constexpr (kOut) {
            x[0] = fmaf(a, x[0], vi[u] * kk.x);
            x[1] = fmaf(a, x[1], vi[u] * kk.y);
            x[2] = fmaf(a, x[2], vi[u] * kk.z);
            x[3] = fmaf(a, x[3], vi[u] * kk.w);
            acc[u][0] = fmaf(x[0], qq.x, acc[u][0]);
            acc[u][1] = fmaf(x[1], qq.y, acc[u][1]);
            acc[u][2] = fmaf(x[2], qq.z, acc[u][2]);
            acc[u][3] = fmaf(x[3], qq.w, acc[u][3]);
          } else if constexpr (decltype(first)::value) {
            x[0] = fmaf(f, x[0], vi[u] * kk.x);
            x[1] = fmaf(f, x[1], vi[u] * kk.y);
            x[2] = fmaf(f, x[2], vi[u] * kk.z);
            x[3] = fmaf(f, x[3], vi[u] * kk.w);
          } else {
            x[0] = fmaf(vi[u], kk.x, x[0]);
            x[1] = fmaf(vi[u], kk.y, x[1]);
            x[2] = fmaf(vi[u], kk.z, x[2]);
            x[3] = fmaf(vi[u], kk.w, x[3]);
          }
        }
      }
      if constexpr (kOut) {
#pragma unroll
        for (int u = 0; u < kR; ++u) {
          const float r = group_sum<4>((acc[u][0] + acc[u][1]) + (acc[u][2] + acc[u][3]));
          if (sub == 0) vs[b][t][rl + 32 * u] = p.scale * r;   // only this row's lanes read v_t[row], and they have
        }
      }
    };
    if constexpr (kOut) {
      for (int t = 0; t < L; ++t) token(t, std::false_type());
    } else {
      token(0, std::true_type());
      for (int t = 1; t < L; ++t) token(t, std::false_type());
    }
    if (more && warp == 0) decays(c0 + kScanTokens, g_next);
    if constexpr (kOut) {
      __syncthreads();
      for (int e = tid; e < L * (kScanRows / 4); e += kScanThreads) {
        const int t = e / (kScanRows / 4), i = 4 * (e - t * (kScanRows / 4));
        if (i0 + i < dv)
          *reinterpret_cast<float4*>(o + ((size_t)(t0 + t) * p.Hv + h) * dv + i0 + i) =
              *reinterpret_cast<const float4*>(&vs[b][t][i]);
      }
    }
  }
  float* to = !kOut ? p.states + slot : it.J == 1 ? p.state_out + srow : nullptr;
#pragma unroll
  for (int u = 0; u < kR; ++u) {
    if (to && row + 32 * u < dv) {
#pragma unroll
      for (int i = 0; i < E / 4; ++i)
        *reinterpret_cast<float4*>(to + 32 * u * DK + 16 * i) =
            make_float4(s[u][4 * i], s[u][4 * i + 1], s[u][4 * i + 2], s[u][4 * i + 3]);
    }
  }
  if (!kOut && i0 == 0 && tid == 0) {
    const double a = exp(sum);
    const float hi = (float)a;
    p.decays[(size_t)blockIdx.x * p.Hv + h] = make_float2(hi, hi < 1e30f ? (float)(a - hi) : 0.f);
  }
}

// The states that enter the segments, in place of the segments' own, and the final ones.
// grid: (ceil(dv dk / 1024), Hv, n_seqs); 256 threads of 4 values. Bound by the bytes of the
// states; eight segments' loads are in flight at a time.
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
  if (!GDN_CHECK(first >= 0 && J > 0 && n < p.n_seqs)) return;
  const size_t own = ((size_t)n * p.Hv + h) * per_state + at, step = (size_t)p.Hv * per_state;
  float* slot = p.states + ((size_t)first * p.Hv + h) * per_state + at;
  const float2* decay = p.decays + (size_t)first * p.Hv + h;
  float4 s = p.state_in ? *reinterpret_cast<const float4*>(p.state_in + own) : make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kAhead = 8;
  float4 x[kAhead];
  float2 a[kAhead];
  auto load = [&](int u, int j) {
    if (j < J) {
      x[u] = *reinterpret_cast<const float4*>(slot + j * step);
      a[u] = decay[(size_t)j * p.Hv];
    }
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u) load(u, u);
  for (int j = 0; j < J; j += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (j + u < J) {
        const float4 own_x = x[u];
        const float2 own_a = a[u];
        load(u, j + u + kAhead);             // in flight for eight segments' time
        *reinterpret_cast<float4*>(slot + (j + u) * step) = s;
        s.x = fmaf(own_a.x, s.x, fmaf(own_a.y, s.x, own_x.x));
        s.y = fmaf(own_a.x, s.y, fmaf(own_a.y, s.y, own_x.y));
        s.z = fmaf(own_a.x, s.z, fmaf(own_a.y, s.z, own_x.z));
        s.w = fmaf(own_a.x, s.w, fmaf(own_a.y, s.w, own_x.w));
      }
    }
  }
  *reinterpret_cast<float4*>(p.state_out + own) = s;
}

}  // namespace lin
}  // namespace gdn
