// A pool of recurrent states in 8 bits: states written into slots (store) and
// read back (load).
//
// Along d_k the values are taken in groups of 32 (16 where d_k = 16). A group
// holds one exponent byte b and 8-bit codes; the value is code 2^(b - 127). The
// codes are e4m3 floats (largest 448) or integers (largest 127), and b is the
// smallest exponent that fits the group's largest magnitude (0 at least), so
//
//   - scaling by 2^(127 - b) is exact and the only rounding is the code's own, to
//     nearest even: at most half a step of 2^-3 relative (e4m3), or 2^(b - 128)
//     absolute (integers);
//   - storing what was loaded gives the same values again, so a sequence that is
//     set aside many times does not drift.
//
// A group with an infinity or a NaN gets b = 255 and loads as NaN throughout.
// Both kernels are bound by the bytes they move; a lane takes 4 consecutive
// values (16 bytes of fp32), so a group is 8 lanes and its largest magnitude
// three shuffles, and keeps kUnroll such accesses in flight.
//
// Measured, 32 heads of 128 x 128, fp32 and e4m3: 64 states stored and loaded again 55.3 us
// (338 MB, 6.1 TB/s); 48 loaded 23.3 us (5.4 TB/s). With 4 accesses in flight 55.9 and 23.2,
// with 16 57.3 and 23.5.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace gdn {
namespace pool {

constexpr int kThreads = 256;
constexpr int kUnroll = 8;
constexpr int kTile = kThreads * 4 * kUnroll;   // values per CTA

struct E4M3 {
  static constexpr uint32_t kMaxMant = 0x600000u;   // 448 = 1.75 * 2^8
  static constexpr int kMaxExp = 8;
  static __device__ __forceinline__ uint32_t encode4(const float* y) {
    const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
    return (uint32_t)lo | ((uint32_t)hi << 16);
  }
  static __device__ __forceinline__ void decode4(uint32_t c, float* y) {
    const __half2 lo(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xffffu), __NV_E4M3));
    const __half2 hi(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> 16), __NV_E4M3));
    const float2 a = __half22float2(lo), b = __half22float2(hi);
    y[0] = a.x; y[1] = a.y; y[2] = b.x; y[3] = b.y;
  }
};
struct I8 {
  static constexpr uint32_t kMaxMant = 0x7e0000u;   // 127 = 1.984375 * 2^6
  static constexpr int kMaxExp = 6;
  static __device__ __forceinline__ uint32_t encode4(const float* y) {
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) c |= ((uint32_t)__float2int_rn(y[i]) & 0xffu) << (8 * i);
    return c;
  }
  static __device__ __forceinline__ void decode4(uint32_t c, float* y) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = (float)(int8_t)(c >> (8 * i));
  }
};

// The exponent byte of a group whose largest magnitude has these bits.
template <typename F>
__device__ __forceinline__ uint32_t exponent_byte(uint32_t amax_bits) {
  const int x = (int)(amax_bits >> 23);
  if (x == 255) return 255u;
  const int b = x - F::kMaxExp + ((amax_bits & 0x7fffffu) > F::kMaxMant ? 1 : 0);
  return b > 0 ? (uint32_t)b : 0u;
}

// Touched once: streaming accesses.
__device__ __forceinline__ float4 fetch4(const float* p) { return ld_stream(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 fetch4(const __nv_bfloat16* p) {
  const uint2 raw = __ldcs(reinterpret_cast<const uint2*>(p));
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store4(float* p, const float* y) {
  st_stream(reinterpret_cast<float4*>(p), make_float4(y[0], y[1], y[2], y[3]));
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* y) {
  __nv_bfloat162 a = __floats2bfloat162_rn(y[0], y[1]), b = __floats2bfloat162_rn(y[2], y[3]);
  __stcs(reinterpret_cast<uint2*>(p), make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b)));
}

// grid: n * tiles, tiles = ceil(per_state / kTile); per_state = Hv dv dk, a
// multiple of 256. G: lanes per group (8, or 4 where dk = 16).
template <typename F, typename TS, int G>
__global__ void __launch_bounds__(kThreads)
store_kernel(const TS* __restrict__ state, const int32_t* __restrict__ slots, int n, int n_slots, int tiles,
             long long per_state, uint32_t* __restrict__ codes, uint8_t* __restrict__ exps) {
  const int i = blockIdx.x / tiles, tile = blockIdx.x - i * tiles;
  const int slot = slots[i];
  if (slot < 0 || slot >= n_slots) return;
  // a slot named twice takes its last state: an earlier one leaves it alone
  int later = 0;
  for (int j = i + 1 + (int)threadIdx.x; j < n; j += kThreads) later |= slots[j] == slot;
  if (__syncthreads_or(later)) return;

  if (!GDN_CHECK(i < n && tile < tiles && (long long)tile * kTile < per_state)) return;
  const long long base = (long long)tile * kTile + threadIdx.x * 4;
  const TS* src = state + (size_t)i * per_state;
  float4 x[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long at = base + u * (kThreads * 4);
    x[u] = at < per_state ? fetch4(src + at) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  uint32_t* cdst = codes + (size_t)slot * (per_state / 4);
  uint8_t* edst = exps + (size_t)slot * (per_state / (4 * G));
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long at = base + u * (kThreads * 4);
    uint32_t m = max(max(__float_as_uint(x[u].x) & 0x7fffffffu, __float_as_uint(x[u].y) & 0x7fffffffu),
                     max(__float_as_uint(x[u].z) & 0x7fffffffu, __float_as_uint(x[u].w) & 0x7fffffffu));
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
    const uint32_t b = exponent_byte<F>(m);
    const float inv = b == 255u ? 0.f : __uint_as_float((254u - b) << 23);   // 2^(127 - b)
    float y[4] = {x[u].x * inv, x[u].y * inv, x[u].z * inv, x[u].w * inv};
    if (at < per_state) {
      cdst[at / 4] = b == 255u ? 0u : F::encode4(y);
      if ((threadIdx.x & (G - 1)) == 0) edst[at / (4 * G)] = (uint8_t)b;
    }
  }
}

// grid: n * tiles
template <typename F, typename TS, int G>
__global__ void __launch_bounds__(kThreads)
load_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ exps,
            const int32_t* __restrict__ slots, int n_slots, int tiles, long long per_state,
            TS* __restrict__ state) {
  const int i = blockIdx.x / tiles, tile = blockIdx.x - i * tiles;
  const int slot = slots[i];
  const bool held = slot >= 0 && slot < n_slots;   // another slot: a sequence without a past, zeros
  if (!GDN_CHECK(tile < tiles && (long long)tile * kTile < per_state)) return;
  const long long base = (long long)tile * kTile + threadIdx.x * 4;
  const uint32_t* csrc = codes + (size_t)(held ? slot : 0) * (per_state / 4);
  const uint8_t* esrc = exps + (size_t)(held ? slot : 0) * (per_state / (4 * G));
  uint32_t c[kUnroll], b[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long at = base + u * (kThreads * 4);
    const bool in = held && at < per_state;
    c[u] = in ? __ldcs(csrc + at / 4) : 0u;
    b[u] = in ? esrc[at / (4 * G)] : 0u;
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long at = base + u * (kThreads * 4);
    float y[4];
    F::decode4(c[u], y);
    const float scale = b[u] == 255u ? __uint_as_float(0x7fc00000u)
                        : b[u] == 0u ? __uint_as_float(0x00400000u)   // 2^-127
                                     : __uint_as_float(b[u] << 23);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] *= scale;
    if (at < per_state) store4(state + (size_t)i * per_state + at, y);
  }
}

}  // namespace pool
}  // namespace gdn
