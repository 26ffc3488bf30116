// Chunked prefill of decayed linear attention on the sm_100a tensor cores, one
// persistent kernel (bf16 or f16 inputs; d_k, d_v up to 128, smaller ones padded
// with zeros by the TMA loads).
//
// Mathematics. A block of up to 128 tokens enters with state S (d_v x d_k). With
// G_r the log-decays summed from the block's first token to r, G_L their total:
//
//   P_rs = scale exp(G_r - G_s) q_r . k_s  (s <= r),   o_r = exp(G_r) scale S q_r + sum_s P_rs v_s
//   S   <- exp(G_L) S + sum_s v_s (exp(G_L - G_s) k_s)^T
//
// Four products a block, each 128 x 128 x 128: Q K^T, Q S^T, P V and V^T K~ with
// K~_s = w_s k_s, w_s = exp(G_L - G_s). No state element ever waits for a sum over
// tokens outside the tensor core; the state itself lives in fp32 registers of the
// compute warps (64 values a thread) and is only read by the tensor core as a
// rounded copy, for o.
//
// Precision. o has 16 bits, so P and the copy of S that Q meets are rounded to the
// input type (half a step each, and no term of o carries both). The state is fp32,
// so K~ is not rounded: it is split into three bf16 terms (8 bits each, 24 in all)
// or two f16 terms (22 bits) that are multiplied with V one after another into one
// accumulator. In f16 powers of two keep what is rounded in the type's range: one from
// the block's largest |k| and w for the terms of K~, one from the largest |S| for the
// copy of S, and one for P where a score passes 2^15.
// Log-decays are summed in fp64 (exp(G_r - G_s) of far tokens is a difference of
// large sums) and clamped at -200, where exp is zero in fp32, so that a reset (-inf)
// does not turn differences into NaN.
//
// Work over a long axis. Heads alone do not fill the GPU, so a sequence is cut into
// segments of `seg` blocks; one item is (sequence, head, segment), item i belongs to
// CTA i mod G. An item has two passes over its segment:
//
//   A  (not for a sequence's last segment) K and V only: the segment's own
//      contribution to the state, published to the workspace with its decay;
//   B  Q, K, V: the outputs, from the state that enters the segment. K and V come
//      from L2 this time.
//
// The states that enter the segments are the running combination of the published
// ones. Two scan warps per CTA compute it: a warp owns 1/16 of one head's state,
// carries it in registers from segment to segment and hands every result to the
// CTA that waits for it. Heads are taken in panels of at most 4 G / 32, so each
// (head, 1/32) of a panel has an owner of its own.
//
// Order and progress. Items are numbered (sequence, panel, segment, head). Every
// wait on another CTA is for work of a lower number -- B(i) and scan(i) for scans
// and publications before i, a publication for the scan of the same slot's last
// but one user, a scan for the reading of a slot two rounds back -- so with all CTAs
// resident (cooperative launch) the lowest unfinished one can always go on. All
// waits are bounded; after one ran out a warp waits no more and runs to its end.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "sm100.cuh"

namespace gdn {
namespace ltc {

using namespace sm100;

constexpr int kB = 128;              // tokens per block
constexpr int kD = 128;              // padded head size
constexpr int kCompute = 256;        // warps 0-7
constexpr int kLoadWarp = 8;         // K, V tiles
constexpr int kMmaWarp = 9;          // tensor-core work
constexpr int kGateWarp = 10;        // Q tiles and the decay tables
constexpr int kScanWarp = 12;        // to 15 (warp 11 has no job: registers go by four warps)
constexpr int kScanWarps = 4;
constexpr int kThreads = 32 * (kScanWarp + kScanWarps);
constexpr int kSlices = 32;          // owners of one head's state
// Registers: 512 threads start with 128 each; the compute warps' share grows by what
// the others give back (256 x 176 + 256 x 80 = 65536, all that the block holds).
constexpr int kRegsCompute = 176, kRegsOther = 80;
static_assert(kCompute * kRegsCompute + (kThreads - kCompute) * kRegsOther <= 65536, "register file");
constexpr int kStateBytes = kD * kD * 4;
constexpr float kMinLog = -200.f;

// ---- shared memory (bytes) ----
constexpr uint32_t kQ = 0;                     // [128][128] as two K-major 128B-swizzled atoms, 16 KB apart
constexpr uint32_t kK = 32768;                 // two buffers
constexpr uint32_t kV = 98304;                 // two buffers
constexpr uint32_t kS = 163840;                // the rounded copy of S; pass A: terms of K~, second half
constexpr uint32_t kML = 196608;               // terms of K~ (half a block); o on its way out
constexpr uint32_t kStage = kS;                // kS and kML together: a state on its way in or out
constexpr uint32_t kTab = 229376;              // float w[128], gam[128], gh[128], gl[128]
constexpr uint32_t kBars = kTab + 2048;
constexpr uint32_t kMisc = kBars + 256;        // words: see Misc
constexpr uint32_t kSmem = kMisc + 256;
static_assert(kSmem <= 227 * 1024, "shared memory budget");

enum Bar { kKvFull = 0, kKvEmpty = 2, kQFull = 4, kOiDone, kTabFull, kTabEmpty, kPFull, kKt0, kKt1, kMlFree, kPt, kOFull,
           kOFree, kUFull, kSReady, kStFull, kNumBars };

struct Misc {
  uint32_t tmem;
  float gam_l;         // exp(G_L) of the block
  float seg_gam;       // exp of the segment's total log-decay, up to this block
  uint32_t big;        // |G| is large somewhere in the block: its low parts are needed
  float red[8];        // reductions over the compute warps (f16)
  float w_max;         // the largest w of the block
};

// ---- tensor memory columns ----
constexpr uint32_t kColP = 0;        // Q K^T, then P in place (16 bits: columns 0-31 and 64-95)
constexpr uint32_t kColOi = 128;     // Q S^T
constexpr uint32_t kColOa = 256;     // P V
constexpr uint32_t kColU = 384;      // V^T K~

// ---- workspace ----
constexpr int kFlagWords = 32;       // per CTA: out_ready[2], scanned[2], in_cnt[2], done
enum Flag { kOutReady = 0, kScanned = 2, kInCnt = 4, kDone = 6 };
struct Workspace {
  __host__ __device__ static constexpr size_t flags_bytes(int ctas) { return (size_t)ctas * kFlagWords * 4; }
  __host__ __device__ static constexpr size_t meta_offset(int ctas) { return flags_bytes(ctas); }       // float per (CTA, parity)
  __host__ __device__ static constexpr size_t slots_offset(int ctas) { return (flags_bytes(ctas) + (size_t)ctas * 8 + 1023) & ~size_t(1023); }
  // per CTA: two published states, two entering states
  __host__ __device__ static constexpr size_t bytes(int ctas) { return slots_offset(ctas) + (size_t)ctas * 4 * kStateBytes; }
};

struct Params {
  const float* g;
  const float* state_in;
  const int32_t* cu_seqlens;
  void* o;
  float* state_out;
  uint8_t* ws;
  int g_stride, n_seqs, total_T, Hqk, Hv, dk, dv, seg, panel;
  float scale;
  long long limit;     // SM cycles that a wait lasts at most
};

// Waits that stop waiting once one has run out. The limit grows with the problem: a
// scan warp may wait for a sequence that comes at the end.
struct Wait {
  long long limit;
  bool ok = true;
  __device__ __forceinline__ explicit Wait(long long l) : limit(l) {}
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    if (ok) ok = mbar_wait(bar, parity, limit);
  }
  __device__ __forceinline__ void flag(const uint32_t* p, uint32_t target) {
    if (ok) ok = wait_flag_geq(p, target, limit);
  }
};

struct Item {
  int n, h, j, J;      // sequence, head, segment of J
  int hp;              // heads in the panel: the next segment's item is this many further
  int t0, len;         // the segment's first token and tokens
  int first;           // the item of segment 0 of this sequence and head
};

// Finds items in increasing order (warp-collective).
struct Walk {
  int n = 0, base = 0;
  __device__ __forceinline__ bool find(const Params& p, int item, Item& it) {
    const int lane = threadIdx.x & 31;
    const int seg_t = p.seg * kB;
    for (;;) {
      if (n >= p.n_seqs) return false;
      int a = 0, len = 0, J = 0;
      if (n + lane < p.n_seqs) {
        a = min(max(p.cu_seqlens[n + lane], 0), p.total_T);
        len = max(min(max(p.cu_seqlens[n + lane + 1], 0), p.total_T) - a, 0);
        J = max(1, (len + seg_t - 1) / seg_t);
      }
      const int cnt = J * p.Hv;
      int incl = cnt;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += x;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, base + incl > item);
      if (hit) {
        const int src = __ffs(hit) - 1;
        n += src;
        base += __shfl_sync(0xffffffffu, incl - cnt, src);
        J = __shfl_sync(0xffffffffu, J, src);
        a = __shfl_sync(0xffffffffu, a, src);
        len = __shfl_sync(0xffffffffu, len, src);
        const int li = item - base, per = J * p.panel, pi = li / per, rem = li - pi * per;
        const int hp = min(p.panel, p.Hv - pi * p.panel);
        it.n = n;
        it.J = J;
        it.hp = hp;
        it.j = rem / hp;
        it.h = pi * p.panel + rem - it.j * hp;
        it.first = item - it.j * hp;
        it.t0 = a + it.j * seg_t;
        it.len = min(seg_t, len - it.j * seg_t);
        return true;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
      n += 32;
    }
  }
};

// 16 columns of 32 lanes: registers to tensor memory (complete after tmem_wait_st).
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Four K-steps with A in TMEM (8 columns a step) and B advancing BSTEP 16-byte units a
// step, from one asm block (as mma_run_warp).
template <uint32_t BSTEP>
__device__ __forceinline__ void mma4_tmem_a_run_warp(uint32_t d_tmem, uint32_t a_tmem, uint64_t b0, uint32_t idesc,
                                                     uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 t, %3, %3;\n\t"
      "mov.b32 a, %1;\n\t"
      "mov.b64 b, %2;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p;\n\t"
      "add.u32 a, a, 8;\n\tadd.s64 b, b, %5;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.u32 a, a, 8;\n\tadd.s64 b, b, %5;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.u32 a, a, 8;\n\tadd.s64 b, b, %5;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b0), "r"(idesc), "r"(acc), "n"(BSTEP)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^e as a float, e clamped to the normal range.
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(min(max(e, -126), 127) + 127) << 23); }
// The exponent e with |x| < 2^(e + 1) (x finite; 128 for infinities and NaN).
__device__ __forceinline__ int exponent_of(float x) { return (int)((__float_as_uint(x) >> 23) & 255u) - 127; }

__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// The scan warps: owner `ow` of 4 G carries its share of each panel's head.
__device__ __forceinline__ void scan_role(const Params& p, int ow, int G) {
  const int lane = threadIdx.x & 31;
  const int hl = ow / kSlices, sl = ow - hl * kSlices;
  const int seg_t = p.seg * kB;
  uint32_t* flags = reinterpret_cast<uint32_t*>(p.ws);
  const float* meta = reinterpret_cast<const float*>(p.ws + Workspace::meta_offset(G));
  uint8_t* slots = p.ws + Workspace::slots_offset(G);
  Wait wait(p.limit);
  int base = 0;
  for (int n0 = 0; n0 < p.n_seqs; n0 += 32) {
    int J = 0;
    if (n0 + lane < p.n_seqs) {
      const int a = min(max(p.cu_seqlens[n0 + lane], 0), p.total_T);
      const int len = max(min(max(p.cu_seqlens[n0 + lane + 1], 0), p.total_T) - a, 0);
      J = max(1, (len + seg_t - 1) / seg_t);
    }
    for (int i = 0; i < 32 && n0 + i < p.n_seqs; ++i) {
      const int Jn = __shfl_sync(0xffffffffu, J, i);
      if (Jn > 1) {
        for (int h0 = 0; h0 < p.Hv; h0 += p.panel) {
          const int hp = min(p.panel, p.Hv - h0);
          if (hl >= hp) continue;
          float4 S[4];
          // word x = v * 256 + t of a slot holds columns 4 v .. 4 v + 3 of thread t's 64
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int t = 128 * (sl & 1) + 32 * u + lane, row = t & 127, col = 64 * (t >> 7) + 4 * (sl >> 1);
            S[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p.state_in && row < p.dv && col < p.dk)
              S[u] = __ldcg(reinterpret_cast<const float4*>(
                  p.state_in + (((size_t)(n0 + i) * p.Hv + h0 + hl) * p.dv + row) * p.dk + col));
          }
          for (int j = 0; j + 1 < Jn; ++j) {
            const int item = base + h0 * Jn + j * hp + hl, c = item % G, r = item / G;
            const int dst = item + hp, c2 = dst % G, r2 = dst / G;
            if (lane == 0) wait.flag(flags + c * kFlagWords + kOutReady + (r & 1), r + 1);
            __syncwarp();
            const float gam = __ldcg(meta + 2 * c + (r & 1));
            const float4* src = reinterpret_cast<const float4*>(slots + (size_t)(4 * c + (r & 1)) * kStateBytes) + 128 * sl;
            float4 L[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) L[u] = __ldcg(src + 32 * u + lane);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              S[u].x = fmaf(gam, S[u].x, L[u].x);
              S[u].y = fmaf(gam, S[u].y, L[u].y);
              S[u].z = fmaf(gam, S[u].z, L[u].z);
              S[u].w = fmaf(gam, S[u].w, L[u].w);
            }
            if (lane == 0 && r2 >= 2) wait.flag(flags + c2 * kFlagWords + kDone, r2 - 1);
            __syncwarp();
            float4* d = reinterpret_cast<float4*>(slots + (size_t)(4 * c2 + 2 + (r2 & 1)) * kStateBytes) + 128 * sl;
#pragma unroll
            for (int u = 0; u < 4; ++u) __stcg(d + 32 * u + lane, S[u]);
            __syncwarp();
            if (lane == 0) {
              red_add_release_gpu(flags + c2 * kFlagWords + kInCnt + (r2 & 1), 1u);
              red_add_release_gpu(flags + c * kFlagWords + kScanned + (r & 1), 1u);
            }
          }
        }
      }
      base += Jn * p.Hv;
    }
  }
}

__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
}
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsCompute));
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
prefill_kernel(const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap km,
               const __grid_constant__ CUtensorMap vm, const __grid_constant__ CUtensorMap om,
               const __grid_constant__ CUtensorMap sim, const __grid_constant__ CUtensorMap som, const Params p) {
  constexpr bool kF16 = std::is_same<T, __half>::value;
  constexpr uint32_t kFmt = Op16<T>::kFmt;
  constexpr int kTerms = kF16 ? 2 : 3;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kBars);
  Misc* misc = reinterpret_cast<Misc*>(sm + kMisc);
  float* tab_w = reinterpret_cast<float*>(sm + kTab);
  float* tab_gam = tab_w + kB;
  float* tab_gh = tab_w + 2 * kB;
  float* tab_gl = tab_w + 3 * kB;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = gridDim.x, cta = blockIdx.x;

  if (smem_u32(sm) & 1023u) {   // the swizzled tiles need it; never seen (no static shared memory)
    if (tid == 0) flag_error(kErrCheck);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      const bool warps = i == kTabEmpty || i == kKt0 || i == kKt1 || i == kPt || i == kOFree || i == kSReady;
      mbar_init(&bars[i], warps ? 8 : i == kTabFull ? 32 : 1);
    }
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&misc->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc->tmem;
  const uint32_t sbase = smem_u32(sm);
  Wait wait(p.limit);
  Walk walk;
  Item it;
  if (warp == kLoadWarp) {
    give_registers();
    // ---------------------------------------------------------- K, V tiles ---
    const uint64_t once = l2_evict_first_policy();
    uint32_t cnt = 0;
    for (int item = cta; walk.find(p, item, it); item += G) {
      const int hq = it.h / (p.Hv / p.Hqk), nb = (it.len + kB - 1) / kB;
      const bool shared_k = p.Hv != p.Hqk;
      for (int pass = it.j + 1 < it.J ? 0 : 1; pass < 2; ++pass) {
        for (int b = 0; b < nb; ++b, ++cnt) {
          const uint32_t s = cnt & 1;
          if (cnt >= 2) wait(&bars[kKvEmpty + s], ((cnt >> 1) - 1) & 1);
          if (!wait.ok) break;
          const int t = it.t0 + b * kB;
          uint64_t* full = &bars[kKvFull + s];
          mbar_arrive_expect_tx_warp(full, 65536);
          uint8_t *kt = sm + kK + s * 32768, *vt = sm + kV + s * 32768;
          // the second pass is the last to read V, and K where no other head shares it
          if (pass == 0 || shared_k) {
            tma_load_3d_warp(kt, &km, full, 0, hq, t);
            tma_load_3d_warp(kt + 16384, &km, full, 64, hq, t);
          } else {
            tma_load_3d_warp_hint(kt, &km, full, 0, hq, t, once);
            tma_load_3d_warp_hint(kt + 16384, &km, full, 64, hq, t, once);
          }
          if (pass == 0) {
            tma_load_3d_warp(vt, &vm, full, 0, it.h, t);
            tma_load_3d_warp(vt + 16384, &vm, full, 64, it.h, t);
          } else {
            tma_load_3d_warp_hint(vt, &vm, full, 0, it.h, t, once);
            tma_load_3d_warp_hint(vt + 16384, &vm, full, 64, it.h, t, once);
          }
        }
      }
    }
    // tiles still on their way land before the CTA ends
    for (uint32_t c = cnt >= 2 ? cnt - 2 : 0; c < cnt; ++c) mbar_wait(&bars[kKvFull + (c & 1)], (c >> 1) & 1, p.limit);
  } else if (warp == kGateWarp) {
    give_registers();
    // ------------------------------------------- Q tiles and decay tables ---
    uint32_t qn = 0, tn = 0;
    for (int item = cta; walk.find(p, item, it); item += G) {
      const int hq = it.h / (p.Hv / p.Hqk), nb = (it.len + kB - 1) / kB;
      for (int pass = it.j + 1 < it.J ? 0 : 1; pass < 2; ++pass) {
        double seg = 0.0;
        for (int b = 0; b < nb; ++b) {
          const int t = it.t0 + b * kB, L = min(kB, it.len - b * kB);
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int s = 4 * lane + e;
            const float gv = s < L ? p.g[(size_t)(t + s) * p.g_stride + it.h] : 0.f;
            x[e] = gv < kMinLog ? kMinLog : gv;
          }
          if (pass == 1) {
            if (qn > 0) wait(&bars[kOiDone], (qn - 1) & 1);
            if (wait.ok) {
              mbar_arrive_expect_tx_warp(&bars[kQFull], 32768);
              tma_load_3d_warp(sm + kQ, &qm, &bars[kQFull], 0, hq, t);
              tma_load_3d_warp(sm + kQ + 16384, &qm, &bars[kQFull], 64, hq, t);
              ++qn;
            }
          }
          double c[4];
          c[0] = x[0]; c[1] = c[0] + x[1]; c[2] = c[1] + x[2]; c[3] = c[2] + x[3];
          double incl = c[3];
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
          }
          const double end = __shfl_sync(0xffffffffu, incl, 31), before = incl - c[3];
          seg += end;
          float w[4], gm[4], gh[4], gl[4], far = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const double Gs = before + c[e], G2 = Gs * 1.4426950408889634;
            w[e] = 4 * lane + e < L ? expf((float)(end - Gs)) : 0.f;
            gm[e] = expf((float)Gs) * p.scale;
            gh[e] = (float)G2;
            gl[e] = (float)(G2 - (double)gh[e]);
            far = fmaxf(far, fabsf(gh[e]));
          }
          // from 64 on half a step of gh alone would move a weight by 2.6e-6 of itself
          const uint32_t big = __any_sync(0xffffffffu, !(far < 64.f));
          if (tn > 0) wait(&bars[kTabEmpty], (tn - 1) & 1);
          reinterpret_cast<float4*>(tab_w)[lane] = make_float4(w[0], w[1], w[2], w[3]);
          reinterpret_cast<float4*>(tab_gam)[lane] = make_float4(gm[0], gm[1], gm[2], gm[3]);
          reinterpret_cast<float4*>(tab_gh)[lane] = make_float4(gh[0], gh[1], gh[2], gh[3]);
          reinterpret_cast<float4*>(tab_gl)[lane] = make_float4(gl[0], gl[1], gl[2], gl[3]);
          float wm = fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3]));
          if constexpr (kF16) {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, off));
          }
          if (lane == 0) {
            misc->w_max = wm;
            misc->gam_l = expf((float)end);
            misc->seg_gam = expf((float)seg);
            misc->big = big;
          }
          mbar_arrive(&bars[kTabFull]);
          ++tn;
        }
      }
    }
    if (qn > 0) mbar_wait(&bars[kQFull], (qn - 1) & 1, p.limit);
  } else if (warp == kMmaWarp) {
    give_registers();
    // ------------------------------------------------- tensor-core work ---
    constexpr uint32_t id_kk = idesc_f16kind(128, 128, false, false, kFmt);
    constexpr uint32_t id_pv = idesc_f16kind(128, 128, false, true, kFmt);
    constexpr uint32_t id_u = idesc_f16kind(128, 128, true, true, kFmt);
    uint32_t cnt = 0, qn = 0, un = 0, bn = 0;
    for (int item = cta; walk.find(p, item, it); item += G) {
      const int nb = (it.len + kB - 1) / kB;
      const bool last = it.j + 1 == it.J;
      for (int pass = last ? 1 : 0; pass < 2; ++pass) {
        for (int b = 0; b < nb; ++b, ++cnt) {
          const uint32_t s = cnt & 1;
          const uint32_t kt = sbase + kK + s * 32768, vt = sbase + kV + s * 32768;
          const bool upd = pass == 0 || last || b + 1 < nb;   // the state after the segment comes from pass A
          wait(&bars[kKvFull + s], (cnt >> 1) & 1);
          if (pass == 1) {
            wait(&bars[kQFull], qn & 1);
            tc_fence_after();
            {
              const uint64_t qd = desc_kmajor(sbase + kQ, 0, 16384), kd = desc_kmajor(kt, 0, 16384);
              mma_run_warp<4, 2, 2>(tmem + kColP, qd, kd, id_kk, 0);
              mma_run_warp<4, 2, 2>(tmem + kColP, desc_advance(qd, 16384), desc_advance(kd, 16384), id_kk, 1);
            }
            mma_commit_warp(&bars[kPFull]);
            wait(&bars[kSReady], qn & 1);
            if (qn > 0) wait(&bars[kOFree], (qn - 1) & 1);
            tc_fence_after();
            {
              const uint64_t qd = desc_kmajor(sbase + kQ, 0, 16384), sd = desc_kmajor(sbase + kS, 0, 16384);
              mma_run_warp<4, 2, 2>(tmem + kColOi, qd, sd, id_kk, 0);
              mma_run_warp<4, 2, 2>(tmem + kColOi, desc_advance(qd, 16384), desc_advance(sd, 16384), id_kk, 1);
            }
            mma_commit_warp(&bars[kOiDone]);
            ++qn;
          }
          auto half = [&](int hf, uint32_t buf) {
            wait(&bars[kKt0 + hf], un & 1);
            tc_fence_after();
            const uint64_t vd = desc_mnmajor(vt, 4 * hf, 128, 16384);
            mma_run_warp<4, 128, 128>(tmem + kColU, vd, desc_mnmajor(kt, 4 * hf, 128, 16384), id_u, hf);
#pragma unroll
            for (int term = 1; term < kTerms; ++term)
              mma_run_warp<4, 128, 128>(tmem + kColU, vd, desc_mnmajor(buf + (term - 1) * 16384, 0, 128, 8192), id_u, 1);
          };
          if (upd) half(0, sbase + kML);
          if (pass == 1) {
            if (upd) mma_commit_warp(&bars[kMlFree]);
            wait(&bars[kPt], bn++ & 1);
            tc_fence_after();
            {
              const uint64_t vd = desc_mnmajor(vt, 0, 128, 16384);
              mma4_tmem_a_run_warp<128>(tmem + kColOa, tmem + kColP, vd, id_pv, 0);
              mma4_tmem_a_run_warp<128>(tmem + kColOa, tmem + kColP + 64, desc_advance(vd, 4 * 2048), id_pv, 1);
            }
            mma_commit_warp(&bars[kOFull]);
          }
          if (upd) {
            half(1, pass == 0 ? sbase + kS : sbase + kML);
            ++un;
            mma_commit_warp(&bars[kUFull]);
          }
          mma_commit_warp(&bars[kKvEmpty + s]);
        }
      }
    }
  } else if (warp >= 8) {
    give_registers();
    // ------------------------------------- states between the segments ---
    if (p.ws && warp >= kScanWarp) scan_role(p, cta * kScanWarps + warp - kScanWarp, G);
  } else {
    // ----------------------------------------------------- compute warps ---
    take_registers();
    const int wg = warp >> 2, w4 = warp & 3, row = 32 * w4 + lane;   // row of every 128-row tile, columns 64 wg ..
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * w4) << 16);
    uint32_t* flags = reinterpret_cast<uint32_t*>(p.ws) + cta * kFlagWords;
    float* meta = reinterpret_cast<float*>(p.ws + Workspace::meta_offset(G)) + 2 * cta;
    uint8_t* slots = p.ws + Workspace::slots_offset(G) + (size_t)cta * 4 * kStateBytes;
    const float log2_scale = log2f(p.scale);
    uint32_t cnt = 0, tn = 0, qn = 0, un = 0, mn = 0, stn = 0;
    uint32_t pubs0 = 0, pubs1 = 0, ins0 = 0, ins1 = 0;   // uses of this CTA's slots, by parity
    float S[64];
    float s_up = 1.f;   // f16: the copy of S is S / s_up

    // kS and kML may be written again: earlier bulk stores have read them
    auto acquire_stage = [&] {
      if (tid == 0) bulk_wait_read_all();
      named_bar_sync(1, kCompute);
    };
    // the largest value over the compute threads (f16)
    auto reduce_max = [&](float m) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      if (lane == 0) misc->red[warp] = m;
      named_bar_sync(1, kCompute);
      m = misc->red[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) m = fmaxf(m, misc->red[i]);
      named_bar_sync(1, kCompute);
      return m;
    };
    // the rounded copy of S
    auto write_copy = [&] {
      float down = 1.f;
      if constexpr (kF16) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 64; ++i) m = fmaxf(m, fabsf(S[i]));
        const int e = exponent_of(reduce_max(m)) - 14;   // the largest below 2^15
        s_up = pow2i(e);
        down = pow2i(-e);
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = kF16 ? S[8 * c + i] * down : S[8 * c + i];
        *reinterpret_cast<uint4*>(sm + kS + wg * 16384 + row * 128 + ((c ^ (row & 7)) << 4)) = pack8<T>(x);
      }
      fence_async_smem();
      arrive_warp(&bars[kSReady]);
    };
    // K~'s terms for tokens 64 hf .. 64 hf + 63 of the block: the first over K itself
    auto make_terms = [&](int hf, uint32_t kt, uint32_t buf, float up) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = (tid >> 4) + 16 * i, c = tid & 15;         // token in the half, 16-byte chunk
        const uint32_t in_row = ((c & 7) ^ (r & 7)) << 4;
        uint4* src = reinterpret_cast<uint4*>(sm + kt + (c >> 3) * 16384 + (64 * hf + r) * 128 + in_row);
        uint8_t* dst = sm + buf + (c >> 3) * 8192 + r * 128 + in_row;
        const float w = tab_w[64 * hf + r] * (kF16 ? up : 1.f);
        float x[8], y[8];
        unpack8<T>(*src, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = w != 0.f ? x[e] * w : 0.f;   // (rows behind the sequence may hold anything)
#pragma unroll
        for (int term = 0; term < kTerms; ++term) {
          const uint4 v = pack8<T>(x);
          if (term == 0)
            *src = v;
          else
            *reinterpret_cast<uint4*>(dst + (term - 1) * 16384) = v;
          if (term + 1 < kTerms) {
            unpack8<T>(v, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] -= y[e];
          }
        }
      }
      fence_async_smem();
      arrive_warp(&bars[kKt0 + hf]);
    };
    // f16: the power of two that brings the block's |w k| below 2^14
    auto term_scale = [&](uint32_t kt, int L) {
      __half2 m = __half2half2(__ushort_as_half(0));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = (tid >> 4) + 16 * i, c = tid & 15;
        if (r < L) {
          const uint4 v =
              *reinterpret_cast<const uint4*>(sm + kt + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
          const __half2* h = reinterpret_cast<const __half2*>(&v);
#pragma unroll
          for (int e = 0; e < 4; ++e) m = __hmax2(m, __habs2(h[e]));
        }
      }
      const float2 f = __half22float2(m);
      return exponent_of(reduce_max(fmaxf(f.x, f.y)) * misc->w_max) - 13;
    };
    // rows of V behind the sequence: zero (their weights are, but they may hold anything)
    auto clear_v = [&](uint32_t vt, int L) {
      for (int i = tid; i < (kB - L) * 16; i += kCompute) {
        const int r = L + (i >> 4), c = i & 15;
        *reinterpret_cast<uint4*>(sm + vt + (c >> 3) * 16384 + r * 128 + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
      }
      fence_async_smem();
    };
    // S <- exp(G_L) S + U
    auto update_state = [&](float gam, float down) {
      wait(&bars[kUFull], un++ & 1);
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float u[32];
        tmem_ld32(tl + kColU + 64 * wg + 32 * c, u);
#pragma unroll
        for (int i = 0; i < 32; ++i) S[32 * c + i] = fmaf(gam, S[32 * c + i], kF16 ? u[i] * down : u[i]);
      }
      tc_fence_before();
    };

    for (int item = cta; walk.find(p, item, it); item += G) {
      const int nb = (it.len + kB - 1) / kB, r = item / G, par = r & 1;
      const bool last = it.j + 1 == it.J;
      if (!last) {
        // --------------------------------------------------------- pass A ---
        acquire_stage();
#pragma unroll
        for (int i = 0; i < 64; ++i) S[i] = 0.f;
        float seg_gam = 1.f;
        for (int b = 0; b < nb; ++b, ++cnt) {
          const uint32_t s = cnt & 1, kt = kK + s * 32768;
          const int L = min(kB, it.len - b * kB);   // (only a last segment has a short block)
          wait(&bars[kTabFull], tn++ & 1);
          wait(&bars[kKvFull + s], (cnt >> 1) & 1);
          const float gam = misc->gam_l;
          seg_gam = misc->seg_gam;
          int e = 0;
          if constexpr (kF16) e = term_scale(kt, L);
          make_terms(0, kt, kML, pow2i(-e));
          make_terms(1, kt, kS, pow2i(-e));
          arrive_warp(&bars[kTabEmpty]);
          update_state(gam, pow2i(e));
        }
        const uint32_t used = par ? pubs1++ : pubs0++;
        if (tid == 0 && used > 0) wait.flag(flags + kScanned + par, kSlices * used);
        named_bar_sync(1, kCompute);
        float4* out = reinterpret_cast<float4*>(slots + (size_t)par * kStateBytes);
#pragma unroll
        for (int v = 0; v < 16; ++v)
          __stcg(out + 256 * v + tid, make_float4(S[4 * v], S[4 * v + 1], S[4 * v + 2], S[4 * v + 3]));
        if (tid == 0) __stcg(meta + par, seg_gam);
        named_bar_sync(1, kCompute);
        if (tid == 0) {
          fence_acq_rel_gpu();
          st_release_gpu(flags + kOutReady + par, r + 1);
        }
      }
      // ----------------------------------------------------------- pass B ---
      // the state that enters
      acquire_stage();
      if (it.j > 0) {
        const uint32_t use = par ? ++ins1 : ++ins0;
        if (lane == 0) wait.flag(flags + kInCnt + par, kSlices * use);
        __syncwarp();
        const float4* in = reinterpret_cast<const float4*>(slots + (size_t)(2 + par) * kStateBytes);
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const float4 x = __ldcg(in + 256 * v + tid);
          S[4 * v] = x.x; S[4 * v + 1] = x.y; S[4 * v + 2] = x.z; S[4 * v + 3] = x.w;
        }
      } else if (p.state_in) {
        const int boxes = (p.dk + 31) / 32;
        fence_async_smem();
        named_bar_sync(1, kCompute);
        if (tid == 0) {
          mbar_arrive_expect_tx(&bars[kStFull], boxes * 16384);
          for (int x = 0; x < boxes; ++x)
            tma_load_3d(sm + kStage + x * 16384, &sim, &bars[kStFull], 32 * x, 0, it.n * p.Hv + it.h);
        }
        wait(&bars[kStFull], stn++ & 1);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const int x = 2 * wg + (c >> 3);
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (x < boxes)
            v = *reinterpret_cast<const float4*>(sm + kStage + x * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
          S[4 * c] = v.x; S[4 * c + 1] = v.y; S[4 * c + 2] = v.z; S[4 * c + 3] = v.w;
        }
        named_bar_sync(1, kCompute);
      } else {
#pragma unroll
        for (int i = 0; i < 64; ++i) S[i] = 0.f;
      }
      if (nb > 0) write_copy();
      if (p.ws) {
        named_bar_sync(1, kCompute);   // every thread has its part
        if (tid == 0) st_release_gpu(flags + kDone, r + 1);
      }
      for (int b = 0; b < nb; ++b, ++cnt, ++qn) {
        const uint32_t s = cnt & 1, kt = kK + s * 32768, vt = kV + s * 32768;
        const int t = it.t0 + b * kB, L = min(kB, it.len - b * kB);
        const bool upd = last || b + 1 < nb;
        wait(&bars[kTabFull], tn++ & 1);
        wait(&bars[kKvFull + s], (cnt >> 1) & 1);
        const float gam = misc->gam_l, row_gam = tab_gam[row] * s_up;
        const bool big = misc->big != 0;
        if (L < kB) clear_v(vt, L);
        int e = 0;
        if constexpr (kF16) {
          if (upd) e = term_scale(kt, L);
        }
        acquire_stage();
        wait(&bars[kPFull], qn & 1);
        tc_fence_after();
        if (upd) make_terms(0, kt, kML, pow2i(-e));
        // P: 32 columns at a time, as packed pairs
        float p_up = 1.f;
        {
          const float gr = tab_gh[row] + log2_scale, grl = tab_gl[row];
          uint32_t u[32];
          auto scores = [&](float down) {
            float top = 0.f;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int cb = 2 * wg + c;               // columns 32 cb ..: zero above the diagonal
              if (cb > w4) {
#pragma unroll
                for (int i = 0; i < 16; ++i) u[16 * c + i] = 0u;
                continue;
              }
              float x[32];
              tmem_ld32(tl + kColP + 32 * cb, x);
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 h4 = *reinterpret_cast<const float4*>(tab_gh + 32 * cb + i);
                float d[4] = {gr - h4.x, gr - h4.y, gr - h4.z, gr - h4.w};
                if (big) {
                  const float4 l4 = *reinterpret_cast<const float4*>(tab_gl + 32 * cb + i);
                  // (the scale's logarithm joins the low parts: gr - h4 alone is exact where it matters)
                  d[0] = (tab_gh[row] - h4.x) + ((grl - l4.x) + log2_scale);
                  d[1] = (tab_gh[row] - h4.y) + ((grl - l4.y) + log2_scale);
                  d[2] = (tab_gh[row] - h4.z) + ((grl - l4.z) + log2_scale);
                  d[3] = (tab_gh[row] - h4.w) + ((grl - l4.w) + log2_scale);
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  const float v = x[i + y] * ex2(d[y]);
                  x[i + y] = (cb < w4 || i + y <= lane) && (!kF16 || row < L) ? v : 0.f;
                  if constexpr (kF16) {
                    top = fmaxf(top, fabsf(x[i + y]));
                    x[i + y] *= down;
                  }
                }
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) u[16 * c + i] = Op16<T>::pack2(x[2 * i], x[2 * i + 1]);
            }
            return top;
          };
          const float top = scores(1.f);
          if constexpr (kF16) {
            if (!named_bar_and(1, kCompute, top < 32768.f)) {
              const int pe = exponent_of(reduce_max(top)) - 14;
              p_up = pow2i(pe);
              scores(pow2i(-pe));
            }
          }
          tmem_st16(tl + kColP + 64 * wg, u);
          tmem_st16(tl + kColP + 64 * wg + 16, u + 16);
          tmem_wait_st();
          tc_fence_before();
          arrive_warp(&bars[kPt]);
        }
        if (upd) {
          wait(&bars[kMlFree], mn++ & 1);
          make_terms(1, kt, kML, pow2i(-e));
        }
        arrive_warp(&bars[kTabEmpty]);
        if (upd) {
          update_state(gam, pow2i(e));
        }
        wait(&bars[kOiDone], qn & 1);
        if (upd && b + 1 < nb) write_copy();
        // o, staged as [token][column] in kML
        wait(&bars[kOFull], qn & 1);
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float x[16], y[16];
          tmem_ld16(tl + kColOi + 64 * wg + 16 * c, x);
          tmem_ld16(tl + kColOa + 64 * wg + 16 * c, y);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = fmaf(row_gam, x[i], kF16 ? y[i] * p_up : y[i]);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            *reinterpret_cast<uint4*>(sm + kML + wg * 16384 + row * 128 + (((2 * c + i) ^ (row & 7)) << 4)) =
                pack8<T>(x + 8 * i);
        }
        tc_fence_before();
        arrive_warp(&bars[kOFree]);
        fence_async_smem();
        named_bar_sync(1, kCompute);
        if (L == kB) {
          if (tid == 0) {
            tma_store_3d(&om, sm + kML, 0, it.h, t);
            if (p.dv > 64) tma_store_3d(&om, sm + kML + 16384, 64, it.h, t);
            bulk_commit_group();
          }
        } else {
          T* o = static_cast<T*>(p.o);
          const int chunks = p.dv / 8;
          for (int i = tid; i < L * chunks; i += kCompute) {
            const int rr = i / chunks, c = i - rr * chunks;
            __stcs(reinterpret_cast<uint4*>(o + ((size_t)(t + rr) * p.Hv + it.h) * p.dv + 8 * c),
                   *reinterpret_cast<const uint4*>(sm + kML + (c >> 3) * 16384 + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)));
          }
        }
      }
      if (last) {
        // the state after the sequence; state_out may be state_in, whose reader is then the first segment
        if (it.J > 1 && tid == 0)
          wait.flag(reinterpret_cast<uint32_t*>(p.ws) + (it.first % G) * kFlagWords + kDone, it.first / G + 1);
        acquire_stage();
#pragma unroll
        for (int c = 0; c < 16; ++c)
          *reinterpret_cast<float4*>(sm + kStage + (2 * wg + (c >> 3)) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4)) =
              make_float4(S[4 * c], S[4 * c + 1], S[4 * c + 2], S[4 * c + 3]);
        fence_async_smem();
        named_bar_sync(1, kCompute);
        if (tid == 0) {
          for (int x = 0; 32 * x < p.dk; ++x)
            tma_store_3d(&som, sm + kStage + x * 16384, 32 * x, 0, it.n * p.Hv + it.h);
          bulk_commit_group();
        }
      }
    }
    if (tid == 0) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace ltc
}  // namespace gdn
