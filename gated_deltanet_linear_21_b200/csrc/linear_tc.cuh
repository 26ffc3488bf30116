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
// Four products a block, each 128 x 128 x 128: Q K^T, Q S^T, P V and K~^T V with
// K~_s = w_s k_s, w_s = exp(G_L - G_s). The state lives, transposed, in fp32 registers
// of the compute warps (64 values a thread); the tensor core reads a rounded copy of it,
// for o alone.
//
// Precision. o has 16 bits, so P and the copy of S that Q meets are rounded to the
// input type (half a step each, and no term of o carries both). The state is fp32, so
// K~ is not rounded but split into terms that are multiplied with V one after another
// into one accumulator. With w = w1 + w2 + w3 (each of the input type's precision)
// packed 16-bit arithmetic gives the terms without leaving the type:
//
//   hi = rn(w1 k), e1 = w1 k - hi (exact in one fma), h2 = rn(w2 k), t4 = w3 k + (w2 k - h2)
//
// 24 bits in bf16. f16 needs hi and rn(w2 k + e1), 22 bits; in bf16 the same two (16
// bits) serve where the state is only read for o, inside a segment that is not a
// sequence's last. In f16 powers of two keep what is rounded in the type's range: one
// from the block's largest |k| and w for the terms of K~, one from the largest |S| for
// the copy of S, and one for P where a score passes 2^15.
// Log-decays are summed in fp64 (exp(G_r - G_s) of far tokens is a difference of large
// sums) and clamped where exp is zero in fp32, so that a reset (-inf) does not turn
// differences into NaN. For tokens r, s of different quarters of the block the weight of
// P is the product of a factor of r and one of s, around the end of s's quarter; inside
// a quarter it is exp(G_r - G_s) itself.
//
// What bounds it. The data move once through HBM at 128 KB a block (fewer where heads
// share k and q); the products' operands pass shared memory (128 bytes a cycle), which
// is the tighter bound. So K~'s terms and P are tensor-memory operands: K~ is read from
// K's tile by ldmatrix with transposition, weighted in registers and stored to tensor
// memory, and no term ever lies in shared memory.
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
// ones. Four scan warps per CTA compute it: a warp owns 1/32 of one head's state,
// carries it in registers from segment to segment and hands every result to the
// CTA that waits for it. Heads are taken in panels of at most 4 G / 32, so each
// (head, 1/32) of a panel has an owner of its own.
//
// Roles. Warps 0-7 compute. Warp 8 walks the items, hands them to the others through a
// ring and loads K, V; warp 9 issues the products; warp 10 loads Q and computes the
// decay tables; warp 11, the courier, waits for and sets the flags in global memory, so
// that the compute warps wait for none of those; warps 12-15 scan.
//
// Order and progress. Items are numbered (sequence, panel, segment, head). Every
// wait on another CTA is for work of a lower number -- B(i) and scan(i) for scans
// and publications before i, a publication for the scan of the same slot's last
// but one user, a scan for the reading of a slot two rounds back -- so with all CTAs
// resident (cooperative launch) the lowest unfinished one can always go on. All
// waits are bounded, the compute warps' barrier among themselves too; a warp whose wait
// ran out leaves its loop.
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
constexpr int kLoadWarp = 8;         // items; K, V tiles
constexpr int kMmaWarp = 9;          // tensor-core work
constexpr int kGateWarp = 10;        // Q tiles and the decay tables
constexpr int kCourierWarp = 11;     // flags in global memory
constexpr int kScanWarp = 12;        // to 15
constexpr int kScanWarps = 4;
constexpr int kThreads = 32 * (kScanWarp + kScanWarps);
constexpr int kSlices = 32;          // owners of one head's state
// Registers: 512 threads start with 128 each; the compute warps' share grows by what
// the others give back (256 x 176 + 256 x 80 = 65536, all that the block holds).
constexpr int kRegsCompute = 176, kRegsOther = 80;
static_assert(kCompute * kRegsCompute + (kThreads - kCompute) * kRegsOther <= 65536, "register file");
constexpr int kStateBytes = kD * kD * 4;
constexpr float kMinLog = -105.f;  // exp is 0 in fp32, subnormals included

// ---- shared memory (bytes) ----
constexpr uint32_t kQ = 0;                     // [128][128] as two K-major 128B-swizzled atoms, 16 KB apart
constexpr uint32_t kK = 32768;                 // two buffers
constexpr uint32_t kV = 98304;                 // two buffers
constexpr uint32_t kS = 163840;                // the rounded copy of S, [d_k][d_v] as two MN-major atoms
constexpr uint32_t kO = 196608;                // o on its way out
constexpr uint32_t kStage = kS;                // kS and kO together: a state on its way in or out
constexpr uint32_t kTab = 229376;              // w (bf16: words wp1[64], wp2[64], wp3[64]; f16: float[128]), then
constexpr uint32_t kTabGam = kTab + 768;       // float gam[128], gp[128], gb[128]
constexpr uint32_t kBars = kTabGam + 1536;
constexpr uint32_t kRing = kBars + 256;        // items
constexpr uint32_t kMisc = kRing + 192;        // words: see Misc
constexpr uint32_t kSmem = kMisc + 256;
static_assert(kSmem <= 227 * 1024, "shared memory budget");
constexpr int kRingItems = 4;

enum Bar { kKvFull = 0, kKvEmpty = 2, kItFull = 4, kItEmpty = 8, kQFull = 12, kTabFull, kTabEmpty, kPFull, kKt, kPt, kUFull,
           kOFull, kStFull, kSlotFree, kPub, kInReady, kGot, kOutOk, kCBar, kNumBars };
static_assert(kNumBars * 8 <= 256, "barriers");

struct Misc {
  uint32_t tmem;
  float gam_l;         // exp(G_L) of the block
  float seg_gam;       // exp of the segment's total log-decay, up to this block
  float w_max;         // the largest w of the block
  float tot[4];        // the quarters' total log-decays (base 2)
  float red[2][8];     // reductions over the compute warps (f16)
};
static_assert(sizeof(Misc) <= 256, "shared memory budget");

// ---- tensor memory columns ----
// The terms of K~ lie where Q S^T and P V go later in the block: each K half (tokens
// 0-63, 64-127) in the 64 columns that the warps which write it also read o from.
constexpr uint32_t kColP = 0;        // Q K^T, then P in place (16 bits: columns 0-31 and 64-95)
constexpr uint32_t kColOi = 128;     // t4, h2; then Q S^T
constexpr uint32_t kColOa = 256;     // hi, e1 (or the second of two terms); then P V
constexpr uint32_t kColU = 384;      // K~^T V
constexpr uint32_t kColHi = kColOa, kColE1 = kColOa + 32, kColT4 = kColOi, kColH2 = kColOi + 32;

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
  // by the whole warp, which agrees on the outcome
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    ok = __all_sync(0xffffffffu, ok && mbar_wait(bar, parity, limit));
  }
  // by one lane
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

static_assert(sizeof(Item) * kRingItems <= 192, "shared memory budget");

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
// 16 lanes x 32 columns, as 8 x 8 matrices of 16-bit pairs: u[2 i + b] of thread t is row
// 8 b + t / 4 of the lanes, column 4 i + t % 4.
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
}
// Four 8 x 8 matrices of 16-bit values, transposed: thread t holds rows 2 (t % 4) and + 1 of
// column t / 4 of each.
__device__ __forceinline__ void ldmatrix_t4(uint32_t saddr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}
// Packed arithmetic on two values of the 16-bit type, rounded to nearest even.
template <typename T> struct Two;
template <> struct Two<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
  }
};
template <> struct Two<__half> {
  static __device__ __forceinline__ uint32_t mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
  }
};
__device__ __forceinline__ uint32_t neg2(uint32_t a) { return a ^ 0x80008000u; }

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
          // word x = v * 256 + t of a slot holds rows (d_v) 64 (t / 128) + 4 v .. + 3 of column t % 128
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int t = 128 * (sl & 1) + 32 * u + lane, col = t & 127, row = 64 * (t >> 7) + 4 * (sl >> 1);
            S[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p.state_in && row < p.dv && col < p.dk) {   // (d_v is a multiple of 4)
              const float* x = p.state_in + (((size_t)(n0 + i) * p.Hv + h0 + hl) * p.dv + row) * p.dk + col;
              S[u] = make_float4(__ldcg(x), __ldcg(x + p.dk), __ldcg(x + 2 * p.dk), __ldcg(x + 3 * p.dk));
            }
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
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kBars);
  Misc* misc = reinterpret_cast<Misc*>(sm + kMisc);
  Item* ring = reinterpret_cast<Item*>(sm + kRing);
  uint32_t* tab_wp = reinterpret_cast<uint32_t*>(sm + kTab);    // bf16: three words of pairs
  float* tab_w = reinterpret_cast<float*>(sm + kTab);           // f16
  float* tab_gam = reinterpret_cast<float*>(sm + kTabGam);      // exp(G_r) scale
  float* tab_gp = tab_gam + kB;                                 // log2 decay from the start of r's quarter to r
  float* tab_gb = tab_gam + 2 * kB;                             // exp of the decay from s to the end of its quarter
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = gridDim.x, cta = blockIdx.x;

  if (smem_u32(sm) & 1023u) {   // the swizzled tiles need it; never seen (no static shared memory)
    if (tid == 0) flag_error(kErrCheck);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      const bool warps = i == kTabEmpty || i == kKt || i == kPt || i == kPub || i == kGot || i == kCBar;
      const bool readers = i >= kItEmpty && i < kItEmpty + kRingItems;
      mbar_init(&bars[i], warps ? 8 : readers ? (p.ws ? 11 : 10) : 1);
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
  // the CTA's i-th item, false behind the last
  auto next_item = [&](uint32_t i, Item& it) {
    wait(&bars[kItFull + (i & 3)], (i >> 2) & 1);
    if (!wait.ok) return false;
    it = ring[i & 3];
    arrive_warp(&bars[kItEmpty + (i & 3)]);
    return it.n >= 0;
  };
  Item it;

  if (warp == kLoadWarp) {
    give_registers();
    // ------------------------------------------------- items; K, V tiles ---
    const uint64_t once = l2_evict_first_policy();
    Walk walk;
    uint32_t cnt = 0;
    bool more = true;
    for (uint32_t i = 0; more && wait.ok; ++i) {
      more = walk.find(p, cta + (int)i * G, it);
      if (!more) it.n = -1;
      if (i >= kRingItems) wait(&bars[kItEmpty + (i & 3)], ((i >> 2) - 1) & 1);
      if (lane == 0) ring[i & 3] = it;
      arrive_warp(&bars[kItFull + (i & 3)]);
      if (!more) break;
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
    for (uint32_t i = 0; next_item(i, it); ++i) {
      const int hq = it.h / (p.Hv / p.Hqk), nb = (it.len + kB - 1) / kB;
      for (int pass = it.j + 1 < it.J ? 0 : 1; pass < 2; ++pass) {
        double seg = 0.0;
        for (int b = 0; b < nb && wait.ok; ++b) {
          const int t = it.t0 + b * kB, L = min(kB, it.len - b * kB);
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int s = 4 * lane + e;
            const float gv = s < L ? p.g[(size_t)(t + s) * p.g_stride + it.h] : 0.f;
            x[e] = gv < kMinLog ? kMinLog : gv;
          }
          if (pass == 1) {
            if (qn > 0) wait(&bars[kOFull], (qn - 1) & 1);
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
          const double q0 = __shfl_sync(0xffffffffu, before, lane & 24), q1 = __shfl_sync(0xffffffffu, incl, lane | 7);
          seg += end;
          float w[4], gm[4], gp[4], gb[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const double Gs = before + c[e];
            w[e] = 4 * lane + e < L ? expf((float)(end - Gs)) : 0.f;
            gm[e] = expf((float)Gs) * p.scale;
            gp[e] = (float)((Gs - q0) * 1.4426950408889634);
            gb[e] = expf((float)(q1 - Gs));
          }
          float wm = fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3]));
          if constexpr (kF16) {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, off));
          }
          if (tn > 0) wait(&bars[kTabEmpty], (tn - 1) & 1);
          if constexpr (kF16) {
            reinterpret_cast<float4*>(tab_w)[lane] = make_float4(w[0], w[1], w[2], w[3]);
          } else {
#pragma unroll
            for (int term = 0; term < 3; ++term) {
              const uint32_t lo = Op16<T>::pack2(w[0], w[1]), hi = Op16<T>::pack2(w[2], w[3]);
              reinterpret_cast<uint2*>(tab_wp + 64 * term)[lane] = make_uint2(lo, hi);
              const float2 a = Op16<T>::unpack2(lo), d = Op16<T>::unpack2(hi);
              w[0] -= a.x; w[1] -= a.y; w[2] -= d.x; w[3] -= d.y;
            }
          }
          reinterpret_cast<float4*>(tab_gam)[lane] = make_float4(gm[0], gm[1], gm[2], gm[3]);
          reinterpret_cast<float4*>(tab_gp)[lane] = make_float4(gp[0], gp[1], gp[2], gp[3]);
          reinterpret_cast<float4*>(tab_gb)[lane] = make_float4(gb[0], gb[1], gb[2], gb[3]);
          if ((lane & 7) == 0) misc->tot[lane >> 3] = (float)((q1 - q0) * 1.4426950408889634);
          if (lane == 0) {
            misc->w_max = wm;
            misc->gam_l = expf((float)end);
            misc->seg_gam = expf((float)seg);
          }
          arrive_warp(&bars[kTabFull]);
          ++tn;
        }
      }
    }
    if (qn > 0) mbar_wait(&bars[kQFull], (qn - 1) & 1, p.limit);
  } else if (warp == kMmaWarp) {
    give_registers();
    // ------------------------------------------------- tensor-core work ---
    constexpr uint32_t id_qk = idesc_f16kind(128, 128, false, false, kFmt);   // both K-major
    constexpr uint32_t id_mn = idesc_f16kind(128, 128, false, true, kFmt);    // B MN-major
    uint32_t cnt = 0, qn = 0, un = 0;
    for (uint32_t i = 0; next_item(i, it); ++i) {
      const int nb = (it.len + kB - 1) / kB;
      const bool last = it.j + 1 == it.J;
      for (int pass = last ? 1 : 0; pass < 2; ++pass) {
        for (int b = 0; b < nb && wait.ok; ++b, ++cnt) {
          const uint32_t s = cnt & 1;
          const uint32_t kt = sbase + kK + s * 32768;
          const uint64_t vd = desc_mnmajor(sbase + kV + s * 32768, 0, 128, 16384);
          const uint64_t vd4 = desc_advance(vd, 4 * 2048);
          const bool upd = pass == 0 || last || b + 1 < nb;   // the state after the segment comes from pass A
          const bool four = !kF16 && (pass == 0 || last);
          wait(&bars[kKvFull + s], (cnt >> 1) & 1);
          if (pass == 1) {
            wait(&bars[kQFull], qn & 1);
            tc_fence_after();
            const uint64_t qd = desc_kmajor(sbase + kQ, 0, 16384), kd = desc_kmajor(kt, 0, 16384);
            mma_run_warp<4, 2, 2>(tmem + kColP, qd, kd, id_qk, 0);
            mma_run_warp<4, 2, 2>(tmem + kColP, desc_advance(qd, 16384), desc_advance(kd, 16384), id_qk, 1);
            mma_commit_warp(&bars[kPFull]);
          }
          if (upd) {
            wait(&bars[kKt], un++ & 1);
            tc_fence_after();
            auto term = [&](uint32_t col, uint32_t acc) {
              mma4_tmem_a_run_warp<128>(tmem + kColU, tmem + col, vd, id_mn, acc);
              mma4_tmem_a_run_warp<128>(tmem + kColU, tmem + col + 64, vd4, id_mn, 1);
            };
            term(kColE1, 0);
            if (four) {
              term(kColH2, 1);
              term(kColT4, 1);
            }
            term(kColHi, 1);
            mma_commit_warp(&bars[kUFull]);
          }
          if (pass == 1) {
            wait(&bars[kPt], qn & 1);
            tc_fence_after();
            const uint64_t qd = desc_kmajor(sbase + kQ, 0, 16384), sd = desc_mnmajor(sbase + kS, 0, 128, 16384);
            mma_run_warp<4, 2, 128>(tmem + kColOi, qd, sd, id_mn, 0);
            mma_run_warp<4, 2, 128>(tmem + kColOi, desc_advance(qd, 16384), desc_advance(sd, 4 * 2048), id_mn, 1);
            mma4_tmem_a_run_warp<128>(tmem + kColOa, tmem + kColP, vd, id_mn, 0);
            mma4_tmem_a_run_warp<128>(tmem + kColOa, tmem + kColP + 64, vd4, id_mn, 1);
            mma_commit_warp(&bars[kOFull]);
            ++qn;
          }
          mma_commit_warp(&bars[kKvEmpty + s]);
        }
      }
    }
  } else if (warp == kCourierWarp) {
    give_registers();
    // ---------------------------------------------- flags in global memory ---
    if (p.ws) {
      uint32_t* all = reinterpret_cast<uint32_t*>(p.ws);
      uint32_t* flags = all + cta * kFlagWords;
      uint32_t pubs0 = 0, pubs1 = 0, ins0 = 0, ins1 = 0, pn = 0;   // uses of this CTA's slots, by parity
      for (uint32_t i = 0; next_item(i, it); ++i) {
        const int par = i & 1;
        const bool last = it.j + 1 == it.J;
        if (!last) {
          const uint32_t used = par ? pubs1++ : pubs0++;
          if (lane == 0 && used > 0) wait.flag(flags + kScanned + par, kSlices * used);
          arrive_warp(&bars[kSlotFree]);
          wait(&bars[kPub], pn++ & 1);
          if (lane == 0) {
            fence_acq_rel_gpu();
            st_release_gpu(flags + kOutReady + par, i + 1);
          }
        }
        if (it.j > 0) {
          const uint32_t use = par ? ++ins1 : ++ins0;
          if (lane == 0) wait.flag(flags + kInCnt + par, kSlices * use);
          arrive_warp(&bars[kInReady]);
        }
        wait(&bars[kGot], i & 1);
        if (lane == 0) {
          fence_acq_rel_gpu();
          st_release_gpu(flags + kDone, i + 1);
        }
        if (last && it.J > 1) {
          // state_out may be state_in, whose reader is then the first segment
          if (lane == 0) wait.flag(all + (it.first % G) * kFlagWords + kDone, it.first / G + 1);
          arrive_warp(&bars[kOutOk]);
        }
      }
    }
  } else if (warp >= kScanWarp) {
    give_registers();
    // ------------------------------------- states between the segments ---
    if (p.ws) scan_role(p, cta * kScanWarps + warp - kScanWarp, G);
  } else {
    take_registers();
    // ----------------------------------------------------- compute warps ---
    // Warp w4 of each half wg has lanes 32 w4 .. of tensor memory: rows (tokens) of P and
    // o, columns (d_k) of K~ and of the state. wg: the half of the tokens of K~, of the
    // columns of P, and of d_v in o and the state.
    const int wg = warp >> 2, w4 = warp & 3, row = 32 * w4 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * w4) << 16);
    float* meta = reinterpret_cast<float*>(p.ws + Workspace::meta_offset(G)) + 2 * cta;
    uint8_t* slots = p.ws + Workspace::slots_offset(G) + (size_t)cta * 4 * kStateBytes;
    const float log2_scale = log2f(p.scale);
    uint32_t cnt = 0, tn = 0, qn = 0, un = 0, stn = 0, pn = 0, inn = 0, okn = 0, bn = 0, rn = 0;
    float S[64];        // S[64 wg + i][row]
    float s_up = 1.f;   // f16: the copy of S is S / s_up

    // the compute warps' barrier
    auto sync = [&] {
      arrive_warp(&bars[kCBar]);
      wait(&bars[kCBar], bn++ & 1);
    };
    // the largest value over the compute threads (f16)
    auto reduce_max = [&](float m) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      float* red = misc->red[rn++ & 1];   // (the one used two reductions ago: a barrier lies between)
      if (lane == 0) red[warp] = m;
      sync();
      m = red[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) m = fmaxf(m, red[i]);
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
    };
    // The terms of K~ for tokens 64 wg .. + 63 and columns 32 w4 .. + 31 of K's tile at kt.
    // Returns the power of two that they were multiplied with (f16).
    const uint32_t ldm_row = 64 * wg + 8 * ((lane >> 4) & 1) + (lane & 7);
    auto make_terms = [&](uint32_t kt, int L, bool four) -> int {
      uint32_t kr[32];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t c = 4 * w4 + 2 * half + ((lane >> 3) & 1);     // 16-byte chunk of K's row
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const uint32_t r = ldm_row + 8 * i;
          ldmatrix_t4(sbase + kt + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4), kr + 16 * half + 2 * i);
        }
      }
      if (L < kB) {   // rows behind the sequence may hold anything
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int t = 64 * wg + 8 * i + 2 * (lane & 3);
          const uint32_t keep = (t < L ? 0xffffu : 0u) | (t + 1 < L ? 0xffff0000u : 0u);
          kr[2 * i] &= keep; kr[2 * i + 1] &= keep; kr[16 + 2 * i] &= keep; kr[17 + 2 * i] &= keep;
        }
      }
      uint32_t w1[8], w2[8], w3[8];
      int e = 0;
      if constexpr (kF16) {
        __half2 m = __half2half2(__ushort_as_half(0));
#pragma unroll
        for (int i = 0; i < 32; ++i) m = __hmax2(m, __habs2(*reinterpret_cast<__half2*>(&kr[i])));
        const float2 f = __half22float2(m);
        // |w k| below 2^14 and w below 2^15
        e = min(13 - exponent_of(reduce_max(fmaxf(f.x, f.y)) * misc->w_max), 14 - exponent_of(misc->w_max));
        const float up = pow2i(e);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float2 w = *reinterpret_cast<const float2*>(tab_w + 64 * wg + 8 * i + 2 * (lane & 3));
          w.x *= up; w.y *= up;
          w1[i] = Op16<T>::pack2(w.x, w.y);
          const float2 x = Op16<T>::unpack2(w1[i]);
          w2[i] = Op16<T>::pack2(w.x - x.x, w.y - x.y);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t at = 32 * wg + 4 * i + (lane & 3);
          w1[i] = tab_wp[at];
          w2[i] = tab_wp[64 + at];
          w3[i] = tab_wp[128 + at];
        }
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t tw = tl + (static_cast<uint32_t>(16 * half) << 16) + 64 * wg;
        uint32_t x[16], y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          x[i] = Two<T>::mul(w1[i >> 1], kr[16 * half + i]);
          y[i] = Two<T>::fma(w1[i >> 1], kr[16 * half + i], neg2(x[i]));
        }
        tmem_st_frag(tw + kColHi, x);
        if (four) {
          tmem_st_frag(tw + kColE1, y);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = Two<T>::mul(w2[i >> 1], kr[16 * half + i]);
          tmem_st_frag(tw + kColH2, x);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            y[i] = Two<T>::fma(w2[i >> 1], kr[16 * half + i], neg2(x[i]));
            if constexpr (!kF16) y[i] = Two<T>::fma(w3[i >> 1], kr[16 * half + i], y[i]);
          }
          tmem_st_frag(tw + kColT4, y);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = Two<T>::fma(w2[i >> 1], kr[16 * half + i], y[i]);
          tmem_st_frag(tw + kColE1, y);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      arrive_warp(&bars[kKt]);
      return e;
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
    // P, packed, over Q K^T. Returns the power of two that it was divided by (f16).
    auto make_scores = [&](int L) -> float {
      const float gr = tab_gp[row] + log2_scale;
      uint32_t u[32];
      auto scores = [&](float down) {
        float top = 0.f, far = 0.f;
#pragma unroll
        for (int c = 1; c >= 0; --c) {
          const int cb = 2 * wg + c;               // columns 32 cb ..: zero above the diagonal
          if (cb > w4) {
#pragma unroll
            for (int i = 0; i < 16; ++i) u[16 * c + i] = 0u;
            continue;
          }
          float x[32];
          tmem_ld32(tl + kColP + 32 * cb, x);
          if (cb == w4) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 h4 = *reinterpret_cast<const float4*>(tab_gp + 32 * cb + i);
              const float d[4] = {gr - h4.x, gr - h4.y, gr - h4.z, gr - h4.w};
#pragma unroll
              for (int y = 0; y < 4; ++y) x[i + y] = i + y <= lane ? x[i + y] * ex2(d[y]) : 0.f;
            }
          } else {
            far = 0.f;
            for (int y = cb + 1; y < w4; ++y) far += misc->tot[y];
            const float a = ex2(gr + far);
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 b4 = *reinterpret_cast<const float4*>(tab_gb + 32 * cb + i);
              x[i] *= b4.x * a; x[i + 1] *= b4.y * a; x[i + 2] *= b4.z * a; x[i + 3] *= b4.w * a;
            }
          }
          if constexpr (kF16) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              top = fmaxf(top, fabsf(x[i]));
              x[i] *= down;
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) u[16 * c + i] = Op16<T>::pack2(x[2 * i], x[2 * i + 1]);
        }
        return row < L ? top : 0.f;
      };
      const float top = scores(1.f);
      float up = 1.f;
      if constexpr (kF16) {
        const float most = reduce_max(top);
        if (most >= 32768.f) {
          const int e = exponent_of(most) - 14;
          up = pow2i(e);
          scores(pow2i(-e));
        }
      }
      tmem_st16(tl + kColP + 64 * wg, u);
      tmem_st16(tl + kColP + 64 * wg + 16, u + 16);
      tmem_wait_st();
      tc_fence_before();
      arrive_warp(&bars[kPt]);
      return up;
    };
    // o of this warp's 32 tokens and 64 columns, through its own part of kO
    uint8_t* o_stage = sm + kO + wg * 16384 + w4 * 4096;
    const int o_chunks = min(8, max(0, p.dv / 8 - 8 * wg));    // 16-byte chunks of these columns
    auto write_o = [&](int t, int h, int L, float row_gam, float up) {
      if (o_chunks == 0) return;
      if (lane == 0) bulk_wait_read_all();
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float x[16], y[16];
        tmem_ld16(tl + kColOi + 64 * wg + 16 * c, x);
        tmem_ld16(tl + kColOa + 64 * wg + 16 * c, y);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = fmaf(row_gam, x[i], kF16 ? y[i] * up : y[i]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          *reinterpret_cast<uint4*>(o_stage + lane * 128 + (((2 * c + i) ^ (lane & 7)) << 4)) = pack8<T>(x + 8 * i);
      }
      tc_fence_before();
      const int rows = min(32, L - 32 * w4);
      if (rows == 32) {
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&om, o_stage, 64 * wg, h, t + 32 * w4);
          bulk_commit_group();
        }
      } else {
        __syncwarp();
        T* o = static_cast<T*>(p.o);
        for (int i = lane; i < rows * o_chunks; i += 32) {
          const int r = i / o_chunks, c = i - r * o_chunks;
          __stcs(reinterpret_cast<uint4*>(o + ((size_t)(t + 32 * w4 + r) * p.Hv + h) * p.dv + 64 * wg + 8 * c),
                 *reinterpret_cast<const uint4*>(o_stage + r * 128 + ((c ^ (r & 7)) << 4)));
        }
      }
    };
    // element (d_v 64 wg + i, d_k row) of a staged state: boxes of 32 columns, 128-byte rows
    auto staged = [&](int i) {
      const int v = 64 * wg + i;
      return reinterpret_cast<float*>(sm + kStage + w4 * 16384 + v * 128 + (((lane >> 2) ^ (v & 7)) << 4) + (lane & 3) * 4);
    };

    for (uint32_t i = 0; next_item(i, it); ++i) {
      const int nb = (it.len + kB - 1) / kB, par = i & 1;
      const bool last = it.j + 1 == it.J;
      if (!last) {
        // --------------------------------------------------------- pass A ---
#pragma unroll
        for (int x = 0; x < 64; ++x) S[x] = 0.f;
        float seg_gam = 1.f;
        for (int b = 0; b < nb && wait.ok; ++b, ++cnt) {
          const uint32_t s = cnt & 1;
          wait(&bars[kTabFull], tn++ & 1);
          wait(&bars[kKvFull + s], (cnt >> 1) & 1);
          const float gam = misc->gam_l;
          seg_gam = misc->seg_gam;
          const int e = make_terms(kK + s * 32768, kB, !kF16);   // (only a last segment has a short block)
          arrive_warp(&bars[kTabEmpty]);
          update_state(gam, pow2i(-e));
        }
        wait(&bars[kSlotFree], pn++ & 1);
        float4* out = reinterpret_cast<float4*>(slots + (size_t)par * kStateBytes);
#pragma unroll
        for (int v = 0; v < 16; ++v)
          __stcg(out + 256 * v + tid, make_float4(S[4 * v], S[4 * v + 1], S[4 * v + 2], S[4 * v + 3]));
        if (tid == 0) __stcg(meta + par, seg_gam);
        arrive_warp(&bars[kPub]);
      }
      // ----------------------------------------------------------- pass B ---
      // the state that enters
      if (it.j > 0) {
        wait(&bars[kInReady], inn++ & 1);
        const float4* in = reinterpret_cast<const float4*>(slots + (size_t)(2 + par) * kStateBytes);
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const float4 x = __ldcg(in + 256 * v + tid);
          S[4 * v] = x.x; S[4 * v + 1] = x.y; S[4 * v + 2] = x.z; S[4 * v + 3] = x.w;
        }
      } else if (p.state_in) {
        const int boxes = (p.dk + 31) / 32;
        if (lane == 0) bulk_wait_read_all();   // (what went out through kS and kO)
        fence_async_smem();
        sync();
        if (tid == 0) {
          mbar_arrive_expect_tx(&bars[kStFull], boxes * 16384);
          for (int x = 0; x < boxes; ++x)
            tma_load_3d(sm + kStage + x * 16384, &sim, &bars[kStFull], 32 * x, 0, it.n * p.Hv + it.h);
        }
        wait(&bars[kStFull], stn++ & 1);
#pragma unroll
        for (int x = 0; x < 64; ++x) S[x] = w4 < boxes ? *staged(x) : 0.f;
        sync();
      } else {
#pragma unroll
        for (int x = 0; x < 64; ++x) S[x] = 0.f;
      }
      if (nb > 0) {
        // kS may be a state's on its way out (thread 0's stores)
        if (i > 0 && !(it.j == 0 && p.state_in)) {
          if (tid == 0) bulk_wait_read_all();
          sync();
        }
        write_copy();
      }
      if (p.ws) arrive_warp(&bars[kGot]);
      for (int b = 0; b < nb && wait.ok; ++b, ++cnt, ++qn) {
        const uint32_t s = cnt & 1;
        const int t = it.t0 + b * kB, L = min(kB, it.len - b * kB);
        const bool upd = last || b + 1 < nb;
        wait(&bars[kTabFull], tn++ & 1);
        wait(&bars[kKvFull + s], (cnt >> 1) & 1);
        const float gam = misc->gam_l, row_gam = tab_gam[row] * s_up;
        if (L < kB) clear_v(kV + s * 32768, L);
        int e = 0;
        if (upd) e = make_terms(kK + s * 32768, L, !kF16 && last);
        wait(&bars[kPFull], qn & 1);
        tc_fence_after();
        const float up = make_scores(L);
        arrive_warp(&bars[kTabEmpty]);
        if (upd) update_state(gam, pow2i(-e));
        wait(&bars[kOFull], qn & 1);
        tc_fence_after();
        write_o(t, it.h, L, row_gam, up);
        if (upd && b + 1 < nb) write_copy();
      }
      if (last) {
        // the state after the sequence
        if (it.J > 1) wait(&bars[kOutOk], okn++ & 1);
        if (lane == 0) bulk_wait_read_all();
        sync();
#pragma unroll
        for (int x = 0; x < 64; ++x) *staged(x) = S[x];
        fence_async_smem();
        sync();
        if (tid == 0) {
          for (int x = 0; 32 * x < p.dk; ++x)
            tma_store_3d(&som, sm + kStage + x * 16384, 32 * x, 0, it.n * p.Hv + it.h);
          bulk_commit_group();
        }
      }
    }
    if (lane == 0) bulk_wait_all();
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
