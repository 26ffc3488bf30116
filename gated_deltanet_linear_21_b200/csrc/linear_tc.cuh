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
// o is computed as rho_r (q_r S + sum_s P'_rs v_s), rho_r = scale exp(G_r), P'_rs =
// exp(-G_s) q_r . k_s, so that both products go to one accumulator and a score's weight
// depends on its column alone. That is exact while exp(-G_s) stays in range; a steep block
// (2^60 or more) takes a power of two 2^-m_r out of its late rows, from P' by the exponent
// and from q_r, after Q K^T, exactly.
//
// Four products a block, each 128 x 128 x 128: Q K^T, Q S^T, P' V and K~^T V with
// K~_s = w_s k_s, w_s = exp(G_L - G_s). The state lives, transposed, in fp32 registers
// of the compute warps (64 values a thread); the tensor core reads a rounded copy of it,
// for o alone.
//
// Precision. o has 16 bits, so P' and the copy of S that Q meets are rounded to the
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
// from the block's largest |w k| for the terms of K~ (where a column's largest is some 2^-11
// of it or less, or w falls by 2^-18, one for each column, and the terms come from fp32 products); 2^-b for the copy of S; and for
// each row r, whose P' and q meet v and that copy in one accumulator, 2^-a_r for P' and
// 2^(b - a_r) for q (rho_r holds 2^a_r). No row's or state's size then bears on another's
// precision: a row's largest score (or q, if that is larger) is at 2^14, or q keeps its size
// and the score is at 2^3 or above; the largest |S| is at 2^5; what is far below rounds to a
// multiple of 2^-24. Rows whose scores outweigh their part of the state lose low bits of q so:
// with |S| at 2^5 that is below 2^-25 of the row's largest score.
// Log-decays are summed in fp64 (exp(G_r - G_s) of far tokens is a difference of large
// sums) and clamped where exp is zero in fp32, so that a reset (-inf) does not turn
// differences into NaN. What meets a token once -- w, rho, exp(-G_s) -- is ex2.approx of them,
// 2^-22 relative. The decays that the state is carried with come back every block where
// the decay is fixed, so they are exp2 in fp64: a block's rounded to fp32 (at most 8 follow
// one another in a segment), a segment's in two floats.
//
// Infinities and NaN. Scores above the diagonal are zeros, and zero times a NaN of V is one: it
// reaches the rows of its column in front of its token, as far as the block goes. It also
// stays in the state (in what a segment adds to it, where that is looked at), so one look an
// item finds it, and those rows are then made again, token by token, from the state that
// entered.
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
// that the compute warps wait for none of those; warps 12-15 scan. Sixteen compute warps
// with half the columns each were slower (560 against 456 us on eight packed sequences).
//
// Measured (bf16): 4096 tokens, 16 heads 55 to 56 us; eight packed sequences of 128 to 8192
// tokens, 32 heads 435 to 448 us, 780 MB, so 1.8 TB/s; 64 of 20 to 300 tokens 175 us; f16, 32768
// tokens, 32 heads 517 to 544 us. A block takes the compute warps 5200 to 5900 cycles in pass B and
// 4000 to 5000 in pass A (f16 some 8 % more: its powers of two), its products 2560 and 2048: what
// bounds it is their instructions and waits. Neither fewer spilled registers nor tiles brought to
// L2 ahead change that. Steep blocks cost more: 4096 tokens with g = -1 62 us (f16 78).
// What finds infinities in V costs 1 to 4 %; looking through each block of V ahead, 7 to 14 %.
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
constexpr int kComputeWarps = 8;     // warps 0-7
constexpr int kCompute = 32 * kComputeWarps;
constexpr int kLoadWarp = 8;         // items; K, V tiles
constexpr int kMmaWarp = 9;          // tensor-core work
constexpr int kGateWarp = 10;        // Q tiles and the decay tables
constexpr int kCourierWarp = 11;     // flags in global memory
constexpr int kScanWarp = 12;        // to 15
constexpr int kScanWarps = 4;
constexpr int kWarps = kScanWarp + kScanWarps;
constexpr int kThreads = 32 * kWarps;
constexpr int kSlices = 32;          // owners of one head's state
// Registers: 512 threads start with 128 each; the compute warps' share grows by what the
// others give back (256 x 176 + 256 x 80 = 65536, all that the block holds).
constexpr int kRegsCompute = 176, kRegsOther = 80;
static_assert(kLoadWarp == kComputeWarps && kComputeWarps % 4 == 0 && kWarps % 4 == 0, "whole groups of four warps");
static_assert(kCompute * kRegsCompute + (kThreads - kCompute) * kRegsOther <= kThreads * 128, "register file");
constexpr int kStateBytes = kD * kD * 4;
constexpr float kInf = __builtin_huge_valf();
constexpr float kMinLog = -105.f;  // exp is 0 in fp32, subnormals included

// A block is steep when its log-decay (base 2) reaches this: P' = exp(-G_s) q_r . k_s and its
// products with V are fp32 and in bf16 have no other scale, so |q . k| |v| stays below 2^67.
constexpr int kSteep = 60;

// ---- shared memory (bytes) ----
constexpr uint32_t kQ = 0;                     // two buffers of [128][128], two K-major 128B-swizzled atoms 16 KB apart;
                                               // o goes out through the buffer that its Q came in
constexpr uint32_t kK = 65536;                 // two buffers
constexpr uint32_t kV = 131072;                // two buffers
constexpr uint32_t kS = 196608;                // the rounded copy of S, [d_k][d_v] as two MN-major atoms
constexpr uint32_t kTab = 229376;              // w (bf16: words wp1[64], wp2[64], wp3[64]; f16: float[128]), then
constexpr uint32_t kTabGam = kTab + 768;       // float gam[128], gp[128], gb[128]
constexpr uint32_t kBars = kTabGam + 1536;
constexpr uint32_t kRing = kBars + 320;        // items
constexpr uint32_t kMisc = kRing + 192;        // words: see Misc
constexpr uint32_t kSmem = kMisc + 256;
static_assert(kSmem <= 227 * 1024, "shared memory budget");
constexpr int kRingItems = 4;

// A barrier's waiters go by the parity of its phase, so none may complete a second phase
// before all of them have seen the first: each next completion has to need something that
// they do after that wait. Hence two barriers for pass A's two accumulators (kUFull,
// kURead) and four, as many as there are ring items, for kGot: the courier may fall behind
// the compute warps by that many and hands its item back after it. kGot is also what keeps
// the courier from the next kInReady and kOutOk until all warps have seen this item's: they
// arrive on it after those waits.
enum Bar { kKvFull = 0, kKvEmpty = 2, kItFull = 4, kItEmpty = 8, kGot = 12, kUFull = 16, kURead = 18, kKt = 20, kHalf = 22,
           kQFull = 24, kQFree = 26, kTabEmpty = 28, kPFull, kSReady, kOFull, kSlotFree, kPub, kInReady, kOutOk, kCBar,
           kLeft, kNumBars };
static_assert(kNumBars * 8 <= 320, "barriers");

struct Misc {
  uint32_t tmem;
  uint32_t dead;       // a wait ran out
  float gam_l;         // exp(G_L) of the block
  float2 seg_gam;      // exp of the segment's total log-decay, in two parts (pass A's last block)
  float w_max, w_min;  // the largest and the smallest w of the block's tokens (f16)
  uint32_t steep;      // exp(-G) reaches 2^kSteep in the block
  int start_i[4];      // the log-decays (base 2) up to each quarter: whole part
  float start_f[4];    // and the rest
  float red[2][2][kComputeWarps];   // reductions over the compute warps (f16)
};
static_assert(sizeof(Misc) <= 256, "shared memory budget");

// ---- tensor memory columns ----
// Each of two terms of K~ has 32 columns for either half of the tokens (0-63, 64-127);
// pass A's other two lie where o goes in pass B. P', packed, takes the first half of either
// 64 columns of Q K^T.
constexpr uint32_t kColP = 0;        // Q K^T, then P' in place
constexpr uint32_t kColO = 128;      // Q S^T + P' V
constexpr uint32_t kColK = 256;      // terms of K~
constexpr uint32_t kColU = 384;      // K~^T V (pass A: every other block's over P)

// ---- workspace ----
constexpr int kFlagWords = 32;       // per CTA: out_ready[2], scanned[2], in_cnt[2], done
enum Flag { kOutReady = 0, kScanned = 2, kInCnt = 4, kDone = 6 };
struct Workspace {
  __host__ __device__ static constexpr size_t flags_bytes(int ctas) { return (size_t)ctas * kFlagWords * 4; }
  __host__ __device__ static constexpr size_t meta_offset(int ctas) { return flags_bytes(ctas); }       // float2 per (CTA, parity)
  __host__ __device__ static constexpr size_t slots_offset(int ctas) { return (flags_bytes(ctas) + (size_t)ctas * 16 + 1023) & ~size_t(1023); }
  // per CTA: two published states, two entering states
  __host__ __device__ static constexpr size_t bytes(int ctas) { return slots_offset(ctas) + (size_t)ctas * 4 * kStateBytes; }
};

struct Params {
  const void *q, *k, *v;
  const float* g;
  const float* state_in;
  const int32_t* cu_seqlens;
  void* o;
  float* state_out;
  uint8_t* ws;
  int g_stride, n_seqs, total_T, Hqk, Hv, dk, dv, seg, panel;
  int items;           // at most, of a cu_seqlens that keeps its rules
  float scale;
  long long limit;     // SM cycles that a wait lasts at most
};

// Waits give up once `dead` is set, and the roles leave their loops; the kernel's end
// reports it. Waits for a flag in global memory set it when their time is over, and for
// those on chip the watchdog (the last warp, once its scan is done) does when the kernel's is:
// so the wait itself, of which there are many, is five instructions long. The limit grows
// with the problem: a scan warp may wait for a sequence that comes at the end.
struct Wait {
  uint32_t dead;       // shared-memory address
  long long limit;
  __device__ __forceinline__ bool ok() const {
    uint32_t d;
    asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(d) : "r"(dead) : "memory");
    return d == 0;
  }
  __device__ __forceinline__ void give_up() const {
    asm volatile("st.volatile.shared.b32 [%0], 1;" ::"r"(dead) : "memory");
  }
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) const {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 d;\n\t"
        "W%=: mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1;\n\t"
        "@p bra D%=;\n\t"
        "ld.volatile.shared.b32 d, [%2];\n\t"
        "setp.eq.u32 q, d, 0;\n\t"
        "@q bra W%=;\n\t"
        "D%=:\n\t}" ::"r"(smem_u32(bar)),
        "r"(parity), "r"(dead)
        : "memory");
  }
  // the watchdog's: for the other warps to leave
  __device__ __forceinline__ void watch(uint64_t* left) const {
    const long long t0 = clock64();
    while (!mbar_try_wait(left, 0)) {
      if (clock64() - t0 > limit) {
        give_up();
        break;
      }
    }
  }
  // on a flag in global memory, by one lane
  __device__ __forceinline__ void flag(const uint32_t* p, uint32_t target) const {
    if (ok() && !wait_flag_geq(p, target, limit)) give_up();
  }
};

struct Item {
  int n, h, j, J;      // sequence, head, segment of J
  int hp;              // heads in the panel: the next segment's item is this many further
  int t0, len;         // the segment's first token and tokens
  int first;           // the item of segment 0 of this sequence and head
};

static_assert(sizeof(Item) * kRingItems <= 192, "shared memory budget");

// Finds items in increasing order (warp-collective). Sequences that overlap, as no valid
// cu_seqlens makes them, may have more items than an int counts: the first sequence that
// passes p.items ends the walk, and the scan's.
struct Walk {
  int n = 0;
  long long base = 0;
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
      const long long cnt = (long long)J * p.Hv;
      long long incl = cnt;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += x;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, base + incl > item);
      if (hit) {
        const int src = __ffs(hit) - 1;
        if (base + __shfl_sync(0xffffffffu, incl, src) > p.items) return false;
        n += src;
        base += __shfl_sync(0xffffffffu, incl - cnt, src);
        J = __shfl_sync(0xffffffffu, J, src);
        a = __shfl_sync(0xffffffffu, a, src);
        len = __shfl_sync(0xffffffffu, len, src);
        const int li = (int)(item - base), per = J * p.panel, pi = li / per, rem = li - pi * per;
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
// Twice 32 columns of 32 lanes, waited for together.
__device__ __forceinline__ void tmem_ld32x2(uint32_t ta, uint32_t tb, float* x, float* y) {
  uint32_t u[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31]), "=r"(u[32]),
        "=r"(u[33]), "=r"(u[34]), "=r"(u[35]), "=r"(u[36]), "=r"(u[37]), "=r"(u[38]), "=r"(u[39]), "=r"(u[40]),
        "=r"(u[41]), "=r"(u[42]), "=r"(u[43]), "=r"(u[44]), "=r"(u[45]), "=r"(u[46]), "=r"(u[47]), "=r"(u[48]),
        "=r"(u[49]), "=r"(u[50]), "=r"(u[51]), "=r"(u[52]), "=r"(u[53]), "=r"(u[54]), "=r"(u[55]), "=r"(u[56]),
        "=r"(u[57]), "=r"(u[58]), "=r"(u[59]), "=r"(u[60]), "=r"(u[61]), "=r"(u[62]), "=r"(u[63])
      : "r"(ta), "r"(tb)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    x[i] = __uint_as_float(u[i]);
    y[i] = __uint_as_float(u[32 + i]);
  }
}
__device__ __forceinline__ uint64_t l2_evict_normal_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}
__device__ __forceinline__ void st_relaxed_gpu(uint32_t* p, uint32_t v) {
  asm volatile("st.relaxed.gpu.global.b32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void red_add_relaxed_gpu(uint32_t* p, uint32_t v) {
  asm volatile("red.relaxed.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t neg2(uint32_t a) { return a ^ 0x80008000u; }

__device__ __forceinline__ void tmem_st1(uint32_t taddr, uint32_t u) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(u) : "memory");
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

// A value that the compiler does not take for a loop's invariant: it would write the loop
// out once for each outcome of a condition on it, and the instruction cache is small.
__device__ __forceinline__ bool each_time(bool x) {
  uint32_t y = x;
  asm volatile("" : "+r"(y));
  return y != 0;
}

__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// The scan warps: owner `ow` of 4 G carries its share of each panel's head.
__device__ __forceinline__ void scan_role(const Params& p, const Wait& wait, int ow, int G) {
  const int lane = threadIdx.x & 31;
  const int hl = ow / kSlices, sl = ow - hl * kSlices;
  const int seg_t = p.seg * kB;
  uint32_t* flags = reinterpret_cast<uint32_t*>(p.ws);
  const float2* meta = reinterpret_cast<const float2*>(p.ws + Workspace::meta_offset(G));
  uint8_t* slots = p.ws + Workspace::slots_offset(G);
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
      if (base + (long long)Jn * p.Hv > p.items) return;   // (as Walk)
      if (Jn > 1) {
        for (int h0 = 0; h0 < p.Hv; h0 += p.panel) {
          const int hp = min(p.panel, p.Hv - h0);
          if (hl >= hp) continue;
          float4 S[4];
          // word x = v * 256 + t of a slot holds rows (d_v) 64 (t / 128) + 4 v .. + 3 of column t % 128
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int col = 32 * u + lane, row = 64 * (sl & 1) + 4 * (sl >> 1);
            S[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p.state_in && row < p.dv && col < p.dk) {   // (d_v is a multiple of 4)
              const float* x = p.state_in + (((size_t)(n0 + i) * p.Hv + h0 + hl) * p.dv + row) * p.dk + col;
              S[u] = make_float4(__ldcg(x), __ldcg(x + p.dk), __ldcg(x + 2 * p.dk), __ldcg(x + 3 * p.dk));
            }
          }
          long long t0 = 0;
          for (int j = 0; j + 1 < Jn;) {
            // One look at the flags of up to two segments: lanes 0 and 1 whether segments j
            // and j + 1 are published, lanes 2 and 3 whether the slots that their results go
            // to have been read.
            const int jl = j + (lane & 1), item = base + h0 * Jn + jl * hp + hl;
            const int at = lane < 2 ? item : item + hp, c = at % G, r = at / G;
            const uint32_t need = lane < 2 ? r + 1 : max(r - 1, 0);
            bool ready = false;
            if (lane < 4 && jl + 1 < Jn && GDN_CHECK(item >= 0 && at < p.items))
              ready = ld_acquire_gpu(flags + c * kFlagWords + (lane < 2 ? kOutReady + (r & 1) : kDone)) >= need;
            const uint32_t bits = __ballot_sync(0xffffffffu, ready);
            const int m = (bits & 5u) != 5u ? 0 : (bits & 10u) != 10u ? 1 : 2;
            if (m == 0) {
              const long long now = clock64();
              if (t0 == 0) t0 = now;
              if (__any_sync(0xffffffffu, now - t0 > p.limit || !wait.ok())) {
                wait.give_up();
                return;
              }
              __nanosleep(20);
              continue;
            }
            t0 = 0;
            float4 L[2][4];
            float2 gam[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (x < m) {
                const int src = item - (lane & 1) * hp + x * hp, cs = src % G, rs = src / G;
                gam[x] = __ldcg(meta + 2 * cs + (rs & 1));
                const float4* from =
                    reinterpret_cast<const float4*>(slots + (size_t)(4 * cs + (rs & 1)) * kStateBytes) + 128 * sl;
#pragma unroll
                for (int u = 0; u < 4; ++u) L[x][u] = __ldcg(from + 32 * u + lane);
              }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (x < m) {
                const int dst = item - (lane & 1) * hp + (x + 1) * hp, cd = dst % G, rd = dst / G;
                float4* to = reinterpret_cast<float4*>(slots + (size_t)(4 * cd + 2 + (rd & 1)) * kStateBytes) + 128 * sl;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  S[u].x = fmaf(gam[x].x, S[u].x, fmaf(gam[x].y, S[u].x, L[x][u].x));
                  S[u].y = fmaf(gam[x].x, S[u].y, fmaf(gam[x].y, S[u].y, L[x][u].y));
                  S[u].z = fmaf(gam[x].x, S[u].z, fmaf(gam[x].y, S[u].z, L[x][u].z));
                  S[u].w = fmaf(gam[x].x, S[u].w, fmaf(gam[x].y, S[u].w, L[x][u].w));
                  __stcg(to + 32 * u + lane, S[u]);
                }
              }
            }
            __syncwarp();
            // lanes 0 (and 1): the published slot is free; 2 (and 3): the entering state is there
            if (lane < 4 && (lane & 1) < m) {
              fence_acq_rel_gpu();
              red_add_relaxed_gpu(flags + c * kFlagWords + (lane < 2 ? kScanned : kInCnt) + (r & 1), 1u);
            }
            j += m;
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

// kWhole: d_k = d_v = 128.
template <typename T, bool kWhole>
__global__ void __launch_bounds__(kThreads, 1)
prefill_kernel(const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap km,
               const __grid_constant__ CUtensorMap vm, const __grid_constant__ CUtensorMap om, const Params p) {
  constexpr bool kF16 = std::is_same<T, __half>::value;
  constexpr uint32_t kFmt = Op16<T>::kFmt;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kBars);
  Misc* misc = reinterpret_cast<Misc*>(sm + kMisc);
  Item* ring = reinterpret_cast<Item*>(sm + kRing);
  uint32_t* tab_wp = reinterpret_cast<uint32_t*>(sm + kTab);    // bf16: three words of pairs
  float* tab_w = reinterpret_cast<float*>(sm + kTab);           // f16
  float* tab_gam = reinterpret_cast<float*>(sm + kTabGam);      // rho_r = exp(G_r) scale
  float* tab_gp = tab_gam + kB;       // minus the log-decay (base 2) from the start of s's quarter to s
  float* tab_gb = tab_gam + 2 * kB;   // exp(-G_s)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = gridDim.x, cta = blockIdx.x;

  if (smem_u32(sm) & 1023u) {   // the swizzled tiles need it; never seen (no static shared memory)
    if (tid == 0) flag_error(kErrCheck);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      const bool warps = (i >= kGot && i < kGot + 4) || i == kURead || i == kURead + 1 || i == kQFree || i == kQFree + 1 ||
                         i == kTabEmpty || i == kSReady || i == kKt || i == kKt + 1 || i == kPub || i == kCBar;
      const bool readers = i >= kItEmpty && i < kItEmpty + kRingItems, both = i == kKvFull || i == kKvFull + 1;
      mbar_init(&bars[i], warps ? kComputeWarps : readers ? kComputeWarps + (p.ws ? 3 : 2) : i == kLeft ? kWarps - 1 : both ? 2 : 1);
    }
    fence_mbar_init();
    misc->dead = 0;
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
  const Wait wait{smem_u32(&misc->dead), p.limit};
  // the CTA's i-th item, false behind the last
  auto next_item = [&](uint32_t i, Item& it) {
    wait(&bars[kItFull + (i & 3)], (i >> 2) & 1);
    if (!wait.ok()) return false;
    it = ring[i & 3];
    if (warp != kCourierWarp) arrive_warp(&bars[kItEmpty + (i & 3)]);
    return it.n >= 0;
  };
  Item it;

  if (warp >= kLoadWarp) {
    // (one instruction for the four warps of a group, as it has to be: before the roles part)
    give_registers();
    if (warp == kLoadWarp) {
      // ------------------------------------------------- items; K, V tiles ---
      const uint64_t once = l2_evict_first_policy(), again = l2_evict_normal_policy();
      Walk walk;
      uint32_t cnt = 0;
      bool more = true;
      for (uint32_t i = 0; more && wait.ok(); ++i) {
        more = walk.find(p, cta + (int)i * G, it);
        if (more) more = GDN_CHECK(it.n < p.n_seqs && it.h >= 0 && it.h < p.Hv && it.j >= 0 && it.j < it.J && it.len >= 0 &&
                                   it.t0 >= 0 && it.t0 + it.len <= p.total_T && it.first >= 0 && it.first < p.items &&
                                   (p.ws || it.J == 1));
        if (!more) it.n = -1;
        if (i >= kRingItems) wait(&bars[kItEmpty + (i & 3)], ((i >> 2) - 1) & 1);
        if (lane == 0) ring[i & 3] = it;
        arrive_warp(&bars[kItFull + (i & 3)]);
        if (!more) break;
        const int hq = it.h / (p.Hv / p.Hqk), nb = (it.len + kB - 1) / kB;
        const bool shared_k = p.Hv != p.Hqk;
#pragma unroll 1
        for (int pass = it.j + 1 < it.J ? 0 : 1; pass < 2; ++pass) {
#pragma unroll 1
          for (int b = 0; b < nb; ++b, ++cnt) {
            const uint32_t s = cnt & 1;
            if (cnt >= 2) wait(&bars[kKvEmpty + s], ((cnt >> 1) - 1) & 1);
            if (!wait.ok()) break;
            const int t = it.t0 + b * kB;
            uint64_t* full = &bars[kKvFull + s];
            mbar_arrive_expect_tx_warp(full, 65536);
            uint8_t *kt = sm + kK + s * 32768, *vt = sm + kV + s * 32768;
            // the second pass is the last to read V, and K where no other head shares it
            const uint64_t pv = pass == 0 ? again : once, pk = pass == 0 || shared_k ? again : once;
            tma_load_3d_warp_hint(kt, &km, full, 0, hq, t, pk);
            tma_load_3d_warp_hint(kt + 16384, &km, full, 64, hq, t, pk);
            tma_load_3d_warp_hint(vt, &vm, full, 0, it.h, t, pv);
            tma_load_3d_warp_hint(vt + 16384, &vm, full, 64, it.h, t, pv);
          }
        }
      }
      // tiles still on their way land before the CTA ends
      for (uint32_t c = cnt >= 2 ? cnt - 2 : 0; c < cnt; ++c) mbar_wait(&bars[kKvFull + (c & 1)], (c >> 1) & 1);
    } else if (warp == kGateWarp) {
      // ------------------------------------------- Q tiles and decay tables ---
      const uint64_t pol = p.Hv != p.Hqk ? l2_evict_normal_policy() : l2_evict_first_policy();
      uint32_t qn = 0, cnt = 0;
#pragma unroll 1
      for (uint32_t i = 0; next_item(i, it); ++i) {
        const int hq = it.h / (p.Hv / p.Hqk), nb = (it.len + kB - 1) / kB;
        const float* gh = p.g + it.h;
#pragma unroll 1
        for (int pass = it.j + 1 < it.J ? 0 : 1; pass < 2; ++pass) {
          double seg = 0.0;
          float g[4];
          // a block's log-decays, four consecutive tokens to a lane, fetched a block ahead
          auto fetch = [&](int b) {
            const int r = b * kB + 4 * lane;
#pragma unroll
            for (int x = 0; x < 4; ++x)
              g[x] = r + x < it.len ? gh[(size_t)(it.t0 + r + x) * p.g_stride] : 0.f;
          };
          fetch(0);
#pragma unroll 1
          for (int b = 0; b < nb && wait.ok(); ++b, ++cnt) {
            const int L = min(kB, it.len - b * kB);
            // G, the log-decays (base 2) from the block's start, in fp64; rounded to fp32 as
            // differences only
            constexpr double kLog2E = 1.4426950408889634;
            double c[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              c[x] = (g[x] < kMinLog ? kMinLog : g[x]) * kLog2E;
              if (x > 0) c[x] += c[x - 1];
            }
            double incl = c[3];
            fetch(b + 1);
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
              const double y = __shfl_up_sync(0xffffffffu, incl, off);
              if (lane >= off) incl += y;
            }
            const double sum = __shfl_sync(0xffffffffu, incl, 31), up = __shfl_up_sync(0xffffffffu, incl, 1);
            const double before = lane > 0 ? up : 0.0;   // (not incl - c[3], which a NaN or +inf of this lane would be)
            const double start = __shfl_sync(0xffffffffu, before, lane & 24), whole = floor(start);
            seg += sum;
            float w[4], wm = 0.f, wl = kInf;
            float4 gam, gb, gp;
            float *const gamx = &gam.x, *const gbx = &gb.x, *const gpx = &gp.x;
            bool flat = true;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const double G = before + c[x];
              w[x] = 4 * lane + x < L ? ex2((float)(sum - G)) : 0.f;
              gamx[x] = ex2((float)G) * p.scale;
              gbx[x] = ex2((float)-G);
              gpx[x] = (float)(start - G);
              flat = flat && G > -kSteep;
              wm = fmaxf(wm, w[x]);
              if (4 * lane + x < L) wl = fminf(wl, w[x]);
            }
            uint2 wp[3];
            if constexpr (kF16) {
#pragma unroll
              for (int off = 16; off > 0; off >>= 1) {
                wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, off));
                wl = fminf(wl, __shfl_xor_sync(0xffffffffu, wl, off));
              }
            } else {
              float v[4] = {w[0], w[1], w[2], w[3]};
#pragma unroll
              for (int term = 0; term < 3; ++term) {
                wp[term] = make_uint2(Op16<T>::pack2(v[0], v[1]), Op16<T>::pack2(v[2], v[3]));
                const float2 lo = Op16<T>::unpack2(wp[term].x), hi = Op16<T>::unpack2(wp[term].y);
                v[0] -= lo.x; v[1] -= lo.y; v[2] -= hi.x; v[3] -= hi.y;
              }
            }
            const uint32_t steep = __any_sync(0xffffffffu, !flat);
            const float rest = (float)(start - whole);
            const double far = exp2(lane == 0 ? sum : seg);   // lane 0: the block's, lane 1: the segment's
            const float far_hi = (float)far;
            const int whole_i = (int)whole;
            // everything is ready before the tables may be written: they are one block's
            if (cnt > 0) wait(&bars[kTabEmpty], (cnt - 1) & 1);
            if constexpr (kF16) {
              reinterpret_cast<float4*>(tab_w)[lane] = make_float4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
              for (int term = 0; term < 3; ++term) reinterpret_cast<uint2*>(tab_wp + 64 * term)[lane] = wp[term];
            }
            reinterpret_cast<float4*>(tab_gam)[lane] = gam;
            reinterpret_cast<float4*>(tab_gp)[lane] = gp;
            reinterpret_cast<float4*>(tab_gb)[lane] = gb;
            if ((lane & 7) == 0) {
              misc->start_i[lane >> 3] = whole_i;
              misc->start_f[lane >> 3] = rest;
            }
            if (lane == 0) {
              misc->w_max = wm;
              misc->w_min = wl;
              misc->steep = steep;
              misc->gam_l = far_hi;
            }
            // (read when the segment is published, before the next item's pass A ends)
            if (lane == 1 && pass == 0 && b + 1 == nb)
              misc->seg_gam = make_float2(far_hi, far_hi < 1e30f ? (float)(far - far_hi) : 0.f);
            arrive_warp(&bars[kKvFull + (cnt & 1)]);   // (the block is there when K, V and these are)
            if (pass == 1) {
              const uint32_t q = qn & 1;
              if (qn >= 2) wait(&bars[kQFree + q], ((qn >> 1) - 1) & 1);
              if (wait.ok()) {
                mbar_arrive_expect_tx_warp(&bars[kQFull + q], 32768);
                tma_load_3d_warp_hint(sm + kQ + q * 32768, &qm, &bars[kQFull + q], 0, hq, it.t0 + b * kB, pol);
                tma_load_3d_warp_hint(sm + kQ + q * 32768 + 16384, &qm, &bars[kQFull + q], 64, hq, it.t0 + b * kB, pol);
                ++qn;
              }
            }
          }
        }
      }
      for (uint32_t q = qn >= 2 ? qn - 2 : 0; q < qn; ++q) mbar_wait(&bars[kQFull + (q & 1)], (q >> 1) & 1);
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------- tensor-core work ---
      constexpr uint32_t id_qk = idesc_f16kind(128, 128, false, false, kFmt);   // both K-major
      constexpr uint32_t id_mn = idesc_f16kind(128, 128, false, true, kFmt);    // B MN-major
      // (one copy of each product's code: the loops of all roles share the instruction cache)
      uint32_t cnt = 0, qn = 0, tn0 = 0, tn1 = 0, un0 = 0, un1 = 0;   // tn, un: uses of kKt and the accumulators
#pragma unroll 1
      for (uint32_t i = 0; next_item(i, it); ++i) {
        const int nb = (it.len + kB - 1) / kB;
        const bool last = it.j + 1 == it.J;
#pragma unroll 1
        for (int pass = last ? 1 : 0; pass < 2; ++pass) {
          const bool a = pass == 0;
#pragma unroll 1
          for (int b = 0; b < nb && wait.ok(); ++b, ++cnt) {
            const bool a = each_time(pass == 0);
            const uint32_t s = cnt & 1;
            const uint64_t vd = desc_mnmajor(sbase + kV + s * 32768, 0, 128, 16384);
            const uint64_t qd = desc_kmajor(sbase + kQ + (qn & 1) * 32768, 0, 16384);
            wait(&bars[kKvFull + s], (cnt >> 1) & 1);
            if (!a) {
              wait(&bars[kQFull + (qn & 1)], (qn >> 1) & 1);
              tc_fence_after();
              const uint64_t kd = desc_kmajor(sbase + kK + s * 32768, 0, 16384);
#pragma unroll 1
              for (int h = 0; h < 2; ++h)
                mma_run_warp<4, 2, 2>(tmem + kColP, desc_advance(qd, 16384 * h), desc_advance(kd, 16384 * h), id_qk, h);
              mma_commit_warp(&bars[kPFull]);
            }
            if (a || last || b + 1 < nb) {   // (the state after another segment comes from pass A)
              const uint32_t q = a ? b & 1 : 0, used = q ? un1++ : un0++;
              if (a && b >= 2) wait(&bars[kURead + q], (used - 1) & 1);
              // Two terms of K~ at a time. Pass A has room for two such pairs, so one is made while
              // the other is multiplied: the block's other two (bf16), or the next block's (f16).
              const int parts = !kF16 && (a || last) ? 2 : 1;
#pragma unroll 1
              for (int part = 0; part < parts; ++part) {
                const uint32_t r = parts == 2 ? part : a ? b & 1 : 0;
                wait(&bars[kKt + r], (r ? tn1++ : tn0++) & 1);
                tc_fence_after();
#pragma unroll 1
                for (int x = 0; x < 4; ++x)   // the smaller term first, either half of the tokens
                  mma4_tmem_a_run_warp<128>(tmem + (q ? kColP : kColU),
                                            tmem + (a && r ? kColO : kColK) + (x < 2 ? 32 : 0) + 64 * (x & 1),
                                            desc_advance(vd, 8192 * (x & 1)), id_mn, part | x);
                if (a || part + 1 < parts) mma_commit_warp(&bars[kHalf + r]);
              }
              mma_commit_warp(&bars[kUFull + q]);
            }
            if (!a) {
              wait(&bars[kSReady], qn & 1);
              tc_fence_after();
              const uint64_t sd = desc_mnmajor(sbase + kS, 0, 128, 16384);
#pragma unroll 1
              for (int h = 0; h < 2; ++h)
                mma_run_warp<4, 2, 128>(tmem + kColO, desc_advance(qd, 16384 * h), desc_advance(sd, 8192 * h), id_mn, h);
#pragma unroll 1
              for (int h = 0; h < 2; ++h)
                mma4_tmem_a_run_warp<128>(tmem + kColO, tmem + kColP + 64 * h, desc_advance(vd, 8192 * h), id_mn, 1);
              mma_commit_warp(&bars[kOFull]);
              ++qn;
            }
            mma_commit_warp(&bars[kKvEmpty + s]);
          }
          if (a) {   // both accumulators are read before pass B reuses their columns
            wait(&bars[kURead], (un0 - 1) & 1);
            if (nb > 1) wait(&bars[kURead + 1], (un1 - 1) & 1);
          }
        }
      }
    } else if (warp == kCourierWarp) {
      // ---------------------------------------------- flags in global memory ---
      if (p.ws) {
        uint32_t* all = reinterpret_cast<uint32_t*>(p.ws);
        uint32_t* flags = all + cta * kFlagWords;
        uint32_t pubs0 = 0, pubs1 = 0, ins0 = 0, ins1 = 0, pn = 0;   // uses of this CTA's slots, by parity
#pragma unroll 1
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
              st_relaxed_gpu(flags + kOutReady + par, i + 1);
            }
          }
          if (it.j > 0) {
            const uint32_t use = par ? ++ins1 : ++ins0;
            if (lane == 0) wait.flag(flags + kInCnt + par, kSlices * use);
            arrive_warp(&bars[kInReady]);
          }
          if (last && it.J > 1) {
            // state_out may be state_in, whose reader is then the first segment
            if (lane == 0) wait.flag(all + (it.first % G) * kFlagWords + kDone, it.first / G + 1);
            arrive_warp(&bars[kOutOk]);
          }
          wait(&bars[kGot + (i & 3)], (i >> 2) & 1);
          if (lane == 0) {
            fence_acq_rel_gpu();
            st_relaxed_gpu(flags + kDone, i + 1);
          }
          arrive_warp(&bars[kItEmpty + (i & 3)]);
        }
      }
    } else if (warp >= kScanWarp) {
      // ------------------------------------- states between the segments ---
      if (p.ws) scan_role(p, wait, cta * kScanWarps + warp - kScanWarp, G);
    }
  } else {
    take_registers();   // waits until the others have given theirs
    // ----------------------------------------------------- compute warps ---
    // Warp w4 of each four has lanes 32 w4 .. of tensor memory: rows (tokens) of P and o,
    // columns (d_k) of K~ and of the state. wg: the half of the tokens of K~, of the
    // columns of P, and of d_v in o and the state.
    const int wg = warp >> 2, w4 = warp & 3, row = 32 * w4 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * w4) << 16) + 64 * wg;   // this warp's 64 columns of a region
    float2* meta = reinterpret_cast<float2*>(p.ws + Workspace::meta_offset(G)) + 2 * cta;
    uint8_t* slots = p.ws + Workspace::slots_offset(G) + (size_t)cta * 4 * kStateBytes;
    uint32_t cnt = 0, qn = 0, rn = 0, phases = 0;   // phases: the parity that each barrier is waited for next
    float S[64];        // S[64 wg + i][row]
    float up = 1.f;     // f16: 2^a of this thread's row
    bool bad = false;   // infinities or NaN in this warp's part of what the item adds to the state

    auto wait_next = [&](int bar) {
      wait(&bars[bar], (phases >> (bar - kUFull)) & 1);
      phases ^= 1u << (bar - kUFull);
    };
    static_assert(kUFull < kHalf && kNumBars - kUFull <= 32, "one word of phases");
    // the compute warps' barrier
    auto sync = [&] {
      arrive_warp(&bars[kCBar]);
      wait_next(kCBar);
    };
    // the largest value over the compute threads (f16); `low`: the smallest over a warp, then the
    // smallest over the w4 of the larger of their two warps'
    auto reduce_max = [&](float m, float* low = nullptr) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (low) *low = fminf(*low, __shfl_xor_sync(0xffffffffu, *low, off));
      }
      float(*red)[kComputeWarps] = misc->red[rn++ & 1];   // (the one used two reductions ago: a barrier lies between)
      if (lane == 0) {
        red[0][warp] = m;
        if (low) red[1][warp] = *low;
      }
      sync();
      m = red[0][0];
#pragma unroll
      for (int i = 1; i < kComputeWarps; ++i) m = fmaxf(m, red[0][i]);
      if (low) {
        *low = fmaxf(red[1][0], red[1][4]);
#pragma unroll
        for (int i = 1; i < 4; ++i) *low = fminf(*low, fmaxf(red[1][i], red[1][4 + i]));
      }
      return m;
    };
    // the rounded copy of S
    auto write_copy = [&](float down) {
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
    // Sixteen registers of K's tile at kt: tokens 64 wg .. + 63, columns 32 w4 + 16 half .. + 15,
    // as transposed pairs of tokens
    const uint32_t ldm_row = 64 * wg + 8 * ((lane >> 4) & 1) + (lane & 7);
    auto load_k = [&](uint32_t kt, int half, uint32_t* kr) {
      const uint32_t c = 4 * w4 + 2 * half + ((lane >> 3) & 1);     // 16-byte chunk of K's row
      const uint32_t at = sbase + kt + (c >> 3) * 16384 + ldm_row * 128 + (((c & 7) ^ (ldm_row & 7)) << 4);
#pragma unroll
      for (int i = 0; i < 8; i += 2) ldmatrix_t4(at + 1024 * i, kr + 2 * i);
    };
    // f16: the two terms of K~ from fp32 products, a power of two for each column; returns that of
    // column `row`. ex: the exponents of each half column's largest product. (They are written
    // behind a barrier that all warps reach after they have read those of an earlier block.)
    auto put_terms_apart = [&](uint32_t kt, uint32_t region) -> int {
      uint8_t* const ex = reinterpret_cast<uint8_t*>(tab_w + kB) + 32 * w4;
      const float* const w = tab_w + 64 * wg + 2 * (lane & 3);
      auto power = [&](int c) { return min(13 - ((int)max(ex[c], ex[kD + c]) - 127), 126); };
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        uint32_t kr[16];
        float m[2] = {0.f, 0.f};
        load_k(kt, half, kr);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 x = Op16<T>::unpack2(kr[i]);
          m[i & 1] = fmaxf(m[i & 1], fmaxf(fabsf(x.x * w[8 * (i >> 1)]), fabsf(x.y * w[8 * (i >> 1) + 1])));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 1));
          m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 2));
          if ((lane & 3) == 0) ex[kD * wg + 16 * half + 8 * i + (lane >> 2)] = (uint8_t)(exponent_of(m[i]) + 127);
        }
      }
      sync();
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        uint32_t kr[16], lo[16];
        load_k(kt, half, kr);
        const float f[2] = {pow2i(power(16 * half + (lane >> 2))), pow2i(power(16 * half + 8 + (lane >> 2)))};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float2 x = Op16<T>::unpack2(kr[i]);
          x.x = x.x * w[8 * (i >> 1)] * f[i & 1];
          x.y = x.y * w[8 * (i >> 1) + 1] * f[i & 1];
          kr[i] = Op16<T>::pack2(x.x, x.y);
          const float2 y = Op16<T>::unpack2(kr[i]);
          lo[i] = Op16<T>::pack2(x.x - y.x, x.y - y.y);
        }
        const uint32_t tw = tl + region + (static_cast<uint32_t>(16 * half) << 16);
        tmem_st_frag(tw, kr);
        tmem_st_frag(tw + 32, lo);
      }
      return power(lane);
    };
    // Two terms of K~ (part 0: hi and, with four of them, e1; part 1: h2 and t4). Returns the
    // power of two that they were multiplied with (f16).
    auto put_terms = [&](uint32_t kt, bool four, int part, uint32_t region, int bar) -> int {
      uint32_t w1[8], w2[8], w3[8];
      int e = 0;
      if constexpr (kF16) {
        // The columns' largest products, with w below 1 so that none overflows. f16 ends at 2^-24:
        // with the block's largest product at 2^13 (w below 2^15) a column's has to be at 2^2 or
        // above, so that hi and its rest have 22 bits beside it and 18 for what is 2^-8 of it,
        // and w at 2^-7 or above for 18 bits of its own: a decay of some 18 bits in the block.
        // Beyond either the terms come from fp32 products, 7 % of a long prompt's time if all do
        // (551 against 517 us, 32768 tokens; with no look 502).
        const int ew = exponent_of(misc->w_max);
        const float ws = pow2i(-ew - 1);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 w = *reinterpret_cast<const float2*>(tab_w + 64 * wg + 8 * i + 2 * (lane & 3));
          w1[i] = Op16<T>::pack2(w.x * ws, w.y * ws);
        }
        float top = 0.f, low = 65504.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t kr[16];
          __half2 m[2] = {__half2half2(__ushort_as_half(0)), __half2half2(__ushort_as_half(0))};
          load_k(kt, half, kr);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t x = Two<T>::mul(w1[i >> 1], kr[i]);
            m[i & 1] = __hmax2(m[i & 1], __habs2(*reinterpret_cast<const __half2*>(&x)));
          }
          __half2 c = __hmax2(__lows2half2(m[0], m[1]), __highs2half2(m[0], m[1]));   // two columns
          c = __hmax2(c, __shfl_xor_sync(0xffffffffu, c, 1));
          c = __hmax2(c, __shfl_xor_sync(0xffffffffu, c, 2));
          const float2 f = __half22float2(c);
          const int col = 32 * w4 + 16 * half + (lane >> 2);
          top = fmaxf(top, fmaxf(f.x, f.y));
          if (kWhole || col < p.dk) low = fminf(low, f.x);
          if (kWhole || col + 8 < p.dk) low = fminf(low, f.y);
        }
        top = reduce_max(top, &low);
        e = min(12 - exponent_of(top) - ew, 14 - ew);
        if (each_time(!(top < kInf) || low * pow2i(e + ew + 1) < 4.f || misc->w_min * pow2i(e) < 0.0078125f)) {
          e = put_terms_apart(kt, region);
          tmem_wait_st();
          tc_fence_before();
          arrive_warp(&bars[kKt + bar]);
          return e;
        }
        const float scale = pow2i(e);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float2 w = *reinterpret_cast<const float2*>(tab_w + 64 * wg + 8 * i + 2 * (lane & 3));
          w.x *= scale; w.y *= scale;
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
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        uint32_t kr[16], x[16], y[16];
        load_k(kt, half, kr);
        const uint32_t tw = tl + region + (static_cast<uint32_t>(16 * half) << 16);
        if (part == 0) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            x[i] = Two<T>::mul(w1[i >> 1], kr[i]);
            y[i] = Two<T>::fma(w1[i >> 1], kr[i], neg2(x[i]));
          }
          if (!four) {
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = Two<T>::fma(w2[i >> 1], kr[i], y[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            x[i] = Two<T>::mul(w2[i >> 1], kr[i]);
            y[i] = Two<T>::fma(w2[i >> 1], kr[i], neg2(x[i]));
            if constexpr (!kF16) y[i] = Two<T>::fma(w3[i >> 1], kr[i], y[i]);
          }
        }
        tmem_st_frag(tw, x);
        tmem_st_frag(tw + 32, y);
      }
      tmem_wait_st();
      tc_fence_before();
      arrive_warp(&bars[kKt + bar]);
      return e;
    };
    // Rows behind the sequence may hold anything: zero in V, and in the patch of K that this
    // warp weighs (Q K^T masks its own).
    auto clear_rows = [&](uint32_t kt, uint32_t vt, int L) {
#pragma unroll 1
      for (int i = tid; i < (kB - L) * 16; i += kCompute) {
        const int r = L + (i >> 4), c = i & 15;
        *reinterpret_cast<uint4*>(sm + vt + (c >> 3) * 16384 + r * 128 + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
      }
#pragma unroll 1
      for (int i = lane; i < 256; i += 32) {
        const int r = 64 * wg + (i >> 2), c = 4 * w4 + (i & 3);
        if (r >= L)
          *reinterpret_cast<uint4*>(sm + kt + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
              make_uint4(0, 0, 0, 0);
      }
      fence_async_smem();
      __syncwarp();
    };
    // S <- exp(G_L) S + U
    auto update_state = [&](int q, float gam, float down) {
      wait_next(kUFull + q);
      tc_fence_after();
      float u[64];
      tmem_ld64(tl + (q ? kColP : kColU), u);
#pragma unroll
      for (int i = 0; i < 64; ++i) S[i] = fmaf(gam, S[i], kF16 ? u[i] * down : u[i]);
      tc_fence_before();
      arrive_warp(&bars[kURead + q]);
    };
    // f16: the powers of two of the copy of S (2^-b, returned) and of this thread's row (P' by
    // `by` = 2^-a, q by 2^(b - a - m), `up` = 2^a), from the largest |S|, |P'| (`top`: of the
    // thread's 64 columns) and |q|; S has to be there. `rows`, 512 bytes of the tables that this
    // block has no use for, holds each half row's exponents of |P'| and |q|. (They are written
    // after Q K^T of this block, which follows every warp's copy of S in the block before.)
    auto row_scales = [&](float top, uint8_t* q, int m, float* rows, float& by) -> float {
      uint4* const qr = reinterpret_cast<uint4*>(q + wg * 16384 + row * 128);
      __half2 mq = __half2half2(__ushort_as_half(0));
#pragma unroll 2
      for (int c = 0; c < 8; ++c) {
        const uint4 x = qr[c ^ (row & 7)];
        mq = __hmax2(__hmax2(__hmax2(mq, __habs2(*reinterpret_cast<const __half2*>(&x.x))),
                             __hmax2(__habs2(*reinterpret_cast<const __half2*>(&x.y)),
                                     __habs2(*reinterpret_cast<const __half2*>(&x.z)))),
                     __habs2(*reinterpret_cast<const __half2*>(&x.w)));
      }
      const float2 f = __half22float2(mq);
      uint16_t* const er = reinterpret_cast<uint16_t*>(rows) + row;
      er[128 * wg] = (uint16_t)((exponent_of(top) + 127) << 8 | (exponent_of(fmaxf(f.x, f.y)) + 127));
      float most;
      bool finite = true;
#pragma unroll 1
      do {   // again where there are infinities: the other values keep their size
        most = 0.f;
#pragma unroll
        for (int i = 0; i < 64; ++i) most = finite || fabsf(S[i]) < kInf ? fmaxf(most, fabsf(S[i])) : most;
        most = reduce_max(most);
        finite = !finite || most < kInf;
      } while (!finite);
      const uint32_t x = er[0], y = er[128];
      const int b = max(exponent_of(most) - 5, -100);
      const int ep = (int)max(x >> 8, y >> 8) - 127, eq = (int)max(x & 255u, y & 255u) - 127 - m;
      // q as it is where the scores have their place beside it
      const int a = m == 0 && ep >= b + 3 && ep <= b + 14 ? b : max(max(ep, b + eq) - 14, max(b - m - 30, -100));
      up = pow2i(a);
      by = pow2i(-a);
      const int c = b - a - m;
      if (__any_sync(0xffffffffu, c != 0)) {
        // (two factors: f16 holds no power below 2^-24)
        const __half2 f1 = __float2half2_rn(pow2i(min(max(c, -14), 15)));
        const __half2 f2 = __float2half2_rn(pow2i(min(max(c + 14, -25), 0) + max(c - 15, 0)));
#pragma unroll 2
        for (int i = 0; i < 8; ++i) {
          uint4 z = qr[i ^ (row & 7)];
          __half2* const h = reinterpret_cast<__half2*>(&z);
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = __hmul2(__hmul2(h[j], f1), f2);
          qr[i ^ (row & 7)] = z;
        }
      }
      return pow2i(-b);
    };
    // P', packed, over Q K^T: 32 rows and 64 columns, zero above the diagonal.
    auto make_scores = [&](uint8_t* q) {
      float down = 1.f, by = 1.f, top = 0.f;
#pragma unroll 1
      for (int pass = kF16 ? 0 : 1; pass < 2; ++pass) {
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          const int cb = 2 * wg + c;
          uint32_t u[16];
          if (cb > w4) {
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = 0u;
          } else {
            float x[32];
            tmem_ld32(tl + kColP + 32 * c, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 b = *reinterpret_cast<const float4*>(tab_gb + 32 * cb + 4 * i);
              x[4 * i] *= b.x; x[4 * i + 1] *= b.y; x[4 * i + 2] *= b.z; x[4 * i + 3] *= b.w;
            }
            if (cb == w4) {
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = i <= lane ? x[i] : 0.f;
            }
            if constexpr (kF16) {
              if (pass == 0) {
#pragma unroll
                for (int i = 0; i < 32; ++i) top = fmaxf(top, fabsf(x[i]));
              }
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] *= by;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = Op16<T>::pack2(x[2 * i], x[2 * i + 1]);
          }
          if (pass == 1) tmem_st16(tl + kColP + 16 * c, u);   // (columns that this warp has read)
        }
        if constexpr (kF16) {
          if (pass == 0) down = row_scales(top, q, 0, tab_gp, by);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      return down;
    };
    // A steep block's: 2^-m_r out of a row of Q, and P' by the exponent; compact, not fast.
    auto make_steep_scores = [&](uint8_t* q, int m_row) {
      if constexpr (!kF16) {
        const float f = m_row > 126 ? 0.f : pow2i(-m_row);
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint4* at = reinterpret_cast<uint4*>(q + wg * 16384 + row * 128 + ((c ^ (row & 7)) << 4));
          float x[8];
          unpack8<T>(*at, x);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= f;
          *at = pack8<T>(x);
        }
      }
      float down = 1.f, by = 1.f, top = 0.f;
#pragma unroll 1
      for (int pass = kF16 ? 0 : 1; pass < 2; ++pass) {
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          const int col = 64 * wg + 8 * c, cb = col >> 5;
          const float far = (float)(-misc->start_i[cb] - m_row) - misc->start_f[cb];
          float x[8];
          tmem_ld8(tl + kColP + 8 * c, x);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] = col + i <= row ? x[i] * ex2(far + tab_gp[col + i]) : 0.f;
            top = fmaxf(top, fabsf(x[i]));
          }
          if (pass == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              tmem_st1(tl + kColP + 4 * c + i, Op16<T>::pack2(x[2 * i] * by, x[2 * i + 1] * by));
          }
        }
        if constexpr (kF16) {
          if (pass == 0) down = row_scales(top, q, m_row, tab_gb, by);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      return down;
    };
    // o of this warp's 32 tokens and 64 columns, through its part of the block's Q buffer
    const int o_chunks = min(8, max(0, p.dv / 8 - 8 * wg));    // 16-byte chunks of these columns
    auto stage_o = [&](uint8_t* o_stage, float rho) {
      if (o_chunks == 0) return;
#pragma unroll 1
      for (int c = 0; c < 8; c += 4) {
        float x[32];
        tmem_ld32(tl + kColO + 8 * c, x);
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] *= rho;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(o_stage + lane * 128 + (((c + i) ^ (lane & 7)) << 4)) = pack8<T>(x + 8 * i);
      }
      tc_fence_before();
    };
    auto send_o = [&](const uint8_t* o_stage, int t, int h, int L) {
      if (o_chunks == 0) return;
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
        T* o = static_cast<T*>(p.o) + ((size_t)(t + 32 * w4) * p.Hv + h) * p.dv + 64 * wg;
        const int c = lane & 7;
        if (c < o_chunks) {
#pragma unroll 1
          for (int r = lane >> 3; r < rows; r += 4)
            __stcs(reinterpret_cast<uint4*>(o + (size_t)r * p.Hv * p.dv + 8 * c),
                   *reinterpret_cast<const uint4*>(o_stage + r * 128 + ((c ^ (r & 7)) << 4)));
        }
        fence_async_smem();   // Q's next tile comes to where these rows lay
      }
    };
    auto not_finite = [&] {
      float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 64; ++i) t[i & 3] = fmaf(S[i], 0.f, t[i & 3]);
      return __any_sync(0xffffffffu, !((t[0] + t[1]) + (t[2] + t[3]) == 0.f)) != 0;
    };
    // Rows of this warp in front of a column's first infinity or NaN in V, in its block: again, by
    // the recurrence, with four of d_k to a lane. A column's NaN is in the state of all four warps
    // that hold it, so each finds its own rows.
    auto mend_rows = [&](int par) {
      if (lane == 0) bulk_wait_all();   // the rows' own way out is over
      __syncwarp();
      const int hq = it.h / (p.Hv / p.Hqk), cols = min(64, p.dv - 64 * wg);
      const T* const q = static_cast<const T*>(p.q) + ((size_t)it.t0 * p.Hqk + hq) * p.dk;
      const T* const k = static_cast<const T*>(p.k) + ((size_t)it.t0 * p.Hqk + hq) * p.dk;
      const size_t at_v = ((size_t)it.t0 * p.Hv + it.h) * p.dv + 64 * wg, step = (size_t)p.Hv * p.dv;
      const T* const v = static_cast<const T*>(p.v) + at_v;
      T* const o = static_cast<T*>(p.o) + at_v;
      int first[2] = {it.len, it.len};   // of columns 2 lane, 2 lane + 1
      if (2 * lane < cols) {
#pragma unroll 4
        for (int t = it.len - 1; t >= 0; --t) {
          const float2 x = Op16<T>::unpack2(*reinterpret_cast<const uint32_t*>(v + t * step + 2 * lane));
          if (!(fabsf(x.x) < kInf)) first[0] = t;
          if (!(fabsf(x.y) < kInf)) first[1] = t;
        }
      }
#pragma unroll 1
      for (int c = 0; c < cols; ++c) {
        const int end = __shfl_sync(0xffffffffu, c & 1 ? first[1] : first[0], c >> 1);
        const int lo = (end & ~(kB - 1)) + 32 * w4, hi = min(lo + 32, end);
        if (end == it.len || lo >= hi) continue;
        float s[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int j = 32 * u + lane;
          s[u] = 0.f;
          if (it.j > 0)
            s[u] = __ldcg(reinterpret_cast<const float*>(slots + (size_t)(2 + par) * kStateBytes) +
                          ((size_t)(c >> 2) * 256 + 128 * wg + j) * 4 + (c & 3));
          else if (p.state_in && j < p.dk)
            s[u] = __ldcs(p.state_in + (((size_t)it.n * p.Hv + it.h) * p.dv + 64 * wg + c) * p.dk + j);
        }
#pragma unroll 1
        for (int t = 0; t < hi; ++t) {
          const float a = expf(p.g[(size_t)(it.t0 + t) * p.g_stride + it.h]), x = to_f32(v[t * step + c]);
          float r = 0.f;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int j = 32 * u + lane;
            if (j >= p.dk) continue;
            s[u] = fmaf(a, s[u], x * to_f32(k[(size_t)t * p.Hqk * p.dk + j]));
            if (t >= lo) r = fmaf(s[u], to_f32(q[(size_t)t * p.Hqk * p.dk + j]), r);
          }
          if (t >= lo) {
            r = group_sum<32>(r);
            if (lane == 0) o[t * step + c] = from_f32<T>(p.scale * r);
          }
        }
      }
      __syncwarp();
    };
#pragma unroll 1
    for (uint32_t i = 0; next_item(i, it); ++i) {
      const int nb = (it.len + kB - 1) / kB, par = i & 1;
      const bool last = it.j + 1 == it.J;
      bad = false;
      // One body for both passes. K~ of a block is made while the tensor core is at the block
      // before it: in pass A the state follows a block behind; in pass B o of the block before
      // leaves tensor memory first, because K~ goes where it was.
#pragma unroll 1
      for (int pass = last ? 1 : 0; pass < 2; ++pass) {
        if (pass == 0) {
#pragma unroll
          for (int x = 0; x < 64; ++x) S[x] = 0.f;
        }
        float gam = 0.f, rho = 0.f;
        int e = 0;
#pragma unroll 1
        for (int b = 0; b <= nb && wait.ok(); ++b) {
          const bool a = each_time(pass == 0), ends = each_time(last);
          const uint32_t s = cnt & 1;
          const int L = min(kB, it.len - b * kB);
          const bool here = each_time(b < nb), upd = each_time(here && (a || ends || b + 1 < nb));
          const bool four = !kF16 && (a || ends);
          const float gam_before = gam, rho_before = rho;
          const int e_before = e;
          float down = 1.f;
          uint8_t* const q_tile = sm + kQ + (qn & 1) * 32768;
          if (here) {
            wait(&bars[kKvFull + s], (cnt >> 1) & 1);
            gam = misc->gam_l;
            if (L < kB) clear_rows(kK + s * 32768, kV + s * 32768, L);
          }
          // K~: two terms, and with four of them two more -- in pass A beside the first, else when
          // those are multiplied
          const int parts = each_time(four && (a || upd)) ? 2 : 1;
#pragma unroll 1
          for (int part = 0; part < parts; ++part) {
            const int r = four ? part : a ? b & 1 : 0;
            if (a ? b >= (four ? 1 : 2) : part == 1) wait_next(kHalf + (a ? r : 0));
            if (a && !four && !here) wait_next(kHalf + (~b & 1));
            if (upd) e = put_terms(kK + s * 32768, four, part, a && r ? kColO : kColK, r);
            if (part + 1 == parts && here && (a || four)) arrive_warp(&bars[kTabEmpty]);
            if (a || part == 1) continue;
            if (!a && b == 0) {
              // the state that enters
              if (it.j > 0) {
                wait_next(kInReady);
                const float4* in = reinterpret_cast<const float4*>(slots + (size_t)(2 + par) * kStateBytes);
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                  const float4 x = __ldcg(in + 256 * v + tid);
                  S[4 * v] = x.x; S[4 * v + 1] = x.y; S[4 * v + 2] = x.z; S[4 * v + 3] = x.w;
                }
              } else {
                const float* in = p.state_in + (((size_t)it.n * p.Hv + it.h) * p.dv + 64 * wg) * p.dk + row;
                if (!p.state_in) {
#pragma unroll
                  for (int x = 0; x < 64; ++x) S[x] = 0.f;
                } else if (kWhole) {
#pragma unroll
                  for (int x = 0; x < 64; ++x) S[x] = __ldcs(in + x * kD);
                } else {
#pragma unroll
                  for (int x = 0; x < 64; ++x) S[x] = row < p.dk && 64 * wg + x < p.dv ? __ldcs(in + x * p.dk) : 0.f;
                }
              }
            }
            if (!a && here) {
              const bool steep = each_time(misc->steep != 0);
              wait_next(kPFull);
              tc_fence_after();
              rho = tab_gam[row];
              if (steep) {
                const float rest = misc->start_f[w4] - tab_gp[row];
                const int m_row = max(0, -kSteep - misc->start_i[w4] - (int)ceilf(rest));
                rho = p.scale * ex2((float)(misc->start_i[w4] + m_row) + rest);
                down = make_steep_scores(q_tile, m_row);
              } else {
                down = make_scores(q_tile);
              }
            }
            if (here && !four) arrive_warp(&bars[kTabEmpty]);
            if (!a) {
              if (here) rho *= up;
              if (b > 0) {
                uint8_t* const o_stage = sm + kQ + (~qn & 1) * 32768 + wg * 16384 + w4 * 4096;
                wait_next(kOFull);
                tc_fence_after();
                stage_o(o_stage, rho_before);
                send_o(o_stage, it.t0 + (b - 1) * kB, it.h, min(kB, it.len - (b - 1) * kB));
              }
              if (here) write_copy(down);
              if (p.ws && b == 0 && !last && !bad) arrive_warp(&bars[kGot + (i & 3)]);
            }
          }
          if (!a) {
            if (b > 0) {   // the Q buffer is free when o has left it
              if (lane == 0) bulk_wait_read_all();
              arrive_warp(&bars[kQFree + (~qn & 1)]);
            }
            if (here) ++qn;
          }
          if (here) ++cnt;
          if (a ? b > 0 : upd) update_state(a ? ~b & 1 : 0, a ? gam_before : gam, pow2i(a ? -e_before : -e));
        }
        if (pass == 0) {
          bad = not_finite();
          wait_next(kSlotFree);
          float4* out = reinterpret_cast<float4*>(slots + (size_t)par * kStateBytes);
#pragma unroll
          for (int v = 0; v < 16; ++v)
            __stcg(out + 256 * v + tid, make_float4(S[4 * v], S[4 * v + 1], S[4 * v + 2], S[4 * v + 3]));
          if (tid == 0) __stcg(meta + par, misc->seg_gam);
          arrive_warp(&bars[kPub]);
        }
      }
      if (last) bad = not_finite();
      if (bad) {
        // (S waits in tensor memory, where the state's products are over)
        const uint32_t* const u = reinterpret_cast<const uint32_t*>(S);
#pragma unroll
        for (int c = 0; c < 64; c += 16) tmem_st16(tl + kColU + c, u + c);
        tmem_wait_st();
        mend_rows(par);
        tmem_ld64(tl + kColU, S);
      }
      // The state that entered is needed no more; nor does the next item's kOutOk come before this.
      if (last && it.J > 1) wait_next(kOutOk);
      if (p.ws && (last || bad)) arrive_warp(&bars[kGot + (i & 3)]);
      if (last) {
        // the state after the sequence: a row of 32 consecutive columns a store. Where it takes
        // the place of state_in, no warp reads that any more.
        if (it.J == 1 && p.state_in == p.state_out) sync();
        float* out = p.state_out + (((size_t)it.n * p.Hv + it.h) * p.dv + 64 * wg) * p.dk + row;
        if (kWhole) {
#pragma unroll
          for (int x = 0; x < 64; ++x) __stcs(out + x * kD, S[x]);
        } else if (row < p.dk) {
#pragma unroll
          for (int x = 0; x < 64; ++x)
            if (64 * wg + x < p.dv) __stcs(out + x * p.dk, S[x]);
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  if (warp < kWarps - 1) {
    arrive_warp(&bars[kLeft]);
  } else {
    wait.watch(&bars[kLeft]);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (tid == 0 && !wait.ok()) flag_error(kErrTimeout);
}

// Waits that nothing ends, one kind a CTA: on chip (CTA 0; the watchdog's time is over after
// max_cycles), for a flag (CTA 1), the scan's for a publication (CTA 2; there the watchdog would
// take 16 times as long, which a check of the time tells). The first warp waits on chip in all
// of them and leaves when another gives up.
__device__ uint32_t g_never_published[8 * kFlagWords];
__device__ int32_t g_two_segments[2] = {0, 2 * kB};
__global__ void __launch_bounds__(96) wait_selftest_kernel(long long max_cycles) {
  __shared__ uint64_t bars[2];   // never completed; the warps that have left
  __shared__ uint32_t dead;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, kind = blockIdx.x;
  if (threadIdx.x == 0) {
    mbar_init(&bars[0], 1);
    mbar_init(&bars[1], 2);
    fence_mbar_init();
    dead = 0;
  }
  __syncthreads();
  const long long t0 = clock64();
  const Wait wait{smem_u32(&dead), max_cycles};
  if (warp == 0) {
    wait(&bars[0], 0);
  } else if (warp == 1 && kind == 1) {
    if (lane == 0) wait.flag(g_never_published, 1u);
  } else if (warp == 1 && kind == 2) {
    Params p = {};
    p.cu_seqlens = g_two_segments;
    p.ws = reinterpret_cast<uint8_t*>(g_never_published);
    p.n_seqs = p.Hqk = p.Hv = p.seg = p.panel = 1;
    p.total_T = 2 * kB;
    p.items = 2;
    p.dk = p.dv = kD;
    p.limit = max_cycles;
    scan_role(p, wait, 0, 8);
  }
  if (warp < 2) {
    arrive_warp(&bars[1]);
  } else {
    Wait{smem_u32(&dead), kind == 0 ? max_cycles : 16 * max_cycles}.watch(&bars[1]);
  }
  __syncthreads();
  if (threadIdx.x == 0 && !wait.ok()) flag_error(clock64() - t0 > 8 * max_cycles ? kErrCheck : kErrTimeout);
}

}  // namespace ltc
}  // namespace gdn
