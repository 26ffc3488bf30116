// C ABI of libgdn.so: argument checks, kernel selection and launches.
// Declared and documented in include/gdn.h.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <set>
#include <string>
#include <algorithm>
#include <type_traits>
#include <utility>

#include "gdn.h"
#include "common.cuh"
#include "decode.cuh"
#include "prefill_simt.cuh"
#include "prefill_pc.cuh"
#include "linear.cuh"
#include "linear_tc.cuh"
#include "state_pool.cuh"

#include <cudaTypedefs.h>

namespace {

thread_local std::string t_last_error;

gdn_status fail(gdn_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
gdn_status fail(gdn_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  t_last_error = buf;
  return s;
}

gdn_status ok() {
  t_last_error.clear();
  return GDN_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool head_dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
bool dtype_ok(gdn_dtype dtype) { return dtype == GDN_BF16 || dtype == GDN_F32 || dtype == GDN_F16; }

// Allow a kernel the full opt-in shared memory, once per (kernel, device), so
// that later calls (including ones inside CUDA-graph capture) only launch.
constexpr size_t kSmemOptIn = 227 * 1024;
template <typename F>
gdn_status allow_smem(F* kern, const char* what) {
  static std::mutex mu;
  static std::set<std::pair<const void*, int>> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  std::lock_guard<std::mutex> lock(mu);
  const auto key = std::make_pair(reinterpret_cast<const void*>(kern), dev);
  if (done.count(key)) return GDN_OK;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemOptIn);
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  done.insert(key);
  return GDN_OK;
}

gdn_status launch_status(const char* what) {
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "%s: launch failed: %s", what, cudaGetErrorString(e));
  return ok();
}

// ---------------------------------------------------------------- decode ---
template <typename TIO, int DK, typename TS>
gdn_status launch_decode(const void* q, const void* k, const void* v, const float* g,
                         const float* beta, TS* state, int B, int Hqk, int Hv, int dv,
                         float scale, void* o, cudaStream_t st) {
  using Sh = gdn::DecodeShape<DK, TS>;
  dim3 grid((unsigned)(B * Hv), (unsigned)((dv + Sh::kRowsPerCta - 1) / Sh::kRowsPerCta));
  gdn::decode_step_kernel<TIO, DK, TS><<<grid, Sh::kWarps * 32, 0, st>>>(
      static_cast<const TIO*>(q), static_cast<const TIO*>(k), static_cast<const TIO*>(v), g, beta,
      state, Hqk, Hv, dv, scale, static_cast<TIO*>(o));
  return launch_status("gdn_decode");
}

template <typename TIO, typename TS>
gdn_status dispatch_decode(const void* q, const void* k, const void* v, const float* g,
                           const float* beta, TS* state, int B, int Hqk, int Hv, int dk,
                           int dv, float scale, void* o, cudaStream_t st) {
  switch (dk) {
    case 16: return launch_decode<TIO, 16, TS>(q, k, v, g, beta, state, B, Hqk, Hv, dv, scale, o, st);
    case 32: return launch_decode<TIO, 32, TS>(q, k, v, g, beta, state, B, Hqk, Hv, dv, scale, o, st);
    case 64: return launch_decode<TIO, 64, TS>(q, k, v, g, beta, state, B, Hqk, Hv, dv, scale, o, st);
    default: return launch_decode<TIO, 128, TS>(q, k, v, g, beta, state, B, Hqk, Hv, dv, scale, o, st);
  }
}

// Host checks shared by the decode entry points; GDN_OK when the call may proceed
// (B == 0 is returned as done through *done).
gdn_status check_decode(const char* fn, const void* q, const void* k, const void* v, const float* g,
                        const float* beta, const void* state, int B, int Hqk, int Hv, int dk, int dv,
                        gdn_dtype dtype, const void* o, bool* done) {
  *done = false;
  if (B < 0) return fail(GDN_ERR_INVALID_ARG, "%s: B=%d < 0", fn, B);
  if (Hqk <= 0 || Hv <= 0 || Hv % Hqk != 0)
    return fail(GDN_ERR_INVALID_ARG, "%s: Hv=%d must be a positive multiple of Hqk=%d", fn, Hv, Hqk);
  if (!head_dim_ok(dk) || !head_dim_ok(dv))
    return fail(GDN_ERR_UNSUPPORTED, "%s: dk=%d, dv=%d (supported: 16, 32, 64, 128)", fn, dk, dv);
  if (!dtype_ok(dtype)) return fail(GDN_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
  if ((int64_t)B * Hv > 0x7fffffff) return fail(GDN_ERR_INVALID_ARG, "%s: B*Hv too large", fn);
  if (B == 0) {
    *done = true;
    return ok();
  }
  if (!q || !k || !v || !g || !beta || !state || !o)
    return fail(GDN_ERR_INVALID_ARG, "%s: pointers must not be NULL", fn);
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(state))
    return fail(GDN_ERR_INVALID_ARG, "%s: q, k, v, o and state must be 16-byte aligned", fn);
  if (!aligned4(g) || !aligned4(beta)) return fail(GDN_ERR_INVALID_ARG, "%s: g and beta must be 4-byte aligned", fn);
  return GDN_OK;
}

// --------------------------------------------------------------- prefill ---
constexpr size_t kSmemLimit = kSmemOptIn;

int simt_slice_rows(int dk, int dv, int C) {
  // widest state slice whose working set fits in shared memory, at most 32 rows
  for (int dvp = dv < 32 ? dv : 32; dvp >= 8; dvp /= 2) {
    if (dv % dvp) continue;
    if ((size_t)gdn::SimtSmem(C, dk, dvp).total * sizeof(float) <= kSmemLimit) return dvp;
  }
  return 0;
}

template <typename TIO>
gdn_status launch_prefill_simt(const void* q, const void* k, const void* v, const float* g,
                               const float* beta, const float* state_in, const int32_t* cu,
                               int n_seqs, int64_t total_T, int Hqk, int Hv, int dk, int dv,
                               float scale, int C, void* o, float* state_out, cudaStream_t st) {
  const int dvp = simt_slice_rows(dk, dv, C);
  if (dvp == 0)
    return fail(GDN_ERR_UNSUPPORTED, "gdn_prefill: dk=%d dv=%d chunk=%d does not fit the SIMT kernel", dk,
                dv, C);
  const size_t smem = (size_t)gdn::SimtSmem(C, dk, dvp).total * sizeof(float);
  auto kern = gdn::prefill_simt_kernel<TIO>;
  if (gdn_status s = allow_smem(kern, "gdn_prefill")) return s;
  dim3 grid((unsigned)(dv / dvp), (unsigned)Hv, (unsigned)n_seqs);
  kern<<<grid, 256, smem, st>>>(static_cast<const TIO*>(q), static_cast<const TIO*>(k),
                                static_cast<const TIO*>(v), g, beta, state_in, cu, Hqk, Hv, dk, dv,
                                dvp, C, scale, static_cast<TIO*>(o), state_out, (long long)total_T);
  return launch_status("gdn_prefill");
}

// ------------------------------------------------- tensor-core prefill ---
// The driver's tensor-map encoder, looked up once per process (thread-safe).
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// 3-D map of 16-bit elements (bf16 or f16) over a token-major [T][H][D] tensor:
// dims (D, H, T), box (box_d, 1, box_t).
bool make_map(CUtensorMap* m, const void* base, int D, int H, int T, int box_d, CUtensorMapDataType type,
              int box_t = gdn::pc::kC) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2};
  cuuint32_t box[3] = {(cuuint32_t)box_d, 1, (cuuint32_t)box_t};
  cuuint32_t estr[3] = {1, 1, 1};
  const int row_bytes = box_d * 2;
  CUtensorMapSwizzle sw = row_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                          : row_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                            : CU_TENSOR_MAP_SWIZZLE_32B;
  auto encode = [&] {
    return enc(m, type, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  if (r == CUDA_ERROR_INVALID_CONTEXT || r == CUDA_ERROR_NOT_INITIALIZED) {
    // A host thread that has made no CUDA call yet: unlike the runtime's own calls the encoder
    // does not make the device's context the thread's.
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = encode();
  }
  return r == CUDA_SUCCESS;
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

// The prefill kernel's two bounded waits -- on a ring flag in global memory and
// on an mbarrier -- each run on something nothing will ever signal, so that the
// timeout path (error word set, kernel returns) can be exercised without a hung
// or faulted GPU.
__device__ uint32_t g_never_set;
__global__ void wait_selftest_kernel(long long max_cycles) {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) {
    gdn::sm100::wait_flag_geq(&g_never_set, 1u, max_cycles);
    gdn::sm100::mbar_init(&bar, 1);
    gdn::sm100::fence_mbar_init();
    gdn::sm100::mbar_wait(&bar, 0, max_cycles);
  }
}

bool uses_pc_prefill(gdn_dtype dtype, int dk, int dv) {
  return (dtype == GDN_BF16 || dtype == GDN_F16) && dk == 128 && dv == 128;
}


template <int DVP, typename T>
gdn_status launch_pc(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const CUtensorMap& om,
                     const gdn::pc::Params& prm, int grid, cudaStream_t st) {
  auto kern = gdn::pc::prefill_pc_kernel<DVP, T>;
  if (gdn_status s = allow_smem(kern, "gdn_prefill")) return s;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(gdn::pc::kThreads);
  cfg.dynamicSmemBytes = gdn::pc::Smem<DVP>::kAlloc;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;   // every CTA co-resident: CTAs wait on one another
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, qm, km, vm, om, prm);
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "gdn_prefill: launch failed: %s", cudaGetErrorString(e));
  return launch_status("gdn_prefill");
}

// Chooses the state slice width DVP and the number of chain CTAs. The kernel
// runs P = NC / slices chains (sequence-heads) at a time, in rounds, and
// prepares packages on the remaining CTAs; its time is about the larger of the
// two sides. Per-chunk costs (SM cycles) measured on B200: a chain step of one
// slice and the preparation of one (head, chunk) item. With several sequences a
// round lasts as long as its longest chain, so P is kept to a multiple or a
// divisor of Hv (whole sequences, or equal parts of one, per round) and a round
// of m sequences is charged the expected longest of m: 2m / (m + 1) times the
// mean length (the lengths are on the device; only their mean is known here).
struct PcPlan {
  int dvp;
  long nc;
};
PcPlan plan_pc(long chains, int64_t total_T, int n_seqs, int Hv, int sms) {
  const double kChainStep[3] = {1950.0, 2300.0, 3100.0};   // DVP 32, 64, 128
  const double kPrepItem = 10500.0;
  const double chunks = std::max(1.0, std::ceil((double)total_T / std::max(1, n_seqs) / 64.0));
  PcPlan best = {128, 1};
  double best_t = 1e300;
  for (int t = 0; t < 3; ++t) {
    const int dvp = 32 << t, slices = 128 / dvp;
    const long p_max = std::min({chains, (long)gdn::pc::kMaxPositions, ((long)sms - 8) / slices});
    for (long pos = 1; pos <= p_max; ++pos) {
      double maxf = 1.0;
      if (n_seqs > 1) {
        if (pos % Hv != 0 && Hv % pos != 0) continue;
        const double m = pos >= Hv ? (double)(pos / Hv) : 1.0;
        maxf = 2.0 * m / (m + 1.0);
      }
      const long nc = pos * slices;
      const double rounds = std::ceil((double)chains / pos);
      const double chain_t = rounds * chunks * maxf * kChainStep[t];
      const double prep_t = chains * chunks * kPrepItem / (double)(sms - nc);
      const double tt = std::max(chain_t, prep_t);
      if (tt < best_t * 0.999) {
        best_t = tt;
        best = {dvp, nc};
      }
    }
  }
  return best;
}

// The plan a launch uses: the model's choice, replaced field by field by the
// caller's request (a field of 0 keeps the model's value), clamped so that no
// position is without a chain, a chain's slices stay in one round and the
// package ring's positions suffice. The request is validated by the caller.
struct PcLaunchPlan {
  int dvp;
  long nc, rounds;
};
bool plan_request_ok(const gdn_plan* req) {
  if (!req) return true;
  return (req->dvp == 0 || req->dvp == 32 || req->dvp == 64 || req->dvp == 128) && req->n_chain_ctas >= 0;
}
PcLaunchPlan resolve_pc(long chains, int64_t total_T, int n_seqs, int Hv, int sms, const gdn_plan* req) {
  PcPlan plan = plan_pc(chains, total_T, n_seqs, Hv, sms);
  if (req && req->dvp != 0 && req->dvp != plan.dvp) {
    // another slice width: keep the model's number of chains per round
    plan.nc = plan.nc / (128 / plan.dvp) * (128 / req->dvp);
    plan.dvp = req->dvp;
  }
  const int dvp = plan.dvp, slices = 128 / dvp;
  long nc = plan.nc;
  if (req && req->n_chain_ctas > 0) nc = std::max(1, std::min(req->n_chain_ctas, sms - 1));
  nc = std::min(nc, (long)sms - 1);
  nc = std::min(nc, chains * slices);
  nc = std::min(nc, (long)gdn::pc::kMaxPositions * slices);
  nc -= nc % slices;
  if (nc < slices) nc = slices;
  return {dvp, nc, (chains * slices + nc - 1) / nc};
}

gdn_status launch_prefill_pc(const void* q, const void* k, const void* v, const float* g, const float* beta,
                             const float* state_in, const int32_t* cu, int n_seqs, int64_t total_T, int Hqk,
                             int Hv, float scale, gdn_dtype dtype, void* o, float* state_out, void* ws,
                             const gdn_plan* req, cudaStream_t st) {
  const long chains = (long)n_seqs * Hv;
  const int sms = sm_count();
  if (sms < 16) return fail(GDN_ERR_CUDA, "gdn_prefill: cannot query the multiprocessor count");
  const PcLaunchPlan lp = resolve_pc(chains, total_T, n_seqs, Hv, sms, req);
  const int dvp = lp.dvp, slices = 128 / dvp;
  const long nc = lp.nc;
  if (lp.rounds > gdn::pc::kMaxRounds)
    return fail(GDN_ERR_UNSUPPORTED, "gdn_prefill: %ld sequence-heads is more than this kernel schedules", chains);
  CUtensorMap qm, km, vm, om;
  const CUtensorMapDataType ty = dtype == GDN_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!make_map(&qm, q, 128, Hqk, (int)total_T, 64, ty) || !make_map(&km, k, 128, Hqk, (int)total_T, 64, ty) ||
      !make_map(&vm, v, 128, Hv, (int)total_T, std::min(dvp, 64), ty) ||
      !make_map(&om, o, 128, Hv, (int)total_T, std::min(dvp, 64), ty))
    return fail(GDN_ERR_CUDA, "gdn_prefill: cuTensorMapEncodeTiled unavailable or failed");
  cudaError_t e = cudaMemsetAsync(ws, 0, gdn::pc::Workspace::zeroed_bytes(nc / slices), st);
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "gdn_prefill: %s", cudaGetErrorString(e));
  gdn::pc::Params prm;
  prm.g = g;
  prm.beta = beta;
  prm.state_in = state_in;
  prm.cu_seqlens = cu;
  prm.o = o;
  prm.state_out = state_out;
  prm.ws = static_cast<uint8_t*>(ws);
  prm.n_seqs = n_seqs;
  prm.Hqk = Hqk;
  prm.Hv = Hv;
  prm.total_T = (int)total_T;
  prm.scale = scale;
  prm.n_chain_ctas = (int)nc;
  if (dtype == GDN_F16) {
    if (dvp == 32) return launch_pc<32, __half>(qm, km, vm, om, prm, sms, st);
    if (dvp == 64) return launch_pc<64, __half>(qm, km, vm, om, prm, sms, st);
    return launch_pc<128, __half>(qm, km, vm, om, prm, sms, st);
  }
  if (dvp == 32) return launch_pc<32, __nv_bfloat16>(qm, km, vm, om, prm, sms, st);
  if (dvp == 64) return launch_pc<64, __nv_bfloat16>(qm, km, vm, om, prm, sms, st);
  return launch_pc<128, __nv_bfloat16>(qm, km, vm, om, prm, sms, st);
}

// ------------------------------------------------------ linear attention ---
// Calls f with a null pointer of the C++ type of dtype.
template <typename F>
gdn_status with_dtype(gdn_dtype dtype, F f) {
  if (dtype == GDN_F32) return f(static_cast<float*>(nullptr));
  if (dtype == GDN_F16) return f(static_cast<__half*>(nullptr));
  return f(static_cast<__nv_bfloat16*>(nullptr));
}
// Calls f with dk as a compile-time constant.
template <typename F>
gdn_status with_dk(int dk, F f) {
  switch (dk) {
    case 16: return f(std::integral_constant<int, 16>());
    case 32: return f(std::integral_constant<int, 32>());
    case 64: return f(std::integral_constant<int, 64>());
    default: return f(std::integral_constant<int, 128>());
  }
}

constexpr int kLinearCtas = 148;   // CTAs that the workspace is laid out for: one on each SM

bool linear_on_tensor_cores(gdn_dtype dtype, int64_t total_T) { return dtype != GDN_F32 && total_T > 0; }

// Blocks of 128 tokens per segment. Fewer make more items, so that one sequence's
// heads fill the GPU and unequal sequences even out; more make fewer hand-overs of a
// state: eight packed sequences of 32 heads take 436 us with up to 8, 458 with up to 4 and
// 447 with up to 12 (32768 tokens, f16: 500, 521 and 502 to 514). The lengths are on the
// device: only their mean is known here.
int linear_segment(int n_seqs, int64_t total_T, int Hv) {
  const int64_t per_seq = std::max<int64_t>(1, (total_T / std::max(1, n_seqs) + 127) / 128);
  const int64_t blocks = per_seq * n_seqs * Hv;
  return (int)std::min<int64_t>(8, std::max<int64_t>(1, (blocks + kLinearCtas - 1) / kLinearCtas));
}

// fp32: tokens per segment, and the workspace of the segments' states (what precedes the
// states holds their decays). Splitting costs a second pass over k and v. Where the
// sequences' heads fill the GPU by themselves only those of twice the mean length are
// split (16 x 300 tokens, 32 heads of 128: 430 us, in segments for four waves 695); where a
// wave of resident CTAs holds two segments of each sequence or more, all of them are in one
// wave (3300 tokens, 16 heads of 64: 96 us, in segments for four waves 119; 4096 tokens, 16
// heads of 128: 307 and 330); in between, in about four. `resident` is what 148 SMs hold of
// the kernels' registers and shared memory with two rows a lane; on another device only the
// choice is off. The rule knows neither how the lengths differ nor what the last wave leaves
// empty: with 32 heads of 128, 8, 9, 10 and 12 sequences of 2000 tokens take 2.12, 1.53,
// 2.27 and 2.45 ms, and four of 20 tokens and four of 4000 2.03 ms.
struct ScanPlan {
  int seg;
  int64_t segments;    // at most
  size_t decay_bytes, bytes;
};
ScanPlan scan_plan(int n_seqs, int64_t total_T, int Hv, int dk, int dv) {
  ScanPlan s;
  const int64_t rows = (dv + gdn::lin::scan_rows(dv) - 1) / gdn::lin::scan_rows(dv);
  const int64_t resident = 148 * (dk == 128 ? 4 : 5), per_wave = resident / (Hv * rows);
  const int64_t want = per_wave > 2 * n_seqs ? per_wave - n_seqs
                       : per_wave > n_seqs   ? 4 * resident / (Hv * rows)
                                             : std::max(1, n_seqs / 2);
  s.seg = (int)std::min<int64_t>(std::max<int64_t>(64, (total_T / want + 16) / 16 * 16), 1 << 30);
  s.segments = total_T / s.seg + n_seqs;
  s.decay_bytes = ((size_t)s.segments * Hv * 8 + 255) & ~size_t(255);
  s.bytes = total_T <= s.seg ? 0 : s.decay_bytes + (size_t)s.segments * Hv * dv * dk * 4;
  return s;
}

template <typename T>
gdn_status launch_linear_tc(const char* fn, const void* q, const void* k, const void* v, int64_t total_T,
                            gdn::ltc::Params prm, CUtensorMapDataType ty, cudaStream_t st) {
  const int sms = sm_count();
  if (sms < 16) return fail(GDN_ERR_CUDA, "%s: cannot query the multiprocessor count", fn);
  const int64_t items = (total_T / (prm.seg * gdn::ltc::kB) + prm.n_seqs) * prm.Hv;   // at most
  const int grid = (int)std::min<int64_t>(prm.ws ? INT64_MAX : items, std::min(sms, kLinearCtas));
  prm.items = (int)items;
  prm.panel = std::min(prm.Hv, gdn::ltc::kScanWarps * grid / gdn::ltc::kSlices);
  if (!prm.ws) prm.panel = prm.Hv;
  // about 2 s, and ten times what the blocks take (4000 cycles each)
  prm.limit = 4000000000ll + (total_T / gdn::ltc::kB + prm.n_seqs) * prm.Hv / grid * 40000;
  CUtensorMap qm, km, vm, om;
  if (!make_map(&qm, q, prm.dk, prm.Hqk, (int)total_T, 64, ty, gdn::ltc::kB) ||
      !make_map(&km, k, prm.dk, prm.Hqk, (int)total_T, 64, ty, gdn::ltc::kB) ||
      !make_map(&vm, v, prm.dv, prm.Hv, (int)total_T, 64, ty, gdn::ltc::kB) ||
      !make_map(&om, prm.o, prm.dv, prm.Hv, (int)total_T, 64, ty, 32))
    return fail(GDN_ERR_CUDA, "%s: cuTensorMapEncodeTiled unavailable or failed", fn);
  auto kern = prm.dk == gdn::ltc::kD && prm.dv == gdn::ltc::kD ? gdn::ltc::prefill_kernel<T, true>
                                                               : gdn::ltc::prefill_kernel<T, false>;
  if (gdn_status s = allow_smem(kern, fn)) return s;
  if (prm.ws) {
    cudaError_t e = cudaMemsetAsync(prm.ws, 0, gdn::ltc::Workspace::flags_bytes(grid), st);
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(gdn::ltc::kThreads);
  cfg.dynamicSmemBytes = gdn::ltc::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;   // with segments CTAs wait on one another: every one co-resident
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = prm.ws ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, qm, km, vm, om, prm);
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  return launch_status(fn);
}

template <typename TS>
gdn_status linear_decode(const char* fn, const void* q, const void* k, const void* v, const float* g, int g_stride,
                         TS* state, int B, int Hqk, int Hv, int dk, int dv, float scale, gdn_dtype dtype, void* o,
                         void* stream) {
  bool done = false;
  // (g stands in for the beta of the shared checks)
  if (gdn_status s = check_decode(fn, q, k, v, g, g, state, B, Hqk, Hv, dk, dv, dtype, o, &done)) return s;
  if (g_stride != 0 && g_stride != Hv)
    return fail(GDN_ERR_INVALID_ARG, "%s: g_stride=%d (0 or Hv=%d)", fn, g_stride, Hv);
  if ((int64_t)B * Hv * 8 > 0x7fffffff) return fail(GDN_ERR_INVALID_ARG, "%s: B*Hv too large", fn);   // (8 CTAs a head at most)
  if (done) return ok();
  if (scale <= 0.f) scale = 1.0f / sqrtf((float)dk);
  return with_dtype(dtype, [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    return with_dk(dk, [&](auto dkc) {
      constexpr int DK = decltype(dkc)::value;
      constexpr int kRows = gdn::lin::LinearDecodeShape<DK, TS>::kRowsPerCta;
      const int parts = (dv + kRows - 1) / kRows;
      gdn::lin::decode_kernel<T, DK, TS>
          <<<(unsigned)(B * Hv) * parts, gdn::lin::kDecodeWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(
              static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), g, g_stride, state, Hqk, Hv,
              dv, parts, scale, static_cast<T*>(o));
      return launch_status(fn);
    });
  });
}

// ------------------------------------------------------------ state pool ---
gdn_status check_pool(const char* fn, const void* state, gdn_dtype state_dtype, const int32_t* slots, int n,
                      int n_slots, int Hv, int dk, int dv, gdn_code code, const void* codes, const uint8_t* exps,
                      bool* done) {
  *done = false;
  if (n < 0 || n_slots < 0) return fail(GDN_ERR_INVALID_ARG, "%s: n=%d, n_slots=%d", fn, n, n_slots);
  if (Hv <= 0) return fail(GDN_ERR_INVALID_ARG, "%s: Hv=%d", fn, Hv);
  if (!head_dim_ok(dk) || !head_dim_ok(dv))
    return fail(GDN_ERR_UNSUPPORTED, "%s: dk=%d, dv=%d (supported: 16, 32, 64, 128)", fn, dk, dv);
  if (state_dtype != GDN_F32 && state_dtype != GDN_BF16)
    return fail(GDN_ERR_INVALID_ARG, "%s: state type %d (GDN_F32 or GDN_BF16)", fn, (int)state_dtype);
  if (code != GDN_CODE_E4M3 && code != GDN_CODE_I8) return fail(GDN_ERR_INVALID_ARG, "%s: unknown code %d", fn, (int)code);
  const int64_t tiles = ((int64_t)Hv * dv * dk + gdn::pool::kTile - 1) / gdn::pool::kTile;
  if (n > 0 && tiles > 0x7fffffff / n) return fail(GDN_ERR_INVALID_ARG, "%s: n*Hv too large", fn);
  if (n == 0) {
    *done = true;
    return ok();
  }
  if (!state || !slots || (n_slots > 0 && (!codes || !exps)))
    return fail(GDN_ERR_INVALID_ARG, "%s: pointers must not be NULL", fn);
  if (!aligned16(state) || !aligned16(codes))
    return fail(GDN_ERR_INVALID_ARG, "%s: state and codes must be 16-byte aligned", fn);
  if (!aligned4(slots)) return fail(GDN_ERR_INVALID_ARG, "%s: slots must be 4-byte aligned", fn);
  return GDN_OK;
}

template <typename F>
gdn_status with_pool_types(gdn_code code, gdn_dtype state_dtype, int dk, F f) {
  auto group = [&](auto c, auto* s) {
    return dk == 16 ? f(c, s, std::integral_constant<int, 4>()) : f(c, s, std::integral_constant<int, 8>());
  };
  auto st = [&](auto c) {
    return state_dtype == GDN_F32 ? group(c, static_cast<float*>(nullptr))
                                  : group(c, static_cast<__nv_bfloat16*>(nullptr));
  };
  return code == GDN_CODE_E4M3 ? st(gdn::pool::E4M3()) : st(gdn::pool::I8());
}

}  // namespace

extern "C" {

size_t gdn_linear_prefill_workspace_bytes(int n_seqs, int64_t total_T, int Hv, int dk, int dv, gdn_dtype dtype) {
  if (n_seqs <= 0 || Hv <= 0 || total_T <= 0 || total_T >= (int64_t(1) << 31) || !head_dim_ok(dk) || !head_dim_ok(dv))
    return 0;   // (gdn_linear_prefill refuses it, or has nothing to do)
  if (!linear_on_tensor_cores(dtype, total_T)) return scan_plan(n_seqs, total_T, Hv, dk, dv).bytes;
  // sequences of one segment need none
  if (total_T <= (int64_t)linear_segment(n_seqs, total_T, Hv) * gdn::ltc::kB) return 0;
  return gdn::ltc::Workspace::bytes(kLinearCtas);
}

gdn_status gdn_linear_prefill(const void* q, const void* k, const void* v, const float* g, int g_stride,
                              const float* state_in, const int32_t* cu_seqlens, int n_seqs, int64_t total_T, int Hqk,
                              int Hv, int dk, int dv, float scale, gdn_dtype dtype, void* o, float* state_out,
                              void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "gdn_linear_prefill";
  if (n_seqs < 0) return fail(GDN_ERR_INVALID_ARG, "%s: n_seqs=%d < 0", fn, n_seqs);
  if (total_T < 0 || total_T >= (int64_t(1) << 31))
    return fail(GDN_ERR_INVALID_ARG, "%s: total_T=%lld out of range", fn, (long long)total_T);
  if (Hqk <= 0 || Hv <= 0 || Hv % Hqk != 0)
    return fail(GDN_ERR_INVALID_ARG, "%s: Hv=%d must be a positive multiple of Hqk=%d", fn, Hv, Hqk);
  if (!head_dim_ok(dk) || !head_dim_ok(dv))
    return fail(GDN_ERR_UNSUPPORTED, "%s: dk=%d, dv=%d (supported: 16, 32, 64, 128)", fn, dk, dv);
  if (!dtype_ok(dtype)) return fail(GDN_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
  if (g_stride != 0 && g_stride != Hv)
    return fail(GDN_ERR_INVALID_ARG, "%s: g_stride=%d (0 or Hv=%d)", fn, g_stride, Hv);
  if (n_seqs > 65535 || Hv > 65535)
    return fail(GDN_ERR_UNSUPPORTED, "%s: n_seqs=%d, Hv=%d (at most 65535 each)", fn, n_seqs, Hv);
  if (n_seqs == 0) return ok();
  if (!cu_seqlens || !state_out)
    return fail(GDN_ERR_INVALID_ARG, "%s: cu_seqlens and state_out must not be NULL", fn);
  if (total_T > 0 && (!q || !k || !v || !g || !o))
    return fail(GDN_ERR_INVALID_ARG, "%s: q, k, v, g and o must not be NULL", fn);
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(state_out) || !aligned16(state_in))
    return fail(GDN_ERR_INVALID_ARG, "%s: q, k, v, o and the states must be 16-byte aligned", fn);
  if (!aligned4(g) || !aligned4(cu_seqlens))
    return fail(GDN_ERR_INVALID_ARG, "%s: g and cu_seqlens must be 4-byte aligned", fn);
  const size_t need = gdn_linear_prefill_workspace_bytes(n_seqs, total_T, Hv, dk, dv, dtype);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return fail(GDN_ERR_INVALID_ARG, "%s: workspace needs %zu bytes (16-byte aligned), got %zu", fn, need,
                workspace_bytes);
  if (scale <= 0.f) scale = 1.0f / sqrtf((float)dk);
  if (linear_on_tensor_cores(dtype, total_T)) {
    const int seg = linear_segment(n_seqs, total_T, Hv);
    if ((total_T / (seg * gdn::ltc::kB) + n_seqs) * Hv > 0x7fff0000)
      return fail(GDN_ERR_UNSUPPORTED, "%s: %d sequences, %lld tokens, %d heads are more than this kernel schedules", fn,
                  n_seqs, (long long)total_T, Hv);
    gdn::ltc::Params prm = {};
    prm.q = q;
    prm.k = k;
    prm.v = v;
    prm.g = g;
    prm.state_in = state_in;
    prm.cu_seqlens = cu_seqlens;
    prm.o = o;
    prm.state_out = state_out;
    prm.ws = need > 0 ? static_cast<uint8_t*>(workspace) : nullptr;
    prm.g_stride = g_stride;
    prm.n_seqs = n_seqs;
    prm.total_T = (int)total_T;
    prm.Hqk = Hqk;
    prm.Hv = Hv;
    prm.dk = dk;
    prm.dv = dv;
    prm.seg = seg;
    prm.scale = scale;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == GDN_F16)
      return launch_linear_tc<__half>(fn, q, k, v, total_T, prm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, st);
    return launch_linear_tc<__nv_bfloat16>(fn, q, k, v, total_T, prm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, st);
  }
  // fp32 (and no tokens at all, where only the states are copied)
  const ScanPlan plan = scan_plan(n_seqs, total_T, Hv, dk, dv);
  gdn::lin::ScanParams prm = {};
  prm.g = g;
  prm.state_in = state_in;
  prm.cu_seqlens = cu_seqlens;
  prm.state_out = state_out;
  prm.decays = static_cast<float2*>(workspace);
  prm.states = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.decay_bytes);
  prm.g_stride = g_stride;
  prm.n_seqs = n_seqs;
  prm.total_T = (int)total_T;
  prm.Hqk = Hqk;
  prm.Hv = Hv;
  prm.dv = dv;
  prm.seg = plan.seg;
  prm.segments = (int)plan.segments;
  prm.scale = scale;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto run = [&](auto dkc, auto rows) {
    constexpr int DK = decltype(dkc)::value, R = decltype(rows)::value;
    const dim3 grid((unsigned)plan.segments, (unsigned)Hv, (unsigned)((dv + 32 * R - 1) / (32 * R)));
    const auto *qf = static_cast<const float*>(q), *kf = static_cast<const float*>(k), *vf = static_cast<const float*>(v);
    auto* of = static_cast<float*>(o);
    if (need > 0) {
      gdn::lin::scan_kernel<DK, R, false><<<grid, gdn::lin::kScanThreads, 0, st>>>(qf, kf, vf, of, prm);
      if (gdn_status s = launch_status(fn)) return s;
      gdn::lin::combine_kernel<<<dim3((unsigned)((dv * DK + 1023) / 1024), (unsigned)Hv, (unsigned)n_seqs), 256, 0, st>>>(
          prm, dv * DK);
      if (gdn_status s = launch_status(fn)) return s;
    }
    gdn::lin::scan_kernel<DK, R, true><<<grid, gdn::lin::kScanThreads, 0, st>>>(qf, kf, vf, of, prm);
    return launch_status(fn);
  };
  return with_dk(dk, [&](auto dkc) {
    return gdn::lin::scan_rows_per_lane(dv) == 2 ? run(dkc, std::integral_constant<int, 2>())
                                                 : run(dkc, std::integral_constant<int, 1>());
  });
}

gdn_status gdn_linear_decode(const void* q, const void* k, const void* v, const float* g, int g_stride, float* state,
                             int B, int Hqk, int Hv, int dk, int dv, float scale, gdn_dtype dtype, void* o,
                             void* stream) {
  return linear_decode("gdn_linear_decode", q, k, v, g, g_stride, state, B, Hqk, Hv, dk, dv, scale, dtype, o, stream);
}

gdn_status gdn_linear_decode_bf16_state(const void* q, const void* k, const void* v, const float* g, int g_stride,
                                        void* state, int B, int Hqk, int Hv, int dk, int dv, float scale,
                                        gdn_dtype dtype, void* o, void* stream) {
  return linear_decode("gdn_linear_decode_bf16_state", q, k, v, g, g_stride, static_cast<__nv_bfloat16*>(state), B,
                       Hqk, Hv, dk, dv, scale, dtype, o, stream);
}

gdn_status gdn_state_store(const void* state, gdn_dtype state_dtype, const int32_t* slots, int n, int n_slots, int Hv,
                           int dk, int dv, gdn_code code, void* codes, uint8_t* exps, void* stream) {
  bool done = false;
  if (gdn_status s = check_pool("gdn_state_store", state, state_dtype, slots, n, n_slots, Hv, dk, dv, code, codes,
                                exps, &done))
    return s;
  if (done) return ok();
  const long long per_state = (long long)Hv * dv * dk;
  const int tiles = (int)((per_state + gdn::pool::kTile - 1) / gdn::pool::kTile);
  return with_pool_types(code, state_dtype, dk, [&](auto c, auto* tag, auto grp) {
    using TS = std::remove_pointer_t<decltype(tag)>;
    gdn::pool::store_kernel<decltype(c), TS, decltype(grp)::value>
        <<<(unsigned)n * tiles, gdn::pool::kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
            static_cast<const TS*>(state), slots, n, n_slots, tiles, per_state, static_cast<uint32_t*>(codes), exps);
    return launch_status("gdn_state_store");
  });
}

gdn_status gdn_state_load(const void* codes, const uint8_t* exps, const int32_t* slots, int n, int n_slots, int Hv,
                          int dk, int dv, gdn_code code, void* state, gdn_dtype state_dtype, void* stream) {
  bool done = false;
  if (gdn_status s = check_pool("gdn_state_load", state, state_dtype, slots, n, n_slots, Hv, dk, dv, code, codes, exps,
                                &done))
    return s;
  if (done) return ok();
  const long long per_state = (long long)Hv * dv * dk;
  const int tiles = (int)((per_state + gdn::pool::kTile - 1) / gdn::pool::kTile);
  return with_pool_types(code, state_dtype, dk, [&](auto c, auto* tag, auto grp) {
    using TS = std::remove_pointer_t<decltype(tag)>;
    gdn::pool::load_kernel<decltype(c), TS, decltype(grp)::value>
        <<<(unsigned)n * tiles, gdn::pool::kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
            static_cast<const uint32_t*>(codes), exps, slots, n_slots, tiles, per_state, static_cast<TS*>(state));
    return launch_status("gdn_state_load");
  });
}

int gdn_version(void) { return (0 << 16) | 5; }

const char* gdn_last_error(void) { return t_last_error.c_str(); }

size_t gdn_prefill_workspace_bytes(int n_seqs, int Hv, int dk, int dv, gdn_dtype dtype) {
  if (n_seqs <= 0 || Hv <= 0 || !uses_pc_prefill(dtype, dk, dv)) return 0;
  return gdn::pc::Workspace::bytes(std::min((long)n_seqs * Hv, (long)gdn::pc::kMaxPositions));
}

gdn_status gdn_prefill_plan(int n_seqs, int64_t total_T, int Hv, int dk, int dv, gdn_dtype dtype, int sm_count_arg,
                            const gdn_plan* requested, int* dvp, int* n_chain_ctas, int* rounds) {
  t_last_error.clear();
  if (!dvp || !n_chain_ctas || !rounds) return fail(GDN_ERR_INVALID_ARG, "gdn_prefill_plan: null output");
  if (!plan_request_ok(requested))
    return fail(GDN_ERR_INVALID_ARG, "gdn_prefill_plan: requested dvp %d (0, 32, 64 or 128), n_chain_ctas %d (>= 0)",
                requested->dvp, requested->n_chain_ctas);
  if (n_seqs <= 0 || Hv <= 0 || total_T < 0)
    return fail(GDN_ERR_INVALID_ARG, "gdn_prefill_plan: n_seqs %d, Hv %d, total_T %lld", n_seqs, Hv,
                (long long)total_T);
  if (!uses_pc_prefill(dtype, dk, dv))
    return fail(GDN_ERR_UNSUPPORTED, "gdn_prefill_plan: the tensor-core kernel takes bf16 or f16 with dk = dv = 128");
  const int sms = sm_count_arg > 0 ? sm_count_arg : sm_count();
  if (sms < 16) return fail(GDN_ERR_INVALID_ARG, "gdn_prefill_plan: %d multiprocessors", sms);
  const PcLaunchPlan lp = resolve_pc((long)n_seqs * Hv, total_T, n_seqs, Hv, sms, requested);
  *dvp = lp.dvp;
  *n_chain_ctas = (int)lp.nc;
  *rounds = (int)std::min(lp.rounds, (long)INT32_MAX);
  return GDN_OK;
}

gdn_status gdn_prefill_ex(const void* q, const void* k, const void* v, const float* g,
                          const float* beta, const float* state_in, const int32_t* cu_seqlens,
                          int n_seqs, int64_t total_T, int Hqk, int Hv, int dk, int dv, float scale,
                          int chunk, gdn_dtype dtype, void* o, float* state_out, void* workspace,
                          size_t workspace_bytes, const gdn_plan* plan, void* stream) {
  if (!plan_request_ok(plan))
    return fail(GDN_ERR_INVALID_ARG, "gdn_prefill: plan dvp %d (0, 32, 64 or 128), n_chain_ctas %d (>= 0)",
                plan->dvp, plan->n_chain_ctas);
  if (n_seqs < 0) return fail(GDN_ERR_INVALID_ARG, "gdn_prefill: n_seqs=%d < 0", n_seqs);
  if (total_T < 0 || total_T >= (int64_t(1) << 31))
    return fail(GDN_ERR_INVALID_ARG, "gdn_prefill: total_T=%lld out of range", (long long)total_T);
  if (Hqk <= 0 || Hv <= 0 || Hv % Hqk != 0)
    return fail(GDN_ERR_INVALID_ARG, "gdn_prefill: Hv=%d must be a positive multiple of Hqk=%d", Hv, Hqk);
  if (!head_dim_ok(dk) || !head_dim_ok(dv))
    return fail(GDN_ERR_UNSUPPORTED, "gdn_prefill: dk=%d, dv=%d (supported: 16, 32, 64, 128)", dk, dv);
  if (!dtype_ok(dtype)) return fail(GDN_ERR_INVALID_ARG, "gdn_prefill: unknown dtype %d", (int)dtype);
  if (n_seqs == 0) return ok();
  if (!cu_seqlens || !state_out)
    return fail(GDN_ERR_INVALID_ARG, "gdn_prefill: cu_seqlens and state_out must not be NULL");
  if (total_T > 0 && (!q || !k || !v || !g || !beta || !o))
    return fail(GDN_ERR_INVALID_ARG, "gdn_prefill: q, k, v, g, beta and o must not be NULL");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(state_out) ||
      !aligned16(state_in))
    return fail(GDN_ERR_INVALID_ARG, "gdn_prefill: q, k, v, o and the states must be 16-byte aligned");
  if (!aligned4(g) || !aligned4(beta) || !aligned4(cu_seqlens))
    return fail(GDN_ERR_INVALID_ARG, "gdn_prefill: g, beta and cu_seqlens must be 4-byte aligned");
  if (scale <= 0.f) scale = 1.0f / sqrtf((float)dk);
  int C = chunk;
  if (C == 0) C = uses_pc_prefill(dtype, dk, dv) ? 64 : 16;
  if (C != 16 && C != 32 && C != 64)
    return fail(GDN_ERR_UNSUPPORTED, "gdn_prefill: chunk=%d (supported: 16, 32, 64)", C);
  const size_t need = gdn_prefill_workspace_bytes(n_seqs, Hv, dk, dv, dtype);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return fail(GDN_ERR_INVALID_ARG, "gdn_prefill: workspace needs %zu bytes (16-byte aligned), got %zu",
                need, workspace_bytes);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (uses_pc_prefill(dtype, dk, dv) && C == 64 && total_T > 0)
    return launch_prefill_pc(q, k, v, g, beta, state_in, cu_seqlens, n_seqs, total_T, Hqk, Hv, scale, dtype, o,
                             state_out, workspace, plan, st);
  if (dtype == GDN_F32)
    return launch_prefill_simt<float>(q, k, v, g, beta, state_in, cu_seqlens, n_seqs, total_T, Hqk,
                                      Hv, dk, dv, scale, C, o, state_out, st);
  if (dtype == GDN_F16)
    return launch_prefill_simt<__half>(q, k, v, g, beta, state_in, cu_seqlens, n_seqs, total_T, Hqk,
                                       Hv, dk, dv, scale, C, o, state_out, st);
  return launch_prefill_simt<__nv_bfloat16>(q, k, v, g, beta, state_in, cu_seqlens, n_seqs, total_T,
                                            Hqk, Hv, dk, dv, scale, C, o, state_out, st);
}

gdn_status gdn_prefill(const void* q, const void* k, const void* v, const float* g,
                       const float* beta, const float* state_in, const int32_t* cu_seqlens,
                       int n_seqs, int64_t total_T, int Hqk, int Hv, int dk, int dv, float scale,
                       int chunk, gdn_dtype dtype, void* o, float* state_out, void* workspace,
                       size_t workspace_bytes, void* stream) {
  return gdn_prefill_ex(q, k, v, g, beta, state_in, cu_seqlens, n_seqs, total_T, Hqk, Hv, dk, dv, scale, chunk,
                        dtype, o, state_out, workspace, workspace_bytes, nullptr, stream);
}

gdn_status gdn_decode(const void* q, const void* k, const void* v, const float* g,
                      const float* beta, float* state, int B, int Hqk, int Hv, int dk, int dv,
                      float scale, gdn_dtype dtype, void* o, void* stream) {
  bool done = false;
  if (gdn_status s = check_decode("gdn_decode", q, k, v, g, beta, state, B, Hqk, Hv, dk, dv, dtype, o, &done))
    return s;
  if (done) return ok();
  if (scale <= 0.f) scale = 1.0f / sqrtf((float)dk);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == GDN_F32)
    return dispatch_decode<float, float>(q, k, v, g, beta, state, B, Hqk, Hv, dk, dv, scale, o, st);
  if (dtype == GDN_F16)
    return dispatch_decode<__half, float>(q, k, v, g, beta, state, B, Hqk, Hv, dk, dv, scale, o, st);
  return dispatch_decode<__nv_bfloat16, float>(q, k, v, g, beta, state, B, Hqk, Hv, dk, dv, scale, o, st);
}

gdn_status gdn_decode_bf16_state(const void* q, const void* k, const void* v, const float* g,
                                 const float* beta, void* state, int B, int Hqk, int Hv, int dk, int dv,
                                 float scale, gdn_dtype dtype, void* o, void* stream) {
  bool done = false;
  if (gdn_status s =
          check_decode("gdn_decode_bf16_state", q, k, v, g, beta, state, B, Hqk, Hv, dk, dv, dtype, o, &done))
    return s;
  if (done) return ok();
  if (scale <= 0.f) scale = 1.0f / sqrtf((float)dk);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto* s16 = static_cast<__nv_bfloat16*>(state);
  if (dtype == GDN_F32)
    return dispatch_decode<float, __nv_bfloat16>(q, k, v, g, beta, s16, B, Hqk, Hv, dk, dv, scale, o, st);
  if (dtype == GDN_F16)
    return dispatch_decode<__half, __nv_bfloat16>(q, k, v, g, beta, s16, B, Hqk, Hv, dk, dv, scale, o, st);
  return dispatch_decode<__nv_bfloat16, __nv_bfloat16>(q, k, v, g, beta, s16, B, Hqk, Hv, dk, dv, scale, o, st);
}

gdn_status gdn_wait_selftest(int max_wait_us, void* stream) {
  if (max_wait_us < 1 || max_wait_us > 1000000)
    return fail(GDN_ERR_INVALID_ARG, "gdn_wait_selftest: max_wait_us=%d outside [1, 1000000]", max_wait_us);
  const long long cycles = (long long)max_wait_us * 2000;   // ~2 GHz SM clock
  wait_selftest_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(cycles);
  if (gdn_status s = launch_status("gdn_wait_selftest")) return s;
  gdn::ltc::wait_selftest_kernel<<<3, 96, 0, static_cast<cudaStream_t>(stream)>>>(cycles);
  return launch_status("gdn_wait_selftest");
}

gdn_status gdn_device_error(void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  unsigned int word = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&word, gdn::g_error_word, sizeof word, 0,
                                            cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "gdn_device_error: %s", cudaGetErrorString(e));
  if (word) {
    unsigned int line = 0;
    e = cudaMemcpyFromSymbolAsync(&line, gdn::g_error_line, sizeof line, 0, cudaMemcpyDeviceToHost, st);
    const unsigned int zero = 0;
    if (e == cudaSuccess)
      e = cudaMemcpyToSymbolAsync(gdn::g_error_word, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess)
      e = cudaMemcpyToSymbolAsync(gdn::g_error_line, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "gdn_device_error: %s", cudaGetErrorString(e));
    if (word & gdn::kErrCheck)
      return fail(GDN_ERR_DEVICE_CHECK, "an index check of the GDN_DEBUG build failed (source line %u, error word 0x%x)",
                  line, word);
    return fail(GDN_ERR_DEVICE_TIMEOUT, "a bounded device wait ran out (error word 0x%x)", word);
  }
  return ok();
}

int gdn_debug_checks(void) {
#ifdef GDN_DEBUG
  return 1;
#else
  return 0;
#endif
}

}  // extern "C"

// ============================================================================
// Allocation-free prefill.
//
// Some callers cannot hand the library any device memory of its own making:
// code that runs where cudaMalloc is not allowed or not wanted -- inside a
// region whose memory was planned ahead of time by an inference runtime, a
// plugin whose host framework owns every allocation, or a real-time loop where
// an allocator call could stall or fail. gdn_prefill needs a workspace (the
// package ring the preparation and chain CTAs exchange data through), so for
// those callers this file keeps one statically sized scratch array in device
// memory and gdn_prefill_noalloc runs the same kernel on it.
//
// The array lives as long as the library is loaded, on every device that
// loads it. Host code must never use the array's name as a device pointer:
// its device address is looked up with cudaGetSymbolAddress, with the device
// current. The address belongs to the CUDA context the module was loaded in,
// so it is cached per device together with that context's id and looked up
// again on every call made outside stream capture (a cheap host-side query);
// a call under capture uses the cached address, which must come from an
// earlier call in the same context. Every call shares the array: the parts
// that must start at zero are cleared by each call on its stream, and two
// calls whose kernels overlap on the GPU (different streams, or different
// host threads) race on it and must be serialised by the caller.
// ============================================================================
namespace {

// The largest workspace gdn_prefill can ask for (the ring of kMaxPositions
// positions), rounded up to whole MiB: every problem gdn_prefill runs fits.
constexpr size_t kNoAllocScratchBytes =
    (gdn::pc::Workspace::bytes(gdn::pc::kMaxPositions) + (size_t(1) << 20) - 1) & ~((size_t(1) << 20) - 1);
static __device__ __align__(256) uint8_t g_noalloc_scratch[kNoAllocScratchBytes];

constexpr int kMaxDevices = 64;
struct NoAllocAddr {
  unsigned long long ctx_id;   // the context the address was looked up in
  void* ptr;
};
std::mutex g_noalloc_mu;
NoAllocAddr g_noalloc_addr[kMaxDevices] = {};

// Id of the calling thread's current CUDA context (driver entry points looked
// up once); false if there is none or the driver lacks the query.
bool current_context_id(unsigned long long* id) {
  static std::once_flag once;
  static PFN_cuCtxGetCurrent_v4000 get_current = nullptr;
  static PFN_cuCtxGetId_v12000 get_id = nullptr;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_current = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(p);
    p = nullptr;
    if (cudaGetDriverEntryPoint("cuCtxGetId", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_id = reinterpret_cast<PFN_cuCtxGetId_v12000>(p);
  });
  if (!get_current || !get_id) return false;
  CUcontext ctx = nullptr;
  if (get_current(&ctx) != CUDA_SUCCESS || !ctx) return false;
  return get_id(ctx, id) == CUDA_SUCCESS;
}

gdn_status noalloc_scratch(cudaStream_t st, void** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "gdn_prefill_noalloc: %s", cudaGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices)
    return fail(GDN_ERR_UNSUPPORTED, "gdn_prefill_noalloc: device %d beyond %d", dev, kMaxDevices);
  // (a runtime call on the stream also makes the device's context current)
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  e = cudaStreamIsCapturing(st, &cap);
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "gdn_prefill_noalloc: %s", cudaGetErrorString(e));
  unsigned long long ctx = 0;
  if (!current_context_id(&ctx))
    return fail(GDN_ERR_CUDA, "gdn_prefill_noalloc: cannot identify the current CUDA context");
  std::lock_guard<std::mutex> lock(g_noalloc_mu);
  NoAllocAddr& a = g_noalloc_addr[dev];
  if (cap == cudaStreamCaptureStatusNone) {
    void* ptr = nullptr;
    e = cudaGetSymbolAddress(&ptr, g_noalloc_scratch);
    if (e != cudaSuccess || !ptr)
      return fail(GDN_ERR_CUDA, "gdn_prefill_noalloc: cudaGetSymbolAddress failed: %s", cudaGetErrorString(e));
    a = {ctx, ptr};
  } else if (!a.ptr || a.ctx_id != ctx) {
    return fail(GDN_ERR_CUDA,
                "gdn_prefill_noalloc: called under stream capture before any call outside capture in this "
                "CUDA context (the scratch address is looked up outside capture)");
  }
  *out = a.ptr;
  return GDN_OK;
}

}  // namespace

extern "C" gdn_status gdn_prefill_noalloc(const void* q, const void* k, const void* v, const float* g,
                                          const float* beta, const float* state_in,
                                          const int32_t* cu_seqlens, int n_seqs, int64_t total_T, int Hqk,
                                          int Hv, int dk, int dv, float scale, int chunk, gdn_dtype dtype,
                                          void* o, float* state_out, void* stream) {
  if (dtype != GDN_BF16 || dk != 128 || dv != 128 || (chunk != 0 && chunk != 64))
    return fail(GDN_ERR_UNSUPPORTED,
                "gdn_prefill_noalloc: only bf16 with dk = dv = 128 and chunk 64 (the tensor-core kernel)");
  if (n_seqs > 0 && Hv > 0) {
    const size_t need = gdn_prefill_workspace_bytes(n_seqs, Hv, dk, dv, dtype);
    if (need > kNoAllocScratchBytes)
      return fail(GDN_ERR_UNSUPPORTED,
                  "gdn_prefill_noalloc: %d sequences x %d heads need %zu bytes of scratch, more than the %zu "
                  "bytes built into the library; use gdn_prefill with a workspace",
                  n_seqs, Hv, need, kNoAllocScratchBytes);
  }
  void* scratch = nullptr;
  if (gdn_status s = noalloc_scratch(static_cast<cudaStream_t>(stream), &scratch)) return s;
  return gdn_prefill(q, k, v, g, beta, state_in, cu_seqlens, n_seqs, total_T, Hqk, Hv, dk, dv, scale, chunk,
                     dtype, o, state_out, scratch, kNoAllocScratchBytes, stream);
}
