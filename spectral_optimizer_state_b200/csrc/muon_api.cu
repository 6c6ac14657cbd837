// C-ABI of libmuon: argument checks, workspace, tensor maps and the launch
// sequence of one Muon step (momentum pass, k Newton-Schulz iterations of
// three tensor-core products each, the last one applying the update).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <vector>

#include "../../include/muon.h"
#include "blocks.h"
#include "device_utils.cuh"
#include "experts.h"
#include "internal.h"

using namespace muon;

namespace {

// ------------------------------------------------------------------ errors
char g_cuda_error[256] = "";
std::mutex g_err_mu;

muon_status cuda_fail(cudaError_t e, const char* what) {
  std::lock_guard<std::mutex> lk(g_err_mu);
  std::snprintf(g_cuda_error, sizeof(g_cuda_error), "%s: %s", what, cudaGetErrorString(e));
  return MUON_ERR_CUDA;
}

#define MUON_CUDA(call, what)                          \
  do {                                                 \
    cudaError_t _e = (call);                           \
    if (_e != cudaSuccess) return cuda_fail(_e, what); \
  } while (0)

// Capture state of `s`: 0 not capturing, 1 capturing into a CUDA graph, -1 unreadable.
int capture_state(cudaStream_t s) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &cs) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  return cs == cudaStreamCaptureStatusNone ? 0 : 1;
}

muon_status refuse_growth(const char* what, const char* why) {
  std::lock_guard<std::mutex> lk(g_err_mu);
  std::snprintf(g_cuda_error, sizeof(g_cuda_error), "%s must grow, but %s", what, why);
  return MUON_ERR_ALLOC;
}

// Records why a device allocation failed (and clears the error) for muon_last_cuda_error.
void note_alloc_failure() {
  const cudaError_t e = cudaGetLastError();
  std::lock_guard<std::mutex> lk(g_err_mu);
  std::snprintf(g_cuda_error, sizeof(g_cuda_error), "device allocation: %s", cudaGetErrorString(e));
}

// ------------------------------------------------------------------ tensor maps
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encoder() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// bf16 buffer [planes][L][rows][pitch] viewed as 4-D {cols, rows, L, planes};
// box {box_cols, box_rows}.  Operand maps use the 128-byte swizzle the UMMA
// descriptors expect; store maps use the 64-byte swizzle of the epilogue's
// 32 x 32 staging tiles.  Out-of-range reads give zeros, stores are clipped.
bool encode_map(CUtensorMap* map, const void* base, int cols, int rows, int L, int planes,
                int pitch, int box_cols, int box_rows,
                CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B) {
  EncodeTiledFn enc = get_encoder();
  if (!enc) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(L), static_cast<cuuint64_t>(planes)};
  const cuuint64_t row_bytes = static_cast<cuuint64_t>(pitch) * 2;
  cuuint64_t strides[3] = {row_bytes, row_bytes * rows, row_bytes * rows * L};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

constexpr float kQuintic[3] = {3.4445f, -4.7750f, 2.0315f};

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
int round8(int x) { return (x + 7) / 8 * 8; }
int round64(int x) { return (x + 63) / 64 * 64; }

// MN-major operand [planes][L][rows][pitch] as the 5-D view {64, rows, pitch/64, L, planes}:
// one box {64, 64, 4, 1, 1} brings 64 rows of four 64-column chunks, chunk after chunk
// (the layout the UMMA descriptor walks with an 8 KB leading-dimension offset).
bool encode_chunked_map(CUtensorMap* map, const void* base, int rows, int L, int planes, int pitch,
                        int chunks = 4) {
  EncodeTiledFn enc = get_encoder();
  if (!enc || pitch % 64) return false;
  cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(pitch / 64),
                        static_cast<cuuint64_t>(L), static_cast<cuuint64_t>(planes)};
  const cuuint64_t row_bytes = static_cast<cuuint64_t>(pitch) * 2;
  cuuint64_t strides[4] = {row_bytes, 128, row_bytes * rows, row_bytes * rows * L};
  cuuint32_t box[5] = {64, 64, static_cast<cuuint32_t>(chunks), 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// One group as the kernels see it.
struct GroupPlan {
  const void* const* g;  // device pointers (G or X)
  float* const* m;       // null for orthogonalise-only
  void* const* w;        // W (step) or Out (orthogonalise)
  int batch, rows, cols, f32, planes;
  int m_rows, n_cols, transposed, pitch_n, pitch_m, nblk;
  long long x_mat, x_plane, a_mat, a_plane;  // elements
  size_t off_x[2], off_a, off_b;             // bytes into the workspace
  int mat_off, part_off;
};

}  // namespace

struct muon_ctx {
  int device = 0;
  int sm_count = 148;
  float coeffs[3 * MUON_MAX_ITERS];
  int k = 5;
  void* ws = nullptr;
  size_t ws_bytes = 0;
  // per-matrix arrays
  int cap_mats = 0;
  size_t cap_parts = 0;
  float* d_nu = nullptr;
  float* d_s1 = nullptr;
  float* d_s2 = nullptr;
  int* d_flags = nullptr;
  unsigned* d_counters = nullptr;
  float* d_partials = nullptr;
  // [0]: the last whole-matrix call's, cleared as one begins; [1]: what expert and block calls have reported
  // since muon_get_status last took it; [2]: what it took
  int* d_status = nullptr;
  unsigned* d_done = nullptr;  // [kMaxProblems][MUON_MAX_BATCH] phase-completion counters
  // MUON_OVERLAP=1: momentum passes of later groups and applies of earlier groups run on a side
  // stream beside the Newton-Schulz launches of other groups.  Off by default: on B200 the
  // co-running elementwise passes slow the GEMM by as much time as they hide (both draw on the
  // same L2 -> SM bandwidth), and one persistent launch for all groups has no gap between them.
  bool overlap = false;
  // MUON_TEST_DROP_SIGNAL=1 at creation: the next persistent Newton-Schulz launch drops one
  // completion signal (test of the bounded waits; used once, then cleared)
  bool drop_signal_once = false;
  cudaStream_t side = nullptr;
  cudaEvent_t ev_fork = nullptr, ev_join = nullptr;
  cudaEvent_t ev_k1[MUON_MAX_GROUPS] = {};
  cudaEvent_t ev_gemm[MUON_MAX_GROUPS] = {};
  bool per_phase = false;       // MUON_LAUNCH=phase: one launch per phase (same work; per-phase timing)
  int last_count = 0;
  cudaStream_t last_stream = nullptr;
  bool pending = false;
  bool captured = false;        // a call was captured into a CUDA graph: the buffers never move again
  // device staging for gradients that arrive from host memory
  void* d_stage = nullptr;
  size_t stage_bytes = 0;
  // scratch of the spectral passes (GEMV partials, norms, cap partials)
  void* d_aux = nullptr;
  size_t aux_bytes = 0;
  // results of the last call as muon_get_status / muon_get_norms report them: the per-matrix
  // arrays of the last run, or the gathered copies of a slab-pipelined host call
  const float* out_nu = nullptr;
  const int* out_flags = nullptr;
  float* d_nu_all = nullptr;
  int* d_flags_all = nullptr;
  int cap_all = 0;
  // per-block results of the block calls
  float* d_nu_blocks = nullptr;
  int* d_flags_blocks = nullptr;
  int cap_blocks = 0;
  std::vector<cudaEvent_t> copy_events;  // one per slab of a host call
  // per-launch timing
  bool profiling = false;
  std::vector<cudaEvent_t> events;  // pool, two per recorded launch
  std::vector<int> rec_kind;        // kind of recorded launch i (events 2i, 2i+1)
};

namespace {

// Record the start event of a profiled launch; returns the slot or -1.
int prof_begin(muon_ctx* c, int kind, cudaStream_t s) {
  if (!c->profiling) return -1;
  const size_t slot = c->rec_kind.size();
  while (c->events.size() < 2 * (slot + 1)) {
    cudaEvent_t e;
    if (cudaEventCreate(&e) != cudaSuccess) return -1;
    c->events.push_back(e);
  }
  c->rec_kind.push_back(kind);
  cudaEventRecord(c->events[2 * slot], s);
  return static_cast<int>(slot);
}

void prof_end(muon_ctx* c, int slot, cudaStream_t s) {
  if (slot >= 0) cudaEventRecord(c->events[2 * slot + 1], s);
}

struct DeviceGuard {
  int prev = -1;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (prev != dev) cudaSetDevice(dev);
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
  }
};

bool finite(float x) { return std::isfinite(x); }

muon_status check_hparams(const muon_hparams* hp) {
  if (!hp) return MUON_ERR_INVALID_ARG;
  if (!finite(hp->lr) || !finite(hp->beta) || !finite(hp->weight_decay) || !finite(hp->eps))
    return MUON_ERR_INVALID_ARG;
  if (hp->eps < 0.f) return MUON_ERR_INVALID_ARG;
  if (!finite(hp->grad_scale) || !(hp->grad_scale > 0.f)) return MUON_ERR_INVALID_ARG;
  if (hp->scale_mode < MUON_SCALE_SQRT_RATIO || hp->scale_mode > MUON_SCALE_RMS_MATCH)
    return MUON_ERR_INVALID_ARG;
  return MUON_OK;
}

muon_status check_group(const muon_group& g, bool need_m) {
  if (g.dtype != MUON_BF16 && g.dtype != MUON_F32) return MUON_ERR_DTYPE;
  if (g.batch < 1 || g.batch > MUON_MAX_BATCH) return MUON_ERR_INVALID_ARG;
  if (g.rows < 1 || g.cols < 1) return MUON_ERR_INVALID_ARG;
  if (g.rows > 32768 || g.cols > 32768 || std::min(g.rows, g.cols) > 8192)
    return MUON_ERR_UNSUPPORTED_SHAPE;
  if (!g.W || !g.G || (need_m && !g.M)) return MUON_ERR_INVALID_ARG;
  for (int l = 0; l < g.batch; ++l) {
    if (!g.W[l] || !g.G[l] || (need_m && !g.M[l])) return MUON_ERR_INVALID_ARG;
  }
  return MUON_OK;
}

float shape_scale(int rows, int cols, int mode) {
  switch (mode) {
    case MUON_SCALE_NONE: return 1.0f;
    case MUON_SCALE_RMS_MATCH: return 0.2f * std::sqrt(static_cast<float>(std::max(rows, cols)));
    default: return std::sqrt(std::max(1.0f, static_cast<float>(rows) / static_cast<float>(cols)));
  }
}

// Make sure the workspace and the per-matrix arrays can hold `plans`.
// Growing a context buffer synchronises the device and allocates; neither is allowed while the
// call's stream is being captured into a CUDA graph, and either would invalidate the capture.  A
// graph captured earlier keeps the buffers' addresses, so once a call has been captured the
// buffers never move again.  In both cases the call is refused before anything is queued (a
// capture in progress stays usable).  A stream whose capture state cannot be read counts as
// capturing: growth would fail on it too.
muon_status may_grow(muon_ctx* c, cudaStream_t s, const char* what) {
  if (capture_state(s) != 0)
    return refuse_growth(what, "the stream is capturing a CUDA graph: make the same call once before capture");
  if (c->captured)
    return refuse_growth(what, "a CUDA graph captured from this context holds its buffers: use another context");
  return MUON_OK;
}

// Called before any work of a call is queued on `s`: remembers that the context's buffers now
// sit in a captured graph.
void note_capture(muon_ctx* c, cudaStream_t s) {
  if (capture_state(s) == 1) c->captured = true;
}

muon_status reserve(muon_ctx* c, std::vector<GroupPlan>& plans, cudaStream_t s) {
  size_t bytes = 0;
  int mats = 0;
  size_t parts = 0;
  for (auto& p : plans) {
    const size_t xb = static_cast<size_t>(p.x_plane) * p.planes * 2;
    const size_t ab = static_cast<size_t>(p.a_plane) * p.planes * 2;
    p.off_x[0] = bytes; bytes = align_up(bytes + xb, 256);
    p.off_x[1] = bytes; bytes = align_up(bytes + xb, 256);
    p.off_a = bytes; bytes = align_up(bytes + ab, 256);
    p.off_b = bytes; bytes = align_up(bytes + ab, 256);
    p.mat_off = mats;
    mats += p.batch;
    p.part_off = static_cast<int>(parts);
    parts += static_cast<size_t>(p.batch) * p.nblk;
  }
  const bool grow_ws = bytes > c->ws_bytes;
  const bool grow_arrays = mats > c->cap_mats || parts > c->cap_parts;
  if (grow_ws || grow_arrays) {
    const muon_status st = may_grow(c, s, "the workspace");
    if (st != MUON_OK) return st;
  }
  note_capture(c, s);
  if (grow_ws) {
    MUON_CUDA(cudaDeviceSynchronize(), "sync before workspace growth");
    if (c->ws) cudaFree(c->ws);
    c->ws = nullptr;
    c->ws_bytes = 0;
    if (cudaMalloc(&c->ws, bytes) != cudaSuccess) {
      note_alloc_failure();
      return MUON_ERR_ALLOC;
    }
    c->ws_bytes = bytes;
  }
  if (grow_arrays) {
    MUON_CUDA(cudaDeviceSynchronize(), "sync before array growth");
    cudaFree(c->d_nu); cudaFree(c->d_s1); cudaFree(c->d_s2); cudaFree(c->d_flags);
    cudaFree(c->d_counters); cudaFree(c->d_partials);
    c->d_nu = c->d_s1 = c->d_s2 = c->d_partials = nullptr;
    c->d_flags = nullptr;
    c->d_counters = nullptr;
    const int cm = std::max(mats, c->cap_mats);
    const size_t cp = std::max(parts, c->cap_parts);
    bool ok = cudaMalloc(&c->d_nu, cm * sizeof(float)) == cudaSuccess &&
              cudaMalloc(&c->d_s1, cm * sizeof(float)) == cudaSuccess &&
              cudaMalloc(&c->d_s2, cm * sizeof(float)) == cudaSuccess &&
              cudaMalloc(&c->d_flags, cm * sizeof(int)) == cudaSuccess &&
              cudaMalloc(&c->d_counters, cm * sizeof(unsigned)) == cudaSuccess &&
              cudaMalloc(&c->d_partials, cp * sizeof(float)) == cudaSuccess;
    if (!ok) {
      note_alloc_failure();
      c->cap_mats = 0;
      c->cap_parts = 0;
      return MUON_ERR_ALLOC;
    }
    MUON_CUDA(cudaMemset(c->d_counters, 0, cm * sizeof(unsigned)), "clear counters");
    MUON_CUDA(cudaMemset(c->d_flags, 0, cm * sizeof(int)), "clear flags");
    c->cap_mats = cm;
    c->cap_parts = cp;
  }
  return MUON_OK;
}

GroupPlan plan_group(const muon_group& g) {
  GroupPlan p{};
  p.g = g.G;
  p.m = g.M;
  p.w = g.W;
  p.batch = g.batch;
  p.rows = g.rows;
  p.cols = g.cols;
  p.f32 = g.dtype == MUON_F32;
  p.planes = p.f32 ? 3 : 1;
  p.transposed = g.rows > g.cols;
  p.m_rows = std::min(g.rows, g.cols);
  p.n_cols = std::max(g.rows, g.cols);
  p.pitch_n = round64(p.n_cols);  // the chunked MN-major view never leaves a row
  p.pitch_m = round8(p.m_rows);
  p.nblk = momentum_blocks_per_matrix(g.rows, g.cols);
  p.x_mat = static_cast<long long>(p.m_rows) * p.pitch_n;
  p.x_plane = p.x_mat * p.batch;
  p.a_mat = static_cast<long long>(p.m_rows) * p.pitch_m;
  p.a_plane = p.a_mat * p.batch;
  return p;
}

uint16_t* ws_at(muon_ctx* c, size_t off) {
  return reinterpret_cast<uint16_t*>(static_cast<char*>(c->ws) + off);
}

enum Phase { PH_GRAM, PH_POLY, PH_UPDATE };

// Fill one GEMM problem for group p, phase ph of iteration `it`.
bool fill_problem(muon_ctx* c, const GroupPlan& p, Phase ph, int it, GemmProblem& q) {
  std::memset(static_cast<void*>(&q), 0, sizeof(q));
  const float a = c->coeffs[3 * it], b = c->coeffs[3 * it + 1], cc = c->coeffs[3 * it + 2];
  const int src = it & 1, dst = (it + 1) & 1;
  (void)dst;
  uint16_t* X = ws_at(c, p.off_x[src]);
  uint16_t* Xn = ws_at(c, p.off_x[dst]);
  uint16_t* A = ws_at(c, p.off_a);
  uint16_t* B = ws_at(c, p.off_b);
  const int m = p.m_rows, n = p.n_cols;
  q.L = p.batch;
  q.nseg = p.planes == 3 ? 6 : 1;
  q.planes = p.planes;
  const bool have_poly = cc != 0.f;
  const CUtensorMapSwizzle sw64 = CU_TENSOR_MAP_SWIZZLE_64B;
  // K-major B operand box height: the tile's N (256, or 128 for narrow tiles)
  const int kb_rows = 256;
  switch (ph) {
    case PH_GRAM:
      // A = s2 * X X^T; with c = 0 the polynomial is linear and the Gram
      // epilogue writes B' = b A + a I directly.
      if (!encode_map(&q.tmA, X, n, m, p.batch, p.planes, p.pitch_n, 64, 128)) return false;
      if (!encode_map(&q.tmB, X, n, m, p.batch, p.planes, p.pitch_n, 64, kb_rows)) return false;
      if (!encode_map(&q.tmB2, X, n, m, p.batch, p.planes, p.pitch_n, 64, kb_rows / 2)) return false;
      if (!encode_map(&q.tmOut, have_poly ? A : B, m, m, p.batch, p.planes, p.pitch_m, 32, 32, sw64))
        return false;
      q.M = m; q.N = m; q.K = n;
      q.b_mn_major = 0; q.sym = 1;
      q.alpha = have_poly ? 1.f : b;
      q.beta = 0.f;
      q.diag = have_poly ? 0.f : a;
      q.mat_scale = it == 0 ? c->d_s2 + p.mat_off : nullptr;
      break;
    case PH_POLY:
      // B' = c A A + b A + a I
      if (!encode_map(&q.tmA, A, m, m, p.batch, p.planes, p.pitch_m, 64, 128)) return false;
      if (!encode_map(&q.tmB, A, m, m, p.batch, p.planes, p.pitch_m, 64, kb_rows)) return false;
      if (!encode_map(&q.tmB2, A, m, m, p.batch, p.planes, p.pitch_m, 64, kb_rows / 2)) return false;
      if (!encode_map(&q.tmOut, B, m, m, p.batch, p.planes, p.pitch_m, 32, 32, sw64)) return false;
      q.M = m; q.N = m; q.K = m;
      q.b_mn_major = 0; q.sym = 1;
      q.alpha = cc; q.beta = b; q.diag = a;
      q.cin = A; q.cin_plane = p.a_plane; q.cin_mat = p.a_mat; q.cin_pitch = p.pitch_m;
      break;
    case PH_UPDATE: {
      // X' = s1 * B' X   (s1 = 1/(nu+eps) on the first iteration, X = U unnormalised)
      if (!encode_map(&q.tmA, B, m, m, p.batch, p.planes, p.pitch_m, 64, 128)) return false;
      // chunked MN-major view: 4 chunks of 64 columns per load
      if (!encode_chunked_map(&q.tmB, X, m, p.batch, p.planes, p.pitch_n, 4)) return false;
      q.M = m; q.N = n; q.K = m;
      q.b_mn_major = 1; q.sym = 0;
      q.alpha = 1.f; q.beta = 0.f; q.diag = 0.f;
      q.mat_scale = it == 0 ? c->d_s1 + p.mat_off : nullptr;
      if (!encode_map(&q.tmOut, Xn, n, m, p.batch, p.planes, p.pitch_n, 32, 32, sw64)) return false;
      break;
    }
  }
  q.tiles_per_matrix = gemm_tiles_per_matrix(q.M, q.N, q.sym);
  q.k_tiles = (q.K + 63) / 64;
  return true;
}

// Spectral cap of one group: per-matrix top singular vectors of the pre-step W
// (u: length rows, v: length cols) and where the coefficients go.
struct CapSpec {
  const float* const* u;
  const float* const* v;
  float* alpha;  // device [batch]
};

muon_status ensure_aux(muon_ctx* c, size_t bytes, cudaStream_t s) {
  if (bytes <= c->aux_bytes) {
    note_capture(c, s);
    return MUON_OK;
  }
  const muon_status st = may_grow(c, s, "the scratch");
  if (st != MUON_OK) return st;
  MUON_CUDA(cudaDeviceSynchronize(), "sync before scratch growth");
  cudaFree(c->d_aux);
  c->d_aux = nullptr;
  c->aux_bytes = 0;
  if (cudaMalloc(&c->d_aux, bytes) != cudaSuccess) {
    note_alloc_failure();
    return MUON_ERR_ALLOC;
  }
  c->aux_bytes = bytes;
  return MUON_OK;
}

muon_status run(muon_ctx* c, std::vector<GroupPlan>& plans, const muon_hparams* hp, bool step,
                float eps, cudaStream_t s, const CapSpec* cap = nullptr, bool clear_status = true) {
  muon_status st = reserve(c, plans, s);
  if (st != MUON_OK) return st;
  if (cap != nullptr) {  // per-block partials of the cap coefficients, sized before any launch
    st = ensure_aux(c, sizeof(double) * plans[0].batch * cap_alpha_blocks(plans[0].m_rows), s);
    if (st != MUON_OK) return st;
  }
  int total = 0;
  for (auto& p : plans) total += p.batch;
  if (clear_status) MUON_CUDA(cudaMemsetAsync(c->d_status, 0, sizeof(int), s), "clear status");

  // K1: momentum / look-ahead / norm over the groups `gs` (one launch per run of groups that share
  // a dtype and fit the launch's pointer tables).
  auto k1 = [&](const std::vector<int>& gs, cudaStream_t strm) -> muon_status {
    size_t i = 0;
    while (i < gs.size()) {
      MomentumParams mp;
      std::memset(static_cast<void*>(&mp), 0, sizeof(mp));
      mp.beta = step ? hp->beta : 0.f;
      mp.gscale = step ? hp->grad_scale : 1.f;
      mp.nesterov = step ? hp->nesterov : 0;
      mp.eps = eps;
      const int f32 = plans[gs[i]].f32;
      int mats = 0;
      for (; i < gs.size() && mp.ngroups < MUON_MAX_GROUPS; ++i) {
        const GroupPlan& p = plans[gs[i]];
        if (p.f32 != f32 || mats + p.batch > MUON_MAX_BATCH) break;
        MomentumGroup& q = mp.grp[mp.ngroups++];
        q.mat0 = mats;
        for (int l = 0; l < p.batch; ++l) {
          mp.g[mats + l] = p.g[l];
          mp.m[mats + l] = step ? p.m[l] : nullptr;
        }
        mats += p.batch;
        q.batch = p.batch;
        q.rows = p.rows;
        q.cols = p.cols;
        q.nblk = p.nblk;
        q.pitch = p.pitch_n;
        q.x = ws_at(c, p.off_x[0]);
        q.x_plane = p.x_plane;
        q.x_mat = p.x_mat;
        q.partials = c->d_partials + p.part_off;
        q.counters = c->d_counters + p.mat_off;
        q.nu = c->d_nu + p.mat_off;
        q.scale1 = c->d_s1 + p.mat_off;
        q.scale2 = c->d_s2 + p.mat_off;
        q.flags = c->d_flags + p.mat_off;
      }
      const int slot = prof_begin(c, MUON_KERNEL_MOMENTUM, strm);
      MUON_CUDA(launch_momentum(mp, f32 != 0, step, f32 ? 3 : 1, strm), "momentum kernel");
      prof_end(c, slot, strm);
    }
    return MUON_OK;
  };
  // Both elementwise launches take the groups last to first (and, inside each launch, the
  // matrices last to first): the momentum pass then writes last the U the Newton-Schulz launch
  // reads first (group 0, matrix 0), and the apply reads first the iterates that launch wrote
  // last, while they are still in L2.
  std::vector<int> all_groups;
  for (int g = static_cast<int>(plans.size()) - 1; g >= 0; --g) all_groups.push_back(g);
  // k Newton-Schulz iterations.  One persistent launch runs every phase of
  // every group (as many as fit in one parameter block), ordered phase by phase;
  // per-(phase, matrix) counters let a tile start as soon as the previous phase
  // of its own matrix has landed.  MUON_LAUNCH=phase runs one launch per phase.
  std::vector<Phase> seq_ph;
  std::vector<int> seq_it;
  for (int it = 0; it < c->k; ++it) {
    for (int ph = PH_GRAM; ph <= PH_UPDATE; ++ph) {
      if (ph == PH_POLY && c->coeffs[3 * it + 2] == 0.f) continue;
      seq_ph.push_back(static_cast<Phase>(ph));
      seq_it.push_back(it);
    }
  }
  const bool persistent = !c->per_phase;
  const int signals_per_tile = kEpilogueWarps;
  const int ng = static_cast<int>(plans.size());
  const int nph = static_cast<int>(seq_ph.size());
  // Launch order of (group, phase) problems.  Persistent launches go group by
  // group: one group's X stays (mostly) L2-resident across its phases, and the
  // next group starts while the last phases of the previous one drain.  (Each
  // phase keeps the matrix order of the previous one, so a matrix's next phase
  // is dispatched a whole phase after its previous one; reversing the order for
  // L2 reuse measured slower because of those dependency waits.)  The per-phase
  // mode runs one launch per phase covering every group.
  struct Item { int g, pi; };
  std::vector<std::vector<Item>> launches;
  // Pipelined schedule (two or more groups, persistent kernel): one launch per group on the
  // caller's stream; the momentum pass of group g+1 and the apply of group g run on the side
  // stream beside them.  Groups whose momentum pass is transposed (tall W, shared-memory
  // tiles that cannot sit beside a GEMM CTA) go first, so the passes that overlap are the
  // ones that fit.
  const bool pipelined = c->overlap && persistent && ng >= 2 && cap == nullptr && c->side != nullptr;
  std::vector<int> order;
  for (int g = 0; g < ng; ++g)
    if (plans[g].transposed) order.push_back(g);
  for (int g = 0; g < ng; ++g)
    if (!plans[g].transposed) order.push_back(g);
  if (pipelined) {
    for (int g : order) {
      std::vector<Item> cur;
      for (int pi = 0; pi < nph; ++pi) cur.push_back({g, pi});
      launches.push_back(cur);
    }
  } else if (persistent) {
    std::vector<Item> cur;
    for (int g = 0; g < ng; ++g) {
      for (int pi = 0; pi < nph; ++pi) {
        if (static_cast<int>(cur.size()) == kMaxProblems) {
          launches.push_back(cur);
          cur.clear();
        }
        cur.push_back({g, pi});
      }
    }
    if (!cur.empty()) launches.push_back(cur);
  } else {
    for (int pi = 0; pi < nph; ++pi) {
      std::vector<Item> cur;
      for (int g = 0; g < ng; ++g) cur.push_back({g, pi});
      launches.push_back(cur);
    }
  }
  GemmParams gp;
  auto run_launch = [&](const std::vector<Item>& items, cudaStream_t strm) -> muon_status {
    std::memset(static_cast<void*>(&gp), 0, sizeof(gp));
    gp.status = c->d_status;
    int tiles = 0;
    int last_of_group[MUON_MAX_GROUPS];
    for (int g = 0; g < ng; ++g) last_of_group[g] = -1;
    for (const Item& itm : items) {
      GemmProblem& q = gp.prob[gp.nprob];
      if (!fill_problem(c, plans[itm.g], seq_ph[itm.pi], seq_it[itm.pi], q))
        return cuda_fail(cudaErrorInvalidValue, "tensor map encoding");
      q.tile_base = tiles;
      tiles += q.tiles_per_matrix * q.L;
      if (persistent) {
        q.done_self = c->d_done + static_cast<size_t>(gp.nprob) * MUON_MAX_BATCH;
        const int prev = last_of_group[itm.g];
        if (prev >= 0) {  // the previous phase of this group is in the same launch
          q.done_dep = gp.prob[prev].done_self;
          q.dep_target = static_cast<unsigned>(signals_per_tile * gp.prob[prev].tiles_per_matrix);
        }
        last_of_group[itm.g] = gp.nprob;
      }
      ++gp.nprob;
    }
    gp.total_tiles = tiles;
    if (persistent && c->drop_signal_once && gp.nprob > 1) {
      gp.drop_signal = 1;
      c->drop_signal_once = false;
    }
    if (persistent)
      MUON_CUDA(cudaMemsetAsync(c->d_done, 0, sizeof(unsigned) * gp.nprob * MUON_MAX_BATCH, strm), "clear counters");
    const int units = std::min(tiles, c->sm_count);
    const int kind = items.size() > static_cast<size_t>(ng) || persistent
                         ? MUON_KERNEL_NS_FUSED
                         : MUON_KERNEL_GRAM + (seq_ph[items[0].pi] - PH_GRAM);
    const int slot = prof_begin(c, kind, strm);
    MUON_CUDA(launch_gemm(gp, units, strm), "newton-schulz gemm");
    prof_end(c, slot, strm);
    return MUON_OK;
  };

  // K5: scale + decoupled decay applied to W (or the plain copy to Out) over the groups `gs`.
  auto k5 = [&](const std::vector<int>& gs, cudaStream_t strm) -> muon_status {
    size_t i = 0;
    while (i < gs.size()) {
      ApplyParams ap;
      std::memset(static_cast<void*>(&ap), 0, sizeof(ap));
      const int f32 = plans[gs[i]].f32;
      ap.planes = plans[gs[i]].planes;
      ap.apply = step ? 1 : 0;
      ap.decay = step ? 1.0f - hp->lr * hp->weight_decay : 1.0f;
      ap.status = c->d_status;
      int mats = 0;
      for (; i < gs.size() && ap.ngroups < MUON_MAX_GROUPS; ++i) {
        const GroupPlan& p = plans[gs[i]];
        if (p.f32 != f32 || mats + p.batch > MUON_MAX_BATCH) break;
        ApplyGroup& q = ap.grp[ap.ngroups++];
        q.mat0 = mats;
        for (int l = 0; l < p.batch; ++l) {
          ap.w[mats + l] = p.w[l];
          if (cap != nullptr) {
            ap.cu[mats + l] = cap->u[l];
            ap.cv[mats + l] = cap->v[l];
          }
        }
        mats += p.batch;
        q.batch = p.batch;
        q.rows = p.rows;
        q.cols = p.cols;
        q.nblk = momentum_blocks_per_matrix(p.rows, p.cols);
        q.o = ws_at(c, p.off_x[c->k & 1]);
        q.o_plane = p.x_plane;
        q.o_mat = p.x_mat;
        q.pitch = p.pitch_n;
        q.lrs = step ? hp->lr * shape_scale(p.rows, p.cols, hp->scale_mode) : 0.f;
        q.flags = step ? c->d_flags + p.mat_off : nullptr;
        q.alpha = cap != nullptr ? cap->alpha : nullptr;
      }
      const int slot = prof_begin(c, MUON_KERNEL_APPLY, strm);
      MUON_CUDA(launch_apply(ap, f32 != 0, strm), "apply kernel");
      prof_end(c, slot, strm);
    }
    return MUON_OK;
  };

  if (pipelined) {
    // caller's stream: K1(first), GEMM(first), GEMM(second) ..., K5(last)
    // side stream:     K1(second) ..., K5(first) ...
    st = k1({order[0]}, s);
    if (st != MUON_OK) return st;
    MUON_CUDA(cudaEventRecord(c->ev_fork, s), "fork");
    MUON_CUDA(cudaStreamWaitEvent(c->side, c->ev_fork, 0), "fork");
    for (int i = 1; i < ng; ++i) {
      st = k1({order[i]}, c->side);
      if (st != MUON_OK) return st;
      MUON_CUDA(cudaEventRecord(c->ev_k1[i], c->side), "momentum done");
    }
    for (int i = 0; i < ng; ++i) {
      if (i > 0) MUON_CUDA(cudaStreamWaitEvent(s, c->ev_k1[i], 0), "wait momentum");
      st = run_launch(launches[i], s);
      if (st != MUON_OK) return st;
      if (i + 1 < ng) {
        MUON_CUDA(cudaEventRecord(c->ev_gemm[i], s), "gemm done");
        MUON_CUDA(cudaStreamWaitEvent(c->side, c->ev_gemm[i], 0), "wait gemm");
        st = k5({order[i]}, c->side);
        if (st != MUON_OK) return st;
      }
    }
    st = k5({order[ng - 1]}, s);
    if (st != MUON_OK) return st;
    MUON_CUDA(cudaEventRecord(c->ev_join, c->side), "join");
    MUON_CUDA(cudaStreamWaitEvent(s, c->ev_join, 0), "join");
  } else {
    st = k1(all_groups, s);
    if (st != MUON_OK) return st;
    for (const auto& items : launches) {
      st = run_launch(items, s);
      if (st != MUON_OK) return st;
    }
    // Spectral cap: alpha_l = u_l^T O_l v_l from the final iterate (one group).
    if (cap != nullptr) {
      const GroupPlan& p = plans[0];
      CapParams cp;
      std::memset(static_cast<void*>(&cp), 0, sizeof(cp));
      for (int l = 0; l < p.batch; ++l) {
        cp.a[l] = p.transposed ? cap->v[l] : cap->u[l];  // wide rows are W's columns when tall
        cp.b[l] = p.transposed ? cap->u[l] : cap->v[l];
      }
      cp.o = ws_at(c, p.off_x[c->k & 1]);
      cp.o_plane = p.x_plane;
      cp.o_mat = p.x_mat;
      cp.pitch = p.pitch_n;
      cp.m = p.m_rows;
      cp.n = p.n_cols;
      cp.planes = p.planes;
      cp.partial = static_cast<double*>(c->d_aux);
      MUON_CUDA(launch_cap_alpha(cp, p.batch, cap->alpha, s), "cap coefficient");
    }
    st = k5(all_groups, s);
    if (st != MUON_OK) return st;
  }
  c->last_count = total;
  c->last_stream = s;
  c->pending = true;
  c->out_nu = c->d_nu;
  c->out_flags = c->d_flags;
  return MUON_OK;
}

// Expert and block calls add to a status word of their own, which nothing but muon_get_status clears (a
// memset a call would cost as much as their smallest kernels, and captured it would wipe what earlier
// replays reported).
int* collected_status(const muon_ctx* c) { return c->d_status + 1; }

__global__ void take_status_kernel(int* word, int* taken) { *taken = atomicExch(word, 0); }

// The last call's status and flags and, with `take`, what expert and block calls have reported since this was
// last asked.
muon_status last_status(muon_ctx* c, int* flags, int capacity, int* count, bool take) {
  DeviceGuard guard(c->device);
  if (count) *count = c->last_count;
  if (!c->pending) return MUON_OK;
  MUON_CUDA(cudaStreamSynchronize(c->last_stream), "stream synchronize");
  int word[2] = {0, 0};
  MUON_CUDA(cudaMemcpy(word, c->d_status, sizeof(word), cudaMemcpyDeviceToHost), "read status");
  if (!take) word[1] = 0;
  if (word[1] != 0) {  // taken in one exchange: what another stream adds meanwhile is kept for the next report
    take_status_kernel<<<1, 1, 0, c->last_stream>>>(collected_status(c), c->d_status + 2);
    MUON_CUDA(cudaGetLastError(), "take status");
    MUON_CUDA(cudaMemcpyAsync(&word[1], c->d_status + 2, sizeof(int), cudaMemcpyDeviceToHost, c->last_stream), "read status");
    MUON_CUDA(cudaStreamSynchronize(c->last_stream), "stream synchronize");
  }
  const int status = word[0] | word[1];
  std::vector<int> f(c->last_count);
  if (c->last_count > 0)
    MUON_CUDA(cudaMemcpy(f.data(), c->out_flags, sizeof(int) * c->last_count, cudaMemcpyDeviceToHost),
              "read flags");
  if (flags) std::memcpy(flags, f.data(), sizeof(int) * std::min(capacity, c->last_count));
  if (status & kStatusTimeout) return MUON_ERR_TIMEOUT;
  if (status & kStatusBadSegments) return MUON_ERR_INVALID_ARG;
  if (status & kStatusNonfinite) return MUON_ERR_NONFINITE;
  for (int v : f)
    if (v & MUON_FLAG_NONFINITE) return MUON_ERR_NONFINITE;
  return MUON_OK;
}

// ------------------------------------------------------------------ experts
// A token matrix or weight stack as the tensor maps see it: `planes` bf16 planes of `mats` matrices.
struct Operand {
  const void* base;
  int mats, rows, cols, planes;
  long long ld, s, plane;  // elements
};

// The caller's matrices when a TMA can read them in place, else their packed copy at `scratch`
// (null while sizes are only counted); *bytes grows by what the copy takes.
bool in_place(const Operand& o, int dtype) {
  return dtype == MUON_BF16 && reinterpret_cast<uintptr_t>(o.base) % 16 == 0 && (o.rows <= 1 || o.ld % 8 == 0) &&
         (o.mats <= 1 || (o.s % 8 == 0 && o.s > 0));
}

Operand packed(const Operand& o, int dtype) {
  Operand q = o;
  q.planes = dtype == MUON_F32 ? 3 : 1;
  q.ld = round8(o.cols);
  q.s = q.ld * o.rows;
  q.plane = q.s * o.mats;
  q.base = nullptr;
  return q;
}

size_t operand_bytes(const Operand& q) { return align_up(static_cast<size_t>(q.plane) * q.planes * 2, 256); }

// 4-D map {cols, rows, mats, planes}, box {box_cols, box_rows, 1, 1}, 128-byte swizzle.
bool encode_operand(CUtensorMap* map, const Operand& o, int box_cols, int box_rows) {
  EncodeTiledFn enc = get_encoder();
  if (!enc) return false;
  auto dim = [](long long v) { return static_cast<cuuint64_t>(std::max(v, 1ll)); };
  cuuint64_t dims[4] = {dim(o.cols), dim(o.rows), dim(o.mats), dim(o.planes)};
  // the stride of a one-element dimension is never used but still checked: any multiple of 16 bytes
  const long long ld = o.rows > 1 ? o.ld : round8(o.cols), sm = o.mats > 1 ? o.s : ld * std::max(o.rows, 1),
                  sp = o.planes > 1 ? o.plane : sm * o.mats;
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(sm) * 2,
                           static_cast<cuuint64_t>(sp) * 2};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(o.base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// fp32 output [mats][rows][cols] as {cols, rows, mats}, box {32, 16, 1}.
bool encode_out_f32(CUtensorMap* map, void* base, int cols, int rows, int mats, long long ld, long long s) {
  EncodeTiledFn enc = get_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(mats)};
  const long long row = rows > 1 ? ld : (cols + 3) / 4 * 4;
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(row) * 4, static_cast<cuuint64_t>(mats > 1 ? s : row * rows) * 4};
  cuuint32_t box[3] = {32, 16, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

muon_status check_experts(const muon_ctx* c, const muon_experts* ex) {
  if (!c || !ex || !ex->offsets) return MUON_ERR_INVALID_ARG;
  if (ex->dtype != MUON_BF16 && ex->dtype != MUON_F32) return MUON_ERR_DTYPE;
  if (ex->experts < 1 || ex->experts > MUON_MAX_EXPERTS || ex->tokens < 0 || ex->rows < 1 || ex->cols < 1)
    return MUON_ERR_INVALID_ARG;
  if (ex->tokens > (1 << 30) || ex->rows > 32768 || ex->cols > 32768) return MUON_ERR_UNSUPPORTED_SHAPE;
  return MUON_OK;
}

// A matrix of `rows` rows of `cols` elements with row stride ld.
bool rows_ok(const void* p, long long ld, int rows, int cols) {
  if (rows == 0) return true;
  return p != nullptr && (rows == 1 || ld >= cols);
}

// A stack whose elements may not overlap (an output), or may not alias within a matrix (an input).
bool stack_ok(const void* p, long long ld, long long s, int mats, int rows, int cols, bool output) {
  if (p == nullptr || (rows > 1 && ld < cols) || (mats > 1 && s < (output ? cols : 1))) return false;
  if (!output || rows == 1 || mats == 1) return true;
  return s >= ld ? s >= ld * (rows - 1) + cols : ld >= s * (mats - 1) + cols;
}

// Whether two CTAs share each tile (256 features).  A pair loads a third less per product but starts
// slower and rounds features up to 256.  Measured with 16 experts (us, single -> pair); where the two cross
// depends on how tiles fill the last round, and the limits lie between the crossings:
//   bf16 products, millions of outputs: 2048 x 2048 weights 4.2: 31.5 -> 33.6, 5.2: 35.4 -> 34.3, 6.0: 36.1 -> 34.5,
//     8.4: 40 -> 37.8; 1536 x 768 4.7: 18.2 -> 18.9, 5.9: 19.1 -> 19.2, 7.9: 21.8 -> 22.5, 12.6: 24.9 -> 23.6, with
//     8 experts 6.1: 15.9 -> 17.2, 9.4: 17.4 -> 17.9; their input gradients 3.1: 17.5 -> 17.4, 4.7: 20 -> 23.5, 5.9:
//     24.9 -> 24.2, 7.9: 28.3 -> 25.7.  640 columns, a sixth of the pairs' features idle: 27.5 -> 28.9.
//   bf16 gradients, tokens an expert: 1536 x 768 384: 40.1 -> 41.6, 448: 42.0 -> 40.7, 496: 45.0 -> 41.7, 768: 51 -> 48;
//     2048 x 2048, 8 experts 384: 64.6 -> 66.5, 512: 71 -> 65.
//   fp32 loads three planes of everything, so pairs pay earlier.  Products, millions of outputs: 640 x 768 0.66:
//     33.5 -> 35.2, 0.98: 43.7 -> 37.4, 1.3: 46.7 -> 39.8, 1.6: 46.8 -> 48.5; 1536 x 768 1.2: 70.4 -> 72.4, 1.6: 71.5 ->
//     73.3, 2.4: 81.4 -> 75.4.  Gradients: 16 tokens 3.1: 17.4 -> 17.6, 3.9: 19.3 -> 18.2, 4.7: 19.8 -> 18.2, 6.3: 24 ->
//     20.8; 128 tokens 3.1: 20.4 -> 20.0, 4.3: 24 -> 20.7.
bool expert_pair(ExpertMode mode, bool f32, long long features, long long rows, long long tokens, long long experts) {
  const long long out = features * (mode == EXPERT_WGRAD ? rows * experts : tokens);  // output elements
  if (f32) return features > 128 && out >= (mode == EXPERT_WGRAD ? 4500000 : 1250000);
  const long long idle = (features + 255) / 256 * 256 - features;
  return 16 * idle <= features && out >= 6000000 && (mode != EXPERT_WGRAD || tokens >= 500 * experts);
}

// Whether fp32 operands are split by the product kernel itself or packed into planes before it.  Packing
// reads 4 and writes 6 bytes of each weight before 6 are loaded, for every tile that loads them; the
// kernel's own split reads 4, but anew for each tile, whose rows are at most 64.  Measured (us, packed ->
// split), products with 16 experts of 1536 x 768: 8 tokens an expert 69.5 -> 43.2, 64 tokens 73.2 -> 47.2, 80
// tokens 74.8 -> 63.7, 128 tokens 78.8 -> 68.4 (79.4 -> 85.8 where the router is uneven); input gradients 64 tokens
// 71.9 -> 47.7, 80 tokens 88.6 -> 80.7, 128 tokens 80.8 -> 87.8; 64 experts, 24 tokens in all 94.2 -> 42.0.
// Gradients pack only tokens, and have more tiles the narrower they are: they split where the packing
// launch is what costs (16 experts, 8 tokens each, millions of elements 3.1: 18.7 -> 16.3, 3.9: 21.4 -> 19.1, 4.1:
// 22.1 -> 20.5, 4.7: 19.4 -> 20.5, 5.5: 21.8 -> 24.5, 9.4: 25.7 -> 37.0; 48 tokens each 3.9: 21.3 -> 20.1, 4.7:
// 19.1 -> 21.6).
bool expert_split(ExpertMode mode, long long outputs, long long tokens, long long experts) {
  return tokens <= 64 * experts && (mode != EXPERT_WGRAD || outputs <= 4000000);
}

// Packs what a TMA cannot read in place, encodes the maps and queues one product launch.
muon_status run_experts(muon_ctx* c, const muon_experts* ex, ExpertMode mode, Operand a, Operand b, ExpertParams& p,
                        cudaStream_t s) {
  const bool f32 = ex->dtype == MUON_F32;
  const long long outputs = static_cast<long long>(p.features) * p.rows * ex->experts;  // of a gradient
  const bool split = f32 && expert_split(mode, outputs, ex->tokens, ex->experts);
  const bool pa = !split && !in_place(a, ex->dtype), pb = !split && !in_place(b, ex->dtype);
  // both operands have the same number of planes: fp32 packs both or neither
  const Operand qa = pa ? packed(a, ex->dtype) : a, qb = pb ? packed(b, ex->dtype) : b;
  const size_t need = (pa ? operand_bytes(qa) : 0) + (pb ? operand_bytes(qb) : 0);
  muon_status st = ensure_aux(c, need, s);
  if (st != MUON_OK) return st;
  char* at = static_cast<char*>(c->d_aux);
  PackParams packs;
  packs.count = 0;
  auto pack = [&](Operand& o, const Operand& q) {
    if (o.rows > 0)
      packs.item[packs.count++] = PackItem{o.base, reinterpret_cast<uint16_t*>(at), o.ld, o.s, q.s, q.plane, o.mats,
                                           o.rows, o.cols, static_cast<int>(q.ld),
                                           o.mats > 1 ? ex->offsets : nullptr, 0};
    o = q;
    o.base = at;
    at += operand_bytes(q);
  };
  if (pa) pack(a, qa);
  if (pb) pack(b, qb);
  if (packs.count > 0) MUON_CUDA(launch_pack(packs, ex->dtype == MUON_F32, c->sm_count, s), "pack kernel");
  bool ok = true;
  if (split) {
    auto pairs = [](const Operand& o) {
      return reinterpret_cast<uintptr_t>(o.base) % 8 == 0 && o.cols % 2 == 0 && (o.rows <= 1 || o.ld % 2 == 0) &&
             (o.mats <= 1 || o.s % 2 == 0);
    };
    p.a = a.base;
    p.b = b.base;
    p.ld_a = a.ld;
    p.s_a = a.s;
    p.ld_b = b.ld;
    p.pairs_a = pairs(a);
    p.pairs_b = pairs(b);
    p.contraction = mode == EXPERT_FORWARD ? a.cols : a.rows;
  } else {
    // nothing is loaded of a matrix without rows, but its map still needs an address
    if (a.rows == 0) a.base = c->d_status;
    if (b.rows == 0) b.base = c->d_status;
    ok = encode_operand(&p.tmA, a, 64, mode == EXPERT_FORWARD ? 128 : 64);
    for (int i = 0; ok && i < kExpertBoxes; ++i)
      ok = encode_operand(&p.tmB[i], b, 64, mode == EXPERT_WGRAD ? 64 : 16 << i);
  }
  if (ok && p.out_f32 && p.vec)
    ok = mode == EXPERT_WGRAD ? encode_out_f32(&p.tmOut, p.out, p.features, p.rows, ex->experts, p.ld_out, p.s_out)
                              : encode_out_f32(&p.tmOut, p.out, p.features, ex->tokens, 1, p.ld_out, 0);
  if (!ok) return cuda_fail(cudaErrorInvalidValue, "tensor map encoding");
  p.offsets = ex->offsets;
  p.experts = ex->experts;
  p.tokens = ex->tokens;
  p.in_f32 = f32;
  p.split = split;
  p.status = collected_status(c);
  const bool pair = !split && expert_pair(mode, f32, p.features, p.rows, ex->tokens, ex->experts);
  const int fm = pair ? 256 : 128;
  const long long nf = (p.features + fm - 1) / fm;
  // more CTAs than the narrowest tiles can number would idle
  const long long most = (pair ? 2 : 1) * nf *
                         (mode == EXPERT_WGRAD ? static_cast<long long>((p.rows + 31) / 32) * ex->experts
                                               : ex->tokens / 32 + std::min(ex->tokens, ex->experts));
  const int sms = pair ? c->sm_count & ~1 : c->sm_count;
  const int ctas = static_cast<int>(std::max(pair ? 2ll : 1ll, std::min<long long>(most, sms)));
  MUON_CUDA(launch_experts(p, mode, pair, ctas, s), "expert product");
  c->last_count = 0;
  c->last_stream = s;
  c->pending = true;
  return MUON_OK;
}

// ------------------------------------------------------------------ blocks
// Largest value an iteration of the coefficient table can reach from singular values of at most 1:
// of X, of A = X X^T, and of b A + c A A with and without a I, each bounded by its spectral norm.
double table_bound(const float* abc, int k) {
  double r = 1.0, most = 1.0;
  for (int i = 0; i < k; ++i) {
    const double a = abc[3 * i], b = abc[3 * i + 1], c = abc[3 * i + 2];
    auto poly = [&](double t) { return std::fabs(a + b * t + c * t * t); };  // of t = sigma^2
    auto rest = [&](double t) { return std::fabs(b * t + c * t * t); };
    double pmax = std::max({poly(0.0), poly(r * r), rest(r * r)}), next = r * poly(r * r);
    if (c != 0.0) {
      const double t = -b / (2.0 * c);
      if (t > 0.0 && t < r * r) pmax = std::max({pmax, poly(t), rest(t)});
    }
    // extrema of sigma poly(sigma^2): a + 3 b t + 5 c t^2 = 0
    auto extremum = [&](double t) {
      if (t > 0.0 && t < r * r) next = std::max(next, std::sqrt(t) * poly(t));
    };
    if (c != 0.0) {
      const double d = 9.0 * b * b - 20.0 * a * c;
      if (d >= 0.0) {
        extremum((-3.0 * b + std::sqrt(d)) / (10.0 * c));
        extremum((-3.0 * b - std::sqrt(d)) / (10.0 * c));
      }
    } else if (b != 0.0) {
      extremum(-a / (3.0 * b));
    }
    most = std::max({most, r * r, pmax, next});
    r = 1.01 * next;  // the products' own rounding
    if (!(most < 1e30)) return 1e30;
  }
  return most;
}

constexpr size_t kBlockMostSmem = 226 * 1024;

// How matrices of rows x cols are cut: sizes, grid, the cluster that holds a block and the shared memory each
// of its CTAs needs.
muon_status plan_blocks(int rows, int cols, int block_rows, int block_cols, int dtype, BlockParams& p, size_t* smem) {
  if (dtype != MUON_BF16 && dtype != MUON_F32) return MUON_ERR_DTYPE;
  if (rows < 1 || cols < 1 || block_rows < 1 || block_cols < 1) return MUON_ERR_INVALID_ARG;
  if (rows > 32768 || cols > 32768) return MUON_ERR_UNSUPPORTED_SHAPE;
  p.block_rows = std::min(block_rows, rows);
  p.block_cols = std::min(block_cols, cols);
  p.rows = rows;
  p.cols = cols;
  p.grid_cols = (cols + p.block_cols - 1) / p.block_cols;
  p.per_matrix = p.grid_cols * ((rows + p.block_rows - 1) / p.block_rows);
  const int m = std::min(p.block_rows, p.block_cols), n = std::max(p.block_rows, p.block_cols);
  if (m > kBlockMaxShort || p.per_matrix > kBlockMost) return MUON_ERR_UNSUPPORTED_SHAPE;
  // Clusters: the fewest CTAs whose shared memory holds the block (blocks of 2048 x 128 in bf16: four CTAs
  // 1767 us, five 2330, eight 3130: an SM holds one CTA of a cluster, and the exchange of the Gram partials
  // does not shrink).  Where eight do not, the exchange takes the place of A, at two barriers more each (with
  // them three CTAs hold that block too, in 1870 us).
  for (int i = 1; i <= kBlockMaxCluster + 1; ++i) {
    p.cluster = std::min(i, kBlockMaxCluster);
    p.slice = round64((n + p.cluster - 1) / p.cluster);
    p.alias = i > kBlockMaxCluster;
    *smem = block_smem_bytes(m, p.slice, p.block_rows > p.block_cols, dtype == MUON_F32, p.cluster, p.alias);
    if (*smem <= kBlockMostSmem) return MUON_OK;
  }
  return MUON_ERR_UNSUPPORTED_SHAPE;
}

muon_status run_blocks(muon_ctx* c, const muon_blocks* bl, const muon_hparams* hp, bool step, float eps,
                       cudaStream_t s) {
  if (!c || !bl || !bl->W || !bl->G || (step && !bl->M)) return MUON_ERR_INVALID_ARG;
  if (bl->batch < 1 || bl->batch > MUON_MAX_BATCH) return MUON_ERR_INVALID_ARG;
  BlockParams p;
  std::memset(static_cast<void*>(&p), 0, sizeof(p));
  size_t smem = 0;
  const muon_status planned = plan_blocks(bl->rows, bl->cols, bl->block_rows, bl->block_cols, bl->dtype, p, &smem);
  if (planned != MUON_OK) return planned;
  if (bl->rows > 1 && (bl->ldw < bl->cols || bl->ldg < bl->cols || (step && bl->ldm < bl->cols)))
    return MUON_ERR_INVALID_ARG;
  const bool f32 = bl->dtype == MUON_F32, tall = p.block_rows > p.block_cols;
  p.ldw = bl->ldw;
  p.ldg = bl->ldg;
  p.ldm = bl->ldm;
  const long long total = static_cast<long long>(p.per_matrix) * bl->batch;
  if (total > kBlockMost) return MUON_ERR_UNSUPPORTED_SHAPE;
  // TMEM is shared by the SM's CTAs: never more than 512 columns between those of this library that fit
  // beside one another (of any launch: two calls may run at once), so that no CTA waits for columns
  // while its cluster waits for it.  Every kernel with TMEM takes at least 77 KB, those with all of it
  // more than the rest of the SM then leaves.
  // A CTA that has its SM alone takes 512 threads (192 blocks of 128 x 768: 241 us, 269 with 256; of 64 x 1024: 162
  // and 175) and asks L2 for the block that follows while it multiplies (768 blocks of 2048 x 128: 1769 us, 1838
  // without); where two share an SM, one loads while the other multiplies, more threads cost 186 instead of
  // 153 us and the request changes nothing (148.2 and 148.5).
  constexpr size_t kTwoPerSm = (228 * 1024) / 2 - 1024, kNoThird = 77 * 1024, kAlone = 152 * 1024;
  const bool alone = smem > kTwoPerSm || p.cluster > 1;
  p.tmem_cols = alone ? 512 : 256;
  p.threads = alone ? 512 : 256;
  p.blocks = static_cast<int>(total);
  p.ahead = alone ? c->sm_count / p.cluster : 0;
  smem = std::max(smem, alone ? kAlone : kNoThird);
  const size_t eb = f32 ? 4 : 2;
  const bool grid_aligned = p.grid_cols == 1 || p.block_cols % 8 == 0;
  // eight elements an access: 16 bytes of bf16, 32 of fp32
  auto row_aligned = [&](long long ld) { return bl->rows == 1 || ld % 8 == 0; };
  p.vec = grid_aligned && row_aligned(bl->ldw) && row_aligned(bl->ldg) && (!step || row_aligned(bl->ldm));
  for (int l = 0; l < bl->batch; ++l) {
    if (!bl->W[l] || !bl->G[l] || (step && !bl->M[l])) return MUON_ERR_INVALID_ARG;
    p.w[l] = bl->W[l];
    p.g[l] = bl->G[l];
    p.m[l] = step ? bl->M[l] : nullptr;
    const uintptr_t wg = reinterpret_cast<uintptr_t>(p.w[l]) | reinterpret_cast<uintptr_t>(p.g[l]);
    if (wg % (8 * eb) || reinterpret_cast<uintptr_t>(p.m[l]) % 32) p.vec = 0;
  }
  // What is written may be given once, or a matrix would be stepped twice at the same time; what is read may not be
  // written by another block at that time: G may be its own W, lying the same way, and no other W nor any M.
  const void* written[2 * MUON_MAX_BATCH];
  const void** end = std::copy(p.w, p.w + bl->batch, written);
  if (step) end = std::copy(p.m, p.m + bl->batch, end);
  std::sort(written, end);
  if (std::adjacent_find(written, end) != end) return MUON_ERR_INVALID_ARG;
  for (int l = 0; l < bl->batch; ++l)
    if (p.g[l] == p.w[l] ? bl->rows > 1 && bl->ldg != bl->ldw : std::binary_search(written, end, p.g[l]))
      return MUON_ERR_INVALID_ARG;
  const double bound = table_bound(c->coeffs, c->k);
  if (!(bound < 32768.0)) return MUON_ERR_INVALID_ARG;
  p.store_scale = static_cast<float>(std::ldexp(1.0, std::min(12, static_cast<int>(std::floor(std::log2(32768.0 / bound))))));
  p.step = step;
  p.beta = step ? hp->beta : 0.f;
  p.gscale = step ? hp->grad_scale : 1.f;
  p.eps = eps;
  p.decay = step ? 1.0f - hp->lr * hp->weight_decay : 1.0f;
  p.lr = step ? hp->lr : 0.f;
  p.nesterov = step ? hp->nesterov : 0;
  p.scale_mode = step ? hp->scale_mode : MUON_SCALE_NONE;
  p.k = c->k;
  std::memcpy(p.abc, c->coeffs, sizeof(float) * 3 * c->k);
  p.status = collected_status(c);
  if (total > c->cap_blocks) {
    const muon_status st = may_grow(c, s, "the per-block results");
    if (st != MUON_OK) return st;
    MUON_CUDA(cudaDeviceSynchronize(), "sync before result growth");
    cudaFree(c->d_nu_blocks);
    cudaFree(c->d_flags_blocks);
    c->d_nu_blocks = nullptr;
    c->d_flags_blocks = nullptr;
    c->cap_blocks = 0;
    if (cudaMalloc(&c->d_nu_blocks, sizeof(float) * total) != cudaSuccess ||
        cudaMalloc(&c->d_flags_blocks, sizeof(int) * total) != cudaSuccess) {
      note_alloc_failure();
      return MUON_ERR_ALLOC;
    }
    c->cap_blocks = static_cast<int>(total);
  }
  note_capture(c, s);
  p.nu = c->d_nu_blocks;
  p.flags = c->d_flags_blocks;
  MUON_CUDA(launch_blocks(p, static_cast<int>(total), tall, f32, smem, s), "block step");
  c->last_count = static_cast<int>(total);
  c->last_stream = s;
  c->pending = true;
  c->out_nu = c->d_nu_blocks;
  c->out_flags = c->d_flags_blocks;
  return MUON_OK;
}

muon_status validate_and_plan(muon_ctx* c, const muon_group* groups, int ngroups, bool step,
                              std::vector<GroupPlan>& plans) {
  if (!c || !groups || ngroups < 1 || ngroups > MUON_MAX_GROUPS) return MUON_ERR_INVALID_ARG;
  plans.clear();
  for (int i = 0; i < ngroups; ++i) {
    muon_status st = check_group(groups[i], step);
    if (st != MUON_OK) return st;
    plans.push_back(plan_group(groups[i]));
  }
  return MUON_OK;
}

}  // namespace

// ====================================================================== C ABI
extern "C" {

int muon_abi_version(void) { return MUON_ABI_VERSION; }

const char* muon_status_string(muon_status s) {
  switch (s) {
    case MUON_OK: return "MUON_OK";
    case MUON_ERR_INVALID_ARG: return "MUON_ERR_INVALID_ARG";
    case MUON_ERR_UNSUPPORTED_SHAPE: return "MUON_ERR_UNSUPPORTED_SHAPE";
    case MUON_ERR_DTYPE: return "MUON_ERR_DTYPE";
    case MUON_ERR_CUDA: return "MUON_ERR_CUDA";
    case MUON_ERR_NONFINITE: return "MUON_ERR_NONFINITE";
    case MUON_ERR_TIMEOUT: return "MUON_ERR_TIMEOUT";
    case MUON_ERR_NO_DEVICE: return "MUON_ERR_NO_DEVICE";
    case MUON_ERR_ALLOC: return "MUON_ERR_ALLOC";
  }
  return "MUON_ERR_UNKNOWN";
}

const char* muon_last_cuda_error(void) { return g_cuda_error; }

muon_status muon_create(muon_ctx** out, int device) {
  if (!out) return MUON_ERR_INVALID_ARG;
  *out = nullptr;
  int n = 0;
  if (cudaGetDeviceCount(&n) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return MUON_ERR_NO_DEVICE;
  }
  if (device < 0 || device >= n) return MUON_ERR_INVALID_ARG;
  cudaDeviceProp prop;
  MUON_CUDA(cudaGetDeviceProperties(&prop, device), "device properties");
  if (prop.major != 10) return MUON_ERR_NO_DEVICE;
  if (!get_encoder()) return MUON_ERR_NO_DEVICE;
  DeviceGuard guard(device);
  muon_ctx* c = new muon_ctx();
  c->device = device;
  c->sm_count = prop.multiProcessorCount;
  for (int i = 0; i < 5; ++i) std::memcpy(&c->coeffs[3 * i], kQuintic, sizeof(kQuintic));
  c->k = 5;

  if (const char* l = std::getenv("MUON_LAUNCH")) {
    if (std::strcmp(l, "phase") == 0) c->per_phase = true;
  }
  if (const char* d = std::getenv("MUON_TEST_DROP_SIGNAL")) {
    if (std::strcmp(d, "1") == 0) c->drop_signal_once = true;
  }
  if (const char* o = std::getenv("MUON_OVERLAP")) {
    if (std::strcmp(o, "1") == 0) c->overlap = true;
  }
  {
    int least = 0, greatest = 0;
    bool ok = cudaDeviceGetStreamPriorityRange(&least, &greatest) == cudaSuccess &&
              cudaStreamCreateWithPriority(&c->side, cudaStreamNonBlocking, least) == cudaSuccess &&
              cudaEventCreateWithFlags(&c->ev_fork, cudaEventDisableTiming) == cudaSuccess &&
              cudaEventCreateWithFlags(&c->ev_join, cudaEventDisableTiming) == cudaSuccess;
    for (int g = 0; ok && g < MUON_MAX_GROUPS; ++g)
      ok = cudaEventCreateWithFlags(&c->ev_k1[g], cudaEventDisableTiming) == cudaSuccess &&
           cudaEventCreateWithFlags(&c->ev_gemm[g], cudaEventDisableTiming) == cudaSuccess;
    if (!ok) {
      cudaGetLastError();
      if (c->side) cudaStreamDestroy(c->side);
      c->side = nullptr;  // everything runs on the caller's stream
    }
  }
  if (cudaMalloc(&c->d_status, 3 * sizeof(int)) != cudaSuccess) {
    note_alloc_failure();
    delete c;
    return MUON_ERR_ALLOC;
  }
  cudaMemset(c->d_status, 0, 3 * sizeof(int));
  if (cudaMalloc(&c->d_done, sizeof(unsigned) * kMaxProblems * MUON_MAX_BATCH) != cudaSuccess) {
    note_alloc_failure();
    cudaFree(c->d_status);
    delete c;
    return MUON_ERR_ALLOC;
  }
  *out = c;
  return MUON_OK;
}

muon_status muon_destroy(muon_ctx* c) {
  if (!c) return MUON_OK;
  DeviceGuard guard(c->device);
  cudaDeviceSynchronize();
  cudaFree(c->ws);
  cudaFree(c->d_nu);
  cudaFree(c->d_s1);
  cudaFree(c->d_s2);
  cudaFree(c->d_flags);
  cudaFree(c->d_counters);
  cudaFree(c->d_partials);
  cudaFree(c->d_status);
  cudaFree(c->d_done);
  cudaFree(c->d_stage);
  cudaFree(c->d_aux);
  cudaFree(c->d_nu_all);
  cudaFree(c->d_flags_all);
  cudaFree(c->d_nu_blocks);
  cudaFree(c->d_flags_blocks);
  for (cudaEvent_t e : c->copy_events) cudaEventDestroy(e);
  for (cudaEvent_t e : c->events) cudaEventDestroy(e);
  for (int g = 0; g < MUON_MAX_GROUPS; ++g) {
    if (c->ev_k1[g]) cudaEventDestroy(c->ev_k1[g]);
    if (c->ev_gemm[g]) cudaEventDestroy(c->ev_gemm[g]);
  }
  if (c->ev_fork) cudaEventDestroy(c->ev_fork);
  if (c->ev_join) cudaEventDestroy(c->ev_join);
  if (c->side) cudaStreamDestroy(c->side);
  delete c;
  return MUON_OK;
}

muon_status muon_set_coeffs(muon_ctx* c, const float* abc, int k) {
  if (!c || !abc || k < 1 || k > MUON_MAX_ITERS) return MUON_ERR_INVALID_ARG;
  for (int i = 0; i < 3 * k; ++i)
    if (!std::isfinite(abc[i])) return MUON_ERR_INVALID_ARG;
  std::memcpy(c->coeffs, abc, sizeof(float) * 3 * k);
  c->k = k;
  return MUON_OK;
}

muon_status muon_get_coeffs(const muon_ctx* c, float* abc, int* k) {
  if (!c || !abc || !k) return MUON_ERR_INVALID_ARG;
  std::memcpy(abc, c->coeffs, sizeof(float) * 3 * c->k);
  *k = c->k;
  return MUON_OK;
}

muon_status muon_step_groups(muon_ctx* c, const muon_group* groups, int ngroups,
                             const muon_hparams* hp, void* stream) {
  std::vector<GroupPlan> plans;
  muon_status st = validate_and_plan(c, groups, ngroups, true, plans);
  if (st != MUON_OK) return st;
  st = check_hparams(hp);
  if (st != MUON_OK) return st;
  DeviceGuard guard(c->device);
  return run(c, plans, hp, true, hp->eps, static_cast<cudaStream_t>(stream));
}

muon_status muon_step(muon_ctx* c, void* const* W, const void* const* G, float* const* M,
                      int batch, int rows, int cols, int dtype, const muon_hparams* hp,
                      void* stream) {
  muon_group g;
  g.W = W;
  g.G = G;
  g.M = M;
  g.batch = batch;
  g.rows = rows;
  g.cols = cols;
  g.dtype = dtype;
  return muon_step_groups(c, &g, 1, hp, stream);
}

muon_status muon_ns_orthogonalize(muon_ctx* c, const void* const* X, void* const* Out, int batch,
                                  int rows, int cols, int dtype, float eps, void* stream) {
  if (!std::isfinite(eps) || eps < 0.f) return MUON_ERR_INVALID_ARG;
  muon_group g;
  g.W = Out;
  g.G = X;
  g.M = nullptr;
  g.batch = batch;
  g.rows = rows;
  g.cols = cols;
  g.dtype = dtype;
  std::vector<GroupPlan> plans;
  muon_status st = validate_and_plan(c, &g, 1, false, plans);
  if (st != MUON_OK) return st;
  for (int l = 0; l < batch; ++l)
    if (Out[l] == X[l]) return MUON_ERR_INVALID_ARG;
  DeviceGuard guard(c->device);
  return run(c, plans, nullptr, false, eps, static_cast<cudaStream_t>(stream));
}

muon_status muon_get_status(muon_ctx* c, int* flags, int capacity, int* count) {
  if (!c || capacity < 0) return MUON_ERR_INVALID_ARG;
  return last_status(c, flags, capacity, count, true);
}

muon_status muon_get_norms(muon_ctx* c, float* nu, int capacity, int* count) {
  if (!c || !nu || capacity < 0) return MUON_ERR_INVALID_ARG;
  DeviceGuard guard(c->device);
  if (count) *count = c->last_count;
  if (!c->pending || c->last_count == 0 || capacity == 0) return MUON_OK;
  MUON_CUDA(cudaStreamSynchronize(c->last_stream), "stream synchronize");
  MUON_CUDA(cudaMemcpy(nu, c->out_nu, sizeof(float) * std::min(capacity, c->last_count),
                       cudaMemcpyDeviceToHost),
            "read norms");
  return MUON_OK;
}

muon_status muon_step_groups_host(muon_ctx* c, const muon_group* groups, int ngroups,
                                  const muon_hparams* hp, float* nu_host, int* flags_host,
                                  void* stream) {
  if (!c || !groups || ngroups < 1 || ngroups > MUON_MAX_GROUPS) return MUON_ERR_INVALID_ARG;
  muon_status st = check_hparams(hp);
  if (st != MUON_OK) return st;
  size_t need = 0;
  for (int i = 0; i < ngroups; ++i) {
    st = check_group(groups[i], true);
    if (st != MUON_OK) return st;
    const size_t eb = groups[i].dtype == MUON_F32 ? 4 : 2;
    need += align_up(static_cast<size_t>(groups[i].rows) * groups[i].cols * eb, 256) * groups[i].batch;
  }
  DeviceGuard guard(c->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (need > c->stage_bytes) {
    MUON_CUDA(cudaStreamSynchronize(s), "sync before staging growth");
    cudaFree(c->d_stage);
    c->d_stage = nullptr;
    c->stage_bytes = 0;
    if (cudaMalloc(&c->d_stage, need) != cudaSuccess) {
      note_alloc_failure();
      return MUON_ERR_ALLOC;
    }
    c->stage_bytes = need;
  }
  // Staging slot of every matrix (256-byte aligned, group after group).
  std::vector<std::vector<const void*>> gptr(ngroups);
  std::vector<std::vector<size_t>> gbytes(ngroups);
  size_t off = 0;
  int total = 0;
  for (int i = 0; i < ngroups; ++i) {
    const size_t eb = groups[i].dtype == MUON_F32 ? 4 : 2;
    const size_t bytes = static_cast<size_t>(groups[i].rows) * groups[i].cols * eb;
    gptr[i].resize(groups[i].batch);
    gbytes[i].assign(groups[i].batch, bytes);
    for (int l = 0; l < groups[i].batch; ++l) {
      gptr[i][l] = static_cast<char*>(c->d_stage) + off;
      off += align_up(bytes, 256);
    }
    total += groups[i].batch;
  }
  if (c->side == nullptr) {
    // one stream: every upload, then one step over all groups
    std::vector<muon_group> dev(groups, groups + ngroups);
    for (int i = 0; i < ngroups; ++i) {
      for (int l = 0; l < groups[i].batch; ++l)
        MUON_CUDA(cudaMemcpyAsync(const_cast<void*>(gptr[i][l]), groups[i].G[l], gbytes[i][l],
                                  cudaMemcpyHostToDevice, s),
                  "gradient upload");
      dev[i].G = gptr[i].data();
    }
    std::vector<GroupPlan> plans;
    st = validate_and_plan(c, dev.data(), ngroups, true, plans);
    if (st != MUON_OK) return st;
    st = run(c, plans, hp, true, hp->eps, s);
    if (st != MUON_OK) return st;
  } else {
    // Slab pipeline: the uploads run on the side stream (copy engine) slab after slab while the
    // caller's stream steps each slab as soon as its gradients have landed, so the PCIe transfer of
    // slab k+1 overlaps the step of slab k.  A slab is up to ~32 MB of one group's gradients.
    constexpr size_t kSlabBytes = size_t(32) << 20;
    struct Slab { int g, l0, n; };
    std::vector<Slab> slabs;
    for (int i = 0; i < ngroups; ++i) {
      const size_t mb = std::max<size_t>(gbytes[i][0], 1);
      const int per = static_cast<int>(std::max<size_t>(1, kSlabBytes / mb));
      for (int l0 = 0; l0 < groups[i].batch; l0 += per)
        slabs.push_back({i, l0, std::min(per, groups[i].batch - l0)});
    }
    while (c->copy_events.size() < slabs.size()) {
      cudaEvent_t e;
      MUON_CUDA(cudaEventCreateWithFlags(&e, cudaEventDisableTiming), "event");
      c->copy_events.push_back(e);
    }
    if (total > c->cap_all) {
      MUON_CUDA(cudaStreamSynchronize(s), "sync before result growth");
      cudaFree(c->d_nu_all);
      cudaFree(c->d_flags_all);
      c->d_nu_all = nullptr;
      c->d_flags_all = nullptr;
      c->cap_all = 0;
      if (cudaMalloc(&c->d_nu_all, sizeof(float) * total) != cudaSuccess ||
          cudaMalloc(&c->d_flags_all, sizeof(int) * total) != cudaSuccess) {
        note_alloc_failure();
        return MUON_ERR_ALLOC;
      }
      c->cap_all = total;
    }
    // the uploads start once everything queued on the caller's stream (e.g. the previous step
    // still reading the staging buffer) is done
    MUON_CUDA(cudaEventRecord(c->ev_fork, s), "fork");
    MUON_CUDA(cudaStreamWaitEvent(c->side, c->ev_fork, 0), "fork");
    for (size_t k = 0; k < slabs.size(); ++k) {
      const Slab& sl = slabs[k];
      for (int l = sl.l0; l < sl.l0 + sl.n; ++l)
        MUON_CUDA(cudaMemcpyAsync(const_cast<void*>(gptr[sl.g][l]), groups[sl.g].G[l], gbytes[sl.g][l],
                                  cudaMemcpyHostToDevice, c->side),
                  "gradient upload");
      MUON_CUDA(cudaEventRecord(c->copy_events[k], c->side), "upload done");
    }
    int first = 0;
    std::vector<int> first_of_group(ngroups, 0);
    for (int i = 1; i < ngroups; ++i) first_of_group[i] = first_of_group[i - 1] + groups[i - 1].batch;
    for (size_t k = 0; k < slabs.size(); ++k) {
      const Slab& sl = slabs[k];
      MUON_CUDA(cudaStreamWaitEvent(s, c->copy_events[k], 0), "wait upload");
      muon_group sg = groups[sl.g];
      sg.W = groups[sl.g].W + sl.l0;
      sg.G = gptr[sl.g].data() + sl.l0;
      sg.M = groups[sl.g].M + sl.l0;
      sg.batch = sl.n;
      std::vector<GroupPlan> plans;
      st = validate_and_plan(c, &sg, 1, true, plans);
      if (st != MUON_OK) return st;
      st = run(c, plans, hp, true, hp->eps, s, nullptr, /*clear_status=*/k == 0);
      if (st != MUON_OK) return st;
      first = first_of_group[sl.g] + sl.l0;
      MUON_CUDA(cudaMemcpyAsync(c->d_nu_all + first, c->d_nu, sizeof(float) * sl.n, cudaMemcpyDeviceToDevice, s),
                "gather norms");
      MUON_CUDA(cudaMemcpyAsync(c->d_flags_all + first, c->d_flags, sizeof(int) * sl.n, cudaMemcpyDeviceToDevice,
                                s),
                "gather flags");
    }
    c->last_count = total;
    c->out_nu = c->d_nu_all;
    c->out_flags = c->d_flags_all;
  }
  if (nu_host)
    MUON_CUDA(cudaMemcpyAsync(nu_host, c->out_nu, sizeof(float) * c->last_count, cudaMemcpyDeviceToHost, s),
              "norm download");
  if (flags_host)
    MUON_CUDA(cudaMemcpyAsync(flags_host, c->out_flags, sizeof(int) * c->last_count, cudaMemcpyDeviceToHost, s),
              "flag download");
  MUON_CUDA(cudaStreamSynchronize(s), "stream synchronize");
  return last_status(c, nullptr, 0, nullptr, false);  // this call's: others' stay for muon_get_status
}

muon_status muon_power_iteration(muon_ctx* c, const void* const* W, float* const* u, float* const* v,
                                 float* sigma, int batch, int rows, int cols, int dtype, int iters,
                                 void* stream) {
  if (!c || !W || !u || !v || !sigma || batch < 1 || batch > MUON_MAX_BATCH || iters < 1 || iters > 10000)
    return MUON_ERR_INVALID_ARG;
  if (rows < 1 || cols < 1) return MUON_ERR_INVALID_ARG;
  if (rows > 32768 || cols > 32768) return MUON_ERR_UNSUPPORTED_SHAPE;
  if (dtype != MUON_BF16 && dtype != MUON_F32) return MUON_ERR_DTYPE;
  for (int l = 0; l < batch; ++l)
    if (!W[l] || !u[l] || !v[l]) return MUON_ERR_INVALID_ARG;
  DeviceGuard guard(c->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  GemvParams gp;
  std::memset(static_cast<void*>(&gp), 0, sizeof(gp));
  gp.rows = rows;
  gp.cols = cols;
  const bool f32 = dtype == MUON_F32;
  for (int l = 0; l < batch; ++l) gp.w[l] = W[l];
  bool fused = cols % 8 == 0 && cols <= power_pass_max_cols();
  for (int l = 0; l < batch && fused; ++l)
    if (reinterpret_cast<uintptr_t>(W[l]) % 16) fused = false;
  if (fused) {
    // one pass over W and one launch per iteration (power_stream_kernel)
    const int nblk = power_pass_blocks(rows, cols, batch, f32, c->sm_count);
    const size_t part_bytes = align_up(2 * sizeof(float) * batch * nblk * cols, 256);
    const size_t tsq_bytes = align_up(sizeof(float) * batch * nblk, 256);
    muon_status st = ensure_aux(c, part_bytes + tsq_bytes + 2 * sizeof(unsigned) * batch, s);
    if (st != MUON_OK) return st;
    gp.partial = static_cast<float*>(c->d_aux);
    float* tsq = reinterpret_cast<float*>(static_cast<char*>(c->d_aux) + part_bytes);
    unsigned* done = reinterpret_cast<unsigned*>(static_cast<char*>(c->d_aux) + part_bytes + tsq_bytes);
    for (int l = 0; l < batch; ++l) {
      gp.x[l] = v[l];
      gp.y[l] = u[l];
    }
    MUON_CUDA(launch_power_iteration_stream(gp, batch, f32, nblk, iters, tsq, done, sigma, c->d_status,
                                            c->sm_count, s),
              "power iteration");
    return MUON_OK;
  }
  gp.rows_per_chunk = 64;
  gp.row_chunks = (rows + 63) / 64;
  const size_t part_bytes = align_up(sizeof(float) * batch * gp.row_chunks * cols, 256);
  muon_status st = ensure_aux(c, part_bytes + sizeof(float) * MUON_MAX_BATCH, s);
  if (st != MUON_OK) return st;
  gp.partial = static_cast<float*>(c->d_aux);
  float* norms = reinterpret_cast<float*>(static_cast<char*>(c->d_aux) + part_bytes);
  MUON_CUDA(launch_normalize(v, batch, cols, norms, s), "normalise start vector");
  for (int i = 0; i < iters; ++i) {
    for (int l = 0; l < batch; ++l) {
      gp.x[l] = v[l];
      gp.y[l] = u[l];
    }
    MUON_CUDA(launch_gemv_rows(gp, batch, f32, s), "W v");
    MUON_CUDA(launch_normalize(u, batch, rows, norms, s), "normalise u");
    for (int l = 0; l < batch; ++l) {
      gp.x[l] = u[l];
      gp.y[l] = v[l];
    }
    MUON_CUDA(launch_gemv_cols(gp, batch, f32, s), "W^T u");
    MUON_CUDA(launch_normalize(v, batch, cols, sigma, s), "normalise v");
  }
  return MUON_OK;
}

muon_status muon_min_singular(muon_ctx* c, const void* const* W, float* const* y, const float* sigma_max,
                              float* sigma_min, int batch, int rows, int cols, int dtype, int iters, void* stream) {
  if (!c || !W || !y || !sigma_max || !sigma_min || batch < 1 || batch > MUON_MAX_BATCH || iters < 0 ||
      iters > 100000)
    return MUON_ERR_INVALID_ARG;
  if (rows < 1 || cols < 1) return MUON_ERR_INVALID_ARG;
  if (rows > 32768 || cols > 32768) return MUON_ERR_UNSUPPORTED_SHAPE;
  if (dtype != MUON_BF16 && dtype != MUON_F32) return MUON_ERR_DTYPE;
  for (int l = 0; l < batch; ++l)
    if (!W[l] || !y[l]) return MUON_ERR_INVALID_ARG;
  DeviceGuard guard(c->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool tall = rows > cols;
  const int m = tall ? cols : rows, n = tall ? rows : cols;  // wide view X is m x n
  const bool f32 = dtype == MUON_F32;
  if (tall) {
    // X X^T y = W^T W y: one streaming pass over W per shifted step (power_stream_kernel with a
    // shift), all passes in one launch when its blocks fit on the GPU at once
    bool stream_ok = cols % 8 == 0 && cols <= power_pass_max_cols();
    for (int l = 0; l < batch && stream_ok; ++l)
      if (reinterpret_cast<uintptr_t>(W[l]) % 16) stream_ok = false;
    const int nblk = stream_ok ? power_pass_blocks(rows, cols, batch, f32, c->sm_count) : 0;
    if (stream_ok && (iters == 0 || power_pass_together(cols, f32, nblk, batch, c->sm_count))) {
      const size_t part_bytes = align_up(2 * sizeof(float) * batch * nblk * cols, 256);
      const size_t tsq_bytes = align_up(sizeof(float) * batch * nblk, 256);
      const size_t cnt_bytes = align_up(2 * sizeof(unsigned) * batch, 256);
      const size_t t_bytes = align_up(sizeof(float) * rows, 256);
      muon_status st = ensure_aux(c, part_bytes + tsq_bytes + cnt_bytes + batch * t_bytes, s);
      if (st != MUON_OK) return st;
      char* base = static_cast<char*>(c->d_aux);
      GemvParams sp;
      std::memset(static_cast<void*>(&sp), 0, sizeof(sp));
      sp.rows = rows;
      sp.cols = cols;
      sp.partial = reinterpret_cast<float*>(base);
      float* tsq = reinterpret_cast<float*>(base + part_bytes);
      unsigned* counters = reinterpret_cast<unsigned*>(base + part_bytes + tsq_bytes);
      for (int l = 0; l < batch; ++l) {
        sp.w[l] = W[l];
        sp.x[l] = y[l];
        sp.y[l] = reinterpret_cast<float*>(base + part_bytes + tsq_bytes + cnt_bytes + l * t_bytes);
      }
      const cudaError_t e = launch_power_iteration_stream(sp, batch, f32, nblk, iters + 1, tsq, counters,
                                                          sigma_min, c->d_status, c->sm_count, s, sigma_max);
      if (e == cudaSuccess) return MUON_OK;
      // no room for the cooperative launch after all (another client on the device): two GEMVs
      if (e != cudaErrorCooperativeLaunchTooLarge) return cuda_fail(e, "shifted iteration");
      (void)cudaGetLastError();
    }
  }
  if (!tall) {
    // X = W: one pass over W per shifted step, column slabs (colslab_kernel), one launch
    bool aligned = true;
    for (int l = 0; l < batch && aligned; ++l)
      if (reinterpret_cast<uintptr_t>(W[l]) % 16) aligned = false;
    const int S = aligned ? colslab_width(rows, cols, batch, f32, c->sm_count) : 0;
    if (S > 0) {
      const int nslab = cols / S;
      const size_t part_bytes = align_up(2 * sizeof(float) * batch * nslab * rows, 256);
      const size_t dsq_bytes = align_up(sizeof(float) * batch * nslab, 256);
      muon_status st = ensure_aux(c, part_bytes + dsq_bytes + 2 * sizeof(unsigned) * batch, s);
      if (st != MUON_OK) return st;
      char* base = static_cast<char*>(c->d_aux);
      GemvParams sp;
      std::memset(static_cast<void*>(&sp), 0, sizeof(sp));
      sp.rows = rows;
      sp.cols = cols;
      sp.partial = reinterpret_cast<float*>(base);
      for (int l = 0; l < batch; ++l) {
        sp.w[l] = W[l];
        sp.x[l] = y[l];
      }
      const cudaError_t e = launch_min_singular_slabs(sp, batch, f32, S, iters, sigma_max,
                                                      reinterpret_cast<float*>(base + part_bytes),
                                                      reinterpret_cast<unsigned*>(base + part_bytes + dsq_bytes),
                                                      sigma_min, c->d_status, s);
      if (e == cudaSuccess) return MUON_OK;
      // no room for the cooperative launch after all (another client on the device): two GEMVs
      if (e != cudaErrorCooperativeLaunchTooLarge) return cuda_fail(e, "shifted iteration (column slabs)");
      (void)cudaGetLastError();
    }
  }
  GemvParams gp;
  std::memset(static_cast<void*>(&gp), 0, sizeof(gp));
  gp.rows = rows;
  gp.cols = cols;
  gp.rows_per_chunk = 64;
  gp.row_chunks = (rows + 63) / 64;
  const size_t part_bytes = align_up(sizeof(float) * batch * gp.row_chunks * cols, 256);
  const size_t w_bytes = align_up(sizeof(float) * n, 256), z_bytes = align_up(sizeof(float) * m, 256);
  muon_status st = ensure_aux(c, part_bytes + batch * (w_bytes + z_bytes), s);
  if (st != MUON_OK) return st;
  char* base = static_cast<char*>(c->d_aux);
  gp.partial = reinterpret_cast<float*>(base);
  float* wv[MUON_MAX_BATCH];
  float* zv[MUON_MAX_BATCH];
  for (int l = 0; l < batch; ++l) {
    gp.w[l] = W[l];
    wv[l] = reinterpret_cast<float*>(base + part_bytes + l * w_bytes);
    zv[l] = reinterpret_cast<float*>(base + part_bytes + batch * w_bytes + l * z_bytes);
  }
  // out <- X^T in (length n) and out <- X in (length m), X the wide view of W
  auto apply_xt = [&](float* const* in, float* const* out) {
    for (int l = 0; l < batch; ++l) {
      gp.x[l] = in[l];
      gp.y[l] = out[l];
    }
    return tall ? launch_gemv_rows(gp, batch, f32, s) : launch_gemv_cols(gp, batch, f32, s);
  };
  auto apply_x = [&](float* const* in, float* const* out) {
    for (int l = 0; l < batch; ++l) {
      gp.x[l] = in[l];
      gp.y[l] = out[l];
    }
    return tall ? launch_gemv_cols(gp, batch, f32, s) : launch_gemv_rows(gp, batch, f32, s);
  };
  MUON_CUDA(launch_normalize(y, batch, m, nullptr, s), "normalise start vector");
  for (int i = 0; i < iters; ++i) {
    MUON_CUDA(apply_xt(y, wv), "X^T y");
    MUON_CUDA(apply_x(wv, zv), "X X^T y");
    MUON_CUDA(launch_shift_normalize(y, zv, batch, m, sigma_max, s), "shifted step");
  }
  MUON_CUDA(apply_xt(y, wv), "X^T y");
  MUON_CUDA(launch_normalize(wv, batch, n, sigma_min, s), "Rayleigh estimate");
  return MUON_OK;
}

muon_status muon_step_capped(muon_ctx* c, void* const* W, const void* const* G, float* const* M,
                             const float* const* u, const float* const* v, int batch, int rows, int cols,
                             int dtype, const muon_hparams* hp, float* alpha, void* stream) {
  if (!u || !v || !alpha) return MUON_ERR_INVALID_ARG;
  muon_group g;
  g.W = W;
  g.G = G;
  g.M = M;
  g.batch = batch;
  g.rows = rows;
  g.cols = cols;
  g.dtype = dtype;
  std::vector<GroupPlan> plans;
  muon_status st = validate_and_plan(c, &g, 1, true, plans);
  if (st != MUON_OK) return st;
  st = check_hparams(hp);
  if (st != MUON_OK) return st;
  for (int l = 0; l < batch; ++l)
    if (!u[l] || !v[l]) return MUON_ERR_INVALID_ARG;
  DeviceGuard guard(c->device);
  CapSpec cap{u, v, alpha};
  return run(c, plans, hp, true, hp->eps, static_cast<cudaStream_t>(stream), &cap);
}

muon_status muon_expert_matmul(muon_ctx* c, const muon_experts* ex, const void* X, long long ldx, const void* W,
                               long long ldw, long long sw, void* Y, long long ldy, int transpose, int clear_rest,
                               void* stream) {
  const muon_status st = check_experts(c, ex);
  if (st != MUON_OK) return st;
  const int in = transpose ? ex->rows : ex->cols, out = transpose ? ex->cols : ex->rows;
  if (!rows_ok(X, ldx, ex->tokens, in) || !rows_ok(Y, ldy, ex->tokens, out) ||
      !stack_ok(W, ldw, sw, ex->experts, ex->rows, ex->cols, false))
    return MUON_ERR_INVALID_ARG;
  if (ex->tokens == 0) {
    c->last_count = 0;
    return MUON_OK;
  }
  if (Y == X || Y == W) return MUON_ERR_INVALID_ARG;
  DeviceGuard guard(c->device);
  ExpertParams p;
  std::memset(static_cast<void*>(&p), 0, sizeof(p));
  p.features = out;
  p.k_tiles = (in + 63) / 64;
  p.out = Y;
  p.ld_out = ldy;
  p.out_f32 = ex->dtype == MUON_F32;
  const int quad = ex->dtype == MUON_F32 ? 4 : 8;  // elements of 16 bytes
  p.vec = (ex->tokens == 1 || ldy % quad == 0) && reinterpret_cast<uintptr_t>(Y) % 16 == 0;
  p.clear_rest = clear_rest != 0;
  p.scale = 1.f;
  return run_experts(c, ex, transpose ? EXPERT_BACKWARD : EXPERT_FORWARD,
                     Operand{W, ex->experts, ex->rows, ex->cols, 1, ldw, sw, 0},
                     Operand{X, 1, ex->tokens, in, 1, ldx, 0, 0}, p, static_cast<cudaStream_t>(stream));
}

static muon_status expert_grad(muon_ctx* c, const muon_experts* ex, const void* dY, long long ldy, const void* X,
                               long long ldx, void* G, long long ldg, long long sg, int out_dtype, float beta,
                               float scale, bool fresh, void* stream) {
  const muon_status st = check_experts(c, ex);
  if (st != MUON_OK) return st;
  if (out_dtype != MUON_F32 && out_dtype != ex->dtype) return MUON_ERR_DTYPE;
  if (!finite(beta) || !finite(scale)) return MUON_ERR_INVALID_ARG;
  if (!rows_ok(dY, ldy, ex->tokens, ex->rows) || !rows_ok(X, ldx, ex->tokens, ex->cols) ||
      !stack_ok(G, ldg, sg, ex->experts, ex->rows, ex->cols, true))
    return MUON_ERR_INVALID_ARG;
  if (G == dY || G == X) return MUON_ERR_INVALID_ARG;
  DeviceGuard guard(c->device);
  ExpertParams p;
  std::memset(static_cast<void*>(&p), 0, sizeof(p));
  p.features = ex->cols;
  p.rows = ex->rows;
  p.out = G;
  p.ld_out = ldg;
  p.s_out = sg;
  p.out_f32 = out_dtype == MUON_F32;
  const int quad = out_dtype == MUON_F32 ? 4 : 8;  // elements of 16 bytes
  p.vec = (ex->rows == 1 || ldg % quad == 0) && (ex->experts == 1 || sg % quad == 0) &&
          reinterpret_cast<uintptr_t>(G) % 16 == 0;
  p.beta = beta;
  p.scale = scale;
  p.clear_rest = fresh;
  return run_experts(c, ex, EXPERT_WGRAD, Operand{X, 1, ex->tokens, ex->cols, 1, ldx, 0, 0},
                     Operand{dY, 1, ex->tokens, ex->rows, 1, ldy, 0, 0}, p, static_cast<cudaStream_t>(stream));
}

muon_status muon_expert_grad(muon_ctx* c, const muon_experts* ex, const void* dY, long long ldy, const void* X,
                             long long ldx, void* G, long long ldg, long long sg, int out_dtype, float beta,
                             float scale, void* stream) {
  return expert_grad(c, ex, dY, ldy, X, ldx, G, ldg, sg, out_dtype, beta, scale, false, stream);
}

muon_status muon_expert_grad_new(muon_ctx* c, const muon_experts* ex, const void* dY, long long ldy, const void* X,
                                 long long ldx, void* G, long long ldg, long long sg, int out_dtype, float scale,
                                 void* stream) {
  return expert_grad(c, ex, dY, ldy, X, ldx, G, ldg, sg, out_dtype, 0.f, scale, true, stream);
}

muon_status muon_check_blocks(int rows, int cols, int block_rows, int block_cols, int dtype) {
  BlockParams p;
  size_t smem = 0;
  return plan_blocks(rows, cols, block_rows, block_cols, dtype, p, &smem);
}

muon_status muon_step_blocks(muon_ctx* c, const muon_blocks* blocks, const muon_hparams* hp, void* stream) {
  if (!c) return MUON_ERR_INVALID_ARG;
  const muon_status st = check_hparams(hp);
  if (st != MUON_OK) return st;
  DeviceGuard guard(c->device);
  return run_blocks(c, blocks, hp, true, hp->eps, static_cast<cudaStream_t>(stream));
}

muon_status muon_ns_orthogonalize_blocks(muon_ctx* c, const muon_blocks* blocks, float eps, void* stream) {
  if (!c || !std::isfinite(eps) || eps < 0.f) return MUON_ERR_INVALID_ARG;
  DeviceGuard guard(c->device);
  return run_blocks(c, blocks, nullptr, false, eps, static_cast<cudaStream_t>(stream));
}

size_t muon_workspace_bytes(const muon_ctx* c) {
  if (!c) return 0;
  return c->ws_bytes + c->stage_bytes + c->aux_bytes;
}

muon_status muon_profile_enable(muon_ctx* c, int on) {
  if (!c) return MUON_ERR_INVALID_ARG;
  c->profiling = on != 0;
  return MUON_OK;
}

muon_status muon_profile_read(muon_ctx* c, muon_profile* out, int reset) {
  if (!c || !out) return MUON_ERR_INVALID_ARG;
  DeviceGuard guard(c->device);
  std::memset(out, 0, sizeof(*out));
  for (size_t i = 0; i < c->rec_kind.size(); ++i) {
    MUON_CUDA(cudaEventSynchronize(c->events[2 * i + 1]), "profile event");
    float ms = 0.f;
    MUON_CUDA(cudaEventElapsedTime(&ms, c->events[2 * i], c->events[2 * i + 1]), "profile elapsed");
    out->launches[c->rec_kind[i]] += 1;
    out->ms[c->rec_kind[i]] += ms;
  }
  if (reset) c->rec_kind.clear();
  return MUON_OK;
}

}  // extern "C"
