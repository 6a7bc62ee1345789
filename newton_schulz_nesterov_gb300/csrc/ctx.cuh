// The handle behind dmuon_handle_t and what every entry point does with it:
// error texts, profiling brackets, pointer checks, the tensor-map encoder.
// Host code, shared by the translation units of the C ABI.
#pragma once

#include <cstdio>
#include <mutex>
#include <string>
#include <vector>

#include <cudaTypedefs.h>

#include "../../include/dmuon.h"
#include "common.cuh"
#include "gram.cuh"
#include "plan.cuh"
#include "small.cuh"

namespace dmuon {

// Cached caller pointer sets per plan (see run()).
constexpr int kPtrSlots = 64;

// cuTensorMapEncodeTiled, looked up once; nullptr if the driver lacks it.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return encode;
}

struct ProfRec {
  cudaEvent_t a, b;
  int kind;
};

// One chunk of the matrix list: a contiguous run [i0, i0 + n) planned and
// launched as a unit.  All chunks share one workspace and run one after the
// other on the stream.
struct Chunk {
  int i0 = 0, n = 0;
  Layout L;                       // sub-list layout (workspace offsets, work lists)
  MatDesc* d_mats = nullptr;
  CUtensorMap* d_maps = nullptr;
  int64_t* d_prefix = nullptr;
  float* d_partials = nullptr;
  float* d_tmax = nullptr;        // per momentum tile: max |U|
  float* d_svec = nullptr;        // per matrix: s/p
  float* d_bvec = nullptr;        // per matrix: beta', the scale of the iterate after the first product
  float* d_pscale = nullptr;      // per matrix: the prescale p of X[0] (kept across steps)
  int* d_redo = nullptr;          // per matrix: X[0] to be rewritten with a new p
  int* d_counters = nullptr;      // per matrix: finished tiles of a fused launch (zeroed before it)
  int4* d_items[3] = {nullptr, nullptr, nullptr};
  int* d_starts[3] = {nullptr, nullptr, nullptr};
  GramDesc* d_gd = nullptr;       // gram plans: per-matrix Gram-space buffers
  CUtensorMap* d_gmaps = nullptr; // gram plans: kGramBufs maps per matrix
};

}  // namespace dmuon

struct dmuon_ctx {
  int device = 0;
  int num_sms = 0;
  // plan
  std::vector<dmuon_shape_t> shapes;   // caller order
  std::vector<int> order;              // plan position -> caller index
  int n_large = 0;                     // plan positions [0, n_large) are chunked
  std::vector<dmuon::SmallDesc> small_descs;  // plan positions [n_large, n)
  dmuon::SmallDesc* d_small = nullptr;
  bool small_path = true;              // requested
  bool small_ok = false;               // small kernel configured on this device
  bool plan_small = false;             // small kernel used by the current plan
  bool plan_gram = false;              // chunks laid out for the Gram-space backend
  bool gram_ok = false;                // Gram-space kernels configured on this device
  std::vector<dmuon::Chunk> chunks;
  size_t ws_bytes = 0, small_bytes = 0;
  void* ws = nullptr;
  void* small = nullptr;
  dmuon::MatPtrs* d_ptrs = nullptr;
  int* d_flags = nullptr;
  int* d_err = nullptr;
  // pointer-set cache: kPtrSlots device slots of n MatPtrs each
  std::vector<dmuon::MatPtrs> slot_ptrs[dmuon::kPtrSlots];
  uint64_t slot_use[dmuon::kPtrSlots] = {};
  bool slot_pending[dmuon::kPtrSlots] = {};
  cudaEvent_t slot_ev[dmuon::kPtrSlots] = {};
  uint64_t use_clock = 0;
  dmuon::MatPtrs* h_stage = nullptr;  // pinned staging, kPtrSlots x n
  cudaStream_t last_stream = nullptr;
  int64_t launches = 0;
  bool profiling = false;
  std::vector<dmuon::ProfRec> prof;
  std::vector<cudaEvent_t> ev_pool;
  std::string last_error;
  unsigned long long wait_timeout_ns = 0;  // 0: kernels' default (4 s)
  int max_clusters = 0;                     // resident 2-CTA clusters (0: pairs unavailable)
  int tile_mode = 0;                        // requested: 0 auto, 1 single CTA, 2 CTA pairs, 3 single CTA 128x128
  int64_t chunk_elems = 0;                  // requested chunk size (0: default)
  bool plan_pair = false;                   // tile kind of the current plan
  int plan_bn = dmuon::kBN;                        // its single-CTA tile width (256, or 128)
  int64_t plan_chunk_elems = 0;             // chunk size of the current plan
  // Overlap of chunk c+1's momentum pass with chunk c's tensor-core phases:
  // a side stream, two alternating chunk workspaces and fork/join events.
  bool overlap = false;                     // requested (off: measured neutral at the power cap)
  bool balanced = true;                     // requested: work items dealt longest-first to the least loaded
  int f16_iters = 3;                        // direct backend: leading iterations with fp16 operands
  int fused = 2;                            // direct backend, one launch per chunk for all products:
                                            // 0 never, 1 always, 2 for chunks of few work items
  bool plan_balanced = true;                // in the current plan
  bool plan_overlap = false;                // in the current plan (needs >= 2 chunks)
  size_t ws_chunk = 0;                      // bytes of one chunk workspace
  cudaStream_t side = nullptr;
  cudaEvent_t ev_fork = nullptr, ev_join = nullptr, ev_norm[2] = {}, ev_gemm[2] = {};
  // AdamW / clipping: descriptor buffer (device), pinned staging, results
  void* aux_dev = nullptr;
  size_t aux_dev_cap = 0;
  uint8_t* aux_host = nullptr;
  size_t aux_host_cap = 0;
  cudaEvent_t aux_ev = nullptr;
  bool aux_pending = false;
  // Operators of a 4-bit block: a wait that ran out (device word, allocated
  // with the handle) and the norm backward's partial sums
  int* d_op_err = nullptr;
  void* op_ws = nullptr;
  size_t op_ws_cap = 0;
  int norm_places[8] = {};
  bool quant_ready = false, norm_ready = false;  // the kernels' limits of shared memory are set
  bool op_ws_captured = false;         // a graph holds op_ws: it stays until the handle goes
  std::vector<void*> op_ws_kept;
};

namespace dmuon {

inline int cuda_err(cudaError_t e) { return e == cudaSuccess ? DMUON_OK : (e == cudaErrorMemoryAllocation ? DMUON_ERR_OOM : DMUON_ERR_CUDA); }

// Record what failed (readable through dmuon_last_error) and return `code`.
inline int fail(dmuon_ctx* h, int code, const char* what, cudaError_t e = cudaSuccess) {
  char buf[384];
  if (e != cudaSuccess)
    std::snprintf(buf, sizeof buf, "%s: %s (%d)", what, cudaGetErrorString(e), (int)e);
  else
    std::snprintf(buf, sizeof buf, "%s", what);
  h->last_error = buf;
  return code;
}

inline cudaEvent_t pool_event(dmuon_ctx* h) {
  if (!h->ev_pool.empty()) { cudaEvent_t e = h->ev_pool.back(); h->ev_pool.pop_back(); return e; }
  cudaEvent_t e = nullptr;
  cudaEventCreate(&e);
  return e;
}

inline bool capturing(cudaStream_t s) {
  cudaStreamCaptureStatus c = cudaStreamCaptureStatusNone;
  return cudaStreamIsCapturing(s, &c) == cudaSuccess && c != cudaStreamCaptureStatusNone;
}

struct LaunchGuard {  // brackets one launch with profiling events (not under capture)
  dmuon_ctx* h; cudaStream_t s; ProfRec r; bool on;
  LaunchGuard(dmuon_ctx* h_, cudaStream_t s_, int kind) : h(h_), s(s_), on(h_->profiling && !capturing(s_)) {
    if (on) { r.a = pool_event(h); r.b = pool_event(h); r.kind = kind; cudaEventRecord(r.a, s); }
  }
  ~LaunchGuard() {
    ++h->launches;
    if (on) { cudaEventRecord(r.b, s); h->prof.push_back(r); }
  }
};

inline int check_ptr(const void* p) {
  if (!p) return DMUON_ERR_ARG;
  if (((uintptr_t)p & 15u) != 0) return DMUON_ERR_ALIGN;
  return DMUON_OK;
}

}  // namespace dmuon
