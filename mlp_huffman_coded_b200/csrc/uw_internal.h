// Host-side internals shared by the libuw translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "uw.h"

namespace uw {

// Device facts cached per device ordinal.
struct DeviceInfo {
  int ordinal = -1;
  int sm_count = 0;
  int major = 0, minor = 0;
  size_t max_smem_optin = 0;
  size_t l2_bytes = 0;
};
uw_status device_info(DeviceInfo* out);  // current device

// Counts every kernel launch issued through the library.
void note_launch(int n = 1);

// Maps a CUDA error to a status (UW_OK for cudaSuccess).
inline uw_status cuda_status(cudaError_t e) { return e == cudaSuccess ? UW_OK : UW_ERR_CUDA; }

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link
// against libcuda).  2-D, row-major: dims {inner, outer}, row stride in bytes.
uw_status make_tensor_map_2d(CUtensorMap* map, CUtensorMapDataType dtype, const void* base,
                             uint64_t inner, uint64_t outer, uint64_t row_stride_bytes,
                             uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle);
// Same, 3-D: dims {d0, d1, d2} (d0 contiguous), byte strides of dims 1 and 2
// (any order, multiples of 16), box {b0, b1, b2}.
uw_status make_tensor_map_3d(CUtensorMap* map, CUtensorMapDataType dtype, const void* base, uint64_t d0,
                             uint64_t d1, uint64_t d2, uint64_t stride1_bytes, uint64_t stride2_bytes, uint32_t b0,
                             uint32_t b1, uint32_t b2, CUtensorMapSwizzle swizzle);

// Workspace layout: [0, 256) header (status word at offset 0), then tile
// counters, split-K partials and the pipeline's intermediate matrix.
constexpr size_t kWsHeader = 256;
// Split-K tile counters: one fixed-size region right after the header, so
// the partial sums start at the same offset for every GEMM plan and one
// GEMM's partials never land on another's counters when calls share a
// workspace.  16384 tiles.
constexpr size_t kCounterBytes = 64 * 1024;
inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Shape of one GEMM launch, shared by every pipeline so that the K split and
// its reduction order are identical for all of them.
struct GemmPlan {
  int64_t N = 0, K = 0;
  int B = 0;
  int KB = 0;        // K / 64
  int n_mtiles = 0;  // ceil(N / 128)
  int n_ntiles = 0;  // ceil(B / 256)
  int ntile = 0;     // batch columns per tile (multiple of 16, <= 256)
  int64_t units = 0; // n_mtiles * n_ntiles * KB
  int grid = 0;      // CTAs (<= SM count, <= units)
  size_t counter_bytes = 0;
  size_t partial_bytes = 0;
};
uw_status gemm_plan(int64_t N, int64_t K, int B, int sm_count, GemmPlan* out);
size_t gemm_ws_bytes(const GemmPlan& p);  // header + counters + partials
size_t pipeline_scratch_bytes(const uw_layout* L, int pipeline);

// Device pointer checks.
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
uw_status check_matrix(const uw_matrix* m);

// Kernel launchers (asynchronous).
uw_status launch_decode(const uw_matrix* m, int mode, void* out, uint32_t* status, cudaStream_t s);
// Full decode of rows[0..n_rows) (device int32) into out [n_rows, cols] BF16.
uw_status launch_decode_rows(const uw_matrix* m, const int32_t* rows, int64_t n_rows, void* out, uint32_t* status,
                             cudaStream_t s);
enum Loader { kLoaderBF16 = 0, kLoaderEXP8 = 1, kLoaderIDX4 = 2, kLoaderPACK = 3 };
struct GemmArgs {
  int loader = kLoaderIDX4;
  int64_t N = 0, K = 0;
  int B = 0;
  const uint8_t* sm = nullptr;
  const uint8_t* aux = nullptr;       // idx4 or exp8
  const uint16_t* wbf16 = nullptr;    // BF16 loader
  const uint32_t* vflags = nullptr;
  const uint32_t* vprefix = nullptr;
  const uint16_t* verbatim = nullptr;
  long long n_verbatim = 0;            // verbatim groups (bounds the slots read)
  int wpr = 0;
  const uint8_t* pack = nullptr;      // direct-palette pack: bodies, then verbatim tails (PACK loader)
  const uint32_t* pack_off = nullptr;
  const uint8_t* palette = nullptr;   // 16 entries (IDX4 / PACK loaders)
  const uint8_t* code_len = nullptr;  // which palette entries are in use
  const uint16_t* x = nullptr;
  uint16_t* y = nullptr;
  const uint16_t* gate = nullptr;     // non-NULL: y = SiLU(gate) * (x W^T)
  void* ws = nullptr;
  size_t ws_bytes = 0;
  int force_mixed_palette = 0;        // testing: use the general lookup
  // Launch with programmatic dependent launch (the kernel streams its weights
  // before waiting for the previous kernel on the stream).  Off when that
  // previous kernel wrote the weights (a decode kernel of the same call).
  bool overlap_previous = true;
};
uw_status launch_gemm(const GemmArgs& a, cudaStream_t s);
uw_status launch_swiglu(const uint16_t* g, const uint16_t* u, uint16_t* h, int64_t n, cudaStream_t s);


// Products grouped by expert.  The device record of one compressed matrix:
// where its pack lies and its palette tables (PaletteTables).
constexpr int kMaxExperts = UW_MAX_EXPERTS;
struct alignas(16) ExpertDesc {
  const uint8_t* pack;       // tile records
  const uint8_t* tails;      // verbatim rows, tile order
  const uint32_t* pack_off;  // per tile: verbatim rows of all earlier tiles
  uint32_t n_verbatim, mixed;
  uint32_t lo0, lo1, hi0, hi1, b7lo0, b7lo1, b7hi0, b7hi1, keep;
  uint32_t reserved[3];
};
static_assert(sizeof(ExpertDesc) == 80, "uw_experts_table_bytes");
uw_status expert_desc(const uw_matrix* m, ExpertDesc* out);

struct GroupedArgs {
  int64_t N = 0, K = 0;
  int E = 1;
  bool swiglu = false;                         // table[0] = gate, table[1] = up
  const void* table[2] = {nullptr, nullptr};   // device ExpertDesc[E]; NULL: `one` is the only group's
  const ExpertDesc* one = nullptr;             // host
  const uint16_t* x = nullptr;
  int x_rows = 0;
  const int32_t* rows = nullptr;     // row of x per slot, NULL: slot s reads row s
  const int32_t* offsets = nullptr;  // first slot of each group, NULL: one group of n_rows
  // The offsets were written before the kernel just ahead on the stream
  // started: they are read, and weights stream, before waiting for it.
  bool offsets_ready = false;
  int n_rows = 0;
  const uint16_t* bias = nullptr;
  const uint16_t* residual = nullptr;
  int activation = UW_ACT_NONE, out_type = UW_OUT_BF16;
  void* y = nullptr;
  void* ws = nullptr;
  size_t ws_bytes = 0;
};
// `scattered`: room for x's rows next to each other too.  0: unsupported
size_t grouped_ws_bytes(int64_t N, int64_t K, int E, int n_rows, bool swiglu, bool scattered);
uw_status launch_grouped(const GroupedArgs& a, cudaStream_t s);

}  // namespace uw
