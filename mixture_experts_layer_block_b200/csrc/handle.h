// handle.h -- the handle behind the C ABI and the host helpers that its entry points share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <initializer_list>
#include <vector>

#include "launch.h"
#include "moe_b200.h"
#include "mx.cuh"

namespace moe {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct MapKey {
  const void* ptr;
  uint64_t inner, outer, stride;
  uint32_t box0, box1;
  int dtype;
  bool operator==(const MapKey& o) const {
    return ptr == o.ptr && inner == o.inner && outer == o.outer && stride == o.stride &&
           box0 == o.box0 && box1 == o.box1 && dtype == o.dtype;
  }
};

struct MapEntry {
  MapKey key;
  CUtensorMap map;
};

constexpr int64_t kDefaultTimeoutNs = 2000000000LL;

}  // namespace moe

struct moe_handle {
  moe_config cfg{};
  int device = 0;
  int num_sms = 0;
  char* ws_mem = nullptr;
  size_t ws_bytes = 0;
  moe::Workspace ws{};
  int max_tiles = 0, max_lag = 0, max_units = 0;
  int64_t sorted_len_max = 0, blocks_len_max = 0;
  size_t gate_smem = 0;
  moe::EncodeTiledFn encode = nullptr;
  std::vector<moe::MapEntry> cache;
  CUtensorMap h_routed{}, h_shared{}, xs_map{}, y_map{};
  CUtensorMap h_routed16{}, h_shared16{}, xs_map16{};  // 16-row boxes for batches of <= 16 tokens
  CUtensorMap h_routed32{}, h_shared32{}, xs_map32{}, y_map32{};  // 32-row boxes (SM-pair tiles)
  int max_routed_tiles = 0;
  int64_t routed_rows = 0, tile_rows = 0;  // rows of xs, and of h and y, for either tile height
  int max_pairs = 0;                       // 2-CTA clusters of the pair kernel that fit at once
  int last_workers = 0, last_tile_m = moe::kBM;
  int last_shape = 0;  // expert-GEMM shape of the last forward: 0 general, 1 small, 2 tail, 3 pair
  int last_kernels = 0;  // kernels launched by the last forward
  bool fused_ok = false;  // batches of <= 16 tokens may run as one fused launch on this device
  bool mx_fused_ok = false;  // the same for moe_forward_mxfp8
  int32_t epoch = 0;      // fused forwards launched (the arrival counter's target / grid size)
  int parts_rows = 0;  // rows of the K-split partial logits buffer
  std::vector<cudaEvent_t> ev;  // kTimingRing x (kNumStages + 1) events around the kernels
  int timed = 0;                // forwards recorded since the last moe_stage_times
  bool timing = false;
  cudaStream_t last_stream = nullptr;
  bool have_forward = false;
  int last_T = 0, last_k = 0, last_lag = 0;
  void* x_stage = nullptr;   // [2 slots][max_tokens][H] bf16 (slot 0 for moe_forward_host)
  float* out_stage = nullptr;  // [2 slots][max_tokens][H] fp32 or bf16
  size_t x_slot_bytes = 0, out_slot_bytes = 0;
  // moe_forward_host_async: copy streams and, per staging slot, the events that order the
  // copy in, the forward and the copy back
  cudaStream_t copy_in = nullptr, copy_out = nullptr;
  cudaEvent_t ev_in[2] = {nullptr, nullptr}, ev_done[2] = {nullptr, nullptr}, ev_out[2] = {nullptr, nullptr};
  bool slot_used[2] = {false, false};
  int async_slot = 0;
  bool async_pending = false;
  int dep_extra_next = 0;
  int64_t timeout_ns = moe::kDefaultTimeoutNs;
  // MXFP8 workspace (MOE_FLAG_MXFP8): x in token order and in tile order, h, with their scales
  moe::MxBuffers mx{};
  CUtensorMap mx_xs_map{}, mx_h_map{}, mx_xs_map32{}, mx_h_map32{};
  // status and abort words of the feed-forward block's kernels: apart from the layer's, which
  // each layer forward resets, because such a call may run beside one on another stream
  moe::DeviceMeta* ffn_meta = nullptr;
  int ffn_pairs = 0;  // 2-CTA clusters of the block's GEMMs that fit on the device at once
  // set by the first moe_ffn_* call that launches, from any thread: from then on moe_get_status waits for the device,
  // since such calls may be under way on any number of streams, in replayed graphs too
  std::atomic<bool> ffn_used{false};
};

namespace moe {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int encode_map(moe_handle* h, CUtensorMap* out, const void* ptr, uint64_t inner, uint64_t outer,
                      uint64_t stride_bytes, uint32_t box0, uint32_t box1,
                      CUtensorMapDataType dtype = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                      CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {stride_bytes};
  cuuint32_t box[2] = {box0, box1};
  cuuint32_t es[2] = {1, 1};
  CUresult r = h->encode(out, dtype, 2, const_cast<void*>(ptr), dims,
                         strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MOE_OK : MOE_ERR_CUDA;
}

inline int check_cuda(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

inline int select_device(moe_handle* h) { return check_cuda(cudaSetDevice(h->device)); }

// A buffer of a call, to tell whether two of them overlap.
struct Span {
  const void* p;
  int64_t bytes;
};

inline bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y ? y - x < (uintptr_t)a.bytes : x - y < (uintptr_t)b.bytes;
}

// Whether one of the buffers that a call writes overlaps another, or one that it reads: kernels read
// and write tiles in no fixed order, so that the results would depend on timing.
inline bool clobbers(std::initializer_list<Span> writes, std::initializer_list<Span> reads) {
  for (const Span* w = writes.begin(); w != writes.end(); ++w) {
    for (const Span* o = w + 1; o != writes.end(); ++o)
      if (overlap(*w, *o)) return true;
    for (const Span& r : reads)
      if (overlap(*w, r)) return true;
  }
  return false;
}

// The handle's device for the length of one call; the caller's device is put back at the end.
class DeviceScope {
 public:
  explicit DeviceScope(int device) {
    if (cudaGetDevice(&old_) != cudaSuccess) old_ = -1;
    rc_ = old_ == device ? MOE_OK : check_cuda(cudaSetDevice(device));
    if (old_ == device) old_ = -1;
  }
  ~DeviceScope() {
    if (old_ >= 0) cudaSetDevice(old_);
  }
  DeviceScope(const DeviceScope&) = delete;
  DeviceScope& operator=(const DeviceScope&) = delete;
  int rc() const { return rc_; }

 private:
  int old_ = -1, rc_ = MOE_OK;
};

}  // namespace moe
