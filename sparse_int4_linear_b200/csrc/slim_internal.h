// Internal launch wrappers shared by the host API (not part of the C ABI).
#pragma once
#include <cuda_runtime.h>
#include <array>
#include <cstdint>
#include <cstddef>
#include <map>
#include <shared_mutex>
#include <mutex>

#include <nvtx3/nvToolsExt.h>

#include "slim.h"

namespace slim {

// An NVTX range over a scope of host code (a call, a pack step, a kernel
// launch); a no-op unless a profiler is attached.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

// Tuning knobs, read from the environment at the library's first call and
// again by slim_tuning_reload():
//   SLIM_NO_STREAM      M <= 16 never uses the single-launch kernel
//   SLIM_STREAM_WARPS   8 or 16 main warps in the single-launch kernel
//   SLIM_PDL_EARLY      the single-launch kernel signals the next launch early
//   SLIM_DECODE_CFG     "WR,KW,S" forces the token-tiled decode kernel's split
//   SLIM_NO_PREFILL     M > 16 stays on the token-tiled decode kernels
//   SLIM_PREFILL_1SM    the prefill path never uses SM pairs
//   SLIM_PREFILL_TILE   "halves,tokens" or "pair,tokens" forces a prefill tile of the
//                       forward and the gated block (where that path has it: one half
//                       64 or 128 tokens in the forward, two 128 or 192, and 64 in the
//                       gated block; pairs 128, 192, 224 or 240 from 256 tokens on)
struct Tuning {
  bool no_stream = false, no_prefill = false, prefill_1sm = false, pdl_early = false;
  int stream_warps = 0;                      // 0: chosen per call
  bool decode_cfg = false;
  int dec_wr = 0, dec_kw = 0, dec_s = 0;
  bool prefill_tile = false, prefill_pair = false;
  int prefill_nh = 0, prefill_tt = 0;
  unsigned generation = 0;                   // bumped by every reload; part of every plan-cache key
};
Tuning tuning();
void reload_tuning();

// Thread-safe memo of host-side plans.  Keys hold the device, the tuning
// generation and every input the plan depends on.
template <size_t N, class V>
class PlanCache {
 public:
  using Key = std::array<long long, N>;
  template <class F>
  V get(const Key& k, F&& make) {
    {
      std::shared_lock<std::shared_mutex> lock(mu_);
      auto it = map_.find(k);
      if (it != map_.end()) return it->second;
    }
    V v = make();
    std::unique_lock<std::shared_mutex> lock(mu_);
    map_.emplace(k, v);
    return v;
  }

 private:
  std::shared_mutex mu_;
  std::map<Key, V> map_;
};

// The calling thread's current CUDA device (-1 if it cannot be read).
int current_device();
// Record a failed CUDA call for slim_last_cuda_error() (per host thread).
void set_last_cuda_error(cudaError_t e);
int last_cuda_error();

cudaError_t launch_pack(const slim_layer& L, const uint16_t* W, cudaStream_t s);
cudaError_t launch_pack_adapter(const slim_layer& L, const uint16_t* Lsrc, const uint16_t* Rsrc,
                                cudaStream_t s);
cudaError_t launch_pack_done(cudaStream_t s);
// 4-bit adapters (layer.adapter_bits == 4): quantize L and R into Lq / Rq.
// The bf16 layouts (Lf, Rf, Rp, Lp) packed after it then hold the
// dequantized values.
cudaError_t launch_quant_adapter(const slim_layer& L, const uint16_t* Lsrc, const uint16_t* Rsrc, cudaStream_t s);
cudaError_t launch_unpack_adapters(const slim_layer& L, int8_t* qL, uint16_t* sL, int8_t* qR, uint16_t* sR,
                                   cudaStream_t s);
cudaError_t launch_unpack_dec(const slim_layer& L, int8_t* q, uint16_t* scales, cudaStream_t s);

// What the forward writes: Y [M][N], or for the gated block H = act(G) U in Y
// [M][N / 2] and, when not null, GU [M][N].
struct GatedOut {
  uint16_t* Y = nullptr;
  bool gated = false;
  int act = 0;
  uint16_t* GU = nullptr;
  // Test aid: the gated kernels also wait that many SM cycles for something
  // that never comes (0: they do not), and so give up.
  long long fail_cycles = 0;
};

// Adapter down-projection T = X L into `T` (bf16 [ceil(M/16)*16][r16]).
cudaError_t launch_adapter_down(const slim_layer& L, const uint16_t* X, int M, uint16_t* T,
                                cudaStream_t s);
// Sparse int4 main product plus the adapter up-projection, bf16 Y.
cudaError_t launch_decode(const slim_layer& L, const uint16_t* X, int M, uint16_t* Y, const uint16_t* T,
                          cudaStream_t s);

// The forward: tensor-core prefill (M > 16, when allowed), the single-launch
// streaming decode (M <= 16, when its plan fits and its workspace fits
// `ws_limit`), else the token-tiled adapter-down + decode pair.  `ws` must be
// zero-filled before its first use (the streaming kernel keeps a control
// block at its start).
size_t forward_ctl_bytes(int r16);
// `allow_prefill` false keeps M > 16 on the token-tiled decode kernels (no
// dequantized-image workspace).
size_t forward_workspace_bytes(const slim_layer& L, int M, bool allow_prefill, size_t ws_limit = SIZE_MAX);
// The most forward_workspace_bytes gives for any M' in [1, M].
size_t forward_workspace_bytes_upto(const slim_layer& L, int M, bool allow_prefill, size_t ws_limit = SIZE_MAX);
cudaError_t launch_forward(const slim_layer& L, const uint16_t* X, int M, uint16_t* Y, void* ws, bool allow_prefill,
                           size_t ws_limit, cudaStream_t s);

// Kernels one launch_forward call launches.
int forward_launches(const slim_layer& L, int M, bool allow_prefill, size_t ws_limit = SIZE_MAX);

// Gated block by streaming the weights once per 16 tokens; reads T = X L
// (row-major, [.][rl16]) of launch_adapter_down, which must be the kernel just
// before it when there is an adapter.  (A plan fits every layer the format
// allows; the query is for tests.)
bool gstream_fits(const slim_layer& L, int M);
cudaError_t launch_gstream(const slim_layer& L, const uint16_t* X, int M, const GatedOut& o, const uint16_t* T,
                           cudaStream_t s);

// Single-launch streaming decode (M <= 16).
bool stream_supported(const slim_layer& L, int M);
size_t stream_workspace_bytes(const slim_layer& L, int M);
cudaError_t launch_stream(const slim_layer& L, const uint16_t* X, int M, uint16_t* Y, void* ws, cudaStream_t s);
// The same with the budget of the waits for T partials in SM cycles, and
// readers that expect the tag of launch seq + tag_skew (a test aid: with
// tag_skew = 1 no CTA writes what they wait for, so every wait gives up).
cudaError_t launch_stream_ex(const slim_layer& L, const uint16_t* X, int M, uint16_t* Y, void* ws,
                             long long t_wait_cycles, uint32_t tag_skew, cudaStream_t s);

// Bytes of the pre-swizzled R^T image: 128-row tiles x ceil(r16/64) atoms,
// padded to whole 512-row blocks (the largest prefill CTA-pair tile).
inline size_t rp_bytes(int N, int r16) {
  return r16 > 0 ? (size_t)((N + 511) / 512) * 4 * 128 * (size_t)((r16 + 63) / 64) * 64 * 2 : 0;
}
cudaError_t launch_pack_rp(const slim_layer& L, const uint16_t* Rsrc, cudaStream_t s);
cudaError_t launch_pack_lp(const slim_layer& L, const uint16_t* Lsrc, cudaStream_t s);
// T = X L on the tensor cores into the prefill kernel's swizzled T tiles.
// (tiles of `tt` tokens).
cudaError_t launch_tgemm(const slim_layer& L, const uint16_t* X, int M, int tt, uint16_t* Tswz, cudaStream_t s);

// Tensor-core prefill forward (M > 16): the dequantized weight images go to
// `img` (prefill_image_bytes(N, K) bytes of workspace).
int prefill_tokens_per_tile(const slim_layer& L, int M, bool gated = false);
constexpr int kPrefillMaxTile = 240;   // widest token tile of the prefill kernels
size_t prefill_image_bytes(int N, int K);
cudaError_t launch_prefill(const slim_layer& L, const uint16_t* X, int M, const GatedOut& o, const uint16_t* Tswz,
                           uint8_t* img, cudaStream_t s);

// Gated feed-forward block H = act(G) U on a layer of two equal fused
// linears; GU (G and U side by side, [M][2F]) is written too when not null.
size_t gated_workspace_bytes(const slim_layer& L, int M);
int gated_launches(const slim_layer& L, int M);
cudaError_t launch_gated(const slim_layer& L, const uint16_t* X, int M, int act, uint16_t* H, uint16_t* GU, void* ws,
                         cudaStream_t s, long long fail_cycles = 0);

// Backward pass of the linears (dY) or, with dY null, of the gated block (GU,
// dH, act); null outputs are not computed.
size_t backward_workspace_bytes(const slim_layer& L, int M);
cudaError_t launch_backward(const slim_layer& L, const uint16_t* X, const uint16_t* dY, const uint16_t* GU,
                            const uint16_t* dH, int act, int M, uint16_t* dX, uint16_t* dL, uint16_t* dR, void* ws,
                            cudaStream_t s);

// Dense 4-bit linear.
size_t w4_dec_bytes(int K, int N, int group);
size_t w4_workspace_bytes(const slim_w4_layer& L, int M);
int w4_launches(const slim_w4_layer& L, int M);
void w4_split(const slim_w4_layer& L, int M, int32_t* plan);   // see slim_w4_plan
cudaError_t launch_w4_pack(const slim_w4_layer& L, const uint16_t* W, cudaStream_t s);
cudaError_t launch_w4_unpack(const slim_w4_layer& L, int8_t* q, uint16_t* scales, cudaStream_t s);
cudaError_t launch_w4(const slim_w4_layer& L, const uint16_t* X, int M, uint16_t* Y, void* ws, cudaStream_t s);

int max_clusters(const void* func, cudaLaunchConfig_t cfg);
// Number of SMs of the current device (cached per device).
int num_sms();
// Compute-capability major of the current device (cached per device; -1 on error).
int device_cc_major();
// Test aid: a one-thread wait on a barrier nothing completes, bounded by
// about wait_us of SM clock (at most the forward's wait budget); records
// SLIM_ERR_TIMEOUT in `status`.
cudaError_t launch_wait_probe(int32_t* status, int wait_us, cudaStream_t s);
// Raise `func`'s dynamic shared-memory limit to at least `smem` bytes (and
// allow cluster sizes above 8 when asked) on the current device.  Function
// attributes belong to a (kernel, device); what was set is remembered per
// pair under a lock, so concurrent first calls from several host threads,
// or one thread driving several GPUs, each get them set.
cudaError_t ensure_func_attrs(const void* func, size_t smem, bool nonportable_cluster = false);

}  // namespace slim
