// Backward pass of the compressed linear and of the gated feed-forward block.
//
// The packed 4-bit 2:4 weight is frozen (thesis Fig. 7.1: the adapters may be
// fine-tuned with the compressed weight fixed); gradients go to X and to the
// adapter factors.  For Y_g = X W_g^T + (X L_g) R_g over the fused linears g:
//
//   dT_g = dY_g R_g^T                 [M][r]
//   dX   = dY W + sum_g dT_g L_g^T    [M][K]
//   dL_g = X^T dT_g                   [K][r]
//   dR_g = (X L_g)^T dY_g             [r][N_g]
//
// and for the gated block H = act(G) U, from the saved G and U,
//   dG = dH U act'(G),  dU = dH act(G)  as dY.
//
// dX sums over N, across which the weight has no 2:4 structure (the pairs lie
// along K), so it is a dense product of 2 M N K operations on tcgen05.  For few
// tokens the weight is expanded inside that product (slim_qgemm.cu); for more
// it is expanded once per call to bf16 [N][K] (the rounding of q * s to bf16 is
// the prefill path's) and multiplied by slim_gemm.cu.  The
// adapter's factors are read from the packed layer's operand images.
//
// Roundings to bf16 besides the outputs: dG and dU (tensor-core operands of
// three products; rounding them once lets all three read 16 bits), T = X L
// and dT (as the forward rounds T), q * s.  All sums are fp32.
#include <algorithm>

#include "slim_act.cuh"
#include "slim_common.cuh"
#include "slim_gemm.h"
#include "slim_internal.h"
#include "slim_qgemm.h"

namespace slim {
namespace {

size_t a1k(size_t x) { return (x + 1023) / 1024 * 1024; }

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// dY [M][2F] = [dH U act'(G), dH act(G)] from GU [M][2F] and dH [M][F]; 8
// columns per thread.  Bound by HBM: 10 bytes per element of dH (2048 x 11008
// in 35 us).
__device__ __forceinline__ void gate_bwd(int block, int blocks, const uint4* __restrict__ GU,
                                         const uint4* __restrict__ dH, int act, int F8, size_t total,
                                         uint4* __restrict__ dY) {
  for (size_t e = (size_t)block * 256 + threadIdx.x; e < total; e += (size_t)blocks * 256) {
    const size_t m = e / F8, c = e % F8;
    const uint4 gv = GU[m * 2 * F8 + c], uv = GU[m * 2 * F8 + F8 + c], hv = dH[e];
    const uint32_t g[4] = {gv.x, gv.y, gv.z, gv.w}, u[4] = {uv.x, uv.y, uv.z, uv.w}, h[4] = {hv.x, hv.y, hv.z, hv.w};
    uint32_t og[4], ou[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float a0, d0, a1, d1;
      act_both(act, bf_lo(g[q]), a0, d0);
      act_both(act, bf_hi(g[q]), a1, d1);
      const float h0 = bf_lo(h[q]), h1 = bf_hi(h[q]);
      og[q] = pack_bf(h0 * bf_lo(u[q]) * d0, h1 * bf_hi(u[q]) * d1);
      ou[q] = pack_bf(h0 * a0, h1 * a1);
    }
    dY[m * 2 * F8 + c] = make_uint4(og[0], og[1], og[2], og[3]);
    dY[m * 2 * F8 + F8 + c] = make_uint4(ou[0], ou[1], ou[2], ou[3]);
  }
}

// Rows of an odd N moved to a pitch a tensor copy can read (a multiple of 16
// bytes), 8 columns per thread; the columns past N are never read.  NaN is made
// quiet, as arithmetic would: nothing in a workspace may look like the tags of
// launch_tag().
__device__ __forceinline__ void pad_rows(int block, int blocks, const uint16_t* __restrict__ src, int N, int P8,
                                         size_t total, uint4* __restrict__ dst) {
  for (size_t e = (size_t)block * 256 + threadIdx.x; e < total; e += (size_t)blocks * 256) {
    const size_t m = e / P8;
    const int c = (int)(e - m * P8) * 8;
    const uint16_t* from = src + m * N + c;
    uint32_t o[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      o[q] = c + q < N ? __ldg(from + q) : 0u;
      if ((o[q] & 0x7FFFu) > 0x7F80u) o[q] |= 0x40u;
    }
    dst[e] = make_uint4(o[0] | o[1] << 16, o[2] | o[3] << 16, o[4] | o[5] << 16, o[6] | o[7] << 16);
  }
}

// Canonical packed weight -> dense bf16 [N][K], zeros at the pruned places.  A
// CTA stages the packed bytes of 16384 columns (6.4 KB, wide loads), then each
// thread expands 8 columns (2 groups of 4, 16 bytes) at a time, so that every
// store is a whole line.  The integers come from the mantissa of 2^23 + u; one
// byte permutation per pair of columns places the two kept values, its
// selectors from a table of the 16 metadata nibbles.  Bound by HBM (0.39 bytes
// read and 2 written per weight) and by the integer pipe about equally: 22016
// x 4096 in 35 us.
constexpr int kExpPieces = 2048;     // pieces of 8 columns a CTA expands at a time
__device__ __forceinline__ void expand(int block, int blocks, const uint4* __restrict__ vals,
                                       const uint4* __restrict__ meta, const uint4* __restrict__ scales, size_t total,
                                       uint4* __restrict__ W) {
  __shared__ __align__(16) uint16_t vs[kExpPieces];
  __shared__ __align__(16) uint8_t ms[kExpPieces];
  __shared__ __align__(16) __half ss[kExpPieces / 16];
  __shared__ uint32_t place[16];
  const int t = threadIdx.x;
  // Bytes of columns 0 .. 3 out of (pair, 0): 4 is a zero byte, the kept
  // columns i0 and i1 (nibble i0 | i1 << 2) get bytes 1, 0 and 3, 2.
  if (t < 16) place[t] = 0x44444444u ^ (0x54u << ((t & 3) * 8)) ^ (0x76u << ((t >> 2) * 8));
  for (size_t b0 = (size_t)block * kExpPieces; b0 < total; b0 += (size_t)blocks * kExpPieces) {
    // 16 bytes of vals, meta, scales serve 8, 16, 128 pieces (a row has a
    // multiple of 16; the last 16 bytes of scales may reach into the padding of
    // their region, whose size is a multiple of 256).
    const int n = (int)min((size_t)kExpPieces, total - b0);
    if (t * 8 < n) reinterpret_cast<uint4*>(vs)[t] = __ldg(vals + b0 / 8 + t);
    if (t < 128) {
      if (t * 16 < n) reinterpret_cast<uint4*>(ms)[t] = __ldg(meta + b0 / 16 + t);
    } else if (t < 128 + kExpPieces / 128) {
      if ((t - 128) * 128 < n) reinterpret_cast<uint4*>(ss)[t - 128] = __ldg(scales + b0 / 128 + (t - 128));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kExpPieces / 256; ++i) {
      const int e = i * 256 + t;
      if (e >= n) break;
      const uint32_t v = (uint32_t)vs[e] ^ 0x8888u;   // nibbles u = q + 8
      const uint32_t mt = ms[e];
      const float s = __half2float(ss[e >> 4]);
      uint32_t o[4];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float f0 = (__uint_as_float(0x4B000000u | ((v >> (8 * q)) & 15u)) - 8388616.f) * s;
        const float f1 = (__uint_as_float(0x4B000000u | ((v >> (8 * q + 4)) & 15u)) - 8388616.f) * s;
        const uint32_t pr = pack_bf(f0, f1), sel = place[(mt >> (4 * q)) & 15u];
        o[2 * q] = __byte_perm(pr, 0u, sel);
        o[2 * q + 1] = __byte_perm(pr, 0u, sel >> 16);
      }
      W[b0 + e] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    __syncthreads();
  }
}

// What the products read and the caller does not have: dY (gate_bwd, pad_rows,
// or the caller's own) by the first n_y CTAs, the expanded weight by the
// others, side by side in one launch.
struct PrepareParams {
  const uint4* GU;
  const uint4* dH;
  const uint16_t* dY;
  uint16_t* y;
  int act, N, pitch;
  size_t y_total;
  int n_y;
  const uint4* vals;
  const uint4* meta;
  const uint4* scales;
  uint4* W;
  size_t w_total;
};
__global__ void __launch_bounds__(256) k_prepare(const PrepareParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.x, n_w = gridDim.x - p.n_y;
  if (b >= p.n_y) expand(b - p.n_y, n_w, p.vals, p.meta, p.scales, p.w_total, p.W);
  else if (p.GU) gate_bwd(b, p.n_y, p.GU, p.dH, p.act, p.N / 16, p.y_total, reinterpret_cast<uint4*>(p.y));
  else pad_rows(b, p.n_y, p.dY, p.N, p.pitch / 8, p.y_total, reinterpret_cast<uint4*>(p.y));
}

// Workspace map.  The first kilobyte is left alone (the decode kernel's
// control block lives there when a forward shares the workspace).
struct BwdWs {
  size_t dY, T, dT, W, total;
};
BwdWs bwd_ws(const slim_layer& L, int M) {
  BwdWs w;
  size_t off = 1024;
  const size_t m = (size_t)std::max(M, 1);
  w.dY = off;   off += a1k(m * ((L.N + 7) / 8 * 8) * 2);
  w.T = off;    off += a1k(m * L.rl16 * 2);
  w.dT = off;   off += a1k(m * L.rl16 * 2);
  w.W = off;    off += qgemm_pays(M, L.K) ? 0 : a1k((size_t)L.N * L.K * 2);
  w.total = off;
  return w;
}

}  // namespace

size_t backward_workspace_bytes(const slim_layer& L, int M) { return bwd_ws(L, M).total; }

// dY not null: the linear's output gradient.  Else GU, dH and act: the gated
// block's.  dX, dL, dR: the wanted gradients (null: not computed).
cudaError_t launch_backward(const slim_layer& L, const uint16_t* X, const uint16_t* dY, const uint16_t* GU,
                            const uint16_t* dH, int act, int M, uint16_t* dX, uint16_t* dL, uint16_t* dR, void* ws,
                            cudaStream_t s) {
  NvtxRange nv("backward");
  uint8_t* wb = static_cast<uint8_t*>(ws);
  const BwdWs w = bwd_ws(L, M);
  const int K = L.K, N = L.N, N8 = (N + 7) / 8 * 8;
  cudaError_t e;
  // Kernels of this call in launch order.  One that waits for its predecessor
  // at its start (`last`: the latest such) sees everything launched before it
  // complete; one whose inputs all come from before that may start early.
  const bool packed = dX && qgemm_pays(M, K);   // dX straight from the packed weight
  int n = 0, last = -1, at_y = -1, at_T = -1, at_dT = -1, at_W = -1;
  uint16_t* W = reinterpret_cast<uint16_t*>(wb + w.W);
  const uint16_t* y = dY;
  int ldy = N;
  {
    // CTAs: up to 16 per SM for each of the two.
    auto blocks = [](size_t work, size_t per) {
      return (int)std::min((work + per - 1) / per, (size_t)num_sms() * 16);
    };
    PrepareParams p = {};
    if (!dY || N != N8) {
      p.y = reinterpret_cast<uint16_t*>(wb + w.dY);
      p.GU = reinterpret_cast<const uint4*>(GU);
      p.dH = reinterpret_cast<const uint4*>(dH);
      p.dY = dY;
      p.act = act;
      p.N = N;
      p.pitch = N8;
      p.y_total = dY ? (size_t)M * (N8 / 8) : (size_t)M * (N / 16);
      p.n_y = blocks(p.y_total, 256);
      y = p.y;
      ldy = N8;
      at_y = n;
    }
    int n_w = 0;
    if (dX && !packed) {
      p.vals = reinterpret_cast<const uint4*>(L.vals);
      p.meta = reinterpret_cast<const uint4*>(L.meta);
      p.scales = reinterpret_cast<const uint4*>(L.scales);
      p.W = reinterpret_cast<uint4*>(W);
      p.w_total = (size_t)N * (K / 8);
      n_w = blocks(p.w_total, kExpPieces);
      at_W = n;
    }
    if (p.n_y + n_w > 0) {
      NvtxRange nr("backward: dY and the expanded weight (k_prepare)");
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)(p.n_y + n_w));
      cfg.blockDim = dim3(256);
      cfg.stream = s;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaLaunchKernelEx(&cfg, k_prepare, p);
      if (e != cudaSuccess) return e;
      last = n++;
    }
  }
  GemmCall base;
  base.n_groups = L.n_groups;
  for (int g = 0; g < SLIM_MAX_GROUPS; ++g) base.group_end[g] = L.group_end[g];
  base.r16 = L.r16;
  base.status = L.status;
  auto rowmajor = [](const void* p, long long rows, long long c, long long pitch) {
    GemmOperand o;
    o.base = p;
    o.layout = GemmLayout::kRowMajor;
    o.rows = rows;
    o.c = c;
    o.pitch = pitch;
    return o;
  };
  auto colmajor = [&](const void* p, long long rows, long long c, long long pitch) {
    GemmOperand o = rowmajor(p, rows, c, pitch);
    o.layout = GemmLayout::kColMajor;
    return o;
  };
  uint16_t* T = reinterpret_cast<uint16_t*>(wb + w.T);
  uint16_t* dT = reinterpret_cast<uint16_t*>(wb + w.dT);
  const int r64 = ceil_div(L.r16, 64) * 64;
  // L^T as images: line (k / 64) * rl16 + j holds column j of L at 64 k, an
  // MN-major tile for a product over j, a K-major one for a product over k.
  GemmOperand lt;
  lt.base = L.Lp;
  lt.layout = GemmLayout::kImage;
  lt.rows = K;
  lt.c = L.rl16;
  lt.blk_lines = L.rl16;
  lt.img_lines = (long long)K / 64 * L.rl16;
  GemmCall gT = base, gdT = base, gdX = base, gdL = base, gdR = base;
  if (L.r16 > 0) {
    gT.I = M;             // T = X L
    gT.J = L.rl16;
    gT.a[0] = rowmajor(X, M, K, K);
    gT.b[0] = lt;
    gT.b[0].layout = GemmLayout::kImageK;
    gT.b[0].rows = L.rl16;
    gT.b[0].c = K;
    gT.C = T;
    gT.ldc = L.rl16;
    gdT.mode = GemmMode::kGroupC;   // dT_g = dY_g R_g^T
    gdT.I = M;
    gdT.J = L.r16;
    gdT.a[0] = rowmajor(y, M, N, ldy);
    gdT.b[0].base = L.Rp;
    gdT.b[0].layout = GemmLayout::kImage;
    gdT.b[0].rows = r64;
    gdT.b[0].c = N;
    gdT.b[0].blk_lines = 128;
    gdT.b[0].cblk_lines = r64 / 64 * 128;
    gdT.b[0].img_lines = (long long)ceil_div(N, 512) * 4 * (r64 / 64) * 128;
    gdT.C = dT;
    gdT.ldc = L.rl16;
    gdL.I = K;            // dL = X^T dT
    gdL.J = L.rl16;
    gdL.a[0] = colmajor(X, K, M, K);
    gdL.b[0] = colmajor(dT, L.rl16, M, L.rl16);
    gdL.C = dL;
    gdL.ldc = L.n_groups * L.r;
    gdL.jb = L.r16;
    gdL.jr = L.r;
    gdR.mode = GemmMode::kGroupJ;   // dR_g = T_g^T dY_g
    gdR.I = L.r;
    gdR.J = N;
    gdR.a[0] = colmajor(T, L.rl16, M, L.rl16);
    gdR.b[0] = colmajor(y, N, M, ldy);
    gdR.C = dR;
    gdR.ldc = N;
  }
  gdX.I = M;              // dX = dY W + dT L^T
  gdX.J = K;
  gdX.a[0] = rowmajor(y, M, N, ldy);
  gdX.b[0] = colmajor(W, K, N, K);
  if (L.r16 > 0) {
    gdX.nseg = 2;
    gdX.a[1] = rowmajor(dT, M, L.rl16, L.rl16);
    gdX.b[1] = lt;
  }
  gdX.C = dX;
  gdX.ldc = K;

  // Products that fit together share a launch.
  struct Wanted {
    const GemmCall* g;
    int* out;                 // launch index of what it writes for later ones (or null)
    int* in[3];               // launch indices of what wrote its inputs (null: nothing in this call)
  };
  auto run = [&](const Wanted* w, int count) -> cudaError_t {
    GemmCall batch[kGemmBatch];
    bool early = last >= 0;
    for (int q = 0; q < count; ++q) {
      batch[q] = *w[q].g;
      for (int* i : w[q].in) early = early && (!i || *i < last);
    }
    if (!early) last = n;
    for (int q = 0; q < count; ++q)
      if (w[q].out) *w[q].out = n;
    ++n;
    return launch_gemms(batch, count, early, s);
  };
  auto run_all = [&](const Wanted* w, int count) -> cudaError_t {
    GemmCall batch[kGemmBatch];
    for (int q = 0; q < count; ++q) batch[q] = *w[q].g;
    if (count > 1 && gemms_fit_together(batch, count)) return run(w, count);
    cudaError_t err = cudaSuccess;
    for (int q = 0; q < count && err == cudaSuccess; ++q) err = run(w + q, 1);
    return err;
  };
  Wanted first[2], then[3];
  int n1 = 0, n2 = 0;
  if (L.r16 > 0 && dR) first[n1++] = {&gT, &at_T, {nullptr, nullptr, nullptr}};
  if (L.r16 > 0 && (dX || dL)) first[n1++] = {&gdT, &at_dT, {&at_y, nullptr, nullptr}};
  if (dX && !packed) then[n2++] = {&gdX, nullptr, {&at_y, &at_W, &at_dT}};
  if (dL) then[n2++] = {&gdL, nullptr, {&at_dT, nullptr, nullptr}};
  if (dR) then[n2++] = {&gdR, nullptr, {&at_T, &at_y, nullptr}};
  e = run_all(first, n1);
  if (e != cudaSuccess) return e;
  if (packed) {
    QGemmCall q;
    q.I = M;
    q.J = K;
    q.c = N;
    q.A = y;
    q.lda = ldy;
    q.C = dX;
    q.ldc = K;
    q.status = L.status;
    q.vals = L.vals;
    q.meta = L.meta;
    q.scales = L.scales;
    if (L.r16 > 0) {
      q.A2 = dT;
      q.B2 = L.Lp;
      q.c2 = L.rl16;
    }
    const bool early = last >= 0 && at_y < last && at_dT < last;
    if (!early) last = n;
    ++n;
    e = launch_qgemm(q, early, s);
    if (e != cudaSuccess) return e;
  }
  // All the rest at once, or dX by itself and the adapters' gradients in the
  // SMs its last wave leaves idle.
  GemmCall rest[3];
  for (int q = 0; q < n2; ++q) rest[q] = *then[q].g;
  if (n2 == 3 && gemms_fit_together(rest, 3)) return run(then, 3);
  if (n2 == 3) {
    e = run(then, 1);
    return e != cudaSuccess ? e : run_all(then + 1, 2);
  }
  return run_all(then, n2);
}

}  // namespace slim
