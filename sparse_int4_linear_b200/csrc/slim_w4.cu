// Linear with dense 4-bit weights (quantized as the compressed layer's, not
// pruned): Y = X W^^T, W^ = q * s with one fp16 scale per row and group of
// 32, 64 or 128 consecutive k.
//
// Packed form: chunks of 16 rows x 128 K, row tile by row tile.  A chunk is
// 1024 bytes of biased nibbles u = q + 8 in the order of the m16n8k16 A
// fragment (one 32-bit word per lane and 16-k step; two 16-byte words per lane
// and chunk), then 16 rows' scales per group, rows g and g + 8 in one 32-bit
// word, the groups of a row pair side by side.
//
//   k_w4_pack    quantization and packing
//   k_w4         few tokens: streams the packed weight once per 16 tokens
//   k_qgemm      up to some hundred tokens (slim_qgemm.cu): expanded inside the
//                product
//   k_w4_expand  more: the weight as bf16 [N][K] for slim_gemm.cu
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "slim_common.cuh"
#include "slim_gemm.h"
#include "slim_internal.h"
#include "slim_qgemm.h"

namespace cg = cooperative_groups;

namespace slim {
namespace {

__host__ __device__ constexpr int w4_chunk(int group) { return 1024 + 32 * (128 / group); }

// ---------------------------------------------------------------- packing
// One CTA per chunk: warp w quantizes row w, lane l the values 4l .. 4l + 3
// (as k_pack: abs-max / 7 to fp16, round half to even, clip to +-7).
__global__ void __launch_bounds__(512) k_w4_pack(const uint16_t* __restrict__ W, int K, int N, int group,
                                                 uint8_t* __restrict__ dec, int32_t* status) {
  __shared__ uint32_t chunk[(1024 + 32 * 4) / 4];
  const int NG = 128 / group, bytes = w4_chunk(group);
  const int rt = blockIdx.x, ck = blockIdx.y;
  const int row = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < bytes / 4; i += blockDim.x) chunk[i] = 0u;
  __syncthreads();
  const int n = rt * 16 + row;
  const bool valid = n < N;
  float w[4] = {0.f, 0.f, 0.f, 0.f};
  if (valid) {
    const uint2 raw = *reinterpret_cast<const uint2*>(W + (size_t)n * K + (size_t)ck * 128 + lane * 4);
    w[0] = __uint_as_float(raw.x << 16);
    w[1] = __uint_as_float(raw.x & 0xFFFF0000u);
    w[2] = __uint_as_float(raw.y << 16);
    w[3] = __uint_as_float(raw.y & 0xFFFF0000u);
  }
  float amax = fmaxf(fmaxf(fabsf(w[0]), fabsf(w[1])), fmaxf(fabsf(w[2]), fabsf(w[3])));
  uint32_t nan = isnan(w[0]) || isnan(w[1]) || isnan(w[2]) || isnan(w[3]);
  // The group's lanes are consecutive: 8, 16 or 32 of them.
  for (int o = group / 8; o > 0; o >>= 1) {
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    nan |= __shfl_xor_sync(0xffffffffu, nan, o);
  }
  const __half s16 = __float2half_rn(__fdiv_rn(amax, 7.0f));
  const float sf = __half2float(s16);
  const bool bad = nan || isinf(sf);
  if (valid && bad) record_status(status, SLIM_ERR_RANGE);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int q = 0;
    if (valid && !bad && sf != 0.f) q = (int)fminf(fmaxf(rintf(__fdiv_rn(w[i], sf)), -7.f), 7.f);
    const int k = lane * 4 + i, j = k >> 4;
    atomicOr(&chunk[(j >> 2) * 128 + frag_lane(row, k & 15) * 4 + (j & 3)], (uint32_t)(q + 8) << frag_shift(row, k & 15));
  }
  if (lane % (group / 4) == 0 && valid && !bad)
    atomicOr(&chunk[256 + (row & 7) * NG + lane / (group / 4)],
             (uint32_t)__half_as_ushort(s16) << (16 * (row >> 3)));
  __syncthreads();
  uint32_t* out = reinterpret_cast<uint32_t*>(dec + ((size_t)rt * (K / 128) + ck) * bytes);
  for (int i = threadIdx.x; i < bytes / 4; i += blockDim.x) out[i] = chunk[i];
}

__global__ void k_w4_done() {}

// Packed -> int8 q [N][K] and fp16 scales [N][K/group].
__global__ void __launch_bounds__(256) k_w4_unpack(const uint8_t* __restrict__ dec, int K, int N, int group,
                                                   int8_t* __restrict__ q, uint16_t* __restrict__ scales) {
  const size_t e = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= (size_t)N * K) return;
  const int n = (int)(e / K), k = (int)(e % K), row = n & 15, kk = k & 127, j = kk >> 4, NG = 128 / group;
  const uint8_t* ch = dec + ((size_t)(n >> 4) * (K / 128) + (k >> 7)) * w4_chunk(group);
  const uint32_t w = reinterpret_cast<const uint32_t*>(ch)[(j >> 2) * 128 + frag_lane(row, kk & 15) * 4 + (j & 3)];
  q[e] = (int8_t)((int)((w >> frag_shift(row, kk & 15)) & 15u) - 8);
  if (k % group == 0) {
    const uint32_t s = reinterpret_cast<const uint32_t*>(ch + 1024)[(row & 7) * NG + kk / group];
    scales[(size_t)n * (K / group) + k / group] = (uint16_t)(s >> (16 * (row >> 3)));
  }
}

// Packed -> bf16(q * s) [N][K] (the prefill path's rounding).  A warp expands
// one chunk: each lane its words (of 16 rows x 128 K), through shared memory
// so that rows are written in whole lines of 256 bytes.  Bound by HBM: 0.5
// bytes read and 2 written per weight (4096 x 11008 in 24 us).
__global__ void __launch_bounds__(256) k_w4_expand(const uint8_t* __restrict__ dec, int NCK, size_t chunks, int K, int N,
                                                   int group, uint16_t* __restrict__ W) {
  __shared__ __align__(16) uint32_t ts[8][16][68];   // 128 bf16 a row, padded
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3, NG = 128 / group;
  uint32_t(*t)[68] = ts[threadIdx.x >> 5];
  for (size_t i = (size_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < chunks; i += (size_t)gridDim.x * 8) {
    const uint8_t* ch = dec + i * w4_chunk(group);
    const uint4 va = __ldg(reinterpret_cast<const uint4*>(ch) + lane), vb = __ldg(reinterpret_cast<const uint4*>(ch) + 32 + lane);
    const uint32_t w[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 s = __half22float2(reinterpret_cast<const __half2*>(ch + 1024)[g * NG + j * 16 / group]);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float sc = (p & 1) ? s.y : s.x;
        const __nv_bfloat162 o =
            __floats2bfloat162_rn((__uint_as_float(0x4B000000u | ((w[j] >> (4 * p)) & 15u)) - 8388616.f) * sc,
                                  (__uint_as_float(0x4B000000u | ((w[j] >> (16 + 4 * p)) & 15u)) - 8388616.f) * sc);
        t[g + 8 * (p & 1)][j * 8 + tq + 4 * (p >> 1)] = *reinterpret_cast<const uint32_t*>(&o);
      }
    }
    __syncwarp();
    const int rt = (int)(i / NCK), ck = (int)(i % NCK);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int row = q * 2 + (lane >> 4), c = lane & 15, n = rt * 16 + row;
      if (n < N)
        *reinterpret_cast<uint4*>(W + (size_t)n * K + (size_t)ck * 128 + c * 8) =
            *reinterpret_cast<const uint4*>(&t[row][c * 4]);
    }
    __syncwarp();
  }
}

// ---------------------------------------------------------------- few tokens
// A CTA owns a range of row tiles and, in a cluster of S, a range of K, which
// it takes in panels whose X fits shared memory (one panel where possible).
// The panel's chunks, tile by tile, are cut into 16 contiguous ranges, one a
// warp: no warp waits for another while it streams, whatever the shape.  A
// warp streams its range through its own ring of bulk copies (stages of up to
// 4 chunks, 2 with more than 8 tokens), expands the nibbles to exact bf16
// integers, multiplies on the tensor cores with the staged X and scales each
// group's sum in fp32; leaving a row tile it keeps the sums it has of it (a
// segment) in shared memory.  Behind one barrier the CTA adds each tile's
// segments in warp order, then the panels, then the S ranks in rank order
// through distributed shared memory: every sum has a fixed order.
//
// Bound by HBM for large layers; the nibbles' expansion (56 integer and 32
// bf16 instructions per chunk and lane) comes next, so the loop around it is
// kept short: copies are issued per stage, every offset is a constant (150
// warp instructions a chunk).  B200, cold L2: 8192 x 28672, group 128, one token
// 29 us = 4.2 TB/s, 24.4 us without the expansion; 16 tokens 49 us; 4096 x
// 4096, group 64, four tokens 5.4 us.
constexpr int kW4Warps = 16;
__host__ __device__ constexpr int w4_stage_chunks(int NT) { return NT == 1 ? 4 : 2; }
constexpr int kW4Stages = 3;       // ring stages a warp has at most
constexpr int kTokStride = 20;     // floats between tokens of a partial tile (16 rows + padding)

struct W4Params {
  const uint16_t* X;
  uint16_t* Y;
  const uint8_t* dec;
  int M, K, N, NRT, NCK;
  int nst;             // ring stages
  int G;               // CTAs along the row tiles
  int P, ckp;          // panels of a rank's K, chunks of a panel (the last ones may have fewer)
  int tmax;            // row tiles of the largest CTA
  int32_t* status;
};

struct W4Smem {
  size_t xs, ring, part, sums, bars, who, total;
};
__host__ __device__ inline W4Smem w4_smem(int slot, int xrows, int ckp, int nst, int tmax, bool keep) {
  W4Smem m;
  size_t off = 0;
  m.ring = off; off += (size_t)kW4Warps * nst * slot;
  m.bars = off; off += (size_t)(kW4Warps * kW4Stages + 2) * 8;   // the rings', X's
  m.who = off;  off += (size_t)(tmax * 8 + 15) / 16 * 16;        // first and last warp of a tile
  m.part = off; off += (size_t)(tmax + kW4Warps) * xrows * kTokStride * 4;
  m.sums = off; off += keep ? (size_t)tmax * xrows * 16 * 4 : 0;
  m.xs = off;   off += (size_t)xrows * (ckp * 128 + 8) * 2;
  m.total = off;
  return m;
}

// m16n8k16 with zero sums to start from.
__device__ __forceinline__ void mma_16816_z(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
}
template <int OFF>
__device__ __forceinline__ uint32_t lds32_so(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1+%2];" : "=r"(v) : "r"(a), "n"(OFF));
  return v;
}

// acc += scaled sums of chunk C of a stage.  wl: the lane's words of the
// stage, sl: its scales', x0 / x1: its X rows at the stage's first k.
template <int NT, int NG, int C>
__device__ __forceinline__ void w4_chunk_mma(float (&acc)[NT][4], uint32_t wl, uint32_t sl, uint32_t x0, uint32_t x1) {
  constexpr int CHUNK = w4_chunk(128 / NG);
  const uint4 va = lds128_so<C * CHUNK>(wl), vb = lds128_so<C * CHUNK + 512>(wl);
  const uint32_t vw[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
  uint32_t sc[4];
  if (NG == 1) {
    sc[0] = lds32_so<C * CHUNK>(sl);
  } else if (NG == 2) {
    lds64_so<C * CHUNK>(sl, sc[0], sc[1]);
  } else {
    const uint4 v = lds128_so<C * CHUNK>(sl);
    sc[0] = v.x; sc[1] = v.y; sc[2] = v.z; sc[3] = v.w;
  }
  float pt[NG][NT][4];
  auto step = [&](auto jc) {      // 16-k steps j and j + 1
    constexpr int j = decltype(jc)::value * 2, q = j * NG / 8;
    constexpr bool first = j % (8 / NG) == 0;     // of its group
    uint32_t b0[4], b1[4], a[4];
    ldmatrix_x4_so<C * 256 + j * 32>(b0, x0);
    if (NT == 2) ldmatrix_x4_so<C * 256 + j * 32>(b1, x1);
    decode_word(vw[j], a);
    const uint4 a0 = make_uint4(a[0], a[1], a[2], a[3]);
    if (first) {
      mma_16816_z(pt[q][0], a0, b0[0], b0[1]);
      if (NT == 2) mma_16816_z(pt[q][NT - 1], a0, b1[0], b1[1]);
    } else {
      mma_16816(pt[q][0], a0, b0[0], b0[1]);
      if (NT == 2) mma_16816(pt[q][NT - 1], a0, b1[0], b1[1]);
    }
    decode_word(vw[j + 1], a);
    const uint4 a1 = make_uint4(a[0], a[1], a[2], a[3]);
    mma_16816(pt[q][0], a1, b0[2], b0[3]);
    if (NT == 2) mma_16816(pt[q][NT - 1], a1, b1[2], b1[3]);
  };
  step(std::integral_constant<int, 0>());
  step(std::integral_constant<int, 1>());
  step(std::integral_constant<int, 2>());
  step(std::integral_constant<int, 3>());
#pragma unroll
  for (int q = 0; q < NG; ++q) {
    const float2 sf = __half22float2(*reinterpret_cast<const __half2*>(&sc[q]));
    const float lo = sf.x, hi = sf.y;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      acc[n][0] = fmaf(lo, pt[q][n][0], acc[n][0]);
      acc[n][1] = fmaf(lo, pt[q][n][1], acc[n][1]);
      acc[n][2] = fmaf(hi, pt[q][n][2], acc[n][2]);
      acc[n][3] = fmaf(hi, pt[q][n][3], acc[n][3]);
    }
  }
}

// Outputs n and n + 1 (n even) of one token.
__device__ __forceinline__ void store_w4(const W4Params& p, int tok, int n, float y0, float y1) {
  if (!dcheck(tok < p.M, p.status)) return;
  uint16_t* yp = p.Y + (size_t)tok * p.N + n;
  if ((p.N & 1) == 0) {
    if (n < p.N) *reinterpret_cast<__nv_bfloat162*>(yp) = __floats2bfloat162_rn(y0, y1);
  } else {
    if (n < p.N) yp[0] = __bfloat16_as_ushort(__float2bfloat16_rn(y0));
    if (n + 1 < p.N) yp[1] = __bfloat16_as_ushort(__float2bfloat16_rn(y1));
  }
}

template <int NT, int NG>
__global__ void __launch_bounds__(kW4Warps * 32, 1) k_w4(const W4Params p) {
  constexpr int GROUP = 128 / NG, CHUNK = w4_chunk(GROUP), SC = w4_stage_chunks(NT), SLOT = SC * CHUNK;
  extern __shared__ __align__(128) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int S = gridDim.x, rank = blockIdx.x, cta = blockIdx.y, tok0 = blockIdx.z * 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int xrows = min(min(16, p.M - tok0), NT * 8), last = xrows - 1;
  const int ck0 = (int)((long long)rank * p.NCK / S), nck = (int)((long long)(rank + 1) * p.NCK / S) - ck0;
  const int t0 = (int)((long long)cta * p.NRT / p.G), nt = (int)((long long)(cta + 1) * p.NRT / p.G) - t0;
  const int nst = p.nst;
  const bool keep = S > 1 || p.P > 1;
  const W4Smem L = w4_smem(SLOT, xrows, p.ckp, nst, p.tmax, keep);
  uint16_t* Xs = reinterpret_cast<uint16_t*>(smem + L.xs);
  float* part = reinterpret_cast<float*>(smem + L.part);
  float* sums = reinterpret_cast<float*>(smem + L.sums);
  int2* who = reinterpret_cast<int2*>(smem + L.who);
  uint8_t* ring = smem + L.ring + (size_t)warp * nst * SLOT;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bars) + warp * kW4Stages;
  uint64_t* xbar = reinterpret_cast<uint64_t*>(smem + L.bars) + kW4Warps * kW4Stages;
  const int xrow = p.ckp * 128 + 8;
  // Warp w's range of a panel of nc chunks a tile starts here; warps without
  // a chunk come last.
  auto start = [&](int w, int nc) {
    const int C = nt * nc, W = min(kW4Warps, C);
    return w >= W ? C : (int)((long long)w * C / W);
  };

  // Copies run ahead of the products (i_*: the next stage's panel, tile,
  // chunk of the tile, and the range's end).  Stages end with their tile.
  int i_n = 0, i_pan = 0, i_rt = 0, i_c = 0, i_nc = 0, i_left = 0;
  auto open_panel = [&]() {
    for (i_left = 0; i_pan < p.P; ++i_pan) {
      i_nc = min(p.ckp, nck - i_pan * p.ckp);
      const int f0 = start(warp, i_nc);
      i_left = start(warp + 1, i_nc) - f0;
      i_rt = f0 / i_nc;
      i_c = f0 - i_rt * i_nc;
      if (i_left > 0) return;
    }
  };
  open_panel();
  auto issue = [&](int slot) {     // the next stage, if there is one
    if (i_left == 0) return;
    const int n = min(min(SC, i_left), i_nc - i_c);
    if (lane == 0 && dcheck(t0 + i_rt < p.NRT && ck0 + i_pan * p.ckp + i_c + n <= p.NCK, p.status)) {
      mbar_expect_tx(bars + slot, (uint32_t)(n * CHUNK));
      bulk_g2s(ring + slot * SLOT, p.dec + ((size_t)(t0 + i_rt) * p.NCK + ck0 + i_pan * p.ckp + i_c) * CHUNK,
               (uint32_t)(n * CHUNK), bars + slot);
    }
    ++i_n;
    i_left -= n;
    i_c += n;
    if (i_c == i_nc) {
      i_c = 0;
      ++i_rt;
    }
    if (i_left == 0) {
      ++i_pan;
      open_panel();
    }
  };
  if (lane == 0) {
    for (int i = 0; i < nst; ++i) mbar_init(bars + i, 1);
    if (warp == 0) mbar_init(xbar, 1);
    fence_mbar_init();
  }
  __syncwarp();
  // The packed weight is constant: start streaming before the wait, with one
  // stage a warp (more would keep X waiting behind it).
  issue(0);
  // X of a panel: one bulk copy per token row, by one thread.
  auto stage_x = [&](int pan) {
    const uint32_t bytes = (uint32_t)min(p.ckp, nck - pan * p.ckp) * 256u;
    const uint16_t* xp = p.X + (size_t)tok0 * p.K + (size_t)(ck0 + pan * p.ckp) * 128;
    mbar_expect_tx(xbar, bytes * (uint32_t)xrows);
    for (int tk = 0; tk < xrows; ++tk) bulk_g2s(Xs + tk * xrow, xp + (size_t)tk * p.K, bytes, xbar);
  };
  if (threadIdx.x == 0) {
    pdl_wait();
    stage_x(0);
  }
  __syncthreads();      // X's barrier is set up, and the previous grid has completed
  pdl_launch_dependents();
  for (int i = 1; i < nst; ++i) issue(i);

  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
  // Rows of X past the staged ones repeat the last (their products land in
  // outputs that are not stored).
  const uint32_t xs_s = smem_u32(Xs);
  const uint32_t xa0 = xs_s + (uint32_t)(min(lane & 7, last) * xrow + (lane >> 3) * 8) * 2u;
  const uint32_t xa1 = xs_s + (uint32_t)(min(8 + (lane & 7), last) * xrow + (lane >> 3) * 8) * 2u;

  const int pstride = xrows * kTokStride;                // floats of one segment
  const uint32_t ring_s = smem_u32(ring), bar_s = smem_u32(bars);
  const uint32_t wl0 = ring_s + lane * 16, sl0 = ring_s + 1024 + g * 4 * NG;
  bool ok = true;
  int it = 0, st = 0, gave_up = 0, gave_pan = 0;   // where a wait gave up: the stage, the panel
  uint32_t ph = 0;
  for (int pan = 0; pan < p.P; ++pan) {
    if (pan > 0) {
      __syncthreads();      // the last panel's X is no longer read
      if (threadIdx.x == 0 && ok) {
        fence_proxy_async_smem();
        stage_x(pan);
      }
    }
    if (ok && !__all_sync(0xffffffffu, mbar_wait(xbar, pan & 1))) {
      ok = false;
      gave_up = it;
      gave_pan = pan;
    }
    const int nc = min(p.ckp, nck - pan * p.ckp);
    const int f0 = start(warp, nc);
    int left = start(warp + 1, nc) - f0, lt = f0 / nc, c = f0 - lt * nc;
    // Segment of warp w and tile lt in slot lt + w: both grow along the stream.
    float* dst = part + (size_t)(lt + warp) * pstride;
    while (left > 0) {
      if (ok) {
        ok = __all_sync(0xffffffffu, mbar_wait_s(bar_s + st * 8, ph));
        if (!ok) {
          gave_up = it;
          gave_pan = pan;
        }
      }
      const int n = min(min(SC, left), nc - c);
      if (ok) {
        const uint32_t wl = wl0 + (uint32_t)(st * SLOT), sl = sl0 + (uint32_t)(st * SLOT);
        const uint32_t x0 = xa0 + (uint32_t)c * 256u, x1 = xa1 + (uint32_t)c * 256u;
        if (n == SC) {
          w4_chunk_mma<NT, NG, 0>(acc, wl, sl, x0, x1);
          w4_chunk_mma<NT, NG, 1>(acc, wl, sl, x0, x1);
          if (SC == 4) {
            w4_chunk_mma<NT, NG, 2>(acc, wl, sl, x0, x1);
            w4_chunk_mma<NT, NG, 3>(acc, wl, sl, x0, x1);
          }
        } else {
#pragma unroll 1
          for (int q = 0; q < n; ++q)
            w4_chunk_mma<NT, NG, 0>(acc, wl + q * CHUNK, sl + q * CHUNK, x0 + q * 256, x1 + q * 256);
        }
        __syncwarp();
        if (lane == 0) fence_proxy_async_smem();
        issue(st);
      }
      ++it;
      if (++st == nst) {
        st = 0;
        ph ^= 1u;
      }
      if (c == 0 && lane == 0) who[lt].x = warp;
      left -= n;
      c += n;
      if (c == nc && lane == 0) who[lt].y = warp;
      if (c == nc || left == 0) {
        // Leaving the tile: a segment whose copies never arrived is NaN, and
        // so is every output of its tile.
        c = 0;
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          const int tk = q * 8 + 2 * t;
          if (!ok) acc[q][0] = acc[q][1] = acc[q][2] = acc[q][3] = NAN;
          if (tk < xrows) {
            dst[tk * kTokStride + g] = acc[q][0];
            dst[tk * kTokStride + g + 8] = acc[q][2];
          }
          if (tk + 1 < xrows) {
            dst[(tk + 1) * kTokStride + g] = acc[q][1];
            dst[(tk + 1) * kTokStride + g + 8] = acc[q][3];
          }
          acc[q][0] = acc[q][1] = acc[q][2] = acc[q][3] = 0.f;
        }
        dst += pstride;
        ++lt;
      }
    }
    __syncthreads();
    // Two rows of one token and tile per thread.
    for (int e = threadIdx.x; e < nt * xrows * 8; e += kW4Warps * 32) {
      const int row = (e & 7) * 2, lt = (e >> 3) / xrows, tk = (e >> 3) - lt * xrows;
      float* sm = sums + ((size_t)lt * xrows + tk) * 16 + row;
      float y0 = pan > 0 ? sm[0] : 0.f, y1 = pan > 0 ? sm[1] : 0.f;
      const int2 ww = who[lt];
      const float* ps = part + (size_t)(lt + ww.x) * pstride + tk * kTokStride + row;
#pragma unroll 4
      for (int w = ww.x; w <= ww.y; ++w, ps += pstride) {
        const float2 v = *reinterpret_cast<const float2*>(ps);
        y0 += v.x;
        y1 += v.y;
      }
      if (S > 1 || pan + 1 < p.P) {
        sm[0] = y0;
        sm[1] = y1;
      } else {
        store_w4(p, tok0 + tk, (t0 + lt) * 16 + row, y0, y1);
      }
    }
  }
  if (!ok && lane == 0) {
    record_status(p.status, SLIM_ERR_TIMEOUT);
    // Let the copies issued and not consumed land before the CTA exits (X's
    // last one is that of the panel where warp 0, which issues them, stopped).
    const long long deadline = clock64() + kWaitBudgetCycles;
    if (warp == 0) drain_phase(xbar, gave_pan & 1, deadline);
    for (int i = gave_up; i < i_n; ++i) drain_phase(bars + i % nst, (i / nst) & 1, deadline);
  }
  if (S > 1) {
    cluster.sync();
    const int E = nt * xrows * 8;
    const int e0 = (int)((long long)rank * E / S), e1 = (int)((long long)(rank + 1) * E / S);
    for (int e = e0 + (int)threadIdx.x; e < e1; e += blockDim.x) {
      const int row = (e & 7) * 2, tk = (e >> 3) % xrows, lt = (e >> 3) / xrows;
      float y0 = 0.f, y1 = 0.f;
      for (int q = 0; q < S; ++q) {
        const float2 v = *reinterpret_cast<const float2*>(cluster.map_shared_rank(sums, q) +
                                                          ((size_t)lt * xrows + tk) * 16 + row);
        y0 += v.x;
        y1 += v.y;
      }
      store_w4(p, tok0 + tk, (t0 + lt) * 16 + row, y0, y1);
    }
    cluster.sync();
  }
}

// ---------------------------------------------------------------- host
constexpr size_t kW4SmemLimit = 220 * 1024;
// Up to 16 tokens the packed weight is streamed once; up to 32 it is streamed
// twice on layers of 2^23 weights or more (which keeps them exact: the product
// rounds q * s).  Measured, 32 tokens, streamed twice against expanded inside the
// product, us a call: 8192 x 28672 96.8 and 107.9, 4096 x 4096 13.6 and 15.3, 4096
// x 2048 10.6 and 12.3; the product would be shorter at 4096 x 11008, 29.0 and
// 24.8, 11008 x 4096, 34.1 and 29.8, 8192 x 8192, 42.1 and 33.7, 28672 x 8192,
// 127.6 and 98.9, and is below the limit: 2048 x 2048 9.7 and 8.5, 1024 x 4096 10.1
// and 6.8.
bool w4_few(const slim_w4_layer& L, int M) { return M <= 16 || (M <= 32 && (long long)L.N * L.K >= 8 << 20); }

struct W4Plan {
  int S = 1, nst = 1, G = 1, NT = 1, P = 1, ckp = 0, tmax = 0;
  size_t smem = 0;
};

W4Plan w4_plan_uncached(const slim_w4_layer& L, int M) {
  W4Plan best;
  const int nsm = num_sms(), NCK = L.K / 128, xr = std::min(M, 16);
  const int NT = xr > 8 ? 2 : 1, SC = w4_stage_chunks(NT), slot = SC * w4_chunk(L.group);
  for (int S = 1; S <= 8 && S <= NCK; S *= 2) {
    W4Plan pl;
    pl.S = S;
    pl.NT = NT;
    const int nck = ceil_div(NCK, S);
    // Few panels; rings of 3 stages, or 2, before more panels.
    for (pl.P = 1; pl.P <= nck && pl.smem == 0; ++pl.P) {
      pl.ckp = ceil_div(nck, pl.P);
      // (The shorter ranks, of NCK / S chunks, have one of the last panel too.)
      if (ceil_div(nck, pl.ckp) != pl.P || (pl.P - 1) * pl.ckp >= NCK / S) continue;
      // Row tiles of a CTA: an even share of the SMs, but no more than 32 (the
      // segments and sums kept in shared memory).
      const bool keep = S > 1 || pl.P > 1;
      pl.G = std::max(std::min(L.n_row_tiles, std::max(1, nsm / S)), ceil_div(L.n_row_tiles, 32));
      pl.tmax = ceil_div(L.n_row_tiles, pl.G);
      for (int nst = 2; nst <= kW4Stages; ++nst) {
        const size_t n = w4_smem(slot, xr, pl.ckp, nst, pl.tmax, keep).total;
        if (n > kW4SmemLimit) break;
        pl.smem = n;
        pl.nst = nst;
      }
    }
    --pl.P;
    best = pl;
    // More ranks only while the row tiles leave half of the SMs idle.
    if (L.n_row_tiles * S * 2 > nsm) break;
  }
  return best;
}

W4Plan w4_plan(const slim_w4_layer& L, int M) {
  static PlanCache<5, W4Plan> cache;
  return cache.get({current_device(), L.K, L.N, L.group, std::min(M, 16)}, [&] { return w4_plan_uncached(L, M); });
}

template <int NT, int NG>
cudaError_t run_w4(cudaLaunchConfig_t& cfg, const W4Plan& pl, const W4Params& p) {
  cudaError_t e = ensure_func_attrs(reinterpret_cast<const void*>(k_w4<NT, NG>), pl.smem);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, k_w4<NT, NG>, p);
}

}  // namespace

size_t w4_dec_bytes(int K, int N, int group) {
  return (size_t)ceil_div(N, 16) * (K / 128) * w4_chunk(group);
}

bool w4_streams(const slim_w4_layer& L, int M) { return w4_few(L, M) && w4_plan(L, M).smem > 0; }

void w4_split(const slim_w4_layer& L, int M, int32_t* plan) {
  const W4Plan pl = M > 0 && w4_streams(L, M) ? w4_plan(L, M) : W4Plan{0, 0, 0, 0, 0, 0, 0, 0};
  plan[0] = pl.S;
  plan[1] = pl.P;
  plan[2] = pl.ckp;
  plan[3] = pl.G;
}

size_t w4_workspace_bytes(const slim_w4_layer& L, int M) {
  if (M <= 0 || w4_streams(L, M) || qgemm_pays(M, L.N)) return 0;
  return 1024 + (size_t)L.N * L.K * 2;
}

int w4_launches(const slim_w4_layer& L, int M) {
  if (M <= 0) return 0;
  return w4_streams(L, M) || qgemm_pays(M, L.N) ? 1 : 2;
}

cudaError_t launch_w4_pack(const slim_w4_layer& L, const uint16_t* W, cudaStream_t s) {
  NvtxRange nv("pack: dense 4-bit weight (k_w4_pack)");
  k_w4_pack<<<dim3(L.n_row_tiles, L.K / 128), 512, 0, s>>>(W, L.K, L.N, L.group, L.dec, L.status);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // k_w4 may start while the kernel before it still runs; this empty one
  // starts only after the packing has completed.
  k_w4_done<<<1, 32, 0, s>>>();
  return cudaGetLastError();
}

cudaError_t launch_w4_unpack(const slim_w4_layer& L, int8_t* q, uint16_t* scales, cudaStream_t s) {
  const size_t total = (size_t)L.N * L.K;
  k_w4_unpack<<<(unsigned)((total + 255) / 256), 256, 0, s>>>(L.dec, L.K, L.N, L.group, q, scales);
  return cudaGetLastError();
}

cudaError_t launch_w4(const slim_w4_layer& L, const uint16_t* X, int M, uint16_t* Y, void* ws, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  const W4Plan pl = w4_plan(L, M);
  if (w4_few(L, M) && pl.smem > 0) {
    NvtxRange nv("dense 4-bit: stream (k_w4)");
    W4Params p;
    p.X = X;
    p.Y = Y;
    p.dec = L.dec;
    p.M = M;
    p.K = L.K;
    p.N = L.N;
    p.NRT = L.n_row_tiles;
    p.NCK = L.K / 128;
    p.nst = pl.nst;
    p.status = L.status;
    p.G = pl.G;
    p.P = pl.P;
    p.ckp = pl.ckp;
    p.tmax = pl.tmax;
    cfg.gridDim = dim3(pl.S, pl.G, ceil_div(M, 16));
    cfg.blockDim = dim3(kW4Warps * 32);
    cfg.dynamicSmemBytes = pl.smem;
    attr[1].val.clusterDim.x = pl.S;
    cfg.numAttrs = pl.S > 1 ? 2 : 1;
    const int ng = 128 / L.group;
    if (pl.NT == 1)
      return ng == 1 ? run_w4<1, 1>(cfg, pl, p) : ng == 2 ? run_w4<1, 2>(cfg, pl, p) : run_w4<1, 4>(cfg, pl, p);
    return ng == 1 ? run_w4<2, 1>(cfg, pl, p) : ng == 2 ? run_w4<2, 2>(cfg, pl, p) : run_w4<2, 4>(cfg, pl, p);
  }
  if (qgemm_pays(M, L.N)) {
    NvtxRange nv("dense 4-bit: expansion and product (k_qgemm)");
    QGemmCall q;
    q.I = M;
    q.J = L.N;
    q.c = L.K;
    q.A = X;
    q.lda = L.K;
    q.C = Y;
    q.ldc = L.N;
    q.dec = L.dec;
    q.group = L.group;
    q.status = L.status;
    return launch_qgemm(q, false, s);
  }
  uint8_t* wb = static_cast<uint8_t*>(ws);
  uint16_t* W = reinterpret_cast<uint16_t*>(wb + 1024);
  {
    NvtxRange nv("dense 4-bit: expand (k_w4_expand)");
    const size_t chunks = (size_t)L.n_row_tiles * (L.K / 128);
    cfg.gridDim = dim3((unsigned)std::min<size_t>((chunks + 7) / 8, (size_t)num_sms() * 5));
    cfg.blockDim = dim3(256);
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, k_w4_expand, (const uint8_t*)L.dec, (int)L.K / 128, chunks, (int)L.K, (int)L.N,
                                       (int)L.group, W);
    if (e != cudaSuccess) return e;
  }
  NvtxRange nv("dense 4-bit: product (k_gemm)");
  GemmCall g;
  g.I = M;
  g.J = L.N;
  g.a[0].base = X;
  g.a[0].rows = M;
  g.a[0].c = g.a[0].pitch = L.K;
  g.b[0].base = W;
  g.b[0].rows = L.N;
  g.b[0].c = g.b[0].pitch = L.K;
  g.C = Y;
  g.ldc = L.N;
  g.status = L.status;
  return launch_gemms(&g, 1, false, s);
}

}  // namespace slim
