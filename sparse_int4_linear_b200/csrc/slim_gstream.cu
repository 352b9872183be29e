// Gated block for few tokens: the gate and up weights streamed once per 16
// tokens, activation and product in the same kernel.
//
// A CTA owns a range of pairs of row tiles (16 gate rows and the 16 up rows
// beside them), in the order gate tile, up tile, gate tile, ...  K is taken in
// panels whose X fits shared memory (one panel where possible).  The chunks of
// a panel (16 rows x 256 K, 1600 bytes), tile by tile, are cut into 16
// contiguous ranges, one a warp: no warp waits for another while it streams,
// and no CTA for another at all.  A warp streams its range through its own
// ring of bulk copies, expands the nibbles to exact bf16 integers, multiplies
// with the sparse tensor cores (mma.sp, the 2-bit metadata selects the staged
// activations) and scales each 128-group's sum in fp32; leaving a row tile it
// adds the sums it has of it (a segment) to a slot in shared memory.  Behind
// one barrier each warp takes pairs of tiles: it adds their segments in warp
// order and the adapter's R^T T^T (dense mma.sync), and stores act(G) U.
// Every sum has a fixed order.
//
// T = X L comes from k_adapter_down, launched just before: it starts this
// kernel as soon as X is known to be complete, and only the end of this kernel
// waits for T.  Bound by HBM; behind it the integer pipe (nibbles) and, with
// two token tiles, shared memory (activation fragments).  B200, cold L2: 4096
// to 2 x 11008, rank 128, one token 13.8 us a call (3.1 TB/s); 8192 to 2 x
// 28672, rank 256, 16 tokens 75 us (2.9 TB/s), one token without an adapter
// 5.1 TB/s.
#include <algorithm>
#include <type_traits>

#include "slim_act.cuh"
#include "slim_common.cuh"
#include "slim_internal.h"

namespace slim {
namespace {

constexpr int kGsWarps = 16;
constexpr int kGsStages = 4;        // ring stages a warp has at most
constexpr int kGsTok = 20;          // floats between tokens of a segment (16 rows + padding)
__host__ __device__ constexpr int gs_stage_chunks(int NT) { return NT == 1 ? 2 : 1; }

struct GsParams {
  const uint16_t* X;
  uint16_t* H;
  uint16_t* GU;
  const uint8_t* dec;
  const uint4* Rf;
  const uint16_t* T;
  int M, K, N, NRT, NKB;
  int r16, rl16;
  int nst;
  int G;               // CTAs
  int P, ckp;          // panels of K, chunks of a panel (the last one may lack some)
  int tmax;            // row tiles of the largest CTA
  int act;
  long long fail_cycles;   // test aid (see GatedOut)
  int32_t* status;
};

struct GsSmem {
  size_t ring, bars, who, part, ts, xs, total;
};
__host__ __device__ inline GsSmem gs_smem(int slot, int xrows, int ckp, int nst, int tmax, int rl16) {
  GsSmem m;
  size_t off = 0;
  m.ring = off; off += (size_t)kGsWarps * nst * slot;
  m.bars = off; off += (size_t)(kGsWarps * kGsStages + 2) * 8;        // the rings', X's, one that never completes
  m.who = off;  off += (size_t)(tmax * 8 + 15) / 16 * 16;             // first and last warp of a tile
  m.part = off; off += (size_t)(tmax + kGsWarps) * xrows * kGsTok * 4;
  m.ts = off;   off += rl16 > 0 ? (size_t)xrows * (rl16 + 8) * 2 : 0;
  m.xs = off;   off += (size_t)xrows * (ckp * 256 + 8) * 2;
  m.total = off;
  return m;
}

// acc += scaled sums of chunk C of a stage.  wl: the lane's words of the
// stage, sl: its scales', x0 / x1: its X rows at the stage's first k.
template <int NT, int C>
__device__ __forceinline__ void gs_chunk(float (&acc)[NT][4], uint32_t wl, uint32_t sl, uint32_t x0, uint32_t x1) {
  constexpr int O = C * kDecChunk;
  const uint4 v0 = lds128_so<O>(wl), v1 = lds128_so<O + 512>(wl), ev = lds128_so<O + 1024>(wl);
  uint32_t sw[2];
  lds64_so<O>(sl, sw[0], sw[1]);
  const uint32_t vw[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  const uint32_t ew[4] = {ev.x, ev.y, ev.z, ev.w};
  float pt[2][NT][4];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int n = 0; n < NT; ++n) pt[q][n][0] = pt[q][n][1] = pt[q][n][2] = pt[q][n][3] = 0.f;
  // One tensor-core chain per scale group; the two interleave.
  auto step = [&](auto jc) {
    constexpr int i = decltype(jc)::value, j = (i >> 1) + (i & 1) * 4, q = i & 1;
    uint32_t a[4], b[4];
    decode_word(vw[j], a);
    ldmatrix_x4_so<C * 512 + j * 64>(b, x0);
    mma_sp_16832<j & 1>(pt[q][0], a, b, ew[j >> 1]);
    if (NT == 2) {
      ldmatrix_x4_so<C * 512 + j * 64>(b, x1);
      mma_sp_16832<j & 1>(pt[q][NT - 1], a, b, ew[j >> 1]);
    }
  };
  step(std::integral_constant<int, 0>());
  step(std::integral_constant<int, 1>());
  step(std::integral_constant<int, 2>());
  step(std::integral_constant<int, 3>());
  step(std::integral_constant<int, 4>());
  step(std::integral_constant<int, 5>());
  step(std::integral_constant<int, 6>());
  step(std::integral_constant<int, 7>());
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float2 s = __half22float2(*reinterpret_cast<const __half2*>(&sw[q]));   // rows g, g + 8
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      acc[n][0] = fmaf(s.x, pt[q][n][0], acc[n][0]);
      acc[n][1] = fmaf(s.x, pt[q][n][1], acc[n][1]);
      acc[n][2] = fmaf(s.y, pt[q][n][2], acc[n][2]);
      acc[n][3] = fmaf(s.y, pt[q][n][3], acc[n][3]);
    }
  }
}

template <int NT>
__global__ void __maxnreg__(112) k_gstream(const GsParams p) {
  constexpr int SC = gs_stage_chunks(NT), SLOT = SC * kDecChunk;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int tok0 = blockIdx.y * 16, xrows = min(p.M - tok0, NT * 8), last = xrows - 1;
  const int NP = p.NRT >> 1;
  const int p0 = (int)((long long)blockIdx.x * NP / p.G), np = (int)((long long)(blockIdx.x + 1) * NP / p.G) - p0;
  const int nt = 2 * np, nst = p.nst;
  const GsSmem L = gs_smem(SLOT, xrows, p.ckp, nst, p.tmax, p.rl16);
  uint16_t* Xs = reinterpret_cast<uint16_t*>(smem + L.xs);
  uint16_t* Ts = reinterpret_cast<uint16_t*>(smem + L.ts);
  float* part = reinterpret_cast<float*>(smem + L.part);
  int2* who = reinterpret_cast<int2*>(smem + L.who);
  uint8_t* ring = smem + L.ring + (size_t)warp * nst * SLOT;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bars) + warp * kGsStages;
  uint64_t* xbar = reinterpret_cast<uint64_t*>(smem + L.bars) + kGsWarps * kGsStages;
  const int xrow = p.ckp * 256 + 8, trow = p.rl16 + 8;
  // The layer's row tile at place lt of this CTA's stream.
  auto tile_at = [&](int lt) { return (lt & 1) * NP + p0 + (lt >> 1); };
  // Warp w's range of a panel (of ckp chunks a tile, whether they exist or
  // not, so that it is the same in every panel) starts here.
  auto start = [&](int w) {
    const int C = nt * p.ckp, W = min(kGsWarps, C);
    return w >= W ? C : (int)((long long)w * C / W);
  };
  const int f0 = start(warp), f1 = start(warp + 1);

  // Copies run ahead of the products: i_* is the next stage's panel, place,
  // chunk and what is left of the range, and how many chunks of the tile exist
  // in it.
  int i_n = 0, i_pan = 0, i_lt = 0, i_c = 0, i_left = 0, i_real = 0;
  auto open_tile = [&]() {      // to the next tile with a chunk to copy
    for (;;) {
      if (i_left == 0) {
        if (i_pan >= p.P || f1 == f0) {
          i_pan = p.P;
          return;
        }
        i_left = f1 - f0;
        i_lt = f0 / p.ckp;
        i_c = f0 - i_lt * p.ckp;
      }
      i_real = min(min(i_left, p.ckp - i_c), p.NKB - i_pan * p.ckp - i_c);
      if (i_real > 0) return;
      i_left -= min(i_left, p.ckp - i_c);
      i_c = 0;
      ++i_lt;
      if (i_left == 0) ++i_pan;
    }
  };
  open_tile();
  auto issue = [&](int slot) {     // the next stage, if there is one
    if (i_pan >= p.P) return;
    const int n = min(SC, i_real);
    if (lane == 0 && dcheck(tile_at(i_lt) < p.NRT && i_pan * p.ckp + i_c + n <= p.NKB, p.status)) {
      mbar_expect_tx(bars + slot, (uint32_t)(n * kDecChunk));
      bulk_g2s(ring + slot * SLOT, p.dec + ((size_t)tile_at(i_lt) * p.NKB + i_pan * p.ckp + i_c) * kDecChunk,
               (uint32_t)(n * kDecChunk), bars + slot);
    }
    ++i_n;
    i_c += n;
    i_left -= n;
    i_real -= n;
    if (i_real == 0) {
      const int skip = i_c < p.ckp ? min(i_left, p.ckp - i_c) : 0;   // chunks the panel lacks
      const bool ends = i_c + skip == p.ckp;
      i_left -= skip;
      if (ends) {
        i_c = 0;
        ++i_lt;
      }
      if (i_left == 0) ++i_pan;
      open_tile();
    }
  };
  if (lane == 0) {
    for (int i = 0; i < nst; ++i) mbar_init(bars + i, 1);
    if (warp == 0) {
      mbar_init(xbar, 1);
      mbar_init(xbar + 1, 1);
    }
    fence_mbar_init();
  }
  __syncwarp();
  // The packed weight is constant: start streaming at once, with one stage a
  // warp (more would keep X waiting behind it).
  issue(0);
  // X of a panel: one bulk copy per token row, by one thread; zeros past K.
  auto stage_x = [&](int pan) {
    const uint32_t bytes = (uint32_t)min(p.ckp * 256, p.K - pan * p.ckp * 256) * 2u;
    const uint16_t* xp = p.X + (size_t)tok0 * p.K + (size_t)pan * p.ckp * 256;
    mbar_expect_tx(xbar, bytes * (uint32_t)xrows);
    for (int tk = 0; tk < xrows; ++tk) bulk_g2s(Xs + tk * xrow, xp + (size_t)tk * p.K, bytes, xbar);
  };
  auto pad_x = [&](int pan) {
    const int have = min(p.ckp * 256, p.K - pan * p.ckp * 256), pad = (have + 255) / 256 * 256 - have;
    for (int i = threadIdx.x; i < xrows * pad; i += kGsWarps * 32) Xs[(i / pad) * xrow + have + i % pad] = 0;
  };
  pad_x(0);
  if (threadIdx.x == 0) {
    // With an adapter k_adapter_down came just before: it has seen X complete.
    if (p.r16 == 0) pdl_wait();
    stage_x(0);
  }
  __syncthreads();
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
  const uint32_t ring_s = smem_u32(ring), bar_s = smem_u32(bars);
  const uint32_t wl0 = ring_s + lane * 16, sl0 = ring_s + 1536 + 8 * g;
  const int pstride = xrows * kGsTok;

  bool ok = p.fail_cycles == 0 || __all_sync(0xffffffffu, mbar_wait(xbar + 1, 0, p.fail_cycles));
  int it = 0, st = 0, gave_up = 0, gave_pan = 0;   // where a wait gave up: the stage, the panel
  uint32_t ph = 0;
  for (int pan = 0; pan < p.P; ++pan) {
    if (pan > 0) {
      __syncthreads();      // the last panel's X is no longer read
      if (threadIdx.x == 0 && ok) {
        fence_proxy_async_smem();
        stage_x(pan);
      }
      if (pan + 1 == p.P) {
        pad_x(pan);
        __syncthreads();
      }
    }
    if (ok && !__all_sync(0xffffffffu, mbar_wait(xbar, pan & 1))) {
      ok = false;
      gave_up = it;
      gave_pan = pan;
    }
    int left = f1 - f0, lt = f0 / p.ckp, c = f0 - lt * p.ckp;
    while (left > 0) {
      const int in_tile = min(left, p.ckp - c), real = min(in_tile, p.NKB - pan * p.ckp - c);
      for (int q = 0; q < real; q += SC) {
        if (ok) {
          ok = __all_sync(0xffffffffu, mbar_wait_s(bar_s + st * 8, ph));
          if (!ok) {
            gave_up = it;
            gave_pan = pan;
          }
        }
        if (ok) {
          const uint32_t wl = wl0 + (uint32_t)(st * SLOT), sl = sl0 + (uint32_t)(st * SLOT);
          const uint32_t x0 = xa0 + (uint32_t)(c + q) * 512u, x1 = xa1 + (uint32_t)(c + q) * 512u;
          gs_chunk<NT, 0>(acc, wl, sl, x0, x1);
          if (SC == 2 && q + 1 < real) gs_chunk<NT, SC - 1>(acc, wl, sl, x0, x1);
          __syncwarp();
          if (lane == 0) fence_proxy_async_smem();
          issue(st);
        }
        ++it;
        if (++st == nst) {
          st = 0;
          ph ^= 1u;
        }
      }
      // Leaving the tile: the segment of warp w and place lt lies in slot
      // lt + w (both grow along the stream), the same in every panel.
      if (pan == 0 && lane == 0) {
        if (c == 0) who[lt].x = warp;
        if (c + in_tile == p.ckp) who[lt].y = warp;
      }
      float* dst = part + (size_t)(lt + warp) * pstride;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tk = n * 8 + 2 * t + (i & 1);
          if (tk < xrows) {
            float* d = dst + tk * kGsTok + g + 8 * (i >> 1);
            *d = pan == 0 ? acc[n][i] : *d + acc[n][i];
          }
          acc[n][i] = 0.f;
        }
      }
      left -= in_tile;
      c = 0;
      ++lt;
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
  // T = X L of the kernel before this one, and with it everything older.
  pdl_wait();
  {
    const int per = p.rl16 / 8;
    for (int i = threadIdx.x; i < xrows * per; i += kGsWarps * 32) {
      const int tk = i / per, c8 = (i - tk * per) * 8;
      *reinterpret_cast<uint4*>(Ts + tk * trow + c8) =
          __ldcg(reinterpret_cast<const uint4*>(p.T + (size_t)(tok0 + tk) * p.rl16 + c8));
    }
  }
  // A CTA one of whose waits gave up stores NaN.
  const bool bad = __syncthreads_or(!ok);
  const int F = p.N >> 1, JS = p.r16 / 16;
  const uint32_t ts_s = smem_u32(Ts);
  const uint32_t tb = ts_s + (uint32_t)((NT == 2 ? min((lane & 7) + ((lane >> 4) & 1) * 8, last) : min(lane & 7, last)) * trow +
                                        ((lane >> 3) & 1) * 8) * 2u;
  for (int pr = warp; pr < np; pr += kGsWarps) {
    float y[2][NT][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int lt = 2 * pr + j;
      const uint4* rf = p.Rf + (size_t)tile_at(lt) * JS * 32 + lane;
      uint4 af[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < JS) af[q] = __ldg(rf + q * 32);
#pragma unroll
      for (int n = 0; n < NT; ++n) y[j][n][0] = y[j][n][1] = y[j][n][2] = y[j][n][3] = 0.f;
      const int2 ww = who[lt];
      const float* ps = part + (size_t)(lt + ww.x) * pstride + g;
#pragma unroll 2
      for (int w = ww.x; w <= ww.y; ++w, ps += pstride) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tk = n * 8 + 2 * t + (i & 1);
            if (tk < xrows) y[j][n][i] += ps[tk * kGsTok + 8 * (i >> 1)];
          }
      }
      // R^T T^T of linear j: T columns [j r16, (j + 1) r16).
      for (int s0 = 0; s0 < JS; s0 += 8) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (s0 + q < JS) {
            uint32_t b[4];
            const uint32_t a = tb + (uint32_t)(j * p.r16 + (s0 + q) * 16) * 2u;
            if (NT == 2) {
              ldmatrix_x4_s(b, a);
            } else {
              asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(b[0]), "=r"(b[1]) : "r"(a));
            }
            mma_16816(y[j][0], af[q], b[0], b[1]);
            if (NT == 2) mma_16816(y[j][NT - 1], af[q], b[2], b[3]);
          }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (s0 + 8 + q < JS) af[q] = __ldg(rf + (s0 + 8 + q) * 32);
      }
    }
    const int n0 = (p0 + pr) * 16 + g;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tk = n * 8 + 2 * t + (i & 1), row = n0 + 8 * (i >> 1);
        if (tk >= xrows || !dcheck(row < F && tok0 + tk < p.M, p.status)) continue;
        const float gv = bad ? NAN : y[0][n][i], uv = bad ? NAN : y[1][n][i];
        p.H[(size_t)(tok0 + tk) * F + row] = __bfloat16_as_ushort(__float2bfloat16_rn(act_fwd(p.act, gv) * uv));
        if (p.GU) {
          p.GU[(size_t)(tok0 + tk) * p.N + row] = __bfloat16_as_ushort(__float2bfloat16_rn(gv));
          p.GU[(size_t)(tok0 + tk) * p.N + F + row] = __bfloat16_as_ushort(__float2bfloat16_rn(uv));
        }
      }
  }
}

// ---------------------------------------------------------------- host
struct GsPlan {
  int NT = 1, P = 1, ckp = 0, nst = 0, G = 1, tmax = 0;
  size_t smem = 0;
};

// One panel of K if its X fits, else the fewest; then the deepest rings.  A
// CTA has an even share of the row tiles on the SMs, up to 64; fewer where an
// adapter of thousands of columns (T in shared memory) leaves no room (at 2
// tiles, 4096 columns and 16 tokens the smallest plan takes 214 KB, so one
// always fits).
//
// Up to 150 KB k_adapter_down's CTAs (74 KB) fit beside this kernel's, which
// then start at once (7B, one token: 13.2 us a call against 17.1 with rings of
// three stages, which leave no room).  That is kept with one token tile and up
// to two panels; more cost more than the wait (70B, 8 tokens: 57 us in
// 160 KB, 49 in 220; 7B, 8 tokens, two panels: 15.4 against 18.0).
GsPlan gs_plan_fit(const slim_layer& L, int M, size_t limit, int most_panels) {
  GsPlan pl;
  pl.NT = M <= 8 ? 1 : 2;
  const int NP = L.n_row_tiles / 2, slot = gs_stage_chunks(pl.NT) * kDecChunk;
  for (int most = 32; most >= 1; most /= 2) {
    pl.G = std::max(std::min(NP, num_sms()), ceil_div(NP, most));
    pl.tmax = 2 * ceil_div(NP, pl.G);
    for (pl.P = 1; pl.P <= std::min(L.n_kblocks, most_panels); ++pl.P) {
      pl.ckp = ceil_div(L.n_kblocks, pl.P);
      if (ceil_div(L.n_kblocks, pl.ckp) != pl.P) continue;
      for (int nst = 2; nst <= kGsStages; ++nst) {
        const size_t n = gs_smem(slot, M, pl.ckp, nst, pl.tmax, L.rl16).total;
        if (n > limit) break;
        pl.smem = n;
        pl.nst = nst;
      }
      if (pl.smem) return pl;
    }
  }
  return pl;
}

GsPlan gs_plan_uncached(const slim_layer& L, int M) {
  if (M <= 8 && L.r16 > 0) {
    const GsPlan pl = gs_plan_fit(L, M, 150 * 1024, 2);
    if (pl.smem) return pl;
  }
  return gs_plan_fit(L, M, 220 * 1024, L.n_kblocks);
}

GsPlan gs_plan(const slim_layer& L, int M) {
  static PlanCache<5, GsPlan> cache;
  return cache.get({current_device(), L.K, L.N, L.rl16, std::min(M, 16)},
                   [&] { return gs_plan_uncached(L, std::min(M, 16)); });
}

template <int NT>
cudaError_t run_gstream(cudaLaunchConfig_t& cfg, const GsParams& p) {
  cudaError_t e = ensure_func_attrs(reinterpret_cast<const void*>(k_gstream<NT>), cfg.dynamicSmemBytes);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, k_gstream<NT>, p);
}

}  // namespace

bool gstream_fits(const slim_layer& L, int M) { return gs_plan(L, M).smem > 0; }

cudaError_t launch_gstream(const slim_layer& L, const uint16_t* X, int M, const GatedOut& o, const uint16_t* T,
                           cudaStream_t s) {
  NvtxRange nv("gated decode: stream, adapter T R, activation and product (k_gstream)");
  const GsPlan pl = gs_plan(L, M);
  if (!pl.smem) return cudaErrorNotSupported;
  GsParams p;
  p.X = X;
  p.H = o.Y;
  p.GU = o.GU;
  p.dec = L.dec;
  p.Rf = reinterpret_cast<const uint4*>(L.Rf);
  p.T = T;
  p.M = M;
  p.K = L.K;
  p.N = L.N;
  p.NRT = L.n_row_tiles;
  p.NKB = L.n_kblocks;
  p.r16 = L.r16;
  p.rl16 = L.rl16;
  p.nst = pl.nst;
  p.G = pl.G;
  p.P = pl.P;
  p.ckp = pl.ckp;
  p.tmax = pl.tmax;
  p.act = o.act;
  p.fail_cycles = o.fail_cycles;
  p.status = L.status;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pl.G, ceil_div(M, 16));
  cfg.blockDim = dim3(kGsWarps * 32);
  cfg.dynamicSmemBytes = pl.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return pl.NT == 1 ? run_gstream<1>(cfg, p) : run_gstream<2>(cfg, p);
}

}  // namespace slim
