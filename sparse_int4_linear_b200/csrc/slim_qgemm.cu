// Products with a packed 4-bit operand, for few token tiles: the weight is
// expanded to bf16 (q * s rounded, as everywhere on the tensor-core paths)
// straight into the MMA's shared-memory operand tiles and never written out,
// so a call moves 0.4 to 0.5 bytes per weight instead of the 4.5 of an expanded
// copy in memory.
//
// A CTA computes 128 tokens x 256 columns, stage by stage of 64 of the
// contraction: sixteen warps expand the weight's tile (packed words prefetched
// into registers two stages ahead), one loads the activations by tensor
// copies, one issues the MMAs (tcgen05, fp32 sums in tensor memory); the
// expanding warps write the result.  The contraction is split over a cluster
// of up to 8 CTAs whose sums are added in rank order through distributed
// shared memory.
//
//   k_qgemm<0>  B(j, c) = W[c][j] of a 2:4 layer (dX = dY W): a tile's rows c
//               are lines of 64 columns j, an MN-major operand; plus the
//               adapter's dT L^T from its images
//   k_qgemm<1>  B(j, c) = W[j][c] of a dense 4-bit layer: K-major
//
// Bound by the expansion's instructions: 0.86 us a stage of 16 K weights at
// K 8192, N 28672 (0.25 of the tensor pipe, a tenth of the memory bandwidth).
// B200, cold L2, 128 tokens: dense 4096 x 11008 27 us against 52 with an
// expanded copy, 8192 x 28672 113 against 212; dX of an 8192 x 8192 2:4 layer
// 37 against 56.
#include <cooperative_groups.h>

#include <algorithm>

#include "slim_internal.h"
#include "slim_qgemm.h"
#include "slim_tcgen05.cuh"

namespace slim {
namespace {

constexpr int QG_ROWS = 128, QG_COLS = 256;
constexpr int QG_EXP = 16;                   // warps 0-15: expansion, then the result
constexpr int QG_THREADS = (QG_EXP + 2) * 32;   // warp 16: copies, warp 17: MMA issue
constexpr int QG_A = QG_ROWS * 128, QG_B = QG_COLS * 128, QG_STAGE = QG_A + QG_B;
constexpr int QG_NST = 4;
constexpr int QG_SMEM = QG_NST * QG_STAGE + (2 * QG_NST + 1) * 8 + 16 + 1024;
static_assert(QG_NST * QG_STAGE >= QG_ROWS * (QG_COLS + 4) * 4, "a rank's sums fit the rings");

struct QgParams {
  int I, J, c, c2;
  int ni, nj;          // tiles
  uint16_t* C;
  int ldc;
  const uint8_t* vals;
  const uint8_t* meta;
  const __half* scales;
  const uint8_t* dec;
  int ng;              // groups of a chunk
  int splits;
  int early;
  int32_t* status;
};

__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr) {
  // MN-major, 128-byte swizzle: lines of 64 rows, 8-line groups 1024 B apart
  // along the contraction (SBO), the next 64 rows 8 KB on (LBO).
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(8192 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// (Ordered among the volatile statements around them, the barriers' too; loads
// of other shared memory may pass them.)
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v));
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w));
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// A nibble u = q + 8 at bits [b, b + 4) of the mantissa of 1.0 reads 1 + u /
// 2^n, n = 23 - b, so q s = fma(that, 2^n s, -(2^n + 8) s): one rounding, of a
// value of 4 + 11 bits, so none; both factors are exact too while 2^n + 8 has
// n - 2 <= 13 significant bits beside the scale's 11.  Nibbles 2, 3 and 4 of a
// word lie well as they are, 0 and 1 after a shift up by two, 5 to 7 after a
// shift down by three: 2.25 instructions per weight.
struct NibScale {
  float m[3], c[3];
  __device__ __forceinline__ explicit NibScale(float s) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int n = 15 - 4 * k;
      m[k] = s * (float)(1 << n);
      c[k] = -s * (float)((1 << n) + 8);
    }
  }
};
struct Nibbles {
  uint32_t lo, mid, hi;
  __device__ __forceinline__ explicit Nibbles(uint32_t w) : lo(w << 8), mid(w), hi(w >> 12) {}
  __device__ __forceinline__ float at(int i, const NibScale& s) const {   // i a constant once unrolled
    const uint32_t w = i < 2 ? lo : i < 5 ? mid : hi;
    const int k = i < 2 ? i : i < 5 ? i - 2 : i - 5;
    return fmaf(__uint_as_float(0x3F800000u | (w & (0xF00u << (4 * k)))), s.m[k], s.c[k]);
  }
};

// Packed words one thread needs of a stage.
template <int SRC>
struct QgWords;
template <>
struct QgWords<0> {      // 32 columns j of one row c
  uint2 v;
  uint32_t m;
  uint16_t s;
};
template <>
struct QgWords<1> {      // 4 steps of 16 c of a row tile
  uint4 v;
  uint2 s;               // the scales of rows g and g + 8, up to two groups of the 64 columns
};

template <int SRC>
__global__ void __launch_bounds__(QG_THREADS, 1)
    k_qgemm(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap ta2,
            const __grid_constant__ CUtensorMap tb2, const __grid_constant__ QgParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + QG_NST * QG_STAGE);
  uint64_t* empty = full + QG_NST;
  uint64_t* acc_full = empty + QG_NST;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(acc_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(acc_full + 1) + 1;
  __shared__ uint32_t place[16];
  float* red = reinterpret_cast<float*>(smem);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int SP = p.splits, split = SP > 1 ? (int)cluster_rank() : 0;
  const int tile = blockIdx.x / SP;
  const int i0 = tile % p.ni * QG_ROWS, j0 = tile / p.ni * QG_COLS;
  const int S0 = ceil_div(p.c, 64), S = S0 + ceil_div(p.c2, 64);
  const int u0 = (int)((long long)split * S / SP), u1 = (int)((long long)(split + 1) * S / SP);

  if (threadIdx.x < 16) {
    // Bytes of columns 0 .. 3 out of (pair, 0): 4 is a zero byte, the kept
    // columns i0 and i1 (nibble i0 | i1 << 2) get bytes 1, 0 and 3, 2.
    const int t = threadIdx.x;
    place[t] = 0x44444444u ^ (0x54u << ((t & 3) * 8)) ^ (0x76u << ((t >> 2) * 8));
  }
  if (threadIdx.x == 0) {
    // A stage is full when its copies have landed and every expanding warp
    // has written its part.
    for (int i = 0; i < QG_NST; ++i) {
      mbar_init(full + i, 1 + QG_EXP);
      mbar_init(empty + i, 1);
    }
    mbar_init(acc_full, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == QG_EXP + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32((const void*)tmem_slot)),
                 "r"(QG_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < QG_EXP) {
    // ---------------------------------------------------------------- expansion
    const int ew = warp;
    const int g = lane >> 2, t = lane & 3;
    constexpr int AHEAD = 2;
    QgWords<SRC> w[AHEAD];
    // SRC 0: lane = row c = 8 (ew % 8) + lane % 8 of a stage, columns 128 (ew
    // / 8) + 32 (lane / 8) on.  SRC 1: row tile ew of the tile's 16.
    const int c = (ew & 7) * 8 + (lane & 7), j = j0 + (ew >> 3) * 128 + (lane >> 3) * 32;
    const int rt = j0 / 16 + ew, ng = p.ng, chunk = 1024 + 32 * ng;
    const bool inside = SRC == 0 ? j < p.J : rt * 16 < p.J;
    const uint8_t* pv = SRC == 0 ? p.vals + (size_t)c * (p.J / 4) + j / 4 : p.dec + (size_t)rt * (p.c / 128) * chunk + lane * 16;
    const uint8_t* ps = SRC == 0 ? reinterpret_cast<const uint8_t*>(p.scales + (size_t)c * (p.J / 128) + j / 128)
                                 : pv - lane * 16 + 1024 + g * ng * 4;
    // Where the lane's pieces go in a stage's tile (the swizzle: 16-byte piece k
    // of line c at k ^ c % 8).
    const uint32_t sm = smem_u32(smem);
    uint32_t off[SRC == 0 ? 4 : 8];
#pragma unroll
    for (int k = 0; k < (SRC == 0 ? 4 : 8); ++k)
      off[k] = SRC == 0 ? (uint32_t)(((j - j0) >> 6) * 8192 + c * 128 + (((((j & 32) >> 3) + k) ^ (c & 7)) << 4))
                        : (uint32_t)(ew * 2048 + g * 128 + ((k ^ g) << 4) + t * 4);
    const uint8_t* pm = p.meta + (size_t)c * (p.J / 8) + j / 8;   // SRC 0 only
    auto fetch = [&](int u, QgWords<SRC>& q) {
      const bool on = inside && u < u1 && (SRC == 1 || u * 64 + c < p.c);
      if constexpr (SRC == 0) {
        q.v = make_uint2(0u, 0u);
        q.m = 0x44444444u;
        q.s = 0;
        if (on) {
          q.v = __ldg(reinterpret_cast<const uint2*>(pv + (size_t)u * (16 * p.J)));
          q.m = __ldg(reinterpret_cast<const uint32_t*>(pm + (size_t)u * (8 * p.J)));
          q.s = __ldg(reinterpret_cast<const uint16_t*>(ps + (size_t)u * p.J));
        }
      } else {
        q.v = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
        q.s = make_uint2(0u, 0u);
        if (on) {
          const size_t at = (size_t)(u >> 1) * chunk;
          q.v = __ldg(reinterpret_cast<const uint4*>(pv + at + (u & 1) * 512));
          const uint32_t* sc = reinterpret_cast<const uint32_t*>(ps + at) + ((u & 1) * ng >> 1);
          q.s.x = __ldg(sc);
          q.s.y = ng == 4 ? __ldg(sc + 1) : q.s.x;
        }
      }
    };
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) fetch(u0 + k, w[k]);
    int st = 0;
    uint32_t ph = 1;
    for (int ub = u0; ub < u1; ub += AHEAD) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int u = ub + k;
        if (u >= u1) break;
        const QgWords<SRC> q = w[k];
        fetch(u + AHEAD, w[k]);
        // (A wait that gives up leaves the stage short of arrivals; the MMA
        // warp's own wait then gives up too.)
        if (!warp_pwait(empty + st, ph, abort_flag)) break;
        const uint32_t bs = sm + (uint32_t)(st * QG_STAGE + QG_A);
        if (u < S0) {
          if constexpr (SRC == 0) {
            const NibScale s(__half2float(__ushort_as_half(q.s)));
            const Nibbles vv[2] = {Nibbles(q.v.x ^ 0x88888888u), Nibbles(q.v.y ^ 0x88888888u)};
#pragma unroll
            for (int h = 0; h < 4; ++h) {       // 8 columns, two groups of 4
              uint32_t o[4];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int i = (h & 1) * 4 + e * 2;
                const uint32_t pr = pack2(vv[h >> 1].at(i, s), vv[h >> 1].at(i + 1, s));
                const uint32_t sel = place[(q.m >> (h * 8 + e * 4)) & 15u];
                o[2 * e] = __byte_perm(pr, 0u, sel);
                o[2 * e + 1] = __byte_perm(pr, 0u, sel >> 16);
              }
              sts128(bs + off[h], o[0], o[1], o[2], o[3]);
            }
          } else {
            const Nibbles ww[4] = {Nibbles(q.v.x), Nibbles(q.v.y), Nibbles(q.v.z), Nibbles(q.v.w)};
            const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&q.s.x));
            const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&q.s.y));
#pragma unroll
            for (int r = 0; r < 2; ++r) {      // row g + 8 r
              const NibScale sa(r ? fa.y : fa.x), sb(r ? fb.y : fb.x);
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // columns 16 j + 8 h + 2 t
                  const int i = 2 * h + r;
                  const NibScale& sc = j < 2 ? sa : sb;
                  sts32(bs + off[2 * j + h] + r * 1024, pack2(ww[j].at(i, sc), ww[j].at(4 + i, sc)));
                }
            }
          }
        }
        fence_proxy_async_smem();   // before the tensor cores read it
        __syncwarp();
        if (lane == 0) mbar_arrive(full + st);
        if (++st == QG_NST) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
    // ---------------------------------------------------------------- result
    // Lanes (rows) 32 (warp % 4) on, columns 64 (warp / 4) on.
    const bool acc_ok = mbar_wait(acc_full, 0);
    tc_fence_after();
    if (!p.early) pdl_wait();   // the output may still be in use by earlier work on the stream
    const bool good = __all_sync(0xffffffffu, acc_ok && !*abort_flag);
    if (!good && lane == 0) {
      *abort_flag = 1;
      record_status(p.status, SLIM_ERR_TIMEOUT);
    }
    const int row = warp % 4 * 32 + lane, i = i0 + row;
    for (int c0 = warp / 4 * 64, c1 = c0 + 64; c0 < c1; c0 += 32) {
      uint32_t v[32];
      if (good) {
        tc_ld32(v, tmem + ((uint32_t)(warp % 4 * 32) << 16) + (uint32_t)c0);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
      } else {
#pragma unroll
        for (int q = 0; q < 32; ++q) v[q] = 0x7FC00000u;   // incomplete sums are stored as NaN
        // (What goes by way of the rings may meet a copy that lands late, so NaN
        // is chosen again where it is stored.)
      }
      if (SP > 1) {
        // This rank's sums, rows padded by 4 floats; the rings are idle (every
        // stage was read by a completed MMA).
        uint4* r = reinterpret_cast<uint4*>(red + (size_t)row * (QG_COLS + 4) + c0);
#pragma unroll
        for (int q = 0; q < 8; ++q) r[q] = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
      } else if (j0 + c0 + 32 <= p.J && (p.ldc & 7) == 0) {
        uint16_t* out = p.C + (size_t)i * p.ldc + j0 + c0;
        if (i < p.I)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[e] = pack2(__uint_as_float(v[8 * q + 2 * e]), __uint_as_float(v[8 * q + 2 * e + 1]));
            reinterpret_cast<uint4*>(out)[q] = make_uint4(o[0], o[1], o[2], o[3]);
          }
      } else {
        // Rows without whole 16-byte pieces: the lanes write a row's columns
        // side by side, by way of the (idle) rings.
        uint32_t* st = reinterpret_cast<uint32_t*>(smem) + warp * 32 * 17;
#pragma unroll
        for (int q = 0; q < 16; ++q)
          st[lane * 17 + q] = pack2(__uint_as_float(v[2 * q]), __uint_as_float(v[2 * q + 1]));
        __syncwarp();
        if (j0 + c0 + lane < p.J) {
          const uint16_t* from = reinterpret_cast<const uint16_t*>(st) + lane;
          uint16_t* to = p.C + (size_t)(i - lane) * p.ldc + j0 + c0 + lane;
          const int n = min(32, p.I - (i - lane));
#pragma unroll 8
          for (int r = 0; r < n; ++r, to += p.ldc) *to = good ? from[r * 34] : (uint16_t)0x7FC0;
        }
        __syncwarp();
      }
    }
  } else if (warp == QG_EXP) {
    // ---------------------------------------------------------------- copies
    const bool one = elect_one();
    if (one) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&ta)) : "memory");
      if (p.c2 > 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&ta2)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tb2)) : "memory");
      }
    }
    __syncwarp();
    if (!p.early) pdl_wait();   // the activations were written by the previous kernels on the stream
    pdl_launch_dependents();
    int st = 0;
    uint32_t ph = 1;
    for (int u = u0; u < u1; ++u) {
      if (!warp_pwait(empty + st, ph, abort_flag)) break;
      if (one) {
        uint8_t* as = smem + st * QG_STAGE;
        if (u < S0) {
          mbar_expect_tx(full + st, QG_A);
          tma_load_2d(as, &ta, u * 64, i0, full + st);
        } else {
          const int c = (u - S0) * 64;
          mbar_expect_tx(full + st, QG_A + QG_B);
          tma_load_2d(as, &ta2, c, i0, full + st);
          for (int b = 0; b < 4; ++b) tma_load_2d(as + QG_A + b * 8192, &tb2, 0, (j0 / 64 + b) * p.c2 + c, full + st);
        }
      }
      __syncwarp();
      if (++st == QG_NST) {
        st = 0;
        ph ^= 1u;
      }
    }
    if (lane == 0 && *abort_flag) {
      // Let the copies in flight land: their stages may lack other arrivals,
      // so time is all there is to wait for.
      const long long t0 = clock64();
      while (clock64() - t0 < 200000) {
      }
    }
  } else {
    // ---------------------------------------------------------------- MMA issue
    const bool one = elect_one();
    const uint32_t base = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(QG_COLS >> 3) << 17) | ((uint32_t)(QG_ROWS >> 4) << 24);
    const uint32_t mn = base | (1u << 16);
    const uint32_t sm = smem_u32(smem);
    int st = 0;
    uint32_t ph = 0;
    for (int u = u0; u < u1; ++u) {
      if (!warp_pwait(full + st, ph, abort_flag)) break;
      tc_fence_after();
      const int kks = min(4, ceil_div(u < S0 ? p.c - u * 64 : p.c2 - (u - S0) * 64, 16));
      if (one) {
        const uint32_t as = sm + (uint32_t)(st * QG_STAGE), bs = as + QG_A;
        for (int kk = 0; kk < kks; ++kk) {
          // (The adapter's images are MN-major too.)
          if (SRC == 0) mma_dense(tmem, sw128_desc(as + kk * 32), mn_desc(bs + kk * 2048), mn, (u - u0) | kk);
          else mma_dense(tmem, sw128_desc(as + kk * 32), sw128_desc(bs + kk * 32), base, (u - u0) | kk);
        }
        tc_commit(empty + st);
      }
      __syncwarp();
      if (++st == QG_NST) {
        st = 0;
        ph ^= 1u;
      }
    }
    if (one) tc_commit(acc_full);
    __syncwarp();
  }
  if (SP > 1) {
    // Rank r adds rows [rows r / SP, rows (r + 1) / SP) over the ranks, in rank
    // order; NaN if a wait of any rank gave up.
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    tc_fence_before();
    cluster.sync();
    bool bad = false;
    for (int q = 0; q < SP; ++q) bad = bad || *cluster.map_shared_rank(const_cast<int*>(abort_flag), q) != 0;
    const int rows = min(QG_ROWS, p.I - i0), r0 = split * rows / SP, r1 = (split + 1) * rows / SP;
    // (A warp reads whole lines of a rank at a time.)
    for (int e = threadIdx.x; e < (r1 - r0) * (QG_COLS / 4); e += QG_THREADS) {
      const int row = r0 + e / (QG_COLS / 4), j = e % (QG_COLS / 4) * 4;
      if (j0 + j >= p.J || !dcheck(i0 + row < p.I, p.status)) continue;
      const size_t off = (size_t)row * (QG_COLS + 4) + j;
      float4 v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < SP) v[q] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(red, q) + off);
      float f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < SP) {
          f[0] += v[q].x; f[1] += v[q].y; f[2] += v[q].z; f[3] += v[q].w;
        }
      if (bad) f[0] = f[1] = f[2] = f[3] = NAN;
      uint16_t* out = p.C + (size_t)(i0 + row) * p.ldc + j0 + j;
      if (j0 + j + 4 <= p.J && (p.ldc & 3) == 0) {
        *reinterpret_cast<uint2*>(out) = make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (j0 + j + q < p.J) out[q] = __bfloat16_as_ushort(__float2bfloat16_rn(f[q]));
      }
    }
    cluster.sync();
  }
  // An early kernel completes no earlier than the one before it.
  if (p.early && threadIdx.x == 0 && blockIdx.x == 0) pdl_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == QG_EXP + 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(QG_COLS) : "memory");
  }
}

CUresult encode_rows64(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* m, const void* base, long long cols,
                       long long rows, long long pitch, int box_rows, bool swizzled) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)pitch * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, estr[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, swizzled ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

template <int SRC>
cudaError_t run_qgemm(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* cluster, const CUtensorMap& ta, const CUtensorMap& ta2,
                      const CUtensorMap& tb2, QgParams& p, int most) {
  const void* f = reinterpret_cast<const void*>(k_qgemm<SRC>);
  cudaError_t e = ensure_func_attrs(f, QG_SMEM);
  if (e != cudaSuccess) return e;
  // The largest split whose clusters all run at once.
  for (p.splits = most; p.splits > 1; --p.splits) {
    cluster->val.clusterDim.x = p.splits;
    cfg.gridDim = dim3(p.splits);
    if (p.ni * p.nj <= max_clusters(f, cfg)) break;
  }
  cluster->val.clusterDim.x = p.splits;
  cfg.gridDim = dim3(p.ni * p.nj * p.splits);
  cfg.numAttrs = p.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_qgemm<SRC>, ta, ta2, tb2, p);
}

}  // namespace

// One token tile: always.  Every further one expands the weight again, which
// pays while the SMs it keeps busy would be idle: a product whose tiles are at
// most half of the SMs for two of them, a quarter for up to four.  Measured,
// here against an expanded copy, us a call: dense 4096 x 4096, 128 tokens 17.8
// and 27.2, 256 tokens (32 tiles) 23 and 28.9, 512 tokens (64) 36.6 and 35.7;
// 4096 x 11008, 128 tokens 27 and 52, 256 tokens (86) 64 and 60; 2048 x 2048,
// 512 tokens (32) 16.4 and 20.0; the backward pass of 4096 x 4096, rank 128,
// 128 tokens 24.7 and 32.2, 256 tokens 33.2 and 38.7, 512 tokens 52.8 and 45.2.
bool qgemm_pays(int I, int J) {
  const int tiles = ceil_div(I, QG_ROWS) * ceil_div(J, QG_COLS), nsm = num_sms();
  return I <= QG_ROWS || (I <= 2 * QG_ROWS && tiles * 2 <= nsm) || (I <= 4 * QG_ROWS && tiles * 4 <= nsm);
}

cudaError_t launch_qgemm(const QGemmCall& g, bool early, cudaStream_t s) {
  auto encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  CUtensorMap ta, ta2 = {}, tb2 = {};
  if (encode_rows64(encode, &ta, g.A, g.c, g.I, g.lda, QG_ROWS, false) != CUDA_SUCCESS) return cudaErrorInvalidValue;
  if (g.A2 && (encode_rows64(encode, &ta2, g.A2, g.c2, g.I, g.c2, QG_ROWS, false) != CUDA_SUCCESS ||
               encode_rows64(encode, &tb2, g.B2, 64, (long long)g.J / 64 * g.c2, 64, 64, true) != CUDA_SUCCESS))
    return cudaErrorInvalidValue;
  QgParams p = {};
  p.I = g.I;
  p.J = g.J;
  p.c = g.c;
  p.c2 = g.A2 ? g.c2 : 0;
  p.ni = ceil_div(g.I, QG_ROWS);
  p.nj = ceil_div(g.J, QG_COLS);
  p.C = g.C;
  p.ldc = g.ldc;
  p.vals = g.vals;
  p.meta = g.meta;
  p.scales = reinterpret_cast<const __half*>(g.scales);
  p.dec = g.dec;
  p.ng = g.dec ? 128 / g.group : 0;
  p.early = early ? 1 : 0;
  p.status = g.status;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(QG_THREADS);
  cfg.dynamicSmemBytes = QG_SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // About one CTA per SM, at least 4 stages each.
  const int stages = ceil_div(p.c, 64) + ceil_div(p.c2, 64);
  const int most = std::max(1, std::min({8, num_sms() / (p.ni * p.nj), stages / 4}));
  return g.dec ? run_qgemm<1>(cfg, &attr[1], ta, ta2, tb2, p, most) : run_qgemm<0>(cfg, &attr[1], ta, ta2, tb2, p, most);
}

}  // namespace slim
