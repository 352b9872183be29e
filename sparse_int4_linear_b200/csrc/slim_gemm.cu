// Dense bf16 products C = A B^T with fp32 accumulators in tensor memory
// (tcgen05.mma kind::f16), for operands in any of the layouts the backward
// pass meets (see slim_gemm.h).
//
// A CTA (CG = 1) owns 128 output rows, a pair of CTAs on an SM pair (CG = 2,
// tcgen05 cta_group::2) 256, and up to 256 output columns.  The contraction
// runs in stages of 64 columns: one producer thread loads both operands by
// tensor copies (128-byte swizzle; operands whose rows are contiguous land as
// MN-major tiles, the others K-major), one thread issues the MMAs, four warps
// write the accumulators out.  A product with few output tiles splits its
// contraction over a cluster of up to 8 CTAs, whose fp32 sums are added in
// rank order through distributed shared memory, so results do not depend on
// timing.
//
// The pairs are persistent and their sums alternate between two halves of
// tensor memory, so that the tensor cores work on the next tile while the last
// one is written (linear backward 11008 x 4096, rank 128, 2048 tokens 198 -> 181
// us, dense 4-bit 4096 x 11008, 1024 tokens 101 -> 93, among other calls with cold
// L2; one after the other they run under the power cap, 213 and 111).
//
// Bound by the tensor cores for the large products (a pair's stage is 256 x
// 256 x 64 MACs = 512 cycles against 32 KB of copies per CTA): dX of 2048
// tokens, 22016 to 4096, 254 us = 1.45 PFLOP/s on B200.  Of 4096 to 11008 (one
// launch by itself, cold) the tensor pipe is active for 86 % of an SM's cycles.  Bound by latency for
// the rank-r ones (a launch, the first copies, a cluster's sums: 5 to 8 us
// each), which therefore share launches.
#include <cooperative_groups.h>

#include <algorithm>

#include "slim_gemm.h"
#include "slim_internal.h"
#include "slim_tcgen05.cuh"

namespace slim {
namespace {

constexpr int GM_ROWS = 128;              // output rows of a CTA
constexpr int GM_THREADS = 192;           // warps 0-3 epilogue, 4 producer, 5 MMA
constexpr int GM_ABYTES = GM_ROWS * 128;  // A tile of a stage: 128 rows x 64 columns
constexpr int GM_SMEM = 200 * 1024;       // ring budget
constexpr int GM_MAX_STAGES = 8;
constexpr int GM_TMEM = 256;

struct GemmParams {
  int I, J, jt;
  int nst;                     // ring stages
  int nseg, clen[2];
  int a_mn, b_mn;              // operand tiles are MN-major
  int a_3d, b_3d;              // ... and come in one copy (see three_d)
  int img[2], blk_lines[2], cblk_lines[2];   // B of segment s is an image (1 kImage, 2 kImageK)
  int mode, n_groups, group_end[SLIM_MAX_GROUPS], r16;
  int cta0;                    // the product's first CTA in the grid
  int ni, nj;                  // output tiles along rows (CG = 2: of a pair) and columns
  int tiles;                   // ... and over the groups
  uint16_t* C;
  int ldc, jb, jr;
  int32_t* status;
};

// The products of a launch.
struct GemmProblem {
  CUtensorMap ta0, tb0, ta1, tb1;
  GemmParams p;
};
struct GemmBatch {
  GemmProblem pr[kGemmBatch];
  int n;
  int splits;                  // CTAs of a cluster sharing a contraction (CG = 1)
  int early;
};

__device__ __forceinline__ uint64_t mn128_desc(uint32_t saddr) {
  // MN-major, 128-byte swizzle: lines of 64 rows, 8-line groups 1024 B apart
  // along the contraction (SBO), the next 64 rows 8 KB on (LBO).
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(8192 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

template <int CG>
__device__ __forceinline__ void mma_plain(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, int acc) {
  if (CG == 2)
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(acc)
                 : "memory");
  else
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(acc)
                 : "memory");
}

// Tensor copies into this CTA's shared memory that complete on the barrier at
// shared::cluster address `bar` (of either CTA of a pair).
template <int CG>
__device__ __forceinline__ void load2(uint32_t dst, const CUtensorMap* m, int x, int y, uint32_t bar) {
  if (CG == 2)
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
                 "[%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar)
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
                 "[%4];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}
template <int CG>
__device__ __forceinline__ void load3(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar) {
  if (CG == 2)
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
                 "[%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
                 "[%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
                 : "memory");
}

// N sums of one output row, from column j on (col0: the batch's first column).
template <int N>
__device__ __forceinline__ void store_row(const GemmParams& p, int i, int j, const float (&v)[N], int col0, bool bad) {
  if (i >= p.I || j >= p.J) return;
  uint16_t* row = p.C + (size_t)i * p.ldc;
  constexpr int V = N < 8 ? 4 : 8;   // columns of a store
  if (j + N <= p.J && (p.ldc & (V - 1)) == 0 && p.jb == p.jr && (col0 & (V - 1)) == 0) {
#pragma unroll
    for (int q = 0; q < N / V; ++q) {
      union {
        __nv_bfloat162 h[V / 2];
        uint4 v8;
        uint2 v4;
      } o;
#pragma unroll
      for (int c = 0; c < V / 2; ++c) {
        o.h[c] = __floats2bfloat162_rn(v[V * q + 2 * c], v[V * q + 2 * c + 1]);
        if (bad) o.h[c] = __halves2bfloat162(__ushort_as_bfloat16(0x7FC0), __ushort_as_bfloat16(0x7FC0));
      }
      if constexpr (V == 8) reinterpret_cast<uint4*>(row + col0 + j)[q] = o.v8;
      else reinterpret_cast<uint2*>(row + col0 + j)[q] = o.v4;
    }
  } else {
    int blk = (col0 + j) / p.jb, in = (col0 + j) - blk * p.jb;
#pragma unroll
    for (int q = 0; q < N; ++q) {
      if (in >= p.jb) {
        in -= p.jb;
        ++blk;
      }
      if (j + q < p.J && in < p.jr)
        row[(size_t)blk * p.jr + in] = bad ? (uint16_t)0x7FC0 : __bfloat16_as_ushort(__float2bfloat16_rn(v[q]));
      ++in;
    }
  }
}

// A warp's 32 rows x 32 columns whose rows are not written in whole 16-byte
// pieces (an odd pitch, columns left out, the last ones): by way of shared
// memory, so that the lanes write a row's columns side by side and not each
// its own row (4096 x 4099, 1024 tokens 78 -> 44 us a dense 4-bit call, against
// 39 for an even pitch; 1024 x 20001 240 -> 86).
constexpr int kRaggedWords = 32 * 17;
__device__ __forceinline__ void store_ragged(const GemmParams& p, uint32_t* st, int i, int j, const float (&v)[32],
                                             int col0, bool bad) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
    st[lane * 17 + q] = *reinterpret_cast<const uint32_t*>(&h);
  }
  __syncwarp();
  const int col = col0 + j + lane, blk = col / p.jb, in = col - blk * p.jb;
  if (j + lane < p.J && in < p.jr) {
    const uint16_t* from = reinterpret_cast<const uint16_t*>(st) + lane;
    uint16_t* to = p.C + (size_t)i * p.ldc + (size_t)blk * p.jr + in;
    const int n = min(32, p.I - i);
#pragma unroll 8
    for (int r = 0; r < n; ++r, to += p.ldc) *to = bad ? (uint16_t)0x7FC0 : from[r * 34];
  }
  __syncwarp();   // (the next tensor-memory load is the whole warp's)
}

// One output tile.  Row tiles fastest, then columns, then groups (kGroupC).
struct GemmTile {
  int i0, j0;          // this CTA's first output row, the tile's first output column
  int cbeg, clen0;     // the first pair of operands' contraction
  int a_row0, col0;
  int S0, S;           // stages of 64 columns: of the first pair of operands, of both
};
template <int CG>
__device__ __forceinline__ GemmTile gemm_tile(const GemmParams& p, int tile, uint32_t rank) {
  GemmTile t;
  t.i0 = tile % p.ni * GM_ROWS * CG + (int)rank * GM_ROWS;
  t.j0 = tile / p.ni % p.nj * p.jt;
  int grp = tile / (p.ni * p.nj);
  if (p.mode == (int)GemmMode::kGroupJ) {
    grp = 0;
    while (grp + 1 < p.n_groups && t.j0 >= p.group_end[grp]) ++grp;
  }
  t.cbeg = p.mode == (int)GemmMode::kGroupC && grp > 0 ? p.group_end[grp - 1] : 0;
  t.clen0 = p.mode == (int)GemmMode::kGroupC ? p.group_end[grp] - t.cbeg : p.clen[0];
  t.a_row0 = t.i0 + (p.mode == (int)GemmMode::kGroupJ ? grp * p.r16 : 0);
  t.col0 = p.mode == (int)GemmMode::kGroupC ? grp * p.r16 : 0;
  t.S0 = ceil_div(t.clen0, 64);
  t.S = t.S0 + (p.nseg > 1 ? ceil_div(p.clen[1], 64) : 0);
  return t;
}

template <int CG>
__global__ void __launch_bounds__(GM_THREADS, 1)
    k_gemm(const __grid_constant__ GemmBatch batch) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  int which = 0;
  while (CG == 1 && which + 1 < batch.n && (int)blockIdx.x >= batch.pr[which + 1].p.cta0) ++which;   // (a pair's is alone)
  const GemmProblem& pb = batch.pr[which];
  const GemmParams& p = pb.p;
  const bool early = batch.early != 0;
  const int jc = p.jt / CG;                       // operand B rows this CTA holds
  const int bbytes = jc * 128, sbytes = GM_ABYTES + bbytes;
  const int NST = p.nst;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + NST * sbytes);   // rank 0's count both CTAs' copies
  uint64_t* empty = full + NST;
  uint64_t* acc_full = empty + NST;       // [2]
  uint64_t* acc_empty = acc_full + 2;     // [2], rank 0's: the pair's 8 epilogue warps have read the sums
  uint64_t* done = acc_empty + 2;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(done + 1) + 1;
  // Where ragged rows are staged: the idle rings, or (the rings of a pair
  // already fill with its next tile) memory of their own.
  uint32_t* ragged = reinterpret_cast<uint32_t*>(CG == 2 ? reinterpret_cast<uint8_t*>(done + 3) : smem);
  float* red = reinterpret_cast<float*>(smem);    // [128][jt + 4] fp32 sums of a rank, in the idle rings

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const int SP = CG == 2 ? 2 : batch.splits;               // CTAs of a cluster
  const int split = CG == 2 ? 0 : (int)cluster_rank();
  // A pair walks the tiles (one pair per two SMs); a cluster of single CTAs has
  // one.  A pair's sums alternate between two halves of tensor memory, so that
  // the next tile's products run while the epilogue writes the last one's.
  const int tile0 = CG == 2 ? (int)blockIdx.x >> 1 : ((int)blockIdx.x - p.cta0) / SP;
  const int tile_end = CG == 2 ? p.tiles : tile0 + 1, tile_step = CG == 2 ? (int)gridDim.x >> 1 : 1;
  const int parts = CG == 2 ? 1 : SP;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * NST + 5; ++i) mbar_init(full + i, full + i == acc_empty || full + i == acc_empty + 1 ? 8 : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    if (CG == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32((const void*)tmem_slot)),
                   "r"(CG * GM_TMEM)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32((const void*)tmem_slot)),
                   "r"(CG * GM_TMEM)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 4) {
    // ---------------------------------------------------------------- producer
    // (The whole warp walks the loop, one elected lane issues, as below.)
    const bool one = elect_one();
    if (one) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&pb.ta0)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&pb.tb0)) : "memory");
      if (p.nseg > 1) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&pb.ta1)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&pb.tb1)) : "memory");
      }
    }
    __syncwarp();
    if (!early) pdl_wait();   // the operands were written by the previous kernels on the stream
    pdl_launch_dependents();    // all that came before the previous kernel has completed
    const uint32_t full0 = CG == 2 ? cluster_addr(full, 0) : smem_u32(full);
    const uint32_t sm = smem_u32(smem);
    int iss = 0, st = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (int tile = tile0; ok && tile < tile_end; tile += tile_step) {
      const GemmTile t = gemm_tile<CG>(p, tile, rank);
      const int a_row0 = t.a_row0, jb = t.j0 + (int)rank * jc;
      const int u0 = (int)((long long)split * t.S / parts), u1 = (int)((long long)(split + 1) * t.S / parts);
      for (int u = u0; u < u1; ++u) {
        if (!__all_sync(0xffffffffu, pwait(empty + st, ph, abort_flag))) {
          ok = false;
          break;
        }
        const int seg = u < t.S0 ? 0 : 1;
        const int c = (seg ? u - t.S0 : u) * 64, ca = c + (seg ? 0 : t.cbeg);
        if (!dcheck(c < (seg ? p.clen[1] : t.clen0), p.status)) {
          *abort_flag = 1;
          ok = false;
          break;
        }
        ++iss;
        if (one) {
          const uint32_t as = sm + (uint32_t)(st * sbytes), bs = as + GM_ABYTES, bar = full0 + 8u * (uint32_t)st;
          if (rank == 0) mbar_expect_tx(full + st, (uint32_t)(CG * sbytes));
          const CUtensorMap* ma = seg ? &pb.ta1 : &pb.ta0;
          const CUtensorMap* mb = seg ? &pb.tb1 : &pb.tb0;
          if (!p.a_mn) load2<CG>(as, ma, ca, a_row0, bar);
          else if (p.a_3d) load3<CG>(as, ma, 0, ca, a_row0 >> 6, bar);
          else {
            load2<CG>(as, ma, a_row0, ca, bar);
            load2<CG>(as + 8192, ma, a_row0 + 64, ca, bar);
          }
          if (!p.b_mn) {
            if (p.img[seg]) load2<CG>(bs, mb, 0, (ca >> 6) * p.blk_lines[seg] + jb, bar);
            else load2<CG>(bs, mb, ca, jb, bar);
          } else if (p.img[seg]) {
            const int cl = p.cblk_lines[seg] ? (ca >> 7) * p.cblk_lines[seg] + (ca & 127) : ca;
            for (int b = 0; b < jc / 64; ++b)
              load2<CG>(bs + b * 8192, mb, 0, (jb / 64 + b) * p.blk_lines[seg] + cl, bar);
          } else if (p.b_3d) {
            load3<CG>(bs, mb, 0, ca, jb >> 6, bar);
          } else {
            for (int b = 0; b < jc / 64; ++b) load2<CG>(bs + b * 8192, mb, jb + 64 * b, ca, bar);
          }
        }
        __syncwarp();
        if (++st == NST) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
    if (lane == 0) {
      if (*abort_flag) {
        // Let the copies still in flight land: rank 0's barriers count both
        // CTAs' bytes, rank 1 gives its own a fixed grace period.
        const long long t0 = clock64(), deadline = t0 + kWaitBudgetCycles;
        if (rank == 0) {
          for (int q = max(0, iss - NST); q < iss; ++q) drain_phase(full + q % NST, (q / NST) & 1, deadline);
        } else {
          while (clock64() - t0 < 200000) {
          }
        }
      }
    }
  } else if (warp == 5) {
    // ---------------------------------------------------------------- MMA issue (both CTAs)
    // The whole warp walks the loop, so that its operands stay in uniform
    // registers; one elected lane issues.
    if (rank == 0) {
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)p.a_mn << 15) | ((uint32_t)p.b_mn << 16) |
                             ((uint32_t)(p.jt >> 3) << 17) | ((uint32_t)((GM_ROWS * CG) >> 4) << 24);
      const uint32_t sm = smem_u32(smem);
      const uint64_t ad0 = p.a_mn ? mn128_desc(sm) : sw128_desc(sm);
      const uint64_t bd0 = p.b_mn ? mn128_desc(sm + GM_ABYTES) : sw128_desc(sm + GM_ABYTES);
      const uint32_t ak = (p.a_mn ? 2048 : 32) >> 4, bk = (p.b_mn ? 2048 : 32) >> 4;   // 16 columns on
      const bool one = elect_one();
      int st = 0, n = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = tile0; ok && tile < tile_end; tile += tile_step, ++n) {
        const GemmTile t = gemm_tile<CG>(p, tile, rank);
        const int u0 = (int)((long long)split * t.S / parts), u1 = (int)((long long)(split + 1) * t.S / parts);
        const uint32_t acc = tmem + (uint32_t)((n & 1) * GM_TMEM);
        if (CG == 2) ok = __all_sync(0xffffffffu, pwait(acc_empty + (n & 1), ((n >> 1) & 1) ^ 1, abort_flag));
        tc_fence_after();
        for (int u = u0; ok && u < u1; ++u) {
          if (!__all_sync(0xffffffffu, pwait(full + st, ph, abort_flag))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int left = u < t.S0 ? t.clen0 - u * 64 : p.clen[1] - (u - t.S0) * 64;
          const uint32_t off = (uint32_t)(st * sbytes) >> 4;
          if (one) {
            if (left > 48) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_plain<CG>(acc, ad0 + off + kk * ak, bd0 + off + kk * bk, idesc, (u - u0) | kk);
            } else {
              for (int kk = 0; kk * 16 < left; ++kk)
                mma_plain<CG>(acc, ad0 + off + kk * ak, bd0 + off + kk * bk, idesc, (u - u0) | kk);
            }
            if (CG == 2) tc_commit2(empty + st);
            else tc_commit(empty + st);
          }
          __syncwarp();
          if (++st == NST) {
            st = 0;
            ph ^= 1u;
          }
        }
        // Always on this CTA's barrier, on the peer's only for complete sums.
        if (one) {
          if (CG == 2) tc_commit2_mask(acc_full + (n & 1), ok ? 3 : 1);
          else tc_commit(acc_full);
        }
        __syncwarp();
      }
      if (CG == 2) {
        // No MMA is in flight when tensor memory is freed.
        if (one) tc_commit2_mask(done, 1);
        __syncwarp();
        mbar_wait(done, 0);
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    int n = 0;
    for (int tile = tile0; tile < tile_end; tile += tile_step, ++n) {
      const GemmTile t = gemm_tile<CG>(p, tile, rank);
      const int i0 = t.i0, j0 = t.j0, col0 = t.col0;
      const uint32_t acc = tmem + (uint32_t)((n & 1) * GM_TMEM);
      // (Of a single CTA the wait ends with its MMAs, complete or not.)
      const bool acc_ok = CG == 2 ? pwait(acc_full + (n & 1), (n >> 1) & 1, abort_flag) : mbar_wait(acc_full, 0);
      tc_fence_after();
      if (!early && n == 0) pdl_wait();   // the output may still be in use by earlier work on the stream
      // Warp-uniform: the tensor-memory loads are .sync.aligned.  A tile whose
      // sums are incomplete is written as NaN.
      const bool good = __all_sync(0xffffffffu, acc_ok && !*abort_flag);
      if (!good && lane == 0) {
        *abort_flag = 1;
        record_status(p.status, SLIM_ERR_TIMEOUT);
      }
      for (int c0 = 0; c0 < p.jt; c0 += 32) {
        uint32_t v[32];
        if (good) {
          tc_ld32(v, acc + ((uint32_t)(warp * 32) << 16) + (uint32_t)c0);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        } else {
#pragma unroll
          for (int q = 0; q < 32; ++q) v[q] = 0u;
        }
        float f[32];
#pragma unroll
        for (int q = 0; q < 32; ++q) f[q] = __uint_as_float(v[q]);
        if (CG == 1 && SP > 1) {
          // Sums of this rank, rows padded by 4 floats (a quarter-warp's 16-byte
          // stores hit distinct banks).  The rings are idle: every copy has
          // been consumed by a completed MMA.
          float4* r = reinterpret_cast<float4*>(red + (size_t)(warp * 32 + lane) * (p.jt + 4) + c0);
#pragma unroll
          for (int q = 0; q < 8; ++q) r[q] = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
        } else {
          const int i = i0 + warp * 32, j = j0 + c0;
          if (j + 32 <= p.J && (p.ldc & 7) == 0 && p.jb == p.jr && (col0 & 7) == 0) store_row<32>(p, i + lane, j, f, col0, !good);
          else store_ragged(p, ragged + warp * kRaggedWords, i, j, f, col0, !good);
        }
      }
      if (CG == 2) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(cluster_addr(acc_empty + (n & 1), 0));
      }
    }
  }
  if (CG == 1 && SP > 1) {
    const GemmTile t = gemm_tile<CG>(p, tile0, 0);
    const int i0 = t.i0, j0 = t.j0, col0 = t.col0;
    // Rank c adds rows [rows c / SP, rows (c + 1) / SP) over the ranks, in rank
    // order; NaN if a wait of any rank gave up.
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    tc_fence_before();
    cluster.sync();
    bool bad = false;
    for (int q = 0; q < SP; ++q) bad = bad || *cluster.map_shared_rank(const_cast<int*>(abort_flag), q) != 0;
    // (A warp reads whole lines of a rank at a time: with 8 columns a thread,
    // half of every line a read, the sums of 8 ranks took twice as long.  Two
    // places a thread keep enough reads in flight.)
    constexpr int U = 2;
    const int rows = min(GM_ROWS, p.I - i0), r0 = split * rows / SP, r1 = (split + 1) * rows / SP, per = p.jt / 4;
    const int lp = __ffs(per) - 1, total = (r1 - r0) * per;   // (a single CTA's jt is a power of two)
    for (int e0 = threadIdx.x; e0 < total; e0 += U * GM_THREADS) {
      float4 a[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int e = e0 + u * GM_THREADS;
        const size_t off = (size_t)(r0 + (e >> lp)) * (p.jt + 4) + (e & (per - 1)) * 4;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < SP && e < total) a[u][q] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(red, q) + off);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int e = e0 + u * GM_THREADS;
        if (e >= total) break;
        float f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < SP) {
            f[0] += a[u][q].x; f[1] += a[u][q].y; f[2] += a[u][q].z; f[3] += a[u][q].w;
          }
        store_row<4>(p, i0 + r0 + (e >> lp), j0 + (e & (per - 1)) * 4, f, col0, bad);
      }
    }
    cluster.sync();
  }
  // An early kernel completes no earlier than the one before it: one thread
  // of the grid waits (all the others give their SM up).
  if (early && threadIdx.x == 0 && blockIdx.x == 0) pdl_wait();
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (CG == 2) cluster_sync_all();   // neither CTA leaves while the other may touch its memory
  if (warp == 5) {
    tc_fence_after();
    if (CG == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(CG * GM_TMEM) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(CG * GM_TMEM) : "memory");
  }
}

// What planning needs to know of a product.
struct GemmShape {
  int I, J, groups;
  long long c_min, c_max;      // shortest and longest contraction of a group
  bool b_rows;                 // B is row-major, the contraction in one piece
};
GemmShape gemm_shape(const GemmCall& g) {
  GemmShape h;
  h.I = g.I;
  h.J = g.J;
  h.groups = g.mode == GemmMode::kGroupC ? g.n_groups : 1;
  h.c_min = h.c_max = g.a[0].c + (g.nseg > 1 ? g.a[1].c : 0);
  if (g.mode == GemmMode::kGroupC) {
    h.c_max = 0;
    for (int q = 0; q < h.groups; ++q) {
      const long long c = g.group_end[q] - (q ? g.group_end[q - 1] : 0);
      h.c_min = std::min(h.c_min, c);
      h.c_max = std::max(h.c_max, c);
    }
  }
  h.b_rows = g.b[0].layout == GemmLayout::kRowMajor && g.nseg == 1;
  return h;
}

// Columns of a pair's tile when pairs of CTAs, each on 256 rows, fill three
// quarters of the SMs by themselves, else 0.  256 columns, or for a row-major
// B the width whose waves of pairs finish first (the constant: a tile's own
// cost in columns; 0, 64 and 128 there are within 2 % at 4096 x 11008, 400 and 1024
// tokens, and 11008 x 4096, 2048).  Measured, pairs against single CTAs, us a call:
// linear backward 11008 x 4096, rank 128, 2048 tokens 181 and 209, 8192 x 8192, 512
// tokens 94 and 103, dense 4-bit 4096 x 11008, 1024 tokens 95 and 119, 1024 x 20000
// 55 and 74.  With 64 CTAs in pairs (left to single CTAs), 4096 x 4096, 512 tokens,
// 36.0 and 37.2, its backward pass 46.3 and 46.6.  Against it: the backward pass of
// 8192 x 1024, rank 256, 500 tokens, whose dX has 128 CTAs in pairs of 20 stages
// each: 45 and 40.
int pair_width(const GemmShape& h) {
  const int nsm = num_sms();
  const long long rows = (long long)ceil_div(h.I, 256) * h.groups;
  if (h.I <= 128 || h.J <= 128 || rows * ceil_div(h.J, 256) * 2 * 4 < nsm * 3) return 0;
  int jt = 256;
  long long best = -1;
  for (int w = 256; w >= (h.b_rows ? 192 : 256); w -= 32) {
    const long long waves = (rows * ceil_div(h.J, w) * 2 + nsm - 1) / nsm;
    if (best < 0 || waves * (w + 64) < best) {
      best = waves * (w + 64);
      jt = w;
    }
  }
  return jt;
}

// Single CTAs of 128 rows and 64 to 256 columns (narrower ones as long as even
// the largest split would leave half of the SMs idle), with the contraction
// split over a cluster so that about one CTA per SM runs (at least 4 stages a
// CTA).
struct SinglePlan {
  int jt[kGemmBatch];
  int splits;
};
SinglePlan single_plan(const GemmShape* h, int n) {
  SinglePlan pl;
  const int nsm = num_sms();
  long long most = 8;
  for (int q = 0; q < n; ++q) {
    pl.jt[q] = h[q].J <= 64 ? 64 : h[q].J <= 128 ? 128 : 256;
    most = std::max(1ll, std::min(most, (h[q].c_min + 63) / 64 / 4));
  }
  auto tiles = [&]() {
    long long t = 0;
    for (int q = 0; q < n; ++q) t += (long long)ceil_div(h[q].I, 128) * ceil_div(h[q].J, pl.jt[q]) * h[q].groups;
    return t;
  };
  for (;;) {
    int widest = 0;
    for (int q = 1; q < n; ++q)
      if (pl.jt[q] > pl.jt[widest]) widest = q;
    if (tiles() * most >= (most > 1 ? nsm * 3 / 4 : nsm / 2) || pl.jt[widest] <= 64) break;
    pl.jt[widest] /= 2;
  }
  pl.splits = (int)std::max(1ll, std::min(nsm / tiles(), most));
  return pl;
}

// A column-major operand whose rows fill whole lines of 64 is read as
// [rows / 64][c][64], so that a tile of several lines is one copy.  (Not
// kGroupJ's A, whose tiles may start inside a line.)
bool three_d(const GemmOperand& o) { return o.layout == GemmLayout::kColMajor && o.rows % 64 == 0; }

CUresult encode_operand(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* m, const GemmOperand& o, int box_rows,
                        bool d3) {
  if (d3) {
    const cuuint64_t d3[3] = {64, (cuuint64_t)o.c, (cuuint64_t)(o.rows / 64)};
    const cuuint64_t s3[2] = {(cuuint64_t)o.pitch * 2, 128};
    const cuuint32_t b3[3] = {64, 64, (cuuint32_t)(box_rows / 64)}, e3[3] = {1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(o.base), d3, s3, b3, e3,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  const cuuint32_t estr[2] = {1, 1};
  cuuint64_t dims[2], strides[1];
  cuuint32_t box[2];
  CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  if (o.layout == GemmLayout::kImage || o.layout == GemmLayout::kImageK) {
    dims[0] = 64;
    dims[1] = (cuuint64_t)o.img_lines;
    strides[0] = 128;
    box[0] = 64;
    box[1] = o.layout == GemmLayout::kImage ? 64 : (cuuint32_t)box_rows;
    sw = CU_TENSOR_MAP_SWIZZLE_NONE;   // the bytes are already swizzled
  } else {
    const bool rm = o.layout == GemmLayout::kRowMajor;
    dims[0] = (cuuint64_t)(rm ? o.c : o.rows);
    dims[1] = (cuuint64_t)(rm ? o.rows : o.c);
    strides[0] = (cuuint64_t)o.pitch * 2;
    box[0] = 64;
    box[1] = rm ? (cuuint32_t)box_rows : 64;
  }
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(o.base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

template <int CG>
cudaError_t run_gemm(cudaLaunchConfig_t& cfg, const GemmBatch& b) {
  cudaError_t e = ensure_func_attrs(reinterpret_cast<const void*>(k_gemm<CG>), cfg.dynamicSmemBytes);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, k_gemm<CG>, b);
}

}  // namespace

bool gemms_fit_together(const GemmCall* g, int n) {
  if (n > kGemmBatch) return false;
  GemmShape h[kGemmBatch];
  for (int q = 0; q < n; ++q) {
    h[q] = gemm_shape(g[q]);
    if (pair_width(h[q])) return false;
  }
  const int together = single_plan(h, n).splits;
  for (int q = 0; q < n; ++q)
    if (single_plan(h + q, 1).splits > 2 * together) return false;
  return true;
}

cudaError_t launch_gemms(const GemmCall* g, int n, bool early, cudaStream_t s) {
  auto encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  GemmShape h[kGemmBatch];
  for (int q = 0; q < n; ++q) h[q] = gemm_shape(g[q]);
  const int wide = n == 1 ? pair_width(h[0]) : 0, cg = wide ? 2 : 1;
  SinglePlan pl = single_plan(h, n);
  if (wide) {
    pl.jt[0] = wide;
    pl.splits = 1;
  }
  GemmBatch b = {};
  b.n = n;
  b.early = early ? 1 : 0;
  size_t smem = 0;
  long long tiles = 0;
  for (int k = 0; k < n; ++k) {
    GemmProblem& pr = b.pr[k];
    GemmParams& p = pr.p;
    const GemmCall& c = g[k];
    const int jc = pl.jt[k] / cg;
    p.I = c.I;
    p.J = c.J;
    p.jt = pl.jt[k];
    p.nseg = c.nseg;
    p.a_mn = c.a[0].layout == GemmLayout::kColMajor;
    p.b_mn = c.b[0].layout == GemmLayout::kColMajor || c.b[0].layout == GemmLayout::kImage;
    p.a_3d = three_d(c.a[0]) && c.mode != GemmMode::kGroupJ;
    p.b_3d = three_d(c.b[0]);
    CUtensorMap* maps[4] = {&pr.ta0, &pr.tb0, &pr.ta1, &pr.tb1};
    for (int q = 0; q < c.nseg; ++q) {
      p.clen[q] = (int)c.a[q].c;
      p.img[q] = c.b[q].layout == GemmLayout::kImage ? 1 : c.b[q].layout == GemmLayout::kImageK ? 2 : 0;
      p.blk_lines[q] = c.b[q].blk_lines;
      p.cblk_lines[q] = c.b[q].cblk_lines;
      if (encode_operand(encode, maps[2 * q], c.a[q], GM_ROWS, q == 0 && p.a_3d) != CUDA_SUCCESS ||
          encode_operand(encode, maps[2 * q + 1], c.b[q], jc, q == 0 && p.b_3d) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    }
    p.mode = (int)c.mode;
    p.n_groups = c.n_groups;
    for (int q = 0; q < SLIM_MAX_GROUPS; ++q) p.group_end[q] = c.group_end[q];
    p.r16 = c.r16;
    p.C = c.C;
    p.ldc = c.ldc;
    p.jb = c.jb;
    p.jr = c.jr;
    p.status = c.status;
    p.ni = ceil_div(c.I, GM_ROWS * cg);
    p.nj = ceil_div(c.J, p.jt);
    p.tiles = p.ni * p.nj * h[k].groups;
    tiles += p.tiles;
    // No more stages than a CTA's share of the contraction has, but room for a
    // rank's sums.
    const int sbytes = GM_ABYTES + jc * 128;
    static_assert(4 * (GM_ABYTES + 256 * 128) >= GM_ROWS * (256 + 4) * 4 &&
                      6 * (GM_ABYTES + 128 * 128) >= GM_ROWS * (128 + 4) * 4 &&
                      8 * (GM_ABYTES + 64 * 128) >= GM_ROWS * (64 + 4) * 4,
                  "a rank's sums fit its rings");
    const int share = (int)std::min<long long>(GM_MAX_STAGES, (h[k].c_max / 64 + 2) / pl.splits + 1);
    const int red = pl.splits > 1 ? ceil_div(GM_ROWS * (p.jt + 4) * 4, sbytes) : 1;
    p.nst = std::min({GM_MAX_STAGES, GM_SMEM / sbytes, std::max({2, share, red})});
    smem = std::max(smem, (size_t)p.nst * sbytes + (2 * p.nst + 5) * 8 + 16 + 1024 + (cg == 2 ? 4 * kRaggedWords * 4 : 0));
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(GM_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cg == 2) {
    cudaError_t e = ensure_func_attrs(reinterpret_cast<const void*>(k_gemm<2>), smem);
    if (e != cudaSuccess) return e;
    // As many pairs as run at once, or one per tile.
    cfg.gridDim = dim3(2);
    const int pairs = std::max(1, max_clusters(reinterpret_cast<const void*>(k_gemm<2>), cfg));
    cfg.gridDim = dim3((unsigned)(2 * std::min<long long>(tiles, pairs)));
    return run_gemm<2>(cfg, b);
  }
  cudaError_t e = ensure_func_attrs(reinterpret_cast<const void*>(k_gemm<1>), smem);
  if (e != cudaSuccess) return e;
  // The largest split whose clusters all run at once (a cluster left for a
  // second wave would double the kernel's time).
  for (b.splits = pl.splits; b.splits > 1; --b.splits) {
    attr[1].val.clusterDim.x = b.splits;
    cfg.gridDim = dim3(b.splits);
    if (tiles <= max_clusters(reinterpret_cast<const void*>(k_gemm<1>), cfg)) break;
  }
  attr[1].val.clusterDim.x = b.splits;
  int at = 0;
  for (int k = 0; k < n; ++k) {
    b.pr[k].p.cta0 = at;
    at += b.pr[k].p.ni * b.pr[k].p.nj * h[k].groups * b.splits;
  }
  cfg.gridDim = dim3(at);
  cfg.numAttrs = b.splits > 1 ? 2 : 1;
  return run_gemm<1>(cfg, b);
}

}  // namespace slim
