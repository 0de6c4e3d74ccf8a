// cross_few.cu -- cross attention of few query columns (bf16): generated rows,
// a handful of candidates.  Bound by reading K and V once from HBM.
//
// An item is up to 8 NT query columns of one (sequence, KV head); a tile is one
// block of 16 keys, which a warp takes whole:
//   S^T[16 keys x 8]  = K q^T           mma.sync m16n8k16, fp32 accumulation
//   P = 2^(S scale log2 e - m)          online per warp, bf16 for the product (as
//                                       V is: an MMA takes one type), summed in
//                                       fp32 before that rounding
//   O^T[D x 8]       += V^T P
// for each of the NT groups of 8 columns.  (With keys on the M side the work is
// proportional to the columns there are; 128 query columns on the M side of a
// tcgen05 MMA took 150 us where this takes what the loads take.)
// A CTA is a worker; its 8 warps take a piece's blocks in turn, each through a
// ring of its own that it refills itself by 2-D tensor loads (128-byte swizzle),
// across pieces too, so that loads stay in flight while a piece ends.  At a
// piece's end the warps' states are added up through shared memory.
#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cross_attention.h"
#include "ptx.cuh"

namespace pa {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kKeys = kBlockSize;
constexpr int kExtra = 16;  // what an item costs besides its blocks, in blocks of a warp (measured: 8 to 24 alike)
constexpr float kGrow = 8.f;  // log2 growth of a maximum before O is rescaled

template <int D>
struct Shape {
  static constexpr int TILE = kKeys * D * 2;          // bytes of a K or V block
  static constexpr int SLOT = 2 * TILE;
  static constexpr int DEPTH = D == 128 ? 3 : 6;      // 192 KB of loads in flight
  static constexpr int SMEM = 1024 + kWarps * DEPTH * SLOT + kWarps * 8 * D * 4;
};

// 2^x, approximate, 0 below the smallest normal number: of a weight (at most 2^8) that
// is rounded to bf16, and of a factor between two maxima
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1) cross_few_kernel(const __grid_constant__ CrossArgs a) {
  using C = Shape<D>;
  constexpr int COLS = 8 * NT, MT = D / 16, DEPTH = C::DEPTH;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* const sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  float* const s_o = reinterpret_cast<float*>(sm + kWarps * DEPTH * C::SLOT);  // [kWarps][8][D], dim d of column c at
                                                                               // d ^ (c / 2 % 4 * 8)
  // q fragments in registers, or where those would spill in shared memory
  constexpr bool Q_SMEM = NT * D >= 512;
  uint2* const s_q = reinterpret_cast<uint2*>(s_o);
  __shared__ __align__(8) uint64_t s_full[kWarps][DEPTH];
  __shared__ int s_flag[kWarps][DEPTH];     // the slot's block id is bad
  __shared__ float2 s_ml[kWarps][8];
  __shared__ int s_bad[kWarps];
  __shared__ int s_abort;
  __shared__ CrossTotal s_total;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, tq = lane & 3;   // MMA fragments: row g (and g + 8), columns 2 tq, 2 tq + 1
  const uint32_t full0 = smem_addr(&s_full[warp][0]);
  const uint32_t slot0 = smem_addr(sm) + warp * DEPTH * C::SLOT;

  if (lane == 0) {
    if (warp == 0) {
      prefetch_tensormap(&a.tm_k);
      prefetch_tensormap(&a.tm_v);
    }
    for (int i = 0; i < DEPTH; ++i) mbar_init(full0 + 8 * i, 1);
    if (warp == 0) s_abort = 0;
    fence_barrier_init();
  }
  const CrossShare share = cross_share<kThreads>(a, COLS, kKeys, kExtra, &s_total);  // (synchronises the CTA)

  // ---- this warp's loads: blocks t0 + warp, + 8, ... of every piece with keys
  CrossWalk ahead(a, share, COLS);
  CrossPiece ip{};
  bool more = true;
  int ib = 0, iend = 0, issued = 0;
  int ids = 0, id_first = 0;                // lane l: the id of block id_first + 8 l
  const uint64_t policy = l2_policy_evict_first();
  auto load_ids = [&]() {
    id_first = ib;
    const int b = ib + kWarps * lane;
    ids = b < iend ? __ldg(a.block_tables + static_cast<size_t>(ip.s) * a.max_blocks_per_seq + b) : 0;
  };
  auto issue = [&]() {
    while (more && ib >= iend) {
      more = ahead.next(a, COLS, kKeys, kExtra, &ip);
      if (more && ip.n > 0) {
        ib = ip.t0 + warp;
        iend = ip.t1;
        if (ib < iend) load_ids();
      }
    }
    if (!more) return;
    if (ib >= id_first + 32 * kWarps) load_ids();
    const int id = __shfl_sync(0xffffffffu, ids, (ib - id_first) / kWarps);
    const int sl = issued % DEPTH;
    const bool bad = id < 0 || id >= a.num_blocks;
    if (lane == 0) {
      const uint32_t bar = full0 + 8 * sl, dst = slot0 + sl * C::SLOT;
      s_flag[warp][sl] = bad;
      if (bad) {
        mbar_arrive(bar);
      } else {
        fence_proxy_async_smem();  // (rows of the slot may have been cleared)
        mbar_arrive_expect_tx(bar, C::SLOT);
        const int y = (id * a.num_kv_heads + ip.kvh) * kKeys;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          tma_load_2d_hint(dst + h * (kKeys * 128), &a.tm_k, h * 64, y, bar, policy);
          tma_load_2d_hint(dst + C::TILE + h * (kKeys * 128), &a.tm_v, h * 64, y, bar, policy);
        }
      }
    }
    ++issued;
    ib += kWarps;
  };
  for (int i = 0; i < DEPTH; ++i) issue();

  CrossWalk walk(a, share, COLS);
  CrossPiece p;
  int taken = 0;
  bool ok = true;
  while (ok && walk.next(a, COLS, kKeys, kExtra, &p)) {
    if (p.n == 0) {
      for (int i = tid; i < p.live * (D / 8); i += kThreads)
        reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) +
                                 (p.base(a) + cross_column(a, i / (D / 8))) * D)[i % (D / 8)] = make_uint4(0, 0, 0, 0);
      continue;
    }
    // q of column 8 nt + g as the B operand (dims 2 tq, + 1 and 2 tq + 8, + 9 of
    // each slice of 16); columns past the last repeat it and are not stored
    uint32_t qb[Q_SMEM ? 1 : NT][Q_SMEM ? 1 : MT][2];
    if constexpr (Q_SMEM) {
      // (the exchange area holds them while the piece lasts, in fragment order)
      __syncthreads();
      for (int i = tid; i < NT * MT * 32; i += kThreads) {
        const int nt = i / (MT * 32), k = i / 32 % MT;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(
            static_cast<const __nv_bfloat16*>(a.q) + (p.base(a) + cross_column(a, min(8 * nt + g, p.live - 1))) * D) + tq;
        s_q[i] = make_uint2(__ldg(src + 8 * k), __ldg(src + 8 * k + 4));
      }
      __syncthreads();
    }
#pragma unroll
    for (int nt = 0; nt < (Q_SMEM ? 0 : NT); ++nt) {
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          static_cast<const __nv_bfloat16*>(a.q) + (p.base(a) + cross_column(a, min(8 * nt + g, p.live - 1))) * D) + tq;
#pragma unroll
      for (int k = 0; k < MT; ++k) {
        qb[nt][k][0] = __ldg(src + 8 * k);
        qb[nt][k][1] = __ldg(src + 8 * k + 4);
      }
    }
    float o[NT][MT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int k = 0; k < MT; ++k) o[nt][k][0] = o[nt][k][1] = o[nt][k][2] = o[nt][k][3] = 0.f;
    }
    bool bad = false;
    for (int b = p.t0 + warp; b < p.t1; b += kWarps) {
      const int sl = taken % DEPTH;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(full0 + 8 * sl, (taken / DEPTH) & 1))) {
        ok = false;
        break;
      }
      ++taken;
      if (s_flag[warp][sl]) {
        bad = true;
      } else {
        const uint32_t kb = slot0 + sl * C::SLOT, vb = kb + C::TILE;
        const int rows = min(kKeys, p.n - b * kKeys);
        if (rows < kKeys) {
          // rows past the end hold stale data, and 0 x NaN would poison O
          for (int i = lane; i < (kKeys - rows) * (D / 8); i += 32) {
            const int r = rows + i / (D / 8), ch = i % (D / 8);
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vb + (ch >> 3) * (kKeys * 128) + r * 128 +
                                                                          ((ch & 7) << 4)),
                         "r"(0)
                         : "memory");
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        const int lr = lane & 7, lm = lane >> 3;  // ldmatrix: row within a matrix, matrix
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
        for (int k = 0; k < MT; ++k) {
          const int key = (lm & 1) * 8 + lr, ch = 2 * k + (lm >> 1);
          uint32_t af[4];
          ldmatrix_x4(kb + (ch >> 3) * (kKeys * 128) + key * 128 + (((ch ^ key) & 7) << 4), af);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (Q_SMEM) {
              const uint2 q2 = s_q[(nt * MT + k) * 32 + lane];
              mma_bf16_16816(s[nt], af, q2.x, q2.y);
            } else {
              mma_bf16_16816(s[nt], af, qb[nt][k][0], qb[nt][k][1]);
            }
          }
        }
        // s[nt]: keys g, g, g + 8, g + 8 x columns 2 tq, 2 tq + 1, 2 tq, 2 tq + 1
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = g + (e >> 1) * 8 < rows ? s[nt][e] * a.scale_log2 : -INFINITY;
          float mx[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
          // (a warp's first block, and the rare growth: the exact maximum)
          if (__any_sync(0xffffffffu, mx[0] > m[nt][0] + kGrow || mx[1] > m[nt][1] + kGrow)) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
              mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], off));
              mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], off));
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if (mx[c] > m[nt][c] + kGrow) {
                const float al = ex2(m[nt][c] - mx[c]);  // (0 while nothing was seen)
                m[nt][c] = mx[c];
                l[nt][c] *= al;
#pragma unroll
                for (int k = 0; k < MT; ++k) {
                  o[nt][k][c] *= al;
                  o[nt][k][c + 2] *= al;
                }
              }
            }
          }
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // (a column that saw only -inf: an offset of 0 keeps its weights at 0)
            const float base = m[nt][e & 1] == -INFINITY ? 0.f : m[nt][e & 1];
            w[e] = ex2(x[e] - base);
          }
          l[nt][0] += w[0] + w[2];
          l[nt][1] += w[1] + w[3];
          const __nv_bfloat162 p0 = __floats2bfloat162_rn(w[0], w[1]), p1 = __floats2bfloat162_rn(w[2], w[3]);
          pb[nt][0] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&p0));
          pb[nt][1] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&p1));
        }
#pragma unroll
        for (int k = 0; k < MT; ++k) {
          const int key = (lm >> 1) * 8 + lr, ch = 2 * k + (lm & 1);
          uint32_t af[4];
          ldmatrix_x4_trans(vb + (ch >> 3) * (kKeys * 128) + key * 128 + (((ch ^ key) & 7) << 4), af);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(o[nt][k], af, pb[nt][0], pb[nt][1]);
        }
      }
      __syncwarp();  // (the slot has been read)
      issue();
    }
    if (!ok && atomicExch(&s_abort, 1) == 0 && a.err_flag) atomicOr(a.err_flag, kErrTimeout);

    // ---- the piece's end: the warps' states, 8 columns at a time
    if (Q_SMEM) __syncthreads();  // (q has been read)
    if (lane == 0) s_bad[warp] = bad;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (8 * nt >= p.live) break;
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        l[nt][0] += __shfl_xor_sync(0xffffffffu, l[nt][0], off);
        l[nt][1] += __shfl_xor_sync(0xffffffffu, l[nt][1], off);
      }
      float* const dst = s_o + (warp * 8 + 2 * tq) * D;
#pragma unroll
      for (int k = 0; k < MT; ++k) {
        const int d = (16 * k + g) ^ (8 * tq);
        dst[d] = o[nt][k][0];
        dst[D + d] = o[nt][k][1];
        dst[d ^ 8] = o[nt][k][2];
        dst[D + (d ^ 8)] = o[nt][k][3];
      }
      if (g == 0) {
        s_ml[warp][2 * tq] = make_float2(m[nt][0], l[nt][0]);
        s_ml[warp][2 * tq + 1] = make_float2(m[nt][1], l[nt][1]);
      }
      __syncthreads();
      ok = *reinterpret_cast<volatile int*>(&s_abort) == 0;
      for (int u = tid; u < 8 * (D / 8); u += kThreads) {
        const int c = u % 8, ch = u / 8;
        if (8 * nt + c >= p.live) continue;
        float M = -INFINITY, L = 0.f, acc[8];
        bool any = false;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          M = fmaxf(M, s_ml[w][c].x);
          any |= s_bad[w] != 0;
        }
#pragma unroll
        for (int d = 0; d < 8; ++d) acc[d] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 ml = s_ml[w][c];
          const float f = ml.x == -INFINITY ? 1.f : ex2(ml.x - M);  // (nothing finite: zeros, or NaN)
          L = fmaf(f, ml.y, L);
          const float4* v = reinterpret_cast<const float4*>(s_o + (w * 8 + c) * D + ((8 * ch) ^ ((c >> 1 & 3) << 3)));
          const float4 v0 = v[0], v1 = v[1];
          acc[0] = fmaf(f, v0.x, acc[0]);
          acc[1] = fmaf(f, v0.y, acc[1]);
          acc[2] = fmaf(f, v0.z, acc[2]);
          acc[3] = fmaf(f, v0.w, acc[3]);
          acc[4] = fmaf(f, v1.x, acc[4]);
          acc[5] = fmaf(f, v1.y, acc[5]);
          acc[6] = fmaf(f, v1.z, acc[6]);
          acc[7] = fmaf(f, v1.w, acc[7]);
        }
        if (any && ch == 0 && c == 0 && a.err_flag) atomicOr(a.err_flag, kErrBlockId);
        if (p.slot < 0) {
          const float inv = 1.f / L;
#pragma unroll
          for (int d = 0; d < 8; ++d) acc[d] = any ? 0.f : acc[d] * inv;
          cross_store8(static_cast<__nv_bfloat16*>(a.out) + (p.base(a) + cross_column(a, 8 * nt + c)) * D + 8 * ch, acc);
        } else {
          cross_store8(a.part_o + static_cast<size_t>(p.slot) * COLS * D + (ch * COLS + 8 * nt + c) * 8, acc);
          if (ch == 0) a.part_ml[static_cast<size_t>(p.slot) * COLS + 8 * nt + c] = make_float2(M, any ? -1.f : L);
        }
      }
      __syncthreads();
    }
    if (ok && p.slot >= 0) {
      int first, pieces;
      cross_chain(s_total, p, &first, &pieces);
      __threadfence();
      __syncthreads();
      if (tid == 0) s_total.old[0][0] = atomicInc(a.count + first, pieces - 1);
      __syncthreads();
      if (s_total.old[0][0] == static_cast<unsigned>(pieces - 1)) {
        __threadfence();
        static_assert(kMergeFloats<COLS> <= kWarps * 8 * D, "the weights go where the exchange was");
        // (with more column groups the partials in flight would spill the tile loop's registers)
        if (NT <= 2 && pieces <= kMergeSharedPieces && p.live * (D / 4) * 16 > kThreads) {
          cross_merge_shared<__nv_bfloat16, D, COLS, 2, 8>(a, p, first, pieces, tid, kThreads, s_o);
          __syncthreads();  // (the weights are read to its end: the next piece's states go there)
        } else {
          // (one column of 64 dims is 16 units)
          cross_merge<__nv_bfloat16, D, COLS, 1, 1, 4, 8, D * 4 <= kThreads>(a, p, first, pieces, 0, tid, kThreads);
        }
      }
    }
  }
  // loads in flight land before the CTA exits (after an abort there may be some)
  for (int i = taken; i < issued; ++i) mbar_wait_bounded(full0 + 8 * (i % DEPTH), (i / DEPTH) & 1);
}

template <int D, int NT>
CrossKernel info() {
  CrossKernel k{};
  k.fn = reinterpret_cast<const void*>(&cross_few_kernel<D, NT>);
  k.threads = kThreads;
  k.ctas_per_sm = 1;
  k.smem = Shape<D>::SMEM;
  k.cols = 8 * NT;
  k.keys = kKeys;
  k.extra = kExtra;
  return k;
}

template <int D>
CrossKernel pick(int columns) {
  return columns <= 8 ? info<D, 1>() : columns <= 16 ? info<D, 2>() : columns <= 24 ? info<D, 3>() : info<D, 4>();
}

}  // namespace

CrossKernel cross_few_kernel_info(int head_dim, int columns) {
  return head_dim == 64 ? pick<64>(columns) : pick<128>(columns);
}

}  // namespace pa
