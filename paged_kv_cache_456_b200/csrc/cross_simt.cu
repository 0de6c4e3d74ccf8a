// cross_simt.cu -- cross attention in fp32 on the CUDA cores.
//
// A CTA (one worker) takes 8 CPT query columns x 64 keys at a time:
//   S = Q K^T           thread: CPT columns x 4 keys, packed fp32 pairs along D
//   P = 2^(S - m)       online, fp32; running max m and sum l per column
//   O = O 2^(dm) + P V  thread: CPT columns x D/16 dims
// Column group cg = tid / 16 belongs to 16 lanes of one warp (kg = tid % 16:
// keys kg + 16 j, dims 4 kg + 64 j), so the row reductions are four shuffles
// and P passes between the two products through shared memory within a warp.
// K of the next tile is fetched (cp.async) while this tile's P V runs, V
// while the next S runs.  CPT = 8 is bound by the fp32 units: 16 LDS.128
// wavefronts feed 64 packed FMAs of a warp (32 cycles of the SM); 4 x 2048 rows
// against 2048 keys, 16 heads of 64: 1806 us, 38 TFLOP/s; heads of 128: 43.
// Fewer columns a (sequence, KV head) take a smaller CPT, more CTAs an SM, and
// come nearer to the loads of K and V: 64 single rows against 1500 states, 16
// heads of 64 (786 MB): 248 us with CPT 1, 743 with 8.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cross_attention.h"
#include "ptx.cuh"

namespace pa {
namespace {

constexpr int kKeys = 64, kThreads = 128;
constexpr int kExtra = 0;  // (1: 6 ragged sequences 18.5 -> 25.6 us, their items being of few tiles)

// CTAs an SM, by shared memory and registers
template <int D, int CPT>
constexpr int kCtas = D == 64 ? (CPT == 8 ? 2 : CPT == 4 ? 3 : 4) : (CPT == 1 ? 3 : 2);

template <int N>
__device__ __forceinline__ void load_p(const float* src, float (&p)[N]) {
  if constexpr (N == 1) {
    p[0] = *src;
  } else if constexpr (N == 2) {
    const float2 v = *reinterpret_cast<const float2*>(src);
    p[0] = v.x, p[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(src + i);
      p[i] = v.x, p[i + 1] = v.y, p[i + 2] = v.z, p[i + 3] = v.w;
    }
  }
}
template <int N>
__device__ __forceinline__ void store_p(float* dst, const float (&p)[N]) {
  if constexpr (N == 1) {
    *dst = p[0];
  } else if constexpr (N == 2) {
    *reinterpret_cast<float2*>(dst) = make_float2(p[0], p[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<float4*>(dst + i) = make_float4(p[i], p[i + 1], p[i + 2], p[i + 3]);
  }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float2 lo2(const float4& x) { return make_float2(x.x, x.y); }
__device__ __forceinline__ float2 hi2(const float4& x) { return make_float2(x.z, x.w); }

template <int D, int CPT>
__global__ void __launch_bounds__(kThreads, kCtas<D, CPT>)
cross_simt_kernel(const __grid_constant__ CrossArgs a) {
  constexpr int CPR = D / 4;  // 16-byte chunks of a row
  constexpr int DJ = D / 64, kCols = 8 * CPT;
  extern __shared__ __align__(16) float smem[];
  float* const sQ = smem;                  // [kCols][D], 16-byte chunk c of row r at c ^ (r / CPT)
  float* const sK = sQ + kCols * D;        // [kKeys][D], chunk c of row r at c ^ (r % 8)
  float* const sV = sK + kKeys * D;        // [kKeys][D]
  float* const sP = sV + kKeys * D;        // [4 warps][kKeys][2 CPT columns]
  const int tid = threadIdx.x, lane = tid & 31;
  const int cg = tid >> 4, kg = tid & 15;
  float* const myP = sP + (tid >> 5) * (kKeys * 2 * CPT) + (lane >> 4) * CPT;
  __shared__ CrossTotal s_total;

  CrossWalk walk(a, cross_share<kThreads>(a, kCols, kKeys, kExtra, &s_total), kCols);
  CrossPiece p;
  while (walk.next(a, kCols, kKeys, kExtra, &p)) {
    if (p.n == 0) {
      for (int c = tid / 16; c < kCols; c += kThreads / 16) {
        if (c >= p.live) break;
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + (p.base(a) + cross_column(a, c)) * D);
        for (int i = tid & 15; i < CPR; i += 16) dst[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      continue;
    }
    const bool bad_block = cross_bad_block(a, p, kKeys, tid, kThreads);
    const int32_t* const table = a.block_tables + static_cast<size_t>(p.s) * a.max_blocks_per_seq;
    // this thread's chunk of RPP rows of each block
    constexpr int RPP = kThreads / CPR;
    const int lc = tid % CPR, lr = tid / CPR;
    const long long head = static_cast<long long>(p.kvh) * kBlockSize * D + lr * D + 4 * lc;
    const long long block = static_cast<long long>(a.num_kv_heads) * kBlockSize * D;
    auto load = [&](float* dst, const void* cache, int t, bool swizzle) {
      const float* const base = static_cast<const float*>(cache) + head;
#pragma unroll
      for (int b = 0; b < kKeys / kBlockSize; ++b) {
        const int key = t * kKeys + b * kBlockSize;
        int id = key < p.n ? __ldg(table + key / kBlockSize) : 0;
        if (id < 0 || id >= a.num_blocks) id = 0;  // (the piece is poisoned)
        const float* const src = base + id * block;
#pragma unroll
        for (int r = 0; r < kBlockSize; r += RPP) {
          const int row = b * kBlockSize + r + lr;
          cp_async16(smem_addr(dst + row * D + 4 * (lc ^ (swizzle ? row & 7 : 0))), src + r * D, key + r + lr < p.n);
        }
      }
      cp_commit();
    };
    __syncthreads();  // (the last piece's Q, K and V have been read)
    for (int i = tid; i < kCols * CPR; i += kThreads) {
      const int c = i / CPR, k = i % CPR;
      const long long x = p.base(a) + cross_column(a, min(c, p.live - 1));
      cp_async16(smem_addr(sQ + c * D + 4 * (k ^ (c / CPT))), static_cast<const float*>(a.q) + x * D + 4 * k,
                 c < p.live);
    }
    load(sK, a.k_cache, p.t0, true);
    load(sV, a.v_cache, p.t0, false);

    float m[CPT], l[CPT];
    float2 o[CPT][2 * DJ];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < 2 * DJ; ++j) o[i][j] = make_float2(0.f, 0.f);
    }
    for (int t = p.t0; t < p.t1; ++t) {
      cp_wait<1>();
      __syncthreads();
      float2 s2[CPT][4];
#pragma unroll
      for (int i = 0; i < CPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s2[i][j] = make_float2(0.f, 0.f);
#pragma unroll 2
      for (int c = 0; c < D / 4; ++c) {
        float4 k4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          k4[j] = *reinterpret_cast<const float4*>(sK + (kg + 16 * j) * D + 4 * (c ^ (kg & 7)));
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          const float4 q4 = *reinterpret_cast<const float4*>(sQ + (cg * CPT + i) * D + 4 * (c ^ cg));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s2[i][j] = __ffma2_rn(lo2(q4), lo2(k4[j]), s2[i][j]);
            s2[i][j] = __ffma2_rn(hi2(q4), hi2(k4[j]), s2[i][j]);
          }
        }
      }
      __syncthreads();
      if (t + 1 < p.t1) load(sK, a.k_cache, t + 1, true); else cp_commit();

      // softmax of this thread's columns x 4 keys
      float x[CPT][4], al[CPT];
      bool grow = false;
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool seen = t * kKeys + kg + 16 * j < p.n;
          x[i][j] = seen ? (s2[i][j].x + s2[i][j].y) * a.scale_log2 : -INFINITY;
          mx = fmaxf(mx, x[i][j]);
        }
#pragma unroll
        for (int off = 8; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        al[i] = 1.f;
        if (mx > m[i]) {
          al[i] = exp2f(m[i] - mx);
          m[i] = mx;
          grow = true;
        }
        const float base = m[i] == -INFINITY ? 0.f : m[i];  // (every score -inf: weights 0)
        l[i] *= al[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[i][j] = exp2f(x[i][j] - base);
          l[i] += x[i][j];
        }
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int i = 0; i < CPT; ++i)
#pragma unroll
          for (int j = 0; j < 2 * DJ; ++j) o[i][j] = __fmul2_rn(o[i][j], make_float2(al[i], al[i]));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float pr[CPT];
#pragma unroll
        for (int i = 0; i < CPT; ++i) pr[i] = x[i][j];
        store_p(myP + (kg + 16 * j) * 2 * CPT, pr);
      }
      __syncwarp();
      cp_wait<1>();
      __syncthreads();
#pragma unroll 4
      for (int k = 0; k < kKeys; ++k) {
        float pr[CPT];
        load_p(myP + k * 2 * CPT, pr);
#pragma unroll
        for (int j = 0; j < DJ; ++j) {
          const float4 v4 = *reinterpret_cast<const float4*>(sV + k * D + 4 * kg + 64 * j);
#pragma unroll
          for (int i = 0; i < CPT; ++i) {
            const float2 pp = make_float2(pr[i], pr[i]);
            o[i][2 * j] = __ffma2_rn(pp, lo2(v4), o[i][2 * j]);
            o[i][2 * j + 1] = __ffma2_rn(pp, hi2(v4), o[i][2 * j + 1]);
          }
        }
      }
      __syncthreads();
      if (t + 1 < p.t1) load(sV, a.v_cache, t + 1, false); else cp_commit();
    }

    const bool bad = __syncthreads_or(bad_block);
    if (bad && tid == 0 && a.err_flag) atomicOr(a.err_flag, kErrBlockId);
#pragma unroll
    for (int off = 8; off; off >>= 1)
#pragma unroll
      for (int i = 0; i < CPT; ++i) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
    if (p.slot < 0) {
      float* const dst = static_cast<float*>(a.out) + p.base(a) * D + 4 * kg;
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        const int c = cg * CPT + i;
        const float inv = 1.f / l[i];
        if (c >= p.live) continue;
#pragma unroll
        for (int j = 0; j < DJ; ++j)
          *reinterpret_cast<float4*>(dst + cross_column(a, c) * D + 64 * j) =
              bad ? make_float4(0.f, 0.f, 0.f, 0.f)
                  : make_float4(o[i][2 * j].x * inv, o[i][2 * j].y * inv, o[i][2 * j + 1].x * inv,
                                o[i][2 * j + 1].y * inv);
      }
    } else {  // (columns past the last too: no one reads them)
      float* const dst = a.part_o + static_cast<size_t>(p.slot) * kCols * D + (kg / 2 * kCols + cg * CPT) * 8 + kg % 2 * 4;
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
#pragma unroll
        for (int j = 0; j < DJ; ++j)
          *reinterpret_cast<float4*>(dst + 8 * i + 8 * j * kCols * 8) =
              make_float4(o[i][2 * j].x, o[i][2 * j].y, o[i][2 * j + 1].x, o[i][2 * j + 1].y);
        if (kg == 0)
          a.part_ml[static_cast<size_t>(p.slot) * kCols + cg * CPT + i] = make_float2(m[i], bad ? -1.f : l[i]);
      }
    }
    if (p.slot >= 0) {
      int first, pieces;
      cross_chain(s_total, p, &first, &pieces);
      __threadfence();
      __syncthreads();
      if (tid == 0) s_total.old[0][0] = atomicInc(a.count + first, pieces - 1);
      __syncthreads();
      if (s_total.old[0][0] == static_cast<unsigned>(pieces - 1)) {
        __threadfence();
        static_assert(kMergeFloats<kCols> <= 4 * kKeys * 2 * CPT, "the weights go where P was");
        if (pieces <= kMergeSharedPieces)
          cross_merge_shared<float, D, kCols, 4, 4>(a, p, first, pieces, tid, kThreads, sP);
        else
          cross_merge<float, D, kCols, 1, 1, 2>(a, p, first, pieces, 0, tid, kThreads);
      }
    }
  }
  cp_wait<0>();
}

template <int D, int CPT>
CrossKernel info() {
  CrossKernel k{};
  k.fn = reinterpret_cast<const void*>(&cross_simt_kernel<D, CPT>);
  k.threads = kThreads;
  k.ctas_per_sm = kCtas<D, CPT>;
  k.smem = (static_cast<size_t>(8 * CPT) * D + 2 * kKeys * D + 4 * kKeys * 2 * CPT) * sizeof(float);
  k.cols = 8 * CPT;
  k.keys = kKeys;
  k.extra = kExtra;
  return k;
}

template <int D>
CrossKernel pick(long long columns) {
  return columns <= 8 ? info<D, 1>() : columns <= 16 ? info<D, 2>() : columns <= 32 ? info<D, 4>() : info<D, 8>();
}

}  // namespace

CrossKernel cross_simt_kernel_info(int head_dim, long long columns) {
  return head_dim == 64 ? pick<64>(columns) : pick<128>(columns);
}

}  // namespace pa
