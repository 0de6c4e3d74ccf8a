// cross_simt.cu -- cross attention in fp32 on the CUDA cores.
//
// A CTA (one worker) takes 64 query columns x 64 keys at a time:
//   S = Q K^T           thread: 8 columns x 4 keys, packed fp32 pairs along D
//   P = 2^(S - m)       online, fp32; running max m and sum l per column
//   O = O 2^(dm) + P V  thread: 8 columns x D/16 dims
// Column group cg = tid / 16 belongs to 16 lanes of one warp (kg = tid % 16:
// keys kg + 16 j, dims 4 kg + 64 j), so the row reductions are four shuffles
// and P passes between the two products through shared memory within a warp.
// K of the next tile is fetched (cp.async) while this tile's P V runs, V
// while the next S runs.  Bound by the fp32 units: 16 LDS.128 wavefronts
// feed 64 packed FMAs of a warp (32 cycles of the SM).
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cross_attention.h"
#include "ptx.cuh"

namespace pa {
namespace {

constexpr int kCols = 64, kKeys = 64, kThreads = 128;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float2 lo2(const float4& x) { return make_float2(x.x, x.y); }
__device__ __forceinline__ float2 hi2(const float4& x) { return make_float2(x.z, x.w); }

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
cross_simt_kernel(const __grid_constant__ CrossArgs a) {
  constexpr int CPR = D / 4;  // 16-byte chunks of a row
  constexpr int DJ = D / 64;
  extern __shared__ __align__(16) float smem[];
  float* const sQ = smem;                  // [kCols][D], 16-byte chunk c of row r at c ^ (r / 8 % 8)
  float* const sK = sQ + kCols * D;        // [kKeys][D], chunk c of row r at c ^ (r % 8)
  float* const sV = sK + kKeys * D;        // [kKeys][D]
  float* const sP = sV + kKeys * D;        // [4 warps][kKeys][16 columns]
  const int tid = threadIdx.x, lane = tid & 31;
  const int cg = tid >> 4, kg = tid & 15;
  float* const myP = sP + (tid >> 5) * (kKeys * 16) + ((lane >> 4) * 8);
  __shared__ CrossTotal s_total;

  CrossWalk walk(a, cross_share<kThreads>(a, kCols, kKeys, &s_total), kCols);
  CrossPiece p;
  while (walk.next(a, kCols, kKeys, &p)) {
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
    auto load = [&](float* dst, const void* cache, int t, bool swizzle) {
      for (int i = tid; i < kKeys * CPR; i += kThreads) {
        const int r = i / CPR, c = i % CPR;
        const int key = t * kKeys + r;
        const bool live = key < p.n;
        int id = live ? __ldg(table + key / kBlockSize) : 0;
        if (id < 0 || id >= a.num_blocks) id = 0;  // (the piece is poisoned)
        const float* row = static_cast<const float*>(cache) +
                       ((static_cast<size_t>(id) * a.num_kv_heads + p.kvh) * kBlockSize + key % kBlockSize) * D;
        cp_async16(smem_addr(dst + r * D + 4 * (c ^ (swizzle ? r & 7 : 0))), row + 4 * c, live);
      }
      cp_commit();
    };
    __syncthreads();  // (the last piece's Q, K and V have been read)
    for (int i = tid; i < kCols * CPR; i += kThreads) {
      const int c = i / CPR, k = i % CPR;
      const long long x = p.base(a) + cross_column(a, min(c, p.live - 1));
      cp_async16(smem_addr(sQ + c * D + 4 * (k ^ ((c >> 3) & 7))), static_cast<const float*>(a.q) + x * D + 4 * k,
                 c < p.live);
    }
    load(sK, a.k_cache, p.t0, true);
    load(sV, a.v_cache, p.t0, false);

    float m[8], l[8];
    float2 o[8][2 * DJ];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < 2 * DJ; ++j) o[i][j] = make_float2(0.f, 0.f);
    }
    for (int t = p.t0; t < p.t1; ++t) {
      cp_wait<1>();
      __syncthreads();
      float2 s2[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s2[i][j] = make_float2(0.f, 0.f);
#pragma unroll 2
      for (int c = 0; c < D / 4; ++c) {
        float4 k4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          k4[j] = *reinterpret_cast<const float4*>(sK + (kg + 16 * j) * D + 4 * (c ^ (kg & 7)));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 q4 = *reinterpret_cast<const float4*>(sQ + (cg * 8 + i) * D + 4 * (c ^ cg));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s2[i][j] = __ffma2_rn(lo2(q4), lo2(k4[j]), s2[i][j]);
            s2[i][j] = __ffma2_rn(hi2(q4), hi2(k4[j]), s2[i][j]);
          }
        }
      }
      __syncthreads();
      if (t + 1 < p.t1) load(sK, a.k_cache, t + 1, true); else cp_commit();

      // softmax of this thread's 8 columns x 4 keys
      float x[8][4], al[8];
      bool grow = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
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
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 2 * DJ; ++j) o[i][j] = __fmul2_rn(o[i][j], make_float2(al[i], al[i]));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float4* dst = reinterpret_cast<float4*>(myP + (kg + 16 * j) * 16);
        dst[0] = make_float4(x[0][j], x[1][j], x[2][j], x[3][j]);
        dst[1] = make_float4(x[4][j], x[5][j], x[6][j], x[7][j]);
      }
      __syncwarp();
      cp_wait<1>();
      __syncthreads();
#pragma unroll 4
      for (int k = 0; k < kKeys; ++k) {
        const float4 pa = *reinterpret_cast<const float4*>(myP + k * 16);
        const float4 pb = *reinterpret_cast<const float4*>(myP + k * 16 + 4);
        const float pr[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
#pragma unroll
        for (int j = 0; j < DJ; ++j) {
          const float4 v4 = *reinterpret_cast<const float4*>(sV + k * D + 4 * kg + 64 * j);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
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
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int off = 8; off; off >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
      const int c = cg * 8 + i;
      if (c >= p.live) continue;
      const long long x = p.base(a) + cross_column(a, c);
      const float inv = p.slot < 0 ? 1.f / l[i] : 1.f;
#pragma unroll
      for (int j = 0; j < DJ; ++j) {
        const float4 v = bad ? make_float4(0.f, 0.f, 0.f, 0.f)
                             : make_float4(o[i][2 * j].x * inv, o[i][2 * j].y * inv, o[i][2 * j + 1].x * inv,
                                           o[i][2 * j + 1].y * inv);
        const int d = 4 * kg + 64 * j;
        if (p.slot < 0)
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + x * D + d) = v;
        else
          *reinterpret_cast<float4*>(a.part_o + static_cast<size_t>(p.slot) * kCols * D + (d / 8 * kCols + c) * 8 +
                                     d % 8) = v;
      }
      if (p.slot >= 0 && kg == 0)
        a.part_ml[static_cast<size_t>(p.slot) * kCols + c] = make_float2(m[i], bad ? -1.f : l[i]);
    }
    if (p.slot >= 0) {
      int first, pieces;
      cross_chain(s_total, p, &first, &pieces);
      __threadfence();
      __syncthreads();
      if (tid == 0) s_total.old[0] = atomicInc(a.count + first, pieces - 1);
      __syncthreads();
      if (s_total.old[0] == static_cast<unsigned>(pieces - 1)) {
        __threadfence();
        cross_merge<float, D, kCols, 1, 1, 2>(a, p, first, pieces, 0, tid, kThreads);
      }
    }
  }
  cp_wait<0>();
}

template <int D>
CrossKernel info() {
  CrossKernel k{};
  k.fn = reinterpret_cast<const void*>(&cross_simt_kernel<D>);
  k.threads = kThreads;
  k.ctas_per_sm = 2;
  k.smem = (static_cast<size_t>(kCols) * D + 2 * kKeys * D + 4 * kKeys * 16) * sizeof(float);
  k.cols = kCols;
  k.keys = kKeys;
  return k;
}

}  // namespace

CrossKernel cross_simt_kernel_info(int head_dim) { return head_dim == 64 ? info<64>() : info<128>(); }

}  // namespace pa
