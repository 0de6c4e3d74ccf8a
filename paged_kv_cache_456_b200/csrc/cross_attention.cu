// cross_attention.cu -- pa_cross_attention's plan and merge kernels and its
// launch.  The query rows of each sequence attend to ALL tokens that the
// sequence's block table lists (an encoder's states, a document), whose
// number does not depend on the number of rows:
//   out[r][h] = sum_i exp(x_i - max x) V_i / sum_i exp(x_i - max x),
//   x_i = scale q[r][h] . K_i,   i = 0 .. n - 1.
// Launches: the plan (one CTA: lengths and block ids checked, the work laid
// out), the attention kernel, the merge of split items, each behind the last
// with programmatic dependent launch.
#include <algorithm>
#include <map>
#include <mutex>
#include <utility>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cross_attention.h"
#include "cross_kernels.h"

namespace pa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanSeqsOnChip = 4096;  // sequences whose starts the plan searches in shared memory
constexpr int kPlanAhead = 4;          // block ids per lane loaded beside a sequence's lengths
constexpr int kFoldThreads = 256;

__global__ void __launch_bounds__(kPlanThreads, 1) cross_plan_kernel(const CrossArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ long long s_start[kPlanSeqsOnChip + 1];
  __shared__ long long s_wsum[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = a.num_seqs;
  const bool on_chip = S <= kPlanSeqsOnChip;
  auto put = [&](int s, long long v) {
    if (on_chip) s_start[s] = v; else a.start[s] = v;
  };
  auto get = [&](int s) -> long long { return on_chip ? s_start[s] : __ldcg(a.start + s); };

  // One warp per sequence: its rows and length, and that every block it
  // attends to is a block of the cache (the first ids are loaded together
  // with the lengths; each load is in bounds of its array whatever the
  // values).  A sequence with a bad length or id keeps its rows and loses its
  // keys: they are written as zeros.
  for (int s = warp; s < S; s += kPlanThreads / 32) {
    const int32_t* row = a.block_tables + static_cast<size_t>(s) * a.max_blocks_per_seq;
    const int r0 = a.query_start[s], r1 = a.query_start[s + 1];
    int n = a.context_lens[s];
    int ids[kPlanAhead];
#pragma unroll
    for (int k = 0; k < kPlanAhead; ++k) {
      const int b = lane + 32 * k;
      ids[k] = b < a.max_blocks_per_seq ? __ldg(row + b) : 0;
    }
    int bit = 0;
    const bool placed = 0 <= r0 && r0 <= r1 && r1 <= a.num_rows;
    if (!placed) {
      bit = kErrQuery;
    } else if (n < 0 || n > a.len_cap) {
      bit = kErrContextLen;
    } else {
      const int nb = (n + kBlockSize - 1) / kBlockSize;  // (at most max_blocks_per_seq)
      bool bad = false;
#pragma unroll
      for (int k = 0; k < kPlanAhead; ++k)
        bad |= lane + 32 * k < nb && !(ids[k] >= 0 && ids[k] < a.num_blocks);
#pragma unroll 4
      for (int b = lane + 32 * kPlanAhead; b < nb; b += 32) {
        const int id = __ldg(row + b);
        bad |= !(id >= 0 && id < a.num_blocks);
      }
      if (r1 > r0 && __any_sync(0xffffffffu, bad)) bit = kErrBlockId;
    }
    if (bit) n = 0;
    if (lane == 0) {
      if (bit && a.err_flag && (bit == kErrQuery || r1 > r0)) atomicOr(a.err_flag, bit);
      const int Q = placed ? r1 - r0 : 0;
      const long long c = static_cast<long long>(Q) << a.group_log2;
      const int ng = static_cast<int>((c + a.cols - 1) / a.cols);
      a.meta[s] = make_int4(placed ? r0 : 0, Q, n, ng);
      put(s, static_cast<long long>(a.num_kv_heads) * ng * cross_tiles(n, a.keys));
    }
  }
  __syncthreads();

  // tiles before each sequence
  const int per = (S + kPlanThreads - 1) / kPlanThreads;
  const int s0 = min(S, tid * per), s1 = min(S, s0 + per);
  long long local = 0;
  for (int s = s0; s < s1; ++s) local += get(s);
  long long incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) s_wsum[warp] = incl;
  __syncthreads();
  long long run = incl - local, W = 0;
  for (int i = 0; i < kPlanThreads / 32; ++i) {
    if (i < warp) run += s_wsum[i];
    W += s_wsum[i];
  }
  for (int s = s0; s < s1; ++s) {
    const long long t = get(s);
    put(s, run);
    run += t;
  }
  __syncthreads();

  const long long workers = max(1LL, min(static_cast<long long>(a.max_workers), W / a.min_tiles));
  if (tid == 0) {
    a.head[0] = W;
    a.head[1] = workers;
  }
  for (int w = tid; w < workers; w += kPlanThreads) {
    const long long lo = w * W / workers, hi = (w + 1) * W / workers;
    int l = 0, u = S - 1;  // the last sequence that starts at lo or before
    while (l < u) {
      const int mid = (l + u + 1) >> 1;
      if (get(mid) <= lo) l = mid; else u = mid - 1;
    }
    const int nt = cross_tiles(__ldcg(&a.meta[l].z), a.keys);
    const long long off = lo - get(l);
    const int item = static_cast<int>(off / nt);
    a.rec[w] = make_int4(l, item, static_cast<int>(off - static_cast<long long>(item) * nt),
                         static_cast<int>(hi - lo));
  }
}

// The merge of an item that worker boundaries cut.  CTAs (w, y): the items in
// which boundary w (between workers w and w + 1) is the first, columns y * 8 +
// warp onwards; a lane takes D / 32 dims.
template <typename T, int D>
__global__ void __launch_bounds__(kFoldThreads) cross_merge_kernel(const CrossArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int DPL = D / 32, AHEAD = 4;
  const long long W = __ldcg(a.head), workers = __ldcg(a.head + 1);
  const int w = blockIdx.x;  // the worker of the item's first piece
  if (w + 1 >= workers) return;
  const int4 rec = __ldcg(a.rec + w + 1);
  if (rec.z == 0) return;    // an item begins at this boundary
  const long long begin = (w + 1) * W / workers - rec.z;
  if (begin < w * W / workers) return;  // not the item's first boundary
  const int4 m = __ldcg(a.meta + rec.x);
  const long long last = begin + cross_tiles(m.z, a.keys) - 1;
  const int pieces = static_cast<int>(((last + 1) * workers - 1) / W) - w + 1;
  const int kvh = rec.y / m.w, grp = rec.y - kvh * m.w;
  const int lane = threadIdx.x & 31;
  for (int c = blockIdx.y * (kFoldThreads / 32) + (threadIdx.x >> 5); c < a.cols;
       c += gridDim.y * (kFoldThreads / 32)) {
    const long long gc = static_cast<long long>(grp) * a.cols + c;
    const int row = static_cast<int>(gc >> a.group_log2);
    if (row >= m.y) break;
    const int h = static_cast<int>(gc) & ((1 << a.group_log2) - 1);
    float M = -INFINITY, L = 0.f, acc[DPL];
#pragma unroll
    for (int d = 0; d < DPL; ++d) acc[d] = 0.f;
    for (int p0 = 0; p0 < pieces; p0 += AHEAD) {
      float2 ml[AHEAD];
      float o[AHEAD][DPL];
      float mn = M;
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int p = min(p0 + k, pieces - 1);
        const size_t at = static_cast<size_t>(p == 0 ? 2 * w + 1 : 2 * (w + p)) * a.cols + c;
        ml[k] = __ldcg(a.part_ml + at);
        if constexpr (DPL == 4) {
          const float4 t = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * D) + lane);
          o[k][0] = t.x, o[k][1] = t.y, o[k][2] = t.z, o[k][3] = t.w;
        } else {
          const float2 t = __ldcg(reinterpret_cast<const float2*>(a.part_o + at * D) + lane);
          o[k][0] = t.x, o[k][1] = t.y;
        }
        if (p0 + k >= pieces) ml[k] = make_float2(-INFINITY, 0.f);  // (a repeat, weighed 0)
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) mn = fmaxf(mn, ml[k].x);
      const float sc = M == -INFINITY ? 0.f : exp2f(M - mn);
      L *= sc;
#pragma unroll
      for (int d = 0; d < DPL; ++d) acc[d] *= sc;
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        if (p0 + k >= pieces) break;
        // (a piece whose scores are all -inf carries zeros, or the NaN that
        // such scores make)
        const float wt = ml[k].x == -INFINITY ? 1.f : exp2f(ml[k].x - mn);
        L = fmaf(wt, ml[k].y, L);
#pragma unroll
        for (int d = 0; d < DPL; ++d) acc[d] = fmaf(wt, o[k][d], acc[d]);
      }
      M = mn;
    }
    const float inv = 1.f / L;
    T* const dst = static_cast<T*>(a.out) +
                   (static_cast<size_t>(m.x + row) * a.num_q_heads + (kvh << a.group_log2) + h) * D +
                   lane * DPL;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int d = 0; d < DPL; ++d) dst[d] = acc[d] * inv;
    } else {
#pragma unroll
      for (int d = 0; d < DPL; d += 2)
        *reinterpret_cast<__nv_bfloat162*>(dst + d) = __floats2bfloat162_rn(acc[d] * inv, acc[d + 1] * inv);
    }
  }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

std::mutex g_mu;
std::map<std::pair<int, const void*>, size_t> g_smem;  // (device, kernel) -> limit set

}  // namespace

CrossKernel cross_kernel(int num_seqs, int num_rows, int group, int head_dim, int elem_bytes) {
  if (elem_bytes == 2) return cross_tc_kernel_info(head_dim);
  return cross_simt_kernel_info(head_dim, elem_bytes);
}

CrossPlan cross_plan(int num_seqs, int num_rows, int num_q_heads, int num_kv_heads, int head_dim,
                     int elem_bytes, int num_sms) {
  const CrossKernel k = cross_kernel(num_seqs, num_rows, num_q_heads / num_kv_heads, head_dim,
                                     elem_bytes);
  CrossPlan p;
  p.cols = k.cols;
  p.keys = k.keys;
  p.max_workers = num_sms * k.ctas_per_sm * k.workers_per_cta;
  p.min_tiles = k.min_tiles;
  const size_t slots = 2 * static_cast<size_t>(p.max_workers);
  p.rec_off = 256;
  p.meta_off = up256(p.rec_off + static_cast<size_t>(p.max_workers) * sizeof(int4));
  p.start_off = up256(p.meta_off + static_cast<size_t>(num_seqs) * sizeof(int4));
  p.ml_off = up256(p.start_off + (static_cast<size_t>(num_seqs) + 1) * sizeof(long long));
  p.o_off = up256(p.ml_off + slots * k.cols * sizeof(float2));
  p.bytes = up256(p.o_off + slots * k.cols * head_dim * sizeof(float));
  return p;
}

cudaError_t launch_cross_attention(CrossArgs& a, int elem_bytes, int num_sms, cudaStream_t stream) {
  const CrossKernel k = cross_kernel(a.num_seqs, a.num_rows, 1 << a.group_log2, a.head_dim, elem_bytes);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    size_t& limit = g_smem[std::make_pair(dev, k.fn)];
    if (limit < k.smem) {
      if ((e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(k.smem))) != cudaSuccess)
        return e;
      limit = k.smem;
    }
  }
  void* params[] = {&a};
  if ((e = cudaLaunchKernel(reinterpret_cast<const void*>(&cross_plan_kernel), dim3(1),
                            dim3(kPlanThreads), params, 0, stream)) != cudaSuccess)
    return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms * k.ctas_per_sm);
  cfg.blockDim = dim3(k.threads);
  cfg.dynamicSmemBytes = k.smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelExC(&cfg, k.fn, params)) != cudaSuccess) return e;
  const void* merge =
      elem_bytes == 4 ? (a.head_dim == 64 ? reinterpret_cast<const void*>(&cross_merge_kernel<float, 64>)
                                          : reinterpret_cast<const void*>(&cross_merge_kernel<float, 128>))
                      : (a.head_dim == 64
                             ? reinterpret_cast<const void*>(&cross_merge_kernel<__nv_bfloat16, 64>)
                             : reinterpret_cast<const void*>(&cross_merge_kernel<__nv_bfloat16, 128>));
  cfg.gridDim = dim3(std::max(1, a.max_workers - 1), std::min(8, std::max(1, a.cols / 8)));
  cfg.blockDim = dim3(kFoldThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelExC(&cfg, merge, params);
}

}  // namespace pa
