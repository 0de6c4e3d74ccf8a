// cross_attention.h -- what the kernels of pa_cross_attention share: the
// arguments, the cut of the work over the CTAs, and the merge of what it cuts.
//
// An item is (sequence, KV head, group of query columns); a column is one
// (query row, query head) pair of the KV head, column c of a sequence being
// row c / G, head c % G.  An item's keys are cut into tiles; an item without
// keys counts one tile (its rows are written as zeros).  All tiles are laid
// end to end in (sequence, KV head, group, tile) order, `extra` units ahead of
// each item's for what an item costs besides its tiles, and cut into equal
// contiguous shares, one per worker (a CTA), so every CTA gets as much work
// however skewed the lengths are.  (A cut inside the units ahead is one at the
// item's first tile.)  The run of one item's tiles inside a share is a piece: a
// piece that is the whole item stores the output, any other stores a partial
// state (m, l, o), and the CTA that stores the last of an item's partials
// merges them, in the order of the keys:
//   M = max_j m_j,  out = sum_j 2^(m_j - M) o_j / sum_j 2^(m_j - M) l_j.
// No CTA waits for another.  A worker has at most two partial pieces, hence
// two slots: slot 2 w for the piece its share begins inside of, 2 w + 1 for
// the one it begins and does not finish.
//
// Every CTA lays the work out for itself (cross_share): that costs it one
// round of loads and a scan, less than a launch ahead of it did (a one-CTA plan
// kernel: 6 us, and 13 us to check 4096 block ids).  Block ids are checked by
// the pieces that attend to them: each item of a sequence covers all its keys,
// so a bad id is met by every row's item, and a piece that meets one poisons
// its item (l = -1).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "pa_internal.h"

namespace pa {

struct CrossArgs {
  const void* q;
  void* out;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;
  int num_seqs, num_rows, num_q_heads, num_kv_heads;
  int group_log2;              // log2 of the query heads per KV head
  int max_blocks_per_seq, num_blocks, len_cap;
  float scale_log2;            // scale * log2(e)
  long long max_units;         // of work that num_rows rows in order can make (set by the launcher)
  int32_t* err_flag;
  // workspace
  unsigned* count;             // [workers][column tiles]: partials stored of the item that begins
                               // in the worker and goes on; zero between calls
  float2* part_ml;             // [slots][columns]: running max (log2 units), sum of weights (< 0: poisoned)
  float* part_o;               // [slots][column tiles][D / 8][columns of a tile][8] (cross_tc.cu: 4 dims for 8)
  CUtensorMap tm_k;            // bf16: caches as [num_blocks * Hkv * 16][D], boxes 16 x 64, SW128
  CUtensorMap tm_v;
  CUtensorMap tm_q;            // (where the kernel asks) q as (D, query heads, rows), boxes 64 x G x 128 / G
};

// A kernel and how it cuts the work.
struct CrossKernel {
  const void* fn;              // __global__ void fn(CrossArgs)
  int threads, ctas_per_sm;
  size_t smem;                 // dynamic shared memory of a CTA
  int cols, keys, extra;       // columns of an item, keys of a tile, units ahead of an item
  bool tma_q;                  // reads q through tm_q
};
// The kernel for a call (host-known sizes only).
CrossKernel cross_kernel(int num_seqs, int num_rows, int group, int head_dim, int elem_bytes);
// fp32, about `columns` query columns a (sequence, KV head): CUDA cores (cross_simt.cu)
CrossKernel cross_simt_kernel_info(int head_dim, long long columns);
CrossKernel cross_tc_kernel_info(int head_dim);  // bf16, many columns: tcgen05 (cross_tc.cu)
// bf16, about `columns` (at most 32) query columns a (sequence, KV head): mma.sync (cross_few.cu)
CrossKernel cross_few_kernel_info(int head_dim, int columns);

// Workspace: the counters first, in a place that no call's sizes change.
constexpr size_t kCrossCountBytes = 16384;
struct CrossLayout {
  size_t ml_off, o_off, bytes;
};
CrossLayout cross_layout(const CrossKernel& k, int head_dim, int num_sms);
// what any call of at most `num_rows` rows needs, however many sequences share them
size_t cross_workspace_bytes(int num_rows, int group, int head_dim, int elem_bytes, int num_sms);
cudaError_t launch_cross_attention(CrossArgs& a, const CrossKernel& k, int num_sms, cudaStream_t stream);

#ifdef __CUDACC__
__device__ __forceinline__ void prefetch_tensormap(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

__device__ __forceinline__ int cross_tiles(int n, int keys) { return n > 0 ? (n + keys - 1) / keys : 1; }

// Sequence s's {first row, rows, keys, groups of `cols` columns}, checked: one
// whose rows are out of order has none, one whose length is bad has no keys.
__device__ __forceinline__ int4 cross_seq(const CrossArgs& a, int s, int cols, int* bit) {
  const int r0 = __ldg(a.query_start + s), r1 = __ldg(a.query_start + s + 1);
  int n = __ldg(a.context_lens + s);
  *bit = 0;
  if (!(0 <= r0 && r0 <= r1 && r1 <= a.num_rows)) {
    *bit = kErrQuery;
    return make_int4(0, 0, 0, 0);
  }
  if (r1 > r0 && (n < 0 || n > a.len_cap)) {
    *bit = kErrContextLen;
    n = 0;
  }
  // (rows * query heads fit in 31 bits)
  return make_int4(r0, r1 - r0, n, (((r1 - r0) << a.group_log2) + cols - 1) / cols);
}

// A worker's share: `left` units from unit `unit` of item `item` of sequence s
// on; the first is unit `at` of all.
struct CrossShare {
  long long at;
  int left, s, item, unit;
};
// (in shared memory: what the end of a piece needs)
struct CrossTotal {
  long long W;       // units of the call
  int workers;       // workers that have some
  // partials stored before this one, per column tile and parity of the piece's
  // slot: a share has at most one cut piece of each, so that no word is written
  // for a later piece while a slow warp still has to read it
  unsigned old[2][2];
  long long scratch[16];  // (a long long per warp, two more; at most 14 warps)
};

// Lays the work out; every thread of the CTA takes part, and is past a
// __syncthreads at the end.  Up to 128 sequences every warp does it for itself
// (a lane has up to four, whose lengths it loads together); more are spread
// over the CTA.
template <int THREADS>
__device__ __forceinline__ CrossShare cross_share(const CrossArgs& a, int cols, int keys, int extra, CrossTotal* total) {
  long long* const scratch = total->scratch;
  constexpr int WARPS = THREADS / 32, MINE = 4;
  const int tid = threadIdx.x, lane = tid & 31, S = a.num_seqs;
  const bool by_warp = S <= 32 * MINE;
  const int parts = by_warp ? 32 : THREADS, part = by_warp ? lane : tid;
  const int per = (S + parts - 1) / parts;
  const int s0 = min(S, part * per), s1 = min(S, s0 + per);
  auto units_of = [&](const int4& m) -> long long {
    return static_cast<long long>(a.num_kv_heads) * m.w * (extra + cross_tiles(m.z, keys));
  };
  long long local = 0;
  int bits = 0;
  int4 mine[MINE];  // (by_warp)
  if (by_warp) {
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
      int bit = 0;
      mine[k] = s0 + k < s1 ? cross_seq(a, s0 + k, cols, &bit) : make_int4(0, 0, 0, 0);
      local += units_of(mine[k]);  // (at most 4 x 2^50)
      bits |= bit;
    }
  } else {
    for (int s = s0; s < s1; ++s) {
      int bit;
      local = min(local + units_of(cross_seq(a, s, cols, &bit)), 1LL << 52);
      bits |= bit;
    }
  }
  long long incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  long long run = incl - local, W;
  if (by_warp) {
    W = __shfl_sync(0xffffffffu, incl, 31);
  } else {
    if (lane == 31) scratch[tid >> 5] = incl;
    __syncthreads();
    W = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
      if (i < (tid >> 5)) run += scratch[i];
      W += scratch[i];
    }
  }
  // Pairs of query_start that go back and forth can each be in order and cover the
  // same rows many times over: such a call is refused, not worked through.
  if (W > a.max_units) {
    W = 0;
    bits |= kErrQuery;
  }
  if (bits && blockIdx.x == 0 && a.err_flag) atomicOr(a.err_flag, bits);
  CrossShare x;
  const int w = blockIdx.x;
  const int workers = static_cast<int>(max(1LL, min(static_cast<long long>(gridDim.x), W)));
  // (64-bit division costs hundreds of cycles: only where it is needed)
  if (W < (1 << 20)) {
    const unsigned u = static_cast<unsigned>(W);
    x.at = w * u / workers;  // (at most 2^11 workers)
    x.left = w < workers ? static_cast<int>((w + 1) * u / workers) - static_cast<int>(x.at) : 0;
  } else {
    x.at = w * W / workers;
    x.left = w < workers ? static_cast<int>((w + 1) * W / workers - x.at) : 0;
  }
  if (tid == 0) {
    total->W = W;
    total->workers = workers;
  }
  // one part's sequences hold the first unit
  const bool owner = run <= x.at && x.at < run + local;
  long long off = x.at - run;
  int fs = 0, fitem = 0, funit = 0;
  auto place = [&](int s, const int4& m) -> bool {
    const long long t = units_of(m);
    if (off >= t) {
      off -= t;
      return false;
    }
    const int nt = extra + cross_tiles(m.z, keys);
    fs = s;
    fitem = off < (1LL << 31) ? static_cast<int>(off) / nt : static_cast<int>(off / nt);
    funit = static_cast<int>(off - static_cast<long long>(fitem) * nt);
    return true;
  };
  if (by_warp) {
    bool done = !owner;
#pragma unroll
    for (int k = 0; k < MINE; ++k)
      if (!done) done = place(s0 + k, mine[k]);
    const unsigned who = __ballot_sync(0xffffffffu, owner);
    const int src = who ? __ffs(who) - 1 : 0;
    x.s = __shfl_sync(0xffffffffu, fs, src);
    x.item = __shfl_sync(0xffffffffu, fitem, src);
    x.unit = __shfl_sync(0xffffffffu, funit, src);
    __syncthreads();
  } else {
    int* const res = reinterpret_cast<int*>(scratch + WARPS);
    if (owner) {
      for (int s = s0; s < s1; ++s) {
        int bit;
        if (place(s, cross_seq(a, s, cols, &bit))) break;
      }
      res[0] = fs;
      res[1] = fitem;
      res[2] = funit;
    }
    __syncthreads();
    x.s = res[0];
    x.item = res[1];
    x.unit = res[2];
  }
  return x;
}

// A run of one item's tiles.
struct CrossPiece {
  int s, kvh, grp;   // sequence, KV head, group of columns
  int t0, t1, nt;    // tiles [t0, t1) of the item's nt
  int n, live;       // keys, live columns of the group
  int row;           // query row of column 0
  int slot;          // partial slot, or -1: the whole item
  long long begin;   // the item's first tile, in units
  // column 0 of the group in q and out, in rows of D elements
  __device__ __forceinline__ long long base(const CrossArgs& a) const {
    return static_cast<long long>(row) * a.num_q_heads + (kvh << a.group_log2);
  }
};

// The pieces of a share, in order.
struct CrossWalk {
  CrossShare x;
  int4 m;
  CrossWalk() = default;
  __device__ __forceinline__ CrossWalk(const CrossArgs& a, const CrossShare& share, int cols) : x(share) {
    int bit;
    m = x.left > 0 ? cross_seq(a, x.s, cols, &bit) : make_int4(0, 0, 0, 0);
  }
  __device__ __forceinline__ bool next(const CrossArgs& a, int cols, int keys, int extra, CrossPiece* p) {
    while (x.left > 0) {
      if (x.item >= a.num_kv_heads * m.w) {
        if (++x.s >= a.num_seqs) return false;
        int bit;
        m = cross_seq(a, x.s, cols, &bit);
        x.item = x.unit = 0;
        continue;
      }
      p->nt = cross_tiles(m.z, keys);
      const int u0 = x.unit, u1 = min(extra + p->nt, u0 + x.left), item = x.item;
      p->begin = x.at - u0 + extra;
      x.at += u1 - u0;
      x.left -= u1 - u0;
      ++x.item;
      x.unit = 0;
      p->t0 = max(0, u0 - extra);
      p->t1 = u1 - extra;
      if (p->t1 <= p->t0) continue;  // (nothing but units ahead)
      p->s = x.s;
      p->kvh = item / m.w;
      p->grp = item - p->kvh * m.w;
      p->n = m.z;
      const int c0 = p->grp * cols;
      p->live = min(cols, (m.y << a.group_log2) - c0);
      p->row = m.x + (c0 >> a.group_log2);
      const int w = blockIdx.x;
      p->slot = p->t0 > 0 ? 2 * w : p->t1 < p->nt ? 2 * w + 1 : -1;
      return true;
    }
    return false;
  }
};
// the workers that hold the pieces of p's item: the first, and how many
__device__ __forceinline__ void cross_chain(const CrossTotal& t, const CrossPiece& p, int* first, int* pieces) {
  if (t.W < (1 << 20)) {
    const unsigned W = static_cast<unsigned>(t.W), b = static_cast<unsigned>(p.begin);
    *first = static_cast<int>(((b + 1) * t.workers - 1) / W);
    *pieces = static_cast<int>(((b + p.nt) * t.workers - 1) / W) - *first + 1;
  } else {
    *first = static_cast<int>(((p.begin + 1) * t.workers - 1) / t.W);
    *pieces = static_cast<int>(((p.begin + p.nt) * t.workers - 1) / t.W) - *first + 1;
  }
}

// column c of a piece's group in q and out, in rows of D elements past the
// piece's base (the group begins at a query row's first head)
__device__ __forceinline__ int cross_column(const CrossArgs& a, int c) {
  return (c >> a.group_log2) * (a.num_q_heads - (1 << a.group_log2)) + c;
}

// Does a block that the piece attends to lie outside the cache?  Thread i of
// `threads` looks at every threads-th id.
__device__ __forceinline__ bool cross_bad_block(const CrossArgs& a, const CrossPiece& p, int keys, int i, int threads) {
  const int32_t* const row = a.block_tables + static_cast<size_t>(p.s) * a.max_blocks_per_seq;
  const int b1 = (min(p.n, p.t1 * keys) + kBlockSize - 1) / kBlockSize;
  bool bad = false;
  for (int b = p.t0 * (keys / kBlockSize) + i; b < b1; b += threads) {
    const int id = __ldg(row + b);
    bad |= !(id >= 0 && id < a.num_blocks);
  }
  return bad;
}

__device__ __forceinline__ void cross_store8(float* dst, const float (&x)[8]) {
  reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void cross_store8(__nv_bfloat16* dst, const float (&x)[8]) {
  __nv_bfloat162 b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(b);
}

__device__ __forceinline__ void cross_store4(float* dst, const float (&x)[4]) {
  *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void cross_store4(__nv_bfloat16* dst, const float (&x)[4]) {
  __nv_bfloat162 b[2] = {__floats2bfloat162_rn(x[0], x[1]), __floats2bfloat162_rn(x[2], x[3])};
  *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(b);
}

// column tile t of the partial of an item's i-th piece (`first`: the worker of
// its first)
template <int TILES>
__device__ __forceinline__ size_t cross_tile(int first, int i, int t) {
  return static_cast<size_t>(i == 0 ? 2 * first + 1 : 2 * (first + i)) * TILES + t;
}
// Dims 4 ch to 4 ch + 3 of column c in a partial of COLS columns: CHUNK dims of a
// column lie together, as many as a lane of the kernel stores at a time (so that
// a warp's stores fill whole 32-byte sectors).
template <int COLS, int CHUNK>
__device__ __forceinline__ int cross_chunk(int ch, int c) {
  return CHUNK == 4 ? (ch * COLS + c) * 4 : (ch / 2 * COLS + c) * 8 + (ch & 1) * 4;
}
// a piece's weight under the item's maximum (a piece that saw nothing finite
// carries zeros, or the NaN that its scores make)
__device__ __forceinline__ float cross_weight(float m, float M) { return m == -INFINITY ? 1.f : exp2f(m - M); }

// The merge of an item's column tile t (of TILES, COLS columns each) by
// `team` threads, once all its partials are stored and visible.  A thread
// takes 4 dims of a column at a time, UNITS of them and AHEAD pieces in flight;
// with LANES, where 16 times as many threads as units are there, 16 lanes share one.
template <typename T, int D, int COLS, int TILES, int UNITS, int AHEAD, int CHUNK = 8, bool LANES = false>
__device__ __forceinline__ void cross_merge(const CrossArgs& a, const CrossPiece& p, int first, int pieces, int t,
                                            int i0, int team) {
  const int live = min(COLS, p.live - t * COLS);
  const int units = live * (D / 4);
  if (LANES && pieces <= 16 && units * 16 <= team) {
    // 16 lanes of a unit, a piece each, summed by a fixed tree
    const int u = i0 / 16, j = i0 % 16;
    const int x = min(u, units - 1), ch = x / (2 * live) * 2 + (x & 1), c = x % (2 * live) >> 1;
    float2 ml = make_float2(-INFINITY, 0.f);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (j < pieces) {
      const size_t pt = cross_tile<TILES>(first, j, t);
      ml = __ldcg(a.part_ml + pt * COLS + c);
      o = __ldcg(reinterpret_cast<const float4*>(a.part_o + pt * COLS * D + cross_chunk<COLS, CHUNK>(ch, c)));
    }
    float M = ml.x;
#pragma unroll
    for (int k = 8; k; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
    const float w = cross_weight(ml.x, M);
    float v[5] = {w * o.x, w * o.y, w * o.z, w * o.w, w * ml.y};
    int bad = ml.y < 0.f;
#pragma unroll
    for (int k = 8; k; k >>= 1) {
#pragma unroll
      for (int d = 0; d < 5; ++d) v[d] += __shfl_xor_sync(0xffffffffu, v[d], k);
      bad |= __shfl_xor_sync(0xffffffffu, bad, k);
    }
    if (j == 0 && u < units) {
      const float inv = 1.f / v[4];
      float r[4];
#pragma unroll
      for (int d = 0; d < 4; ++d) r[d] = bad ? 0.f : v[d] * inv;
      cross_store4(static_cast<T*>(a.out) + (p.base(a) + cross_column(a, t * COLS + c)) * D + ch * 4, r);
    }
    return;
  }
  for (int u0 = i0; u0 < units; u0 += UNITS * team) {
    int c[UNITS], ch[UNITS];
    float M[UNITS], L[UNITS], acc[UNITS][4];
    bool bad[UNITS];
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const int x = min(u0 + u * team, units - 1);  // (a repeat is stored twice, alike)
      ch[u] = x / (2 * live) * 2 + (x & 1);         // (the two chunks of a stored 8 side by side)
      c[u] = x % (2 * live) >> 1;
      M[u] = -INFINITY;
      L[u] = 0.f;
      bad[u] = false;
#pragma unroll
      for (int d = 0; d < 4; ++d) acc[u][d] = 0.f;
    }
    for (int j0 = 0; j0 < pieces; j0 += AHEAD) {
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const size_t pt = cross_tile<TILES>(first, min(j0 + j, pieces - 1), t);
#pragma unroll
        for (int u = 0; u < UNITS; ++u) M[u] = fmaxf(M[u], __ldcg(a.part_ml + pt * COLS + c[u]).x);
      }
    }
    for (int j0 = 0; j0 < pieces; j0 += AHEAD) {
      float2 ml[AHEAD][UNITS];
      float4 o[AHEAD][UNITS];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        if (j0 + j >= pieces) break;
        const size_t pt = cross_tile<TILES>(first, j0 + j, t);
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          ml[j][u] = __ldcg(a.part_ml + pt * COLS + c[u]);
          o[j][u] = __ldcg(reinterpret_cast<const float4*>(
              a.part_o + pt * COLS * D + cross_chunk<COLS, CHUNK>(ch[u], c[u])));
        }
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        if (j0 + j >= pieces) break;
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          bad[u] |= ml[j][u].y < 0.f;
          const float w = cross_weight(ml[j][u].x, M[u]);
          L[u] = fmaf(w, ml[j][u].y, L[u]);
          acc[u][0] = fmaf(w, o[j][u].x, acc[u][0]);
          acc[u][1] = fmaf(w, o[j][u].y, acc[u][1]);
          acc[u][2] = fmaf(w, o[j][u].z, acc[u][2]);
          acc[u][3] = fmaf(w, o[j][u].w, acc[u][3]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const float inv = 1.f / L[u];
#pragma unroll
      for (int d = 0; d < 4; ++d) acc[u][d] = bad[u] ? 0.f : acc[u][d] * inv;
      cross_store4(static_cast<T*>(a.out) + (p.base(a) + cross_column(a, t * COLS + c[u])) * D + ch[u] * 4, acc[u]);
    }
  }
}

// The same by a whole CTA of `team` threads with room for the pieces' weights
// in shared memory (kMergeFloats<COLS>): a column's maximum,
// weights and sum are worked out once, and the pass over the partials holds
// nothing but them in flight.
constexpr int kMergeSharedPieces = 31;
template <int COLS>
constexpr int kMergeFloats = (2 * kMergeSharedPieces + 1) * COLS;
template <typename T, int D, int COLS, int UNITS, int AHEAD>
__device__ __forceinline__ void cross_merge_shared(const CrossArgs& a, const CrossPiece& p, int first, int pieces,
                                                   int i0, int team, float* s) {
  float* const s_w = s;                                   // [pieces][COLS]: maximum, then weight
  float* const s_l = s_w + kMergeSharedPieces * COLS;     // [pieces][COLS]
  float* const s_inv = s_l + kMergeSharedPieces * COLS;   // [COLS]: 1 / sum, -1: poisoned
  const int live = p.live;
  for (int i = i0; i < pieces * COLS; i += team) {
    const float2 ml = __ldcg(a.part_ml + cross_tile<1>(first, i / COLS, 0) * COLS + i % COLS);
    s_w[i] = ml.x;
    s_l[i] = ml.y;
  }
  __syncthreads();
  for (int c = i0; c < live; c += team) {
    float M = -INFINITY, L = 0.f;
    bool bad = false;
    for (int j = 0; j < pieces; ++j) M = fmaxf(M, s_w[j * COLS + c]);
    for (int j = 0; j < pieces; ++j) {
      const float w = cross_weight(s_w[j * COLS + c], M), l = s_l[j * COLS + c];
      bad |= l < 0.f;
      L = fmaf(w, l, L);
      s_w[j * COLS + c] = w;
    }
    s_inv[c] = bad ? -1.f : 1.f / L;
  }
  __syncthreads();
  const int units = live * (D / 4);
  for (int u0 = i0; u0 < units; u0 += UNITS * team) {
    int c[UNITS], ch[UNITS];
    float acc[UNITS][4];
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const int x = min(u0 + u * team, units - 1);  // (a repeat is stored twice, alike)
      ch[u] = x / (2 * live) * 2 + (x & 1);         // (the two chunks of a stored 8 side by side)
      c[u] = x % (2 * live) >> 1;
#pragma unroll
      for (int d = 0; d < 4; ++d) acc[u][d] = 0.f;
    }
    for (int j0 = 0; j0 < pieces; j0 += AHEAD) {
      float4 o[AHEAD][UNITS];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        if (j0 + j >= pieces) break;
#pragma unroll
        for (int u = 0; u < UNITS; ++u)
          o[j][u] = __ldcg(reinterpret_cast<const float4*>(a.part_o + cross_tile<1>(first, j0 + j, 0) * COLS * D +
                                                           (ch[u] / 2 * COLS + c[u]) * 8 + (ch[u] & 1) * 4));
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        if (j0 + j >= pieces) break;
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          const float w = s_w[(j0 + j) * COLS + c[u]];
          acc[u][0] = fmaf(w, o[j][u].x, acc[u][0]);
          acc[u][1] = fmaf(w, o[j][u].y, acc[u][1]);
          acc[u][2] = fmaf(w, o[j][u].z, acc[u][2]);
          acc[u][3] = fmaf(w, o[j][u].w, acc[u][3]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const float inv = s_inv[c[u]];
#pragma unroll
      for (int d = 0; d < 4; ++d) acc[u][d] = inv == -1.f ? 0.f : acc[u][d] * inv;
      cross_store4(static_cast<T*>(a.out) + (p.base(a) + cross_column(a, c[u])) * D + ch[u] * 4, acc[u]);
    }
  }
}
#endif

}  // namespace pa
