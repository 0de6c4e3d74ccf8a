// cross_attention.h -- what the kernels of pa_cross_attention share: the
// arguments, the work's layout in the workspace, and the walk over a worker's
// share of it.
//
// An item is (sequence, KV head, group of `cols` query columns); a column is
// one (query row, query head) pair of the KV head, column c of a sequence
// being row c / G, head c % G.  An item's keys are cut into tiles of `keys`;
// an item without keys counts one tile (its rows are written as zeros).  All
// tiles are laid end to end in (sequence, KV head, group, tile) order and cut
// into equal contiguous shares, one per worker, so every worker gets the same
// number of tiles however skewed the lengths are.  The run of one item's
// tiles inside a share is a piece: a piece that is the whole item stores the
// output, any other stores a partial state (m, l, o) for the merge kernel:
//   M = max_j m_j,  out = sum_j 2^(m_j - M) o_j / sum_j 2^(m_j - M) l_j.
// A worker has at most two partial pieces, hence two partial slots: slot 2 w
// for the piece its share begins inside of, 2 w + 1 for the one it begins and
// does not finish.  Nothing in the workspace outlives a call or needs zeroing.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
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
  int num_seqs, num_rows, num_q_heads, num_kv_heads, head_dim;
  int group_log2;              // log2 of the query heads per KV head
  int max_blocks_per_seq, num_blocks, len_cap;
  float scale_log2;            // scale * log2(e)
  int32_t* err_flag;
  // the cut of the work
  int cols, keys;              // columns of an item, keys of a tile
  int max_workers;             // workers of the launch
  int min_tiles;               // a worker's share is at least this long
  // workspace
  long long* head;             // {tiles, workers}
  int4* rec;                   // [max_workers]: {sequence, item, tile, tiles of the share}
  int4* meta;                  // [num_seqs]: {first row, rows, keys, groups of columns}
  long long* start;            // [num_seqs + 1]: tiles before each sequence
  float2* part_ml;             // [2 max_workers][cols]: running max (log2 units), sum of weights
  float* part_o;               // [2 max_workers][cols][head_dim]
  CUtensorMap tm_k;            // caches as [num_blocks * Hkv * 16][head_dim] (tensor loads)
  CUtensorMap tm_v;
};

// How the work of a call is cut, and by which kernel it is done.
struct CrossPlan {
  int cols, keys, max_workers, min_tiles;
  size_t rec_off, meta_off, start_off, ml_off, o_off, bytes;
};
CrossPlan cross_plan(int num_seqs, int num_rows, int num_q_heads, int num_kv_heads, int head_dim,
                     int elem_bytes, int num_sms);
cudaError_t launch_cross_attention(CrossArgs& a, int elem_bytes, int num_sms, cudaStream_t stream);

#ifdef __CUDACC__
// A run of one item's tiles.
struct CrossPiece {
  int s, kvh, grp;   // sequence, KV head, group of columns
  int t0, t1, nt;    // tiles [t0, t1) of the item's nt
  int q0, Q, n;      // first query row, rows, keys
  int slot;          // partial slot, or -1: the whole item
};

__device__ __forceinline__ int cross_tiles(int n, int keys) { return n > 0 ? (n + keys - 1) / keys : 1; }

// The pieces of worker w's share, in order.
struct CrossWalk {
  int s, item, tile, left, w;
  int4 m;
  __device__ __forceinline__ CrossWalk(const CrossArgs& a, int worker) : w(worker) {
    // (written by the plan kernel while this grid may already have been
    // launched: read through L2, never through the read-only path)
    const int4 r = __ldcg(a.rec + worker);
    s = r.x;
    item = r.y;
    tile = r.z;
    left = worker < __ldcg(a.head + 1) ? r.w : 0;
    m = left > 0 ? __ldcg(a.meta + s) : make_int4(0, 0, 0, 0);
  }
  __device__ __forceinline__ bool next(const CrossArgs& a, CrossPiece* p) {
    if (left <= 0) return false;
    while (item >= a.num_kv_heads * m.w) {
      if (++s >= a.num_seqs) return false;
      m = __ldcg(a.meta + s);
      item = tile = 0;
    }
    p->s = s;
    p->kvh = item / m.w;
    p->grp = item - p->kvh * m.w;
    p->q0 = m.x;
    p->Q = m.y;
    p->n = m.z;
    p->nt = cross_tiles(m.z, a.keys);
    p->t0 = tile;
    p->t1 = min(p->nt, tile + left);
    p->slot = tile > 0 ? 2 * w : p->t1 < p->nt ? 2 * w + 1 : -1;
    left -= p->t1 - p->t0;
    ++item;
    tile = 0;
    return true;
  }
};
#endif

}  // namespace pa
