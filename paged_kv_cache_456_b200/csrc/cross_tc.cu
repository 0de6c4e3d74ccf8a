// cross_tc.cu -- cross attention of many query columns on the tcgen05 tensor
// cores (bf16).
//
// An item is 256 query columns of one (sequence, KV head), two tiles A and B
// of 128 (the M side of an MMA), which share every tile of 128 keys:
//   S_t[128 x 128] = Q_t K^T              TMEM, fp32
//   P_t = 2^(S_t scale log2 e - m)        one thread per column; bf16, into
//                                         the TMEM columns S_t was read from
//   O_t[128 x D]  += P_t V                TMEM, fp32
// The running maximum m (log2 units) is raised, and O_t rescaled, only when a
// score exceeds it by 2^8; the sum of the weights is taken in fp32 before
// they are rounded for the product.
//
// Roles (12 warps, one CTA per SM, one worker each):
//   warps 0-3, 4-7  softmax of tile A, of tile B: thread c owns column c (TMEM
//                   lane c): its q row, S row, P row and O row;
//   warp 8          producer: K and V tiles into one ring by 2-D tensor loads
//                   (16-row blocks found through the block table);
//   warp 9          MMA issue, in the order  P_A V, S_A', P_B V, S_B'  where '
//                   is the next tile of the worker's share, of the next piece
//                   at a piece's end: one tile's softmax always runs beside
//                   the other's MMAs.  P is handed over in halves of 64 keys,
//                   so that its product starts half a softmax early;
//   warp 10         the q rows of each next piece, once its last scores are done
//                   (warp 11 completes the third warpgroup).
// The softmax of a tile takes the last running maximum on trust: the first
// half's weights are computed while the tile's own maximum is, and computed
// again in the rare case that it exceeds the running one by 2^8 or more.
// The output leaves straight from registers, 32 bytes (a whole sector) a lane and
// store; whole rows by way of a staging area took as long.
// Tried and slower (4 x 4096 x 4096, 32 heads; this form 0.90 ms): S in two
// buffers of 64 keys a tile, whose MMAs cost a third more operand traffic (0.96
// to 1.25 ms); an MMA warp for each tile, whose softmaxes then fall into step
// (1.03 ms); an eighth to a half of the weights from a cubic on the FMA units
// (0.94 to 0.99 ms).
// A piece with at most 128 columns leaves tile B out.  Every mbarrier wait is
// bounded, by what it waits for: one tile's work, or for the q warp and a
// warpgroup whose column tile is left out the tiles of whole pieces.  A wait that
// runs out sets PA_ERRBIT_TIMEOUT and every role leaves.
#include <cstdint>
#include <type_traits>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cross_attention.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace pa {
namespace {

constexpr int kCols = 128, kTiles = 2, kKeys = 128;
// What an item costs besides its tiles (0, 1, 2, 3: 16 ragged sequences 69.0, 58.2, 59.4,
// 61.2 us; 32 of 128 rows against 700 keys 83, 81, 77, 76).
constexpr int kExtra = 1;
constexpr int kBlocks = kKeys / kBlockSize;  // blocks of a K/V tile
constexpr int kWg = 128;                     // threads of a softmax warpgroup
constexpr int kProducerWarp = 8, kMmaWarp = 9, kQWarp = 10, kThreads = 384;
// registers: 168 a thread at launch (384 x 168 = 64512), then 192 for the two
// softmax warpgroups and 120 for the third (256 x 192 + 128 x 120 = 64512)
constexpr int kRegsSoftmax = 192, kRegsRest = 120;
constexpr int kTmemCols = 512;               // S_t at 128 t, O_t at 256 + 128 t
constexpr float kGrow = 8.f;                 // log2 growth of a maximum before O is rescaled

template <int D>
struct Shape {
  static constexpr int KB = D / 64;             // 128-byte blocks of a row
  static constexpr int QT = kCols * D * 2;      // bytes of a Q tile
  static constexpr int KT = kKeys * D * 2;      // bytes of a K or V tile
  static constexpr int HALF = kKeys * 128;      // bytes of a 64-element half of it
  static constexpr int NS = D == 128 ? 4 : 8;   // ring slots
  static constexpr int SMEM = 1024 + kTiles * QT + NS * KT + 256;
};

__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// a bounded wait whose outcome the whole warp shares
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity) {
  bool ok = try_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = global_timer_ns();
    while (!(ok = try_wait(bar, parity)) && global_timer_ns() - t0 <= kWaitLimitNs) {
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// The same for a wait through `tiles` tiles of other roles' work: that many
// times the limit of one, given up as soon as another role gives up (which each
// of them does within the limit of one tile).
__device__ __forceinline__ bool wait_long(uint32_t bar, uint32_t parity, int tiles, const int* abort) {
  bool ok = try_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = global_timer_ns(), limit = kWaitLimitNs * static_cast<uint64_t>(tiles + 1);
    while (!(ok = try_wait(bar, parity)) && *reinterpret_cast<const volatile int*>(abort) == 0 &&
           global_timer_ns() - t0 <= limit) {
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// 2^x; results below the smallest normal number are 0 (they are weights of at
// most 2^8, rounded to bf16)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// a 3-D tensor load (coordinate x a multiple of 16 bytes' worth of elements)
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// ---- pieces of the softmax: 32 scores of a column -----------------------------
__device__ __forceinline__ void maxima(const uint32_t (&s)[32], float (&m)[4]) {
#pragma unroll
  for (int k = 0; k < 32; k += 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = max3(m[i], __uint_as_float(s[k + i]), __uint_as_float(s[k + i + 4]));
  }
}
// 2^(s mul - m) as bf16 pairs in w[at, at + 16), added up in l before the rounding.
// (An MMA takes both operands in one type, and V is bf16.  Adding up the weights as
// rounded instead would take two instructions more a pair, in the chain that this
// kernel waits for, and gains little: the output's error falls by 1.5 % over 100
// keys and 0.1 to 0.5 % over 1100 or 4096, computed in 64 bits for values of mean 0
// to 2 deviations.)
__device__ __forceinline__ void weights(const uint32_t (&s)[32], float mul, float m, uint32_t (&w)[32], int at,
                                        float2 (&l)[2]) {
  // (a column that saw only -inf: an offset of 0 keeps its weights at 0)
  const float nm = m == -INFINITY ? 0.f : -m;
  const float2 mul2 = make_float2(mul, mul), nm2 = make_float2(nm, nm);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float2 x =
        __ffma2_rn(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), mul2, nm2);
    const float2 y = make_float2(ex2(x.x), ex2(x.y));
    l[e & 1] = __fadd2_rn(l[e & 1], y);
    w[at + e] = pack_bf16(y.x, y.y);
  }
}
__device__ __forceinline__ void store_p(uint32_t addr, const uint32_t (&w)[32]) {
  tc::tmem_st32(addr, w);
  tc::tmem_wait_st();
}

__device__ __forceinline__ int live_tiles(const CrossPiece& p) { return p.live > kCols ? 2 : 1; }
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A warp's walk over the share and the piece it is at live in shared memory:
// in registers they would be held through the tile loops, which have none to
// spare.  One lane steps; a piece's fields are read again where they are used.
struct WarpWalk {
  CrossWalk walk;
  CrossPiece piece[2];  // (the softmax steps to the next piece while it is at one)
  __device__ __forceinline__ bool next(const CrossArgs& a, bool with_keys, int to = 0) {
    bool ok = false;
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
      while ((ok = walk.next(a, kTiles * kCols, kKeys, kExtra, &piece[to])) && with_keys && piece[to].n == 0) {
      }
    ok = __any_sync(0xffffffffu, ok);
    __syncwarp();
    return ok;
  }
  __device__ __forceinline__ CrossPiece get(int from = 0) const {
    CrossPiece p;
    static_assert(sizeof(CrossPiece) % 4 == 0, "copied by words");
    const volatile int* const src = reinterpret_cast<const volatile int*>(&piece[from]);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(CrossPiece) / 4); ++i) reinterpret_cast<int*>(&p)[i] = src[i];
    return p;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) cross_tc_kernel(const __grid_constant__ CrossArgs a) {
  using C = Shape<D>;
  constexpr int KB = C::KB, QT = C::QT, KT = C::KT, HALF = C::HALF, NS = C::NS;
  constexpr uint32_t IDESC_S = tc::idesc_bf16_f32(kCols, kKeys, false);
  constexpr uint32_t IDESC_O = tc::idesc_bf16_f32(kCols, D, true);

  extern __shared__ unsigned char smem_raw[];
  unsigned char* const sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  unsigned char* const sQ = sm;                  // [kTiles][QT]
  unsigned char* const sR = sQ + kTiles * QT;    // [NS][KT]: K and V tiles in turn
  const uint32_t b0 = smem_addr(sR + NS * KT);
  // barriers: full[NS] empty[NS] | per tile: sfull, p[2], odone, qfull, qempty, sync | drain
  auto FULL = [&](int i) { return b0 + 8 * i; };
  auto EMPTY = [&](int i) { return b0 + 8 * (NS + i); };
  auto TB = [&](int t, int i) { return b0 + 8 * (2 * NS + 7 * t + i); };
  enum { SFULL = 0, P0 = 1, ODONE = 3, QFULL = 4, QEMPTY = 5, SYNC = 6 };
  const uint32_t DRAIN = b0 + 8 * (2 * NS + 7 * kTiles);
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ CrossTotal s_total;
  __shared__ WarpWalk s_walk[kThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    prefetch_tensormap(&a.tm_k);
    prefetch_tensormap(&a.tm_v);
    prefetch_tensormap(&a.tm_q);
    for (int i = 0; i < NS; ++i) {
      mbar_init(FULL(i), 1);
      mbar_init(EMPTY(i), 1);
    }
    for (int t = 0; t < kTiles; ++t) {
      mbar_init(TB(t, SFULL), 1);
      mbar_init(TB(t, P0), kWg);
      mbar_init(TB(t, P0 + 1), kWg);
      mbar_init(TB(t, ODONE), 1);
      mbar_init(TB(t, QFULL), 1);
      mbar_init(TB(t, QEMPTY), 1);
      mbar_init(TB(t, SYNC), kWg);
    }
    mbar_init(DRAIN, 1);
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(smem_addr(&s_tmem), kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  {
    const CrossShare share = cross_share<kThreads>(a, kTiles * kCols, kKeys, kExtra, &s_total);  // (synchronises the CTA)
    if (lane == 0) s_walk[warp].walk = CrossWalk(a, share, kTiles * kCols);
    __syncwarp();
  }
  WarpWalk& walk = s_walk[warp];
  tc::fence_after_sync();
  const uint32_t tmem = s_tmem;

  auto timeout = [&]() {
    if (atomicExch(&s_abort, 1) == 0 && a.err_flag) atomicOr(a.err_flag, kErrTimeout);
  };
  auto aborted = [&]() { return __any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&s_abort) != 0); };

  if (warp >= 8) {
    regs_dec<kRegsRest>();
    if (warp == kProducerWarp) {
      // ---------------- producer: K(0) V(0) K(1) V(1) ... over all steps ----------------
      const int oob = a.num_blocks * a.num_kv_heads * kBlockSize;  // a row past the caches: zeros
      int idx = 0;
      bool ok = true;
      auto issue = [&](const CUtensorMap* map, int y) -> bool {
        const int st = idx % NS;
        if (idx >= NS && !wait_all(EMPTY(st), ((idx / NS) - 1) & 1)) return false;
        if (lane == 0) mbar_arrive_expect_tx(FULL(st), KT);
        __syncwarp();
        if (lane < kBlocks) {
          const uint32_t dst = smem_addr(sR + st * KT) + lane * kBlockSize * 128;
#pragma unroll
          for (int h = 0; h < KB; ++h) tma_load_2d(dst + h * HALF, map, h * 64, y, FULL(st));
        }
        ++idx;
        return true;
      };
      while (ok && walk.next(a, true)) {
        const CrossPiece p = walk.get();
        const int32_t* const table = a.block_tables + static_cast<size_t>(p.s) * a.max_blocks_per_seq;
        auto rows_of = [&](int j) -> int {  // this lane's block of tile j
          const int b = j * kBlocks + lane;
          int y = oob;
          if (lane < kBlocks && j < p.t1 && b * kBlockSize < p.n) {
            const int id = __ldg(table + b);
            if (id >= 0 && id < a.num_blocks) y = (id * a.num_kv_heads + p.kvh) * kBlockSize;
          }
          return y;
        };
        int ynext = rows_of(p.t0);
        for (int j = p.t0; j < p.t1; ++j) {
          const int y = ynext;
          ynext = rows_of(j + 1);
          if (aborted() || !issue(&a.tm_k, y) || !issue(&a.tm_v, y)) {
            ok = false;
            break;
          }
        }
      }
      if (!ok) timeout();
      // every load issued lands before the CTA can exit
      for (int i = max(0, idx - NS); i < idx; ++i) wait_all(FULL(i % NS), (i / NS) & 1);
    } else if (warp == kMmaWarp) {
      // ---------------- MMA issue --------------------------------------------------------
      const uint64_t qdesc = tc::sdesc_sw128(smem_addr(sQ), 16, 1024);
      const uint64_t kdesc = tc::sdesc_sw128(smem_addr(sR), 16, 1024);
      const uint64_t vdesc = tc::sdesc_sw128(smem_addr(sR), HALF, 1024);
      int step = 0;                       // K of this step in ring index 2 step, V in 2 step + 1
      int pn[kTiles] = {0, 0}, qn[kTiles] = {0, 0};
      bool ok = true;
      // S_t of the step `s`, whose K has landed
      auto issue_s = [&](int t, int s, bool last, bool q_done) {
        const int st = (2 * s) % NS;
        const uint64_t qd = tc::sdesc_advance(qdesc, t * QT), kd = tc::sdesc_advance(kdesc, st * KT);
        if (tc::elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t qo = (k / 4) * (kCols * 128) + (k % 4) * 32, ko = (k / 4) * HALF + (k % 4) * 32;
            tc::mma_bf16_ss(tmem + t * kKeys, tc::sdesc_advance(qd, qo), tc::sdesc_advance(kd, ko), IDESC_S, k > 0);
          }
          tc::commit(TB(t, SFULL));
          if (last) tc::commit(EMPTY(st));
          if (q_done) tc::commit(TB(t, QEMPTY));
        }
        __syncwarp();
      };
      // (of a piece this warp needs its tiles and which column tiles live)
      int left = 0, live = 0, nleft = 0, nlive = 0;
      auto advance = [&]() {
        nleft = nlive = 0;
        if (walk.next(a, true)) {
          const CrossPiece y = walk.get();
          nleft = y.t1 - y.t0;
          nlive = live_tiles(y);
        }
      };
      advance();
      bool begun = false;  // O of the piece holds a product
      left = nleft;
      live = nlive;
      if (left > 0) {
        ok = wait_all(FULL(0), 0);
        for (int t = 0; t < live && ok; ++t) {
          ok = wait_all(TB(t, QFULL), (qn[t]++) & 1);
          tc::fence_after_sync();
          if (ok) issue_s(t, 0, t == live - 1, left == 1);
        }
      }
      while (left > 0 && ok) {
        const bool same = left > 1;
        if (same) {
          nleft = left - 1;
          nlive = live;
        } else {
          advance();
        }
        const int vi = 2 * step + 1, ki = vi + 1;
        const uint64_t vd = tc::sdesc_advance(vdesc, (vi % NS) * KT);
        if (aborted()) { ok = false; break; }
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          if (t < live) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (!wait_all(TB(t, P0 + h), pn[t] & 1)) { ok = false; break; }
              if (t == 0 && h == 0 && !wait_all(FULL(vi % NS), (vi / NS) & 1)) { ok = false; break; }
              tc::fence_after_sync();
              if (tc::elect_one()) {
#pragma unroll
                for (int k = 4 * h; k < 4 * h + 4; ++k)
                  tc::mma_bf16_ts(tmem + kTiles * kKeys + t * 128, tmem + t * kKeys + k * 8,
                                  tc::sdesc_advance(vd, k * 16 * 128), IDESC_O, (begun || k > 0) ? 1u : 0u);
                if (h == 1) {
                  if (!same) tc::commit(TB(t, ODONE));
                  if (t == live - 1) tc::commit(EMPTY(vi % NS));
                }
              }
              __syncwarp();
            }
            if (!ok) break;
            ++pn[t];
          }
          if (t < nlive) {
            if (t == 0 && !wait_all(FULL(ki % NS), (ki / NS) & 1)) { ok = false; break; }
            if (!same && !wait_all(TB(t, QFULL), (qn[t]++) & 1)) { ok = false; break; }
            tc::fence_after_sync();
            issue_s(t, step + 1, t == nlive - 1, nleft == 1);
          }
        }
        ++step;
        begun = same;
        left = nleft;
        live = nlive;
      }
      if (!ok) timeout();
      // every MMA issued has completed before the TMEM can be freed
      if (tc::elect_one()) tc::commit(DRAIN);
      wait_all(DRAIN, 0);
      __syncwarp();
    } else if (warp == kQWarp) {
      // ---------------- q rows: 128 / G rows x G heads a tile, by tensor loads (columns past
      // the sequence's last get other rows, or zeros past the tensor's end) -------------
      int qn[kTiles] = {0, 0}, before = 0;  // (the last piece's tiles)
      bool ok = true;
      const int rows = kCols >> a.group_log2;
      while (ok && walk.next(a, true)) {
        const CrossPiece p = walk.get();
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          if (t >= live_tiles(p) || !ok) continue;
          // (a wait through the last piece)
          if (aborted() || (qn[t] > 0 && !wait_long(TB(t, QEMPTY), (qn[t] - 1) & 1, before, &s_abort))) {
            ok = false;
            continue;
          }
          ++qn[t];
          if (lane == 0) {
            mbar_arrive_expect_tx(TB(t, QFULL), QT);
#pragma unroll
            for (int h = 0; h < KB; ++h)
              tma_load_3d(smem_addr(sQ + t * QT) + h * (kCols * 128), &a.tm_q, h * 64, p.kvh << a.group_log2,
                          p.row + t * rows, TB(t, QFULL));
          }
          __syncwarp();
        }
        before = p.t1 - p.t0;
      }
      if (!ok) timeout();
      for (int t = 0; t < kTiles; ++t)  // (the last loads land before the CTA can exit)
        if (qn[t] > 0) wait_all(TB(t, QFULL), (qn[t] - 1) & 1);
    }
  } else {
    regs_inc<kRegsSoftmax>();
    // ---------------- softmax: warpgroup t serves tile t, thread col its column -------
    const int t = warp / 4, col = tid % kWg;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16);
    const uint32_t s_addr = lane_base + t * kKeys, o_addr = lane_base + kTiles * kKeys + t * 128;
    const bool wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
    int step = 0, sn = 0, on = 0, syncs = 0;
    int passed = 0;  // tiles of the pieces since this warpgroup's last one
    bool ok = true;
    auto group_sync = [&]() -> bool {  // the 128 threads of this warpgroup
      mbar_arrive(TB(t, SYNC));
      return wait_all(TB(t, SYNC), (syncs++) & 1);
    };
    // Scores in log2 units are s * mul: under a positive scale the maximum commutes
    // with the rounded product; another scale is applied to the scores one by one.
    const float mul = a.scale_log2 > 0.f ? a.scale_log2 : 1.f;
    // The piece at hand is walk.piece[at].  What a piece needs beside its tiles is done
    // while the tensor cores have the scores in hand: its block ids are checked behind
    // its first tile's weights, the walk goes on behind its second's.
    int at = 1;
    bool looked = false, more = false;
    while (ok) {
      if (!looked) more = walk.next(a, false, at ^ 1);
      looked = false;
      at ^= 1;
      if (!more) break;
      int left, tiles;  // keys from this tile on, tiles to go
      bool bad = false;
      {
        const CrossPiece p = walk.get(at);
        const bool mine = t < live_tiles(p);
        if (p.n == 0) {
          if (mine && t * kCols + col < p.live) {
            uint4* const dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) +
                                                        (p.base(a) + cross_column(a, t * kCols + col)) * D);
            for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0, 0, 0, 0);
          }
          continue;
        }
        tiles = p.t1 - p.t0;
        left = p.n - p.t0 * kKeys;
        if (!mine) {
          step += tiles;
          passed += tiles;
          continue;
        }
      }
      // (the first scores come when the pieces without this column tile are done)
      if (passed > 0 && !wait_long(TB(t, SFULL), sn & 1, passed, &s_abort)) { ok = false; break; }
      passed = 0;
      float m_run = -INFINITY;
      float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      bool begun = false;
      for (; tiles > 0; --tiles, left -= kKeys, ++step, begun = true) {
        // Rows past the end in the last block hold stale data, and 0 x NaN
        // would poison O: tile A's warpgroup clears them before its first P V,
        // while the scores are on their way
        if (t == 0 && left < kKeys && left % kBlockSize) {
          const int vi = 2 * step + 1;
          if (!wait_all(FULL(vi % NS), (vi / NS) & 1)) { ok = false; break; }
          unsigned char* const vt = sR + (vi % NS) * KT;
          const int nr = kBlockSize - left % kBlockSize;
          for (int i = col; i < nr * 8 * KB; i += kWg) {
            const int h = i / (nr * 8), r = left + (i / 8) % nr;
            *reinterpret_cast<uint4*>(vt + h * HALF + r * 128 + ((i % 8) << 4)) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (aborted() || !wait_all(TB(t, SFULL), (sn++) & 1)) { ok = false; break; }
        tc::fence_after_sync();
        const bool plain = left >= kKeys && a.scale_log2 > 0.f;
        // 32 scores of another tile made ready to be scaled by mul (keys past the end: -inf)
        auto prepare = [&](uint32_t (&x)[32], int c) {
          const float f = a.scale_log2 > 0.f ? 1.f : a.scale_log2;
#pragma unroll
          for (int k = 0; k < 32; ++k)
            x[k] = 32 * c + k < left ? __float_as_uint(__uint_as_float(x[k]) * f) : 0xff800000u;
        };
        uint32_t s2[32], s3[32], w[32];
        float2 lh[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        // The first half's weights under the running maximum (in a piece's first
        // tile there is none yet: they are computed again below), and the
        // tile's own maximum beside them; the second half's scores stay.
        auto front = [&](auto plain_tag) {
          constexpr bool PLAIN = decltype(plain_tag)::value;
          uint32_t s0[32], s1[32];
          tc::tmem_ld32(s_addr, s0);
          tc::tmem_wait_ld(s0);
          tc::tmem_ld32(s_addr + 32, s1);
          if (!PLAIN) prepare(s0, 0);
          maxima(s0, m4);
          weights(s0, mul, m_run, w, 0, lh);
          tc::tmem_wait_ld(s1);
          tc::tmem_ld32(s_addr + 64, s2);
          if (!PLAIN) prepare(s1, 1);
          maxima(s1, m4);
          weights(s1, mul, m_run, w, 16, lh);
          tc::tmem_wait_ld(s2);
          tc::tmem_ld32(s_addr + 96, s3);
          if (!PLAIN) prepare(s2, 2);
          maxima(s2, m4);
          tc::tmem_wait_ld(s3);
          if (!PLAIN) prepare(s3, 3);
          maxima(s3, m4);
        };
        if (plain) front(std::true_type{}); else front(std::false_type{});
        const float mx = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]) * mul;
        const bool grow = mx > m_run + kGrow;
        if (!begun || __any_sync(0xffffffffu, grow)) {
          float al = 1.f;
          if (grow) {
            al = ex2(m_run - mx);  // (0 while nothing was seen)
            m_run = mx;
          }
          l2[0] = __fmul2_rn(l2[0], make_float2(al, al));
          l2[1] = __fmul2_rn(l2[1], make_float2(al, al));
          lh[0] = lh[1] = make_float2(0.f, 0.f);
          if (begun) {
            // (S of this tile was issued behind P V of the last one: O is complete)
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
              tc::tmem_ld32(o_addr + i * 32, w);
              tc::tmem_wait_ld(w);
#pragma unroll
              for (int k = 0; k < 32; ++k) w[k] = __float_as_uint(__uint_as_float(w[k]) * al);
              tc::tmem_st32(o_addr + i * 32, w);
            }
          }
          uint32_t s0[32], s1[32];  // the first half again
          tc::tmem_ld32(s_addr, s0);
          tc::tmem_wait_ld(s0);
          if (!plain) prepare(s0, 0);
          weights(s0, mul, m_run, w, 0, lh);
          tc::tmem_ld32(s_addr + 32, s1);
          tc::tmem_wait_ld(s1);
          if (!plain) prepare(s1, 1);
          weights(s1, mul, m_run, w, 16, lh);
        }
        store_p(s_addr, w);
        tc::fence_before_sync();
        mbar_arrive(TB(t, P0));
        weights(s2, mul, m_run, w, 0, lh);
        weights(s3, mul, m_run, w, 16, lh);
        store_p(s_addr + 32, w);
        tc::fence_before_sync();
        mbar_arrive(TB(t, P0 + 1));
        l2[0] = __fadd2_rn(l2[0], lh[0]);
        l2[1] = __fadd2_rn(l2[1], lh[1]);
        if (!begun) {
          bad = __any_sync(0xffffffffu, cross_bad_block(a, walk.get(at), kKeys, lane, 32));
        } else if (!looked) {
          more = walk.next(a, false, at ^ 1);
          looked = true;
        }
      }
      if (!ok) break;
      // ---- the piece's O
      const CrossPiece p = walk.get(at);
      const float2 la = __fadd2_rn(l2[0], l2[1]);
      const float l_run = la.x + la.y;
      if (bad && lane == 0 && a.err_flag) atomicOr(a.err_flag, kErrBlockId);
      const size_t pt = static_cast<size_t>(max(p.slot, 0)) * kTiles + t;
      // A piece of a cut item: if every other piece has stored its partial, this
      // one is merged with them straight from tensor memory, else it is stored
      // (most items are cut in two, and the part a share begins with is long done).
      int first = blockIdx.x, pieces = 1;
      bool store = false;
      float wgt = 1.f, L = l_run, M = m_run;  // this piece's weight, the item's sum and maximum
      bool zero = bad;
      // Of the y-th other piece: its slot, m and l, dims from 32 q on.  Of two pieces the
      // other's dims are read 32 ahead of their use, into v; its weight is wv.
      int mine = 0;
      float wv = 0.f;
      auto slot_of = [&](int y) { return cross_tile<kTiles>(first, y + (y >= mine), t); };
      auto ml_of = [&](int y) { return a.part_ml + slot_of(y) * kCols + col; };
      auto dims_of = [&](int q, int y) {
        return reinterpret_cast<const float4*>(a.part_o + slot_of(y) * kCols * D) + 8 * q * kCols + col;
      };
      if (p.slot >= 0) {
        cross_chain(s_total, p, &first, &pieces);
        if (col == 0) s_total.old[t][p.slot & 1] = atomicAdd(a.count + 2 * first + t, 0u);
        if (!group_sync()) { ok = false; break; }
        store = s_total.old[t][p.slot & 1] != static_cast<unsigned>(pieces - 1);
        if (!store) {
          __threadfence();
          mine = blockIdx.x - first;
          const float2 ml0 = __ldcg(ml_of(0));
          M = fmaxf(M, ml0.x);
          for (int y = 1; y < pieces - 1; ++y) M = fmaxf(M, __ldcg(ml_of(y)).x);
          L = 0.f;
          for (int x = 0; x < pieces; ++x) {
            const float2 ml = x == mine ? make_float2(m_run, bad ? -1.f : l_run)
                              : x == (mine == 0) ? ml0 : __ldcg(ml_of(x - (x > mine)));
            zero |= ml.y < 0.f;
            L = fmaf(cross_weight(ml.x, M), ml.y, L);
          }
          wv = cross_weight(ml0.x, M);
          wgt = cross_weight(m_run, M);
          if (col == 0) a.count[2 * first + t] = 0;
        }
      }
      if (!wait_all(TB(t, ODONE), (on++) & 1)) { ok = false; break; }
      tc::fence_after_sync();
      const float inv = 1.f / L;
      const bool live = t * kCols + col < p.live;
      __nv_bfloat16* const dst = static_cast<__nv_bfloat16*>(a.out) +
                                 (p.base(a) + (live ? cross_column(a, t * kCols + col) : 0)) * D;
      auto emit = [&](int q, const uint32_t (&o)[32]) {  // dims 32 q to 32 q + 31 of the output
        if (!live) return;
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // 16 dims (32 bytes) at a time
          uint32_t v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            v[e] = zero ? 0u
                        : pack_bf16(__uint_as_float(o[16 * i + 2 * e]) * inv, __uint_as_float(o[16 * i + 2 * e + 1]) * inv);
          uint4* const to = reinterpret_cast<uint4*>(dst + 32 * q + 16 * i);
          if (wide) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]),
                         "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                         : "memory");
          } else {
            to[0] = make_uint4(v[0], v[1], v[2], v[3]);
            to[1] = make_uint4(v[4], v[5], v[6], v[7]);
          }
        }
      };
      // (every lane runs the warp-wide TMEM loads; only live columns are stored)
      const bool pair = pieces == 2 && !store;
      if (pair) {  // w_0 o_0 + w_1 o_1
        float4 v[8];
        const float4* const head = dims_of(0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __ldcg(head + i * kCols);
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          tc::tmem_ld32(o_addr + 32 * q, o);
          tc::tmem_wait_ld(o);
          const bool go_on = q + 1 < D / 32;
          const float4* const src = dims_of(q + 1, 0);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float own = __uint_as_float(o[4 * i + e]);
              o[4 * i + e] = __float_as_uint(mine == 0 ? fmaf(wv, x[e], wgt * own) : fmaf(wgt, own, wv * x[e]));
            }
            if (go_on) v[i] = __ldcg(src + i * kCols);
          }
          emit(q, o);
        }
      }
#pragma unroll 1
      for (int q = 0; q < (pair ? 0 : D / 32); ++q) {
        uint32_t o[32];
        tc::tmem_ld32(o_addr + 32 * q, o);
        tc::tmem_wait_ld(o);
        const int pq = (8 * q * kCols + col) * 4;  // these dims in a partial
        if (store) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(a.part_o + pt * kCols * D + pq + i * kCols * 4) =
                make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          continue;
        }
        if (pieces > 1) {
          float acc[32];
          float4 v[8];
#pragma unroll
          for (int k = 0; k < 32; ++k) acc[k] = 0.f;
          for (int x = 0; x < pieces; ++x) {
            if (x == mine) {
#pragma unroll
              for (int k = 0; k < 32; ++k) acc[k] = fmaf(wgt, __uint_as_float(o[k]), acc[k]);
              continue;
            }
            const int y = x - (x > mine);
            const float wx = cross_weight(__ldcg(ml_of(y)).x, M);
            const float4* const src = dims_of(q, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __ldcg(src + i * kCols);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              acc[4 * i] = fmaf(wx, v[i].x, acc[4 * i]);
              acc[4 * i + 1] = fmaf(wx, v[i].y, acc[4 * i + 1]);
              acc[4 * i + 2] = fmaf(wx, v[i].z, acc[4 * i + 2]);
              acc[4 * i + 3] = fmaf(wx, v[i].w, acc[4 * i + 3]);
            }
          }
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(acc[k]);
        }
        emit(q, o);
      }
      tc::fence_before_sync();  // (O has been read before this warpgroup's next P lets it be written)
      if (store) {
        a.part_ml[pt * kCols + col] = make_float2(m_run, bad ? -1.f : l_run);
        __threadfence();
        if (!group_sync()) { ok = false; break; }
        if (col == 0) s_total.old[t][p.slot & 1] = atomicInc(a.count + 2 * first + t, pieces - 1);
        if (!group_sync()) { ok = false; break; }
        if (s_total.old[t][p.slot & 1] == static_cast<unsigned>(pieces - 1)) {
          __threadfence();
          cross_merge<__nv_bfloat16, D, kCols, kTiles, 4, 2, 4>(a, p, first, pieces, t, col, kWg);
        }
      }
    }
    if (!ok) timeout();
  }

  // every role is out of its loop; the MMAs have completed
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kTmemCols);
}

template <int D>
CrossKernel info() {
  CrossKernel k{};
  k.fn = reinterpret_cast<const void*>(&cross_tc_kernel<D>);
  k.threads = kThreads;
  k.ctas_per_sm = 1;
  k.smem = Shape<D>::SMEM;
  k.cols = kTiles * kCols;
  k.keys = kKeys;
  k.extra = kExtra;
  k.tma_q = true;
  return k;
}

}  // namespace

CrossKernel cross_tc_kernel_info(int head_dim) { return head_dim == 64 ? info<64>() : info<128>(); }

}  // namespace pa
