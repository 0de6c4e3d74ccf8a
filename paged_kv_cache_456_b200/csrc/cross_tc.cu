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
//   warps 10, 11    none (they complete the third warpgroup);
//   warp 9          MMA issue, in the order  P_A V, S_A', P_B V, S_B'  where '
//                   is the next tile of the worker's share, of the next piece
//                   at a piece's end: one tile's softmax always runs beside
//                   the other's MMAs.  P is handed over in halves of 64 keys,
//                   so that its product starts half a softmax early.
// A piece with at most 128 columns leaves tile B out.  Every mbarrier wait is
// bounded; a wait that runs out sets PA_ERRBIT_TIMEOUT and every role leaves.
#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cross_attention.h"
#include "cross_kernels.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace pa {
namespace {

constexpr int kCols = 128, kTiles = 2, kKeys = 128;
constexpr int kBlocks = kKeys / kBlockSize;  // blocks of a K/V tile
constexpr int kWg = 128;                     // threads of a softmax warpgroup
constexpr int kProducerWarp = 8, kMmaWarp = 9, kThreads = 384;
// registers: 168 a thread at launch (384 x 168 = 64512), then 208 for the two
// softmax warpgroups and 80 for the third (256 x 208 + 128 x 80 = 63488)
constexpr int kRegsSoftmax = 208, kRegsRest = 80;
constexpr int kTmemCols = 512;               // S_t at 128 t, O_t at 256 + 128 t
constexpr float kGrow = 8.f;                 // log2 growth of a maximum before O is rescaled

template <int D>
struct Shape {
  static constexpr int KB = D / 64;             // 128-byte blocks of a row
  static constexpr int QT = kCols * D * 2;      // bytes of a Q tile
  static constexpr int KT = kKeys * D * 2;      // bytes of a K or V tile
  static constexpr int HALF = kKeys * 128;      // bytes of a 64-element half of it
  static constexpr int NS = D == 128 ? 5 : 8;   // ring slots
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
__device__ __forceinline__ void st_wide(void* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool fill) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(fill ? 16 : 0)
               : "memory");
}

template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ int live_tiles(const CrossArgs& a, const CrossPiece& p) {
  return (static_cast<long long>(p.Q) << a.group_log2) - static_cast<long long>(p.grp) * (kTiles * kCols) > kCols
             ? 2 : 1;
}
// the next piece that has keys
__device__ __forceinline__ bool next_keys(CrossWalk& w, const CrossArgs& a, CrossPiece* p) {
  while (w.next(a, p))
    if (p->n > 0) return true;
  return false;
}

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
  // barriers: full[NS] empty[NS] | per tile: sfull, p[2], odone, qfull | drain
  auto FULL = [&](int i) { return b0 + 8 * i; };
  auto EMPTY = [&](int i) { return b0 + 8 * (NS + i); };
  auto TB = [&](int t, int i) { return b0 + 8 * (2 * NS + 5 * t + i); };
  enum { SFULL = 0, P0 = 1, ODONE = 3, QFULL = 4 };
  const uint32_t DRAIN = b0 + 8 * (2 * NS + 5 * kTiles);
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(FULL(i), 1);
      mbar_init(EMPTY(i), 1);
    }
    for (int t = 0; t < kTiles; ++t) {
      mbar_init(TB(t, SFULL), 1);
      mbar_init(TB(t, P0), kWg);
      mbar_init(TB(t, P0 + 1), kWg);
      mbar_init(TB(t, ODONE), 1);
      mbar_init(TB(t, QFULL), kWg);
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
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s_tmem;

  asm volatile("griddepcontrol.wait;" ::: "memory");  // (the plan)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  auto timeout = [&]() {
    if (atomicExch(&s_abort, 1) == 0 && a.err_flag) atomicOr(a.err_flag, kErrTimeout);
  };
  auto aborted = [&]() { return __any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&s_abort) != 0); };
  CrossWalk walk(a, blockIdx.x);

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
    CrossPiece p;
    while (ok && next_keys(walk, a, &p)) {
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
    auto issue_s = [&](int t, int s, bool last) {
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
      }
      __syncwarp();
    };
    CrossPiece cur, nxt;
    bool have = next_keys(walk, a, &cur);
    int live = have ? live_tiles(a, cur) : 0, nlive = 0;
    if (have) {
      ok = wait_all(FULL(0), 0);
      for (int t = 0; t < live && ok; ++t) {
        ok = wait_all(TB(t, QFULL), (qn[t]++) & 1);
        tc::fence_after_sync();
        if (ok) issue_s(t, 0, t == live - 1);
      }
    }
    int j = cur.t0;
    while (have && ok) {
      const bool same = j + 1 < cur.t1;
      bool have_next = same;
      if (same) {
        nlive = live;
      } else {
        have_next = next_keys(walk, a, &nxt);
        nlive = have_next ? live_tiles(a, nxt) : 0;
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
                                tc::sdesc_advance(vd, k * 16 * 128), IDESC_O, (j > cur.t0 || k > 0) ? 1u : 0u);
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
        if (have_next && t < nlive) {
          if (t == 0 && !wait_all(FULL(ki % NS), (ki / NS) & 1)) { ok = false; break; }
          if (!same && !wait_all(TB(t, QFULL), (qn[t]++) & 1)) { ok = false; break; }
          tc::fence_after_sync();
          issue_s(t, step + 1, t == nlive - 1);
        }
      }
      ++step;
      if (same) {
        ++j;
      } else {
        cur = nxt;
        j = cur.t0;
        live = nlive;
        have = have_next;
      }
    }
    if (!ok) timeout();
    // every MMA issued has completed before the TMEM can be freed
    if (tc::elect_one()) tc::commit(DRAIN);
    wait_all(DRAIN, 0);
    __syncwarp();
  }
  } else {
    regs_inc<kRegsSoftmax>();
    // ---------------- softmax: warpgroup t serves tile t, thread col its column -------
    const int t = warp / 4, col = tid % kWg;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16);
    const uint32_t s_addr = lane_base + t * kKeys, o_addr = lane_base + kTiles * kKeys + t * 128;
    const bool wide_out = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
    const bool wide_part = reinterpret_cast<uintptr_t>(a.part_o) % 32 == 0;
    int step = 0, sn = 0, on = 0;
    bool ok = true;
    // this column's (row, head) in piece y as an index into q and out, -1: none
    auto column_of = [&](const CrossPiece& y) -> long long {
      const long long gc = static_cast<long long>(y.grp) * (kTiles * kCols) + t * kCols + col;
      const long long r = gc >> a.group_log2;
      if (r >= y.Q) return -1;
      return (y.q0 + r) * a.num_q_heads + (y.kvh << a.group_log2) + (gc & ((1 << a.group_log2) - 1));
    };
    auto load_q = [&](long long c) {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + (c >= 0 ? c : 0) * D;
      const uint32_t qb = smem_addr(sQ + t * QT) + col * 128;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        cp_async16_zfill(qb + (i / 8) * (kCols * 128) + (((i % 8) ^ (col % 8)) << 4), src + i * 8, c >= 0);
    };
    auto hand_q = [&]() {
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      mbar_arrive(TB(t, QFULL));
    };
    CrossPiece p, nxt;
    bool have = walk.next(a, &p), q_handed = false;
    while (have && ok) {
      const bool have_next = walk.next(a, &nxt);
      const bool mine = t < live_tiles(a, p);
      const long long c = column_of(p);
      if (p.n == 0) {
        if (mine && c >= 0) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + c * D);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0, 0, 0, 0);
        }
      } else if (!mine) {
        step += p.t1 - p.t0;
      } else {
        // (Q of a piece that follows another with keys was handed over there)
        if (!q_handed) {
          load_q(c);
          hand_q();
        }
        q_handed = false;
        const bool ahead = have_next && nxt.n > 0 && t < live_tiles(a, nxt);
        float m_run = -INFINITY;
        float2 l2[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) l2[i] = make_float2(0.f, 0.f);
        for (int j = p.t0; j < p.t1; ++j, ++step) {
          if (aborted() || !wait_all(TB(t, SFULL), (sn++) & 1)) { ok = false; break; }
          tc::fence_after_sync();
          uint32_t sv[2][64];
          tc::tmem_ld64(s_addr, sv[0]);
          tc::tmem_ld64(s_addr + 64, sv[1]);
          tc::tmem_wait_ld(sv[0]);
          tc::tmem_wait_ld(sv[1]);
          if (j == p.t1 - 1 && ahead) load_q(column_of(nxt));  // (its last S of this piece is complete)
          const int kb = j * kKeys;
          // Scores in log2 units are sv * mul: whole tiles under a positive
          // scale keep the raw scores (the maximum commutes with the rounded
          // product); otherwise they are scaled here, and keys past the end
          // set to -inf.
          float mul = a.scale_log2;
          if (kb + kKeys > p.n || !(mul > 0.f)) {
#pragma unroll
            for (int k = 0; k < kKeys; ++k)
              sv[k / 64][k % 64] =
                  kb + k < p.n ? __float_as_uint(__uint_as_float(sv[k / 64][k % 64]) * mul) : 0xff800000u;
            mul = 1.f;
          }
          float m8[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) m8[i] = -INFINITY;
#pragma unroll
          for (int k = 0; k < kKeys; k += 16) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              m8[i] = max3(m8[i], __uint_as_float(sv[k / 64][k % 64 + i]),
                           __uint_as_float(sv[k / 64][k % 64 + i + 8]));
          }
          const float mx = fmaxf(max3(max3(m8[0], m8[1], m8[2]), m8[3], m8[4]), max3(m8[5], m8[6], m8[7])) * mul;
          const bool grow = mx > m_run + kGrow;
          if (__any_sync(0xffffffffu, grow)) {
            float al = 1.f;
            if (grow) {
              al = ex2(m_run - mx);  // (0 while nothing was seen)
              m_run = mx;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) l2[i] = __fmul2_rn(l2[i], make_float2(al, al));
            if (j > p.t0) {
              // (S of this tile was issued behind P V of the last one: O is complete)
#pragma unroll 1
              for (int i = 0; i < D / 32; ++i) {
                uint32_t r[32];
                tc::tmem_ld32(o_addr + i * 32, r);
                tc::tmem_wait_ld(r);
#pragma unroll
                for (int k = 0; k < 32; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * al);
                tc::tmem_st32(o_addr + i * 32, r);
              }
            }
          }
          // (a column that saw only -inf: an offset of 0 keeps its weights at 0)
          const float nm = m_run == -INFINITY ? 0.f : -m_run;
          const float2 mul2 = make_float2(mul, mul), nm2 = make_float2(nm, nm);
          // Rows past the end in the last block hold stale data, and 0 x NaN
          // would poison O: tile A's warpgroup clears them before its first P V
          const int tail = p.n % kBlockSize;
          if (t == 0 && tail && p.n - kb < kKeys) {
            const int vi = 2 * step + 1;
            if (!wait_all(FULL(vi % NS), (vi / NS) & 1)) { ok = false; break; }
            unsigned char* const vt = sR + (vi % NS) * KT;
            const int r0 = p.n - kb, nr = kBlockSize - tail;
            for (int i = col; i < nr * 8 * KB; i += kWg) {
              const int h = i / (nr * 8), r = r0 + (i / 8) % nr;
              *reinterpret_cast<uint4*>(vt + h * HALF + r * 128 + ((i % 8) << 4)) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float2 x = __ffma2_rn(
                  make_float2(__uint_as_float(sv[h][2 * e]), __uint_as_float(sv[h][2 * e + 1])), mul2, nm2);
              const float2 y = make_float2(ex2(x.x), ex2(x.y));
              l2[e & 3] = __fadd2_rn(l2[e & 3], y);
              const __nv_bfloat162 pp = __float22bfloat162_rn(y);
              w[e] = *reinterpret_cast<const uint32_t*>(&pp);
            }
            tc::tmem_st32(s_addr + 32 * h, w);
            tc::tmem_wait_st();
            tc::fence_before_sync();
            mbar_arrive(TB(t, P0 + h));
          }
        }
        if (!ok) break;
        if (ahead) {
          // the next piece's first S runs while this piece's O goes out
          hand_q();
          q_handed = true;
        }
        const float2 la = __fadd2_rn(__fadd2_rn(l2[0], l2[1]), __fadd2_rn(l2[2], l2[3]));
        const float l_run = la.x + la.y;
        if (!wait_all(TB(t, ODONE), (on++) & 1)) { ok = false; break; }
        tc::fence_after_sync();
        const bool whole = p.slot < 0;
        const float inv = 1.f / l_run;
        const size_t at = whole ? 0 : static_cast<size_t>(p.slot) * (kTiles * kCols) + t * kCols + col;
        // (every lane runs the warp-wide TMEM loads; only live columns store)
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          uint32_t o[64];
          tc::tmem_ld64(o_addr + 64 * h, o);
          tc::tmem_wait_ld(o);
          if (c < 0) continue;
          if (whole) {
            uint4* const dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + c * D + 64 * h);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const __nv_bfloat162 pp = __floats2bfloat162_rn(__uint_as_float(o[16 * i + 2 * e]) * inv,
                                                                __uint_as_float(o[16 * i + 2 * e + 1]) * inv);
                w[e] = *reinterpret_cast<const uint32_t*>(&pp);
              }
              st_wide(dst + 2 * i, w, wide_out);
            }
          } else {
            float4* const dst = reinterpret_cast<float4*>(a.part_o + at * D + 64 * h);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = o[8 * i + e];
              st_wide(dst + 2 * i, w, wide_part);
            }
          }
        }
        if (!whole && c >= 0) a.part_ml[at] = make_float2(m_run, l_run);
        tc::fence_before_sync();  // (O has been read before this warpgroup's next P lets it be written)
      }
      p = nxt;
      have = have_next;
    }
    if (!ok) timeout();
    asm volatile("cp.async.wait_all;" ::: "memory");  // (a Q left in flight by an abort)
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
  k.workers_per_cta = 1;
  k.smem = Shape<D>::SMEM;
  k.cols = kTiles * kCols;
  k.keys = kKeys;
  k.min_tiles = 1;
  return k;
}

}  // namespace

CrossKernel cross_tc_kernel_info(int head_dim) { return head_dim == 64 ? info<64>() : info<128>(); }

}  // namespace pa
