// rope_append.cu -- rotary positions applied on the way into the paged cache.
//
// For token t, a q or k head row x and pair i of its rotary_dim / 2 rotated
// pairs (a, b) = (x[i], x[i + rotary_dim / 2]) or (x[2 i], x[2 i + 1]):
//   theta  = positions[axis(i)][t] * inv_freq[i]
//   (a, b) <- rot_scale * (a cos theta - b sin theta, a sin theta + b cos theta)
// Dims from rotary_dim on are copied.  A q row goes to q_out, a k row to its
// cache slot, and the v row is copied to its slot beside it.
//
// Memory-bound: every row is read and written once, about 3 fp32 operations
// an element.  What is not a stream is kept off it:
//   * the angles.  A token's cos and sin are the same for all its heads, so a
//     CTA computes them once into shared memory, rotary_dim / 2 per token.
//     theta is formed and reduced as a fraction of a turn in pairs of doubles (a
//     plain fp64 product is off by theta 2^-53: 1e-4 at 2^40), and goes to fp32 in
//     two parts, so that sine and cosine carry the error of sincospif (1 ulp)
//     and one rounding, at positions of up to 2^53.
//   * the slots: one division per token (and warp that works on it), not per
//     element.
// A thread's unit of work is two 16-byte chunks of one row: the two halves of
// the same 8 (bf16) or 4 (fp32) pairs, or two chunks to copy.
//
// Two kernels.  Where a row's units divide a warp (every power-of-two head_dim
// up to 512 bf16 or 256 fp32 elements, with any rotary_dim that leaves whole
// units), a warp takes a token, or a slice of its rows: a lane keeps the same
// place in every row, its angles in registers, and three or four rows in flight; no
// division a row, no barrier.  Other shapes take a CTA per few tokens, its units laid
// end to end, angles read from shared memory per unit.  Measured on what both
// can do, 16384 tokens of 48 rows of 256 bytes (402 MB): 68.5 us (90 %
// of the copy rate) against 81; one token of as many rows: 2.8 against 2.4 us.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "pa_internal.h"
#include "rope_append.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kUnitsAhead = 2;  // units a thread has in flight
constexpr size_t kMaxSmem = 40 * 1024;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float x, float* y) { *y = x; }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16* y) { *y = __float2bfloat16_rn(x); }

template <typename T>
union Chunk {
  uint4 v;
  T e[16 / sizeof(T)];
};

// 1 / (2 pi), rounded to double, and what that leaves
constexpr double kTurnsPerRadian = 0.15915494309189535, kTurnsPerRadianLow = -9.839338337591243e-18;

// rot_scale (cos, sin) of pair p of token t
__device__ __forceinline__ float2 angle(const RopeArgs& a, int p, long long t) {
  int axis = 0;
  if (a.pair_axis) {
    axis = a.pair_axis[p];
    if (axis < 0 || axis >= a.num_axes) {  // (a pair without an axis is not turned)
      if (a.err_flag) atomicOr(a.err_flag, kErrAxis);
      return make_float2(a.rot_scale, 0.f);
    }
  }
  // the product exactly (hi + lo), times 1 / (2 pi) in two doubles: turns + rest
  const double pos = static_cast<double>(a.positions[axis * a.num_tokens + t]), freq = a.inv_freq[p];
  const double hi = pos * freq, lo = fma(pos, freq, -hi);
  const double turns = hi * kTurnsPerRadian;
  const double rest = fma(hi, kTurnsPerRadianLow, fma(lo, kTurnsPerRadian, fma(hi, kTurnsPerRadian, -turns)));
  double part = (turns - rint(turns)) + rest;
  part = 2. * (part - rint(part));  // half turns, in [-1, 1]
  // to fp32 in two parts: sine and cosine of the first, turned by the second (below 2^-25 half turns)
  const float x = static_cast<float>(part), d = 3.14159265f * static_cast<float>(part - x);
  float s0, c0;
  sincospif(x, &s0, &c0);
  const float s = fmaf(d, c0, s0), c = fmaf(-d, s0, c0);
  return make_float2(c * a.rot_scale, s * a.rot_scale);
}

// One unit of work: two chunks of one row (the second missing where c1 < 0).
struct Unit {
  int tok = -1;   // token within the CTA (-1: no unit)
  int part;       // 0: q, 1: key, 2: value
  int head;
  int c0, c1;     // chunks of the row
  bool rotated;
};

template <typename T, bool ADJACENT>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeArgs a) {
  constexpr int VE = 16 / sizeof(T);
  extern __shared__ float smem[];
  const int tpc = a.tokens_per_cta, half = a.rotary_dim / 2;
  float* const s_cos = smem;               // [tpc][half]
  float* const s_sin = s_cos + tpc * half;
  long long* const s_row = reinterpret_cast<long long*>(s_sin + tpc * half);  // [tpc]
  const int tid = threadIdx.x;
  const long long t0 = static_cast<long long>(blockIdx.x) * tpc;
  const int nt = static_cast<int>(a.num_tokens - t0 < tpc ? a.num_tokens - t0 : tpc);

  // units of a row: rotated ones, then the copied rest two chunks at a time
  const int chunks = a.head_dim / VE;
  const int ur = a.rotary_dim / (2 * VE);
  const int rest = chunks - 2 * ur, uc = (rest + 1) / 2;
  const int uv = (chunks + 1) / 2;
  const int uq = ur + uc;
  const int nq = a.q ? a.num_q_heads * uq : 0;
  const int nk = a.key ? a.num_kv_heads * uq : 0;
  const int nv = a.key ? a.num_kv_heads * uv : 0;
  const int per_token = nq + nk + nv;
  const int begin = blockIdx.y * a.units_per_slice;
  const int end = min(nt * per_token, begin + a.units_per_slice);

  // the slots first: the copies' addresses need them
  if (tid < nt) {
    long long row = -1;
    if (a.key) {
      const long long slot = a.slot_mapping[t0 + tid];
      if (slot >= a.num_slots) {
        if (blockIdx.y == 0 && a.err_flag) atomicOr(a.err_flag, kErrSlot);
      } else if (slot >= 0) {
        const long long blk = slot / a.block_size;
        row = blk * a.num_kv_heads * a.block_size + (slot - blk * a.block_size);
      }
    }
    s_row[tid] = row;
  }

  auto locate = [&](int i) -> Unit {
    Unit u;
    if (i >= end) return u;
    u.tok = i / per_token;
    int r = i - u.tok * per_token;
    u.part = r < nq ? 0 : r < nq + nk ? 1 : 2;
    r -= u.part == 0 ? 0 : u.part == 1 ? nq : nq + nk;
    const int width = u.part == 2 ? uv : uq;
    u.head = r / width;
    const int w = r - u.head * width;
    u.rotated = u.part != 2 && w < ur;
    if (u.rotated) {
      u.c0 = w;
      u.c1 = w + ur;
    } else {  // the n chunks from `first` on, the two halves of them side by side
      const int first = u.part == 2 ? 0 : 2 * ur, n = chunks - first, k = u.part == 2 ? w : w - ur;
      u.c0 = first + k;
      u.c1 = k + (n + 1) / 2 < n ? u.c0 + (n + 1) / 2 : -1;
    }
    return u;
  };
  auto source = [&](const Unit& u) -> const uint4* {
    const void* p = u.part == 0 ? a.q : u.part == 1 ? a.key : a.value;
    const long long stride = u.part == 0 ? a.q_stride : u.part == 1 ? a.key_stride : a.value_stride;
    return reinterpret_cast<const uint4*>(static_cast<const T*>(p) + (t0 + u.tok) * stride +
                                          static_cast<long long>(u.head) * a.head_dim);
  };
  // (after the barrier: the slots are in shared memory; null: a padding token)
  auto destination = [&](const Unit& u) -> uint4* {
    if (u.part == 0)
      return reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + (t0 + u.tok) * a.q_out_stride +
                                      static_cast<long long>(u.head) * a.head_dim);
    const long long row = s_row[u.tok];
    if (row < 0) return nullptr;
    T* const cache = static_cast<T*>(u.part == 1 ? a.k_cache : a.v_cache);
    return reinterpret_cast<uint4*>(cache + (row + static_cast<long long>(u.head) * a.block_size) *
                                                a.head_dim);
  };

  Unit u[kUnitsAhead];
  Chunk<T> x0[kUnitsAhead], x1[kUnitsAhead];
  auto load = [&](int i) {
#pragma unroll
    for (int k = 0; k < kUnitsAhead; ++k) {
      u[k] = locate(i + k * kThreads);
      if (u[k].tok >= 0) {
        const uint4* const src = source(u[k]);
        x0[k].v = src[u[k].c0];
        if (u[k].c1 >= 0) x1[k].v = src[u[k].c1];
      }
    }
  };
  load(begin + tid);

  // the angles of this CTA's tokens
  for (int i = tid; i < nt * half; i += kThreads) {
    const int tok = i / half, p = i - tok * half;
    const float2 cs = angle(a, p, t0 + tok);
    s_cos[i] = cs.x;
    s_sin[i] = cs.y;
  }
  __syncthreads();

  for (int i = begin + tid; i < end; i += kUnitsAhead * kThreads) {
    if (i != begin + tid) load(i);
#pragma unroll
    for (int k = 0; k < kUnitsAhead; ++k) {
      if (u[k].tok < 0) continue;
      if (u[k].rotated) {
        const int p0 = u[k].tok * half;
        if constexpr (ADJACENT) {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            Chunk<T>& x = n ? x1[k] : x0[k];
            const int p = p0 + (n ? u[k].c1 : u[k].c0) * (VE / 2);
#pragma unroll
            for (int j = 0; j < VE / 2; ++j) {
              const float c = s_cos[p + j], s = s_sin[p + j];
              const float xa = to_f32(x.e[2 * j]), xb = to_f32(x.e[2 * j + 1]);
              from_f32(fmaf(xa, c, -(xb * s)), &x.e[2 * j]);
              from_f32(fmaf(xa, s, xb * c), &x.e[2 * j + 1]);
            }
          }
        } else {
          const int p = p0 + u[k].c0 * VE;
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            const float c = s_cos[p + j], s = s_sin[p + j];
            const float xa = to_f32(x0[k].e[j]), xb = to_f32(x1[k].e[j]);
            from_f32(fmaf(xa, c, -(xb * s)), &x0[k].e[j]);
            from_f32(fmaf(xa, s, xb * c), &x1[k].e[j]);
          }
        }
      }
      uint4* const dst = destination(u[k]);
      if (dst) {
        dst[u[k].c0] = x0[k].v;
        if (u[k].c1 >= 0) dst[u[k].c1] = x1[k].v;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// A warp per (token, slice of its rows); UPR = units of a row, a divisor of 32.
// ---------------------------------------------------------------------------
constexpr int kWarps = 2;      // per CTA
constexpr int kMaxHalf = 256;  // rotated pairs, at most
constexpr long long kL2Bytes = 126LL << 20;
constexpr int kWarpsWanted = 12;  // warps an SM, before a token's rows are cut
constexpr int kTokensAtOnce = 16;  // tokens an SM up to which no warp waits for another's place

// AHEAD: the rows that a lane has in flight.
template <typename T, bool ADJACENT, bool STREAM, int AHEAD>
__global__ void __launch_bounds__(kWarps * 32) rope_append_warp_kernel(const RopeArgs a, int upr, int slices) {
  constexpr int VE = 16 / sizeof(T);
  extern __shared__ float smem[];
  const int lane = threadIdx.x & 31, half = a.rotary_dim / 2;
  float* const s_cos = smem + (threadIdx.x >> 5) * 2 * half;
  float* const s_sin = s_cos + half;
  const long long g = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const long long t = g / slices;
  const int slice = static_cast<int>(g - t * slices);
  if (t >= a.num_tokens) return;

  // this lane's chunks of every row it takes
  const int w = lane % upr, ur = a.rotary_dim / (2 * VE), chunks = a.head_dim / VE;
  const int rows_per_it = 32 / upr, sub = lane / upr;
  const int Hq = a.q ? a.num_q_heads : 0, Hkv = a.key ? a.num_kv_heads : 0;
  const int rows = Hq + 2 * Hkv;
  const int its = (rows + rows_per_it - 1) / rows_per_it;
  const int it0 = slice * its / slices, it1 = (slice + 1) * its / slices;

  long long cache_row = -1;  // the token's row in the caches of KV head 0
  if (a.key) {
    const long long slot = a.slot_mapping[t];
    if (slot >= a.num_slots) {
      if (slice == 0 && lane == 0 && a.err_flag) atomicOr(a.err_flag, kErrSlot);
    } else if (slot >= 0) {
      const long long blk = slot / a.block_size;
      cache_row = blk * Hkv * a.block_size + (slot - blk * a.block_size);
    }
  }
  // A row: 0 .. Hq - 1 the q heads, then the key heads, then the value heads.
  // Rotated units take chunks w and w + ur; the rest of a row (a value row:
  // all of it) is copied, two chunks half of it apart.
  struct Row {
    const uint4* src;
    uint4* dst;
    int c0, c1;
    bool turn;
  };
  auto locate = [&](int it) -> Row {
    Row r{nullptr, nullptr, 0, 0, false};
    const int row = it * rows_per_it + sub;
    if (it >= it1 || row >= rows) return r;
    const T* src;
    T* dst;
    const bool val = row >= Hq + Hkv;
    if (row < Hq) {
      src = static_cast<const T*>(a.q) + t * a.q_stride + row * a.head_dim;
      dst = static_cast<T*>(a.q_out) + t * a.q_out_stride + row * a.head_dim;
    } else {
      if (cache_row < 0) return r;
      const int h = row - Hq - (val ? Hkv : 0);
      src = (val ? static_cast<const T*>(a.value) + t * a.value_stride : static_cast<const T*>(a.key) + t * a.key_stride) +
            h * a.head_dim;
      dst = static_cast<T*>(val ? a.v_cache : a.k_cache) +
            (cache_row + static_cast<long long>(h) * a.block_size) * a.head_dim;
    }
    r.turn = !val && w < ur;
    const int first = val ? 0 : 2 * ur, k = val ? w : w - ur;
    r.c0 = r.turn ? w : first + k;
    r.c1 = r.turn ? w + ur : first + k + (chunks - first) / 2;
    r.src = reinterpret_cast<const uint4*>(src);
    r.dst = reinterpret_cast<uint4*>(dst);
    return r;
  };
  Row row[AHEAD];
  Chunk<T> x0[AHEAD], x1[AHEAD];
  auto load = [&](int it) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      row[k] = locate(it + k);
      if (row[k].src) {
        x0[k].v = STREAM ? __ldcs(row[k].src + row[k].c0) : row[k].src[row[k].c0];
        x1[k].v = STREAM ? __ldcs(row[k].src + row[k].c1) : row[k].src[row[k].c1];
      }
    }
  };
  load(it0);

  // the token's angles: half / 32 pairs a lane, then each lane reads its own
  for (int p = lane; p < half; p += 32) {
    const float2 cs = angle(a, p, t);
    s_cos[p] = cs.x;
    s_sin[p] = cs.y;
  }
  __syncwarp();
  float c[VE], s[VE];
  if (w < ur) {
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      // (adjacent pairs: the first half of them in chunk w, the second in w + ur)
      const int p = ADJACENT ? (w + (j < VE / 2 ? 0 : ur)) * (VE / 2) + j % (VE / 2) : w * VE + j;
      c[j] = s_cos[p];
      s[j] = s_sin[p];
    }
  }
  for (int it = it0; it < it1; it += AHEAD) {
    if (it != it0) load(it);
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      if (!row[k].src) continue;
      if (row[k].turn) {
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          if constexpr (ADJACENT) {
            T* const e = (j < VE / 2 ? x0[k].e : x1[k].e) + 2 * (j % (VE / 2));
            const float xa = to_f32(e[0]), xb = to_f32(e[1]);
            from_f32(fmaf(xa, c[j], -(xb * s[j])), e);
            from_f32(fmaf(xa, s[j], xb * c[j]), e + 1);
          } else {
            const float xa = to_f32(x0[k].e[j]), xb = to_f32(x1[k].e[j]);
            from_f32(fmaf(xa, c[j], -(xb * s[j])), &x0[k].e[j]);
            from_f32(fmaf(xa, s[j], xb * c[j]), &x1[k].e[j]);
          }
        }
      }
      if (STREAM) {
        __stcs(row[k].dst + row[k].c0, x0[k].v);
        __stcs(row[k].dst + row[k].c1, x1[k].v);
      } else {
        row[k].dst[row[k].c0] = x0[k].v;
        row[k].dst[row[k].c1] = x1[k].v;
      }
    }
  }
}

}  // namespace

// Launch shape.  The warp kernel: a token's rows are cut into slices where the
// tokens alone would leave the SMs without warps (each slice computes the
// token's angles again: that costs no bandwidth, only a few hundred cycles that
// the rows' own loads cover).  The CTA kernel: as many tokens as give each
// thread about four units; where that leaves fewer CTAs than fill the GPU twice,
// slices of one unit per thread of one token.
cudaError_t launch_rope_append(RopeArgs a, int elem_bytes, bool adjacent, int num_sms,
                               cudaStream_t stream) {
  const int ve = 16 / elem_bytes;
  const int chunks = a.head_dim / ve, ur = a.rotary_dim / (2 * ve);
  const int uq = ur + (chunks - 2 * ur + 1) / 2, uv = (chunks + 1) / 2;
  auto divides = [](int x) { return x > 0 && 32 % x == 0; };
  if (chunks % 2 == 0 && divides(chunks / 2) && a.rotary_dim / 2 <= kMaxHalf) {
    const int upr = chunks / 2, rows_per_it = 32 / upr;  // (what is copied of a row: whole units too)
    const int rows = (a.q ? a.num_q_heads : 0) + (a.key ? 2 * a.num_kv_heads : 0);
    const int its = (rows + rows_per_it - 1) / rows_per_it;
    const long long want = static_cast<long long>(num_sms) * kWarpsWanted;
    const long long slices = std::min<long long>(its, std::max<long long>(1, want / a.num_tokens));
    const long long ctas = (a.num_tokens * slices + kWarps - 1) / kWarps;
    if (ctas < (1LL << 31)) {
      const size_t smem = kWarps * a.rotary_dim * sizeof(float);
      auto go = [&](auto kernel) {
        kernel<<<static_cast<unsigned>(ctas), kWarps * 32, smem, stream>>>(a, upr, static_cast<int>(slices));
      };
      // Tokens that all have a place at once gain from a fourth row in flight (2048
      // tokens of 80 rows: 16.9 us, 18.1 with three; 1024 of 48: 6.1, 6.4), more lose
      // by the registers it takes (8192 of 20: 17.9, 15.3 with three).
      const bool few = a.num_tokens <= static_cast<long long>(num_sms) * kTokensAtOnce;
      auto pick = [&](auto elem, auto stream_tag) {
        using T = decltype(elem);
        constexpr bool S = decltype(stream_tag)::value;
        if constexpr (!S) {
          if (few) {
            adjacent ? go(rope_append_warp_kernel<T, true, S, 4>) : go(rope_append_warp_kernel<T, false, S, 4>);
            return;
          }
        }
        adjacent ? go(rope_append_warp_kernel<T, true, S, 3>) : go(rope_append_warp_kernel<T, false, S, 3>);
      };
      // More than the L2 holds (126 MB): read and written under the streaming
      // policy (402 MB: 67 us, 70 without); less may be read again from it (84 MB
      // held by the L2: 12.8 us, 14.4 streamed).
      const bool big = 2LL * a.num_tokens * rows * a.head_dim * elem_bytes > kL2Bytes;
      if (elem_bytes == 2)
        big ? pick(__nv_bfloat16(), std::true_type{}) : pick(__nv_bfloat16(), std::false_type{});
      else
        big ? pick(float(), std::true_type{}) : pick(float(), std::false_type{});
      return cudaGetLastError();
    }
  }
  const long long per_token = (a.q ? static_cast<long long>(a.num_q_heads) * uq : 0) +
                              (a.key ? static_cast<long long>(a.num_kv_heads) * (uq + uv) : 0);
  const size_t token_smem = a.rotary_dim * sizeof(float) + sizeof(long long);
  long long tpc = std::min<long long>({4 * kThreads / per_token, kThreads,
                                       static_cast<long long>(kMaxSmem / token_smem)});
  if (tpc < 1) tpc = 1;
  long long slice = per_token * tpc;
  if ((a.num_tokens + tpc - 1) / tpc < 2LL * num_sms) {
    tpc = 1;
    slice = std::max<long long>(kThreads, (per_token + 65534) / 65535);
  }
  const long long slices = (per_token * tpc + slice - 1) / slice;
  a.tokens_per_cta = static_cast<int>(tpc);
  a.units_per_slice = static_cast<int>(slice);
  const size_t smem = static_cast<size_t>(tpc) * token_smem;
  const dim3 grid(static_cast<unsigned>((a.num_tokens + tpc - 1) / tpc), static_cast<unsigned>(slices));
  auto go = [&](auto kernel) { kernel<<<grid, kThreads, smem, stream>>>(a); };
  if (elem_bytes == 2)
    adjacent ? go(rope_append_kernel<__nv_bfloat16, true>) : go(rope_append_kernel<__nv_bfloat16, false>);
  else
    adjacent ? go(rope_append_kernel<float, true>) : go(rope_append_kernel<float, false>);
  return cudaGetLastError();
}

}  // namespace pa
