// cross_attention.cu -- pa_cross_attention: the choice of the kernel and its
// launch.  The query rows of each sequence attend to ALL tokens that the
// sequence's block table lists (an encoder's states, a document), whose
// number does not depend on the number of rows:
//   out[r][h] = sum_i exp(x_i - max x) V_i / sum_i exp(x_i - max x),
//   x_i = scale q[r][h] . K_i,   i = 0 .. n - 1.
#include "cross_attention.h"

#include <algorithm>
#include <exception>
#include <map>
#include <mutex>
#include <utility>

namespace pa {
namespace {

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// bf16: up to this many query columns a (sequence, KV head), on average, go to
// the kernel that streams K and V past them.
constexpr int kFewColumns = 32;

std::mutex g_mu;
std::map<std::pair<int, const void*>, bool> g_ready;  // (device, kernel): its shared memory limit is set

}  // namespace

namespace {

// the kernel for `columns` query columns a (sequence, KV head), on average
CrossKernel kernel_of(long long columns, int head_dim, int elem_bytes) {
  if (elem_bytes == 4) return cross_simt_kernel_info(head_dim, columns);
  if (columns <= kFewColumns) return cross_few_kernel_info(head_dim, static_cast<int>(columns));
  return cross_tc_kernel_info(head_dim);
}

}  // namespace

CrossKernel cross_kernel(int num_seqs, int num_rows, int group, int head_dim, int elem_bytes) {
  const long long columns =
      num_seqs > 0 ? (static_cast<long long>(num_rows) * group + num_seqs - 1) / num_seqs : 0;
  return kernel_of(columns, head_dim, elem_bytes);
}

CrossLayout cross_layout(const CrossKernel& k, int head_dim, int num_sms) {
  const size_t slots = 2 * static_cast<size_t>(num_sms) * k.ctas_per_sm;
  CrossLayout l;
  l.ml_off = kCrossCountBytes;
  l.o_off = up256(l.ml_off + slots * k.cols * sizeof(float2));
  l.bytes = up256(l.o_off + slots * k.cols * head_dim * sizeof(float));
  return l;
}

// Fewer sequences put more columns on each, up to all rows on one, and with
// them another kernel and layout: the largest of those that up to `num_rows`
// rows can reach.
size_t cross_workspace_bytes(int num_rows, int group, int head_dim, int elem_bytes, int num_sms) {
  constexpr long long kLastChoice = 65;  // (from here on the kernel is the same)
  const long long most = std::min(static_cast<long long>(num_rows) * group, kLastChoice);
  size_t bytes = 0;
  for (long long columns = 0; columns <= most; ++columns)
    bytes = std::max(bytes, cross_layout(kernel_of(columns, head_dim, elem_bytes), head_dim, num_sms).bytes);
  return bytes;
}

cudaError_t launch_cross_attention(CrossArgs& a, const CrossKernel& k, int num_sms, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  try {
    std::lock_guard<std::mutex> lock(g_mu);
    bool& ready = g_ready[std::make_pair(dev, k.fn)];
    if (!ready) {
      if ((e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(k.smem))) != cudaSuccess)
        return e;
      ready = true;
    }
  } catch (const std::exception&) {  // (the map's memory, the lock: nothing passes a C entry)
    return cudaErrorMemoryAllocation;
  }
  const long long groups = ((static_cast<long long>(a.num_rows) << a.group_log2) / k.cols + a.num_seqs);
  a.max_units = groups * a.num_kv_heads * (k.extra + (a.len_cap > 0 ? (a.len_cap + k.keys - 1) / k.keys : 1));
  void* params[] = {&a};
  return cudaLaunchKernel(k.fn, dim3(num_sms * k.ctas_per_sm), dim3(k.threads), params, k.smem, stream);
}

}  // namespace pa
