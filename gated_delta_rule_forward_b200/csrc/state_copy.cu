// Page copies of a state pool [layers][pages][page]: copying, forking,
// compacting and clearing recurrent states (bandwidth-bound).
//
// The page pairs arrive as kernel arguments, so a call needs no device index
// array and takes what its host lists hold when it is made; a captured graph
// holds them by value.  One block copies 32 KB of one page of one layer, eight
// float4 loads in flight per thread; the pair is the fastest-varying block
// index, so that a page forked to many is read from DRAM once and from L2 by
// the blocks beside it.  1.2 GB moved: 185 us, 6.54 TB/s; one page of 16 heads to
// eight others: 4.7 us in a graph, 9.3 us a call, which the host's part bounds.
#include "state_copy.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 8;
constexpr int kBlockVec = kThreads * kUnroll;   // float4 per block

template <int MAX>
struct Pairs {
  int n;
  int src[MAX], dst[MAX];
};

template <int MAX>
__global__ void __launch_bounds__(kThreads) state_copy_kernel(float4 *pool, size_t page_vec, int pages, int blocks_per_page,
                                                               const __grid_constant__ Pairs<MAX> pairs) {
  const long x = blockIdx.x;
  const int i = static_cast<int>(x % pairs.n);
  const long y = x / pairs.n;
  const int blk = static_cast<int>(y % blocks_per_page);
  const size_t layer = y / blocks_per_page;
  const int src = pairs.src[i], dst = pairs.dst[i];
  float4 *d = pool + (layer * pages + dst) * page_vec;
  const float4 *s = pool + (layer * pages + max(src, 0)) * page_vec;
  const size_t base = static_cast<size_t>(blk) * kBlockVec + threadIdx.x;
  float4 v[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const size_t at = base + u * kThreads;
    v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (src >= 0 && at < page_vec) v[u] = s[at];
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const size_t at = base + u * kThreads;
    if (at < page_vec) d[at] = v[u];
  }
}

}  // namespace
}  // namespace gdr

cudaError_t gdr_launch_state_copy(float *pool, size_t page_floats, int layers, int pages, const gdr::CopyPairs &pairs,
                                  cudaStream_t s) {
  using namespace gdr;
  const size_t vec = page_floats / 4;
  const long per_page = static_cast<long>((vec + kBlockVec - 1) / kBlockVec);
  const long blocks = per_page * layers * pairs.n;
  auto launch = [&](auto few) {
    few.n = pairs.n;
    for (int i = 0; i < pairs.n; ++i) {
      few.src[i] = pairs.src[i];
      few.dst[i] = pairs.dst[i];
    }
    state_copy_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(reinterpret_cast<float4 *>(pool), vec, pages,
                                                                         static_cast<int>(per_page), few);
  };
  if (pairs.n <= kFewCopyPairs) launch(Pairs<kFewCopyPairs>());
  else launch(Pairs<kMaxCopyPairs>());
  return cudaGetLastError();
}
