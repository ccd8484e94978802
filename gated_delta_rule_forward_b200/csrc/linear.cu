// Linear attention with a decay per head: the plan of a call, the chain of its
// segments' start states, the sum over shared heads' gradients, and the order
// of the launches.  The runs themselves are in linear_chunk.cu (bf16) and
// linear_token.cu (fp32).
#include "linear.cuh"
#include "linear_chunk.cuh"
#include "tc_util.cuh"

namespace gdr {
namespace {

// ---------------------------------------------------------------------------
// Start states from the segments' end states, in place: per element and
// sequence X_g <- S_g, S_{g+1} = lambda^{len_g} S_g + X_g, and the state after the
// last segment where it is wanted.  The loads of several segments are issued
// together; only the fused multiply-adds depend on one another.
constexpr int kChainThreads = 256;

__global__ void __launch_bounds__(kChainThreads) linear_chain_kernel(const LinProblem p) {
  tc::griddep_launch_dependents();
  const LinRun &r = p.run[blockIdx.z];
  const int e4 = blockIdx.x * kChainThreads + threadIdx.x;   // float4 of the state
  tc::griddep_wait();
  const size_t page_vec = static_cast<size_t>(r.da) * r.dc / 4;
  if (e4 >= static_cast<int>(page_vec)) return;
  for (int u = blockIdx.y; u < p.N * p.H; u += gridDim.y) {
    const int n = u / p.H, h = u - n * p.H;
    int len = p.T, x = n * p.G, nseg = p.G;
    if (p.cu) {
      const int t0 = lin_cu(p, n);
      len = max(lin_cu(p, n + 1) - t0, 0);
      x = t0 / p.seg + n;
      nseg = max(1, (len + p.seg - 1) / p.seg);
    }
    if (nseg == 1) continue;
    const int tail = len - (nseg - 1) * p.seg;   // tokens of the last segment
    const float ld = __ldg(p.log_decay + h);
    const float2 full = lin_pow64_parts(ld, p.seg), ftail = tail == p.seg ? full : lin_pow64_parts(ld, tail);
    const int page = lin_page(p, n);
    float4 cur = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r.s0 && page >= 0) {
      const float *src = r.s0 + (static_cast<size_t>(page) * p.H + h) * page_vec * 4;
      if (r.s0_t) {
        const int row = e4 * 4 / r.dc, col = e4 * 4 % r.dc;
        cur = make_float4(src[(col + 0) * r.da + row], src[(col + 1) * r.da + row], src[(col + 2) * r.da + row],
                          src[(col + 3) * r.da + row]);
      } else {
        cur = *reinterpret_cast<const float4 *>(src + 4 * e4);
      }
    }
    float4 *X = reinterpret_cast<float4 *>(r.X) + (static_cast<size_t>(x) * p.H + h) * page_vec + e4;
    const size_t xs = p.H * page_vec;
    float4 *fin = r.s_final && page >= 0
                      ? reinterpret_cast<float4 *>(r.s_final) + (static_cast<size_t>(page) * p.H + h) * page_vec + e4 : nullptr;
    constexpr int U = 8;
    for (int i0 = 0; i0 < nseg; i0 += U) {
      float4 d[U];
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (i0 + k < nseg - (fin ? 0 : 1)) d[k] = X[(r.reverse ? nseg - 1 - (i0 + k) : i0 + k) * xs];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i = i0 + k;
        if (i >= nseg) break;
        X[(r.reverse ? nseg - 1 - i : i) * xs] = cur;
        if (i == nseg - 1 && !fin) break;
        const float2 f = i == (r.reverse ? 0 : nseg - 1) ? ftail : full;   // the sequence's last segment may be short
        cur.x = fmaf(f.x, cur.x, fmaf(f.y, cur.x, d[k].x));
        cur.y = fmaf(f.x, cur.y, fmaf(f.y, cur.y, d[k].y));
        cur.z = fmaf(f.x, cur.z, fmaf(f.y, cur.z, d[k].z));
        cur.w = fmaf(f.x, cur.w, fmaf(f.y, cur.w, d[k].w));
      }
    }
    if (fin) *fin = cur;
  }
}

// ---------------------------------------------------------------------------
// Sum over the value heads that share a key head: 4 elements per thread, the
// group's values read in head order (so the order of the sum is fixed).
template <typename IO>
__global__ void __launch_bounds__(256) group_sum_kernel(const float *__restrict__ x, IO *__restrict__ y, long rows,
                                                        int Hk, int G, int d, const int *cu, int N, int zero_rest) {
  const long i = static_cast<long>(blockIdx.x) * 256 + threadIdx.x;   // 4 elements of one (row, key head)
  const int d4 = d / 4;
  const long rh = i / d4;
  const long row = rh / Hk;
  if (row >= rows) return;
  const bool none = cu && (row < __ldg(cu) || row >= __ldg(cu + N));   // a row of no sequence
  if (none && !zero_rest) return;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (!none) {
    const float4 *src = reinterpret_cast<const float4 *>(x) + rh * G * d4 + i % d4;
    s = src[0];
    for (int g = 1; g < G; ++g) {
      const float4 v = src[static_cast<size_t>(g) * d4];
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
  }
  IO *dst = y + i * 4;
  st_io<IO>(dst, s.x);
  st_io<IO>(dst + 1, s.y);
  st_io<IO>(dst + 2, s.z);
  st_io<IO>(dst + 3, s.w);
}

}  // namespace
}  // namespace gdr

cudaError_t gdr_launch_linear_chain(const gdr::LinProblem &p, bool pdl, cudaStream_t s) {
  using namespace gdr;
  const int elems = p.run[0].da * p.run[0].dc;   // the same for every run of a call
  cudaLaunchConfig_t cfg = {};
  const long pairs = static_cast<long>(p.N) * p.H;
  cfg.gridDim = dim3((elems / 4 + kChainThreads - 1) / kChainThreads, static_cast<unsigned>(pairs < 65535 ? pairs : 65535), p.nrun);
  cfg.blockDim = dim3(kChainThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, linear_chain_kernel, p);
}

cudaError_t gdr_launch_linear_group_sum(const float *x, void *y, const gdr::LinProblem &p, int Hk, int d, cudaStream_t s) {
  using namespace gdr;
  const int G = p.H / Hk;
  const long rows = static_cast<long>(p.B) * p.T;
  const long threads = rows * Hk * (d / 4);
  const unsigned grid = static_cast<unsigned>((threads + 255) / 256);
  if (p.bf16_io)
    group_sum_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(x, static_cast<__nv_bfloat16 *>(y), rows, Hk, G, d, p.cu, p.N, p.zero_rest);
  else
    group_sum_kernel<float><<<grid, 256, 0, s>>>(x, static_cast<float *>(y), rows, Hk, G, d, p.cu, p.N, p.zero_rest);
  return cudaGetLastError();
}

// A dense batch: CTAs of one (run, segment, head), each with an SM of its own (or, fp32 at value
// widths of 64, half of one).  Times in us on a B200: a round of CTAs costs `start`, a
// step of 64 (bf16) or 16 (fp32) tokens `step2` with outputs and `step1` in phase 1.
// bf16 has the clock it has under load, and less of a cost where half of the SMs stay idle, whose
// power the others get.
// (bf16: 64 sequences of 32 chunks: whole 66 us, in two segments each 58, in four 74; 192 runs of
// 32 chunks whole 110, in two 139; 16 of 1024 in nine segments 345, in eight 348, in 18 349, in
// four 491.)
namespace {
struct PlanCost {
  float start, step1, step2, step2_half;
};
constexpr PlanCost kChunkCost = {5.f, 1.15f, 2.1f, 1.9f}, kTokenCost = {4.f, 4.3f, 6.1f, 6.1f};
// a phase 2 that chains its states, for each segment before the last, and the kernel
constexpr float kSelfChain = 1.4f, kChainKernel = 3.5f;

int plan_dense(const gdr::LinProblem &p, const PlanCost &cost, int steps, int slots) {   // segments per sequence
  const long units = static_cast<long>(p.N) * p.H * p.nrun;
  float best = 0.f;
  int G = 1;
  for (int g = 1; g == 1 || (g <= steps && units * g <= 2l * slots); ++g) {
    const int len = (steps + g - 1) / g;
    const long rounds = (units * g + slots - 1) / slots;
    float t = rounds * (cost.start + len * (2 * units * g <= slots ? cost.step2_half : cost.step2));
    if (g > 1) t += rounds * (cost.start + len * cost.step1) + (g <= gdr::kLinSelfChain ? kSelfChain * (g - 1) : kChainKernel);
    if (g == 1 || t < best) {
      best = t;
      G = g;
    }
  }
  return G;
}
}  // namespace

void gdr_linear_plan(gdr::LinProblem *p, int sms) {
  const long total = static_cast<long>(p->B) * p->T;
  const int step = p->bf16_io ? 64 : 16;
  long seg;
  if (!p->cu) {
    const int steps = (p->T + step - 1) / step;
    bool narrow = true;
    for (int i = 0; i < p->nrun; ++i) narrow = narrow && p->run[i].dc == 64;
    const int g = plan_dense(*p, p->bf16_io ? kChunkCost : kTokenCost, steps, !p->bf16_io && narrow ? 2 * sms : sms);
    seg = static_cast<long>(step) * ((steps + g - 1) / g);
  } else {
    // lengths unknown here: segments that give every SM one (a packed bf16 batch of 9200 tokens, 16 heads:
    // 1024 tokens 83 us, 512: 95, 2048: 111)
    seg = (total * p->H * p->nrun / sms + step - 1) / step * step;
    if (seg < 4 * step) seg = 4 * step;
  }
  if (seg > p->T) seg = p->T;
  if (seg < 1) seg = 1;
  p->seg = static_cast<int>(seg);
  p->G = p->T > 0 ? (p->T + p->seg - 1) / p->seg : 1;
  p->items = p->cu ? p->T / p->seg + p->N : p->N * p->G;
}

// Segment states of all runs, twice where phase 2 may chain them itself.
static size_t run_floats(const gdr::LinProblem &p, int i) {
  return gdr::lin_segmented(p) ? static_cast<size_t>(gdr::lin_blocks(p)) * p.run[i].da * p.run[i].dc : 0;
}
size_t gdr_linear_workspace_bytes(const gdr::LinProblem &p) {
  size_t floats = 0;
  for (int i = 0; i < p.nrun; ++i) floats += run_floats(p, i) * (gdr::lin_self_chains(p) ? 2 : 1);
  return floats * sizeof(float);
}

cudaError_t gdr_launch_linear(gdr::LinProblem &p, void *ws, cudaStream_t s, std::string *err) {
  float *X = static_cast<float *>(ws);
  for (int i = 0; i < p.nrun; ++i) {
    p.run[i].X = X;
    X += run_floats(p, i);
    if (!gdr::lin_self_chains(p)) continue;
    p.run[i].XS = X;
    X += run_floats(p, i);
  }
  const bool segmented = gdr::lin_segmented(p);
  const bool chunk = p.bf16_io && p.T > 0;   // no tokens: the token kernel copies the states
  gdr::LinChunkMaps maps;
  if (chunk && !gdr_linear_chunk_maps(p, &maps)) return *err = "tensor map: ", cudaErrorInvalidValue;
  auto phase = [&](bool phase1, bool pdl) {
    return chunk ? gdr_launch_linear_chunk(p, maps, phase1, pdl, s) : gdr_launch_linear_token(p, phase1, pdl, s);
  };
  cudaError_t e;
  // (phase 2's segments read the start state side by side: an end state in its place is written by the chain kernel, or
  // in a packed forward they read phase 1's copy of it)
  p.chained = segmented && !gdr::lin_self_chains(p);
  for (int i = 0; i < p.nrun; ++i)
    if (segmented && p.run[i].s0 && p.run[i].s0 == p.run[i].s_final) {
      p.s0_copied = !p.chained && chunk && p.cu && p.nrun == 1;
      p.chained |= !p.s0_copied;
    }
  if (segmented) {
    if ((e = phase(true, false)) != cudaSuccess) return *err = "segment states: ", e;
    if (p.chained && (e = gdr_launch_linear_chain(p, true, s)) != cudaSuccess) return *err = "segment chain: ", e;
  }
  if ((e = phase(false, segmented)) != cudaSuccess) return *err = "runs: ", e;
  return cudaSuccess;
}
