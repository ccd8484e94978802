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
  const int h = blockIdx.y % p.H;
  const LinRun &r = p.run[blockIdx.y / p.H];
  const int e4 = blockIdx.x * kChainThreads + threadIdx.x;   // float4 of the state
  tc::griddep_wait();
  const float ld = __ldg(p.log_decay + h);
  const float full = static_cast<float>(exp(static_cast<double>(ld) * p.seg));
  const size_t page_elems = static_cast<size_t>(r.da) * r.dc;
  if (static_cast<size_t>(e4) * 4 >= page_elems) return;
  for (int n = blockIdx.z; n < p.N; n += gridDim.z) {
    int t0 = 0, len = p.T, x0 = n * p.G;
    if (p.cu) {
      t0 = lin_cu(p, n);
      len = max(lin_cu(p, n + 1) - t0, 0);
      x0 = t0 / p.seg + n;
    }
    const int nseg = max(1, (len + p.seg - 1) / p.seg);
    if (nseg == 1) continue;
    const int tail = len - (nseg - 1) * p.seg;   // tokens of the last segment
    const float ftail = tail == p.seg ? full : static_cast<float>(exp(static_cast<double>(ld) * tail));
    const int page = lin_page(p, n);
    float4 cur = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r.s0 && page >= 0) {
      const float *src = r.s0 + (static_cast<size_t>(page) * p.H + h) * page_elems;
      if (r.s0_t) {
        const int row = e4 * 4 / r.dc, col = e4 * 4 % r.dc;
        cur = make_float4(src[(col + 0) * r.da + row], src[(col + 1) * r.da + row], src[(col + 2) * r.da + row],
                          src[(col + 3) * r.da + row]);
      } else {
        cur = *reinterpret_cast<const float4 *>(src + 4 * e4);
      }
    }
    const size_t step = static_cast<size_t>(p.H) * page_elems / 4;
    float4 *X = reinterpret_cast<float4 *>(r.X) + (static_cast<size_t>(x0) * p.H + h) * (page_elems / 4) + e4;
    float4 *fin = r.s_final && page >= 0 ? reinterpret_cast<float4 *>(
        r.s_final + (static_cast<size_t>(page) * p.H + h) * page_elems) + e4 : nullptr;
    constexpr int U = 8;
    for (int i0 = 0; i0 < nseg; i0 += U) {
      float4 d[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u < nseg - (fin ? 0 : 1)) d[u] = X[(r.reverse ? nseg - 1 - (i0 + u) : i0 + u) * step];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u;
        if (i >= nseg) break;
        X[(r.reverse ? nseg - 1 - i : i) * step] = cur;
        if (i == nseg - 1 && !fin) break;
        const float f = i == (r.reverse ? 0 : nseg - 1) ? ftail : full;   // the sequence's last segment may be short
        cur.x = fmaf(f, cur.x, d[u].x);
        cur.y = fmaf(f, cur.y, d[u].y);
        cur.z = fmaf(f, cur.z, d[u].z);
        cur.w = fmaf(f, cur.w, d[u].w);
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
                                                        int Hk, int G, int d, const int *cu, int N) {
  const long i = static_cast<long>(blockIdx.x) * 256 + threadIdx.x;   // 4 elements of one (row, key head)
  const int d4 = d / 4;
  const long rh = i / d4;
  const long row = rh / Hk;
  if (row >= rows) return;
  if (cu && (row < __ldg(cu) || row >= __ldg(cu + N))) return;   // a row of no sequence
  const float4 *src = reinterpret_cast<const float4 *>(x) + rh * G * d4 + i % d4;
  float4 s = src[0];
  for (int g = 1; g < G; ++g) {
    const float4 v = src[static_cast<size_t>(g) * d4];
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
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
  cfg.gridDim = dim3((elems / 4 + kChainThreads - 1) / kChainThreads, p.H * p.nrun, p.N < 65535 ? p.N : 65535);
  cfg.blockDim = dim3(kChainThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, linear_chain_kernel, p);
}

cudaError_t gdr_launch_linear_group_sum(const float *x, void *y, bool bf16, int B, int T, int Hk, int G, int d,
                                        const int *cu, int N, cudaStream_t s) {
  using namespace gdr;
  const long rows = static_cast<long>(B) * T;
  const long threads = rows * Hk * (d / 4);
  const unsigned grid = static_cast<unsigned>((threads + 255) / 256);
  if (bf16) group_sum_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(x, static_cast<__nv_bfloat16 *>(y), rows, Hk, G, d, cu, N);
  else group_sum_kernel<float><<<grid, 256, 0, s>>>(x, static_cast<float *>(y), rows, Hk, G, d, cu, N);
  return cudaGetLastError();
}

void gdr_linear_plan(gdr::LinProblem *p, int sms) {
  const long total = static_cast<long>(p->B) * p->T;
  long seg;
  if (p->bf16_io) {
    // One CTA per SM and (run, segment, head).
    const long slots = sms, heads = static_cast<long>(p->H) * p->nrun;
    if (!p->cu) {
      const long per_seq = slots / (heads * p->N > 0 ? heads * p->N : 1);   // segments per sequence that fit
      seg = per_seq <= 1 ? p->T : (p->T + per_seq - 1) / per_seq;
    } else {
      seg = total * heads / slots;
    }
    if (seg < 128) seg = 128;
  } else {
    // Token kernel: one warp per (run, segment, head, 8 columns), 12 or so resident
    // per SM; segments of at least 64 tokens until the device is full.
    long warps = 0;
    for (int i = 0; i < p->nrun; ++i) warps += static_cast<long>(p->H) * (p->run[i].dc / 8);
    const long slots = 12L * sms;
    seg = (total * warps + slots - 1) / slots;        // tokens per segment that fill the slots
    if (!p->cu && static_cast<long>(p->N) * warps >= slots) seg = p->T;
  }
  seg = (seg + 63) / 64 * 64;
  if (seg < 64) seg = 64;
  const long whole = (p->T + 63) / 64 * 64;
  if (seg > whole) seg = whole > 0 ? whole : 64;
  p->seg = static_cast<int>(seg);
  p->G = p->T > 0 ? (p->T + p->seg - 1) / p->seg : 1;
  p->items = p->cu ? p->T / p->seg + p->N : p->N * p->G;
}

// Segment states of all runs, when any sequence may have more than one segment.
size_t gdr_linear_workspace_bytes(const gdr::LinProblem &p) {
  if (p.T <= p.seg) return 0;
  size_t floats = 0;
  for (int i = 0; i < p.nrun; ++i) floats += static_cast<size_t>(p.items) * p.H * p.run[i].da * p.run[i].dc;
  return floats * sizeof(float);
}

cudaError_t gdr_launch_linear(gdr::LinProblem &p, void *ws, cudaStream_t s, std::string *err) {
  float *X = static_cast<float *>(ws);
  for (int i = 0; i < p.nrun; ++i) {
    p.run[i].X = X;
    X += static_cast<size_t>(p.items) * p.H * p.run[i].da * p.run[i].dc;
  }
  const bool segmented = p.T > p.seg;
  const bool chunk = p.bf16_io && p.T > 0;   // no tokens: the token kernel copies the states
  gdr::LinChunkMaps maps;
  if (chunk && !gdr_linear_chunk_maps(p, &maps)) return *err = "tensor map: ", cudaErrorInvalidValue;
  auto phase = [&](bool phase1, bool pdl) {
    return chunk ? gdr_launch_linear_chunk(p, maps, phase1, pdl, s) : gdr_launch_linear_token(p, phase1, pdl, s);
  };
  cudaError_t e;
  if (segmented) {
    if ((e = phase(true, false)) != cudaSuccess) return *err = "segment states: ", e;
    if ((e = gdr_launch_linear_chain(p, true, s)) != cudaSuccess) return *err = "segment chain: ", e;
  }
  if ((e = phase(false, segmented)) != cudaSuccess) return *err = "runs: ", e;
  return cudaSuccess;
}
