// Linear attention with a decay per head, token by token in fp32: the exact
// path, used for fp32 tensors.
//
// One warp owns one (run, segment, head) and eight columns of the state; the
// da x 8 fp32 slice lives in registers (lane l holds rows l, l + 32, ...).  Per
// token S <- lambda S + b c^T and y = S^T a, the eight column sums reduced over
// the lanes by halving exchanges (9 shuffles instead of 40).  Token t + 1's
// loads are in flight while token t is computed.
#include "linear.cuh"
#include "tc_util.cuh"

namespace gdr {
namespace {

constexpr int kWarps = 4;

template <int DA, typename IO, bool PHASE1>
__global__ void __launch_bounds__(kWarps * 32) linear_token_kernel(const LinProblem p, int ir) {
  constexpr int R = DA / 32;
  tc::griddep_wait();   // in every thread: this grid may not end before the one it depends on
  const LinRun &r = p.run[ir];
  const int lane = threadIdx.x & 31;
  const int groups = r.dc / 8;
  const long gw = static_cast<long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (gw >= static_cast<long>(p.items) * p.H * groups) return;
  const int cg = static_cast<int>(gw % groups);
  const long xh = gw / groups;
  const int h = static_cast<int>(xh % p.H), x = static_cast<int>(xh / p.H);
  const LinItem it = lin_item(p, x);
  if (!it.ok) return;
  const bool last = r.reverse ? it.g == 0 : it.g == it.nseg - 1;    // in the run's order
  if (PHASE1 && last && (it.nseg == 1 || !r.s_final)) return;
  const int c0 = cg * 8, dc = r.dc;
  const float ld = __ldg(p.log_decay + h);
  // lambda as a sum of two fp32 values: its own rounding, compounded over a memory of
  // thousands of tokens, would be the largest error of the state (6e-4 at log_decay = -1e-4)
  const double lam64 = exp(static_cast<double>(ld));
  const float lam = static_cast<float>(lam64), lam_lo = static_cast<float>(lam64 - lam);
  const int page = lin_page(p, it.n);

  float S[R][8];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int c = 0; c < 8; ++c) S[i][c] = 0.f;
  if (!PHASE1) {
    if (it.nseg > 1) {   // the chain kernel wrote every segment's start, the first one's too
      const float *src = r.X + (static_cast<size_t>(x) * p.H + h) * DA * dc;
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) S[i][c] = src[static_cast<size_t>(lane + 32 * i) * dc + c0 + c];
    } else if (r.s0 && page >= 0) {
      const float *src = r.s0 + (static_cast<size_t>(page) * p.H + h) * DA * dc;
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const size_t row = lane + 32 * i, col = c0 + c;
          S[i][c] = src[r.s0_t ? col * DA + row : row * dc + col];
        }
    }
  }

  const LinTensor &ta = p.t[r.ia], &tb = p.t[r.ib], &tcn = p.t[r.ic];
  const long long row0 = it.t0;
  const IO *pa = static_cast<const IO *>(ta.p) + it.b * ta.sb + row0 * ta.st + (h / ta.div) * ta.sh + lane;
  const IO *pb = static_cast<const IO *>(tb.p) + it.b * tb.sb + row0 * tb.st + (h / tb.div) * tb.sh + lane;
  const IO *pc = static_cast<const IO *>(tcn.p) + it.b * tcn.sb + row0 * tcn.st + (h / tcn.div) * tcn.sh + c0;
  const size_t yrow = static_cast<size_t>(it.b) * p.T + it.t0;

  struct Tok {
    float a[R], b[R], c[8];
  };
  auto load = [&](int t, Tok &d) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (!PHASE1) d.a[i] = ld_io<IO>(pa + t * ta.st + 32 * i);
      d.b[i] = r.bscale * ld_io<IO>(pb + t * tb.st + 32 * i);
    }
    ld8<IO>(pc + t * tcn.st, d.c);
  };
  const int beg = it.g * p.seg, end = min(it.len, beg + p.seg);
  const int count = end - beg;
  Tok cur, nxt;
  if (count > 0) load(r.reverse ? end - 1 : beg, cur);
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    const int t = r.reverse ? end - 1 - i : beg + i;
    if (i + 1 < count) load(r.reverse ? t - 1 : t + 1, nxt);
    float y[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) y[c] = 0.f;
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (r.reverse) S[k][c] = fmaf(cur.b[k], cur.c[c], S[k][c]);
        else S[k][c] = fmaf(lam, S[k][c], fmaf(lam_lo, S[k][c], cur.b[k] * cur.c[c]));
        if (!PHASE1) y[c] = fmaf(S[k][c], cur.a[k], y[c]);
        if (r.reverse) S[k][c] = fmaf(lam, S[k][c], lam_lo * S[k][c]);
      }
    if (!PHASE1) {
      // lanes with bit 4, 3, 2 clear keep the lower half of the columns each time
      float z4[4], z2[2], z;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float give = lane & 16 ? y[c] : y[c + 4];
        z4[c] = (lane & 16 ? y[c + 4] : y[c]) + __shfl_xor_sync(0xffffffffu, give, 16);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float give = lane & 8 ? z4[c] : z4[c + 2];
        z2[c] = (lane & 8 ? z4[c + 2] : z4[c]) + __shfl_xor_sync(0xffffffffu, give, 8);
      }
      {
        const float give = lane & 4 ? z2[0] : z2[1];
        z = (lane & 4 ? z2[1] : z2[0]) + __shfl_xor_sync(0xffffffffu, give, 4);
      }
      z += __shfl_xor_sync(0xffffffffu, z, 2);
      z += __shfl_xor_sync(0xffffffffu, z, 1);
      if ((lane & 3) == 0) {
        const int col = c0 + ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
        const size_t at = ((yrow + t) * p.H + h) * dc + col;
        if (r.y_f32) static_cast<float *>(r.y)[at] = r.yscale * z;
        else st_io<IO>(static_cast<IO *>(r.y) + at, r.yscale * z);
      }
    }
    cur = nxt;
  }

  float *dst = nullptr;
  if (PHASE1) dst = r.X + (static_cast<size_t>(x) * p.H + h) * DA * dc;
  else if (it.nseg == 1 && r.s_final && page >= 0) dst = r.s_final + (static_cast<size_t>(page) * p.H + h) * DA * dc;
  if (dst) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float4 *d4 = reinterpret_cast<float4 *>(dst + static_cast<size_t>(lane + 32 * i) * dc + c0);
      d4[0] = make_float4(S[i][0], S[i][1], S[i][2], S[i][3]);
      d4[1] = make_float4(S[i][4], S[i][5], S[i][6], S[i][7]);
    }
  }
}

template <typename IO, bool PHASE1>
cudaError_t launch_run(const LinProblem &p, int ir, bool pdl, cudaStream_t s) {
  const LinRun &r = p.run[ir];
  const long warps = static_cast<long>(p.items) * p.H * (r.dc / 8);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((warps + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return r.da == 128 ? cudaLaunchKernelEx(&cfg, linear_token_kernel<128, IO, PHASE1>, p, ir)
                     : cudaLaunchKernelEx(&cfg, linear_token_kernel<64, IO, PHASE1>, p, ir);
}

}  // namespace
}  // namespace gdr

cudaError_t gdr_launch_linear_token(const gdr::LinProblem &p, bool phase1, bool pdl, cudaStream_t s) {
  using namespace gdr;
  for (int i = 0; i < p.nrun; ++i) {
    cudaError_t e;
    // only the first launch may be a programmatic dependent: the runs of one phase do not wait for
    // one another, but each has to come after everything before the phase
    const bool dep = pdl && i == 0;
    if (p.bf16_io) e = phase1 ? launch_run<__nv_bfloat16, true>(p, i, dep, s) : launch_run<__nv_bfloat16, false>(p, i, dep, s);
    else e = phase1 ? launch_run<float, true>(p, i, dep, s) : launch_run<float, false>(p, i, dep, s);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}
