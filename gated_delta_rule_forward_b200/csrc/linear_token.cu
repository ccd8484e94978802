// Linear attention with a decay per head, token by token in fp32: the exact
// path, used for fp32 tensors (and for the state copies of a call without
// tokens).
//
// One CTA owns one (run, segment, head), one warp of it eight columns of the
// state; the da x 8 fp32 slice lives in registers (lane l holds rows l, l + 32,
// ...; columns in pairs).  Tokens come through shared memory eight at a time,
// the next eight on their way while these are computed.  Per token
// S <- lambda S + b c^T and y = S^T a, the eight column sums reduced over the lanes
// by halving exchanges (9 shuffles instead of 40).  Bound by issue: about 80
// instructions a token and warp.
#include "linear.cuh"
#include "tc_util.cuh"

namespace gdr {
namespace {

using tc::fma_f32x2;
using tc::mul_f32x2;
using tc::pair_f32;
using tc::unpair_f32;

constexpr int TT = 8;   // tokens a tile

__device__ __forceinline__ void copy16(uint32_t dst, const float *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <int DA, int DC, bool PHASE1>
__global__ void __launch_bounds__(DC * 4) linear_token_kernel(const __grid_constant__ LinProblem p, int ir,
                                                              bool beside) {
  constexpr int R = DA / 32, NT = DC * 4;
  __shared__ __align__(16) float ta[2][PHASE1 ? 1 : TT][DA], tb[2][TT][DA], tcol[2][TT][DC];
  // In every thread, at the start or (a run beside the phase's first) at the end: a grid may not
  // end before the one it depends on.
  if (!beside) tc::griddep_wait();
  tc::griddep_launch_dependents();
  const LinRun &r = p.run[ir];
  const int tid = threadIdx.x, lane = tid & 31, c0 = 8 * (tid >> 5);
  const LinItem it = lin_item(p, blockIdx.x);
  const int h = it.h;
  const bool rev = r.reverse != 0;
  const bool last = rev ? it.g == 0 : it.g == it.nseg - 1;    // in the run's order
  if (!it.ok || (PHASE1 && last && (it.nseg == 1 || !r.s_final))) {
    if (beside) tc::griddep_wait();
    return;
  }
  const float ld = __ldg(p.log_decay + h);
  const int page = lin_page(p, it.n);

  uint64_t S[R][4];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) S[i][c] = 0;
  if (!PHASE1) {
    const float *start = r.X + static_cast<size_t>(it.slot) * DA * DC;
    if (it.nseg > 1 && !p.chained) {
      float *mine = r.XS + static_cast<size_t>(it.slot) * DA * DC;
      lin_self_chain(p, r, it, page, last, DA, DC, mine, tid, NT);
      start = mine;
      __syncthreads();
    }
    const bool whole = it.nseg == 1, t = whole && r.s0_t;
    if (whole) start = r.s0 && page >= 0 ? r.s0 + (static_cast<size_t>(page) * p.H + h) * DA * DC : nullptr;
    if (start)
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int row = lane + 32 * i, col = c0 + 2 * c;
          S[i][c] = t ? pair_f32(start[col * DA + row], start[(col + 1) * DA + row])
                      : *reinterpret_cast<const uint64_t *>(start + row * DC + col);
        }
  }

  const LinTensor &la = p.t[r.ia], &lb = p.t[r.ib], &lc = p.t[r.ic];
  const float *pa = static_cast<const float *>(la.p) + it.b * la.sb + it.t0 * la.st + (h / la.div) * la.sh;
  const float *pb = static_cast<const float *>(lb.p) + it.b * lb.sb + it.t0 * lb.st + (h / lb.div) * lb.sh;
  const float *pc = static_cast<const float *>(lc.p) + it.b * lc.sb + it.t0 * lc.st + (h / lc.div) * lc.sh;
  const int count = it.end - it.beg;
  auto token = [&](int i) { return rev ? it.end - 1 - i : it.beg + i; };   // in the run's order
  auto fetch = [&](int i0, int buf) {   // tokens i0 .. i0 + TT - 1, those of the segment
    const int n = min(TT, count - i0);
    for (int k = tid; k < n * (DA / 4); k += NT) {
      const int t = k / (DA / 4), d = 4 * (k % (DA / 4));
      copy16(tc::smem_u32(&tb[buf][t][d]), pb + token(i0 + t) * lb.st + d);
      if (!PHASE1) copy16(tc::smem_u32(&ta[buf][t][d]), pa + token(i0 + t) * la.st + d);
    }
    for (int k = tid; k < n * (DC / 4); k += NT) {
      const int t = k / (DC / 4), d = 4 * (k % (DC / 4));
      copy16(tc::smem_u32(&tcol[buf][t][d]), pc + token(i0 + t) * lc.st + d);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // lambda as one of the two fp32 values beside it, chosen token by token so that their running product
  // stays within a rounding of the exact power (one fixed value's rounding, compounded over a memory of
  // 10^4 tokens, would be an error of 6e-4)
  const double lam64 = exp(static_cast<double>(ld));
  const float lam0 = static_cast<float>(lam64);
  const double off = lam64 - lam0;
  const float lam1 = off == 0. || lam0 == 0.f ? lam0 : __int_as_float(__float_as_int(lam0) + (off < 0. ? -1 : 1));
  const float share = lam1 == lam0 ? 0.f : static_cast<float>(off / (static_cast<double>(lam1) - lam0));
  float owed = 0.f;

  // lanes with bit 4, 3, 2 clear keep the lower half of the columns each time
  const int ycol = c0 + ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
  float *y = static_cast<float *>(r.y) + ((static_cast<size_t>(it.b) * p.T + it.t0) * p.H + h) * DC + ycol;
  const size_t ystep = static_cast<size_t>(p.H) * DC;
  const float bscale = r.bscale, yscale = r.yscale;
  if (count > 0) fetch(0, 0);
  for (int i0 = 0, buf = 0; i0 < count; i0 += TT, buf ^= 1) {
    if (i0 + TT < count) {
      fetch(i0 + TT, buf ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    const int n = min(TT, count - i0);
#pragma unroll 2
    for (int t = 0; t < n; ++t) {
      owed += share;
      const bool up = owed > 0.5f;
      owed -= up ? 1.f : 0.f;
      const float lam = up ? lam1 : lam0;
      const uint64_t l2 = pair_f32(lam, lam);
      uint64_t c[4], y2[4] = {0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = *reinterpret_cast<const uint64_t *>(&tcol[buf][t][c0 + 2 * k]);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float b = bscale * tb[buf][t][lane + 32 * i];
        const uint64_t b2 = pair_f32(b, b);
        uint64_t a2 = 0;
        if (!PHASE1) {
          const float a = ta[buf][t][lane + 32 * i];
          a2 = pair_f32(a, a);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          S[i][k] = rev ? fma_f32x2(b2, c[k], S[i][k]) : fma_f32x2(l2, S[i][k], mul_f32x2(b2, c[k]));
          if (!PHASE1) y2[k] = fma_f32x2(a2, S[i][k], y2[k]);
          if (rev) S[i][k] = mul_f32x2(l2, S[i][k]);
        }
      }
      if (!PHASE1) {
        float v[8], z4[4], z2[2], z;
#pragma unroll
        for (int k = 0; k < 4; ++k) unpair_f32(y2[k], v[2 * k], v[2 * k + 1]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          z4[k] = (lane & 16 ? v[k + 4] : v[k]) + __shfl_xor_sync(0xffffffffu, lane & 16 ? v[k] : v[k + 4], 16);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          z2[k] = (lane & 8 ? z4[k + 2] : z4[k]) + __shfl_xor_sync(0xffffffffu, lane & 8 ? z4[k] : z4[k + 2], 8);
        z = (lane & 4 ? z2[1] : z2[0]) + __shfl_xor_sync(0xffffffffu, lane & 4 ? z2[0] : z2[1], 4);
        z += __shfl_xor_sync(0xffffffffu, z, 2);
        z += __shfl_xor_sync(0xffffffffu, z, 1);
        if ((lane & 3) == 0) y[token(i0 + t) * ystep] = yscale * z;
      }
    }
    __syncthreads();   // this tile is read before the one after the next replaces it
  }

  float *dst = nullptr;
  if (PHASE1) dst = r.X + static_cast<size_t>(it.slot) * DA * DC;
  else if (it.nseg == 1 && r.s_final && page >= 0) dst = r.s_final + (static_cast<size_t>(page) * p.H + h) * DA * DC;
  if (dst) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) *reinterpret_cast<uint64_t *>(dst + (lane + 32 * i) * DC + c0 + 2 * c) = S[i][c];
  }
  if (beside) tc::griddep_wait();
}

template <int DA, int DC, bool PHASE1>
cudaError_t launch_run(const LinProblem &p, int ir, bool pdl, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(lin_blocks(p)));
  cfg.blockDim = dim3(DC * 4);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, linear_token_kernel<DA, DC, PHASE1>, p, ir, ir > 0);
}

template <bool PHASE1>
cudaError_t launch_shape(const LinProblem &p, int ir, bool pdl, cudaStream_t s) {
  const LinRun &r = p.run[ir];
  if (r.da == 128 && r.dc == 128) return launch_run<128, 128, PHASE1>(p, ir, pdl, s);
  if (r.da == 128) return launch_run<128, 64, PHASE1>(p, ir, pdl, s);
  if (r.dc == 128) return launch_run<64, 128, PHASE1>(p, ir, pdl, s);
  return launch_run<64, 64, PHASE1>(p, ir, pdl, s);
}

}  // namespace
}  // namespace gdr

cudaError_t gdr_launch_linear_token(const gdr::LinProblem &p, bool phase1, bool pdl, cudaStream_t s) {
  for (int i = 0; i < p.nrun; ++i) {
    // the first run waits for the phase before; the others start once all of its CTAs are past that wait, run
    // beside it and end after it
    const bool dep = pdl || i > 0;
    const cudaError_t e = phase1 ? gdr::launch_shape<true>(p, i, dep, s) : gdr::launch_shape<false>(p, i, dep, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}
