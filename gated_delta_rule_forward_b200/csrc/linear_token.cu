// Linear attention with a decay per head, token by token in fp32: the exact
// path, used for fp32 tensors (and for the state copies of a call without
// tokens).
//
// One CTA owns one (run, segment, head), one warp of it eight columns of the
// state; the da x 8 fp32 slice lives in registers (eight lanes share the rows of two
// columns; rows in pairs).  Tokens come through shared memory sixteen at a time, the
// next sixteen on their way while these are computed.  Per token S <- lambda S + b c^T
// and y = S^T a; the sums of four tokens' columns go over the lanes together, seven
// exchanges for eight of them.  (A reverse run is the same recurrence with the first
// token's decay moved to the end.)
//
// Bound by the FMA pipe: 3 d^2 multiplications and additions a token are 200 ns of an
// SM at d = 128; it takes 380 (the pipe 57% active).  Two sequences of 500 tokens, 4
// heads: 33 us in a graph, their backward 70; 74 of 300, 8 heads: 460 us.  With a column's rows
// over all 32 lanes (nine exchanges a token) the forwards were 43 and 636.
#include "linear.cuh"
#include "tc_util.cuh"

namespace gdr {
namespace {

using tc::fma_f32x2;
using tc::mul_f32x2;
using tc::pair_f32;
using tc::unpair_f32;

constexpr int TT = 16;   // tokens a tile
constexpr int NC = 2;    // columns a lane

__device__ __forceinline__ void copy16(uint32_t dst, const float *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <int DA, int DC, bool PHASE1>
constexpr int smem_floats = 2 * TT * ((PHASE1 ? 1 : 2) * DA + DC);

template <int DA, int DC, bool PHASE1>
__device__ __forceinline__ void token_run(const LinProblem &p, const LinRun &r, unsigned block, float *smem) {
  constexpr int R = DA / 32, NT = DC * 8 / NC, HC = NC / 2;
  float(*tb)[TT][DA] = reinterpret_cast<float(*)[TT][DA]>(smem);
  float(*tcol)[TT][DC] = reinterpret_cast<float(*)[TT][DC]>(smem + 2 * TT * DA);
  float(*ta)[TT][DA] = reinterpret_cast<float(*)[TT][DA]>(smem + 2 * TT * (DA + DC));   // (not in phase 1)
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  if (!PHASE1 && p.zero_rest && !r.y_f32)
    lin_zero_rest(p, r.y, static_cast<size_t>(p.H) * DC * 4, lin_cu(p, 0), lin_cu(p, p.N), block, gridDim.x / p.nrun);
  if (tid >= NT) return;   // a narrow run beside wide ones
  const LinItem it = lin_item(p, block);
  const int h = it.h;
  const bool rev = r.reverse != 0;
  const bool last = rev ? it.g == 0 : it.g == it.nseg - 1;    // in the run's order
  if (!it.ok || (PHASE1 && last && (it.nseg == 1 || !r.s_final))) return;
  const float ld = __ldg(p.log_decay + h);
  const int page = lin_page(p, it.n);

  // S[j][k][c]: rows row0 + 32 j + 2 k (+ 1), column col0 + c
  const int row0 = 4 * (lane & 7), col0 = 4 * NC * (tid >> 5) + NC * (lane >> 3);
  uint64_t S[R][2][NC];
#pragma unroll
  for (int j = 0; j < R; ++j)
#pragma unroll
    for (int k = 0; k < 2 * NC; ++k) S[j][k / NC][k % NC] = 0;
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
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int row = row0 + 32 * j + 2 * k;
          if (t) {
#pragma unroll
            for (int c = 0; c < NC; ++c) S[j][k][c] = *reinterpret_cast<const uint64_t *>(start + (col0 + c) * DA + row);
          } else {
#pragma unroll
            for (int c = 0; c < NC; c += 2) {
              const float2 x = *reinterpret_cast<const float2 *>(start + row * DC + col0 + c);
              const float2 y = *reinterpret_cast<const float2 *>(start + (row + 1) * DC + col0 + c);
              S[j][k][c] = pair_f32(x.x, y.x);
              S[j][k][c + 1] = pair_f32(x.y, y.y);
            }
          }
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
  auto decay = [&]() {
    owed += share;
    const bool up = owed > 0.5f;
    owed -= up ? 1.f : 0.f;
    return up ? lam1 : lam0;
  };
  // of four tokens' columns each lane of a row group sums up HC: token yt, columns col0 + HC yc ..
  const int yc = (lane >> 2) & 1, yt = lane & 3;
  float *y = static_cast<float *>(r.y) + ((static_cast<size_t>(it.b) * p.T + it.t0) * p.H + h) * DC + col0 + HC * yc;
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
#pragma unroll 1
    for (int t0 = 0; t0 < n; t0 += 4) {
      float v[4][NC] = {};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int t = t0 + u;
        if (t >= n) break;
        const float lam = rev && i0 + t == 0 ? 1.f : decay();
        const uint64_t l2 = pair_f32(lam, lam);
        uint64_t c[NC], y2[NC] = {};
#pragma unroll
        for (int e = 0; e < NC; ++e) {
          const float x = bscale * tcol[buf][t][col0 + e];
          c[e] = pair_f32(x, x);
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
          const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(&tb[buf][t][row0 + 32 * j]);
          ulonglong2 a = {0, 0};
          if (!PHASE1) a = *reinterpret_cast<const ulonglong2 *>(&ta[buf][t][row0 + 32 * j]);
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < NC; ++e) {
              const uint64_t b2 = k ? b.y : b.x;
              uint64_t &s = S[j][k][e];
              s = fma_f32x2(l2, s, mul_f32x2(b2, c[e]));
              if (!PHASE1) y2[e] = fma_f32x2(k ? a.y : a.x, s, y2[e]);
            }
        }
        if (!PHASE1)
#pragma unroll
          for (int e = 0; e < NC; ++e) {
            float lo, hi;
            unpair_f32(y2[e], lo, hi);
            v[u][e] = lo + hi;
          }
      }
      if (!PHASE1) {
#pragma unroll
        for (int c = 0; c < HC; ++c) {
          float z4[4], z2[2], z;
#pragma unroll
          for (int u = 0; u < 4; ++u)
            z4[u] = (yc ? v[u][HC + c] : v[u][c]) + __shfl_xor_sync(0xffffffffu, yc ? v[u][c] : v[u][HC + c], 4);
#pragma unroll
          for (int u = 0; u < 2; ++u)
            z2[u] = (lane & 2 ? z4[u + 2] : z4[u]) + __shfl_xor_sync(0xffffffffu, lane & 2 ? z4[u] : z4[u + 2], 2);
          z = (lane & 1 ? z2[1] : z2[0]) + __shfl_xor_sync(0xffffffffu, lane & 1 ? z2[0] : z2[1], 1);
          if (t0 + yt < n) y[token(i0 + t0 + yt) * ystep + c] = yscale * z;
        }
      }
    }
    __syncthreads();   // this tile is read before the one after the next replaces it
  }

  if (rev && count > 0) {   // a reverse state is left with the decay to the next token applied
    const float lam = decay();
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int k = 0; k < 2 * NC; ++k) S[j][k / NC][k % NC] = mul_f32x2(pair_f32(lam, lam), S[j][k / NC][k % NC]);
  }
  float *dst = nullptr;
  if (PHASE1) dst = r.X + static_cast<size_t>(it.slot) * DA * DC;
  else if (it.nseg == 1 && r.s_final && page >= 0) dst = r.s_final + (static_cast<size_t>(page) * p.H + h) * DA * DC;
  if (dst) {
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float *to = dst + (row0 + 32 * j + 2 * k) * DC + col0;
#pragma unroll
        for (int c = 0; c < NC; c += 2) {
          float2 x, y;
          unpair_f32(S[j][k][c], x.x, y.x);
          unpair_f32(S[j][k][c + 1], x.y, y.y);
          *reinterpret_cast<float2 *>(to + c) = x;
          *reinterpret_cast<float2 *>(to + DC + c) = y;
        }
      }
  }
}

// All runs of a phase in one launch.  A forward has one run, (DA, DC); a backward dq's, dk's and dv's, the last (DA, DC)
// and, if MIXED, the others (DC, DA).
template <int DA, int DC, bool MIXED>
constexpr int kBlock = (MIXED && DA > DC ? DA : DC) * 8 / NC;

template <int DA, int DC, bool PHASE1, bool MIXED>
__global__ void __launch_bounds__(kBlock<DA, DC, MIXED>) linear_token_kernel(const __grid_constant__ LinProblem p) {
  constexpr int own = smem_floats<DA, DC, PHASE1>, other = MIXED ? smem_floats<DC, DA, PHASE1> : 0;
  __shared__ __align__(16) float smem[own > other ? own : other];
  unsigned block;
  const LinRun &r = lin_run<!MIXED>(p, block);
  if (MIXED && r.dc != DC) token_run<DC, DA, PHASE1>(p, r, block, smem);
  else token_run<DA, DC, PHASE1>(p, r, block, smem);
}

template <int DA, int DC, bool PHASE1, bool MIXED>
cudaError_t launch(const LinProblem &p, bool pdl, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(lin_blocks(p) * p.nrun));
  cfg.blockDim = dim3(kBlock<DA, DC, MIXED>);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, linear_token_kernel<DA, DC, PHASE1, MIXED>, p);
}

template <int DA, int DC>
cudaError_t launch_kind(const LinProblem &p, bool phase1, bool pdl, cudaStream_t s) {
  if (DA != DC && p.nrun == kLinMaxRuns)
    return phase1 ? launch<DA, DC, true, DA != DC>(p, pdl, s) : launch<DA, DC, false, DA != DC>(p, pdl, s);
  return phase1 ? launch<DA, DC, true, false>(p, pdl, s) : launch<DA, DC, false, false>(p, pdl, s);
}

}  // namespace
}  // namespace gdr

cudaError_t gdr_launch_linear_token(const gdr::LinProblem &p, bool phase1, bool pdl, cudaStream_t s) {
  const gdr::LinRun &r = p.run[p.nrun - 1];   // o's or dv's: (dk, dv)
  if (r.da == 128 && r.dc == 128) return gdr::launch_kind<128, 128>(p, phase1, pdl, s);
  if (r.da == 128) return gdr::launch_kind<128, 64>(p, phase1, pdl, s);
  if (r.dc == 128) return gdr::launch_kind<64, 128>(p, phase1, pdl, s);
  return gdr::launch_kind<64, 64>(p, phase1, pdl, s);
}
