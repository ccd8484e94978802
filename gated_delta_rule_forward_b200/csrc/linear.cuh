// Linear attention with a decay per head: the problem description shared by
// its kernels, and the device helpers that read it.
//
// With lambda = exp(log_decay[h]) the operator is
//     S_t = lambda S_{t-1} + k_t v_t^T,     o_t = scale S_t^T q_t,
// and its gradients are three more runs of the same recurrence:
//     dq_t = scale S_t dO_t                        = run(a = dO, b = v,  c = k)
//     dv_s = dS_s^T k_s                            = reverse run(a = k,  b = q,  c = dO)
//     dk_s = dS_s v_s                              = reverse run(a = v,  b = dO, c = q)
//     dS_t = scale q_t dO_t^T + lambda dS_{t+1}    (the reverse runs' state, or its transpose)
// so every kernel here computes a "run" of three tensors a, b, c:
//     forward:  S <- lambda S + bscale b c^T,  y = yscale S^T a
//     reverse:  S <- S + bscale b c^T,         y = yscale S^T a,   S <- lambda S
// with S [da][dc].  The reverse state is carried with the decay to the next
// (earlier) token applied, so that what a run leaves is the gradient of the
// initial state, and its start is the gradient of the final state.
//
// Long sequences are cut into segments of `seg` tokens that run side by side:
// phase 1 leaves every segment's end state from a zero start, those are chained
// into start states (by each segment of phase 2 for itself where there are few,
// by a kernel in between otherwise), and phase 2 runs all segments from them.
#pragma once

#include <string>

#include "common.cuh"

namespace gdr {

constexpr int kLinMaxRuns = 3;

// A [B, T, heads, d] tensor with unit stride along d; value head h reads head h / div.
struct LinTensor {
  const void *p;
  long long sb, st, sh;   // elements
  int div;
};

struct LinRun {
  int ia, ib, ic;       // indexes into LinProblem::t
  int da, dc;
  int reverse;
  float bscale, yscale;
  void *y;              // [B, T, H, dc], dense
  int y_f32;            // y in fp32 instead of the I/O type
  const float *s0;      // start state [.., H, da, dc], or null (zeros)
  int s0_t;             // s0 is laid out [.., H, dc, da]
  float *s_final;       // end state [.., H, da, dc], or null
  float *X;             // segment states [slots, da, dc], used when segmented
  float *XS;            // and the start states that phase 2 makes of them
};

struct LinProblem {
  int nrun;
  LinRun run[kLinMaxRuns];
  LinTensor t[4];
  bool bf16_io;
  int B, T, H, N;        // N sequences: N = B, or the packed ones of B = 1
  const int *cu;         // [N + 1] token offsets of the packed sequences, or null
  const int *slots;      // [N] page of each sequence's state, or null (page n)
  int pages;
  const float *log_decay;   // [H]
  int seg;               // tokens per segment
  int G;                 // segments of a sequence (packed: at most)
  int items;             // (sequence, segment) pairs (packed: an upper bound)
  int chained;           // X holds start states already (the chain kernel ran)
  int s0_copied;         // phase 1 leaves the sequences' start states in their first segments' XS (a packed forward in place)
  int zero_rest;         // the outputs' rows of no packed sequence become zeros
  int fault;             // the bf16 kernels' first block leaves out what its waits wait for (failure tests)
};

// A run's blocks are its segments of every head; each has a state in X.
inline long lin_blocks(const LinProblem &p) { return static_cast<long>(p.items) * p.H; }
inline bool lin_segmented(const LinProblem &p) { return p.G > 1; }
// Segments up to which phase 2 chains the states itself.  In a packed bf16 forward whose sequences have one on
// average G is only a bound, and those that run whole then start beside phase 1, as they do not behind a chain
// kernel: 16 ragged prompts of 9200 tokens, 16 heads, 69 us for 75, of 128 x 128 71 for 82.  (Two sequences in five
// segments each: 66 for 61; the packed backward 286 for 283, fp32 527 for 519.)
constexpr int kLinSelfChain = 4, kLinSelfChainPacked = 16;
inline bool lin_self_chains(const LinProblem &p) {
  return p.G <= kLinSelfChain || (p.G <= kLinSelfChainPacked && p.cu && p.bf16_io && p.nrun == 1 && p.N >= p.G);
}

#ifdef __CUDACC__
// One segment of one (sequence, head).  `ok` is false for an index past the last one.
struct LinItem {
  bool ok;
  int n, h, g, nseg, b;
  int t0, len;   // the sequence's first token within its batch row, its length
  int beg, end;  // the segment's tokens within the sequence
  int slot, step;   // its entry of X, and the distance to the next segment's
};

__device__ __forceinline__ int lin_cu(const LinProblem &p, int n) { return min(max(__ldg(p.cu + n), 0), p.T); }

// Packed: sequence n's items start at cu[n] / seg + n: consecutive starts differ by at
// least the sequence's segments (and by at least one for an empty sequence), so
// a packed batch needs no table.  The search is 32-ary, one probe per lane;
// offsets are clamped to [0, T], so that any cu_seqlens stays within the rows.
__device__ __forceinline__ LinItem lin_item(const LinProblem &p, int block) {
  LinItem it;
  // neighbouring heads in neighbouring blocks: they read neighbouring rows
  const int x = block / p.H;
  it.h = block - x * p.H;
  it.slot = block;
  it.step = p.H;
  if (!p.cu) {
    it.n = x / p.G;
    it.g = x - it.n * p.G;
    it.nseg = p.G;
    it.b = it.n;
    it.t0 = 0;
    it.len = p.T;
    it.beg = it.g * p.seg;
    it.end = min(p.T, it.beg + p.seg);
    it.ok = true;
    return it;
  }
  const int lane = threadIdx.x & 31;
  int lo = 0, cnt = p.N;
  bool found = true;
  while (true) {
    const int step = (cnt + 31) / 32;
    const int i = lane * step;
    const bool le = i < cnt && lin_cu(p, lo + i) / p.seg + lo + i <= x;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    if (m == 0) {
      found = false;
      break;
    }
    const int k = 31 - __clz(m);
    lo += k * step;
    cnt = min(step, cnt - k * step);
    if (step == 1) break;
  }
  it.n = lo;
  it.b = 0;
  it.t0 = lin_cu(p, lo);
  it.len = max(lin_cu(p, lo + 1) - it.t0, 0);
  it.nseg = max(1, (it.len + p.seg - 1) / p.seg);
  it.g = x - (it.t0 / p.seg + lo);
  it.ok = found && it.g < it.nseg;
  it.beg = it.g * p.seg;
  it.end = min(it.len, it.beg + p.seg);
  return it;
}

// The run a block of a phase's launch belongs to, and its block in that run: the runs' blocks in turn where one
// body does all runs, which then read their common tensors together, one run's after another's where a run has a
// body of its own, which neighbouring SMs then share.  (bf16 backward of 8 sequences of 2048 tokens, 8 heads, for seconds: 112
// us in turn, 116 one after another; of 128 x 64, after a rest, 166 and 100.  The run's index as comparisons: as a quotient,
// 4 sequences of 4096, 16 heads, take 218 us for 208.)
template <bool IN_TURN>
__device__ __forceinline__ const LinRun &lin_run(const LinProblem &p, unsigned &block) {
  const unsigned blocks = gridDim.x / p.nrun;
  const unsigned i = IN_TURN ? blockIdx.x % p.nrun : (blockIdx.x >= blocks) + (blockIdx.x >= 2 * blocks);
  block = IN_TURN ? blockIdx.x / p.nrun : blockIdx.x - i * blocks;
  return p.run[i == 0 ? 0 : i == 1 ? 1 : 2];
}

// This block's share of the zeros in a run's output rows of no sequence: [0, first) and [end, T), the offsets
// cu[0] and cu[N].
__device__ __forceinline__ void lin_zero_rest(const LinProblem &p, void *y, size_t row_bytes, int first, int end,
                                              unsigned block, unsigned blocks) {
  uint4 *const v = static_cast<uint4 *>(y);
  const size_t row = row_bytes / 16, step = static_cast<size_t>(blocks) * blockDim.x;
  const size_t mine = static_cast<size_t>(block) * blockDim.x + threadIdx.x;
  for (size_t i = mine; i < first * row; i += step) v[i] = make_uint4(0u, 0u, 0u, 0u);
  for (size_t i = end * row + mine; i < p.T * row; i += step) v[i] = make_uint4(0u, 0u, 0u, 0u);
}

// lambda^n by way of 64 bits.
__device__ __forceinline__ float lin_pow64(float log_decay, int n) {
  return static_cast<float>(exp(static_cast<double>(log_decay) * n));
}

// The same as hi + lo, lo above zero where the power is, for a chain of many segments: one fp32 value, always off the same way
// by up to 2^-25, would be their states' largest error (147 segments: 2.4e-6 of the end state).
__device__ __forceinline__ float2 lin_pow64_parts(float log_decay, int n) {
  const double x = exp(static_cast<double>(log_decay) * n);
  const float hi = __double2float_rd(x);
  return make_float2(hi, fmaxf(static_cast<float>(x - hi), hi * 0x1p-60f));
}

// Page of sequence n's state, or -1 where its slot lies outside the pool.
__device__ __forceinline__ int lin_page(const LinProblem &p, int n) {
  if (!p.slots) return n;
  const int s = __ldg(p.slots + n);
  return s >= 0 && s < p.pages ? s : -1;
}

// A segment's start state from the start state of its sequence and the end states (from
// zero) of the segments before it in the run's order, and after the last segment the
// end state of the sequence where it is wanted.  The whole block; `to` may be read by it after a
// barrier.  (So few segments may take lambda's powers as one fp32 value each.)
__device__ __forceinline__ void lin_self_chain(const LinProblem &p, const LinRun &r, const LinItem &it, int page,
                                               bool last, int da, int dc, float *to, int tid, int threads) {
  const float ld = __ldg(p.log_decay + it.h);
  const size_t elems = static_cast<size_t>(da) * dc;
  const float *X = r.X + static_cast<size_t>(it.slot - it.g * it.step) * elems;   // segment 0's
  const int before = r.reverse ? it.nseg - 1 - it.g : it.g;
  const bool fin = last && r.s_final && page >= 0;
  const size_t at_page = (static_cast<size_t>(page < 0 ? 0 : page) * p.H + it.h) * elems;
  float f[kLinSelfChain];
  {   // the decay over the run's k-th segment; a lane computes one of them
    const int k = tid & 3, seg = r.reverse ? it.nseg - 1 - k : k;
    static_assert(kLinSelfChain == 4, "lanes");
    const float x = k < before + fin ? lin_pow64(ld, min(it.len, (seg + 1) * p.seg) - seg * p.seg) : 0.f;
#pragma unroll
    for (int i = 0; i < kLinSelfChain; ++i) f[i] = __shfl_sync(0xffffffffu, x, i);
  }
  for (int e = 4 * tid; e < static_cast<int>(elems); e += 4 * threads) {
    float4 d[kLinSelfChain];
#pragma unroll
    for (int k = 0; k < kLinSelfChain; ++k) {
      const int seg = r.reverse ? it.nseg - 1 - k : k;
      if (k < before + fin) d[k] = *reinterpret_cast<const float4 *>(X + static_cast<size_t>(seg) * it.step * elems + e);
    }
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r.s0 && page >= 0) {
      const float *src = r.s0 + at_page;
      const int row = e / dc, col = e - row * dc;
      if (r.s0_t) s = make_float4(src[(col + 0) * da + row], src[(col + 1) * da + row], src[(col + 2) * da + row],
                                  src[(col + 3) * da + row]);
      else s = *reinterpret_cast<const float4 *>(src + e);
    }
#pragma unroll
    for (int k = 0; k < kLinSelfChain; ++k) {
      if (k == before) *reinterpret_cast<float4 *>(to + e) = s;
      if (k >= before + fin) continue;
      s.x = fmaf(f[k], s.x, d[k].x);
      s.y = fmaf(f[k], s.y, d[k].y);
      s.z = fmaf(f[k], s.z, d[k].z);
      s.w = fmaf(f[k], s.w, d[k].w);
    }
    if (fin) *reinterpret_cast<float4 *>(r.s_final + at_page + e) = s;
  }
}

// The same for any number of segments of a forward, their loads four at a time.  (With a copied start state the
// first segment's is there already.)
__device__ __forceinline__ void lin_self_chain_long(const LinProblem &p, const LinRun &r, const LinItem &it, int page,
                                                    bool last, int da, int dc, float *to, int tid, int threads) {
  const float ld = __ldg(p.log_decay + it.h);
  const size_t elems = static_cast<size_t>(da) * dc;
  const float *X = r.X + static_cast<size_t>(it.slot - it.g * it.step) * elems;   // segment 0's
  const bool fin = last && r.s_final && page >= 0;
  const size_t at_page = (static_cast<size_t>(page < 0 ? 0 : page) * p.H + it.h) * elems;
  const int steps = it.g + fin;
  if (p.s0_copied && it.g == 0) return;
  const float *s0 = p.s0_copied           ? r.XS + static_cast<size_t>(it.slot - it.g * it.step) * elems
                    : r.s0 && page >= 0 ? r.s0 + at_page
                                        : nullptr;
  float full, ftail;   // the decays over a segment and over the sequence's last one, each computed by a lane
  {
    const float x = lin_pow64(ld, tid & 1 ? it.len - (it.nseg - 1) * p.seg : p.seg);
    full = __shfl_sync(0xffffffffu, x, 0);
    ftail = __shfl_sync(0xffffffffu, x, 1);
  }
  constexpr int U = 4;
  for (int e = 4 * tid; e < static_cast<int>(elems); e += 4 * threads) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (s0) s = *reinterpret_cast<const float4 *>(s0 + e);
#pragma unroll 1
    for (int k0 = 0; k0 < steps; k0 += U) {
      float4 d[U];
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (k0 + k < steps) d[k] = *reinterpret_cast<const float4 *>(X + static_cast<size_t>(k0 + k) * it.step * elems + e);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (k0 + k >= steps) break;
        if (k0 + k == it.g) *reinterpret_cast<float4 *>(to + e) = s;
        const float f = k0 + k == it.nseg - 1 ? ftail : full;
        s.x = fmaf(f, s.x, d[k].x);
        s.y = fmaf(f, s.y, d[k].y);
        s.z = fmaf(f, s.z, d[k].z);
        s.w = fmaf(f, s.w, d[k].w);
      }
    }
    *reinterpret_cast<float4 *>(fin ? r.s_final + at_page + e : to + e) = s;
  }
}

// lambda as hi + lo, off by a few roundings (2^-24) of the smaller of lambda and 1 - lambda: above 1/2 from
// e = lambda - 1 = t (t + 2), t = exp(x) - 1 at half the decay by its Taylor series to x^8 (|x| < 0.35: the
// next term is 6e-10 of it).  lo is above zero where lambda is, so that an infinite state stays one.  In every
// thread and without a branch: with expm1f, or in one warp for all, decoding 256 rows of 16 heads of
// 64 x 64 takes 16.4 and 15.8 us for 15.4, with one fp32 lambda 15.2.
__device__ __forceinline__ float2 lin_decay(float log_decay) {
  const float x = 0.5f * log_decay;
  float e = 1.f / 40320.f;
  e = fmaf(e, x, 1.f / 5040.f);
  e = fmaf(e, x, 1.f / 720.f);
  e = fmaf(e, x, 1.f / 120.f);
  e = fmaf(e, x, 1.f / 24.f);
  e = fmaf(e, x, 1.f / 6.f);
  e = fmaf(e, x, 0.5f);
  e = fmaf(e * x, x, x);
  e = fmaf(e, e, 2.f * e);
  const float near = __fadd_rd(1.f, e);   // and e - (near - 1): both differences exact
  const bool small = log_decay > -0.6931472f;
  const float hi = small ? near : expf(log_decay);
  const float lo = small ? e - (near - 1.f) : 0.f;
  return make_float2(hi, fmaxf(lo, hi * 0x1p-60f));
}
#endif

}  // namespace gdr

// Launchers.  `phase1`: end states of the segments from zero, into X (of a
// sequence's last one, in the run's order, only where its end state is wanted);
// otherwise the runs themselves.
cudaError_t gdr_launch_linear_token(const gdr::LinProblem &p, bool phase1, bool pdl, cudaStream_t s);
cudaError_t gdr_launch_linear_chain(const gdr::LinProblem &p, bool pdl, cudaStream_t s);

// A whole call: the plan (segment length) is gdr_linear_plan's, `ws` holds
// gdr_linear_workspace_bytes.
void gdr_linear_plan(gdr::LinProblem *p, int sms);
size_t gdr_linear_workspace_bytes(const gdr::LinProblem &p);
cudaError_t gdr_launch_linear(gdr::LinProblem &p, void *ws, cudaStream_t s, std::string *err);

// y[b,t,hk,:] = sum over the group's p.H / Hk heads of x[b,t,hk * G + i,:], for the tokens of the packed
// sequences (all tokens when p.cu is null; zeros in the other rows when p.zero_rest).
cudaError_t gdr_launch_linear_group_sum(const float *x, void *y, const gdr::LinProblem &p, int Hk, int d, cudaStream_t s);

namespace gdr {
struct LinDecodeProblem {
  int N, Hk, H, dk, dv, pages;
  bool bf16_io;
  const void *q, *k, *v;      // [N, Hk, dk], [N, Hk, dk], [N, H, dv], dense
  const float *log_decay;     // [H]
  const int *slots;           // [N] or null
  float *state;               // [pages, H, dk, dv]
  void *o;                    // [N, H, dv]
  float scale;
};
}  // namespace gdr
cudaError_t gdr_launch_linear_decode(const gdr::LinDecodeProblem &p, int sms, cudaStream_t s);
