// Linear attention with a decay per head in chunks of C = 64 tokens on the
// tensor cores (bf16 tensors), for any run of three tensors a, b, c (linear.cuh).
//
// With w and Gamma powers of lambda, D_ts = lambda^|t-s| on the run's side of
// the diagonal and S the state at the chunk's start in the run's order, per chunk
//     Y = yscale (Gamma_t (a_t S) + bscale sum_s D_ts (a_t . b_s) c_s),
//     S <- lambda^n S + bscale sum_s w_s b_s c_s^T,
//     forward: Gamma_t = lambda^{t+1}, w_s = lambda^{n-1-s};  reverse: the two exchanged.
// One CTA sweeps the chunks of one (run, segment, head) in order; everything is
// held transposed, so that M = 128 of the MMAs is the value width and the state
// is their tensor-memory operand:
//     P    [t][s]   = a b^T          M64  N64  K = da   (tensor memory)
//     O1^T [dc][t]  = S^T a^T        M128 N64  K = da   (S^T in bf16 in tensor memory)
//     O2^T [dc][t]  = c^T P^T        M128 N64  K = 64   (P back through shared memory in bf16)
//     dS^T [dc][da] = c^T (w b)      M128 N = da, K = 64
// The last three go to the tensor pipe in one go, and Y^T = yscale (Gamma_t O1^T + O2^T).
// The fp32 state lives in registers: lane dc of a warp quad, half of da per
// thread; S <- lambda^n S + dS is one pass over it.
//
// Rounding.  The products' inputs are exact bf16 except three: w b, P and the
// S^T operand.  w b enters the state, which is fp32, so it is split into three
// bf16 terms (24 bits, three MMAs): the state keeps fp32 accuracy; where the
// state is not kept (a later segment starts from phase 1's), two terms do, 2^-8
// of what follows.  P and S^T enter only Y, on disjoint parts of its sum, and
// are rounded once to bf16, like Y itself.
//
// Two CTAs share an SM (107 KB of shared memory, 256 tensor-memory columns, nine
// warps of 112 registers each).  One warp issues the copies and the MMAs; the
// others hand over to it through mbarriers only, so that the next chunk's P is
// formed while this one's outputs are written.
#include "linear.cuh"
#include "linear_chunk.cuh"
#include "tc_util.cuh"
#include "tma_host.cuh"

// Device-side error word of this file (see gdr_device_status()).
__device__ int g_gdr_linear_error = 0;

namespace gdr {
namespace tc {
namespace {

constexpr int C = 64;
constexpr int UNROLL_W = 2;
constexpr int NCOMPUTE = 8;                       // compute warps; one more issues copies and MMAs
constexpr int NTHREADS = 32 * (NCOMPUTE + 1);
constexpr uint32_t TILE = 16384;        // 64 rows of two 128-byte atoms
constexpr uint32_t OFF_A = 0;           // a (phase 1: the second c buffer)
constexpr uint32_t OFF_C = TILE;
constexpr uint32_t OFF_B = 2 * TILE;    // two buffers; the first term of w b replaces b in place
constexpr uint32_t OFF_M = 4 * TILE;    // second and third terms of w b; then each warp's 2 KB of output rows
constexpr uint32_t OFF_L = 5 * TILE;
constexpr uint32_t OFF_P = 6 * TILE;    // bf16 P, rows t, 8 KB
constexpr uint32_t OFF_PW = OFF_P + 8192;      // lambda^0 .. lambda^64, then what fp32 loses of them
constexpr uint32_t OFF_D = OFF_PW + 2 * 65 * 4 + 8;   // yscale bscale lambda^d at 64 + d, zeros for d < 0
constexpr uint32_t OFF_BAR = OFF_D + 128 * 4;
constexpr uint32_t SMEM_BYTES = OFF_BAR + 128 + 1024;
static_assert(OFF_BAR % 16 == 0 && 2 * (SMEM_BYTES + 1024) <= 233472, "two CTAs per SM");
constexpr uint32_t COL_DS = 0;     // dS^T, 128 columns
constexpr uint32_t COL_P = 0;      // P, 64 columns: read before dS^T is formed, formed after dS^T is read
constexpr uint32_t COL_S = 128;    // S^T in bf16, 64 columns
constexpr uint32_t COL_O2 = 128;   // O2^T over S^T: formed after O1^T, read before the next S^T
constexpr uint32_t COL_O1 = 192;   // O1^T, 64 columns
constexpr uint32_t TMEM_COLS = 256;

// Bounded wait that also gives up once another thread has.
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t phase, volatile int *abort) {
  if (mbar_try_wait(bar, phase)) return true;
  const long long start = clock64();
  while (!mbar_try_wait(bar, phase)) {
    if (*abort) return false;
    if (clock64() - start > (1ll << 31)) {
      *abort = 1;
      return false;
    }
  }
  return true;
}

// lambda^64 as one of the two fp32 values beside it, chosen chunk by chunk so that their
// running product stays within a rounding of the exact power: one fixed value's rounding,
// compounded over a memory of hundreds of chunks, would be the state's largest error.
struct ChunkDecay {
  float below, above, frac, acc;   // lambda^64 = below + frac (above - below)
  __device__ __forceinline__ void init(float hi, float lo) {   // lambda^64 = hi + lo, |lo| at most half a step
    const int step = lo < 0.f ? -1 : 1;
    const float other = lo == 0.f || hi == 0.f ? hi : __int_as_float(__float_as_int(hi) + step);
    below = hi;
    above = other;
    frac = other == hi ? 0.f : lo / (other - hi);
    acc = 0.f;
  }
  __device__ __forceinline__ float next() {
    acc += frac;
    const bool up = acc > 0.5f;
    acc -= up ? 1.f : 0.f;
    return up ? above : below;
  }
};

// w x of two bf16 values x as a sum of bf16 pairs: two terms keep 16 significant bits,
// three keep 24.
__device__ __forceinline__ void split_pair(uint32_t x, uint64_t w, uint64_t minus_one, bool three, uint32_t &hi,
                                           uint32_t &mid, uint32_t &lo) {
  const uint64_t p = mul_f32x2(pair_f32(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)), w);
  float a, b;
  unpair_f32(p, a, b);
  hi = pack_bf16x2(a, b);
  const uint64_t r = fma_f32x2(pair_f32(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)), minus_one, p);
  unpair_f32(r, a, b);
  mid = pack_bf16x2(a, b);
  if (three) {
    unpair_f32(fma_f32x2(pair_f32(__uint_as_float(mid << 16), __uint_as_float(mid & 0xffff0000u)), minus_one, r), a, b);
    lo = pack_bf16x2(a, b);
  }
}

template <int DA, int DC, bool PHASE1>
__global__ void __launch_bounds__(NTHREADS, 2)
    linear_chunk_kernel(const __grid_constant__ LinProblem p, const __grid_constant__ LinChunkMaps maps,
                        const LinRunSel sel) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + (-smem_u32(smem_raw) & 1023u);   // an offset, so that accesses stay shared ones
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ri = sel.run[blockIdx.x % sel.n];
  const int xh = blockIdx.x / sel.n;
  const int h = xh % p.H, x = xh / p.H;
  const LinRun &r = p.run[ri];
  const bool rev = r.reverse != 0;
  const LinItem it = lin_item(p, x);
  const bool last = rev ? it.g == 0 : it.g == it.nseg - 1;   // in the run's order
  if (!it.ok || (PHASE1 && last)) {
    griddep_launch_dependents();
    griddep_wait();
    return;
  }

  float *pw = reinterpret_cast<float *>(sm + OFF_PW), *pw_lo = pw + 65;
  float *dtab = reinterpret_cast<float *>(sm + OFF_D);
  uint64_t *bar_a = reinterpret_cast<uint64_t *>(sm + OFF_BAR);   // a landed
  uint64_t *bar_b = bar_a + 1;       // [2] b landed
  uint64_t *bar_c = bar_a + 3;       // [2] c landed (the second one in phase 1 only)
  uint64_t *bar_p = bar_a + 5;       // P formed
  uint64_t *bar_o1 = bar_a + 6;      // O1^T formed
  uint64_t *bar_o = bar_a + 7;       // O2^T formed
  uint64_t *bar_kv = bar_a + 8;      // dS^T formed
  uint64_t *bar_ready = bar_a + 9;   // P, w b and S^T written (8 warps)
  uint64_t *bar_ds = bar_a + 10;     // dS^T read (8 warps)
  uint64_t *bar_drain = bar_a + 11;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar_a + 12);
  volatile int *abort = reinterpret_cast<volatile int *>(bar_a + 13);

  if (warp == 0) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  if (tid == 32) {
    for (int i = 0; i < 9; ++i) mbar_init(bar_a + i, 1);
    mbar_init(bar_ready, NCOMPUTE);
    mbar_init(bar_ds, NCOMPUTE);
    mbar_init(bar_drain, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (tid >= 64 && tid < 64 + 65) {
    const int m = tid - 64;
    const double e = m == 0 ? 1.0 : exp(static_cast<double>(__ldg(p.log_decay + h)) * m);
    const float hi = static_cast<float>(e);
    pw[m] = hi;
    pw_lo[m] = static_cast<float>(e - hi);
    if (m < C) {
      dtab[C + m] = r.bscale * r.yscale * hi;
      dtab[m] = 0.f;
    }
  }
  // value widths of 64: the upper 64 lanes of the M = 128 products read zeros
  if (DC == 64)
    for (int i = tid; i < 512; i += NTHREADS) {
      reinterpret_cast<uint4 *>(sm + OFF_C + 8192)[i] = make_uint4(0u, 0u, 0u, 0u);
      if (PHASE1) reinterpret_cast<uint4 *>(sm + OFF_A + 8192)[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();

  const int beg = it.g * p.seg, end = min(it.len, beg + p.seg);
  const int nch = (end - beg + C - 1) / C;
  const int page = lin_page(p, it.n);
  float *const final_page = !PHASE1 && last && r.s_final && page >= 0
                                ? r.s_final + (static_cast<size_t>(page) * p.H + h) * DA * DC : nullptr;
  // a state that leaves in fp32 takes all three terms; one that only makes bf16 outputs, two
  const bool three = PHASE1 || final_page;
  auto chunk_row = [&](int i) { return beg + C * (rev ? nch - 1 - i : i); };
  bool ok = true;

  if (warp == NCOMPUTE) {
    // ---------------------------------------------------------------- issuer: copies and MMAs
    if (lane == 0) {
      const CUtensorMap *ma = &maps.m[r.ia], *mb = &maps.m[r.ib], *mc = &maps.m[r.ic];
      const int ha = h / p.t[r.ia].div, hb = h / p.t[r.ib].div, hc = h / p.t[r.ic].div;
      const uint32_t base = smem_u32(sm);
      uint32_t issued_a = 0, issued_b = 0, issued_c = 0;
      auto load_a = [&](int i) {
        mbar_expect_tx(bar_a, DA * 128);
        for (int d = 0; d < DA / 64; ++d)
          tma_load_4d(sm + OFF_A + 8192 * d, ma, bar_a, 64 * d, ha, it.t0 + chunk_row(i), it.b);
        ++issued_a;
      };
      auto load_b = [&](int i) {
        uint64_t *bar = bar_b + (i & 1);
        mbar_expect_tx(bar, DA * 128);
        for (int d = 0; d < DA / 64; ++d)
          tma_load_4d(sm + OFF_B + TILE * (i & 1) + 8192 * d, mb, bar, 64 * d, hb, it.t0 + chunk_row(i), it.b);
        ++issued_b;
      };
      auto load_c = [&](int i) {
        const int buf = PHASE1 ? i & 1 : 0;
        mbar_expect_tx(bar_c + buf, DC * 128);
        for (int d = 0; d < DC / 64; ++d)
          tma_load_4d(sm + (buf ? OFF_A : OFF_C) + 8192 * d, mc, bar_c + buf, 64 * d, hc, it.t0 + chunk_row(i), it.b);
        ++issued_c;
      };
      // P = a b^T once both landed
      auto issue_p = [&](int i) -> bool {
        if (!wait_or_abort(bar_a, i & 1, abort) || !wait_or_abort(bar_b + (i & 1), (i >> 1) & 1, abort)) return false;
        const uint32_t a = base + OFF_A, b = base + OFF_B + TILE * (i & 1);
#pragma unroll
        for (int kk = 0; kk < DA / 16; ++kk) {
          const uint32_t o = (kk >> 2) * 8192 + (kk & 3) * 32;
          mma_ss(tmem + COL_P, sdesc(a + o, 16, 1024), sdesc(b + o, 16, 1024), idesc_bf16(C, C, false, false), kk > 0);
        }
        mma_commit(bar_p);
        return true;
      };
      if (nch > 0) {
        if (!PHASE1) load_a(0);
        load_b(0);
        load_c(0);
        if (nch > 1) {
          load_b(1);
          if (PHASE1) load_c(1);
        }
        if (!PHASE1) ok = issue_p(0);
      }
      for (int i = 0; ok && i < nch; ++i) {
        const uint32_t ph = i & 1, ct = base + (PHASE1 && ph ? OFF_A : OFF_C);
        const uint32_t term[3] = {base + OFF_B + TILE * ph, base + OFF_M, base + OFF_L};
        // the chunk after the next: into L2, while the buffers it will land in are in use
        if (!PHASE1 && i + 1 < nch)
          for (int d = 0; d < DC / 64; ++d) tma_prefetch_4d(mc, 64 * d, hc, it.t0 + chunk_row(i + 1), it.b);
        if (!PHASE1 && i + 2 < nch)
          for (int d = 0; d < DA / 64; ++d) tma_prefetch_4d(ma, 64 * d, ha, it.t0 + chunk_row(i + 2), it.b);
        if (!(ok = wait_or_abort(bar_ready, ph, abort))) break;
        tc_fence_after();
        if (!PHASE1) {   // O1^T = S^T a^T
#pragma unroll
          for (int kk = 0; kk < DA / 16; ++kk)
            mma_ts(tmem + COL_O1, tmem + COL_S + 8 * kk, sdesc(base + OFF_A + (kk >> 2) * 8192 + (kk & 3) * 32, 16, 1024),
                   idesc_bf16(128, C, false, false), kk > 0);
          mma_commit(bar_o1);
        }
        if (!(ok = wait_or_abort(bar_c + (PHASE1 ? ph : 0), PHASE1 ? (i >> 1) & 1 : ph, abort))) break;
        // dS^T = c^T (w b)
#pragma unroll
        for (int t = 0; t < 3; ++t)
          if (t < 2 || three)
#pragma unroll
            for (int kk = 0; kk < C / 16; ++kk)
              mma_ss(tmem + COL_DS, sdesc(ct + kk * 2048, 8192, 1024), sdesc(term[t] + kk * 2048, 8192, 1024),
                     idesc_bf16(128, DA, true, true), t + kk > 0);
        mma_commit(bar_kv);
        if (!PHASE1) {
          // O2^T = c^T P^T goes where S^T was read from: once O1^T is complete, while dS^T is under way
          if (!(ok = wait_or_abort(bar_o1, ph, abort))) break;
#pragma unroll
          for (int kk = 0; kk < C / 16; ++kk)
            mma_ss(tmem + COL_O2, sdesc(ct + kk * 2048, 8192, 1024), sdesc(base + OFF_P + kk * 32, 16, 1024),
                   idesc_bf16(128, C, true, false), kk > 0);
          mma_commit(bar_o);
          if (i + 1 < nch) load_a(i + 1);
        }
        if (!(ok = wait_or_abort(bar_kv, ph, abort))) break;
        if (i + 2 < nch) {
          load_b(i + 2);
          if (PHASE1) load_c(i + 2);
        }
        if (!PHASE1 && i + 1 < nch) {
          if (!(ok = wait_or_abort(bar_o, ph, abort))) break;
          load_c(i + 1);
          // P takes dS^T's columns once those are read
          if (!(ok = wait_or_abort(bar_ds, ph, abort))) break;
          tc_fence_after();
          ok = issue_p(i + 1);
        }
      }
      if (!ok) {
        // a wait gave up: report it, then let the MMAs and copies in flight finish
        // (each wait again bounded) before shared and tensor memory are released
        atomicOr(&g_gdr_linear_error, 1);
        mma_commit(bar_drain);
        mbar_wait(bar_drain, 0);
        if (issued_a) mbar_wait(bar_a, (issued_a - 1) & 1);
        for (int b = 0; b < 2; ++b) {
          const uint32_t nb = (issued_b + 1 - b) / 2, nc = PHASE1 ? (issued_c + 1 - b) / 2 : b ? 0 : issued_c;
          if (nb) mbar_wait(bar_b + b, (nb - 1) & 1);
          if (nc) mbar_wait(bar_c + b, (nc - 1) & 1);
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- compute warps
    const int quad = warp & 3, half = warp >> 2;
    const float bscale = r.bscale, yscale = r.yscale;
    const bool y_f32 = r.y_f32 != 0;
    // thread (quad, lane, half) holds S[da = half DA/2 + j][dc = 32 quad + lane], in pairs along da
    constexpr int SN = DA / 2;
    const int dcr = 32 * quad + lane, da0 = half * SN;
    const bool has_c = dcr < DC;
    uint64_t S[SN / 2];
#pragma unroll
    for (int j = 0; j < SN / 2; ++j) S[j] = 0;
    griddep_wait();   // the chain kernel's start states
    if (!PHASE1 && has_c) {
      if (it.nseg > 1) {
        const float *src = r.X + ((static_cast<size_t>(x) * p.H + h) * DA + da0) * DC + dcr;
#pragma unroll
        for (int j = 0; j < SN / 2; ++j) S[j] = pair_f32(src[2 * j * DC], src[(2 * j + 1) * DC]);
      } else if (r.s0 && page >= 0) {
        const float *src = r.s0 + (static_cast<size_t>(page) * p.H + h) * DA * DC;
        if (r.s0_t) {
          const float4 *s4 = reinterpret_cast<const float4 *>(src + static_cast<size_t>(dcr) * DA + da0);
#pragma unroll
          for (int j = 0; j < SN / 4; ++j) {
            const float4 f = s4[j];
            S[2 * j] = pair_f32(f.x, f.y);
            S[2 * j + 1] = pair_f32(f.z, f.w);
          }
        } else {
          src += da0 * DC + dcr;
#pragma unroll
          for (int j = 0; j < SN / 2; ++j) S[j] = pair_f32(src[2 * j * DC], src[(2 * j + 1) * DC]);
        }
      }
    }
    const uint32_t lrow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    ChunkDecay decay;
    decay.init(pw[C], pw_lo[C]);
    auto store_operand = [&]() {   // S^T to tensor memory in bf16: columns da / 2
#pragma unroll
      for (int q = 0; q < SN / 32; ++q) {
        uint32_t u[16];
#pragma unroll
        for (int m = 0; m < 16; ++m) {
          float a, b;
          unpair_f32(S[16 * q + m], a, b);
          u[m] = pack_bf16x2(a, b);
        }
        tmem_st16(lrow + COL_S + half * (SN / 2) + 16 * q, u);
      }
      tmem_wait_st();
    };
    if (!PHASE1) store_operand();

    for (int i = 0; i < nch; ++i) {
      const uint32_t ph = i & 1;
      const int row0 = chunk_row(i), n = min(C, end - row0);
      uint8_t *bt = sm + OFF_B + TILE * ph;

      // 1. P with its decays, to bf16 (rows 16 quad .. of the M = 64 layout, columns 32 half ..)
      if (!PHASE1) {
        ok = __all_sync(0xffffffffu, wait_or_abort(bar_p, ph, abort));
        if (!ok) break;
        tc_fence_after();
        float v[16];
        tmem_ld_frag4(lrow + COL_P + 32 * half, v);
        tmem_wait_ld();
        uint32_t u[4][2];   // column groups of 8 x rows lane / 4 (+ 8)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int t = 16 * quad + (lane >> 2) + 8 * k, s = 32 * half + 8 * j + 2 * (lane & 3);
            float y[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int d = rev ? s + e - t : t - s - e;
              const float w = dtab[C + d];
              y[e] = d >= 0 && s + e < n ? v[4 * j + 2 * k + e] * w : 0.f;
            }
            u[j][k] = pack_bf16x2(y[0], y[1]);
          }
        const int t = 16 * quad + (lane & 15), ch = 4 * half + (lane >> 4);
        stmatrix4(smem_u32(sm + OFF_P + sw128(t, ch)), u[0][0], u[0][1], u[1][0], u[1][1]);
        stmatrix4(smem_u32(sm + OFF_P + sw128(t, ch + 2)), u[2][0], u[2][1], u[3][0], u[3][1]);
      }
      // 2. w b in bf16 terms; rows behind the sequence's end become zeros, in c too
      ok = __all_sync(0xffffffffu, wait_or_abort(bar_b + ph, (i >> 1) & 1, abort));
      if (!ok) break;
      {
        const int row = tid & 63, piece = tid >> 6;   // four threads per row
        if (row < n) {
          const float w = pw[rev ? row + 1 : n - 1 - row] * bscale;
          const uint64_t w2 = pair_f32(w, w), minus_one = pair_f32(-1.f, -1.f);
#pragma unroll UNROLL_W
          for (int jj = 0; jj < DA / 32; ++jj) {
            const int j = piece * (DA / 32) + jj;
            const uint32_t off = (j >> 3) * 8192 + sw128(row, j & 7);
            uint4 v = *reinterpret_cast<const uint4 *>(bt + off), mid, lo;
            split_pair(v.x, w2, minus_one, three, v.x, mid.x, lo.x);
            split_pair(v.y, w2, minus_one, three, v.y, mid.y, lo.y);
            split_pair(v.z, w2, minus_one, three, v.z, mid.z, lo.z);
            split_pair(v.w, w2, minus_one, three, v.w, mid.w, lo.w);
            *reinterpret_cast<uint4 *>(bt + off) = v;
            *reinterpret_cast<uint4 *>(sm + OFF_M + off) = mid;
            if (three) *reinterpret_cast<uint4 *>(sm + OFF_L + off) = lo;
          }
        }
        if (n < C) {
          ok = __all_sync(0xffffffffu, wait_or_abort(bar_c + (PHASE1 ? ph : 0), PHASE1 ? (i >> 1) & 1 : ph, abort));
          if (!ok) break;
          if (row >= n) {
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int jj = 0; jj < DA / 32; ++jj) {
              const int j = piece * (DA / 32) + jj;
              const uint32_t off = (j >> 3) * 8192 + sw128(row, j & 7);
              *reinterpret_cast<uint4 *>(bt + off) = zero;
              *reinterpret_cast<uint4 *>(sm + OFF_M + off) = zero;
              *reinterpret_cast<uint4 *>(sm + OFF_L + off) = zero;
            }
#pragma unroll
            for (int jj = 0; jj < DC / 32; ++jj) {
              const int j = piece * (DC / 32) + jj;
              *reinterpret_cast<uint4 *>(sm + (PHASE1 && ph ? OFF_A : OFF_C) + (j >> 3) * 8192 + sw128(row, j & 7)) = zero;
            }
          }
        }
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_ready);

      // 3. S <- lambda^n S + dS
      ok = __all_sync(0xffffffffu, wait_or_abort(bar_kv, ph, abort));
      if (!ok) break;
      tc_fence_after();
      {
        const float g = n == C ? decay.next() : pw[n];
        const uint64_t g2 = pair_f32(g, g);
#pragma unroll
        for (int q = 0; q < SN / 16; ++q) {
          float v[16];
          tmem_ld16(lrow + COL_DS + da0 + 16 * q, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e) S[8 * q + e] = fma_f32x2(g2, S[8 * q + e], pair_f32(v[2 * e], v[2 * e + 1]));
        }
      }
      tc_fence_before();   // dS^T is read before the next product overwrites it
      if (PHASE1) continue;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_ds);

      // 4. the output: this warp's 32 columns dc and 32 tokens t, through its 2 KB of
      // shared memory (rows t of 64 bytes, 16-byte chunks XOR-ed with t / 2) unless in fp32
      ok = __all_sync(0xffffffffu, wait_or_abort(bar_o, ph, abort));
      if (!ok) break;
      tc_fence_after();
      if (quad * 32 < DC) {
        uint8_t *stage = sm + OFF_M + 2048 * warp;
        const size_t y0 = ((static_cast<size_t>(it.b) * p.T + it.t0 + row0) * p.H + h) * DC + 32 * quad;
        const size_t ystep = static_cast<size_t>(p.H) * DC;
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) {   // 16 lanes of tensor memory x 16 columns: dc = 32 quad + 16 hh .., t = t0 ..
          const int hh = qq & 1, t0 = 32 * half + 16 * (qq >> 1);
          float v1[8], v2[8];
          const uint32_t at = lrow + (static_cast<uint32_t>(16 * hh) << 16) + t0;
          tmem_ld_frag2(at + COL_O1, v1);
          tmem_ld_frag2(at + COL_O2, v2);
          tmem_wait_ld();
          uint32_t u[2][2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int t = t0 + 8 * j + 2 * (lane & 3);
            const uint64_t g2 = pair_f32(yscale * pw[rev ? max(n - 1 - t, 0) : t + 1],
                                         yscale * pw[rev ? max(n - 2 - t, 0) : t + 2]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float ya, yb;
              unpair_f32(fma_f32x2(g2, pair_f32(v1[4 * j + 2 * k], v1[4 * j + 2 * k + 1]),
                                   pair_f32(v2[4 * j + 2 * k], v2[4 * j + 2 * k + 1])), ya, yb);
              if (y_f32) {
                float *y = static_cast<float *>(r.y) + y0 + 16 * hh + 8 * k + (lane >> 2);
                if (t < n) y[t * ystep] = ya;
                if (t + 1 < n) y[(t + 1) * ystep] = yb;
              } else {
                u[j][k] = pack_bf16x2(ya, yb);
              }
            }
          }
          if (!y_f32) {
            // matrix m: tokens t0 + 8 (m / 2) .., columns 16 hh + 8 (m & 1) ..; its row q = token
            const int tt = 16 * (qq >> 1) + 8 * (lane >> 4) + (lane & 7), ch = 2 * hh + ((lane >> 3) & 1);
            stmatrix4_trans(smem_u32(stage + tt * 64 + ((ch ^ (tt >> 1)) & 3) * 16), u[0][0], u[0][1], u[1][0], u[1][1]);
          }
        }
        if (!y_f32) {
          __syncwarp();
          __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(r.y) + y0 + 8 * (lane & 3);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int tt = 8 * k + (lane >> 2), t = 32 * half + tt;
            const uint4 v = *reinterpret_cast<const uint4 *>(stage + tt * 64 + (((lane & 3) ^ (tt >> 1)) & 3) * 16);
            if (t < n) *reinterpret_cast<uint4 *>(y + t * ystep) = v;
          }
        }
      }
      // the quad's two warps share its lanes: O2^T is read by both before S^T replaces it, and
      // the output rows lie where all warps write w b next
      tc_fence_before();
      named_bar_sync(1, 32 * NCOMPUTE);
      if (i + 1 < nch) store_operand();
    }
    float *dst = PHASE1 ? r.X + (static_cast<size_t>(x) * p.H + h) * DA * DC : final_page;
    if (dst && has_c && ok) {
      dst += da0 * DC + dcr;
#pragma unroll
      for (int j = 0; j < SN / 2; ++j) {
        float a, b;
        unpair_f32(S[j], a, b);
        dst[2 * j * DC] = a;
        dst[(2 * j + 1) * DC] = b;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

template <int DA, int DC, bool PHASE1>
cudaError_t launch(const LinProblem &p, const LinChunkMaps &maps, const LinRunSel &sel, bool pdl, cudaStream_t s) {
  auto kern = linear_chunk_kernel<DA, DC, PHASE1>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long>(p.items) * p.H * sel.n));
  cfg.blockDim = dim3(NTHREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p, maps, sel);
}

template <bool PHASE1>
cudaError_t launch_shape(int da, int dc, const LinProblem &p, const LinChunkMaps &m, const LinRunSel &sel, bool pdl,
                         cudaStream_t s) {
  if (da == 128 && dc == 128) return launch<128, 128, PHASE1>(p, m, sel, pdl, s);
  if (da == 128 && dc == 64) return launch<128, 64, PHASE1>(p, m, sel, pdl, s);
  if (da == 64 && dc == 128) return launch<64, 128, PHASE1>(p, m, sel, pdl, s);
  return launch<64, 64, PHASE1>(p, m, sel, pdl, s);
}

}  // namespace

// [B, T, heads, d] bf16 tensor with any batch, token and head strides: boxes of 64 (d) x 64 tokens.
static bool strided_map(CUtensorMap *m, const LinTensor &t, int B, int T, int heads, int d) {
  auto enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)t.sh * 2, (cuuint64_t)t.st * 2, (cuuint64_t)t.sb * 2};
  const cuuint32_t box[4] = {64, 1, 64, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(t.p), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc
}  // namespace gdr

bool gdr_linear_chunk_maps(const gdr::LinProblem &p, gdr::LinChunkMaps *maps) {
  bool done[4] = {};
  for (int i = 0; i < p.nrun; ++i) {
    const gdr::LinRun &r = p.run[i];
    const int idx[3] = {r.ia, r.ib, r.ic}, d[3] = {r.da, r.da, r.dc};
    for (int j = 0; j < 3; ++j) {
      if (done[idx[j]]) continue;
      const gdr::LinTensor &t = p.t[idx[j]];
      if (!gdr::tc::strided_map(&maps->m[idx[j]], t, p.B, p.T, p.H / t.div, d[j])) return false;
      done[idx[j]] = true;
    }
  }
  return true;
}

cudaError_t gdr_launch_linear_chunk(const gdr::LinProblem &p, const gdr::LinChunkMaps &maps, bool phase1, bool pdl,
                                    cudaStream_t s) {
  // one launch for all runs of a shape, so that they read their common tensors at about the same time
  bool done[gdr::kLinMaxRuns] = {};
  for (int i = 0; i < p.nrun; ++i) {
    if (done[i]) continue;
    gdr::LinRunSel sel = {};
    for (int j = i; j < p.nrun; ++j)
      if (!done[j] && p.run[j].da == p.run[i].da && p.run[j].dc == p.run[i].dc) {
        sel.run[sel.n++] = j;
        done[j] = true;
      }
    // a programmatic dependent waits for the one launch before it, so only the phase's first one may be it
    const cudaError_t e = phase1 ? gdr::tc::launch_shape<true>(p.run[i].da, p.run[i].dc, p, maps, sel, pdl && i == 0, s)
                                 : gdr::tc::launch_shape<false>(p.run[i].da, p.run[i].dc, p, maps, sel, pdl && i == 0, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

int gdr_linear_read_device_error(cudaStream_t stream) {
  int h = 0, zero = 0;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return -1;
  if (cudaMemcpyFromSymbol(&h, g_gdr_linear_error, sizeof(int)) != cudaSuccess) return -1;
  if (h) cudaMemcpyToSymbol(g_gdr_linear_error, &zero, sizeof(int));
  return h;
}
