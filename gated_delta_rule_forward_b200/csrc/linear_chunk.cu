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
// bf16 terms (24 bits, three MMAs): the state keeps fp32 accuracy.  P and S^T
// enter only Y, on disjoint parts of its sum, and are rounded once to bf16,
// like Y itself.
//
// Two CTAs share an SM (107 KB of shared memory, 256 tensor-memory columns, 128
// registers a thread each), so that one's copies, MMAs and register passes
// overlap the other's; within a CTA the steps follow one another.
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
constexpr int NTHREADS = 256;
constexpr uint32_t TILE = 16384;        // 64 rows of two 128-byte atoms
constexpr uint32_t OFF_A = 0;           // a (phase 1: the second c buffer)
constexpr uint32_t OFF_C = TILE;
constexpr uint32_t OFF_B = 2 * TILE;    // two buffers; the first term of w b replaces b in place
constexpr uint32_t OFF_M = 4 * TILE;    // second and third terms of w b; then each warp's 2 KB of output rows
constexpr uint32_t OFF_L = 5 * TILE;
constexpr uint32_t OFF_P = 6 * TILE;    // bf16 P, rows t, 8 KB
constexpr uint32_t OFF_PW = OFF_P + 8192;      // lambda^0 .. lambda^64, then what fp32 loses of them
constexpr uint32_t OFF_D = OFF_PW + 2 * 65 * 4 + 8;   // bscale lambda^d at 64 + d, zeros for d < 0
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

// Three bf16 terms of eight fp32 values (24 significant bits together), as 16-byte chunks.
__device__ __forceinline__ void split3(const float (&x)[8], uint4 &hi, uint4 &mid, uint4 &lo) {
  uint32_t h[4], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    const float r0 = x[2 * i] - __uint_as_float(h[i] << 16), r1 = x[2 * i + 1] - __uint_as_float(h[i] & 0xffff0000u);
    m[i] = pack_bf16x2(r0, r1);
    l[i] = pack_bf16x2(r0 - __uint_as_float(m[i] << 16), r1 - __uint_as_float(m[i] & 0xffff0000u));
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  mid = make_uint4(m[0], m[1], m[2], m[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

template <int DA, int DC, bool PHASE1>
__global__ void __launch_bounds__(NTHREADS, 2)
    linear_chunk_kernel(const __grid_constant__ LinProblem p, const __grid_constant__ LinChunkMaps maps,
                        const LinRunSel sel) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = warp & 3, half = warp >> 2;
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
  uint64_t *bar_a = reinterpret_cast<uint64_t *>(sm + OFF_BAR);
  uint64_t *bar_b = bar_a + 1;    // [2]
  uint64_t *bar_c = bar_a + 3;    // [2], the second one in phase 1 only
  uint64_t *bar_p = bar_a + 5, *bar_o1 = bar_a + 6, *bar_o = bar_a + 7, *bar_kv = bar_a + 8;
  uint64_t *bar_drain = bar_a + 9;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar_a + 10);
  volatile int *abort = reinterpret_cast<volatile int *>(bar_a + 11);

  if (warp == 0) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  if (tid == 32) {
    for (int i = 0; i < 10; ++i) mbar_init(bar_a + i, 1);
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
      dtab[C + m] = r.bscale * hi;
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
  auto chunk_row = [&](int i) { return beg + C * (rev ? nch - 1 - i : i); };
  const CUtensorMap *ma = &maps.m[r.ia], *mb = &maps.m[r.ib], *mc = &maps.m[r.ic];
  const int ha = h / p.t[r.ia].div, hb = h / p.t[r.ib].div, hc = h / p.t[r.ic].div;
  uint32_t issued_a = 0, issued_b = 0, issued_c = 0;   // copies (thread 0)
  auto load_a = [&](int i) {
    mbar_expect_tx(bar_a, DA * 128);
    for (int d = 0; d < DA / 64; ++d) tma_load_4d(sm + OFF_A + 8192 * d, ma, bar_a, 64 * d, ha, it.t0 + chunk_row(i), it.b);
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
  if (tid == 0 && nch > 0) {
    if (!PHASE1) load_a(0);
    load_b(0);
    load_c(0);
    if (nch > 1) {
      load_b(1);
      if (PHASE1) load_c(1);
    }
  }

  // ---- start state: thread (quad, lane, half) holds S[da = half DA/2 + j][dc = 32 quad + lane]
  constexpr int SN = DA / 2;
  const int dcr = 32 * quad + lane, da0 = half * SN;
  const bool has_c = dcr < DC;
  float S[SN];
#pragma unroll
  for (int j = 0; j < SN; ++j) S[j] = 0.f;
  const int page = lin_page(p, it.n);
  if (!PHASE1 && has_c) {
    griddep_wait();   // the chain kernel's start states
    if (it.nseg > 1) {
      const float *src = r.X + ((static_cast<size_t>(x) * p.H + h) * DA + da0) * DC + dcr;
#pragma unroll
      for (int j = 0; j < SN; ++j) S[j] = src[j * DC];
    } else if (r.s0 && page >= 0) {
      const float *src = r.s0 + (static_cast<size_t>(page) * p.H + h) * DA * DC;
      if (r.s0_t) {
        const float4 *s4 = reinterpret_cast<const float4 *>(src + static_cast<size_t>(dcr) * DA + da0);
#pragma unroll
        for (int j = 0; j < SN / 4; ++j) {
          const float4 f = s4[j];
          S[4 * j] = f.x; S[4 * j + 1] = f.y; S[4 * j + 2] = f.z; S[4 * j + 3] = f.w;
        }
      } else {
        src += da0 * DC + dcr;
#pragma unroll
        for (int j = 0; j < SN; ++j) S[j] = src[j * DC];
      }
    }
  } else if (!has_c || PHASE1) {
    griddep_wait();
  }
  const uint32_t lrow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
  auto store_operand = [&]() {   // S^T to tensor memory in bf16: columns da / 2
#pragma unroll
    for (int q = 0; q < SN / 32; ++q) {
      uint32_t u[16];
#pragma unroll
      for (int m = 0; m < 16; ++m) u[m] = pack_bf16x2(S[32 * q + 2 * m], S[32 * q + 2 * m + 1]);
      tmem_st16(lrow + COL_S + half * (SN / 2) + 16 * q, u);
    }
    tmem_wait_st();
  };
  auto issue_p = [&]() {   // P = a b^T of the chunk in the a and b buffers
    return [&](int i) {
      const uint32_t a = smem_u32(sm + OFF_A), b = smem_u32(sm + OFF_B + TILE * (i & 1));
#pragma unroll
      for (int kk = 0; kk < DA / 16; ++kk) {
        const uint32_t o = (kk >> 2) * 8192 + (kk & 3) * 32;
        mma_ss(tmem + COL_P, sdesc(a + o, 16, 1024), sdesc(b + o, 16, 1024), idesc_bf16(C, C, false, false), kk > 0);
      }
      mma_commit(bar_p);
    };
  }();

  bool ok = true;
  if (!PHASE1) {
    store_operand();
    if (tid == 0 && nch > 0) {
      ok = wait_or_abort(bar_a, 0, abort) && wait_or_abort(bar_b, 0, abort);
      if (ok) issue_p(0);
    }
    __syncwarp();
  }

  bool bad = false;
  for (int i = 0; i < nch; ++i) {
    const uint32_t ph = i & 1;
    const int row0 = chunk_row(i), n = min(C, end - row0);
    uint8_t *bt = sm + OFF_B + TILE * (i & 1);
    const uint32_t ct_off = PHASE1 && (i & 1) ? OFF_A : OFF_C;
    const int cbuf = PHASE1 ? i & 1 : 0;
    const uint32_t cph = PHASE1 ? (i >> 1) & 1 : ph;

    // 1. P with its decays, to bf16 (rows 16 quad + lane of the M = 64 layout)
    if (!PHASE1) {
      ok = ok && wait_or_abort(bar_p, ph, abort);
      ok = __all_sync(0xffffffffu, ok);
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
    // 2. w b in three bf16 terms; rows behind the sequence's end become zeros, in c too
    ok = ok && wait_or_abort(bar_b + (i & 1), (i >> 1) & 1, abort);
    {
      const int row = tid & 63, part = tid >> 6;
      const float w = row < n ? pw[rev ? row + 1 : n - 1 - row] * r.bscale : 0.f;
#pragma unroll
      for (int jj = 0; jj < DA / 32; ++jj) {
        const int j = part * (DA / 32) + jj;
        const uint32_t off = (j >> 3) * 8192 + sw128(row, j & 7);
        float f[8];
        unpack8(*reinterpret_cast<const uint4 *>(bt + off), f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = row < n ? f[e] * w : 0.f;
        uint4 hi, mid, lo;
        split3(f, hi, mid, lo);
        *reinterpret_cast<uint4 *>(bt + off) = hi;
        *reinterpret_cast<uint4 *>(sm + OFF_M + off) = mid;
        *reinterpret_cast<uint4 *>(sm + OFF_L + off) = lo;
      }
      if (n < C) {
        ok = ok && wait_or_abort(bar_c + cbuf, cph, abort);
        if (row >= n)
#pragma unroll
          for (int jj = 0; jj < DC / 32; ++jj) {
            const int j = part * (DC / 32) + jj;
            *reinterpret_cast<uint4 *>(sm + ct_off + (j >> 3) * 8192 + sw128(row, j & 7)) = make_uint4(0u, 0u, 0u, 0u);
          }
      }
    }
    fence_async_smem();
    tc_fence_before();
    if ((bad = __syncthreads_or(!ok))) break;

    // 3. O1^T = S^T a^T, O2^T = c^T P^T and dS^T = c^T (w b)
    if (tid == 0) {
      tc_fence_after();
      const uint32_t ct = smem_u32(sm + ct_off);
      if (!PHASE1) {
        const uint32_t a = smem_u32(sm + OFF_A);
#pragma unroll
        for (int kk = 0; kk < DA / 16; ++kk)
          mma_ts(tmem + COL_O1, tmem + COL_S + 8 * kk, sdesc(a + (kk >> 2) * 8192 + (kk & 3) * 32, 16, 1024),
                 idesc_bf16(128, C, false, false), kk > 0);
        mma_commit(bar_o1);
      }
      ok = wait_or_abort(bar_c + cbuf, cph, abort);
      if (ok) {
        const uint32_t part[3] = {smem_u32(bt), smem_u32(sm + OFF_M), smem_u32(sm + OFF_L)};
#pragma unroll
        for (int t = 0; t < 3; ++t)
#pragma unroll
          for (int kk = 0; kk < C / 16; ++kk)
            mma_ss(tmem + COL_DS, sdesc(ct + kk * 2048, 8192, 1024), sdesc(part[t] + kk * 2048, 8192, 1024),
                   idesc_bf16(128, DA, true, true), t + kk > 0);
        mma_commit(bar_kv);
      }
      // O2^T goes where S^T was read from: once O1^T is complete, while dS^T is under way
      if (!PHASE1 && ok && (ok = wait_or_abort(bar_o1, ph, abort))) {
        const uint32_t pt = smem_u32(sm + OFF_P);
#pragma unroll
        for (int kk = 0; kk < C / 16; ++kk)
          mma_ss(tmem + COL_O2, sdesc(ct + kk * 2048, 8192, 1024), sdesc(pt + kk * 32, 16, 1024),
                 idesc_bf16(128, C, true, false), kk > 0);
        mma_commit(bar_o);
      }
    }
    __syncwarp();

    // 4. S <- lambda^n S + dS
    ok = ok && wait_or_abort(bar_kv, ph, abort);
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
    if (tid == 0 && ok) {
      if (i + 2 < nch) {
        load_b(i + 2);
        if (PHASE1) load_c(i + 2);
      }
      if (!PHASE1 && i + 1 < nch) load_a(i + 1);
    }
    __syncwarp();
    {
      const float g = pw[n], gl = pw_lo[n];
#pragma unroll
      for (int q = 0; q < SN / 32; ++q) {
        float v[32];
        tmem_ld32(lrow + COL_DS + da0 + 32 * q, v);
#pragma unroll
        for (int e = 0; e < 32; ++e) S[32 * q + e] = fmaf(g, S[32 * q + e], fmaf(gl, S[32 * q + e], v[e]));
      }
    }
    if (PHASE1) {
      tc_fence_before();   // dS^T is read before the next chunk's product overwrites it
      continue;
    }

    // 5. the output: this warp's 32 columns dc and 32 tokens t, through its 2 KB of
    // shared memory (rows t of 64 bytes, 16-byte chunks XOR-ed with t / 2) unless in fp32
    ok = ok && wait_or_abort(bar_o, ph, abort);
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
    if (tid == 0 && ok && i + 1 < nch) load_c(i + 1);
    __syncwarp();
    if (quad * 32 < DC) {
      uint8_t *stage = sm + OFF_M + 2048 * warp;
      const size_t y0 = ((static_cast<size_t>(it.b) * p.T + it.t0 + row0) * p.H + h) * DC + 32 * quad;
      const size_t ystep = static_cast<size_t>(p.H) * DC;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {   // 16 lanes of tensor memory: dc = 32 quad + 16 hh ..
        float v1[16], v2[16];
        const uint32_t at = lrow + (static_cast<uint32_t>(16 * hh) << 16) + 32 * half;
        tmem_ld_frag4(at + COL_O1, v1);
        tmem_ld_frag4(at + COL_O2, v2);
        tmem_wait_ld();
        uint32_t u[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = 32 * half + 8 * j + 2 * (lane & 3);
          const float g0 = pw[rev ? max(n - 1 - t, 0) : t + 1], g1 = pw[rev ? max(n - 2 - t, 0) : t + 2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float y0v = r.yscale * fmaf(g0, v1[4 * j + 2 * k], v2[4 * j + 2 * k]);
            const float y1v = r.yscale * fmaf(g1, v1[4 * j + 2 * k + 1], v2[4 * j + 2 * k + 1]);
            if (r.y_f32) {
              float *y = static_cast<float *>(r.y) + y0 + 16 * hh + 8 * k + (lane >> 2);
              if (t < n) y[t * ystep] = y0v;
              if (t + 1 < n) y[(t + 1) * ystep] = y1v;
            } else {
              u[j][k] = pack_bf16x2(y0v, y1v);
            }
          }
        }
        if (!r.y_f32) {
          // matrix m: tokens 8 (j + m / 2) .., columns 16 hh + 8 (m & 1) ..; row q = token
          const int t = 8 * (lane >> 4) + (lane & 7), ch = 2 * hh + ((lane >> 3) & 1);
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const int tt = 8 * j + t;
            stmatrix4_trans(smem_u32(stage + tt * 64 + ((ch ^ (tt >> 1)) & 3) * 16), u[j][0], u[j][1], u[j + 1][0],
                            u[j + 1][1]);
          }
        }
      }
      if (!r.y_f32) {
        __syncwarp();
        __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(r.y) + y0 + 8 * (lane & 3);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int tt = 8 * k + (lane >> 2), t = 32 * half + tt;
          const uint4 row = *reinterpret_cast<const uint4 *>(stage + tt * 64 + (((lane & 3) ^ (tt >> 1)) & 3) * 16);
          if (t < n) *reinterpret_cast<uint4 *>(y + t * ystep) = row;
        }
      }
    }
    tc_fence_before();
    if ((bad = __syncthreads_or(!ok))) break;
    if (tid == 0 && i + 1 < nch) {
      tc_fence_after();
      ok = wait_or_abort(bar_a, (i + 1) & 1, abort) && wait_or_abort(bar_b + ((i + 1) & 1), ((i + 1) >> 1) & 1, abort);
      if (ok) issue_p(i + 1);
    }
    __syncwarp();
    if (i + 1 < nch) store_operand();
  }

  bad = __syncthreads_or(bad || !ok);
  if (bad) {
    if (tid == 0) {
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
  } else {
    float *dst = nullptr;
    if (PHASE1) dst = r.X + (static_cast<size_t>(x) * p.H + h) * DA * DC;
    else if (last && r.s_final && page >= 0) dst = r.s_final + (static_cast<size_t>(page) * p.H + h) * DA * DC;
    if (dst && has_c) {
      dst += da0 * DC + dcr;
#pragma unroll
      for (int j = 0; j < SN; ++j) dst[j * DC] = S[j];
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
