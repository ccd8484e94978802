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
//     dS^T [dc][da] = c^T (w b)      M128 N = da, K = 64
//     O1^T [dc][t]  = S^T a^T        M128 N64  K = da   (S^T in bf16 in tensor memory)
//     O2^T [dc][t]  = c^T P^T        M128 N64  K = 64   (P back through shared memory in bf16)
// and Y^T = yscale (Gamma_t O1^T + O2^T).  The fp32 state lives in registers of
// 16 warps: lane dc of a quad, a quarter of da per thread; S <- lambda^n S + dS
// is one pass over it.
//
// Rounding.  The products' inputs are exact bf16 except three: w b, P and the
// S^T operand.  w b enters the state, which is fp32, so it is split into three
// bf16 terms (24 bits, three MMAs): the state keeps fp32 accuracy; where the
// state is not kept (a later segment starts from phase 1's), two terms do, 2^-8
// of what follows.  P and S^T enter only Y, on disjoint parts of its sum, and
// are rounded once to bf16, like Y itself.
//
// One CTA has the SM.  Its warps are specialised and hand over through
// mbarriers, so that three chunks are under way at once:
//     copies (1 warp)    a, b, c of the chunks to come, each into the stage of one that is done
//     prep   (8 warps)   P and w b of chunk i + 1
//     MMAs   (1 warp)    dS(i), P(i + 1), O1(i), O2(i)
//     finish (16 warps)  S after chunk i, its bf16 operand, the output rows of chunk i
// Only S -> operand -> O1 is a chain from chunk to chunk.
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
constexpr int NFINISH = 16, NPREP = 8;   // warps 0 .. 15 and 16 .. 23, then the MMA and the copy warp
constexpr int NTHREADS = 32 * (NFINISH + NPREP + 2);
constexpr uint32_t TILE = 16384;        // 64 rows of two 128-byte atoms
// Shared memory.  The copies run NST chunks ahead; what is made of a chunk has two
// buffers (the third term of w b, with all runs' tensors in flight, one).
template <bool PHASE1>
struct Smem {
  static constexpr int NST = PHASE1 ? 4 : 3;
  static constexpr uint32_t B = 0;               // in a stage: b; the first term of w b replaces it in place
  static constexpr uint32_t CT = TILE;
  static constexpr uint32_t A = 2 * TILE;
  static constexpr uint32_t STAGE = (PHASE1 ? 2 : 3) * TILE;
  static constexpr uint32_t M = NST * STAGE;     // second term of w b, two buffers
  static constexpr uint32_t L = M + 2 * TILE;    // third term
  static constexpr int NL = PHASE1 ? 2 : 1;
  static constexpr uint32_t P = L + NL * TILE;   // bf16 P, rows t, 8 KB, two buffers
  static constexpr uint32_t Y = P + (PHASE1 ? 0 : 2 * 8192);      // 1 KB of output rows per finishing warp
  static constexpr uint32_t PW = Y + (PHASE1 ? 0 : 1024 * NFINISH);   // lambda^0 .. lambda^64, then what fp32 loses of them
  static constexpr uint32_t BAR = PW + 2 * 65 * 4 + 8;
  static constexpr uint32_t BYTES = BAR + 208 + 1024;
  static_assert(BAR % 16 == 0 && P % 1024 == 0 && BYTES <= 232448, "one CTA per SM");
};
constexpr uint32_t COL_DS = 0;     // dS^T, 128 columns
constexpr uint32_t COL_S = 128;    // S^T in bf16, 64 columns
constexpr uint32_t COL_P = 192;    // P, 64 columns
constexpr uint32_t COL_O = 256;    // two buffers of O1^T and O2^T, 64 columns each
constexpr uint32_t TMEM_COLS = 512;

// Shared-memory matrix descriptors (sdesc()) in halves: `lo` of an address is followed by
// that of an address o bytes on at + o / 16, so that the one thread that issues the MMAs
// spends one addition on each (built from scratch they took it 100 cycles an MMA).
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);   // sbo 1024, version 1, SWIZZLE_128B
template <bool ACC>
__device__ __forceinline__ void mma_ss_lo(uint32_t d_tmem, uint32_t alo, uint32_t blo, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(alo), "r"(blo), "r"(idesc), "n"(ACC ? 1 : 0), "r"(DESC_HI)
      : "memory");
}
template <bool ACC>
__device__ __forceinline__ void mma_ts_lo(uint32_t d_tmem, uint32_t a_tmem, uint32_t blo, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(blo), "r"(idesc), "n"(ACC ? 1 : 0), "r"(DESC_HI)
      : "memory");
}
// D (+)= A B over K steps of 16, A and B advancing by ao and bo bytes a step; steps
// 4 .. 7 of a K-major operand lie in the next atom, 8 KB on.
template <int STEPS, bool ACC0, bool A_ATOMS, bool B_ATOMS>
__device__ __forceinline__ void mma_ss_steps(uint32_t d, uint32_t alo, uint32_t ao, uint32_t blo, uint32_t bo,
                                             uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < STEPS; ++kk) {
    const uint32_t a = alo + (A_ATOMS ? (kk >> 2) * 512 + (kk & 3) * (ao / 16) : kk * (ao / 16));
    const uint32_t b = blo + (B_ATOMS ? (kk >> 2) * 512 + (kk & 3) * (bo / 16) : kk * (bo / 16));
    if (kk == 0) mma_ss_lo<ACC0>(d, a, b, idesc);
    else mma_ss_lo<true>(d, a, b, idesc);
  }
}

// Waits in the barrier's own time limit (about a millisecond), which leaves the issue
// slots to the other warps; a loop of short ones took more of them than the arithmetic.
__device__ __forceinline__ bool try_wait_long(uint64_t *bar, uint32_t phase) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000000;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(phase)
      : "memory");
  return ok != 0;
}
// Bounded wait (a second or so) that also gives up once another thread has.
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t phase, volatile int *abort) {
  if (try_wait_long(bar, phase)) return true;
  const long long start = clock64();
  while (!try_wait_long(bar, phase)) {
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
__global__ void __launch_bounds__(NTHREADS, 1)
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

  using M = Smem<PHASE1>;
  constexpr int NST = M::NST;
  float *pw = reinterpret_cast<float *>(sm + M::PW), *pw_lo = pw + 65;
  // per stage (chunk i: barrier i % NST, phase (i / NST) & 1)
  uint64_t *bar_load = reinterpret_cast<uint64_t *>(sm + M::BAR);   // a, b and c landed
  uint64_t *bar_free = bar_load + 4;     // every MMA that reads them complete
  // per buffer (chunk i: barrier i & 1, phase (i >> 1) & 1)
  uint64_t *bar_ready = bar_load + 8;    // P and w b written (8 warps)
  uint64_t *bar_kv = bar_load + 10;      // dS^T formed
  uint64_t *bar_o = bar_load + 12;       // O1^T and O2^T formed
  uint64_t *bar_oread = bar_load + 14;   // and read (16 warps)
  // one each (chunk i: phase i & 1)
  uint64_t *bar_p = bar_load + 16;       // P formed
  uint64_t *bar_ds = bar_load + 17;      // dS^T read (16 warps)
  uint64_t *bar_s = bar_load + 18;       // S^T of the chunk's start in tensor memory (16 warps)
  uint64_t *bar_drain = bar_load + 19;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar_load + 20);
  volatile int *abort = reinterpret_cast<volatile int *>(bar_load + 21);

  if (warp == 0) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  if (tid == 32) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(bar_load + i, 1);
      mbar_init(bar_free + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_ready + i, NPREP);
      mbar_init(bar_kv + i, 1);
      mbar_init(bar_o + i, 1);
      mbar_init(bar_oread + i, NFINISH);
    }
    mbar_init(bar_p, 1);
    mbar_init(bar_ds, NFINISH);
    mbar_init(bar_s, NFINISH);
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
  }
  // value widths of 64: the upper 64 lanes of the M = 128 products read zeros
  if (DC == 64)
    for (int i = tid; i < 512 * NST; i += NTHREADS)
      reinterpret_cast<uint4 *>(sm + M::STAGE * (i >> 9) + M::CT + 8192)[i & 511] = make_uint4(0u, 0u, 0u, 0u);
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

  if (warp == NFINISH + NPREP + 1) {
    // ---------------------------------------------------------------- copies
    if (lane == 0) {
      const CUtensorMap *ma = &maps.m[r.ia], *mb = &maps.m[r.ib], *mc = &maps.m[r.ic];
      const int ha = h / p.t[r.ia].div, hb = h / p.t[r.ib].div, hc = h / p.t[r.ic].div;
      constexpr uint32_t bytes = (PHASE1 ? 0 : DA * 128) + DA * 128 + DC * 128;
      int i = 0;
      for (; i < nch; ++i) {
        const int st = i % NST, row = it.t0 + chunk_row(i);
        uint8_t *dst = sm + M::STAGE * st;
        if (i >= NST && !wait_or_abort(bar_free + st, (i / NST - 1) & 1, abort)) break;
        mbar_expect_tx(bar_load + st, bytes);
        for (int d = 0; d < DA / 64; ++d) {
          tma_load_4d(dst + M::B + 8192 * d, mb, bar_load + st, 64 * d, hb, row, it.b);
          if (!PHASE1) tma_load_4d(dst + M::A + 8192 * d, ma, bar_load + st, 64 * d, ha, row, it.b);
        }
        for (int d = 0; d < DC / 64; ++d) tma_load_4d(dst + M::CT + 8192 * d, mc, bar_load + st, 64 * d, hc, row, it.b);
        if (i + NST < nch) {   // and the chunk that comes into this stage next, as far as L2
          const int ahead = it.t0 + chunk_row(i + NST);
          for (int d = 0; d < DA / 64; ++d) {
            tma_prefetch_4d(mb, 64 * d, hb, ahead, it.b);
            if (!PHASE1) tma_prefetch_4d(ma, 64 * d, ha, ahead, it.b);
          }
          for (int d = 0; d < DC / 64; ++d) tma_prefetch_4d(mc, 64 * d, hc, ahead, it.b);
        }
      }
      // nothing may land in shared memory after the CTA (each wait bounded)
      for (int j = i > NST ? i - NST : 0; j < i; ++j) mbar_wait(bar_load + j % NST, (j / NST) & 1);
    }
  } else if (warp == NFINISH + NPREP) {
    // ---------------------------------------------------------------- MMAs
    if (lane == 0) {
      const uint32_t base = smem_u32(sm);
      bool ok = true;
      auto issue_p = [&](int i) -> bool {   // P = a b^T once both landed
        if (!wait_or_abort(bar_load + i % NST, (i / NST) & 1, abort)) return false;
        const uint32_t sb = base + M::STAGE * (i % NST);
        mma_ss_steps<DA / 16, false, true, true>(tmem + COL_P, desc_lo(sb + M::A, 16), 32, desc_lo(sb + M::B, 16), 32,
                                                 idesc_bf16(C, C, false, false));
        mma_commit(bar_p);
        return true;
      };
      if (!PHASE1 && nch > 0) ok = issue_p(0);
      for (int i = 0; ok && i < nch; ++i) {
        const int st = i % NST, bf = i & 1;
        const uint32_t bph = (i >> 1) & 1, sb = base + M::STAGE * st;
        const uint32_t clo = desc_lo(sb + M::CT, 8192);
        // dS^T = c^T (w b)
        if (!(ok = wait_or_abort(bar_load + st, (i / NST) & 1, abort) && wait_or_abort(bar_ready + bf, bph, abort))) break;
        if (i > 0 && !(ok = wait_or_abort(bar_ds, (i - 1) & 1, abort))) break;
        tc_fence_after();
        constexpr uint32_t id_kv = idesc_bf16(128, DA, true, true);
        mma_ss_steps<C / 16, false, false, false>(tmem + COL_DS, clo, 2048, desc_lo(sb + M::B, 8192), 2048, id_kv);
        mma_ss_steps<C / 16, true, false, false>(tmem + COL_DS, clo, 2048, desc_lo(base + M::M + TILE * bf, 8192), 2048,
                                                 id_kv);
        if (three)
          mma_ss_steps<C / 16, true, false, false>(tmem + COL_DS, clo, 2048,
                                                   desc_lo(base + M::L + TILE * (i % M::NL), 8192), 2048, id_kv);
        mma_commit(bar_kv + bf);
        if (PHASE1) {
          mma_commit(bar_free + st);
          continue;
        }
        // the next chunk's P (this one's has been read)
        if (i + 1 < nch && !(ok = issue_p(i + 1))) break;
        // O1^T = S^T a^T, O2^T = c^T P^T
        if (!(ok = wait_or_abort(bar_s, i & 1, abort))) break;
        if (i >= 2 && !(ok = wait_or_abort(bar_oread + bf, ((i - 2) >> 1) & 1, abort))) break;
        tc_fence_after();
        const uint32_t co = tmem + COL_O + 128 * bf, alo = desc_lo(sb + M::A, 16);
#pragma unroll
        for (int kk = 0; kk < DA / 16; ++kk) {
          const uint32_t a = alo + (kk >> 2) * 512 + (kk & 3) * 2;
          if (kk == 0) mma_ts_lo<false>(co, tmem + COL_S, a, idesc_bf16(128, C, false, false));
          else mma_ts_lo<true>(co, tmem + COL_S + 8 * kk, a, idesc_bf16(128, C, false, false));
        }
        mma_ss_steps<C / 16, false, false, false>(co + 64, clo, 2048, desc_lo(base + M::P + 8192 * bf, 16), 32,
                                                  idesc_bf16(128, C, true, false));
        mma_commit(bar_o + bf);
        mma_commit(bar_free + st);
      }
      if (!ok) {   // a wait gave up: the MMAs in flight finish before the memory they use is released
        mma_commit(bar_drain);
        mbar_wait(bar_drain, 0);
      }
    }
  } else if (warp >= NFINISH) {
    // ---------------------------------------------------------------- prep: P and w b
    const int quad = warp & 3, half = (warp - NFINISH) >> 2;
    const int row = tid & 63, piece = (tid >> 6) & 3;   // w b: four threads per row
    const float bscale = r.bscale;
    const uint32_t lrow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    // P: rows t = 16 quad + lane / 4 (+ 8), columns s = 32 half + 8 j + 2 (lane % 4) (+ 1); the decays
    // are the same for every chunk
    uint64_t dec[4][2];
    if (!PHASE1) {
      const float f = bscale * r.yscale;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int t = 16 * quad + (lane >> 2) + 8 * k, s = 32 * half + 8 * j + 2 * (lane & 3);
          const int d = rev ? s - t : t - s, d1 = rev ? d + 1 : d - 1;
          dec[j][k] = pair_f32(d >= 0 ? f * pw[max(d, 0)] : 0.f, d1 >= 0 ? f * pw[max(d1, 0)] : 0.f);
        }
    }
    const uint64_t minus_one = pair_f32(-1.f, -1.f);
    for (int i = 0; i < nch; ++i) {
      const int st = i % NST, bf = i & 1;
      uint8_t *sb = sm + M::STAGE * st, *mid_t = sm + M::M + TILE * bf, *lo_t = sm + M::L + TILE * (i % M::NL);
      const int n = min(C, end - chunk_row(i));
      if (!__all_sync(0xffffffffu, wait_or_abort(bar_load + st, (i / NST) & 1, abort))) break;
      // this chunk's buffers are those of the products of two chunks ago (a single third-term buffer: of
      // the last one), which P's and b's arrival do not imply
      if (i >= 2 && !__all_sync(0xffffffffu, wait_or_abort((PHASE1 ? bar_kv : bar_o) + bf, ((i - 2) >> 1) & 1, abort))) break;
      if (M::NL == 1 && three && i >= 1 &&
          !__all_sync(0xffffffffu, wait_or_abort(bar_kv + (bf ^ 1), ((i - 1) >> 1) & 1, abort))) break;
      if (!PHASE1) {
        if (!__all_sync(0xffffffffu, wait_or_abort(bar_p, i & 1, abort))) break;
        tc_fence_after();
        float v[16];
        tmem_ld_frag4(lrow + COL_P + 32 * half, v);
        tmem_wait_ld();
        uint32_t u[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float y0, y1;
            unpair_f32(mul_f32x2(pair_f32(v[4 * j + 2 * k], v[4 * j + 2 * k + 1]), dec[j][k]), y0, y1);
            if (n < C) {   // whatever lies behind the sequence's end has no part in this
              const int s = 32 * half + 8 * j + 2 * (lane & 3);
              y0 = s < n ? y0 : 0.f;
              y1 = s + 1 < n ? y1 : 0.f;
            }
            u[j][k] = pack_bf16x2(y0, y1);
          }
        const int t = 16 * quad + (lane & 15), ch = 4 * half + (lane >> 4);
        stmatrix4(smem_u32(sm + M::P + 8192 * bf + sw128(t, ch)), u[0][0], u[0][1], u[1][0], u[1][1]);
        stmatrix4(smem_u32(sm + M::P + 8192 * bf + sw128(t, ch + 2)), u[2][0], u[2][1], u[3][0], u[3][1]);
      }
      if (row < n) {
        const float w = pw[rev ? row + 1 : n - 1 - row] * bscale;
        const uint64_t w2 = pair_f32(w, w);
#pragma unroll
        for (int jj = 0; jj < DA / 32; ++jj) {
          const int j = piece * (DA / 32) + jj;
          const uint32_t off = (j >> 3) * 8192 + sw128(row, j & 7);
          uint4 v = *reinterpret_cast<const uint4 *>(sb + M::B + off), mid, lo;
          split_pair(v.x, w2, minus_one, three, v.x, mid.x, lo.x);
          split_pair(v.y, w2, minus_one, three, v.y, mid.y, lo.y);
          split_pair(v.z, w2, minus_one, three, v.z, mid.z, lo.z);
          split_pair(v.w, w2, minus_one, three, v.w, mid.w, lo.w);
          *reinterpret_cast<uint4 *>(sb + M::B + off) = v;
          *reinterpret_cast<uint4 *>(mid_t + off) = mid;
          if (three) *reinterpret_cast<uint4 *>(lo_t + off) = lo;
        }
      } else {   // rows behind the sequence's end: zeros, in c too
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int jj = 0; jj < DA / 32; ++jj) {
          const int j = piece * (DA / 32) + jj;
          const uint32_t off = (j >> 3) * 8192 + sw128(row, j & 7);
          *reinterpret_cast<uint4 *>(sb + M::B + off) = zero;
          *reinterpret_cast<uint4 *>(mid_t + off) = zero;
          *reinterpret_cast<uint4 *>(lo_t + off) = zero;
        }
#pragma unroll
        for (int jj = 0; jj < DC / 32; ++jj) {
          const int j = piece * (DC / 32) + jj;
          *reinterpret_cast<uint4 *>(sb + M::CT + (j >> 3) * 8192 + sw128(row, j & 7)) = zero;
        }
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_ready + bf);
    }
  } else {
    // ---------------------------------------------------------------- finish: the state and the outputs
    const int quad = warp & 3, part = warp >> 2;
    // thread (quad, lane, part) holds S[da = part DA/4 + j][dc = 32 quad + lane], in pairs along da
    constexpr int SN = DA / 4;
    const int dcr = 32 * quad + lane, da0 = part * SN;
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
    auto store_operand = [&]() {   // S^T to tensor memory in bf16 (columns da / 2), and the hand-over
      uint32_t u[SN / 2];
#pragma unroll
      for (int m = 0; m < SN / 2; ++m) {
        float a, b;
        unpair_f32(S[m], a, b);
        u[m] = pack_bf16x2(a, b);
      }
      if constexpr (SN == 32) tmem_st16(lrow + COL_S + part * 16, u);
      else tmem_st8(lrow + COL_S + part * 8, u);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_s);
    };
    if (!PHASE1) store_operand();
    // the output: this warp's 32 columns dc and 16 tokens t, through its 1 KB of shared
    // memory (rows t of 64 bytes, 16-byte chunks XOR-ed with t / 2) unless in fp32.
    // Fragment tiles: lane holds dc = 16 hh + lane / 4 (+ 8), t = 8 j + 2 (lane % 4) (+ 1).
    const bool has_y = !PHASE1 && quad * 32 < DC, y_f32 = r.y_f32 != 0;
    const float yscale = r.yscale;
    const size_t ystep = static_cast<size_t>(p.H) * DC;
    const int tf = 16 * part + 2 * (lane & 3), tr = 16 * part + (lane >> 2);
    const uint32_t stage = smem_u32(sm + M::Y + 1024 * warp);
    // stmatrix: matrix m = tokens 8 (m / 2) .., columns 8 (m & 1) ..; its row q = token
    const int tq = 8 * (lane >> 4) + (lane & 7), cq = (lane >> 3) & 1;
    const uint32_t put0 = stage + tq * 64 + (((cq ^ (tq >> 1)) & 3) << 4), put1 = stage + tq * 64 + ((((2 + cq) ^ (tq >> 1)) & 3) << 4);
    const uint32_t get = stage + (lane >> 2) * 64 + ((((lane & 3) ^ (lane >> 3)) & 3) << 4);   // and 512 bytes on: token + 8
    // row tr's address in this chunk, advanced chunk by chunk; full chunks' decays
    uint8_t *yrow = nullptr;
    const long long yadvance = (rev ? -C : C) * static_cast<long long>(ystep) * (y_f32 ? 4 : 2);
    uint64_t gam[2] = {0, 0};
    auto gamma = [&](int n, uint64_t (&g)[2]) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = tf + 8 * j;
        g[j] = pair_f32(yscale * pw[rev ? max(n - 1 - t, 0) : t + 1], yscale * pw[rev ? max(n - 2 - t, 0) : t + 2]);
      }
    };
    if (has_y && nch > 0) {
      const size_t row = static_cast<size_t>(it.b) * p.T + it.t0 + chunk_row(0);
      if (y_f32) yrow = reinterpret_cast<uint8_t *>(static_cast<float *>(r.y) + (row + tf) * ystep + h * DC + 32 * quad + (lane >> 2));
      else yrow = reinterpret_cast<uint8_t *>(static_cast<__nv_bfloat16 *>(r.y) + (row + tr) * ystep + h * DC + 32 * quad + 8 * (lane & 3));
      gamma(C, gam);
    }
    bool ok = true;
    for (int i = 0; i < nch; ++i) {
      const int bf = i & 1;
      const uint32_t bph = (i >> 1) & 1;
      const int n = min(C, end - chunk_row(i));
      // S <- lambda^n S + dS
      if (!(ok = __all_sync(0xffffffffu, wait_or_abort(bar_kv + bf, bph, abort)))) break;
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
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_ds);
      if (PHASE1) continue;

      // its operand for the next chunk, once O1^T has been formed from this one's
      if (!(ok = __all_sync(0xffffffffu, wait_or_abort(bar_o + bf, bph, abort)))) break;
      tc_fence_after();
      if (i + 1 < nch) store_operand();
      if (!has_y) {
        if (lane == 0) mbar_arrive(bar_oread + bf);
        continue;
      }
      if (n < C) gamma(n, gam);
      const uint32_t col = lrow + COL_O + 128 * bf + 16 * part;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {   // 16 lanes of tensor memory: dc = 32 quad + 16 hh ..
        float v1[8], v2[8];
        const uint32_t at = col + (static_cast<uint32_t>(16 * hh) << 16);
        tmem_ld_frag2(at, v1);
        tmem_ld_frag2(at + 64, v2);
        tmem_wait_ld();
        if (hh == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_oread + bf);
        }
        uint64_t y[2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            y[j][k] = fma_f32x2(gam[j], pair_f32(v1[4 * j + 2 * k], v1[4 * j + 2 * k + 1]),
                                pair_f32(v2[4 * j + 2 * k], v2[4 * j + 2 * k + 1]));
        float a, b;
        if (y_f32) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float *dst = reinterpret_cast<float *>(yrow) + 8 * j * ystep + 16 * hh + 8 * k;
              unpair_f32(y[j][k], a, b);
              if (tf + 8 * j < n) dst[0] = a;
              if (tf + 8 * j + 1 < n) dst[ystep] = b;
            }
        } else {
          uint32_t u[2][2];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              unpair_f32(y[j][k], a, b);
              u[j][k] = pack_bf16x2(a, b);
            }
          stmatrix4_trans(hh ? put1 : put0, u[0][0], u[0][1], u[1][0], u[1][1]);
        }
      }
      if (!y_f32) {
        __syncwarp();
        uint4 v0, v1;
        ld_shared_v4(get, v0);
        ld_shared_v4(get + 512, v1);
        if (n == C) {
          *reinterpret_cast<uint4 *>(yrow) = v0;
          *reinterpret_cast<uint4 *>(yrow + 16 * ystep) = v1;
        } else {
          if (tr < n) *reinterpret_cast<uint4 *>(yrow) = v0;
          if (tr + 8 < n) *reinterpret_cast<uint4 *>(yrow + 16 * ystep) = v1;
        }
        __syncwarp();   // read before the next chunk's rows are put there
      }
      if (n < C) gamma(C, gam);
      yrow += yadvance;
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
  if (tid == 0 && *abort) atomicOr(&g_gdr_linear_error, 1);
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

template <int DA, int DC, bool PHASE1>
cudaError_t launch(const LinProblem &p, const LinChunkMaps &maps, const LinRunSel &sel, bool pdl, cudaStream_t s) {
  constexpr uint32_t SMEM = Smem<PHASE1>::BYTES;
  auto kern = linear_chunk_kernel<DA, DC, PHASE1>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long>(p.items) * p.H * sel.n));
  cfg.blockDim = dim3(NTHREADS);
  cfg.dynamicSmemBytes = SMEM;
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
