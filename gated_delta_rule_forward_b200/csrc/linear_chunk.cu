// Linear attention with a decay per head in chunks of C = 64 tokens on the
// tensor cores (bf16 tensors), for any run of three tensors a, b, c (linear.cuh).
//
// With w and Gamma powers of lambda, D_ts = lambda^|t-s| on the run's side of
// the diagonal and S the state at the chunk's start in the run's order, per chunk
//     Y = yscale (Gamma_t (a_t S) + bscale sum_s D_ts (a_t . b_s) c_s),
//     S <- lambda^n S + bscale sum_s w_s b_s c_s^T,
//     forward: Gamma_t = lambda^{t+1}, w_s = lambda^{n-1-s};  reverse: the two exchanged.
// One CTA sweeps the chunks of one (run, segment, head) in order; everything is
// held transposed, so that M = 128 of the MMAs is the value width and both the
// state and the weighted values are tensor-memory operands:
//     P    [t][s]   = a b^T          M64  N64  K = da   (into tensor memory)
//     dS^T [dc][da] = (w c)^T b      M128 N = da, K = 64
//     O1^T [dc][t]  = S^T a^T        M128 N64  K = da
//     O2^T [dc][t]  = c^T P^T        M128 N64  K = 64   (P back through shared memory in bf16)
// and Y^T = yscale (Gamma_t O1^T + O2^T).  The fp32 state lives in registers of
// 8 warps: lane dc of a quad, half of da per thread; S <- lambda^n S + dS
// is one pass over it.  c is weighted on its way into tensor memory, rather than b in
// place, which takes 64 KB of a chunk's 272 KB off shared memory.
//
// Rounding.  The products' inputs are exact bf16 except three: w c, P and the
// S^T operand.  w c enters the state, which is fp32, so it is split into three
// bf16 terms (24 bits, three MMAs): the state keeps fp32 accuracy; where the
// state is not kept (a later segment starts from phase 1's), two terms do, 2^-8
// of what follows.  P and S^T enter only Y, on disjoint parts of its sum, and
// are rounded once to bf16, like Y itself.
//
// One CTA has the SM.  Its warps are specialised and hand over through
// mbarriers, so that three chunks are under way at once:
//     copies (1 warp)    a, b, c of the chunks to come, each into the stage of one that is done
//     prep   (8 warps)   w c of chunk i + 1
//     MMAs   (3 warps)   P(i + 1);  dS(i);  O1(i), O2(i)
//     state  (8 warps)   S after chunk i, its bf16 operand
//     output (8 warps)   P of chunk i + 1 to bf16, the rows of chunk i
// Only S -> operand -> O1 is a chain from chunk to chunk.
//
// Measured on a B200 (bf16, d = 128): 65536 tokens of 16 heads, both phases, 306 us in thirty
// calls after a rest and 363 to 373 us after seconds of them, when the power limit holds the clock at
// 1.30 GHz; 8 sequences of 2048 tokens, 8 heads, 59 us forward and 112 us backward (1.73 GHz; 53 and 108 after a rest).
// With 192 runs of 32 chunks the tensor pipe is active 43% of the time and 54% of the issue
// slots are taken (1.73 GHz); a chunk takes about 2500 cycles, and value widths of 64 hardly
// less (144 runs of 32 chunks: 67 us for 72).  So neither the tensor pipe nor DRAM (42% at most)
// bounds it, nor shared memory, whose 208 KB a chunk (48 copied in, 32 read for P, 16 a term of dS, 16 for O1, 24 for O2,
// 16 of c weighted, 8 of P and 32 of output rows through it) are 1625 cycles at 128 bytes a clock: the
// hand-overs from one kind of warp to the next do, and the issue slots of the slowest kind.
// Dropped after measurement: O1 and O2 in one accumulator (64k 385 us, backward
// 118), one issuing warp for all products (404), weighting with packed bf16 arithmetic (no change).
#include <atomic>
#include <type_traits>

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
// warps 0-7 state, 8-15 output, 16-23 prep, then one for the copies and one for each of
// the three kinds of products
constexpr int NSTATE = 8, NOUT = 8, NPREP = 8;
constexpr int W_OUT = NSTATE, W_PREP = W_OUT + NOUT, W_COPY = W_PREP + NPREP, W_MMA_P = W_COPY + 1,
              W_MMA_DS = W_COPY + 2;   // and the last warp: O
constexpr int NTHREADS = 32 * (W_COPY + 4);
// registers a thread: 72 at launch, moved to the threads that hold the state
constexpr int R_STATE = 112, R_OUT = 64, R_PREP = 56, R_CTL = 40;
static_assert(32 * (NSTATE * R_STATE + NOUT * R_OUT + NPREP * R_PREP + 4 * R_CTL) <= 72 * NTHREADS, "register split");
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
constexpr uint32_t TILE = 16384;        // 64 rows of two 128-byte atoms
// Shared memory.  The copies run NST chunks ahead.
template <bool PHASE1>
struct Smem {
  static constexpr int NST = PHASE1 ? 6 : 4;
  static constexpr uint32_t B = 0;               // in a stage
  static constexpr uint32_t CT = TILE;
  static constexpr uint32_t A = 2 * TILE;
  static constexpr uint32_t STAGE = (PHASE1 ? 2 : 3) * TILE;
  static constexpr uint32_t P = NST * STAGE;     // bf16 P, rows t, 8 KB, two buffers
  static constexpr uint32_t Y = P + (PHASE1 ? 0 : 2 * 8192);      // 2 KB of output rows per output warp
  static constexpr uint32_t PW = Y + (PHASE1 ? 0 : 2048 * NOUT);   // lambda^0 .. lambda^64, then what fp32 loses of them
  static constexpr uint32_t BAR = PW + 2 * 65 * 4 + 8;
  // barriers per stage
  static constexpr uint32_t LOAD = BAR;              // a, b and c landed
  static constexpr uint32_t FREE = LOAD + 8 * NST;   // the products that read them complete (dS^T; O1^T and O2^T, which P came before)
  // per buffer of two
  static constexpr uint32_t READY = FREE + 8 * NST;  // w c written (8 warps)
  static constexpr uint32_t KV = READY + 16;         // dS^T formed
  static constexpr uint32_t OUT = KV + 16;           // O1^T and O2^T formed
  // one each
  static constexpr uint32_t OREAD = OUT + 16;        // O1^T and O2^T read (8 warps)
  static constexpr uint32_t PREAD = OREAD + 8;       // P read (8 warps)
  static constexpr uint32_t PBF = PREAD + 8;         // two: P written in bf16 (8 warps)
  static constexpr uint32_t PF = PBF + 16;           // two: P formed
  static constexpr uint32_t DS = PF + 16;            // two: dS^T read (8 warps)
  static constexpr uint32_t SOP = DS + 16;           // S^T of the chunk's start in tensor memory (8 warps)
  static constexpr uint32_t DRAIN = SOP + 8;
  static constexpr uint32_t PTAIL = DRAIN + 24;      // P of the short chunk formed (once)
  static constexpr uint32_t CREAD = PTAIL + 8;       // c of the short chunk read (8 warps, once)
  static constexpr uint32_t SLOT = CREAD + 8;        // tensor-memory address
  static constexpr uint32_t ABORT = SLOT + 4;        // a wait gave up
  static constexpr uint32_t BYTES = ABORT + 4 + 1024;
  static_assert(BAR % 16 == 0 && P % 1024 == 0 && BYTES <= 232448, "one CTA per SM");
};
// Tensor memory columns.
template <bool PHASE1>
struct Tmem {
  static constexpr uint32_t DS = 0;      // dS^T, 128 (phase 1: two buffers)
  static constexpr uint32_t S = 128;     // S^T in bf16, 64
  static constexpr uint32_t P = 192;     // P, 64
  static constexpr uint32_t O = 256;     // O1^T and O2^T, 64 each
  // (w c)^T in bf16, 32 columns a term: two buffers of two terms (phase 1: of three);
  // beside the outputs there is room for one buffer of three
  static constexpr uint32_t W = PHASE1 ? 256 : 384;
  __device__ static constexpr uint32_t term(int buf, int t) { return W + (PHASE1 ? 128 : 64) * buf + 32 * t; }
};
constexpr uint32_t TMEM_COLS = 512;

// The MMAs are issued by the lane that elect.sync picks, with the predicate inside the
// instruction and everything around it done by the whole warp: descriptors then stay in
// uniform registers, and an issue takes 26 cycles (measured, M64 N64) where the same
// instruction inside `if (lane == 0)` takes 50 to 100, more than it executes.  Descriptors
// (sdesc()) come in halves: `lo` of an address is followed by that of an address o bytes
// on at + o / 16.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);   // sbo 1024, version 1, SWIZZLE_128B
__device__ __forceinline__ void mma_ss_lo(uint32_t d_tmem, uint32_t alo, uint32_t blo, uint32_t idesc, uint32_t acc,
                                          uint32_t e) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(alo), "r"(blo), "r"(idesc), "r"(acc), "r"(DESC_HI), "r"(e)
      : "memory");
}
__device__ __forceinline__ void mma_ts_lo(uint32_t d_tmem, uint32_t a_tmem, uint32_t blo, uint32_t idesc, uint32_t acc,
                                          uint32_t e) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(blo), "r"(idesc), "r"(acc), "r"(DESC_HI), "r"(e)
      : "memory");
}
// Four K steps (64 of K), A and B advancing by `as` and `bs` a step.
template <bool TS>
__device__ __forceinline__ void mma4(uint32_t d, uint32_t a, uint32_t as, uint32_t b, uint32_t bs, uint32_t idesc,
                                     uint32_t acc, uint32_t e) {
#pragma unroll
  for (uint32_t k = 0; k < 4; ++k) {
    if (TS) mma_ts_lo(d, a + as * k, b + bs * k, idesc, k == 0 ? acc : 1, e);
    else mma_ss_lo(d, a + as * k, b + bs * k, idesc, k == 0 ? acc : 1, e);
  }
}
__device__ __forceinline__ void commit_one(uint32_t bar, uint32_t e) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(e)
      : "memory");
}

// Barriers by their 32-bit shared-memory addresses: with 24 warps waiting and arriving
// several times a chunk, generic pointers cost more integer instructions than the
// arithmetic took.
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void expect_at(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Waits up to the given limit (a millisecond), which leaves the issue slots to others.
__device__ __forceinline__ bool try_wait_at(uint32_t bar, uint32_t phase) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000000;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(phase)
      : "memory");
  return ok != 0;
}
// Bounded wait (a second or so) that also gives up once another thread has (the word at
// `abort`).
__device__ __forceinline__ uint32_t clock32() {
  uint32_t c;
  asm volatile("mov.u32 %0, %%clock;" : "=r"(c));
  return c;
}
__device__ __forceinline__ bool wait_at(uint32_t bar, uint32_t phase, uint32_t abort) {
  if (__builtin_expect(try_wait_at(bar, phase), 1)) return true;
  const uint32_t start = clock32();
#pragma unroll 1
  while (!try_wait_at(bar, phase)) {
    uint32_t gave_up;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(gave_up) : "r"(abort) : "memory");
    if (__builtin_expect(gave_up || clock32() - start > 0x80000000u, 0)) {
      asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(abort), "r"(1u) : "memory");
      return false;
    }
  }
  return true;
}
// The same, asking again at once: an issue slot now and then, for a shorter way from the
// last operand to the product.
__device__ __forceinline__ bool spin_at(uint32_t bar, uint32_t phase, uint32_t abort) {
  const uint32_t start = clock32();
  while (true) {
    uint32_t ok, gave_up;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(phase)
        : "memory");
    if (ok) return true;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(gave_up) : "r"(abort) : "memory");
    if (__builtin_expect(gave_up || clock32() - start > 0x80000000u, 0)) {
      asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(abort), "r"(1u) : "memory");
      return false;
    }
  }
}
// The same by a whole warp.
__device__ __forceinline__ bool warp_wait_at(uint32_t bar, uint32_t phase, uint32_t abort) {
  return __all_sync(0xffffffffu, wait_at(bar, phase, abort));
}
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
// A ring of N barriers or stages: index and phase of one chunk after another.
template <int N>
struct Ring {
  uint32_t at = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      phase ^= 1;
    }
  }
};

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
template <int TERMS>
__device__ __forceinline__ void split_pair(uint32_t x, float w0, float w1, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
  const float a = __uint_as_float(x << 16) * w0, b = __uint_as_float(x & 0xffff0000u) * w1;
  hi = pack_bf16x2(a, b);
  const float ra = a - __uint_as_float(hi << 16), rb = b - __uint_as_float(hi & 0xffff0000u);
  mid = pack_bf16x2(ra, rb);
  if (TERMS == 3)
    lo = pack_bf16x2(ra - __uint_as_float(mid << 16), rb - __uint_as_float(mid & 0xffff0000u));
}

// YF32: y in fp32 (the value heads' shares of a shared head's gradient).
// LONG: phase 2 chains any number of segments (kLinSelfChain otherwise) or from copied start states, whose code costs
// the others registers.
template <int DA, int DC, bool PHASE1, bool YF32, bool LONG>
__device__ __forceinline__ void chunk_run(const LinProblem &p, const LinChunkMaps &maps, const LinRun &r, unsigned block) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + (-smem_u32(smem_raw) & 1023u);   // an offset, so that accesses stay shared ones
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // uniform in the compiler's eyes, and so the branches on it
  if (warp == W_COPY && lane < 3) prefetch_tmap(&maps.m[lane == 0 ? r.ib : lane == 1 ? r.ic : r.ia]);
  const bool rev = r.reverse != 0;
  const bool zero_rest = !PHASE1 && !YF32 && p.zero_rest;
  int rest_first = 0, rest_end = p.T;
  if (zero_rest) rest_first = lin_cu(p, 0), rest_end = lin_cu(p, p.N);
  const LinItem it = lin_item(p, block);
  if (zero_rest) lin_zero_rest(p, r.y, static_cast<size_t>(p.H) * DC * 2, rest_first, rest_end, block, gridDim.x / p.nrun);
  const int h = it.h;
  const bool last = rev ? it.g == 0 : it.g == it.nseg - 1;   // in the run's order
  if (!it.ok || (PHASE1 && last && (it.nseg == 1 || !r.s_final))) {
    griddep_launch_dependents();
    griddep_wait();
    return;
  }

  using M = Smem<PHASE1>;
  using T = Tmem<PHASE1>;
  constexpr int NST = M::NST;
  float *pw = reinterpret_cast<float *>(sm + M::PW), *pw_lo = pw + 65;
  const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(sm), 0), abort = base + M::ABORT;

  if (warp == 0) {
    tmem_alloc(reinterpret_cast<uint32_t *>(sm + M::SLOT), TMEM_COLS);
    tmem_relinquish();
  }
  // host fault injection: the first block copies no first chunk (phase 1), or forms no P, so that its waits run out
  const bool faulty = p.fault && blockIdx.x == 0;
  const int beg = it.beg, end = it.end;
  const int nch = __shfl_sync(0xffffffffu, (end - beg + C - 1) / C, 0);
  // copies of one chunk into its stage, and of the chunk that comes there next as far as L2
  const int row_first = it.t0 + beg + (rev ? C * (nch - 1) : 0), row_step = rev ? -C : C;
  auto copy_chunk = [&](int i, uint32_t at) {
    const CUtensorMap *ma = &maps.m[r.ia], *mb = &maps.m[r.ib], *mc = &maps.m[r.ic];
    const int ha = h / p.t[r.ia].div, hb = h / p.t[r.ib].div, hc = h / p.t[r.ic].div;
    constexpr uint32_t bytes = (PHASE1 ? 0 : DA * 128) + DA * 128 + DC * 128;
    const uint32_t bar = base + M::LOAD + 8 * at, dst = base + M::STAGE * at;
    const int row = row_first + i * row_step;
    expect_at(bar, bytes);
    for (int d = 0; d < DA / 64; ++d) {
      load_box(dst + M::B + 8192 * d, mb, bar, 64 * d, hb, row, it.b);
      if (!PHASE1) load_box(dst + M::A + 8192 * d, ma, bar, 64 * d, ha, row, it.b);
    }
    for (int d = 0; d < DC / 64; ++d) load_box(dst + M::CT + 8192 * d, mc, bar, 64 * d, hc, row, it.b);
    if (i + NST < nch) {
      const int ahead = row + NST * row_step;
      for (int d = 0; d < DA / 64; ++d) {
        tma_prefetch_4d(mb, 64 * d, hb, ahead, it.b);
        if (!PHASE1) tma_prefetch_4d(ma, 64 * d, ha, ahead, it.b);
      }
      for (int d = 0; d < DC / 64; ++d) tma_prefetch_4d(mc, 64 * d, hc, ahead, it.b);
    }
  };
  if (tid == 32 * W_COPY) {
    auto init = [&](uint32_t at, int n, uint32_t count) {
      for (int i = 0; i < n; ++i) mbar_init(reinterpret_cast<uint64_t *>(sm + at + 8 * i), count);
    };
    init(M::LOAD, NST, 1);
    init(M::FREE, NST, PHASE1 ? 1 : 2);
    init(M::READY, 2, NPREP);
    init(M::KV, 2, 1);
    init(M::OUT, 2, 1);
    init(M::OREAD, 1, NOUT);
    init(M::PF, 2, 1);
    init(M::PREAD, 1, NOUT);
    init(M::PBF, 2, NOUT);
    init(M::DS, 2, NSTATE);
    init(M::SOP, 1, NSTATE);
    init(M::DRAIN, 3, 1);
    init(M::PTAIL, 1, 1);
    init(M::CREAD, 1, NPREP);
    *reinterpret_cast<uint32_t *>(sm + M::ABORT) = 0;
    fence_mbar_init();
    // the first chunks: their tensors are inputs of the call, whatever grid this one depends on
    for (int i = PHASE1 && faulty ? 1 : 0; i < NST && i < nch; ++i) copy_chunk(i, i);
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
  const uint32_t tmem = *reinterpret_cast<uint32_t *>(sm + M::SLOT);   // 0: the CTA holds all of tensor memory (the MMA warp writes it so)

  const int page = lin_page(p, it.n);
  // (the end state of a sequence with several segments is made from phase 1's)
  float *const final_page = !PHASE1 && it.nseg == 1 && r.s_final && page >= 0
                                ? r.s_final + (static_cast<size_t>(page) * p.H + h) * DA * DC : nullptr;
  // a state that leaves in fp32 takes all three terms; one that only makes bf16 outputs, two
  const bool three = PHASE1 || __shfl_sync(0xffffffffu, final_page != nullptr, 0);
  const int tail_i = rev ? 0 : nch - 1, tail_n = end - beg - C * (nch - 1);   // the only chunk that may be short

  // The grid before: phase 1's states, or the chain kernel's.  Whoever reads them waits here itself.  (A sequence
  // that runs whole reads only what the call was given, complete before phase 1 began, and may run beside it.)
  const float *start = r.X + static_cast<size_t>(it.slot) * DA * DC;
  if (PHASE1 || it.nseg > 1) griddep_wait();
  griddep_launch_dependents();
  if (PHASE1 && p.s0_copied && it.g == 0) {
    const float4 *src = reinterpret_cast<const float4 *>(r.s0 + (static_cast<size_t>(max(page, 0)) * p.H + h) * DA * DC);
    float4 *dst = reinterpret_cast<float4 *>(r.XS + static_cast<size_t>(it.slot) * DA * DC);
    for (int e = tid; e < DA * DC / 4; e += NTHREADS) dst[e] = page >= 0 ? src[e] : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (!PHASE1 && it.nseg > 1 && !p.chained) {
    float *mine = r.XS + static_cast<size_t>(it.slot) * DA * DC;
    if (LONG) lin_self_chain_long(p, r, it, page, last, DA, DC, mine, tid, NTHREADS);
    else lin_self_chain(p, r, it, page, last, DA, DC, mine, tid, NTHREADS);
    start = mine;
    __syncthreads();
  }

  if (warp >= W_COPY) regs_dec<R_CTL>();
  if (warp == W_COPY) {
    // ---------------------------------------------------------------- copies
    if (lane == 0) {
      int i = min(nch, NST);   // the first ones are under way
      Ring<NST> st;
      for (; i < nch; ++i, st.next()) {
        if (!wait_at(base + M::FREE + 8 * st.at, st.phase, abort)) break;
        copy_chunk(i, st.at);
      }
      // nothing may land in shared memory after the CTA (each wait bounded)
      for (int j = i > NST ? i - NST : PHASE1 && faulty ? 1 : 0; j < i; ++j)
        mbar_wait(reinterpret_cast<uint64_t *>(sm + M::LOAD) + j % NST, (j / NST) & 1);
    }
    // what follows this grid follows the one before it, whether or not any of its blocks had to wait
    if (blockIdx.x == gridDim.x - 1) griddep_wait();
  } else if (warp > W_COPY) {
    // ---------------------------------------------------------------- MMAs
    // A warp for each kind, so that none waits behind another's operands; a product's
    // operands are all handed over through barriers, so their order needs no more.
    // No barrier may complete a phase that some waiter has not yet seen: each waiter of
    // phase k of a barrier comes, by some chain of hand-overs, before its phase k + 1.
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t phase) {
      ok = ok && __all_sync(0xffffffffu, spin_at(base + bar, phase, abort));
      return ok;
    };
    Ring<NST> st;
    Ring<2> bf;
    if (warp == W_MMA_P) {   // P = a b^T, as soon as the chunk before's is read
      for (int i = 0; !PHASE1 && !faulty && i < nch; ++i, st.next(), bf.next()) {
        if (i > 0 && !wait(M::PREAD, (i - 1) & 1)) break;
        if (!wait(M::LOAD + 8 * st.at, st.phase)) break;
        tc_fence_after();
        const uint32_t sb = base + M::STAGE * st.at, alo = desc_lo(sb + M::A, 16), blo = desc_lo(sb + M::B, 16);
        const uint32_t e = elect_one();
#pragma unroll
        for (uint32_t d = 0; d < DA / 64; ++d)
          mma4<false>(T::P, alo + 512 * d, 2, blo + 512 * d, 2, idesc_bf16(C, C, false, false), d, e);
        commit_one(base + M::PF + 8 * bf.at, e);
        if (i == tail_i) commit_one(base + M::PTAIL, e);
      }
    } else if (warp == W_MMA_DS) {   // dS^T = (w c)^T b
      for (int i = 0; i < nch; ++i, st.next(), bf.next()) {
        if (!wait(M::LOAD + 8 * st.at, st.phase) || !wait(M::READY + 8 * bf.at, bf.phase)) break;
        if (PHASE1 ? i >= 2 && !wait(M::DS + 8 * bf.at, bf.phase ^ 1)
                   : i >= 1 && !wait(M::DS + 8 * (bf.at ^ 1), bf.phase ^ (bf.at ^ 1))) break;
        tc_fence_after();
        const uint32_t blo = desc_lo(base + M::STAGE * st.at + M::B, 8192);
        const uint32_t wcol = T::term(PHASE1 || !three ? bf.at : 0, 0), ds = T::DS + (PHASE1 ? 128 * bf.at : 0);
        const uint32_t e = elect_one();
#pragma unroll
        for (uint32_t t = 0; t < 2; ++t) mma4<true>(ds, wcol + 32 * t, 8, blo, 128, idesc_bf16(128, DA, false, true), t, e);
        if (three) mma4<true>(ds, wcol + 64, 8, blo, 128, idesc_bf16(128, DA, false, true), 1, e);
        commit_one(base + M::KV + 8 * bf.at, e);
        commit_one(base + M::FREE + 8 * st.at, e);
      }
    } else {   // O1^T = S^T a^T, O2^T = c^T P^T
      for (int i = 0; !PHASE1 && i < nch; ++i, st.next(), bf.next()) {
        if (!wait(M::LOAD + 8 * st.at, st.phase) || !wait(M::PBF + 8 * bf.at, bf.phase)) break;
        // the short chunk's rows of c behind the end are zeros once its dS^T is formed
        if (i == tail_i && tail_n < C && !wait(M::KV + 8 * bf.at, bf.phase)) break;
        if (!wait(M::SOP, i & 1)) break;
        if (i > 0 && !wait(M::OREAD, (i - 1) & 1)) break;
        tc_fence_after();
        const uint32_t sb = base + M::STAGE * st.at, alo = desc_lo(sb + M::A, 16);
        const uint32_t e = elect_one();
#pragma unroll
        for (uint32_t d = 0; d < DA / 64; ++d)
          mma4<true>(T::O, T::S + 32 * d, 8, alo + 512 * d, 2, idesc_bf16(128, C, false, false), d, e);
        mma4<false>(T::O + 64, desc_lo(sb + M::CT, 8192), 128, desc_lo(base + M::P + 8192 * bf.at, 16), 2,
                    idesc_bf16(128, C, true, false), 0, e);
        commit_one(base + M::OUT + 8 * bf.at, e);
        commit_one(base + M::FREE + 8 * st.at, e);
      }
    }
    // the MMAs in flight finish before the memory they use is released, also where a wait gave up and nobody
    // else waits for them
    commit_one(base + M::DRAIN + 8 * (warp - W_MMA_P), elect_one());
    mbar_wait(reinterpret_cast<uint64_t *>(sm + M::DRAIN) + (warp - W_MMA_P), 0);
  } else if (warp >= W_PREP) {
    // ---------------------------------------------------------------- prep: w c
    regs_dec<R_PREP>();
    const int quad = warp & 3, half = (warp - W_PREP) >> 2;
    const float bscale = r.bscale;
    const bool has_c = 32 * quad < DC;
    const int s0 = 32 * half + 2 * (lane & 3);   // this thread's tokens: s0 + 8 j (+ 1), j = 0 .. 3
    // w c: lanes dc = 32 quad + 16 g + lane / 4 (+ 8), tokens s0 + 8 j (+ 1); full chunks' weights
    float wgt[4][2];
    auto weights = [&](int n) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int s = s0 + 8 * j;
        wgt[j][0] = bscale * pw[rev ? s + 1 : max(n - 1 - s, 0)];
        wgt[j][1] = bscale * pw[rev ? s + 2 : max(n - 2 - s, 0)];
      }
    };
    weights(C);
    // ldmatrix of c: matrix m = tokens 8 (j + m / 2) .., columns 8 (m & 1) ..; its row q = token
    const int sq = 32 * half + 8 * (lane >> 4) + (lane & 7), dq = 32 * quad + 8 * ((lane >> 3) & 1);
    const uint32_t get0 = base + M::CT + (dq >> 6) * 8192 + sw128(sq, (dq & 63) >> 3);
    const uint32_t get1 = base + M::CT + ((dq + 16) >> 6) * 8192 + sw128(sq, ((dq + 16) & 63) >> 3);
    auto weigh = [&](uint32_t stage, uint32_t col, int n, auto terms) {
      constexpr int TERMS = decltype(terms)::value;
      uint32_t v[2][8];
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int j = 0; j < 4; j += 2)
          ldmatrix4_trans((g ? get1 : get0) + stage + 1024 * j, v[g][2 * j], v[g][2 * j + 1], v[g][2 * j + 2], v[g][2 * j + 3]);
      if (n < C)   // tokens behind the sequence's end count for nothing, whatever they hold
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int s = s0 + 8 * (j >> 1);
          const uint32_t keep = s + 1 < n ? 0xffffffffu : s < n ? 0xffffu : 0u;
          v[0][j] &= keep;
          v[1][j] &= keep;
        }
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t t1[8], t2[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) split_pair<TERMS>(v[g][j], wgt[j >> 1][0], wgt[j >> 1][1], v[g][j], t1[j], t2[j]);
        const uint32_t at = col + (static_cast<uint32_t>(16 * g) << 16);
        tmem_st_frag4(at, v[g]);
        tmem_st_frag4(at + 32, t1);
        if (TERMS == 3) tmem_st_frag4(at + 64, t2);
      }
    };
    const uint32_t wlane = tmem + (static_cast<uint32_t>(quad * 32) << 16) + 16 * half;
    if (!has_c) {   // value widths of 64: the upper lanes' operand is zero
      const uint32_t zero[8] = {};
      for (int t = 0; t < (PHASE1 ? 8 : 4); ++t)   // every column of the buffers
        for (int g = 0; g < 2; ++g) tmem_st_frag4(wlane + (static_cast<uint32_t>(16 * g) << 16) + T::term(0, t), zero);
      tmem_wait_st();   // here: an empty sequence has no chunk to wait in, and the CTA frees the memory at once
    }
    Ring<NST> st;
    Ring<2> bf;
    for (int i = 0; i < nch; ++i, st.next(), bf.next()) {
      const int n = i == tail_i ? tail_n : C;
      if (!warp_wait_at(base + M::LOAD + 8 * st.at, st.phase, abort)) break;
      // the buffer is that of the product of two chunks ago (one buffer of three terms: of the last chunk)
      if (!PHASE1 && three) {
        if (i >= 1 && !warp_wait_at(base + M::KV + 8 * (bf.at ^ 1), bf.phase ^ (bf.at ^ 1), abort)) break;
      } else {
        if (i >= 2 && !warp_wait_at(base + M::KV + 8 * bf.at, bf.phase ^ 1, abort)) break;
      }
      tc_fence_after();
      if (n < C) weights(n);
      if (has_c) {
        const uint32_t col = wlane + T::term(PHASE1 || !three ? bf.at : 0, 0);
        if (three) weigh(M::STAGE * st.at, col, n, std::integral_constant<int, 3>());
        else weigh(M::STAGE * st.at, col, n, std::integral_constant<int, 2>());
      }
      tmem_wait_st();
      if (n < C) {
        // rows behind the sequence's end, which the products read as well, become zeros (once all of c is
        // read and P is formed; the output warps clear P of them)
        __syncwarp();
        if (lane == 0) arrive_at(base + M::CREAD);
        if (!PHASE1 && !warp_wait_at(base + M::PTAIL, 0, abort)) break;
        if (!warp_wait_at(base + M::CREAD, 0, abort)) break;
        uint8_t *sb = sm + M::STAGE * st.at;
        const int row = tid & 63, piece = (tid >> 6) & 3;
        if (row >= n) {
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
          for (int j = piece; j < DA / 8; j += 4) *reinterpret_cast<uint4 *>(sb + M::B + (j >> 3) * 8192 + sw128(row, j & 7)) = zero;
          for (int j = piece; j < DC / 8; j += 4) *reinterpret_cast<uint4 *>(sb + M::CT + (j >> 3) * 8192 + sw128(row, j & 7)) = zero;
        }
        weights(C);
        fence_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_at(base + M::READY + 8 * bf.at);
    }
  } else if (warp >= W_OUT) {
    // ---------------------------------------------------------------- P and the output
    regs_dec<R_OUT>();
    // this warp's 32 columns dc and 32 tokens t, through its 2 KB of shared memory (rows t of
    // 64 bytes, 16-byte chunks XOR-ed with t / 2) unless in fp32.  Fragment tiles: lane
    // holds dc = 16 hh + lane / 4 (+ 8), t = 16 tt + 8 j + 2 (lane % 4) (+ 1).
    const int quad = warp & 3, half = (warp - W_OUT) >> 2;
    const uint32_t lrow = tmem + (static_cast<uint32_t>(quad * 32) << 16) + T::O + 32 * half;
    const float yscale = r.yscale;
    const size_t ystep = static_cast<size_t>(p.H) * DC;
    const int tf = 32 * half + 2 * (lane & 3), tr = 32 * half + (lane >> 2);
    const uint32_t stage = base + M::Y + 2048 * (warp - W_OUT);
    // stmatrix: matrix m = tokens 8 (m / 2) .., columns 8 (m & 1) ..; its row q = token
    const int tq = 8 * (lane >> 4) + (lane & 7), cq = (lane >> 3) & 1;
    const uint32_t put0 = stage + tq * 64 + (((cq ^ (tq >> 1)) & 3) << 4), put1 = stage + tq * 64 + ((((2 + cq) ^ (tq >> 1)) & 3) << 4);
    const uint32_t get = stage + (lane >> 2) * 64 + ((((lane & 3) ^ (lane >> 3)) & 3) << 4);   // every 512 bytes on: token + 8
    // full chunks' decays
    uint64_t gam[4];
    auto gamma = [&](int n) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = tf + 8 * j;
        gam[j] = pair_f32(yscale * pw[rev ? max(n - 1 - t, 0) : t + 1], yscale * pw[rev ? max(n - 2 - t, 0) : t + 2]);
      }
    };
    gamma(C);
    // this lane's row in the chunk, advanced chunk by chunk
    uint8_t *yrow;
    const long long yadvance = (rev ? -C : C) * static_cast<long long>(ystep) * (YF32 ? 4 : 2);
    {
      const size_t row = static_cast<size_t>(it.b) * p.T + it.t0 + beg + (rev ? C * (nch - 1) : 0);
      if (YF32) yrow = reinterpret_cast<uint8_t *>(static_cast<float *>(r.y) + (row + tf) * ystep + h * DC + 32 * quad + (lane >> 2));
      else yrow = reinterpret_cast<uint8_t *>(static_cast<__nv_bfloat16 *>(r.y) + (row + tr) * ystep + h * DC + 32 * quad + 8 * (lane & 3));
    }
    // P: rows t = 16 quad + lane / 4 (+ 8), columns s0 + 8 j (+ 1); the decays are the same for every chunk
    const int s0 = tf;
    uint64_t dec[4][2];
    {
      const float f = r.bscale * yscale;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int t = 16 * quad + (lane >> 2) + 8 * k, s = s0 + 8 * j;
          const int d = rev ? s - t : t - s, d1 = rev ? d + 1 : d - 1;
          dec[j][k] = pair_f32(d >= 0 ? f * pw[max(d, 0)] : 0.f, d1 >= 0 ? f * pw[max(d1, 0)] : 0.f);
        }
    }
    // stmatrix of P: matrix m = rows 8 (m & 1) .., columns 8 (m / 2) ..
    const int tp = 16 * quad + (lane & 15), cp = 4 * half + (lane >> 4);
    const uint32_t pput0 = base + M::P + sw128(tp, cp), pput1 = base + M::P + sw128(tp, cp + 2);
    const uint32_t plane = tmem + (static_cast<uint32_t>(quad * 32) << 16) + T::P + 32 * half;
    Ring<2> bf, obf;   // of P's chunk, and of the output's, one behind
    for (int i = 0; !PHASE1 && i <= nch; ++i, bf.next()) {
      if (i < nch) {   // P of chunk i, with its decays
        const int n = i == tail_i ? tail_n : C;
        if (!warp_wait_at(base + M::PF + 8 * bf.at, bf.phase, abort)) break;
        tc_fence_after();
        float v[16];
        tmem_ld_frag4(plane, v);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_at(base + M::PREAD);
        uint32_t u[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float y0, y1;
            unpair_f32(mul_f32x2(pair_f32(v[4 * j + 2 * k], v[4 * j + 2 * k + 1]), dec[j][k]), y0, y1);
            u[j][k] = pack_bf16x2(y0, y1);
          }
        if (n < C)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t keep = s0 + 8 * j + 1 < n ? 0xffffffffu : s0 + 8 * j < n ? 0xffffu : 0u;
            u[j][0] &= keep;
            u[j][1] &= keep;
          }
        // (the buffer's last reader, the product of two chunks ago, was waited for with its output)
        stmatrix4(pput0 + 8192 * bf.at, u[0][0], u[0][1], u[1][0], u[1][1]);
        stmatrix4(pput1 + 8192 * bf.at, u[2][0], u[2][1], u[3][0], u[3][1]);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) arrive_at(base + M::PBF + 8 * bf.at);
      }
      if (i == 0) continue;
      // the output of chunk i - 1
      const int n = i - 1 == tail_i ? tail_n : C;
      if (!warp_wait_at(base + M::OUT + 8 * obf.at, obf.phase, abort)) break;
      tc_fence_after();
      obf.next();
      if (32 * quad >= DC) {   // a value width of 64: nothing of it in these lanes
        if (lane == 0) arrive_at(base + M::OREAD);
        continue;
      }
      if (n < C) gamma(n);
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        float v1[2][8], v2[2][8];   // 16 lanes of tensor memory each: dc = 32 quad + 16 hh ..
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          tmem_ld_frag2(lrow + (static_cast<uint32_t>(16 * hh) << 16) + 16 * tt, v1[hh]);
          tmem_ld_frag2(lrow + (static_cast<uint32_t>(16 * hh) << 16) + 16 * tt + 64, v2[hh]);
        }
        tmem_wait_ld();
        if (tt == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_at(base + M::OREAD);
        }
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t u[2][2];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float a, b;
              unpair_f32(fma_f32x2(gam[2 * tt + j], pair_f32(v1[hh][4 * j + 2 * k], v1[hh][4 * j + 2 * k + 1]),
                                   pair_f32(v2[hh][4 * j + 2 * k], v2[hh][4 * j + 2 * k + 1])), a, b);
              if (YF32) {
                float *dst = reinterpret_cast<float *>(yrow) + (16 * tt + 8 * j) * ystep + 16 * hh + 8 * k;
                if (tf + 16 * tt + 8 * j < n) dst[0] = a;
                if (tf + 16 * tt + 8 * j + 1 < n) dst[ystep] = b;
              } else {
                u[j][k] = pack_bf16x2(a, b);
              }
            }
          if (!YF32) stmatrix4_trans((hh ? put1 : put0) + 1024 * tt, u[0][0], u[0][1], u[1][0], u[1][1]);
        }
      }
      if (!YF32) {
        __syncwarp();
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) ld_shared_v4(get + 512 * k, v[k]);
        if (n == C) {
#pragma unroll
          for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4 *>(yrow + 16 * k * ystep) = v[k];
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (tr + 8 * k < n) *reinterpret_cast<uint4 *>(yrow + 16 * k * ystep) = v[k];
        }
        __syncwarp();   // read before the next chunk's rows are put there
      }
      if (n < C) gamma(C);
      yrow += yadvance;
    }
  } else {
    // ---------------------------------------------------------------- state
    regs_inc<R_STATE>();
    // thread (quad, lane, half) holds S[da = half DA/2 + j][dc = 32 quad + lane], in pairs along da
    const int quad = warp & 3, half = warp >> 2;
    constexpr int SN = DA / 2;
    const int dcr = 32 * quad + lane, da0 = half * SN;
    const bool has_c = dcr < DC;
    uint64_t S[SN / 2];
#pragma unroll
    for (int j = 0; j < SN / 2; ++j) S[j] = 0;
    if (!PHASE1 && has_c) {
      if (it.nseg > 1) {
        const float *src = start + static_cast<size_t>(da0) * DC + dcr;
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
#pragma unroll
      for (int q = 0; q < SN / 32; ++q) {
        uint32_t u[16];
#pragma unroll
        for (int m = 0; m < 16; ++m) {
          float a, b;
          unpair_f32(S[16 * q + m], a, b);
          u[m] = pack_bf16x2(a, b);
        }
        tmem_st16(lrow + T::S + half * (SN / 2) + 16 * q, u);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_at(base + M::SOP);
    };
    if (!PHASE1) store_operand();
    bool ok = true;
    Ring<2> bf;
    for (int i = 0; i < nch; ++i, bf.next()) {
      const int n = i == tail_i ? tail_n : C;
      // S <- lambda^n S + dS
      if (!(ok = warp_wait_at(base + M::KV + 8 * bf.at, bf.phase, abort))) break;
      tc_fence_after();
      {
        const float g = n == C ? decay.next() : pw[n];
        const uint64_t g2 = pair_f32(g, g);
#pragma unroll
        for (int q = 0; q < SN / 32; ++q) {
          float v[32];
          tmem_ld32(lrow + T::DS + (PHASE1 ? 128 * bf.at : 0) + da0 + 32 * q, v);
          if (q == SN / 32 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_at(base + M::DS + 8 * bf.at);
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) S[16 * q + e] = fma_f32x2(g2, S[16 * q + e], pair_f32(v[2 * e], v[2 * e + 1]));
        }
      }
      // its operand for the next chunk, once O1^T has been formed from this one's
      if (PHASE1 || i + 1 == nch) continue;
      if (!(ok = warp_wait_at(base + M::OUT + 8 * bf.at, bf.phase, abort))) break;
      tc_fence_after();
      store_operand();
    }
    float *dst = PHASE1 ? r.X + static_cast<size_t>(it.slot) * DA * DC : final_page;
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
  if (tid == 0 && *reinterpret_cast<volatile uint32_t *>(sm + M::ABORT)) atomicOr(&g_gdr_linear_error, 1);
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// All runs of a phase in one launch.  A forward has one run, (DA, DC); a backward dq's, dk's and dv's, the last (DA, DC),
// the others (DC, DA) and with y in fp32 if YF32, which a MIXED kernel has a second body for.
template <int DA, int DC, bool PHASE1, bool MIXED, bool YF32, bool LONG>
__global__ void __launch_bounds__(NTHREADS, 1)
    linear_chunk_kernel(const __grid_constant__ LinProblem p, const __grid_constant__ LinChunkMaps maps) {
  unsigned block;
  const LinRun &r = lin_run<!MIXED>(p, block);
  if (MIXED && (r.dc != DC || r.y_f32)) chunk_run<DC, DA, PHASE1, YF32, LONG>(p, maps, r, block);
  else chunk_run<DA, DC, PHASE1, false, LONG>(p, maps, r, block);
}

template <int DA, int DC, bool PHASE1, bool MIXED, bool YF32, bool LONG>
cudaError_t launch(const LinProblem &p, const LinChunkMaps &maps, bool pdl, cudaStream_t s) {
  constexpr uint32_t SMEM = Smem<PHASE1>::BYTES;
  auto kern = linear_chunk_kernel<DA, DC, PHASE1, MIXED, YF32, LONG>;
  // the kernel's limit on the current device, set by the first call there
  static std::atomic<unsigned long long> set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (!(set.load(std::memory_order_relaxed) & bit)) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM)) != cudaSuccess) return e;
    set.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(lin_blocks(p) * p.nrun));
  cfg.blockDim = dim3(NTHREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p, maps);
}

template <int DA, int DC>
cudaError_t launch_kind(const LinProblem &p, const LinChunkMaps &m, bool phase1, bool pdl, cudaStream_t s) {
  const bool backward = p.nrun == kLinMaxRuns;
  if (backward && phase1 && DA != DC) return launch<DA, DC, true, DA != DC, false, false>(p, m, pdl, s);
  if (phase1) return launch<DA, DC, true, false, false, false>(p, m, pdl, s);
  if (backward && p.run[0].y_f32) return launch<DA, DC, false, true, true, false>(p, m, pdl, s);
  if (backward && DA != DC) return launch<DA, DC, false, DA != DC, false, false>(p, m, pdl, s);
  if (!p.chained && (p.G > kLinSelfChain || p.s0_copied)) return launch<DA, DC, false, false, false, true>(p, m, pdl, s);   // (a forward)
  return launch<DA, DC, false, false, false, false>(p, m, pdl, s);
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
  const gdr::LinRun &r = p.run[p.nrun - 1];   // o's or dv's: (dk, dv)
  if (r.da == 128 && r.dc == 128) return gdr::tc::launch_kind<128, 128>(p, maps, phase1, pdl, s);
  if (r.da == 128) return gdr::tc::launch_kind<128, 64>(p, maps, phase1, pdl, s);
  if (r.dc == 128) return gdr::tc::launch_kind<64, 128>(p, maps, phase1, pdl, s);
  return gdr::tc::launch_kind<64, 64>(p, maps, phase1, pdl, s);
}

int gdr_linear_read_device_error(cudaStream_t stream) {
  int h = 0, zero = 0;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return -1;
  if (cudaMemcpyFromSymbol(&h, g_gdr_linear_error, sizeof(int)) != cudaSuccess) return -1;
  if (h) cudaMemcpyToSymbol(g_gdr_linear_error, &zero, sizeof(int));
  return h;
}
