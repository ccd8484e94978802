// One token of linear attention with a decay per head, on a pool of states
// (bandwidth-bound: the fp32 state is read once and written once, and q, k, v
// and o are about 1% of its bytes).
//
//     S <- lambda S + k v^T,   o = scale S^T q
//
// The same lambda multiplies a state for thousands of steps, so its error compounds over
// the state's memory of 1 / (1 - lambda) of them: one fp32 value of it is off by up to
// 2^-25, which a decay of -1e-6 makes 3%.  It is taken as hi + lo (lin_decay):
//     S <- hi S + (lo S + k v^T).
//
// The value columns are independent, so a (row, head) may be cut into slices of
// columns, one CTA of 256 threads each: thread (rg, cq) holds columns
// 4 cq .. 4 cq + 3 of rows rg, rg + RG, ..., with all its float4 loads issued
// before the first is used.  Whole rows (512 bytes per warp) where the batch
// fills the device by itself; 32-column slices (128-byte row pieces) otherwise,
// which puts four times the SMs on a small batch (3 rows of 8 heads of 128 x 128 in a
// graph: 2.05 us in slices, 2.9 whole; 16 rows: 3.3 and 3.2; 36: 5.0 and 4.9).  256 rows
// of 16 heads: 85.3 us, 6.27 TB/s; 3 rows of 8 heads called one by one: 11.8 us, the
// host's part of a call.
#include "linear.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 256;

template <int DK, int W, typename IO>
__global__ void __launch_bounds__(kThreads) linear_decode_kernel(const LinDecodeProblem p) {
  constexpr int TPR = W / 4, RG = kThreads / TPR, RPT = DK / RG;
  static_assert(RPT >= 1 && DK % RG == 0 && TPR <= 32, "shape");
  __shared__ float kf[DK], qf[DK];
  __shared__ __align__(16) float red[kThreads / 32][W];
  const int tid = threadIdx.x, cq = tid % TPR, rg = tid / TPR;
  const int slices = p.dv / W;
  const int sl = blockIdx.x % slices;
  const long nh = blockIdx.x / slices;
  const int n = static_cast<int>(nh / p.H), h = static_cast<int>(nh % p.H);
  const int page = p.slots ? __ldg(p.slots + n) : n;
  IO *o = static_cast<IO *>(p.o) + nh * p.dv + sl * W;
  if (page < 0 || page >= p.pages) {   // a padding row: zeros, no state
    if (tid < W) st_io<IO>(o + tid, 0.f);
    return;
  }
  float *S = p.state + (static_cast<size_t>(page) * p.H + h) * DK * p.dv + sl * W + 4 * cq;
  float4 s[RPT];
#pragma unroll
  for (int r = 0; r < RPT; ++r) s[r] = *reinterpret_cast<const float4 *>(S + static_cast<size_t>(rg + RG * r) * p.dv);

  const size_t qrow = (static_cast<size_t>(n) * p.Hk + h / (p.H / p.Hk)) * DK;
  if (tid < DK) kf[tid] = ld_io<IO>(static_cast<const IO *>(p.k) + qrow + tid);
  else if (tid < 2 * DK) qf[tid - DK] = ld_io<IO>(static_cast<const IO *>(p.q) + qrow + tid - DK);
  float v[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) v[c] = ld_io<IO>(static_cast<const IO *>(p.v) + nh * p.dv + sl * W + 4 * cq + c);
  const float2 lam = lin_decay(__ldg(p.log_decay + h));
  __syncthreads();
  auto update = [&](float s, float kv) { return fmaf(lam.x, s, fmaf(lam.y, s, kv)); };

  float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const int i = rg + RG * r;
    const float k = kf[i], q = qf[i];
    s[r].x = update(s[r].x, k * v[0]);
    s[r].y = update(s[r].y, k * v[1]);
    s[r].z = update(s[r].z, k * v[2]);
    s[r].w = update(s[r].w, k * v[3]);
    *reinterpret_cast<float4 *>(S + static_cast<size_t>(i) * p.dv) = s[r];
    y[0] = fmaf(s[r].x, q, y[0]);
    y[1] = fmaf(s[r].y, q, y[1]);
    y[2] = fmaf(s[r].z, q, y[2]);
    y[3] = fmaf(s[r].w, q, y[3]);
  }
  // the warp's row groups (lanes TPR apart), then the eight warps
#pragma unroll
  for (int m = TPR; m < 32; m *= 2)
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] += __shfl_xor_sync(0xffffffffu, y[c], m);
  if ((tid & 31) < TPR) *reinterpret_cast<float4 *>(&red[tid >> 5][4 * cq]) = make_float4(y[0], y[1], y[2], y[3]);
  __syncthreads();
  if (tid < W) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) t += red[w][tid];
    st_io<IO>(o + tid, p.scale * t);
  }
}

template <int DK, typename IO>
cudaError_t launch_dk(const LinDecodeProblem &p, int sms, cudaStream_t s) {
  const long nh = static_cast<long>(p.N) * p.H;
  if (2 * nh <= sms) {
    linear_decode_kernel<DK, 32, IO><<<static_cast<unsigned>(nh * (p.dv / 32)), kThreads, 0, s>>>(p);
  } else if (p.dv == 128) {
    linear_decode_kernel<DK, 128, IO><<<static_cast<unsigned>(nh), kThreads, 0, s>>>(p);
  } else {
    linear_decode_kernel<DK, 64, IO><<<static_cast<unsigned>(nh), kThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace gdr

cudaError_t gdr_launch_linear_decode(const gdr::LinDecodeProblem &p, int sms, cudaStream_t s) {
  using namespace gdr;
  if (p.dk == 128) return p.bf16_io ? launch_dk<128, __nv_bfloat16>(p, sms, s) : launch_dk<128, float>(p, sms, s);
  return p.bf16_io ? launch_dk<64, __nv_bfloat16>(p, sms, s) : launch_dk<64, float>(p, sms, s);
}
