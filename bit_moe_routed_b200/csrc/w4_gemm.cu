// C = x . W^T for up to 64 rows of x and 4-bit weights with group scales (w4.cuh): the linear
// layers of a decode step (ai-muninn.com post, "一張 22G 老卡跑 284B": decode is bound by
// reading the weights, so the weights are what gets small).
//
// One block a SM takes a contiguous range of items (16 rows of W times 8 or 16 rows of x); all
// of its warps share an item's reduction, so even a matrix of a few thousand rows has every
// SM reading.  More than 8 rows of x take two B sets per decoded word (64 registers instead
// of 32), which halves how often the codes are decoded and fetched from L2; the decode, not
// the MMAs, is what bounds a large batch.
#include "w4.cuh"

namespace bitmoe {
namespace {

struct W4GemmParams {
  W4Stream st;
  const uint16_t* x;
  float* C;
  int M, slots;
};

template <int NB>
struct GemmJob {
  const W4GemmParams& p;
  __device__ __forceinline__ int matrix(int) const { return 0; }
  __device__ __forceinline__ void ready() const {}
  __device__ __forceinline__ const uint16_t* row(int set, int slot, int col) const {
    const int m = (slot * NB + set) * kW4Cols + col;
    return m < p.M ? p.x + (size_t)m * p.st.K : nullptr;
  }
  __device__ __forceinline__ void store(int slot, int unit, int col, int r, float a, float b) const {
    const int m = slot * NB * kW4Cols + col, n = unit * kW4Rows + r;
    if (m >= p.M) return;
    float* c = p.C + (size_t)m * p.st.rows + n;
    if (n < p.st.rows) c[0] = a;
    if (n + 8 < p.st.rows) c[8] = b;
  }
  __device__ __forceinline__ void batch_done(int, int, int) const {}
};

template <typename T, int G, bool ZP, int NB>
__global__ void __launch_bounds__(kW4MaxWarps * 32, 1) w4_gemm_kernel(const __grid_constant__ W4GemmParams p) {
  extern __shared__ __align__(128) uint8_t w4_smem[];
  const long long total = (long long)p.slots * p.st.upe;
  const int lo = (int)(blockIdx.x * total / gridDim.x), hi = (int)((blockIdx.x + 1) * total / gridDim.x);
  GemmJob<NB> job{p};
  w4_stream<T, T, G, ZP, NB, false, false>(p.st, w4_smem, lo, hi, job);
}

template <typename T, int G, bool ZP, int NB>
cudaError_t launch_one(const W4GemmParams& p, int blocks, int warps, cudaStream_t s) {
  auto kern = w4_gemm_kernel<T, G, ZP, NB>;
  const size_t smem = w4_stream_smem(warps);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)blocks), dim3((unsigned)warps * 32), smem, s, false, p);
}
template <typename T, int G, bool ZP>
cudaError_t launch_nb(const W4GemmParams& p, int nb, int blocks, int warps, cudaStream_t s) {
  return nb == 1 ? launch_one<T, G, ZP, 1>(p, blocks, warps, s) : launch_one<T, G, ZP, 2>(p, blocks, warps, s);
}
template <typename T, int G>
cudaError_t launch_z(const W4GemmParams& p, int nb, int blocks, int warps, cudaStream_t s) {
  return p.st.m0.zeros ? launch_nb<T, G, true>(p, nb, blocks, warps, s)
                       : launch_nb<T, G, false>(p, nb, blocks, warps, s);
}
template <typename T>
cudaError_t launch_g(const W4GemmParams& p, int group, int nb, int blocks, int warps, cudaStream_t s) {
  if (group == 32) return launch_z<T, 32>(p, nb, blocks, warps, s);
  if (group == 64) return launch_z<T, 64>(p, nb, blocks, warps, s);
  return launch_z<T, 128>(p, nb, blocks, warps, s);
}

}  // namespace

cudaError_t launch_w4_gemm(const W4GemmLaunch& a, cudaStream_t s, int num_sms) {
  W4GemmParams p{};
  const W4Split sp = w4_split(a.K);
  p.st.m0 = {a.codes, a.scales, a.zeros};
  p.st.K = a.K;
  p.st.rows = a.N;
  p.st.upe = (a.N + kW4Rows - 1) / kW4Rows;
  p.st.passes = sp.passes;
  p.st.kw = sp.kw;
  p.st.teams = sp.teams;
  p.st.vec = w4_vec(a.scales, a.zeros, a.K, a.group);
  p.x = a.x;
  p.C = a.C;
  p.M = a.M;
  const int nb = a.M > kW4Cols ? 2 : 1;
  p.slots = (a.M + nb * kW4Cols - 1) / (nb * kW4Cols);
  const long long total = (long long)p.slots * p.st.upe;
  const int blocks = (int)(total < num_sms ? total : num_sms);
  return a.f16 ? launch_g<FP16>(p, a.group, nb, blocks, sp.warps(), s)
               : launch_g<BF16>(p, a.group, nb, blocks, sp.warps(), s);
}

}  // namespace bitmoe
