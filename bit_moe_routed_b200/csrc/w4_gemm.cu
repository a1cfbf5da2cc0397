// C = x . W^T for up to 64 rows of x and 4-bit weights with group scales (w4.cuh): the linear
// layers of a decode step (ai-muninn.com post, "一張 22G 老卡跑 284B": decode is bound by
// reading the weights, so the weights are what gets small).
//
// One block a SM takes a contiguous range of items, 16 rows of W times a slot of rows of x; all of
// its warps share an item's reduction, so even a matrix of a few thousand rows has every SM
// reading.  Slots after the first decode the codes again; they come from L2 by then.
#include <type_traits>

#include "w4_wide.cuh"

namespace bitmoe {
namespace {

// Up to 4 rows of x take the whole-number form, more the 16-bit one, 16 rows a slot.  Both, in us
// (8192 x 4096, G = 128, bf16): 1 row 7.3 and 10.2, 4 rows 9.5 and 10.6, 5 rows 12.6 and 11.0,
// 16 rows 19.5 and 15.0, 64 rows 62 and 32.
constexpr int kW4WholeRows = 4;
constexpr int kW4WideRows = 16;

struct W4GemmParams {
  W4Stream st;
  const uint16_t* x;
  float* C;
  int M, slots;
};

// COLS: rows of x in a slot.
template <int COLS>
struct GemmJob {
  const W4GemmParams& p;
  static constexpr int kLastPart = 0;
  __device__ __forceinline__ void range(int part, int& lo, int& hi) const {
    const unsigned total = (unsigned)(p.slots * p.st.upe);  // below 2^23: 32 bits hold the products
    lo = part == 0 ? (int)(blockIdx.x * total / gridDim.x) : 0;
    hi = part == 0 ? (int)((blockIdx.x + 1) * total / gridDim.x) : 0;
  }
  __device__ __forceinline__ int matrix(int) const { return 0; }
  template <typename Wait>
  __device__ __forceinline__ bool plan(Wait) const { return true; }
  __device__ __forceinline__ bool same_rows() const { return false; }
  __device__ __forceinline__ int rows(int slot) const { return min(COLS, p.M - slot * COLS); }
  __device__ __forceinline__ const uint16_t* row(int slot, int col) const {
    const int m = slot * COLS + col;
    return m < p.M ? p.x + (size_t)m * p.st.K : nullptr;
  }
  __device__ __forceinline__ void store(int slot, int unit, int col, int r, float a, float b) const {
    const int m = slot * COLS + col, n = unit * kW4Rows + r;
    if (m >= p.M) return;
    float* c = p.C + (size_t)m * p.st.rows + n;
    if (n < p.st.rows) c[0] = a;
    if (n + 8 < p.st.rows) c[8] = b;
  }
  __device__ __forceinline__ void before_add(int) const {}
  __device__ __forceinline__ void finish(int) const {}
};

template <typename T, int G, bool ZP, bool RING>
__global__ void __launch_bounds__(kW4MaxThreads, 1) w4_gemm_kernel(const __grid_constant__ W4GemmParams p) {
  extern __shared__ uint8_t w4_raw[];
  uint8_t* smem = w4_raw + ((1024 - (ptx::smem_u32(w4_raw) & 1023)) & 1023);
  w4_init(p.st, smem, w4_smem<G, ZP, RING>(p.st));
  __syncthreads();
  GemmJob<kW4Cols> job{p};
  if (w4_roles<T, T, G, ZP, RING, false>(p.st, smem, job)) w4_consume<T, T, G, ZP, RING, false>(p.st, smem, job);
}

template <typename T, typename O, int G, bool ZP, bool RING>
__global__ void __launch_bounds__(kW4MaxThreads, 1) w4_gemm_wide_kernel(const __grid_constant__ W4GemmParams p) {
  extern __shared__ uint8_t w4_raw[];
  uint8_t* smem = w4_raw + ((1024 - (ptx::smem_u32(w4_raw) & 1023)) & 1023);
  w4_init(p.st, smem, w4_smem<G, ZP, RING>(p.st));
  __syncthreads();
  GemmJob<kW4WideRows> job{p};
  if (w4_roles_wide<T, G, ZP, RING, false>(p.st, smem, job))
    w4_consume_wide<O, T, T, G, ZP, RING, false>(p.st, smem, job);
}

template <typename T, int G, bool ZP, bool RING>
cudaError_t launch_one(const W4GemmParams& p, int blocks, int warps, cudaStream_t s) {
  using O = std::conditional_t<std::is_same_v<T, FP16>, WideFP16, WideBF16>;
  auto kern = p.M > kW4WholeRows ? w4_gemm_wide_kernel<T, O, G, ZP, RING> : w4_gemm_kernel<T, G, ZP, RING>;
  const size_t smem = (size_t)w4_smem<G, ZP, RING>(p.st).bytes() + kW4SmemPad;
  static std::atomic<unsigned long long> allowed[2];
  cudaError_t e = w4_allow_smem(kern, allowed[p.M > kW4WholeRows]);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)blocks), dim3((unsigned)w4_threads(warps)), smem, s, false, p);
}
template <typename T, int G>
cudaError_t launch_z(const W4GemmParams& p, int blocks, int warps, cudaStream_t s) {
  if (p.st.zeros0)
    return p.st.ring_scales ? launch_one<T, G, true, true>(p, blocks, warps, s)
                            : launch_one<T, G, true, false>(p, blocks, warps, s);
  return p.st.ring_scales ? launch_one<T, G, false, true>(p, blocks, warps, s)
                          : launch_one<T, G, false, false>(p, blocks, warps, s);
}
template <typename T>
cudaError_t launch_g(const W4GemmParams& p, int group, int blocks, int warps, cudaStream_t s) {
  if (group == 32) return launch_z<T, 32>(p, blocks, warps, s);
  if (group == 64) return launch_z<T, 64>(p, blocks, warps, s);
  return launch_z<T, 128>(p, blocks, warps, s);
}

}  // namespace

cudaError_t launch_w4_gemm(const W4GemmLaunch& a, cudaStream_t s, int num_sms) {
  W4GemmParams p{};
  if (!w4_set_stream(p.st, {a.codes, a.scales, a.zeros}, nullptr, 1, a.N, a.K, a.group))
    return cudaErrorInvalidValue;
  p.st.wait_ns = a.wait_ns;
  p.st.status = a.status;
  p.x = a.x;
  p.C = a.C;
  p.M = a.M;
  const int cols = a.M > kW4WholeRows ? kW4WideRows : kW4Cols;
  p.slots = (a.M + cols - 1) / cols;
  const long long total = (long long)p.slots * p.st.upe;
  const int warps = p.st.kw * p.st.teams;
  const int blocks = (int)(total < num_sms ? total : num_sms);
  return a.f16 ? launch_g<FP16>(p, a.group, blocks, warps, s) : launch_g<BF16>(p, a.group, blocks, warps, s);
}

}  // namespace bitmoe
