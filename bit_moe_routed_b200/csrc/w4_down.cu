// Kernel 2 of the 4-bit layer (w4_layer.cuh): the down product and the weighted sum; above
// kW4InlineT tokens the sum is a kernel of its own.
#include "w4_layer.cuh"

namespace bitmoe {
namespace {

__global__ void __launch_bounds__(256) w4_sum_kernel(const __grid_constant__ W4LayerParams p) {
  ptx::griddep_wait();
  const int i = blockIdx.x * 256 + threadIdx.x, per = p.d / 4;
  if (i < p.T * per) w4_sum4(p, p.w_out + i / per * p.k, i / per, i % per * 4);
}

template <typename S, int G, bool ZP, bool RING, bool WIDE>
__global__ void __launch_bounds__(kW4MaxThreads, 1) w4_down_kernel(const __grid_constant__ W4LayerParams p) {
  extern __shared__ uint8_t w4_raw[];
  uint8_t* smem = w4_raw + ((1024 - (ptx::smem_u32(w4_raw) & 1023)) & 1023);
  ptx::griddep_launch_dependents();
  const W4Smem M = w4_smem<G, ZP, RING>(p.st);
  w4_init(p.st, smem, M);
  const uint32_t ready = ptx::smem_u32(smem + M.bars()) + 8 * kW4BarPlan;
  DownJob job{{p, w4_plan_at(p, smem + M.bytes()), smem + M.few(), ready},
                               reinterpret_cast<int*>(smem), reinterpret_cast<int*>(smem + M.counter()),
              reinterpret_cast<const volatile int*>(smem + M.abort_flag())};
  __syncthreads();
  if (!(WIDE ? w4_roles_wide<FP32, G, ZP, RING, false>(p.st, smem, job)
             : w4_roles<FP32, S, G, ZP, RING, false>(p.st, smem, job)))
    return;
  if (!w4_few(p.T, p.k)) w4_plan(p, job.L, smem + M.part(), ready, false);
  ptx::griddep_wait();  // h and the counts
  if constexpr (WIDE)
    w4_consume_wide<WideFP16, FP32, S, G, ZP, RING, false>(p.st, smem, job);
  else
    w4_consume<FP32, S, G, ZP, RING, false>(p.st, smem, job);
  job.finish(threadIdx.x);
}

template <typename S, int G, bool ZP, bool RING, bool WIDE>
struct DownLaunch {
  static cudaError_t run(const W4LayerParams& p, int blocks, cudaStream_t s) {
    return w4_launch<DownLaunch, G, ZP, RING>(w4_down_kernel<S, G, ZP, RING, WIDE>, p, true, blocks, s);
  }
};

}  // namespace

cudaError_t launch_w4_down(const W4LayerParams& p, bool f16, int group, bool wide, int blocks, cudaStream_t s) {
  const cudaError_t e = w4_pick<DownLaunch>(f16, group, wide, p, blocks, s);
  if (e != cudaSuccess || p.T <= kW4InlineT) return e;
  const unsigned sum_blocks = (unsigned)(((long long)p.T * (p.d / 4) + 255) / 256);
  return launch_pdl(w4_sum_kernel, dim3(sum_blocks), dim3(256), 0, s, true, p);
}

}  // namespace bitmoe
