// Kernel 1 of the 4-bit layer (w4_layer.cuh): routing, grouping, gate and up products,
// silu(g) u.
#include "w4_layer.cuh"

namespace bitmoe {
namespace {

template <typename T, int G, bool ZP, bool RING, bool WIDE>
__global__ void __launch_bounds__(kW4MaxThreads, 1) w4_gate_up_kernel(const __grid_constant__ W4LayerParams p) {
  extern __shared__ uint8_t w4_raw[];
  uint8_t* smem = w4_raw + ((1024 - (ptx::smem_u32(w4_raw) & 1023)) & 1023);
  ptx::griddep_launch_dependents();
  const W4Smem M = w4_smem<G, ZP, RING>(p.st);
  w4_init(p.st, smem, M);
  const uint32_t ready = ptx::smem_u32(smem + M.bars()) + 8 * kW4BarPlan;
  GateUpJob job{{p, w4_plan_at(p, smem + M.bytes()), smem + M.few(), ready}};
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.units2; i += blockDim.x) p.cnt[i] = 0;
  __syncthreads();
  if (!(WIDE ? w4_roles_wide<T, G, ZP, RING, true>(p.st, smem, job) : w4_roles<T, T, G, ZP, RING, true>(p.st, smem, job)))
    return;
  if (!w4_few(p.T, p.k)) w4_plan(p, job.L, smem + M.part(), ready, blockIdx.x == 0);
  if constexpr (WIDE)
    w4_consume_wide<std::conditional_t<std::is_same_v<T, FP16>, WideFP16, WideBF16>, T, T, G, ZP, RING, true>(p.st, smem, job);
  else
    w4_consume<T, T, G, ZP, RING, true>(p.st, smem, job);
}

template <typename T, int G, bool ZP, bool RING, bool WIDE>
struct GateUpLaunch {
  static cudaError_t run(const W4LayerParams& p, int blocks, cudaStream_t s) {
    return w4_launch<GateUpLaunch, G, ZP, RING>(w4_gate_up_kernel<T, G, ZP, RING, WIDE>, p, false, blocks, s);
  }
};

}  // namespace

cudaError_t launch_w4_gate_up(const W4LayerParams& p, bool f16, int group, bool wide, int blocks, cudaStream_t s) {
  return w4_pick<GateUpLaunch>(f16, group, wide, p, blocks, s);
}

}  // namespace bitmoe
