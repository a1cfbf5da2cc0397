// The whole MoE layer for up to 64 tokens on 4-bit weights with group scales, in two kernels.
//
// Per token: the top-k of its router scores, g = Wg[e] x, u = Wu[e] x, h = silu(g) u,
// y = Wd[e] h for each selected expert e (and the shared one), and
// out = y_shared + sum_j w_j y_j with w_j = sigmoid(s_j) / sum sigmoid(s) (tcti.cn post,
// "补齐软件栈缺失": the router picks k routed experts beside an always-on shared one;
// dpshk.com article, "核心实现三": an expert is read once for all its tokens).
//
//   kernel 1  routing, grouping by expert, gate and up products, silu(g) u
//   kernel 2  routing and grouping again, down product, weighted sum
//
// Both are w4_stream loops over (slot, unit) items, a slot being an expert with up to 8 of
// its (token, choice) pairs, the shared expert's slots first, then the experts in ascending
// order.  What bounds them is reading the active experts' codes once.  Every block works out
// the routing and the slots for itself from the scores (one warp a token): that costs about
// a microsecond in shared memory, where a kernel of its own would cost a launch and a round
// trip through L2, and it lets kernel 2 start its weight copies before kernel 1 has
// finished.  The blocks' slots agree because pairs are ranked in (token, choice) order.
// h goes to kernel 2 as two bf16 terms, high and low: 16 significant bits, so that the fp32
// output keeps about 6e-7 of relative error, at one more MMA per fragment, which the loop
// has room for; bf16 alone would leave 1.7e-3.  Its terms cannot overflow where fp16's could.
// The weighted sum runs where the last slot of 16 output rows finishes (an acq_rel count, as
// in the single-token kernel), always in the order shared, j = 0..k-1.
#include "single_token.cuh"
#include "w4.cuh"

namespace bitmoe {
namespace {

struct W4LayerParams {
  W4Stream st;
  const float* scores;
  int T, E, k, P, shared;  // P = T * k pairs; row P + t is token t's shared-expert row
  int slots_cap;
  const uint16_t* x;       // kernel 1
  uint16_t *hh, *hl;       // h, high and low bf16 terms [rows][f]
  int32_t* idx;
  float* w_out;
  float* y;                // [rows][d] fp32
  int* cnt;                // arrivals per 16 output rows
  int units2;
  float* out;
  int f, d;
};

// The slots in shared memory: 8 pairs, the expert and the count of each; the pairs' weights.
struct W4Plan {
  uint16_t* pair;  // [slots][8]
  int16_t* e;
  int16_t* n;
  float* w;        // [P]
  int slots;
};
__host__ __device__ inline int w4_slots_cap(int T, int k, int E, int shared) {
  const int P = T * k;
  const int routed = P < E + P / kW4Cols ? P : E + P / kW4Cols;
  return routed + (shared ? (T + kW4Cols - 1) / kW4Cols : 0);
}
inline size_t w4_plan_smem(int T, int k, int E, int shared) {
  return (size_t)w4_slots_cap(T, k, E, shared) * 20 + (size_t)T * k * 4 + 16 + 4 * kW4Batch * kW4MaxWarps;
}

__device__ __forceinline__ void w4_route(const float* scores, int E, int k, int lane, int* slot_e,
                                         float* w, int* pos) {
  if (E <= 256)
    route_token_warp<8>(scores, E, k, lane, slot_e, nullptr, nullptr, w, pos, nullptr, nullptr, nullptr, nullptr);
  else if (E <= 512)
    route_token_warp<16>(scores, E, k, lane, slot_e, nullptr, nullptr, w, pos, nullptr, nullptr, nullptr, nullptr);
  else
    route_token_warp<32>(scores, E, k, lane, slot_e, nullptr, nullptr, w, pos, nullptr, nullptr, nullptr, nullptr);
}

// Routing and slots.  scratch: shared memory that the stream uses later (at least
// 8 P + 8 E + 256 bytes a warp).  With `emit` the block writes idx and w.
__device__ __forceinline__ W4Plan w4_plan(const W4LayerParams& p, uint8_t* at, uint8_t* scratch,
                                          bool emit) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  W4Plan L;
  L.w = reinterpret_cast<float*>(at);
  L.pair = reinterpret_cast<uint16_t*>(at + (((size_t)p.P * 4 + 15) & ~(size_t)15));
  L.e = reinterpret_cast<int16_t*>(L.pair + (size_t)p.slots_cap * 8);
  L.n = L.e + p.slots_cap;
  int* se = reinterpret_cast<int*>(scratch);  // expert of a pair
  int* rank = se + p.P;                       // its place among the expert's pairs
  int* cnt = rank + p.P;                      // pairs, then first slot, of an expert
  int* base = cnt + p.E;
  int* tmp = base + p.E + warp * 64;
  const int ss = p.shared ? (p.T + kW4Cols - 1) / kW4Cols : 0;
  for (int i = threadIdx.x; i < p.E; i += blockDim.x) cnt[i] = 0;
  for (int t = warp; t < p.T; t += warps) {
    w4_route(p.scores + (size_t)t * p.E, p.E, p.k, lane, tmp, L.w + t * p.k, tmp + 32);
    __syncwarp();
    if (lane < p.k) se[t * p.k + lane] = tmp[tmp[32 + lane]];
    __syncwarp();
  }
  __syncthreads();
  if (emit)
    for (int i = threadIdx.x; i < p.P; i += blockDim.x) {
      p.idx[i] = se[i];
      p.w_out[i] = L.w[i];
    }
  if (warp == 0) {
    // ranks in pair order
    for (int i0 = 0; i0 < p.P; i0 += 32) {
      const int i = i0 + lane;
      const int e = i < p.P ? se[i] : -1 - lane;
      const unsigned same = __match_any_sync(0xffffffffu, e);
      const int before = __popc(same & ((1u << lane) - 1u));
      int c = 0;
      if (i < p.P) {
        c = cnt[e];
        rank[i] = c + before;
      }
      __syncwarp();
      if (i < p.P && before == 0) cnt[e] = c + __popc(same);
      __syncwarp();
    }
    int run = ss;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < p.E ? (cnt[e] + kW4Cols - 1) / kW4Cols : 0;
      int inc = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += v;
      }
      if (e < p.E) base[e] = run + inc - n;
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) tmp[0] = run;
  }
  __syncthreads();
  L.slots = *(base + p.E);  // warp 0's tmp[0]
  for (int i = threadIdx.x; i < p.P; i += blockDim.x) {
    const int e = se[i], r = rank[i], s = base[e] + r / kW4Cols;
    L.pair[s * 8 + r % kW4Cols] = (uint16_t)i;
    if (r % kW4Cols == 0) {
      L.e[s] = (int16_t)e;
      L.n[s] = (int16_t)min(kW4Cols, cnt[e] - r);
    }
  }
  if (p.shared)
    for (int t = threadIdx.x; t < p.T; t += blockDim.x) {
      const int s = t / kW4Cols;
      L.pair[t] = (uint16_t)(p.P + t);
      if (t % kW4Cols == 0) {
        L.e[s] = (int16_t)p.E;
        L.n[s] = (int16_t)min(kW4Cols, p.T - t);
      }
    }
  __syncthreads();  // the scratch is the stream's from here on
  return L;
}

__device__ __forceinline__ int w4_atom_add_acq_rel(int* p, int v) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v)
               : "memory");
  return old;
}

struct GateUpJob {
  const W4LayerParams& p;
  const W4Plan& L;
  __device__ __forceinline__ int matrix(int slot) const { return L.e[slot]; }
  __device__ __forceinline__ void ready() const {}
  __device__ __forceinline__ const uint16_t* row(int, int slot, int col) const {
    if (col >= L.n[slot]) return nullptr;
    const int pr = L.pair[slot * 8 + col];
    const int tok = pr < p.P ? pr / p.k : pr - p.P;
    return p.x + (size_t)tok * p.d;
  }
  __device__ __forceinline__ void store(int slot, int unit, int col, int r, float g, float u) const {
    if (col >= L.n[slot]) return;
    const float h = g / (1.0f + expf(-g)) * u;
    const __nv_bfloat16 hi = __float2bfloat16_rn(h);
    const float hf = __bfloat162float(hi);
    // an infinite or NaN h has no low term
    const __nv_bfloat16 lo = __float2bfloat16_rn(fabsf(hf) <= 3.4e38f ? h - hf : 0.f);
    const size_t at = (size_t)L.pair[slot * 8 + col] * p.f + unit * 8 + r;
    p.hh[at] = __bfloat16_as_ushort(hi);
    p.hl[at] = __bfloat16_as_ushort(lo);
  }
  __device__ __forceinline__ void batch_done(int, int, int) const {}
};

struct DownJob {
  const W4LayerParams& p;
  const W4Plan& L;
  int* last;
  __device__ __forceinline__ int matrix(int slot) const { return L.e[slot]; }
  __device__ __forceinline__ void ready() const { ptx::griddep_wait(); }  // h and the counts
  __device__ __forceinline__ const uint16_t* row(int set, int slot, int col) const {
    if (col >= L.n[slot]) return nullptr;
    return (set ? p.hl : p.hh) + (size_t)L.pair[slot * 8 + col] * p.f;
  }
  __device__ __forceinline__ void store(int slot, int unit, int col, int r, float a, float b) const {
    if (col >= L.n[slot]) return;
    float* y = p.y + (size_t)L.pair[slot * 8 + col] * p.d + unit * kW4Rows + r;
    y[0] = a;
    y[8] = b;
  }
  __device__ __forceinline__ void batch_done(int, int u0, int nb) const {
    __syncthreads();
    if (threadIdx.x < nb)
      last[threadIdx.x] = w4_atom_add_acq_rel(p.cnt + u0 + threadIdx.x, 1) == L.slots - 1;
    __syncthreads();
    for (int q = 0; q < nb; ++q) {
      if (!last[q]) continue;
      for (int i = threadIdx.x; i < p.T * 4; i += blockDim.x) {
        const int t = i >> 2, m = (u0 + q) * kW4Rows + 4 * (i & 3);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.shared) a = __ldcg(reinterpret_cast<const float4*>(p.y + (size_t)(p.P + t) * p.d + m));
        for (int j = 0; j < p.k; ++j) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(p.y + (size_t)(t * p.k + j) * p.d + m));
          const float w = L.w[t * p.k + j];
          a.x = fmaf(w, v.x, a.x);
          a.y = fmaf(w, v.y, a.y);
          a.z = fmaf(w, v.z, a.z);
          a.w = fmaf(w, v.w, a.w);
        }
        *reinterpret_cast<float4*>(p.out + (size_t)t * p.d + m) = a;
      }
    }
  }
};

template <typename T, int G, bool ZP>
__global__ void __launch_bounds__(kW4MaxWarps * 32, 1) w4_gate_up_kernel(const __grid_constant__ W4LayerParams p) {
  extern __shared__ __align__(128) uint8_t w4_smem[];
  ptx::griddep_launch_dependents();
  uint8_t* at = w4_smem + (size_t)(blockDim.x >> 5) * (kW4Stages * kW4StageBytes + 2 * kW4Batch * 512);
  const W4Plan L = w4_plan(p, at, w4_smem, blockIdx.x == 0);
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.units2; i += blockDim.x) p.cnt[i] = 0;
  const long long total = (long long)L.slots * p.st.upe;
  const int lo = (int)(blockIdx.x * total / gridDim.x), hi = (int)((blockIdx.x + 1) * total / gridDim.x);
  GateUpJob job{p, L};
  w4_stream<T, T, G, ZP, 1, false, true>(p.st, w4_smem, lo, hi, job);
}

template <typename S, int G, bool ZP>
__global__ void __launch_bounds__(kW4MaxWarps * 32, 1) w4_down_kernel(const __grid_constant__ W4LayerParams p) {
  extern __shared__ __align__(128) uint8_t w4_smem[];
  uint8_t* at = w4_smem + (size_t)(blockDim.x >> 5) * (kW4Stages * kW4StageBytes + 2 * kW4Batch * 512);
  int* last = reinterpret_cast<int*>(at);
  const W4Plan L = w4_plan(p, at + 4 * kW4Batch * kW4MaxWarps, w4_smem, false);
  const long long total = (long long)L.slots * p.st.upe;
  const int lo = (int)(blockIdx.x * total / gridDim.x), hi = (int)((blockIdx.x + 1) * total / gridDim.x);
  DownJob job{p, L, last};
  w4_stream<BF16, S, G, ZP, 2, true, false>(p.st, w4_smem, lo, hi, job);
}

template <typename T, int G, bool ZP>
cudaError_t launch_both(const W4LayerParams& p1, const W4LayerParams& p2, int warps1, int warps2,
                        int blocks, cudaStream_t s) {
  auto k1 = w4_gate_up_kernel<T, G, ZP>;
  auto k2 = w4_down_kernel<T, G, ZP>;
  const size_t plan = w4_plan_smem(p1.T, p1.k, p1.E, p1.shared);
  const size_t smem1 = w4_stream_smem(warps1) + plan, smem2 = w4_stream_smem(warps2) + plan;
  cudaError_t e = cudaFuncSetAttribute(k1, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem1);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k2, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem2);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k1, dim3((unsigned)blocks), dim3((unsigned)warps1 * 32), smem1, s, false, p1);
  if (e != cudaSuccess) return e;
  return launch_pdl(k2, dim3((unsigned)blocks), dim3((unsigned)warps2 * 32), smem2, s, true, p2);
}
template <typename T, int G>
cudaError_t launch_z(const W4LayerParams& p1, const W4LayerParams& p2, int warps1, int warps2,
                     int blocks, cudaStream_t s) {
  return p1.st.m0.zeros ? launch_both<T, G, true>(p1, p2, warps1, warps2, blocks, s)
                        : launch_both<T, G, false>(p1, p2, warps1, warps2, blocks, s);
}
template <typename T>
cudaError_t launch_g(const W4LayerParams& p1, const W4LayerParams& p2, int group, int warps1,
                     int warps2, int blocks, cudaStream_t s) {
  if (group == 32) return launch_z<T, 32>(p1, p2, warps1, warps2, blocks, s);
  if (group == 64) return launch_z<T, 64>(p1, p2, warps1, warps2, blocks, s);
  return launch_z<T, 128>(p1, p2, warps1, warps2, blocks, s);
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

W4LayerLayout w4_layer_layout(int T, int k, int shared, int d, int f) {
  W4LayerLayout L{};
  const size_t R = (size_t)T * k + (shared ? T : 0);
  size_t o = 0;
  L.hh = o;
  o = up256(o + R * f * 2);
  L.hl = o;
  o = up256(o + R * f * 2);
  L.y = o;
  o = up256(o + R * d * 4);
  L.cnt = o;
  o = up256(o + (size_t)(d / kW4Rows) * 4);
  L.total = o;
  return L;
}

cudaError_t launch_w4_layer(const W4LayerLaunch& a, cudaStream_t s, int num_sms) {
  const W4LayerLayout L = w4_layer_layout(a.T, a.k, a.shared, a.d, a.f);
  W4LayerParams p{};
  p.scores = a.scores;
  p.T = a.T;
  p.E = a.E;
  p.k = a.k;
  p.P = a.T * a.k;
  p.shared = a.shared;
  p.slots_cap = w4_slots_cap(a.T, a.k, a.E, a.shared);
  p.x = a.x;
  p.hh = reinterpret_cast<uint16_t*>(a.ws + L.hh);
  p.hl = reinterpret_cast<uint16_t*>(a.ws + L.hl);
  p.y = reinterpret_cast<float*>(a.ws + L.y);
  p.cnt = reinterpret_cast<int*>(a.ws + L.cnt);
  p.idx = a.idx;
  p.w_out = a.w_out;
  p.out = a.out;
  p.f = a.f;
  p.d = a.d;
  p.units2 = a.d / kW4Rows;
  W4LayerParams p1 = p, p2 = p;
  const W4Split s1 = w4_split(a.d), s2 = w4_split(a.f);
  p1.st.m0 = {a.gate_codes, a.gate_scales, a.gate_zeros};
  p1.st.m1 = {a.up_codes, a.up_scales, a.up_zeros};
  p1.st.K = a.d;
  p1.st.rows = a.f;
  p1.st.upe = a.f / 8;
  p1.st.passes = s1.passes;
  p1.st.kw = s1.kw;
  p1.st.teams = s1.teams;
  p1.st.vec = w4_vec(a.gate_scales, a.gate_zeros, a.d, a.group) &&
              w4_vec(a.up_scales, a.up_zeros, a.d, a.group);
  p2.st.m0 = {a.down_codes, a.down_scales, a.down_zeros};
  p2.st.K = a.f;
  p2.st.rows = a.d;
  p2.st.upe = p.units2;
  p2.st.passes = s2.passes;
  p2.st.kw = s2.kw;
  p2.st.teams = s2.teams;
  p2.st.vec = w4_vec(a.down_scales, a.down_zeros, a.f, a.group);
  return a.f16 ? launch_g<FP16>(p1, p2, a.group, s1.warps(), s2.warps(), num_sms, s)
               : launch_g<BF16>(p1, p2, a.group, s1.warps(), s2.warps(), num_sms, s);
}

}  // namespace bitmoe
