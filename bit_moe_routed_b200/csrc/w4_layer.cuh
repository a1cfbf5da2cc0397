// The whole MoE layer for up to 64 tokens on 4-bit weights with group scales, in two kernels.
//
// Per token: the top-k of its router scores, g = Wg[e] x, u = Wu[e] x, h = silu(g) u,
// y = Wd[e] h for each selected expert e (and the shared one), and
// out = y_shared + sum_j w_j y_j with w_j = sigmoid(s_j) / sum sigmoid(s) (tcti.cn post,
// "补齐软件栈缺失": the router picks k routed experts beside an always-on shared one;
// dpshk.com article, "核心实现三": an expert is read once for all its tokens).
//
//   kernel 1  routing, grouping by expert, gate and up products, silu(g) u
//   kernel 2  routing and grouping again, down product, weighted sum (up to 8 tokens; with
//             more a third, small one adds up)
//
// Both products are streams (w4.cuh) over (slot, unit) items, a slot being an expert with a few
// of its (token, choice) pairs, the shared expert's slots first, then the experts.  The floor is
// reading the active experts' codes once.  Every block works out the routing and the slots for
// itself from the scores, one warp a token: that costs 2 to 5 us in shared memory, most of it
// behind the first copies or kernel 1's last units, where a kernel of its own would cost a launch
// and a round trip through L2, and it lets kernel 2 start its weight copies before kernel 1 has
// finished.  The blocks' slots agree because pairs are ranked in (token, choice) order.
// h stays fp32 in the workspace and enters the down product as x does the first two, with 30 or
// 22 significant bits (w4.cuh, w4_wide.cuh); in 16 bits it would leave 1.7e-3 (bf16) of relative
// error in an fp32 output.
// Every sum has one order: slices, then y_shared and j = 0..k-1, so a call is deterministic.
//
// Measured (device, us; d = 4096, f = 2048, E = 256, k = 6, a shared expert, G = 128): 1 token 40
// (2.3 TB/s), 16 tokens 202, 64 tokens 540, both with Zipf(1) routing.
#pragma once
#include <type_traits>

#include "single_token.cuh"
#include "w4_wide.cuh"

namespace bitmoe {

struct W4LayerParams {
  W4Stream st;
  const float* scores;
  int T, E, k, P, shared;  // P = T * k pairs; row P + t is token t's shared-expert row
  int sc, sc_log2;         // most pairs of a slot: 4, 8 or 16
  int shared_slots;
  unsigned inv_k;          // pair / k = pair * inv_k >> 16 (pair < 2048, k <= 32)
  int slots_cap;
  const uint16_t* x;       // kernel 1
  float* h;                // [rows][f]
  int32_t* idx;
  float* w_out;
  float* y;                // [rows][d] fp32
  int* cnt;                // arrivals per 16 output rows
  int units2;
  float* out;
  int f, d;
};

namespace {

// The slots in shared memory: up to sc pairs, the expert and the count of each; the
// pairs' weights.  The shared expert's slots, the first, are known without them: slot s has
// tokens s * sc and up.
struct W4Plan {
  uint16_t* pair;  // [slots][sc]
  int16_t* e;
  uint8_t* n;
  float* w;        // [P]
  int* total;      // slots
};
inline int w4_slots_cap(int T, int k, int E, int shared, int sc) {
  const int P = T * k;
  const int routed = P < E + P / sc ? P : E + P / sc;
  return routed + (shared ? (T + sc - 1) / sc : 0);
}
inline size_t w4_plan_smem(const W4LayerParams& p) {
  return (size_t)p.slots_cap * (2 * p.sc + 3) + (size_t)p.P * 4 + 16 + 16;
}
__device__ __forceinline__ W4Plan w4_plan_at(const W4LayerParams& p, uint8_t* at) {
  W4Plan L;
  L.total = reinterpret_cast<int*>(at);
  L.w = reinterpret_cast<float*>(at + 16);
  L.pair = reinterpret_cast<uint16_t*>(at + 16 + (((size_t)p.P * 4 + 15) & ~(size_t)15));
  L.e = reinterpret_cast<int16_t*>(L.pair + (size_t)p.slots_cap * p.sc);
  L.n = reinterpret_cast<uint8_t*>(L.e + p.slots_cap);
  return L;
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

// Routing and slots, by the consuming warps, which then let the copying warp at them.
// scratch: the memory of the stream's sums (2 KB a warp; it takes 4 P + 4 E + 256 bytes a warp,
// at most 14.6 KB of the 18 KB of the fewest warps, 9, with 64 tokens, k = 32, E = 1024).  With
// `emit` the block writes idx and w.
__device__ __forceinline__ void w4_plan(const W4LayerParams& p, const W4Plan& L, uint8_t* scratch, uint32_t ready,
                                        bool emit) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warps = p.st.kw * p.st.teams, threads = warps * 32;
  int* tmp = reinterpret_cast<int*>(scratch) + warp * 64;
  int* sum = reinterpret_cast<int*>(scratch);  // a warp's slots (after the routing)
  uint16_t* se = reinterpret_cast<uint16_t*>(scratch + warps * 256);  // expert of a pair
  uint16_t* rank = se + p.P;                   // its place among the expert's pairs
  uint16_t* cnt = rank + p.P;                  // pairs of an expert
  uint16_t* base = cnt + p.E;                  // its first slot
  const int ss = p.shared_slots;
  for (int i = threadIdx.x; i < p.E; i += threads) cnt[i] = 0;
  for (int t = warp; t < p.T; t += warps) {
    w4_route(p.scores + (size_t)t * p.E, p.E, p.k, lane, tmp, L.w + t * p.k, tmp + 32);
    __syncwarp();
    if (lane < p.k) se[t * p.k + lane] = (uint16_t)tmp[tmp[32 + lane]];
    __syncwarp();
  }
  w4_sync(p.st);
  if (emit)
    for (int i = threadIdx.x; i < p.P; i += threads) {
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
        rank[i] = (uint16_t)(c + before);
      }
      __syncwarp();
      if (i < p.P && before == 0) cnt[e] = (uint16_t)(c + __popc(same));
      __syncwarp();
    }
  }
  w4_sync(p.st);
  // first slots: each warp takes a run of experts, 32 at a time
  const int per = (p.E + 32 * warps - 1) / (32 * warps) * 32;
  int run = 0;
  for (int e0 = warp * per; e0 < min(p.E, (warp + 1) * per); e0 += 32) {
    const int e = e0 + lane;
    const int n = e < p.E ? (cnt[e] + p.sc - 1) >> p.sc_log2 : 0;
    int inc = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += v;
    }
    if (e < p.E) base[e] = (uint16_t)(run + inc - n);
    run += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) sum[warp] = run;
  w4_sync(p.st);
  for (int i = threadIdx.x; i < p.P; i += threads) {
    const int e = se[i], r = rank[i];
    int s = ss + base[e] + (r >> p.sc_log2);
    for (int w = 0; w < e / per; ++w) s += sum[w];
    L.pair[s * p.sc + (r & (p.sc - 1))] = (uint16_t)i;
    if ((r & (p.sc - 1)) == 0) {
      L.e[s] = (int16_t)e;
      L.n[s] = (uint8_t)min(p.sc, cnt[e] - r);
    }
  }
  if (threadIdx.x == 0) {
    int s = ss;
    for (int w = 0; w < warps; ++w) s += sum[w];
    *L.total = s;
  }
  w4_sync(p.st);  // the scratch is the stream's from here on
  // the copying and adding warps may read the slots
  if (threadIdx.x == 0) ptx::mbar_arrive(ready);
}

// The same for up to 4 tokens with up to 32 pairs, by the adding warps, while the consuming ones
// begin with the shared expert: no expert has more pairs than a slot takes, so a slot is an
// expert, in the order in which the pairs name them.  scratch: 256 bytes a warp and 32 ints.
__host__ __device__ inline bool w4_few(int T, int k) { return T <= kW4Cols && T * k <= 32; }
__device__ __forceinline__ void w4_plan_few(const W4LayerParams& p, const W4Plan& L, uint8_t* scratch,
                                            uint32_t ready, int tid, bool emit) {
  const int warp = tid >> 5, lane = tid & 31, ss = p.shared ? 1 : 0;
  int* se = reinterpret_cast<int*>(scratch);
  int* tmp = se + 32 + warp * 64;
  for (int t = warp; t < p.T; t += kW4SumThreads / 32) {
    w4_route(p.scores + (size_t)t * p.E, p.E, p.k, lane, tmp, L.w + t * p.k, tmp + 32);
    __syncwarp();
    if (lane < p.k) se[t * p.k + lane] = tmp[tmp[32 + lane]];
    __syncwarp();
  }
  asm volatile("bar.sync 3, %0;" ::"n"(kW4SumThreads) : "memory");
  if (warp == 0) {
    const int e = lane < p.P ? se[lane] : -1 - lane;
    const unsigned same = __match_any_sync(0xffffffffu, e), lower = (1u << lane) - 1u;
    const bool first = lane < p.P && (same & lower) == 0;
    const unsigned firsts = __ballot_sync(0xffffffffu, first);
    const int s = ss + __popc(firsts & ((1u << (__ffs(same) - 1)) - 1u));
    if (lane < p.P) {
      L.pair[s * kW4Cols + __popc(same & lower)] = (uint16_t)lane;
      if (first) {
        L.e[s] = (int16_t)e;
        L.n[s] = (uint8_t)__popc(same);
      }
      if (emit) {
        p.idx[lane] = e;
        p.w_out[lane] = L.w[lane];
      }
    }
    if (lane == 0) *L.total = ss + __popc(firsts);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ready);
  }
}

// What both kernels' jobs share: the slots, and the block's items.  A block takes its share of
// the shared expert's units first: that needs no routing, and those units, with the most rows
// of x, are spread evenly.  Up to 2 tokens all units cost the same and kernel 2, whose routing is
// done by the time that kernel 1 has finished, takes one run of everything, a slot less to load
// h for (1 token, d = f = 512: 20 us a layer against 23; 4 tokens, d = 4096, f = 2048: 120
// against 111, so there the shared units stay first).
struct LayerJob {
  const W4LayerParams& p;
  W4Plan L;
  uint8_t* scratch;  // for w4_plan_few
  uint32_t ready;    // barrier: the slots are known
  static constexpr int kLastPart = 1;
  // at most 2^22 items: 32 bits hold the products
  __device__ __forceinline__ void whole_range(int part, int& lo, int& hi) const {
    lo = hi = 0;
    if (part == 0) return;
    const unsigned all = (unsigned)(*L.total * p.st.upe), G = gridDim.x, b = blockIdx.x;
    lo = (int)(b * all / G);
    hi = (int)((b + 1) * all / G);
  }
  __device__ __forceinline__ void shared_first_range(int part, int& lo, int& hi) const {
    const unsigned S = (unsigned)(p.shared_slots * p.st.upe), G = gridDim.x, b = blockIdx.x;
    const unsigned s0 = b * S / G, s1 = (b + 1) * S / G;
    lo = (int)s0;
    hi = (int)s1;
    if (part == 0) return;
    const unsigned all = (unsigned)(*L.total * p.st.upe);
    if (all - S >= G) {  // whole shares of everything, less the block's shared items
      lo = (int)(S + b * all / G - s0);
      hi = (int)(S + (b + 1) * all / G - s1);
    } else {
      lo = (int)(S + b * (all - S) / G);
      hi = (int)(S + (b + 1) * (all - S) / G);
    }
  }
  __device__ __forceinline__ int matrix(int slot) const { return slot < p.shared_slots ? p.E : L.e[slot]; }
  template <typename Wait>
  __device__ __forceinline__ bool plan(Wait wait) const { return wait(); }
  __device__ __forceinline__ int rows(int slot) const {
    return slot < p.shared_slots ? min(p.sc, p.T - slot * p.sc) : L.n[slot];
  }
  // the y row (and row of h) of a column
  __device__ __forceinline__ int pair(int slot, int col) const {
    return slot < p.shared_slots ? p.P + slot * p.sc + col : L.pair[slot * p.sc + col];
  }
};

__device__ __forceinline__ int w4_atom_add_acq_rel(int* p, int v) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v)
               : "memory");
  return old;
}

struct GateUpJob : LayerJob {
  __device__ __forceinline__ void range(int part, int& lo, int& hi) const { shared_first_range(part, lo, hi); }
  __device__ __forceinline__ const uint16_t* row(int slot, int col) const {
    if (col >= rows(slot)) return nullptr;
    const int pr = pair(slot, col);
    return p.x + (size_t)(pr < p.P ? (int)((unsigned)pr * p.inv_k >> 16) : pr - p.P) * p.d;
  }
  __device__ __forceinline__ void store(int slot, int unit, int col, int r, float g, float u) const {
    p.h[(size_t)pair(slot, col) * p.f + unit * 8 + r] = g / (1.0f + expf(-g)) * u;
  }
  __device__ __forceinline__ bool same_rows() const { return p.T == 1; }
  __device__ __forceinline__ void before_add(int tid) const {
    if (w4_few(p.T, p.k)) w4_plan_few(p, L, scratch, ready, tid, blockIdx.x == 0);
  }
  __device__ __forceinline__ void finish(int) const {}
};

// The weighted sum of four outputs of token t.
__device__ __forceinline__ void w4_sum4(const W4LayerParams& p, const float* w, int t, int m) {
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.shared) a = __ldcg(reinterpret_cast<const float4*>(p.y + (size_t)(p.P + t) * p.d + m));
  for (int j0 = 0; j0 < p.k; j0 += 8) {
    float4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j0 + j < p.k)
        v[j] = __ldcg(reinterpret_cast<const float4*>(p.y + (size_t)(t * p.k + j0 + j) * p.d + m));
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j0 + j < p.k) {
        const float c = w[j0 + j];
        a.x = fmaf(c, v[j].x, a.x);
        a.y = fmaf(c, v[j].y, a.y);
        a.z = fmaf(c, v[j].z, a.z);
        a.w = fmaf(c, v[j].w, a.w);
      }
  }
  *reinterpret_cast<float4*>(p.out + (size_t)t * p.d + m) = a;
}

// Up to kW4InlineT tokens the block that finishes a unit's last slot adds the unit's rows up,
// all of its threads together, after its last store.  With more tokens the last blocks would
// have most of the sum to themselves; there a third kernel does it.
constexpr int kW4InlineT = 8;
struct DownJob : LayerJob {
  int* list;   // [units2], in memory that the stream has finished with
  int* count;  // 0 at the start
  const volatile int* aborted;  // a wait of the block has run out: nothing to add up
  __device__ __forceinline__ void range(int part, int& lo, int& hi) const {
    if (p.T <= kW4SetRows)
      whole_range(part, lo, hi);
    else
      shared_first_range(part, lo, hi);
  }
  __device__ __forceinline__ const float* row(int slot, int col) const {
    return col < rows(slot) ? p.h + (size_t)pair(slot, col) * p.f : nullptr;
  }
  __device__ __forceinline__ void store(int slot, int unit, int col, int r, float a, float b) const {
    float* y = p.y + (size_t)pair(slot, col) * p.d + unit * kW4Rows + r;
    y[0] = a;
    y[8] = b;
  }
  __device__ __forceinline__ bool same_rows() const { return false; }
  __device__ __forceinline__ void before_add(int tid) const {
    if (w4_few(p.T, p.k)) w4_plan_few(p, L, scratch, ready, tid, false);
    ptx::griddep_wait();
  }
  // by all consuming and adding threads
  __device__ __forceinline__ void finish(int tid) const {
    if (p.T > kW4InlineT) return;
    const int threads = p.st.kw * p.st.teams * 32 + kW4SumThreads;
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");  // every store
    if (*aborted) return;
    for (int part = 0; part < 2; ++part) {
      int lo, hi;
      range(part, lo, hi);
      for (int i = lo + tid; i < hi; i += threads) {
        const int u = i % p.st.upe;
        if (w4_atom_add_acq_rel(p.cnt + u, 1) == *L.total - 1) list[atomicAdd(count, 1)] = u;
      }
    }
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
    const int work = *count * p.T * 4;
    for (int i = tid; i < work; i += threads) {
      const int t = (i >> 2) % p.T;
      w4_sum4(p, L.w + t * p.k, t, list[(i >> 2) / p.T] * kW4Rows + 4 * (i & 3));
    }
  }
};

}  // namespace

// Kernel 1 and kernel 2 (w4_gate_up.cu, w4_down.cu); wide: the 16-bit form.
cudaError_t launch_w4_gate_up(const W4LayerParams& p, bool f16, int group, bool wide, int blocks, cudaStream_t s);
cudaError_t launch_w4_down(const W4LayerParams& p, bool f16, int group, bool wide, int blocks, cudaStream_t s);

namespace {
// The instantiation of F<T, G, ZP, RING, WIDE> for a call.
template <template <typename, int, bool, bool, bool> class F, typename T, int G, bool ZP>
cudaError_t w4_pick_rw(bool wide, const W4LayerParams& p, int blocks, cudaStream_t s) {
  if (wide)
    return p.st.ring_scales ? F<T, G, ZP, true, true>::run(p, blocks, s) : F<T, G, ZP, false, true>::run(p, blocks, s);
  return p.st.ring_scales ? F<T, G, ZP, true, false>::run(p, blocks, s) : F<T, G, ZP, false, false>::run(p, blocks, s);
}
template <template <typename, int, bool, bool, bool> class F, typename T, int G>
cudaError_t w4_pick_z(bool wide, const W4LayerParams& p, int blocks, cudaStream_t s) {
  return p.st.zeros0 ? w4_pick_rw<F, T, G, true>(wide, p, blocks, s) : w4_pick_rw<F, T, G, false>(wide, p, blocks, s);
}
template <template <typename, int, bool, bool, bool> class F, typename T>
cudaError_t w4_pick_g(int group, bool wide, const W4LayerParams& p, int blocks, cudaStream_t s) {
  if (group == 32) return w4_pick_z<F, T, 32>(wide, p, blocks, s);
  if (group == 64) return w4_pick_z<F, T, 64>(wide, p, blocks, s);
  return w4_pick_z<F, T, 128>(wide, p, blocks, s);
}
template <template <typename, int, bool, bool, bool> class F>
cudaError_t w4_pick(bool f16, int group, bool wide, const W4LayerParams& p, int blocks, cudaStream_t s) {
  return f16 ? w4_pick_g<F, FP16>(group, wide, p, blocks, s) : w4_pick_g<F, BF16>(group, wide, p, blocks, s);
}
// Id: a type of the kernel's own, so that each has its `allowed`.
template <typename Id, int G, bool ZP, bool RING, typename Kernel>
cudaError_t w4_launch(Kernel kern, const W4LayerParams& p, bool overlap, int blocks, cudaStream_t s) {
  const size_t smem = w4_smem<G, ZP, RING>(p.st).bytes() + w4_plan_smem(p) + kW4SmemPad;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = w4_allow_smem(kern, allowed);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)blocks), dim3((unsigned)w4_threads(p.st.kw * p.st.teams)), smem, s, overlap, p);
}
}  // namespace
}  // namespace bitmoe
