// Host side of the 4-bit layer: the workspace, the parameters of its two kernels.
#include "w4_layer.cuh"

namespace bitmoe {
namespace {

// Whether a call takes the 16-bit form: where an expert has four pairs and more on average (32
// tokens, 16 experts, k = 4, d = 2048, f = 1408: 87 us against 121 in whole numbers).
bool w4_wide(int T, int k, int E) { return T > 8 && T * k >= 4 * E; }

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

W4LayerLayout w4_layer_layout(int T, int k, int shared, int d, int f) {
  W4LayerLayout L{};
  const size_t R = (size_t)T * k + (shared ? T : 0);
  size_t o = 0;
  L.h = o;
  o = up256(o + R * f * 4);
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
  p.x = a.x;
  p.h = reinterpret_cast<float*>(a.ws + L.h);
  p.y = reinterpret_cast<float*>(a.ws + L.y);
  p.cnt = reinterpret_cast<int*>(a.ws + L.cnt);
  p.idx = a.idx;
  p.w_out = a.w_out;
  p.out = a.out;
  p.f = a.f;
  p.d = a.d;
  p.units2 = a.d / kW4Rows;
  p.st.wait_ns = a.wait_ns;
  p.st.status = a.status;
  W4LayerParams p1 = p, p2 = p;
  const bool wide = w4_wide(a.T, a.k, a.E);
  p1.sc = wide ? 8 * kW4WideSets : kW4Cols;
  p2.sc = wide ? 8 : kW4Cols;
  p1.sc_log2 = wide ? 4 : 2;
  p2.sc_log2 = wide ? 3 : 2;
  p1.shared_slots = a.shared ? (a.T + p1.sc - 1) / p1.sc : 0;
  p2.shared_slots = a.shared ? (a.T + p2.sc - 1) / p2.sc : 0;
  p1.inv_k = p2.inv_k = (65536u + a.k - 1) / a.k;
  p1.slots_cap = w4_slots_cap(a.T, a.k, a.E, a.shared, p1.sc);
  p2.slots_cap = w4_slots_cap(a.T, a.k, a.E, a.shared, p2.sc);
  const long long n = a.E + a.shared;
  const W4Mat gate{a.gate_codes, a.gate_scales, a.gate_zeros}, up{a.up_codes, a.up_scales, a.up_zeros};
  if (!w4_set_stream(p1.st, gate, &up, n, a.f, a.d, a.group) ||
      !w4_set_stream(p2.st, {a.down_codes, a.down_scales, a.down_zeros}, nullptr, n, a.d, a.f, a.group))
    return cudaErrorInvalidValue;
  const cudaError_t e = launch_w4_gate_up(p1, a.f16, a.group, wide, num_sms, s);
  return e == cudaSuccess ? launch_w4_down(p2, a.f16, a.group, wide, num_sms, s) : e;
}

}  // namespace bitmoe
