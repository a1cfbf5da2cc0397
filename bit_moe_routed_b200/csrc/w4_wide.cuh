// The stream of w4.cuh for slots of more rows of x: up to 16 a slot, in 16-bit operands.
//
// The whole-number form spends four MMA columns on a row of x, so past a few rows the tensor
// core and the decodes of one slot after another set its pace.  Here q - z becomes a bf16 or
// fp16 operand (an integer of at most 8 bits: exact), x enters as it is, and one decode serves
// two MMAs of 8 rows each: 9 (fp16) or 11 (bf16) instructions a word of 8 codes instead of 3,
// but for 16 rows of x instead of 4.  The group's sum is fp32 in the tensor core, the scale
// follows in fp32.  fp32 rows (TERMS: the hidden state) take two fp16 terms, high and low, after
// a power of two per slice as in the whole-number form: 22 significant bits, 8 rows a slot.
#pragma once
#include "w4.cuh"

namespace bitmoe {
namespace {

constexpr int kW4WideSets = 2;  // B sets of a warp, 8 columns each, 32 registers each

struct WideBF16 {
  static constexpr bool kHalf = false;
  static constexpr uint32_t kOne = 0x43004300u;  // 128: one unit in the last place is 1
};
struct WideFP16 {
  static constexpr bool kHalf = true;
  static constexpr uint32_t kOne = 0x64006400u;   // 1024: likewise
  static constexpr uint32_t kHigh = 0x54005400u;  // 64: here a nibble at bit 4 counts in ones
  static constexpr uint32_t kDiff = 0x63806380u;  // 960
};
template <typename O>
__device__ __forceinline__ uint32_t w4_sub2(uint32_t a, uint32_t b) {
  if constexpr (O::kHalf) {
    const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}
// (v & mask) | bits in one instruction
__device__ __forceinline__ uint32_t w4_set(uint32_t v, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(mask), "r"(bits));
  return r;
}
// A word's 8 codes less the zero point as the pairs (0,4) (1,5) (2,6) (3,7).  lo, hi: the zero
// point over the bases of a nibble at bit 0 and (fp16) at bit 4.
template <typename O>
__device__ __forceinline__ void w4_decode16(uint32_t v, uint32_t lo, uint32_t hi, uint32_t (&a)[4]) {
  if constexpr (O::kHalf) {
    const uint32_t u = v >> 8;
    a[0] = w4_sub2<O>(w4_set(v, 0x000F000Fu, O::kOne), lo);
    a[1] = w4_sub2<O>(w4_set(v, 0x00F000F0u, O::kHigh), hi);
    a[2] = w4_sub2<O>(w4_set(u, 0x000F000Fu, O::kOne), lo);
    a[3] = w4_sub2<O>(w4_set(u, 0x00F000F0u, O::kHigh), hi);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = w4_sub2<O>(w4_set(v >> (4 * i), 0x000F000Fu, O::kOne), lo);
  }
}
template <typename O, bool ZP>
__device__ __forceinline__ void w4_offsets(int z, uint32_t& lo, uint32_t& hi) {
  lo = O::kOne | (ZP ? (uint32_t)z * 0x00010001u : 0x00080008u);
  if constexpr (O::kHalf) hi = ZP ? w4_sub2<O>(lo, O::kDiff) : (O::kHigh + 0x00800080u);
}
template <typename O>
__device__ __forceinline__ void w4_mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (O::kHalf)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3},"
        " {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3},"
        " {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One task: 16 rows times SETS sets; tot[n]: rows g and g + 8, columns 2t and 2t + 1 as the MMA
// has them.
template <typename O, typename S, int G, bool ZP, int SETS>
__device__ __forceinline__ void w4_task16(uint32_t at, const W4RowScales<G, ZP>& r0, const W4RowScales<G, ZP>& r1,
                                          const uint32_t (&bx)[kW4WideSets][8][4], uint32_t pair,
                                          float (&tot)[kW4WideSets][4]) {
  constexpr int SG = G / 32;
#pragma unroll
  for (int b = 0; b < kW4Chunk / G; ++b) {
    uint32_t w0[SG], w1[SG];
    w4_lds(at ^ (uint32_t)(b * (G / 2)), w0);
    w4_lds((at ^ (uint32_t)(b * (G / 2))) + pair, w1);
    uint32_t lo0, hi0, lo1, hi1;
    w4_offsets<O, ZP>(ZP ? r0.zero(b) : 8, lo0, hi0);
    w4_offsets<O, ZP>(ZP ? r1.zero(b) : 8, lo1, hi1);
    float acc[SETS][4];
#pragma unroll
    for (int n = 0; n < SETS; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
    for (int i = 0; i < SG; ++i) {
      uint32_t a0[4], a1[4];
      w4_decode16<O>(w0[i], lo0, hi0, a0);
      w4_decode16<O>(w1[i], lo1, hi1, a1);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < SETS; ++n)
          w4_mma16<O>(acc[n], a0[2 * h], a1[2 * h], a0[2 * h + 1], a1[2 * h + 1], bx[n][SG * b + i][2 * h],
                      bx[n][SG * b + i][2 * h + 1]);
    }
    const float s0 = r0.template scale<S>(b), s1 = r1.template scale<S>(b);
#pragma unroll
    for (int n = 0; n < SETS; ++n) {
      tot[n][0] = b == 0 ? s0 * acc[n][0] : fmaf(s0, acc[n][0], tot[n][0]);
      tot[n][1] = b == 0 ? s0 * acc[n][1] : fmaf(s0, acc[n][1], tot[n][1]);
      tot[n][2] = b == 0 ? s1 * acc[n][2] : fmaf(s1, acc[n][2], tot[n][2]);
      tot[n][3] = b == 0 ? s1 * acc[n][3] : fmaf(s1, acc[n][3], tot[n][3]);
    }
  }
}

// B set of a 16-bit row (NULL: zeros), in the order in which the codes of a word come apart.
template <int G>
__device__ __forceinline__ void w4_load_b16(uint32_t (&bx)[8][4], const uint16_t* row, int valid, int t) {
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (row != nullptr && s / (G / 32) < valid) v = *reinterpret_cast<const uint4*>(row + w4_step<G>(s, t));
    bx[s][0] = ptx::prmt(v.x, v.z, 0x5410);
    bx[s][1] = ptx::prmt(v.x, v.z, 0x7632);
    bx[s][2] = ptx::prmt(v.y, v.w, 0x5410);
    bx[s][3] = ptx::prmt(v.y, v.w, 0x7632);
  }
}
// Both sets of an fp32 row: its high and low fp16 terms after a power of two that brings the
// slice's largest element to [2^14, 2^15).  Returns the power that takes sums back.  inf and
// NaN pass in the high term.
template <int G>
__device__ __forceinline__ float w4_load_b_terms(uint32_t (&bx)[kW4WideSets][8][4], const float* row, int valid, int t) {
  float top = 0.f;
#pragma unroll
  for (int s = 0; s < 8; ++s)
    if (row != nullptr && s / (G / 32) < valid) {
      float v[8];
      w4_load8<FP32>(row + w4_step<G>(s, t), v);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (fabsf(v[j]) <= 3.402823466e38f) top = fmaxf(top, fabsf(v[j]));
    }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const int up = top > 0.f ? min(126, 14 + 127 - (int)(__float_as_uint(top) >> 23)) : 0;
  const float scale = __uint_as_float((uint32_t)(127 + up) << 23);
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (row != nullptr && s / (G / 32) < valid) w4_load8<FP32>(row + w4_step<G>(s, t), v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = v[i] * scale, y = v[i + 4] * scale;
      const __half2 hi = __floats2half2_rn(x, y);
      const float2 f = __half22float2(hi);
      const __half2 lo = __floats2half2_rn(fabsf(f.x) <= 65504.f ? x - f.x : 0.f, fabsf(f.y) <= 65504.f ? y - f.y : 0.f);
      bx[0][s][i] = *reinterpret_cast<const uint32_t*>(&hi);
      bx[1][s][i] = *reinterpret_cast<const uint32_t*>(&lo);
    }
  }
  return __uint_as_float((uint32_t)(127 - up) << 23);
}

// The consuming warps; as w4_consume, with a unit a team between two sums and, of each unit, the
// lanes' four sums a set ([set][lane] as float4; TERMS: the terms' sum, one set).
template <typename O, typename T, typename S, int G, bool ZP, bool RING, bool DUAL, typename Job>
__device__ __forceinline__ void w4_consume_wide(const W4Stream& p, uint8_t* smem, const Job& job) {
  constexpr bool TERMS = sizeof(typename T::Raw) == 4;
  constexpr int NG = kW4Chunk / G;
  constexpr int ROWS = DUAL ? 8 : kW4Rows;
  constexpr bool RAGGED = !DUAL;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int kw = warp % p.kw, team = warp / p.kw;
  const int UB = p.teams;
  const W4Smem L = w4_smem<G, ZP, RING>(p);
  const uint32_t bars = ptx::smem_u32(smem + L.bars());
  float* const sums_at = reinterpret_cast<float*>(smem + L.part()) + warp * 256 + lane * 4;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L.abort_flag());
  const int ngr = p.K / G;
  const uint32_t stage_bytes = (uint32_t)p.kw * kW4StageBytes;
  const uint32_t lane_at = ptx::smem_u32(smem) + kw * (ROWS * 128) + w4_lane_offset<G>(g, t);
  const uint32_t pair = DUAL ? stage_bytes / 2 : 1024u;
  const int row = w4_row<G>(g);
  const uint32_t gpitch = (uint32_t)(p.kw * NG), zstage = gpitch * kW4Rows;
  const uint32_t lane_zp = ptx::smem_u32(smem + L.zero_points()) + row * gpitch + kw * NG;
  const uint32_t lane_sp = ptx::smem_u32(smem + L.scales()) + 2 * (row * gpitch + kw * NG);
  uint32_t bx[kW4WideSets][8][4];
  float back[2] = {1.f, 1.f};  // TERMS: what takes the sums of columns 2t and 2t + 1 back
  int buf = 0, seq0 = 0;
  uint32_t taken = 1;
  bool ok = true;
  int lo, hi;
  job.range(0, lo, hi);
  for (int part = 0, item = lo; part < 2;) {
    if (item >= hi) {
      if (++part == 2) break;
      if (!job.plan([&] { return w4_wait(bars + 8 * kW4BarPlan, 0, p, abort_flag); })) break;
      job.range(1, item, hi);
      continue;
    }
    const int slot = item / p.upe, first = item - slot * p.upe;
    const int units = min(p.upe - first, hi - item), n_rows = job.rows(slot);
    const int base = job.matrix(slot) * p.rows;
    for (int u0 = first; u0 < first + units; u0 += UB) {
      const int nb = min(UB, first + units - u0);
      if (ok) ok = w4_wait(bars + 8 * (kW4BarTaken + buf), taken, p, abort_flag);
      for (int pass = 0; pass < p.passes; ++pass, seq0 += nb) {
        if (team >= nb) continue;
        const int chunk = pass * p.kw + kw;
        const int left = p.K - chunk * kW4Chunk;
        const int valid = left <= 0 ? 0 : min(left, kW4Chunk) / G;
        W4Quarter<G, ZP> quarter0, quarter1;
        if (!RING && valid > 0) {
          const int r = (u0 + team) * ROWS + row;
          const size_t at0 = (size_t)(base + r) * ngr + (size_t)chunk * NG, at1 = DUAL ? at0 : at0 + (size_t)8 * ngr;
          if (!RAGGED || r < p.rows) quarter0.load(p.scales0 + at0, p.zeros0 + at0, valid, t);
          if (!RAGGED || r + 8 < p.rows)
            quarter1.load((DUAL ? p.scales1 : p.scales0) + at1, (DUAL ? p.zeros1 : p.zeros0) + at1, valid, t);
        }
        if (valid > 0 && (p.passes > 1 || u0 == first)) {
          if constexpr (TERMS) {
            const float* r = job.row(slot, g);
            const float f = w4_load_b_terms<G>(bx, r ? r + (size_t)chunk * kW4Chunk : nullptr, valid, t);
            back[0] = __shfl_sync(0xffffffffu, f, 8 * t);
            back[1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
          } else {
#pragma unroll
            for (int n = 0; n < kW4WideSets; ++n) {
              const uint16_t* r = job.row(slot, n * 8 + g);
              w4_load_b16<G>(bx[n], r ? r + (size_t)chunk * kW4Chunk : nullptr, valid, t);
            }
          }
        }
        const int seq = seq0 + team, stage = seq & (p.stages - 1);
        if (ok) ok = w4_wait(bars + 8 * stage, (uint32_t)(seq / p.stages) & 1u, p, abort_flag);
        if (!ok) continue;
        const uint32_t at = lane_at + stage * stage_bytes;
        float tot[kW4WideSets][4];
        if (valid > 0) {
          W4RowScales<G, ZP> r0, r1;
          if (!RING) {
            quarter0.whole(r0, lane);
            quarter1.whole(r1, lane);
          } else {
            const uint32_t zp = lane_zp + stage * zstage, sp = lane_sp + stage * (2 * zstage);
            r0.load_ring(sp, zp);
            r1.load_ring(sp + 16 * gpitch, zp + 8 * gpitch);
          }
          if (TERMS || n_rows > 8)
            w4_task16<O, S, G, ZP, kW4WideSets>(at, r0, r1, bx, pair, tot);
          else
            w4_task16<O, S, G, ZP, 1>(at, r0, r1, bx, pair, tot);
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars + 8 * (kW4MaxRing + stage));
        if (valid == 0) continue;
        if constexpr (TERMS) {
          tot[0][0] = (tot[0][0] + tot[1][0]) * back[0], tot[0][2] = (tot[0][2] + tot[1][2]) * back[0];
          tot[0][1] = (tot[0][1] + tot[1][1]) * back[1], tot[0][3] = (tot[0][3] + tot[1][3]) * back[1];
        }
#pragma unroll
        for (int n = 0; n < (TERMS ? 1 : kW4WideSets); ++n) {
          if (n == 1 && n_rows <= 8) break;
          float4* out = reinterpret_cast<float4*>(sums_at + buf * (p.kw * p.teams * 256) + n * 128);
          float4 v = make_float4(tot[n][0], tot[n][1], tot[n][2], tot[n][3]);
          if (pass > 0) {
            const float4 o = *out;
            v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
          }
          *out = v;
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bars + 8 * (kW4BarSums + buf));
      buf = (buf + 1) % kW4Bufs;
      if (buf == 0) taken ^= 1;
    }
    item += units;
  }
}

// The adding warps take the batches in turn, a lane of theirs for a lane of the MMA.
template <typename T, int G, bool ZP, bool RING, bool DUAL, typename Job>
__device__ __forceinline__ void w4_add_wide(const W4Stream& p, uint8_t* smem, const Job& job, int tid) {
  constexpr bool TERMS = sizeof(typename T::Raw) == 4;
  const int lane = tid & 31, g = lane >> 2, t = lane & 3;
  int turn = tid >> 5;  // batches until the warp's next
  const W4Smem L = w4_smem<G, ZP, RING>(p);
  const uint32_t bars = ptx::smem_u32(smem + L.bars());
  const float* const sums_at = reinterpret_cast<const float*>(smem + L.part()) + lane * 4;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L.abort_flag());
  int buf = 0;
  uint32_t there = 0;
  for (int part = 0; part < 2; ++part) {
    int lo, hi;
    if (part == 1 && !job.plan([&] { return w4_wait(bars + 8 * kW4BarPlan, 0, p, abort_flag); })) return;
    job.range(part, lo, hi);
    for (int item = lo; item < hi;) {
      const int slot = item / p.upe, first = item - slot * p.upe;
      const int units = min(p.upe - first, hi - item), n_rows = job.rows(slot);
      const int sets = TERMS || n_rows <= 8 ? 1 : 2;
      for (int u0 = first; u0 < first + units; u0 += p.teams) {
        const int nb = min(p.teams, first + units - u0);
        const bool last = part == Job::kLastPart && item + units >= hi && u0 + p.teams >= first + units;
        const bool mine = turn == 0 || last;  // all three share the last batch
        if (mine && !w4_wait(bars + 8 * (kW4BarSums + buf), there, p, abort_flag)) return;
        for (int i = last ? tid >> 5 : 0; i < nb * sets && mine; i += last ? kW4SumThreads / 32 : 1) {
          const int q = sets == 2 ? i >> 1 : i, n = sets == 2 ? i & 1 : 0;
          const float4* at = reinterpret_cast<const float4*>(sums_at + ((buf * p.teams + q) * p.kw) * 256 + n * 128);
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int k = 0; k < p.kw; ++k) {
            const float4 v = at[k * 64];
            a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
          }
          const int mr = w4_row<G>(g), col = n * 8 + 2 * t;
          if (col < n_rows) job.store(slot, u0 + q, col, mr, a.x, a.z);
          if (col + 1 < n_rows) job.store(slot, u0 + q, col + 1, mr, a.y, a.w);
        }
        __syncwarp();
        if (lane == 0 && turn == 0 && !last) ptx::mbar_arrive(bars + 8 * (kW4BarTaken + buf));
        turn = turn == 0 ? kW4SumThreads / 32 - 1 : turn - 1;
        buf = (buf + 1) % kW4Bufs;
        if (buf == 0) there ^= 1;
      }
      item += units;
    }
  }
}

// As w4_roles.
template <typename T, int G, bool ZP, bool RING, bool DUAL, typename Job>
__device__ __forceinline__ bool w4_roles_wide(const W4Stream& p, uint8_t* smem, const Job& job) {
  const int warp = threadIdx.x >> 5, warps = p.kw * p.teams, group = (warps + 3) / 4 * 4;
  if (warp >= group) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == group) {
      w4_produce<G, ZP, RING, DUAL, 1>(p, smem, job);
    } else {
      const int tid = threadIdx.x - 32 * group - 32;
      job.before_add(tid);
      w4_add_wide<T, G, ZP, RING, DUAL>(p, smem, job, tid);
      job.finish(warps * 32 + tid);
    }
    return false;
  }
  asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
  return warp < warps;
}

}  // namespace
}  // namespace bitmoe
