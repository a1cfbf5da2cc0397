// 4-bit weights with group scales (w4): the streaming product that the GEMM (w4_gemm.cu) and
// the whole-layer kernels (w4_layer.cu) share.
//
// A matrix is codes [N][K/2] (two 4-bit codes per byte, the low nibble the even element),
// scales [N][K/G] in the activations' type and, optionally, zero points [N][K/G]:
//   W[n][k] = (q[n][k] - z[n][k/G]) s[n][k/G],   z = 8 where there are no zero points.
// A row's dot product is taken group by group: sum_g s[n][g] * (sum_{k in g} (q - z) x[k]).
// q - z is an integer of at most 8 bits, exact in bf16 and in fp16, so the inner sums run on
// the tensor core (mma.sync m16n8k16, 16-bit operands, fp32 sums) with exact products and
// the scale is applied to the group's sum in fp32: nothing is rounded to 16 bits on the way.
//
// What bounds it is reading the codes once (K/2 bytes a row); the decode of a 32-bit word to
// four operand registers (11 instructions) takes about two thirds of the issue slots that
// the memory rate leaves, so the loop around it is kept bare:
//   - a task is 16 rows x 256 reduction elements (2 KB of codes).  A warp keeps one slice of
//     256 elements for all its tasks, so the B operand, up to 8 rows of x in that slice, sits
//     in 32 registers for the whole slot and no activation passes through shared memory;
//   - codes come by 16-byte cp.async into a ring of the warp's own, four tasks deep (96 KB a
//     SM in flight), with no barrier between warps;
//   - within a group, lane t of a quad takes a quarter of the group's elements (its 4, 8 or
//     16 bytes of codes) whichever k those are: the k order inside a dot product is free as
//     long as A and B agree, and this one makes the fragment a straight read of the row;
//   - the warps that share a unit (16 rows) leave their sums in shared memory, and every four
//     units or so the block adds them in a fixed order.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.cuh"
#include "ptx.cuh"

namespace bitmoe {
namespace {

constexpr int kW4Chunk = 256;      // reduction elements of a task
constexpr int kW4Rows = 16;        // rows of a task (the MMA's M)
constexpr int kW4Stages = 4;       // ring of a warp
constexpr int kW4StageBytes = kW4Rows * kW4Chunk / 2;
constexpr int kW4MaxWarps = 16;
constexpr int kW4Batch = 4;        // tasks of a warp between two block-wide sums (one B set)
constexpr int kW4Cols = 8;         // rows of x per B set (the MMA's N)

struct W4Mat {
  const uint8_t* codes;
  const void* scales;
  const uint8_t* zeros;  // NULL: 8
};

// How a block's warps split the reduction: nchunk slices, `passes` rounds of kw warps; `teams`
// groups of kw warps take units in turn.
struct W4Split {
  int nchunk, passes, kw, teams;
  int warps() const { return kw * teams; }
};
inline W4Split w4_split(int K) {
  W4Split s;
  s.nchunk = (K + kW4Chunk - 1) / kW4Chunk;
  s.passes = (s.nchunk + kW4MaxWarps - 1) / kW4MaxWarps;
  s.kw = (s.nchunk + s.passes - 1) / s.passes;
  s.teams = kW4MaxWarps / s.kw;
  return s;
}
// whether a row's scales (and zero points) of a slice can be loaded at once: rows of whole
// slices, bases on the load's alignment
inline bool w4_vec(const void* scales, const uint8_t* zeros, int K, int group) {
  const int ng = kW4Chunk / group;
  return K % kW4Chunk == 0 && reinterpret_cast<uintptr_t>(scales) % (2 * ng) == 0 &&
         reinterpret_cast<uintptr_t>(zeros) % ng == 0;
}
// ring and partial sums of a block (both kernels' first regions of shared memory)
inline size_t w4_stream_smem(int warps) {
  return (size_t)warps * (kW4Stages * kW4StageBytes + 2 * kW4Batch * 512);
}

struct BF16 {
  static constexpr uint32_t kMagic = 0x43004300u;  // 128 in both halves: one unit in the last place is 1
  __device__ static float to_float(uint32_t bits) { return __uint_as_float(bits << 16); }
  __device__ static uint32_t sub2(uint32_t a, uint32_t b) {
    __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a),
                               *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
  }
  __device__ static void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    ptx::mma_m16n8k16_bf16(c, a[0], a[1], a[2], a[3], b0, b1);
  }
};
struct FP16 {
  static constexpr uint32_t kMagic = 0x64006400u;  // 1024 in both halves
  __device__ static float to_float(uint32_t bits) {
    return __half2float(__ushort_as_half((unsigned short)bits));
  }
  __device__ static uint32_t sub2(uint32_t a, uint32_t b) {
    __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
  }
  __device__ static void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    ptx::mma_m16n8k16_f16(c, a[0], a[1], a[2], a[3], b0, b1);
  }
};

// Where 16-byte piece c (0..7) of row r lies in a stage of 128-byte rows, such that the
// fragment reads (16, 8 or 4 bytes a lane for G = 128, 64, 32) meet no bank twice.
template <int G>
__device__ __forceinline__ uint32_t w4_piece(int r, int c) {
  const int p = G == 128 ? c ^ ((r & 1) << 2) ^ ((r >> 1) & 3) : G == 64 ? c ^ ((r & 3) << 1) : c ^ (r & 7);
  return (uint32_t)(r * 128 + p * 16);
}

// The scales and zero points of one row in one slice, as loaded.
template <int G, bool ZP>
struct W4RowScales {
  static constexpr int NG = kW4Chunk / G;  // groups in a slice: 2, 4, 8
  uint32_t s[NG / 2];
  uint32_t z[NG == 8 ? 2 : 1];
  // at: (row * groups + first group); vec: the row pitch and the bases allow whole loads
  __device__ __forceinline__ void load(const W4Mat& m, size_t at, int valid, bool vec) {
    const uint16_t* sp = reinterpret_cast<const uint16_t*>(m.scales) + at;
    if (vec) {
      if constexpr (NG == 2) {
        s[0] = __ldg(reinterpret_cast<const uint32_t*>(sp));
      } else if constexpr (NG == 4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(sp));
        s[0] = v.x, s[1] = v.y;
      } else {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(sp));
        s[0] = v.x, s[1] = v.y, s[2] = v.z, s[3] = v.w;
      }
      if constexpr (ZP) {
        const uint8_t* zp = m.zeros + at;
        if constexpr (NG == 2) {
          z[0] = __ldg(reinterpret_cast<const uint16_t*>(zp));
        } else if constexpr (NG == 4) {
          z[0] = __ldg(reinterpret_cast<const uint32_t*>(zp));
        } else {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(zp));
          z[0] = v.x, z[1] = v.y;
        }
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < NG / 2; ++i) {
      const uint32_t lo = 2 * i < valid ? __ldg(sp + 2 * i) : 0u;
      const uint32_t hi = 2 * i + 1 < valid ? __ldg(sp + 2 * i + 1) : 0u;
      s[i] = lo | (hi << 16);
    }
    if constexpr (ZP) {
      z[0] = 0;
      if constexpr (NG == 8) z[1] = 0;
#pragma unroll
      for (int i = 0; i < NG; ++i)
        if (i < valid) z[i / 4] |= (uint32_t)__ldg(m.zeros + at + i) << (8 * (i % 4));
    }
  }
  __device__ __forceinline__ uint32_t scale_bits(int b) const {
    return (b & 1) ? s[b / 2] >> 16 : s[b / 2] & 0xFFFFu;
  }
  // the group's offset (magic + zero point) in both halves; zero points 0..127
  template <typename T>
  __device__ __forceinline__ uint32_t offset2(int b) const {
    if constexpr (!ZP) return T::kMagic + 0x00080008u;
    const uint32_t v = (z[b / 4] >> (8 * (b % 4))) & 0x7Fu;
    return T::kMagic | v | (v << 16);
  }
};

// One task: rows g and g+8 of the stage times the B sets, group by group.  HL: the two sets
// are the high and low terms of the same rows and share the sums.
template <typename T, typename S, int G, bool ZP, int NB, bool HL>
__device__ __forceinline__ void w4_task(const uint8_t* stage, const W4RowScales<G, ZP>& r0,
                                        const W4RowScales<G, ZP>& r1,
                                        const uint32_t (&bx)[NB][8][4], int valid, int lane,
                                        float (&tot)[HL ? 1 : NB][4]) {
  constexpr int SG = G / 32;  // 32-bit words of a lane per group and row
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int b = 0; b < kW4Chunk / G; ++b) {
    if (b >= valid) break;
    uint32_t w0[SG], w1[SG];
    if constexpr (G == 128) {
      const uint4 a = *reinterpret_cast<const uint4*>(stage + w4_piece<G>(g, 4 * b + t));
      const uint4 c = *reinterpret_cast<const uint4*>(stage + w4_piece<G>(g + 8, 4 * b + t));
      w0[0] = a.x, w0[1] = a.y, w0[2] = a.z, w0[3] = a.w;
      w1[0] = c.x, w1[1] = c.y, w1[2] = c.z, w1[3] = c.w;
    } else if constexpr (G == 64) {
      const uint2 a = *reinterpret_cast<const uint2*>(stage + w4_piece<G>(g, 2 * b + (t >> 1)) + 8 * (t & 1));
      const uint2 c = *reinterpret_cast<const uint2*>(stage + w4_piece<G>(g + 8, 2 * b + (t >> 1)) + 8 * (t & 1));
      w0[0] = a.x, w0[1] = a.y;
      w1[0] = c.x, w1[1] = c.y;
    } else {
      w0[0] = *reinterpret_cast<const uint32_t*>(stage + w4_piece<G>(g, b) + 4 * t);
      w1[0] = *reinterpret_cast<const uint32_t*>(stage + w4_piece<G>(g + 8, b) + 4 * t);
    }
    const uint32_t o0 = r0.template offset2<T>(b), o1 = r1.template offset2<T>(b);
    float acc[NB][4];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
#pragma unroll
    for (int i = 0; i < SG; ++i) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int sh = 8 * h;
        const uint32_t a[4] = {
            T::sub2(((w0[i] >> sh) & 0x000F000Fu) | T::kMagic, o0),
            T::sub2(((w1[i] >> sh) & 0x000F000Fu) | T::kMagic, o1),
            T::sub2(((w0[i] >> (sh + 4)) & 0x000F000Fu) | T::kMagic, o0),
            T::sub2(((w1[i] >> (sh + 4)) & 0x000F000Fu) | T::kMagic, o1)};
#pragma unroll
        for (int n = 0; n < NB; ++n)
          T::mma(acc[n], a, bx[n][SG * b + i][2 * h], bx[n][SG * b + i][2 * h + 1]);
      }
    }
    const float s0 = S::to_float(r0.scale_bits(b)), s1 = S::to_float(r1.scale_bits(b));
    if constexpr (HL) {
#pragma unroll
      for (int n = 1; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[0][i] += acc[n][i];
    }
#pragma unroll
    for (int n = 0; n < (HL ? 1 : NB); ++n) {
      tot[n][0] = fmaf(s0, acc[n][0], tot[n][0]);
      tot[n][1] = fmaf(s0, acc[n][1], tot[n][1]);
      tot[n][2] = fmaf(s1, acc[n][2], tot[n][2]);
      tot[n][3] = fmaf(s1, acc[n][3], tot[n][3]);
    }
  }
}

// B set of one row's slice: the row's elements in the order in which the codes of a word come
// apart, (0,4) (1,5) (2,6) (3,7).  row NULL: zeros.
template <int G>
__device__ __forceinline__ void w4_load_b(uint32_t (&bx)[8][4], const uint16_t* row, int chunk,
                                          int valid, int t) {
  constexpr int SG = G / 32;
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    const int b = s / SG, i = s % SG;
    if (row != nullptr && b < valid)
      v = *reinterpret_cast<const uint4*>(row + (size_t)chunk * kW4Chunk + G * b + (G / 4) * t + 8 * i);
    bx[s][0] = ptx::prmt(v.x, v.z, 0x5410);
    bx[s][1] = ptx::prmt(v.x, v.z, 0x7632);
    bx[s][2] = ptx::prmt(v.y, v.w, 0x5410);
    bx[s][3] = ptx::prmt(v.y, v.w, 0x7632);
  }
}

// The streaming product of one block over its items [lo, hi): item = slot * upe + unit, a slot
// being an expert (or the matrix) with up to 8 * NX rows of x, a unit 16 rows of the matrix, or
// 8 rows of m0 and the same 8 of m1 (DUAL).  Job supplies the slots and takes the sums:
//   matrix(slot)            the slot's matrix (its rows start at matrix * rows)
//   ready()                 called once, after the first copies are under way, before any B load
//   row(set, slot, col)     the B row of a column, NULL past the last
//   store(slot, unit, col, r, a, b)   the sums of rows r and r + 8 of the unit, by one thread
//   batch_done(slot, u0, n) called by all threads after the stores of units u0 .. u0 + n
struct W4Stream {
  W4Mat m0, m1;
  int K, rows, upe;      // rows of a matrix; units of a slot
  int passes, kw, teams; // the block's split (w4_split)
  bool vec;              // scales and zero points can be loaded whole slices at a time
};

template <typename T, typename S, int G, bool ZP, int NB, bool HL, bool DUAL, typename Job>
__device__ __forceinline__ void w4_stream(const W4Stream& p, uint8_t* smem, int lo, int hi, Job& job) {
  constexpr int NX = HL ? 1 : NB;              // sums per task
  constexpr int BATCH = kW4Batch / NX;         // tasks of a warp per block-wide sum
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int kw = warp % p.kw, team = warp / p.kw;
  const int UB = BATCH * p.teams;
  uint8_t* ring = smem + warp * (kW4Stages * kW4StageBytes);
  float* part = reinterpret_cast<float*>(smem + (size_t)(blockDim.x >> 5) * (kW4Stages * kW4StageBytes));
  const uint32_t ring_u32 = ptx::smem_u32(ring);
  const size_t pitch = (size_t)p.K / 2;
  const int ngr = p.K / G;

  // where the next copy comes from: the warp's tasks in the order in which it takes them
  int c_item = lo, c_nb = 0, c_pass = 0, c_q = 0, c_slot = 0, c_u0 = 0;
  bool c_done = false;
  auto c_batch = [&]() {  // the batch that starts at c_item
    if (c_item >= hi) {
      c_done = true;
      return;
    }
    c_slot = c_item / p.upe;
    c_u0 = c_item - c_slot * p.upe;
    c_nb = min(UB, min(p.upe - c_u0, hi - c_item));
    c_pass = 0;
    c_q = team;
  };
  auto c_settle = [&]() {  // step over batches and passes in which this team has no unit left
    while (!c_done && c_q >= c_nb) {
      if (team < c_nb && ++c_pass < p.passes) {
        c_q = team;
      } else {
        c_item += c_nb;
        c_batch();
      }
    }
  };
  auto issue = [&](int stage) {
    if (!c_done) {
      const int chunk = c_pass * p.kw + kw;
      const int left = p.K - chunk * kW4Chunk;
      if (left > 0) {
        const int piece = lane & 7, unit = c_u0 + c_q;
        const bool ok = piece * 32 < left;
        const size_t col = (size_t)chunk * (kW4Chunk / 2) + (ok ? piece * 16 : 0);
        const size_t first = (size_t)job.matrix(c_slot) * p.rows;
        const uint32_t dst = ring_u32 + stage * kW4StageBytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = (lane >> 3) + 4 * i;
          const uint8_t* src;
          if (DUAL)
            src = (i < 2 ? p.m0.codes : p.m1.codes) + (first + unit * 8 + (r & 7)) * pitch + col;
          else
            src = p.m0.codes + (first + min(unit * kW4Rows + r, p.rows - 1)) * pitch + col;
          ptx::cp_async_16_zfill(dst + w4_piece<G>(r, piece), src, ok ? 16u : 0u);
        }
      }
      c_q += p.teams;
      c_settle();
    }
    ptx::cp_async_commit();
  };
  c_batch();
  c_settle();
#pragma unroll
  for (int s = 0; s < kW4Stages - 1; ++s) issue(s);
  job.ready();

  uint32_t bx[NB][8][4];
  int b_slot = -1, stage = 0, buf = 0;
  for (int item = lo; item < hi;) {
    const int slot = item / p.upe, u0 = item - slot * p.upe;
    const int nb = min(UB, min(p.upe - u0, hi - item));
    const size_t first = (size_t)job.matrix(slot) * p.rows;
    for (int pass = 0; pass < p.passes; ++pass) {
      const int chunk = pass * p.kw + kw;
      const int left = p.K - chunk * kW4Chunk;
      const int valid = left <= 0 ? 0 : min(left, kW4Chunk) / G;  // groups of this slice
      if (valid > 0 && (p.passes > 1 || slot != b_slot)) {
#pragma unroll
        for (int n = 0; n < NB; ++n) w4_load_b<G>(bx[n], job.row(n, slot, g), chunk, valid, t);
        b_slot = slot;
      }
      for (int q = team; q < nb; q += p.teams) {
        const int unit = u0 + q;
        W4RowScales<G, ZP> r0, r1;
        if (valid > 0) {
          const size_t gr0 = (size_t)chunk * W4RowScales<G, ZP>::NG;
          if (DUAL) {
            const size_t at = (first + unit * 8 + g) * ngr + gr0;
            r0.load(p.m0, at, valid, p.vec);
            r1.load(p.m1, at, valid, p.vec);
          } else {
            r0.load(p.m0, (first + min(unit * kW4Rows + g, p.rows - 1)) * ngr + gr0, valid, p.vec);
            r1.load(p.m0, (first + min(unit * kW4Rows + g + 8, p.rows - 1)) * ngr + gr0, valid, p.vec);
          }
        }
        ptx::cp_async_wait_group<kW4Stages - 2>();
        __syncwarp();  // every lane's copies of this task have landed, and its reads of the last are done
        issue((stage + kW4Stages - 1) % kW4Stages);
        if (valid > 0) {
          float tot[NX][4];
#pragma unroll
          for (int n = 0; n < NX; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) tot[n][i] = 0.f;
          w4_task<T, S, G, ZP, NB, HL>(ring + stage * kW4StageBytes, r0, r1, bx, valid, lane, tot);
          // (c0, c2) and (c1, c3): rows g and g+8 of one column together
#pragma unroll
          for (int n = 0; n < NX; ++n) {
            float4* at = reinterpret_cast<float4*>(
                part + ((((size_t)buf * UB + q) * p.kw + kw) * NX + n) * 128 + lane * 4);
            float4 v = make_float4(tot[n][0], tot[n][2], tot[n][1], tot[n][3]);
            if (pass > 0) {
              const float4 o = *at;
              v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
            }
            *at = v;
          }
        }
        stage = (stage + 1) % kW4Stages;
      }
    }
    __syncthreads();
    // the warps' sums of every (unit, set, column, row pair), in slice order
    for (int i = threadIdx.x; i < nb * NX * 64; i += blockDim.x) {
      const int q = i / (NX * 64), n = (i / 64) % NX, l = (i % 64) / 2, j = i & 1;
      const float2* at = reinterpret_cast<const float2*>(
                             part + (((size_t)buf * UB + q) * p.kw * NX + n) * 128) + l * 2 + j;
      float a = 0.f, b = 0.f;
#pragma unroll 4
      for (int c = 0; c < p.kw; ++c) {
        const float2 v = at[(size_t)c * NX * 64];
        a += v.x;
        b += v.y;
      }
      job.store(slot, u0 + q, 8 * n + 2 * (l & 3) + j, l >> 2, a, b);
    }
    job.batch_done(slot, u0, nb);
    item += nb;
    buf ^= 1;
  }
  ptx::cp_async_wait_all();
}

}  // namespace
}  // namespace bitmoe
