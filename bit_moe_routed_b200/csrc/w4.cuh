// 4-bit weights with group scales (w4): the streaming product that the GEMM (w4_gemm.cu) and
// the whole-layer kernels (w4_layer.cu) share.
//
// A matrix is codes [N][K/2] (two 4-bit codes per byte, the low nibble the even element),
// scales [N][K/G] in the activations' type and, optionally, zero points [N][K/G]:
//   W[n][k] = (q[n][k] - z[n][k/G]) s[n][k/G],   z = 8 where there are no zero points.
// A row's dot product is taken group by group: sum_g s[n][g] * (sum_{k in g} (q - z) x[k]).
//
// The floor is reading the codes once (K/2 bytes a row): 88 clocks of a SM for 2 KB at the
// measured copy rate.  What bounds the loop is issuing instructions: made into bf16 or fp16
// operands of the tensor core, a word of 8 codes costs 9 to 11, and 2 KB took 370 in all.  So
// the product of a few rows of x runs in whole numbers: x goes, per row and slice of 256
// elements, into fixed point of 31 bits, taken apart into four signed bytes, and mma.sync
// m16n8k32 (8-bit integers, 32-bit sums; 2.1 clocks a SM, as the 16-bit m16n8k16 takes for half
// the reduction) multiplies code bytes with them, four columns a row of x.  A word of codes
// costs 3 instructions, 2 KB some 200, and a group's sum is exact.  Fixed point is off by at
// most 2^-30 of the slice's largest |x| per element: nothing for bf16 (fp16) elements down to
// 2^-22 (2^-19) of that, and below them less than a rounding of the largest to fp32.  The scale,
// and everything after it, is applied in fp32.  More rows of x: w4_wide.cuh.
//
// Measured (device, CUDA graph of calls on three sets of data): 65536 x 4096, G = 128, 4 rows:
// 36 us, 3.8 TB/s of 6.46, the 16-bit form 52 us; 4096 x 4096, 1 row: 6.0 us.
//
//   - a task is 16 rows x 256 reduction elements (2 KB of codes).  A warp keeps one slice of
//     256 elements for all its tasks, so the B operand, up to 4 rows of x in that slice, sits
//     in 16 registers per two rows for the whole slot;
//   - one warp of its own brings a unit (16 rows) for all the warps that share it with one or
//     two TMA boxes of up to 32 KB into a ring of 64 KB; it alone walks the list of units;
//   - within a group, lane t of a quad takes a quarter of the group's elements (its 4, 8 or
//     16 bytes of codes) whichever k those are: the k order inside a dot product is free as
//     long as A and B agree, and this one makes the fragment a straight read of the row;
//   - scales and zero points come with the codes by TMA where their rows are aligned for it;
//     elsewhere they are prefetched to L2 and loaded a task ahead;
//   - the warps that share a unit leave their sums in shared memory, where three warps of
//     their own add them in a fixed order and store the results while the others go on.
// A sum that comes out NaN (an infinity or NaN in x or in a scale) is taken again by one
// thread in floating point, so that infinities keep their sign.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "internal.cuh"
#include "ptx.cuh"
#include "waits.cuh"

namespace bitmoe {

// What the blocks of a stream know of its matrices.
struct W4Stream {
  CUtensorMap map0, map1;      // codes (w4_code_map)
  CUtensorMap smap0, smap1;    // scales and zero points (w4_group_map), with ring_scales
  CUtensorMap zmap0, zmap1;
  const uint8_t *codes0, *codes1;
  const uint16_t *scales0, *scales1;
  const uint8_t *zeros0, *zeros1;
  int K, rows, upe;        // rows of a matrix; units of a slot
  int passes, kw, teams;   // the block's split (w4_split)
  int stages;              // stages of the ring, a power of two
  bool ring_scales;        // scales and zero points come through the ring (the kernels' RING)
  long long wait_ns;
  int* status;
};

namespace {

constexpr int kW4Chunk = 256;      // reduction elements of a task
constexpr int kW4Rows = 16;        // rows of a task (the MMA's M)
constexpr int kW4Stages = 2;       // units under way per team of warps (4: the same times)
constexpr int kW4StageBytes = kW4Rows * kW4Chunk / 2;
constexpr int kW4MaxWarps = 16;
constexpr int kW4SetRows = 2;      // rows of x per B set: 4 bytes each fill the MMA's 8 columns
constexpr int kW4Sets = 2;         // B sets of a warp
constexpr int kW4Cols = kW4Sets * kW4SetRows;  // rows of x in a slot
constexpr int kW4Batch = 2;        // units a team works on between two sums (1: 18% slower at 16 tokens; 3: 16%)
constexpr int kW4Sums = 64 * kW4Sets;  // floats of a warp's sums of a unit

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
// Shared memory of a block of W consuming warps: the ring of codes (at a 1024-byte boundary),
// of scales and of zero points, the buffers of partial sums, the sums of bytes of x, the
// barriers, the abort flag and a counter; what the kernel adds comes after.
constexpr int kW4MaxRing = kW4Stages * kW4MaxWarps;  // most stages (one warp a unit)
constexpr int kW4Bufs = 4;                           // buffers of partial sums (2: 4% slower)
constexpr int kW4PartBytes = 1024;                   // of a warp in one of them
constexpr int kW4BarSums = 2 * kW4MaxRing, kW4BarTaken = kW4BarSums + kW4Bufs, kW4BarPlan = kW4BarTaken + kW4Bufs;
constexpr int kW4ByteSums = 512;                     // of a warp's sums of x's bytes (two sets)
struct W4Smem {
  int warps, groups;  // groups: per slice, 0 where scales do not come through the ring
  bool zeros;
  __host__ __device__ int scales() const { return warps * kW4Stages * kW4StageBytes; }
  __host__ __device__ int zero_points() const { return scales() + warps * kW4Stages * groups * kW4Rows * 2; }
  __host__ __device__ int part() const { return zero_points() + (zeros ? warps * kW4Stages * groups * kW4Rows : 0); }
  __host__ __device__ int byte_sums() const { return part() + warps * kW4Bufs * kW4PartBytes; }
  __host__ __device__ int bars() const { return byte_sums() + (zeros ? warps * kW4ByteSums : 0); }
  __host__ __device__ int abort_flag() const { return bars() + (kW4BarPlan + 1) * 8; }
  __host__ __device__ int counter() const { return abort_flag() + 4; }
  __host__ __device__ int few() const { return abort_flag() + 16; }  // scratch of the adding warps
  __host__ __device__ int bytes() const { return few() + 1024; }
};
constexpr int kW4SmemPad = 1024;  // for the alignment of the ring
// A block: the consuming warps, rounded up to a warpgroup of 4, and one more warpgroup: the
// copying warp and three that add up.  20 warps launch with 96 registers a thread; the last
// group keeps 64 and the consuming ones get 104: 4 * 104 + 64 = 5 * 96 on each of the SM's four
// partitions.
constexpr int kW4MaxThreads = (kW4MaxWarps + 4) * 32;
constexpr int kW4SumThreads = 96;
inline int w4_threads(int warps) { return ((warps + 3) / 4 * 4 + 4) * 32; }

struct BF16 {
  using Raw = uint16_t;
  __device__ static float to_float(uint32_t bits) { return __uint_as_float(bits << 16); }
};
struct FP16 {
  using Raw = uint16_t;
  __device__ static float to_float(uint32_t bits) {
    return __half2float(__ushort_as_half((unsigned short)bits));
  }
};
struct FP32 {
  using Raw = float;
};
// 8 consecutive elements of a row as fp32
template <typename T>
__device__ __forceinline__ void w4_load8(const typename T::Raw* at, float (&v)[8]) {
  if constexpr (sizeof(typename T::Raw) == 4) {
    const float4 a = __ldcg(reinterpret_cast<const float4*>(at));
    const float4 b = __ldcg(reinterpret_cast<const float4*>(at) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(at);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = T::to_float(w[i] & 0xFFFFu);
      v[2 * i + 1] = T::to_float(w[i] >> 16);
    }
  }
}
template <typename T>
__device__ __forceinline__ float w4_load1(const typename T::Raw* at) {
  if constexpr (sizeof(typename T::Raw) == 4)
    return __ldcg(at);
  else
    return T::to_float(*at);
}

// (v & mask) ^ bits in one instruction
__device__ __forceinline__ uint32_t w4_pick(uint32_t v, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(v), "r"(mask), "r"(bits));
  return r;
}
// A word's 8 codes as bytes, the even elements in `even`, the odd ones in `odd`: without zero
// points signed, 16 (q - 8) (the nibble with its top bit flipped is q - 8 in two's complement at
// the top of the byte); with them unsigned, q.
template <bool ZP>
__device__ __forceinline__ void w4_decode(uint32_t v, uint32_t& even, uint32_t& odd) {
  if constexpr (ZP) {
    even = v & 0x0F0F0F0Fu;
    odd = (v >> 4) & 0x0F0F0F0Fu;
  } else {
    even = w4_pick(v * 16u, 0xF0F0F0F0u, 0x80808080u);
    odd = w4_pick(v, 0xF0F0F0F0u, 0x80808080u);
  }
}
// Sums start at the bits of 1.5 * 2^23, so that a sum below 2^22 either way, read as fp32, is
// itself plus that number: a subtraction on the multiply-add pipe in place of a conversion.
// (A group's is at most 128 elements * 128 * 128.)  With zero points they start at that less
// the zero point times the sum of the group's bytes of x, which leaves sum (q - z) x.
constexpr int kW4Magic = 0x4B400000;
__device__ __forceinline__ float w4_sum(int c) { return __int_as_float(c) - 12582912.0f; }
// D += A B on bytes, B signed, A signed or (ZP) not; without `volatile`: a function of its
// operands that the compiler may move between the decodes.
template <bool ZP>
__device__ __forceinline__ void w4_mma(int (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  if constexpr (ZP)
    asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0, %1, %2, %3},"
        " {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3},"
        " {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// The matrix row (0..7) that the MMA's row g holds.  TMA writes 16-byte piece c of row r at
// c ^ r of the row's 128 bytes; with this order the lanes that one shared-memory access
// serves together (2, 4 or 8 rows by 16, 8 or 4 bytes a lane) meet no bank twice.
template <int G>
__device__ __forceinline__ int w4_row(int g) {
  return G == 128 ? ((g & 1) << 2) | (g >> 1) : G == 64 ? ((g & 3) << 1) | (g >> 2) : g;
}
// A lane's byte offset of group 0 in a stage's first 8 rows; group b is at offset ^ b * G / 2.
template <int G>
__device__ __forceinline__ uint32_t w4_lane_offset(int g, int t) {
  const int r = w4_row<G>(g);
  const int c = G == 128 ? t : G == 64 ? t >> 1 : 0;
  return (uint32_t)(r * 128 + ((c ^ r) << 4) + (G == 64 ? 8 * (t & 1) : G == 32 ? 4 * t : 0));
}

__device__ __forceinline__ void w4_lds(uint32_t at, uint32_t (&w)[4]) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
}
__device__ __forceinline__ void w4_lds(uint32_t at, uint32_t (&w)[2]) {
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
}
__device__ __forceinline__ void w4_lds(uint32_t at, uint32_t (&w)[1]) {
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at));
}

// The scales and zero points of one row in one slice, as loaded.
template <int G, bool ZP>
struct W4RowScales {
  static constexpr int NG = kW4Chunk / G;  // groups in a slice: 2, 4, 8
  uint32_t s[NG / 2];
  uint32_t z[NG == 8 ? 2 : 1];
  // from a stage of the ring
  __device__ __forceinline__ void load_ring(uint32_t sp, uint32_t zp) {
    w4_lds(sp, s);
    if constexpr (ZP) {
      if constexpr (NG == 2)
        asm volatile("ld.shared.u16 %0, [%1];" : "=r"(z[0]) : "r"(zp));
      else
        w4_lds(zp, z);
    }
  }
  template <typename S>
  __device__ __forceinline__ float scale(int b) const {
    return S::to_float((b & 1) ? s[b / 2] >> 16 : s[b / 2] & 0xFFFFu);
  }
  __device__ __forceinline__ int zero(int b) const { return (int)((z[b / 4] >> (8 * (b % 4))) & 0x7Fu); }
};
// A lane's quarter of them (two groups, one, or of two groups one), loaded from memory at any
// alignment; the quad puts them together where they are used.
template <int G, bool ZP>
struct W4Quarter {
  static constexpr int NG = kW4Chunk / G;
  uint32_t s = 0, z = 0;
  __device__ __forceinline__ void load(const uint16_t* sp, const uint8_t* zp, int valid, int t) {
    const int i = NG == 8 ? 2 * t : NG == 4 ? t : t & 1;
    s = i < valid ? __ldg(sp + i) : 0u;
    if (NG == 8 && i + 1 < valid) s |= (uint32_t)__ldg(sp + i + 1) << 16;
    if constexpr (ZP) {
      z = i < valid ? __ldg(zp + i) : 0u;
      if (NG == 8 && i + 1 < valid) z |= (uint32_t)__ldg(zp + i + 1) << 8;
    }
  }
  __device__ __forceinline__ void whole(W4RowScales<G, ZP>& r, int lane) const {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < (NG == 2 ? 2 : 4); ++i) v[i] = __shfl_sync(0xffffffffu, s, (lane & 28) | i);
#pragma unroll
    for (int i = 0; i < NG / 2; ++i) r.s[i] = NG == 8 ? v[i] : ptx::prmt(v[2 * i], v[2 * i + 1], 0x5410);
    if constexpr (ZP) {
#pragma unroll
      for (int i = 0; i < (NG == 2 ? 2 : 4); ++i) v[i] = __shfl_sync(0xffffffffu, z, (lane & 28) | i);
      if constexpr (NG == 8) {
        r.z[0] = ptx::prmt(v[0], v[1], 0x5410);
        r.z[1] = ptx::prmt(v[2], v[3], 0x5410);
      } else if constexpr (NG == 4) {
        r.z[0] = ptx::prmt(ptx::prmt(v[0], v[1], 0x0040), ptx::prmt(v[2], v[3], 0x0040), 0x5410);
      } else {
        r.z[0] = ptx::prmt(v[0], v[1], 0x0040);
      }
    }
  }
};

// One task: 16 rows times the B sets, group by group; `at` is the lane's group 0 in the first
// 8 rows, the other 8 are `pair` bytes on.  tot[n]: the lane's two bytes of one row of x in
// set n (columns 2t and 2t + 1, weights 1 and 256), for matrix rows g and g + 8.
// Groups past the row's end have codes and x of zero, and scales of zero.
// xsum: with zero points, in shared memory, the lane's two columns' sums of bytes of every
// group: [set][group][8 columns].
template <typename S, int G, bool ZP, int SETS>
__device__ __forceinline__ void w4_task(uint32_t at, const W4RowScales<G, ZP>& r0,
                                        const W4RowScales<G, ZP>& r1,
                                        const uint32_t (&bx)[kW4Sets][8][2], uint32_t pair, uint32_t xsum,
                                        float (&tot)[kW4Sets][2]) {
  constexpr int SG = G / 32;  // 32-bit words of a lane per group and row
  constexpr int NG = kW4Chunk / G;
  // all codes first; then two groups at a time, step by step in turn, so that two chains of
  // MMAs and decodes are under way
  uint32_t w0[NG][SG], w1[NG][SG];
#pragma unroll
  for (int b = 0; b < NG; ++b) {
    w4_lds(at ^ (uint32_t)(b * (G / 2)), w0[b]);
    w4_lds((at ^ (uint32_t)(b * (G / 2))) + pair, w1[b]);
  }
#pragma unroll
  for (int b0 = 0; b0 < NG; b0 += 2) {
    int acc[2][SETS][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int n = 0; n < SETS; ++n) {
        if constexpr (ZP) {
          uint32_t sum[2];
          w4_lds(xsum + (n * NG + b0 + j) * 32, sum);
          const int z0 = r0.zero(b0 + j), z1 = r1.zero(b0 + j);
          acc[j][n][0] = kW4Magic - z0 * (int)sum[0];
          acc[j][n][1] = kW4Magic - z0 * (int)sum[1];
          acc[j][n][2] = kW4Magic - z1 * (int)sum[0];
          acc[j][n][3] = kW4Magic - z1 * (int)sum[1];
        } else {
          acc[j][n][0] = acc[j][n][1] = acc[j][n][2] = acc[j][n][3] = kW4Magic;
        }
      }
#pragma unroll
    for (int i = 0; i < SG; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t a[4];
        w4_decode<ZP>(w0[b0 + j][i], a[0], a[2]);
        w4_decode<ZP>(w1[b0 + j][i], a[1], a[3]);
#pragma unroll
        for (int n = 0; n < SETS; ++n) w4_mma<ZP>(acc[j][n], a, bx[n][SG * (b0 + j) + i]);
      }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int b = b0 + j;
      const float s0 = r0.template scale<S>(b), s1 = r1.template scale<S>(b);
#pragma unroll
      for (int n = 0; n < SETS; ++n) {
        const float f0 = fmaf(w4_sum(acc[j][n][1]), 256.f, w4_sum(acc[j][n][0]));
        const float f1 = fmaf(w4_sum(acc[j][n][3]), 256.f, w4_sum(acc[j][n][2]));
        tot[n][0] = b == 0 ? s0 * f0 : fmaf(s0, f0, tot[n][0]);
        tot[n][1] = b == 0 ? s1 * f1 : fmaf(s1, f1, tot[n][1]);
      }
    }
  }
}

// Where step s (32 elements) of lane t starts in a slice.
template <int G>
__device__ __forceinline__ int w4_step(int s, int t) {
  return G * (s / (G / 32)) + (G / 4) * t + 8 * (s % (G / 32));
}
// B set: byte g % 4 of the fixed-point elements of the slice of one row (NULL: zeros).  A power
// of two brings the slice's largest element to [2^29, 2^30); the digits are balanced, so all
// four are signed bytes.  The four lanes that hold the bytes of one row convert a quarter of
// the elements each and exchange bytes.  Returns the power that takes sums back, or NaN where
// the slice holds an infinity or NaN.
template <typename T, int G>
__device__ __forceinline__ float w4_load_b(uint32_t (&bx)[8][2], const typename T::Raw* row, int valid, int g, int t) {
  constexpr int SG = G / 32;
  const int p = g & 3;  // the lane's quarter, steps 2p and 2p + 1, and its byte
  float v[2][8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = 2 * p + i;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (row != nullptr && s / SG < valid) w4_load8<T>(row + w4_step<G>(s, t), v[i]);
  }
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float f = fabsf(v[i][j]);
      top = f <= 3.402823466e38f ? fmaxf(top, f) : __uint_as_float(0x7F800000u);
    }
#pragma unroll
  for (int off = 1; off < 16; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  const bool odd = !(top <= 3.402823466e38f);
  const int up = top > 0.f && !odd ? min(126, 29 + 127 - (int)(__float_as_uint(top) >> 23)) : 0;
  const float scale = __uint_as_float((uint32_t)(127 + up) << 23);
  uint32_t d[2][8];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      d[i][j] = (uint32_t)((odd ? 0 : __float2int_rn(v[i][j] * scale)) + 0x00808080);
  // r[m]: the lane's byte of quarter p ^ m, from the lane that converted it
  const uint32_t flip = p < 3 ? 0x80808080u : 0u;
  uint32_t r[4][2][2];
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const uint32_t sel = (uint32_t)((p ^ m) * 0x11 + 0x40);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // the even elements, the odd ones
        const uint32_t w = ptx::prmt(ptx::prmt(d[i][h], d[i][2 + h], sel), ptx::prmt(d[i][4 + h], d[i][6 + h], sel), 0x5410);
        r[m][i][h] = (m == 0 ? w : __shfl_xor_sync(0xffffffffu, w, 4 * m)) ^ flip;
      }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // quarter Q is r[p ^ Q]
      const bool p0 = p & 1, p1 = p & 2;
      const uint32_t a0 = p0 ? r[1][i][h] : r[0][i][h], a1 = p0 ? r[0][i][h] : r[1][i][h];
      const uint32_t a2 = p0 ? r[3][i][h] : r[2][i][h], a3 = p0 ? r[2][i][h] : r[3][i][h];
      bx[i][h] = p1 ? a2 : a0;
      bx[2 + i][h] = p1 ? a3 : a1;
      bx[4 + i][h] = p1 ? a0 : a2;
      bx[6 + i][h] = p1 ? a1 : a3;
    }
  return odd ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)(127 - up) << 23);
}

// The sums of a B set's bytes by group and column, to shared memory [group][8 columns].
template <int G>
__device__ __forceinline__ void w4_byte_sums(const uint32_t (&bx)[8][2], int* to, int g, int t) {
  constexpr int SG = G / 32, NG = kW4Chunk / G;
#pragma unroll
  for (int b = 0; b < NG; ++b) {
    int sum = 0;
#pragma unroll
    for (int i = 0; i < SG; ++i) {
      sum = __dp4a((int)bx[SG * b + i][0], 0x01010101, sum);
      sum = __dp4a((int)bx[SG * b + i][1], 0x01010101, sum);
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if (t == (b & 3)) to[b * 8 + g] = sum;
  }
}

// A row's product in floating point, by one thread: where a sum is not a number.
template <typename T, typename S, int G, bool ZP>
__device__ __noinline__ float w4_slow_dot(const typename T::Raw* x, const uint8_t* codes,
                                          const uint16_t* scales, const uint8_t* zeros, int K) {
  float sum = 0.f;
  for (int b = 0; b < K / G; ++b) {
    const float z = ZP ? (float)(zeros[b] & 0x7F) : 8.f, s = S::to_float(scales[b]);
    for (int k = b * G; k < (b + 1) * G; ++k) {
      const int q = (codes[k >> 1] >> (4 * (k & 1))) & 15;
      sum = fmaf(w4_load1<T>(x + k), ((float)q - z) * s, sum);
    }
  }
  return sum;
}

// The streaming product of one block over its items: item = slot * upe + unit, a slot
// being an expert (or the matrix) with up to kW4Cols rows of x, a unit 16 rows of the matrix, or
// 8 rows of the first matrix and the same 8 of the second (DUAL).  Job supplies the slots and
// takes the sums:
//   range(part, lo, hi)     the block's items, in two parts [lo, hi); kLastPart: the last that
//                           can hold any
//   matrix(slot)            the slot's matrix (its rows start at matrix * rows)
//   plan(wait)              called by every warp before part 1; wait() is true once the slots are
//                           known (false if a wait has run out)
//   same_rows()             every slot has the same rows of x
//   rows(slot)              rows of x in the slot
//   row(slot, col)          row `col` of x (0 .. kW4Cols - 1) in the slot, NULL past the last
//   store(slot, unit, col, r, a, b)   the sums of rows r and r + 8 of the unit (DUAL: row r of
//                           both matrices), by one thread

// Barrier of the consuming warps.
__device__ __forceinline__ void w4_sync(const W4Stream& p) {
  asm volatile("bar.sync 1, %0;" ::"r"(p.kw * p.teams * 32) : "memory");
}
template <int G, bool ZP, bool RING>
__host__ __device__ __forceinline__ W4Smem w4_smem(const W4Stream& p) {
  return W4Smem{p.kw * p.teams, RING ? kW4Chunk / G : 0, ZP};
}

// Barriers, flag and counter of the block; the caller synchronises the block before w4_roles.
__device__ __forceinline__ void w4_init(const W4Stream& p, uint8_t* smem, const W4Smem& L) {
  const uint32_t bars = ptx::smem_u32(smem + L.bars());
  for (int i = threadIdx.x; i < p.stages; i += blockDim.x) {
    ptx::mbar_init(bars + 8 * i, 1);                    // full: the copy
    ptx::mbar_init(bars + 8 * (kW4MaxRing + i), p.kw);  // empty: the warps of a unit
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kW4Bufs; ++i) {
      ptx::mbar_init(bars + 8 * (kW4BarSums + i), L.warps);                 // sums there
      ptx::mbar_init(bars + 8 * (kW4BarTaken + i), 1);         // sums taken
    }
    ptx::mbar_init(bars + 8 * kW4BarPlan, 1);  // the slots are known
    *reinterpret_cast<int*>(smem + L.abort_flag()) = 0;
    *reinterpret_cast<int*>(smem + L.counter()) = 0;
  }
  ptx::fence_mbar_init();
}
// A wait of a whole warp: true once the phase is complete, false if a wait has run out.  The
// hardware may park the warp for most of it (polling it takes the same times).
__device__ __forceinline__ bool w4_wait(uint32_t bar, uint32_t parity, const W4Stream& p, volatile int* abort_flag) {
  constexpr uint32_t kPark = 20000;  // ns
  if (__all_sync(0xffffffffu, ptx::mbar_try_wait_for(bar, parity, p.wait_ns < kPark ? (uint32_t)p.wait_ns : kPark)))
    return true;
  return wait_warp(bar, parity, p.wait_ns, abort_flag, p.status);
}

// The copying warp: every unit (and pass) of the block's items in the order in which the
// consuming warps take them.  A stage is [slice][row][128 bytes] (DUAL: the first matrix's
// slices, then the second's); its scales and zero points are [row][group] with the groups of
// the pass.  Where those are not aligned for TMA they go to L2 at the same time (a row's share
// of this pass, a sector a lane): the consuming warps' loads, one task ahead, then find them
// there; left to DRAM, whose latency under load is longer than a task, they would set the pace.
// One warp has to keep up with the memory here, a unit every 700 clocks at some 8 clocks an
// instruction, so a unit takes as few of them as it can.
// BATCH: units a team works on between two sums.
template <int G, bool ZP, bool RING, bool DUAL, int BATCH, typename Job>
__device__ __forceinline__ void w4_produce(const W4Stream& p, uint8_t* smem, const Job& job) {
  constexpr int ROWS = DUAL ? 8 : kW4Rows;
  const int lane = threadIdx.x & 31;
  const W4Smem L = w4_smem<G, ZP, RING>(p);
  const uint32_t ring = ptx::smem_u32(smem), bars = ptx::smem_u32(smem + L.bars());
  const uint32_t sring = ptx::smem_u32(smem + L.scales()), zring = ptx::smem_u32(smem + L.zero_points());
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L.abort_flag());
  const int ngr = p.K / G;
  const bool whole = p.K % kW4Chunk == 0;
  const uint32_t bytes = (uint32_t)p.kw * kW4StageBytes;
  const uint32_t zbytes = (uint32_t)(p.kw * (kW4Chunk / G) * kW4Rows), sbytes = 2 * zbytes;
  const uint32_t tx = bytes + (RING ? sbytes + (ZP ? zbytes : 0u) : 0u);
  if (lane == 0) {
    ptx::prefetch_tmap(&p.map0);
    if (DUAL) ptx::prefetch_tmap(&p.map1);
  }
  // lanes 2r and 2r + 1 bring row r's scales to L2, every second sector each
  const int r = DUAL ? (lane >> 1) & 7 : lane >> 1;
  const uint16_t* const scales = DUAL && lane >= 16 ? p.scales1 : p.scales0;
  const uint8_t* const zeros = DUAL && lane >= 16 ? p.zeros1 : p.zeros0;
  const int step = ROWS * ngr;  // groups from one unit to the next (K <= 2^20)
  int stage = 0, seq = 0;
  uint32_t parity = 1;  // a fresh barrier's "previous" phase counts as complete
  bool ok = true;
  for (int part = 0; part < 2; ++part) {
    int lo, hi;
    if (part == 1 && !job.plan([&] { return w4_wait(bars + 8 * kW4BarPlan, 0, p, abort_flag); })) break;
    job.range(part, lo, hi);
    for (int item = lo; item < hi && ok;) {
      const int slot = item / p.upe, first = item - slot * p.upe;
      const int units = min(p.upe - first, hi - item);
      const int batch = p.passes > 1 ? BATCH * p.teams : units;
      for (int u0 = 0; u0 < units && ok; u0 += batch) {
        const int nb = min(batch, units - u0);
        for (int pass = 0; pass < p.passes && ok; ++pass) {
          const int g0 = pass * p.kw * (kW4Chunk / G);  // the pass's groups of a row
          const int gn = min(ngr - g0, p.kw * (kW4Chunk / G));
          int y = job.matrix(slot) * p.rows + (first + u0) * ROWS;
          int rows_left = p.rows - (first + u0) * ROWS - r;
          const uint16_t* sp = scales + (size_t)(y + r) * ngr + g0;
          const uint8_t* zp = zeros + (size_t)(y + r) * ngr + g0;
          for (int q = 0; q < nb; ++q) {
            const uint32_t full = bars + 8 * stage, empty = full + 8 * kW4MaxRing;
            ok = w4_wait(empty, parity, p, abort_flag);
            if (!ok) break;
            const uint32_t dst = ring + stage * bytes;
            if (lane == 0) ptx::mbar_arrive_expect_tx(full, tx);
            if (whole) {
              if (lane == 0) {
                ptx::tma_load_3d(dst, &p.map0, 0, y, pass * p.kw, full);
                if (DUAL) ptx::tma_load_3d(dst + bytes / 2, &p.map1, 0, y, pass * p.kw, full);
              }
            } else {
              __syncwarp();  // the barrier expects the bytes before any lane's copy
              if (lane < p.kw) {
                const int x = (pass * p.kw + lane) * (kW4Chunk / 2);
                ptx::tma_load_2d(dst + lane * (ROWS * 128), &p.map0, x, y, full);
                if (DUAL) ptx::tma_load_2d(dst + bytes / 2 + lane * (ROWS * 128), &p.map1, x, y, full);
              }
            }
            if (RING) {
              if (lane == 0) {
                const uint32_t sd = sring + stage * sbytes, zd = zring + stage * zbytes;
                ptx::tma_load_2d(sd, &p.smap0, g0, y, full);
                if (DUAL) ptx::tma_load_2d(sd + sbytes / 2, &p.smap1, g0, y, full);
                if (ZP) {
                  ptx::tma_load_2d(zd, &p.zmap0, g0, y, full);
                  if (DUAL) ptx::tma_load_2d(zd + zbytes / 2, &p.zmap1, g0, y, full);
                }
              }
            } else if (rows_left > 0) {
              for (int i = 16 * (lane & 1); i < gn + 15; i += 32) ptx::prefetch_l2(sp + min(i, gn - 1));
              if (ZP)
                for (int i = 32 * (lane & 1); i < gn + 31; i += 64) ptx::prefetch_l2(zp + min(i, gn - 1));
            }
            y += ROWS;
            rows_left -= ROWS;
            sp += step;
            zp += step;
            ++seq;
            if (++stage == p.stages) {
              stage = 0;
              parity ^= 1;
            }
          }
        }
      }
      item += units;
    }
  }
  // every copy lands before the block can end
  if (lane == 0)
    for (int i = max(0, seq - p.stages); i < seq; ++i)
      drain_wait(bars + 8 * (i & (p.stages - 1)), (uint32_t)(i / p.stages) & 1u);
}

// The consuming warps.  T: type of x; S: of the scales.
template <typename T, typename S, int G, bool ZP, bool RING, bool DUAL, typename Job>
__device__ __forceinline__ void w4_consume(const W4Stream& p, uint8_t* smem, const Job& job) {
  constexpr int NG = kW4Chunk / G;
  constexpr int ROWS = DUAL ? 8 : kW4Rows;     // rows of a unit in a matrix
  constexpr bool RAGGED = !DUAL;               // the last unit may reach past the matrix
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int kw = warp % p.kw, team = warp / p.kw;
  const int UB = kW4Batch * p.teams;
  const W4Smem L = w4_smem<G, ZP, RING>(p);
  const uint32_t bars = ptx::smem_u32(smem + L.bars());
  float* const sums_at = reinterpret_cast<float*>(smem + L.part());
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L.abort_flag());
  const int ngr = p.K / G;
  const uint32_t stage_bytes = (uint32_t)p.kw * kW4StageBytes;
  const uint32_t lane_at = ptx::smem_u32(smem) + kw * (ROWS * 128) + w4_lane_offset<G>(g, t);
  const uint32_t pair = DUAL ? stage_bytes / 2 : 1024u;
  const int row = w4_row<G>(g);  // the lane's first row of a unit
  // its groups in a stage of the ring of scales; the second row is 8 rows or half a stage on
  const uint32_t gpitch = (uint32_t)(p.kw * NG), zstage = gpitch * kW4Rows;
  const uint32_t lane_zp = ptx::smem_u32(smem + L.zero_points()) + row * gpitch + kw * NG;
  const uint32_t lane_sp = ptx::smem_u32(smem + L.scales()) + 2 * (row * gpitch + kw * NG);
  const size_t step = (size_t)p.teams * ROWS * ngr;  // groups from one unit of the team to the next
  int* const byte_sums = reinterpret_cast<int*>(smem + L.byte_sums() + (ZP ? warp * kW4ByteSums : 0));
  const uint32_t xsum = ptx::smem_u32(byte_sums) + 8 * t;
  uint32_t bx[kW4Sets][8][2];
  float back[kW4Sets];  // what takes the lane's sums back from fixed point
  int buf = 0, seq0 = 0;       // seq0: place of the batch's first unit in the ring's sequence
  uint32_t taken = 1;          // parity of the sums' barrier of buffer 0 (fresh: complete)
  bool ok = true;              // no wait has run out
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
        const int chunk = pass * p.kw + kw;
        const int left = p.K - chunk * kW4Chunk;
        const int valid = left <= 0 ? 0 : min(left, kW4Chunk) / G;  // groups of this slice
        // scales that do not come through the ring: the first unit's, then one task ahead
        W4Quarter<G, ZP> next0, next1;
        size_t at0 = 0;
        int rows_left = 0;
        auto load_scales = [&](int q) {
          if (q >= nb || valid == 0) return;
          const size_t at1 = DUAL ? at0 : at0 + (size_t)8 * ngr;
          if (!RAGGED || rows_left > 0) next0.load(p.scales0 + at0, p.zeros0 + at0, valid, t);
          if (!RAGGED || rows_left > 8)
            next1.load((DUAL ? p.scales1 : p.scales0) + at1, (DUAL ? p.zeros1 : p.zeros0) + at1, valid, t);
          at0 += step;
          if (RAGGED) rows_left -= p.teams * ROWS;
        };
        if (!RING) {
          const int r = (u0 + team) * ROWS + row;
          at0 = (size_t)(base + r) * ngr + (size_t)chunk * NG;
          rows_left = p.rows - r;
          load_scales(team);
        }
        if (valid > 0 && (p.passes > 1 || (u0 == first && (seq0 == 0 || !job.same_rows())))) {
#pragma unroll
          for (int n = 0; n < kW4Sets; ++n) {
            if (n * kW4SetRows >= n_rows) break;
            const typename T::Raw* r = job.row(slot, n * kW4SetRows + (g >> 2));
            const float f = w4_load_b<T, G>(bx[n], r ? r + (size_t)chunk * kW4Chunk : nullptr, valid, g, t);
            // columns 2t and 2t + 1: bytes 0 and 1 or (odd t) 2 and 3 of row t / 2
            back[n] = __shfl_sync(0xffffffffu, f, (t >> 1) * 16) * ((t & 1) ? 65536.f : 1.f) * (ZP ? 1.f : 0.0625f);
            if constexpr (ZP) w4_byte_sums<G>(bx[n], byte_sums + n * (8 * NG), g, t);
          }
          if constexpr (ZP) __syncwarp();
        }
        float* sums = sums_at + ((buf * UB + team) * p.kw + kw) * kW4Sums + lane * 2;
        for (int q = team; q < nb; q += p.teams, sums += p.teams * p.kw * kW4Sums) {
          const W4Quarter<G, ZP> now0 = next0, now1 = next1;
          if (!RING) load_scales(q + p.teams);
          const int seq = seq0 + q, stage = seq & (p.stages - 1);
          const uint32_t parity = (uint32_t)(seq / p.stages) & 1u;
          if (ok) ok = w4_wait(bars + 8 * stage, parity, p, abort_flag);
          if (!ok) continue;
          float tot[kW4Sets][2];
          const uint32_t at = lane_at + stage * stage_bytes;
          if (valid > 0) {  // as many sets as the slot has rows for
            W4RowScales<G, ZP> r0, r1;
            if (!RING) {
              now0.whole(r0, lane);
              now1.whole(r1, lane);
            } else {
              const uint32_t zp = lane_zp + stage * zstage, sp = lane_sp + stage * (2 * zstage);
              r0.load_ring(sp, zp);
              r1.load_ring(sp + 16 * gpitch, zp + 8 * gpitch);
            }
            if (n_rows <= kW4SetRows)
              w4_task<S, G, ZP, 1>(at, r0, r1, bx, pair, xsum, tot);
            else
              w4_task<S, G, ZP, kW4Sets>(at, r0, r1, bx, pair, xsum, tot);
          }
          __syncwarp();  // every lane has read the stage
          if (lane == 0) ptx::mbar_arrive(bars + 8 * (kW4MaxRing + stage));
          if (valid == 0) continue;
#pragma unroll
          for (int n = 0; n < kW4Sets; ++n) {
            if (n * kW4SetRows >= n_rows) break;
            float2* out = reinterpret_cast<float2*>(sums + n * 64);
            float2 v = make_float2(tot[n][0] * back[n], tot[n][1] * back[n]);
            if (pass > 0) {
              const float2 o = *out;
              v.x += o.x, v.y += o.y;
            }
            *out = v;
          }
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

// The adding warps take the batches of the consuming warps' sums in turn.  A row of x has two
// lanes of a quad, its low and its high bytes.  Lane (sub, r) takes every fourth slice of row
// pair r, for each row of x; the four of a row pair join what they have, and lane group `sub`
// stores row `sub` of x.  `tid`: 0 .. kW4SumThreads - 1.
template <typename T, typename S, int G, bool ZP, bool RING, bool DUAL, typename Job>
__device__ __forceinline__ void w4_add(const W4Stream& p, uint8_t* smem, const Job& job, int tid) {
  constexpr int ROWS = DUAL ? 8 : kW4Rows;
  int turn = tid >> 5;  // batches until the warp's next
  const int r = tid & 7, sub = (tid >> 3) & 3, mr = w4_row<G>(r);
  const int UB = kW4Batch * p.teams, ngr = p.K / G;
  const W4Smem L = w4_smem<G, ZP, RING>(p);
  const uint32_t bars = ptx::smem_u32(smem + L.bars());
  const float* const sums_at = reinterpret_cast<const float*>(smem + L.part());
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
      for (int u0 = first; u0 < first + units; u0 += UB) {
        const int nb = min(UB, first + units - u0);
        const bool last = part == Job::kLastPart && item + units >= hi && u0 + UB >= first + units;
        const bool mine = turn == 0 || last;  // all three share the last batch
        if (mine && !w4_wait(bars + 8 * (kW4BarSums + buf), there, p, abort_flag)) return;
        for (int q = last ? tid >> 5 : 0; q < nb && mine; q += last ? kW4SumThreads / 32 : 1) {
          const float4* at = reinterpret_cast<const float4*>(sums_at + (buf * UB + q) * p.kw * kW4Sums + r * 8);
          float a = 0.f, b = 0.f;  // of column `sub`
#pragma unroll
          for (int c = 0; c < kW4Cols; ++c) {
            if (c >= n_rows) break;
            float x = 0.f, y = 0.f;
#pragma unroll 4
            for (int k = sub; k < p.kw; k += 4) {
              const float4 v = at[k * (kW4Sums / 4) + (c >> 1) * 16 + (c & 1)];
              x += v.x + v.z;
              y += v.y + v.w;
            }
            x += __shfl_xor_sync(0xffffffffu, x, 8);
            y += __shfl_xor_sync(0xffffffffu, y, 8);
            x += __shfl_xor_sync(0xffffffffu, x, 16);
            y += __shfl_xor_sync(0xffffffffu, y, 16);
            if (c == sub) a = x, b = y;
          }
          if (sub >= n_rows) continue;
          const int unit = u0 + q;
          if (a != a || b != b) {
            const typename T::Raw* x = job.row(slot, sub);
            const size_t r0 = (size_t)job.matrix(slot) * p.rows + unit * ROWS + mr, r1 = DUAL ? r0 : r0 + 8;
            if (a != a && unit * ROWS + mr < p.rows)
              a = w4_slow_dot<T, S, G, ZP>(x, p.codes0 + r0 * (p.K / 2), p.scales0 + r0 * ngr, p.zeros0 + r0 * ngr, p.K);
            if (b != b && unit * ROWS + mr + (DUAL ? 0 : 8) < p.rows)
              b = w4_slow_dot<T, S, G, ZP>(x, (DUAL ? p.codes1 : p.codes0) + r1 * (p.K / 2),
                                           (DUAL ? p.scales1 : p.scales0) + r1 * ngr,
                                           (DUAL ? p.zeros1 : p.zeros0) + r1 * ngr, p.K);
          }
          job.store(slot, unit, sub, mr, a, b);
        }
        __syncwarp();
        if ((tid & 31) == 0 && turn == 0 && !last) ptx::mbar_arrive(bars + 8 * (kW4BarTaken + buf));
        turn = turn == 0 ? kW4SumThreads / 32 - 1 : turn - 1;
        buf = (buf + 1) % kW4Bufs;
        if (buf == 0) there ^= 1;
      }
      item += units;
    }
  }
}

// Splits the block into its roles and runs the copying and the adding warps; true in the
// consuming warps.  Job adds: before_add(thread) and finish(thread), which the adding warps call
// before their first and after their last batch.
template <typename T, typename S, int G, bool ZP, bool RING, bool DUAL, typename Job>
__device__ __forceinline__ bool w4_roles(const W4Stream& p, uint8_t* smem, const Job& job) {
  const int warp = threadIdx.x >> 5, warps = p.kw * p.teams, group = (warps + 3) / 4 * 4;
  if (warp >= group) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == group) {
      w4_produce<G, ZP, RING, DUAL, kW4Batch>(p, smem, job);
    } else {
      const int tid = threadIdx.x - 32 * group - 32;
      job.before_add(tid);
      w4_add<T, S, G, ZP, RING, DUAL>(p, smem, job, tid);
      job.finish(warps * 32 + tid);
    }
    return false;
  }
  asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
  return warp < warps;
}

// Allows a kernel a SM's whole shared memory, once a device (bit `device` of `allowed`).
constexpr int kW4MaxSmem = 227 * 1024;
template <typename Kernel>
cudaError_t w4_allow_smem(Kernel kern, std::atomic<unsigned long long>& allowed) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (allowed.load(std::memory_order_relaxed) >> dev & 1)) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kW4MaxSmem);
  if (e == cudaSuccess) allowed.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

// Host side: the map of a matrix's codes, [matrices * rows][K/2] bytes, with the 128-byte
// swizzle.  Rows of whole slices: (128 bytes, row, slice), kw slices a box; otherwise one slice
// a box.  Past the edges it reads zeros.
inline bool w4_code_map(CUtensorMap* m, const uint8_t* codes, long long rows, int K, int kw, int box_rows) {
  EncodeTiledFn fn = tensor_map_encode_fn();
  if (fn == nullptr) return false;
  const bool whole = K % kW4Chunk == 0;
  const cuuint64_t dims[3] = {whole ? 128u : (cuuint64_t)K / 2, (cuuint64_t)rows, (cuuint64_t)(K / kW4Chunk)};
  const cuuint64_t strides[2] = {(cuuint64_t)K / 2, 128u};
  const cuuint32_t box[3] = {128u, (cuuint32_t)box_rows, (cuuint32_t)kw};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, whole ? 3 : 2, const_cast<uint8_t*>(codes), dims, strides,
            box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The map of one value a group, [rows][groups] (bytes: 2 for scales, 1 for zero points): boxes
// of a pass's groups x box_rows rows.
inline bool w4_group_map(CUtensorMap* m, const void* base, int bytes, long long rows, int ngr, int box_groups,
                         int box_rows) {
  EncodeTiledFn fn = tensor_map_encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)ngr, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ngr * bytes};
  const cuuint32_t box[2] = {(cuuint32_t)box_groups, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1u, 1u};
  return fn(m, bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Fills in what a stream knows of its matrices: one, or two of the same shape.
struct W4Mat {
  const uint8_t* codes;
  const void* scales;
  const uint8_t* zeros;
};
inline bool w4_set_stream(W4Stream& st, const W4Mat& a, const W4Mat* b, long long matrices, int rows,
                          int K, int group) {
  const W4Split s = w4_split(K);
  const int box_rows = b ? 8 : kW4Rows, ngr = K / group, box = s.kw * (kW4Chunk / group);
  st.K = K;
  st.rows = rows;
  st.upe = (rows + box_rows - 1) / box_rows;
  st.passes = s.passes;
  st.kw = s.kw;
  st.teams = s.teams;
  st.stages = kW4Stages;
  while (2 * st.stages <= kW4Stages * s.teams) st.stages *= 2;
  const W4Mat* ms[2] = {&a, b};
  CUtensorMap* maps[2][3] = {{&st.map0, &st.smap0, &st.zmap0}, {&st.map1, &st.smap1, &st.zmap1}};
  // rows and boxes of scales and zero points whole 16-byte pieces
  const int unit = a.zeros ? 16 : 8;
  st.ring_scales = ngr % unit == 0 && box % unit == 0;
  for (const W4Mat* m : ms) {
    if (m == nullptr) continue;
    st.ring_scales = st.ring_scales && reinterpret_cast<uintptr_t>(m->scales) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(m->zeros) % 16 == 0;
  }
  for (int i = 0; i < 2 && ms[i]; ++i) {
    const W4Mat& m = *ms[i];
    if (!w4_code_map(maps[i][0], m.codes, matrices * rows, K, s.kw, box_rows)) return false;
    if (!st.ring_scales) continue;
    if (!w4_group_map(maps[i][1], m.scales, 2, matrices * rows, ngr, box, box_rows)) return false;
    if (m.zeros && !w4_group_map(maps[i][2], m.zeros, 1, matrices * rows, ngr, box, box_rows)) return false;
  }
  st.codes0 = a.codes;
  st.scales0 = static_cast<const uint16_t*>(a.scales);
  st.zeros0 = a.zeros;
  if (b) {
    st.codes1 = b->codes;
    st.scales1 = static_cast<const uint16_t*>(b->scales);
    st.zeros1 = b->zeros;
  }
  return true;
}

}  // namespace
}  // namespace bitmoe
