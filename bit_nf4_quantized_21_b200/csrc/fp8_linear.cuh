// fp8_linear.cuh -- the frozen linear layer over a weight held in 8-bit
// floating point (E4M3) with one fp32 scale for each block of 128 x 128, the
// activations quantised on the way in with one scale for each 1 x 128.
//
//   quantiser: s = fp32(absmax / 448), r = fp32(1 / s), q = E4M3_rne(fp32(x r))
//   forward:   Y[m, n]  = sum over blocks kb of sx[m, kb] sw[n/128, kb] D_kb[m, n],
//              D_kb[m, n] = sum over k in block kb of qx[m, k] qw[n, k]
//   dX:        the same with the contraction over n: dX[m, k] = sum over
//              blocks nb of sg[m, nb] sw[nb, k/128] sum over n in nb of qg[m, n] qw[n, k]
//
// Products of E4M3 values are exact in the tensor core's fp32 accumulator;
// each block's sum is scaled and added in fp32; the output is rounded once.
//
// k_fp8_gemm (many tokens).  A pair of SMs (tcgen05.mma cta_group::2,
// kind::f8f6f4) owns a 256 x 256 output tile; each CTA brings its 128
// activation rows and its 128-row half of the weight tile by TMA, 32 KB per
// block of 128 in a ring of six.  A block's product cannot stay in the tensor
// core's accumulator (the scales differ from block to block): it goes into
// tensor memory, and eight warps take it out and add it to fp32 sums in
// registers, acc = fma(D, sx sw, acc), packed in pairs; a thread holds 128
// outputs of one row, inside one scale block of the weight.  Tensor memory
// holds two such products and no more, so a place has to be free again soon:
// four accumulators of 128 columns instead of two of 256 (a place waits for
// half as much work), an issuing thread for each (a thread that waits after
// issuing MMAs stalls until they drain), and the place is handed back as soon
// as its values are in registers, before they are used.  The scales come
// through shared memory, two blocks ahead (one block ahead, their way was
// what every block waited for: 2048 x 11008 x 4096 took 99 us).  The grid is
// one pair per two SMs and walks the tiles, so that a tile's output is written
// while the next one's products are already running.  The same weight bytes
// serve both directions: a tile of 128 rows x 128 bytes is a K-major operand
// forward and an MN-major one in dX.  Where there are few tiles they are 128
// columns wide, a whole block to an accumulator, three in flight.
//   Measured on the device (calls in a graph, each on inputs that are not in
// L2, the quantiser ahead of the product): 2048 x 11008 x 4096 forward 90 us
// (2.05 PFLOP/s; 85 without the quantiser, 97 with fp32 in and out), dX 99 us;
// one after the other from the public entry, where power and launches count,
// 108 (1.71 PFLOP/s) and 116.  1000 x 4100 x 4040 28.6 us (N = 4096, whose rows
// TMA can write: 25.7).  Fewer tokens leave most pairs idle while each walks
// its contraction alone: 64 x 4096 x 4096 16.6 us (its bytes: 2.7), 256 x
// 11008 x 4096 22.8 (8.0), dX of 1 to 64 tokens x 28672 x 512 73 (2.2) and
// x 28672 x 8192 77 to 113 (36).
//   With many tokens, what bounds it now is the epilogue warps' way for a half
// of a block: notice that it is there, take 64 columns out (one warp in a
// quarter of the tensor memory at a time), hand the place back, 32 packed
// multiply-adds; 0.24 us, where the MMAs need 0.14.
//
// k_fp8_gemv (few tokens, forward), HBM bound: the weight streams once from
// global memory straight into the registers of legacy warp-level MMAs
// (m16n8k32; 16 weight rows x 8 tokens): at these token counts the tensor
// work is 1/100 of what the stream takes, and a warp's fragment loads are
// whole 64-byte pieces of its rows.  The tokens' codes sit in shared memory.
// Behind the quantiser the kernel is a programmatic dependent launch: its
// first weights travel while the activations are quantised.
//   Measured the same way: 1 x 28672 x 8192 43 us (5.5 TB/s of weight, a
// copy's rate is 6.57), 8 x 28672 x 8192 45.5 us; 16 tokens 66, 23 tokens 116
// (fewer blocks on their way as fragments of more tokens fill the registers;
// from 24 on their codes pass shared memory at this width and the other kernel
// takes 62).  7 x 4096 x 4096 8.2 us (two launches and a CTA's one round over
// its rows).
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "ptx.cuh"

namespace qlora {

constexpr int kF8Block = 128;
constexpr float kF8Max = 448.0f;

// ------------------------------------------------------------- quantiser
// E4M3 codes of (lo, hi), round to nearest even, saturating; NaN stays NaN
__device__ __forceinline__ uint32_t f8_pack2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint2 f8_pack8(const float (&f)[8], float r) {
  return make_uint2(f8_pack2(f[0] * r, f[1] * r) | (f8_pack2(f[2] * r, f[3] * r) << 16),
                    f8_pack2(f[4] * r, f[5] * r) | (f8_pack2(f[6] * r, f[7] * r) << 16));
}
// Largest magnitude as the bits of a float: for magnitudes the order of the
// bits is the order of the values, and infinities and NaN come out on top.
__device__ __forceinline__ uint32_t f8_magnitude(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  return m;
}
// scale and reciprocal of a block; a scale below the smallest normal number
// stands for a block of zeros
__device__ __forceinline__ void f8_scale(float absmax, float& s, float& r) {
  s = __fdiv_rn(absmax, kF8Max);
  r = 0.0f;
  if (s < 1.17549435e-38f) s = 0.0f; else r = __frcp_rn(s);
}

struct Fp8QuantArgs {
  const void* x;
  int64_t ldx, rows, cols;
  uint8_t* codes;
  int64_t ldq;
  float* scale;
  int vec;              // 16-byte loads are aligned for every row
  int* status;
};

// elements [c, c + 8) of a row, zeros past its end
template <typename T>
__device__ __forceinline__ void f8_load8(const T* row, int64_t c, int64_t cols, int vec, float (&f)[8]) {
  if (vec && c + 8 <= cols) {
    if (sizeof(T) == 2) {
      const uint4 v = *reinterpret_cast<const uint4*>(row + c);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    } else {
      const float4 a = reinterpret_cast<const float4*>(row + c)[0], b = reinterpret_cast<const float4*>(row + c)[1];
      f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
      f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c + i < cols ? static_cast<float>(row[c + i]) : 0.0f;
  }
}

// Blocks of 1 x 128: sixteen lanes per block, eight elements each.  HBM
// bound (reads 2 or 4 bytes, writes 1 per element): 2048 x 11008 bf16 20 us
// (its bytes at the copy's rate: 10.3), 2048 x 4096 9.4 (3.8), fp32 9.7 (6.4).
// A CTA takes 16 rows of
// one block column, so that the scales, which go out block-major ([cols /
// 128][rows], the order in which the GEMM reads them), leave as one run.
constexpr int kF8QuantThreads = 256;
constexpr int kF8QuantRows = kF8QuantThreads / 16;
template <typename T>
__global__ void __launch_bounds__(kF8QuantThreads) k_fp8_quant_rows(const Fp8QuantArgs a) {
  __shared__ float scales[kF8QuantRows];
  griddep_launch_dependents();            // the product behind may bring its weights meanwhile
  const uint32_t blocks = static_cast<uint32_t>((a.cols + kF8Block - 1) / kF8Block);
  const uint32_t kb = blockIdx.x % blocks;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / blocks) * kF8QuantRows;
  const int r = threadIdx.x >> 4;
  const int64_t row = row0 + r, c = static_cast<int64_t>(kb) * kF8Block + (threadIdx.x & 15) * 8;
  const bool in = row < a.rows && c < a.cols;
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = 0.0f;
  if (in) f8_load8(static_cast<const T*>(a.x) + row * a.ldx, c, a.cols, a.vec, f);
  uint32_t m = f8_magnitude(f);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  float s, rc;
  f8_scale(__uint_as_float(m), s, rc);
  if (in) *reinterpret_cast<uint2*>(a.codes + row * a.ldq + c) = f8_pack8(f, rc);
  if ((threadIdx.x & 15) == 0) {
    scales[r] = s;
    if (m >= 0x7F800000u && a.status) atomicOr(a.status, QLORA_DEV_NONFINITE);
  }
  __syncthreads();
  if (threadIdx.x < kF8QuantRows && row0 + threadIdx.x < a.rows)
    a.scale[static_cast<int64_t>(kb) * a.rows + row0 + threadIdx.x] = scales[threadIdx.x];
}

// Blocks of 128 x 128: one CTA per block, 64 elements per thread in registers.
// 11008 x 4096 fp32 41 us (its bytes at the copy's rate: 34), bf16 72 us (21).
template <typename T>
__global__ void __launch_bounds__(256) k_fp8_quant_blocks(const Fp8QuantArgs a) {
  __shared__ uint32_t red[8];
  const int64_t nkb = (a.cols + kF8Block - 1) / kF8Block;
  const int64_t nb = blockIdx.x / nkb, kb = blockIdx.x % nkb;
  const int64_t c = kb * kF8Block + (threadIdx.x & 15) * 8;
  const int64_t r0 = nb * kF8Block + (threadIdx.x >> 4);
  float f[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = r0 + 16 * i;
    if (row < a.rows) {
      f8_load8(static_cast<const T*>(a.x) + row * a.ldx, c, a.cols, a.vec, f[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] = 0.0f;
    }
    m = max(m, f8_magnitude(f[i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, red[i]);
  float s, r;
  f8_scale(__uint_as_float(m), s, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = r0 + 16 * i;
    if (row < a.rows && c < a.cols) *reinterpret_cast<uint2*>(a.codes + row * a.ldq + c) = f8_pack8(f[i], r);
  }
  if (threadIdx.x == 0) {
    a.scale[nb * nkb + kb] = s;
    if (m >= 0x7F800000u && a.status) atomicOr(a.status, QLORA_DEV_NONFINITE);
  }
}

// --------------------------------------------------- few tokens: the stream
struct Fp8GemvArgs {
  const uint8_t* w;
  int64_t ldw, N, K;
  const float* sw;       // [ceil(N/128)][ceil(K/128)]
  const uint8_t* x;
  int64_t ldx;
  int M;
  const float* sx;       // [ceil(K/128)][M]
  void* y;
  int64_t ldy;
  int y_f32;
  int after_quant;       // launched as a dependent of the quantiser
};

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes of a row from byte k, zeros from byte `end` on (rows are 16-byte
// aligned and at least `end` rounded up to 16 long)
__device__ __forceinline__ uint4 f8_bytes16(const uint8_t* row, int64_t k, int64_t end) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (k < end) {
    v = *reinterpret_cast<const uint4*>(row + k);
    if (k + 16 > end) {
      const int n = static_cast<int>(end - k);     // 1 .. 15 bytes stay
      auto keep = [n](uint32_t w, int at) {
        const int b = n - at;
        return b >= 4 ? w : b <= 0 ? 0u : w & ((1u << (8 * b)) - 1u);
      };
      v.x = keep(v.x, 0); v.y = keep(v.y, 4); v.z = keep(v.z, 8); v.w = keep(v.w, 12);
    }
  }
  return v;
}

constexpr int kF8GemvWarps = 16;
constexpr int kF8GemvThreads = 32 * kF8GemvWarps;
constexpr int kF8GemvRows = 16;

// Shared memory of a launch: the tokens' codes (rows `xs` bytes apart: 64
// more than a multiple of 128, so that the eight rows that a load takes lie
// in different banks), their scales, the warps' sums of one tile.
struct Fp8GemvSmem {
  uint32_t xs, off_scale, off_part, bytes;
};
__host__ __device__ inline Fp8GemvSmem fp8_gemv_smem(int M, int64_t K, int nt) {
  Fp8GemvSmem s;
  const uint32_t blocks = static_cast<uint32_t>((K + kF8Block - 1) / kF8Block);
  s.xs = blocks * kF8Block + 64;
  s.off_scale = s.xs * static_cast<uint32_t>(M);
  s.off_part = s.off_scale + blocks * nt * 8 * 4;
  s.bytes = s.off_part + kF8GemvWarps * kF8GemvRows * (nt * 8 + 1) * 4;
  return s;
}

// A weight load: read once, kept out of L1
__device__ __forceinline__ uint4 f8_stream16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// One CTA per SM.  Its tiles of 16 weight rows are shared out by blocks of the
// contraction: warp w takes blocks w, w + 16, ...; every warp has the weights
// of a few blocks on their way (2 KB each), across the end of a tile too.
// The contraction's order inside a block is free as long as both operands
// follow it: lane quad c holds bytes 16c .. 16c + 15 and 64 + 16c .. of each
// of its rows, and MMA i takes 8 of them.
template <int NT>
__global__ void __launch_bounds__(kF8GemvThreads, 1) k_fp8_gemv(const Fp8GemvArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const Fp8GemvSmem lay = fp8_gemv_smem(a.M, a.K, NT);
  float* sxs = reinterpret_cast<float*>(smem_raw + lay.off_scale);      // [block][NT * 8]
  float* part = reinterpret_cast<float*>(smem_raw + lay.off_part);      // [warp][row][NT * 8 + 1]
  constexpr int kPitch = NT * 8 + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int blocks = static_cast<int>((a.K + kF8Block - 1) / kF8Block);
  const int tiles = static_cast<int>((a.N + kF8GemvRows - 1) / kF8GemvRows);
  const int grid = static_cast<int>(gridDim.x);
  const bool busy = warp < blocks;

  constexpr int kAhead = NT == 1 ? 4 : NT == 2 ? 3 : 2;      // blocks on their way (as many as registers hold)
  uint4 buf[kAhead][4];
  float bsw[kAhead];
  int pt = blockIdx.x, pk = warp;            // the next block to fetch
  auto fetch = [&](uint4 (&v)[4], float& s) {
    if (busy && pt < tiles) {
      const int64_t n0 = static_cast<int64_t>(pt) * kF8GemvRows;
      const uint8_t* w0 = a.w + min(n0 + g, a.N - 1) * a.ldw;
      const uint8_t* w1 = a.w + min(n0 + g + 8, a.N - 1) * a.ldw;
      const int64_t k = static_cast<int64_t>(pk) * kF8Block + 16 * c;
      if (static_cast<int64_t>(pk + 1) * kF8Block <= a.K) {
        v[0] = f8_stream16(w0 + k);
        v[1] = f8_stream16(w1 + k);
        v[2] = f8_stream16(w0 + k + 64);
        v[3] = f8_stream16(w1 + k + 64);
      } else {                               // bytes past the last column may hold anything
        v[0] = f8_bytes16(w0, k, a.K);
        v[1] = f8_bytes16(w1, k, a.K);
        v[2] = f8_bytes16(w0, k + 64, a.K);
        v[3] = f8_bytes16(w1, k + 64, a.K);
      }
      s = a.sw[n0 / kF8Block * blocks + pk];
      pk += kF8GemvWarps;
      if (pk >= blocks) { pk = warp; pt += grid; }
    }
  };
#pragma unroll
  for (int b = 0; b < kAhead; ++b) fetch(buf[b], bsw[b]);
  if (a.after_quant) griddep_wait();         // the activations come from the kernel ahead, the weights do not
  for (int i = threadIdx.x; i < a.M * blocks * 8; i += kF8GemvThreads) {
    const int tok = i / (blocks * 8);
    const int64_t k = static_cast<int64_t>(i % (blocks * 8)) * 16;
    *reinterpret_cast<uint4*>(smem_raw + tok * lay.xs + k) = f8_bytes16(a.x + tok * a.ldx, k, a.K);
  }
  for (int i = threadIdx.x; i < blocks * NT * 8; i += kF8GemvThreads) {
    const int tok = i % (NT * 8);
    sxs[i] = tok < a.M ? a.sx[static_cast<int64_t>(i / (NT * 8)) * a.M + tok] : 0.0f;
  }
  __syncthreads();

  float acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] = 0.0f;
  // the tile's sums over the warps, in warp order
  auto finish = [&](int tile) {
    float* mine = part + warp * kF8GemvRows * kPitch;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      mine[g * kPitch + t * 8 + 2 * c] = acc[t][0];
      mine[g * kPitch + t * 8 + 2 * c + 1] = acc[t][1];
      mine[(g + 8) * kPitch + t * 8 + 2 * c] = acc[t][2];
      mine[(g + 8) * kPitch + t * 8 + 2 * c + 1] = acc[t][3];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = 0.0f;
    }
    __syncthreads();
    const int64_t n0 = static_cast<int64_t>(tile) * kF8GemvRows;
    for (int i = threadIdx.x; i < kF8GemvRows * NT * 8; i += kF8GemvThreads) {
      const int r = i % kF8GemvRows, tok = i / kF8GemvRows;
      if (tok < a.M && n0 + r < a.N) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < kF8GemvWarps; ++k) s += part[(k * kF8GemvRows + r) * kPitch + tok];
        const int64_t at = tok * a.ldy + n0 + r;
        if (a.y_f32) static_cast<float*>(a.y)[at] = s;
        else static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(s);
      }
    }
    __syncthreads();
  };
  if (!busy) {                               // fewer blocks than warps: zeros to every sum
    for (int tile = blockIdx.x; tile < tiles; tile += grid) finish(tile);
    return;
  }
  int tile = blockIdx.x, kb = warp;
  while (tile < tiles) {
#pragma unroll
    for (int b = 0; b < kAhead; ++b) {
      if (tile >= tiles) break;
      const uint4 p0 = buf[b][0], q0 = buf[b][1], p1 = buf[b][2], q1 = buf[b][3];
      const float s = bsw[b];
      const uint8_t* xk = smem_raw + kb * kF8Block + 16 * c;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int tok = t * 8 + g;
        uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
        if (tok < a.M) {
          x0 = *reinterpret_cast<const uint4*>(xk + tok * lay.xs);
          x1 = *reinterpret_cast<const uint4*>(xk + tok * lay.xs + 64);
        }
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        mma_e4m3(d, p0.x, q0.x, p0.y, q0.y, x0.x, x0.y);
        mma_e4m3(d, p0.z, q0.z, p0.w, q0.w, x0.z, x0.w);
        mma_e4m3(d, p1.x, q1.x, p1.y, q1.y, x1.x, x1.y);
        mma_e4m3(d, p1.z, q1.z, p1.w, q1.w, x1.z, x1.w);
        const float2 sx = *reinterpret_cast<const float2*>(sxs + kb * (NT * 8) + t * 8 + 2 * c);
        const float s0 = s * sx.x, s1 = s * sx.y;
        acc[t][0] = fmaf(d[0], s0, acc[t][0]);
        acc[t][1] = fmaf(d[1], s1, acc[t][1]);
        acc[t][2] = fmaf(d[2], s0, acc[t][2]);
        acc[t][3] = fmaf(d[3], s1, acc[t][3]);
      }
      fetch(buf[b], bsw[b]);
      kb += kF8GemvWarps;
      if (kb >= blocks) {
        finish(tile);
        kb = warp;
        tile += grid;
      }
    }
  }
}

// ---------------------------------------------- many tokens: the 2-SM GEMM
constexpr int kF8EpiWarps = 8;
constexpr int kF8ProdWarp = 8;
constexpr int kF8IssueWarp = 9;                  // .. 12: an issuer per accumulator
constexpr int kF8ScaleWarp = 13;
constexpr int kF8ActWarp = 14;
constexpr int kF8Threads = 32 * 16;
// registers per thread: what the launch gives everyone, then the epilogue's
// two warpgroups take what the two others hand back
constexpr int kF8Regs = 128, kF8EpiRegs = 208, kF8RoleRegs = 48;
static_assert(256 * kF8EpiRegs + 256 * kF8RoleRegs <= kF8Threads * kF8Regs, "register split");
constexpr uint32_t kF8OpBytes = 128 * 128;       // 16 KB: 128 rows x 128 bytes
constexpr uint32_t kF8StageBytes = 4096;         // per epilogue warp: 32 rows x 128 bytes of output
constexpr uint32_t kF8ScaleBytes = (128 + 4) * 4; // 128 row scales, the weight's two (and padding)
// What depends on a tile's width, 128 HALVES columns: a block's product takes
// HALVES accumulators.
template <int MODE, int HALVES>
struct F8Cfg {
  // (dX takes whole boxes of 128 columns, the swizzle's width, also for its narrow tiles)
  static constexpr uint32_t kWBytes = MODE == 0 ? kF8OpBytes / 2 * HALVES : kF8OpBytes;
  static constexpr uint32_t kSlotBytes = kF8OpBytes + kWBytes;
  static constexpr int kRing = 6;
  static constexpr int kAccs = HALVES == 2 ? 4 : 3;
  static constexpr uint32_t kInFlight = kAccs / HALVES;         // blocks that the accumulators hold
  static constexpr uint32_t kScaleLag = 2;
  static constexpr uint32_t kScaleRing = kInFlight + kScaleLag;
  static constexpr uint32_t kOffStage = kRing * kSlotBytes;
  static constexpr uint32_t kOffScale = kOffStage + kF8EpiWarps * kF8StageBytes;
  static constexpr uint32_t kOffBar = kOffScale + kScaleRing * kF8ScaleBytes;
  static constexpr uint32_t kSmem = kOffBar + 256 /*bars*/;
  static_assert(kOffBar % 8 == 0, "barriers");
  // An issuer takes every kInFlight-th block and waits for a slot by the
  // parity of its phase: it must be the one that waited for the phase before.
  static_assert(kRing % kInFlight == 0, "an issuer comes back to its own slots");
  static_assert(kSmem <= 227 * 1024, "fp8 GEMM shared memory");
};
constexpr uint32_t kF8TmemCols = 512;
constexpr int kF8GroupM = 8;

struct Fp8GemmArgs {
  int64_t M;             // activation rows
  int64_t out_cols;      // N (forward) or K (dX)
  int64_t ctr;           // contraction length
  const float* sa;       // activation scales [ceil(ctr/128)][M]
  const float* sw;       // weight scales [ceil(N/128)][ceil(K/128)]
  int64_t sw_cols;       // ceil(K/128)
  void* out;
  int64_t ldo;
  int out_f32;
  int tma_out;           // tm_out maps the output (rows that start and end on 16 bytes)
  int tiles_m, tiles_n;
  int after_quant;       // launched as a dependent of the quantiser
  int* status;
};

// D[tmem] (+)= A[smem] * B[smem]^T over a 2-SM pair, E4M3 x E4M3 -> fp32, K = 32
__device__ __forceinline__ void umma_e4m3_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::f8f6f4: E4M3 x E4M3 (format 0) -> fp32
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, int b_mn_major) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn_major) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// 32 lanes x 32 bits, 32 consecutive columns per thread
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23,"
      " %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// acc += d * s on two fp32 values at once, each rounded once
__device__ __forceinline__ void fma_f32x2(uint64_t& acc, uint32_t d0, uint32_t d1, uint64_t s2) {
  asm("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\tfma.rn.f32x2 %0, d, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(d0), "r"(d1), "l"(s2));
}

// four bytes from global to shared memory without passing a register (zero
// where `in` does not hold; the address is not read then)
__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
// one of the arrivals that a barrier counts, once this thread's copies have landed
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// whether a phase is complete, without waiting
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// one thread of a converged warp, always the same one
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
// output tile t: groups of kF8GroupM tile rows, a group's columns one after
// the other, so that the tiles in flight share rows and columns in L2
__device__ __forceinline__ void f8_tile(int t, const Fp8GemmArgs& a, int& tm, int& tn) {
  const int per = kF8GroupM * a.tiles_n;
  const int g = t / per, r = t % per;
  const int h = min(kF8GroupM, a.tiles_m - g * kF8GroupM);
  tm = g * kF8GroupM + r % h;
  tn = r / h;
}

// MODE 0: forward (weight tile K-major), 1: dX (weight tile MN-major)
template <int MODE, int HALVES>
__global__ void __launch_bounds__(kF8Threads, 1)
    k_fp8_gemm(const __grid_constant__ CUtensorMap tm_act, const __grid_constant__ CUtensorMap tm_w,
               const __grid_constant__ CUtensorMap tm_out, const Fp8GemmArgs args) {
  using C = F8Cfg<MODE, HALVES>;
  constexpr uint32_t kDepth = C::kInFlight;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = smem_raw;
  if (smem_u32(base) % 1024 != 0) {      // the swizzled tiles' alignment (no room to round up)
    if (threadIdx.x == 0 && args.status) atomicOr(args.status, QLORA_DEV_TIMEOUT);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + C::kOffBar);
  uint64_t* full = bars;                         // [ring] leader: both CTAs' tiles landed
  uint64_t* empty = full + C::kRing;              // [ring] local: the issuers' MMAs done with the slot
  uint64_t* acc_full = empty + C::kRing;          // [4] local: accumulator holds its half of a block's product
  uint64_t* acc_empty = acc_full + C::kAccs;      // [4] leader: both CTAs have taken it out
  uint64_t* drained = acc_empty + C::kAccs;       // local: every MMA issued is done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* act_count = tmem_slot + 2;  // activation tiles asked for

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
  const int tiles = args.tiles_m * args.tiles_n;
  const int KB = static_cast<int>((args.ctr + kF8Block - 1) / kF8Block);
  const int mine = pair < tiles ? (tiles - pair + pairs - 1) / pairs : 0;   // this pair's tiles
  const uint32_t total = static_cast<uint32_t>(mine) * KB;                 // blocks over all of them (host: < 2^31)

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kRing; ++i) { mbar_init(smem_u32(&full[i]), 1); mbar_init(smem_u32(&empty[i]), HALVES); }
    for (int i = 0; i < C::kAccs; ++i) {
      mbar_init(smem_u32(&acc_full[i]), i % HALVES == 0 ? 1 + 32 : 1);   // the first half also brings the block's scales
      mbar_init(smem_u32(&acc_empty[i]), 2 * kF8EpiWarps);
    }
    mbar_init(smem_u32(drained), C::kAccs);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kF8ProdWarp) {
    if (lane == 0) { tma_prefetch_desc(&tm_act); tma_prefetch_desc(&tm_w); tma_prefetch_desc(&tm_out); }
    __syncwarp();
    tmem_alloc_pair(smem_u32(tmem_slot), kF8TmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();   // both CTAs' barriers initialised before any cross-CTA use
  tc_fence_after();
  const uint32_t tmem_d = *tmem_slot;
  auto leader_bar = [&](uint64_t* b) { return mapa_shared(smem_u32(b), 0); };
  if (threadIdx.x == 0) QLORA_CHECK_ONLY(C::kSmem <= dyn_smem_bytes(), 200);

  if (warp >= kF8EpiWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kF8RoleRegs));
    if (warp == kF8ProdWarp || warp == kF8ActWarp) {
      // ---------------------------------------------------------- producers
      // One thread brings the weight's tiles, another the activations' (one
      // thread for both took 0.37 us per block of a 128-column tile, against
      // 0.27).
      const bool weights = warp == kF8ProdWarp;
      uint32_t it = 0;
      if (lane == 0) {
        bool live = true;
        if (!weights && args.after_quant) griddep_wait();   // the activations come from the kernel ahead
        for (int t = pair; t < tiles && live; t += pairs) {
          int tm, tn;
          f8_tile(t, args, tm, tn);
          const int32_t m0 = tm * 256 + static_cast<int32_t>(rank) * 128;
          const int32_t c0 = (2 * tn + static_cast<int32_t>(rank)) * (64 * HALVES);   // this CTA's half of the output columns
          for (int kb = 0; kb < KB; ++kb, ++it) {
            const uint32_t s = it % C::kRing;
            if (it >= C::kRing && !mbar_wait(smem_u32(&empty[s]), (it / C::kRing + 1) & 1, abort_flag, args.status)) {
              live = false;
              break;
            }
            const uint32_t fb = leader_bar(&full[s]);
            if (weights && leader) mbar_arrive_expect_tx(smem_u32(&full[s]), 2 * C::kSlotBytes);
            const uint32_t dst = smem_u32(base) + s * C::kSlotBytes;
            // (a skipped load leaves the slot's wait to run out: bounded, the launch aborts)
            if (it == 0 && blockIdx.x == 0 && qlora_stalled()) continue;
            if (!QLORA_CHECK((s + 1) * C::kSlotBytes <= C::kOffStage && m0 >= 0 && c0 >= 0, 201)) continue;
            if (!weights) tma_load_2d_pair(dst, &tm_act, fb, kb * kF8Block, m0);
            else if (MODE == 0) tma_load_2d_pair(dst + kF8OpBytes, &tm_w, fb, kb * kF8Block, c0);
            else tma_load_2d_pair(dst + kF8OpBytes, &tm_w, fb, c0, kb * kF8Block);
          }
        }
        if (!weights) *act_count = it;
      }
      __syncwarp();
      named_bar_sync(1, 64);                                // both producers are through
      if (weights && lane == 0 && *abort_flag && leader) {
        // loads still in flight land before the CTA can exit
        it = max(it, *act_count);
        for (uint32_t i = it > C::kRing ? it - C::kRing : 0; i < it; ++i) {
          const uint64_t t1 = global_ns();
          while (!mbar_try_wait_cluster(smem_u32(&full[i % C::kRing]), (i / C::kRing) & 1) &&
                 global_ns() - t1 < qlora_drain_limit()) {}
        }
      }
    } else if (warp == kF8ScaleWarp) {
      // ------------------------------------------------------- scale warp
      // The scales of block `it` (128 rows' and the weight's two) into slot
      // it % (depth + lag), `lag` blocks ahead, by copies that count towards
      // the accumulator's barrier when they land (no registers: a value that
      // is spilled is waited for).  The slot is free: block it - lag has been
      // computed, so its accumulator was free before, so the epilogue is
      // through with block it - lag - depth.  Loads in the epilogue's own
      // warps stalled its multiply-adds (390 cycles for 64 columns against 150).
      const int64_t sw_step = MODE == 0 ? 1 : args.sw_cols, sw_run = MODE == 0 ? args.sw_cols : 1;
      const int64_t runs = (args.out_cols + kF8Block - 1) / kF8Block;
      if (args.after_quant) griddep_wait();
      uint32_t it = 0, slot = 0;
      bool live = true;
      for (int t = pair; t < tiles && live; t += pairs) {
        int tm, tn;
        f8_tile(t, args, tm, tn);
        const int64_t row = static_cast<int64_t>(tm) * 256 + rank * 128 + lane;
        const int64_t ob = HALVES == 2 ? 2 * static_cast<int64_t>(tn) + (lane & 1) : tn;
        const float* sa = args.sa;
        const float* sw = args.sw + (ob < runs ? ob * sw_run : 0);
        for (int kb = 0; kb < KB; ++kb, ++it) {
          if (it >= C::kScaleLag) {
            const uint32_t b = it - C::kScaleLag;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&acc_full[HALVES * (b % kDepth)]), (b / kDepth) & 1, abort_flag,
                                                   args.status))) {
              live = false;
              break;
            }
          }
          QLORA_CHECK_ONLY(C::kOffScale + (slot + 1) * kF8ScaleBytes <= C::kOffBar, 203);
          const uint32_t dst = smem_u32(base) + C::kOffScale + slot * kF8ScaleBytes + 4 * lane;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool in = row + 32 * i < args.M;
            cp_async4(dst + 128 * i, in ? sa + row + 32 * i : args.sa, in);
          }
          if (lane < 2) cp_async4(dst + 512, sw, true);
          cp_async_arrive(smem_u32(&acc_full[HALVES * (it % kDepth)]));
          slot = slot + 1 == C::kScaleRing ? 0 : slot + 1;
          sa += args.M;
          sw += sw_step;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp >= kF8IssueWarp && warp < kF8IssueWarp + C::kAccs && leader) {
      // --------------------------------------------- MMA issuers (leader)
      // Issuer j owns accumulator j: half j % HALVES of the blocks j / HALVES,
      // j / HALVES + depth, ...  The half: columns 64 (j % HALVES) .. of each
      // CTA's weight rows.
      // The whole warp runs the loop, so that the descriptors are uniform
      // values; one elected thread issues.
      const uint32_t j = warp - kF8IssueWarp, half = j % HALVES;
      constexpr uint32_t idesc = idesc_e4m3(256, 128, MODE);
      const uint32_t dcol = tmem_d + 128u * j;
      for (uint32_t it = j / HALVES; it < total; it += kDepth) {
        const uint32_t s = it % C::kRing, use = it / kDepth;
        bool ok = mbar_wait(smem_u32(&full[s]), (it / C::kRing) & 1, abort_flag, args.status);
        ok = ok && (use == 0 || mbar_wait(smem_u32(&acc_empty[j]), (use + 1) & 1, abort_flag, args.status));
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        tc_fence_after();
        const uint32_t ab = smem_u32(base) + s * C::kSlotBytes, wb = ab + kF8OpBytes + half * (MODE == 0 ? 8192u : 64u);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t adesc = sw128_desc(ab + k * 32, 16, 1024);
            const uint64_t bdesc = MODE == 0 ? sw128_desc(wb + k * 32, 16, 1024) : sw128_desc(wb + k * 4096, 16384, 1024);
            umma_e4m3_pair(dcol, adesc, bdesc, idesc, k > 0 ? 1u : 0u);
          }
          umma_commit_pair(smem_u32(&acc_full[j]), 0x3);
          umma_commit_pair(smem_u32(&empty[s]), 0x3);
        }
        __syncwarp();
      }
      if (elect_one()) umma_commit_pair(smem_u32(drained), 0x3);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // Warp w: rows 32 (w % 4) .. of this CTA; of each accumulator the 64
    // columns that come from CTA p = w / 4's weight rows, so that a warp's
    // 64 HALVES output columns lie in one scale block.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kF8EpiRegs));
    const int q = warp & 3, p = warp >> 2;
    const uint32_t taddr = tmem_d + (static_cast<uint32_t>(q * 32) << 16) + 64u * p;
    const uint32_t freed = leader_bar(&acc_empty[0]), filled = smem_u32(&acc_full[0]);
    bool ahead = false;
    uint8_t* stage = base + C::kOffStage + warp * kF8StageBytes;
    uint32_t it = 0;
    bool live = true;
    for (int t = pair; t < tiles && live; t += pairs) {
      int tm, tn;
      f8_tile(t, args, tm, tn);
      const int64_t row0 = static_cast<int64_t>(tm) * 256 + rank * 128 + q * 32;
      const int64_t col = (2 * static_cast<int64_t>(tn) + p) * (64 * HALVES);
      uint64_t acc[32 * HALVES];
#pragma unroll
      for (int i = 0; i < 32 * HALVES; ++i) acc[i] = 0;
      for (int kb = 0; kb < KB && live; ++kb, ++it) {
        uint64_t s2 = 0;
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
          const uint32_t buf = HALVES * (it % kDepth) + h;
          // (votes: the lanes of a warp take the same way out of an aborted launch)
          if (!__all_sync(0xFFFFFFFFu, ahead) &&
              !__all_sync(0xFFFFFFFFu, mbar_wait(filled + 8 * buf, (it / kDepth) & 1, abort_flag, args.status))) {
            live = false;
            break;
          }
          tc_fence_after();
          uint32_t r[64];
          tmem_ld32(taddr + 128u * buf, r);
          tmem_ld32(taddr + 128u * buf + 32, r + 32);
          tmem_ld_wait();
          if (h == 0) {
            const float* slot = reinterpret_cast<const float*>(base + C::kOffScale + (it % C::kScaleRing) * kF8ScaleBytes);
            const float s = slot[32 * q + lane] * slot[128 + p];
            asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(s));
          }
          // the product is in registers: the next one may overwrite it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(freed + 8 * buf);
          // whether the next product is there already, asked now and looked at after the additions
          const uint32_t next = HALVES * it + h + 1;             // counted in accumulators
          ahead = mbar_test(filled + 8 * (next % C::kAccs), (next / C::kAccs) & 1);
#pragma unroll
          for (int i = 0; i < 32; ++i) fma_f32x2(acc[32 * h + i], r[2 * i], r[2 * i + 1], s2);
        }
      }
      if (!live) break;
      // Out through shared memory, 128 bytes of each of the warp's 32 rows at
      // a time (128-byte swizzle), so that global memory sees whole rows of a
      // box: by a TMA store, or by the lanes where rows do not start and end on
      // 16 bytes.
      const int per = args.out_f32 ? 32 : 64;                      // columns of a box
#pragma unroll
      for (int b = 0; b < 2 * HALVES; ++b) {
        if (!args.out_f32 && b >= HALVES) break;
        if (lane == 0) bulk_wait_read();                           // the box before has been read
        __syncwarp();
        QLORA_CHECK_ONLY(C::kOffStage + (warp + 1) * kF8StageBytes <= C::kOffScale, 202);
        uint8_t* line = stage + lane * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint4 v;
          if (args.out_f32) {
            const uint64_t x = acc[16 * b + 2 * c], y = acc[16 * b + 2 * c + 1];
            v = make_uint4(static_cast<uint32_t>(x), static_cast<uint32_t>(x >> 32), static_cast<uint32_t>(y),
                           static_cast<uint32_t>(y >> 32));
          } else {
            uint32_t pk[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint64_t x = acc[(32 * b + 4 * c + i) % (32 * HALVES)];
              pk[i] = pack_bf16x2(__uint_as_float(static_cast<uint32_t>(x)), __uint_as_float(static_cast<uint32_t>(x >> 32)));
            }
            v = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
          *reinterpret_cast<uint4*>(line + ((c ^ (lane & 7)) << 4)) = v;
        }
        const int64_t bx = col + b * per;
        if (args.tma_out) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && bx < args.out_cols && row0 < args.M) {
            tma_store_2d(&tm_out, smem_u32(stage), static_cast<int32_t>(bx), static_cast<int32_t>(row0));
            bulk_commit();
          }
        } else {
          __syncwarp();
          const int64_t left = args.out_cols - bx;
          for (int r = 0; r < 32 && row0 + r < args.M; ++r) {
            const uint32_t v = *reinterpret_cast<const uint32_t*>(stage + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
            if (args.out_f32) {
              if (lane < left) static_cast<float*>(args.out)[(row0 + r) * args.ldo + bx + lane] = __uint_as_float(v);
            } else {
              __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(args.out) + (row0 + r) * args.ldo + bx + 2 * lane;
              if (2 * lane < left) dst[0] = __ushort_as_bfloat16(static_cast<uint16_t>(v));
              if (2 * lane + 1 < left) dst[1] = __ushort_as_bfloat16(static_cast<uint16_t>(v >> 16));
            }
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) bulk_wait_read();   // the stores have read their boxes before the CTA can exit
  }

  // Single-lane roles leave their warps diverged; the cluster barrier is
  // warp-aligned, and tensor memory must not be released under running MMAs
  // (on an aborted launch some may be: wait for the issuers' last commit).
  __syncwarp();
  if (warp == kF8ProdWarp) {
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait_cluster(smem_u32(drained), 0) && global_ns() - t0 < qlora_wait_limit()) {}
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == kF8ProdWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_d, kF8TmemCols);
  }
}

using Fp8Gemm = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, Fp8GemmArgs);

}  // namespace qlora
