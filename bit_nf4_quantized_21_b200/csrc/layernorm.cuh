// layernorm.cuh -- layer norm over the last dimension, forward and backward,
// with the reduction of the weight's and the bias's gradient.
//
//   mean = sum x / C        rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//   y  = (x - mean) rstd w + b
//   xh = (x - mean) rstd    g = dy w
//   dx = rstd (g - mean(g) - xh mean(g xh))
//   dw = sum over rows of dy xh        db = sum over rows of dy
//
// Every sum is fp32; the variance is the sum of squared differences from
// the mean (a second sweep over registers), never sum(x^2) - mean^2, which
// loses everything when the mean is far above the spread.  A row is read
// from memory once and held in registers between the sweeps; outputs are
// rounded once.
//
// HBM bound: 2 elements moved per element forward, 3 backward.  A group of
// GROUP threads owns a row (a warp for short rows, so that no block barrier
// is needed; up to 1024 threads for long ones), each thread PER chunks of
// VEC elements.  VEC is 16 bytes when the row length, strides and pointers
// allow it, otherwise one element.  Rows that do not fit the registers take
// the streaming kernels, which read a row again from L1/L2 per sweep.
//
// The backward walks rows with a fixed grid: a thread keeps the same columns
// for every row, so its share of dw and db accumulates in registers and is
// written once per block as a row of partials; k_ln_finish adds the partials
// in a fixed order (no atomics: results do not depend on scheduling).
//
// Measured on the device (calls in a graph, each on inputs that are not in L2)
// against a copy's rate of 6.57 TB/s, bf16 unless said.  Forward 8192 x 8192
// 48 us (5.6 TB/s; the copy would take 40.9), 4096 x 4096 16.8 us (10.2), fp32
// 26 us (20.4), 16 x 4096 2.9 us (two dependent trips to memory and a launch).
// Backward 8192 x 8192 77 us (61.3), 4096 x 4096 26 us (15.3; 21.7 without the
// parameters' gradients: writing one row of partials per block and adding them
// up is the rest), fp32 40 us (30.7).  Rows that are not 16-byte aligned take
// single-element loads and stores and never the ring: 8000 x 1500 bf16 31 us
// forward (7.3) and 56 backward (11.0), 1237 x 2051 fp32 19 us backward (4.6).
// The streaming kernels: 4096 x 12288 fp32 88 us forward (61) and 262 backward
// (92; 149 without the parameters' gradients), 2048 x 12001 bf16 50 (15) and
// 120 (22).
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "ptx.cuh"
#include "f32x2.cuh"

namespace qlora {

constexpr int kLnMaxParts = 592;     // most partial rows of dw/db that a backward call writes

struct LnArgs {
  const void* x;
  int64_t ldx;
  const void* w;        // nullable: ones
  const void* b;        // nullable: zeros
  int w_bf16;
  int64_t rows, cols;
  float eps;
  void* y;              // forward
  int64_t ldy;
  float* mean;          // forward: written when non-null; backward: read
  float* rstd;
  const void* dy;       // backward
  int64_t lddy;
  void* dx;
  int64_t lddx;
  float* part;          // [parts][2][cols] partials of dw, db; null: not wanted
  int stages;           // ring kernels: rows in shared memory
  int* status;
};

template <typename T> struct LnElem;
template <> struct LnElem<float> { static constexpr int kVec = 4; };
template <> struct LnElem<__nv_bfloat16> { static constexpr int kVec = 8; };

// VEC consecutive elements as loaded (16 bytes, or one element)
template <typename T, int VEC> struct LnRaw;
template <> struct LnRaw<__nv_bfloat16, 8> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
};
template <> struct LnRaw<float, 4> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; }
};
template <> struct LnRaw<__nv_bfloat16, 1> {
  __nv_bfloat16 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *p; }
  __device__ __forceinline__ void zero() { v = __float2bfloat16_rn(0.0f); }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = __bfloat162float(v); }
};
template <> struct LnRaw<float, 1> {
  float v;
  __device__ __forceinline__ void load(const float* p) { v = *p; }
  __device__ __forceinline__ void zero() { v = 0.0f; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = v; }
};

__device__ __forceinline__ void ln_store(__nv_bfloat16* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                            pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void ln_store(float* p, const float (&f)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void ln_store(__nv_bfloat16* p, const float (&f)[1]) { *p = __float2bfloat16_rn(f[0]); }
__device__ __forceinline__ void ln_store(float* p, const float (&f)[1]) { *p = f[0]; }

// VEC parameters (weight or bias, bf16 or fp32) from column c; `fill` when absent
template <int VEC>
__device__ __forceinline__ void ln_param(const void* p, int bf16, int64_t c, float fill, float (&f)[VEC]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = fill;
  } else if (VEC == 1) {
    f[0] = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[c]) : static_cast<const float*>(p)[c];
  } else if (bf16) {
    const uint2* q = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + c);
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const uint2 u = q[i];
      f[4 * i] = __uint_as_float(u.x << 16);
      f[4 * i + 1] = __uint_as_float(u.x & 0xFFFF0000u);
      f[4 * i + 2] = __uint_as_float(u.y << 16);
      f[4 * i + 3] = __uint_as_float(u.y & 0xFFFF0000u);
    }
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + c);
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const float4 u = q[i];
      f[4 * i] = u.x; f[4 * i + 1] = u.y; f[4 * i + 2] = u.z; f[4 * i + 3] = u.w;
    }
  }
}

// Sums of two values over a group of GROUP threads, the same in every thread
// of the group.  `red` holds one float2 per warp; consecutive calls of a
// block alternate between two such buffers, so one barrier per call is
// enough (a buffer is written again only after the next call's barrier).
template <int GROUP>
__device__ __forceinline__ float2 ln_group_sum(float2 v, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
    v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
  }
  if (GROUP == 32) return v;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  __syncthreads();
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < GROUP / 64; ++i) {
    const float4 u = reinterpret_cast<const float4*>(red)[i];   // two warps' sums
    s.x += u.x + u.z;
    s.y += u.y + u.w;
  }
  return s;
}
// the same for one value; `red` as one float per warp
template <int GROUP>
__device__ __forceinline__ float ln_group_sum1(float v, float2* red2) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (GROUP == 32) return v;
  float* red = reinterpret_cast<float*>(red2);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < GROUP / 128; ++i) {
    const float4 u = reinterpret_cast<const float4*>(red)[i];   // four warps' sums
    s += (u.x + u.y) + (u.z + u.w);
  }
  return s;
}

template <int GROUP> constexpr int ln_block() { return GROUP < 128 ? 128 : GROUP; }
// backward: eight warps' rows, whose partials the block adds up itself
template <int GROUP> constexpr int ln_bwd_block() { return GROUP < 128 ? 256 : GROUP; }

template <typename T, int VEC, int GROUP, int PER>
__global__ void __launch_bounds__(ln_block<GROUP>()) k_ln_fwd(const LnArgs a) {
  constexpr int kRows = ln_block<GROUP>() / GROUP;
  __shared__ __align__(16) float2 red[2][32];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / GROUP;
  const int t = threadIdx.x % GROUP;
  if (row >= a.rows) return;            // whole warps only: a group of a warp, or the block's one row
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  LnRaw<T, VEC> raw[PER];
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int64_t c = static_cast<int64_t>(t + i * GROUP) * VEC;
    if (c < a.cols) raw[i].load(x + c); else raw[i].zero();
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    float f[VEC];
    raw[i].get(f);
#pragma unroll
    for (int e = 0; e < VEC; ++e) s += f[e];
  }
  const float inv = 1.0f / static_cast<float>(a.cols);
  const float mean = ln_group_sum1<GROUP>(s, red[0]) * inv;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int64_t c = static_cast<int64_t>(t + i * GROUP) * VEC;
    float f[VEC];
    raw[i].get(f);
    if (c < a.cols) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = f[e] - mean;
        s = fmaf(d, d, s);
      }
    }
  }
  const float rstd = 1.0f / sqrtf(ln_group_sum1<GROUP>(s, red[1]) * inv + a.eps);
  T* y = static_cast<T*>(a.y) + row * a.ldy;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int64_t c = static_cast<int64_t>(t + i * GROUP) * VEC;
    if (c < a.cols) {
      float f[VEC], w[VEC], b[VEC];
      raw[i].get(f);
      ln_param<VEC>(a.w, a.w_bf16, c, 1.0f, w);
      ln_param<VEC>(a.b, a.w_bf16, c, 0.0f, b);
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = fmaf((f[e] - mean) * rstd, w[e], b[e]);
      ln_store(y + c, f);
    }
  }
  if (t == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

// Any row length: a block per row, the row read again per sweep.
constexpr int kLnStreamThreads = 512;
template <typename T>
__global__ void __launch_bounds__(kLnStreamThreads) k_ln_fwd_stream(const LnArgs a) {
  __shared__ __align__(16) float2 red[2][32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const float inv = 1.0f / static_cast<float>(a.cols);
  float s = 0.0f;
  for (int64_t c = threadIdx.x; c < a.cols; c += kLnStreamThreads) s += static_cast<float>(x[c]);
  const float mean = ln_group_sum1<kLnStreamThreads>(s, red[0]) * inv;
  s = 0.0f;
  for (int64_t c = threadIdx.x; c < a.cols; c += kLnStreamThreads) {
    const float d = static_cast<float>(x[c]) - mean;
    s = fmaf(d, d, s);
  }
  const float rstd = 1.0f / sqrtf(ln_group_sum1<kLnStreamThreads>(s, red[1]) * inv + a.eps);
  T* y = static_cast<T*>(a.y) + row * a.ldy;
  for (int64_t c = threadIdx.x; c < a.cols; c += kLnStreamThreads) {
    float w[1], b[1], f[1];
    ln_param<1>(a.w, a.w_bf16, c, 1.0f, w);
    ln_param<1>(a.b, a.w_bf16, c, 0.0f, b);
    f[0] = fmaf((static_cast<float>(x[c]) - mean) * rstd, w[0], b[0]);
    ln_store(y + c, f);
  }
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

// One group's sums of dw and db as row `group` of the partials.
template <int VEC, int GROUP, int PER>
__device__ __forceinline__ void ln_write_part(const LnArgs& a, int64_t group, int t, const float (&dw)[PER][VEC],
                                              const float (&db)[PER][VEC]) {
  float* pw = a.part + group * 2 * a.cols;
  float* pb = pw + a.cols;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int64_t c = static_cast<int64_t>(t + i * GROUP) * VEC;
    if (c < a.cols) {
      if (VEC == 1) {
        pw[c] = dw[i][0];
        pb[c] = db[i][0];
      } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
          *reinterpret_cast<float4*>(pw + c + e) =
              make_float4(dw[i][e], dw[i][(e + 1) % VEC], dw[i][(e + 2) % VEC], dw[i][(e + 3) % VEC]);
          *reinterpret_cast<float4*>(pb + c + e) =
              make_float4(db[i][e], db[i][(e + 1) % VEC], db[i][(e + 2) % VEC], db[i][(e + 3) % VEC]);
        }
      }
    }
  }
}

// Backward, rows in registers.  The grid walks the rows; the loads of the
// next row are in flight while the current one is reduced.
template <typename T, int VEC, int GROUP, int PER>
__global__ void __launch_bounds__(ln_bwd_block<GROUP>(), PER > 8 ? 3 : GROUP <= 512 ? 2 : 1) k_ln_bwd(const LnArgs a) {
  constexpr int kRows = ln_bwd_block<GROUP>() / GROUP;
  __shared__ __align__(16) float2 red[2][32];
  const int t = threadIdx.x % GROUP;
  const int64_t group = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / GROUP;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  float dw[PER][VEC], db[PER][VEC];
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[i][e] = db[i][e] = 0.0f;
  const float inv = 1.0f / static_cast<float>(a.cols);
  LnRaw<T, VEC> rx[PER], rd[PER];
  float mean = 0.0f, rstd = 0.0f;
  auto fetch = [&](int64_t row) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int64_t c = static_cast<int64_t>(t + i * GROUP) * VEC;
      if (c < a.cols) { rx[i].load(x + c); rd[i].load(dy + c); } else { rx[i].zero(); rd[i].zero(); }
    }
    mean = a.mean[row];
    rstd = a.rstd[row];
  };
  // a group of a warp ends its loop by itself; a group of a block has one row per block
  int64_t row = group;
  if (row < a.rows) fetch(row);
  int buf = 0;
  for (; row < a.rows; row += step) {
    LnRaw<T, VEC> x[PER], d[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) { x[i] = rx[i]; d[i] = rd[i]; }
    const float mu = mean, rs = rstd;
    if (row + step < a.rows) fetch(row + step);
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int64_t c = static_cast<int64_t>(t + i * GROUP) * VEC;
      if (c < a.cols) {
        float fx[VEC], fd[VEC], w[VEC];
        x[i].get(fx);
        d[i].get(fd);
        ln_param<VEC>(a.w, a.w_bf16, c, 1.0f, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = (fx[e] - mu) * rs, g = fd[e] * w[e];
          s.x += g;
          s.y = fmaf(g, xh, s.y);
          dw[i][e] = fmaf(fd[e], xh, dw[i][e]);
          db[i][e] += fd[e];
        }
      }
    }
    s = ln_group_sum<GROUP>(s, red[buf]);
    buf ^= 1;
    const float m1 = s.x * inv, m2 = s.y * inv;
    T* dx = static_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int64_t c = static_cast<int64_t>(t + i * GROUP) * VEC;
      if (c < a.cols) {
        float fx[VEC], fd[VEC], w[VEC], o[VEC];
        x[i].get(fx);
        d[i].get(fd);
        ln_param<VEC>(a.w, a.w_bf16, c, 1.0f, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = (fx[e] - mu) * rs;
          o[e] = rs * (fmaf(fd[e], w[e], -m1) - xh * m2);
        }
        ln_store(dx + c, o);
      }
    }
  }
  griddep_launch_dependents();             // k_ln_finish
  if (!a.part) return;
  if (kRows == 1) {
    ln_write_part<VEC, GROUP, PER>(a, group, t, dw, db);
  } else {
    // one row of partials per block: the warps' sums added in warp order
    constexpr int kCols = GROUP * PER * VEC;
    __shared__ float sums[kRows][kRows == 1 ? 1 : kCols];
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < PER; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) sums[threadIdx.x / GROUP][(t + i * GROUP) * VEC + e] = which ? db[i][e] : dw[i][e];
      __syncthreads();
      float* p = a.part + (static_cast<int64_t>(blockIdx.x) * 2 + which) * a.cols;
      for (int c = threadIdx.x; c < a.cols; c += ln_bwd_block<GROUP>()) {
        float v = sums[0][c];
#pragma unroll
        for (int k = 1; k < kRows; ++k) v += sums[k][c];
        p[c] = v;
      }
    }
  }
}

// ------------------------------------------------------ rows through a ring
// Many rows of 16-byte aligned chunks: a block walks its rows, which arrive in
// a ring in shared memory by bulk copies (one thread asks for a whole row),
// several rows ahead.  Registers alone kept 16 to 32 KB per SM on their way
// and reached 3 TB/s; the ring keeps up to 200 KB.  A slot is refilled after
// the block barrier of its row's first reduction, which every thread reaches
// with the row in registers.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}
constexpr int kLnMaxStages = 8;
// After a wait that gave up: the loads still under way land before the block
// can exit (bounded).  By the thread that asked for them.
__device__ __noinline__ void ln_drain(uint64_t* full, int stages, int64_t asked) {
  for (int64_t i = asked > stages ? asked - stages : 0; i < asked; ++i) {
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait(smem_u32(&full[i % stages]), static_cast<uint32_t>((i / stages) & 1)) &&
           global_ns() - t0 < qlora_drain_limit()) {}
  }
}

// The ring kernels' arithmetic per byte is what keeps them from the memory's
// rate: packed pairs of fp32 halve its instructions.
// VEC elements from shared memory as pairs; zeros past the last column
template <typename T, int VEC>
__device__ __forceinline__ void ln_pairs(const T* p, bool in, f32x2 (&v)[VEC / 2]) {
  LnRaw<T, VEC> raw;
  if (in) raw.load(p); else raw.zero();
  float f[VEC];
  raw.get(f);
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) v[i] = pair2(f[2 * i], f[2 * i + 1]);
}
template <int VEC>
__device__ __forceinline__ void ln_param_pairs(const void* p, int bf16, int64_t c, float fill, f32x2 (&v)[VEC / 2]) {
  float f[VEC];
  ln_param<VEC>(p, bf16, c, fill, f);
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) v[i] = pair2(f[2 * i], f[2 * i + 1]);
}
template <typename T, int VEC>
__device__ __forceinline__ void ln_store_pairs(T* p, const f32x2 (&v)[VEC / 2]) {
  float f[VEC];
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    const float2 u = unpair2(v[i]);
    f[2 * i] = u.x;
    f[2 * i + 1] = u.y;
  }
  ln_store(p, f);
}

// FULL: the row is exactly GROUP * PER chunks, so no thread is past its end.
template <typename T, int GROUP, int PER, bool FULL>
__global__ void __launch_bounds__(GROUP, 1024 / GROUP) k_ln_fwd_ring(const LnArgs a) {
  constexpr int VEC = LnElem<T>::kVec, H = VEC / 2;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) float2 red[2][32];
  __shared__ uint64_t full[kLnMaxStages];
  __shared__ int abort_word;
  __shared__ int asked;                    // rows asked for (thread 0's; kept out of its registers)
  const int t = threadIdx.x;
  const int cols = static_cast<int>(a.cols);
  const uint32_t row_bytes = static_cast<uint32_t>(cols * sizeof(T));
  const int mine = static_cast<int>((a.rows - blockIdx.x + gridDim.x - 1) / gridDim.x);   // rows of this block
  if (t == 0) {
    for (int i = 0; i < a.stages; ++i) mbar_init(smem_u32(&full[i]), 1);
    abort_word = 0;
    asked = 0;
    fence_mbar_init();
  }
  __syncthreads();
  auto ask = [&](int i, int s) {       // row i of this block into slot s
    asked = i + 1;
    mbar_arrive_expect_tx(smem_u32(&full[s]), row_bytes);
    bulk_load(smem_u32(ring) + s * row_bytes, static_cast<const T*>(a.x) + static_cast<int64_t>(blockIdx.x + i * gridDim.x) * a.ldx, row_bytes,
              smem_u32(&full[s]));
  };
  if (t == 0) {
    // (the test hook: the first row never comes, its barrier only expects it)
    const bool stall = blockIdx.x == 0 && qlora_stalled();
    if (stall) mbar_arrive_expect_tx(smem_u32(&full[0]), row_bytes);
    for (int i = stall ? 1 : 0; i < a.stages && i < mine; ++i) ask(i, i);
  }
  f32x2 w[PER][H], b[PER][H];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int c = (t + k * GROUP) * VEC;
    if (FULL || c < cols) {
      ln_param_pairs<VEC>(a.w, a.w_bf16, c, 1.0f, w[k]);
      ln_param_pairs<VEC>(a.b, a.w_bf16, c, 0.0f, b[k]);
    }
  }
  const float inv = 1.0f / static_cast<float>(cols);
  int s = 0;
  uint32_t parity = 0;
  bool came = true;                        // every row so far
  for (int i = 0; i < mine; ++i) {
    const int64_t row = static_cast<int>(blockIdx.x + i * gridDim.x);
    // A wait that gives up says so in *status.  Every later wait then gives up
    // at once, and no more rows are asked for (a slot whose row has not come
    // is still in its old phase), so the launch runs out quickly.
    came = mbar_wait(smem_u32(&full[s]), parity, &abort_word, a.status) && came;
    const T* src = reinterpret_cast<const T*>(ring + s * row_bytes);
    f32x2 v[PER][H], acc = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int c = (t + k * GROUP) * VEC;
      ln_pairs<T, VEC>(src + c, FULL || c < cols, v[k]);
#pragma unroll
      for (int e = 0; e < H; ++e) acc = add2(acc, v[k][e]);
    }
    float2 sum = unpair2(acc);
    const float mean = ln_group_sum1<GROUP>(sum.x + sum.y, red[0]) * inv;
    if (t == 0 && i + a.stages < mine && came) ask(i + a.stages, s);
    const f32x2 neg = pair2(-mean, -mean);
    acc = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      if (FULL || (t + k * GROUP) * VEC < cols) {
#pragma unroll
        for (int e = 0; e < H; ++e) {
          v[k][e] = add2(v[k][e], neg);
          acc = fma2(v[k][e], v[k][e], acc);
        }
      }
    }
    sum = unpair2(acc);
    const float rstd = 1.0f / sqrtf(ln_group_sum1<GROUP>(sum.x + sum.y, red[1]) * inv + a.eps);
    const f32x2 scale = pair2(rstd, rstd);
    T* y = static_cast<T*>(a.y) + row * a.ldy;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int c = (t + k * GROUP) * VEC;
      if (FULL || c < cols) {
#pragma unroll
        for (int e = 0; e < H; ++e) v[k][e] = fma2(mul2(v[k][e], scale), w[k][e], b[k][e]);
        ln_store_pairs<T, VEC>(y + c, v[k]);
      }
    }
    if (t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    if (++s == a.stages) { s = 0; parity ^= 1; }
  }
  if (t == 0 && *const_cast<volatile int*>(&abort_word)) ln_drain(full, a.stages, asked);
}

template <typename T, int GROUP, int PER, bool FULL>
__global__ void __launch_bounds__(GROUP) k_ln_bwd_ring(const LnArgs a) {
  constexpr int VEC = LnElem<T>::kVec, H = VEC / 2;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) float2 red[2][32];
  __shared__ uint64_t full[kLnMaxStages];
  __shared__ int abort_word;
  __shared__ int asked;                    // rows asked for (thread 0's; kept out of its registers)
  const int t = threadIdx.x;
  const int cols = static_cast<int>(a.cols);
  const uint32_t row_bytes = static_cast<uint32_t>(cols * sizeof(T));
  const int mine = static_cast<int>((a.rows - blockIdx.x + gridDim.x - 1) / gridDim.x);
  if (t == 0) {
    for (int i = 0; i < a.stages; ++i) mbar_init(smem_u32(&full[i]), 1);
    abort_word = 0;
    asked = 0;
    fence_mbar_init();
  }
  __syncthreads();
  auto ask = [&](int i, int s) {       // rows i of x and dy into slot s
    asked = i + 1;
    const int64_t row = static_cast<int>(blockIdx.x + i * gridDim.x);
    const uint32_t bar = smem_u32(&full[s]), dst = smem_u32(ring) + 2 * s * row_bytes;
    mbar_arrive_expect_tx(bar, 2 * row_bytes);
    bulk_load(dst, static_cast<const T*>(a.x) + row * a.ldx, row_bytes, bar);
    bulk_load(dst + row_bytes, static_cast<const T*>(a.dy) + row * a.lddy, row_bytes, bar);
  };
  if (t == 0) {
    // (the test hook: the first row never comes, its barrier only expects it)
    const bool stall = blockIdx.x == 0 && qlora_stalled();
    if (stall) mbar_arrive_expect_tx(smem_u32(&full[0]), row_bytes);
    for (int i = stall ? 1 : 0; i < a.stages && i < mine; ++i) ask(i, i);
  }
  f32x2 w[PER][H], dw[PER][H], db[PER][H];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int c = (t + k * GROUP) * VEC;
#pragma unroll
    for (int e = 0; e < H; ++e) w[k][e] = dw[k][e] = db[k][e] = 0;
    if (FULL || c < cols) ln_param_pairs<VEC>(a.w, a.w_bf16, c, 1.0f, w[k]);
  }
  const float inv = 1.0f / static_cast<float>(cols);
  int s = 0;
  uint32_t parity = 0;
  bool came = true;                        // every row so far
  float mu = a.mean[blockIdx.x], rs = a.rstd[blockIdx.x];
  for (int i = 0; i < mine; ++i) {
    const int64_t row = static_cast<int>(blockIdx.x + i * gridDim.x);
    const int64_t next = i + 1 < mine ? row + gridDim.x : row;
    const float mu_next = a.mean[next], rs_next = a.rstd[next];
    came = mbar_wait(smem_u32(&full[s]), parity, &abort_word, a.status) && came;   // (as in the forward)
    const T* xs = reinterpret_cast<const T*>(ring + 2 * s * row_bytes);
    const T* ds = reinterpret_cast<const T*>(ring + (2 * s + 1) * row_bytes);
    const f32x2 neg = pair2(-mu, -mu), scale = pair2(rs, rs);
    f32x2 xh[PER][H], g[PER][H], sg = 0, sgx = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      // (past the last column w and dy are zero, so nothing is added)
      const int c = (t + k * GROUP) * VEC;
      ln_pairs<T, VEC>(xs + c, FULL || c < cols, xh[k]);
      ln_pairs<T, VEC>(ds + c, FULL || c < cols, g[k]);
#pragma unroll
      for (int e = 0; e < H; ++e) {
        xh[k][e] = mul2(add2(xh[k][e], neg), scale);
        dw[k][e] = fma2(g[k][e], xh[k][e], dw[k][e]);
        db[k][e] = add2(db[k][e], g[k][e]);
        g[k][e] = mul2(g[k][e], w[k][e]);
        sg = add2(sg, g[k][e]);
        sgx = fma2(g[k][e], xh[k][e], sgx);
      }
    }
    const float2 p = unpair2(sg), q = unpair2(sgx);
    const float2 sum = ln_group_sum<GROUP>(make_float2(p.x + p.y, q.x + q.y), red[i & 1]);
    if (t == 0 && i + a.stages < mine && came) ask(i + a.stages, s);
    const float m1 = -sum.x * inv, m2 = -sum.y * inv;
    const f32x2 n1 = pair2(m1, m1), n2 = pair2(m2, m2);
    T* dx = static_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int c = (t + k * GROUP) * VEC;
      if (FULL || c < cols) {
#pragma unroll
        for (int e = 0; e < H; ++e) g[k][e] = mul2(fma2(xh[k][e], n2, add2(g[k][e], n1)), scale);
        ln_store_pairs<T, VEC>(dx + c, g[k]);
      }
    }
    mu = mu_next;
    rs = rs_next;
    if (++s == a.stages) { s = 0; parity ^= 1; }
  }
  if (t == 0 && *const_cast<volatile int*>(&abort_word)) ln_drain(full, a.stages, asked);
  griddep_launch_dependents();             // k_ln_finish
  if (a.part) {
    float fw[PER][VEC], fb[PER][VEC];
#pragma unroll
    for (int k = 0; k < PER; ++k)
#pragma unroll
      for (int e = 0; e < H; ++e) {
        const float2 u = unpair2(dw[k][e]), v = unpair2(db[k][e]);
        fw[k][2 * e] = u.x; fw[k][2 * e + 1] = u.y;
        fb[k][2 * e] = v.x; fb[k][2 * e + 1] = v.y;
      }
    ln_write_part<VEC, GROUP, PER>(a, blockIdx.x, t, fw, fb);
  }
}

// Any row length: the columns' partials (k_ln_bwd_cols: a thread per column
// and a run of rows per block row of the grid), then dx with a block per row.
// In that order, because dX may be X or dY.
template <typename T>
__global__ void __launch_bounds__(kLnStreamThreads) k_ln_bwd_stream(const LnArgs a) {
  __shared__ __align__(16) float2 red[2][32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
  const float mu = a.mean[row], rs = a.rstd[row];
  float2 s = make_float2(0.0f, 0.0f);
  for (int64_t c = threadIdx.x; c < a.cols; c += kLnStreamThreads) {
    float w[1];
    ln_param<1>(a.w, a.w_bf16, c, 1.0f, w);
    const float g = static_cast<float>(dy[c]) * w[0];
    s.x += g;
    s.y = fmaf(g, (static_cast<float>(x[c]) - mu) * rs, s.y);
  }
  s = ln_group_sum<kLnStreamThreads>(s, red[0]);
  const float inv = 1.0f / static_cast<float>(a.cols);
  const float m1 = s.x * inv, m2 = s.y * inv;
  T* dx = static_cast<T*>(a.dx) + row * a.lddx;
  for (int64_t c = threadIdx.x; c < a.cols; c += kLnStreamThreads) {
    float w[1], o[1];
    ln_param<1>(a.w, a.w_bf16, c, 1.0f, w);
    const float xh = (static_cast<float>(x[c]) - mu) * rs;
    o[0] = rs * (fmaf(static_cast<float>(dy[c]), w[0], -m1) - xh * m2);
    ln_store(dx + c, o);
  }
}

constexpr int kLnColThreads = 128;
template <typename T>
__global__ void __launch_bounds__(kLnColThreads) k_ln_bwd_cols(const LnArgs a) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kLnColThreads + threadIdx.x;
  if (c >= a.cols) return;
  float dw = 0.0f, db = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float d = static_cast<float>(static_cast<const T*>(a.dy)[row * a.lddy + c]);
    const float xh = (static_cast<float>(static_cast<const T*>(a.x)[row * a.ldx + c]) - a.mean[row]) * a.rstd[row];
    dw = fmaf(d, xh, dw);
    db += d;
  }
  float* pw = a.part + static_cast<int64_t>(blockIdx.y) * 2 * a.cols;
  pw[c] = dw;
  pw[a.cols + c] = db;
}

// dw and db from the partial rows, which are read as rows of 2 cols values:
// 32 of them per block, 16 bytes per thread, 32 threads down the rows with
// all their loads in flight; the threads' sums are added in a fixed order.
struct LnFinishArgs {
  const float* part;
  int parts;
  int64_t cols;
  void* dw;             // nullable
  void* db;             // nullable
  int out_bf16;
  int dependent;        // launched behind the kernel that writes the partials
};
constexpr int kLnFinishThreads = 256;
constexpr int kLnFinishCols = 32, kLnFinishLanes = kLnFinishThreads * 4 / kLnFinishCols;
constexpr int kLnFinishLoads = (kLnMaxParts + kLnFinishLanes - 1) / kLnFinishLanes;
__global__ void __launch_bounds__(kLnFinishThreads) k_ln_finish(const LnFinishArgs a) {
  __shared__ float sm[kLnFinishLanes][kLnFinishCols + 1];
  const int x = (threadIdx.x % 8) * 4, y = threadIdx.x / 8;
  const int64_t width = 2 * a.cols, c0 = static_cast<int64_t>(blockIdx.x) * kLnFinishCols + x;
  if (a.dependent) griddep_wait();
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c0 + 4 <= width && width % 4 == 0) {
    float4 v[kLnFinishLoads];
#pragma unroll
    for (int i = 0; i < kLnFinishLoads; ++i) {
      const int p = y + i * kLnFinishLanes;
      v[i] = p < a.parts ? *reinterpret_cast<const float4*>(a.part + p * width + c0) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll
    for (int i = 0; i < kLnFinishLoads; ++i) { s.x += v[i].x; s.y += v[i].y; s.z += v[i].z; s.w += v[i].w; }
  } else {
    for (int p = y; p < a.parts; p += kLnFinishLanes) {
      const float* q = a.part + p * width + c0;
      if (c0 < width) s.x += q[0];
      if (c0 + 1 < width) s.y += q[1];
      if (c0 + 2 < width) s.z += q[2];
      if (c0 + 3 < width) s.w += q[3];
    }
  }
  sm[y][x] = s.x; sm[y][x + 1] = s.y; sm[y][x + 2] = s.z; sm[y][x + 3] = s.w;
  __syncthreads();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kLnFinishCols + threadIdx.x;
  if (threadIdx.x < kLnFinishCols && c < width) {
    float v = sm[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < kLnFinishLanes; ++i) v += sm[i][threadIdx.x];
    void* out = c < a.cols ? a.dw : a.db;
    const int64_t at = c < a.cols ? c : c - a.cols;
    if (!out) return;
    if (a.out_bf16) static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
    else static_cast<float*>(out)[at] = v;
  }
}

}  // namespace qlora
