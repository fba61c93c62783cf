// distill.cuh -- distillation from a teacher's top logits: the loss of a row
// of student logits against a short list of teacher logits, and its gradient.
//
// Row i: student logits z over the vocabulary, teacher logits t_j for listed
// entries id_j (a negative id marks an unused place), temperature tau:
//   p_j = softmax over the listed entries of t_j / tau
//   q_v = exp(z_v / tau - lse),  lse = log sum_v exp(z_v / tau)
//   loss = w tau^2 sum_j p_j (log p_j - log q_{id_j})
//   dloss/dz_v = w tau (q_v - sum_{j: id_j = v} p_j)
// (each listed place is a term of its own, so an id listed twice counts
// twice).  A row of weight 0, or with no listed entry left, has loss 0 and a
// gradient of zeros whatever its logits are.
//
// One sweep computes the running maximum m and the sum of exp((z - m) / tau)
// together, fp32 throughout: exponentials in base 2 of (z - m) log2(e) / tau.
// The maximum is subtracted before the scale is applied, so logits masked
// with the type's lowest value neither overflow nor, where a row holds
// nothing else, make anything but a uniform softmax.  The gradient is a second sweep over
// the row, which by then sits in L2 (rows in flight: a few per SM, tens of
// MB in 126 MB), so a call that returns both reads the logits from memory
// once.  Bound: HBM (one read, and one write of the gradient), closely
// followed by the special-function unit, 16 exponentials per clock per SM.
//
// A row belongs to a cluster of CTAs, each sweeping a slice of the
// vocabulary: one CTA when there are rows enough to fill the GPU, up to
// eight for few rows; the CTAs exchange (m, s) through distributed shared
// memory and combine them in rank order, so the result does not depend on
// scheduling.  Rows may start at any element: the vector part of a row runs
// from its first 16-byte boundary, the ragged ends element by element.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "ptx.cuh"

#define QLORA_DEV_INDEX 4

namespace qlora {

constexpr int kDiThreads = 512;
constexpr int kDiWarps = kDiThreads / 32;
constexpr int kDiMaxTop = 1024;
constexpr int kDiBatch = 4;            // 16-byte loads in flight per thread

struct DistillArgs {
  const void* z;
  int64_t ldz, rows, vocab;
  const void* ids;
  int ids64;
  const void* t;
  int t_bf16;
  int top;
  const float* weight;       // nullable: ones
  float tau;
  float scale2;              // log2(e) / tau
  float* loss;               // forward
  float* lse;                // forward: written (nullable)
  const float* lse_in;       // backward
  const float* grad;         // backward, nullable: ones
  void* dz;                  // gradient (forward: nullable)
  int64_t lddz;
  int slices;                // CTAs per row (forward: the cluster size)
  int* status;
};

__device__ __forceinline__ float di_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <typename T> struct DiVec;
template <> struct DiVec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
};
template <> struct DiVec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
};

// Running (maximum, sum of exp2((z - maximum) scale2)).  A sum whose maximum
// is still -inf uses the reference 0: every term exp2(-inf) is 0, and a NaN
// among the terms stays in the sum.
struct DiSum {
  float max, sum;
};
__device__ __forceinline__ float di_ref(float max) { return max == -INFINITY ? 0.0f : max; }
__device__ __forceinline__ DiSum di_merge(DiSum a, DiSum b, float scale2) {
  const float m = fmaxf(a.max, b.max);
  const float ref = di_ref(m);
  // an empty side adds its sum (0, or NaN) as it is
  const float ea = a.max == -INFINITY ? 1.0f : di_exp2((a.max - ref) * scale2);
  const float eb = b.max == -INFINITY ? 1.0f : di_exp2((b.max - ref) * scale2);
  return DiSum{m, a.sum * ea + b.sum * eb};
}

__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// max and sum over the block, the same in every thread; red holds one float
// per warp and is free again after the call's last barrier
__device__ __forceinline__ float di_block_max(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < kDiWarps; ++i) v = fmaxf(v, red[i]);
  return v;
}
__device__ __forceinline__ float di_block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < kDiWarps; ++i) v += red[i];
  return v;
}

// FWD: the loss and the normaliser, and the gradient when dz is given.
// Otherwise the gradient alone, from a given normaliser (no exchange between
// the CTAs of a row).
template <typename T, bool FWD>
__global__ void __launch_bounds__(kDiThreads, 2) k_distill(const DistillArgs a) {
  constexpr int N = DiVec<T>::N;
  __shared__ __align__(16) int s_id[kDiMaxTop];     // vocabulary index, or -1
  __shared__ float s_t[kDiMaxTop];                  // t / tau
  __shared__ float s_p[kDiMaxTop];                  // p
  __shared__ float s_z[kDiMaxTop];                  // the student's logit at the entry
  __shared__ float red[kDiWarps];
  __shared__ float2 red2[kDiWarps];
  __shared__ float2 s_mine;                         // this CTA's (max, sum) for its cluster

  const int64_t row = blockIdx.x / a.slices;
  const int slice = static_cast<int>(blockIdx.x % a.slices);   // rank in the cluster (forward)
  const int tid = threadIdx.x;
  const T* z = static_cast<const T*>(a.z) + row * a.ldz;
  T* dz = a.dz ? static_cast<T*>(a.dz) + row * a.lddz : nullptr;

  // the row's vector part: [head, head + N * chunks); this CTA's chunks [c0, c1)
  const uintptr_t za = reinterpret_cast<uintptr_t>(z), da = reinterpret_cast<uintptr_t>(dz);
  int64_t head = static_cast<int64_t>(((16 - (za & 15)) & 15) / sizeof(T));
  if (head > a.vocab || (dz && ((za ^ da) & 15))) head = a.vocab;   // no common 16-byte boundary: element by element
  const int64_t chunks = (a.vocab - head) / N;
  const int64_t per = (chunks + a.slices - 1) / a.slices;
  const int64_t c0 = min(chunks, slice * per), c1 = min(chunks, c0 + per);
  // the ragged ends: [0, head) and [tail, vocab), spread over the slices' threads
  const int64_t tail = head + chunks * N;
  const int64_t ragged = head + (a.vocab - tail);
  const int64_t rag0 = static_cast<int64_t>(slice) * kDiThreads + tid, rstep = static_cast<int64_t>(a.slices) * kDiThreads;
  auto ragged_at = [&](int64_t i) { return i < head ? i : tail + (i - head); };
  const uint4* zv = reinterpret_cast<const uint4*>(z + head);

  // ---------------------------------------------------------- the teacher
  float tmax = -INFINITY;
  bool bad = false;
  for (int j = tid; j < a.top; j += kDiThreads) {
    const int64_t e = row * a.top + j;
    const int64_t id = a.ids64 ? static_cast<const int64_t*>(a.ids)[e] : static_cast<const int32_t*>(a.ids)[e];
    const float t = (a.t_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.t)[e])
                              : static_cast<const float*>(a.t)[e]) / a.tau;
    const bool ok = id >= 0 && id < a.vocab;
    bad |= id >= a.vocab;
    s_id[j] = ok ? static_cast<int>(id) : -1;
    s_t[j] = ok ? t : -INFINITY;
    s_z[j] = ok ? static_cast<float>(z[id]) : 0.0f;
    if (ok) tmax = fmaxf(tmax, t);
  }
  if (tid < 4 && a.top + tid < kDiMaxTop) s_id[a.top + tid] = -1;   // the scan below reads whole groups of four
  if (bad && a.status) atomicOr(a.status, QLORA_DEV_INDEX);
  tmax = di_block_max(tmax, red);
  const float tref = tmax == -INFINITY ? 0.0f : tmax;
  float tsum = 0.0f;
  for (int j = tid; j < a.top; j += kDiThreads) {
    const float e = s_id[j] >= 0 ? expf(s_t[j] - tref) : 0.0f;
    s_p[j] = e;
    tsum += e;
  }
  tsum = di_block_sum(tsum, red);
  const bool empty = tsum == 0.0f;       // nothing listed (a NaN is not nothing)
  const float tinv = empty ? 0.0f : 1.0f / tsum;
  for (int j = tid; j < a.top; j += kDiThreads) s_p[j] *= tinv;
  const float weight = a.weight ? a.weight[row] : 1.0f;

  // ------------------------------------------------------ the normaliser
  // q = exp2((z - ref) scale2 - l2)
  float ref, l2;
  if (FWD) {
    DiSum acc{-INFINITY, 0.0f};
    auto take = [&](float m, auto&& each) {
      // `m`: the batch's maximum; `each(max)`: its sum of exponentials
      if (m > acc.max) {
        if (acc.max != -INFINITY) acc.sum *= di_exp2((acc.max - m) * a.scale2);
        acc.max = m;
      }
      acc.sum += each(di_ref(acc.max));
    };
    for (int64_t c = c0 + tid; c < c1; c += kDiBatch * kDiThreads) {
      uint4 v[kDiBatch];
#pragma unroll
      for (int b = 0; b < kDiBatch; ++b) {
        const int64_t at = c + b * kDiThreads;
        v[b] = zv[at < c1 ? at : c];     // past the end: the batch's first chunk again, not summed
      }
      float m = -INFINITY;
#pragma unroll
      for (int b = 0; b < kDiBatch; ++b) {
        float f[N];
        DiVec<T>::unpack(v[b], f);
#pragma unroll
        for (int e = 0; e < N; ++e) m = fmaxf(m, f[e]);
      }
      take(m, [&](float top) {
        float s = 0.0f;
#pragma unroll
        for (int b = 0; b < kDiBatch; ++b) {
          if (c + b * kDiThreads < c1) {
            float f[N];
            DiVec<T>::unpack(v[b], f);
#pragma unroll
            for (int e = 0; e < N; ++e) s += di_exp2((f[e] - top) * a.scale2);
          }
        }
        return s;
      });
    }
    for (int64_t i = rag0; i < ragged; i += rstep) {
      const float f = static_cast<float>(z[ragged_at(i)]);
      take(fmaxf(f, -INFINITY), [&](float top) { return di_exp2((f - top) * a.scale2); });
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const DiSum other{__shfl_xor_sync(0xFFFFFFFFu, acc.max, o), __shfl_xor_sync(0xFFFFFFFFu, acc.sum, o)};
      // the lower lane's part first in both lanes, so that both hold the same sum
      acc = (tid & o) ? di_merge(other, acc, a.scale2) : di_merge(acc, other, a.scale2);
    }
    if ((tid & 31) == 0) red2[tid >> 5] = make_float2(acc.max, acc.sum);
    __syncthreads();
    acc = DiSum{red2[0].x, red2[0].y};
#pragma unroll
    for (int i = 1; i < kDiWarps; ++i) acc = di_merge(acc, DiSum{red2[i].x, red2[i].y}, a.scale2);
    if (a.slices > 1) {
      if (tid == 0) s_mine = make_float2(acc.max, acc.sum);
      cluster_sync();
      const uint32_t mine = smem_u32(&s_mine);
      acc = DiSum{-INFINITY, 0.0f};
      for (int r = 0; r < a.slices; ++r) {
        const float2 o = ld_cluster_f2(mapa_shared(mine, static_cast<uint32_t>(r)));
        acc = di_merge(acc, DiSum{o.x, o.y}, a.scale2);
      }
    }
    ref = di_ref(acc.max);
    l2 = log2f(acc.sum);

    if (slice == 0) {
      const float zlog = logf(acc.sum);
      float kl = 0.0f;
      const float tlog = logf(tsum);
      for (int j = tid; j < a.top; j += kDiThreads) {
        const float p = s_p[j];
        // p = 0 contributes nothing even where q = 0; a NaN p stays
        if (!(p == 0.0f)) kl += p * (((s_t[j] - tref) - tlog) - ((s_z[j] - ref) / a.tau - zlog));
      }
      kl = di_block_sum(kl, red);
      if (tid == 0) {
        const float f = weight * (a.tau * a.tau);
        a.loss[row] = (empty || weight == 0.0f) ? 0.0f : f * kl;
        if (a.lse) a.lse[row] = ref / a.tau + zlog;
      }
    }
  } else {
    ref = a.lse_in[row] * a.tau;
    l2 = 0.0f;
  }

  // --------------------------------------------------------- the gradient
  if (dz) {
    float f = weight * a.tau;
    if (!FWD && a.grad) f *= a.grad[row];
    const bool none = empty || weight == 0.0f || f == 0.0f;
    uint4* dv = reinterpret_cast<uint4*>(dz + head);
    __syncthreads();                     // s_p, and the entries' logits before dz may overwrite z
    if (none) {
      for (int64_t c = c0 + tid; c < c1; c += kDiThreads) dv[c] = make_uint4(0, 0, 0, 0);
      for (int64_t i = rag0; i < ragged; i += rstep) DiVec<T>::store(dz + ragged_at(i), 0.0f);
    } else {
      for (int64_t c = c0 + tid; c < c1; c += kDiBatch * kDiThreads) {
        uint4 v[kDiBatch];
#pragma unroll
        for (int b = 0; b < kDiBatch; ++b) {
          const int64_t at = c + b * kDiThreads;
          if (at < c1) v[b] = zv[at];
        }
#pragma unroll
        for (int b = 0; b < kDiBatch; ++b) {
          const int64_t at = c + b * kDiThreads;
          if (at < c1) {
            float g[N];
            DiVec<T>::unpack(v[b], g);
#pragma unroll
            for (int e = 0; e < N; ++e) g[e] = f * di_exp2(fmaf(g[e] - ref, a.scale2, -l2));
            dv[at] = DiVec<T>::pack(g);
          }
        }
      }
      for (int64_t i = rag0; i < ragged; i += rstep) {
        const int64_t at = ragged_at(i);
        DiVec<T>::store(dz + at, f * di_exp2(fmaf(static_cast<float>(z[at]) - ref, a.scale2, -l2)));
      }
      __syncthreads();                   // the sweep's writes come before the listed entries'
      for (int j = tid; j < a.top; j += kDiThreads) {
        const int id = s_id[j];
        // the CTA that swept the entry's place writes it
        bool mine = false;
        if (id >= 0) {
          if (id >= head && id < tail) {
            const int64_t c = (id - head) / N;
            mine = c >= c0 && c < c1;
          } else {
            const int64_t i = id < head ? id : head + (id - tail);
            mine = (i / kDiThreads) % a.slices == slice;
          }
        }
        if (mine) {
          float p = 0.0f;                // every place that lists this id, in list order
          for (int k = 0; k < a.top; k += 4) {
            const int4 o = *reinterpret_cast<const int4*>(&s_id[k]);
            if (o.x == id) p += s_p[k];
            if (o.y == id) p += s_p[k + 1];
            if (o.z == id) p += s_p[k + 2];
            if (o.w == id) p += s_p[k + 3];
          }
          DiVec<T>::store(dz + id, f * (di_exp2(fmaf(s_z[j] - ref, a.scale2, -l2)) - p));
        }
      }
    }
  }
  // a CTA's shared memory stays until every CTA of the cluster has read it
  if (FWD && a.slices > 1) cluster_sync();
}

}  // namespace qlora
