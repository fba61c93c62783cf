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
// The maximum is subtracted before the scale is applied, the student's and the
// teacher's alike, so logits masked with the type's lowest value neither
// overflow nor, where a row or a list holds nothing else, make anything but a
// uniform softmax.  The gradient is a second sweep over the row, which by then
// sits in L2 (rows in flight: a few per SM, tens of MB in 126 MB), so a call
// that returns both reads the logits from memory once.  Bound: HBM (one read,
// and one write of the gradient), closely followed by the special-function
// unit, 16 exponentials per clock per SM.
//
// A row belongs to a cluster of CTAs, each sweeping a slice of the
// vocabulary: one CTA when there are rows enough to fill the GPU, up to
// eight for few rows; the CTAs exchange (m, s) through distributed shared
// memory and combine them in rank order, so the result does not depend on
// scheduling.  In a CTA eight warps sweep while a ninth works through the
// teacher's list, whose chain of dependent loads would otherwise be most of
// a short row's time.  Rows may start at any element: the vector part of a row runs
// from its first 16-byte boundary, the ragged ends element by element.
//
// Measured on the device (calls in a graph, each on inputs that are not in L2)
// against a copy's rate of 6.57 TB/s: loss and gradient in one call 4096 x
// 32768 bf16 108 us (5.0 TB/s; the copy would take 82), fp32 207 us (163),
// 1024 x 131072 bf16 124 us (82); loss alone 4096 x 32768 bf16 56 us (41),
// fp32 88 us (82), 6 x 131072 5.1 us; gradient alone 4096 x 32768 bf16 91 us
// (82), fp32 177 us (163), 777 x 50021 bf16 34.5 us (24), fp32 61 us (47).
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "ptx.cuh"
#include "f32x2.cuh"

#define QLORA_DEV_INDEX 4

namespace qlora {

constexpr int kDiWarps = 8;                      // sweep the vocabulary
constexpr int kDiSweep = kDiWarps * 32;
constexpr int kDiThreads = kDiSweep + 32;        // and one warp for the teacher's list
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

// A 16-byte chunk of logits: N values as N / 2 pairs of fp32 (packed
// arithmetic: half the instructions, the same roundings).
__device__ __forceinline__ uint32_t di_max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <typename T> struct DiVec;
template <> struct DiVec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float max(const uint4& v) {
    // a NaN loses against a number; the sum brings it back
    uint32_t m = di_max_bf16x2(di_max_bf16x2(v.x, v.y), di_max_bf16x2(v.z, v.w));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  }
  static __device__ __forceinline__ void pairs(const uint4& v, f32x2 (&f)[4]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pair2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint4 pack(const f32x2 (&f)[4]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpair2(f[i]);
      u[i] = pack_bf16x2(x.x, x.y);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
};
template <> struct DiVec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float max(const uint4& v) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
  static __device__ __forceinline__ void pairs(const uint4& v, f32x2 (&f)[2]) {
    f[0] = pair2(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = pair2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  static __device__ __forceinline__ uint4 pack(const f32x2 (&f)[2]) {
    const float2 x = unpair2(f[0]), y = unpair2(f[1]);
    return make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(y.x), __float_as_uint(y.y));
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

__device__ __forceinline__ float di_warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
__device__ __forceinline__ float di_warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// FWD: the loss and the normaliser, and the gradient when dz is given.
// Otherwise the gradient alone, from a given normaliser (no exchange between
// the CTAs of a row).
template <typename T, bool FWD>
__global__ void __launch_bounds__(kDiThreads, 4) k_distill(const DistillArgs a) {
  constexpr int N = DiVec<T>::N;
  __shared__ __align__(16) int s_id[kDiMaxTop];     // vocabulary index, or -1
  __shared__ float s_t[kDiMaxTop];                  // t, then t - the largest
  __shared__ float s_p[kDiMaxTop];                  // p
  __shared__ float s_z[kDiMaxTop];                  // the student's logit at the entry
  __shared__ float2 red[kDiWarps];                  // the warps' (max, sum)
  __shared__ float2 s_mine;                         // this CTA's (max, sum) for its cluster
  __shared__ int s_empty;                           // no listed entry has weight

  const int64_t row = blockIdx.x / a.slices;
  const int slice = static_cast<int>(blockIdx.x % a.slices);   // rank in the cluster (forward)
  const int tid = threadIdx.x, lane = tid & 31;
  const bool teacher = tid >= kDiSweep;
  const T* z = static_cast<const T*>(a.z) + row * a.ldz;
  T* dz = a.dz ? static_cast<T*>(a.dz) + row * a.lddz : nullptr;

  // the row's vector part: [head, head + N * chunks); this CTA's chunks [c0, c1)
  const uintptr_t za = reinterpret_cast<uintptr_t>(z), da = reinterpret_cast<uintptr_t>(dz);
  int64_t head = static_cast<int64_t>(((16 - (za & 15)) & 15) / sizeof(T));
  if (head > a.vocab || (dz && ((za ^ da) & 15))) head = a.vocab;   // no common 16-byte boundary: element by element
  const int chunks = static_cast<int>((a.vocab - head) / N);
  const int per = (chunks + a.slices - 1) / a.slices;
  const int c0 = min(chunks, slice * per), c1 = min(chunks, c0 + per);
  // the ragged ends: [0, head) and [tail, vocab), spread over the slices' threads
  const int64_t tail = head + static_cast<int64_t>(chunks) * N;
  const int64_t ragged = head + (a.vocab - tail);
  const int64_t rag0 = static_cast<int64_t>(slice) * kDiSweep + tid, rstep = static_cast<int64_t>(a.slices) * kDiSweep;
  auto ragged_at = [&](int64_t i) { return i < head ? i : tail + (i - head); };
  const uint4* zv = reinterpret_cast<const uint4*>(z + head);
  const f32x2 scale = pair2(a.scale2, a.scale2);

  DiSum acc{-INFINITY, 0.0f};
  float tsum = 0.0f;
  if (teacher) {
    // -------------------------------------------------------- the teacher
    float tmax = -INFINITY;
    bool bad = false;
    for (int j = lane; j < a.top; j += 32) {
      const int64_t e = row * a.top + j;
      const int64_t id = a.ids64 ? static_cast<const int64_t*>(a.ids)[e] : static_cast<const int32_t*>(a.ids)[e];
      const float t = a.t_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.t)[e])
                               : static_cast<const float*>(a.t)[e];
      const bool ok = id >= 0 && id < a.vocab;
      bad |= id >= a.vocab;
      s_id[j] = ok ? static_cast<int>(id) : -1;
      s_t[j] = ok ? t : -INFINITY;
      s_z[j] = ok ? static_cast<float>(z[id]) : 0.0f;
      if (ok) tmax = fmaxf(tmax, t);
    }
    if (lane < 4 && a.top + lane < kDiMaxTop) s_id[a.top + lane] = -1;   // the scan below reads whole groups of four
    if (bad && a.status) atomicOr(a.status, QLORA_DEV_INDEX);
    tmax = di_warp_max(tmax);
    const float tref = tmax == -INFINITY ? 0.0f : tmax;
    for (int j = lane; j < a.top; j += 32) {
      const float d = s_t[j] - tref;                 // (t / tau first would overflow for the type's lowest and highest values)
      const float e = s_id[j] >= 0 ? expf(d / a.tau) : 0.0f;
      s_t[j] = d;
      s_p[j] = e;
      tsum += e;
    }
    tsum = di_warp_sum(tsum);
    const float tinv = tsum == 0.0f ? 0.0f : 1.0f / tsum;              // (a NaN is not nothing)
    for (int j = lane; j < a.top; j += 32) s_p[j] *= tinv;
    if (lane == 0) s_empty = tsum == 0.0f ? 1 : 0;
  } else if (FWD) {
    // -------------------------------------------------------- the sweep
    // `m`: a batch's maximum; `each(max)`: its sum of exponentials
    auto take = [&](float m, auto&& each) {
      if (m > acc.max) {
        if (acc.max != -INFINITY) acc.sum *= di_exp2((acc.max - m) * a.scale2);
        acc.max = m;
      }
      acc.sum += each(di_ref(acc.max));
    };
    auto chunk_sum = [&](const uint4& v, f32x2 neg, f32x2& s2) {
      f32x2 f[N / 2];
      DiVec<T>::pairs(v, f);
#pragma unroll
      for (int e = 0; e < N / 2; ++e) {
        const float2 x = unpair2(mul2(add2(f[e], neg), scale));
        s2 = add2(s2, pair2(di_exp2(x.x), di_exp2(x.y)));
      }
    };
    int c = c0 + tid;
    for (; c + (kDiBatch - 1) * kDiSweep < c1; c += kDiBatch * kDiSweep) {
      uint4 v[kDiBatch];
#pragma unroll
      for (int b = 0; b < kDiBatch; ++b) v[b] = zv[c + b * kDiSweep];
      float m = DiVec<T>::max(v[0]);
#pragma unroll
      for (int b = 1; b < kDiBatch; ++b) m = fmaxf(m, DiVec<T>::max(v[b]));
      take(m, [&](float top) {
        f32x2 s2 = 0;
        const f32x2 neg = pair2(-top, -top);
#pragma unroll
        for (int b = 0; b < kDiBatch; ++b) chunk_sum(v[b], neg, s2);
        const float2 s = unpair2(s2);
        return s.x + s.y;
      });
    }
    for (; c < c1; c += kDiSweep) {
      const uint4 v = zv[c];
      take(fmaxf(DiVec<T>::max(v), -INFINITY), [&](float top) {
        f32x2 s2 = 0;
        chunk_sum(v, pair2(-top, -top), s2);
        const float2 s = unpair2(s2);
        return s.x + s.y;
      });
    }
    for (int64_t i = rag0; i < ragged; i += rstep) {
      const float f = static_cast<float>(z[ragged_at(i)]);
      take(fmaxf(f, -INFINITY), [&](float top) { return di_exp2((f - top) * a.scale2); });
    }
    // the warp's sum: the largest maximum, then every lane's part against it
    const float m = di_warp_max(acc.max);
    const float part = acc.max == -INFINITY ? acc.sum : acc.sum * di_exp2((acc.max - di_ref(m)) * a.scale2);
    const float sum = di_warp_sum(part);
    if (lane == 0) red[tid >> 5] = make_float2(m, sum);
  }

  const float weight = a.weight ? a.weight[row] : 1.0f;
  // q = exp2((z - ref) scale2 - l2)
  float ref, l2;
  if (FWD) {
    __syncthreads();
    acc = DiSum{red[0].x, red[0].y};
#pragma unroll
    for (int i = 1; i < kDiWarps; ++i) acc.max = fmaxf(acc.max, red[i].x);
    {
      const float2 mine = red[lane % kDiWarps];
      float part = lane < kDiWarps ? mine.y : 0.0f;
      if (lane < kDiWarps && mine.x != -INFINITY) part *= di_exp2((mine.x - di_ref(acc.max)) * a.scale2);
      acc.sum = di_warp_sum(part);
    }
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

    if (teacher && slice == 0) {
      const float zlog = logf(acc.sum), tlog = logf(tsum);
      float kl = 0.0f;
      for (int j = lane; j < a.top; j += 32) {
        const float p = s_p[j];
        // p = 0 contributes nothing even where q = 0; a NaN p stays.  The sum is
        // of tau / 2 times p (log p - log q): divided by tau, or added up whole,
        // student logits of the type's lowest value overflow where the loss does not
        if (!(p == 0.0f)) kl += 0.5f * p * ((s_t[j] - (s_z[j] - ref)) + a.tau * (zlog - tlog));
      }
      kl = di_warp_sum(kl);
      if (lane == 0) {
        const float f = weight * a.tau * 2.0f;
        a.loss[row] = (s_empty || weight == 0.0f) ? 0.0f : f * kl;
        if (a.lse) a.lse[row] = ref / a.tau + zlog;
      }
    }
  } else {
    ref = a.lse_in[row] * a.tau;
    l2 = 0.0f;
    if (a.dz == a.z) __syncthreads();    // the entries' logits are taken before dz overwrites them
  }

  // --------------------------------------------------------- the gradient
  if (dz) {
    float f = weight * a.tau;
    if (!FWD && a.grad) f *= a.grad[row];
    uint4* dv = reinterpret_cast<uint4*>(dz + head);
    auto zeros = [&]() {
      for (int c = c0 + tid; c < c1; c += kDiSweep) dv[c] = make_uint4(0, 0, 0, 0);
      for (int64_t i = rag0; i < ragged; i += rstep) DiVec<T>::store(dz + ragged_at(i), 0.0f);
    };
    const bool none = weight == 0.0f || f == 0.0f || (FWD && s_empty);
    if (none) {
      if (!teacher) zeros();
    } else {
      if (!teacher) {
        const f32x2 neg = pair2(-ref, -ref), nl2 = pair2(-l2, -l2), ff = pair2(f, f);
        for (int c = c0 + tid; c < c1; c += kDiBatch * kDiSweep) {
          uint4 v[kDiBatch];
#pragma unroll
          for (int b = 0; b < kDiBatch; ++b)
            if (c + b * kDiSweep < c1) v[b] = zv[c + b * kDiSweep];
#pragma unroll
          for (int b = 0; b < kDiBatch; ++b) {
            if (c + b * kDiSweep < c1) {
              f32x2 g[N / 2];
              DiVec<T>::pairs(v[b], g);
#pragma unroll
              for (int e = 0; e < N / 2; ++e) {
                const float2 x = unpair2(fma2(add2(g[e], neg), scale, nl2));
                g[e] = mul2(pair2(di_exp2(x.x), di_exp2(x.y)), ff);
              }
              __stcs(dv + c + b * kDiSweep, DiVec<T>::pack(g));   // (leaves L2 to the logits that are read twice)
            }
          }
        }
        for (int64_t i = rag0; i < ragged; i += rstep) {
          const int64_t at = ragged_at(i);
          DiVec<T>::store(dz + at, f * di_exp2(fmaf(static_cast<float>(z[at]) - ref, a.scale2, -l2)));
        }
      }
      __syncthreads();                   // the sweep's writes come before the listed entries'
      if (!FWD && s_empty) {             // (the backward learns it from the teacher's warp only here)
        if (!teacher) zeros();
        return;
      }
      for (int j = tid; j < a.top; j += kDiThreads) {
        const int id = s_id[j];
        // the CTA that swept the entry's place writes it
        bool mine = false;
        if (id >= 0) {
          if (id >= head && id < tail) {
            const int c = static_cast<int>((id - head) / N);
            mine = c >= c0 && c < c1;
          } else {
            const int64_t i = id < head ? id : head + (id - tail);
            mine = (i / kDiSweep) % a.slices == slice;
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
