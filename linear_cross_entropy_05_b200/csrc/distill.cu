// Distillation from a teacher's top logits: the two small kernels around the
// logit pass (fwd.cu, PICK) and the stripe backward (bwd_stripe.cu, PICK).
//
// For a token with teacher entries (id_k, t_k), k < K, and a temperature T:
//   p_k    = exp(t_k / T) / sum_j exp(t_j / T)   over the row's live entries
//   lse    = log sum_v exp(z_v / T),   z_v = E_i . C_v
//   loss   = T^2 sum_k p_k (log p_k - z_{id_k} / T + lse)
//   dloss / dz_v = T (exp(z_v / T - lse) - sum_{k: id_k = v} p_k)
// An entry is live unless its id is ignore_index or its logit -inf.  The
// teacher's side costs N K (8 + 4) bytes, nothing beside the logit pass; it
// is kept in double; the weights are rounded to float once.
//
// distill_targets  one block per row: p, sum p log p, and the entries sorted
//                  by id, so that the logit and gradient tiles, which walk
//                  the vocabulary in order, meet them one after another.  For
//                  the backward also the copy of E that it reads: 4 N D bytes
//                  beside products of 6 N V D.
// distill_finalize merges the splits' (max, sum, weighted logits) into lse
//                  and loss; 32 rows x 16 split lanes per block, so the
//                  [split][row] partials are read in whole lines.  The block
//                  that finishes last adds up the mean, in a fixed order.
// distill_parts    adds up dE from the parts that few tokens' stripes leave
//                  (deterministic mode), in the order of the parts.
// distill_mark     NaN to the gradients of a backward in which a bounded wait
//                  gave up: tiles that were not reached hold what was there
//                  before (distill_parts does it too, which saves few tokens'
//                  calls a launch).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace cce {

namespace {

// Reduction of one double per thread over the block (whole warps; buf holds
// one per warp), in a fixed order; every thread gets the result.
template <bool MAX>
__device__ __forceinline__ double block_reduce(double v, double* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmax(v, u) : v + u;
  }
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  __syncthreads();  // buf may still be read from an earlier reduction
  if ((tid & 31) == 0) buf[tid >> 5] = v;
  __syncthreads();
  double r = buf[0];
  for (int i = 1; i < (int)(blockDim.x * blockDim.y >> 5); ++i) r = MAX ? fmax(r, buf[i]) : r + buf[i];
  return r;
}

}  // namespace

constexpr int FIN_PARTS = 16;

// n_sort: K rounded up to a power of two (the sort network's size)
__global__ void __launch_bounds__(256) distill_targets_kernel(const TargetArgs a, int n_sort) {
  extern __shared__ double smem_d[];
  double* sx = smem_d;                                                     // [K] t / T, -inf if not live
  unsigned long long* key = reinterpret_cast<unsigned long long*>(sx + a.K);  // [n_sort] id << 32 | position
  double* buf = reinterpret_cast<double*>(key + n_sort);                   // [8]
  const int row = blockIdx.x;
  const size_t base = (size_t)row * a.K;
  const int tid = threadIdx.x;

  int bad = 0;
  double top = -INFINITY;
  for (int k = tid; k < n_sort; k += blockDim.x) {
    unsigned id = INT_MAX;
    if (k < a.K) {
      const long long raw = a.ids[base + k];
      const float t = a.teacher_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.teacher)[base + k])
                                     : reinterpret_cast<const float*>(a.teacher)[base + k];
      double x = -INFINITY;
      if (raw != a.ignore_index && t != -INFINITY) {
        if (raw < 0 || raw >= a.V || !(t < INFINITY)) {
          bad = 1;  // an id outside the vocabulary, a NaN or +inf logit
        } else {
          id = (unsigned)raw;
          x = (double)t * a.inv_temperature;
        }
      }
      sx[k] = x;
      top = fmax(top, x);
    }
    key[k] = ((unsigned long long)id << 32) | (unsigned)k;
  }
  bad = __syncthreads_or(bad);
  top = block_reduce<true>(top, buf);
  const int kind = bad ? ROW_BAD : (top == -INFINITY ? ROW_EMPTY : ROW_LIVE);
  if (tid == 0) {
    a.row_kind[row] = kind;
    if (bad) atomicOr(a.status + ST_FLAGS, SF_BAD_LABEL);
    if (kind != ROW_LIVE) a.stats[row] = make_double2(0.0, 0.0);
  }
  if (a.E_live) {
    const uint4* src = reinterpret_cast<const uint4*>(a.E) + (size_t)row * (a.D / 8);
    uint4* dst = reinterpret_cast<uint4*>(a.E_live) + (size_t)row * (a.D / 8);
#pragma unroll 4
    for (int i = tid; i < a.D / 8; i += blockDim.x) dst[i] = kind == ROW_LIVE ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
  }
  if (kind != ROW_LIVE) {
    for (int k = tid; k < a.K; k += blockDim.x) {
      a.tgt_id[base + k] = INT_MAX;
      a.tgt_w[base + k] = 0.f;
    }
    return;
  }

  double s = 0.0, sxw = 0.0;  // sum of exp(x - top) and of exp(x - top) (x - top)
  for (int k = tid; k < a.K; k += blockDim.x) {
    const double d = sx[k] - top;
    const double e = exp(d);
    s += e;
    if (e > 0.0) sxw += e * d;
  }
  s = block_reduce<false>(s, buf);
  sxw = block_reduce<false>(sxw, buf);

  // bitonic sort by id (then position)
  for (int size = 2; size <= n_sort; size <<= 1) {
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      __syncthreads();
      for (int i = tid; i < (n_sort >> 1); i += blockDim.x) {
        const int lo = 2 * i - (i & (stride - 1));
        const int hi = lo + stride;
        const bool up = (lo & size) == 0;
        const unsigned long long ka = key[lo], kb = key[hi];
        if ((ka > kb) == up) {
          key[lo] = kb;
          key[hi] = ka;
        }
      }
    }
  }
  __syncthreads();
  const double inv = 1.0 / s;
  double sum_w = 0.0;
  for (int k = tid; k < a.K; k += blockDim.x) {
    const unsigned long long kk = key[k];
    const double x = sx[(unsigned)kk & 0xffffu];
    a.tgt_id[base + k] = (int)(kk >> 32);
    const float w = x == -INFINITY ? 0.f : (float)(exp(x - top) * inv);
    a.tgt_w[base + k] = w;
    sum_w += (double)w;
  }
  sum_w = block_reduce<false>(sum_w, buf);
  if (tid == 0) a.stats[row] = make_double2(sxw / s - log(s), sum_w);
}

__global__ void __launch_bounds__(32 * FIN_PARTS) distill_finalize_kernel(const DistillFinArgs a) {
  __shared__ float sm[FIN_PARTS][32];
  __shared__ double ss[FIN_PARTS][32];
  __shared__ double sd[FIN_PARTS][32];
  __shared__ int s_last;
  const int lane = threadIdx.x, part = threadIdx.y;
  const int row = blockIdx.x * 32 + lane;
  // (sums relative to 2^ms(M): see lse_fold_columns)
  auto ms = [&](float m) { return __fmul_rn(m, a.scale2); };
  float M = -INFINITY;
  double s = 0.0, dot = 0.0;
  if (row < a.N) {
    for (int r = part; r < a.n_part; r += FIN_PARTS) {
      const float2 p = a.partial[(size_t)r * a.N + row];
      dot += a.dot[(size_t)r * a.N + row];
      const float m = fmaxf(M, p.x);
      if (m != -INFINITY) s = s * (double)exp2f(ms(M) - ms(m)) + (double)p.y * (double)exp2f(ms(p.x) - ms(m));
      M = m;
    }
  }
  sm[part][lane] = M;
  ss[part][lane] = s;
  sd[part][lane] = dot;
  __syncthreads();
  if (part == 0 && row < a.N) {
    for (int q = 1; q < FIN_PARTS; ++q) M = fmaxf(M, sm[q][lane]);
    s = 0.0;
    dot = 0.0;
    for (int q = 0; q < FIN_PARTS; ++q) {
      if (sm[q][lane] != -INFINITY) s += ss[q][lane] * (double)exp2f(ms(sm[q][lane]) - ms(M));
      dot += sd[q][lane];
    }
    const double T = (double)a.temperature;
    // M / T, and what the rounding of ms left of the shift
    constexpr double kLn2 = 0.69314718055994530942;
    const double L = (double)M / T + kLn2 * ((double)ms(M) - (double)M * (double)a.scale2) + log(s);
    const int kind = a.row_kind[row];
    double loss = 0.0;
    // (lse is weighted by the rounded weights too: their rounding then meets
    // log-probabilities and not logits)
    const double2 st = a.stats[row];
    if (kind == ROW_LIVE) loss = T * T * (st.x - dot / T + st.y * L);
    float lse = (float)L, out = (float)loss;
    if (kind == ROW_BAD) out = __int_as_float(0x7fc00000);
    // a bounded wait gave up: some partials may be an earlier call's
    if (a.status[ST_FLAGS] & SF_TIMEOUT) lse = out = __int_as_float(0x7fc00000);
    a.lse[row] = lse;
    a.loss[row] = out;
  }
  if (!a.mean) return;

  // the mean, by the last block to get here
  __threadfence();
  __syncthreads();
  const int tid = part * 32 + lane;
  if (tid == 0) s_last = atomicAdd(a.status + ST_NEXT_TILE, 1ull) == gridDim.x - 1ull;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  double sum = 0.0, n = 0.0;
  for (int i = tid; i < a.N; i += 32 * FIN_PARTS) {
    if (a.row_kind[i] != ROW_EMPTY) {
      sum += (double)__ldcg(a.loss + i);
      n += 1.0;
    }
  }
  double* buf = &sd[0][0];
  sum = block_reduce<false>(sum, buf);
  n = block_reduce<false>(n, buf);
  if (tid == 0) {
    *a.mean = (float)(sum / n);
    *a.inv_count = (float)(1.0 / n);
  }
}

// If a wait gave up: NaN to both gradients (a pattern of both types).
__device__ __forceinline__ bool mark_if_failed(const GradOuts& o) {
  if (!(__ldcg(o.status + ST_FLAGS) & SF_TIMEOUT)) return false;
  const uint4 nan4 = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
  const size_t stride = (size_t)gridDim.x * blockDim.x, i0 = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  for (size_t i = i0; i < o.dE_bytes / 16; i += stride) reinterpret_cast<uint4*>(o.dE)[i] = nan4;
  for (size_t i = i0; i < o.dC_bytes / 16; i += stride) reinterpret_cast<uint4*>(o.dC)[i] = nan4;
  return true;
}

__global__ void __launch_bounds__(256) distill_mark_kernel(const GradOuts o) { mark_if_failed(o); }

cudaError_t launch_distill_mark(const GradOuts& o, int sms, cudaStream_t stream) {
  distill_mark_kernel<<<sms, 256, 0, stream>>>(o);
  return cudaGetLastError();
}

// dE = the sum of the parts (plus dE itself with `accumulate`), in their order.
// part4: float4s from one part to the next.
__global__ void __launch_bounds__(256) distill_parts_kernel(const float4* __restrict__ parts, int n_parts, size_t part4,
                                                            const GradOuts o, size_t n4, int bf16, int accumulate) {
  if (mark_if_failed(o)) return;
  void* out = o.dE;
  const size_t stride = (size_t)gridDim.x * blockDim.x;
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n4; i += stride) {
    float4 v = __ldg(parts + i);
#pragma unroll 8
    for (int p = 1; p < n_parts; ++p) {
      const float4 x = __ldg(parts + p * part4 + i);
      v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
    }
    if (!bf16) {
      float4* dst = reinterpret_cast<float4*>(out) + i;
      if (accumulate) v = make_float4(v.x + dst->x, v.y + dst->y, v.z + dst->z, v.w + dst->w);
      *dst = v;
    } else {
      uint2* dst = reinterpret_cast<uint2*>(out) + i;
      if (accumulate) {
        const uint2 old = *dst;
        const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&old.x));
        const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&old.y));
        v = make_float4(v.x + a.x, v.y + a.y, v.z + b.x, v.w + b.y);
      }
      const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
      *dst = make_uint2(*reinterpret_cast<const unsigned*>(&lo), *reinterpret_cast<const unsigned*>(&hi));
    }
  }
}

cudaError_t launch_distill_parts(const float* parts, int n_parts, size_t part_floats, const GradOuts& o, size_t n,
                                 bool bf16, bool accumulate, int sms, cudaStream_t stream) {
  const size_t blocks = (n / 4 + 255) / 256;
  distill_parts_kernel<<<(unsigned)(blocks < (size_t)sms * 8 ? blocks : (size_t)sms * 8), 256, 0, stream>>>(
      reinterpret_cast<const float4*>(parts), n_parts, part_floats / 4, o, n / 4, bf16 ? 1 : 0, accumulate ? 1 : 0);
  return cudaGetLastError();
}

cudaError_t launch_distill_targets(const TargetArgs& a, cudaStream_t stream) {
  int n_sort = 32;
  while (n_sort < a.K) n_sort <<= 1;
  const int least = a.E_live ? 128 : 32;
  const int threads = n_sort / 2 < least ? least : (n_sort / 2 > 256 ? 256 : n_sort / 2);
  const size_t smem = (size_t)a.K * 8 + (size_t)n_sort * 8 + 64;
  distill_targets_kernel<<<a.N, threads, smem, stream>>>(a, n_sort);
  return cudaGetLastError();
}

cudaError_t launch_distill_finalize(const DistillFinArgs& a, cudaStream_t stream) {
  distill_finalize_kernel<<<(a.N + 31) / 32, dim3(32, FIN_PARTS), 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace cce
