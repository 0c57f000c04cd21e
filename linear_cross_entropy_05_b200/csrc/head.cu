// The head's logits of up to 512 tokens at a time, for choosing among them:
// the k largest (top_logits) or one drawn token per row (sample).
//
//   z_iv = E_i . C_v;  x_iv = z_iv / T_i;
//   log-probability of v: x_iv - log sum_w exp(x_iw)
//
// head_logits   C is read once per 512 tokens, which is what bounds the call
//               below about 256 tokens (2 V D bytes); above, the products.
//               (256 tokens at a time: 262 us for 256 tokens x 2304 x 256000,
//               the time of 1.18 GB of C and 0.26 GB of logits; 512 at a time
//               the products' time covers them.)
//               The vocabulary is the M side of the tensor-core tiles and the
//               tokens are the N side, so a batch of 16 multiplies 16 columns
//               and not 256.  CTA pairs (cta_group::2): 256 vocabulary rows x
//               up to 256 tokens in TMEM, double buffered; 128 rows of C and
//               half of the tokens' rows of E per CTA and stage.  The logits
//               go to the workspace in fp32, with the largest of each group
//               of 32 vocabulary entries and, for each of a few hundred bins
//               of groups (the ones that one epilogue warp meets), the largest
//               and sum exp(x - largest).
// head_select   one block per token.  Almost no row needs its logits again:
//               the k-th largest bin maximum is no larger than the k-th
//               largest logit, so only the bins, and of these the groups, that
//               reach it are read, and their few candidates are sorted in
//               shared memory; a draw without filters walks the bins' sums,
//               the groups' of one share, and reads one group.  Rows that
//               this does not settle (more than kCap candidates: a wide
//               nucleus, a row full of ties) take exact passes over the row.
//
// A logit is one accumulator's sum over all of D, whose truncated additions
// leave the largest 8e-6 short (relatively) at D = 8192.  The distillation
// forward hands its accumulator over every 1024 of D; here a thread would have
// to hold 64 sums beside the 96 registers that 576 threads leave it, and parts
// kept in tensor memory for few tokens only would make a token's logits depend
// on how many others are in the call.
//
// A drawn token is decided by comparing u with a quotient of sums of up to V
// exponentials; these sums are formed in double (a group's 32 in 2^-51
// fixed point, so that no order of summation shows), because float sums would
// move the borders between tokens by more than a rare token's own width.  Rows
// whose token does not hang on them (row_exact) take float exponentials
// (head_logits, 193 tokens x 896 x 151936: 92 us; in double 142 us).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "common.cuh"
#include "ptx.cuh"

namespace cce {

namespace {

constexpr int HL_EPI_WARPS = 16;                 // four per TMEM lane group, taking 32-token chunks in turn
constexpr int HL_THREADS = 64 + 32 * HL_EPI_WARPS;
constexpr int HL_CHUNKS = 8 / (HL_EPI_WARPS / 4); // 32-token chunks of a warp: of at most eight in 256 tokens
constexpr int HL_MAX_STAGES = 12;
constexpr double kLog2e = 1.4426950408889634074;

// Order-preserving map of floats that are not NaN to unsigned.
__device__ __forceinline__ unsigned order_key(float x) {
  const unsigned b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(unsigned k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
constexpr unsigned kKeyPosInf = 0xff800000u;  // order_key(+inf)
constexpr unsigned kKeyNegInf = 0x007fffffu;  // order_key(-inf)

// 2^-t for t >= 0, off by a few units of 2^-53: t = k / 1024 + r with
// |r| <= 1 / 2048, 2^-(k / 1024) from a table (and the exponent) and 2^-r from
// its series up to r^3 (the next term is below 6e-16).  A fraction of the
// double operations of a general exp2.
constexpr int kExpTab = HEAD_EXP_TAB;
__device__ __forceinline__ void fill_exp_table(double* tab) {
  for (int i = threadIdx.x; i < kExpTab; i += blockDim.x) tab[i] = exp2(-(double)i / kExpTab);
}
// 2^-t + add, for t <= 1000
__device__ __forceinline__ double exp2_neg_plus(double t, double add, const double* tab) {
  constexpr double kRound = 6755399441055744.0 / kExpTab;  // 1.5 2^52 / 1024: adding it rounds to multiples of 1 / 1024
  const double u = t + kRound;
  const int k = __double2loint(u);
  const double r = t - (u - kRound);
  // (-ln 2)^n / n!
  double q = fma(r, -5.5504108664821580e-2, 2.4022650695910071e-1);
  q = fma(q, r, -6.9314718055994531e-1);
  q = fma(q, r, 1.0);
  const double w = tab[k & (kExpTab - 1)];
  return fma(q, __hiloint2double(__double2hiint(w) - ((k >> 10) << 20), __double2loint(w)), add);
}
__device__ __forceinline__ double exp2_neg(double t, const double* tab) {
  return t < 1000.0 ? exp2_neg_plus(t, 0.0, tab) : 0.0;
}

// Whether a row's token hangs on sums over the whole vocabulary: a draw
// without top-k whose mass is shared out (no filter, or top-p).  Its groups'
// sums are formed in double; for the other rows they only enter the
// log-sum-exp, and float exponentials do.
__device__ __forceinline__ bool row_exact(const HeadArgs& a, int row) {
  if (!a.u || !((a.temperature ? a.temperature[row] : a.temperature_all) > 0.f)) return false;
  const int k = a.top_k ? a.top_k[row] : a.top_k_all;
  if (k > 0 && k < a.V) return false;
  return (a.top_p ? a.top_p[row] : a.top_p_all) < 1.f || !((a.min_p ? a.min_p[row] : a.min_p_all) > 0.f);
}

// (NaN if any is)
__device__ __forceinline__ float warp_max(float x) {
  float m;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}

// Sums over the warp of eight columns at once: each exchange halves the columns
// that a lane carries; lanes 4 j .. 4 j + 3 end with column j's.
__device__ __forceinline__ float warp_sums(float (&v)[8], int lane) {
#pragma unroll
  for (int n = 4, o = 16; n >= 1; n >>= 1, o >>= 1) {
    const bool upper = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  float r = v[0];
  r += __shfl_xor_sync(0xffffffffu, r, 2);
  r += __shfl_xor_sync(0xffffffffu, r, 1);
  return r;
}

__device__ __forceinline__ double row_scale(const HeadArgs& a, int n) {
  const float t = a.temperature ? a.temperature[n] : a.temperature_all;
  // (an infinite temperature keeps a scale above 0, so that a logit of -inf still weighs nothing)
  return t > 0.f ? fmax(kLog2e / (double)t, 1e-300) : kLog2e;  // greedy rows: log-probability at temperature 1
}

}  // namespace

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(HL_THREADS, 1)
    head_logits_kernel(const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmC32,
                       const __grid_constant__ CUtensorMap tmE, const HeadArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int S = a.stages;
  const uint32_t stage_bytes = (uint32_t)(A_STAGE_BYTES + a.nt * 64);  // [128 voc][64 d] and [nt / 2 tok][64 d]
  double* tab = reinterpret_cast<double*>(smem + (size_t)S * stage_bytes);
  double* scale = tab + kExpTab;                                          // [HEAD_ROWS] log2(e) / T
  float* scale_f = reinterpret_cast<float*>(scale + HEAD_ROWS);           // [HEAD_ROWS]
  // running largest logit and sum exp of each epilogue warp's share of the
  // vocabulary, for its columns [warp][chunk][lane]
  double* bin_sum = reinterpret_cast<double*>(scale_f + HEAD_ROWS);
  float* bin_max = reinterpret_cast<float*>(bin_sum + HL_EPI_WARPS * HL_CHUNKS * 32);
  unsigned* exact = reinterpret_cast<unsigned*>(bin_max + HL_EPI_WARPS * HL_CHUNKS * 32);  // a bit per row: row_exact
  uint64_t* bars = reinterpret_cast<uint64_t*>(exact + HEAD_ROWS / 32);
  uint64_t* full = bars;                    // leader: both CTAs' copies landed
  uint64_t* empty = full + HL_MAX_STAGES;   // each CTA: stage free again
  uint64_t* tfull = empty + HL_MAX_STAGES;  // each CTA [2]: accumulator ready
  uint64_t* tempty = tfull + 2;             // leader [2]: both epilogues done with it
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  // This pair's block of tokens, and its vocabulary entries: whole groups, as
  // many for every pair as can be; the last tile is loaded as far as it
  // reaches.  The pairs of one share of the vocabulary and different blocks
  // walk it together, so that C is read from memory once (one pair taking the
  // blocks in turn for each tile found 14 % of the second block's C in L2).
  const int pair = blockIdx.x >> 1;
  const int row0 = pair % a.n_blk * a.nt;  // first row of the block
  const int va = pair / a.n_blk * a.pair_rows, vb = (int)min((long long)a.V, (long long)va + a.pair_rows);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * HL_EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  if (threadIdx.x == 32) {
    tma_prefetch_map(&tmC);
    tma_prefetch_map(&tmC32);
    tma_prefetch_map(&tmE);
  }
  for (int n = threadIdx.x; n < HEAD_ROWS; n += HL_THREADS) {  // (whole warps)
    const bool live = n < a.n_rows;
    scale[n] = live ? row_scale(a, a.n0 + n) : 1.0;
    // (an infinite temperature's 1e-300 would be 0, and -inf * 0 NaN; the least
    // float makes exp2(d * scale) 1 for every finite d, and 0 for -inf)
    scale_f[n] = fmaxf((float)scale[n], 1.4e-45f);
    const unsigned bits = __ballot_sync(0xffffffffu, live && row_exact(a, a.n0 + n));
    if (lane == 0) exact[n >> 5] = bits;
  }
  fill_exp_table(tab);
  for (int i = threadIdx.x; i < HL_EPI_WARPS * HL_CHUNKS * 32; i += HL_THREADS) {
    bin_max[i] = -INFINITY;
    bin_sum[i] = 0.0;
  }
  if (blockIdx.x == 0) {  // for head_select
    for (int i = threadIdx.x; i < kExpTab; i += HL_THREADS) a.exp_tab[i] = exp2(-(double)i / kExpTab);
    for (int i = threadIdx.x; i < a.n_rows; i += HL_THREADS) a.scales[i] = row_scale(a, a.n0 + i);
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const WaitCtl wc{abort_flag, a.wait_limit_ns};
  const int nkb = (a.D + BK - 1) / BK;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer (both CTAs) ----------------
      // C passes through L2 once: first to leave, so that what head_select reads
      // (and its code) stays
      const uint64_t once = l2_policy_evict_first();
      int stage = 0;
      uint32_t phase = 0, armed = 0;
      for (int v0 = a.withhold_loads ? vb : va; v0 < vb; v0 += BN) {
        // groups of this tile (of 8), and of this CTA's half of it
        const int groups = min(BN / 32, (vb - v0 + 31) / 32);
        const int mine = min(BM / 32, max(0, groups - (int)rank * (BM / 32)));
        const uint32_t bytes = (uint32_t)(groups * 32 * BK * 2 + 2 * a.nt * 64);
        const int y = v0 + (int)rank * BM;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, wc)) goto producer_done;
          uint8_t* X = smem + (size_t)stage * stage_bytes;
          if (leader) mbar_arrive_expect_tx(&full[stage], bytes);
          if (mine == BM / 32)
            tma_load_2d_pair_hint(X, &tmC, &full[stage], kb * BK, y, once);
          else  // (what the other rows of the stage hold only reaches logits that nobody reads)
            for (int g = 0; g < mine; ++g)
              tma_load_2d_pair_hint(X + g * 4096, &tmC32, &full[stage], kb * BK, y + g * 32, once);
          tma_load_2d_pair(X + A_STAGE_BYTES, &tmE, &full[stage], kb * BK, a.n0 + row0 + (int)rank * (a.nt / 2));
          armed |= 1u << stage;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    producer_done:
      if (leader) {
        int dummy = 0;
        WaitCtl exit_wc{&dummy, a.wait_limit_ns};
        for (int s = 0; s < S; ++s)
          if (armed & (1u << s)) mbar_wait(&full[s], (s < stage) ? phase : (phase ^ 1u), exit_wc);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ---------------- UMMA issuer (leader only) ----------------
      const uint32_t idesc = idesc_bf16_f32(2 * BM, a.nt, false, false);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      for (int v0 = va; v0 < vb; v0 += BN) {
        if (!mbar_wait(&tempty[acc], acc_phase ^ 1u, wc)) goto mma_done;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * 256);
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&full[stage], phase, wc)) goto mma_done;
          tc_fence_after();
          const uint32_t xa = smem_u32(smem + (size_t)stage * stage_bytes);
          const uint32_t ya = xa + A_STAGE_BYTES;
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)
            umma_bf16_pair(d_tmem, sdesc_sw128(xa + k * 32, 16, 1024), sdesc_sw128(ya + k * 32, 16, 1024), idesc,
                           (kb | k) != 0);
          umma_commit_pair_mc(&empty[stage], 0x3);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        umma_commit_pair_mc(&tfull[acc], 0x3);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
    mma_done:
      umma_commit_pair_mc(drain, 0x1);
      {
        int dummy = 0;
        WaitCtl exit_wc{&dummy, a.wait_limit_ns};
        mbar_wait(drain, 0, exit_wc);
      }
    }
  } else {
    // ---------------- epilogue: one vocabulary entry (TMEM lane) per thread ----------------
    const int lg = warp & 3;
    const int hsel = (warp - 2) >> 2;
    const uint32_t lane_addr = (uint32_t)(lg * 32) << 16;
    const uint32_t tempty_leader0 = mapa_shared(smem_u32(&tempty[0]), 0);
    const uint32_t tempty_leader1 = mapa_shared(smem_u32(&tempty[1]), 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    const int n_chunk = (min(a.nt, a.n_rows - row0) + 31) / 32;
    for (int v0 = va; v0 < vb; v0 += BN) {
      const bool ready = __all_sync(0xffffffffu, mbar_wait(&tfull[acc], acc_phase, wc));
      if (!ready) break;
      tc_fence_after();
      const int v = v0 + (int)rank * BM + lg * 32 + lane;
      const int grp = v >> 5;
      const bool in = v < vb;
      for (int c = hsel; c < n_chunk && v - lane < vb; c += HL_EPI_WARPS / 4) {
        float x[32];
        tmem_ld32(tmem_base + lane_addr + (uint32_t)(acc * 256 + c * 32), x);
        const int row = row0 + c * 32;  // of the chunk's first token (a multiple of 32)
        const int n_here = min(32, a.n_rows - row);
        float* dst = a.logits + (size_t)row * a.ld + v;
        const bool in_double = exact[row >> 5] != 0u;  // (for all of the 32)
        if (v - lane + 32 > vb) {  // V ends inside this group
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = in ? x[j] : -INFINITY;
        }
        // lane j keeps column j's maximum and sum
        float my_max = 0.f;
        unsigned my_hi = 0u, my_lo = 0u;
        float my_tail = 0.f;
#pragma unroll
        for (int j0 = 0; j0 < 32; j0 += 8) {
          if (j0 < n_here) {
            float m[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              // -0 becomes +0, so that equal logits have equal keys
              x[j0 + j] += 0.f;
              if (in && j0 + j < n_here) dst[(size_t)(j0 + j) * a.ld] = x[j0 + j];
              m[j] = warp_max(x[j0 + j]);
            }
            // double: each exponential in fixed point, units of 2^-51 in two
            // words, so that a group's 32 are summed exactly by integer
            // reductions.  float: the largest logit's own (1 each) are counted
            // and the others summed apart from them, so that a log-probability
            // near 0 keeps its relative precision
            if (!in_double) {
              float e[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float d = x[j0 + j] - m[j];
                const float p = ex2_approx(d * scale_f[row + j0 + j]);
                const bool below = d < 0.f;
                e[j] = below ? p : 0.f;
                const unsigned others = __ballot_sync(0xffffffffu, below);  // (counted below)
                my_max = lane == j0 + j ? m[j] : my_max;
                my_hi = lane == j0 + j ? others : my_hi;
              }
              const float tail = __shfl_sync(0xffffffffu, warp_sums(e, lane), (lane & 7) * 4);
              my_tail = (lane >> 3) == (j0 >> 3) ? tail : my_tail;
            } else {
              // (m widened by the lane of its column; terms below 2^-80 of the
              // largest round to nothing)
#pragma unroll
              for (int j = 0; j < 8; ++j) my_max = lane == j0 + j ? m[j] : my_max;
              const double mine = (double)my_max;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const double wide_m = __shfl_sync(0xffffffffu, mine, j0 + j);
                double t = (wide_m - (double)x[j0 + j]) * scale[row + j0 + j];
                t = __hiloint2double(min(__double2hiint(t), 0x40540000), __double2loint(t));  // at most about 80
                const double w = exp2_neg_plus(t, 2.0, tab);  // in [2, 3]: the fraction's 52 bits are e in units of 2^-51
                const unsigned whi = (unsigned)__double2hiint(w) & 0xfffffu, wlo = (unsigned)__double2loint(w);
                const unsigned hi = __reduce_add_sync(0xffffffffu, (whi << 6) | (wlo >> 26));
                const unsigned lo = __reduce_add_sync(0xffffffffu, wlo & 0x3ffffffu);
                my_hi = lane == j0 + j ? hi : my_hi;
                my_lo = lane == j0 + j ? lo : my_lo;
              }
            }
          }
        }
        if (lane < n_here) {
          // a NaN becomes +inf, which marks the row (its logits are not looked at then)
          my_max = my_max == my_max ? my_max : INFINITY;
          const size_t at = (size_t)(row + lane) * a.n_grp + grp;
          a.gmax[at] = my_max;
          // this warp's own sum over the tiles
          const int i = ((warp - 2) * HL_CHUNKS + c / (HL_EPI_WARPS / 4)) * 32 + lane;
          const float old = bin_max[i], top = fmaxf(old, my_max);
          double mass = (double)__popc(~my_hi) + (double)my_tail;
          if (in_double) {
            mass = ((double)my_hi * 67108864.0 + (double)my_lo) * (1.0 / 2251799813685248.0);
            a.gmass[at] = mass;
          }
          const double f = scale[row + lane];
          if (my_max > -INFINITY)
            bin_sum[i] = bin_sum[i] * exp2_neg(((double)top - (double)old) * f, tab) +
                         mass * exp2_neg(((double)top - (double)my_max) * f, tab);
          bin_max[i] = top;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(acc ? tempty_leader1 : tempty_leader0);
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    // this warp's bin: its share of the vocabulary, every eighth group of it
    const int bin = pair / a.n_blk * 8 + (int)rank * 4 + lg;
    for (int c = hsel; c < n_chunk; c += HL_EPI_WARPS / 4) {
      const int i = ((warp - 2) * HL_CHUNKS + c / (HL_EPI_WARPS / 4)) * 32 + lane, row = row0 + c * 32 + lane;
      if (row < a.n_rows) {
        a.bmax[(size_t)row * a.n_bin + bin] = bin_max[i];
        a.bmass[(size_t)row * a.n_bin + bin] = bin_sum[i];
      }
    }
  }

  // ---------------- teardown ----------------
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicOr(a.status + ST_FLAGS, SF_TIMEOUT);
}

// ----------------------------------------------------------------------------
// head_select
// ----------------------------------------------------------------------------
namespace {

constexpr int HS_THREADS = 512;
constexpr int HS_WARPS = HS_THREADS / 32;
constexpr int kCap = 4096;       // candidates sorted in shared memory
constexpr int kGrpCap = 8192;    // group keys kept in shared memory (V up to 262144; the others are read again)

struct SelectShared {
  unsigned long long cand[kCap];  // (~key) << 32 | id: ascending = falling logit, then rising id
  union {
    double mass[kCap];
    int list[2 * kCap];           // groups to read
  };
  double tab[kExpTab];
  double red[HS_WARPS];
  unsigned ured[3][HS_WARPS];
  int rank[HS_THREADS];
  int count;
  unsigned found_key;
  int found_rank;
  int out_i;
  unsigned gkey[kGrpCap];
};

// A row's view of head_logits' results.
struct Row {
  const float* z;       // [V]
  const float* gmax;    // [n_grp]
  const double* gmass;  // [n_grp] (rows of a chunk with exact ones)
  int V, n_grp;
  int share;            // groups of a share of the vocabulary; bin b holds every eighth of share b / 8
  unsigned key[2];      // this thread's bins' largest logits (bins threadIdx.x, + HS_THREADS)
  unsigned top, low;    // the largest key, and the smallest that is not of an empty bin
  float zmax;
  double scale;         // log2(e) / T
  const double* tab;
};

__device__ __forceinline__ unsigned grp_key(const Row& r, const SelectShared& s, int g) {
  return g < kGrpCap ? s.gkey[g] : order_key(__ldg(r.gmax + g));
}
// The groups' keys to shared memory, for the paths that go through all groups.
__device__ void load_group_keys(const Row& r, SelectShared& s) {
  const int n = min(r.n_grp, kGrpCap);
  for (int g0 = threadIdx.x; g0 < n; g0 += 8 * HS_THREADS) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = g0 + j * HS_THREADS < n ? __ldg(r.gmax + g0 + j * HS_THREADS) : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (g0 + j * HS_THREADS < n) s.gkey[g0 + j * HS_THREADS] = order_key(v[j]);
  }
  __syncthreads();
}
// exp((z - zmax) / T)
__device__ __forceinline__ double mass_of(const Row& r, float z) {
  return exp2_neg(((double)r.zmax - (double)z) * r.scale, r.tab);
}

__device__ __forceinline__ double block_sum(double v, SelectShared& s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = v;
  __syncthreads();
  // every warp adds the warps' sums in the same tree
  v = s.red[threadIdx.x & (HS_WARPS - 1)];
#pragma unroll
  for (int o = HS_WARPS / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <bool MAX>
__device__ __forceinline__ unsigned block_pick(unsigned v, SelectShared& s) {
  v = MAX ? __reduce_max_sync(0xffffffffu, v) : __reduce_min_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.ured[0][threadIdx.x >> 5] = v;
  __syncthreads();
  v = s.ured[0][threadIdx.x & (HS_WARPS - 1)];
  return MAX ? __reduce_max_sync(0xffffffffu, v) : __reduce_min_sync(0xffffffffu, v);
}
// Exclusive prefix sum of one double per thread; total to every thread.
__device__ __forceinline__ double block_scan(double v, SelectShared& s, double& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  double inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();
  if (lane == 31) s.red[w] = inc;
  __syncthreads();
  double before = 0.0;
  total = 0.0;
#pragma unroll
  for (int i = 0; i < HS_WARPS; ++i) {
    if (i < w) before += s.red[i];
    total += s.red[i];
  }
  const double ex = __shfl_up_sync(0xffffffffu, inc, 1);
  return before + (lane ? ex : 0.0);
}

// A key that at least `want` bin maxima reach, and not many more: halving by
// counting threads, until the number is near `want` or the keys are
// exhausted; 0 if fewer than 3 / 2 `want` threads have a bin that holds anything
// (then the bound would be a poor one).  (A radix select's first digits put
// every group into one bin: 8000 additions to one word a digit, 77 us for one
// row of 256000 entries.)
__device__ unsigned bin_threshold(const Row& r, int want, SelectShared& s) {
  const unsigned mine = max(r.key[0], r.key[1]);
  unsigned lo = r.low, hi = r.top + 1u;  // count(lo) >= want > count(hi)
  if (2 * __syncthreads_count(mine >= lo) < 3 * want) return 0u;
  while (hi - lo > 1u) {
    const unsigned mid = lo + (hi - lo) / 2u;
    const int c = __syncthreads_count(mine >= mid);
    if (c >= want) {
      lo = mid;
      if (c <= want + min(want / 2, 128) + 16) break;
    } else {
      hi = mid;
    }
  }
  return lo;
}

// The same over all groups (1 <= want <= n_grp), with three counts a pass that
// split the keys between one that is reached often enough and one that is not
// into four.
__device__ unsigned group_threshold(const Row& r, int want, SelectShared& s) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  unsigned lo = 0u, hi = r.top + 1u;
  const int enough = want + min(want / 2, 128) + 16;
  while (hi - lo > 1u) {
    const unsigned step = max(1u, (hi - lo) / 4u);
    const unsigned t1 = lo + step, t2 = min(hi, t1 + step), t3 = min(hi, t2 + step);
    unsigned c1 = 0u, c2 = 0u, c3 = 0u;
#pragma unroll 4
    for (int g = threadIdx.x; g < r.n_grp; g += HS_THREADS) {
      const unsigned k = grp_key(r, s, g);
      c1 += k >= t1;
      c2 += k >= t2;
      c3 += k >= t3;
    }
    c1 = __reduce_add_sync(0xffffffffu, c1);
    c2 = __reduce_add_sync(0xffffffffu, c2);
    c3 = __reduce_add_sync(0xffffffffu, c3);
    __syncthreads();
    if (lane == 0) {
      s.ured[0][w] = c1;
      s.ured[1][w] = c2;
      s.ured[2][w] = c3;
    }
    __syncthreads();
    const unsigned half = lane < HS_WARPS ? 1u : 0u;
    c1 = __reduce_add_sync(0xffffffffu, half * s.ured[0][lane & (HS_WARPS - 1)]);
    c2 = __reduce_add_sync(0xffffffffu, half * s.ured[1][lane & (HS_WARPS - 1)]);
    c3 = __reduce_add_sync(0xffffffffu, half * s.ured[2][lane & (HS_WARPS - 1)]);
    int c_lo = INT_MAX;
    if ((int)c3 >= want) {
      lo = t3;
      c_lo = (int)c3;
    } else if ((int)c2 >= want) {
      lo = t2;
      hi = t3;
      c_lo = (int)c2;
    } else if ((int)c1 >= want) {
      lo = t1;
      hi = t2;
      c_lo = (int)c1;
    } else {
      hi = t1;
    }
    if (c_lo <= enough) break;
  }
  return lo;
}

// Appends every entry with key >= thr to s.cand (as far as it fits); their
// number, or one above kCap, is returned to all threads.  by_bins: the groups
// to read are looked up among the bins that reach thr, else among all (whose
// keys have been loaded).
__device__ int gather_candidates(const Row& r, unsigned thr, bool by_bins, SelectShared& s) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  constexpr int kBins = 2 * HS_THREADS;
  int* groups = s.list + kBins;  // room for 2 kCap - kBins
  __syncthreads();
  if (threadIdx.x == 0) {
    s.count = 0;
    s.found_rank = 0;
    s.out_i = 0;
  }
  __syncthreads();
  // one addition per warp for the lanes that have a group
  auto add_groups = [&](bool has, int g) {
    const unsigned who = __ballot_sync(0xffffffffu, has);
    if (who == 0u) return;
    int at = 0;
    if (lane == 0) at = atomicAdd(&s.found_rank, __popc(who));
    at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1u));
    if (has && at < 2 * kCap - kBins) groups[at] = g;
  };
  if (by_bins) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool has = r.key[i] >= thr;
      const unsigned who = __ballot_sync(0xffffffffu, has);
      int at = 0;
      if (lane == 0 && who) at = atomicAdd(&s.out_i, __popc(who));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1u));
      if (has) s.list[at] = threadIdx.x + i * HS_THREADS;
    }
    __syncthreads();
    // a lane per group of a bin, four bins a turn
    const int n_bins = s.out_i;
    for (int i = w; i < n_bins; i += 4 * HS_WARPS) {
      for (int t = 0; t * 8 < r.share; t += 32) {
        unsigned key[4];
        int g[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int bin = i + q * HS_WARPS < n_bins ? s.list[i + q * HS_WARPS] : 0;
          const int in_share = (t + lane) * 8 + (bin & 7);
          g[q] = (bin >> 3) * r.share + in_share;
          const bool there = i + q * HS_WARPS < n_bins && in_share < r.share && g[q] < r.n_grp;
          key[q] = there ? order_key(__ldg(r.gmax + g[q])) : 0u;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) add_groups(key[q] >= thr, g[q]);
      }
    }
  } else {
    for (int g0 = 0; g0 < r.n_grp; g0 += HS_THREADS) {
      const int g = g0 + (int)threadIdx.x;
      add_groups(g < r.n_grp && grp_key(r, s, g) >= thr, g);
    }
  }
  __syncthreads();
  const int n_list = s.found_rank;
  if (n_list > kCap) return kCap + 1;  // a candidate at least from each
  for (int i = w; i < n_list; i += 8 * HS_WARPS) {
    // eight groups a turn, so that their loads overlap
    float z[8];
    int v[8], total = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int at = i + q * HS_WARPS;
      v[q] = at < n_list ? groups[at] * 32 + lane : r.V;
      z[q] = v[q] < r.V ? __ldg(r.z + v[q]) : 0.f;
    }
    unsigned hits[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      hits[q] = __ballot_sync(0xffffffffu, v[q] < r.V && order_key(z[q]) >= thr);
      total += __popc(hits[q]);
    }
    int at = 0;
    if (lane == 0) at = atomicAdd(&s.count, total);
    at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int mine = at + __popc(hits[q] & ((1u << lane) - 1u));
      if ((hits[q] >> lane & 1u) && mine < kCap)
        s.cand[mine] = ((unsigned long long)(~order_key(z[q])) << 32) | (unsigned)v[q];
      at += __popc(hits[q]);
    }
  }
  __syncthreads();
  return s.count;
}

// Candidates: every entry not below some key that at least `want` groups reach
// (their number as of gather_candidates); thr: that key, or `floor` if that is
// larger.
__device__ int gather_top_groups(const Row& r, int want, unsigned floor, unsigned& thr, SelectShared& s) {
  thr = bin_threshold(r, want, s);
  if (thr) {
    thr = max(floor, thr);
    return gather_candidates(r, thr, true, s);
  }
  load_group_keys(r, s);
  thr = max(floor, want < r.n_grp ? group_threshold(r, want, s) : 0u);
  return gather_candidates(r, thr, false, s);
}

// How many of n <= HS_THREADS values value(0 .. n - 1) are below this thread's,
// value(threadIdx.x).  The comparisons of a value are shared by HS_THREADS / n
// threads.
template <typename Fn>
__device__ int block_rank(int n, Fn value, SelectShared& s) {
  int m = 32;
  while (m < n) m <<= 1;
  const int i = threadIdx.x & (m - 1), parts = HS_THREADS / m, part = threadIdx.x / m;
  __syncthreads();
  s.rank[threadIdx.x] = 0;
  __syncthreads();
  if (i < n) {
    const auto mine = value(i);
    int c = 0;
#pragma unroll 8
    for (int j = part; j < n; j += parts) c += value(j) < mine;
    if (c) atomicAdd(&s.rank[i], c);
  }
  __syncthreads();
  return s.rank[threadIdx.x];
}

// Sorts s.cand[0 .. n) ascending (n <= kCap; the rest up to a power of two is filled).
__device__ void sort_candidates(SelectShared& s, int n) {
  if (n <= HS_THREADS) {
    const int rank = block_rank(n, [&](int i) { return s.cand[i]; }, s);
    const unsigned long long mine = (int)threadIdx.x < n ? s.cand[threadIdx.x] : 0ull;
    __syncthreads();
    if ((int)threadIdx.x < n) s.cand[rank] = mine;
    __syncthreads();
    return;
  }
  __syncthreads();
  int size2 = 1;
  while (size2 < n) size2 <<= 1;
  __syncthreads();
  for (int i = n + (int)threadIdx.x; i < size2; i += HS_THREADS) s.cand[i] = ~0ull;
  for (int size = 2; size <= size2; size <<= 1) {
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      __syncthreads();
      for (int i = threadIdx.x; i < (size2 >> 1); i += HS_THREADS) {
        const int lo = 2 * i - (i & (stride - 1));
        const int hi = lo + stride;
        const bool up = (lo & size) == 0;
        const unsigned long long ka = s.cand[lo], kb = s.cand[hi];
        if ((ka > kb) == up) {
          s.cand[lo] = kb;
          s.cand[hi] = ka;
        }
      }
    }
  }
  __syncthreads();
}
__device__ __forceinline__ unsigned cand_key(unsigned long long c) { return ~(unsigned)(c >> 32); }

// ---- the whole row: where bins, groups and candidates do not settle it ----

// f(id, logit) for the entries [a, b) of this warp, four loads at a time.
template <typename F>
__device__ __forceinline__ void warp_stream(const Row& r, int a, int b, F f) {
  for (int v0 = a + (int)(threadIdx.x & 31); v0 < b; v0 += 128) {
    float z[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] = v0 + 32 * j < b ? __ldg(r.z + v0 + 32 * j) : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (v0 + 32 * j < b) f(v0 + 32 * j, z[j]);
  }
}
// A sixteenth of [a, b), in whole groups, rounded up.
__device__ __forceinline__ int part_of(int a, int b) { return ((b - a) / HS_WARPS + 32) & ~31; }

// Sum of weight(id, logit) over each warp's part of [a, b), to s.red.
template <typename F>
__device__ void part_sums(const Row& r, int a, int b, F weight, SelectShared& s) {
  const int w = threadIdx.x >> 5, part = part_of(a, b);
  double m = 0.0;
  warp_stream(r, min(b, a + w * part), min(b, a + w * part + part), [&](int v, float z) { m += weight(v, z); });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.red[w] = m;
  __syncthreads();
}

// The first id of [a, b) at which the cumulated weight is above `left` (the
// last with any weight if none is); s.red holds part_sums of that range.
template <typename F>
__device__ int locate(const Row& r, int a, int b, double left, F weight, SelectShared& s) {
  while (true) {
    // the part that holds it: the last with any weight that begins at or below it
    const int part = part_of(a, b);
    int at = 0;
    double run = 0.0, skipped = 0.0;
    for (int i = 0; i < HS_WARPS; ++i) {
      if (s.red[i] > 0.0 && run <= left) {
        at = i;
        skipped = run;
      }
      run += s.red[i];
    }
    left -= skipped;
    a = min(b, a + at * part);
    b = min(b, a + part);
    if (b - a <= 256) break;
    part_sums(r, a, b, weight, s);
  }
  const int lane = threadIdx.x & 31;
  int last = a;
  for (int v0 = a; v0 < b; v0 += 32) {  // (every warp alike)
    const int v = v0 + lane;
    const double own = v < b ? weight(v, __ldg(r.z + v)) : 0.0;
    double inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    const unsigned any = __ballot_sync(0xffffffffu, own > 0.0);
    const unsigned over = __ballot_sync(0xffffffffu, own > 0.0 && inc > left);
    if (over) return v0 + __ffs((int)over) - 1;
    if (any) last = v0 + 31 - __clz((int)any);
    left -= __shfl_sync(0xffffffffu, inc, 31);
  }
  return last;
}

// A prefix of the falling order: the entries above `key` and those with that
// key and an id up to `id`.
struct Border {
  unsigned key;
  int id;
};
__device__ __forceinline__ bool within(const Border& e, unsigned key, int v) {
  return key > e.key || (key == e.key && v <= e.id);
}

// Appends the entries of the row that take(id, key) accepts to s.cand; their
// number (at most kCap are kept).
template <typename F>
__device__ int gather_if(const Row& r, F take, SelectShared& s) {
  const int w = threadIdx.x >> 5, part = part_of(0, r.V);
  __syncthreads();
  if (threadIdx.x == 0) s.count = 0;
  __syncthreads();
  warp_stream(r, min(r.V, w * part), min(r.V, w * part + part), [&](int v, float z) {
    const unsigned key = order_key(z);
    if (take(v, key)) {
      const int at = atomicAdd(&s.count, 1);
      if (at < kCap) s.cand[at] = ((unsigned long long)(~key) << 32) | (unsigned)v;
    }
  });
  __syncthreads();
  return min(s.count, kCap);
}

// The shortest prefix that holds `need` (> 0) entries, or (MASS) `need` of the
// mass sum exp((z - zmax) / T).  Three thresholds a pass close in on the key
// where it ends, until at most kCap entries are left to sort, or one key.
template <bool MASS>
__device__ Border find_border(const Row& r, double need, SelectShared& s) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, part = part_of(0, r.V);
  // measure(>= lo) >= need > measure(>= hi); so many entries reach either
  unsigned lo = 0u, hi = r.top + 1u;
  double above = 0.0;
  int n_lo = r.V, n_hi = 0;
  float reach = fmaxf(fmaxf(r.zmax - key_value(r.low), 1e-6f * fabsf(r.zmax)), 1e-30f);
  for (int pass = 0; n_lo - n_hi > kCap && hi - lo > 1u; ++pass) {
    unsigned t[3];  // rising
    if (lo == 0u && pass < 16) {
      // no lower end yet: steps from the largest that grow
      const float z0 = pass == 0 ? r.zmax : key_value(hi);
#pragma unroll
      for (int i = 0; i < 3; ++i) t[i] = order_key(fmaxf(z0 - reach * (i == 0 ? 4.f : i == 1 ? 2.f : 1.f), -FLT_MAX));
      reach *= 8.f;
    } else if (pass < 32) {
      // quarters of the logits between them
      const float a = key_value(lo), b = key_value(hi - 1u), d = b * 0.25f - a * 0.25f;
#pragma unroll
      for (int i = 0; i < 3; ++i) t[i] = order_key(a + d * (float)(i + 1));
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i) t[i] = lo + (unsigned)(((unsigned long long)(hi - lo) * (i + 1)) >> 2);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) t[i] = min(max(t[i], lo + 1u), hi - 1u);
    double m[3] = {0.0, 0.0, 0.0};
    int c[3] = {0, 0, 0};
    warp_stream(r, min(r.V, w * part), min(r.V, w * part + part), [&](int, float z) {
      const unsigned key = order_key(z);
      if (key >= t[0]) {
        const double e = MASS ? mass_of(r, z) : 0.0;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          if (key >= t[i]) {
            ++c[i];
            if (MASS) m[i] += e;
          }
        }
      }
    });
    int n[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      n[i] = __reduce_add_sync(0xffffffffu, c[i]);
      __syncthreads();
      if (lane == 0) s.ured[0][w] = (unsigned)n[i];
      __syncthreads();
      n[i] = (int)__reduce_add_sync(0xffffffffu, lane < HS_WARPS ? s.ured[0][lane] : 0u);
      m[i] = MASS ? block_sum(m[i], s) : (double)n[i];
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {  // (rising: the last that still holds it)
      if (m[i] >= need && t[i] > lo) {
        lo = t[i];
        n_lo = n[i];
      }
    }
#pragma unroll
    for (int i = 2; i >= 0; --i) {
      if (!(m[i] >= need) && t[i] < hi) {
        hi = t[i];
        n_hi = n[i];
        above = m[i];
      }
    }
  }
  const int left = n_lo - n_hi;
  if (left > kCap) {
    // one key, of which the lowest ids belong to it
    const double one = MASS ? mass_of(r, key_value(lo)) : 1.0;
    const double want = ceil((need - above) / one);
    const int n = want >= 1.0 ? (want < (double)left ? (int)want : left) : 1;
    if (n == left) return Border{lo, r.V};
    auto is_tie = [&](int, float z) { return order_key(z) == lo ? 1.0 : 0.0; };
    part_sums(r, 0, r.V, is_tie, s);
    return Border{lo, locate(r, 0, r.V, (double)n - 0.5, is_tie, s)};
  }
  const int c = gather_if(r, [&](int, unsigned key) { return key >= lo && key < hi; }, s);
  sort_candidates(s, c);
  // the entries before which less than `need` has come
  constexpr int PER = kCap / HS_THREADS;
  const int i0 = threadIdx.x * PER;
  double e[PER], sum = 0.0, total;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    e[j] = i0 + j < c ? (MASS ? mass_of(r, key_value(cand_key(s.cand[i0 + j]))) : 1.0) : 0.0;
    sum += e[j];
  }
  double before = above + block_scan(sum, s, total);
  unsigned keep = 0u;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    if (i0 + j < c && before < need) keep = (unsigned)(i0 + j + 1);
    before += e[j];
  }
  const int n = (int)block_pick<true>(keep, s);
  if (n == 0) return Border{min(hi, r.top), r.V};  // (does not happen: `above` is less than `need`)
  const unsigned long long last = s.cand[n - 1];
  return Border{cand_key(last), (int)(unsigned)last};
}

// The k largest entries (k <= kCap, k <= V) as candidates: at least these,
// sorted; their number.
__device__ int top_candidates(const Row& r, int k, SelectShared& s) {
  int c = kCap + 1;
  unsigned thr;
  if (r.n_grp >= k || r.V <= kCap) c = gather_top_groups(r, k, 0u, thr, s);
  if (c > kCap) {
    const Border e = find_border<false>(r, (double)k, s);
    c = gather_if(r, [&](int v, unsigned key) { return within(e, key, v); }, s);
  }
  sort_candidates(s, c);
  return c;
}

// Settles row-wide what the sorted candidates could not: the prefix that top-k
// (k > 0) and top-p leave, and the draw from it, in the order of ids, without
// the entries below min_p.
__device__ int wide_draw(const Row& r, int k, double p, double min_p, double u, double total, SelectShared& s) {
  Border e{0u, r.V};
  auto kept = [&](int v, float z) {
    if (!within(e, order_key(z), v)) return 0.0;
    const double m = mass_of(r, z);
    return m >= min_p ? m : 0.0;
  };
  auto sum_parts = [&]() {
    double t = 0.0;
    for (int i = 0; i < HS_WARPS; ++i) t += s.red[i];
    return t;
  };
  if (k > 0) {
    e = find_border<false>(r, (double)k, s);
    if (p < 1.0) {
      part_sums(r, 0, r.V, [&](int v, float z) { return within(e, order_key(z), v) ? mass_of(r, z) : 0.0; }, s);
      total = sum_parts();
    }
  }
  if (p < 1.0) {
    const Border q = find_border<true>(r, fmax(p * total, 1e-300), s);
    if (q.key > e.key || (q.key == e.key && q.id < e.id)) e = q;
  }
  part_sums(r, 0, r.V, kept, s);
  return locate(r, 0, r.V, u * sum_parts(), kept, s);
}

// Draw without filters: the first id whose cumulated mass passes u times the
// whole, from the bins' sums (mass[]: this thread's bins'), the groups' sums of
// one share and one group's logits.
__device__ int plain_draw(const Row& r, const double (&mass)[2], double u, double& total, SelectShared& s) {
  const int lane = threadIdx.x & 31;
  // a share's sum: that of its eight bins
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    double m = mass[i];
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
    if ((lane & 7) == 0) s.mass[(threadIdx.x + i * HS_THREADS) / 8] = m;
  }
  __syncthreads();
  constexpr int kShares = HEAD_BINS / 8;
  double m = threadIdx.x < kShares ? s.mass[threadIdx.x] : 0.0;
  double before = block_scan(m, s, total);
  double left = u * total;
  // the share that holds the target: the last that begins at or below it
  unsigned at = block_pick<true>(m > 0.0 && before <= left ? threadIdx.x + 1u : 0u, s);
  const int share = at ? (int)at - 1 : 0;
  if ((int)threadIdx.x == share) s.red[0] = before;
  __syncthreads();
  left -= s.red[0];
  __syncthreads();
  // its groups, and the first of them that passes the target (else the last with any mass)
  const int ga = share * r.share, gb = min(r.n_grp, ga + r.share);
  int best = ga;
  double best_left = left;
  for (int g0 = ga; g0 < gb; g0 += HS_THREADS) {
    const int g = g0 + (int)threadIdx.x;
    m = g < gb ? __ldg(r.gmass + g) * mass_of(r, __ldg(r.gmax + g)) : 0.0;
    double here;
    before = block_scan(m, s, here);
    const unsigned over = block_pick<false>(m > 0.0 && before + m > left ? threadIdx.x : 0x7fffffffu, s);
    at = over != 0x7fffffffu ? over + 1u : block_pick<true>(m > 0.0 ? threadIdx.x + 1u : 0u, s);
    if (at) {
      best = g0 + (int)at - 1;
      if (threadIdx.x + 1u == at) s.red[0] = before;
      __syncthreads();
      best_left = left - s.red[0];
      __syncthreads();
    }
    if (over != 0x7fffffffu) break;
    left -= here;
  }
  // its entries (every warp alike)
  const int v = best * 32 + lane;
  const double own = v < r.V ? mass_of(r, __ldg(r.z + v)) : 0.0;
  double inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  const unsigned any = __ballot_sync(0xffffffffu, own > 0.0);
  const unsigned over = __ballot_sync(0xffffffffu, own > 0.0 && inc > best_left);
  return best * 32 + (over ? __ffs((int)over) - 1 : 31 - __clz((int)any));
}

// Draw from sorted candidates that hold every kept entry; k = 0: no top-k.
__device__ int draw_from_candidates(const Row& r, int c, int k, double p, double min_p, double u, double total,
                                    SelectShared& s) {
  if (k > 0) c = min(c, k);
  if (c <= HS_THREADS) {
    // an entry per thread
    const int i = threadIdx.x;
    const unsigned long long mine = i < c ? s.cand[i] : 0ull;
    double e = i < c ? mass_of(r, key_value(cand_key(mine))) : 0.0, sum;
    const double before = block_scan(e, s, sum);
    if (k > 0) total = sum;
    // (both filters leave a prefix)
    const int n = __syncthreads_count(i < c && (i == 0 || p >= 1.0 || before < p * total) && e >= min_p);
    if (n <= 1) return (int)(unsigned)s.cand[0];
    const int rank = block_rank(n, [&](int x) { return (unsigned)s.cand[x]; }, s);
    if (i < n) {
      s.cand[rank] = mine & 0xffffffffull;
      s.mass[rank] = e;
    }
    __syncthreads();
    e = i < n ? s.mass[i] : 0.0;
    const double cum = block_scan(e, s, sum) + e;
    unsigned first = block_pick<false>(e > 0.0 && cum > u * sum ? (unsigned)i : 0x7fffffffu, s);
    if (first == 0x7fffffffu) first = block_pick<true>(e > 0.0 ? (unsigned)i : 0u, s);
    return (int)s.cand[first];
  }
  constexpr int PER = kCap / HS_THREADS;
  // masses in falling order and what comes before each
  const int i0 = threadIdx.x * PER;
  double e[PER], m = 0.0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    e[j] = i0 + j < c ? mass_of(r, key_value(cand_key(s.cand[i0 + j]))) : 0.0;
    m += e[j];
  }
  double sum;
  double before = block_scan(m, s, sum);
  if (k > 0) total = sum;
  int keep = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    if (i0 + j < c && (i0 + j == 0 || p >= 1.0 || before < p * total) && e[j] >= min_p) ++keep;
    before += e[j];
  }
  // (both filters leave a prefix)
  const int n = (int)(block_sum((double)keep, s) + 0.5);
  if (n <= 1) return (int)(unsigned)s.cand[0];
  // the kept entries in the order of ids; their keys are needed for the masses
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += HS_THREADS) {
    const unsigned long long cc = s.cand[i];
    s.mass[i] = mass_of(r, key_value(cand_key(cc)));
    s.cand[i] = ((cc & 0xffffffffull) << 32) | (unsigned)i;
  }
  sort_candidates(s, n);
  m = 0.0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    e[j] = i0 + j < n ? s.mass[(unsigned)s.cand[i0 + j]] : 0.0;
    m += e[j];
  }
  before = block_scan(m, s, sum);
  const double target = u * sum;
  unsigned pick = 0xffffffffu;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    before += e[j];
    if (i0 + j < n && e[j] > 0.0 && before > target) pick = min(pick, (unsigned)(i0 + j));
  }
  pick = block_pick<false>(pick, s);
  if (pick == 0xffffffffu) pick = (unsigned)(n - 1);
  return (int)(s.cand[pick] >> 32);
}

__device__ int sample_row(const Row& r, const double (&mass)[2], int k, double p, double min_p, double u,
                          double& total, bool greedy, SelectShared& s) {
  if (k >= r.V || k < 0) k = 0;
  if (greedy || k == 1) {
    // the lowest id among the largest logits
    unsigned g_first = 0x7fffffffu;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (r.key[i] == r.top) {
        const int bin = threadIdx.x + i * HS_THREADS, g0 = (bin >> 3) * r.share;
        for (int j = bin & 7; j < r.share && g0 + j < r.n_grp; j += 8)
          if (order_key(__ldg(r.gmax + g0 + j)) == r.top) {
            g_first = min(g_first, (unsigned)(g0 + j));
            break;
          }
      }
    const int g = min((int)block_pick<false>(g_first, s), r.n_grp - 1);
    const int v = g * 32 + (int)(threadIdx.x & 31);
    const unsigned eq = __ballot_sync(0xffffffffu, v < r.V && order_key(__ldg(r.z + v)) == r.top);
    return g * 32 + __ffs((int)eq) - 1;
  }
  if (k == 0 && p >= 1.0 && !(min_p > 0.0)) return plain_draw(r, mass, u, total, s);
  if (k > 0 && k <= kCap) {
    const int c = top_candidates(r, k, s);
    return draw_from_candidates(r, c, k, p, min_p, u, total, s);
  }
  if (k == 0) {
    // entries below min_p of the largest are out (a little slack, in the mass
    // too, whose rounding is far apart in logits at a large T: their own masses
    // decide); of the others, groups in growing numbers until their candidates
    // hold p of the mass
    unsigned floor_key = 0u;
    if (min_p > 0.0) {
      const double t = (double)r.zmax + (log2(min_p) - 0x1p-50) / r.scale;
      floor_key = min(r.top, order_key((float)(t - 1e-6 * (fabs(t) + fabs((double)r.zmax) + 1.0))));
    }
    for (int want = 64; want <= 4096; want <<= 3) {
      unsigned thr = floor_key;
      int c;
      if (p < 1.0)
        c = gather_top_groups(r, want, floor_key, thr, s);
      else
        c = gather_candidates(r, thr, true, s);
      if (c > kCap) break;
      double m = 0.0;
      for (int i = threadIdx.x; i < c; i += HS_THREADS) m += mass_of(r, key_value(cand_key(s.cand[i])));
      m = block_sum(m, s);
      if (thr == floor_key || m >= p * total) {
        sort_candidates(s, c);
        return draw_from_candidates(r, c, 0, p, min_p, u, total, s);
      }
    }
  }
  return wide_draw(r, k, p, min_p, u, total, s);
}

}  // namespace

__global__ void __launch_bounds__(HS_THREADS, 2) head_select_kernel(const HeadArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SelectShared& s = *reinterpret_cast<SelectShared*>(smem_raw);
  const int n = blockIdx.x;          // row of this chunk
  const int row = a.n0 + n;
  const float qnan = __int_as_float(0x7fc00000);
  Row r;
  r.z = a.logits + (size_t)n * a.ld;
  r.gmax = a.gmax + (size_t)n * a.n_grp;
  r.gmass = a.gmass + (size_t)n * a.n_grp;
  r.V = a.V;
  r.n_grp = a.n_grp;
  r.scale = __ldg(a.scales + n);
  r.tab = s.tab;
  for (int i = threadIdx.x; i < kExpTab; i += HS_THREADS) s.tab[i] = __ldg(a.exp_tab + i);
  r.share = a.pair_rows / 32;
  float bmax[2];
  double mass[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int bin = threadIdx.x + i * HS_THREADS;
    bmax[i] = bin < a.n_bin ? __ldg(a.bmax + (size_t)n * a.n_bin + bin) : -INFINITY;
    mass[i] = bin < a.n_bin ? __ldg(a.bmass + (size_t)n * a.n_bin + bin) : 0.0;
    r.key[i] = order_key(bmax[i]);
  }
  r.top = block_pick<true>(max(r.key[0], r.key[1]), s);
  r.zmax = key_value(r.top);
  const unsigned own = max(r.key[0], r.key[1]);
  r.low = block_pick<false>(own > kKeyNegInf ? own : 0xffffffffu, s);
  const bool timeout = (a.status[ST_FLAGS] & SF_TIMEOUT) != 0;
  const bool broken = r.top >= kKeyPosInf || r.top <= kKeyNegInf;  // an infinite (or NaN) logit on top
  if (timeout || broken) {
    if (threadIdx.x == 0 && !timeout) atomicOr(a.status + ST_FLAGS, SF_NONFINITE);
    if (a.u) {
      if (threadIdx.x == 0) {
        a.token[row] = -1;
        a.logp[row] = qnan;
      }
    } else {
      for (int i = threadIdx.x; i < a.k; i += HS_THREADS) {
        a.values[(size_t)row * a.k + i] = qnan;
        a.ids[(size_t)row * a.k + i] = -1;
      }
      if (threadIdx.x == 0) a.lse[row] = qnan;
    }
    return;
  }
  // sum exp((z - zmax) / T) (a draw without filters adds its shares up itself)
#pragma unroll
  for (int i = 0; i < 2; ++i) mass[i] *= mass_of(r, bmax[i]);
  double total = block_sum(mass[0] + mass[1], s);
  constexpr double kLn2 = 0.69314718055994530942;

  if (!a.u) {
    const int c = top_candidates(r, a.k, s);
    for (int i = threadIdx.x; i < a.k; i += HS_THREADS) {
      const unsigned long long cc = i < c ? s.cand[i] : 0ull;
      a.values[(size_t)row * a.k + i] = key_value(cand_key(cc));
      a.ids[(size_t)row * a.k + i] = (int64_t)(unsigned)cc;
    }
    if (threadIdx.x == 0) a.lse[row] = (float)((double)r.zmax + log(total));
    return;
  }
  const float t = a.temperature ? a.temperature[row] : a.temperature_all;
  const int k = a.top_k ? a.top_k[row] : a.top_k_all;
  // settings outside their ranges act as the nearest inside; NaN as "off" (u: 0)
  double p = (double)(a.top_p ? a.top_p[row] : a.top_p_all);
  p = p < 1.0 ? fmax(p, 0.0) : 1.0;
  double min_p = (double)(a.min_p ? a.min_p[row] : a.min_p_all);
  min_p = min_p > 0.0 ? fmin(min_p, 1.0) : 0.0;
  const double u = fmax((double)a.u[row], 0.0);
  int token = sample_row(r, mass, k, p, min_p, u, total, !(t > 0.f), s);
  if (threadIdx.x == 0) {
    token = min(max(token, 0), a.V - 1);  // (an index into the row whatever the workspace holds)
    a.token[row] = token;
    a.logp[row] = (float)(((double)__ldg(r.z + token) - (double)r.zmax) * r.scale * kLn2 - log(total));
  }
}

// shared memory behind the stages: scales, table, row bits, barriers
constexpr int kHeadExtra = HL_EPI_WARPS * HL_CHUNKS * 32 * 12 + HEAD_ROWS * 12 + kExpTab * 8 + HEAD_ROWS / 8 + 8 * (2 * HL_MAX_STAGES + 5) + 16;

int head_logits_stages(int nt) {
  const int fit = (227 * 1024 - 1024 - kHeadExtra) / (A_STAGE_BYTES + nt * 64);
  return fit < HL_MAX_STAGES ? fit : HL_MAX_STAGES;
}

// tmC, tmC32: C in boxes of {64, 128} and {64, 32}; tmE: E in boxes of {64, nt / 2}; grid: an even number of CTAs.
cudaError_t launch_head_logits(const CUtensorMap& tmC, const CUtensorMap& tmC32, const CUtensorMap& tmE,
                               const HeadArgs& a, int grid, cudaStream_t stream) {
  const size_t smem = 1024 + (size_t)a.stages * (A_STAGE_BYTES + a.nt * 64) + kHeadExtra;
  cudaError_t e = cudaFuncSetAttribute(head_logits_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  head_logits_kernel<<<grid, HL_THREADS, smem, stream>>>(tmC, tmC32, tmE, a);
  return cudaGetLastError();
}

cudaError_t launch_head_select(const HeadArgs& a, cudaStream_t stream) {
  const size_t smem = sizeof(SelectShared);
  cudaError_t e = cudaFuncSetAttribute(head_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  head_select_kernel<<<a.n_rows, HS_THREADS, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace cce
