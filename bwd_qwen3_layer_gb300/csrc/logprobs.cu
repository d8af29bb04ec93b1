// Log probabilities of given tokens with each row's entropy and most likely classes,
// and their gradient. With m = max z, x = z - m, s = sum exp(x), u = sum x exp(x):
//   log p_t = x_t - log s,  H = log s - u / s,
//   dz_j = a (1[j = t] - p_j) - b p_j (log p_j + H).
//
// Forward: one read of the logits, bound by HBM where there are many rows (2045 x 151936
// bf16: 96 us, 95 % of the copy rate), by the trips behind the pass where there are few
// (one row with 5 alternatives 6 us, 64 x 151936 fp32 with 20: 15, of which the pass 8;
// 301 x 32001 with 8: 12). A cluster of up to 8 CTAs takes a row; a thread keeps its own
// m, s, u over 32-byte vectors of the row, rescaled when its maximum moves; the threads'
// meet in the warp, the CTA and, through distributed shared memory, the cluster's first
// CTA, always in the same order. What runs once per row is kept short: fetching unrolled
// code costs such a launch more than its loops do (wider unrolls there: 6 -> 9 us).
//
// Most likely classes. A class is a 64-bit key, the logit in the order of unsigned numbers
// above the complement of the index: keys are distinct, equal logits go to the lower index.
// A thread's maximum is known from the pass. The n best threads of a CTA hold the n best
// classes of its share, and a class worth listing is at least as good as the n-th best
// thread's maximum (found bit by bit): those threads' vectors (n of 256 threads') are read
// once more, from L2, and what passes, a few more than n as a rule, is put in order by
// counting who is better. The first CTA orders the cluster's lists in the same way. Should
// more pass than there is room for, equal logits are the reason (a mask of the type's
// lowest value, a row of one value): then the better classes are listed alone and of the
// equal ones the first, found by reading the row from its beginning. If the better ones
// alone are too many (they fill few threads' vectors), the CTA looks for its n best one
// after the other.
#include <cooperative_groups.h>
#include <limits.h>
#include <math.h>

#include "internal.h"
#include "kl_common.cuh"

namespace cg = cooperative_groups;

namespace kl {
namespace {

constexpr int LP_THREADS = 256;
constexpr int LP_WARPS = LP_THREADS / 32;
constexpr int LP_U = 2;            // vectors a thread looks at together
constexpr int LP_ROOM = 1024;      // classes a CTA puts in order
constexpr float LP_LOG2E = 1.4426950408889634f;
constexpr float LP_FAR = -1e30f;   // stands for x = -inf, whose exponential is 0 and whose product with that must be too

struct LpParams {
  const void* z;
  int64_t ldz;
  const int32_t* tokens;
  float* logprob;
  float* entropy;
  float* norm;
  int32_t* top_id;
  float* top_lp;
  int N, V, top;
  uint32_t* err;
};

__device__ __forceinline__ float lp_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lp_max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Aligned 32-byte vectors of T: 8 floats or 16 bf16, as floats.
template <typename T> struct LpVec;
template <> struct LpVec<float> {
  static constexpr int N = 8;
  uint32_t w[8];
  static constexpr uint32_t NONE = 0xff800000u;          // -infinity
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(w[i]); }
  __device__ __forceinline__ float max() const {
    float m = get(0);
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, get(i));
    return m;
  }
};
template <> struct LpVec<__nv_bfloat16> {
  static constexpr int N = 16;
  uint32_t w[8];
  static constexpr uint32_t NONE = 0xff80ff80u;
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16); }
  __device__ __forceinline__ float max() const {
    uint32_t m = w[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
};
template <typename T>
__device__ __forceinline__ LpVec<T> lp_load(const T* p) {
  LpVec<T> v;
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
               : "l"(p));
  return v;
}
// A row is `head` classes before the first aligned vector, `vecs` such vectors and `tail` classes behind them.
template <typename T>
struct LpRow {
  static constexpr int N = LpVec<T>::N;
  const T* z;
  int V, head, vecs, tail;
  __device__ __forceinline__ LpRow(const T* z_, int V_) : z(z_), V(V_) {
    head = min(static_cast<int>((0u - reinterpret_cast<uintptr_t>(z_)) & 31u) / static_cast<int>(sizeof(T)), V);
    vecs = (V - head) / N;
    tail = V - head - vecs * N;
  }
  __device__ __forceinline__ const T* at(int vec) const { return z + head + vec * N; }
  // class `i` of the two ends
  __device__ __forceinline__ int end(int i) const { return i < head ? i : V - tail + (i - head); }
  __device__ __forceinline__ LpVec<T> load(int vec) const {
    if (vec < vecs) return lp_load(at(vec));
    LpVec<T> v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v.w[e] = LpVec<T>::NONE;
    return v;
  }
};

// A class's key; 0 for a logit of -infinity. (A NaN gets a high one: such a row's list means nothing.)
__device__ __forceinline__ uint32_t lp_order(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);             // -0 becomes 0
  return z == -INFINITY ? 0 : b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t lp_key(float z, int j) {
  const uint32_t order = lp_order(z);
  return order ? static_cast<uint64_t>(order) << 32 | static_cast<uint32_t>(~j) : 0;
}
__device__ __forceinline__ int lp_class(uint64_t key) { return static_cast<int>(~static_cast<uint32_t>(key)); }
__device__ __forceinline__ float lp_logit(uint64_t key) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  return __uint_as_float(o >> 31 ? o & 0x7fffffffu : ~o);
}

struct LpSum {
  float m, s, u;
};
// The summary of two sets of logits. An empty one is (-inf, 0, 0); one without any number above -inf but
// with a NaN (-inf, NaN, 0).
__device__ __forceinline__ LpSum lp_merge(const LpSum& a, const LpSum& b) {
  LpSum r;
  r.m = fmaxf(a.m, b.m);
  if (r.m == -INFINITY) {
    r.s = a.s + b.s;
    r.u = 0.f;
    return r;
  }
  const float da = fmaxf(a.m - r.m, LP_FAR), db = fmaxf(b.m - r.m, LP_FAR);
  const float fa = lp_ex2(da * LP_LOG2E), fb = lp_ex2(db * LP_LOG2E);
  r.s = a.s * fa + b.s * fb;
  r.u = fa * fmaf(a.s, da, a.u) + fb * fmaf(b.s, db, b.u);
  return r;
}

// The summary of a warp's, in every lane; the sums in the same order in every lane. FAR as in lp_merge: nothing,
// or a NaN, stays what it is where no number is above -inf.
__device__ __forceinline__ LpSum lp_warp_sum(LpSum a) {
  float m = a.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float d = fmaxf(a.m - m, LP_FAR), f = lp_ex2(d * LP_LOG2E);
  float u = f * fmaf(a.s, d, a.u), s = f * a.s;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    u += __shfl_xor_sync(0xffffffffu, u, o);
  }
  return {m, s, u};
}

// How many of the `n` keys at `keys` (n a multiple of 4, shared memory) are better than `key`.
__device__ __forceinline__ int lp_rank(const uint64_t* keys, int n, uint64_t key) {
  int rank = 0;
  for (int i = 0; i < n; i += 4) {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(keys + i), b = *reinterpret_cast<const ulonglong2*>(keys + i + 2);
    rank += (a.x > key) + (a.y > key) + (b.x > key) + (b.y > key);
  }
  return rank;
}

// Pairs of floats: one instruction for two logits.
__device__ __forceinline__ uint64_t lp_pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void lp_unpair(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t lp_add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t lp_mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t lp_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

constexpr int LP_CLUSTER = 8;                  // CTAs per row at most
struct LpShared {
  LpSum warp_sum[LP_WARPS];
  LpSum sum[LP_CLUSTER];                       // (first CTA) the CTAs'
  int chosens, count;                          // how many threads and classes may be listed
  uint64_t round[LP_WARPS];
  uint16_t chosen[LP_THREADS];                 // threads that hold classes to list
  alignas(16) uint64_t top[LP_THREADS];        // (first CTA) the CTAs' classes in order, n each, 0 behind the last
  alignas(16) uint64_t keys[LP_ROOM];
};
static_assert(LP_CLUSTER * KL_LOGPROBS_MAX_TOP <= LP_THREADS, "a thread per listed class");
static_assert(LP_THREADS + KL_LOGPROBS_MAX_TOP <= LP_ROOM, "room for the first equal classes");

// TOP: alternatives are wanted. Four CTAs on an SM have the registers for the next vectors; without alternatives
// five do (2045 x 151936 bf16: 96 us with five, 105 with four, 102 with the eight that come of no bound, whose
// next vectors the compiler does not hold; 64 x 151936 fp32 with 20: 14.8 with four, 17.5 with five, 18.9 with eight).
constexpr int LP_SLOTS = 4;
template <typename T, bool TOP>
__global__ void __launch_bounds__(LP_THREADS, TOP ? LP_SLOTS : LP_SLOTS + 1) token_logprobs_kernel(const __grid_constant__ LpParams p) {
  pdl_wait();
  __shared__ LpShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int CL = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int n = blockIdx.x / CL, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const LpRow<T> row(static_cast<const T*>(p.z) + static_cast<int64_t>(n) * p.ldz, p.V);
  constexpr int NV = LpVec<T>::N;

  if (TOP) sh.top[tid] = 0;
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");   // the first CTA runs and its list is empty
  const int step = CL * LP_THREADS, i0 = rank * LP_THREADS + tid;
  const bool ends = rank == CL - 1;            // this CTA has the row's ends too

  // this thread's summary, over LP_U vectors at a time: one look at the maximum for all of them, the next
  // ones on their way
  LpSum a = {-INFINITY, 0.f, 0.f};
  LpVec<T> next[LP_U];
#pragma unroll
  for (int k = 0; k < LP_U; ++k) next[k] = row.load(i0 + k * step);
  // what the row's end needs, before it is needed
  const int tok = p.tokens[n];
  float ztok = 0.f;
  if (tok >= 0 && tok < p.V) ztok = Elem<T>::to_f(row.z[tok]);
#pragma unroll 1
  for (int i = i0; i < row.vecs; i += LP_U * step) {
    LpVec<T> v[LP_U];
#pragma unroll
    for (int k = 0; k < LP_U; ++k) {
      v[k] = next[k];
      next[k] = row.load(i + (LP_U + k) * step);
    }
    float cm = v[0].max();
#pragma unroll
    for (int k = 1; k < LP_U; ++k) cm = fmaxf(cm, v[k].max());
    if (cm > a.m) {
      const float d = fmaxf(a.m - cm, LP_FAR), f = lp_ex2(d * LP_LOG2E);
      a.u = f * fmaf(a.s, d, a.u);
      a.s *= f;
      a.m = cm;
    }
    // (no number above -inf so far: as from 0, so that a NaN is not lost)
    const float base = a.m == -INFINITY ? 0.f : -a.m;
    const uint64_t neg = lp_pair(base, base), scale = lp_pair(LP_LOG2E, LP_LOG2E);
    uint64_t s2 = 0, u2 = 0;
#pragma unroll
    for (int k = 0; k < LP_U; ++k)
#pragma unroll
      for (int e = 0; e < NV; e += 2) {
        float x0, x1, e0, e1;
        lp_unpair(lp_add2(lp_pair(v[k].get(e), v[k].get(e + 1)), neg), x0, x1);
        const uint64_t x = lp_pair(lp_max_nan(x0, LP_FAR), lp_max_nan(x1, LP_FAR));
        lp_unpair(lp_mul2(x, scale), e0, e1);
        const uint64_t ex = lp_pair(lp_ex2(e0), lp_ex2(e1));
        s2 = lp_add2(s2, ex);
        u2 = lp_fma2(ex, x, u2);
      }
    float s0, s1, u0, u1;
    lp_unpair(s2, s0, s1);
    lp_unpair(u2, u0, u1);
    a.s += s0 + s1;
    a.u += u0 + u1;
  }
  if (ends && tid < row.head + row.tail) {     // a class of the ends each
    const float z = Elem<T>::to_f(row.z[row.end(tid)]);
    a = lp_merge(a, {fmaxf(z, -INFINITY), z == -INFINITY ? 0.f : z - z + 1.f, 0.f});
  }
  pdl_launch_dependents();
  // threads of a warp, warps of the CTA, CTAs of the cluster
  const uint32_t mine = TOP ? lp_order(a.m) : 0;
  a = lp_warp_sum(a);
  if (lane == 0) sh.warp_sum[warp] = a;
  if (tid == 0) sh.chosens = sh.count = 0;
  __syncthreads();
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  LpShared& first = *cluster.map_shared_rank(&sh, 0);
  if (warp == LP_WARPS - 1) {
    const LpSum t = lp_warp_sum(lane < LP_WARPS ? sh.warp_sum[lane] : LpSum{-INFINITY, 0.f, 0.f});
    if (lane == 0) first.sum[rank] = t;
  }
  if (TOP) {
    // the greatest number that at least n threads' maxima reach, bit by bit; one that just n reach will do
    uint32_t lowest = 0;
#pragma unroll 1
    for (uint32_t bit = 1u << 31; bit >= (sizeof(T) == 2 ? 1u << 16 : 1u); bit >>= 1) {
      const int reach = __syncthreads_count(mine >= (lowest | bit));
      if (reach >= p.top) lowest |= bit;
      if (reach == p.top) break;
    }
    if (mine != 0 && mine >= lowest) sh.chosen[atomicAdd(&sh.chosens, 1)] = static_cast<uint16_t>(tid);
    const uint32_t above = lowest + (sizeof(T) == 2 ? 1u << 16 : 1u);        // better ones are at least this
    uint32_t least = lowest;                     // 0 if there are fewer than n: everything passes
    int count;
#pragma unroll 1
    for (;;) {
      const uint64_t last = static_cast<uint64_t>(least) << 32;
      auto list = [&](float z, int j) {
        const uint64_t key = lp_key(z, j);
        if (key == 0 || key < last) return;
        const int at = atomicAdd(&sh.count, 1);
        if (at < LP_ROOM) sh.keys[at] = key;
      };
      __syncthreads();
      // the chosen threads' vectors once more, in quarters, spread over all threads: a trip or two to L2 as a rule
      constexpr int NQ = NV / 4;
      const int chosen = sh.chosens, each = (row.vecs + step - 1) / step;
#pragma unroll 1
      for (int k = tid; k < chosen * each * 4; k += LP_THREADS) {
        const int vec = k >> 2, i = rank * LP_THREADS + sh.chosen[vec % chosen] + vec / chosen * step;
        if (i >= row.vecs) continue;
        const T* q = row.at(i) + (k & 3) * NQ;
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(q));
        const int j = static_cast<int>(q - row.z);
        if (sizeof(T) == 4) {
          list(__uint_as_float(w.x), j);
          list(__uint_as_float(w.y), j + 1);
        } else {
          list(__uint_as_float(w.x << 16), j);
          list(__uint_as_float(w.x & 0xffff0000u), j + 1);
          list(__uint_as_float(w.y << 16), j + 2);
          list(__uint_as_float(w.y & 0xffff0000u), j + 3);
        }
      }
      if (ends && tid < row.head + row.tail) list(Elem<T>::to_f(row.z[row.end(tid)]), row.end(tid));
      __syncthreads();
      count = sh.count;
      if (count <= LP_ROOM || least == above) break;
      least = above;                             // the better ones alone
      __syncthreads();
      if (tid == 0) sh.count = 0;
    }
    if (count <= LP_ROOM) {
      if (tid < 4 && count + tid < ((count + 3) & ~3)) sh.keys[count + tid] = 0;
      __syncthreads();
      for (int i = tid; i < count; i += LP_THREADS) {
        const uint64_t key = sh.keys[i];
        const int r = lp_rank(sh.keys, (count + 3) & ~3, key);
        if (r < p.top) first.top[rank * p.top + r] = key;
      }
      if (least != lowest && count < p.top) {
        // and the first of the equal ones, LP_THREADS classes at a time: the ones before the vectors, the CTA's
        // vectors, the ones behind
        __syncthreads();                         // the keys have been read
        if (tid == 0) sh.count = 0;
        __syncthreads();
        const int blocks = (row.vecs + LP_THREADS - 1) / LP_THREADS;
        int found = 0;
#pragma unroll 1
        for (int b = ends ? -1 : 0; b <= (ends ? blocks * NV : blocks * NV - 1) && found < p.top - count; ++b) {
          int j = row.head + b * LP_THREADS + tid, behind = row.head + row.vecs * NV;
          if (b < 0) j = tid, behind = row.head;
          else if (b == blocks * NV) j = behind + tid, behind = p.V;
          else if (b / NV % CL != rank) continue;
          const uint64_t key = j < behind ? lp_key(Elem<T>::to_f(row.z[j]), j) : 0;
          const uint32_t o = static_cast<uint32_t>(key >> 32);
          if (key && o >= lowest && o < above) sh.keys[atomicAdd(&sh.count, 1)] = key;
          __syncthreads();
          found = sh.count;                      // below n and a thread each more
          __syncthreads();
        }
        if (tid < 4 && found + tid < ((found + 3) & ~3)) sh.keys[found + tid] = 0;
        __syncthreads();
        for (int i = tid; i < found; i += LP_THREADS) {
          const uint64_t key = sh.keys[i];
          const int r = count + lp_rank(sh.keys, (found + 3) & ~3, key);
          if (r < p.top) first.top[rank * p.top + r] = key;
        }
      }
    } else {
      // one after the other, each the best behind the one before
      uint64_t before = ~0ull;
      for (int k = 0; k < p.top; ++k) {
        uint64_t b = 0;
        auto look = [&](int j) {
          const uint64_t key = lp_key(Elem<T>::to_f(row.z[j]), j);
          if (key < before && key > b) b = key;
        };
#pragma unroll 1
        for (int i = i0; i < row.vecs; i += step)
#pragma unroll 1
          for (int e = 0; e < NV; ++e) look(row.head + i * NV + e);
        if (ends && tid < row.head + row.tail) look(row.end(tid));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const uint64_t c = __shfl_xor_sync(0xffffffffu, b, o);
          b = c > b ? c : b;
        }
        __syncthreads();
        if (lane == 0) sh.round[warp] = b;
        __syncthreads();
        for (int w = 0; w < LP_WARPS; ++w) b = sh.round[w] > b ? sh.round[w] : b;
        before = b;
        if (tid == 0) first.top[rank * p.top + k] = b;
        if (b == 0) break;
      }
    }
  }
  cluster.sync();
  if (rank == 0) {
    const LpSum t = lp_warp_sum(lane < CL ? sh.sum[lane] : LpSum{-INFINITY, 0.f, 0.f});
    const bool empty = t.m == -INFINITY && t.s == 0.f;
    const float ls = empty ? -INFINITY : logf(t.s);
    if (tid == 0) {
      float lp = 0.f;
      if (tok >= 0 && tok < p.V) lp = empty ? -INFINITY : ztok - t.m - ls;
      else if (tok != -1) record_error(p.err, KL_DEVERR_TARGET);
      p.logprob[n] = lp;
      if (p.entropy) p.entropy[n] = empty ? 0.f : ls - t.u / t.s;
      if (p.norm) {
        p.norm[2 * static_cast<int64_t>(n)] = t.m;
        p.norm[2 * static_cast<int64_t>(n) + 1] = ls;
      }
    }
    if (TOP) {
      // the CTAs' lists in one order, a thread per class
      const int all = CL * p.top;
      const uint64_t key = sh.top[tid];
      const int have = __syncthreads_count(key != 0);
      int32_t* id = p.top_id + static_cast<int64_t>(n) * p.top;
      float* out = p.top_lp + static_cast<int64_t>(n) * p.top;
      if (key) {
        const int r = lp_rank(sh.top, (all + 3) & ~3, key);
        if (r < p.top) {
          id[r] = lp_class(key);
          out[r] = lp_logit(key) - t.m - ls;
        }
      }
      if (tid < p.top && tid >= have) {        // no class is left
        id[tid] = -1;
        out[tid] = -INFINITY;
      }
    }
  }
}

struct LpBwdParams {
  const void* z;
  int64_t ldz;
  const int32_t* tokens;
  const float* norm;
  const float* entropy;
  const float* dlp;
  const float* dent;
  void* dz;
  int64_t lddz;
  int N, V, parts;
  uint32_t* err;
};

// Backward: one read and one write of a part of a row, bound by HBM. Vectors of eight classes, aligned in z;
// where dz's lie as z's do they are written whole, else (rows of other strides or types whose alignment
// differs) class by class.
constexpr int LB_U = 4;                        // vectors a thread has under way
constexpr float LB_FAR = -1e4f;                // as LP_FAR: p is 0, and the entropy's weight times this is finite (up to 3e34)
constexpr int LB_PART = LP_THREADS * 8 * LB_U; // classes a CTA takes

template <typename T, typename U>
__global__ void __launch_bounds__(LP_THREADS) token_logprobs_bwd_kernel(const __grid_constant__ LpBwdParams p) {
  pdl_enter();
  const int n = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
  const T* z = static_cast<const T*>(p.z) + static_cast<int64_t>(n) * p.ldz;
  U* dz = static_cast<U*>(p.dz) + static_cast<int64_t>(n) * p.lddz;
  const float m = p.norm[2 * static_cast<int64_t>(n)], ls = p.norm[2 * static_cast<int64_t>(n) + 1];
  int t = p.tokens[n];
  if (t < -1 || t >= p.V) {
    if (threadIdx.x == 0 && part == 0) record_error(p.err, KL_DEVERR_TARGET);
    t = -1;
  }
  const float a = t >= 0 && p.dlp ? p.dlp[n] : 0.f, b = p.dent ? p.dent[n] : 0.f, H = p.dent ? p.entropy[n] : 0.f;
  // zeros: no logit above -inf, or no weight, whatever the logits are (padding may hold NaN)
  const bool none = (m == -INFINITY && ls == -INFINITY) || (a == 0.f && b == 0.f);
  auto grad = [&](float zj, int j) {
    const float x = lp_max_nan(zj - m - ls, LB_FAR), q = lp_ex2(x * LP_LOG2E);
    float d = -q * fmaf(b, x + H, a);
    if (j == t) d += a;
    return none ? 0.f : d;
  };
  constexpr int ZA = 8 * sizeof(T), DA = 8 * sizeof(U);         // bytes of a vector
  const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(z) & (ZA - 1)) / sizeof(T));
  const bool both = lead == static_cast<int>((reinterpret_cast<uintptr_t>(dz) & (DA - 1)) / sizeof(U));
  if (!both) {
    for (int j = part * LB_PART + threadIdx.x; j < min(p.V, (part + 1) * LB_PART); j += LP_THREADS)
      dz[j] = Elem<U>::from_f(grad(Elem<T>::to_f(z[j]), j));
    return;
  }
  uint32_t v[LB_U][ZA / 4];
  const int j0 = part * LB_PART + threadIdx.x * 8 - lead;
  auto whole = [&](int j) { return j >= 0 && j + 8 <= p.V; };
#pragma unroll
  for (int k = 0; k < LB_U; ++k) {
    const int j = j0 + k * LP_THREADS * 8;
    if (!whole(j)) continue;
    if (sizeof(T) == 4)
      asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(v[k][0]), "=r"(v[k][1]), "=r"(v[k][2]), "=r"(v[k][3]), "=r"(v[k][4 % (ZA / 4)]), "=r"(v[k][5 % (ZA / 4)]),
                     "=r"(v[k][6 % (ZA / 4)]), "=r"(v[k][7 % (ZA / 4)])
                   : "l"(z + j));
    else
      asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v[k][0]), "=r"(v[k][1]), "=r"(v[k][2]), "=r"(v[k][3])
                   : "l"(z + j));
  }
#pragma unroll
  for (int k = 0; k < LB_U; ++k) {
    const int j = j0 + k * LP_THREADS * 8;
    if (!whole(j)) {                           // an end of the row, or behind it
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j + e >= 0 && j + e < p.V) dz[j + e] = Elem<U>::from_f(grad(Elem<T>::to_f(z[j + e]), j + e));
      continue;
    }
    float g[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t w = sizeof(T) == 4 ? v[k][e % (ZA / 4)] : e & 1 ? v[k][e >> 1] & 0xffff0000u : v[k][e >> 1] << 16;
      g[e] = grad(__uint_as_float(w), j + e);
    }
    if (sizeof(U) == 4)
      asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dz + j), "f"(g[0]), "f"(g[1]),
                   "f"(g[2]), "f"(g[3]), "f"(g[4]), "f"(g[5]), "f"(g[6]), "f"(g[7])
                   : "memory");
    else
      asm volatile("st.global.L1::no_allocate.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(dz + j), "r"(pack_bf16x2(g[0], g[1])),
                   "r"(pack_bf16x2(g[2], g[3])), "r"(pack_bf16x2(g[4], g[5])), "r"(pack_bf16x2(g[6], g[7]))
                   : "memory");
  }
}

template <typename... A, typename... B>
kl_status launch_cluster(void (*kern)(A...), int grid, int cluster, cudaStream_t st, B&&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(LP_THREADS);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  KL_CUDA(cudaLaunchKernelEx(&cfg, kern, args...));
  return KL_OK;
}

}  // namespace

kl_status token_logprobs(int N, int V, int dtype, const void* z, int64_t ldz, const int32_t* tokens, int n_top,
                         float* logprob, float* entropy, float* norm, int32_t* top_id, float* top_logprob,
                         cudaStream_t st) {
  const LpParams p = {z, ldz, tokens, logprob, entropy, norm, top_id, top_logprob, N, V, n_top, device_error_word()};
  // CTAs per row: as many as run at once, each with a vector for every thread at least (301 x 32001: 12 us with
  // two, 17 with four, of which a part waits; 64 x 151936: 15 with eight, 21 where only three run on an SM)
  const int per = LP_THREADS * 32 / static_cast<int>(dtype_size(dtype));
  int cl = 1;
  while (cl < LP_CLUSTER && 2 * static_cast<int64_t>(N) * cl <= LP_SLOTS * num_sms() && static_cast<int64_t>(cl) * per < V) cl *= 2;
  ProfScope ps("token_logprobs", st, 0.0, static_cast<double>(N) * V * dtype_size(dtype));
  if (dtype == KL_F32)
    return n_top ? launch_cluster(token_logprobs_kernel<float, true>, N * cl, cl, st, p)
                 : launch_cluster(token_logprobs_kernel<float, false>, N * cl, cl, st, p);
  return n_top ? launch_cluster(token_logprobs_kernel<__nv_bfloat16, true>, N * cl, cl, st, p)
               : launch_cluster(token_logprobs_kernel<__nv_bfloat16, false>, N * cl, cl, st, p);
}

kl_status token_logprobs_bwd(int N, int V, int dtype, const void* z, int64_t ldz, const int32_t* tokens,
                             const float* norm, const float* entropy, const float* dlp, const float* dent, int dz_dtype,
                             void* dz, int64_t lddz, cudaStream_t st) {
  const int parts = (V + 7 + LB_PART - 1) / LB_PART;       // up to seven classes less in the first vector
  const int64_t grid = static_cast<int64_t>(N) * parts;
  if (grid > 2147483647LL) return set_error(KL_ERR_UNSUPPORTED, "token_logprobs_bwd: %d rows of %d classes", N, V);
  const LpBwdParams p = {z, ldz, tokens, norm, entropy, dlp, dent, dz, lddz, N, V, parts, device_error_word()};
  ProfScope ps("token_logprobs_bwd", st, 0.0, static_cast<double>(N) * V * (dtype_size(dtype) + dtype_size(dz_dtype)));
  const int g = static_cast<int>(grid);
  if (dtype == KL_F32 && dz_dtype == KL_F32) launch_pdl(token_logprobs_bwd_kernel<float, float>, g, LP_THREADS, 0, st, p);
  else if (dtype == KL_F32) launch_pdl(token_logprobs_bwd_kernel<float, __nv_bfloat16>, g, LP_THREADS, 0, st, p);
  else if (dz_dtype == KL_F32) launch_pdl(token_logprobs_bwd_kernel<__nv_bfloat16, float>, g, LP_THREADS, 0, st, p);
  else launch_pdl(token_logprobs_bwd_kernel<__nv_bfloat16, __nv_bfloat16>, g, LP_THREADS, 0, st, p);
  KL_CUDA(cudaGetLastError());
  return KL_OK;
}

}  // namespace kl
