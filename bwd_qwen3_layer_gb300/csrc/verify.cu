// Drafted tokens judged by the target's probabilities (speculative decoding's
// accept-or-resample rule, from given random numbers):
//   draft t of row r is accepted iff u_r q_r(t) < p_r(t);
//   at the first rejection the next token is drawn from max(0, p_r - q_r), after
//   the last accepted draft from p: the smallest index i with
//   C_i = sum_{j <= i} w_j > u sum_j w_j.
//
// Only one row of p (and q) per request is read whole: V x 4 B each, bound by
// HBM for many requests and by latency for one. A cluster of 8 or 16 CTAs takes
// one request: each finds the row itself (at most a few gathers), sums its share
// of the weights, the sums meet in distributed shared memory, and the CTA in whose
// range the cumulative sum crosses u x total looks for the place: its warps' sums
// name a stretch of about a thousand weights, which the CTA sums once more (from
// L2), one vector per lane.
//
// An index must not depend on how a sum is split, so sums are held far beyond
// the weights' own precision: p - q as an error-free pair of floats (two-sum,
// Knuth), sums, prefix sums and comparisons in such pairs, a lane's running sum in
// three floats. The error of a sum, relative to it, whatever V is: a lane's 4 to 32
// elements are added as a tree of at most 5 levels, whose roundings (each at most
// 2^-24 of itself) come to 30 x 2^-48 at most; joining such groups loses below
// 2^-60 of them; the joins of lanes, warps and CTAs are 16 additions of pairs, 2^-46
// each. Below 2^-41 in all, some 2^-47 as a rule. fp64
// is slow on this part (an addition takes 63 cycles, an SM starts two a cycle):
// with every thread's sums in it 64 requests of 151936 classes took 82 us, with
// the warps' prefix sums alone 26, without it 19 (rows in L2; 21.4 where they are
// not). The acceptance test is exact: the product of two floats fits a double.
#include "internal.h"
#include "kl_common.cuh"

namespace kl {
namespace {

// CTAs per request (one cluster) and warps per CTA, by how many clusters are
// resident together (V = 151936, p and q in fp32 and in L2; rows that are not in it
// after the stroke):
//   up to 7 requests   16 CTAs of 16 warps, an SM each: one 7.1 us / 6.9, seven 7.3 /
//                      9.2; eight CTAs for one 8.1; from 8 requests on they take two
//                      rounds (8: 11.3)
//   up to 14           8 of 16 warps: 8.5 to 8.6 us / 10.8 to 11.3, 8 of 8 warps 9.8
//                      to 11.3; 16 requests take two rounds (12.5)
//   more               8 of 8 warps, four CTAs per SM: 16 requests 11.1 us / 14.8, 64
//                      19.2 / 21.4, 128 34 / 35.5
// With 5000 classes all splits lie close: 5.8 to 6.3 us for 1 to 16 requests in fp32
// (6.5 to 6.9 in bf16), 7.2 for 64.
constexpr int DV_CL = 8, DV_CL_FEW = 16;
constexpr int DV_WARPS_MANY = 8, DV_WARPS_FEW = 16;
constexpr int DV_FEW = 7, DV_SOME = 14;

struct VerifyParams {
  const void* p;
  const void* q;
  int64_t ldp, ldq;
  const int32_t* tokens;
  const int32_t* cu;
  const float* ua;
  const float* us;
  int32_t* acc;
  int32_t* next;
  int B, T, V;
  uint32_t* err;
};

template <typename T>
__device__ __forceinline__ float dv_ld(const void* base, int64_t i) {
  return Elem<T>::to_f(static_cast<const T*>(base)[i]);
}

// E elements (one, or a 16-byte vector), all of them in the row.
template <typename T, int E>
__device__ __forceinline__ void dv_load_whole(const T* x, float (&f)[E]) {
  if constexpr (E == 1) {
    f[0] = Elem<T>::to_f(*x);
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(x));
    if constexpr (sizeof(T) == 4) {
      f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y);
      f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
    } else {
      const float2 x0 = unpack_bf16x2(a.x), x1 = unpack_bf16x2(a.y), x2 = unpack_bf16x2(a.z), x3 = unpack_bf16x2(a.w);
      f[0] = x0.x; f[1] = x0.y; f[2] = x1.x; f[3] = x1.y;
      f[4] = x2.x; f[5] = x2.y; f[6] = x3.x; f[7] = x3.y;
    }
  }
}
// E elements of a row starting at column i: columns outside [0, V) give zero.
template <typename T, int E>
__device__ __forceinline__ void dv_load(const T* row, int64_t i, int V, float (&f)[E]) {
  if (i >= 0 && i + E <= V) {
    dv_load_whole<T, E>(row + i, f);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = i + e >= 0 && i + e < V ? Elem<T>::to_f(row[i + e]) : 0.f;
  }
}

// A number as an unevaluated pair of floats, hi + lo (about 48 bits).
struct Pair {
  float hi, lo;
};
// a + b, and its rounding error
__device__ __forceinline__ Pair dv_two_sum(float a, float b) {
  const float s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Pair dv_norm(Pair v) {   // |lo| at most half a step of hi
  const float s = v.hi + v.lo;
  return {s, v.lo - (s - v.hi)};
}
__device__ __forceinline__ Pair dv_join(Pair a, Pair b) {   // not normed
  const Pair s = dv_two_sum(a.hi, b.hi);
  return {s.hi, s.lo + (a.lo + b.lo)};
}
__device__ __forceinline__ Pair dv_plus(Pair a, Pair b) { return dv_norm(dv_join(a, b)); }
// The sum of N pairs (N a power of two) as a tree: an error that is added up one by
// one grows with the square of their number, one of a tree with that of its levels.
template <int N>
__device__ __forceinline__ Pair dv_tree(const Pair (&v)[N]) {
  if constexpr (N == 1) {
    return v[0];
  } else {
    Pair half[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) half[i] = dv_join(v[2 * i], v[2 * i + 1]);
    return dv_tree<N / 2>(half);
  }
}
// A running sum of pairs: the errors' sum has an error term of its own, so that its
// precision does not depend on how many are added.
struct Sum {
  float hi = 0.f, lo = 0.f, rest = 0.f;
  __device__ __forceinline__ void add(Pair v) {
    const Pair a = dv_two_sum(hi, v.hi), b = dv_two_sum(lo, a.lo), c = dv_two_sum(b.hi, v.lo);
    hi = a.hi;
    lo = c.hi;
    rest += b.lo + c.lo;
  }
  __device__ __forceinline__ Pair value() const {
    const Pair s = dv_norm({hi, lo});
    return dv_norm({s.hi, s.lo + rest});
  }
};
// a > b for normed pairs: where the leading parts are close their difference is
// exact, and where they are not it decides.
__device__ __forceinline__ bool dv_above(Pair a, Pair b) { return (a.hi - b.hi) + (a.lo - b.lo) > 0.f; }
__device__ __forceinline__ Pair dv_times(float u, Pair a) {
  const float p = __fmul_rn(u, a.hi);
  return dv_norm({p, fmaf(u, a.hi, -p) + u * a.lo});
}
__device__ __forceinline__ Pair dv_shfl(Pair v, int lane) {
  return {__shfl_sync(0xffffffffu, v.hi, lane), __shfl_sync(0xffffffffu, v.lo, lane)};
}
// The sum of the warp's 32 pairs, in every lane.
__device__ __forceinline__ Pair dv_warp_sum(Pair v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = dv_plus(v, {__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
  return v;
}
// Inclusive prefix sums over the first N lanes of a warp (N a power of two).
template <int N>
__device__ __forceinline__ Pair dv_warp_scan(Pair v, int lane) {
#pragma unroll
  for (int o = 1; o < N; o <<= 1) {
    const Pair x = {__shfl_up_sync(0xffffffffu, v.hi, o), __shfl_up_sync(0xffffffffu, v.lo, o)};
    if (lane >= o) v = dv_plus(x, v);
  }
  return v;
}

// Which weights a request's token is drawn from.
enum { DV_P = 0, DV_REST = 1, DV_REST_LOOKUP = 2 };   // p; max(0, p - q); p without the draft

// The weight p - q (or p) as an error-free pair; zero where it is not positive.
__device__ __forceinline__ void dv_weight(int kind, float p, float q, int64_t col, int draft, float& w, float& we) {
  w = p;
  we = 0.f;
  if (kind == DV_REST) {
    w = p - q;
    const float b = w - p;
    we = (p - (w - b)) - (q + b);
  } else if (kind == DV_REST_LOOKUP && col == draft) {
    w = 0.f;
  }
  if (!(w > 0.f)) w = we = 0.f;
}

// The two halves of a cluster-wide barrier: shared memory of another CTA may be
// written once that CTA runs, so every CTA arrives at its start and waits just
// before its first such write.
__device__ __forceinline__ void dv_cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void dv_cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void st_cluster_pair(uint32_t addr, Pair v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.hi), "f"(v.lo) : "memory");
}

// One warp: lane i holds the sum s of part i (zero where there is none) and the sum
// incl of the parts up to it. The part whose cumulative sum crosses x: the first i with
// before + incl_i > x; if rounding leaves none, the last one with a positive sum;
// -1 if there is none. `before` becomes the sum in front of it.
__device__ __forceinline__ int dv_cross(Pair s, Pair incl, int lane, Pair x, Pair& before) {
  const Pair up = dv_plus(before, incl);
  const unsigned some = __ballot_sync(0xffffffffu, s.hi > 0.f);
  const unsigned over = __ballot_sync(0xffffffffu, s.hi > 0.f && dv_above(up, x));
  if (!some) return -1;
  const int i = over ? __ffs(over) - 1 : 31 - __clz(some);
  if (i > 0) before = dv_plus(before, dv_shfl(incl, i - 1));
  return i;
}

// What the first warp tells the others: the part to look into (below 0: none),
// the sum in front of it and the value to cross.
struct VerifySmem {
  Pair slots[2][DV_CL_FEW];          // the CTAs' sums, written by each of them (one array per attempt)
  Pair parts[32];                // the warps' sums
  Pair before, x;
  int part, accepted, kind;
};

// A row (and the draft's): where it starts, its first column's place in a vector.
template <typename T>
struct DvRow {
  const T* p;
  const T* q;
  int mis, V, draft;
};

template <typename T, int E, int KIND>
__device__ __forceinline__ Pair dv_vector(const DvRow<T>& r, int64_t col, const float (&fp)[E], const float (&fq)[E]) {
  Pair v[E];
#pragma unroll
  for (int e = 0; e < E; ++e) dv_weight(KIND, fp[e], fq[e], col + e, r.draft, v[e].hi, v[e].lo);
  return dv_tree<E>(v);
}

// Sum of the warp's vectors j0 .. j1 - 1, lane by lane: the whole ones four at a
// time, the row's first and last one, which columns outside it may share, apart.
template <typename T, int E, int KIND>
__device__ __forceinline__ Pair dv_sum_kind(const DvRow<T>& r, int j0, int j1) {
  constexpr int U = 4;
  const int lane = threadIdx.x & 31;
  const int lo = max(j0, r.mis ? 1 : 0);
  const int hi = min(j1, static_cast<int>((static_cast<int64_t>(r.V) + r.mis) / E));
  Sum sum;
  auto one = [&](int j) {
    const int64_t col = static_cast<int64_t>(j) * E - r.mis;
    float fp[E], fq[E] = {};
    dv_load<T, E>(r.p, col, r.V, fp);
    if (KIND == DV_REST) dv_load<T, E>(r.q, col, r.V, fq);
    sum.add(dv_vector<T, E, KIND>(r, col, fp, fq));
  };
  int j = lo + lane;
  for (; j + 32 * (U - 1) < hi; j += 32 * U) {
    float fp[U][E], fq[U][E] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t col = static_cast<int64_t>(j + 32 * u) * E - r.mis;
      dv_load_whole<T, E>(r.p + col, fp[u]);
      if (KIND == DV_REST) dv_load_whole<T, E>(r.q + col, fq[u]);
    }
    Pair v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = dv_vector<T, E, KIND>(r, static_cast<int64_t>(j + 32 * u) * E - r.mis, fp[u], fq[u]);
    sum.add(dv_tree<U>(v));
  }
  for (; j < hi; j += 32) one(j);
  if (lane == 0 && j0 < lo && j0 < j1) one(j0);
  if (lane == 31 && j1 > hi && j1 - 1 >= lo) one(j1 - 1);
  return dv_warp_sum(sum.value());
}
template <typename T, int E>
__device__ __forceinline__ Pair dv_sum(const DvRow<T>& r, int kind, int j0, int j1) {
  if (kind == DV_REST) return dv_sum_kind<T, E, DV_REST>(r, j0, j1);
  if (kind == DV_REST_LOOKUP) return dv_sum_kind<T, E, DV_REST_LOOKUP>(r, j0, j1);
  return dv_sum_kind<T, E, DV_P>(r, j0, j1);
}

template <typename T, int E, int WARPS, int CL>
__device__ __forceinline__ void dv_request(const VerifyParams& p, VerifySmem& s, int b, int rank, const DvRow<T>& row, int kind,
                                           int accepted) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // columns in vectors of E: vector j holds columns E j - mis ..
  const int nv = static_cast<int>((static_cast<int64_t>(p.V) + row.mis + E - 1) / E);
  const int per_cta = (nv + CL - 1) / CL;
  const int per_warp = (per_cta + WARPS - 1) / WARPS;
  const int c0 = min(nv, rank * per_cta), c1 = min(nv, c0 + per_cta);
  const int w0 = min(c1, c0 + warp * per_warp), w1 = min(c1, w0 + per_warp);
  const float u = p.us[b];

  for (int attempt = 0; attempt < 2; ++attempt) {
    const Pair sum = dv_sum<T, E>(row, kind, w0, w1);
    if (lane == 0) s.parts[warp] = sum;
    if (attempt == 0) dv_cluster_wait();
    __syncthreads();
    Pair mine = {0.f, 0.f}, upto = mine;
    if (warp == 0) {
      if (lane < WARPS) mine = s.parts[lane];
      upto = dv_warp_scan<WARPS>(mine, lane);
      const Pair cta = dv_shfl(upto, WARPS - 1);
      if (lane < CL) st_cluster_pair(mapa_shared(smem_u32(&s.slots[attempt][rank]), lane), cta);
    }
    cluster_sync_all();
    if (warp == 0) {
      Pair part = {0.f, 0.f}, before = part;
      if (lane < CL) part = s.slots[attempt][lane];
      const Pair incl = dv_warp_scan<CL>(part, lane);
      const Pair total = dv_shfl(incl, CL - 1);
      const Pair x = dv_times(u, total);
      int next = kind;
      int owner = total.hi > 0.f && total.hi < INFINITY ? dv_cross(part, incl, lane, x, before) : -1;
      if (owner < 0 && attempt == 0 && kind != DV_P && !(total.hi > 0.f)) {
        next = -1;                                   // nothing left of p - q anywhere: p itself
      } else if (owner < 0) {
        if (rank == 0 && lane == 0) {
          p.acc[b] = accepted;
          p.next[b] = -1;
        }
      } else if (owner == rank) {
        owner = max(0, dv_cross(mine, upto, lane, x, before));
        if (lane == 0) {
          s.before = before;
          s.x = x;
        }
      } else {
        owner = -1;
      }
      if (lane == 0) {
        s.part = owner;
        s.kind = next;
      }
    }
    __syncthreads();
    if (s.kind < 0) {
      kind = DV_P;
      continue;
    }
    const int ow = s.part;
    if (ow < 0) return;
    // that warp's stretch once more, spread over the CTA: warp w takes its w-th part
    const int s0 = min(c1, c0 + ow * per_warp), s1 = min(c1, s0 + per_warp);
    const int piece = (s1 - s0 + WARPS - 1) / WARPS;
    const int p0 = min(s1, s0 + warp * piece), p1 = min(s1, p0 + piece);
    const Pair again = dv_sum<T, E>(row, kind, p0, p1);
    if (lane == 0) s.parts[warp] = again;
    __syncthreads();
    const Pair x = s.x;
    Pair front = s.before;
    const Pair stretch = lane < WARPS ? s.parts[lane] : Pair{0.f, 0.f};
    const int pw = max(0, dv_cross(stretch, dv_warp_scan<WARPS>(stretch, lane), lane, x, front));
    if (warp != pw) return;
    // this warp's piece in order, 32 vectors at a time
    int64_t found = -1, last = -1;
    Sum upto_here;
    upto_here.add(front);
    for (int j0 = p0; j0 < p1 && found < 0; j0 += 32) {
      const int j = j0 + lane;
      const int64_t col = static_cast<int64_t>(j) * E - row.mis;
      Pair w[E];
#pragma unroll
      for (int e = 0; e < E; ++e) w[e] = {0.f, 0.f};
      if (j < p1) {
        float fp[E], fq[E] = {};
        dv_load<T, E>(row.p, col, p.V, fp);
        if (kind == DV_REST) dv_load<T, E>(row.q, col, p.V, fq);
#pragma unroll
        for (int e = 0; e < E; ++e) dv_weight(kind, fp[e], fq[e], col + e, row.draft, w[e].hi, w[e].lo);
      }
      const Pair incl = dv_warp_scan<32>(dv_norm(dv_tree<E>(w)), lane), before = upto_here.value();
      Pair at = {__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
      at = lane ? dv_plus(before, at) : before;      // everything in front of this lane's vector
      int64_t hit = -1, pos = -1;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        at = dv_plus(at, w[e]);
        if (w[e].hi > 0.f) {
          pos = col + e;
          if (hit < 0 && dv_above(at, x)) hit = col + e;
        }
      }
      const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0), any = __ballot_sync(0xffffffffu, pos >= 0);
      if (hits) found = __shfl_sync(0xffffffffu, hit, __ffs(hits) - 1);
      if (any) last = __shfl_sync(0xffffffffu, pos, 31 - __clz(any));
      upto_here.add(dv_shfl(incl, 31));
    }
    if (lane == 0) {
      p.acc[b] = accepted;
      p.next[b] = static_cast<int32_t>(found >= 0 ? found : last);   // rounding at the very end: the last positive weight
    }
    return;
  }
}

template <typename T, int WARPS, int CL>
__global__ void __launch_bounds__(32 * WARPS, WARPS == DV_WARPS_MANY ? 4 : 1) draft_verify_kernel(const VerifyParams p) {
  pdl_enter();
  __shared__ VerifySmem s;
  const int b = blockIdx.x / CL, rank = static_cast<int>(cluster_ctarank());
  const int r0 = min(max(p.cu[b], 0), p.T), r1 = min(max(p.cu[b + 1], r0), p.T);
  if (r1 <= r0) {                       // the whole cluster leaves here
    if (rank == 0 && threadIdx.x == 0) {
      p.acc[b] = 0;
      p.next[b] = -1;
    }
    return;
  }
  dv_cluster_arrive();
  if (threadIdx.x < 32) {
    // the first draft that is not accepted, 32 at a time
    int acc = r1 - 1 - r0;
    for (int i0 = 0; i0 < r1 - 1 - r0; i0 += 32) {
      const int i = i0 + static_cast<int>(threadIdx.x);
      bool no = false;
      if (i < r1 - 1 - r0) {
        const int64_t row = r0 + i;
        const int t = p.tokens[row + 1];
        no = true;
        if (t >= 0 && t < p.V) {
          const double pt = dv_ld<T>(p.p, row * p.ldp + t);
          const double qt = p.q ? dv_ld<T>(p.q, row * p.ldq + t) : 1.f;
          no = !(static_cast<double>(p.ua[row]) * qt < pt);
        } else if (rank == 0) {
          record_error(p.err, KL_DEVERR_TARGET);
        }
      }
      const unsigned m = __ballot_sync(0xffffffffu, no);
      if (m) {
        acc = i0 + __ffs(m) - 1;
        break;
      }
    }
    if (threadIdx.x == 0) s.accepted = acc;
  }
  __syncthreads();
  const int accepted = s.accepted;
  const int64_t row = r0 + accepted;
  const bool rejected = row < r1 - 1;
  const int kind = !rejected ? DV_P : p.q ? DV_REST : DV_REST_LOOKUP;
  const int draft = rejected ? p.tokens[row + 1] : -1;
  DvRow<T> w;
  w.p = static_cast<const T*>(p.p) + row * p.ldp;
  w.q = kind == DV_REST ? static_cast<const T*>(p.q) + row * p.ldq : nullptr;
  w.V = p.V;
  w.draft = draft;
  constexpr int E = 16 / sizeof(T);
  // 16-byte vectors where both rows start at the same place of one (a row of an
  // odd vocabulary starts anywhere); element by element where they do not
  w.mis = static_cast<int>((reinterpret_cast<uintptr_t>(w.p) & 15u) / sizeof(T));
  if (!w.q || w.mis == static_cast<int>((reinterpret_cast<uintptr_t>(w.q) & 15u) / sizeof(T))) {
    dv_request<T, E, WARPS, CL>(p, s, b, rank, w, kind, accepted);
  } else {
    w.mis = 0;
    dv_request<T, 1, WARPS, CL>(p, s, b, rank, w, kind, accepted);
  }
}

}  // namespace

kl_status draft_verify(const kl_verify_cfg& c, const void* p, int64_t ldp, const void* q, int64_t ldq,
                       const int32_t* tokens, const int32_t* cu, const float* ua, const float* us, int32_t* acc,
                       int32_t* next, cudaStream_t st) {
  VerifyParams v = {p, q, ldp, ldq, tokens, cu, ua, us, acc, next, c.B, c.T, c.V, device_error_word()};
  using Kernel = void (*)(VerifyParams);
  const bool f32 = c.dtype == KL_F32, few = c.B <= DV_FEW, some = c.B <= DV_SOME;
  Kernel k;
  if (few)
    k = f32 ? Kernel(draft_verify_kernel<float, DV_WARPS_FEW, DV_CL_FEW>) : Kernel(draft_verify_kernel<__nv_bfloat16, DV_WARPS_FEW, DV_CL_FEW>);
  else if (some)
    k = f32 ? Kernel(draft_verify_kernel<float, DV_WARPS_FEW, DV_CL>) : Kernel(draft_verify_kernel<__nv_bfloat16, DV_WARPS_FEW, DV_CL>);
  else
    k = f32 ? Kernel(draft_verify_kernel<float, DV_WARPS_MANY, DV_CL>) : Kernel(draft_verify_kernel<__nv_bfloat16, DV_WARPS_MANY, DV_CL>);
  const int cl = few ? DV_CL_FEW : DV_CL;
  // 16 CTAs are above the portable size; set at every call, as the device may differ
  if (few) KL_CUDA(cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cl;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c.B * cl);
  cfg.blockDim = dim3(32 * (some ? DV_WARPS_FEW : DV_WARPS_MANY));
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const double es = static_cast<double>(dtype_size(c.dtype));
  ProfScope ps("draft_verify", st, 0.0, static_cast<double>(c.B) * c.V * es * (q ? 2 : 1));
  KL_CUDA(cudaLaunchKernelEx(&cfg, k, v));
  return KL_OK;
}

}  // namespace kl
