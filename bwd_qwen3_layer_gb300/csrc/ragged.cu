// What surrounds the attention of a ragged step over the paged cache: the step's
// block tables, positions and slots from the requests' lengths, and the new
// tokens' rotation with the cache write.
//
//   ragged_plan_kernel  one cluster. Every CTA scans the requests itself (rows,
//                       blocks wanted and given back, 1024 requests at a time,
//                       the prefix sums in its shared memory) and takes its share
//                       of the rows, of the new table entries and, after a cluster
//                       barrier, when nobody reads the list any more, of the
//                       blocks given back; the first CTA updates the counts.
//                       Few requests are bound by latency, three dependent reads
//                       and a scan (64 decoding requests 5.5 us); many rows and
//                       blocks by a search of the prefix sums for each of them (700
//                       requests of 41,893 rows with 2,631 blocks taken and 17,271
//                       given back: 14.8 us, the state restored before each call).
//   ragged_qkv_kernel   one CTA per row: all its q, k and v heads, 16 bytes a
//                       thread and plane half, the row's 64 (cos, sin) pairs
//                       formed once in shared memory while the heads are on
//                       their way. Bound by HBM.
#include "internal.h"
#include "kl_common.cuh"
#include "rope.cuh"

namespace kl {
namespace {

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
constexpr int RP_THREADS = 1024;
constexpr int RP_WARPS = RP_THREADS / 32;
// CTAs of the cluster: eight (the portable most) where the rows or the requests
// would keep one busy for long, else one.
constexpr int RP_CLUSTER = 8;
constexpr int RP_ONE_CTA_ROWS = 4096;

constexpr long long RP_PAST = 1LL << 30;     // no table row reaches this position
struct PlanParams {
  const int32_t* n_new;
  const int32_t* ctx;
  int32_t* table;
  int32_t* held;
  int32_t* free_list;
  int32_t* n_free;
  int32_t* cu;
  int32_t* pos;
  int32_t* slots;
  int32_t* missing;
  int B, T, bs, max_blocks, n_blocks;
  uint32_t* err;
};

// What one request asks for.
struct PlanReq {
  int n;       // rows
  int ctx, held, want;
  int take;    // blocks it lacks
  int back;    // blocks it gives back
};
__device__ __forceinline__ PlanReq plan_req(const PlanParams& p, int b) {
  PlanReq r = {0, 0, 0, 0, 0, 0};
  if (b >= p.B) return r;
  const int n = p.n_new[b];
  r.ctx = max(p.ctx[b], 0);
  r.held = min(max(p.held[b], 0), p.max_blocks);
  r.n = max(n, 0);
  // in 32 bits unsigned, where ctx + n fits: a division of 64 takes 0.3 us
  if (n > 0) r.want = static_cast<int>(min((static_cast<uint32_t>(r.ctx) + n - 1) / p.bs + 1, static_cast<uint32_t>(p.max_blocks)));
  r.take = max(r.want - r.held, 0);
  r.back = n < 0 ? r.held : 0;
  return r;
}

struct PlanSmem {
  long long sums[3][RP_WARPS], most[RP_WARPS];
  // the chunk's requests: exclusive prefix sums within the chunk and their lengths
  long long row[RP_THREADS + 1], take[RP_THREADS + 1], back[RP_THREADS];
  int ctx[RP_THREADS], held[RP_THREADS], want[RP_THREADS];
};

// Exclusive prefix sums of three values per thread over the CTA; totals in t.
__device__ void plan_scan(PlanSmem& s, long long (&v)[3], long long (&t)[3]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long incl[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    incl[k] = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl[k], o);
      if (lane >= o) incl[k] += x;
    }
  }
  __syncthreads();                                  // the previous chunk is done with the sums and the lists
  if (lane == 31)
#pragma unroll
    for (int k = 0; k < 3; ++k) s.sums[k][warp] = incl[k];
  __syncthreads();
  if (warp < 3) {
    const long long mine = s.sums[warp][lane];
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    s.sums[warp][lane] = x;                         // inclusive over the warps
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    t[k] = s.sums[k][RP_WARPS - 1];
    v[k] = incl[k] - v[k] + (warp ? s.sums[k][warp - 1] : 0);
  }
}

// The last i in [0, n) with list[i] <= x (list[0] <= x).
template <typename T>
__device__ __forceinline__ int plan_find(const T* list, int n, long long x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (list[m] <= x) lo = m; else hi = m;
  }
  return lo;
}

__global__ void __launch_bounds__(RP_THREADS) ragged_plan_kernel(const PlanParams p) {
  pdl_enter();
  __shared__ PlanSmem s;
  const int rank = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(gridDim.x);
  const int tid = threadIdx.x, gtid = rank * RP_THREADS + tid, gstride = ctas * RP_THREADS;
  const bool one_round = p.B <= RP_THREADS;
  const int n_free = min(max(*p.n_free, 0), p.n_blocks);
  long long row0 = 0, take0 = 0, mine = 0;
  bool bad_page = false;      // a position past its table row, or a block outside the pool
  auto slot_of = [&](int blk, int at, int lb) {
    if (blk < 0) return -1;
    if (blk >= p.n_blocks) {
      bad_page = true;
      return -1;
    }
    return blk * p.bs + (at - lb * p.bs);
  };
  // the chunk's requests, their prefix sums in shared memory
  auto load = [&](int base, long long (&t)[3]) -> PlanReq {
    const PlanReq r = plan_req(p, base + tid);
    long long v[3] = {r.n, r.take, r.back};
    plan_scan(s, v, t);
    s.row[tid] = v[0];
    s.take[tid] = v[1];
    s.back[tid] = v[2];
    s.ctx[tid] = r.ctx;
    s.held[tid] = r.held;
    s.want[tid] = r.want;
    if (tid == 0) {
      s.row[RP_THREADS] = t[0];
      s.take[RP_THREADS] = t[1];
    }
    __syncthreads();
    return r;
  };
  PlanReq r = {0, 0, 0, 0, 0, 0};
  long long t[3] = {0, 0, 0};

  for (int base = 0; base < p.B; base += RP_THREADS) {
    r = load(base, t);
    const int here = min(p.B - base, RP_THREADS);
    if (rank == 0 && tid < here) p.cu[base + tid] = static_cast<int32_t>(min(row0 + s.row[tid], static_cast<long long>(p.T)));
    // blocks granted: the largest prefix of the wishes that the list can give
    if (r.take > 0 && take0 + s.take[tid + 1] <= n_free) mine = take0 + s.take[tid + 1];
    // the new table entries: the k-th block taken comes from the list's end; a
    // request whose last block is not there has none of them
    for (long long k = gtid; k < t[1]; k += gstride) {
      const int i = plan_find(s.take, here, k);
      const int lb = s.held[i] + static_cast<int>(k - s.take[i]);
      const bool granted = take0 + s.take[i + 1] <= n_free;
      p.table[static_cast<int64_t>(base + i) * p.max_blocks + lb] = granted ? p.free_list[n_free - 1 - static_cast<int>(take0 + k)] : -1;
    }
    // the rows
    const int rows = static_cast<int>(max(0LL, min(t[0], static_cast<long long>(p.T) - row0)));
#pragma unroll 4
    for (int k = gtid; k < rows; k += gstride) {
      const int i = plan_find(s.row, here, k);
      const long long pos = s.ctx[i] + (k - s.row[i]);
      const int at = static_cast<int>(min(pos, RP_PAST)), lb = at / p.bs;    // RP_PAST: past any table row
      int slot = -1;
      if (lb < s.held[i]) {
        slot = slot_of(p.table[static_cast<int64_t>(base + i) * p.max_blocks + lb], at, lb);
      } else if (lb < s.want[i]) {
        // a block taken in this step, read where the table entry comes from
        if (take0 + s.take[i + 1] <= n_free)
          slot = slot_of(p.free_list[n_free - 1 - static_cast<int>(take0 + s.take[i] + (lb - s.held[i]))], at, lb);
      } else {
        bad_page = true;
      }
      p.pos[row0 + k] = static_cast<int32_t>(pos);
      p.slots[row0 + k] = slot;
    }
    row0 += t[0];
    take0 += t[1];
  }
  if (bad_page) record_error(p.err, KL_DEVERR_PAGE);
  // the blocks granted in all, found by every CTA for itself
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine = max(mine, static_cast<long long>(__shfl_xor_sync(0xffffffffu, mine, o)));
  if ((tid & 31) == 0) s.most[tid >> 5] = mine;
  if (ctas > 1) cluster_sync_all();                 // nobody reads the list any more
  else __syncthreads();
  long long granted = 0;
  for (int w = 0; w < RP_WARPS; ++w) granted = max(granted, s.most[w]);

  // ended requests' blocks go behind what is left of the list
  long long back = n_free - granted;
  for (int base = 0; base < p.B; base += RP_THREADS) {
    if (!one_round) r = load(base, t);
    const int here = min(p.B - base, RP_THREADS);
    for (long long k = gtid; k < t[2]; k += gstride) {
      const int i = plan_find(s.back, here, k);
      if (back + k < p.n_blocks)                    // a list that was consistent never grows past the pool
        p.free_list[back + k] = p.table[static_cast<int64_t>(base + i) * p.max_blocks + (k - s.back[i])];
    }
    back += t[2];
  }
  if (!one_round && ctas > 1) cluster_sync_all();   // nobody reads the counts any more
  if (rank != 0) return;
  // the counts: with one round of requests they are at hand still
  long long upto = 0;
  for (int base = 0; base < p.B; base += RP_THREADS) {
    if (!one_round) r = load(base, t);
    if (base + tid < p.B) p.held[base + tid] = r.back ? 0 : upto + s.take[tid + 1] <= granted ? max(r.held, r.want) : r.held;
    upto += t[1];
  }
  if (tid == 0) {
    p.cu[p.B] = static_cast<int32_t>(min(row0, static_cast<long long>(p.T)));
    *p.n_free = static_cast<int32_t>(min(back, static_cast<long long>(p.n_blocks)));
    *p.missing = static_cast<int32_t>(min(take0 - granted, 2147483647LL));
    if (row0 > p.T) record_error(p.err, KL_DEVERR_ROWS);
  }
}

// ---------------------------------------------------------------------------
// norm, rotation and cache write
// ---------------------------------------------------------------------------
// 128 threads with five heads each in flight, six CTAs per SM: 63 us for 8189 rows
// of 64 / 8 heads (5.3 TB/s); 256 with three and four 75, 320 with two and three 76.
// Bulk copies through shared memory by persistent CTAs took 64.5.
constexpr int RQ_THREADS = 128;
constexpr int RQ_D = 128;
constexpr int RQ_LANES = 8;        // threads per head: 8 planes (16 elements) each
constexpr int RQ_MAX = 5;          // heads a thread has in flight

struct QkvParams {
  const __nv_bfloat16* q_pre;
  const __nv_bfloat16* k_pre;
  const __nv_bfloat16* v;
  const __nv_bfloat16* gq;
  const __nv_bfloat16* gk;
  const int32_t* cu;
  const int32_t* pos;
  const int32_t* slots;
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_pool;
  __nv_bfloat16* v_pool;
  float eps;
  int B, T, Hq, Hkv, inter, pool_rows;
  uint32_t* err;
  RopeFreq f;
};

__device__ __forceinline__ void rq_unpack(const uint4& a, float (&f)[8]) {
  const float2 x0 = unpack_bf16x2(a.x), x1 = unpack_bf16x2(a.y), x2 = unpack_bf16x2(a.z), x3 = unpack_bf16x2(a.w);
  f[0] = x0.x; f[1] = x0.y; f[2] = x1.x; f[3] = x1.y;
  f[4] = x2.x; f[5] = x2.y; f[6] = x3.x; f[7] = x3.y;
}
__device__ __forceinline__ uint4 rq_pack(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// One head's eighth: thread l of a head's eight holds planes 8 l .. 8 l + 7, that
// is elements 8 l .. and 64 + 8 l .. (planes (i, i + 64)), or 16 l .. 16 l + 15
// (planes (2i, 2i + 1)): offsets ia and ib. xa, xb: its elements, normed (gva,
// gvb: its gains) and turned by the row's (cos, sin). Called by whole
// warps; `turn` is off for values, which stay as they are.
__device__ __forceinline__ void rq_turn(uint4& xa, uint4& xb, const uint4& gva, const uint4& gvb, bool norm, bool turn, int inter,
                                        int ia, float eps, const float2* cs) {
  float a[8], b[8];
  rq_unpack(xa, a);
  rq_unpack(xb, b);
  if (norm) {                                       // the same for all threads: the shuffles are convergent
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
#pragma unroll
    for (int o = RQ_LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (turn) {
      const float r = rsqrtf(ss / static_cast<float>(RQ_D) + eps);   // two ulp; the result is rounded to bf16
      float ga[8], gb[8];
      rq_unpack(gva, ga);
      rq_unpack(gvb, gb);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] = a[e] * r * ga[e];
        b[e] = b[e] * r * gb[e];
      }
    }
  }
  if (!turn) return;
  const int l8 = inter ? ia >> 1 : ia;              // 8 l
  if (inter) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 c0 = cs[l8 + e], c1 = cs[l8 + 4 + e];
      const float x0 = a[2 * e], y0 = a[2 * e + 1], x1 = b[2 * e], y1 = b[2 * e + 1];
      a[2 * e] = x0 * c0.x - y0 * c0.y;
      a[2 * e + 1] = x0 * c0.y + y0 * c0.x;
      b[2 * e] = x1 * c1.x - y1 * c1.y;
      b[2 * e + 1] = x1 * c1.y + y1 * c1.x;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 c = cs[l8 + e];
      const float x = a[e], z = b[e];
      a[e] = x * c.x - z * c.y;
      b[e] = x * c.y + z * c.x;
    }
  }
  xa = rq_pack(a);
  xb = rq_pack(b);
}

// One CTA per row. Heads in the order q, k, v; each element is read and written by
// one thread, so q_out may be q_pre.
__global__ void __launch_bounds__(RQ_THREADS, 6) ragged_qkv_kernel(const __grid_constant__ QkvParams p) {
  pdl_enter();
  __shared__ float2 cs[RQ_D / 2];
  const int row = blockIdx.x;
  const int heads = p.Hq + 2 * p.Hkv;
  const int l = threadIdx.x % RQ_LANES, h0 = threadIdx.x / RQ_LANES;
  constexpr int STEP = RQ_THREADS / RQ_LANES;
  const int ia = p.inter ? 16 * l : 8 * l, ib = p.inter ? 16 * l + 8 : 64 + 8 * l;
  auto src = [&](int h) {
    return h < p.Hq ? p.q_pre + (static_cast<int64_t>(row) * p.Hq + h) * RQ_D
           : h < p.Hq + p.Hkv ? p.k_pre + (static_cast<int64_t>(row) * p.Hkv + (h - p.Hq)) * RQ_D
                              : p.v + (static_cast<int64_t>(row) * p.Hkv + (h - p.Hq - p.Hkv)) * RQ_D;
  };
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  const bool norm = p.gq != nullptr;
  const uint4 gqa = norm ? *reinterpret_cast<const uint4*>(p.gq + ia) : none, gqb = norm ? *reinterpret_cast<const uint4*>(p.gq + ib) : none;
  const uint4 gka = norm ? *reinterpret_cast<const uint4*>(p.gk + ia) : none, gkb = norm ? *reinterpret_cast<const uint4*>(p.gk + ib) : none;
  // a row past the last request is read too (the tensors have it), not written
  const int rows = p.cu[p.B], pos = p.pos[row];
  int slot = p.slots[row];
  for (int base = 0; base < heads; base += RQ_MAX * STEP) {
    uint4 xa[RQ_MAX], xb[RQ_MAX];
#pragma unroll
    for (int j = 0; j < RQ_MAX; ++j) {
      const int h = base + j * STEP + h0;
      xa[j] = xb[j] = make_uint4(0u, 0u, 0u, 0u);
      if (h < heads) {
        const __nv_bfloat16* x = src(h);
        xa[j] = *reinterpret_cast<const uint4*>(x + ia);
        xb[j] = *reinterpret_cast<const uint4*>(x + ib);
      }
    }
    if (base == 0) {
      if (row >= rows) return;
      if (slot >= p.pool_rows) {
        if (threadIdx.x == 0) record_error(p.err, KL_DEVERR_PAGE);
        slot = -1;
      }
      if (threadIdx.x < RQ_D / 2) {
        float c, sn;
        rope_cos_sin(pos, p.f.turn[threadIdx.x], 1.0f, &c, &sn);
        cs[threadIdx.x] = make_float2(c, sn);
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < RQ_MAX; ++j) {
      const int h = base + j * STEP + h0;
      const bool turn = h < p.Hq + p.Hkv;
      rq_turn(xa[j], xb[j], h < p.Hq ? gqa : gka, h < p.Hq ? gqb : gkb, norm, turn, p.inter, ia, p.eps, cs);
      if (h >= heads || (h >= p.Hq && slot < 0)) continue;
      __nv_bfloat16* y = h < p.Hq ? p.q_out + (static_cast<int64_t>(row) * p.Hq + h) * RQ_D
                         : turn ? p.k_pool + (static_cast<int64_t>(slot) * p.Hkv + (h - p.Hq)) * RQ_D
                                : p.v_pool + (static_cast<int64_t>(slot) * p.Hkv + (h - p.Hq - p.Hkv)) * RQ_D;
      *reinterpret_cast<uint4*>(y + ia) = xa[j];
      *reinterpret_cast<uint4*>(y + ib) = xb[j];
    }
  }
}

}  // namespace

kl_status ragged_check(const kl_ragged_cfg* rc) {
  if (!rc) return set_error(KL_ERR_INVALID_ARG, "ragged: null configuration");
  if (rc->B < 1 || rc->T < 1 || rc->block_size < 1 || rc->max_blocks < 1 || rc->n_blocks < 1)
    return set_error(KL_ERR_INVALID_ARG, "ragged: bad sizes (B %d, T %d, block %d, table %d, pool %d)", rc->B, rc->T,
                     rc->block_size, rc->max_blocks, rc->n_blocks);
  if (rc->T > (1 << 24) || rc->B > (1 << 24))
    return set_error(KL_ERR_UNSUPPORTED, "ragged: too many rows or requests (%d, %d)", rc->T, rc->B);
  const double rows = static_cast<double>(rc->n_blocks) * rc->block_size;
  if (rows >= 2147483647.0)
    return set_error(KL_ERR_UNSUPPORTED, "ragged: pool rows (%.0f) beyond 32-bit indexing", rows);
  if (static_cast<double>(rc->max_blocks) * rc->block_size > 1073741824.0)
    return set_error(KL_ERR_UNSUPPORTED, "ragged: a table row of %d blocks of %d tokens above 2^30 positions", rc->max_blocks,
                     rc->block_size);
  return KL_OK;
}

kl_status ragged_heads_check(const kl_ragged_cfg* rc, int Hq, int Hkv, int d, int dtype) {
  KL_TRY(ragged_check(rc));
  if (Hq < 1 || Hkv < 1 || Hq % Hkv) return set_error(KL_ERR_INVALID_ARG, "ragged: bad head counts %d / %d", Hq, Hkv);
  if (d != RQ_D || dtype != KL_BF16)
    return set_error(KL_ERR_UNSUPPORTED, "ragged: bf16 with head dim 128 only (got dtype %d, d %d)", dtype, d);
  if (Hq / Hkv > 128) return set_error(KL_ERR_UNSUPPORTED, "ragged: %d query heads per kv head above 128", Hq / Hkv);
  const double rows = static_cast<double>(rc->n_blocks) * rc->block_size * Hkv;
  if (rows >= 2147483647.0)
    return set_error(KL_ERR_UNSUPPORTED, "ragged: pool rows (%.0f) beyond 32-bit indexing", rows);
  return KL_OK;
}

kl_status ragged_plan(const kl_ragged_cfg& rc, const int32_t* n_new, const int32_t* ctx, int32_t* table, int32_t* held,
                      int32_t* free_list, int32_t* n_free, int32_t* cu, int32_t* pos, int32_t* slots, int32_t* missing,
                      cudaStream_t st) {
  PlanParams p = {n_new, ctx, table, held, free_list, n_free, cu, pos, slots, missing,
                  rc.B, rc.T, rc.block_size, rc.max_blocks, rc.n_blocks, device_error_word()};
  const int ctas = rc.T > RP_ONE_CTA_ROWS || rc.B > RP_THREADS ? RP_CLUSTER : 1;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(RP_THREADS);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  ProfScope ps("ragged_plan", st, 0.0, 20.0 * rc.B + 8.0 * rc.T);
  KL_CUDA(cudaLaunchKernelEx(&cfg, ragged_plan_kernel, p));
  return KL_OK;
}

kl_status ragged_qkv_rope(const kl_ragged_cfg& rc, int Hq, int Hkv, const void* q_pre, const void* k_pre, const void* v,
                          const void* gq, const void* gk, float eps, float base, int inter, const int32_t* cu,
                          const int32_t* pos, const int32_t* slots, void* q_out, void* kp, void* vp, cudaStream_t st) {
  QkvParams p;
  p.q_pre = static_cast<const __nv_bfloat16*>(q_pre);
  p.k_pre = static_cast<const __nv_bfloat16*>(k_pre);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.gq = static_cast<const __nv_bfloat16*>(gq);
  p.gk = static_cast<const __nv_bfloat16*>(gk);
  p.cu = cu;
  p.pos = pos;
  p.slots = slots;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_pool = static_cast<__nv_bfloat16*>(kp);
  p.v_pool = static_cast<__nv_bfloat16*>(vp);
  p.eps = eps;
  p.B = rc.B;
  p.T = rc.T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.inter = inter;
  p.pool_rows = rc.n_blocks * rc.block_size;
  p.err = device_error_word();
  p.f = rope_freq(RQ_D, base);
  ProfScope ps("ragged_qkv_rope", st, 0.0, 2.0 * 2 * rc.T * (Hq + 2.0 * Hkv) * RQ_D);
  launch_pdl(ragged_qkv_kernel, rc.T, RQ_THREADS, 0, st, p);
  KL_CUDA(cudaGetLastError());
  return KL_OK;
}

}  // namespace kl
