// Log probabilities of given tokens with each row's entropy and most likely classes,
// and their gradient. With m = max z, s = sum exp(z - m), u = sum (z - m) exp(z - m):
//   log p_t = z_t - m - log s,  H = log s - u / s,
//   dz_j = a (1[j = t] - p_j) - b p_j (log p_j + H).
// One CTA per row; the alternatives one after the other, each the best class behind
// the one before.
#include <limits.h>
#include <math.h>

#include "internal.h"
#include "kl_common.cuh"

namespace kl {
namespace {

constexpr int LP_THREADS = 256;
constexpr int LP_WARPS = LP_THREADS / 32;

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

template <typename T>
__global__ void __launch_bounds__(LP_THREADS) token_logprobs_kernel(const __grid_constant__ LpParams p) {
  pdl_enter();
  __shared__ float red[3][LP_WARPS];
  __shared__ int red_i[LP_WARPS];
  const int n = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* z = static_cast<const T*>(p.z) + static_cast<int64_t>(n) * p.ldz;
  float m = -INFINITY;
  for (int i = threadIdx.x; i < p.V; i += LP_THREADS) m = fmaxf(m, Elem<T>::to_f(z[i]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[0][warp] = m;
  __syncthreads();
  for (int w = 0; w < LP_WARPS; ++w) m = fmaxf(m, red[0][w]);
  float s = 0.f, u = 0.f;
  for (int i = threadIdx.x; i < p.V; i += LP_THREADS) {
    const float x = Elem<T>::to_f(z[i]) - m, e = expf(x);
    s += e;
    if (!(e == 0.f)) u += e * x;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    u += __shfl_xor_sync(0xffffffffu, u, o);
  }
  if (lane == 0) {
    red[1][warp] = s;
    red[2][warp] = u;
  }
  __syncthreads();
  s = u = 0.f;
  for (int w = 0; w < LP_WARPS; ++w) {
    s += red[1][w];
    u += red[2][w];
  }
  const bool some = m > -INFINITY || s > 0.f;   // all -inf: s is NaN
  bool nan = false;
  if (!some) {                                  // -inf everywhere, or NaN somewhere
    for (int i = threadIdx.x; i < p.V; i += LP_THREADS) nan |= isnan(Elem<T>::to_f(z[i]));
    nan = __syncthreads_or(nan);
  }
  const bool empty = !some && !nan;
  const float ls = empty ? -INFINITY : logf(s);
  if (threadIdx.x == 0) {
    const int t = p.tokens[n];
    float lp = 0.f;
    if (t >= 0 && t < p.V) lp = empty ? -INFINITY : Elem<T>::to_f(z[t]) - m - ls;
    else if (t != -1) record_error(p.err, KL_DEVERR_TARGET);
    p.logprob[n] = lp;
    if (p.entropy) p.entropy[n] = empty ? 0.f : ls - u / s;
    if (p.norm) {
      p.norm[2 * n] = m;
      p.norm[2 * n + 1] = ls;
    }
  }
  float last = INFINITY;
  int last_i = -1;
  for (int k = 0; k < p.top; ++k) {
    float b = -INFINITY;
    int bi = INT_MAX;
    for (int i = threadIdx.x; i < p.V; i += LP_THREADS) {
      const float x = Elem<T>::to_f(z[i]);
      if ((x < last || (x == last && i > last_i)) && x > b) {
        b = x;
        bi = i;
      }
    }
    auto better = [&](float x, int i) {
      if (x > b || (x == b && i < bi)) {
        b = x;
        bi = i;
      }
    };
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) better(__shfl_xor_sync(0xffffffffu, b, o), __shfl_xor_sync(0xffffffffu, bi, o));
    __syncthreads();
    if (lane == 0) {
      red[0][warp] = b;
      red_i[warp] = bi;
    }
    __syncthreads();
    for (int w = 0; w < LP_WARPS; ++w) better(red[0][w], red_i[w]);
    last = b;
    last_i = bi;
    if (threadIdx.x == 0) {
      p.top_id[static_cast<int64_t>(n) * p.top + k] = b > -INFINITY ? bi : -1;
      p.top_lp[static_cast<int64_t>(n) * p.top + k] = b > -INFINITY ? b - m - ls : -INFINITY;
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
  int N, V;
  uint32_t* err;
};

template <typename T, typename U>
__global__ void __launch_bounds__(LP_THREADS) token_logprobs_bwd_kernel(const __grid_constant__ LpBwdParams p) {
  pdl_enter();
  const int n = blockIdx.x;
  const T* z = static_cast<const T*>(p.z) + static_cast<int64_t>(n) * p.ldz;
  U* dz = static_cast<U*>(p.dz) + static_cast<int64_t>(n) * p.lddz;
  const float m = p.norm[2 * n], ls = p.norm[2 * n + 1];
  const bool empty = m == -INFINITY && ls == -INFINITY;
  int t = p.tokens[n];
  if (t < -1 || t >= p.V) {
    if (threadIdx.x == 0) record_error(p.err, KL_DEVERR_TARGET);
    t = -1;
  }
  const float a = t >= 0 && p.dlp ? p.dlp[n] : 0.f, b = p.dent ? p.dent[n] : 0.f, H = p.dent ? p.entropy[n] : 0.f;
  for (int i = threadIdx.x; i < p.V; i += LP_THREADS) {
    const float x = Elem<T>::to_f(z[i]) - m - ls, e = expf(x);
    float d = e == 0.f ? 0.f : -e * (a + b * (x + H));
    if (i == t) d += a;
    dz[i] = Elem<U>::from_f(empty ? 0.f : d);
  }
}

}  // namespace

kl_status token_logprobs(int N, int V, int dtype, const void* z, int64_t ldz, const int32_t* tokens, int n_top,
                         float* logprob, float* entropy, float* norm, int32_t* top_id, float* top_logprob,
                         cudaStream_t st) {
  const LpParams p = {z, ldz, tokens, logprob, entropy, norm, top_id, top_logprob, N, V, n_top, device_error_word()};
  ProfScope ps("token_logprobs", st, 0.0, static_cast<double>(N) * V * dtype_size(dtype));
  if (dtype == KL_F32) launch_pdl(token_logprobs_kernel<float>, N, LP_THREADS, 0, st, p);
  else launch_pdl(token_logprobs_kernel<__nv_bfloat16>, N, LP_THREADS, 0, st, p);
  KL_CUDA(cudaGetLastError());
  return KL_OK;
}

kl_status token_logprobs_bwd(int N, int V, int dtype, const void* z, int64_t ldz, const int32_t* tokens,
                             const float* norm, const float* entropy, const float* dlp, const float* dent, int dz_dtype,
                             void* dz, int64_t lddz, cudaStream_t st) {
  const LpBwdParams p = {z, ldz, tokens, norm, entropy, dlp, dent, dz, lddz, N, V, device_error_word()};
  ProfScope ps("token_logprobs_bwd", st, 0.0, static_cast<double>(N) * V * (dtype_size(dtype) + dtype_size(dz_dtype)));
  if (dtype == KL_F32 && dz_dtype == KL_F32) launch_pdl(token_logprobs_bwd_kernel<float, float>, N, LP_THREADS, 0, st, p);
  else if (dtype == KL_F32) launch_pdl(token_logprobs_bwd_kernel<float, __nv_bfloat16>, N, LP_THREADS, 0, st, p);
  else if (dz_dtype == KL_F32) launch_pdl(token_logprobs_bwd_kernel<__nv_bfloat16, float>, N, LP_THREADS, 0, st, p);
  else launch_pdl(token_logprobs_bwd_kernel<__nv_bfloat16, __nv_bfloat16>, N, LP_THREADS, 0, st, p);
  KL_CUDA(cudaGetLastError());
  return KL_OK;
}

}  // namespace kl
