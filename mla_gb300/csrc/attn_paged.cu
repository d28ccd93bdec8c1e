// Attention of a few new tokens per sequence over the paged 8-bit cache.
//
// Scores s_j = scale * (kscale * (q_nope . code_j) + q_pe . kpe_j), softmax in
// float32 over the visible keys, o = sum_j p_j vscale * code_j.  One CTA per
// (head, query), tiles of 128 keys: a thread forms one key's score, then one
// value dimension's sum.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace mla {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float decode1(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

__global__ void __launch_bounds__(128) paged_attn_simple(const PagedAttnArgs a) {
  __shared__ float q[192], s[128];
  __shared__ float red[4];
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.x, row = blockIdx.y, b = row / a.T, t = row - b * a.T;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int p0 = a.P[b];
  const bool idle = p0 < 0 || p0 > a.P_max;
  bool bad = p0 < -1 || p0 > a.P_max;
  const int qi = idle ? -1 : p0 + t;  // this query's position
  for (int d = tid; d < 192; d += 128) q[d] = __bfloat162float(a.q[row * a.q_row + h * 192 + d]);
  __syncthreads();
  float m = -INFINITY, l = 0.f, o = 0.f;
  const int start = a.window ? max(0, qi - a.window + 1) : 0;
  for (int k0 = 0; k0 <= qi; k0 += 128) {
    if (a.window && k0 >= a.sinks && k0 + 127 < start) continue;
    const int j = k0 + tid;
    const bool seen = j <= qi && (!a.window || j >= start || j < a.sinks);
    float x = -INFINITY;
    if (seen) {
      const int id = a.c.table[(size_t)b * a.c.max_pages + j / a.c.page];
      bad |= id < 0 || id >= a.c.n_pages;
      const int pid = min(max(id, 0), a.c.n_pages - 1);
      const uint8_t* kc = a.c.k_codes + (((size_t)pid * a.c.heads + h) * a.c.page + j % a.c.page) * 128;
      const __nv_bfloat16* kp = a.c.k_pe + ((size_t)pid * a.c.page + j % a.c.page) * 64;
      float acc = 0.f, acc2 = 0.f;
      for (int d = 0; d < 128; ++d) acc = fmaf(q[d], decode1(kc[d]), acc);
      for (int d = 0; d < 64; ++d) acc2 = fmaf(q[128 + d], __bfloat162float(kp[d]), acc2);
      x = (acc * a.c.k_scales[(size_t)pid * a.c.heads + h] + acc2) * (a.scale * kLog2e);
    }
    float mx = warp_max(x);
    if (lane == 0) red[warp] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float m_new = fmaxf(m, mx), ref = m_new == -INFINITY ? 0.f : m_new;
    s[tid] = exp2f(x - ref);
    __syncthreads();
    const float alpha = exp2f(m - ref);
    m = m_new;
    l *= alpha;
    o *= alpha;
    for (int i = 0; i < 128 && k0 + i <= qi; ++i) {
      const int jj = k0 + i;
      if (a.window && jj < start && jj >= a.sinks) continue;
      const int id = a.c.table[(size_t)b * a.c.max_pages + jj / a.c.page];
      const int pid = min(max(id, 0), a.c.n_pages - 1);
      const uint8_t* vc = a.c.v_codes + (((size_t)pid * a.c.heads + h) * a.c.page + jj % a.c.page) * 128;
      l += s[i];
      o = fmaf(s[i] * a.c.v_scales[(size_t)pid * a.c.heads + h], decode1(vc[tid]), o);
    }
    __syncthreads();
  }
  a.o[row * a.o_row + h * 128 + tid] = __float2bfloat16_rn(l > 0.f ? o / l : 0.f);
  if (bad) atomicOr(a.status, kStatusBadLength);
}

}  // namespace

cudaError_t launch_paged_attention(const PagedAttnArgs& a, const DevStatusHost& st, int num_sms, cudaStream_t stream,
                                   int* launches) {
  (void)st;
  (void)num_sms;
  if (!a.status_cleared) {
    const cudaError_t e = cudaMemsetAsync(a.status, 0, 256, stream);
    if (e != cudaSuccess) return e;
  }
  ++*launches;
  return launch_pdl(paged_attn_simple, dim3(a.c.heads, a.B * a.T), dim3(128), 0, stream, a);
}

}  // namespace mla
