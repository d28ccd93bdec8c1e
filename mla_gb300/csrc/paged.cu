// Appending to the paged 8-bit cache.
//
// Per touched page and head: the new tokens' keys and values are read once
// (a warp takes a token's 128 keys in its lower and 128 values in its upper
// 16 lanes, 16 bytes a lane), held in registers while their largest magnitude
// is reduced over the page's warps, and written as E4M3 codes of x * 2^-k with
// the smallest k in [-60, 60] that keeps amax <= 448 * 2^k.  A page that
// already holds tokens keeps the larger of 2^k and its scale; when 2^k is the
// larger, its codes are decoded and coded again at the new scale.  Scales are
// powers of two, so that a code and its re-expression differ only where the
// larger scale drops bits; a page that something else has filled may bring any
// positive scale, by which the new tokens are divided then.
// The rotary keys (one per token, shared by the heads) are rotated by a
// further row of CTAs, angles as in the RoPE table.  The kernel is held to 64
// registers: the division by a foreign scale would take it to 97, with fewer
// warps to load (8 x 4096 tokens 345 us where they take 259).
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace mla {

namespace {

constexpr int kFloorExp = -60, kCeilExp = 60;

// Sequence b's new tokens: positions p .. p + n - 1 from source row `row` on.
// n = 0 for an idle sequence; bad = arguments that no append can take.
struct AppendSeq {
  int p, n, row;
  bool bad;
  __device__ __forceinline__ AppendSeq(const PagedAppendArgs& a, int b) {
    p = a.P ? a.P[b] : a.p0;
    row = a.cu ? a.cu[b] : b * a.T;
    n = a.cu ? a.cu[b + 1] - row : a.T;
    const long long cap = (long long)a.c.max_pages * a.c.page;
    bad = p < -1 || p > a.p_max || n < 0 || n > a.T || row < 0 || (long long)row + n > a.N ||
          (p >= 0 && (long long)p + n > cap);
    if (bad || p < 0) n = 0;
  }
};

// The smallest k in [-60, 60] with top <= 448 * 2^k (448 = 1.75 * 2^8), top >= 0.
__device__ __forceinline__ int block_exp(float top) {
  const uint32_t u = __float_as_uint(top);
  const int k = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(kCeilExp, max(kFloorExp, k));
}

__device__ __forceinline__ float exp2_int(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }

__device__ __forceinline__ uint32_t code2(float x0, float x1) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float2 decode2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xffffu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// 8 bf16 -> 8 codes of x * r
__device__ __forceinline__ uint2 code8(const uint4& u, float r) {
  const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y), c = unpack_bf16x2(u.z), d = unpack_bf16x2(u.w);
  return make_uint2(code2(a.x * r, a.y * r) | code2(b.x * r, b.y * r) << 16,
                    code2(c.x * r, c.y * r) | code2(d.x * r, d.y * r) << 16);
}

// y rounded towards zero from a value that is y + rest: to odd, so that the
// rounding of y to a code (4 bits of 24) has the value's own answer
__device__ __forceinline__ float to_odd(float y, float rest) {
  return rest > 0.f || rest < 0.f ? __uint_as_float(__float_as_uint(y) | 1u) : y;
}
// x / s and c * r for a rounding to a code
__device__ __forceinline__ float quotient(float x, float s) {
  const float y = __fdiv_rz(x, s);
  return to_odd(y, fmaf(-y, s, x));
}
__device__ __forceinline__ float product(float c, float r) {
  const float y = __fmul_rz(c, r);
  return to_odd(y, fmaf(c, r, -y));
}

// The two rare forms of a page's rows, 8 elements of n rows each.  New tokens
// in a page whose scale is not a power of two: divided by it.
__device__ __forceinline__ void divide_rows(const __nv_bfloat16* src, long long src_step, uint8_t* dst, int dst_step,
                                            int n, float scale) {
#pragma unroll 1
  for (int i = 0; i < n; ++i, src += src_step, dst += dst_step) {
    const uint4 x = *reinterpret_cast<const uint4*>(src);
    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
    uint32_t out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack_bf16x2(in[e]);
      out[e] = code2(quotient(f.x, scale), quotient(f.y, scale));
    }
    *reinterpret_cast<uint2*>(dst) = make_uint2(out[0] | out[1] << 16, out[2] | out[3] << 16);
  }
}
// Codes that a growing scale re-expresses, r = old scale / new scale.
__device__ __forceinline__ void rescale_rows(uint8_t* at, int step, int n, float r) {
#pragma unroll 1
  for (int i = 0; i < n; ++i, at += step) {
    const uint2 x = *reinterpret_cast<const uint2*>(at);
    const uint32_t in[4] = {x.x, x.x >> 16, x.y, x.y >> 16};
    uint32_t out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = decode2(in[e]);
      out[e] = code2(product(f.x, r), product(f.y, r));
    }
    *reinterpret_cast<uint2*>(at) = make_uint2(out[0] | out[1] << 16, out[2] | out[3] << 16);
  }
}

// keys or values of sequence b's new token t, head h
__device__ __forceinline__ const __nv_bfloat16* source(const PagedAppendArgs& a, int b, int h, int t, int row,
                                                       bool is_v) {
  return is_v ? a.v + b * a.v_seq + (a.v_seq ? t : row + t) * a.v_token + h * a.v_head
              : a.k + b * a.k_seq + (a.k_seq ? t : row + t) * a.k_token + h * a.k_head;
}

// larger |x| of two pairs of bf16, element by element, NaN ignored
__device__ __forceinline__ __nv_bfloat162 top_pair(__nv_bfloat162 m, uint32_t u) {
  const uint32_t a = u & 0x7fff7fffu;
  return __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&a));
}

// Grid: x = (sequence, touched page), y = head group, and one row of CTAs more
// for the rotary keys.  2^w_log warps share a head, each holding up to 8 tokens.
__global__ void __launch_bounds__(512, 2) paged_append_kernel(const PagedAppendArgs a, int pages_per_seq, int w_log) {
  __shared__ float red[16][2];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int warps = blockDim.x >> 5;
  const int page = a.c.page, page_log = 31 - __clz(page);

  if (blockIdx.x == 0 && blockIdx.y == 0) {
    // every sequence and page number of the call, for the status word
    int bad = 0;
    for (int i = tid; i < a.B * pages_per_seq; i += blockDim.x) {
      const int b = i / pages_per_seq, j = i - b * pages_per_seq;
      const AppendSeq s(a, b);
      bad |= s.bad;
      const int pi = (s.p >> page_log) + j;
      if (s.n > 0 && pi * page < s.p + s.n) {
        const int pid = a.c.table[(size_t)b * a.c.max_pages + pi];
        bad |= pid < 0 || pid >= a.c.n_pages;
      }
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) {
      if (!a.status_cleared) {
        a.status[0] = bad ? kStatusBadLength : 0u;
        a.status[kStatusExtraWord] = 0u;
      } else if (bad) {
        atomicOr(a.status, kStatusBadLength);
      }
    }
  }

  const int b = blockIdx.x / pages_per_seq, j = blockIdx.x - b * pages_per_seq;
  const AppendSeq s(a, b);
  const int pi = (s.p >> page_log) + j;
  const int base = pi * page;                        // the page's first position
  if (s.n == 0 || base >= s.p + s.n) return;
  const int pid = a.c.table[(size_t)b * a.c.max_pages + pi];
  if (pid < 0 || pid >= a.c.n_pages) return;
  const int slot0 = max(s.p - base, 0);              // first new slot = tokens already in the page
  const int n = min(s.p + s.n, base + page) - (base + slot0);
  const int t0 = base + slot0 - s.p;                 // the new token in slot0

  if (blockIdx.y == gridDim.y - 1) {
    for (int i = warp; i < n; i += warps) {
      const long long r = (long long)(s.row + t0 + i) * a.pe_token;
      const float x1 = a.pe ? __bfloat162float(a.pe[r + lane]) : a.pe_f32[r + lane];
      const float x2 = a.pe ? __bfloat162float(a.pe[r + lane + 32]) : a.pe_f32[r + lane + 32];
      const float2 cs = rope_cos_sin(base + slot0 + i, a.inv_freq[lane]);
      __nv_bfloat16* d = a.c.k_pe + ((size_t)pid * page + slot0 + i) * 64;
      d[lane] = __float2bfloat16_rn(x1 * cs.x - x2 * cs.y);
      d[lane + 32] = __float2bfloat16_rn(x2 * cs.x + x1 * cs.y);
    }
    return;
  }

  const int h = blockIdx.y * (warps >> w_log) + (warp >> w_log), W = 1 << w_log, wi = warp & (W - 1);
  const bool live = h < a.c.heads;
  const bool is_v = lane >= 16;
  const int col = (lane & 15) * 8;
  constexpr int kRows = 8;
  uint4 u[kRows];
  float top = 0.f;
  float* scale_at = nullptr;
  float old = 0.f;  // the scale that the page's tokens have
  const int mine = (n - wi + W - 1) >> w_log;  // this warp's tokens: wi, wi + W, ..
  if (live) {
    const long long token = is_v ? a.v_token : a.k_token;
    const __nv_bfloat16* src = source(a, b, h, t0, s.row, is_v);
    const __nv_bfloat16* at = src + wi * token + col;
    const long long step = token << w_log;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      u[i] = i < mine ? *reinterpret_cast<const uint4*>(at) : make_uint4(0u, 0u, 0u, 0u);
      at += step;
    }
    scale_at = (is_v ? a.c.v_scales : a.c.k_scales) + (size_t)pid * a.c.heads + h;
    if (slot0 > 0) old = *scale_at;
    __nv_bfloat162 m0 = __floats2bfloat162_rn(0.f, 0.f), m1 = m0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      m0 = top_pair(top_pair(m0, u[i].x), u[i].y);
      m1 = top_pair(top_pair(m1, u[i].z), u[i].w);
    }
    const float2 f = __bfloat1622float2(__hmax2(m0, m1));
    top = fmaxf(f.x, f.y);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  if (W > 1) {
    if ((lane & 15) == 0) red[warp][is_v] = top;
    __syncthreads();
    for (int i = 0; i < W; ++i) top = fmaxf(top, red[warp - wi + i][is_v]);
  }
  if (!live) return;
  const float need = exp2_int(block_exp(top)), scale = fmaxf(need, old);
  if (wi == 0 && (lane & 15) == 0) *scale_at = scale;
  uint8_t* dst = (is_v ? a.c.v_codes : a.c.k_codes) + (((size_t)pid * a.c.heads + h) << page_log) * 128 + col;
  const uint32_t bits = __float_as_uint(scale);
  if (!(bits & 0x7fffffu) && bits - (1u << 23) < 253u << 23) {  // a power of two that has a reciprocal
    const float r = __uint_as_float((254u << 23) - bits);
    uint8_t* at = dst + (slot0 + wi) * 128;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (i < mine) *reinterpret_cast<uint2*>(at) = code8(u[i], r);
      at += 128 << w_log;
    }
  } else {
    divide_rows(source(a, b, h, t0 + wi, s.row, is_v) + col, (is_v ? a.v_token : a.k_token) << w_log,
                dst + (slot0 + wi) * 128, 128 << w_log, mine, scale);
  }
  if (slot0 > 0 && need > old) rescale_rows(dst + wi * 128, 128 << w_log, (slot0 - wi + W - 1) >> w_log, old / need);
}

// Grid: x = (sequence, page of 16 positions), y = head: a warp per 2
// positions, 8 codes a lane and step.  The rotary key of a position is
// copied into each head's row.
__global__ void __launch_bounds__(256) paged_gather_kernel(const PagedGatherArgs a, int blocks) {
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x / blocks, h = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j0 = (blockIdx.x - b * blocks) * 16;
  if (j0 + 16 <= a.from && j0 >= a.first) return;
  const int id = a.c.table[(size_t)b * a.c.max_pages + j0 / a.c.page];
  const bool bad = id < 0 || id >= a.c.n_pages;
  if (bad && threadIdx.x == 0 && h == 0) atomicOr(a.status, kStatusBadLength);
  const int pid = bad ? 0 : id;
  const float ks = a.c.k_scales[(size_t)pid * a.c.heads + h], vs = a.c.v_scales[(size_t)pid * a.c.heads + h];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = j0 + warp * 2 + i;
    if (j >= a.P || (j < a.from && j >= a.first)) continue;
    const int slot = j & (a.c.page - 1);
    const size_t row = (((size_t)pid * a.c.heads + h) * a.c.page + slot) * 128;
    const size_t dst = ((size_t)b * a.c.heads + h) * a.cap + j;
    // lanes 0..15: 8 key codes each, 16..31: 8 value codes; then the 64 rotary values
    const bool is_v = lane >= 16;
    const int col = (lane & 15) * 8;
    const uint2 c = *reinterpret_cast<const uint2*>((is_v ? a.c.v_codes : a.c.k_codes) + row + col);
    const float s = is_v ? vs : ks;
    const float2 x0 = decode2(c.x), x1 = decode2(c.x >> 16), x2 = decode2(c.y), x3 = decode2(c.y >> 16);
    const uint4 u = make_uint4(pack_bf16x2(x0.x * s, x0.y * s), pack_bf16x2(x1.x * s, x1.y * s),
                               pack_bf16x2(x2.x * s, x2.y * s), pack_bf16x2(x3.x * s, x3.y * s));
    *reinterpret_cast<uint4*>((is_v ? a.v + dst * 128 : a.k + dst * 192) + col) = u;
    if (lane < 8)
      *reinterpret_cast<uint4*>(a.k + dst * 192 + 128 + lane * 8) =
          *reinterpret_cast<const uint4*>(a.c.k_pe + ((size_t)pid * a.c.page + slot) * 64 + lane * 8);
  }
}

}  // namespace

cudaError_t launch_paged_gather(const PagedGatherArgs& a, cudaStream_t stream) {
  const int blocks = (a.P + 15) / 16;
  const long long gx = (long long)a.B * blocks;
  if (gx > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(paged_gather_kernel, dim3((unsigned)gx, a.c.heads), dim3(256), 0, stream, a, blocks);
}

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream) {
  const int most = min(a.T, a.N);  // a sequence has no more rows than the call
  const int pages_per_seq = paged_append_pages(most, a.c.page);
  // 8 tokens a warp: one warp per head for a few new tokens, else page / 8
  const int w_log = most <= 8 ? 0 : a.c.page == 16 ? 1 : a.c.page == 32 ? 2 : a.c.page == 64 ? 3 : 4;
  const int W = 1 << w_log, warps = W > 8 ? W : 8;
  const long long gx = (long long)a.B * pages_per_seq;
  if (gx > 1 << 24) return cudaErrorInvalidValue;
  const int gy = (a.c.heads * W + warps - 1) / warps + 1;
  return launch_pdl(paged_append_kernel, dim3((unsigned)gx, gy), dim3(warps * 32), 0, stream, a,
                    pages_per_seq, w_log);
}

}  // namespace mla
