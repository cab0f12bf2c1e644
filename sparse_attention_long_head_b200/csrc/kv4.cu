// Writing to and reading from the 4-bit paged key/value cache (format:
// kv4.cuh).
//
// Quantisation of a group of 64 channels x:
//     m = min x,  s = bf16((max x - min x) / 15),
//     n = clamp(rint((x - m) / s), 0, 15)  (ties to even),  x ~ s n + m.
// m is exact in bf16 (it is one of the values).  s is rounded to bf16: 15 s
// then misses the range by at most 15 s 2^-8 = 0.06 s, far less than the half
// step that n itself may be off.  Both quotients are formed in fp32 and, where
// that comes next to a border between two results, again in fp64, so that s
// and n are those of the exact quotients.  s = 0 (a constant group) gives
// n = 0; an infinity or NaN in the group gives s = m = NaN, so that the group
// reads back as NaN.
//
// Both kernels are bound by memory: 4 d bytes of bf16 K and V and 9/8 d bytes
// of cache per token and head.  Eight lanes take one group of one slot (16
// bytes of K and of V each), so every access is a full 32- or 128-byte piece.
#include <cuda_bf16.h>

#include "kv4.cuh"

namespace vs {

constexpr int kKv4Threads = 256;

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Codes of this lane's eight channels and the pair of the group that the
// eight lanes of an aligned octet hold (the whole warp must call it).
__device__ __forceinline__ uint32_t quantize8(const uint4& u, uint32_t& pair) {
  float x[8];
  unpack8(u, x);
  float lo = x[0], hi = x[0];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    bad |= !(fabsf(x[i]) <= 3.402823466e38f);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const uint32_t bads = __ballot_sync(0xffffffffu, bad);
  const int lane = threadIdx.x & 31;
  if ((bads >> (lane & 24)) & 0xffu) {
    pair = 0x7fc07fc0u;
    return 0u;
  }
  const double lo64 = lo;
  // (hi - lo) / 15 to within 2^-22: the bf16 it rounds to, unless its low half
  // is next to 0x8000, it is subnormal or hi - lo overflowed
  float range = (hi - lo) * (1.f / 15.f);
  const int low = (int)(__float_as_uint(range) & 0xffffu) - 0x8000;
  if ((low < 8 && low > -8) || !(range > 1e-30f && range < 1e37f))
    range = (float)(((double)hi - lo64) / 15.0);
  const __nv_bfloat16 sb = __float2bfloat16_rn(range);
  const float s = __bfloat162float(sb);
  pair = (uint32_t)__bfloat16_as_ushort(sb) | (__float_as_uint(lo) & 0xffff0000u);
  if (s == 0.f) return 0u;
  const float r = 1.f / s;
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = (x[i] - lo) * r;
    float n = rintf(q);
    // near a half (or not a number: x - m or 1 / s overflowed), decide exactly
    if (!(fabsf(q - n) < 0.4999f)) n = (float)rint(((double)x[i] - lo64) / (double)s);
    word |= (uint32_t)(int)fminf(fmaxf(n, 0.f), 15.f) << (4 * i);
  }
  return word;
}

__global__ void __launch_bounds__(kKv4Threads) kv4_append_kernel(Kv4AppendArgs a) {
  const Kv4Cache& c = a.c;
  const int b = blockIdx.y;
  int64_t tok0;
  int n, len;
  bool ok = seq_range(a.cu, a.total, a.max_new, b, tok0, n);
  ok = kv4_len(c, b, len) && ok;
  // room: the new slots are [len - n, len)
  ok = ok && n <= len && len <= 64 * c.table_ld && ((!a.acc && !a.pos) || len <= a.ld);
  if (!ok) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.status, VS_DEVFLAG_BOUNDS);
    return;
  }
  const int start = len - n;
  const uint32_t stride = gridDim.x * blockDim.x;
  const uint32_t first = blockIdx.x * blockDim.x + threadIdx.x;
  const uint32_t line = c.Hkv * c.GR * 8;  // jobs a token: a lane's eight channels of K and of V
  const uint32_t jobs = n * line;          // below 2^31
  const uint4* K = static_cast<const uint4*>(a.K) + tok0 * (a.kv_stride / 8);
  const uint4* V = static_cast<const uint4*>(a.V) + tok0 * (a.kv_stride / 8);
  for (uint32_t base = first - (threadIdx.x & 31); base < jobs; base += stride) {
    const uint32_t e = base + (threadIdx.x & 31);
    const bool live = e < jobs;
    const uint32_t ec = live ? e : jobs - 1;
    const uint32_t t = ec / line, x = ec - t * line;  // x: 16-byte piece of the token's row
    const int w = x & 7, g = (x >> 3) & (c.GR - 1), head = x / (8 * c.GR);
    const int64_t src = (int64_t)t * (a.kv_stride / 8) + x;
    const uint4 ku = __ldg(K + src), vu = __ldg(V + src);
    uint32_t kp, vp;
    const uint32_t kw = quantize8(ku, kp), vw = quantize8(vu, vp);
    if (!live) continue;
    const int slot = start + (int)t;
    uint8_t* page = kv4_page(c, b, slot >> 6, head);
    if (!page) {
      atomicOr(a.status, VS_DEVFLAG_BOUNDS);
      continue;
    }
    const int r = slot & 63;
    *reinterpret_cast<uint32_t*>(page + kv4_code_off(c.GR, 0, g, r) + 4 * w) = kw;
    *reinterpret_cast<uint32_t*>(page + kv4_code_off(c.GR, 1, g, r) + 4 * w) = vw;
    if (w == 0) {
      *reinterpret_cast<uint32_t*>(page + kv4_pair_off(c.GR, 0, g, r)) = kp;
      *reinterpret_cast<uint32_t*>(page + kv4_pair_off(c.GR, 1, g, r)) = vp;
    }
  }
  if (!a.acc && !a.pos) return;
  const int pos0 = (a.n_tokens ? a.n_tokens[b] : len) - n;
  for (uint32_t e = first; e < (uint32_t)n * c.Hkv; e += stride) {
    const int head = e / n, t = e - head * n;
    const int64_t out = ((int64_t)b * c.Hkv + head) * a.ld + start + t;
    if (a.acc) {
      float sum = 0.f;
      if (a.Av)
        for (int h = head * a.G; h < (head + 1) * a.G; ++h)
          sum += __ldg(a.Av + (int64_t)h * a.total + tok0 + t);
      a.acc[out] = sum;
    }
    if (a.pos) a.pos[out] = pos0 + t;
  }
}

__global__ void __launch_bounds__(kKv4Threads) kv4_read_kernel(Kv4ReadArgs a) {
  const Kv4Cache& c = a.c;
  const int b = blockIdx.y;
  int64_t tok0;
  int n, len;
  bool ok = seq_range(a.cu, a.total, a.max_read, b, tok0, n);
  ok = kv4_len(c, b, len) && ok;
  const int start = a.start ? a.start[b] : 0;
  ok = ok && start >= 0 && start <= len - n && len <= 64 * c.table_ld;
  if (!ok) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.status, VS_DEVFLAG_BOUNDS);
    return;
  }
  const uint32_t stride = gridDim.x * blockDim.x;
  const uint32_t line = c.Hkv * c.GR * 8, jobs = n * line;  // as in the append
  uint4* K = static_cast<uint4*>(a.K) + tok0 * (a.kv_stride / 8);
  uint4* V = static_cast<uint4*>(a.V) + tok0 * (a.kv_stride / 8);
  for (uint32_t e = blockIdx.x * blockDim.x + threadIdx.x; e < jobs; e += stride) {
    const uint32_t t = e / line, x = e - t * line;
    const int w = x & 7, g = (x >> 3) & (c.GR - 1), head = x / (8 * c.GR);
    const int slot = start + (int)t, r = slot & 63;
    const uint8_t* page = kv4_page(c, b, slot >> 6, head);
    const int64_t dst = (int64_t)t * (a.kv_stride / 8) + x;
    if (!page) {
      atomicOr(a.status, VS_DEVFLAG_BOUNDS);
      continue;
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint32_t word =
          __ldg(reinterpret_cast<const uint32_t*>(page + kv4_code_off(c.GR, kv, g, r)) + w);
      const uint32_t pair =
          __ldg(reinterpret_cast<const uint32_t*>(page + kv4_pair_off(c.GR, kv, g, r)));
      const float s = kv4_step(pair), m = kv4_min(pair);
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)  // s n is exact in fp32, so one rounding each: + m, then bf16
        o[i] = pack2(fmaf((float)((word >> (8 * i)) & 15u), s, m),
                     fmaf((float)((word >> (8 * i + 4)) & 15u), s, m));
      (kv ? V : K)[dst] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// Blocks per sequence: enough for the longest one, at most about 16 blocks an
// SM in all (each then strides over its share).
static int kv4_blocks(int B, int64_t jobs) {
  const int64_t most = ceil_div(16LL * device_sm_count(), B);
  const int64_t want = (jobs + kKv4Threads - 1) / kKv4Threads;
  return (int)(want < 1 ? 1 : (want < most ? want : most));
}

cudaError_t launch_kv4_append(const Kv4AppendArgs& a) {
  const dim3 grid(kv4_blocks(a.c.B, (int64_t)a.max_new * a.c.Hkv * a.c.GR * 8), a.c.B);
  kv4_append_kernel<<<grid, kKv4Threads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4ReadArgs& a) {
  const dim3 grid(kv4_blocks(a.c.B, (int64_t)a.max_read * a.c.Hkv * a.c.GR * 8), a.c.B);
  kv4_read_kernel<<<grid, kKv4Threads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace vs
