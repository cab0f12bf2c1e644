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
// The floor of both kernels is memory: 4 d bytes of bf16 K and V and 9/8 d bytes
// of cache per token and head.  50,413 tokens of 8 heads, d = 128 (265 MB):
// append 90 us, bound by instruction issue (3.2 of 4 a cycle, some 370 per warp
// and 512 values; the ALU pipe at 69%), read 54 us, 4.9 TB/s.  Eight
// lanes take one group of one slot (16 bytes of K and of V each), so every access
// is a full 32- or 128-byte piece.
#include <cuda_bf16.h>

#include "kv4.cuh"

namespace vs {

constexpr int kKv4Threads = 256;

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {  // NaN if either is
  const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<__nv_bfloat162*>(&a),
                                       *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&a),
                                       *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ __nv_bfloat162 abs2(uint32_t a) {
  a &= 0x7fff7fffu;
  return *reinterpret_cast<__nv_bfloat162*>(&a);
}
__device__ __forceinline__ float bf16_at(const uint32_t (&v)[4], int i) {
  return __uint_as_float(i & 1 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
}

// Two fp32 in one register pair; one instruction for both (append 93 -> 90 us).
__device__ __forceinline__ uint64_t pair2(uint32_t lo, uint32_t hi) {
  return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ uint64_t both(float x) {
  return pair2(__float_as_uint(x), __float_as_uint(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Adding this to x in [0, 2^22) leaves rint(x) in the low bits.
constexpr float kRound = 12582912.f;  // 1.5 2^23
constexpr uint32_t kRoundBits = 0x4b400000u;

// Codes of this lane's eight channels and the pair of the group that the
// eight lanes of an aligned octet hold (the whole warp must call it).  No
// conversion instructions (their unit is narrow): rounding and integers come
// from the addition of kRound.
__device__ __forceinline__ uint32_t quantize8(const uint4& u, uint32_t& pair) {
  const uint32_t v[4] = {u.x, u.y, u.z, u.w};
  const uint32_t mn = min2(min2(v[0], v[1]), min2(v[2], v[3]));
  const uint32_t mx = max2(max2(v[0], v[1]), max2(v[2], v[3])) ^ 0x80008000u;
  uint32_t ends = min2(__byte_perm(mn, mx, 0x5410), __byte_perm(mn, mx, 0x7632));  // min, -max
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) ends = min2(ends, __shfl_xor_sync(0xffffffffu, ends, o));
  const float lo = __uint_as_float(ends << 16), hi = -__uint_as_float(ends & 0xffff0000u);
  if (!(lo > -INFINITY && hi < INFINITY)) {  // also where either is NaN
    pair = 0x7fc07fc0u;
    return 0u;
  }
  // (hi - lo) / 15 to within 2^-22: the bf16 it rounds to, unless its low half
  // is next to 0x8000 or it is not well inside the normal range
  float range = (hi - lo) * (1.f / 15.f);
  const int low = (int)(__float_as_uint(range) & 0xffffu) - 0x8000;
  const bool normal = range > 1e-30f && range < 1e37f;
  if ((low < 8 && low > -8) || !normal) range = (float)(((double)hi - (double)lo) / 15.0);
  const __nv_bfloat16 sb = __float2bfloat16_rn(range);
  const float s = __bfloat162float(sb);
  pair = (uint32_t)__bfloat16_as_ushort(sb) | (ends << 16);
  if (s == 0.f) return 0u;
  // q = (x - lo) / s, the product corrected once by the remainder: a quotient
  // that is a whole number and a half comes out as such, and no other does,
  // for (x - lo) - (n + 1/2) s is a multiple of the smallest unit in the last
  // place among x, lo and s / 2, hence 0 or above 2^-24 (x - lo) -- unless x
  // or lo is below 2^-16 of the range (and not 0; 2^-15 is tested).
  const float tiny = range * (15.f * 0x1p-15f);
  bool exact = normal && (fabsf(lo) >= tiny || lo == 0.f);
  const __nv_bfloat162 least = __hmin2(__hmin2(abs2(v[0]), abs2(v[1])), __hmin2(abs2(v[2]), abs2(v[3])));
  if (!(fminf(__low2float(least), __high2float(least)) >= tiny)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) exact &= fabsf(bf16_at(v, i)) >= tiny || bf16_at(v, i) == 0.f;
  }
  const float r = __fdividef(1.f, s);  // to 2^-22
  const uint64_t r2 = both(r), minus_s = both(-s), minus_lo = both(-lo), round2 = both(kRound);
  uint32_t word = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    const uint64_t d = add2(pair2(v[i] << 16, v[i] & 0xffff0000u), minus_lo);
    const uint64_t q = mul2(d, r2);
    const uint64_t x = add2(fma2(fma2(q, minus_s, d), r2, q), round2);  // below 15.1
    word = (word * 16u + (uint32_t)(x >> 32)) * 16u + (uint32_t)x;
  }
  word -= kRoundBits * 0x11111111u;  // of all eight
  if (!exact) {  // quotients next to a half, or overflowed, in 64 bits
    word = 0;
    for (int i = 7; i >= 0; --i) {
      const float d = bf16_at(v, i) - lo, q = d * r;
      float n = (q + kRound) - kRound;
      if (!normal || !(fabsf(q - n) < 0.4999f))
        n = (float)rint(fmin(((double)bf16_at(v, i) - (double)lo) / (double)s, 15.0));
      word = word * 16u + (uint32_t)n;
    }
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
  // job e = t line + x is 16-byte piece x of token t's row; both move on by
  // `stride` jobs without a division
  const uint32_t dt = stride / line, dx = stride - dt * line;
  uint32_t t = first / line, x = first - t * line;
  auto load = [&](uint32_t t, uint32_t x, uint4& k, uint4& v) {
    const int64_t src = (int64_t)t * (a.kv_stride / 8) + x;
    k = __ldg(K + src);
    v = __ldg(V + src);
  };
  uint4 kn = make_uint4(0, 0, 0, 0), vn = kn;  // the next job's, loaded one turn ahead
  if (first < jobs) load(t, x, kn, vn);
  for (uint32_t base = first - (threadIdx.x & 31); base < jobs; base += stride) {
    const bool live = base + (threadIdx.x & 31) < jobs;
    const uint4 ku = kn, vu = vn;
    const int slot = start + (int)t;
    const int w = x & 7, g = (x >> 3) & (c.GR - 1), head = x >> (c.GR == 1 ? 3 : 4);
    t += dt;
    x += dx;
    if (x >= line) {
      x -= line;
      ++t;
    }
    if (base + stride + (threadIdx.x & 31) < jobs) load(t, x, kn, vn);
    uint32_t kp, vp;
    const uint32_t kw = quantize8(ku, kp), vw = quantize8(vu, vp);
    if (!live) continue;
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

// Code i of a word as a float.
__device__ __forceinline__ float code(uint32_t word, int i) {
  return __uint_as_float(((word >> (4 * i)) & 15u) | kRoundBits) - kRound;
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
  const uint32_t dt = stride / line, dx = stride - dt * line;
  uint32_t e = blockIdx.x * blockDim.x + threadIdx.x, t = e / line, x = e - t * line;
  for (; e < jobs; e += stride, t += dt, x += dx) {
    if (x >= line) {
      x -= line;
      ++t;
    }
    const int w = x & 7, g = (x >> 3) & (c.GR - 1), head = x >> (c.GR == 1 ? 3 : 4);
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
        o[i] = pack2(fmaf(code(word, 2 * i), s, m), fmaf(code(word, 2 * i + 1), s, m));
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
