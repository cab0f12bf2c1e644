// The 4-bit paged key/value cache: format and addressing shared by its kernels
// (kv4.cu, kv4_evict.cu).
//
// A page holds 64 slots (tokens) of every KV head; the bytes of one (page,
// head) are contiguous, so that a page of one head is one bulk copy:
//   key codes   [d/64][64 slots][32 bytes]
//   value codes [d/64][64 slots][32 bytes]
//   key pairs   [d/64][64 slots] (s, m) as two bf16
//   value pairs [d/64][64 slots] (s, m)
// A slot's 64 channels of a group are eight 32-bit words; word w, nibble j
// (bits 4j..4j+3) is channel 8w + j, and code n stands for s n + m.
#pragma once
#include <cstdint>

#include "internal.h"

namespace vs {

constexpr int kKv4Page = 64;            // slots per page
constexpr int kKv4Group = 64;           // channels per (s, m) pair
constexpr int kKv4Codes = 64 * 32;      // bytes of codes per group and page
constexpr int kKv4Pairs = 64 * 4;       // bytes of pairs per group and page
constexpr int kKv4GroupBytes = 2 * (kKv4Codes + kKv4Pairs);  // K and V: 4608

struct Kv4Cache {
  uint8_t* pool;         // [n_pages][Hkv][GR * kKv4GroupBytes]
  int n_pages;
  const int32_t* table;  // [B][table_ld] page of slots [64 i, 64 i + 64)
  int64_t table_ld;
  const int32_t* lens;   // [B] slots in use
  int B, Hkv, GR;        // GR: groups per head, d / 64
  int max_len;           // host bound on lens
};

// Slots in use of sequence b; a length outside [0, max_len] counts as 0 and
// returns false (callers flag VS_DEVFLAG_BOUNDS).
__device__ __forceinline__ bool kv4_len(const Kv4Cache& c, int b, int& n) {
  n = c.lens[b];
  if (n >= 0 && n <= c.max_len) return true;
  n = 0;
  return false;
}

// The bytes of (page, head), or null for a page outside the pool.
__device__ __forceinline__ uint8_t* kv4_page(const Kv4Cache& c, int b, int page, int head) {
  const int id = __ldg(c.table + (int64_t)b * c.table_ld + page);
  if (id < 0 || id >= c.n_pages) return nullptr;
  return c.pool + ((int64_t)id * c.Hkv + head) * (c.GR * kKv4GroupBytes);
}

// Byte offsets inside a (page, head); kv 0: keys, 1: values.
__host__ __device__ __forceinline__ int kv4_code_off(int GR, int kv, int g, int slot) {
  return (kv * GR + g) * kKv4Codes + slot * 32;
}
__host__ __device__ __forceinline__ int kv4_pair_off(int GR, int kv, int g, int slot) {
  return 2 * GR * kKv4Codes + (kv * GR + g) * kKv4Pairs + slot * 4;
}

__device__ __forceinline__ float kv4_step(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float kv4_min(uint32_t pair) {
  return __uint_as_float(pair & 0xffff0000u);
}

// A second kernel that starts while the first drains (programmatic dependent
// launch): the first calls launch_dependents, the second waits for all of the
// first's writes before it touches anything.
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_previous_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <class... P, class... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t stream,
                                A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

struct Kv4AppendArgs {
  Kv4Cache c;
  const void* K;
  const void* V;
  int64_t kv_stride, total;
  const int32_t* cu;
  int max_new;
  const int32_t* n_tokens;  // or null: the lengths
  const float* Av;          // [Hq][total] or null
  int G;                    // query heads per KV head
  float* acc;               // [B][Hkv][ld] or null
  int32_t* pos;             // likewise
  int64_t ld;
  int* status;
  cudaStream_t stream;
};
cudaError_t launch_kv4_append(const Kv4AppendArgs& a);

struct Kv4ReadArgs {
  Kv4Cache c;
  const int32_t* start;  // [B] first slot, or null: 0
  const int32_t* cu;
  int64_t total;
  int max_read;
  void* K;
  void* V;
  int64_t kv_stride;
  int* status;
  cudaStream_t stream;
};
cudaError_t launch_kv4_read(const Kv4ReadArgs& a);

struct Kv4DecodeArgs {
  Kv4Cache c;
  const void* Q;
  int64_t q_stride;
  int Hq, G;
  float scale;
  int window, sinks;  // window 0: every slot
  void* O;
  float* lse;           // [Hq][B] or null
  const float* acc_in;  // [B][Hkv][ld] or null
  float* acc_out;       // or null
  int64_t ld;
  void* ws;
  cudaStream_t stream;
};
size_t kv4_decode_ws_bytes(int B, int Hq, int Hkv, int d, int max_len, bool weights);
cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a);

struct Kv4EvictArgs {
  Kv4Cache c;
  const int32_t* n_tokens;
  const float* acc_in;
  const int32_t* pos_in;
  int64_t ld_in;
  int keep, sinks, recent;
  int32_t* lens_out;
  float* acc_out;
  int32_t* pos_out;
  int64_t ld_out;
  void* ws;
  cudaStream_t stream;
};
size_t kv4_evict_ws_bytes(int B, int Hkv, int max_len, int keep);
cudaError_t launch_kv4_evict(const Kv4EvictArgs& a);

}  // namespace vs
