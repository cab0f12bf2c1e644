// Eviction from the 4-bit paged cache by accumulated attention weight.
//
// Of a (sequence, KV head) row's n slots k = min(n, keep) stay: first those
// whose position is fixed (the first `sinks` tokens and the last `recent`
// ones), then by accumulated weight, descending (NaN after -inf), ties to the
// lower slot.  Attention does not depend on the order of the slots, so slots
// below k that stay do not move: the i-th slot below k that goes is
// overwritten by the i-th slot at or above k that stays.  Sources and
// destinations are disjoint, so all moves run at once, and a cache at its
// budget moves only as many slots as it lost.
//
// Bound by latency and by the weights and positions read once (8 bytes a
// slot); a cluster of 1 to 8 CTAs takes a row.  Each CTA keeps its slice of
// the row as order-preserving 32-bit keys in shared memory; the boundary key
// is found by a most-significant-digit search (digits of 11, 11 and 10 bits)
// over histograms that the cluster sums through distributed shared memory;
// then slots are counted and listed by warp ballots in slot order.
#include <cooperative_groups.h>

#include "kv4.cuh"

namespace vs {

namespace cg = cooperative_groups;

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvMaxCluster = 8;
constexpr int kEvBins = 2048;
// a row gets a cluster wide enough for slices of this many slots, up to 8 CTAs
constexpr int kEvSlice = 4096;

// Larger keys stay first: fixed slots, then +inf .. -inf, then NaN.
__device__ __forceinline__ uint32_t evict_key(float w, bool fixed) {
  if (fixed) return 0xffffffffu;
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);  // -0 ties with 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct EvictShared {
  uint32_t hist[kEvBins];
  uint32_t warp_a[kEvWarps], warp_b[kEvWarps];
  uint32_t total_a, total_b;  // read by the cluster
  uint32_t digit, above;
};

__global__ void __launch_bounds__(kEvThreads) kv4_evict_kernel(Kv4EvictArgs a, int32_t* lists,
                                                              int64_t list_ld) {
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const Kv4Cache& c = a.c;
  const int row = blockIdx.x / C;  // b * Hkv + head
  const int b = row / c.Hkv, head = row % c.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  extern __shared__ uint32_t keys[];
  __shared__ EvictShared sh;
  int* status = static_cast<int*>(a.ws);

  int n;
  const bool ok = kv4_len(c, b, n) && n <= 64 * c.table_ld && n <= a.ld_in;
  if (!ok) {  // uniform over the cluster: an empty row
    if (rank == 0 && tid == 0) {
      atomicOr(status, VS_DEVFLAG_BOUNDS);
      if (head == 0) a.lens_out[b] = 0;
    }
    return;
  }
  const int k = min(n, a.keep);
  const float* acc = a.acc_in + (int64_t)row * a.ld_in;
  const int32_t* pos = a.pos_in + (int64_t)row * a.ld_in;
  float* acc_out = a.acc_out + (int64_t)row * a.ld_out;
  int32_t* pos_out = a.pos_out + (int64_t)row * a.ld_out;
  if (rank == 0 && tid == 0 && head == 0) a.lens_out[b] = k;
  if (n == k) {
    for (int t = rank * kEvThreads + tid; t < n; t += C * kEvThreads) {
      acc_out[t] = acc[t];
      pos_out[t] = pos[t];
    }
    return;
  }
  // this CTA's slots [s0, s1), this warp's [w0, w1), in multiples of 32
  const int slice = ((n + C - 1) / C + 31) / 32 * 32;
  const int s0 = min(rank * slice, n), s1 = min(s0 + slice, n);
  const int wper = ((s1 - s0 + kEvWarps - 1) / kEvWarps + 31) / 32 * 32;
  const int w0 = min(s0 + warp * wper, s1), w1 = min(w0 + wper, s1);
  const int64_t newest = (int64_t)a.n_tokens[b] - a.recent;
  for (int t = s0 + tid; t < s1; t += kEvThreads) {
    const int p = pos[t];
    keys[t - s0] = evict_key(acc[t], p < a.sinks || p >= newest);
  }
  __syncthreads();

  // boundary key: the k-th largest.  `need` slots are still to be found among
  // those whose key begins with `prefix`.
  uint32_t prefix = 0, need = k;
  int shift = 32;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10, bins = 1 << bits;
    const int high = shift;  // bits above this digit are fixed to prefix
    shift -= bits;
    for (int i = tid; i < bins; i += kEvThreads) sh.hist[i] = 0;
    __syncthreads();
    for (int t = tid; t < s1 - s0; t += kEvThreads) {
      const uint32_t x = keys[t];
      if (pass == 0 || (x >> high) == prefix) atomicAdd(&sh.hist[(x >> shift) & (bins - 1)], 1u);
    }
    cl.sync();
    // sums over the cluster, thread i taking bins of its own contiguous piece,
    // highest bins first
    const int per = bins / kEvThreads;  // 4 or 2
    uint32_t mine = 0, part[4];
    for (int j = 0; j < per; ++j) {
      const int bin = bins - 1 - (tid * per + j);
      uint32_t x = 0;
      for (int r = 0; r < C; ++r) x += cl.map_shared_rank(sh.hist, r)[bin];
      part[j] = x;
      mine += x;
    }
    // exclusive prefix over the threads
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sh.warp_a[warp] = incl;
    __syncthreads();
    uint32_t before = incl - mine;
    for (int w = 0; w < warp; ++w) before += sh.warp_a[w];
    for (int j = 0; j < per; ++j) {
      if (before < need && need <= before + part[j]) {
        sh.digit = bins - 1 - (tid * per + j);
        sh.above = before;
      }
      before += part[j];
    }
    cl.sync();  // also: the histograms are read before they are cleared
    prefix = (prefix << bits) | sh.digit;
    need -= sh.above;
  }
  const uint32_t bound = prefix;  // `need` of the slots with this key stay, the lowest ones

  // ranks in slot order: of boundary keys first, then of holes and movers
  auto exchange = [&](uint32_t x, uint32_t y, uint32_t& before_x, uint32_t& before_y) {
    // x, y: this warp's counts -> counts of all earlier warps of the cluster
    if (lane == 0) {
      sh.warp_a[warp] = x;
      sh.warp_b[warp] = y;
    }
    __syncthreads();
    before_x = before_y = 0;
    uint32_t all_x = 0, all_y = 0;
    for (int w = 0; w < kEvWarps; ++w) {
      if (w == warp) {
        before_x = all_x;
        before_y = all_y;
      }
      all_x += sh.warp_a[w];
      all_y += sh.warp_b[w];
    }
    if (tid == 0) {
      sh.total_a = all_x;
      sh.total_b = all_y;
    }
    cl.sync();
    for (int r = 0; r < rank; ++r) {
      before_x += *cl.map_shared_rank(&sh.total_a, r);
      before_y += *cl.map_shared_rank(&sh.total_b, r);
    }
    cl.sync();  // read before the next exchange writes
  };
  const uint32_t below_lane = (1u << lane) - 1u;
  uint32_t eq = 0, eq_before, none;
  for (int t = w0 + lane; t - lane < w1; t += 32)
    eq += __popc(__ballot_sync(0xffffffffu, t < w1 && keys[t - s0] == bound));
  exchange(eq, 0, eq_before, none);
  // stays(t) for a warp's 32 slots at once; `seen`: boundary keys before them
  auto stays = [&](int t, uint32_t& seen) {
    const uint32_t x = t < w1 ? keys[t - s0] : 0u;
    const bool tie = t < w1 && x == bound;
    const uint32_t ties = __ballot_sync(0xffffffffu, tie);
    const bool s = t < w1 && (x > bound || (tie && seen + __popc(ties & below_lane) < need));
    seen += __popc(ties);
    return s;
  };
  uint32_t seen = eq_before, holes = 0, movers = 0, hole_at, mover_at;
  for (int t = w0 + lane; t - lane < w1; t += 32) {
    const bool s = stays(t, seen);
    holes += __popc(__ballot_sync(0xffffffffu, t < w1 && t < k && !s));
    movers += __popc(__ballot_sync(0xffffffffu, t >= k && s));
  }
  exchange(holes, movers, hole_at, mover_at);
  int32_t* hole_list = lists + (int64_t)row * 2 * list_ld;
  int32_t* mover_list = hole_list + list_ld;
  seen = eq_before;
  for (int t = w0 + lane; t - lane < w1; t += 32) {
    const bool s = stays(t, seen);
    const bool hole = t < w1 && t < k && !s, mover = t >= k && s;
    const uint32_t hb = __ballot_sync(0xffffffffu, hole), mb = __ballot_sync(0xffffffffu, mover);
    if (hole) hole_list[hole_at + __popc(hb & below_lane)] = t;
    if (mover) mover_list[mover_at + __popc(mb & below_lane)] = t;
    if (s && t < k) {
      acc_out[t] = acc[t];
      pos_out[t] = pos[t];
    }
    hole_at += __popc(hb);
    mover_at += __popc(mb);
  }
  // the moves: as many movers as holes in the whole row
  if (warp == kEvWarps - 1 && lane == 0) sh.total_b = hole_at;  // this CTA's last warp: all so far
  __threadfence();
  cl.sync();
  const int moves = (int)*cl.map_shared_rank(&sh.total_b, C - 1);
  // sixteen lanes a move: 16-byte pieces of the codes, then the pairs
  const int sub = tid & 15, codes = 4 * c.GR;
  for (int i = (rank * kEvThreads + tid) / 16; i < moves; i += C * kEvThreads / 16) {
    const int dst = __ldcg(hole_list + i), src = __ldcg(mover_list + i);
    uint8_t* pd = kv4_page(c, b, dst >> 6, head);
    const uint8_t* ps = kv4_page(c, b, src >> 6, head);
    if (!pd || !ps) {
      if (sub == 0) atomicOr(status, VS_DEVFLAG_BOUNDS);
    } else if (sub < codes) {  // piece: (K or V, group, half of 32 bytes)
      const int kv = sub / (2 * c.GR), g = (sub >> 1) % c.GR, off = 16 * (sub & 1);
      *reinterpret_cast<uint4*>(pd + kv4_code_off(c.GR, kv, g, dst & 63) + off) =
          *reinterpret_cast<const uint4*>(ps + kv4_code_off(c.GR, kv, g, src & 63) + off);
    } else if (sub < codes + 2 * c.GR) {
      const int kv = (sub - codes) / c.GR, g = (sub - codes) % c.GR;
      *reinterpret_cast<uint32_t*>(pd + kv4_pair_off(c.GR, kv, g, dst & 63)) =
          *reinterpret_cast<const uint32_t*>(ps + kv4_pair_off(c.GR, kv, g, src & 63));
    }
    if (sub == 14) acc_out[dst] = acc[src];
    if (sub == 15) pos_out[dst] = pos[src];
  }
  cl.sync();  // no CTA leaves while another may still read its shared memory
}

size_t kv4_evict_ws_bytes(int B, int Hkv, int max_len, int keep) {
  const int64_t list = max_len < keep ? max_len : keep;  // as many holes as slots kept at most
  return align_up(kStatusBytes + sizeof(int32_t) * 2 * (size_t)B * Hkv * (size_t)list, 256);
}

cudaError_t launch_kv4_evict(const Kv4EvictArgs& a) {
  cudaError_t e = cudaMemsetAsync(a.ws, 0, sizeof(int), a.stream);
  if (e != cudaSuccess) return e;
  int C = 1;
  while (C < kEvMaxCluster && (int64_t)C * kEvSlice < a.c.max_len) C *= 2;
  const int64_t slice = (ceil_div(a.c.max_len, C) + 31) / 32 * 32;
  const size_t smem = sizeof(uint32_t) * (size_t)slice;
  e = cudaFuncSetAttribute(kv4_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t list = a.c.max_len < a.keep ? a.c.max_len : a.keep;
  int32_t* lists = reinterpret_cast<int32_t*>(static_cast<char*>(a.ws) + kStatusBytes);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.c.B * a.c.Hkv * C));
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = C;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_evict_kernel, a, lists, list);
}

}  // namespace vs
