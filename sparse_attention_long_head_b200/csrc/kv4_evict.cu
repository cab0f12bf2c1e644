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
// Two kernels.  The first finds who stays, one cluster of 1 to 8 CTAs a row: each
// thread keeps up to 32 slots of the row as order-preserving 32-bit keys in
// registers (at 32 of them some 25 words a thread go through local memory once),
// the boundary key is found digit by digit (four of 8 bits) over
// histograms that the cluster sums through distributed shared memory, and
// ballots in slot order give the lists of holes and of the slots that fill
// them.  Bound by latency (some ten cluster barriers and the row read once, 8
// bytes a slot).  The second moves, 16 lanes a move over the whole device.
// On new data 256 rows of 4200 to 4352 slots cut to 4096 take 34 us, 16 rows of
// 100,000 to 131,072 slots cut to 8192 take 63 to 65 us (123,000 moves of 144
// bytes in pieces of 32 and 4); by themselves the kernels take 16 and 16 (three
// dependent loads a move), 36 and 27.  Data that L2 still holds: 27 and 60 in all.
#include <cooperative_groups.h>

#include "kv4.cuh"

namespace vs {

namespace cg = cooperative_groups;

constexpr int kEvMaxCluster = 8;

// Larger keys stay first: fixed slots, then +inf .. -inf, then NaN.
__device__ __forceinline__ uint32_t evict_key(float w, bool fixed) {
  if (fixed) return 0xffffffffu;
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);  // -0 ties with 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct EvictShared {
  uint32_t hist[4][256];  // one per digit, read by the cluster
  uint32_t merged[256];
  uint32_t warp_a[32], warp_b[32];
  uint32_t total_a, total_b;  // read by the cluster
};

// Where a histogram keeps digit d: lane l of a warp reads digits 255 - 8 l - i,
// i = 0..7, without bank conflicts.
__device__ __forceinline__ uint32_t bin_at(uint32_t d) {
  return 32 * ((255 - d) & 7) + ((255 - d) >> 3);
}

// kEvThreads threads of V slots each.
template <int kEvThreads, int V>
__global__ void __launch_bounds__(kEvThreads, kEvThreads == 512 ? 2 : 1)
    kv4_evict_kernel(Kv4EvictArgs a, int32_t* counts, int32_t* lists, int64_t list_ld) {
  launch_dependents();  // every CTA is resident or done by the time the moves start
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  auto sync_all = [&]() {
    if (C == 1) __syncthreads();
    else cl.sync();
  };
  const Kv4Cache& c = a.c;
  constexpr int kEvWarps = kEvThreads / 32;
  const int row = blockIdx.x / C;  // b * Hkv + head
  const int b = row / c.Hkv, head = row % c.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ EvictShared sh;
  int* status = static_cast<int*>(a.ws);

  int n;
  const bool ok = kv4_len(c, b, n) && n <= 64 * c.table_ld && n <= a.ld_in;
  if (!ok) {  // uniform over the cluster: an empty row
    if (rank == 0 && tid == 0) {
      atomicOr(status, VS_DEVFLAG_BOUNDS);
      if (head == 0) a.lens_out[b] = 0;
      counts[row] = 0;
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
    if (rank == 0 && tid == 0) counts[row] = 0;
    for (int t = rank * kEvThreads + tid; t < n; t += C * kEvThreads) {
      acc_out[t] = acc[t];
      pos_out[t] = pos[t];
    }
    return;
  }
  // this CTA's slots [s0, s1); this warp's [w0, w1), at most 32 V of them;
  // key j of a lane is slot w0 + 32 j + lane
  const int slice = ((n + C - 1) / C + 31) / 32 * 32;
  const int s0 = min(rank * slice, n), s1 = min(s0 + slice, n);
  const int wper = ((s1 - s0 + kEvWarps - 1) / kEvWarps + 31) / 32 * 32;
  const int w0 = min(s0 + warp * wper, s1), w1 = min(w0 + wper, s1);
  const int64_t newest = (int64_t)a.n_tokens[b] - a.recent;
  for (int i = tid; i < 4 * 256; i += kEvThreads) sh.hist[i >> 8][i & 255] = 0;
  uint32_t key[V];
  {
    const float* pa = acc + w0 + lane;
    const int32_t* pp = pos + w0 + lane;
    float w[V];
    int p[V];
    if (w0 + 32 * V <= n) {  // no guards: one address, all loads in flight
#pragma unroll
      for (int j = 0; j < V; ++j) w[j] = __ldg(pa + 32 * j);
#pragma unroll
      for (int j = 0; j < V; ++j) p[j] = __ldg(pp + 32 * j);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const bool in = w0 + 32 * j + lane < n;
        w[j] = in ? __ldg(pa + 32 * j) : 0.f;
        p[j] = in ? __ldg(pp + 32 * j) : 0;
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = evict_key(w[j], p[j] < a.sinks || p[j] >= newest);
  }
  auto live = [&](int j) { return w0 + 32 * j + lane < w1; };

  // Boundary key: the k-th largest.  `need` slots are still to be found among
  // the `equal` ones whose key begins with `prefix`.
  uint32_t prefix = 0, need = k, equal = n;
  int low = 32;  // bits below the digits found so far
  __syncthreads();  // the histograms are zero
#pragma unroll
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (w0 + 32 * j >= w1) break;  // uniform over the warp
      if (live(j) && (pass == 0 || (key[j] >> (shift + 8)) == prefix))
        atomicAdd(&sh.hist[pass][bin_at((key[j] >> shift) & 255u)], 1u);
    }
    sync_all();
    const uint32_t* merged = sh.hist[pass];
    if (C > 1) {
      if (tid < 256) {
        uint32_t x[kEvMaxCluster];
#pragma unroll
        for (int r = 0; r < kEvMaxCluster; ++r)  // all reads in flight
          x[r] = r < C ? cl.map_shared_rank(sh.hist[pass], r)[tid] : 0u;
        uint32_t sum = 0;
#pragma unroll
        for (int r = 0; r < kEvMaxCluster; ++r) sum += x[r];
        sh.merged[tid] = sum;
      }
      __syncthreads();
      merged = sh.merged;
    }
    // every warp takes the same decision: lane l holds bins 255 - 8 l downwards
    uint32_t part[8], mine = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      part[i] = merged[32 * i + lane];  // bin 255 - (8 lane + i)
      mine += part[i];
    }
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    uint32_t before = incl - mine, digit = 0, count = 0, above = 0;
    const bool here = before < need && need <= incl;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (before < need && need <= before + part[i]) {
        digit = 255 - (8 * lane + i);
        count = part[i];
        above = before;
      }
      before += part[i];
    }
    const int from = __ffs(__ballot_sync(0xffffffffu, here)) - 1;  // need <= the sum of all bins
    prefix = (prefix << 8) | __shfl_sync(0xffffffffu, digit, from);
    equal = __shfl_sync(0xffffffffu, count, from);
    need -= __shfl_sync(0xffffffffu, above, from);
    low = shift;
    if (equal == need) break;  // uniform over the cluster: all that begin with prefix stay
  }
  // Larger keys stay, and `need` of the `equal` slots with this key, the lowest
  // ones (all of them, from this key up, where the search ended early).
  const uint32_t bound = prefix << low;

  // this warp's counts x, y -> the counts of all earlier warps of the cluster
  auto exchange = [&](uint32_t x, uint32_t y, uint32_t& before_x, uint32_t& before_y) {
    if (lane == 0) {
      sh.warp_a[warp] = x;
      sh.warp_b[warp] = y;
    }
    __syncthreads();
    uint32_t ax = lane < kEvWarps ? sh.warp_a[lane] : 0u, bx = lane < kEvWarps ? sh.warp_b[lane] : 0u;
#pragma unroll
    for (int o = 1; o < kEvWarps; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, ax, o), v = __shfl_up_sync(0xffffffffu, bx, o);
      if (lane >= o) {
        ax += u;
        bx += v;
      }
    }
    before_x = __shfl_sync(0xffffffffu, ax, warp) - x;
    before_y = __shfl_sync(0xffffffffu, bx, warp) - y;
    if (C == 1) {
      __syncthreads();  // read before the next exchange writes
      return;
    }
    if (tid == kEvWarps - 1) {
      sh.total_a = ax;
      sh.total_b = bx;
    }
    cl.sync();
    uint32_t ox = lane < rank ? *cl.map_shared_rank(&sh.total_a, lane) : 0u;
    uint32_t oy = lane < rank ? *cl.map_shared_rank(&sh.total_b, lane) : 0u;
    before_x += __reduce_add_sync(0xffffffffu, ox);
    before_y += __reduce_add_sync(0xffffffffu, oy);
    cl.sync();  // read before the next exchange writes, and before any CTA leaves
  };
  const uint32_t below_lane = (1u << lane) - 1u;
  uint32_t ties_before = 0;  // boundary keys of earlier warps
  if (equal != need) {       // uniform over the cluster
    uint32_t eq = 0, none;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (w0 + 32 * j >= w1) break;
      eq += __popc(__ballot_sync(0xffffffffu, live(j) && key[j] == bound));
    }
    exchange(eq, 0, ties_before, none);
  }
  // who stays: bit j of `stay` for key j
  uint32_t stay = 0;
  uint32_t holes = 0, movers = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (w0 + 32 * j >= w1) break;
    const int t = w0 + 32 * j + lane;
    const bool tie = t < w1 && key[j] == bound;
    bool s = t < w1 && (key[j] > bound || tie);
    if (equal != need) {
      const uint32_t ties = __ballot_sync(0xffffffffu, tie);
      if (tie && ties_before + __popc(ties & below_lane) >= need) s = false;
      ties_before += __popc(ties);
    }
    if (s) stay |= 1u << j;
    holes += __popc(__ballot_sync(0xffffffffu, t < w1 && t < k && !s));
    movers += __popc(__ballot_sync(0xffffffffu, t >= k && s));
  }
  uint32_t hole_at, mover_at;
  exchange(holes, movers, hole_at, mover_at);
  if (rank == C - 1 && warp == kEvWarps - 1 && lane == 0) counts[row] = (int)(hole_at + holes);
  int32_t* hole_list = lists + (int64_t)row * 2 * list_ld;
  int32_t* mover_list = hole_list + list_ld;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (w0 + 32 * j >= w1) break;
    const int t = w0 + 32 * j + lane;
    const bool s = (stay >> j) & 1u;
    const bool hole = t < w1 && t < k && !s, mover = t >= k && s;
    const uint32_t hb = __ballot_sync(0xffffffffu, hole), mb = __ballot_sync(0xffffffffu, mover);
    if (hole) hole_list[hole_at + __popc(hb & below_lane)] = t;
    if (mover) mover_list[mover_at + __popc(mb & below_lane)] = t;
    hole_at += __popc(hb);
    mover_at += __popc(mb);
  }
  // the entries of the slots that keep their place, a few loads in flight
  constexpr int kBatch = V < 8 ? V : 8;
#pragma unroll
  for (int j0 = 0; j0 < V; j0 += kBatch) {
    if (w0 + 32 * j0 >= min(k, w1)) break;  // uniform over the warp
    float w[kBatch];
    int p[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int t = 32 * (j0 + j);
      const bool in = w0 + t + lane < k;  // k <= n
      w[j] = in ? __ldg(acc + w0 + lane + t) : 0.f;
      p[j] = in ? __ldg(pos + w0 + lane + t) : 0;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int t = w0 + 32 * (j0 + j) + lane;
      if (((stay >> (j0 + j)) & 1u) && t < k) {
        acc_out[t] = w[j];
        pos_out[t] = p[j];
      }
    }
  }
}

// The moves of row blockIdx.y: sixteen lanes a move (16-byte pieces of the
// codes, the pairs, the entries of acc and pos).  One move a lane and turn, as
// many blocks as are resident at once: two moves in flight take the same, four
// at half the threads 5% more, two or four times the blocks 2% and 5% more.
constexpr int kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads, 8)
    kv4_move_kernel(Kv4EvictArgs a, const int32_t* counts, const int32_t* lists, int64_t list_ld) {
  wait_for_previous_kernel();
  const Kv4Cache& c = a.c;
  const int row = blockIdx.y, b = row / c.Hkv, head = row % c.Hkv;
  const int moves = __ldcg(counts + row);
  const int32_t* hole_list = lists + (int64_t)row * 2 * list_ld;
  const int32_t* mover_list = hole_list + list_ld;
  const int groups = gridDim.x * (kMoveThreads / 16);
  const int sub = threadIdx.x & 15, codes = 4 * c.GR;
  // what this lane copies: offset of its piece in slot 0's, and per slot
  int off = 0, step = 0;
  if (sub < codes) {
    off = kv4_code_off(c.GR, sub / (2 * c.GR), (sub >> 1) % c.GR, 0) + 16 * (sub & 1);
    step = 32;
  } else if (sub < codes + 2 * c.GR) {
    off = kv4_pair_off(c.GR, (sub - codes) / c.GR, (sub - codes) % c.GR, 0);
    step = 4;
  }
  for (int i = blockIdx.x * (kMoveThreads / 16) + threadIdx.x / 16; i < moves; i += groups) {
    const int dst = __ldcg(hole_list + i), src = __ldcg(mover_list + i);
    if (sub == 14) {
      a.acc_out[(int64_t)row * a.ld_out + dst] = __ldg(a.acc_in + (int64_t)row * a.ld_in + src);
      continue;
    }
    if (sub == 15) {
      a.pos_out[(int64_t)row * a.ld_out + dst] = __ldg(a.pos_in + (int64_t)row * a.ld_in + src);
      continue;
    }
    uint8_t* pd = kv4_page(c, b, dst >> 6, head);
    const uint8_t* ps = kv4_page(c, b, src >> 6, head);
    if (!pd || !ps) {
      if (sub == 0) atomicOr(static_cast<int*>(a.ws), VS_DEVFLAG_BOUNDS);
      continue;
    }
    pd += off + step * (dst & 63);
    ps += off + step * (src & 63);
    if (step == 32) *reinterpret_cast<uint4*>(pd) = *reinterpret_cast<const uint4*>(ps);
    else if (step == 4) *reinterpret_cast<uint32_t*>(pd) = *reinterpret_cast<const uint32_t*>(ps);
  }
}

// As many moves at most: holes are among the `keep` first slots, what fills
// them among the others.
static int64_t evict_moves(int max_len, int keep) {
  if (keep >= max_len) return 0;
  return keep < max_len - keep ? keep : max_len - keep;
}

size_t kv4_evict_ws_bytes(int B, int Hkv, int max_len, int keep) {
  const size_t rows = (size_t)B * Hkv;
  return align_up(kStatusBytes + sizeof(int32_t) * rows * (1 + 2 * (size_t)evict_moves(max_len, keep)),
                  256);
}

template <int kEvThreads, int V>
static cudaError_t launch_evict_impl(const Kv4EvictArgs& a, int C, int32_t* counts, int32_t* lists,
                                     int64_t list_ld) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.c.B * a.c.Hkv * C));
  cfg.blockDim = dim3(kEvThreads);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = C;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_evict_kernel<kEvThreads, V>, a, counts, lists, list_ld);
}

cudaError_t launch_kv4_evict(const Kv4EvictArgs& a) {
  cudaError_t e = cudaMemsetAsync(a.ws, 0, sizeof(int), a.stream);
  if (e != cudaSuccess) return e;
  const int rows = a.c.B * a.c.Hkv, sms = device_sm_count();
  int32_t* counts = reinterpret_cast<int32_t*>(static_cast<char*>(a.ws) + kStatusBytes);
  int32_t* lists = counts + rows;
  const int64_t list = evict_moves(a.c.max_len, a.keep);
  // Rows of up to 8192 slots take one CTA of 512 threads (two fit an SM, and no
  // cluster barrier is needed).  Longer rows take clusters: as many CTAs as the
  // slots need, more while the device has SMs to spare, of 512 threads (at most
  // 15 clusters of 8 CTAs of 1024 threads fit the device: 16 rows of 131072
  // slots took two turns, 70 against 67 us), above 131072 slots of 1024.
  const int n = a.c.max_len;
  int C = 1;
  if (n > 8192)
    while (C < kEvMaxCluster && (C * 16384 < n || 2 * rows * C <= sms)) C *= 2;
  if (n <= 2048) e = launch_evict_impl<512, 4>(a, C, counts, lists, list);
  else if (n <= 8192) e = launch_evict_impl<512, 16>(a, C, counts, lists, list);
  else if (C * 4096 >= n) e = launch_evict_impl<1024, 4>(a, C, counts, lists, list);
  else if (C * 16384 >= n) e = launch_evict_impl<512, 32>(a, C, counts, lists, list);
  else e = launch_evict_impl<1024, 32>(a, C, counts, lists, list);
  if (e != cudaSuccess || list == 0) return e;
  const int64_t per_block = kMoveThreads / 16;
  const int64_t want = (list + per_block - 1) / per_block, cap = ceil_div(8LL * sms, rows);
  return launch_after(kv4_move_kernel, dim3((unsigned)(want < cap ? want : cap), rows),
                      kMoveThreads, a.stream, a, (const int*)counts, (const int*)lists, list);
}

}  // namespace vs
