// Single-token attention over the 4-bit paged cache (format: kv4.cuh).
//
// For query head h of sequence b over the visible slots t of its KV head:
//     S_t = scale q . k_t,  O = sum_t softmax(S)_t v_t,   k_t, v_t = s n + m
// per group of 64 channels.  Neither K nor V is ever formed:
//     q . k = sum_g [ s q.n + m (q.1) ],   O = sum_g [ (p s) . n + (p . m) ],
// so the codes n go to the tensor cores as they are and s, m multiply scores
// and weights.  A code needs no conversion: the bits of an integer below 256
// are a bf16 too, n 2^-133 (subnormal below 128; the first normal binade
// continues the same line), which the tensor cores multiply exactly.  A word
// therefore gives its eight codes by four ANDs and one shift: bits 0..3 are n,
// bits 4..7 are 16 n.  The other operand makes up for the 2^-133: q is scaled
// by a power of two per head (max |q| to 2^118) and the weights carry 2^48
// throughout (in the exponential's argument, so that O and l share it).  The
// 16 of odd codes goes into q, and for V into the row's final factor.
// V is centred on code 8 (a second MMA with the constant -8 per V tile), so
// that the rounding of p s to bf16, the only rounding below fp32, acts on
// n - 8, as it would on the values themselves, and the running sums stay small.
//
// Its floor is the cache's bytes: 72 per slot, KV head and group (64 codes and
// pairs of K and V), at G = Hq / Hkv query heads each.  4 sequences of 120,000
// to 131,072 slots, 32/8 heads, d = 128 take 116 to 121 us on new data (73 to 76% of
// a copy; 109 us where the same cache is read again and L2 still holds a part);
// what bounds it there is instructions, 217 per 16 slots: the ALU pipe is busy
// 54% of the cycles and an issue slot 50%, with three warps a scheduler.  mma.sync m16n8k16 is
// used, not tcgen05: with 8 or 16 columns of useful work (the query heads of
// one KV head) the tensor rate is far from the bound, and operands made in
// registers go straight in, without a trip through shared or tensor memory.
//
// One CTA per SM.  All visible pages of all (sequence, KV head) rows form one
// list, cut into equal ranges, one per CTA, and these into one per warp.  A warp
// streams its pages (one contiguous bulk copy each) through two slots of its
// own and keeps its own online softmax; it writes the O of rows that lie
// wholly in its range and leaves an fp32 part of the others (at most two: the
// first and the last).  No warp waits for another before its range is done.
// Then the CTA joins its warps' parts row by row; a row that several CTAs share
// leaves one part per CTA, and the CTA that arrives last joins them in their
// order, so results do not depend on the timing.  No CTA waits for another.
#include <cuda_bf16.h>

#include "kv4.cuh"
#include "ptx.cuh"

namespace vs {

// 12 and 8 warps leave 168 and 255 registers a thread (three and two warps a
// scheduler), which the accumulators of 8 and 16 query heads need.  Two page
// slots each: 221 KB of shared memory at d = 128 with 12 warps.
template <int NT>
struct DecodeShape {
  static constexpr int kWarps = NT == 1 ? 12 : 8;
  static constexpr int kThreads = 32 * kWarps;
};
constexpr int kDecMaxWarps = 12;

// The weights carry 2^kShift (up to 2^8 more while the running maximum lags):
// V steps s from 2^-40 (below, the products with codes of 2^-133 lose bits) to
// 2^40, and minima m below 2^44 (above, 2^56 (15 s + m) summed over 2^24 slots
// overflows).
constexpr float kShift = 48.f;
constexpr int kDecMinPages = 12;  // per CTA, where the list is short

// Workspace: status and tickets (zeroed by the call), then two parts a CTA and
// two a warp, the rows' log2-sum-exp and the scores (the last two only where
// weights are asked for).
struct DecodeLayout {
  int HT = 0;       // query heads a row: 4, 8 or 16
  int HC = 1;       // rows per KV head
  int Gp = 0;       // scores per slot and KV head (G rounded up to even)
  int64_t slots = 0;
  size_t off_tick = 0, off_part = 0, off_lse = 0, off_score = 0, total = 0;
  size_t part_floats = 0;

  static DecodeLayout make(int B, int Hq, int Hkv, int d, int max_len, bool weights, int sms) {
    DecodeLayout L;
    const int G = Hq / Hkv;
    L.HT = G <= 4 ? 4 : G <= 8 ? 8 : 16;
    L.HC = (G + L.HT - 1) / L.HT;
    L.Gp = (G + 1) / 2 * 2;
    L.slots = (int64_t)ceil_div(max_len, kKv4Page) * kKv4Page;
    L.part_floats = (size_t)L.HT * (d + 2);
    L.off_tick = kStatusBytes;
    L.off_part = align_up(L.off_tick + sizeof(int) * (size_t)B * Hkv * L.HC, 256);
    L.off_lse = align_up(
        L.off_part + sizeof(float) * 2 * (size_t)sms * (1 + kDecMaxWarps) * L.part_floats, 256);
    L.off_score = L.off_lse;
    L.total = L.off_lse;
    if (weights) {
      L.off_score = align_up(L.off_lse + sizeof(float) * (size_t)B * Hq, 256);
      L.total = L.off_score + sizeof(float) * (size_t)B * Hkv * (size_t)L.slots * L.Gp;
    }
    return L;
  }
};

struct DecodeParams {
  Kv4Cache c;
  const __nv_bfloat16* Q;
  int64_t q_stride;
  int Hq, G, HC, Gp;
  float scale;  // times log2(e)
  int window, sinks;
  __nv_bfloat16* O;
  float* lse;
  int* status;
  int* ticket;
  float* parts;       // [gridDim][2] of the CTAs
  float* warp_parts;  // [gridDim][warps][2]
  float* lse2;   // [B][Hq] log2-sum-exp, or null
  float* score;  // [B][Hkv][slots][Gp] scores times scale, or null
  int64_t slots;
  uint64_t wait_limit_ns;
};

// Visible pages of a sequence of n slots: the pages of the first `sinks`
// slots that lie before the window's, then the window's (or all).
struct Visible {
  int first, gap, pages;  // page k of the list is k < first ? k : k + gap
};
__device__ __forceinline__ Visible visible_pages(int n, int window, int sinks) {
  const int np = (n + kKv4Page - 1) / kKv4Page;
  if (window == 0 || n <= window) return {np, 0, np};
  const int lo = (n - window) / kKv4Page;
  const int ns = min((min(sinks, n) + kKv4Page - 1) / kKv4Page, lo);
  return {ns, lo - ns, ns + np - lo};
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// D += A B, one m16n8k16 bf16 tile.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two 16 x 16 matrices of bytes, transposed; lane i gives the address of row i
// (mod 16) of matrix i / 16.  Lane (gid, tig) gets of matrix m, in r[2 m] and
// r[2 m + 1], the bytes of rows 4 tig .. 4 tig + 3 in columns gid and gid + 8.
__device__ __forceinline__ void load_bytes_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Transposes an 8 x 8 matrix of 16-bit values held one row per four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The same with nothing added: D = A B.
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Codes at bits 0..3 and at bits 4..7 of both 16-bit halves, as bf16 pairs
// n 2^-133 and 16 n 2^-133.
__device__ __forceinline__ uint32_t codes_lo(uint32_t x) { return x & 0x000f000fu; }
__device__ __forceinline__ uint32_t codes_hi(uint32_t x) { return x & 0x00f000f0u; }
constexpr uint32_t kMinus8 = 0x80088008u;    // -8 2^-133 twice
constexpr uint32_t kMinus128 = 0x80808080u;  // -128 2^-133 twice

// 2^(field - 127) as a float, field in [1, 254].
__device__ __forceinline__ float pow2_field(int field) {
  return __uint_as_float((uint32_t)field << 23);
}

__device__ __forceinline__ void axpy(float4& y, float a, const float4& x) {
  y.x = fmaf(a, x.x, y.x);
  y.y = fmaf(a, x.y, y.y);
  y.z = fmaf(a, x.z, y.z);
  y.w = fmaf(a, x.w, y.w);
}

// Where a CTA's or warp's walk over the list of pages stands.
struct Cursor {
  int b, head, hc;  // sequence, KV head, chunk of its query heads
  int k;            // page in the row's list
  Visible v;
};

__device__ __forceinline__ void cursor_load(const DecodeParams& P, Cursor& q) {
  int n;
  kv4_len(P.c, q.b, n);
  q.v = visible_pages(n, P.window, P.sinks);
}
// Moves the cursor on by `by` pages (it stays valid only within the list).
__device__ __forceinline__ void cursor_add(const DecodeParams& P, Cursor& q, int by) {
  q.k += by;
  while (q.k >= q.v.pages) {
    q.k -= q.v.pages;
    if (++q.hc < P.HC) continue;
    q.hc = 0;
    if (++q.head < P.c.Hkv) continue;
    q.head = 0;
    do {
      if (++q.b >= P.c.B) return;
      cursor_load(P, q);
    } while (q.v.pages == 0);
  }
}

// What a warp needs to know of a page in one of its slots.
struct PageNote {
  int b, head, hc;     // the row
  int k, pages, page;  // place in the row's list, the list's length, page (-1: not in the pool)
};

// A row that other CTAs have pages of too.
struct SharedRow {
  int start;      // list position of the row's first page
  int c0, parts;  // first CTA, and how many (0: no such row)
  int b, h0, heads, ticket;
};

__device__ __forceinline__ void write_lse(const DecodeParams& P, int b, int h, float M, float L) {
  const float l2 = L > 0.f ? M + (log2f(L) - kShift) : (L == 0.f ? -INFINITY : L);
  if (P.lse) P.lse[(int64_t)h * P.c.B + b] = l2 * 0.6931471805599453f;
  if (P.lse2) P.lse2[(int64_t)b * P.Hq + h] = l2;
}

// One warp joins head h of the parts x0 .. x1 in their order: M and L in every
// lane, four channels of the numerator in each of the first D / 4.
template <int D, int HR, class F>
__device__ __forceinline__ void join_parts(int x0, int x1, int h, int lane, F part_of, float& M,
                                           float& L, float4& num) {
  constexpr int kFew = 4;
  if (x1 - x0 < kFew) {  // few parts (short rows): one trip to memory for everything
    float m = -INFINITY, l = 0.f;
    if (lane <= x1 - x0) {
      m = __ldcg(part_of(x0 + lane) + HR * D + h);
      l = __ldcg(part_of(x0 + lane) + HR * D + HR + h);
    }
    float4 y[kFew];
#pragma unroll
    for (int x = 0; x < kFew; ++x)
      if (x <= x1 - x0 && 4 * lane < D)
        y[x] = __ldcg(reinterpret_cast<const float4*>(part_of(x0 + x) + h * D + 4 * lane));
    M = m;
#pragma unroll
    for (int o = kFew / 2; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    M = __shfl_sync(0xffffffffu, M, 0);
    const float f = ex2_approx(m - (M == -INFINITY ? 0.f : M));
    L = 0.f;
    num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int x = 0; x < kFew; ++x) {
      const float fx = __shfl_sync(0xffffffffu, f, x), lx = __shfl_sync(0xffffffffu, l, x);
      if (x <= x1 - x0) {
        L = fmaf(fx, lx, L);
        if (4 * lane < D) axpy(num, fx, y[x]);
      }
    }
    return;
  }
  M = -INFINITY;
  for (int x = x0 + lane; x <= x1; x += 32) M = fmaxf(M, __ldcg(part_of(x) + HR * D + h));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float base = M == -INFINITY ? 0.f : M;
  L = 0.f;
  num = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = x0; p0 <= x1; p0 += 32) {
    const int parts = min(32, x1 - p0 + 1);
    float f = 0.f, fl = 0.f;
    if (lane < parts) {
      const float* p = part_of(p0 + lane) + HR * D + h;
      f = ex2_approx(__ldcg(p) - base);
      fl = f * __ldcg(p + HR);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) fl += __shfl_xor_sync(0xffffffffu, fl, o);
    L += fl;
#pragma unroll 8
    for (int x = 0; x < parts; ++x) {
      const float fx = __shfl_sync(0xffffffffu, f, x);
      if (4 * lane < D)
        axpy(num, fx, __ldcg(reinterpret_cast<const float4*>(part_of(p0 + x) + h * D + 4 * lane)));
    }
  }
}

// A row's query heads are the 8 NT columns of the MMAs.  PACK (up to four
// heads): columns 0..3 and 4..7 are the same heads over two tiles of slots, as
// two softmax states that are joined at the row's end, so that one set of
// scores, weights and pairs covers 32 slots.  Per 16 slots that saves some 20%
// of the instructions, which is what bounds the loop.
template <int GR, int NT, bool PACK>
__global__ void __launch_bounds__(DecodeShape<NT>::kThreads, 1)
    kv4_decode_kernel(const DecodeParams P) {
  static_assert(!PACK || NT == 1, "packing is for few heads");
  constexpr int D = 64 * GR, HT = 8 * NT;
  constexpr int HR = PACK ? 4 : HT;  // query heads a row
  constexpr int kSub = HT / HR;      // softmax states of a head in a warp
  constexpr int kWarps = DecodeShape<NT>::kWarps, kThreads = DecodeShape<NT>::kThreads;
  constexpr int kPart = HR * (D + 2);  // floats of a part: O [HR][D], m and l [HR]
  constexpr int kChunk = GR * kKv4GroupBytes;
  // tiles of 16 slots a step (their chains of dependent instructions overlap),
  // and sets of scores
  constexpr int TT = PACK ? 4 : 2, U = TT / kSub;
  extern __shared__ __align__(128) uint8_t smem[];  // [warp][2][kChunk]
  __shared__ __align__(8) uint64_t bars[2 * kWarps];
  __shared__ PageNote s_note[2 * kWarps];
  __shared__ int s_abort, s_last[2];
  __shared__ int s_sum[kWarps], s_long[kWarps];
  __shared__ int s_start[2];
  __shared__ SharedRow s_row[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const Kv4Cache& c = P.c;
  const int RPS = c.Hkv * P.HC;  // rows per sequence

  launch_dependents();
  if (tid == 0) {
    s_abort = 0;
    s_row[0].parts = s_row[1].parts = 0;
    for (int i = 0; i < 2 * kWarps; ++i) mbar_init(smem_u32(&bars[i]), 1);
    fence_mbar_init();
  }
  // the list's length, and where this CTA's range starts: thread i sums a
  // contiguous piece of the sequences
  const int per = (c.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, c.B), b1 = min(b0 + per, c.B);
  int mine = 0, longest = 0;
  for (int b = b0; b < b1; ++b) {
    int n;
    const bool ok = kv4_len(c, b, n);
    if (blockIdx.x == 0 && !ok) atomicOr(P.status, VS_DEVFLAG_BOUNDS);
    const int pages = visible_pages(n, P.window, P.sinks).pages;
    mine += pages * RPS;
    longest = max(longest, pages);
  }
  int incl = mine;  // over the lanes, then over the warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 31) {
    s_sum[warp] = incl;
    s_long[warp] = longest;
  }
  __syncthreads();
  int total = 0, before = incl - mine;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
    longest = max(longest, s_long[w]);
  }
  // Rows of no more pages than there are warps, and no more rows than CTAs: a
  // row each, so that no CTAs share one.  Else equal ranges of the list.
  const bool by_row = longest <= kWarps && c.B * RPS <= (int)gridDim.x;
  const int share = max(kDecMinPages, (total + (int)gridDim.x - 1) / (int)gridDim.x);
  int f0 = min((int64_t)blockIdx.x * share, (int64_t)total);
  int f1 = min((int64_t)f0 + share, (int64_t)total);
  if (by_row) {
    const int b = blockIdx.x / RPS;
    f0 = f1 = 0;
    if (b < c.B) {
      int n;
      kv4_len(c, b, n);
      f1 = visible_pages(n, P.window, P.sinks).pages;
      if (tid == 0) {
        s_start[0] = b;
        s_start[1] = (blockIdx.x - b * RPS) * f1;
      }
    }
  } else {
    int at = before;
    if (f0 < f1 && at <= f0 && f0 < at + mine) {
      int b = b0;
      for (;; ++b) {
        int n;
        kv4_len(c, b, n);
        const int p = visible_pages(n, P.window, P.sinks).pages * RPS;
        if (f0 < at + p) break;
        at += p;
      }
      s_start[0] = b;
      s_start[1] = f0 - at;
    }
  }
  // rows without a visible slot: nobody's range covers them
  for (int b = blockIdx.x; b < c.B; b += gridDim.x) {
    int n;
    kv4_len(c, b, n);
    if (n > 0) continue;
    for (int e = tid; e < P.Hq * D; e += kThreads)
      P.O[(int64_t)b * P.q_stride + e] = __float2bfloat16_rn(0.f);
    if (P.lse)
      for (int h = tid; h < P.Hq; h += kThreads) P.lse[(int64_t)h * c.B + b] = -INFINITY;
  }
  __syncthreads();
  if (f0 >= f1) return;

  Cursor seg;  // where the CTA's range starts
  seg.b = s_start[0];
  cursor_load(P, seg);
  seg.k = s_start[1] % seg.v.pages;
  seg.head = s_start[1] / seg.v.pages / P.HC;
  seg.hc = s_start[1] / seg.v.pages % P.HC;
  const int count = f1 - f0;
  const int wper = (count + kWarps - 1) / kWarps;  // pages a warp
  const WaitCtx wc{P.wait_limit_ns, P.status, &s_abort};

  // ------------------------------------------------- this warp's own pages
  {
    const int w0 = min(warp * wper, count), pages = min(wper, count - w0);
    Cursor next = seg;  // of the next page to fetch
    int issued = 0;
    int id = 0;  // of the next page, looked up one page ahead of its use
    auto next_page = [&]() { return next.k < next.v.first ? next.k : next.k + next.v.gap; };
    auto look_up = [&]() { id = __ldg(c.table + (int64_t)next.b * c.table_ld + next_page()); };
    if (pages > 0) {
      cursor_add(P, next, w0);
      look_up();
    }
    auto bar = [&](int s) { return smem_u32(&bars[2 * warp + s]); };
    auto issue = [&]() {  // page `issued` into slot issued mod 2
      if (issued >= pages) return;
      const int s = issued & 1;
      if (lane == 0) {
        PageNote& pn = s_note[2 * warp + s];
        pn.b = next.b;
        pn.head = next.head;
        pn.hc = next.hc;
        pn.k = next.k;
        pn.pages = next.v.pages;
        const bool valid = id >= 0 && id < c.n_pages;
        pn.page = valid ? next_page() : -1;
        if (valid) {
          mbar_arrive_expect_tx(bar(s), kChunk);
          bulk_load(smem_u32(smem + (2 * warp + s) * kChunk),
                    c.pool + ((int64_t)id * c.Hkv + next.head) * kChunk, kChunk, bar(s));
        } else {
          atomicOr(P.status, VS_DEVFLAG_BOUNDS);
          mbar_arrive(bar(s));
        }
      }
      if (++issued < pages) {
        cursor_add(P, next, 1);
        look_up();
      }
    };
    issue();
    issue();

    int row_b = -1, row_head = 0, row_hc = 0, row_k0 = 0, row_k1 = 0, row_pages = 0;
    bool first_row = true;
    int n = 0, lo_slot = 0, heads = 0, h0 = 0;
    uint32_t qf[NT][GR][2][4];
    float qs[NT][GR][2], sl[NT][2];
    float o[NT][GR][4][4];  // O^T tiles, centred on code 8, in units of 2^-133
    float m[NT][2], nb[NT][2], l[NT][2], r[NT][GR][2];  // p = 2^(score sl + nb)
    bool ok = true;
    int i = 0;
    for (;; ++i) {
      const int st = i & 1;
      PageNote pn{};
      if (i < pages) {
        if (ok) ok = mbar_wait(bar(st), (uint32_t)(i >> 1) & 1u, wc);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        pn = s_note[2 * warp + st];
      }
      if (i >= pages || pn.b != row_b || pn.head != row_head || pn.hc != row_hc) {
        if (row_b >= 0) {
          // ------------------------------------------- the row is done here
          const bool whole_row = row_k0 == 0 && row_k1 == row_pages;
          float* part = P.warp_parts +
                        (size_t)(2 * (blockIdx.x * kWarps + warp) + (first_row ? 0 : 1)) * kPart;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float M = m[nt][y], L = l[nt][y], f = 1.f;
#pragma unroll
              for (int s = 4; s < 32; s <<= 1) L += __shfl_xor_sync(0xffffffffu, L, s);
              if (PACK) {  // the two halves' states
                const float M2 = __shfl_xor_sync(0xffffffffu, M, 2);
                const float top = fmaxf(M, M2);
                f = ex2_approx(M - (top == -INFINITY ? 0.f : top));
                M = top;
                L *= f;
                L += __shfl_xor_sync(0xffffffffu, L, 2);
              }
              const int h = (PACK ? 2 * (tig & 1) : 8 * nt + 2 * tig) + y;
              const bool mine = h < heads && (!PACK || tig < 2);
              const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);  // NaN stays
              if (mine && gid == 0) {
                if (whole_row) {
                  write_lse(P, row_b, h0 + h, M, L);
                } else {
                  part[HR * D + h] = M;
                  part[HR * D + HR + h] = L;
                }
              }
              __nv_bfloat16* orow =
                  P.O + (int64_t)row_b * P.q_stride + (int64_t)(h0 + h) * D + 2 * gid;
#pragma unroll
              for (int g = 0; g < GR; ++g) {
                float rs = r[nt][g][y];
#pragma unroll
                for (int s = 4; s < 32; s <<= 1) rs += __shfl_xor_sync(0xffffffffu, rs, s);
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // odd codes count 16 n
                  float lo = fmaf(o[nt][g][j][y] * 0x1p100f, 0x1p33f, rs);
                  float hi = fmaf(o[nt][g][j][y + 2] * 0x1p100f, 0x1p29f, rs);
                  if (PACK) {
                    lo *= f;
                    hi *= f;
                    lo += __shfl_xor_sync(0xffffffffu, lo, 2);
                    hi += __shfl_xor_sync(0xffffffffu, hi, 2);
                  }
                  if (mine) {
                    if (whole_row)
                      *reinterpret_cast<uint32_t*>(orow + 64 * g + 16 * j) =
                          pack_bf16x2(lo * inv, hi * inv);
                    else
                      *reinterpret_cast<float2*>(part + h * D + 64 * g + 16 * j + 2 * gid) =
                          make_float2(lo, hi);
                  }
                }
              }
            }
          first_row = false;
        }
        if (i >= pages) break;
        row_b = pn.b;
        row_head = pn.head;
        row_hc = pn.hc;
        row_k0 = pn.k;
        row_pages = pn.pages;
        kv4_len(c, row_b, n);
        lo_slot = P.window > 0 && n > P.window ? n - P.window : 0;
        heads = min(HR, P.G - row_hc * HR);
        h0 = row_head * P.G + row_hc * HR;  // first query head of the row
        // Q as the B operand of S^T = K Q^T: head gid (mod HR), channels in the
        // order the words' codes give, scaled by f = 2^(field - 127), odd codes' by f / 16.
        // For this lane's heads: the groups' sums of q, in the units f 2^-133 of
        // the scores, and what takes scores from these units to base 2.
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t big = 0;
#pragma unroll
          for (int g = 0; g < GR; ++g)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              uint4 u = make_uint4(0, 0, 0, 0);
              const int h = PACK ? gid & 3 : 8 * nt + gid;
              if (h < heads)
                u = __ldg(reinterpret_cast<const uint4*>(P.Q + (int64_t)row_b * P.q_stride +
                                                         (int64_t)(h0 + h) * D + 64 * g +
                                                         8 * (2 * tig + w)));
              qf[nt][g][w][0] = __byte_perm(u.x, u.z, 0x5410);  // channels 0, 4
              qf[nt][g][w][1] = __byte_perm(u.x, u.z, 0x7632);  // 1, 5
              qf[nt][g][w][2] = __byte_perm(u.y, u.w, 0x5410);
              qf[nt][g][w][3] = __byte_perm(u.y, u.w, 0x7632);
              // largest exponent, as the bits of |q|
              const uint32_t x = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                                          __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
              big = max(big, max(x & 0xffffu, x >> 16));
            }
          big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
          // max |q| f in [2^118, 2^119); f at most 2^127, and at least 2^6 (for |q|
          // from 2^113 on), where the scale of the scores ends
          const int field = min(254, max(133, 372 - (int)(big >> 7)));
          const float f = pow2_field(field);
#pragma unroll
          for (int g = 0; g < GR; ++g) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float a = __uint_as_float(qf[nt][g][w][i] << 16) * f;
                const float b = __uint_as_float(qf[nt][g][w][i] & 0xffff0000u) * f;
                sum += a + b;
                qf[nt][g][w][i] =
                    i & 1 ? pack_bf16x2(a * 0.0625f, b * 0.0625f) : pack_bf16x2(a, b);
              }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            sum *= 0x1p-100f;
            qs[nt][g][0] = __shfl_sync(0xffffffffu, sum, 8 * tig) * 0x1p-33f;
            qs[nt][g][1] = __shfl_sync(0xffffffffu, sum, 8 * tig + 4) * 0x1p-33f;
          }
          const float back = P.scale * pow2_field(387 - field);  // scale 2^133 / f
          sl[nt][0] = __shfl_sync(0xffffffffu, back, 8 * tig);
          sl[nt][1] = __shfl_sync(0xffffffffu, back, 8 * tig + 4);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int g = 0; g < GR; ++g) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
              for (int j = 0; j < 4; ++j) o[nt][g][j][x] = 0.f;
            r[nt][g][0] = r[nt][g][1] = 0.f;
          }
          m[nt][0] = m[nt][1] = -INFINITY;
          l[nt][0] = l[nt][1] = nb[nt][0] = nb[nt][1] = 0.f;
        }
      }
      row_k1 = pn.k + 1;
      if (pn.page >= 0) {
        const uint8_t* pg = smem + (2 * warp + st) * kChunk;
        const int t0 = pn.page * kKv4Page;
        // every slot of the page visible?
        const bool whole = t0 + kKv4Page <= n && (t0 >= lo_slot || t0 + kKv4Page <= P.sinks);
        auto hidden = [&](int t) { return t >= n || (t < lo_slot && t >= P.sinks); };
        // TT tiles of 16 slots a step, looped where a page has more: a short row
        // runs the code from a cold instruction cache.
        const int mine = PACK ? 16 * (tig >> 1) + gid : gid;  // slot of this lane's row gid
        const int vrow = 2 * ((lane >> 2) & 3) + ((lane >> 1) & 1) + 8 * (lane & 1);
        const int tiles = min(4, (n - t0 + 15) / 16);
#pragma unroll 1
        for (int tl = 0; tl < tiles; tl += TT) {
          const uint8_t* kc = pg + kv4_code_off(GR, 0, 0, 16 * tl + gid) + 8 * tig;
          const uint8_t* pr = pg + kv4_pair_off(GR, 0, 0, 16 * tl + mine);
          // rows of the byte matrices: slots in the order that makes bytes 0 and
          // 2 of a register slots 2 tig, 2 tig + 1, and bytes 1 and 3 those + 8
          const uint32_t vc =
              smem_u32(pg + kv4_code_off(GR, 1, 0, 16 * tl + vrow)) + 16 * (lane >> 4);
          float sc[U][NT][4];
#pragma unroll
          for (int g = 0; g < GR; ++g)
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const uint32_t pa =
                  *reinterpret_cast<const uint32_t*>(pr + g * kKv4Pairs + 64 * kSub * u);
              const uint32_t pb =
                  *reinterpret_cast<const uint32_t*>(pr + g * kKv4Pairs + 64 * kSub * u + 32);
              const float sa = kv4_step(pa), sb = kv4_step(pb);
              const float ma = kv4_min(pa), mb = kv4_min(pb);
              float cacc[kSub][NT][4];
#pragma unroll
              for (int v = 0; v < kSub; ++v) {
                const uint8_t* kt = kc + g * kKv4Codes + 512 * (kSub * u + v);
                const uint2 wa = *reinterpret_cast<const uint2*>(kt);
                const uint2 wb = *reinterpret_cast<const uint2*>(kt + 256);
                const uint32_t xa = wa.x >> 8, xb = wb.x >> 8, ya = wa.y >> 8, yb = wb.y >> 8;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  mma_bf16_first(cacc[v][nt], codes_lo(wa.x), codes_lo(wb.x), codes_hi(wa.x),
                                 codes_hi(wb.x), qf[nt][g][0][0], qf[nt][g][0][1]);
                  mma_bf16(cacc[v][nt], codes_lo(xa), codes_lo(xb), codes_hi(xa), codes_hi(xb),
                           qf[nt][g][0][2], qf[nt][g][0][3]);
                  mma_bf16(cacc[v][nt], codes_lo(wa.y), codes_lo(wb.y), codes_hi(wa.y),
                           codes_hi(wb.y), qf[nt][g][1][0], qf[nt][g][1][1]);
                  mma_bf16(cacc[v][nt], codes_lo(ya), codes_lo(yb), codes_hi(ya), codes_hi(yb),
                           qf[nt][g][1][2], qf[nt][g][1][3]);
                }
              }
              // q.k = sum_g s (q.n) + m (q.1)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  const float mm = x < 2 ? ma : mb, ss = x < 2 ? sa : sb, qq = qs[nt][g][x & 1];
                  const float qn = kSub == 2 && tig >= 2 ? cacc[kSub - 1][nt][x] : cacc[0][nt][x];
                  sc[u][nt][x] = fmaf(ss, qn, g == 0 ? mm * qq : fmaf(mm, qq, sc[u][nt][x]));
                }
            }
          const int ta = t0 + 16 * tl + mine;  // slot of this lane's row gid in set 0
          if (!whole) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if (hidden(ta + 16 * kSub * u)) sc[u][nt][0] = sc[u][nt][1] = -INFINITY;
                if (hidden(ta + 16 * kSub * u + 8)) sc[u][nt][2] = sc[u][nt][3] = -INFINITY;
              }
          }
          if (P.score) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const int hh = row_hc * HR + (PACK ? 2 * (tig & 1) : 8 * nt + 2 * tig);
              if (hh < P.Gp) {
                float* dst = P.score + (((int64_t)row_b * c.Hkv + row_head) * P.slots + ta) * P.Gp + hh;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                  for (int y = 0; y < 2; ++y)
                    *reinterpret_cast<float2*>(dst + (16 * kSub * u + 8 * y) * P.Gp) = make_float2(
                        sc[u][nt][2 * y] * sl[nt][0], sc[u][nt][2 * y + 1] * sl[nt][1]);
              }
            }
          }
          // Online softmax.  The running maximum follows only when a score
          // passes it by 2^8: the weights have room, and the lanes' maxima need
          // not be joined for every tile.
          bool need = false;
          float mx[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float x = -INFINITY;
#pragma unroll
              for (int u = 0; u < U; ++u) x = fmax3(x, sc[u][nt][y], sc[u][nt][y + 2]);
              mx[nt][y] = x * sl[nt][y];
              need |= mx[nt][y] > m[nt][y] + 8.f;
            }
          if (__any_sync(0xffffffffu, need)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                float x = mx[nt][y];
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                if (x > m[nt][y]) {
                  const float f = ex2_approx(m[nt][y] - x);  // 0 at first
                  m[nt][y] = x;
                  nb[nt][y] = kShift - x;
                  l[nt][y] *= f;
#pragma unroll
                  for (int g = 0; g < GR; ++g) {
                    r[nt][g][y] *= f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                      o[nt][g][j][y] *= f;
                      o[nt][g][j][y + 2] *= f;
                    }
                  }
                }
              }
          }
          float p[U][NT][4];
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                p[u][nt][x] = ex2_approx(fmaf(sc[u][nt][x], sl[nt][x & 1], nb[nt][x & 1]));
                l[nt][x & 1] += p[u][nt][x];
              }
          const uint32_t first_half = gid < 4 ? ~0u : 0u;  // columns of a pack's first tile
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int g = 0; g < GR; ++g) {
              uint32_t pa =
                  *reinterpret_cast<const uint32_t*>(pr + (GR + g) * kKv4Pairs + 64 * kSub * u);
              uint32_t pb =
                  *reinterpret_cast<const uint32_t*>(pr + (GR + g) * kKv4Pairs + 64 * kSub * u + 32);
              if (!whole) {  // 0 * NaN of a slot never written
                if (hidden(ta + 16 * kSub * u)) pa = 0;
                if (hidden(ta + 16 * kSub * u + 8)) pb = 0;
              }
              const float sa = kv4_step(pa), sb = kv4_step(pb);
              const float ca = fmaf(8.f, sa, kv4_min(pa)), cb = fmaf(8.f, sb, kv4_min(pb));
              uint32_t bf[NT][2];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                bf[nt][0] = transpose8(pack_bf16x2(p[u][nt][0] * sa, p[u][nt][1] * sa));
                bf[nt][1] = transpose8(pack_bf16x2(p[u][nt][2] * sb, p[u][nt][3] * sb));
#pragma unroll
                for (int y = 0; y < 2; ++y)
                  r[nt][g][y] = fmaf(p[u][nt][y], ca, fmaf(p[u][nt][y + 2], cb, r[nt][g][y]));
              }
              // V^T as the A operand: a register is one tile of 16 channels, the
              // low codes of its bytes in rows 0..7, the high ones in rows 8..15
#pragma unroll
              for (int v = 0; v < kSub; ++v) {
                const uint32_t keep = v == 0 ? first_half : ~first_half;
                uint32_t x[4];
                load_bytes_t(x, vc + g * kKv4Codes + 512 * (kSub * u + v));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  const uint32_t b0 = PACK ? bf[nt][0] & keep : bf[nt][0];
                  const uint32_t b1 = PACK ? bf[nt][1] & keep : bf[nt][1];
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    mma_bf16(o[nt][g][j], codes_lo(x[j]), codes_hi(x[j]), codes_lo(x[j] >> 8),
                             codes_hi(x[j] >> 8), b0, b1);
                }
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  mma_bf16(o[nt][g][j], kMinus8, kMinus128, kMinus8, kMinus128, bf[nt][0], bf[nt][1]);
            }
        }
      }
      __syncwarp();
      issue();
    }
    // copies not awaited (only after a wait gave up) land before shared memory is released
    if (lane == 0 && !ok)
      for (; i < issued; ++i)
        mbar_wait_drain(bar(i & 1), (uint32_t)(i >> 1) & 1u, P.wait_limit_ns);
  }

  // ------------------------------------- the parts of the CTA's warps, by row
  // One (row, head) a warp and turn: a lane per part, then D / 4 lanes with
  // four channels each.
  __syncthreads();
  const int w_lane = 4 * lane;  // first channel of this lane
  auto finish = [&](int b, int h, float M, float L, const float4& num) {
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);  // NaN stays
    if (w_lane < D)
      *reinterpret_cast<uint2*>(P.O + (int64_t)b * P.q_stride + (int64_t)h * D + w_lane) =
          make_uint2(pack_bf16x2(num.x * inv, num.y * inv), pack_bf16x2(num.z * inv, num.w * inv));
    if (lane == 0) write_lse(P, b, h, M, L);
  };
  int turn = 0, wa = 0, wb = 0;
  for (int at = 0; at < count;) {
    const int k0 = seg.k, k1 = min(seg.v.pages, k0 + (count - at));
    // the warps with pages of it
    while ((wa + 1) * wper <= at) ++wa;
    while ((wb + 1) * wper < at + (k1 - k0)) ++wb;
    const bool shared = k0 > 0 || k1 < seg.v.pages;
    const int heads = min(HR, P.G - seg.hc * HR), h0 = seg.head * P.G + seg.hc * HR;
    if (shared || wa != wb) {
      // the CTA's part: its first row's or its last row's
      float* out = P.parts + (size_t)(2 * blockIdx.x + (at > 0 ? 1 : 0)) * kPart;
      // the heads go round the warps: this warp's first is the one at its turn
      int h = warp - turn;
      if (h < 0) h += kWarps;
      turn = (turn + heads) % kWarps;
      for (; h < heads; h += kWarps) {
        // a warp's part of the row is its first unless its range starts before the row
        auto part_of = [&](int w) {
          return P.warp_parts +
                 (size_t)(2 * (blockIdx.x * kWarps + w) + (w * wper < at ? 1 : 0)) * kPart;
        };
        float M, L;
        float4 num;
        join_parts<D, HR>(wa, wb, h, lane, part_of, M, L, num);
        if (!shared) {
          finish(seg.b, h0 + h, M, L, num);
        } else {
          if (w_lane < D) *reinterpret_cast<float4*>(out + h * D + w_lane) = num;
          if (lane == 0) {
            out[HR * D + h] = M;
            out[HR * D + HR + h] = L;
          }
        }
      }
      if (shared && tid == 0) {
        // list positions of the row give the CTAs that share it
        SharedRow& sr = s_row[at > 0 ? 1 : 0];
        sr.start = f0 + at - k0;
        sr.c0 = sr.start / share;
        sr.parts = (sr.start + seg.v.pages - 1) / share - sr.c0 + 1;
        sr.b = seg.b;
        sr.h0 = h0;
        sr.heads = heads;
        sr.ticket = (seg.b * c.Hkv + seg.head) * P.HC + seg.hc;
      }
    }
    at += k1 - k0;
    if (at < count) cursor_add(P, seg, k1 - k0);
  }
  // ---------------------------------------------------- rows of several CTAs
  __threadfence();
  __syncthreads();
  if (tid < 2) {
    const SharedRow& sr = s_row[tid];
    s_last[tid] = sr.parts > 0 && atomicAdd(P.ticket + sr.ticket, 1) == sr.parts - 1;
  }
  __syncthreads();
  if (!s_last[0] && !s_last[1]) return;
  __threadfence();
  turn = 0;
  for (int x = 0; x < 2; ++x) {
    if (!s_last[x]) continue;
    const SharedRow sr = s_row[x];
    int h = warp - turn;
    if (h < 0) h += kWarps;
    turn = (turn + sr.heads) % kWarps;
    for (; h < sr.heads; h += kWarps) {
      // CTA x's part is its first unless its range starts before the row
      auto part_of = [&](int cta) {
        return P.parts + (size_t)(2 * cta + ((int64_t)cta * share < sr.start ? 1 : 0)) * kPart;
      };
      float M, L;
      float4 num;
      join_parts<D, HR>(sr.c0, sr.c0 + sr.parts - 1, h, lane, part_of, M, L, num);
      finish(sr.b, sr.h0 + h, M, L, num);
    }
  }
}

// acc_out = acc_in + sum over the KV head's query heads of the softmax weight,
// per slot; invisible slots keep their sum.  Bound by memory: a float per query
// head and two for acc per slot; 236,000 slots of 8 heads (4 query heads each):
// 14 us, 3.2 TB/s.  Two slots a thread, so that their loads overlap: one or four
// take 2 us longer.  W: floats of a score load (Gp is a multiple).
constexpr int kWeightsTurn = 512;  // slots of a block and turn
template <int W>
__global__ void __launch_bounds__(256) kv4_weights_kernel(DecodeParams P, const float* acc_in,
                                                          float* acc_out, int64_t ld) {
  constexpr int kSlots = kWeightsTurn / 256;
  constexpr int kHeads = 128;  // log-sum-exps kept; a load per slot for further heads
  __shared__ float s_lse2[kHeads];
  const Kv4Cache& c = P.c;
  const int b = blockIdx.y / c.Hkv, head = blockIdx.y % c.Hkv;
  int n;
  kv4_len(c, b, n);
  const int lo_slot = P.window > 0 && n > P.window ? n - P.window : 0;
  const float* lse2 = P.lse2 + (int64_t)b * P.Hq + (int64_t)head * P.G;
  const int64_t row = (int64_t)b * c.Hkv + head;
  wait_for_previous_kernel();
  if (threadIdx.x < P.G && threadIdx.x < kHeads) s_lse2[threadIdx.x] = __ldcg(lse2 + threadIdx.x);
  __syncthreads();
  for (int t0 = blockIdx.x * kWeightsTurn + threadIdx.x; t0 < n; t0 += gridDim.x * kWeightsTurn) {
    float sum[kSlots], w[kSlots] = {};
    bool seen[kSlots];
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
      const int t = t0 + 256 * u;
      sum[u] = acc_in && t < n ? acc_in[row * ld + t] : 0.f;
      seen[u] = t < n && (t >= lo_slot || t < P.sinks) && kv4_page(c, b, t >> 6, head);
    }
    for (int h = 0; h < P.G; h += W) {
      float x[kSlots][W] = {};
#pragma unroll
      for (int u = 0; u < kSlots; ++u) {
        const int t = t0 + 256 * u;
        if (t >= n) continue;
        const float* s = P.score + (row * P.slots + t) * P.Gp + h;
        if constexpr (W == 4)
          *reinterpret_cast<float4*>(x[u]) = __ldcs(reinterpret_cast<const float4*>(s));
        else
          *reinterpret_cast<float2*>(x[u]) = __ldcs(reinterpret_cast<const float2*>(s));
      }
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if (h + i >= P.G) continue;
        const float l = h + i < kHeads ? s_lse2[h + i] : __ldcg(lse2 + h + i);
#pragma unroll
        for (int u = 0; u < kSlots; ++u) w[u] += ex2_approx(x[u][i] - l);
      }
    }
#pragma unroll
    for (int u = 0; u < kSlots; ++u)
      if (t0 + 256 * u < n) acc_out[row * ld + t0 + 256 * u] = seen[u] ? sum[u] + w[u] : sum[u];
  }
}

size_t kv4_decode_ws_bytes(int B, int Hq, int Hkv, int d, int max_len, bool weights) {
  return DecodeLayout::make(B, Hq, Hkv, d, max_len, weights, device_sm_count()).total;
}

template <int GR, int NT, bool PACK>
static cudaError_t launch_decode_impl(const DecodeParams& P, int grid, cudaStream_t stream) {
  auto kern = kv4_decode_kernel<GR, NT, PACK>;
  constexpr int smem = DecodeShape<NT>::kWarps * 2 * GR * kKv4GroupBytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<grid, DecodeShape<NT>::kThreads, smem, stream>>>(P);
  return cudaGetLastError();
}

cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a) {
  const int sms = device_sm_count(), d = a.c.GR * 64;
  const DecodeLayout L =
      DecodeLayout::make(a.c.B, a.Hq, a.c.Hkv, d, a.c.max_len, a.acc_out != nullptr, sms);
  char* ws = static_cast<char*>(a.ws);
  // status word and tickets
  cudaError_t e = cudaMemsetAsync(ws, 0, L.off_part, a.stream);
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)a.c.B * a.c.Hkv * L.HC;
  // no more CTAs than the longest possible list fills
  const int64_t most = rows * (L.slots / kKv4Page);
  const int64_t by_pages = (most + kDecMinPages - 1) / kDecMinPages;
  const int64_t want = by_pages > rows ? by_pages : rows;
  const int grid = (int)(want < 1 ? 1 : (want < sms ? want : sms));
  DecodeParams P;
  P.c = a.c;
  P.Q = static_cast<const __nv_bfloat16*>(a.Q);
  P.q_stride = a.q_stride;
  P.Hq = a.Hq;
  P.G = a.G;
  P.HC = L.HC;
  P.Gp = L.Gp;
  P.scale = a.scale * 1.4426950408889634f;
  P.window = a.window;
  P.sinks = a.sinks;
  P.O = static_cast<__nv_bfloat16*>(a.O);
  P.lse = a.lse;
  P.status = reinterpret_cast<int*>(ws);
  P.ticket = reinterpret_cast<int*>(ws + L.off_tick);
  P.parts = reinterpret_cast<float*>(ws + L.off_part);
  P.warp_parts = P.parts + 2 * (size_t)grid * L.part_floats;
  P.lse2 = a.acc_out ? reinterpret_cast<float*>(ws + L.off_lse) : nullptr;
  P.score = a.acc_out ? reinterpret_cast<float*>(ws + L.off_score) : nullptr;
  P.slots = L.slots;
  P.wait_limit_ns = kDefaultWaitLimitNs;
  if (L.HT == 4)
    e = a.c.GR == 1 ? launch_decode_impl<1, 1, true>(P, grid, a.stream)
                    : launch_decode_impl<2, 1, true>(P, grid, a.stream);
  else if (L.HT == 8)
    e = a.c.GR == 1 ? launch_decode_impl<1, 1, false>(P, grid, a.stream)
                    : launch_decode_impl<2, 1, false>(P, grid, a.stream);
  else
    e = a.c.GR == 1 ? launch_decode_impl<1, 2, false>(P, grid, a.stream)
                    : launch_decode_impl<2, 2, false>(P, grid, a.stream);
  if (e != cudaSuccess || !a.acc_out) return e;
  const int64_t per_row = (L.slots + kWeightsTurn - 1) / kWeightsTurn;
  const int64_t cap = ceil_div(32LL * sms, a.c.B * a.c.Hkv);
  const dim3 wgrid((unsigned)(per_row < cap ? per_row : cap), a.c.B * a.c.Hkv);
  return launch_after(L.Gp % 4 == 0 ? kv4_weights_kernel<4> : kv4_weights_kernel<2>, wgrid, 256,
                      a.stream, P, a.acc_in, a.acc_out, a.ld);
}

}  // namespace vs
