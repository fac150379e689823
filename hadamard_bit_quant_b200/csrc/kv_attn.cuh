// Attention over the paged 8-bit key/value cache: few query rows per key/value head (single tokens, drafts).
//
//   O_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = exp(scale * q_r . k_j - m_r)  over the keys j that row r sees,
// with k_j = (u_j - 128) * s of the key's block. Rows of one request that share a key/value head (its query
// heads times its new tokens) are taken 16 at a time, so the cache is read once for all of them.
//
// The bound is the cache read: D bytes of keys and D of values for each token and head. The kernel is a stream over
// tiles of 32 tokens:
//   * two or three CTAs per SM, each with an equal share of all tiles of all requests and heads (the long axis is
//     split wherever the share ends), tiles dealt to its 6 or 4 warps in turn;
//   * each warp has a ring of its own in shared memory, filled with 16-byte cp.async, and its own reference
//     maximum, sum and output in registers: no barrier while it streams. The next run's first tiles are fetched before
//     the warps' results of this one are added up;
//   * codes become fp16 exactly (0x6400 | u is 1024 + u; minus 1152), the query rows are scaled by a power of
//     two into fp16's range (exact but for what lies 2^-25 below the row's largest value), and both products
//     run on mma.m16n8k16 with fp32 sums, the tokens (then the channels) as the 16 rows and the query rows as the 8
//     columns: with 8 query rows nothing is padded, where a 128-row tcgen05 tile would be 15/16 padding;
//   * a block's key scale multiplies the scores; its value scale s enters as an addend log2(s) of the exponent. So
//     the second product takes weights p s, relative to a reference of their own row: nothing that a row does not see
//     has a part in how they are rounded. The sum of the p, relative to a reference of the scores alone, is that of the
//     weights times 1 / s. Both references are raised only when a tile outgrows the weights' by 2^8: then no lane has to ask
//     the others for the tile's maxima. Weights stay below 2^15 and are rounded to fp16 (11 bits), finer than the bf16 output.
// At the end of a run the warps' results are joined through shared memory: weighted values relative to the largest weights'
// reference, and the log2 of the sums. A run that is only a part of its row's keys goes to the workspace in the same form,
// and kv_combine_kernel joins the parts.
// Measured, of HBM's copy rate on the codes, queries and outputs: 128 requests of up to 4096 tokens, 32 query heads on 8 of
// 128: 143 us, 5.6 TB/s (86 %); one of 131072: 57 us, 4.7 TB/s (72 %); 16 of up to 2048, 32 heads each their own: 44.5 us,
// 4.35 TB/s (66 %). What is left there is the start (lengths, table, first tiles: 4 us one after the other), the
// SMs' unequal share of the bandwidth (42 to 64 us for equal work) and the joining (3 us). Many short requests are
// bound by the instructions at the beginnings and ends of runs: 2048 of 100 tokens 195 us where the bytes take 64.
#pragma once
#include "hbl_common.cuh"
#include <cuda_fp16.h>

namespace hbl {
namespace kv {

constexpr int kAttnTile = 32;         // tokens of a warp's tile
constexpr int kAttnRows = 16;         // most query rows of a tile
// log2 of how far the weights' reference is set below the largest weight, and of how far that may then grow: together fp16's
// range, so that small weights, of which there may be many, are rounded as late as its least value allows.
constexpr float kHead = 7.f, kLag = 8.f;
// log2 of how far a block's value scale may lie below that of the row's largest weight before the scores' reference is brought
// up to date (the sum, relative to it, stays below 2^103 for each key). With one that lies further below the block then counts
// as that far: its weights are zero in fp16 either way, and the p that the sum gets back from them neither vanish nor
// overflow. kLeastScale: log2 of the least value scale that is told apart (appending makes none below 2^-100); kZeroScale
// stands for that of 0, which leaves the weights' reference as it is.
constexpr float kSpread = 88.f, kLeastScale = -110.f, kZeroScale = -2e30f;
constexpr float kNothing = -1e30f;    // references of a row that has seen no key
constexpr int kMaxAttnCtas = 480;     // workspace is laid out for this many
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnArgs {
  const uint16_t* Q;                  // T x Hq x D, q_stride elements from token to token
  long long q_stride;
  const int32_t* cu_q;                // B + 1
  const int32_t* kv_lens;             // B
  const int32_t* table;               // B x max_pages
  const uint8_t* kcodes;
  const uint8_t* vcodes;
  const float* kscale;
  const float* vscale;
  uint16_t* O;                        // T x Hq x D
  float* lse;                         // T x Hq or null
  long long* prefix;                  // workspace: tiles before each request, B + 1
  float* part_mz;                     // workspace: [cta][2][16] the weights' reference of a part and log2 of its sum
  float* part_o;                      // workspace: [cta][2][16][D] weighted values relative to that reference
  float scale_log2;                   // softmax scale * log2(e)
  int T, Hq, Hkv, group, B, max_pages, page_log2, num_pages, causal, window, ctas;
  int few_rows;                       // requests with more rows per key/value head than this go to kv_prefill_kernel
  int most_rows;                      // (>= few_rows) and those with more than this break the caller's bound: no kernel's
  int tile_rows;                      // query rows that kv_attn_kernel takes at a time: 8 or 16
  uint32_t group_mul;                 // division by group: see by_group
  int group_shift;
  int row_tiles;                      // > 0: one CTA for each request, head and of so many row tiles, nothing is split
};

// n / group for 0 <= n < 2^31 by one multiplication: with 2^shift >= group, group_mul = floor(2^32 (2^shift - group) / group) + 1.
HBL_DEVINL int by_group(const AttnArgs& a, int n) {
  return (int)((__umulhi((uint32_t)n, a.group_mul) + (uint32_t)n) >> a.group_shift);
}

// A request as the kernels see it: whatever the arrays hold, rows stay inside Q and keys inside the table.
struct Request {
  int row0, q, kv;
  int rt, lo, tiles;                  // for kv_attn_kernel: row tiles, first tile of keys, tiles of keys (0: not its request)
  bool few;                           // rows that kv_attn_kernel takes
};

HBL_DEVINL Request request_of(const AttnArgs& a, int b) {
  Request r;
  r.row0 = min(max(a.cu_q[b], 0), a.T);
  r.q = min(max(a.cu_q[b + 1], r.row0), a.T) - r.row0;
  r.kv = (int)min((long long)max(a.kv_lens[b], 0), (long long)a.max_pages << a.page_log2);
  r.few = (long long)r.q * a.group <= a.few_rows;
  r.rt = (r.q * a.group + a.tile_rows - 1) >> (a.tile_rows == 8 ? 3 : 4);
  // tiles from the first key that any of its rows sees to the last
  r.lo = a.window > 0 ? max(r.kv - r.q + 1 - a.window, 0) / kAttnTile : 0;
  r.tiles = r.q > 0 && r.few ? (r.kv + kAttnTile - 1) / kAttnTile - r.lo : 0;
  return r;
}
HBL_DEVINL bool prefill_request(const AttnArgs& a, const Request& r) {
  return !r.few && (long long)r.q * a.group <= a.most_rows;
}
HBL_DEVINL long long tiles_of(const AttnArgs& a, const Request& r) { return (long long)r.tiles * r.rt * a.Hkv; }

// Rows beyond the caller's bound belong to no kernel that was launched for them.
HBL_DEVINL void check_bound(const AttnArgs& a, const Request& r) {
  if ((long long)r.q * a.group > a.most_rows) set_device_error(HBL_ERR_INVALID_ARG);
}

HBL_DEVINL void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
HBL_DEVINL void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}
HBL_DEVINL void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N> HBL_DEVINL void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

HBL_DEVINL uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
HBL_DEVINL uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
HBL_DEVINL float2 lds64f(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];\n" : "=f"(v.x), "=f"(v.y) : "r"(a));
  return v;
}
HBL_DEVINL float lds32f(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(v) : "r"(a));
  return v;
}

// Two codes (bytes i, i + 1 of w) as fp16 values u - 128, exactly.
HBL_DEVINL uint32_t sub1152(uint32_t h) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
HBL_DEVINL uint32_t codes_lo(uint32_t w) { return sub1152(__byte_perm(w, 0x64646464u, 0x4140)); }
HBL_DEVINL uint32_t codes_hi(uint32_t w) { return sub1152(__byte_perm(w, 0x64646464u, 0x4342)); }

HBL_DEVINL uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

HBL_DEVINL void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

HBL_DEVINL float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

HBL_DEVINL float log2_scale(float s) { return s > 0.f ? fmaxf(__log2f(s), kLeastScale) : kZeroScale; }

// 1 / l, and 0 for a row without keys.
HBL_DEVINL float over(float l) { return l > 0.f || l != l ? __fdividef(1.f, l) : 0.f; }

// The power of two that brings a row's largest magnitude into [2^14, 2^15), and its inverse.
HBL_DEVINL void row_power(float amax, float* up, float* down) {
  int e = (int)(__float_as_uint(amax) >> 23) - 127;       // exponent; -127 for zero and subnormals
  e = min(max(e, -100), 127);
  *up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
  *down = __uint_as_float((uint32_t)(127 - 14 + e) << 23);
}

// Shared memory of a CTA: each warp's ring of stages (32 tokens of keys, then of values, and 4 scales),
// then the buffer through which the warps' outputs are added, four rows at a time.
template <int D> struct AttnCfg {
  // Warps of a block and blocks of an SM. Twelve warps hold enough bytes in flight; more and smaller blocks hide each
  // other's beginnings and ends of runs, but leave more parts to be joined. Measured, 6 x 2 against 4 x 3: D = 64, 32
  // requests of 5 rows, windows of 1024: 27.4 / 24.8 us; D = 128, one request of 131072: 56.2 / 57.1 us.
  static constexpr int kWarps = D == 64 ? 4 : 6, kCtas = 12 / kWarps;
  static constexpr int kKBytes = kAttnTile * D;
  static constexpr int kStageBytes = 2 * kKBytes + 16;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kMerge = kWarps * 4 * D * 4;
  static constexpr int kSmem = kRing + kMerge + kWarps * kAttnRows * 8;
};

// 16-byte chunk c of token row r of a tile lies at chunk c ^ swz(r), chosen for the reads of a quarter-warp (two
// neighbouring g, four t): keys are read as rows g, chunks t, values as rows 2t + e, chunks g. With 8 chunks to a row
// both then touch every bank once; with 4 chunks the keys do, the values twice.
template <int D> HBL_DEVINL constexpr uint32_t swz(int r) {
  return D == 128 ? (uint32_t)((((r ^ (r >> 2)) & 1) << 2) | (r & 2)) : (uint32_t)((r >> 1) & 3);
}
template <int D> HBL_DEVINL uint32_t tile_at(int r, int c) { return (uint32_t)(r * D) + (((uint32_t)c ^ swz<D>(r)) << 4); }

HBL_DEVINL uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}

// Consecutive tiles [lo, hi) of one request, head and row tile, taken by one CTA.
struct Run {
  Request rq;
  int b, h, rt, lo, hi;
};

template <int D, int NT>   // NT: column tiles of 8 query rows
__global__ void __launch_bounds__(AttnCfg<D>::kWarps * 32, AttnCfg<D>::kCtas) kv_attn_kernel(const AttnArgs a) {
  using C = AttnCfg<D>;
  constexpr int kAttnWarps = C::kWarps;
  constexpr int NK = D / 16;          // k-steps of the score product
  constexpr int NJ = D / 16;          // row tiles of the output product
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long sh[kAttnWarps];
  __shared__ int s_b;
  __shared__ long long s_off;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  // the kernel that joins the parts may take its place as soon as there is room; it waits for this one's end
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");

  Run run;
  long long at, left;                 // tile within the request, over (head, row tile, tile); tiles of this CTA to go
  if (a.row_tiles > 0) {
    const int rt = (int)(blockIdx.x % a.row_tiles), i = (int)(blockIdx.x / a.row_tiles), h = i % a.Hkv;
    run.b = i / a.Hkv;
    run.rq = request_of(a, run.b);
    if (rt == 0 && h == 0 && threadIdx.x == 0) check_bound(a, run.rq);
    if (!run.rq.few || rt >= run.rq.rt) return;
    if (run.rq.tiles == 0) {          // no key at all
      const int row_lo = rt * 8 * NT, rows = min(8 * NT, run.rq.q * a.group - row_lo);
      for (int k = threadIdx.x; k < rows * (D / 8); k += blockDim.x) {
        const int r = row_lo + k / (D / 8);
        const int tok = by_group(a, r);
        const size_t out = (size_t)(run.rq.row0 + tok) * a.Hq + (size_t)(h * a.group + r - tok * a.group);
        reinterpret_cast<uint4*>(a.O + out * D)[k % (D / 8)] = make_uint4(0, 0, 0, 0);
        if (a.lse && k % (D / 8) == 0) a.lse[out] = -INFINITY;
      }
      return;
    }
    at = ((long long)h * run.rq.rt + rt) * run.rq.tiles;
    left = run.rq.tiles;
  } else {
    // this CTA's share [w0, w1) of all tiles, and the request in which it begins
    const int per = (a.B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) sum += tiles_of(a, request_of(a, b));
    long long ex = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, ex, o);
      if (lane >= o) ex += y;
    }
    if (lane == 31) sh[warp] = ex;
    __syncthreads();
    long long total = 0, before = 0;
#pragma unroll
    for (int i = 0; i < kAttnWarps; ++i) {
      if (i < warp) before += sh[i];
      total += sh[i];
    }
    ex += before - sum;
    if (blockIdx.x == 0) {
      long long x = ex;
      for (int b = b0; b < b1; ++b) {
        a.prefix[b] = x;
        x += tiles_of(a, request_of(a, b));
      }
      if (threadIdx.x == 0) a.prefix[a.B] = total;
    }
    const long long n = min(total, (long long)a.ctas);      // no CTA before this one is without a tile
    if (blockIdx.x >= n) return;
    const long long w0 = total * blockIdx.x / n, w1 = total * (blockIdx.x + 1) / n;
    if (ex <= w0 && w0 < ex + sum) {
      long long x = ex;
      for (int b = b0; b < b1; ++b) {
        const long long tiles = tiles_of(a, request_of(a, b));
        if (w0 < x + tiles) { s_b = b; s_off = w0 - x; break; }
        x += tiles;
      }
    }
    __syncthreads();
    run.b = s_b;
    run.rq = request_of(a, run.b);
    at = s_off;
    left = w1 - w0;
  }

  uint8_t* ring = smem + warp * (C::kStages * C::kStageBytes);
  const uint32_t ring_u = (uint32_t)__cvta_generic_to_shared(ring);
  float* merge = reinterpret_cast<float*>(smem + C::kRing);                        // [warp][4][D], chunks permuted
  float2* merge_mz = reinterpret_cast<float2*>(smem + C::kRing + C::kMerge);       // [warp][8 NT]

  // The run that begins at tile `at` of request run.b; every other one is an item from its beginning, found without a
  // division (with four in 64 bits: 16 requests 45 us instead of 43, 2048 of 100 tokens 219 instead of 197).
  auto take = [&](Run& r) {
    r.hi = (int)min((long long)r.rq.tiles, r.lo + left);
    left -= r.hi - r.lo;
  };
  auto open = [&](Run& r) {
    const int item = (int)(at / r.rq.tiles);
    r.lo = (int)(at % r.rq.tiles);
    r.h = item / r.rq.rt;
    r.rt = item % r.rq.rt;
    take(r);
  };
  auto open_next = [&](Run& r) {
    r.lo = 0;
    if (++r.rt == r.rq.rt) {
      r.rt = 0;
      if (++r.h == a.Hkv) {
        r.h = 0;
        do r.rq = request_of(a, ++r.b); while (r.rq.tiles == 0);    // the next request with any tiles
      }
    }
    take(r);
  };

  // Copies of one tile: 32 token rows of keys and of values, and the scales of its (at most two) pages. Rows behind
  // the last key are not fetched; a page outside the cache is recorded, its scales marked -1, which masks its keys. A
  // tile's half lies within one page, so its chunks are consecutive in memory and the offsets below constants.
  const uint32_t dst0 = tile_at<D>(lane / (D / 16), lane % (D / 16));                       // of even copies
  const uint32_t dst1 = tile_at<D>(lane / (D / 16) + 512 / D, lane % (D / 16)) - 512u;      // of odd ones
  const uint32_t block = (uint32_t)D << a.page_log2, step = block * (uint32_t)a.Hkv;        // bytes of a page's head, of a page
  const uint32_t pmask = (1u << a.page_log2) - 1u;
  auto issue = [&](const Run& r, int j, int stage) {
    const uint32_t s0 = ring_u + stage * C::kStageBytes;
    const int key0 = (r.rq.lo + j) * kAttnTile;
    const int32_t* table = a.table + (size_t)r.b * a.max_pages;
    int id[2];
    id[0] = __ldg(table + (key0 >> a.page_log2));
    id[1] = key0 + 16 < r.rq.kv ? __ldg(table + ((key0 + 16) >> a.page_log2)) : 0;
    bool ok[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      ok[e] = id[e] >= 0 && id[e] < a.num_pages;
      if (!ok[e]) set_device_error(HBL_ERR_INVALID_ARG);
    }
    if (lane < 4) {
      const int e = lane & 1;
      const uint32_t dst = s0 + 2 * C::kKBytes + 4 * lane;
      if (e ? ok[1] : ok[0])
        cp_async4(dst, (lane < 2 ? a.kscale : a.vscale) + (size_t)(e ? id[1] : id[0]) * a.Hkv + r.h);
      else
        asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(dst), "f"(-1.f) : "memory");
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (!ok[e]) continue;
      const int key = key0 + 16 * e;
      const uint64_t src = (uint64_t)(uint32_t)id[e] * step + (uint64_t)r.h * block + ((uint32_t)key & pmask) * D + 16 * lane;
      const uint8_t *ks = a.kcodes + src, *vs = a.vcodes + src;
      const int rows = r.rq.kv - key;                       // keys of this half and behind it
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        const uint32_t dst = s0 + 16 * e * D + 512 * k + ((k & 1) ? dst1 : dst0);
        if (512 * k / D + lane / (D / 16) < rows) {
          cp_async16(dst, ks + 512 * k);
          cp_async16(dst + C::kKBytes, vs + 512 * k);
        }
      }
    }
  };
  auto fill = [&](const Run& r) {
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) {
      const int j = r.lo + warp + s * kAttnWarps;
      if (j < r.hi) issue(r, j, s);
      cp_commit();
    }
  };

  // A run's query rows (row g of each column tile), asked for ahead of its first tiles: behind them they would wait for
  // everything that the whole GPU has just asked for. (With two column tiles there are no registers to hold them.)
  uint32_t raw[NT][NK][2];
  auto queries = [&](const Run& r) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int row = min(r.rt * 8 * NT + 8 * i + g, r.rq.q * a.group - 1), tok = by_group(a, row);
      const uint16_t* q = a.Q + (size_t)(r.rq.row0 + tok) * (size_t)a.q_stride + (size_t)(r.h * a.group + row - tok * a.group) * D;
#pragma unroll
      for (int c = 0; c < NK / 4; ++c) {
        const uint4* p = reinterpret_cast<const uint4*>(q + 16 * (t4 + 4 * c));
        const uint4 x = __ldg(p), y = __ldg(p + 1);
        const uint32_t ws[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          raw[i][4 * c + k][0] = ws[2 * k];
          raw[i][4 * c + k][1] = ws[2 * k + 1];
        }
      }
    }
  };
  open(run);
  if constexpr (NT == 1) queries(run);
  fill(run);
  bool first_item = true;
  while (true) {
    const Request& rq = run.rq;
    const int row_lo = run.rt * 8 * NT, rows = min(8 * NT, rq.q * a.group - row_lo);
    // keys that every row, and that any row, of the tile sees
    const int tok_a = by_group(a, row_lo), tok_b = by_group(a, row_lo + rows - 1), pos0 = rq.kv - rq.q;
    const int all_last = a.causal ? min(rq.kv, pos0 + tok_a + 1) : rq.kv;
    const int any_last = a.causal ? min(rq.kv, pos0 + tok_b + 1) : rq.kv;
    const int all_first = a.window > 0 ? max(pos0 + tok_b + 1 - a.window, 0) : 0;
    const int any_first = a.window > 0 ? max(pos0 + tok_a + 1 - a.window, 0) : 0;

    // query fragments: row g of each column tile, scaled by a power of two into fp16
    uint32_t qf[NT][NK][2];
    float qs[NT][2];
    if constexpr (NT > 1) queries(run);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(raw[i][k][e] << 16)),
                                   fabsf(__uint_as_float(raw[i][k][e] & 0xffff0000u))));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      float up, down;
      row_power(amax, &up, &down);
      down *= a.scale_log2;
#pragma unroll
      for (int e = 0; e < 2; ++e) qs[i][e] = __shfl_sync(0xffffffffu, down, 8 * t4 + 4 * e);   // of rows 2 t4 + e
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          qf[i][k][e] = pack_half(__uint_as_float(raw[i][k][e] << 16) * up, __uint_as_float(raw[i][k][e] & 0xffff0000u) * up);
    }

    // this thread's rows are 8 i + 2 t4 + e; output tile jj holds the channels 2 NJ g + 2 jj and the next one
    float o[NT][NJ][4], m[NT][2], ref[NT][2], l[NT][2];      // weights' reference, scores', and the sum relative to that
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int jj = 0; jj < NJ; ++jj)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][jj][e] = 0.f;
      m[i][0] = m[i][1] = ref[i][0] = ref[i][1] = kNothing;
      l[i][0] = l[i][1] = 0.f;
    }

    int stage = 0;
    for (int j = run.lo + warp; j < run.hi; j += kAttnWarps) {
      const int ahead = j + (C::kStages - 1) * kAttnWarps;
      if (ahead < run.hi) issue(run, ahead, stage == 0 ? C::kStages - 1 : stage - 1);
      cp_commit();
      cp_wait<C::kStages - 1>();
      __syncwarp();
      const uint32_t s0 = ring_u + stage * C::kStageBytes;
      const int key0 = (rq.lo + j) * kAttnTile;
      if (key0 < any_last && key0 + kAttnTile > any_first) {
        // scores: token tile h holds the keys key0 + 16 h + g and 8 more of its rows, and lies within a page
        float s[NT][2][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) s[i][hh][0] = s[i][hh][1] = s[i][hh][2] = s[i][hh][3] = 0.f;
#pragma unroll
        for (int c = 0; c < NK / 4; ++c)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const uint4 x = lds128(s0 + tile_at<D>(16 * hh + g, t4 + 4 * c)), y = lds128(s0 + tile_at<D>(16 * hh + g + 8, t4 + 4 * c));
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t kf[4] = {codes_lo(xs[k]), codes_lo(ys[k]), codes_hi(xs[k]), codes_hi(ys[k])};
#pragma unroll
              for (int i = 0; i < NT; ++i) mma_f16(s[i][hh], kf, qf[i][4 * c + k][0], qf[i][4 * c + k][1]);
            }
          }
        const float2 ks = lds64f(s0 + 2 * C::kKBytes);
        const float2 vs = lds64f(s0 + 2 * C::kKBytes + 8);
        float lv[2] = {log2_scale(vs.x), log2_scale(vs.y)};
        const bool whole = key0 >= all_first && key0 + kAttnTile <= all_last && ks.x >= 0.f && ks.y >= 0.f;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[i][0][e] *= ks.x * qs[i][e & 1];
            s[i][1][e] *= ks.y * qs[i][e & 1];
          }
        if (!whole) {
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int pos = pos0 + by_group(a, min(row_lo + 8 * i + 2 * t4 + e, rq.q * a.group - 1));
              const int last = a.causal ? min(rq.kv, pos + 1) : rq.kv;
              const int first = a.window > 0 ? pos + 1 - a.window : 0;
#pragma unroll
              for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                  const int key = key0 + 16 * hh + 8 * f + g;
                  if (key < first || key >= last || (hh ? ks.y : ks.x) < 0.f) s[i][hh][2 * f + e] = -INFINITY;
                }
            }
          // a half of which no row sees anything: its page's scale says nothing
          if (key0 >= any_last || key0 + 16 <= any_first || !(ks.x >= 0.f)) lv[0] = lv[1];
          if (key0 + 16 >= any_last || key0 + 32 <= any_first || !(ks.y >= 0.f)) lv[1] = lv[0];
        }
        // references: raised when any lane's weights have outgrown them
        auto addend = [&](int i, int e, int hh) { return fmaxf(lv[hh] - m[i][e], -ref[i][e] - kSpread); };
        const float quiet = fminf(lv[0], lv[1]);
        bool grown = false;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float s0 = fmaxf(s[i][0][e], s[i][0][e + 2]), s1 = fmaxf(s[i][1][e], s[i][1][e + 2]);
            grown |= fmaxf(s0 + lv[0], s1 + lv[1]) > m[i][e] + (kHead + kLag) || quiet < m[i][e] - ref[i][e] - kSpread;
          }
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float s0 = fmaxf(s[i][0][e], s[i][0][e + 2]), s1 = fmaxf(s[i][1][e], s[i][1][e + 2]);
              float y = fmaxf(s0 + lv[0], s1 + lv[1]), ys = fmaxf(s0, s1);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) {
                y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
                ys = fmaxf(ys, __shfl_xor_sync(0xffffffffu, ys, d));
              }
              const float mn = fmaxf(m[i][e], y - kHead), rn = fmaxf(ref[i][e], ys);
              const float alpha = exp2_fast(m[i][e] - mn);
              l[i][e] *= exp2_fast(ref[i][e] - rn);
              m[i][e] = mn;
              ref[i][e] = rn;
#pragma unroll
              for (int jj = 0; jj < NJ; ++jj) {
                o[i][jj][e] *= alpha;
                o[i][jj][e + 2] *= alpha;
              }
            }
        }
        uint32_t pf[NT][2][2];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const float add[2] = {addend(i, 0, hh), addend(i, 1, hh)};
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = exp2_fast(s[i][hh][e] + add[e & 1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) l[i][e] = __fmaf_rn(p[e] + p[e + 2], exp2_fast(-ref[i][e] - add[e]), l[i][e]);
            // a token's two rows side by side; transposed, a row's two tokens
            pf[i][hh][0] = transpose8(pack_half(p[0], p[1]));
            pf[i][hh][1] = transpose8(pack_half(p[2], p[3]));
          }
        }
        // outputs, 16 tokens at a time: this thread reads the tokens 2 t4 + {0, 1, 8, 9}, channels 2 NJ g and on
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t v[4][NJ / 2];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 16 * hh + 2 * t4 + (e & 1) + 8 * (e >> 1);
            if constexpr (D == 128) {
              const uint4 w = lds128(s0 + C::kKBytes + tile_at<D>(r, g));
              v[e][0] = w.x; v[e][1] = w.y; v[e][2] = w.z; v[e][3] = w.w;
            } else {
              const uint2 w = lds64(s0 + C::kKBytes + tile_at<D>(r, g >> 1) + 8 * (g & 1));
              v[e][0] = w.x; v[e][1] = w.y;
            }
          }
#pragma unroll
          for (int k = 0; k < NJ / 2; ++k)
#pragma unroll
            for (int f = 0; f < 2; ++f) {                   // channels 4 k + 2 f and the next
              const uint32_t sel = f ? 0x7362 : 0x5140;
              const uint32_t c0 = __byte_perm(v[0][k], v[1][k], sel), c8 = __byte_perm(v[2][k], v[3][k], sel);
              const uint32_t vf[4] = {codes_lo(c0), codes_hi(c0), codes_lo(c8), codes_hi(c8)};
#pragma unroll
              for (int i = 0; i < NT; ++i) mma_f16(o[i][2 * k + f], vf, pf[i][hh][0], pf[i][hh][1]);
            }
        }
      }
      __syncwarp();
      stage = stage + 1 == C::kStages ? 0 : stage + 1;
    }
    // the ring is this run's no longer
    const bool more = left > 0;
    Run next = run;
    cp_wait<0>();
    __syncwarp();
    if (more) {
      open_next(next);
      if constexpr (NT == 1) queries(next);
      fill(next);
    }

    // join the warps' results
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], d);
        if (g == 0) merge_mz[warp * 8 * NT + 8 * i + 2 * t4 + e] = make_float2(m[i][e], ref[i][e] + __log2f(l[i][e]));
      }
    const bool final_ = run.lo == 0 && run.hi == rq.tiles;
    const size_t slot = ((size_t)blockIdx.x * 2 + (first_item ? 0 : 1)) * kAttnRows;
#pragma unroll
    for (int pass = 0; pass < 2 * NT; ++pass) {             // rows 4 pass .. 4 pass + 3
      if (4 * pass >= rows) break;
      if ((t4 >> 1) == (pass & 1)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* dst = merge + (warp * 4 + 2 * (t4 & 1) + e) * D;
#pragma unroll
          for (int c = 0; c < NJ / 2; ++c) {
            const auto& u = o[pass >> 1][2 * c];
            const auto& w = o[pass >> 1][2 * c + 1];
            const int ch = (NJ / 2) * g + c;                // chunk of four channels, moved by the row pair
            *reinterpret_cast<float4*>(dst + 4 * (ch ^ (t4 & 1))) = make_float4(u[e], u[e + 2], w[e], w[e + 2]);
          }
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < D; i += blockDim.x) {   // 4 rows x D / 4 chunks
        const int rr = i / (D / 4), ch = i % (D / 4), r = 4 * pass + rr;
        if (r < rows) {
          float M = kNothing, Z = -INFINITY, L = 0.f;
#pragma unroll
          for (int k = 0; k < kAttnWarps; ++k) {
            M = fmaxf(M, merge_mz[k * 8 * NT + r].x);
            Z = fmaxf(Z, merge_mz[k * 8 * NT + r].y);
          }
          Z = Z == -INFINITY ? 0.f : Z;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < kAttnWarps; ++k) {
            const float2 mz = merge_mz[k * 8 * NT + r];
            const float f = exp2_fast(mz.x - M);
            const float4 v = *reinterpret_cast<const float4*>(merge + (k * 4 + rr) * D + 4 * (ch ^ (rr >> 1)));
            L += exp2_fast(mz.y - Z);
            acc.x += v.x * f; acc.y += v.y * f; acc.z += v.z * f; acc.w += v.w * f;
          }
          const int d = 4 * ch;
          if (final_) {
            const int row = row_lo + r;
            const int tok = by_group(a, row);
            const size_t out = (size_t)(rq.row0 + tok) * a.Hq + (size_t)(run.h * a.group + row - tok * a.group);
            const float root = exp2_fast(0.5f * (M - Z)), inv = root * over(L);   // 2^(M - Z) itself may have no place in fp32
            uint2 y;
            y.x = (uint32_t)float_to_bf16_bits(acc.x * inv * root) | ((uint32_t)float_to_bf16_bits(acc.y * inv * root) << 16);
            y.y = (uint32_t)float_to_bf16_bits(acc.z * inv * root) | ((uint32_t)float_to_bf16_bits(acc.w * inv * root) << 16);
            *reinterpret_cast<uint2*>(a.O + out * D + d) = y;
            if (a.lse && ch == 0) a.lse[out] = L == 0.f ? -INFINITY : Z * kLn2 + logf(L);
          } else {
            *reinterpret_cast<float4*>(a.part_o + (slot + r) * D + d) = acc;
            if (ch == 0) *reinterpret_cast<float2*>(a.part_mz + 2 * (slot + r)) = make_float2(M, Z + __log2f(L));
          }
        }
      }
      __syncthreads();
    }
    first_item = false;
    if (!more) break;
    run = next;
  }
}

// Joins the parts of rows whose keys were split between CTAs, and writes the rows that see nothing at all. KW
// warps for each (request, key/value head, row), `rows` of them for each request and head, or (rows = 0) for each
// (token, query head); each takes every KW-th part, and what it has to read of them depends on nothing but their numbers.
template <int D, int KW>
__global__ void __launch_bounds__(256) kv_combine_kernel(const AttnArgs a, const int rows) {
  constexpr int V = D / 32;                                 // channels of a lane
  constexpr int kPer = 8 / KW;                              // rows of a block
  __shared__ float s_acc[kPer][KW][D];
  __shared__ float2 s_mz[kPer][KW];
  __shared__ float s_l[kPer][KW];
  const int lane = threadIdx.x & 31, k = (threadIdx.x >> 5) % KW, half = threadIdx.x / (32 * KW);
  const long long i = (long long)blockIdx.x * kPer + half;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  int b, r, h;
  bool mine;                                                // the row is there and is to be written here
  if (rows > 0) {
    const long long pair = i / rows;
    r = (int)(i - pair * rows);
    b = (int)(pair / a.Hkv);
    h = (int)(pair - (long long)b * a.Hkv);
    mine = b < a.B;
  } else {
    const int t = (int)(i / a.Hq), head = (int)(i - (long long)t * a.Hq);
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu_q[mid] <= t) lo = mid; else hi = mid;
    }
    b = lo;
    h = by_group(a, head);
    mine = t < a.T;
    r = mine ? (t - request_of(a, b).row0) * a.group + head - h * a.group : 0;
    mine = mine && r >= 0;
  }
  size_t row = 0;
  float M = kNothing, Z = -INFINITY, L = 0.f, acc[V] = {};   // weighted values relative to 2^M, sum relative to 2^Z
  if (mine) {
    const Request rq = request_of(a, b);
    if (r == 0 && h == 0 && k == 0 && lane == 0) check_bound(a, rq);
    mine = rq.few && r < rq.q * a.group;
    const int tok = by_group(a, r);
    row = (size_t)(rq.row0 + tok) * a.Hq + (size_t)(h * a.group + r - tok * a.group);
    if (mine && rq.tiles > 0) {
      const long long total = a.prefix[a.B], n = min(total, (long long)a.ctas);
      const long long x0 = a.prefix[b] + (long long)(h * rq.rt + r / a.tile_rows) * rq.tiles, x1 = x0 + rq.tiles - 1;
      // CTA c holds the tiles from total * c / n on
      const int c0 = (int)(((x0 + 1) * n + total - 1) / total) - 1;
      const int c1 = (int)(((x1 + 1) * n + total - 1) / total) - 1;
      mine = c0 < c1;                                       // else written by that CTA
      if (mine) {
        // the first part is its CTA's last item, unless the CTA begins with it; every other one is its CTA's first
        const int tail = total * c0 / n != x0;
        for (int c = c0 + k; c <= c1; c += 4 * KW) {        // four parts at a time, all asked for before the first is used
          float2 mz[4];
          float v[4][V];
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const int at = c + p * KW;
            mz[p] = make_float2(kNothing, -INFINITY);
#pragma unroll
            for (int e = 0; e < V; ++e) v[p][e] = 0.f;
            if (at <= c1) {
              const size_t slot = ((size_t)at * 2 + (at == c0 ? tail : 0)) * kAttnRows + r % a.tile_rows;
              mz[p] = *reinterpret_cast<const float2*>(a.part_mz + 2 * slot);
              const float* o = a.part_o + slot * D + V * lane;
              if constexpr (V == 4) *reinterpret_cast<float4*>(v[p]) = *reinterpret_cast<const float4*>(o);
              else *reinterpret_cast<float2*>(v[p]) = *reinterpret_cast<const float2*>(o);
            }
          }
          const float mn = fmaxf(M, fmaxf(fmaxf(mz[0].x, mz[1].x), fmaxf(mz[2].x, mz[3].x)));
          const float zn = fmaxf(Z, fmaxf(fmaxf(mz[0].y, mz[1].y), fmaxf(mz[2].y, mz[3].y)));
          const float f0 = exp2_fast(M - mn), mu = zn == -INFINITY ? 0.f : zn;
          M = mn;
          L *= exp2_fast(Z - mu);
          Z = zn;
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] *= f0;
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const float f = exp2_fast(mz[p].x - mn);
            L += exp2_fast(mz[p].y - mu);
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] += v[p][e] * f;
          }
        }
      }
    }
  }
  if constexpr (KW > 1) {
#pragma unroll
    for (int e = 0; e < V; ++e) s_acc[half][k][V * lane + e] = acc[e];
    if (lane == 0) {
      s_mz[half][k] = make_float2(M, Z);
      s_l[half][k] = L;
    }
    __syncthreads();
    M = kNothing;
    Z = -INFINITY;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      M = fmaxf(M, s_mz[half][w].x);
      Z = fmaxf(Z, s_mz[half][w].y);
    }
    const float mu = Z == -INFINITY ? 0.f : Z;
    L = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      const float f = exp2_fast(s_mz[half][w].x - M);
      L += s_l[half][w] * exp2_fast(s_mz[half][w].y - mu);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += s_acc[half][w][V * lane + e] * f;
    }
  }
  if (!mine || k != 0) return;
  Z = Z == -INFINITY ? 0.f : Z;
  const float root = exp2_fast(0.5f * (M - Z)), inv = root * over(L);
#pragma unroll
  for (int e = 0; e < V; e += 2)
    *reinterpret_cast<uint32_t*>(a.O + row * D + V * lane + e) = (uint32_t)float_to_bf16_bits(acc[e] * inv * root) |
                                                                 ((uint32_t)float_to_bf16_bits(acc[e + 1] * inv * root) << 16);
  if (a.lse && lane == 0) a.lse[row] = L == 0.f ? -INFINITY : Z * kLn2 + logf(L);
}

}  // namespace kv
}  // namespace hbl
