// Attention over the paged 8-bit key/value cache: few query rows per key/value head (single tokens, drafts).
//
//   O_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = exp(scale * q_r . k_j - m_r)  over the keys j that row r sees,
// with k_j = (u_j - 128) * s of the key's block. Rows of one request that share a key/value head (its query
// heads times its new tokens) are taken 16 at a time, so the cache is read once for all of them.
//
// The bound is the cache read: D bytes of keys and D of values for each token and head, with
// 4 * 16 * D multiply-adds on them. The kernel is therefore a stream over tiles of 32 tokens:
//   * one CTA per SM, each with an equal share of all tiles of all requests and heads (the long axis is
//     split wherever the share ends), tiles dealt to 8 warps in turn;
//   * each warp has a ring of its own in shared memory, filled with 16-byte cp.async, and its own running
//     maximum, sum and output in registers: no barrier while it streams;
//   * codes become fp16 exactly (0x6400 | u is 1024 + u; minus 1152), the query rows are scaled by a power of
//     two into fp16's range (exact but for what lies 2^-25 below the row's largest value), and both products
//     run on mma.m16n8k16 with fp32 sums. A 128-row tcgen05 tile would be at least 7/8 padding here;
//   * a block's key scale multiplies the scores, its value scale the probabilities, relative to the largest
//     value scale met so far, which keeps them inside fp16's range; they are rounded to fp16 (11 bits), finer than the
//     bf16 output.
// At the end of a run the warps' results are added through shared memory. A run that is only a part of its
// row's keys goes to the workspace, and kv_combine_kernel joins the parts.
#pragma once
#include "hbl_common.cuh"
#include <cuda_fp16.h>

namespace hbl {
namespace kv {

constexpr int kAttnWarps = 8;
constexpr int kAttnTile = 32;         // tokens of a warp's tile
constexpr int kAttnRows = 16;         // query rows of a tile
constexpr int kMaxAttnCtas = 256;     // workspace is laid out for this many
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
  float* part_ml;                     // workspace: [cta][2][16] maximum and sum
  float* part_o;                      // workspace: [cta][2][16][D]
  float scale_log2;                   // softmax scale * log2(e)
  int T, Hq, Hkv, group, B, max_pages, page_log2, num_pages, causal, window, ctas;
  int few_rows;                       // requests with more rows per key/value head than this go to kv_prefill_kernel
  int most_rows;                      // and those with more than this break the caller's bound
};

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
  r.rt = (int)(((long long)r.q * a.group + kAttnRows - 1) / kAttnRows);
  // tiles from the first key that any of its rows sees to the last
  r.lo = a.window > 0 ? max(r.kv - r.q + 1 - a.window, 0) / kAttnTile : 0;
  r.tiles = r.q > 0 && r.few ? (r.kv + kAttnTile - 1) / kAttnTile - r.lo : 0;
  return r;
}
HBL_DEVINL bool prefill_request(const AttnArgs& a, const Request& r) {
  return !r.few && (long long)r.q * a.group <= a.most_rows;
}
HBL_DEVINL long long tiles_of(const AttnArgs& a, const Request& r) { return (long long)r.tiles * r.rt * a.Hkv; }

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

// The power of two that brings a row's largest magnitude into [2^14, 2^15), and its inverse.
HBL_DEVINL void row_power(float amax, float* up, float* down) {
  int e = (int)(__float_as_uint(amax) >> 23) - 127;       // exponent; -127 for zero and subnormals
  e = min(max(e, -100), 120);
  *up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
  *down = __uint_as_float((uint32_t)(127 - 14 + e) << 23);
}

// Shared memory of a CTA: each warp's ring of stages (32 tokens of keys, then of values, and 4 scales),
// then the buffer through which the warps' outputs are added.
template <int D> struct AttnCfg {
  static constexpr int kKBytes = kAttnTile * D;
  static constexpr int kStageBytes = 2 * kKBytes + 16;
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kRing = kAttnWarps * kStages * kStageBytes;
  static constexpr int kMerge = kAttnWarps * 8 * D * 4;
  static constexpr int kSmem = kRing + kMerge + kAttnWarps * kAttnRows * 8;
};

// 16-byte chunk c of token row r of a tile lies at chunk c ^ swz(r): the key reads (rows 4g + i, chunks t)
// and the value reads (rows 8t + e, chunk g) of a quarter-warp then fall on different banks.
template <int D> HBL_DEVINL uint32_t tile_at(int r, int c) {
  if constexpr (D == 128) return (uint32_t)(r * 128 + ((c ^ (r & 7) ^ ((r >> 3) << 1)) & 7) * 16);
  else return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3) ^ (r >> 3)) & 3) * 16);
}

template <int D>
__global__ void __launch_bounds__(kAttnWarps * 32, 1) kv_attn_kernel(const AttnArgs a) {
  using C = AttnCfg<D>;
  constexpr int NK = D / 16;          // k-steps of the score product
  constexpr int NJ = D / 8;           // column tiles of the output
  constexpr int CPR = D / 16;         // 16-byte chunks of a token row
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long sh[9];
  __shared__ int s_b;
  __shared__ long long s_off;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const int P = 1 << a.page_log2;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");

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

  uint8_t* ring = smem + warp * (C::kStages * C::kStageBytes);
  const uint32_t ring_u = (uint32_t)__cvta_generic_to_shared(ring);
  float* merge = reinterpret_cast<float*>(smem + C::kRing);                        // [warp][8][D], chunks permuted
  float2* merge_ml = reinterpret_cast<float2*>(smem + C::kRing + C::kMerge);       // [warp][16]

  int b = s_b;
  Request rq = request_of(a, b);
  long long at = s_off;               // tile within the request, over (head, row tile, tile)
  bool first_item = true;
  for (long long w = w0; w < w1;) {
    while (at >= tiles_of(a, rq)) {   // the next request with any tiles
      at = 0;
      rq = request_of(a, ++b);
    }
    const int item = (int)(at / rq.tiles), lo = (int)(at % rq.tiles);
    const int h = item / rq.rt, rt = item % rq.rt;
    const int hi = (int)min((long long)rq.tiles, lo + (w1 - w));
    // tiles [lo, hi) of this item; token tile j starts at key (rq.lo + j) * 32
    const int row_lo = rt * kAttnRows, rows = min(kAttnRows, rq.q * a.group - row_lo);
    // keys that row r of the tile sees: [first, last)
    int first[2], last[2], tok[2], head[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = min(row_lo + g + 8 * i, rq.q * a.group - 1);
      tok[i] = r / a.group;
      head[i] = h * a.group + r % a.group;
      const int pos = rq.kv - rq.q + tok[i];
      last[i] = a.causal ? max(min(rq.kv, pos + 1), 0) : rq.kv;
      first[i] = a.window > 0 ? max(pos + 1 - a.window, 0) : 0;
    }
    // keys that every row of the tile sees
    const int tok_a = row_lo / a.group, tok_b = (row_lo + rows - 1) / a.group;
    const int all_last = a.causal ? min(rq.kv, rq.kv - rq.q + tok_a + 1) : rq.kv;
    const int any_last = a.causal ? min(rq.kv, rq.kv - rq.q + tok_b + 1) : rq.kv;
    const int all_first = a.window > 0 ? max(rq.kv - rq.q + tok_b + 1 - a.window, 0) : 0;
    const int any_first = a.window > 0 ? max(rq.kv - rq.q + tok_a + 1 - a.window, 0) : 0;

    // query fragments, scaled by a power of two into fp16
    uint32_t qf[NK][4];
    float qs[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint16_t* q = a.Q + (size_t)(rq.row0 + tok[i]) * (size_t)a.q_stride + (size_t)head[i] * D;
      uint32_t raw[NK][2];
      float amax = 0.f;
#pragma unroll
      for (int c = 0; c < NK / 4; ++c) {
        const uint4* p = reinterpret_cast<const uint4*>(q + 16 * (t4 + 4 * c));
        const uint4 x = __ldg(p), y = __ldg(p + 1);
        const uint32_t ws[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          raw[4 * c + k][0] = ws[2 * k];
          raw[4 * c + k][1] = ws[2 * k + 1];
        }
      }
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(raw[k][e] << 16)),
                                   fabsf(__uint_as_float(raw[k][e] & 0xffff0000u))));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      float up;
      row_power(amax, &up, &qs[i]);
      qs[i] *= a.scale_log2;
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          qf[k][2 * e + i] = pack_half(__uint_as_float(raw[k][e] << 16) * up,
                                       __uint_as_float(raw[k][e] & 0xffff0000u) * up);
    }

    float o[NJ][4];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, vref = 0.f;

    // Copies of one tile: 32 token rows of keys and of values, and the scales of its (at most two) pages.
    // A page outside the cache is recorded and its scales marked -1, which masks its keys.
    const int32_t* table = a.table + (size_t)b * a.max_pages;
    auto issue = [&](int j, int stage) {
      const uint32_t s0 = ring_u + stage * C::kStageBytes;
      const int key0 = (rq.lo + j) * kAttnTile;
      int id[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = key0 + 16 * e;
        id[e] = key < rq.kv ? __ldg(table + (key >> a.page_log2)) : 0;
        if (id[e] < 0 || id[e] >= a.num_pages) {
          set_device_error(HBL_ERR_INVALID_ARG);
          id[e] = -1;
        }
      }
      if (lane < 4) {
        const int p = id[lane & 1];
        const uint32_t dst = s0 + 2 * C::kKBytes + 4 * lane;
        if (p >= 0) cp_async4(dst, (lane < 2 ? a.kscale : a.vscale) + (size_t)p * a.Hkv + h);
        else asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(dst), "f"(-1.f) : "memory");
      }
#pragma unroll
      for (int k = 0; k < CPR; ++k) {
        const int i = lane + 32 * k, r = i / CPR, c = i % CPR, key = key0 + r;
        const int p = id[r >> 4];
        if (key < rq.kv && p >= 0) {
          const size_t src = ((((size_t)p * a.Hkv + h) << a.page_log2) + (size_t)(key & (P - 1))) * D + 16 * c;
          cp_async16(s0 + tile_at<D>(r, c), a.kcodes + src);
          cp_async16(s0 + C::kKBytes + tile_at<D>(r, c), a.vcodes + src);
        }
      }
    };

    const int j0 = lo + warp;
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) {
      if (j0 + s * kAttnWarps < hi) issue(j0 + s * kAttnWarps, s);
      cp_commit();
    }
    int stage = 0;
    for (int j = j0; j < hi; j += kAttnWarps) {
      const int ahead = j + (C::kStages - 1) * kAttnWarps;
      if (ahead < hi) issue(ahead, stage == 0 ? C::kStages - 1 : stage - 1);
      cp_commit();
      cp_wait<C::kStages - 1>();
      __syncwarp();
      const uint32_t s0 = ring_u + stage * C::kStageBytes;
      const int key0 = (rq.lo + j) * kAttnTile;
      if (key0 < any_last && key0 + kAttnTile > any_first) {
        // scores: tile i holds the keys 4c + i of its columns c
        float s[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
          for (int c = 0; c < NK / 4; ++c) {
            const uint4 w = lds128(s0 + tile_at<D>(4 * g + i, t4 + 4 * c));
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f16(s[i], qf[4 * c + k], codes_lo(ws[k]), codes_hi(ws[k]));
          }
        }
        // this thread's keys are 8 t4 .. 8 t4 + 7, all of one page
        const float ks = lds32f(s0 + 2 * C::kKBytes + 4 * (t4 >> 1));
        float vs = lds32f(s0 + 2 * C::kKBytes + 8 + 4 * (t4 >> 1));
        const int key = key0 + 8 * t4;
        const bool whole = key0 >= all_first && key0 + kAttnTile <= all_last && !__any_sync(0xffffffffu, ks < 0.f);
        const float f[2] = {qs[0] * ks, qs[1] * ks};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][e] *= f[e >> 1];
        if (!whole) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int k = key + i + 4 * (e & 1);
              if (k < first[e >> 1] || k >= last[e >> 1] || ks < 0.f) s[i][e] = -INFINITY;
            }
        }
        // a half tile of which no row sees anything: its page's scale says nothing
        const int half0 = key0 + 16 * (t4 >> 1);
        if (half0 >= any_last || half0 + 16 <= any_first || ks < 0.f) vs = 0.f;
        float vmax = fmaxf(vs, __shfl_xor_sync(0xffffffffu, vs, 2));
        const float vnew = fmaxf(vref, vmax);
        const float vr = vnew > 0.f ? __fdividef(vs, vnew) : 0.f;
        const float shrink = vref == vnew ? 1.f : __fdividef(vref, vnew);
        vref = vnew;
        float alpha[2], mu[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1])),
                          fmaxf(fmaxf(s[2][2 * e], s[2][2 * e + 1]), fmaxf(s[3][2 * e], s[3][2 * e + 1])));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          const float mn = fmaxf(m[e], x);
          mu[e] = mn == -INFINITY ? 0.f : mn;
          alpha[e] = exp2_fast(m[e] - mu[e]);
          m[e] = mn;
        }
        uint32_t pf[2][4];
        float ls[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = exp2_fast(s[i][e] - mu[e >> 1]);
            ls[e >> 1] += p[e];
            p[e] *= vr;
          }
          pf[i >> 1][2 * (i & 1)] = pack_half(p[0], p[1]);
          pf[i >> 1][2 * (i & 1) + 1] = pack_half(p[2], p[3]);
        }
        l[0] = l[0] * alpha[0] + ls[0];
        l[1] = l[1] * alpha[1] + ls[1];
        const float ao[2] = {alpha[0] * shrink, alpha[1] * shrink};
        if (__any_sync(0xffffffffu, ao[0] != 1.f || ao[1] != 1.f)) {
#pragma unroll
          for (int jj = 0; jj < NJ; ++jj)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[jj][e] *= ao[e >> 1];
        }
        // output: column tile jj holds the channels NJ * c + jj of its columns c
#pragma unroll
        for (int half = 0; half < 2; ++half) {            // keys 8 t4 + {0, 4, 1, 5}, then {2, 6, 3, 7}
          uint32_t v[4][NJ / 4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 8 * t4 + 2 * half + (e >> 1) + 4 * (e & 1);
            if constexpr (D == 128) {
              const uint4 w = lds128(s0 + C::kKBytes + tile_at<D>(r, g));
              v[e][0] = w.x; v[e][1] = w.y; v[e][2] = w.z; v[e][3] = w.w;
            } else {
              const uint2 w = lds64(s0 + C::kKBytes + tile_at<D>(r, g >> 1) + 8 * (g & 1));
              v[e][0] = w.x; v[e][1] = w.y;
            }
          }
#pragma unroll
          for (int k = 0; k < NJ / 4; ++k) {
            const uint32_t a0 = __byte_perm(v[0][k], v[1][k], 0x5140), a1 = __byte_perm(v[0][k], v[1][k], 0x7362);
            const uint32_t b0 = __byte_perm(v[2][k], v[3][k], 0x5140), b1 = __byte_perm(v[2][k], v[3][k], 0x7362);
            mma_f16(o[4 * k + 0], pf[half], codes_lo(a0), codes_lo(b0));
            mma_f16(o[4 * k + 1], pf[half], codes_hi(a0), codes_hi(b0));
            mma_f16(o[4 * k + 2], pf[half], codes_lo(a1), codes_lo(b1));
            mma_f16(o[4 * k + 3], pf[half], codes_hi(a1), codes_hi(b1));
          }
        }
      }
      __syncwarp();
      stage = stage + 1 == C::kStages ? 0 : stage + 1;
    }
    cp_wait<0>();
    __syncwarp();

    // add the warps' results
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      if (t4 == 0) merge_ml[warp * kAttnRows + g + 8 * e] = make_float2(m[e], l[e]);
    }
    const bool final_ = lo == 0 && hi == rq.tiles;
    const size_t slot = ((size_t)blockIdx.x * 2 + (first_item ? 0 : 1)) * kAttnRows;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      // rows 8e .. 8e + 7: this thread's channels are 2 NJ t4 + jj (columns 2 t4) and NJ more; 16-byte chunk c
      // of that run of 2 NJ lies at c ^ (4 (g & 1) + t4)
      if (8 * e < rows) {
#pragma unroll
        for (int c = 0; c < NJ / 2; ++c) {
          const int jj = 4 * (c % (NJ / 4)), col = c / (NJ / 4);
          const float4 v = make_float4(o[jj][2 * e + col] * vref, o[jj + 1][2 * e + col] * vref,
                                       o[jj + 2][2 * e + col] * vref, o[jj + 3][2 * e + col] * vref);
          const int pc = c ^ ((4 * (g & 1) + t4) & (NJ / 2 - 1));
          *reinterpret_cast<float4*>(merge + (warp * 8 + g) * D + 2 * NJ * t4 + 4 * pc) = v;
        }
      }
      __syncthreads();
      if (8 * e < rows) {
        for (int i = threadIdx.x; i < 8 * (D / 4); i += blockDim.x) {
          const int gr = i / (D / 4), ch = i % (D / 4), r = 8 * e + gr;
          if (r < rows) {
            const int tt = ch / (NJ / 2), pc = (ch % (NJ / 2)) ^ ((4 * (gr & 1) + tt) & (NJ / 2 - 1));
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int k = 0; k < kAttnWarps; ++k) M = fmaxf(M, merge_ml[k * kAttnRows + r].x);
            const float mu = M == -INFINITY ? 0.f : M;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kAttnWarps; ++k) {
              const float2 ml = merge_ml[k * kAttnRows + r];
              const float f = exp2_fast(ml.x - mu);
              const float4 v = *reinterpret_cast<const float4*>(merge + (k * 8 + gr) * D + 2 * NJ * tt + 4 * pc);
              L += ml.y * f;
              acc.x += v.x * f; acc.y += v.y * f; acc.z += v.z * f; acc.w += v.w * f;
            }
            const int d = 4 * ch;
            if (final_) {
              const int rr = row_lo + r;
              const size_t out = (size_t)(rq.row0 + rr / a.group) * a.Hq + (size_t)(h * a.group + rr % a.group);
              const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
              uint2 y;
              y.x = (uint32_t)float_to_bf16_bits(acc.x * inv) | ((uint32_t)float_to_bf16_bits(acc.y * inv) << 16);
              y.y = (uint32_t)float_to_bf16_bits(acc.z * inv) | ((uint32_t)float_to_bf16_bits(acc.w * inv) << 16);
              *reinterpret_cast<uint2*>(a.O + out * D + d) = y;
              if (a.lse && ch == 0) a.lse[out] = L > 0.f || L != L ? M * kLn2 + logf(L) : -INFINITY;
            } else {
              *reinterpret_cast<float4*>(a.part_o + (slot + r) * D + d) = acc;
              if (ch == 0) {
                a.part_ml[2 * (slot + r)] = M;
                a.part_ml[2 * (slot + r) + 1] = L;
              }
            }
          }
        }
      }
      __syncthreads();
    }
    first_item = false;
    w += hi - lo;
    at += hi - lo;
  }
}

// Joins the parts of rows whose keys were split between CTAs, and writes the rows that see nothing at all.
// One warp per (request, key/value head, row), `rows` of them for each request and head.
template <int D>
__global__ void __launch_bounds__(256) kv_combine_kernel(const AttnArgs a, const int rows) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lo = (int)(i / ((long long)rows * a.Hkv)), r = (int)(i % rows), h = (int)(i / rows % a.Hkv);
  if (lo >= a.B) return;
  const Request rq = request_of(a, lo);
  if (r == 0 && h == 0 && lane == 0 && (long long)rq.q * a.group > a.most_rows) set_device_error(HBL_ERR_INVALID_ARG);
  if (!rq.few || r >= rq.q * a.group) return;
  const int rt = r / kAttnRows;
  const size_t row = (size_t)(rq.row0 + r / a.group) * a.Hq + (size_t)(h * a.group + r % a.group);
  float M = -INFINITY, L = 0.f;
  constexpr int V = D / 32;                                 // channels of a lane
  float acc[V] = {};
  if (rq.tiles > 0) {
    const long long total = a.prefix[a.B];
    const long long x0 = a.prefix[lo] + (long long)(h * rq.rt + rt) * rq.tiles, x1 = x0 + rq.tiles - 1;
    // CTA c holds the tiles from total * c / n on
    const long long n = min(total, (long long)a.ctas);
    const int c0 = (int)(((x0 + 1) * n + total - 1) / total) - 1;
    const int c1 = (int)(((x1 + 1) * n + total - 1) / total) - 1;
    if (c0 == c1) return;                                   // written by that CTA
    for (int c = c0; c <= c1; ++c) {
      const bool begins = c > c0 || total * c / n == x0;   // the CTA's first item, or its last
      const size_t slot = ((size_t)c * 2 + (begins ? 0 : 1)) * kAttnRows + r % kAttnRows;
      const float m = a.part_ml[2 * slot], l = a.part_ml[2 * slot + 1];
      const float mn = fmaxf(M, m), mu = mn == -INFINITY ? 0.f : mn;
      const float f0 = exp2_fast(M - mu), f1 = exp2_fast(m - mu);
      M = mn;
      L = L * f0 + l * f1;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = acc[i] * f0 + a.part_o[slot * D + V * lane + i] * f1;
    }
  }
  const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
#pragma unroll
  for (int i = 0; i < V; i += 2)
    *reinterpret_cast<uint32_t*>(a.O + row * D + V * lane + i) =
        (uint32_t)float_to_bf16_bits(acc[i] * inv) | ((uint32_t)float_to_bf16_bits(acc[i + 1] * inv) << 16);
  if (a.lse && lane == 0) a.lse[row] = L > 0.f || L != L ? M * kLn2 + logf(L) : -INFINITY;
}

}  // namespace kv
}  // namespace hbl
