// Attention over the paged 8-bit key/value cache: many query rows per key/value head (prompts and chunks of
// prompts), on the 5th-generation tensor cores.
//
// Same sums as kv_attn.cuh. Here the products bound it: 4 D multiply-add pairs for each row and key, beside
// one exponential. One CTA takes 256 rows (query tokens times the heads that share a key/value head) of one
// request and streams the keys in tiles of 128:
//   * warps 8..11 read the codes, turn them into fp16 exactly and store them 128B-swizzled (keys and
//     values have the same layout: token rows of 64 channels; the keys are read K-major, the values MN-major);
//   * warp 13 keeps the block scales a few tiles ahead;
//   * warps 12 and 14, one for each half of the rows, issue tcgen05.mma kind::f16: S = Q K^T into TMEM, 64 keys a
//     step (of which two are held), then O += P V with P as the A operand from TMEM;
//   * warps 0..3 and 4..7 (a thread for each of 128 rows, twice) turn S into P in place. While one half's
//     softmax runs, the tensor cores work for the other half: S, P and O of both fill the 512 TMEM columns.
// A block's value scale s enters as an addend of the exponent, log2(s), which costs nothing: P holds weights p s, relative to
// a reference of their own row, 2^7 below the largest. It is raised only when that has grown by 2^8, so the outputs in
// TMEM are rarely rescaled; weights stay below 2^15 and are rounded to fp16. The sum of the p is fp32, relative to a
// reference of the scores alone: each group's weights times 1 / s. Nothing that a row does not see has a part in its result.
// Measured: 2048-row chunks of four requests over up to 8192 keys, 32 query heads on 8 of 128: 735 us, 865 TFLOP/s (52 % of
// the burst cuBLAS rate, 62 % of the sustained one); one prompt of 2048, 32 heads of their own: 69 us, of which
// 9 us for each 256-row item are its beginning and end. A step of 64 keys takes 2340 cycles, of which the tensor cores work
// 1264 (QK with N = 64 is bound by its shared-memory operands, 49 cycles an instruction) and the special function units 1090;
// a scheduler has two softmax warps, a converting one and an issuing one, and what is left is their latencies:
// without the exponentials the kernel would take 14 % less, without the maxima 10 %, without QK 8 %, without the loads 6 %.
// Every wait is bounded, as in gemm_tc.cuh.
#pragma once
#include "gemm_tc.cuh"
#include "kv_attn.cuh"

namespace hbl {
namespace kv {

constexpr int kPreRows = 256;            // query rows of a CTA, in two halves of 128
constexpr int kPreKeys = 128;            // keys of a tile
constexpr int kPreStep = 64;             // keys of a step: scores of two steps are held for each half
constexpr int kPreThreads = 512;
constexpr int kPreGroups = kPreKeys / 16;
constexpr int kPreStepGroups = kPreStep / 16;
constexpr int kPreRing = 4;              // tiles whose scales are held
constexpr int kPreApart = 8;             // the first step's bit, of a tile's: a scale so far below the largest (see kSpread)

template <int D> struct __align__(1024) PreSmem {
  static constexpr int kPanels = D / 64;
  uint8_t q[2][kPanels][128 * 128];
  uint8_t k[2][kPanels][kPreKeys * 128];
  uint8_t v[2][kPanels][kPreKeys * 128];
  // of each tile: [0, 8) key scales of the 16-key groups, [8, 16) log2 of their value scales, [16] bits: the groups that
  // are not in the cache, and from kPreApart the two steps
  float scale[kPreRing][32];
  uint64_t q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2][2], p_full[2][2], o_full[2], o_last[2];
  uint64_t drained[2];
  float down[kPreRows];                  // a row's inverse power of two times the softmax scale
  long long sh[33];
  int item_b;
  int item_off;
  uint32_t tmem_base;
  int abort;
};

// One lane of a converged warp issues; the operands stay warp-uniform, so they need no transfer to uniform
// registers for each instruction.
HBL_DEVINL void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n.reg .pred p, e;\nsetp.ne.b32 p, %4, 0;\nelect.sync _|e, 0xffffffff;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
HBL_DEVINL void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n.reg .pred p, e;\nsetp.ne.b32 p, %4, 0;\nelect.sync _|e, 0xffffffff;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
HBL_DEVINL void commit(uint64_t* bar) {
  asm volatile(
      "{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(tc::su32(bar))
      : "memory");
}

// tc::mbar_wait, but the hardware holds the thread for up to a millisecond at a time: a warp that polls takes issue
// slots from the softmax warps of its scheduler.
HBL_DEVINL bool try_long(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000000;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(tc::su32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
HBL_DEVINL bool wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (try_long(bar, parity)) return true;
  const long long t0 = clock64();
  while (!try_long(bar, parity)) {
    if (*abort) return false;
    if (clock64() - t0 > tc::kSpinLimit) {
      *abort = 1;
      set_device_error(HBL_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

// Instruction descriptor: D fp32, A and B fp16, M = 128, N = n; bit 16: B is MN-major.
HBL_DEVINL uint32_t idesc_f16(int n, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
// An MN-major 128B-swizzled tile: rows (k) of 128 bytes, 8-row groups 1024 bytes apart, the next 64 columns
// `lead` bytes on.
HBL_DEVINL uint64_t smem_desc_mn(uint32_t saddr, uint32_t lead) {
  return (tc::smem_desc_sw128(saddr) & ~((uint64_t)0x3fff << 16)) | ((uint64_t)(lead >> 4) << 16);
}

#define HBL_TMEM_LD16(addr, r)                                                                                   \
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}," \
               " [%16];\n"                                                                                       \
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), \
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),        \
                 "=r"(r[15])                                                                                     \
               : "r"(addr)                                                                                       \
               : "memory")

#define HBL_TMEM_ST16(addr, r)                                                                                   \
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"   \
               "%15,%16};\n" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),      \
               "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),       \
               "r"(r[14]), "r"(r[15])                                                                            \
               : "memory")

HBL_DEVINL uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// As exp2_fast and pack_half, but kept in the order in which they are written.
HBL_DEVINL float exp2_ordered(float x) {
  float y;
  asm volatile("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
HBL_DEVINL uint32_t pack_ordered(float lo, float hi) {
  uint32_t r;
  asm volatile("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

HBL_DEVINL float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The block starts with 128 registers a thread; the converting warps hold 64 bytes in flight for each of keys and
// values, so the others hand theirs over: 2 x 120 + 152 + 112 for four warpgroups of 128 threads.
constexpr int kPreRegsSoftmax = 120, kPreRegsConvert = 152, kPreRegsRest = 112;
static_assert(2 * kPreRegsSoftmax + kPreRegsConvert + kPreRegsRest <= 4 * 128, "registers of the launch");
template <int N> HBL_DEVINL void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N)); }
template <int N> HBL_DEVINL void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N)); }

HBL_DEVINL void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }
HBL_DEVINL void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// The keys that a half's rows see lie in the tiles [lo, hi).
struct TileRange { int lo, hi; };
HBL_DEVINL TileRange tiles_seen(const AttnArgs& a, const Request& rq, int row_a, int row_b) {
  if (row_a > row_b) return {0, 0};
  const int pos0 = rq.kv - rq.q;
  const int last = a.causal ? min(rq.kv, pos0 + by_group(a, row_b) + 1) : rq.kv;
  const int first = a.window > 0 ? max(pos0 + by_group(a, row_a) + 1 - a.window, 0) : 0;
  if (last <= first) return {0, 0};
  return {first / kPreKeys, (last + kPreKeys - 1) / kPreKeys};
}

// Lane g (mod 8) looks up the page of the 16-key group g of a tile: -2 behind the last key, -1 where the page is not in
// the cache. The tables are fetched a tile before the codes are, and looked at only then: a warp stops at the first use
// of what it loads, and no load is to wait for another one.
struct PageLookup {
  int id = -2, raw = -2;
  bool beyond = true;
  HBL_DEVINL void fetch(const AttnArgs& a, const int32_t* table, int kv, int j, int lane) {
    const int key = j * kPreKeys + 16 * (lane & 7);
    beyond = key >= kv;
    raw = beyond ? -2 : __ldg(table + (key >> a.page_log2));
  }
  HBL_DEVINL void settle(const AttnArgs& a) { id = beyond ? -2 : raw < 0 || raw >= a.num_pages ? -1 : raw; }
};

template <int D>
__global__ void __launch_bounds__(kPreThreads, 1) kv_prefill_kernel(const AttnArgs a) {
  using S_t = PreSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  S_t& S = *reinterpret_cast<S_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &S.abort;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&S.q_full[i], 128);
      tc::mbar_init(&S.k_full[i], 129);
      tc::mbar_init(&S.k_empty[i], 2);
      tc::mbar_init(&S.v_full[i], 128);
      tc::mbar_init(&S.v_empty[i], 2);
      tc::mbar_init(&S.s_full[i][0], 1);
      tc::mbar_init(&S.s_full[i][1], 1);
      tc::mbar_init(&S.p_full[i][0], 128);
      tc::mbar_init(&S.p_full[i][1], 128);
      tc::mbar_init(&S.o_full[i], 1);
      tc::mbar_init(&S.o_last[i], 1);
      tc::mbar_init(&S.drained[i], 1);
    }
    S.abort = 0;
    S.item_b = -1;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 12) {
    tc::tmem_alloc(&S.tmem_base, 512);
    tc::tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;\n" ::: "memory");

  // the item of this CTA: request, head and row tile (longest first within a request)
  auto items_of = [&](int b) {
    const Request r = request_of(a, b);
    return prefill_request(a, r) ? (long long)((r.q * (long long)a.group + kPreRows - 1) / kPreRows) * a.Hkv : 0ll;
  };
  {
    const int per = (a.B + kPreThreads - 1) / kPreThreads;
    const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) sum += items_of(b);
    long long ex = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, ex, o);
      if (lane >= o) ex += y;
    }
    if (lane == 31) S.sh[warp] = ex;
    __syncthreads();
    for (int i = 0; i < warp; ++i) ex += S.sh[i];
    ex -= sum;
    if (ex <= blockIdx.x && blockIdx.x < ex + sum) {
      long long x = ex;
      for (int b = b0; b < b1; ++b) {
        const long long n = items_of(b);
        if (blockIdx.x < x + n) {
          S.item_b = b;
          S.item_off = (int)(blockIdx.x - x);
          break;
        }
        x += n;
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  if (S.item_b < 0) {                    // more CTAs were launched than there are items
    if (warp == 12) tc::tmem_dealloc(tmem, 512);
    return;
  }
  const int b = S.item_b;
  const Request rq = request_of(a, b);
  const int nrows = rq.q * a.group;
  const int rts = (nrows + kPreRows - 1) / kPreRows;
  const int rt = rts - 1 - S.item_off / a.Hkv, h = S.item_off % a.Hkv;
  const int row0 = rt * kPreRows;
  TileRange half[2];
#pragma unroll
  for (int w = 0; w < 2; ++w)
    half[w] = tiles_seen(a, rq, row0 + 128 * w, min(row0 + 128 * w + 127, nrows - 1));
  // tiles of the CTA; a half without keys has an empty range
  int lo = 0x7fffffff, hi = 0;
#pragma unroll
  for (int w = 0; w < 2; ++w)
    if (half[w].lo < half[w].hi) {
      lo = min(lo, half[w].lo);
      hi = max(hi, half[w].hi);
    }

  if (warp < 8) {
    // ----- a row's softmax -----
    regs_down<kPreRegsSoftmax>();
    const int w = warp >> 2;
    const int r = row0 + 128 * w + (threadIdx.x & 127);
    const bool live = r < nrows;
    const int tok = by_group(a, min(r, nrows - 1)), head = h * a.group + min(r, nrows - 1) - tok * a.group;
    const int pos = rq.kv - rq.q + tok;
    const int last = a.causal ? max(min(rq.kv, pos + 1), 0) : rq.kv;
    const int first = a.window > 0 ? max(pos + 1 - a.window, 0) : 0;
    {
      // The warp's 32 rows in fp16, each brought into its range by a power of two, to shared memory: two (D = 64: four)
      // rows at a time, a lane for each 16 bytes, so that the loads are whole lines.
      constexpr int LPR = D / 8, RPI = 32 / LPR;           // lanes of a row, rows of a step
      const int base = row0 + 128 * w + 32 * (warp & 3), c = lane % LPR;
      uint4 x[32 / RPI];
#pragma unroll
      for (int i = 0; i < 32 / RPI; ++i) {
        const int rr = min(base + RPI * i + lane / LPR, nrows - 1), t = by_group(a, rr);
        x[i] = __ldg(reinterpret_cast<const uint4*>(a.Q + (size_t)(rq.row0 + t) * (size_t)a.q_stride +
                                                    (size_t)(h * a.group + rr - t * a.group) * D) + c);
      }
      {
#pragma unroll
        for (int i = 0; i < 32 / RPI; ++i) {
          const uint32_t ws[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          float amax = 0.f, up, down;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(ws[k] << 16)), fabsf(__uint_as_float(ws[k] & 0xffff0000u))));
#pragma unroll
          for (int d = 1; d < LPR; d <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
          row_power(amax, &up, &down);
          const int rr = 32 * (warp & 3) + RPI * i + lane / LPR;
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            o[k] = pack_half(__uint_as_float(ws[k] << 16) * up, __uint_as_float(ws[k] & 0xffff0000u) * up);
          sts128(tc::su32(&S.q[w][c >> 3][rr * 128 + (((c & 7) ^ (rr & 7)) << 4)]), make_uint4(o[0], o[1], o[2], o[3]));
          if (c == 0) S.down[128 * w + rr] = down * a.scale_log2;
        }
      }
      fence_async_smem();
      tc::mbar_arrive(&S.q_full[w]);
      __syncwarp();
    }
    const float qs = S.down[threadIdx.x];
    const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t s_addr = lane_base + (uint32_t)(128 * w), o_addr = lane_base + (uint32_t)(256 + 128 * w);
    // keys that every row of this warp sees, for the tiles that need no mask
    const int lane_lo = __reduce_max_sync(0xffffffffu, first), lane_hi = __reduce_min_sync(0xffffffffu, last);
    float m = kNothing, ref = kNothing, l = 0.f;             // weights' reference, scores', and the sum relative to that
    bool ok = true;
    const int steps = 2 * (half[w].hi - half[w].lo);
    for (int n = 0; n < steps; ++n) {
      ok = __all_sync(0xffffffffu, wait(&S.s_full[w][n & 1], (uint32_t)(n >> 1) & 1u, abort));
      if (!ok) break;
      tc::tc_fence_after();
      const int j = half[w].lo + (n >> 1), key0 = j * kPreKeys + kPreStep * (n & 1);
      const uint32_t src = s_addr + (uint32_t)(kPreStep * (n & 1));
      uint32_t x[kPreStep];
      HBL_TMEM_LD32(src, x);
      HBL_TMEM_LD32(src + 32u, (x + 32));
      const uint32_t sc = tc::su32(&S.scale[(j - lo) % kPreRing][0]) + 16u * (n & 1);
      const uint4 kq = lds128(sc), vq = lds128(sc + 32);
      const uint32_t bits = __float_as_uint(S.scale[(j - lo) % kPreRing][16]);
      const uint32_t bad = (bits >> (kPreStepGroups * (n & 1))) & 15u;
      // never zero, so that a masked score (minus infinity) stays one when it is multiplied
      const float least = 1.17549435e-38f;
      const float f[4] = {fmaxf(__uint_as_float(kq.x) * qs, least), fmaxf(__uint_as_float(kq.y) * qs, least),
                          fmaxf(__uint_as_float(kq.z) * qs, least), fmaxf(__uint_as_float(kq.w) * qs, least)};
      // addends of the exponent, relative to the reference; see kSpread
      float add[4];
      auto addends = [&](const uint4& lv) {
        const float lowest = -ref - kSpread;
        add[0] = fmaxf(__uint_as_float(lv.x) - m, lowest);
        add[1] = fmaxf(__uint_as_float(lv.y) - m, lowest);
        add[2] = fmaxf(__uint_as_float(lv.z) - m, lowest);
        add[3] = fmaxf(__uint_as_float(lv.w) - m, lowest);
      };
      addends(vq);
      tc::tc_wait_ld();
      if (!(key0 >= lane_lo && key0 + kPreStep <= lane_hi && bad == 0)) {
        const int c_lo = first - key0, c_hi = last - key0;      // the columns that this row sees
#pragma unroll
        for (int i = 0; i < kPreStep; ++i)
          if (i < c_lo || i >= c_hi || (bad >> (i >> 4)) & 1) x[i] = 0xff800000u;
      }
      float mt = -INFINITY, z[kPreStepGroups];
#pragma unroll
      for (int g = 0; g < kPreStepGroups; ++g) {
        float y[5];
#pragma unroll
        for (int i = 0; i < 5; ++i)
          y[i] = max3(__uint_as_float(x[16 * g + 3 * i]), __uint_as_float(x[16 * g + 3 * i + 1]),
                      __uint_as_float(x[16 * g + 3 * i + 2]));
        z[g] = fmaxf(max3(y[0], y[1], y[2]), max3(y[3], y[4], __uint_as_float(x[16 * g + 15])));
        mt = fmaxf(mt, __fmaf_rn(z[g], f[g], add[g]));
      }
      if (__any_sync(0xffffffffu, mt > kHead + kLag) || (bits >> (kPreApart + (n & 1)) & 1)) {
        const uint4 lv = lds128(sc + 32);
        const float u[4] = {z[0] * f[0], z[1] * f[1], z[2] * f[2], z[3] * f[3]};
        const float most = fmaxf(fmaxf(u[0] + __uint_as_float(lv.x), u[1] + __uint_as_float(lv.y)),
                                 fmaxf(u[2] + __uint_as_float(lv.z), u[3] + __uint_as_float(lv.w)));
        const float mn = mt > kHead + kLag ? fmaxf(m, most - kHead) : m, rn = fmaxf(ref, fmaxf(fmaxf(u[0], u[1]), fmaxf(u[2], u[3])));
        const float ao = exp2_fast(m - mn);
        l *= exp2_fast(ref - rn);
        m = mn;
        ref = rn;
        addends(lv);
        if (n > 0 && __any_sync(0xffffffffu, ao != 1.f)) {
          // Once the products so far are complete. Those up to the last but one are (this step's scores were issued behind
          // them), and the next one waits for this step, so the phase is either this one or just over.
          ok = __all_sync(0xffffffffu, wait(&S.o_full[w], (uint32_t)(n - 1) & 1u, abort));
          if (!ok) break;
          tc::tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < D / 16; ++k) {
            uint32_t o[16];
            HBL_TMEM_LD16(o_addr + 16u * k, o);
            tc::tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * ao);
            HBL_TMEM_ST16(o_addr + 16u * k, o);
          }
        }
      }
      // from weights to p: a block's 1 / s, and the references
      const float back[4] = {exp2_fast(-ref - add[0]), exp2_fast(-ref - add[1]), exp2_fast(-ref - add[2]), exp2_fast(-ref - add[3])};
      // A pair's exponentials take the special function unit 16 cycles; the arithmetic of the pair kLag in front is issued
      // in their shadow, in this order, and never waits for them.
      constexpr int kPairs = kPreStep / 2, kLag = 4;
      uint32_t p[16];
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int i = 0; i < kPairs + kLag; ++i) {
        if (i < kPairs) {
          const float ag = add[i >> 3];
          const float2 y = __ffma2_rn(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])),
                                      make_float2(f[i >> 3], f[i >> 3]), make_float2(ag, ag));
          x[2 * i] = __float_as_uint(exp2_ordered(y.x));
          x[2 * i + 1] = __float_as_uint(exp2_ordered(y.y));
        }
        if (i >= kLag) {
          const int q = i - kLag;
          const float2 e = make_float2(__uint_as_float(x[2 * q]), __uint_as_float(x[2 * q + 1]));
          p[q & 15] = pack_ordered(e.x, e.y);
          sum[q & 1] = q & 6 ? __fadd2_rn(sum[q & 1], e) : e;
          if ((q & 7) == 7) {
            const float2 t = __fadd2_rn(sum[0], sum[1]);
            l = __fmaf_rn(t.x + t.y, back[q >> 3], l);
          }
          if ((q & 15) == 15) HBL_TMEM_ST16(src + 16u * (q >> 4), p);
        }
      }
      tc::tc_wait_st();
      tc::tc_fence_before();
      tc::mbar_arrive(&S.p_full[w][n & 1]);
    }
    // ----- the row's output -----
    const bool any = steps > 0;
    if (any) ok = ok && __all_sync(0xffffffffu, wait(&S.o_last[w], 0, abort));
    if (ok && !*abort) {
      tc::tc_fence_after();
      const bool some = l > 0.f || l != l;
      const float root = exp2_fast(0.5f * (m - ref)), inv = over(l) * root;    // 2^(m - ref) itself may have no place in fp32
      const size_t out = (size_t)(rq.row0 + tok) * a.Hq + head;
      // Each lane has a row; through the place of the half's queries, whose last use is over, a warp's stores become whole
      // lines (two or four rows at a time).
      constexpr int LPR = D / 8, RPI = 32 / LPR;
      const int rr = threadIdx.x & 127;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x[32];
        if (any) {
          HBL_TMEM_LD32(o_addr + 32u * c, x);
          tc::tc_wait_ld();
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float e0 = some ? __uint_as_float(x[8 * k + 2 * i]) * inv * root : 0.f;
            const float e1 = some ? __uint_as_float(x[8 * k + 2 * i + 1]) * inv * root : 0.f;
            y[i] = (uint32_t)float_to_bf16_bits(e0) | ((uint32_t)float_to_bf16_bits(e1) << 16);
          }
          const int ch = 4 * c + k;
          sts128(tc::su32(&S.q[w][ch >> 3][rr * 128 + (((ch & 7) ^ (rr & 7)) << 4)]), make_uint4(y[0], y[1], y[2], y[3]));
        }
      }
      __syncwarp();
      const int base = row0 + 128 * w + 32 * (warp & 3), c = lane % LPR;
#pragma unroll 4
      for (int i = 0; i < 32 / RPI; ++i) {
        const int r2 = 32 * (warp & 3) + RPI * i + lane / LPR, row = base + RPI * i + lane / LPR;
        const uint4 v = lds128(tc::su32(&S.q[w][c >> 3][r2 * 128 + (((c & 7) ^ (r2 & 7)) << 4)]));
        const int t = by_group(a, row);
        if (row < nrows)
          reinterpret_cast<uint4*>(a.O + ((size_t)(rq.row0 + t) * a.Hq + (size_t)(h * a.group + row - t * a.group)) * D)[c] = v;
      }
      if (live && a.lse) a.lse[out] = some ? ref * kLn2 + logf(l) : -INFINITY;
    }
  } else if (warp < 12) {
    // ----- codes to fp16 -----
    regs_up<kPreRegsConvert>();
    // Thread t converts 16 codes of a row, the channels [16 q, 16 q + 16) of panel `pan`, in each of NS sweeps. The
    // 8 threads of a store phase hold an even and an odd row, whose chunks 2 q ^ row fall on different banks.
    const int t = threadIdx.x - 256, q = t & 3;
    const int pan = D == 128 ? (t >> 3) & 1 : 0, r0 = D == 128 ? ((t >> 4) << 1) | ((t >> 2) & 1) : t >> 2;
    constexpr int RPS = 128 * 64 / (D * 4);              // token rows of one sweep of the 128 threads
    constexpr int NS = kPreKeys / RPS;                   // sweeps of a tile
    const int32_t* table = a.table + (size_t)b * a.max_pages;
    const uint32_t pmask = (1u << a.page_log2) - 1u;
    const size_t block = (size_t)D << a.page_log2;       // bytes of a page's head
    const size_t mine = h * block + (size_t)(r0 & pmask) * D + (size_t)(64 * pan + 16 * q);
    const uint8_t* kbase = a.kcodes + mine;
    const uint8_t* vbase = a.vcodes + mine;
    const uint32_t step = (uint32_t)(a.Hkv * block), pbytes = pmask * D;
    PageLookup look;
    // Keys that no row sees are fetched too, from some page: their codes are finite, and they count for nothing.
    auto load = [&](const uint8_t* base, uint4 (&x)[NS]) {
      uint32_t pb = pbytes;
      asm volatile("" : "+r"(pb));                       // the sweeps' addresses are not to be kept in registers
      const int known = max(look.id, 0);
      int id[NS];
#pragma unroll
      for (int s = 0; s < NS; ++s) id[s] = __shfl_sync(0xffffffffu, known, RPS * s / 16 + (RPS > 16 ? r0 >> 4 : 0));
#pragma unroll
      for (int s = 0; s < NS; ++s) x[s] = ldg_stream(base + (uint64_t)(uint32_t)id[s] * step + ((RPS * s * D) & pb));
    };
    const uint32_t to = (uint32_t)(pan * kPreKeys * 128 + r0 * 128);
    const uint32_t c0 = to + (((2 * q) ^ (r0 & 7)) << 4), c1 = to + (((2 * q + 1) ^ (r0 & 7)) << 4);
    auto store = [&](uint8_t (*dst)[kPreKeys * 128], const uint4 (&x)[NS]) {
      const uint32_t base = tc::su32(&dst[0][0]);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        sts128(base + c0 + RPS * 128 * s, make_uint4(codes_lo(x[s].x), codes_hi(x[s].x), codes_lo(x[s].y), codes_hi(x[s].y)));
        sts128(base + c1 + RPS * 128 * s, make_uint4(codes_lo(x[s].z), codes_hi(x[s].z), codes_lo(x[s].w), codes_hi(x[s].w)));
      }
    };
    uint4 kx[NS], vx[NS];
    if (lo < hi) {
      look.fetch(a, table, rq.kv, lo, lane);
      look.settle(a);
      load(kbase, kx);
      load(vbase, vx);
      if (lo + 1 < hi) look.fetch(a, table, rq.kv, lo + 1, lane);
    }
    for (int j = lo; j < hi; ++j) {
      const int n = j - lo, st = n & 1;
      const uint32_t ph = (uint32_t)(n >> 1) & 1u;
      if (n >= 2 && !__all_sync(0xffffffffu, wait(&S.k_empty[st], ph ^ 1u, abort))) break;
      store(S.k[st], kx);
      fence_async_smem();
      tc::mbar_arrive(&S.k_full[st]);
      if (j + 1 < hi) {
        look.settle(a);
        load(kbase, kx);
      }
      if (n >= 2 && !__all_sync(0xffffffffu, wait(&S.v_empty[st], ph ^ 1u, abort))) break;
      store(S.v[st], vx);
      fence_async_smem();
      tc::mbar_arrive(&S.v_full[st]);
      if (j + 1 < hi) {
        load(vbase, vx);
        if (j + 2 < hi) look.fetch(a, table, rq.kv, j + 2, lane);
      }
    }
  } else {
    // ----- tensor cores -----
    regs_down<kPreRegsRest>();
    if (warp == 12 || warp == 14) {
      const int w = (warp - 12) >> 1;
      const TileRange mine = w ? half[1] : half[0];
      const uint32_t id_s = idesc_f16(kPreStep, false), id_o = idesc_f16(D, true);
      constexpr int kTileUnits = D / 64 * kPreKeys * 128 / 16;      // descriptors count in 16 bytes: a tile of Q, K or V
      constexpr int kStepUnits = kPreStep * 128 / 16;               // the second step's rows in a panel
      const uint64_t q_d = tc::smem_desc_sw128(tc::su32(&S.q[w][0][0])), k_d = tc::smem_desc_sw128(tc::su32(&S.k[0][0][0]));
      const uint64_t v_d = smem_desc_mn(tc::su32(&S.v[0][0][0]), kPreKeys * 128);
      const uint32_t s_t = tmem + 128u * w, o_t = tmem + 256u + 128u * w;
      auto all = [](bool x) { return __all_sync(0xffffffffu, x) != 0; };
      // tile t of the CTA: its stage and the phase of its barriers
      auto full = [&](uint64_t* bar, int t) { return all(wait(bar + (t & 1), (uint32_t)(t >> 1) & 1u, abort)); };
      auto scores = [&](int t, int part) {
        const uint64_t kd = k_d + (t & 1) * kTileUnits + part * kStepUnits;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int at = (k >> 2) * (kPreKeys * 128 / 16) + (k & 3) * 2;
          mma_f16_ss(s_t + kPreStep * part, q_d + at, kd + at, id_s, k > 0);
        }
        commit(&S.s_full[w][part]);
      };
      auto outputs = [&](int t, int part, bool first) {
        const uint64_t vd = v_d + (t & 1) * kTileUnits + part * kStepUnits;
#pragma unroll
        for (int k = 0; k < kPreStep / 16; ++k)
          mma_f16_ts(o_t, s_t + kPreStep * part + 8u * k, vd + k * (2048 / 16), id_o, (!first || k > 0) ? 1u : 0u);
        commit(&S.o_full[w]);
      };
      // tiles that only the other half sees: passed on when they have come
      auto skip = [&](int t) {
        if (!full(S.k_full, t)) return false;
        if (lane == 0) tc::mbar_arrive(&S.k_empty[t & 1]);
        if (!full(S.v_full, t)) return false;
        if (lane == 0) tc::mbar_arrive(&S.v_empty[t & 1]);
        return true;
      };
      const int tiles = max(hi - lo, 0), seen = mine.hi - mine.lo, t0 = seen > 0 ? mine.lo - lo : tiles, t1 = t0 + seen;
      bool ok = true;
      for (int t = 0; t < t0 && ok; ++t) ok = skip(t);
      if (ok && seen > 0 && (ok = all(wait(&S.q_full[w], 0, abort)) && full(S.k_full, t0))) {
        tc::tc_fence_after();
#pragma unroll 1
        for (int part = 0; part < 2; ++part) scores(t0, part);
        commit(&S.k_empty[t0 & 1]);
      }
      // The outputs of a step, then the scores of the step after next, into the place of the probabilities just used:
      // while the tensor cores do that, the scores of the next step are ready for the softmax.
      // One copy of the code for both steps of a tile: the warps of a block share the instruction caches.
#pragma unroll 1
      for (int n = 0; n < 2 * seen && ok; ++n) {
        const int t = t0 + (n >> 1), part = n & 1;
        if (part == 0) ok = full(S.v_full, t);
        ok = ok && all(wait(&S.p_full[w][part], (uint32_t)(n >> 1) & 1u, abort));
        if (!ok) break;
        tc::tc_fence_after();
        outputs(t, part, n == 0);
        if (part) commit(&S.v_empty[t & 1]);
        if (n == 2 * seen - 1) commit(&S.o_last[w]);
        if (t + 1 == t1) continue;
        if (part == 0) {
          if (!(ok = full(S.k_full, t + 1))) break;
          tc::tc_fence_after();
        }
        scores(t + 1, part);
        if (part) commit(&S.k_empty[(t + 1) & 1]);
      }
      for (int t = t1; t < tiles && ok; ++t) ok = skip(t);
      commit(&S.drained[w]);
      // outstanding products read shared memory: wait (bounded) until they are done
      const long long c0 = clock64();
      while (!tc::mbar_try_wait(&S.drained[w], 0) && clock64() - c0 < tc::kSpinLimit) {
      }
    } else if (warp == 13) {
      // ----- block scales -----
      // Lane g (mod 8) holds those of group g. The scales of a group that no row of the CTA sees are 1, whatever its page has.
      const int32_t* table = a.table + (size_t)b * a.max_pages;
      const int any_first = a.window > 0 ? max(rq.kv - rq.q + by_group(a, row0) + 1 - a.window, 0) : 0;
      const int any_last = a.causal ? rq.kv - rq.q + by_group(a, min(row0 + kPreRows, nrows) - 1) + 1 : rq.kv;
      float ks = 1.f, vs = 1.f, top = 0.f;                   // top: the largest value scale so far
      bool absent = false;
      PageLookup look;
      auto load = [&](int j) {
        look.settle(a);
        const int key = j * kPreKeys + 16 * (lane & 7);
        ks = vs = 1.f;
        absent = look.id == -1;
        if (look.id >= 0 && key + 16 > any_first && key < any_last) {
          ks = __ldg(a.kscale + (size_t)look.id * a.Hkv + h);
          vs = __ldg(a.vscale + (size_t)look.id * a.Hkv + h);
        }
      };
      if (lo < hi) {
        look.fetch(a, table, rq.kv, lo, lane);
        load(lo);
        if (lo + 1 < hi) look.fetch(a, table, rq.kv, lo + 1, lane);
      }
      for (int j = lo; j < hi; ++j) {
        const int n = j - lo, st = n & 1;
        const float lv = log2_scale(vs);
        const unsigned bad = __ballot_sync(0xffffffffu, absent) & 0xffu;
        top = fmaxf(top, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vs))));    // scales are not negative
        const unsigned apart = __ballot_sync(0xffffffffu, lv < fmaxf(log2_scale(top), kLeastScale) - kSpread);
        // the ring's place is free: k_full of tile n - 1 was signalled behind the scores of tile n - 3, which wait for
        // the probabilities of tile n - 4, its last user
        if (lane < kPreGroups) {
          float* dst = S.scale[n % kPreRing];
          dst[lane] = ks;
          dst[8 + lane] = lv;
          if (lane == 0) {
            dst[16] = __uint_as_float(bad | (apart & 0x0fu ? 1u << kPreApart : 0u) | (apart & 0xf0u ? 2u << kPreApart : 0u));
            if (bad) set_device_error(HBL_ERR_INVALID_ARG);
          }
        }
        if (n >= 2 && !__all_sync(0xffffffffu, wait(&S.k_empty[st], ((uint32_t)(n >> 1) & 1u) ^ 1u, abort))) break;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&S.k_full[st]);
        if (j + 1 < hi) {
          load(j + 1);
          if (j + 2 < hi) look.fetch(a, table, rq.kv, j + 2, lane);
        }
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

}  // namespace kv
}  // namespace hbl
