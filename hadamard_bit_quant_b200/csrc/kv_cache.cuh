// The paged 8-bit key/value cache: page planning, appending and reading back.
//
// The cache of one attention layer is a set of pages. A page holds P
// consecutive tokens of one request; for each key/value head it is one block
// of P x D unsigned codes u and one fp32 scale s, and the block stands for the
// values (u - 128) * s. Keys and values have a cache each.
//
// The scale rule is the absmax rule of the 8-bit quantiser (architecture
// walkthrough, section 3.4, Eq. 7) taken over a block instead of a token:
//   s = max(gamma / 127, 2^-100),  u = 128 + rint(x / s),
// without that rule's epsilon, because a block's codes are rescaled when a
// louder token joins it and must then divide by the very scale they are
// multiplied with.
#pragma once
#include "hbl_common.cuh"

namespace hbl {
namespace kv {

constexpr float kScaleFloor = 7.888609052210118e-31f;   // 2^-100: no division by zero, no overflow of 1 / s
constexpr int kZero = 128;                              // the code of the value 0
constexpr int kMaxRequests = 8192;

// ---------------------------------------------------------------------------
// Page planning.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;   // most threads of a block
constexpr int kPlanCtas = 8;          // blocks of the cluster that takes a large step

// Exclusive prefix sum over the block; *total gets the sum. `sh` holds 33 values.
HBL_DEVINL long long block_scan(long long v, long long* sh, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int nw = blockDim.x >> 5;
    long long w = lane < nw ? sh[lane] : 0;
    const long long w0 = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    sh[lane] = w - w0;
    if (lane == 31) sh[32] = w;
  }
  __syncthreads();
  *total = sh[32];
  return sh[warp] + x - v;
}

// Largest b in [0, B) with a[b] <= i (a ascending, a[0] = 0).
HBL_DEVINL int find_row(const int* a, int B, int i) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

struct PlanArgs {
  const int32_t* new_lens;
  int32_t* kv_lens;
  int32_t* table;
  int32_t* free_pages;
  int32_t* free_count;
  int32_t* cu_q;
  int32_t* slots;
  int32_t* refused;
  int B, page_log2, num_pages, max_pages, T;
};

// One step of the page table (see hbl_kv_plan). Every quantity is a prefix sum over the requests: rows of
// new tokens, pages wanted, pages given back. With those sums in shared memory, each slot, each
// new table entry and each page returned to the stack is found by itself with a binary search. A large step is taken by a
// cluster of blocks: each forms the (short) sums for itself and takes its part of the rest; the lengths and the count,
// which all of them read, are written behind a cluster barrier. Nothing here moves enough bytes to matter: it is bound
// by its chain of dependent loads and barriers (4 requests of 5 rows: 3.7 us a step; 512 requests, 49 K rows: 10 us, by
// one block 33 us).
__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(PlanArgs a) {
  extern __shared__ int sm[];
  int* cu = sm;                       // [B + 1] first row of each request
  int* want = cu + a.B + 1;           // [B + 1] pages taken by the requests before this one
  int* gone = want + a.B + 1;         // [B + 1] pages given back by the requests before this one
  int* len = gone + a.B + 1;          // [B] cached tokens before the step; ~ of it where the request is refused
  __shared__ long long sh[33];
  __shared__ int s_used;
  uint32_t rank, ranks;
  asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctaid.x;\n" : "=r"(ranks));
  const int tid = (int)(rank * blockDim.x + threadIdx.x), threads = (int)(ranks * blockDim.x);
  const int P = 1 << a.page_log2, lg = a.page_log2;
  const long long cap = (long long)a.max_pages << lg;
  const int per = (a.B + (int)blockDim.x - 1) / (int)blockDim.x;
  const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
  auto pages = [&](long long n) { return (int)((n + P - 1) >> lg); };
  if (threadIdx.x == 0) s_used = 0;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int F = min(max(*a.free_count, 0), a.num_pages);

  // rows of new tokens
  long long sum = 0, total;
  for (int b = b0; b < b1; ++b) {
    len[b] = (int)min((long long)max(a.kv_lens[b], 0), cap);
    sum += max(a.new_lens[b], 0);
  }
  long long x = block_scan(sum, sh, &total);
  for (int b = b0; b < b1; ++b) {
    cu[b] = (int)min(x, (long long)a.T);
    x += max(a.new_lens[b], 0);
  }
  if (threadIdx.x == 0) cu[a.B] = (int)min(total, (long long)a.T);
  __syncthreads();

  // pages wanted (low word) and given back (high word); a request that cannot grow at all wants none
  auto pages_of = [&](int b, bool* wide) {
    const long long n = len[b], q = a.new_lens[b], after = max(n + q, 0ll);
    *wide = q > 0 && (after > cap || cu[b + 1] - cu[b] < q);
    if (*wide) return 0ll;
    const int more = pages(after) - pages(n);
    return more >= 0 ? (long long)more : (long long)(-more) << 32;
  };
  bool wide;
  sum = 0;
  for (int b = b0; b < b1; ++b) sum += pages_of(b, &wide);
  x = block_scan(sum, sh, &total);
  const int R = (int)(total >> 32), stock = (int)min((long long)F + R, 0x7fffffffll);
  for (int b = b0; b < b1; ++b) {
    const long long y = pages_of(b, &wide);
    const int take = (int)(y & 0xffffffff), nd = (int)(x & 0xffffffff);
    want[b] = nd;
    gone[b] = (int)(x >> 32);
    const bool ok = !wide && (take == 0 || (long long)nd + take <= stock);
    if (ok && take) atomicMax(&s_used, nd + take);
    if (!ok) len[b] = ~len[b];
    x += y;
  }
  if (threadIdx.x == 0) {
    want[a.B] = (int)(total & 0xffffffff);
    gone[a.B] = R;
  }
  __syncthreads();
  const int used = s_used;

  // i-th page given back in this step, and i-th page handed out: those given back first, then the stack from its top
  auto released = [&](int i) {
    const int b = find_row(gone, a.B, i);
    return a.table[(size_t)b * a.max_pages + (size_t)(pages(len[b]) - (gone[b + 1] - gone[b]) + (i - gone[b]))];
  };
  auto handed = [&](int i) { return i < R ? released(i) : a.free_pages[F - 1 - (i - R)]; };

  // indexes run in 32 bits without a sign: one step behind the last of 2^31 - 1 rows is no int
  for (uint32_t i = tid; i < (uint32_t)a.T; i += threads) {
    const int t = (int)i;
    int slot = -1;
    if (t < cu[a.B]) {
      const int b = find_row(cu, a.B, t), n = len[b];
      if (n >= 0) {
        const int pos = n + (t - cu[b]), pi = pos >> lg, held = pages(n);
        const int id = pi < held ? a.table[(size_t)b * a.max_pages + pi] : handed(want[b] + pi - held);
        if (id >= 0 && id < a.num_pages) slot = (id << lg) + (pos & (P - 1));
        else set_device_error(HBL_ERR_INVALID_ARG);
      }
    }
    a.slots[t] = slot;
  }
  for (uint32_t n = tid; n < (uint32_t)used; n += threads) {
    const int i = (int)n, b = find_row(want, a.B, i);
    a.table[(size_t)b * a.max_pages + (size_t)(pages(len[b]) + (i - want[b]))] = handed(i);
  }
  // what was given back and not handed out again: the last of it lies deepest, so a step that is undone
  // leaves the stack as it was
  for (uint32_t n = (uint32_t)used + tid; n < (uint32_t)R; n += threads) {
    const int i = (int)n;
    const long long at = (long long)F + (R - 1 - i);
    if (at < a.num_pages) a.free_pages[at] = released(i);
    else set_device_error(HBL_ERR_INVALID_ARG);
  }
  for (int b = tid; b <= a.B; b += threads) {
    a.cu_q[b] = cu[b];
    if (b < a.B) a.refused[b] = len[b] < 0;
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  for (int b = tid; b < a.B; b += threads)
    a.kv_lens[b] = len[b] < 0 ? ~len[b] : (int)max((long long)len[b] + a.new_lens[b], 0ll);
  if (tid == 0) *a.free_count = min(stock - used, a.num_pages);
}

// ---------------------------------------------------------------------------
// Appending.
// ---------------------------------------------------------------------------

// A code 128 + rint(x / s), ties to even, of the exact quotient, in the low byte of the result. t holds the
// integer r nearest to x * (1/s) behind 1.5 * 2^23 + 128; r is within one of the answer. The remainder x - r s is exact in fp32
// (it is a multiple of half an ulp of s and not larger than s), so comparing it with s / 2 decides; it is
// hardly ever as large.
HBL_DEVINL uint32_t code_of(float x, float s, float inv, float h) {
  const float magic = 12583040.0f;
  float t = __fmaf_rn(x, inv, magic);
  const float d = __fmaf_rn(-__fsub_rn(t, magic), s, x);
  if (fabsf(d) >= h) {
    const bool odd = __float_as_uint(t) & 1u;               // 128 is even
    if (fabsf(d) > h || odd) t = __fadd_rn(t, copysignf(1.f, d));
  }
  return __float_as_uint(t);
}

// Two bf16 values as the cache takes them: there is no code for NaN (0 is stored) or infinity (the largest
// finite value is stored).
HBL_DEVINL uint32_t finite2(uint32_t w) {
#pragma unroll
  for (int e = 0; e < 32; e += 16) {
    const uint32_t v = (w >> e) & 0x7fffu;
    if (v > 0x7f80u) w &= ~(0xffffu << e);
    else if (v == 0x7f80u) w -= 1u << e;
  }
  return w;
}
// Larger magnitudes of two pairs of bf16 values; NaN is the largest of all.
HBL_DEVINL uint32_t max_abs2(uint32_t m, uint32_t w) {
  const __nv_bfloat162 x = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&m),
                                       __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)));
  return *reinterpret_cast<const uint32_t*>(&x);
}

// The 8 codes of 8 bf16 values: code_of's first step for each, and its second only if any of them needs it.
HBL_DEVINL uint2 codes8(const uint4& x, float s, float inv, float h) {
  const float magic = 12583040.0f;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[8];
  bool close = false;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float v = __uint_as_float(k & 1 ? w[k >> 1] & 0xffff0000u : w[k >> 1] << 16);
    const float t = __fmaf_rn(v, inv, magic);
    close |= fabsf(__fmaf_rn(-__fsub_rn(t, magic), s, v)) >= h;
    c[k] = __float_as_uint(t);
  }
  if (close) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      c[k] = code_of(__uint_as_float(k & 1 ? w[k >> 1] & 0xffff0000u : w[k >> 1] << 16), s, inv, h);
  }
  return make_uint2(__byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410));
}

struct AppendArgs {
  const uint16_t *k, *v;              // keys, values
  long long kstride, vstride;         // elements from token to token
  uint8_t *kcodes, *vcodes;
  float *kscale, *vscale;
  const int32_t* slots;
  int T, H, page_log2, num_pages;
};

constexpr int kAppendThreads = 256;
constexpr int kAppendSpan = 128;      // most tokens of a block's span; its last run may go on for a page
// The tokens of one run, handled by `NT` threads (a warp or the block) of which this is number `tid`.
// `reduce` gives all of them the largest of their values. What fits in registers is read once.
template <int D, int NT, int HELD, typename Reduce>
HBL_DEVINL void append_run(const uint16_t* x, long long stride, int n, int off, int P, uint8_t* codes, float* scale, int tid,
                           Reduce reduce) {
  constexpr int VPT = D / 8;          // vectors of a token
  const int total = n * VPT;
  const float held = off > 0 ? *scale : 0.f;
  const float before = held >= 0.f && held < INFINITY ? held : 0.f;
  auto vec = [&](int i) { return __ldg(reinterpret_cast<const uint4*>(x + (size_t)(i / VPT) * (size_t)stride) + i % VPT); };
  uint4 v[HELD];
  uint32_t m = 0;
  {
    const uint16_t* p = x + (size_t)(tid / VPT) * (size_t)stride + 8 * (tid % VPT);
#pragma unroll
    for (int k = 0; k < HELD; ++k, p += (NT / VPT) * stride)
      v[k] = tid + k * NT < total ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int k = 0; k < HELD; ++k) m = max_abs2(max_abs2(max_abs2(max_abs2(m, v[k].x), v[k].y), v[k].z), v[k].w);
  for (int i = tid + HELD * NT; i < total; i += NT) {
    const uint4 w = vec(i);
    m = max_abs2(max_abs2(max_abs2(max_abs2(m, w.x), w.y), w.z), w.w);
  }
  uint32_t top = reduce(max(m & 0xffffu, m >> 16));
  const bool odd = top >= 0x7f80u;    // NaN or infinity among them: once more, with what is stored for those
  if (odd) {
    m = 0;
    for (int i = tid; i < total; i += NT) {
      const uint4 w = vec(i);
      m = max_abs2(max_abs2(max_abs2(max_abs2(m, finite2(w.x)), finite2(w.y)), finite2(w.z)), finite2(w.w));
    }
    top = reduce(max(m & 0xffffu, m >> 16));
#pragma unroll
    for (int k = 0; k < HELD; ++k)
      v[k] = make_uint4(finite2(v[k].x), finite2(v[k].y), finite2(v[k].z), finite2(v[k].w));
  }
  const float s = fmaxf(before, fmaxf(__fdiv_rn(__uint_as_float(top << 16), 127.f), kScaleFloor));
  const float inv = __frcp_rn(s), h = 0.5f * s;
  if (s != before) {                  // what the block held before the run
    for (int i = tid; i < off * (D / 4); i += NT) {
      const uint32_t w = reinterpret_cast<uint32_t*>(codes)[i];
      uint32_t c[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        c[k] = code_of(__fmul_rn((float)((int)((w >> (8 * k)) & 255u) - kZero), before), s, inv, h);
      reinterpret_cast<uint32_t*>(codes)[i] =
          __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    }
  }
  uint2* dst = reinterpret_cast<uint2*>(codes + (size_t)off * D);
#pragma unroll
  for (int k = 0; k < HELD; ++k)
    if (tid + k * NT < total) dst[tid + k * NT] = codes8(v[k], s, inv, h);
  for (int i = tid + HELD * NT; i < total; i += NT) {
    uint4 w = vec(i);
    if (odd) w = make_uint4(finite2(w.x), finite2(w.y), finite2(w.z), finite2(w.w));
    dst[i] = codes8(w, s, inv, h);
  }
  if (tid == 0) *scale = s;           // every thread has read it: it lies behind a reduction
}

// A run is a row of tokens in consecutive slots of one page. A block takes the runs that begin in its span of
// tokens, for one head's keys or values: a single long one with all its threads, several (or a short one) with a
// warp each. It finds the run's absmax, raises the block's scale to it if it must (rescaling the codes that the
// block held before the run), and writes the run's codes; the values are read once, for both. The bound is HBM, two bytes
// read and one written for each value: 8192 tokens, 32 heads of 128, pages of 64: 51 us, 3.9 TB/s (60 % of a copy;
// reading them twice, a warp to a run: 235 us); 16 single tokens: 3.0 us.
// HELD: 16-byte vectors that a thread holds, as many as a page gives it.
template <int D, int HELD>
__global__ void __launch_bounds__(kAppendThreads, 4) kv_append_kernel(const AppendArgs a, const int span) {
  constexpr int kWords = kAppendThreads / 32;
  __shared__ unsigned s_head[kWords], s_on[kWords];         // bit t: a run begins at token t0 + t; a run goes on there
  __shared__ int s_slot[kAppendThreads];
  __shared__ uint32_t s_max[2][kWords];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // heads first, then keys and values: blocks that run together read whole token rows
  const uint32_t unit = blockIdx.x / (uint32_t)a.H;
  const int h = (int)(blockIdx.x - unit * (uint32_t)a.H), P = 1 << a.page_log2, t0 = (int)(unit >> 1) * span;
  const bool keys = (unit & 1) == 0;
  const uint32_t slots = (uint32_t)a.num_pages << a.page_log2;
  {
    const int t = t0 + (int)threadIdx.x;
    const int now = t < a.T ? a.slots[t] : -1, last = t > 0 && t < a.T ? a.slots[t - 1] : -1;
    const bool valid = now >= 0 && (uint32_t)now < slots;
    const bool on = valid && (now & (P - 1)) != 0 && last == now - 1;
    if (now >= 0 && !valid) set_device_error(HBL_ERR_INVALID_ARG);
    s_slot[threadIdx.x] = now;
    const unsigned goes_on = __ballot_sync(0xffffffffu, on);
    const unsigned begins = __ballot_sync(0xffffffffu, valid && !on && (int)threadIdx.x < span);
    if (lane == 0) {
      s_head[warp] = begins;
      s_on[warp] = goes_on;
    }
  }
  __syncthreads();
  const unsigned heads = lane < kWords ? s_head[lane] : 0u, on = lane < kWords ? s_on[lane] : 0u;
  int upto = __popc(heads);           // runs that begin in this lane's word or before it
#pragma unroll
  for (int d = 1; d < kWords; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += y;
  }
  const int runs = __shfl_sync(0xffffffffu, upto, kWords - 1);
  if (runs == 0) return;
  const uint16_t* x = keys ? a.k : a.v;
  const long long stride = keys ? a.kstride : a.vstride;
  // Token, slot and length of the i-th run, by a whole warp: lane l looks at the tokens 32 l to 32 l + 31.
  auto run_at = [&](int i, int* slot, int* n) {
    const int word = __ffs(__ballot_sync(0xffffffffu, lane < kWords && upto > i)) - 1;
    unsigned bits = __shfl_sync(0xffffffffu, heads, word);
    for (int skip = i - (__shfl_sync(0xffffffffu, upto, word) - __popc(bits)); skip > 0; --skip) bits &= bits - 1;
    const int t = 32 * word + __ffs(bits) - 1;
    // the first token behind t where no run goes on
    unsigned stop = lane < kWords ? ~on : 0u;
    if (lane < word) stop = 0;
    else if (lane == word) stop &= ~(0xffffffffu >> (31 - (t & 31)));
    const int end = __reduce_min_sync(0xffffffffu, stop ? 32 * lane + __ffs(stop) - 1 : kAppendThreads);
    *slot = s_slot[t];
    *n = end - t;
    return t0 + t;
  };
  auto codes_at = [&](int slot) {
    return (keys ? a.kcodes : a.vcodes) + (((size_t)(slot >> a.page_log2) * a.H + h) << a.page_log2) * D;
  };
  auto scale_at = [&](int slot) { return (keys ? a.kscale : a.vscale) + (size_t)(slot >> a.page_log2) * a.H + h; };
  static_assert(kAppendThreads >= kAppendSpan + 128, "the last run of a span ends within the tokens looked at");
  int slot, n;
  if (runs == 1) {
    const int t = run_at(0, &slot, &n);
    if (n * (D / 8) > 4 * 32) {
      int pass = 0;
      append_run<D, kAppendThreads, HELD>(x + (size_t)t * (size_t)stride + (size_t)h * D, stride, n, slot & (P - 1), P,
                                          codes_at(slot), scale_at(slot), threadIdx.x, [&](uint32_t m) {
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) s_max[pass][warp] = m;
        __syncthreads();
        m = __reduce_max_sync(0xffffffffu, lane < kWords ? s_max[pass][lane] : 0u);
        pass ^= 1;
        return m;
      });
      return;
    }
  }
  for (int i = warp; i < runs; i += kWords) {
    const int t = run_at(i, &slot, &n);
    append_run<D, 32, HELD>(x + (size_t)t * (size_t)stride + (size_t)h * D, stride, n, slot & (P - 1), P, codes_at(slot),
                            scale_at(slot), lane, [&](uint32_t m) { return __reduce_max_sync(0xffffffffu, m); });
  }
}

// ---------------------------------------------------------------------------
// Reading back.
// ---------------------------------------------------------------------------
struct ReadArgs {
  const uint8_t *kcodes, *vcodes;
  const float *kscale, *vscale;
  uint16_t *k, *v;                    // T x H x D; either may be null
  const int32_t* slots;
  int T, H, page_log2, num_pages;
};

constexpr int kReadItems = 4;         // vectors of 8 values of a thread

// bf16((u - 128) * s), the product rounded to fp32 first. A thread's four 8-byte loads of codes are all
// issued before the first is used. Bound by HBM: 8192 tokens, 32 heads of 128: 33.9 us, 5.9 TB/s.
template <int D>
__global__ void __launch_bounds__(256) kv_read_kernel(const ReadArgs a) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const bool keys = blockIdx.y == 0;
  uint16_t* out = keys ? a.k : a.v;
  if (!out) return;
  const uint8_t* codes = keys ? a.kcodes : a.vcodes;
  const float* scale = keys ? a.kscale : a.vscale;
  const uint32_t rows = (uint32_t)a.T * (uint32_t)a.H;
  const uint32_t slots = (uint32_t)a.num_pages << a.page_log2, pmask = (1u << a.page_log2) - 1u;
  const uint32_t row0 = (uint32_t)(blockIdx.x * (size_t)(256 * kReadItems / (D / 8))) + threadIdx.x / (D / 8);
  const int c = 8 * (int)(threadIdx.x % (D / 8));
  uint2 w[kReadItems];
  float s[kReadItems];
#pragma unroll
  for (int i = 0; i < kReadItems; ++i) {
    const uint32_t row = row0 + (uint32_t)(i * (256 / (D / 8)));
    w[i] = make_uint2(0, 0);
    s[i] = 0.f;
    if (row < rows) {
      const uint32_t t = row / (uint32_t)a.H, h = row - t * (uint32_t)a.H;
      const int slot = a.slots[t];
      if (slot >= 0 && (uint32_t)slot >= slots) {
        set_device_error(HBL_ERR_INVALID_ARG);
      } else if (slot >= 0) {
        const size_t block = (size_t)((uint32_t)slot >> a.page_log2) * a.H + h;
        w[i] = __ldg(reinterpret_cast<const uint2*>(codes + ((block << a.page_log2) + ((uint32_t)slot & pmask)) * D + c));
        s[i] = __ldg(scale + block);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kReadItems; ++i) {
    const uint32_t row = row0 + (uint32_t)(i * (256 / (D / 8)));
    if (row >= rows) break;
    uint32_t r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // a byte in the low bits of 2^23, minus 2^23 + 128: the value of the code, exactly
      const uint32_t u = k < 2 ? w[i].x : w[i].y;
      const float lo = __uint_as_float(__byte_perm(u, 0x4b000000u, k & 1 ? 0x7552 : 0x7550)) - 8388736.0f;
      const float hi = __uint_as_float(__byte_perm(u, 0x4b000000u, k & 1 ? 0x7553 : 0x7551)) - 8388736.0f;
      const __nv_bfloat162 p = __floats2bfloat162_rn(__fmul_rn(lo, s[i]), __fmul_rn(hi, s[i]));
      r[k] = *reinterpret_cast<const uint32_t*>(&p);
    }
    *reinterpret_cast<uint4*>(out + (size_t)row * D + c) = make_uint4(r[0], r[1], r[2], r[3]);
  }
}

}  // namespace kv
}  // namespace hbl
