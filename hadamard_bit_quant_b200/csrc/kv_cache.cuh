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
constexpr int kPlanThreads = 1024;

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
// new tokens, pages wanted, pages given back. With those three sums in shared memory, each slot, each
// new table entry and each page returned to the stack is found by itself with a binary search.
__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(PlanArgs a) {
  extern __shared__ int sm[];
  int* cu = sm;                       // [B + 1] first row of each request
  int* want = cu + a.B + 1;           // [B + 1] pages taken by the requests before this one
  int* gone = want + a.B + 1;         // [B + 1] pages given back by the requests before this one
  __shared__ long long sh[33];
  __shared__ int s_used;
  const int P = 1 << a.page_log2, lg = a.page_log2;
  const long long cap = (long long)a.max_pages << lg;
  const int per = (a.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
  if (threadIdx.x == 0) s_used = 0;

  auto len_of = [&](int b) { return min(max((long long)a.kv_lens[b], 0ll), cap); };
  auto pages = [&](long long n) { return (n + P - 1) >> lg; };

  // rows of new tokens
  long long sum = 0, total;
  for (int b = b0; b < b1; ++b) sum += max(a.new_lens[b], 0);
  long long x = block_scan(sum, sh, &total);
  for (int b = b0; b < b1; ++b) {
    cu[b] = (int)min(x, (long long)a.T);
    x += max(a.new_lens[b], 0);
  }
  if (threadIdx.x == 0) cu[a.B] = (int)min(total, (long long)a.T);
  __syncthreads();

  // pages wanted and given back; a request that cannot grow wants none
  long long need = 0, back = 0;
  for (int b = b0; b < b1; ++b) {
    const long long n = len_of(b), q = a.new_lens[b], after = max(n + q, 0ll);
    if (q > 0 && (after > cap || cu[b + 1] - cu[b] < q)) continue;
    need += max(pages(after) - pages(n), 0ll);
    back += max(pages(n) - pages(after), 0ll);
  }
  long long need_all, back_all;
  const long long need0 = block_scan(need, sh, &need_all), back0 = block_scan(back, sh, &back_all);
  const int F = min(max(*a.free_count, 0), a.num_pages);
  const long long stock = F + back_all;
  {
    long long nd = need0, bk = back0;
    for (int b = b0; b < b1; ++b) {
      const long long n = len_of(b), q = a.new_lens[b], after = max(n + q, 0ll);
      const bool wide = q > 0 && (after > cap || cu[b + 1] - cu[b] < q);
      const long long take = wide ? 0 : max(pages(after) - pages(n), 0ll);
      want[b] = (int)min(nd, 0x7fffffffll);
      gone[b] = (int)min(bk, 0x7fffffffll);
      const bool ok = !wide && (take == 0 || nd + take <= stock);
      if (ok && take) atomicMax(&s_used, (int)(nd + take));
      a.refused[b] = ok ? 0 : 1;
      nd += take;
      if (!wide) bk += max(pages(n) - pages(after), 0ll);
    }
  }
  if (threadIdx.x == 0) {
    want[a.B] = (int)min(need_all, 0x7fffffffll);
    gone[a.B] = (int)min(back_all, 0x7fffffffll);
  }
  __syncthreads();
  const int used = s_used, R = gone[a.B];

  // i-th page given back in this step, and i-th page handed out: those given back first, then the stack from its top
  auto released = [&](int i) {
    const int b = find_row(gone, a.B, i);
    const long long after = max(len_of(b) + a.new_lens[b], 0ll);
    return a.table[(size_t)b * a.max_pages + (size_t)(pages(after) + (i - gone[b]))];
  };
  auto handed = [&](int i) { return i < R ? released(i) : a.free_pages[F - 1 - (i - R)]; };

  for (int t = threadIdx.x; t < a.T; t += kPlanThreads) {
    int slot = -1;
    if (t < cu[a.B]) {
      const int b = find_row(cu, a.B, t);
      if (a.refused[b] == 0) {
        const long long n = len_of(b), pos = n + (t - cu[b]);
        const int pi = (int)(pos >> lg), held = (int)pages(n);
        const int id = pi < held ? a.table[(size_t)b * a.max_pages + pi] : handed(want[b] + pi - held);
        if (id >= 0 && id < a.num_pages) slot = (id << lg) + (int)(pos & (P - 1));
        else set_device_error(HBL_ERR_INVALID_ARG);
      }
    }
    a.slots[t] = slot;
  }
  for (int i = threadIdx.x; i < used; i += kPlanThreads) {
    const int b = find_row(want, a.B, i);
    a.table[(size_t)b * a.max_pages + (size_t)(pages(len_of(b)) + (i - want[b]))] = handed(i);
  }
  // what was given back and not handed out again: the last of it lies deepest, so a step that is undone
  // leaves the stack as it was
  for (int i = used + threadIdx.x; i < R; i += kPlanThreads) {
    const int at = F + (R - 1 - i);
    if (at < a.num_pages) a.free_pages[at] = released(i);
    else set_device_error(HBL_ERR_INVALID_ARG);
  }
  for (int b = threadIdx.x; b <= a.B; b += kPlanThreads) a.cu_q[b] = cu[b];
  __syncthreads();
  for (int b = b0; b < b1; ++b) {
    const long long n = len_of(b);
    a.kv_lens[b] = (int)(a.refused[b] ? n : max(n + a.new_lens[b], 0ll));
  }
  if (threadIdx.x == 0) *a.free_count = (int)min(stock - used, (long long)a.num_pages);
}

// ---------------------------------------------------------------------------
// Appending.
// ---------------------------------------------------------------------------

// rint(x / s), ties to even, of the exact quotient. r = rint(x * (1/s)) is within one of it; the remainder
// x - r s is exact in fp32 (it is a multiple of half an ulp of s and not larger than s), so comparing it
// with s / 2 decides.
HBL_DEVINL float quotient(float x, float s, float inv) {
  float r = rintf(__fmul_rn(x, inv));
  const float d = __fmaf_rn(-r, s, x), h = 0.5f * s;
  const bool odd = ((int)r) & 1;
  if (fabsf(d) > h || (fabsf(d) == h && odd)) r += copysignf(1.f, d);
  return r;
}

// A bf16 value as the cache takes it: there is no code for NaN (0 is stored) or infinity (the largest
// finite value is stored).
HBL_DEVINL float finite(float x) {
  const float big = __uint_as_float(0x7f7f0000u);   // largest finite bf16
  return x != x ? 0.f : fminf(fmaxf(x, -big), big);
}
HBL_DEVINL float lo_bf16(uint32_t w) { return finite(__uint_as_float(w << 16)); }
HBL_DEVINL float hi_bf16(uint32_t w) { return finite(__uint_as_float(w & 0xffff0000u)); }

struct AppendArgs {
  const uint16_t* x[2];               // keys, values
  long long stride[2];                // elements from token to token
  uint8_t* codes[2];
  float* scale[2];
  const int32_t* slots;
  int T, H, page_log2, num_pages;
};

// One warp for each (first token of a run, head, keys or values). A run is a row of tokens in consecutive
// slots of one page: the warp finds the run's absmax, raises the block's scale to it if it must (rescaling
// the codes that the block held before the run), and writes the run's codes.
template <int D>
__global__ void __launch_bounds__(256) kv_append_kernel(AppendArgs a) {
  constexpr int LPT = D / 8;          // lanes of a token, 8 values each
  constexpr int TPW = 32 / LPT;       // tokens side by side in a warp
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int lane = threadIdx.x & 31, h = blockIdx.y, kind = blockIdx.z;
  const int t0 = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t0 >= a.T) return;
  const int P = 1 << a.page_log2;
  const int slot = a.slots[t0];
  if (slot < 0) return;
  if (slot >= (a.num_pages << a.page_log2)) {
    if (lane == 0) set_device_error(HBL_ERR_INVALID_ARG);
    return;
  }
  const int off = slot & (P - 1);
  if (t0 > 0 && off > 0 && a.slots[t0 - 1] == slot - 1) return;   // not the first of its run
  int n = 1;
  while (true) {
    const int m = n + lane;
    const bool in = off + m < P && t0 + m < a.T && a.slots[t0 + m] == slot + m;
    const unsigned out = ~__ballot_sync(0xffffffffu, in);
    if (out) { n += __ffs(out) - 1; break; }
    n += 32;
  }
  const uint16_t* x = a.x[kind] + (size_t)t0 * (size_t)a.stride[kind] + (size_t)h * D + 8 * (lane % LPT);
  float gamma = 0.f;
  for (int i = lane / LPT; i < n; i += TPW) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(x + (size_t)i * (size_t)a.stride[kind]));
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) gamma = fmaxf(gamma, fmaxf(fabsf(lo_bf16(ws[k])), fabsf(hi_bf16(ws[k]))));
  }
  gamma = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(gamma)));
  const size_t block = (size_t)(slot >> a.page_log2) * a.H + h;
  uint8_t* codes = a.codes[kind] + block * (size_t)P * D;
  float before = off > 0 ? a.scale[kind][block] : 0.f;
  if (!(before >= 0.f && before <= 3.4e38f)) before = 0.f;
  const float s = fmaxf(before, fmaxf(__fdiv_rn(gamma, 127.f), kScaleFloor));
  const float inv = __frcp_rn(s);
  if (off > 0 && s != before) {
    for (int i = lane; i < off * (D / 4); i += 32) {
      uint32_t w = reinterpret_cast<uint32_t*>(codes)[i], o = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float v = __fmul_rn((float)((int)((w >> (8 * k)) & 255u) - kZero), before);
        o |= (uint32_t)((int)quotient(v, s, inv) + kZero) << (8 * k);
      }
      reinterpret_cast<uint32_t*>(codes)[i] = o;
    }
  }
  for (int i = lane / LPT; i < n; i += TPW) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(x + (size_t)i * (size_t)a.stride[kind]));
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    uint32_t o[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t c0 = (uint32_t)((int)quotient(lo_bf16(ws[k]), s, inv) + kZero);
      const uint32_t c1 = (uint32_t)((int)quotient(hi_bf16(ws[k]), s, inv) + kZero);
      o[k >> 1] |= (c0 | (c1 << 8)) << (16 * (k & 1));
    }
    *reinterpret_cast<uint2*>(codes + (size_t)(off + i) * D + 8 * (lane % LPT)) = make_uint2(o[0], o[1]);
  }
  __syncwarp();
  if (lane == 0) a.scale[kind][block] = s;
}

// ---------------------------------------------------------------------------
// Reading back.
// ---------------------------------------------------------------------------
struct ReadArgs {
  const uint8_t* codes[2];
  const float* scale[2];
  uint16_t* out[2];                   // T x H x D; either may be null
  const int32_t* slots;
  int T, H, page_log2, num_pages;
};

// Eight values a thread: one 8-byte load of codes, one 16-byte store. bf16((u - 128) * s), the product
// rounded to fp32 first.
template <int D>
__global__ void __launch_bounds__(256) kv_read_kernel(ReadArgs a) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int kind = blockIdx.y;
  if (!a.out[kind]) return;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long row = i / (D / 8);
  if (row >= (long long)a.T * a.H) return;
  const int t = (int)(row / a.H), h = (int)(row % a.H), c = (int)(i % (D / 8)) * 8;
  const int slot = a.slots[t];
  uint4 o = make_uint4(0, 0, 0, 0);
  if (slot >= (a.num_pages << a.page_log2)) {
    set_device_error(HBL_ERR_INVALID_ARG);
  } else if (slot >= 0) {
    const size_t block = (size_t)(slot >> a.page_log2) * a.H + h;
    const int off = slot & ((1 << a.page_log2) - 1);
    const uint2 w = *reinterpret_cast<const uint2*>(a.codes[kind] + ((block << a.page_log2) + off) * D + c);
    const float s = a.scale[kind][block];
    uint32_t r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t v = (k < 2 ? w.x : w.y) >> (16 * (k & 1));
      const float lo = __fmul_rn((float)((int)(v & 255u) - kZero), s);
      const float hi = __fmul_rn((float)((int)((v >> 8) & 255u) - kZero), s);
      r[k] = (uint32_t)float_to_bf16_bits(lo) | ((uint32_t)float_to_bf16_bits(hi) << 16);
    }
    o = make_uint4(r[0], r[1], r[2], r[3]);
  }
  *reinterpret_cast<uint4*>(a.out[kind] + row * D + c) = o;
}

}  // namespace kv
}  // namespace hbl
