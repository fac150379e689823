// Host side of the paged 8-bit key/value cache: argument checks, workspace layout and launches. Included by
// hbl_api.cu after its own helpers.
#pragma once
#include <algorithm>
#include <cmath>
#include "kv_cache.cuh"
#include "kv_attn.cuh"
#include "kv_prefill.cuh"

namespace hbl {
namespace {

inline bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// Pages of 16, 32, 64 or 128 tokens; slot numbers stay in an int32.
int check_pages(int page, int num_pages) {
  if (page != 16 && page != 32 && page != 64 && page != 128) return HBL_ERR_SHAPE;
  if (num_pages < 1 || (long long)num_pages * page >= (1ll << 31)) return HBL_ERR_SHAPE;
  return HBL_OK;
}

int check_heads(int T, int H, int D) {
  if (T < 0 || H < 1 || H > 65535 || (D != 64 && D != 128)) return HBL_ERR_SHAPE;
  if ((long long)T * H >= (1ll << 31)) return HBL_ERR_SHAPE;
  return HBL_OK;
}

int check_table(int B, int max_pages, int page) {
  if (B < 0 || B > kv::kMaxRequests || max_pages < 1 || (long long)B * max_pages >= (1ll << 31)) return HBL_ERR_SHAPE;
  return (long long)max_pages * page > (1ll << 30) ? HBL_ERR_SHAPE : HBL_OK;
}

struct KvWs {
  size_t prefix, mz, o, total;
};

KvWs kv_ws_layout(int B, int D) {
  KvWs L;
  size_t off = 0;
  const size_t rows = (size_t)kv::kMaxAttnCtas * 2 * kv::kAttnRows;
  L.prefix = off; off = align_up(off + ((size_t)B + 1) * 8, 256);
  L.mz = off; off = align_up(off + rows * 8, 256);
  L.o = off; off = align_up(off + rows * D * 4, 256);
  L.total = off;
  return L;
}

// Rows per key/value head up to which a request is streamed by kv_attn_kernel, two tiles of 16 that both read the
// cache; more go to the tensor-core kernel, which reads it once for 256 rows but gives a request's head to one CTA.
constexpr int kFewRows = 32;

// Rows of all query heads together up to which that holds for every request. Measured for one request, tensor-core kernel / this
// one, us: 8 rows of 64 heads on 8 over 131072 keys (512 in all): 1720 / 244; 64 rows of 32 on 8 over 32768 (2048): 616 / 238; 512
// rows of 8 on 2 over 8192 (4096): 162 / 126; 192 rows of 32 on 8 over 4096 (6144): 89 / 107; 1024 rows of 8 on 2 over 1024
// (8192): 34 / 53; 2048 rows of 4 on 1 over 2048 (8192): 52 / 76.
constexpr int kFewInAll = 6144;

// Most cached tokens of a request, and most CTAs, for which kv_attn_kernel leaves each item to one CTA: one request of 130
// tokens, 32 heads of 128, takes 4.4 us so and 8.1 us with the parts joined by a second kernel.
constexpr int kWholeKeys = 512, kWholeCtas = 4096;

// Three kernels, each of which takes the requests that are its own: which those are is known on the GPU only.
// The host leaves out what its bound on the rows rules out.
template <int D>
int launch_kv_attention(const kv::AttnArgs& a, cudaStream_t s) {
  if (a.most_rows > a.few_rows) {
    // every request wastes less than one tile of rows
    const long long rows = (long long)a.T * a.group;
    const long long items = rows / kv::kPreRows + std::min<long long>(a.B, rows / (a.few_rows + 1));
    if (items > 0) {
      const size_t smem = sizeof(kv::PreSmem<D>) + 1024;
      ensure_smem_attr(kv::kv_prefill_kernel<D>, smem);
      ProfScope ps("kv_prefill", s);
      launch_pdl(kv::kv_prefill_kernel<D>, dim3((unsigned)(items * a.Hkv)), dim3(kv::kPreThreads), smem, s, a);
    }
  }
  {
    auto kernel = a.tile_rows == 8 ? kv::kv_attn_kernel<D, 1> : kv::kv_attn_kernel<D, 2>;
    ensure_smem_attr(kernel, kv::AttnCfg<D>::kSmem);
    ProfScope ps("kv_attn", s);
    launch_pdl(kernel, dim3(a.ctas), dim3(kv::AttnCfg<D>::kWarps * 32), kv::AttnCfg<D>::kSmem, s, a);
  }
  if (a.row_tiles == 0) {
    ProfScope ps("kv_combine", s);
    // few rows have many parts, many rows have few
    const long long by_request = (long long)a.B * a.Hkv * a.few_rows, by_token = (long long)a.T * a.Hq;
    const int rows = by_request <= by_token ? a.few_rows : 0;
    const long long all = std::min(by_request, by_token);
    if (all <= 256) launch_pdl(kv::kv_combine_kernel<D, 8>, dim3((unsigned)all), dim3(256), 0, s, a, rows);
    else if (all <= 1024) launch_pdl(kv::kv_combine_kernel<D, 2>, dim3((unsigned)((all + 3) / 4)), dim3(256), 0, s, a, rows);
    else launch_pdl(kv::kv_combine_kernel<D, 1>, dim3((unsigned)((all + 7) / 8)), dim3(256), 0, s, a, rows);
  }
  return launch_status();
}

}  // namespace
}  // namespace hbl

extern "C" {

int hbl_kv_plan(const int32_t* new_lens, int B, int page, int num_pages, int max_pages, int T, int32_t* kv_lens,
                int32_t* block_table, int32_t* free_pages, int32_t* free_count, int32_t* cu_q, int32_t* slots,
                int32_t* refused, hbl_stream stream) {
  int st = check_pages(page, num_pages);
  if (st) return st;
  if (T < 0 || (st = check_table(B, max_pages, page))) return HBL_ERR_SHAPE;
  if (B == 0) return HBL_OK;
  if (!new_lens || !kv_lens || !block_table || !free_pages || !free_count || !cu_q || !refused || (T > 0 && !slots))
    return HBL_ERR_INVALID_ARG;
  for (const void* p : {(const void*)new_lens, (const void*)kv_lens, (const void*)block_table,
                        (const void*)free_pages, (const void*)free_count, (const void*)cu_q, (const void*)slots,
                        (const void*)refused})
    if (misaligned(p, 4)) return HBL_ERR_INVALID_ARG;
  DeviceState* d = nullptr;
  if ((st = ensure_device(&d))) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const kv::PlanArgs a{new_lens, kv_lens, block_table, free_pages, free_count, cu_q, slots, refused,
                       B, ilog2(page), num_pages, max_pages, T};
  const size_t smem = 4 * ((size_t)B + 1) * 4;
  // for the largest batch whatever this one is: the kernel's static arrays count too, so the limit is short of 48 KB
  ensure_smem_attr(kv::kv_plan_kernel, 4 * ((size_t)kv::kMaxRequests + 1) * 4);
  // a thread for each request or row up to a block's 1024; beyond that a cluster of blocks shares the rows
  const int most = std::max(B, T), threads = most <= 128 ? 128 : most <= 512 ? 512 : kv::kPlanThreads;
  const int ctas = T > 2 * kv::kPlanThreads ? kv::kPlanCtas : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  ProfScope ps("kv_plan", s);
  if (cudaLaunchKernelEx(&cfg, kv::kv_plan_kernel, a) != cudaSuccess) {
    cudaGetLastError();
    return HBL_ERR_CUDA;
  }
  return launch_status();
}

int hbl_kv_append(const hbl_bf16* K, const hbl_bf16* V, int T, int Hkv, int D, long long k_stride,
                  long long v_stride, const int32_t* slots, int page, int num_pages, uint8_t* kcodes,
                  uint8_t* vcodes, float* kscale, float* vscale, hbl_stream stream) {
  int st = check_pages(page, num_pages);
  if (st || (st = check_heads(T, Hkv, D))) return st;
  if (T == 0) return HBL_OK;
  if (k_stride < (long long)Hkv * D || v_stride < (long long)Hkv * D || k_stride % 8 || v_stride % 8)
    return HBL_ERR_SHAPE;
  if (!K || !V || !slots || !kcodes || !vcodes || !kscale || !vscale) return HBL_ERR_INVALID_ARG;
  if (misaligned16(K) || misaligned16(V) || misaligned16(kcodes) || misaligned16(vcodes)) return HBL_ERR_INVALID_ARG;
  if (misaligned(slots, 4) || misaligned(kscale, 4) || misaligned(vscale, 4)) return HBL_ERR_INVALID_ARG;
  DeviceState* d = nullptr;
  if ((st = ensure_device(&d))) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const kv::AppendArgs a{K, V, k_stride, v_stride, kcodes, vcodes, kscale, vscale, slots, T, Hkv, ilog2(page), num_pages};
  // Spans of a page (64 tokens at least) when there are many tokens, so that a run fills a block; shorter ones, down to a
  // token for each warp, until the grid has four blocks for each SM. Measured for other multiples (us, at 1 / 4 / 16): 8
  // requests of 512 tokens, 8 heads of 128, pages of 128: 19.5 / 8.7 / 12.8; 7 of 300, 8 heads of 64, pages of 64: 5.3 /
  // 5.1 / 8.8; 256 single tokens, 32 heads of 128: 16.5 / 11.3 / 11.9.
  int span = std::max(page, 64);
  while (span > 8 && (long long)((T + span - 1) / span) * Hkv * 2 < 4ll * d->sm_count) span /= 2;
  const long long blocks = (long long)((T + span - 1) / span) * Hkv * 2;
  if (blocks >= (1ll << 31)) return HBL_ERR_SHAPE;
  const dim3 grid((unsigned)blocks);
  ProfScope ps("kv_append", s);
  // what a run of a page holds for each thread: of a block, or of a warp where a page is a short run (16 tokens)
  const bool many = page * D > 8192 || page * D == 16 * 128;
  auto kernel = D == 64 ? (many ? kv::kv_append_kernel<64, 8> : kv::kv_append_kernel<64, 4>)
                        : (many ? kv::kv_append_kernel<128, 8> : kv::kv_append_kernel<128, 4>);
  launch_pdl(kernel, grid, dim3(kv::kAppendThreads), 0, s, a, span);
  return launch_status();
}

int hbl_kv_read(const int32_t* slots, int T, int Hkv, int D, int page, int num_pages, const uint8_t* kcodes,
                const uint8_t* vcodes, const float* kscale, const float* vscale, hbl_bf16* K, hbl_bf16* V,
                hbl_stream stream) {
  int st = check_pages(page, num_pages);
  if (st || (st = check_heads(T, Hkv, D))) return st;
  if (T == 0 || (!K && !V)) return HBL_OK;
  if (!slots || (K && (!kcodes || !kscale)) || (V && (!vcodes || !vscale))) return HBL_ERR_INVALID_ARG;
  if (misaligned16(K) || misaligned16(V) || misaligned16(kcodes) || misaligned16(vcodes)) return HBL_ERR_INVALID_ARG;
  if (misaligned(slots, 4) || misaligned(kscale, 4) || misaligned(vscale, 4)) return HBL_ERR_INVALID_ARG;
  DeviceState* d = nullptr;
  if ((st = ensure_device(&d))) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const kv::ReadArgs a{kcodes, vcodes, kscale, vscale, K, V, slots, T, Hkv, ilog2(page), num_pages};
  const long long vectors = (long long)T * Hkv * (D / 8), per = 256 * kv::kReadItems;
  const dim3 grid((unsigned)((vectors + per - 1) / per), 2);
  ProfScope ps("kv_read", s);
  if (D == 64) launch_pdl(kv::kv_read_kernel<64>, grid, dim3(256), 0, s, a);
  else launch_pdl(kv::kv_read_kernel<128>, grid, dim3(256), 0, s, a);
  return launch_status();
}

size_t hbl_kv_attention_workspace_bytes(int B, int D) {
  if (B < 0 || (D != 64 && D != 128)) return 0;
  return kv_ws_layout(B, D).total;
}

int hbl_kv_attention(const hbl_bf16* Q, int T, int Hq, int Hkv, int D, long long q_stride, const int32_t* cu_q,
                     const int32_t* kv_lens, int B, int max_q, int max_kv, const int32_t* block_table,
                     int max_pages, int page, int num_pages, const uint8_t* kcodes, const uint8_t* vcodes,
                     const float* kscale, const float* vscale, float scale, int causal, int window, hbl_bf16* O,
                     float* lse, void* ws, size_t ws_bytes, hbl_stream stream) {
  int st = check_pages(page, num_pages);
  if (st || (st = check_heads(T, Hq, D)) || (st = check_heads(T, Hkv, D))) return st;
  if (Hq % Hkv != 0 || q_stride < (long long)Hq * D || q_stride % 8) return HBL_ERR_SHAPE;
  // positions, rows and windows (cut to the table's reach below) then add up within an int
  if ((long long)T * Hq >= (1ll << 30) || (st = check_table(B, max_pages, page))) return HBL_ERR_SHAPE;
  if (max_q < 0 || max_kv < 0) return HBL_ERR_SHAPE;
  if ((causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal)) return HBL_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale * kv::kLog2e)) return HBL_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return HBL_OK;
  if (!Q || !cu_q || !kv_lens || !block_table || !kcodes || !vcodes || !kscale || !vscale || !O)
    return HBL_ERR_INVALID_ARG;
  if (misaligned16(Q) || misaligned16(kcodes) || misaligned16(vcodes) || misaligned16(O)) return HBL_ERR_INVALID_ARG;
  for (const void* p : {(const void*)cu_q, (const void*)kv_lens, (const void*)block_table, (const void*)kscale,
                        (const void*)vscale, (const void*)lse})
    if (misaligned(p, 4)) return HBL_ERR_INVALID_ARG;
  const KvWs L = kv_ws_layout(B, D);
  if (!ws || ws_bytes < L.total) return HBL_ERR_WORKSPACE;
  if (misaligned(ws, 256)) return HBL_ERR_INVALID_ARG;
  DeviceState* d = nullptr;
  if ((st = ensure_device(&d))) return st;
  uint8_t* w = static_cast<uint8_t*>(ws);
  const int most_q = max_q > 0 && max_q < T ? max_q : T;    // no request has more than all: rows of a head then stay below 2^30
  kv::AttnArgs a{Q, q_stride, cu_q, kv_lens, block_table, kcodes, vcodes, kscale, vscale, O, lse,
                       reinterpret_cast<long long*>(w + L.prefix), reinterpret_cast<float*>(w + L.mz),
                       reinterpret_cast<float*>(w + L.o), scale * kv::kLog2e, T, Hq, Hkv, Hq / Hkv, B, max_pages,
                       ilog2(page), num_pages, causal, window < max_pages * page ? window : 0,
                       std::min((D == 64 ? kv::AttnCfg<64>::kCtas : kv::AttnCfg<128>::kCtas) * d->sm_count, kv::kMaxAttnCtas), std::max(kFewRows, Hq / Hkv),
                       most_q * (Hq / Hkv), 0, 0, 0, 0};
  // The tensor-core kernel gives 256 rows of a head to one CTA for the whole length of their keys: with few such items most
  // of the GPU would wait for them, and kv_attn_kernel, which splits the keys, takes every row.
  if ((long long)T * Hq <= kFewInAll) a.few_rows = a.most_rows;
  a.few_rows = std::min(a.few_rows, a.most_rows);           // a request beyond the caller's bound is nobody's
  a.group_shift = ilog2(a.group);
  a.group_mul = (uint32_t)((((1ull << a.group_shift) - (uint64_t)a.group) << 32) / (uint64_t)a.group + 1);
  a.tile_rows = a.few_rows <= 8 ? 8 : 16;
  // Few enough keys for one CTA to be through with them before a second kernel could have joined the parts: each item
  // is left whole (at most kWholeCtas of them, so that the grid stays a few waves).
  const long long most_kv = std::min<long long>(max_kv ? max_kv : 1ll << 40, (long long)max_pages * page);
  const int row_tiles = (a.few_rows + a.tile_rows - 1) / a.tile_rows;
  if (most_kv <= kWholeKeys && (long long)B * Hkv * row_tiles <= kWholeCtas) {
    a.row_tiles = row_tiles;
    a.ctas = B * Hkv * row_tiles;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return D == 64 ? launch_kv_attention<64>(a, s) : launch_kv_attention<128>(a, s);
}

}  // extern "C"
