// C ABI of the attention step around the linears: rotary positions, the paged FP8
// key / value cache (append, attention) and low-rank adapters. Argument checks and the
// construction-time objects; nothing here touches the device except through the launches.
#include <math.h>
#include <stdlib.h>

#include "internal.h"

using namespace fp8w8a8;

struct fp8_rope_plan {
  int head_dim;
  int interleaved;
  RopeTable table;
};

struct fp8_kv_cache {
  int device;
  int cu_count;
  KvCache c;
};

struct fp8_lora_plan {
  int device;
  int cu_count;
  LoraWeights w;
};

namespace {

constexpr int64_t kMaxGridThreads = (int64_t)1 << 32;
constexpr int64_t kMaxHeads = 65535;      // a grid dimension
constexpr int64_t kMaxRequests = FP8W8A8_MAX_REQUESTS;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A [tokens, heads, head_dim] view: every row of a head 16-byte aligned.
int check_rows(const fp8_rows* r) {
  if (!r || !r->data) return FP8W8A8_ERR_INVALID_ARG;
  if (r->heads < 1 || r->heads > kMaxHeads) return FP8W8A8_ERR_BAD_SHAPE;
  if (!aligned(r->data, 16) || r->token_stride % 8 != 0 || r->head_stride % 8 != 0) return FP8W8A8_ERR_MISALIGNED;
  return FP8W8A8_OK;
}

// An output's rows must not lie on each other.
int check_rows_out(const fp8_rows* r, const fp8_rows* in, int64_t head_dim) {
  const int st = check_rows(r);
  if (st != FP8W8A8_OK) return st;
  if (r->heads != in->heads) return FP8W8A8_ERR_BAD_SHAPE;
  if (r->token_stride < head_dim || (r->heads > 1 && r->head_stride < head_dim)) return FP8W8A8_ERR_BAD_SHAPE;
  return FP8W8A8_OK;
}

int check_batch(int64_t requests, int64_t tokens) {
  if (requests < 0 || requests > kMaxRequests) return FP8W8A8_ERR_BAD_SHAPE;
  if (tokens < 0 || tokens >= FP8W8A8_MAX_ROWS) return FP8W8A8_ERR_BAD_SHAPE;
  return FP8W8A8_OK;
}

bool table_fits(const KvCache& c, int64_t table_pages) {
  return table_pages >= 1 && table_pages <= FP8W8A8_MAX_PLACES / c.page_tokens;
}

// The ragged batch of a cache call: request lengths, row offsets and the page table.
int check_paged(const KvCache& c, int64_t requests, int64_t tokens, const int32_t* table, int64_t table_pages,
                const int32_t* lengths, const int32_t* starts) {
  if (!table || !lengths || !starts) return FP8W8A8_ERR_INVALID_ARG;
  const int st = check_batch(requests, tokens);
  if (st != FP8W8A8_OK) return st;
  if (!table_fits(c, table_pages)) return FP8W8A8_ERR_BAD_SHAPE;
  if (!aligned(table, 4) || !aligned(lengths, 4) || !aligned(starts, 4)) return FP8W8A8_ERR_MISALIGNED;
  return FP8W8A8_OK;
}

RopeTensor rope_tensor(const fp8_rows* x, const fp8_rows* y) {
  if (!x) return RopeTensor{nullptr, nullptr, 0, 0, 0, 0, 0};
  return RopeTensor{static_cast<const uint16_t*>(x->data), static_cast<uint16_t*>(y->data), x->token_stride,
                    x->head_stride, y->token_stride, y->head_stride, (int)x->heads};
}

RowsIn rows_in(const fp8_rows* x) {
  return RowsIn{static_cast<const uint16_t*>(x->data), x->token_stride, x->head_stride};
}

}  // namespace

extern "C" {

int fp8_rope_create(int64_t head_dim, int axes, const int64_t* widths, double base, int layout, fp8_rope_plan** out) {
  if (!out || !widths) return FP8W8A8_ERR_INVALID_ARG;
  if (layout != FP8W8A8_ROPE_INTERLEAVED && layout != FP8W8A8_ROPE_HALVES) return FP8W8A8_ERR_INVALID_ARG;
  if (!(base > 1.0) || !isfinite(base)) return FP8W8A8_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return FP8W8A8_ERR_BAD_SHAPE;
  if (axes < 1 || axes > FP8W8A8_MAX_AXES) return FP8W8A8_ERR_BAD_SHAPE;
  int64_t columns = 0;
  for (int i = 0; i < axes; ++i) {
    if (widths[i] < 2 || widths[i] % 2 != 0 || widths[i] > head_dim - columns) return FP8W8A8_ERR_BAD_SHAPE;
    columns += widths[i];
  }
  fp8_rope_plan* p = static_cast<fp8_rope_plan*>(calloc(1, sizeof(fp8_rope_plan)));
  if (!p) return FP8W8A8_ERR_HIP;
  p->head_dim = (int)head_dim;
  p->interleaved = layout == FP8W8A8_ROPE_INTERLEAVED;
  p->table.columns = (int32_t)columns;
  p->table.axes = axes;
  int at = 0;
  for (int i = 0; i < axes; ++i) {
    p->table.begin[i] = 2 * at;
    p->table.half[i] = (int32_t)(widths[i] / 2);
    for (int j = 0; j < widths[i] / 2; ++j, ++at) {
      // whole turns per unit of position, in two fp32 parts
      const double turns = pow(base, -2.0 * j / (double)widths[i]) / (2.0 * M_PI);
      p->table.hi[at] = (float)turns;
      p->table.lo[at] = (float)(turns - (double)p->table.hi[at]);
      p->table.axis[at] = (uint8_t)i;
    }
  }
  *out = p;
  return FP8W8A8_OK;
}

int fp8_rope_run(const fp8_rope_plan* plan, int64_t tokens, const int32_t* positions, const fp8_rows* q,
                 const fp8_rows* q_out, const fp8_rows* k, const fp8_rows* k_out, void* stream) {
  if (!plan || !positions || (k && !k_out)) return FP8W8A8_ERR_INVALID_ARG;
  if (tokens < 0 || tokens >= FP8W8A8_MAX_ROWS) return FP8W8A8_ERR_BAD_SHAPE;
  int st = check_rows(q);
  if (st == FP8W8A8_OK) st = check_rows_out(q_out, q, plan->head_dim);
  if (st == FP8W8A8_OK && k) st = check_rows(k);
  if (st == FP8W8A8_OK && k) st = check_rows_out(k_out, k, plan->head_dim);
  if (st != FP8W8A8_OK) return st;
  if (!aligned(positions, 4)) return FP8W8A8_ERR_MISALIGNED;
  if (tokens == 0) return FP8W8A8_OK;
  // at most one wavefront per token and head
  if (tokens * (q->heads + (k ? k->heads : 0)) * 64 >= kMaxGridThreads) return FP8W8A8_ERR_BAD_SHAPE;
  int cus = 0;
  st = current_device_ok(&cus);
  if (st != FP8W8A8_OK) return st;
  hipError_t e = launch_rope(plan->head_dim, plan->interleaved != 0, plan->table, tokens, positions,
                             rope_tensor(q, q_out), rope_tensor(k, k_out), cus > 0 ? cus : 256,
                             static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8W8A8_OK : FP8W8A8_ERR_HIP;
}

void fp8_rope_destroy(fp8_rope_plan* plan) { free(plan); }

int fp8_kv_cache_create(int device, int64_t pages, int64_t page_tokens, int64_t heads, int64_t head_dim, void* k_codes,
                        void* v_codes, float* k_scale, float* v_scale, fp8_kv_cache** out) {
  if (!out || !k_codes || !v_codes || !k_scale || !v_scale) return FP8W8A8_ERR_INVALID_ARG;
  if (pages < 1 || pages > INT32_MAX || heads < 1 || heads > kMaxHeads) return FP8W8A8_ERR_BAD_SHAPE;
  if (page_tokens != 32 && page_tokens != 64 && page_tokens != 128) return FP8W8A8_ERR_BAD_SHAPE;
  if (head_dim != 64 && head_dim != 128) return FP8W8A8_ERR_BAD_SHAPE;
  if (!aligned(k_codes, 16) || !aligned(v_codes, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return FP8W8A8_ERR_MISALIGNED;
  int cus = 0;
  int st = query_device(device, &cus);
  if (st != FP8W8A8_OK) return st;
  fp8_kv_cache* p = static_cast<fp8_kv_cache*>(calloc(1, sizeof(fp8_kv_cache)));
  if (!p) return FP8W8A8_ERR_HIP;
  p->device = device;
  p->cu_count = cus > 0 ? cus : 256;
  p->c = KvCache{static_cast<uint8_t*>(k_codes), static_cast<uint8_t*>(v_codes), k_scale, v_scale, (int)pages,
                 (int)heads, (int)page_tokens, (int)head_dim};
  *out = p;
  return FP8W8A8_OK;
}

void fp8_kv_cache_destroy(fp8_kv_cache* cache) { free(cache); }

int fp8_kv_append(const fp8_kv_cache* cache, int64_t requests, int64_t tokens, const fp8_rows* k, const fp8_rows* v,
                  const int32_t* table, int64_t table_pages, const int32_t* lengths, const int32_t* starts,
                  void* stream) {
  if (!cache) return FP8W8A8_ERR_INVALID_ARG;
  int st = check_rows(k);
  if (st == FP8W8A8_OK) st = check_rows(v);
  if (st == FP8W8A8_OK) st = check_paged(cache->c, requests, tokens, table, table_pages, lengths, starts);
  if (st != FP8W8A8_OK) return st;
  if (k->heads != cache->c.heads || v->heads != cache->c.heads) return FP8W8A8_ERR_BAD_SHAPE;
  if (requests == 0 || tokens == 0) return FP8W8A8_OK;
  // the pages that may receive tokens, a workgroup of up to 512 threads each
  if ((tokens / cache->c.page_tokens + 2 * requests) * 512 >= kMaxGridThreads) return FP8W8A8_ERR_BAD_SHAPE;
  st = plan_device_current(cache->device);
  if (st != FP8W8A8_OK) return st;
  hipError_t e = launch_kv_append(cache->c, requests, tokens, rows_in(k), rows_in(v), table, table_pages, lengths,
                                  starts, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8W8A8_OK : FP8W8A8_ERR_HIP;
}

size_t fp8_kv_attend_workspace_bytes(const fp8_kv_cache* cache, int64_t requests, int64_t tokens, int64_t heads,
                                     int64_t table_pages) {
  if (!cache || requests <= 0 || tokens <= 0 || check_batch(requests, tokens) != FP8W8A8_OK) return 0;
  if (heads < 1 || heads > kMaxHeads || heads % cache->c.heads != 0 || !table_fits(cache->c, table_pages)) return 0;
  const AttendCut cut = kv_attend_cut(cache->c, requests, tokens, heads, table_pages, cache->cu_count);
  return kv_attend_fits(cache->c, cut, tokens, heads) ? kv_attend_workspace_bytes(cache->c, cut, heads) : 0;
}

int fp8_kv_attend(const fp8_kv_cache* cache, int64_t requests, int64_t tokens, const fp8_rows* q, const int32_t* table,
                  int64_t table_pages, const int32_t* lengths, const int32_t* starts, float scale, int causal,
                  void* out_bf16, void* workspace, size_t workspace_bytes, void* stream) {
  if (!cache || !out_bf16) return FP8W8A8_ERR_INVALID_ARG;
  int st = check_rows(q);
  if (st == FP8W8A8_OK) st = check_paged(cache->c, requests, tokens, table, table_pages, lengths, starts);
  if (st != FP8W8A8_OK) return st;
  if (q->heads % cache->c.heads != 0) return FP8W8A8_ERR_BAD_SHAPE;
  if (!(scale > 0.0f) || !isfinite(scale)) return FP8W8A8_ERR_INVALID_ARG;
  if (!aligned(out_bf16, 16)) return FP8W8A8_ERR_MISALIGNED;
  if (requests == 0 || tokens == 0) return FP8W8A8_OK;
  const AttendCut cut = kv_attend_cut(cache->c, requests, tokens, q->heads, table_pages, cache->cu_count);
  if (!kv_attend_fits(cache->c, cut, tokens, q->heads)) return FP8W8A8_ERR_BAD_SHAPE;
  const size_t need = kv_attend_workspace_bytes(cache->c, cut, q->heads);
  if (need > 0) {
    if (!workspace) return FP8W8A8_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return FP8W8A8_ERR_MISALIGNED;
    if (workspace_bytes < need) return FP8W8A8_ERR_WORKSPACE_TOO_SMALL;
  }
  st = plan_device_current(cache->device);
  if (st != FP8W8A8_OK) return st;
  hipError_t e = launch_kv_attend(cache->c, cut, requests, tokens, q->heads, rows_in(q), table, table_pages, lengths,
                                  starts, scale, causal != 0, static_cast<uint16_t*>(out_bf16), workspace,
                                  static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8W8A8_OK : FP8W8A8_ERR_HIP;
}

int fp8_lora_create(int device, int64_t adapters, int64_t rank, int64_t n, int64_t k, const void* a_bf16,
                    const void* b_bf16, const float* scale, fp8_lora_plan** out) {
  if (!out || !a_bf16 || !b_bf16 || !scale) return FP8W8A8_ERR_INVALID_ARG;
  if (adapters < 1 || adapters > INT32_MAX) return FP8W8A8_ERR_BAD_SHAPE;
  if (rank < 8 || rank > FP8W8A8_MAX_RANK || rank % 8 != 0) return FP8W8A8_ERR_BAD_SHAPE;
  if (n < 16 || k < 16 || n > FP8W8A8_MAX_DIM || k > FP8W8A8_MAX_DIM || n % 16 != 0 || k % 16 != 0)
    return FP8W8A8_ERR_BAD_SHAPE;
  if (!aligned(a_bf16, 16) || !aligned(b_bf16, 16) || !aligned(scale, 4)) return FP8W8A8_ERR_MISALIGNED;
  int cus = 0;
  int st = query_device(device, &cus);
  if (st != FP8W8A8_OK) return st;
  fp8_lora_plan* p = static_cast<fp8_lora_plan*>(calloc(1, sizeof(fp8_lora_plan)));
  if (!p) return FP8W8A8_ERR_HIP;
  p->device = device;
  p->cu_count = cus > 0 ? cus : 256;
  p->w = LoraWeights{static_cast<const uint16_t*>(a_bf16), static_cast<const uint16_t*>(b_bf16), scale, (int)adapters,
                     (int)rank, (int)k, (int)n};
  *out = p;
  return FP8W8A8_OK;
}

int fp8_lora_run(const fp8_lora_plan* plan, int64_t requests, int64_t tokens, const void* x_bf16,
                 const void* base_bf16, const int32_t* starts, const int32_t* adapter, void* out_bf16, void* stream) {
  if (!plan || !x_bf16 || !base_bf16 || !starts || !adapter || !out_bf16) return FP8W8A8_ERR_INVALID_ARG;
  int st = check_batch(requests, tokens);
  if (st != FP8W8A8_OK) return st;
  if (!aligned(x_bf16, 16) || !aligned(base_bf16, 16) || !aligned(out_bf16, 16) || !aligned(starts, 4) ||
      !aligned(adapter, 4))
    return FP8W8A8_ERR_MISALIGNED;
  if (requests == 0 || tokens == 0) return FP8W8A8_OK;
  // workgroups of 1024 threads where few tokens stand in a request, of 256 where many do
  if ((tokens <= 16 * requests ? (tokens / 16 + requests) * 1024 : (tokens / 32 + requests) * 256) >= kMaxGridThreads)
    return FP8W8A8_ERR_BAD_SHAPE;
  st = plan_device_current(plan->device);
  if (st != FP8W8A8_OK) return st;
  hipError_t e = launch_lora(plan->w, requests, tokens, static_cast<const uint16_t*>(x_bf16),
                             static_cast<const uint16_t*>(base_bf16), starts, adapter,
                             static_cast<uint16_t*>(out_bf16), plan->cu_count, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8W8A8_OK : FP8W8A8_ERR_HIP;
}

void fp8_lora_destroy(fp8_lora_plan* plan) { free(plan); }

}  // extern "C"
