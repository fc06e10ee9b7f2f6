// Append of new keys and values to a paged FP8 cache, with one scale for each page and head.
//
// New token t of a request with length L after the append and n new tokens stands at place
// L - n + t. For every page that receives tokens, and every head,
//   fresh = max(fl32(amax of the page's new values / 448), 2^-60),
//   s     = max(s_old, fresh) if tokens stood in the page before, else fresh,
//   new   = e4m3fn_rne_sat(fl32(x / s)),
//   old   = e4m3fn_rne_sat(fl32(fl32(dec(old) * s_old) / s)) where s grew.
// The floor of 2^-60 keeps every scale a normal number whose logarithm the attention may
// use; values below it are zero codes.
//
// HBM-bound: 2 bytes read, 1 written per element. One workgroup takes one page of one head,
// K and V: each lane loads 8 columns of 4 consecutive tokens of both, the maxima meet in LDS,
// and the values are quantised from the registers. K codes leave in rows [token, dim]. V
// codes leave in rows [dim, token], the operand order of the attention's second product: 4 x 4
// bytes are turned in registers and the page passes through LDS, so that whole pages are
// stored 16 bytes per lane; a partly filled page is stored byte by byte. Values are read once and
// codes not again soon: both go past the caches. 32760 tokens, 16 heads of 128: 90 us with
// inputs that change from call to call, 4.5 TB/s (on inputs that stand in the caches 64.5 us; K
// and V in workgroups of their own, with ordinary stores, took 96).
// One token of 64 requests, 8.7 us, is a chain of loads: offsets, page number, scale, old codes.
#include "gemm_common.h"
#include "internal.h"
#include "quant_row.h"
#include "ragged.h"

namespace fp8w8a8 {
namespace {

struct AppendArgs {
  KvCache c;
  Ragged r;
  RowsIn in[2];  // keys, values
  const int32_t* table;
  const int32_t* lengths;
  int table_pages;
};

// Codes of one dword's four values once more, at the larger scale.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float s_old, float s) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  return qrow::pack4(lo[0] * s_old / s, lo[1] * s_old / s, hi[0] * s_old / s, hi[1] * s_old / s);
}

// The codes of a page's first `first` tokens at the new scale, and no other byte: 16 codes of a
// chunk of K are of one token, of V of 16 neighbouring ones.
template <int PAGE, int DIM, bool VALUES>
__device__ __forceinline__ void rescale_page(uint8_t* codes, int tid, int first, float s_old, float s) {
  constexpr int kThreads = PAGE * DIM / 32;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = tid + h * kThreads;
    const int live = VALUES ? min(16, first - i * 16 % PAGE) : i * 16 / DIM < first ? 16 : 0;
    if (live <= 0) continue;
    uint32_t* chunk = reinterpret_cast<uint32_t*>(codes + 16 * i);
    const uint4 old = *reinterpret_cast<const uint4*>(chunk);
    const uint32_t w[4] = {old.x, old.y, old.z, old.w};
    uint32_t y[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) y[d] = rescale4(w[d], s_old, s);
    if (live == 16) {
      *reinterpret_cast<uint4*>(chunk) = make_uint4(y[0], y[1], y[2], y[3]);
      continue;
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if (live >= 4 * d + 4) chunk[d] = y[d];
      else
        for (int e = 4 * d; e < live; ++e) codes[16 * i + e] = (uint8_t)(y[d] >> (8 * (e & 3)));
    }
  }
}

template <int PAGE, int DIM>
__global__ __launch_bounds__(PAGE* DIM / 32) void kv_append_kernel(AppendArgs a) {
  constexpr int kThreads = PAGE * DIM / 32;
  constexpr int kWaves = kThreads / 64;
  constexpr int kChunks = DIM / 8;
  __shared__ float wave_amax[2][kWaves];
  __shared__ __attribute__((aligned(16))) uint32_t turned[DIM * PAGE / 4];
  const int tid = threadIdx.x, lane = tid & 63;
  constexpr int kShift = __builtin_ctz(PAGE);
  const int head = blockIdx.y;
  const Request q = request_of_slot<2>(a.r, 1, kShift, blockIdx.x, lane, a.lengths);
  const int64_t length = q.value;
  const int64_t begin = length - q.rows;  // place of the request's first new token
  if (q.index < 0 || q.rows == 0 || begin < 0) return;
  const int64_t page_index = (begin >> kShift) + q.tile;
  const int64_t page_begin = page_index << kShift;
  if (page_begin >= length || page_index >= a.table_pages) return;
  const int chunk = tid % kChunks, tok = tid / kChunks * 4;
  const int first = (int)max((int64_t)0, begin - page_begin);       // first new place in the page
  const int last = (int)min((int64_t)PAGE, length - page_begin);    // one past the last
  const int64_t row = q.row0 + page_begin + tok - begin;              // of this lane's first token
  uint4 x[2][4];
#pragma unroll
  for (int v = 0; v < 2; ++v)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const bool live = tok + t >= first && tok + t < last;
      x[v][t] = make_uint4(0, 0, 0, 0);
      if (live)
        x[v][t] = __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const v4u*>(
                                                a.in[v].x + (row + t) * a.in[v].token + head * a.in[v].head + chunk * 8)));
    }
  const int page = a.table[(int64_t)q.index * a.table_pages + page_index];
  if (page < 0 || page >= a.c.pages) return;
  const int64_t unit = (int64_t)page * a.c.heads + head;
  uint8_t *k = a.c.k + unit * (PAGE * DIM), *v = a.c.v + unit * (PAGE * DIM);
  float* const scales[2] = {a.c.k_scale + unit, a.c.v_scale + unit};
  float s_old[2], s[2], r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    s_old[i] = first > 0 ? *scales[i] : 0.0f;
    float amax = qrow::absmax16(qrow::absmax16(0.0f, x[i][0], x[i][1]), x[i][2], x[i][3]);
    amax = qrow::wave_max(amax);
    if (lane == 0) wave_amax[i][tid >> 6] = amax;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float amax = wave_amax[i][0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) amax = fmaxf(amax, wave_amax[i][w]);
    s[i] = fmaxf(s_old[i], fmaxf(amax / 448.0f, 0x1p-60f));
    r[i] = 1.0f / s[i];
    if (s[i] != s_old[i] && tid == 0) *scales[i] = s[i];
  }
  if (first > 0) {
    if (s[0] != s_old[0]) rescale_page<PAGE, DIM, false>(k, tid, first, s_old[0], s[0]);
    if (s[1] != s_old[1]) rescale_page<PAGE, DIM, true>(v, tid, first, s_old[1], s[1]);
  }
  // s is at least 2^-60, so that the fast quotient is the rounded one wherever it is no zero code
  uint32_t code[2][4][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t w[4] = {x[i][t].x, x[i][t].y, x[i][t].z, x[i][t].w};
      const auto over = [&](float y) { return qrow::quotient<qrow::Mode::kFast>(y, s[i], r[i]); };
#pragma unroll
      for (int j = 0; j < 2; ++j)
        code[i][t][j] = qrow::pack4(over(qrow::bf16_lo(w[2 * j])), over(qrow::bf16_hi(w[2 * j])),
                                 over(qrow::bf16_lo(w[2 * j + 1])), over(qrow::bf16_hi(w[2 * j + 1])));
    }
#pragma unroll
  for (int t = 0; t < 4; ++t)
    if (tok + t >= first && tok + t < last)
      __builtin_nontemporal_store((unsigned long long)code[0][t][0] | ((unsigned long long)code[0][t][1] << 32), reinterpret_cast<unsigned long long*>(k + (tok + t) * DIM + chunk * 8));
  if (first > 0 || last < PAGE) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (tok + t >= first && tok + t < last)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[(chunk * 8 + e) * PAGE + tok + t] = (uint8_t)(code[1][t][e >> 2] >> (8 * (e & 3)));
    return;
  }
  // column e of the four tokens as one dword
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    uint32_t d = 0;
#pragma unroll
    for (int t = 0; t < 4; ++t) d |= (code[1][t][e >> 2] >> (8 * (e & 3)) & 0xffu) << (8 * t);
    turned[(chunk * 8 + e) * (PAGE / 4) + tok / 4] = d;
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h)
    __builtin_nontemporal_store(reinterpret_cast<const v4u*>(turned)[tid + h * kThreads], reinterpret_cast<v4u*>(v) + tid + h * kThreads);
}

template <int PAGE, int DIM>
void launch(const AppendArgs& a, int64_t slots, hipStream_t stream) {
  kv_append_kernel<PAGE, DIM><<<dim3((unsigned)slots, (unsigned)a.c.heads), dim3(PAGE * DIM / 32), 0, stream>>>(a);
}

}  // namespace

hipError_t launch_kv_append(const KvCache& c, int64_t requests, int64_t tokens, const RowsIn& k, const RowsIn& v,
                            const int32_t* table, int64_t table_pages, const int32_t* lengths, const int32_t* starts,
                            hipStream_t stream) {
  const AppendArgs a{c, {starts, (int)requests, (int)tokens}, {k, v}, table, lengths, (int)table_pages};
  const int shift = __builtin_ctz(c.page_tokens);
  const int64_t slots = ragged_slots(tokens, requests, 1, shift, 2);
  if (c.head_dim == 64) {
    if (shift == 5) launch<32, 64>(a, slots, stream);
    else if (shift == 6) launch<64, 64>(a, slots, stream);
    else launch<128, 64>(a, slots, stream);
  } else {
    if (shift == 5) launch<32, 128>(a, slots, stream);
    else if (shift == 6) launch<64, 128>(a, slots, stream);
    else launch<128, 128>(a, slots, stream);
  }
  return hipGetLastError();
}

}  // namespace fp8w8a8
