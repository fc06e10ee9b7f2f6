// Attention over the paged FP8 cache: for query row x of a request with n new tokens and
// length L, and the key / value head its query head shares,
//   out = sum_j softmax_j(scale * q . k_j) v_j,   j < L (or j <= L - n + x where causal),
// with k and v dequantised (code * page scale). Tokens on a page that the table does not
// name are masked; a row with no token left gives zeros.
//
// Both products run on the matrix cores, transposed: S^T = K Q^T and O^T = V^T P^T, so that
// a lane holds one query row (its column) of either and 32 neighbouring tokens of the
// scores, and the softmax and its rescaling need nothing from other lanes but the maximum of
// the lane that holds the other 32 tokens of a tile of 64. The tokens of a score tile are
// dealt to matrix rows so (token_of_row) that the probabilities already stand where the
// second product wants them.
//
//   * Scores: K codes widen to bf16 exactly in registers and the queries stay as they are, so
//     that a score is the fp32 sum of exact products. (The FP8 matrix instructions would take
//     the codes as they are, with each query split into two e4m3 numbers, in the same time.
//     But they align the products of a group to the largest and cut them there: one product of
//     2048 and 63 of 0.633 summed to 0.93 too little, and beside an outlying channel scores of 64
//     came out 0.02 off.)
//   * Softmax: the exponent carries the V scale of the token's page,
//     p' = 2^(score * log2 e + log2(v_scale) - m), so that O^T sums p' times V codes and
//     needs no scaling by pages; the denominator sums p' / v_scale. m is a bound, not the
//     maximum: it moves (and O and l are rescaled) only when a lane's p' of a tile sum to
//     more than 2^40, or its p' / v_scale to more than 2^90, so that a tile needs no maximum.
//     It moves to the largest score * log2 e + max(log2(v_scale), -60): p' is then at most 1 and
//     p' / v_scale at most 2^60, whatever V scales a request holds, and the denominator of 2^30
//     tokens stays within fp32 with its inverse.
//   * Output: p' is rounded once to bf16, which keeps 8 bits over the whole range of fp32
//     (fp16 would keep 11, but lose what lies 2^-32 below a row's largest, all there is in a
//     column whose strongest tokens hold zero); the denominator is a sum in fp32 (see powers).
//     V codes widen to bf16 exactly, sums are fp32.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "gemm_common.h"
#include "internal.h"
#include "ragged.h"

namespace fp8w8a8 {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kTile = 64;          // tokens of a score tile
constexpr float kNone = -1e30f;    // the running maximum before any token
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMost = 0x1p40f;   // a lane's p' of a tile may sum to this before m moves,
constexpr float kWeight = 0x1p-50f;  // and its p' / v_scale, its share of the denominator, to kMost / kWeight
constexpr float kLeastLog = -60.0f;  // of a V scale's logarithm in the bound

struct AttendArgs {
  KvCache c;
  Ragged r;
  RowsIn q;
  const int32_t* table;
  const int32_t* lengths;
  uint16_t* out;    // [rows, heads, dim]
  float* part_out;  // [parts, part_rows * heads, dim + 2]: a part's O, then m and l, where parts > 1
  int table_pages, heads, group, shift, causal, parts, slots;
  int skip;       // slots before this launch's first, served by another launch (of one request only)
  int part_rows;  // rows of part_out: the tensor's, or with skipped slots those that may be left of the request's
  float scale;
};

// Matrix row m of a score tile (of two, a = 0, 1, that make 64 tokens) is this token: lanes of
// the lower half then hold tokens 0..31 in order, 16 of each tile, those of the upper 32..63.
__device__ __forceinline__ int token_of_row(int a, int m) {
  return 32 * ((m >> 2) & 1) + 16 * a + 4 * (m >> 3) + (m & 3);
}
// Matrix row m of output tile b is this column of V, so that a lane ends with 16 neighbours.
__device__ __forceinline__ int dim_of_row(int b, int m) { return 32 * b + 16 * ((m >> 2) & 1) + 4 * (m >> 3) + (m & 3); }

// Their inverses: the matrix row (of 64) of a token, and (of DIM) of a column.
__device__ __forceinline__ int row_of_token(int t) {
  return 32 * ((t >> 4) & 1) + 8 * ((t >> 2) & 3) + 4 * (t >> 5) + (t & 3);
}
__device__ __forceinline__ int row_of_dim(int d) { return (d & ~31) + 8 * ((d >> 2) & 3) + 4 * ((d >> 4) & 1) + (d & 3); }

__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32, 64); }

__device__ __forceinline__ v8bf widen(int w0, int w1) {
  const v2bf16 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
  const v2bf16 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
  const v2bf16 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
  const v2bf16 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// p' of a lane's N scores, rounded to bf16, and the sum of the rounded ones: the weights of a row
// then sum to one, and values that are all alike come back as they are (with the sum of the
// unrounded ones a row that one token rules is off by up to 2^-8 in all its columns). By
// two-element dot products, or, DOTS false, by additions of the widened halves: the dot products go
// through the matrix cores, and beside another wavefront's products one takes 38 cycles, two
// additions and the widening 20. Where a wavefront's softmax runs beside such products all the time
// (kv_attend_teams) the additions are quicker (32760 x 32760, 16 heads of 128: 7.33 ms against 7.47;
// 1560 x 32760: 438 us against 453), elsewhere the dot products (6 ragged causal requests, 32 heads
// of 64: 122 us against 131). Sums of the unrounded p' would take 7.08 ms and 423 us.
template <int N, bool DOTS, class Scores>
__device__ __forceinline__ float powers(const Scores& s, float c, float add, v8bf (&p)[N / 8]) {
  float sum[2] = {0.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s(e), c, add));
    const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s(e + 1), c, add));
    const v2bf16 h = __builtin_convertvector((v2f){x, y}, v2bf16);
    if constexpr (DOTS) {
      const v2bf16 one = {(__bf16)1.0f, (__bf16)1.0f};
      sum[e / 2 % 2] = __builtin_amdgcn_fdot2_f32_bf16(h, one, sum[e / 2 % 2], false);
    } else {
      const uint32_t w = __builtin_bit_cast(uint32_t, h);
      sum[0] += __uint_as_float(w << 16);
      sum[1] += __uint_as_float(w & 0xffff0000u);
    }
    p[e / 8][e % 8] = h[0];
    p[e / 8][e % 8 + 1] = h[1];
  }
  return sum[0] + sum[1];
}

// 2^x for x <= 0 in two equal factors: a product with both keeps what the power alone, zero below
// 2^-126, would lose (a denominator may stand far above or below 1, see softmax_step).
__device__ __forceinline__ float root_power(float x) { return __builtin_amdgcn_exp2f(0.5f * x); }

// Only the first `live` of a lane's N tokens count.
template <int N, class Scores>
__device__ __forceinline__ void mask(const Scores& s, int live) {
#pragma unroll
  for (int e = 0; e < N; ++e) s.set(e, e < live ? s(e) : -INFINITY);
}

// A tile's scores of N tokens per lane -> p', with m and l of the lane's row brought up to date
// and O through `rescale`. s(e): the e-th score; c: score units of the tokens' page; lv, rv:
// log2 and inverse of its V scale; `over`: the largest over the lanes that share a row; `first`:
// no tile came before, so that the bound is sure to move. `rescale` multiplies O by the square of its
// argument.
template <int N, bool DOTS, class Scores, class Over, class Rescale>
__device__ __forceinline__ void softmax_step(bool first, const Scores& s, float c, float lv, float rv, v8bf (&p)[N / 8],
                                             float& m, float& l, const Over& over, const Rescale& rescale) {
  float sum = INFINITY;
  if (!first) sum = powers<N, DOTS>(s, c, lv - m, p);
  if (__builtin_expect(__any(!(fmaxf(sum, sum * rv * kWeight) <= kMost)), 0)) {
    float mx = s(0);
#pragma unroll
    for (int e = 1; e < N; ++e) mx = fmaxf(mx, s(e));
    const float up = fmaxf(m, over(__builtin_fmaf(mx, c, fmaxf(lv, kLeastLog))));
    const float fix = root_power(m - up);
    m = up;
    l = l * fix * fix;
    rescale(fix);
    sum = powers<N, DOTS>(s, c, lv - m, p);
  }
  l += sum * rv;
}

// The scores of a lane: 16 in each of two 32-row tiles, or 4 in each of four 16-row tiles.
struct Tiles32 {
  v16f (&s)[2];
  __device__ __forceinline__ float operator()(int e) const { return s[e >> 4][e & 15]; }
  __device__ __forceinline__ void set(int e, float x) const { s[e >> 4][e & 15] = x; }
};
struct Tiles16 {
  v4f (&s)[4];
  __device__ __forceinline__ float operator()(int e) const { return s[e >> 2][e & 3]; }
  __device__ __forceinline__ void set(int e, float x) const { s[e >> 2][e & 3] = x; }
};

// What one wavefront holds of 32 query rows (packed: the query heads of a key head side by
// side, token by token). Lane: row lane % 32, and half lane / 32 of a tile's tokens.
template <int DIM>
struct Rows {
  static constexpr int kSteps = DIM / 16;  // matrix steps over the head dimension
  static constexpr int kOut = DIM / 32;    // output tiles
  v8bf q[kSteps];
  v16f o[kOut];
  float m, l;  // bound and sum

  // p: the row's DIM values, or null for a row that is not there
  __device__ __forceinline__ void load(const uint16_t* p, int half) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
      q[i] = __builtin_bit_cast(v8bf, p ? reinterpret_cast<const uint4*>(p)[2 * i + half] : make_uint4(0, 0, 0, 0));
#pragma unroll
    for (int b = 0; b < kOut; ++b) o[b] = v16f{};
    m = kNone;
    l = 0.0f;
  }

  // Scores of a lane's 32 tokens -> p', with m, l and O brought up to date (see softmax_step).
  template <bool DOTS>
  __device__ __forceinline__ void softmax(bool first, v16f (&s)[2], float c, float lv, float rv, v8bf (&p)[4]) {
    softmax_step<32, DOTS>(first, Tiles32{s}, c, lv, rv, p, m, l, [](float x) { return fmaxf(x, __shfl_xor(x, 32, 64)); },
                             [&](float fix) {
#pragma unroll
                               for (int b = 0; b < kOut; ++b)
#pragma unroll
                                 for (int e = 0; e < 16; ++e) o[b][e] = o[b][e] * fix * fix;
                             });
  }
};

// A lane's 4 N codes of V with those past the first `live` tokens cleared: what stands in
// unused slots may be no number.
template <int N, class V>
__device__ __forceinline__ void clear_past(V& v, int live) {
#pragma unroll
  for (int d = 0; d < N; ++d) {
    const int n = live - 4 * d;
    v[d] = n >= 4 ? v[d] : n <= 0 ? 0 : v[d] & ((1 << (8 * n)) - 1);
  }
}

// A lane's 4 N codes of V with those that are no number cleared: on the tiles that some rows of
// a causal request see further into than others, a place that a row must not see would reach
// it as 0 times NaN.
template <int N, class V>
__device__ __forceinline__ void clear_nan(V& v) {
#pragma unroll
  for (int d = 0; d < N; ++d) {
    const uint32_t w = (uint32_t)v[d], top = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // of codes 0x7f, 0xff
    v[d] = (int)(w & ~(top | (top - (top >> 7))));
  }
}

// Page numbers and scales of 64 pages of a request, one per lane, fetched together; a tile's
// are then read across lanes. A page that holds no place below `seen` is not looked at, whether
// the table names it or not: its codes and scales may be anything.
struct Window {
  int id;           // -1: not named
  int lo, hi;       // byte offset of the page's codes of a head (page 0's where not named)
  float c, lv, rv;  // exponent units of a score; log2 and inverse of the V scale

  __device__ __forceinline__ void load_ids(const AttendArgs& a, const int32_t* row, int seen, int first, int lane) {
    const int j = first + lane;
    const int p = j < (seen + (1 << a.shift) - 1) >> a.shift ? row[j] : -1;
    id = p >= 0 && p < a.c.pages ? p : -1;
  }
  __device__ __forceinline__ void load_scales(const AttendArgs& a, int kv, int64_t page_bytes) {
    const int64_t unit = (int64_t)max(id, 0) * a.c.heads + kv;
    lo = (int)(unit * page_bytes);
    hi = (int)(unit * page_bytes >> 32);
    // the append's scales are at least 2^-60; of a page of the request that it has not filled yet
    // (places a causal row must not see) the scale may be no number
    const float v = id >= 0 ? fminf(fmaxf(a.c.v_scale[unit], 0x1p-100f), 0x1p120f) : 1.0f;
    const float k = id >= 0 ? a.c.k_scale[unit] : 1.0f;
    c = fmaxf(k * (a.scale * kLog2e), 0x1p-126f);
    lv = __builtin_amdgcn_logf(v);
    rv = 1.0f / v;
  }
};

__device__ __forceinline__ int read_lane(int x, int i) { return __builtin_amdgcn_readlane(x, i); }
__device__ __forceinline__ float read_lane(float x, int i) { return __int_as_float(read_lane(__float_as_int(x), i)); }

// A page's value for this lane's 32 tokens of a tile: page `i` of the window, or with pages of
// 32 tokens page i + 1 for the upper half.
template <bool SMALL, typename T>
__device__ __forceinline__ T of_half(T x, int i, int half) {
  const T lo = read_lane(x, i);
  if constexpr (!SMALL) return lo;
  const T hi = read_lane(x, i + 1);
  return half ? hi : lo;
}

// Whether both or one of the pages of a tile are not named.
template <bool SMALL>
__device__ __forceinline__ bool unnamed(int ids, int i) {
  return (read_lane(ids, i) | (SMALL ? read_lane(ids, i + 1) : 0)) < 0;
}

// The rows of one workgroup's tile: the first packed row of the request's, their number, the
// places that the whole tile and its first row see.
struct Span {
  int req, row0, first, rows, seen, seen_first, length, count;
};

// Inclusive sums over the lanes.
__device__ __forceinline__ int wave_sums(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);  // from 1, 2, 4, 8 lanes below in a row of 16
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // the last of a row, to the next
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // the last of the lower 32, to the upper
  return x;
}

// The slot-th tile of up to 64 requests in falling order of the tokens that it sees: workgroups
// start in this order, and none that takes long starts late (6 ragged causal requests, 32 heads
// of 64: 148.4 -> 134.1 us). A lane holds a request; at_least(t) of its tiles see at
// least t score tiles, and the slot's t is the largest with more than `slot` of them in all.
__device__ __forceinline__ Request request_by_length(const AttendArgs& a, int shift, int slot, int lane) {
  const int i = min(lane, a.r.requests - 1);
  const int begin = clamp_row(a.r.starts[i], a.r.rows), end = clamp_row(a.r.starts[i + 1], a.r.rows);
  const int value = a.lengths[i], length = min(max(value, 0), a.table_pages << a.shift);
  const int rows = lane < a.r.requests ? max(0, end - begin) : 0;
  const int tiles = (int)(((uint32_t)rows * a.group + (1u << shift) - 1) >> shift);
  auto at_least = [&](int t) {
    if (t == 0) return tiles;
    const int past = (t - 1) * kTile;  // tokens that do not suffice
    if (past >= length) return 0;
    // the tile's last row sees max(value, 0) - rows + token + 1
    const int token = past - (max(value, 0) - rows);
    return !a.causal || token <= 0 ? tiles : tiles - min(tiles, (int)((int64_t)token * a.group >> shift));
  };
  auto all = [&](int t) { return read_lane(wave_sums(at_least(t)), 63); };
  if (slot >= all(0)) return Request{-1, 0, 0, 0, 0};
  int lo = 0, hi = (a.table_pages << a.shift) / kTile + 2;
  while (hi - lo > 1) {
    const int t = (lo + hi) >> 1;
    if (all(t) > slot) lo = t;
    else hi = t;
  }
  const int more = at_least(lo + 1), same = at_least(lo) - more;
  const int r = slot - read_lane(wave_sums(more), 63), before = wave_sums(same);
  const int c = __popcll(__ballot(before <= r));
  const int tile = tiles - 1 - more - (r - (before - same));
  return Request{c, read_lane(begin, c), read_lane(rows, c), read_lane(tile, c), read_lane(value, c)};
}

template <int TILE_ROWS>
__device__ __forceinline__ bool find_span(const AttendArgs& a, int slot, int lane, Span& w) {
  constexpr int kShift = __builtin_ctz(TILE_ROWS);
  const Request q = TILE_ROWS > 16 && a.r.requests <= 64
                        ? request_by_length(a, kShift, slot, lane)
                        : request_of_slot<1>(a.r, a.group, kShift, slot, lane, a.lengths);
  if (q.index < 0) return false;
  w.req = q.index;
  w.row0 = q.row0;
  w.count = q.rows;
  w.first = q.tile << kShift;
  const int64_t all = (int64_t)w.count * a.group;
  if (w.first >= all) return false;
  w.rows = (int)min((int64_t)TILE_ROWS, all - w.first);
  const int cap = a.table_pages << a.shift;
  w.length = max(q.value, 0);
  // places seen by the tile's last and first row
  const int last = a.causal ? w.length - w.count + (w.first + w.rows - 1) / a.group + 1 : w.length;
  const int head = a.causal ? w.length - w.count + w.first / a.group + 1 : w.length;
  w.seen = min(max(last, 0), cap);
  w.seen_first = min(max(head, 0), cap);
  return true;
}

// Store a wavefront's rows: a lane's 16 neighbouring columns of each output tile.
template <int DIM>
__device__ __forceinline__ void store_rows(const AttendArgs& a, const Rows<DIM>& r, int64_t row_head, int part_row0,
                                           int part, int half) {
  if (a.parts == 1) {
    const float inv = r.l > 0.0f ? 1.0f / r.l : 0.0f;
    uint16_t* out = a.out + row_head * DIM + 16 * half;
#pragma unroll
    for (int b = 0; b < DIM / 32; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(r.o[b][8 * h + 2 * e] * inv, r.o[b][8 * h + 2 * e + 1] * inv);
        reinterpret_cast<uint4*>(out + 32 * b)[h] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    return;
  }
  const int64_t all = (int64_t)a.part_rows * a.heads;
  row_head -= (int64_t)part_row0 * a.heads;
  float* out = a.part_out + (part * all + row_head) * DIM;
#pragma unroll
  for (int b = 0; b < DIM / 32; ++b)
#pragma unroll
    for (int h = 0; h < 4; ++h)
      reinterpret_cast<float4*>(out + 32 * b + 16 * half)[h] =
          make_float4(r.o[b][4 * h], r.o[b][4 * h + 1], r.o[b][4 * h + 2], r.o[b][4 * h + 3]);
  if (half == 0) {
    float* ml = a.part_out + a.parts * all * DIM + (part * all + row_head) * 2;
    ml[0] = r.m;
    ml[1] = r.l;
  }
}

// Workgroup -> (slot, key head, part), XCD by XCD: the workgroups of one XCD serve as few key
// heads and parts as possible, so that those at work together share K and V in its L2. Few rows:
// neighbouring slots, often of one request, on one XCD.
__device__ __forceinline__ void place(const AttendArgs& a, int& slot, int& kv, int& part) {
  const int n = gridDim.x, id = blockIdx.x;
  const int q = n / kXcds, r = n % kXcds, xcd = id % kXcds;
  const int logical = xcd * q + min(xcd, r) + id / kXcds;
  slot = logical % a.slots;
  const int rest = logical / a.slots;
  part = rest % a.parts;
  kv = rest / a.parts;
}

// Many rows, whose slots fall in length: where key heads times parts are no multiple of the XCDs,
// 2, 4 or 8 of these take turns with the slots of some heads and parts, so that each gets long and
// short ones; who begins changes from one head and part to the next, so that all get nearly as many. (In
// runs of neighbouring slots instead: 2 causal requests, 16380 and 8000 rows, 4 heads of 64 on 2 480
// us against 300; 8 of up to 2000 on 6000, 20 heads of 128 on 5 466 against 401.) An XCD's unused
// workgroups are its last: dealt out between the others they leave some of its CUs two (12 heads of
// 128, 7800 rows on 7800, 362 us: 1.46 times that).
struct Deal {
  int slots, turns, each;  // log2 of the XCDs that take turns; heads and parts of each such set

  __host__ __device__ __forceinline__ Deal(int groups, int slots) : slots(slots) {
    static_assert(kXcds == 8, "powers of two");
    const int d = __builtin_ctz(groups | kXcds);
    turns = 3 - d;
    each = groups >> d;
  }
  // the XCD's first slot of the set's i-th head and part: the bits of i reversed, spread evenly
  __host__ __device__ __forceinline__ int first(int xcd, int i) const {
    const int mask = (1 << turns) - 1;
    return (xcd + ((0x73516240u >> 4 * (i & mask) & 7) >> (3 - turns))) & mask;
  }
  // slots of the set's i-th head and part that fall to an XCD, and all of its slots
  __host__ __device__ __forceinline__ int of_group(int xcd, int i) const {
    return (slots - first(xcd, i) + (1 << turns) - 1) >> turns;
  }
  __host__ __forceinline__ int64_t of_xcd(int xcd) const {
    int64_t n = (int64_t)(each >> turns) * slots;  // 1 << turns heads and parts have one turn at every slot
    for (int i = each >> turns << turns; i < each; ++i) n += of_group(xcd, i);
    return n;
  }
};
__device__ __forceinline__ bool place_in_turns(const AttendArgs& a, int& slot, int& kv, int& part) {
  const Deal d(a.c.heads * a.parts, a.slots);
  const int xcd = blockIdx.x % kXcds;
  int j = blockIdx.x / kXcds, i = j / d.slots << d.turns;
  j %= d.slots;
  for (; j >= d.of_group(xcd, i); ++i) j -= d.of_group(xcd, i);
  if (i >= d.each) return false;
  const int g = (xcd >> d.turns) * d.each + i;
  slot = a.skip + (j << d.turns) + d.first(xcd, i);
  part = g % a.parts;
  kv = g / a.parts;
  return true;
}

// A wavefront's row of set x: where it stands, whether it is there, and the places it sees.
struct Place {
  int64_t row_head;
  int limit;
  bool there;
};

template <int DIM>
__device__ __forceinline__ Place start_rows(const AttendArgs& a, const Span& w, int kv, int in_tile, int half,
                                            Rows<DIM>& r) {
  Place p;
  p.there = in_tile < w.rows;
  const int packed = w.first + in_tile;
  const int token = packed / a.group, head = kv * a.group + packed % a.group;
  r.load(p.there ? a.q.x + (w.row0 + token) * a.q.token + head * a.q.head : nullptr, half);
  p.limit = !p.there ? 0 : a.causal ? min(w.seen, max(w.length - w.count + token + 1, 0)) : w.seen;
  p.row_head = (int64_t)(w.row0 + token) * a.heads + head;
  return p;
}

// Rows of a workgroup's tile where there are many: 32 to a wavefront.
constexpr int kThreadRows(int threads) { return threads / 2; }

// Swizzle of the 16-byte chunks of an LDS row of N chunks (see swz): rows that fill a line of
// all banks are told apart by their low bits.
template <int N>
__device__ __forceinline__ int spread(int r) {
  if constexpr (N == 16) return r & 15;
  else return swz<128>(r);
}

// The tiles of a workgroup that shares them through LDS: 16 codes of K and of V to a lane and
// tile (THREADS = 4 DIM lanes), loaded ahead, widened to bf16 once for all wavefronts and left
// in LDS, K rows in the order of token_of_row and V rows in that of dim_of_row, chunks swizzled
// so that operand reads are conflict free.
template <int DIM, bool SMALL>
struct Feed {
  static constexpr int kThreads = 4 * DIM;
  static constexpr int kBytes = kTile * DIM * 2;  // of a widened tile of K, and of V
  static constexpr int kChunks = DIM / 8;         // 16-byte chunks of a widened K row; of a V row 8

  const AttendArgs& a;
  const Span& w;
  const int32_t* row;  // the request's page numbers
  int kv, lane, half, last;
  int64_t page_bytes;
  int k_off, v_off, k_dst, v_dst;  // this lane's place within a page, and in LDS
  int v_token;                     // of a tile, the first of its codes of V
  int up;                          // 1 on a tile's second page (pages of 32 tokens: the upper half of the wavefronts)
  Window now, ahead;               // of the tile in use, and of the tile being loaded
  int now_first, ahead_first;
  v4i raw_k, raw_v;

  __device__ __forceinline__ Feed(const AttendArgs& a, const Span& w, int kv, int lane, int t0, int t1)
      : a(a), w(w), row(a.table + (int64_t)w.req * a.table_pages), kv(kv), lane(lane), half(lane >> 5), last(t1 - 1) {
    page_bytes = (int64_t)DIM << a.shift;
    const int kt = threadIdx.x / (DIM / 16), kc = threadIdx.x % (DIM / 16), kr = row_of_token(kt);
    k_off = (SMALL ? kt & 31 : kt) * DIM + 16 * kc;
    k_dst = kr * DIM * 2 + ((2 * kc ^ spread<kChunks>(kr)) << 4);
    up = SMALL ? __builtin_amdgcn_readfirstlane(threadIdx.x / (2 * DIM)) : 0;
    const int vd = SMALL ? threadIdx.x / 2 % DIM : threadIdx.x / 4;
    const int vc = SMALL ? threadIdx.x % 2 + 2 * up : threadIdx.x % 4, vr = row_of_dim(vd);
    v_off = (vd << a.shift) + 16 * (SMALL ? vc & 1 : vc);
    v_dst = vr * 128 + ((2 * vc ^ spread<8>(vr)) << 4);
    v_token = 16 * vc;
    now_first = ahead_first = page_of(t0) & ~63;
    now.load_ids(a, row, w.seen, now_first, lane);
    now.load_scales(a, kv, page_bytes);
    ahead = now;
  }
  __device__ __forceinline__ int page_of(int t) const { return (t * kTile) >> a.shift; }
  // The windows for the use of tile t and the load of tile u.
  __device__ __forceinline__ void move(int t, int u) {
    if (page_of(t) - now_first >= 64) {
      now = ahead;
      now_first = ahead_first;
      asm volatile("");  // one tile in 32: a branch, and no selects in every tile
    }
    if (page_of(min(u, last)) - ahead_first >= 64) {
      ahead_first += 64;
      ahead.load_ids(a, row, w.seen, ahead_first, lane);
      ahead.load_scales(a, kv, page_bytes);
    }
  }
  // This lane's codes of tile u. Past the last tile that one is loaded again: without branches
  // around them the waits stay with the loads they are for.
  __device__ __forceinline__ void load(int u) {
    const int t = min(u, last), i = page_of(t) - ahead_first;
    const int64_t page = offset_of(i + up);
    // a page of 128 tokens holds two tiles
    const int second = a.shift == 7 ? (t & 1) * kTile : 0;
    raw_k = *reinterpret_cast<const v4i*>(a.c.k + page + (uint32_t)(k_off + second * DIM));
    raw_v = *reinterpret_cast<const v4i*>(a.c.v + page + (uint32_t)(v_off + second));
  }
  __device__ __forceinline__ int64_t offset_of(int i) const {
    return (int64_t)(((uint64_t)(uint32_t)read_lane(ahead.hi, i) << 32) | (uint32_t)read_lane(ahead.lo, i));
  }
  // What stands in unused slots of V may be no number.
  __device__ __forceinline__ void clear(int u) {
    const int t = min(u, last), i = page_of(t) - ahead_first;
    const bool named = read_lane(ahead.id, i + up) >= 0;
    if ((t + 1) * kTile > w.seen_first || !named) {
      clear_past<4>(raw_v, named ? w.seen - t * kTile - v_token : 0);
      if (a.causal) clear_nan<4>(raw_v);
    }
  }
  // Half h of this lane's codes, widened, to a tile in LDS.
  __device__ __forceinline__ void leave_k(uint8_t* tile, int h) const {
    *reinterpret_cast<v8bf*>(tile + (k_dst ^ (h << 4))) = widen(raw_k[2 * h], raw_k[2 * h + 1]);
  }
  __device__ __forceinline__ void leave_v(uint8_t* tile, int h) const {
    *reinterpret_cast<v8bf*>(tile + (v_dst ^ (h << 4))) = widen(raw_v[2 * h], raw_v[2 * h + 1]);
  }
  // The x-th operand of the output product of a tile (of V), and of its scores (of K).
  static __device__ __forceinline__ v8bf v_operand(const uint8_t* tile, int x, int lane) {
    const int r = 32 * (x % (DIM / 32)) + (lane & 31);
    return *reinterpret_cast<const v8bf*>(tile + r * 128 + (((4 * (lane >> 5) + x / (DIM / 32)) ^ spread<8>(r)) << 4));
  }
  static __device__ __forceinline__ v8bf k_operand(const uint8_t* tile, int x, int lane) {
    const int r = 32 * (x & 1) + (lane & 31);
    return *reinterpret_cast<const v8bf*>(tile + r * DIM * 2 + (((x & ~1) | (lane >> 5)) ^ spread<kChunks>(r)) * 16);
  }
};

// The softmax of tile t's scores in the row order of kv_attend_tiles and kv_attend_teams.
template <bool DOTS, int DIM, bool SMALL>
__device__ __forceinline__ void tile_softmax(const AttendArgs& a, const Feed<DIM, SMALL>& f, Rows<DIM>& r, v16f (&s)[2],
                                             v8bf (&p)[4], int t, int t0, int whole, int limit) {
  const int i = f.page_of(t) - f.now_first;
  // through LDS, whose time is not short here, where a wavefront needs two pages' values
  auto of = [&](float x) { return SMALL ? __shfl(x, i + f.half, 64) : read_lane(x, i); };
  const float c = of(f.now.c), lv = of(f.now.lv), rv = of(f.now.rv);
  if (t >= whole || unnamed<SMALL>(f.now.id, i))
    mask<32>(Tiles32{s}, of_half<SMALL>(f.now.id, i, f.half) < 0 ? 0 : limit - t * kTile - 32 * f.half);
  r.template softmax<DOTS>(t == t0, s, c, lv, rv, p);
}

// Many rows, heads of 64: four wavefronts of 32 rows. A tile is loaded two tiles ahead and
// left in LDS one ahead (two buffers, one barrier to a tile); three workgroups to a CU keep
// the matrix cores and the vector units busy beside each other. (A tile's 32 exponentials to
// a lane take longer than its products here, and in the turns of kv_attend_teams the matrix
// cores would wait for them: 6 ragged causal requests of 32 heads 143 against 168 us. The
// softmax in halves of 32 tokens, the output product of one under the exponentials of the
// other: 149 against 146.5; four workgroups to a CU in 128 registers, with spills: 169.)
// Bound by the vector instructions: of those 6 requests' 122 us they take 57% of all cycles,
// products 31%, and 14% of the CUs' time passes before the first and after the last workgroups.
template <int DIM, bool SMALL>
__global__ __launch_bounds__(4 * DIM, 3) void kv_attend_tiles(AttendArgs a) {
  typedef Feed<DIM, SMALL> F;
  constexpr int kOut = DIM / 32;
  __shared__ __attribute__((aligned(1024))) uint8_t k_tile[2][F::kBytes], v_tile[2][F::kBytes];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int slot, kv, part;
  if (!place_in_turns(a, slot, kv, part)) return;
  Span w;
  if (!find_span<kThreadRows(F::kThreads)>(a, slot, lane, w)) return;
  Rows<DIM> r;
  const Place pl = start_rows<DIM>(a, w, kv, 32 * wave + (lane & 31), lane >> 5, r);
  const int tiles = (w.seen + kTile - 1) / kTile;
  const int t0 = (int)((int64_t)tiles * part / a.parts), t1 = (int)((int64_t)tiles * (part + 1) / a.parts);
  const int whole = w.seen_first / kTile;  // tiles that every row sees whole

  if (t0 < t1) {
    F f(a, w, kv, lane, t0, t1);
    auto leave = [&](int t) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f.leave_k(k_tile[t & 1], h);
        f.leave_v(v_tile[t & 1], h);
      }
    };
    f.load(t0);
    f.clear(t0);
    leave(t0);
    f.move(t0, t0 + 1);
    f.load(t0 + 1);
    for (int t = t0; t < t1; ++t) {
      __syncthreads();
      v16f s[2] = {};
#pragma unroll
      for (int x = 0; x < DIM / 8; ++x)
        s[x & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(F::k_operand(k_tile[t & 1], x, lane), r.q[x / 2], s[x & 1], 0,
                                                           0, 0);
      f.clear(t + 1);
      leave(t + 1);
      f.move(t, t + 2);
      f.load(t + 2);
      v8bf p[4];
      tile_softmax<true>(a, f, r, s, p, t, t0, whole, pl.limit);
#pragma unroll
      for (int x = 0; x < 4 * kOut; ++x)
        r.o[x % kOut] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(F::v_operand(v_tile[t & 1], x, lane), p[x / kOut],
                                                                r.o[x % kOut], 0, 0, 0);
    }
  }
  r.l += other_half(r.l);
  if (pl.there) store_rows<DIM>(a, r, pl.row_head, a.skip ? w.row0 : 0, part, lane >> 5);
}

// All of the workgroup's LDS writes so far are there for what follows.
__device__ __forceinline__ void phase_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Many rows, heads of 128: eight wavefronts of 32 rows; two stand on each SIMD, one of each
// team (wave / 4), and take turns with the matrix cores. Between two barriers one team
// multiplies (the output product of tile t - 1 and the scores of tile t) while the other does
// the softmax of its scores.
//
//   interval    2 t                    2 t + 1                2 t + 2
//   team 0      multiply(t)            softmax(t)             multiply(t + 1)
//   team 1      softmax(t - 1)         multiply(t)            softmax(t)
//
// multiply(t) leaves its share of tile t + 2 in LDS (loaded an interval before) and loads the
// next: the tile is whole two intervals before its first use, so that the first operands of a
// multiply are read ahead of its barrier. K of a tile is read in multiply(t) and V in
// multiply(t + 1), by both teams, and written over three and four tiles later: each time after
// the barrier that follows its last reader.
//
// Bound by power: at 32760 x 32760 and 16 heads a CU takes 1760 cycles for each of 8192 intervals, the
// ends of its workgroups among them, 1024 of them products, and the clock, 2.4 GHz where it may,
// settles at 1.9 (1165 to 1210 TFLOP/s; cycles that are saved come back in part only, since the
// clock falls: 5% fewer are 3.4% of the time).
template <int DIM, bool SMALL>
__global__ __launch_bounds__(4 * DIM, 2) void kv_attend_teams(AttendArgs a) {
  typedef Feed<DIM, SMALL> F;
  constexpr int kOut = DIM / 32;
  __shared__ __attribute__((aligned(1024))) uint8_t k_tile[3][F::kBytes], v_tile[4][F::kBytes];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int team = wave >> 2;
  int slot, kv, part;
  if (!place_in_turns(a, slot, kv, part)) return;
  Span w;
  if (!find_span<kThreadRows(F::kThreads)>(a, slot, lane, w)) return;
  Rows<DIM> r;
  const Place pl = start_rows<DIM>(a, w, kv, 32 * wave + (lane & 31), lane >> 5, r);
  const int tiles = (w.seen + kTile - 1) / kTile;
  const int t0 = (int)((int64_t)tiles * part / a.parts), t1 = (int)((int64_t)tiles * (part + 1) / a.parts);
  const int whole = w.seen_first / kTile;  // tiles that every row sees whole

  if (t0 < t1) {
    F f(a, w, kv, lane, t0, t1);
    // Operands are read kAhead products before their use, and this wavefront's share of tile
    // t + 2 and the load of tile t + 3 go between the products a piece at a time. The order is
    // the one written: left to itself the compiler reads each operand right before its product
    // and waits out the LDS latency every time.
    constexpr int kOutProducts = 4 * kOut, kAll = kOutProducts + DIM / 8, kAhead = 6;
    v16f s[2];
    v8bf p[4] = {}, op[kAll];
    int k_slot = t0 % 3;  // of K of the tile about to be multiplied; V's is its number modulo 4
    auto operand = [&](int x, int t) {
      return x < kOutProducts ? F::v_operand(v_tile[(t - 1) & 3], x, lane)
                              : F::k_operand(k_tile[k_slot], x - kOutProducts, lane);
    };
    auto multiply = [&](auto first, int t) {
      constexpr int kFrom = decltype(first)::value ? kOutProducts : 0;
      uint8_t* k_to = k_tile[k_slot == 0 ? 2 : k_slot - 1];
      uint8_t* v_to = v_tile[(t + 2) & 3];
      // before the other team's vector work wherever both could issue (7.76 -> 7.40 ms)
      __builtin_amdgcn_s_setprio(1);
      s[0] = v16f{};
      s[1] = v16f{};
#pragma unroll
      for (int x = kFrom; x < kAll; ++x) {
        __builtin_amdgcn_sched_barrier(0);
        if (x < kOutProducts)
          r.o[x % kOut] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(op[x], p[x / kOut], r.o[x % kOut], 0, 0, 0);
        else
          s[x & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(op[x], r.q[(x - kOutProducts) / 2], s[x & 1], 0, 0, 0);
        if (x + kAhead < kAll) op[x + kAhead] = operand(x + kAhead, t);
        const int y = x - kOutProducts;  // by the score products, which every call has
        if (y == 0 || y == 1) f.leave_k(k_to, y);
        if (y == 2 || y == 3) f.leave_v(v_to, y - 2);
        if (y == 4) f.load(t + 3);
      }
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(0);
      k_slot = k_slot == 2 ? 0 : k_slot + 1;
    };

#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f.move(t0, t0 + u);
      f.load(t0 + u);
      f.clear(t0 + u);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f.leave_k(k_tile[(k_slot + u) % 3], h);
        f.leave_v(v_tile[(t0 + u) & 3], h);
      }
    }
    f.move(t0, t0 + 2);
    f.load(t0 + 2);
    f.clear(t0 + 2);
    f.move(t0, t0 + 3);
    phase_barrier();
    if (team == 1) phase_barrier();
#pragma unroll
    for (int x = 0; x < kAhead; ++x) op[kOutProducts + x] = operand(kOutProducts + x, t0);
    multiply(std::true_type{}, t0);
    for (int t = t0; t < t1; ++t) {
      phase_barrier();
      f.clear(t + 3);
      f.move(t, t + 4);
      tile_softmax<false>(a, f, r, s, p, t, t0, whole, pl.limit);
#pragma unroll
      for (int x = 0; x < kAhead; ++x) op[x] = operand(x, t + 1);
      phase_barrier();
      multiply(std::false_type{}, t + 1);  // past the last tile: scores of what stands there, unused
    }
    if (team == 0) phase_barrier();  // as many barriers as team 1
  }
  r.l += other_half(r.l);
  if (pl.there) store_rows<DIM>(a, r, pl.row_head, a.skip ? w.row0 : 0, part, lane >> 5);
}

// Few rows: tiles of 16 rows, whose NW wavefronts take the tokens' tiles in turn, straight
// from memory to registers (nothing is shared), and are joined in LDS at the end. The products
// run in 16 x 16 tiles, a lane holding row lane % 16 and 16 neighbouring tokens, those of its
// group lane / 16 of four: matrix row m of score tile 2 i + a is token 16 (m / 4) + 8 i + 4 a +
// m % 4, that of output tile b column (DIM / 4) (m / 4) + 4 b + m % 4. A load takes 64
// neighbouring bytes of 16 rows.
//
// HBM-bound with many requests: one token of 64 requests of up to 4096, 16 heads of 128 streams
// 684 MB in 126 us, 5.4 TB/s (a large copy: 5.0), the join 4 us more. With few, a chain of loads
// that need each other (offsets, page numbers, codes): one token of one request 7.3 us, its
// launch among them. K of the next tile is asked for before the softmax of this one, and V
// before the products of its scores; three workgroups to a CU cover the rest.
template <int DIM, int NW, bool SMALL>
__global__ __launch_bounds__(64 * NW, 3) void kv_attend_few(AttendArgs a) {
  constexpr int kChunks = DIM / 64;  // 16-byte chunks of a K row to a lane
  constexpr int kOut = DIM / 16;
  __shared__ float join_o[NW][64][DIM / 4 + 1];
  __shared__ float join_m[NW][64], join_l[NW][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, group = lane >> 4, half = lane >> 5;
  int slot, kv, part;
  place(a, slot, kv, part);
  Span w;
  if (!find_span<16>(a, slot, lane, w)) return;

  const int tiles = (w.seen + kTile - 1) / kTile;
  const int t0 = (int)((int64_t)tiles * part / a.parts), t1 = (int)((int64_t)tiles * (part + 1) / a.parts);
  const int whole = w.seen_first / kTile;
  const int64_t page_bytes = (int64_t)DIM << a.shift;
  const int32_t* row = a.table + (int64_t)w.req * a.table_pages;
  auto page_of = [&](int t) { return (t * kTile) >> a.shift; };

  Window now;
  int first = page_of(t0 + wave) & ~63;
  if (t0 + wave < t1) now.load_ids(a, row, w.seen, first, lane);

  // the rows, while the page numbers arrive
  const bool there = col < w.rows;
  const int packed = w.first + col;
  const int token = packed / a.group, head = kv * a.group + packed % a.group;
  const uint16_t* src_q = a.q.x + (w.row0 + token) * a.q.token + head * a.q.head + 16 * group;
  const int limit = !there ? 0 : a.causal ? min(w.seen, max(w.length - w.count + token + 1, 0)) : w.seen;
  v8bf q[2 * kChunks];
#pragma unroll
  for (int n = 0; n < 2 * kChunks; ++n)
    q[n] = __builtin_bit_cast(
        v8bf, there ? *reinterpret_cast<const uint4*>(src_q + 64 * (n >> 1) + 8 * (n & 1)) : make_uint4(0, 0, 0, 0));

  // this lane's places within a tile: K row and chunk, V row and chunk
  const int k_tok = 16 * (col >> 2) + (col & 3);                // + 8 i + 4 a
  const int k_up = k_tok >> 5;                                  // its page, where a tile spans two
  const uint32_t k_off = (SMALL ? k_tok & 31 : k_tok) * DIM + 16 * group;
  const uint32_t v_off = (((DIM / 4) * (col >> 2) + (col & 3)) << a.shift) + (SMALL ? 16 * (group & 1) : 16 * group);
  auto base_of = [&](int t, int up) {
    const int id = max(of_half<SMALL>(now.id, page_of(t) - first, up), 0);
    return ((int64_t)id * a.c.heads + kv) * page_bytes;
  };
  v4i k[4][kChunks], v[kOut];
  auto load_k = [&](int t) {
    const uint8_t* src = a.c.k + base_of(t, k_up) + (k_off + (a.shift == 7 ? (t & 1) * kTile * DIM : 0));
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int n = 0; n < kChunks; ++n) k[x][n] = *reinterpret_cast<const v4i*>(src + 4 * x * DIM + 64 * n);
  };
  auto load_v = [&](int t) {
    const uint8_t* src = a.c.v + base_of(t, half) + (v_off + (a.shift == 7 ? (t & 1) * kTile : 0));
#pragma unroll
    for (int b = 0; b < kOut; ++b) v[b] = *reinterpret_cast<const v4i*>(src + ((4 * b) << a.shift));
  };

  v4f o[kOut] = {};
  float m = kNone, l = 0.0f;
  if (t0 + wave < t1) {
    load_k(t0 + wave);
    now.load_scales(a, kv, page_bytes);
  }
  for (int t = t0 + wave; t < t1; t += NW) {
    load_v(t);
    v4f s[4] = {};
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int n = 0; n < kChunks; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          s[x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(k[x][n][2 * h], k[x][n][2 * h + 1]), q[2 * n + h], s[x], 0,
                                                         0, 0);
    const int i = page_of(t) - first;
    const int id = of_half<SMALL>(now.id, i, half);
    const bool some = t >= whole || unnamed<SMALL>(now.id, i);
    const float c = of_half<SMALL>(now.c, i, half);
    const float lv = of_half<SMALL>(now.lv, i, half), rv = of_half<SMALL>(now.rv, i, half);
    if (t + NW < t1) {
      if (page_of(t + NW) - first >= 64) {
        first = page_of(t + NW) & ~63;
        now.load_ids(a, row, w.seen, first, lane);
        load_k(t + NW);
        now.load_scales(a, kv, page_bytes);
      } else {
        load_k(t + NW);
      }
    }
    v8bf p[2];
    const int at = t * kTile + 16 * group;
    auto over = [](float x) {
      x = fmaxf(x, __shfl_xor(x, 16, 64));
      return fmaxf(x, __shfl_xor(x, 32, 64));
    };
    auto rescale = [&](float fix) {
#pragma unroll
      for (int b = 0; b < kOut; ++b) o[b] = o[b] * fix * fix;
    };
    if (some) {
      mask<16>(Tiles16{s}, id < 0 ? 0 : limit - at);
#pragma unroll
      for (int b = 0; b < kOut; ++b) {
        clear_past<4>(v[b], id < 0 ? 0 : w.seen - at);
        if (a.causal) clear_nan<4>(v[b]);
      }
    }
    softmax_step<16, true>(t == t0 + wave, Tiles16{s}, c, lv, rv, p, m, l, over, rescale);
#pragma unroll
    for (int b = 0; b < kOut; ++b)
#pragma unroll
      for (int n = 0; n < 2; ++n)
        o[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(v[b][2 * n], v[b][2 * n + 1]), p[n], o[b], 0, 0, 0);
  }
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);

  // Join the wavefronts: each leaves its O, bound and sum, and joins a share of the columns.
  join_m[wave][lane] = m;
  join_l[wave][lane] = l;
#pragma unroll
  for (int b = 0; b < kOut; ++b)
#pragma unroll
    for (int e = 0; e < 4; ++e) join_o[wave][lane][4 * b + e] = o[b][e];
  __syncthreads();
  if (!there) return;
  float top = kNone, sum = 0.0f, wt[NW];
#pragma unroll
  for (int x = 0; x < NW; ++x) top = fmaxf(top, join_m[x][lane]);
#pragma unroll
  for (int x = 0; x < NW; ++x) {
    wt[x] = root_power(join_m[x][lane] - top);
    sum += wt[x] * join_l[x][lane] * wt[x];
  }
  // a part leaves O as it is
  const float inv = a.parts > 1 ? 1.0f : sum > 0.0f ? 1.0f / sum : 0.0f;
  constexpr int kShare = DIM / 4 / NW;  // columns of a lane's DIM / 4
  const int64_t row_head = (int64_t)(w.row0 + token) * a.heads + head;
  const int column = (DIM / 4) * group + kShare * wave;
  float y[kShare];
#pragma unroll
  for (int e = 0; e < kShare; ++e) {
    float z = 0.0f;
#pragma unroll
    for (int x = 0; x < NW; ++x) z += wt[x] * join_o[x][lane][kShare * wave + e] * wt[x];
    y[e] = z * inv;
  }
  if (a.parts == 1) {
#pragma unroll
    for (int e = 0; e < kShare; e += 4)
      *reinterpret_cast<uint2*>(a.out + row_head * DIM + column + e) =
          make_uint2(pack_bf16x2(y[e], y[e + 1]), pack_bf16x2(y[e + 2], y[e + 3]));
    return;
  }
  const int64_t all = (int64_t)a.part_rows * a.heads;
#pragma unroll
  for (int e = 0; e < kShare; e += 4)
    *reinterpret_cast<float4*>(a.part_out + (part * all + row_head) * DIM + column + e) =
        make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
  if (group == 0 && wave == 0) {
    float* ml = a.part_out + a.parts * all * DIM + (part * all + row_head) * 2;
    ml[0] = top;
    ml[1] = sum;
  }
}

// The parts of each row and head joined: out = sum_i w_i O_i / sum_i w_i l_i, w_i = 2^(m_i - max m).
// (Of O_i / l_i and weights l_i 2^(m_i - max m) those under V scales of 2^100 would pass below fp32.)
// One wavefront per row and head, lane i holding the weight of part i (at most kMaxParts). Rows
// of no request, or of a skipped slot (the last tiles of the only request), were not written by
// any part and are left alone. Eight parts are on their way at a time: bound by the parts' way
// back from memory (1560 rows, 16 heads of 128, 2 parts: 12 us).
constexpr int kMaxParts = 64;
template <int DIM>
__global__ __launch_bounds__(256) void kv_attend_join(AttendArgs a, int row_shift) {
  constexpr int kCols = DIM / 64;
  typedef float Cols __attribute__((ext_vector_type(kCols)));
  const int lane = threadIdx.x & 63;
  const int64_t all = (int64_t)a.part_rows * a.heads;
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (i >= all) return;
  const float2 ml = lane < a.parts ? reinterpret_cast<const float2*>(a.part_out + a.parts * all * DIM)[lane * all + i]
                                   : make_float2(kNone, 0.0f);
  int row = (int)(i / a.heads);
  const int head = (int)(i % a.heads);
  if (a.skip) {
    const int begin = clamp_row(a.r.starts[0], a.r.rows), rows = max(0, clamp_row(a.r.starts[1], a.r.rows) - begin);
    const int64_t units = (int64_t)rows * a.group;
    const int64_t left = ((units + (1 << row_shift) - 1) >> row_shift) - a.skip;  // tiles
    if (row >= rows || ((int64_t)row * a.group + head % a.group) >> row_shift >= left) return;
    row += begin;
  } else {
    const Request q = request_of_slot<0>(a.r, 1, 0, row, lane, a.lengths);
    if (q.index < 0 || q.tile >= q.rows) return;
  }
  float m = ml.x, sum = 0.0f;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  const float wt = root_power(ml.x - m), wl = wt * ml.y * wt;
  const Cols* po = reinterpret_cast<const Cols*>(a.part_out + i * DIM) + lane;
  Cols o = {};
  for (int p0 = 0; p0 < a.parts; p0 += 8) {  // weights past the last part are zero
    Cols y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = po[min(p0 + j, a.parts - 1) * all * (DIM / kCols)];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float w = read_lane(wt, p0 + j);
      sum += read_lane(wl, p0 + j);
      o += w * y[j] * w;
    }
  }
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  uint16_t* out = a.out + ((int64_t)row * a.heads + head) * DIM + lane * kCols;
  if constexpr (DIM == 128) *reinterpret_cast<uint32_t*>(out) = pack_bf16x2(o[0] * inv, o[1] * inv);
  else *out = (uint16_t)pack_bf16x2(o[0] * inv, 0.0f);
}

template <int DIM, bool SMALL>
void launch(AttendArgs a, const AttendCut& x, hipStream_t stream) {
  auto attend = [&] {
    const int groups = a.c.heads * a.parts;
    int64_t most = 0;  // workgroups of an XCD
    for (int xcd = 0; xcd < kXcds; ++xcd) most = std::max(most, Deal(groups, a.slots).of_xcd(xcd));
    const dim3 grid((unsigned)(x.rows == 16 ? (int64_t)a.slots * groups : kXcds * most));
    if (x.rows == 16) kv_attend_few<DIM, 4, SMALL><<<grid, dim3(256), 0, stream>>>(a);
    else if constexpr (DIM == 64) kv_attend_tiles<DIM, SMALL><<<grid, dim3(Feed<DIM, SMALL>::kThreads), 0, stream>>>(a);
    else kv_attend_teams<DIM, SMALL><<<grid, dim3(Feed<DIM, SMALL>::kThreads), 0, stream>>>(a);
  };
  if (x.whole) {
    a.parts = 1;
    a.slots = (int)x.whole;
    attend();
    a.skip = (int)x.whole;
    a.parts = x.parts;
    a.slots = (int)(x.slots - x.whole);
  }
  attend();
  if (x.parts > 1) {
    const int64_t all = x.part_rows * a.heads;
    kv_attend_join<DIM><<<dim3((unsigned)((all + 3) / 4)), dim3(256), 0, stream>>>(a, x.shift);
  }
}

}  // namespace

AttendCut kv_attend_cut(const KvCache& c, int64_t requests, int64_t tokens, int64_t heads, int64_t table_pages, int cus) {
  const int group = (int)(heads / c.heads);
  const int64_t tiles = (table_pages * c.page_tokens + kTile - 1) / kTile;
  AttendCut x;
  // Up to 64 rows a request, some workgroups of 16 rows that each read its tokens are quicker than
  // one that shares them through LDS with most of its 128 or 256 rows empty (16 heads of 128 on up to
  // 4096 tokens: up to 32 rows of 32 requests 100 us against 179, 40 of 16 67 against 102, 60 of 16 78
  // against 106; of one request on 32760 tokens 24 rows 34 against 64, 64 55 against 68). The rule goes
  // by rows alone: it gives grids that do not fill the CUs to the larger tiles although the smaller
  // ones would be quicker there too (256 rows on 4096 27 us against 36; 1024 on 1024, 8 heads, 16
  // against 32).
  const bool few = tokens * group <= 64 * requests;
  x.rows = few ? 16 : kThreadRows(4 * c.head_dim);
  x.shift = __builtin_ctz(x.rows);
  x.slots = ragged_slots(tokens, requests, group, x.shift, 1);
  x.whole = 0;
  x.part_rows = tokens;
  // workgroups that will hold a tile: of several requests about half have a partly filled one
  const int64_t filled = requests == 1 ? (tokens * group + x.rows - 1) >> x.shift
                                       : (tokens * group >> x.shift) + (requests + 1) / 2;
  const int64_t busy = std::max<int64_t>(1, std::min(x.slots, few ? std::max(requests, filled) : filled)) * c.heads;
  if (few) {
    // A part for every CU as long as each of its wavefronts has two tiles (one token of one
    // request of 16 heads and 4096 tokens: 1 part 26.4 us, 8 11.8, 32 12.8; of 32760 tokens: 1 part
    // 187 us, 16 31.2, 24 34.4); requests of different lengths also even out over up to sixteen
    // workgroups to a CU of four tiles a wavefront (32 requests of up to 4096 tokens: 1 part 82.6
    // us, 4 72.9, 12 82.6; 64 requests: 138, 130.5 and 154).
    const int64_t spread = std::min<int64_t>(tiles / 8, cus / busy);
    const int64_t even = requests > 1 ? std::min<int64_t>(tiles / 16, 16 * (int64_t)cus / busy) : 1;
    x.parts = (int)std::min<int64_t>(std::max<int64_t>({1, spread, even}), kMaxParts);
    while (x.parts > 1 && !kv_attend_fits(c, x, tokens, heads)) --x.parts;
    return x;
  }
  // In tiles' time. Heads of 128: rounds of one workgroup to a CU, each its share of the tiles
  // and what it starts and ends with (about 6 tiles). Heads of 64: three to a CU, which
  // together get through 1.4 times what one does. And the join: 2 tiles and the parts' way out
  // and back. (1560 rows on 32760 tokens, 16 heads of 128: 1 part 740 us, 2 437, 4 450, 8 490; 256
  // rows on 4096: 99, 62, 42 and 35.5; 2000 rows on 2000 tokens, 16 heads of 64: 1 part 36 us, 2 47.)
  const int at_once = (c.head_dim == 64 ? 3 : 1) * cus;
  auto rounds = [&](int64_t units, int p) {
    const double one = (double)tiles / p + 6, wgs = (double)units * p, all = std::ceil(wgs / at_once) * one;
    return c.head_dim == 64 ? std::max(all, wgs * one / (1.4 * cus)) : all;
  };
  // Where the last round of whole workgroups would be far from full (one request, whose tiles
  // take alike), its rows are a second launch in parts (4680 rows on 4680 tokens, 16 heads of 128,
  // 304 workgroups: 252 -> 194 us).
  const int64_t full = requests == 1 ? busy / at_once * at_once / c.heads : 0;
  double best = 0;
  x.parts = 1;
  AttendCut y = x;
  for (int64_t whole : {(int64_t)0, full}) {
    const int64_t units = busy - whole * c.heads;
    const double before = whole ? rounds(whole * c.heads, 1) + 4 : 0;
    if (units <= 0 || (whole && whole >= x.slots)) continue;
    y.whole = whole;
    if (whole) y.part_rows = std::min(tokens, (((x.slots - whole) << x.shift) + group - 1) / group);
    for (int p = whole ? 2 : 1; p <= 32 && p <= std::max<int64_t>(1, tiles / 4); ++p) {
      const double rows = (double)units / busy * (double)tokens;
      const double join = p == 1 ? 0 : 2 + 1.3e-4 * p * rows * (double)heads;
      const double time = before + rounds(units, p) + join;
      y.parts = p;
      // parts never make a call too large that fits without
      if ((p == 1 && !whole) || (time < best && kv_attend_fits(c, y, tokens, heads))) {
        best = time;
        x = y;
      }
    }
  }
  return x;
}

size_t kv_attend_workspace_bytes(const KvCache& c, const AttendCut& x, int64_t heads) {
  return x.parts == 1 ? 0 : (size_t)x.parts * x.part_rows * heads * (c.head_dim + 2) * sizeof(float);
}

bool kv_attend_fits(const KvCache& c, const AttendCut& x, int64_t tokens, int64_t heads) {
  const int64_t most = (int64_t)1 << 23;  // workgroups of 512 threads in a grid
  // packed rows are counted in 32 bits
  return tokens * (heads / c.heads) < INT32_MAX - 128 && x.slots * c.heads * x.parts + 8 * kXcds < most &&
         (x.parts == 1 || (x.part_rows * heads + 3) / 4 < most);
}

hipError_t launch_kv_attend(const KvCache& c, const AttendCut& x, int64_t requests, int64_t tokens, int64_t heads,
                            const RowsIn& q, const int32_t* table, int64_t table_pages, const int32_t* lengths,
                            const int32_t* starts, float scale, bool causal, uint16_t* out, void* workspace,
                            hipStream_t stream) {
  const AttendArgs a{c,
                     {starts, (int)requests, (int)tokens},
                     q,
                     table,
                     lengths,
                     out,
                     static_cast<float*>(workspace),
                     (int)table_pages,
                     (int)heads,
                     (int)(heads / c.heads),
                     c.page_tokens == 32 ? 5 : c.page_tokens == 64 ? 6 : 7,
                     causal ? 1 : 0,
                     x.parts,
                     (int)x.slots,
                     0,
                     (int)x.part_rows,
                     scale};
  const bool small = c.page_tokens == 32;
  if (c.head_dim == 64) {
    if (small) launch<64, true>(a, x, stream);
    else launch<64, false>(a, x, stream);
  } else {
    if (small) launch<128, true>(a, x, stream);
    else launch<128, false>(a, x, stream);
  }
  return hipGetLastError();
}

}  // namespace fp8w8a8
