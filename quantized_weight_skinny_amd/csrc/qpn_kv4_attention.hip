// Attention of a verify step's rows over the 4-bit paged cache of
// include/qpn_decode.h.
//
// Mathematics. One kv head's query rows (rows of the sequence x query heads
// of the group) form 16-row tiles. A wavefront takes 32 tokens at a time and
// computes S^T = K Q^T (tokens x rows) and O^T += V^T P^T (elements x rows)
// with v_mfma_f32_16x16x32_f16, with p = 2^(s f - m), f = scale * log2(e) *
// k_scale, under a running reference m per row.
//
// Layouts that need no shuffle. Lane l = (i, g) = (l % 16, l / 16):
//  - K as the A operand of step c: token i, elements g * D/4 + 8c .. + 7: the
//    lane's D/8 bytes of the token's row are contiguous.
//  - the result of S^T: row (query) i, tokens 4g .. 4g + 3 of a 16-token half.
//  - P^T as the B operand: row i, contraction places 8g .. 8g + 7. Place
//    8g + j stands for token 4g + j of the first half (j < 4) and 4g + j - 4
//    of the second, so a lane's eight p are its own eight s.
//  - V^T as the A operand of block n: element i * D/16 + n at the same eight
//    tokens. The cache interleaves four tokens' D/16 elements, so the lane's
//    codes of four tokens are contiguous, and pairs of tokens are brought
//    together by swapping nibbles, before they are decoded.
//  - the result of O^T: row i, elements (4g + r) * D/16 + n: over n contiguous.
//
// E2M1 x E4M3 is exact in fp16, so fp16 rounds only q (bf16 rows are scaled
// by a power of two first: exact but for elements 2^-24 below their row's
// largest) and p. p is kept between 2^8 (at the reference) and 2^15: a row's
// reference moves only when a score passes it by 2^7, which a wavefront sees
// with one vote, and p as small as 2^-22 of the largest is a normal fp16.
#include "qpn_device.hpp"
#include "qpn_decode_internal.hpp"

namespace qpn {
namespace {

constexpr int kW = kAttnWaves;
constexpr float kNoToken = -1e30f;  // a row's reference before it has seen a token
constexpr float kBias = 8.0f, kHeadroom = 15.0f;

struct AttnParams {
  const uint8_t* cache;  // the layer
  int64_t page_bytes;
  int32_t pages, page_shift, seg_bytes, kv_heads, group;
  const void* q;
  int64_t q_ts, q_hs;
  void* out;
  float* lse;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* kv_len;
  const int32_t* q_start;
  int32_t batch, rows, max_q, max_kv, window, slots, min_chunk, q_aligned;
  int64_t max_units;
  float f, v_scale;  // f: scale * log2(e) * k_scale
  int4* sched;       // [batch]: first unit, splits, row tiles, -
  float* part;       // [unit][16 NQ][DIM], then [unit][16 NQ][2]
};

// One sequence's share of the work.
struct Seq {
  int len, qs, ql, lo, tiles, rt;  // tokens, first row, rows, first tile, tiles, row tiles
};

__device__ __forceinline__ Seq sequence(const AttnParams& a, int b, int rows_per_tile) {
  Seq s;
  s.len = min(max(a.kv_len[b], 0), a.max_kv);
  if (a.q_start) {
    s.qs = min(max(a.q_start[b], 0), a.rows);
    s.ql = min(min(max(a.q_start[b + 1] - s.qs, 0), a.max_q), a.rows - s.qs);
  } else {
    s.qs = b * a.max_q;
    s.ql = a.max_q;
  }
  // the first token that the sequence's first row sees
  const int first = a.window ? max(0, s.len - s.ql - a.window + 1) : 0;
  s.lo = first / kTileTokens;
  s.tiles = (s.len + kTileTokens - 1) / kTileTokens - s.lo;
  s.rt = (s.ql * a.group + rows_per_tile - 1) / rows_per_tile;
  return s;
}

__device__ __forceinline__ long long wave_sum(long long v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

// The codes and scales of 32 tokens as a lane holds them.
template <int DIM>
struct Tile {
  static constexpr int kWords = DIM / 32;  // dwords of codes a lane has of 16 tokens
  uint32_t k[2][kWords], v[2][kWords], ks[2], vs[2];
};

// A page's segment, read with raw buffer loads: its base and range and the
// place of a half in it sit in scalar registers, a lane's offsets do not
// change, so an address costs no vector instruction; and nothing past the
// segment can be read.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t segment_of(const uint8_t* seg, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(seg), 0, bytes, Stream::kRsrcWord3);
}

template <int WORDS>
__device__ __forceinline__ void load_words(uint32_t (&r)[WORDS], __amdgpu_buffer_rsrc_t seg, int lane_at, int at) {
  if constexpr (WORDS == 2) {
    const auto x = __builtin_amdgcn_raw_buffer_load_b64(seg, lane_at, at, Stream::kStreaming);
    r[0] = x[0], r[1] = x[1];
  } else {
#pragma unroll
    for (int j = 0; j < WORDS / 4; ++j) {
      const u4 x = __builtin_amdgcn_raw_buffer_load_b128(seg, lane_at + 16 * j, at, Stream::kStreaming);
#pragma unroll
      for (int e = 0; e < 4; ++e) r[4 * j + e] = x[e];
    }
  }
}

// Half `h` (16 tokens from offset `off` of a page's segment `seg`): the keys,
// and the values.
template <int DIM>
__device__ __forceinline__ void load_keys(Tile<DIM>& t, int h, __amdgpu_buffer_rsrc_t seg, int off, int page, int lane) {
  const int i = lane & 15, g = lane >> 4;
  load_words(t.k[h], seg, i * (DIM / 2) + g * (DIM / 8), off * (DIM / 2));
  const int lane_at = i * (DIM / 16) + g * (DIM / 64), at = page * DIM + off * (DIM / 16);
  if constexpr (DIM == 64)
    t.ks[h] = __builtin_amdgcn_raw_buffer_load_b8(seg, lane_at, at, Stream::kStreaming);
  else if constexpr (DIM == 128)
    t.ks[h] = __builtin_amdgcn_raw_buffer_load_b16(seg, lane_at, at, Stream::kStreaming);
  else
    t.ks[h] = __builtin_amdgcn_raw_buffer_load_b32(seg, lane_at, at, Stream::kStreaming);
}

template <int DIM>
__device__ __forceinline__ void load_vals(Tile<DIM>& t, int h, __amdgpu_buffer_rsrc_t seg, int off, int page, int lane) {
  const int i = lane & 15, g = lane >> 4;
  load_words(t.v[h], seg, lane_v<DIM>(i, g), page * (DIM / 2) + off * (DIM / 2));
  t.vs[h] = __builtin_amdgcn_raw_buffer_load_b32(seg, g * (DIM / 4) + (i * DIM / 256) * 4,
                                                 page * DIM + page * (DIM / 16) + off * (DIM / 16), Stream::kStreaming);
}

// The larger of three (two). The compiler's fmaxf first quiets each operand
// that it has not computed itself, an instruction each.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
__device__ __forceinline__ float max2(float a, float b) {
  float r;
  asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

__device__ __forceinline__ h2 splat(_Float16 x) { return h2{x, x}; }

// S^T of 32 tokens against the row tiles: step c of both halves meets each
// query fragment q(n, c) once.
template <int DIM, int NQ, typename Q>
__device__ __forceinline__ void scores(const Tile<DIM>& t, const Q& q, f4 (&s)[2][NQ]) {
  h2 sc[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    sc[h][0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(t.ks[h], 1.0f, false);
    if constexpr (DIM == 256) sc[h][1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(t.ks[h], 1.0f, true);
#pragma unroll
    for (int n = 0; n < NQ; ++n) s[h][n] = f4{0.f, 0.f, 0.f, 0.f};
  }
#pragma unroll
  for (int c = 0; c < DIM / 32; ++c) {
    const h8 k0 = decode_fp4x8(t.k[0][c], splat(sc[0][c / 4][(c / 2) & 1]));
    const h8 k1 = decode_fp4x8(t.k[1][c], splat(sc[1][c / 4][(c / 2) & 1]));
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const h8 x = q(n, c);
      s[0][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, x, s[0][n], 0, 0, 0);
      s[1][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, x, s[1][n], 0, 0, 0);
    }
  }
}

// Two dwords, x of even and y of odd elements: byte b holds element 2b (or
// 2b + 1) of two tokens.
__device__ __forceinline__ void pair_up(uint32_t a, uint32_t b, uint32_t& x, uint32_t& y) {
  constexpr uint32_t m = 0x0F0F0F0Fu;
  x = (a & m) | ((b << 4) & ~m);
  y = ((a >> 4) & m) | (b & ~m);
}

template <int I>
__device__ __forceinline__ h2 code_pair(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, I);
}

// Four elements' (2B, 2B + 1 of x and y: blocks n0 .. ) fragments and products.
template <int B, int NQ, int BLOCKS>
__device__ __forceinline__ void values_byte(const uint32_t (&x)[4], const uint32_t (&y)[4], const h2 (&sc)[4], int n0,
                                            const h8 (&p)[NQ], f4 (&o)[NQ][BLOCKS]) {
  const h8 even = cat(code_pair<B>(x[0]) * sc[0], code_pair<B>(x[1]) * sc[1], code_pair<B>(x[2]) * sc[2],
                      code_pair<B>(x[3]) * sc[3]);
  const h8 odd = cat(code_pair<B>(y[0]) * sc[0], code_pair<B>(y[1]) * sc[1], code_pair<B>(y[2]) * sc[2],
                     code_pair<B>(y[3]) * sc[3]);
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    o[n][n0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(even, p[n], o[n][n0], 0, 0, 0);
    o[n][n0 + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(odd, p[n], o[n][n0 + 1], 0, 0, 0);
  }
}

// O^T += V^T P^T over 32 tokens.
template <int DIM, int NQ>
__device__ __forceinline__ void values(const Tile<DIM>& t, const uint32_t (&vs)[2], const h8 (&p)[NQ],
                                       f4 (&o)[NQ][DIM / 16]) {
  h2 sc[4];  // tokens 0,1 and 2,3 of the lane's quad in each half
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    sc[2 * h] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(vs[h], 1.0f, false);
    sc[2 * h + 1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(vs[h], 1.0f, true);
  }
  uint32_t x[4], y[4];
  if constexpr (DIM == 64) {
    // a token has two bytes: dword 0 holds tokens 0 and 1, dword 1 tokens 2 and 3
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int d = 0; d < 2; ++d) pair_up(t.v[h][d], t.v[h][d] >> 16, x[2 * h + d], y[2 * h + d]);
    values_byte<0>(x, y, sc, 0, p, o);
    values_byte<1>(x, y, sc, 2, p, o);
  } else {
    constexpr int kTokenWords = DIM / 128;
#pragma unroll
    for (int w = 0; w < kTokenWords; ++w) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const auto word = [&](int tok) { return t.v[h][tok * kTokenWords + w]; };
        pair_up(word(0), word(1), x[2 * h], y[2 * h]);
        pair_up(word(2), word(3), x[2 * h + 1], y[2 * h + 1]);
      }
      values_byte<0>(x, y, sc, 8 * w, p, o);
      values_byte<1>(x, y, sc, 8 * w + 2, p, o);
      values_byte<2>(x, y, sc, 8 * w + 4, p, o);
      values_byte<3>(x, y, sc, 8 * w + 6, p, o);
    }
  }
}

// 8 consecutive outputs, rounded once to the type of q.
template <bool BF16>
__device__ __forceinline__ void store_out8(void* out, int64_t at, const float (&x)[8]) {
  u4 w;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = round16<BF16>(x[2 * j]) | static_cast<uint32_t>(round16<BF16>(x[2 * j + 1])) << 16;
  *reinterpret_cast<u4*>(static_cast<uint16_t*>(out) + at) = w;
}

// Wavefronts a SIMD is to hold: the output tiles and what a step needs fit
// 512 / waves registers (NQ * DIM / 4 of them for the output).
constexpr int waves_per_simd(int dim, int nq) {
  return dim == 256 || nq >= (dim == 64 ? 4 : 3) ? 2 : nq * dim <= 128 ? 4 : 3;
}

// Workgroup u takes unit u: of one sequence, a run of tiles, a row tile and a
// kv head. The units are counted out on the device from the lengths, so a
// captured call follows them: with `total` tiles to do over all sequences, row
// tiles and heads, a unit is max(min_chunk, ceil(total / slots)) tiles, and
// every sequence is cut into whole units. Heads run fastest (neighbouring
// workgroups read neighbouring segments of one page), then row tiles: with 8
// heads or a multiple, the row tiles that read the same tokens land on the same XCD.
template <int DIM, int NQ, bool BF16>
__global__ __launch_bounds__(kW * 64, waves_per_simd(DIM, NQ)) void kv4_attention_kernel(const AttnParams a) {
  constexpr int kRows = 16 * NQ, kBlocks = DIM / 16, kSteps = DIM / 32;
  constexpr int kPad = DIM + 4;
  constexpr bool kQueriesInLds = NQ * DIM > 128;
  union Shared {
    float red[kW][16][kPad];
    u4 q[kQueriesInLds ? NQ * kSteps * 64 : 1];
  };
  __shared__ Shared sh;
  __shared__ float2 ml[kW][kRows];
  __shared__ float fs[kRows];
  auto& red = sh.red;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int unit = blockIdx.x;

  // Which sequence, and how long a unit is.
  long long total = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    const int b = b0 + lane;
    if (b < a.batch) {
      const Seq s = sequence(a, b, kRows);
      total += static_cast<long long>(max(s.tiles, 1)) * s.rt;
    }
  }
  total = wave_sum(total) * a.kv_heads;
  // no sequence is longer than 2^30 tokens: a chunk that is cut there holds any
  // (the same in every lane: held in a scalar register, like all that follows from it)
  const int chunk = __builtin_amdgcn_readfirstlane(
      max(a.min_chunk, static_cast<int>(min((total + a.slots - 1) / a.slots, 1ll << 26))));
  int b = -1, base = 0, splits = 0;
  for (int b0 = 0, before = 0; b0 < a.batch; b0 += 64) {
    const int bl = b0 + lane;
    int n = 0, units = 0;
    if (bl < a.batch) {
      const Seq s = sequence(a, bl, kRows);
      n = max(1, (s.tiles + chunk - 1) / chunk);
      units = n * s.rt * a.kv_heads;
    }
    int sum = units;  // inclusive running sum over the lanes
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int x = __shfl_up(sum, o);
      if (lane >= o) sum += x;
    }
    const int first = before + sum - units;
    const unsigned long long hit = __ballot(unit >= first && unit < first + units);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      b = b0 + l;
      base = __builtin_amdgcn_readlane(first, l);
      splits = __builtin_amdgcn_readlane(n, l);
      break;
    }
    before += __builtin_amdgcn_readlane(sum, 63);
  }
  if (b < 0) return;  // the grid is the largest number of units
  b = __builtin_amdgcn_readfirstlane(b);
  const Seq s = sequence(a, b, kRows);
  int rest = unit - base;
  const int head = rest % a.kv_heads;
  rest /= a.kv_heads;
  const int rtile = rest % s.rt, split = rest / s.rt;
  if (rest == 0 && head == 0 && tid == 0) a.sched[b] = int4{base, splits, s.rt, 0};

  // The rows: row r of the row tile is query row r / group, head r % group.
  const int row0 = rtile * kRows, nrows = min(s.ql * a.group - row0, kRows);
  int pos[NQ];
  h8 qreg[kQueriesInLds ? 1 : NQ][kSteps];
  float f[NQ], m[NQ], l[NQ];
  f4 o[NQ][kBlocks];
  // one tile's fragments as a wavefront's lanes hold them, and its factor
  auto load_queries = [&](int n, h8 (&q)[kSteps]) {
    const int r = n * 16 + i;
    const int qi = (row0 + r) / a.group, hh = (row0 + r) - qi * a.group;
    const bool live = r < nrows;
    const int64_t at = static_cast<int64_t>(s.qs + (live ? qi : 0)) * a.q_ts +
                       static_cast<int64_t>(head * a.group + (live ? hh : 0)) * a.q_hs + g * (DIM / 4);
    uint16_t raw[DIM / 4];
    const uint16_t* src = static_cast<const uint16_t*>(a.q) + at;
    if (a.q_aligned) {
#pragma unroll
      for (int c = 0; c < kSteps; ++c) {
        const u4 x = *reinterpret_cast<const u4*>(src + c * 8);
#pragma unroll
        for (int e = 0; e < 8; ++e) raw[c * 8 + e] = static_cast<uint16_t>(x[e / 2] >> (16 * (e & 1)));
      }
    } else {
#pragma unroll
      for (int e = 0; e < DIM / 4; ++e) raw[e] = src[e];
    }
    float factor = a.f;
    if constexpr (BF16) {
      // a power of two that brings the row's largest magnitude to [1, 2)
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < DIM / 4; ++e) top = max(top, static_cast<uint32_t>(raw[e]) & 0x7FFFu);
      top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16)));
      top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32)));
      // (a row below 2^-60 by 2^60; inf and NaN stay themselves)
      const int e2 = min(max(static_cast<int>(top >> 7), 67), 252) - 127;
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
      factor = a.f * __uint_as_float(static_cast<uint32_t>(127 + e2) << 23);
#pragma unroll
      for (int e = 0; e < DIM / 4; ++e) {
        const float x = __uint_as_float(static_cast<uint32_t>(raw[e]) << 16);
        q[e / 8][e % 8] = live ? static_cast<_Float16>(x * down) : static_cast<_Float16>(0.f);
      }
    } else {
#pragma unroll
      for (int e = 0; e < DIM / 4; ++e)
        q[e / 8][e % 8] = live ? __builtin_bit_cast(_Float16, raw[e]) : static_cast<_Float16>(0.f);
    }
    return factor;
  };
  if constexpr (kQueriesInLds) {
    for (int n = wave; n < NQ; n += kW) {
      h8 q[kSteps];
      const float factor = load_queries(n, q);
#pragma unroll
      for (int c = 0; c < kSteps; ++c) sh.q[(n * kSteps + c) * 64 + lane] = __builtin_bit_cast(u4, q[c]);
      if (g == 0) fs[n * 16 + i] = factor;
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NQ; ++n) f[n] = fs[n * 16 + i];
  } else {
#pragma unroll
    for (int n = 0; n < NQ; ++n) f[n] = load_queries(n, qreg[n]);
  }
  const auto query = [&](int n, int c) -> h8 {
    if constexpr (kQueriesInLds)
      return __builtin_bit_cast(h8, sh.q[(n * kSteps + c) * 64 + lane]);
    else
      return qreg[n][c];
  };
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    pos[n] = s.len - s.ql + (row0 + n * 16 + i) / a.group;
    m[n] = kNoToken;
    l[n] = 0.f;
#pragma unroll
    for (int j = 0; j < kBlocks; ++j) o[n][j] = f4{0.f, 0.f, 0.f, 0.f};
  }

  // The unit's tiles, cut to what this row tile's rows see at all.
  const int first_pos = s.len - s.ql + row0 / a.group, last_pos = s.len - s.ql + (row0 + nrows - 1) / a.group;
  const int win = a.window;
  int t0 = s.lo + split * chunk, t1 = min(t0 + chunk, s.lo + s.tiles);
  t1 = min(t1, last_pos / kTileTokens + (last_pos >= 0));
  if (win) t0 = max(t0, max(0, first_pos - win + 1) / kTileTokens);
  const int mine = t1 > t0 + wave && a.pages > 0 ? (t1 - t0 - wave + kW - 1) / kW : 0;  // this wavefront's tiles
  const int page = 1 << a.page_shift;
  const int32_t* table = a.table + static_cast<int64_t>(b) * a.table_stride;
  const uint8_t* head_base = a.cache + static_cast<int64_t>(head) * a.seg_bytes;

  // Page indices of the wavefront's next 64 tiles, one lane each; -1: none.
  int pid[2] = {-1, -1};
  auto pages_from = [&](int j0) {
    const int j = j0 + lane;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int tok = (t0 + wave + j * kW) * kTileTokens + 16 * h;
      int p = -1;
      if (j < mine && tok < s.len) p = table[tok >> a.page_shift];
      pid[h] = p >= 0 && p < a.pages ? p : -1;
    }
  };
  // Keys and values of tile j, the pages having been looked up.
  Tile<DIM> t;
  int pg[2] = {-1, -1};   // the pages of the tile in hand
  const auto token_of = [&](int j) { return (t0 + wave + j * kW) * kTileTokens; };
  const auto segment = [&](int p) {
    return segment_of(head_base + static_cast<int64_t>(max(p, 0)) * a.page_bytes, a.seg_bytes);
  };
  auto look_up = [&](int (&next)[2], int j) {
    if ((j & 63) == 0) pages_from(j);
#pragma unroll
    for (int h = 0; h < 2; ++h) next[h] = __builtin_amdgcn_readlane(pid[h], j & 63);
  };
  auto keys = [&](const int (&p)[2], int j) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      load_keys<DIM>(t, h, segment(p[h]), (token_of(j) + 16 * h) & (page - 1), page, lane);
  };
  auto vals = [&](const int (&p)[2], int j) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      load_vals<DIM>(t, h, segment(p[h]), (token_of(j) + 16 * h) & (page - 1), page, lane);
  };
  if (mine > 0) {
    look_up(pg, 0);
    keys(pg, 0);
    vals(pg, 0);
  }
  // The keys of the next tile are on their way during this one's softmax and
  // values, its values during the next one's scores: one set of registers
  // each, and the other wavefronts of the SIMD to fill what is left.
  for (int j = 0; j < mine; ++j) {
    const int tok = token_of(j);
    f4 sc[2][NQ];
    scores<DIM, NQ>(t, query, sc);
    __builtin_amdgcn_sched_barrier(0);
    int next[2] = {-1, -1};
    if (j + 1 < mine) {
      look_up(next, j + 1);
      keys(next, j + 1);
    }
    __builtin_amdgcn_sched_barrier(0);
    uint32_t vs[2] = {t.vs[0], t.vs[1]};
    const bool whole =
        tok + kTileTokens - 1 <= first_pos && (win == 0 || tok > last_pos - win) && pg[0] >= 0 && pg[1] >= 0;
    if (!whole) {
      // Scores of unseen tokens become -inf whatever the cache holds there,
      // and the values of tokens past the end or of absent pages are zeroed:
      // such bytes may decode to NaN, which a p of 0 would not remove. Bit b
      // of a mask stands for token tok + 4 g + b.
      const int at = tok + 4 * g;
      const auto up_to = [](int x) -> uint32_t { return x < 0 ? 0u : x >= 31 ? ~0u : (2u << x) - 1u; };
      const uint32_t held = up_to(s.len - 1 - at) & ((pg[0] >= 0 ? 0xFFFFu : 0u) | (pg[1] >= 0 ? 0xFFFF0000u : 0u));
      const auto bit = [](uint32_t w, int b) { return static_cast<uint32_t>(static_cast<int32_t>(w << (31 - b)) >> 31); };
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) vs[h] &= ~(0xFFu << (8 * e)) | bit(held, 16 * h + e);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const uint32_t seen = held & up_to(pos[n] - at) & (win ? ~up_to(pos[n] - win - at) : ~0u);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t k = bit(seen, 16 * h + e);
            sc[h][n][e] = __uint_as_float((__float_as_uint(sc[h][n][e]) & k) | (0xFF800000u & ~k));
          }
      }
    }
    float far = -__builtin_inff();
    float top[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      top[n] = max3(max3(sc[0][n][0], sc[0][n][1], sc[0][n][2]), sc[0][n][3], sc[1][n][0]);
      top[n] = max2(max3(top[n], sc[1][n][1], sc[1][n][2]), sc[1][n][3]);
      far = max2(far, fmaf(top[n], f[n], -m[n]));
    }
    if (__any(far > kHeadroom)) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float mx = fmaxf(m[n], fmaf(top[n], f[n], -kBias));
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float down = __builtin_amdgcn_exp2f(m[n] - mx);
        m[n] = mx;
        l[n] *= down;
#pragma unroll
        for (int d = 0; d < kBlocks; ++d) o[n][d] *= down;
      }
    }
    h8 p[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // (the sum takes p before it is rounded: lse keeps its 32 bits)
        const float x = __builtin_amdgcn_exp2f(fmaf(sc[e / 4][n][e % 4], f[n], -m[n]));
        l[n] += x;
        p[n][e] = static_cast<_Float16>(x);
      }
    }
    values<DIM, NQ>(t, vs, p, o);
    __builtin_amdgcn_sched_barrier(0);
    if (j + 1 < mine) vals(next, j + 1);
    __builtin_amdgcn_sched_barrier(0);
    pg[0] = next[0], pg[1] = next[1];
  }

  // Join the wavefronts: a row's reference becomes the largest of the four.
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    l[n] += __shfl_xor(l[n], 16);
    l[n] += __shfl_xor(l[n], 32);
    if (g == 0) ml[wave][n * 16 + i] = float2{m[n], l[n]};
  }
  __syncthreads();
  const int64_t part_rows = static_cast<int64_t>(unit) * kRows;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    float mx = ml[0][n * 16 + i].x;
#pragma unroll
    for (int w = 1; w < kW; ++w) mx = fmaxf(mx, ml[w][n * 16 + i].x);
    const float down = __builtin_amdgcn_exp2f(m[n] - mx);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int d = 0; d < kBlocks; d += 4)
        *reinterpret_cast<f4*>(&red[wave][i][(g * 4 + r) * kBlocks + d]) =
            f4{o[n][d][r] * down, o[n][d + 1][r] * down, o[n][d + 2][r] * down, o[n][d + 3][r] * down};
    __syncthreads();
    // 8 elements a thread
#pragma unroll
    for (int x = tid; x < 16 * DIM / 8; x += kW * 64) {
      const int r = x / (DIM / 8), d = x % (DIM / 8) * 8, row = n * 16 + r;
      if (row < nrows) {
        float mr = ml[0][row].x;
#pragma unroll
        for (int w = 1; w < kW; ++w) mr = fmaxf(mr, ml[w][row].x);
        float lr = 0.f;
#pragma unroll
        for (int w = 0; w < kW; ++w) lr += ml[w][row].y * __builtin_amdgcn_exp2f(ml[w][row].x - mr);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[e] = red[0][r][d + e];
#pragma unroll
          for (int w = 1; w < kW; ++w) v[e] += red[w][r][d + e];
        }
        if (splits > 1) {
          float* dst = a.part + (part_rows + row) * DIM + d;
          *reinterpret_cast<f4*>(dst) = f4{v[0], v[1], v[2], v[3]};
          *reinterpret_cast<f4*>(dst + 4) = f4{v[4], v[5], v[6], v[7]};
          if (d == 0) {
            float2* mld = reinterpret_cast<float2*>(a.part + a.max_units * kRows * DIM);
            mld[part_rows + row] = float2{mr, lr};
          }
        } else {
          const int qi = (row0 + row) / a.group, hh = (row0 + row) - qi * a.group;
          const int64_t at = static_cast<int64_t>(s.qs + qi) * (a.kv_heads * a.group) + head * a.group + hh;
          const float up = lr > 0.f ? a.v_scale / lr : (lr == 0.f ? 0.f : lr);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= up;
          store_out8<BF16>(a.out, at * DIM + d, v);
          if (d == 0 && a.lse)
            a.lse[at] = lr == 0.f ? -__builtin_inff() : (__builtin_amdgcn_logf(lr) + mr) * 0.69314718055994531f;
        }
      }
    }
    __syncthreads();
  }
}

// Joins the units of the sequences that were cut: one wavefront a (row, query
// head), in the order of the units.
template <int DIM, bool BF16>
__global__ __launch_bounds__(256) void kv4_attention_join_kernel(const AttnParams a, int unit_rows) {
  constexpr int kPer = 8, kLanes = DIM / kPer;  // lanes that hold a row; the others take other units
  constexpr int kGroups = 64 / kLanes;
  const int lane = threadIdx.x & 63;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int heads = a.kv_heads * a.group;
  if (id >= static_cast<int64_t>(a.rows) * heads) return;
  const int row = static_cast<int>(id / heads), head = static_cast<int>(id - static_cast<int64_t>(row) * heads);
  int b, qs;
  if (a.q_start) {
    // the last sequence that starts at or before the row
    int lo = 0, hi = a.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (a.q_start[mid] <= row) lo = mid;
      else hi = mid - 1;
    }
    b = lo;
    qs = a.q_start[b];
    if (row < qs || row - qs >= a.max_q || row >= a.q_start[b + 1]) return;  // a row of no sequence
  } else {
    b = row / a.max_q;
    qs = b * a.max_q;
  }
  const int4 sc = a.sched[b];
  if (sc.y <= 1) return;  // written by its only unit
  const int r = (row - qs) * a.group + head % a.group;
  const int rtile = r / unit_rows;
  const int step = sc.z * a.kv_heads;
  const int64_t first = sc.x + rtile * a.kv_heads + head / a.group;
  const float2* ml = reinterpret_cast<const float2*>(a.part + a.max_units * unit_rows * DIM) + r % unit_rows;
  float mx = kNoToken;
  for (int s = lane; s < sc.y; s += 64) mx = fmaxf(mx, ml[(first + static_cast<int64_t>(s) * step) * unit_rows].x);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
  float l = 0.f, v[kPer] = {};
  const int gr = lane / kLanes, d = lane % kLanes * kPer;
#pragma unroll 4
  for (int s = gr; s < sc.y; s += kGroups) {
    const int64_t at = (first + static_cast<int64_t>(s) * step) * unit_rows;
    const float2 x = ml[at];
    const float* src = a.part + (at + r % unit_rows) * DIM + d;
    const f4 v0 = *reinterpret_cast<const f4*>(src), v1 = *reinterpret_cast<const f4*>(src + 4);
    const float w = __builtin_amdgcn_exp2f(x.x - mx);
    l += w * x.y;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] += w * v0[e];
      v[4 + e] += w * v1[e];
    }
  }
#pragma unroll
  for (int o = kLanes; o < 64; o <<= 1) {
    l += __shfl_xor(l, o);
#pragma unroll
    for (int e = 0; e < kPer; ++e) v[e] += __shfl_xor(v[e], o);
  }
  if (gr != 0) return;
  const float up = l > 0.f ? a.v_scale / l : (l == 0.f ? 0.f : l);
#pragma unroll
  for (int e = 0; e < kPer; ++e) v[e] *= up;
  store_out8<BF16>(a.out, id * DIM + d, v);
  if (d == 0 && a.lse)
    a.lse[id] = l == 0.f ? -__builtin_inff() : (__builtin_amdgcn_logf(l) + mx) * 0.69314718055994531f;
}

template <int DIM, int NQ, bool BF16>
hipError_t launch_as(const AttnParams& a, hipStream_t stream) {
  kv4_attention_kernel<DIM, NQ, BF16><<<dim3(static_cast<uint32_t>(a.max_units)), dim3(kW * 64), 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // a sequence of at most min_chunk tiles is one unit
  if (a.max_kv <= a.min_chunk * kTileTokens) return hipSuccess;
  const int64_t heads = static_cast<int64_t>(a.rows) * a.kv_heads * a.group;
  kv4_attention_join_kernel<DIM, BF16>
      <<<dim3(static_cast<uint32_t>((heads + 3) / 4)), dim3(256), 0, stream>>>(a, 16 * NQ);
  return hipGetLastError();
}

template <int DIM, bool BF16>
hipError_t launch_nq(int nq, const AttnParams& a, hipStream_t stream) {
  switch (nq) {
    case 1: return launch_as<DIM, 1, BF16>(a, stream);
    case 2: return launch_as<DIM, 2, BF16>(a, stream);
    default: break;
  }
  if constexpr (DIM != 256)
    if (nq == 3) return launch_as<DIM, 3, BF16>(a, stream);
  if constexpr (DIM == 64)
    if (nq == 4) return launch_as<DIM, 4, BF16>(a, stream);
  return hipErrorInvalidValue;
}

template <bool BF16>
hipError_t launch_dim(int dim, int nq, const AttnParams& a, hipStream_t stream) {
  switch (dim) {
    case 64: return launch_nq<64, BF16>(nq, a, stream);
    case 128: return launch_nq<128, BF16>(nq, a, stream);
    case 256: return launch_nq<256, BF16>(nq, a, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_kv4_attention(const qpn_kv4_cache& c, const qpn_kv4_attention_args& x, const AttentionPlan& p,
                                void* workspace, hipStream_t stream) {
  AttnParams a;
  a.page_bytes = static_cast<int64_t>(qpn_kv4_page_bytes(c.page_size, c.kv_heads, c.head_dim));
  a.cache = static_cast<const uint8_t*>(c.data) + a.page_bytes * c.pages * x.layer;
  a.pages = static_cast<int32_t>(c.pages);
  a.page_shift = __builtin_ctz(c.page_size);
  a.seg_bytes = static_cast<int32_t>(kv4_segment_bytes(c.page_size, c.head_dim));
  a.kv_heads = c.kv_heads;
  a.group = x.heads / c.kv_heads;
  a.q = x.q, a.q_ts = x.q_token_stride, a.q_hs = x.q_head_stride;
  a.q_aligned = reinterpret_cast<uintptr_t>(x.q) % 16 == 0 && x.q_token_stride % 8 == 0 && x.q_head_stride % 8 == 0;
  a.out = x.out, a.lse = x.lse;
  a.table = x.table, a.table_stride = x.table_stride;
  a.kv_len = x.kv_len, a.q_start = x.q_start;
  a.batch = x.batch, a.rows = x.rows, a.max_q = x.max_q_len < x.rows ? x.max_q_len : x.rows;
  a.max_kv = x.max_kv_len, a.window = x.window;
  a.slots = p.slots, a.min_chunk = p.min_chunk, a.max_units = p.max_units;
  a.f = x.scale * 1.44269504088896341f * c.k_scale;
  a.v_scale = c.v_scale;
  a.sched = static_cast<int4*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + p.sched_bytes);
  return x.dtype == QPN_DT_BF16 ? launch_dim<true>(c.head_dim, p.tiles16, a, stream)
                                : launch_dim<false>(c.head_dim, p.tiles16, a, stream);
}

}  // namespace qpn
