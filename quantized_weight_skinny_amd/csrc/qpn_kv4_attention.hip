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
// E2M1 x E4M3 is exact in fp16, so fp16 rounds only q (bf16 rows are scaled by
// a power of two first, their largest to 2^15: all eight bits of an element
// stay down to 2^-32 of its row's largest, and what a smaller one loses is at
// most 2^-40 of that) and p. p is kept between 2^8 (at the reference) and 2^15: a row's
// reference moves only when a score passes it by 2^7, which a wavefront sees
// with one vote, and p as small as 2^-22 of the largest is a normal fp16.
//
// What bounds it. For 32 tokens of 128 elements the codes take 64 conversions
// and 64 multiplications (the conversion's own scale is a power of two, the
// blocks' are not) and 16 instructions to pair V's; every row tile adds 8
// exponentials at two slots each, 24 adds and multiply-adds, 4 conversions, 6
// for the maximum and 16 MFMAs. At three row tiles (8 rows of 5 heads) the
// counters give 364 vector instructions a tile, all of the kernel's, that issue for
// 1570 cycles; the loop takes 1810 cycles a tile and SIMD, with two wavefronts,
// which a SIMD needs: one alone issues a vector instruction every 8 cycles, two
// or more every 4 to 5. So 131072 tokens of 8 heads (151 MB) take 26 us of vector
// instructions against 25 us of memory, and the call 46: the loop is 30 of it,
// the rest the launch (1 to 2), the shares' counting (3), first loads (3), joining
// wavefronts (4) and pieces (6). At one row tile (one row, four wavefronts a
// SIMD) 24 sequences' 180 MB take 39 us.
#include <algorithm>

#include "qpn_device.hpp"
#include "qpn_decode_internal.hpp"

namespace qpn {
namespace {

constexpr int kW = kAttnWaves;
constexpr float kNoToken = -1e30f;  // a row's reference before it has seen a token
constexpr float kBias = 8.0f, kHeadroom = 15.0f;
constexpr float kLeast = 1.17549435e-38f, kMost = 3.40282347e+38f;  // fp32's normal range
// What a run costs besides its tiles, in tiles: its queries, the first loads'
// latency and the joining of the wavefronts (4 to 6 us where a tile takes 0.2
// to 0.4). 48 ragged sequences 127 us with 0, 87 with 12, 81 with 20.
constexpr int kRunCost = 20;

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
  int32_t batch, rows, max_q, max_kv, window, row_tiles, groups, min_share, q_aligned;
  float f, v_scale;  // f: scale * log2(e) * k_scale
  struct Cut* cuts;  // [groups]; groups 0: no join
  float* part;       // [2 groups][16 NQ][DIM], then [2 groups][16 NQ][2]
};

// The run that a workgroup's share begins inside of (rows 0: it begins with
// one): its pieces are those of workgroups first .. last, its rows `rows` of
// kv head `head`'s from row `row0` of the sequence whose rows begin at `qs`.
struct Cut {
  int rows, first, last, qs, row0, head, pad[2];
};
static_assert(sizeof(Cut) == 32, "the workspace holds 32 bytes a workgroup");

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
  s.tiles = max(1, (s.len + kTileTokens - 1) / kTileTokens - s.lo);  // an empty sequence is one tile that holds nothing
  s.rt = (s.ql * a.group + rows_per_tile - 1) / rows_per_tile;
  return s;
}

// Lane l's sequence, in scalar registers.
__device__ __forceinline__ Seq lane_of(const Seq& s, int l) {
  const auto get = [&](int x) { return __builtin_amdgcn_readlane(x, l); };
  return Seq{get(s.len), get(s.qs), get(s.ql), get(s.lo), get(s.tiles), get(s.rt)};
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

// A lane's byte offsets in a segment's four arrays.
template <int DIM>
struct LaneOffsets {
  int k, v, ks, vs;
  __device__ __forceinline__ LaneOffsets(int lane, int page) {
    const int i = lane & 15, g = lane >> 4;
    k = i * (DIM / 2) + g * (DIM / 8);
    v = page * (DIM / 2) + lane_v<DIM>(i, g);
    ks = page * DIM + i * (DIM / 16) + g * (DIM / 64);
    vs = page * DIM + page * (DIM / 16) + g * (DIM / 4) + (i * DIM / 256) * 4;
  }
};

// Half `h` (16 tokens), whose codes begin `codes` and whose scales begin
// `scales` bytes into their arrays: the keys, and the values.
template <int DIM>
__device__ __forceinline__ void load_keys(Tile<DIM>& t, int h, __amdgpu_buffer_rsrc_t seg, const LaneOffsets<DIM>& at,
                                          int codes, int scales) {
  load_words(t.k[h], seg, at.k, codes);
  if constexpr (DIM == 64)
    t.ks[h] = __builtin_amdgcn_raw_buffer_load_b8(seg, at.ks, scales, Stream::kStreaming);
  else if constexpr (DIM == 128)
    t.ks[h] = __builtin_amdgcn_raw_buffer_load_b16(seg, at.ks, scales, Stream::kStreaming);
  else
    t.ks[h] = __builtin_amdgcn_raw_buffer_load_b32(seg, at.ks, scales, Stream::kStreaming);
}

template <int DIM>
__device__ __forceinline__ void load_vals(Tile<DIM>& t, int h, __amdgpu_buffer_rsrc_t seg, const LaneOffsets<DIM>& at,
                                          int codes, int scales) {
  load_words(t.v[h], seg, at.v, codes);
  t.vs[h] = __builtin_amdgcn_raw_buffer_load_b32(seg, at.vs, scales, Stream::kStreaming);
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

// The kernel's arguments, to be read again from where they lie.
typedef const AttnParams __attribute__((address_space(4))) * ParamsPtr;
__device__ __forceinline__ const AttnParams& reread(const AttnParams&) {
  ParamsPtr p = (ParamsPtr)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const AttnParams*)p;
}

// The work is the tiles of all (sequence, row tile, kv head), laid end to end
// in that order. Where a sequence may be long, each of `groups` workgroups (as
// many as the device holds at once) takes an equal share of that line, at
// least min_share tiles, whatever the lengths: a share may begin inside one
// run of tiles and end inside another. A run that lies in one share is
// written as it is; the pieces of any other go to the workspace, at most two a
// workgroup (the end of a run in slot 2 w, the beginning of one in slot
// 2 w + 1), and the join kernel adds them. The line is measured out on the
// device from the lengths, so a captured call follows them. Where every
// sequence is short (groups 0), a workgroup takes a run, and no length but its
// own matters.
template <int DIM, int NQ, bool BF16>
__global__ __launch_bounds__(kW * 64, attn_waves_per_simd(DIM, NQ)) void kv4_attention_kernel(const AttnParams params) {

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
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  int tid = threadIdx.x, lane = tid & 63;
  const int group_id = blockIdx.x;

  const AttnParams& a0 = params;
  // This workgroup's share [at, end) of the line, and the sequence b, whose
  // tiles begin at `base`, that the share begins in.
  int b = 0, base = 0, at, end, share = 0;
  Seq seq = {0, 0, 0, 0, 0, 0};
  if (a0.groups == 0) {
    const int per = a0.row_tiles * a0.kv_heads;
    b = group_id / per;
    seq = sequence(a0, b, kRows);
    at = (group_id - b * per) * (seq.tiles + kRunCost);
    end = at + seq.tiles + kRunCost;
    if (at >= seq.rt * a0.kv_heads * (seq.tiles + kRunCost)) return;  // fewer row tiles than the longest has
  } else {
    int total = 0;
    // of the last 64 sequences: a lane's, its part of the line, and the running sum
    Seq lanes = {0, 0, 0, 0, 0, 0};
    int mine = 0, sum = 0;
    const auto count = [&](int b0) {
      mine = 0;
      if (b0 + lane < a0.batch) {
        lanes = sequence(a0, b0 + lane, kRows);
        mine = (lanes.tiles + kRunCost) * lanes.rt * a0.kv_heads;
      }
      sum = mine;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int x = __shfl_up(sum, o);
        if (lane >= o) sum += x;
      }
    };
    for (int b0 = 0; b0 < a0.batch; b0 += 64) {
      count(b0);
      total += __builtin_amdgcn_readlane(sum, 63);
    }
    share = max(a0.min_share, (total + a0.groups - 1) / a0.groups);
    at = group_id * share;  // groups * share is at most 2^31 - 1, as the line is
    end = min(at + share, total);
    if (at >= total) {
      if (tid == 0) a0.cuts[group_id].rows = 0;
      return;
    }
    int before = 0;
    for (int b0 = 0; b0 < a0.batch; b0 += 64) {
      if (a0.batch > 64) count(b0);
      const int all = __builtin_amdgcn_readlane(sum, 63);
      if (at < before + all) {
        const int l = __builtin_ctzll(__ballot(at < before + sum));
        b = b0 + l;
        base = before + __builtin_amdgcn_readlane(sum, l) - __builtin_amdgcn_readlane(mine, l);
        seq = lane_of(lanes, l);
        break;
      }
      before += all;
    }
  }
  bool first_run = true;
  while (true) {
    // (what follows from the lane is worked out again for every run: kept from
    // one to the next it would take registers that the occupancy needs;
    // and so are the arguments, which come from the scalar cache)
    asm volatile("" : "+v"(tid), "+v"(lane));
    const AttnParams& a = reread(params);
    const int i = lane & 15, g = lane >> 4;
    const Seq s = seq;
    const int cost = s.tiles + kRunCost;
    const int run = (at - base) / cost, from = at - base - run * cost, to = min(cost, from + end - at);
    const int tile0 = max(0, from - kRunCost), tiles = max(0, to - kRunCost) - tile0;
    at += to - from;
    const int rtile = run / a.kv_heads, head = run - rtile * a.kv_heads;
    const bool alone = tiles == s.tiles;  // the whole run
    // The rows: row r of the row tile is query row r / group, head r % group.
    const int row0 = rtile * kRows, nrows = min(s.ql * a.group - row0, kRows);
    if (first_run && a.groups && tid == 0) {
      // where this run's first tile and its last lie on the line
      const int begin = base + run * cost + kRunCost;
      a.cuts[group_id] = Cut{tile0 > 0 ? nrows : 0, begin / share, (begin + s.tiles - 1) / share, s.qs, row0, head,
                             {0, 0}};
    }
    first_run = false;
    if (tiles > 0) {
      h8 qreg[kQueriesInLds ? 1 : NQ][kSteps];
      float f[NQ], m[NQ], l[NQ];
      f4 o[NQ][kBlocks];
      // Row tile n's queries as a wavefront's lanes hold them: a lane's part of its
      // row in memory, eight elements of it as they lie there, and as a fragment.
      const auto row_of = [&](int n) {
        const int r = n * 16 + i;
        const int qi = (row0 + r) / a.group, hh = (row0 + r) - qi * a.group;
        const bool live = r < nrows;  // (a row past the last loads the first)
        const int64_t row_at = static_cast<int64_t>(s.qs + (live ? qi : 0)) * a.q_ts +
                               static_cast<int64_t>(head * a.group + (live ? hh : 0)) * a.q_hs + g * (DIM / 4);
        return static_cast<const uint16_t*>(a.q) + row_at;
      };
      const auto eight = [&](const uint16_t* src, int c) {
        u4 x;
        if (a.q_aligned) {
          x = *reinterpret_cast<const u4*>(src + c * 8);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = src[c * 8 + 2 * e] | static_cast<uint32_t>(src[c * 8 + 2 * e + 1]) << 16;
        }
        return x;
      };
      // bf16: the exponent (a row below 2^-111 takes that of 2^-111; inf and NaN stay
      // themselves) less which a row's largest magnitude is in [2^15, 2^16): the
      // top of fp16, whose smallest step is then 2^-39 of it.
      const auto larger = [](uint32_t top, const u4& x) {
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(max(top, x[e] & 0x7FFFu), (x[e] >> 16) & 0x7FFFu);
        return top;
      };
      const auto exponent = [](uint32_t top) {
        top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16)));
        top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32)));
        return min(max(static_cast<int>(top >> 7), 16), 254) - (127 + 15);
      };
      const auto fragment = [&](int n, u4 x, int e2) {
        if (n * 16 + i >= nrows) x = u4{0u, 0u, 0u, 0u};
        if constexpr (BF16) {
          const float down = __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
          h8 q;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            q[2 * e] = static_cast<_Float16>(__uint_as_float(x[e] << 16) * down);
            q[2 * e + 1] = static_cast<_Float16>(__uint_as_float(x[e] & 0xFFFF0000u) * down);
          }
          return q;
        } else {
          return __builtin_bit_cast(h8, x);
        }
      };
      // (kept in fp32's normal range: 0 or inf times a score, -inf or 0, would be NaN. Products of
      // queries and codes are below 2^36, so that the least normal factor makes them all as good as 0.)
      const auto factor = [&](int e2) {
        if constexpr (!BF16) return a.f;
        return fminf(fmaxf(a.f * __uint_as_float(static_cast<uint32_t>(127 + e2) << 23), kLeast), kMost);
      };
      // They are asked for before the first keys and values and made into
      // fragments while those come; in LDS, wavefront n does tile n for all four.
      // Two tiles (of 128 at three wavefronts a SIMD, of 256) would have too many
      // registers on the way (made as the others the compiler spills 8 of 168 at
      // 128 in bf16 and 16 of 256 at 256): those queries come first, eight elements
      // at a time, bf16 rows twice, and the first keys wait for them.
      static_assert(NQ <= kW, "a wavefront prepares one tile");
      constexpr bool kQueriesFirst = NQ == 2 && DIM >= 128;
      u4 raw[kQueriesFirst ? 1 : kQueriesInLds ? 1 : NQ][kQueriesFirst ? 1 : kSteps];
      if constexpr (kQueriesFirst) {
        if (wave < NQ) {
          const uint16_t* src = row_of(wave);
          int e2 = 0;
          if constexpr (BF16) {
            uint32_t top = 0;
#pragma unroll 1
            for (int c = 0; c < kSteps; ++c) top = larger(top, eight(src, c));
            e2 = exponent(top);
          }
#pragma unroll 1
          for (int c = 0; c < kSteps; ++c)
            sh.q[(wave * kSteps + c) * 64 + lane] = __builtin_bit_cast(u4, fragment(wave, eight(src, c), e2));
          if (g == 0) fs[wave * 16 + i] = factor(e2);
        }
      } else if constexpr (kQueriesInLds) {
        if (wave < NQ) {
          const uint16_t* src = row_of(wave);
#pragma unroll
          for (int c = 0; c < kSteps; ++c) raw[0][c] = eight(src, c);
        }
      } else {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          const uint16_t* src = row_of(n);
#pragma unroll
          for (int c = 0; c < kSteps; ++c) raw[n][c] = eight(src, c);
        }
      }

      // The tiles in hand, cut to what this row tile's rows see at all.
      const int first_pos = s.len - s.ql + row0 / a.group, last_pos = s.len - s.ql + (row0 + nrows - 1) / a.group;
      const int win = a.window;
      int t0 = s.lo + tile0, t1 = t0 + tiles;
      t1 = min(t1, last_pos / kTileTokens + (last_pos >= 0));
      if (win) t0 = max(t0, max(0, first_pos - win + 1) / kTileTokens);
      const int mine = t1 > t0 + wave && a.pages > 0 ? (t1 - t0 - wave + kW - 1) / kW : 0;  // this wavefront's tiles
      const int page = 1 << a.page_shift;
      const int32_t* table = a.table + static_cast<int64_t>(b) * a.table_stride;
      const uint8_t* head_base = a.cache + static_cast<int64_t>(head) * a.seg_bytes;

      // The page segments of the wavefront's next 64 tiles, a lane each, and which
      // of their halves have none. A half's loads take their base from here and
      // their place in the page from the token, in scalar registers throughout.
      uint64_t base_of[2], absent[2] = {0, 0};
      auto pages_from = [&](int j0) {
        const int j = j0 + lane;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int tok = (t0 + wave + j * kW) * kTileTokens + 16 * h;
          int p = -1;
          if (j < mine && tok < s.len) p = table[tok >> a.page_shift];
          const bool none = p < 0 || p >= a.pages;
          base_of[h] = reinterpret_cast<uint64_t>(head_base) + static_cast<uint64_t>(none ? 0 : p) * a.page_bytes;
          absent[h] = __ballot(none);
        }
      };
      // Tile j's place: the segments of its halves and their tokens' offsets in
      // the codes and in the scales. Past the last tile the segments are empty:
      // loads there bring zeros and no traffic, and as every step has the same
      // loads, a wait for the older ones need not be a wait for all.
      struct Place {
        __amdgpu_buffer_rsrc_t seg[2];
        int codes[2], scales[2];
      };
      const auto place = [&](int j) {
        Place r;
        if ((j & 63) == 0) pages_from(j);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(base_of[h]), j & 63);
          const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(base_of[h] >> 32), j & 63);
          r.seg[h] = segment_of(reinterpret_cast<const uint8_t*>(static_cast<uint64_t>(hi) << 32 | lo),
                                j < mine ? a.seg_bytes : 0);
          const int off = ((t0 + wave + j * kW) * kTileTokens + 16 * h) & (page - 1);
          r.codes[h] = off * (DIM / 2);
          r.scales[h] = off * (DIM / 16);
        }
        return r;
      };
      Tile<DIM> t;
      const LaneOffsets<DIM> lane_at(lane, page);
      if (mine > 0) {
        const Place r = place(0);
#pragma unroll
        for (int h = 0; h < 2; ++h) load_keys<DIM>(t, h, r.seg[h], lane_at, r.codes[h], r.scales[h]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int h = 0; h < 2; ++h) load_vals<DIM>(t, h, r.seg[h], lane_at, r.codes[h], r.scales[h]);
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_sched_barrier(0);
      const auto exponent_of = [&](const u4 (&x)[kQueriesFirst ? 1 : kSteps]) {
        uint32_t top = 0;
        if constexpr (BF16) {
#pragma unroll
          for (const u4& w : x) top = larger(top, w);
          return exponent(top);
        }
        return 0;
      };
      if constexpr (kQueriesInLds) {
        if constexpr (!kQueriesFirst) {
          if (wave < NQ) {
            const int e2 = exponent_of(raw[0]);
#pragma unroll
            for (int c = 0; c < kSteps; ++c)
              sh.q[(wave * kSteps + c) * 64 + lane] = __builtin_bit_cast(u4, fragment(wave, raw[0][c], e2));
            if (g == 0) fs[wave * 16 + i] = factor(e2);
          }
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NQ; ++n) f[n] = fs[n * 16 + i];
      } else {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          const int e2 = exponent_of(raw[n]);
#pragma unroll
          for (int c = 0; c < kSteps; ++c) qreg[n][c] = fragment(n, raw[n][c], e2);
          f[n] = factor(e2);
        }
      }
      const auto query = [&](int n, int c) -> h8 {
        if constexpr (kQueriesInLds)
          return __builtin_bit_cast(h8, sh.q[(n * kSteps + c) * 64 + lane]);
        else
          return qreg[n][c];
      };
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        m[n] = kNoToken;
        l[n] = 0.f;
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) o[n][j] = f4{0.f, 0.f, 0.f, 0.f};
      }

      // The keys of the next tile are on their way during this one's softmax and
      // values, its values during the next one's scores: one set of registers
      // each, and the other wavefronts of the SIMD to fill what is left.
      //
      // A SIMD serves the older of its wavefronts first, and the workgroup that
      // came second to a compute unit would end a third later than the first. So
      // a wavefront's priority falls with every quarter of its tiles: whoever is
      // behind goes first.
      const int quarter = (mine + 3) / 4;
      __builtin_amdgcn_s_setprio(3);
      // (At three row tiles of 128, whose registers hold two tiles, the whole next
      // tile is asked for before this one's scores: 57 -> 54 us over 131072 tokens.
      // Two tiles would spill at two and three row tiles of 64, one and two of 128 and
      // two of 256; they would fit at one and four of 64 and one of 256, which were
      // not measured.)
      constexpr bool kTwo = NQ * DIM == 384;
      auto step = [&](Tile<DIM>& t, Tile<DIM>& u, int j) {
        if (j == quarter) __builtin_amdgcn_s_setprio(2);
        if (j == 2 * quarter) __builtin_amdgcn_s_setprio(1);
        if (j == 3 * quarter) __builtin_amdgcn_s_setprio(0);
        const int tok = (t0 + wave + j * kW) * kTileTokens;
        Place r;
        bool none0, none1;  // before place(j + 1) looks up the next 64
        if constexpr (kTwo) {
          none0 = absent[0] >> (j & 63) & 1, none1 = absent[1] >> (j & 63) & 1;
          r = place(j + 1);
#pragma unroll
          for (int h = 0; h < 2; ++h) load_keys<DIM>(u, h, r.seg[h], lane_at, r.codes[h], r.scales[h]);
#pragma unroll
          for (int h = 0; h < 2; ++h) load_vals<DIM>(u, h, r.seg[h], lane_at, r.codes[h], r.scales[h]);
          __builtin_amdgcn_sched_barrier(0);
        }
        f4 sc[2][NQ];
        scores<DIM, NQ>(t, query, sc);
        if constexpr (!kTwo) {
          none0 = absent[0] >> (j & 63) & 1, none1 = absent[1] >> (j & 63) & 1;
          __builtin_amdgcn_sched_barrier(0);
          r = place(j + 1);
#pragma unroll
          for (int h = 0; h < 2; ++h) load_keys<DIM>(t, h, r.seg[h], lane_at, r.codes[h], r.scales[h]);
          __builtin_amdgcn_sched_barrier(0);
        }
        uint32_t vs[2] = {t.vs[0], t.vs[1]};
        const bool whole =
            tok + kTileTokens - 1 <= first_pos && (win == 0 || tok > last_pos - win) && !none0 && !none1;
        if (!whole) {
          // Scores of unseen tokens become -inf whatever the cache holds there,
          // and the values of tokens past the end, of absent pages or in front of
          // all rows' windows are zeroed: such bytes may decode to NaN, which a p of
          // 0 would not remove. Bit b of a mask stands for token tok + 4 g + b.
          const int mine0 = tok + 4 * g;
          const auto up_to = [](int x) -> uint32_t { return x < 0 ? 0u : x >= 31 ? ~0u : (2u << x) - 1u; };
          const uint32_t held = up_to(s.len - 1 - mine0) & (win ? ~up_to(first_pos - win - mine0) : ~0u) &
                                ((none0 ? 0u : 0xFFFFu) | (none1 ? 0u : 0xFFFF0000u));
          const auto bit = [](uint32_t w, int b) {
            return static_cast<uint32_t>(static_cast<int32_t>(w << (31 - b)) >> 31);
          };
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) vs[h] &= ~(0xFFu << (8 * e)) | bit(held, 16 * h + e);
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            // (the row's position is worked out here, for the few tiles that need it)
            const int pos = s.len - s.ql + (row0 + n * 16 + i) / a.group;
            const uint32_t seen = held & up_to(pos - mine0) & (win ? ~up_to(pos - win - mine0) : ~0u);
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
        if constexpr (!kTwo) {
#pragma unroll
          for (int h = 0; h < 2; ++h) load_vals<DIM>(t, h, r.seg[h], lane_at, r.codes[h], r.scales[h]);
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      if constexpr (kTwo) {
        Tile<DIM> u;
        for (int j = 0; j < mine; j += 2) {
          step(t, u, j);
          if (j + 1 >= mine) break;
          step(u, t, j + 1);
        }
      } else {
        for (int j = 0; j < mine; ++j) step(t, t, j);
      }

      const AttnParams& z = reread(params);
      // Join the wavefronts: a row's reference becomes the largest of the four.
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        l[n] += __shfl_xor(l[n], 16);
        l[n] += __shfl_xor(l[n], 32);
        if (g == 0) ml[wave][n * 16 + i] = float2{m[n], l[n]};
      }
      __syncthreads();
      const int64_t part_rows = static_cast<int64_t>(2 * group_id + (tile0 == 0)) * kRows;
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
            if (!alone) {
              float* dst = z.part + (part_rows + row) * DIM + d;
              *reinterpret_cast<f4*>(dst) = f4{v[0], v[1], v[2], v[3]};
              *reinterpret_cast<f4*>(dst + 4) = f4{v[4], v[5], v[6], v[7]};
              if (d == 0) {
                float2* mld = reinterpret_cast<float2*>(z.part + static_cast<int64_t>(2 * z.groups) * kRows * DIM);
                mld[part_rows + row] = float2{mr, lr};
              }
            } else {
              const int qi = (row0 + row) / z.group, hh = (row0 + row) - qi * z.group;
              const int64_t row_at = static_cast<int64_t>(s.qs + qi) * (z.kv_heads * z.group) + head * z.group + hh;
              const float up = lr > 0.f ? z.v_scale / lr : (lr == 0.f ? 0.f : lr);
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] *= up;
              store_out8<BF16>(z.out, row_at * DIM + d, v);
              if (d == 0 && z.lse)
                z.lse[row_at] = lr == 0.f ? -__builtin_inff() : (__builtin_amdgcn_logf(lr) + mr) * 0.69314718055994531f;
            }
          }
        }
        __syncthreads();
      }
    }
    if (at >= end) break;
    if (at - base >= cost * s.rt * reread(params).kv_heads) {
      // the next sequence that has rows
      base = at;
      do seq = sequence(reread(params), ++b, kRows);
      while (seq.rt == 0);
    }
  }
}

// Joins the pieces of the runs that were cut, in the order of the line, one
// wavefront a row: a run of n + 1 pieces has n workgroups that begin inside
// of it, and these share its rows. (A workgroup for every four rows of every
// one of them, most of which had nothing to do, took 9 us; this takes 5.)
constexpr int kJoinWaves = 16;

template <int DIM, int NQ, bool BF16>
__global__ __launch_bounds__(kJoinWaves * 64) void kv4_attention_join_kernel(const AttnParams a) {
  constexpr int kRows = 16 * NQ;
  constexpr int kPer = 8, kLanes = DIM / kPer;  // lanes that hold a row; the others take other pieces
  constexpr int kGroups = 64 / kLanes;
  const int lane = threadIdx.x & 63, w = blockIdx.x;
  const Cut c = a.cuts[w];
  if (c.rows == 0) return;  // else first < w <= last
  const int gr = lane / kLanes, d = lane % kLanes * kPer;
  const float2* ml = reinterpret_cast<const float2*>(a.part + static_cast<int64_t>(2 * a.groups) * kRows * DIM);
  const int n = c.last - c.first;
  for (int r = w - c.first - 1 + __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6) * n; r < c.rows;
       r += n * kJoinWaves) {
    const auto piece = [&](int x) { return (2 * x + (x == c.first)) * kRows + r; };
    // every kLanes lanes take each kGroups-th piece, under a reference of their
    // own. (The kernel is short enough for the fetching of its code to count: eight
    // pieces at once after a pass for the largest reference took 1.4 to 3 us more
    // where runs are cut into few pieces, and 0.3 less where one is cut into 64.)
    float mx = kNoToken, l = 0.f, v[kPer] = {};
#pragma unroll 3
    for (int x = c.first + gr; x <= c.last; x += kGroups) {
      const float2 q = ml[piece(x)];
      const float* src = a.part + static_cast<int64_t>(piece(x)) * DIM + d;
      const f4 v0 = *reinterpret_cast<const f4*>(src), v1 = *reinterpret_cast<const f4*>(src + 4);
      const float top = fmaxf(mx, q.x), down = __builtin_amdgcn_exp2f(mx - top), p = __builtin_amdgcn_exp2f(q.x - top);
      mx = top;
      l = l * down + p * q.y;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = v[e] * down + p * v0[e];
        v[4 + e] = v[4 + e] * down + p * v1[e];
      }
    }
    const float own = mx;
#pragma unroll
    for (int o = kLanes; o < 64; o <<= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
    const float down = __builtin_amdgcn_exp2f(own - mx);
    l *= down;
#pragma unroll
    for (int e = 0; e < kPer; ++e) v[e] *= down;
#pragma unroll 1
    for (int o = kLanes; o < 64; o <<= 1) {
      l += __shfl_xor(l, o);
#pragma unroll
      for (int e = 0; e < kPer; ++e) v[e] += __shfl_xor(v[e], o);
    }
    if (gr == 0) {
      const float up = l > 0.f ? a.v_scale / l : (l == 0.f ? 0.f : l);
#pragma unroll
      for (int e = 0; e < kPer; ++e) v[e] *= up;
      const int qi = (c.row0 + r) / a.group, hh = (c.row0 + r) - qi * a.group;
      const int64_t to = static_cast<int64_t>(c.qs + qi) * (a.kv_heads * a.group) + c.head * a.group + hh;
      store_out8<BF16>(a.out, to * DIM + d, v);
      if (d == 0 && a.lse)
        a.lse[to] = l == 0.f ? -__builtin_inff() : (__builtin_amdgcn_logf(l) + mx) * 0.69314718055994531f;
    }
  }
}

template <int DIM, int NQ, bool BF16>
hipError_t launch_as(const AttnParams& a, hipStream_t stream) {
  const uint32_t grid = a.groups ? a.groups : static_cast<uint32_t>(a.batch) * a.row_tiles * a.kv_heads;
  kv4_attention_kernel<DIM, NQ, BF16><<<dim3(grid), dim3(kW * 64), 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.groups == 0) return e;
  kv4_attention_join_kernel<DIM, NQ, BF16>
      <<<dim3(static_cast<uint32_t>(a.groups)), dim3(kJoinWaves * 64), 0, stream>>>(a);
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
  // (no length is above 2^30; a position less the window stays inside 32 bits)
  a.max_kv = x.max_kv_len, a.window = x.window < (1 << 30) ? x.window : 1 << 30;
  a.row_tiles = p.row_tiles, a.groups = p.groups, a.min_share = p.min_share;
  a.f = std::min(std::min(x.scale * 1.44269504088896341f, kMost) * c.k_scale, kMost);
  if (x.dtype == QPN_DT_F16) a.f = std::max(a.f, kLeast);  // (bf16: with each row's power of two)
  a.v_scale = c.v_scale;
  a.cuts = static_cast<Cut*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + p.cut_bytes);
  return x.dtype == QPN_DT_BF16 ? launch_dim<true>(c.head_dim, p.tiles16, a, stream)
                                : launch_dim<false>(c.head_dim, p.tiles16, a, stream);
}

}  // namespace qpn
