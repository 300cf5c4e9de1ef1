// Attention of chunks of new tokens over the 4-bit paged cache and themselves
// (include/qpn_prompt.h).
//
// Mathematics. One kv head's query rows (new tokens x query heads of the
// group) form tiles of 128, a workgroup's, 32 a wavefront. Tokens come 64 at a
// time: first the cached ones, decoded to fp16 (E2M1 x E4M3 is exact there),
// then the new ones in their own type. Each 64 go to LDS once for all 128
// rows, and a wavefront computes S^T = K Q^T and O^T += V^T P^T with
// v_mfma_f32_32x32x16, p = 2^(s f - m) under a running reference m per row.
//
// Layouts that need no shuffle. Lane l = (i, h) = (l % 32, l / 32):
//  - S^T has the row i of the wavefront in a lane, at tokens 8 a + 4 h + b of
//    32 (a, b = 0 .. 3): a row's statistics are a lane's, but for one exchange
//    with lane l ^ 32.
//  - P^T as the B operand wants 8 tokens of 16 in lane (i, h): its own are
//    4 h + b and 8 + 4 h + b, so the contraction's places stand for these, and
//  - V^T as the A operand has them together: LDS holds a 16's quads of tokens in the
//    order 0, 2, 1, 3 along each element's row. The rows' 16-byte pieces are
//    permuted by the row number, so that neither a read of neighbouring
//    elements nor a write of every eighth meets one bank.
//
// f = scale * log2(e) (* k_scale for the cache); v_scale multiplies O once,
// between the cached and the new tokens.
//
// What is rounded, and why. The matrix instructions take 16-bit operands, so p is
// rounded before its product with the values: to fp16 for cached tokens, whose values fp16
// holds exactly, and to their own type for new ones. Taken apart into two such halves it
// would need 16 more of a step's 32 matrix instructions, which are 38 % of the
// cycles already. It adds 2e-4 (fp16) or 1.1e-3 (bf16) of a result to the rounding of the result
// itself, 2.1e-4 or 1.6e-3: together 2.9e-4 and 2.0e-3, heads of 256 2.1e-3 (2-norms).
//
// What bounds it, at 2048 new tokens after 30000 (40 heads on 8 of 128, 1.3 Tflop):
// 1505 to 1560 us, 0.86 PFLOP/s of the 1.35 that a large product reaches. The matrix
// instructions take 38 % of the cycles and the vector ones (exponentials, the
// decoding) 49 %, with little overlap; the clock is at 2.0 GHz under load (over zeros,
// which draw less power: 1356 us where it took 1514). Heads of 64: 1015 us, where exponentials
// are twice as many for each product. 128 rows a workgroup and 64 tokens: 256 threads with
// O, Q and P in registers, two workgroups a compute unit, so that one decodes while
// the other multiplies. Where this took 1723 us, two LDS buffers and one barrier a step
// took 1724, a raised priority around the products 1704 to 1750, more LDS reads ahead 1790
// and the next step's products in between this one's exponentials 1674, but heads of
// 256 spill then (980 instead of 275): none is worth its cost.
// One short run is its steps' latency: 5 tokens after 300 19 us.
#include <algorithm>

#include "qpn_device.hpp"
#include "qpn_prompt_internal.hpp"
#include "qpn_decode_internal.hpp"

namespace qpn {
namespace {

typedef float f16v __attribute__((ext_vector_type(16)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef u4 u4_anywhere __attribute__((aligned(2)));

constexpr int kThreads = 256, kRows = kChunkRows, kTokens = kChunkTokens;
// Steps a share has at least: every share of a run writes and joins a piece of it. With 1,
// 2, 4, 8: 5 rows after 1000 tokens 16.7, 18.1, 20.7, 27 us; 60 after 3000 34, 34, 35, 39; 8
// sequences of 1 to 100 after 100 to 3000 38, 38, 40, 49; 24 ragged ones 299, 297, 295, 294.
constexpr int kMinShare = 4;
constexpr float kNoToken = -1e30f;  // a row's reference before it has seen a token
constexpr float kBias = 8.0f, kHeadroom = 15.0f;
constexpr float kLeast = 1.17549435e-38f, kMost = 3.40282347e+38f;  // fp32's normal range
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;

struct ChunkParams {
  const uint8_t* cache;  // the layer
  int64_t page_bytes;
  int32_t pages, page_shift, seg_bytes, kv_heads, group;
  const void *q, *k, *v;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;
  void* out;
  float* lse;
  const int32_t* table;
  int64_t table_stride;
  const int32_t *kv_len, *q_start;
  int32_t batch, rows, max_q, max_kv, window, tiles, groups;
  float f, k_scale, v_scale;  // f: scale * log2(e)
  struct Cut* cuts;           // [groups]; groups 0: a workgroup a run, no join
  float* part;                // [2 groups][kRows][DIM], then [2 groups][kRows][2]
};

// The run that a workgroup's share begins inside of (rows 0: it begins with
// one): its pieces are those of shares first .. last, its rows `rows` of kv
// head `head`'s from row `row0` of the sequence whose new tokens begin at `qs`.
struct Cut {
  int rows, first, last, qs, row0, head, pad[2];
};
static_assert(sizeof(Cut) == 32, "the workspace holds 32 bytes a share");

// A sequence: its new tokens qs .. qs + ql - 1, its `len` cached ones, its row
// tiles and what they cost: row tile j first + more * j, in sixteenths of a step of
// 64 tokens.
struct Sequence {
  int qs, ql, len, tiles, first, more;
};

// What a run costs besides its steps, in steps: queries, the first loads, the output. 24
// ragged sequences take 351 us with 0, 318 with 1, 296 with 3, 300 with 6; 8 of 1 to 100 rows after
// 100 to 3000 47, 40, 40, 34; one of 2048 rows the same with all.
constexpr int kRunCost = 3;

__device__ __forceinline__ Sequence sequence(const ChunkParams& a, int b) {
  Sequence s;
  if (a.q_start) {
    s.qs = min(max(a.q_start[b], 0), a.rows);
    s.ql = min(min(max(a.q_start[b + 1] - s.qs, 0), a.max_q), a.rows - s.qs);
  } else {
    s.qs = b * a.max_q;
    s.ql = a.max_q;
  }
  s.len = a.pages > 0 ? min(max(a.kv_len[b], 0), a.max_kv) : 0;
  s.tiles = (s.ql * a.group + kRows - 1) / kRows;
  // a window's row tile sees the window and its own rows, another all cached tokens and the new ones up to it
  const int seen = a.window ? min(a.window + kRows / a.group, s.len + s.ql) : s.len;
  s.first = 16 * (seen / kTokens + 1 + kRunCost);
  s.more = a.window ? 0 : 16 * kRows / kTokens / a.group;
  return s;
}

// The cost of the first j row tiles.
__device__ __forceinline__ int64_t cost_of(const Sequence& s, int64_t j) {
  return s.first * j + s.more * (j * (j - 1) / 2);
}

__device__ __forceinline__ Sequence lane_of(const Sequence& s, int l) {
  const auto get = [&](int x) { return __builtin_amdgcn_readlane(x, l); };
  return Sequence{get(s.qs), get(s.ql), get(s.len), get(s.tiles), get(s.first), get(s.more)};
}

__device__ __forceinline__ int64_t lane_of(int64_t x, int l) {
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(x), l);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(static_cast<uint64_t>(x) >> 32), l);
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// Sums over the lanes up to each.
__device__ __forceinline__ int64_t scan(int64_t x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Where place `at` of a line lies to which sequence b adds line(sequence): the
// sequence and the place at which its part begins (false: behind the line).
template <typename Line>
__device__ __forceinline__ bool find_sequence(const ChunkParams& a, int64_t at, Line line, int& b, int64_t& base,
                                              Sequence& s) {
  const int lane = threadIdx.x & 63;
  int64_t before = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    Sequence mine = {0, 0, 0, 0, 0, 0};
    int64_t part = 0;
    if (b0 + lane < a.batch) {
      mine = sequence(a, b0 + lane);
      part = line(mine);
    }
    const int64_t sum = scan(part);
    const uint64_t past = __ballot(at < before + sum);
    if (past) {
      const int l = __builtin_ctzll(past);
      b = b0 + l;
      base = before + lane_of(sum - part, l);
      s = lane_of(mine, l);
      return true;
    }
    before += lane_of(sum, 63);
  }
  return false;
}

// The kernel's arguments, to be read again from where they lie.
typedef const ChunkParams __attribute__((address_space(4))) * ParamsPtr;
__device__ __forceinline__ const ChunkParams& reread(const ChunkParams&) {
  ParamsPtr p = (ParamsPtr)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const ChunkParams*)p;
}

__device__ __forceinline__ h2 splat(_Float16 x) { return h2{x, x}; }

// Two dwords, x of even and y of odd elements: byte b holds element 2b (or
// 2b + 1) of two tokens.
__device__ __forceinline__ void pair_up(uint32_t a, uint32_t b, uint32_t& x, uint32_t& y) {
  constexpr uint32_t m = 0x0F0F0F0Fu;
  x = (a & m) | ((b << 4) & ~m);
  y = ((a >> 4) & m) | (b & ~m);
}

template <int I>
__device__ __forceinline__ uint32_t scaled_pair(uint32_t w, h2 s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, I) * s);
}

// LDS of a workgroup, in 16-bit units.
template <int DIM>
struct Tiles {
  static constexpr int kKeyStride = DIM + 8;
  alignas(16) uint16_t k[kTokens * kKeyStride];
  alignas(16) uint16_t v[DIM * kTokens];
  uint32_t odd[2];  // tokens of the 64 whose values hold inf or NaN, where some row may not see them
};

// The place of quad q (tokens 4 q .. 4 q + 3) in element d's row of V^T.
__device__ __forceinline__ int value_at(int d, int q) {
  const int order = ((q & 1) << 1) | ((q >> 1) & 1);
  const int piece = (q >> 2) * 2 + (order >> 1);
  return d * kTokens + ((piece ^ ((d ^ (d >> 3)) & 7)) * 8) + (order & 1) * 4;
}

template <bool BF16>
struct Half;
template <>
struct Half<false> {
  typedef h8 vec;
  static __device__ __forceinline__ f16v mfma(u4 a, u4 b, f16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t round2(float x, float y) {
    return __builtin_bit_cast(uint32_t, h2{static_cast<_Float16>(x), static_cast<_Float16>(y)});
  }
  static constexpr uint32_t kExponent = 0x7C00u;
};
template <>
struct Half<true> {
  static __device__ __forceinline__ f16v mfma(u4 a, u4 b, f16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t round2(float x, float y) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{x, y}), b2));
  }
  static constexpr uint32_t kExponent = 0x7F80u;
};

// inf and NaN among two 16-bit values become 0; whether there were any.
template <bool BF16>
__device__ __forceinline__ bool strike_odd(uint32_t& x) {
  constexpr uint32_t e = Half<BF16>::kExponent;
  const bool lo = (x & e) == e, hi = (x >> 16 & e) == e;
  x &= (lo ? 0xFFFF0000u : ~0u) & (hi ? 0xFFFFu : ~0u);
  return lo || hi;
}

template <int DIM, bool BF16>
__global__ __launch_bounds__(kThreads, DIM == 256 ? 1 : 2) void kv4_chunk_kernel(const ChunkParams params) {
  constexpr int kSteps = DIM / 16, kBlocks = DIM / 32;
  constexpr int kKeyUnits = (kTokens * DIM / 32 + kThreads - 1) / kThreads;  // of 32 elements, a thread
  constexpr int kPerToken = DIM / 32;
  constexpr int kValueWords = DIM / 32;                       // dwords of a quad's codes a thread has
  constexpr int kNewUnits = kTokens * DIM / 8 / kThreads;     // 16 bytes of a new token's key, a thread
  constexpr int kNewQuads = kTokens / 4 * DIM / 8 / kThreads; // 8 elements of four new tokens' values, a thread
  constexpr int kQuadUnits = kNewQuads > 0 ? kNewQuads : 1;
  __shared__ Tiles<DIM> sh;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  int tid = threadIdx.x, lane = tid & 63;

  // The work is the steps of all (sequence, kv head, row tile), laid end to end in
  // that order. Each of `groups` workgroups, as many as the device holds at once,
  // takes an equal share of that line, whatever the lengths: a share may begin inside
  // of one run of steps and end inside another. A run that lies in one share is written
  // as it is; the pieces of any other go to the workspace, at most two a share (the end
  // of a run in slot 2 w, the beginning of one in slot 2 w + 1), and the join kernel adds
  // them. Workgroups go round the eight dies; each die takes an eighth of the line, so
  // that the row tiles of a head, which read the same tokens, meet in its cache.
  int b = 0, share_of = 0;
  int64_t base = 0, at = 0, end = 1, share = 0;
  Sequence seq;
  {
  const ChunkParams& a = params;
  if (a.groups == 0) {
    const int64_t t = a.tiles - 1 - blockIdx.x / a.kv_heads;  // a sequence's last rows, which see most, go first
    if (!find_sequence(a, t, [](const Sequence& x) { return static_cast<int64_t>(x.tiles); }, b, base, seq)) return;
    at = (blockIdx.x % a.kv_heads) * cost_of(seq, seq.tiles) + cost_of(seq, t - base);
    end = at + seq.first + seq.more * (t - base);
    base = 0;
  } else {
    const auto line = [&](const Sequence& x) { return a.kv_heads * cost_of(x, x.tiles); };
    int64_t total = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
      int64_t part = 0;
      if (b0 + lane < a.batch) part = line(sequence(a, b0 + lane));
      total += lane_of(scan(part), 63);
    }
    share_of = blockIdx.x % 8 * (a.groups / 8) + blockIdx.x / 8;
    share = max((total + a.groups - 1) / a.groups, static_cast<int64_t>(16 * kMinShare));
    at = share_of * share;
    end = min(at + share, total);
    if (at >= total) {
      if (tid == 0) a.cuts[share_of].rows = 0;
      return;
    }
    find_sequence(a, at, line, b, base, seq);
  }
  }
  bool first_run = true;
  while (true) {
  // (what follows from the lane is worked out again for every run: kept from one
  // to the next it would take registers; and so are the arguments, which come from
  // the scalar cache)
  asm volatile("" : "+v"(tid), "+v"(lane));
  const ChunkParams& a = reread(params);
  const int i = lane & 31, h = lane >> 5;
  // The run: its kv head and row tile, and the part [from, to) of its cost.
  const int64_t head_cost = cost_of(seq, seq.tiles);
  const int head = static_cast<int>((at - base) / head_cost);
  const int64_t in_head = at - base - head * head_cost;
  int low = 0, high = seq.tiles - 1;  // the last row tile that begins at in_head or before
  while (low < high) {
    const int mid = (low + high + 1) / 2;
    if (cost_of(seq, mid) <= in_head) low = mid;
    else high = mid - 1;
  }
  const int cost = seq.first + seq.more * low;
  const int from = static_cast<int>(in_head - cost_of(seq, low));
  const int to = static_cast<int>(min(static_cast<int64_t>(cost), from + end - at));
  struct { int b, qs, ql, len, row0; } rt = {b, seq.qs, seq.ql, seq.len, low * kRows};
  const int nrows = min(rt.ql * a.group - rt.row0, kRows);
  const int win = a.window;
  const bool alone = from == 0 && to == cost;
  if (first_run && a.groups && tid == 0) {
    const int64_t begin = at - from;
    a.cuts[share_of] = Cut{from > 0 ? nrows : 0, static_cast<int>(begin / share),
                           static_cast<int>((begin + cost - 1) / share), rt.qs, rt.row0, head, {0, 0}};
  }
  first_run = false;
  at += to - from;

  // The tokens that the tile's rows see, in steps of 64: cached ones from step
  // c0 to c1, then new ones from n0 to n1.
  const int q_first = rt.row0 / a.group, q_last = (rt.row0 + nrows - 1) / a.group;
  int c0 = 0, c1 = (rt.len + kTokens - 1) / kTokens, n0 = 0, n1 = q_last / kTokens + 1;
  if (win) {
    c0 = min(max(rt.len + q_first - win + 1, 0) / kTokens, c1);
    n0 = max(q_first - win + 1, 0) / kTokens;
  }
  const int steps = c1 - c0 + n1 - n0;
  const int s0 = static_cast<int>(static_cast<int64_t>(steps) * from / cost);
  const int s1 = static_cast<int>(static_cast<int64_t>(steps) * to / cost);
  // this workgroup's share of them
  const int cb = c0 + min(s0, c1 - c0), ce = c0 + min(s1, c1 - c0);
  const int nb = n0 + max(s0 - (c1 - c0), 0), ne = n0 + max(s1 - (c1 - c0), 0);

  // This lane's row.
  const int r = wave * 32 + i;
  const bool live = r < nrows, busy = wave * 32 < nrows;  // (the wavefront has rows)
  const int qi = (rt.row0 + (live ? r : 0)) / a.group, hh = rt.row0 + (live ? r : 0) - qi * a.group;
  const int w_first = (rt.row0 + wave * 32) / a.group, w_last = (rt.row0 + min(wave * 32 + 31, nrows - 1)) / a.group;
  const uint16_t* q_row = static_cast<const uint16_t*>(a.q) + static_cast<int64_t>(rt.qs + qi) * a.q_ts +
                          static_cast<int64_t>(head * a.group + hh) * a.q_hs + h * 8;
  u4 q[kSteps];
  f16v o[kBlocks];
  float m = kNoToken, l = 0.f;
#pragma unroll
  for (int n = 0; n < kBlocks; ++n) o[n] = 0.f;

  const auto load_queries = [&] {
#pragma unroll
    for (int c = 0; c < kSteps; ++c) q[c] = *reinterpret_cast<const u4_anywhere*>(q_row + c * 16);
  };

  // One step: scores of the 64 tokens in LDS against the wavefront's rows,
  // their softmax, the values. `whole`: every row sees every token. Else a row
  // sees token t of the 64 where lo <= t <= hi and bit t of `held` is set.
  const auto step = [&](auto type, float f, bool whole, uint64_t held, int lo, int hi) {
    using H = decltype(type);
    f16v s[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) s[x] = 0.f;
#pragma unroll
    for (int c = 0; c < kSteps; ++c) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const u4 key = *reinterpret_cast<const u4*>(&sh.k[(x * 32 + i) * Tiles<DIM>::kKeyStride + c * 16 + h * 8]);
        s[x] = H::mfma(key, q[c], s[x]);
      }
      // (else the compiler asks for all keys at once, and has no registers for them)
      if (DIM == 256 && c % 4 == 3) __builtin_amdgcn_sched_barrier(0);
    }
    if (!whole) {
      const uint64_t mine = held >> (4 * h);
      const int from = lo - 4 * h, to = hi - 4 * h;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int t = x * 32 + e / 4 * 8 + e % 4;
          const bool seen = t >= from && t <= to && (mine >> t & 1);
          s[x][e] = seen ? s[x][e] : -__builtin_inff();
        }
    }
    float top = s[0][0];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, s[x][e]);
    // (a row's reference moves only when a score passes it by 2^7)
    if (__any(fmaf(top, f, -m) > kHeadroom)) {
      float mx = fmaxf(m, fmaf(top, f, -kBias));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float down = __builtin_amdgcn_exp2f(m - mx);
      m = mx;
      l *= down;
#pragma unroll
      for (int n = 0; n < kBlocks; ++n) o[n] *= down;
    }
    u4 p[4];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const float p0 = __builtin_amdgcn_exp2f(fmaf(s[x][e], f, -m));
        const float p1 = __builtin_amdgcn_exp2f(fmaf(s[x][e + 1], f, -m));
        l += p0 + p1;  // (before they are rounded: lse keeps its 32 bits)
        p[x * 2 + e / 8][e % 8 / 2] = H::round2(p0, p1);
      }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
#pragma unroll
      for (int n = 0; n < kBlocks; ++n) {
        const int d = n * 32 + i;
        const u4 val = *reinterpret_cast<const u4*>(&sh.v[d * kTokens + (((2 * c + h) ^ ((d ^ (d >> 3)) & 7)) * 8)]);
        o[n] = H::mfma(val, p[c], o[n]);
      }
      if (DIM == 256) __builtin_amdgcn_sched_barrier(0);
    }
  };

  // ---- cached tokens
  if (cb < ce) {
    const int page = 1 << a.page_shift;
    const int32_t* table = a.table + static_cast<int64_t>(rt.b) * a.table_stride;
    const uint8_t* head_base = a.cache + static_cast<int64_t>(head) * a.seg_bytes;
    // a lane's token's page (-1: none)
    const auto page_of = [&](int c) {
      const int t = c * kTokens + lane;
      int p = -1;
      if (c < ce && t < rt.len) p = table[t >> a.page_shift];
      return p < a.pages ? p : -1;
    };
    u4 kc[kKeyUnits];
    uint32_t ks[kKeyUnits], vc[kValueWords], vs;
    const auto load_cached = [&](int c, int pg) {
#pragma unroll
      for (int j = 0; j < kKeyUnits; ++j) {
        const int unit = min(j * kThreads + tid, kTokens * kPerToken - 1), t = unit / kPerToken, part = unit % kPerToken;
        const int p = max(__shfl(pg, t), 0), off = (c * kTokens + t) & (page - 1);
        const uint8_t* seg = head_base + p * a.page_bytes;
        kc[j] = *reinterpret_cast<const u4*>(seg + off * (DIM / 2) + part * 16);
        ks[j] = *reinterpret_cast<const uint16_t*>(seg + page * DIM + off * (DIM / 16) + part * 2);
      }
      const int qd = tid / 16, e = tid % 16;
      const int p = max(__shfl(pg, qd * 4), 0), off = (c * kTokens + qd * 4) & (page - 1);
      const uint8_t* seg = head_base + p * a.page_bytes;
      const uint8_t* codes = seg + page * (DIM / 2) + lane_v<DIM>(e, off / 4);
      if constexpr (kValueWords == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(codes);
        vc[0] = x.x, vc[1] = x.y;
      } else {
#pragma unroll
        for (int j = 0; j < kValueWords / 4; ++j) {
          const u4 x = *reinterpret_cast<const u4*>(codes + 16 * j);
#pragma unroll
          for (int y = 0; y < 4; ++y) vc[4 * j + y] = x[y];
        }
      }
      vs = *reinterpret_cast<const uint32_t*>(seg + page * DIM + page * (DIM / 16) + off / 4 * (DIM / 4) + (e * DIM / 256) * 4);
    };
    // `guard`: some row may not see some token that is there, so a value scale of NaN must not meet its p of 0
    const auto store_cached = [&](uint64_t held, bool guard) {
#pragma unroll
      for (int j = 0; j < kKeyUnits; ++j) {
        const int unit = j * kThreads + tid, t = unit / kPerToken, part = unit % kPerToken;
        if (kTokens * kPerToken % kThreads != 0 && unit >= kTokens * kPerToken) break;
        const h2 sc = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(ks[j], 1.0f, false);
        uint16_t* dst = &sh.k[t * Tiles<DIM>::kKeyStride + part * 32];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          *reinterpret_cast<h8*>(dst + x * 8) = decode_fp4x8(kc[j][x], splat(sc[x / 2]));
      }
      // tokens that are not there have scales of 0, whatever the cache holds: their p is 0, and must meet no NaN
      const int qd = tid / 16, e = tid % 16;
      const uint32_t there = static_cast<uint32_t>(held >> (4 * qd)) & 15u;
      uint32_t scales = vs & ((there & 1u) * 0xFFu | (there >> 1 & 1u) * 0xFF00u | (there >> 2 & 1u) * 0xFF0000u |
                              (there >> 3) * 0xFF000000u);
      if (guard) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if ((scales >> (8 * x) & 0x7Fu) == 0x7Fu) {
            scales &= ~(0xFFu << (8 * x));
            atomicOr(&sh.odd[qd / 8], 1u << (qd % 8 * 4 + x));
          }
      }
      const h2 s01 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(scales, 1.0f, false);
      const h2 s23 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(scales, 1.0f, true);
      const auto put = [&](int d, uint32_t x, uint32_t y) {
        *reinterpret_cast<uint2*>(&sh.v[value_at(d, qd)]) = uint2{x, y};
      };
      uint32_t x0, y0, x1, y1;
      if constexpr (DIM == 64) {
        pair_up(vc[0], vc[0] >> 16, x0, y0);
        pair_up(vc[1], vc[1] >> 16, x1, y1);
        const int d = e * 4;
        put(d, scaled_pair<0>(x0, s01), scaled_pair<0>(x1, s23));
        put(d + 1, scaled_pair<0>(y0, s01), scaled_pair<0>(y1, s23));
        put(d + 2, scaled_pair<1>(x0, s01), scaled_pair<1>(x1, s23));
        put(d + 3, scaled_pair<1>(y0, s01), scaled_pair<1>(y1, s23));
      } else {
        constexpr int kTokenWords = DIM / 128;
#pragma unroll
        for (int w = 0; w < kTokenWords; ++w) {
          pair_up(vc[w], vc[kTokenWords + w], x0, y0);
          pair_up(vc[2 * kTokenWords + w], vc[3 * kTokenWords + w], x1, y1);
          const int d = e * (DIM / 16) + w * 8;
          put(d, scaled_pair<0>(x0, s01), scaled_pair<0>(x1, s23));
          put(d + 1, scaled_pair<0>(y0, s01), scaled_pair<0>(y1, s23));
          put(d + 2, scaled_pair<1>(x0, s01), scaled_pair<1>(x1, s23));
          put(d + 3, scaled_pair<1>(y0, s01), scaled_pair<1>(y1, s23));
          put(d + 4, scaled_pair<2>(x0, s01), scaled_pair<2>(x1, s23));
          put(d + 5, scaled_pair<2>(y0, s01), scaled_pair<2>(y1, s23));
          put(d + 6, scaled_pair<3>(x0, s01), scaled_pair<3>(x1, s23));
          put(d + 7, scaled_pair<3>(y0, s01), scaled_pair<3>(y1, s23));
        }
      }
    };

    int pg = page_of(cb);
    load_cached(cb, pg);
    load_queries();
    float f = a.f * a.k_scale;
    if constexpr (BF16) {
      // rows are scaled by the power of two that takes their largest to [2^15, 2^16), the top of fp16
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < kSteps; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(max(top, q[c][e] & 0x7FFFu), (q[c][e] >> 16) & 0x7FFFu);
      top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32)));
      const int e2 = min(max(static_cast<int>(top >> 7), 16), 254) - (127 + 15);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
#pragma unroll
      for (int c = 0; c < kSteps; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          q[c][e] = Half<false>::round2(__uint_as_float(q[c][e] << 16) * down,
                                        __uint_as_float(q[c][e] & 0xFFFF0000u) * down);
      f *= __uint_as_float(static_cast<uint32_t>(127 + e2) << 23);
    }
    // (0 or inf times a score, -inf or 0, would be NaN. Products of queries and codes are below 2^36: a factor
    // below the normal range makes them all as good as 0, and so does the least normal one)
    f = fminf(fmaxf(f, kLeast), kMost);
    uint64_t held = __ballot(pg >= 0);
    pg = page_of(cb + 1);
    if (win) {
      if (tid < 2) sh.odd[tid] = 0;
      __syncthreads();
    }
    for (int c = cb; c < ce; ++c) {
      const bool guard = win != 0 && c * kTokens <= rt.len + q_last - win;
      store_cached(held, guard);
      const uint64_t now = held;
      if (c + 1 < ce) {
        held = __ballot(pg >= 0);
        load_cached(c + 1, pg);
        pg = page_of(c + 2);
      }
      __syncthreads();
      if (busy) {
        const int t0 = c * kTokens;
        const bool whole = now == ~uint64_t(0) && (win == 0 || t0 > rt.len + w_last - win);
        step(Half<false>{}, f, whole, now, win ? rt.len + qi - win + 1 - t0 : 0, kTokens);
      }
      bool struck = false;
      if (guard) {
        const uint32_t odd0 = sh.odd[0], odd1 = sh.odd[1];
        struck = (odd0 | odd1) != 0;
        // What was struck comes back for the rows that see it: 16 elements of NaN for each such scale.
        for (uint64_t left = busy ? static_cast<uint64_t>(odd1) << 32 | odd0 : 0; left; left &= left - 1) {
          const int t = c * kTokens + __builtin_ctzll(left), off = t & (page - 1);
          const uint8_t* at = head_base + table[t >> a.page_shift] * a.page_bytes + page * DIM + page * (DIM / 16) +
                              off / 4 * (DIM / 4) + off % 4;
          if (t <= rt.len + qi - win) continue;
#pragma unroll
          for (int n = 0; n < kBlocks; ++n)
#pragma unroll
            for (int y = 0; y < 2; ++y)
              if ((at[(n * 2 + y) * 4] & 0x7F) == 0x7F)
#pragma unroll
                for (int e = 0; e < 8; ++e) o[n][y * 8 + e] = __builtin_nanf("");
        }
      }
      __syncthreads();
      if (struck) {
        if (tid < 2) sh.odd[tid] = 0;
        __syncthreads();
      }
    }
#pragma unroll
    for (int n = 0; n < kBlocks; ++n) o[n] *= a.v_scale;
  }

  // ---- new tokens
  if (nb < ne) {
    const uint16_t* kb = static_cast<const uint16_t*>(a.k) + rt.qs * a.k_ts + head * a.k_hs;
    const uint16_t* vb = static_cast<const uint16_t*>(a.v) + rt.qs * a.v_ts + head * a.v_hs;
    u4 kn[kNewUnits], vn[kQuadUnits][4];
    const auto load_new_keys = [&](int c) {
      // (tokens past the last are the last again: no row sees them)
#pragma unroll
      for (int j = 0; j < kNewUnits; ++j) {
        const int unit = j * kThreads + tid, t = min(c * kTokens + unit / (DIM / 8), rt.ql - 1);
        kn[j] = *reinterpret_cast<const u4_anywhere*>(kb + t * a.k_ts + unit % (DIM / 8) * 8);
      }
    };
    const auto load_new_values = [&](int c) {
#pragma unroll
      for (int j = 0; j < kQuadUnits; ++j) {
        const int unit = min(j * kThreads + tid, kTokens / 4 * DIM / 8 - 1);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int t = min(c * kTokens + unit / (DIM / 8) * 4 + x, rt.ql - 1);
          vn[j][x] = *reinterpret_cast<const u4_anywhere*>(vb + t * a.v_ts + unit % (DIM / 8) * 8);
        }
      }
    };
    const auto store_new_keys = [&] {
#pragma unroll
      for (int j = 0; j < kNewUnits; ++j) {
        const int unit = j * kThreads + tid;
        *reinterpret_cast<u4*>(&sh.k[unit / (DIM / 8) * Tiles<DIM>::kKeyStride + unit % (DIM / 8) * 8]) = kn[j];
      }
    };
    // `guard`: some row may not see some token of these, so their values must be finite
    const auto store_new_values = [&](bool guard) {
#pragma unroll
      for (int j = 0; j < kQuadUnits; ++j) {
        const int unit = j * kThreads + tid, qd = unit / (DIM / 8), d = unit % (DIM / 8) * 8;
        if (kTokens / 4 * DIM / 8 % kThreads != 0 && unit >= kTokens / 4 * DIM / 8) break;
        if (guard) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            bool odd = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w = vn[j][x][e];
              odd |= strike_odd<BF16>(w);
              vn[j][x][e] = w;
            }
            if (odd) atomicOr(&sh.odd[qd / 8], 1u << (qd % 8 * 4 + x));
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // element 2e (2e + 1) of tokens 0, 1 and of 2, 3
          constexpr uint32_t kLow = 0x05040100u, kHigh = 0x07060302u;
          const uint32_t w0 = vn[j][0][e], w1 = vn[j][1][e], w2 = vn[j][2][e], w3 = vn[j][3][e];
          *reinterpret_cast<uint2*>(&sh.v[value_at(d + 2 * e, qd)]) =
              uint2{__builtin_amdgcn_perm(w1, w0, kLow), __builtin_amdgcn_perm(w3, w2, kLow)};
          *reinterpret_cast<uint2*>(&sh.v[value_at(d + 2 * e + 1, qd)]) =
              uint2{__builtin_amdgcn_perm(w1, w0, kHigh), __builtin_amdgcn_perm(w3, w2, kHigh)};
        }
      }
    };
    constexpr bool kAhead = DIM < 256;  // (heads of 256 have no registers left for the next tokens)
    if constexpr (kAhead) {
      load_new_keys(nb);
      load_new_values(nb);
    }
    load_queries();
    if (tid < 2) sh.odd[tid] = 0;
    __syncthreads();
    for (int c = nb; c < ne; ++c) {
      const int t0 = c * kTokens;
      const bool guard = t0 + kTokens - 1 > q_first || (win != 0 && t0 <= q_last - win);
      if constexpr (kAhead) {
        store_new_keys();
        store_new_values(guard);
        if (c + 1 < ne) {
          load_new_keys(c + 1);
          load_new_values(c + 1);
        }
      } else {
        load_new_keys(c);
        store_new_keys();
        __builtin_amdgcn_sched_barrier(0);
        load_new_values(c);
        store_new_values(guard);
      }
      __syncthreads();
      const uint32_t odd0 = sh.odd[0], odd1 = sh.odd[1];
      if (busy) {
        const bool whole = t0 + kTokens - 1 <= w_first && (win == 0 || t0 > w_last - win);
        const int lo = win ? qi - win + 1 - t0 : 0, hi = qi - t0;
        step(Half<BF16>{}, a.f, whole, ~uint64_t(0), lo, hi);
        // What was struck comes back for the rows that see it (a row that sees inf or NaN is inf or NaN).
        for (uint64_t left = static_cast<uint64_t>(odd1) << 32 | odd0; left; left &= left - 1) {
          const int t = __builtin_ctzll(left);
          const uint16_t* src = vb + min(t0 + t, rt.ql - 1) * a.v_ts + 4 * h;
          if (t < lo || t > hi) continue;
#pragma unroll
          for (int n = 0; n < kBlocks; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint32_t x = src[n * 32 + e / 4 * 8 + e % 4];
              if ((x & Half<BF16>::kExponent) == Half<BF16>::kExponent) o[n][e] += widen16<BF16>(x);
            }
        }
      }
      __syncthreads();
      if ((odd0 | odd1) != 0) {
        if (tid < 2) sh.odd[tid] = 0;
        __syncthreads();
      }
    }
  }

  if (busy) {
    l += __shfl_xor(l, 32);
    const int64_t row_at = static_cast<int64_t>(rt.qs + qi) * (a.kv_heads * a.group) + head * a.group + hh;
    if (live && !alone) {
      const int64_t slot = (2 * share_of + (from == 0)) * kRows + r;
      if (h == 0) reinterpret_cast<float2*>(a.part + static_cast<int64_t>(2 * a.groups) * kRows * DIM)[slot] = float2{m, l};
      float* dst = a.part + slot * DIM + 4 * h;
#pragma unroll
      for (int n = 0; n < kBlocks; ++n)
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          *reinterpret_cast<f4*>(dst + n * 32 + e * 2) = f4{o[n][e], o[n][e + 1], o[n][e + 2], o[n][e + 3]};
    } else if (live) {
      const float up = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
      uint16_t* dst = static_cast<uint16_t*>(a.out) + row_at * DIM + 4 * h;
#pragma unroll
      for (int n = 0; n < kBlocks; ++n)
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          *reinterpret_cast<uint2*>(dst + n * 32 + e * 2) = uint2{Half<BF16>::round2(o[n][e] * up, o[n][e + 1] * up),
                                                                  Half<BF16>::round2(o[n][e + 2] * up, o[n][e + 3] * up)};
      if (h == 0 && a.lse) a.lse[row_at] = l == 0.f ? -__builtin_inff() : (__builtin_amdgcn_logf(l) + m) * kLn2;
    }
  }
  if (at >= end) break;
  if (at - base >= a.kv_heads * head_cost) {
    // the next sequence that has rows
    base = at;
    do seq = sequence(a, ++b);
    while (seq.tiles == 0);
  }
  }
}

// Joins the pieces of the runs that were cut, in the order of the line, a
// wavefront a row: a run of n + 1 pieces has n shares that begin inside of it, and
// these share its rows.
constexpr int kJoinWaves = 16;

template <int DIM, bool BF16>
__global__ __launch_bounds__(kJoinWaves * 64) void kv4_chunk_join_kernel(const ChunkParams a) {
  constexpr int kLanes = DIM / 4, kAtOnce = 64 / kLanes;  // lanes that hold a row, four elements each; pieces at once
  const int lane = threadIdx.x & 63, w = blockIdx.x;
  const Cut c = a.cuts[w];
  if (c.rows == 0) return;  // else first < w <= last
  const int gr = lane / kLanes, d = lane % kLanes * 4;
  const float2* ml = reinterpret_cast<const float2*>(a.part + static_cast<int64_t>(2 * a.groups) * kRows * DIM);
  const int n = c.last - c.first;
  for (int r = w - c.first - 1 + __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6) * n; r < c.rows;
       r += n * kJoinWaves) {
    float mx = kNoToken, l = 0.f;
    f4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int x = c.first + gr; x <= c.last; x += kAtOnce) {
      const int64_t slot = (2 * x + (x == c.first)) * static_cast<int64_t>(kRows) + r;
      const float2 q = ml[slot];
      const f4 piece = *reinterpret_cast<const f4*>(a.part + slot * DIM + d);
      const float top = fmaxf(mx, q.x), down = __builtin_amdgcn_exp2f(mx - top), p = __builtin_amdgcn_exp2f(q.x - top);
      mx = top;
      l = l * down + p * q.y;
      v = v * down + piece * p;
    }
    const float own = mx;
#pragma unroll
    for (int o = kLanes; o < 64; o <<= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
    const float down = __builtin_amdgcn_exp2f(own - mx);
    l *= down;
    v *= down;
#pragma unroll
    for (int o = kLanes; o < 64; o <<= 1) {
      l += __shfl_xor(l, o);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += __shfl_xor(v[e], o);
    }
    if (gr != 0) continue;
    const int qi = (c.row0 + r) / a.group, hh = c.row0 + r - qi * a.group;
    const int64_t row_at = static_cast<int64_t>(c.qs + qi) * (a.kv_heads * a.group) + c.head * a.group + hh;
    const float up = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row_at * DIM + d) =
        uint2{Half<BF16>::round2(v[0] * up, v[1] * up), Half<BF16>::round2(v[2] * up, v[3] * up)};
    if (d == 0 && a.lse) a.lse[row_at] = l == 0.f ? -__builtin_inff() : (__builtin_amdgcn_logf(l) + mx) * kLn2;
  }
}

template <int DIM, bool BF16>
hipError_t launch_as(const ChunkParams& a, hipStream_t stream) {
  const uint32_t grid = a.groups ? a.groups : static_cast<uint32_t>(a.tiles) * a.kv_heads;
  kv4_chunk_kernel<DIM, BF16><<<dim3(grid), dim3(kThreads), 0, stream>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.groups == 0) return e;
  kv4_chunk_join_kernel<DIM, BF16><<<dim3(static_cast<uint32_t>(a.groups)), dim3(kJoinWaves * 64), 0, stream>>>(a);
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_dim(int dim, const ChunkParams& a, hipStream_t stream) {
  switch (dim) {
    case 64: return launch_as<64, BF16>(a, stream);
    case 128: return launch_as<128, BF16>(a, stream);
    case 256: return launch_as<256, BF16>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_kv4_chunk(const qpn_kv4_cache& c, const qpn_kv4_chunk_args& x, const ChunkPlan& p, void* workspace,
                            hipStream_t stream) {
  ChunkParams a;
  a.page_bytes = static_cast<int64_t>(qpn_kv4_page_bytes(c.page_size, c.kv_heads, c.head_dim));
  a.cache = static_cast<const uint8_t*>(c.data) + a.page_bytes * c.pages * x.layer;
  a.pages = static_cast<int32_t>(c.pages);
  a.page_shift = __builtin_ctz(c.page_size);
  a.seg_bytes = static_cast<int32_t>(kv4_segment_bytes(c.page_size, c.head_dim));
  a.kv_heads = c.kv_heads;
  a.group = x.heads / c.kv_heads;
  a.q = x.q, a.k = x.k, a.v = x.v;
  a.q_ts = x.q_token_stride, a.q_hs = x.q_head_stride;
  a.k_ts = x.k_token_stride, a.k_hs = x.k_head_stride;
  a.v_ts = x.v_token_stride, a.v_hs = x.v_head_stride;
  a.out = x.out, a.lse = x.lse;
  a.table = x.table, a.table_stride = x.table_stride;
  a.kv_len = x.kv_len, a.q_start = x.q_start;
  a.batch = x.batch, a.rows = x.rows, a.max_q = x.max_q_len < x.rows ? x.max_q_len : x.rows;
  constexpr int kWindow = (1 << 30) + (1 << 21);  // no position is above 2^30 + 2^20, and one less this stays inside 32 bits
  a.max_kv = x.max_kv_len, a.window = x.window < kWindow ? x.window : kWindow;
  a.tiles = p.tiles, a.groups = p.groups;
  a.f = std::min(x.scale * kLog2e, kMost), a.k_scale = c.k_scale, a.v_scale = c.v_scale;
  a.cuts = static_cast<Cut*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + p.cut_bytes);
  return x.dtype == QPN_DT_BF16 ? launch_dim<true>(c.head_dim, a, stream) : launch_dim<false>(c.head_dim, a, stream);
}

}  // namespace qpn
