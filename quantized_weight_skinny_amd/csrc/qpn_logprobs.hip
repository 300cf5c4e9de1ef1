// Log-probabilities of given tokens, entropies and the first tokens of rows of
// logits (include/qpn_prompt.h).
//
// Mathematics. With f = log2(e) / t and a reference m, a lane keeps
// s = sum 2^((x - m) f) and w = sum 2^((x - m) f) (x - m) f over its elements in
// one pass; a larger m' scales them by d = 2^((m - m') f), after w has been
// given (m - m') f times s. Then log2 p = (x - m) f - log2 s, and the entropy
// is log2 s - w / s, both times ln 2. A lane adds 128 elements at most in 32 bits
// before they go to its sums of 64, in which wavefronts and slices of a row are added, too.
//
// The first tokens are found in the same pass. Every wavefront keeps a list of
// candidates above a bound, which at least `top` of the slice's elements so far
// reach; a wavefront's elements come in the order of their index, so a later one
// that equals the bound comes after these. The first bound is the top-th largest of
// all lanes' maxima over the slice's first 4096 elements: a fourth of the candidates
// follow that bounds from a wavefront's own 1024 would let through (64 rows of 50021
// with 64 first tokens 26 us, with such bounds 39; 255 of 151936 with twenty 49 and
// 57). A list is cut back to `top` (by a search over the keys' bits, with votes)
// when it passes twice that, which raises the bound. Rising rows, whose every
// element passes, cost more and are no less right.
//
// What bounds it: some 16 vector instructions an element, exponential and
// comparisons among them: 2048 rows of 151936 bf16 with five first tokens 150 to 190
// us, 3.3 to 4.1 TB/s, where the bytes alone take 101. Small calls are two launches and
// their latency: one row of 151936 with twenty 18 us (8.0 + 10.5 for the kernels), 37
// of 50021 fp32 16 us (5.0 + 3.9).
#include "qpn_decode_internal.hpp"
#include "qpn_device.hpp"
#include "qpn_prompt_internal.hpp"

namespace qpn {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kEach = kLogprobsStep / kThreads;  // elements a lane takes at a time
// Such steps whose sums are 32 bits: of 128 elements (2048 rows of 151936, 37 steps, 167.2 us; all
// of a row's in 32 bits 166.4).
constexpr int kFlush = 8;
constexpr int kList = 128;               // candidates that a wavefront keeps
constexpr int kShort = 80;               // ... and those that a cut leaves
constexpr int kAtOnce = 8 * 64;          // ... and what it may add before it looks
constexpr int kKeys = (kList + kAtOnce) / 64;
typedef u4 u4_anywhere __attribute__((aligned(2)));
constexpr float kLowest = -3.402823466e38f;

struct Stat {
  double sum, dot;  // s and w under the reference max
  float max;
  int before;       // elements that come before the given token
};
static_assert(sizeof(Stat) == 24, "the workspace holds 24 bytes a slice");

struct LogprobsParams {
  qpn_logprobs_args a;
  int slices, length;  // of a row, and a slice's elements
  Stat* stats;         // [rows][slices]
  uint64_t* lists;     // [rows][slices][top]: keys in descending order, 0 past the last
};

struct Bf16 {
  uint16_t bits;
};
template <typename T>
__device__ __forceinline__ float widen(T x) {
  if constexpr (sizeof(T) == 4) return x;
  else if constexpr (__is_same(T, Bf16)) return widen16<true>(x.bits);
  else return static_cast<float>(x);
}

// A lane's 16 bytes of elements as fp32. (Made quiet once here: a maximum of a
// signalling NaN would be NaN, and the compiler quiets each operand it does not know.)
template <typename T>
__device__ __forceinline__ void widen_piece(const u4& w, float* x) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __builtin_canonicalizef(__uint_as_float(w[e]));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __builtin_canonicalizef(widen16<__is_same(T, Bf16)>(w[e] & 0xFFFFu));
      x[2 * e + 1] = __builtin_canonicalizef(widen16<__is_same(T, Bf16)>(w[e] >> 16));
    }
  }
}

// Larger keys come first: the logit's order (-0 as 0, NaN as -inf), then the lower index.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x == x ? x + 0.0f : -__builtin_inff());
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t order) {
  return __uint_as_float(order ^ ((order & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ uint64_t key_of(float x, int index) {
  return static_cast<uint64_t>(order_of(x)) << 32 | ~static_cast<uint32_t>(index);
}
constexpr uint32_t kMinusInf = 0x007FFFFFu;  // order_of(-inf)

// Cuts a wavefront's list of n keys (all different, 0: none; 64 KEYS at most) back to the `top` largest, or
// some more, kShort at most; top <= n. Returns the order of a bound that at least `top`
// of them reach and all that stay. The bound is found bit by bit from above: 16
// bits of the logits' order tell most lists apart, the index those of equal logits.
template <int KEYS>
__device__ __forceinline__ uint32_t cut_list(uint64_t* list, int& n, int top) {
  const int lane = threadIdx.x & 63;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the list holds other lanes' keys
  uint64_t key[KEYS];
#pragma unroll
  for (int j = 0; j < KEYS; ++j) key[j] = j * 64 + lane < n ? list[j * 64 + lane] : 0;
  const auto reach = [&](uint64_t x) {
    int count = 0;
#pragma unroll
    for (int j = 0; j < KEYS; ++j) {
      if (j * 64 >= n) break;
      count += __popcll(__ballot(key[j] >= x));
    }
    return count;
  };
  uint64_t bound = 0;
#pragma unroll 1
  for (int bit = 63; bit >= 0; --bit) {
    const uint64_t next = bound | uint64_t(1) << bit;
    if (reach(next) >= top) bound = next;
    if ((bit & 15) == 0 && reach(bound) <= kShort) break;
  }
  bound = max(bound, uint64_t(1));  // (places without a key go, too)
  int at = 0;
#pragma unroll
  for (int j = 0; j < KEYS; ++j) {
    if (j * 64 >= n) break;
    const uint64_t stays = __ballot(key[j] >= bound);
    const int mine = at + __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(stays >> 32),
                                                    __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(stays), 0));
    if (key[j] >= bound) list[mine] = key[j];
    at += __popcll(stays);
  }
  n = at;
  return static_cast<uint32_t>(bound >> 32);
}

// Adds the lanes' keys where `take` to the wavefront's list.
__device__ __forceinline__ void add_keys(uint64_t* list, int& n, bool take, uint64_t key) {
  const uint64_t all = __ballot(take);
  if (take)
    list[n + __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(all >> 32),
                                       __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(all), 0))] = key;
  n += __popcll(all);
}

// The wavefronts' lists (counts[w] keys each) as one, in descending order: `put`
// gets each key among the first `top` and its place. Returns how many there are.
template <typename Put>
__device__ __forceinline__ int merge_lists(const uint64_t (*lists)[kList + kAtOnce], const int* counts, int top, Put put) {
  int total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) total += counts[w];
#pragma unroll 1
  for (int mine = threadIdx.x; mine < total; mine += kThreads) {
    int w = 0, at = mine;
    while (at >= counts[w]) at -= counts[w++];
    const uint64_t key = lists[w][at];
    int place = 0;
#pragma unroll 1
    for (int o = 0; o < kWaves; ++o) {
      const int n = counts[o];
#pragma unroll 8
      for (int j = 0; j < n; ++j) place += lists[o][j] > key;
    }
    if (place < top) put(key, place);
  }
  return min(total, top);
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) x = fmaxf(x, __shfl_xor(x, o));
  return x;
}
__device__ __forceinline__ double wave_add(double x) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o);
  return x;
}

__device__ __forceinline__ float factor_of(const LogprobsParams& p, int row) {
  const float t = p.a.temperature ? p.a.temperature[row] : 1.0f;
  return fminf(1.44269504088896341f / (t > 0.f ? t : 1.0f), -kLowest);
}

// 2^((x - m) f), and the exponent: 0 for x of -inf and NaN, whatever m and f.
__device__ __forceinline__ float weight(float x, float m, float f, float& t) {
  t = fmaxf((x - m) * f, -1000.0f);
  return __builtin_amdgcn_exp2f(t);
}

// s and w under another reference, d = (m - m') f of 0 or below (2^-1000 is 0).
template <typename F>
__device__ __forceinline__ void move_reference(F& s, F& w, float d) {
  d = fmaxf(d, -1000.0f);  // (also of inf - inf)
  const float down = __builtin_amdgcn_exp2f(d);
  w = down > 0.f ? (w + s * d) * down : F(0);
  s *= down;
}

// One slice of one row.
template <typename T, bool TOP>
__global__ __launch_bounds__(kThreads) void logprobs_slices_kernel(const LogprobsParams p) {
  constexpr int kPiece = 16 / sizeof(T), kPieces = kEach / kPiece;
  __shared__ Stat joined[kWaves];
  __shared__ uint64_t lists[TOP ? kWaves : 1][kList + kAtOnce];
  __shared__ int counts[kWaves];
  __shared__ uint32_t maxima[TOP ? kThreads : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int row = blockIdx.x / p.slices, slice = blockIdx.x - row * p.slices;
  const T* x0 = static_cast<const T*>(p.a.logits) + row * p.a.row_stride;
  const int begin = slice * p.length, end = min(begin + p.length, p.a.vocab);
  u4 raw[kPieces];
  constexpr int kWaveStep = kEach * 64;
  const auto load = [&](int at) {
    const T* from = x0 + at + lane * kPiece;
    if (at + kWaveStep <= end) {
#pragma unroll
      for (int j = 0; j < kPieces; ++j) raw[j] = *reinterpret_cast<const u4_anywhere*>(from + j * 64 * kPiece);
    } else {
#pragma unroll
      for (int j = 0; j < kPieces; ++j)
        if (at + (j * 64 + lane + 1) * kPiece <= end) raw[j] = *reinterpret_cast<const u4_anywhere*>(from + j * 64 * kPiece);
    }
  };
  const int at0 = begin + wave * kWaveStep;
  if (at0 < end) load(at0);
  const float f = factor_of(p, row);
  const int token = p.a.tokens ? p.a.tokens[row] : -1;
  const bool given = token >= 0 && token < p.a.vocab;
  // An element comes before the token where it is at least the token's logit
  // (in front of it) or larger (behind it).
  float reach = __builtin_inff(), above = __builtin_inff();
  if (given) {
    reach = value_of(order_of(widen<T>(x0[token])));
    above = reach == __builtin_inff() ? __builtin_nanf("") : value_of(order_of(reach) + 1);
    // (of -inf, all in front: the rows' kernel adds them, NaN among them)
    if (reach == -__builtin_inff()) reach = __builtin_nanf("");
  }
  float m = kLowest, s = 0.f, w = 0.f;
  float m_sum = kLowest;  // the reference of sum and dot
  double sum = 0.0, dot = 0.0;
  int before = 0, n = 0, steps = 0;
  float bound = -__builtin_inff();
  bool first = true;
  uint64_t* list = lists[TOP ? wave : 0];
  // (a short list is cut by a hundred instructions, and a bound that rises early spares most steps)
  const int enough = min(2 * p.a.top + 8, kList);

  const auto flush = [&] {
    move_reference(sum, dot, (m_sum - m) * f);
    sum += s, dot += w;
    m_sum = m, s = 0.f, w = 0.f, steps = 0;
  };
  // (each wavefront takes a first step, of -inf alone where it has no elements)
  for (int at = at0; at < end || (TOP && first); at += kWaveStep * kWaves) {
    float x[kEach];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) widen_piece<T>(raw[j], &x[j * kPiece]);
    if (at + kWaveStep > end) {
      // the end of the slice: what is past it is -inf, a piece across it comes one by one
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const int e0 = at + j * 64 * kPiece + lane * kPiece;
        if (e0 + kPiece > end) {
#pragma unroll
          for (int e = 0; e < kPiece; ++e) x[j * kPiece + e] = e0 + e < end ? widen<T>(x0[e0 + e]) : -__builtin_inff();
        }
      }
    }
    if (at + kWaveStep * kWaves < end) load(at + kWaveStep * kWaves);
    float most = x[0];
#pragma unroll
    for (int e = 1; e < kEach; ++e) most = fmaxf(most, x[e]);
    const float top = fmaxf(m, most);
    if (__any(top > m)) {
      move_reference(s, w, (m - top) * f);
      m = top;
    }
    const auto index = [&](int e) { return at + e / kPiece * (64 * kPiece) + lane * kPiece + e % kPiece; };
    const bool mixed = token >= at && token < at + kWaveStep;
    const float least = at > token ? above : reach;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      float t;
      const float y = weight(x[e], m, f, t);
      s += y;
      w = fmaf(y, t, w);
    }
    if (++steps == kFlush) flush();
    // (for a likely token, most steps hold none that comes before it)
    if (mixed) {
#pragma unroll
      for (int e = 0; e < kEach; ++e) before += x[e] >= (index(e) >= token ? above : reach);
    } else if (__any(most >= least)) {
#pragma unroll
      for (int e = 0; e < kEach; ++e) before += x[e] >= least;
    }
    if constexpr (TOP) {
      bool equal = false;  // elements that equal the bound count
      if (first) {
        // the upper 16 bits of the top-th largest of all lanes' maxima
        maxima[threadIdx.x] = order_of(most);
        __syncthreads();
        uint32_t each[kWaves];
#pragma unroll
        for (int o = 0; o < kWaves; ++o) each[o] = maxima[o * 64 + lane];
        uint32_t b = 0;
#pragma unroll 1
        for (int bit = 31; bit >= 16; --bit) {
          const uint32_t next = b | 1u << bit;
          int reached = 0;
#pragma unroll
          for (int o = 0; o < kWaves; ++o) reached += static_cast<int>(__popcll(__ballot(each[o] >= next)));
          if (reached >= p.a.top) b = next;
        }
        if (b > kMinusInf) bound = value_of(b), equal = true;
        first = false;
      }
      if (__any(equal ? most >= bound : most > bound)) {
#pragma unroll
        for (int part = 0; part < kEach / 8; ++part) {
          // (the eight elements of a part lie in front of the next part's for all lanes)
          const float* y = &x[part * 8];
          float z = y[0];
#pragma unroll
          for (int e = 1; e < 8; ++e) z = fmaxf(z, y[e]);
          if (!__any(equal ? z >= bound : z > bound)) continue;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const bool take = equal ? y[e] >= bound : y[e] > bound;
            if (__any(take)) add_keys(list, n, take, key_of(y[e], index(part * 8 + e)));
          }
          if (n > enough) {
            bound = value_of(cut_list<kKeys>(list, n, p.a.top));
            equal = false;
          }
        }
      }
    }
  }

  // Lanes, then wavefronts.
  flush();
  const float most = wave_max(m);
  move_reference(sum, dot, (m - most) * f);
  sum = wave_add(sum), dot = wave_add(dot);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) before += __shfl_xor(before, o);
  if (lane == 0) {
    joined[wave] = Stat{sum, dot, most, before};
    counts[wave] = n;
  }
  __syncthreads();
  const int64_t at = static_cast<int64_t>(row) * p.slices + slice;
  if (threadIdx.x == 0) {
    Stat r = joined[0];
#pragma unroll
    for (int o = 1; o < kWaves; ++o) {
      Stat y = joined[o];
      const float top = fmaxf(r.max, y.max);
      move_reference(r.sum, r.dot, (r.max - top) * f);
      move_reference(y.sum, y.dot, (y.max - top) * f);
      r = Stat{r.sum + y.sum, r.dot + y.dot, top, r.before + y.before};
    }
    p.stats[at] = r;
  }
  if constexpr (TOP) {
    uint64_t* out = p.lists + at * p.a.top;
    const int found = merge_lists(lists, counts, p.a.top, [&](uint64_t key, int place) { out[place] = key; });
    for (int j = found + threadIdx.x; j < p.a.top; j += kThreads) out[j] = 0;
  }
}

// A row's slices as one, and its results.
template <typename T, bool TOP>
__global__ __launch_bounds__(kThreads) void logprobs_rows_kernel(const LogprobsParams p) {
  __shared__ uint64_t keys[TOP ? kLogprobsKeys : 1], first[TOP ? 64 : 1];
  __shared__ int infinite, found, left;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int row = blockIdx.x;
  const T* x0 = static_cast<const T*>(p.a.logits) + row * p.a.row_stride;
  // (asked for early: each of these waits for the one before)
  const int token = p.a.tokens ? p.a.tokens[row] : -1;
  const float given_t = p.a.temperature ? p.a.temperature[row] : 1.0f;
  const bool given = token >= 0 && token < p.a.vocab;
  const float given_x = given ? widen<T>(x0[token]) : 0.f;
  const float f = factor_of(p, row);
  if (threadIdx.x == 0) infinite = 0, found = 0;
  // every wavefront adds all slices
  Stat r{0.0, 0.0, kLowest, 0};
  for (int c = lane; c < p.slices; c += 64) {
    Stat y = p.stats[static_cast<int64_t>(row) * p.slices + c];
    const float top = fmaxf(r.max, y.max);
    move_reference(r.sum, r.dot, (r.max - top) * f);
    move_reference(y.sum, y.dot, (y.max - top) * f);
    r = Stat{r.sum + y.sum, r.dot + y.dot, top, r.before + y.before};
  }
  const float most = wave_max(r.max);
  move_reference(r.sum, r.dot, (r.max - most) * f);
  r.sum = wave_add(r.sum), r.dot = wave_add(r.dot), r.max = most;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) r.before += __shfl_xor(r.before, o);
  const int total = p.slices * p.a.top;
  if constexpr (TOP) {
    const uint64_t* in = p.lists + static_cast<int64_t>(row) * total;
    for (int j = threadIdx.x; j < total; j += kThreads) keys[j] = in[j];
  }
  __syncthreads();
  if (r.max == __builtin_inff()) {
    // infinite logits share the probability
    int count = 0;
    for (int e = threadIdx.x; e < p.a.vocab; e += kThreads) count += widen<T>(x0[e]) == __builtin_inff();
    if (count) atomicAdd(&infinite, count);
    __syncthreads();
    r.sum = infinite, r.dot = 0.0;
  }
  // log p = ((x - max) / t) - ln s
  const double t = given_t > 0.f ? given_t : 1.0f, log_sum = r.sum > 0.0 ? log(r.sum) : 0.0;
  const auto log_p = [&](float x) -> float {
    if (!(x > -__builtin_inff())) return -__builtin_inff();
    if (x == r.max) return static_cast<float>(-log_sum);
    return static_cast<float>((static_cast<double>(x) - static_cast<double>(r.max)) / t - log_sum);
  };
  if (threadIdx.x == 0) {
    if (p.a.logprobs) p.a.logprobs[row] = given ? log_p(given_x) : 0.f;
    // (all in front of a logit of -inf or NaN come before it)
    if (p.a.rank) p.a.rank[row] = given ? r.before + (given_x > -__builtin_inff() ? 0 : token) : -1;
    if (p.a.entropy) p.a.entropy[row] = r.sum > 0.0 ? static_cast<float>(fmax(log_sum - r.dot / r.sum * 0.69314718055994530942, 0.0)) : 0.f;
  }
  if constexpr (TOP) {
    // the first `top` of all slices', or some more
    if (wave == 0) {
      int n = total;
      if (p.slices > 1) cut_list<kLogprobsKeys / 64>(keys, n, p.a.top);
      if (lane == 0) left = n;
    }
    __syncthreads();
    for (int j = threadIdx.x; j < left; j += kThreads) {
      const uint64_t key = keys[j];
      int place = 0;
#pragma unroll 8
      for (int i = 0; i < left; ++i) place += keys[i] > key;
      if (key != 0 && place < p.a.top) {
        first[place] = key;
        atomicAdd(&found, 1);
      }
    }
    __syncthreads();
    // fewer tokens than asked for are above -inf: the others in the order of their index
    if (found < p.a.top && wave == 0) {
      int n = found;
      for (int e0 = 0; e0 < p.a.vocab && n < p.a.top; e0 += 64) {
        const bool low = e0 + lane < p.a.vocab && !(widen<T>(x0[e0 + lane]) > -__builtin_inff());
        const uint64_t all = __ballot(low);
        const int place = n + __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(all >> 32),
                                                        __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(all), 0));
        if (low && place < p.a.top) first[place] = key_of(-__builtin_inff(), e0 + lane);
        n += __popcll(all);
      }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < p.a.top; j += kThreads) {
      const int64_t at = static_cast<int64_t>(row) * p.a.top + j;
      p.a.top_tokens[at] = static_cast<int32_t>(~static_cast<uint32_t>(first[j]));
      p.a.top_logprobs[at] = log_p(value_of(static_cast<uint32_t>(first[j] >> 32)));
    }
  }
}

template <typename T>
hipError_t launch_as(const LogprobsParams& p, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(p.a.rows) * p.slices), rows(static_cast<uint32_t>(p.a.rows));
  if (p.a.top > 0) {
    logprobs_slices_kernel<T, true><<<grid, dim3(kThreads), 0, stream>>>(p);
  } else {
    logprobs_slices_kernel<T, false><<<grid, dim3(kThreads), 0, stream>>>(p);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.a.top > 0) {
    logprobs_rows_kernel<T, true><<<rows, dim3(kThreads), 0, stream>>>(p);
  } else {
    logprobs_rows_kernel<T, false><<<rows, dim3(kThreads), 0, stream>>>(p);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_token_logprobs(const qpn_logprobs_args& a, const LogprobsPlan& plan, void* workspace,
                                 hipStream_t stream) {
  LogprobsParams p;
  p.a = a;
  p.slices = plan.slices, p.length = plan.length;
  p.stats = static_cast<Stat*>(workspace);
  p.lists = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(workspace) + plan.stat_bytes);
  switch (a.dtype) {
    case QPN_DT_F16: return launch_as<_Float16>(p, stream);
    case QPN_DT_BF16: return launch_as<Bf16>(p, stream);
    default: return launch_as<float>(p, stream);
  }
}

}  // namespace qpn
