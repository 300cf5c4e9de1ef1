// Verification of drafted tokens (include/qpn_decode.h).
//
// One pass over all rows of logits takes each row's maximum, its lowest index
// and the sum of exponentials (32-bit exponentials, 64-bit sums of them):
// that is all the accept tests need. Only one row a sequence (two with a
// draft) is then read again, for the place of u_sample among the running
// sums. A vocabulary's running sums lie closer together than 32 bits tell
// apart, so these weights and sums are 64-bit, a chunk a workgroup: the chunk
// sums of p and q; then, for a rejected draft with a row of its own, those of
// max(p - q, 0), for which both totals must be known; then one workgroup a
// sequence finds the chunk and the token in it.
//
// These kernels are short, and most of their time is latency. For few
// sequences the accept tests are repeated by every workgroup of the second
// pass, 16 wavefronts for its rows at once, instead of taking a launch. (The
// last workgroup of each row and sequence, found by a counter, making them in
// the first pass measured 13.6 us instead of 5.0 for 8 rows, and 52 instead of
// 32 for 480: the counter's round trip is added to every workgroup.) And a
// launch fetches each line of its code from memory, so a kernel of few
// workgroups holds one copy of the 64-bit exponential, in a loop (4 us of the
// last pass, when that took 16.8).
//
// Measured, fp16, 151936 tokens. 1 sequence of 7 drafts without rows: first
// pass 4.8 us, sums 7.4, last pass 6.9; 32 such sequences with draft logits:
// 31.5 (146 MB, 4.6 TB/s), accept tests 5.2, sums 18.7, rest 16.8, last 10.9.
#include "qpn_decode_internal.hpp"
#include "qpn_device.hpp"

namespace qpn {
namespace {

constexpr int kT = 256;          // threads of the first pass
constexpr int kChunk = 4096;     // elements a workgroup takes of a row
constexpr int kPer = kChunk / kT;
constexpr int kD = 1024;         // threads of the passes that draw
constexpr int kDrawPer = kChunk / kD;
constexpr int kDrawWaves = kD / 64;
constexpr int kMaxDrafts = 64;
typedef u4 u4_anywhere __attribute__((aligned(2)));

struct Stat {
  float max;
  int idx;
  double sum;
};
static_assert(sizeof(Stat) == 16, "the workspace holds 16 bytes a chunk");

// Running sums over a wavefront's lanes by data-parallel moves (lane l gets
// the value of lane l - n of its row of 16, then of the rows before): six
// steps of three instructions, against two trips through LDS each for a
// shuffled 64-bit value.
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double x) {
  const long long b = __builtin_bit_cast(long long, x);
  const int lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, ROWS, 0xF, false);
  const int hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, static_cast<unsigned long long>(static_cast<uint32_t>(hi)) << 32 |
                                        static_cast<uint32_t>(lo));
}
__device__ __forceinline__ double wave_scan(double x) {
  x += moved<0x111, 0xF>(x);  // one lane up in the row
  x += moved<0x112, 0xF>(x);  // two
  x += moved<0x114, 0xF>(x);  // four
  x += moved<0x118, 0xF>(x);  // eight
  x += moved<0x142, 0xA>(x);  // the last lane of rows 0 and 2, to rows 1 and 3
  x += moved<0x143, 0xC>(x);  // lane 31, to rows 2 and 3
  return x;
}
__device__ __forceinline__ double lane_value(double x, int l) {
  const long long b = __builtin_bit_cast(long long, x);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(b), l);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(b >> 32), l);
  return __builtin_bit_cast(double, static_cast<unsigned long long>(hi) << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double x) { return lane_value(wave_scan(x), 63); }

// What the accept tests leave to the passes that draw a token.
enum : int { kDone = 0, kFromP = 1, kFromRest = 2 };
struct Verdict {
  int accepted, how;
  int skip;             // the rejected draft, struck from p where no draft row is given; -1: none
  float t;              // the temperature (1 for probabilities)
  float p_max, q_max;   // maxima of the rows that the token is picked from
  int pad[2];
};
static_assert(sizeof(Verdict) == 32, "the workspace holds 32 bytes a sequence");

struct VerifyParams {
  qpn_verify_args a;
  int chunks, decided;
  Verdict* verdicts;  // [batch]
  Stat* stats;        // [batch][drafts + 1][chunks], then [batch][drafts][chunks]
  double* sums;       // [batch][3][chunks]: of p, of q, of what q leaves over
};

template <typename T>
__device__ __forceinline__ float widen(T x);
template <>
__device__ __forceinline__ float widen<_Float16>(_Float16 x) { return static_cast<float>(x); }
template <>
__device__ __forceinline__ float widen<float>(float x) { return x; }
struct Bf16 {
  uint16_t bits;
};
template <>
__device__ __forceinline__ float widen<Bf16>(Bf16 x) { return widen16<true>(x.bits); }

// A logit as it counts: NaN as -inf.
template <typename T>
__device__ __forceinline__ float logit(T x) {
  const float v = widen<T>(x);
  return v == v ? v : -__builtin_inff();
}

// A probability as it counts: NaN and negative as 0.
__device__ __forceinline__ double probability(float x) { return x > 0.f ? static_cast<double>(x) : 0.0; }

// e^x for x <= 0 in 64 bits: x = n ln 2 + r, |r| <= ln(2) / 2, the Taylor sum
// of e^r to r^13 / 13! (its rest is below 2^-57), and a shift of the exponent. Twenty
// instructions, against the library's checks for arguments that do not occur.
// n ln 2 is taken off in two parts (the reduction of Cody and Waite, Software
// Manual for the Elementary Functions, 1980): ln 2 rounded to 40 places after
// the point, whose product with n, at most 11 bits, is exact, and what is left.
__device__ __forceinline__ double exp64(double x) {
  constexpr double kLn2 = 762123384786.0 / 1099511627776.0, kLn2Rest = -1.7239444525614835e-13;
  x = fmax(x, -800.0);
  const double n = rint(x * 1.4426950408889634074);
  double r = fma(n, -kLn2, x);
  r = fma(n, -kLn2Rest, r);
  double p = 1.0 / 6227020800.0;
  p = fma(p, r, 1.0 / 479001600.0);
  p = fma(p, r, 1.0 / 39916800.0);
  p = fma(p, r, 1.0 / 3628800.0);
  p = fma(p, r, 1.0 / 362880.0);
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return ldexp(p, static_cast<int>(n));
}

// e^((x - max) / t): 1 at the maximum (also an infinite one), 0 at -inf.
__device__ __forceinline__ double weight(float x, float max, double inv_t) {
  if (x == -__builtin_inff()) return 0.0;
  return x == max ? 1.0 : exp64((static_cast<double>(x) - static_cast<double>(max)) * inv_t);
}

// (max, lowest index of it), folded over lanes that are `o` apart.
__device__ __forceinline__ void fold_max(float& m, int& idx, int o) {
  const float m2 = __shfl_xor(m, o);
  const int i2 = __shfl_xor(idx, o);
  if (m2 > m || (m2 == m && i2 < idx)) m = m2, idx = i2;
}

template <typename T>
__device__ __forceinline__ const T* target_row(const VerifyParams& p, int b, int i) {
  return static_cast<const T*>(p.a.target) + b * p.a.target_batch_stride + i * p.a.target_row_stride;
}
template <typename T>
__device__ __forceinline__ const T* draft_row(const VerifyParams& p, int b, int i) {
  return static_cast<const T*>(p.a.draft) + b * p.a.draft_batch_stride + i * p.a.draft_row_stride;
}

__device__ __forceinline__ int drafts_of(const VerifyParams& p, int b) {
  return p.a.num_draft ? min(max(p.a.num_draft[b], 0), p.a.drafts) : p.a.drafts;
}
// 0: greedy
__device__ __forceinline__ float temperature_of(const VerifyParams& p, int b) {
  const float t = p.a.temperature ? p.a.temperature[b] : 1.0f;
  return t > 0.f ? t : 0.f;
}

// log x for x > 0, to 32 bits.
__device__ __forceinline__ float log_of(double x) {
  const float m = __builtin_amdgcn_logf(static_cast<float>(__builtin_amdgcn_frexp_mant(x)));
  return (static_cast<float>(__builtin_amdgcn_frexp_exp(x)) + m) * 0.69314718055994531f;
}

// One row's chunks as one, by a wavefront (all its lanes return it).
__device__ __forceinline__ Stat join_stats(const Stat* s, int chunks, float scale) {
  const int lane = threadIdx.x & 63;
  Stat r{-__builtin_inff(), 0x7FFFFFFF, 0.0};
  // e^((x - m) / t) for two maxima; 0 for -inf, also under -inf
  const auto ratio = [&](float x, float m) {
    return x == -__builtin_inff() ? 0.f : x == m ? 1.f : __builtin_amdgcn_exp2f((x - m) * scale);
  };
#pragma unroll 1
  for (int c = lane; c < chunks; c += 64) {
    const Stat x = s[c];
    const float m = fmaxf(r.max, x.max);
    r.sum = r.sum * ratio(r.max, m) + x.sum * ratio(x.max, m);
    if (x.max > r.max || (x.max == r.max && x.idx < r.idx)) r.idx = x.idx;
    r.max = m;
  }
  const float mine = r.max;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) fold_max(r.max, r.idx, o);
  r.sum = wave_sum(r.sum * ratio(mine, r.max));
  return r;
}

// The accept tests of sequence b, its rows joined a wavefront each, then one
// thread a draft; and (where `write`) the verdict and the outputs that follow:
// all but the place of a token that is still to be drawn.
template <typename T, bool PROBS>
__device__ Verdict decide(const VerifyParams& p, int b, bool write) {
  __shared__ int rejected_at;
  __shared__ Stat p_rows[kMaxDrafts + 1], q_rows[kMaxDrafts];
  const int n = drafts_of(p, b);
  const float t = PROBS ? 1.f : temperature_of(p, b);
  const int tid = threadIdx.x, places = p.a.drafts + 1;
  const double inv_t = 1.0 / (t > 0.f ? t : 1.f);
  // a draft's token, its logits and its number are on their way while the rows are joined
  const bool with_q = p.a.draft && t > 0.f;  // (a greedy sequence has no use for the draft's rows)
  int d = -1;
  float u = 0.f;
  float x_p = 0.f, x_q = 0.f;
  if (tid < n) {
    const int64_t at = static_cast<int64_t>(b) * p.a.drafts + tid;
    d = p.a.draft_tokens[at];
    u = p.a.u_accept[at];
    if (d >= 0 && d < p.a.vocab) {
      x_p = widen<T>(target_row<T>(p, b, tid)[d]);
      if (with_q) x_q = widen<T>(draft_row<T>(p, b, tid)[d]);
    }
  }
  if constexpr (!PROBS) {
    const float scale = 1.44269504088896341f / (t > 0.f ? t : 1.f);
    const int rows = n + 1 + (with_q ? n : 0);
#pragma unroll 1
    for (int r = tid >> 6; r < rows; r += kDrawWaves) {
      const int64_t row = r <= n ? static_cast<int64_t>(b) * places + r
                                 : static_cast<int64_t>(p.a.batch) * places + static_cast<int64_t>(b) * p.a.drafts +
                                       (r - n - 1);
      const Stat x = join_stats(p.stats + row * p.chunks, p.chunks, scale);
      if ((tid & 63) == 0) (r <= n ? p_rows[r] : q_rows[r - n - 1]) = x;
    }
  }
  if (tid == 0) rejected_at = n;
  __syncthreads();
  double pd = 0.0;  // p of the draft
  if (tid < n) {
    bool ok = false;
    if (d >= 0 && d < p.a.vocab) {
      double qd = 1.0;
#pragma unroll 1
      for (int k = 0; k < (with_q ? 2 : 1); ++k) {
        const float x = k ? x_q : x_p;
        double y;
        if constexpr (PROBS) {
          y = probability(x);
        } else {
          const Stat r = (k ? q_rows : p_rows)[tid];
          y = r.sum > 0.0 ? weight(x == x ? x : -__builtin_inff(), r.max, inv_t) / r.sum : 0.0;
        }
        if (k) qd = y;
        else pd = y;
      }
      ok = static_cast<double>(u) * qd < pd;
      if constexpr (!PROBS)
        if (t == 0.f) ok = p_rows[tid].idx == d;
    }
    if (!ok) atomicMin(&rejected_at, tid);
  }
  __syncthreads();
  const int accepted = rejected_at;
  Verdict v{accepted, kFromP, -1, t > 0.f ? t : 1.f, 0.f, 0.f, {0, 0}};
  int token = -1;
  double token_p = 1.0;
  if constexpr (!PROBS) {
    const Stat r = p_rows[accepted];
    v.p_max = r.max;
    if (t == 0.f || r.max == -__builtin_inff()) {
      v.how = kDone;
      if (r.max > -__builtin_inff()) token = r.idx, token_p = 1.0 / r.sum;
    }
  }
  if (accepted < n && v.how != kDone) {
    if (p.a.draft) {
      v.how = kFromRest;
      if constexpr (!PROBS) v.q_max = q_rows[accepted].max;
    } else {
      v.skip = p.a.draft_tokens[static_cast<int64_t>(b) * p.a.drafts + accepted];
    }
  }
  if (write && tid < places && (tid != accepted || v.how == kDone)) {
    const int64_t at = static_cast<int64_t>(b) * places + tid;
    p.a.tokens[at] = tid < accepted ? d : tid == accepted ? token : -1;
    if (p.a.logprobs)
      p.a.logprobs[at] = log_of(tid < accepted ? pd : tid == accepted ? token_p : 1.0);
  }
  if (write && tid == 0) {
    p.a.accepted[b] = accepted;
    p.verdicts[b] = v;
  }
  return v;
}

// Maximum and sum of exponentials of one chunk of one row, read in 16-byte
// vectors from wherever the row begins: the chunks, and so the bits of the
// result, do not depend on a row's place in memory.
template <typename T>
__global__ __launch_bounds__(kT) void verify_rows_kernel(const VerifyParams p, int target_rows) {
  constexpr int kVec = 16 / sizeof(T), kLoads = kPer / kVec;
  __shared__ float wmax[kT / 64];
  __shared__ int widx[kT / 64];
  __shared__ double wsum[kT / 64];
  const int row = blockIdx.x / p.chunks, c = blockIdx.x - row * p.chunks;
  const bool is_target = row < target_rows;
  const int b = is_target ? row / (p.a.drafts + 1) : (row - target_rows) / p.a.drafts;
  const int i = is_target ? row - b * (p.a.drafts + 1) : row - target_rows - b * p.a.drafts;
  const int n = drafts_of(p, b);
  const float t = temperature_of(p, b);
  // (a greedy sequence does not use its draft's logits)
  if (is_target ? i > n : i >= n || t == 0.f) return;
  const T* src = is_target ? target_row<T>(p, b, i) : draft_row<T>(p, b, i);
  const float scale = 1.44269504088896341f / (t > 0.f ? t : 1.f);
  float x[kPer];
  float m = -__builtin_inff();
  int idx = 0x7FFFFFFF;
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int e0 = c * kChunk + (j * kT + threadIdx.x) * kVec;
    if (e0 + kVec <= p.a.vocab) {
      const u4 w = *reinterpret_cast<const u4_anywhere*>(src + e0);
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        // (a cast of the vector element itself would read the vector's first)
        const uint32_t bits = sizeof(T) == 4 ? w[e] : w[e / 2] >> (16 * (e & 1));
        if constexpr (sizeof(T) == 4)
          x[j * kVec + e] = logit<T>(__builtin_bit_cast(T, bits));
        else
          x[j * kVec + e] = logit<T>(__builtin_bit_cast(T, static_cast<uint16_t>(bits)));
      }
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        x[j * kVec + e] = e0 + e < p.a.vocab ? logit<T>(src[e0 + e]) : -__builtin_inff();
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e)
      if (x[j * kVec + e] > m) m = x[j * kVec + e], idx = e0 + e;
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) fold_max(m, idx, o);
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = m, widx[threadIdx.x >> 6] = idx;
  __syncthreads();
  m = wmax[0], idx = widx[0];
#pragma unroll
  for (int w = 1; w < kT / 64; ++w)
    if (wmax[w] > m || (wmax[w] == m && widx[w] < idx)) m = wmax[w], idx = widx[w];
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const float w = x[e] == m ? 1.f : __builtin_amdgcn_exp2f((x[e] - m) * scale);
    s += x[e] == -__builtin_inff() ? 0.f : w;
  }
  double sum = wave_sum(s);
  if ((threadIdx.x & 63) == 0) wsum[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.0;
#pragma unroll
    for (int w = 0; w < kT / 64; ++w) sum += wsum[w];
    p.stats[static_cast<int64_t>(row) * p.chunks + c] = Stat{m, idx, sum};
  }
}

// Two sums over the workgroup, to every thread.
__device__ __forceinline__ void block_sum2(double& a, double& b, double (&buf)[kDrawWaves][2]) {
  a = wave_sum(a), b = wave_sum(b);
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6][0] = a, buf[threadIdx.x >> 6][1] = b;
  __syncthreads();
  a = b = 0.0;
#pragma unroll 4
  for (int w = 0; w < kDrawWaves; ++w) a += buf[w][0], b += buf[w][1];
}

// The weights of this thread's places e0 + j * step of the row that a token is
// drawn from: of p without the struck draft, and of q where qr is given.
// SMALL: with one copy of the exponential, for a kernel of few workgroups.
template <typename T, bool PROBS, bool SMALL>
__device__ __forceinline__ void weights(const VerifyParams& p, const Verdict& v, const T* pr, const T* qr, int e0,
                                        int step, double (&wp)[kDrawPer], double (&wq)[kDrawPer]) {
  float x[kDrawPer], y[kDrawPer];
#pragma unroll
  for (int j = 0; j < kDrawPer; ++j) {
    const int e = e0 + j * step;
    const bool in = e < p.a.vocab;
    if constexpr (PROBS) {
      wp[j] = in && e != v.skip ? probability(widen<T>(pr[e])) : 0.0;
      wq[j] = in && qr ? probability(widen<T>(qr[e])) : 0.0;
    } else {
      x[j] = in && e != v.skip ? logit<T>(pr[e]) : -__builtin_inff();
      y[j] = in && qr ? logit<T>(qr[e]) : -__builtin_inff();
    }
  }
  if constexpr (!PROBS) {
    static_assert(kDrawPer == 4, "four places are told apart below");
    const double inv_t = 1.0 / v.t;
#pragma unroll
    for (int j = 0; j < 4; ++j) wq[j] = 0.0;
    if constexpr (SMALL) {
#pragma unroll 1
      for (int k = 0; k < (qr ? 8 : 4); ++k) {
        const int j = k & 3;
        const float xs = j == 0 ? x[0] : j == 1 ? x[1] : j == 2 ? x[2] : x[3];
        const float ys = j == 0 ? y[0] : j == 1 ? y[1] : j == 2 ? y[2] : y[3];
        const double w = weight(k < 4 ? xs : ys, k < 4 ? v.p_max : v.q_max, inv_t);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (k == i) wp[i] = w;
          if (k == 4 + i) wq[i] = w;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) wp[j] = weight(x[j], v.p_max, inv_t);
      if (qr) {
#pragma unroll
        for (int j = 0; j < 4; ++j) wq[j] = weight(y[j], v.q_max, inv_t);
      }
    }
  }
}

// What the draft leaves over of a token, from weights and factors. Both products
// are rounded before the difference: in a fused multiply-add one of them would
// not be, and where the rows agree the rounding of the other would be left over,
// to be drawn from instead of p. The sums and the pick call this one function, so
// that a chunk whose sum is above 0 has a token whose share is.
__device__ __forceinline__ double left_over(double wp, double scale_p, double wq, double scale_q) {
#pragma clang fp contract(off)
  const double p = wp * scale_p, q = wq * scale_q;
  return fmax(p - q, 0.0);
}

// The accept tests alone, a workgroup a sequence.
template <typename T>
__global__ __launch_bounds__(kD) void verify_decide_kernel(const VerifyParams p) {
  decide<T, false>(p, blockIdx.x, true);
}

// Chunk sums of the row that a token is picked from. REST false: of p and,
// where its draft was rejected, of q; of probabilities, which need no totals,
// also of what q leaves over. REST true: of what q leaves over.
template <typename T, bool PROBS, bool REST>
__global__ __launch_bounds__(kD) void verify_sums_kernel(const VerifyParams p) {
  __shared__ double buf[kDrawWaves][2];
  const int b = blockIdx.x / p.chunks, c = blockIdx.x - b * p.chunks;
  const Verdict v = REST || p.decided ? p.verdicts[b] : decide<T, PROBS>(p, b, c == 0);
  if (v.how == kDone || (REST && v.how != kFromRest)) return;
  const T* pr = target_row<T>(p, b, v.accepted);
  const T* qr = v.how == kFromRest ? draft_row<T>(p, b, v.accepted) : nullptr;
  double* sums = p.sums + static_cast<int64_t>(b) * 3 * p.chunks;
  double wp[kDrawPer], wq[kDrawPer];
  weights<T, PROBS, false>(p, v, pr, qr, c * kChunk + threadIdx.x, kD, wp, wq);
  double scale_p = 1.0, scale_q = 1.0;
  if constexpr (REST) {
    double zp = 0.0, zq = 0.0;  // (verify_pick_kernel adds them in the same order)
#pragma unroll 1
    for (int j = threadIdx.x; j < p.chunks; j += kD) zp += sums[j], zq += sums[p.chunks + j];
    block_sum2(zp, zq, buf);
    scale_p = zp > 0.0 ? 1.0 / zp : 0.0;
    scale_q = zq > 0.0 ? 1.0 / zq : 0.0;
    __syncthreads();
  }
  double sp = 0.0, sq = 0.0;
#pragma unroll
  for (int j = 0; j < kDrawPer; ++j) {
    if constexpr (REST) {
      sp += left_over(wp[j], scale_p, wq[j], scale_q);
    } else {
      sp += wp[j];
      sq += PROBS ? left_over(wp[j], 1.0, wq[j], 1.0) : wq[j];
    }
  }
  block_sum2(sp, sq, buf);
  if (threadIdx.x == 0) {
    if constexpr (REST) {
      sums[2 * p.chunks + c] = sp;
    } else {
      sums[c] = sp;
      sums[(PROBS ? 2 : 1) * p.chunks + c] = sq;
    }
  }
}

// The token that u_sample picks, one workgroup a sequence: from max(p - q, 0)
// for a rejected draft with a row, else from p (without v.skip). The first
// wavefront finds the chunk, then all of them its token.
template <typename T, bool PROBS>
__global__ __launch_bounds__(kD) void verify_pick_kernel(const VerifyParams p) {
  __shared__ double w[kChunk];
  __shared__ double wsum[kDrawWaves];
  __shared__ double s_left, s_scale_p, s_scale_q, s_zp;
  __shared__ int s_chunk, s_rest, found, last;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Verdict v = p.verdicts[b];
  if (v.how == kDone) return;
  const T* pr = target_row<T>(p, b, v.accepted);
  const T* qr = v.how == kFromRest ? draft_row<T>(p, b, v.accepted) : nullptr;
  if (wave == 0) {
    const double* sums = p.sums + static_cast<int64_t>(b) * 3 * p.chunks;
    const float u = p.a.u_sample[b];
    // the totals of p, q and of what is left over, those of p and q in the order
    // of the pass that summed that (a thread's places, lanes, wavefronts): with
    // totals of another order all that rounding left of a chunk there could be
    // gone here
    double z[3] = {0.0, 0.0, 0.0};
#pragma unroll 1
    for (int w0 = 0; w0 < min(p.chunks, kD); w0 += 64) {
      double x[3] = {0.0, 0.0, 0.0};
#pragma unroll 1
      for (int j = w0 + lane; j < p.chunks; j += kD) {
        x[0] += sums[j];
        if (qr) {
          if constexpr (!PROBS) x[1] += sums[p.chunks + j];
          x[2] += sums[2 * p.chunks + j];
        }
      }
#pragma unroll
      for (int k = 0; k < 3; ++k) z[k] += wave_sum(x[k]);
    }
    const bool rest = qr && z[2] > 0.0;  // nothing left over: from p
    const double* cs = rest ? sums + 2 * p.chunks : sums;
    const double aim = static_cast<double>(u) * (rest ? z[2] : z[0]);
    // the first chunk whose running sum exceeds the aim; by rounding there may
    // be none: then the last that holds anything, and all of it
    int chunk = -1;
    double run = 0.0, before = -__builtin_inf();
#pragma unroll 1
    for (int j0 = 0; j0 < p.chunks; j0 += 64) {
      const double x = j0 + lane < p.chunks ? cs[j0 + lane] : 0.0;
      const double sum = run + wave_scan(x);
      const unsigned long long over = __ballot(x > 0.0 && sum > aim), some = __ballot(x > 0.0);
      if (over) {
        const int l = __builtin_ctzll(over);
        chunk = j0 + l;
        before = lane_value(sum - x, l);
        break;
      }
      if (some) chunk = j0 + 63 - __builtin_clzll(some);
      run = lane_value(sum, 63);
    }
    if (lane == 0) {
      s_chunk = chunk;
      s_left = aim - before;
      s_rest = rest;
      s_zp = z[0];
      s_scale_p = !PROBS && rest ? 1.0 / z[0] : 1.0;
      s_scale_q = !PROBS && rest && z[1] > 0.0 ? 1.0 / z[1] : PROBS && rest ? 1.0 : 0.0;
      found = 0x7FFFFFFF, last = -1;
    }
  }
  __syncthreads();
  int token = -1;
  const int chunk = s_chunk;
  if (chunk >= 0) {
    double wp[kDrawPer], wq[kDrawPer];
    weights<T, PROBS, true>(p, v, pr, s_rest ? qr : nullptr, chunk * kChunk + tid, kD, wp, wq);
#pragma unroll
    for (int j = 0; j < kDrawPer; ++j) w[j * kD + tid] = left_over(wp[j], s_scale_p, wq[j], s_scale_q);
    __syncthreads();
    double mine = 0.0;
#pragma unroll
    for (int j = 0; j < kDrawPer; ++j) mine += w[tid * kDrawPer + j];
    double sum = wave_scan(mine);
    if (lane == 63) wsum[wave] = sum;
    __syncthreads();
    sum -= mine;
#pragma unroll
    for (int k = 0; k < kDrawWaves - 1; ++k) sum += k < wave ? wsum[k] : 0.0;
    int hit = 0x7FFFFFFF, end = -1;
#pragma unroll
    for (int j = 0; j < kDrawPer; ++j) {
      const double x = w[tid * kDrawPer + j];
      sum += x;
      if (x > 0.0) {
        end = tid * kDrawPer + j;
        if (sum > s_left && hit == 0x7FFFFFFF) hit = end;
      }
    }
    // lanes lie in order: one of each wavefront speaks for it (1024 atomics on
    // one place took 6 us)
    const unsigned long long hits = __ballot(hit != 0x7FFFFFFF), ends = __ballot(end >= 0);
    if (hits && lane == static_cast<int>(__builtin_ctzll(hits))) atomicMin(&found, hit);
    if (ends && lane == 63 - static_cast<int>(__builtin_clzll(ends))) atomicMax(&last, end);
    __syncthreads();
    token = chunk * kChunk + (found != 0x7FFFFFFF ? found : last);
  }
  if (tid < 2) {
    // lane 0: the token's weight in p; lane 1: that of the struck draft, which is in no sum
    const int e = tid == 0 ? token : v.skip;
    double x = 0.0;
    if (e >= 0 && e < p.a.vocab) {
      if constexpr (PROBS) x = probability(widen<T>(pr[e]));
      else x = weight(logit<T>(pr[e]), v.p_max, 1.0 / v.t);
    }
    const double struck = __shfl_xor(x, 1);
    if (tid == 0) {
      if (token < 0 && struck > 0.0) token = v.skip, x = struck;  // it is all that p is
      const int64_t at = static_cast<int64_t>(b) * (p.a.drafts + 1) + v.accepted;
      p.a.tokens[at] = token;
      if (p.a.logprobs) p.a.logprobs[at] = log_of(token < 0 ? 1.0 : PROBS ? x : x / (s_zp + struck));
    }
  }
}

template <typename T>
hipError_t launch_logits(const VerifyParams& p, hipStream_t stream) {
  const int target_rows = p.a.batch * (p.a.drafts + 1);
  const bool with_draft = p.a.draft && p.a.drafts > 0;
  const int rows = target_rows + (with_draft ? p.a.batch * p.a.drafts : 0);
  verify_rows_kernel<T><<<dim3(static_cast<uint32_t>(rows) * p.chunks), kT, 0, stream>>>(p, target_rows);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid(static_cast<uint32_t>(p.a.batch) * p.chunks);
  if (p.decided) {
    verify_decide_kernel<T><<<dim3(p.a.batch), kD, 0, stream>>>(p);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  verify_sums_kernel<T, false, false><<<grid, kD, 0, stream>>>(p);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (with_draft) {
    verify_sums_kernel<T, false, true><<<grid, kD, 0, stream>>>(p);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  verify_pick_kernel<T, false><<<dim3(p.a.batch), kD, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_verify(const qpn_verify_args& a, const VerifyPlan& plan, void* workspace, hipStream_t stream) {
  VerifyParams p;
  p.a = a;
  p.chunks = plan.chunks;
  // Up to one workgroup a slot (two a compute unit) each makes its sequence's
  // accept tests itself, beyond that a launch of their own makes them once.
  // Whole calls, inside against launched: 152 workgroups 19.4 and 20.7 us, 494
  // 25.0 and 25.8, 608 29.6 and 27.5, 1824 61 and 53 (3 drafts, fp16).
  p.decided = !a.probabilities && a.batch * plan.chunks > 2 * kComputeUnits;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.verdicts = reinterpret_cast<Verdict*>(ws);
  p.stats = reinterpret_cast<Stat*>(ws += plan.verdict_bytes);
  p.sums = reinterpret_cast<double*>(ws + plan.stat_bytes);
  if (a.probabilities) {
    verify_sums_kernel<float, true, false><<<dim3(static_cast<uint32_t>(a.batch) * p.chunks), kD, 0, stream>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    verify_pick_kernel<float, true><<<dim3(a.batch), kD, 0, stream>>>(p);
    return hipGetLastError();
  }
  switch (a.dtype) {
    case QPN_DT_F16: return launch_logits<_Float16>(p, stream);
    case QPN_DT_BF16: return launch_logits<Bf16>(p, stream);
    default: return launch_logits<float>(p, stream);
  }
}

}  // namespace qpn
