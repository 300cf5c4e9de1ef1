// Verification of drafted tokens (include/qpn_decode.h).
//
// One pass over all rows of logits takes each row's maximum, its lowest index
// and the sum of exponentials (32-bit exponentials, 64-bit sums of them):
// that is all the accept tests need. Only one row a sequence (two with a
// draft) is then read again, for the place of u_sample among the running
// sums. A vocabulary's running sums lie closer together than 32 bits tell
// apart, so these weights and sums are 64-bit, spread over the workgroups in
// chunks: chunk sums, then (with a draft's logits) the chunk sums of
// max(p - q, 0), for which both rows' totals must be known, then one
// workgroup a sequence finds the chunk and the token in it. The kernels after
// the first repeat the accept tests, a few hundred values from the cache,
// instead of handing them over in a launch of their own.
#include "qpn_decode_internal.hpp"
#include "qpn_device.hpp"

namespace qpn {
namespace {

constexpr int kT = 256;          // threads
constexpr int kChunk = 4096;     // elements a workgroup takes of a row
constexpr int kPer = kChunk / kT;
constexpr int kMaxDrafts = 64;

struct Stat {
  float max;
  int idx;
  double sum;
};
static_assert(sizeof(Stat) == 16, "the workspace holds 16 bytes a chunk");

struct VerifyParams {
  qpn_verify_args a;
  int chunks;
  Stat* stats;   // [batch][drafts + 1][chunks], then [batch][drafts][chunks]
  double* sums;  // [batch][3][chunks]: of p, of q, of what q leaves over
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
__device__ __forceinline__ double exp64(double x) {
  x = fmax(x, -800.0);
  const double n = rint(x * 1.4426950408889634074);
  double r = fma(n, -6.93147180369123816490e-01, x);  // ln 2 in two parts: n times the first is exact
  r = fma(n, -1.90821492927058770002e-10, r);
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

// Maximum and sum of exponentials of one chunk of one row. The chunk grid is
// laid on 16-byte boundaries of memory, so that rows of any alignment are
// read in whole vectors but for their first and last.
template <typename T>
__global__ __launch_bounds__(kT) void verify_stats_kernel(const VerifyParams p, int target_rows) {
  constexpr int kVec = 16 / sizeof(T), kLoads = kPer / kVec;
  __shared__ float wmax[kT / 64];
  __shared__ int widx[kT / 64];
  __shared__ double wsum[kT / 64];
  const int row = blockIdx.x / p.chunks, c = blockIdx.x - row * p.chunks;
  int b, i;
  const T* src;
  const bool is_target = row < target_rows;
  if (is_target) {
    b = row / (p.a.drafts + 1), i = row - b * (p.a.drafts + 1);
    if (i > drafts_of(p, b)) return;
    src = target_row<T>(p, b, i);
  } else {
    b = (row - target_rows) / p.a.drafts, i = (row - target_rows) - b * p.a.drafts;
    if (i >= drafts_of(p, b) || temperature_of(p, b) == 0.f) return;
    src = draft_row<T>(p, b, i);
  }
  const float t = temperature_of(p, b);
  const float scale = 1.44269504088896341f / (t > 0.f ? t : 1.f);
  const int lead = static_cast<int>(reinterpret_cast<uintptr_t>(src) / sizeof(T)) & (kVec - 1);
  float x[kPer];
  float m = -__builtin_inff();
  int idx = 0x7FFFFFFF;
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int e0 = c * kChunk + (j * kT + threadIdx.x) * kVec - lead;
    if (e0 >= 0 && e0 + kVec <= p.a.vocab) {
      const u4 w = __builtin_nontemporal_load(reinterpret_cast<const u4*>(src + e0));
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
        x[j * kVec + e] = e0 + e >= 0 && e0 + e < p.a.vocab ? logit<T>(src[e0 + e]) : -__builtin_inff();
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
  double sum = s;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o);
  if ((threadIdx.x & 63) == 0) wsum[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.0;
#pragma unroll
    for (int w = 0; w < kT / 64; ++w) sum += wsum[w];
    p.stats[static_cast<int64_t>(row) * p.chunks + c] = Stat{m, idx, sum};
  }
}

// One row's chunks as one, by a wavefront (all lanes return it).
__device__ __forceinline__ Stat join_stats(const Stat* s, int chunks, float t) {
  const int lane = threadIdx.x & 63;
  const double inv_t = 1.0 / (t > 0.f ? t : 1.f);
  Stat r{-__builtin_inff(), 0x7FFFFFFF, 0.0};
  for (int c = lane; c < chunks; c += 64) {
    const Stat x = s[c];
    if (x.max > r.max || (x.max == r.max && x.idx < r.idx)) r.max = x.max, r.idx = x.idx;
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) fold_max(r.max, r.idx, o);
  for (int c = lane; c < chunks; c += 64) r.sum += s[c].sum * weight(s[c].max, r.max, inv_t);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) r.sum += __shfl_xor(r.sum, o);
  return r;
}

// What the accept tests say of a sequence.
struct Verdict {
  int accepted, n;
  float t;             // 0: greedy
  float p_max, q_max;  // maxima of the rows that the token is picked from
  int best;            // the target row's largest logit
  double p_sum;        // 32-bit precise
};

struct VerdictShared {
  int ok[kMaxDrafts + 1];
  float pmax[kMaxDrafts + 1], qmax[kMaxDrafts + 1];
  int best[kMaxDrafts + 1];
  double psum[kMaxDrafts + 1];
};

template <typename T, bool PROBS>
__device__ Verdict decide(const VerifyParams& p, int b, VerdictShared& sh) {
  const int n = drafts_of(p, b), wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const float t = temperature_of(p, b);
  const double inv_t = 1.0 / (t > 0.f ? t : 1.f);
  for (int i = wave; i <= n; i += kT / 64) {
    const int d = i < n ? p.a.draft_tokens[static_cast<int64_t>(b) * p.a.drafts + i] : 0;
    const bool known = d >= 0 && d < p.a.vocab;
    const T* pr = target_row<T>(p, b, i);
    bool ok = false;
    Stat ps{0.f, 0, 0.0}, qs{0.f, 0, 0.0};
    if constexpr (PROBS) {
      if (i < n && known) {
        const double pd = probability(widen<T>(pr[d]));
        const double qd = p.a.draft ? probability(widen<T>(draft_row<T>(p, b, i)[d])) : 1.0;
        ok = static_cast<double>(p.a.u_accept[static_cast<int64_t>(b) * p.a.drafts + i]) * qd < pd;
      }
    } else {
      ps = join_stats(p.stats + (static_cast<int64_t>(b) * (p.a.drafts + 1) + i) * p.chunks, p.chunks, t);
      if (i < n && t == 0.f) {
        ok = known && ps.idx == d;
      } else if (i < n) {
        if (p.a.draft)
          qs = join_stats(p.stats + (static_cast<int64_t>(p.a.batch) * (p.a.drafts + 1) +
                                     static_cast<int64_t>(b) * p.a.drafts + i) * p.chunks, p.chunks, t);
        if (known) {
          const double pd = ps.sum > 0.0 ? weight(logit<T>(pr[d]), ps.max, inv_t) / ps.sum : 0.0;
          double qd = 1.0;
          if (p.a.draft) qd = qs.sum > 0.0 ? weight(logit<T>(draft_row<T>(p, b, i)[d]), qs.max, inv_t) / qs.sum : 0.0;
          ok = static_cast<double>(p.a.u_accept[static_cast<int64_t>(b) * p.a.drafts + i]) * qd < pd;
        }
      }
    }
    if (lane == 0) {
      sh.ok[i] = ok;
      sh.pmax[i] = ps.max, sh.qmax[i] = qs.max;
      sh.best[i] = ps.idx;
      sh.psum[i] = ps.sum;
    }
  }
  __syncthreads();
  int a = 0;
  while (a < n && sh.ok[a]) ++a;
  return Verdict{a, n, t, sh.pmax[a], sh.qmax[a], sh.best[a], sh.psum[a]};
}

// The unnormalized weights of place `e` of the row the token is picked from:
// of p (without the rejected draft `skip`, where no draft row is given) and of q.
template <typename T, bool PROBS>
__device__ __forceinline__ double p_weight(const T* row, int e, float max, double inv_t, int skip) {
  if (e == skip) return 0.0;
  if constexpr (PROBS)
    return probability(widen<T>(row[e]));
  else
    return weight(logit<T>(row[e]), max, inv_t);
}

// Sums over a chunk of up to two quantities, to thread 0.
__device__ __forceinline__ void block_sum2(double& a, double& b, double (*buf)[2]) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) a += __shfl_xor(a, o), b += __shfl_xor(b, o);
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6][0] = a, buf[threadIdx.x >> 6][1] = b;
  __syncthreads();
  a = b = 0.0;
#pragma unroll
  for (int w = 0; w < kT / 64; ++w) a += buf[w][0], b += buf[w][1];
}

// LEFT false: the chunk's sums of p and of q (and, of probabilities, of what
// q leaves over at once); true: of what q leaves over.
template <typename T, bool PROBS, bool LEFT>
__global__ __launch_bounds__(kT) void verify_sums_kernel(const VerifyParams p) {
  __shared__ VerdictShared sh;
  __shared__ double buf[kT / 64][2];
  const int b = blockIdx.x / p.chunks, c = blockIdx.x - b * p.chunks;
  const Verdict v = decide<T, PROBS>(p, b, sh);
  const bool rejected = v.accepted < v.n;
  if constexpr (!PROBS)
    if (v.t == 0.f) return;  // greedy: nothing is drawn
  const bool with_q = rejected && p.a.draft;
  if (LEFT && !with_q) return;
  const double inv_t = 1.0 / (v.t > 0.f ? v.t : 1.f);
  const T* pr = target_row<T>(p, b, v.accepted);
  const T* qr = with_q ? draft_row<T>(p, b, v.accepted) : nullptr;
  const int skip =
      rejected && !p.a.draft ? p.a.draft_tokens[static_cast<int64_t>(b) * p.a.drafts + v.accepted] : -1;
  double* sums = p.sums + static_cast<int64_t>(b) * 3 * p.chunks;
  double inv_p = 0.0, inv_q = 0.0;
  if constexpr (LEFT) {
    double zp = 0.0, zq = 0.0;
    for (int j = threadIdx.x; j < p.chunks; j += kT) zp += sums[j], zq += sums[p.chunks + j];
    block_sum2(zp, zq, buf);
    inv_p = zp > 0.0 ? 1.0 / zp : 0.0;
    inv_q = zq > 0.0 ? 1.0 / zq : 0.0;
    __syncthreads();
  }
  double sp = 0.0, sq = 0.0;
#pragma unroll 4
  for (int j = 0; j < kPer; ++j) {
    const int e = c * kChunk + j * kT + threadIdx.x;
    if (e >= p.a.vocab) break;
    const double wp = p_weight<T, PROBS>(pr, e, v.p_max, inv_t, skip);
    const double wq = with_q ? p_weight<T, PROBS>(qr, e, v.q_max, inv_t, -1) : 0.0;
    if constexpr (LEFT) {
      sp += fmax(wp * inv_p - wq * inv_q, 0.0);
    } else if constexpr (PROBS) {
      sp += wp;
      sq += fmax(wp - wq, 0.0);
    } else {
      sp += wp;
      sq += wq;
    }
  }
  block_sum2(sp, sq, buf);
  if (threadIdx.x == 0) {
    if constexpr (LEFT) {
      sums[2 * p.chunks + c] = sp;
    } else if constexpr (PROBS) {
      sums[c] = sp;
      sums[2 * p.chunks + c] = sq;
    } else {
      sums[c] = sp;
      sums[p.chunks + c] = sq;
    }
  }
}

// Inclusive running sum over the workgroup's threads, in thread order.
__device__ __forceinline__ double block_scan(double x, double* wsum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 63) wsum[wave] = x;
  __syncthreads();
  for (int w = 0; w < wave; ++w) x += wsum[w];
  return x;
}

// One workgroup a sequence: the token and the outputs.
template <typename T, bool PROBS>
__global__ __launch_bounds__(kT) void verify_pick_kernel(const VerifyParams p) {
  __shared__ VerdictShared sh;
  __shared__ double wsum[kT / 64];
  __shared__ double buf[kT / 64][2];
  __shared__ int found, last;
  __shared__ double before;
  const int b = blockIdx.x, tid = threadIdx.x;
  const Verdict v = decide<T, PROBS>(p, b, sh);
  const bool rejected = v.accepted < v.n, greedy = !PROBS && v.t == 0.f;
  const double inv_t = 1.0 / (v.t > 0.f ? v.t : 1.f);
  const T* pr = target_row<T>(p, b, v.accepted);
  int token = -1;
  if (greedy) {
    if (v.p_max > -__builtin_inff()) token = v.best;
  } else {
    const int32_t d = rejected ? p.a.draft_tokens[static_cast<int64_t>(b) * p.a.drafts + v.accepted] : -1;
    int skip = rejected && !p.a.draft ? d : -1;
    bool with_q = rejected && p.a.draft;
    const T* qr = with_q ? draft_row<T>(p, b, v.accepted) : nullptr;
    const double* sums = p.sums + static_cast<int64_t>(b) * 3 * p.chunks;
    // the totals of p, q and of what is left over
    double zp = 0.0, zq = 0.0, zl = 0.0, none = 0.0;
    for (int j = tid; j < p.chunks; j += kT) {
      zp += sums[j];
      if (with_q) {
        if constexpr (!PROBS) zq += sums[p.chunks + j];
        zl += sums[2 * p.chunks + j];
      }
    }
    block_sum2(zp, zq, buf);
    __syncthreads();
    block_sum2(zl, none, buf);
    const double inv_p = PROBS ? 1.0 : (zp > 0.0 ? 1.0 / zp : 0.0), inv_q = PROBS ? 1.0 : (zq > 0.0 ? 1.0 / zq : 0.0);
    double total = with_q ? zl : zp;
    bool rest_of_p = false;  // nothing is left over: from p
    if (!(total > 0.0) && rejected) {
      if (with_q) {
        with_q = false;
        total = zp;
      } else {
        // p without the draft is nothing: the draft is all there is
        rest_of_p = true;
        skip = -1;
      }
    }
    if (rest_of_p) {
      const bool known = d >= 0 && d < p.a.vocab;
      if (tid == 0 && known && p_weight<T, PROBS>(pr, d, v.p_max, inv_t, -1) > 0.0) found = d;
      else if (tid == 0) found = -1;
      __syncthreads();
      token = found;
    } else if (total > 0.0) {
      const double* cs = with_q ? sums + 2 * p.chunks : sums;
      const double aim = static_cast<double>(p.a.u_sample[b]) * total;
      // the first chunk whose running sum exceeds the aim (or the last that holds anything)
      if (tid == 0) found = 0x7FFFFFFF, last = -1;
      __syncthreads();
      double run = 0.0;
      for (int j0 = 0; j0 < p.chunks; j0 += kT) {
        const int j = j0 + tid;
        const double x = j < p.chunks ? cs[j] : 0.0;
        const double sum = run + block_scan(x, wsum);
        if (j < p.chunks && x > 0.0) {
          if (sum > aim) atomicMin(&found, j);
          atomicMax(&last, j);
        }
        __syncthreads();
        if (found == j) before = sum - x;
        run += wsum[0] + wsum[1] + wsum[2] + wsum[3];
        __syncthreads();
        if (found != 0x7FFFFFFF) break;
      }
      const bool whole = found == 0x7FFFFFFF;  // rounding: past the end, the last token that counts
      const int c = whole ? last : found;
      const double left = whole ? __builtin_inf() : aim - before;
      __syncthreads();
      if (tid == 0) found = 0x7FFFFFFF, last = -1;
      double w[kPer], mine = 0.0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int e = c * kChunk + tid * kPer + j;
        w[j] = 0.0;
        if (e < p.a.vocab) {
          w[j] = p_weight<T, PROBS>(pr, e, v.p_max, inv_t, skip);
          if (with_q) w[j] = fmax(w[j] * inv_p - p_weight<T, PROBS>(qr, e, v.q_max, inv_t, -1) * inv_q, 0.0);
        }
        mine += w[j];
      }
      double sum = block_scan(mine, wsum) - mine;
      int hit = 0x7FFFFFFF, end = -1;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        sum += w[j];
        if (w[j] > 0.0) {
          end = c * kChunk + tid * kPer + j;
          if (sum > left && hit == 0x7FFFFFFF) hit = end;
        }
      }
      if (hit != 0x7FFFFFFF) atomicMin(&found, hit);
      if (end >= 0) atomicMax(&last, end);
      __syncthreads();
      token = found != 0x7FFFFFFF ? found : last;
    }
  }
  // outputs: place tid
  const int places = p.a.drafts + 1;
  if (tid < places) {
    int out = -1;
    if (tid < v.accepted) out = p.a.draft_tokens[static_cast<int64_t>(b) * p.a.drafts + tid];
    else if (tid == v.accepted) out = token;
    p.a.tokens[static_cast<int64_t>(b) * places + tid] = out;
    if (p.a.logprobs) {
      double lp = 0.0;
      if (out >= 0) {
        const T x = target_row<T>(p, b, tid)[out];
        if constexpr (PROBS) {
          lp = log(probability(widen<T>(x)));
        } else {
          const float y = logit<T>(x);
          lp = (y == sh.pmax[tid] ? 0.0 : (static_cast<double>(y) - static_cast<double>(sh.pmax[tid])) * inv_t) -
               log(sh.psum[tid]);
        }
      }
      p.a.logprobs[static_cast<int64_t>(b) * places + tid] = static_cast<float>(lp);
    }
  }
  if (tid == 0) p.a.accepted[b] = v.accepted;
}

template <typename T>
hipError_t launch_logits(const VerifyParams& p, hipStream_t stream) {
  const int target_rows = p.a.batch * (p.a.drafts + 1);
  const int rows = target_rows + (p.a.draft ? p.a.batch * p.a.drafts : 0);
  verify_stats_kernel<T><<<dim3(static_cast<uint32_t>(rows) * p.chunks), kT, 0, stream>>>(p, target_rows);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid(static_cast<uint32_t>(p.a.batch) * p.chunks);
  verify_sums_kernel<T, false, false><<<grid, kT, 0, stream>>>(p);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (p.a.draft && p.a.drafts > 0) {
    verify_sums_kernel<T, false, true><<<grid, kT, 0, stream>>>(p);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  verify_pick_kernel<T, false><<<dim3(p.a.batch), kT, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_verify(const qpn_verify_args& a, const VerifyPlan& plan, void* workspace, hipStream_t stream) {
  VerifyParams p;
  p.a = a;
  p.chunks = plan.chunks;
  p.stats = static_cast<Stat*>(workspace);
  p.sums = reinterpret_cast<double*>(static_cast<uint8_t*>(workspace) + plan.stat_bytes);
  if (a.probabilities) {
    verify_sums_kernel<float, true, false><<<dim3(static_cast<uint32_t>(a.batch) * p.chunks), kT, 0, stream>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    verify_pick_kernel<float, true><<<dim3(a.batch), kT, 0, stream>>>(p);
    return hipGetLastError();
  }
  switch (a.dtype) {
    case QPN_DT_F16: return launch_logits<_Float16>(p, stream);
    case QPN_DT_BF16: return launch_logits<Bf16>(p, stream);
    default: return launch_logits<float>(p, stream);
  }
}

}  // namespace qpn
