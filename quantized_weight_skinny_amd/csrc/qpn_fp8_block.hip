// Products of 8-bit codes with a scale for each block of 128
// (include/qpn_prompt.h): the quantizer, the product of a few rows and the
// product of many.
//
// Mathematics. v_mfma_f32_16x16x128_f8f6f4 takes 128 places of k at once, one
// block of either operand's scales: started from zero it gives the block's
// sums, and one multiply-add each adds them, times (x scale * w scale), to the
// fp32 result. w is the A operand (16 outputs), x the B operand (16 rows), so a
// lane's results are one row of x at four neighbouring outputs: one factor for
// all four, and stores of four. Lane l = (i, g) = (l % 16, l / 16) holds row i;
// which 32 of the 128 places it holds is free as long as both operands agree:
// the 16-byte pieces g and g + 4.
//
// What the instruction keeps of a sum. It adds the products of codes with some
// 12 bits below the largest of them, not 24: blocks of normal values come out
// 1.4e-5 of the result off (the 2-norms), measured, and the same for
// v_mfma_f32_16x16x32_fp8_fp8. That is a tenth and less of the rounding to
// fp16 or bf16; where large products of a block cancel it is 2^-11 of what has
// cancelled, which may be more than the rounding. An fp32 result is the choice of a
// caller who minds: there the codes are brought to fp16, which holds them exactly, for
// v_mfma_f32_16x16x32_f16, whose sums are fp32 (EXACT below). At half the rate, 2048 x
// 34816 x 5120 takes 674 us then instead of 397, which is why 16-bit results do not have it.
#include <algorithm>

#include "qpn_decode_internal.hpp"
#include "qpn_device.hpp"
#include "qpn_prompt_internal.hpp"

namespace qpn {
namespace {

typedef int i8 __attribute__((ext_vector_type(8)));
typedef const float __attribute__((address_space(4))) * scalar_ptr;  // read through the scalar cache

// ------------------------------------------------------------------ quantizer

// 8 elements of type DT from element `at` of a row; those from `end` on are 0.
template <int DT>
__device__ __forceinline__ void load8(const void* row, int64_t at, int64_t end, bool vec, float (&v)[8]) {
  if constexpr (DT == QPN_DT_F32) {
    const float* p = static_cast<const float*>(row) + at;
    if (vec && at + 8 <= end) {
      const f4 a = *reinterpret_cast<const f4*>(p), b = *reinterpret_cast<const f4*>(p + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = at + e < end ? p[e] : 0.f;
    }
  } else {
    constexpr bool kBf16 = DT == QPN_DT_BF16;
    const uint16_t* p = static_cast<const uint16_t*>(row) + at;
    if (vec && at + 8 <= end) {
      const u4 x = *reinterpret_cast<const u4*>(p);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[2 * e] = widen16<kBf16>(x[e] & 0xFFFFu), v[2 * e + 1] = widen16<kBf16>(x[e] >> 16);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = at + e < end ? widen16<kBf16>(p[e]) : 0.f;
    }
  }
}

// The magnitude as it counts for a block's scale: 0 for inf and NaN.
__device__ __forceinline__ float counted(float x) {
  const float a = fabsf(x);
  return a < __builtin_inff() ? a : 0.f;
}

// The exponent e of the scale 2^e: amax = f 2^q with 1 <= f < 2, and 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exponent(float amax) {
  if (amax == 0.f) return 0;
  const uint32_t b = __float_as_uint(amax);
  const int q = static_cast<int>(b >> 23) - 127;  // (a subnormal amax gets the least scale)
  return max(q - 8 + ((b & 0x7FFFFFu) > 0x600000u), -126);
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Codes of 8 elements: exact quotients (a multiplication by a power of two),
// rounded to nearest even by the conversion; nothing is above 448.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
  float q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) q[e] = fabsf(v[e]) < __builtin_inff() ? v[e] * inv : __builtin_nanf("");
  uint2 r;
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  r.x = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
  r.y = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], w, true);
  return r;
}

__device__ __forceinline__ void store_codes8(uint8_t* row, int64_t at, int64_t end, bool vec, uint2 c) {
  if (vec && at + 8 <= end) {
    *reinterpret_cast<uint2*>(row + at) = c;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (at + e < end) row[at + e] = static_cast<uint8_t>((e < 4 ? c.x : c.y) >> (8 * (e & 3)));
  }
}

struct QuantizeParams {
  const void* x;
  uint8_t* codes;
  float* scales;
  int64_t rows, k, stride, code_stride, scale_row_stride, scale_block_stride;
  int32_t blocks, load_vec, store_vec;
};

// A row's block of 128 is 16 lanes', a load of 16 bytes each: 17408 x 5120 52 us (5.1
// TB/s; a copy reaches 6.2), fp32 78 (5.7). 2048 x 5120 of bf16 take 8 to 11 us for 31 MB
// that take 5 and 65 % of that in waiting, as its wavefronts are over after one
// load; a small call is a launch, 3 us.
template <int DT>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const QuantizeParams a) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 16 + threadIdx.x / 16;
  const int64_t row = t / a.blocks;
  if (row >= a.rows) return;
  const int block = static_cast<int>(t - row * a.blocks);
  const int64_t at = static_cast<int64_t>(block) * kScaleBlock + threadIdx.x % 16 * 8;
  const int size = DT == QPN_DT_F32 ? 4 : 2;
  float v[8];
  load8<DT>(static_cast<const char*>(a.x) + row * a.stride * size, at, a.k, a.load_vec, v);
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, counted(v[e]));
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
  const int e2 = scale_exponent(amax);
  store_codes8(a.codes + row * a.code_stride, at, a.k, a.store_vec, codes8(v, pow2(-e2)));
  if (threadIdx.x % 16 == 0) a.scales[row * a.scale_row_stride + block * a.scale_block_stride] = pow2(e2);
}

// 128 x 128 elements are one workgroup's: 17408 x 5120 of bf16 51 us (5.2 TB/s), fp32 82
// (5.5), 151936 x 5120 428 (5.5).
template <int DT>
__global__ __launch_bounds__(256) void quantize_blocks_kernel(const QuantizeParams a) {
  __shared__ float top[4];
  const int64_t rb = blockIdx.x / a.blocks;
  const int block = static_cast<int>(blockIdx.x - rb * a.blocks);
  const int64_t at = static_cast<int64_t>(block) * kScaleBlock + threadIdx.x % 16 * 8;
  const int size = DT == QPN_DT_F32 ? 4 : 2;
  float amax = 0.f;
  float v[8][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t row = rb * kScaleBlock + j * 16 + threadIdx.x / 16;
    load8<DT>(static_cast<const char*>(a.x) + min(row, a.rows - 1) * a.stride * size, at, a.k, a.load_vec, v[j]);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, counted(v[j][e]));  // (the last row again changes nothing)
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
  if (threadIdx.x % 64 == 0) top[threadIdx.x / 64] = amax;
  __syncthreads();
  const int e2 = scale_exponent(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t row = rb * kScaleBlock + j * 16 + threadIdx.x / 16;
    if (row < a.rows) store_codes8(a.codes + row * a.code_stride, at, a.k, a.store_vec, codes8(v[j], pow2(-e2)));
  }
  if (threadIdx.x == 0) a.scales[rb * a.scale_row_stride + block * a.scale_block_stride] = pow2(e2);
}

// ------------------------------------------------------------------ products

struct ProductParams {
  const uint8_t *x, *w;
  const float *xs, *ws;
  void* y;
  float* partial;  // [splits][m][n] where splits > 1
  int64_t x_stride, xs_row, xs_block, w_stride, ws_row, ws_block, y_stride;
  int64_t m, n, n_first;  // (many rows: the tiles' first output)
  int32_t k, blocks, splits, tiles, y_dtype, y_vec;
};

// 32 codes of one row: a lane's part of a block, as fp16 where EXACT.
template <bool EXACT>
struct Frag {
  u4 c[2];
  __device__ __forceinline__ Frag() = default;
  __device__ __forceinline__ Frag(const u4& c0, const u4& c1) : c{c0, c1} {}
};
template <>
struct Frag<true> {
  h8 c[4];
  __device__ __forceinline__ Frag() = default;
  __device__ __forceinline__ Frag(const u4& c0, const u4& c1)
      : c{decode_fp8x8(c0[0], c0[1]), decode_fp8x8(c0[2], c0[3]), decode_fp8x8(c1[0], c1[1]), decode_fp8x8(c1[2], c1[3])} {}
};

// A lane's part of a block that begins at `at` less the lane's place, from memory: pieces past the end of k are zeros.
template <bool EXACT>
__device__ __forceinline__ Frag<EXACT> short_frag(const uint8_t* row, int64_t at, int k) {
  const u4 zero = {0u, 0u, 0u, 0u};
  return Frag<EXACT>(at < k ? *reinterpret_cast<const u4*>(row + at) : zero,
                     at + 64 < k ? *reinterpret_cast<const u4*>(row + at + 64) : zero);
}

// The block's sums.
__device__ __forceinline__ f4 block_sums(const Frag<true>& w, const Frag<true>& x) {
  f4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 4; ++j) s = __builtin_amdgcn_mfma_f32_16x16x32_f16(w.c[j], x.c[j], s, 0, 0, 0);
  return s;
}
__device__ __forceinline__ f4 block_sums(const Frag<false>& w, const Frag<false>& x) {
  const u4 &a0 = w.c[0], &a1 = w.c[1], &b0 = x.c[0], &b1 = x.c[1];
  const i8 a = {(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3], (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]};
  const i8 b = {(int)b0[0], (int)b0[1], (int)b0[2], (int)b0[3], (int)b1[0], (int)b1[1], (int)b1[2], (int)b1[3]};
  // both operands E4M3, no scales of the instruction's own
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// A block's factor, x scale * w scale, serves its sums as it is where it is a normal number.
// Where one is not, few rows take the way of add_scaled at once, and tiles once their loop is
// over (the test takes an instruction a factor: 2048 x 34816 x 5120 402 us with and without it;
// the other way inside the loop would have the compiler spill the tile of 256).
__device__ __forceinline__ bool ordinary(float factor) {
  return __builtin_amdgcn_classf(factor, 0x108);  // +normal, -normal
}
__device__ __forceinline__ bool finite_not_zero(float scale) {
  return __builtin_amdgcn_classf(scale, 0x198);  // normal and subnormal
}

// acc += sums * xs * sw where it may not be: the scales' mantissas are multiplied first,
// their exponents enter last, so that nothing leaves the range but a result that does.
__device__ __forceinline__ void add_scaled(f4& acc, const f4& sums, float xs, float sw) {
  const float factor = xs * sw;
  const bool as_it_is = ordinary(factor);
  const float m = __builtin_amdgcn_frexp_mantf(xs) * __builtin_amdgcn_frexp_mantf(sw);
  const int e = __builtin_amdgcn_frexp_expf(xs) + __builtin_amdgcn_frexp_expf(sw);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float one = fmaf(sums[j], factor, acc[j]), other = acc[j] + __builtin_ldexpf(sums[j] * m, e);
    acc[j] = as_it_is ? one : other;
  }
}

// Four neighbouring outputs of one row.
__device__ __forceinline__ void store4(const ProductParams& p, int64_t row, int64_t n, const f4& v) {
  if (row >= p.m) return;
  const int64_t at = row * p.y_stride + n;
  if (p.y_dtype == QPN_DT_F32) {
    float* y = static_cast<float*>(p.y) + at;
    if (p.y_vec && n + 4 <= p.n) {
      *reinterpret_cast<f4*>(y) = v;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < p.n) y[r] = v[r];
    }
    return;
  }
  uint16_t h[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) h[r] = p.y_dtype == QPN_DT_BF16 ? round16<true>(v[r]) : round16<false>(v[r]);
  uint16_t* y = static_cast<uint16_t*>(p.y) + at;
  if (p.y_vec && n + 4 <= p.n) {
    *reinterpret_cast<uint2*>(y) = uint2{h[0] | static_cast<uint32_t>(h[1]) << 16, h[2] | static_cast<uint32_t>(h[3]) << 16};
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n + r < p.n) y[r] = h[r];
  }
}

// 64 lanes x 16 bytes from memory to LDS, past the registers: lane l's go to
// dst + 16 l. M0 holds the place in LDS; the compiler does not track it, and
// nothing else here uses it.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
typedef __attribute__((address_space(3))) void* lds_void;
__device__ __forceinline__ void lds_dma(const uint8_t* base, uint32_t offset, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %2" ::"v"(offset), "s"(dst), "s"(base)
               : "memory", "m0");
}
// The same of 4 bytes a lane.
__device__ __forceinline__ void lds_dma4(const float* base, uint32_t offset, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, %2" ::"v"(offset), "s"(dst), "s"(base)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// Few rows: a workgroup takes 16 outputs, its wavefronts every WAVES-th block of k
// each; their sums are added in LDS in the order of the wavefronts. A block's
// codes come to LDS, kRing blocks a wavefront on their way, and only from there
// to the lanes that multiply them: neighbouring lanes hold neighbouring rows, and a
// load of 16 bytes from each costs the cache 64 accesses instead of 16 (16 rows x
// 5120 x 17408 34 us, with the memory's rate reached by neither more wavefronts
// nor more loads on their way). A wavefront's part of LDS is its own: no barrier.
//
// The weight's bytes bound it: one row x 34816 x 5120 29 us with the quantizer, 6.2
// TB/s; 16 rows x 5120 x 17408 20 us where half of the weight is in the last-level cache
// from the call before, 24 to 26 where all of it comes from memory (3.6 TB/s: 320
// workgroups on 256 compute units, and the quantizer's launch). fp32 results cost 1 us
// more there. Small calls are two launches: one row x 7168 x 5120 11 us for 6 us of bytes.
template <int MT, int WAVES, bool EXACT>
__global__ __launch_bounds__(WAVES * 64) void few_rows_kernel(const ProductParams p) {
  constexpr int kRing = 2, kTile = 16 * kScaleBlock;
  struct Slot {
    uint8_t w[kTile], x[MT][kTile];
    float scales[64];  // of all rows of x
  };
  constexpr int kLoads = 2 + 2 * MT + 1;
  __shared__ union {
    alignas(16) Slot ring[WAVES][kRing];
    f4 red[WAVES][MT][64];
  } sh;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const uint8_t* w = p.w + n0 * p.w_stride;
  const scalar_ptr ws = (scalar_ptr)(p.ws + n0 / kScaleBlock * p.ws_row);
  // what a lane brings: of rows lane / 8 and 8 + lane / 8 of a tile, one piece
  const uint32_t piece = ((lane & 7) ^ (lane >> 3)) * 16;
  uint32_t from_w[2], from_x[MT][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    from_w[h] = static_cast<uint32_t>(min(static_cast<int64_t>(h * 8 + lane / 8), p.n - 1 - n0) * p.w_stride) + piece;
#pragma unroll
    for (int t = 0; t < MT; ++t)
      from_x[t][h] = static_cast<uint32_t>(min(static_cast<int64_t>(t * 16 + h * 8 + lane / 8), p.m - 1) * p.x_stride) + piece;
  }
  const uint32_t from_s = static_cast<uint32_t>(min(static_cast<int64_t>(lane), p.m - 1) * p.xs_row * 4);
  const uint32_t ring0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void)(&sh.ring[wave][0])));
  const auto bring = [&](int b, int slot) {
    const uint32_t to = __builtin_amdgcn_readfirstlane(ring0 + slot * static_cast<uint32_t>(sizeof(Slot)));
    const int64_t at = static_cast<int64_t>(b) * kScaleBlock;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      lds_dma(w + at, from_w[h], to + h * 1024);
#pragma unroll
      for (int t = 0; t < MT; ++t) lds_dma(p.x + at, from_x[t][h], to + (1 + t) * kTile + h * 1024);
    }
    lds_dma4(p.xs + b * p.xs_block, from_s, to + (1 + MT) * kTile);
  };
  f4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = f4{0.f, 0.f, 0.f, 0.f};
  const int slot0 = i * kScaleBlock + ((g ^ (i & 7)) * 16), slot1 = i * kScaleBlock + (((g + 4) ^ (i & 7)) * 16);
  const auto frag = [&](const uint8_t* tile) {
    return Frag<EXACT>(*reinterpret_cast<const u4*>(tile + slot0), *reinterpret_cast<const u4*>(tile + slot1));
  };
  const int whole = p.k / kScaleBlock;  // blocks that are not cut by the end of k
  static_assert(kRing == 2, "the loop below keeps one block on its way");
  if (wave < whole) bring(wave, 0);
  int slot = 0;
#pragma unroll 1
  for (int b = wave; b < whole; b += WAVES, slot ^= 1) {
    if (b + WAVES < whole) {
      bring(b + WAVES, slot ^ 1);
      __builtin_amdgcn_s_waitcnt(vmcnt_only(kLoads));
    } else {
      __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const Slot& r = sh.ring[wave][slot];
    const float sw = ws[b * p.ws_block];
    const Frag<EXACT> wf = frag(r.w);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const float xs = r.scales[t * 16 + i], factor = xs * sw;
      const f4 sums = block_sums(wf, frag(r.x[t]));
      if (__all(ordinary(factor))) acc[t] += sums * factor;
      else add_scaled(acc[t], sums, xs, sw);
    }
    // (the reads are over before their place is asked to be filled again)
    __builtin_amdgcn_s_waitcnt(lgkmcnt_only(0));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  if (whole < p.blocks && whole % WAVES == wave) {
    // the short last block, piece by piece: those past the end of k are zeros
    const int64_t at = static_cast<int64_t>(whole) * kScaleBlock + g * 16;
    const float sw = ws[whole * p.ws_block];
    const Frag<EXACT> wf = short_frag<EXACT>(w + min(static_cast<int64_t>(i), p.n - 1 - n0) * p.w_stride, at, p.k);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int64_t row = min(static_cast<int64_t>(t * 16 + i), p.m - 1);
      add_scaled(acc[t], block_sums(wf, short_frag<EXACT>(p.x + row * p.x_stride, at, p.k)),
                 p.xs[row * p.xs_row + whole * p.xs_block], sw);
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < MT; ++t) sh.red[wave][t][lane] = acc[t];
  __syncthreads();
  for (int t = wave; t < MT; t += WAVES) {
    f4 v = sh.red[0][t][lane];
#pragma unroll
    for (int o = 1; o < WAVES; ++o) v += sh.red[o][t][lane];
    store4(p, t * 16 + i, n0 + 4 * g, v);
  }
}

// Many rows: MW x NW wavefronts of TM x TN tiles of 16 x 16 each. Both
// operands' 128 bytes of a block go to LDS, the next block's while this one is
// multiplied. A row's eight 16-byte pieces lie in LDS at piece ^ (row % 8), so
// that neighbouring rows' reads meet different banks.
//
// Within a block the products of one row tile are issued while the sums of the
// one before are scaled, and the next one's codes are on their way: a result
// that is used at once costs the pipeline's depth (2048 x 34816 x 5120: 534 us
// before, 404 to 440 since). At 256 x 256 that takes all registers: the last tile
// of rows begins early enough to be whole (its rows are computed twice, to the same
// bits), and one offset serves all of a thread's rows of x.
//
// What bounds it there (2048 x 34816 x 5120, 394 to 402 us with the quantizer, 1.85
// PFLOP/s): of the cycles, matrix instructions take 46 % and vector ones 40 %, four
// multiply-adds a lane for each instruction's sums among them, at a clock of 2.0 to 2.1
// GHz under load (over zeros, which draw less power: 372 us where it took 397).
// Tiles of 64 wait: matrix instructions 8 % and vector ones 15 % of the cycles at 777 x
// 1795 x 1296, 19.5 us for an fp32 result, of which rows of an odd length cost 2.6
// (16.9 at 1796) and fp16 instructions little (17.2 for bf16). With four blocks in LDS
// instead of two, fewer workgroups fit: 21 us.
//
// Workgroups go round the eight dies. Each die takes an eighth of the tiles, row
// tiles first: its 32 compute units read 8 x 4 tiles' rows between them rather
// than 1 x 32, from a cache that holds a fraction of either operand.
template <int MW, int NW, int TM, int TN, bool EXACT>
__global__ __launch_bounds__(MW * NW * 64, 2) void many_rows_kernel(const ProductParams p) {
  constexpr int kThreads = MW * NW * 64, kM = MW * TM * 16, kN = NW * TN * 16;
  constexpr bool kWhole = kM == 256;  // every tile's rows are there
  constexpr int kStage = (kM + kN) * kScaleBlock, kRowsAtOnce = kThreads / 8;
  constexpr int kLoadsX = kM / kRowsAtOnce, kLoadsW = kN / kRowsAtOnce;
  static_assert(kM % kRowsAtOnce == 0 && kN % kRowsAtOnce == 0 && kRowsAtOnce % 8 == 0, "whole loads of either operand");
  static_assert(kScaleBlock % (TN * 16) == 0, "a wavefront's outputs share their scale");
  __shared__ alignas(16) uint8_t lds[2][kStage];  // x rows, then w rows
  __shared__ alignas(16) float scales[2][kM];     // of x: a wavefront's rows t * 16 + i at i * TM + t
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int m_tiles = static_cast<int>((p.m + kM - 1) / kM);
  const int per_die = (gridDim.x + 7) / 8, tile = blockIdx.x % 8 * per_die + blockIdx.x / 8;
  if (tile >= p.tiles) return;  // (the grid is a multiple of 8)
  const int64_t m_first = static_cast<int64_t>(tile % m_tiles) * kM;
  const int64_t m0 = kWhole ? min(m_first, p.m - kM) : m_first, n0 = p.n_first + tile / m_tiles * static_cast<int64_t>(kN);
  const int wm = wave % MW, wn = wave / MW;
  const int split = blockIdx.y;
  const int b0 = static_cast<int>(static_cast<int64_t>(p.blocks) * split / p.splits);
  const int b1 = static_cast<int>(static_cast<int64_t>(p.blocks) * (split + 1) / p.splits);
  const uint8_t* x = p.x + m0 * p.x_stride;
  const uint8_t* w = p.w + n0 * p.w_stride;
  // the rows and pieces that this thread brings: row tid / 8 of every kRowsAtOnce
  const uint32_t piece = ((tid & 7) ^ (tid >> 3 & 7)) * 16;
  uint32_t from_x[kWhole ? 1 : kLoadsX], from_w[kLoadsW];
#pragma unroll
  for (int j = 0; j < (kWhole ? 1 : kLoadsX); ++j)
    from_x[j] = static_cast<uint32_t>(min(static_cast<int64_t>(j * kRowsAtOnce + tid / 8), p.m - 1 - m0) * p.x_stride) + piece;
#pragma unroll
  for (int j = 0; j < kLoadsW; ++j)
    from_w[j] = static_cast<uint32_t>(min(static_cast<int64_t>(j * kRowsAtOnce + tid / 8), p.n - 1 - n0) * p.w_stride) + piece;
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void)(&lds[0][0]))) + wave * 1024;
  const auto x_rows = [&](int b, int j) {
    return x + static_cast<int64_t>(b) * kScaleBlock + (kWhole ? j * kRowsAtOnce * p.x_stride : 0);
  };
  // Load j of this wavefront's of a whole block.
  const auto bring = [&](int b, int buf, int j) {
    const uint32_t to = __builtin_amdgcn_readfirstlane(lds0 + buf * kStage + j * kThreads * 16);
    if (j < kLoadsX) lds_dma(x_rows(b, j), from_x[kWhole ? 0 : j], to);
    else lds_dma(w + static_cast<int64_t>(b) * kScaleBlock, from_w[j - kLoadsX], to);
  };
  // The short last block: pieces past the end of k are zeros.
  const auto bring_short = [&](int b, int buf) {
    const bool in = b * kScaleBlock + static_cast<int>(piece) < p.k;
#pragma unroll
    for (int j = 0; j < kLoadsX + kLoadsW; ++j) {
      const uint8_t* from = j < kLoadsX ? x_rows(b, j) + from_x[kWhole ? 0 : j]
                                        : w + static_cast<int64_t>(b) * kScaleBlock + from_w[j < kLoadsX ? 0 : j - kLoadsX];
      u4 v = {0u, 0u, 0u, 0u};
      if (in) v = *reinterpret_cast<const u4*>(from);
      *reinterpret_cast<u4*>(&lds[buf][(j * kThreads + tid) * 16]) = v;
    }
  };
  // x's scales: 64 rows a wavefront's, by the first kM / 64 of them.
  const uint32_t scale_slot = wave * 64 + lane, scale_part = scale_slot / (TM * 16), in_part = scale_slot % (TM * 16);
  const uint32_t from_s = static_cast<uint32_t>(
      min(static_cast<int64_t>(scale_part * (TM * 16) + in_part % TM * 16 + in_part / TM), p.m - 1 - m0) * p.xs_row * 4);
  const uint32_t scales0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void)(&scales[0][0]))) + wave * 256;
  const auto bring_scales = [&](int b, int buf) {
    if (wave < kM / 64)
      lds_dma4(p.xs + m0 * p.xs_row + b * p.xs_block, from_s, __builtin_amdgcn_readfirstlane(scales0 + buf * kM * 4));
  };
  const int64_t w_block = n0 + wn * TN * 16 < p.n ? (n0 + wn * TN * 16) / kScaleBlock : 0;
  const scalar_ptr ws = (scalar_ptr)(p.ws + w_block * p.ws_row);
  f4 acc[TM][TN];
#pragma unroll
  for (int t = 0; t < TM; ++t)
#pragma unroll
    for (int u = 0; u < TN; ++u) acc[t][u] = f4{0.f, 0.f, 0.f, 0.f};
  const int slot0 = ((g ^ (i & 7)) * 16), slot1 = (((g + 4) ^ (i & 7)) * 16);
  constexpr int kLoads = kLoadsX + kLoadsW;
  float sw = 0.f;
  bool plain = true;
  if (b0 < b1) {
    bring_scales(b0, 0);
    sw = ws[b0 * p.ws_block];
    if ((b0 + 1) * kScaleBlock <= p.k) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) bring(b0, 0, j);
    } else {
      bring_short(b0, 0);
    }
  }
  for (int b = b0; b < b1; ++b) {
    const int buf = (b - b0) & 1;
    __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
    __syncthreads();
    const uint8_t* xt = &lds[buf][(wm * TM * 16 + i) * kScaleBlock];
    const uint8_t* wt = &lds[buf][(kM + wn * TN * 16 + i) * kScaleBlock];
    const auto frag = [&](const uint8_t* rows) {
      return Frag<EXACT>(*reinterpret_cast<const u4*>(rows + slot0), *reinterpret_cast<const u4*>(rows + slot1));
    };
    Frag<EXACT> wf[TN], xf[2];
    xf[0] = frag(xt);
#pragma unroll
    for (int u = 0; u < TN; ++u) wf[u] = frag(wt + u * 16 * kScaleBlock);
    typedef float row_scales __attribute__((ext_vector_type(TM)));
    const row_scales s = *reinterpret_cast<const row_scales*>(&scales[buf][(wm * 16 + i) * TM]) * sw;
#pragma unroll
    for (int t = 0; t < TM; ++t) plain &= ordinary(s[t]);
    const bool more = b + 1 < b1, whole = (b + 2) * kScaleBlock <= p.k;
    if (more) {
      bring_scales(b + 1, buf ^ 1);
      sw = ws[(b + 1) * p.ws_block];
      if (!whole) bring_short(b + 1, buf ^ 1);
    }
    f4 sums[2][TN];
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t <= TM; ++t) {
      if (t + 1 < TM) xf[(t + 1) & 1] = frag(xt + (t + 1) * 16 * kScaleBlock);
      // (the next block's loads are spread over the first half of this one: all at once they stand in the way of LDS reads)
      if (t < TM / 2 && more && whole) {
#pragma unroll
        for (int j = kLoads * t / (TM / 2); j < kLoads * (t + 1) / (TM / 2); ++j) bring(b + 1, buf ^ 1, j);
      }
#pragma unroll
      for (int u = 0; u < TN; ++u) {
        if (t < TM) sums[t & 1][u] = block_sums(wf[u], xf[t & 1]);
        if (t > 0) {
          acc[t - 1][u] += sums[(t - 1) & 1][u] * s[t - 1];
          asm volatile("" : "+v"(acc[t - 1][u]));  // (here: the compiler would gather them behind the loads)
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  // Factors outside the normal range were met: the wavefront's sums once more, from memory, unless the scales
  // were zeros, infinities or NaN themselves.
  if (!__all(plain)) {
    const auto row_of = [&](int t) { return min(m0 + (wm * TM + t) * 16 + i, p.m - 1); };
    bool left = false;
    for (int b = b0; b < b1; ++b) {
      const float one = ws[b * p.ws_block];
      for (int t = 0; t < TM; ++t) {
        const float xs = p.xs[row_of(t) * p.xs_row + b * p.xs_block];
        left |= !ordinary(xs * one) && finite_not_zero(xs) && finite_not_zero(one);
      }
    }
    if (__any(left)) {
#pragma unroll
      for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int u = 0; u < TN; ++u) acc[t][u] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int b = b0; b < b1; ++b) {
        const int64_t at = static_cast<int64_t>(b) * kScaleBlock + g * 16;
        const float one = ws[b * p.ws_block];
        Frag<EXACT> wf[TN];
#pragma unroll
        for (int u = 0; u < TN; ++u)
          wf[u] = short_frag<EXACT>(p.w + min(n0 + (wn * TN + u) * 16 + i, p.n - 1) * p.w_stride, at, p.k);
#pragma unroll
        for (int t = 0; t < TM; ++t) {
          const Frag<EXACT> xf = short_frag<EXACT>(p.x + row_of(t) * p.x_stride, at, p.k);
          const float xs = p.xs[row_of(t) * p.xs_row + b * p.xs_block];
#pragma unroll
          for (int u = 0; u < TN; ++u) {
            add_scaled(acc[t][u], block_sums(wf[u], xf), xs, one);
            asm volatile("" : "+v"(acc[t][u]));
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    const int64_t row = m0 + (wm * TM + t) * 16 + i;
#pragma unroll
    for (int u = 0; u < TN; ++u) {
      const int64_t n = n0 + (wn * TN + u) * 16 + 4 * g;
      if (p.splits == 1) {
        store4(p, row, n, acc[t][u]);
      } else if (row < p.m) {
        float* d = p.partial + (split * p.m + row) * p.n + n;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n + r < p.n) d[r] = acc[t][u][r];
      }
    }
  }
}

// Adds the partial sums of a split k, in the order of k.
__global__ __launch_bounds__(256) void join_kernel(const ProductParams p) {
  const int64_t quads = (p.n + 3) / 4;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t row = at / quads, n = (at - row * quads) * 4;
  if (row >= p.m) return;
  f4 v = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < p.splits; ++s) {
    const float* d = p.partial + (s * p.m + row) * p.n + n;
    if (p.n % 4 == 0) {
      v += *reinterpret_cast<const f4*>(d);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < p.n) v[r] += d[r];
    }
  }
  store4(p, row, n, v);
}

template <int MT, bool EXACT>
hipError_t launch_few(int waves, uint32_t grid, const ProductParams& p, hipStream_t stream) {
  switch (waves) {
    case 4: few_rows_kernel<MT, 4, EXACT><<<dim3(grid), dim3(256), 0, stream>>>(p); break;
    case 8:
      if constexpr (MT < 4) few_rows_kernel<MT, 8, EXACT><<<dim3(grid), dim3(512), 0, stream>>>(p);
      else return hipErrorInvalidValue;
      break;
    default:
      if constexpr (MT == 1) few_rows_kernel<MT, 16, EXACT><<<dim3(grid), dim3(1024), 0, stream>>>(p);
      else return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_block_quantize(const void* x, int32_t dtype, int64_t rows, int64_t k, int64_t stride,
                                     int32_t block_rows, uint8_t* codes, int64_t code_stride, float* scales,
                                     int64_t scale_row_stride, int64_t scale_block_stride, hipStream_t stream) {
  QuantizeParams a;
  a.x = x, a.codes = codes, a.scales = scales;
  a.rows = rows, a.k = k, a.stride = stride, a.code_stride = code_stride;
  a.scale_row_stride = scale_row_stride, a.scale_block_stride = scale_block_stride;
  a.blocks = static_cast<int32_t>((k + kScaleBlock - 1) / kScaleBlock);
  const int per16 = dtype == QPN_DT_F32 ? 4 : 8;
  a.load_vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && (stride % per16 == 0 || rows == 1);
  a.store_vec = reinterpret_cast<uintptr_t>(codes) % 8 == 0 && (code_stride % 8 == 0 || rows == 1);
  if (block_rows == 1) {
    const dim3 grid(static_cast<uint32_t>((rows * a.blocks + 15) / 16));
    switch (dtype) {
      case QPN_DT_F16: quantize_rows_kernel<QPN_DT_F16><<<grid, dim3(256), 0, stream>>>(a); break;
      case QPN_DT_BF16: quantize_rows_kernel<QPN_DT_BF16><<<grid, dim3(256), 0, stream>>>(a); break;
      default: quantize_rows_kernel<QPN_DT_F32><<<grid, dim3(256), 0, stream>>>(a); break;
    }
  } else {
    const dim3 grid(static_cast<uint32_t>((rows + kScaleBlock - 1) / kScaleBlock * a.blocks));
    switch (dtype) {
      case QPN_DT_F16: quantize_blocks_kernel<QPN_DT_F16><<<grid, dim3(256), 0, stream>>>(a); break;
      case QPN_DT_BF16: quantize_blocks_kernel<QPN_DT_BF16><<<grid, dim3(256), 0, stream>>>(a); break;
      default: quantize_blocks_kernel<QPN_DT_F32><<<grid, dim3(256), 0, stream>>>(a); break;
    }
  }
  return hipGetLastError();
}

hipError_t launch_fp8_block_gemm(const qpn_fp8_block_gemm_args& a, const Fp8BlockPlan& plan, void* workspace,
                                 hipStream_t stream) {
  ProductParams p = {};
  uint8_t* base = static_cast<uint8_t*>(workspace);
  float* own_scales = reinterpret_cast<float*>(base + plan.code_bytes);
  if (a.x_dtype == QPN_DT_E4M3) {
    p.x = static_cast<const uint8_t*>(a.x), p.x_stride = a.x_stride;
    p.xs = a.x_scales, p.xs_row = a.x_scale_row_stride, p.xs_block = a.x_scale_block_stride;
  } else {
    p.x = base, p.x_stride = a.k;
    p.xs = own_scales, p.xs_row = 1, p.xs_block = a.m;  // a block's scales of neighbouring rows lie together
    if (a.k > 0) {
      const hipError_t e = launch_fp8_block_quantize(a.x, a.x_dtype, a.m, a.k, a.x_stride, 1, base, a.k, own_scales, 1,
                                                     a.m, stream);
      if (e != hipSuccess) return e;
    }
  }
  p.w = a.w, p.w_stride = a.w_stride;
  p.ws = a.w_scales, p.ws_row = a.w_scale_row_stride, p.ws_block = a.w_scale_block_stride;
  p.y = a.y, p.y_stride = a.y_stride, p.y_dtype = a.y_dtype;
  const int size = a.y_dtype == QPN_DT_F32 ? 4 : 2;
  p.y_vec = reinterpret_cast<uintptr_t>(a.y) % (4 * size) == 0 && (a.y_stride % 4 == 0 || a.m == 1);
  p.m = a.m, p.n = a.n, p.k = static_cast<int32_t>(a.k), p.blocks = plan.blocks, p.splits = plan.splits;
  p.partial = reinterpret_cast<float*>(base + plan.code_bytes + plan.scale_bytes);
  if (plan.m_tiles > 0) {
    const uint32_t grid = static_cast<uint32_t>((a.n + 15) / 16);
    const bool exact = a.y_dtype == QPN_DT_F32;
    switch (plan.m_tiles) {
      case 1: return exact ? launch_few<1, true>(plan.waves, grid, p, stream) : launch_few<1, false>(plan.waves, grid, p, stream);
      case 2: return exact ? launch_few<2, true>(plan.waves, grid, p, stream) : launch_few<2, false>(plan.waves, grid, p, stream);
      case 3: return exact ? launch_few<3, true>(plan.waves, grid, p, stream) : launch_few<3, false>(plan.waves, grid, p, stream);
      default: return exact ? launch_few<4, true>(plan.waves, grid, p, stream) : launch_few<4, false>(plan.waves, grid, p, stream);
    }
  }
  const bool exact = a.y_dtype == QPN_DT_F32;
  const auto launch = [&](int tile, int64_t first, int64_t last) {
    p.n_first = first;
    p.tiles = static_cast<int32_t>((a.m + tile - 1) / tile * ((last - first + tile - 1) / tile));
    const dim3 grid(static_cast<uint32_t>((p.tiles + 7) / 8 * 8), static_cast<uint32_t>(plan.splits));
    if (tile == 256)
      many_rows_kernel<2, 4, 8, 4, false><<<grid, dim3(512), 0, stream>>>(p);
    else if (tile == 128 && exact)
      many_rows_kernel<2, 2, 4, 4, true><<<grid, dim3(256), 0, stream>>>(p);
    else if (tile == 128)
      many_rows_kernel<2, 2, 4, 4, false><<<grid, dim3(256), 0, stream>>>(p);
    else if (exact)
      many_rows_kernel<2, 2, 2, 2, true><<<grid, dim3(256), 0, stream>>>(p);
    else
      many_rows_kernel<2, 2, 2, 2, false><<<grid, dim3(256), 0, stream>>>(p);
    return hipGetLastError();
  };
  // (fp32 results: 16 fp16 fragments beside 128 sums would not fit the registers)
  if (!exact && plan.wide > 0) {
    const hipError_t e = launch(256, 0, std::min(plan.wide, a.n));
    if (e != hipSuccess || plan.wide >= a.n) return e;
    return launch(128, plan.wide, a.n);
  }
  hipError_t e = launch(plan.tile, 0, a.n);
  if (e != hipSuccess || plan.splits == 1) return e;
  const int64_t quads = a.m * ((a.n + 3) / 4);
  join_kernel<<<dim3(static_cast<uint32_t>((quads + 255) / 256)), dim3(256), 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace qpn
