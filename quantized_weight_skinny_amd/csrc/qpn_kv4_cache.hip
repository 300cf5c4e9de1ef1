// The 4-bit paged cache of include/qpn_decode.h: quantizing keys and values
// into it, reading them back, and copying pages.
#include "qpn_decode_internal.hpp"
#include "qpn_device.hpp"

namespace qpn {
namespace {

constexpr int kThreads = 256;

struct PoolRef {
  uint8_t* layer;
  int64_t page_bytes, slots;  // slots: pages * page_size
  int32_t page_shift, page, kv_heads, dim, seg_bytes;
};

PoolRef pool_ref(const qpn_kv4_cache& c, int32_t layer) {
  PoolRef p;
  p.page_bytes = static_cast<int64_t>(qpn_kv4_page_bytes(c.page_size, c.kv_heads, c.head_dim));
  p.layer = static_cast<uint8_t*>(c.data) + p.page_bytes * c.pages * layer;
  p.slots = c.pages * c.page_size;
  p.page_shift = __builtin_ctz(c.page_size);
  p.page = c.page_size;
  p.kv_heads = c.kv_heads;
  p.dim = c.head_dim;
  p.seg_bytes = static_cast<int32_t>(kv4_segment_bytes(c.page_size, c.head_dim));
  return p;
}

// Where block `blk` (16 elements) of one head's token at `slot` lies: its codes
// (K: 8 bytes; V: pieces of dim / 32 bytes, dim / 8 apart) and its scale byte.
struct BlockRef {
  uint8_t *codes, *scale;
};

template <int DIM, bool V>
__device__ __forceinline__ BlockRef block_ref(const PoolRef& p, int64_t slot, int head, int blk) {
  uint8_t* seg = p.layer + (slot >> p.page_shift) * p.page_bytes + static_cast<int64_t>(head) * p.seg_bytes;
  const int off = static_cast<int>(slot) & (p.page - 1);
  BlockRef r;
  if constexpr (V) {
    // the block's 256 / DIM groups of D / 16 elements
    r.codes = seg + p.page * (DIM / 2) + (off >> 2) * (2 * DIM) + blk * (256 / DIM) * (DIM / 8) + (off & 3) * (DIM / 32);
    r.scale = seg + p.page * DIM + p.page * (DIM / 16) + (off >> 2) * (DIM / 4) + blk * 4 + (off & 3);
  } else {
    r.codes = seg + off * (DIM / 2) + blk * 8;
    r.scale = seg + p.page * DIM + off * (DIM / 16) + blk;
  }
  return r;
}

template <int DIM, bool V>
__device__ __forceinline__ void store_block(const BlockRef& r, uint32_t lo, uint32_t hi, uint32_t sc) {
  if constexpr (!V || DIM == 256) {
    *reinterpret_cast<uint2*>(r.codes) = make_uint2(lo, hi);
  } else if constexpr (DIM == 128) {
    *reinterpret_cast<uint32_t*>(r.codes) = lo;
    *reinterpret_cast<uint32_t*>(r.codes + 16) = hi;
  } else {
    *reinterpret_cast<uint16_t*>(r.codes) = static_cast<uint16_t>(lo);
    *reinterpret_cast<uint16_t*>(r.codes + 8) = static_cast<uint16_t>(lo >> 16);
    *reinterpret_cast<uint16_t*>(r.codes + 16) = static_cast<uint16_t>(hi);
    *reinterpret_cast<uint16_t*>(r.codes + 24) = static_cast<uint16_t>(hi >> 16);
  }
  *r.scale = static_cast<uint8_t>(sc);
}

template <int DIM, bool V>
__device__ __forceinline__ uint2 load_block(const BlockRef& r) {
  if constexpr (!V || DIM == 256) {
    return *reinterpret_cast<const uint2*>(r.codes);
  } else if constexpr (DIM == 128) {
    return make_uint2(*reinterpret_cast<const uint32_t*>(r.codes), *reinterpret_cast<const uint32_t*>(r.codes + 16));
  } else {
    const auto at = [&](int o) { return static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(r.codes + o)); };
    return make_uint2(at(0) | at(8) << 16, at(16) | at(24) << 16);
  }
}

// One block of 16 values (as 16-bit words): its scale byte and its codes (two
// dwords). `plain`: the tensor scale is far enough from the ends of fp32 for
// the quotients below.
//
// The codes are those of fp32 division and the nearest-even rule. A division
// an element would be a third of the kernel's instructions, so the block
// divides once: with r = 1 / d correctly rounded and q = x * r, off by at most
// an ulp, q + (x - q d) r, the residual exact in a fused multiply-add, is the
// correctly rounded x / d. (Where x r overflows the correction gives NaN, which
// the conversion takes to the largest code, as it does an infinite quotient.)
// Blocks with an infinity or NaN take the division.
// 16389 tokens of 2 x 1024 elements: 37 us with divisions and a comparison
// for every midpoint, 21 us so (4.1 TB/s of values in and codes out).
template <bool BF16>
__device__ __forceinline__ uint32_t quantize_block(const u4 (&w)[2], float s_t, bool plain, uint32_t& lo, uint32_t& hi) {
  // magnitudes of 16-bit floats are ordered as their bits are
  typedef unsigned short us2 __attribute__((ext_vector_type(2)));
  us2 top2 = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t x = w[j / 4][j % 4] & 0x7FFF7FFFu;
    top2 = __builtin_elementwise_max(top2, __builtin_bit_cast(us2, x));
  }
  const uint32_t top = max(static_cast<uint32_t>(top2[0]), static_cast<uint32_t>(top2[1]));
  constexpr uint32_t kInf = BF16 ? 0x7F80u : 0x7C00u;
  float v[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = widen16<BF16>((w[e / 8][e / 2 % 4] >> (16 * (e & 1))) & 0xFFFFu);
  float amax = widen16<BF16>(top);
  if (top > kInf) {
    // the largest that is a number
    amax = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(v[e]));
  }
  const uint32_t sc = encode_e4m3(amax / 6.0f / s_t);
  const float d = decode_e4m3(sc) * s_t;
  lo = 0u, hi = 0u;
  if (plain && top < kInf && d != 0.f) {
    const float r = 1.0f / d;
    float q[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float q0 = v[e] * r;
      // (a zero keeps its sign)
      q[e] = copysignf(fmaf(fmaf(-q0, d, v[e]), r, q0), v[e]);
    }
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, q[0], q[1], 1.0f, 0);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, q[2], q[3], 1.0f, 1);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, q[4], q[5], 1.0f, 2);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, q[6], q[7], 1.0f, 3);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, q[8], q[9], 1.0f, 0);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, q[10], q[11], 1.0f, 1);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, q[12], q[13], 1.0f, 2);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, q[14], q[15], 1.0f, 3);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint32_t c = d == 0.f ? ((__float_as_uint(v[e]) >> 28) & 0x8u) : encode_e2m1(v[e] / d);
      if (e < 8) lo |= c << (4 * e);
      else hi |= c << (4 * (e - 8));
    }
  }
  return sc;
}

struct Source {
  const uint16_t* data;
  int64_t ts, hs;
  int32_t aligned;  // rows start on 16 bytes
  float scale;
  bool plain;       // the scale lies between 2^-60 and 2^60
};

template <int DIM, bool BF16, bool V>
__device__ __forceinline__ void append_block(const PoolRef& p, const Source& s, int64_t t, int64_t slot, int head,
                                             int blk) {
  const uint16_t* src = s.data + t * s.ts + head * s.hs + blk * 16;
  u4 w[2];
  if (s.aligned) {
#pragma unroll
    for (int j = 0; j < 2; ++j) w[j] = reinterpret_cast<const u4*>(src)[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j / 4][j % 4] = src[2 * j] | static_cast<uint32_t>(src[2 * j + 1]) << 16;
  }
  uint32_t lo, hi;
  const uint32_t sc = quantize_block<BF16>(w, s.scale, s.plain, lo, hi);
  store_block<DIM, V>(block_ref<DIM, V>(p, slot, head, blk), lo, hi, sc);
}

// A thread a block of 16 elements of K or V; blocks of one token run fastest.
template <int DIM, bool BF16>
__global__ __launch_bounds__(kThreads) void kv4_append_kernel(const PoolRef p, const Source k, const Source v,
                                                              const int64_t* __restrict__ slots, int64_t tokens) {
  const int per = p.kv_heads * (DIM / 16);
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t t = idx / per;
  if (t >= tokens) return;
  const int64_t slot = slots[t];
  if (slot < 0 || slot >= p.slots) return;
  const int w = static_cast<int>(idx - t * per), head = w / (DIM / 16), blk = w % (DIM / 16);
  if (blockIdx.y == 0)
    append_block<DIM, BF16, false>(p, k, t, slot, head, blk);
  else
    append_block<DIM, BF16, true>(p, v, t, slot, head, blk);
}

template <int DIM, typename Out, bool BF16, bool V>
__device__ __forceinline__ void read_block(const PoolRef& p, float scale, int64_t slot, int head, int blk, Out* dst) {
  float x[16];
  if (slot < 0 || slot >= p.slots) {
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = 0.f;
  } else {
    const BlockRef r = block_ref<DIM, V>(p, slot, head, blk);
    const uint2 c = load_block<DIM, V>(r);
    const h2 sc = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(static_cast<uint32_t>(*r.scale), 1.0f, false);
    const h8 a = decode_fp4x8(c.x, h2{sc.x, sc.x}), b = decode_fp4x8(c.y, h2{sc.x, sc.x});
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = static_cast<float>(a[e]) * scale, x[8 + e] = static_cast<float>(b[e]) * scale;
  }
  if constexpr (sizeof(Out) == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) reinterpret_cast<f4*>(dst)[j] = f4{x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]};
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      u4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float lo = x[8 * j + 2 * e], hi = x[8 * j + 2 * e + 1];
        if constexpr (!BF16) {  // fp16 saturates; a NaN passes
          lo = fabsf(lo) > 65504.f ? copysignf(65504.f, lo) : lo;
          hi = fabsf(hi) > 65504.f ? copysignf(65504.f, hi) : hi;
        }
        w[e] = round16<BF16>(lo) | static_cast<uint32_t>(round16<BF16>(hi)) << 16;
      }
      reinterpret_cast<u4*>(dst)[j] = w;
    }
  }
}

template <int DIM, typename Out, bool BF16>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(const PoolRef p, float k_scale, float v_scale,
                                                            const int64_t* __restrict__ slots, int64_t tokens,
                                                            Out* __restrict__ k, Out* __restrict__ v) {
  const int per = p.kv_heads * (DIM / 16);
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t t = idx / per;
  if (t >= tokens) return;
  const int64_t slot = slots[t];
  const int w = static_cast<int>(idx - t * per), head = w / (DIM / 16), blk = w % (DIM / 16);
  if (blockIdx.y == 0)
    read_block<DIM, Out, BF16, false>(p, k_scale, slot, head, blk, k + idx * 16);
  else
    read_block<DIM, Out, BF16, true>(p, v_scale, slot, head, blk, v + idx * 16);
}

// 16-byte vectors: page_bytes is a multiple of 16.
constexpr int kCopyVectors = 4;  // a thread's loads in flight

__global__ __launch_bounds__(kThreads) void kv4_copy_pages_kernel(uint8_t* data, int64_t layer_bytes,
                                                                  int64_t page_bytes, int32_t pages,
                                                                  const int32_t* __restrict__ src,
                                                                  const int32_t* __restrict__ dst, int32_t pieces) {
  const int64_t pair = blockIdx.x / pieces;
  const int piece = static_cast<int>(blockIdx.x - pair * pieces);
  const int s = src[pair], d = dst[pair];
  if (s < 0 || s >= pages || d < 0 || d >= pages || s == d) return;
  uint8_t* layer = data + layer_bytes * blockIdx.y;
  const u4* from = reinterpret_cast<const u4*>(layer + page_bytes * s);
  u4* to = reinterpret_cast<u4*>(layer + page_bytes * d);
  const int vectors = static_cast<int>(page_bytes / 16);
  const int v0 = piece * (kThreads * kCopyVectors) + threadIdx.x;
  u4 x[kCopyVectors];
#pragma unroll
  for (int j = 0; j < kCopyVectors; ++j)
    if (v0 + j * kThreads < vectors) x[j] = __builtin_nontemporal_load(from + v0 + j * kThreads);
#pragma unroll
  for (int j = 0; j < kCopyVectors; ++j)
    if (v0 + j * kThreads < vectors) __builtin_nontemporal_store(x[j], to + v0 + j * kThreads);
}

template <int DIM>
hipError_t append_dim(const PoolRef& p, const Source& k, const Source& v, int32_t dtype, const int64_t* slots,
                      int64_t tokens, hipStream_t stream) {
  const int64_t threads = tokens * p.kv_heads * (DIM / 16);
  const dim3 grid(static_cast<uint32_t>((threads + kThreads - 1) / kThreads), 2);
  if (dtype == QPN_DT_BF16)
    kv4_append_kernel<DIM, true><<<grid, kThreads, 0, stream>>>(p, k, v, slots, tokens);
  else
    kv4_append_kernel<DIM, false><<<grid, kThreads, 0, stream>>>(p, k, v, slots, tokens);
  return hipGetLastError();
}

template <int DIM>
hipError_t read_dim(const PoolRef& p, const qpn_kv4_cache& c, int32_t dtype, const int64_t* slots, int64_t tokens,
                    void* k, void* v, hipStream_t stream) {
  const int64_t threads = tokens * p.kv_heads * (DIM / 16);
  const dim3 grid(static_cast<uint32_t>((threads + kThreads - 1) / kThreads), 2);
  if (dtype == QPN_DT_F32)
    kv4_read_kernel<DIM, float, false><<<grid, kThreads, 0, stream>>>(p, c.k_scale, c.v_scale, slots, tokens,
                                                                      static_cast<float*>(k), static_cast<float*>(v));
  else if (dtype == QPN_DT_BF16)
    kv4_read_kernel<DIM, uint16_t, true><<<grid, kThreads, 0, stream>>>(
        p, c.k_scale, c.v_scale, slots, tokens, static_cast<uint16_t*>(k), static_cast<uint16_t*>(v));
  else
    kv4_read_kernel<DIM, uint16_t, false><<<grid, kThreads, 0, stream>>>(
        p, c.k_scale, c.v_scale, slots, tokens, static_cast<uint16_t*>(k), static_cast<uint16_t*>(v));
  return hipGetLastError();
}

// Tokens a launch takes at most, so that its grid stays below 2^31 workgroups' threads.
int64_t tokens_per_launch(int kv_heads, int dim) { return (int64_t(1) << 30) / (kv_heads * (dim / 16)); }

}  // namespace

hipError_t launch_kv4_append(const qpn_kv4_cache& c, int32_t layer, const void* k, const void* v, int32_t dtype,
                             int64_t tokens, int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs,
                             const int64_t* slots, hipStream_t stream) {
  const PoolRef p = pool_ref(c, layer);
  const auto source = [](const void* x, int64_t ts, int64_t hs, float scale) {
    const bool al = reinterpret_cast<uintptr_t>(x) % 16 == 0 && ts % 8 == 0 && hs % 8 == 0;
    return Source{static_cast<const uint16_t*>(x), ts, hs, al, scale, scale > 0x1p-60f && scale < 0x1p60f};
  };
  const int64_t most = tokens_per_launch(c.kv_heads, c.head_dim);
  for (int64_t t = 0; t < tokens; t += most) {
    const int64_t n = tokens - t < most ? tokens - t : most;
    const Source ks = source(static_cast<const uint16_t*>(k) + t * k_ts, k_ts, k_hs, c.k_scale);
    const Source vs = source(static_cast<const uint16_t*>(v) + t * v_ts, v_ts, v_hs, c.v_scale);
    const hipError_t e = c.head_dim == 64    ? append_dim<64>(p, ks, vs, dtype, slots + t, n, stream)
                         : c.head_dim == 128 ? append_dim<128>(p, ks, vs, dtype, slots + t, n, stream)
                                             : append_dim<256>(p, ks, vs, dtype, slots + t, n, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_kv4_read(const qpn_kv4_cache& c, int32_t layer, const int64_t* slots, int64_t tokens, int32_t dtype,
                           void* k, void* v, hipStream_t stream) {
  const PoolRef p = pool_ref(c, layer);
  const int64_t most = tokens_per_launch(c.kv_heads, c.head_dim);
  const int64_t row = static_cast<int64_t>(c.kv_heads) * c.head_dim * (dtype == QPN_DT_F32 ? 4 : 2);
  for (int64_t t = 0; t < tokens; t += most) {
    const int64_t n = tokens - t < most ? tokens - t : most;
    void* kt = static_cast<uint8_t*>(k) + t * row;
    void* vt = static_cast<uint8_t*>(v) + t * row;
    const hipError_t e = c.head_dim == 64    ? read_dim<64>(p, c, dtype, slots + t, n, kt, vt, stream)
                         : c.head_dim == 128 ? read_dim<128>(p, c, dtype, slots + t, n, kt, vt, stream)
                                             : read_dim<256>(p, c, dtype, slots + t, n, kt, vt, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_kv4_copy_pages(const qpn_kv4_cache& c, const int32_t* src, const int32_t* dst, int64_t count,
                                 hipStream_t stream) {
  const int64_t page_bytes = static_cast<int64_t>(qpn_kv4_page_bytes(c.page_size, c.kv_heads, c.head_dim));
  const int pieces = static_cast<int>((page_bytes / 16 + kThreads * kCopyVectors - 1) / (kThreads * kCopyVectors));
  const int64_t most = (int64_t(1) << 22) / pieces;  // pairs a launch
  for (int64_t i = 0; i < count; i += most) {
    const int64_t n = count - i < most ? count - i : most;
    for (int32_t layer = 0; layer < c.layers; layer += 65535) {
      const int32_t layers = c.layers - layer < 65535 ? c.layers - layer : 65535;
      kv4_copy_pages_kernel<<<dim3(static_cast<uint32_t>(n * pieces), layers), kThreads, 0, stream>>>(
          static_cast<uint8_t*>(c.data) + page_bytes * c.pages * layer, page_bytes * c.pages, page_bytes,
          static_cast<int32_t>(c.pages), src + i, dst + i, pieces);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace qpn
