// act_pack.cuh -- activations kept in 8 bits between the forward and the
// backward pass.
//
// A row of `cols` values is cut into blocks of 128 (the last one may be
// shorter).  Each block keeps one power of two 2^e, the smallest with
// amax <= 127 * 2^e, and each value the whole number rint(x / 2^e) in
// [-127, 127].  The power of two makes both directions exact but for that one
// rounding: dividing by it is exact in fp32, code * 2^e has at most 7
// significant bits and so is exact in bf16 too, and packing what was unpacked
// gives the same codes.  Against a scale of amax / 127 the rounding step is up
// to twice as wide (1.5 times on average).  The error of a value is at most
// half a step, 2^(e-1) <= amax / 127.
//
// (Values that would round to 2^128, in a block of power 2^122, stop at 63 * 2^122.)
//
// Stored: e + 127 in a byte (1 .. 249; a block of zeros has 1).  A block that
// holds an infinity or a NaN is stored as 255 and reads back as NaN
// throughout, so that a fault in the activations stays visible.
//
// The floor of both directions is HBM traffic (3 bytes a value in bf16).  For rows of
// whole blocks unpacking is near it (16K x 16 rows of 128, bf16: 17 us of 15.4;
// fp32 29 us of 25.6); packing is bound by its instructions (23 us, fp32 37 us: 0.74
// issues a cycle with DRAM at 40 %).  Rows that are not whole blocks take more and
// narrower accesses, single values where their length is odd (17 to 55 % of HBM).
// A block belongs to a group of lanes, the fewest that hold it at LV values a lane (8
// bf16 or 4 fp32 values: 16 bytes), so that short rows fill their warps too; a
// thread has its kPackPasses blocks' values in flight together.  Rows whose
// length is a multiple of 128 are blocks one after the other and need no row
// arithmetic.
#pragma once

#include "common.cuh"

#include <type_traits>

namespace gdn2 {

constexpr int kPackCols = 128;     // values that share a power of two
constexpr int kPackThreads = 256;
constexpr int kPackPasses = 3;     // blocks per group of lanes, in flight together
constexpr int kPackNonFinite = 255;

// e + 127 of a block from the bits of its largest absolute value (as an
// unsigned number; it orders like the value, infinities and NaN above all).
// With amax = 1.M * 2^(E-127): amax <= 127 * 2^e, 127 = 1.984375 * 2^6, is
// e >= E - 127 - 6, or one more if 1.M > 1.984375; adding 0x1FFFF carries into
// the exponent exactly in that case.  Powers below 2^-126 are not used, so
// that 2^e and 2^-e are both normal numbers.
__device__ __forceinline__ int pack_exponent(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return kPackNonFinite;
  return max(1, (int)((amax_bits + 0x1FFFFu) >> 23) - 6);
}
constexpr int kPackTop = 249;   // the power 2^122, that of fp32's largest values
// 2^-e, and 2^e (NaN for a block that was not finite), from e + 127
__device__ __forceinline__ float pack_inverse(int e127) { return __uint_as_float((uint32_t)(254 - e127) << 23); }
__device__ __forceinline__ float pack_power(int e127) {
  return __uint_as_float(e127 >= kPackNonFinite ? 0x7FC00000u : (uint32_t)e127 << 23);
}

// The code of x in its low byte: adding 1.5 * 2^23 rounds x / 2^e to the nearest
// whole number (ties to even) and leaves it in the mantissa's low bits.
__device__ __forceinline__ uint32_t pack_code(float x, float inv) {
  return __float_as_uint(fmaf(x, inv, 12582912.f));
}
// Where 64 * 2^122 would read back as infinity, codes stop at 63; a block that
// is not finite has none.
__device__ __forceinline__ uint32_t pack_code_rare(float x, float inv, int e127) {
  return e127 == kPackTop ? (uint32_t)max(-63, min(63, __float2int_rn(x * inv))) : 0u;
}
// Four low bytes in one word.
__device__ __forceinline__ uint32_t four_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// The values of the codes in bytes i and i + 1 (i = 0 or 2) of a word: a code
// becomes fp32 by its place in the mantissa of 2^23 (one byte permute, and
// 8388736 = 2^23 + 128 off again, exact), cheaper than a conversion instruction.
template <int I>
__device__ __forceinline__ float2 code_values(uint32_t word, float power) {
  const uint32_t u = word ^ 0x80808080u;
  const float2 f = make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540 + I)),
                               __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7541 + I)));
  return __fmul2_rn(__fadd2_rn(f, make_float2(-8388736.f, -8388736.f)), make_float2(power, power));
}

// The larger of each half of two words of bf16 pairs, NaN above all.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

struct PackArgs {
  const void* x;        // [rows, cols] (pack)
  void* y;              // [rows, cols] (unpack)
  int8_t* codes;        // [rows, cols]
  uint8_t* exps;        // [rows, blocks]
  long long total;      // rows * blocks
  int cols, blocks;     // blocks per row
  int group;            // lanes per block: a power of two, 1 .. 32
  int step_rows, step_blocks;   // kPackThreads / group blocks on: whole rows, and blocks
};

// Where the thread's blocks begin, their lengths (0: there is none), their numbers:
// one division for the first, the others a fixed step on.
struct PackBlock {
  size_t base;
  int len;
  long long n;
};
__device__ __forceinline__ void pack_blocks(const PackArgs& a, PackBlock (&b)[kPackPasses]) {
  const int groups = kPackThreads / a.group;
  long long n = (long long)blockIdx.x * kPackPasses * groups + threadIdx.x / a.group;
  if (a.blocks == 1) {
    const size_t first = (size_t)n * a.cols;
#pragma unroll
    for (int u = 0; u < kPackPasses; ++u) {
      b[u].n = n + u * groups;
      b[u].len = b[u].n < a.total ? a.cols : 0;
      b[u].base = b[u].len ? first + (size_t)(u * groups * a.cols) : 0;
    }
    return;
  }
  long long row = a.total <= 0xffffffffll ? (long long)((uint32_t)n / (uint32_t)a.blocks) : n / a.blocks;
  int cb = (int)(n - row * a.blocks);
#pragma unroll
  for (int u = 0; u < kPackPasses; ++u) {
    const bool is = n < a.total;
    b[u].n = n;
    b[u].len = is ? min(kPackCols, a.cols - cb * kPackCols) : 0;
    b[u].base = is ? (size_t)row * a.cols + (size_t)cb * kPackCols : 0;
    n += groups;
    row += a.step_rows;
    cb += a.step_blocks;
    if (cb >= a.blocks) {
      cb -= a.blocks;
      ++row;
    }
  }
}

// A lane's LV values of a block.  VEC: values LV l .. LV l + LV - 1 by one
// access (rows a multiple of LV long: such a run never straddles the row's end
// and is aligned); else values l, l + group, ... (l: the lane within its group).
template <typename T, int LV>
union PackVec {
  typename std::conditional<sizeof(T) * LV == 16, uint4, typename std::conditional<sizeof(T) * LV == 8, uint2, uint32_t>::type>::type v;
  T e[LV];
};

template <typename IO, int LV, bool VEC>
__global__ void __launch_bounds__(kPackThreads) act_pack_kernel(const PackArgs a) {
  const int l = threadIdx.x & (a.group - 1);
  PackVec<IO, LV> w[kPackPasses];
  PackBlock b[kPackPasses];
  pack_blocks(a, b);
#pragma unroll
  for (int u = 0; u < kPackPasses; ++u) {
    const IO* p = static_cast<const IO*>(a.x) + b[u].base;
    w[u].v = decltype(w[u].v){};
    if (VEC) {
      if (LV * l < b[u].len) w[u].v = reinterpret_cast<const decltype(w[u].v)*>(p)[l];
    } else {
#pragma unroll
      for (int j = 0; j < LV; ++j)
        if (l + a.group * j < b[u].len) w[u].e[j] = p[l + a.group * j];
    }
  }
  // the largest absolute value's bits: bf16 in pairs, upper and lower half
  uint32_t m[kPackPasses];
#pragma unroll
  for (int u = 0; u < kPackPasses; ++u) {
    const uint32_t* words = reinterpret_cast<const uint32_t*>(&w[u].v);
    m[u] = 0;
#pragma unroll
    for (int j = 0; j < LV * (int)sizeof(IO) / 4; ++j)
      m[u] = sizeof(IO) == 2 ? max_bf16x2(m[u], words[j] & 0x7FFF7FFFu) : max(m[u], words[j] & 0x7FFFFFFFu);
  }
  for (int o = a.group / 2; o > 0; o /= 2)
#pragma unroll
    for (int u = 0; u < kPackPasses; ++u) {
      const uint32_t k = __shfl_xor_sync(0xffffffffu, m[u], o);
      m[u] = sizeof(IO) == 2 ? max_bf16x2(m[u], k) : max(m[u], k);
    }
#pragma unroll
  for (int u = 0; u < kPackPasses; ++u) {
    if (b[u].len == 0) continue;
    if (sizeof(IO) == 2) m[u] = max(m[u] & 0xFFFF0000u, m[u] << 16);
    const int e = pack_exponent(m[u]);
    const float inv = pack_inverse(e);
    int8_t* q = a.codes + b[u].base;
    uint32_t c[LV];
    if (e < kPackTop) {
#pragma unroll
      for (int j = 0; j < LV; ++j) c[j] = pack_code(to_f32(w[u].e[j]), inv);
    } else {
#pragma unroll
      for (int j = 0; j < LV; ++j) c[j] = pack_code_rare(to_f32(w[u].e[j]), inv, e);
    }
    if (VEC) {
      PackVec<int8_t, LV> r;
      uint32_t* words = reinterpret_cast<uint32_t*>(&r.v);
#pragma unroll
      for (int j = 0; j < LV / 4; ++j) words[j] = four_bytes(c[4 * j], c[4 * j + 1], c[4 * j + 2], c[4 * j + 3]);
      if (LV * l < b[u].len) reinterpret_cast<decltype(r.v)*>(q)[l] = r.v;
    } else {
#pragma unroll
      for (int j = 0; j < LV; ++j)
        if (l + a.group * j < b[u].len) q[l + a.group * j] = (int8_t)(c[j] & 0xFFu);
    }
    if (l == 0) a.exps[b[u].n] = (uint8_t)e;
  }
}

template <typename IO, int LV, bool VEC>
__global__ void __launch_bounds__(kPackThreads) act_unpack_kernel(const PackArgs a) {
  const int l = threadIdx.x & (a.group - 1);
  PackVec<int8_t, LV> c[kPackPasses];
  float p2[kPackPasses];
  PackBlock b[kPackPasses];
  pack_blocks(a, b);
#pragma unroll
  for (int u = 0; u < kPackPasses; ++u) {
    p2[u] = b[u].len > 0 ? pack_power(a.exps[b[u].n]) : 0.f;
    const int8_t* p = a.codes + b[u].base;
    if (VEC) {
      c[u].v = decltype(c[u].v){};
      if (LV * l < b[u].len) c[u].v = reinterpret_cast<const decltype(c[u].v)*>(p)[l];
    } else {
#pragma unroll
      for (int j = 0; j < LV; ++j) c[u].e[j] = l + a.group * j < b[u].len ? p[l + a.group * j] : (int8_t)0;
    }
  }
#pragma unroll
  for (int u = 0; u < kPackPasses; ++u) {
    IO* q = static_cast<IO*>(a.y) + b[u].base;
    if (VEC) {
      PackVec<IO, LV> w;
      const uint32_t* words = reinterpret_cast<const uint32_t*>(&c[u].v);
#pragma unroll
      for (int j = 0; j < LV; j += 4) {
        const float2 lo = code_values<0>(words[j / 4], p2[u]), hi = code_values<2>(words[j / 4], p2[u]);
        w.e[j] = from_f32<IO>(lo.x);
        w.e[j + 1] = from_f32<IO>(lo.y);
        w.e[j + 2] = from_f32<IO>(hi.x);
        w.e[j + 3] = from_f32<IO>(hi.y);
      }
      if (LV * l < b[u].len) reinterpret_cast<decltype(w.v)*>(q)[l] = w.v;
    } else {
#pragma unroll
      for (int j = 0; j < LV; ++j)
        if (l + a.group * j < b[u].len) q[l + a.group * j] = from_f32<IO>((float)c[u].e[j] * p2[u]);
    }
  }
}

}  // namespace gdn2
