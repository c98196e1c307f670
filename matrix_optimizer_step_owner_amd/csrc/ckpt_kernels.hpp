// Activation checkpoints in 8 bits (gfx950).
//
// Each row of an activation is cut into blocks of kCkptBlock columns.  A block
// is held as whole numbers q in [-127, 127] and one power of two 2^e, the
// smallest e >= -126 with max |x| <= 127 * 2^e:
//   q = x / 2^e rounded to the nearest, ties to even;  x is held as q * 2^e.
// The error is at most 2^(e-1), half a step: under max|x| / 127 where e > -126,
// as max|x| > 127 * 2^(e-1) there.  e stops at
// 121, above which q * 2^e could pass the largest float, and q at 127: only
// values beyond 127.5 * 2^121 are then off by more (by under one step).  A power of
// two makes the division exact and q * 2^e a bf16 number (seven bits of
// magnitude), so the checkpoint restores without a second rounding and the
// weight gradient can multiply it in bf16 as it stands.  e is stored as the
// byte e + 127; 255 marks a block with an infinity or a NaN, which restores as
// NaN throughout.
//
// Bound by HBM: x is read once and one byte and 1/128 written per value.
// Sixteen lanes take one block, eight values each, and find its maximum with
// four lane exchanges; a thread has kCkptUnits blocks' loads in flight (two:
// four were 3% slower, one 3-9% on bf16).  Activations are read, and restored,
// once: both pass the L2s by (restoring 8192 x 27648 bf16: 5.9 -> 6.5 TB/s;
// streaming the codes gained nothing).  8192 x 27648 bf16: quantize 4.5 TB/s,
// restore 6.5.
#pragma once

#include "common.hpp"
#include "grouped_kernels.hpp"

namespace mfsdp {

constexpr int kCkptUnits = 2;   // blocks per 16-lane group

struct CkptArgs {
  void* x;             // rows x k, row stride ld (read by quantize, written by restore)
  int8_t* codes;       // rows x k, contiguous
  uint8_t* scales;     // rows x nb
  int64_t ld;
  uint32_t units;      // rows * nb, under 2^29 in one launch
  int32_t k, nb;
  int32_t vec;         // rows of x start on 16 bytes and k is a multiple of 8
};

// One block of this 16-lane group: its row, first column and how many columns
// it has.
struct CkptUnit {
  int64_t row;
  int c0, left;
  __device__ __forceinline__ CkptUnit(const CkptArgs& a, uint32_t u) {
    row = u / static_cast<uint32_t>(a.nb);
    c0 = static_cast<int>(u - static_cast<uint32_t>(row) * a.nb) * kCkptBlock;
    left = min(kCkptBlock, a.k - c0);
  }
};

// First column of half h (four values) of a lane's eight: eight (bf16) or twice
// four (fp32) consecutive columns, so that 16 lanes' 16-byte accesses are
// contiguous.
template <class E>
__device__ __forceinline__ int ckpt_col(int l16, int h) {
  return E::kVec == 8 ? l16 * 8 + h * 4 : h * 64 + l16 * 4;
}

__device__ __forceinline__ uint32_t ckpt_unit0() {
  return blockIdx.x * (16 * kCkptUnits) + (threadIdx.x >> 4);
}

template <class E>
__global__ __launch_bounds__(256) void ckpt_quantize_kernel(CkptArgs a) {
  using S = typename E::storage_t;
  const int l16 = threadIdx.x & 15;
  const uint32_t unit0 = ckpt_unit0();
  const bool vec = a.vec != 0;
  float v[kCkptUnits][8];
#pragma unroll
  for (int i = 0; i < kCkptUnits; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (unit0 + 16 * i >= a.units) continue;
    const CkptUnit u(a, unit0 + 16 * i);
    const S* src = static_cast<const S*>(a.x) + u.row * a.ld + u.c0;
    if (!vec) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j * 16 + l16 < u.left) v[i][j] = E::to_f32(src[j * 16 + l16]);
    } else if constexpr (E::kVec == 8) {
      if (l16 * 8 < u.left) Vec16<E>::unpack(gld_stream(src + l16 * 8), v[i]);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = ckpt_col<E>(l16, h);
        float t[4] = {0.f, 0.f, 0.f, 0.f};
        if (c < u.left) Vec16<E>::unpack(gld_stream(src + c), t);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][4 * h + j] = t[j];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kCkptUnits; ++i) {
    if (unit0 + 16 * i >= a.units) continue;   // whole 16-lane groups leave together
    // largest magnitude by its bits: infinities and NaN come out on top
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[i][j]) & 0x7fffffffu);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1)
      top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d, 16)));
    // max = m 2^p, 1 <= m < 2: e = p - 6 while m <= 127/64, else p - 5; the
    // biased exponent is clamped to [1, 248] (e = -126 .. 121)
    int be = static_cast<int>(top >> 23) - 6 + ((top & 0x7fffffu) > 0x7e0000u ? 1 : 0);
    be = min(max(be, 1), 248);
    const bool bad = top >= 0x7f800000u;
    const float inv = __uint_as_float(static_cast<uint32_t>(254 - be) << 23);   // 2^-e
    const CkptUnit u(a, unit0 + 16 * i);
    int8_t* dst = a.codes + u.row * a.k + u.c0;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int q = bad ? 0 : static_cast<int>(fminf(fmaxf(rintf(v[i][j] * inv), -127.f), 127.f));
      w[j >> 2] |= static_cast<uint32_t>(q & 0xff) << (8 * (j & 3));
    }
    if (!vec) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j * 16 + l16 < u.left) dst[j * 16 + l16] = static_cast<int8_t>(w[j >> 2] >> (8 * (j & 3)));
    } else if constexpr (E::kVec == 8) {
      if (l16 * 8 < u.left) *reinterpret_cast<uint2*>(dst + l16 * 8) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = ckpt_col<E>(l16, h);
        if (c < u.left) *reinterpret_cast<uint32_t*>(dst + c) = w[h];
      }
    }
    if (l16 == 0) a.scales[unit0 + 16 * i] = static_cast<uint8_t>(bad ? 255 : be);
  }
}

template <class E>
__global__ __launch_bounds__(256) void ckpt_restore_kernel(CkptArgs a) {
  using S = typename E::storage_t;
  const int l16 = threadIdx.x & 15;
  const uint32_t unit0 = ckpt_unit0();
  const bool vec = a.vec != 0;
  uint32_t w[kCkptUnits][2];
  uint32_t b[kCkptUnits];
#pragma unroll
  for (int i = 0; i < kCkptUnits; ++i) {
    w[i][0] = w[i][1] = b[i] = 0;
    if (unit0 + 16 * i >= a.units) continue;
    const CkptUnit u(a, unit0 + 16 * i);
    const int8_t* src = a.codes + u.row * a.k + u.c0;
    b[i] = a.scales[unit0 + 16 * i];
    if (!vec) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j * 16 + l16 < u.left)
          w[i][j >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(src[j * 16 + l16])) << (8 * (j & 3));
    } else if constexpr (E::kVec == 8) {
      if (l16 * 8 < u.left) {
        const uint2 t = *reinterpret_cast<const uint2*>(src + l16 * 8);
        w[i][0] = t.x;
        w[i][1] = t.y;
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = ckpt_col<E>(l16, h);
        if (c < u.left) w[i][h] = *reinterpret_cast<const uint32_t*>(src + c);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kCkptUnits; ++i) {
    if (unit0 + 16 * i >= a.units) continue;
    const CkptUnit u(a, unit0 + 16 * i);
    S* dst = static_cast<S*>(a.x) + u.row * a.ld + u.c0;
    const float s = ckpt_scale(b[i]);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = static_cast<float>(static_cast<int8_t>(w[i][j >> 2] >> (8 * (j & 3)))) * s;
    if (!vec) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j * 16 + l16 < u.left) dst[j * 16 + l16] = E::from_f32(v[j]);
    } else if constexpr (E::kVec == 8) {
      if (l16 * 8 < u.left) gst_stream(dst + l16 * 8, Vec16<E>::pack(v));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = ckpt_col<E>(l16, h);
        const float t[4] = {v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
        if (c < u.left) gst_stream(dst + c, Vec16<E>::pack(t));
      }
    }
  }
}

}  // namespace mfsdp
