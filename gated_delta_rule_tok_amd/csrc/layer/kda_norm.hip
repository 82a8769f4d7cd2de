// kda_norm.hip -- the residual's addition and the RMS norm, with a bf16 or an
// e4m3 output:
//   s = x + r,  r <- bf16(s),  y = s w / sqrt(mean(s^2) + eps)
//   bf16(y), or e4m3(y / c) with c = max|y| / 448 over a row or 128 channels.
//
// Bound by the bytes (7 to 8 per element with a residual): one workgroup per
// row keeps the whole row in registers between the sum of squares and the
// output, so every byte moves once.  A thread holds VPT pieces of 8 adjacent
// channels; 16 adjacent threads hold a group of 128.
//
// The quotient y / c = 448 (s w) / max|s w| does not depend on the row's norm,
// so it is formed from t = s w alone, as n = 448 t, q = n / m by a reciprocal
// and one step of refinement.  t and n are exact without a residual (two 8-bit
// factors and 7 * 2^6), and a quotient half way between two e4m3 values is then
// found as such and goes to the even one.
//
// Rows of any finite size are taken: see where var is formed.
#include "kda_layer_internal.h"
#include "kda_mfma.h"

namespace kda {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr float kFp8Max = 448.f;
constexpr int kGridX = 1 << 20;  // rows per grid row (a grid dimension holds fewer than 2^32 threads)

__device__ __forceinline__ uint32_t round2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// 16 or 8 bytes at any address (the memory pipe takes them unaligned: rows of
// odd length cost 2-byte accesses otherwise)
struct __attribute__((packed, aligned(1))) Bytes16 { uint32_t v[4]; };
struct __attribute__((packed, aligned(1))) Bytes8 { uint32_t v[2]; };

// 8 adjacent elements from p, of which n exist (the others are zeros)
template <bool VEC>
__device__ __forceinline__ void load8f(const uint16_t* p, int n, float* f) {
  if (VEC) {
    unpack8(n > 0 ? *reinterpret_cast<const uint4*>(p) : uint4{0, 0, 0, 0}, f);
  } else if (n >= 8) {
    const Bytes16 b = *reinterpret_cast<const Bytes16*>(p);
    unpack8(uint4{b.v[0], b.v[1], b.v[2], b.v[3]}, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < n ? bf16_to_f32(p[i]) : 0.f;
  }
}

template <bool VEC>
__device__ __forceinline__ void store8(uint16_t* p, int n, const float* f) {
  const uint32_t v[4] = {round2(f[0], f[1]), round2(f[2], f[3]), round2(f[4], f[5]), round2(f[6], f[7])};
  if (VEC) {
    if (n > 0) *reinterpret_cast<uint4*>(p) = uint4{v[0], v[1], v[2], v[3]};
  } else if (n >= 8) {
    *reinterpret_cast<Bytes16*>(p) = Bytes16{{v[0], v[1], v[2], v[3]}};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = uint16_t(v[i / 2] >> (16 * (i & 1)));
  }
}

// Sum (or maximum) over the workgroup, the same in every thread; the waves'
// parts are joined in wave order.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float* red) {
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    const float w = __shfl_xor(v, o);
    v = MAX ? fmaxf(v, w) : v + w;
  }
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float r = red[0];
  for (int i = 1; i < waves; ++i) r = MAX ? fmaxf(r, red[i]) : r + red[i];
  return r;
}

template <int VPT, bool VEC, bool RES, bool FP8>
__global__ __launch_bounds__(1024) void norm_kernel(NormParams np) {
  __shared__ float red[3][16];
  const int t = threadIdx.x;
  const int64_t row = int64_t(blockIdx.y) * kGridX + blockIdx.x;
  if (row >= np.rows) return;
  const uint16_t* x = np.x + row * np.x_row;
  uint16_t* r = RES ? np.res + row * np.r_row : nullptr;
  float s[VPT][8], w[VPT][8];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = 8 * (t + i * int(blockDim.x));
    load8f<VEC>(x + c, np.dim - c, s[i]);
    if (RES) load8f<VEC>(r + c, np.dim - c, w[i]);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = 8 * (t + i * int(blockDim.x));
    if (RES) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] += w[i][j];
      store8<VEC>(r + c, np.dim - c, s[i]);
    }
    load8f<VEC>(np.w + c, np.dim - c, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(s[i][j], s[i][j], sum);
  }
  sum = block_reduce<false>(sum, red[0]);
  // Squares that fp32 may not hold (the same for the whole row): the row times a
  // power of two, which leaves y as it is.  2^-80 brings its largest element, 2^50
  // at least, to 2^-30 .. 2^48; 2^70 brings the least bf16 to 2^-63 and, where eps
  // counts, keeps eps times its square below 2^60.
  float var = sum / float(np.dim) + np.eps;
  if (var > 0x1p100f || var < 0x1p-80f) {
    const float p = var > 1.f ? 0x1p-80f : 0x1p70f;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[i][j] *= p;
        sum = fmaf(s[i][j], s[i][j], sum);
      }
    var = block_reduce<false>(sum, red[1]) / float(np.dim) + np.eps * p * p;
  }
  const float rstd = var == 0.f ? 0.f : 1.f / sqrtf(var);  // a row of zeros without eps: zeros
  if (!FP8) {
    uint16_t* o = static_cast<uint16_t*>(np.out) + row * np.o_row;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = 8 * (t + i * int(blockDim.x));
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] = s[i][j] * rstd * w[i][j];
      store8<VEC>(o + c, np.dim - c, s[i]);
    }
    return;
  }
  uint8_t* o = static_cast<uint8_t*>(np.out) + row * np.o_row;
  float m[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    m[i] = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s[i][j] *= w[i][j];
      m[i] = fmaxf(m[i], fabsf(s[i][j]));
    }
  }
  if (np.group) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
      for (int d = 8; d; d >>= 1) m[i] = fmaxf(m[i], __shfl_xor(m[i], d));
    }
  } else {
    float a = m[0];
#pragma unroll
    for (int i = 1; i < VPT; ++i) a = fmaxf(a, m[i]);
    a = block_reduce<true>(a, red[2]);
#pragma unroll
    for (int i = 0; i < VPT; ++i) m[i] = a;
  }
  const int groups = np.group ? (np.dim + 127) / 128 : 1;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = 8 * (t + i * int(blockDim.x)), n = np.dim - c;
    if (n <= 0) continue;
    if (np.group ? (c & 127) == 0 : c == 0)
      np.scale[row * groups + (np.group ? c >> 7 : 0)] = m[i] * rstd / kFp8Max;
    // a power of two keeps 448 t and 1 / m in range; a group of zeros is divided by one
    const float p2 = m[i] < 0x1p-60f ? 0x1p60f : m[i] > 0x1p60f ? 0x1p-60f : 1.f;
    const float d = m[i] > 0.f ? m[i] * p2 : 1.f, inv = 1.f / d;
    const float k = rstd == 0.f ? 0.f : kFp8Max * p2;  // (beside an infinity: zeros, as in bf16)
    float z[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float nn = s[i][j] * k, q = nn * inv;
      z[j] = fmaf(fmaf(-q, d, nn), inv, q);
    }
    uint2 b;
    b.x = __builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], 0, false);
    b.x = __builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], b.x, true);
    b.y = __builtin_amdgcn_cvt_pk_fp8_f32(z[4], z[5], 0, false);
    b.y = __builtin_amdgcn_cvt_pk_fp8_f32(z[6], z[7], b.y, true);
    if (VEC) {
      *reinterpret_cast<uint2*>(o + c) = b;
    } else if (n >= 8) {
      *reinterpret_cast<Bytes8*>(o + c) = Bytes8{{b.x, b.y}};
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) o[c + j] = uint8_t((j < 4 ? b.x : b.y) >> (8 * (j & 3)));
    }
  }
}

template <int VPT, bool VEC>
hipError_t launch(const NormParams& p, hipStream_t st) {
  NormParams arg = p;
  void* args[] = {&arg};
  const void* f;
  if (p.res)
    f = p.fp8 ? reinterpret_cast<const void*>(&norm_kernel<VPT, VEC, true, true>)
              : reinterpret_cast<const void*>(&norm_kernel<VPT, VEC, true, false>);
  else
    f = p.fp8 ? reinterpret_cast<const void*>(&norm_kernel<VPT, VEC, false, true>)
              : reinterpret_cast<const void*>(&norm_kernel<VPT, VEC, false, false>);
  const dim3 grid(uint32_t(p.rows < kGridX ? p.rows : kGridX), uint32_t((p.rows + kGridX - 1) / kGridX));
  const int pieces = (p.dim + 7) / 8, threads = ((pieces + VPT - 1) / VPT + 63) / 64 * 64;
  return hipLaunchKernel(f, grid, dim3(threads), args, 0, st);
}

// Pieces of a row per thread: one for few rows (latency), two for many (a
// reduction over half the waves): 1 x 7168 3.0 us with one, 3.4 with four; 4096
// x 2048 12.1 / 11.4 us with one / two, 16384 x 7168 to e4m3 154 / 150 us (5.5
// TB/s; a copy reaches 5.1), 16384 x 5120 118 / 120.
template <bool VEC>
hipError_t pick(const NormParams& p, hipStream_t st) {
  const int pieces = (p.dim + 7) / 8;
  if (pieces <= 1024 && p.rows < 256) return launch<1, VEC>(p, st);
  if (pieces <= 2048) return launch<2, VEC>(p, st);
  return launch<4, VEC>(p, st);
}

}  // namespace

hipError_t launch_norm(const NormParams& p, hipStream_t stream) {
  // whole pieces at aligned addresses, where every row of every operand has them
  const bool many = p.rows > 1;
  const auto at = [](const void* q) { return reinterpret_cast<uintptr_t>(q); };
  const bool vec = p.dim % 8 == 0 && at(p.x) % 16 == 0 && at(p.res) % 16 == 0 && at(p.w) % 16 == 0 &&
                   at(p.out) % (p.fp8 ? 8 : 16) == 0 && !(many && p.x_row % 8) &&
                   !(many && p.res && p.r_row % 8) && !(many && p.o_row % 8);
  return vec ? pick<true>(p, stream) : pick<false>(p, stream);
}

}  // namespace kda
