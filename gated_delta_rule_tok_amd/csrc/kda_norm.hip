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
// so it is formed from t = s w alone, with a correctly rounded division: t is
// exact without a residual (two 8-bit factors), and then a quotient half way
// between two e4m3 values is a tie in fp32 too and goes to the even one.
#include "kda_layer_internal.h"
#include "kda_mfma.h"

namespace kda {
namespace {

constexpr float kFp8Max = 448.f;
constexpr int kGridX = 1 << 20;  // rows per grid row (a grid dimension holds fewer than 2^32 threads)

// 8 adjacent elements from p, of which n exist (n <= 0: none, zeros)
template <bool VEC>
__device__ __forceinline__ void load8f(const uint16_t* p, int n, float* f) {
  if (VEC) {
    if (n > 0) {
      unpack8(*reinterpret_cast<const uint4*>(p), f);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < n ? bf16_to_f32(p[i]) : 0.f;
  }
}

template <bool VEC>
__device__ __forceinline__ void store8(uint16_t* p, int n, const float* f) {
  if (VEC) {
    if (n > 0)
      *reinterpret_cast<uint4*>(p) =
          uint4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                pack_bf16x2(f[6], f[7])};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = f32_to_bf16(f[i]);
  }
}

// Sum (or maximum) over the workgroup, the same in every thread; the waves'
// parts are joined in wave order.
template <int THREADS, bool MAX>
__device__ __forceinline__ float block_reduce(float v, float* red) {
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    const float w = __shfl_xor(v, o);
    v = MAX ? fmaxf(v, w) : v + w;
  }
  if (THREADS == 64) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float r = red[0];
#pragma unroll
  for (int i = 1; i < THREADS / 64; ++i) r = MAX ? fmaxf(r, red[i]) : r + red[i];
  return r;
}

template <int THREADS, int VPT, bool VEC, bool RES, bool FP8>
__global__ __launch_bounds__(THREADS) void norm_kernel(NormParams np) {
  __shared__ float red[2][16];
  const int t = threadIdx.x;
  const int64_t row = int64_t(blockIdx.y) * kGridX + blockIdx.x;
  if (row >= np.rows) return;
  const uint16_t* x = np.x + row * np.x_row;
  uint16_t* r = RES ? np.res + row * np.r_row : nullptr;
  float s[VPT][8], w[VPT][8];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = 8 * (t + i * THREADS);
    load8f<VEC>(x + c, np.dim - c, s[i]);
    if (RES) {
      float f[8];
      load8f<VEC>(r + c, np.dim - c, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] += f[j];
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) load8f<VEC>(np.w + 8 * (t + i * THREADS), np.dim - 8 * (t + i * THREADS), w[i]);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = 8 * (t + i * THREADS);
    if (RES) store8<VEC>(r + c, np.dim - c, s[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += s[i][j] * s[i][j];
  }
  sum = block_reduce<THREADS, false>(sum, red[0]);
  const float rstd = 1.f / sqrtf(sum / float(np.dim) + np.eps);
  if (!FP8) {
    uint16_t* o = static_cast<uint16_t*>(np.out) + row * np.o_row;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = 8 * (t + i * THREADS);
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
    a = block_reduce<THREADS, true>(a, red[1]);
#pragma unroll
    for (int i = 0; i < VPT; ++i) m[i] = a;
  }
  const int groups = np.group ? (np.dim + 127) / 128 : 1;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = 8 * (t + i * THREADS), n = np.dim - c;
    if (n <= 0) continue;
    const float c8 = m[i] * rstd / kFp8Max;
    if (np.group ? (c & 127) == 0 : c == 0) np.scale[row * groups + (np.group ? c >> 7 : 0)] = c8;
    const float d = m[i] > 0.f ? m[i] : 1.f;
    float z[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = kFp8Max * s[i][j] / d;
    uint2 b;
    b.x = __builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], 0, false);
    b.x = __builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], b.x, true);
    b.y = __builtin_amdgcn_cvt_pk_fp8_f32(z[4], z[5], 0, false);
    b.y = __builtin_amdgcn_cvt_pk_fp8_f32(z[6], z[7], b.y, true);
    if (VEC) {
      *reinterpret_cast<uint2*>(o + c) = b;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) o[c + j] = uint8_t((j < 4 ? b.x : b.y) >> (8 * (j & 3)));
    }
  }
}

template <int THREADS, int VPT, bool VEC>
hipError_t launch(const NormParams& p, hipStream_t st) {
  NormParams arg = p;
  void* args[] = {&arg};
  const void* f;
  if (p.res)
    f = p.fp8 ? reinterpret_cast<const void*>(&norm_kernel<THREADS, VPT, VEC, true, true>)
              : reinterpret_cast<const void*>(&norm_kernel<THREADS, VPT, VEC, true, false>);
  else
    f = p.fp8 ? reinterpret_cast<const void*>(&norm_kernel<THREADS, VPT, VEC, false, true>)
              : reinterpret_cast<const void*>(&norm_kernel<THREADS, VPT, VEC, false, false>);
  const dim3 grid(uint32_t(p.rows < kGridX ? p.rows : kGridX), uint32_t((p.rows + kGridX - 1) / kGridX));
  return hipLaunchKernel(f, grid, dim3(THREADS), args, 0, st);
}

template <bool VEC>
hipError_t pick(const NormParams& p, hipStream_t st) {
  if (p.dim <= 512) return launch<64, 1, VEC>(p, st);
  if (p.dim <= 2048) return launch<256, 1, VEC>(p, st);
  if (p.dim <= 4096) return launch<256, 2, VEC>(p, st);
  if (p.dim <= 8192) return launch<256, 4, VEC>(p, st);
  if (p.dim <= 16384) return launch<1024, 2, VEC>(p, st);
  return launch<1024, 4, VEC>(p, st);
}

}  // namespace

hipError_t launch_norm(const NormParams& p, hipStream_t stream) {
  // 16-byte accesses where every row of every operand starts on 16 bytes (8
  // for an e4m3 output) and ends with a whole piece of 8
  const auto at = [](const void* q) { return reinterpret_cast<uintptr_t>(q); };
  const bool many = p.rows > 1;
  const bool vec = p.dim % 8 == 0 && at(p.x) % 16 == 0 && at(p.res) % 16 == 0 && at(p.w) % 16 == 0 &&
                   at(p.out) % (p.fp8 ? 8 : 16) == 0 && !(many && p.x_row % 8) &&
                   !(many && p.res && p.r_row % 8) && !(many && p.o_row % 8);
  return vec ? pick<true>(p, stream) : pick<false>(p, stream);
}

}  // namespace kda
