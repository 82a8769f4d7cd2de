// kda_gdr_serial.hip -- the delta rule with one decay per head, token after
// token: the decode step on a pool of states, and prefills of a few tokens per
// sequence.
//
// One workgroup holds V columns of one state in registers and, per token, does
// in one pass over them
//   x = k~^T S,  y = q~^T S,  u = beta (v - a x),
//   o = scale (a y + (q~ . k~) u),  S <- a S + k~ u^T
// (o from the old state, so that k and q share one reduction and one barrier).
// A decode step is bound by the state's bytes, read and written once: every
// load of the state is issued before anything else, 16 bytes per lane, 32 KB in
// flight per workgroup.  256 sequences x 16 heads, fp32: 111 us, 4.8 TB/s (a
// copy reaches 5.1).
#include "kda_gdr.h"

namespace kda {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));

// two numbers rounded to bf16 (one instruction; NaN stays NaN)
__device__ __forceinline__ uint32_t round2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

template <bool BF16, int V>
__global__ __launch_bounds__(256) void serial_kernel(GdrParams p) {
  constexpr int E = BF16 ? 8 : 4;   // columns per thread (16 bytes)
  constexpr int TPR = V / E;        // threads across a row
  constexpr int R = kD * TPR / 256; // rows (key channels) per thread
  __shared__ float kq[4][2][kD];    // a copy per wave: no barrier before its use
  __shared__ float red[2][4][2][V];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int S = kD / V;
  const int item = blockIdx.x / S, col = (blockIdx.x % S) * V + (tid % TPR) * E;
  const int n = item / p.Hv, h = item % p.Hv, hk = h / (p.Hv / p.Hk);
  const int row0 = tid / TPR * R;
  int t0, t1;
  int64_t slot = n;
  if (p.idx) {
    slot = p.idx[n];
    if (slot < 0 || slot >= p.slots) return;
    t0 = n;
    t1 = n + 1;
  } else {
    gdr_range(p, n, t0, t1);
  }
  const size_t base = (size_t(slot) * p.Hv + h) * (kD * kD) + size_t(row0) * kD + col;
  float s[R][E];
  if (p.s0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (BF16) {
        unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.s0) + base + r * kD), s[r]);
      } else {
        const f32x4 f = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p.s0) + base + r * kD);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[r][e] = f[e];
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < E; ++e) s[r][e] = 0.f;
  }
  const float A_log = p.A_log[h], dt_bias = p.dt_bias[h];
  for (int t = t0; t < t1; ++t) {
    const uint32_t kw = *reinterpret_cast<const uint32_t*>(p.k + t * p.k_t + hk * p.k_h + 2 * lane);
    const uint32_t qw = *reinterpret_cast<const uint32_t*>(p.q + t * p.q_t + hk * p.q_h + 2 * lane);
    const uint16_t* vp = p.v + t * p.v_t + h * p.v_h + col;
    float v[E];
    if (BF16) {
      unpack8(*reinterpret_cast<const uint4*>(vp), v);
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(vp);
      v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
    }
    const float decay = expf(gdr_log_decay(bf16_to_f32(p.a[t * p.a_t + h * p.a_h]), A_log, dt_bias));
    const float beta = gdr_sigmoid(bf16_to_f32(p.beta[t * p.b_t + h * p.b_h]));
    float k0 = bf16_lo(kw), k1 = bf16_hi(kw), q0 = bf16_lo(qw), q1 = bf16_hi(qw);
    float kk, qq, qk;
    const auto sums = [&] {
      kk = k0 * k0 + k1 * k1, qq = q0 * q0 + q1 * q1, qk = q0 * k0 + q1 * k1;
#pragma unroll
      for (int o = 32; o; o >>= 1) {
        kk += __shfl_xor(kk, o);
        qq += __shfl_xor(qq, o);
        qk += __shfl_xor(qk, o);
      }
    };
    sums();
    float ke = kNormEps, qe = kNormEps;
    if (fmaxf(kk, qq) > 0x1p100f) {  // (the same in every lane) squares that fp32 may not hold
      if (kk > 0x1p100f) k0 *= 0x1p-70f, k1 *= 0x1p-70f, ke = 0.f;  // 1e-6 2^-140 is nothing beside them
      if (qq > 0x1p100f) q0 *= 0x1p-70f, q1 *= 0x1p-70f, qe = 0.f;
      sums();
    }
    const float rk = 1.f / sqrtf(kk + ke), rq = 1.f / sqrtf(qq + qe);
    qk *= rk * rq;
    *reinterpret_cast<float2*>(&kq[wave][0][2 * lane]) = float2{k0 * rk, k1 * rk};
    *reinterpret_cast<float2*>(&kq[wave][1][2 * lane]) = float2{q0 * rq, q1 * rq};
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    float x[E] = {}, y[E] = {};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float kr = kq[wave][0][row0 + r], qr = kq[wave][1][row0 + r];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x[e] = fmaf(kr, s[r][e], x[e]);
        y[e] = fmaf(qr, s[r][e], y[e]);
      }
    }
#pragma unroll
    for (int o = TPR; o < 64; o <<= 1)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x[e] += __shfl_xor(x[e], o);
        y[e] += __shfl_xor(y[e], o);
      }
    const int par = t & 1;  // two buffers: a wave ahead writes the other one
    if (lane < TPR) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        red[par][wave][0][lane * E + e] = x[e];
        red[par][wave][1][lane * E + e] = y[e];
      }
    }
    __syncthreads();
    float u[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = (tid % TPR) * E + e;
      const float xs = (red[par][0][0][c] + red[par][1][0][c]) + (red[par][2][0][c] + red[par][3][0][c]);
      const float ys = (red[par][0][1][c] + red[par][1][1][c]) + (red[par][2][1][c] + red[par][3][1][c]);
      u[e] = beta * (v[e] - decay * xs);
      y[e] = p.scale * (decay * ys + qk * u[e]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float kr = kq[wave][0][row0 + r];
#pragma unroll
      for (int e = 0; e < E; ++e) s[r][e] = fmaf(kr, u[e], decay * s[r][e]);
    }
    if (tid < TPR) {
      uint16_t* o = p.out + t * p.o_t + h * p.o_h + col;
      if (BF16)
        *reinterpret_cast<uint4*>(o) = uint4{round2(y[0], y[1]), round2(y[2], y[3]),
                                             round2(y[E - 4], y[E - 3]), round2(y[E - 2], y[E - 1])};
      else
        *reinterpret_cast<uint2*>(o) = uint2{round2(y[0], y[1]), round2(y[2], y[3])};
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (BF16)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.sT) + base + r * kD) =
          uint4{round2(s[r][0], s[r][1]), round2(s[r][2], s[r][3]),
                round2(s[r][E - 4], s[r][E - 3]), round2(s[r][E - 2], s[r][E - 1])};
    else
      *reinterpret_cast<f32x4*>(static_cast<float*>(p.sT) + base + r * kD) =
          f32x4{s[r][0], s[r][1], s[r][2], s[r][3]};
  }
}

}  // namespace

hipError_t launch_gdr_serial(const GdrParams& p, hipStream_t stream) {
  GdrParams arg = p;
  void* args[] = {&arg};
  const int64_t pairs = int64_t(p.N) * p.Hv;
  // Columns per workgroup: few states are spread over more workgroups (1 x 16:
  // 4.9 us with 32 columns, 5.0 with 64, 5.6 with 128; 256 x 16, fp32, 114, 111
  // and 110), a bf16 state of 64 columns is too little for one (128 x 32: 61 us
  // against 58 with 128, 93 with 32).
  const int cols = pairs <= 64 ? 32 : p.state_bf16 && pairs >= 512 ? 128 : 64;
  const void* f = cols == 32   ? (p.state_bf16 ? reinterpret_cast<const void*>(&serial_kernel<true, 32>)
                                               : reinterpret_cast<const void*>(&serial_kernel<false, 32>))
                  : cols == 64 ? (p.state_bf16 ? reinterpret_cast<const void*>(&serial_kernel<true, 64>)
                                               : reinterpret_cast<const void*>(&serial_kernel<false, 64>))
                               : reinterpret_cast<const void*>(&serial_kernel<true, 128>);
  return hipLaunchKernel(f, dim3(uint32_t(pairs * (kD / cols))), dim3(256), args, 0, stream);
}

}  // namespace kda
