// kda_gdr_chunk.hip -- the delta rule with one decay per head, in chunks of 64
// tokens.
//
// With G the running sum of log a in a chunk, S the state entering it and
// k~, q~ the normalised rows:
//   A[t,s] = beta_t e^(G_t-G_s) (k~_t . k~_s), s < t;      T = (I + A)^-1
//   R_t = beta_t (v_t - e^(G_t) k~_t^T S);                 U = T R
//   o_t = scale (e^(G_t) q~_t^T S + sum_{s<=t} e^(G_t-G_s) (q~_t . k~_s) U_s)
//   S'  = e^(G_C) S + sum_s e^(G_C-G_s) k~_s U_s^T
// Every exponent is a sum of decays, so no factor exceeds 1 whatever the gate.
//
// Two launches.  prep_kernel, one workgroup per (chunk, value head), forms
// what does not depend on the state, for all chunks at once: T, the matrix P
// in front of U, the coefficients of every token, and K, Q and K^T as operands.
// scan_kernel walks the chunks of a sequence with the state in registers.
//
// What bounds it.  A chunk depends on the one before, 4 us with an fp32 state;
// 8 x 2048 tokens, 16 heads, fp32 state: prep 71 us, scan 142 us (medians of a
// trace, which vary by 5% from one to the next; 219 MB of inputs and outputs: 43 us at the rate of a copy).  With more
// states than compute units it is the bytes too: 32 ragged prompts, 32 heads,
// bf16 state, prep 228 us and scan 285 us for 1.7 GB, the operands that prep
// writes and scan reads among them.
//
// Precision.  Operands are fp16 (11 bits), sums fp32; prep_kernel spills three
// registers.
//  * A row of K or Q, times a power of two that brings its largest element to
//    [1, 2), is exact in fp16 (bf16 has 8 bits; elements below 2^-14 of the
//    largest are off by 2^-25 of it at most).  Norms, decays and the powers of
//    two are fp32 coefficients on sums or on the other factor.
//  * S, R, U and T have to be cut.  With an fp32 state each is two pieces,
//    x = x0 + x1 (22 bits), and a product of two of them is x0 y0 + x0 y1 +
//    x1 y0; with a bf16 state one piece: 2^-11 per factor beside the 2^-8 of
//    the stored state.  out, which is bf16, takes one piece of S, U and P.
//  * Range: everything in a column of the state (S, V, R, U) scales together,
//    so each column carries a power of two per chunk that brings the larger of
//    its |S| and |v| to [2^7, 2^8).  ||S_t|| grows by at most |v| per token
//    (the map is a contraction), hence |U| <= (1 + sqrt(128) + 64) 2^8 < 2^15:
//    no finite input overflows, and what fp16 loses below 2^-14 is under 2^-28
//    of the column's largest element.  T and P are at most 1.
#include <algorithm>
#include <type_traits>

#include "kda_gdr.h"

namespace kda {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kC = kGdrChunk;
constexpr int kUnits = 6;        // 16 x 32 pieces of a lower triangle of 64: row tile w has w / 2 + 1
constexpr int kKUnits = 16, kHeadUnits = 3 * kKUnits;  // K, Q and K^T of one (chunk, key head)
constexpr int kMaxTri = 3 * kUnits;  // T in two pieces and P, of one (chunk, value head)
constexpr int kCoefs = 5 * kC;   // floats of one (chunk, value head)
// coefficient rows, rk and rq the factors that make a scaled row a unit one:
// beta; beta e^G rk; e^G rq; rk e^(G_C - G); e^(G_C)
enum { kBeta, kKs, kQs, kUs, kEnd };

__device__ __forceinline__ f32x4 mfma32h(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma4(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f16x8 cath(f16x4 lo, f16x4 hi) {
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// First slot of sequence n (see GdrLayout).
__device__ __forceinline__ int64_t first_slot(const GdrParams& p, int n) {
  return int64_t(min(max(p.cu[n], 0), p.T)) / kC + n;
}

// NP fp16 pieces of four numbers
template <int NP>
__device__ __forceinline__ void cut4(f32x4 x, f16x4* o) {
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const f16x2 a = __builtin_convertvector((f32x2{x[0], x[1]}), f16x2);
    const f16x2 b = __builtin_convertvector((f32x2{x[2], x[3]}), f16x2);
    o[i] = f16x4{a[0], a[1], b[0], b[1]};
    if (i + 1 < NP) {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = fmaf(float(o[i][j]), -1.f, x[j]);
    }
  }
}

// unit index of (row tile w, k-step s) in a triangle
__device__ __forceinline__ constexpr int unit_of(int w, int s) { return (w < 2 ? w : 2 * w - 2) + s; }

// ---- prep -------------------------------------------------------------------

constexpr int kPitch = 68;  // floats per row of the LDS matrices (bank spread)

struct PrepLds {
  union {
    f16x8 kf[4][4][64];     // K as operand units [tile][k-step][lane], until A and P are formed
    float A[kC][kPitch];    // A below the diagonal; T in the diagonal blocks; T_ij in block (j, i)
  };
  _Float16 P[kC][72];
  float tmp[4][16][16];
  double G[kC];
  float rk[kC], rq[kC], beta[kC];
};

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// acc += X Y for 16 x 16 fp32 blocks in LDS
__device__ __forceinline__ f32x4 block_mul(const float* X, int xp, const float* Y, int yp, f32x4 acc,
                                           int l16, int g4) {
#pragma unroll
  for (int k = 0; k < 16; k += 4) acc = mfma4(X[l16 * xp + k + g4], Y[(k + g4) * yp + l16], acc);
  return acc;
}

// One row of K or Q, this lane's 32 channels of it, times the power of two that
// brings its largest element to [1, 2) (2^127 where that is no normal number, a
// row of zeros among them), in fp16, and the factor that makes this scaled row a
// unit one.  The sum of squares is the scaled row's: that of a row as it came
// may pass fp32, as may its products with other rows.  The factor is at most 1:
// W = factor U stays in fp16.
__device__ __forceinline__ void scale_row(const bf16x8 (&row)[4], f16x8 (&half)[4], float& unit) {
  float big = 0.f;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    float f[8];
    unpack8(__builtin_bit_cast(uint4, row[s]), f);
#pragma unroll
    for (int j = 0; j < 8; ++j) big = fmaxf(big, fabsf(f[j]));
  }
  big = fmaxf(big, __shfl_xor(big, 16));
  big = fmaxf(big, __shfl_xor(big, 32));
  const uint32_t e = __float_as_uint(big) >> 23;
  const float down = __uint_as_float((254u - min(e, 253u)) << 23);
  float sum = 0.f;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const u32x4 x = __builtin_bit_cast(u32x4, row[s]);
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 f = {bf16_lo(x[i]) * down, bf16_hi(x[i]) * down};
      sum = fmaf(f[0], f[0], sum);
      sum = fmaf(f[1], f[1], sum);
      o[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, f16x2));
    }
    half[s] = __builtin_bit_cast(f16x8, o);
  }
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
  // (beyond 2^40 the sum is nothing beside 1e-6 down^2, which may pass fp32)
  const bool small = down > 0x1p40f;
  unit = 1.f / sqrtf(small ? kNormEps : sum + kNormEps * down * down) * (small ? __uint_as_float(e << 23) : 1.f);
}

template <int NP>
__global__ __launch_bounds__(256, 4) void prep_kernel(GdrParams p, GdrLayout lay) {
  __shared__ PrepLds L;
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g4 = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t slot = blockIdx.x / p.Hv;
  const int h = blockIdx.x % p.Hv, group = p.Hv / p.Hk, hk = h / group;
  // the last sequence whose first slot is not behind this one, 64 candidates at
  // a time; its range comes from the same loads where 64 hold them all
  int lo = 0, t0, t1;
  if (p.N <= 64) {
    gdr_range(p, min(lane, p.N - 1), t0, t1);
    lo = 63 - __builtin_clzll(__ballot(lane < p.N && t0 / kC + lane <= slot) | 1);
    t0 = __builtin_amdgcn_readlane(t0, lo);
    t1 = __builtin_amdgcn_readlane(t1, lo);
  } else {
    for (int span = p.N; span > 1;) {
      const int step = (span + 63) / 64, n = lo + lane * step;
      const bool in = lane * step < span && first_slot(p, min(n, p.N - 1)) <= slot;
      const int k = 63 - __builtin_clzll(__ballot(in) | 1);
      lo += k * step;
      span = min(step, span - k * step);
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    gdr_range(p, lo, t0, t1);
  }
  const int64_t off = (slot - (t0 / kC + lo)) * kC;
  if (off < 0 || off >= t1 - t0) return;  // no chunk has this slot
  t0 += int(off);
  const int len = min(kC, t1 - t0);
  const bool first = h % group == 0;  // writes K, Q and K^T for the key head's value heads
  f16x8* units = reinterpret_cast<f16x8*>(p.ws + lay.head) + (size_t(slot) * p.Hk + hk) * (kHeadUnits * 64) + lane;

  // rows of K and Q as operands: lane l row l % 16 of tile w, channels 32 s + 8
  // (l / 16); rows behind the end repeat the last one, with factors of 0
  // (every load of the workgroup's inputs is issued before the first is used)
  bf16x8 kraw[4], qraw[4];
  const int r0 = 16 * w + l16;
  {
    const int64_t t = t0 + min(r0, len - 1);
    const uint16_t* kp = p.k + t * p.k_t + hk * p.k_h + 8 * g4;
    const uint16_t* qp = p.q + t * p.q_t + hk * p.q_h + 8 * g4;
#pragma unroll
    for (int s = 0; s < 4; ++s) kraw[s] = *reinterpret_cast<const bf16x8*>(kp + 32 * s);
#pragma unroll
    for (int s = 0; s < 4; ++s) qraw[s] = *reinterpret_cast<const bf16x8*>(qp + 32 * s);
  }
  const int64_t tg = t0 + min(lane, len - 1);  // gates: lane = token
  const uint16_t raw_a = p.a[tg * p.a_t + h * p.a_h], raw_beta = p.beta[tg * p.b_t + h * p.b_h];
  const float A_log = p.A_log[h], dt_bias = p.dt_bias[h];
  // G in fp64, so that differences of large sums keep their small terms, and times log2(e)
  if (w == 0) {
    double G = lane < len ? double(gdr_log_decay(bf16_to_f32(raw_a), A_log, dt_bias)) * 1.4426950408889634074 : 0.0;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const double u = __shfl_up(G, o);
      if (lane >= o) G += u;
    }
    L.G[lane] = G;
    L.beta[lane] = lane < len ? gdr_sigmoid(bf16_to_f32(raw_beta)) : 0.f;
  }
  f16x8 kf[4], qf[4];
  {
    float rk, rq;
    scale_row(kraw, kf, rk);
    scale_row(qraw, qf, rq);
#pragma unroll
    for (int s = 0; s < 4; ++s) L.kf[w][s][lane] = kf[s];
    if (first) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        units[(4 * w + s) * 64] = kf[s];
        units[(kKUnits + 4 * w + s) * 64] = qf[s];
      }
    }
    if (g4 == 0) {
      L.rk[r0] = r0 < len ? rk : 0.f;
      L.rq[r0] = r0 < len ? rq : 0.f;
    }
  }
  __syncthreads();
  // K transposed, as operand units [state tile r][k-step z]: lane l the channel
  // of row l % 16 of tile r (see scan_kernel), tokens 32 z + 4 (l / 16) .. + 3
  // and 16 further on
  if (first) {
    const _Float16* kl = reinterpret_cast<const _Float16*>(&L.kf[0][0][0]);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int unit = 4 * w + u, r = unit >> 1;
      const int c = 32 * (r >> 1) + 8 * (l16 >> 2) + 4 * (r & 1) + (l16 & 3);
      f16x8 e;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // token t's channel c: tile t / 16, k-step c / 32, lane t % 16 + 16 (c / 8 % 4)
        const int tile = 2 * (unit & 1) + (j >> 2), row = 4 * g4 + (j & 3);
        e[j] = kl[((tile * 4 + (c >> 5)) * 64 + row + 16 * ((c >> 3) & 3)) * 8 + (c & 7)];
      }
      units[(2 * kKUnits + unit) * 64] = e;
    }
  }
  const double Gend = L.G[kC - 1];  // tokens behind the end add nothing
  if (tid < kC) {
    const float eG = ex2(float(L.G[tid])), b = L.beta[tid], rk = L.rk[tid], rq = L.rq[tid];
    float* co = reinterpret_cast<float*>(p.ws + lay.coef) + (size_t(slot) * p.Hv + h) * kCoefs + tid;
    co[kBeta * kC] = b;
    co[kKs * kC] = b * eG * rk;
    co[kQs * kC] = eG * rq;
    co[kUs * kC] = rk * ex2(float(Gend - L.G[tid]));
    co[kEnd * kC] = ex2(float(Gend));
  }
  // A and P, row tile w (Q first, so that its rows' registers are free for K's products)
  f32x4 kk[4], qk[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    qk[j] = f32x4{};
    if (j <= w) {
#pragma unroll
      for (int s = 0; s < 4; ++s) qk[j] = mfma32h(qf[s], L.kf[j][s][lane], qk[j]);
    }
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    kk[j] = f32x4{};
    if (j <= w) {
#pragma unroll
      for (int s = 0; s < 4; ++s) kk[j] = mfma32h(kf[s], L.kf[j][s][lane], kk[j]);
    }
  }
  __syncthreads();  // kf is read: A takes its place
  // (the rows' factors first, and selects after the products: conditions around
  // LDS reads become branches, and the reads wait for each other)
  double Gt[4];
  float bt[4], qt[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 16 * w + 4 * g4 + i;
    Gt[i] = L.G[t];
    bt[i] = L.beta[t] * L.rk[t];
    qt[i] = L.rq[t];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int s = 16 * j + l16;
    if (j > w) {  // P's unit of 32 columns may reach one tile further than the triangle
      if (j == w + 1 && j % 2 == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) L.P[16 * w + 4 * g4 + i][s] = 0;
      }
      continue;
    }
    const double Gs = L.G[s];
    const float rs = L.rk[s];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * w + 4 * g4 + i;
      const float e = ex2(float(Gt[i] - Gs)) * rs, a = bt[i] * e * kk[j][i], q = qt[i] * e * qk[j][i];
      L.A[t][s] = s < t ? a : 0.f;
      L.P[t][s] = (_Float16)(s <= t ? q : 0.f);
    }
  }
  // T: the diagonal blocks by forward substitution, a column per lane
  {
    wave_sync();
    __builtin_amdgcn_sched_barrier(0);
    float x[16];
    const float* a = &L.A[16 * w][16 * w];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      // (a few rows' elements of A at a time: all 120 in flight spill)
      if (i % 6 == 5) __builtin_amdgcn_sched_barrier(0);
      float v = i == l16 ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < i; ++j) v = fmaf(-a[i * kPitch + j], x[j], v);
      x[i] = v;
    }
    wave_sync();
    if (g4 == 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) L.A[16 * w + i][16 * w + l16] = x[i];
    }
  }
  // blocks below it, by distance from the diagonal: T_ij = -T_ii sum_{j<=k<i} A_ik T_kj
  for (int d = 1; d < 4; ++d) {
    __syncthreads();
    if (w >= d) {
      const int j = w - d;
      f32x4 acc = {};
      for (int k = j; k < w; ++k) {
        const float* Tkj = k == j ? &L.A[16 * j][16 * j] : &L.A[16 * j][16 * k];
        acc = block_mul(&L.A[16 * w][16 * k], kPitch, Tkj, kPitch, acc, l16, g4);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) L.tmp[w][4 * g4 + i][l16] = acc[i];
      wave_sync();
      const f32x4 t = block_mul(&L.A[16 * w][16 * w], kPitch, &L.tmp[w][0][0], 16, f32x4{}, l16, g4);
#pragma unroll
      for (int i = 0; i < 4; ++i) L.A[16 * j + 4 * g4 + i][16 * w + l16] = -t[i];
    }
  }
  __syncthreads();
  // T and P as operand units of row tile w: slots 4 half .. are tokens 16 (2 s + half) + 4 g4 ..
  f16x8* tri = reinterpret_cast<f16x8*>(p.ws + lay.tri) + (size_t(slot) * p.Hv + h) * (kMaxTri * 64) + lane;
  for (int s = 0; s <= w / 2; ++s) {
    f16x4 t[2][NP], pp[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int cb = 2 * s + half;
      const float* src = cb < w ? &L.A[16 * cb + l16][16 * w + 4 * g4] : &L.A[16 * w + l16][16 * cb + 4 * g4];
      const f32x4 f = cb <= w ? f32x4{src[0], src[1], src[2], src[3]} : f32x4{};
      cut4<NP>(f, t[half]);
      pp[half] = *reinterpret_cast<const f16x4*>(&L.P[16 * w + l16][16 * cb + 4 * g4]);
    }
    const int u = unit_of(w, s);
#pragma unroll
    for (int i = 0; i < NP; ++i) tri[(u * NP + i) * 64] = cath(t[0][i], t[1][i]);
    tri[(kUnits * NP + u) * 64] = cath(pp[0], pp[1]);
  }
}

// ---- scan -------------------------------------------------------------------
//
// Three kinds of it.  kWhole: whole sequences.  With few states and long
// sequences most of the machine would idle, so there sequences are cut into
// segments (kda_segment.hip has the table and the combine): a segment maps the
// state S entering it to P S + R, and kSummary forms R (from zeros) and P (from
// the identity, with values 0) as 256 columns, of all segments but a sequence's
// last at once, without outputs; after the combine kRerun walks all segments at
// once, each from its state.
//
// A wave owns 16 value columns of one state for the whole sequence and
// needs nothing of the other waves' columns: S, R and U stay in its registers
// from the accumulators of one product to the operands of the next, without
// LDS.  An accumulator tile holds, in lane l, rows 4 (l / 16) + i of column l %
// 16; an operand takes 8 k-slots per lane, in any order that both operands
// share.  Two accumulator tiles side by side are such an operand, with the k
// order "4 (l / 16) + i of the first tile, then of the second": T, P and K^T
// are laid out that way by prep_kernel.  For K and Q, whose units hold 8
// adjacent channels per lane, the state's rows are permuted instead: row 4 g +
// i of state tile r is channel 32 (r / 2) + 8 g + 4 (r % 2) + i.
//
// K, Q, K^T, T and P are operands of every wave alike: the workgroup stages a
// chunk's units (1 KB each, in lane order) in LDS, the next chunk's while this
// one is computed, by loads that write LDS directly; one barrier per chunk.

// s_waitcnt operands: at most 0 or 16 vector memory accesses outstanding, the
// other counters as they are (vmcnt in bits 3:0 and 15:14)
constexpr int kVmcnt0 = 0x0f70, kVmcnt16 = 0x4f70;

template <int NP>
struct Stage {
  static constexpr int kTri = kUnits * (NP + 1), kAll = kHeadUnits + kTri;
  u32x4 unit[kAll][64];
  f32x4 coef[kCoefs / 4 + 48];  // two loads of 64 lanes
};

constexpr int kRsrcWord3 = 0x00020000;  // raw buffer, 32-bit offsets
// 16 bytes per lane from base + off + 16 * lane (off scalar) to dst + 16 * lane
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const char* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, -1, kRsrcWord3);
}
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t base, int off, void* dst, int lane16) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(base, (__attribute__((address_space(3))) void*)dst, 16, lane16, off, 0, 0);
}

// The largest of a lane's |x| and of the lanes that share its column
__device__ __forceinline__ float over_column(float m) {
  m = fmaxf(m, __shfl_xor(m, 16));
  return fmaxf(m, __shfl_xor(m, 32));
}

enum { kWhole, kSummary, kRerun };
constexpr uint32_t kRankGrid = 256;

template <int NP, int W, int KIND>
__global__ __launch_bounds__(64 * W, W / 4) void scan_kernel(GdrParams p, GdrLayout lay) {
  __shared__ Stage<NP> L[2];
  constexpr int kSlices = (KIND == kSummary ? 2 : 1) * kD / (16 * W);
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g4 = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = p.Hv / p.Hk;
  // the value heads of a key head on one XCD: its units of K and Q are in that L2
  const int item = work_item(blockIdx.x, gridDim.x, kSlices * group);
  const int m = item / (kSlices * p.Hv), h = item / kSlices % p.Hv, hk = h / group;
  const int col = ((item % kSlices * W + w) * 16 + l16) % kD;  // this lane's value column
  const bool map = KIND == kSummary && item % kSlices >= kSlices / 2;  // a column of P
  int n = m, t0, t1;
  bool last = true;
  int64_t slot0;
  if (KIND == kWhole) {
    // With more workgroups than fit at once the longest sequences go first
    // (ties by index): 32 ragged prompts, 32 heads 291 us against 322.
    if (p.N > 1 && p.N <= 64 && gridDim.x > kRankGrid) {
      int len = -1;
      if (lane < p.N) {
        gdr_range(p, lane, t0, t1);
        len = t1 - t0;
      }
      int rank = 0;
      for (int j = 0; j < p.N; ++j) {
        const int other = __builtin_amdgcn_readlane(len, j);
        rank += other > len || (other == len && j < lane);
      }
      n = __builtin_ctzll(__ballot(lane < p.N && rank == m));
    }
    gdr_range(p, n, t0, t1);
    slot0 = first_slot(p, n);
  } else {
    const int4 e = *reinterpret_cast<const int4*>(p.seg + 4 * m);
    n = e.x;
    last = e.w & 1;
    if (n < 0 || (KIND == kSummary && last)) return;
    t0 = e.y;
    t1 = e.z;
    slot0 = first_slot(p, n) + (t0 - min(max(p.cu[n], 0), p.T)) / kC;
  }
  const int nc = (t1 - t0 + kC - 1) / kC;

  f32x4 S[8];                // the column's state times sc
  float sc = 1.f, inv = 1.f;  // a power of two and its inverse
  const size_t sbase = (size_t(n) * p.Hv + h) * (kD * kD) + col;
  const auto state_at = [&](int r, int i) {
    return sbase + size_t(32 * (r >> 1) + 8 * g4 + 4 * (r & 1) + i) * kD;
  };
  if (KIND == kSummary) {
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[r][i] = map && 32 * (r >> 1) + 8 * g4 + 4 * (r & 1) + i == col ? 1.f : 0.f;
  } else if (KIND == kRerun) {
    const float* s0 = p.starts + (size_t(m) * p.Hv + h) * (kD * kD) + col;
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[r][i] = s0[state_at(r, i) - sbase];
  } else if (!p.s0) {
#pragma unroll
    for (int r = 0; r < 8; ++r) S[r] = f32x4{};
  } else if (p.state_bf16) {
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[r][i] = bf16_to_f32(static_cast<const uint16_t*>(p.s0)[state_at(r, i)]);
  } else {
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[r][i] = static_cast<const float*>(p.s0)[state_at(r, i)];
  }

  const char* headb = p.ws + lay.head + (size_t(slot0) * p.Hk + hk) * (kHeadUnits * 1024);
  const char* trib = p.ws + lay.tri + (size_t(slot0) * p.Hv + h) * (kMaxTri * 1024);
  const char* cob = p.ws + lay.coef + (size_t(slot0) * p.Hv + h) * (kCoefs * 4);
  const char* vb = reinterpret_cast<const char*>(p.v + int64_t(t0) * p.v_t + h * p.v_h);
  char* ob = reinterpret_cast<char*>(p.out + int64_t(t0) * p.o_t + h * p.o_h);
  // in bytes: the strides, and where this lane's column of its first row is
  const uint32_t v_t = 2 * uint32_t(p.v_t), o_t = 2 * uint32_t(p.o_t);
  const uint32_t v_lane = 4 * g4 * v_t + 2 * col, o_lane = 4 * g4 * o_t + 2 * col;

  const auto fetch = [&](int c, Stage<NP>& d) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t head = rsrc_of(headb + size_t(c) * p.Hk * (kHeadUnits * 1024));
    const __amdgpu_buffer_rsrc_t tri = rsrc_of(trib + size_t(c) * p.Hv * (kMaxTri * 1024));
    const __amdgpu_buffer_rsrc_t co = rsrc_of(cob + size_t(c) * p.Hv * (kCoefs * 4));
    const int lane16 = lane * 16;
#pragma unroll
    for (int i = 0; i < kHeadUnits / W; ++i) {
      if (KIND == kSummary && W * i >= kKUnits && W * i < 2 * kKUnits) continue;  // Q
      load_lds(head, (w + W * i) * 1024, &d.unit[w + W * i][0], lane16);
    }
    constexpr int kTri = KIND == kSummary ? kUnits * NP : Stage<NP>::kTri;
#pragma unroll
    for (int i = 0; i < (kTri + W - 1) / W; ++i) {
      const int u = min(w + W * i, kTri - 1);  // (the last one more than once)
      load_lds(tri, u * 1024, &d.unit[kHeadUnits + u][0], lane16);
    }
    load_lds(co, (w & 1) * 1024, &d.coef[64 * (w & 1)], w & 1 ? min(lane16, kCoefs * 4 - 1024 - 16) : lane16);
  };
  // The chunk's values in this lane's column.  Rows behind the sequence's end are
  // zeros, or rows of it where rows overlap: their coefficients are 0.  (No row
  // is inside the buffer for a column of P.)
  uint32_t v[4][4];
  const auto fetch_values = [&](int c) __attribute__((always_inline)) {
    c = min(c, nc - 1);
    uint32_t row = v_t;
    asm("" : "+s"(row));  // (16 multiples of it are not worth 16 registers)
    const uint32_t end = uint32_t(min(kC, t1 - t0 - c * kC) - 1);
    const __amdgpu_buffer_rsrc_t vc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(vb + int64_t(c) * kC * p.v_t * 2), 0, map ? 0 : int(end * v_t + 2 * kD), kRsrcWord3);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[rt][i] = __builtin_amdgcn_raw_buffer_load_b16(vc, int(v_lane + uint32_t(16 * rt + i) * row), 0, 0);
  };
  if (nc > 0) {
    fetch(0, L[0]);
    fetch_values(0);
  }
  __builtin_amdgcn_s_waitcnt(kVmcnt0);
  __syncthreads();
  const auto step = [&](int c, const Stage<NP>& d, Stage<NP>& dn, auto whole) __attribute__((always_inline)) {
    // one register for the units' base (the second stage lies past the offsets that an LDS access holds)
    typedef const __attribute__((address_space(3))) char* lds_t;
    lds_t ub = (lds_t)(&d.unit[0][lane]), cb0 = (lds_t)(&d.coef[g4]);
    asm("" : "+v"(ub));
    asm("" : "+v"(cb0));
    const auto op = [&](int u) { return *reinterpret_cast<const __attribute__((address_space(3))) f16x8*>(ub + u * 1024); };
    const auto coef = [&](int k, int rt) {
      return *reinterpret_cast<const __attribute__((address_space(3))) f32x4*>(cb0 + (k * (kC / 4) + 4 * rt) * 16);
    };
    // (unconditional: the waits for values count the loads behind them)
    if (whole()) fetch(min(c + 1, nc - 1), dn);
    // Bring the larger of |S| and |v| in the column to [2^7, 2^8) (zeros and the smallest columns
    // are left below), unless it is between 2^3 and there in every column of the wave.
    {
      float ms = 0.f, mv = 0.f;
#pragma unroll
      for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) ms = fmaxf(ms, fabsf(S[r][i]));
#pragma unroll
      for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int i = 0; i < 4; ++i) mv = fmaxf(mv, fabsf(bf16_lo(v[rt][i])));
      const float big = over_column(fmaxf(ms * inv, mv));
      const uint32_t e = __float_as_uint(big) >> 23, now = max(e, 27u) - 7u, old = __float_as_uint(inv) >> 23;
      if (__any(now > old || now + 4 < old)) {
        // (to the true size and from there: sc * inv alone passes fp32 where a
        // large column was erased and zeros follow)
        sc = __uint_as_float((254u - now) << 23);
#pragma unroll
        for (int r = 0; r < 8; ++r) S[r] = S[r] * inv * sc;
        inv = __uint_as_float(now << 23);
      }
    }
    // K S and Q S
    f32x4 ks[4] = {}, qs[4] = {};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      f16x4 lo[NP], hi[NP];
      f16x8 b[NP];
      cut4<NP>(S[2 * s], lo);
      cut4<NP>(S[2 * s + 1], hi);
#pragma unroll
      for (int i = 0; i < NP; ++i) b[i] = cath(lo[i], hi[i]);
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) {
        const f16x8 k = op(4 * rt + s), q = op(kKUnits + 4 * rt + s);
#pragma unroll
        for (int i = 0; i < NP; ++i) ks[rt] = mfma32h(k, b[i], ks[rt]);
        if (KIND != kSummary) qs[rt] = mfma32h(q, b[0], qs[rt]);
      }
    }
    // R = beta V - beta e^G K~ S, and U = T R
    f16x4 r[4][NP];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      const f32x4 cb = coef(kBeta, rt), ck = coef(kKs, rt);
      f32x4 x;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = (cb[i] * sc) * bf16_lo(v[rt][i]) - ck[i] * ks[rt][i];
      cut4<NP>(x, r[rt]);
    }
    if (whole()) fetch_values(c + 1);
    f32x4 u[4] = {};
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
#pragma unroll
      for (int z = 0; z <= rt / 2; ++z)
#pragma unroll
        for (int a = 0; a < NP; ++a) {
          const f16x8 t = op(kHeadUnits + unit_of(rt, z) * NP + a);
#pragma unroll
          for (int b = 0; a + b < NP; ++b) u[rt] = mfma32h(t, cath(r[2 * z][b], r[2 * z + 1][b]), u[rt]);
        }
    // the state's update with W = rk e^(G_C - G) U
    const float end = coef(kEnd, 0)[0];
    f16x4 up[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      cut4<1>(u[rt], &up[rt]);
      cut4<NP>(coef(kUs, rt) * u[rt], r[rt]);
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      S[t] *= end;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const f16x8 k = op(2 * kKUnits + 2 * t + z);
#pragma unroll
        for (int b = 0; b < NP; ++b) S[t] = mfma32h(k, cath(r[2 * z][b], r[2 * z + 1][b]), S[t]);
      }
    }
    if (KIND == kSummary) {
      __builtin_amdgcn_s_waitcnt(kVmcnt0);
      __syncthreads();
      return;
    }
    // out = scale (e^G Q~ S + P U)
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      qs[rt] *= coef(kQs, rt);
#pragma unroll
      for (int z = 0; z <= rt / 2; ++z)
        qs[rt] = mfma32h(op(kHeadUnits + kUnits * NP + unit_of(rt, z)), cath(up[2 * z], up[2 * z + 1]), qs[rt]);
      qs[rt] *= p.scale * inv;
    }
    char* oc = ob + int64_t(c) * kC * p.o_t * 2;
    uint32_t orow = o_t;
    asm("" : "+s"(orow));
    const auto store = [&](int rt, int i) __attribute__((always_inline)) {
      *reinterpret_cast<bf16*>(oc + uint64_t(16 * rt + i) * orow + o_lane) = (bf16)qs[rt][i];
    };
    if (whole()) {
      // This wave's loads of the next chunk into LDS have to be there before the
      // barrier, its stores need not: these 16 are its last accesses to memory
      // (nothing is scheduled across the lines around them).
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int i = 0; i < 4; ++i) store(rt, i);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(kVmcnt16);
      __syncthreads();
    } else {
      const int len = t1 - t0 - c * kC;
#pragma unroll
      for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (16 * rt + 4 * g4 + i < len) store(rt, i);
    }
  };
  // whole chunks, then the rest
  const int full = (t1 - t0) / kC;
  for (int c = 0; c < full; c += 2) {
    step(c, L[0], L[1], std::true_type{});
    if (c + 1 < full) step(c + 1, L[1], L[0], std::true_type{});
  }
  if (full < nc) step(full, L[full & 1], L[0], std::false_type{});
#pragma unroll
  for (int r = 0; r < 8; ++r) S[r] *= inv;
  if (KIND == kSummary) {
    float* out = p.summ + ((size_t(m) * p.Hv + h) * 2 + map) * (kD * kD) + col;
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) out[state_at(r, i) - sbase] = S[r][i];
  } else if (!last) {
    return;
  } else if (p.state_bf16) {
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) static_cast<uint16_t*>(p.sT)[state_at(r, i)] = f32_to_bf16(S[r][i]);
  } else {
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) static_cast<float*>(p.sT)[state_at(r, i)] = S[r][i];
  }
}

// ---- launches -----------------------------------------------------------------

template <int NP, int W, int KIND>
hipError_t launch_scan(const GdrParams& p, GdrLayout lay, int64_t seqs, hipStream_t st) {
  GdrParams arg = p;
  void* args[] = {&arg, &lay};
  const int64_t wgs = seqs * p.Hv * (KIND == kSummary ? 2 : 1) * kD / (16 * W);
  return hipLaunchKernel(reinterpret_cast<const void*>(&scan_kernel<NP, W, KIND>), dim3(uint32_t(wgs)),
                         dim3(64 * W), args, 0, st);
}

template <int NP>
hipError_t launch_prep(const GdrParams& p, GdrLayout lay, hipStream_t st) {
  GdrParams arg = p;
  void* args[] = {&arg, &lay};
  return hipLaunchKernel(reinterpret_cast<const void*>(&prep_kernel<NP>), dim3(uint32_t(lay.slots * p.Hv)),
                         dim3(256), args, 0, st);
}

template <int NP>
hipError_t launch_whole(const GdrParams& p, const GdrLayout& lay, int cus, hipStream_t st) {
  if (hipError_t e = launch_prep<NP>(p, lay, st); e != hipSuccess) return e;
  // A workgroup fills a compute unit's LDS, so with at most half as many states
  // as units two workgroups of 64 columns each take one: 8 x 2048 tokens, 16
  // heads 129 us against 155, 1 x 8192, 8 heads 280 against 366; above that one
  // of 128 columns and two waves per SIMD: 32 ragged prompts, 32 heads 326
  // against 417 (sequences in index order).
  return 2 * int64_t(p.N) * p.Hv <= cus ? launch_scan<NP, 4, kWhole>(p, lay, p.N, st)
                                        : launch_scan<NP, 8, kWhole>(p, lay, p.N, st);
}

// The segment-parallel schedule, five launches.  Factors keep 22 bits whatever
// the state's type: P and R are multiplied on.
hipError_t launch_segments(const GdrParams& p, const GdrLayout& lay, int L, hipStream_t st) {
  SegParams sp{};
  sp.cu = p.cu;
  sp.N = p.N;
  sp.T = p.T;
  sp.H = p.Hv;
  sp.L = L;
  sp.M = p.N + p.T / L;
  sp.table = reinterpret_cast<int32_t*>(p.ws + lay.table);
  sp.first = reinterpret_cast<int32_t*>(p.ws + lay.first);
  sp.count = reinterpret_cast<int32_t*>(p.ws + lay.count);
  sp.s0 = p.s0;
  sp.s0_bf16 = p.state_bf16;
  sp.summ = reinterpret_cast<const float*>(p.ws + lay.summ);
  sp.starts = reinterpret_cast<float*>(p.ws + lay.starts);
  GdrParams q = p;
  q.seg = sp.table;
  q.summ = reinterpret_cast<float*>(p.ws + lay.summ);
  q.starts = sp.starts;
  if (hipError_t e = launch_seg_plan(sp, st); e != hipSuccess) return e;
  if (hipError_t e = launch_prep<2>(q, lay, st); e != hipSuccess) return e;
  if (hipError_t e = launch_scan<2, 4, kSummary>(q, lay, sp.M, st); e != hipSuccess) return e;
  if (hipError_t e = launch_seg_combine(sp, st); e != hipSuccess) return e;
  return launch_scan<2, 4, kRerun>(q, lay, sp.M, st);
}

constexpr int kSegSlots = 160;      // (segment, head) pairs that the workspace holds
constexpr int kSegMinTokens = 2048;  // of a call that takes segments

// Tokens per segment, or 0 for whole sequences.  Measured, whole / segments
// (us): 1 x 8192 tokens, 8 heads 305 / 157; 1 x 2048, 8 heads 110 / 74; 1 x
// 16384, 16 heads 693 / 385; 2 x 4096, 16 heads 243 / 192 (207 with the shorter
// segments that fewer states take); 1 x 4096, 32 heads 189 / 191; 1 x 2048, 16
// heads 88 / 88; 1 x 1024, 2 heads 49 / 58.
int segment_length(int64_t T, int Hv, int64_t N) {
  const int64_t pairs = N * Hv;
  if (pairs > 32 || T < (pairs > 8 ? 4096 : 2048) * N) return 0;
  const int64_t target = std::max<int64_t>(1, (pairs > 16 ? 96 : 128) / Hv);
  const int64_t L = std::max<int64_t>(256, ((T + target - 1) / target + kC - 1) / kC * kC);
  return (N + T / L) * Hv <= kSegSlots ? int(L) : 0;
}

}  // namespace

GdrLayout gdr_layout(int64_t T, int Hk, int Hv, int64_t N) {
  GdrLayout l{};
  l.slots = T / kC + N;
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  l.head = 0;
  l.tri = l.head + up(size_t(l.slots) * Hk * kHeadUnits * 1024);
  l.coef = l.tri + up(size_t(l.slots) * Hv * kMaxTri * 1024);
  l.table = l.coef + up(size_t(l.slots) * Hv * kCoefs * 4);
  // one size for every head count, so that the workspace's size grows with each argument
  const size_t seg = T >= kSegMinTokens ? kSegSlots : 0, state = size_t(kD) * kD * 4;
  l.first = l.table + up(16 * seg);
  l.count = l.first + up(4 * seg);
  l.summ = l.count + up(4 * seg);
  l.starts = l.summ + 2 * seg * state;
  l.total = l.starts + seg * state;
  return l;
}

hipError_t launch_gdr_chunked(const GdrParams& p, int cus, hipStream_t stream) {
  const GdrLayout lay = gdr_layout(p.T, p.Hk, p.Hv, p.N);
  if (const int L = segment_length(p.T, p.Hv, p.N); L > 0) return launch_segments(p, lay, L, stream);
  return p.state_bf16 ? launch_whole<1>(p, lay, cus, stream) : launch_whole<2>(p, lay, cus, stream);
}

}  // namespace kda
