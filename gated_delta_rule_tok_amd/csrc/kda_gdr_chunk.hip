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
// in front of U, the coefficients of every token, and K transposed.
// scan_kernel, one workgroup per (sequence, value head, slice of the value
// columns), walks the chunks with the state in registers: four products per
// chunk.
//
// Precision.  q, k and v are bf16, so products with them take the raw rows
// (exact operands) and fp32 norms and decays as coefficients on fp32 sums;
// only S, R, U, T and P have to be rounded to become operands.  Each is cut
// into NP bf16 pieces (x = x0 + x1 (+ x2), 8 bits each): NP = 3 for an fp32
// state (24 bits, all of fp32), NP = 2 for a bf16 state (16 bits: 2^-17 per
// factor, against the 2^-9 of the rounded state and output).  A product of two
// cut factors sums the piece products i + j < NP.
#include "kda_gdr.h"

namespace kda {
namespace {

constexpr int kC = kGdrChunk;
constexpr int kUnits = 6;        // 16 x 32 pieces of a lower triangle of 64: row tile w has w / 2 + 1
constexpr int kUnit = 64 * 8;    // bf16 of one such operand unit (1 KB)
constexpr int kMaxPieces = 3;
constexpr int kTriElems = 2 * kUnits * kMaxPieces * kUnit;  // T and P of one (chunk, head)
constexpr int kCoefs = 5 * kC;   // floats of one (chunk, head)
// coefficient rows: beta; beta e^G rk; scale e^G rq; rk e^(G_C - G); e^(G_C)
enum { kBeta, kKs, kQs, kUs, kEnd };

__device__ __forceinline__ f32x4 mfma4(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// First slot of sequence n (see GdrLayout).
__device__ __forceinline__ int64_t first_slot(const GdrParams& p, int n) {
  return int64_t(min(max(p.cu[n], 0), p.T)) / kC + n;
}

// x as NP bf16 pieces
template <int NP>
__device__ __forceinline__ void cut(float x, bf16* o) {
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    o[i] = (bf16)x;
    x -= (float)o[i];
  }
}

// unit index of (row tile w, k-step s)
__device__ __forceinline__ int unit_of(int w, int s) { return (w < 2 ? w : 2 * w - 2) + s; }

// ---- prep -------------------------------------------------------------------

constexpr int kPitch = 68;  // floats per row of the LDS matrices (bank spread)

struct PrepLds {
  uint4 kf[4][4][64];       // K as operand units [tile][k-step][lane]
  float A[kC][kPitch];      // A below the diagonal; T in the diagonal blocks; T_ij in block (j, i)
  float P[kC][kPitch];
  float tmp[4][16][17];
  double G[kC];
  float rk[kC], rq[kC], beta[kC];
};

// acc += X Y for 16 x 16 fp32 blocks in LDS
__device__ __forceinline__ f32x4 block_mul(const float* X, int xp, const float* Y, int yp, f32x4 acc,
                                           int l16, int g4) {
#pragma unroll
  for (int k = 0; k < 16; k += 4) acc = mfma4(X[l16 * xp + k + g4], Y[(k + g4) * yp + l16], acc);
  return acc;
}

template <int NP>
__device__ __forceinline__ void store_unit(uint16_t* base, int unit, int lane, const float* f) {
  bf16 o[8][NP];
#pragma unroll
  for (int j = 0; j < 8; ++j) cut<NP>(f[j], o[j]);
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const bf16x8 v = {o[0][i], o[1][i], o[2][i], o[3][i], o[4][i], o[5][i], o[6][i], o[7][i]};
    *reinterpret_cast<bf16x8*>(base + (size_t(unit) * NP + i) * kUnit + lane * 8) = v;
  }
}

template <int NP>
__global__ __launch_bounds__(256) void prep_kernel(GdrParams p, GdrLayout lay) {
  __shared__ PrepLds L;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, l16 = lane & 15, g4 = lane >> 4;
  const int64_t slot = blockIdx.x / p.Hv;
  const int h = blockIdx.x % p.Hv, group = p.Hv / p.Hk, hk = h / group;
  int lo = 0, hi = p.N - 1;  // the last sequence whose first slot is not behind this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (first_slot(p, mid) <= slot) lo = mid; else hi = mid - 1;
  }
  int t0, t1;
  gdr_range(p, lo, t0, t1);
  const int64_t off = (slot - first_slot(p, lo)) * kC;
  if (off < 0 || off >= t1 - t0) return;  // no chunk has this slot
  t0 += int(off);
  const int len = min(kC, t1 - t0);

  // rows of K and Q as operands: lane l row l % 16 of tile w, channels 32 s + 8 (l / 16)
  bf16x8 kf[4], qf[4];
  {
    const int r = 16 * w + l16;
    const bool ok = r < len;
    const int64_t t = t0 + (ok ? r : 0);
    const uint16_t* kp = p.k + t * p.k_t + hk * p.k_h + 8 * g4;
    const uint16_t* qp = p.q + t * p.q_t + hk * p.q_h + 8 * g4;
    float sk = 0.f, sq = 0.f;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const uint4 a = ok ? *reinterpret_cast<const uint4*>(kp + 32 * s) : uint4{0, 0, 0, 0};
      const uint4 b = ok ? *reinterpret_cast<const uint4*>(qp + 32 * s) : uint4{0, 0, 0, 0};
      L.kf[w][s][lane] = a;
      kf[s] = __builtin_bit_cast(bf16x8, a);
      qf[s] = __builtin_bit_cast(bf16x8, b);
      float f[8];
      unpack8(a, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sk = fmaf(f[j], f[j], sk);
      unpack8(b, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sq = fmaf(f[j], f[j], sq);
    }
    sk += __shfl_xor(sk, 16);
    sq += __shfl_xor(sq, 16);
    sk += __shfl_xor(sk, 32);
    sq += __shfl_xor(sq, 32);
    if (g4 == 0) {
      L.rk[r] = ok ? 1.f / sqrtf(sk + kNormEps) : 0.f;
      L.rq[r] = ok ? 1.f / sqrtf(sq + kNormEps) : 0.f;
    }
  }
  if (w == 0) {  // gates: lane = token; G in fp64, so that differences of large sums keep their small terms
    const bool ok = lane < len;
    const int64_t t = t0 + (ok ? lane : 0);
    const float la = gdr_log_decay(bf16_to_f32(p.a[t * p.a_t + h * p.a_h]), p.A_log[h], p.dt_bias[h]);
    double G = ok ? double(la) : 0.0;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const double u = __shfl_up(G, o);
      if (lane >= o) G += u;
    }
    L.G[lane] = G;
    L.beta[lane] = ok ? gdr_sigmoid(bf16_to_f32(p.beta[t * p.b_t + h * p.b_h])) : 0.f;
  }
  __syncthreads();
  // K transposed, as operand units [tile of 16 channels][k-step of 32 tokens]: lane l channel l % 16,
  // tokens 32 s + 8 (l / 16); once per key head
  if (h % group == 0) {
    uint16_t* kt = reinterpret_cast<uint16_t*>(p.ws + lay.kt) + (size_t(slot) * p.Hk + hk) * (kD * kC);
    const uint16_t* kl = reinterpret_cast<const uint16_t*>(&L.kf[0][0][0]);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int unit = 4 * w + u, c = 16 * (unit >> 1) + l16, tok = 32 * (unit & 1) + 8 * g4;
      uint16_t e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)  // token t's channel c: tile t / 16, k-step c / 32, lane t % 16 + 16 (c / 8 % 4)
        e[j] = kl[((((tok + j) >> 4) * 4 + (c >> 5)) * 64 + ((tok + j) & 15) + 16 * ((c >> 3) & 3)) * 8 + (c & 7)];
      *reinterpret_cast<uint4*>(kt + unit * kUnit + lane * 8) =
          uint4{uint32_t(e[0]) | uint32_t(e[1]) << 16, uint32_t(e[2]) | uint32_t(e[3]) << 16,
                uint32_t(e[4]) | uint32_t(e[5]) << 16, uint32_t(e[6]) | uint32_t(e[7]) << 16};
    }
  }
  const double Gend = L.G[kC - 1];  // tokens behind the end add nothing
  if (tid < kC) {
    const float eG = expf(float(L.G[tid])), rk = L.rk[tid], b = L.beta[tid];
    float* co = reinterpret_cast<float*>(p.ws + lay.coef) + (size_t(slot) * p.Hv + h) * kCoefs + tid;
    co[kBeta * kC] = b;
    co[kKs * kC] = b * eG * rk;
    co[kQs * kC] = p.scale * eG * L.rq[tid];
    co[kUs * kC] = rk * expf(float(Gend - L.G[tid]));
    co[kEnd * kC] = expf(float(Gend));
  }
  // A and P, row tile w
  for (int j = 0; j < 4; ++j) {
    f32x4 kk = {}, qk = {};
    if (j <= w) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const bf16x8 b = __builtin_bit_cast(bf16x8, L.kf[j][s][lane]);
        kk = mfma32(kf[s], b, kk);
        qk = mfma32(qf[s], b, qk);
      }
    }
    const int s = 16 * j + l16;
    const double Gs = L.G[s];
    const float rs = L.rk[s];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * w + 4 * g4 + i;
      const float e = s <= t ? expf(float(L.G[t] - Gs)) * rs : 0.f;
      if (j <= w) L.A[t][s] = s < t ? L.beta[t] * L.rk[t] * e * kk[i] : 0.f;
      L.P[t][s] = s <= t ? p.scale * L.rq[t] * e * qk[i] : 0.f;
    }
  }
  // T: the diagonal blocks by forward substitution, a column per lane
  {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    float x[16];
    const float* a = &L.A[16 * w][16 * w];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = i == l16 ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < i; ++j) v = fmaf(-a[i * kPitch + j], x[j], v);
      x[i] = v;
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
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
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      const f32x4 t = block_mul(&L.A[16 * w][16 * w], kPitch, &L.tmp[w][0][0], 17, f32x4{}, l16, g4);
#pragma unroll
      for (int i = 0; i < 4; ++i) L.A[16 * j + 4 * g4 + i][16 * w + l16] = -t[i];
    }
  }
  __syncthreads();
  // T and P as operand units of row tile w
  uint16_t* tri = reinterpret_cast<uint16_t*>(p.ws + lay.tri) + (size_t(slot) * p.Hv + h) * kTriElems;
  for (int s = 0; s <= w / 2; ++s) {
    const int c0 = 32 * s + 8 * g4, cb = c0 >> 4;
    float f[8];
    const float* src = cb < w ? &L.A[16 * cb + l16][16 * w + (c0 & 15)] : &L.A[16 * w + l16][c0];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = cb <= w ? src[j] : 0.f;
    store_unit<NP>(tri, unit_of(w, s), lane, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = L.P[16 * w + l16][c0 + j];
    store_unit<NP>(tri + kUnits * kMaxPieces * kUnit, unit_of(w, s), lane, f);
  }
}

// ---- scan -------------------------------------------------------------------

constexpr int kSPitch = kD + 8;  // bf16 per column of the state's pieces
constexpr int kUPitch = kC + 8;  // bf16 per column of the chunk's R and U

template <int NP, int CT>
struct ScanLds {
  bf16 S[NP][16 * CT][kSPitch];
  bf16 R[NP][16 * CT][kUPitch];
  bf16 U[NP][16 * CT][kUPitch];
  bf16 W[NP][16 * CT][kUPitch];  // U with the coefficients of the state's update
};

template <int NP, int PITCH, int COLS>
__device__ __forceinline__ void put4(bf16 (&dst)[NP][COLS][PITCH], int col, int row, f32x4 x) {
  bf16 o[4][NP];
#pragma unroll
  for (int i = 0; i < 4; ++i) cut<NP>(x[i], o[i]);
#pragma unroll
  for (int i = 0; i < NP; ++i) *reinterpret_cast<bf16x4*>(&dst[i][col][row]) = bf16x4{o[0][i], o[1][i], o[2][i], o[3][i]};
}

// acc[ct] += X Y, X in NP-piece operand units, Y in columns of LDS
template <int NP, int CT>
__device__ __forceinline__ void tri_mul(f32x4 (&acc)[CT], const bf16x8 (&x)[2][NP],
                                        const bf16 (&y)[NP][16 * CT][kUPitch], int steps, int l16, int g4) {
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (s < steps) {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int b = 0; b < NP; ++b) {
          const bf16x8 f = *reinterpret_cast<const bf16x8*>(&y[b][16 * ct + l16][32 * s + 8 * g4]);
#pragma unroll
          for (int a = 0; a + b < NP; ++a) acc[ct] = mfma32(x[s][a], f, acc[ct]);
        }
    }
  }
}

// One token row operand of K or Q
__device__ __forceinline__ void load_rows(bf16x8 (&f)[4], const uint16_t* base, bool ok) {
#pragma unroll
  for (int s = 0; s < 4; ++s)
    f[s] = ok ? *reinterpret_cast<const bf16x8*>(base + 32 * s) : bf16x8{};
}

template <int NP, int CT>
__global__ __launch_bounds__(256) void scan_kernel(GdrParams p, GdrLayout lay) {
  __shared__ __align__(16) ScanLds<NP, CT> L;
  constexpr int kSlices = kD / (16 * CT);
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, l16 = lane & 15, g4 = lane >> 4;
  const int item = work_item(blockIdx.x, gridDim.x, kSlices);
  const int n = item / (kSlices * p.Hv), h = item / kSlices % p.Hv, hk = h / (p.Hv / p.Hk);
  const int col0 = item % kSlices * (16 * CT);
  int t0, t1;
  gdr_range(p, n, t0, t1);
  const int nc = (t1 - t0 + kC - 1) / kC;

  // the state: key channels 32 w + 16 r + 4 g4 + i, columns col0 + 16 ct + l16
  f32x4 S[2][CT];
  const size_t sbase = (size_t(n) * p.Hv + h) * (kD * kD) + col0 + l16;
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const size_t e = sbase + size_t(32 * w + 16 * r + 4 * g4 + i) * kD + 16 * ct;
        S[r][ct][i] = !p.s0 ? 0.f
                            : p.state_bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p.s0)[e])
                                           : static_cast<const float*>(p.s0)[e];
      }
  const int64_t slot0 = first_slot(p, n);
  const uint16_t* ktb = reinterpret_cast<const uint16_t*>(p.ws + lay.kt) + (size_t(slot0) * p.Hk + hk) * (kD * kC) + lane * 8;
  const uint16_t* trib = reinterpret_cast<const uint16_t*>(p.ws + lay.tri) + (size_t(slot0) * p.Hv + h) * kTriElems + lane * 8;
  const float* cob = reinterpret_cast<const float*>(p.ws + lay.coef) + (size_t(slot0) * p.Hv + h) * kCoefs;
  const int steps = w / 2 + 1;

  for (int c = 0; c < nc; ++c) {
    const int tok = t0 + c * kC, len = min(kC, t1 - tok);
    const uint16_t* kt = ktb + size_t(c) * p.Hk * (kD * kC);
    const uint16_t* tri = trib + size_t(c) * p.Hv * kTriElems;
    const float* co = cob + size_t(c) * p.Hv * kCoefs;
    const bool rok = 16 * w + l16 < len;
    const int64_t rt = tok + (rok ? 16 * w + l16 : 0);
    bf16x8 kf[4], qf[4];
    load_rows(kf, p.k + rt * p.k_t + hk * p.k_h + 8 * g4, rok);
    f32x4 v[CT];
    const int tr = 16 * w + 4 * g4;  // this lane's four token rows
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool ok = tr + i < len;
      const uint16_t* vp = p.v + int64_t(tok + (ok ? tr + i : 0)) * p.v_t + h * p.v_h + col0 + l16;
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) v[ct][i] = ok ? bf16_to_f32(vp[16 * ct]) : 0.f;
    }
    const f32x4 cb = *reinterpret_cast<const f32x4*>(co + kBeta * kC + tr);
    const f32x4 ck = *reinterpret_cast<const f32x4*>(co + kKs * kC + tr);
    const f32x4 cq = *reinterpret_cast<const f32x4*>(co + kQs * kC + tr);
    const f32x4 cu = *reinterpret_cast<const f32x4*>(co + kUs * kC + tr);
    const float end = co[kEnd * kC];
    bf16x8 tf[2][NP], pf[2][NP], ktf[2][2];
    load_rows(qf, p.q + rt * p.q_t + hk * p.q_h + 8 * g4, rok);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const size_t u = (size_t(unit_of(w, min(s, steps - 1))) * NP + i) * kUnit;
        tf[s][i] = *reinterpret_cast<const bf16x8*>(tri + u);
        pf[s][i] = *reinterpret_cast<const bf16x8*>(tri + kUnits * kMaxPieces * kUnit + u);
      }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int s = 0; s < 2; ++s) ktf[r][s] = *reinterpret_cast<const bf16x8*>(kt + (4 * w + 2 * r + s) * kUnit);

    // the state's pieces
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) put4<NP>(L.S, 16 * ct + l16, 32 * w + 16 * r + 4 * g4, S[r][ct]);
    __syncthreads();
    // K S and Q S, rows of token tile w
    f32x4 ks[CT] = {}, qs[CT] = {};
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int b = 0; b < NP; ++b) {
          const bf16x8 f = *reinterpret_cast<const bf16x8*>(&L.S[b][16 * ct + l16][32 * s + 8 * g4]);
          ks[ct] = mfma32(kf[s], f, ks[ct]);
          qs[ct] = mfma32(qf[s], f, qs[ct]);
        }
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) put4<NP>(L.R, 16 * ct + l16, tr, cb * v[ct] - ck * ks[ct]);
    __syncthreads();
    f32x4 u[CT] = {};
    tri_mul<NP, CT>(u, tf, L.R, steps, l16, g4);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      put4<NP>(L.U, 16 * ct + l16, tr, u[ct]);
      put4<NP>(L.W, 16 * ct + l16, tr, cu * u[ct]);
    }
    __syncthreads();
    // the state's update, key rows 32 w ..
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) S[r][ct] *= end;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int b = 0; b < NP; ++b) {
          const bf16x8 f = *reinterpret_cast<const bf16x8*>(&L.W[b][16 * ct + l16][32 * s + 8 * g4]);
#pragma unroll
          for (int r = 0; r < 2; ++r) S[r][ct] = mfma32(ktf[r][s], f, S[r][ct]);
        }
    // the outputs
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) qs[ct] *= cq;
    tri_mul<NP, CT>(qs, pf, L.U, steps, l16, g4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (tr + i < len) {
        uint16_t* o = p.out + int64_t(tok + tr + i) * p.o_t + h * p.o_h + col0 + l16;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) o[16 * ct] = f32_to_bf16(qs[ct][i]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const size_t e = sbase + size_t(32 * w + 16 * r + 4 * g4 + i) * kD + 16 * ct;
        if (p.state_bf16)
          static_cast<uint16_t*>(p.sT)[e] = f32_to_bf16(S[r][ct][i]);
        else
          static_cast<float*>(p.sT)[e] = S[r][ct][i];
      }
}

template <int NP>
hipError_t launch(const GdrParams& p, int cus, hipStream_t st) {
  GdrParams arg = p;
  GdrLayout lay = gdr_layout(p.T, p.Hk, p.Hv, p.N);
  void* args[] = {&arg, &lay};
  if (hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&prep_kernel<NP>),
                                     dim3(uint32_t(lay.slots * p.Hv)), dim3(256), args, 0, st);
      e != hipSuccess)
    return e;
  const int64_t pairs = int64_t(p.N) * p.Hv;
  if (pairs * 4 >= cus)
    return hipLaunchKernel(reinterpret_cast<const void*>(&scan_kernel<NP, 2>), dim3(uint32_t(pairs * 4)),
                           dim3(256), args, 0, st);
  return hipLaunchKernel(reinterpret_cast<const void*>(&scan_kernel<NP, 1>), dim3(uint32_t(pairs * 8)),
                         dim3(256), args, 0, st);
}

}  // namespace

GdrLayout gdr_layout(int64_t T, int Hk, int Hv, int64_t N) {
  GdrLayout l{};
  l.slots = T / kC + N;
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  l.kt = 0;
  l.tri = l.kt + up(size_t(l.slots) * Hk * kD * kC * 2);
  l.coef = l.tri + up(size_t(l.slots) * Hv * kTriElems * 2);
  l.total = l.coef + up(size_t(l.slots) * Hv * kCoefs * 4);
  return l;
}

hipError_t launch_gdr_chunked(const GdrParams& p, int cus, hipStream_t stream) {
  return p.state_bf16 ? launch<2>(p, cus, stream) : launch<3>(p, cus, stream);
}

}  // namespace kda
