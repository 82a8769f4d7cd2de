// kda_moe.hip -- a mixture-of-experts layer for a decode step's tokens, experts in
// microscaled 4-bit numbers (include/kda_mx4.h has the formulas).
//
// Bound by the bytes of the experts that are hit, each read once.  Four launches:
//   logits   x router^T in fp64, (tile of 16 experts) x (slice of k) per workgroup
//   route    a token per workgroup: slices joined, scores, choice; the last one to
//            finish lists the experts that are hit and their tokens
//   up       16 rows of G and of U of one expert per workgroup, waves share k:
//            h = gate silu(G x) (U x), as two bf16 pieces
//   down     16 rows of W_down of every expert that is hit per workgroup: the sum
//            over experts ends where it is made, nothing goes through memory
//
// The router in fp64: which experts are chosen does not depend on the order of a
// sum, and with a whole-number result there is no rounding to hide behind.  It
// costs 0.75 us of the fp64 matrix pipe per 16 tokens at 256 x 7168.
#include "kda_mx4_dev.h"
#include "kda_mx4_internal.h"

namespace kda {
namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kRouterWaves = 4;
constexpr int kMaxExperts = 1024;

// v_mfma_f64_16x16x4_f64: lane l holds element (l % 16, k = l / 16) of A and B and
// rows l / 16 + 4 j of column l % 16 of the result (checked on the device).
__device__ __forceinline__ f64x4 mfma64(double a, double b, f64x4 c) {
  return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}

__global__ __launch_bounds__(64 * kRouterWaves) void logits_kernel(MoeParams p) {
  __shared__ double red[kRouterWaves][4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int e0 = blockIdx.x * 16, slice = blockIdx.y, m0 = blockIdx.z * 16;
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) p.head[0] = 0;
  const uint16_t* er = p.router + size_t(min(e0 + l16, p.E - 1)) * p.K;
  const uint16_t* xr = p.x + min(m0 + l16, p.M - 1) * p.x_row;
  const int end = min((slice + 1) * p.slice_blocks, p.K / 32);
  f64x4 acc = {};
  for (int b = slice * p.slice_blocks + wave; b < end; b += kRouterWaves) {
    const u32x4 a = *reinterpret_cast<const u32x4*>(er + 32 * b + 8 * g);
    const u32x4 x = *reinterpret_cast<const u32x4*>(xr + 32 * b + 8 * g);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc = mfma64(double(bf16_lo(a[i])), double(bf16_lo(x[i])), acc);
      acc = mfma64(double(bf16_hi(a[i])), double(bf16_hi(x[i])), acc);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) red[wave][j][lane] = acc[j];
  __syncthreads();
  // thread -> expert, token of the tile
  const int e = threadIdx.x & 15, t = threadIdx.x >> 4;
  double s = 0;
#pragma unroll
  for (int w = 0; w < kRouterWaves; ++w) s += red[w][e >> 2][(e & 3) * 16 + t];
  if (e0 + e < p.E && m0 + t < p.M) p.logits[(size_t(slice) * p.M + m0 + t) * p.E + e0 + e] = s;
}

constexpr int kRouteThreads = 256;

// Largest (or sum) over the workgroup, in a fixed order.
template <bool MAX>
__device__ double block_reduce(double v, double* red) {
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    const double w = __shfl_xor(v, o);
    v = MAX ? fmax(v, w) : v + w;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double r = red[0];
  for (int i = 1; i < kRouteThreads / 64; ++i) r = MAX ? fmax(r, red[i]) : r + red[i];
  return r;
}

// The experts that are hit, in order, with their tokens in order; shared experts
// behind them.  One workgroup.
__device__ void list_experts(const MoeParams& p, uint64_t* mask, int32_t* count) {
  const int t = threadIdx.x;
  for (int e = t; e < p.E; e += kRouteThreads) mask[e] = 0;
  __shared__ uint64_t live;
  if (t == 0) live = 0;
  __syncthreads();
  const int pairs = p.M * p.top;
  for (int i = t; i < pairs; i += kRouteThreads) {
    const int e = __hip_atomic_load(p.ids + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (e >= 0) {
      atomicOr(reinterpret_cast<unsigned long long*>(&mask[e]), 1ull << (i / p.top));
      if (i % p.top == 0) atomicOr(reinterpret_cast<unsigned long long*>(&live), 1ull << (i / p.top));
    }
  }
  __syncthreads();
  if (t < 64) {  // one wave: running numbers of slots and of pairs, 64 experts at a time
    int slot = 0, begin = 0;
    for (int e0 = 0; e0 < p.E + p.S; e0 += 64) {
      const int e = e0 + t;
      const uint64_t m = e < p.E ? mask[e] : e < p.E + p.S ? live : 0;
      const int n = __popcll(m);
      const uint64_t hit = __ballot(n > 0);
      int sum = n;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(sum, o);
        if (t >= o) sum += u;
      }
      if (n) {
        const int s = slot + __popcll(hit & ((1ull << t) - 1));
        p.slot_expert[s] = e;
        p.slot_begin[s] = begin + sum - n;
      }
      if (e < p.E) count[e] = begin + sum - n;
      slot += __popcll(hit);
      begin += __shfl(sum, 63);
    }
    if (t == 0) {
      p.slot_begin[slot] = begin;
      p.head[1] = slot;
    }
  }
  __syncthreads();
  int routed = 0;  // pairs of chosen experts: where the shared ones begin
  for (int w = 0; w < p.M; ++w) routed += (live >> w) & 1 ? p.top : 0;
  for (int i = t; i < pairs; i += kRouteThreads) {
    const int e = __hip_atomic_load(p.ids + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (e < 0) continue;
    const int token = i / p.top;
    const int at = count[e] + __popcll(mask[e] & ((1ull << token) - 1));
    p.pairs[at] = token;
    p.pair_gate[at] = __hip_atomic_load(p.gates + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  const int lives = __popcll(live);
  for (int i = t; i < p.S * p.M; i += kRouteThreads) {
    const int s = i / p.M, token = i % p.M;
    if (!((live >> token) & 1)) continue;
    const int at = routed + s * lives + __popcll(live & ((1ull << token) - 1));
    p.pairs[at] = token;
    p.pair_gate[at] = 1.f;
  }
}

__global__ __launch_bounds__(kRouteThreads) void route_kernel(MoeParams p) {
  __shared__ double key[kMaxExperts], score[kMaxExperts], red[kRouteThreads / 64], chosen[32];
  __shared__ int last;
  const int m = blockIdx.x, t = threadIdx.x;
  if (p.idx && p.idx[m] < 0) {
    if (t < p.top) {
      __hip_atomic_store(p.ids + m * p.top + t, -1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(p.gates + m * p.top + t, 0.f, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  } else {
    double most = -INFINITY;
    for (int e = t; e < p.E; e += kRouteThreads) {
      double l = 0;
      for (int s = 0; s < p.slices; ++s) l += p.logits[(size_t(s) * p.M + m) * p.E + e];
      score[e] = l;
      most = fmax(most, l);
    }
    if (p.softmax) {
      most = block_reduce<true>(most, red);
      double sum = 0;
      for (int e = t; e < p.E; e += kRouteThreads) {
        const double l = score[e];
        key[e] = l;
        score[e] = exp(l - most);
        sum += score[e];
      }
      sum = block_reduce<false>(sum, red);
      for (int e = t; e < p.E; e += kRouteThreads) score[e] /= sum;
    } else {
      for (int e = t; e < p.E; e += kRouteThreads) {
        const double l = score[e];
        key[e] = l;
        score[e] = 1.0 / (1.0 + exp(-l));
      }
    }
    // The order is that of the scores plus the bias; without one the logits have the
    // same, also where scores have run into 0 or 1.  No NaN comes before a number.
    for (int e = t; e < p.E; e += kRouteThreads) {
      const double v = p.bias ? score[e] + double(p.bias[e]) : key[e];
      key[e] = v == v ? v : -INFINITY;
    }
    __syncthreads();
    for (int e = t; e < p.E; e += kRouteThreads) {
      const double v = key[e];
      int rank = 0;
      for (int f = 0; f < p.E; ++f) rank += key[f] > v || (key[f] == v && f < e) ? 1 : 0;
      if (rank < p.top) {
        chosen[rank] = score[e];
        __hip_atomic_store(p.ids + m * p.top + rank, e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    __syncthreads();
    if (t < p.top) {
      double sum = 1;
      if (p.renorm) {
        sum = 0;
        for (int j = 0; j < p.top; ++j) sum += chosen[j];
      }
      __hip_atomic_store(p.gates + m * p.top + t, float(chosen[t] / sum * double(p.route_scale)), __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  __threadfence();
  __syncthreads();
  if (t == 0)
    last = __hip_atomic_fetch_add(p.head, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == p.M - 1;
  __syncthreads();
  if (last) list_experts(p, reinterpret_cast<uint64_t*>(key), reinterpret_cast<int32_t*>(score));
}

// h is kept in the order in which down's operands take it: element 32 g + 8 d + e of
// a run of 128 at 32 d + 8 g + e, so that a load of operand d is 64 adjacent bytes a
// token.  Rows are whole runs.
__device__ __forceinline__ int h_place(int i) {
  return (i & ~127) | ((i >> 3) & 3) << 5 | ((i >> 5) & 3) << 3 | (i & 7);
}
__device__ __forceinline__ int h_row(int inter) { return (inter + 127) & ~127; }

constexpr int kUpWaves = 8, kUpSteps = 2;

template <int RQ>
__device__ __forceinline__ void up_tile(const MoeParams& p, char* lds, int expert, int i0, int begin, int n) {
  constexpr int STEPS = kUpSteps;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int nb = p.K / kMxBlock, units = (nb + 4 * STEPS - 1) / (4 * STEPS);
  const int per = (units + kUpWaves - 1) / kUpWaves, first = wave * per, cnt = max(0, min(per, units - first));
  const uint8_t *codes[2], *scales[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const size_t r = (size_t(expert) * 2 + i) * p.I + i0 + l16;
    codes[i] = p.w_up + r * (p.K / 2);
    scales[i] = p.s_up + r * nb;
  }
  f32x4 acc[2] = {};
  char* xl = lds + wave * 4096;
  if (cnt) {
    Piece<STEPS> buf[2][2];
    XRows<RQ> x;
    const auto load = [&](Piece<STEPS>(&b)[2], int unit) {
#pragma unroll
      for (int i = 0; i < 2; ++i) load_piece<STEPS>(b[i], codes[i], scales[i], nb, unit, g);
    };
    load(buf[0], first);
    const uint16_t* row[RQ];
#pragma unroll
    for (int q = 0; q < RQ; ++q) row[q] = p.x + int64_t(p.pairs[begin + min(4 * q + g, n - 1)]) * p.x_row;
    load_x<RQ>(x, row, first * STEPS * 128, p.K, l16);
    const auto use = [&](Piece<STEPS>(&b)[2], int unit) {
#pragma unroll
      for (int j = 0; j < STEPS; ++j) {
        stage_x<RQ>(xl, x, l16, g);
        load_x<RQ>(x, row, (unit * STEPS + j + 1) * 128, p.K, l16);
        wave_lds_fence();
        bf16x8 o[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) o[d] = x_operand(xl, d, l16, g);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float sc = scale_of(b[i].s[j], g);
#pragma unroll
          for (int d = 0; d < 4; ++d) acc[i] = mfma32(dequant8(b[i].w[j][d], sc), o[d], acc[i]);
        }
        wave_lds_fence();
      }
    };
    int i = 0;
    for (; i + 2 <= cnt; i += 2) {
      load(buf[1], first + i + 1);
      use(buf[0], first + i);
      load(buf[0], first + min(i + 2, cnt - 1));
      use(buf[1], first + i + 1);
    }
    if (i < cnt) use(buf[0], first + i);
  }
  f32x4(*red)[2][64] = reinterpret_cast<f32x4(*)[2][64]>(lds);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) red[wave][i][lane] = acc[i];
  __syncthreads();
  if (threadIdx.x < 256) {
    const int r = threadIdx.x & 15, m = threadIdx.x >> 4;
    const float* at = reinterpret_cast<const float*>(&red[0][0][(r >> 2) * 16 + m]) + (r & 3);
    float a = at[0], u = at[256];
#pragma unroll
    for (int w = 1; w < kUpWaves; ++w) a += at[w * 512], u += at[w * 512 + 256];
    if (m < n) {
      const float h = a / (1.f + __expf(-a)) * u * p.pair_gate[begin + m];
      const uint16_t hi = f32_to_bf16(h);
      const size_t o = size_t(begin + m) * h_row(p.I) + h_place(i0 + r);
      p.h_hi[o] = hi;
      p.h_lo[o] = f32_to_bf16(h - bf16_to_f32(hi));
    }
  }
}

__global__ __launch_bounds__(64 * kUpWaves) void up_kernel(MoeParams p) {
  __shared__ __align__(16) char lds[kUpWaves * 4096];
  const int slot = blockIdx.y;
  if (slot >= p.head[1]) return;
  const int begin = p.slot_begin[slot] + 16 * blockIdx.z, n = min(16, p.slot_begin[slot + 1] - begin);
  if (n <= 0) return;
  const int expert = p.slot_expert[slot];
  if (n <= 4)
    up_tile<1>(p, lds, expert, 16 * blockIdx.x, begin, n);
  else
    up_tile<4>(p, lds, expert, 16 * blockIdx.x, begin, n);
}

constexpr int kDownWaves = 8, kDownSteps = 2;

// h of one token for STEPS steps: its two pieces' operands.
struct HPiece {
  bf16x8 hi[kDownSteps][4], lo[kDownSteps][4];
};

__global__ __launch_bounds__(64 * kDownWaves) void down_kernel(MoeParams p) {
  constexpr int STEPS = kDownSteps;
  extern __shared__ __align__(16) char lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int nb = p.I / kMxBlock, units = (nb + 4 * STEPS - 1) / (4 * STEPS);
  const int slots = p.head[1], jobs = slots * units;
  const int per = (jobs + kDownWaves - 1) / kDownWaves, first = wave * per, cnt = max(0, min(per, jobs - first));
  // [wave][token][16]: this wave's sums
  f32x4* y = reinterpret_cast<f32x4*>(lds) + wave * p.M * 4;
  for (int i = lane; i < p.M * 4; i += 64) y[i] = f32x4{};
  wave_lds_fence();
  const int hrow = h_row(p.I);

  const auto load_w = [&](Piece<STEPS>& b, int job) {
    const int expert = p.slot_expert[job / units];
    const size_t r = size_t(expert) * p.K + n0 + l16;
    load_piece<STEPS>(b, p.w_down + r * (p.I / 2), p.s_down + r * nb, nb, job % units, g);
  };
  const auto load_h = [&](HPiece& h, int at, int unit) {
    const uint16_t *hi = p.h_hi + size_t(at) * hrow, *lo = p.h_lo + size_t(at) * hrow;
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      const int b = (unit * STEPS + j) * 4 + g;
      const bool in = b < nb;
      const int k = in ? (unit * STEPS + j) * 128 + 8 * g : 0;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        h.hi[j][d] = *reinterpret_cast<const bf16x8*>(hi + (in ? k + 32 * d : 0));
        h.lo[j][d] = *reinterpret_cast<const bf16x8*>(lo + (in ? k + 32 * d : 0));
        if (!in) h.hi[j][d] = h.lo[j][d] = bf16x8{};
      }
    }
  };
  Piece<STEPS> buf[2];
  const auto use = [&](const Piece<STEPS>& b, int job) {
    const int slot = job / units, unit = job % units;
    const int begin = p.slot_begin[slot], n = p.slot_begin[slot + 1] - begin;
    for (int t0 = 0; t0 < n; t0 += 16) {
      const int at = begin + min(t0 + l16, n - 1);
      HPiece h;
      load_h(h, at, unit);
      const int token = p.pairs[at];
      f32x4 acc = {};
#pragma unroll
      for (int j = 0; j < STEPS; ++j) {
        const float sc = scale_of(b.s[j], g);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const bf16x8 w = dequant8(b.w[j][d], sc);
          acc = mfma32(w, h.hi[j][d], acc);
          acc = mfma32(w, h.lo[j][d], acc);
        }
      }
      if (t0 + l16 < n) y[token * 4 + g] += acc;
      wave_lds_fence();
    }
  };
  if (cnt) {
    load_w(buf[0], first);
    int i = 0;
    for (; i + 2 <= cnt; i += 2) {
      load_w(buf[1], first + i + 1);
      use(buf[0], first + i);
      load_w(buf[0], first + min(i + 2, cnt - 1));
      use(buf[1], first + i + 1);
    }
    if (i < cnt) use(buf[0], first + i);
  }
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(lds);
  for (int i = threadIdx.x; i < p.M * 16; i += 64 * kDownWaves) {
    const int m = i >> 4;
    if (p.idx && p.idx[m] < 0) continue;
    float s = all[i];
#pragma unroll
    for (int w = 1; w < kDownWaves; ++w) s += all[w * p.M * 16 + i];
    p.out[m * p.out_row + n0 + (i & 15)] = f32_to_bf16(s);
  }
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

// Slices of the router's sums: about 256 workgroups for 16 tokens, whatever the
// number of tokens (the size of the workspace grows with it and never falls).
MoeLayout moe_layout(int M, int K, int I, int E, int S, int top) {
  MoeLayout l{};
  const int nb = K / kMxBlock, tiles = (E + 15) / 16;
  int slices = 256 / tiles;
  if (slices > (nb + kRouterWaves - 1) / kRouterWaves) slices = (nb + kRouterWaves - 1) / kRouterWaves;
  if (slices < 1) slices = 1;
  l.slice_blocks = (nb + slices - 1) / slices;
  l.slices = (nb + l.slice_blocks - 1) / l.slice_blocks;
  l.slots = (int64_t(M) * top < E ? M * top : E) + S;
  const size_t pairs = size_t(M) * (top + S), hrow = (size_t(I) + 127) & ~size_t(127);
  size_t at = 0;
  const auto part = [&](size_t bytes) {
    const size_t here = at;
    at = up256(at + bytes);
    return here;
  };
  l.head = part(2 * 4);
  l.logits = part(size_t(l.slices) * M * E * 8);
  l.slot_expert = part(size_t(l.slots) * 4);
  l.slot_begin = part(size_t(l.slots + 1) * 4);
  l.pairs = part(pairs * 4);
  l.pair_gate = part(pairs * 4);
  l.h_hi = part(pairs * hrow * 2);
  l.h_lo = part(pairs * hrow * 2);
  l.total = at;
  return l;
}

hipError_t launch_moe(const MoeParams& p, int cus, hipStream_t st) {
  MoeParams arg = p;
  void* args[] = {&arg};
  const auto go = [&](const void* f, dim3 grid, int threads, size_t lds) {
    return hipLaunchKernel(f, grid, dim3(threads), args, lds, st);
  };
  const int tiles = (p.M + 15) / 16, slots = (p.M * p.top < p.E ? p.M * p.top : p.E) + p.S;
  hipError_t e = go(reinterpret_cast<const void*>(&logits_kernel), dim3((p.E + 15) / 16, p.slices, tiles),
                    64 * kRouterWaves, 0);
  if (e != hipSuccess) return e;
  e = go(reinterpret_cast<const void*>(&route_kernel), dim3(p.M), kRouteThreads, 0);
  if (e != hipSuccess) return e;
  e = go(reinterpret_cast<const void*>(&up_kernel), dim3(p.I / 16, slots, tiles), 64 * kUpWaves, 0);
  if (e != hipSuccess) return e;
  return go(reinterpret_cast<const void*>(&down_kernel), dim3(p.K / 16), 64 * kDownWaves,
            size_t(kDownWaves) * p.M * 64);
}

}  // namespace kda
