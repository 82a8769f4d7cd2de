// kda_moe.hip -- a mixture-of-experts layer for a decode step's tokens, experts in
// microscaled 4-bit numbers (include/kda_mx4.h has the formulas).
//
// Bound by the bytes of the experts that are hit, each read once.  Four launches:
//   logits   x router^T in fp64, (tile of 16 experts) x (slice of k) per workgroup
//   route    a token per workgroup: slices joined, scores, choice; the last one to
//            finish lists the experts that are hit and their tokens, as slots
//   up       h = gate silu(G x) (U x), as three bf16 pieces: a workgroup walks through
//            a run of (slot, 16 rows of G and of U), its waves share k
//   down     16 rows of W_down of all slots per workgroup, or of a part of them where
//            the rows are few; the sum over experts ends there
//
// The router in fp64: which experts are chosen does not depend on the order of a
// sum, and with a whole-number result there is no rounding to hide behind.  It
// costs 0.75 us of the fp64 matrix pipe per 16 tokens at 256 x 7168.
//
// 7168 x 512, 8 + 1 of 256 experts: one token 30 us (logits 5.5, route 5.7, up 13.5, down
// 8: each a launch and a chain of round trips, 50 MB in all), 64 tokens 335 to 361 us by
// how many experts they hit (up 194, 4.2 TB/s; down 128, 3.2 TB/s: its third piece of h
// costs 11 us; a copy reaches 5.0).  What it took, each as measured then: whole lines
// through LDS instead of operands as they are wanted (404 to 286 us on tokens that hit half
// the experts: the address unit was the bound), units of 256 of k in down (139 to 111:
// instructions were), short code, since single-token launches run each line of it once.
#include "kda_mx4_dev.h"
#include "kda_mx4_internal.h"

namespace kda {
namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kRouterWaves = 4;
constexpr int kMaxExperts = 1024;
constexpr int kWaves = 8;  // of the workgroups of up and down
constexpr int kDownSteps4 = 2, kDownSteps16 = 1;  // 128s of k in a unit of down, by tokens a slot

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
  if (blockIdx.x == 0 && blockIdx.z == 0) {  // counters of the launches behind this one
    if (slice == 0 && threadIdx.x == 0) p.head[0] = 0;
    for (int i = slice * (64 * kRouterWaves) + threadIdx.x; i < p.K / 16; i += gridDim.y * (64 * kRouterWaves))
      p.done[i] = 0;
  }
  const uint16_t* er = p.router + size_t(min(e0 + l16, p.E - 1)) * p.K;
  const uint16_t* xr = p.x + min(m0 + l16, p.M - 1) * p.x_row;
  const int end = min((slice + 1) * p.slice_blocks, p.K / 32);
  f64x4 acc = {};
  constexpr int kAtOnce = 4;  // blocks of 32 whose loads are under way together
  for (int b0 = slice * p.slice_blocks + wave; b0 < end; b0 += kAtOnce * kRouterWaves) {
    u32x4 a[kAtOnce], x[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int b = min(b0 + u * kRouterWaves, end - 1);
      a[u] = *reinterpret_cast<const u32x4*>(er + 32 * b + 8 * g);
      x[u] = *reinterpret_cast<const u32x4*>(xr + 32 * b + 8 * g);
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      if (b0 + u * kRouterWaves >= end) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc = mfma64(double(bf16_lo(a[u][i])), double(bf16_lo(x[u][i])), acc);
        acc = mfma64(double(bf16_hi(a[u][i])), double(bf16_hi(x[u][i])), acc);
      }
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

// Slot number `slot`: the expert and tokens c * chunk .. of those in mask; its pairs
// begin at `begin`.
__device__ __forceinline__ void write_slot(const MoeParams& p, int slot, int expert, uint64_t mask, int c, int begin) {
  for (int i = 0; i < c * p.chunk; ++i) mask &= mask - 1;
  MoeSlot o;
  o.expert = expert, o.begin = begin + c * p.chunk, o.n = min(__popcll(mask), p.chunk), o.unused = 0;
  uint32_t token = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    o.token[q] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (mask) token = uint32_t(__builtin_ctzll(mask));  // (the last one is repeated)
      mask &= mask - 1;
      o.token[q] |= token << (8 * i);
    }
  }
  p.slot[slot] = o;
}

// Agent-scope accesses go past the caches that other workgroups do not see, so that
// what is written with them is there once vmcnt says so: no cache has to be written
// back or emptied around the counter that announces it.
__device__ __forceinline__ void stores_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
template <typename T>
__device__ __forceinline__ void put(T* p, T v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
template <typename T>
__device__ __forceinline__ T get(const T* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
// Whether this workgroup is the last of n to come here (counter: 0 before the first).
__device__ __forceinline__ bool come_last(int32_t* counter, int n) {
  __shared__ int last;
  stores_done();
  __syncthreads();
  if (threadIdx.x == 0)
    last = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == n - 1;
  __syncthreads();
  return last;
}

constexpr int kMaxSlots = 64 * 32 + 16 * 16;

// The experts that are hit, in order, with their tokens in order; shared experts
// behind them.  One workgroup.
struct RouteLds {
  double key[kMaxExperts], next[kMaxExperts];  // the order: of the sums, then of the logits
  double score[kMaxExperts], red[kRouteThreads / 64], chosen[32];
  int chosen_id[32];
  int16_t best[kMaxExperts / 64 * 32];
};
struct ListLds {
  uint64_t mask[kMaxExperts + 16];
  uint16_t first[kMaxExperts + 16], slot_of[kMaxSlots];  // expert * 16 + chunk
  int16_t ids[64 * 32];
  float gates[64 * 32];
  uint64_t live;
  int total[kRouteThreads / 64];
};
__device__ void list_slots(const MoeParams& p, ListLds& L) {
  const int t = threadIdx.x, lane = t & 63, every = p.E + p.S;
  for (int e = t; e < p.E; e += kRouteThreads) L.mask[e] = 0;
  if (t == 0) L.live = 0;
  __syncthreads();
  const int pairs = p.M * p.top;
  for (int i = t; i < pairs; i += kRouteThreads) {
    const int e = get(p.ids + i);
    L.gates[i] = get(p.gates + i);
    L.ids[i] = int16_t(e);
    if (e >= 0) {
      const int token = i / p.top;
      atomicOr(reinterpret_cast<unsigned long long*>(&L.mask[e]), 1ull << token);
      if (i == token * p.top) atomicOr(reinterpret_cast<unsigned long long*>(&L.live), 1ull << token);
    }
  }
  __syncthreads();
  if (t < p.S) L.mask[p.E + t] = L.live;
  __syncthreads();
  // running numbers of slots (upper half) and pairs (lower), an expert a thread
  int before = 0;
  for (int e0 = 0; e0 < every; e0 += kRouteThreads) {
    const int e = e0 + t, n = e < every ? __popcll(L.mask[e]) : 0, c = (n + p.chunk - 1) / p.chunk;
    int sum = c << 16 | n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(sum, o);
      if (lane >= o) sum += u;
    }
    if (lane == 63) L.total[t >> 6] = sum;
    __syncthreads();
    int at = before + sum - (c << 16 | n);
#pragma unroll
    for (int w = 0; w < kRouteThreads / 64; ++w) {
      if (w < t >> 6) at += L.total[w];
      before += L.total[w];
    }
    __syncthreads();
    if (n) L.first[e] = uint16_t(at & 0xffff);
    for (int i = 0; i < c; ++i) L.slot_of[(at >> 16) + i] = uint16_t(e * 16 + i);
  }
  const int slots = before >> 16, lives = __popcll(L.live);
  if (t == 0) p.head[1] = slots;
  __syncthreads();
  for (int i = t; i < slots; i += kRouteThreads) {
    const int e = L.slot_of[i] >> 4;
    write_slot(p, i, e, L.mask[e], L.slot_of[i] & 15, L.first[e]);
  }
  for (int i = t; i < pairs; i += kRouteThreads) {
    const int e = L.ids[i];
    if (e >= 0) p.pair_gate[L.first[e] + __popcll(L.mask[e] & ((1ull << (i / p.top)) - 1))] = L.gates[i];
  }
  for (int i = t; i < p.S * lives; i += kRouteThreads) p.pair_gate[lives * p.top + i] = 1.f;
}

// Numbers in the order of v (logits and sums; finite ones are far from 1e300), a NaN behind
// minus infinity.
__device__ __forceinline__ double order_of(double v) {
  return v != v ? -INFINITY : v == -INFINITY ? -1e300 : v;
}
// Of two experts whose sums are the same: whether f comes before e.
__device__ __forceinline__ bool next_before(const RouteLds& L, int f, int e) {
  const double a = L.next[f], b = L.next[e];
  return a > b || (a == b && f < e);
}
// The top largest keys, of equal ones the largest next, of equal ones of these the first:
// each wave ranks 64 adjacent experts at a time, then the best of those are ranked among
// each other.
__device__ __forceinline__ void choose(const MoeParams& p, RouteLds& L, int m) {
  const int t = threadIdx.x, lane = t & 63;
  for (int e0 = t & ~63; e0 < p.E; e0 += kRouteThreads) {
    const int e = e0 + lane, end = min(64, p.E - e0);
    const double v = L.key[min(e, p.E - 1)];
    int rank = 0, same = 0;
#pragma unroll 8
    for (int i = 0; i < end; ++i) {
      const double o = L.key[e0 + i];
      rank += o > v ? 1 : 0;
      same += o == v ? 1 : 0;
    }
    if (lane < end && same > 1)
      for (int i = 0; i < end; ++i) rank += L.key[e0 + i] == v && next_before(L, e0 + i, e) ? 1 : 0;
    if (lane < end && rank < p.top) L.best[(e0 >> 6) * p.top + rank] = int16_t(e);
  }
  __syncthreads();
  const int whole = (p.E - 1) >> 6, n = whole * p.top + min(p.top, p.E - 64 * whole);
  for (int i = t; i < n; i += kRouteThreads) {
    const int e = L.best[i];
    const double v = L.key[e];
    int rank = 0, same = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const double o = L.key[L.best[j]];
      rank += o > v ? 1 : 0;
      same += o == v ? 1 : 0;
    }
    if (same > 1)
      for (int j = 0; j < n; ++j) rank += L.key[L.best[j]] == v && next_before(L, L.best[j], e) ? 1 : 0;
    if (rank < p.top) {
      L.chosen[rank] = L.score[e];
      L.chosen_id[rank] = e;
      put(p.ids + m * p.top + rank, e);
    }
  }
}

__global__ __launch_bounds__(kRouteThreads) void route_kernel(MoeParams p) {
  __shared__ union {
    RouteLds route;
    ListLds list;
  } L;
  double *score = L.route.score, *red = L.route.red, *chosen = L.route.chosen;
  double *key = L.route.key, *next = L.route.next;
  int* chosen_id = L.route.chosen_id;
  const int m = blockIdx.x, t = threadIdx.x;
  if (p.idx && p.idx[m] < 0) {
    if (t < p.top) {
      put(p.ids + m * p.top + t, -1);
      put(p.gates + m * p.top + t, 0.f);
    }
  } else {
    double most = -INFINITY;
    for (int e = t; e < p.E; e += kRouteThreads) {
      double l = 0;
#pragma unroll 8
      for (int s = 0; s < p.slices; ++s) l += p.logits[(size_t(s) * p.M + m) * p.E + e];
      score[e] = l;
      most = fmax(most, l);
    }
    if (p.softmax) {
      most = block_reduce<true>(most, red);
      double sum = 0;
      for (int e = t; e < p.E; e += kRouteThreads) {
        const double l = score[e];
        next[e] = order_of(l);
        score[e] = exp(l - most);
        sum += score[e];
      }
      sum = block_reduce<false>(sum, red);
      for (int e = t; e < p.E; e += kRouteThreads) score[e] /= sum;
    } else {
      for (int e = t; e < p.E; e += kRouteThreads) {
        const double l = score[e];
        next[e] = order_of(l);
        score[e] = 1.0 / (1.0 + exp(-l));
      }
    }
    // The order is that of the scores plus the bias.  Where 64 bits hold two sums as the
    // same (scores that have run into 0 or 1, or a bias that is far larger) that of the
    // logits, which is theirs for equal biases; sums that are infinite are the same indeed.
    for (int e = t; e < p.E; e += kRouteThreads) {
      const double v = score[e] + (p.bias ? double(p.bias[e]) : 0.0);
      key[e] = order_of(v);
      if (isinf(v)) next[e] = 0;
    }
    __syncthreads();
    choose(p, L.route, m);
    __syncthreads();
    if (t < p.top) {
      double sum = 1;
      if (p.renorm) {
        sum = 0;
        for (int j = 0; j < p.top; ++j) sum += chosen[j];
      }
      const float gate = float(chosen[t] / sum * double(p.route_scale));
      put(p.gates + m * p.top + t, gate);
      if (p.M == 1) p.pair_gate[t] = gate;
    }
  }
  if (p.M == 1) {  // the choice is the list
    const int n = p.idx && p.idx[0] < 0 ? 0 : p.top + p.S;
    if (t < n) {
      write_slot(p, t, t < p.top ? chosen_id[t] : p.E + t - p.top, 1, 0, t);
      if (t >= p.top) p.pair_gate[t] = 1.f;
    }
    if (t == 0) p.head[1] = n;
    return;
  }
  if (come_last(p.head, p.M)) list_slots(p, L.list);
}

// Data that a launch before this one wrote, read through the scalar cache.
template <typename T>
__device__ __forceinline__ const __attribute__((address_space(4))) T* scalar(const T* p) {
  return (const __attribute__((address_space(4))) T*)(p);
}
struct SlotView {
  int expert, begin, n;
  uint32_t t0, t1, t2, t3;
  __device__ __forceinline__ SlotView(const MoeSlot* p) {
    const auto* s = scalar(p);
    expert = s->expert, begin = s->begin, n = s->n;
    t0 = s->token[0], t1 = s->token[1], t2 = s->token[2], t3 = s->token[3];
  }
  // tokens 4 q + g and i, of a lane
  template <int Q>
  __device__ __forceinline__ int token4(int g) const {
    return ((Q == 0 ? t0 : Q == 1 ? t1 : Q == 2 ? t2 : t3) >> (8 * g)) & 0xff;
  }
  __device__ __forceinline__ int token(int i) const {
    const uint32_t lo = i & 4 ? t1 : t0, hi = i & 4 ? t3 : t2;
    return ((i & 8 ? hi : lo) >> (8 * (i & 3))) & 0xff;
  }
};

// A workgroup's items are adjacent (slot, tile of 16 rows) pairs; the units of k of a
// wave, item after item, go through a ring of U, so that the next item's loads are
// under way while this one is joined.
template <int RQ, int STEPS, int U, bool TINY>
__global__ __launch_bounds__(64 * kWaves, 4) void up_kernel(MoeParams p) {
  constexpr int kX = STEPS * RQ * 1024, kWave = kX + 2 * kPieceLds<STEPS>;
  __shared__ __align__(16) char lds[kWaves * kWave];
  __shared__ f32x4 red[kWaves][2][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int tiles = p.I / 16;
  const uint32_t items = scalar(p.head)[1] * tiles;
  const uint32_t lo = items * blockIdx.x >> p.up_log2, hi = items * (blockIdx.x + 1) >> p.up_log2;
  if (lo >= hi) return;
  const int nb = p.K / kMxBlock, units = (nb + 4 * STEPS - 1) / (4 * STEPS);
  const int first = units * wave / kWaves, cnt = units * (wave + 1) / kWaves - first;
  char *xl = lds + wave * kWave, *wl = xl + kX;
  const uint32_t row_bytes = p.K / 2, code_row = (lane >> 2) * row_bytes, scale_row = (lane >> 2) * nb;
  const int slot0 = lo / tiles, tile0 = lo - slot0 * tiles;

  struct Unit {
    Piece<STEPS> w[2];
    XRows<RQ> x[STEPS];
  } buf[U];
  // what is loaded next; n of the slot that is loaded and of the one that is used
  int n_load = 0, n_use = 0, left_items = hi - lo, slot = slot0, tile = tile0, unit = 0;
  const uint8_t *codes[2], *scales[2];
  uint32_t row[RQ];
  const auto aim_slot = [&](const SlotView& s) {
    n_load = s.n;
    const uint32_t x_bytes = uint32_t(p.x_row) * 2;
    row[0] = s.token4<0>(g) * x_bytes;
    if (RQ > 1) {
      row[1 % RQ] = s.token4<1>(g) * x_bytes;
      row[2 % RQ] = s.token4<2>(g) * x_bytes;
      row[3 % RQ] = s.token4<3>(g) * x_bytes;
    }
  };
  const auto aim_tile = [&](int expert) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const size_t r = (size_t(expert) * 2 + i) * p.I + tile * 16;
      codes[i] = p.w_up + r * row_bytes;
      scales[i] = p.s_up + r * nb;
    }
  };
  // (Loads behind the last unit to keep the number in flight constant, so that the waits
  // could count them, cost more than waiting for all: other waves fill the time.)
  const auto load = [&](Unit& b) {
    if (left_items == 0) return;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      load_piece<STEPS, TINY>(b.w[i], codes[i], code_row, scales[i], scale_row, nb, first + unit, lane & 3);
#pragma unroll
    for (int j = 0; j < STEPS; ++j) load_x<RQ>(b.x[j], p.x, row, ((first + unit) * STEPS + j) * 128, p.K, l16, n_load);
    if (++unit == cnt) {
      unit = 0;
      if (--left_items > 0) {
        if (++tile == tiles) tile = 0, ++slot;
        const SlotView s(p.slot + slot);
        if (tile == 0) aim_slot(s);
        aim_tile(s.expert);
      }
    }
  };
  f32x4 acc[2] = {};
  const auto use = [&](Unit& b, int unit) {
#pragma unroll
    for (int i = 0; i < 2; ++i) stage_piece<STEPS, TINY>(wl + i * kPieceLds<STEPS>, b.w[i], nb, first + unit, lane);
#pragma unroll
    for (int j = 0; j < STEPS; ++j)
      stage_x<RQ>(xl + j * (RQ * 1024), b.x[j], ((first + unit) * STEPS + j) * 128, p.K, l16, g, n_use);
    wave_lds_fence();
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      bf16x8 o[4];
#pragma unroll
      for (int d = 0; d < 4; ++d) o[d] = x_operand<RQ>(xl + j * (RQ * 1024), d, l16, g);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const char* at = wl + i * kPieceLds<STEPS>;
        const float sc = scale_of(scale_operand<STEPS>(at, j, l16, g));
        const u32x4 c = codes_operand(at, j, l16, g);
#pragma unroll
        for (int d = 0; d < 4; ++d) acc[i] = mfma32(dequant8(c[d], sc), o[d], acc[i]);
      }
    }
    wave_lds_fence();
  };
  int items_left = hi - lo;
  // joins the waves' sums of an item
  int at_slot = slot0, at_tile = tile0;
  const auto join = [&]() {
    __syncthreads();  // the last item's are read
    red[wave][0][lane] = acc[0], red[wave][1][lane] = acc[1];
    acc[0] = acc[1] = f32x4{};
    __syncthreads();
    if (wave < RQ) {
      const int n = lane & 15, m = 4 * wave + g;  // row of the tile, pair of the slot
      const SlotView s(p.slot + at_slot);
      if (4 * wave < s.n) {
        const auto* gate4 = scalar(p.pair_gate) + s.begin + 4 * wave;
        const float g0 = gate4[0], g1 = gate4[1], g2 = gate4[2], g3 = gate4[3];
        const float gate = g & 2 ? (g & 1 ? g3 : g2) : (g & 1 ? g1 : g0);
        const float* at = reinterpret_cast<const float*>(&red[0][0][(n >> 2) * 16 + m]) + (n & 3);
        float a = at[0], u = at[256];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) a += at[w * 512], u += at[w * 512 + 256];
        if (m < s.n) {
          const float h = a / (1.f + __expf(-a)) * u * gate;
          // all 24 bits of h, 8 to a piece: cut, not rounded, so that the rest is exact and
          // the first never passes bf16's largest
          const size_t plane = size_t(p.M) * (p.top + p.S) * p.I;
          uint16_t* o = p.h + size_t(s.begin + m) * p.I + at_tile * 16 + n;
          float rest = h;
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            const uint32_t piece = __float_as_uint(rest) & 0xffff0000u;
            o[i * plane] = uint16_t(piece >> 16);
            rest -= __uint_as_float(piece);
          }
        }
      }
    }
    if (++at_tile == tiles) {
      at_tile = 0, ++at_slot;
      if (items_left > 1) n_use = scalar(p.slot + at_slot)->n;
    }
  };
  if (cnt == 0) {  // (fewer units than waves)
    for (; items_left > 0; --items_left) join();
    return;
  }
  {
    const SlotView s(p.slot + slot0);
    aim_slot(s);
    aim_tile(s.expert);
    n_use = s.n;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) load(buf[u]);
  int at_unit = 0;
  for (;;) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      use(buf[u], at_unit);
      load(buf[u]);
      if (++at_unit == cnt) {
        join();
        if (--items_left == 0) return;
        at_unit = 0;
      }
    }
  }
}

// The operands of h in LDS: with 4 tokens a slot the three pieces of a step as rows 4 i +
// token, which are columns of one MFMA (and added up when the slot is done); with 16 one
// piece of all steps after the other.
template <int RQ, int STEPS>
constexpr int kDownH = RQ == 1 ? 3 * 1024 : STEPS * RQ * 1024;

template <int RQ, int STEPS, int U, bool TINY>
__global__ __launch_bounds__(64 * kWaves, 4) void down_kernel(MoeParams p) {
  extern __shared__ __align__(16) char lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16, part = blockIdx.y;
  const int nb = p.I / kMxBlock, units = (nb + 4 * STEPS - 1) / (4 * STEPS);
  const uint32_t jobs = scalar(p.head)[1] * units;
  // this wave's run of (slot, unit of k)
  const uint32_t share = part * kWaves + wave, shares = p.parts * kWaves;
  const int first = jobs * share / shares, end = jobs * (share + 1) / shares;
  constexpr int kH = kDownH<RQ, STEPS>, kWave = kH + kPieceLds<STEPS>;
  char *hl = lds + wave * kWave, *wl = hl + kH;
  // [wave][token][16]: this wave's sums
  f32x4* y = reinterpret_cast<f32x4*>(lds + kWaves * kWave) + wave * p.M * 4;
  for (int i = lane; i < p.M * 4; i += 64) y[i] = f32x4{};
  wave_lds_fence();
  if (first < end) {
    struct Unit {
      Piece<STEPS> w;
      XRows<RQ> h[3][STEPS];
    } buf[U];
    // what is loaded next
    const uint32_t row_bytes = p.I / 2, code_row = (lane >> 2) * row_bytes, scale_row = (lane >> 2) * nb;
    const int slot0 = first / units;
    int job = first, slot = slot0, unit = first - slot0 * units;
    const uint8_t *codes, *scales;
    const uint16_t* h;
    const size_t plane = size_t(p.M) * (p.top + p.S) * p.I;
    uint32_t row[RQ];
    int n_load = 0, n_use = 0;  // of the slot that is loaded and of the one that is used
    const auto aim = [&]() {
      const SlotView s(p.slot + slot);
      n_load = s.n;
      const size_t r = size_t(s.expert) * p.K + n0;
      codes = p.w_down + r * row_bytes;
      scales = p.s_down + r * nb;
      h = p.h + size_t(s.begin) * p.I;
#pragma unroll
      for (int q = 0; q < RQ; ++q) row[q] = uint32_t(min(4 * q + g, s.n - 1)) * (p.I * 2);
    };
    const auto load = [&](Unit& b) {
      if (job == end) return;
      load_piece<STEPS, TINY>(b.w, codes, code_row, scales, scale_row, nb, unit, lane & 3);
#pragma unroll
      for (int j = 0; j < STEPS; ++j)
#pragma unroll
        for (int i = 0; i < 3; ++i)
          load_x<RQ>(b.h[i][j], h + i * plane, row, (unit * STEPS + j) * 128, p.I, l16, n_load);
      if (++job < end && ++unit == units) {
        unit = 0;
        ++slot;
        aim();
      }
    };
    f32x4 acc = {};
    const auto use = [&](Unit& b, int unit) {
      stage_piece<STEPS, TINY>(wl, b.w, nb, unit, lane);
      const auto weights = [&](int j, bf16x8(&w)[4]) {
        const float sc = scale_of(scale_operand<STEPS>(wl, j, l16, g));
        const u32x4 c = codes_operand(wl, j, l16, g);
#pragma unroll
        for (int d = 0; d < 4; ++d) w[d] = dequant8(c[d], sc);
      };
      if (RQ == 1) {
        const int r = l16 < 12 ? l16 : l16 - 4;  // (the last four columns are not used)
#pragma unroll
        for (int j = 0; j < STEPS; ++j) {
#pragma unroll
          for (int i = 0; i < 3; ++i)
            stage_x<RQ>(hl, b.h[i][j], (unit * STEPS + j) * 128, p.I, l16, g, n_use, 4 * i);
          wave_lds_fence();
          bf16x8 w[4];
          weights(j, w);
#pragma unroll
          for (int d = 0; d < 4; ++d) acc = mfma32(w[d], x_operand_of(hl, r, d, g), acc);
          wave_lds_fence();
        }
        return;
      }
      bf16x8 w[STEPS][4];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
#pragma unroll
        for (int j = 0; j < STEPS; ++j)
          stage_x<RQ>(hl + j * (RQ * 1024), b.h[i][j], (unit * STEPS + j) * 128, p.I, l16, g, n_use);
        wave_lds_fence();
#pragma unroll
        for (int j = 0; j < STEPS; ++j) {
          if (i == 0) weights(j, w[j]);
#pragma unroll
          for (int d = 0; d < 4; ++d) acc = mfma32(w[j][d], x_operand<RQ>(hl + j * (RQ * 1024), d, l16, g), acc);
        }
        wave_lds_fence();
      }
    };
    int at = first, at_slot = slot0, at_unit = unit;
    const auto step = [&](Unit& b) {
      use(b, at_unit);
      load(b);
      ++at;
      if (++at_unit == units || at == end) {
        const SlotView s(p.slot + at_slot);
        if (RQ == 1) {  // columns t, 4 + t and 8 + t
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] += __shfl_xor(acc[i], 4) + __shfl_xor(acc[i], 8);
        }
        if (l16 < s.n) y[s.token(l16) * 4 + g] += acc;
        wave_lds_fence();
        acc = f32x4{};
        ++at_slot;
        at_unit = 0;
        if (at < end) n_use = scalar(p.slot + at_slot)->n;
      }
    };
    aim();
    n_use = n_load;
#pragma unroll
    for (int u = 0; u < U; ++u) load(buf[u]);
    for (bool more = true; more;) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!more) break;
        step(buf[u]);
        more = at != end;
      }
    }
  }
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(lds + kWaves * kWave);
  if (p.parts > 1) {
    // a part's sums to the workspace; who comes last adds them up, in their order
    for (int i = threadIdx.x; i < p.M * 16; i += 64 * kWaves) {
      float s = all[i];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) s += all[w * p.M * 16 + i];
      put(p.sums + (size_t(part) * p.M + (i >> 4)) * p.K + n0 + (i & 15), s);
    }
    if (!come_last(p.done + blockIdx.x, p.parts)) return;
  }
  for (int i = threadIdx.x; i < p.M * 16; i += 64 * kWaves) {
    const int m = i >> 4;
    if (p.idx && p.idx[m] < 0) continue;
    float s = 0.f;
    if (p.parts > 1) {
      for (int q = 0; q < p.parts; ++q) s += get(p.sums + (size_t(q) * p.M + m) * p.K + n0 + (i & 15));
    } else {
#pragma unroll
      for (int w = 0; w < kWaves; ++w) s += all[w * p.M * 16 + i];
    }
    p.out[m * p.out_row + n0 + (i & 15)] = f32_to_bf16(s);
  }
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

int moe_slots(int M, int E, int S, int top, int chunk) {
  const int pairs = M * top, most = E + pairs / chunk;
  return (pairs < most ? pairs : most) + S * ((M + chunk - 1) / chunk);
}

// Parts of down's sum over slots: two workgroups per compute unit of 256 (a number that is
// known without a device, as the workspace's size has to be), while a part has a unit of k
// for each of its waves.  (Twice the parts, one unit for two waves: one token, 8 of 64
// experts of 1024 x 256, 15.3 us instead of 13.9; 8 + 1 of 128 of 2048 x 512 19.6 / 19.2.)
int moe_parts(int M, int K, int I, int E, int S, int top, int chunk) {
  const int unit = 128 * (chunk == 4 ? kDownSteps4 : kDownSteps16);
  const int tiles = K / 16, units = (I + unit - 1) / unit;
  const int64_t shares = int64_t(moe_slots(M, E, S, top, chunk)) * units / kWaves;
  int parts = 512 / tiles;
  if (parts > shares) parts = int(shares);
  if (parts > kMoeMostParts) parts = kMoeMostParts;
  return parts < 1 ? 1 : parts;
}

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
  const size_t pairs = size_t(M) * (top + S);
  size_t most = 512 / (K / 16);
  if (most > kMoeMostParts) most = kMoeMostParts;
  size_t at = 0;
  const auto part = [&](size_t bytes) {
    const size_t here = at;
    at = up256(at + bytes);
    return here;
  };
  l.head = part(2 * 4);
  l.done = part(size_t(K / 16) * 4);
  l.logits = part(size_t(l.slices) * M * E * 8);
  l.slot = part(size_t(moe_slots(M, E, S, top, 4)) * sizeof(MoeSlot));
  l.pair_gate = part((pairs + 16) * 4);
  l.h = part(pairs * I * 3 * 2);
  l.sums = part(most > 1 ? most * M * K * 4 : 0);
  l.total = at;
  return l;
}

hipError_t launch_moe(const MoeParams& params, int cus, hipStream_t st) {
  MoeParams p = params;
  // Tokens per slot: 4 where an expert has about three at most (of all rows, padding among
  // them: the host knows no better).  us with 4 / 16, all experts as likely: 7168 x 512,
  // 8 + 1 of 256 experts, 16 tokens 160 / 224, 64 tokens 361 / 453; 4096 x 1024, 4 + 1 of
  // 64, 40 tokens 134 / 151; 2048 x 1024, 8 of 128, 32 tokens 110 / 128, 64 tokens 149 /
  // 149; 2080 x 1056, 4 of 40, 21 tokens 67 / 70, 32 tokens 75 / 75, 64 tokens 107 / 91.
  // What has more tokens than a slot is read once for each slot, from the L2 mostly: by
  // workgroups that run at the same time.
  p.chunk = p.M <= 4 || p.M * p.top <= 3 * p.E ? 4 : 16;
  p.parts = moe_parts(p.M, p.K, p.I, p.E, p.S, p.top, p.chunk);
  void* args[] = {&p};
  const auto go = [&](auto* f, dim3 grid, int threads, size_t lds) {
    return hipLaunchKernel(reinterpret_cast<const void*>(f), grid, dim3(threads), args, lds, st);
  };
  hipError_t e = go(&logits_kernel, dim3((p.E + 15) / 16, p.slices, (p.M + 15) / 16), 64 * kRouterWaves, 0);
  if (e != hipSuccess) return e;
  e = go(&route_kernel, dim3(p.M), kRouteThreads, 0);
  if (e != hipSuccess) return e;
  // a power of two of workgroups, about two per compute unit
  const int64_t items = int64_t(moe_slots(p.M, p.E, p.S, p.top, p.chunk)) * (p.I / 16);
  p.up_log2 = 0;
  while ((int64_t(1) << p.up_log2) < items && (2 << p.up_log2) <= 2 * cus) ++p.up_log2;
  const dim3 up(1u << p.up_log2), down(p.K / 16, p.parts);
  const size_t sums = size_t(kWaves) * p.M * 64;
  // Units of 256 of k with 4 tokens a slot: a unit costs about 100 instructions whatever
  // its size, and down of 64 tokens, 7168 x 512, 256 experts, took 139 us with 128 and 111
  // with 256, both with two pieces of h.  One in flight, but two in up, whose items are
  // shorter: registers for other waves fill the time as well as loads ahead do (16 tokens a
  // slot, 64 x 2080 x 1056, 40 experts, two pieces of h: 79 us against 85 with two units;
  // with three pieces two units do not fit in 128 registers).
  if (p.chunk == 4) {
    e = go(p.K < 128 ? &up_kernel<1, 2, 2, true> : &up_kernel<1, 2, 2, false>, up, 64 * kWaves, 0);
    if (e != hipSuccess) return e;
    return go(p.I < 128 ? &down_kernel<1, kDownSteps4, 1, true> : &down_kernel<1, kDownSteps4, 1, false>, down,
              64 * kWaves, sums + kWaves * (kDownH<1, kDownSteps4> + kPieceLds<kDownSteps4>));
  }
  e = go(p.K < 128 ? &up_kernel<4, 1, 1, true> : &up_kernel<4, 1, 1, false>, up, 64 * kWaves, 0);
  if (e != hipSuccess) return e;
  return go(p.I < 128 ? &down_kernel<4, kDownSteps16, 1, true> : &down_kernel<4, kDownSteps16, 1, false>, down,
            64 * kWaves, sums + kWaves * (kDownH<4, kDownSteps16> + kPieceLds<kDownSteps16>));
}

}  // namespace kda
