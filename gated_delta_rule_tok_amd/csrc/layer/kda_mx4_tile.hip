// kda_mx4_tile.hip -- products of many rows x with weights, both in microscaled
// 4-bit numbers:  y[m, n] = sum_k x[m, k] w[n, k].
//
// The floor for many rows is the scaled 4-bit MFMA (32x32x64: 32 cycles).  A
// workgroup makes BM x BN outputs from operands in LDS: stages of 128 of k that loads
// fill directly, three or seven ahead of the one in use, and the scales of 512 of k at a
// time.  A wave has the operands of its next half stage on the way while it issues the
// MFMAs of one, over the barrier between stages too.
//
// The loads are written in assembly: with the builtin the compiler waits for every
// load into LDS before each read of it, which leaves one stage in flight.  Their
// count in flight is waited on by hand.
//
// 8192 x 7168 x 7168: 226 us where the same call is repeated, 244 to 274 between other
// kernels, 3.1 to 3.7 PFLOP/s; the MFMAs are busy 42 to 47% of the cycles, at 1.9 GHz (84
// us would do at 2.4 GHz).  896 tiles on 256 units are four rounds
// where 3.5 would do, a round's stores (6 us) overlap nothing, and a stage of 1024 MFMA
// cycles takes about 1600 with a workgroup alone.  Steps: operands read where they are
// used 271 us; read ahead of 16 MFMAs, but with a branch behind them, over which the
// compiler moves all MFMAs, 263; no such branch 241; one add per load's LDS address and
// half of a stage's loads in the next one's time 223; eight waves instead of four the
// same, 6% less on single rounds.
#include <type_traits>

#include "kda_mx4_dev.h"
#include "kda_mx4_internal.h"

namespace kda {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// 16 bytes per lane from base + soff + voff to LDS at lds + more + 16 * lane
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // (m0 is reserved: no variable is ever in it)
__device__ __forceinline__ void load_lds(i32x4 base, uint32_t voff, uint32_t soff, uint32_t lds, uint32_t more) {
  asm volatile("s_add_u32 m0, %0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :: "s"(lds), "v"(voff), "s"(base), "s"(soff), "i"(more)
               : "memory", "scc", "m0");
}
#pragma clang diagnostic pop
// bytes: behind them loads give zeros
__device__ __forceinline__ i32x4 rsrc_of(const void* p, uint64_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  return i32x4{__builtin_amdgcn_readfirstlane(int(uint32_t(a))), __builtin_amdgcn_readfirstlane(int(a >> 32)),
               __builtin_amdgcn_readfirstlane(int(uint32_t(bytes < 0xffffffffu ? bytes : 0xffffffffu))), 0x00020000};
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)(p)));
}

// NS stages of 128 of k; scales of 512 of k for those in flight and the one in use
template <int BM, int BN, int NS>
struct TileLds {
  static constexpr int kScales = NS == 4 ? 2 : 4;
  char code[NS][(BM + BN) * 64];  // x's rows, then w's
  char scale[kScales][(BM + BN) * 16];
};

template <int N>
__device__ __forceinline__ void wait_loads() {  // at most N loads under way, and none from LDS
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"(N) : "memory");
}

// WN: waves along w's rows; two along x's.  DIRECT: each row's scales are at 4-byte
// addresses, and the stages whole.  Otherwise the words around them are loaded, and a
// stage's scales put together from two: 4096 x 4128 x 4096 47 us (50 by
// way of registers, whose wait empties the wave's loads once in four stages).
template <int BM, int BN, int NS, int WN, bool DIRECT>
__global__ __launch_bounds__(128 * WN) void tile_kernel(Mx4Params p) {
  constexpr int kWaves = 2 * WN;
  constexpr int FM = BM / 64, FN = BN / (32 * WN);          // 32 x 32 tiles of a wave, either way
  constexpr int kLoads = (BM + BN) / (16 * kWaves);         // per wave and stage
  constexpr int kScaleLoads = (BM + BN) / (64 * kWaves);    // per wave and four stages
  static_assert(kScaleLoads * 64 * kWaves == BM + BN, "");
  __shared__ __align__(16) TileLds<BM, BN, NS> L;
  char* smem = L.code[0];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l32 = lane & 31, half = lane >> 5;
  // Workgroups go to the 8 XCDs round robin: each XCD takes a run of tiles, and walks
  // it in columns of 8 tiles of x, so that what its workgroups read at a time stays in
  // its L2.
  const int tm = int((p.M + BM - 1) / BM), tn = (p.N + BN - 1) / BN;
  int id = blockIdx.x;
  {
    const int total = tm * tn, per = total / 8, more = total % 8, xcd = id & 7, k = id >> 3;
    id = xcd * per + min(xcd, more) + k;
  }
  const int panel = id / (8 * tn), width = min(8, tm - 8 * panel), in = id - panel * 8 * tn;
  const int64_t m0 = int64_t(8 * panel + in % width) * BM;
  const int n0 = in / width * BN;
  const uint32_t row_bytes = p.K / 2, nb = p.K / kMxBlock;
  const uint64_t m_left = uint64_t(p.M - m0), n_left = uint64_t(p.N - n0);
  const uint8_t *xs = p.xs + size_t(m0) * nb, *ws = p.ws + size_t(n0) * nb;
  // bytes of the first row's scales behind a word's begin (what is read of the words beside
  // an operand's scales is not used)
  const uint32_t x_turn = DIRECT ? 0 : reinterpret_cast<uintptr_t>(xs) & 3,
                 w_turn = DIRECT ? 0 : reinterpret_cast<uintptr_t>(ws) & 3;
  const i32x4 xb = rsrc_of(static_cast<const uint8_t*>(p.x) + size_t(m0) * row_bytes, m_left * row_bytes),
              wb = rsrc_of(p.w + size_t(n0) * row_bytes, n_left * row_bytes),
              xsb = rsrc_of(xs - x_turn, (x_turn + m_left * nb + 3) & ~uint64_t(3)),
              wsb = rsrc_of(ws - w_turn, (w_turn + n_left * nb + 3) & ~uint64_t(3));
  const int mlast = int(p.M - 1 - m0 < BM ? p.M - 1 - m0 : BM - 1), nlast = min(p.N - 1 - n0, BN - 1);
  // this lane's source of each load of a stage; rows behind the last repeat it
  uint32_t off[kLoads], soff[kScaleLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = (wave * kLoads + i) * 16 + (lane >> 2);  // row of the stage
    const uint32_t piece = (lane & 3) ^ bank_turn(r);
    off[i] = uint32_t(r < BM ? min(r, mlast) : min(r - BM, nlast)) * row_bytes + piece * 16;
  }
#pragma unroll
  for (int i = 0; i < kScaleLoads; ++i) {
    const int r = (wave * kScaleLoads + i) * 64 + lane;
    soff[i] = (r < BM ? x_turn + min(r, mlast) * nb : w_turn + min(r - BM, nlast) * nb) & ~3u;
  }
  const int T = (nb + 3) / 4;
  // (a wave's loads are all of x or all of w)
  static_assert(BM == BN, "");
  const i32x4 code_base = wave < kWaves / 2 ? xb : wb, scale_base = wave < kWaves / 2 ? xsb : wsb;
  const uint32_t code0 = lds_address(L.code[0]) + wave * (kLoads * 1024),
                 scale0 = lds_address(L.scale[0]) + wave * (kScaleLoads * 1024);
  // Stages behind the last are loaded too, from where the last one is: a loop without
  // branches whose waits count the same loads every time.
  const auto issue = [&](int t, int i) {
    load_lds(code_base, off[i], min(t, T - 1) * 64, code0 + (t & (NS - 1)) * sizeof(L.code[0]), i * 1024);
  };
  // The scales of four stages are 16 bytes a row (or the words where they begin).
  const auto issue_scales = [&](int t) {
    if ((t & 3) || t > T) return;  // (the word behind a row's last may be wanted)
#pragma unroll
    for (int i = 0; i < kScaleLoads; ++i)
      load_lds(scale_base, soff[i], 4 * t, scale0 + ((t >> 2) & (L.kScales - 1)) * sizeof(L.scale[0]), i * 1024);
  };
  f32x16 acc[FM][FN] = {};
  const int xr = wave / WN * (BM / 2) + l32, wr = BM + wave % WN * (BN / WN) + l32;  // rows of the stage
  struct Frags {
    u32x4 a[FN], b[FM];
  } f[2];
  struct Scales {
    uint32_t x[FM], w[FN];
  } sc, word;
  // fragment i of stage t, half s (0, 1): w's, then x's
  const auto read = [&](Frags& f, int t, int s, int i) {
    const int r = i < FN ? wr + 32 * i : xr + 32 * (i - FN);
    const u32x4 v = *reinterpret_cast<const u32x4*>(L.code[t & (NS - 1)] + r * 64 + ((2 * s + half) ^ bank_turn(r)) * 16);
    if (i < FN)
      f.a[i] = v;
    else
      f.b[i - FN] = v;
  };
  const auto read_scale = [&](Scales& o, int t, int i) {
    const int r = i < FN ? wr + 32 * i : xr + 32 * (i - FN);
    const uint32_t v = *reinterpret_cast<const uint32_t*>(L.scale[(t >> 2) & (L.kScales - 1)] + 4 * (t & 3) + r * 16);
    if (i < FN)
      o.w[i] = v;
    else
      o.x[i - FN] = v;
  };
  // A stage's scales, shifted for this lane's half, from the word that was read last; where
  // the rows are not at word addresses from that and the one before it, with zeros behind
  // the row's end, so that what is read of its codes there counts nothing.
  const uint32_t turn_w = (w_turn + (wr - BM) * nb) & 3, turn_x = (x_turn + xr * nb) & 3;  // (32 rows on the same)
  const uint32_t end_mask = nb & 3 ? (1u << (8 * (nb & 3))) - 1 : ~0u;
  const auto scales_of = [&](const Scales& read, int t) {
    const uint32_t mask = t == T - 1 ? end_mask : ~0u;
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      sc.w[i] = DIRECT ? read.w[i] : __builtin_amdgcn_alignbyte(read.w[i], word.w[i], turn_w) & mask;
      sc.w[i] >>= 8 * half;
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      sc.x[i] = DIRECT ? read.x[i] : __builtin_amdgcn_alignbyte(read.x[i], word.x[i], turn_x) & mask;
      sc.x[i] >>= 8 * half;
    }
    word = read;
  };
  constexpr int kAhead = DIRECT ? 0 : 1;  // the word that completes stage t's scales: t + kAhead
  // The products of one half stage; between(n) is issued behind the n-th of them: a wave
  // alone on its SIMD issues everything else in the MFMAs' time or instead of them.
  const auto multiply = [&](const Frags& f, auto s, const Scales& c, const auto& between) {
    constexpr int kByte = 2 * decltype(s)::value;  // of the shifted scales
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            codes8(f.a[j]), codes8(f.b[i]), acc[i][j], 4, 4, kByte, int(c.w[j]), kByte, int(c.x[i]));
        __builtin_amdgcn_sched_barrier(0);
        between(i * FN + j);
        __builtin_amdgcn_sched_barrier(0);
      }
  };
#pragma unroll
  for (int t = 0; t < NS; ++t) {
    issue_scales(t);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (t + 1 < NS || i < kLoads - kLoads / 2) issue(t, i);  // (the rest comes in the loop)
  }
  wait_loads<(NS - 2) * kLoads>();  // the first stage
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  constexpr int kReads = FN + FM, kSlots = FM * FN;  // fragments of a half stage; MFMAs
#pragma unroll
  for (int i = 0; i < kReads; ++i) {
    read(f[0], 0, 0, i);
    if (!DIRECT) read_scale(word, 0, i);
  }
  Scales next;
#pragma unroll
  for (int i = 0; i < kReads; ++i) read_scale(next, kAhead, i);
  scales_of(next, 0);
  // Reads in the first half of a half stage's MFMAs, loads in the second half: those of
  // stage t + NS where stage t's last read is done, the rest in front of the next wait.
  constexpr int kEach = (2 * kReads + kSlots - 1) / kSlots, kLoadsEach = (kLoads + kSlots - 1) / kSlots;
  constexpr int kLate = kLoads / 2;  // of a stage's loads, in the next one's time
  for (int t = 0; t < T; ++t) {
    // (the one branch, in front: the compiler moves MFMAs behind one, all at once)
    issue_scales(t + NS);
    multiply(f[0], std::integral_constant<int, 0>{}, sc, [&](int n) {
#pragma unroll
      for (int i = n * kEach; i < (n + 1) * kEach && i < kReads; ++i) read(f[1], t, 1, i);
#pragma unroll
      for (int i = (n - kSlots / 2) * kLoadsEach; i < (n - kSlots / 2 + 1) * kLoadsEach; ++i)
        if (i >= 0 && i < kLate) issue(t + NS - 1, kLoads - kLate + i);
    });
    // stage t + 1 is in LDS (those behind it may be under way), and every wave has read
    // all of stage t, which the loads may overwrite
    wait_loads<(NS - 2) * kLoads>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    multiply(f[1], std::integral_constant<int, 1>{}, sc, [&](int n) {
#pragma unroll
      for (int i = n * kEach; i < (n + 1) * kEach && i < kReads; ++i) {
        read(f[0], t + 1, 0, i);
        read_scale(next, t + 1 + kAhead, i);
      }
#pragma unroll
      for (int i = (n - kSlots / 2) * kLoadsEach; i < (n - kSlots / 2 + 1) * kLoadsEach; ++i)
        if (i >= 0 && i < kLoads - kLate) issue(t + NS, i);
    });
    scales_of(next, t + 1);
  }
  wait_loads<0>();
  // y by rows of 16-byte pieces, through LDS: 32 tokens of this wave at a time
  __syncthreads();
  constexpr int kPitch = BN / WN * 2 + 16;  // bytes
  char* mine = smem + wave * 32 * kPitch;
  const int64_t mw = m0 + wave / WN * (BM / 2);
  const int nw = n0 + wave % WN * (BN / WN);
  const bool vec = p.y_row % 8 == 0 && reinterpret_cast<uintptr_t>(p.y) % 16 == 0;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // rows (of w) 8 q + 4 half .. + 3 of this lane's token
        const f32x4 v{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        *reinterpret_cast<bf16x4*>(mine + l32 * kPitch + (32 * j + 8 * q + 4 * half) * 2) = to_bf16x4(v);
      }
    wave_lds_fence();
    constexpr int kPieces = BN / WN / 8;  // 16-byte pieces of a token
#pragma unroll
    for (int q = 0; q < 32 * kPieces / 64; ++q) {
      const int at = q * 64 + lane, r = at / kPieces, c = at % kPieces;
      const int64_t m = mw + 32 * i + r;
      const int n = nw + 8 * c;
      const u32x4 v = *reinterpret_cast<const u32x4*>(mine + r * kPitch + c * 16);
      if (m >= p.M || n >= p.N) continue;
      uint16_t* y = p.y + m * p.y_row + n;
      if (vec && n + 8 <= p.N) {
        *reinterpret_cast<u32x4*>(y) = v;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (n + e < p.N) y[e] = uint16_t(v[e / 2] >> (16 * (e & 1)));
      }
    }
    wave_lds_fence();
  }
}

template <int BM, int BN, int NS, int WN>
hipError_t launch(const Mx4Params& p, hipStream_t st) {
  const auto at = [](const void* q) { return reinterpret_cast<uintptr_t>(q); };
  const bool direct = p.K % 128 == 0 && at(p.xs) % 4 == 0 && at(p.ws) % 4 == 0;
  const void* f = direct ? reinterpret_cast<const void*>(&tile_kernel<BM, BN, NS, WN, true>)
                         : reinterpret_cast<const void*>(&tile_kernel<BM, BN, NS, WN, false>);
  Mx4Params arg = p;
  void* args[] = {&arg};
  const int64_t tiles = ((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
  return hipLaunchKernel(f, dim3(uint32_t(tiles)), dim3(128 * WN), args, 0, st);
}

}  // namespace

static int64_t tiles_of(const Mx4Params& p, int side) {
  return ((p.M + side - 1) / side) * ((p.N + side - 1) / side);
}

// Tiles of 64 x 64 and more against the streaming form (us, 64 x 64 / streaming): where
// they are half the compute units and more, 128 x 2048 x 4096 5.8 / 6.0, 64 x 7168 x 8200
// 18.8 / 20.4, 64 x 7168 x 14336 20 / 29, 300 x 4128 x 2050 11.3 / 16.3, 512 x 7168 x 1536
// 13.2 / 15.2, but 128 x 7168 x 1536 (48 tiles) 13.1 / 6.9, 64 x 7168 x 7168 (112) 18.6 /
// 16.7; with 32 tokens and fewer half a tile's work is for nothing: 32 x 7168 x 8200 15.4 /
// 14.8, 20 x 2080 x 12000 9.3 / 8.2.
bool mx4_in_tiles(const Mx4Params& p, int cus) { return p.M > 32 && 2 * tiles_of(p, 64) >= cus; }

// The side of a tile (us, 64 / 128 / 256): the smallest that two workgroups a compute unit
// (of 64), one (of 128) hold at once: a stage's round trip counts, not its MFMAs.  512 x
// 2048 x 2048 5.9 / 8.0 / 14.7, 256 x 7168 x 7168 18.6 / 21.6 / 42, 1024 x 7168 x 1536 15.7 /
// 22.4; 300 x 2080 x 8200 18.4 / 10.1 / 17.7, 512 x 7168 x 7168 35 / 24.8 / 43; 1024 x 7168 x
// 7168 - / 46 / 44, 2048 x 2048 x 7168 - / 33 / 22.
hipError_t launch_mx4_tile(const Mx4Params& p, int cus, hipStream_t stream) {
  if (tiles_of(p, 64) <= 2 * cus) return launch<64, 64, 8, 1>(p, stream);
  if (tiles_of(p, 128) <= cus) return launch<128, 128, 8, 2>(p, stream);
  return launch<256, 256, 4, 4>(p, stream);
}

}  // namespace kda
