// kda_mx4_tile.hip -- products of many rows x with weights, both in microscaled
// 4-bit numbers:  y[m, n] = sum_k x[m, k] w[n, k].
//
// Bound by the scaled 4-bit MFMA (32x32x64: 32 cycles).  A workgroup of four waves
// makes BM x BN outputs, each wave a quarter, from operands in LDS: four stages of
// 128 of k that loads fill directly, three ahead of the one in use, and the scales
// of 512 of k at a time.  A wave of 128 x 128 outputs reads 8 KB of LDS for 16
// MFMAs, 64 of LDS's 128 bytes a cycle with four waves.
//
// LDS holds a row's 64 bytes of a stage as four pieces of 16, at piece ^ (row / 2)
// % 4, so that 8 adjacent rows' pieces are in different banks; a load into LDS
// places lanes in order, so the permutation is made by the addresses that it reads.
//
// The loads are written in assembly: with the builtin the compiler waits for every
// load into LDS before each read of it, which leaves one stage in flight.  Their
// count in flight is waited on by hand (see Stage).
#include "kda_mx4_dev.h"
#include "kda_mx4_internal.h"

namespace kda {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kStages = 4;

// 16 bytes per lane from base + soff + voff to LDS at lds + 16 * lane
__device__ __forceinline__ void load_lds(i32x4 base, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :: "s"(lds), "v"(voff), "s"(base), "s"(soff)
               : "memory");
}
__device__ __forceinline__ i32x4 rsrc_of(const void* p) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  return i32x4{__builtin_amdgcn_readfirstlane(int(uint32_t(a))), __builtin_amdgcn_readfirstlane(int(a >> 32)), -1,
               0x00020000};
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)(p)));
}

template <int BM, int BN>
struct TileLds {
  char code[kStages][(BM + BN) * 64];  // x's rows, then w's
  char scale[2][(BM + BN) * 16];
};

template <int BM, int BN>
__global__ __launch_bounds__(256, 1) void tile_kernel(Mx4Params p) {
  constexpr int FM = BM / 64, FN = BN / 64;          // 32 x 32 tiles of a wave, either way
  constexpr int kLoads = (BM + BN) / 64;             // per wave and stage
  constexpr int kScaleLoads = (BM + BN) / 256;       // per wave and four stages
  __shared__ __align__(16) TileLds<BM, BN> L;
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
  const i32x4 xb = rsrc_of(static_cast<const uint8_t*>(p.x) + size_t(m0) * row_bytes),
              wb = rsrc_of(p.w + size_t(n0) * row_bytes), xsb = rsrc_of(p.xs + size_t(m0) * nb),
              wsb = rsrc_of(p.ws + size_t(n0) * nb);
  const int mlast = int(p.M - 1 - m0 < BM ? p.M - 1 - m0 : BM - 1), nlast = min(p.N - 1 - n0, BN - 1);
  // this lane's source of each load of a stage; rows behind the last repeat it
  uint32_t off[kLoads], soff[kScaleLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = (wave * kLoads + i) * 16 + (lane >> 2);  // row of the stage
    const uint32_t piece = ((lane & 3) ^ (r >> 1)) & 3;
    off[i] = uint32_t(r < BM ? min(r, mlast) : min(r - BM, nlast)) * row_bytes + piece * 16;
  }
#pragma unroll
  for (int i = 0; i < kScaleLoads; ++i) {
    const int r = (wave * kScaleLoads + i) * 64 + lane;
    soff[i] = uint32_t(r < BM ? min(r, mlast) : min(r - BM, nlast)) * nb;
  }
  const int T = p.K / 128;
  const uint32_t code0 = lds_address(L.code[0]), scale0 = lds_address(L.scale[0]);
  // The scales of four stages are 16 bytes a row; the last ones of a row are its last
  // 16 bytes, so that no load passes its end.
  const auto issue = [&](int t) {
    if ((t & 3) == 0) {
#pragma unroll
      for (int i = 0; i < kScaleLoads; ++i) {
        const int c = wave * kScaleLoads + i;
        load_lds(c * 64 < BM ? xsb : wsb, soff[i], min(uint32_t(4 * t), nb - 16),
                 scale0 + ((t >> 2) & 1) * sizeof(L.scale[0]) + c * 1024);
      }
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int c = wave * kLoads + i;
      load_lds(c * 16 < BM ? xb : wb, off[i], t * 64, code0 + (t & 3) * sizeof(L.code[0]) + c * 1024);
    }
  };
  f32x16 acc[FM][FN] = {};
  const int xr = (wave >> 1) * (BM / 2) + l32, wr = BM + (wave & 1) * (BN / 2) + l32;  // rows of the stage
  issue(0);
  if (T > 1) issue(1);
  if (T > 2) issue(2);
  for (int t = 0; t < T; ++t) {
    // stage t is in LDS: the loads of the two stages behind it may be under way; and
    // what this wave read of stage t - 1 has arrived, so that it may be overwritten
    if (t + 2 < T) {
      if (kLoads == 8)
        asm volatile("s_waitcnt vmcnt(16) lgkmcnt(0)" ::: "memory");
      else
        asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)" ::: "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    }
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (t + 3 < T) issue(t + 3);  // into the stage that every wave has left
    const char* code = L.code[t & 3];
    const int sd = 4 * t - int(min(uint32_t(4 * (t & ~3)), nb - 16));  // this stage's scales in the row's 16 bytes
    const char* scale = L.scale[(t >> 2) & 1] + sd;
    uint32_t sx[FM], sw[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) sx[i] = *reinterpret_cast<const uint32_t*>(scale + (xr + 32 * i) * 16) >> (8 * half);
#pragma unroll
    for (int i = 0; i < FN; ++i) sw[i] = *reinterpret_cast<const uint32_t*>(scale + (wr + 32 * i) * 16) >> (8 * half);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      u32x4 a[FN], b[FM];
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const int r = wr + 32 * i;
        a[i] = *reinterpret_cast<const u32x4*>(code + r * 64 + (((2 * s + half) ^ (r >> 1)) & 3) * 16);
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int r = xr + 32 * i;
        b[i] = *reinterpret_cast<const u32x4*>(code + r * 64 + (((2 * s + half) ^ (r >> 1)) & 3) * 16);
      }
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          if (s == 0)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(codes8(a[j]), codes8(b[i]), acc[i][j], 4, 4, 0,
                                                                        int(sw[j]), 0, int(sx[i]));
          else
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(codes8(a[j]), codes8(b[i]), acc[i][j], 4, 4, 2,
                                                                        int(sw[j]), 2, int(sx[i]));
        }
    }
  }
  // y by rows of 16-byte pieces, through LDS: 32 tokens of this wave at a time
  __syncthreads();
  constexpr int kPitch = BN / 2 * 2 + 16;  // bytes
  char* mine = smem + wave * 32 * kPitch;
  const int64_t mw = m0 + (wave >> 1) * (BM / 2);
  const int nw = n0 + (wave & 1) * (BN / 2);
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
    constexpr int kPieces = BN / 16;  // 16-byte pieces of a token
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

template <int BM, int BN>
hipError_t launch(const Mx4Params& p, hipStream_t st) {
  const void* f = reinterpret_cast<const void*>(&tile_kernel<BM, BN>);
  Mx4Params arg = p;
  void* args[] = {&arg};
  const int64_t tiles = ((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
  return hipLaunchKernel(f, dim3(uint32_t(tiles)), dim3(256), args, 0, st);
}

}  // namespace

bool mx4_tile_ok(const Mx4Params& p) {
  return p.K % 128 == 0 && p.K >= 512 && reinterpret_cast<uintptr_t>(p.xs) % 4 == 0 &&
         reinterpret_cast<uintptr_t>(p.ws) % 4 == 0;
}

hipError_t launch_mx4_tile(const Mx4Params& p, int cus, hipStream_t stream) {
  const int64_t big = ((p.M + 255) / 256) * ((p.N + 255) / 256);
  if (2 * big > cus) return launch<256, 256>(p, stream);
  return launch<128, 128>(p, stream);
}

}  // namespace kda
