// MX4 x MX4 products (gfx950): both operands stay in 4 bits with their block
// scales and meet in the scaled matrix instructions, at four times the rate of
// 16-bit ones.
//
// A workgroup computes BM x BN outputs; per step of 256 along K both operand
// tiles lie in LDS as blocks of 16 rows x 128 values, in lane order (lane
// 16q + r: row r, MX block q), so every LDS access is one run of 1 KiB. A
// lane's 32 values share one scale, as the instruction wants it. The packed
// weights have this order already; the activations get it from the addresses
// their loads use.
#include "lutq_mx_device.h"

namespace lutq {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8 widen(u32x4 v) {
  return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

template <int DT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64) void mx_tile4_kernel(MxParams p, int mtiles) {
  constexpr int kWaves = WM * WN;
  constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
  constexpr int kStepChunks = 2;
  constexpr int XB = BM / 16 * kStepChunks / kWaves, WB = BN / 16 * kStepChunks / kWaves;
  __shared__ u32x4 xs[2][BM / 16 * kStepChunks][kWave];
  __shared__ u32x4 ws[2][BN / 16 * kStepChunks][kWave];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int wm = wave % WM, wn = wave / WM;
  const unsigned id = xcd_contiguous(blockIdx.x, gridDim.x);
  const int row0 = (int)(id % mtiles) * BM, nt = (int)(id / mtiles);
  const MxWeights& w = p.w;
  const int kb = w.K / kMxBlock;
  const uint8_t* x = static_cast<const uint8_t*>(p.x);

  // LDS blocks this wave fetches: block b is tile b / 2, chunk b % 2 of the step
  size_t xrow[XB], wtile[WB];
#pragma unroll
  for (int i = 0; i < XB; ++i) {
    const int row = row0 + (wave * XB + i) / kStepChunks * 16 + r;
    xrow[i] = (size_t)(row < p.M ? row : p.M - 1);
  }
#pragma unroll
  for (int i = 0; i < WB; ++i) {
    const int t = nt * (BN / 16) + (wave * WB + i) / kStepChunks;
    wtile[i] = (size_t)(t < w.ntile ? t : w.ntile - 1);
  }
  // and the scales of the tiles it multiplies
  size_t srow[MI];
  uint32_t stile[NI];
#pragma unroll
  for (int m = 0; m < MI; ++m) {
    const int row = row0 + (wm * MI + m) * 16 + r;
    srow[m] = (size_t)(row < p.M ? row : p.M - 1) * kb;
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int t = nt * (BN / 16) + wn * NI + i;
    stile[i] = (uint32_t)(t < w.ntile ? t : w.ntile - 1);
  }

  f32x4 acc[NI][MI];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int m = 0; m < MI; ++m) acc[i][m] = f32x4{0, 0, 0, 0};

  const int steps = (w.nchunk + kStepChunks - 1) / kStepChunks;
  u32x4 xr[XB], wr[WB];
  uint32_t sx[2][MI][kStepChunks], sw[2][NI];
  auto fetch = [&](int s, int stage) {
#pragma unroll
    for (int i = 0; i < XB; ++i) {
      const int b = (s * kStepChunks + (wave * XB + i) % kStepChunks) * 4 + q;
      const u32x4* src = reinterpret_cast<const u32x4*>(x + xrow[i] * p.ldx + (size_t)b * kMxSlotBytes);
      xr[i] = *(b < kb ? src : &mx_zero16);
    }
#pragma unroll
    for (int i = 0; i < WB; ++i) {
      // a chunk past the last: any valid one, the activations are zero there
      int c = s * kStepChunks + (wave * WB + i) % kStepChunks;
      c = c < w.nchunk ? c : w.nchunk - 1;
      wr[i] = *reinterpret_cast<const u32x4*>(w.codes + (wtile[i] * w.nchunk + c) * kMxBlockBytes +
                                              lane * kMxSlotBytes);
    }
#pragma unroll
    for (int m = 0; m < MI; ++m)
#pragma unroll
      for (int c = 0; c < kStepChunks; ++c) {
        const int b = (s * kStepChunks + c) * 4 + q;
        const uint32_t v = p.xscales[srow[m] + (b < kb ? b : kb - 1)];
        sx[stage][m][c] = b < kb ? v : 127u;  // not a NaN of another block
      }
#pragma unroll
    for (int i = 0; i < NI; ++i)
      sw[stage][i] = *reinterpret_cast<const uint16_t*>(
          w.scales + ((size_t)stile[i] * w.nquad + s / 2) * (kWave * 4) + lane * 4 + (s & 1) * 2);
  };
  auto put = [&](int stage) {
#pragma unroll
    for (int i = 0; i < XB; ++i) xs[stage][wave * XB + i][lane] = xr[i];
#pragma unroll
    for (int i = 0; i < WB; ++i) ws[stage][wave * WB + i][lane] = wr[i];
  };
  fetch(0, 0);
  put(0);
  auto step = [&](int s, int stage) {
    __syncthreads();
    const bool more = s + 1 < steps;
    if (more) fetch(s + 1, stage ^ 1);
#pragma unroll
    for (int c = 0; c < kStepChunks; ++c) {
      i32x8 b[MI];
#pragma unroll
      for (int m = 0; m < MI; ++m) b[m] = widen(xs[stage][(wm * MI + m) * kStepChunks + c][lane]);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const i32x8 a = widen(ws[stage][(wn * NI + i) * kStepChunks + c][lane]);
#pragma unroll
        for (int m = 0; m < MI; ++m) {
          if (c == 0)
            acc[i][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                a, b[m], acc[i][m], 4, 4, 0, (int)sw[stage][i], 0, (int)sx[stage][m][c]);
          else
            acc[i][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                a, b[m], acc[i][m], 4, 4, 1, (int)sw[stage][i], 0, (int)sx[stage][m][c]);
        }
      }
    }
    if (more) put(stage ^ 1);
  };
  int s = 0;
  for (; s + 1 < steps; s += 2) {
    step(s, 0);
    step(s + 1, 1);
  }
  if (s < steps) step(s, 0);

#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int t = nt * (BN / 16) + wn * NI + i;
    if (t >= w.ntile) continue;
    const int n = t * 16 + 4 * q;
    const f32x4 f = row_factors(w.rows, n, 0);
#pragma unroll
    for (int m = 0; m < MI; ++m) {
      const int row = row0 + (wm * MI + m) * 16 + r;
      if (row < p.M)
        store4<DT>(static_cast<uint16_t*>(p.y) + (size_t)row * w.N, n, w.N, acc[i][m] * f);
    }
  }
}

template <int DT, int BM, int BN, int WM, int WN>
hipError_t go(const MxParams& p, hipStream_t s) {
  const long long mt = (p.M + BM - 1) / BM, nt = (p.w.ntile + BN / 16 - 1) / (BN / 16);
  if (mt * nt > 0x7FFFFFFF) return hipErrorInvalidValue;
  mx_tile4_kernel<DT, BM, BN, WM, WN><<<dim3((unsigned)(mt * nt)), WM * WN * 64, 0, s>>>(p, (int)mt);
  return hipGetLastError();
}

template <int DT>
hipError_t pick(const MxParams& p, int cus, hipStream_t s) {
  if (p.M <= 64) return go<DT, 64, 128, 2, 4>(p, s);
  return go<DT, 256, 256, 2, 4>(p, s);
}

}  // namespace

hipError_t launch_mx_tile4(const MxParams& p, int dtype, int cus, hipStream_t s) {
  return dtype == kF16 ? pick<kF16>(p, cus, s) : pick<kBf16>(p, cus, s);
}

}  // namespace lutq
