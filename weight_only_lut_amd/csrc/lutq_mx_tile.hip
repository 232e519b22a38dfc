// MX4 products for many rows: tiles of the output through LDS (gfx950).
//
// A workgroup computes BM rows of activations x BN weight rows. Per chunk of
// 128 along K the activations' tile lies in LDS (256 bytes a row, its sixteen
// 16-byte pieces exchanged by the row's low bits so that the 16 rows of a
// fragment read hit all 64 banks once); the weights go from memory to
// registers in 4 bits and are decoded there, since a wave's share is used by
// at most two waves. Both are fetched one chunk ahead.
// Compiled once per activation type (LUTQ_MX_TYPE).
#include "lutq_mx_device.h"

namespace lutq {
namespace {

constexpr int DT = LUTQ_MX_TYPE;
typedef Mx16<DT> T;
typedef T::frag frag;

template <int MODE, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64) void mx_tile_kernel(MxParams p, int mtiles, int ntiles) {
  constexpr bool kUp = MODE == kMxUp;
  constexpr int kThreads = WM * WN * 64;
  constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
  constexpr int kLoads = BM * 16 / kThreads;  // 16-byte pieces per thread and chunk
  __shared__ u32x4 xs[2][BM * 16];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int wm = wave % WM, wn = wave / WM;
  const unsigned id = xcd_contiguous(blockIdx.x, gridDim.x);
  int mt, nt;
  if constexpr (MODE == kMxDense) {
    mt = id % mtiles;
    nt = id / mtiles;
  } else {
    nt = id % ntiles;
    mt = id / ntiles;
  }
  int expert = 0, row0 = mt * BM, rows;
  if constexpr (MODE == kMxDense) {
    rows = p.M - row0 < BM ? p.M - row0 : BM;
  } else {
    if (mt >= p.tiles[0]) return;
    const int32_t* t = p.tiles + 4 + 4 * mt;
    expert = t[0];
    row0 = t[1];
    rows = t[2];
  }
  const MxWeights& w = p.w;

  // this thread's pieces: row and (swizzled) column of piece i * kThreads + tid
  const uint16_t* xp[kLoads];
  const int slot = threadIdx.x & 15;
  int col[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int row = (i * kThreads + (int)threadIdx.x) >> 4;
    long long src = row0 + (row < rows ? row : rows - 1);  // rows past the end are computed, not stored
    if constexpr (kUp) src = p.order[src] / p.topk;
    col[i] = (slot ^ (row & 15)) * 8;
    xp[i] = static_cast<const uint16_t*>(p.x) + src * p.ldx + col[i];
  }
  const uint8_t* codes = w.codes + expert * w.expert_codes;
  const uint8_t* scales = w.scales + expert * w.expert_scales;
  const float* rowf = w.rows + expert * w.expert_rows;
  const int half = w.ntile / 2;
  const int limit = kUp ? half : w.ntile;
  int tile[NI];  // for the up mode the second half of a wave's tiles are the up rows of the first
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    constexpr int kSpan = kUp ? NI / 2 : NI;
    int t = nt * (WN * kSpan) + wn * kSpan + i % kSpan;
    t = t < limit ? t : limit - 1;
    tile[i] = t + (kUp && i >= kSpan ? half : 0);
  }

  f32x4 acc[NI][MI];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int m = 0; m < MI; ++m) acc[i][m] = f32x4{0, 0, 0, 0};

  u32x4 xr[kLoads];
  auto load_x = [&](int c) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const u32x4* src = reinterpret_cast<const u32x4*>(xp[i] + (size_t)c * kChunk);
      xr[i] = *(c * kChunk + col[i] < w.K ? src : &mx_zero16);
    }
  };
  u32x4 cd[2][NI];
  uint32_t sc[2][NI];
  auto load_w = [&](int c, u32x4* d, uint32_t* s) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      d[i] = *reinterpret_cast<const u32x4*>(codes + ((size_t)tile[i] * w.nchunk + c) * kMxBlockBytes +
                                             lane * kMxSlotBytes);
      s[i] = scales[((size_t)tile[i] * w.nquad + c / 4) * (kWave * 4) + lane * 4 + c % 4];
    }
  };
  auto store_x = [&](int stage) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) xs[stage][i * kThreads + threadIdx.x] = xr[i];
  };
  load_x(0);
  load_w(0, cd[0], sc[0]);
  store_x(0);
  const int base = (wm * MI * 16 + r) * 16;
  auto step = [&](int c, int stage) {
    __syncthreads();
    const bool more = c + 1 < w.nchunk;
    if (more) {
      load_x(c + 1);
      load_w(c + 1, cd[stage ^ 1], sc[stage ^ 1]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      frag b[MI];
#pragma unroll
      for (int m = 0; m < MI; ++m)
        b[m] = __builtin_bit_cast(frag, xs[stage][base + m * 256 + ((4 * q + j) ^ r)]);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const frag a = T::decode(cd[stage][i][j], mx_scale<DT>(sc[stage][i]));
#pragma unroll
        for (int m = 0; m < MI; ++m) acc[i][m] = T::mfma(a, b[m], acc[i][m]);
      }
    }
    if (more) store_x(stage ^ 1);
  };
  int c = 0;
  for (; c + 1 < w.nchunk; c += 2) {
    step(c, 0);
    step(c + 1, 1);
  }
  if (c < w.nchunk) step(c, 0);

  constexpr int kOut = kUp ? NI / 2 : NI;
  const int N = kUp ? half * 16 : w.N;
#pragma unroll
  for (int i = 0; i < kOut; ++i) {
    const int t = nt * (WN * kOut) + wn * kOut + i;
    if (t >= limit) continue;
    const int n = t * 16 + 4 * q;
    const f32x4 f = row_factors(rowf, n, T::kShift);
    f32x4 fu = f;
    if constexpr (kUp) fu = row_factors(rowf, half * 16 + n, T::kShift);
#pragma unroll
    for (int m = 0; m < MI; ++m) {
      const int row = (wm * MI + m) * 16 + r;
      if (row >= rows) continue;
      f32x4 v = acc[i][m] * f;
      if constexpr (kUp) {
        const f32x4 u = acc[i + kOut][m] * fu;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = silu_mul(v[e], u[e]);
      }
      if constexpr (MODE == kMxDown) {
        const int pair = p.order[row0 + row];
        v *= p.weights[pair];
        store4(static_cast<float*>(p.y) + (size_t)pair * N, n, N, v);
      } else {
        store4<DT>(static_cast<uint16_t*>(p.y) + (size_t)(row0 + row) * N, n, N, v);
      }
    }
  }
}

template <int MODE, int BM, int BN, int WM, int WN>
hipError_t go(const MxParams& p, hipStream_t s) {
  const int span = (MODE == kMxUp ? BN / 2 : BN) / 16;
  const int tiles = MODE == kMxUp ? p.w.ntile / 2 : p.w.ntile;
  const long long nt = (tiles + span - 1) / span;
  const long long mt = MODE == kMxDense ? (p.M + BM - 1) / BM : p.max_tiles;
  if (nt * mt > 0x7FFFFFFF) return hipErrorInvalidValue;
  mx_tile_kernel<MODE, BM, BN, WM, WN><<<dim3((unsigned)(nt * mt)), WM * WN * 64, 0, s>>>(p, (int)mt, (int)nt);
  return hipGetLastError();
}

}  // namespace

template <>
hipError_t mx_tile<DT>(const MxParams& p, int mode, int cus, hipStream_t s) {
  switch (mode) {
    case kMxDense: return go<kMxDense, 256, 256, 2, 4>(p, s);
    case kMxUp: return go<kMxUp, 128, 256, 2, 4>(p, s);
    default: return go<kMxDown, 128, 256, 2, 4>(p, s);
  }
}

}  // namespace lutq
