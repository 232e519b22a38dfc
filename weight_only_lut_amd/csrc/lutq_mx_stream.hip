// MX4 products for few rows: the packed weights stream once past 16 to 64
// rows of activations (gfx950).
//
// y[m][n] = rows[n] * sum_k x[m][k] * (level * relative scale)[n][k]. Bound by
// the weights' bytes, 0.53 per value. A workgroup owns NT tiles of 16 weight
// rows and splits K over its waves: a wave's load is one contiguous 1 KiB
// block of codes, its 64 blocks' scales one byte per lane, and the sums of the
// waves meet in LDS in a fixed order. Everything goes to the matrix cores,
// also at one row: 16 columns cost no more than one there, and the decode
// (16 conversions per KiB and lane) is the same for either.
//
// The experts' modes keep h = silu(g) * u in fp32 (a few KB) and split it into
// two bf16 fragments on the way into the down product, at no cost where bytes
// bound it: of the operator's roundings only the last remains, and h has the
// range of fp32 also in fp16 models.
// Compiled once per activation type (LUTQ_MX_TYPE).
#include <type_traits>

#include "lutq_mx_device.h"

namespace lutq {
namespace {

constexpr int DT = LUTQ_MX_TYPE;


// MODE (see MxMode): dense, up, down and up-pair. For the up modes half of
// the NT tiles are gate rows and half the up rows that meet them.
template <int MODE, int W, int NT, int MT, int U>
__global__ __launch_bounds__(W * 64) void mx_stream_kernel(MxParams p) {
  __shared__ f32x4 red[W][NT * MT][kWave];
  constexpr bool kUp = MODE == kMxUp || MODE == kMxUpPair;
  constexpr bool kDown = MODE == kMxDown;  // x is h
  typedef Mx16<kDown ? kBf16 : DT> T;
  typedef typename T::frag frag;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  int expert = 0, row0 = 0, rows = 0;
  if constexpr (MODE == kMxDense) {
    row0 = blockIdx.y * 16 * MT;
    rows = p.M - row0 < 16 * MT ? p.M - row0 : 16 * MT;
  } else if constexpr (MODE == kMxUpPair) {
    row0 = blockIdx.y;
    rows = 1;
    expert = p.ids[row0];
    if ((unsigned)expert >= (unsigned)p.experts) return;
  } else {
    if ((int)blockIdx.y >= p.tiles[0]) return;
    const int32_t* t = p.tiles + 4 + 4 * blockIdx.y;
    expert = t[0];
    row0 = t[1];
    rows = t[2];
  }
  typedef std::conditional_t<kDown, float, uint16_t> X;
  constexpr int kVec = kDown ? 8 : 4;  // 16-byte loads of a lane's 32 values
  const X* xp[MT];
  bool live[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int m = mt * 16 + r;
    live[mt] = m < rows;
    long long src = row0 + (live[mt] ? m : 0);
    if constexpr (MODE == kMxUp) src = p.order[src] / p.topk;
    if constexpr (MODE == kMxUpPair) src = row0 / p.topk;
    xp[mt] = static_cast<const X*>(p.x) + src * p.ldx + 32 * q;
  }
  const MxWeights& w = p.w;
  const uint8_t* codes = w.codes + expert * w.expert_codes;
  const uint8_t* scales = w.scales + expert * w.expert_scales;
  const float* rowf = w.rows + expert * w.expert_rows;
  int tile[NT];
  const int half = w.ntile / 2;  // up modes: F / 16
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    int t;
    if constexpr (kUp) {
      t = (int)blockIdx.x * (NT / 2) + i % (NT / 2);
      t = (t < half ? t : half - 1) + (i < NT / 2 ? 0 : half);
    } else {
      t = (int)blockIdx.x * NT + i;
      t = t < w.ntile ? t : w.ntile - 1;
    }
    tile[i] = t;
  }
  f32x4 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[i][mt] = f32x4{0, 0, 0, 0};

  const int per = (w.nchunk + W - 1) / W;
  const int c0 = wave * per;
  const int c1 = c0 + per < w.nchunk ? c0 + per : w.nchunk;
  for (int c = c0; c < c1; c += U) {
    u32x4 cd[U][NT];
    uint32_t sc[U][NT];
    u32x4 xf[U][MT][kVec];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int cc = c + u < c1 ? c + u : c1 - 1;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        cd[u][i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(
            codes + ((size_t)tile[i] * w.nchunk + cc) * kMxBlockBytes + lane * kMxSlotBytes));
        sc[u][i] = scales[((size_t)tile[i] * w.nquad + cc / 4) * (kWave * 4) + lane * 4 + cc % 4];
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const bool in = live[mt] && cc * kChunk + 32 * q < w.K;
        const u32x4* src = reinterpret_cast<const u32x4*>(xp[mt] + (size_t)cc * kChunk);
#pragma unroll
        for (int j = 0; j < kVec; ++j) xf[u][mt][j] = in ? src[j] : u32x4{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c + u < c1) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const float s = mx_scale<T::kType>(sc[u][i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const frag a = T::decode(cd[u][i][j], s);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              if constexpr (kDown) {
                frag hi, lo;
                split_bf16(__builtin_bit_cast(f32x4, xf[u][mt][2 * j]),
                           __builtin_bit_cast(f32x4, xf[u][mt][2 * j + 1]), hi, lo);
                acc[i][mt] = T::mfma(a, lo, acc[i][mt]);
                acc[i][mt] = T::mfma(a, hi, acc[i][mt]);
              } else {
                acc[i][mt] = T::mfma(a, __builtin_bit_cast(frag, xf[u][mt][j]), acc[i][mt]);
              }
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) red[wave][i * MT + mt][lane] = acc[i][mt];
  __syncthreads();

  // a slot: four outputs n of one row m
  constexpr int kTiles = kUp ? NT / 2 : NT;
  for (int s = threadIdx.x; s < kTiles * MT * kWave; s += W * 64) {
    const int l = s & 63, im = s >> 6, mt = im % MT, i = im / MT;
    const int m = mt * 16 + (l & 15);
    if (m >= rows) continue;
    f32x4 v = red[0][im][l];
#pragma unroll
    for (int k = 1; k < W; ++k) v += red[k][im][l];
    const int t = (int)blockIdx.x * kTiles + i;
    if (t >= (kUp ? half : w.ntile)) continue;
    const int n = t * 16 + 4 * (l >> 4);
    v *= row_factors(rowf, n, T::kShift);
    if constexpr (kUp) {
      f32x4 u = red[0][im + kTiles * MT][l];
#pragma unroll
      for (int k = 1; k < W; ++k) u += red[k][im + kTiles * MT][l];
      u *= row_factors(rowf, half * 16 + n, T::kShift);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = silu_mul(v[e], u[e]);
      const int F = half * 16;
      store4(static_cast<float*>(p.y) + (size_t)(row0 + m) * F, n, F, v);
    } else if constexpr (MODE == kMxDown) {
      const int pair = p.order[row0 + m];
      v *= p.weights[pair];
      store4(static_cast<float*>(p.y) + (size_t)pair * w.N, n, w.N, v);
    } else {
      store4<DT>(static_cast<uint16_t*>(p.y) + (size_t)(row0 + m) * w.N, n, w.N, v);
    }
  }
}

// The down products of one token's k <= 16 experts and their weighted sum in
// one workgroup per NT tiles: pair j owns column j of the MFMAs, so one
// accumulator holds all the experts' outputs apart, and the waves split the
// k * nchunk blocks of weights between them.
template <int W, int NT, int U>
__global__ __launch_bounds__(W * 64) void mx_down_token_kernel(MxParams p) {
  __shared__ f32x4 red[W][NT][kWave];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int token = blockIdx.y, k = p.topk;
  const MxWeights& w = p.w;
  const int32_t* ids = p.ids + (size_t)token * k;
  typedef Mx16<kBf16> T;
  typedef T::frag frag;
  const float* h = static_cast<const float*>(p.x) + (size_t)token * k * p.ldx + 32 * q;
  int tile[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int t = (int)blockIdx.x * NT + i;
    tile[i] = t < w.ntile ? t : w.ntile - 1;
  }
  f32x4 acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = f32x4{0, 0, 0, 0};
  const int units = k * w.nchunk, per = (units + W - 1) / W;
  const int u0 = wave * per;
  const int u1 = u0 + per < units ? u0 + per : units;
  for (int b = u0; b < u1; b += U) {
    u32x4 cd[U][NT];
    uint32_t sc[U][NT];
    f32x4 xf[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = b + u < u1 ? b + u : u1 - 1;
      const int j = at / w.nchunk, cc = at - j * w.nchunk;
      const int id = ids[j];
      const bool valid = (unsigned)id < (unsigned)p.experts;
      const size_t e = valid ? id : 0;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        cd[u][i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(
            w.codes + e * w.expert_codes + ((size_t)tile[i] * w.nchunk + cc) * kMxBlockBytes +
            lane * kMxSlotBytes));
        sc[u][i] = w.scales[e * w.expert_scales + ((size_t)tile[i] * w.nquad + cc / 4) * (kWave * 4) +
                            lane * 4 + cc % 4];
      }
      // column j alone is not zero; nothing was written to h of an absent pair
      const bool in = r == j && valid && b + u < u1 && cc * kChunk + 32 * q < w.K;
      const f32x4* src = reinterpret_cast<const f32x4*>(h + (size_t)j * p.ldx + (size_t)cc * kChunk);
#pragma unroll
      for (int s = 0; s < 8; ++s) xf[u][s] = in ? src[s] : f32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        frag hi, lo;
        split_bf16(xf[u][2 * j], xf[u][2 * j + 1], hi, lo);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const frag a = T::decode(cd[u][i][j], mx_scale<kBf16>(sc[u][i]));
          acc[i] = T::mfma(a, lo, acc[i]);
          acc[i] = T::mfma(a, hi, acc[i]);
        }
      }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) red[wave][i][lane] = acc[i];
  __syncthreads();
  // lane (q, j): the outputs n = 4q .. 4q + 3 of pair j; the sum over the
  // pairs runs over the 16 lanes of a row in the order of j
  for (int s = threadIdx.x; s < NT * 4; s += W * 64) {
    const int i = s >> 2, qq = s & 3;
    const int t = (int)blockIdx.x * NT + i;
    if (t >= w.ntile) continue;
    const int n = t * 16 + 4 * qq;
    f32x4 sum = {0, 0, 0, 0};
    for (int j = 0; j < k; ++j) {
      const int id = ids[j];
      if ((unsigned)id >= (unsigned)p.experts) continue;
      f32x4 v = red[0][i][qq * 16 + j];
#pragma unroll
      for (int x = 1; x < W; ++x) v += red[x][i][qq * 16 + j];
      v *= row_factors(w.rows + id * w.expert_rows, n, T::kShift);
      sum += v * p.weights[(size_t)token * k + j];
    }
    store4<DT>(static_cast<uint16_t*>(p.y) + (size_t)token * w.N, n, w.N, sum);
  }
}

template <int MODE, int W, int NT, int MT, int U>
hipError_t go(const MxParams& p, hipStream_t s) {
  constexpr bool kUp = MODE == kMxUp || MODE == kMxUpPair;
  const int tiles = kUp ? p.w.ntile / 2 : p.w.ntile, per = kUp ? NT / 2 : NT;
  const dim3 g((unsigned)((tiles + per - 1) / per), 1);
  MxParams q = p;
  // grid.y holds 65535 at most
  if constexpr (MODE == kMxDense) {
    const int step = 65535 * 16 * MT;
    for (int m0 = 0; m0 < p.M; m0 += step) {
      q.M = p.M - m0 < step ? p.M - m0 : step;
      q.x = static_cast<const uint16_t*>(p.x) + (size_t)m0 * p.ldx;
      q.y = static_cast<uint16_t*>(p.y) + (size_t)m0 * p.w.N;
      const unsigned gy = (unsigned)((q.M + 16 * MT - 1) / (16 * MT));
      mx_stream_kernel<MODE, W, NT, MT, U><<<dim3(g.x, gy), W * 64, 0, s>>>(q);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  } else {
    const unsigned gy = MODE == kMxUpPair ? (unsigned)p.pairs : (unsigned)p.max_tiles;
    mx_stream_kernel<MODE, W, NT, MT, U><<<dim3(g.x, gy), W * 64, 0, s>>>(q);
    return hipGetLastError();
  }
}

}  // namespace

template <>
hipError_t mx_stream<DT>(const MxParams& p, int mode, int cus, hipStream_t s) {
  switch (mode) {
    case kMxDense:
      if (p.M <= 16) return go<kMxDense, 8, 1, 1, 4>(p, s);
      if (p.M <= 32) return go<kMxDense, 8, 2, 2, 2>(p, s);
      return go<kMxDense, 8, 2, 4, 1>(p, s);
    case kMxUp: return go<kMxUp, 8, 2, 1, 4>(p, s);
    case kMxDown: return go<kMxDown, 8, 1, 1, 4>(p, s);
    case kMxUpPair: return go<kMxUpPair, 8, 2, 1, 4>(p, s);
    default: {
      const dim3 g((unsigned)p.w.ntile, (unsigned)p.M);
      mx_down_token_kernel<8, 1, 4><<<g, 512, 0, s>>>(p);
      return hipGetLastError();
    }
  }
}

}  // namespace lutq
