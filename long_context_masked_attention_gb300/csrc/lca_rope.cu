// lca_rope.cu — rotary positions: rows of query and key heads whose pairs of
// values are turned by an angle that grows with the token's position, and the
// gradients turned back; entry points and kernel.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/lca_attn.h"
#include "lca_host.h"
#include "lca_paged.cuh"

namespace lca {
namespace {

constexpr int kPairs = kHeadDim / 2;
constexpr int kThreads = 256;

struct RopeArgs {
  const uint16_t* x[2];  // queries, keys
  uint16_t* y[2];
  long long x_stride[2], y_stride[2];
  int heads[2];
  const int* positions;
  long long items;  // rows x chunks x parts
  int chunks, per;  // of a row's heads, and heads in each
  int pairs;        // that turn
  bool in_place[2];
  float scale;
  uint64_t turns[kPairs];  // a pair's turns per position, modulo 1, times 2^64
};

template <int N>
struct Bits;
template <>
struct Bits<8> {
  using V = uint4;
};
template <>
struct Bits<4> {
  using V = uint2;
};
template <>
struct Bits<2> {
  using V = uint32_t;
};
template <>
struct Bits<1> {
  using V = uint16_t;
};

template <typename T>
__device__ __forceinline__ float to_float(uint16_t x) {
  return static_cast<float>(*reinterpret_cast<const T*>(&x));
}
template <typename T>
__device__ __forceinline__ uint16_t to_bits(float x) {
  const T y = static_cast<T>(x);
  return *reinterpret_cast<const uint16_t*>(&y);
}

// Turns the pairs of every head of a row, y = scale (a cos - b sin, b cos + a
// sin); one reading and one writing of the rows, which bounds it.
//
// The angle is position x frequency, and only its fraction of a turn matters.
// In 32 bits a position of 2^19 leaves 2^-5 of the fastest pair's angle; here
// the frequency is turns x 2^64 modulo 2^64, the product wraps as whole turns do,
// and its upper 32 bits are the fraction exactly to 2^-32 of a turn.  cos and
// sin of it are 32-bit ones.
//
// A warp has one row's heads, or a chunk of them: each lane finds two pairs' cos
// and sin, once for all heads, and the lanes pass them on.  A lane
// then has one unit of every (32 / lanes of a head)-th head: kVec values and
// the kVec that they pair with, and the loads of four heads are under way at once.
//  * half layout: pairs (i, i + r/2), units of 8, 4, 2 or 1 values as r/2
//    allows, so that no unit is partly turned; what lies behind r is halved into
//    units of the same kind, which are copied.
//  * interleaved: pairs (2i, 2i + 1) are 32-bit words, a unit is the words of two
//    16-byte pieces, and each word is turned or kept.
// With kVec = 1 a head has 64 units, two parts of 32 lanes.
//
// Measured: 32K rows of 64 + 8 heads 183 us (6.6 TB/s read and written, 0.97 of a
// copy's rate), 8K rows of 24 + 8 heads, 64 of 128 values turned, 22.8 us (5.9 TB/s,
// start and end counted), 64 rows 3.3 us, which is a launch.
template <typename T, int kVec, bool kInter>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  using V = typename Bits<kVec>::V;
  constexpr int kUnits = kPairs / kVec;                  // of a head
  constexpr int kLanes = kUnits < 32 ? kUnits : 32;      // for a head
  constexpr int kParts = kUnits / kLanes, kStep = 32 / kLanes, kAtOnce = 4;
  const int lane = threadIdx.x & 31;
  const long long warps = gridDim.x * static_cast<long long>(kThreads / 32);
  for (long long it = blockIdx.x * static_cast<long long>(kThreads / 32) + (threadIdx.x >> 5); it < a.items; it += warps) {
    const int part = kParts > 1 ? static_cast<int>(it % kParts) : 0;
    const long long rc = kParts > 1 ? it / kParts : it;
    const long long row = rc / a.chunks;
    const int chunk = static_cast<int>(rc - row * a.chunks);
    // two pairs' cos and sin
    const long long pos = a.positions[row];
    float c2[2] = {1.f, 1.f}, s2[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (2 * lane + k < a.pairs) {
        const uint64_t turn = static_cast<uint64_t>(pos) * a.turns[2 * lane + k];
        sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &s2[k], &c2[k]);
        c2[k] *= fabsf(a.scale);
        s2[k] *= a.scale;  // negative: turned back
      }
    const int unit = lane % kLanes + 32 * part;
    const bool turned = kInter || unit < a.pairs / kVec;
    float c[kVec], s[kVec];
    bool own[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int p = kInter ? 4 * unit + (j & 3) + 32 * (j >> 2) : min(unit * kVec + j, kPairs - 1);
      own[j] = p < a.pairs;
      const float c0 = __shfl_sync(~0u, c2[0], p >> 1), c1 = __shfl_sync(~0u, c2[1], p >> 1);
      const float s0 = __shfl_sync(~0u, s2[0], p >> 1), s1 = __shfl_sync(~0u, s2[1], p >> 1);
      c[j] = (p & 1) ? c1 : c0;
      s[j] = (p & 1) ? s1 : s0;
    }
    int lo, hi;  // the unit's two places in a head
    if (kInter) {
      lo = 8 * unit, hi = 64 + 8 * unit;
    } else if (turned) {
      lo = kVec * unit, hi = a.pairs + kVec * unit;
    } else {
      lo = a.pairs + kVec * unit, hi = kPairs + kVec * unit;  // 2 pairs + (kVec unit - pairs), and 64 - pairs more
    }
    const int h0 = chunk * a.per + lane / kLanes, h1 = min((chunk + 1) * a.per, a.heads[0] + a.heads[1]);
    for (int h = h0; h < h1; h += kStep * kAtOnce) {
      V x[kAtOnce], z[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int head = h + u * kStep;
        if (head < h1) {
          const int w = head >= a.heads[0];
          const uint16_t* src = a.x[w] + row * a.x_stride[w] + (head - (w ? a.heads[0] : 0)) * kHeadDim;
          x[u] = *reinterpret_cast<const V*>(src + lo);
          z[u] = *reinterpret_cast<const V*>(src + hi);
        }
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int head = h + u * kStep;
        if (head >= h1) continue;
        const int w = head >= a.heads[0];
        if (!turned && a.in_place[w]) continue;
        alignas(16) uint16_t p[kVec], q[kVec];
        *reinterpret_cast<V*>(p) = x[u];
        *reinterpret_cast<V*>(q) = z[u];
        if (turned) {
#pragma unroll
          for (int j = 0; j < kVec; ++j) {
            uint16_t& first = kInter ? (j < 4 ? p : q)[2 * (j & 3)] : p[j];
            uint16_t& second = kInter ? (j < 4 ? p : q)[2 * (j & 3) + 1] : q[j];
            const float f = to_float<T>(first), g = to_float<T>(second);
            const uint16_t r0 = to_bits<T>(fmaf(c[j], f, -s[j] * g)), r1 = to_bits<T>(fmaf(c[j], g, s[j] * f));
            if (!kInter || own[j]) first = r0, second = r1;
          }
        }
        uint16_t* dst = a.y[w] + row * a.y_stride[w] + (head - (w ? a.heads[0] : 0)) * kHeadDim;
        *reinterpret_cast<V*>(dst + lo) = *reinterpret_cast<const V*>(p);
        *reinterpret_cast<V*>(dst + hi) = *reinterpret_cast<const V*>(q);
      }
    }
  }
}

template <typename T>
void launch(const RopeArgs& a, int vec, bool inter, int grid, cudaStream_t st) {
  if (inter)
    rope_kernel<T, 8, true><<<grid, kThreads, 0, st>>>(a);
  else if (vec == 8)
    rope_kernel<T, 8, false><<<grid, kThreads, 0, st>>>(a);
  else if (vec == 4)
    rope_kernel<T, 4, false><<<grid, kThreads, 0, st>>>(a);
  else if (vec == 2)
    rope_kernel<T, 2, false><<<grid, kThreads, 0, st>>>(a);
  else
    rope_kernel<T, 1, false><<<grid, kThreads, 0, st>>>(a);
}

constexpr double kMostFrequency = 1048576.0;  // radians per position
constexpr long long kMostStride = 1LL << 38;
constexpr int kMostHeads = 0xFFFFFF;  // a row's elements stay in 32 bits

// Turns per position modulo 1 as a 64-bit fraction: w / (2 pi) in twice the
// 53 bits of a double, since a position multiplies what is lost by up to 2^31.
uint64_t turns_of(double w) {
  const double hi = 0.15915494309189535, lo = -9.839338337591243e-18;  // 1 / (2 pi)
  const double p = w * hi, e = std::fma(w, hi, -p) + w * lo;
  constexpr double k64 = 18446744073709551616.0;  // 2^64
  const double whole = static_cast<double>(static_cast<int64_t>(p));  // p is below 2^18
  return static_cast<uint64_t>((p - whole) * k64) + static_cast<uint64_t>(static_cast<int64_t>(e * k64));
}

// Bytes from the first element of the rows to the last.
long long extent(int n, long long stride, int heads) {
  return n == 0 || heads == 0 ? 0 : ((n - 1) * stride + static_cast<long long>(heads) * kHeadDim) * 2;
}

bool rows_ok(const lca_rope_rows* r, int n_rows) {
  if (r->heads < 0) return false;
  if (r->heads == 0) return true;
  const long long row = static_cast<long long>(r->heads) * kHeadDim;
  for (const int64_t s : {r->x_stride, r->y_stride})
    if (s < row || s % 8 != 0 || s > kMostStride || (n_rows > 1 && static_cast<double>(n_rows - 1) * s > 1e15)) return false;
  return true;
}

bool rows_memory(const lca_rope_rows* r) {
  if (r->heads == 0) return true;
  return r->x && r->y && aligned16(r->x) && aligned16(r->y) && device_input(r->x) && device_input(r->y);
}

}  // namespace
}  // namespace lca

using namespace lca;

extern "C" {

lca_status lca_rope_frequencies(const lca_rope_table* t, double* inv_freq, float* scale) {
  if (!t || !inv_freq || !scale) return LCA_ERR_INVALID_ARG;
  const int r = t->rot_dim;
  if (r < 2 || r % 2 != 0 || r > kHeadDim) return LCA_ERR_INVALID_ARG;
  if (!(t->base > 1.0) || !std::isfinite(t->base) || !(t->factor >= 1.0) || !std::isfinite(t->factor))
    return LCA_ERR_INVALID_ARG;
  const bool bands = t->scaling == LCA_ROPE_YARN || t->scaling == LCA_ROPE_BANDS;
  if (t->scaling < LCA_ROPE_PLAIN || t->scaling > LCA_ROPE_BANDS) return LCA_ERR_INVALID_ARG;
  if (bands && (t->original_len < 1 || !(t->slow > 0.0) || !(t->fast > t->slow) || !std::isfinite(t->fast)))
    return LCA_ERR_INVALID_ARG;
  if (t->scaling == LCA_ROPE_NTK && r == 2) return LCA_ERR_INVALID_ARG;  // its exponent is r / (r - 2)
  constexpr double kTwoPi = 6.283185307179586;
  const double base = t->scaling == LCA_ROPE_NTK ? t->base * std::pow(t->factor, r / (r - 2.0)) : t->base;
  if (!std::isfinite(base)) return LCA_ERR_INVALID_ARG;
  double low = 0, high = 0;  // YARN: pairs that make `fast` and `slow` turns in original_len positions
  if (t->scaling == LCA_ROPE_YARN) {
    auto pair_of = [&](double n) { return r * std::log(t->original_len / (n * kTwoPi)) / (2 * std::log(t->base)); };
    low = std::max(std::floor(pair_of(t->fast)), 0.0);
    high = std::min(std::ceil(pair_of(t->slow)), r - 1.0);
  }
  for (int i = 0; i < r / 2; ++i) {
    const double w = std::pow(base, -2.0 * i / r);
    double keep = 1.0;  // of the unscaled frequency
    if (t->scaling == LCA_ROPE_LINEAR) keep = 0.0;
    if (t->scaling == LCA_ROPE_YARN) keep = 1.0 - std::min(std::max((i - low) / std::max(high - low, 1e-3), 0.0), 1.0);
    if (t->scaling == LCA_ROPE_BANDS)
      keep = std::min(std::max((t->original_len * w / kTwoPi - t->slow) / (t->fast - t->slow), 0.0), 1.0);
    inv_freq[i] = w * keep + w / t->factor * (1.0 - keep);
  }
  *scale = t->scaling == LCA_ROPE_YARN ? static_cast<float>(0.1 * std::log(t->factor) + 1.0) : 1.0f;
  return LCA_OK;
}

lca_status lca_rope(const lca_rope_rows* q, const lca_rope_rows* k, const int32_t* positions, int32_t n_rows, int32_t d,
                    int32_t dtype, const lca_rope_desc* rope, int32_t back, void* stream) {
  const lca_rope_rows none{};
  if (!q) q = &none;
  if (!k) k = &none;
  if (!rope || n_rows < 0 || (dtype != LCA_BF16 && dtype != LCA_F16)) return LCA_ERR_INVALID_ARG;
  if (d != kHeadDim) return LCA_ERR_UNSUPPORTED;
  const int r = rope->rot_dim;
  if (r < 2 || r % 2 != 0 || r > kHeadDim || !rope->inv_freq) return LCA_ERR_INVALID_ARG;
  if (!std::isfinite(rope->scale) || rope->scale < 0.f) return LCA_ERR_INVALID_ARG;
  for (int i = 0; i < r / 2; ++i)
    if (!(rope->inv_freq[i] >= 0.0 && rope->inv_freq[i] <= kMostFrequency)) return LCA_ERR_INVALID_ARG;
  if (!rows_ok(q, n_rows) || !rows_ok(k, n_rows)) return LCA_ERR_INVALID_ARG;
  if (static_cast<long long>(q->heads) + k->heads > kMostHeads) return LCA_ERR_UNSUPPORTED;
  const int heads = q->heads + k->heads;
  if (n_rows == 0 || heads == 0) return LCA_OK;
  if (!rows_memory(q) || !rows_memory(k) || !positions || (reinterpret_cast<uintptr_t>(positions) & 3u) != 0 ||
      !device_input(positions))
    return LCA_ERR_INVALID_ARG;
  {  // rows written must not be rows that others are read from; a part's own rows may be written in place
    const lca_rope_rows* t[2] = {q, k};
    auto apart = [](const void* x, long long nx, const void* y, long long ny) {
      const auto a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
      return nx == 0 || ny == 0 || a + static_cast<uintptr_t>(nx) <= b || b + static_cast<uintptr_t>(ny) <= a;
    };
    // rows of one stride that leave room for each other's (parts of one wider row) do not meet
    auto woven = [&](const void* x, int hx, long long sx, const void* y, int hy, long long sy) {
      if (sx != sy || n_rows < 2) return false;
      const auto a = static_cast<long long>(reinterpret_cast<uintptr_t>(x)), b = static_cast<long long>(reinterpret_cast<uintptr_t>(y));
      const long long step = 2 * sx, off = ((b - a) % step + step) % step;  // y's row after x's
      return off >= 256LL * hx && off + 256LL * hy <= step;
    };
    for (int i = 0; i < 2; ++i) {
      if (t[i]->heads == 0) continue;
      if (!apart(t[i]->y, extent(n_rows, t[i]->y_stride, t[i]->heads), positions, 4LL * n_rows)) return LCA_ERR_INVALID_ARG;
      for (int j = 0; j < 2; ++j) {
        if (t[j]->heads == 0) continue;
        const long long ny = extent(n_rows, t[i]->y_stride, t[i]->heads);
        const bool same = i == j && t[i]->x == t[i]->y && (t[i]->x_stride == t[i]->y_stride || n_rows == 1);
        if (!same && !apart(t[i]->y, ny, t[j]->x, extent(n_rows, t[j]->x_stride, t[j]->heads)) &&
            !woven(t[i]->y, t[i]->heads, t[i]->y_stride, t[j]->x, t[j]->heads, t[j]->x_stride))
          return LCA_ERR_INVALID_ARG;
        if (i < j && !apart(t[i]->y, ny, t[j]->y, extent(n_rows, t[j]->y_stride, t[j]->heads)) &&
            !woven(t[i]->y, t[i]->heads, t[i]->y_stride, t[j]->y, t[j]->heads, t[j]->y_stride))
          return LCA_ERR_INVALID_ARG;
      }
    }
  }
  const int sms = num_sms();
  if (sms <= 0) return LCA_ERR_CUDA;
  RopeArgs a{};
  const lca_rope_rows* t[2] = {q, k};
  for (int w = 0; w < 2; ++w) {
    a.x[w] = static_cast<const uint16_t*>(t[w]->x);
    a.y[w] = static_cast<uint16_t*>(t[w]->y);
    a.x_stride[w] = t[w]->x_stride;
    a.y_stride[w] = t[w]->y_stride;
    a.heads[w] = t[w]->heads;
    a.in_place[w] = t[w]->x == t[w]->y;
  }
  a.positions = positions;
  a.pairs = r / 2;
  const float scale = rope->scale > 0.f ? rope->scale : 1.f;
  a.scale = back ? -scale : scale;
  for (int i = 0; i < a.pairs; ++i) a.turns[i] = turns_of(rope->inv_freq[i]);
  const bool inter = rope->interleaved != 0;
  int vec = 8;
  if (!inter)
    while (a.pairs % vec != 0) vec /= 2;
  const int lanes = std::min(kPairs / vec, 32), parts = kPairs / vec / lanes, step = 32 / lanes;
  // a warp takes all heads of a row where there are rows enough to fill the
  // GPU with warps, so that cos and sin are found once; few rows are cut up
  const long long want = cdiv(32LL * sms, static_cast<long long>(n_rows) * parts);
  const int chunks = static_cast<int>(std::min<long long>(want, cdiv(heads, step)));
  a.per = static_cast<int>(cdiv(cdiv(heads, chunks), step) * step);
  a.chunks = static_cast<int>(cdiv(heads, a.per));
  a.items = static_cast<long long>(n_rows) * a.chunks * parts;
  const int grid = static_cast<int>(std::min<long long>(cdiv(a.items, kThreads / 32), sms * 8LL));
  note_launches(1);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == LCA_F16)
    launch<__half>(a, vec, inter, grid, st);
  else
    launch<__nv_bfloat16>(a, vec, inter, grid, st);
  LCA_CUDA(cudaGetLastError());
  return LCA_OK;
}

}  // extern "C"
