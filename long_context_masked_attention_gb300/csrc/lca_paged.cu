// lca_paged.cu — kernels of the paged cache: the batch plan, the writing of
// new keys and values into their pages, and attention over the pages.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "lca_paged.h"
#include "sm103.cuh"

namespace lca {
namespace {

// ------------------------------------------------------------------ batch plan
// Two exclusive sums over the requests (new tokens; pages they need) place
// every row and every fresh page.  What bounds the call is latency, not its
// few bytes, so it is one launch without a second pass: each block runs the
// sums over all requests itself, 1024 at a time, and from each such tile
// writes only its own share of the rows and of the fresh pages (256 at a
// time, round robin), finding a row's request by bisection in shared memory.
constexpr int kPlanThreads = 1024;
constexpr int kPlanShare = 256;

// Inclusive sum over the block of a pair of 64-bit values.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long (*part)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(~0u, a, d), y = __shfl_up_sync(~0u, b, d);
    if (lane >= d) a += x, b += y;
  }
  if (lane == 31) part[warp][0] = a, part[warp][1] = b;
  __syncthreads();
  if (warp == 0) {
    long long x = part[lane][0], y = part[lane][1];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long u = __shfl_up_sync(~0u, x, d), w = __shfl_up_sync(~0u, y, d);
      if (lane >= d) x += u, y += w;
    }
    part[lane][0] = x, part[lane][1] = y;
  }
  __syncthreads();
  if (warp > 0) a += part[warp - 1][0], b += part[warp - 1][1];
}

// Largest s in [0, n) with start[s] <= x.
__device__ __forceinline__ int bisect(const long long* start, int n, long long x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int pages_of(long long tokens, int page_size) {
  return static_cast<int>((tokens + page_size - 1) / page_size);
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PagedPlanArgs a) {
  __shared__ long long part[32][2];
  __shared__ long long row0[kPlanThreads + 1], page0[kPlanThreads + 1];  // exclusive sums of the tile
  __shared__ int ctx_s[kPlanThreads];
  const int tid = threadIdx.x;
  const long long room = static_cast<long long>(a.max_pages) * a.page_size;
  const int taken = min(max(a.taken[0], 0), a.n_free);
  long long rows = 0, pages = 0;  // sums before the tile
  int bad = 0;
  for (int base = 0; base < a.n_seq; base += kPlanThreads) {
    const int n = min(kPlanThreads, a.n_seq - base);
    long long nw = 0, fresh = 0, ctx = 0, want_len = 0;
    int wrong = 0;
    if (tid < n) {
      const int c = a.ctx_len[base + tid], w = a.new_len[base + tid];
      nw = max(w, 0);
      ctx = min(static_cast<long long>(max(c, 0)), room);
      want_len = min(ctx + nw, room);
      wrong = c < 0 || w < 0 || c > room || ctx + nw > room;
      fresh = max(pages_of(want_len, a.page_size) - pages_of(ctx, a.page_size), 0);
    }
    long long ir = nw, ip = fresh;
    block_scan2(ir, ip, part);
    if (tid < n) {
      row0[tid] = rows + ir - nw;
      page0[tid] = pages + ip - fresh;
      ctx_s[tid] = static_cast<int>(ctx);
      if (rows + ir > a.n_rows) wrong = 1;
      if (blockIdx.x == 0) {
        if (base == 0 && tid == 0) a.q_start[0] = 0;
        a.q_start[base + tid + 1] = static_cast<int>(min(rows + ir, static_cast<long long>(a.n_rows)));
        a.k_len[base + tid] = static_cast<int>(want_len);
      }
    }
    if (tid == n - 1) row0[n] = rows + ir, page0[n] = pages + ip;
    bad += __syncthreads_count(wrong);

    // this block's share of the tile's rows
    const long long r_end = min(row0[n], static_cast<long long>(a.n_rows));
    const int sub = tid / kPlanShare, in = tid % kPlanShare;
    constexpr int kSubs = kPlanThreads / kPlanShare;
    const long long step = static_cast<long long>(gridDim.x) * kSubs, me = blockIdx.x * kSubs + sub;
    for (long long s = rows / kPlanShare + (me - rows / kPlanShare % step + step) % step; s * kPlanShare < r_end;
         s += step) {
      const long long r = s * kPlanShare + in;
      if (r < rows || r >= r_end) continue;
      const int i = bisect(row0, n, r);
      const long long pos = ctx_s[i] + (r - row0[i]);
      int slot = -1;
      if (pos < room) {
        const int c = static_cast<int>(pos / a.page_size);
        const int have = pages_of(ctx_s[i], a.page_size);
        int page;
        if (c < have) {
          page = a.block_table[(base + i) * a.table_stride + c];
        } else {
          const long long f = taken + page0[i] + (c - have);
          page = f < a.n_free ? a.free_pages[f] : -1;
        }
        if (page >= 0 && page < a.n_pages) slot = page * a.page_size + static_cast<int>(pos % a.page_size);
      }
      a.slots[r] = slot;
      a.positions[r] = static_cast<int>(min(pos, 0x7FFFFFFFLL));
    }
    // and of its fresh pages
    for (long long s = pages / kPlanShare + (me - pages / kPlanShare % step + step) % step; s * kPlanShare < page0[n];
         s += step) {
      const long long f = s * kPlanShare + in;
      if (f < pages || f >= page0[n]) continue;
      const int i = bisect(page0, n, f);
      const int have = pages_of(ctx_s[i], a.page_size);
      int page = taken + f < a.n_free ? a.free_pages[taken + f] : -1;
      if (page < 0 || page >= a.n_pages) page = -1;
      a.block_table[(base + i) * a.table_stride + have + (f - page0[i])] = page;
    }
    rows = row0[n];
    pages = page0[n];
    __syncthreads();  // the tile's arrays are reused
  }
  // rows behind the last request
  const long long first = min(rows, static_cast<long long>(a.n_rows));
  for (long long r = first + blockIdx.x * static_cast<long long>(kPlanThreads) + tid; r < a.n_rows;
       r += static_cast<long long>(gridDim.x) * kPlanThreads) {
    a.slots[r] = -1;
    a.positions[r] = 0;
  }
  if (blockIdx.x == 0 && tid == 0) {
    if (a.n_seq == 0) a.q_start[0] = 0;
    const long long left = a.n_free - taken;
    a.state[0] = static_cast<int>(taken + min(pages, left));
    a.state[1] = static_cast<int>(min(max(pages - left, 0LL), 0x7FFFFFFFLL));
    a.state[2] = bad;
    a.state[3] = static_cast<int>(first);
  }
}

// ------------------------------------------------------------------ write
// Copies 16-byte pieces: 16 threads per (row, head) for K and V together.
__global__ void __launch_bounds__(256) paged_write_kernel(const PagedWriteArgs a) {
  const long long n = static_cast<long long>(a.n_rows) * a.Hkv * 16;
  for (long long t = blockIdx.x * 256LL + threadIdx.x; t < n; t += gridDim.x * 256LL) {
    const int piece = static_cast<int>(t & 15);
    const long long rh = t >> 4;
    const int head = static_cast<int>(rh % a.Hkv);
    const long long row = rh / a.Hkv;
    const int slot = __ldg(a.slots + row);
    if (slot < 0 || slot >= a.n_slots) continue;
    const uint4 x = a.k[row * a.k_stride + head * 16 + piece], y = a.v[row * a.v_stride + head * 16 + piece];
    const long long at = slot / a.page_size * a.page_stride + slot % a.page_size * a.token_stride +
                         head * a.head_stride + piece;
    a.kc[at] = x;
    a.vc[at] = y;
  }
}

// ------------------------------------------------------------------ attention
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f(__half& y, float x) { y = __float2half_rn(x); }

// Clamps the requests' lengths to what the tensors hold and flags those that
// needed it.
__global__ void paged_seqs_kernel(const PagedAttnArgs a) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= a.n_seq) return;
  const int r0 = a.q_start[i], r1 = a.q_start[i + 1], kl = a.k_len[i];
  const long long room = static_cast<long long>(a.max_pages) * a.page_size;
  PagedSeq s{};
  s.q_off = min(max(r0, 0), a.Tq);
  s.q_len = min(max(r1, s.q_off), a.Tq) - s.q_off;
  s.k_len = static_cast<int>(min(static_cast<long long>(max(kl, 0)), room));
  if (r0 < 0 || r1 < r0 || r1 > a.Tq || kl < 0 || kl > room) raise_status(a.status, kStatusDeviceArg, 50);
  a.seqs[i] = s;
}

// One warp per (row, query head), one key at a time, online softmax in base 2.
template <typename T>
__global__ void __launch_bounds__(256) paged_rows_kernel(const PagedAttnArgs a) {
  const long long w = blockIdx.x * 8LL + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= static_cast<long long>(a.Tq) * a.Hq) return;
  const int head = static_cast<int>(w % a.Hq), row = static_cast<int>(w / a.Hq);
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  int lo = 0, hi = a.n_seq;  // the last request that starts at or before the row
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.seqs[mid].q_off <= row) lo = mid; else hi = mid;
  }
  const PagedSeq sq = a.n_seq > 0 ? a.seqs[lo] : PagedSeq{};
  if (row >= sq.q_off && row < sq.q_off + sq.q_len) {
    SegInfo sg{};
    sg.q_len = sq.q_len;
    sg.k_len = sq.k_len;
    const Span sp = row_span(a.mask, sg, row - sq.q_off);
    const T* q = static_cast<const T*>(a.q) + row * a.q_stride + head * kHeadDim + lane * 4;
    float qf[4];
    for (int k = 0; k < 4; ++k) qf[k] = to_f(q[k]) * a.scale_log2;
    const int j0 = sp.a1 < sp.b1 ? min(sp.a0 < sp.b0 ? sp.a0 : sp.a1, sp.a1) : sp.a0;
    const int j1 = max(sp.a0 < sp.b0 ? sp.b0 : 0, sp.a1 < sp.b1 ? sp.b1 : 0);
    for (int j = j0; j < j1; ++j) {
      if (!((j >= sp.a0 && j < sp.b0) || (j >= sp.a1 && j < sp.b1))) continue;
      const int page = a.table[lo * a.table_stride + j / a.page_size];
      const bool ok = page >= 0 && page < a.n_pages;
      if (!ok && lane == 0) raise_status(a.status, kStatusDeviceArg, 51);
      const long long at = (ok ? page : 0) * a.page_stride + j % a.page_size * a.token_stride +
                           head / a.G * a.head_stride + lane * 4;
      const T *kr = static_cast<const T*>(a.kc) + at, *vr = static_cast<const T*>(a.vc) + at;
      float s = 0.f;
      for (int k = 0; k < 4; ++k) s += ok ? qf[k] * to_f(kr[k]) : 0.f;
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
      const float mn = fmaxf(m, s), f = exp2f(m - mn), p = exp2f(s - mn);
      l = l * f + p;
      for (int k = 0; k < 4; ++k) acc[k] = acc[k] * f + (ok ? p * to_f(vr[k]) : 0.f);
      m = mn;
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  T* o = static_cast<T*>(a.o) + w * kHeadDim + lane * 4;
  for (int k = 0; k < 4; ++k) from_f(o[k], acc[k] * inv);
  if (lane == 0)
    a.lse[static_cast<long long>(head) * a.Tq + row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

void launch_paged_plan(const PagedPlanArgs& a, int num_sms, cudaStream_t st) {
  // a block per 4096 rows: below that, one block's own writes cost less than
  // the sums each further block would repeat
  const int grid = std::max(1, std::min(num_sms, static_cast<int>((static_cast<long long>(a.n_rows) + 4095) / 4096)));
  note_launches(1);
  paged_plan_kernel<<<grid, kPlanThreads, 0, st>>>(a);
}

void launch_paged_write(const PagedWriteArgs& a, int num_sms, cudaStream_t st) {
  const long long n = (static_cast<long long>(a.n_rows) * a.Hkv * 16 + 255) / 256;
  if (n == 0) return;
  note_launches(1);
  paged_write_kernel<<<static_cast<int>(std::min<long long>(n, num_sms * 8LL)), 256, 0, st>>>(a);
}

void launch_paged_attn(const PagedAttnArgs& a, bool fp16, int, cudaStream_t st) {
  if (a.n_seq > 0) {
    note_launches(1);
    paged_seqs_kernel<<<(a.n_seq + 255) / 256, 256, 0, st>>>(a);
  }
  const int grid = static_cast<int>((static_cast<long long>(a.Tq) * a.Hq + 7) / 8);
  note_launches(1);
  if (fp16)
    paged_rows_kernel<__half><<<grid, 256, 0, st>>>(a);
  else
    paged_rows_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
}

}  // namespace lca
