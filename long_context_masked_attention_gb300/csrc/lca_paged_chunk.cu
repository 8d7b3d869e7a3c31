// lca_paged_chunk.cu — attention of many rows over a 16-bit paged cache
// (lca_paged_chunk.cuh), the first kernel of every call of attention over a
// paged cache, and the join of divided items.
#include "lca_paged_chunk.cuh"

namespace lca {
namespace {

// Sums over the requests and their row blocks: block0[i] = row blocks of the
// requests before i, line[b] = key tiles of the row blocks before b (one head;
// at least one per block, so that rows without keys are written) and
// kItemCost more for each block.
__device__ void place_items(const PagedAttnArgs& a) {
  __shared__ long long part[32];
  const int tid = threadIdx.x;
  long long at = 0;
  for (int base = 0; base < a.n_seq; base += 1024) {
    const int i = base + tid;
    const long long n = i < a.n_seq ? row_blocks(a, paged_seg(a, i).q_len) : 0;
    long long total;
    const long long inc = block_scan(n, part, total);
    // rows that overlap (a bad q_start) can make more blocks than there is room for
    if (i < a.n_seq) a.block0[i] = static_cast<int>(min(at + inc - n, static_cast<long long>(a.max_blocks)));
    at += total;
  }
  const int blocks = static_cast<int>(min(at, static_cast<long long>(a.max_blocks)));
  if (tid == 0) a.block0[a.n_seq] = blocks;
  __syncthreads();
  at = 0;
  for (int base = 0; base < blocks; base += 1024) {
    const int b = base + tid;
    long long n = 0;
    if (b < blocks) {
      int i = 0;  // the last request whose blocks start at or before b
      for (int hi = a.n_seq; hi - i > 1;) {
        const int mid = (i + hi) >> 1;
        if (a.block0[mid] <= b) i = mid; else hi = mid;
      }
      const SegInfo sg = paged_seg(a, i);
      const int tok = (b - a.block0[i]) * 2 * a.tpt;
      if (tok < sg.q_len) {
        const Tiles t = tiles_of(hull(a, sg.q_len, sg.k_len, tok, min(tok + 2 * a.tpt, sg.q_len)));
        n = max(t.n0 + t.n1, 1) + kItemCost;
      }
    }
    long long total;
    const long long inc = block_scan(n, part, total);
    if (b < blocks) a.line[b] = at + inc - n;
    at += total;
  }
  if (tid == 0) a.line[blocks] = at;
}

// First kernel of a call: clears the status and the counts, reports lengths
// that the tensors do not hold, and places the items of many rows.
__global__ void __launch_bounds__(1024) paged_begin_kernel(const __grid_constant__ PagedAttnArgs a, bool many) {
  launch_dependents();
  for (int i = threadIdx.x; i <= kPagedMaxSpans; i += 1024) a.arrived[i] = 0;  // and the claims behind them
  if (many && threadIdx.x < kPagedMaxChunkCtas) a.cuts[threadIdx.x].last = -1;
  if (threadIdx.x < 4) a.status[threadIdx.x] = 0;
  __syncthreads();
  const int room = a.max_pages * a.page_size;
  for (int i = threadIdx.x; i < a.n_seq; i += 1024) {
    const int r0 = a.q_start[i], r1 = a.q_start[i + 1], kl = a.k_len[i];
    if (r0 < 0 || r1 < r0 || r1 > a.Tq || kl < 0 || kl > room) paged_report(a.status, kStatusDeviceArg, 50);
    if (a.ctx_len) {
      const int c = a.ctx_len[i];
      if (c < 0 || c > room || paged_seg(a, i).q_len < paged_rows(a, i).q_len)
        paged_report(a.status, kStatusDeviceArg, 52);
    }
  }
  if (many) place_items(a);
}

// Joins the pieces of the item that starts in CTA blockIdx.x's span and ends
// in a later one's: 32 rows per block, four rows per warp.  Bound by trips to
// L2, so the loads of two pieces of all four rows are under way at once; launched
// alone and cold 6.5 us for 32 requests of 5 tokens, 10.9 for 8 prompts.
constexpr int kJoinRows = 32;
template <typename T, bool k8>
__global__ void __launch_bounds__(8 * kJoinRows, 3) paged_join_kernel(const __grid_constant__ PagedAttnArgs a) {
  launch_dependents();
  grid_wait();
  const int c0 = blockIdx.x;
  const PagedCut cut = a.cuts[c0];
  if (cut.last < 0) return;
  const int lane = threadIdx.x & 31;
  const int row0 = blockIdx.y * kJoinRows + (threadIdx.x >> 5) * 4;  // of the item's two sub-tiles
  auto token_of = [&](int row) { return cut.tok0 + (row >> 7) * a.tpt + (row & 127) / a.G; };
  if (token_of(row0) >= cut.q_len || (row0 & 127) >= a.tpt * a.G) return;  // nor do the three after it have a token
  auto piece = [&](int k) {
    return a.chunk_parts + (2 * (c0 + k) + (k == 0 ? cut.late : 0)) * static_cast<long long>(kPagedChunkPartFloats);
  };
  float m, l, o[4][4];
  join_rows<256, 4, 2>(cut.last - c0 + 1, piece, row0, m, l, o);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float mr = __shfl_sync(~0u, m, 8 * r), lr = __shfl_sync(~0u, l, 8 * r);
    const int row = row0 + r, token = token_of(row);
    if (token >= cut.q_len || (row & 127) >= a.tpt * a.G) continue;
    const int head = cut.head * a.G + (row & 127) % a.G;
    const float inv = lr == 0.f ? 0.f : 1.f / lr;
    T* dst = static_cast<T*>(a.o) + (static_cast<long long>(cut.q_off + token) * a.Hq + head) * kHeadDim + 4 * lane;
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(Half2<T>::pack(o[r][0] * inv, o[r][1] * inv), Half2<T>::pack(o[r][2] * inv, o[r][3] * inv));
    if (lane == 0)
      a.lse[static_cast<long long>(head) * a.Tq + cut.q_off + token] =
          lr == 0.f ? -INFINITY : (mr + log2f(lr) - kBias<Operand<T, k8>>) * kLn2;
  }
}

}  // namespace

cudaError_t launch_paged_begin(const PagedAttnArgs& a, bool many, cudaStream_t st) {
  note_launches(1);
  paged_begin_kernel<<<1, 1024, 0, st>>>(a, many);
  return cudaGetLastError();
}

cudaError_t launch_paged_chunk(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const PagedAttnArgs& a, bool fp16, int num_sms, cudaStream_t st) {
  return fp16 ? launch_chunk<__half, false>(tq, tk, tv, a, num_sms, st)
              : launch_chunk<__nv_bfloat16, false>(tq, tk, tv, a, num_sms, st);
}

cudaError_t launch_paged_join(const PagedAttnArgs& a, bool fp16, bool eight, int num_sms, cudaStream_t st) {
  const dim3 grid(std::min(num_sms, kPagedMaxChunkCtas), 256 / kJoinRows);
  note_launches(1);
  const auto kernel = fp16    ? (eight ? paged_join_kernel<__half, true> : paged_join_kernel<__half, false>)
                      : eight ? paged_join_kernel<__nv_bfloat16, true>
                              : paged_join_kernel<__nv_bfloat16, false>;
  return launch_after(kernel, grid, 8 * kJoinRows, 0, st, a);
}

}  // namespace lca
