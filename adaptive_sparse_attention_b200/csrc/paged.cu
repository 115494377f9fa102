// paged.cu -- the bookkeeping and the writes of a paged key-value cache: block tables and slot
// maps from the requests' lengths (page_tables_kernel), and the new tokens' keys and values into
// their slots (paged_append_kernel).
#include "entmax_attn.h"
#include "kernels.h"

namespace ea {
namespace {

constexpr int kTableThreads = 512;
constexpr int kTableWarps = kTableThreads / 32;
constexpr int kSlots = 4;  // consecutive slots per thread, one search for all
constexpr unsigned kFull = 0xffffffffu;

struct Grow {
  int have, need, add;  // pages held, pages needed, new tokens
  bool ok;              // the lengths make sense and the table row holds the pages
};

__device__ __forceinline__ Grow grow_of(const PageTables& P, int b) {
  Grow r;
  const int len = P.lens[b], add = P.new_lens[b];
  r.add = max(add, 0);
  const int64_t total = static_cast<int64_t>(len) + r.add;
  r.have = len > 0 ? (len - 1) / P.page_size + 1 : 0;
  r.need = r.have;
  r.ok = len >= 0 && add >= 0 && total <= P.table_tokens &&
         (!P.padded || add <= P.n_new);
  if (r.ok) r.need = total > 0 ? static_cast<int>((total - 1) / P.page_size) + 1 : 0;
  return r;
}

// Sums of new tokens stop at 2^31 - 1, so that the prefix sums never fall: no lengths send a search
// or an index outside.  (The pages add up to less than 2^31, see the host checks.)
__device__ __forceinline__ int add_tokens(int a, int b) {  // both >= 0
  return static_cast<int>(min(static_cast<unsigned>(a) + static_cast<unsigned>(b), 0x7fffffffu));
}

// Block-wide exclusive scans of two values at once, x by add_tokens; totals in tx, ty.
__device__ __forceinline__ void scan2(int& x, int& y, int2* buf, int& tx, int& ty) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(kFull, x, o), b = __shfl_up_sync(kFull, y, o);
    if (lane >= o) {
      x = add_tokens(x, a);
      y += b;
    }
  }
  if (lane == 31) buf[warp] = make_int2(x, y);
  x = __shfl_up_sync(kFull, x, 1);
  y = __shfl_up_sync(kFull, y, 1);
  if (lane == 0) x = y = 0;
  __syncthreads();
  int bx = 0, by = 0;
  tx = ty = 0;
#pragma unroll
  for (int w = 0; w < kTableWarps; ++w) {
    const int2 v = buf[w];
    if (w < warp) {
      bx = add_tokens(bx, v.x);
      by += v.y;
    }
    tx = add_tokens(tx, v.x);
    ty += v.y;
  }
  x = add_tokens(x, bx);
  y += by;
}

// A request as the blocks look it up.
struct Entry {
  int token;  // its first new token
  int page;   // its first entry of the free list, counted from free_start
  int len;    // tokens held, -1 if it is not served
  int have;   // pages held
};
// last b with e[b].FIELD <= v (nondecreasing, e[0].FIELD <= v)
template <int Entry::*FIELD>
__device__ __forceinline__ int last_at_most(const Entry* e, int n, int v) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (e[mid].*FIELD <= v) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Every block scans the B lengths itself (a few KB from L2, no second launch and no order between
// blocks), then writes its share of the new table entries and of the slots.  Bound by the launch
// and three dependent loads for small batches (64 requests of one token: 5 us), by the scan, the
// search and the writes of 8 bytes a token for large ones (1000 requests, 236K tokens: 6.8 us).
__global__ void __launch_bounds__(kTableThreads) page_tables_kernel(const PageTables P) {
  extern __shared__ __align__(16) char smem[];
  Entry* req = reinterpret_cast<Entry*>(smem);  // [B + 1], the last holds the totals
  __shared__ int2 buf[kTableWarps];
  __shared__ int served_pages;
  const int tid = threadIdx.x;
  serial_wait();
  const int start = *P.free_start;
  const int avail = start >= 0 && start <= P.n_free ? P.n_free - start : 0;
  if (tid == 0) served_pages = 0;
  {
    const int per = (P.B + kTableThreads - 1) / kTableThreads;
    const int b0 = min(tid * per, P.B), b1 = min(b0 + per, P.B);
    int toks = 0, pages = 0;
    for (int b = b0; b < b1; ++b) {
      const Grow r = grow_of(P, b);
      toks = add_tokens(toks, r.add);
      pages += r.need - r.have;
    }
    int x = toks, y = pages, tx, ty;
    scan2(x, y, buf, tx, ty);
    for (int b = b0; b < b1; ++b) {
      const Grow r = grow_of(P, b);
      const int x1 = add_tokens(x, r.add), y1 = y + r.need - r.have;
      // A request is served if its lengths fit, its tokens lie inside the slots and its pages
      // inside the free list.  Requests that take pages are served in order until the list is
      // exhausted.
      const bool ok = r.ok && x1 < 0x7fffffff && (P.padded || x1 <= P.n_new) &&
                      (r.need == r.have || y1 <= avail);
      req[b] = {x, y, ok ? P.lens[b] : -1, r.have};
      x = x1;
      y = y1;
    }
    if (tid == 0) req[P.B] = {tx, ty, -1, 0};
    __syncthreads();
  }
  const int step = gridDim.x * kTableThreads;  // at most 148 blocks
  const int me = blockIdx.x * kTableThreads + tid;
  // slots
  const int64_t n_slots = P.padded ? static_cast<int64_t>(P.B) * P.n_new : P.n_new;
  for (int64_t i0 = static_cast<int64_t>(me) * kSlots; i0 < n_slots;
       i0 += static_cast<int64_t>(step) * kSlots) {
    int b, t;  // of slot i0
    if (!P.padded) {
      b = last_at_most<&Entry::token>(req, P.B, static_cast<int>(i0));
      t = static_cast<int>(i0) - req[b].token;
    } else if (n_slots <= 0x7fffffff) {
      b = static_cast<int>(i0) / P.n_new;
      t = static_cast<int>(i0) - b * P.n_new;
    } else {
      b = static_cast<int>(i0 / P.n_new);
      t = static_cast<int>(i0 - static_cast<int64_t>(b) * P.n_new);
    }
    Entry r = req[b];
    int add = req[b + 1].token - r.token;
    int64_t slot[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j, ++t) {
      // on to the request of slot i0 + j: the next one with a new token, or the next row
      while (t >= (P.padded ? P.n_new : add) && b + 1 < P.B) {
        r = req[++b];
        add = req[b + 1].token - r.token;
        t = 0;
      }
      slot[j] = -1;
      if (r.len >= 0 && t < add) {
        const int pos = r.len + t;
        const int blk = pos / P.page_size;
        const int page = blk < r.have ? P.tables[b * P.table_stride + blk]
                                      : P.free_pages[start + r.page + (blk - r.have)];
        if (page >= 0)
          slot[j] = static_cast<int64_t>(page) * P.page_size + (pos - blk * P.page_size);
      }
    }
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (i0 + j < n_slots) P.slots[i0 + j] = slot[j];
  }
  // new table entries
  const int n_pages = min(req[P.B].page, avail);
  for (int j = me; j < n_pages; j += step) {
    const int b = last_at_most<&Entry::page>(req, P.B, j);
    const Entry r = req[b];
    if (r.len >= 0)
      P.tables[b * P.table_stride + r.have + (j - r.page)] = P.free_pages[start + j];
  }
  if (blockIdx.x == 0) {
    int most = 0;
    for (int b = tid; b < P.B; b += kTableThreads) {
      const Entry r = req[b], next = req[b + 1];
      P.lens_out[b] = r.len >= 0 ? r.len + (next.token - r.token) : P.lens[b];
      P.cu_new[b] = r.token;
      if (r.len >= 0 && next.page > r.page) most = max(most, next.page);
    }
    if (most) atomicMax(&served_pages, most);  // a maximum does not depend on the order
    __syncthreads();
    if (tid == 0) {
      P.cu_new[P.B] = req[P.B].token;
      *P.free_next = start + served_pages;
    }
  }
}

// The copies of one chunk of tokens: a block takes kTokens tokens of one kv head of k or v, VPR
// threads per row of VPR 16-byte vectors, kAppendRows rows in flight per thread.  A pure copy:
// bound by HBM (32192 tokens of 8 heads, d = 128: 41 us, 6.4 TB/s; with one row in flight 57 us).
// The rows of consecutive tokens are consecutive in a [Hkv, N, d] input and, within a page, in a
// [pages, Hkv, page_size, d] cache.  The grid is (chunks of tokens, kv heads, k or v), so that no
// index needs a 64-bit division.
constexpr int kAppendThreads = 256;
constexpr int kAppendRows = 4;  // rows per thread
template <int VPR>  // 16-byte vectors per row
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const PagedAppend P) {
  constexpr int kStep = kAppendThreads / VPR;
  const int lane = threadIdx.x % VPR;
  const int h = blockIdx.y;
  const char* src = static_cast<const char*>(blockIdx.z ? P.v : P.k) + lane * 16 +
                    h * P.stride_h;
  char* dst = static_cast<char*>(blockIdx.z ? P.v_cache : P.k_cache) + lane * 16 +
              h * P.head_stride;
  const int n0 = blockIdx.x * (kStep * kAppendRows) + threadIdx.x / VPR;
  serial_wait();
  int64_t slot[kAppendRows];
  uint4 x[kAppendRows];
#pragma unroll
  for (int i = 0; i < kAppendRows; ++i) {
    const int n = n0 + i * kStep;
    slot[i] = n < P.n_tokens ? P.slots[n] : -1;
    const int b = P.T == P.n_tokens ? 0 : n / P.T, t = n - b * P.T;
    if (n < P.n_tokens)
      x[i] = *reinterpret_cast<const uint4*>(src + b * P.stride_b + t * P.stride_t);
  }
#pragma unroll
  for (int i = 0; i < kAppendRows; ++i) {
    if (slot[i] < 0) continue;  // a padding row
    if (slot[i] >= P.n_slots) {
      if (lane == 0) atomicMax(P.status, ENTMAX_ATTN_ERANGE);
      continue;
    }
    // num_pages and page_size are ints, so the page of a valid slot is too
    int64_t page;
    if (P.n_slots <= 0x7fffffff) page = static_cast<int>(slot[i]) / P.page_size;
    else page = slot[i] / P.page_size;
    const int off = static_cast<int>(slot[i] - page * P.page_size);
    *reinterpret_cast<uint4*>(dst + page * P.page_stride + off * P.slot_stride) = x[i];
  }
}

}  // namespace

cudaError_t launch_page_tables(const PageTables& P, cudaStream_t s) {
  const int64_t n_slots = P.padded ? static_cast<int64_t>(P.B) * P.n_new : P.n_new;
  const int64_t want = (n_slots - 1) / (kTableThreads * kSlots) + 1;
  const int grid = static_cast<int>(want < 1 ? 1 : want > 148 ? 148 : want);
  const size_t smem = sizeof(Entry) * (P.B + 1);
  if (smem > 48 * 1024) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e =
        allow_smem(page_tables_kernel, sizeof(Entry) * (kMaxRequests + 1), done);
    if (e != cudaSuccess) return e;
  }
  return launch_serial(page_tables_kernel, dim3(grid), dim3(kTableThreads), smem, s, 1, P);
}

cudaError_t launch_paged_append(const PagedAppend& P, int row_bytes, cudaStream_t s) {
  const int vpr = row_bytes / 16;
  const int per_block = kAppendThreads / vpr * kAppendRows;
  const dim3 grid(static_cast<unsigned>((P.n_tokens - 1) / per_block + 1),
                  static_cast<unsigned>(P.Hkv), 2);
  const dim3 block(kAppendThreads);
  switch (vpr) {
    case 8: return launch_serial(paged_append_kernel<8>, grid, block, 0, s, 1, P);
    case 16: return launch_serial(paged_append_kernel<16>, grid, block, 0, s, 1, P);
    default: return launch_serial(paged_append_kernel<32>, grid, block, 0, s, 1, P);
  }
}

}  // namespace ea
