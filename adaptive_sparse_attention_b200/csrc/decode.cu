// decode.cu -- alpha-entmax attention of one new token per request over a paged key-value cache
// (the serving form of the forward pass).  For request b with n = seq_lens[b] keys and query head
// h of kv head h / G:
//   z_j = c q . k_j, c = (alpha - 1) / sqrt(d);   p_j = [z_j - tau]_+^beta, sum_j p_j = 1;
//   o = sum_j p_j v_j
// with key j in slot j % page_size of page block_tables[b][j / page_size].
//
// Two kernels.  decode_scores_kernel reads every key once and keeps, per (request, head), the keys
// that can carry p > 0 (z > max - 1, since p <= 1 gives tau >= max - 1).  decode_join_kernel joins
// them: the max over all parts, tau, and o from the values of the keys with z > tau.  A softmax
// would have to read every value too; here the values of keys with p = 0 are never read, so the
// traffic is that of the keys alone unless the supports are wide.
//
// What bounds it: HBM reads of the keys.  The cache is split in units of 16 keys of one kv head;
// all units of the batch are dealt to the grid's warps in equal contiguous runs, whatever the
// requests' lengths, so one long request and many ragged ones load the GPU alike, and the lengths
// are needed on the device only.  A run that crosses from one (request, kv head) to the next is
// cut there into parts; part (warp w, group g) has the number w + g, which is unique because
// every cut advances w or g.
#include <cuda_bf16.h>

#include "common.cuh"
#include "entmax_attn.h"
#include "kernels.h"

namespace ea {
namespace {

constexpr int kScoreThreads = 128;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kJoinThreads = 128;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kWarpList = 512;  // candidates a warp of the join keeps in shared memory
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ int clamped_len(const DecodeProblem& P, int b) {
  const int n = P.lens[b];
  return n < 0 || n > P.max_len ? 0 : n;
}

// Inclusive scan of x over the block's threads; *total gets the block's sum.  buf: one int per
// warp.  Every thread of the block calls it.
template <int WARPS>
__device__ __forceinline__ int block_scan(int x, int* buf, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // buf may still be read by the previous call
  if (lane == 31) buf[warp] = x;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += buf[w];
    sum += buf[w];
  }
  *total = sum;
  return x + before;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// Scores of 16 keys x 8 NT heads.  Lane 4 g + t holds, of key rows g and g + 8, the 16-byte chunks
// t, t + 4, t + 8, ... (four lanes read 64 contiguous bytes of a row).  bf16: the chunk's four
// bf16 pairs are the A fragments of two m16n8k16 products whose k index is permuted the same way
// in q's B fragments, so the keys go from global memory to the tensor cores without shared
// memory.  mma.sync suffices: the products take a fraction of the time the keys' bytes do, and
// the M = 128 tile of tcgen05 would be filled by the G heads of one group to a sixteenth.
// fp32: true fp32 products on the CUDA cores, q from shared memory, summed over the four lanes.
// Either way lane 4 g + t ends with rows g, g + 8 of heads 2 t, 2 t + 1 of every 8.
template <typename T, int D, int NT>
struct Scorer;

template <int D, int NT>
struct Scorer<__nv_bfloat16, D, NT> {
  static constexpr int kChunks = D / 32;  // 16-byte chunks per lane and row
  uint32_t bq[NT][kChunks][4];
  __device__ __forceinline__ void load_q(const __nv_bfloat16* q, int64_t stride_h, int heads,
                                         float*) {
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (n * 8 + g < heads)
          x = *reinterpret_cast<const uint4*>(q + (n * 8 + g) * stride_h + c * 32 + t * 8);
        bq[n][c][0] = x.x;
        bq[n][c][1] = x.y;
        bq[n][c][2] = x.z;
        bq[n][c][3] = x.w;
      }
  }
  __device__ __forceinline__ void scores(const uint4 (&a)[2][kChunks], float (&acc)[NT][4],
                                         const float*) const {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        mma_bf16(acc[n], a[0][c].x, a[1][c].x, a[0][c].y, a[1][c].y, bq[n][c][0], bq[n][c][1]);
        mma_bf16(acc[n], a[0][c].z, a[1][c].z, a[0][c].w, a[1][c].w, bq[n][c][2], bq[n][c][3]);
      }
    }
  }
};

template <int D, int NT>
struct Scorer<float, D, NT> {
  static constexpr int kChunks = D / 16;
  int heads_;
  // q of the group's heads into the warp's shared-memory rows [8 NT][D]
  __device__ __forceinline__ void load_q(const float* q, int64_t stride_h, int heads, float* sq) {
    __syncwarp();
    heads_ = heads;
    for (int i = threadIdx.x & 31; i < heads * (D / 4); i += 32)
      reinterpret_cast<float4*>(sq)[i] = *reinterpret_cast<const float4*>(
          q + (i / (D / 4)) * stride_h + (i % (D / 4)) * 4);
    __syncwarp();
  }
  __device__ __forceinline__ void scores(const uint4 (&a)[2][kChunks], float (&acc)[NT][4],
                                         const float* sq) const {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        float s0 = 0.f, s1 = 0.f;
        if (n * 8 + h < heads_) {  // uniform
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const float4 x =
                *reinterpret_cast<const float4*>(sq + (n * 8 + h) * D + c * 16 + t * 4);
            s0 = fmaf(__uint_as_float(a[0][c].x), x.x, s0);
            s0 = fmaf(__uint_as_float(a[0][c].y), x.y, s0);
            s0 = fmaf(__uint_as_float(a[0][c].z), x.z, s0);
            s0 = fmaf(__uint_as_float(a[0][c].w), x.w, s0);
            s1 = fmaf(__uint_as_float(a[1][c].x), x.x, s1);
            s1 = fmaf(__uint_as_float(a[1][c].y), x.y, s1);
            s1 = fmaf(__uint_as_float(a[1][c].z), x.z, s1);
            s1 = fmaf(__uint_as_float(a[1][c].w), x.w, s1);
          }
          s0 += __shfl_xor_sync(kFull, s0, 1);
          s1 += __shfl_xor_sync(kFull, s1, 1);
          s0 += __shfl_xor_sync(kFull, s0, 2);
          s1 += __shfl_xor_sync(kFull, s1, 2);
        }
        if (h >> 1 == t) {
          acc[n][h & 1] = s0;
          acc[n][2 + (h & 1)] = s1;
        }
      }
    }
  }
};

// The two key rows a lane reads of one unit, and whether they exist.
template <int CH>
struct Unit {
  uint4 a[2][CH];
};

// Walks the block table for one key row of a lane: the row of unit u + 1 is 16 keys further on.
struct RowCursor {
  int blk, off;
  __device__ __forceinline__ void start(int key, int page) {
    blk = key / page;
    off = key - blk * page;
  }
  __device__ __forceinline__ void advance(int page) {
    off += 16;
    if (off >= page) {
      if (page >= 16) {
        off -= page;
        ++blk;
      } else {
        const int n = off / page;
        blk += n;
        off -= n * page;
      }
    }
  }
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kScoreThreads, 4) decode_scores_kernel(const DecodeProblem P) {
  using S = Scorer<T, D, NT>;
  constexpr int CH = S::kChunks;
  // 8 KB of keys in flight per warp
  constexpr int DEPTH = 8192 / (16 * D * static_cast<int>(sizeof(T)));
  extern __shared__ __align__(16) char smem[];
  float* sq_all = reinterpret_cast<float*>(smem);  // fp32 only: [warps][8 NT][D]
  int* pre = reinterpret_cast<int*>(
      smem + (sizeof(T) == 4 ? kScoreWarps * 8 * NT * D * sizeof(float) : 0));  // [B + 1]
  __shared__ int scan_buf[kScoreWarps];
  asm volatile("griddepcontrol.launch_dependents;");

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  {  // prefix sums of the requests' unit counts
    const int per = (P.B + kScoreThreads - 1) / kScoreThreads;
    const int b0 = min(tid * per, P.B), b1 = min(b0 + per, P.B);
    int sum = 0;
    for (int b = b0; b < b1; ++b) sum += (clamped_len(P, b) + 15) >> 4;
    int total;
    int at = block_scan<kScoreWarps>(sum, scan_buf, &total) - sum;
    for (int b = b0; b < b1; ++b) {
      pre[b] = at;
      at += (clamped_len(P, b) + 15) >> 4;
    }
    if (tid == 0) pre[P.B] = total;
    __syncthreads();
  }
  if (blockIdx.x == 0) {  // for the join
    for (int b = tid; b <= P.B; b += kScoreThreads) P.pre[b] = pre[b];
    for (int b = tid; b < P.B; b += kScoreThreads)
      if (P.lens[b] < 0 || P.lens[b] > P.max_len) atomicMax(P.status, ENTMAX_ATTN_ERANGE);
  }
  const int HG = P.Hkv * P.head_blocks;  // groups per request
  const int64_t N = static_cast<int64_t>(pre[P.B]) * HG;
  const int64_t nw = min(static_cast<int64_t>(gridDim.x) * kScoreWarps, N);
  const int w = blockIdx.x * kScoreWarps + warp;
  if (w >= nw) return;
  int64_t u = w * N / nw;
  const int64_t u_end = (w + 1) * N / nw;
  float* sq = sq_all + warp * 8 * NT * D;

  while (u < u_end) {
    // the request of unit u: the last b with pre[b] <= u / HG (empty requests have pre[b + 1] =
    // pre[b] and are never last)
    const int v = static_cast<int>(u / HG);
    int lo = 0, hi = P.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= v) lo = mid;
      else hi = mid - 1;
    }
    const int b = lo;
    const int nb = pre[b + 1] - pre[b];
    const int64_t r = u - static_cast<int64_t>(pre[b]) * HG;
    const int hg = static_cast<int>(r / nb);
    const int first = static_cast<int>(r - static_cast<int64_t>(hg) * nb);
    const int last = static_cast<int>(min(static_cast<int64_t>(nb), first + (u_end - u)));
    u += last - first;
    const int hk = hg / P.head_blocks, hb = hg - hk * P.head_blocks;
    const int h0 = hk * P.G + hb * 8 * NT;               // first query head of the part
    const int heads = min(8 * NT, P.G - hb * 8 * NT);    // its query heads
    const int len = clamped_len(P, b);
    const int32_t* table = P.tables + b * P.table_stride;
    const T* kbase = static_cast<const T*>(P.k) + hk * P.head_stride + t * (16 / sizeof(T));
    S sc;
    sc.load_q(static_cast<const T*>(P.q) + b * P.q_stride_b + h0 * P.q_stride_h, P.q_stride_h,
              heads, sq);

    float m[NT][2];
    int cnt[NT][2];
    bool bad[NT][2];
    int2* cand[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[n][e] = -INFINITY;
        cnt[n][e] = 0;
        bad[n][e] = false;
        const int h = n * 8 + 2 * t + e;
        cand[n][e] = P.cand + (static_cast<int64_t>(b) * P.Hq + h0 + min(h, heads - 1)) *
                                  P.cand_stride + first * 16;
      }
    bool bad_page = false;

    // Pipeline: the keys of the next DEPTH units are in registers or on their way, the page
    // numbers of the unit after those too.
    RowCursor cur[2];
    cur[0].start(first * 16 + g, P.page_size);
    cur[1].start(first * 16 + g + 8, P.page_size);
    int fetch = first;  // unit the cursors stand at
    int page[2], off[2];
    auto next_pages = [&]() {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        page[i] = -1;
        off[i] = cur[i].off;
        if (fetch < last && fetch * 16 + g + 8 * i < len) {
          page[i] = table[cur[i].blk];
          if (page[i] < 0 || page[i] >= P.num_pages) {
            page[i] = -1;
            bad_page = true;
          }
        }
        cur[i].advance(P.page_size);
      }
      ++fetch;
    };
    Unit<CH> unit[DEPTH];
    auto load_unit = [&](Unit<CH>& x) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const T* row = kbase + page[i] * P.page_stride + off[i] * P.slot_stride;
#pragma unroll
        for (int c = 0; c < CH; ++c)
          x.a[i][c] = page[i] >= 0 ? load_stream(row + c * (64 / sizeof(T)))
                                   : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    next_pages();
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) {
      load_unit(unit[i]);
      next_pages();
    }
    for (int blk0 = first; blk0 < last; blk0 += DEPTH) {
#pragma unroll
      for (int i = 0; i < DEPTH; ++i) {
        const int blk = blk0 + i;
        if (blk < last) {
          float acc[NT][4];
          sc.scores(unit[i].a, acc, sq);
          load_unit(unit[i]);
          next_pages();
          const int key = blk * 16 + g;
          bool pass = false;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool live = n * 8 + 2 * t + (e & 1) < heads && key + (e >> 1) * 8 < len;
              const float z = live ? P.c * acc[n][e] : -INFINITY;
              acc[n][e] = z;
              bad[n][e & 1] |= !(z < INFINITY);
              pass |= z > m[n][e & 1] - 1.f;
            }
          if (__any_sync(kFull, pass)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float x = fmaxf(acc[n][e], acc[n][2 + e]);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
                m[n][e] = fmaxf(m[n][e], x);
#pragma unroll
                for (int i2 = 0; i2 < 2; ++i2) {
                  const float z = acc[n][2 * i2 + e];
                  const bool in = z > m[n][e] - 1.f;
                  const unsigned mine = __ballot_sync(kFull, in) & (0x11111111u << t);
                  if (in)
                    cand[n][e][cnt[n][e] + __popc(mine & ((1u << lane) - 1u))] =
                        make_int2(__float_as_int(z), key + 8 * i2);
                  cnt[n][e] += __popc(mine);
                }
              }
          }
        }
      }
    }
    bad_page = __any_sync(kFull, bad_page);
    if (bad_page && lane == 0) atomicMax(P.status, ENTMAX_ATTN_ERANGE);
    int2* part = P.parts + (static_cast<int64_t>(w) + static_cast<int64_t>(b) * HG + hg) *
                               (8 * NT);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool nan =
            (__ballot_sync(kFull, bad[n][e]) & (0x11111111u << t)) != 0u || bad_page;
        if (g == 0)
          part[n * 8 + 2 * t + e] = make_int2(cnt[n][e], __float_as_int(nan ? NAN : m[n][e]));
      }
  }
}

// max that keeps a NaN of either side
__device__ __forceinline__ float max_nan(float a, float b) {
  return (a != a || b != b) ? NAN : fmaxf(a, b);
}

// One block per (request, query head).
template <typename T, int D, int BK>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const DecodeProblem P) {
  extern __shared__ __align__(16) char smem[];
  int* start = reinterpret_cast<int*>(smem);  // [parts of the group + 1]: prefix sums of counts
  __shared__ float2 list[kJoinWarps][kWarpList];  // (z, key bits), one list per warp
  __shared__ float sums[2][kJoinWarps][4];
  __shared__ float red[kJoinWarps];
  __shared__ int scan_buf[kJoinWarps];
  __shared__ __align__(16) float oacc[kJoinWarps][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x, b = blockIdx.y;
  const int hk = h / P.G, in_group = h - hk * P.G;
  const int hb = in_group / P.heads_per_block, col = in_group - hb * P.heads_per_block;
  const int64_t row = static_cast<int64_t>(b) * P.Hq + h;
  T* out = static_cast<T*>(P.out) + row * D;
  const int raw_len = P.lens[b];
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const int len = clamped_len(P, b);
  if (len == 0) {  // no key: o = 0 and tau = +inf; a length out of range: NaN
    const float x = raw_len == 0 ? 0.f : NAN;
    for (int i = tid; i < D; i += kJoinThreads) store_elem(out, i, x);
    if (tid == 0) P.tau[row] = raw_len == 0 ? INFINITY : NAN;
    return;
  }
  const int HG = P.Hkv * P.head_blocks;
  const int64_t N = static_cast<int64_t>(P.pre[P.B]) * HG;
  const int64_t nw = min(static_cast<int64_t>(P.score_warps), N);
  const int nb = (len + 15) >> 4;
  const int hg = hk * P.head_blocks + hb;
  const int64_t A = static_cast<int64_t>(P.pre[b]) * HG + static_cast<int64_t>(hg) * nb;
  // the warps whose runs hold the group's first and last unit: the last w with w N / nw <= unit
  const int64_t w0 = ((A + 1) * nw - 1) / N, w1 = ((A + nb) * nw - 1) / N;
  const int np = static_cast<int>(w1 - w0) + 1;
  const int2* part = P.parts + (w0 + static_cast<int64_t>(b) * HG + hg) * P.heads_per_block + col;

  float m = -INFINITY;
  for (int i = tid; i < np; i += kJoinThreads)
    m = max_nan(m, __int_as_float(part[static_cast<int64_t>(i) * P.heads_per_block].y));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(kFull, m, o));
  if (lane == 0) red[warp] = m;
  __syncthreads();
  m = red[0];
#pragma unroll
  for (int i = 1; i < kJoinWarps; ++i) m = max_nan(m, red[i]);
  if (!(m > -INFINITY)) {  // NaN, or every score -inf: p is not defined
    for (int i = tid; i < D; i += kJoinThreads) store_elem(out, i, NAN);
    if (tid == 0) P.tau[row] = NAN;
    return;
  }
  // Candidates of the parts that reach the window, as one sequence of E entries
  int E = 0;
  for (int i0 = 0; i0 < np; i0 += kJoinThreads) {
    const int i = i0 + tid;
    int n = 0;
    if (i < np) {
      const int2 x = part[static_cast<int64_t>(i) * P.heads_per_block];
      if (__int_as_float(x.y) > m - 1.f) n = x.x;
    }
    int total;
    const int incl = block_scan<kJoinWarps>(n, scan_buf, &total);
    if (i < np) start[i] = E + incl - n;
    E += total;
  }
  if (tid == 0) start[np] = E;
  __syncthreads();
  const int2* cand = P.cand + row * P.cand_stride;
  auto entry = [&](int e) {  // the e-th candidate: in the last part that starts at or before e
    int lo = 0, hi = np - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (start[mid] <= e) lo = mid;
      else hi = mid - 1;
    }
    const int64_t u = (w0 + lo) * N / nw;  // the part's first unit
    const int64_t k0 = u > A ? (u - A) * 16 : 0;
    return cand[k0 + e - start[lo]];
  };
  // Each warp compacts its entries with z > m - 1 into its list, in a fixed order.
  int n_list = 0;
  for (int e0 = warp * 32; e0 < E; e0 += kJoinThreads) {
    const int e = e0 + lane;
    int2 x = make_int2(__float_as_int(-INFINITY), 0);
    if (e < E) x = entry(e);
    const bool in = __int_as_float(x.x) > m - 1.f;
    const unsigned bal = __ballot_sync(kFull, in);
    const int at = n_list + __popc(bal & ((1u << lane) - 1u));
    if (in && at < kWarpList) list[warp][at] = make_float2(__int_as_float(x.x), __int_as_float(x.y));
    n_list += __popc(bal);
  }
  __syncwarp();
  const bool over = __syncthreads_or(n_list > kWarpList);

  // tau
  Search sr;
  sr.init(m, len, P.alpha);
  for (int it = 0; it < P.n_iter; ++it) {
    const float tau = sr.tau;
    float s0 = 0.f, s1 = 0.f, s2 = 0.f;
    auto add = [&](float z) {
      const float y = z - tau;
      if (y > 0.f) {
        float p0, p1, p2;
        entmax_powers<BK>(y, P.beta, p0, p1, p2);
        s0 += p0;
        s1 += p1;
        s2 += p2;
      }
    };
    if (!over) {
      for (int e = lane; e < n_list; e += 32) add(list[warp][e].x);
    } else {
      for (int e = tid; e < E; e += kJoinThreads) add(__int_as_float(entry(e).x));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s0 += __shfl_xor_sync(kFull, s0, o);
      s1 += __shfl_xor_sync(kFull, s1, o);
      s2 += __shfl_xor_sync(kFull, s2, o);
    }
    if (lane == 0) {
      sums[it & 1][warp][0] = s0;
      sums[it & 1][warp][1] = s1;
      sums[it & 1][warp][2] = s2;
    }
    __syncthreads();  // two buffers: the next step writes the other one
    s0 = s1 = s2 = 0.f;
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) {
      s0 += sums[it & 1][i][0];
      s1 += sums[it & 1][i][1];
      s2 += sums[it & 1][i][2];
    }
    sr.step<BK>(s0, s1, s2, P.beta);
    if (sr.settled()) break;
  }
  const float tau = sr.tau;

  // o: 16-byte chunks of the value rows, D sizeof(T) / 16 lanes per row
  constexpr int LPR = D * sizeof(T) / 16;  // lanes per value row (8, 16 or 32)
  constexpr int RPW = 32 / LPR;            // value rows per warp load
  constexpr int EPL = 16 / sizeof(T);      // elements per lane
  float o[EPL] = {};
  const int32_t* table = P.tables + b * P.table_stride;
  const T* vbase = static_cast<const T*>(P.v) + hk * P.head_stride + (lane % LPR) * EPL;
  const int n_mine = over ? E : n_list;
  for (int e0 = over ? warp * 32 : 0; e0 < n_mine; e0 += over ? kJoinThreads : 32) {
    const int e = e0 + lane;
    float p = 0.f;
    int64_t at = 0;
    if (e < n_mine) {
      float z;
      int key;
      if (over) {
        const int2 x = entry(e);
        z = __int_as_float(x.x);
        key = x.y;
      } else {
        z = list[warp][e].x;
        key = __float_as_int(list[warp][e].y);
      }
      p = entmax_p<BK>(z - tau, P.beta);
      if (p > 0.f) {
        const int blk = key / P.page_size;
        at = table[blk] * P.page_stride + (key - blk * P.page_size) * P.slot_stride;
      }
    }
    unsigned live = __ballot_sync(kFull, p > 0.f);
    while (live) {  // RPW rows at a time: this lane's is the (lane / LPR)-th of the set bits
      unsigned rest = live;
      int src = -1;
#pragma unroll
      for (int i = 0; i < RPW; ++i) {
        const int bit = rest ? __ffs(rest) - 1 : -1;
        if (i == lane / LPR) src = bit;
        rest &= rest - 1u;
      }
      live = rest;
      const float pw = __shfl_sync(kFull, p, src & 31);
      const int64_t from = __shfl_sync(kFull, at, src & 31);
      if (src >= 0) {
        const uint4 x = load_stream(vbase + from);
        const T* xv = reinterpret_cast<const T*>(&x);
#pragma unroll
        for (int i = 0; i < EPL; ++i) o[i] = fmaf(pw, load_elem(xv, i), o[i]);
      }
    }
  }
#pragma unroll
  for (int s = LPR; s < 32; s <<= 1)
#pragma unroll
    for (int i = 0; i < EPL; ++i) o[i] += __shfl_xor_sync(kFull, o[i], s);
  if (lane < LPR)
#pragma unroll
    for (int i = 0; i < EPL; ++i) oacc[warp][lane * EPL + i] = o[i];
  __syncthreads();
  for (int i = tid; i < D; i += kJoinThreads) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kJoinWarps; ++k) s += oacc[k][i];
    store_elem(out, i, s);
  }
  if (tid == 0) P.tau[row] = tau;
}

template <typename T, int D, int NT>
cudaError_t launch_scores(const DecodeProblem& P, cudaStream_t s) {
  const size_t smem = (sizeof(T) == 4 ? kScoreWarps * 8 * NT * D * sizeof(float) : 0) +
                      sizeof(int) * (P.B + 1);
  auto kern = decode_scores_kernel<T, D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  kern<<<kDecodeScoreWarps / kScoreWarps, kScoreThreads, smem, s>>>(P);
  return cudaGetLastError();
}

template <typename T, int D, int BK>
cudaError_t launch_join(const DecodeProblem& P, cudaStream_t s) {
  // parts of one group: at most one per warp, and at most one per unit
  const int np = min(kDecodeScoreWarps, (P.max_len + 15) / 16);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(P.Hq, P.B);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = sizeof(int) * (np + 1);
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_join_kernel<T, D, BK>, P);
}

template <typename T, int D>
cudaError_t launch_decode_t(const DecodeProblem& P, cudaStream_t s) {
  cudaError_t e = P.heads_per_block == 8 ? launch_scores<T, D, 1>(P, s)
                                         : launch_scores<T, D, 2>(P, s);
  if (e != cudaSuccess) return e;
  switch (beta_kind(P.beta)) {
    case kBetaOne: return launch_join<T, D, kBetaOne>(P, s);
    case kBetaTwo: return launch_join<T, D, kBetaTwo>(P, s);
    case kBetaNear3: return launch_join<T, D, kBetaNear3>(P, s);
    default: return launch_join<T, D, kBetaGeneral>(P, s);
  }
}

}  // namespace

cudaError_t launch_decode(const DecodeProblem& P, int dtype, int d, cudaStream_t s) {
  if (dtype == ENTMAX_ATTN_FP32)
    return d == 64 ? launch_decode_t<float, 64>(P, s) : launch_decode_t<float, 128>(P, s);
  return d == 64 ? launch_decode_t<__nv_bfloat16, 64>(P, s)
                 : launch_decode_t<__nv_bfloat16, 128>(P, s);
}

}  // namespace ea
