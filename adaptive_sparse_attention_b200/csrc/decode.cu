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
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kWarpList = 256;  // candidates a warp of the join keeps in shared memory
constexpr int kNewtonSteps = 64;  // a bound that no search reaches
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
  // q of head group hg of request b
  __device__ __forceinline__ void load_q(const DecodeProblem& P, int b, int hg, float*) {
    const int hk = hg / P.head_blocks, first = (hg - hk * P.head_blocks) * 8 * NT;
    const int heads = P.G - first;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(P.q) + b * P.q_stride_b +
                             (hk * P.G + first) * P.q_stride_h;
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (n * 8 + g < heads)
          x = *reinterpret_cast<const uint4*>(q + (n * 8 + g) * P.q_stride_h + c * 32 + t * 8);
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
  // q of head group hg of request b into the warp's shared-memory rows [8 NT][D]
  __device__ __forceinline__ void load_q(const DecodeProblem& P, int b, int hg, float* sq) {
    const int hk = hg / P.head_blocks, first = (hg - hk * P.head_blocks) * 8 * NT;
    heads_ = min(8 * NT, P.G - first);
    const float* q = static_cast<const float*>(P.q) + b * P.q_stride_b +
                     (hk * P.G + first) * P.q_stride_h;
    __syncwarp();
    for (int i = threadIdx.x & 31; i < heads_ * (D / 4); i += 32)
      reinterpret_cast<float4*>(sq)[i] = *reinterpret_cast<const float4*>(
          q + (i / (D / 4)) * P.q_stride_h + (i % (D / 4)) * 4);
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

// One warp scores units [first, last) of 16 keys of head group hg of request b and appends the
// candidates of each head to the group's lists at the run's first key, a count and a max per head
// to part.  sq: the warp's (or block's) shared-memory q rows, fp32 only.
template <typename T, int D, int NT>
__device__ __forceinline__ void score_run(const DecodeProblem& P,
                                          const Scorer<T, D, NT>& sc, const float* sq, int b,
                                          int hg, int len, int first, int last, int2* part) {
  using S = Scorer<T, D, NT>;
  constexpr int CH = S::kChunks;
  // 8 KB of keys in flight per warp
  constexpr int DEPTH = 8192 / (16 * D * static_cast<int>(sizeof(T)));
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int hk = hg / P.head_blocks, hb = hg - hk * P.head_blocks;
  const int h0 = hk * P.G + hb * 8 * NT;
  const int heads = min(8 * NT, P.G - hb * 8 * NT);
  const int32_t* table = P.tables + b * P.table_stride;
  const T* kbase = static_cast<const T*>(P.k) + hk * P.head_stride + t * (16 / sizeof(T));

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

  // Pipeline: the keys of the next DEPTH units are in registers or on their way, the page numbers
  // of the unit after those too.
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
  uint4 unit[DEPTH][2][CH];
  auto load_unit = [&](uint4 (&x)[2][CH]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const T* row = kbase + page[i] * P.page_stride + off[i] * P.slot_stride;
#pragma unroll
      for (int c = 0; c < CH; ++c)
        x[i][c] = page[i] >= 0 ? load_stream(row + c * (64 / sizeof(T)))
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
        sc.scores(unit[i], acc, sq);
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
              for (int r = 0; r < 2; ++r) {
                const float z = acc[n][2 * r + e];
                const bool in = z > m[n][e] - 1.f;
                const unsigned mine = __ballot_sync(kFull, in) & (0x11111111u << t);
                if (in)
                  cand[n][e][cnt[n][e] + __popc(mine & ((1u << lane) - 1u))] =
                      make_int2(__float_as_int(z), key + 8 * r);
                cnt[n][e] += __popc(mine);
              }
            }
        }
      }
    }
  }
  bad_page = __any_sync(kFull, bad_page);
  if (bad_page && lane == 0) atomicMax(P.status, ENTMAX_ATTN_ERANGE);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const bool nan = (__ballot_sync(kFull, bad[n][e]) & (0x11111111u << t)) != 0u || bad_page;
      if (g == 0)
        part[n * 8 + 2 * t + e] = make_int2(cnt[n][e], __float_as_int(nan ? NAN : m[n][e]));
    }
}

// max that keeps a NaN of either side
__device__ __forceinline__ float max_nan(float a, float b) {
  return (a != a || b != b) ? NAN : fmaxf(a, b);
}

// x^beta for x > 0 (or 0 where x <= 0), to a few units of the last place: near beta = 3 the cube
// times x^(beta - 3), whose exponent is small enough for the fast logarithm's error.
template <int BK>
__device__ __forceinline__ float power(float x, float beta) {
  if (!(x > 0.f)) return 0.f;
  if (BK == kBetaOne) return x;
  if (BK == kBetaTwo) return x * x;
  if (BK == kBetaNear3) return (x * x) * (x * exp2f((beta - 3.f) * __log2f(x)));
  return exp2f(beta * log2f(x));
}

struct JoinSmem {
  float2 list[kJoinWarps][kWarpList];  // (z, key bits): each warp's candidates
  float2 sums[2][kJoinWarps];
  float sums2[2][kJoinWarps];
  float red[kJoinWarps];
  float2 live[kJoinWarps][32];  // (p, -) and offsets of the values being added
  int64_t from[kJoinWarps][32];
  __align__(16) float o[kJoinWarps][128];
};

// One block joins the parts of one (request, query head): part(i) is its i-th count and max,
// key0(i) the first key of part i in the candidate list.
template <typename T, int D, int BK, typename Part, typename Key0>
__device__ __forceinline__ void join_head(const DecodeProblem& P, JoinSmem& sm, int b, int h,
                                          int len, int np, const Part& part, const Key0& key0) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hk = h / P.G;
  const int64_t row = static_cast<int64_t>(b) * P.Hq + h;
  T* out = static_cast<T*>(P.out) + row * D;

  float m = -INFINITY;
  for (int i = tid; i < np; i += kJoinThreads) m = max_nan(m, __int_as_float(part(i).y));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(kFull, m, o));
  if (lane == 0) sm.red[warp] = m;
  __syncthreads();
  m = sm.red[0];
#pragma unroll
  for (int i = 1; i < kJoinWarps; ++i) m = max_nan(m, sm.red[i]);
  if (!(m > -INFINITY)) {  // NaN, or every score -inf: p is not defined
    for (int i = tid; i < D; i += kJoinThreads) store_elem(out, i, NAN);
    if (tid == 0) P.tau[row] = NAN;
    return;
  }

  // Each warp compacts the entries with z > m - 1 of a contiguous range of parts, in order: the
  // first kWarpList into shared memory, the others back to the front of the range (an entry only
  // moves forward, over entries that the warp has read already).
  int2* cand = P.cand + row * P.cand_stride;
  const int i_end = static_cast<int>(static_cast<int64_t>(warp + 1) * np / kJoinWarps);
  const int i_beg = static_cast<int>(static_cast<int64_t>(warp) * np / kJoinWarps);
  int2* spill = cand + (i_beg < i_end ? key0(i_beg) : 0);
  int n_list = 0;
  for (int i0 = i_beg; i0 < i_end; i0 += 32) {
    int n = 0;
    int64_t k0 = 0;
    if (i0 + lane < i_end) {
      const int2 x = part(i0 + lane);
      if (__int_as_float(x.y) > m - 1.f) n = x.x;
      k0 = key0(i0 + lane);
    }
    int start = n;  // of this lane's part in the sequence of the 32 parts' entries
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, start, o);
      if (lane >= o) start += y;
    }
    const int total = __shfl_sync(kFull, start, 31);
    start -= n;
    const int64_t shift = k0 - start;
    constexpr int U = 4;  // loads in flight per lane
    for (int e0 = 0; e0 < total; e0 += 32 * U) {
      int2 x[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int e = e0 + 32 * j + lane;
        int lo = 0;  // the last part that starts at or before e
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          if (__shfl_sync(kFull, start, lo + o) <= e) lo += o;
        const int64_t at = __shfl_sync(kFull, shift, lo) + e;
        x[j] = make_int2(__float_as_int(-INFINITY), 0);
        if (e < total) x[j] = cand[at];
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const bool in = __int_as_float(x[j].x) > m - 1.f;
        const unsigned bal = __ballot_sync(kFull, in);
        const int at = n_list + __popc(bal & ((1u << lane) - 1u));
        if (in) {
          if (at < kWarpList)
            sm.list[warp][at] = make_float2(__int_as_float(x[j].x), __int_as_float(x[j].y));
          else
            spill[at - kWarpList] = x[j];
        }
        n_list += __popc(bal);
      }
    }
  }
  __syncwarp();
  auto entry = [&](int e) {
    if (e < kWarpList) return sm.list[warp][e];
    const int2 x = spill[e - kWarpList];
    return make_float2(__int_as_float(x.x), __int_as_float(x.y));
  };

  // tau.  For beta >= 1 by Newton's steps on the norm g(tau) = (sum [z - tau]_+^beta)^(1/beta) = 1
  // from tau = m - 1, where g >= 1: g is convex and falling (a norm of functions that are), so
  // the iterates rise to the root and never pass it, and it is linear in tau while the support
  // stays and the scores tie, so the steps are few: with S0, S1 the sums of the powers beta and
  // beta - 1, (g - 1) / -g' = (S0 - S0^(1 - 1/beta)) / S1.  They run until tau has settled (4 or 5
  // steps on normal scores, 14 at most over a wide sweep of sizes and spreads at beta = 1), so
  // n_iter does not enter.  For beta < 1 g is not convex, and the bracketed search of the
  // attention passes is used.
  float tau;
  if (BK != kBetaGeneral || P.beta >= 1.f) {
    tau = m - 1.f;
    for (int it = 0; it < kNewtonSteps; ++it) {
      float s0 = 0.f, s1 = 0.f;
      for (int e = lane; e < n_list; e += 32) {
        const float y = entry(e).x - tau;
        if (BK == kBetaOne) {
          if (y > 0.f) {
            s0 += y;
            s1 += 1.f;
          }
        } else if (BK == kBetaTwo) {
          const float x = fmaxf(y, 0.f);
          s1 += x;
          s0 = fmaf(x, x, s0);
        } else if (y > 0.f) {
          const float p = power<BK>(y, P.beta);
          s0 += p;
          s1 += __fdividef(p, y);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        s0 += __shfl_xor_sync(kFull, s0, o);
        s1 += __shfl_xor_sync(kFull, s1, o);
      }
      if (lane == 0) sm.sums[it & 1][warp] = make_float2(s0, s1);
      __syncthreads();  // two buffers: the next step writes the other one
      s0 = s1 = 0.f;
#pragma unroll
      for (int i = 0; i < kJoinWarps; ++i) {
        s0 += sm.sums[it & 1][i].x;
        s1 += sm.sums[it & 1][i].y;
      }
      float step;
      if (BK == kBetaOne) step = (s0 - 1.f) / s1;
      else if (BK == kBetaTwo) step = (s0 - sqrtf(s0)) / s1;
      else step = (s0 - exp2f((1.f - 1.f / P.beta) * log2f(s0))) / s1;
      tau += step;
      if (!(step > 2.f * FLT_EPSILON * fmaxf(fabsf(tau), m - tau))) break;
    }
  } else {
    Search sr;
    sr.init(m, len, P.alpha);
    for (int it = 0; it < P.n_iter; ++it) {
      float s0 = 0.f, s1 = 0.f, s2 = 0.f;
      for (int e = lane; e < n_list; e += 32) {
        const float y = entry(e).x - sr.tau;
        if (y > 0.f) {
          float p0, p1, p2;
          entmax_powers<BK>(y, P.beta, p0, p1, p2);
          s0 += p0;
          s1 += p1;
          s2 += p2;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        s0 += __shfl_xor_sync(kFull, s0, o);
        s1 += __shfl_xor_sync(kFull, s1, o);
        s2 += __shfl_xor_sync(kFull, s2, o);
      }
      if (lane == 0) {
        sm.sums[it & 1][warp] = make_float2(s0, s1);
        sm.sums2[it & 1][warp] = s2;
      }
      __syncthreads();
      s0 = s1 = s2 = 0.f;
#pragma unroll
      for (int i = 0; i < kJoinWarps; ++i) {
        s0 += sm.sums[it & 1][i].x;
        s1 += sm.sums[it & 1][i].y;
        s2 += sm.sums2[it & 1][i];
      }
      sr.step<BK>(s0, s1, s2, P.beta);
      if (sr.settled()) break;
    }
    tau = sr.tau;
  }

  // o: each warp adds the values of its entries with p > 0, in 16-byte chunks, D sizeof(T) / 16
  // lanes per row, four rows per lane group in flight
  constexpr int LPR = D * sizeof(T) / 16;  // lanes per value row (8, 16 or 32)
  constexpr int RPW = 32 / LPR;            // value rows per warp load
  constexpr int EPL = 16 / sizeof(T);      // elements per lane
  constexpr int U = 4;
  float o[EPL] = {};
  const int32_t* table = P.tables + b * P.table_stride;
  const T* vbase = static_cast<const T*>(P.v) + hk * P.head_stride + (lane % LPR) * EPL;
  for (int e0 = 0; e0 < n_list; e0 += 32) {
    float p = 0.f;
    int key = 0;
    if (e0 + lane < n_list) {
      const float2 x = entry(e0 + lane);
      p = power<BK>(x.x - tau, P.beta);
      key = __float_as_int(x.y);
    }
    const unsigned live = __ballot_sync(kFull, p > 0.f);
    if (!live) continue;
    const int n = __popc(live);
    if (p > 0.f) {
      const int at = __popc(live & ((1u << lane) - 1u));
      const int blk = key / P.page_size;
      sm.live[warp][at].x = p;
      sm.from[warp][at] = table[blk] * P.page_stride + (key - blk * P.page_size) * P.slot_stride;
    }
    __syncwarp();
    for (int i0 = 0; i0 < n; i0 += RPW * U) {
      uint4 x[U];
      float w[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * RPW + lane / LPR;
        w[j] = 0.f;
        x[j] = make_uint4(0u, 0u, 0u, 0u);
        if (i < n) {
          w[j] = sm.live[warp][i].x;
          x[j] = load_stream(vbase + sm.from[warp][i]);
        }
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const T* v = reinterpret_cast<const T*>(&x[j]);
#pragma unroll
        for (int i = 0; i < EPL; ++i) o[i] = fmaf(w[j], load_elem(v, i), o[i]);
      }
    }
    __syncwarp();
  }
#pragma unroll
  for (int s = LPR; s < 32; s <<= 1)
#pragma unroll
    for (int i = 0; i < EPL; ++i) o[i] += __shfl_xor_sync(kFull, o[i], s);
  if (lane < LPR)
#pragma unroll
    for (int i = 0; i < EPL; ++i) sm.o[warp][lane * EPL + i] = o[i];
  __syncthreads();
  for (int i = tid; i < D; i += kJoinThreads) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kJoinWarps; ++k) s += sm.o[k][i];
    store_elem(out, i, s);
  }
  if (tid == 0) P.tau[row] = tau;
}

// o and tau of a request without keys (o = 0, tau = +inf) or with a length out of range (NaN)
template <typename T, int D>
__device__ __forceinline__ void write_empty(const DecodeProblem& P, int b, int h, bool valid) {
  const int64_t row = static_cast<int64_t>(b) * P.Hq + h;
  T* out = static_cast<T*>(P.out) + row * D;
  for (int i = threadIdx.x; i < D; i += kJoinThreads) store_elem(out, i, valid ? 0.f : NAN);
  if (threadIdx.x == 0) P.tau[row] = valid ? INFINITY : NAN;
}

// ------------------------------------------------------------------ split: two kernels --

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kScoreThreads, 4) decode_scores_kernel(const DecodeProblem P) {
  extern __shared__ __align__(16) char smem[];
  float* sq_all = reinterpret_cast<float*>(smem);  // fp32 only: [warps][8 NT][D]
  int* pre = reinterpret_cast<int*>(
      smem + (sizeof(T) == 4 ? kScoreWarps * 8 * NT * D * sizeof(float) : 0));  // [B + 1]
  __shared__ int scan_buf[kScoreWarps];
  asm volatile("griddepcontrol.launch_dependents;");

  const int tid = threadIdx.x, warp = tid >> 5;
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
    Scorer<T, D, NT> sc;
    sc.load_q(P, b, hg, sq);
    score_run<T, D, NT>(P, sc, sq, b, hg, clamped_len(P, b), first, last,
                        P.parts + (static_cast<int64_t>(w) + static_cast<int64_t>(b) * HG + hg) *
                                      (8 * NT));
  }
}

// One block per (request, query head).
template <typename T, int D, int BK>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const DecodeProblem P) {
  __shared__ JoinSmem sm;
  const int h = blockIdx.x, b = blockIdx.y;
  const int hk = h / P.G, in_group = h - hk * P.G;
  const int hb = in_group / P.heads_per_block, col = in_group - hb * P.heads_per_block;
  const int raw_len = P.lens[b], len = clamped_len(P, b);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (len == 0) {
    write_empty<T, D>(P, b, h, raw_len == 0);
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
  const int2* parts = P.parts + (w0 + static_cast<int64_t>(b) * HG + hg) * P.heads_per_block + col;
  join_head<T, D, BK>(
      P, sm, b, h, len, static_cast<int>(w1 - w0) + 1,
      [&](int i) { return parts[static_cast<int64_t>(i) * P.heads_per_block]; },
      [&](int i) -> int64_t { return i > 0 ? ((w0 + i) * N / nw - A) * 16 : 0; });
}

template <typename T, int D, int NT>
cudaError_t launch_scores(const DecodeProblem& P, cudaStream_t s) {
  const size_t smem = (sizeof(T) == 4 ? kScoreWarps * 8 * NT * D * sizeof(float) : 0) +
                      sizeof(int) * (P.B + 1);
  auto kern = decode_scores_kernel<T, D, NT>;
  if (smem > 47 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  kern<<<kDecodeScoreWarps / kScoreWarps, kScoreThreads, smem, s>>>(P);
  return cudaGetLastError();
}

template <typename T, int D, int BK>
cudaError_t launch_join(const DecodeProblem& P, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(P.Hq, P.B);
  cfg.blockDim = dim3(kJoinThreads);
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
