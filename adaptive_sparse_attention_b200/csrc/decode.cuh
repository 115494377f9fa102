// decode.cuh -- alpha-entmax attention of one new token per request over a paged key-value cache
// (the serving form of the forward pass).  For request b with n = seq_lens[b] keys and query head
// h of kv head h / G:
//   z_j = c q . k_j, c = (alpha - 1) / sqrt(d);   p_j = [z_j - tau]_+^beta, sum_j p_j = 1;
//   o = sum_j p_j v_j
// with key j in slot j % page_size of page block_tables[b][j / page_size].
//
// Two steps.  The scores: every key is read once (for each 16 query heads of its kv head; the form for
// more than 8 spills registers, and one request of 32768 keys and 8 kv heads takes 34.9 us with 16
// query heads each, 24.3 with 8), and per (request, head) the keys that can carry
// p > 0 are kept (z > max - 1, since p <= 1 gives tau >= max - 1).  The join: the max m over all
// parts, tau, and o from the values of the keys with z > tau.  A softmax would have to read every
// value too; here the values of keys with p = 0 are never read, so the traffic is that of the keys
// alone unless the supports are wide.  Both steps run in one kernel (decode_cluster_kernel) for
// small batches, else in two (decode_scores_kernel and a join); choose_decode_kernels picks.
//
// p is made of the differences z - tau, so the join works with z - m and t = tau - m in [-1, 0),
// which fp32 resolves whatever the size of the scores (z - m is exact for z >= m / 2 > 0), and adds
// m only to the tau that it returns: with tau itself 100000 tied keys at z = 30 had a sum of p off
// by 5% (alpha = 2).
//
// What bounds it: HBM reads of the keys; for small calls the chain of dependent reads (length,
// page, keys, candidates, page, value), about 9 us.  In the split kernels the cache is cut in units
// of 16 keys of one kv head; all units of the batch are dealt to the grid's warps in contiguous
// runs of one length, whatever the requests' lengths, so one long request and many ragged ones load
// the GPU alike, and the lengths are needed on the device only.  A run that crosses from one
// (request, kv head) to the next is cut there into parts; part (warp w, group g) has the number w +
// g, which is unique because every cut advances w or g.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"
#include "entmax_attn.h"
#include "kernels.h"

namespace ea {
namespace {

constexpr int kScoreThreads = 128;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kNewtonSteps = 64;  // bounds that no search reaches
constexpr int kHalvings = 64;
constexpr int kSolo = 256;  // candidates of a head that one warp takes alone
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

// 16 bytes that are read once.  (Not ld.global.nc: a block may be set up while the kernel before it
// still writes the cache, so the cache is not read-only for all of this kernel's life.)
__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// The address of this block's shared variable in block `rank` of the cluster.
__device__ __forceinline__ uint32_t remote(const void* p, int rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}

// Stores to the shared memory of another block.
__device__ __forceinline__ void store_remote(uint32_t a, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(x) : "memory");
}
__device__ __forceinline__ void store_remote(uint32_t a, int x) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}
__device__ __forceinline__ void store_remote(uint32_t a, int2 x) {
  asm volatile("st.shared::cluster.v2.s32 [%0], {%1, %2};" ::"r"(a), "r"(x.x), "r"(x.y)
               : "memory");
}
__device__ __forceinline__ void store_remote(uint32_t a, float2 x) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(x.x), "f"(x.y)
               : "memory");
}
// max that keeps a NaN of either side
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// An int that compares as the float does, and back.
__device__ __forceinline__ int ordered(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) {
  return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}

// x = *p if go
__device__ __forceinline__ void load_stream_if(uint4& x, const void* p, bool go) {
  asm volatile(
      "{ .reg .pred q; setp.ne.s32 q, %5, 0;\n\t"
      "@q ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4]; }"
      : "+r"(x.x), "+r"(x.y), "+r"(x.z), "+r"(x.w)
      : "l"(p), "r"(static_cast<int>(go))
      : "memory");
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
  // q of head group hg of request b into registers
  __device__ __forceinline__ void load_q(const DecodeProblem& P, int b, int hg, float*, int,
                                         int) {
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
      float other[4] = {};  // two chains of products: half the latency of one
      acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        mma_bf16(acc[n], a[0][c].x, a[1][c].x, a[0][c].y, a[1][c].y, bq[n][c][0], bq[n][c][1]);
        mma_bf16(other, a[0][c].z, a[1][c].z, a[0][c].w, a[1][c].w, bq[n][c][2], bq[n][c][3]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] += other[i];
    }
  }
};

template <int D, int NT>
struct Scorer<float, D, NT> {
  static constexpr int kChunks = D / 16;
  int heads_;
  // q of head group hg of request b into shared-memory rows [8 NT][D], by thread i of n; the
  // threads that share the rows synchronise before and after
  __device__ __forceinline__ void load_q(const DecodeProblem& P, int b, int hg, float* sq, int i,
                                         int n) {
    const int hk = hg / P.head_blocks, first = (hg - hk * P.head_blocks) * 8 * NT;
    heads_ = min(8 * NT, P.G - first);
    const float* q = static_cast<const float*>(P.q) + b * P.q_stride_b +
                     (hk * P.G + first) * P.q_stride_h;
    for (; i < heads_ * (D / 4); i += n)
      reinterpret_cast<float4*>(sq)[i] = *reinterpret_cast<const float4*>(
          q + (i / (D / 4)) * P.q_stride_h + (i % (D / 4)) * 4);
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
  __device__ __forceinline__ void advance_in_pages_of_16(int page) {
    off += 16;
    if (off >= page) {
      off -= page;
      ++blk;
    }
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
// to part (SHARE: shared memory, of every block of the cluster).  sq: the warp's (or block's)
// shared-memory q rows, fp32 only.  SHARE: the warps of a cluster of `blocks` blocks, all at the
// same heads, tell each other the largest score that they have met (known, one copy per block), so
// that each keeps few candidates beside those of the end: which ones depends on the timing, but the
// join drops all of them again.
// ONE_PAGE: page_size is a multiple of 16, so a unit lies in one page: one lookup for both rows of a
// lane (33 requests with d = 64: 28.3 against 26.9 us; 64 of 16384 tokens 263 against 259).
template <typename T, int D, int NT, bool SHARE, bool ONE_PAGE>
__device__ __forceinline__ void score_run(const DecodeProblem& P,
                                          const Scorer<T, D, NT>& sc, const float* sq, int b,
                                          int hg, int len, int first, int last, int2* part,
                                          int64_t part_stride, int* known, int blocks) {
  using S = Scorer<T, D, NT>;
  constexpr int CH = S::kChunks;
  // 8 KB of keys in flight per warp, in registers: 128 KB per SM with 16 warps, which reads at 6.2
  // TB/s.  (Asynchronous copies into 12 KB of shared memory per warp were slower: 64 requests of
  // 16384 tokens 445 against 342 us.)
  constexpr int DEPTH = 8192 / (16 * D * static_cast<int>(sizeof(T)));
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int hk = hg / P.head_blocks, hb = hg - hk * P.head_blocks;
  const int h0 = hk * P.G + hb * 8 * NT;
  const int heads = min(8 * NT, P.G - hb * 8 * NT);
  const int32_t* table = P.tables + b * P.table_stride;
  const T* kbase = static_cast<const T*>(P.k) + hk * P.head_stride + t * (16 / sizeof(T));

  float m[NT][2];     // the largest score known, from which the threshold follows
  float own[NT][2];   // this lane's largest score; NaN once it has met one
  float none[NT][2];  // added to the scores: -inf for columns without a head
  int cnt[NT][2];
  int2* cand[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[n][e] = own[n][e] = -INFINITY;
      cnt[n][e] = 0;
      const int h = n * 8 + 2 * t + e;
      none[n][e] = h < heads ? 0.f : -INFINITY;
      cand[n][e] = P.cand + (static_cast<int64_t>(b) * P.Hq + h0 + min(h, heads - 1)) *
                                P.cand_stride + first * 16;
    }
  bool bad_page = false;

  // Pipeline: the keys of the next DEPTH units are in registers or on their way, the page numbers
  // of the unit after those too.  No load is predicated per row: rows past the last key take the
  // page of the last key, and a page that does not exist page 0 (the part is then marked NaN), so
  // every address lies in the cache; their scores are masked below.
  const int page_size = P.page_size, last_blk = (len - 1) / page_size;
  RowCursor cur[2];
  cur[0].start(first * 16 + g, page_size);
  cur[1].start(first * 16 + g + 8, page_size);
  int fetch = first;  // unit the cursors stand at
  int page[2], off[2];
  auto next_pages = [&]() {
    off[0] = cur[0].off;
    page[0] = table[min(cur[0].blk, last_blk)];
    if (ONE_PAGE) {
      off[1] = off[0] + 8;
      page[1] = page[0];
      cur[0].advance_in_pages_of_16(page_size);
    } else {
      off[1] = cur[1].off;
      page[1] = table[min(cur[1].blk, last_blk)];
      cur[0].advance(page_size);
      cur[1].advance(page_size);
    }
  };
  uint4 unit[DEPTH][2][CH];
  auto load_unit = [&](uint4 (&x)[2][CH]) {
    const bool go = fetch < last;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool exists = static_cast<unsigned>(page[i]) < static_cast<unsigned>(P.num_pages);
      bad_page |= !exists;
      const T* row = kbase + (exists ? page[i] : 0) * P.page_stride + off[i] * P.slot_stride;
#pragma unroll
      for (int c = 0; c < CH; ++c) load_stream_if(x[i][c], row + c * (64 / sizeof(T)), go);
    }
    ++fetch;
  };
  next_pages();
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int c = 0; c < CH; ++c) unit[i][r][c] = make_uint4(0u, 0u, 0u, 0u);
    load_unit(unit[i]);
    next_pages();
  }
  // known is set in every block
  if (SHARE) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
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
          for (int e = 0; e < 2; ++e) {
            acc[n][e] = fmaf(P.c, acc[n][e], none[n][e]);
            acc[n][2 + e] = fmaf(P.c, acc[n][2 + e], none[n][e]);
          }
        if (blk * 16 + 16 > len) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key + 8 * (e >> 1) >= len) acc[n][e] = -INFINITY;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float top = max_nan(acc[n][e], acc[n][2 + e]);
            own[n][e] = max_nan(own[n][e], top);
            pass |= top - m[n][e] > -1.f;
          }
        if (__any_sync(kFull, pass)) {
          bool above = false;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (SHARE)
                m[n][e] = fmaxf(
                    m[n][e], unordered(*static_cast<volatile int*>(known + n * 8 + 2 * t + e)));
              above |= fmaxf(acc[n][e], acc[n][2 + e]) > m[n][e];
            }
          if (__any_sync(kFull, above)) {  // a new maximum
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float x = fmaxf(acc[n][e], acc[n][2 + e]);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
                if (SHARE && x > m[n][e] && g < blocks)  // lane 4 g + t tells block g
                  asm volatile("red.relaxed.cluster.shared::cluster.max.s32 [%0], %1;" ::"r"(
                                   remote(known + n * 8 + 2 * t + e, g)),
                               "r"(ordered(x))
                               : "memory");
                m[n][e] = fmaxf(m[n][e], x);
              }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const float z = acc[n][2 * r + e];
                const bool in = z - m[n][e] > -1.f;  // also where m - 1 rounds to m
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
  bad_page = __any_sync(kFull, bad_page);
  if (bad_page && lane == 0) atomicMax(P.status, ENTMAX_ATTN_ERANGE);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = own[n][e];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) x = max_nan(x, __shfl_xor_sync(kFull, x, o));
      // NaN also stands for +inf and for a page that does not exist
      const int2 y = make_int2(cnt[n][e], __float_as_int(x < INFINITY && !bad_page ? x : NAN));
      int2* to = part + (n * 8 + 2 * t + e) * part_stride;
      if (SHARE) {  // lane 4 g + t tells block g
        if (g < blocks) store_remote(remote(to, g), y);
      } else if (g == 0) {
        *to = y;
      }
    }
}

// x^beta for x > 0 (or 0 where x <= 0), to a few units of the last place: near beta = 3 the cube
// times x^(beta - 3), whose exponent is small enough for the fast logarithm's error.
__device__ __forceinline__ float tiny_power(float x, float f) {  // x^f for |f| <= kNearIntFrac
  return exp2f(f * __log2f(fmaxf(x, 1e-30f)));
}
template <int BK>
__device__ __forceinline__ float power(float x, float beta) {
  if (!(x > 0.f)) return 0.f;
  if (BK == kBetaOne) return x;
  if (BK == kBetaTwo) return x * x;
  if (BK == kBetaNear3) return (x * x) * (x * tiny_power(x, beta - 3.f));
  return exp2f(beta * log2f(x));
}

// Shared memory of a join by C blocks of W warps.
template <int W, int C = 1>
struct JoinSmem {
  static constexpr int kList = 256;  // candidates per warp kept here
  struct Row {
    int64_t from;  // offset of a value row
    float p;
  };
  union {
    float2 list[W][kList];  // (z - m or p, key bits)
    float o[W][128];        // after the lists: partial sums of o
  };
  float2 all[W > 1 ? kSolo : 1];  // all candidates, when they are few
  Row rows[W][32];
  float2 sums[2][C * W];
  float2 bound;  // m and the bound of t, one pair for the whole join
  float red[W];
  int count[C * W];
  float co[C > 1 ? C : 1][C > 1 ? 128 : 1];  // the blocks' sums of o
};

// What orders the C W warps of a join.
template <int W, int C>
__device__ __forceinline__ void join_sync() {
  if (C > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else if (W == 1) {
    __syncwarp();
  } else {
    __syncthreads();
  }
}

// x into *p of every block of the join, by one warp
template <int C, typename V>
__device__ __forceinline__ void share(V* p, V x) {
  const int lane = threadIdx.x & 31;
  if (C > 1) {
    if (lane < C) store_remote(remote(p, lane), x);
  } else if (lane == 0) {
    *p = x;
  }
}

// One step towards t from the left, for beta >= 1 (here tau stands for t, z for z - m): Newton's on
// the norm g(tau) = (sum [z - tau]_+^beta)^(1/beta), which is 1 at tau.  g is convex and falling (a norm of
// functions that are), so from a point where g >= 1 the iterates rise to the root and never pass
// it, and g is linear in tau while the support stays and the scores tie, so they are few: 4 or 5
// on normal scores, 14 at most over a wide sweep of sizes and spreads at beta = 1.  With s0, s1
// the sums of the powers beta and beta - 1, (g - 1) / -g' = (s0 - s0^(1 - 1/beta)) / s1; near the
// root (s0 - 1) / (beta s1) to first order, which does not cancel.
template <int BK>
__device__ __forceinline__ float norm_step(float s0, float s1, float beta) {
  float rise;
  if (BK == kBetaOne) rise = s0 - 1.f;
  else if (s0 < 1.01f) rise = (s0 - 1.f) * (BK == kBetaTwo ? 0.5f : 1.f / beta);
  else if (BK == kBetaTwo) rise = s0 - s0 * rsqrtf(s0);
  else rise = s0 - exp2f((1.f - 1.f / beta) * __log2f(s0));
  return __fdividef(rise, s1);
}
// adds x^beta and x^(beta - 1) for x = [z - tau]_+
template <int BK>
__device__ __forceinline__ void norm_add(float x, float beta, float& s0, float& s1) {
  float q;  // x^(beta - 1), 0 at x = 0
  if (BK == kBetaOne) q = x > 0.f ? 1.f : 0.f;
  else if (BK == kBetaTwo) q = x;
  else if (BK == kBetaNear3) q = x * (x * tiny_power(x, beta - 3.f));
  else q = x > 0.f ? exp2f((beta - 1.f) * log2f(x)) : 0.f;
  s1 += q;
  s0 = fmaf(q, x, s0);
}
__device__ __forceinline__ void warp_sum2(float& a, float& b) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(kFull, a, o);
    b += __shfl_xor_sync(kFull, b, o);
  }
}

// The parts of one (request, query head): part i holds the candidates of the keys from key0(i) on.
struct Parts {
  const int2* info;      // (count, max bits) of each
  int np;                // number of parts
  int most;              // no more than this, whatever the workspace holds
  int run, off, nb;      // part i starts at unit i run - off of the nb units of the request
  __device__ __forceinline__ int2 part(int i) const { return info[i]; }
  __device__ __forceinline__ int key0(int i) const { return min(max(i * run - off, 0), nb) * 16; }
};

// From the maxima of a head's parts: its largest score m, and a lower bound of t = tau - m.  The
// maxima are scores of the head, and the tau of a part of the keys is at most that of all (more keys
// only add to the sum), so a few of the steps above on up to 256 of them give a bound far above -1:
// of 20000 normal scores at alpha = 1.333, 184 lie above tau, 226 above the bound from 64 maxima
// and 3496 above m - 1.  Where at most half of the parts reach above m - 1 the candidates are few
// and the bound is -1.  (The parts' counts do not enter: in the cluster kernel they depend on
// the timing, and the bound decides in which order the sums below add.)  Every warp computes both,
// so that they need no barrier; red: where there may be more than 256 parts, whose maximum the block
// takes together.
struct Bounds {
  float m, floor;  // floor: of t
};
template <int BK, int W>
__device__ __forceinline__ Bounds part_bounds(const DecodeProblem& P, float* red,
                                              const Parts& parts) {
  const int np = parts.np;
  constexpr int R = 8;
  const int lane = threadIdx.x & 31;
  float x[R];
  Bounds r;
  r.m = -INFINITY;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    x[j] = lane + 32 * j < np ? __int_as_float(parts.part(lane + 32 * j).y) : -INFINITY;
    r.m = max_nan(r.m, x[j]);
  }
  if (np > 32 * R)
    for (int i = 32 * R + (W == 1 ? lane : threadIdx.x); i < np; i += 32 * W)
      r.m = max_nan(r.m, __int_as_float(parts.part(i).y));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) r.m = max_nan(r.m, __shfl_xor_sync(kFull, r.m, o));
  if (W > 1 && parts.most > 32 * R) {
    if (lane == 0) red[threadIdx.x >> 5] = r.m;
    __syncthreads();
    r.m = red[lane % W];
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) r.m = max_nan(r.m, __shfl_xor_sync(kFull, r.m, o));
  }
  r.floor = -1.f;
  int n = 0;  // parts that reach above m - 1
#pragma unroll
  for (int j = 0; j < R; ++j) {
    x[j] -= r.m;  // an m of -inf or NaN is refused by the join
    n += __popc(__ballot_sync(kFull, x[j] > -1.f));
  }
  if (2 * n > min(np, 32 * R) && (BK != kBetaGeneral || P.beta >= 1.f)) {
    for (int it = 0; it < 3; ++it) {
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (32 * j < np) norm_add<BK>(fmaxf(x[j] - r.floor, 0.f), P.beta, s0, s1);
      warp_sum2(s0, s1);
      r.floor += norm_step<BK>(s0, s1, P.beta);
    }
    // the steps' rounding: s0 and s1 add 8 terms and 5 partial sums, 13 units of 2^-24 each
    r.floor = fmaxf(r.floor - 16.f * FLT_EPSILON, -1.f);
  }
  return r;
}

// C blocks (a cluster) of W warps, or one warp of a block for W = 1, join the parts of one
// (request, query head) with these bounds.
template <typename T, int D, int BK, int W, int C>
__device__ __forceinline__ void join_head(const DecodeProblem& P, JoinSmem<W, C>& sm, int rank,
                                          int b, int h, int len, Bounds bound,
                                          const Parts& parts) {
  const int np = parts.np;
  constexpr int kThreads = 32 * W;
  constexpr int kAll = C * W;  // warps of the join
  constexpr int kList = JoinSmem<W, C>::kList;
  const int lane = threadIdx.x & 31, warp = W == 1 ? 0 : threadIdx.x >> 5;
  const int me = rank * W + warp;
  float m = bound.m, floor = bound.floor;
  const int tid = W == 1 ? lane : threadIdx.x;
  const int hk = h / P.G;
  const int64_t row = static_cast<int64_t>(b) * P.Hq + h;
  T* out = static_cast<T*>(P.out) + row * D;
  auto undefined = [&]() {
    if (rank == 0) {
      for (int i = tid; i < D; i += kThreads) store_elem(out, i, NAN);
      if (tid == 0) P.tau[row] = NAN;
    }
  };

  // Each warp compacts the entries above the bound of a contiguous range of parts, in order and as
  // (z - m, key): the first kList into shared memory, the others back to the front of the range (an
  // entry only moves forward, over places that the warp has read already, since it reads them in
  // order).
  int2* cand = P.cand + row * P.cand_stride;
  const int i_end = (me + 1) * np / kAll;
  const int i_beg = me * np / kAll;
  int2* spill = cand + (i_beg < i_end ? parts.key0(i_beg) : 0);
  const unsigned below = (1u << lane) - 1u;
  int n_list = 0;
  for (int i0 = i_beg; i0 < i_end; i0 += 32) {
    // 32 parts as one sequence of chunks of up to 32 entries: lane i's part owns the chunks from
    // first on, chunk c of it is at cand[base + 32 c ..), its entries end at 32 c + lane < limit
    int n = 0, first, base = 0;
    if (i0 + lane < i_end) {
      const int2 x = parts.part(i0 + lane);
      base = parts.key0(i0 + lane);
      if (__int_as_float(x.y) - m > floor)
        n = min(max(x.x, 0), min(parts.run, parts.nb - (base >> 4)) * 16);
    }
    const int chunks = (n + 31) >> 5;
    first = chunks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, first, o);
      if (lane >= o) first += y;
    }
    const int total = __shfl_sync(kFull, first, 31);
    first -= chunks;
    base -= 32 * first;
    const int limit = 32 * first + n;
    constexpr int U = 8;  // loads in flight per lane
    for (int c0 = 0; c0 < total; c0 += U) {
      int2 x[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int c = c0 + j;
        // its part is the last that starts at or before it (a part without chunks starts where
        // the next one does)
        const int own = 31 - __clz(__ballot_sync(kFull, first <= c));
        const int at = __shfl_sync(kFull, base, own) + 32 * c + lane;
        const int end = __shfl_sync(kFull, limit, own);
        x[j] = make_int2(__float_as_int(-INFINITY), 0);
        if (c < total && 32 * c + lane < end) x[j] = cand[at];
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const float z = __int_as_float(x[j].x) - m;
        const bool in = z > floor;
        const unsigned bal = __ballot_sync(kFull, in);
        const int at = n_list + __popc(bal & below);
        if (in) {
          if (at < kList) sm.list[warp][at] = make_float2(z, __int_as_float(x[j].y));
          else spill[at - kList] = make_int2(__float_as_int(z), x[j].y);
        }
        n_list += __popc(bal);
      }
    }
  }
  // When the candidates are few, the first warp takes them all and finds tau and the p by itself,
  // with no sum over the warps or blocks per step, and deals the values to add to its block's
  // warps.
  // All blocks and warps go by one m and bound, so that each takes the same barriers and no block
  // leaves while another stores into its shared memory, whatever another call that was given the same
  // workspace wrote in between.
  bool solo = W == 1;
  if (W > 1) {
    share<C>(&sm.count[me], n_list);
    if (me == 0) share<C>(&sm.bound, make_float2(m, floor));
    join_sync<W, C>();
    m = sm.bound.x;
    floor = sm.bound.y;
  }
  if (!(m > -INFINITY)) return undefined();  // a NaN, or every score -inf: p is not defined
  if (W > 1) {
    // inclusive scan of the counts, lane l holding those of warps K l .. K l + K - 1
    constexpr int K = kAll > 32 ? kAll / 32 : 1;
    int x = 0;
#pragma unroll
    for (int i = 0; i < K; ++i)
      if (K * lane + i < kAll) x += sm.count[K * lane + i];
    const int own = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    const int total = __shfl_sync(kFull, x, 31);
    if (total <= kSolo) {
      int at = __shfl_sync(kFull, x - own, me / K);
      for (int i = 0; i < me % K; ++i) at += sm.count[me / K * K + i];
      for (int e = lane; e < n_list; e += 32) {  // n_list <= kSolo <= kList
        if (C > 1) store_remote(remote(&sm.all[at + e], 0), sm.list[warp][e]);
        else sm.all[at + e] = sm.list[warp][e];
      }
      n_list = total;
      solo = true;
      join_sync<W, C>();
      if (C > 1 && rank != 0) return;
    }
  }
  __syncwarp();
  if (solo && n_list == 0) return undefined();  // only where another call writes the workspace
  const bool deal = W > 1 && solo;
  float2* list = deal ? sm.all : sm.list[warp];
  auto entry = [&](int e) {
    if (e < kList) return list[e];  // all of them when solo: kSolo <= kList
    const int2 x = spill[e - kList];
    return make_float2(__int_as_float(x.x), __int_as_float(x.y));
  };
  auto set_entry = [&](int e, float z, int key) {
    if (e < kList) list[e] = make_float2(z, __int_as_float(key));
    else spill[e - kList] = make_int2(__float_as_int(z), key);
  };

  // tau - m, called tau from here on: for beta >= 1 by the steps of norm_step from the lower bound,
  // until it has settled; for beta < 1 by bisection, because the sum falls with an infinite slope at
  // every score, where steps by derivatives stall short of the root (the attention passes' search
  // left sums of p up to 2000 off).
  // A list of up to 32 candidates (quick) is held one per lane, and their values' places are looked
  // up while tau is found.
  float tau = 0.f;
  int n_live = 0;  // candidates with p > 0
  const int32_t* table = P.tables + b * P.table_stride;
  auto value_row = [&](float2 x) -> int64_t {  // offset of the value of list entry x
    const int key = min(static_cast<unsigned>(__float_as_int(x.y)),
                        static_cast<unsigned>(len - 1));
    const int blk = key / P.page_size, page = table[blk];
    return (static_cast<unsigned>(page) < static_cast<unsigned>(P.num_pages) ? page : 0) *
               P.page_stride +
           (key - blk * P.page_size) * P.slot_stride;
  };
  const bool quick = solo && n_list <= 32 && (BK != kBetaGeneral || P.beta >= 1.f);
  if (deal && warp != 0) {
    // waits for the first warp below
  } else if (quick) {
    float z = -INFINITY;
    int64_t from = 0;
    if (lane < n_list) {
      const float2 x = entry(lane);
      z = x.x;
      from = value_row(x);
    }
    tau = floor;
    for (int it = 0; it < kNewtonSteps; ++it) {
      float s0 = 0.f, s1 = 0.f;
      norm_add<BK>(fmaxf(z - tau, 0.f), P.beta, s0, s1);
      warp_sum2(s0, s1);
      const float step = norm_step<BK>(s0, s1, P.beta);
      tau += step;
      if (!(step > 2.f * FLT_EPSILON * fabsf(tau))) break;
    }
    const float p = power<BK>(z - tau, P.beta);
    const unsigned live = __ballot_sync(kFull, p > 0.f);
    if (p > 0.f) sm.rows[0][__popc(live & below)] = {from, p};
    n_live = __popc(live);
  } else if (BK != kBetaGeneral || P.beta >= 1.f) {
    tau = floor;
    for (int it = 0; it < kNewtonSteps; ++it) {
      float s0 = 0.f, s1 = 0.f;
      for (int e0 = lane; e0 < n_list; e0 += 128) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = e0 + 32 * j;
          x[j] = e < n_list ? fmaxf(entry(e).x - tau, 0.f) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) norm_add<BK>(x[j], P.beta, s0, s1);
      }
      warp_sum2(s0, s1);
      if (W > 1 && !solo) {
        share<C>(&sm.sums[it & 1][me], make_float2(s0, s1));
        join_sync<W, C>();  // two buffers: the next step writes the other one
        s0 = s1 = 0.f;
#pragma unroll
        for (int i = lane % kAll; i < kAll; i += 32) {
          const float2 x = sm.sums[it & 1][i];
          s0 += x.x;
          s1 += x.y;
        }
#pragma unroll
        for (int o = (kAll < 32 ? kAll : 32) / 2; o > 0; o >>= 1) {
          s0 += __shfl_xor_sync(kFull, s0, o);
          s1 += __shfl_xor_sync(kFull, s1, o);
        }
      }
      const float step = norm_step<BK>(s0, s1, P.beta);
      tau += step;
      if (!(step > 2.f * FLT_EPSILON * fabsf(tau))) break;
    }
  } else {
    // [-1, -n^(1 - alpha)] holds the root: p <= 1, and n keys at most 0 have it at the upper end when
    // all tie there (moved by the rounding of the power).  Halved until its ends are neighbours, by
    // the geometric mean while they lie far apart: 24 to 35 steps.
    float lo = -1.f, hi = -0.9999f * fmaxf(exp2f((1.f - P.alpha) * log2f(len)), FLT_MIN);
    float over = INFINITY, under = 1.f;  // how far the sum is from 1 at lo and at hi
    for (int it = 0; it < kHalvings; ++it) {
      const float mid = lo < 4.f * hi ? -sqrtf(-lo) * sqrtf(-hi) : 0.5f * (lo + hi);
      if (!(mid > lo && mid < hi)) break;
      float s0 = 0.f;
      for (int e = lane; e < n_list; e += 32) s0 += power<BK>(entry(e).x - mid, P.beta);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s0 += __shfl_xor_sync(kFull, s0, o);
      if (W > 1 && !solo) {
        share<C>(&sm.sums[it & 1][me], make_float2(s0, 0.f));
        join_sync<W, C>();
        s0 = 0.f;
        for (int i = 0; i < kAll; ++i) s0 += sm.sums[it & 1][i].x;
      }
      if (s0 > 1.f) {
        lo = mid;
        over = s0 - 1.f;
      } else {
        hi = mid;
        under = 1.f - s0;
      }
    }
    tau = over < under ? lo : hi;
  }

  // The entries with p > 0 move to the front of the list, p in the place of z ...
  if (!quick && (!deal || warp == 0)) {
    for (int e0 = 0; e0 < n_list; e0 += 32) {
      float p = 0.f;
      int key = 0;
      if (e0 + lane < n_list) {
        const float2 x = entry(e0 + lane);
        p = power<BK>(x.x - tau, P.beta);
        key = __float_as_int(x.y);
      }
      const unsigned live = __ballot_sync(kFull, p > 0.f);
      if (p > 0.f) set_entry(n_live + __popc(live & below), p, key);
      n_live += __popc(live);
    }
  }
  if (deal) {
    if (threadIdx.x == 0) sm.count[0] = n_live;
    __syncthreads();
    n_live = sm.count[0];
  } else {
    __syncwarp();
  }
  const int step = deal ? W : 1, mine = deal ? warp : 0;  // this warp's entries: mine + i step
  n_live = (n_live - mine + step - 1) / step;
  // ... and their values are added in 16-byte chunks, D sizeof(T) / 16 lanes per row, four rows
  // per lane group in flight.
  constexpr int LPR = D * sizeof(T) / 16;  // lanes per value row (8, 16 or 32)
  constexpr int RPW = 32 / LPR;            // value rows per warp load
  constexpr int EPL = 16 / sizeof(T);      // elements per lane
  constexpr int U = 4;
  float o[EPL] = {};
  const typename JoinSmem<W, C>::Row* rows = quick ? sm.rows[0] + mine : sm.rows[warp];
  const int row_step = quick ? step : 1;
  const T* vbase = static_cast<const T*>(P.v) + hk * P.head_stride + (lane % LPR) * EPL;
  for (int e0 = 0; e0 < n_live; e0 += 32) {
    const int n = min(32, n_live - e0);
    if (!quick) {
      if (lane < n) {
        const float2 x = entry(mine + (e0 + lane) * step);
        sm.rows[warp][lane] = {value_row(x), x.x};
      }
      __syncwarp();
    }
    for (int i0 = 0; i0 < n; i0 += RPW * U) {
      uint4 x[U];
      float w[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * RPW + lane / LPR;
        w[j] = 0.f;
        x[j] = make_uint4(0u, 0u, 0u, 0u);
        if (i < n) {
          w[j] = rows[i * row_step].p;
          x[j] = load_stream(vbase + rows[i * row_step].from);
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
  join_sync<W, 1>();  // the lists are no longer needed
  if (lane < LPR)
#pragma unroll
    for (int i = 0; i < EPL; ++i) sm.o[warp][lane * EPL + i] = o[i];
  join_sync<W, 1>();
  for (int i = tid; i < D; i += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) s += sm.o[k][i];
    if (C > 1 && !solo) store_remote(remote(&sm.co[rank][i], 0), s);
    else store_elem(out, i, s);
  }
  if (C > 1 && !solo) {
    join_sync<W, C>();
    if (rank == 0)
      for (int i = tid; i < D; i += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < C; ++k) s += sm.co[k][i];
        store_elem(out, i, s);
      }
  }
  if (rank == 0 && tid == 0) P.tau[row] = m + tau;
}

// o and tau of a request without keys (o = 0, tau = +inf) or with a length out of range (NaN)
template <typename T, int D>
__device__ __forceinline__ void write_empty(const DecodeProblem& P, int b, int h, bool valid,
                                            int tid, int threads) {
  const int64_t row = static_cast<int64_t>(b) * P.Hq + h;
  T* out = static_cast<T*>(P.out) + row * D;
  for (int i = tid; i < D; i += threads) store_elem(out, i, valid ? 0.f : NAN);
  if (tid == 0) P.tau[row] = valid ? INFINITY : NAN;
}

// ------------------------------------------------------------------ split: two kernels --

// The split kernels keep the parts of one head of the groups (the first, second, ... of each
// group) side by side: this many.
__device__ __forceinline__ int64_t split_part_stride(const DecodeProblem& P) {
  return P.score_warps + static_cast<int64_t>(P.B) * P.Hkv * P.head_blocks;
}

// 1.6 GB of keys (64 requests of 8000 to 16384 tokens) take 250 us, 6.4 TB/s, the copy rate; 268 MB
// (one request of 131072) 48 us, 5.6 TB/s: the ramp-up and the tail of 28 units per warp.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kScoreThreads, 4) decode_scores_kernel(const DecodeProblem P) {
  extern __shared__ __align__(16) char smem[];
  float* sq_all = reinterpret_cast<float*>(smem);  // fp32 only: [warps][8 NT][D]
  int* pre = reinterpret_cast<int*>(
      smem + (sizeof(T) == 4 ? kScoreWarps * 8 * NT * D * sizeof(float) : 0));  // [B + 1]
  __shared__ int scan_buf[kScoreWarps];
  const int tid = threadIdx.x, warp = tid >> 5;
  serial_wait();
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
  const int N = pre[P.B] * HG;           // below 2^31, see decode_layout
  const int run = (N + P.score_warps - 1) / P.score_warps;
  const int w = blockIdx.x * kScoreWarps + warp;
  int u = w * run;  // at most score_warps more than N
  const int u_end = min(u + run, N);
  float* sq = sq_all + warp * 8 * NT * D;

  while (u < u_end) {
    // the request of unit u: the last b with pre[b] <= u / HG (empty requests have pre[b + 1] =
    // pre[b] and are never last)
    const int v = u / HG;
    int lo = 0, hi = P.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= v) lo = mid;
      else hi = mid - 1;
    }
    const int b = lo;
    const int nb = pre[b + 1] - pre[b];
    const int r = u - pre[b] * HG;
    const int hg = r / nb;
    const int first = r - hg * nb;
    const int last = min(nb, first + (u_end - u));
    u += last - first;
    Scorer<T, D, NT> sc;
    __syncwarp();
    sc.load_q(P, b, hg, sq, tid & 31, 32);
    __syncwarp();
    auto score = [&](auto one_page) {
      score_run<T, D, NT, false, decltype(one_page)::value>(
          P, sc, sq, b, hg, clamped_len(P, b), first, last,
          P.parts + (static_cast<int64_t>(w) + static_cast<int64_t>(b) * HG + hg),
          split_part_stride(P), nullptr, 1);
    };
    if (P.page_size % 16 == 0) score(std::true_type());
    else score(std::false_type());
  }
}

// The parts of one (request, query head) in the score kernel's numbering.
__device__ __forceinline__ Parts split_parts(const DecodeProblem& P, int b, int h, int len) {
  const int hk = h / P.G, in_group = h - hk * P.G;
  const int hb = in_group / P.heads_per_block, col = in_group - hb * P.heads_per_block;
  const int HG = P.Hkv * P.head_blocks, hg = hk * P.head_blocks + hb;
  Parts r;
  r.nb = (len + 15) >> 4;
  r.most = r.nb;
  // What is read from the workspace is clamped throughout the join and decides about no barrier (see
  // join_head), so that one that another call overwrites meanwhile spoils the results but sends no
  // access outside and leaves no block waiting.
  const int units = min(max(P.pre[P.B], r.nb), static_cast<int>(P.B * (P.cand_stride >> 4)));
  r.run = (units * HG + P.score_warps - 1) / P.score_warps;
  const int A = min(max(P.pre[b], 0), units - r.nb) * HG + hg * r.nb;  // the group's first unit
  const int w0 = A / r.run;
  r.off = A - w0 * r.run;
  r.np = (A + r.nb - 1) / r.run - w0 + 1;
  r.info = P.parts + col * split_part_stride(P) + w0 + static_cast<int64_t>(b) * HG + hg;
  return r;
}

// A cluster of C blocks of 8 warps per (request, query head).  About 8 us with few candidates, 20
// us for 128 heads with up to 14000 (lengths to 20000, alpha = 1.333, no spikes): a chain of reads.
constexpr int kJoinWarps = 8;
template <typename T, int D, int BK, int C>
__global__ void __launch_bounds__(32 * kJoinWarps) decode_join_kernel(const DecodeProblem P) {
  __shared__ JoinSmem<kJoinWarps, C> sm;
  const int rank = C > 1 ? blockIdx.x : 0;
  const int h = blockIdx.y, b = blockIdx.z;
  serial_wait();
  const int raw_len = P.lens[b], len = clamped_len(P, b);
  if (len == 0) {
    if (rank == 0) write_empty<T, D>(P, b, h, raw_len == 0, threadIdx.x, 32 * kJoinWarps);
    return;
  }
  // every block runs before any stores into its shared memory
  if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const Parts parts = split_parts(P, b, h, len);
  const Bounds bound = part_bounds<BK, kJoinWarps>(P, sm.red, parts);
  if (C > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  join_head<T, D, BK, kJoinWarps, C>(P, sm, rank, b, h, len, bound, parts);
}

// One warp per head, up to eight heads to a block.  DEFER: a head with more than kWarpEntries
// candidates is left to the whole block, unless half of the warps have one.  (Not in the cluster
// kernel, where the counts depend on the timing; its requests are short.)
constexpr int kWarpEntries = 768;
struct ManySmem {
  union {
    JoinSmem<kJoinWarps> block;
    JoinSmem<1> warp[kJoinWarps];
  };
  Bounds bound[kJoinWarps];
  int heavy;
};
// Head(w) gives the b, h, length and parts of warp w's head; valid: this warp has one.
struct HeadRef {
  int b, h, len;
  Parts parts;
};
template <typename T, int D, int BK, bool DEFER, typename Head>
__device__ __forceinline__ void join_many(const DecodeProblem& P, ManySmem& sm, bool valid,
                                          const Head& head) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (DEFER) {
    if (threadIdx.x == 0) sm.heavy = 0;
    __syncthreads();
  }
  if (valid) {
    const HeadRef r = head(warp);
    const Bounds bound = part_bounds<BK, 1>(P, nullptr, r.parts);
    int n = 0;
    if (DEFER)
      for (int i = lane; i < r.parts.np; i += 32) {
        const int2 x = r.parts.part(i);
        if (__int_as_float(x.y) - bound.m > bound.floor) n += x.x;
      }
    if (DEFER && __reduce_add_sync(kFull, n) > kWarpEntries) {
      if (lane == 0) {
        sm.bound[warp] = bound;
        atomicOr(&sm.heavy, 1 << warp);
      }
    } else {
      join_head<T, D, BK, 1, 1>(P, sm.warp[warp], 0, r.b, r.h, r.len, bound, r.parts);
    }
  }
  if (!DEFER) return;
  __syncthreads();
  const int todo = sm.heavy;
  if (__popc(todo) >= kJoinWarps / 2) {
    if (todo >> warp & 1) {
      const HeadRef r = head(warp);
      join_head<T, D, BK, 1, 1>(P, sm.warp[warp], 0, r.b, r.h, r.len, sm.bound[warp], r.parts);
    }
    return;
  }
  for (int left = todo; left; left &= left - 1) {
    const int w = __ffs(left) - 1;
    const HeadRef r = head(w);
    join_head<T, D, BK, kJoinWarps, 1>(P, sm.block, 0, r.b, r.h, r.len, sm.bound[w], r.parts);
    __syncthreads();  // shared memory of this head
  }
}

template <typename T, int D, int BK>
__global__ void __launch_bounds__(32 * kJoinWarps) decode_join_many_kernel(const DecodeProblem P) {
  __shared__ ManySmem sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t rows = static_cast<int64_t>(P.B) * P.Hq;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kJoinWarps;
  serial_wait();
  auto head = [&](int w) {
    HeadRef r;
    r.b = static_cast<int>((row0 + w) / P.Hq);
    r.h = static_cast<int>(row0 + w - static_cast<int64_t>(r.b) * P.Hq);
    r.len = clamped_len(P, r.b);
    r.parts = split_parts(P, r.b, r.h, r.len);
    return r;
  };
  bool valid = row0 + warp < rows;
  if (valid) {
    const int b = static_cast<int>((row0 + warp) / P.Hq);
    const int h = static_cast<int>(row0 + warp - static_cast<int64_t>(b) * P.Hq);
    const int raw_len = P.lens[b];
    if (clamped_len(P, b) == 0) {
      write_empty<T, D>(P, b, h, raw_len == 0, lane, 32);
      valid = false;
    }
  }
  join_many<T, D, BK, true>(P, sm, valid, head);
}

template <typename T, int D, int NT>
cudaError_t launch_scores(const DecodeProblem& P, cudaStream_t s) {
  auto bytes = [](int B) {
    return (sizeof(T) == 4 ? kScoreWarps * 8 * NT * D * sizeof(float) : 0) + sizeof(int) * (B + 1);
  };
  auto kern = decode_scores_kernel<T, D, NT>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kern, bytes(kMaxRequests), done);
  if (e != cudaSuccess) return e;
  const size_t smem = bytes(P.B);
  return launch_serial(kern, dim3(kDecodeScoreWarps / kScoreWarps), dim3(kScoreThreads), smem, s,
                       1, P);
}

template <typename T, int D, int BK>
cudaError_t launch_join(const DecodeProblem& P, cudaStream_t s) {
  const dim3 block(32 * kJoinWarps);
  if (P.join_blocks == 0) {
    const int64_t rows = static_cast<int64_t>(P.B) * P.Hq;
    const dim3 grid(static_cast<unsigned>((rows + kJoinWarps - 1) / kJoinWarps));
    return launch_serial(decode_join_many_kernel<T, D, BK>, grid, block, 0, s, 1, P);
  }
  const dim3 grid(P.join_blocks, P.Hq, P.B);
  return P.join_blocks == 4
             ? launch_serial(decode_join_kernel<T, D, BK, 4>, grid, block, 0, s, 4, P)
             : launch_serial(decode_join_kernel<T, D, BK, 1>, grid, block, 0, s, 1, P);
}

// ------------------------------------------------------------------ cluster: one kernel --

// A cluster of P.cluster (1 to 8) blocks scores one (request, head group), each of its warps an
// equal run of units, and after a cluster barrier its blocks join the group's heads.  One launch
// and no prefix sums: less latency than the split kernels, as long as all clusters run at once.
// One request of 1000 tokens takes 8.6 us, 4 of 16384 30 us (4.4 TB/s); a block alone on its SM
// reads 44 GB/s, 64 KB in flight over a latency of 1.4 us.
constexpr int kClusterBlocks = 8;  // at most
template <typename T, int D, int NT, int BK>
__global__ void __launch_bounds__(32 * kJoinWarps, 2) decode_cluster_kernel(const DecodeProblem P) {
  __shared__ union {
    JoinSmem<kJoinWarps> block;
    ManySmem many;
  } sm;
  __shared__ __align__(16) float sq[sizeof(T) == 4 ? 8 * NT * D : 4];
  __shared__ int known[8 * NT];  // ordered(): the largest score of each head in the cluster so far
  __shared__ int2 info[8 * NT * kClusterBlocks * kJoinWarps];  // [head][part]
  const int tid = threadIdx.x, warp = tid >> 5;
  const int blocks = P.cluster, rank = blockIdx.x;  // the cluster is the x extent of the grid
  const int hg = blockIdx.y, b = blockIdx.z;
  if (tid < 8 * NT) known[tid] = ordered(-INFINITY);
  serial_wait();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const int raw_len = P.lens[b], len = clamped_len(P, b);
  Parts parts;
  parts.np = parts.most = blocks * kJoinWarps;
  parts.nb = (len + 15) >> 4;
  parts.run = (parts.nb + parts.np - 1) / parts.np;
  parts.off = 0;
  if (len > 0) {
    Scorer<T, D, NT> sc;
    sc.load_q(P, b, hg, sq, tid, 32 * kJoinWarps);
    if (sizeof(T) == 4) __syncthreads();
    const int i = rank * kJoinWarps + warp;
    auto score = [&](auto one_page) {
      score_run<T, D, NT, true, decltype(one_page)::value>(
          P, sc, sq, b, hg, len, min(i * parts.run, parts.nb), min((i + 1) * parts.run, parts.nb),
          info + i, parts.np, known, blocks);
    };
    if (P.page_size % 16 == 0) score(std::true_type());
    else score(std::false_type());
  } else {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (raw_len != 0 && rank == 0 && hg == 0 && tid == 0)
      atomicMax(P.status, ENTMAX_ATTN_ERANGE);
  }
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  // the block's heads: rank, rank + blocks, ...
  const int hk = hg / P.head_blocks, hb = hg - hk * P.head_blocks;
  const int h0 = hk * P.G + hb * 8 * NT, heads = min(8 * NT, P.G - hb * 8 * NT);
  if (len == 0) {
    for (int col = rank; col < heads; col += blocks)
      write_empty<T, D>(P, b, h0 + col, raw_len == 0, tid, 32 * kJoinWarps);
  } else if (heads <= blocks) {
    if (rank >= heads) return;
    parts.info = info + rank * parts.np;
    const Bounds bound = part_bounds<BK, kJoinWarps>(P, sm.block.red, parts);
    join_head<T, D, BK, kJoinWarps, 1>(P, sm.block, 0, b, h0 + rank, len, bound, parts);
  } else {
    for (int c0 = rank; c0 < heads; c0 += blocks * kJoinWarps) {
      auto head = [&](int w) {
        HeadRef r{b, h0 + c0 + w * blocks, len, parts};
        r.parts.info = info + (c0 + w * blocks) * parts.np;
        return r;
      };
      join_many<T, D, BK, false>(P, sm.many, c0 + warp * blocks < heads, head);
    }
  }
}

template <typename T, int D, int NT, int BK>
cudaError_t launch_cluster(const DecodeProblem& P, cudaStream_t s) {
  return launch_serial(decode_cluster_kernel<T, D, NT, BK>,
                       dim3(P.cluster, P.Hkv * P.head_blocks, P.B), dim3(32 * kJoinWarps), 0, s,
                       P.cluster, P);
}

template <typename T, int D, int BK>
cudaError_t launch_decode_k(const DecodeProblem& P, cudaStream_t s) {
  if (P.cluster)
    return P.heads_per_block == 8 ? launch_cluster<T, D, 1, BK>(P, s)
                                  : launch_cluster<T, D, 2, BK>(P, s);
  const cudaError_t e = P.heads_per_block == 8 ? launch_scores<T, D, 1>(P, s)
                                               : launch_scores<T, D, 2>(P, s);
  if (e != cudaSuccess) return e;
  return launch_join<T, D, BK>(P, s);
}

template <typename T, int D>
cudaError_t launch_decode_t(const DecodeProblem& P, cudaStream_t s) {
  switch (beta_kind(P.beta)) {
    case kBetaOne: return launch_decode_k<T, D, kBetaOne>(P, s);
    case kBetaTwo: return launch_decode_k<T, D, kBetaTwo>(P, s);
    case kBetaNear3: return launch_decode_k<T, D, kBetaNear3>(P, s);
    default: return launch_decode_k<T, D, kBetaGeneral>(P, s);
  }
}

}  // namespace
}  // namespace ea
