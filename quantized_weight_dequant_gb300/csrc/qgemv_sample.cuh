// Sampling the next token of each row: temperature, top-k, top-p and min-p from one random number.
//
// With w_i = 2^((l_i - max l) log2(e) / T) the tokens that stay are a beginning of the order (logit descending,
// index ascending), cut by a count (top-k) and by a sum of weights (top-p), and a floor under the weights
// (min-p); the draw is the first index whose running sum of kept weights exceeds u times their sum.  Nothing is
// sorted: a cut is found by histograms over ever finer ranges of the logits, and the draw by sums of the warps'
// pieces of the row.
//
//  * Weights are whole numbers of 2^-43, computed to 2^-32 of the largest, and their sums are exact: the result
//    does not depend on which thread adds what.  32-bit weights are not enough: an error of 2^-24 in a
//    few heavy tokens moves the borders of all the others, and of 10^4 draws some would go to a neighbour.
//  * A row belongs to a cluster of CTAs, each with a piece of it in index order, each warp with a piece of that.
//  * Histogram 0 goes by z = (max - l) log2(e) / T, 40 buckets for each halving of the weight (where weights
//    matter; coarser behind 2^-45): monotone in the logit, so its buckets are ranges of the order.  The
//    bucket with the border is then divided by the logits' bits, 2048 ways at a time, until the border falls between two
//    ranges or within one value, whose equals are counted by index.
//  * What takes part after a cut is listed, so that it is found once: in the cluster's first CTA where it holds all, in every CTA's own
//    list, or, of more, the border's bucket alone.  (Going over the rows every time: 64 rows of 128000 fp32 with mixed settings
//    136 us, with lists 68; 509 of 50001 in bf16 with top-p 376 and 161.)
//  * Instructions and shared memory's adds bound the passes with weights, the meetings of a cluster the rest: one row of 32000
//    takes 10.1 us, of which the logits' bytes are nothing; 64 rows of 128000 without limits 34 (4.8 at the copy's rate), with
//    top-k 50 22, with the largest logit alone 9.2.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/qgemv.h"
#include "qgemv_ptx.cuh"

namespace qg {

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kSampleBuckets = 2048;
constexpr int kSampleGroups = 32;  // of 64 buckets
constexpr int kSampleNothing = 1801;  // the first bucket whose tokens weigh nothing: 45 halvings, 40 buckets each, to the nearest
constexpr int kSampleMaxCluster = 8;
// Candidates that are compared each with each (8 x 50001, top-k 400 and top-p 0.9: 23.3 us, with 512 44.9; top-k 200: 21.8, with 128
// 22.6), and that one CTA's list holds: so many that a second CTA finds room on the SM.
constexpr int kSampleFew = 256;
constexpr int kSampleList = 4096;
constexpr int kSampleUnit = 43;    // weights in units of 2^-43: 2^20 of them stay below 2^64
constexpr uint32_t kTableFirst = 119 << 7, kTableValues = 15 << 7;  // bf16: magnitudes of 2^-8 up to 2^7
constexpr float kInf = __builtin_huge_valf();

struct alignas(16) SampleSmem {
  uint32_t count[kSampleBuckets], lo[kSampleBuckets], hi[kSampleBuckets];  // hi:lo a 64-bit sum
  uint64_t group_mass[kSampleGroups];
  uint32_t group_count[kSampleGroups];  // beside masses
  uint64_t warp_sum[kSampleWarps];
  uint64_t cta_sum[2];    // for the cluster
  uint32_t found[2];      // for the cluster
  uint32_t others;        // add_values
  uint32_t mine, listed;  // candidates of this CTA's piece, and in its list
  uint64_t best_warp[kSampleWarps];
  uint64_t best;          // for the cluster
  uint4 edge[2];          // the row's first and last 16 bytes, with -inf in the places of what is not the row's
  float scale[2];         // of the row: hi, lo
  uint64_t pick_before, pick_mass, pick_target, pick_total;
  uint32_t pick_bucket, pick_count, pick_first;  // pick_first: tokens up to the end of the bucket's group (MASS)
  uint64_t pow[64];
  float list_logit[kSampleList];
  uint32_t list_index[kSampleList];
};

__host__ __device__ constexpr size_t sample_table_bytes(int type) { return type == QGEMV_OUT_BF16 ? 2 * kTableValues * 8 : 0; }

// ---------------------------------------------------------------------------- cluster
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// (.aligned: whole warps come here, whatever their lanes did before)
__device__ __forceinline__ void cluster_arrive_all() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_all() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_meet() {
  cluster_arrive_all();
  cluster_wait_all();
}
__device__ __forceinline__ uint32_t remote_u32(const void* p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t remote_u64(const void* p, uint32_t rank) {
  uint32_t a;
  uint64_t v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void store_remote(const void* p, uint32_t rank, uint32_t v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ uint64_t warp_scan64(uint64_t v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// floor(u total), and whether that is all of it, for u in (0, 1): 24 bits times 64, shifted.  (Every thread needs it: in 64-bit
// floats, of which an SM does two a cycle, it takes the CTA 3400 cycles.)
__device__ __forceinline__ uint64_t share_of(float u, uint64_t total, bool& whole) {
  const uint32_t b = __float_as_uint(u), e = b >> 23;
  const uint64_t mant = (b & 0x7fffff) | (e ? 0x800000 : 0);
  const int shift = 150 - static_cast<int>(max(e, 1u));  // u = mant 2^-shift, shift >= 24
  const uint64_t hi = __umul64hi(total, mant), lo = total * mant;
  if (shift >= 64) {
    if (shift >= 128) {
      whole = false;
      return 0;
    }
    whole = lo == 0 && (shift == 64 || hi << (128 - shift) == 0);
    return shift == 64 ? hi : hi >> (shift - 64);
  }
  whole = lo << (64 - shift) == 0;
  return hi << (64 - shift) | lo >> shift;
}

// log(part / total) to fp32's precision: near 1 by what is missing, which a quotient of 24 bits has lost.
__device__ __forceinline__ float log_share(uint64_t part, uint64_t total) {
  const uint64_t rest = total - part;
  const float q = static_cast<float>(static_cast<double>(min(part, rest)) / static_cast<double>(total));
  return part > rest ? log1pf(-q) : logf(q);
}

// ---------------------------------------------------------------------------- logits
template <int T>
constexpr int kVec = T == QGEMV_OUT_F32 ? 4 : 8;  // logits in 16 bytes

// -0 as 0, so that equal logits have equal bits.  (NaN stays: it is above nothing, in the last bucket and of weight 0, like -inf.)
__device__ __forceinline__ float usual(float l) { return l + 0.f; }

template <int T>
__device__ __forceinline__ void unpack(const uint4& v, float (&l)[kVec<T>]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (T == QGEMV_OUT_F32) {
      l[j] = __uint_as_float(w[j]);
    } else if constexpr (T == QGEMV_OUT_F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      l[2 * j] = f.x, l[2 * j + 1] = f.y;
    } else {
      l[2 * j] = __uint_as_float(w[j] << 16), l[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}
// Back, for values that `unpack` gave (or -inf or 0).
template <int T>
__device__ __forceinline__ uint4 repack(const float (&l)[kVec<T>]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (T == QGEMV_OUT_F32) {
      w[j] = __float_as_uint(l[j]);
    } else if constexpr (T == QGEMV_OUT_F16) {
      const __half2 h = __floats2half2_rn(l[2 * j], l[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      w[j] = __float_as_uint(l[2 * j]) >> 16 | (__float_as_uint(l[2 * j + 1]) & 0xffff0000u);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The logit's place in the order: smaller for larger logits.
__device__ __forceinline__ uint32_t rank_key(float l) {
  const uint32_t b = __float_as_uint(l);
  return b & 0x80000000u ? b : ~(b | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k : ~k & 0x7fffffffu); }

// 2^(j/64) in units of 2^-52.
__constant__ const uint64_t kPow[64] = {
    4503599627370496ull, 4552640611975265ull, 4602215617889652ull, 4652330460224456ull, 4702991017412879ull,
    4754203231900066ull, 4805973110840145ull, 4858306726800864ull, 4911210218475899ull, 4964689791404917ull,
    5018751718701482ull, 5073402341788886ull, 5128648071143992ull, 5184495387049181ull, 5240950840352481ull,
    5298021053235979ull, 5355712719992597ull, 5414032607811327ull, 5472987557571019ull, 5532584484642807ull,
    5592830379701282ull, 5653732309544490ull, 5715297417922861ull, 5777532926377168ull, 5840446135085607ull,
    5904044423720103ull, 5968335252311938ull, 6033326162126810ull, 6099024776549417ull, 6165438801977672ull,
    6232576028726661ull, 6300444331942437ull, 6369051672525773ull, 6438406098065967ull, 6508515743784820ull,
    6579388833490889ull, 6651033680544135ull, 6723458688831074ull, 6796672353750547ull, 6870683263210221ull,
    6945500098633947ull, 7021131635980086ull, 7097586746770917ull, 7174874399133264ull, 7253003658850448ull,
    7331983690425701ull, 7411823758157149ull, 7492533227224511ull, 7574121564787629ull, 7656598341096955ull,
    7739973230616135ull, 7824256013156818ull, 7909456575025820ull, 7995584910184779ull, 8082651121422441ull,
    8170665421539708ull, 8259638134547591ull, 8349579696878213ull, 8440500658608991ull, 8532411684700150ull,
    8625323556245722ull, 8719247171738151ull, 8814193548346688ull, 8910173823209688ull};

// What the weights of a row go by: its largest logit, and 64 log2(e) / T in two floats.
struct RowScale {
  float m, hi, lo;
  float least;  // a finite logit of weight 0, as which lower ones (and NaN) count
  bool sharp;   // every logit but the largest has weight 0: that is infinite, or neighbouring numbers are that far apart
};

__device__ __forceinline__ RowScale row_scale(float m, float hi, float lo) {
  RowScale r{m, hi, lo, 0.f, false};
  const float far = 64.f * (kSampleUnit + 2) / hi;
  r.sharp = !(fabsf(m) * 5.9604645e-08f < far);  // (the next lower logit is |m| 2^-24 away at least)
  r.least = m - far * 1.0001f - fabsf(m) * 2.4e-7f;
  return r;
}

// 2^43 w, rounded down, for a row that is not sharp.  y = (l - m) 64 log2(e) / T as a sum of two floats; y = k + f with k whole and
// |f| <= 1/2; 2^(f/64) - 1 by its series in g = f ln(2)/64, |g| < 0.0055, as a sum of two floats again, and that in whole numbers
// of 2^-22 and of 2^-44; times 2^(k/64) = 2^(k >> 6) times one of 64 constants.  Right to 2^-32 of the largest weight, weights
// near 1 to 2^-31.8 of themselves as a root of the mean square; the mean is right to 2^-37 (against 80 bits, over 6 10^7 arguments).
// Conversions between floats and whole numbers are additions of 1.5 2^23 units, since the converting instructions go at a quarter
// of the rate.  45 instructions: with 117 (64-bit shifts and products as they come) 64 rows of 128000 took 56 us.
__device__ __forceinline__ uint64_t weight_of(float l, const RowScale& r, const uint64_t* pow, float& y) {
  l = fmaxf(l, r.least);
  const float d = l - r.m;
  const float back = d - l;
  const float off = (l - (d - back)) + (-r.m - back);  // l - m = d + off
  const float p = d * r.hi;
  y = p;
  const float e = fmaf(off, r.hi, fmaf(d, r.lo, fmaf(d, r.hi, -p)));
  const float kf = p + 12582912.f;
  const int kb = __float_as_int(kf);  // 0x4b400000 + k
  const float f = p - (kf - 12582912.f);
  constexpr float kL = 0.0108304247f;  // ln(2) / 64
  const float g = f * kL;
  const float q = fmaf(g * g, fmaf(g, 1.f / 6.f, 0.5f), fmaf(e, kL, fmaf(f, kL, -g)));
  const float x = g + q, left = (g - x) + q;  // 2^(f/64) - 1 = x + left
  const float a = x + 3.f;                    // units of 2^-22
  const float b = ((x - (a - 3.f)) + left) + 7.152557373046875e-07f;  // 1.5 2^-21: units of 2^-44
  const int n1 = __float_as_int(a) - 0x40400000, n2 = __float_as_int(b) - 0x35400000;
  uint64_t t = pow[kb & 63];
  const int c = static_cast<int>(t >> 22);  // units of 2^-30
  asm("mad.wide.s32 %0, %1, %2, %0;" : "+l"(t) : "r"(c), "r"(n1));
  asm("mad.wide.s32 %0, %1, 1024, %0;" : "+l"(t) : "r"(__mulhi(c, n2)));
  uint64_t w;
  asm("shr.u64 %0, %1, %2;" : "=l"(w) : "l"(t), "r"((0x4b400000 + 639 - kb) >> 6));  // 9 - (k >> 6); from 64 on 0
  return w;
}

// Histogram 0: 40 buckets for each halving of the weight, behind 2^-45 16 for each doubling of the distance.
__device__ __forceinline__ int linear_bucket(float y) { return __float_as_int(fmaf(y, -0.625f, 12582912.f)) - 0x4b400000; }  // to the nearest
__device__ __forceinline__ int bucket_of(float l, const RowScale& r) {
  const float y = (l - r.m) * r.hi;  // 64 for each halving
  if (!(y > -2880.f)) {
    if (l == r.m) return 0;  // infinite
    const float z = y * -0.015625f;
    if (!(z < 65536.f)) return kSampleBuckets - 1;
    return kSampleNothing + ((__float_as_int(z) - __float_as_int(45.f)) >> 19);
  }
  return linear_bucket(y);
}

// The tokens that stay, a beginning of the order: those of smaller buckets, and of `bucket` those of smaller keys and of `key`
// the indexes up to `index`.  Logits from `sure` on are of smaller buckets (NaN: none is known to be), those up to `never` of larger
// ones: few need more than two comparisons.
struct Cut {
  int bucket;
  uint32_t key, index;
  float sure, never;
};
__device__ __forceinline__ Cut cut_in(int bucket, const RowScale& r) {
  Cut c{bucket, 0xffffffffu, 0xffffffffu, __int_as_float(0x7fffffff), -kInf};
  auto z_at = [](int b) { return b < kSampleNothing ? (static_cast<float>(b) - 0.5f) / 40.f : __int_as_float(__float_as_int(45.f) + ((b - kSampleNothing) << 19)); };
  const float wide = 1e-5f * fabsf(r.m);
  // buckets are monotone in the logit: a logit of a smaller bucket proves it of all larger ones
  const float sure = r.m - z_at(bucket) * (64.f * 0.99999f) / r.hi + wide, never = r.m - z_at(bucket + 1) * (64.f * 1.00001f) / r.hi - wide;
  if (sure == sure && bucket_of(sure, r) < bucket) c.sure = sure;
  if (never == never && bucket < kSampleBuckets - 1 && bucket_of(never, r) > bucket) c.never = never;
  return c;
}
__device__ __forceinline__ bool stays(const Cut& c, float l, uint32_t i, const RowScale& r) {
  if (l >= c.sure) return true;
  if (l <= c.never) return false;
  const int b = bucket_of(l, r);
  if (b != c.bucket) return b < c.bucket;
  const uint32_t k = rank_key(l);
  return k < c.key || (k == c.key && i <= c.index);
}
// What both leave.
__device__ __forceinline__ Cut both_cuts(const Cut& a, const Cut& b) {
  if (a.bucket != b.bucket) return a.bucket < b.bucket ? a : b;
  if (a.key != b.key) return a.key < b.key ? a : b;
  return a.index < b.index ? a : b;
}

// A cluster's view of one row.  HELD: each CTA has its piece in shared memory, with what does not take part as -inf.
template <int T, bool HELD>
struct SampleRow {
  SampleSmem& s;
  const void* row;       // global
  const uint4* vecs;     // 16 bytes each; the first holds logits before the row's, too, where the row begins inside it
  uint32_t rank, ctas;
  int before_row;        // how many
  int V;
  int last;              // vector of the row
  int begin_at, end, whole;  // this CTA's vectors, and how many a warp has
  int lo, hi;            // this warp's
  int lane, warp;
  RowScale r;
  const uint64_t* table;  // bf16: weights of the values of 15 octaves, positive ones first
  bool listed = false;   // the candidates are, in s.list_*
  bool parted = false;   // only those of the border's bucket are, and
  uint64_t above = 0;    // this thread's sum of the smaller buckets' weights
  bool alone = false;    // those of the whole cluster in its first CTA, and the others have nothing to do
  uint64_t goal = 0;     // of few listed candidates, the mass at which top-p ends, once it is known
  int turn = 0;
  bool reading = false;  // others may still be reading this CTA's histogram

  // The weight of a logit of a row that is not sharp, and y = (l - m) 64 log2(e) / T.
  __device__ __forceinline__ uint64_t weight_y(float l, float& y) const {
    if constexpr (T == QGEMV_OUT_BF16) {
      const uint32_t b = __float_as_uint(l) >> 16, i = (b & 0x7fff) - kTableFirst;
      if (table && i < kTableValues) {
        y = (l - r.m) * r.hi;
        return table[i + (b >> 15) * kTableValues];
      }
    }
    return weight_of(l, r, s.pow, y);
  }
  __device__ __forceinline__ uint64_t sharp_weight(float l) const { return l == r.m ? 1ull << kSampleUnit : 0; }
  __device__ __forceinline__ uint64_t weight(float l) const {
    float y;
    return r.sharp ? sharp_weight(l) : weight_y(l, y);
  }
  // bf16 has few values: their weights are computed once (a weight is 45 instructions, a row has thousands of equal logits).
  __device__ __forceinline__ void fill(uint64_t* to) {
    for (int i = threadIdx.x; i < 2 * static_cast<int>(kTableValues); i += kSampleThreads) {
      const uint32_t v = i < static_cast<int>(kTableValues) ? kTableFirst + i : 0x8000u + kTableFirst + i - kTableValues;
      const float l = __uint_as_float(v << 16);
      float y;
      to[i] = l > r.m ? 0 : weight_of(l, r, s.pow, y);
    }
    __syncthreads();
  }

  __device__ __forceinline__ int index_of(int v) const { return v * kVec<T> - before_row; }

  // Vector v as the row has it.
  __device__ __forceinline__ void load_global(int v, float (&l)[kVec<T>]) const {
    const int i0 = index_of(v);
    if (i0 >= 0 && i0 + kVec<T> <= V) {
      unpack<T>(vecs[v], l);
#pragma unroll
      for (int j = 0; j < kVec<T>; ++j) l[j] = usual(l[j]);
    } else {
#pragma unroll
      for (int j = 0; j < kVec<T>; ++j) {
        l[j] = -kInf;
        if (i0 + j >= 0 && i0 + j < V) {
          if constexpr (T == QGEMV_OUT_F32) {
            l[j] = static_cast<const float*>(row)[i0 + j];
          } else {
            const uint32_t b = static_cast<const uint16_t*>(row)[i0 + j];
            if constexpr (T == QGEMV_OUT_F16)
              l[j] = __half2float(__ushort_as_half(static_cast<unsigned short>(b)));
            else
              l[j] = __uint_as_float(b << 16);
          }
          l[j] = usual(l[j]);
        }
      }
    }
  }
  __device__ __forceinline__ const uint4* where(int v) const {
    const uint4* at = vecs + v;
    if (!HELD && v == last) at = &s.edge[1];
    if (!HELD && v == 0) at = &s.edge[0];
    return at;
  }
  __device__ __forceinline__ uint4 load(int v) const { return *where(v); }

  template <int U>
  __device__ __forceinline__ void read(int v0, uint4 (&raw)[U]) const {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (v0 + 32 * u < hi) raw[u] = load(v0 + 32 * u);
  }
  // f(logits, index of the first, how many) of this warp's piece, U vectors' reads in flight together; of the candidates, one by one,
  // once they are listed
  template <int U, class F, class G>
  __device__ __forceinline__ void each(F f, G g) const {
    if (listed) {
      for (uint32_t i = threadIdx.x; i < s.listed; i += kSampleThreads) g(s.list_logit[i], s.list_index[i]);
      return;
    }
    uint4 next[U];
    if (!HELD) read<U>(lo + lane, next);
    for (int v0 = lo + lane; v0 < hi; v0 += 32 * U) {
      uint4 raw[U];
      if (HELD) {
        read<U>(v0, raw);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = next[u];
        read<U>(v0 + 32 * U, next);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (v0 + 32 * u >= hi) break;
        float l[kVec<T>];
        unpack<T>(raw[u], l);
        if (!HELD) {
#pragma unroll
          for (int j = 0; j < kVec<T>; ++j) l[j] = usual(l[j]);
        }
        f(l, static_cast<uint32_t>(index_of(v0 + 32 * u)));
      }
    }
  }
  // f(logit, index) where pick(logit) says so, which few do
  template <class P, class F>
  __device__ __forceinline__ void each_of(P pick, F f) const {
    each<2>(
        [&](const float (&l)[kVec<T>], uint32_t i) {
          uint32_t some = 0;
#pragma unroll
          for (int j = 0; j < kVec<T>; ++j) some |= static_cast<uint32_t>(pick(l[j])) << j;
          while (some) {
            const int j = __ffs(some) - 1;
            some &= some - 1;
            float one = l[0];
#pragma unroll
            for (int q = 1; q < kVec<T>; ++q)
              if (j == q) one = l[q];
            f(one, i + j);
          }
        },
        [&](float l, uint32_t i) {
          if (pick(l)) f(l, i);
        });
  }
  // f(weight, y, logit, index) of the tokens that `in` keeps (ALL: of all), whose weights are computed four at a time; y: as weight_of
  // gives it
  template <bool ALL, class F>
  __device__ __forceinline__ void each_weight(const Cut& in, F f) const {
    each<2>(
        [&](const float (&l)[kVec<T>], uint32_t i) {
#pragma unroll
          for (int h = 0; h < kVec<T>; h += 4) {
            bool here[4] = {true, true, true, true}, any = ALL;
            if (!ALL) {
#pragma unroll
              for (int j = 0; j < 4; ++j) any |= here[j] = stays(in, l[h + j], i + h + j, r);
            }
            if (!any) continue;
            uint64_t w[4];
            float y[4];
            if (r.sharp) {
#pragma unroll
              for (int j = 0; j < 4; ++j) w[j] = sharp_weight(l[h + j]), y[j] = 0.f;
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) w[j] = weight_y(l[h + j], y[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (here[j]) f(w[j], y[j], l[h + j], i + h + j);
          }
        },
        [&](float l, uint32_t i) {
          if (!ALL && !stays(in, l, i, r)) return;
          float y = 0.f;
          const uint64_t w = r.sharp ? sharp_weight(l) : weight_y(l, y);
          f(w, y, l, i);
        });
  }

  __device__ __forceinline__ void meet() {
    if (ctas > 1)
      cluster_meet();
    else
      __syncthreads();
  }

  // An empty histogram.
  __device__ __forceinline__ void begin() {
    if (reading) cluster_wait_all();
    reading = false;
    uint4* h = reinterpret_cast<uint4*>(s.count);
    for (int i = threadIdx.x; i < 3 * kSampleBuckets / 4; i += kSampleThreads) h[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  __device__ __forceinline__ void settle() {
    if (reading) cluster_wait_all();
    reading = false;
  }

  __device__ __forceinline__ void add_mass(int b, uint64_t w) const {
    if (!w) return;
    const uint32_t wl = static_cast<uint32_t>(w), old = atomicAdd(&s.lo[b], wl);
    const uint32_t wh = static_cast<uint32_t>(w >> 32) + (old + wl < old);
    if (wh) atomicAdd(&s.hi[b], wh);
  }

  // The first bucket of the histogram, over the whole cluster, at which the running count (mass) reaches aim(sum) - `before`;
  // s.pick_* say which and what it holds.
  template <bool MASS, class A>
  __device__ void pick(A aim, uint64_t before) {
    __syncthreads();
    {  // sums of the 32 groups: 16 threads each
      const int g = threadIdx.x / 16, at = threadIdx.x % 16;
      uint64_t m = 0;
      uint32_t c = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int b = g * 64 + j * 16 + at;
        if (MASS) m += static_cast<uint64_t>(s.hi[b]) << 32 | s.lo[b];
        c += s.count[b];
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) {
        if (MASS) m += __shfl_xor_sync(0xffffffffu, m, o);
        c += __shfl_xor_sync(0xffffffffu, c, o);
      }
      if (at == 0) s.group_mass[g] = MASS ? m : c, s.group_count[g] = c;
    }
    meet();
    if (warp == 0) {
      const uint32_t last = ctas - 1;
      uint64_t v = s.group_mass[lane];
      uint32_t some = s.group_count[lane];
      if (ctas > 1) {
        uint64_t part[kSampleMaxCluster];
        uint32_t n[kSampleMaxCluster];
#pragma unroll
        for (uint32_t q = 0; q < kSampleMaxCluster; ++q) {
          part[q] = remote_u64(&s.group_mass[lane], min(q, last));
          if (MASS) n[q] = remote_u32(&s.group_count[lane], min(q, last));
        }
        v = some = 0;
#pragma unroll
        for (uint32_t q = 0; q < kSampleMaxCluster; ++q)
          if (q < ctas) v += part[q], some += MASS ? n[q] : 0;
      }
      uint64_t run = warp_scan64(v, lane);
      const uint64_t total = __shfl_sync(0xffffffffu, run, 31), target = aim(total);
      uint32_t hit = __ballot_sync(0xffffffffu, before + run >= target);
      const int g = hit ? __ffs(hit) - 1 : 31;
      before += __shfl_sync(0xffffffffu, run - v, g);
      some = __reduce_add_sync(0xffffffffu, lane <= g ? some : 0);
      // the group's 64 buckets, two a lane
      const int b0 = g * 64 + 2 * lane;
      uint64_t bm[2] = {}, bc = 0;  // bc: counts in halves
      if (ctas > 1) {
        uint64_t c[kSampleMaxCluster], lo[kSampleMaxCluster], hi[kSampleMaxCluster];
#pragma unroll
        for (uint32_t q = 0; q < kSampleMaxCluster; ++q) {
          c[q] = remote_u64(&s.count[b0], min(q, last));
          if (MASS) lo[q] = remote_u64(&s.lo[b0], min(q, last)), hi[q] = remote_u64(&s.hi[b0], min(q, last));
        }
#pragma unroll
        for (uint32_t q = 0; q < kSampleMaxCluster; ++q) {
          if (q >= ctas) continue;
          bc += c[q];
          if (MASS) {
            bm[0] += hi[q] << 32 | (lo[q] & 0xffffffffu);
            bm[1] += (hi[q] & 0xffffffff00000000ull) | lo[q] >> 32;
          }
        }
      } else {
        bc = static_cast<uint64_t>(s.count[b0 + 1]) << 32 | s.count[b0];
        if (MASS) {
          bm[0] = static_cast<uint64_t>(s.hi[b0]) << 32 | s.lo[b0];
          bm[1] = static_cast<uint64_t>(s.hi[b0 + 1]) << 32 | s.lo[b0 + 1];
        }
      }
      const uint64_t v0 = MASS ? bm[0] : bc & 0xffffffffu, v1 = MASS ? bm[1] : bc >> 32;
      run = warp_scan64(v0 + v1, lane);
      hit = __ballot_sync(0xffffffffu, before + run >= target);
      const int at = hit ? __ffs(hit) - 1 : 31;
      const bool second = before + run - v1 < target;
      if (lane == at) {
        s.pick_before = before + run - v1 - (second ? 0 : v0);
        s.pick_bucket = b0 + (second ? 1 : 0);
        s.pick_mass = second ? v1 : v0;
        s.pick_count = static_cast<uint32_t>(second ? bc >> 32 : bc);
        s.pick_target = target;
        s.pick_total = total;
        s.pick_first = some;
      }
    }
    __syncthreads();
    if (ctas > 1) {
      cluster_arrive_all();
      reading = true;
    }
  }

  // An empty list again, once all CTAs have seen how long it was.
  __device__ __forceinline__ void forget() {
    meet();
    if (threadIdx.x == 0) s.mine = 0;
    __syncthreads();
  }

  // The candidates, those of `c`'s bucket and smaller ones that `in` keeps, go into lists, in no order (what follows goes by logits
  // and indexes): into that of the cluster's first CTA where it holds them, which then goes on alone, else into each CTA's own.  Where
  // one of those is too short nothing is listed, and a later list begins empty.
  __device__ void list(const Cut& c, const Cut& in) {
    settle();
    each_of([&](float l) { return l > c.never; },
            [&](float l, uint32_t i) {
              if (i >= static_cast<uint32_t>(V) || (!(l >= c.sure) && bucket_of(l, r) > c.bucket) || !stays(in, l, i, r)) return;
              const uint32_t at = atomicAdd(&s.mine, 1u);
              if (at < kSampleList) s.list_logit[at] = l, s.list_index[at] = i;
            });
    __syncthreads();
    const uint32_t n = s.mine;
    uint32_t all = n, most = n, base = 0;
    if (ctas > 1) {
      cluster_meet();
      uint32_t part[kSampleMaxCluster];
#pragma unroll
      for (uint32_t q = 0; q < kSampleMaxCluster; ++q) part[q] = remote_u32(&s.mine, min(q, ctas - 1));
      all = most = 0;
#pragma unroll
      for (uint32_t q = 0; q < kSampleMaxCluster; ++q) {
        if (q >= ctas) continue;
        if (q < rank) base += part[q];
        all += part[q];
        most = max(most, part[q]);
      }
    }
    if (most > kSampleList) {
      forget();
      return;
    }
    listed = true;
    alone = ctas == 1;
    if (threadIdx.x == 0) s.listed = n;
    if (all <= kSampleList && ctas > 1) {
      if (rank != 0)
        for (uint32_t i = threadIdx.x; i < n; i += kSampleThreads) {
          store_remote(&s.list_logit[base + i], 0, __float_as_uint(s.list_logit[i]));
          store_remote(&s.list_index[base + i], 0, s.list_index[i]);
        }
      else if (threadIdx.x == 0)
        s.listed = all;
      cluster_meet();
      alone = true;
      ctas = 1;
    }
    __syncthreads();
  }

  // Where the candidates are too many for lists: those of `c`'s bucket alone are listed, and the weights (from floor_w on) of the smaller
  // buckets' summed.
  __device__ void split(const Cut& c, const Cut& in, uint64_t floor_w) {
    settle();
    uint64_t sum = 0;
    each<2>(
        [&](const float (&l)[kVec<T>], uint32_t i) {
#pragma unroll
          for (int h = 0; h < kVec<T>; h += 4) {
            bool here[4], any = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              here[j] = l[h + j] > c.never && stays(in, l[h + j], i + h + j, r);
              if (here[j] && !(l[h + j] >= c.sure)) {
                const int b = bucket_of(l[h + j], r);
                here[j] = b < c.bucket;
                if (b == c.bucket && i + h + j < static_cast<uint32_t>(V)) {
                  const uint32_t at = atomicAdd(&s.mine, 1u);
                  if (at < kSampleList) s.list_logit[at] = l[h + j], s.list_index[at] = i + h + j;
                }
              }
              any |= here[j];
            }
            if (!any) continue;
            uint64_t w[4];
            float y;
            if (r.sharp) {
#pragma unroll
              for (int j = 0; j < 4; ++j) w[j] = sharp_weight(l[h + j]);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) w[j] = weight_y(l[h + j], y);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += here[j] && w[j] >= floor_w ? w[j] : 0;
          }
        },
        [](float, uint32_t) {});
    __syncthreads();
    uint32_t most = s.mine;
    if (ctas > 1) {
      cluster_meet();
      for (uint32_t q = 0; q < ctas; ++q) most = max(most, remote_u32(&s.mine, q));
    }
    if (most > kSampleList) {
      forget();
      return;
    }
    above = sum;
    listed = parted = true;
    if (threadIdx.x == 0) s.listed = s.mine;
    __syncthreads();
  }

  // The first index at which the running sum of `weigh` exceeds `aim(all)`; sum(): this thread's part of it; `take` is called by one thread of the cluster with
  // the index, its weight and the sum.
  template <bool FINAL, class S, class W, class A, class K>
  __device__ void locate(S sum, W weigh, A aim, K take) {
    if (listed && !(FINAL && parted)) {  // the running sum over ranges of indexes
      uint32_t first = 0;
      uint64_t target = 0, before = 0, total = 0;
      for (int shift = max(0, 32 - __clz(V - 1) - 11), width = 32;; width = shift, shift = max(0, shift - 11)) {
        begin();
        for (uint32_t e = threadIdx.x; e < s.listed; e += kSampleThreads) {
          const uint32_t i = s.list_index[e];
          if (i >= first && (width == 32 || (i - first) >> width == 0)) add_mass(static_cast<int>((i - first) >> shift), weigh(s.list_logit[e], i));
        }
        pick<true>([&](uint64_t sum) { return width == 32 ? aim(sum) + 1 : target; }, before);
        if (width == 32) total = s.pick_total;
        target = s.pick_target;
        before = s.pick_before;
        first += s.pick_bucket << shift;
        if (shift == 0) break;
      }
      settle();
      if (threadIdx.x == 0 && (alone || rank == 0)) take(first, s.pick_mass, total);
      return;
    }
    const uint64_t mine = warp_sum64(listed ? above : sum());
    settle();
    __syncthreads();
    if (lane == 0) s.warp_sum[warp] = mine;
    __syncthreads();
    if (listed) {
      for (uint32_t e = threadIdx.x; e < s.listed; e += kSampleThreads) {
        const uint32_t i = s.list_index[e];
        const uint64_t w = weigh(s.list_logit[e], i);
        const int piece = (static_cast<int>(i + before_row) / kVec<T> - begin_at) / whole;
        if (w) atomicAdd(reinterpret_cast<unsigned long long*>(&s.warp_sum[piece]), static_cast<unsigned long long>(w));
      }
      __syncthreads();
    }
    uint64_t before = 0, cta = 0;
#pragma unroll
    for (int q = 0; q < kSampleWarps; ++q) {
      const uint64_t v = s.warp_sum[q];
      if (q < warp) before += v;
      cta += v;
    }
    uint64_t total = cta;
    if (ctas > 1) {
      if (threadIdx.x == 0) s.cta_sum[turn] = cta;
      cluster_meet();
      total = 0;
#pragma unroll
      for (uint32_t q = 0; q < kSampleMaxCluster; ++q) {
        const uint64_t v = q < ctas ? remote_u64(&s.cta_sum[turn], q) : 0;
        if (q < rank) before += v;
        total += v;
      }
    }
    const uint64_t target = aim(total);
    uint64_t start = before;  // of this CTA
#pragma unroll
    for (int q = 0; q < kSampleWarps; ++q) start -= q < warp ? s.warp_sum[q] : 0;
    if (target < start || target >= start + cta) return;
    // the piece of a warp with the target in it is divided among all warps, and the part with the target gone through in order
    int piece = 0;
    for (; piece + 1 < kSampleWarps && target >= start + s.warp_sum[piece]; ++piece) start += s.warp_sum[piece];
    __syncthreads();
    const int from = min(end, begin_at + piece * whole), to = min(end, from + whole);
    const int step = (to - from + kSampleWarps - 1) / kSampleWarps;
    const int f0 = min(to, from + warp * step), f1 = min(to, f0 + step);
    auto weights = [&](int v, uint64_t(&w)[kVec<T>]) {
      float l[kVec<T>];
      if (v < f1) unpack<T>(load(v), l);
      uint64_t all = 0;
#pragma unroll
      for (int j = 0; j < kVec<T>; ++j) {
        w[j] = v < f1 ? weigh(usual(l[j]), static_cast<uint32_t>(index_of(v) + j)) : 0;
        all += w[j];
      }
      return all;
    };
    uint64_t part = 0, w[kVec<T>];
    for (int v = f0; v < f1; v += 32) part += weights(v + lane, w);
    part = warp_sum64(part);
    if (lane == 0) s.warp_sum[warp] = part;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kSampleWarps; ++q) start += q < warp ? s.warp_sum[q] : 0;
    if (target < start || target >= start + part) return;
    for (int v = f0; v < f1; v += 32) {
      const uint64_t all = weights(v + lane, w), run = start + warp_scan64(all, lane);
      const uint32_t hit = __ballot_sync(0xffffffffu, run > target);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          uint64_t at = run - all;
          bool open = true;
#pragma unroll
          for (int j = 0; j < kVec<T>; ++j) {
            at += w[j];
            if (open && at > target) {
              take(static_cast<uint32_t>(index_of(v + lane) + j), w[j], total);
              open = false;
            }
          }
        }
        return;
      }
      start = __shfl_sync(0xffffffffu, run, 31);
    }
  }

  __device__ __forceinline__ bool few() const { return listed && alone && s.listed <= kSampleFew; }

  // All that is left for few candidates, a thread to each: its place in the order and the mass before it by comparison with all others,
  // what is kept (k: at most so many; p_goal(mass of those): the mass at which top-p ends, and no limit where that is all ones), and
  // the running sum by index in the same way.  (Every cut by histograms and every draw of such a list is two meetings and two
  // passes over 2048 buckets: 1 x 32000 with k 50 and p 0.9 15.5 us for 10.1.  512 candidates take twice as long this way.)
  template <class P, class A, class K>
  __device__ void finish(uint32_t k, P p_goal, uint64_t floor_w, A aim, K take) {
    uint64_t* key = reinterpret_cast<uint64_t*>(s.count);
    uint64_t* mass = reinterpret_cast<uint64_t*>(s.lo);
    const int n = static_cast<int>(s.listed), e = threadIdx.x;
    const bool in = e < n;
    uint64_t mine = ~0ull, w = 0;
    if (in) {
      mine = static_cast<uint64_t>(rank_key(s.list_logit[e])) << 32 | s.list_index[e];
      w = weight(s.list_logit[e]);
      key[e] = mine;
      mass[e] = w;
    }
    __syncthreads();
    uint32_t place = 0;
    uint64_t before = 0;
    if (warp * 32 < n) {
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const bool less = key[j] < mine;
        place += less;
        before += less ? mass[j] : 0;
      }
    }
    auto sum = [&](uint64_t v) {  // over the CTA
      v = warp_sum64(v);
      if (lane == 0) s.warp_sum[warp] = v;
      __syncthreads();
      v = 0;
#pragma unroll
      for (int q = 0; q < kSampleWarps; ++q) v += s.warp_sum[q];
      __syncthreads();
      return v;
    };
    const uint64_t end = p_goal(sum(in && place < k ? w : 0));
    const uint64_t kept = in && place < k && before < end && w >= floor_w ? w : 0;
    if (in) mass[e] = kept;
    const uint64_t total = sum(kept), target = aim(total);
    if (warp * 32 >= n) return;
    uint64_t run = 0;
    const uint32_t index = static_cast<uint32_t>(mine);
#pragma unroll 4
    for (int j = 0; j < n; ++j) run += static_cast<uint32_t>(key[j]) <= index ? mass[j] : 0;
    if (kept && run > target && run - kept <= target) take(index, kept, total);
  }

  // Lists the tokens that can be among the first k: those whose bucket is no larger than that of the k-th largest of the threads' largest
  // logits, `top`.
  __device__ void list_first(uint32_t k, float top) {
    begin();
    if (top > -kInf) atomicAdd(&s.count[bucket_of(top, r)], 1u);
    pick<false>([&](uint64_t) { return static_cast<uint64_t>(k); }, 0);
    if (s.pick_total >= k) list(cut_in(static_cast<int>(s.pick_bucket), r), Cut{kSampleBuckets, 0, 0, -kInf, -kInf});
  }

  // add(weight, y, ...) of all tokens' sums for the histogram: those of the table's values are counted, in the place of the list, and a
  // count times a weight added, one add instead of three for each token.
  template <class A>
  __device__ void add_values(A add) {
    uint32_t* seen = s.list_index;
    static_assert(2 * kTableValues <= kSampleList);
    for (int i = threadIdx.x; i < static_cast<int>(2 * kTableValues); i += kSampleThreads) seen[i] = 0;
    if (threadIdx.x == 0) s.others = 0;
    __syncthreads();
    const auto add_one = [&](float l) {
      float y;
      const uint64_t w = weight_of(l, r, s.pow, y);
      add(w, y, 1u);
    };
    constexpr int U = 2;
    uint4 next[U];
    read<U>(lo + lane, next);
    for (int v0 = lo + lane; v0 < hi; v0 += 32 * U) {
      uint4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u] = next[u];
      read<U>(v0 + 32 * U, next);
      uint32_t others = 0;  // a bit each
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (v0 + 32 * u >= hi) break;
        const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t b = j % 2 ? w[j / 2] >> 16 : w[j / 2] & 0xffff, at = (b & 0x7fff) - kTableFirst;
          if (at < kTableValues)
            atomicAdd(&seen[at + (b >> 15) * kTableValues], 1u);
          else
            others |= static_cast<uint32_t>(__uint_as_float(b << 16) > r.least) << (8 * u + j);
        }
      }
      while (others) {
        const int k = __ffs(others) - 1;
        others &= others - 1;
        const float l = usual(__uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(where(v0 + 32 * (k / 8)))[k % 8]) << 16));
        const uint32_t at = atomicAdd(&s.others, 1u);
        if (at < kSampleList)
          s.list_logit[at] = l;  // all threads will share these
        else
          add_one(l);
      }
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < min(s.others, static_cast<uint32_t>(kSampleList)); i += kSampleThreads) add_one(s.list_logit[i]);
    for (int i = threadIdx.x; i < static_cast<int>(2 * kTableValues); i += kSampleThreads) {
      const uint32_t n = seen[i], b = i < static_cast<int>(kTableValues) ? kTableFirst + i : 0x8000u + kTableFirst + i - kTableValues;
      if (n) add(table[i], (__uint_as_float(b << 16) - r.m) * r.hi, n);
    }
  }

  // The cut after `aim(sum)` tokens (MASS: after the shortest beginning that has that mass) of those that `in` keeps.  In CTAs that
  // have nothing more to do then (alone, and not the first) it means nothing.
  template <bool MASS, class A>
  __device__ Cut cut_at(A aim, const Cut& in, uint64_t floor_w = 0) {
    begin();
    if constexpr (MASS) {
      const auto add_n = [&](uint64_t w, float y, uint32_t n) {
        if (!w) return;
        const int b = linear_bucket(y);
        atomicAdd(&s.count[b], n);
        add_mass(b, w * n);
      };
      const auto add = [&](uint64_t w, float y, float, uint32_t) { add_n(w, y, 1); };
      bool by_value = false;
      if constexpr (T == QGEMV_OUT_BF16) by_value = table && !listed && in.bucket == kSampleBuckets;
      if (by_value)
        add_values(add_n);
      else if (in.bucket == kSampleBuckets)
        each_weight<true>(in, add);
      else
        each_weight<false>(in, add);
    } else {
      each_of([&](float) { return true; }, [&](float l, uint32_t i) { if (stays(in, l, i, r)) atomicAdd(&s.count[bucket_of(l, r)], 1u); });
    }
    pick<MASS>(aim, 0);
    const uint64_t target = s.pick_target;
    uint64_t before = s.pick_before;
    uint64_t part = MASS ? s.pick_mass : s.pick_count;
    Cut c = cut_in(static_cast<int>(s.pick_bucket), r);
    // A count that ends among tokens of weight 0 (those a mask took out among them) cuts nothing that can be drawn.
    if (!MASS && c.bucket >= kSampleNothing) return c;
    if (!listed) {
      // (up to 3/4 of all lists, as the CTAs' parts are not equal: with a half and with the whole every case is within 1.5 %)
      const bool fit = MASS ? s.pick_first <= kSampleList * ctas * 3 / 4 : before + part <= kSampleList;
      if (fit) list(c, in);
      if constexpr (MASS) {
        if (!listed) split(c, in, floor_w);  // (one CTA can have most of the candidates: what a mask leaves is often one range)
        if (few()) {
          goal = target;
          return c;
        }
      }
    }
    if ((alone && rank != 0) || before + part == target) return c;
    // the bucket's logits lie between these
    uint32_t klo = c.sure < kInf ? rank_key(c.sure) : 0, khi = c.never > -kInf ? rank_key(c.never) : 0xffffffffu;
    for (;;) {
      const int bits = 32 - __clz(khi - klo);
      const int shift = max(0, bits - 11);
      begin();
      each_of([&](float l) { return !(l >= c.sure) && l > c.never; },
              [&](float l, uint32_t i) {
                const uint32_t k = rank_key(l);
                if (k < klo || k > khi || bucket_of(l, r) != c.bucket || !stays(in, l, i, r)) return;
                const int b = static_cast<int>((k - klo) >> shift);
                atomicAdd(&s.count[b], 1u);
                if (MASS) add_mass(b, weight(l));
              });
      pick<MASS>([&](uint64_t) { return target; }, before);
      before = s.pick_before;
      part = MASS ? s.pick_mass : s.pick_count;
      klo += s.pick_bucket << shift;
      khi = klo + ((1u << shift) - 1);
      c.key = khi;
      if (s.pick_count == 1 || before + part == target) return c;
      if (shift == 0) break;
    }
    // equal logits: the first of them by index
    uint64_t n = target - before;
    if (MASS) {
      const uint64_t one = part / s.pick_count;
      n = (n + one - 1) / one;
    }
    const int f = turn;
    const float equal = key_logit(klo);
    const auto is = [&](float l, uint32_t i) { return static_cast<uint64_t>(l == equal && stays(in, l, i, r)); };
    locate<false>(
        [&] {
          uint64_t mine = 0;
          each_of([&](float l) { return l == equal; }, [&](float l, uint32_t i) { mine += is(l, i); });
          return mine;
        },
        is, [&](uint64_t) { return n - 1; }, [&](uint32_t i, uint64_t, uint64_t) { s.found[f] = i; });
    turn ^= 1;
    meet();
    uint32_t at = 0xffffffffu;
    for (uint32_t q = 0; q < ctas; ++q) at = min(at, ctas > 1 ? remote_u32(&s.found[f], q) : s.found[f]);
    c.index = at;
    return c;
  }
};

template <int T, bool HELD>
__global__ void __launch_bounds__(kSampleThreads, 2) sample_kernel(const __grid_constant__ qgemv_sample_t p) {
  extern __shared__ __align__(16) uint8_t sample_smem[];
  SampleSmem& s = *reinterpret_cast<SampleSmem*>(sample_smem);
  constexpr int E = kVec<T>;
  const uint32_t ctas = cluster_ctas(), rank = cluster_rank();
  const int64_t m = blockIdx.x / ctas;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  const uint8_t* at_row = static_cast<const uint8_t*>(p.logits) + m * p.stride * (16 / E);
  const int skip = static_cast<int>((reinterpret_cast<uintptr_t>(at_row) & 15) / (16 / E));
  const uint4* global = reinterpret_cast<const uint4*>(at_row - skip * (16 / E));
  uint4* held = reinterpret_cast<uint4*>(sample_smem + sizeof(SampleSmem) + sample_table_bytes(T));
  const int vectors = (skip + p.V + E - 1) / E;
  const int c0 = static_cast<int>(static_cast<int64_t>(vectors) * rank / ctas), c1 = static_cast<int>(static_cast<int64_t>(vectors) * (rank + 1) / ctas);
  const int per = (c1 - c0 + kSampleWarps - 1) / kSampleWarps;
  SampleRow<T, HELD> row{s, at_row, global, rank, ctas, skip, p.V, vectors - 1};
  uint64_t* table = reinterpret_cast<uint64_t*>(sample_smem + sizeof(SampleSmem));
  row.begin_at = c0, row.end = c1, row.whole = per;
  row.lo = min(c1, c0 + warp * per);
  row.hi = min(c1, row.lo + per);
  row.lane = lane;
  row.warp = warp;
  if (threadIdx.x < 2) s.found[threadIdx.x] = 0xffffffffu;
  if (threadIdx.x == 2) s.mine = 0;
  if (threadIdx.x < 64) s.pow[threadIdx.x] = kPow[threadIdx.x];
  pdl_wait();
  const float temperature = p.temperature ? p.temperature[m] : 1.f, top_p = p.top_p ? p.top_p[m] : 1.f;
  const float min_p = p.min_p ? p.min_p[m] : 0.f, u = p.u[m];
  const int32_t k = p.top_k ? p.top_k[m] : 0;
  // the largest logit and its first index; the piece into shared memory
  float top = -kInf;
  int at = -1;
#pragma unroll 4
  for (int v = row.lo + lane; v < row.hi; v += 32) {
    float l[E];
    row.load_global(v, l);
    if (HELD)
      held[v - c0] = repack<T>(l);
    else if (v == 0 || v == vectors - 1)
      s.edge[v != 0] = repack<T>(l);
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (l[j] > top) top = l[j], at = row.index_of(v) + j;
  }
  if (HELD) row.vecs = held - c0;
  uint64_t best = at < 0 ? 0 : static_cast<uint64_t>(~rank_key(top)) << 32 | (0xffffffffu - static_cast<uint32_t>(at));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) s.best_warp[warp] = best;
  if (threadIdx.x == kSampleThreads - 1) {
    const double c = 64.0 * 1.4426950408889634 / fmin(fmax(static_cast<double>(temperature), 5.421010862427522e-20), 1.152921504606847e18);
    s.scale[0] = static_cast<float>(c), s.scale[1] = static_cast<float>(c - s.scale[0]);
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kSampleWarps; ++q) best = max(best, s.best_warp[q]);
  if (ctas > 1) {
    if (threadIdx.x == 0) s.best = best;
    cluster_meet();
#pragma unroll
    for (uint32_t q = 0; q < kSampleMaxCluster; ++q)
      if (q < ctas) best = max(best, remote_u64(&s.best, q));
  }
  if (best != 0) row.r = row_scale(key_logit(~static_cast<uint32_t>(best >> 32)), s.scale[0], s.scale[1]);
  if (best == 0 || !(temperature > 0.f)) {
    if (rank == 0 && threadIdx.x == 0) {
      p.tokens[m] = best ? static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(best)) : -1;
      if (p.logprobs) p.logprobs[m] = best ? 0.f : -kInf;
    }
  } else {
    const bool limited = k > 0 && k < p.V;
    row.table = T == QGEMV_OUT_BF16 && !row.r.sharp && !(limited && k <= kSampleList) ? table : nullptr;  // a list's weights are fewer than the table's
    if (row.table) row.fill(table);
    Cut cut{kSampleBuckets, 0, 0, -kInf, -kInf};
    if (limited && k <= static_cast<int>(ctas) * kSampleThreads / 2) row.list_first(static_cast<uint32_t>(k), top);
    const uint64_t floor_w = min_p > 0.f ? static_cast<uint64_t>(ceilf(fminf(min_p, 1.f) * 8796093022208.f)) : 0;  // 2^43 times it is exact
    const auto p_goal = [&](uint64_t total) {
      bool whole = true;
      const uint64_t t = top_p > 0.f ? share_of(top_p, total, whole) : 0;
      return max(t + !whole, static_cast<uint64_t>(1));
    };
    const auto aim = [&](uint64_t total) {
      bool whole;
      return u >= 1.f ? total - 1 : u > 0.f ? share_of(u, total, whole) : 0;
    };
    const auto take = [&](uint32_t i, uint64_t w, uint64_t total) {
      p.tokens[m] = static_cast<int32_t>(i);
      if (p.logprobs) p.logprobs[m] = log_share(w, total);
    };
    if (!row.few()) {
      if (limited && !(row.alone && rank != 0)) cut = row.template cut_at<false>([&](uint64_t) { return static_cast<uint64_t>(k); }, cut);
      if (top_p < 1.f && !(row.alone && rank != 0)) cut = both_cuts(cut, row.template cut_at<true>(p_goal, cut, floor_w));
    }
    if (row.alone && rank != 0) {
      // the first CTA has all that is left
    } else if (row.goal || (row.few() && cut.bucket == kSampleBuckets)) {
      row.finish(
          limited ? static_cast<uint32_t>(k) : 0xffffffffu, [&](uint64_t total) { return row.goal ? row.goal : top_p < 1.f ? p_goal(total) : ~0ull; }, floor_w, aim, take);
    } else {
      row.template locate<true>(
          [&] {
            uint64_t mine = 0;
            if (cut.bucket == kSampleBuckets && floor_w == 0)
              row.template each_weight<true>(cut, [&](uint64_t w, float, float, uint32_t) { mine += w; });
            else
              row.template each_weight<false>(cut, [&](uint64_t w, float, float, uint32_t) { mine += w >= floor_w ? w : 0; });
            return mine;
          },
          [&](float l, uint32_t i) -> uint64_t {
            if (!stays(cut, l, i, row.r)) return 0;
            const uint64_t w = row.weight(l);
            return w >= floor_w ? w : 0;
          },
          aim, take);
    }
  }
  if (ctas > 1) cluster_meet();  // no CTA leaves while another reads its shared memory
}

}  // namespace qg
