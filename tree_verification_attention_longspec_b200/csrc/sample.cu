// Sampling from logits (temperature, top-k, top-p, min-p) with given uniform numbers, and
// the acceptance of a verified draft tree whose nodes are sampled that way.
//
// For a row of logits l, its largest value top, and temperature t > 0:
//   w_i = exp((l_i - top) / t), 1 for the largest
//   top-k keeps the first k in the order (larger logit, then smaller index);
//   top-p keeps, of those, the i with (sum of w before i in that order) < p * (sum of w kept
//   by top-k), and always the first; min-p keeps the i with w_i >= min_p.
//   token = the first kept i, in index order, with sum_{j <= i} w_j > u * Z, Z the kept sum.
// Each of the three keeps a beginning of the one order, so what is kept is a threshold
// (key, index) and no sort is needed.
//
// Weights are integers, round(w * 2^43): sums of them are exact in 64 bits (2^20 entries
// at most), so they come out the same in any order, atomics included, and the token is a
// function of the inputs alone. w itself is computed in fp64 (relative error below 2^-41):
// an fp32 exponential's 1e-7 would move the borders of a flat 128k-entry distribution by
// more than the gap that one row in a thousand leaves to its uniform number.
//
// One cluster of 1 to 8 CTAs per row; each keeps its share of the row in shared memory
// (what does not fit is read again), so that HBM is read once, and the passes over it
// meet through distributed shared memory:
//   load       the largest logit;
//   histogram  (top-k or top-p) entries counted in 4096 bins of x = (top - l) / t. Counts
//              give top-k's border bin; with each bin's largest and smallest weight they
//              bound where top-p's border lies, with its middle one they guess it;
//   weigh      the exact sums above and below those bins, whose own entries are listed;
//   decide     one CTA of the cluster sorts the list (64-bit (key, index)), finds the last
//              entry kept, and the CTA that the uniform number falls on; that one finds the
//              warp's run and the entry, weighing one run again. The exact sums show whether
//              the listed bins did hold the border.
// Rows of bf16 with top-k or top-p take a shorter way, `resolve_keys`: one bin per value,
// so that counts times weights decide without a list. Rows whose border bins hold more
// entries than the list (long runs of equal logits), or missed the border, take `select`
// instead: exact histograms of the weights, level by level down to one key.
//
// The row is read once from HBM, but HBM does not bound it: a cluster's life is a chain of
// phases (load, largest, histogram, its sums, borders, weights, decision, find), each behind
// a cluster barrier, with one shared-memory atomic an entry in the histogram and up to 10
// fp64 instructions an entry in the weights. Measured (B200): 256 rows of 128,256 bf16 96
// us (0.7 TB/s; the list's way took 238; 53 of them are the loads and barriers alone, as greedy
// rows show), 123 where the largest logits are 32 or more and `key_map` counts a second time,
// 64 rows of 152,064 bf16 with the tree walk 32 us, 534 rows of 128,256 with it 166 us, 8 rows
// of 32,000 fp32 21 us.
#include <cooperative_groups.h>

#include "ls_device.cuh"
#include "ls_verify_attn.h"
#include "sample_plan.cuh"
#include "tree_walk.cuh"

namespace ls {

namespace cg = cooperative_groups;

struct SampleArgs {
  const void* logits;
  int64_t row_stride;  // elements
  const float* uniform;
  const float* temperature;  // nullptr: 1
  const int32_t* top_k;      // nullptr: off
  const float* top_p;        // nullptr: off
  const float* min_p;        // nullptr: off
  int32_t* out;
  int32_t V, seg, cap;  // entries of the row, of a CTA's share, of the part kept in shared memory
  int32_t vec;          // rows start on 16-byte boundaries
};

namespace {

constexpr int kThreads = 512;  // two CTAs an SM: one's loads run under the other's arithmetic
constexpr int kWarps = kThreads / 32;
constexpr int kBins = kThreads;  // of `select`: one per thread
constexpr int kFine = 4096;      // bins of the first histogram
constexpr int kFinePer = kFine / kThreads;
constexpr int kFineUnit = 128;   // of them for one unit of x, where x spans the weights' whole range
constexpr int kList = 1024;      // entries of the border bins kept aside, two per thread
constexpr int kMaxVocab = 1 << 20;  // sums of 2^43 stay below 2^63
constexpr int kWeightBits = 43;
constexpr float kMaxX = 30.6f;  // exp(-30.6) is below half a unit
// a weight's three parts: a CTA's share is at most kMaxSeg entries, so their sums fit 32 bits
constexpr int kPartBits = 15;
constexpr int kLut = 1024;  // e^(-b / 32) * 2^43
constexpr int kKeys = 4096;  // bins of the histogram over bf16 values
constexpr int kKeysPer = kKeys / kThreads;  // of a group; the cluster has a group for each thread of a CTA
constexpr int kTable = kKeys / 2;           // weights that fit the histogram's place
constexpr int kMags = kKeys / 2;            // magnitudes of `plain_map`: 16 octaves of 128
constexpr int kMagEnd = 0x4200;             // their end, 32
constexpr int kTiny = 256;                  // entries below them kept aside
constexpr int kDataBytes = 76 * 1024;  // of the row, in shared memory
// It arrives in pieces of two 16-byte vectors a thread.
constexpr int kPieceVecs = 2, kPieces = (kDataBytes / 16 + kPieceVecs * kThreads - 1) / (kPieceVecs * kThreads);

using u64 = unsigned long long;

// Order-preserving key of a float: larger value, larger key (-0 and +0 get one key). NaN has
// no place in it: its weight is 0, and where entries are counted it is taken for -inf.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ uint32_t order_key(float x) { return key_of(x == x ? x : -INFINITY); }

// Place of an entry in the order: larger key first, then smaller index.
__device__ __forceinline__ u64 place_of(uint32_t key, uint32_t i) { return ((u64)~key << 32) | i; }

// The two ways to a row's threshold share the memory (a cluster barrier lies between).
struct Fast {
  uint32_t hist[kFine];  // later the sorted list (u64[kList])
  u64 list[kList];
};
struct Keys {
  union {
    uint32_t hist[kKeys];
    double weight[kTable];  // later: of the bins kept
  };
  u64 mass[kThreads];  // of this CTA's groups of bins
  uint32_t n_tiny;
  uint16_t small[kTiny];  // bits of the entries without a bin
};
struct Slow {
  u64 hist[kBins];          // this CTA's measure of each bin
  uint32_t part[3][kBins];  // its parts while they are added up
  uint32_t list[kList];
};
static_assert(sizeof(uint32_t) * kFine >= sizeof(u64) * kList && kList == 2 * kThreads, "sorted list");

// What the first histogram tells: top-k's border bin (kFine - 1: none) with the entries
// before it and in it, and the bins [lo, hi] that should hold top-p's border.
struct Borders {
  int bk;
  uint32_t above, in;
  int lo, hi;
};
// What the list decides: the place of the last entry kept, and the CTA whose share holds the
// target, with the sum before it. ok = 0: nothing (the list is too short, or elsewhere).
struct Verdict {
  u64 last, target, pre;
  int ok, owner;
};

// What the histogram over bf16 values decides: `edge` is the last value kept, `m` of its
// entries with it (each of weight w); ok = 0: nothing (values too small to have a bin).
struct KeyVerdict {
  u64 target, w;
  float edge;
  uint32_t m, bin;
  int ok;
};

struct Shared {
  double lut[kLut];
  union {
    Fast f;
    Keys k;
    Slow s;
  };
  u64 wsum[kWarps], scan[kWarps];
  u64 total;          // this CTA's sum
  u64 ws[3][kWarps];  // the warps' sums of `resolve`: kept for certain, under min-p, below the border
  u64 tot[3];         // and the CTA's
  u64 above, inside;  // measure before the border bin, and in it
  u64 last, before;
  Borders borders;
  Verdict verdict;
  KeyVerdict keys;
  uint32_t lpart[3][kWarps], cpart[3][kWarps];  // kept weights of the list, by run of this CTA and by CTA
  uint32_t n_list, kmin, kmax;                  // listed entries; `select`: keys of the border bin
  uint32_t bin, bins[3], in_range[2], cut;
  u64 tiny;  // weight of the entries without a bin
  uint32_t cwarp[kWarps];
  float fmax[kWarps], fmin[kWarps], fsum[kWarps];
  float top, low;
};

template <bool F32>
struct Row {
  const void* g;      // this CTA's share in global memory
  const void* s;      // its first `cap` entries in shared memory
  int n, cap;
  // entries i and i + 1 (i even); -inf past the share
  __device__ __forceinline__ void pair(int i, float& a, float& b) const {
    if (i + 1 < cap) {
      if constexpr (F32) {
        const float2 v = *reinterpret_cast<const float2*>(static_cast<const float*>(s) + i);
        a = v.x;
        b = v.y;
      } else {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(s) + i);
        a = __uint_as_float(v << 16);
        b = __uint_as_float(v & 0xffff0000u);
      }
      return;
    }
    a = i < n ? load(i) : -INFINITY;
    b = i + 1 < n ? load(i + 1) : -INFINITY;
  }
  // entries i .. of 16 bytes, all in shared memory
  __device__ __forceinline__ void vector(int i, float (&x)[F32 ? 4 : 8]) const {
    if constexpr (F32) {
      const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(s) + i);
      x[0] = v.x;
      x[1] = v.y;
      x[2] = v.z;
      x[3] = v.w;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(s) + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(w[e] << 16);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ uint4 words(int i) const {
    return *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(s) + (F32 ? 4 : 2) * i);
  }
  __device__ __forceinline__ float one(int i) const {
    if (i >= cap) return load(i);
    if constexpr (F32)
      return static_cast<const float*>(s)[i];
    else
      return bf16_to_f32(static_cast<const uint16_t*>(s)[i]);
  }
  __device__ __forceinline__ float load(int i) const {
    if constexpr (F32)
      return static_cast<const float*>(g)[i];
    else
      return bf16_to_f32(static_cast<const uint16_t*>(g)[i]);
  }
};

// What is kept so far: keys above `key`, and those equal to it up to entry `index`.
struct Keep {
  uint32_t key, index;
  __device__ __forceinline__ bool has(uint32_t k, uint32_t i) const { return k > key || (k == key && i <= index); }
};

// sum += w where a < b (and c >= d): one predicated addition, w having been computed anyway.
__device__ __forceinline__ void add_below(double& sum, double w, float a, float b) {
  asm("{\n\t.reg .pred p;\n\tsetp.lt.f32 p, %2, %3;\n\t@p add.rn.f64 %0, %0, %1;\n\t}"
      : "+d"(sum)
      : "d"(w), "f"(a), "f"(b));
}
__device__ __forceinline__ void add_below(double& sum, double w, float a, float b, float c, float d) {
  asm("{\n\t.reg .pred p;\n\tsetp.lt.f32 p, %2, %3;\n\tsetp.ge.and.f32 p, %4, %5, p;\n\t@p add.rn.f64 %0, %0, %1;\n\t}"
      : "+d"(sum)
      : "d"(w), "f"(a), "f"(b), "f"(c), "f"(d));
}

// Packed bf16 pairs, NaN skipped.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// sum += the double at shared address `at`, where a > b and a >= c.
__device__ __forceinline__ void add_above(double& sum, uint32_t at, float a, float b, float c) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .f64 v;\n\tmov.f64 v, 0d0000000000000000;\n\tsetp.gt.f32 p, %2, %3;\n\t"
      "setp.ge.and.f32 p, %2, %4, p;\n\t@p ld.shared.f64 v, [%1];\n\tadd.rn.f64 %0, %0, v;\n\t}"
      : "+d"(sum)
      : "r"(at), "f"(a), "f"(b), "f"(c)
      : "memory");
}

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <class T>
__device__ __forceinline__ T warp_scan(T v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T w = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += w;
  }
  return v;
}

template <bool F32>
class Sampler {
 public:
  __device__ Sampler(const SampleArgs& a, Shared& sh, void* data)
      : a_(a), sh_(sh), cl_(cg::this_cluster()), tid_(threadIdx.x), lane_(tid_ & 31), warp_(tid_ >> 5) {
    rank_ = (int)cl_.block_rank();
    size_ = (int)cl_.num_blocks();
    row_id_ = blockIdx.x / size_;
    lo_ = rank_ * a.seg;
    r_.n = max(0, min(a.seg, a.V - lo_));
    r_.cap = min(r_.n, a.cap) & ~1;
    const int64_t at = row_id_ * a.row_stride + lo_;
    r_.g = F32 ? static_cast<const void*>(static_cast<const float*>(a.logits) + at)
               : static_cast<const void*>(static_cast<const uint16_t*>(a.logits) + at);
    r_.s = data;
    // each warp's run of entries, in index order: whole steps of 16-byte reads where it is long
    const int per = (r_.n + kWarps - 1) / kWarps, whole = per >= 16 * 64 ? 32 * kPer : 64;
    run_ = (per + whole - 1) / whole * whole;
    w0_ = min(r_.n, warp_ * run_);
    w1_ = min(r_.n, w0_ + run_);
  }

  // A CTA's shared memory lives until its peers have read it: `leave` says that this CTA has,
  // `end` waits for the others'. (One that is done then makes room while another goes on.)
  __device__ __forceinline__ void leave() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    left_ = true;
  }
  __device__ __forceinline__ void end() {
    __syncwarp();
    if (!left_) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }

  __device__ void run() {
    load();
    for (int i = tid_; i < kLut; i += kThreads) sh_.lut[i] = exp(-(double)i / 32.0) * (double)(1ull << kWeightBits);
    const float t = a_.temperature != nullptr ? a_.temperature[row_id_] : 1.0f;
    int k = a_.top_k != nullptr ? a_.top_k[row_id_] : 0;
    if (k <= 0 || k >= a_.V) k = 0;
    const float p = a_.top_p != nullptr ? a_.top_p[row_id_] : 1.0f;
    // bf16 rows to be cut are counted while they arrive
    const bool cuts = k > 0 || p < 1.0f, counted = !F32 && cuts && t > 0.f && a_.vec;
    if (counted)
      count_arriving();
    else
      extremes();
    if (top_ == -INFINITY) {  // nothing above -inf
      if (rank_ == 0 && tid_ == 0) a_.out[row_id_] = 0;
      return;
    }
    if (!(t > 0.f)) {  // greedy: the first entry of the largest value
      const float top = top_;
      auto first = [top](float x, uint32_t) { return x == top ? 1ull : 0ull; };
      u64 before;
      sums(first, &before);
      leave();
      const int i = find(first, before, 0ull, w0_, w1_, sh_.wsum[warp_]);
      if (i >= 0) a_.out[row_id_] = i;
      return;
    }
    inv_t_ = 1.0 / (double)t;
    inv_f_ = (float)inv_t_;
    top_d_ = (double)top_;
    const uint32_t least = least_key(a_.min_p != nullptr ? a_.min_p[row_id_] : 0.0f, t);
    const float u = a_.uniform[row_id_];
    if constexpr (!F32) {
      if (cuts && !wide()) {
        KeyMap map;
        if (counted) {
          if (plain_map(t, &map) && resolve_keys(map, k, p, least, u)) return;
          cl_.sync();
        }
        if (key_map(t, &map)) {
          count_all(map);
          if (resolve_keys(map, k, p, least, u)) return;
        }
      }
      cl_.sync();  // the memory changes hands
    }
    if (!wide() && resolve(k, p, least, u)) return;
    cl_.sync();  // the memory changes hands
    Keep keep{0u, 0xffffffffu};
    if (k > 0) keep = select<false>(keep, top_ - low_, (u64)k, 0.0);
    if (p < 1.0f) keep = select<true>(keep, fminf(31.0f * t, top_ - low_), 0ull, (double)p);
    auto kept = [this, keep, least](float x, uint32_t i) {
      const uint32_t key = key_of(x);
      return key >= least && keep.has(key, i) ? weight_any(x) : 0ull;
    };
    u64 before;
    const u64 z = sums(kept, &before);
    leave();
    const int i = find(kept, before, target_of(u, z), w0_, w1_, sh_.wsum[warp_]);
    if (i >= 0) a_.out[row_id_] = i;
  }

 private:
  static constexpr int kPer = F32 ? 4 : 8;  // entries of 16 bytes
  const SampleArgs& a_;
  Shared& sh_;
  cg::cluster_group cl_;
  int tid_, lane_, warp_, rank_, size_, lo_, run_, w0_, w1_;
  bool left_ = false;  // the same in all threads
  int64_t row_id_;
  Row<F32> r_;
  float top_, low_;  // largest and smallest logit

  double inv_t_, top_d_;
  float inv_f_;

  // round(2^43 exp((l - top) / t)), as a double, where x = (top - l) / t is below 32 (xf: x in
  // fp32). exp(-x) = e^(-b / 32) * e^r with b the integer nearest to 32 x, |r| <= 2^-6, the
  // first factor from a table and the second by its Taylor polynomial to degree 5
  // (remainder 2^-36 / 720 = 2^-45). Adding and taking off 2^52 rounds to an integer.
  __device__ __forceinline__ double weight_in(float l, float xf) const {
    const int b = __float_as_int(fmaf(fminf(xf, 31.9f), 32.0f, 12582912.0f)) - 0x4b400000;
    const double fb = __hiloint2double(0x42e00000, b) - 140737488355328.0;  // (2^47 + b / 32) - 2^47
    const double r = fma((double)l - top_d_, inv_t_, fb);
    double e = fma(r, 1.0 / 120.0, 1.0 / 24.0);
    e = fma(e, r, 1.0 / 6.0);
    e = fma(e, r, 0.5);
    e = fma(e, r, 1.0);
    e = fma(e, r, 1.0);
    return fma(e, sh_.lut[b], 4503599627370496.0) - 4503599627370496.0;
  }
  // 0 beyond the range, and for NaN: of l, or of -inf under an infinite temperature
  __device__ __forceinline__ u64 weight(float l) const {
    const float xf = (top_ - l) * inv_f_;
    return xf < kMaxX ? (u64)weight_in(l, xf) : 0ull;
  }
  // The same for the rows that `resolve` leaves to `select`: top_ may be +inf, and x may not come
  // out of fp32 (`wide`).
  __device__ __forceinline__ u64 weight_any(float l) const {
    if (l == top_) return 1ull << kWeightBits;
    if (!wide()) return weight(l);
    const float xf = (float)((top_d_ - (double)l) * inv_t_);
    return xf < kMaxX ? (u64)weight_in(l, xf) : 0ull;
  }
  // Temperatures above 10^36, under which logits 2^128 apart are less than kMaxX units apart, and
  // those below 2^-128, whose reciprocals pass fp32.
  __device__ __forceinline__ bool wide() const { return inv_f_ < 1e-36f || inv_f_ == INFINITY; }

  __device__ __forceinline__ static u64 target_of(float u, u64 z) {
    const double at = u > 0.f ? (double)u * (double)z : 0.0;
    return at < (double)z ? min((u64)at, z - 1) : z - 1;
  }

  // The least key that min-p keeps: exp((l - top) / t) >= m, in fp64, for no lesser one.
  __device__ uint32_t least_key(float m, float t) const {
    if (!(m > 0.f) || top_ == INFINITY || inv_t_ == 0.0) return 0u;  // (t = inf: every finite logit weighs 1)
    const double x_min = m < 1.f ? log((double)m) : 0.0;
    auto keeps = [&](uint32_t key) { return ((double)of_key(key) - top_d_) * inv_t_ >= x_min; };
    uint32_t key = key_of((float)(top_d_ + x_min * (double)t));  // off by rounding
    const uint32_t most = key_of(top_);
    for (int i = 0; i < 4 && key < most && !keeps(key); ++i) ++key;
    for (int i = 0; i < 4 && keeps(key - 1); ++i) --key;
    return min(key, most);
  }

  // f(16 bytes) over this warp's run where they lie in shared memory, g(value) over the rest
  template <class F, class G>
  __device__ __forceinline__ void each_words(F f, G g) const {
    const int whole = w0_ + max(0, min(w1_, r_.cap) - w0_) / kPer * kPer;
    for (int i = w0_ + kPer * lane_; i < whole; i += 32 * kPer) f(r_.words(i));
    for (int i = whole + lane_; i < w1_; i += 32) g(r_.one(i));
  }
  // f(values, entry of the first) over this warp's run, 16 bytes a lane and step (NaN, which
  // weighs nothing, beyond its end)
  template <class F>
  __device__ __forceinline__ void each_vector(F f) const {
    const int whole = w0_ + max(0, min(w1_, r_.cap) - w0_) / kPer * kPer;
    float x[kPer];
    for (int i = w0_ + kPer * lane_; i < whole; i += 32 * kPer) {
      r_.vector(i, x);
      f(x, (uint32_t)(lo_ + i));
    }
#pragma unroll
    for (int e = 1; e < kPer; ++e) x[e] = __uint_as_float(0x7fffffffu);
    for (int i = whole + lane_; i < w1_; i += 32) {
      x[0] = r_.one(i);
      f(x, (uint32_t)(lo_ + i));
    }
  }
  // f(value, entry of the row) over this warp's run
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    const int whole = w0_ + max(0, min(w1_, r_.cap) - w0_) / kPer * kPer;
    for (int i = w0_ + kPer * lane_; i < whole; i += 32 * kPer) {
      float x[kPer];
      r_.vector(i, x);
#pragma unroll
      for (int e = 0; e < kPer; ++e) f(x[e], (uint32_t)(lo_ + i + e));
    }
    for (int i = whole + lane_; i < w1_; i += 32) f(r_.one(i), (uint32_t)(lo_ + i));
  }

  // Starts the copy of the share into shared memory; `extremes` waits for it.
  __device__ void load() {
    const int n_vec = a_.vec ? r_.cap / kPer : 0;
    uint8_t* to = static_cast<uint8_t*>(const_cast<void*>(r_.s));
    const uint8_t* from = static_cast<const uint8_t*>(r_.g);
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
#pragma unroll
      for (int e = 0; e < kPieceVecs; ++e) {
        const int v = (c * kPieceVecs + e) * kThreads + tid_;
        if (v < n_vec)
          asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(at + 16 * v), "l"(from + 16 * (int64_t)v) : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    for (int i = n_vec * kPer + tid_; i < r_.cap; i += kThreads) {
      if constexpr (F32)
        reinterpret_cast<float*>(to)[i] = static_cast<const float*>(r_.g)[i];
      else
        reinterpret_cast<uint16_t*>(to)[i] = static_cast<const uint16_t*>(r_.g)[i];
    }
  }

  // The largest and smallest of what `take` saw; NaN skipped.
  struct Ends {
    float mx = -INFINITY, mn = INFINITY;
    uint32_t m2 = 0xff80ff80u, n2 = 0x7f807f80u;  // -inf, +inf
    __device__ __forceinline__ void take(float x) {
      mx = fmaxf(mx, x);
      mn = fminf(mn, x);
    }
    __device__ __forceinline__ void take(const uint4& v) {  // of bf16
      m2 = max_bf16x2(m2, max_bf16x2(max_bf16x2(v.x, v.y), max_bf16x2(v.z, v.w)));
      n2 = min_bf16x2(n2, min_bf16x2(min_bf16x2(v.x, v.y), min_bf16x2(v.z, v.w)));
    }
    __device__ __forceinline__ void join() {
      mx = fmaxf(mx, fmaxf(__uint_as_float(m2 << 16), __uint_as_float(m2 & 0xffff0000u)));
      mn = fminf(mn, fminf(__uint_as_float(n2 << 16), __uint_as_float(n2 & 0xffff0000u)));
    }
  };

  // The row's largest and smallest logit.
  __device__ void extremes() {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    Ends ends;
    if constexpr (F32)
      each([&](float x, uint32_t) { ends.take(x); });
    else
      each_words([&](const uint4& v) { ends.take(v); }, [&](float x) { ends.take(x); });
    share_ends(ends);
  }
  // top_ and low_ from the threads' ends; a barrier of the cluster.
  __device__ void share_ends(Ends& ends) {
    if constexpr (!F32) ends.join();
    float mx = ends.mx, mn = ends.mn;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    }
    if (lane_ == 0) {
      sh_.fmax[warp_] = mx;
      sh_.fmin[warp_] = mn;
    }
    __syncthreads();
    if (warp_ == 0) {
      mx = lane_ < kWarps ? sh_.fmax[lane_] : -INFINITY;
      mn = lane_ < kWarps ? sh_.fmin[lane_] : INFINITY;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      }
      if (lane_ == 0) {
        sh_.top = mx;
        sh_.low = mn;
      }
    }
    cl_.sync();
    top_ = -INFINITY;
    low_ = INFINITY;
    for (int c = 0; c < size_; ++c) {
      const Shared* o = cl_.map_shared_rank(&sh_, c);
      top_ = fmaxf(top_, o->top);
      low_ = fminf(low_, o->low);
    }
  }

  // Sum of f over the row; *before: its part in the shares and runs before this warp's.
  template <class F>
  __device__ u64 sums(F f, u64* before) {
    u64 s = 0;
    each([&](float x, uint32_t i) { s += f(x, i); });
    s = warp_sum64(s);
    if (lane_ == 0) sh_.wsum[warp_] = s;
    __syncthreads();
    u64 in_cta = 0, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp_) in_cta += sh_.wsum[w];
      all += sh_.wsum[w];
    }
    if (tid_ == 0) sh_.total = all;
    cl_.sync();
    u64 z = 0, pre = 0;
    for (int c = 0; c < size_; ++c) {
      const u64 o = cl_.map_shared_rank(&sh_, c)->total;
      if (c < rank_) pre += o;
      z += o;
    }
    *before = pre + in_cta;
    return z;
  }

  // The entry of [i0, i1) at which the running sum of f, which is `before` at i0 and grows by
  // `sum` over it, first exceeds `target`: returned by one lane of the warp that holds it, -1
  // by every other thread.
  template <class F>
  __device__ int find(F f, u64 before, u64 target, int i0, int i1, u64 sum) {
    if (target < before || target >= before + sum) return -1;
    for (; i0 < i1; i0 += 64) {
      const int i = i0 + 2 * lane_;
      u64 wa = 0, wb = 0;
      if (i < i1) {
        float x, y;
        r_.pair(i, x, y);
        wa = f(x, (uint32_t)(lo_ + i));
        if (i + 1 < i1) wb = f(y, (uint32_t)(lo_ + i + 1));
      }
      const u64 inc = warp_scan(wa + wb, lane_);
      const u64 step = __shfl_sync(0xffffffffu, inc, 31);
      if (target < before + step) {
        const u64 start = before + inc - wa - wb;
        if (target >= start && target < start + wa) return lo_ + i;
        if (target >= start + wa && target < start + wa + wb) return lo_ + i + 1;
        return -1;
      }
      before += step;
    }
    return -1;
  }

  // Sums of weights by 32-bit atomics: three parts, each of fewer than 2^17 entries.
  __device__ __forceinline__ static void add_parts(uint32_t (&part)[3][kWarps], int at, u64 w) {
    constexpr uint32_t m = (1u << kPartBits) - 1u;
    atomicAdd(&part[0][at], (uint32_t)w & m);
    atomicAdd(&part[1][at], (uint32_t)(w >> kPartBits) & m);
    atomicAdd(&part[2][at], (uint32_t)(w >> (2 * kPartBits)));
  }
  __device__ __forceinline__ static u64 parts(const uint32_t (&part)[3][kWarps], int at) {
    return (u64)part[0][at] + ((u64)part[1][at] << kPartBits) + ((u64)part[2][at] << (2 * kPartBits));
  }

  // The first histogram (bin b holds the entries whose x is nearest to b * step; logits of
  // few bits then lie in the middle of their bins, which the guess wants): top-k's border bin
  // with the entries before it and in it (none where k entries outnumber those with a weight),
  // and the bins [lo, hi] one of which holds top-p's border.
  __device__ Borders borders(float per, float step, uint32_t k, float p) {
    uint32_t* hist = sh_.f.hist;
    for (int i = tid_; i < kFine / 4; i += kThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    const float top = top_;
    each([&](float x, uint32_t) {
      const float v = fmaf(top - x, per, 0.5f);
      if (v < (float)(kFine - 1)) atomicAdd(&hist[(int)v], 1u);  // what lies beyond has no weight
    });
    cl_.sync();
    // Each CTA adds up its share of the bins over the cluster, in place (no other CTA reads
    // that share of its histogram), and one CTA looks through the sums: with other rows' CTAs
    // on the same SMs, what a cluster does twice costs time.
    if (size_ > 1) {
      const int share = kFine / 4 / size_;
      for (int i = rank_ * share + tid_; i < (rank_ + 1) * share; i += kThreads) {
        uint4 v[kMaxCluster];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < size_) v[r] = reinterpret_cast<const uint4*>(cl_.map_shared_rank(&sh_, r)->f.hist)[i];
#pragma unroll
        for (int r = 1; r < kMaxCluster; ++r)
          if (r < size_) {
            v[0].x += v[r].x;
            v[0].y += v[r].y;
            v[0].z += v[r].z;
            v[0].w += v[r].w;
          }
        reinterpret_cast<uint4*>(hist)[i] = v[0];
      }
      cl_.sync();
    }
    if (rank_ == 0) look(step, k, p);
    cl_.sync();
    return cl_.map_shared_rank(&sh_, 0)->borders;
  }

  // The borders from the summed histogram, into this CTA's sh_.borders.
  __device__ void look(float step, uint32_t k, float p) {
    uint32_t c[kFinePer];
#pragma unroll
    for (int e = 0; e < kFinePer / 4; ++e) {
      const int i = tid_ * (kFinePer / 4) + e;
      const Shared* o = cl_.map_shared_rank(&sh_, i / (kFine / 4 / size_));
      const uint4 v = reinterpret_cast<const uint4*>(o->f.hist)[i];
      c[4 * e] = v.x;
      c[4 * e + 1] = v.y;
      c[4 * e + 2] = v.z;
      c[4 * e + 3] = v.w;
    }
    if (tid_ == 0) {
      sh_.borders = Borders{kFine - 1, 0u, 0u, 0, -1};
      sh_.bins[0] = sh_.bins[1] = sh_.bins[2] = kFine - 2;
      sh_.in_range[0] = sh_.in_range[1] = 0u;
    }
    uint32_t own = 0;
#pragma unroll
    for (int e = 0; e < kFinePer; ++e) own += c[e];
    const uint32_t inc = warp_scan(own, lane_);
    if (lane_ == 31) sh_.cwarp[warp_] = inc;
    __syncthreads();
    uint32_t before = inc - own;
    for (int w = 0; w < warp_; ++w) before += sh_.cwarp[w];
#pragma unroll
    for (int e = 0; e < kFinePer; ++e) {
      const int b = kFinePer * tid_ + e;
      if (k > 0 && b < kFine - 1 && before < k && k <= before + c[e]) sh_.borders = Borders{b, before, c[e], 0, -1};
      before += c[e];
    }
    __syncthreads();
    const int bk = sh_.borders.bk;
    const uint32_t above = sh_.borders.above;
    if (p < 0.f) return;
    // The weight of each bin's middle, times its entries that top-k leaves; the bin's largest
    // and smallest are off from it by the same factors in every bin.
    float v[kFinePer], sum = 0.f;
#pragma unroll
    for (int e = 0; e < kFinePer; ++e) {
      const int b = kFinePer * tid_ + e;
      uint32_t cnt = b < bk ? c[e] : 0u;
      if (b == bk && b < kFine - 1) cnt = k - above;
      if (b == kFine - 1) cnt = 0u;
      sum += (float)cnt * __expf(-(float)b * step);
      v[e] = sum;
    }
    float pre = warp_scan(sum, lane_), all = 0.f;
    if (lane_ == 31) sh_.fsum[warp_] = pre;
    pre -= sum;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp_) pre += sh_.fsum[w];
      all += sh_.fsum[w];
    }
    // The first bins whose running sums reach the goal: for certain in [bins[0], bins[1]]
    // (widened by far more than the rounding of bins and sums), and most likely, by the
    // middles, near bins[2]: their sums are off by the entries' places in their bins, which
    // nearly average out.
    const float off = __expf(step) * 1.0002f;
    const float goal[3] = {p * all / off, p * all * off, p * all};
    uint32_t first[3] = {kFine - 2, kFine - 2, kFine - 2};
#pragma unroll
    for (int e = kFinePer - 1; e >= 0; --e)
#pragma unroll
      for (int q = 0; q < 3; ++q)
        if (pre + v[e] >= goal[q]) first[q] = kFinePer * tid_ + e;
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      first[q] = __reduce_min_sync(0xffffffffu, first[q]);
      if (lane_ == 0 && first[q] < kFine - 2) atomicMin(&sh_.bins[q], first[q]);
    }
    __syncthreads();
    // the widest of three ranges whose entries the list holds: the certain one where it is
    // short, else two bins on either side of the likely one, or one
    const int a = (int)sh_.bins[0], z = min((int)sh_.bins[1], bk), mid = (int)sh_.bins[2];
    const int from[3] = {a, max(a, mid - 2), max(a, mid - 1)}, to[3] = {z, min(z, mid + 2), min(z, mid + 1)};
    uint32_t in_range[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < kFinePer; ++e) {
      const int b = kFinePer * tid_ + e;
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (b >= from[q] && b <= to[q]) in_range[q] += c[e];
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      in_range[q] = __reduce_add_sync(0xffffffffu, in_range[q]);
      if (lane_ == 0 && in_range[q]) atomicAdd(&sh_.in_range[q], in_range[q]);
    }
    __syncthreads();
    const int q = sh_.in_range[0] <= kList / 4 ? 0 : sh_.in_range[1] <= kList - kList / 8 ? 1 : 2;
    if (tid_ == 0) {
      sh_.borders.lo = from[q];
      sh_.borders.hi = to[q];
    }
  }

  // Sorts v[0 .. n) ascending; n2: a power of two of at least 64, n and at most 2 * kThreads, up
  // to which v is padded with ~0. Short lists by counting the entries before each (n steps,
  // all independent: 8% off a call with top-k, whose lists are short; at 400 entries 3% more
  // than the other), longer ones bitonic: a warp holds 64 entries in registers, so that distances below 64 are shuffles
  // and only the longer ones go through shared memory and the CTA's barrier.
  __device__ void sort(u64* v, uint32_t n, uint32_t n2) {
    if (n <= (uint32_t)kThreads / 2) {
      const u64 own = v[min((uint32_t)tid_, n2 - 1)];
      uint32_t at = 0;
      if (64u * (tid_ / 64) < n)  // whole warps
#pragma unroll 8
        for (uint32_t j = 0; j < n2; j += 2) {
          const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(v + j);
          at += (w.x < own ? 1u : 0u) + (w.y < own ? 1u : 0u);
        }
      __syncthreads();
      if ((uint32_t)tid_ < n) v[at] = own;  // places differ
      __syncthreads();
      return;
    }
    const uint32_t i = 64 * warp_ + lane_;  // this thread's entries: i and i + 32
    const bool works = 64u * warp_ < n2;    // whole warps
    u64 a = 0, b = 0;
    if (works) {
      a = v[i];
      b = v[i + 32];
    }
    for (uint32_t k = 2; k <= n2; k *= 2) {
      const bool up_a = (i & k) == 0, up_b = ((i + 32) & k) == 0;
      for (uint32_t j = k / 2; j > 0; j /= 2) {
        if (j >= 64) {
          if (works) {
            v[i] = a;
            v[i + 32] = b;
          }
          __syncthreads();
          if (works) {
            const u64 x = v[i ^ j], y = v[(i + 32) ^ j];
            const bool low = (i & j) == 0;
            a = (a < x) == (low == up_a) ? a : x;
            b = (b < y) == (low == up_b) ? b : y;
          }
          __syncthreads();
        } else if (works) {
          if (j == 32) {
            if ((a > b) == up_a) {
              const u64 x = a;
              a = b;
              b = x;
            }
          } else {
            const u64 x = __shfl_xor_sync(0xffffffffu, a, j), y = __shfl_xor_sync(0xffffffffu, b, j);
            const bool low = (lane_ & j) == 0;
            a = (a < x) == (low == up_a) ? a : x;
            b = (b < y) == (low == up_b) ? b : y;
          }
        }
      }
    }
    if (works) {
      v[i] = a;
      v[i + 32] = b;
    }
    __syncthreads();
  }

  // Rank 0, after the cluster's sums and lists are there: the verdict, into its sh_.verdict.
  __device__ void decide(const Borders& at, bool cut, bool nucleus, int k, float p, uint32_t least, float u) {
    if (tid_ == 0) sh_.verdict.ok = 0;
    u64 keep_all = 0, under = 0, rest = 0;
    uint32_t n = 0, from[kMaxCluster];
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
      from[c] = n;
      if (c < size_) {
        const Shared* o = cl_.map_shared_rank(&sh_, c);
        keep_all += o->tot[0];
        under += o->tot[1];
        rest += o->tot[2];
        n += o->n_list;
      }
    }
    if (n == 0 || n > (uint32_t)kList) return;
    u64* v = reinterpret_cast<u64*>(sh_.f.hist);  // read by no other CTA any more
    uint32_t n2 = 64;
    while (n2 < n) n2 *= 2;
    for (uint32_t j = tid_; j < n; j += kThreads) {
      int c = 0;
      uint32_t at_c = 0;
#pragma unroll
      for (int q = 1; q < kMaxCluster; ++q)
        if (q < size_ && from[q] <= j) {
          c = q;
          at_c = from[q];
        }
      v[j] = cl_.map_shared_rank(&sh_, c)->f.list[j - at_c];
    }
    for (uint32_t j = n + tid_; j < n2; j += kThreads) v[j] = ~0ull;
    __syncthreads();
    sort(v, n, n2);
    const uint32_t j0 = 2 * tid_;
    u64 w[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) w[e] = j0 + e < n ? weight(of_key(~(uint32_t)(v[j0 + e] >> 32))) : 0ull;
    u64 before = warp_scan(w[0] + w[1], lane_);
    if (lane_ == 31) sh_.scan[warp_] = before;
    __syncthreads();
    before -= w[0] + w[1];
    for (int i = 0; i < warp_; ++i) before += sh_.scan[i];
    // the list in order: top-p's bins, then top-k's border bin (the same, or a later one)
    const uint32_t start_k = cut ? n - at.in : n;
    const uint32_t end = cut ? start_k + ((uint32_t)k - at.above) : n;  // top-k keeps those before
    const uint32_t lim = nucleus ? min(end, cut && at.hi < at.bk ? start_k : n) : end;
    uint32_t m = end;
    if (nucleus) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // weight before entries `end` and `lim` (both at most kList)
        const u64 b = e ? before + w[0] : before;
        if (j0 + e == end) sh_.last = b;
        if (j0 + e == lim) sh_.before = b;
      }
      if (tid_ == kThreads - 1) {
        if (end == kList) sh_.last = before + w[0] + w[1];
        if (lim == kList) sh_.before = before + w[0] + w[1];
      }
      __syncthreads();
      const u64 sure = keep_all + under, z = sure + rest + sh_.last;
      const double g = ceil((double)p * (double)z);
      const u64 goal = g >= 1.0 ? min((u64)g, z) : 1ull;
      // the border lies inside the list, or it is not decided here
      const bool inside = sure < goal && sure + sh_.before >= goal;
      m = (uint32_t)__syncthreads_count(j0 < lim && sure + before < goal);
      m += (uint32_t)__syncthreads_count(j0 + 1 < lim && sure + before + w[0] < goal);
      if (!inside) return;
    }
    const u64 last = v[m - 1];  // m >= 1: k exceeds the entries above its bin, and sure < goal
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (j0 + e >= m) continue;
      const u64 place = v[j0 + e];
      if (~(uint32_t)(place >> 32) >= least) add_parts(sh_.cpart, (int)(uint32_t)place / a_.seg, w[e]);
    }
    __syncthreads();
    if (tid_ == 0) {
      u64 z = keep_all;
      for (int c = 0; c < size_; ++c) z += parts(sh_.cpart, c);
      Verdict o{last, target_of(u, z), 0, 1, 0};
      u64 mine = cl_.map_shared_rank(&sh_, 0)->tot[0] + parts(sh_.cpart, 0);
      while (o.owner < size_ - 1 && o.target >= o.pre + mine) {
        o.pre += mine;
        ++o.owner;
        mine = cl_.map_shared_rank(&sh_, o.owner)->tot[0] + parts(sh_.cpart, o.owner);
      }
      sh_.verdict = o;
    }
  }

  // ---- bf16 rows: one bin per value
  //
  // Logits of 8 significant bits have few values: those that weigh anything lie within
  // [top - 31 t, top], some 4000 of them down to 2^-13. Bins for each, in falling order, make
  // the histogram exact: thresholds and sums come from counts times weights, without a list,
  // and what is left to do for the entries themselves is to add up the kept ones' weights by
  // runs, from a table, in the one CTA that holds the token. Smaller magnitudes have no bin:
  // their few entries' weights are added up one by one, which does unless the threshold falls
  // among them; then `resolve` decides.
  //
  // Bins for magnitudes from 2^-11 to 32 (`plain`) ask for no largest logit, so rows inside
  // are counted while they arrive; others once it is known, in bins below it (`key_map`).
  // 256 rows of 128,256, top-p 0.9, stage by stage (us): launches 10, load 10, count 29 (a
  // shared-memory atomic an entry), sums over the cluster 10, border 9, kept weight by CTA
  // 11, by run 12, the token 7.
  struct KeyMap {
    int ptop, pos, zero, neg0, least, count;  // bins: ptop - magnitude (`pos` of them) | zero | neg0 + magnitude
    __device__ __forceinline__ int bin(uint32_t u) const {  // of a bf16's bits; not in [0, count): none
      const int mag = (int)(u & 0x7fffu);
      if (mag < least) return mag == 0 ? zero : -1;
      return (u & 0x8000u) ? neg0 + mag : ptop - mag;
    }
    // the same of bits whose magnitude is at least `least`
    __device__ __forceinline__ int large_bin(uint32_t u) const {
      const int neg = (int)(u << 16) >> 31;
      return ((int)(u & 0x7fffu) ^ ~neg) + (neg ? neg0 : ptop + 1);
    }
    __device__ __forceinline__ int after_tiny() const { return zero >= 0 ? zero + 1 : pos; }  // bins below those without one
    __device__ __forceinline__ float tiny_end() const { return __uint_as_float((uint32_t)least << 16); }  // their magnitudes are less
    __device__ __forceinline__ float value(int b) const {
      if (b < pos) return __uint_as_float((uint32_t)(ptop - b) << 16);
      return b == zero ? 0.f : -__uint_as_float((uint32_t)(b - neg0) << 16);
    }
  };
  // Bins that do not depend on the row: magnitudes from 2^-11 to 32. Smaller ones, 0 too, have none.
  __device__ __forceinline__ static KeyMap plain() {
    return KeyMap{kMagEnd - 1, kMags, -1, 2 * kMags - kMagEnd, kMagEnd - kMags, kKeys};
  }
  // Counts the row in them while it arrives, each thread the vectors that it copies itself, and
  // finds its ends.
  __device__ void count_arriving() {
    const KeyMap map = plain();
    uint32_t* hist = sh_.k.hist;
    for (int i = tid_; i < kKeys / 4; i += kThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid_ == 0) {
      sh_.k.n_tiny = 0u;
      sh_.tiny = 0ull;
    }
    __syncthreads();
    Ends ends;
    auto count = [&](uint32_t bits) {
      const int b = map.bin(bits);
      if ((uint32_t)b < (uint32_t)kKeys) {
        atomicAdd(&hist[b], 1u);
      } else if (b == -1) {
        const uint32_t at = atomicAdd(&sh_.k.n_tiny, 1u);
        if (at < kTiny) sh_.k.small[at] = (uint16_t)bits;
      }
    };
    const int n_vec = r_.cap / kPer;
    auto piece = [&](int c) {
#pragma unroll
      for (int e = 0; e < kPieceVecs; ++e) {
        const int i = (c * kPieceVecs + e) * kThreads + tid_;
        if (i >= n_vec) break;
        const uint4 v = r_.words(i * kPer);
        ends.take(v);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t small = 0x7fff7fffu;
#pragma unroll
        for (int q = 0; q < 4; ++q) small = __vminu2(small, w[q] & 0x7fff7fffu);
        if (min(small & 0xffffu, small >> 16) < (uint32_t)map.least) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            count(w[q] & 0xffffu);
            count(w[q] >> 16);
          }
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int a = map.large_bin(w[q] & 0xffffu), b = map.large_bin(w[q] >> 16);
            if ((uint32_t)a < (uint32_t)kKeys) atomicAdd(&hist[a], 1u);
            if ((uint32_t)b < (uint32_t)kKeys) atomicAdd(&hist[b], 1u);
          }
        }
      }
    };
    static_assert(kPieces == 5, "the waits below");
    asm volatile("cp.async.wait_group 4;" ::: "memory");
    piece(0);
    asm volatile("cp.async.wait_group 3;" ::: "memory");
    piece(1);
    asm volatile("cp.async.wait_group 2;" ::: "memory");
    piece(2);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    piece(3);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    piece(4);
    for (int i = n_vec * kPer + tid_; i < r_.n; i += kThreads) {  // the share's end, and what has no room
      const float x = r_.load(i);
      ends.take(x);
      count(__float_as_uint(x) >> 16);
    }
    share_ends(ends);
  }
  // `plain`, where it holds what weighs anything in this row (whose histogram is there).
  __device__ bool plain_map(float t, KeyMap* k) {
    if (!(inv_f_ > 0.f && inv_f_ < INFINITY)) return false;
    const float end = __uint_as_float((uint32_t)kMagEnd << 16);
    bool fits = true;
    for (int c = 0; c < size_; ++c) fits &= cl_.map_shared_rank(&sh_, c)->k.n_tiny <= kTiny;
    if (!fits || !(top_ < end) || !(low_ > -end || top_ - kMaxX * t > -end)) return false;
    *k = plain();
    const uint32_t n = sh_.k.n_tiny;
    for (uint32_t j = tid_; j < n; j += kThreads) {
      const u64 w = weight(__uint_as_float((uint32_t)sh_.k.small[j] << 16));
      if (w) atomicAdd(&sh_.tiny, w);
    }
    return true;
  }
  // The map for this row; false where its range of values has no room.
  __device__ bool key_map(float t, KeyMap* k) const {
    if (!(inv_f_ > 0.f && inv_f_ < INFINITY)) return false;
    const float low = top_ - kMaxX * t;  // below it, weights are 0
    if (!(low < top_) || top_ == INFINITY) return false;
    const int last = low < 0.f ? (int)min(__float_as_uint(-low) >> 16, 0x7f7eu) + 1 : 0;  // largest magnitude below 0
    if (top_ > 0.f) {
      const int p = (int)(__float_as_uint(top_) >> 16);
      // bins: p - least + 1, the zero, last - least + 1
      const int least = max(1, last > 0 ? (p + last + 4 - kKeys) / 2 : p + 2 - kKeys);
      if (least > p) return false;
      const int zero = p - least + 1;
      *k = KeyMap{p, zero, zero, zero + 1 - least, least, last >= least ? zero + 2 - least + last : zero + 1};
    } else if (top_ == 0.f) {
      const int least = max(1, last + 2 - kKeys);
      *k = KeyMap{-1, 0, 0, 1 - least, least, last >= least ? 2 - least + last : 1};
    } else {
      const int p = (int)(__float_as_uint(-top_) >> 16);
      *k = KeyMap{-1, 0, -1, -p, p, last - p + 1};
    }
    return k->count <= kKeys && k->count > 0;
  }

  // Counts the row in the map's bins.
  __device__ void count_all(const KeyMap& map) {
    uint32_t* hist = sh_.k.hist;
    for (int i = tid_; i < kKeys / 4; i += kThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid_ == 0) {
      sh_.tiny = 0ull;
      sh_.k.n_tiny = 0u;
    }
    __syncthreads();
    u64 tiny = 0;
    uint32_t n_tiny = 0;
    auto count = [&](uint32_t bits) {
      const int b = map.bin(bits);
      if ((uint32_t)b < (uint32_t)map.count) {
        atomicAdd(&hist[b], 1u);
      } else if (b == -1) {
        tiny += weight(__uint_as_float(bits << 16));
        ++n_tiny;
      }
    };
    each_words(
        [&](const uint4& v) {
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t small = 0x7fff7fffu;
#pragma unroll
          for (int e = 0; e < 4; ++e) small = __vminu2(small, w[e] & 0x7fff7fffu);
          if (min(small & 0xffffu, small >> 16) < (uint32_t)map.least) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              count(w[e] & 0xffffu);
              count(w[e] >> 16);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int a = map.large_bin(w[e] & 0xffffu), b = map.large_bin(w[e] >> 16);
              if ((uint32_t)a < (uint32_t)map.count) atomicAdd(&hist[a], 1u);
              if ((uint32_t)b < (uint32_t)map.count) atomicAdd(&hist[b], 1u);
            }
          }
        },
        [&](float x) { count(__float_as_uint(x) >> 16); });
    if (tiny) atomicAdd(&sh_.tiny, tiny);
    if (n_tiny) atomicAdd(&sh_.k.n_tiny, n_tiny);
    cl_.sync();
  }

  // The row's token from the CTAs' counts; false where they do not tell. The sums over the
  // cluster decide the border; every CTA's own counts then give its kept weight, and only the
  // one that the target falls in goes through its entries again.
  __device__ bool resolve_keys(const KeyMap& map, int k, float p, uint32_t least, float u) {
    uint4* hist = reinterpret_cast<uint4*>(sh_.k.hist);
    const int share = kKeys / 4 / size_, in_share = rank_ * share + tid_;  // groups of four bins
    static_assert(kKeys / 4 / 2 <= kThreads, "a thread adds up four bins");
    uint4 own = make_uint4(0u, 0u, 0u, 0u);  // this CTA's counts where the sums take their place
    if (tid_ < 2) sh_.tot[tid_] = 0ull;
    if (size_ > 1) {
      if (tid_ < share) {
        uint4 v[kMaxCluster];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < size_) v[r] = reinterpret_cast<const uint4*>(cl_.map_shared_rank(&sh_, r)->k.hist)[in_share];
        own = hist[in_share];
#pragma unroll
        for (int r = 1; r < kMaxCluster; ++r)
          if (r < size_) {
            v[0].x += v[r].x;
            v[0].y += v[r].y;
            v[0].z += v[r].z;
            v[0].w += v[r].w;
          }
        hist[in_share] = v[0];
      }
      __syncthreads();
    }
    {  // its groups' weights, size_ threads a group
      const int g = tid_ / size_, b0 = (rank_ * (kThreads / size_) + g) * kKeysPer;
      u64 mass = 0;
      for (int e = tid_ % size_; e < kKeysPer; e += size_) {
        const uint32_t c = sh_.k.hist[b0 + e];
        if (c) mass += c * weight(map.value(b0 + e));
      }
      for (int o = size_ / 2; o > 0; o /= 2) mass += __shfl_xor_sync(0xffffffffu, mass, o);
      if (tid_ % size_ == 0) sh_.k.mass[g] = mass;
    }
    cl_.sync();
    if (rank_ == 0) look_keys(map, (uint32_t)k, p, least, u);
    cl_.sync();
    const KeyVerdict o = cl_.map_shared_rank(&sh_, 0)->keys;
    if (!o.ok) return false;
    const int whole = (int)o.bin;  // bins kept whole
    const float least_f = least > 0u ? of_key(least) : -INFINITY, edge = o.edge;
    const uint32_t cut = edge >= least_f ? o.m : 0u;  // of the edge's own entries, the first `cut` are kept
    {  // this CTA's kept weight but for the edge's entries, and their number
      // (those without a bin are kept all or none: `ok` says so)
      u64 keep = tid_ == 0 && whole >= map.after_tiny() && least_f <= -map.tiny_end() ? sh_.tiny : 0ull;
      auto four = [&](uint4 v, int b) {
#pragma unroll 1  // (code that runs once costs its fetching)
        for (int e = 0; e < 4; ++e, ++b) {
          if (v.x && b < whole && map.value(b) >= least_f) keep += v.x * weight(map.value(b));
          if (b == whole) sh_.tot[1] = v.x;
          v = make_uint4(v.y, v.z, v.w, 0u);
        }
      };
#pragma unroll 1
      for (int i = tid_; i < kKeys / 4 + kThreads; i += kThreads) {
        const bool rest = i >= kKeys / 4;  // at last, the counts that the sums replaced
        const int at = rest ? in_share : i;
        if ((rest ? size_ > 1 && tid_ < share : size_ == 1 || i / share != rank_) && 4 * at <= whole)
          four(rest ? own : hist[at], 4 * at);
      }
      if (__any_sync(0xffffffffu, keep != 0ull)) {
        keep = warp_sum64(keep);
        if (lane_ == 0) atomicAdd(&sh_.tot[0], keep);
      }
    }
    cl_.sync();
    // the CTA, the warp's run, and the part of it that the target falls in; `pre`: kept weight
    // before it, `seen`: the edge's entries before it
    auto kept_of = [&](u64 whole_w, uint32_t n, uint32_t seen) {
      return whole_w + (u64)(min(seen + n, cut) - min(seen, cut)) * o.w;
    };
    u64 pre = 0, cta_w[kMaxCluster];
    uint32_t seen = 0, cta_n[kMaxCluster];
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c)
      if (c < size_) {
        const Shared* q = cl_.map_shared_rank(&sh_, c);
        cta_w[c] = q->tot[0];
        cta_n[c] = (uint32_t)q->tot[1];
      }
    leave();
    int owner = -1;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c)
      if (c < size_ && owner < 0) {
        const u64 mine = kept_of(cta_w[c], cta_n[c], seen);
        if (o.target < pre + mine) {
          owner = c;
        } else {
          pre += mine;
          seen += cta_n[c];
        }
      }
    if (owner != rank_) return true;
    // Weights of the values kept whole, where the histogram was: those above a positive edge, or
    // above a negative one but for the smallest magnitudes, as many as there is room for.
    const int tm = top_ > 0.f ? (int)(__float_as_uint(top_) >> 16) : 0;
    const int em = (int)(__float_as_uint(fabsf(edge)) >> 16);
    KeyMap tab{tm, tm - em, -1, 0, 0, tm - em <= kTable ? tm - em : 0};  // of a positive edge
    if (!(edge > 0.f)) {
      // the least magnitude in it: those from it to the top's and to the edge's have room
      const int least_mag = max(max(1, max(tm, em) - kTable + 1),
                                top_ > 0.f ? (tm + em + 3 - kTable) / 2 : (int)(__float_as_uint(-top_) >> 16 & 0x7fffu));
      const int pos = top_ > 0.f ? max(0, tm - least_mag + 1) : 0;
      tab = KeyMap{tm, pos, -1, pos - least_mag, least_mag, edge < 0.f ? pos + max(0, em - least_mag + 1) : 0};
    }
    for (int b = tid_; b < tab.count; b += kThreads) sh_.k.weight[b] = (double)weight(tab.value(b));
    __syncthreads();
    auto weight_at = [&](float x) {  // of x > edge
      const int b = tab.bin(__float_as_uint(x) >> 16);
      return (uint32_t)b < (uint32_t)tab.count ? sh_.k.weight[b] : (double)weight(x);
    };
    double keep = 0.0;
    uint32_t equal = 0;
    auto add = [&](float x) {
      if (x > edge && x >= least_f) keep += weight_at(x);
      equal += x == edge ? 1u : 0u;
    };
    const uint32_t table = (uint32_t)__cvta_generic_to_shared(sh_.k.weight);
    const float low = fmaxf(edge, least_f);
    each_words(
        [&](const uint4& v) {
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          const uint32_t m2 = max_bf16x2(max_bf16x2(w[0], w[1]), max_bf16x2(w[2], w[3]));
          if (!(fmaxf(__uint_as_float(m2 << 16), __uint_as_float(m2 & 0xffff0000u)) >= low)) return;
          bool slow = tab.count == 0;  // not all in the table
          if (tab.least > 0) {
            uint32_t small = 0x7fff7fffu;
#pragma unroll
            for (int e = 0; e < 4; ++e) small = __vminu2(small, w[e] & 0x7fff7fffu);
            slow |= min(small & 0xffffu, small >> 16) < (uint32_t)tab.least;
          }
          if (slow) {
#pragma unroll 1
            for (int e = 0; e < 4; ++e) {
              const uint32_t x = e == 0 ? w[0] : e == 1 ? w[1] : e == 2 ? w[2] : w[3];
              add(__uint_as_float(x << 16));
              add(__uint_as_float(x & 0xffff0000u));
            }
          } else if (tab.least == 0) {  // positive ones only
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = __uint_as_float(w[e] << 16), y = __uint_as_float(w[e] & 0xffff0000u);
              add_above(keep, table + 8u * (uint32_t)(tm - (int)(w[e] & 0xffffu)), x, edge, least_f);
              add_above(keep, table + 8u * (uint32_t)(tm - (int)(w[e] >> 16)), y, edge, least_f);
              equal += x == edge ? 1u : 0u;
              equal += y == edge ? 1u : 0u;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = __uint_as_float(w[e] << 16), y = __uint_as_float(w[e] & 0xffff0000u);
              add_above(keep, table + 8u * (uint32_t)tab.large_bin(w[e] & 0xffffu), x, edge, least_f);
              add_above(keep, table + 8u * (uint32_t)tab.large_bin(w[e] >> 16), y, edge, least_f);
              equal += x == edge ? 1u : 0u;
              equal += y == edge ? 1u : 0u;
            }
          }
        },
        add);
    const u64 s_keep = warp_sum64((u64)keep);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane_ == 0) {
      sh_.ws[0][warp_] = s_keep;
      sh_.cwarp[warp_] = equal;
    }
    __syncthreads();
    // Of 32 parts in order, a lane's own weighing `w` and holding `n` of the edge's entries: the
    // kept weight and the edge's entries before it, and whether the target falls in it.
    auto place = [&](u64 w, uint32_t n, u64* before, uint32_t* same) {
      *same = seen + warp_scan(n, lane_) - n;
      const u64 mine = kept_of(w, n, *same);
      *before = pre + warp_scan(mine, lane_) - mine;
      return o.target >= *before && o.target < *before + mine;
    };
    u64 at;
    uint32_t same;
    const bool is_run = place(lane_ < kWarps ? sh_.ws[0][lane_] : 0ull, lane_ < kWarps ? sh_.cwarp[lane_] : 0u, &at, &same);
    const int w = __ffs(__ballot_sync(0xffffffffu, is_run)) - 1;
    if (w < 0) return true;  // not reached: the runs' sums are the CTA's
    pre = __shfl_sync(0xffffffffu, at, w);
    seen = __shfl_sync(0xffffffffu, same, w);
    // that run again, a part for each warp and of that for each lane
    const int r0 = min(r_.n, w * run_), r1 = min(r_.n, r0 + run_);
    const int per = (run_ + kThreads - 1) / kThreads;
    const int i0 = min(r1, r0 + tid_ * per), i1 = min(r1, i0 + per);
    auto whole_weight = [&](float x) { return x > edge && x >= least_f ? (u64)weight_at(x) : 0ull; };
    u64 s = 0;
    uint32_t n = 0;
    for (int i = i0; i < i1; ++i) {
      const float x = r_.one(i);
      s += whole_weight(x);
      n += x == edge ? 1u : 0u;
    }
    const u64 warp_s = warp_sum64(s);
    const uint32_t warp_n = __reduce_add_sync(0xffffffffu, n);
    if (lane_ == 0) {
      sh_.scan[warp_] = warp_s;
      sh_.cpart[0][warp_] = warp_n;
    }
    __syncthreads();
    place(lane_ < kWarps ? sh_.scan[lane_] : 0ull, lane_ < kWarps ? sh_.cpart[0][lane_] : 0u, &at, &same);
    pre = __shfl_sync(0xffffffffu, at, warp_);
    seen = __shfl_sync(0xffffffffu, same, warp_);
    if (place(s, n, &at, &same)) {
      for (int i = i0; i < i1; ++i) {
        const float x = r_.one(i);
        u64 mine = whole_weight(x);
        if (x == edge) mine = same++ < cut ? o.w : 0ull;
        if (o.target >= at && o.target < at + mine) a_.out[row_id_] = lo_ + i;
        at += mine;
      }
    }
    return true;
  }

  // Rank 0: the summed histogram's verdict, into its sh_.keys. Thread t has group t. The group
  // that holds a border is looked through by eight lanes, a bin each: every other CTA of the
  // cluster waits for this one.
  __device__ void look_keys(const KeyMap& map, uint32_t k, float p, uint32_t least, float u) {
    const int groups = kThreads / size_;  // of a CTA
    const Shared* o = cl_.map_shared_rank(&sh_, tid_ / groups);
    const u64 bins = o->k.mass[tid_ % groups];
    u64 tiny = 0;
    uint32_t n_tiny = 0;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < size_) {
        const Shared* q = cl_.map_shared_rank(&sh_, r);
        tiny += q->tiny;
        n_tiny += q->k.n_tiny;
      }
    // The entries without a bin count to the group of the bin after them (if there is none, to
    // the end): a border among them is not found there.
    const int bt = map.after_tiny(), gt = bt / kKeysPer;
    u64 mass = bins + (tid_ == gt ? tiny : 0ull), end = gt >= kThreads ? tiny : 0ull;
    // of group g, lane e's bin: its entries, and (none where there are none) their weight
    auto count_of = [&](int g) {
      return lane_ < kKeysPer ? cl_.map_shared_rank(&sh_, g / groups)->k.hist[kKeysPer * g + lane_] : 0u;
    };
    // top-k's border: bins before bk are kept whole, `room` entries of it
    int bk = kKeys;  // none: there are fewer entries
    uint32_t room = 0;
    bool found = true;
    if (tid_ == 0) sh_.bins[0] = sh_.bins[1] = kThreads;  // the borders' groups
    if (k > 0) {
      uint32_t own = tid_ == gt ? n_tiny : 0u;
#pragma unroll
      for (int e = 0; e < kKeysPer / 4; ++e) {
        const uint4 v = reinterpret_cast<const uint4*>(o->k.hist)[tid_ * (kKeysPer / 4) + e];
        own += v.x + v.y + v.z + v.w;
      }
      const uint32_t inc = warp_scan(own, lane_);
      if (lane_ == 31) sh_.cwarp[warp_] = inc;
      __syncthreads();
      const uint32_t warps = lane_ < warp_ ? sh_.cwarp[lane_] : 0u;
      const uint32_t before = __reduce_add_sync(0xffffffffu, warps) + inc - own;
      if (k > before && k <= before + own) {
        sh_.bins[0] = (uint32_t)tid_;
        sh_.cut = k - before;
      }
      __syncthreads();
      const int g = (int)sh_.bins[0];
      if (g < kThreads) {
        const int b = kKeysPer * g + lane_;
        const bool past = g == gt && b >= bt;  // lanes after the entries without a bin
        const uint32_t c = count_of(g), upto = warp_scan(c, lane_) + (past ? n_tiny : 0u), left = sh_.cut;  // of the group
        const int e = __ffs(__ballot_sync(0xffffffffu, upto >= left)) - 1;
        const uint32_t first = __shfl_sync(0xffffffffu, upto - c, e);
        const bool over = __shfl_sync(0xffffffffu, past ? 1 : 0, e);
        bk = kKeysPer * g + e;
        // Zeros have a bin ahead of all entries without one, but the positive ones of those come
        // before them in the order: how many zeros are kept is not told from the counts.
        found = left > first && !(bk == map.zero && map.pos > 0 && n_tiny > 0u);
        room = left - first;
        if (warp_ == g / 32) {  // its weight is what is kept of it
          const uint32_t kept = lane_ < e ? c : lane_ == e ? room : 0u;
          const u64 w = warp_sum64(kept ? kept * weight(map.value(b)) : 0ull);
          if (tid_ == g) mass = w + (over ? tiny : 0ull);
        }
        if (tid_ > g) mass = 0;
        end = 0;
      } else if (n_tiny > 0u && gt >= kThreads) {
        found = false;  // maybe among them
      }
    } else {
      __syncthreads();
    }
    const u64 minc = warp_scan(mass, lane_);
    if (lane_ == 31) sh_.scan[warp_] = minc;
    __syncthreads();
    const u64 sums = lane_ < kWarps ? sh_.scan[lane_] : 0ull, upto = warp_scan(sums, lane_);
    const u64 all = __shfl_sync(0xffffffffu, upto, kWarps - 1) + end;
    const u64 before = __shfl_sync(0xffffffffu, upto - sums, warp_) + minc - mass;
    u64 goal = all;  // the border holds the goal-th unit of weight: the last kept
    if (p < 1.0f) {
      const double g = ceil((double)p * (double)all);
      goal = g >= 1.0 ? min((u64)g, all) : 1ull;
    }
    if (goal > before && goal <= before + mass) {
      sh_.bins[1] = (uint32_t)tid_;
      sh_.above = before;
    }
    if (tid_ == 0) sh_.keys.ok = 0;
    __syncthreads();
    const int g = (int)sh_.bins[1];
    if (g == kThreads || !found) return;
    const float least_f = least > 0u ? of_key(least) : -INFINITY;
    const int b = kKeysPer * g + lane_;
    if (warp_ == 0) {
      uint32_t c = count_of(g);
      if (b >= bk) c = b == bk ? room : 0u;
      const u64 w = c ? weight(map.value(b)) : 0ull, extra = g == gt && b >= bt && bk >= bt ? tiny : 0ull;
      const u64 at = sh_.above + extra + warp_scan(c * w, lane_) - c * w;
      if (at < goal && goal <= at + c * w) {
        uint32_t m = (uint32_t)((float)(goal - at) / (float)w);  // off by less than one: at most 2^20
        while (m * w < goal - at) ++m;
        while (m > 1u && (m - 1u) * w >= goal - at) --m;
        const u64 z = at + m * w;  // kept, but for min-p
        // no border among the entries without a bin: top-p's at a zero between them, or min-p's
        const bool amid = b == map.zero || (b >= bt && least_f > -map.tiny_end() && least_f < map.tiny_end());
        sh_.keys = KeyVerdict{target_of(u, z), w, map.value(b), m, (uint32_t)b, n_tiny == 0u || !amid ? 1 : 0};
      }
    }
    if (least == 0u) return;
    __syncthreads();
    if (!sh_.keys.ok || sh_.keys.edge >= least_f) return;
    // min-p ends before the border: the bins down to it, of the groups before the border's whole
    u64 kept = tid_ == 0 && (int)sh_.keys.bin >= bt && least_f <= -map.tiny_end() ? tiny : 0ull;
    if (tid_ <= g && map.value(kKeysPer * tid_) >= least_f) {
      if (tid_ < g && map.value(kKeysPer * tid_ + kKeysPer - 1) >= least_f) {
        kept += bins;
      } else {
#pragma unroll 1
        for (int e = 0; e < kKeysPer; ++e) {
          const float x = map.value(kKeysPer * tid_ + e);
          const uint32_t c = x >= least_f ? o->k.hist[kKeysPer * tid_ + e] : 0u;
          if (c) kept += c * weight(x);
        }
      }
    }
    kept = warp_sum64(kept);
    if (lane_ == 0) sh_.wsum[warp_] = kept;
    __syncthreads();
    if (warp_ == 0) {
      const u64 z = warp_sum64(lane_ < kWarps ? sh_.wsum[lane_] : 0ull);
      if (lane_ == 0) sh_.keys.target = target_of(u, z);
    }
  }

  // The row's token, by way of the list; false where the list does not hold the border (then
  // nothing is written). k = 0: no top-k; `least`: the least key that min-p keeps.
  __device__ bool resolve(int k, float p, uint32_t least, float u) {
    // infinite logits and temperatures beyond fp32's reciprocals have no finite x
    if (top_ == INFINITY || !(inv_f_ > 0.f && inv_f_ < INFINITY)) return false;
    const bool nucleus = p < 1.0f;
    Borders at{kFine - 1, 0u, 0u, 0, -1};
    float per = 0.f;
    if (tid_ < 3 * kWarps) (&sh_.lpart[0][0])[tid_] = (&sh_.cpart[0][0])[tid_] = 0u;
    if (tid_ == 0) sh_.n_list = 0u;
    __syncthreads();
    if (k > 0 || nucleus) {
      const float range = (top_ - low_) * inv_f_;
      float unit = (float)kFineUnit;  // finer bins where the row spans less than them all
      for (int i = 0; i < 12 && range * unit * 2.0f <= (float)(kFine - 2); ++i) unit *= 2.0f;
      per = inv_f_ * unit;
      if (!(per < INFINITY)) return false;
      at = borders(per, 1.0f / unit, (uint32_t)k, nucleus ? p : -1.0f);
    }
    const int bk = at.bk, lo = at.lo, hi = at.hi;
    const bool cut = at.in > 0;  // top-k drops entries that have a weight
    const bool any = nucleus || cut;
    // Exact sums: kept for certain, above top-p's border but under min-p, and below the border
    // (a thread's in fp64: at most 2^8 integers up to 2^43). An entry's bin is the whole part
    // of v, so bins are told apart by v.
    u64 s_keep = 0, s_under = 0, s_rest = 0;
    const float least_f = least > 0u ? of_key(least) : -INFINITY, top = top_, inv_f = inv_f_;
    double d_keep = 0.0, d_sure = 0.0, d_all = 0.0;
    if (any) {
      const float f_sure = (float)(nucleus ? lo : bk), f_lo = (float)lo, f_hi = (float)(hi + 1);
      const float f_bk = (float)bk, f_cut = cut ? (float)(bk + 1) : 0.f;  // f_bk <= v < f_cut: top-k's border bin
      const float f_end = nucleus ? f_bk : f_sure;                       // no weight is asked for from there on
      // what is below all of them concerns nobody: with top-k alone, most of the row
      const float f_last = fmaxf(fmaxf(f_end, f_hi), f_cut);
      each_vector([&](float (&x)[kPer], uint32_t i) {
        float v[kPer], least_v = INFINITY;
        bool in_list = false;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          v[e] = fmaf(top - x[e], per, 0.5f);
          least_v = fminf(least_v, v[e]);
          in_list |= (v[e] >= f_lo && v[e] < f_hi) || (v[e] >= f_bk && v[e] < f_cut);
        }
        if (!(least_v < f_last)) return;
        if (in_list) {
#pragma unroll
          for (int e = 0; e < kPer; ++e)
            if ((v[e] >= f_lo && v[e] < f_hi) || (v[e] >= f_bk && v[e] < f_cut)) {
              const uint32_t to = atomicAdd(&sh_.n_list, 1u);
              if (to < kList) sh_.f.list[to] = place_of(key_of(x[e]), i + e);
              v[e] = INFINITY;  // its weight is added up later
            }
        }
        if (!(least_v < f_end)) return;
        if (nucleus) {
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            const double w = weight_in(x[e], (top - x[e]) * inv_f);
            add_below(d_all, w, v[e], f_end);
            add_below(d_sure, w, v[e], f_sure);
            add_below(d_keep, w, v[e], f_sure, x[e], least_f);
          }
        } else {
#pragma unroll
          for (int e = 0; e < kPer; ++e)
            if (v[e] < f_sure) add_below(d_keep, weight_in(x[e], (top - x[e]) * inv_f), v[e], f_sure, x[e], least_f);
        }
      });
      s_rest = (u64)(d_all - d_sure);
      s_under = (u64)(d_sure - d_keep);
    } else {
      each_vector([&](float (&x)[kPer], uint32_t) {
        float most = -INFINITY;
#pragma unroll
        for (int e = 0; e < kPer; ++e) most = fmaxf(most, x[e]);
        if (!(most >= least_f)) return;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const float xf = (top - x[e]) * inv_f;
          add_below(d_keep, weight_in(x[e], xf), xf, kMaxX, x[e], least_f);
        }
      });
    }
    s_keep = (u64)d_keep;
    if (!nucleus) s_under = 0;
    s_keep = warp_sum64(s_keep);
    s_under = warp_sum64(s_under);
    s_rest = warp_sum64(s_rest);
    if (lane_ == 0) {
      sh_.ws[0][warp_] = s_keep;
      sh_.ws[1][warp_] = s_under;
      sh_.ws[2][warp_] = s_rest;
    }
    __syncthreads();
    if (warp_ < 3) {
      const u64 v = warp_sum64(lane_ < kWarps ? sh_.ws[warp_][lane_] : 0ull);
      if (lane_ == 0) sh_.tot[warp_] = v;
    }
    cl_.sync();
    Verdict o{~0ull, 0, 0, 1, 0};
    if (any) {
      if (rank_ == 0) decide(at, cut, nucleus, k, p, least, u);
      cl_.sync();
      o = cl_.map_shared_rank(&sh_, 0)->verdict;
      if (!o.ok) return false;
    } else {
      u64 tot[kMaxCluster], z = 0;
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        tot[c] = c < size_ ? cl_.map_shared_rank(&sh_, c)->tot[0] : 0ull;
        z += tot[c];
      }
      o.target = target_of(u, z);
      u64 pre = 0;
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        if (o.target >= pre && o.target < pre + tot[c]) {
          o.owner = c;
          o.pre = pre;
        }
        pre += tot[c];
      }
    }
    leave();
    if (o.owner != rank_) return true;
    if (any) {
      // the list's kept weights by run of this CTA
      for (uint32_t j = tid_; j < sh_.n_list; j += kThreads) {
        const u64 place = sh_.f.list[j];
        const uint32_t key = ~(uint32_t)(place >> 32);
        if (place <= o.last && key >= least) add_parts(sh_.lpart, ((int)(uint32_t)place - lo_) / run_, weight(of_key(key)));
      }
      __syncthreads();
    }
    u64 pre = o.pre;
    const u64 target = o.target, last = o.last;
    int w = 0;
    u64 run = sh_.ws[0][0] + parts(sh_.lpart, 0);
    while (w < kWarps - 1 && target >= pre + run) {
      pre += run;
      ++w;
      run = sh_.ws[0][w] + parts(sh_.lpart, w);
    }
    // that warp's run, weighed again by all warps
    const int r0 = min(r_.n, w * run_), r1 = min(r_.n, r0 + run_);
    const int sub = (run_ / 64 + kWarps - 1) / kWarps * 64;
    const int i0 = min(r1, r0 + warp_ * sub), i1 = min(r1, i0 + sub);
    auto kept = [this, last, least](float x, uint32_t i) {
      const uint32_t key = key_of(x);
      return key >= least && place_of(key, i) <= last ? weight(x) : 0ull;
    };
    u64 s = 0;
    for (int i = i0 + 2 * lane_; i < i1; i += 64) {
      float x, y;
      r_.pair(i, x, y);
      s += kept(x, (uint32_t)(lo_ + i));
      if (i + 1 < i1) s += kept(y, (uint32_t)(lo_ + i + 1));
    }
    s = warp_sum64(s);
    if (lane_ == 0) sh_.scan[warp_] = s;
    __syncthreads();
    for (int i = 0; i < warp_; ++i) pre += sh_.scan[i];
    const int i = find(kept, pre, target, i0, i1, s);
    if (i >= 0) a_.out[row_id_] = i;
    return true;
  }

  // Adds the CTAs' histograms, and finds the bin b with (measure of the bins before it)
  // < goal <= (that and its own); bin 0 holds the largest keys. MASS: the goal is
  // p * total, fixed here at the first level. False: the row's measure is below the goal.
  template <bool MASS>
  __device__ bool border(bool first, double p, u64* goal) {
    __syncthreads();
    u64 h = sh_.s.part[0][tid_];
    if (MASS) h += ((u64)sh_.s.part[1][tid_] << kPartBits) + ((u64)sh_.s.part[2][tid_] << (2 * kPartBits));
    sh_.s.hist[tid_] = h;
    cl_.sync();
    h = 0;
    for (int c = 0; c < size_; ++c) h += cl_.map_shared_rank(&sh_, c)->s.hist[tid_];
    u64 inc = h;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane_ >= o) inc += v;
    }
    if (lane_ == 31) sh_.wsum[warp_] = inc;
    __syncthreads();
    u64 pre = 0, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp_) pre += sh_.wsum[w];
      all += sh_.wsum[w];
    }
    if (MASS && first) {
      const double g = ceil(p * (double)all);
      *goal = g >= 1.0 ? min((u64)g, all) : 1ull;
    }
    inc += pre;
    if (inc - h < *goal && *goal <= inc) {
      sh_.bin = (uint32_t)tid_;
      sh_.above = inc - h;
      sh_.inside = h;
    }
    cl_.sync();  // the border is known, and no CTA reads another's histogram any more
    return all >= *goal;
  }

  __device__ __forceinline__ void clear() {
    sh_.s.part[0][tid_] = 0u;
    sh_.s.part[1][tid_] = 0u;
    sh_.s.part[2][tid_] = 0u;
    __syncthreads();
  }

  template <bool MASS>
  __device__ __forceinline__ void count(uint32_t bin, float x) {
    if (MASS) {
      const u64 w = weight_any(x);
      if (w == 0ull) return;
      constexpr uint32_t m = (1u << kPartBits) - 1u;
      const uint32_t a = (uint32_t)w & m, b = (uint32_t)(w >> kPartBits) & m, c = (uint32_t)(w >> (2 * kPartBits));
      if (a) atomicAdd(&sh_.s.part[0][bin], a);
      if (b) atomicAdd(&sh_.s.part[1][bin], b);
      if (c) atomicAdd(&sh_.s.part[2][bin], c);
    } else {
      atomicAdd(&sh_.s.part[0][bin], 1u);
    }
  }

  // Narrows `keep` to the first entries, in order, that top-k (goal of them) or top-p
  // (MASS: until p of the kept weight lies before) leaves. `range`: the distance from the
  // largest logit that the first histogram spreads over its bins.
  template <bool MASS>
  __device__ Keep select(Keep keep, float range, u64 goal, double p) {
    const float per = range > 0.f ? (float)(kBins - 1) / range : 0.f, top = top_;
    auto bin_of = [per, top](float x) {  // does not fall as x falls
      if (x == top) return 0;
      const float v = (top - x) * per;
      return v < (float)(kBins - 1) ? (int)v : kBins - 1;
    };
    clear();
    each([&](float x, uint32_t i) {
      if (keep.has(order_key(x), i)) count<MASS>((uint32_t)bin_of(x), x);
    });
    if (!border<MASS>(true, p, &goal)) return keep;
    // the border bin's keys: listed aside where they fit, and their range
    const int b0 = (int)sh_.bin;
    u64 above = sh_.above;
    if (tid_ == 0) {
      sh_.n_list = 0u;
      sh_.kmin = 0xffffffffu;
      sh_.kmax = 0u;
    }
    __syncthreads();
    each([&](float x, uint32_t i) {
      const uint32_t k = order_key(x);
      if (bin_of(x) == b0 && keep.has(k, i)) {
        const uint32_t at = atomicAdd(&sh_.n_list, 1u);
        if (at < kList) sh_.s.list[at] = k;
        atomicMin(&sh_.kmin, k);
        atomicMax(&sh_.kmax, k);
      }
    });
    cl_.sync();
    uint32_t k0 = 0xffffffffu, k1 = 0u;
    for (int c = 0; c < size_; ++c) {
      const Shared* o = cl_.map_shared_rank(&sh_, c);
      k0 = min(k0, o->kmin);
      k1 = max(k1, o->kmax);
    }
    const uint32_t n_list = sh_.n_list;
    // the remaining goal inside [k0, k1], until a bin is one key
    while (true) {
      goal -= above;
      int shift = 0;
      while (((k1 - k0) >> shift) >= (uint32_t)kBins) ++shift;
      clear();
      if (n_list <= kList) {
        for (uint32_t j = tid_; j < n_list; j += kThreads) {
          const uint32_t k = sh_.s.list[j];
          if (k >= k0 && k <= k1) count<MASS>((k1 - k) >> shift, of_key(k));
        }
      } else {
        each([&](float x, uint32_t i) {
          const uint32_t k = order_key(x);
          if (k >= k0 && k <= k1 && keep.has(k, i)) count<MASS>((k1 - k) >> shift, x);
        });
      }
      border<MASS>(false, p, &goal);
      above = sh_.above;
      const uint32_t b = sh_.bin;
      k1 -= b << shift;
      if (shift == 0) break;
      const uint32_t width = (1u << shift) - 1u;
      k0 = k1 - k0 > width ? k1 - width : k0;
    }
    // of the entries with key k1: the first m, in index order
    const u64 each_w = MASS ? weight_any(of_key(k1)) : 1ull;
    const u64 m = (goal - above + each_w - 1) / each_w, c = sh_.inside / each_w;
    Keep out{k1, k1 == keep.key ? keep.index : 0xffffffffu};
    if (m < c) {
      auto same = [keep, k1](float x, uint32_t i) {
        const uint32_t k = order_key(x);
        return k == k1 && keep.has(k, i) ? 1ull : 0ull;
      };
      u64 before;
      sums(same, &before);
      const int i = find(same, before, m - 1, w0_, w1_, sh_.wsum[warp_]);
      if (i >= 0)
        for (int o = 0; o < size_; ++o) cl_.map_shared_rank(&sh_, o)->cut = (uint32_t)i;
      cl_.sync();
      out.index = sh_.cut;
    }
    return out;
  }
};

template <bool F32>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Shared& sh = *reinterpret_cast<Shared*>(smem + kDataBytes);
  {
    Sampler<F32> s(a, sh, smem);
    s.run();
    s.end();
  }
}

struct WalkArgs {
  const int32_t* token;  // [N] the target's token at every node
  const int32_t* draft;
  const int32_t* parent;
  const int32_t* cu_tree;
  int32_t* accept_len;
  int32_t* accept_path;
  int32_t* next_token;
  int32_t B, T, N;
};

__global__ void __launch_bounds__(kMaxTree) sampled_walk_kernel(const __grid_constant__ WalkArgs a) {
  const int b = blockIdx.x, tid = threadIdx.x;
  Plan p{};
  p.B = a.B;
  p.T = a.T;
  p.N = a.N;
  int base = 0, n = 0;
  bool ok = tree_range(p, a.cu_tree, b, &base, &n);
  __shared__ int32_t token[kMaxTree], parent[kMaxTree], draft[kMaxTree], first_match[kMaxTree], path[kMaxTree], len_s;
  if (tid < n) {  // inputs that the sampling kernel does not write
    parent[tid] = a.parent[base + tid];
    draft[tid] = a.draft[base + tid];
  }
  first_match[tid] = INT32_MAX;
  const bool bad_link = tid < n && (tid == 0 ? parent[tid] != -1 : (parent[tid] < 0 || parent[tid] >= tid));
  ok = ok && n > 0 && !__syncthreads_or(bad_link);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (ok && tid < n) token[tid] = a.token[base + tid];
  __syncthreads();
  if (ok) {  // the same for the whole CTA
    const int len = walk_tree(token, parent, draft, first_match, n, path);
    if (tid == 0) len_s = len;
  } else if (tid == 0) {
    len_s = -1;
  }
  __syncthreads();
  const int len = len_s;
  if (tid < a.T) a.accept_path[(int64_t)b * a.T + tid] = tid <= len ? path[tid] : -1;
  if (tid == 0) {
    a.accept_len[b] = len;
    a.next_token[b] = ok ? token[path[len]] : -1;
  }
}

bool al4(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 3u) == 0; }

int check_sample(const void* logits, int64_t row_stride, const float* uniform, const ls_sample_opts* o, const void* out,
                 int64_t rows, int32_t vocab, int32_t dtype) {
  if (rows < 0 || vocab < 1) return LS_ERR_INVALID_ARG;
  if (dtype != LS_DTYPE_BF16 && dtype != LS_DTYPE_F32) return LS_ERR_INVALID_ARG;
  if (vocab > kMaxVocab || rows > (1 << 27)) return LS_ERR_UNSUPPORTED;
  if (row_stride < vocab && rows > 1) return LS_ERR_INVALID_ARG;
  if (rows == 0) return LS_OK;
  if (logits == nullptr || uniform == nullptr || out == nullptr) return LS_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(logits) & (dtype == LS_DTYPE_F32 ? 3u : 1u)) != 0 || !al4(uniform) || !al4(out))
    return LS_ERR_INVALID_ARG;
  if (o != nullptr && (!al4(o->temperature) || !al4(o->top_k) || !al4(o->top_p) || !al4(o->min_p)))
    return LS_ERR_INVALID_ARG;
  return LS_OK;
}

template <bool F32>
int launch_sample(const SampleArgs& a, int64_t rows, int cluster, cudaStream_t st) {
  constexpr int smem = kDataBytes + (int)sizeof(Shared);
  static_assert(2 * (smem + 1024) <= 233472, "two CTAs an SM");
  static bool configured[kMaxConfigured] = {};  // per template instance
  if (configure_once(sample_kernel<F32>, smem, configured) != cudaSuccess) return LS_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<F32>, a) == cudaSuccess ? LS_OK : LS_ERR_CUDA;
}

// The sampling launch; arguments checked.
int run_sample(const void* logits, int64_t row_stride, const float* uniform, const ls_sample_opts* o, int32_t* out,
               int64_t rows, int32_t vocab, int32_t dtype, cudaStream_t st) {
  const bool f32 = dtype == LS_DTYPE_F32;
  const int elt = f32 ? 4 : 2, cap = kDataBytes / elt;
  SampleArgs a{};
  a.logits = logits;
  a.row_stride = row_stride;
  a.uniform = uniform;
  if (o != nullptr) {
    a.temperature = o->temperature;
    a.top_k = o->top_k;
    a.top_p = o->top_p;
    a.min_p = o->min_p;
  }
  a.out = out;
  a.V = vocab;
  a.cap = cap;
  a.vec = (reinterpret_cast<uintptr_t>(logits) & 15u) == 0 && (row_stride * elt) % 16 == 0 ? 1 : 0;
  int sms = 0, major = 0;
  const int rd = device_info(&sms, &major);
  if (rd != LS_OK) return rd;
  if (major != 10) return LS_ERR_UNSUPPORTED;
  const int cluster = sample_cluster(rows, vocab, cap, sms);
  a.seg = sample_share(vocab, cluster);
  (void)cudaGetLastError();
  return f32 ? launch_sample<true>(a, rows, cluster, st) : launch_sample<false>(a, rows, cluster, st);
}

}  // namespace

}  // namespace ls

extern "C" {

int ls_sample(const void* logits, int64_t row_stride, const float* uniform, const ls_sample_opts* opts, int32_t* out,
              int64_t rows, int32_t vocab, int32_t logits_dtype, void* stream) {
  const int rc = ls::check_sample(logits, row_stride, uniform, opts, out, rows, vocab, logits_dtype);
  if (rc != LS_OK || rows == 0) return rc;
  return ls::run_sample(logits, row_stride, uniform, opts, out, rows, vocab, logits_dtype,
                        static_cast<cudaStream_t>(stream));
}

int ls_tree_accept_sample(const void* logits, const float* uniform, const ls_sample_opts* opts,
                          const int32_t* tree_tokens, const int32_t* tree_parent, const int32_t* cu_tree,
                          int32_t total_nodes, int32_t* node_token, int32_t* accept_len, int32_t* accept_path,
                          int32_t* next_token, const ls_accept_dims* dims, void* stream) {
  if (dims == nullptr || dims->batch < 1 || dims->tree_size < 1 || dims->vocab < 1) return LS_ERR_INVALID_ARG;
  if (dims->tree_size > ls::kMaxTree) return LS_ERR_UNSUPPORTED;
  const int64_t most = (int64_t)dims->batch * dims->tree_size;
  if (most > (1 << 27)) return LS_ERR_UNSUPPORTED;
  const int64_t n = cu_tree != nullptr ? (int64_t)total_nodes : most;
  if (n < 0 || n > most) return LS_ERR_INVALID_ARG;
  const int rc = ls::check_sample(logits, dims->vocab, uniform, opts, node_token, n, dims->vocab, dims->logits_dtype);
  if (rc != LS_OK) return rc;
  if (accept_len == nullptr || accept_path == nullptr || next_token == nullptr) return LS_ERR_INVALID_ARG;
  if (n > 0 && (tree_tokens == nullptr || tree_parent == nullptr)) return LS_ERR_INVALID_ARG;
  if (!ls::al4(tree_tokens) || !ls::al4(tree_parent) || !ls::al4(cu_tree) || !ls::al4(accept_len) ||
      !ls::al4(accept_path) || !ls::al4(next_token))
    return LS_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n > 0) {
    const int e = ls::run_sample(logits, dims->vocab, uniform, opts, node_token, n, dims->vocab, dims->logits_dtype, st);
    if (e != LS_OK) return e;
  }
  ls::WalkArgs w;
  w.token = node_token;
  w.draft = tree_tokens;
  w.parent = tree_parent;
  w.cu_tree = cu_tree;
  w.accept_len = accept_len;
  w.accept_path = accept_path;
  w.next_token = next_token;
  w.B = dims->batch;
  w.T = dims->tree_size;
  w.N = (int32_t)n;
  // a programmatic dependent of the sampling kernel: it reads its own inputs before waiting
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(dims->batch);
  cfg.blockDim = dim3(ls::kMaxTree);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = n > 0 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, ls::sampled_walk_kernel, w) != cudaSuccess) return LS_ERR_CUDA;
  return LS_OK;
}

}  // extern "C"
