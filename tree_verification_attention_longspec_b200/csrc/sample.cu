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
// function of the inputs alone. w itself is computed in fp64 (relative error below 2^-46):
// an fp32 exponential's 1e-7 would move the borders of a flat 128k-entry distribution by
// more than the gap that one row in a thousand leaves to its uniform number.
//
// One cluster of 1 to 8 CTAs per row; each keeps its share of the row in shared memory
// (what does not fit is read again), so that HBM is read once, and the passes over it
// meet through distributed shared memory. A threshold is found by a histogram of 1024
// bins, linear in the distance to the largest logit, then by further ones over the keys
// of the one bin that holds the border, whose members are listed aside.
#include <cooperative_groups.h>

#include <algorithm>

#include "ls_device.cuh"
#include "ls_verify_attn.h"
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

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = kThreads;  // one per thread
constexpr int kList = 4096;      // keys of a border bin kept aside
constexpr int kMaxCluster = 8;
constexpr int kMaxVocab = 1 << 20;  // sums of 2^43 stay below 2^63
constexpr int kWeightBits = 43;
// a weight's three parts: a CTA's share is at most 2^17 entries, so their sums fit 32 bits
constexpr int kPartBits = 15;
constexpr int kMaxSeg = 1 << 17;
constexpr int kDataBytes = 160 * 1024;

using u64 = unsigned long long;

// Order-preserving key of a float: larger value, larger key (-0 and +0 get one key).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

struct Shared {
  u64 hist[kBins];          // this CTA's measure of each bin
  uint32_t part[3][kBins];  // its parts while they are added up
  uint32_t list[kList];
  uint32_t n_list;
  uint32_t kmin, kmax;  // keys of the border bin
  u64 wsum[kWarps + 1];
  u64 total;  // this CTA's sum
  u64 above;  // measure before the border bin, and in it
  u64 inside;
  uint32_t bin;
  float fmax[kWarps], fmin[kWarps];
  float top, low;
  uint32_t cut;  // index threshold found by the CTA that owns it
};

// 2^43 * exp(x) rounded, x <= 0. exp by 2^n * 2^f, f in [-1/2, 1/2], and the Taylor
// polynomial of 2^f = exp(f ln 2) to degree 11 (remainder (ln2/2)^12/12! = 6e-15).
__device__ __forceinline__ u64 weight_of(double x) {
  if (!(x > -30.6)) return 0ull;  // below half a unit
  const double magic = 6755399441055744.0;  // 1.5 * 2^52
  const double y = x * 1.4426950408889634074;
  const double t = y + magic;
  const int n = __double2loint(t);
  const double f = y - (t - magic);
  double p = 4.4455382718708100e-10;  // (ln 2)^k / k!, k = 11 .. 0
  p = fma(p, f, 7.0549116208011210e-09);
  p = fma(p, f, 1.0178086009239696e-07);
  p = fma(p, f, 1.3215486790144305e-06);
  p = fma(p, f, 1.5252733804059838e-05);
  p = fma(p, f, 1.5403530393381606e-04);
  p = fma(p, f, 1.3333558146428441e-03);
  p = fma(p, f, 9.6181291076284770e-03);
  p = fma(p, f, 5.5504108664821576e-02);
  p = fma(p, f, 2.4022650695910070e-01);
  p = fma(p, f, 6.9314718055994530e-01);
  p = fma(p, f, 1.0);
  return __double2ull_rn(p * __hiloint2double((1023 + kWeightBits + n) << 20, 0));
}

template <bool F32>
struct Row {
  const void* g;      // this CTA's share in global memory
  const void* s;      // its first `cap` entries in shared memory
  int n, cap;
  // entries i and i + 1 (i even); -inf past the share and for NaN
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
  __device__ __forceinline__ float load(int i) const {
    float x;
    if constexpr (F32)
      x = static_cast<const float*>(g)[i];
    else
      x = bf16_to_f32(static_cast<const uint16_t*>(g)[i]);
    return x == x ? x : -INFINITY;
  }
};

// What is kept so far: keys above `key`, and those equal to it up to entry `index`.
struct Keep {
  uint32_t key, index;
  __device__ __forceinline__ bool has(uint32_t k, uint32_t i) const { return k > key || (k == key && i <= index); }
};

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
    // each warp's run of entries, in index order; two entries a lane and step
    const int per = (r_.n + kWarps - 1) / kWarps;
    run_ = (per + 63) / 64 * 64;
    w0_ = min(r_.n, warp_ * run_);
    w1_ = min(r_.n, w0_ + run_);
  }

  __device__ void run() {
    load();
    const float t = a_.temperature != nullptr ? a_.temperature[row_id_] : 1.0f;
    if (top_ == -INFINITY) {  // nothing above -inf
      if (rank_ == 0 && tid_ == 0) a_.out[row_id_] = 0;
      return;
    }
    if (!(t > 0.f)) {  // greedy: the first entry of the largest value
      const float top = top_;
      auto first = [top](float x, uint32_t) { return x == top ? 1ull : 0ull; };
      u64 before;
      sums(first, &before);
      const int i = find(first, before, 0ull);
      if (i >= 0) a_.out[row_id_] = i;
      return;
    }
    inv_t_ = 1.0 / (double)t;
    Keep keep{0u, 0xffffffffu};
    const int k = a_.top_k != nullptr ? a_.top_k[row_id_] : 0;
    if (k > 0 && k < a_.V) keep = select<false>(keep, top_ - low_, (u64)k, 0.0);
    const float p = a_.top_p != nullptr ? a_.top_p[row_id_] : 1.0f;
    if (p < 1.0f) keep = select<true>(keep, fminf(31.0f * t, top_ - low_), 0ull, (double)p);
    const float mp = a_.min_p != nullptr ? a_.min_p[row_id_] : 0.0f;
    const double x_min = mp > 0.f ? (mp < 1.f ? log((double)mp) : 0.0) : -1e300;
    auto kept = [this, keep, x_min](float x, uint32_t i) {
      if (!keep.has(key_of(x), i)) return 0ull;
      const double e = exponent(x);
      return e >= x_min ? weight_of(e) : 0ull;
    };
    u64 before;
    const u64 z = sums(kept, &before);
    const float u = a_.uniform[row_id_];
    const double at = u > 0.f ? (double)u * (double)z : 0.0;
    const u64 target = at < (double)z ? min((u64)at, z - 1) : z - 1;
    const int i = find(kept, before, target);
    if (i >= 0) a_.out[row_id_] = i;
  }

 private:
  const SampleArgs& a_;
  Shared& sh_;
  cg::cluster_group cl_;
  int tid_, lane_, warp_, rank_, size_, lo_, run_, w0_, w1_;
  int64_t row_id_;
  Row<F32> r_;
  float top_, low_;  // largest value; smallest above -inf
  double inv_t_;

  // (l - top) / t; 0 for the largest (also +inf), -inf for -inf
  __device__ __forceinline__ double exponent(float x) const {
    if (x == top_) return 0.0;
    if (x == -INFINITY || top_ == INFINITY) return -INFINITY;
    return ((double)x - (double)top_) * inv_t_;
  }

  // f(value, entry of the row) over this warp's run, two entries a lane and step
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    for (int i = w0_ + 2 * lane_; i < w1_; i += 64) {
      float x, y;
      r_.pair(i, x, y);
      f(x, (uint32_t)(lo_ + i));
      if (i + 1 < w1_) f(y, (uint32_t)(lo_ + i + 1));
    }
  }

  // The share into shared memory, and the row's largest and smallest finite-or-+inf value.
  __device__ void load() {
    float mx = -INFINITY, mn = INFINITY;
    auto take = [&](float x) {
      mx = fmaxf(mx, x);
      if (x > -INFINITY) mn = fminf(mn, x);
    };
    constexpr int kPer = F32 ? 4 : 8;
    const int n_vec = a_.vec ? r_.cap / kPer : 0;
    constexpr int kFly = 4;
    for (int v0 = tid_; v0 < n_vec; v0 += kFly * kThreads) {
      uint4 w[kFly];
#pragma unroll
      for (int u = 0; u < kFly; ++u)
        if (v0 + u * kThreads < n_vec) w[u] = __ldcs(static_cast<const uint4*>(r_.g) + v0 + u * kThreads);
#pragma unroll
      for (int u = 0; u < kFly; ++u) {
        if (v0 + u * kThreads < n_vec) {
          uint32_t q[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (F32) {
              float x = __uint_as_float(q[e]);
              if (!(x == x)) {
                x = -INFINITY;
                q[e] = 0xff800000u;
              }
              take(x);
            } else {
              float x = __uint_as_float(q[e] << 16), y = __uint_as_float(q[e] & 0xffff0000u);
              if (!(x == x)) {
                x = -INFINITY;
                q[e] = (q[e] & 0xffff0000u) | 0xff80u;
              }
              if (!(y == y)) {
                y = -INFINITY;
                q[e] = (q[e] & 0xffffu) | 0xff800000u;
              }
              take(x);
              take(y);
            }
          }
          reinterpret_cast<uint4*>(const_cast<void*>(r_.s))[v0 + u * kThreads] = make_uint4(q[0], q[1], q[2], q[3]);
        }
      }
    }
    for (int i = n_vec * kPer + tid_; i < r_.n; i += kThreads) {
      const float x = r_.load(i);
      take(x);
      if (i < r_.cap) {
        if constexpr (F32)
          static_cast<float*>(const_cast<void*>(r_.s))[i] = x;
        else
          static_cast<uint16_t*>(const_cast<void*>(r_.s))[i] = (uint16_t)(__float_as_uint(x) >> 16);
      }
    }
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
    if (tid_ == 0) {
      for (int w = 1; w < kWarps; ++w) {
        mx = fmaxf(mx, sh_.fmax[w]);
        mn = fminf(mn, sh_.fmin[w]);
      }
      sh_.top = mx;
      sh_.low = mn;
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
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
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

  // The entry at which the running sum of f first exceeds `target`: returned by one lane of
  // the warp whose run holds it (after `sums` of the same f), -1 by every other thread.
  template <class F>
  __device__ int find(F f, u64 before, u64 target) {
    if (target < before || target >= before + sh_.wsum[warp_]) return -1;
    for (int i0 = w0_; i0 < w1_; i0 += 64) {
      const int i = i0 + 2 * lane_;
      u64 wa = 0, wb = 0;
      if (i < w1_) {
        float x, y;
        r_.pair(i, x, y);
        wa = f(x, (uint32_t)(lo_ + i));
        if (i + 1 < w1_) wb = f(y, (uint32_t)(lo_ + i + 1));
      }
      u64 inc = wa + wb;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane_ >= o) inc += v;
      }
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

  // Adds the CTAs' histograms, and finds the bin b with (measure of the bins before it)
  // < goal <= (that and its own); bin 0 holds the largest keys. MASS: the goal is
  // p * total, fixed here at the first level. False: the row's measure is below the goal.
  template <bool MASS>
  __device__ bool border(bool first, double p, u64* goal) {
    __syncthreads();
    u64 h = sh_.part[0][tid_];
    if (MASS) h += ((u64)sh_.part[1][tid_] << kPartBits) + ((u64)sh_.part[2][tid_] << (2 * kPartBits));
    sh_.hist[tid_] = h;
    cl_.sync();
    h = 0;
    for (int c = 0; c < size_; ++c) h += cl_.map_shared_rank(&sh_, c)->hist[tid_];
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
    sh_.part[0][tid_] = 0u;
    sh_.part[1][tid_] = 0u;
    sh_.part[2][tid_] = 0u;
    __syncthreads();
  }

  template <bool MASS>
  __device__ __forceinline__ void count(uint32_t bin, float x) {
    if (MASS) {
      const u64 w = weight_of(exponent(x));
      if (w == 0ull) return;
      constexpr uint32_t m = (1u << kPartBits) - 1u;
      const uint32_t a = (uint32_t)w & m, b = (uint32_t)(w >> kPartBits) & m, c = (uint32_t)(w >> (2 * kPartBits));
      if (a) atomicAdd(&sh_.part[0][bin], a);
      if (b) atomicAdd(&sh_.part[1][bin], b);
      if (c) atomicAdd(&sh_.part[2][bin], c);
    } else {
      atomicAdd(&sh_.part[0][bin], 1u);
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
      if (keep.has(key_of(x), i)) count<MASS>((uint32_t)bin_of(x), x);
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
      const uint32_t k = key_of(x);
      if (bin_of(x) == b0 && keep.has(k, i)) {
        const uint32_t at = atomicAdd(&sh_.n_list, 1u);
        if (at < kList) sh_.list[at] = k;
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
          const uint32_t k = sh_.list[j];
          if (k >= k0 && k <= k1) count<MASS>((k1 - k) >> shift, of_key(k));
        }
      } else {
        each([&](float x, uint32_t i) {
          const uint32_t k = key_of(x);
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
    const u64 each_w = MASS ? weight_of(exponent(of_key(k1))) : 1ull;
    const u64 m = (goal - above + each_w - 1) / each_w, c = sh_.inside / each_w;
    Keep out{k1, k1 == keep.key ? keep.index : 0xffffffffu};
    if (m < c) {
      auto same = [keep, k1](float x, uint32_t i) {
        const uint32_t k = key_of(x);
        return k == k1 && keep.has(k, i) ? 1ull : 0ull;
      };
      u64 before;
      sums(same, &before);
      const int i = find(same, before, m - 1);
      if (i >= 0)
        for (int o = 0; o < size_; ++o) cl_.map_shared_rank(&sh_, o)->cut = (uint32_t)i;
      cl_.sync();
      out.index = sh_.cut;
    }
    return out;
  }
};

template <bool F32>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const __grid_constant__ SampleArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Shared& sh = *reinterpret_cast<Shared*>(smem + kDataBytes);
  {
    Sampler<F32> s(a, sh, smem);
    s.run();
  }
  cg::this_cluster().sync();  // a CTA's shared memory lives until its peers have read it
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
  static_assert(smem <= 232448, "shared memory");
  if (cudaFuncSetAttribute(sample_kernel<F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return LS_ERR_CUDA;
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
  // the fewest CTAs whose shared memory holds the row; more while the rows leave SMs idle
  int cluster = 1;
  while (cluster < kMaxCluster && (vocab + cluster - 1) / cluster > std::min(cap, kMaxSeg) - 8) cluster *= 2;
  while (cluster < kMaxCluster && rows * cluster * 2 <= 148 && vocab / cluster >= 8192) cluster *= 2;
  a.seg = ((vocab + cluster - 1) / cluster + 7) / 8 * 8;
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
