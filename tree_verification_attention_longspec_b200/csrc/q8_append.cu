// New keys and values into the 8-bit paged cache.
//
// Per scale block (scale_block tokens of one kv head, keys and values apart) that a
// sequence's new rows x touch:
//   amax = max |x| over them (NaN skipped), e = the least integer in [-60, 64] with
//   amax <= 448 * 2^e, unit = 2^e;
//   a block that already holds tokens keeps its scale s where s >= unit; where s < unit its
//   earlier codes c become the codes nearest to c * (s / unit) and its scale becomes unit;
//   code = nearest e4m3 of x / scale (ties to even, saturated).
// Units are powers of two, so x / unit and, between units, c * (s / unit) are exact before their
// one rounding, and a scale that grows costs the earlier codes nothing but bits that fall
// below e4m3's smallest: a block's content depends on what is in it, hardly on the calls
// that brought it. (Where another writer's s is none, quotient and product are rounded to odd
// first, so that the code is still the nearest to the exact value.) (A tighter scale, amax / 448, gains under one bit of range and none of
// precision, the codes being floating point.)
//
// A team of 1, 2, 4 or 8 warps per block, head and tensor, so that a lane holds at most 8
// loads of 8 values: all are in flight at once, give amax, and are rounded from registers.
// Bytes bound it: each row is read once and its codes written once. Measured (B200): 16,384
// new rows of 8 heads, 101 MB: 23 us, 4.4 TB/s (16 loads a lane and half the warps an SM:
// 26.2; one warp per block that reads the rows past 16 loads twice: 27.1); a few accepted
// rows each of 8 sequences: 10 us, the launch.
#include <algorithm>

#include "q8_device.cuh"

namespace ls {
namespace {

constexpr int kWarps = 8;
constexpr int kKeep = 8;  // 16-byte loads of a lane

// Rows that sequence b, of `len` tokens, appends.
__device__ __forceinline__ int appended(const AppendArgs& a, int b, int len) {
  int n = a.cu_new != nullptr ? a.cu_new[b + 1] - a.cu_new[b] : a.accept_len[b] + 1;
  n = min(n, a.max_new);
  const int64_t room = (int64_t)a.kv.max_pages * a.kv.page_size - len;
  return n <= 0 || len < 0 ? 0 : (int)min((int64_t)n, max(room, (int64_t)0));
}

// The lengths after the call, by one CTA.
__device__ void new_lengths(const AppendArgs& a) {
  __shared__ int32_t part[kWarps * 32];
  const int per = (a.B + kWarps * 32 - 1) / (kWarps * 32);
  const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
  int sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int len = a.cu[b + 1] - a.cu[b];
    sum += len + appended(a, b, len);
  }
  part[threadIdx.x] = sum;
  __syncthreads();
  int at = 0;
  for (int t = 0; t < min((int)threadIdx.x, a.B); ++t) at += part[t];
  if (threadIdx.x == 0) a.cu_out[0] = 0;
  for (int b = b0; b < b1; ++b) {
    const int len = a.cu[b + 1] - a.cu[b];
    at += len + appended(a, b, len);
    a.cu_out[b + 1] = at;
  }
}

// Eight bf16 values times a power of two as codes (the products are exact).
__device__ __forceinline__ uint2 encode(const uint4& v, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    c[k] = f32x2_e4m3x2(__uint_as_float(w[k] << 16) * s, __uint_as_float(w[k] & 0xffff0000u) * s);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Quotients and products that fp32 does not hold are rounded to odd (towards zero, then the
// last bit set): 24 bits of which the last says that there is more are rounded to a code's 4
// as the exact value would be, where fp32's nearest could land on the middle of two codes.
__device__ __forceinline__ float to_odd(float towards_zero, float rest) {
  return rest > 0.f || rest < 0.f ? __uint_as_float(__float_as_uint(towards_zero) | 1u) : towards_zero;  // (NaN, infinity: as they are)
}
__device__ __forceinline__ float quotient(float x, float s) {
  const float q = __fdiv_rz(x, s);
  return to_odd(q, fmaf(-q, s, x));
}
__device__ __forceinline__ float product(float x, float s) {
  const float q = __fmul_rz(x, s);
  return to_odd(q, fmaf(x, s, -q));
}

// Eight bf16 values over s as codes.
__device__ __forceinline__ uint2 encode_over(const uint4& v, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    c[k] = f32x2_e4m3x2(quotient(__uint_as_float(w[k] << 16), s), quotient(__uint_as_float(w[k] & 0xffff0000u), s));
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32, 4) q8_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kLanes = D / 8;       // lanes of a row
  constexpr int kRows = 32 / kLanes;  // rows a step
  if (blockIdx.x == gridDim.x - 1) {
    if (a.cu_out != nullptr) new_lengths(a);
    return;
  }
  const int lane = threadIdx.x & 31;
  const KvQ8& kv = a.kv;
  const int warp = threadIdx.x >> 5, team = 1 << a.team_shift, mate = warp & (team - 1);  // of the block's warps
  const uint32_t unit = (blockIdx.x * kWarps + warp) >> a.team_shift;                     // (block, tensor, head)
  __shared__ uint32_t mates[kWarps];
  const int h = (int)(unit % (uint32_t)a.Hkv);
  const bool val = (unit / (uint32_t)a.Hkv) & 1;  // values, or keys
  int id = (int)(unit / (uint32_t)a.Hkv >> 1);
  // the touched blocks of all sequences in order: which one is number id?
  int b = -1, len = 0, n = 0, block = 0;
  for (int base = 0; base < a.B; base += 32) {
    const int bb = base + lane;
    const int l = bb < a.B ? a.cu[bb + 1] - a.cu[bb] : 0;
    const int c = bb < a.B ? appended(a, bb, l) : 0;
    const int touched = c > 0 ? ((l + c - 1) >> kv.scale_shift) - (l >> kv.scale_shift) + 1 : 0;
    int upto = touched;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const uint32_t here = __ballot_sync(0xffffffffu, id < upto);
    if (here) {
      const int at = __ffs(here) - 1;
      b = base + at;
      len = __shfl_sync(0xffffffffu, l, at);
      n = __shfl_sync(0xffffffffu, c, at);
      block = (len >> kv.scale_shift) + id - __shfl_sync(0xffffffffu, upto - touched, at);
      break;
    }
    id -= __shfl_sync(0xffffffffu, upto, 31);
  }
  if (b < 0) return;
  const int first = block * kv.scale_block;  // its first token
  const int p0 = max(len, first), p1 = min(len + n, first + kv.scale_block);
  const int64_t stride = (int64_t)a.Hkv * D;
  const int col = (lane % kLanes) * 8, sub = lane / kLanes;
  const int i0 = mate * kKeep * kRows + sub;  // this lane's rows, from p0: i0, i0 + kRows, ...

  // The source row of token p0 + i: the next one, or where the path names it.
  const int32_t* path = a.cu_new != nullptr ? nullptr : a.accept_path + (size_t)b * a.T + (p0 - len);
  int row_base, row_end;  // rows of the sequence
  if (path == nullptr) {
    row_base = a.cu_new[b] + (p0 - len);
    row_end = a.rows;
  } else {
    Plan pl{};
    pl.B = a.B;
    pl.T = a.T;
    pl.N = a.rows;
    tree_range(pl, a.cu_tree, b, &row_base, &row_end);
    row_end += row_base;
  }
  const uint16_t* src = (val ? a.v_new : a.k_new) + h * D + col;
  auto source = [&](int i) -> int {  // -1: none
    if (p0 + i >= p1) return -1;
    const int r = path != nullptr ? path[i] : i;
    return r >= 0 && row_base >= 0 && r < row_end - row_base ? row_base + r : -1;
  };
  auto fetch = [&](int r) {
    return r >= 0 ? *reinterpret_cast<const uint4*>(src + (int64_t)r * stride) : make_uint4(0u, 0u, 0u, 0u);
  };
  uint4 keep[kKeep];
  uint32_t there = 0u;  // bit s: row of step s exists
#pragma unroll
  for (int s = 0; s < kKeep; ++s) {
    const int r = source(i0 + s * kRows);
    keep[s] = fetch(r);
    there |= r >= 0 ? 1u << s : 0u;
  }
  // the block's place in the cache, while the rows are on their way
  const int page_no = first / kv.page_size;  // below max_pages: p0 is in the cache
  const int32_t page = kv.page_table[(size_t)b * kv.max_pages + page_no];
  if ((uint32_t)page >= (uint32_t)kv.num_pages) return;  // not a page of this cache: dropped
  const int64_t row0 = (int64_t)page * kv.page_size + (first - page_no * kv.page_size);  // row of token `first`
  uint8_t* codes = (val ? kv.v_pages : kv.k_pages) + row0 * stride + h * D + col;
  float* scale_at = (val ? kv.v_scale : kv.k_scale) + (row0 >> kv.scale_shift) * a.Hkv + h;
  const bool held = p0 > first;
  const float old = held ? *scale_at : 0.f;

  // the largest magnitude: bf16 pairs compared as such (NaN skipped)
  uint32_t most = 0u;
  auto take = [&](const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) asm("max.bf16x2 %0, %0, %1;" : "+r"(most) : "r"(w[e] & 0x7fff7fffu));
  };
#pragma unroll
  for (int s = 0; s < kKeep; ++s) take(keep[s]);
  float amax = fmaxf(__uint_as_float(most << 16), __uint_as_float(most & 0xffff0000u));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (team > 1) {  // (all of them are here: what returned above depends on the block alone)
    if (lane == 0) mates[warp] = __float_as_uint(amax);
    asm volatile("bar.sync %0, %1;" ::"r"(1 + (warp >> a.team_shift)), "r"(32 * team) : "memory");
    for (int w = 0; w < team; ++w) amax = fmaxf(amax, __uint_as_float(mates[warp - mate + w]));
  }
  // 448 = 1.75 * 2^8: amax = m * 2^k with 1 <= m < 2 needs e = k - 8, one more where m > 1.75
  int e = kMinScaleExp;
  if (amax > 0.f) {
    e = exponent_of(amax) - 8 + ((__float_as_uint(amax) & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = min(max(e, kMinScaleExp), kMaxScaleExp);
  }
  const float need = pow2f(e);
  const float now = held ? fmaxf(old, need) : need;
  if (held && old < now) {  // the earlier tokens' codes in the new unit
    const float ratio = old > 0.f ? old / now : 0.f;
#pragma unroll 1
    for (int p = first + mate * kRows + sub; p < p0; p += team * kRows) {
      uint2* at = reinterpret_cast<uint2*>(codes + (int64_t)(p - first) * stride);
      uint2 c = *at;
      uint32_t* cw = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t lo = e4m3x2_f16x2(cw[k]), hi = e4m3x2_f16x2_hi(cw[k]);
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        cw[k] = (uint32_t)f32x2_e4m3x2(product(x.x, ratio), product(x.y, ratio)) |
                ((uint32_t)f32x2_e4m3x2(product(y.x, ratio), product(y.y, ratio)) << 16);
      }
      *at = c;
    }
  }
  if (mate == 0 && lane == 0 && !(held && old == now)) *scale_at = now;
  codes += (int64_t)(p0 - first + i0) * stride;
  auto store = [&](int s, const uint2& c) { *reinterpret_cast<uint2*>(codes + (int64_t)s * kRows * stride) = c; };
  // a power of two (every scale of this kernel's) divides by a multiplication, exactly
  if ((__float_as_uint(now) & 0x7fffffu) == 0u && now >= 1.17549435e-38f) {
    const float inv = 1.f / now;
#pragma unroll
    for (int s = 0; s < kKeep; ++s)
      if (there >> s & 1u) store(s, encode(keep[s], inv));
  } else {
    // another writer's scale, kept: divisions, in a loop of their own (unrolled with the rest
    // they were most of the kernel's code, and its time)
#pragma unroll 1
    for (int s = 0; s < kKeep; ++s) {
      const int r = source(i0 + s * kRows);
      if (r >= 0) store(s, encode_over(fetch(r), now));
    }
  }
}

template <int D>
cudaError_t launch_d(AppendArgs a, cudaStream_t stream) {
  // warps of a block: its rows (or as many as a sequence appends) over what one holds
  constexpr int kHold = kKeep * (32 / (D / 8));
  a.team_shift = 0;
  while ((kHold << a.team_shift) < std::min(a.kv.scale_block, a.max_new)) ++a.team_shift;
  static_assert(kWarps * kHold >= 128, "a team is in one CTA");
  const int64_t warps = (a.blocks * 2 * a.Hkv) << a.team_shift;
  const int64_t ctas = (warps + kWarps - 1) / kWarps + 1;  // the last one: the lengths
  if (warps > INT32_MAX) return cudaErrorInvalidValue;
  q8_append_kernel<D><<<(unsigned)ctas, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_q8_append(const AppendArgs& a, cudaStream_t stream) {
  return a.d == 64 ? launch_d<64>(a, stream) : launch_d<128>(a, stream);
}

}  // namespace ls
