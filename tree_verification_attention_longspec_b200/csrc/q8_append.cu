// New keys and values into the 8-bit paged cache.
//
// Per scale block (scale_block tokens of one kv head, keys and values apart) that a
// sequence's new rows x touch:
//   amax = max |x| over them (NaN skipped), e = the least integer in [-60, 64] with
//   amax <= 448 * 2^e, unit = 2^e;
//   a block that already holds tokens keeps its scale s where s >= unit; where s < unit its
//   earlier codes c become the codes nearest to c * (s / unit) and its scale becomes unit;
//   code = nearest e4m3 of x / scale (ties to even, saturated).
// Units are powers of two, so x / unit and c * (s / unit) are exact before their one
// rounding, and a scale that grows costs the earlier codes nothing but bits that fall
// below e4m3's smallest: a block's content depends on what is in it, hardly on the calls
// that brought it. (A tighter scale, amax / 448, gains under one bit of range and none of
// precision, the codes being floating point.)
//
// One warp per block, head and tensor: lanes hold 8 values each, rows in a first pass give
// amax and stay in registers (up to 16 loads, the rest are read again), a second rounds.
#include "q8_device.cuh"

namespace ls {
namespace {

constexpr int kWarps = 8;
constexpr int kKeep = 16;  // 16-byte loads a lane keeps between the passes

template <int D>
__global__ void __launch_bounds__(kWarps * 32) q8_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kLanes = D / 8;         // lanes of a row
  constexpr int kRows = 32 / kLanes;    // rows a step
  const int lane = threadIdx.x & 31;
  const KvQ8& kv = a.kv;
  auto count = [&](int b, int len) -> int {  // rows that sequence b appends
    int n;
    if (a.cu_new != nullptr) {
      n = a.cu_new[b + 1] - a.cu_new[b];
    } else {
      n = a.accept_len[b] + 1;
    }
    const int64_t room = (int64_t)kv.max_pages * kv.page_size - len;
    n = min(n, a.max_new);
    return n <= 0 || len < 0 ? 0 : (int)min((int64_t)n, max(room, (int64_t)0));
  };
  if (blockIdx.x == gridDim.x - 1) {  // the lengths after the call
    if (a.cu_out == nullptr) return;
    __shared__ int32_t part[kWarps * 32];
    const int per = (a.B + kWarps * 32 - 1) / (kWarps * 32);
    const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
    int sum = 0;
    for (int b = b0; b < b1; ++b) {
      const int len = a.cu[b + 1] - a.cu[b];
      sum += len + count(b, len);
    }
    part[threadIdx.x] = sum;
    __syncthreads();
    int at = 0;
    for (int t = 0; t < (int)threadIdx.x; ++t) at += part[t];
    if (threadIdx.x == 0) a.cu_out[0] = 0;
    for (int b = b0; b < b1; ++b) {
      const int len = a.cu[b + 1] - a.cu[b];
      at += len + count(b, len);
      a.cu_out[b + 1] = at;
    }
    return;
  }
  int64_t id = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int h = (int)(id % a.Hkv);
  id /= a.Hkv;
  const bool val = id & 1;  // values, or keys
  id >>= 1;
  const int bl = (int)(id % a.blocks);
  const int64_t b64 = id / a.blocks;
  if (b64 >= a.B) return;
  const int b = (int)b64;
  const int len = a.cu[b + 1] - a.cu[b];
  const int n = count(b, len);
  const int block = len / kv.scale_block + bl;  // of the sequence
  const int first = block * kv.scale_block;     // its first token
  const int p0 = max(len, first), p1 = min(len + n, first + kv.scale_block);
  if (p0 >= p1) return;
  const int page_no = first / kv.page_size;  // below max_pages: p0 is in the cache
  const int32_t page = kv.page_table[(size_t)b * kv.max_pages + page_no];
  if ((uint32_t)page >= (uint32_t)kv.num_pages) return;  // not a page of this cache: dropped
  const int64_t row0 = (int64_t)page * kv.page_size + (first - page_no * kv.page_size);  // row of token `first`
  const int64_t stride = (int64_t)a.Hkv * D;
  uint8_t* codes = (val ? kv.v_pages : kv.k_pages) + row0 * stride + h * D;
  float* scale_at = (val ? kv.v_scale : kv.k_scale) + row0 / kv.scale_block * a.Hkv + h;
  const uint16_t* src = (val ? a.v_new : a.k_new) + h * D;
  // source row of the token at position p, -1 where the path names none
  int tree_base = 0, tree_n = 0;
  if (a.cu_new == nullptr) {
    Plan pl{};
    pl.B = a.B;
    pl.T = a.T;
    pl.N = a.rows;
    tree_range(pl, a.cu_tree, b, &tree_base, &tree_n);
  }
  auto source = [&](int p) -> int {
    const int i = p - len;
    if (a.cu_new != nullptr) {
      const int r = a.cu_new[b] + i;
      return (uint32_t)r < (uint32_t)a.rows ? r : -1;
    }
    const int node = a.accept_path[(size_t)b * a.T + i];
    return (uint32_t)node < (uint32_t)tree_n ? tree_base + node : -1;
  };
  const int col = (lane % kLanes) * 8, sub = lane / kLanes;
  const int steps = (p1 - p0 + kRows - 1) / kRows;
  const bool held = p0 > first;
  const float old = held ? *scale_at : 0.f;

  uint4 keep[kKeep];
  float amax = 0.f;
  auto fetch = [&](int s, uint4& v) -> bool {
    const int p = p0 + s * kRows + sub;
    const int r = p < p1 ? source(p) : -1;
    v = make_uint4(0u, 0u, 0u, 0u);
    if (r >= 0) v = *reinterpret_cast<const uint4*>(src + (int64_t)r * stride + col);
    return r >= 0;
  };
  uint32_t there = 0u;  // bit s: row of step s exists
  for (int s0 = 0; s0 < steps; s0 += kKeep) {
#pragma unroll
    for (int s = 0; s < kKeep; ++s) {
      const bool ok = s0 + s < steps && fetch(s0 + s, keep[s]);
      if (!ok) keep[s] = make_uint4(0u, 0u, 0u, 0u);
      if (s0 == 0 && ok) there |= 1u << s;
    }
#pragma unroll
    for (int s = 0; s < kKeep; ++s) {
      const uint32_t w[4] = {keep[s].x, keep[s].y, keep[s].z, keep[s].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u))));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  // 448 = 1.75 * 2^8: amax = m * 2^k with 1 <= m < 2 needs e = k - 8, one more where m > 1.75
  int e = kMinScaleExp;
  if (amax > 0.f) {
    const uint32_t bits = __float_as_uint(amax);
    e = exponent_of(amax) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = min(max(e, kMinScaleExp), kMaxScaleExp);
  }
  const float need = pow2f(e);
  const float now = held ? fmaxf(old, need) : need;
  if (held && old < now) {  // the earlier tokens' codes in the new unit
    const float ratio = old > 0.f ? old / now : 0.f;
    for (int p = first + sub; p < p0; p += kRows) {
      uint2* at = reinterpret_cast<uint2*>(codes + (int64_t)(p - first) * stride + col);
      uint2 c = *at;
      uint32_t* cw = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t lo = e4m3x2_f16x2(cw[k]), hi = e4m3x2_f16x2_hi(cw[k]);
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        cw[k] = (uint32_t)f32x2_e4m3x2(x.x * ratio, x.y * ratio) |
                ((uint32_t)f32x2_e4m3x2(y.x * ratio, y.y * ratio) << 16);
      }
      *at = c;
    }
  }
  if (lane == 0 && !(held && old == now)) *scale_at = now;
  auto store = [&](int s, const uint4& v) {
    const int p = p0 + s * kRows + sub;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)  // a division: exact where the scale is a power of two
      c[k] = f32x2_e4m3x2(__fdiv_rn(__uint_as_float(w[k] << 16), now),
                          __fdiv_rn(__uint_as_float(w[k] & 0xffff0000u), now));
    *reinterpret_cast<uint2*>(codes + (int64_t)(p - first) * stride + col) =
        make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  };
  if (steps <= kKeep) {
#pragma unroll
    for (int s = 0; s < kKeep; ++s)
      if (there >> s & 1u) store(s, keep[s]);
  } else {
    for (int s = 0; s < steps; ++s) {
      uint4 v;
      if (fetch(s, v)) store(s, v);
    }
  }
}

template <int D>
cudaError_t launch_d(const AppendArgs& a, cudaStream_t stream) {
  const int64_t warps = (int64_t)a.B * a.blocks * 2 * a.Hkv;
  const int64_t ctas = (warps + kWarps - 1) / kWarps + 1;  // the last one: the lengths
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  q8_append_kernel<D><<<(unsigned)ctas, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_q8_append(const AppendArgs& a, cudaStream_t stream) {
  return a.d == 64 ? launch_d<64>(a, stream) : launch_d<128>(a, stream);
}

}  // namespace ls
