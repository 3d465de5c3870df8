// Attention partials over the 8-bit cache for units of few query rows.
//
// The same partials as partials_tc.cu (prefix keys with no mask, then the tree block under
// the ancestor mask, one online softmax), with cached keys kc * ks and values vc * vs, the
// scales ks, vs shared by a block of tokens and kv head:
//   x_j = scale * log2(e) * ks_j <q, kc_j>          score in the log2 domain
//   p_j = 2^(x_j + log2 vs_j - m + kOff)            weight times its value's scale
//   O += p_j vc_j,   l += p_j / vs_j
// m is the running maximum of x_j + log2 vs_j (raised only when exceeded by kRaise), so p_j
// lies in f16's range, p and the codes are f16 operands (the codes exactly) and the scales
// cost one FMA a score. out = O / l, lse = m - kOff + log2 l.
//
// Decoding and small trees read each cached byte for few rows: HBM bounds them. So no
// shared memory on the way: every warp streams its own keys from global memory into
// registers, 16 at a step, two steps ahead (8 KB a warp in flight at d = 128), converts
// them there and feeds mma.sync with the cache as the A operand: S^T = K Q^T with 16 keys
// by 8 rows, O^T += V^T P^T with 16 dimensions by 8 rows, so that 8 rows cost half of what
// a 16-row A operand would. The order of d inside a K step and of V's rows is free, and is
// chosen so that a lane's operands are contiguous bytes: 32 of each of its two keys, 16 of
// each of its four values (byte pairs of two keys by PRMT). P^T comes out of S^T's
// accumulators by movmatrix. (mma.sync: with 8 to 16 rows tcgen05's 128-row tile would be
// nine tenths padding, and its operands would have to be converted through shared memory.)
//
// A chunk's 128-key blocks go round the CTA's 8 warps in steps of 16 keys; the warps'
// (m, l, O) are merged in shared memory at the end and leave as the chunk's partial.
#include "q8_device.cuh"
#include "sm100.cuh"

namespace ls {
namespace {
using sm100::ex2_approx;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 16;                // keys a warp takes at a time
constexpr int kStride = kWarps * kStep;  // keys between a warp's steps
constexpr float kRaise = 6.0f;           // log2 units that a score may exceed the running maximum by
constexpr float kOff = 9.0f;             // so weights stay below 2^15
static_assert(kStride == kBlockN, "a block is one step of every warp");

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint4 load16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load8(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// 16 cached keys and values as one lane holds them: with n = lane / 4, c = lane % 4, key
// words of keys n and n + 8 (d = 16 c + 64 h .. + 15), value words of keys 2c, 2c + 1,
// 2c + 8, 2c + 9 (d = n * D / 8 .. + D / 8 - 1).
template <int D>
struct Frag {
  uint32_t k[2][D / 16];
  uint32_t v[4][D / 32];
  float ks, vs;
};

template <int D>
constexpr int smem_bytes(int rows) {
  return kWarps * rows * (D + 4) * 4;  // the warps' O (rows padded by 16 bytes)
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1) q8_rows_kernel(const __grid_constant__ Q8Args a) {
  constexpr int R = 8 * NT;          // rows of a unit
  constexpr int kKS = D / 16;        // K steps of a score
  constexpr int kMT = D / 16;        // 16-row tiles of O^T
  constexpr int kVB = D / 8;         // value bytes of a lane
  constexpr int kPad = D + 4;
  extern __shared__ __align__(16) float so[];  // [warp][R][kPad]
  __shared__ float sm[kWarps][R], sl[kWarps][R];
  __shared__ uint32_t vis[R][4];  // tree nodes visible to the row
  __shared__ int cut[R];          // window: first attended key the row sees
  __shared__ int16_t par[kMaxTree];
  __shared__ uint32_t bad_s;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Plan& p = a.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = lane >> 2, c4 = lane & 3;
  const int32_t* cu = plan_cu(p, a.cu);
  const ChunkCoord c = locate_chunk(p, cu, blockIdx.x);
  if (!c.valid) return;  // more CTAs than the device lengths need: the combine reports it
  int tree_base, tree_n;
  tree_range(p, a.cu_tree, c.b, &tree_base, &tree_n);
  const int row0 = c.rgi * R;                     // first row of the unit: node row0 / g, head row0 % g
  const int rows = min(R, tree_n * p.g - row0);   // rows that exist
  if (rows <= 0) {
    if (tid == 0) a.chunk_status[blockIdx.x] = 0u;
    return;
  }
  const int seq_len = cu[c.b + 1] - cu[c.b];
  const KvQ8& kv = a.kv;
  const int64_t stride = (int64_t)p.Hkv * D;  // bytes of a cache row, elements of a tree row

  // ---- the cache, two steps ahead
  const uint8_t* kbase = kv.k_pages + c.kh * D + 16 * c4;
  const uint8_t* vbase = kv.v_pages + c.kh * D + kVB * n;
  // cache row of the step's first key (a step never crosses a page: both are multiples of 16)
  auto find = [&](int key) -> int32_t { return key < c.key_end ? q8_row(kv, c.b, c.key_skip + key) : 0; };
  auto load = [&](Frag<D>& f, int key, int32_t row) {
    if (key >= c.key_end) return;
    const uint8_t* k0 = kbase + (int64_t)(row + n) * stride;
#pragma unroll
    for (int hf = 0; hf < D / 64; ++hf) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 x = load16(k0 + 8 * j * stride + 64 * hf);
        f.k[j][4 * hf] = x.x;
        f.k[j][4 * hf + 1] = x.y;
        f.k[j][4 * hf + 2] = x.z;
        f.k[j][4 * hf + 3] = x.w;
      }
    }
    const uint8_t* v0 = vbase + (int64_t)(row + 2 * c4) * stride;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint8_t* vp = v0 + ((j & 1) + 8 * (j >> 1)) * stride;
      if constexpr (D == 128) {
        const uint4 x = load16(vp);
        f.v[j][0] = x.x;
        f.v[j][1] = x.y;
        f.v[j][2] = x.z;
        f.v[j][3] = x.w;
      } else {
        const uint2 x = load8(vp);
        f.v[j][0] = x.x;
        f.v[j][1] = x.y;
      }
    }
    const size_t s = (size_t)(row / kv.scale_block) * p.Hkv + c.kh;
    f.ks = __ldg(kv.k_scale + s);
    f.vs = __ldg(kv.v_scale + s);
  };
  int key = c.key_begin + warp * kStep;
  Frag<D> f0, f1;
  int32_t r0 = find(key), r1 = find(key + kStride);
  load(f0, key, r0);
  load(f1, key + kStride, r1);
  r0 = find(key + 2 * kStride);

  // ---- per-row masks
  const bool win = p.window > 0 && c.key_begin < 2 * kBlockN && c.key_end > c.key_begin;
  if (tid == 0) bad_s = 0u;
  if (c.has_tree || win)
    for (int x = tid; x < tree_n; x += kThreads) {
      const int32_t pp = a.parent[(size_t)tree_base + x];
      par[x] = (int16_t)(pp >= -1 && pp < tree_n ? pp : kMaxTree);
    }
  __syncthreads();
  if (tid < R) {
    uint32_t m[4] = {0u, 0u, 0u, 0u};
    int depth = 0;
    if ((c.has_tree || win) && tid < rows) {
      int x = (row0 + tid) / p.g;
      for (int step = 0; step <= kMaxTree; ++step) {
        m[x >> 5] |= 1u << (x & 31);
        const int pp = par[x];
        if (x == 0) {
          if (pp != -1) bad_s = 1u;
          break;
        }
        if (pp < 0 || pp >= x) {  // not a rooted tree with parents before their children
          bad_s = 1u;
          break;
        }
        x = pp;
        ++depth;
      }
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) vis[tid][w] = m[w];
    cut[tid] = win ? window_cut(p, seq_len, depth) : 0;
  }
  // ---- Q^T as B operands: row n of each row tile, f16, scaled by a power of two a row
  if (a.after_prep) asm volatile("griddepcontrol.wait;" ::: "memory");
  uint32_t q[NT][kKS][2];
  float cs[NT][2];  // score factor of rows 2c, 2c + 1: softmax scale * log2(e) / the row's power of two
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = 8 * t + n;
    uint2 w[kKS];
    float amax = 0.f;
    if (r < rows) {
      const int node = (row0 + r) / p.g, j = (row0 + r) % p.g;
      const uint16_t* qp = a.q + ((size_t)(tree_base + node) * p.Hq + c.kh * p.g + j) * D + 16 * c4;
#pragma unroll
      for (int s = 0; s < kKS; ++s) {
        w[s] = *reinterpret_cast<const uint2*>(qp + 64 * (s / 4) + 4 * (s % 4));
        amax = fmaxf(amax, fmaxf(fmaxf(fabsf(__uint_as_float(w[s].x << 16)), fabsf(__uint_as_float(w[s].x & 0xffff0000u))),
                                 fmaxf(fabsf(__uint_as_float(w[s].y << 16)), fabsf(__uint_as_float(w[s].y & 0xffff0000u)))));
      }
    } else {
#pragma unroll
      for (int s = 0; s < kKS; ++s) w[s] = make_uint2(0u, 0u);
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int sh = f16_shift(amax);
    const float mul = pow2f(sh), inv = pow2f(-sh);
#pragma unroll
    for (int s = 0; s < kKS; ++s) {
      q[t][s][0] = pack_f16x2(__uint_as_float(w[s].x << 16) * mul, __uint_as_float(w[s].x & 0xffff0000u) * mul);
      q[t][s][1] = pack_f16x2(__uint_as_float(w[s].y << 16) * mul, __uint_as_float(w[s].y & 0xffff0000u) * mul);
    }
    cs[t][0] = p.scale_log2 * __shfl_sync(0xffffffffu, inv, 8 * c4);
    cs[t][1] = p.scale_log2 * __shfl_sync(0xffffffffu, inv, 8 * c4 + 4);
  }
  __syncthreads();  // vis, cut
  int cuts[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    cuts[t][0] = cut[8 * t + 2 * c4];
    cuts[t][1] = cut[8 * t + 2 * c4 + 1];
  }

  float o[NT][kMT][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int i = 0; i < kMT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][i][e] = 0.f;
    m[t][0] = m[t][1] = -INFINITY;
    l[t][0] = l[t][1] = 0.f;
  }

  // x: scores (log2 units, value scale folded in, -inf where masked) of keys n (e = 0, 1)
  // and n + 8 (e = 2, 3) for rows 2c, 2c + 1. Raises the maxima, adds to the sums (rv = 1 /
  // value scale) and returns P^T as B operands.
  auto weigh = [&](float (&x)[NT][4], float rv, uint32_t (&b)[NT][2]) {
    bool up = false;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) up |= fmaxf(x[t][e], x[t][e + 2]) > m[t][e] + kRaise;
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(x[t][e], x[t][e + 2]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float now = fmaxf(m[t][e], mx);
          f[e] = m[t][e] == now ? 1.f : ex2_approx(m[t][e] - now);  // 0 from m = -inf
          m[t][e] = now;
          l[t][e] *= f[e];
        }
#pragma unroll
        for (int i = 0; i < kMT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][i][e] *= f[e & 1];
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      // a row that has seen no key yet keeps m = -inf, and its weights are 0
      const float ma = (m[t][0] == -INFINITY ? 0.f : m[t][0]) - kOff, mb = (m[t][1] == -INFINITY ? 0.f : m[t][1]) - kOff;
      const float p0 = ex2_approx(x[t][0] - ma), p1 = ex2_approx(x[t][1] - mb);
      const float p2 = ex2_approx(x[t][2] - ma), p3 = ex2_approx(x[t][3] - mb);
      l[t][0] = fmaf(p0 + p2, rv, l[t][0]);
      l[t][1] = fmaf(p1 + p3, rv, l[t][1]);
      b[t][0] = transpose8x8(pack_f16x2(p0, p1));
      b[t][1] = transpose8x8(pack_f16x2(p2, p3));
    }
  };

  // ---- prefix steps
  auto compute = [&](Frag<D>& f, int k0) {
    float s[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
#pragma unroll
    for (int i = 0; i < kKS; ++i) {
      const uint32_t a0 = e4m3x2_f16x2(f.k[0][i]), a1 = e4m3x2_f16x2(f.k[1][i]);
      const uint32_t a2 = e4m3x2_f16x2_hi(f.k[0][i]), a3 = e4m3x2_f16x2_hi(f.k[1][i]);
#pragma unroll
      for (int t = 0; t < NT; ++t) mma16816(s[t], a0, a1, a2, a3, q[t][i][0], q[t][i][1]);
    }
    // scales: a key's below f32's normals counts as 2^-126 (its scores are 0 either way), a
    // value's as the nearer end of [2^-60, 2^64]
    const float ks = fmaxf(f.ks, 1.17549435e-38f);
    const float vs = fminf(fmaxf(f.vs, 8.6736174e-19f), 1.8446744e19f);
    const float lv = log2f(vs), rv = 1.f / vs;
    const bool edge = k0 + kStep > c.key_end;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = fmaf(s[t][e], ks * cs[t][e & 1], lv);
    if (edge || win) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int kk = k0 + n + 8 * (e >> 1);
          if (kk >= c.key_end || kk < cuts[t][e & 1]) s[t][e] = -INFINITY;
        }
      if (edge) {  // rows past the sequence hold anything: no NaN into the product
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (k0 + 2 * c4 + (j & 1) + 8 * (j >> 1) >= c.key_end)
#pragma unroll
            for (int w = 0; w < D / 32; ++w) f.v[j][w] = 0u;
      }
    }
    uint32_t b[NT][2];
    weigh(s, rv, b);
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {  // four value bytes: tiles 2w (bytes 0, 1) and 2w + 1 (2, 3)
      const uint32_t xa = __byte_perm(f.v[0][w], f.v[1][w], 0x5140), xb = __byte_perm(f.v[2][w], f.v[3][w], 0x5140);
      const uint32_t ya = __byte_perm(f.v[0][w], f.v[1][w], 0x7362), yb = __byte_perm(f.v[2][w], f.v[3][w], 0x7362);
      const uint32_t x0 = e4m3x2_f16x2(xa), x1 = e4m3x2_f16x2_hi(xa), x2 = e4m3x2_f16x2(xb), x3 = e4m3x2_f16x2_hi(xb);
      const uint32_t y0 = e4m3x2_f16x2(ya), y1 = e4m3x2_f16x2_hi(ya), y2 = e4m3x2_f16x2(yb), y3 = e4m3x2_f16x2_hi(yb);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        mma16816(o[t][2 * w], x0, x1, x2, x3, b[t][0], b[t][1]);
        mma16816(o[t][2 * w + 1], y0, y1, y2, y3, b[t][0], b[t][1]);
      }
    }
  };
  while (key < c.key_end) {
    compute(f0, key);
    r1 = find(key + 3 * kStride);
    load(f0, key + 2 * kStride, r0);
    if (key + kStride < c.key_end) compute(f1, key + kStride);
    r0 = find(key + 4 * kStride);
    load(f1, key + 3 * kStride, r1);
    key += 2 * kStride;
  }

  // ---- the tree block: bf16 keys and values, 16 a step, scaled into f16 by powers of two
  // (a key's own, and one for the step's values, which then act as a value scale)
  if (c.has_tree) {
    for (int x0 = warp * kStep; x0 < tree_n; x0 += kStride) {
      float s[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
      uint32_t kh[2][kKS][2];
      float kinv[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int x = x0 + n + 8 * j;
        uint2 w[kKS];
        float amax = 0.f;
        const uint16_t* kp = a.k_tree + (int64_t)(tree_base + x) * stride + c.kh * D + 16 * c4;
#pragma unroll
        for (int i = 0; i < kKS; ++i) {
          w[i] = x < tree_n ? *reinterpret_cast<const uint2*>(kp + 64 * (i / 4) + 4 * (i % 4)) : make_uint2(0u, 0u);
          amax = fmaxf(amax, fmaxf(fmaxf(fabsf(__uint_as_float(w[i].x << 16)), fabsf(__uint_as_float(w[i].x & 0xffff0000u))),
                                   fmaxf(fabsf(__uint_as_float(w[i].y << 16)), fabsf(__uint_as_float(w[i].y & 0xffff0000u)))));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int sh = f16_shift(amax);
        const float mul = pow2f(sh);
        kinv[j] = pow2f(-sh);
#pragma unroll
        for (int i = 0; i < kKS; ++i) {
          kh[j][i][0] = pack_f16x2(__uint_as_float(w[i].x << 16) * mul, __uint_as_float(w[i].x & 0xffff0000u) * mul);
          kh[j][i][1] = pack_f16x2(__uint_as_float(w[i].y << 16) * mul, __uint_as_float(w[i].y & 0xffff0000u) * mul);
        }
      }
#pragma unroll
      for (int i = 0; i < kKS; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) mma16816(s[t], kh[0][i][0], kh[1][i][0], kh[0][i][1], kh[1][i][1], q[t][i][0], q[t][i][1]);
      // values: D / 8 of each of four nodes
      uint32_t vw[4][kVB / 2];
      float vmax = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int x = x0 + 2 * c4 + (j & 1) + 8 * (j >> 1);
        const uint16_t* vp = a.v_tree + (int64_t)(tree_base + x) * stride + c.kh * D + kVB * n;
#pragma unroll
        for (int i = 0; i < kVB / 8; ++i) {
          const uint4 w = x < tree_n ? *reinterpret_cast<const uint4*>(vp + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
          vw[j][4 * i] = w.x;
          vw[j][4 * i + 1] = w.y;
          vw[j][4 * i + 2] = w.z;
          vw[j][4 * i + 3] = w.w;
        }
#pragma unroll
        for (int i = 0; i < kVB / 2; ++i)
          vmax = fmaxf(vmax, fmaxf(fabsf(__uint_as_float(vw[j][i] << 16)), fabsf(__uint_as_float(vw[j][i] & 0xffff0000u))));
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, off));
      // all-zero values (or ones too small to matter in the sums) leave the weights as they are
      const int vsh = min(max(f16_shift(vmax), -kMaxScaleExp), -kMinScaleExp);
      const float vmul = pow2f(vsh), lv = (float)-vsh;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int x = x0 + n + 8 * (e >> 1);
          const uint32_t* mask = vis[8 * t + 2 * c4 + (e & 1)];
          const bool see = x < tree_n && ((mask[x >> 5] >> (x & 31)) & 1u);
          s[t][e] = see ? fmaf(s[t][e] * kinv[e >> 1], cs[t][e & 1], lv) : -INFINITY;
        }
      uint32_t b[NT][2];
      weigh(s, vmul, b);
#pragma unroll
      for (int i = 0; i < kMT; ++i) {  // values 2i (low half of word i) and 2i + 1
        const uint32_t a0 = pack_f16x2(__uint_as_float(vw[0][i] << 16) * vmul, __uint_as_float(vw[1][i] << 16) * vmul);
        const uint32_t a1 = pack_f16x2(__uint_as_float(vw[0][i] & 0xffff0000u) * vmul, __uint_as_float(vw[1][i] & 0xffff0000u) * vmul);
        const uint32_t a2 = pack_f16x2(__uint_as_float(vw[2][i] << 16) * vmul, __uint_as_float(vw[3][i] << 16) * vmul);
        const uint32_t a3 = pack_f16x2(__uint_as_float(vw[2][i] & 0xffff0000u) * vmul, __uint_as_float(vw[3][i] & 0xffff0000u) * vmul);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma16816(o[t][i], a0, a1, a2, a3, b[t][0], b[t][1]);
      }
    }
  }

  // ---- the warps' results joined: rows' maxima and sums, then O^T weighted
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float s = l[t][e];
      s += __shfl_xor_sync(0xffffffffu, s, 4);
      s += __shfl_xor_sync(0xffffffffu, s, 8);
      s += __shfl_xor_sync(0xffffffffu, s, 16);
      if (n == 0) {
        sm[warp][8 * t + 2 * c4 + e] = m[t][e];
        sl[warp][8 * t + 2 * c4 + e] = s;
      }
    }
#pragma unroll
    for (int i = 0; i < kMT; ++i) {
      float* at = so + (size_t)(warp * R + 8 * t + 2 * c4) * kPad + kVB * n + 2 * i;
      *reinterpret_cast<float2*>(at) = make_float2(o[t][i][0], o[t][i][2]);
      *reinterpret_cast<float2*>(at + kPad) = make_float2(o[t][i][1], o[t][i][3]);
    }
  }
  __syncthreads();
  const size_t slot = (size_t)blockIdx.x * p.slot_rows;
  for (int idx = tid; idx < rows * (D / 4); idx += kThreads) {
    const int r = idx / (D / 4), d = idx % (D / 4) * 4;
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w][r]);
    const float ref = M == -INFINITY ? 0.f : M;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2_approx(sm[w][r] - ref);  // 0 for a warp that saw no key
      L = fmaf(sl[w][r], f, L);
      const float4 v = *reinterpret_cast<const float4*>(so + (size_t)(w * R + r) * kPad + d);
      acc.x = fmaf(v.x, f, acc.x);
      acc.y = fmaf(v.y, f, acc.y);
      acc.z = fmaf(v.z, f, acc.z);
      acc.w = fmaf(v.w, f, acc.w);
    }
    const float inv = M == -INFINITY ? 0.f : 1.f / L;
    *reinterpret_cast<float4*>(a.o_part + (slot + r) * D + d) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (d == 0) a.lse_part[slot + r] = M == -INFINITY ? -INFINITY : M - kOff + log2f(L);
  }
  if (tid == 0) a.chunk_status[blockIdx.x] = bad_s ? kErrBadTree : 0u;
}

template <int D, int NT>
cudaError_t launch(const Q8Args& a, cudaStream_t stream) {
  const int smem = smem_bytes<D>(8 * NT);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(q8_rows_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.p.n_chunks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.after_prep ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, q8_rows_kernel<D, NT>, a);
}

}  // namespace

cudaError_t launch_q8_rows(const Q8Args& a, cudaStream_t stream) {
  if (a.p.n_chunks == 0) return cudaSuccess;
  if (a.p.d == 64) return a.p.slot_rows == 8 ? launch<64, 1>(a, stream) : launch<64, 2>(a, stream);
  return a.p.slot_rows == 8 ? launch<128, 1>(a, stream) : launch<128, 2>(a, stream);
}

}  // namespace ls
