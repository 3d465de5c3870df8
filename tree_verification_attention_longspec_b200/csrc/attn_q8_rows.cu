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
// cost one FMA a score. out = O / l, lse = m - kOff + log2 l. As f16, p_j is off by 2^-11 of
// itself or by 2^-25, whichever is more: w_j vs_j by max(2^-11 w_j vs_j, 2^-34 M) with M the
// row's largest, so blocks of values far below another's (2^23 at equal weights) lose bits in
// dimensions where the other holds zeros.
//
// Decoding and small trees read each cached byte for few rows: HBM bounds them, and what
// keeps HBM busy is bytes in flight. Every warp streams its own keys, 16 at a step, through
// its own ring in shared memory (cp.async, no barrier but the warp's own; 128 KB to 150 KB an
// SM under way), converts them in registers and feeds mma.sync with the cache as the A
// operand: S^T = K Q^T with 16 keys by 8 rows, O^T += V^T P^T with 16 dimensions by 8 rows,
// so that 8 rows cost half of what a 16-row A operand would. The order of d inside a K step
// and of V's rows is free, and is chosen so that a lane's operands are contiguous bytes: 32
// of each of its two keys, 16 of each of its four values (byte pairs of two keys by PRMT).
// P^T comes out of S^T's accumulators by movmatrix. (mma.sync: with 8 to 16 rows tcgen05's
// 128-row tile would be nine tenths padding, and its operands would have to be converted
// through shared memory. The other kernel takes over above kQ8MaxRows. 32 rows a head here and
// there: 65,536 tokens of 8 heads 60 and 73 us, 8,192 tokens 23.6 and 25.6, 1,024 tokens 17.4
// and 21.5; 48 rows: 81 and 73, 25.6 and 25.6, 17.4 and 21.5.)
//
// A chunk's keys go round the CTA's warps in steps of 16; the warps' (m, l, O) are merged in
// shared memory at the end and leave as the chunk's partial, which combine.cu joins.
//
// Measured, both launches of the call together (B200, copy rate 6.5 TB/s): 8 sequences of
// 32k tokens, 4 heads, 8 rows a head: 57 us, 4.7 TB/s; one sequence of 64k tokens: 25 us for
// 67 MB, of which the loop over keys takes 13 (5.2 TB/s) and launch, the first loads' chain
// (lengths, page table, cache), the merge and the combine the rest.
#include "q8_device.cuh"
#include "sm100.cuh"

namespace ls {
namespace {
using sm100::ex2_approx;

constexpr int kStep = 16;                // keys a warp takes at a time
constexpr float kRaise = 6.0f;           // log2 units that a score may exceed the running maximum by
constexpr float kOff = 9.0f;             // so weights stay below 2^15

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Of two packed bf16 values: the larger magnitude, and both times mul as f16.
__device__ __forceinline__ float largest(uint32_t w) {
  return fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xffff0000u)));
}
__device__ __forceinline__ uint32_t f16_of(uint32_t w, float mul) {
  return pack_f16x2(__uint_as_float(w << 16) * mul, __uint_as_float(w & 0xffff0000u) * mul);
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// (The hint brings a whole key of two neighbouring heads: 57.7 -> 56.7 us for 8 sequences of
// 32k tokens against 128 bytes, which is what no hint gives as well.)
__device__ __forceinline__ void copy16(uint32_t to, const uint8_t* from) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const float* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}

// 16 cached keys and values as one lane multiplies them: with n = lane / 4, c = lane % 4, key
// words of keys n and n + 8 (d = 16 c + 64 h .. + 15), value words of keys 2c, 2c + 1,
// 2c + 8, 2c + 9 (d = n * D / 8 .. + D / 8 - 1).
template <int D>
struct Frag {
  uint32_t k[2][D / 16];
  uint32_t v[4][D / 32];
  float ks, vs;
};

// A warp's ring: kStages steps of 16 keys, 16 values and their scales. Chunk ch (16 bytes) of
// key k's row sits at ch ^ f(k), which makes the fragments' reads free of bank conflicts at
// d = 128 (at d = 64 two rows share a line, and the values' reads meet two to a bank).
template <int D, int NT>
struct Ring {
  static constexpr int kStages = D == 128 ? (NT == 1 ? 3 : 4) : (NT == 1 ? 5 : 6);
  static constexpr int kTile = kStep * D;         // bytes of a step's keys (or values)
  static constexpr int kStage = 2 * kTile + 16;   // and the two scales
  static constexpr int kBytes = kStages * kStage;  // a warp's
  static __device__ __forceinline__ int place(int key, int ch) {
    const int f = D == 128 ? (key & 7) ^ ((key & 1) << 2) : (key >> 1) & 3;
    return key * D + ((ch ^ f) << 4);
  }
};

// What a step costs is a chain of dependent instructions, so as many warps as their registers
// allow: two CTAs of 8 an SM for units of 8 rows (one streams while the other starts or
// ends), one of 12 for 16 rows.
constexpr int warps_of(int nt) { return nt == 1 ? 8 : 12; }
constexpr int ctas_of(int nt) { return nt == 1 ? 2 : 1; }

// A tree of at most kQ8MaxRows rows has at most that many nodes: two steps.
constexpr int kTreeSteps = 2;
static_assert(kTreeSteps * kStep >= kQ8MaxRows, "tree steps");

// The warps' rings, and the tree parts' O.
template <int D, int NT>
constexpr int smem_bytes() {
  return warps_of(NT) * Ring<D, NT>::kBytes + kTreeSteps * 8 * NT * (D + 4) * 4;
}

template <int D, int NT>
__global__ void __launch_bounds__(32 * warps_of(NT), ctas_of(NT)) q8_rows_kernel(const __grid_constant__ Q8Args a) {
  constexpr int kWarps = warps_of(NT), kThreads = 32 * kWarps;
  constexpr int kStride = kWarps * kStep;  // keys between a warp's steps
  constexpr int R = 8 * NT;          // rows of a unit
  constexpr int kKS = D / 16;        // K steps of a score
  constexpr int kMT = D / 16;        // 16-row tiles of O^T
  constexpr int kVB = D / 8;         // value bytes of a lane
  constexpr int kPad = D + 4;
  using Rg = Ring<D, NT>;
  static_assert(ctas_of(NT) * (smem_bytes<D, NT>() + 8192) <= 228 * 1024, "shared memory");
  static_assert(R * kPad * 4 <= Rg::kBytes, "a warp's O takes its ring's place");
  extern __shared__ __align__(16) uint8_t smem[];  // the warps' rings
  __shared__ float sm[kWarps + kTreeSteps][R], sl[kWarps + kTreeSteps][R];  // the warps', then the tree's
  __shared__ uint2 qs[NT][kKS][32];
  __shared__ float q_inv[R];
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

  // ---- the cache, kStages - 1 steps ahead
  uint8_t* ring = smem + warp * Rg::kBytes;
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  constexpr int kChunks = D / 16, kCopies = kStep * kChunks / 32;  // 16-byte chunks of a row; a lane's of a tile
  const int ch = lane % kChunks, kr = lane / kChunks;              // this lane's chunk, and row of the first copy
  const uint8_t* kbase = kv.k_pages + c.kh * D + 16 * ch + kr * stride;
  const uint8_t* vbase = kv.v_pages + c.kh * D + 16 * ch + kr * stride;
  const float* sbase = (lane ? kv.v_scale : kv.k_scale) + c.kh;
#if defined(LS_DEBUG)
  uint32_t dbg = 0u;
  LS_DCHECK(dbg, (int64_t)blockIdx.x < p.n_chunks && p.slot_rows == R && c.b < p.B && c.kh < p.Hkv);
  LS_DCHECK(dbg, tree_base >= 0 && tree_base + tree_n <= p.N && (row0 + rows - 1) / p.g < tree_n);
  LS_DCHECK(dbg, c.key_begin == c.key_end || (c.key_begin % kStep == 0 && c.key_skip % kStep == 0));
  LS_DCHECK(dbg, c.key_skip + c.key_end <= seq_len);
#endif
  // cache row of the step's first key (a step never crosses a page: both are multiples of 16)
  auto find = [&](int key) -> int32_t {
    LS_DCHECK(dbg, key >= c.key_end || q8_page_exists(kv, c.b, c.key_skip + key));
    return key < c.key_end ? q8_row(kv, c.b, c.key_skip + key) : 0;
  };
  auto copy = [&](int stage, int key, int32_t row) {
    if (key < c.key_end) {
      LS_DCHECK(dbg, row >= 0 && row + kStep <= kv.num_pages * kv.page_size && row % kStep == 0);
      const uint32_t to = ring_at + stage * Rg::kStage;
      const int64_t from = (int64_t)row * stride;
      const uint8_t *kp = kbase + from, *vp = vbase + from;
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        const int at = Rg::place(kr + i * (32 / kChunks), ch);
        copy16(to + at, kp);
        copy16(to + Rg::kTile + at, vp);
        kp += stride * (32 / kChunks);
        vp += stride * (32 / kChunks);
      }
      if (lane < 2) copy4(to + 2 * Rg::kTile + 4 * lane, sbase + (int64_t)(row >> kv.scale_shift) * p.Hkv);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // Lane l holds the row of this warp's step 32 * batch + l: one table read for 32 steps, and
  // the next batch's is under way (a read a step held every copy up by its latency).
  const int key0 = c.key_begin + warp * kStep;
  auto find_batch = [&](int batch) { return find(key0 + (32 * batch + lane) * kStride); };
  int32_t rows_now = find_batch(0), rows_next = find_batch(1);
  int ahead = 0;  // the next step to copy
  auto copy_next = [&](int stage) {
    copy(stage, key0 + ahead * kStride, __shfl_sync(0xffffffffu, rows_now, ahead & 31));
    if ((++ahead & 31) == 0) {
      rows_now = rows_next;
      rows_next = find_batch((ahead >> 5) + 1);
    }
  };
#pragma unroll
  for (int s = 0; s < Rg::kStages - 1; ++s) copy_next(s);

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
  // ---- Q^T as B operands, in shared memory (every warp multiplies by the same ones): row n of
  // each row tile, f16, scaled by a power of two a row; warp t makes tile t's
  if (a.after_prep) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp < NT) {
    const int r = 8 * warp + n;
    uint2 w[kKS];
    float amax = 0.f;
    if (r < rows) {
      const int node = (row0 + r) / p.g, j = (row0 + r) % p.g;
      const uint16_t* qp = a.q + ((size_t)(tree_base + node) * p.Hq + c.kh * p.g + j) * D + 16 * c4;
#pragma unroll
      for (int s = 0; s < kKS; ++s) {
        w[s] = *reinterpret_cast<const uint2*>(qp + 64 * (s / 4) + 4 * (s % 4));
        amax = fmaxf(amax, fmaxf(largest(w[s].x), largest(w[s].y)));
      }
    } else {
#pragma unroll
      for (int s = 0; s < kKS; ++s) w[s] = make_uint2(0u, 0u);
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int sh = f16_shift(amax);
    const float mul = pow2f(sh);
#pragma unroll
    for (int s = 0; s < kKS; ++s) qs[warp][s][lane] = make_uint2(f16_of(w[s].x, mul), f16_of(w[s].y, mul));
    if (c4 == 0) q_inv[r] = pow2f(-sh);
  }
  __syncthreads();
  float cs[NT][2];  // score factor of rows 2c, 2c + 1: softmax scale * log2(e) / the row's power of two
  int cuts[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    cuts[t][0] = cut[8 * t + 2 * c4];
    cuts[t][1] = cut[8 * t + 2 * c4 + 1];
    cs[t][0] = p.scale_log2 * q_inv[8 * t + 2 * c4];
    cs[t][1] = p.scale_log2 * q_inv[8 * t + 2 * c4 + 1];
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
  auto compute = [&](const uint8_t* tile, int k0) {
    Frag<D> f;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int hf = 0; hf < D / 64; ++hf) {
        const uint4 x = *reinterpret_cast<const uint4*>(tile + Rg::place(n + 8 * j, c4 + 4 * hf));
        f.k[j][4 * hf] = x.x;
        f.k[j][4 * hf + 1] = x.y;
        f.k[j][4 * hf + 2] = x.z;
        f.k[j][4 * hf + 3] = x.w;
      }
    f.ks = reinterpret_cast<const float*>(tile + 2 * Rg::kTile)[0];
    f.vs = reinterpret_cast<const float*>(tile + 2 * Rg::kTile)[1];
    float s[NT][4], s2[NT][4];  // two chains of products
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = s2[t][e] = 0.f;
#pragma unroll
    for (int i = 0; i < kKS; ++i) {
      const uint32_t a0 = e4m3x2_f16x2(f.k[0][i]), a1 = e4m3x2_f16x2(f.k[1][i]);
      const uint32_t a2 = e4m3x2_f16x2_hi(f.k[0][i]), a3 = e4m3x2_f16x2_hi(f.k[1][i]);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint2 q = qs[t][i][lane];
        mma16816(i & 1 ? s2[t] : s[t], a0, a1, a2, a3, q.x, q.y);
      }
    }
    // scales: a key's below f32's normals counts as 2^-126 (its scores are 0 either way), a
    // value's as the nearer end of [2^-60, 2^64]
    const float ks = fmaxf(f.ks, 1.17549435e-38f);
    const float vs = fminf(fmaxf(f.vs, 8.6736174e-19f), 1.8446744e19f);
    const float lv = lg2_approx(vs), rv = rcp_approx(vs);  // off by 2^-22, like the exponentials
    const bool edge = k0 + kStep > c.key_end;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = fmaf(s[t][e] + s2[t][e], ks * cs[t][e & 1], lv);
    if (edge || win) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int kk = k0 + n + 8 * (e >> 1);
          if (kk >= c.key_end || kk < cuts[t][e & 1]) s[t][e] = -INFINITY;
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int kk = 2 * c4 + (j & 1) + 8 * (j >> 1);
      if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(tile + Rg::kTile + Rg::place(kk, n));
        f.v[j][0] = x.x;
        f.v[j][1] = x.y;
        f.v[j][2] = x.z;
        f.v[j][3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(tile + Rg::kTile + Rg::place(kk, n >> 1) + 8 * (n & 1));
        f.v[j][0] = x.x;
        f.v[j][1] = x.y;
      }
    }
    if (edge) {  // rows past the sequence hold anything: no NaN into the product
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (k0 + 2 * c4 + (j & 1) + 8 * (j >> 1) >= c.key_end)
#pragma unroll
          for (int w = 0; w < D / 32; ++w) f.v[j][w] = 0u;
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
  int stage = 0;
  for (int key = key0; key < c.key_end; key += kStride) {
    asm volatile("cp.async.wait_group %0;" ::"n"(Rg::kStages - 2) : "memory");
    __syncwarp();  // the stage is there for every lane, and every lane is done with the one before
    copy_next(stage == 0 ? Rg::kStages - 1 : stage - 1);
    compute(ring + stage * Rg::kStage, key);
    stage = stage == Rg::kStages - 1 ? 0 : stage + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
  // This warp's result into its ring's place: its rows' maxima and sums, and O^T. (The tree
  // block starts anew: carried along, its registers spilled into the loop above.)
  auto part_of = [&](int part) {
    return reinterpret_cast<float*>(smem + min(part, kWarps) * Rg::kBytes) + max(part - kWarps, 0) * R * kPad;
  };
  auto put = [&](int part) {
    float* to = part_of(part);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float s = l[t][e];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        if (n == 0) {
          sm[part][8 * t + 2 * c4 + e] = m[t][e];
          sl[part][8 * t + 2 * c4 + e] = s;
        }
      }
#pragma unroll
      for (int i = 0; i < kMT; ++i) {
        float* at = to + (8 * t + 2 * c4) * kPad + kVB * n + 2 * i;
        *reinterpret_cast<float2*>(at) = make_float2(o[t][i][0], o[t][i][2]);
        *reinterpret_cast<float2*>(at + kPad) = make_float2(o[t][i][1], o[t][i][3]);
      }
    }
  };
  put(warp);

  // ---- the tree block, a step for each of the last warps: bf16 keys and values, scaled into
  // f16 by powers of two (a key's own, and one for the step's values, which then acts as their
  // scale). Both are read twice, for the power and for the product, rather than held.
  const int tree_step = kWarps - 1 - warp, x0 = tree_step * kStep;
  if (c.has_tree && x0 < tree_n) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][i][e] = 0.f;
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
    }
    float s[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
    auto key_word = [&](int j, int i) {
      const int x = x0 + n + 8 * j;
      const uint16_t* kp = a.k_tree + (int64_t)(tree_base + x) * stride + c.kh * D + 16 * c4;
      return x < tree_n ? *reinterpret_cast<const uint2*>(kp + 64 * (i / 4) + 4 * (i % 4)) : make_uint2(0u, 0u);
    };
    float kmul[2], kinv[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < kKS; ++i) amax = fmaxf(amax, fmaxf(largest(key_word(j, i).x), largest(key_word(j, i).y)));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      kmul[j] = pow2f(f16_shift(amax));
      kinv[j] = pow2f(-f16_shift(amax));
    }
#pragma unroll
    for (int i = 0; i < kKS; ++i) {
      const uint2 w0 = key_word(0, i), w1 = key_word(1, i);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint2 q = qs[t][i][lane];
        mma16816(s[t], f16_of(w0.x, kmul[0]), f16_of(w1.x, kmul[1]), f16_of(w0.y, kmul[0]), f16_of(w1.y, kmul[1]), q.x,
                 q.y);
      }
    }
    auto value_word = [&](int j, int i) {  // values 2i and 2i + 1 of the lane's node j
      const int x = x0 + 2 * c4 + (j & 1) + 8 * (j >> 1);
      const uint16_t* vp = a.v_tree + (int64_t)(tree_base + x) * stride + c.kh * D + kVB * n;
      return x < tree_n ? *reinterpret_cast<const uint32_t*>(vp + 2 * i) : 0u;
    };
    float vmax = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < kVB / 2; ++i) vmax = fmaxf(vmax, largest(value_word(j, i)));
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
    for (int i = 0; i < kMT; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = f16_of(value_word(j, i), vmul);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        mma16816(o[t][i], __byte_perm(w[0], w[1], 0x5410), __byte_perm(w[0], w[1], 0x7632),
                 __byte_perm(w[2], w[3], 0x5410), __byte_perm(w[2], w[3], 0x7632), b[t][0], b[t][1]);
    }
    put(kWarps + tree_step);
  }

  // ---- the warps' results joined: rows' maxima and sums, then O^T weighted
  __syncthreads();
  const int parts = kWarps + (c.has_tree ? (tree_n + kStep - 1) / kStep : 0);
  const size_t slot = (size_t)blockIdx.x * p.slot_rows;
  for (int idx = tid; idx < rows * (D / 4); idx += kThreads) {
    const int r = idx / (D / 4), d = idx % (D / 4) * 4;
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < parts; ++w) M = fmaxf(M, sm[w][r]);
    const float ref = M == -INFINITY ? 0.f : M;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < parts; ++w) {
      const float f = ex2_approx(sm[w][r] - ref);  // 0 for a warp that saw no key
      L = fmaf(sl[w][r], f, L);
      const float4 v = *reinterpret_cast<const float4*>(part_of(w) + r * kPad + d);
      acc.x = fmaf(v.x, f, acc.x);
      acc.y = fmaf(v.y, f, acc.y);
      acc.z = fmaf(v.z, f, acc.z);
      acc.w = fmaf(v.w, f, acc.w);
    }
    const float inv = M == -INFINITY ? 0.f : 1.f / L;
    *reinterpret_cast<float4*>(a.o_part + (slot + r) * D + d) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (d == 0) a.lse_part[slot + r] = M == -INFINITY ? -INFINITY : M - kOff + log2f(L);
  }
  uint32_t status = bad_s ? kErrBadTree : 0u;
#if defined(LS_DEBUG)
  status |= __syncthreads_or((int)dbg) ? kErrIndex : 0u;
#endif
  if (tid == 0) a.chunk_status[blockIdx.x] = status;
}

template <int D, int NT>
cudaError_t launch(const Q8Args& a, cudaStream_t stream) {
  const int smem = smem_bytes<D, NT>();
  static bool configured[kMaxConfigured] = {};  // per template instance
  const cudaError_t e = configure_once(q8_rows_kernel<D, NT>, smem, configured);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.p.n_chunks);
  cfg.blockDim = dim3(32 * warps_of(NT));
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
