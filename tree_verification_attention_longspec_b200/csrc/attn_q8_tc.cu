// Attention partials over the 8-bit cache on the 5th-generation tensor cores.
//
// The computation, the work split and the partials are partials_tc.cu's: one CTA per chunk,
// a 256-row unit as two 128-row query tiles in ping-pong (or, for a unit of at most 128
// rows, both tiles on its rows and alternate key blocks), S_t and O_t in TMEM, P over the
// scores, the tree block last. What the 8-bit cache changes:
//
// Operands. tcgen05 takes both operands of a product in one type. The codes are exact in
// f16, so K and V become f16 tiles in shared memory, Q becomes f16 in place (each row times
// a power of two that brings its largest element to [2^14, 2^15): exact down to 2^-29 of
// it), and so do the tree block's keys and values (a power of two for each of the two
// tiles). P is f16 too: 11 bits where bf16 has 8, as long as it is at least 2^-14 (see Scales).
// Scales. A score is s * ck + lv in the log2 domain, ck the key block's scale times the
// softmax scale over the row's power of two, lv = log2 of the value scale; both are constant
// over 16 keys (no scale block is shorter), so they cost one multiplier and one addend a
// group. P = 2^(s * ck + lv - m + kOff) then carries the value scale, the product needs
// none, and the row's sum takes it out again, 1 / vs a group. m is the running maximum of
// s * ck + lv, raised when exceeded by kRaise, so P stays below 2^15. What this costs: a weight
// times its scale that is below 2^-23 of the row's largest such product (M) is a subnormal f16,
// off by up to 2^-25, which is 2^-34 M; a block of much smaller values than another's loses
// bits to it, in dimensions where that one holds zeros.
//
// Warp roles (384 threads, one CTA per SM):
//   warps 0-3, 4-7  softmax of tile 0, of tile 1
//   warp 8          TMA producer: Q, then the blocks' codes (page by page) into a raw ring;
//                   the blocks' scales into a table
//   warp 9          MMA issuer
//   warps 10, 11    converters: raw tile -> swizzled f16 tile (cvt.f16x2.e4m3x2, two codes an
//                   instruction; rows past the sequence become zeros, so that whatever they
//                   hold meets weight 0 as 0), and the tree's keys and values from
//                   global memory
// By halves. S, P and the running maximum go by 64 keys: while a tile's softmax works at one
// half of its scores, the tensor core replaces the other, whose P it has used (O_t += P V of
// that half, then Q K^T of the next block's into its place), so neither waits for the other's
// turn. Whole blocks at a time left every softmax warp idle for half the period. (Q K^T at
// N = 64 reads Q twice as often; the tensor core has the time.) A raise of the maximum, rare,
// waits for the last half's product before it rescales O_t.
// Issue. All lanes of the MMA warp go along and one issues, so that descriptors stay in uniform
// registers: from one lane's an MMA took 60 cycles to issue, and the issuer was what bound the
// kernel (107 us against 84.5).
//
// Rings. A block holds its V and the next K for its whole length, so two more f16 tiles let the
// converters run a block ahead; the raw ring gets what is left (three and four: 82.5 us, four
// and two: 80.9).
//
// Measured (B200): 64 nodes, 28 heads over 4, 65,536 tokens: 77 us on the device (85 a call
// with the combine), 780 TFLOP/s, 0.47 of the measured bf16 rate; 64 nodes over 16,384 tokens:
// 32 us (37 a call). A
// half takes a softmax warp some 1,700 cycles, in which its SM quarter's two warps issue twice
// 430 instructions and 64 exponentials a row (1,024 cycles of the MUFU), and two quarters a
// converter's 350 (there being no 8-bit operand for K without Q and P in 8 bits too). Tried,
// and no faster here: an eighth to a third of the exponentials by polynomial on the FMA pipe
// (84.9 to 86 from 84.5), a higher threshold of raises (no change), registers moved from the converters to the softmax (428: the
// converters spill), four converter warps. The converter's loop is not unrolled: the roles
// share the code cache (92 us with, 88 without).
// Every wait is bounded; on a timeout the CTA raises an abort flag, all roles drain their
// in-flight copies and MMAs, TMEM is freed, and the chunk status reports it.
#include "q8_device.cuh"
#include "sm100.cuh"
#include "tensor_maps.cuh"

namespace ls {
namespace {
using namespace sm100;

constexpr int kThreads = 384;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kConvertWarp = 10;  // and 11
constexpr int kConverters = 64;   // threads
constexpr int kTiles = 2;         // 128-row query tiles per CTA
constexpr int kHalf = 64;         // keys per P half
constexpr int kGroup = 16;        // keys that share their scales for certain
constexpr int kGroups = kBlockN / kGroup;
constexpr int kTables = 8;  // scale tables in flight: a block's is written after the softmax of the eighth before it
constexpr float kRaise = 6.0f;  // log2 units that a score may exceed the running maximum by
constexpr float kOff = 9.0f;    // so P stays below 2^15
static_assert(kUnitRows == kTiles * 128, "a unit is two 128-row tiles");

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kPanelBytes = 128 * 128;             // 128 rows x 64 f16, 128B-swizzled
  static constexpr int kTileBytes = kPanels * kPanelBytes;  // 128 rows x D f16
  static constexpr int kRawBytes = 128 * D;                 // 128 rows x D codes
  static constexpr int kSlots = D == 128 ? 4 : 6;           // f16 tiles
  static constexpr int kRaw = D == 128 ? 2 : 8;             // raw tiles
  // Q: [panel][kUnitRows rows][128 B]; tile t is rows [128 t, 128 t + 128) of each panel
  static constexpr int kQPanelBytes = kUnitRows * 128;
  static constexpr int kQOff = 0;
  static constexpr int kSlotOff = kPanels * kQPanelBytes;
  static constexpr int kRawOff = kSlotOff + kSlots * kTileBytes;
  static constexpr int kBarOff = kRawOff + kRaw * kRawBytes;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS = 0;    // S_t / P_t at 128 t
  static constexpr uint32_t kColO = 256;  // O_t at 256 + D t
  static_assert(kPanels * kQPanelBytes >= 128 * D * 4 && kSlots * kTileBytes >= 128 * D * 4, "epilogue staging");
};

struct alignas(64) TcParams {
  CUtensorMap tmap_q;
  CUtensorMap tmap_k;  // codes
  CUtensorMap tmap_v;
  CUtensorMap tmap_o;  // o_part as [n_chunks * 256 rows][d] fp32, stores of 128 rows x 32 floats
  Q8Args a;
};

struct Bars {
  uint64_t q_full;                      // the unit's Q rows are in shared memory (bf16)
  uint64_t raw_full[8], raw_empty[8];   // raw tiles
  uint64_t full[6], empty[6];           // f16 tiles
  uint64_t table_full[kTables];         // a block's scales
  uint64_t s_full[kTiles][2];           // half h of S_t(j) is in TMEM (and O_t holds every PV but the last half's)
  uint64_t p_full[kTiles][2];           // half h of P_t(j) is in TMEM
  uint64_t pv_done[kTiles];             // O_t holds one more half
  uint64_t o_full[kTiles];              // every MMA of tile t finished
  uint64_t tree_full;                   // tree_max is there
  uint64_t mask_full;                   // the tree's Ancestors are, in raw tile mask_slot's place
  uint32_t tmem_base;
  uint32_t abort;
  uint32_t tree_err;                    // a parent link that is not a rooted tree's
  uint32_t dbg;                         // index-checking builds: kErrIndex once a check failed
  int32_t mask_slot;
  float kc[kTables][kGroups];           // key scales of the block's groups
  float lv[kTables][kGroups];           // log2 of the value scales
  float rv[kTables][kGroups];           // 1 / value scale
  uint32_t tree_max[2];                 // largest magnitudes of the tree's keys and values (float bits)
  int8_t q_shift[kUnitRows];            // log2 of the row's power of two
  int16_t parent[kMaxTree];             // the sequence's tree (chunks that hold the tree block)
};
static_assert(Cfg<128>::kRaw <= 8 && Cfg<64>::kRaw <= 8 && Cfg<128>::kSlots <= 6 && Cfg<64>::kSlots <= 6, "barriers");

// The dynamic window of a CTA less 1 KB; the layout is aligned up to 1024 bytes inside it
// (the 128-byte swizzle atom repeats every 1024 bytes).
constexpr int kSmemWindow = 232448;
template <int D>
constexpr int smem_need() {
  return Cfg<D>::kBarOff + (int)sizeof(Bars) + 1024;
}
static_assert(smem_need<128>() <= kSmemWindow && smem_need<64>() <= kSmemWindow, "shared memory");

// Instruction descriptor for kind::f16 with f16 A/B and an fp32 accumulator.
constexpr uint32_t umma_idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4)                                 // D: f32 (A, B: f16 = 0)
         | ((b_mn_major ? 1u : 0u) << 16)          // B major-ness (A is K-major)
         | (static_cast<uint32_t>(N >> 3) << 17)   // N / 8
         | (static_cast<uint32_t>(M >> 4) << 24);  // M / 16
}

// True in one lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// Largest magnitude of eight bf16 values, as the bits of one (ordered like the values), in
// both halves of m; NaN is skipped.
__device__ __forceinline__ void take_max(uint32_t (&m)[4], const uint4& w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) asm("max.bf16x2 %0, %0, %1;" : "+r"(m[e]) : "r"(u[e] & 0x7fff7fffu));
}
__device__ __forceinline__ float join_max(const uint32_t (&m)[4]) {
  float x = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) x = fmaxf(x, fmaxf(__uint_as_float(m[e] << 16), __uint_as_float(m[e] & 0xffff0000u)));
  return x;
}

// The largest finite magnitude of n rows of D bf16 values, by one warp; for the rare tree with an
// infinite key. (Not inlined: where its code lay between the others', the kernel ran 5% longer.)
template <int D>
__device__ __noinline__ float finite_max(const uint16_t* from, int n, int stride) {
  uint32_t m = 0u;
#pragma unroll 1
  for (int i = threadIdx.x & 31; i < n * D; i += 32) {
    const uint32_t u = from[(size_t)(i / D) * stride + i % D] & 0x7fffu;
    m = u < 0x7f80u ? max(m, u) : m;
  }
  return __uint_as_float(__reduce_max_sync(0xffffffffu, m) << 16);
}

// Eight bf16 values times mul, as f16.
__device__ __forceinline__ uint4 f16_of_bf16(const uint4& w, float mul) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint32_t r[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    r[e] = pack_f16x2(__uint_as_float(u[e] << 16) * mul, __uint_as_float(u[e] & 0xffff0000u) * mul);
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// P for 64 scores of four groups: 2^(s * ck + cm), packed to f16 pairs; adds each group's
// sum, times rv, to l. A masked score (-inf) gives 0.
__device__ __forceinline__ void make_p(const float (&s)[kHalf], const float* ck, const float* cm, const float* rv,
                                       uint32_t (&pk)[kHalf / 2], float& l) {
#pragma unroll
  for (int g = 0; g < kHalf / kGroup; ++g) {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int e = g * kGroup / 2; e < (g + 1) * kGroup / 2; ++e) {
      float x0, x1;
      fma2_bc(x0, x1, s[2 * e], s[2 * e + 1], ck[g], cm[g]);
      const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
      add2(s0, s1, p0, p1);
      pk[e] = pack_f16x2(p0, p1);
    }
    l = fmaf(s0 + s1, rv[g], l);
  }
}

// Tree mask (LongSpec, gist.science summary, section 2C, "Baum-Maskierung"): the nodes that
// each of the tree's n nodes sees, itself and its ancestors, as bits, by one warp. Every link
// is checked (node 0 is the root with parent -1, any other node's parent lies below it); false
// in a lane that found a bad one, which then counts as a root. Seven rounds of pointer jumping
// cover 128 levels; a lane's nodes are lane, lane + 32, ...: `up` and `seen` hold all of them
// between rounds.
struct Ancestors {
  uint32_t seen[kMaxTree][4];
  int32_t up[kMaxTree];
};
__device__ __forceinline__ bool find_ancestors(Ancestors* t, const int32_t* parent, int n, int lane) {
  bool good = true;
  for (int x = lane; x < kMaxTree; x += 32) {
    const int pp = x < n ? parent[x] : -1;
    const bool fine = x == 0 || x >= n ? pp == -1 : pp >= 0 && pp < x;
    good &= fine;
    t->up[x] = fine ? pp : -1;
#pragma unroll
    for (int w = 0; w < 4; ++w) t->seen[x][w] = x >> 5 == w ? 1u << (x & 31) : 0u;
  }
  __syncwarp();
  for (int round = 0; round < 7; ++round) {
    uint32_t more[kMaxTree / 32][4];
    int32_t next[kMaxTree / 32];
#pragma unroll
    for (int q = 0; q < kMaxTree / 32; ++q) {
      const int y = t->up[lane + 32 * q];
      next[q] = y >= 0 ? t->up[y] : -1;
#pragma unroll
      for (int w = 0; w < 4; ++w) more[q][w] = y >= 0 ? t->seen[y][w] : 0u;
    }
    __syncwarp();
#pragma unroll
    for (int q = 0; q < kMaxTree / 32; ++q) {
      t->up[lane + 32 * q] = next[q];
#pragma unroll
      for (int w = 0; w < 4; ++w) t->seen[lane + 32 * q][w] |= more[q][w];
    }
    __syncwarp();
  }
  return good;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) q8_tc_kernel(const __grid_constant__ TcParams P) {
  using C = Cfg<D>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kBarOff);
  const Q8Args& a = P.a;
  const Plan& p = a.p;
  const KvQ8& kv = a.kv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint64_t wait_ns = (uint64_t)p.wait_ns;  // limit of every bounded wait below

  const int32_t* cu = plan_cu(p, a.cu);  // kernel parameters when the host gave lengths
  const ChunkCoord c = locate_chunk(p, cu, blockIdx.x);
  if (!c.valid) return;  // more CTAs than the device lengths need: the combine reports it
  const int n_keys = c.key_end - c.key_begin;
  const int nb = (n_keys + kBlockN - 1) / kBlockN;     // prefix blocks
  const int tail_end = n_keys - (nb - 1) * kBlockN;    // keys of the last one
  const bool has_tree = c.has_tree;
  const int nbt = nb + (has_tree ? 1 : 0);  // blocks, the tree block (block nb) last
  const int seq_len = cu[c.b + 1] - cu[c.b];
  // sliding window: a row at depth d sees the attended keys from window_cut(d) on, which
  // is below 2 * 128, so only the chunks that start there cut rows individually
  const bool win_rows = p.window > 0 && nb > 0 && c.key_begin < 2 * kBlockN;
  int tree_base, tree_n;  // the sequence's tree nodes (none if cu_tree is bad: the combine reports it)
  tree_range(p, a.cu_tree, c.b, &tree_base, &tree_n);
  const int tok0 = c.rgi * p.tpu;                         // first tree node of the unit
  const int rows_here = min(p.tpu, tree_n - tok0) * p.g;  // rows of the unit that exist
  const bool alt = unit_alternates(rows_here);            // both tiles on these rows
  if (rows_here <= 0) {  // a unit past the sequence's tree: nothing to attend for
    if (tid == 0) a.chunk_status[blockIdx.x] = 0u;
    return;
  }
  if (nbt == 0) {  // empty key range: an empty partial (two of them when the tiles alternate)
    for (int r = tid; r < rows_here; r += kThreads) {
      a.lse_part[(size_t)blockIdx.x * kUnitRows + r] = -INFINITY;
      if (alt) a.lse_part[(size_t)blockIdx.x * kUnitRows + 128 + r] = -INFINITY;
    }
    if (tid == 0) a.chunk_status[blockIdx.x] = 0u;
    return;
  }
  volatile uint32_t* abort = &bars->abort;

  // The tiles in the order that the MMA thread uses them: K(j), V(j) for j = 0, 1, ...; with
  // alternate blocks K(0), K(1), then V(j) and K(j + 2) for j = 0, 1, ... (no K past the
  // last block).
  const int n_tiles = 2 * nbt;
  const int pro = nbt < 2 ? nbt : 2, pairs = nbt > 2 ? nbt - 2 : 0;
  auto tile_of = [&](int ld, int* j, int* val) {
    if (!alt) {
      *j = ld >> 1;
      *val = ld & 1;
    } else if (ld < pro) {
      *j = ld;
      *val = 0;
    } else if (ld - pro < 2 * pairs) {
      const int r = ld - pro;
      *j = (r >> 1) + ((r & 1) ? 2 : 0);
      *val = (r & 1) ? 0 : 1;
    } else {
      *j = pairs + (ld - pro - 2 * pairs);
      *val = 1;
    }
  };
  // When the tree kernel writes q and k_tree (rotated), this grid may start before that grid
  // ends: the prefix loads go ahead, Q and the tree block wait for it.
  auto wait_prior = [&]() {
    if (a.after_prep) asm volatile("griddepcontrol.wait;" ::: "memory");
  };

  // Block j's scale table, lane g writing group g's entries (one whole warp).
  auto write_scales = [&](int j, float k, float lv, float rv) {
    if (lane < kGroups) {
      bars->kc[j % kTables][lane] = k;
      bars->lv[j % kTables][lane] = lv;
      bars->rv[j % kTables][lane] = rv;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->table_full[j % kTables]);
  };

  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_map(&P.tmap_q);
    tma_prefetch_map(&P.tmap_k);
    tma_prefetch_map(&P.tmap_v);
    mbar_init(&bars->q_full, 1);
    for (int s = 0; s < C::kRaw; ++s) {
      mbar_init(&bars->raw_full[s], 1);
      mbar_init(&bars->raw_empty[s], 2);
    }
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&bars->full[s], 2);
      mbar_init(&bars->empty[s], 1);
    }
    for (int s = 0; s < kTables; ++s) mbar_init(&bars->table_full[s], 1);
    for (int t = 0; t < kTiles; ++t) {
      mbar_init(&bars->s_full[t][0], 1);
      mbar_init(&bars->s_full[t][1], 1);
      mbar_init(&bars->pv_done[t], 1);
      mbar_init(&bars->p_full[t][0], 128);
      mbar_init(&bars->p_full[t][1], 128);
      mbar_init(&bars->o_full[t], 1);
    }
    mbar_init(&bars->tree_full, 8);
    mbar_init(&bars->mask_full, 1);
    bars->tree_max[0] = bars->tree_max[1] = 0u;
    bars->abort = 0u;
    bars->tree_err = 0u;
    bars->dbg = 0u;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    if (lane == 0) tma_prefetch_map(&P.tmap_o);
    __syncwarp();
    tmem_alloc(&bars->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  // The producer, which made the barriers, does not wait for the others to see them: its first
  // loads are on their way meanwhile.
  tc_fence_before_sync();
  if (warp == kProducerWarp) {
    __syncwarp();
    asm volatile("bar.arrive 4, 384;" ::: "memory");
  } else {
    asm volatile("bar.sync 4, 384;" ::: "memory");
  }
  tc_fence_after_sync();
  const uint32_t tbase = warp == kProducerWarp ? 0u : bars->tmem_base;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------------ TMA producer
    // a box is bh rows (a page, or 128 rows of a larger one); lane l issues box l of a block
    const int bh = kv.page_size < kBlockN ? kv.page_size : kBlockN;
    const int n_boxes = kBlockN / bh;
    int issued = 0, slot = 0, use = 0;
    bool ok = true;
#if defined(LS_DEBUG)
    // the unit's nodes lie inside the tree tensors (rows of the Q box past the last read zeros),
    // its keys inside the sequence, its partial inside o_part
    if (lane == 0 && !(tok0 >= 0 && tok0 < tree_n && tree_base >= 0 && tree_base + tree_n <= p.N &&
                       c.key_skip + c.key_end <= seq_len && (int64_t)blockIdx.x < p.n_chunks && c.b < p.B && c.kh < p.Hkv))
      bars->dbg = kErrIndex;
#endif
    // A block's scales are read when its keys are asked for, and go into the table one block
    // later, when they have come.
    float ks = 1.f, vs = 1.f;
    int scaled = -1;  // the block whose scales ks, vs hold
    auto put_scales = [&]() {
      if (scaled < 0) return;
      const float v = fminf(fmaxf(vs, 8.6736174e-19f), 1.8446744e19f);
      write_scales(scaled, fmaxf(ks, 1.17549435e-38f), log2f(v), 1.f / v);
      scaled = -1;
    };
    if (lane == 0 && !a.after_prep) {
      mbar_arrive_expect_tx(&bars->q_full, C::kPanels * 128 * p.g * p.tpu);
#pragma unroll
      for (int pn = 0; pn < C::kPanels; ++pn)
        tma_load_4d(smem + C::kQOff + pn * C::kQPanelBytes, &P.tmap_q, &bars->q_full, pn * 64, 0, c.kh, tree_base + tok0);
    }
    bool q_issued = !a.after_prep;
    for (int ld = 0; ld < n_tiles && ok; ++ld) {
      if (!q_issued && (ld == 2 || issued > 0)) {
        // the first tile is on its way: now Q, once the tree kernel has written it
        wait_prior();
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars->q_full, C::kPanels * 128 * p.g * p.tpu);
#pragma unroll
          for (int pn = 0; pn < C::kPanels; ++pn)
            tma_load_4d(smem + C::kQOff + pn * C::kQPanelBytes, &P.tmap_q, &bars->q_full, pn * 64, 0, c.kh, tree_base + tok0);
        }
        q_issued = true;
      }
      int j, val;
      tile_of(ld, &j, &val);
      if (j == nb) continue;  // the tree block comes through the converters
      // this lane's page box; boxes past the sequence's end read some page (made zeros later)
      int prow = 0;
      if (lane < n_boxes) {
        const int key = c.key_skip + c.key_begin + j * kBlockN + lane * bh;
        prow = q8_row(kv, c.b, key);
#if defined(LS_DEBUG)
        // a box with keys of the sequence is a page's of the cache, and any box lies inside it
        if ((key < c.key_skip + c.key_end && !q8_page_exists(kv, c.b, key)) || prow < 0 ||
            prow + bh > kv.num_pages * kv.page_size)
          bars->dbg = kErrIndex;
#endif
      }
      if (!val) {
        put_scales();
        const int key = lane * kGroup;  // lane g: group g's row, from the lane that has its box
        const int row = __shfl_sync(0xffffffffu, prow, min(key / bh, 31)) + key % bh;
        ks = vs = 1.f;
        if (lane < kGroups && c.key_begin + j * kBlockN + key < c.key_end) {
          const size_t at = (size_t)(row >> kv.scale_shift) * p.Hkv + c.kh;
          ks = __ldg(kv.k_scale + at);
          vs = __ldg(kv.v_scale + at);
        }
        scaled = j;
      }
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bars->raw_empty[slot], (use & 1) ^ 1, abort, wait_ns));
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&bars->raw_full[slot], C::kRawBytes);
      __syncwarp();
      if (lane < n_boxes)
        tma_load_3d(smem + C::kRawOff + slot * C::kRawBytes + lane * bh * D, val ? &P.tmap_v : &P.tmap_k,
                    &bars->raw_full[slot], 0, c.kh, prow);
      ++issued;
      if (++slot == C::kRaw) {
        slot = 0;
        ++use;
      }
    }
    put_scales();
    if (has_tree && ok) {  // where the next raw tile would go
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bars->raw_empty[slot], (use & 1) ^ 1, abort, wait_ns));
      if (ok) {
        Ancestors* t = reinterpret_cast<Ancestors*>(smem + C::kRawOff + slot * C::kRawBytes);
        if (!find_ancestors(t, a.parent + tree_base, tree_n, lane)) bars->tree_err = 1u;
        if (lane == 0) {
          bars->mask_slot = slot;
          mbar_arrive(&bars->mask_full);
        }
      }
    }
    if (!q_issued) {  // no prefix tile at all
      wait_prior();
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars->q_full, C::kPanels * 128 * p.g * p.tpu);
#pragma unroll
        for (int pn = 0; pn < C::kPanels; ++pn)
          tma_load_4d(smem + C::kQOff + pn * C::kQPanelBytes, &P.tmap_q, &bars->q_full, pn * 64, 0, c.kh, tree_base + tok0);
      }
    }
    // make sure no copy is still writing shared memory when the CTA ends
    if (lane == 0) {
      drain_wait(&bars->q_full, 0);
      const int first = issued > C::kRaw ? issued - C::kRaw : 0;
      for (int seq = first; seq < issued; ++seq) drain_wait(&bars->raw_full[seq % C::kRaw], (seq / C::kRaw) & 1);
    }
    __syncwarp();
  } else if (warp >= kConvertWarp) {
    // ------------------------------------------------------------------ converters
    const int ct = tid - kConvertWarp * 32;  // 0 .. 63
    const bool first_warp = warp == kConvertWarp;
    int slot = 0, use = 0, raw = 0, raw_use = 0;
    bool ok = true;
    for (int ld = 0; ld < n_tiles && ok; ++ld) {
      int j, val;
      tile_of(ld, &j, &val);
      auto wait_slot = [&]() {
        return __all_sync(0xffffffffu, mbar_wait_bounded(&bars->empty[slot], (use & 1) ^ 1, abort, wait_ns));
      };
      uint8_t* dst = smem + C::kSlotOff + slot * C::kTileBytes;
      if (j < nb) {
        ok = wait_slot() && __all_sync(0xffffffffu, mbar_wait_bounded(&bars->raw_full[raw], raw_use & 1, abort, wait_ns));
        if (!ok) break;
        const uint8_t* src = smem + C::kRawOff + raw * C::kRawBytes;
        const int lim = j == nb - 1 ? tail_end : kBlockN;
        // A thread takes one 16-byte chunk column of every kRows-th row (kRows a multiple of 8,
        // so that the swizzle stays its own: chunk q of a panel row sits at q ^ (row & 7)). At
        // d = 128, eight lanes hold four chunks of two rows each: their stores then cover all
        // bank groups, and only the (half as many) loads meet two to a bank.
        constexpr int kChunks = D / 16, kRows = kConverters / kChunks, kIter = 128 / kRows, kBatch = 8;
        const int cc = D == 128 ? (ct & 3) | ((ct >> 1) & 4) : ct & 3;
        const int row0 = D == 128 ? ((ct >> 2) & 1) | ((ct >> 3) & 2) | ((ct >> 3) & 4) : ct >> 2;
        uint8_t* line = dst + (cc / 4) * C::kPanelBytes + row0 * 128;
        uint8_t* first = line + (((2 * (cc & 3)) ^ (row0 & 7)) << 4);
        uint8_t* second = line + (((2 * (cc & 3) + 1) ^ (row0 & 7)) << 4);
        src += row0 * D + cc * 16;
#pragma unroll 1  // (unrolled, 92 us instead of 89 for 64 nodes over 64k tokens: the roles share the code cache)
        for (int it = 0; it < kIter; it += kBatch) {
          uint4 w[kBatch];
#pragma unroll
          for (int e = 0; e < kBatch; ++e) w[e] = *reinterpret_cast<const uint4*>(src + (it + e) * kRows * D);
          if (lim < kBlockN) {
#pragma unroll
            for (int e = 0; e < kBatch; ++e)
              if (row0 + (it + e) * kRows >= lim) w[e] = make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll
          for (int e = 0; e < kBatch; ++e) {
            const int at = (it + e) * kRows * 128;
            *reinterpret_cast<uint4*>(first + at) =
                make_uint4(e4m3x2_f16x2(w[e].x), e4m3x2_f16x2_hi(w[e].x), e4m3x2_f16x2(w[e].y), e4m3x2_f16x2_hi(w[e].y));
            *reinterpret_cast<uint4*>(second + at) =
                make_uint4(e4m3x2_f16x2(w[e].z), e4m3x2_f16x2_hi(w[e].z), e4m3x2_f16x2(w[e].w), e4m3x2_f16x2_hi(w[e].w));
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->raw_empty[raw]);
        if (++raw == C::kRaw) {
          raw = 0;
          ++raw_use;
        }
      } else {
        // The tree block: bf16 rows from global memory, times a power of two for the tile (its
        // largest magnitude has been found by the softmax warps). The first rows are on their
        // way before the tile's place is free. Keys past the tree are masked whatever they
        // hold; values there become zeros.
        constexpr int kChunks = D / 8;  // 16-byte chunks of a bf16 row
        constexpr int kIter = 128 * kChunks / kConverters, kBatch = 8;
        const int used = (tree_n * kChunks + kConverters - 1) / kConverters;  // of the iterations
        if (!val) {
          wait_prior();
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bars->tree_full, 0, abort, wait_ns));
          if (!ok) break;
        }
        const uint16_t* from = (val ? a.v_tree : a.k_tree) + ((size_t)tree_base * p.Hkv + c.kh) * D;
        float most = __uint_as_float(bars->tree_max[0]);
        if (most == INFINITY) {  // a node's infinity is no measure for the others (each warp looks by itself)
          most = finite_max<D>(a.k_tree + ((size_t)tree_base * p.Hkv + c.kh) * D, tree_n, p.Hkv * D);
        }
        const int vsh = min(max(f16_shift(__uint_as_float(bars->tree_max[1])), -kMaxScaleExp), -kMinScaleExp);
        const int ksh = f16_shift(most);
        if (first_warp && !val) write_scales(j, pow2f(-ksh), (float)-vsh, pow2f(vsh));  // all groups alike
        const float mul = pow2f(val ? vsh : ksh);
#pragma unroll 1
        for (int it = 0; it < used; it += kBatch) {
          uint4 w[kBatch];
#pragma unroll
          for (int e = 0; e < kBatch; ++e) {
            const int i = ct + (it + e) * kConverters, row = i / kChunks;
            w[e] = make_uint4(0u, 0u, 0u, 0u);
            if (row < tree_n) w[e] = *reinterpret_cast<const uint4*>(from + (size_t)row * p.Hkv * D + i % kChunks * 8);
          }
          if (it == 0) ok = wait_slot();
          if (!ok) break;
#pragma unroll
          for (int e = 0; e < kBatch; ++e) {
            const int i = ct + (it + e) * kConverters, row = i / kChunks, cc = i % kChunks;
            *reinterpret_cast<uint4*>(dst + (cc / 8) * C::kPanelBytes + row * 128 + (((cc % 8) ^ (row & 7)) << 4)) =
                f16_of_bf16(w[e], mul);
          }
        }
        if (!ok) break;
        if (val) {
#pragma unroll 1
          for (int it = (used + kBatch - 1) / kBatch * kBatch; it < kIter; ++it) {
            const int i = ct + it * kConverters, row = i / kChunks, cc = i % kChunks;
            *reinterpret_cast<uint4*>(dst + (cc / 8) * C::kPanelBytes + row * 128 + (((cc % 8) ^ (row & 7)) << 4)) =
                make_uint4(0u, 0u, 0u, 0u);
          }
        }
      }
      fence_proxy_async_smem();  // the tile is read by the tensor core
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->full[slot]);
      if (++slot == C::kSlots) {
        slot = 0;
        ++use;
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ Q to f16 (warps 0-7)
    // Thread r converts row r of the unit in place: 16-byte chunks of the row, in an order
    // that starts at the lane, so that a warp's accesses spread over the banks. The rows
    // after the box's tpu * g become zeros, so that no stale shared memory enters an MMA.
    if (warp < 8) {
      if (has_tree) {
        // the largest magnitudes of the tree block's keys and values, while Q and the first
        // keys are on their way
        wait_prior();
        constexpr int kChunks = D / 8;
        uint4 w[2][kChunks / 2];  // 128 rows over 256 threads
#pragma unroll
        for (int val = 0; val < 2; ++val) {
          const uint16_t* from = (val ? a.v_tree : a.k_tree) + ((size_t)tree_base * p.Hkv + c.kh) * D;
#pragma unroll
          for (int e = 0; e < kChunks / 2; ++e) {
            const int i = tid + 256 * e, row = i / kChunks;
            w[val][e] = make_uint4(0u, 0u, 0u, 0u);
            if (row < tree_n) w[val][e] = *reinterpret_cast<const uint4*>(from + (size_t)row * p.Hkv * D + i % kChunks * 8);
          }
        }
#pragma unroll
        for (int val = 0; val < 2; ++val) {
          uint32_t m[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int e = 0; e < kChunks / 2; ++e) take_max(m, w[val][e]);
          const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(join_max(m)));
          if (lane == 0) atomicMax(&bars->tree_max[val], most);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->tree_full);
      }
      const bool got = __all_sync(0xffffffffu, mbar_wait_bounded(&bars->q_full, 0, abort, wait_ns));
      if (got) {
        const bool row_there = tid < p.tpu * p.g;
        uint8_t* line = smem + C::kQOff + tid * 128;
        uint4 w[C::kPanels * 8];
        uint32_t m[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < C::kPanels * 8; ++i) {
          w[i] = make_uint4(0u, 0u, 0u, 0u);
          if (row_there)
            w[i] = *reinterpret_cast<const uint4*>(line + (i / 8) * C::kQPanelBytes + (((i + lane) & 7) << 4));
          take_max(m, w[i]);
        }
        const int sh = f16_shift(join_max(m));
        const float mul = pow2f(sh);
        bars->q_shift[tid] = (int8_t)sh;
#pragma unroll
        for (int i = 0; i < C::kPanels * 8; ++i)
          *reinterpret_cast<uint4*>(line + (i / 8) * C::kQPanelBytes + (((i + lane) & 7) << 4)) = f16_of_bf16(w[i], mul);
      }
      fence_proxy_async_smem();
      // the tree of the sequence, for the rows' depths; a parent outside [-1, T) is stored
      // as a value that fails the walk's checks
      if (win_rows) {
        for (int x = tid; x < tree_n; x += 256) {
          const int32_t pp = a.parent[(size_t)tree_base + x];
          bars->parent[x] = (int16_t)(pp >= -1 && pp < tree_n ? pp : kMaxTree);
        }
      }
    }
    // Q and the tree are in shared memory: warps 0-7 and the MMA warp meet at barrier 1
    asm volatile("bar.sync 1, 288;" ::: "memory");

    if (warp == kMmaWarp) {
      // ---------------------------------------------------------------- MMA issuer
      // The whole warp goes along and one lane issues, so that what an MMA is given (the same in
      // all lanes) stays in uniform registers: moved there from one lane's, each took 60 cycles.
      const bool lead = elect_one();
      const uint32_t tb = __reduce_max_sync(0xffffffffu, tbase);
      const int blocks = (int)__reduce_max_sync(0xffffffffu, (uint32_t)nbt);
      const bool by_turns = __any_sync(0xffffffffu, alt);
      constexpr uint32_t idesc_qk = umma_idesc_f16(128, kHalf, false);
      constexpr uint32_t idesc_pv = umma_idesc_f16(128, D, true);
      // A descriptor differs from another of the same kind only in its start-address
      // field (address >> 4 in the low 14 bits; shared addresses stay below 256 KB, so
      // adding an offset never carries out of it): build the bases once, add offsets.
      const uint64_t dq0 = umma_sdesc_sw128(smem_u32(smem + C::kQOff), 16, 1024);
      constexpr uint32_t kQPanel16 = C::kQPanelBytes >> 4, kQTile16 = (128 * 128) >> 4;
      const uint64_t dk0 = umma_sdesc_sw128(smem_u32(smem + C::kSlotOff), 16, 1024);
      const uint64_t dv0 = umma_sdesc_sw128(smem_u32(smem + C::kSlotOff), C::kPanelBytes, 1024);
      constexpr uint32_t kTile16 = C::kTileBytes >> 4, kPanel16 = C::kPanelBytes >> 4;
      auto commit = [&](uint64_t* bar) {
        if (lead) umma_commit(bar);
      };
      // half h of S_t = Q_t K^T into that half of tile t's score buffer; K sits in ring slot `slot`
      auto issue_qk = [&](int t, int slot, int h) {
        const uint64_t dq = dq0 + (uint64_t)((by_turns ? 0 : t) * kQTile16);  // both tiles read tile 0's Q rows by turns
        const uint64_t dk = dk0 + (uint64_t)(slot * kTile16 + h * ((kHalf * 128) >> 4));
        const uint32_t tS = tb + C::kColS + t * kBlockN + h * kHalf;
        if (lead) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t koff = (kk & 3) * 2;  // 32 bytes per K step inside a panel (16-byte units)
            umma_ss(tS, dq + (kk >> 2) * kQPanel16 + koff, dk + (kk >> 2) * kPanel16 + koff, idesc_qk,
                    kk > 0 ? 1u : 0u);
          }
          umma_commit(&bars->s_full[t][h]);
        }
      };
      // O_t += P_t V over keys [64h, 64h+64) of block j: four K = 16 steps, P from TMEM
      auto issue_pv = [&](int t, int slot, int j, int h) {
        const uint64_t dv = dv0 + (uint64_t)(slot * kTile16);
        const uint32_t tP = tb + C::kColS + t * kBlockN + h * kHalf;
        const uint32_t tO = tb + C::kColO + t * D;
        if (lead) {
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {
            const int kk = 4 * h + k4;
            umma_ts(tO, tP + k4 * 8, dv + kk * (2048 / 16), idesc_pv, (j > 0 || kk > 0) ? 1u : 0u);
          }
          umma_commit(&bars->pv_done[t]);
        }
      };
      // P written by the softmax warps' tcgen05.st: their wait::st, fence and arrive pair
      // with this wait and the fence after it before an MMA reads P
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool got = __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort, wait_ns));
        tc_fence_after_sync();
        return got;
      };
      // K, V written by the converters, whose proxy fence precedes their arrival
      auto wait_tile = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort, wait_ns));
      };
      int slot = 0, use = 0;  // ring position of the next tile, in consumption order
      auto advance = [&]() {
        if (++slot == C::kSlots) {
          slot = 0;
          use ^= 1;
        }
      };
      bool ok = true;
      if (by_turns) {
        // alternate blocks: tile t takes blocks t, t + 2, ...; S_t = Q K(t)^T first, then
        // for j = 0, 1, ...: PV of block j for tile j % 2 and that tile's next QK^T, by halves
        for (int t = 0; t < kTiles && t < blocks && ok; ++t) {
          ok = wait_tile(&bars->full[slot], use);
          if (!ok) break;
          issue_qk(t, slot, 0);
          issue_qk(t, slot, 1);
          commit(&bars->empty[slot]);
          advance();
        }
        for (int j = 0; j < blocks && ok; ++j) {
          const int t = j & 1, i = j >> 1;  // tile and its own block count
          ok = wait_tile(&bars->full[slot], use);  // V(j)
          if (!ok) break;
          const int sv = slot;
          advance();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = ok && wait(&bars->p_full[t][h], i & 1);
            if (ok) issue_pv(t, sv, i, h);
            if (ok && h == 1) commit(&bars->empty[sv]);
            if (ok && j + 2 < blocks) {
              if (h == 0) ok = wait_tile(&bars->full[slot], use);  // K(j + 2)
              if (ok) issue_qk(t, slot, h);
            }
          }
          if (!ok) break;
          if (j + 2 < blocks) {
            commit(&bars->empty[slot]);
            advance();
          } else if (t == 0) {
            commit(&bars->o_full[0]);  // tile 0's last PV; no QK^T follows it
          }
        }
      } else {
        ok = wait_tile(&bars->full[slot], use);  // K(0)
        if (ok) {
#pragma unroll
          for (int x = 0; x < 2 * kTiles; ++x) issue_qk(x % kTiles, slot, x / kTiles);
          commit(&bars->empty[slot]);
          advance();
        }
        for (int j = 0; j < blocks && ok; ++j) {
          const int sv = slot, uv = use;  // V(j)
          advance();
          const bool more = j + 1 < blocks;
          const int sk = slot, uk = use;  // K(j+1), when there is one
          ok = wait_tile(&bars->full[sv], uv);
#pragma unroll
          for (int x = 0; x < 2 * kTiles; ++x) {  // halves, of each both tiles
            const int h = x / kTiles, t = x % kTiles;
            ok = ok && wait(&bars->p_full[t][h], j & 1);
            if (ok) issue_pv(t, sv, j, h);
            // V(j) is free once both tiles' PV have read it: released before the next QK^T,
            // so that its refill (a few microseconds in flight) starts that much earlier
            if (ok && x == 3) commit(&bars->empty[sv]);
            if (ok && !more && x == 2) commit(&bars->o_full[0]);  // tile 0's epilogue may start
            if (ok && more) {
              if (x == 0) ok = wait_tile(&bars->full[sk], uk);
              if (ok) issue_qk(t, sk, h);
            }
          }
          if (!ok) break;
          if (more) {
            commit(&bars->empty[sk]);
            advance();
          }
        }
      }
      // tile 0's last PV precedes tile 1's in issue order, so o_full[1] completes last
      commit(&bars->o_full[1]);
      if (lead) drain_wait(&bars->o_full[1], 0);
      __syncwarp();
    } else {
      // ---------------------------------------------------------------- softmax / epilogue
      const int t = warp >> 2;                 // query tile
      const int row = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
      const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t tS = tbase + lane_base + C::kColS + t * kBlockN;
      const uint32_t tO = tbase + lane_base + C::kColO + t * D;
      float m = -INFINITY, l = 0.f;  // running maximum (log2 units) of this row, its sum of weights
      const int ur = alt ? row : t * 128 + row;  // row of the unit (both tiles' rows when alternating)
      const bool has_row = ur < rows_here;
      const float cs = p.scale_log2 * pow2f(-(int)bars->q_shift[ur]);
      const int node = tok0 + ur / p.g;   // its tree node
      int cut = 0;                        // window: first attended key this row sees
      if (win_rows && has_row) {
        int x = node, depth = 0;
        for (int step = 0; step < kMaxTree && x > 0; ++step) {
          const int pp = bars->parent[x];
          if (pp < 0 || pp >= x) break;  // not a rooted tree: the tree block's chunk reports it
          x = pp;
          ++depth;
        }
        cut = window_cut(p, seq_len, depth);
      }
      bool ok = true;
      // blocks of this tile: all of them, or every other one (from block t) when alternating
      const int n_mine = alt ? (nbt - t + 1) / 2 : nbt;
      // Half a block at a time: while this warp works at one half, the tensor core computes the
      // other half's next scores, so that neither waits for the other's turn.
#pragma unroll 1
      for (int n = 0; n < 2 * n_mine; ++n) {
        const int i = n >> 1, h = n & 1;
        const int j = alt ? 2 * i + t : i;  // the block
        const int tb = j % kTables;
        const uint32_t tH = tS + h * kHalf;
        // the block's scales first (they came long ago), then its scores
        constexpr int kHG = kHalf / kGroup;  // groups of a half
        float ck[kHG], cm[kHG], rv[kHG];
        const bool scaled = h != 0 || mbar_wait_bounded(&bars->table_full[tb], (j / kTables) & 1, abort, wait_ns);
#pragma unroll
        for (int g = 0; g < kHG; ++g) {
          // not 0 (a row or a block of zeros), so that a masked score stays -inf
          ck[g] = fmaxf(bars->kc[tb][kHG * h + g] * cs, 1.17549435e-38f);
          cm[g] = bars->lv[tb][kHG * h + g];
          rv[g] = bars->rv[tb][kHG * h + g];
        }
        ok = __all_sync(0xffffffffu, scaled && mbar_wait_bounded(&bars->s_full[t][h], i & 1, abort, wait_ns));
        if (!ok) break;
        tc_fence_after_sync();
        float x[kHalf];
        {
          uint32_t r[2][32];
          tmem_ld32(tH, r[0]);
          tmem_ld32(tH + 32, r[1]);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < kHalf; ++e) x[e] = __uint_as_float(r[e >> 5][e & 31]);
        }
        if (j >= nb - 1 || win_rows) {  // the sequence's last prefix block, the tree's, or a window's first
          if (j == nb) {  // keys = the sequence's tree nodes; a padding row sees none
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bars->mask_full, 0, abort, wait_ns));
            if (!ok) break;
            const Ancestors* t = reinterpret_cast<const Ancestors*>(smem + C::kRawOff + bars->mask_slot * C::kRawBytes);
            const uint32_t am[2] = {has_row ? t->seen[node][2 * h] : 0u, has_row ? t->seen[node][2 * h + 1] : 0u};
#pragma unroll
            for (int e = 0; e < kHalf; ++e)
              if (!((am[e >> 5] >> (e & 31)) & 1u)) x[e] = -INFINITY;
          } else {
            const int shift = win_rows ? cut - (c.key_begin + j * kBlockN) - kHalf * h : 0;  // masked leading columns
            const int lim = (j == nb - 1 ? tail_end : kBlockN) - kHalf * h;                  // and from here on
#pragma unroll
            for (int e = 0; e < kHalf; ++e)
              if (e < shift || e >= lim) x[e] = -INFINITY;
          }
        }
        float mx = -INFINITY;
#pragma unroll
        for (int g = 0; g < kHG; ++g) {
          float m0 = fmax3(x[16 * g], x[16 * g + 1], x[16 * g + 2]), m1 = fmax3(x[16 * g + 3], x[16 * g + 4], x[16 * g + 5]);
#pragma unroll
          for (int e = 6; e < 14; e += 4) {
            m0 = fmax3(m0, x[16 * g + e], x[16 * g + e + 1]);
            m1 = fmax3(m1, x[16 * g + e + 2], x[16 * g + e + 3]);
          }
          m0 = fmax3(m0, x[16 * g + 14], x[16 * g + 15]);
          mx = fmaxf(mx, fmaf(fmaxf(m0, m1), ck[g], cm[g]));
        }
        const bool raise = mx > m + kRaise;
        const bool any_raise = __any_sync(0xffffffffu, raise);
        const float m_new = raise ? mx : m;
        // a row that has seen no visible key yet (a padding row of a tree-only chunk)
        // keeps m = -inf; its P is 0 against any finite reference
        const float m_off = (m_new == -INFINITY ? 0.f : m_new) - kOff;
#pragma unroll
        for (int g = 0; g < kHG; ++g) cm[g] -= m_off;
        if (any_raise) {
          // the maximum moved up: rescale what O_t and l hold. O_t is idle once the last
          // half's PV has completed (those before it precede S_t in the tensor core's order),
          // and this half's waits for this warpgroup's P. f = 1 where m is unchanged, 0
          // before the first half.
          const float f = m == m_new ? 1.f : ex2_approx(m - m_new);
          if (n > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bars->pv_done[t], (n - 1) & 1, abort, wait_ns));
            if (!ok) break;
            tc_fence_after_sync();
#pragma unroll
            for (int q = 0; q < D / 16; ++q) {
              uint32_t o[16];
              tmem_ld16(tO + 16 * q, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(tO + 16 * q, o);
            }
          }
          l *= f;
          m = m_new;
        }
        uint32_t pk[kHalf / 2];
        make_p(x, ck, cm, rv, pk, l);
        tmem_st32(tH, pk);  // over the half's scores
        tmem_wait_st();
        tc_fence_before_sync();
        mbar_arrive(&bars->p_full[t][h]);
      }
      // -------------------------------------------------------------- epilogue
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bars->o_full[t], 0, abort, wait_ns));
      // Each warpgroup stages its normalised 128 x D tile in shared memory as D/32 panels
      // of 128 rows x 128 B, swizzled like the tensor map (16-byte chunk q of row r at
      // q ^ (r & 7): conflict-free for the per-row writes), and one thread stores the
      // panels to o_part with TMA. Tile 0 finishes while tile 1's last PV may still read
      // V from the slot ring, so it stages over the Q tiles (every QK has completed by
      // o_full[0]); tile 1, last of all, stages over the ring. Rows past the unit's last
      // row are stored too: they stay inside the chunk's 256-row slot, which no one reads.
      const bool ok_all = bar_and(2 + t, 128, ok);
      if (ok_all) {
        tc_fence_after_sync();
        constexpr int kOPanels = D / 32;  // 128-byte panels of an fp32 row
        uint8_t* stage = smem + (t == 0 ? C::kQOff : C::kSlotOff);
        const float inv = 1.f / l;
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {  // panel q = columns [32 q, 32 q + 32)
          uint32_t r[32];
          tmem_ld32(tO + 32 * q, r);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4*>(stage + q * (128 * 128) + row * 128 + ((e ^ (row & 7)) << 4)) =
                make_float4(__uint_as_float(r[4 * e]) * inv, __uint_as_float(r[4 * e + 1]) * inv,
                            __uint_as_float(r[4 * e + 2]) * inv, __uint_as_float(r[4 * e + 3]) * inv);
        }
        // this tile's partial: rows [128 t, 128 t + 128) of the chunk's slot
        if (has_row) a.lse_part[(size_t)blockIdx.x * kUnitRows + t * 128 + row] = m - kOff + log2f(l);
        fence_proxy_async_smem();  // the staged tile is read by the TMA unit
        asm volatile("bar.sync %0, 128;" ::"r"(2 + t) : "memory");
        if ((warp & 3) == 0 && lane == 0 && (alt || t * 128 < rows_here)) {
#pragma unroll
          for (int q = 0; q < kOPanels; ++q)
            tma_store_2d(&P.tmap_o, stage + q * (128 * 128), 32 * q, (int)blockIdx.x * kUnitRows + t * 128);
          bulk_commit();
          bulk_wait_all();  // the shared memory must stay until the TMA has read it
        }
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tbase, C::kTmemCols);
  }
  if (tid == 0)
    a.chunk_status[blockIdx.x] = (bars->abort ? kErrTimeout : 0u) | (bars->tree_err ? kErrBadTree : 0u) | bars->dbg;
}

// The codes of K or V viewed as [rows][H_kv][D] bytes; boxes of box_rows rows of one head.
bool make_code_map(CUtensorMap* map, const void* base, int D, int Hkv, int64_t rows, int box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hkv, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)Hkv * D};
  cuuint32_t box[3] = {(cuuint32_t)D, 1, (cuuint32_t)box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(const Q8Args& a, cudaStream_t stream) {
  TcParams P;
  P.a = a;
  const int box_rows = a.kv.page_size < kBlockN ? a.kv.page_size : kBlockN;
  const int64_t rows = (int64_t)a.kv.num_pages * a.kv.page_size;
  if (!make_q_map(&P.tmap_q, a.q, D, a.p) || !make_code_map(&P.tmap_k, a.kv.k_pages, D, a.p.Hkv, rows, box_rows) ||
      !make_code_map(&P.tmap_v, a.kv.v_pages, D, a.p.Hkv, rows, box_rows) ||
      !make_o_map(&P.tmap_o, a.o_part, D, (int64_t)a.p.n_chunks * kUnitRows))
    return cudaErrorInvalidValue;
  const int smem = smem_need<D>();
  static bool configured[kMaxConfigured] = {};  // per template instance
  const cudaError_t e = configure_once(q8_tc_kernel<D>, smem, configured);
  if (e != cudaSuccess) return e;
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
  return cudaLaunchKernelEx(&cfg, q8_tc_kernel<D>, P);
}

}  // namespace

cudaError_t launch_q8_tc(const Q8Args& a, cudaStream_t stream) {
  if (a.p.n_chunks == 0) return cudaSuccess;
  return a.p.d == 64 ? launch<64>(a, stream) : launch<128>(a, stream);
}

}  // namespace ls
