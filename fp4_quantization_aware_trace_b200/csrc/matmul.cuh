// matmul.cuh -- the product of two captured FP4 operands, dense or grouped.
// Included by trace_fp4.cu inside its anonymous namespace.
//
// out[r, j] = s_a[g] s_w[g] sum_k a[r, k] w[g n + j, k], both operands E2M1
// codes with block scales along k.  The tensor core's block-scaled FP4
// instruction (tcgen05.mma, 64 k-elements each) multiplies codes and scales
// and accumulates in fp32 in tensor memory; the global scales are applied
// once, before the one rounding to bf16.
//
// The matrix w supplies the 128 rows (M) of a tile and the tokens its
// columns (N, a multiple of 16 up to 256): a group that ends inside a tile
// costs only the columns it has, and a decode batch is a narrow N instead of
// 128 mostly empty rows.  So the accumulator is transposed: lane = output
// column j, tensor-memory column = token.
//
// One persistent CTA per SM walks tiles; its warps are specialised:
//   warp 0      copies both operands' codes by TMA, 256 k-elements (128 bytes
//               per row, 128-byte swizzle) per stage of a shared-memory ring,
//               and tiled scales whose 128-row block is the tile's own;
//   warp 1      moves a stage's scales to tensor memory and issues its products;
//   warp 3      finds the CTA's tiles ahead of the others and posts them;
//   warps 4-11  read finished accumulators and write bf16 rows of out;
//   warps 12-15 copy all other scales into the ring in the 128 x 4 tiled order
//               the tensor core wants, from either layout and at any row (a
//               group starts anywhere), and zero what lies past the last k.
// Large products are done by pairs of CTAs (M = 256, N up to 256): each CTA
// copies its own rows of w and half of the tokens, so a stage moves 39 KB into
// an SM for 512 cycles of products and not 47 KB for 384.  Their scales all
// come by TMA, and warps 12-15 write out with the others.
//
// Tensor memory (512 columns) holds one accumulator of 256 or 192 tokens and 5
// or more stages of scales, or two accumulators of up to 128: of a large one the
// next tile's products wait until it has been read out (120 cycles of reads in a
// bubble of 1500), which costs less than two of 192 with only two stages of
// NVFP4 scales beside them (16384 x 4096 x 2048: 92 us).  The issuing warp's own
// instructions are what a stage costs besides: 12 copies of scales and 4
// products issue in 250 cycles if nothing is waited for in between.
//
// Measured, back to back in a graph (of 4 times the measured bf16 rate, or of
// the measured copy bandwidth):
//   16384 x 4096 x 2048 NVFP4                65 us   4.2 PFLOP/s, 0.64
//   4099 x 4096 x 4096 MXFP4                 28.2 us 4.9 PFLOP/s, 0.74
//   65536 x 1536 x 2048, 128 experts NVFP4   130 us  3.2 PFLOP/s, 0.59
//   512 x 1536 x 2048, 128 experts NVFP4     41 us   5.6 TB/s, 0.85
//   1 x 4096 x 4096 NVFP4                    7.0 us  one wave: launch and latency
// What bounds the large ones: the tensor core is busy a little over half of the
// time; reading an accumulator out, and the traffic of the output beside that of
// the operands, take the rest (without any output 16384 x 4096 x 2048 takes 45
// us).  With calls back to back for a second the 1 kW limit lowers the clock to
// 1.6 GHz and the first takes 78 us.
#pragma once

constexpr int kMmThreads = 512;
constexpr int kMmM = 128;            // w rows of a tile
constexpr int kMmStageBytes = 128;   // code bytes per row and stage: 256 elements
constexpr int kMmMaxStages = 8;
constexpr uint32_t kMmTurnPiece = 16 * 32 * 2;        // an output piece: 16 tokens x 32 columns
constexpr uint32_t kMmTurnBytes = 12 * kMmTurnPiece;  // one for each of up to 12 warps
constexpr uint32_t kMmBox = 32 * 32 * 2;             // 32 rows x 32 columns of out, for each of 12 warps
// CTAs that share a tile's k: clusters of 8 take 5 us longer to launch than
// clusters of 4 (29 x 2048 x 4096: 12.9 us with 8, 7.6 with 4, 10.7 with 1).
constexpr uint32_t kMmMaxSplit = 4;
constexpr uint32_t kMmTokens = 192, kMmPairTokens = 256;  // of the largest tiles
constexpr uint32_t kMmPairBox = kMmPairTokens / 4;        // token rows a CTA of a pair copies at a time
constexpr uint32_t kMmTmemCols = 512;
// Polls of one wait before a CTA gives up (each try_wait itself suspends):
// a guard, every wait ends as its copies and products do.
constexpr uint32_t kMmPolls = 1u << 20;

struct MmShape {
  int64_t rows, n;
  uint32_t cols, scols;        // k-elements, scale columns
  int32_t groups, matrices;
  uint32_t nt;                 // tokens of a full tile (multiple of 16)
  uint32_t n_tiles;            // ceil(n / 128), of pairs ceil(n / 256)
  uint32_t w_blocks;           // ceil(n / 128): of pairs, a matrix's 128-row blocks of scales
  uint32_t ksteps;             // stages of a whole product
  uint32_t stages, accs, sf_slots;
  uint32_t n_lo, step_hi, step_lo;  // see MmWalk; from one of a CTA's (a team's) tiles to its next
  uint32_t split;              // CTAs of a cluster that share one tile's k (1: none)
  uint8_t a_tiled, w_tiled;
  uint8_t a_bytes, w_bytes;    // row-major scales that are not 4-byte words
};

__device__ uint32_t g_matmul_gave_up;  // counts waits that ran out of polls; never cleared

// The product of two global scales as m * p * q, |m| in [1, 2) and p, q powers
// of two: ga * gw itself may leave fp32's range where sum * ga * gw does not
// (a small activation against a large weight).  |sum| is 0 or in
// [2^-20, 2^54], so with the exponents halved no step over- or underflows
// unless the result does; past +-250 the result is 0 or infinite anyway.
// Exponents within +-60 leave nothing to lose: one factor then, the same bits.
struct OutScale {
  float m, p, q;
  bool one;  // p and q are 1
  __device__ __forceinline__ float apply(float sum) const {
    return one ? sum * m : ((sum * m) * p) * q;
  }
};

// 16 sums of a lane to bf16 pairs.
template <bool MX>
__device__ __forceinline__ void scaled_bf16(const uint32_t* v, const OutScale& s, uint32_t* w) {
  if (MX || s.one) {
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      float lo = __uint_as_float(v[2 * x]), hi = __uint_as_float(v[2 * x + 1]);
      if (!MX) lo *= s.m, hi *= s.m;
      w[x] = cvt_bf16x2(lo, hi);
    }
  } else {
#pragma unroll
    for (int x = 0; x < 8; ++x)
      w[x] = cvt_bf16x2(s.apply(__uint_as_float(v[2 * x])), s.apply(__uint_as_float(v[2 * x + 1])));
  }
}

__device__ __forceinline__ OutScale make_out_scale(float ga, float gw) {
  const double d = (double)ga * (double)gw;  // exact
  OutScale s{(float)d, 1.0f, 1.0f, true};
  int e = ((__double2hiint(d) >> 20) & 0x7FF) - 1023;
  if (e == -1023 || e == 1024 || (e >= -60 && e <= 60)) return s;  // zero or not finite, or plain
  s.one = false;
  s.m = (float)__hiloint2double((__double2hiint(d) & 0x800FFFFF) | (1023 << 20), __double2loint(d));
  e = max(-252, min(e, 250));
  s.p = __int_as_float((e / 2 + 127) << 23);
  s.q = __int_as_float((e - e / 2 + 127) << 23);
  return s;
}

// ---------------------------------------------------------------------------
// Instructions
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}

// The same shared-memory address in another CTA of the cluster.
__device__ __forceinline__ uint32_t peer_smem(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// Only what tcgen05 instructions read or wrote hangs on this arrival (a
// cluster-scope release would order memory that nobody shares, and cost more
// than a stage's products).
__device__ __forceinline__ void mbar_arrive_peer(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float ld_peer(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// Every thread of every CTA of the cluster, with its earlier writes seen.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// One lane of a converged warp; ptxas knows that a branch on it leaves a
// single thread and keeps the operands of what it issues in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0u;
}

// A value that every lane of a warp holds, said to be so: what the tensor core
// and the copy engine are given has to be in uniform registers.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// Up to 256 polls for a phase to end.
__device__ __forceinline__ bool mbar_poll(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 c;\n\tmov.u32 c, 256;\n\t"
      "again:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra over;\n\tsub.u32 c, c, 1;\n\tsetp.ne.u32 q, c, 0;\n\t@q bra again;\n\t"
      "over:\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0u;
}

// Whether a phase has ended, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0u;
}

// Bounded wait of a warp for a phase (lanes may name different barriers);
// false once any wait of the CTA has given up.  60 cycles where the phase has
// ended, against 90 of a loop over single polls.
__device__ __forceinline__ bool mm_wait(uint32_t bar, uint32_t parity, volatile uint32_t* gave_up) {
  for (uint32_t i = 0; i < kMmPolls / 256u; ++i) {
    if (__all_sync(0xFFFFFFFFu, mbar_poll(bar, parity))) return true;
    if (__any_sync(0xFFFFFFFFu, *gave_up != 0u)) break;
  }
  *gave_up = 1u;
  if (threadIdx.x % 32u == 0u) atomicAdd(&g_matmul_gave_up, 1u);
  return false;
}

__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// CG 2: `bar` may lie in the other CTA of the pair.
template <int CG>
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int32_t x,
                                            int32_t y, uint32_t bar) {
  if (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Shared memory to a box of a tensor; rows and columns outside it are not
// written.  The thread that issues waits for its stores to have been read.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int32_t x,
                                             int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   map),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// A contiguous copy, counted on the stage's barrier (whose expected bytes
// include it); addresses and size are multiples of 16.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// `bytes` <= 4 of a word; the rest of it becomes zero.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

// Shared-memory matrix descriptors: codes with 128-byte rows in the 128-byte
// swizzle (8-row groups 1024 bytes apart); scales as 32 rows of 16 bytes
// (8-row groups 128 bytes apart, no swizzle).  The upper words are constants,
// the lower ones hold the address in 16-byte units.
constexpr uint32_t kCodeDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kScaleDescHigh = (128u >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t code_desc(uint32_t smem) {
  return ((smem & 0x3FFFFu) >> 4) | (1u << 16);
}
__device__ __forceinline__ uint32_t scale_desc(uint32_t smem) { return (smem & 0x3FFFFu) >> 4; }

// Instruction descriptor: E2M1 x E2M1, K-major, M = 128 per CTA, N = n; the
// scale type (the ids of the bytes used in a scale word are added later).
template <bool MX, int CG>
__device__ __forceinline__ uint32_t mm_idesc(uint32_t n) {
  return (1u << 7) | (1u << 10) | ((n >> 3) << 17) | (MX ? 1u << 23 : 0u) |
         ((CG * 128u >> 4) << 24);
}

// Columns of a product of `tokens` tokens: whole 16s in each CTA's share.
template <int CG>
__device__ __forceinline__ uint32_t mm_width(uint32_t tokens) {
  return (tokens + 16u * CG - 1u) / (16u * CG) * (16u * CG);
}

// D += A B on one CTA's tensor core or (CG 2) on a pair's: each CTA then
// holds its 128 rows of A, half the rows of B, and its rows of D.
#define TRACE_MMA_FP4(GROUP, KIND, VEC)                                                       \
  asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %6, 0;\n\t"           \
               "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"                            \
               "tcgen05.mma.cta_group::" GROUP ".kind::" KIND ".block_scale.scale_vec::" VEC   \
               " [%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(d),                               \
               "r"(a), "r"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)add),               \
               "n"(kCodeDescHigh)                                                              \
               : "memory")
template <bool MX, int CG>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                        uint32_t sa, uint32_t sb, bool add) {
  if (MX && CG == 1) TRACE_MMA_FP4("1", "mxf4", "2X");
  if (MX && CG == 2) TRACE_MMA_FP4("2", "mxf4", "2X");
  if (!MX && CG == 1) TRACE_MMA_FP4("1", "mxf4nvf4", "4X");
  if (!MX && CG == 2) TRACE_MMA_FP4("2", "mxf4nvf4", "4X");
}
#undef TRACE_MMA_FP4

// 512 bytes of scales to 4 columns of tensor memory (CG 2: each CTA of the
// pair its own).
template <int CG>
__device__ __forceinline__ void scales_to_tmem(uint32_t tmem, uint32_t desc) {
  if (CG == 1)
    asm volatile("{\n\t.reg .b64 a;\n\tmov.b64 a, {%1, %2};\n\t"
                 "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], a;\n\t}" ::"r"(tmem),
                 "r"(desc), "n"(kScaleDescHigh)
                 : "memory");
  else
    asm volatile("{\n\t.reg .b64 a;\n\tmov.b64 a, {%1, %2};\n\t"
                 "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], a;\n\t}" ::"r"(tmem),
                 "r"(desc), "n"(kScaleDescHigh)
                 : "memory");
}

// The barrier's phase ends when every product and copy issued so far by this
// thread has (CG 2: the barrier at this address in both CTAs).
template <int CG>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  if (CG == 1)
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

// 32 lanes x 16 columns of an accumulator: a lane's row (output column) and 16
// tokens.  (All of a tile in 120 cycles; in the shape that a transposing store
// takes, 16 lanes x 256 bits, 420.)
__device__ __forceinline__ void tmem_ld_32x16(uint32_t addr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(addr));
}

// Every load so far has arrived; no use of the words moves in front of the
// wait, through which they pass.
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_arrived(uint32_t* v) {
  asm volatile(""
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                 "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                 "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])::"memory");
}

// A position in a ring of `size` slots and the parity of its current round.
struct Ring {
  uint32_t at = 0, parity = 0;
  __device__ __forceinline__ void next(uint32_t size) {
    if (++at == size) {
      at = 0;
      parity ^= 1u;
    }
  }
};

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------
// `first_tile[g]`: token tiles before group g.  A tile number counts token
// tiles, and w tiles within one: neighbours share their tokens, and the CTAs
// that run at a time share one or a few groups' matrices in L2.
struct MmTile {
  int32_t group;
  int64_t row0;       // first token row
  uint32_t lead;      // rows in front that belong to earlier groups
  uint32_t tokens;    // rows up to the group's last in this tile
  uint32_t j0;        // first output column
  bool product;       // false: a group without a matrix, its rows are zero
  bool end;           // behind the last tile
};

// Offsets are clamped to the rows there are, whatever they hold.  One group may
// have some too: a batch padded around it.
__device__ __forceinline__ int64_t mm_bound(const int64_t* offs, int32_t g, const MmShape& sh) {
  if (offs == nullptr) return g == 0 ? 0 : sh.rows;
  const int64_t v = offs[g];
  return v < 0 ? 0 : (v > sh.rows ? sh.rows : v);
}

// The row that a group's tiles are counted from: a pair's lie at multiples of
// 128 (and the first begins at a multiple of 64), so that the copy engine can
// take tiled scales as they are, at most two blocks for a tile.
template <int CG>
__device__ __forceinline__ int64_t mm_start(int64_t bound) {
  return CG == 2 ? bound & ~(int64_t)127 : bound;
}

// A CTA's walk over its tiles without a division per tile: neighbours differ in
// `lo`, the w tile (of transposed products, the token tile).
struct MmWalk {
  uint32_t hi, lo, d_hi, d_lo, n_lo;
  __device__ __forceinline__ MmWalk(uint32_t t0, const MmShape& sh)
      : hi(t0 / sh.n_lo), d_hi(sh.step_hi), d_lo(sh.step_lo), n_lo(sh.n_lo) {
    lo = t0 - hi * n_lo;
  }
  __device__ __forceinline__ void next() {
    hi += d_hi;
    lo += d_lo;
    if (lo >= n_lo) {
      lo -= n_lo;
      ++hi;
    }
  }
};

// For a converged warp: with several groups its lanes search the table
// together, 32 entries at a time.
template <int CG>
__device__ __forceinline__ MmTile mm_tile(uint32_t tt, uint32_t jt, const uint32_t* first_tile,
                                          const int64_t* offs, const MmShape& sh) {
  MmTile m;
  uint32_t lo = 0;  // the last group that starts at or before tt
  for (uint32_t span = (uint32_t)sh.groups; span > 1u;) {
    const uint32_t step = (span + 31u) / 32u, probe = threadIdx.x % 32u * step;
    const bool in = probe < span && first_tile[lo + probe] <= tt;
    const uint32_t skip = (__popc(__ballot_sync(0xFFFFFFFFu, in)) - 1u) * step;
    lo += skip;
    span = min(step, span - skip);
  }
  m.group = (int32_t)lo;
  const int64_t begin = mm_bound(offs, m.group, sh);
  const uint32_t first = sh.groups > 1 ? first_tile[lo] : 0u;
  const int64_t from = mm_start<CG>(begin) + (int64_t)(tt - first) * sh.nt;
  m.row0 = CG == 2 && begin - from >= 64 ? from + 64 : from;
  m.lead = begin > m.row0 ? (uint32_t)(begin - m.row0) : 0u;
  const int64_t end = mm_bound(offs, m.group + 1, sh), to = end < from + sh.nt ? end : from + sh.nt;
  // (no tile of a valid table is empty; one of offsets that go down could be)
  m.tokens = from >= 0 && to > m.row0 ? (uint32_t)(to - m.row0) : 0u;
  m.j0 = jt * (CG * kMmM);
  m.product = m.group < sh.matrices && m.tokens > 0u;
  m.end = false;
  return m;
}

// One warp finds the CTA's tiles ahead of the others (a tile's group, its bounds
// and global scales are some 1000 cycles of dependent loads) and posts them.
constexpr uint32_t kMmPosts = 3;
struct MmPosts {
  MmTile tile[kMmPosts];
  OutScale scale[kMmPosts];
  u64 posted[kMmPosts], taken[kMmPosts];
};

// The next posted tile, for a warp; false behind the last one (or when the CTA
// has given up).
__device__ __forceinline__ bool mm_next(Ring* at, MmPosts* posts, MmTile* m, OutScale* scale,
                                        volatile uint32_t* gave_up) {
  if (!mm_wait(smem_u32(&posts->posted[at->at]), at->parity, gave_up)) return false;
  *m = posts->tile[at->at];
  if (scale != nullptr) *scale = posts->scale[at->at];
  __syncwarp();
  if (threadIdx.x % 32u == 0u) mbar_arrive(smem_u32(&posts->taken[at->at]));
  at->next(kMmPosts);
  return !m->end;
}

// first_tile[0 .. groups] by a scan over the CTA.
template <int CG>
__device__ __forceinline__ void mm_table(uint32_t* first_tile, uint32_t* warp_sum,
                                         const int64_t* offs, const MmShape& sh) {
  const uint32_t lane = threadIdx.x % 32u, warp = threadIdx.x / 32u;
  uint32_t carry = 0u;
  for (int32_t g0 = 0; g0 < sh.groups; g0 += kMmThreads) {
    const int32_t g = g0 + (int32_t)threadIdx.x;
    uint32_t tiles = 0u;
    if (g < sh.groups) {
      const int64_t begin = mm_bound(offs, g, sh), end = mm_bound(offs, g + 1, sh);
      if (end > begin) tiles = (uint32_t)((end - mm_start<CG>(begin) + sh.nt - 1) / sh.nt);
    }
    uint32_t sum = tiles;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= (uint32_t)d) sum += v;
    }
    if (lane == 31u) warp_sum[warp] = sum;
    __syncthreads();
    uint32_t base = carry, all = 0u;
    for (uint32_t w = 0; w < kMmThreads / 32; ++w) {
      if (w < warp) base += warp_sum[w];
      all += warp_sum[w];
    }
    if (g < sh.groups) first_tile[g] = base + sum - tiles;
    carry += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) first_tile[sh.groups] = carry;
  __syncthreads();
}

// ---------------------------------------------------------------------------
// Scales of one 128-row block for one stage: ATOMS pieces of 512 bytes (128
// rows x 4 scale columns), `apart` bytes from one to the next.  Each of the
// four scale warps copies a quarter of the rows, one 4-byte word per lane and
// piece.
// ---------------------------------------------------------------------------
struct ScaleSrc {
  const uint8_t* row;  // this lane's row (null: past the array's end)
  uint32_t step;       // bytes from one group of 4 columns to the next
  bool bulk;           // the block is one of the tiled layout's own: TMA's work
  bool bytes;          // rows without 4-byte alignment
};

// Whether the copy engine takes stage k of a block: 512-byte pieces as they
// are, none of them with columns past the last.
__device__ __forceinline__ bool scales_bulk(bool tiled, int64_t row0) {
  return tiled && row0 % 128 == 0;
}

__device__ __forceinline__ ScaleSrc scale_src(const uint8_t* base, bool tiled, bool bytes,
                                              int64_t row0, int64_t rows, uint32_t scols,
                                              uint32_t quarter, uint32_t lane) {
  ScaleSrc s;
  s.bytes = bytes;
  s.step = tiled ? 512u : 4u;
  s.bulk = scales_bulk(tiled, row0);
  const uint32_t ct = (scols + 3u) / 4u;
  const int64_t r = row0 + 32u * quarter + lane;
  s.row = r >= rows ? nullptr
          : tiled   ? base + (size_t)(r / 128) * ct * 512u + (size_t)(r % 32) * 16u +
                        (size_t)(r % 128 / 32) * 4u
                    : base + (size_t)r * scols;
  return s;
}

// `at`: this lane's word of the first piece.
template <int ATOMS>
__device__ __forceinline__ void copy_scales(const ScaleSrc& s, const uint8_t* base, uint32_t at,
                                            uint32_t apart, uint32_t k, uint32_t scols) {
  const uint32_t c0 = k * (4u * ATOMS);
  if (c0 + 4u * ATOMS <= scols && !s.bytes) {
    if (s.bulk || s.row == nullptr) return;  // rows past the end reach no output
    const uint8_t* from = s.row + (size_t)(k * ATOMS) * s.step;
#pragma unroll
    for (uint32_t j = 0; j < (uint32_t)ATOMS; ++j) cp_async4(at + j * apart, from + j * s.step, 4u);
    return;
  }
  for (uint32_t j = 0; j < (uint32_t)ATOMS; ++j) {
    const uint32_t c = c0 + 4u * j;
    const uint32_t take = s.row == nullptr || c >= scols ? 0u : min(4u, scols - c);
    if (!s.bytes) {
      cp_async4(at + j * apart, take ? s.row + (size_t)(c / 4u) * s.step : base, take);
    } else {
      uint32_t w = 0u;
      for (uint32_t i = 0; i < take; ++i) w |= (uint32_t)s.row[c + i] << (8u * i);
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + j * apart), "r"(w) : "memory");
    }
  }
}

// ---------------------------------------------------------------------------
// The kernel.  RB: 128-row blocks of token scales (1 up to 128 tokens, else
// 2).  CG: CTAs that share a tile.  With CG 2 a pair holds 256 rows of w and
// the same tokens: each CTA copies its own 128 rows of w, half of the tokens'
// codes and all of their scales, every part by TMA and counted on the leader's
// barrier, and the leader's warp 1 issues for both.
//   TR (pairs, one group without offsets, rows of out in whole 16 bytes): called with the operands
// exchanged, so the "tokens" of these comments are columns of out and the rows
// of w its rows.  A lane then holds 16 columns of a row and not 16 rows of a
// column, nothing has to be turned, and a warp hands 32 x 32 of them to the copy
// engine (65536 x 2048 x 256: 52 us, 72 without; 16384 x 4096 x 2048: 65 and 67).
// Not for several groups, whose tiles end at any row.
//   W16: rows of out are whole 16 bytes.  Others are written in words of two
// columns where a piece is whole and k is not long, else one column at a time.
// That is bound by the instructions (45231 x n x 224, 4 experts: 104 us with n =
// 2446 and 117 with 2447, 67 with 2448; one column at a time 136.  65536 x 1534 x
// 2048, 32 experts: 128 and 140; 4099 x 4001 x 4096, where the stores come beside
// the next tile's products: 37.6 and 36.6).  Kernels of their own, because the
// registers of both would not fit one: as it is, all of them use up to 128 without
// spills but the NVFP4 pairs with rows not in whole 16 bytes, which spill 8 bytes
// (28 of loads).
// ---------------------------------------------------------------------------
struct MmMaps {
  CUtensorMap a, w;    // codes
  CUtensorMap as, ws;  // CG 2: tiled scales, a row per 128-row block
  CUtensorMap out;     // TR
};

template <bool MX, int RB, int CG, bool TR, bool W16>
__global__ void __launch_bounds__(kMmThreads, 1)
    k_matmul(const __grid_constant__ MmMaps maps, const uint8_t* __restrict__ as,
             const uint8_t* __restrict__ ws, const float* __restrict__ ag,
             const float* __restrict__ wg, const int64_t* __restrict__ offs, MmShape sh,
             uint16_t* __restrict__ out) {
  constexpr uint32_t ATOMS = MX ? 2 : 4;  // groups of 4 scale columns per stage
  constexpr uint32_t w_code = kMmM * kMmStageBytes;
  constexpr uint32_t block_bytes = ATOMS * 512u;  // a block's scales per stage
  constexpr bool PAIR = CG == 2;
  constexpr uint32_t OUT = PAIR ? 3u : 2u;  // warps that write out, per quarter of a tile's rows
  constexpr uint32_t PIECES = ((PAIR ? kMmPairTokens : RB == 2 ? kMmTokens : 128u) / 16u + OUT - 1u) / OUT;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) u64 full[kMmMaxStages], empty[kMmMaxStages], acc_full[2], acc_empty[2];
  __shared__ __align__(8) MmPosts posts;
  __shared__ uint32_t tmem_base_s, warp_sum[kMmThreads / 32];
  __shared__ volatile uint32_t gave_up;
  const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32u, 0), lane = threadIdx.x % 32u;
  const uint32_t x_code = sh.nt / CG * kMmStageBytes;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t stage_at = (w_code + x_code + block_bytes * (1u + RB) + 1023u) & ~1023u;
  uint8_t* ring_p = smem_raw + (ring - smem_u32(smem_raw));
  uint8_t* after = ring_p + sh.stages * stage_at;  // pieces being turned, the table
  uint32_t* first_tile = reinterpret_cast<uint32_t*>(after + kMmTurnBytes);
  const uint32_t rank = cluster_rank();  // in a pair, or among the CTAs of a split

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < sh.stages; ++s) {
      // the TMA thread, and the scale lanes
      mbar_init(smem_u32(&full[s]), PAIR ? 1 : 1 + 128);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (uint32_t a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&acc_full[a]), 1);
      mbar_init(smem_u32(&acc_empty[a]), 4 * OUT * CG);
    }
    for (uint32_t a = 0; a < kMmPosts; ++a) {
      mbar_init(smem_u32(&posts.posted[a]), 1);
      // the warps that copy, that issue and that write out
      mbar_init(smem_u32(&posts.taken[a]), 1 + (PAIR ? (rank == 0 ? 1 : 0) : 1 + 4) + 4 * OUT);
    }
    gave_up = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0 && elect_one()) {
    tma_prefetch_map(&maps.w);
    tma_prefetch_map(&maps.a);
    if (PAIR) tma_prefetch_map(&maps.ws), tma_prefetch_map(&maps.as);
    if (TR) tma_prefetch_map(&maps.out);
  }
  if (warp == 1) {
    if (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(&tmem_base_s)),
                   "r"(kMmTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(&tmem_base_s)),
                   "r"(kMmTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (PAIR) cluster_sync();  // the other CTA's barriers exist
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  pdl_begin();  // nothing before this read or wrote what another kernel may
  uint32_t token_tiles = (uint32_t)((sh.rows + sh.nt - 1) / sh.nt);
  if (sh.groups > 1) {
    mm_table<CG>(first_tile, warp_sum, offs, sh);
    token_tiles = first_tile[sh.groups];
  }
  const uint32_t tmem = uniform(tmem_base_s);
  const uint32_t acc_cols = (sh.nt + 31u) & ~31u;
  constexpr uint32_t sf_cols = 4u * ATOMS * (1u + RB);  // tensor-memory columns of a stage's scales
  const uint32_t sf_base = tmem + sh.accs * acc_cols;
  // this CTA's part of k
  const uint32_t team = PAIR ? 2u : sh.split;
  const uint32_t k_rank = PAIR ? 0u : rank;
  const uint32_t k0 = k_rank * sh.ksteps / sh.split, k1 = (k_rank + 1u) * sh.ksteps / sh.split;
  const uint32_t j_rank = PAIR ? rank * kMmM : 0u;

  if (warp == 0) {
    Ring r;
    r.parity = 1u;  // the first round finds every slot empty
    bool ok = true;
    const uint32_t c4s = (sh.scols + 3u) / 4u, bulk_steps = sh.scols / (4u * ATOMS);
    MmTile m;
    Ring next;
    while (ok && mm_next(&next, &posts, &m, nullptr, &gave_up)) {
      if (!m.product) continue;
      const int64_t wr = m.group * sh.n + m.j0 + j_rank;
      const int32_t w_row = (int32_t)uniform((uint32_t)wr);
      if (PAIR) {
        // blocks of 128 rows that the tile's scales lie in
        const uint32_t width = mm_width<CG>(m.tokens);
        const bool two = (uint32_t)(m.row0 % 128) + width > 128u;
        const int32_t wb = (int32_t)uniform((uint32_t)m.group * sh.w_blocks + (m.j0 + j_rank) / 128u);
        const int32_t row = (int32_t)uniform((uint32_t)m.row0), xb = row / 128;
        const int32_t xr = row + (int32_t)uniform(rank * (width / 2u));
        // token codes in boxes of 64 rows, as many as the tile has
        const bool more = width / 2u > kMmPairBox;
        const uint32_t bytes = 2u * (w_code + (more ? 2u : 1u) * kMmPairBox * kMmStageBytes +
                                     (two ? 3u : 2u) * block_bytes);
        for (uint32_t k = 0; k < sh.ksteps; ++k, r.next(sh.stages)) {
          const uint32_t at = uniform(ring + r.at * stage_at), sc = at + w_code + x_code;
          const uint32_t own = smem_u32(&full[r.at]), bar = peer_smem(own, 0);
          if (!(ok = mm_wait(smem_u32(&empty[r.at]), r.parity, &gave_up))) break;
          if (!elect_one()) continue;
          if (rank == 0) mbar_expect(own, bytes);
          tma_load_2d<CG>(at, &maps.w, (int32_t)(k * kMmStageBytes), w_row, bar);
          tma_load_2d<CG>(at + w_code, &maps.a, (int32_t)(k * kMmStageBytes), xr, bar);
          if (more)
            tma_load_2d<CG>(at + w_code + kMmPairBox * kMmStageBytes, &maps.a,
                            (int32_t)(k * kMmStageBytes), xr + (int32_t)kMmPairBox, bar);
          tma_load_2d<CG>(sc, &maps.ws, (int32_t)(k * ATOMS * 64u), wb, bar);
          tma_load_2d<CG>(sc + block_bytes, &maps.as, (int32_t)(k * ATOMS * 64u), xb, bar);
          if (two)
            tma_load_2d<CG>(sc + 2u * block_bytes, &maps.as, (int32_t)(k * ATOMS * 64u), xb + 1,
                            bar);
        }
        continue;
      }
      const bool w_bulk = scales_bulk(sh.w_tiled, wr) && wr < sh.n * sh.matrices;
      const bool x_bulk = scales_bulk(sh.a_tiled, m.row0);
      const bool two = RB == 2 && m.tokens > 128u;
      const uint8_t* w_from = ws + (size_t)(wr / 128) * c4s * 512u;
      const uint8_t* x_from = as + (size_t)(m.row0 / 128) * c4s * 512u;
      const uint32_t bulk_bytes = (w_bulk ? block_bytes : 0u) +
                                  (x_bulk ? (two ? 2u : 1u) * block_bytes : 0u);
      for (uint32_t k = k0; k < k1; ++k, r.next(sh.stages)) {
        const uint32_t bar = smem_u32(&full[r.at]), at = uniform(ring + r.at * stage_at);
        if (!(ok = mm_wait(smem_u32(&empty[r.at]), r.parity, &gave_up))) break;
        if (!elect_one()) continue;
        const bool bulk = k < bulk_steps;
        mbar_expect(bar, w_code + x_code + (bulk ? bulk_bytes : 0u));
        tma_load_2d<CG>(at, &maps.w, (int32_t)(k * kMmStageBytes), w_row, bar);
        tma_load_2d<CG>(at + w_code, &maps.a, (int32_t)(k * kMmStageBytes), (int32_t)m.row0, bar);
        if (bulk) {
          const uint32_t sc = at + w_code + x_code;
          if (w_bulk) bulk_copy(sc, w_from + (size_t)k * block_bytes, block_bytes, bar);
          if (x_bulk) {
            bulk_copy(sc + block_bytes, x_from + (size_t)k * block_bytes, block_bytes, bar);
            if (two)
              bulk_copy(sc + 2u * block_bytes, x_from + (size_t)c4s * 512u + (size_t)k * block_bytes,
                        block_bytes, bar);
          }
        }
      }
    }
    if (gave_up)  // let the copies in flight land before the CTA leaves
      for (int z = 0; z < 1000; ++z) __nanosleep(1000);
  } else if (warp >= 12 && !PAIR) {
    const uint32_t quarter = warp - 12u;
    Ring r;
    r.parity = 1u;
    bool ok = true;
    MmTile m;
    Ring next;
    while (ok && mm_next(&next, &posts, &m, nullptr, &gave_up)) {
      if (!m.product) continue;
      const int64_t wr = m.group * sh.n + m.j0 + j_rank;
      const ScaleSrc sw = scale_src(ws, sh.w_tiled, sh.w_bytes, wr, sh.n * sh.matrices, sh.scols,
                                    quarter, lane);
      const ScaleSrc s0 = scale_src(as, sh.a_tiled, sh.a_bytes, m.row0, sh.rows, sh.scols, quarter,
                                    lane);
      const bool two = RB == 2 && m.tokens > 128u;
      const ScaleSrc s1 = scale_src(as, sh.a_tiled, sh.a_bytes, m.row0 + 128, sh.rows, sh.scols,
                                    quarter, lane);
      const uint32_t word = w_code + x_code + 16u * lane + 4u * quarter;
      for (uint32_t k = k0; k < k1; ++k, r.next(sh.stages)) {
        if (!(ok = mm_wait(smem_u32(&empty[r.at]), r.parity, &gave_up))) break;
        const uint32_t at = ring + r.at * stage_at + word, bar = smem_u32(&full[r.at]);
        copy_scales<ATOMS>(sw, ws, at, 512u, k, sh.scols);
        // rows past the tile's last token reach no output
        if (32u * quarter < m.tokens)
          copy_scales<ATOMS>(s0, as, at + block_bytes, 512u, k, sh.scols);
        if (two && 128u + 32u * quarter < m.tokens)
          copy_scales<ATOMS>(s1, as, at + 2u * block_bytes, 512u, k, sh.scols);
        if (sw.bytes || s0.bytes) {  // plain stores: nothing that arrives by itself
          asm volatile("cp.async.wait_all;" ::: "memory");
          mbar_arrive(bar);
        } else {
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar)
                       : "memory");
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 1 && (!PAIR || rank == 0)) {
    Ring r, acc, sf, sf_last;  // sf_last: the stage that used the scale slot before
    acc.parity = 1u;
    uint32_t begun = 0;  // scale slots used so far, up to sf_slots
    const bool sf_wait = sh.sf_slots < sh.stages;
    // What a stage has to wait for: that it is full, and that the scale slot's
    // last reader is done; half of the lanes wait for each (with a slot for
    // every stage the first says the second).  The next stage's barriers are
    // tested before this stage's instructions are issued, so that the answer
    // has arrived when they have been.
    uint32_t bar = smem_u32(&full[0]), parity = 0u;
    bool ok = true, ready = false, any = false;
    uint32_t at = ring, freed = 0u, freed_parity = 0u;
    MmTile m;
    Ring next;
    while (ok && mm_next(&next, &posts, &m, nullptr, &gave_up)) {
      if (!m.product) continue;
      const uint32_t width = uniform(mm_width<CG>(m.tokens));
      const uint32_t d = uniform(tmem + acc.at * acc_cols), idesc = mm_idesc<MX, CG>(width);
      // tokens that start in the middle of a block: two columns of scales on
      const uint32_t shift = PAIR ? uniform((uint32_t)(m.row0 % 128) / 32u) : 0u;
      if (!(ok = mm_wait(smem_u32(&acc_empty[acc.at]), acc.parity, &gave_up))) break;
      for (uint32_t k = k0; k < k1; ++k) {
        if (!__all_sync(0xFFFFFFFFu, ready)) ok = ok && mm_wait(bar, parity, &gave_up);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        // scales written by cp.async and plain stores: seen by the copies below
        if (!PAIR) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        const uint32_t sa = sf_base + sf.at * sf_cols, sb = sa + 4u * ATOMS;
        const uint32_t sd = scale_desc(at + w_code + x_code);
        const uint32_t da = code_desc(at), db = code_desc(at + w_code);
        const uint32_t left = sh.cols - k * 256u, more = k - k0;
        freed = smem_u32(&empty[r.at]), freed_parity = r.parity;
        any = true;
        r.next(sh.stages);
        sf.next(sh.sf_slots);
        at = r.at == 0u ? ring : at + stage_at;
        bar = smem_u32(&full[r.at]), parity = r.parity;
        if (sf_wait && ++begun >= sh.sf_slots) {
          if (lane >= 16u) bar = smem_u32(&empty[sf_last.at]), parity = sf_last.parity;
          sf_last.next(sh.stages);
        }
        ready = mbar_test(bar, parity);
        if (elect_one()) {
          // A second block that the tile does not reach is copied all the same:
          // into columns that no product reads.
#pragma unroll
          for (uint32_t j = 0; j < ATOMS; ++j) {
            scales_to_tmem<CG>(sa + 4u * j, sd + 32u * j);
            scales_to_tmem<CG>(sb + 4u * RB * j, sd + 32u * (ATOMS + j));
            if (RB == 2) scales_to_tmem<CG>(sb + 4u * (RB * j + 1u), sd + 32u * (2u * ATOMS + j));
          }
          if (left >= 256u) {
#pragma unroll
            for (uint32_t j = 0; j < 4u; ++j) {
              const uint32_t c = MX ? j / 2u : j;  // piece with this product's scales
              const uint32_t id = MX ? (j & 1u) * 2u : 0u;
              mma_fp4<MX, CG>(d, da + 2u * j, db + 2u * j, idesc | (id << 4) | (id << 29),
                              sa + 4u * c, sb + 4u * RB * c + shift, j > 0u || more > 0u);
            }
          } else {  // the end of k, 64 elements at a time
#pragma unroll 1
            for (uint32_t j = 0; 64u * j < left; ++j) {
              const uint32_t c = MX ? j / 2u : j;
              const uint32_t id = MX ? (j & 1u) * 2u : 0u;
              mma_fp4<MX, CG>(d, da + 2u * j, db + 2u * j, idesc | (id << 4) | (id << 29),
                              sa + 4u * c, sb + 4u * RB * c + shift, j > 0u || more > 0u);
            }
          }
          mma_commit<CG>(freed);
        }
      }
      if (!ok) break;
      if (elect_one()) mma_commit<CG>(smem_u32(&acc_full[acc.at]));
      acc.next(sh.accs);
    }
    // the products in flight must end before tensor memory is freed
    if (any) mm_wait(freed, freed_parity, &gave_up);
  } else if (warp == 3) {
    Ring at;
    at.parity = 1u;
    for (MmWalk t(blockIdx.x / team, sh);; t.next()) {
      MmTile m;
      m.end = t.hi >= (TR ? sh.n_tiles : token_tiles);
      OutScale scale{1.0f, 1.0f, 1.0f, true};
      if (!m.end) {
        m = mm_tile<CG>(TR ? t.lo : t.hi, TR ? t.hi : t.lo, first_tile, offs, sh);
        if (!MX && m.product) scale = make_out_scale(ag[m.group], wg[m.group]);
      }
      if (!mm_wait(smem_u32(&posts.taken[at.at]), at.parity, &gave_up)) break;
      if (lane == 0) {
        posts.tile[at.at] = m;
        posts.scale[at.at] = scale;
        mbar_arrive(smem_u32(&posts.posted[at.at]));
      }
      __syncwarp();
      at.next(kMmPosts);
      if (m.end) break;
    }
  } else if (warp >= 4 && warp < 4u + 4u * OUT) {
    // OUT warps per 32 lanes of tensor memory, each every OUT-th 16 tokens
    const uint32_t q = warp % 4u, odd = warp / 4u - 1u;
    // (TR: each every OUT-th 32, which it hands on row by row from 2 KB of its own.)
    uint8_t* box = after + (warp - 4u) * kMmBox;
    // A piece of 16 tokens x 32 columns is turned as [token pair][column] words.
    uint32_t* mine = reinterpret_cast<uint32_t*>(after + (warp - 4u) * kMmTurnPiece);
    // Written out, a lane takes 8 columns of two tokens; the halves of its 32
    // bytes in an order that has 8 lanes read different banks.
    const uint32_t pair = lane / 4u, col = (lane % 4u) * 8u, flip = pair % 2u * 4u;
    Ring acc;
    bool ok = true;
    MmTile m;
    OutScale scale;
    Ring next;
    while (ok && mm_next(&next, &posts, &m, &scale, &gave_up)) {
      if (m.product) {
        if (!(ok = mm_wait(smem_u32(&acc_full[acc.at]), acc.parity, &gave_up))) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      }
      const uint32_t d = tmem + acc.at * acc_cols + (q << 21);
      const uint32_t j0 = m.j0 + j_rank + 32u * q;
      uint16_t* to = out + (size_t)m.row0 * sh.n + j0;
      const uint32_t c0 = (m.lead & ~15u) + 16u * odd;
      // This warp's pieces of 32 columns x 16 tokens: all of them leave tensor
      // memory at once, and the accumulator is free before any is stored.
      uint32_t v[PIECES][16];
      if (m.product) {
#pragma unroll
        for (uint32_t i = 0; i < PIECES; ++i)
          tmem_ld_32x16(TR ? d + 32u * (odd + OUT * (i / 2u)) + 16u * (i % 2u) : d + c0 + 16u * OUT * i,
                        v[i]);
        tmem_wait_ld();
#pragma unroll
        for (uint32_t i = 0; i < PIECES; ++i) tmem_arrived(v[i]);
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          if (PAIR)
            mbar_arrive_peer(peer_smem(smem_u32(&acc_empty[acc.at]), 0));
          else
            mbar_arrive(smem_u32(&acc_empty[acc.at]));
        }
        acc.next(sh.accs);
      } else {
#pragma unroll
        for (uint32_t i = 0; i < PIECES; ++i)
#pragma unroll
          for (int x = 0; x < 16; ++x) v[i][x] = 0u;
      }
      if (TR) {
#pragma unroll
        for (uint32_t i = 0; i + 1u < PIECES; i += 2u) {
          const uint32_t c = 32u * (odd + OUT * (i / 2u));
          if (c >= m.tokens) break;
          uint32_t w[16];
          scaled_bf16<MX>(v[i], scale, w);
          scaled_bf16<MX>(v[i + 1u], scale, w + 8);
          if (elect_one()) bulk_wait_read();  // what was handed on from this box
          __syncwarp();
          // the four parts of a row in the order of the 64-byte swizzle
#pragma unroll
          for (uint32_t x = 0; x < 4u; ++x)
            *reinterpret_cast<uint4*>(box + lane * 64u + ((x ^ (lane / 2u % 4u)) * 16u)) =
                make_uint4(w[4u * x], w[4u * x + 1u], w[4u * x + 2u], w[4u * x + 3u]);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          // rows and columns past the last are not written
          if (elect_one() && (int64_t)j0 < sh.n) {
            tma_store_2d(&maps.out, smem_u32(box), (int32_t)m.row0 + (int32_t)c, (int32_t)j0);
            bulk_commit();
          }
        }
        continue;
      }
#pragma unroll
      for (uint32_t i = 0; i < PIECES; ++i) {
        const uint32_t c = c0 + 16u * OUT * i;
        if (c >= m.tokens) break;
        if (sh.split > 1u) {  // this CTA's part of the sum, [token][128] in the free ring
          float* part = reinterpret_cast<float*>(ring_p) + 32u * q;
#pragma unroll
          for (uint32_t x = 0; x < 16u; ++x)
            part[(c + x) * 128u + lane] = __uint_as_float(v[i][x]);
          continue;
        }
        uint32_t w[8];
        scaled_bf16<MX>(v[i], scale, w);
        __syncwarp();
#pragma unroll
        for (uint32_t x = 0; x < 8u; ++x) mine[32u * x + lane] = w[x];
        __syncwarp();
        if (!W16 && sh.cols <= 2048u && m.lead <= c && c + 16u <= m.tokens &&
            (int64_t)j0 + 32 <= sh.n) {
          // Words of two columns, a token by each half of the warp.  In a row at an
          // odd element they begin with the second column; its first and last
          // columns follow by themselves.
          const uint32_t half = lane / 16u;
          const uint32_t x = 2u * (lane % 16u) + ((uint32_t)sh.n & ((uint32_t)m.row0 + c + half) & 1u);
          const uint32_t *lo = mine + x, *hi = mine + min(x + 1u, 31u), sel = half ? 0x7632u : 0x5410u;
          uint32_t v2[8];
#pragma unroll
          for (uint32_t p = 0; p < 8u; ++p) v2[p] = __byte_perm(lo[32u * p], hi[32u * p], sel);
          uint16_t* at = to + (size_t)(c + half) * sh.n + x;
          const size_t step = 2u * (size_t)sh.n;
          if (x < 31u) {
#pragma unroll
            for (uint32_t p = 0; p < 8u; ++p, at += step) *reinterpret_cast<uint32_t*>(at) = v2[p];
          }
          if (((uint32_t)sh.n & 1u) && (((uint32_t)m.row0 + c + lane) & 1u))
            to[(size_t)(c + lane % 16u) * sh.n + 31u * half] =
                (uint16_t)(mine[lane % 16u / 2u * 32u + 31u * half] >> (lane % 2u * 16u));
          continue;
        }
        if (!W16) {
          const uint32_t last = min(c + 16u, m.tokens);
          if ((int64_t)j0 + lane < sh.n)
#pragma unroll 4
            for (uint32_t row = max(c, m.lead); row < last; ++row)
              to[(size_t)row * sh.n + lane] =
                  (uint16_t)(mine[(row - c) / 2u * 32u + lane] >> ((row - c) % 2u * 16u));
          continue;
        }
        const uint4 a = *reinterpret_cast<const uint4*>(mine + 32u * pair + col + flip);
        const uint4 b = *reinterpret_cast<const uint4*>(mine + 32u * pair + col + (4u - flip));
        const uint4 lo = flip ? b : a, hi = flip ? a : b;  // columns + 0..3 and + 4..7
        const uint32_t row = c + 2u * pair;
        if ((int64_t)j0 + col < sh.n) {
          uint16_t* at = to + (size_t)row * sh.n + col;
          if (row >= m.lead && row < m.tokens)
            *reinterpret_cast<uint4*>(at) =
                make_uint4(__byte_perm(lo.x, lo.y, 0x5410), __byte_perm(lo.z, lo.w, 0x5410),
                           __byte_perm(hi.x, hi.y, 0x5410), __byte_perm(hi.z, hi.w, 0x5410));
          if (row + 1u >= m.lead && row + 1u < m.tokens)
            *reinterpret_cast<uint4*>(at + sh.n) =
                make_uint4(__byte_perm(lo.x, lo.y, 0x7632), __byte_perm(lo.z, lo.w, 0x7632),
                           __byte_perm(hi.x, hi.y, 0x7632), __byte_perm(hi.z, hi.w, 0x7632));
        }
      }
    }
    if (TR && elect_one()) bulk_wait_read();  // shared memory outlives its readers
  }
  if (sh.split > 1u) {
    // Every CTA of the cluster holds a part of the sums of one tile; each adds
    // up every split-th token, the parts in the order of k.
    cluster_sync();
    if (!gave_up) {
      const MmTile m = posts.tile[0];
      const OutScale scale = posts.scale[0];
      const uint32_t j = threadIdx.x % 128u;
      for (uint32_t tk = rank + threadIdx.x / 128u * sh.split; tk < m.tokens;
           tk += kMmThreads / 128u * sh.split) {
        const uint32_t word = ring + (tk * 128u + j) * 4u;
        float v[kMmMaxSplit], sum = 0.0f;  // the parts, read at once
#pragma unroll
        for (uint32_t s = 0; s < kMmMaxSplit; ++s)
          if (s < sh.split) v[s] = ld_peer(peer_smem(word, s));
#pragma unroll
        for (uint32_t s = 0; s < kMmMaxSplit; ++s)
          if (s < sh.split) sum += v[s];
        if (!MX) sum = scale.apply(sum);
        if ((int64_t)m.j0 + j < sh.n)
          out[(size_t)(m.row0 + tk) * sh.n + m.j0 + j] = (uint16_t)cvt_bf16x2(sum, 0.0f);
      }
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  // no CTA leaves while another reads its memory, signals it or multiplies its stages
  if (PAIR || sh.split > 1u) cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 1) {
    if (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(kMmTmemCols));
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(kMmTmemCols));
  }
}

// ---------------------------------------------------------------------------
// Scales for pairs from a layout that the copy engine cannot take: row-major,
// or tiled with matrices that do not begin at a 128-row block or rows of scales
// that end inside a piece of four columns.  To the 128 x 4 tiled layout, each
// matrix from a block of its own, zeros past the last row and column.  A CTA
// takes 128 rows x 16 pieces, 64 bytes of a row at a time.  Bound by the launch
// and one latency of memory (operands of 16384 x 2048 and 4096 x 2048: 5 of
// 74 us with the product, which takes 179 us on the rows as they are).
// ---------------------------------------------------------------------------
struct RetileSrc {
  const uint8_t* src;
  uint8_t* dst;
  int64_t rows;      // of a matrix
  uint32_t blocks;   // 128-row blocks of a matrix
  uint32_t ctas;     // of all matrices: 0 if the operand stays as it is
  uint8_t tiled, bytes;
};

__global__ void __launch_bounds__(kThreads)
    k_retile_scales(RetileSrc a, RetileSrc w, uint32_t scols) {
  __shared__ uint32_t words[16 * 128];
  pdl_begin();
  const bool first = blockIdx.x < a.ctas;
  const RetileSrc& s = first ? a : w;
  const uint32_t cta = first ? blockIdx.x : blockIdx.x - a.ctas;
  const uint32_t pieces = (scols + 3u) / 4u, runs = (pieces + 15u) / 16u;
  const uint32_t block = cta / runs, p0 = (cta - block * runs) * 16u;
  const uint32_t matrix = block / s.blocks;
  const int64_t r0 = (int64_t)(block - matrix * s.blocks) * 128;  // in its matrix
  uint32_t v[8], keep[8], to[8];
#pragma unroll
  for (uint32_t i = 0; i < 8u; ++i) {  // eight loads on their way at once
    // neighbours along a row, or in the tiled order
    const uint32_t x = threadIdx.x + kThreads * i;
    const uint32_t p = s.tiled ? x / 128u : x % 16u;
    const uint32_t r = s.tiled ? x % 4u * 32u + x % 128u / 4u : x / 16u, c = 4u * (p0 + p);
    const uint32_t take = r0 + r < s.rows && c < scols ? min(4u, scols - c) : 0u;
    const u64 row = (u64)(matrix * s.rows + r0) + r;
    const u64 at = take == 0u ? 0u
                   : s.tiled  ? ((row / 128u) * pieces + p0 + p) * 512u + row % 32u * 16u +
                                   row % 128u / 32u * 4u
                              : row * scols + c;
    to[i] = p * 128u + r % 32u * 4u + r / 32u;
    keep[i] = take == 4u ? 0xFFFFFFFFu : (1u << (8u * take)) - 1u;
    if (!s.bytes) {
      v[i] = *reinterpret_cast<const uint32_t*>(s.src + at);
    } else {
      v[i] = 0u;
      for (uint32_t b = 0; b < take; ++b) v[i] |= (uint32_t)s.src[at + b] << (8u * b);
    }
  }
#pragma unroll
  for (uint32_t i = 0; i < 8u; ++i) words[to[i]] = v[i] & keep[i];
  __syncthreads();
#pragma unroll
  for (uint32_t i = 0; i < 2u; ++i) {
    const uint32_t x = threadIdx.x + kThreads * i;  // 16 bytes each
    if (p0 + x / 32u < pieces)
      *reinterpret_cast<uint4*>(s.dst + ((size_t)block * pieces + p0) * 512u + 16u * x) =
          *reinterpret_cast<const uint4*>(words + 4u * x);
  }
}
