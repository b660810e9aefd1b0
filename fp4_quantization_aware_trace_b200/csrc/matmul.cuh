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
//   warp 0     copies both operands' codes by TMA, 256 k-elements (128 bytes
//              per row, 128-byte swizzle) per stage of a shared-memory ring,
//              and tiled scales whose 128-row block is the tile's own;
//   warps 8-11 copy all other scales into the ring in the 128 x 4 tiled order
//              the tensor core wants, from either layout and at any row (a
//              group starts anywhere), and zero what lies past the last k;
//   warp 1     moves a stage's scales to tensor memory and issues its
//              products;
//   warps 4-7  read finished accumulators and write bf16 rows of out, while
//              the next tile runs on the other accumulator.
// Each role is one warp that runs alone on its scheduler, so a stage costs it
// its instructions' latencies: ring positions are counters and not quotients,
// and the loops over a stage's parts are unrolled.
#pragma once

constexpr int kMmThreads = 384;
constexpr int kMmM = 128;            // w rows of a tile
constexpr int kMmStageBytes = 128;   // code bytes per row and stage: 256 elements
constexpr int kMmMaxStages = 8;
constexpr uint32_t kMmTmemCols = 512;
// Polls of one wait before a CTA gives up (each try_wait itself suspends):
// a guard, every wait ends as its copies and products do.
constexpr uint32_t kMmPolls = 1u << 22;

struct MmShape {
  int64_t rows, n;
  uint32_t cols, scols;        // k-elements, scale columns
  int32_t groups, matrices;
  uint32_t nt;                 // tokens of a full tile (multiple of 16)
  uint32_t n_tiles;            // ceil(n / 128)
  uint32_t ksteps;             // stages of a whole product
  uint32_t stages, accs, sf_slots;
  uint8_t a_tiled, w_tiled;
  uint8_t a_bytes, w_bytes;    // row-major scales that are not 4-byte words
  uint8_t out16;               // rows of out are 16-byte aligned
};

__device__ uint32_t g_matmul_gave_up;  // set if a wait ran out of polls

// The product of two global scales as m * p * q, m in [1, 2) and p, q powers
// of two: ga * gw itself may leave fp32's range where sum * ga * gw does not
// (a small activation against a large weight).  |sum| is 0 or in
// [2^-20, 2^54], so with the exponents halved no step over- or underflows
// unless the result does; past +-250 the result is 0 or infinite anyway.
struct OutScale {
  float m, p, q;
  __device__ __forceinline__ float apply(float sum) const { return ((sum * m) * p) * q; }
};

__device__ __forceinline__ OutScale make_out_scale(float ga, float gw) {
  const double d = (double)ga * (double)gw;  // exact
  OutScale s{(float)d, 1.0f, 1.0f};
  int e = ((__double2hiint(d) >> 20) & 0x7FF) - 1023;
  if (e == -1023 || e == 1024) return s;  // zero or not finite
  s.m = (float)__hiloint2double((__double2hiint(d) & 0x000FFFFF) | (1023 << 20), __double2loint(d));
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

// One lane of a converged warp; ptxas knows that a branch on it leaves a
// single thread and keeps the operands of what it issues in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0u;
}

// Bounded wait for a phase; false once any wait of the CTA has given up.
// The lanes of a warp agree on the answer.
__device__ __forceinline__ bool mm_wait(uint32_t bar, uint32_t parity, volatile uint32_t* gave_up) {
  bool ok = false;
  for (uint32_t i = 0; i < kMmPolls; ++i) {
    if ((ok = mbar_try_wait(bar, parity))) break;
    if ((i & 255u) == 255u && *gave_up) break;
  }
  if (__all_sync(0xFFFFFFFFu, ok)) return true;
  *gave_up = 1u;
  g_matmul_gave_up = 1u;
  return false;
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int32_t x,
                                            int32_t y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
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
// (8-row groups 128 bytes apart, no swizzle).
__device__ __forceinline__ u64 code_desc(uint32_t smem) {
  return (u64)((smem & 0x3FFFFu) >> 4) | ((u64)1 << 16) | ((u64)(1024 >> 4) << 32) |
         ((u64)1 << 46) | ((u64)2 << 61);
}
__device__ __forceinline__ u64 scale_desc(uint32_t smem) {
  return (u64)((smem & 0x3FFFFu) >> 4) | ((u64)(128 >> 4) << 32) | ((u64)1 << 46);
}

// Instruction descriptor: E2M1 x E2M1, K-major, M = 128, N = n; the scale
// type and which bytes of the scale words the instruction uses (ids).
template <bool MX>
__device__ __forceinline__ uint32_t mm_idesc(uint32_t n) {
  return (1u << 7) | (1u << 10) | ((n >> 3) << 17) | (MX ? 1u << 23 : 0u) | ((128u >> 4) << 24);
}

template <bool MX>
__device__ __forceinline__ void mma_fp4(uint32_t d, u64 a, u64 b, uint32_t idesc, uint32_t sa,
                                        uint32_t sb, bool add) {
  if (MX)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)add)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, "
        "[%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)add)
        : "memory");
}

__device__ __forceinline__ void scales_to_tmem(uint32_t tmem, u64 desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
               : "memory");
}

// The barrier's phase ends when every product and copy issued so far by this
// thread has.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
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
  uint32_t tokens;    // rows of this tile that belong to the group
  uint32_t j0;        // first output column
  bool product;       // false: a group without a matrix, its rows are zero
};

__device__ __forceinline__ int64_t mm_bound(const int64_t* offs, int32_t g, const MmShape& sh) {
  if (offs == nullptr) return g == 0 ? 0 : sh.rows;
  const int64_t v = offs[g];
  return v < 0 ? 0 : (v > sh.rows ? sh.rows : v);
}

__device__ __forceinline__ MmTile mm_tile(uint32_t t, const uint32_t* first_tile,
                                          const int64_t* offs, const MmShape& sh) {
  MmTile m;
  const uint32_t tt = t / sh.n_tiles;
  int32_t lo = 0, hi = sh.groups - 1;  // the last group that starts at or before tt
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) / 2;
    if (first_tile[mid] <= tt) lo = mid; else hi = mid - 1;
  }
  m.group = lo;
  m.row0 = mm_bound(offs, lo, sh) + (int64_t)(tt - first_tile[lo]) * sh.nt;
  const int64_t left = mm_bound(offs, lo + 1, sh) - m.row0;
  m.tokens = left < (int64_t)sh.nt ? (uint32_t)left : sh.nt;
  m.j0 = (t - tt * sh.n_tiles) * kMmM;
  m.product = lo < sh.matrices;
  return m;
}

// first_tile[0 .. groups] by a scan over the CTA.
__device__ __forceinline__ void mm_table(uint32_t* first_tile, uint32_t* warp_sum,
                                         const int64_t* offs, const MmShape& sh) {
  const uint32_t lane = threadIdx.x % 32u, warp = threadIdx.x / 32u;
  uint32_t carry = 0u;
  for (int32_t g0 = 0; g0 < sh.groups; g0 += kMmThreads) {
    const int32_t g = g0 + (int32_t)threadIdx.x;
    uint32_t tiles = 0u;
    if (g < sh.groups) {
      const int64_t cnt = mm_bound(offs, g + 1, sh) - mm_bound(offs, g, sh);
      if (cnt > 0) tiles = (uint32_t)((cnt + sh.nt - 1) / sh.nt);
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
// The kernel; RB: 128-row blocks of token scales (1 up to 128 tokens, else 2)
// ---------------------------------------------------------------------------
template <bool MX, int RB>
__global__ void __launch_bounds__(kMmThreads, 1)
    k_matmul(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap w_map,
             const uint8_t* __restrict__ as, const uint8_t* __restrict__ ws,
             const float* __restrict__ ag, const float* __restrict__ wg,
             const int64_t* __restrict__ offs, MmShape sh, uint16_t* __restrict__ out) {
  constexpr uint32_t ATOMS = MX ? 2 : 4;  // groups of 4 scale columns per stage
  constexpr uint32_t w_code = kMmM * kMmStageBytes;
  constexpr uint32_t block_bytes = ATOMS * 512u;  // a block's scales per stage
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) u64 full[kMmMaxStages], empty[kMmMaxStages], acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_base_s, warp_sum[kMmThreads / 32];
  __shared__ volatile uint32_t gave_up;
  const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32u, 0), lane = threadIdx.x % 32u;
  const uint32_t x_code = sh.nt * kMmStageBytes;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t stage_at = (w_code + x_code + block_bytes * (1u + RB) + 1023u) & ~1023u;
  uint8_t* after = smem_raw + (ring - smem_u32(smem_raw)) + sh.stages * stage_at;
  uint16_t* turn = reinterpret_cast<uint16_t*>(after);               // [4][32][40] bf16
  uint32_t* first_tile = reinterpret_cast<uint32_t*>(after + 4 * 32 * 40 * 2);

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < sh.stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1 + 128);  // the TMA thread and the scale lanes
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (uint32_t a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&acc_full[a]), 1);
      mbar_init(smem_u32(&acc_empty[a]), 4);
    }
    gave_up = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_begin();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_base_s)),
                 "r"(kMmTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  mm_table(first_tile, warp_sum, offs, sh);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base_s;
  const uint32_t tiles = first_tile[sh.groups] * sh.n_tiles;
  const uint32_t acc_cols = (sh.nt + 31u) & ~31u;
  constexpr uint32_t sf_cols = 4u * ATOMS * (1u + RB);  // tensor-memory columns of a stage's scales
  const uint32_t sf_base = tmem + sh.accs * acc_cols;

  if (warp == 0) {
    Ring r;
    r.parity = 1u;  // the first round finds every slot empty
    bool ok = true;
    const uint32_t c4s = (sh.scols + 3u) / 4u, bulk_steps = sh.scols / (4u * ATOMS);
    for (uint32_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const MmTile m = mm_tile(t, first_tile, offs, sh);
      if (!m.product) continue;
      const int64_t wr = m.group * sh.n + m.j0;
      const bool w_bulk = scales_bulk(sh.w_tiled, wr), x_bulk = scales_bulk(sh.a_tiled, m.row0);
      const bool two = RB == 2 && m.tokens > 128u;
      const uint8_t* w_from = ws + (size_t)(wr / 128) * c4s * 512u;
      const uint8_t* x_from = as + (size_t)(m.row0 / 128) * c4s * 512u;
      const uint32_t bulk_bytes = (w_bulk ? block_bytes : 0u) +
                                  (x_bulk ? (two ? 2u : 1u) * block_bytes : 0u);
      for (uint32_t k = 0; k < sh.ksteps; ++k, r.next(sh.stages)) {
        const uint32_t bar = smem_u32(&full[r.at]), at = ring + r.at * stage_at;
        if (!(ok = mm_wait(smem_u32(&empty[r.at]), r.parity, &gave_up))) break;
        if (!elect_one()) continue;
        const bool bulk = k < bulk_steps;
        mbar_expect(bar, w_code + x_code + (bulk ? bulk_bytes : 0u));
        tma_load_2d(at, &w_map, (int32_t)(k * kMmStageBytes), (int32_t)wr, bar);
        tma_load_2d(at + w_code, &a_map, (int32_t)(k * kMmStageBytes), (int32_t)m.row0, bar);
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
    if (!ok)  // let the copies in flight land before the CTA leaves
      for (int z = 0; z < 1000; ++z) __nanosleep(1000);
  } else if (warp >= 8) {
    const uint32_t quarter = warp - 8u;
    Ring r;
    r.parity = 1u;
    bool ok = true;
    for (uint32_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const MmTile m = mm_tile(t, first_tile, offs, sh);
      if (!m.product) continue;
      const int64_t wr = m.group * sh.n + m.j0;
      const ScaleSrc sw = scale_src(ws, sh.w_tiled, sh.w_bytes, wr, sh.n * sh.matrices, sh.scols,
                                    quarter, lane);
      const ScaleSrc s0 = scale_src(as, sh.a_tiled, sh.a_bytes, m.row0, sh.rows, sh.scols, quarter,
                                    lane);
      const bool two = RB == 2 && m.tokens > 128u;
      const ScaleSrc s1 = scale_src(as, sh.a_tiled, sh.a_bytes, m.row0 + 128, sh.rows, sh.scols,
                                    quarter, lane);
      const uint32_t word = w_code + x_code + 16u * lane + 4u * quarter;
      for (uint32_t k = 0; k < sh.ksteps; ++k, r.next(sh.stages)) {
        if (!(ok = mm_wait(smem_u32(&empty[r.at]), r.parity, &gave_up))) break;
        const uint32_t at = ring + r.at * stage_at + word, bar = smem_u32(&full[r.at]);
        copy_scales<ATOMS>(sw, ws, at, 512u, k, sh.scols);
        copy_scales<ATOMS>(s0, as, at + block_bytes, 512u, k, sh.scols);
        if (two) copy_scales<ATOMS>(s1, as, at + 2u * block_bytes, 512u, k, sh.scols);
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
  } else if (warp == 1) {
    Ring r, acc, sf, sf_last;  // sf_last: the stage that used the scale slot before
    acc.parity = 1u;
    uint32_t begun = 0;  // scale slots used so far, up to sf_slots
    bool ok = true;
    Ring last;
    bool any = false;
    for (uint32_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const MmTile m = mm_tile(t, first_tile, offs, sh);
      if (!m.product) continue;
      if (!(ok = mm_wait(smem_u32(&acc_empty[acc.at]), acc.parity, &gave_up))) break;
      const uint32_t d = tmem + acc.at * acc_cols;
      const uint32_t idesc = mm_idesc<MX>((m.tokens + 15u) & ~15u);
      const bool two = RB == 2 && m.tokens > 128u;
      uint32_t left = sh.cols;
      for (uint32_t k = 0; k < sh.ksteps; ++k, r.next(sh.stages), sf.next(sh.sf_slots)) {
        // the scale slot's last reader must be done
        if (begun == sh.sf_slots) {
          if (!(ok = mm_wait(smem_u32(&empty[sf_last.at]), sf_last.parity, &gave_up))) break;
          sf_last.next(sh.stages);
        } else {
          ++begun;
        }
        if (!(ok = mm_wait(smem_u32(&full[r.at]), r.parity, &gave_up))) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        // scales written by cp.async and plain stores: seen by the copy below
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        last = r;
        any = true;
        left -= 256u;  // wraps only after the last step
        if (!elect_one()) continue;
        const uint32_t at = ring + r.at * stage_at;
        const uint32_t slot = sf_base + sf.at * sf_cols;
        const u64 sd = scale_desc(at + w_code + x_code);
#pragma unroll
        for (uint32_t j = 0; j < ATOMS; ++j) {
          scales_to_tmem(slot + 4u * j, sd + 32u * j);
          scales_to_tmem(slot + 4u * ATOMS + 4u * RB * j, sd + 32u * (ATOMS + j));
          if (two)
            scales_to_tmem(slot + 4u * ATOMS + 4u * (RB * j + 1u), sd + 32u * (2u * ATOMS + j));
        }
        const u64 da = code_desc(at), db = code_desc(at + w_code);
#pragma unroll
        for (uint32_t j = 0; j < 4u; ++j) {
          const uint32_t c = MX ? j / 2u : j;  // piece with this product's scales
          const uint32_t id = MX ? (j & 1u) * 2u : 0u;
          if (left + 256u > 64u * j)
            mma_fp4<MX>(d, da + 2u * j, db + 2u * j, idesc | (id << 4) | (id << 29),
                        slot + 4u * c, slot + 4u * ATOMS + 4u * RB * c, (k | j) != 0u);
        }
        mma_commit(smem_u32(&empty[r.at]));
      }
      if (!ok) break;
      if (elect_one()) mma_commit(smem_u32(&acc_full[acc.at]));
      acc.next(sh.accs);
    }
    // the products in flight must end before tensor memory is freed
    if (any) mm_wait(smem_u32(&empty[last.at]), last.parity, &gave_up);
  } else if (warp >= 4) {
    const uint32_t q = warp - 4u;  // this warp's 32 lanes of tensor memory
    uint16_t* mine = turn + q * 32u * 40u;
    Ring acc;
    bool ok = true;
    for (uint32_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const MmTile m = mm_tile(t, first_tile, offs, sh);
      OutScale scale{1.0f, 1.0f, 1.0f};
      if (m.product) {
        if (!MX) scale = make_out_scale(ag[m.group], wg[m.group]);
        if (!(ok = mm_wait(smem_u32(&acc_full[acc.at]), acc.parity, &gave_up))) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      }
      const uint32_t d = tmem + acc.at * acc_cols + (q << 21);
      const uint32_t j0 = m.j0 + 32u * q;
      for (uint32_t c0 = 0; c0 < m.tokens; c0 += 32u) {
        uint32_t v[32];
        if (m.product) {
          tmem_ld16(d + c0, v);
          tmem_ld16(d + c0 + 16u, v + 16);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) v[x] = 0u;
        }
        __syncwarp();
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          const float f = MX ? __uint_as_float(v[x]) : scale.apply(__uint_as_float(v[x]));
          mine[x * 40 + lane] = (uint16_t)cvt_bf16x2(f, 0.0f);
        }
        __syncwarp();
        const uint32_t last = min(32u, m.tokens - c0);
        if (sh.out16) {
#pragma unroll
          for (uint32_t p = 0; p < 4u; ++p) {
            const uint32_t tok = p * 8u + lane / 4u, col = (lane % 4u) * 8u;
            if (tok < last && (int64_t)j0 + col < sh.n)
              *reinterpret_cast<uint4*>(out + (size_t)(m.row0 + c0 + tok) * sh.n + j0 + col) =
                  *reinterpret_cast<const uint4*>(mine + tok * 40u + col);
          }
        } else if ((int64_t)j0 + lane < sh.n) {
          for (uint32_t tok = 0; tok < last; ++tok)
            out[(size_t)(m.row0 + c0 + tok) * sh.n + j0 + lane] = mine[tok * 40u + lane];
        }
      }
      if (m.product) {
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&acc_empty[acc.at]));
        acc.next(sh.accs);
      }
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kMmTmemCols));
}
