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
//   warp 0  copies both operands' codes by TMA, 256 k-elements (128 bytes per
//           row, 128-byte swizzle) per stage of a shared-memory ring;
//   warps 2, 3 copy the block scales into the ring in the 128 x 4 tiled
//           order the tensor core wants, from either layout and at any row
//           (a group starts anywhere), and zero what lies past the last k;
//   warp 1  moves a stage's scales to tensor memory and issues its products;
//   warps 4-7 read finished accumulators and write bf16 rows of out, while
//           the next tile runs on the other accumulator.
#pragma once

constexpr int kMmThreads = 256;
constexpr int kMmM = 128;            // w rows of a tile
constexpr int kMmStageBytes = 128;   // code bytes per row and stage: 256 elements
constexpr int kMmScaleLag = 3;       // stages the scale copies run ahead (<= stages - 1)
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

// Bounded wait for a phase; false once any wait of the CTA has given up.
__device__ __forceinline__ bool mm_wait(uint32_t bar, uint32_t parity, volatile uint32_t* gave_up) {
  for (uint32_t i = 0; i < kMmPolls; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 255u && *gave_up) return false;
  }
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

// bytes <= 4 (16) of a word; the rest of it becomes zero.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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

// first_tile[0 .. groups] by a scan over the CTA (256 threads).
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
// Scales of one 128-row block for one stage, into ATOMS atoms of 512 bytes
// (128 rows x 4 scale columns each).  `half` picks which rows (or atoms) this
// warp copies: two warps share the work.
// ---------------------------------------------------------------------------
struct ScaleSrc {
  const uint8_t* base;
  const uint8_t* row[2];  // this lane's rows 32 (2 half + q) + lane; null: not in the array
  uint32_t step;          // bytes from one group of 4 columns to the next
  bool words16;           // the block is one of the tiled layout's own
  bool bytes;             // no 4-byte alignment
};

__device__ __forceinline__ ScaleSrc scale_src(const uint8_t* base, bool tiled, bool bytes,
                                              int64_t row0, int64_t rows, uint32_t scols,
                                              uint32_t half, uint32_t lane) {
  ScaleSrc s;
  s.base = base;
  s.bytes = bytes;
  s.step = tiled ? 512u : 4u;
  s.words16 = tiled && row0 % 128 == 0;
  const uint32_t ct = (scols + 3u) / 4u;
#pragma unroll
  for (uint32_t q = 0; q < 2u; ++q) {
    const int64_t r = row0 + 32u * (2u * half + q) + lane;
    s.row[q] = nullptr;
    if (r < rows)
      s.row[q] = tiled ? base + (size_t)(r / 128) * ct * 512u + (size_t)(r % 32) * 16u +
                             (size_t)(r % 128 / 32) * 4u
                       : base + (size_t)r * scols;
  }
  return s;
}

template <int ATOMS>
__device__ __forceinline__ void copy_scales(const ScaleSrc& s, int64_t row0, uint32_t dst,
                                            uint32_t dst_step, uint32_t kstep, uint32_t scols,
                                            uint32_t half, uint32_t lane) {
#pragma unroll
  for (uint32_t j = 0; j < (uint32_t)ATOMS; ++j) {
    const uint32_t c4 = kstep * ATOMS + j;  // group of 4 scale columns
    const uint32_t valid = 4u * c4 >= scols ? 0u : min(4u, scols - 4u * c4);
    const uint32_t to = dst + j * dst_step;
    if (s.words16 && valid == 4u) {
      if (j % 2u == half) {
        const uint32_t ct = (scols + 3u) / 4u;
        cp_async16(to + 16u * lane, s.base + ((size_t)(row0 / 128) * ct + c4) * 512u + 16u * lane);
      }
      continue;
    }
#pragma unroll
    for (uint32_t q = 0; q < 2u; ++q) {
      const uint32_t at = to + 16u * lane + 4u * (2u * half + q);
      const uint32_t take = s.row[q] != nullptr ? valid : 0u;
      if (!s.bytes) {
        cp_async4(at, take ? s.row[q] + (size_t)c4 * s.step : s.base, take);
      } else {
        uint32_t w = 0u;
        for (uint32_t i = 0; i < take; ++i) w |= (uint32_t)s.row[q][4u * c4 + i] << (8u * i);
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(w) : "memory");
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
template <bool MX>
__global__ void __launch_bounds__(kMmThreads, 1)
    k_matmul(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap w_map,
             const uint8_t* __restrict__ as, const uint8_t* __restrict__ ws,
             const float* __restrict__ ag, const float* __restrict__ wg,
             const int64_t* __restrict__ offs, MmShape sh, uint16_t* __restrict__ out) {
  constexpr uint32_t ATOMS = MX ? 2 : 4;  // groups of 4 scale columns per stage
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) u64 full[kMmMaxStages], empty[kMmMaxStages], acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_base_s, warp_sum[kMmThreads / 32];
  __shared__ volatile uint32_t gave_up;
  const uint32_t warp = threadIdx.x / 32u, lane = threadIdx.x % 32u;
  const uint32_t rb = (sh.nt + 127u) / 128u;  // 128-row blocks of token scales
  const uint32_t w_code = kMmM * kMmStageBytes, x_code = sh.nt * kMmStageBytes;
  const uint32_t stage_bytes = w_code + x_code + ATOMS * 512u * (1u + rb);
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t stage_at = (stage_bytes + 1023u) & ~1023u;
  uint8_t* after = smem_raw + (ring - smem_u32(smem_raw)) + sh.stages * stage_at;
  uint16_t* turn = reinterpret_cast<uint16_t*>(after);               // [4][32][40] bf16
  uint32_t* first_tile = reinterpret_cast<uint32_t*>(after + 4 * 32 * 40 * 2);

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < sh.stages; ++s) {
      mbar_init(smem_u32(&full[s]), 3);  // the TMA thread and two scale warps
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
  const uint32_t sf_cols = 4u * ATOMS * (1u + rb);  // tensor-memory columns of a stage's scales
  const uint32_t sf_base = tmem + sh.accs * acc_cols;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t i = 0;  // stages filled so far
      bool ok = true;
      for (uint32_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const MmTile m = mm_tile(t, first_tile, offs, sh);
        if (!m.product) continue;
        const int32_t wr = (int32_t)(m.group * sh.n + m.j0);
        for (uint32_t k = 0; k < sh.ksteps; ++k, ++i) {
          const uint32_t s = i % sh.stages;
          if (i >= sh.stages &&
              !(ok = mm_wait(smem_u32(&empty[s]), (i / sh.stages - 1u) & 1u, &gave_up)))
            break;
          const uint32_t at = ring + s * stage_at, bar = smem_u32(&full[s]);
          mbar_expect(bar, w_code + x_code);
          tma_load_2d(at, &w_map, (int32_t)(k * kMmStageBytes), wr, bar);
          tma_load_2d(at + w_code, &a_map, (int32_t)(k * kMmStageBytes), (int32_t)m.row0, bar);
        }
      }
      if (!ok)  // let the copies in flight land before the CTA leaves
        for (int z = 0; z < 1000; ++z) __nanosleep(1000);
    }
  } else if (warp == 2 || warp == 3) {
    const uint32_t half = warp - 2u;
    uint32_t i = 0;
    bool ok = true;
    const auto publish = [&](uint32_t done) {  // this warp's copies of stage number `done` are in
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&full[done % sh.stages]));
    };
    for (uint32_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const MmTile m = mm_tile(t, first_tile, offs, sh);
      if (!m.product) continue;
      const int64_t wr = (int64_t)m.group * sh.n + m.j0;
      const ScaleSrc sw = scale_src(ws, sh.w_tiled, sh.w_bytes, wr, sh.n * sh.matrices, sh.scols,
                                    half, lane);
      const ScaleSrc s0 = scale_src(as, sh.a_tiled, sh.a_bytes, m.row0, sh.rows, sh.scols, half,
                                    lane);
      const bool two = m.tokens > 128u;
      const ScaleSrc s1 = scale_src(as, sh.a_tiled, sh.a_bytes, m.row0 + 128, two ? sh.rows : 0,
                                    sh.scols, half, lane);
      for (uint32_t k = 0; k < sh.ksteps; ++k, ++i) {
        const uint32_t s = i % sh.stages;
        if (i >= sh.stages &&
            !(ok = mm_wait(smem_u32(&empty[s]), (i / sh.stages - 1u) & 1u, &gave_up)))
          break;
        const uint32_t at = ring + s * stage_at + w_code + x_code;
        copy_scales<ATOMS>(sw, wr, at, 512u, k, sh.scols, half, lane);
        const uint32_t ax = at + ATOMS * 512u;
        copy_scales<ATOMS>(s0, m.row0, ax, 512u * rb, k, sh.scols, half, lane);
        if (two) copy_scales<ATOMS>(s1, m.row0 + 128, ax + 512u, 512u * rb, k, sh.scols, half, lane);
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (i >= (uint32_t)kMmScaleLag) {
          asm volatile("cp.async.wait_group %0;" ::"n"(kMmScaleLag) : "memory");
          publish(i - kMmScaleLag);
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (ok)
      for (uint32_t d = i > (uint32_t)kMmScaleLag ? i - kMmScaleLag : 0u; d < i; ++d) publish(d);
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t i = 0, n_acc = 0;  // stages used, tiles begun
      bool ok = true;
      for (uint32_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const MmTile m = mm_tile(t, first_tile, offs, sh);
        if (!m.product) continue;
        const uint32_t a = n_acc % sh.accs;
        if (n_acc >= sh.accs &&
            !(ok = mm_wait(smem_u32(&acc_empty[a]), (n_acc / sh.accs - 1u) & 1u, &gave_up)))
          break;
        ++n_acc;
        const uint32_t d = tmem + a * acc_cols;
        const uint32_t idesc = mm_idesc<MX>((m.tokens + 15u) & ~15u);
        const uint32_t blocks = m.tokens > 128u ? 2u : 1u;
        for (uint32_t k = 0; k < sh.ksteps; ++k, ++i) {
          const uint32_t s = i % sh.stages;
          // the scale slot's last reader must be done
          if (i >= sh.sf_slots) {
            const uint32_t p = i - sh.sf_slots;
            if (!(ok = mm_wait(smem_u32(&empty[p % sh.stages]), (p / sh.stages) & 1u, &gave_up)))
              break;
          }
          if (!(ok = mm_wait(smem_u32(&full[s]), (i / sh.stages) & 1u, &gave_up))) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t at = ring + s * stage_at;
          const uint32_t sf = sf_base + (i % sh.sf_slots) * sf_cols;
          const uint32_t sfx = sf + 4u * ATOMS;
          const uint32_t asc = at + w_code + x_code, axs = asc + ATOMS * 512u;
          for (uint32_t j = 0; j < ATOMS; ++j) {
            scales_to_tmem(sf + 4u * j, scale_desc(asc + 512u * j));
            for (uint32_t b = 0; b < blocks; ++b)
              scales_to_tmem(sfx + 4u * (j * rb + b), scale_desc(axs + 512u * (j * rb + b)));
          }
          const uint32_t left = sh.cols - k * 256u;
          const uint32_t mmas = left >= 256u ? 4u : (left + 63u) / 64u;
          const u64 da = code_desc(at), db = code_desc(at + w_code);
          for (uint32_t j = 0; j < mmas; ++j) {
            const uint32_t c = MX ? j / 2u : j;  // atom of this product's scales
            const uint32_t id = MX ? (j & 1u) * 2u : 0u;
            mma_fp4<MX>(d, da + 2u * j, db + 2u * j, idesc | (id << 4) | (id << 29), sf + 4u * c,
                        sfx + 4u * rb * c, (k | j) != 0u);
          }
          mma_commit(smem_u32(&empty[s]));
        }
        if (ok) mma_commit(smem_u32(&acc_full[a]));
      }
      // the products in flight must end before tensor memory is freed
      if (i > 0) {
        const uint32_t p = i - 1u;
        mm_wait(smem_u32(&empty[p % sh.stages]), (p / sh.stages) & 1u, &gave_up);
      }
    }
  } else {
    const uint32_t q = warp - 4u;  // this warp's 32 lanes of tensor memory
    uint16_t* mine = turn + q * 32u * 40u;
    uint32_t n_acc = 0;
    bool ok = true;
    for (uint32_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const MmTile m = mm_tile(t, first_tile, offs, sh);
      const uint32_t a = n_acc % sh.accs;
      OutScale scale{1.0f, 1.0f, 1.0f};
      if (m.product) {
        if (!(ok = mm_wait(smem_u32(&acc_full[a]), (n_acc / sh.accs) & 1u, &gave_up))) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        ++n_acc;
        if (!MX) scale = make_out_scale(ag[m.group], wg[m.group]);
      }
      const uint32_t d = tmem + a * acc_cols + (q << 21);
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
        if (lane == 0) mbar_arrive(smem_u32(&acc_empty[a]));
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
