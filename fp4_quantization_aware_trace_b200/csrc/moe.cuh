// moe.cuh -- the routing sort, tokens into expert order and back with the
// routing weights, and their gradients.  Included by trace_fp4.cu inside its
// anonymous namespace.
//
// A slot is one (token, choice) pair, numbered token * k + choice.  The sort
// gives each slot a row; rows of one expert are contiguous and in slot order
// (a stable counting sort: no atomic decides an order, so a run repeats bit
// for bit).  Slots whose expert id is outside [0, E) are dropped: they fill
// the last group, group E, and carry no row.
#pragma once

constexpr int kSortMaxWarps = 32;
constexpr uint32_t kSortSmem = 96u * 1024u;  // per-warp counters
constexpr uint32_t kSortChunk = 4096u;       // slots per CTA; one CTA sorts as many alone
constexpr uint32_t kSortMaxChunks = 256u;    // beyond that chunks grow: every CTA reads all counts

// The counter a slot belongs to: its expert, or E for a dropped one.
template <typename ID>
__device__ __forceinline__ uint32_t sort_key(const ID* __restrict__ ids, uint32_t slot,
                                             uint32_t E) {
  const ID v = ids[slot];
  return v >= (ID)0 && (long long)v < (long long)E ? (uint32_t)v : E;
}

// First pass of a sort over several CTAs: counts of one chunk of slots,
// counts[e][chunk].
template <typename ID>
__global__ void __launch_bounds__(512)
    k_moe_count(const ID* __restrict__ ids, uint32_t slots, uint32_t chunk, uint32_t E,
                uint32_t* __restrict__ counts) {
  extern __shared__ uint32_t hist[];
  pdl_begin();
  for (uint32_t e = threadIdx.x; e <= E; e += blockDim.x) hist[e] = 0u;
  __syncthreads();
  const uint32_t first = blockIdx.x * chunk, last = min(first + chunk, slots);
  for (uint32_t s0 = first + threadIdx.x; s0 < last; s0 += 8u * blockDim.x) {
    uint32_t key[8];  // eight loads on their way at a time
#pragma unroll
    for (uint32_t i = 0; i < 8u; ++i)
      if (s0 + i * blockDim.x < last) key[i] = sort_key(ids, s0 + i * blockDim.x, E);
#pragma unroll
    for (uint32_t i = 0; i < 8u; ++i)
      if (s0 + i * blockDim.x < last) atomicAdd(&hist[key[i]], 1u);
  }
  __syncthreads();
  for (uint32_t e = threadIdx.x; e <= E; e += blockDim.x)
    counts[(size_t)e * gridDim.x + blockIdx.x] = hist[e];
}

// Keys of 128 slots from s0 on, 32 apart (n past the end: no counter).
template <typename ID>
__device__ __forceinline__ void sort_keys(const ID* __restrict__ ids, uint32_t s0, uint32_t hi,
                                          uint32_t E, uint32_t n, uint32_t* key) {
  const uint32_t s = s0 + threadIdx.x % 32u;
#pragma unroll
  for (uint32_t i = 0; i < 4u; ++i) key[i] = s + 32u * i < hi ? sort_key(ids, s + 32u * i, E) : n;
}

// Lanes of the warp with this lane's key (< 2^bits), a ballot per bit: the
// match instruction would take 20 us of a sort of 65536 x 8 slots.
__device__ __forceinline__ uint32_t same_key(uint32_t key, uint32_t bits) {
  uint32_t same = 0xFFFFFFFFu;
  for (uint32_t b = 0; b < bits; ++b) {
    const bool one = key >> b & 1u;
    const uint32_t ones = __ballot_sync(0xFFFFFFFFu, one);
    same &= one ? ones : ~ones;
  }
  return same;
}

// Second pass (the only one when a single CTA holds every slot).  Each warp
// owns a contiguous piece of the CTA's chunk and counts it; the counters
// then become each warp's next row per expert: rows of earlier experts +
// this expert's rows in earlier chunks + in earlier warps.  In the last
// walk the lanes of one expert rank themselves by lane, which is slot order.
// Bound by latencies, so what does not depend on one another is asked for
// together: a warp's keys, and the counts of all chunks of five experts; and the
// warps' counters of an expert are scanned by a warp, not by a thread (65536 x 8
// slots, 128 experts: 12.8 us for both passes; 17.4 us with the counts of one
// expert at a time and a thread for each expert's counters).  A sort by one CTA
// takes a warp for every 64 slots or 32 experts (1 x 8 slots, 128 experts: 2.3 us,
// with 32 warps 3.9).
constexpr uint32_t kSortAtOnce = 5u;  // experts of a warp whose counts are read together
template <typename ID>
__global__ void __launch_bounds__(32 * kSortMaxWarps)
    k_moe_place(const ID* __restrict__ ids, uint32_t slots, uint32_t chunk, uint32_t E,
                const uint32_t* __restrict__ counts, int64_t* __restrict__ offsets,
                int32_t* __restrict__ rows, int32_t* __restrict__ slot_of) {
  extern __shared__ uint32_t next[];  // [warps][stride], all[E + 1], earlier[E + 1]
  __shared__ uint32_t part[kSortMaxWarps];
  __shared__ uint32_t carry;
  const uint32_t n = E + 1u, stride = n | 1u, warps = blockDim.x / 32u;
  const uint32_t warp = threadIdx.x / 32u, lane = threadIdx.x % 32u;
  uint32_t* all = next + warps * stride;
  uint32_t* earlier = all + n;
  const uint32_t first = blockIdx.x * chunk, last = min(first + chunk, slots);
  const uint32_t piece = (last - first + warps * 32u - 1u) / (warps * 32u) * 32u;
  const uint32_t lo = min(first + warp * piece, last), hi = min(lo + piece, last);
  const bool once = hi - lo <= 128u;  // all of the warp's keys are held
  pdl_begin();
  uint32_t key[4];
  sort_keys(ids, lo, hi, E, n, key);
  for (uint32_t i = threadIdx.x; i < warps * stride; i += blockDim.x) next[i] = 0u;
  if (threadIdx.x == 0) carry = 0u;
  if (counts != nullptr)
    for (uint32_t e0 = warp; e0 < n; e0 += kSortAtOnce * warps) {
      uint32_t total[kSortAtOnce] = {}, before[kSortAtOnce] = {};
      for (uint32_t c0 = 0; c0 < gridDim.x; c0 += 128u) {
        uint32_t v[kSortAtOnce][4];
#pragma unroll
        for (uint32_t x = 0; x < kSortAtOnce; ++x)
#pragma unroll
          for (uint32_t i = 0; i < 4u; ++i) {
            const uint32_t e = e0 + x * warps, c = c0 + lane + 32u * i;
            v[x][i] = e < n && c < gridDim.x ? counts[(size_t)e * gridDim.x + c] : 0u;
          }
#pragma unroll
        for (uint32_t x = 0; x < kSortAtOnce; ++x)
#pragma unroll
          for (uint32_t i = 0; i < 4u; ++i) {
            total[x] += v[x][i];
            before[x] += c0 + lane + 32u * i < blockIdx.x ? v[x][i] : 0u;
          }
      }
#pragma unroll
      for (uint32_t x = 0; x < kSortAtOnce; ++x) {
        const uint32_t t = __reduce_add_sync(0xFFFFFFFFu, total[x]);
        const uint32_t u = __reduce_add_sync(0xFFFFFFFFu, before[x]);
        if (lane == 0 && e0 + x * warps < n) all[e0 + x * warps] = t, earlier[e0 + x * warps] = u;
      }
    }
  __syncthreads();
  uint32_t* mine = next + warp * stride;
  for (uint32_t s0 = lo; s0 < hi; s0 += 128u) {
    if (!once) sort_keys(ids, s0, hi, E, n, key);
#pragma unroll
    for (uint32_t i = 0; i < 4u; ++i)
      if (key[i] < n) atomicAdd(&mine[key[i]], 1u);
  }
  __syncthreads();
  const bool few = warps <= 8u;  // warps, whose counters of an expert a thread walks
  if (counts == nullptr && !few) {  // this CTA's counts are all there are
    for (uint32_t e = warp; e < n; e += warps) {
      const uint32_t t = __reduce_add_sync(0xFFFFFFFFu, lane < warps ? next[lane * stride + e] : 0u);
      if (lane == 0) all[e] = t;
    }
    __syncthreads();
  }
  // exclusive scan of the totals over the CTA: earlier[e] becomes the chunk's
  // first row of expert e
  for (uint32_t e0 = 0; e0 < n; e0 += blockDim.x) {
    const uint32_t e = e0 + threadIdx.x;
    uint32_t total = 0u;
    if (e < n) {
      if (counts != nullptr || !few)
        total = all[e];
      else
        for (uint32_t w = 0; w < warps; ++w) total += next[w * stride + e];
    }
    uint32_t sum = total;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= (uint32_t)d) sum += v;
    }
    if (lane == 31u) part[warp] = sum;
    __syncthreads();
    const uint32_t before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? part[lane] : 0u);
    const uint32_t at = carry + before + sum - total;
    __syncthreads();
    if (threadIdx.x == blockDim.x - 1u) carry = at + total;
    if (e < n) {
      if (blockIdx.x == 0) offsets[e] = (int64_t)at;
      uint32_t row = counts != nullptr ? at + earlier[e] : at;
      if (few)
        for (uint32_t w = 0; w < warps; ++w) {
          const uint32_t v = next[w * stride + e];
          next[w * stride + e] = row;
          row += v;
        }
      else
        earlier[e] = row;
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) offsets[n] = (int64_t)slots;
  if (!few) {  // of each expert the warps' counters, a lane each
    for (uint32_t e = warp; e < n; e += warps) {
      const uint32_t v = lane < warps ? next[lane * stride + e] : 0u;
      uint32_t sum = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= (uint32_t)d) sum += u;
      }
      if (lane < warps) next[lane * stride + e] = earlier[e] + sum - v;
    }
    __syncthreads();
  }
  const uint32_t bits = 32u - (uint32_t)__clz((int)n);
  for (uint32_t s0 = lo; s0 < hi; s0 += 128u) {
    if (!once) sort_keys(ids, s0, hi, E, n, key);
#pragma unroll
    for (uint32_t i = 0; i < 4u; ++i) {
      if (s0 + 32u * i >= hi) break;
      const uint32_t s = s0 + 32u * i + lane, e = key[i];
      const uint32_t same = same_key(e, bits);
      if (e < n) {
        const uint32_t r = mine[e] + __popc(same & ((1u << lane) - 1u));
        rows[s] = e < E ? (int32_t)r : -1;
        slot_of[r] = e < E ? (int32_t)s : -1;
      }
      __syncwarp();
      if (e < n && lane == (uint32_t)__ffs((int)same) - 1u) mine[e] += __popc(same);
      __syncwarp();
    }
  }
}

// The work of one warp in the token kernels: 512 columns (32 bytes per lane)
// of one token.
struct MoeShape {
  uint32_t tokens, k, slots;
  uint32_t lanes;  // 32-byte words per row
  uint32_t segs;   // warps per row
};

// Tokens into expert order: y[rows[t, j]] = x[t], each x word read once;
// rows without a slot are zeroed by the warp of the token with that number.
__global__ void __launch_bounds__(kThreads)
    k_moe_dispatch(const V8* __restrict__ x, MoeShape sh, const int32_t* __restrict__ rows,
                   const int32_t* __restrict__ slot_of, V8* __restrict__ y) {
  pdl_begin();
  const uint32_t lane = threadIdx.x % 32u;
  const u64 units = (u64)sh.tokens * sh.segs;
  for (u64 u = (u64)blockIdx.x * (kThreads / 32) + threadIdx.x / 32u; u < units;
       u += (u64)gridDim.x * (kThreads / 32)) {
    const uint32_t t = (uint32_t)(u / sh.segs), w = (uint32_t)(u % sh.segs) * 32u + lane;
    const bool in = w < sh.lanes;
    const V8 v = in ? ld_block_stream(x + (size_t)t * sh.lanes + w) : zero_block();
    for (uint32_t j = 0; j < sh.k; ++j) {
      const uint32_t s = t * sh.k + j;
      const int32_t r = rows[s];
      if (in && (uint32_t)r < sh.slots) st_block(y + (size_t)r * sh.lanes + w, v);
      if (in && slot_of[s] < 0) st_block(y + (size_t)s * sh.lanes + w, zero_block());
    }
  }
}

// Back to token order: out[t] = sum_j weights[t, j] y[rows[t, j]] in fp32, in
// the order of j, rounded once; weights == NULL sums with weight one (the
// gradient of dispatch).  Bound by reads of rows in no order: 302 MB (8192 x 8
// rows of 2048) in 59 us.  Two CTAs per SM, each warp with eight rows of 1 KB
// on their way, and a walk over the units that reads the next row numbers
// early; a CTA for every eight units (32 per SM) takes 67 us, half as many
// columns per warp with twice the warps 61 us.
constexpr int kCombinePerSm = 2;
__global__ void __launch_bounds__(kThreads, kCombinePerSm)
    k_moe_combine(const V8* __restrict__ y, MoeShape sh, const int32_t* __restrict__ rows,
                  const float* __restrict__ weights, V8* __restrict__ out) {
  constexpr uint32_t kBatch = 8u;  // rows on their way at a time
  pdl_begin();
  const uint32_t lane = threadIdx.x % 32u;
  const u64 units = (u64)sh.tokens * sh.segs, stride = (u64)gridDim.x * (kThreads / 32);
  u64 u = (u64)blockIdx.x * (kThreads / 32) + threadIdx.x / 32u;
  // Lane j holds the row number and weight of choice j of a batch for all; a
  // unit's first ones are read while the unit before it waits for its rows.
  int32_t row = -1;
  float f = 0.0f;
  auto choices = [&](uint32_t t, uint32_t j0) {
    const uint32_t s = t * sh.k + j0 + lane;
    const bool has = lane < kBatch && j0 + lane < sh.k;
    row = has ? rows[s] : -1;
    f = weights == nullptr ? 1.0f : has ? weights[s] : 0.0f;
  };
  if (u < units) choices((uint32_t)(u / sh.segs), 0u);
  for (; u < units; u += stride) {
    const uint32_t t = (uint32_t)(u / sh.segs), w = (uint32_t)(u % sh.segs) * 32u + lane;
    const bool in = w < sh.lanes;
    float acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
    for (uint32_t j0 = 0; j0 < sh.k; j0 += kBatch) {
      if (j0 > 0u) choices(t, j0);
      const int32_t my_row = row;
      const float my_f = f;
      V8 v[kBatch];
#pragma unroll
      for (uint32_t q = 0; q < kBatch; ++q) {
        const uint32_t r = (uint32_t)__shfl_sync(0xFFFFFFFFu, my_row, q);
        if (in && r < sh.slots) v[q] = ld_block_stream(y + (size_t)r * sh.lanes + w);
      }
      if (j0 + kBatch >= sh.k && u + stride < units)
        choices((uint32_t)((u + stride) / sh.segs), 0u);
#pragma unroll
      for (uint32_t q = 0; q < kBatch; ++q) {
        const uint32_t r = (uint32_t)__shfl_sync(0xFFFFFFFFu, my_row, q);
        const float wq = __shfl_sync(0xFFFFFFFFu, my_f, q);
        if (!(in && r < sh.slots)) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          acc[2 * i] = __fmaf_rn(wq, bf16_lo(v[q].w[i]), acc[2 * i]);
          acc[2 * i + 1] = __fmaf_rn(wq, bf16_hi(v[q].w[i]), acc[2 * i + 1]);
        }
      }
    }
    if (!in) continue;
    V8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.w[i] = cvt_bf16x2(acc[2 * i], acc[2 * i + 1]);
    st_block(out + (size_t)t * sh.lanes + w, o);
  }
}

// Gradients of combine, one warp per slot (the k slots of a token are
// neighbours, so its dout row comes from L1 after the first):
// dy[rows[s]] = weights[s] dout[t], dweights[s] = <dout[t], y[rows[s]]> in
// fp32 (each lane in column order, then a fixed tree).
__global__ void __launch_bounds__(kThreads)
    k_moe_combine_bwd(const V8* __restrict__ dout, const V8* __restrict__ y, MoeShape sh,
                      const int32_t* __restrict__ rows, const int32_t* __restrict__ slot_of,
                      const float* __restrict__ weights, V8* __restrict__ dy,
                      float* __restrict__ dweights) {
  pdl_begin();
  const uint32_t lane = threadIdx.x % 32u;
  for (uint32_t s = blockIdx.x * (kThreads / 32) + threadIdx.x / 32u; s < sh.slots;
       s += gridDim.x * (kThreads / 32)) {
    const uint32_t t = s / sh.k;
    const int32_t r = rows[s];
    const bool live = (uint32_t)r < sh.slots;
    float dot = 0.0f;
    if (live) {
      const float f = weights[s];
      for (uint32_t w = lane; w < sh.lanes; w += 32u) {
        const V8 a = ld_block_l1(dout + (size_t)t * sh.lanes + w);
        const V8 b = ld_block_stream(y + (size_t)r * sh.lanes + w);
        V8 o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dot = __fmaf_rn(bf16_lo(a.w[i]), bf16_lo(b.w[i]), dot);
          dot = __fmaf_rn(bf16_hi(a.w[i]), bf16_hi(b.w[i]), dot);
          o.w[i] = cvt_bf16x2(f * bf16_lo(a.w[i]), f * bf16_hi(a.w[i]));
        }
        st_block(dy + (size_t)r * sh.lanes + w, o);
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, d);
    if (lane == 0) dweights[s] = dot;
    if (slot_of[s] < 0)
      for (uint32_t w = lane; w < sh.lanes; w += 32u)
        st_block(dy + (size_t)s * sh.lanes + w, zero_block());
  }
}
