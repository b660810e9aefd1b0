// matmul.cuh -- the product of two captured FP4 operands, dense or grouped.
// Included by trace_fp4.cu inside its anonymous namespace.
#pragma once

struct MmShape {
  int64_t rows, n;
  uint32_t cols;
  int32_t groups, matrices;
  int a_tiled, w_tiled;
};

// Scale byte (r, c) of a [rows, scols] scale matrix in either layout.
__device__ __forceinline__ size_t scale_at(int64_t r, uint32_t c, uint32_t scols, int tiled) {
  if (!tiled) return (size_t)r * scols + c;
  return ((size_t)(r / 128) * ((scols + 3u) / 4u) + c / 4u) * 512u + (size_t)(r % 32) * 16u +
         (size_t)(r % 128 / 32) * 4u + c % 4u;
}

__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const uint32_t m = c & 7u;
  const float v = m < 2u ? 0.5f * (float)m : (float)(2u + (m & 1u)) * (float)(1u << (m >> 1)) * 0.25f;
  return c & 8u ? -v : v;
}

template <bool MX>
__device__ __forceinline__ float scale_value(uint32_t b) {
  if (MX) return b == 0u ? 0x1p-127f : __uint_as_float(b << 23);
  float v, unused;
  e4m3x2_to_f32(b, v, unused);
  return v;
}

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

// One output per thread, straight from the definition.
template <bool MX>
__global__ void k_matmul_simple(const uint8_t* __restrict__ ac, const uint8_t* __restrict__ as,
                                const float* __restrict__ ag, const int64_t* __restrict__ offs,
                                const uint8_t* __restrict__ wc, const uint8_t* __restrict__ ws,
                                const float* __restrict__ wg, MmShape sh,
                                uint16_t* __restrict__ out) {
  pdl_begin();
  const uint32_t bs = MX ? 32u : 16u, scols = sh.cols / bs;
  const uint64_t total = (uint64_t)sh.rows * (uint64_t)sh.n;
  for (uint64_t i = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (uint64_t)gridDim.x * blockDim.x) {
    const int64_t r = (int64_t)(i / (uint64_t)sh.n), j = (int64_t)(i % (uint64_t)sh.n);
    int32_t g = 0;
    if (offs != nullptr) {
      int32_t lo = 0, hi = sh.groups;  // the first group whose end is past r
      while (lo < hi) {
        const int32_t mid = (lo + hi) / 2;
        if (offs[mid + 1] > r) hi = mid; else lo = mid + 1;
      }
      g = lo;
      if (g == sh.groups) continue;
    }
    float acc = 0.0f;
    if (g < sh.matrices) {
      const int64_t wr = (int64_t)g * sh.n + j;
      for (uint32_t b = 0; b < scols; ++b) {
        const float sa = scale_value<MX>(as[scale_at(r, b, scols, sh.a_tiled)]);
        const float sw = scale_value<MX>(ws[scale_at(wr, b, scols, sh.w_tiled)]);
        float sum = 0.0f;
        for (uint32_t q = 0; q < bs / 2u; ++q) {
          const uint32_t x = ac[(size_t)r * (sh.cols / 2u) + b * (bs / 2u) + q];
          const uint32_t y = wc[(size_t)wr * (sh.cols / 2u) + b * (bs / 2u) + q];
          sum = __fmaf_rn(e2m1_value(x & 15u), e2m1_value(y & 15u), sum);
          sum = __fmaf_rn(e2m1_value(x >> 4), e2m1_value(y >> 4), sum);
        }
        acc = __fmaf_rn(sum, sa * sw, acc);
      }
      if (!MX) acc = make_out_scale(ag[g], wg[g]).apply(acc);
    }
    out[i] = (uint16_t)cvt_bf16x2(acc, 0.0f);
  }
}
