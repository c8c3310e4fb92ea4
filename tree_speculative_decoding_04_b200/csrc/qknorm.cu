// qknorm.cu -- tree_qk_norm_rope: the packed projection rows of the step's M+1
// tree nodes become attention-ready queries and cache rows in one pass: every
// query and key head is normalised by its root mean square, scaled by its
// weight and rotated to its node's tree position, and the key and value heads
// go straight to the cache columns behind the committed prefix.
//
// Tree positions kv_len + depth: "Batch Speculative Decoding Done Right",
// methodology, position-ID contiguity.  For head x of node u, with R rotated
// elements:
//   y = x / sqrt(mean(x^2) + eps) * (offset + w)
//   (y[i], y[i + R/2]) turns by (kv_len + depth[u]) * theta^(-2i/R), i < R/2
//
// Each element is read once and written once: 84.6 MB for 16 x 129 rows of 64 + 8 + 8
// heads of 128, which take 16.8 us (5.0 TB/s; 13.1 us at the copy rate).  A single token
// takes 2.7 us, a launch's length.
#include <algorithm>

#include "tv_common.cuh"

namespace tv {
namespace {

// Threads of a row's CTA: many while the rows fit the GPU at once (three such CTAs to an
// SM: registers), and few beyond that, so that more rows are in flight and the last wave is
// short.  320 / 128 threads, 64 + 16 heads of 128: 144 rows 3.1 / 3.9 us, 432 rows 4.8 /
// 5.3 us, 576 rows 7.3 / 6.2 us, 2048 rows 19.8 / 16.8 us; 32 + 16 heads of 128, 2048 rows
// 16.7 / 11.7 us.
constexpr int kNormThreads = 320, kNormManyRows = 128, kNormBlocks = 3;

struct QkNormParams {
  const uint16_t* qkv;
  int64_t stride;  // elements between projection rows
  const uint16_t* q_weight;
  const uint16_t* k_weight;
  float offset, eps;
  const int32_t* depth;
  uint16_t* q_out;
  uint16_t* k;
  uint16_t* v;
  int64_t S_cap;
  const int32_t* kv_start;
  const int32_t* kv_len;
  const int32_t* slot;
  int n_slots, M, Hq, Hkv, R;
  RopeFreqs rope;
};

__device__ __forceinline__ void unpack8(const uint4& a, float (&x)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// The bf16 values that x was unpacked from, bit by bit.
__device__ __forceinline__ uint4 bits8(const float (&x)[8]) {
  auto two = [&](int i) { return __byte_perm(__float_as_uint(x[i]), __float_as_uint(x[i + 1]), 0x7632); };
  return make_uint4(two(0), two(2), two(4), two(6));
}

// One CTA per projection row.  D / 16 lanes share a head; each holds two 16-byte
// chunks of it: the two ends of eight rotated pairs, or two chunks past R.  A warp
// takes 512 / D heads at a time and requests the next ones before it works on
// these, the first before the angles and weights are laid out in shared memory.
template <int D>
__global__ void __launch_bounds__(kNormThreads, kNormBlocks) qk_norm_rope_kernel(const __grid_constant__ QkNormParams p) {
  constexpr int kLanes = D / 16, kHeads = 32 / kLanes;
  // Of a pair (x, y) with angle t and weights u, v:  x' = x (u cos t) + y (-v sin t),
  // y' = y (v cos t) + x (u sin t); the four factors of a query's and of a key's pairs,
  // the first four pairs of every lane's eight before the second four (no bank conflicts).
  __shared__ __align__(16) float turn[2][4][D / 2], weight[2][D];
  const int n = p.M + 1;
  const int64_t row = blockIdx.x;
  const int b = (int)(row / n), r = (int)(row - (int64_t)b * n);
  const int half = p.R / 2;
  const int lane = threadIdx.x & 31, step = (blockDim.x >> 5) * kHeads;
  const int c = lane % kLanes;
  const bool rot = c < p.R / 16;
  const int c0 = rot ? c : 2 * c;          // past R: chunks R/8 + 2 (c - R/16) and the next
  const int c1 = rot ? c + p.R / 16 : 2 * c + 1;
  const int heads = p.Hq + 2 * p.Hkv;
  const uint4* src = reinterpret_cast<const uint4*>(p.qkv + row * p.stride);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  pdl_wait_primary();
  pdl_launch_dependents();
  int h = (threadIdx.x >> 5) * kHeads + lane / kLanes;
  uint4 a = h < heads ? __ldg(src + h * (D / 8) + c0) : zero;
  uint4 e = h < heads ? __ldg(src + h * (D / 8) + c1) : zero;
  auto scale = [&](int k, int i) {  // (no weight: a scale of one)
    const uint16_t* w = k ? p.k_weight : p.q_weight;
    return w ? p.offset + __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(w)[i]) : 1.f;
  };
  const int depth = p.depth[row];
  const int sl = cache_slot(p.slot, b, p.n_slots);
  if (sl < 0) return;
  const int32_t ks = p.kv_start[sl], kl = p.kv_len[sl];
  if (!geometry_ok(ks, kl, p.M, p.S_cap)) return;
  for (int i = p.R + threadIdx.x; i < D; i += blockDim.x) {
    weight[0][i] = scale(0, i);
    weight[1][i] = scale(1, i);
  }
  for (int i = threadIdx.x; i < half; i += blockDim.x) {
    float cs, sn;
    rope_cos_sin(kl + depth, p.rope.f[i], cs, sn);
    const int at = ((i >> 2 & 1) * (half / 8) + (i >> 3)) * 4 + (i & 3);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float u = scale(k, i), v = scale(k, i + half);
      turn[k][0][at] = u * cs;
      turn[k][1][at] = -v * sn;
      turn[k][2][at] = v * cs;
      turn[k][3][at] = u * sn;
    }
  }
  __syncthreads();
  const int64_t col = ((int64_t)sl * p.Hkv * p.S_cap + ks + kl + r) * D;  // of the slot's first cache head
  for (int first = 0; first < heads; first += step, h += step) {  // whole warps stay together for the shuffles
    float x[8], y[8];
    unpack8(a, x);
    unpack8(e, y);
    if (h + step < heads) {
      a = __ldg(src + (h + step) * (D / 8) + c0);
      e = __ldg(src + (h + step) * (D / 8) + c1);
    }
    uint64_t ss2 = 0;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const uint64_t u = f2_pack(x[i], x[i + 1]), v = f2_pack(y[i], y[i + 1]);
      ss2 = f2_fma(v, v, f2_fma(u, u, ss2));
    }
    float ss, s1;
    f2_unpack(ss2, ss, s1);
    ss += s1;
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    if (h >= heads) continue;
    if (h >= p.Hq + p.Hkv) {
      uint4* dst = reinterpret_cast<uint4*>(p.v + col + (int64_t)(h - p.Hq - p.Hkv) * p.S_cap * D);
      dst[c0] = bits8(x);
      dst[c1] = bits8(y);
      continue;
    }
    const float inv = rsqrtf(ss * (1.f / D) + p.eps);
    const uint64_t inv2 = f2_pack(inv, inv);
    const bool is_q = h < p.Hq;
    const int kind = is_q ? 0 : 1;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const int at = rot ? (i >> 2) * (half / 8) + c : 0;
      float4 t[4];
      if (rot) {
#pragma unroll
        for (int k = 0; k < 4; ++k) t[k] = reinterpret_cast<const float4*>(turn[kind][k])[at];
      } else {
        t[0] = reinterpret_cast<const float4*>(weight[kind])[2 * c0 + (i >> 2)];
        t[2] = reinterpret_cast<const float4*>(weight[kind])[2 * c1 + (i >> 2)];
        t[1] = t[3] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const uint64_t u = f2_mul(f2_pack(x[i + j], x[i + j + 1]), inv2);
        const uint64_t v = f2_mul(f2_pack(y[i + j], y[i + j + 1]), inv2);
        auto of = [&](int k) { return j ? f2_pack(t[k].z, t[k].w) : f2_pack(t[k].x, t[k].y); };
        f2_unpack(rot ? f2_fma(u, of(0), f2_mul(v, of(1))) : f2_mul(u, of(0)), x[i + j], x[i + j + 1]);
        f2_unpack(rot ? f2_fma(v, of(2), f2_mul(u, of(3))) : f2_mul(v, of(2)), y[i + j], y[i + j + 1]);
      }
    }
    uint4* dst = is_q ? reinterpret_cast<uint4*>(p.q_out + (row * p.Hq + h) * D)
                      : reinterpret_cast<uint4*>(p.k + col + (int64_t)(h - p.Hq) * p.S_cap * D);
    dst[c0] = pack8(x);
    dst[c1] = pack8(y);
  }
}

}  // namespace
}  // namespace tv

extern "C" tv_status tree_qk_norm_rope(const uint16_t* qkv, int64_t qkv_stride, const uint16_t* q_weight,
                                       const uint16_t* k_weight, float weight_offset, float eps, uint16_t* q_out,
                                       uint16_t* k, uint16_t* v, int64_t S_cap, const int32_t* kv_start,
                                       const int32_t* kv_len, const int32_t* depth, int B, int M, int Hq, int Hkv,
                                       int D, int rotary_dim, float rope_theta, const int32_t* slot, int n_slots,
                                       tv_stream_t stream) {
  using namespace tv;
  if (B < 0 || M < 0 || Hq <= 0 || Hkv <= 0 || S_cap < 0 || !(eps >= 0.f) || !isfinite(weight_offset))
    return TV_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return TV_ERR_UNSUPPORTED;
  if (rotary_dim < 0 || rotary_dim > D) return TV_ERR_INVALID_ARG;
  if (rotary_dim % 16 != 0) return TV_ERR_UNSUPPORTED;
  if (rotary_dim > 0 && !(rope_theta > 1.0f && isfinite(rope_theta))) return TV_ERR_INVALID_ARG;
  if (M + 1 > kMaxRows || S_cap > 0x7fffffffLL) return TV_ERR_UNSUPPORTED;
  if (slot && n_slots < 1) return TV_ERR_INVALID_ARG;
  const int64_t width = ((int64_t)Hq + 2 * (int64_t)Hkv) * D;
  if (width > 0x7fffffffLL) return TV_ERR_UNSUPPORTED;
  const int64_t rows = (int64_t)B * (M + 1);
  if (rows > 0x7fffffffLL) return TV_ERR_UNSUPPORTED;
  if (B == 0) return TV_OK;
  if (!qkv || !q_out || !k || !v || !kv_start || !kv_len || !depth) return TV_ERR_INVALID_ARG;
  if (qkv_stride < width || qkv_stride % 8 != 0) return TV_ERR_INVALID_ARG;
  if (!aligned16(qkv) || !aligned16(q_weight) || !aligned16(k_weight) || !aligned16(q_out) || !aligned16(k) ||
      !aligned16(v))
    return TV_ERR_INVALID_ARG;
  QkNormParams p;
  p.qkv = qkv;
  p.stride = qkv_stride;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.offset = weight_offset;
  p.eps = eps;
  p.depth = depth;
  p.q_out = q_out;
  p.k = k;
  p.v = v;
  p.S_cap = S_cap;
  p.kv_start = kv_start;
  p.kv_len = kv_len;
  p.slot = slot;
  p.n_slots = slot ? n_slots : B;
  p.M = M;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.R = rotary_dim;
  // (a program's layers share their base: the last table is kept per thread)
  thread_local struct {
    float theta = 0.f;
    int dim = 0;
    RopeFreqs f;
  } last;
  if (rotary_dim > 0 && (last.theta != rope_theta || last.dim != rotary_dim)) {
    rope_freqs((double)rope_theta, rotary_dim, last.f);
    last.theta = rope_theta;
    last.dim = rotary_dim;
  }
  p.rope = last.f;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto kern = D == 64 ? qk_norm_rope_kernel<64> : qk_norm_rope_kernel<128>;
  int sms = 0;
  const tv_status r = current_sms(sms);
  if (r != TV_OK) return r;
  // a warp per group of heads, as far as the threads go
  const int per_warp = 512 / D, groups = (Hq + 2 * Hkv + per_warp - 1) / per_warp;
  const int warps = std::min((rows > (int64_t)kNormBlocks * sms ? kNormManyRows : kNormThreads) / 32, groups);
  return launch(kern, dim3((unsigned)rows), dim3(32 * warps), 0, s, 1, true, p);
}
