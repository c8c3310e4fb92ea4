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
// heads of 128, which take 20 us (4.2 TB/s, 13.1 us at the copy rate; instruction issue
// 70 % busy: the conversions, weights and rotation of 16 elements a lane).  A single token
// takes 3.3 us, a launch's length.
#include <algorithm>

#include "tv_common.cuh"

namespace tv {
namespace {

constexpr int kNormThreads = 320;

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

// One CTA per projection row.  D / 16 lanes share a head; each holds two 16-byte
// chunks of it: the two ends of eight rotated pairs, or two chunks past R.  A warp
// takes 512 / D heads at a time and requests the next ones before it works on
// these, the first before the angles and weights are laid out in shared memory.
template <int D>
__global__ void __launch_bounds__(kNormThreads, 4) qk_norm_rope_kernel(const __grid_constant__ QkNormParams p) {
  constexpr int kLanes = D / 16, kHeads = 32 / kLanes;
  __shared__ __align__(16) float cs[D / 2], sn[D / 2], weight[2][D];
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
  for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) {  // (no weight: a scale of one)
    const uint16_t* w = i < D ? p.q_weight : p.k_weight;
    weight[i / D][i % D] = w ? p.offset + __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(w)[i % D]) : 1.f;
  }
  const int depth = p.depth[row];
  const int sl = cache_slot(p.slot, b, p.n_slots);
  if (sl < 0) return;
  const int32_t ks = p.kv_start[sl], kl = p.kv_len[sl];
  if (!geometry_ok(ks, kl, p.M, p.S_cap)) return;
  for (int i = threadIdx.x; i < half; i += blockDim.x) rope_cos_sin(kl + depth, p.rope.f[i], cs[i], sn[i]);
  __syncthreads();
  const int64_t col = ((int64_t)sl * p.Hkv * p.S_cap + ks + kl + r) * D;  // of the slot's first cache head
  for (int first = 0; first < heads; first += step, h += step) {  // whole warps stay together for the shuffles
    float x[8], y[8];
    unpack8(a, x);
    unpack8(e, y);
    const uint4 a0 = a, e0 = e;
    if (h + step < heads) {
      a = __ldg(src + (h + step) * (D / 8) + c0);
      e = __ldg(src + (h + step) * (D / 8) + c1);
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += x[i] * x[i] + y[i] * y[i];
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    if (h >= heads) continue;
    if (h >= p.Hq + p.Hkv) {
      uint4* dst = reinterpret_cast<uint4*>(p.v + col + (int64_t)(h - p.Hq - p.Hkv) * p.S_cap * D);
      dst[c0] = a0;
      dst[c1] = e0;
      continue;
    }
    const float inv = rsqrtf(ss * (1.f / D) + p.eps);
    const bool is_q = h < p.Hq;
    const float4* w0 = reinterpret_cast<const float4*>(weight[is_q ? 0 : 1]) + 2 * c0;
    const float4* w1 = reinterpret_cast<const float4*>(weight[is_q ? 0 : 1]) + 2 * c1;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 u = w0[i / 4], v = w1[i / 4];
      const float wu[4] = {u.x, u.y, u.z, u.w}, wv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[i + j] *= inv * wu[j];
        y[i + j] *= inv * wv[j];
      }
    }
    if (rot) {
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const float4 u = reinterpret_cast<const float4*>(cs)[2 * c + i / 4];
        const float4 v = reinterpret_cast<const float4*>(sn)[2 * c + i / 4];
        const float co[4] = {u.x, u.y, u.z, u.w}, si[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float s = x[i + j], t = y[i + j];
          x[i + j] = fmaf(s, co[j], -t * si[j]);
          y[i + j] = fmaf(t, co[j], s * si[j]);
        }
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
  // a warp per group of heads, up to kNormThreads: two or three groups each for wide rows
  const int per_warp = 512 / D, groups = (Hq + 2 * Hkv + per_warp - 1) / per_warp;
  const int warps = std::min(kNormThreads / 32, groups);
  return launch(kern, dim3((unsigned)rows), dim3(32 * warps), 0, s, 1, true, p);
}
