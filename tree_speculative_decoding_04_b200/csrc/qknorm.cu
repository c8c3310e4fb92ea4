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
// Bound by HBM for large batches (each element is read once and written once),
// by the launch for small ones.
#include <algorithm>

#include "tv_common.cuh"

namespace tv {
namespace {

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
// chunks of it: the two ends of eight rotated pairs, or two chunks past R.
template <int D>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const __grid_constant__ QkNormParams p) {
  constexpr int kLanes = D / 16;
  pdl_wait_primary();
  pdl_launch_dependents();
  __shared__ float cs[D / 2], sn[D / 2];
  const int n = p.M + 1;
  const int64_t row = blockIdx.x;
  const int b = (int)(row / n), r = (int)(row % n);
  const int sl = cache_slot(p.slot, b, p.n_slots);
  if (sl < 0) return;
  const int32_t ks = p.kv_start[sl], kl = p.kv_len[sl];
  if (!geometry_ok(ks, kl, p.M, p.S_cap)) return;
  const int half = p.R / 2;
  if ((int)threadIdx.x < half)
    rope_cos_sin(kl + p.depth[row], p.rope.f[threadIdx.x], cs[threadIdx.x], sn[threadIdx.x]);
  __syncthreads();

  const int c = threadIdx.x % kLanes;
  const bool rot = c < p.R / 16;
  const int c0 = rot ? c : 2 * c;          // past R: chunks R/8 + 2 (c - R/16) and the next
  const int c1 = rot ? c + p.R / 16 : 2 * c + 1;
  const int heads = p.Hq + 2 * p.Hkv;
  for (int h = threadIdx.x / kLanes; h < (heads + 7) / 8 * 8; h += blockDim.x / kLanes) {
    const bool in = h < heads;  // whole warps stay together for the shuffles
    const uint4* src = reinterpret_cast<const uint4*>(p.qkv + row * p.stride + (int64_t)h * D);
    const uint4 a = in ? src[c0] : make_uint4(0, 0, 0, 0);
    const uint4 e = in ? src[c1] : make_uint4(0, 0, 0, 0);
    float x[8], y[8];
    unpack8(a, x);
    unpack8(e, y);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += x[i] * x[i] + y[i] * y[i];
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    if (!in) continue;
    if (h >= p.Hq + p.Hkv) {
      uint4* dst = reinterpret_cast<uint4*>(p.v + (((int64_t)sl * p.Hkv + h - p.Hq - p.Hkv) * p.S_cap + ks + kl + r) * D);
      dst[c0] = a;
      dst[c1] = e;
      continue;
    }
    const float inv = rsqrtf(ss * (1.f / D) + p.eps);
    const uint16_t* wt = h < p.Hq ? p.q_weight : p.k_weight;
    float w0[8], w1[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w0[i] = w1[i] = 1.f;
    if (wt) {
      unpack8(reinterpret_cast<const uint4*>(wt)[c0], w0);
      unpack8(reinterpret_cast<const uint4*>(wt)[c1], w1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w0[i] += p.offset;
        w1[i] += p.offset;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s = x[i] * inv * w0[i], t = y[i] * inv * w1[i];
      if (rot) {
        const float co = cs[8 * c + i], si = sn[8 * c + i];
        const float s2 = fmaf(s, co, -t * si);
        t = fmaf(t, co, s * si);
        s = s2;
      }
      x[i] = s;
      y[i] = t;
    }
    uint4* dst = h < p.Hq
                     ? reinterpret_cast<uint4*>(p.q_out + (row * p.Hq + h) * D)
                     : reinterpret_cast<uint4*>(p.k + (((int64_t)sl * p.Hkv + h - p.Hq) * p.S_cap + ks + kl + r) * D);
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
  return launch(kern, dim3((unsigned)rows), dim3(256), 0, s, 1, true, p);
}
