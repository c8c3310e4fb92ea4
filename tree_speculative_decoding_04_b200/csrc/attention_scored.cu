// attention_scored.cu -- tree_attention_scored: tree attention whose scores are
// capped by a tanh, limited to a window of positions or biased by distance.
//
// "EAGLE-Pangu: Accelerator-Safe Tree Speculative Decoding on Ascend NPUs",
// methodology C (tree mask), and "Batch Speculative Decoding Done Right",
// methodology (position-ID contiguity): node u sits at position kv_len +
// depth(u), prefix column j at position j, so distances inside the tree are
// differences of depth.
//
// One warp per query row; an online softmax over the keys of the row.
#include <algorithm>

#include "tv_common.cuh"

namespace tv {
namespace {

struct ScoredParams {
  const uint16_t *q, *k, *v;
  const int32_t *kv_start, *kv_len, *depth, *slot;
  const uint32_t* anc;
  int32_t* status;
  const float* slopes;
  uint16_t* out;
  int64_t S_cap, rows;
  int M, Hq, Hkv, G, W, n_slots, window;
  float scale, cap;
};

template <int D>
__global__ void __launch_bounds__(128) scored_rows_kernel(const __grid_constant__ ScoredParams p) {
  constexpr int E = D / 32;
  pdl_wait_primary();
  pdl_launch_dependents();
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= p.rows) return;
  const int n = p.M + 1;
  const int h = (int)(row % p.Hq);
  const int64_t node = row / p.Hq;
  const int b = (int)(node / n);
  const int sl = cache_slot(p.slot, b, p.n_slots);
  const int32_t ks = sl >= 0 ? p.kv_start[sl] : -1, kl = sl >= 0 ? p.kv_len[sl] : 0;
  float o[E], qv[E];
  float m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  if (p.status[b] == 0 && geometry_ok(ks, kl, p.M, p.S_cap)) {
    const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(p.q) + row * D + lane * E;
    for (int e = 0; e < E; ++e) qv[e] = __bfloat162float(q[e]);
    const int64_t base = (((int64_t)sl * p.Hkv + h / p.G) * p.S_cap + ks) * D + lane * E;
    const __nv_bfloat16* K = reinterpret_cast<const __nv_bfloat16*>(p.k) + base;
    const __nv_bfloat16* V = reinterpret_cast<const __nv_bfloat16*>(p.v) + base;
    const int du = p.depth ? p.depth[node] : 0;
    const float slope = p.slopes ? p.slopes[h] : 0.f;
    const int first = p.window > 0 ? (int)max((int64_t)0, (int64_t)kl + du - p.window + 1) : 0;
    for (int j = first; j < kl + n; ++j) {
      int dist = kl + du - j;
      if (j >= kl) {
        const int r = j - kl;
        if (!((p.anc[node * p.W + (r >> 5)] >> (r & 31)) & 1u)) continue;
        dist = du - (p.depth ? p.depth[(int64_t)b * n + r] : 0);
        if (p.window > 0 && dist >= p.window) continue;
      }
      float s = 0.f;
      for (int e = 0; e < E; ++e) s += qv[e] * __bfloat162float(K[(int64_t)j * D + e]);
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      s *= p.scale;
      if (p.cap > 0.f) s = p.cap * tanhf(s / p.cap);
      s -= slope * (float)dist;
      const float mn = fmaxf(m, s);
      const float cr = m == -INFINITY ? 0.f : expf(m - mn), w = expf(s - mn);
      l = l * cr + w;
      for (int e = 0; e < E; ++e) o[e] = o[e] * cr + w * __bfloat162float(V[(int64_t)j * D + e]);
      m = mn;
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) + row * D + lane * E;
  for (int e = 0; e < E; ++e) out[e] = __float2bfloat16_rn(o[e] * inv);
  if (sl < 0 && lane == 0) atomicOr(&p.status[b], kSeqBadGeometry);
}

}  // namespace
}  // namespace tv

extern "C" size_t tree_attention_scored_workspace_size(int B, int M, int Hq, int Hkv, int D, int64_t S_cap,
                                                       int window) {
  return 0;
}

extern "C" tv_status tree_attention_scored(const uint16_t* q, const uint16_t* k, const uint16_t* v, int64_t S_cap,
                                           const int32_t* kv_start, const int32_t* kv_len, const uint32_t* anc_mask,
                                           const int32_t* depth, int32_t* status, int B, int M, int Hq, int Hkv,
                                           int D, float scale, float softcap, int window, const float* alibi_slopes,
                                           uint16_t* out, void* workspace, size_t workspace_bytes,
                                           const int32_t* slot, int n_slots, tv_stream_t stream) {
  using namespace tv;
  if (B < 0 || M < 0 || Hq <= 0 || Hkv <= 0 || S_cap < 0 || !(scale > 0.f) || !isfinite(scale)) return TV_ERR_INVALID_ARG;
  if (Hq % Hkv != 0 || window < 0 || !(softcap >= 0.f) || !isfinite(softcap)) return TV_ERR_INVALID_ARG;
  if (slot && n_slots < 1) return TV_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return TV_ERR_UNSUPPORTED;
  if (M + 1 > kMaxRows || S_cap > 0x7fffffffLL) return TV_ERR_UNSUPPORTED;
  if (B == 0) return TV_OK;
  if (!q || !k || !v || !kv_start || !kv_len || !anc_mask || !status || !out) return TV_ERR_INVALID_ARG;
  if ((window > 0 || alibi_slopes) && !depth) return TV_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return TV_ERR_INVALID_ARG;
  ScoredParams p;
  p.q = q;
  p.k = k;
  p.v = v;
  p.kv_start = kv_start;
  p.kv_len = kv_len;
  p.depth = depth;
  p.slot = slot;
  p.anc = anc_mask;
  p.status = status;
  p.slopes = alibi_slopes;
  p.out = out;
  p.S_cap = S_cap;
  p.M = M;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.W = (M + 1 + 31) / 32;
  p.n_slots = slot ? n_slots : B;
  p.window = window;
  p.scale = scale;
  p.cap = softcap;
  p.rows = (int64_t)B * (M + 1) * Hq;
  const int64_t blocks = (p.rows + 3) / 4;
  if (blocks > 0x7fffffffLL) return TV_ERR_UNSUPPORTED;
  auto kern = D == 64 ? scored_rows_kernel<64> : scored_rows_kernel<128>;
  return launch(kern, dim3((unsigned)blocks), dim3(128), 0, reinterpret_cast<cudaStream_t>(stream), 1, true, p);
}
