// sample.cu -- tree_accept_sample: each tree node's next token is drawn from
// the teacher's filtered distribution (temperature, top-k, top-p, min-p) with a
// given random number, then the longest path whose drafts are the drawn tokens
// is accepted.  Every token that leaves the step is so a draw of the teacher
// itself, whatever the draft proposed.
//
// Definition, for a row l with m = max l, in the order (l descending, index
// ascending): w = exp((l - m) / T); the kept tokens are a prefix of that order
// (top-k: the first k; top-p: while the weight before a token is below p times
// the top-k tokens' weight; min-p: while w >= min_p; the first always); the
// drawn token is the first kept one, in vocabulary order, whose inclusive
// weight exceeds u times the kept weight.
//
// A prefix is named by its last key t (a float's order-preserving bits) and the
// number c of tokens equal to t that belong to it.  Weights are formed in double
// precision and summed as 64-bit fixed-point integers: the sums do not depend
// on the order or the split of the work, and their error is far below the
// weight of any token that can be drawn.
#include <algorithm>

#include "tv_common.cuh"

namespace tv {
namespace {

constexpr int kSampleThreads = 512;
constexpr int kMaxVocab = 1 << 18;  // fixed-point weights of one row stay below 2^63

struct SampleParams {
  const void* logits;
  int64_t stride;
  int V, n;
  const float* uniform;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* token;
  float* logprob;
  int shift;  // weight 1 is 2^shift
};

__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

template <typename T>
__device__ __forceinline__ T block_sum(T v, T* red) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  T s = 0;
  for (int i = 0; i < kSampleThreads / 32; ++i) s += red[i];
  return s;
}

template <bool BF16>
struct Row {
  const void* base;
  int V;
  float m;
  double c;  // log2(e) / T
  int shift;
  // NaN counts as -inf (never drawn); -0 as +0
  __device__ __forceinline__ float at(int i) const {
    float x;
    if (BF16)
      x = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base)[i]);
    else
      x = reinterpret_cast<const float*>(base)[i];
    return x == x ? x + 0.f : -INFINITY;
  }
  __device__ __forceinline__ unsigned long long weight(float x) const {
    if (x == m) return 1ull << shift;
    if (x == -INFINITY || m == INFINITY) return 0ull;
    return (unsigned long long)__double2ull_rn(exp2(((double)x - (double)m) * c) * (double)(1ull << shift));
  }
};

// One CTA per row.
template <bool BF16>
__global__ void __launch_bounds__(kSampleThreads) sample_kernel(const __grid_constant__ SampleParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  typedef unsigned long long u64;
  __shared__ u64 red[kSampleThreads / 32];
  __shared__ float redf[kSampleThreads / 32];
  __shared__ u64 seg[kSampleThreads];
  __shared__ int cnt[kSampleThreads];
  __shared__ int s_tok;
  const int64_t row = blockIdx.x;
  const int b = (int)(row / p.n), tid = threadIdx.x;
  Row<BF16> r;
  r.base = BF16 ? (const void*)(reinterpret_cast<const uint16_t*>(p.logits) + row * p.stride)
                : (const void*)(reinterpret_cast<const float*>(p.logits) + row * p.stride);
  r.V = p.V;
  r.shift = p.shift;
  float mx = -INFINITY;
  for (int i = tid; i < p.V; i += kSampleThreads) mx = fmaxf(mx, r.at(i));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
  if ((tid & 31) == 0) redf[tid >> 5] = mx;
  if (tid == 0) s_tok = p.V;
  __syncthreads();
  for (int i = 0; i < kSampleThreads / 32; ++i) mx = fmaxf(mx, redf[i]);
  r.m = mx;
  if (mx == -INFINITY) {  // no token can be drawn
    if (tid == 0) {
      p.token[row] = -1;
      if (p.logprob) p.logprob[row] = -INFINITY;
    }
    return;
  }
  const float T = p.temperature[b];
  const bool greedy = !(T > 0.f);
  r.c = greedy ? 1.0 : 1.4426950408889634 / (double)T;
  const int k = greedy ? 1 : (p.top_k ? p.top_k[b] : 0);
  const float tp = p.top_p ? p.top_p[b] : 1.f, mp = p.min_p ? p.min_p[b] : 0.f;

  uint32_t t = 0;
  int c = p.V;  // keys above t, and the first c tokens with key t
  const uint32_t mkey = order_key(mx);
  if (k > 0 && k < p.V) {
    u64 above = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t mid = t | (1u << bit);
      u64 cn = 0;
      for (int i = tid; i < p.V; i += kSampleThreads) cn += order_key(r.at(i)) >= mid;
      cn = block_sum(cn, red);
      if (cn >= (u64)k) t = mid;
      else above = cn;
    }
    u64 cn = 0;
    for (int i = tid; i < p.V; i += kSampleThreads) cn += order_key(r.at(i)) > t;
    c = k - (int)block_sum(cn, red);
  }
  if (tp < 1.f) {
    if (!(tp > 0.f)) {
      t = mkey;
      c = 1;
    } else {
      // mass(lo): weight of the kept tokens with key >= lo, and above it
      auto mass_above = [&](uint32_t lo) {
        u64 s = 0;
        for (int i = tid; i < p.V; i += kSampleThreads) {
          const float x = r.at(i);
          if (order_key(x) > lo) s += r.weight(x);
        }
        return block_sum(s, red);
      };
      auto ties = [&](uint32_t key) {
        u64 s = 0;
        for (int i = tid; i < p.V; i += kSampleThreads) s += order_key(r.at(i)) == key;
        return block_sum(s, red);
      };
      const u64 ct = min((u64)c, ties(t));
      const u64 at = mass_above(t), wt = r.weight(key_value(t));
      const double pz = (double)tp * (double)(at + ct * wt);
      uint32_t t2 = t;
      u64 ct2 = ct, a2 = at;
      if ((double)at >= pz) {  // the boundary lies above t
        uint32_t lo = 0;       // largest key with mass(key >= lo) >= pz
        for (int bit = 31; bit >= 0; --bit) {
          const uint32_t mid = lo | (1u << bit);
          if (mid <= t || (double)mass_above(mid - 1) >= pz) lo = mid;
        }
        t2 = lo;
        a2 = mass_above(t2);
        ct2 = ties(t2);
      }
      const u64 w2 = r.weight(key_value(t2));
      // ties kept while the weight before them is below pz
      u64 l = 0, h = ct2;
      while (l < h) {
        const u64 mid = (l + h) / 2;
        if ((double)(a2 + mid * w2) < pz) l = mid + 1;
        else h = mid;
      }
      t = t2;
      c = (int)l;
    }
  }
  if (mp > 0.f) {
    if (mp > 1.f) {
      t = mkey;
      c = 1;
    } else {
      const float cut = __double2float_ru((double)mx + log2((double)mp) / r.c);
      const uint32_t ck = order_key(cut + 0.f);
      if (ck > t) {
        t = min(ck, mkey);
        c = p.V;
      }
    }
  }
  // the draw, in vocabulary order: thread tid owns a contiguous segment
  const int per = (p.V + kSampleThreads - 1) / kSampleThreads;
  const int lo = min(p.V, tid * per), hi = min(p.V, lo + per);
  const u64 wt = r.weight(key_value(t));
  u64 s = 0;
  int nt = 0;
  for (int i = lo; i < hi; ++i) {
    const float x = r.at(i);
    const uint32_t key = order_key(x);
    if (key > t) s += r.weight(x);
    nt += key == t;
  }
  __syncthreads();
  seg[tid] = s;
  cnt[tid] = nt;
  __syncthreads();
  u64 before = 0, total = 0;
  int tb = 0, ta = 0;
  for (int i = 0; i < kSampleThreads; ++i) {
    const int kept = max(0, min(cnt[i], c - ta));
    const u64 w = seg[i] + kept * wt;
    if (i < tid) {
      before += w;
      tb += cnt[i];
    }
    total += w;
    ta += cnt[i];
  }
  const double target = (double)p.uniform[row] * (double)total;
  int found = p.V, last = -1;
  u64 cum = before;
  for (int i = lo; i < hi; ++i) {
    const float x = r.at(i);
    const uint32_t key = order_key(x);
    u64 w = 0;
    if (key > t) w = r.weight(x);
    else if (key == t && tb++ < c) w = wt;
    if (w == 0) continue;
    last = i;
    cum += w;
    if (found == p.V && (double)cum > target) found = i;
  }
  if (found < p.V) atomicMin(&s_tok, found);
  __syncthreads();
  cnt[tid] = last;
  __syncthreads();
  if (tid == 0) {
    int tok = s_tok;
    if (tok == p.V)
      for (int i = 0; i < kSampleThreads; ++i) tok = cnt[i] >= 0 ? cnt[i] : tok;
    const float x = r.at(tok);
    p.token[row] = tok;
    if (p.logprob)
      p.logprob[row] = (float)((x == mx ? 0.0 : ((double)x - (double)mx) * r.c * 0.6931471805599453) -
                               log((double)total / (double)(1ull << p.shift)));
  }
}

}  // namespace
}  // namespace tv

extern "C" size_t tree_accept_sample_workspace_size(int B, int M, int V) {
  return B > 0 && M >= 0 && V > 0 ? 16 : 0;
}

extern "C" tv_status tree_accept_sample(const void* logits, int logits_type, int64_t logits_stride,
                                        const float* uniform, const float* temperature, const int32_t* top_k,
                                        const float* top_p, const float* min_p, const int32_t* draft,
                                        const int32_t* parent, const int32_t* depth, const uint32_t* anc_mask,
                                        int32_t* status, int B, int M, int V, int max_depth, int32_t* token,
                                        float* logprob, int32_t* accept_len, int32_t* path, int32_t* bonus,
                                        void* workspace, size_t workspace_bytes, tv_stream_t stream) {
  using namespace tv;
  if (B < 0 || M < 0 || V < 1 || max_depth < 0 || logits_stride < V) return TV_ERR_INVALID_ARG;
  if (logits_type != TV_LOGITS_F32 && logits_type != TV_LOGITS_BF16) return TV_ERR_INVALID_ARG;
  if (M + 1 > kMaxRows || V > kMaxVocab) return TV_ERR_UNSUPPORTED;
  if (B == 0) return TV_OK;
  if (!logits || !uniform || !temperature || !draft || !parent || !depth || !anc_mask || !status || !token ||
      !accept_len || !path || !bonus)
    return TV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(logits) & (logits_type == TV_LOGITS_F32 ? 3u : 1u)) != 0) return TV_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)B * (M + 1);
  if (rows > 0x7fffffffLL) return TV_ERR_UNSUPPORTED;
  if (!workspace || !aligned16(workspace) || workspace_bytes < tree_accept_sample_workspace_size(B, M, V))
    return TV_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  SampleParams p;
  p.logits = logits;
  p.stride = logits_stride;
  p.V = V;
  p.n = M + 1;
  p.uniform = uniform;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.token = token;
  p.logprob = logprob;
  p.shift = V <= (1 << 17) ? 46 : 45;
  auto kern = logits_type == TV_LOGITS_F32 ? sample_kernel<false> : sample_kernel<true>;
  tv_status r = launch(kern, dim3((unsigned)rows), dim3(kSampleThreads), 0, s, 1, true, p);
  if (r != TV_OK) return r;
  return launch_accept_walk(token, draft, parent, depth, anc_mask, status, B, M, max_depth, accept_len, path, bonus,
                            s);
}
