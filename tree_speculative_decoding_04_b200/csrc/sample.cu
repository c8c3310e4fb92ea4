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
// Launches, each over the whole GPU:
//   stream  one pass over the logits (a chunk of 1024 per warp, loads of 128 bytes
//           that need no alignment): the maximum of every 128 tokens and, for rows
//           that need the weight of all tokens, each chunk's weight relative to its
//           maximum
//   finish  a block per row.  No filter: the chunk in which the target falls is
//           read again.  Filters: no token below a bound can be kept or matter
//           (top-k: the k-th largest of the 128-token maxima bounds the k-th largest
//           token; top-p: once these maxima alone weigh enough, so do the tokens above
//           them; min-p: its threshold), so only 128-token blocks that reach it are
//           read again; the tokens that do go to a list in shared memory, in
//           vocabulary order (were it to overflow, they are walked in L2 instead),
//           and a radix selection over histograms of (count, weight) finds the kept
//           prefix; up to 256 tokens are simply compared with each other.  Rows whose
//           top-p keeps too many tokens for this go through two more launches:
//   weigh   a histogram of the weights, to 2^-16, over 1/32-octave bins below the row's
//           maximum; the block that brings a row's last segment finds the bins in
//           which the border must lie (one or two)
//   border  a list of the tokens down to the border's bins, or, if those are too many,
//           of the tokens in the border's bins and exact sums of what each chunk keeps
//           for sure; the last block of a row settles the list and draws
//   walk    tree_accept's acceptance walk, on the drawn tokens
// Weights are doubles: a token's share of a flat vocabulary is 2^-18, and a sum in fp32
// would move the borders between tokens by as much.  A weight 2^-e has a relative error
// below 2^-48 (1 + e / 16): the series' remainder is 2^-48.6, and the roundings of l - m and
// of log2e / T move the exponent by 2^-51.5 e at most.  The finish's histograms hold weights
// as 64-bit fixed-point numbers in units of 2^-46 (2^-45 beyond 2^17 tokens), and all other
// sums run in a fixed order, so results do not depend on the order of the work.
//
// What bounds it.  16 x 129 rows of 128256 fp32 logits (1059 MB, 164 us at the copy rate)
// take 248 us with min-p and 297 us with top-k (one pass, 4 TB/s and the finish), 403 us
// at a plain temperature and 1050 us with top-p.  The pass that weighs every token is bound
// by instruction issue (65 %: 29 instructions a token, a double exponential among them;
// 2.6 TB/s), border by that and by the settling of its rows (147 us per 516 rows; stream
// 104, finish 16, weigh 56).  Weighing only the sure tokens there, moved together first,
// was no faster (1077 us).  A few rows are bound by launches and block-wide steps: 8 rows
// of 151936 take 14 us with min-p, 17 at a plain temperature, 22 with top-k and 48 with a
// top-p that keeps too many tokens for the finish.
#include <algorithm>
#include <climits>

#include "tv_common.cuh"

namespace tv {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 1024;             // tokens per warp and pass
constexpr int kSub = 128;                // tokens per recorded maximum
constexpr int kMaxVocab = 1 << 18;       // fixed-point weights of one row stay below 2^63
constexpr int kMaxSubs = kMaxVocab / kSub;
static_assert(kMaxVocab / kChunk <= kThreads, "one thread per chunk in the finish");
constexpr int kListCap = 384;            // listed tokens per warp
constexpr int kBins = 1024;
constexpr int kTab = 32, kTabCopies = 16;

struct RowState;

struct SampleParams {
  const void* logits;
  int64_t stride, rows;
  int V, n, nseg, nsub, nchunk;
  const float* uniform;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* token;
  float* logprob;
  float* sub;    // [rows][nsub] maxima of 128 tokens
  double* sum;   // [rows][nchunk] weight of a chunk relative to its maximum; after border: what it keeps for sure
  // rows whose top-p keeps many tokens
  int* marked;         // [0] how many, [1], [2] segments taken by weigh and border, [4 + i] their rows
  RowState* st;        // [rows]
  u64* hist;           // [rows][kBins] weights in units of 2^-18 of the bin's top
  double* over;        // [rows][nchunk] weight of a chunk's tokens above the border's bins
  float* list_x;       // [rows][kRowList] tokens in the border's bins
  int* list_i;
  int shift;     // weight 1 is 2^shift in the histograms
};

constexpr int kRowList = kWarps * kListCap;

struct RowState {
  double total;           // weight of all tokens
  float m, scale;         // maximum; bins per unit of logit
  int bin0, bin1;         // the border's bins, first and last
  int listed;             // tokens in them
  int weighed, bordered;  // segments that have arrived
};

struct Shared {
  double tab[kTab * kTabCopies];
  double cs;
  double redd[kWarps];
  u64 red[kWarps];
  float sub[kMaxSubs];
  uint32_t cnt[kBins], lo[kBins], hi[kBins];
  float lval[kWarps][kListCap];
  int lidx[kWarps][kListCap];
  uint16_t blk[kWarps][kMaxSubs / kWarps + 32];  // 128-token blocks that a warp reads
  int len[kWarps];
  int found, found2, last, last2;
  u64 found_mass;
};

__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// The table of 2^(i / 32), in 16 copies: lane l reads copy l % 16, whose two banks
// no lane of its half-warp shares.
__device__ __forceinline__ void fill_table(double* tab) {
  for (int i = threadIdx.x; i < kTab * kTabCopies; i += kThreads) tab[i] = exp2((double)(i / kTabCopies) / kTab);
}

// 2^(d c) for -1000 <= d c <= 0, c32 = 32 c: 32 d c = n + r, |r| <= 1/2, with r formed
// from d in one rounding; 2^(r / 32) by the first six terms of its series (the next is
// below 2^-48 of the result), 2^(n / 32) from the table and the exponent field.
__device__ __forceinline__ double pow2_in_range(double d, double c32, const double* tab) {
  const double magic = 6755399441055744.0;  // 1.5 * 2^52: rounds to an integer
  const double t = fma(d, c32, magic);
  const int n = __double2loint(t);
  const double r = fma(d, c32, magic - t);
  // ln2^i / i! / 32^i
  double q = 0.0013333558146428443 / 33554432.0;
  q = fma(q, r, 0.0096181291076284772 / 1048576.0);
  q = fma(q, r, 0.055504108664821580 / 32768.0);
  q = fma(q, r, 0.24022650695910071 / 1024.0);
  q = fma(q, r, 0.69314718055994531 / 32.0);
  const double v = tab[(n & (kTab - 1)) * kTabCopies + (threadIdx.x & (kTabCopies - 1))] * fma(q, r, 1.0);
  return __hiloint2double(__double2hiint(v) + (n >> 5) * (1 << 20), __double2loint(v));
}

// Weight of logit x relative to the maximum m, c = log2(e) / T; 0 below 2^-1000.
// The distance to the maximum comes first: c has no bound (T may be as small as a
// float goes), so a product of c with x or m alone would lose the difference.
__device__ __forceinline__ double weight(float x, float m, double c, const double* tab) {
  if (x == m) return x == -INFINITY ? 0.0 : 1.0;
  if (x == -INFINITY || m == INFINITY) return 0.0;
  const double d = (double)x - (double)m;
  return d * c > -1000.0 ? pow2_in_range(d, kTab * c, tab) : 0.0;
}

// The same without branches, for many tokens of one finite maximum: what lies 900
// octaves below the maximum (-inf and NaN among it) counts as if it lay there.
struct Weigher {
  double m, c32;
  float far;
  // Not where 900 octaves below the maximum is beyond the finite floats, and not where
  // they span fewer than 128 steps of the floats at m: `far`, rounded to a float, would be
  // the maximum itself, or more than 1000 octaves below it.
  static __device__ __forceinline__ bool fits(float m, double c) {
    return m < INFINITY && (double)m - 900.0 / c > -1e38 && fabs((double)m) * c < 900.0 * 65536.0;
  }
  __device__ __forceinline__ Weigher(float m_, double c) : m((double)m_), c32(kTab * c) {
    far = (float)((double)m_ - 900.0 / c);
  }
  __device__ __forceinline__ double operator()(float x, const double* tab) const {
    return pow2_in_range((double)fmaxf(x, far) - m, c32, tab);
  }
};

// NaN counts as -inf (never drawn); -0 as +0
__device__ __forceinline__ float clean(float x) { return x == x ? x + 0.f : -INFINITY; }

template <bool BF16>
__device__ __forceinline__ float logit(const SampleParams& p, int64_t row, int i) {
  if (BF16) return clean(__bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.logits)[row * p.stride + i]));
  return clean(reinterpret_cast<const float*>(p.logits)[row * p.stride + i]);
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ double warp_scan(double v) {  // inclusive
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const double o = __shfl_up_sync(0xffffffffu, v, off);
    if ((int)(threadIdx.x & 31) >= off) v += o;
  }
  return v;
}
__device__ __forceinline__ u64 warp_scan(u64 v) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const u64 o = __shfl_up_sync(0xffffffffu, v, off);
    if ((int)(threadIdx.x & 31) >= off) v += o;
  }
  return v;
}

// 1/32-octave bin of a token below the row's finite maximum (monotone in x), and
// where in it the token lies.
__device__ __forceinline__ int bin_of(float x, float m, float scale, float& frac) {
  const float d = (m - x) * scale;
  const int bin = (int)fminf(d, (float)(kBins - 1));
  frac = d - (float)bin;
  return bin;
}

// Settings of a row's sequence.
struct Rule {
  float T, top_p, min_p;
  int k;  // 0: off
  bool greedy, use_p, use_m, plain, need_total;  // plain: no filter
  double c;  // log2(e) / T
};
__device__ __forceinline__ Rule rule_of(const SampleParams& p, int b) {
  Rule r;
  r.T = p.temperature[b];
  r.greedy = !(r.T > 0.f);
  r.c = r.greedy ? 1.0 : 1.4426950408889634 / (double)r.T;
  const int k = p.top_k ? p.top_k[b] : 0;
  r.k = k > 0 && k < p.V ? k : 0;
  r.top_p = p.top_p ? p.top_p[b] : 1.f;
  r.min_p = p.min_p ? p.min_p[b] : 0.f;
  r.use_p = r.top_p < 1.f;  // false for NaN
  r.use_m = r.min_p > 0.f;
  r.plain = !r.greedy && r.k == 0 && !r.use_p && !r.use_m;
  r.need_total = r.plain || (!r.greedy && r.k == 0 && r.use_p);
  return r;
}

// The tokens that may matter to a row with filters: the list, or (overflown) the
// 128-token blocks that reach the bound.  Warp w owns a contiguous range of the
// vocabulary; walk() visits it in order, 32 tokens at a time.
template <bool BF16>
struct Source {
  const SampleParams& p;
  Shared& sh;
  int64_t row;
  float bound;
  bool listed;

  template <class F>
  __device__ __forceinline__ void blocks(F f) const {  // f(first token, x[4]) for each of the warp's blocks
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b0 = (int)((int64_t)p.nsub * w / kWarps), b1 = (int)((int64_t)p.nsub * (w + 1) / kWarps);
    int n = 0;
    for (int base = b0; base < b1; base += 32) {
      const bool in = base + lane < b1 && sh.sub[min(base + lane, b1 - 1)] >= bound;
      const unsigned m = __ballot_sync(0xffffffffu, in);
      if (in) sh.blk[w][n + __popc(m & ((1u << lane) - 1u))] = (uint16_t)(base + lane);
      n += __popc(m);
    }
    __syncwarp();
    for (int k0 = 0; k0 < n; k0 += 4) {  // four blocks' loads in flight
      float x[4][4];
      int first[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        first[k] = k0 + k < n ? sh.blk[w][k0 + k] * kSub : p.V;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = first[k] + j * 32 + lane;
          x[k][j] = i < p.V ? logit<BF16>(p, row, i) : -INFINITY;
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (first[k] < p.V) f(first[k], x[k]);
    }
    __syncwarp();
  }
  template <class F>
  __device__ __forceinline__ void walk(F f) const {  // f(x, index, present), warp-collective
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (listed) {
      for (int i0 = 0; i0 < sh.len[w]; i0 += 32) {
        const bool in = i0 + lane < sh.len[w];
        f(in ? sh.lval[w][i0 + lane] : -INFINITY, in ? sh.lidx[w][i0 + lane] : 0, in);
      }
    } else {
      blocks([&](int first, const float(&x)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) f(x[j], first + j * 32 + lane, x[j] >= bound && x[j] > -INFINITY);
      });
    }
  }
};

// The maxima of the 128-token blocks, for select().
struct Maxima {
  const SampleParams& p;
  Shared& sh;
  template <class F>
  __device__ __forceinline__ void walk(F f) const {
    for (int i = threadIdx.x; i < p.nsub; i += kThreads) f(sh.sub[i], i, true);
  }
};

// A border of the order: keys above t, and the first c of the `ties` tokens with key t.
struct Border {
  uint32_t t;
  int c, ties;
};

// The key in [lo, hi] at which the tokens from the top first count `want` (MASS =
// false) or first weigh `want` (MASS), by histograms over ever narrower key
// ranges.  key(x, index): keys outside the range are left out.  above: the count
// or weight above `hi` on entry, above the found key on return; ties: tokens with
// that key.  False if all tokens together do not reach it.  COARSE: one histogram;
// t is the lower end of the range that holds the key.
template <bool MASS, bool COARSE = false, class Src, class Key>
__device__ bool select(const Src& src, Shared& sh, Key key, uint32_t lo, uint32_t hi, double want, float m, double c,
                       int shift, uint32_t& t, u64& above, int& ties) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  for (;;) {
    const uint32_t range = hi - lo;
    const int sh_bits = max(0, 32 - __clz(range) - 10);
    __syncthreads();
    for (int i = tid; i < kBins; i += kThreads) {
      sh.cnt[i] = 0;
      if (MASS) sh.lo[i] = sh.hi[i] = 0;
    }
    if (tid == 0) sh.found = -1;
    __syncthreads();
    src.walk([&](float x, int i, bool in) {
      const uint32_t k = in ? key(x, i) : 0u;
      if (!in || k < lo || k > hi) return;
      const int bin = (int)((k - lo) >> sh_bits);
      atomicAdd(&sh.cnt[bin], 1u);
      if (MASS) {
        const u64 wt = (u64)__double2ull_rn(weight(x, m, c, sh.tab) * (double)(1ull << shift));
        const uint32_t l = (uint32_t)wt, old = atomicAdd(&sh.lo[bin], l);
        const uint32_t h = (uint32_t)(wt >> 32) + (old + l < old ? 1u : 0u);
        if (h) atomicAdd(&sh.hi[bin], h);
      }
    });
    __syncthreads();
    // from the top: thread i sums bins 1023 - 4 i .. 1020 - 4 i
    u64 v[4], s = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int bin = kBins - 1 - 4 * tid - j;
      v[j] = MASS ? ((u64)sh.hi[bin] << 32) + sh.lo[bin] : sh.cnt[bin];
      s += v[j];
    }
    u64 incl = warp_scan(s);
    if (lane == 31) sh.red[w] = incl;
    __syncthreads();
    for (int i = 0; i < w; ++i) incl += sh.red[i];
    u64 cum = above + incl - s;
    if ((double)cum < want && (double)(cum + s) >= want) {  // one thread at most
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if ((double)(cum + v[j]) >= want) {
          sh.found = kBins - 1 - 4 * tid - j;
          sh.found_mass = cum;
          break;
        }
        cum += v[j];
      }
    }
    __syncthreads();
    const int bin = sh.found;
    if (bin < 0) return false;
    above = sh.found_mass;
    ties = (int)sh.cnt[bin];
    lo += (uint32_t)bin << sh_bits;
    if (COARSE || sh_bits == 0) break;
    hi = min(hi, lo + ((1u << sh_bits) - 1u));
  }
  t = lo;
  return true;
}

// How many of `ties` tokens of weight wt, behind a weight of `above`, have less than
// `want` before them (at least one).
__device__ __forceinline__ int tokens_below(u64 above, u64 wt, int ties, double want) {
  u64 l = 0, h = (u64)ties;
  while (l < h) {
    const u64 mid = (l + h) / 2;
    if ((double)(above + mid * wt) < want) l = mid + 1;
    else h = mid;
  }
  return max(1, (int)l);
}

// Inclusive scan of one double per thread, and the total, in a fixed order.
__device__ __forceinline__ double block_scan(double v, Shared& sh, double& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  double incl = warp_scan(v);
  __syncthreads();
  if (lane == 31) sh.redd[w] = incl;
  __syncthreads();
  double before = 0.0, all = 0.0;
  for (int i = 0; i < kWarps; ++i) {
    if (i < w) before += sh.redd[i];
    all += sh.redd[i];
  }
  total = all;
  return before + incl;
}

// The last of the c first (in vocabulary order) among the tokens with key t.
template <class Src, class Key>
__device__ int tie_limit(const Src& src, Shared& sh, Key key, uint32_t t, int c) {
  uint32_t end = 0;
  u64 above = 0;
  int one;
  select<false>(
      src, sh, [&](float x, int i) { return key(x, i) == t ? (uint32_t)(kMaxVocab - i) : 0u; }, 1u, kMaxVocab, (double)c,
      0.f, 0.0, 0, end, above, one);
  return kMaxVocab - (int)end;
}

template <bool BF16>
__device__ __forceinline__ void put(const SampleParams& p, int64_t row, int tok, double lp) {
  p.token[row] = tok;
  if (p.logprob) p.logprob[row] = (float)lp;
}

// Draws from a row whose chunks weigh `own` (thread i: chunk i).  kept(x, index):
// the token counts.
template <bool BF16, class Kept>
__device__ void draw(const SampleParams& p, Shared& sh, int64_t row, double own, float m, double c, Kept kept) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  double total;
  const double incl = block_scan(own, sh, total);
  const double target = (double)p.uniform[row] * total;
  if (tid == 0) {
    sh.found = sh.found2 = INT_MAX;
    sh.last = sh.last2 = 0;  // (a row's maximum weighs 1; whatever the sums are, an index stays inside the row)
  }
  __syncthreads();
  if (own > 0.0) {
    if (incl > target) atomicMin(&sh.found, tid);
    atomicMax(&sh.last, tid);
  }
  __syncthreads();
  const int chunk = sh.found != INT_MAX ? sh.found : sh.last;
  if (tid == chunk) sh.cs = incl - own;
  // a warp takes 128 tokens of the chunk
  float x[4];
  double v[4], s = 0.0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = chunk * kChunk + w * 128 + j * 32 + lane;
    x[j] = i < p.V ? logit<BF16>(p, row, i) : -INFINITY;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = chunk * kChunk + w * 128 + j * 32 + lane;
    v[j] = warp_scan(kept(x[j], i) ? weight(x[j], m, c, sh.tab) : 0.0);
    s += __shfl_sync(0xffffffffu, v[j], 31);
  }
  if (lane == 0) sh.redd[w] = s;
  __syncthreads();
  double cum = sh.cs;
  for (int i = 0; i < w; ++i) cum += sh.redd[i];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = chunk * kChunk + w * 128 + j * 32 + lane;
    const bool has = kept(x[j], i) && weight(x[j], m, c, sh.tab) > 0.0;
    if (has && cum + v[j] > target) atomicMin(&sh.found2, i);
    if (has) atomicMax(&sh.last2, i);
    cum += __shfl_sync(0xffffffffu, v[j], 31);
  }
  __syncthreads();
  if (tid == 0) {
    // (a target at the very end of the chunk: its last kept token)
    const int tok = sh.found2 != INT_MAX ? sh.found2 : sh.last2;
    const float xt = logit<BF16>(p, row, tok);
    put<BF16>(p, row, tok, (xt == m ? 0.0 : ((double)xt - (double)m) * c * 0.69314718055994531) - log(total));
  }
}

// A row with filters, from the tokens that reach `bound`.  total: the weight of all
// tokens, for top-p without top-k.  LIST: false is returned where the list
// overflows.
template <bool BF16, bool LIST>
__device__ bool filtered(const SampleParams& p, Shared& sh, int64_t row, const Rule& r, float m, float bound, float cut,
                         double total) {
  constexpr int kDrop = BF16 ? 16 : 0;  // a bf16's key has 16 bits
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const double c = r.c;
  const uint32_t mkey = order_key(m);
  auto key = [](float x, int) { return order_key(x) >> kDrop; };
  Source<BF16> src{p, sh, row, bound, false};
  int len = 0;
  src.blocks([&](int first, const float(&x)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = x[j] >= bound && x[j] > -INFINITY;
      const unsigned b = __ballot_sync(0xffffffffu, in);
      const int at = len + __popc(b & ((1u << lane) - 1u));
      if (in && at < kListCap) {
        sh.lval[w][at] = x[j];
        sh.lidx[w][at] = first + j * 32 + lane;
      }
      len += __popc(b);
    }
  });
  if (lane == 0) sh.len[w] = len;
  src.listed = __syncthreads_and(len <= kListCap) != 0;
  if (LIST && !src.listed) return false;
  int present = 0;
  for (int i = 0; i < kWarps; ++i) present += sh.len[i];

  if (present <= kThreads) {
    // A short list: thread i takes its i-th token and finds the token's place in the
    // order, and the weight before it, by comparing with all others.
    int at = threadIdx.x, lw = 0;
    while (lw < kWarps - 1 && at >= sh.len[lw]) at -= sh.len[lw++];
    const bool in = (int)threadIdx.x < present;
    const float x = in ? sh.lval[lw][at] : -INFINITY;
    const int idx = in ? sh.lidx[lw][at] : 0;
    const u64 wx = in ? (u64)__double2ull_rn(weight(x, m, c, sh.tab) * (double)(1ull << p.shift)) : 0ull;
    float* fx = reinterpret_cast<float*>(sh.cnt);  // [256] logits, [256] weights
    u64* fw = reinterpret_cast<u64*>(sh.lo);
    fx[threadIdx.x] = x;
    fw[threadIdx.x] = wx;
    __syncthreads();
    int rank = 0;
    u64 ahead = 0;
#pragma unroll 4
    for (int j = 0; j < present; ++j) {
      const float y = fx[j];
      const bool first = y > x || (y == x && j < (int)threadIdx.x);
      rank += first;
      ahead += first ? fw[j] : 0ull;
    }
    bool kept = in && (r.k == 0 || rank < r.k);
    if (r.use_p) {
      u64 s = kept ? wx : 0ull;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      if (lane == 0) sh.red[w] = s;
      __syncthreads();
      double base = total * (double)(1ull << p.shift);
      if (r.k > 0) {
        u64 all = 0;
        for (int i = 0; i < kWarps; ++i) all += sh.red[i];
        base = (double)all;
      }
      kept = kept && (rank == 0 || (double)ahead < (double)r.top_p * base);
    }
    kept = kept && (x >= cut || x == m);
    const double v = kept ? weight(x, m, c, sh.tab) : 0.0;
    const double incl = block_scan(v, sh, total);
    if (threadIdx.x == 0) {
      sh.found = INT_MAX;
      sh.last = -1;
    }
    __syncthreads();
    if (v > 0.0) {
      if (incl > (double)p.uniform[row] * total) atomicMin(&sh.found, (int)threadIdx.x);
      atomicMax(&sh.last, (int)threadIdx.x);
    }
    __syncthreads();
    if ((int)threadIdx.x == (sh.found != INT_MAX ? sh.found : sh.last))
      put<BF16>(p, row, idx, (x == m ? 0.0 : ((double)x - (double)m) * c * 0.69314718055994531) - log(total));
    return true;
  }

  // ---------------------------------------------------------------- the kept prefix
  const uint32_t klo = order_key(bound) >> kDrop, khi = mkey >> kDrop;
  Border e{klo, INT_MAX, 0};  // everything present
  if (r.k > 0 && present > r.k) {
    u64 above = 0;
    select<false>(src, sh, key, klo, khi, (double)r.k, m, c, p.shift, e.t, above, e.ties);
    e.c = r.k - (int)above;
  }
  auto value = [&](uint32_t t) { return BF16 ? key_value(t << 16 | ((t & 0x8000u) ? 0u : 0xffffu)) : key_value(t); };
  auto fixed = [&](float x) { return (u64)__double2ull_rn(weight(x, m, c, sh.tab) * (double)(1ull << p.shift)); };
  if (r.use_p) {
    double base = total * (double)(1ull << p.shift);
    if (r.k > 0) {  // the weight of the top k
      u64 s = 0;
      src.walk([&](float x, int, bool in) {
        if (in && order_key(x) >> kDrop >= e.t) s += fixed(x);
      });
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      __syncthreads();
      if (lane == 0) sh.red[w] = s;
      __syncthreads();
      u64 all = 0;
      for (int i = 0; i < kWarps; ++i) all += sh.red[i];
      if (e.c < e.ties) all -= (u64)(e.ties - e.c) * fixed(value(e.t));
      base = (double)all;
    }
    const double want = (double)r.top_p * base;
    uint32_t t;
    int ties;
    u64 above = 0;
    if (select<true>(src, sh, key, e.t, khi, want, m, c, p.shift, t, above, ties)) {
      // tokens of key t that are kept: while the weight before them is below `want`
      const int q = tokens_below(above, fixed(value(t)), t == e.t ? min(e.c, ties) : ties, want);
      e = Border{t, q, ties};
    }
  }
  const int tie_end = e.c < e.ties ? tie_limit(src, sh, key, e.t, e.c) : INT_MAX;

  // ---------------------------------------------------------------- the draw
  auto kept = [&](float x, int i, bool in) -> double {
    const uint32_t k = order_key(x) >> kDrop;
    if (!in || k < e.t || (k == e.t && i > tie_end) || !(x >= cut || x == m)) return 0.0;
    return weight(x, m, c, sh.tab);
  };
  double s = 0.0;
  src.walk([&](float x, int i, bool in) { s += kept(x, i, in); });
  s = warp_sum(s);
  __syncthreads();
  if (lane == 0) sh.redd[w] = s;
  __syncthreads();
  total = 0.0;
  for (int i = 0; i < kWarps; ++i) total += sh.redd[i];
  const double target = (double)p.uniform[row] * total;
  int owner = -1, last_w = 0;
  double cum = 0.0, before = 0.0;
  for (int i = 0; i < kWarps; ++i) {
    if (sh.redd[i] > 0.0) last_w = i;
    if (owner < 0 && cum + sh.redd[i] > target) {
      owner = i;
      before = cum;
    }
    cum += sh.redd[i];
  }
  const bool at_end = owner < 0;  // a target at the very end: the last kept token
  if (at_end) owner = last_w;
  if (w == owner) {
    int tok = -1, last = -1;
    float tx = m, lx = m;
    src.walk([&](float x, int i, bool in) {
      if (tok >= 0) return;
      const double v = kept(x, i, in);
      const double sc = warp_scan(v);
      const unsigned has = __ballot_sync(0xffffffffu, v > 0.0);
      const unsigned hit = __ballot_sync(0xffffffffu, v > 0.0 && !at_end && before + sc > target);
      if (has) {
        last = __shfl_sync(0xffffffffu, i, 31 - __clz(has));
        lx = __shfl_sync(0xffffffffu, x, 31 - __clz(has));
      }
      if (hit) {
        tok = __shfl_sync(0xffffffffu, i, __ffs(hit) - 1);
        tx = __shfl_sync(0xffffffffu, x, __ffs(hit) - 1);
      }
      before += __shfl_sync(0xffffffffu, sc, 31);
    });
    if (tok < 0) {
      tok = last;
      tx = lx;
    }
    if (lane == 0)
      put<BF16>(p, row, tok, (tx == m ? 0.0 : ((double)tx - (double)m) * c * 0.69314718055994531) - log(total));
  }
  return true;
}

__device__ __forceinline__ float min_p_cut(const Rule& r, float m) {
  return r.use_m ? fmaxf(-INFINITY, __double2float_ru((double)m + log2((double)r.min_p) / r.c)) : -INFINITY;
}

template <bool BF16>
__device__ void finish_row(const SampleParams& p, Shared& sh, int64_t row) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const Rule r = rule_of(p, (int)(row / p.n));
  float mx = -INFINITY;
  for (int i = tid; i < p.nsub; i += kThreads) {
    const float s = __ldcg(p.sub + row * p.nsub + i);
    sh.sub[i] = s;
    mx = fmaxf(mx, s);
  }
  const uint32_t wk = __reduce_max_sync(0xffffffffu, order_key(mx));
  if (lane == 0) sh.red[w] = wk;
  if (tid == 0) sh.found = sh.found2 = INT_MAX;
  __syncthreads();
  uint32_t mkey = 0;
  for (int i = 0; i < kWarps; ++i) mkey = max(mkey, (uint32_t)sh.red[i]);
  const float m = key_value(mkey);
  if (m == -INFINITY) {  // no token can be drawn
    if (tid == 0) put<BF16>(p, row, -1, -INFINITY);
    return;
  }
  if (r.greedy || r.k == 1 || (r.use_p && !(r.top_p > 0.f)) || r.min_p > 1.f) {  // the first token of the order
    for (int i = tid; i < p.nsub; i += kThreads)
      if (sh.sub[i] == m) {
        atomicMin(&sh.found, i);
        break;
      }
    __syncthreads();
    const int i = sh.found * kSub + tid;
    if (tid < kSub && i < p.V && logit<BF16>(p, row, i) == m) atomicMin(&sh.found2, i);
    __syncthreads();
    if (tid == 0) put<BF16>(p, row, sh.found2, 0.0);
    return;
  }
  double own = 0.0, total = 0.0;
  if (r.need_total) {
    if (tid < p.nchunk) {
      float cm = -INFINITY;
      for (int i = tid * (kChunk / kSub); i < min(p.nsub, (tid + 1) * (kChunk / kSub)); ++i) cm = fmaxf(cm, sh.sub[i]);
      own = __ldcg(p.sum + row * p.nchunk + tid) * weight(cm, m, r.c, sh.tab);
    }
    if (r.plain) {
      draw<BF16>(p, sh, row, own, m, r.c, [](float, int) { return true; });
      return;
    }
    block_scan(own, sh, total);
  }
  const float cut = min_p_cut(r, m);
  float bound = -INFINITY;
  const Maxima maxima{p, sh};
  auto key = [](float x, int) { return order_key(x); };
  uint32_t lowest = 0xffffffffu, t;
  for (int i = tid; i < p.nsub; i += kThreads) lowest = min(lowest, order_key(sh.sub[i]));
  lowest = __reduce_min_sync(0xffffffffu, lowest);
  __syncthreads();
  if (lane == 0) sh.red[w] = lowest;
  __syncthreads();
  for (int i = 0; i < kWarps; ++i) lowest = min(lowest, (uint32_t)sh.red[i]);
  u64 above = 0;
  int ties;
  if (r.k > 0 && r.k <= p.nsub) {
    // a value that at least k of the maxima reach
    if (select<false, true>(maxima, sh, key, lowest, mkey, (double)r.k, m, r.c, p.shift, t, above, ties)) bound = key_value(t);
  } else if (r.k == 0 && r.use_p) {
    // a value such that the maxima that reach it weigh top_p of all (2^-40 is more
    // than the sums' errors)
    const double want = (double)r.top_p * total * (double)(1ull << p.shift) * (1.0 + 1e-12);
    const bool few =
        select<true, true>(maxima, sh, key, lowest, mkey, want, m, r.c, p.shift, t, above, ties) &&
        filtered<BF16, true>(p, sh, row, r, m, key_value(t), cut, total);
    if (few) return;
    if (Weigher::fits(m, r.c)) {  // on to the weighing
      u64* h = p.hist + row * kBins;
      for (int i = tid; i < kBins; i += kThreads) __stcg(h + i, 0ull);
      if (tid == 0) {
        RowState st = {};
        st.total = total;
        st.m = m;
        st.scale = (float)fmin(32.0 * r.c, 3e38);
        p.st[row] = st;
        p.marked[4 + atomicAdd(p.marked, 1)] = (int)row;
      }
      return;
    }
  }
  if (!r.use_p) bound = fmaxf(bound, cut);  // (top-p's base holds all of the top k)
  filtered<BF16, false>(p, sh, row, r, m, fminf(bound, m), cut, total);
}

// A warp's chunk of 1024 logits.  Lane's tokens: 32 j + lane (fp32), 64 j +
// 2 lane and the next (bf16); token(e) is the index of x[e] in the chunk, and block
// s of 128 tokens is x[4 s .. 4 s + 3].
template <bool BF16>
__device__ __forceinline__ int chunk_token(int e) {
  const int lane = threadIdx.x & 31;
  return BF16 ? (e >> 1) * 64 + 2 * lane + (e & 1) : e * 32 + lane;
}
template <bool BF16>
__device__ __forceinline__ void load_chunk(const SampleParams& p, int64_t row, int chunk, uint32_t (&raw)[BF16 ? 16 : 32]) {
  const int lane = threadIdx.x & 31, i0 = chunk * kChunk;
  if (BF16) {
    const uint16_t* src = reinterpret_cast<const uint16_t*>(p.logits) + row * p.stride + i0;
    if ((reinterpret_cast<uintptr_t>(src) & 3u) == 0 && i0 + kChunk <= p.V) {
#pragma unroll
      for (int j = 0; j < 16; ++j) raw[j] = __ldg(reinterpret_cast<const uint32_t*>(src) + j * 32 + lane);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int i = j * 64 + 2 * lane;
        const uint32_t a = i0 + i < p.V ? __ldg(src + i) : 0xff80u, b = i0 + i + 1 < p.V ? __ldg(src + i + 1) : 0xff80u;
        raw[j] = a | b << 16;
      }
    }
  } else {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(p.logits) + row * p.stride + i0;
    if (i0 + kChunk <= p.V) {
#pragma unroll
      for (int j = 0; j < 32; ++j) raw[j] = __ldg(src + j * 32 + lane);
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) raw[j] = i0 + j * 32 + lane < p.V ? __ldg(src + j * 32 + lane) : 0xff800000u;
    }
  }
}
template <bool BF16>
__device__ __forceinline__ void unpack_chunk(const uint32_t (&raw)[BF16 ? 16 : 32], float (&x)[32]) {
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    const uint32_t v = raw[BF16 ? e >> 1 : e];
    x[e] = __uint_as_float(!BF16 ? v : ((e & 1) ? v & 0xffff0000u : v << 16));
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 3) stream_kernel(const __grid_constant__ SampleParams p) {
  __shared__ double tab[kTab * kTabCopies];
  const int tid = threadIdx.x, lane = tid & 31;
  fill_table(tab);
  pdl_wait_primary();
  pdl_launch_dependents();
  if (blockIdx.x == 0 && tid < 4) p.marked[tid] = 0;
  __syncthreads();
  const int64_t units = p.rows * p.nchunk, step = (int64_t)gridDim.x * kWarps;
  int64_t unit = (int64_t)blockIdx.x * kWarps + (tid >> 5);
  for (; unit < units; unit += step) {
    const int64_t row = unit / p.nchunk;
    const int chunk = (int)(unit - row * p.nchunk);
    uint32_t raw[BF16 ? 16 : 32];
    load_chunk<BF16>(p, row, chunk, raw);
    const Rule r = rule_of(p, (int)(row / p.n));
    float x[32];
    unpack_chunk<BF16>(raw, x);
    uint32_t top = 0, mine = 0;
#pragma unroll
    for (int s = 0; s < kChunk / kSub; ++s) {  // (a maximum skips NaN)
      const uint32_t k = __reduce_max_sync(
          0xffffffffu, order_key(clean(fmaxf(fmaxf(x[4 * s], x[4 * s + 1]), fmaxf(x[4 * s + 2], x[4 * s + 3])))));
      if (lane == s) mine = k;
      top = max(top, k);
    }
    const int sub0 = chunk * (kChunk / kSub);
    if (lane < kChunk / kSub && sub0 + lane < p.nsub) __stcg(p.sub + row * p.nsub + sub0 + lane, key_value(mine));
    if (r.need_total) {
      const float cm = key_value(top);
      double s = 0.0;
      if (Weigher::fits(cm, r.c)) {
        const Weigher wt(cm, r.c);
#pragma unroll
        for (int e0 = 0; e0 < 32; e0 += 8) {
          double v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = wt(x[e0 + e], tab);
          s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        }
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) s += weight(clean(x[e]), cm, r.c, tab);
      }
      s = warp_sum(s);
      if (lane == 0) __stcg(p.sum + row * p.nchunk + chunk, s);
    }
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 4) finish_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  fill_table(sh.tab);
  pdl_wait_primary();
  pdl_launch_dependents();
  __syncthreads();
  finish_row<BF16>(p, sh, blockIdx.x);
}

// Has this block brought the row's last segment?  (Block-uniform.)
__device__ __forceinline__ bool last_segment(int* count, int nseg) {
  __shared__ int arrived;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) arrived = atomicAdd(count, 1);
  __syncthreads();
  const bool last = arrived == nseg - 1;
  if (last) __threadfence();
  __syncthreads();
  return last;
}

// The next segment of the marked rows for this block, requested one ahead.  (Taken
// in turn: a block that has finished a row is late, and with a fixed share of the
// segments it would be the last of its next rows too, and finish them all.)
struct Segments {
  int* taken;
  int units, ahead;
  __device__ __forceinline__ Segments(int* taken_, int units_) : taken(taken_), units(units_) {
    ahead = threadIdx.x == 0 ? atomicAdd(taken, 1) : 0;
  }
  __device__ __forceinline__ int next() {  // -1: none left
    __shared__ int unit;
    __syncthreads();
    if (threadIdx.x == 0) {
      unit = ahead < units ? ahead : -1;
      ahead = atomicAdd(taken, 1);
    }
    __syncthreads();
    return unit;
  }
};

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 4) weigh_kernel(const __grid_constant__ SampleParams p) {
  __shared__ uint32_t hist_s[kBins];  // (8192 tokens of at most 2^18 each stay below 2^32)
  __shared__ u64 red[2 * kWarps];
  __shared__ int too_many;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  pdl_wait_primary();
  pdl_launch_dependents();
  const int units = __ldcg(p.marked) * p.nseg;
  if (units == 0) return;
  Segments segments(p.marked + 1, units);
  for (int unit = segments.next(); unit >= 0; unit = segments.next()) {
    const int64_t row = __ldcg(p.marked + 4 + unit / p.nseg);
    const int chunk = unit % p.nseg * kWarps + w;
    for (int i = tid; i < kBins; i += kThreads) hist_s[i] = 0;
    __syncthreads();
    const float m = __ldcg(&p.st[row].m), scale = __ldcg(&p.st[row].scale);
    if (chunk < p.nchunk) {
      uint32_t raw[BF16 ? 16 : 32];
      load_chunk<BF16>(p, row, chunk, raw);
      float x[32];
      unpack_chunk<BF16>(raw, x);
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        float frac;
        const int bin = bin_of(fmaxf(x[e], -INFINITY), m, scale, frac);
        const uint32_t v = (uint32_t)fast_exp2(fmaf(frac, -1.f / 32.f, 18.f));
        if (v) atomicAdd(&hist_s[bin], v);
      }
    }
    __syncthreads();
    u64* hist = p.hist + row * kBins;
    for (int i = tid; i < kBins; i += kThreads)
      if (hist_s[i]) atomicAdd(hist + i, (u64)hist_s[i]);
    if (!last_segment(&p.st[row].weighed, p.nseg)) continue;
    // thread i sums bins 4 i .. 4 i + 3: weights in units of 2^-46, and tokens (in all
    // bins but the last a token counts between 2^(18 - 1/32) and 2^18)
    u64 v[4], s = 0, tokens = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u64 h = __ldcg(hist + 4 * tid + j);
      v[j] = (u64)((double)h * (double)fast_exp2(28.f - (float)(4 * tid + j) / 32.f));
      s += v[j];
      tokens += (h + 255999) / 256000;
    }
    u64 incl = warp_scan(s), listed = warp_scan(tokens);
    if (lane == 31) {
      red[w] = incl;
      red[kWarps + w] = listed;
    }
    if (tid == 0) too_many = 0;
    __syncthreads();
    for (int i = 0; i < w; ++i) {
      incl += red[i];
      listed += red[kWarps + i];
    }
    // Each weight is good to 2^-16: its 18 bits, the exponent's two fp32 roundings
    // (of up to 32: 2^-18) and the exponentials'.  The border lies behind the last
    // bin up to which the sum is surely too small, and not behind the first up to
    // which it surely suffices.
    const double want = (double)p.top_p[row / p.n] * __ldcg(&p.st[row].total) * 70368744177664.0, slack = 1.0 / 16384.0;
    const double first = want * (1.0 - slack), last = want * (1.0 + slack);
    u64 cum = incl - s;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const double c0 = (double)cum, c1 = (double)(cum + v[j]);
      if ((c0 < first && c1 >= first) || (tid == kThreads - 1 && j == 3 && c1 < first)) p.st[row].bin0 = 4 * tid + j;
      if ((c0 < last && c1 >= last) || (tid == kThreads - 1 && j == 3 && c1 < last)) {
        p.st[row].bin1 = 4 * tid + j;
        too_many = listed > kRowList || 4 * tid + j == kBins - 1;
      }
      cum += v[j];
    }
    __syncthreads();
    // where all that may be kept fits the list, all of it is listed
    if (tid == 0 && !too_many) p.st[row].bin0 = 0;
    __syncthreads();
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 3) border_kernel(const __grid_constant__ SampleParams p) {
  constexpr int kDrop = BF16 ? 16 : 0;
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  fill_table(sh.tab);
  pdl_wait_primary();
  pdl_launch_dependents();
  __syncthreads();
  const int units = __ldcg(p.marked) * p.nseg;
  if (units == 0) return;
  Segments segments(p.marked + 2, units);
  for (int unit = segments.next(); unit >= 0; unit = segments.next()) {
    const int64_t row = __ldcg(p.marked + 4 + unit / p.nseg);
    const int chunk = unit % p.nseg * kWarps + w;
    const Rule r = rule_of(p, (int)(row / p.n));
    const double c = r.c;
    const float m = __ldcg(&p.st[row].m), scale = __ldcg(&p.st[row].scale), cut = min_p_cut(r, m);
    const int bin0 = __ldcg(&p.st[row].bin0), bin1 = __ldcg(&p.st[row].bin1);
    auto over_cut = [&](float x) { return x >= cut || x == m; };
    if (chunk < p.nchunk) {
      uint32_t raw[BF16 ? 16 : 32];
      load_chunk<BF16>(p, row, chunk, raw);
      float x[32];
      unpack_chunk<BF16>(raw, x);
      double keep = 0.0, over = 0.0;
      uint32_t listed = 0;  // bit e: x[e] goes to the list
      const Weigher wt(m, c);
#pragma unroll
      for (int e0 = 0; e0 < 32; e0 += 8) {
        // eight tokens at a time: their weights' chains of dependent steps overlap
        uint32_t sure = 0;
#pragma unroll
        for (int e = e0; e < e0 + 8; ++e) {
          x[e] = fmaxf(x[e], -INFINITY);
          float frac;
          const int bin = bin_of(x[e], m, scale, frac);
          sure |= bin < bin0 ? 1u << e : 0u;
          listed |= bin >= bin0 && bin <= bin1 && x[e] > -INFINITY ? 1u << e : 0u;
        }
        if (!__any_sync(0xffffffffu, sure != 0)) continue;
        double v[8];
#pragma unroll
        for (int e = e0; e < e0 + 8; ++e) v[e - e0] = wt(x[e], sh.tab);
#pragma unroll
        for (int e = e0; e < e0 + 8; ++e) {
          const double s = (sure >> e) & 1u ? v[e - e0] : 0.0;
          over += s;
          keep += over_cut(x[e]) ? s : 0.0;
        }
      }
      over = warp_sum(over);
      keep = warp_sum(keep);
      if (lane == 0) {
        __stcg(p.over + row * p.nchunk + chunk, over);
        __stcg(p.sum + row * p.nchunk + chunk, keep);
      }
      int mine = __popc(listed), at = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, at, off);
        if (lane >= off) at += o;
      }
      const int count = __shfl_sync(0xffffffffu, at, 31);
      int first = 0;
      if (lane == 0 && count) first = atomicAdd(&p.st[row].listed, count);
      at += __shfl_sync(0xffffffffu, first, 0) - mine;
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if ((listed >> e) & 1u) {
          if (at < kRowList) {
            __stcg(p.list_x + row * kRowList + at, clean(x[e]));
            __stcg(p.list_i + row * kRowList + at, chunk * kChunk + chunk_token<BF16>(e));
          }
          ++at;
        }
    }
    if (!last_segment(&p.st[row].bordered, p.nseg)) continue;
    const int n = __ldcg(&p.st[row].listed);
    const double unit_w = (double)(1ull << p.shift);
    const double total = __ldcg(&p.st[row].total);
    double sure;
    block_scan(tid < p.nchunk ? __ldcg(p.over + row * p.nchunk + tid) : 0.0, sh, sure);
    const double want = (double)r.top_p * total * unit_w;
    u64 above = (u64)__double2ull_rn(sure * unit_w);
    bool settled = n <= kRowList && (double)above < want;
    Border e{0u, INT_MAX, 0};
    const Source<BF16> src{p, sh, row, -INFINITY, true};
    auto key = [](float x, int) { return order_key(x) >> kDrop; };
    auto fixed = [&](float x) { return (u64)__double2ull_rn(weight(x, m, c, sh.tab) * unit_w); };
    int tie_end = INT_MAX;
    if (settled) {
      // the bins' tokens, in any order, dealt to the warps in turn
      for (int i = tid; i < n; i += kThreads) {
        sh.lval[i % kWarps][i / kWarps] = __ldcg(p.list_x + row * kRowList + i);
        sh.lidx[i % kWarps][i / kWarps] = __ldcg(p.list_i + row * kRowList + i);
      }
      if (tid < kWarps) sh.len[tid] = (n - tid + kWarps - 1) / kWarps;
      __syncthreads();
      uint32_t klo = 0xffffffffu, khi = 0;
      for (int i = tid; i < n; i += kThreads) {
        const uint32_t k = order_key(sh.lval[i % kWarps][i / kWarps]) >> kDrop;
        klo = min(klo, k);
        khi = max(khi, k);
      }
      klo = __reduce_min_sync(0xffffffffu, klo);
      khi = __reduce_max_sync(0xffffffffu, khi);
      if (lane == 0) sh.red[w] = (u64)klo << 32 | khi;
      __syncthreads();
      for (int i = 0; i < kWarps; ++i) {
        klo = min(klo, (uint32_t)(sh.red[i] >> 32));
        khi = max(khi, (uint32_t)sh.red[i]);
      }
      uint32_t t;
      int ties;
      settled = n > 0 && select<true>(src, sh, key, klo, khi, want, m, c, p.shift, t, above, ties);
      if (settled) {
        const float xt = BF16 ? key_value(t << 16 | ((t & 0x8000u) ? 0u : 0xffffu)) : key_value(t);
        e = Border{t, tokens_below(above, fixed(xt), ties, want), ties};
        if (e.c < e.ties) tie_end = tie_limit(src, sh, key, e.t, e.c);
      }
    }
    if (!settled) {
      // the bins hold too many tokens to list (equal logits, or a top_p so close to 1
      // that the border is among the lightest): walk the row
      for (int i = tid; i < p.nsub; i += kThreads) sh.sub[i] = __ldcg(p.sub + row * p.nsub + i);
      __syncthreads();
      filtered<BF16, false>(p, sh, row, r, m, -INFINITY, cut, total);
      __syncthreads();
      continue;
    }
    auto in_bins = [&](float x, int i) {
      const uint32_t k = order_key(x) >> kDrop;
      return k > e.t || (k == e.t && i <= tie_end);
    };
    // the bins' kept tokens join their chunks
    __syncthreads();
    sh.lo[tid] = sh.hi[tid] = 0;
    __syncthreads();
    src.walk([&](float x, int i, bool in) {
      if (!in || !in_bins(x, i) || !over_cut(x)) return;
      const u64 v = fixed(x);
      const uint32_t l = (uint32_t)v, old = atomicAdd(&sh.lo[i / kChunk], l);
      const uint32_t h = (uint32_t)(v >> 32) + (old + l < old ? 1u : 0u);
      if (h) atomicAdd(&sh.hi[i / kChunk], h);
    });
    __syncthreads();
    const double own = tid < p.nchunk ? __ldcg(p.sum + row * p.nchunk + tid) +
                                            (double)(((u64)sh.hi[tid] << 32) + sh.lo[tid]) / unit_w
                                      : 0.0;
    draw<BF16>(p, sh, row, own, m, c, [&](float x, int i) {
      float frac;
      const int bin = bin_of(x, m, scale, frac);
      return x > -INFINITY && over_cut(x) && (bin < bin0 || (bin <= bin1 && in_bins(x, i)));
    });
    __syncthreads();
  }
}

struct SamplePlan {
  int64_t rows;
  int nseg, nsub, nchunk;
  size_t sub, sum, over, marked, st, hist, list_x, list_i, bytes;  // workspace offsets
};
SamplePlan plan_sample(int B, int M, int V) {
  SamplePlan s;
  s.rows = (int64_t)B * (M + 1);
  s.nsub = (V + kSub - 1) / kSub;
  s.nchunk = (V + kChunk - 1) / kChunk;
  s.nseg = (s.nchunk + kWarps - 1) / kWarps;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += ((size_t)s.rows * bytes + 511) / 256 * 256;
    return o;
  };
  s.sub = take(s.nsub * sizeof(float));
  s.sum = take(s.nchunk * sizeof(double));
  s.over = take(s.nchunk * sizeof(double));
  s.marked = take(sizeof(int));  // (the rounding holds the count as well)
  s.st = take(sizeof(RowState));
  s.hist = take(kBins * sizeof(u64));
  s.list_x = take(kRowList * sizeof(float));
  s.list_i = take(kRowList * sizeof(int));
  s.bytes = at;
  return s;
}

template <bool BF16>
tv_status launch_sample(const SampleParams& p, int sms, cudaStream_t s) {
  const int smem = (int)sizeof(Shared);
  tv_status r = allow_shared(reinterpret_cast<const void*>(finish_kernel<BF16>), smem);
  if (r == TV_OK && p.top_p) r = allow_shared(reinterpret_cast<const void*>(border_kernel<BF16>), smem);
  if (r != TV_OK) return r;
  // as many blocks as are resident at once (launch bounds; the finish's shared memory
  // fits four times)
  static_assert(4 * (sizeof(Shared) + 1024) <= 228 * 1024, "four blocks to an SM");
  auto blocks = [&](int64_t n, int per_sm) { return dim3((unsigned)std::min<int64_t>(n, per_sm * (int64_t)sms)); };
  const int64_t units = p.rows * p.nchunk;
  r = launch(stream_kernel<BF16>, blocks((units + kWarps - 1) / kWarps, 3), dim3(kThreads), 0, s, 1, true, p);
  if (r == TV_OK) r = launch(finish_kernel<BF16>, dim3((unsigned)p.rows), dim3(kThreads), smem, s, 1, true, p);
  if (r != TV_OK || !p.top_p) return r;
  r = launch(weigh_kernel<BF16>, blocks(p.rows * p.nseg, 4), dim3(kThreads), 0, s, 1, true, p);
  if (r == TV_OK) r = launch(border_kernel<BF16>, blocks(p.rows * p.nseg, 3), dim3(kThreads), smem, s, 1, true, p);
  return r;
}

}  // namespace
}  // namespace tv

extern "C" size_t tree_accept_sample_workspace_size(int B, int M, int V) {
  return B > 0 && M >= 0 && M < tv::kMaxRows && V > 0 && V <= tv::kMaxVocab ? tv::plan_sample(B, M, V).bytes : 0;
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
  if (rows * tv::plan_sample(1, 0, V).nseg > 0x3fffffff) return TV_ERR_UNSUPPORTED;  // segments are counted in 32 bits
  if (!workspace || !aligned16(workspace) || workspace_bytes < tree_accept_sample_workspace_size(B, M, V))
    return TV_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int sms = 0;
  tv_status r = current_sms(sms);
  if (r != TV_OK) return r;
  const SamplePlan lp = plan_sample(B, M, V);
  char* ws = static_cast<char*>(workspace);
  SampleParams p;
  p.logits = logits;
  p.stride = logits_stride;
  p.rows = rows;
  p.V = V;
  p.n = M + 1;
  p.nseg = lp.nseg;
  p.nsub = lp.nsub;
  p.nchunk = lp.nchunk;
  p.uniform = uniform;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.token = token;
  p.logprob = logprob;
  p.sub = reinterpret_cast<float*>(ws + lp.sub);
  p.sum = reinterpret_cast<double*>(ws + lp.sum);
  p.over = reinterpret_cast<double*>(ws + lp.over);
  p.marked = reinterpret_cast<int*>(ws + lp.marked);
  p.st = reinterpret_cast<RowState*>(ws + lp.st);
  p.hist = reinterpret_cast<u64*>(ws + lp.hist);
  p.list_x = reinterpret_cast<float*>(ws + lp.list_x);
  p.list_i = reinterpret_cast<int*>(ws + lp.list_i);
  p.shift = V <= (1 << 17) ? 46 : 45;
  r = logits_type == TV_LOGITS_F32 ? launch_sample<false>(p, sms, s) : launch_sample<true>(p, sms, s);
  if (r != TV_OK) return r;
  return launch_accept_walk(token, draft, parent, depth, anc_mask, status, B, M, max_depth, accept_len, path, bonus,
                            s);
}
