// attention_scored.cu -- tree_attention_scored: tree attention whose scores are
// capped by a tanh, limited to a window of positions or biased by distance.
//
// "EAGLE-Pangu: Accelerator-Safe Tree Speculative Decoding on Ascend NPUs",
// methodology C (tree mask), and "Batch Speculative Decoding Done Right",
// methodology (position-ID contiguity): node u sits at position kv_len +
// depth(u), prefix column j at position j, so distances inside the tree are
// differences of depth.
//
// For a query row (node u, head h) and a key x, in the log2 domain:
//   s  = scale log2e (q.k)                          no cap
//   s  = cap log2e tanh(scale (q.k) / cap)          cap
//   s -= slope_h log2e (pos(u) - pos(x))            bias
//   out = sum_x 2^(s - r) v_x / sum_x 2^(s - r)     for any reference r
//
// Work.  The G (M+1) query rows of a (sequence, kv head) form tiles of 128, the
// keys it can see (from the root's window on) tiles of 80.  A CTA takes an
// item: two query tiles and a range of key tiles.  Each of its two pipes (a
// softmax warpgroup with a TMEM block of its own) owns one query tile and both
// read every K/V tile; where only one query tile is left, the pipes share it
// and take the even and the odd key tiles.  While one pipe's softmax runs, the
// tensor core works for the other.
//
// Warps (384 threads, one CTA per SM, kept for several items):
//   0     requests K and V tiles into one ring of slots in the order of their use
//   1     TMEM owner; works out the CTA's next item one ahead
//   2, 3  issue the MMAs of a pipe each:
//           S = Q K^T   M = 128, N = 80, A and B from shared memory -> TMEM
//           O += P V    M = 128, N = D,  A = P from TMEM, V from shared memory
//   4-11  the pipes' softmax warps: thread t owns TMEM lane t, one query row
// TMEM columns of a pipe: S [0, 80), P [80, 120), O [128, 128 + D).  Tiles of 80
// keys leave P columns of its own beside S, so the next S is formed while the
// softmax still works on this one.  (Tiles of 128 keys with P written over S: PV
// and the next QK lay between two softmax phases of a pipe, 1.0 us after 1.1-1.4
// us of softmax; 129 query rows x 64 heads x 8 sequences of 4096-16384 keys took
// 551 us, and 530 us with tiles of 80 keys, both with equal ranges dealt in turn.)
// With few query rows a tile has 64 keys and its softmax is shared by a pipe's four
// warps (kFewRows).
// What bounds it: the softmax warps, two to a scheduler, 1.3-1.45 us per pair of tiles
// (tensor pipe 42 %, MUFU 39 %).  Four to a scheduler, each with half of a row's
// columns, took 616 us: twice the TMEM accesses at half the width.  (517 us now, 670
// TFLOP/s, 0.40 of a plain bf16 GEMM's rate; a window of 4096 keys for 6 x 4 rows x 8 heads x 8
// sequences, 135 MB, 36.7 us: 3.7 TB/s with 5 us before the first tile and 6 us of
// epilogue and merge.)
#include <algorithm>
#include <climits>

#include "attention_common.cuh"
#include "tcgen05.cuh"

namespace tv {
namespace {

constexpr int kQRows = 128;
// The few-row form: up to 32 query rows per kv head, and few keys.  All four softmax
// warps of a pipe get the same rows, and each forms the weights of 16 of the 64 keys of a
// tile, so a tile's softmax takes 0.5 us instead of 1.0-1.4.  Longer ranges stream their
// keys at the rate of HBM either way, and there the wider tiles are the better ones.
// Few-row / general form, 8 kv heads of 4 query heads, by keys per SM: 8 sequences of up to
// 4096 keys, single tokens (1770) 28.0 / 28.2 us, 16 of 4096 (3540) 58.3 / 53.5 us; 6 rows
// and a window of 4096, 8 sequences (1770) 37.4 / 36.6 us, 5 (1110) 27.9 / 29.1 us,
// 2 (440) 17.3 / 20.5 us; one sequence of 4096 keys (220) 13.5 / 17.2 us.
constexpr int kFewRows = 32, kFewKeys = 1500;  // query rows; keys per SM
constexpr int keys_of(bool few) { return few ? 64 : 80; }  // keys per tile
constexpr int kQHalf = kQRows * 128;       // of a query tile
constexpr int kRingBytes = 140 * 1024;
constexpr int kMaxSlots = 14;
constexpr int kThreads = 384;
constexpr int kColO = 128;                 // TMEM column of O in a pipe's 256
// A row's reference moves once a score lies more than 2^kGrow above it (the
// weights are floats in bf16 and sums in fp32: a large weight is as exact as a
// small one, and 2^24 leaves both far from their limits).
constexpr float kGrow = 24.0f;
constexpr int kMaxBatch = 4096;
constexpr int kMinTiles = 6;               // no cut nearer to a row's ends than this many key tiles
constexpr int kSecondItem = 14;            // what a CTA's second item costs on top, in key tiles of a lone query tile

// Which scores an instance computes.
//   kCapLow: capped with cap * log2e <= kLowCap: every exponent lies within that of
//   a fixed reference, so no maximum is kept and O is never rescaled
enum Mode { kPlain = 0, kCapLow = 1, kCapHigh = 2, kBias = 3, kCapBias = 4 };
constexpr float kLowCap = 85.f;

// tanh(z) / z for |z| <= kPolyLim as a polynomial in z^2 (least relative error on
// that range, found by iteratively reweighted least squares at Chebyshev nodes:
// 5.7e-7), on the FMA pipe.  Beyond it tanh(z) = 1 - 2 / (e^2z + 1).
constexpr double kPolyLim = 0.75;
constexpr double kPoly[5] = {0.999999463558197, -0.3332825005054474, 0.13258983194828033, -0.050056301057338715,
                             0.012929631397128105};

struct ScoredParams {
  const uint16_t* q;
  const int32_t *kv_start, *kv_len, *depth, *slot;
  const uint32_t* anc;
  int32_t* status;
  const float* slopes;
  uint16_t* out;
  int64_t S_cap;
  int B, M, Hq, Hkv, G, W, n_slots, window;
  int rows;         // G * (M + 1) query rows of a (sequence, kv head)
  int nqt, npairs;  // query tiles, and items' pairs of them
  int rec_rows;     // rows of a partial record
  int grid;         // CTAs
  float inv_g;      // 1 / G
  float scale_log2, ref;
  float c[5];       // capped score = x * (c0 + c1 x^2 + ...), x = q.k
  float x_lim, z2, cap_log2;  // |x| of the polynomial's range; e^2z = 2^(z2 x); cap * log2e
  uint64_t wait_limit_ns;
  float* ws_o;      // records [CTA][0: cut at its start, 1: only at its end][pipe][D / 4][rec_rows] float4
  float2* ws_ml;    // [CTA][2][pipe][rec_rows] (reference, sum)
  int2* ws_row;     // [row of work] the first and the last CTA with a piece; (-1, -1): one had it all
};

// A sequence's place in the cache, the first key that its root sees and the key
// tiles from there (0: bad slot or geometry).  Its status has no part in this:
// a call's CTAs form the plan at different times, and a sequence may fail in
// between.
struct Geo {
  int sl, ks, kl, first, nt;
};

template <int KEYS>
__device__ __forceinline__ Geo sequence(const ScoredParams& p, int b) {
  Geo g{cache_slot(p.slot, b, p.n_slots), 0, 0, 0, 0};
  if (g.sl < 0) return g;
  g.ks = __ldcg(p.kv_start + g.sl);
  g.kl = __ldcg(p.kv_len + g.sl);
  if (!geometry_ok(g.ks, g.kl, p.M, p.S_cap)) return g;
  if (p.window > 0) g.first = max(0, g.kl - (p.window - 1));
  g.nt = (g.kl - g.first + p.M + 1 + KEYS - 1) / KEYS;
  return g;
}

// How the work is dealt.  The rows of work are the pairs of query tiles of every
// (sequence, kv head), in this order.  The CTAs take consecutive shares of them, so a
// row may be cut between CTAs; the pieces are joined by the merge kernel.
//   by cost  (per = 0) a row costs its key tiles, twice for a full pair (a lone query
//            tile takes half the time), and every CTA takes the same cost
//   by piece (per > 0) a row makes equal pieces of at most `per` key tiles, and every
//            CTA takes one piece
// A share by cost crosses from row to row, and every further item costs its queries' way
// into shared memory (2-3 us), the filling and draining of the pipes (2 us) and an
// epilogue (1.3-2.5 us); pieces are uneven.  So: pieces where there is a CTA for every
// row and the longest piece costs no more than an even share and kSecondItem, and shares
// by cost elsewhere.  Measured by piece / by cost, with the longest piece and the even
// share in key tiles: window of 4096 keys, 8 kv heads, 11 sequences (52, 31) 54.3 / 50.2
// us, 14 sequences (52, 39) 55.6 / 57.2 us, 8 sequences (26, 22) 37.5 / 42.3 us; biases, 3
// query tiles, 8 sequences (52, 33) 59.0 / 54.4 us.  Equal ranges of every sequence dealt
// in turn took 172 us for 32 sequences with biases that take 137 us so, and 563 us for
// 129 query rows x 64 heads x 8 sequences that took 510 us so.
__device__ __forceinline__ int tiles_of(int nt) { return max(nt, 1); }  // (a sequence without keys has rows to zero)

struct Shares {  // (the host has checked that all of it fits in 31 bits)
  int total, even;      // all rows, in the unit of the shares; a CTA's share,
  int extra, ctas;      // plus one for the first `extra`; CTAs that take part
  int per, head, pair;  // of one unit of a row: units of its kv head and of a full pair
  // `units`: the sum of units_of over the sequences
  __device__ __forceinline__ void set(const ScoredParams& p, int units, int per_) {
    per = per_;
    head = per ? p.npairs : p.nqt;
    pair = per ? 1 : 2;
    total = units * p.Hkv * head;
    ctas = total;
    // (at least two units by cost, so that every border inside a row is a cut of its own)
    if (!per && p.nqt > 1) ctas = max(1, min(total / 2, max(total / (2 * kMinTiles), p.B * p.Hkv * p.npairs)));
    if (!per && p.nqt == 1) ctas = max(total / kMinTiles, p.B * p.Hkv);
    ctas = min(p.grid, ctas);
    even = (uint32_t)total / (uint32_t)ctas;
    extra = total - even * ctas;
  }
  __device__ __forceinline__ int units_of(int nt) const {
    return per ? (int)((uint32_t)(nt + per - 1) / (uint32_t)per) : nt;
  }
  __device__ __forceinline__ int begin(int cta) const { return even * cta + min(cta, extra); }
  // the key tile at which a row of nt tiles, n units, that begins at `start` is cut for a border
  __device__ __forceinline__ int cut(int border, int start, int nt, int n, bool dual) const {
    const int d = border - start;
    if (d <= 0) return 0;
    if (per) return d >= n ? nt : (int)((uint64_t)nt * d / n);
    const int t = dual ? (d + 1) >> 1 : d;
    if (t >= nt) return nt;
    if (nt < 2 * kMinTiles) return 2 * t < nt ? 0 : nt;
    return t < kMinTiles ? 0 : (nt - t < kMinTiles ? nt : t);
  }
};

// One item: a pair of query tiles (or a last one alone) and a range of key tiles.
struct Item {
  int index;  // -1: no more
  int b, hk, qt0, dual, whole, rec;  // whole: the range is all of the row; else its record
  int kl, first, sl;         // first: the range's first key
  int nt;                    // key tiles (0: nothing to compute, zero rows)
  int row0;                  // cache column of the first key
};

struct Shared {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2], q_full;
  uint64_t item_full[2], item_empty[2];
  uint64_t drain;
  uint32_t tmem;
  Item item[2];
  float2 join_ml[kQRows];
  float depth[kMaxRows];
  uint32_t anc[2 * kQRows][kMaxRows / 32 + 1];  // ancestor words of the softmax threads' rows
};
constexpr int kItemReaders = 3 + 8;  // the producer warp, both MMA threads, the softmax warps
static_assert(4 * kQHalf + kRingBytes + sizeof(Shared) <= 232448, "shared memory of a CTA");

// Row of q and out ([B][M+1][Hq]) of the gr-th query row of (b, hk).  gr / G by a
// reciprocal: exact for G (M+1) < 2^21, which the host checks.
__device__ __forceinline__ int node_of(const ScoredParams& p, int gr) { return (int)(((float)gr + 0.5f) * p.inv_g); }
__device__ __forceinline__ int64_t query_row(const ScoredParams& p, int b, int hk, int gr) {
  const int node = node_of(p, gr);
  return ((int64_t)b * (p.M + 1) + node) * p.Hq + hk * p.G + (gr - node * p.G);
}

// Whether some thread of the 256 softmax threads says so (a barrier of them all).
__device__ __forceinline__ bool any_of_softmax(bool mine) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, 3, 256, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)mine)
      : "memory");
  return any != 0;
}

// The tensor core takes the weights in bf16, and a row's sum takes them as they are after
// that rounding: the output is then a mean of the V rows whatever the weights' scale (a
// reference far from the maximum rounds the largest weight too, and with the sum of the
// unrounded ones a row of one key would be up to 2^-8 off that key's V).
__device__ __forceinline__ uint64_t weights_of(uint32_t pk) {
  return f2_pack(__uint_as_float(pk << 16), __uint_as_float(pk & 0xffff0000u));
}

// One capped score (log2) from the raw product x.
__device__ __forceinline__ float cap_score(float x, const ScoredParams& p) {
  const float t = x * x;
  float g = p.c[4];
#pragma unroll
  for (int i = 3; i >= 0; --i) g = fmaf(g, t, p.c[i]);
  return fabsf(x) <= p.x_lim ? x * g : p.cap_log2 * (1.f - __fdividef(2.f, fast_exp2(x * p.z2) + 1.f));
}

// 16 scores of a row, minus `sub`, from the raw products x of keys kc .. kc+15, in
// the general form.  ok: the keys that count (used where `edge`; what the others
// hold may be anything, and is replaced at the end).  slope2, pos: the row's bias per position
// (log2) and its position; dep: the tree rows' depths.
template <int MODE>
__device__ __forceinline__ void chunk_scores(float (&x)[16], const ScoredParams& p, bool edge, uint32_t ok, float sub,
                                             float slope2, int pos, int kc, int kl, int M, const float* dep) {
  constexpr bool CAP = MODE == kCapLow || MODE == kCapHigh || MODE == kCapBias;
  constexpr bool BIAS = MODE == kBias || MODE == kCapBias;
  bool far = false;
  if (CAP) {
    float a[2] = {fabsf(x[0]), fabsf(x[1])};
#pragma unroll
    for (int j = 2; j < 16; j += 2) a[(j >> 1) & 1] = fmax3(a[(j >> 1) & 1], fabsf(x[j]), fabsf(x[j + 1]));
    far = __any_sync(0xffffffffu, fmaxf(a[0], a[1]) > p.x_lim);
  }
  if (far) {
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = cap_score(x[j], p);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint64_t v = f2_pack(x[2 * j], x[2 * j + 1]);
      uint64_t g = f2_pack(p.scale_log2, p.scale_log2);
      if (CAP) {
        const uint64_t t = f2_mul(v, v);
        g = f2_pack(p.c[4], p.c[4]);
#pragma unroll
        for (int i = 3; i >= 0; --i) g = f2_fma(g, t, f2_pack(p.c[i], p.c[i]));
      }
      f2_unpack(f2_mul(v, g), x[2 * j], x[2 * j + 1]);
    }
  }
  if (BIAS && kc + 16 > kl) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int t = kc + j - kl;  // tree row
      const float off = t < 0 ? (float)t : dep[min(t, M)];  // the key's position less kl
      x[j] += fmaf(slope2, off - (float)(pos - kl), -sub);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] += BIAS ? fmaf(-slope2, (float)(pos - (kc + j)), -sub) : -sub;
  }
  if (edge) {
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = (ok >> j) & 1u ? x[j] : -INFINITY;
  }
}

template <int D, int MODE, bool FEW>
__global__ void __launch_bounds__(kThreads, 1)
    scored_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                  const __grid_constant__ ScoredParams p) {
  constexpr bool BIAS = MODE == kBias || MODE == kCapBias;
  constexpr bool CAP = MODE == kCapLow || MODE == kCapHigh || MODE == kCapBias;
  constexpr bool TRACK = MODE != kCapLow;  // a running maximum is kept
  constexpr int kHalves = D / 64;
  constexpr int kKeys = keys_of(FEW), kColP = kKeys;
  constexpr int kHalf = kKeys * 128;       // one 64-column half of a K or V tile: rows of 128 B
  constexpr int kChunks = FEW ? 1 : kKeys / 16;  // 16-key chunks that a softmax warp works on
  constexpr int kTile = kHalves * kHalf;   // K or V tile
  constexpr int kQTile = kHalves * kQHalf;
  constexpr int kSlots = kRingBytes / kTile < kMaxSlots ? kRingBytes / kTile : kMaxSlots;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* q_s = smem;                // [2][halves][128][128 B]
  uint8_t* ring = smem + 2 * kQTile;  // [slots][halves][80][128 B]
  Shared* sh = reinterpret_cast<Shared*>(ring + kRingBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], 2);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(&sh->s_full[q], 1);
      mbar_init(&sh->s_free[q], 4);
      mbar_init(&sh->p_full[q], 4);
      mbar_init(&sh->pv_done[q], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->item_full[i], 1);
      mbar_init(&sh->item_empty[i], kItemReaders);
    }
    mbar_init(&sh->q_full, 8);
    mbar_init(&sh->drain, 2);
    fence_mbar_init();
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(&sh->tmem, 512);
    tmem_relinquish();
  }
  pdl_wait_primary();
  pdl_launch_dependents();

  // ---------------------------------------------------------------- the CTA's share
  int* nt_s = reinterpret_cast<int*>(ring);
  int4* geo_s = reinterpret_cast<int4*>(ring + 4 * kMaxBatch);
  for (int b = tid; b < p.B; b += kThreads) {
    const int st = __ldcg(p.status + b);
    const Geo g = sequence<kKeys>(p, b);
    nt_s[b] = g.nt;
    geo_s[b] = make_int4(g.sl, g.ks, g.kl, st);
  }
  __syncthreads();
  const bool aligned_ok = (smem_u32(smem) & 1023u) == 0;  // the swizzled tiles need it (else all sequences fail)
  // Warp 1 walks the rows of the share.  Its place: a sequence with its geometry and
  // status, the units of the sequences before it, and the row inside the sequence.
  struct Place {
    int before, lo, hi;  // units of earlier sequences; the share
    int b, hk, pair, count;
    bool fresh;          // g and st are of another sequence
    Geo g;
    int st, n;           // units of a row
  } at = {};
  Shares shares = {};
  // The next item of the share.
  auto next = [&]() -> Item {
    Item it = {};
    it.index = -1;
    while (at.b < p.B && at.before * p.Hkv * shares.head < at.hi) {
      if (at.fresh) {
        at.st = __ldcg(p.status + at.b);
        at.g = sequence<kKeys>(p, at.b);
        at.n = shares.units_of(tiles_of(at.g.nt));
        at.fresh = false;
      }
      const int nt = tiles_of(at.g.nt);
      const bool dual = 2 * at.pair + 1 < p.nqt;
      const int start = at.before * p.Hkv * shares.head + at.n * (at.hk * shares.head + at.pair * shares.pair);
      if (start >= at.hi) break;
      const int t0 = shares.cut(at.lo, start, nt, at.n, dual), t1 = shares.cut(at.hi, start, nt, at.n, dual);
      if (t0 < t1) {
        it.index = at.count++;
        it.b = at.b;
        it.hk = at.hk;
        it.qt0 = 2 * at.pair;
        it.dual = dual;
        it.whole = t0 == 0 && t1 == nt;
        it.rec = 2 * (2 * blockIdx.x + (t0 > 0 ? 0 : 1));
        it.sl = at.g.sl;
        it.kl = at.g.kl;
        it.first = at.g.first + t0 * kKeys;
        it.row0 = at.g.ks + it.first;
        it.nt = aligned_ok && at.st == 0 && at.g.nt > 0 ? t1 - t0 : 0;
        if (p.ws_row && lane == 0) {
          int2* row = p.ws_row + ((int64_t)at.b * p.Hkv + at.hk) * p.npairs + at.pair;
          if (t0 == 0) __stcg(&row->x, it.whole ? -1 : (int)blockIdx.x);
          if (t1 == nt) __stcg(&row->y, it.whole ? -1 : (int)blockIdx.x);
        }
      }
      if (++at.pair == p.npairs) {
        at.pair = 0;
        if (++at.hk == p.Hkv) {
          at.hk = 0;
          at.before += at.n;
          ++at.b;
          at.fresh = true;
        }
      }
      if (t0 < t1) break;
    }
    return it;
  };
  if (warp == 1) {
    int tiles = 0, longest = 0;
    for (int b = lane; b < p.B; b += 32) {
      tiles += tiles_of(nt_s[b]);
      longest = max(longest, tiles_of(nt_s[b]));
    }
    tiles = __reduce_add_sync(0xffffffffu, tiles);
    longest = __reduce_max_sync(0xffffffffu, longest);
    const int heads = p.Hkv * p.npairs;
    int per = 0, units = tiles;
    if (p.B * heads <= p.grid) {
      per = longest;
      units = p.B;
      if (p.ws_row) {
        // the shortest pieces, of 32 lengths from an even share on, that the CTAs can take
        const int least = max(kMinTiles, (int)((uint32_t)(tiles * heads + p.grid - 1) / (uint32_t)p.grid));
        const int mine = least + lane * ((least + 15) >> 4);
        int n = 0;
#pragma unroll 4
        for (int b = 0; b < p.B; ++b) n += (uint32_t)(tiles_of(nt_s[b]) + mine - 1) / (uint32_t)mine;
        const unsigned m = __ballot_sync(0xffffffffu, n * heads <= p.grid);
        if (m) {
          per = __shfl_sync(0xffffffffu, mine, __ffs(m) - 1);
          units = __shfl_sync(0xffffffffu, n, __ffs(m) - 1);
        }
        const int full = p.nqt > 1 ? 2 : 1;
        if (((int64_t)full * min(per, longest) - kSecondItem) * p.grid > tiles * p.Hkv * p.nqt) {
          per = 0;
          units = tiles;
        }
      }
    }
    shares.set(p, units, per);
    // the sequence in which the share begins
    at.b = p.B;
    if ((int)blockIdx.x < shares.ctas) {
      at.lo = shares.begin(blockIdx.x);
      at.hi = shares.begin(blockIdx.x + 1);
      const int seq = p.Hkv * shares.head;
      int before = 0;
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        const int own = b < p.B ? shares.units_of(tiles_of(nt_s[b])) : 0;
        int incl = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, incl, off);
          if (lane >= off) incl += o;
        }
        const unsigned m = __ballot_sync(0xffffffffu, b < p.B && (before + incl) * seq > at.lo);
        if (m) {
          const int src = __ffs(m) - 1;
          at.b = b0 + src;
          at.before = __shfl_sync(0xffffffffu, before + incl - own, src);
          at.n = __shfl_sync(0xffffffffu, own, src);
          const int4 v = geo_s[at.b];
          at.g = Geo{v.x, v.y, v.z, 0, nt_s[at.b]};
          at.g.first = p.window > 0 ? max(0, at.g.kl - (p.window - 1)) : 0;
          at.st = v.w;
          // the kv head, and the pair, in which it begins
          const uint32_t inside = at.lo - at.before * seq;
          at.hk = inside / (uint32_t)(at.n * shares.head);
          at.pair = (inside - at.hk * at.n * shares.head) / (uint32_t)(at.n * shares.pair);
          break;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    const Item it = next();
    if (lane == 0) {
      sh->item[0] = it;
      mbar_arrive(&sh->item_full[0]);
    }
    __syncwarp();
  }
  fence_async_smem();  // the plan's scratch lies in the ring, which the copies write next
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem;
  const uint64_t lim = p.wait_limit_ns;
  // Waits for a role's `n`-th item.  A role that gives up on a wait of its own still
  // takes its items, so the next one comes once every reader is through with the one
  // before the last: warp 1 waits for that longer than a reader's own waits can add
  // up to, and the readers longer than warp 1, so that all of them see the same list.
  constexpr uint64_t kListWait = 8 * kWaitLimitNs;
  auto next_item = [&](int n) -> Item {
    Item it = {};
    it.index = -1;
    if (mbar_wait(&sh->item_full[n & 1], (n >> 1) & 1, 4 * kListWait)) it = sh->item[n & 1];
    return it;
  };
  // Ring order of an item's tiles: K_0 (and K_1 where the pipes take turns), then
  // V_j, K_{j + la} in turn.  Key tiles are taken from the last to the first: with
  // a bias by distance the largest scores come first, and the reference seldom
  // moves.
  auto k_idx = [](const Item& it, int j) {
    const int la = it.dual ? 1 : 2;
    return j < la ? j : 2 * j - la + 1;
  };
  auto v_idx = [](const Item& it, int j) { return j + min((it.dual ? 1 : 2) + j, it.nt); };

  if (warp < 4) {
    if (warp == 1) {
      // -------------------------------------------------------------- items
      bool stuck = false;
      for (int n = 1;; ++n) {
        const Item it = next();
        if (n >= 2 && !stuck)
          stuck = !__all_sync(0xffffffffu, mbar_wait(&sh->item_empty[n & 1], ((n >> 1) - 1) & 1, kListWait));
        if (stuck) {  // nobody takes these any more: zero rows; the merge still needs the rows' places
          if (it.index < 0) break;
          if (lane == 0) atomicOr(&p.status[it.b], kSeqTimeout);
          const int rows = it.whole ? min(it.dual ? 2 * kQRows : kQRows, p.rows - it.qt0 * kQRows) : 0;
          for (int e = lane; e < rows * (D / 8); e += 32)
            reinterpret_cast<uint4*>(p.out + query_row(p, it.b, it.hk, it.qt0 * kQRows + e / (D / 8)) * D)[e % (D / 8)] =
                make_uint4(0, 0, 0, 0);
          continue;
        }
        if (lane == 0) {
          sh->item[n & 1] = it;
          mbar_arrive(&sh->item_full[n & 1]);
        }
        __syncwarp();
        if (it.index < 0) break;
        if (it.nt > 0) {  // the query rows on their way to L2 while the item before is at work
          const int rows = min(it.dual ? 2 * kQRows : kQRows, p.rows - it.qt0 * kQRows);
          for (int e = lane; e < rows * kHalves; e += 32)
            prefetch_l2(p.q + query_row(p, it.b, it.hk, it.qt0 * kQRows + e / kHalves) * D + e % kHalves * 64);
        }
      }
    } else if (warp == 0) {
      // -------------------------------------------------------------- K and V stream
      // The warp walks the ring; lane 0 requests K tiles, lane 1 V tiles (the copies
      // one thread issues are processed one after another).
      uint32_t idx = 0;  // ring entries so far
      bool failed = false;
      for (int n = 0;; ++n) {
        const Item it = next_item(n);
        if (it.index < 0) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->item_empty[n & 1]);
        const int zc = it.sl * p.Hkv + it.hk, la = it.dual ? 1 : 2;
        for (int kj = 0, vj = 0; vj < it.nt && !failed; ++idx) {
          const uint32_t s = idx % kSlots;
          if (idx >= (uint32_t)kSlots &&
              !__all_sync(0xffffffffu, mbar_wait(&sh->empty[s], ((idx / kSlots) - 1) & 1, lim))) {
            failed = true;
            break;
          }
          // The first query tiles come before the ring's fill: every CTA starts with
          // both, and the products wait for the queries.
          if (idx == 2 && kj + vj == 2 && !__all_sync(0xffffffffu, mbar_wait(&sh->q_full, 0, lim))) {
            failed = true;
            break;
          }
          const bool is_k = kj < it.nt && kj - vj < la;
          const int j = is_k ? kj++ : vj++;
          if (lane == (is_k ? 0 : 1)) {
            const CUtensorMap* map = is_k ? &tmk : &tmv;
            mbar_arrive_expect_tx(&sh->full[s], kTile);
            const int row = it.row0 + (it.nt - 1 - j) * kKeys;
            if (D == 128)
              tma_load_4d(ring + s * kTile, map, &sh->full[s], 0, row, 0, zc);
            else
              tma_load_3d(ring + s * kTile, map, &sh->full[s], 0, row, zc);
          }
          __syncwarp();
        }
      }
      // Every copy must land before the shared memory is released, one that no MMA waits
      // for as well: a pipe may still give up after this warp is through.
      for (uint32_t i = 1; i <= (uint32_t)kSlots && i <= idx; ++i)
        mbar_wait(&sh->full[(idx - i) % kSlots], ((idx - i) / kSlots) & 1);
    } else if (lane == 0) {
      // -------------------------------------------------------------- MMA issue, one thread per pipe
      const int q = warp - 2;
      const uint32_t idesc_s = idesc_bf16(128, kKeys, 0), idesc_o = idesc_bf16(128, D, 1);
      const uint32_t t_q = tmem + q * 256;
      uint32_t base = 0, step0 = 0, busy = 0;  // ring entries, steps and items with work so far
      bool ok = true;
      for (int n = 0;; ++n) {
        const Item it = next_item(n);
        if (it.index < 0) break;
        mbar_arrive(&sh->item_empty[n & 1]);
        if (it.nt == 0 || !ok) continue;
        const bool dual = it.dual;
        const int steps = dual ? it.nt : (it.nt + 1 - q) / 2;
        // Each pipe waits for every entry of the ring in its order, the other pipe's as
        // well: a barrier's parity tells a landed copy from a pending one only to who
        // has seen the slot's copy before.  A slot is free once both pipes are through
        // with it: with their products, or by having seen that it is the other's.
        const int la = dual ? 1 : 2;
        int seen = 0, kj = 0, vj = 0;
        auto see = [&](int entry) -> bool {
          for (; seen <= entry; ++seen) {
            const uint32_t idx = base + seen, s = idx % kSlots;
            if (!mbar_wait(&sh->full[s], (idx / kSlots) & 1, lim)) return false;
            const bool is_k = kj < it.nt && kj - vj < la;
            const int j = is_k ? kj++ : vj++;
            if (!dual && (j & 1) != q) mbar_arrive(&sh->empty[s]);
          }
          return true;
        };
        auto qk = [&](int i) -> bool {
          const int entry = k_idx(it, dual ? i : 2 * i + q);
          const uint32_t s = (base + entry) % kSlots, st = step0 + i;
          if (!see(entry)) return false;
          if (st > 0 && !mbar_wait(&sh->s_free[q], (st - 1) & 1, lim)) return false;
          tc_fence_after();
          const uint64_t da = sw128_desc(smem_u32(q_s + (dual ? q : 0) * kQTile), 16);
          const uint64_t db = sw128_desc(smem_u32(ring + s * kTile), 16);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss(t_q, da + (uint64_t)((k >> 2) * (kQHalf / 16) + (k & 3) * 2),
                   db + (uint64_t)((k >> 2) * (kHalf / 16) + (k & 3) * 2), idesc_s, k > 0 ? 1u : 0u);
          tc_commit(&sh->s_full[q]);
          tc_commit(&sh->empty[s]);
          return true;
        };
        ok = mbar_wait(&sh->q_full, busy & 1, lim) && (steps == 0 || qk(0));
        for (int i = 0; i < steps && ok; ++i) {
          if (i + 1 < steps && !(ok = qk(i + 1))) break;
          const int entry = v_idx(it, dual ? i : 2 * i + q);
          const uint32_t s = (base + entry) % kSlots;
          ok = see(entry) && mbar_wait(&sh->p_full[q], (step0 + i) & 1, lim);
          if (!ok) break;
          tc_fence_after();
          const uint64_t db = sw128_desc(smem_u32(ring + s * kTile), kHalf);
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            mma_ts(t_q + kColO, t_q + kColP + k * 8, db + (uint64_t)(k * (16 * 128 / 16)), idesc_o,
                   (i > 0 || k > 0) ? 1u : 0u);
          tc_commit(&sh->pv_done[q]);
          tc_commit(&sh->empty[s]);
        }
        ok = ok && see(2 * it.nt - 1);
        ++busy;
        base += 2 * it.nt;
        step0 += steps;
      }
      // every MMA issued retires before TMEM and shared memory are released
      tc_commit(&sh->drain);
      mbar_wait(&sh->drain, 0);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int pipe = (warp - 4) >> 2;
    const int r = (warp & 3) * 32 + lane;
    const int stid = tid - 128;  // of the 256 softmax threads
    const uint32_t t_row = tmem + pipe * 256 + ((uint32_t)((warp & 3) * 32) << 16), t_o = t_row + kColO;
    const uint32_t t_s = t_row + (FEW ? (warp & 3) * 16 : 0), t_p = t_row + kColP + (FEW ? (warp & 3) * 8 : 0);
    if (FEW) {  // the other warps' keys have no weight in this warp's rows
      uint32_t z[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) z[e] = 0u;
      tmem_st32(t_row + kColP, z);
      tmem_wait_st();
    }
    uint32_t base = 0, step0 = 0;  // ring entries and steps of earlier items
    bool to = false;  // a wait ran out: zero rows from here on
    for (int n_item = 0;; ++n_item) {
    const Item g = next_item(n_item);
    if (g.index < 0) break;
    const bool dual = !FEW && g.dual;
    const int nt = g.nt, hk = g.hk, b = g.b;
    const int qt = dual ? g.qt0 + pipe : g.qt0;
    const int gr = FEW ? lane : qt * kQRows + r;
    const bool row_ok = gr < p.rows;
    const bool warp_live = __any_sync(0xffffffffu, row_ok);
    const int u = min(node_of(p, min(gr, p.rows - 1)), p.M);
    if (nt > 0) {  // query rows -> swizzled shared memory; the tree rows' depths
      // A thread brings one 16-byte column of every 16th (D = 128) or 32nd row, all
      // its requests in flight at once.
      // Few rows: every warp's 32 TMEM lanes get the same ones.
      constexpr int kC = D / 8, kStep = 256 / kC, kN = (FEW ? 1 : 2) * kQRows / kStep;
      constexpr int kLoads = FEW ? kFewRows / kStep : kN;
      const int c = stid % kC, r0 = stid / kC;
      uint4 v[kLoads];
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int gr = g.qt0 * kQRows + r0 + k * kStep;
        v[k] = make_uint4(0, 0, 0, 0);
        if (gr < p.rows && (FEW || dual || k < kN / 2))
          v[k] = __ldg(reinterpret_cast<const uint4*>(p.q + query_row(p, b, hk, gr) * D) + c);
      }
      constexpr int kW = kMaxRows / 32;
      uint32_t a[kW];
      const int64_t node = (int64_t)b * (p.M + 1) + u;
#pragma unroll
      for (int i = 0; i < kW; ++i) a[i] = i < p.W ? __ldg(p.anc + node * p.W + i) : 0u;
      const int d = p.depth && stid <= p.M ? __ldg(p.depth + (int64_t)b * (p.M + 1) + stid) : 0;
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const int row = r0 + k * kStep, rr = row & (kQRows - 1);
        if (FEW || dual || k < kN / 2)
          *reinterpret_cast<uint4*>(q_s + (row / kQRows) * kQTile + (c >> 3) * kQHalf + rr * 128 +
                                    (((c & 7) ^ (rr & 7)) << 4)) = v[k % kLoads];
      }
#pragma unroll
      for (int i = 0; i < kW; ++i) sh->anc[stid][i] = a[i];
      if (stid <= p.M) sh->depth[stid] = (float)d;
      fence_async_smem();
      tc_fence_before();
      asm volatile("bar.sync 3, 256;" ::: "memory");
      if (lane == 0) mbar_arrive(&sh->q_full);
    }
    const int du = (p.window > 0 || BIAS) && nt > 0 ? (int)sh->depth[u] : 0;
    const float slope2 =
        BIAS ? __ldg(p.slopes + hk * p.G + (row_ok ? gr - u * p.G : 0)) * 1.4426950408889634f : 0.f;
    const int pos = g.kl + du;
    const int lo = p.window > 0 ? max(0, pos - (p.window - 1)) : 0;  // first prefix key of the row
    const int n = dual ? nt : (pipe == 0 ? (nt + 1) / 2 : nt / 2);
    float m = TRACK ? -INFINITY : p.ref, l = 0.f;
    uint64_t l2[2] = {0ull, 0ull};
    for (int i = 0; i < n && !to; ++i) {
      const int j = dual ? i : 2 * i + pipe;
      if (!__all_sync(0xffffffffu, mbar_wait(&sh->s_full[pipe], (step0 + i) & 1, lim))) {
        to = true;
        break;
      }
      tc_fence_after();
      const int key0 = g.first + (nt - 1 - j) * kKeys;  // of the sequence
      const int wkey0 = key0 + (FEW ? (warp & 3) * 16 : 0);  // of the warp's chunks
      // S is read: the next S may be formed while this one's weights are
      auto free_s = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->s_free[pipe]);
      };
      // the products with the weights before these are done: P and O are free
      auto wait_pv = [&]() -> bool {
        if (i > 0 && !__all_sync(0xffffffffu, mbar_wait(&sh->pv_done[pipe], (step0 + i - 1) & 1, lim))) return false;
        tc_fence_after();
        return true;
      };
      bool s_kept = true;
      if (warp_live) {
        const bool edge = __any_sync(0xffffffffu, wkey0 + kChunks * 16 > g.kl || wkey0 < lo);
        bool done = false;
        // A tile inside the prefix: the exponents with the reference at hand, in one
        // pass.  The general path takes over if a row has no reference yet (no key so
        // far), a score lies outside the polynomial's range or above the reference's
        // headroom.
        if (!edge && (!TRACK || __all_sync(0xffffffffu, m != -INFINITY))) {
          const float sub = m;
          const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2);
          const uint64_t step2 = f2_pack(2.f * slope2, 2.f * slope2);
          uint32_t x[kChunks][16];
#pragma unroll
          for (int c = 0; c < kChunks; ++c) tmem_ld16(t_s + c * 16, x[c]);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) tmem_wait_ld16(x[c]);
          // exponents of a pair of keys
          auto exponents = [&](int c, int e, float base, uint64_t& add, float& a0, float& a1) {
            const uint64_t v = f2_pack(__uint_as_float(x[c][2 * e]), __uint_as_float(x[c][2 * e + 1]));
            uint64_t gf = sc2;
            if (CAP) {
              const uint64_t t = f2_mul(v, v);
              gf = f2_pack(p.c[4], p.c[4]);
#pragma unroll
              for (int d = 3; d >= 0; --d) gf = f2_fma(gf, t, f2_pack(p.c[d], p.c[d]));
            }
            if (BIAS)
              add = (e & 3) == 0 ? f2_pack(fmaf(slope2, (float)(2 * e), base), fmaf(slope2, (float)(2 * e + 1), base))
                                 : f2_add(add, step2);
            f2_unpack(f2_fma(v, gf, add), a0, a1);
          };
          // Does a score lie outside?  The largest product says so (its magnitude, for
          // the polynomial), except with a bias, where the exponents are formed first.
          float am[2] = {0.f, 0.f}, sm[2] = {-INFINITY, -INFINITY};
          if (CAP || !BIAS) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float x0 = __uint_as_float(x[c][2 * e]), x1 = __uint_as_float(x[c][2 * e + 1]);
                if (CAP) am[e & 1] = fmax3(am[e & 1], fabsf(x0), fabsf(x1));
                else sm[e & 1] = fmax3(sm[e & 1], x0, x1);
              }
          }
          if (BIAS) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              const float base = -slope2 * (float)(pos - wkey0 - 16 * c) - sub;
              uint64_t add = 0;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                float a0, a1;
                exponents(c, e, base, add, a0, a1);
                sm[e & 1] = fmax3(sm[e & 1], a0, a1);
                x[c][2 * e] = __float_as_uint(a0);
                x[c][2 * e + 1] = __float_as_uint(a1);
              }
            }
          }
          const float amx = fmaxf(am[0], am[1]), smx = fmaxf(sm[0], sm[1]);
          const bool redo = (CAP && amx > p.x_lim) || (BIAS && smx > kGrow) ||
                            (MODE == kPlain && smx * p.scale_log2 - sub > kGrow) ||
                            (MODE == kCapHigh && cap_score(amx, p) - sub > kGrow);
          if (!__any_sync(0xffffffffu, redo)) {
            free_s();
            s_kept = false;
            done = true;
            uint32_t pk[kChunks][8];
            uint64_t sub2 = f2_pack(-sub, -sub);
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                float a0 = __uint_as_float(x[c][2 * e]), a1 = __uint_as_float(x[c][2 * e + 1]);
                if (!BIAS) exponents(c, e, 0.f, sub2, a0, a1);
                pk[c][e] = pack_bf16x2(fast_exp2(a0), fast_exp2(a1));
                l2[e & 1] = f2_add(l2[e & 1], weights_of(pk[c][e]));
              }
            if (!wait_pv()) {
              to = true;
              break;
            }
#pragma unroll
            for (int c = 0; c < kChunks; ++c) tmem_st8(t_p + c * 8, pk[c]);
          }
        }
        if (!done) {
          // the keys kc .. kc+15 that the row may read
          auto allowed = [&](int kc) -> uint32_t {
            const int np = g.kl - kc;
            uint32_t w = np >= 32 ? ~0u : (np <= 0 ? 0u : (1u << np) - 1u);
            if (lo > kc) w &= lo - kc >= 32 ? 0u : ~0u << (lo - kc);
            const int r0 = kc - g.kl;  // tree row of bit 0
            if (r0 > -32 && r0 <= p.M) {
              const uint32_t* a = sh->anc[stid];
              uint32_t t;
              if (r0 <= 0) {
                t = a[0] << -r0;
              } else {
                const int wi = r0 >> 5, sft = r0 & 31;
                t = a[wi] >> sft;
                if (sft && wi + 1 < p.W) t |= a[wi + 1] << (32 - sft);
              }
              if (p.M + 1 - r0 < 32) t &= (1u << (p.M + 1 - r0)) - 1u;
              if (p.window > 0)
                for (uint32_t s = t; s; s &= s - 1) {
                  const int bit = __ffs(s) - 1;
                  if (du - (int)sh->depth[r0 + bit] >= p.window) t &= ~(1u << bit);
                }
              w |= t;
            }
            return w;
          };
          // scores of keys kc .. kc+15 less `sub`
          auto scores = [&](int c, float sub, float (&x)[16]) {
            uint32_t raw[16];
            tmem_ld16(t_s + c * 16, raw);
            const uint32_t ok = edge ? allowed(wkey0 + 16 * c) : ~0u;
            tmem_wait_ld16(raw);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(raw[e]);
            chunk_scores<MODE>(x, p, edge, ok, sub, slope2, pos, wkey0 + 16 * c, g.kl, p.M, sh->depth);
          };
          if (TRACK) {  // first the maximum; the scores wait in S's place
            float mx = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
              float x[16];
              scores(c, 0.f, x);
              float a[2] = {fmaxf(mx, x[0]), x[1]};
#pragma unroll
              for (int e = 2; e < 16; e += 2) a[(e >> 1) & 1] = fmax3(a[(e >> 1) & 1], x[e], x[e + 1]);
              mx = fmaxf(a[0], a[1]);
              uint32_t back[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) back[e] = __float_as_uint(x[e]);
              tmem_st16(t_s + c * 16, back);
            }
            tmem_wait_st();
            if (!wait_pv()) {
              to = true;
              break;
            }
            // The reference follows the maximum lazily: O is rescaled (a TMEM access of
            // the whole warp, each row by its own factor) only when some row's maximum
            // has grown by more than 2^kGrow; then every row's follows.
            const bool grow = __any_sync(0xffffffffu, mx > m + kGrow) ? mx > m : false;
            const bool scale_o = grow && m != -INFINITY;
            if (__any_sync(0xffffffffu, scale_o)) {
              const float corr = scale_o ? fast_exp2(m - mx) : 1.f;
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(t_o + c * 32, o);
                tmem_wait_ld32(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                tmem_st32(t_o + c * 32, o);
              }
              float s0, s1, s2, s3;
              f2_unpack(l2[0], s0, s1);
              f2_unpack(l2[1], s2, s3);
              l = (l + ((s0 + s1) + (s2 + s3))) * corr;
              l2[0] = l2[1] = 0ull;
            }
            if (grow) m = mx;
          } else if (!wait_pv()) {
            to = true;
            break;
          }
          const float sub = m == -INFINITY ? 0.f : m;
#pragma unroll 1
          for (int c = 0; c < kChunks; ++c) {
            float x[16];
            if (TRACK) {
              uint32_t raw[16];
              tmem_ld16(t_s + c * 16, raw);
              tmem_wait_ld16(raw);
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(raw[e]) - sub;
            } else {
              scores(c, sub, x);
            }
            uint32_t pk[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              pk[e] = pack_bf16x2(fast_exp2(x[2 * e]), fast_exp2(x[2 * e + 1]));
              l2[e & 1] = f2_add(l2[e & 1], weights_of(pk[e]));
            }
            tmem_st8(t_p + c * 8, pk);
          }
        }
        tmem_wait_st();
      } else if (!wait_pv()) {  // (no row of this warp is real; a parity wait must not fall behind)
        to = true;
        break;
      }
      if (s_kept) free_s();
      // V rows behind the step's may hold anything: zero them (where the pipes share
      // the tile, both do, each before its own product)
      const int kend = g.kl + p.M + 1 - key0;
      if (kend < kKeys) {
        const uint32_t idx = base + v_idx(g, j), s = idx % kSlots;
        if (!__all_sync(0xffffffffu, mbar_wait(&sh->full[s], (idx / kSlots) & 1, lim))) {
          to = true;
          break;
        }
        uint8_t* vt = ring + s * kTile;
        for (int e = r; e < (kKeys - kend) * (D / 8); e += kQRows) {
          const int row = kend + e / (D / 8), c = e % (D / 8);
          *reinterpret_cast<uint4*>(vt + (c >> 3) * kHalf + row * 128 + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->p_full[pipe]);
    }
    {
      float s0, s1, s2, s3;
      f2_unpack(l2[0], s0, s1);
      f2_unpack(l2[1], s2, s3);
      l += (s0 + s1) + (s2 + s3);
    }
    if (n > 0 && !to && !mbar_wait(&sh->pv_done[pipe], (step0 + n - 1) & 1, lim)) to = true;
    to = __any_sync(0xffffffffu, to);
    bool have = n > 0 && !to;
    if (to && lane == 0) atomicOr(&p.status[b], kSeqTimeout);
    tc_fence_after();
    // Both pipes' products have read the query tile.  Where they shared it, a row is the sum
    // of the two (with few rows, of all eight warps): if one gave up, none of it counts.
    if (!dual && any_of_softmax(to)) have = false;
    if (!have) {
      m = -INFINITY;
      l = 0.f;
    }
    // ---------------------------------------------------------------- epilogue
    // Pipes that shared a query tile join: the second hands its O, reference and
    // sum to the first through the query tiles' memory.
    float4* join_o = reinterpret_cast<float4*>(q_s);  // [D / 4][128]
    float w0 = 1.f, w1 = 0.f;
    if (!dual) {
      if (pipe == 1) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (have) {
            tmem_ld32(t_o + c * 32, o);
            tmem_wait_ld32(o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            join_o[(c * 8 + e) * kQRows + r] =
                make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]),
                            __uint_as_float(o[4 * e + 3]));
        }
        sh->join_ml[r] = make_float2(m, l);
      }
      asm volatile("bar.sync 3, 256;" ::: "memory");
      if (pipe == 0) {
        const float2 o = sh->join_ml[r];
        const float mm = fmaxf(m, o.x), ms = mm == -INFINITY ? 0.f : mm;
        w0 = fast_exp2(m - ms);  // 0 for a pipe without keys
        w1 = fast_exp2(o.x - ms);
        l = l * w0 + o.y * w1;
        m = mm;
      }
    }
    if (FEW && pipe == 0) {
      // The warps' parts of the keys join as well: each row's four sums of O, then the
      // D / 8 columns of all rows dealt to the pipe's threads.
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (have) {
          tmem_ld32(t_o + c * 32, o);
          tmem_wait_ld32(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float4& x = join_o[(c * 8 + e) * kQRows + r];
          x = make_float4(fmaf(x.x, w1, __uint_as_float(o[4 * e]) * w0), fmaf(x.y, w1, __uint_as_float(o[4 * e + 1]) * w0),
                          fmaf(x.z, w1, __uint_as_float(o[4 * e + 2]) * w0),
                          fmaf(x.w, w1, __uint_as_float(o[4 * e + 3]) * w0));
        }
      }
      sh->join_ml[r] = make_float2(m, l);
      asm volatile("bar.sync 1, 128;" ::: "memory");
      for (int e = r; e < p.rows * (D / 8); e += kQRows) {
        const int c = e / p.rows, row = e - c * p.rows;
        float2 ml[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) ml[i] = sh->join_ml[32 * i + row];
        const float mm = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), ms = mm == -INFINITY ? 0.f : mm;
        float sum = 0.f;
        float4 a[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float w = fast_exp2(ml[i].x - ms);
          sum = fmaf(ml[i].y, w, sum);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 x = join_o[(2 * c + h) * kQRows + 32 * i + row];
            a[h] = make_float4(fmaf(x.x, w, a[h].x), fmaf(x.y, w, a[h].y), fmaf(x.z, w, a[h].z), fmaf(x.w, w, a[h].w));
          }
        }
        if (g.whole) {
          const float inv = sum > 0.f ? 1.f / sum : 0.f;
          reinterpret_cast<uint4*>(p.out + query_row(p, b, hk, row) * D)[c] =
              make_uint4(pack_bf16x2(a[0].x * inv, a[0].y * inv), pack_bf16x2(a[0].z * inv, a[0].w * inv),
                         pack_bf16x2(a[1].x * inv, a[1].y * inv), pack_bf16x2(a[1].z * inv, a[1].w * inv));
        } else {
          float4* dst = reinterpret_cast<float4*>(p.ws_o) + (int64_t)g.rec * (D / 4) * p.rec_rows;
          __stcg(dst + (2 * c) * p.rec_rows + row, a[0]);
          __stcg(dst + (2 * c + 1) * p.rec_rows + row, a[1]);
          if (c == 0) __stcg(p.ws_ml + (int64_t)g.rec * p.rec_rows + row, make_float2(mm, sum));
        }
      }
    }
    if (!FEW && (dual || pipe == 0)) {
      const bool whole = g.whole;
      const float inv = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
      w0 *= inv;
      w1 *= inv;
      uint8_t* stage = q_s + pipe * kQTile;  // of a pair: this pipe's query tile, [128 rows][2 D bytes], chunks rotated
      const int64_t rec = g.rec + pipe;
      float4* dst = reinterpret_cast<float4*>(p.ws_o) + rec * (D / 4) * p.rec_rows;
      uint4* out_row = reinterpret_cast<uint4*>(p.out + query_row(p, b, hk, min(gr, p.rows - 1)) * D);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (have) {
          tmem_ld32(t_o + c * 32, o);
          tmem_wait_ld32(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        float4 a[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          a[e] = make_float4(__uint_as_float(o[4 * e]) * w0, __uint_as_float(o[4 * e + 1]) * w0,
                             __uint_as_float(o[4 * e + 2]) * w0, __uint_as_float(o[4 * e + 3]) * w0);
          if (!dual) {
            const float4 x = join_o[(c * 8 + e) * kQRows + r];
            a[e] = make_float4(fmaf(x.x, w1, a[e].x), fmaf(x.y, w1, a[e].y), fmaf(x.z, w1, a[e].z),
                               fmaf(x.w, w1, a[e].w));
          }
        }
        if (whole) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 x = a[2 * e], y = a[2 * e + 1];
            const int chunk = c * 4 + e;
            const uint4 v = make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w), pack_bf16x2(y.x, y.y),
                                       pack_bf16x2(y.z, y.w));
            if (dual)
              *reinterpret_cast<uint4*>(stage + r * (2 * D) + ((chunk ^ (r & 7)) << 4)) = v;
            else if (row_ok)
              out_row[chunk] = v;
          }
        } else if (row_ok) {
#pragma unroll
          for (int e = 0; e < 8; ++e) __stcg(dst + (int64_t)(c * 8 + e) * p.rec_rows + r, a[e]);
        }
      }
      if (whole && dual) {
        asm volatile("bar.sync %0, 128;" ::"r"(1 + pipe) : "memory");
        const int rows = min(kQRows, p.rows - qt * kQRows);
        for (int e = r; e < rows * (D / 8); e += kQRows) {
          const int rr = e / (D / 8), chunk = e % (D / 8);
          reinterpret_cast<uint4*>(p.out + query_row(p, b, hk, qt * kQRows + rr) * D)[chunk] =
              *reinterpret_cast<const uint4*>(stage + rr * (2 * D) + ((chunk ^ (rr & 7)) << 4));
        }
      } else if (!whole && row_ok) {
        __stcg(p.ws_ml + rec * p.rec_rows + r, make_float2(m, l));
      }
    }
    if (g.sl < 0 && stid == 0) atomicOr(&p.status[b], kSeqBadGeometry);
    base += 2 * nt;
    step0 += n;
    // the query tiles and depths are free for the next item
    asm volatile("bar.sync 3, 256;" ::: "memory");
    if (lane == 0) mbar_arrive(&sh->item_empty[n_item & 1]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (!aligned_ok && tid == 0)
    for (int b = 0; b < p.B; ++b) atomicOr(&p.status[b], kSeqTimeout);
}

// Joins the records of the rows that were cut: out = sum_i 2^(m_i - m) O_i / sum_i
// 2^(m_i - m) l_i.  Block x: a query tile of a (sequence, kv head); one thread per
// row and four columns.
template <int D>
__global__ void __launch_bounds__(256) scored_merge_kernel(const __grid_constant__ ScoredParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  const int qt = blockIdx.x % p.nqt, hk = blockIdx.x / p.nqt % p.Hkv, b = blockIdx.x / p.nqt / p.Hkv;
  const int2 ctas = __ldcg(p.ws_row + ((int64_t)b * p.Hkv + hk) * p.npairs + qt / 2);
  if (ctas.x < 0) return;
  const int nr = ctas.y - ctas.x + 1;
  // the pieces lie in CTAs one after another, the first at its end, the others at their starts
  auto record = [&](int i) -> int64_t { return 2 * (2 * (ctas.x + i) + (i == 0)) + (qt & 1); };
  const int rows = min(kQRows, p.rows - qt * kQRows);
  const bool fail = p.status[b] != 0;
  const float4* ws_o = reinterpret_cast<const float4*>(p.ws_o);
  for (int e = blockIdx.y * 256 + tid; e < rows * (D / 4); e += gridDim.y * 256) {
    const int r = e % rows, c = e / rows;
    float mx = -INFINITY, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 8;  // records in flight
    for (int i0 = 0; i0 < nr; i0 += U) {
      float2 ml[U];
      float4 o[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        ml[i] = make_float2(-INFINITY, 0.f);
        o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i0 + i < nr) {
          const int64_t rec = record(i0 + i);
          ml[i] = __ldcg(p.ws_ml + rec * p.rec_rows + r);
          o[i] = __ldcg(ws_o + (rec * (D / 4) + c) * p.rec_rows + r);
        }
      }
      float mm = mx;
#pragma unroll
      for (int i = 0; i < U; ++i) mm = fmaxf(mm, ml[i].x);
      const float ms = mm == -INFINITY ? 0.f : mm;
      const float w = fast_exp2(mx - ms);
      l *= w;
      a = make_float4(a.x * w, a.y * w, a.z * w, a.w * w);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const float wi = fast_exp2(ml[i].x - ms);
        l = fmaf(wi, ml[i].y, l);
        a = make_float4(fmaf(wi, o[i].x, a.x), fmaf(wi, o[i].y, a.y), fmaf(wi, o[i].z, a.z), fmaf(wi, o[i].w, a.w));
      }
      mx = mm;
    }
    const float inv = !fail && l > 0.f ? 1.f / l : 0.f;
    uint2 v = make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
    if (fail) v = make_uint2(0u, 0u);
    *reinterpret_cast<uint2*>(p.out + query_row(p, b, hk, qt * kQRows + r) * D + 4 * c) = v;
  }
}

// [BH][S_cap][D] bf16 in boxes of `keys` rows: 64 columns (D = 64), or both 64-column
// halves of a row (D = 128), landing as [half][row][128 B], 128-byte swizzle.
bool encode_scored_map(CUtensorMap* map, const void* base, int64_t BH, int64_t S_cap, int D, int keys) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  const cuuint64_t S = (cuuint64_t)std::max<int64_t>(S_cap, 1);
  if (D == 128) {
    cuuint64_t dims[4] = {64, S, 2, (cuuint64_t)BH};
    cuuint64_t strides[3] = {256, 128, S * 256};
    cuuint32_t box[4] = {64, (cuuint32_t)keys, 2, 1}, estr[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  cuuint64_t dims[3] = {64, S, (cuuint64_t)BH};
  cuuint64_t strides[2] = {128, S * 128};
  cuuint32_t box[3] = {64, (cuuint32_t)keys, 1}, estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Grid and workspace of a shape (lengths are known on the device only).
struct ScoredPlan {
  int few, grid, nqt, npairs, merge, rec_rows;
  size_t ml_off, row_off, ws_bytes;  // records, (reference, sum) pairs, rows' CTAs
};

tv_status plan_scored(int B, int M, int Hq, int Hkv, int D, int64_t S_cap, int window, ScoredPlan& lp) {
  const int rows = (Hq / Hkv) * (M + 1);
  lp.nqt = (rows + kQRows - 1) / kQRows;
  lp.npairs = (lp.nqt + 1) / 2;
  lp.rec_rows = std::min(kQRows, rows);
  int64_t keys = std::max<int64_t>(S_cap, 1);
  if (window > 0) keys = std::min<int64_t>(keys, (int64_t)window - 1 + M + 1);
  // shorter rows are never cut
  // the dealing counts the key tiles of all rows of work in 31 bits
  if ((double)((keys + keys_of(true) - 1) / keys_of(true)) * Hkv * B * lp.nqt > (double)(1 << 30))
    return TV_ERR_UNSUPPORTED;
  const tv_status r = current_sms(lp.grid);
  if (r != TV_OK) return r;
  lp.few = rows <= kFewRows && keys * B * Hkv <= (int64_t)kFewKeys * lp.grid;
  const int64_t tiles = (keys + keys_of(lp.few) - 1) / keys_of(lp.few);
  lp.merge = tiles >= 2 * kMinTiles;
  const size_t recs = lp.merge ? 4 * (size_t)lp.grid * lp.rec_rows : 0;
  lp.ml_off = recs * D * sizeof(float);
  lp.row_off = lp.ml_off + recs * sizeof(float2);
  lp.ws_bytes = lp.merge ? lp.row_off + (size_t)B * Hkv * lp.npairs * sizeof(int2) : 0;
  return TV_OK;
}

template <int D, bool FEW>
auto scored_kernel_of(int mode) {
  return mode == kPlain     ? scored_kernel<D, kPlain, FEW>
         : mode == kCapLow  ? scored_kernel<D, kCapLow, FEW>
         : mode == kCapHigh ? scored_kernel<D, kCapHigh, FEW>
         : mode == kBias    ? scored_kernel<D, kBias, FEW>
                            : scored_kernel<D, kCapBias, FEW>;
}

template <int D>
tv_status launch_scored(int mode, const CUtensorMap& tmk, const CUtensorMap& tmv, const ScoredParams& p,
                        const ScoredPlan& lp, cudaStream_t s) {
  auto kern = lp.few ? scored_kernel_of<D, true>(mode) : scored_kernel_of<D, false>(mode);
  const size_t smem = 2 * (D / 64) * kQHalf + kRingBytes + sizeof(Shared);
  tv_status r = allow_shared(reinterpret_cast<const void*>(kern), (int)smem);
  if (r != TV_OK) return r;
  const int64_t units = (int64_t)p.B * p.Hkv * p.nqt;
  r = launch(kern, dim3((unsigned)p.grid), dim3(kThreads), smem, s, 1, true, tmk, tmv, p);
  if (r != TV_OK || !lp.merge) return r;
  // About eight blocks an SM, and at least one for each query tile: a block whose tile has
  // no pieces leaves at once.
  const int parts = std::max(1, (int)std::min<int64_t>((lp.rec_rows * (D / 4) + 255) / 256, 8 * lp.grid / units));
  return launch(scored_merge_kernel<D>, dim3((unsigned)units, parts), dim3(256), 0, s, 1, true, p);
}

}  // namespace
}  // namespace tv

extern "C" size_t tree_attention_scored_workspace_size(int B, int M, int Hq, int Hkv, int D, int64_t S_cap,
                                                       int window) {
  using namespace tv;
  if (B <= 0 || M < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || (D != 64 && D != 128) || M + 1 > kMaxRows ||
      S_cap < 0 || window < 0 || (int64_t)(Hq / Hkv) * (M + 1) >= (1 << 21))
    return 0;
  ScoredPlan lp;
  return plan_scored(B, M, Hq, Hkv, D, S_cap, window, lp) == TV_OK ? lp.ws_bytes : 0;
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
  if (M + 1 > kMaxRows || S_cap > 0x7fffffffLL || B > kMaxBatch) return TV_ERR_UNSUPPORTED;
  // the polynomial's coefficients hold (scale / softcap)^8
  if (softcap > 0.f && scale / softcap > 1e4f) return TV_ERR_UNSUPPORTED;
  if ((int64_t)(Hq / Hkv) * (M + 1) >= (1 << 21)) return TV_ERR_UNSUPPORTED;
  if (B == 0) return TV_OK;
  if (!q || !k || !v || !kv_start || !kv_len || !anc_mask || !status || !out) return TV_ERR_INVALID_ARG;
  if ((window > 0 || alibi_slopes) && !depth) return TV_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return TV_ERR_INVALID_ARG;
  ScoredPlan lp;
  tv_status r = plan_scored(B, M, Hq, Hkv, D, S_cap, window, lp);
  if (r != TV_OK) return r;
  if (lp.ws_bytes > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < lp.ws_bytes))
    return TV_ERR_INVALID_ARG;
  ScoredParams p = {};
  p.q = q;
  p.kv_start = kv_start;
  p.kv_len = kv_len;
  p.depth = depth;
  p.slot = slot;
  p.anc = anc_mask;
  p.status = status;
  p.slopes = alibi_slopes;
  p.out = out;
  p.S_cap = S_cap;
  p.B = B;
  p.M = M;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.W = (M + 1 + 31) / 32;
  p.n_slots = slot ? n_slots : B;
  p.window = window;
  p.inv_g = 1.f / (float)p.G;
  p.rows = p.G * (M + 1);
  p.nqt = lp.nqt;
  p.npairs = lp.npairs;
  p.rec_rows = lp.rec_rows;
  // rows that are never cut want no more CTAs than there are rows
  p.grid = lp.merge ? lp.grid : (int)std::min<int64_t>(lp.grid, (int64_t)B * Hkv * lp.npairs);
  const double log2e = 1.4426950408889634;
  p.scale_log2 = (float)(scale * log2e);
  int mode = alibi_slopes ? kBias : kPlain;
  if (softcap > 0.f) {
    const double z = (double)scale / softcap, cap2 = softcap * log2e;
    double f = scale * log2e;
    for (int i = 0; i < 5; ++i, f *= z * z) p.c[i] = (float)(kPoly[i] * f);
    p.x_lim = (float)std::min(kPolyLim / z, 3e38);
    p.z2 = (float)(2.0 * z * log2e);
    p.cap_log2 = (float)cap2;
    mode = alibi_slopes ? kCapBias : (cap2 <= kLowCap ? kCapLow : kCapHigh);
    // exponents lie in [-cap2 - ref, cap2 - ref], inside [-110, 60]
    p.ref = (float)std::min(cap2, 110.0 - cap2);
  }
  p.wait_limit_ns = pipeline_wait_limit_ns();
  if (lp.merge) {
    p.ws_o = static_cast<float*>(workspace);
    p.ws_ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) + lp.ml_off);
    p.ws_row = reinterpret_cast<int2*>(static_cast<char*>(workspace) + lp.row_off);
  }
  CUtensorMap tmk, tmv;
  const int64_t BH = (int64_t)p.n_slots * Hkv;
  if (BH > 0x7fffffffLL) return TV_ERR_UNSUPPORTED;
  if (!encode_scored_map(&tmk, k, BH, S_cap, D, keys_of(lp.few)) ||
      !encode_scored_map(&tmv, v, BH, S_cap, D, keys_of(lp.few)))
    return record_cuda_error(cudaErrorInvalidValue);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return D == 64 ? launch_scored<64>(mode, tmk, tmv, p, lp, s) : launch_scored<128>(mode, tmk, tmv, p, lp, s);
}
