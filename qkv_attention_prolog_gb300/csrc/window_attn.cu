// Causal attention of prompts over their own keys, with a sliding window and sinks (16-bit q, k, v).
//
//   S = Q K^T,  P = 2^(S * scale * log2(e) - m),  O = P V,  l = sum P;  out = O / l
//
// per 128-key tile with a running maximum m.  Bound by the tensor cores (4 * 128 operations a
// visible pair of a head) and next to them by the exponentials, one for each pair.  A CTA stays on
// its SM and takes one item after another: two tiles of 128 query rows against the same stream of
// key tiles, so that one tile's products run while the other's softmax does:
//
//   warp 0          loads an item's Q and its K and V tiles, two stages, by TMA
//   warp 1          issues the products (tcgen05): S_i = Q_i K^T, then O_i += P_i V
//   warp 2          works out the items ahead of the others (the divisions and searches of an item
//                   took each role 4000 cycles, as long as a step)
//   warps 4..7      softmax of tile 0, a thread a row; warps 8..11 of tile 1
//
// Tensor memory holds S_0, S_1 and O_0, O_1 (128 columns each); P overwrites the S it came from, in
// 16 bits, and is the second product's operand where it lies.  A tile's rows are (token, head of
// the group): 128 / G tokens of all G query heads that share a k/v head, so every key tile is read
// once for the group, short sequences fill rows, and the band of half-visible tiles is as narrow
// as the tokens are few.
//
// m lags: it is raised, and O rescaled by the row's own thread, only when a score is more than 2^8
// beyond it.  P is rounded to the type of V (the products take two operands of one type); l adds
// the unrounded fp32 values, and O is fp32.
//
// 8192 tokens of one k/v head, 128 items: 101 us a CTA each, 67 shared.
//
// A step takes 1.6 us where all of a tile is visible.  One prompt of 8192 tokens (32 heads on 8, bf16)
// 355 us in short loops, 378, 1.45 PFLOP/s, in long ones; in a window of 2048 178 and 189 us, 1.28; 16
// prompts of up to 1024 in a window of 256, 213 MB, 73 us: three steps an item, as long again for its
// start and its output.  What did
// not pay: two issuing warps (499 -> 540 us for 8192), a row's columns shared by two threads (377 ->
// 504: the products then run at half their rate), waits on several barriers by one warp's lanes at
// a time (384 -> 366 us one after another), the softmax loops unrolled (206 -> 184 us rolled, window
// 2048: the instructions did not fit their cache), the output by four warps of their own while the
// next item runs (128 registers for all: prompts 75 -> 80, 8192 tokens 353 -> 367 us).
//
// Rows behind the sequence's end in its last tile of V are set to zero before the product.  Where V
// holds infinities or NaN at positions that some rows of a tile see and others do not, 0 * inf
// spoils the others: items with a row whose weights are finite and whose result is not are marked,
// and the CTA goes through them once more, with care: what is not finite is cleared from the tiles of
// V before the products, and comes to the rows that see it at the end (8192 tokens: 360 us, with one
// NaN in V 1120, V all NaN 1380; rows worked out again key by key took 299 ms).  A row that sees
// a NaN in K has no finite weights, and stays as it is.
#include "attn_tile.cuh"

namespace mlap {

namespace {

constexpr int kThreads = 384;
constexpr int kPlans = 4;                  // items worked out ahead
constexpr int kReaders = 10;               // warps that read a plan
constexpr int kStage = 32 * 128;           // a softmax warp's rows, half of their columns in 16 bits
constexpr int kMarks = 256;                // items whose marks are kept (the others share them)
// Key tiles of an item that some of its rows do not see whole: the 255 positions behind its first row,
// and as many in front of the windows, with up to seven columns behind the sinks, in tiles of 128.
constexpr int kPartly = 8;

// Items to go through with care, and what such an item's tiles of V held that is not finite, each word
// or byte by one of tile 0's softmax warps.
struct Care {
  uint64_t noted, read;                    // by these warps; by all eight
  uint32_t marks[2 * kMarks / 32];         // of items' tiles
  uint32_t marked;                         // any
  int32_t column[kPartly];                 // where the tiles begin that some rows do not see whole
  uint32_t keys[kPartly][kTile / 32];      // their keys with values that are not finite
  uint8_t kinds[4][3][kHeadDim / 8];       // channels with infinities, negative ones, NaN in the others
};
constexpr int kSmemBytes = (2 + 2 * kStages) * kOperand + 8 * kStage + 1024 + 256 + kPlans * 64 +
                           static_cast<int>(sizeof(Care)) + (kCountedSeqs + 1) * 4;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");

struct Bars {
  uint64_t q_full, q_empty, k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t s_full[2], p_full[2][2], o_done[2], drain, plan_full[kPlans], plan_empty[kPlans];
  uint64_t parted[2];                      // the softmax warps of a tile among themselves
  uint32_t tmem;
  int abort;
  int last[2];                             // the tile's other parts are all there
};
static_assert(sizeof(Bars) <= 256, "barriers");

struct __align__(16) Plan {
  int64_t row0;
  int32_t len, hk;
  int32_t tok0, tiles, steps, valid;       // tiles 0: no further item; valid: columns of the last step
  int32_t sink_end, sink_cols, shift, from;          // from: the first of the item's steps
  TilePart part;                           // (with care the item is whole; first: bits of marked tiles)
};
static_assert(sizeof(Plan) == 64, "four 16-byte reads");

struct Smem {
  uint8_t *q, *k, *v;                      // two Q tiles, the stages of K and V
  Bars* bar;
  Plan* plans;
  uint8_t* staged;
  Care* care;
  int* first;
};
__device__ __forceinline__ Smem smem_of(uint8_t* raw) {
  const uint32_t at = smem_u32(raw);
  Smem s;
  s.q = raw + (((at + 1023u) & ~1023u) - at);
  s.k = s.q + 2 * kOperand;
  s.v = s.k + kStages * kOperand;
  s.bar = reinterpret_cast<Bars*>(s.v + kStages * kOperand);
  s.plans = reinterpret_cast<Plan*>(s.v + kStages * kOperand + 256);
  s.staged = reinterpret_cast<uint8_t*>(s.plans + kPlans);
  s.care = reinterpret_cast<Care*>(s.staged + 8 * kStage);
  s.first = reinterpret_cast<int*>(s.care + 1);
  return s;
}

// What a CTA takes of the items.  Whole ones, a round of one for each CTA at a time, there and back;
// fewer items than CTAs are shared by key tiles where that pays, and what is left after whole rounds
// where a window keeps the items alike (16384 tokens of one k/v head, window 4096: 110 us, shared 100).
// Without one the rounds' long items even out with the short ones left (8192 tokens of two k/v heads
// 106 us, shared 132).
struct Items {
  int items, whole, shared;                // rounds of whole ones; what is left
  bool counted, split;
  int share, lo, hi, t_lo, place;          // the stretch; its first item and where it begins
};

__device__ __forceinline__ Block block_at(const AttnParams& p, const Smem& sm, bool counted, int tpt, int at,
                                          int* hk, SeqRows* s) {      // of item `at`; no tiles: there is none
  *hk = at % p.Nk;
  const int block = at / p.Nk;
  const int b = counted ? seq_of_block(sm.first, p.rag.B, block) : block % p.rag.B;
  const int index = counted ? block - sm.first[b] : block / p.rag.B;
  *s = seq_rows(p.rag, b);
  return index < blocks_of(*s, tpt) ? block_of(p, *s, index, tpt, 0x7fffffff, 1, 8) : Block{};
}

// All threads of the CTA.
__device__ __forceinline__ Items items_of(const AttnParams& p, const Smem& sm, int tpt, int most, bool may_split) {
  Items it;
  const int ctas = gridDim.x;
  it.counted = p.rag.B <= kCountedSeqs;
  it.items = it.counted ? sm.first[p.rag.B] * p.Nk : most;
  it.whole = it.items / ctas;
  it.shared = it.items - it.whole * ctas;
  it.split = false;
  it.share = 1;
  it.lo = it.hi = it.t_lo = it.place = 0;
  const bool even = p.window > 0 && 4 * static_cast<int64_t>(p.window) <= p.rag.max_new;
  if (may_split && (it.whole == 0 || even) && it.shared > 0) {
    int* line = reinterpret_cast<int*>(sm.staged);        // (for the moment)
    int hk;
    SeqRows s;
    Block k{};
    if (static_cast<int>(threadIdx.x) < it.shared) {
      k = block_at(p, sm, it.counted, tpt, it.whole * ctas + threadIdx.x, &hk, &s);
      line[threadIdx.x + 1] = k.tiles > 0 ? k.steps + kGap : 0;
    }
    if (threadIdx.x == 0) line[0] = sm.bar->last[0] = 0;
    __syncthreads();
    if (k.steps > 0) atomicMax(&sm.bar->last[0], k.steps);
    if (threadIdx.x >> 5 == 2) sum_line(line, it.shared);
    __syncthreads();
    const int total = line[it.shared];
    it.share = stretch_of(total, sm.bar->last[0], ctas, &it.split);
    if (static_cast<int>(blockIdx.x) * it.share < total) {
      it.lo = blockIdx.x * it.share;
      it.hi = min(it.lo + it.share, total);
      it.t_lo = seq_of_block(line, it.shared, it.lo);
      it.place = line[it.t_lo];
    }
    __syncthreads();
  }
  return it;
}

// w * f + acc for two 16-bit values.
template <bool BF16>
__device__ __forceinline__ uint32_t fma_16x2(uint32_t w, uint32_t f, uint32_t acc) {
  uint32_t d;
  if constexpr (BF16) {
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(w), "r"(f), "r"(acc));
  } else {
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(w), "r"(f), "r"(acc));
  }
  return d;
}

struct Maps {
  const CUtensorMap *q, *k, *v, *k8, *v8;
};

// What a role has counted: plans, Q tiles, steps, steps of its own tile.
struct Past {
  int plans, items, steps, own;
};

// Whether every row at positions pos_lo .. pos_hi of a block sees the whole tile from column u on.
__device__ __forceinline__ bool seen_by_all(const AttnParams& p, const Block& k, int pos_lo, int pos_hi, int u) {
  const Seen seen(p, k, pos_lo, pos_hi);
  const bool sinks = k.sink_cols > 0 ? u + kTile <= k.sink_end : u + kTile <= p.sinks && u + kTile - 1 <= seen.to;
  return sinks || seen.all(u, kTile);
}

// Clears what is not finite from 32 rows of a tile of V.  Returns a word of the rows that held any, and
// adds their kinds to the lane's channels 8 (lane & 15) .. + 7: bytes of infinities, negative ones, NaN.
template <bool BF16>
__device__ __noinline__ uint32_t clear_rows(uint8_t* rows, uint32_t* kinds, int lane) {
  constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
  uint8_t* at = rows + ((lane >> 3) & 1) * kHalf + (lane >> 4) * 128;
  uint32_t found = 0u;
#pragma unroll 1
  for (int k0 = 0; k0 < 16; k0 += 4) {     // two rows at a time
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = 2 * (k0 + k);
      v[k] = *reinterpret_cast<const uint4*>(at + r * 128 + (((lane & 7) ^ ((r + (lane >> 4)) & 7)) << 4));
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = 2 * (k0 + k);
      uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w}, odd[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) odd[i] = __vcmpeq2(w[i] & (kExp * 0x10001u), kExp * 0x10001u);
      const bool any = (odd[0] | odd[1] | odd[2] | odd[3]) != 0u;
      const uint32_t lanes = __ballot_sync(0xffffffffu, any);
      found |= (lanes & 0xffffu ? 1u << r : 0u) | (lanes >> 16 ? 2u << r : 0u);
      if (!any) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t nan = odd[i] & ~__vcmpeq2(w[i] & 0x7fff7fffu, kExp * 0x10001u);
        const uint32_t neg = w[i] >> 15 & 0x00010001u, is = odd[i] & 0x00010001u, n = nan & 0x00010001u;
        const uint32_t bits = (is & ~n & ~neg) | (is & ~n & neg) << 8;
        const uint32_t low = (bits & 0x101u) | (n << 16 & 0x10000u), high = bits >> 16 | (n & 0x10000u);
        *kinds |= low << (2 * i) | high << (2 * i + 1);
        w[i] &= ~odd[i];
      }
      *reinterpret_cast<uint4*>(at + r * 128 + (((lane & 7) ^ ((r + (lane >> 4)) & 7)) << 4)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  fence_proxy_async_shared();
  return found;
}

// Brings what clear_rows found in an item to a row's O in tensor memory (at `to`).  A warp's 32 rows;
// row: whether the lane has one, at position pos; partly: tiles that some rows do not see whole.
template <bool BF16>
__device__ __noinline__ void add_cleared(const AttnParams& p, const Block& blk, const Care* care, int partly,
                                         const void* v_head, bool row, int pos, uint32_t to) {
  using H = Half16<BF16>;
#pragma unroll 1
  for (int q = 0; q < 8; ++q) {            // 16 channels at a time
    uint32_t raw[16];
    float o[16];
    tmem_ld_32x32b_x16(to + q * 16, raw);
    tmem_ld_wait();
    uint32_t kind[3] = {0u, 0u, 0u};
#pragma unroll
    for (int k = 0; k < 12; ++k) kind[k % 3] |= reinterpret_cast<const uint16_t*>(care->kinds[k / 3][k % 3])[q];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      o[e] = __uint_as_float(raw[e]);
      if ((kind[0] >> e) & 1u) o[e] += INFINITY;
      if ((kind[1] >> e) & 1u) o[e] -= INFINITY;
      if ((kind[2] >> e) & 1u) o[e] = NAN;
    }
    // Values that the row sees, so small that finite ones never add up to an infinity: four keys at a
    // time, which a warp's rows look at together, until nothing but NaN is left.
    constexpr uint32_t kSmall = BF16 ? 0x0d800d80u : 0x04000400u, kInf = BF16 ? 0x7f807f80u : 0x7c007c00u;
    uint32_t sum[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    bool closed = false;
    for (int d = 0; d < partly && !closed; ++d) {
      for (int w = 0; w < kTile / 32 && !closed; ++w) {
        const int u = care->column[d] + 32 * w;
        const uint32_t mine = row ? care->keys[d][w] & sees(p, blk, pos, u) : 0u;
        for (uint32_t rest = __reduce_or_sync(0xffffffffu, mine); rest != 0u && !closed;) {
          uint4 x[4][2];
          uint32_t bit[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            bit[k] = rest & (0u - rest);
            rest ^= bit[k];
            if (bit[k] == 0u) continue;
            const int64_t key = key_of(blk, u + __ffs(bit[k]) - 1);
            const uint4* at = reinterpret_cast<const uint4*>(
                static_cast<const typename H::T*>(v_head) + key * p.Nk * kHeadDim) + 2 * q;
            x[k][0] = at[0];
            x[k][1] = at[1];
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if ((mine & bit[k]) == 0u) continue;
            const uint32_t v[8] = {x[k][0].x, x[k][0].y, x[k][0].z, x[k][0].w,
                                   x[k][1].x, x[k][1].y, x[k][1].z, x[k][1].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] = fma_16x2<BF16>(v[e], kSmall, sum[e]);
          }
          uint32_t nan = ~0u;
#pragma unroll
          for (int e = 0; e < 8; ++e) nan &= __vcmpgtu2(sum[e] & 0x7fff7fffu, kInf);
          closed = __all_sync(0xffffffffu, !row || nan == ~0u);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float f = H::to_f(reinterpret_cast<const typename H::T*>(sum)[e]);
      if (!(fabsf(f) < INFINITY)) o[e] += f;
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 16; ++e) raw[e] = __float_as_uint(o[e]);
    tmem_st_32x32b_x16(to + q * 16, raw);
  }
  tmem_st_wait();
}

// The CTA's items, or (CARE) the marked ones of them once more, whole whatever their parts were.  The
// pipelines run on from one walk to the next.
template <bool BF16, bool CARE>
__device__ __forceinline__ Past walk(const Maps& maps, const AttnParams& p, const Smem& sm, const Items& it, int tpt,
                                     float* slots, uint32_t* arrived, Past past) {
  using H = Half16<BF16>;
  Bars* bar = sm.bar;
  Care* care = sm.care;
  uint8_t *sq = sm.q, *sk = sm.k, *sv = sm.v;
  volatile int* abort_flag = &bar->abort;
  // (the shuffle tells the compiler that the warp's index is the same for all its lanes)
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int group = p.Nq / p.Nk;
  const uint32_t tmem = uniform(bar->tmem);

  // The n-th item of this CTA; null: there is none, or a wait gave up.  Every role walks the items
  // alike; the pipelines run on from one to the next.  Each reads what it needs and hands the plan
  // back: what is done once per item is code that the caches have dropped since the last one.
  auto take = [&](int n) -> const Plan* {
    if (!warp_wait(&bar->plan_full[n % kPlans], (n / kPlans) & 1, abort_flag)) return nullptr;
    const Plan* at = &sm.plans[n % kPlans];
    return uniform(at->tiles) > 0 ? at : nullptr;
  };
  auto give_back = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar->plan_empty[n % kPlans]);
  };

  if (warp == 2) {
    // -------------------------------------------------------------------- items
    int n = past.plans;
    auto put = [&](const Plan& plan) {
      if (!warp_wait(&bar->plan_empty[n % kPlans], ((n / kPlans) & 1) ^ 1, abort_flag)) return false;
      if (lane == 0) {
        sm.plans[n % kPlans] = plan;
        mbar_arrive(&bar->plan_full[n % kPlans]);
      }
      ++n;
      return true;
    };
    bool ok = true;
    const int rounds = it.whole + (it.shared > 0 && !it.split), ctas = gridDim.x;
    int next = it.t_lo, place = it.place, number = 0;
    for (int r = 0; ok; ++r) {
      const bool part = r >= rounds;
      if (part && (!it.split || place >= it.hi)) break;
      const int at = part ? it.whole * ctas + next++ : dealt(r);
      if (at >= it.items) continue;
      Plan plan{};
      SeqRows s;
      const Block k = block_at(p, sm, it.counted, tpt, at, &plan.hk, &s);
      if (k.tiles == 0) continue;
      plan.row0 = s.row0;
      plan.len = s.len;
      plan.tok0 = k.tok0;
      plan.tiles = k.tiles;
      plan.steps = k.steps;
      plan.valid = s.len - k.shift - (k.steps - 1) * kTile;
      plan.sink_end = k.sink_end;
      plan.sink_cols = k.sink_cols;
      plan.shift = k.shift;
      plan.part.parts = 1;
      if (part) {
        const int a0 = place + kGap, from = max(it.lo - a0, 0), to = min(it.hi - a0, k.steps);
        place = a0 + k.steps;
        if (to - from <= 0) continue;      // nothing but empty places
        if (!CARE) {
          plan.from = from;
          plan.steps = to - from;
          if (to < k.steps) plan.valid = kTile;
          plan.part = part_of(a0, k.steps, it.share, static_cast<int>(blockIdx.x));
        }
      }
      if (CARE) {                          // tiles that this CTA wrote and marked
        const int mark = number++ % kMarks;
        plan.part.first = (care->marks[mark >> 4] >> (2 * (mark & 15))) & 3u;
        if (plan.part.first == 0) continue;
      }
      ok = put(plan);
    }
    if (ok) put(Plan{});                   // the end
    past.plans = n;
  } else if (warp == 0) {
    // -------------------------------------------------------------------- loads
    int n = past.plans, nq = past.items, nk = past.steps, nv = nk;       // tiles requested so far
    bool ok = true;
    for (; ok; ++n) {
      const Plan* at = take(n);
      if (at == nullptr) break;
      const Plan plan = *at;
      give_back(n);
      Block blk;
      blk.sink_cols = plan.sink_cols;
      blk.shift = plan.shift;
      const int row0 = static_cast<int>(plan.row0), hk = plan.hk;
      ok = warp_wait(&bar->q_empty, (nq & 1) ^ 1, abort_flag);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bar->q_full, plan.tiles * 2 * group * tpt * 128);
        for (int i = 0; i < plan.tiles; ++i)
          for (int h = 0; h < 2; ++h)
            tma_load_3d(sq + i * kOperand + h * kHalf, maps.q, &bar->q_full, h * 64, hk * group,
                        row0 + plan.tok0 + i * tpt);
      }
      ++nq;
      for (int j = 0; j < plan.steps; ++j) {
        const int st = nk % kStages;
        const uint32_t ph = ((nk / kStages) & 1) ^ 1;
        const int u = (plan.from + j) * kTile, z = row0 + key_of(blk, u);
        // a tile with sinks and keys of the window comes eight rows at a time
        const bool mixed = u < blk.sink_cols && u + kTile > blk.sink_cols;
        auto load = [&](uint8_t* dst, const CUtensorMap* whole, const CUtensorMap* eight,
                        uint64_t* full) {
          mbar_arrive_expect_tx(full, kOperand);
          for (int h = 0; h < 2; ++h) {
            if (!mixed) {
              tma_load_3d(dst + h * kHalf, whole, full, h * 64, hk, z);
              continue;
            }
            for (int r = 0; r < kTile; r += 8)
              tma_load_3d(dst + h * kHalf + r * 128, eight, full, h * 64, hk, row0 + key_of(blk, u + r));
          }
        };
        ok = warp_wait(&bar->k_empty[st], ph, abort_flag);
        if (!ok) break;
        if (lane == 0) load(sk + st * kOperand, maps.k, maps.k8, &bar->k_full[st]);
        ++nk;
        ok = warp_wait(&bar->v_empty[st], ph, abort_flag);
        if (!ok) break;
        if (lane == 0) load(sv + st * kOperand, maps.v, maps.v8, &bar->v_full[st]);
        ++nv;
      }
    }
    give_back(n);                          // (the end)
    past = Past{n + 1, nq, nv, 0};
    if (*abort_flag && lane == 0) {
      // give up cleanly: what was requested lands before the CTA exits (bounded)
      const uint64_t t0 = globaltimer_ns();
      auto landed = [&](uint64_t* full, uint32_t parity) {
        while (!mbar_try_wait(full, parity) && globaltimer_ns() - t0 < 20000000ull) {
        }
      };
      if (nq > 0) landed(&bar->q_full, (nq - 1) & 1);
      for (int i = nk > kStages ? nk - kStages : 0; i < nk; ++i)
        landed(&bar->k_full[i % kStages], (i / kStages) & 1);
      for (int i = nv > kStages ? nv - kStages : 0; i < nv; ++i)
        landed(&bar->v_full[i % kStages], (i / kStages) & 1);
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------------- products
    const uint32_t base = BF16 ? idesc_bf16_f32(kTile, kTile) : idesc_f16_f32(kTile, kTile);
    const uint32_t id_s = base | (p.scale_log2 < 0.f ? kIdescNegateA : 0u);
    const uint32_t id_o = base | kIdescNMajorB;
    // descriptors differ in the start address alone, in units of 16 bytes
    const uint64_t dq = sdesc_kmajor_sw128(smem_u32(sq));
    const uint64_t dk = sdesc_kmajor_sw128(smem_u32(sk));
    const uint64_t dv = sdesc_nmajor_sw128(smem_u32(sv), kHalf);
    auto scores = [&](int i, int st) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_bf16_ss(tmem + i * kTile, dq + i * (kOperand / 16) + (h * kHalf + k * 32) / 16,
                       dk + st * (kOperand / 16) + (h * kHalf + k * 32) / 16, id_s,
                       (h | k) ? 1u : 0u);
      umma_commit(&bar->s_full[i]);
    };
    int n = past.plans, nq = past.items, at = past.steps;      // items and steps so far
    int done0 = at, done1 = past.own;      // steps of either tile
    bool ok = true;
    for (; ok; ++n) {
      const Plan* plan = take(n);
      if (plan == nullptr) break;
      // (known to be the same for all lanes: the loop and the descriptors stay in uniform registers)
      const bool two = uniform(plan->tiles) == 2;
      const int steps = uniform(plan->steps), valid = uniform(plan->valid);
      give_back(n);
      ok = warp_wait(lane == 0 ? &bar->q_full : &bar->k_full[at % kStages],
                     lane == 0 ? nq & 1 : (at / kStages) & 1, abort_flag);
      if (!ok) break;
      ++nq;
      tc_fence_after_sync();
      if (elect_one()) {
        scores(0, at % kStages);
        if (two) scores(1, at % kStages);
        umma_commit(&bar->k_empty[at % kStages]);
        if (steps == 1) umma_commit(&bar->q_empty);
      }
      for (int j = 0; ok && j < steps; ++j, ++at) {
        const int st = at % kStages, nx = (at + 1) % kStages;
        const bool more = j + 1 < steps;
        ok = warp_wait(&bar->v_full[st], (at / kStages) & 1, abort_flag);
        if (more) ok = ok && warp_wait(&bar->k_full[nx], ((at + 1) / kStages) & 1, abort_flag);
        ok = ok && warp_wait(&bar->p_full[0][0], done0 & 1, abort_flag);
        if (!ok) break;
        ++done0;
        if (!more && valid < kTile) {      // the sequence ends inside this tile
          for (int e = valid * 16 + lane; e < kTile * 16; e += 32)
            *reinterpret_cast<uint4*>(sv + st * kOperand + ((e >> 3) & 1) * kHalf + (e >> 4) * 128 +
                                      (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_shared();
          __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i == 1) {
            if (!two) break;
            ok = warp_wait(&bar->p_full[1][0], done1 & 1, abort_flag);
            if (!ok) break;
            ++done1;
          }
          tc_fence_after_sync();
          auto values = [&](int k0) {
#pragma unroll
            for (int k = k0; k < k0 + 4; ++k)
              umma_f16_ts(tmem + 2 * kTile + i * kTile, tmem + i * kTile + k * 8,
                          dv + st * (kOperand / 16) + k * (2048 / 16), id_o, (j | k) ? 1u : 0u);
          };
          if (elect_one()) values(0);
          // (P comes in two halves of 64 keys, the second while the first one's products run)
          ok = warp_wait(&bar->p_full[i][1], (i == 0 ? done0 - 1 : done1 - 1) & 1, abort_flag);
          if (!ok) break;
          tc_fence_after_sync();
          if (elect_one()) {
            values(4);
            umma_commit(&bar->o_done[i]);
            if (i == 1 || !two) umma_commit(&bar->v_empty[st]);
            if (more) {
              scores(i, nx);
              if (i == 1 || !two) {
                umma_commit(&bar->k_empty[nx]);
                if (j + 2 == steps) umma_commit(&bar->q_empty);   // the item's last scores
              }
            }
          }
        }
      }
    }
    give_back(n);                          // (the end)
    past = Past{n + 1, nq, at, done1};
    if (*abort_flag && lane == 0) {        // the products issued so far end before the CTA does
      umma_commit(&bar->drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(&bar->drain, 0) && globaltimer_ns() - t0 < 20000000ull) {
      }
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------------- softmax, a thread a row
    const int i = (warp >> 2) - 1;
    const int row = threadIdx.x & (kTile - 1);
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;     // this warp's 32 lanes
    const uint32_t ts = tmem + i * kTile + lanes, to = tmem + (2 + i) * kTile + lanes;
    const float c = fmaxf(fabsf(p.scale_log2), 1.17549435e-38f);    // (positive for a scale of 0)
    const int row_tok = row / group, row_head = row - row_tok * group;
    // tokens of this warp's rows, behind the tile's first
    const int warp_lo = (warp & 3) * 32 / group, warp_hi = ((warp & 3) * 32 + 31) / group;
    int n = past.plans, done = past.own;   // steps of this tile so far
    int cared = 0;                         // items whose tiles were cleared
    bool ok = true;
    for (; ok; ++n) {
      const Plan* at = take(n);
      if (at == nullptr) break;
      const Plan plan = *at;
      give_back(n);
      if (plan.tiles <= i) {
        if (CARE) {                        // (no warp runs ahead of what has been noted)
          ok = warp_wait(&care->noted, cared++ & 1, abort_flag);
          if (lane == 0) mbar_arrive(&care->read);
        }
        continue;
      }
      Block blk;
      blk.sink_end = plan.sink_end;
      blk.sink_cols = plan.sink_cols;
      blk.shift = plan.shift;
      const int tile_tok = plan.tok0 + i * tpt;
      const int tok = tile_tok + row_tok;
      const int tok_lo = tile_tok + warp_lo, tok_hi = tile_tok + warp_hi;
      const Seen seen(p, blk, tok_lo, tok_hi);
      // (rows of no token hold what is left in shared memory: they never raise m, which is their warp's
      // decision for all of its rows)
      float m = row < group * tpt && tok < plan.len ? -INFINITY : INFINITY, l = 0.f;
      int partly = 0;                      // tiles that some of the item's rows do not see whole
      uint32_t kinds = 0u;
      if (CARE && i == 0 && cared > 0) {   // (what was noted of the last item has been read)
        ok = warp_wait(&care->read, (cared - 1) & 1, abort_flag);
        if (!ok) break;
      }
      for (int j = 0; j < plan.steps; ++j, ++done) {
        ok = warp_wait(&bar->s_full[i], done & 1, abort_flag);
        if (!ok) break;
        tc_fence_after_sync();
        const int u = (plan.from + j) * kTile;
        const bool all = seen.all(u, kTile);
        if (CARE) {                        // tile 0's warps clear V before its first product
          const bool whole = seen_by_all(p, blk, plan.tok0, plan.tok0 + plan.tiles * tpt - 1, u);
          if (i == 0) {
            ok = warp_wait(&bar->v_full[done % kStages], (done / kStages) & 1, abort_flag);
            if (!ok) break;
            uint32_t rest = 0u;
            uint8_t* rows = sv + (done % kStages) * kOperand + (warp & 3) * 32 * 128;
            const uint32_t found = clear_rows<BF16>(rows, whole ? &kinds : &rest, lane);
            if (!whole && lane == 0) {
              care->column[min(partly, kPartly - 1)] = u;
              care->keys[min(partly, kPartly - 1)][warp & 3] = found;
            }
            if (j + 1 == plan.steps) {
              const uint32_t k = kinds | __shfl_xor_sync(0xffffffffu, kinds, 16);
              if (lane < 16)
                for (int e = 0; e < 3; ++e) care->kinds[warp & 3][e][lane] = static_cast<uint8_t>(k >> (8 * e));
              __syncwarp();
              if (lane == 0) mbar_arrive(&care->noted);
            }
          }
          if (!whole) ++partly;
        }
        float top = -INFINITY;
#pragma unroll 1
        for (int q = 0; q < kTile; q += 64) {          // 64 columns at a time
          uint32_t s[2][32];
          tmem_ld_32x32b_x32(ts + q, s[0]);
          tmem_ld_32x32b_x32(ts + q + 32, s[1]);
          tmem_ld_wait();
          if (!all) {
            // some of the warp's rows do not see all of the tile: their columns go back as -inf
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              if (seen.all(u + q + k * 32, 32)) continue;
              const uint32_t see = sees(p, blk, tok, u + q + k * 32);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(see & (1u << e))) s[k][e] = __float_as_uint(-INFINITY);
              tmem_st_32x32b_x32(ts + q + k * 32, s[k]);
            }
          }
          float mx[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t* x = &s[k >> 1][(k & 1) * 16];
            mx[k] = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
#pragma unroll
            for (int e = 2; e < 16; e += 2)
              mx[k] = max3(mx[k], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
          }
          top = max3(top, fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        }
        if (!all) tmem_st_wait();
        top *= c;                          // (-inf stays: c > 0)
        if (__any_sync(0xffffffffu, top > m + kLag)) {
          const float mn = fmaxf(m, top);
          const float f = mn == -INFINITY ? 1.f : exp2_approx(m - mn);
          m = mn;
          l *= f;
          if (j > 0) {
            ok = warp_wait(&bar->o_done[i], (done - 1) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after_sync();
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              uint32_t o[16];
              tmem_ld_32x32b_x16(to + q * 16, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st_32x32b_x16(to + q * 16, o);
            }
          }
        }
        const float neg = m == -INFINITY ? 0.f : -m;
        const float2 c2 = make_float2(c, c), neg2 = make_float2(neg, neg);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
        for (int q = 0; q < kTile; q += 64) {
          uint32_t s[2][32];
          tmem_ld_32x32b_x32(ts + q, s[0]);
          tmem_ld_32x32b_x32(ts + q + 32, s[1]);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float2 x = make_float2(__uint_as_float(s[k][2 * e]), __uint_as_float(s[k][2 * e + 1]));
              x = fma_x2(x, c2, neg2);
              x.x = exp2_approx(x.x);
              x.y = exp2_approx(x.y);
              sum[k] = add_x2(sum[k], x);
              pk[e] = H::pack(x.x, x.y);
            }
            tmem_st_32x32b_x16(ts + (q >> 1) + k * 16, pk);
          }
          tmem_st_wait();
          tc_fence_before_sync();
          mbar_arrive(&bar->p_full[i][q >> 6]);
        }
        const float2 s2 = add_x2(sum[0], sum[1]);
        l += s2.x + s2.y;
      }
      // ---- out = O / l, through shared memory: a row's 256 bytes lie in one thread, and stores of
      // single rows kept the memory pipeline, and with it the next item's first step, for 4000
      // cycles
      if (!ok || !warp_wait(&bar->o_done[i], (done - 1) & 1, abort_flag)) break;
      tc_fence_after_sync();
      if (!CARE && plan.part.parts > 1) {
        // the part goes to the workspace; the last one's warps bring the sum of all back to O
        auto slot = [&](int k) {
          return slots + (static_cast<int64_t>(plan.part.slot(k)) * 2 + i) * kTilePartFloats;
        };
        float4* to_o = reinterpret_cast<float4*>(slot(plan.part.part)) + row;
#pragma unroll 1
        for (int q = 0; q < 8; ++q) {
          uint32_t o[16];
          tmem_ld_32x32b_x16(to + q * 16, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 4; ++e)
            __stcg(to_o + (q * 4 + e) * kTile,
                   make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                               __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3])));
        }
        __stcg(reinterpret_cast<float2*>(slot(plan.part.part) + kTile * kHeadDim) + row, make_float2(m, l));
        mbar_arrive(&bar->parted[i]);
        ok = warp_wait(&bar->parted[i], 0, abort_flag);
        if (!ok) break;
        if (row == 0) bar->last[i] = last_part(arrived, plan.part, i);
        mbar_arrive(&bar->parted[i]);
        ok = warp_wait(&bar->parted[i], 1, abort_flag);
        if (!ok) break;
        if (bar->last[i] == 0) {
          tc_fence_before_sync();
          continue;
        }
        const int parts = plan.part.parts;
        auto ml = [&](int k) {
          return __ldcg(reinterpret_cast<const float2*>(slot(k) + kTile * kHeadDim) + row);
        };
        m = -INFINITY;
        l = 0.f;
#pragma unroll 4
        for (int k = 0; k < parts; ++k) m = fmaxf(m, ml(k).x);
#pragma unroll 4
        for (int k = 0; k < parts; ++k) {
          const float2 x = ml(k);
          l = fmaf(x.y, x.x == -INFINITY ? 0.f : exp2_approx(x.x - m), l);
        }
#pragma unroll 1
        for (int q = 0; q < 8; ++q) {
          float o[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0.f;
#pragma unroll 1
          for (int k0 = 0; k0 < parts; k0 += 4) {              // the loads of four parts at a time
            float mk[4];
            float4 v[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int kk = k0 + k < parts ? k0 + k : parts - 1;
              mk[k] = ml(kk).x;
              const float4* from = reinterpret_cast<const float4*>(slot(kk)) + q * 4 * kTile + row;
#pragma unroll
              for (int e = 0; e < 4; ++e) v[k][e] = __ldcg(from + e * kTile);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float down = mk[k] == -INFINITY || k0 + k >= parts ? 0.f : exp2_approx(mk[k] - m);
              if (down == 0.f) continue;   // (a part that the row saw nothing of, or none)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                o[4 * e] = fmaf(v[k][e].x, down, o[4 * e]);
                o[4 * e + 1] = fmaf(v[k][e].y, down, o[4 * e + 1]);
                o[4 * e + 2] = fmaf(v[k][e].z, down, o[4 * e + 2]);
                o[4 * e + 3] = fmaf(v[k][e].w, down, o[4 * e + 3]);
              }
            }
          }
          tmem_st_32x32b_x16(to + q * 16, reinterpret_cast<const uint32_t(&)[16]>(o));
        }
        tmem_st_wait();
      }
      if (CARE) {
        ok = warp_wait(&care->noted, cared++ & 1, abort_flag);
        if (!ok) break;
        add_cleared<BF16>(p, blk, care, min(partly, kPartly),
                          static_cast<const typename H::T*>(p.v) + (plan.row0 * p.Nk + plan.hk) * kHeadDim,
                          row < group * tpt && tok < plan.len, tok, to);
        if (lane == 0) mbar_arrive(&care->read);
      }
      const bool mine = row < group * tpt && tok < plan.len && (!CARE || (plan.part.first >> i) & 1);
      const int h = plan.hk * group + row_head;
      const float inv = 1.f / l;           // (a row sees itself at least)
      const int64_t at_out = mine ? ((plan.row0 + tok) * p.Nq + h) * kHeadDim : -1;
      int64_t to_out[8];                   // of the rows that this lane stores a piece of
#pragma unroll
      for (int k = 0; k < 8; ++k) to_out[k] = __shfl_sync(0xffffffffu, at_out, 4 * k + (lane >> 3));
      uint8_t* stage = sm.staged + (warp - 4) * kStage;
      const float2 inv2 = make_float2(inv, inv);
      uint32_t odd = 0u;                   // NaN if anything is not finite
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t o[2][32];
#pragma unroll
        for (int q = 0; q < 2; ++q) tmem_ld_32x32b_x32(to + half * 64 + q * 32, o[q]);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 8; ++k) {      // 8 columns: a 16-byte piece
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t* x = &o[k >> 2][(k & 3) * 8 + 2 * e];
            const float2 v = make_float2(__uint_as_float(x[0]), __uint_as_float(x[1]));
            const float2 y = mul_x2(v, inv2);
            w[e] = H::pack(y.x, y.y);
            odd = fma_16x2<BF16>(w[e], 0u, odd);
          }
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((k ^ (lane & 7)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = 4 * k + (lane >> 3), c8 = lane & 7;
          const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + ((c8 ^ (r & 7)) << 4));
          if (to_out[k] >= 0)
            *reinterpret_cast<uint4*>(static_cast<typename H::T*>(p.out) + to_out[k] + half * 64 +
                                      c8 * 8) = v;
        }
        __syncwarp();
      }
      tc_fence_before_sync();              // O is read before the next item's first P is announced
      if (!CARE) {
        const bool spoilt = mine && l < INFINITY && (odd & 0x7fff7fffu) != 0u;
        if (__any_sync(0xffffffffu, spoilt) && lane == 0) {
          const int mark = n % kMarks;
          atomicOr(&care->marks[mark >> 4], 1u << (2 * (mark & 15) + i));
          care->marked = 1u;
        }
      }
    }
    give_back(n);                          // (the end)
    past = Past{n + 1, 0, 0, done};
  }
  return past;
}

template <bool BF16>
__device__ __noinline__ void walk_again(const CUtensorMap* q, const CUtensorMap* k, const CUtensorMap* v,
                                        const CUtensorMap* k8, const CUtensorMap* v8, const AttnParams* at,
                                        uint8_t* smem_raw, int tpt, int most, bool may_split, Past past) {
  const Smem sm = smem_of(smem_raw);
  const AttnParams& p = *at;
  walk<BF16, true>(Maps{q, k, v, k8, v8}, p, sm, items_of(p, sm, tpt, most, may_split), tpt, nullptr, nullptr,
                   past);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    window_attn_kernel(const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ CUtensorMap tmK8,
                       const __grid_constant__ CUtensorMap tmV8, const __grid_constant__ AttnParams p, int tpt,
                       int most, int may_split, float* slots, uint32_t* arrived) {
  using H = Half16<BF16>;
  extern __shared__ uint8_t smem_raw[];
  const Smem sm = smem_of(smem_raw);
  Bars* bar = sm.bar;
  volatile int* abort_flag = &bar->abort;
  // (the shuffle tells the compiler that the warp's index is the same for all its lanes)
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    mbar_init(&bar->q_full, 1);
    mbar_init(&bar->q_empty, 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar->k_full[i], 1);
      mbar_init(&bar->k_empty[i], 1);
      mbar_init(&bar->v_full[i], 1);
      mbar_init(&bar->v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->s_full[i], 1);
      mbar_init(&bar->p_full[i][0], kTile);
      mbar_init(&bar->p_full[i][1], kTile);
      mbar_init(&bar->o_done[i], 1);
      mbar_init(&bar->parted[i], kTile);
    }
    mbar_init(&bar->drain, 1);
    for (int i = 0; i < kPlans; ++i) {
      mbar_init(&bar->plan_full[i], 1);
      mbar_init(&bar->plan_empty[i], kReaders);
    }
    mbar_init(&sm.care->noted, 4);
    mbar_init(&sm.care->read, 8);
    sm.care->marked = 0u;
    bar->abort = 0;
    fence_mbarrier_init();
  }
  if (warp == 3)
    for (int i = lane; i < 2 * kMarks / 32; i += 32) sm.care->marks[i] = 0u;
  if (warp == 1) {
    tmem_alloc(&bar->tmem, 512);
    tmem_relinquish();
  }
  grid_dependency_wait();
  if (p.rag.B <= kCountedSeqs) count_blocks(p.rag, tpt, sm.first);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.rag.B; i += kThreads)
      if (seq_rows(p.rag, i).bad) atomicOr(p.err, kErrIndexRange);

  const Past past = walk<BF16, false>(Maps{&tmQ, &tmK, &tmV, &tmK8, &tmV8}, p, sm,
                                      items_of(p, sm, tpt, most, may_split), tpt, slots, arrived, Past{});
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (sm.care->marked != 0u && *abort_flag == 0) {
    walk_again<BF16>(&tmQ, &tmK, &tmV, &tmK8, &tmV8, &p, smem_raw, tpt, most, may_split, past);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
  }
  if (warp == 1) tmem_dealloc(bar->tmem, 512);
  if (threadIdx.x == 0 && *abort_flag) atomicOr(p.err, kErrTimeout);
}

}  // namespace

// Where items may be longer than a split costs, and there may be fewer of them than CTAs.
bool window_splits(const AttnParams& p) {
  const int64_t tpt = window_attn_tokens(p.Nq / p.Nk), blocks = (p.rag.max_new + 2 * tpt - 1) / (2 * tpt);
  int64_t keys = p.rag.max_new;
  if (p.window > 0 && p.window + 2 * tpt + p.sinks < keys) keys = p.window + 2 * tpt + p.sinks;
  return keys > (kSplitCost - kGap + kMinShare) * kTile && blocks * p.Nk * p.rag.B < 4 * kSplitCtas;
}

cudaError_t launch_window_attn(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                               const CUtensorMap& k8, const CUtensorMap& v8, const AttnParams& p,
                               uint32_t* header, void* ws, cudaStream_t stream, int sm_count) {
  const int tpt = window_attn_tokens(p.Nq / p.Nk);
  const int64_t per_seq = (p.rag.max_new + 2 * tpt - 1) / (2 * tpt);
  const int64_t items = per_seq * p.Nk * p.rag.B;
  if (items > 0x7fffffffLL - sm_count) return cudaErrorInvalidConfiguration;
  const bool split = window_splits(p);
  const int ctas = split && sm_count > kSplitCtas ? kSplitCtas : sm_count;
  auto kern = p.bf16 ? window_attn_kernel<true> : window_attn_kernel<false>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items < ctas && !split ? items : ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, q, k, v, k8, v8, p, tpt, static_cast<int>(items),
                            static_cast<int>(split), static_cast<float*>(ws), header + 1);
}

}  // namespace mlap
