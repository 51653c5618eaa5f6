// Attention of a few query rows per sequence over the paged 8-bit cache (decode and drafts).
//
//   x[t] = scale * log2(e) * ks * (q . kc[t]),   P[t] = 2^(x[t] + log2(vs) - m),
//   out  = (sum_t P[t] vc[t]) / (sum_t P[t] / vs)
//
// with kc, vc the int8 codes and ks, vs the scales of the token's page: one pass over the codes
// with a running maximum m.  The value scale goes into the exponent, so P stays in the range of
// the largest weighted value whatever the pages' scales are, and the sum of the weights takes it
// out again in fp32.
//
// What bounds it is the stream of codes, 256 bytes per token and k/v head, against 4 * rows * 128
// multiply-adds: the tensor cores' register path (mma.sync m16n8k16, 16-bit operands, fp32 sums) has
// the rate for 8 or 16 rows, and its operands come from registers, where int8 becomes 16 bits by a
// byte permute and one packed instruction, exactly: V's codes f16, K's the type of q, which enters the
// first product as it is (scaled into f16's range, bf16 rows lost bits to the largest one beside
// them).  Both products run transposed, S^T = K q^T and O^T = V^T P^T, so that the tokens and the
// channels fill the 16 rows of the instruction and the query rows its 8 columns: eight rows (one
// token of up to eight heads) cost half of what rows as the 16-row operand would, and P turns from
// the first product's layout to the second's by an 8x8 register transpose (movmatrix).  Each of a
// CTA's four warps streams its own pairs of 16-token steps (the largest run of tokens that a page
// is sure to hold whole) by TMA into a ring of two pairs, and joins the others at the end, so no
// barrier stands between the loads and the products.
//
// The work is a line of steps: sequence by sequence, row tile by row tile, head by head, in equal
// stretches for all CTAs (three on each SM), so ragged batches and single long sequences load all
// SMs alike.  Up to eight heads walk the line together, one CTA each: the 128-byte rows of a token's
// heads lie side by side, and read at one time they are one visit to their memory rows.  64
// sequences of up to 8192 tokens, 598 MB: 101 us so, 122 us with every head in its own place on the
// line.  A tile's start and join cost about as much as kTileGap steps; the line counts them in (98 us).
// Where there are stretches enough, each tile begins with one, and none has parts of two (one user
// over 131071 tokens 63 -> 58 us, over 600 tokens 13 -> 10).
//
// A segment that covers a tile's keys whole writes the output.  Otherwise the parts meet in a tree
// of eights: a part goes to the workspace, and whoever arrives last at a node joins its children,
// always in the order of the stretches, and goes on to the next level, so nobody waits and the
// result does not depend on who comes when.  A node's arrivals are counted in four bits of the
// workspace's header, which are zero again when the call ends.  The next segment's pages and first
// copies are requested before that.
//
// Measured: 64 sequences of up to 8192 tokens (32 heads on 8) 98 us, 6.1 TB/s (57 of 4608, where no
// tile is split, stream at 7.2 TB/s); one over 131071 tokens 53 us: the first product at 4.4, the
// median block's last one at 42, the last join at the end; one over 600 tokens 8.6, of which 2 lay
// out the line, 3 come before the first product and 2 are the join (a loop over the children that
// waited for each one's loads took 0.5 more).  Four drafted tokens of seven heads, 28
// rows, take two tiles of 16 and read the codes twice: 96 sequences within a window of 1024 take
// 43 us.  Nothing is full there: DRAM at a third of its rate, 42 % of the issue slots (about a thousand
// instructions for each pair of steps, a third of them int8 to 16 bits); a tile's start and join, over a
// quarter of the line, and the chain of a pair's two products are what is left.  What did not pay:
// tiles of 32 rows (255 registers, q's fragments in shared memory, two CTAs an SM): 16 x 8 tokens
// over 8000 100 -> 89 us, but those drafts 46 -> 59 and one sequence's 8 tokens over 1000 13 -> 18;
// more stretches than resident CTAs (131071 tokens 69 -> 108 us, all of it parts and joins); two
// CTAs an SM for 16-row tiles (4 tokens over 1024: 49 -> 55 us).
#include "attn_common.cuh"
#include "attn_ptx.cuh"
#include "attn_tile.cuh"

namespace mlap {

namespace {

constexpr int kWarps = 4;
constexpr int kStages = 4;                 // 16-token steps a warp keeps in flight (two pairs)
constexpr int kStepTokens = 16;
constexpr int kMaxRows = 16;               // query rows (token, head of the group) of a tile
constexpr int kStepBytes = kStepTokens * kHeadDim * 2;
constexpr int kWarpBytes = kStages * kStepBytes;
constexpr int kPitch = kHeadDim + 4;       // floats between rows while the warps join
// Steps of a stretch at least: a pair for each warp while eight parts of that hold every tile, else
// two (600 tokens 9.2 us and 10.1 with two; 2000, of which one pair each makes a tree of two levels,
// 11.4 and 10.3).
constexpr int kLeastShare = 8;
// What a tile costs beyond its steps, in steps (none, 12, 24, 40: 64 sequences of up to 8192 tokens
// 100.9, 99.4, 98.2, 98.8 us; 96 sequences' drafts in a window of 1024 50.3, 48.6, 46.5, 49.2).
constexpr int kTileGap = 24;
// A stretch grows up to this many steps where tiles can begin with one then (32 sequences of 500
// tokens: 14 us, 19 with the shares of the even line).
constexpr int kWholeShare = 64;
// P is held 2^kHead above its own scale and m may lag kLag behind the true maximum: the largest P
// is 2^(kHead + kLag), inside f16's range, and the smallest normal one 2^-(14 + kHead).
constexpr float kHead = 6.f, kLag = 8.f;

struct SeqWork {
  SeqRows s;
  int sink_steps, near_step;               // steps [0, sink_steps) and from near_step on
  int steps;                               // of both
  int tiles;                               // tiles of a head's rows
  bool beyond;                             // tokens past the block table
};

__device__ __forceinline__ SeqWork seq_work(const AttnParams& p, int b, int tile_rows) {
  SeqWork w;
  w.s = seq_rows(p.rag, b);
  const int g = p.Nq / p.Nk;
  w.tiles = (w.s.len * g + tile_rows - 1) / tile_rows;
  const int cap = p.pg.max_blocks * p.pg.block_size;
  int end = w.s.ctx + w.s.len;             // positions of the keys
  w.beyond = w.s.len > 0 && end > cap;
  if (end > cap) end = cap;
  const int last = (end + kStepTokens - 1) / kStepTokens;
  int near = 0;
  if (p.window > 0 && w.s.ctx >= p.window) near = w.s.ctx - p.window + 1;
  const int sink_end = p.sinks < near ? p.sinks : near;
  w.sink_steps = (sink_end + kStepTokens - 1) / kStepTokens;
  w.near_step = near / kStepTokens;
  if (w.near_step < w.sink_steps) w.near_step = w.sink_steps;
  if (w.sink_steps > last) w.sink_steps = last;
  const int n = last - w.near_step;
  w.steps = w.s.len > 0 ? w.sink_steps + (n > 0 ? n : 0) : 0;
  // rows of a sequence without keys are still to be written (zeros): one step that loads nothing
  if (w.s.len > 0 && w.steps == 0) w.steps = 1;
  return w;
}

// Divisions of the line's places: they fit 32 bits but on the longest lines.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b))
                              : a / b;
}

// The line of steps.  A tile takes kTileGap empty places of it (for its start and its join) and then one
// for each step, or, with whole set, as many as whole stretches hold (the last ones are empty then).
struct Line {
  int64_t total;
  int64_t share;                           // places of a stretch
  bool whole;
  int outer;                               // groups of heads, one after another on the line
  int groups;                              // stretches
};

__device__ __forceinline__ int64_t whole_places(int steps, int64_t share) {
  return quotient(steps + share - 1, share) * share;
}
__device__ __forceinline__ int64_t places_of(const Line& l, const SeqWork& w) {
  return l.whole ? whole_places(w.steps, l.share) : w.steps + kTileGap;
}
__device__ __forceinline__ int64_t work_of(const Line& l, const SeqWork& w) {
  return places_of(l, w) * w.tiles * l.outer;
}

// Workspace of the parts, for each of a group's heads: slot 2c for the part that opens stretch c,
// 2c + 1 for a later one.
struct Parts {
  float* out;                              // (slots, kMaxRows, 128), in units of 2^(m - kHead)
  float* ml;                               // (slots, kMaxRows, 2): m and the sum
  uint32_t* arrived;                       // four bits for each block
  int inner;                               // heads that walk the line together
  int outer;                               // groups of them
  FastDiv groups;                          // by the number of stretches
};

// Sum over the block of a value of each thread; *before: that of the threads before this one.
__device__ __forceinline__ int64_t block_scan(int64_t mine, int64_t* wsum, int64_t* before) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  int64_t total = 0;
  *before = inc - mine;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) *before += wsum[w];
    total += wsum[w];
  }
  return total;
}

// Lays out the line.  All threads of the block; *begin, *places: what of it are the sequences
// [t * per_thread, ...) of thread t, *w: the last of them.  Tiles begin with a stretch where there
// are stretches enough for that: then no block has parts of two tiles, whose starts and joins would
// come one after another.
__device__ __forceinline__ Line lay_line(const AttnParams& p, const Parts& parts, int tile_rows, int per_thread,
                                         bool report, int64_t* begin, int64_t* places, SeqWork* last) {
  __shared__ int64_t wsum[4][kWarps];
  const int b0 = threadIdx.x * per_thread;
  int64_t mine = 0, before;
  Line l;
  l.whole = false;
  l.outer = parts.outer;
  l.groups = static_cast<int>(gridDim.y);
  SeqWork w{};
  bool deep = false;
  for (int b = b0; b < b0 + per_thread && b < p.rag.B; ++b) {
    w = seq_work(p, b, tile_rows);
    mine += static_cast<int64_t>(w.steps + kTileGap) * w.tiles * l.outer;
    deep |= w.steps > 8 * kLeastShare;
    if (report && (w.s.bad || w.beyond)) atomicOr(p.err, kErrIndexRange);
  }
  l.total = block_scan(mine, wsum[0], &before);
  const int64_t up = l.total + l.groups - 1;
  l.share = up >> 32 == 0 ? static_cast<int64_t>(div_fast(static_cast<uint32_t>(up), parts.groups)) : up / l.groups;
  const int least = __syncthreads_or(deep) ? 2 * kLeastShare : kLeastShare;
  if (l.share < least) l.share = least;
  if (per_thread == 1) {
    int64_t share = l.share;
    for (int k = 1; k == 1 || (k < 4 && share <= kWholeShare); ++k, share *= 2) {
      int64_t before2;
      const int64_t m2 = whole_places(w.steps, share) * w.tiles * l.outer;
      const int64_t t2 = block_scan(m2, wsum[k], &before2);
      if (t2 <= share * l.groups) {
        l.whole = true;
        l.share = share;
        l.total = t2;
        before = before2;
        mine = m2;
        break;
      }
    }
  }
  *begin = before;
  *places = mine;
  *last = w;
  return l;
}

template <bool BF16>
__device__ __forceinline__ void mma_16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// 8x8 transpose over the warp: lane (g, c) gives row g, columns 2c and 2c + 1, and gets row g's of
// the transposed matrix.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// 16 tokens of one head of a page, swizzled by 128 bytes.
__device__ __forceinline__ void load_run(void* dst, const CUtensorMap* map, uint64_t* bar, int head,
                                         int row, int page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(head), "r"(row), "r"(page)
      : "memory");
}

// What a step's products need of its page, worked out once by one lane.
struct Meta {
  float f;                                 // ks * scale * log2(e)
  float lv;                                // log2 |vs|
  float inv;                               // 1 / |vs|
  float sign;                              // of vs; 0: vs counts as 0
  int t0;                                  // first token
  int page, row;                           // and where it lies; page -1: nothing of it is visible
  int pad;
};
constexpr int kBatch = 32;                 // steps whose page ids a warp holds, one a lane
constexpr int kMetaBytes = 2 * kBatch * static_cast<int>(sizeof(Meta));
constexpr int kSmemBytes = 1024 + kWarps * (kWarpBytes + kMetaBytes);   // (the ring's alignment)
static_assert(kWarps * kMaxRows * (kPitch + 2) * 4 + 4 <= kWarps * kWarpBytes, "joining fits the ring");


// The part that a stretch holds of a tile: number k of count, the first one in slot slot0.
struct Part {
  int k, count, slot0, first;              // first: stretch of part 0
  __device__ __forceinline__ int64_t slot(int i) const {
    return i == 0 ? slot0 : 2 * (first + i);         // later parts open their stretch
  }
};

// A segment: one tile's rows over the steps [j0, j1) of its sequence that a stretch holds.
struct Seg {
  int64_t token0;                          // the sequence's first row of q and out
  int ctx, len, sink_steps, near_step;
  int b, tile, hk;
  int j0, j1;                              // j1 = 0: no more segments
  Part part;
};
struct Cursor {                            // where the block is on the line
  int64_t lo, hi;                          // its stretch
  int64_t a0;                              // place where the next segment's tile begins
  int b, item;                             // its sequence, its number there
  int group, head;                         // the stretch; this block's of a group's heads
  int64_t places;                          // of a tile of sequence b
  SeqWork w;                               // of sequence b
};

// The cursor's start, by the thread whose sequences (the first one is b, at place begin) hold it.
__device__ __forceinline__ void start_cursor(const AttnParams& p, const Line& l, int tile_rows, int b,
                                             int64_t begin, SeqWork w, bool only, Cursor* cur) {
  cur->group = static_cast<int>(blockIdx.y);
  cur->head = static_cast<int>(blockIdx.x);
  const int64_t lo = cur->group * l.share;
  cur->lo = lo;
  cur->hi = lo + l.share < l.total ? lo + l.share : l.total;
  if (!only) {
    w = seq_work(p, b, tile_rows);
    while (lo >= begin + work_of(l, w)) {
      begin += work_of(l, w);
      w = seq_work(p, ++b, tile_rows);
    }
  }
  const int64_t places = places_of(l, w), item = quotient(lo - begin, places);
  cur->b = b;
  cur->w = w;
  cur->item = static_cast<int>(item);
  cur->places = places;
  cur->a0 = begin + item * places;
}

__device__ __forceinline__ void advance(const AttnParams& p, const Line& l, int tile_rows, Cursor* cur) {
  cur->a0 += cur->places;
  if (++cur->item == cur->w.tiles * l.outer && cur->a0 < cur->hi) {
    cur->item = 0;
    do cur->w = seq_work(p, ++cur->b, tile_rows);
    while (cur->w.steps == 0);             // (a later sequence has work: the line is not at its end)
    cur->places = places_of(l, cur->w);
  }
}

// The segment at the cursor, which moves behind it.  One thread.
__device__ __forceinline__ void next_seg(const AttnParams& p, const Line& l, int inner, int tile_rows,
                                         Cursor* cur, Seg* sg) {
  const int64_t lo = cur->lo, hi = cur->hi;
  const int64_t a0 = cur->a0 + (l.whole ? 0 : kTileGap);     // place of the tile's first step
  if (a0 >= hi) {
    sg->j0 = sg->j1 = 0;
    return;
  }
  const int steps = cur->w.steps, tile = l.outer == 1 ? cur->item : cur->item / l.outer;
  sg->token0 = cur->w.s.row0;
  sg->ctx = cur->w.s.ctx;
  sg->len = cur->w.s.len;
  sg->sink_steps = cur->w.sink_steps;
  sg->near_step = cur->w.near_step;
  sg->b = cur->b;
  sg->tile = tile;
  sg->hk = (cur->item - tile * l.outer) * inner + cur->head;
  sg->j0 = a0 < lo ? static_cast<int>(lo - a0) : 0;
  sg->j1 = steps < hi - a0 ? steps : static_cast<int>(hi - a0);
  Part pt;
  pt.first = cur->group;
  if (a0 < lo) pt.first = static_cast<int>(quotient(a0, l.share));
  pt.slot0 = 2 * pt.first + (pt.first * l.share < a0 ? 1 : 0);
  pt.k = cur->group - pt.first;
  pt.count = pt.k + 1;                     // (the stretches behind this one)
  if (a0 + steps > hi) pt.count += static_cast<int>(quotient(a0 + steps - hi + l.share - 1, l.share));
  sg->part = pt;
  advance(p, l, tile_rows, cur);
}

// Page id of step i of this warp's, two batches ahead of the requests: -1: no page or nothing
// visible.  A warp's steps are every kWarps-th pair of the segment's.
__device__ __forceinline__ int warp_steps(const Seg& sg) {
  return (sg.j1 - sg.j0 + 2 * kWarps - 1) / (2 * kWarps) * 2;   // (the last may lie behind j1)
}
__device__ __forceinline__ int place_of(const Seg& sg, int warp, int i) {
  return sg.j0 + ((i >> 1) * kWarps + warp) * 2 + (i & 1);
}
__device__ __forceinline__ int token_of(const Seg& sg, int place) {
  return (place < sg.sink_steps ? place : sg.near_step + (place - sg.sink_steps)) * kStepTokens;
}
template <int ROWS>
__device__ __forceinline__ int64_t load_id(const AttnParams& p, const Seg& sg, int group, int warp,
                                           int i) {
  const int j = place_of(sg, warp, i);
  if (i >= warp_steps(sg) || j >= sg.j1) return -1;
  const int t0 = token_of(sg, j), blk = static_cast<int>(div_fast(t0 >> 4, p.pg.runs));
  const int last = sg.tile * ROWS + ROWS < sg.len * group ? sg.tile * ROWS + ROWS : sg.len * group;
  const int lo = sg.ctx + sg.tile * ROWS / group, hi = sg.ctx + (last - 1) / group;
  if (blk >= p.pg.max_blocks || t0 > hi ||
      (p.window > 0 && lo - (t0 + kStepTokens - 1) >= p.window && t0 >= p.sinks))
    return -1;
  return p.pg.table[static_cast<int64_t>(sg.b) * p.pg.max_blocks + blk];
}

// What a thread holds of a segment's result: a row's sums in units of 2^(top - kHead).
template <int NT>
struct Held {
  static constexpr int kRows = 8 * NT, kThreadsRow = kWarps * 32 / kRows, kQuads = 32 / kThreadsRow;
  float4 acc[kQuads];
  float top, sum;
};

// A segment's result goes out, or up the tree: node i of level v stands for parts i * 8^v.
template <bool BF16, int NT>
__device__ __forceinline__ void finish(const AttnParams& p, const Seg& sg, const Parts& parts, Held<NT>& r,
                                       int* flag) {
  using H = Half16<BF16>;
  using T = typename H::T;
  constexpr int kThreadsRow = Held<NT>::kThreadsRow, kQuads = Held<NT>::kQuads;
  const int row = threadIdx.x / kThreadsRow, col = (threadIdx.x % kThreadsRow) * 4;
  const int group = p.Nq / p.Nk, rows = sg.len * group, row0 = sg.tile * Held<NT>::kRows;
  const Part part = sg.part;
  const int head = sg.hk % parts.inner;
  auto slot = [&](int i) { return (part.slot(i) * parts.inner + head) * kMaxRows + row; };
  int node = part.k, nodes = part.count;
  bool last = true;
  for (int level = 0; nodes > 1; ++level, node >>= 3, nodes = (nodes + 7) >> 3) {
    const int base = node & ~7;            // the first child under this node's parent
    const int kids = nodes - base < 8 ? nodes - base : 8;
    if (kids == 1) continue;               // alone under its parent
    const int64_t mine = slot(node << (3 * level));
#pragma unroll
    for (int q4 = 0; q4 < kQuads; ++q4)
      __stcg(reinterpret_cast<float4*>(parts.out + mine * kHeadDim + q4 * (4 * kThreadsRow) + col),
             r.acc[q4]);
    if (col == 0) __stcg(reinterpret_cast<float2*>(parts.ml + mine * 2), make_float2(r.top, r.sum));
    __syncthreads();
    if (threadIdx.x == 0) {
      // The parent's counter is that of a stretch which one of its parts opens (any part but the
      // first does): part 8j, or 1 for j = 0, on level 0; above, the parts level + 1 behind 64j.
      const int at = level == 0 ? (base == 0 ? 1 : base) : (base << (3 * level)) + level + 1;
      const int stretch = (part.first + at) * parts.inner + head;
      const uint32_t one = 1u << (4 * (stretch & 7));
      uint32_t* w = parts.arrived + (stretch >> 3);
      const uint32_t old = arrive(w, one); // behind the block's stores, before its loads
      const bool full = ((old >> (4 * (stretch & 7))) & 15u) == static_cast<uint32_t>(kids - 1);
      if (full) atomicSub(w, one * kids);  // zero again for the next call
      *flag = full;
    }
    __syncthreads();
    last = *flag != 0;
    if (!last) break;
    // all loads of the children before the first use: one trip to the L2, not one for each
    float f[8];
    float2 ml[8];
    float4 v[2][8];
    auto fetch = [&](int q4) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float4* from = reinterpret_cast<const float4*>(
            parts.out + slot((base + (k < kids ? k : 0)) << (3 * level)) * kHeadDim + col);
        v[0][k] = __ldcg(from + q4 * kThreadsRow);
        v[1][k] = __ldcg(from + (q4 + 1) * kThreadsRow);
      }
    };
#pragma unroll
    for (int k = 0; k < 8; ++k)
      ml[k] = __ldcg(reinterpret_cast<const float2*>(
          parts.ml + slot((base + (k < kids ? k : 0)) << (3 * level)) * 2));
    fetch(0);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k >= kids) ml[k] = make_float2(-INFINITY, 0.f);
    r.top = -INFINITY;
    r.sum = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) r.top = fmaxf(r.top, ml[k].x);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      f[k] = ml[k].x == -INFINITY ? 0.f : exp2_approx(ml[k].x - r.top);
      r.sum = fmaf(ml[k].y, f[k], r.sum);
    }
#pragma unroll
    for (int q4 = 0; q4 < kQuads; q4 += 2) {
      if (q4 > 0) fetch(q4);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float4& a = r.acc[q4 + u];
        a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (k >= kids) continue;
          a.x = fmaf(v[u][k].x, f[k], a.x);
          a.y = fmaf(v[u][k].y, f[k], a.y);
          a.z = fmaf(v[u][k].z, f[k], a.z);
          a.w = fmaf(v[u][k].w, f[k], a.w);
        }
      }
    }
  }
  if (last && row0 + row < rows) {
    const int tok = (row0 + row) / group;
    T* dst = static_cast<T*>(p.out) +
             ((sg.token0 + tok) * p.Nq + sg.hk * group + (row0 + row - tok * group)) * kHeadDim + col;
    // a sum of 0: no key seen (a NaN sum stays NaN)
    const float rinv = r.sum == 0.f ? 0.f : 1.f / r.sum;
#pragma unroll
    for (int q4 = 0; q4 < kQuads; ++q4)
      *reinterpret_cast<uint2*>(dst + q4 * (4 * kThreadsRow)) =
          make_uint2(H::pack(r.acc[q4].x * rinv, r.acc[q4].y * rinv),
                     H::pack(r.acc[q4].z * rinv, r.acc[q4].w * rinv));
  }
}

template <bool BF16, int NT>
__global__ void __launch_bounds__(kWarps * 32, 3) paged_decode_kernel(
    const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const AttnParams p,
    const Parts parts) {
  using H = Half16<BF16>;
  using T = typename H::T;
  constexpr int kRows = 8 * NT;            // NT: eight-row tiles, 1 or 2
  extern __shared__ uint8_t raw_smem[];
  uint8_t* smem = raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023);
  __shared__ uint64_t arrived[kWarps][2];  // a warp's pairs of steps
  __shared__ int gave_up[kWarps];
  __shared__ Line line;
  __shared__ Cursor cur;
  __shared__ Seg segs[3];                  // the last, this and the next one
  __shared__ int flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int group = p.Nq / p.Nk;
  const int bs = p.pg.block_size;
  uint8_t* ring = smem + warp * kWarpBytes;
  Meta* meta = reinterpret_cast<Meta*>(smem + kWarps * kWarpBytes + warp * kMetaBytes);
  auto check_id = [&](int64_t id) -> int {
    if (id < -1 || id >= p.pg.block_num) {
      atomicOr(p.err, kErrIndexRange);
      return -1;
    }
    return static_cast<int>(id);
  };
  if (threadIdx.x == 0) {
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  if (lane == 0) {
    mbar_init(&arrived[warp][0], 1);
    mbar_init(&arrived[warp][1], 1);
    gave_up[warp] = 0;
    fence_mbarrier_init();
  }
  __syncthreads();
  uint32_t phases = 0;                     // bit i: parity of pair slot i's next arrival
  bool dead = false;                       // a copy did not arrive
  grid_dependency_wait();
  {
    const int per_thread = (p.rag.B + kWarps * 32 - 1) / (kWarps * 32);
    int64_t begin, places;
    SeqWork w;
    const Line l = lay_line(p, parts, kRows, per_thread, (blockIdx.x | blockIdx.y) == 0, &begin, &places, &w);
    const int64_t lo = blockIdx.y * l.share;
    if (lo >= l.total) return;
    if (begin <= lo && lo < begin + places) {            // one thread
      line = l;
      start_cursor(p, l, kRows, threadIdx.x * per_thread, begin, w, per_thread == 1, &cur);
      next_seg(p, l, parts.inner, kRows, &cur, &segs[0]);
    }
    __syncthreads();
    if (segs[0].j1 == 0) return;           // nothing but a tile's empty places
  }
  Held<NT> held;
  int64_t id = load_id<kRows>(p, segs[0], group, warp, lane);
  int64_t id_next = load_id<kRows>(p, segs[0], group, warp, kBatch + lane);
  int now = 0, before = 2, after = 1;
  for (int k = 0;; ++k) {
    const Seg& sg = segs[now];
    if (sg.j1 == 0) break;
    const int n = dead ? 0 : warp_steps(sg);
    const int rows = sg.len * group, row0 = sg.tile * kRows;
    const int row_last = row0 + kRows - 1 < rows ? row0 + kRows - 1 : rows - 1;
    const int pos_lo = sg.ctx + row0 / group, pos_hi = sg.ctx + row_last / group;
    float ks = 0.f, vs = 0.f;
    auto load_scales = [&](int64_t page) {
      const bool ok = page >= 0 && page < p.pg.block_num;
      ks = ok ? p.pg.k_scale[page * p.Nk + sg.hk] : 0.f;
      vs = ok ? p.pg.v_scale[page * p.Nk + sg.hk] : 0.f;
    };
    auto put_place = [&](int i, int64_t id) {            // of this lane's step i of the batch
      const int t0 = token_of(sg, place_of(sg, warp, i));
      const int row = t0 - static_cast<int>(div_fast(t0 >> 4, p.pg.runs)) * bs;
      reinterpret_cast<int4*>(meta + (i & (2 * kBatch - 1)))[1] = make_int4(t0, check_id(id), row, 0);
    };
    auto put_scales = [&](int i) {
      constexpr float units = BF16 ? kCodeUnits : 1.f;
      const float vabs = fmaxf(fabsf(vs), kTinyScale);
      reinterpret_cast<float4*>(meta + (i & (2 * kBatch - 1)))[0] =
          make_float4(fmaf(ks, 0.f, ks * units * p.scale_log2),  // (an infinite scale gives NaN: code 0 * inf is)
                      fmaf(vs, 0.f, __log2f(vabs)), __fdividef(1.f, vabs),
                      vs <= -kTinyScale ? -1.f : fabsf(vs) < kTinyScale ? 0.f : 1.f);
    };
    // Fragments.  A row's 16-byte piece i lies at i ^ (row & 7).  k: rows g and g + 8, pieces 2c and
    // 2c + 1; v: rows 2c, 2c + 1, 2c + 8, 2c + 9, piece g: no bank twice in eight lanes' reads.
    const uint32_t kr = g * 128 + (((2 * c) ^ g) << 4);
    const uint32_t vr = 2048 + 2 * c * 128 + ((g ^ (2 * c)) << 4);
    auto issue_pair = [&](int i) {           // i even
      if (i < n) {
        if (i > 0 && (i & (kBatch - 1)) == 0) {
          put_place(i + lane, id_next);
          put_scales(i + lane);            // (requested with the previous batch)
          id_next = load_id<kRows>(p, sg, group, warp, i + kBatch + lane);
          __syncwarp();
        }
        __syncwarp();                      // the slot's last pair has been read
        const int4* at = reinterpret_cast<const int4*>(meta + (i & (2 * kBatch - 1)));
        const int4 a = at[1], b = at[3];
        uint64_t* bar = &arrived[warp][(i >> 1) & 1];
        const int runs = (a.y >= 0) + (b.y >= 0);
        if (lane == 0 && runs != 0) mbar_arrive_expect_tx(bar, runs * kStepBytes);
        __syncwarp();
        const int page = lane & 2 ? b.y : a.y, row = lane & 2 ? b.z : a.z;
        if (lane < 4 && page >= 0)         // step a's k and v, step b's
          load_run(ring + (i & (kStages - 1)) * kStepBytes + lane * (kStepBytes / 2),
                   lane & 1 ? &vmap : &kmap, bar, sg.hk, row, page);
      }
    };
    put_place(lane, id);
    issue_pair(0);
    load_scales(id);
    if (k > 0) finish<BF16, NT>(p, segs[before], parts, held, &flag);   // of the last segment
    if (threadIdx.x == 0) next_seg(p, line, parts.inner, kRows, &cur, &segs[after]);

    // q rows 8t + g, the channels of this lane's k pieces: step s holds four of them
    uint32_t qb[NT][8][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int row = row0 + 8 * t + g;
      const int tok = row / group;
      const bool ok = row < rows;
      const T* q = static_cast<const T*>(p.q) +
                   ((sg.token0 + tok) * p.Nq + sg.hk * group + (row - tok * group)) * kHeadDim + c * 32;
#pragma unroll
      for (int h = 0; h < 4; ++h) {          // 8 channels at a time
        uint4 raw = make_uint4(0u, 0u, 0u, 0u);
        if (ok) raw = *reinterpret_cast<const uint4*>(q + h * 8);
        qb[t][2 * h][0] = raw.x;
        qb[t][2 * h][1] = raw.y;
        qb[t][2 * h + 1][0] = raw.z;
        qb[t][2 * h + 1][1] = raw.w;
      }
    }
    put_scales(lane);
    __syncwarp();

    // rows 8t + 2c + e: positions, running maximum and sum; O^T tile i: channels 16g + 2i, + 1
    int pos[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) pos[t][e] = sg.ctx + (row0 + 8 * t + 2 * c + e) / group;
    float o[NT][8][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][i][e] = 0.f;
    }

    for (int i = 0; i < n; i += 2) {
      issue_pair(i + 2);
      if (((i + 2) & (kBatch - 1)) == kBatch / 2) load_scales(id_next);   // of the next batch
      const float4* mp = reinterpret_cast<const float4*>(meta + (i & (2 * kBatch - 1)));
      const int2 ta = *reinterpret_cast<const int2*>(mp + 1);
      const int2 tb = *reinterpret_cast<const int2*>(mp + 3);
      if ((ta.y & tb.y) < 0) continue;          // (nothing was requested either)
      const int slot = (i >> 1) & 1;
      if (!warp_wait(&arrived[warp][slot], (phases >> slot) & 1, &gave_up[warp])) {
        dead = true;
        break;
      }
      phases ^= 1u << slot;
      const uint8_t* src = ring + (i & (kStages - 1)) * kStepBytes;
      float s[NT][2][4];                     // [tile][step of the pair]: tokens g, g + 8; rows 2c, 2c+1
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][h][e] = 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint8_t* k = src + h * kStepBytes + (kr ^ (half << 4));
          const uint4 ka = *reinterpret_cast<const uint4*>(k);
          const uint4 kb = *reinterpret_cast<const uint4*>(k + 8 * 128);
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            const uint32_t u = word(ka, q4), v = word(kb, q4);
            const uint32_t a[4] = {codes16<BF16, 0x4140>(u), codes16<BF16, 0x4140>(v),
                                   codes16<BF16, 0x4342>(u), codes16<BF16, 0x4342>(v)};
#pragma unroll
            for (int t = 0; t < NT; ++t)
              mma_16<BF16>(s[t][h], a, qb[t][half * 4 + q4][0], qb[t][half * 4 + q4][1]);
          }
        }
      }
      // x + log2 |vs|; hidden keys to -inf
      const float4 fa = mp[0], fb = mp[2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[t][0][e] = fmaf(s[t][0][e], fa.x, fa.y);
          s[t][1][e] = fmaf(s[t][1][e], fb.x, fb.y);
        }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t0 = h ? tb.x : ta.x, live = (h ? tb.y : ta.y) >= 0;
        const bool all = live && t0 + kStepTokens - 1 <= pos_lo &&
                         (p.window == 0 || pos_hi - t0 < p.window || t0 + kStepTokens <= p.sinks);
        if (!all) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int tok = t0 + g + (e >> 1) * 8, ps = pos[t][e & 1];
              const bool see = live && tok <= ps &&
                               (p.window == 0 || ps - tok < p.window || tok < p.sinks);
              if (!see) s[t][h][e] = -INFINITY;
            }
        }
      }
      float mx[NT][2];
      bool grow = false;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = fmaxf(fmaxf(s[t][0][e], s[t][0][2 + e]), fmaxf(s[t][1][e], s[t][1][2 + e]));
          mx[t][e] = v;
          grow |= v > m[t][e] + kLag;
        }
      if (__any_sync(0xffffffffu, grow)) {   // rare once the largest scores are behind
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = mx[t][e];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
            const float mn = fmaxf(m[t][e], v);
            const float f2 = mn == -INFINITY ? 1.f : exp2_approx(m[t][e] - mn);
            m[t][e] = mn;
            l[t][e] *= f2;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              o[t][k][e] *= f2;
              o[t][k][2 + e] *= f2;
            }
          }
      }
      uint32_t pb[NT][2][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float o0 = (m[t][0] == -INFINITY ? 0.f : -m[t][0]) + kHead;
        const float o1 = (m[t][1] == -INFINITY ? 0.f : -m[t][1]) + kHead;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float p0 = exp2_approx(s[t][h][0] + o0), p1 = exp2_approx(s[t][h][1] + o1);
          const float p2 = exp2_approx(s[t][h][2] + o0), p3 = exp2_approx(s[t][h][3] + o1);
          const float inv = h ? fb.z : fa.z, sg = h ? fb.w : fa.w;
          l[t][0] = fmaf(p0 + p2, inv, l[t][0]);
          l[t][1] = fmaf(p1 + p3, inv, l[t][1]);
          pb[t][h][0] = transpose8x8(Half16<false>::pack(p0 * sg, p1 * sg));
          pb[t][h][1] = transpose8x8(Half16<false>::pack(p2 * sg, p3 * sg));
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* v = src + h * kStepBytes + vr;
        const uint4 va = *reinterpret_cast<const uint4*>(v);
        const uint4 vb = *reinterpret_cast<const uint4*>(src + h * kStepBytes + ((vr + 128) ^ 16));
        const uint4 vc = *reinterpret_cast<const uint4*>(v + 1024);
        const uint4 vd = *reinterpret_cast<const uint4*>(src + h * kStepBytes + ((vr + 128) ^ 16) + 1024);
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {     // four of this lane's sixteen channels: two tiles
          const uint32_t x0 = word(va, q4) ^ 0x80808080u, x1 = word(vb, q4) ^ 0x80808080u;
          const uint32_t x2 = word(vc, q4) ^ 0x80808080u, x3 = word(vd, q4) ^ 0x80808080u;
          const uint32_t ab0 = __byte_perm(x0, x1, 0x5140), ab1 = __byte_perm(x0, x1, 0x7362);
          const uint32_t cd0 = __byte_perm(x2, x3, 0x5140), cd1 = __byte_perm(x2, x3, 0x7362);
          const uint32_t a0[4] = {codes_f16<0x4140>(ab0), codes_f16<0x4342>(ab0),
                                  codes_f16<0x4140>(cd0), codes_f16<0x4342>(cd0)};
          const uint32_t a1[4] = {codes_f16<0x4140>(ab1), codes_f16<0x4342>(ab1),
                                  codes_f16<0x4140>(cd1), codes_f16<0x4342>(cd1)};
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma_16<false>(o[t][q4 * 2], a0, pb[t][h][0], pb[t][h][1]);
            mma_16<false>(o[t][q4 * 2 + 1], a1, pb[t][h][0], pb[t][h][1]);
          }
        }
      }
    }
    if (dead && lane == 0) {               // the copies in flight end before the block does
      atomicOr(p.err, kErrTimeout);
      volatile int late = 0;
      for (int e = 0; e < 2; ++e) mbar_wait(&arrived[warp][e], (phases >> e) & 1, &late);
    }
    __syncwarp();

    // ---- join the warps: rows' maxima and sums first, then the outputs in units of the largest m
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], d);
    __syncthreads();                         // every warp is done with its ring
    id = load_id<kRows>(p, segs[after], group, warp, lane);          // of the next segment
    id_next = load_id<kRows>(p, segs[after], group, warp, kBatch + lane);
    float* wo = reinterpret_cast<float*>(smem);                     // (kWarps, kRows, kPitch)
    float* wm = wo + kWarps * kRows * kPitch;                       // (kWarps, kRows)
    float* wl = wm + kWarps * kRows;
    if (g == 0) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          wm[warp * kRows + 8 * t + 2 * c + e] = m[t][e];
          wl[warp * kRows + 8 * t + 2 * c + e] = l[t][e];
        }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * t + 2 * c + e;
        float top = -INFINITY;
#pragma unroll
        for (int k2 = 0; k2 < kWarps; ++k2) top = fmaxf(top, wm[k2 * kRows + row]);
        const float f2 = m[t][e] == -INFINITY ? 0.f : exp2_approx(m[t][e] - top);
        float* dst = wo + (warp * kRows + row) * kPitch + 16 * g;
#pragma unroll
        for (int k = 0; k < 4; ++k)          // channels 16g + 4k .. + 3: tiles 2k and 2k + 1
          *reinterpret_cast<float4*>(dst + 4 * k) =
              make_float4(o[t][2 * k][e] * f2, o[t][2 * k][2 + e] * f2, o[t][2 * k + 1][e] * f2,
                          o[t][2 * k + 1][2 + e] * f2);
      }
    __syncthreads();
    constexpr int kThreadsRow = Held<NT>::kThreadsRow, kQuads = Held<NT>::kQuads;
    const int row = threadIdx.x / kThreadsRow, col = (threadIdx.x % kThreadsRow) * 4;
    held.top = -INFINITY;
    held.sum = 0.f;
#pragma unroll
    for (int k2 = 0; k2 < kWarps; ++k2) held.top = fmaxf(held.top, wm[k2 * kRows + row]);
#pragma unroll
    for (int k2 = 0; k2 < kWarps; ++k2) {
      const float mk = wm[k2 * kRows + row];
      held.sum = fmaf(wl[k2 * kRows + row], mk == -INFINITY ? 0.f : exp2_approx(mk - held.top), held.sum);
    }
#pragma unroll
    for (int q4 = 0; q4 < kQuads; ++q4) {
      held.acc[q4] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k2 = 0; k2 < kWarps; ++k2) {
        const float4 v = *reinterpret_cast<const float4*>(
            wo + (k2 * kRows + row) * kPitch + q4 * (4 * kThreadsRow) + col);
        held.acc[q4].x += v.x;
        held.acc[q4].y += v.y;
        held.acc[q4].z += v.z;
        held.acc[q4].w += v.w;
      }
    }

    fence_proxy_async_shared();
    __syncthreads();                       // the ring is free for the next segment's copies
    before = now;
    now = after;
    after = 3 - before - now;
  }
  finish<BF16, NT>(p, segs[before], parts, held, &flag);
}

constexpr size_t kSlotBytes = (kMaxRows * kHeadDim + kMaxRows * 2) * sizeof(float);

}  // namespace

size_t paged_decode_workspace() { return 2 * kMaxStretches * kSlotBytes; }

cudaError_t launch_paged_decode(const CUtensorMap& k, const CUtensorMap& v, const AttnParams& p,
                                uint32_t* header, void* ws, cudaStream_t stream, int sm_count) {
  int stretches = sm_count * 3;            // all resident at once (registers and shared memory)
  if (stretches > kMaxStretches) stretches = kMaxStretches;
  Parts parts;
  parts.out = static_cast<float*>(ws);
  parts.ml = parts.out + static_cast<size_t>(2) * kMaxStretches * kMaxRows * kHeadDim;
  parts.arrived = header + 1;
  // heads that walk the line together: the most, up to eight, that divide the heads
  parts.inner = p.Nk < 8 ? p.Nk : 8;
  while (p.Nk % parts.inner) --parts.inner;
  stretches -= stretches % parts.inner;
  parts.outer = p.Nk / parts.inner;
  parts.groups = fast_div(static_cast<uint32_t>(stretches / parts.inner));
  // eight rows a tile while a sequence's rows of a head fit them
  const bool one = static_cast<int64_t>(p.rag.max_new) * (p.Nq / p.Nk) <= 8;
  auto kern = p.bf16 ? (one ? paged_decode_kernel<true, 1> : paged_decode_kernel<true, 2>)
                     : (one ? paged_decode_kernel<false, 1> : paged_decode_kernel<false, 2>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(parts.inner), static_cast<unsigned>(stretches / parts.inner));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, k, v, p, parts);
}

}  // namespace mlap
