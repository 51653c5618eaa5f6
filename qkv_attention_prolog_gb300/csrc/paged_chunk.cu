// Attention of many query rows per sequence (chunks of prompts) over the paged 8-bit cache.
//
//   x[t] = scale * log2(e) * ks * (q . kc[t]),   P[t] = 2^(x[t] + log2(vs) - m),
//   out  = (sum_t P[t] vc[t]) / (sum_t P[t] / vs)
//
// with the codes kc, vc and the scales ks, vs of the token's page (the sign of vs goes to the codes),
// as in paged_decode.cu, on the tensor cores' tcgen05 path, as in window_attn.cu: two tiles of 128
// query rows against one stream of 128-key tiles, S and O in tensor memory, P in place of S.
//
//   warp 0          issues the products: S_i = Q_i K^T in q's type, then O_i += P_i V in f16
//   warps 4..7      softmax of tile 0, a thread a row; warps 8..11 of tile 1
//   warps 1..3 and 12..14 expand the codes, exactly: a tile's K rows from the pages to q's type, its
//                   V rows to f16, in the operands' swizzled layout, two stages; the first of them
//                   requests an item's Q by TMA
//   warp 15         looks up the pages and scales of the tiles' eight runs of 16 tokens, ahead
//
// A step (128 keys of both tiles) takes 2.1 us, and as much with one tile: it is bound by the chain
// score product, softmax, value product of a tile, which the other one's fills, and which the
// expanders' instructions on the same schedulers lengthen (window_attn.cu, without them, 1.6 us).
// Rows of no page and rows behind the sequence's end become zeros, so nothing that is masked
// reaches a product.
//
// Items (256 rows of a head) are dealt whole while there is one for each CTA; what is left, fewer
// than CTAs, is split by steps, and the parts meet in the workspace.  2 x 1000 tokens over 8192,
// 256 items: 246 us, 1.16 PFLOP/s (before K's codes became q's type 297, without the split 328).  256 tokens over 50000,
// 32 items: 187 us.  116 prompts of up to 143 tokens, items of one or two steps: 79 us; bf16 queries
// scaled into f16's range took a third longer in shared memory, twice as long in registers (2 x 1000
// over 8192: 255 and 268).
// What did not pay: three expanding warps (353 us) or seven without a warp of look-ups
// (380), other orders of the issuing warp's waits (the same).
#include "attn_tile.cuh"

namespace mlap {

namespace {

constexpr int kThreads = 512;
constexpr int kExpandWarps = 6;            // warps 1..3 and 12..14
constexpr int kExpanders = kExpandWarps * 32;
constexpr int kPasses = (kTile / 4 + kExpandWarps - 1) / kExpandWarps;   // four-row groups of each
constexpr int kRuns = kTile / 16;          // runs of 16 tokens of a tile: one page each
constexpr int kInfos = 4;                  // tiles whose scales are kept
constexpr float kHead = 6.f;               // P is held 2^6 above its own scale (f16 operands)

struct Run {                               // 16 tokens of one page
  int64_t off;                             // byte offset of the first row in the caches, or -1
  int32_t flags;                           // (first run of a tile) kLive, kSame, kPlain
  float sign;                              // of vs; 0: vs counts as 0
  float f, lv, inv, pad;                   // ks * scale * log2(e), log2|vs|, 1/|vs|
};
constexpr int kLive = 1;                   // every run has a page
constexpr int kSame = 2;                   // all runs have the same scales, f > 0
constexpr int kPlain = 4;                  // every value scale is positive

struct Bars {
  uint64_t q_full, q_empty, k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t s_full[2], p_full[2][2], o_done[2], drain;
  uint64_t info_full[kInfos], info_empty[kInfos];
  uint32_t tmem;
  int abort;
  uint64_t parted[2];                      // the softmax warps of a tile among themselves
  int last[2];                             // the tile's other parts are all there
  int longest;                             // steps of a shared item
};
constexpr int kBarBytes = 384;
static_assert(sizeof(Bars) <= kBarBytes, "barriers");
constexpr int kInfoBytes = kInfos * kRuns * static_cast<int>(sizeof(Run));
constexpr int kSmemBytes =
    (2 + 2 * kStages) * kOperand + 1024 + kBarBytes + kInfoBytes + (kCountedSeqs + 1) * 4 +
    (kSplitCtas + 1) * 4;
// What a CTA works on: an item's steps [from, from + blk.steps).
struct Piece {
  Block blk;
  TilePart part;
  int hk, b;
  int from;
};

// 16 bytes, or zeros without an access; no branch, so that several are in flight.
__device__ __forceinline__ uint4 load_or_zero(const int8_t* at, bool ok) {
  uint4 v;
  asm volatile(
      "{\n.reg .pred P;\n"
      "setp.ne.b32 P, %5, 0;\n"
      "mov.b32 %0, 0;\nmov.b32 %1, 0;\nmov.b32 %2, 0;\nmov.b32 %3, 0;\n"
      "@P ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n}\n"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "l"(at), "r"(static_cast<int>(ok))
      : "memory");
  return v;
}

// Sixteen codes (piece c of row r) into an operand tile: 128-byte rows of 64 elements, two halves,
// 128-byte swizzle.
template <bool BF16>
__device__ __forceinline__ void put_codes(uint8_t* tile, int r, int c, uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint8_t* row = tile + (c >> 2) * kHalf + r * 128;
  const int at = (c & 3) * 2, swz = r & 7;
  *reinterpret_cast<uint4*>(row + ((at ^ swz) << 4)) =
      make_uint4(codes16<BF16, 0x4140>(w[0]), codes16<BF16, 0x4342>(w[0]), codes16<BF16, 0x4140>(w[1]),
                 codes16<BF16, 0x4342>(w[1]));
  *reinterpret_cast<uint4*>(row + (((at + 1) ^ swz) << 4)) =
      make_uint4(codes16<BF16, 0x4140>(w[2]), codes16<BF16, 0x4342>(w[2]), codes16<BF16, 0x4140>(w[3]),
                 codes16<BF16, 0x4342>(w[3]));
}

// The same sixteen elements, negated or (sign 0) cleared.
__device__ __forceinline__ void sign_codes(uint8_t* tile, int r, int c, float sign) {
  uint8_t* row = tile + (c >> 2) * kHalf + r * 128;
  const uint32_t flip = sign < 0.f ? 0x80008000u : 0u, keep = sign == 0.f ? 0u : ~0u;
  for (int e = 0; e < 2; ++e) {
    uint4* at = reinterpret_cast<uint4*>(row + ((((c & 3) * 2 + e) ^ (r & 7)) << 4));
    const uint4 v = *at;
    *at = make_uint4((v.x ^ flip) & keep, (v.y ^ flip) & keep, (v.z ^ flip) & keep,
                     (v.w ^ flip) & keep);
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const AttnParams p, int tpt, int most, float* slots, uint32_t* arrived) {
  using H = Half16<BF16>;
  using T = typename H::T;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* sq = smem;                                // two Q tiles
  uint8_t* sk = sq + 2 * kOperand;
  uint8_t* sv = sk + kStages * kOperand;
  Bars* bar = reinterpret_cast<Bars*>(sv + kStages * kOperand);
  Run* info = reinterpret_cast<Run*>(sv + kStages * kOperand + kBarBytes);
  int* first = reinterpret_cast<int*>(info + kInfos * kRuns);
  int* line = first + kCountedSeqs + 1;              // places before each of the shared items
  volatile int* abort_flag = &bar->abort;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int group = p.Nq / p.Nk;
  const int bs = p.pg.block_size;
  const int capacity = p.pg.max_blocks * bs;

  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmQ);
    mbar_init(&bar->q_full, 1);
    mbar_init(&bar->q_empty, 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar->k_full[i], kExpanders);
      mbar_init(&bar->k_empty[i], 1);
      mbar_init(&bar->v_full[i], kExpanders);
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
    for (int i = 0; i < kInfos; ++i) {
      mbar_init(&bar->info_full[i], 1);
      mbar_init(&bar->info_empty[i], 1);
    }
    bar->abort = 0;
    bar->longest = 0;
    fence_mbarrier_init();
  }
  if (warp == 0) {
    tmem_alloc(&bar->tmem, 512);
    tmem_relinquish();
  }
  grid_dependency_wait();
  const bool counted = p.rag.B <= kCountedSeqs;
  if (counted) count_blocks(p.rag, tpt, first);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = uniform(bar->tmem);
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.rag.B; b += kThreads) {
      const SeqRows s = seq_rows(p.rag, b);
      if (s.bad || (s.len > 0 && s.ctx + s.len > capacity)) atomicOr(p.err, kErrIndexRange);
    }

  const int items = counted ? uniform(first[p.rag.B]) * p.Nk : most;
  auto block_at = [&](int n, int* hk, int* b) {      // of item n
    *hk = n % p.Nk;
    const int at = n / p.Nk;
    *b = counted ? seq_of_block(first, p.rag.B, at) : at % p.rag.B;
    const int index = counted ? at - first[*b] : at / p.rag.B;
    const SeqRows s = seq_rows(p.rag, *b);
    return index < blocks_of(s, tpt) ? block_of(p, s, index, tpt, capacity, 16, 16) : Block{};
  };
  const int ctas = gridDim.x, whole = items / ctas;  // rounds of whole items
  const int shared = items - whole * ctas;
  {                                        // the line: an item's empty places, then its steps
    const int t = threadIdx.x;
    int hk, b, n = 0;
    if (t < shared) {
      const Block k = block_at(whole * ctas + t, &hk, &b);
      n = k.tiles > 0 ? k.steps + kGap : 0;
      line[t + 1] = n;
      atomicMax(&bar->longest, k.steps);
    }
    if (t == 0) line[0] = 0;
    __syncthreads();
    if (warp == 0) sum_line(line, shared);
    __syncthreads();
  }
  const int total = line[shared];
  bool split;
  int share = stretch_of(total, bar->longest, ctas, &split);
  share = uniform(split ? share : 1);
  int lo = 0, hi = 0, t_lo = 0, t_hi = 0;  // the stretch, and the shared items that it touches
  if (!split) {
    t_lo = min(static_cast<int>(blockIdx.x), shared);
    t_hi = min(t_lo + 1, shared);
    lo = line[t_lo];
    hi = line[t_hi];
  } else if (static_cast<int>(blockIdx.x) * share < total) {
    lo = blockIdx.x * share;
    hi = min(lo + share, total);
    t_lo = seq_of_block(line, shared, lo);
    t_hi = seq_of_block(line, shared, hi - 1) + 1;
  }
  // Every role walks the pieces alike; the pipelines run on from one to the next.
  const int rounds = uniform(whole + t_hi - t_lo);
  auto piece_of = [&](int round) {
    Piece x;
    const bool all = round < whole;
    const int t = t_lo + round - whole;
    x.blk = uniform_block(block_at(all ? dealt(round) : whole * ctas + t, &x.hk, &x.b));
    x.part = TilePart{0, 1, 0, 0};
    x.from = 0;
    if (!all && split) {
      const int n = x.blk.steps, a0 = line[t] + kGap;  // place of its first step
      const int j0 = lo > a0 ? min(lo - a0, n) : 0, j1 = min(max(hi - a0, 0), n);
      if (n == 0) {                        // no keys: the stretch with its last place writes zeros
        if (a0 - 1 < lo || a0 - 1 >= hi) x.blk.tiles = 0;
        return x;
      }
      x.part = part_of(a0, n, share, static_cast<int>(blockIdx.x));
      x.from = j0;
      x.blk.steps = uniform(j1 - j0);
      if (x.blk.steps <= 0) x.blk.steps = x.blk.tiles = 0;   // nothing but empty places
    }
    return x;
  };

  if (warp == 0) {
    // -------------------------------------------------------------------- products
    const uint32_t id_s = BF16 ? idesc_bf16_f32(kTile, kTile) : idesc_f16_f32(kTile, kTile);
    const uint32_t id_o = idesc_f16_f32(kTile, kTile) | kIdescNMajorB;
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
    int nq = 0, at = 0;                    // items and steps so far
    int done0 = 0, done1 = 0;              // steps of either tile
    bool ok = true;
    for (int r = 0; ok && r < rounds; ++r) {
      const Block blk = piece_of(r).blk;
      if (blk.steps == 0) continue;
      const bool two = blk.tiles == 2;
      ok = warp_wait(lane == 0 ? &bar->q_full : &bar->k_full[at % kStages],
                     lane == 0 ? nq & 1 : (at / kStages) & 1, abort_flag);
      if (!ok) break;
      ++nq;
      tc_fence_after_sync();
      if (elect_one()) {
        scores(0, at % kStages);
        if (two) scores(1, at % kStages);
        umma_commit(&bar->k_empty[at % kStages]);
        if (blk.steps == 1) umma_commit(&bar->q_empty);
      }
      for (int j = 0; ok && j < blk.steps; ++j, ++at) {
        const int st = at % kStages, nx = (at + 1) % kStages;
        const bool more = j + 1 < blk.steps;
        ok = warp_wait(&bar->v_full[st], (at / kStages) & 1, abort_flag);
        if (more) ok = ok && warp_wait(&bar->k_full[nx], ((at + 1) / kStages) & 1, abort_flag);
        ok = ok && warp_wait(&bar->p_full[0][0], done0 & 1, abort_flag);
        if (!ok) break;
        ++done0;
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
            if (i == 1 || !two) {
              umma_commit(&bar->v_empty[st]);
              umma_commit(&bar->info_empty[at % kInfos]);
            }
            if (more) {
              scores(i, nx);
              if (i == 1 || !two) {
                umma_commit(&bar->k_empty[nx]);
                if (j + 2 == blk.steps) umma_commit(&bar->q_empty);   // the item's last scores
              }
            }
          }
        }
      }
    }
    if (*abort_flag && lane == 0) {        // the products issued so far end before the CTA does
      umma_commit(&bar->drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(&bar->drain, 0) && globaltimer_ns() - t0 < 20000000ull) {
      }
    }
  } else if (warp < 4 || (warp >= 12 && warp < 15)) {
    // -------------------------------------------------------------------- codes
    const int ew = warp < 4 ? warp - 1 : warp - 9;   // 0 .. 5
    // a warp takes four rows at a time, eight lanes each: group 6i + ew, inside one run
    const int piece = lane & 7, sub = lane >> 3;
    const int64_t pitch = static_cast<int64_t>(p.Nk) * kHeadDim;
    int nq = 0, at = 0;                    // items and tiles so far
    bool ok = true;
    for (int r = 0; ok && r < rounds; ++r) {
      const Piece pc = piece_of(r);
      const Block blk = pc.blk;
      const int hk = pc.hk;
      if (blk.steps == 0) continue;
      if (ew == 0) {                       // Q (rows of no token are whatever lies there)
        ok = warp_wait(&bar->q_empty, (nq & 1) ^ 1, abort_flag);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar->q_full, blk.tiles * 2 * group * tpt * 128);
          for (int i = 0; i < blk.tiles; ++i)
            for (int h = 0; h < 2; ++h)
              tma_load_3d(sq + i * kOperand + h * kHalf, &tmQ, &bar->q_full, h * 64, hk * group,
                          static_cast<int>(blk.s.row0) + blk.tok0 + i * tpt);
        }
        ++nq;
      }

      uint4 k[kPasses], v[kPasses];
      const int64_t lane_off = sub * pitch + piece * 16;
      auto fetch = [&](const int8_t* cache, int n, uint4 (&x)[kPasses]) {
        int64_t off[kPasses];
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const int g = kExpandWarps * i + ew;
          off[i] = g < kTile / 4 ? info[(n % kInfos) * kRuns + (g >> 2)].off : -1;
        }
#pragma unroll
        for (int i = 0; i < kPasses; ++i)
          x[i] = load_or_zero(cache + off[i] + lane_off + ((kExpandWarps * i + ew) & 3) * 4 * pitch,
                              off[i] >= 0);
      };
      auto put_k = [&](uint8_t* tile, const uint4 (&x)[kPasses]) {
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const int g = kExpandWarps * i + ew;
          if (g < kTile / 4) put_codes<BF16>(tile, 4 * g + sub, piece, x[i]);
        }
      };
      auto put_v = [&](uint8_t* tile, const uint4 (&x)[kPasses]) {
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const int g = kExpandWarps * i + ew;
          if (g < kTile / 4) put_codes<false>(tile, 4 * g + sub, piece, x[i]);
        }
      };
      // v rows of negative scales change their sign, those whose scale counts as 0 vanish
      auto put_signs = [&](uint8_t* tile, int n) {
        for (int i = 0; i < kPasses; ++i) {
          const int g = kExpandWarps * i + ew;
          if (g >= kTile / 4) break;
          const float sign = info[(n % kInfos) * kRuns + (g >> 2)].sign;
          if (sign != 1.f) sign_codes(tile, 4 * g + sub, piece, sign);
        }
      };
      ok = warp_wait(&bar->info_full[at % kInfos], (at / kInfos) & 1, abort_flag);
      if (!ok) break;
      fetch(p.pg.k, at, k);
      fetch(p.pg.v, at, v);
      for (int j = 0; j < blk.steps; ++j, ++at) {
        const int st = at % kStages;
        const uint32_t ph = ((at / kStages) & 1) ^ 1;
        const bool more = j + 1 < blk.steps;
        ok = warp_wait(&bar->k_empty[st], ph, abort_flag);
        if (!ok) break;
        put_k(sk + st * kOperand, k);
        fence_proxy_async_shared();
        mbar_arrive(&bar->k_full[st]);
        if (more) {
          ok = warp_wait(&bar->info_full[(at + 1) % kInfos], ((at + 1) / kInfos) & 1, abort_flag);
          if (!ok) break;
          fetch(p.pg.k, at + 1, k);
        }
        ok = warp_wait(&bar->v_empty[st], ph, abort_flag);
        if (!ok) break;
        put_v(sv + st * kOperand, v);
        if (!(info[(at % kInfos) * kRuns].flags & kPlain)) put_signs(sv + st * kOperand, at);
        fence_proxy_async_shared();
        mbar_arrive(&bar->v_full[st]);
        if (more) fetch(p.pg.v, at + 1, v);
      }
    }
    if (*abort_flag && ew == 0 && lane == 0 && nq > 0) {     // Q lands before the CTA exits
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(&bar->q_full, (nq - 1) & 1) && globaltimer_ns() - t0 < 20000000ull) {
      }
    }
  } else if (warp == 15) {
    // -------------------------------------------------------------------- pages and scales
    const int64_t pitch = static_cast<int64_t>(p.Nk) * kHeadDim;
    const bool mine = lane < kRuns;        // a run each
    const float units = BF16 ? kCodeUnits : 1.f;
    int at = 0;                            // tiles so far
    bool ok = true;
    for (int r = 0; ok && r < rounds; ++r) {
      const Piece pc = piece_of(r);
      const Block blk = pc.blk;
      const int hk = pc.hk, b = pc.b;
      if (blk.steps == 0) continue;
      const int rows_end = blk.tok0 + blk.tiles * tpt;
      const int pos_hi = blk.s.ctx + (rows_end < blk.s.len ? rows_end : blk.s.len) - 1;
      auto load_id = [&](int j) -> int64_t {
        if (!mine || j >= blk.steps) return -1;
        const int t0 = key_of(blk, (pc.from + j) * kTile + lane * 16);
        // (pages that no row of the block sees are left alone)
        if (t0 >= capacity || t0 > pos_hi ||
            (p.window > 0 && blk.pos0 - (t0 + 15) >= p.window && t0 >= p.sinks))
          return -1;
        return p.pg.table[static_cast<int64_t>(b) * p.pg.max_blocks + div_fast(t0 >> 4, p.pg.runs)];
      };
      float ks = 0.f, vs = 0.f;
      auto load_scales = [&](int64_t id) {
        const bool fine = id >= 0 && id < p.pg.block_num;
        ks = fine ? p.pg.k_scale[id * p.Nk + hk] : 0.f;
        vs = fine ? p.pg.v_scale[id * p.Nk + hk] : 0.f;
      };
      // page ids two tiles and scales one tile ahead of their use
      int64_t id = load_id(0), id1 = load_id(1);
      load_scales(id);
      for (int j = 0; j < blk.steps; ++j, ++at) {
        ok = warp_wait(&bar->info_empty[at % kInfos], ((at / kInfos) & 1) ^ 1, abort_flag);
        if (!ok) break;
        const int t0 = key_of(blk, (pc.from + j) * kTile + (lane & (kRuns - 1)) * 16);
        if (id < -1 || id >= p.pg.block_num) atomicOr(p.err, kErrIndexRange);
        Run x;
        const float vabs = fmaxf(fabsf(vs), kTinyScale);
        const int in = t0 - static_cast<int>(div_fast(t0 >> 4, p.pg.runs)) * bs;   // row of the page
        x.off = id < 0 || id >= p.pg.block_num ? -1 : (id * bs + in) * pitch + hk * kHeadDim;
        x.f = fmaf(ks, 0.f, ks * units * p.scale_log2);  // (an infinite scale gives NaN: code 0 * inf is)
        x.lv = fmaf(vs, 0.f, __log2f(vabs));
        x.inv = __fdividef(1.f, vabs);
        x.sign = vs <= -kTinyScale ? -1.f : fabsf(vs) < kTinyScale ? 0.f : 1.f;
        x.pad = 0.f;
        const bool live = __all_sync(0xffffffffu, !mine || x.off >= 0);
        const float f0 = __shfl_sync(0xffffffffu, x.f, 0), lv0 = __shfl_sync(0xffffffffu, x.lv, 0);
        const bool same = __all_sync(0xffffffffu, !mine || (x.f > 0.f && x.f == f0 && x.lv == lv0));
        const bool plain = __all_sync(0xffffffffu, !mine || x.sign == 1.f || x.off < 0);
        x.flags = (live ? kLive : 0) | (live && same ? kSame : 0) | (plain ? kPlain : 0);
        if (mine) info[(at % kInfos) * kRuns + lane] = x;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->info_full[at % kInfos]);
        id = id1;
        load_scales(id);
        id1 = load_id(j + 2);
      }
    }
  } else {
    // -------------------------------------------------------------------- softmax, a thread a row
    const int i = (warp >> 2) - 1;
    const int row = threadIdx.x & (kTile - 1);
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;     // this warp's 32 lanes
    const uint32_t ts = tmem + i * kTile + lanes, to = tmem + (2 + i) * kTile + lanes;
    const int row_tok = row / group, row_head = row - row_tok * group;
    // tokens of this warp's rows, behind the tile's first
    const int warp_lo = (warp & 3) * 32 / group, warp_hi = ((warp & 3) * 32 + 31) / group;
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
    int done = 0;                          // steps of this tile so far
    int at = 0;                            // tiles of the kernel so far
    bool ok = true;
    for (int r = 0; ok && r < rounds; ++r) {
      const Piece pc = piece_of(r);
      const Block& blk = pc.blk;
      const int hk = pc.hk;
      if (blk.tiles <= i) {
        at += blk.steps;
        continue;
      }
      const int tok = blk.tok0 + i * tpt + row_tok, pos = blk.s.ctx + tok;
      const int pos_lo = blk.pos0 + i * tpt + warp_lo, pos_hi = blk.pos0 + i * tpt + warp_hi;
      const Seen seen(p, blk, pos_lo, pos_hi);
      // (rows of no token hold what is left in shared memory: they never raise m, which is their warp's
      // decision for all of its rows)
      const bool mine = row < group * tpt && tok < blk.s.len;
      float m = mine ? -INFINITY : INFINITY, l = 0.f;
      for (int j = 0; j < blk.steps; ++j, ++done, ++at) {
        ok = warp_wait(&bar->s_full[i], done & 1, abort_flag);
        if (!ok) break;
        tc_fence_after_sync();
        const int u = (pc.from + j) * kTile;
        const Run* run = info + (at % kInfos) * kRuns;
        // Where all runs have the same scales their factors wait for the exponential; otherwise the
        // scores are scaled run by run and put back, as they are where a row does not see them all.
        const int flags = run[0].flags;
        const bool same = flags & kSame, all = (flags & kLive) && seen.all(u, kTile);
        const float f = same ? run[0].f : 1.f, lv = same ? run[0].lv : 0.f;
        float top = -INFINITY;
#pragma unroll 1
        for (int q = 0; q < kTile; q += 64) {          // 64 columns, four runs, at a time
          uint32_t s[2][32];
          tmem_ld_32x32b_x32(ts + q, s[0]);
          tmem_ld_32x32b_x32(ts + q + 32, s[1]);
          tmem_ld_wait();
          const Run* rq = run + q / 16;
          if (!same) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const float2 fl = *reinterpret_cast<const float2*>(&rq[g].f);
              const float2 f2 = make_float2(fl.x, fl.x), lv2 = make_float2(fl.y, fl.y);
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                uint32_t* x = &s[g >> 1][(g & 1) * 16 + e];
                const float2 y =
                    fma_x2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), f2, lv2);
                x[0] = __float_as_uint(y.x);
                x[1] = __float_as_uint(y.y);
              }
            }
          }
          if (!all) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t see = sees(p, blk, pos, u + q + k * 32);
              if (rq[2 * k].off < 0) see &= 0xffff0000u;
              if (rq[2 * k + 1].off < 0) see &= 0x0000ffffu;
              if (__all_sync(0xffffffffu, see == ~0u)) continue;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(see & (1u << e))) s[k][e] = __float_as_uint(-INFINITY);
            }
          }
          if (!same || !all) {
            tmem_st_32x32b_x32(ts + q, s[0]);
            tmem_st_32x32b_x32(ts + q + 32, s[1]);
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
        if (!same || !all) tmem_st_wait();
        top = fmaf(top, f, lv);
        if (__any_sync(0xffffffffu, top > m + kLag)) {
          const float mn = fmaxf(m, top);
          const float down = mn == -INFINITY ? 1.f : exp2_approx(m - mn);
          m = mn;
          l *= down;
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
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * down);
              tmem_st_32x32b_x16(to + q * 16, o);
            }
          }
        }
        const float off = lv + kHead - (m == -INFINITY ? 0.f : m);
        const float2 f2 = make_float2(f, f), off2 = make_float2(off, off);
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
            for (int h = 0; h < 2; ++h) {  // a run each
              float2 sum = make_float2(0.f, 0.f);
              const float inv = run[q / 16 + 2 * k + h].inv;
#pragma unroll
              for (int e = 8 * h; e < 8 * h + 8; ++e) {
                float2 x = make_float2(__uint_as_float(s[k][2 * e]), __uint_as_float(s[k][2 * e + 1]));
                x = fma_x2(x, f2, off2);
                x.x = exp2_approx(x.x);
                x.y = exp2_approx(x.y);
                sum = add_x2(sum, x);
                pk[e] = Half16<false>::pack(x.x, x.y);
              }
              l = fmaf(sum.x + sum.y, inv, l);
            }
            tmem_st_32x32b_x16(ts + (q >> 1) + k * 16, pk);
          }
          tmem_st_wait();
          tc_fence_before_sync();
          mbar_arrive(&bar->p_full[i][q >> 6]);
        }
      }
      if (!ok) break;
      // ---- out = O / l; zeros for a row that saw nothing (a NaN sum stays NaN)
      const int h = hk * group + row_head;
      uint4* dst = reinterpret_cast<uint4*>(
          static_cast<T*>(p.out) + ((blk.s.row0 + tok) * p.Nq + h) * kHeadDim);
      if (blk.steps == 0) {
        if (mine)
          for (int e = 0; e < 16; ++e) dst[e] = make_uint4(0u, 0u, 0u, 0u);
        continue;
      }
      ok = warp_wait(&bar->o_done[i], (done - 1) & 1, abort_flag);
      if (!ok) break;
      tc_fence_after_sync();
      auto slot = [&](int k) { return slots + (static_cast<int64_t>(pc.part.slot(k)) * 2 + i) * (kSlotFloats / 2); };
      bool write = true;
      if (pc.part.parts > 1) {
        float4* to_o = reinterpret_cast<float4*>(slot(pc.part.part)) + row;
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
        __stcg(reinterpret_cast<float2*>(slot(pc.part.part) + kTile * kHeadDim) + row, make_float2(m, l));
        mbar_arrive(&bar->parted[i]);
        ok = warp_wait(&bar->parted[i], 0, abort_flag);
        if (!ok) break;
        if (row == 0) bar->last[i] = last_part(arrived, pc.part, i);
        mbar_arrive(&bar->parted[i]);
        ok = warp_wait(&bar->parted[i], 1, abort_flag);
        if (!ok) break;
        write = bar->last[i] != 0;
        if (write) {                       // m and l of all parts
          float2 ml[kMostParts];
          m = -INFINITY;
          l = 0.f;
#pragma unroll
          for (int k = 0; k < kMostParts; ++k) {
            ml[k] = make_float2(-INFINITY, 0.f);
            if (k < pc.part.parts)
              ml[k] = __ldcg(reinterpret_cast<const float2*>(slot(k) + kTile * kHeadDim) + row);
          }
#pragma unroll
          for (int k = 0; k < kMostParts; ++k) m = fmaxf(m, ml[k].x);
#pragma unroll
          for (int k = 0; k < kMostParts; ++k)
            l = fmaf(ml[k].y, ml[k].x == -INFINITY ? 0.f : exp2_approx(ml[k].x - m), l);
        }
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
      for (int q = 0; write && q < 8; ++q) {
        float o[16];
        if (pc.part.parts == 1) {
          tmem_ld_32x32b_x16(to + q * 16, reinterpret_cast<uint32_t(&)[16]>(o));
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0.f;
#pragma unroll 1
          for (int k0 = 0; k0 < pc.part.parts; k0 += 4) {           // the loads of four parts at a time
            float mk[4];
            float4 v[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int kk = k0 + k < pc.part.parts ? k0 + k : pc.part.parts - 1;
              mk[k] = __ldcg(reinterpret_cast<const float2*>(slot(kk) + kTile * kHeadDim) + row).x;
              const float4* from = reinterpret_cast<const float4*>(slot(kk)) + q * 4 * kTile + row;
#pragma unroll
              for (int e = 0; e < 4; ++e) v[k][e] = __ldcg(from + e * kTile);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float down = mk[k] == -INFINITY || k0 + k >= pc.part.parts ? 0.f : exp2_approx(mk[k] - m);
              if (down == 0.f) continue;   // (a part that saw nothing, or none)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                o[4 * e] = fmaf(v[k][e].x, down, o[4 * e]);
                o[4 * e + 1] = fmaf(v[k][e].y, down, o[4 * e + 1]);
                o[4 * e + 2] = fmaf(v[k][e].z, down, o[4 * e + 2]);
                o[4 * e + 3] = fmaf(v[k][e].w, down, o[4 * e + 3]);
              }
            }
          }
        }
        if (mine) {                        // 32 bytes at a time: whole sectors
          uint32_t w[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) w[k] = H::pack(o[2 * k] * inv, o[2 * k + 1] * inv);
          store_32(dst + q * 2, w, wide);
        }
      }
      tc_fence_before_sync();              // O is read before the next item's first P is announced
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 0) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0 && *abort_flag) atomicOr(p.err, kErrTimeout);
}

int64_t items_of(const AttnParams& p, int tpt) {
  return ((p.rag.max_new + 2 * tpt - 1) / (2 * tpt)) * static_cast<int64_t>(p.Nk) * p.rag.B;
}

}  // namespace

// From four 16-row tiles a block on.  Both paths, this one second, 32 heads on 8:
//   three tiles (12 tokens)   16 x 8000: 136, 116 us   64 x 2000: 146, 125   1 x 50000: 59, 81
//                             1 x 1000: 12, 21         96 in a window of 1024: 105, 122
//   four tiles (16 tokens)    16 x 8000: 173, 116      64 x 2000: 188, 124   1 x 1000: 13, 21
//   six tiles (24 tokens)     16 x 8000: 252, 116      96 in a window of 1024: 188, 122
// (How long the contexts are is known on the device alone.)
bool paged_chunk_pays(const AttnParams& p) {
  const int group = p.Nq / p.Nk, tpt = window_attn_tokens(group);
  const int64_t small = (static_cast<int64_t>(p.rag.max_new) * group + 15) / 16;   // 16-row tiles
  const int64_t blocks = (p.rag.max_new + 2 * tpt - 1) / (2 * tpt);
  return small > 3 * blocks;
}

cudaError_t launch_paged_chunk(const CUtensorMap& q, const AttnParams& p, uint32_t* header, void* ws, cudaStream_t stream,
                               int sm_count) {
  const int tpt = window_attn_tokens(p.Nq / p.Nk);
  const int64_t items = items_of(p, tpt);
  const int ctas = sm_count < kSplitCtas ? sm_count : kSplitCtas;
  if (items > 0x7fffffffLL - ctas) return cudaErrorInvalidConfiguration;
  auto kern = p.bf16 ? paged_chunk_kernel<true> : paged_chunk_kernel<false>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, q, p, tpt, static_cast<int>(items), static_cast<float*>(ws),
                            header + 1);
}

}  // namespace mlap
