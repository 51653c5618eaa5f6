// Append: q, k, v split, optional RmsNorm, RoPE, int8 codes of k and v under one scale for each
// page and head, and their store into the pages.
//
//   z = rope(norm(x)) for q and k;   s = max(old, max|new| / 127);   code = rne(value / s)
//
// A unit is (sequence, page of it that receives tokens, head, k or v): one owner takes the maximum
// over all of the page's new tokens, settles the scale, brings the page's earlier codes to it
// where it grew, and writes the new codes, so no two blocks meet at a scale and the result does
// not depend on any order.  Blocks behind the units rotate q, a warp for eight heads of a token
// with the token's cos and sin held in registers.  Inside a warp eight lanes own one head row, each
// both members of its RoPE pairs (elements 8l..8l+7 and 64+8l..64+8l+7).
//
// Where a page receives at most 16 tokens a warp takes the unit, otherwise a CTA of eight.  16384
// tokens (32 + 8 + 8 heads) into pages of 16: 87 us with warps, 135 with CTAs; 12 new tokens for
// each of 256 sequences: 20 against 39 us; 24 for each of 64: 23 against 15 us.
//
// Bound by memory: 16 prompts of up to 1024 tokens move 256 MB in 52 us (4.9 TB/s), pages' rows
// coming from the L2 the second time.  Held instead in shared memory (64 KB, three CTAs on an SM)
// they cost 56 us, in registers 97; half a row's elements in each lane (sixteen lanes a row) 71;
// two CTAs on an SM 62, five 63 (four spill 44 bytes a thread, 240 where warps take units).
//
// Every product and sum is rounded on its own (no contraction), in one fixed order, so the codes
// are the same whole numbers that the operator's definition in 32-bit arithmetic gives.
#include "attn_common.cuh"

namespace mlap {

namespace {

constexpr int kWarps = 8;
constexpr int kQHeads = 8;                 // query heads of a token that a warp takes

struct Row16 {                 // this lane's 16 elements of a head row
  float a[8], b[8];
};
struct Raw16 {                 // the same as they lie in memory
  uint4 a, b;
};

template <bool BF16>
__device__ __forceinline__ Raw16 load_raw(const void* base, int64_t elem, int l8) {
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const typename Half16<BF16>::T*>(base) + elem);
  return Raw16{p[l8], p[8 + l8]};
}

template <bool BF16>
__device__ __forceinline__ Row16 widen(const Raw16& raw) {
  using H = Half16<BF16>;
  const typename H::T* ea = reinterpret_cast<const typename H::T*>(&raw.a);
  const typename H::T* eb = reinterpret_cast<const typename H::T*>(&raw.b);
  Row16 r;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    r.a[e] = H::to_f(ea[e]);
    r.b[e] = H::to_f(eb[e]);
  }
  return r;
}

// y = x / sqrt(mean x^2 + eps) * gamma over the row's eight lanes.
template <bool BF16>
__device__ __forceinline__ void norm_row(Row16* r, const void* gamma, float eps, int l8,
                                         unsigned mask) {
  float s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    s[e] = __fadd_rn(__fmul_rn(r->a[e], r->a[e]), __fmul_rn(r->b[e], r->b[e]));
#pragma unroll
  for (int w = 4; w > 0; w >>= 1) {
#pragma unroll
    for (int e = 0; e < w; ++e) s[e] = __fadd_rn(s[e], s[e + w]);
  }
  float ss = s[0];
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) ss = __fadd_rn(ss, __shfl_xor_sync(mask, ss, o));
  const float ms = __fadd_rn(__fmul_rn(ss, 1.0f / static_cast<float>(kHeadDim)), eps);
  const float rinv = __frcp_rn(__fsqrt_rn(ms));
  const Row16 g = widen<BF16>(load_raw<BF16>(gamma, 0, l8));
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    r->a[e] = __fmul_rn(__fmul_rn(r->a[e], rinv), g.a[e]);
    r->b[e] = __fmul_rn(__fmul_rn(r->b[e], rinv), g.b[e]);
  }
}

template <bool BF16>
__device__ __forceinline__ void rope_row(Row16* r, const Raw16& cos, const Raw16& sin) {
  const Row16 c = widen<BF16>(cos), s = widen<BF16>(sin);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = r->a[e], y = r->b[e];
    r->a[e] = __fadd_rn(__fmul_rn(x, c.a[e]), __fmul_rn(-y, s.a[e]));
    r->b[e] = __fadd_rn(__fmul_rn(y, c.b[e]), __fmul_rn(x, s.b[e]));
  }
}

// Largest magnitude (a NaN counts as nothing).
__device__ __forceinline__ float row_amax(const Row16& r) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fmaxf(fabsf(r.a[e]), fabsf(r.b[e])));
  return m;
}

__device__ __forceinline__ uint2 codes8(const float (&x)[8], float f) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    int c = __float2int_rn(__fmul_rn(x[e], f));
    c = c < -127 ? -127 : (c > 127 ? 127 : c);
    w[e >> 2] |= static_cast<uint32_t>(c & 0xff) << (8 * (e & 3));
  }
  return make_uint2(w[0], w[1]);
}

// This lane's 16 elements of token `row`, head h of k or v, as they enter the quantisation.
struct RawValue {
  Raw16 x, c, s;
};
template <bool BF16>
__device__ __forceinline__ RawValue load_value(const KvAppendParams& p, int64_t row, int h, bool is_v,
                                               int l8) {
  const int heads = p.Nq + 2 * p.pg.Nk;
  RawValue v;
  v.x = load_raw<BF16>(p.qkv, (row * heads + p.Nq + (is_v ? p.pg.Nk : 0) + h) * kHeadDim, l8);
  if (!is_v) {
    v.c = load_raw<BF16>(p.cos, row * kHeadDim, l8);
    v.s = load_raw<BF16>(p.sin, row * kHeadDim, l8);
  }
  return v;
}
template <bool BF16>
__device__ __forceinline__ Row16 value_of(const KvAppendParams& p, const RawValue& v, bool is_v, int l8,
                                          unsigned mask) {
  Row16 r = widen<BF16>(v.x);
  if (!is_v) {
    if (p.gamma_k != nullptr) norm_row<BF16>(&r, p.gamma_k, p.eps, l8, mask);
    rope_row<BF16>(&r, v.c, v.s);
  }
  return r;
}

// UW: warps of a unit (1 or kWarps).  Blocks [0, unit_blocks) take units, the rest q rows.
template <bool BF16, int UW>
__global__ void __launch_bounds__(kWarps * 32, 4) kv_append_kernel(const KvAppendParams p,
                                                                int pages_per_seq,
                                                                int64_t unit_blocks) {
  using H = Half16<BF16>;
  __shared__ float wmax[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l8 = lane & 7, sub = lane >> 3;
  const unsigned mask = 0xffu << (lane & 24);
  grid_dependency_wait();

  if (blockIdx.x >= unit_blocks) {         // ---- q: a warp takes kQHeads heads of a token, four at a
                                           // time, with the token's tables in registers
    const int64_t last = p.rag.cu[p.rag.B];
    const int64_t first = p.rag.cu[0] < 0 ? 0 : p.rag.cu[0];
    const int64_t rows = last < p.rag.T ? last : p.rag.T;
    const int parts = (p.Nq + kQHeads - 1) / kQHeads;
    const int64_t at = (blockIdx.x - unit_blocks) * kWarps + warp;
    const int64_t row = first + at / parts;
    const int h0 = static_cast<int>(at % parts) * kQHeads + sub;
    if (row >= rows) return;
    const int64_t src = (row * (p.Nq + 2 * p.pg.Nk) + h0) * kHeadDim;
    const Raw16 c = load_raw<BF16>(p.cos, row * kHeadDim, l8);
    const Raw16 s = load_raw<BF16>(p.sin, row * kHeadDim, l8);
    Raw16 raw[kQHeads / 4];
#pragma unroll
    for (int k = 0; k < kQHeads / 4; ++k)
      if (h0 + 4 * k < p.Nq) raw[k] = load_raw<BF16>(p.qkv, src + 4 * k * kHeadDim, l8);
#pragma unroll
    for (int k = 0; k < kQHeads / 4; ++k) {
      if (h0 + 4 * k >= p.Nq) break;
      Row16 r = widen<BF16>(raw[k]);
      if (p.gamma_q != nullptr) norm_row<BF16>(&r, p.gamma_q, p.eps, l8, mask);
      rope_row<BF16>(&r, c, s);
      uint4* dst = reinterpret_cast<uint4*>(static_cast<typename H::T*>(p.q_out) +
                                            (row * p.Nq + h0 + 4 * k) * kHeadDim);
      dst[l8] = make_uint4(H::pack(r.a[0], r.a[1]), H::pack(r.a[2], r.a[3]),
                           H::pack(r.a[4], r.a[5]), H::pack(r.a[6], r.a[7]));
      dst[8 + l8] = make_uint4(H::pack(r.b[0], r.b[1]), H::pack(r.b[2], r.b[3]),
                               H::pack(r.b[4], r.b[5]), H::pack(r.b[6], r.b[7]));
    }
    return;
  }

  // ---- a unit: (sequence b, its page_slot-th touched page, head, k or v)
  const int64_t unit = UW == 1 ? static_cast<int64_t>(blockIdx.x) * kWarps + warp
                               : static_cast<int64_t>(blockIdx.x);
  const int heads2 = 2 * p.pg.Nk;
  const int hv = static_cast<int>(unit % heads2);
  const int64_t bp = unit / heads2;
  const int slot = static_cast<int>(bp % pages_per_seq);
  const int64_t b = bp / pages_per_seq;
  if (b >= p.rag.B) return;                              // whole warps (UW = 1) or whole blocks
  const bool is_v = hv >= p.pg.Nk;
  const int h = is_v ? hv - p.pg.Nk : hv;
  const SeqRows s = seq_rows(p.rag, static_cast<int>(b));
  const int tid = UW == 1 ? lane : threadIdx.x;
  if (s.bad && tid == 0 && slot == 0 && hv == 0) atomicOr(p.err, kErrIndexRange);
  const int bs = p.pg.block_size;
  const int blk = s.ctx / bs + slot;
  const int pos0 = slot == 0 ? s.ctx : blk * bs;         // first new position in the page
  int pos1 = s.ctx + s.len;
  if (pos0 >= pos1) return;
  if (pos1 > blk * bs + bs) pos1 = blk * bs + bs;
  bool bad = false;
  const int64_t page = page_of(p.pg, static_cast<int>(b), blk, &bad);
  if (bad && tid == 0 && hv == 0) atomicOr(p.err, kErrIndexRange);
  if (page < 0) return;
  const int r0 = pos0 - blk * bs, r1 = pos1 - blk * bs;  // rows of the page
  const int64_t tok0 = s.row0 + (pos0 - s.ctx);
  const int first = (UW == 1 ? 0 : warp * 4) + sub;
  constexpr int kStep = UW * 4;

  // A warp that owns its unit keeps the first row; the others are worked out twice (their second
  // reading comes from the L2).
  const int n = r1 - r0;
  const int again = UW == 1 ? first + kStep : first;
  Row16 own{};
  float m = 0.f;
  if (UW == 1 && first < n) {
    own = value_of<BF16>(p, load_value<BF16>(p, tok0 + first, h, is_v, l8), is_v, l8, mask);
    m = row_amax(own);
  }
  for (int i = again; i < n; i += kStep)
    m = fmaxf(m, row_amax(value_of<BF16>(p, load_value<BF16>(p, tok0 + i, h, is_v, l8), is_v, l8, mask)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float* scale = (is_v ? p.pg.v_scale : p.pg.k_scale) + page * p.pg.Nk + h;
  const float held = *scale;                             // read by every thread before the barrier
  if (UW > 1) {
    if (lane == 0) wmax[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < UW; ++w) m = fmaxf(m, wmax[w]);
  }
  const float old = r0 > 0 ? held : 0.f;
  const float sc = fmaxf(old, __fmul_rn(m, static_cast<float>(1.0 / 127.0)));
  const float inv = sc > 0.f ? __frcp_rn(sc) : 0.f;
  int8_t* codes = (is_v ? p.pg.v : p.pg.k) + (page * bs * p.pg.Nk + h) * kHeadDim;
  const int64_t pitch = static_cast<int64_t>(p.pg.Nk) * kHeadDim;
  __syncwarp();
  if (tid == 0) *scale = sc;
  if (r0 > 0 && sc > old) {                              // earlier codes to the grown scale
    const float ratio = __fdiv_rn(old, sc);
    for (int i = first; i < r0; i += kStep) {
      uint4* row = reinterpret_cast<uint4*>(codes + i * pitch) + l8;
      uint4 w = *row;
      const int8_t* c = reinterpret_cast<const int8_t*>(&w);
      float x[8], y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = static_cast<float>(c[e]);
        y[e] = static_cast<float>(c[8 + e]);
      }
      const uint2 lo = codes8(x, ratio), hi = codes8(y, ratio);
      *row = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
  }
  auto put = [&](int i, const Row16& r) {
    uint2* row = reinterpret_cast<uint2*>(codes + (r0 + i) * pitch);
    row[l8] = codes8(r.a, inv);
    row[8 + l8] = codes8(r.b, inv);
  };
  if (UW == 1 && first < n) put(first, own);
  for (int i = again; i < n; i += kStep)
    put(i, value_of<BF16>(p, load_value<BF16>(p, tok0 + i, h, is_v, l8), is_v, l8, mask));
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t stream) {
  const int bs = p.pg.block_size;
  // pages that max_new tokens can touch, starting anywhere in a page
  const int pages = bs > 0 ? (p.rag.max_new + bs - 2) / bs + 1 : 0;
  const int rows = p.rag.max_new < bs ? p.rag.max_new : bs;
  const bool few = rows <= 16;
  const int64_t units = static_cast<int64_t>(p.rag.B) * pages * 2 * p.pg.Nk;
  const int64_t ub = few ? (units + kWarps - 1) / kWarps : units;
  const int64_t qwarps = p.rag.T * ((p.Nq + kQHeads - 1) / kQHeads);
  const int64_t qb = (qwarps + kWarps - 1) / kWarps;
  if (ub + qb > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (ub + qb == 0) return cudaSuccess;
  auto kern = p.bf16 ? (few ? kv_append_kernel<true, 1> : kv_append_kernel<true, kWarps>)
                     : (few ? kv_append_kernel<false, 1> : kv_append_kernel<false, kWarps>);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ub + qb));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p, pages, ub);
}

}  // namespace mlap
