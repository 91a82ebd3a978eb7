// Chunk attention over a cache with 8-bit history on the tcgen05 tensor cores
// (sm_103a).
//
// Row r of a kv head is token r / G, query head r % G.  A unit is 256 rows of one
// (request, kv head): two tiles of 128, the M of an MMA.  It goes over the tokens
// it sees 128 at a time: first the history's tiles (two pages each), then those of
// the BF16 tokens, which are one line: sink, window, chunk.  All tiles of all
// units, in order, are one list that is cut into equal parts, one for each CTA
// (one per SM); units that a cut goes through leave partial records, which
// merge_kernel joins.
//
// S = Q·K^T and O += P·V are tcgen05.mma with fp32 accumulators in tensor memory
// (S of each row tile 128 columns, P over the first half of its S, O 128), Q, K, V
// in shared memory, 128-byte swizzled.  Warps:
//   0-7   softmax, four for each row tile, a thread per row
//   8-11  producers: history codes from global memory through registers to FP16
//         tiles (both code types are exact there), BF16 tokens by cp.async as they
//         are; K and V tiles alternate in a ring of five
//   12    the MMAs: S of the step after next is issued behind O of this one, so the
//         tensor cores work on one row tile while the other's softmax runs
// Steps (a row tile and a token tile) go to the two softmax groups in turn.  A unit
// of at most 128 rows has one row tile: then its token tiles go to the groups in
// turn, each with its own S and O, joined at the end.
//
// Scales.  The key scale of a block multiplies the logits of its 16 tokens, and the
// value scale enters the exponent: P = 2^(x + log2 s_V - M) in FP16, with M its
// own running maximum (less 8; raised when a row passes it by 6, so that O is seldom
// rescaled).  The row sum l is relative to the maximum m of the bare logits:
// Σ of a block's P times 2^(M - log2 s_V - m); a block whose scale is so small
// that P would underflow (2^-60 below what counts) is taken as larger, P then is
// 0 in FP16 all the same.  So P keeps 11 bits for whatever counts in O, whatever the
// scales.  BF16 tokens take the same road with s_V = 1 and P in BF16 (8 bits, as
// their values have): the operands of an MMA have one type, and BF16 values do not
// fit FP16's range.  Q is FP16 (times a power of two, exact) for the history and is
// loaded again as BF16 for the rest.
#include "oscar_kv8.cuh"
#include "oscar_tcgen05.cuh"

namespace oscar {

namespace {

using namespace tcgen05;

constexpr int ROWS = 256, TILE = 128;
constexpr int THREADS = 416, PROD0 = 256, MMA_WARP = 12;
constexpr int NBUF = 5, REGION = 16384, BUF = 2 * REGION;  // a tile: two regions of 64 channels, [128 rows][128 B]
constexpr int NINFO = 4, NALPHA = 3;
constexpr int OFF_Q = 0, OFF_BUF = 2 * BUF, OFF_BAR = OFF_BUF + NBUF * BUF;
enum {
  B_FULL = 0, B_EMPTY = B_FULL + NBUF, B_INFO = B_EMPTY + NBUF, B_S = B_INFO + NINFO, B_P = B_S + 2, B_O = B_P + 2,
  B_QFULL = B_O + 2, B_QEMPTY, B_DRAIN, NBARS
};
// A token tile's scales: x = S·a·(2^exponent of the row), b = log2 s_V.
struct Info {
  float2 cs[8];
  uint8_t valid[4], nanv[4];  // two bits a producer warp: blocks that count, blocks whose value scale is NaN
  uint32_t pad[2];
};
constexpr int OFF_INFO = OFF_BAR + 192, OFF_ALPHA = OFF_INFO + NINFO * (int)sizeof(Info);
constexpr int OFF_XCH = OFF_ALPHA + NALPHA * ROWS, OFF_MISC = OFF_XCH + TILE * 12;
struct Misc {
  uint32_t tmem;
  int abort, bad_v, n;
  long long lo, hi, at, W;
  int b, h, rt, pad;
};
constexpr int SMEM = OFF_MISC + (int)sizeof(Misc);
static_assert(NBARS * 8 <= 192 && sizeof(Info) == 80 && OFF_XCH % 4 == 0 && OFF_MISC % 8 == 0, "layout");
static_assert(SMEM <= 227 * 1024, "shared memory");
constexpr int S_COL = 0, O_COL = 256, TMEM_COLS = 512;
constexpr float C0 = INV_SQRT_D * LOG2E;
constexpr float NONE = -1e30f, LAZY = 6.f, HEAD = 8.f, FAR = 60.f;
// D fp32, M = N = 128; operand type 0: FP16, 1: BF16; bit 16: V is MN-major
constexpr uint32_t idesc(int type, int mn) {
  return (1u << 4) | ((uint32_t)type << 7) | ((uint32_t)type << 10) | ((uint32_t)mn << 16) | ((uint32_t)(TILE >> 3) << 17) |
         ((uint32_t)(TILE >> 4) << 24);
}

// ---------------------------------------------------------------- the work list
// Sum over r = 1 .. n of ceil((w + r c) / 128); c is 32, 64, 128 or 256.
__device__ __forceinline__ long long tiles_sum(int w, long long n, int c) {
  const int a = w + TILE - 1;
  if (c >= TILE) return n * (a / TILE) + (c / TILE) * (n * (n + 1) / 2);
  const int p = TILE / c, e = a % TILE / c;
  auto f = [&](long long x) {  // sum of floor(r / p) over r = 1 .. x
    const long long q = x / p;
    return p * (q * (q - 1) / 2) + q * (x % p + 1);
  };
  return n * (a / TILE) + f(n + e) - f(e);
}

struct Geo {
  int T, c, RT;  // tokens, tokens of a unit, units of a (request, kv head)
  __device__ explicit Geo(const Kv8Prefill& a) : T(a.T), c(ROWS / a.cv.G), RT((int)(((long long)a.T * a.cv.G + ROWS - 1) / ROWS)) {}
};

struct Lens {
  int L, H, nh, w;  // tokens, history; history tiles; BF16 tokens in the cache
  bool ok;
  __device__ void load(const CacheView& cv, int b) {
    const Kv8Req r = kv8_req(cv, b);
    L = r.L, H = r.H, ok = r.ok;
    nh = (H + TILE - 1) / TILE;
    w = L - H;
  }
  __device__ long long before(const Geo& g, int rt) const { return (long long)rt * nh + tiles_sum(w, rt, g.c); }
  __device__ long long per_head(const Geo& g) const {
    return (long long)g.RT * nh + tiles_sum(w, g.RT - 1, g.c) + ((long long)w + g.T + TILE - 1) / TILE;
  }
};

// The units of a CTA's part of the list, one after the other.
struct Walk {
  const Kv8Prefill& a;
  Geo geo;
  Lens r;
  long long lo, hi, at;  // the part; where the unit begins
  int b, h, rt;
  int n, i0, i1;   // the unit's tiles, and those of them in the part
  int t0, t1;      // its tokens
  bool two;        // two row tiles
  __device__ Walk(const Kv8Prefill& args, const Misc* m)
      : a(args), geo(args), lo(m->lo), hi(m->hi), at(m->at), b(m->b), h(m->h), rt(m->rt) {
    if (more()) {
      r.load(a.cv, b);
      unit();
    }
  }
  __device__ bool more() const { return at < hi; }
  __device__ void unit() {
    t0 = rt * geo.c;
    t1 = geo.T - t0 < geo.c ? geo.T : t0 + geo.c;
    two = (t1 - t0) * a.cv.G > TILE;
    n = r.nh + (r.w + t1 + TILE - 1) / TILE;
    i0 = at < lo ? (int)(lo - at) : 0;
    i1 = hi - at < n ? (int)(hi - at) : n;
  }
  __device__ void next() {
    at += n;
    if (++rt == geo.RT) {
      rt = 0;
      if (++h == a.cv.Hkv) {
        h = 0;
        ++b;
        if (more()) r.load(a.cv, b);
      }
    }
    if (more()) unit();
  }
  __device__ int hist_end() const { return i1 < r.nh ? i1 : r.nh; }  // tiles i0 .. here are history
  __device__ int line_begin() const { return i0 > r.nh ? i0 : r.nh; }
};

// What the merge needs to know of the unit that begins in a CTA's part and ends
// in a later one's.
struct Split {
  int b, h, rt, last;  // last: the CTA with its last tile, -1: no such unit
};

// By warp 0: the CTA's part.  pre: [B] in shared memory.
__device__ void plan(const Kv8Prefill& a, Misc* m, long long* pre, int lane) {
  const Geo g(a);
  const CacheView& cv = a.cv;
  long long W = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    long long x = 0;
    if (b < a.B) {
      Lens r;
      r.load(cv, b);
      if (!r.ok && blockIdx.x == 0) record_error(cv.err, OSCAR_ERR_STATE);
      x = r.per_head(g) * cv.Hkv;
    }
    long long inc = x;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const long long y = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += y;
    }
    if (b < a.B) pre[b] = W + inc - x;
    W += __shfl_sync(0xffffffffu, inc, 31);
  }
  __syncwarp();
  if (lane) return;
  Balanced bl;
  bl.W = W;
  bl.n = W < (long long)gridDim.x ? (int)W : (int)gridDim.x;
  m->W = W;
  m->n = bl.n;
  m->lo = m->hi = m->at = 0;
  if ((int)blockIdx.x >= bl.n) return;
  m->lo = balanced_lo(bl, blockIdx.x);
  m->hi = balanced_lo(bl, blockIdx.x + 1);
  const int b = balanced_request(pre, a.B, m->lo);
  Lens r;
  r.load(cv, b);
  const long long per = r.per_head(g), in = m->lo - pre[b];
  const int h = (int)(in / per);
  const long long x = in - h * per;
  int rt = 0, top = g.RT - 1;
  while (rt < top) {  // the last unit that begins at or before x
    const int mid = (rt + top + 1) >> 1;
    if (r.before(g, mid) <= x) rt = mid; else top = mid - 1;
  }
  m->b = b;
  m->h = h;
  m->rt = rt;
  m->at = pre[b] + h * per + r.before(g, rt);
}

// -------------------------------------------------------------------- producers
// Bytes (0, 1) and (2, 3) of w as FP16 pairs.
template <int TYPE>
__device__ __forceinline__ void halves(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (TYPE == OSCAR_KV8_E4M3) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {  // 1024 + (code + 128), less 1152
    const uint32_t u = w ^ 0x80808080u;
    asm("add.rn.f16x2 %0, %1, %2;\n" : "=r"(lo) : "r"(prmt(u, 0x64646464u, 0x4140)), "r"(0xE480E480u));
    asm("add.rn.f16x2 %0, %1, %2;\n" : "=r"(hi) : "r"(prmt(u, 0x64646464u, 0x4342)), "r"(0xE480E480u));
  }
}

__device__ __forceinline__ uint32_t saddr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void st16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// A lane's codes of one side of a block: chunk i ^ (K: gid & 1, V: 2 (gid & 1)) in
// x[i], which spreads a warp's 16-byte stores evenly over the banks.
struct Codes {
  uint4 x[4];
};
template <int SIDE>
__device__ __forceinline__ void load_codes(Codes& c, const uint8_t* block, bool on, int lane) {
  const uint4* src = (const uint4*)(block + SIDE * (KV8_BLK * D)) + lane;
  const int flip = SIDE == 0 ? (lane >> 2 & 1) : 2 * (lane >> 2 & 1);
#pragma unroll
  for (int i = 0; i < 4; ++i) c.x[i] = on ? __ldcg(src + 32 * (i ^ flip)) : make_uint4(0u, 0u, 0u, 0u);
}

// Block `blk` of a K tile (rows are tokens, K-major) and of a V tile (rows are
// tokens, MN-major): the same place for the same token and channel.
template <int TYPE>
__device__ __forceinline__ void store_k(uint32_t tile, const Codes& c, int blk, int lane) {
  const int gid = lane >> 2, tq = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo[4], hi[4];
    halves<TYPE>(c.x[i].x, lo[0], hi[0]);
    halves<TYPE>(c.x[i].y, lo[1], hi[1]);
    halves<TYPE>(c.x[i].z, lo[2], hi[2]);
    halves<TYPE>(c.x[i].w, lo[3], hi[3]);
    const int piece = (4 * ((i ^ gid) & 1) + tq) ^ gid;
    const uint32_t at = tile + (i >> 1) * REGION + (16 * blk + gid) * 128 + piece * 16;
    st16(at, lo[0], lo[1], lo[2], lo[3]);
    st16(at + 8 * 128, hi[0], hi[1], hi[2], hi[3]);
  }
}
template <int TYPE>
__device__ __forceinline__ void store_v(uint32_t tile, const Codes& c, int blk, int lane) {
  const int gid = lane >> 2, tq = lane & 3;
#pragma unroll
  for (int s = 0; s < 2; ++s) {  // channels 16 gid + 8 (s ^ gid & 1) .. + 7
    uint32_t o[2][2][4];         // token 8h + 2tq + l
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          halves<TYPE>(prmt(((const uint32_t*)&c.x[2 * s + i])[2 * e + h], 0, 0x3120), o[h][0][2 * i + e], o[h][1][2 * i + e]);
    const int piece = 2 * (gid & 3) + (s ^ (gid & 1));
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int l = 0; l < 2; ++l) {
        const int t = 2 * tq + l;
        st16(tile + (gid >> 2) * REGION + (16 * blk + 8 * h + t) * 128 + ((piece ^ t) * 16), o[h][l][0], o[h][l][1], o[h][l][2],
             o[h][l][3]);
      }
  }
}

__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(to), "l"(from), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t not_finite2(uint32_t w) {  // of either half
  return (uint32_t)((w & 0x7f80u) == 0x7f80u) | (uint32_t)((w & 0x7f800000u) == 0x7f800000u);
}

template <int TYPE>
struct Producer {
  const Kv8Prefill& a;
  uint8_t* smem;
  uint64_t* bars;
  Misc* misc;
  int t, wp, lane;  // thread of 128, warp of 4
  bool ok = true;
  int gt = 0, qn = 0;  // token tiles, loads of Q
  // Copies under way whose barrier has not been told: at most two.  cut: tokens
  // from, to of a V tile whose values are zeroed where they are not finite.
  struct Pending {
    int bar, buf, from, to;
  } pend[2];
  int npend = 0;

  __device__ Producer(const Kv8Prefill& args, uint8_t* s, int tid)
      : a(args), smem(s), bars((uint64_t*)(s + OFF_BAR)), misc((Misc*)(s + OFF_MISC)), t(tid - PROD0), wp((tid - PROD0) >> 5), lane(tid & 31) {}

  __device__ bool wait(int bar, int phase) {
    if (ok) ok = __all_sync(0xffffffffu, wait_bar(&bars[bar], phase & 1, &misc->abort, a.wait_polls));
    return ok;
  }
  __device__ bool wait_empty(int item) { return item < NBUF ? ok : wait(B_EMPTY + item % NBUF, item / NBUF - 1); }

  __device__ void tell(const Pending& p) {
    if (p.from < p.to) {  // this thread's own pieces
#pragma unroll 1
      for (int i = 0; i < 16; ++i) {
        const int tok = 8 * i + (t >> 4), ch = t & 15;
        uint4* x = (uint4*)(smem + OFF_BUF + p.buf * BUF + (ch >> 3) * REGION + tok * 128 + (((ch & 7) ^ (tok & 7)) << 4));
        if (tok < p.from || tok >= p.to) continue;
        uint32_t w[4] = {x->x, x->y, x->z, x->w};
        uint32_t bad = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bad |= not_finite2(w[j]);
          if ((w[j] & 0x7f80u) == 0x7f80u) w[j] &= 0xffff0000u;
          if ((w[j] & 0x7f800000u) == 0x7f800000u) w[j] &= 0x0000ffffu;
        }
        if (bad) {
          *x = make_uint4(w[0], w[1], w[2], w[3]);
          *(volatile int*)&misc->bad_v = 1;
        }
      }
    }
    fence_proxy_async();
    arrive(&bars[p.bar]);
  }
  __device__ void push(int bar, int buf, int from, int to) {
    copies_commit();
    if (npend == 2) {
      copies_wait<2>();
      tell(pend[0]);
      pend[0] = pend[1];
      npend = 1;
    }
    const Pending p = {bar, buf, from, to};
    if (npend == 0) pend[0] = p; else pend[1] = p;
    ++npend;
  }
  __device__ void flush() {
    copies_wait<0>();
    if (npend > 0) tell(pend[0]);
    if (npend > 1) tell(pend[1]);
    npend = 0;
  }

  __device__ void info(float2 cs, int valid, int nanv) {
    Info* f = (Info*)(smem + OFF_INFO) + (gt & (NINFO - 1));
    if (lane < 2) f->cs[2 * wp + lane] = cs;
    if (lane == 0) {
      f->valid[wp] = (uint8_t)valid;
      f->nanv[wp] = (uint8_t)nanv;
    }
    __syncwarp();
    if (lane == 0) arrive(&bars[B_INFO + (gt & (NINFO - 1))]);
  }

  // Rows of the unit, 16 lanes a row: token and head of row i, 16-byte piece t & 15.
  __device__ const uint4* q_piece(const Walk& u, int row, bool& on) const {
    const int G = a.cv.G, tok = u.t0 + row / G;
    on = tok < u.t1;
    return (const uint4*)(a.q + (((size_t)u.b * u.geo.T + (on ? tok : u.t0)) * a.cv.Hq + u.h * G + (on ? row % G : 0)) * D) + (t & 15);
  }
  __device__ uint32_t q_place(int row) const {
    const int ch = t & 15;
    return saddr(smem + OFF_Q) + (row >> 7) * BUF + (ch >> 3) * REGION + (row & 127) * 128 + (((ch & 7) ^ (row & 7)) << 4);
  }

  // Q in FP16, each row times the power of two that takes its largest finite value to
  // [2^14, 2^15) (not beyond 2^125): what is lost lies 2^38 below it.
  __device__ void load_q16(const Walk& u) {
    if (qn > 0 && !wait(B_QEMPTY, qn - 1)) return;
    int8_t* al = (int8_t*)(smem + OFF_ALPHA) + qn % NALPHA * ROWS;
    const int rows = u.two ? ROWS : TILE;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 32) {
      uint4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        bool on;
        const uint4* p = q_piece(u, r0 + 8 * i + (t >> 4), on);
        x[i] = on ? *p : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = r0 + 8 * i + (t >> 4);
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t mx = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = w[j] & 0x7fffu, hi = w[j] >> 16 & 0x7fffu;
          mx = max(mx, lo < 0x7f80u ? lo : 0u);
          mx = max(mx, hi < 0x7f80u ? hi : 0u);
        }
#pragma unroll
        for (int d = 1; d < 16; d *= 2) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const int e = max((int)(mx >> 7), 16);
        const float f = pow2i(141 - e);
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          asm("cvt.rn.f16x2.f32 %0, %1, %2;\n"
              : "=r"(o[j])
              : "f"(__uint_as_float(w[j] & 0xffff0000u) * f), "f"(__uint_as_float(w[j] << 16) * f));
        st16(q_place(row), o[0], o[1], o[2], o[3]);
        if ((t & 15) == 0) al[row] = (int8_t)(e - 141);
      }
    }
    ++qn;
    fence_proxy_async();
    arrive(&bars[B_QFULL]);
  }

  // The page of tile `i` that this warp's blocks are in: -1 if none counts.
  __device__ int page_of(const Walk& u, int i) const {
    const int pg = 2 * i + (wp >> 1);
    if (i >= u.hist_end() || pg * PAGE >= u.r.H) return -1;
    const int id = a.cv.page_table[(size_t)u.b * a.cv.max_pages_per_req + pg];
    if (id >= 0 && id < a.cv.num_pages) return id;
    if (lane == 0 && !(wp & 1)) record_error(a.cv.err, id < 0 ? OSCAR_ERR_NO_PAGE : OSCAR_ERR_RANGE);
    return -1;
  }

  __device__ void history(const Walk& u) {
    const int end = u.hist_end(), sub = 2 * wp % KV8_PAGE_BLOCKS;
    Codes k[2], v[2];
    float2 sc = make_float2(0.f, 0.f);
    int now = page_of(u, u.i0), next = page_of(u, u.i0 + 1);
    int valid = 0;
    auto on = [&](int i, int pid, int j) { return pid >= 0 && (8 * i + 2 * wp + j) * KV8_BLK < u.r.H; };
    auto load_k = [&](int i, int pid) {
      const uint8_t* base = kv8_head(a.cv, pid < 0 ? 0 : pid, u.h);
      valid = (int)on(i, pid, 0) + 2 * (int)on(i, pid, 1);
#pragma unroll
      for (int j = 0; j < 2; ++j) load_codes<0>(k[j], base + (sub + j) * KV8_BLOCK_BYTES, valid >> j & 1, lane);
      if (lane < 2 && (valid >> lane & 1)) sc = __ldcg((const float2*)(base + KV8_OFF_SCALES) + sub + lane);
    };
    auto load_v = [&](int i, int pid) {
      const uint8_t* base = kv8_head(a.cv, pid < 0 ? 0 : pid, u.h);
#pragma unroll
      for (int j = 0; j < 2; ++j) load_codes<1>(v[j], base + (sub + j) * KV8_BLOCK_BYTES, on(i, pid, j), lane);
    };
    load_k(u.i0, now);
    load_v(u.i0, now);
    load_q16(u);
    for (int i = u.i0; i < end && ok; ++i, ++gt) {
      const int after = page_of(u, i + 2);
      const uint32_t kb = 2 * gt % NBUF, vb = (2 * gt + 1) % NBUF;
      if (!wait_empty(2 * gt)) return;
      {
        const bool bad = lane < 2 && (valid >> lane & 1) && sc.y != sc.y;
        const uint32_t nanv = __ballot_sync(0xffffffffu, bad);
        float lsv = bad || !(lane < 2 && (valid >> lane & 1)) ? 0.f : log2f(sc.y);
        info(make_float2(sc.x * C0, lsv), valid, (int)nanv);
      }
      const uint32_t kt = saddr(smem + OFF_BUF) + kb * BUF, vt = saddr(smem + OFF_BUF) + vb * BUF;
#pragma unroll
      for (int j = 0; j < 2; ++j) store_k<TYPE>(kt, k[j], 2 * wp + j, lane);
      fence_proxy_async();
      arrive(&bars[B_FULL + kb]);
      load_k(i + 1, next);
      if (!wait_empty(2 * gt + 1)) return;
#pragma unroll
      for (int j = 0; j < 2; ++j) store_v<TYPE>(vt, v[j], 2 * wp + j, lane);
      fence_proxy_async();
      arrive(&bars[B_FULL + vb]);
      load_v(i + 1, next);
      next = after;
    }
  }

  // The unit's tiles of BF16 tokens: token s of the line is in the sink, in the window
  // (which begins at ring slot H mod 256) or in the chunk.
  __device__ void line(const Walk& u) {
    const CacheView& cv = a.cv;
    if (qn > 0 && !wait(B_QEMPTY, qn - 1)) return;
    const int rows = u.two ? ROWS : TILE;
#pragma unroll 4
    for (int row = t >> 4; row < rows; row += 8) {
      bool on;
      const uint4* p = q_piece(u, row, on);
      copy16(q_place(row), p, on);
    }
    ++qn;
    push(B_QFULL, 0, 0, 0);
    const size_t head = (size_t)u.b * cv.Hkv + u.h;
    const int nsink = u.r.L < SINK ? u.r.L : SINK, all = u.r.w + u.t1;
    for (int i = u.line_begin(); i < u.i1 && ok; ++i, ++gt) {
      const int s0 = (i - u.r.nh) * TILE;
#pragma unroll 1
      for (int side = 0; side < 2; ++side) {
        const int item = 2 * gt + side, buf = item % NBUF;
        if (!wait_empty(item)) return;
        if (side == 0) info(make_float2(C0, 0.f), 3, 0);
        const __nv_bfloat16* sink = (side ? cv.sink_v : cv.sink_k) + head * SINK * D;
        const __nv_bfloat16* ring = (side ? cv.ring_v : cv.ring_k) + head * RECENT * D;
        const __nv_bfloat16* fresh = (side ? a.v : a.k) + ((size_t)u.b * u.geo.T * cv.Hkv + u.h) * D;
        const int ch = t & 15;
        const uint32_t to = saddr(smem + OFF_BUF) + buf * BUF + (ch >> 3) * REGION;
#pragma unroll 4
        for (int j = 0; j < 16; ++j) {
          const int tok = 8 * j + (t >> 4), s = s0 + tok;
          const bool on = s < all;
          const __nv_bfloat16* p = s < nsink   ? sink + (size_t)s * D
                                   : s < u.r.w ? ring + (size_t)((u.r.H + s - nsink) & (RECENT - 1)) * D
                                               : fresh + (size_t)(on ? s - u.r.w : 0) * cv.Hkv * D;
          copy16(to + tok * 128 + (((ch & 7) ^ (tok & 7)) << 4), p + 8 * ch, on);
        }
        // tokens that only some of the unit's rows see: chunk tokens behind its first
        const int from = u.r.w + u.t0 + 1 - s0, cut_to = all - s0 < TILE ? all - s0 : TILE;
        push(B_FULL + buf, buf, side ? (from > 0 ? from : 0) : 0, side ? cut_to : 0);
      }
    }
    flush();
  }

  __device__ void run() {
    Walk u(a, misc);
    for (; u.more() && ok; u.next()) {
      if (u.i0 < u.hist_end()) history(u);
      if (ok && u.line_begin() < u.i1) line(u);
    }
    copies_wait<0>();
  }
};

// -------------------------------------------------------------------- MMA issue
struct Steps {
  Walk u;
  int tile, half, g, gt;
  __device__ Steps(const Kv8Prefill& a, const Misc* m) : u(a, m), tile(u.more() ? u.i0 : 0), half(0), g(0), gt(0) {}
  __device__ bool more() const { return u.more(); }
  __device__ bool hist() const { return tile < u.r.nh; }
  __device__ void advance() {
    ++g;
    if (u.two && !half) {
      half = 1;
      return;
    }
    half = 0;
    ++gt;
    if (++tile == u.i1) {
      u.next();
      if (u.more()) tile = u.i0;
    }
  }
};

__device__ void issue(const Kv8Prefill& a, uint8_t* smem) {
  uint64_t* bars = (uint64_t*)(smem + OFF_BAR);
  Misc* misc = (Misc*)(smem + OFF_MISC);
  const uint32_t tmem = misc->tmem, qbase = saddr(smem + OFF_Q), bbase = saddr(smem + OFF_BUF);
  Steps s(a, misc), p(a, misc);
  bool new_q = true, started[2] = {false, false};
  int qn = 0, np[2] = {0, 0};
  auto wait = [&](int bar, int phase) { return wait_bar(&bars[bar], phase & 1, &misc->abort, a.wait_polls); };
  auto scores = [&]() -> bool {
    const bool hist = s.hist();
    if (new_q && !wait(B_QFULL, qn++)) return false;
    const int item = 2 * s.gt, buf = item % NBUF, w = s.g & 1;
    if (!s.half && !wait(B_FULL + buf, item / NBUF)) return false;
    fence_after();
    const uint32_t q = qbase + (s.u.two ? w : 0) * BUF, k = bbase + buf * BUF, id = idesc(hist ? 0 : 1, 0);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      const uint32_t off = (ks >> 2) * REGION + (ks & 3) * 32;
      mma_ss(tmem + S_COL + TILE * w, sdesc(q + off), sdesc(k + off), id, ks > 0);
    }
    commit(&bars[B_S + w]);
    const long long at = s.u.at;
    const int gt = s.gt;
    s.advance();
    if (s.gt != gt) commit(&bars[B_EMPTY + buf]);
    new_q = !s.more() || s.u.at != at || s.hist() != hist;
    if (new_q) commit(&bars[B_QEMPTY]);
    return true;
  };
  auto values = [&]() -> bool {
    const int w = p.g & 1, item = 2 * p.gt + 1, buf = item % NBUF;
    if (!wait(B_P + w, np[w]++)) return false;
    if (!p.half && !wait(B_FULL + buf, item / NBUF)) return false;
    fence_after();
    const uint32_t v = bbase + buf * BUF, id = idesc(p.hist() ? 0 : 1, 1);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
      mma_ts(tmem + O_COL + TILE * w, tmem + S_COL + TILE * w + 8 * kk, sdesc_mn(v + kk * 2048, REGION), id, started[w] || kk > 0);
    started[w] = true;
    const long long at = p.u.at;
    const int gt = p.gt;
    p.advance();
    if (p.gt != gt) commit(&bars[B_EMPTY + buf]);
    if (!p.more() || p.u.at != at) {
      for (int i = 0; i < 2; ++i) {
        if (started[i]) commit(&bars[B_O + i]);
        started[i] = false;
      }
    }
    return true;
  };
  bool ok = true;
  for (int i = 0; i < 2; ++i)
    if (ok && s.more()) ok = scores();
  while (ok && p.more()) {
    ok = values();
    if (ok && s.more()) ok = scores();
  }
  // all that was issued has ended before the tensor memory is given back
  commit(&bars[B_DRAIN]);
  mbar_wait(&bars[B_DRAIN], 0);
}

// ---------------------------------------------------------------------- softmax
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&v)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(at),
               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
               "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
               : "memory");
}

// A row's running state.
struct Row {
  float m, l, M;
};

// Tokens of a tile that a row takes: `seen` first ones, and of those the blocks in `valid`.
// P of the tile to tensor memory, sums into the state.  EVERY: all of them.
template <bool F16, bool EVERY>
__device__ __forceinline__ void weigh(Row& st, uint32_t sa, uint32_t oa, const Info* f, float al, int seen, uint32_t valid,
                                      uint32_t nanv, bool first) {
  float cb[8], mb[8];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32];
    tmem_ld32(sa + 32 * c, r);
    tmem_ld_wait_regs(r);
#pragma unroll
    for (int hb = 0; hb < 2; ++hb) {
      const int b = 2 * c + hb;
      float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        const float x = __uint_as_float(r[16 * hb + j]), y = __uint_as_float(r[16 * hb + j + 1]);
        m0 = fmaxf(m0, EVERY || 16 * b + j < seen ? x : -INFINITY);
        m1 = fmaxf(m1, EVERY || 16 * b + j + 1 < seen ? y : -INFINITY);
      }
      mb[b] = EVERY || (valid >> b & 1) ? fmaxf(m0, m1) : -INFINITY;
    }
  }
  float mx = NONE, tx = NONE;
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const float2 cs = f->cs[b];
    cb[b] = cs.x * al;
    const float x = mb[b] * cb[b];
    mx = fmaxf(mx, x);
    tx = fmaxf(tx, x + cs.y);
  }
  const float mn = fmaxf(st.m, mx);
  st.l *= ex2(st.m - mn);
  st.m = mn;
  if (first) {
    st.M = tx - HEAD;
  } else if (__any_sync(0xffffffffu, tx > st.M + (HEAD + LAZY))) {
    const float Mn = fmaxf(st.M, tx - HEAD), g = ex2(st.M - Mn);
    st.M = Mn;
    // S of this step is complete, so is every MMA issued before it: O has all steps before
#pragma unroll 1
    for (int c = 0; c < TILE; c += 32) {
      uint32_t v[32];
      tmem_ld32(oa + c, v);
      tmem_ld_wait_regs(v);
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * g);
      tmem_st32(oa + c, v);
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32], o[16];
    tmem_ld32(sa + 32 * c, r);
    tmem_ld_wait_regs(r);
#pragma unroll
    for (int hb = 0; hb < 2; ++hb) {
      const int b = 2 * c + hb;
      const float shift = max_nan(f->cs[b].y - st.M, -st.m - FAR);
      float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        float x = ex2(fmaf(__uint_as_float(r[16 * hb + j]), cb[b], shift));
        float y = ex2(fmaf(__uint_as_float(r[16 * hb + j + 1]), cb[b], shift));
        if (!EVERY) {
          if (!(valid >> b & 1) || 16 * b + j >= seen) x = 0.f;
          if (!(valid >> b & 1) || 16 * b + j + 1 >= seen) y = 0.f;
        }
        sum0 += x;
        sum1 += y;
        if (!EVERY && (nanv >> b & 1)) x = y = NAN;
        o[8 * hb + j / 2] = pack2<F16>(x, y);
      }
      st.l = fmaf(sum0 + sum1, ex2(-shift - st.m), st.l);
    }
    tmem_st16(sa + 16 * c, o);
  }
  tmem_st_wait();
}

// Adds the values that are not finite of the chunk tokens j0 .. j1 - 1 to a row's channels c0 .. c0 + 31
// (they were left out of the product: other rows do not see them).
__device__ __noinline__ void add_bad(const Kv8Prefill& a, int b, int h, int j0, int j1, int c0, float* o) {
  for (int j = j0; j < j1; ++j) {
    const __nv_bfloat16* v = a.v + (((size_t)b * a.T + j) * a.cv.Hkv + h) * D + c0;
    for (int c = 0; c < 32; ++c) {
      const float x = __bfloat162float(v[c]);
      if (!(fabsf(x) <= 3.4e38f)) o[c] += x;
    }
  }
}

// The rows of a unit, or (part) their record.  oa: this group's O; other: the
// second group's, to be joined (its factor g1), or 0.
__device__ __forceinline__ void write_row(const Kv8Prefill& a, const Walk& u, const Row& st, uint32_t oa, float g0, uint32_t other,
                                          float g1, int row, float* rec, bool bad_v, bool ok) {
  const int G = a.cv.G, tok = u.t0 + row / G;
  const bool on = tok < u.t1;
  const size_t at = ((size_t)u.b * u.geo.T + (on ? tok : u.t0)) * a.cv.Hq + u.h * G + row % G;
  const float lg = log2f(st.l);
  float f = rec ? 1.f : st.l == 0.f ? 0.f : ex2(st.M - st.m - lg);
  if (!ok) f = NAN;
  int j0 = 0, j1 = 0;
  if (bad_v) {
    const int s0 = (u.line_begin() - u.r.nh) * TILE - u.r.w, s1 = (u.i1 - u.r.nh) * TILE - u.r.w;
    j0 = max(u.t0 + 1, s0);
    j1 = min(tok + 1, s1);
  }
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    float o[32];
    {
      uint32_t v[32];
      if (g0 != 0.f) {
        tmem_ld32(oa + c, v);
        tmem_ld_wait_regs(v);
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = g0 != 0.f ? __uint_as_float(v[j]) * g0 : 0.f;
    }
    if (other) {
      uint32_t v[32];
      tmem_ld32(other + c, v);
      tmem_ld_wait_regs(v);
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = fmaf(__uint_as_float(v[j]), g1, o[j]);
    }
    if (bad_v && on) add_bad(a, u.b, u.h, j0, j1, c, o);
    if (on && rec) {
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        *(float4*)(rec + PART_O + c + j) = make_float4(o[j] * f, o[j + 1] * f, o[j + 2] * f, o[j + 3] * f);
    } else if (on) {
#pragma unroll
      for (int j = 0; j < 32; j += 8) {
        uint4 x;
        x.x = pack2<false>(o[j] * f, o[j + 1] * f);
        x.y = pack2<false>(o[j + 2] * f, o[j + 3] * f);
        x.z = pack2<false>(o[j + 4] * f, o[j + 5] * f);
        x.w = pack2<false>(o[j + 6] * f, o[j + 7] * f);
        *(uint4*)(a.out + at * D + c + j) = x;
      }
    }
    __syncwarp();
  }
  if (on && rec) {
    rec[0] = st.m;
    rec[1] = ok ? st.l : NAN;
    rec[2] = st.M;
  } else if (on && a.lse) {
    a.lse[at] = ok ? (st.l == 0.f ? -INFINITY : (st.m + lg) * LN2) : NAN;
  }
  __syncwarp();
}

__device__ float* record(const Kv8Prefill& a, int cta, int slot, int row) {
  return a.part + ((size_t)(2 * cta + slot) * ROWS + row) * PART_STRIDE;
}

__device__ void softmax(const Kv8Prefill& a, uint8_t* smem, int tid) {
  uint64_t* bars = (uint64_t*)(smem + OFF_BAR);
  Misc* misc = (Misc*)(smem + OFF_MISC);
  const int warp = tid >> 5, wg = warp >> 2, row = tid & 127;
  const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16, tmem = misc->tmem + lanes;
  const uint32_t sa = tmem + S_COL + TILE * wg, oa = tmem + O_COL + TILE * wg;
  float* xch = (float*)(smem + OFF_XCH) + row * 3;
  auto wait = [&](int bar, int phase) {
    return (bool)__all_sync(0xffffffffu, wait_bar(&bars[bar], phase & 1, &misc->abort, a.wait_polls));
  };
  bool ok = true;
  int g = 0, gt = 0, ns = 0, no = 0, qn = 0;
  Split split = {0, 0, 0, -1};
  Walk u(a, misc);
  for (; u.more(); u.next()) {
    const int nt = u.i1 - u.i0, hist_end = u.hist_end();
    const int urow = (u.two ? TILE * wg : 0) + row, trow = u.t0 + urow / a.cv.G;
    Row st = {NONE, 0.f, NONE};
    float al = 0.f;
    int cnt = 0;
    for (int i = u.i0 + (u.two ? 0 : (wg - g) & 1); i < u.i1 && ok; i += u.two ? 1 : 2) {
      const int tile = gt + i - u.i0;
      ok = wait(B_INFO + (tile & (NINFO - 1)), tile / NINFO) && wait(B_S + wg, ns);
      if (!ok) break;
      ++ns;
      fence_after();
      const Info* f = (const Info*)(smem + OFF_INFO) + (tile & (NINFO - 1));
      if (i < u.r.nh) {
        if (cnt == 0) al = pow2i(((const int8_t*)(smem + OFF_ALPHA))[qn % NALPHA * ROWS + urow]);
        uint32_t valid = 0, nanv = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          valid |= (uint32_t)f->valid[j] << (2 * j);
          nanv |= (uint32_t)f->nanv[j] << (2 * j);
        }
        if (valid == 0xff && nanv == 0) weigh<true, true>(st, sa, oa, f, al, TILE, valid, nanv, cnt == 0);
        else weigh<true, false>(st, sa, oa, f, al, TILE, valid, nanv, cnt == 0);
      } else {
        const int seen = u.r.w + trow + 1 - (i - u.r.nh) * TILE;
        if (__all_sync(0xffffffffu, seen >= TILE)) weigh<false, true>(st, sa, oa, f, 1.f, TILE, 0xff, 0, cnt == 0);
        else weigh<false, false>(st, sa, oa, f, 1.f, seen, 0xff, 0, cnt == 0);
      }
      fence_before();
      __syncwarp();
      if ((tid & 31) == 0) arrive(&bars[B_P + wg]);
      ++cnt;
    }
    if (ok && cnt > 0) {
      ok = wait(B_O + wg, no);
      ++no;
      fence_after();
    }
    const bool begins = u.i0 == 0, ends = u.i1 == u.n;
    if (begins && !ends) {
      Balanced bl;
      bl.W = misc->W;
      bl.n = misc->n;
      split = {u.b, u.h, u.rt, balanced_owner(bl, u.at + u.n - 1)};
    }
    float* rec = begins && ends ? nullptr : record(a, blockIdx.x, begins ? 1 : 0, urow);
    const bool bad_v = *(volatile int*)&misc->bad_v != 0 && u.line_begin() < u.i1;
    if (u.two) {
      write_row(a, u, st, oa, 1.f, 0, 0.f, urow, rec, bad_v, ok);
    } else {
      if (wg == 1) {
        xch[0] = st.m;
        xch[1] = ok ? st.l : NAN;
        xch[2] = cnt > 0 ? st.M : -INFINITY;
      }
      fence_before();
      asm volatile("bar.sync 3, 256;\n" ::: "memory");
      fence_after();
      if (wg == 0) {
        const float m1 = xch[0], l1 = xch[1], M1 = xch[2];
        const bool one = M1 != -INFINITY;  // the other group had a tile
        Row j;
        j.m = fmaxf(st.m, m1);
        j.l = st.l * ex2(st.m - j.m) + l1 * ex2(m1 - j.m);
        j.M = cnt > 0 ? fmaxf(st.M, M1) : M1;
        write_row(a, u, j, oa, cnt > 0 ? ex2(st.M - j.M) : 0.f, one ? oa + TILE : 0, one ? ex2(M1 - j.M) : 0.f, urow, rec, bad_v, ok);
        fence_before();
      }
      asm volatile("bar.sync 3, 256;\n" ::: "memory");
    }
    gt += nt;
    g += u.two ? 2 * nt : nt;
    qn += (int)(u.i0 < hist_end) + (int)(u.line_begin() < u.i1);
  }
  if (tid == 0) a.splits[blockIdx.x] = make_int4(split.b, split.h, split.rt, split.last);
}

template <int TYPE>
__global__ void __launch_bounds__(THREADS, 1) attend_kernel(const __grid_constant__ Kv8Prefill a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = (uint64_t*)(smem + OFF_BAR);
  Misc* misc = (Misc*)(smem + OFF_MISC);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (saddr(smem) & 1023) {  // the swizzled tiles begin on 1024 bytes; there is no room to move them
    if (tid == 0) {
      a.splits[blockIdx.x] = make_int4(0, 0, 0, -1);
      record_error(a.cv.err, OSCAR_ERR_CUDA);
    }
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(&bars[B_FULL + i], 128);
      mbar_init(&bars[B_EMPTY + i], 1);
    }
    for (int i = 0; i < NINFO; ++i) mbar_init(&bars[B_INFO + i], 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[B_S + i], 1);
      mbar_init(&bars[B_P + i], 4);
      mbar_init(&bars[B_O + i], 1);
    }
    mbar_init(&bars[B_QFULL], 128);
    mbar_init(&bars[B_QEMPTY], 1);
    mbar_init(&bars[B_DRAIN], 1);
    misc->abort = misc->bad_v = 0;
  }
  if (warp == MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(saddr(&misc->tmem)), "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 0) plan(a, misc, (long long*)(smem + OFF_BUF), tid);
  fence_proxy_async();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = misc->tmem;
  if (warp == MMA_WARP) {
    if (tid % 32 == 0) issue(a, smem);
    __syncwarp();
  } else if (tid >= PROD0) {
    Producer<TYPE>(a, smem, tid).run();
  } else {
    softmax(a, smem, tid);
  }
  fence_before();
  __syncthreads();
  if (tid == 0 && misc->abort) record_error(a.cv.err, OSCAR_ERR_TIMEOUT);
  if (warp == MMA_WARP) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
  }
}

// Joins the records of the unit that begins in part blockIdx.x; a warp per row, a lane
// per four channels.
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Kv8Prefill a) {
  pdl_wait();
  pdl_launch_dependents();
  const int4 d = a.splits[blockIdx.x];
  if (d.w < 0) return;
  const int lane = threadIdx.x & 31, row = blockIdx.y * 8 + (threadIdx.x >> 5), G = a.cv.G;
  const int tok = d.z * (ROWS / G) + row / G;
  if (tok >= a.T) return;
  const int first = blockIdx.x, n = d.w - first + 1;
  float m = NONE, L = 0.f;
  for (int k = lane; k < n; k += 32) m = fmaxf(m, record(a, first + k, k == 0, row)[0]);
  for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
  for (int k = lane; k < n; k += 32) {
    const float* r = record(a, first + k, k == 0, row);
    L += r[1] * ex2(r[0] - m);
  }
  for (int s = 16; s; s >>= 1) L += __shfl_xor_sync(0xffffffffu, L, s);
  const float lg = log2f(L);
  float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = 0; k < n; ++k) {
    const float* r = record(a, first + k, k == 0, row);
    const float f = L == 0.f ? 0.f : ex2(r[2] - m - lg);
    const float4 x = *(const float4*)(r + PART_O + 4 * lane);
    o[0] = fmaf(x.x, f, o[0]);
    o[1] = fmaf(x.y, f, o[1]);
    o[2] = fmaf(x.z, f, o[2]);
    o[3] = fmaf(x.w, f, o[3]);
  }
  const size_t at = ((size_t)d.x * a.T + tok) * a.cv.Hq + d.y * G + row % G;
  *(uint2*)(a.out + at * D + 4 * lane) = make_uint2(pack2<false>(o[0], o[1]), pack2<false>(o[2], o[3]));
  if (lane == 0 && a.lse) a.lse[at] = L == 0.f ? -INFINITY : (m + lg) * LN2;
}

template <int TYPE>
cudaError_t launch_attend(const Kv8Prefill& a, cudaStream_t st) {
  static int limit[MAX_DEVICES];
  const cudaError_t e = raise_smem_limit(attend_kernel<TYPE>, limit, SMEM);
  return e != cudaSuccess ? e : launch_pdl(attend_kernel<TYPE>, dim3(a.grid), dim3(THREADS), SMEM, st, a);
}

}  // namespace

Kv8PrefillScratch kv8_prefill_scratch(int grid) {
  Kv8PrefillScratch s;
  s.off_part = ((size_t)grid * sizeof(int4) + 255) & ~(size_t)255;
  s.total = s.off_part + (size_t)grid * 2 * ROWS * PART_STRIDE * sizeof(float);
  return s;
}

cudaError_t launch_kv8_prefill(const Kv8Prefill& a, int type, cudaStream_t st, Profiler* prof) {
  prof_begin(prof, OSCAR_KERNEL_PREFILL_ATTN, st);
  cudaError_t e = type == OSCAR_KV8_E4M3 ? launch_attend<OSCAR_KV8_E4M3>(a, st) : launch_attend<OSCAR_KV8_INT8>(a, st);
  prof_end(prof, OSCAR_KERNEL_PREFILL_ATTN, st);
  if (e != cudaSuccess) return e;
  prof_begin(prof, OSCAR_KERNEL_PREFILL_MERGE, st);
  e = launch_pdl(join_kernel, dim3(a.grid, ROWS / 8), dim3(256), 0, st, a);
  prof_end(prof, OSCAR_KERNEL_PREFILL_MERGE, st);
  return e;
}

}  // namespace oscar
