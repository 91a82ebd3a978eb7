// Chunk attention over a cache with 8-bit history on the tcgen05 tensor cores
// (sm_103a).
//
// Row r of a kv head is token r / G, query head r % G.  A unit is 256 rows of one
// (request, kv head): two tiles of 128, the M of an MMA.  It goes over the tokens
// it sees 128 at a time: first the history's tiles (two pages each), then those of
// the BF16 tokens, which are one line: sink, window, chunk.  All tiles of all
// units, in order, are one list that is cut into equal parts, one for each CTA
// (one per SM); units that a cut goes through leave partial records, which
// join_kernel joins.
//
// S = Q·K^T and O += P·V are tcgen05.mma with fp32 accumulators in tensor memory
// (S of each row tile 128 columns, P over the first half of its S, O 128), Q, K, V
// in shared memory, 128-byte swizzled.  Warps:
//   0-7   softmax, four for each row tile, a thread per row
//   8-15  producers, four for keys and four for values: history codes from global
//         memory through registers to FP16 tiles (both code types are exact there),
//         BF16 tokens by cp.async as they are; K and V tiles alternate in a ring of five
//   18    goes ahead of them: what a tile is, its scales, pages into the L2
//   19    the MMAs: S of the step after next is issued behind O of this one, so the
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
// scales.  For BF16 tokens P is BF16 (8 bits, as their values have): the operands
// of an MMA have one type, and BF16 values do not fit FP16's range.  Their values
// are taken as they are and may be as large as fp32 goes, so P is kept small
// instead: M lies `room` above m, P then adds up to 1 or less over all tokens that a row can
// see, and O stays below the largest value.  (Nothing is lost to that: BF16 reaches
// 2^-126, a row's largest P is 2^-room, some 2^-23, or at least 2^-32 of that.  A unit with
// both kinds of token has its O taken to the new M once.)  Q is FP16 (times a power of
// two, exact) for the history and is loaded again as BF16 for the rest.
//
// What bounds it.  The MMAs of a step take 1024 cycles, the softmax some 1600 to 1900,
// and each waits for the other's barriers (a look at shared memory takes 250 to 300
// cycles while MMAs read their operands there: S = Q·K^T takes all of its bandwidth).
// Two row tiles in flight hide part of that, tensor memory has no place for a third.
// Measured (several GB300s, bf16 burst peak 1894 TFLOP/s): 2048 tokens over 100K, 32/8 heads,
// 2660 to 2820 us by the card, 1270 to 1200 TFLOP/s; 1024 over 50K 715 us; a prompt of 8191
// 550 us, 1000 TFLOP/s of the causal half; 64 tokens over 100K 114 us, 4 x 509 tokens over 0.3K
// to 9K 361 us.  Few rows: 16 requests with 5 tokens over 8K to 32K 181 us (3.7 TB/s; the FP16
// tiles are written to shared memory and read by MMAs of 128 rows, which with the waits
// takes most of its cycles), 5 tokens over 1K 17 us (two launches, the list, three
// dependent trips to memory, instructions that are not in the caches).
//
// One MMA warp, not one a row tile (prompt 631 -> 584 at the time, but 2048 tokens over 100K
// 3090 -> 3580).  Token tiles of 128, not 64: an MMA with N = 64 takes as long.
#include "oscar_kv8.cuh"
#include "oscar_tcgen05.cuh"

namespace oscar {

namespace {

using namespace tcgen05;

constexpr int ROWS = 256, TILE = 128;
constexpr int PROD = 256, SIDE = 128;  // producer threads: 128 for K, 128 for V
// Warps 16, 17 fill the last group up.  With few rows warps 0 and 4 have all of the softmax: the MMAs
// are issued on another quarter of the SM (16 requests with 5 tokens 189 -> 182 us).
constexpr int PROD0 = 256, ISSUE0 = 16, SCOUT_WARP = 18, MMA_WARP = 19, THREADS = 640;
// Registers a thread: 256·136 + 256·88 + 128·32 are the 640·96 of the launch.  (128 for the softmax and
// 96 for the producers: prompt 572 -> 616 us, 2048 tokens over 100K 2745 -> 2800.)
constexpr int REGS_SOFTMAX = 136, REGS_PROD = 88, REGS_MMA = 32;
constexpr int NBUF = 5, REGION = 16384, BUF = 2 * REGION;  // a tile: two regions of 64 channels, [128 rows][128 B]
constexpr int NINFO = 4, NALPHA = 3, NUNIT = 8;
constexpr int OFF_Q = 0, OFF_BUF = 2 * BUF, OFF_BAR = OFF_BUF + NBUF * BUF;
enum {
  B_FULL = 0, B_EMPTY = B_FULL + NBUF, B_INFO = B_EMPTY + NBUF, B_S = B_INFO + NINFO, B_P = B_S + 2, B_O = B_P + 4,
  B_QFULL = B_O + 2, B_QEMPTY, B_OTHER, B_TAKEN, B_DRAIN, NBARS
};
// A token tile's scales: x = S·a·(2^exponent of the row), b = log2 s_V.
struct Info {
  float2 cs[8];
  uint8_t marks[8];  // of the blocks: 1 it counts, 2 its value scale is NaN
  uint32_t flags, pad;
};
constexpr uint32_t ALL_COUNT = 0x01010101u;  // four marks
// What the MMA warp needs to know of a token tile.
enum { F_HIST = 1, F_TWO = 2, F_NEWQ = 4, F_ENDQ = 8, F_ENDU = 16 };
// A unit, as the softmax needs it (the scout follows the work list for it: its state does
// not fit into the registers of a softmax thread).
struct alignas(16) Unit {
  int tiles, hist;  // its tiles in this part, the first of them history
  int line;         // of the BF16 tokens in its first other tile, those that its first row sees
  int flags;        // U_TWO: two row tiles; U_BEGINS, U_ENDS: it does so in this part
  int b, h, t0, t1; // tokens t0 .. t1 - 1
  int c0, c1;       // chunk tokens in this part's tiles
  int pad[2];
};
enum { U_TWO = 1, U_BEGINS = 2, U_ENDS = 4 };
constexpr int OFF_INFO = OFF_BAR + 240, OFF_UNIT = OFF_INFO + NINFO * (int)sizeof(Info), OFF_ALPHA = OFF_UNIT + NUNIT * (int)sizeof(Unit);
constexpr int OFF_XCH = OFF_ALPHA + NALPHA * ROWS, OFF_MISC = OFF_XCH + TILE * 8;
struct Misc {
  uint32_t tmem;
  int abort, bad_v, tiles;  // tiles: in the part
  long long lo, hi, at;
  int b, h, rt, pad;
};
constexpr int SMEM = OFF_MISC + (int)sizeof(Misc);
static_assert(NBARS * 8 <= 240 && sizeof(Info) == 80 && sizeof(Unit) == 48 && OFF_UNIT % 16 == 0 && OFF_XCH % 8 == 0 && OFF_MISC % 8 == 0, "layout");
static_assert(SMEM <= 227 * 1024, "shared memory");
constexpr int S_COL = 0, O_COL = 256, TMEM_COLS = 512;
constexpr float C0 = INV_SQRT_D * LOG2E;
// From here on (base 2) a logit has a bit of fraction left in 32 bits, and what one rounding more or less, of the
// exponent, the maximum and M, adds up to would soon be more than FP16 has room for above P: the row is NaN.
constexpr float TOO_LARGE = 4194304.f;
constexpr float NONE = -3.402823466e38f, LAZY = 6.f, HEAD = 8.f, FAR = 60.f, SPARE = 32.f;
// D fp32, M = N = 128; operand type 0: FP16, 1: BF16; bit 16: V is MN-major
constexpr uint32_t idesc(int type, int mn) {
  return (1u << 4) | ((uint32_t)type << 7) | ((uint32_t)type << 10) | ((uint32_t)mn << 16) | ((uint32_t)(TILE >> 3) << 17) |
         ((uint32_t)(TILE >> 4) << 24);
}

extern __shared__ __align__(1024) uint8_t smem[];
__device__ __forceinline__ uint64_t* barrier(int i) { return (uint64_t*)(smem + OFF_BAR) + i; }
__device__ __forceinline__ Misc* the_misc() { return (Misc*)(smem + OFF_MISC); }

// ---------------------------------------------------------------- the work list
// (64-bit divisions take hundreds of cycles, and every CTA begins with these sums.)
__device__ __forceinline__ long long quotient(long long a, long long b) {  // a >= 0, b > 0
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}
// Sum over r = 1 .. n of ceil((w + r c) / 128), c = 2^lc one of 32, 64, 128, 256.
__device__ __forceinline__ long long tiles_sum(int w, long long n, int lc) {
  const int a = w + TILE - 1;
  if (lc >= 7) return n * (a >> 7) + ((n * (n + 1) / 2) << (lc - 7));
  const int lp = 7 - lc, e = (a & (TILE - 1)) >> lc;
  auto f = [&](long long x) {  // sum of floor(r / 2^lp) over r = 1 .. x
    const long long q = x >> lp;
    return (q * (q - 1) / 2 << lp) + q * ((x & ((1 << lp) - 1)) + 1);
  };
  return n * (a >> 7) + f(n + e) - f(e);
}
// Where part i of n begins in a list of W, and whose part place x is in.
__device__ __forceinline__ long long part_begin(long long W, int n, int i) { return quotient(i * W, n); }
__device__ __forceinline__ int part_of(long long W, int n, long long x) { return (int)(quotient((x + 1) * n + W - 1, W) - 1); }

// Loading Q and writing the rows takes a unit about as long as so many tiles.  (4 x 509 tokens
// over a history / prompt of 8191: with 2 367 / 564 us, 3 348 / 560, 4 346 / 570, 6 341 / 582.)
constexpr int UNIT_COST = 3;

struct Lens {
  int L, H;  // tokens, history
  bool ok;
  __device__ void load(const CacheView& cv, int b) {
    const Kv8Req r = kv8_req(cv, b);
    L = r.L, H = r.H, ok = r.ok;
  }
  // (Not kept: the producers have no register to spare.)
  __device__ int nh() const { return (H + TILE - 1) / TILE; }  // history tiles
  __device__ int w() const { return L - H; }                   // BF16 tokens in the cache
  // Places in the list: a unit has UNIT_COST empty ones and then its tiles.
  __device__ long long before(const Kv8Prefill& a, int rt) const { return (long long)rt * (UNIT_COST + nh()) + tiles_sum(w(), rt, 8 - a.lg); }
  __device__ long long per_head(const Kv8Prefill& a) const {
    return (long long)a.units * (UNIT_COST + nh()) + tiles_sum(w(), a.units - 1, 8 - a.lg) + ((long long)w() + a.T + TILE - 1) / TILE;
  }
};

// The units of a CTA's part of the list, one after the other.
struct Walk {
  const Kv8Prefill& a;
  Lens r;
  int at, len;     // where the unit begins, from the part's begin; the part's length
  int b, h, rt;
  int n, i0, i1;   // the unit's tiles, and those of them in the part
  __device__ Walk(const Kv8Prefill& args, const Misc* m)
      : a(args), at((int)(m->at - m->lo)), len((int)(m->hi - m->lo)), b(m->b), h(m->h), rt(m->rt) {
    if (more()) {
      r.load(a.cv, b);
      unit();
      if (i0 >= i1) next();
    }
  }
  __device__ bool more() const { return at < len; }
  __device__ int t0() const { return rt << (8 - a.lg); }  // its tokens t0 .. t1 - 1
  __device__ int t1() const { return min(t0() + (ROWS >> a.lg), a.T); }
  __device__ bool two() const { return ((t1() - t0()) << a.lg) > TILE; }  // two row tiles
  __device__ void unit() {
    n = r.nh() + (r.w() + t1() + TILE - 1) / TILE;
    const int first = at + UNIT_COST;
    i0 = max(-first, 0);
    i1 = min(len - first, n);
  }
  __device__ void next() {  // the next unit with a tile in the part
    do {
      at += UNIT_COST + n;
      if (++rt == a.units) {
        rt = 0;
        if (++h == a.cv.Hkv) {
          h = 0;
          ++b;
          if (more()) r.load(a.cv, b);
        }
      }
      if (more()) unit();
    } while (more() && i0 >= i1);
  }
  __device__ int hist_end() const { return min(i1, r.nh()); }  // tiles i0 .. here are history
  __device__ int line_begin() const { return max(i0, r.nh()); }
};

// By warp 0: the CTA's part, and (splits) the unit that begins in it and ends in a later
// one's: request, head, unit and the CTA with its last tile, -1 if there is none.
// pre: [B] in shared memory.
__device__ void plan(const Kv8Prefill& a, Misc* m, long long* pre, int lane) {
  const CacheView& cv = a.cv;
  long long W = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    long long x = 0;
    if (b < a.B) {
      Lens r;
      r.load(cv, b);
      if (!r.ok && blockIdx.x == 0) record_error(cv.err, OSCAR_ERR_STATE);
      x = r.per_head(a) * cv.Hkv;
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
  const int parts = W < (long long)gridDim.x ? (int)W : (int)gridDim.x;
  const bool any = (int)blockIdx.x < parts;
  const long long lo = any ? part_begin(W, parts, blockIdx.x) : 0, hi = any ? part_begin(W, parts, blockIdx.x + 1) : 0;
  if (lane == 0) {
    m->lo = lo;
    m->hi = hi;
    m->at = 0;
    m->tiles = 0;
    if (!any) a.splits[blockIdx.x] = make_int4(0, 0, 0, -1);
  }
  if (!any || lane > 1) return;
  // lane 0 finds the part's first unit, lane 1 its last
  const long long at = lane == 0 ? lo : hi - 1;
  const int b = balanced_request(pre, a.B, at);
  Lens r;
  r.load(cv, b);
  const long long per = r.per_head(a), in = at - pre[b];
  const int h = (int)quotient(in, per);
  const long long x = in - h * per;
  int rt = 0, top = a.units - 1;
  while (rt < top) {  // the last unit that begins at or before x
    const int mid = (rt + top + 1) >> 1;
    if (r.before(a, mid) <= x) rt = mid; else top = mid - 1;
  }
  const long long begin = pre[b] + h * per + r.before(a, rt);
  // tiles in front of the part, and in front of its end
  const long long in_unit = (lane == 0 ? lo : hi) - begin - UNIT_COST;
  const long long real = begin - UNIT_COST * (((long long)b * cv.Hkv + h) * a.units + rt) + (in_unit > 0 ? in_unit : 0);
  const long long real_hi = __shfl_sync(3u, real, 1);
  if (lane == 0) {
    m->tiles = (int)(real_hi - real);
    m->b = b;
    m->h = h;
    m->rt = rt;
    m->at = begin;
  } else {
    const int t1 = min((rt + 1) << (8 - a.lg), a.T);
    const long long first = begin + UNIT_COST, end = first + r.nh() + (r.w() + t1 + TILE - 1) / TILE;
    a.splits[blockIdx.x] = make_int4(b, h, rt, first >= lo && first < hi && end > hi ? part_of(W, parts, end - 1) : -1);
  }
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

// Where a row's 16-byte piece t & 15 stands in Q.
__device__ __forceinline__ uint32_t q_place(uint32_t q, int t, int row) {
  const int ch = t & 15;
  return q + (row >> 7) * BUF + (ch >> 3) * REGION + (row & 127) * 128 + (((ch & 7) ^ (row & 7)) << 4);
}

// Q, copied as it is, to FP16 in its place, by 256 threads with the pieces that each copied: a
// row times the power of two that takes its largest finite value to [2^14, 2^15) (not
// beyond 2^125).  What is lost lies 2^38 below it.  (Two or four rows at a time take registers
// from the loop behind it: 16 requests with 5 tokens 188 -> 195 to 213 us.)
__device__ __forceinline__ void convert_q(uint32_t q, int8_t* al, int t, int rows) {
#pragma unroll 1
  for (int row = t >> 4; row < rows; row += 16) {
    const uint32_t at = q_place(q, t, row);
    uint32_t w[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
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
    st16(at, o[0], o[1], o[2], o[3]);
    if ((t & 15) == 0) al[row] = (int8_t)(e - 141);
  }
}

// Whether a phase is over.
__device__ __forceinline__ bool passed(uint64_t* bar, uint32_t parity) {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(r)
               : "r"(saddr(bar)), "r"(parity)
               : "memory");
  return r != 0;
}

template <int TYPE>
struct Producer {
  const Kv8Prefill& a;
  int t, wp, lane, side;  // thread of 256, warp of its side's four; K: 0, V: 1
  bool ok = true;
  int gt = 0, qn = 0;  // token tiles, loads of Q
  // Copies under way whose barrier has not been told: at most two.  from, to: tokens of a V
  // tile whose values are zeroed where they are not finite.
  struct Pending {
    int bar, buf, from, to;
  };
  struct Copies {
    Pending p[2];
    int n = 0;
  };

  __device__ Producer(const Kv8Prefill& args, int tid)
      : a(args), t(tid - PROD0), wp(((tid - PROD0) >> 5) & 3), lane(tid & 31),
        side((int)__shfl_sync(0xffffffffu, (tid - PROD0) / SIDE, 0)) {}

  __device__ bool wait(int bar, int phase) {
    if (ok) ok = __all_sync(0xffffffffu, wait_bar(barrier(bar), phase & 1, &the_misc()->abort, a.wait_polls));
    return ok;
  }
  __device__ bool wait_empty(int item) { return item < NBUF ? ok : wait(B_EMPTY + item % NBUF, item / NBUF - 1); }
  // The MMAs that free a buffer may need copies that nobody has been told of: it does not
  // wait with any.
  __device__ bool wait_empty(int item, Copies& c) {
    if (c.n > 0 && item >= NBUF && !__all_sync(0xffffffffu, passed(barrier(B_EMPTY + item % NBUF), (item / NBUF - 1) & 1))) flush(c);
    return wait_empty(item);
  }

  // A full buffer is told by the 128 threads of its side and once more: K by the scout, with
  // what the tile is, V by its first thread.
  __device__ void told(int bar) {
    arrive(barrier(bar));
    if (t == SIDE && bar < B_FULL + NBUF) arrive(barrier(bar));
  }
  __device__ void tell(const Pending& p) {
    if (p.from < p.to) {  // this thread's own pieces
#pragma unroll 1
      for (int i = 0; i < 16; ++i) {
        const int tok = 8 * i + (t % SIDE >> 4), ch = t & 15;
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
          *(volatile int*)&the_misc()->bad_v = 1;
        }
      }
    }
    fence_proxy_async();
    told(p.bar);
  }
  __device__ void push(Copies& c, const Pending& p) {
    copies_commit();
    if (c.n == 2) {
      copies_wait<2>();
      tell(c.p[0]);
      c.p[0] = c.p[1];
      c.n = 1;
    }
    if (c.n == 0) c.p[0] = p; else c.p[1] = p;
    ++c.n;
  }
  __device__ void flush(Copies& c) {
    copies_wait<0>();
    if (c.n > 0) tell(c.p[0]);
    if (c.n > 1) tell(c.p[1]);
    c.n = 0;
  }

  // Rows of the unit, 16 lanes a row: token and head of row i, 16-byte piece t & 15.
  __device__ const uint4* q_piece(const Walk& u, int row, bool& on) const {
    const int G = a.cv.G, tok = u.t0() + (row >> a.lg);
    on = tok < u.t1();
    return (const uint4*)(a.q + (((size_t)u.b * a.T + (on ? tok : u.t0())) * a.cv.Hq + u.h * G + (on ? row & (G - 1) : 0)) * D) + (t & 15);
  }
  // The unit's rows of Q on their way to their places, as they are.
  __device__ bool copy_q(const Walk& u) {
    if (qn > 0 && !wait(B_QEMPTY, qn - 1)) return false;
    const int rows = u.two() ? ROWS : TILE;
#pragma unroll 4
    for (int row = t >> 4; row < rows; row += 16) {
      bool on;
      const uint4* p = q_piece(u, row, on);
      copy16(q_place(saddr(smem + OFF_Q), t, row), p, on);
    }
    return true;
  }
  // The history's tiles, one side of them.  A warp has blocks 2 wp, 2 wp + 1, its lanes their
  // codes of the next tile in registers.
  template <int S>
  __device__ void history(const Walk& u) {
    const CacheView& cv = a.cv;
    const int end = u.hist_end(), blocks = u.r.H / KV8_BLK, sub = 2 * wp % KV8_PAGE_BLOCKS;
    const int32_t* pages = cv.page_table + (size_t)u.b * cv.max_pages_per_req;
    const int last_page = (u.r.H - 1) / PAGE;
    const uint8_t* head = kv8_head(cv, 0, u.h);  // in page 0
    Codes c[2];
    // The entry of the page with the warp's blocks of tile i (any entry, where there are none).  It
    // is looked at a tile later: what is made of a load at once takes its time.
    auto entry = [&](int i) { return pages[min(2 * i + (wp >> 1), last_page)]; };
    auto good = [&](int id, int i) {
      if (i >= end || 8 * i + 2 * wp >= blocks) return -1;
      return id >= 0 && id < cv.num_pages ? id : -1;
    };
    auto there = [&](int pid, int i, int j) { return pid >= 0 && 8 * i + 2 * wp + j < blocks; };
    auto load = [&](int pid, int i, int j) {
      load_codes<S>(c[j], head + (pid < 0 ? 0 : (size_t)pid * cv.page_bytes) + (sub + j) * KV8_BLOCK_BYTES, there(pid, i, j), lane);
    };
    int now = good(entry(u.i0), u.i0), next = entry(u.i0 + 1), far = entry(u.i0 + 2);
    if (!copy_q(u)) return;
    copies_commit();
    next = good(next, u.i0 + 1);
    copies_wait<0>();
    // (The first codes behind it, from pages that the scout has fetched: 64 tokens over 100K 116.3 -> 115.1 us.)
    convert_q(saddr(smem + OFF_Q), (int8_t*)(smem + OFF_ALPHA) + qn % NALPHA * ROWS, t, u.two() ? ROWS : TILE);
    ++qn;
    fence_proxy_async();
    arrive(barrier(B_QFULL));
    load(now, u.i0, 0);
    load(now, u.i0, 1);
    const uint32_t base = saddr(smem + OFF_BUF);
#pragma unroll 1
    for (int i = u.i0; i < end && ok; ++i, ++gt) {
      const int item = 2 * gt + S, buf = item % NBUF;
      if (!wait_empty(item)) return;
      const int after = far;
      far = entry(i + 3);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (S == 0) store_k<TYPE>(base + buf * BUF, c[j], 2 * wp + j, lane);
        else store_v<TYPE>(base + buf * BUF, c[j], 2 * wp + j, lane);
        load(next, i + 1, j);
      }
      const int ahead = good(after, i + 2);
      fence_proxy_async();
      told(B_FULL + buf);
      now = next;
      next = ahead;
    }
  }

  // The unit's tiles of BF16 tokens: token s of the line is in the sink, in the window
  // (which begins at ring slot H mod 256) or in the chunk.
  __device__ void line(const Walk& u) {
    const CacheView& cv = a.cv;
    if (!copy_q(u)) return;
    ++qn;
    Copies copies;
    push(copies, {B_QFULL, 0, 0, 0});
    const size_t head = (size_t)u.b * cv.Hkv + u.h;
    const int nsink = u.r.L < SINK ? u.r.L : SINK, all = u.r.w() + u.t1();
    for (int i = u.line_begin(); i < u.i1 && ok; ++i, ++gt) {
      const int s0 = (i - u.r.nh()) * TILE;
      const int item = 2 * gt + side, buf = item % NBUF;
      if (!wait_empty(item, copies)) return;
      const __nv_bfloat16* sink = (side ? cv.sink_v : cv.sink_k) + head * SINK * D;
      const __nv_bfloat16* ring = (side ? cv.ring_v : cv.ring_k) + head * RECENT * D;
      const __nv_bfloat16* fresh = (side ? a.v : a.k) + ((size_t)u.b * a.T * cv.Hkv + u.h) * D;
      const int ch = t & 15;
      const uint32_t to = saddr(smem + OFF_BUF) + buf * BUF + (ch >> 3) * REGION;
#pragma unroll 4
      for (int j = 0; j < 16; ++j) {
        const int tok = 8 * j + (t % SIDE >> 4), s = s0 + tok;
        const bool on = s < all;
        const __nv_bfloat16* p = s < nsink   ? sink + (size_t)s * D
                                 : s < u.r.w() ? ring + (size_t)((u.r.H + s - nsink) & (RECENT - 1)) * D
                                             : fresh + (size_t)(on ? s - u.r.w() : 0) * cv.Hkv * D;
        copy16(to + tok * 128 + (((ch & 7) ^ (tok & 7)) << 4), p + 8 * ch, on);
      }
      // tokens that only some of the unit's rows see: chunk tokens behind its first
      const int from = u.r.w() + u.t0() + 1 - s0, cut_to = all - s0 < TILE ? all - s0 : TILE;
      push(copies, {B_FULL + buf, buf, side ? (from > 0 ? from : 0) : 0, side ? cut_to : 0});
    }
    flush(copies);
  }

  __device__ void run() {
    Walk u(a, the_misc());
    for (; u.more() && ok; u.next()) {
      if (u.i0 < u.hist_end()) {
        if (side == 0) history<0>(u);
        else history<1>(u);
      }
      if (ok && u.line_begin() < u.i1) line(u);
    }
    copies_wait<0>();
  }
};

// One warp goes ahead of the producers: it says what each tile is, makes the scales from the
// history's, reports bad pages and brings pages into the L2 (the producers' registers
// have room for one tile, the memory takes longer than one).
__device__ void scout(const Kv8Prefill& a, int lane) {
  const CacheView& cv = a.cv;
  int gt = 0, un = 0;
  for (Walk u(a, the_misc()); u.more(); u.next(), ++un) {
    const int end = u.hist_end(), blocks = u.r.H / KV8_BLK, last_page = max(u.r.H - 1, 0) / PAGE;
    const int32_t* pages = cv.page_table + (size_t)u.b * cv.max_pages_per_req;
    // lanes 0 - 7: the blocks of a tile
    auto entry = [&](int i) { return i < end ? pages[min(2 * i + (lane >> 2 & 1), last_page)] : -1; };
    auto good = [&](int id, int i) {
      if (i >= end || lane >= 8 || 8 * i + lane >= blocks) return -1;
      if (id >= 0 && id < cv.num_pages) return id;
      if ((lane & 3) == 0) record_error(cv.err, id < 0 ? OSCAR_ERR_NO_PAGE : OSCAR_ERR_RANGE);
      return -1;
    };
    auto page = [&](int id) { return kv8_head(cv, id, u.h); };
    auto scale = [&](int id) {
      return id >= 0 ? __ldcg((const float2*)(page(id) + KV8_OFF_SCALES) + (lane & 3)) : make_float2(0.f, 0.f);
    };
    auto fetch = [&](int id) {
      if (id >= 0 && (lane & 3) == 0) bulk_prefetch_l2(page(id), KV8_HEAD_BYTES);
    };
    int now = good(entry(u.i0), u.i0), next = good(entry(u.i0 + 1), u.i0 + 1), far = entry(u.i0 + 2);
    float2 sc = scale(now);
    fetch(now);
    fetch(next);
#pragma unroll 1
    for (int i = u.i0; i < u.i1; ++i, ++gt) {
      const int item = 2 * gt, buf = item % NBUF;
      if (item >= NBUF &&
          !__all_sync(0xffffffffu, wait_bar(barrier(B_EMPTY + buf), (item / NBUF - 1) & 1, &the_misc()->abort, a.wait_polls)))
        return;
      if (i == u.i0 && lane == 0) {
        // NUNIT: the place's last unit lies six tiles or more behind the last tile whose O is
        // done, so both softmax groups have left it
        Unit* x = (Unit*)(smem + OFF_UNIT) + (un & (NUNIT - 1));
        x->tiles = u.i1 - u.i0;
        x->hist = max(end - u.i0, 0);
        const int s0 = (u.line_begin() - u.r.nh()) * TILE;
        x->line = u.r.w() + u.t0() + 1 - s0;
        x->flags = (u.two() ? U_TWO : 0) | (u.i0 == 0 ? U_BEGINS : 0) | (u.i1 == u.n ? U_ENDS : 0);
        x->b = u.b, x->h = u.h, x->t0 = u.t0(), x->t1 = u.t1();
        x->c0 = s0 - u.r.w(), x->c1 = (u.i1 - u.r.nh()) * TILE - u.r.w();
      }
      Info* f = (Info*)(smem + OFF_INFO) + (gt & (NINFO - 1));
      const bool hist = i < end, bad = now >= 0 && sc.y != sc.y;
      if (lane < 8) {
        f->cs[lane] = !hist ? make_float2(C0, 0.f) : make_float2(sc.x * C0, now < 0 || bad ? 0.f : log2f(sc.y));
        f->marks[lane] = (uint8_t)(!hist ? 1 : now < 0 ? 0 : bad ? 3 : 1);
      }
      if (lane == 0)
        f->flags = (hist ? F_HIST : 0) | (u.two() ? F_TWO : 0) | (i == u.i0 || i == end ? F_NEWQ : 0) |
                   (i + 1 == end || i + 1 == u.i1 ? F_ENDQ : 0) | (i + 1 == u.i1 ? F_ENDU : 0);
      __syncwarp();
      if (lane == 0) {
        arrive(barrier(B_INFO + (gt & (NINFO - 1))));
        arrive(barrier(B_FULL + buf));
      }
      now = next;
      sc = scale(now);
      next = good(far, i + 2);
      fetch(next);
      far = entry(i + 3);
    }
  }
}

// -------------------------------------------------------------------- MMA issue
// A whole warp, one lane elected for the instructions: with every value the same in
// all lanes (`same` tells the compiler so) an MMA takes the 64 cycles of its
// arithmetic, issued from a divergent branch 150.  It learns what a tile is from
// the scout's flags: anything slower than the MMAs would hold them up.
__device__ __forceinline__ uint64_t desc(uint32_t lo, uint64_t hi) { return hi | lo; }
__device__ __forceinline__ uint32_t same(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n .reg .pred P;\n elect.sync _|P, 0xffffffff;\n selp.u32 %0, 1, 0, P;\n}\n" : "=r"(p));
  return p != 0;
}

// Loops: the warp comes by once a step, and unrolled it would wait for its
// instructions, which the other warps' code has pushed out of the cache.
__device__ __forceinline__ void scores_mma(uint32_t d, uint32_t q, uint32_t k, uint64_t hi, uint32_t id) {
#pragma unroll 1
  for (int half = 0; half < 2; ++half, q += REGION >> 4, k += REGION >> 4)
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) mma_ss(d, desc(q + 2 * ks, hi), desc(k + 2 * ks, hi), id, half | ks);
}
__device__ __forceinline__ void values_mma(uint32_t d, uint32_t p, uint32_t v, uint64_t hi, uint32_t id, uint32_t add) {
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) mma_ts(d, p + 8 * kk, desc(v + kk * (2048 >> 4), hi), id, add | kk);  // 64 tokens
}

__device__ void issue(const Kv8Prefill& a) {
  Misc* misc = the_misc();
  const Info* infos = (const Info*)(smem + OFF_INFO);
  const uint32_t tmem = same(misc->tmem), qlo = saddr(smem + OFF_Q) >> 4, blo = saddr(smem + OFF_BUF) >> 4;
  const uint64_t hi = sdesc(0), hi_mn = sdesc_mn(0, REGION);
  const int total = (int)same((uint32_t)misc->tiles);
  // of S and of O: tiles done, second row tile's turn, step, ring place and its phase
  struct {
    int tile, half, step, buf, phase;
    uint32_t flags;
  } s = {0, 0, 0, 0, 0, 0}, p = {0, 0, 0, 1, 0, 0};
  uint32_t started = 0, pphase = 0, qphase = 0;
  auto wait = [&](int bar, uint32_t phase) {
    return (bool)__all_sync(0xffffffffu, wait_bar(barrier(bar), phase & 1, &misc->abort, a.wait_polls));
  };
  // What S of the next step needs: waits for it, or (look) only looks.
  auto learn_s = [&](bool look) -> bool {
    if (s.half) return true;
    if (look ? !__all_sync(0xffffffffu, passed(barrier(B_FULL + s.buf), s.phase)) : !wait(B_FULL + s.buf, s.phase)) return false;
    s.flags = same(infos[s.tile & (NINFO - 1)].flags);
    if (s.flags & F_NEWQ) {
      if (look ? !__all_sync(0xffffffffu, passed(barrier(B_QFULL), qphase)) : !wait(B_QFULL, qphase)) return false;
      qphase ^= 1;
    }
    return true;
  };
  auto learn_p = [&]() -> bool {
    if (p.half) return true;
    if (!wait(B_FULL + p.buf, p.phase)) return false;
    p.flags = same(infos[p.tile & (NINFO - 1)].flags);
    return true;
  };
  auto scores = [&]() {
    const uint32_t w = s.step & 1, q = qlo + (s.flags & F_TWO ? w * (BUF >> 4) : 0), k = blo + s.buf * (BUF >> 4);
    const bool last = !(s.flags & F_TWO) || s.half;  // of the tile's steps
    if (elect()) {
      scores_mma(tmem + S_COL + TILE * w, q, k, hi, s.flags & F_HIST ? idesc(0, 0) : idesc(1, 0));
      commit(barrier(B_S + w));
      if (last) commit(barrier(B_EMPTY + s.buf));
      if (last && (s.flags & F_ENDQ)) commit(barrier(B_QEMPTY));
    }
    __syncwarp();
    ++s.step;
    s.half = !last;
    if (last) {
      ++s.tile;
      s.buf += 2;
      if (s.buf >= NBUF) s.buf -= NBUF, s.phase ^= 1;
    }
  };
  auto values = [&](int part) {  // tokens 64 part .. + 63
    const uint32_t w = p.step & 1, v = blo + p.buf * (BUF >> 4) + part * (4 * 2048 >> 4);
    const bool last = part && (!(p.flags & F_TWO) || p.half), end = last && (p.flags & F_ENDU);
    const uint32_t add = part | (started >> w & 1);
    started |= 1u << w;
    if (elect()) {
      values_mma(tmem + O_COL + TILE * w, tmem + S_COL + TILE * w + 32 * part, v, hi_mn, p.flags & F_HIST ? idesc(0, 1) : idesc(1, 1), add);
      if (last) commit(barrier(B_EMPTY + p.buf));
      if (end && (started & 1)) commit(barrier(B_O));
      if (end && (started & 2)) commit(barrier(B_O + 1));
    }
    __syncwarp();
    if (!part) return;
    if (end) started = 0;
    ++p.step;
    p.half = !last;
    if (last) {
      ++p.tile;
      p.buf += 2;
      if (p.buf >= NBUF) p.buf -= NBUF, p.phase ^= 1;
    }
  };
  // S runs up to two steps ahead of O, but waits for K or Q only when there is no O left to
  // issue: K may need the buffer of a V, and Q's loading may not hold up a unit's end.
  // A look at shared memory takes some 250 cycles beside the MMAs, so it is taken before the
  // second half of P is awaited, where S can follow O at once (4 x 509 tokens 359 -> 354 us, 2048 over
  // 100K 2790 -> 2735; not in BF16 tiles: prompt 560 -> 541).
  bool ok = true;
  while (ok && p.tile < total) {
    while (s.tile < total && s.step - p.step < 2) {
      const bool must = s.step == p.step;
      if (!learn_s(!must)) {
        ok = !must;
        break;
      }
      fence_after();
      scores();
    }
    if (!ok) break;
    const uint32_t w = p.step & 1, phase = pphase >> w;
    pphase ^= 1u << w;
    ok = learn_p() && wait(B_P + 2 * w, phase);
    if (!ok) break;
    fence_after();
    values(0);
    const bool more = (p.flags & F_HIST) && s.tile < total && s.step - p.step < 3 && learn_s(true);
    ok = wait(B_P + 2 * w + 1, phase);
    if (!ok) break;
    fence_after();
    values(1);
    if (more) scores();
  }
  // all that was issued has ended before the tensor memory is given back
  if (elect()) commit(barrier(B_DRAIN));
  __syncwarp();
  mbar_wait(barrier(B_DRAIN), 0);
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

__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t (&r)[16]) {  // and waits
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
               "tcgen05.wait::ld.sync.aligned;\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                 "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(at)
               : "memory");
}

// A row's running state.
struct Row {
  float m, l, M;
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two fp32 values in one register pair: one instruction works on both.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 16 columns of S, and their largest.
__device__ __forceinline__ void tmem_ld16_max(uint32_t at, uint32_t (&r)[16], float& m) {
  asm volatile("tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, %16, [%17];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                 "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=f"(m)
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void tmem_ld16_async(uint32_t at, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                 "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void after_wait(uint32_t (&r)[16]) {  // uses of r stay behind the wait
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                    "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t at, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Tokens of two blocks that a row takes: `seen` first ones, and of those the blocks whose mark
// (a byte each) says so.  EVERY: all of them.
struct Taken {
  uint32_t marks;
  int seen;
  __device__ __forceinline__ bool operator()(int b, int j) const { return (marks >> (8 * b) & 1) && 16 * b + j < seen; }
  __device__ __forceinline__ bool nan(int b) const { return marks >> (8 * b) & 2; }
};

// P of block b of two from its S, to `at`; its sum.
template <bool F16, bool EVERY>
__device__ __forceinline__ uint64_t exponentials(const uint32_t (&r)[16], int b, uint32_t at, float cb, float shift, const Taken& taken) {
  const uint64_t cb2 = pair(cb, cb), shift2 = pair(shift, shift);
  uint64_t sum = 0;  // two zeros
  uint32_t o[8];
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    float y, z;
    unpair(fma2(pair(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), cb2, shift2), y, z);
    y = ex2(y);
    z = ex2(z);
    if (!EVERY) {
      if (!taken(b, j)) y = 0.f;
      if (!taken(b, j + 1)) z = 0.f;
    }
    sum = add2(sum, pair(y, z));
    if (!EVERY && taken.nan(b)) y = z = NAN;
    o[j / 2] = pack2<F16>(y, z);
  }
  tmem_st8(at, o);
  return sum;
}
// Adds a sum of P to the state.
__device__ __forceinline__ void add_sum(Row& st, uint64_t sum, float shift) {
  float s0, s1;
  unpair(sum, s0, s1);
  st.l = fmaf(s0 + s1, ex2(-shift - st.m), st.l);
}

// Largest of a block's taken logits, where not all are.
__device__ __forceinline__ float largest(const uint32_t (&r)[16], int b, const Taken& taken) {
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < 16; ++j) m = fmaxf(m, taken(b, j) ? __uint_as_float(r[j]) : -INFINITY);
  return m;
}

// P of the tile to tensor memory, in two halves (said(i): tells of one), sums into the
// state.  S is read twice, the registers do not hold all of it.  Two blocks at a time, in loops that
// are not unrolled: the loops of all roles then fit into the instruction caches together
// (unrolled, warps stood for instructions as long as for shared memory: 16 requests with
// 5 tokens 238 -> 228 us, 4 with 509 420 -> 355, a prompt of 8191 636 -> 594, 2048 tokens over
// 100K 2820 -> 2720).  The largest of the history are found without a loop (with: 2720 -> 2840),
// and the load behind its last pair is made and thrown away (2770 with a branch; BF16
// tiles have the branch, without it the prompt takes 635).
template <bool F16, bool EVERY, typename Said>
__device__ __forceinline__ void weigh(Row& st, uint32_t sa, uint32_t oa, const Info* f, float al, int seen, bool first, float room, Said said) {
  uint32_t r[2][16];
  const float4* cs = (const float4*)f->cs;
  const uint16_t* marks = (const uint16_t*)f->marks;
  float4 sc;
  float mx = NONE, tx = NONE;
#pragma unroll (F16 ? 4 : 1)
  for (int h = 3; h >= 0; --h) {
    float mb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) tmem_ld16_max(sa + 32 * h + 16 * i, r[i], mb[i]);
    if (F16) {
      sc = cs[h];
      sc.x *= al, sc.z *= al;
    }
    const Taken taken = {EVERY ? 0u : F16 ? marks[h] : 0x0101u, seen - 32 * h};
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 2; ++i) after_wait(r[i]);
    if (!EVERY)
#pragma unroll
      for (int i = 0; i < 2; ++i) mb[i] = largest(r[i], i, taken);
    asm volatile("" : "+f"(mb[0]), "+f"(mb[1])::"memory");
    if (F16) {
      const float y = mb[0] * sc.x, z = mb[1] * sc.z;
      mx = max3(mx, y, z);
      tx = max3(tx, y + sc.y, z + sc.w);
    } else {
      mx = max3(mx, mb[0] * C0, mb[1] * C0);
    }
  }
  const float mn = fmaxf(st.m, mx);
  st.l *= ex2(st.m - mn);
  st.m = mn;
  // M, were it chosen now; BF16 tokens also lower what a history of large values has left
  const float aim = F16 ? tx - HEAD : mn + room;
  const bool off = aim > st.M + LAZY || (!F16 && st.M > aim + SPARE);
  if (first) {
    st.M = aim;
  } else if (__any_sync(0xffffffffu, off)) {
    const float Mn = F16 || !off ? fmaxf(st.M, aim) : aim;
    const float g = ex2(0.5f * (st.M - Mn));  // twice: from small scales to BF16 tokens it is 2^-150
    st.M = Mn;
    // S of this step is complete, so is every MMA issued before it: O has all steps before
#pragma unroll 1
    for (int c = 0; c < TILE; c += 16) {
      uint32_t v[16];
      tmem_ld16(oa + c, v);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * g * g);
      tmem_st16(oa + c, v);
    }
  }
  const float line_shift = -st.M;
  uint64_t sum = 0;
#pragma unroll 1
  for (int h = 0; h < 4; ++h) {
    const Taken taken = {EVERY ? 0u : F16 ? marks[h] : 0x0101u, seen - 32 * h};
    float4 nc;
    if (F16) nc = cs[(h + 1) & 3];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (F16) {
        const float shift = max_nan((b ? sc.w : sc.y) - st.M, -st.m - FAR);
        add_sum(st, exponentials<F16, EVERY>(r[b], b, sa + 16 * h + 8 * b, b ? sc.z : sc.x, shift, taken), shift);
      } else {
        sum = add2(sum, exponentials<F16, EVERY>(r[b], b, sa + 16 * h + 8 * b, C0, line_shift, taken));
      }
      if (F16 || h < 3) tmem_ld16_async(sa + 32 * ((h + 1) & 3) + 16 * b, r[b]);
    }
    if (F16) {
      sc = nc;
      sc.x *= al, sc.z *= al;
    }
    if (h & 1) {
      tmem_st_wait();
      said(h >> 1);
    }
    tmem_ld_wait();
#pragma unroll
    for (int b = 0; b < 2; ++b) after_wait(r[b]);
  }
  if (!F16) add_sum(st, sum, line_shift);
}

__device__ __forceinline__ void store32(__nv_bfloat16* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {  // aligned to 32 bytes
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    ((uint4*)p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    ((uint4*)p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
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

// The record of a unit that is not whole in a part: O by groups of four channels, [32][256]
// rows (neighbouring lanes have neighbouring rows), then each row's log2 of the sum of
// exponentials and its M.
struct Record {
  float* p;
  __device__ Record(const Kv8Prefill& a, int cta, int slot) : p(a.part + (size_t)(2 * cta + slot) * ROWS * PART_STRIDE) {}
  __device__ float4* o(int group, int row) const { return (float4*)p + group * ROWS + row; }
  __device__ float& lg(int row) const { return p[ROWS * D + row]; }
  __device__ float& M(int row) const { return p[ROWS * D + ROWS + row]; }
};

// A row of a unit (lg: its log2 of the sum of exponentials), or its record where the
// unit is not whole here.  O = h0²·[oa] + h1²·[ob], either address 0 where there is no such part.  (Addresses are
// the same for the warp, factors are not: a tensor-memory load is the whole warp's, so no
// branch around one may look at a row's factor.)
__device__ __forceinline__ void write_row(const Kv8Prefill& a, const Unit* u, int row, float lg, float M, uint32_t oa, float h0,
                                          uint32_t ob, float h1, bool bad_v) {
  const int G = a.cv.G, tok = u->t0 + (row >> a.lg);
  const bool on = tok < u->t1, whole = (u->flags & (U_BEGINS | U_ENDS)) == (U_BEGINS | U_ENDS);
  const size_t at = ((size_t)u->b * a.T + (on ? tok : u->t0)) * a.cv.Hq + u->h * G + (row & (G - 1));
  const Record rec(a, blockIdx.x, u->flags & U_BEGINS ? 1 : 0);
  const bool wide = ((uintptr_t)a.out & 31) == 0;
  // The factor's root, taken twice: for values of 2^-100 it is below 2^-126.  Nothing seen: zeros, and -infinity as the lse.
  const float f = lg == -INFINITY ? 0.f : ex2(0.5f * (M - lg));
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    float o[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) o[j] = 0.f;
    uint32_t v[32];
    if (oa) {
      tmem_ld32(oa + c, v);
      tmem_ld_wait_regs(v);
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = __uint_as_float(v[j]) * h0 * h0;
    }
    if (ob) {
      tmem_ld32(ob + c, v);
      tmem_ld_wait_regs(v);
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = fmaf(__uint_as_float(v[j]) * h1, h1, o[j]);
    }
    if (bad_v && on) {
      float x[32];
      for (int j = 0; j < 32; ++j) x[j] = o[j];
      add_bad(a, u->b, u->h, max(u->t0 + 1, u->c0), min(tok + 1, u->c1), c, x);
      for (int j = 0; j < 32; ++j) o[j] = x[j];
    }
    if (on && !whole) {
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        *rec.o((c + j) >> 2, row) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
    } else if (on) {
#pragma unroll
      for (int j = 0; j < 32; j += 16) {
        uint32_t x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = pack2<false>(o[j + 2 * i] * f * f, o[j + 2 * i + 1] * f * f);
        store32(a.out + at * D + c + j, x, wide);
      }
    }
    __syncwarp();
  }
  if (on && !whole) {
    rec.lg(row) = lg;
    rec.M(row) = M;
  } else if (on && a.lse) {
    a.lse[at] = lg * LN2;
  }
  __syncwarp();
}

// After a wait that ran out: NaN in the group's rows of unit `un` of the part and those behind it.
__device__ __noinline__ void abandon(const Kv8Prefill& a, const Misc* m, int un, int wg, int row) {
  const int G = a.cv.G;
  int i = 0;
  for (Walk u(a, m); u.more(); u.next(), ++i) {
    const int urow = (u.two() ? TILE * wg : 0) + row, tok = u.t0() + (urow >> a.lg);
    if (i < un || (!u.two() && wg == 1) || tok >= u.t1()) continue;
    if (u.i0 > 0 || u.i1 < u.n) {
      Record(a, blockIdx.x, u.i0 == 0 ? 1 : 0).lg(urow) = NAN;
      continue;
    }
    const size_t at = ((size_t)u.b * a.T + tok) * a.cv.Hq + u.h * G + urow % G;
    for (int c = 0; c < D; ++c) a.out[at * D + c] = __float2bfloat16_rn(NAN);
    if (a.lse) a.lse[at] = NAN;
  }
}

// log2 of 2^a + 2^b.
__device__ __forceinline__ float add_logs(float a, float b) {
  const float m = fmaxf(a, b);
  return m == -INFINITY ? (a == b ? m : NAN) : m + log2f(ex2(a - m) + ex2(b - m));
}

__device__ void softmax(const Kv8Prefill& a, int tid) {
  Misc* misc = the_misc();
  const int warp = tid >> 5, wg = warp >> 2, row = tid & 127;
  const uint32_t tmem = misc->tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  const uint32_t sa = tmem + S_COL + TILE * wg, oa = tmem + O_COL + TILE * wg;
  const int total = misc->tiles;
  auto wait = [&](int bar, int phase) {
    return (bool)__all_sync(0xffffffffu, wait_bar(barrier(bar), phase & 1, &misc->abort, a.wait_polls));
  };
  bool ok = true;
  // token tiles and steps done; this group's S and O so far; exchanges; units, loads of Q
  int gt = 0, g = 0, ns = 0, no = 0, nx = 0, un = 0, qn = 0;
  while (gt < total) {
    if (ok) ok = wait(B_INFO + (gt & (NINFO - 1)), gt / NINFO);
    if (!ok) break;
    const Unit* u = (const Unit*)(smem + OFF_UNIT) + (un & (NUNIT - 1));
    const int tiles = u->tiles, hist = u->hist, two = u->flags & U_TWO;
    const int urow = (two ? TILE * wg : 0) + row, line = u->line + (urow >> a.lg);
    // What O has in rows behind the unit's last token is not written: a warp that has no other
    // rows leaves its P as it is (16 requests with 5 tokens: 229 -> 200 us).
    const bool rows = __any_sync(0xffffffffu, u->t0 + (urow >> a.lg) < u->t1);
    Row st = {NONE, 0.f, NONE};
    float al = 0.f;
    int cnt = 0;
    for (int i = two ? 0 : (wg - g) & 1; i < tiles; i += two ? 1 : 2) {
      const int tile = gt + i;
      // S of a tile tells that all about it is there: the MMAs began after the producers had
      // told of K, which they do last
      ok = wait(B_S + wg, ns);
      if (!ok) break;
      ++ns;
      fence_after();
      const Info* f = (const Info*)(smem + OFF_INFO) + (tile & (NINFO - 1));
      auto said = [&](int h) {
        fence_before();
        __syncwarp();
        if ((tid & 31) == 0) arrive(barrier(B_P + 2 * wg + h));
      };
      if (!rows) {
        if ((tid & 31) == 0) arrive(barrier(B_P + 2 * wg)), arrive(barrier(B_P + 2 * wg + 1));
      } else if (i < hist) {
        if (cnt == 0) al = pow2i(((const int8_t*)(smem + OFF_ALPHA))[qn % NALPHA * ROWS + urow]);
        const uint32_t* marks = (const uint32_t*)f->marks;
        if (marks[0] == ALL_COUNT && marks[1] == ALL_COUNT) weigh<true, true>(st, sa, oa, f, al, TILE, cnt == 0, a.room, said);
        else weigh<true, false>(st, sa, oa, f, al, TILE, cnt == 0, a.room, said);
      } else {
        const int seen = line - (i - hist) * TILE;
        if (__all_sync(0xffffffffu, seen >= TILE)) weigh<false, true>(st, sa, oa, f, 1.f, seen, cnt == 0, a.room, said);
        else weigh<false, false>(st, sa, oa, f, 1.f, seen, cnt == 0, a.room, said);
      }
      ++cnt;
    }
    if (ok && cnt > 0) {
      ok = wait(B_O + wg, no);
      ++no;
      fence_after();
    }
    const bool bad_v = *(volatile int*)&misc->bad_v != 0 && tiles > hist;
    float lg = st.m != NONE && fabsf(st.m) >= TOO_LARGE ? NAN : st.l == 0.f ? -INFINITY : st.m + log2f(st.l);
    if (!ok) break;
    if (two) {
      if (rows) write_row(a, u, urow, lg, st.M, oa, 1.f, 0, 0.f, bad_v);
    } else {
      float2* other = (float2*)(smem + OFF_XCH) + row;
      if (wg == 1) {
        *other = make_float2(lg, cnt > 0 ? st.M : -INFINITY);
        fence_before();
        __syncwarp();
        if ((tid & 31) == 0) arrive(barrier(B_OTHER));
        ok = wait(B_TAKEN, nx);
        if (!ok) break;
      } else {
        ok = wait(B_OTHER, nx);
        if (!ok) break;
        fence_after();
        const float2 x = *other;
        const bool one = __any_sync(0xffffffffu, x.y != -INFINITY);  // the other group had a tile (the same for all rows)
        const float M = cnt > 0 ? fmaxf(st.M, x.y) : x.y;
        if (rows) write_row(a, u, urow, add_logs(lg, x.x), M, cnt > 0 ? oa : 0, ex2(0.5f * (st.M - M)), one ? oa + TILE : 0,
                  ex2(0.5f * (x.y - M)), bad_v);
        fence_before();
        __syncwarp();
        if ((tid & 31) == 0) arrive(barrier(B_TAKEN));
      }
      ++nx;
    }
    gt += tiles;
    g += two ? 2 * tiles : tiles;
    qn += (int)(hist > 0) + (int)(tiles > hist);
    ++un;
  }
  if (!ok) abandon(a, misc, un, wg, row);
}

template <int TYPE>
__global__ void __launch_bounds__(THREADS, 1) attend_kernel(const __grid_constant__ Kv8Prefill a) {
  Misc* misc = the_misc();
  const int tid = threadIdx.x, warp = (int)same(tid >> 5);
  if (saddr(smem) & 1023) {  // the swizzled tiles begin on 1024 bytes; there is no room to move them
    if (tid == 0) {
      a.splits[blockIdx.x] = make_int4(0, 0, 0, -1);
      record_error(a.cv.err, OSCAR_ERR_CUDA);
    }
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(barrier(B_FULL + i), SIDE + 1);
      mbar_init(barrier(B_EMPTY + i), 1);
    }
    for (int i = 0; i < NINFO; ++i) mbar_init(barrier(B_INFO + i), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(barrier(B_S + i), 1);
      mbar_init(barrier(B_P + 2 * i), 4);
      mbar_init(barrier(B_P + 2 * i + 1), 4);
      mbar_init(barrier(B_O + i), 1);
    }
    mbar_init(barrier(B_QFULL), PROD);
    mbar_init(barrier(B_QEMPTY), 1);
    mbar_init(barrier(B_OTHER), 4);
    mbar_init(barrier(B_TAKEN), 4);
    mbar_init(barrier(B_DRAIN), 1);
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
  if (warp >= ISSUE0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(REGS_MMA));
    if (warp == MMA_WARP) issue(a);
    if (warp == SCOUT_WARP) scout(a, tid & 31);
  } else if (tid >= PROD0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(REGS_PROD));
    Producer<TYPE>(a, tid).run();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(REGS_SOFTMAX));
    softmax(a, tid);
  }
  fence_before();
  __syncthreads();
  if (tid == 0 && misc->abort) record_error(a.cv.err, OSCAR_ERR_TIMEOUT);
  if (warp == MMA_WARP) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
  }
}

// Joins the records of the unit that begins in part blockIdx.x, 16 rows a CTA; a thread has
// four channels of a row.  (64 tokens over 100K: 20 MB of records, some 5 of 115 us with the
// launch.  Joining in the last CTA of a unit would need counters that are zero before the
// call, which the scratch does not have.)
constexpr int JOIN_ROWS = 16;
__global__ void __launch_bounds__(512) join_kernel(const __grid_constant__ Kv8Prefill a) {
  __shared__ float s[KV8_PREFILL_MAX_GRID][JOIN_ROWS];
  pdl_wait();
  pdl_launch_dependents();
  const int4 d = a.splits[blockIdx.x];
  if (d.w < 0) return;
  // (In bounds whatever another call may have put there meanwhile, should two share a scratch.)
  if (d.w <= (int)blockIdx.x || d.w >= (int)gridDim.x || (unsigned)d.x >= (unsigned)a.B || (unsigned)d.y >= (unsigned)a.cv.Hkv ||
      (unsigned)d.z >= (unsigned)a.units)
    return;
  const int r16 = threadIdx.x % JOIN_ROWS, group = threadIdx.x / JOIN_ROWS, row = blockIdx.y * JOIN_ROWS + r16, G = a.cv.G;
  const int tok = d.z * (ROWS / G) + row / G;
  if (d.z * (ROWS / G) + (int)blockIdx.y * JOIN_ROWS / G >= a.T) return;  // none of the CTA's rows
  const int first = blockIdx.x, n = d.w - first + 1;
  const bool on = tok < a.T;
  for (int k = group; k < n; k += 32) s[k][r16] = on ? Record(a, first + k, k == 0).lg(row) : -INFINITY;
  __syncthreads();
  float m = -INFINITY, L = 0.f;
  bool nan = false;
  for (int k = 0; k < n; ++k) {
    m = fmaxf(m, s[k][r16]);
    nan |= s[k][r16] != s[k][r16];
  }
  const bool none = m == -INFINITY;  // nothing seen
  for (int k = 0; k < n; ++k) L += none ? 0.f : ex2(s[k][r16] - m);
  const float lg = nan ? NAN : none ? -INFINITY : m + log2f(L);
  __syncthreads();
  for (int k = group; k < n; k += 32)  // roots, taken twice
    s[k][r16] = none && !nan ? 0.f : on ? ex2(0.5f * (Record(a, first + k, k == 0).M(row) - lg)) : 0.f;
  __syncthreads();
  if (!on) return;
  float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int k = 0; k < n; ++k) {
    const float f = s[k][r16];
    const float4 x = *Record(a, first + k, k == 0).o(group, row);
    o[0] = fmaf(x.x * f, f, o[0]);
    o[1] = fmaf(x.y * f, f, o[1]);
    o[2] = fmaf(x.z * f, f, o[2]);
    o[3] = fmaf(x.w * f, f, o[3]);
  }
  const size_t at = ((size_t)d.x * a.T + tok) * a.cv.Hq + d.y * G + row % G;
  *(uint2*)(a.out + at * D + 4 * group) = make_uint2(pack2<false>(o[0], o[1]), pack2<false>(o[2], o[3]));
  if (group == 0 && a.lse) a.lse[at] = lg * LN2;
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

cudaError_t launch_kv8_prefill(Kv8Prefill a, int type, cudaStream_t st, Profiler* prof) {
  a.lg = 0;
  while (1 << a.lg < a.cv.G) ++a.lg;
  a.units = (int)((((long long)a.T << a.lg) + ROWS - 1) / ROWS);
  const long long most = SINK + RECENT + (long long)a.cv.max_pages_per_req * PAGE + a.T;  // tokens that a row can see
  a.room = LAZY;
  for (long long n = 1; n < most; n *= 2) a.room += 1.f;
  prof_begin(prof, OSCAR_KERNEL_PREFILL_ATTN, st);
  cudaError_t e = type == OSCAR_KV8_E4M3 ? launch_attend<OSCAR_KV8_E4M3>(a, st) : launch_attend<OSCAR_KV8_INT8>(a, st);
  prof_end(prof, OSCAR_KERNEL_PREFILL_ATTN, st);
  if (e != cudaSuccess) return e;
  prof_begin(prof, OSCAR_KERNEL_PREFILL_MERGE, st);
  e = launch_pdl(join_kernel, dim3(a.grid, ROWS / JOIN_ROWS), dim3(32 * JOIN_ROWS), 0, st, a);
  prof_end(prof, OSCAR_KERNEL_PREFILL_MERGE, st);
  return e;
}

}  // namespace oscar
