// Writing and evicting in a cache with 8-bit history (sm_103a).
#include "oscar_kv8.cuh"

namespace oscar {

namespace {

// ------------------------------------------------------------------- append
constexpr int AW = 16;  // warps per append CTA

// One side of a block, 64 BF16 values per lane in the order of the layout:
// K: w[c][r][j]  row 8r + gid, channels 32c + 8tq + 2j, + 1
// V: w[2h + l][i][j]  row 8h + 2tq + l, channels 16gid + 8i + 2j, + 1
struct SideRows {
  uint4 w[4][2];
};

__device__ __forceinline__ uint32_t word(const uint4& x, int j) { return ((const uint32_t*)&x)[j]; }

// Row(t): the address of token t's 128 channels.
template <typename Row>
__device__ __forceinline__ void load_side(SideRows& S, int side, int lane, Row row) {
  const int gid = lane >> 2, tq = lane & 3;
  if (side == 0) {
    const uint4* r0 = (const uint4*)(row(gid)) + tq;
    const uint4* r1 = (const uint4*)(row(8 + gid)) + tq;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      S.w[c][0] = r0[4 * c];
      S.w[c][1] = r1[4 * c];
    }
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint4* r = (const uint4*)(row(8 * (t >> 1) + 2 * tq + (t & 1))) + 2 * gid;
      S.w[t][0] = r[0];
      S.w[t][1] = r[1];
    }
  }
}

// x qmax / am rounded to the nearest 8-bit value, ties to even, exactly, without
// a division per value.  f = qmax / am has one rounding, so the product x f is
// within 2^-24 of the quotient.  x and am have 8 significant bits and a
// midpoint between codes at most 8: a quotient that is not a midpoint is at
// least 2^-16 away from one (2^-13 for e4m3), relative.  So the exact product is
// first rounded to a grid that holds the midpoints and is finer than that, which
// puts the midpoints back in their places and moves nothing across one.
struct Factor {
  float f, g;
};

// Two fp32 values in one register pair: one instruction works on both.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Codes of two values, in the low two bytes.
//  e4m3: with g = -17 f (about), c = x g is a multiple of 16 ulp(x f), d is
//    x f + c rounded to such multiples, and d - c, exact, the multiple next to x f:
//    20 bits of it.
//  int8: adding 192 rounds x f to multiples of 2^-16 (2^-15 from 64 on, 2^-17 below
//    -64); adding the rest of 1.5 2^23 rounds that to an integer, whose low byte
//    is the code.
template <int TYPE>
__device__ __forceinline__ uint32_t codes2(uint64_t x, Factor k) {
  uint32_t r;
  if (TYPE == OSCAR_KV8_E4M3) {
    const uint64_t c = mul2(x, pair(k.g, k.g));
    const uint64_t y = fma2(c, pair(-1.f, -1.f), fma2(x, pair(k.f, k.f), c));
    asm("{\n .reg .f32 a, b;\n .reg .b16 t;\n mov.b64 {a, b}, %1;\n cvt.rn.satfinite.e4m3x2.f32 t, b, a;\n"
        " cvt.u32.u16 %0, t;\n}\n"
        : "=r"(r)
        : "l"(y));
  } else {
    const float rest = 12582912.f - 192.f;
    const uint64_t y = add2(fma2(x, pair(k.f, k.f), pair(192.f, 192.f)), pair(rest, rest));
    asm("{\n .reg .b32 a, b;\n mov.b64 {a, b}, %1;\n prmt.b32 %0, a, b, 0x0040;\n}\n" : "=r"(r) : "l"(y));
  }
  return r;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// A warp quantises one side of a block and writes codes and scale.
template <int TYPE>
__device__ __forceinline__ void quantise_side(const SideRows& S, int side, uint8_t* block, float* scale, int lane) {
  const float qmax = TYPE == OSCAR_KV8_E4M3 ? 448.f : 127.f;
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) mx = max_abs2(mx, word(S.w[i][r], j));
  mx = max(mx >> 16, mx & 0xffffu);
  mx = __reduce_max_sync(0xffffffffu, mx);
  // an infinity or NaN in the block: NaN as its scale, so that whatever reads the block shows it
  const bool bad = mx >= 0x7f80u;
  const float am = fmaxf(__uint_as_float(mx << 16), KV8_TINY);
  const int e = (int)((__float_as_uint(am) >> 23) & 0xffu) - 127;  // am = 2^e x [1, 2)
  const float unit = __uint_as_float((__float_as_uint(am) & 0x007fffffu) | 0x3f800000u);
  Factor k;
  k.f = ldexpf(__fdiv_rn(qmax, unit), -e);
  k.g = -17.f * k.f;
  uint4* dst = (uint4*)(block + side * (KV8_BLK * D)) + lane;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint4 o;
    uint32_t* ow = (uint32_t*)&o;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t x, y;
        float a, b, p, q;
        if (side == 0) {  // bytes: row 8r + gid, channels + l
          x = word(S.w[c][0], 2 * s + h);
          y = word(S.w[c][1], 2 * s + h);
          a = bf_lo(x), b = bf_hi(x), p = bf_lo(y), q = bf_hi(y);
        } else {  // bytes: channel + r, token 8h + 2tq + l
          const int j = 2 * c + s;  // channel pair 16gid + 2j
          x = word(S.w[2 * h][j >> 2], j & 3);
          y = word(S.w[2 * h + 1][j >> 2], j & 3);
          a = bf_lo(x), b = bf_lo(y), p = bf_hi(x), q = bf_hi(y);
        }
        ow[2 * s + h] = bad ? 0u : prmt(codes2<TYPE>(pair(a, b), k), codes2<TYPE>(pair(p, q), k), 0x5410);
      }
    dst[32 * c] = o;
  }
  if (lane == 0) *scale = bad ? __uint_as_float(0x7fffffffu) : __fdiv_rn(am, qmax);
}

// The lengths an append leaves, and whether it can be done at all: `err` is
// the reason if not.
struct AppendPlan {
  int L, H, L1, H1;
  int err;
};

__device__ __forceinline__ AppendPlan append_lengths(const CacheView& cv, int b, int T, bool early = false) {
  AppendPlan p;
  const Kv8Req r = kv8_req(cv, b, early);
  p.L = r.L;
  p.H = r.H;
  p.err = r.ok ? 0 : OSCAR_ERR_STATE;
  const long long L1 = (long long)r.L + T;
  // a window of at most 256 tokens that starts on a block: its last 16 blocks
  const long long last = L1 > SINK ? (L1 - SINK - 1) / KV8_BLK : -1;
  long long H1 = (last + 1 - KV8_RING_BLOCKS) * KV8_BLK;
  if (H1 < r.H) H1 = r.H;
  if (!p.err && (H1 + PAGE - 1) / PAGE > cv.max_pages_per_req) p.err = OSCAR_ERR_RANGE;
  p.L1 = (int)L1;
  p.H1 = (int)H1;
  return p;
}

// And the pages that take the blocks.  Every thread of the block calls it.
__device__ __forceinline__ AppendPlan append_plan(const CacheView& cv, int b, int T, bool early = false) {
  AppendPlan p = append_lengths(cv, b, T, early);
  int bad = 0;
  if (!p.err && p.H1 > p.H)
    for (int pg = p.H / PAGE + (int)threadIdx.x; pg < (p.H1 + PAGE - 1) / PAGE; pg += blockDim.x) {
      const int32_t* at = cv.page_table + (size_t)b * cv.max_pages_per_req + pg;
      const int id = early ? __ldcg(at) : *at;
      if (id < 0) bad |= 1;
      if (id >= cv.num_pages) bad |= 2;
    }
  if (__syncthreads_or(bad)) p.err = __syncthreads_or(bad & 1) ? OSCAR_ERR_NO_PAGE : OSCAR_ERR_RANGE;
  return p;
}

// The plan in blocks of 16 positions.
struct AppendBlocks {
  int first, last;  // blocks with a new token
  int old_last;     // last block with a token before the call
  int h0, h1;       // history before and after
};

__device__ __forceinline__ AppendBlocks append_blocks(const AppendPlan& p) {
  AppendBlocks k;
  k.old_last = p.L > SINK ? (p.L - SINK - 1) / KV8_BLK : -1;
  k.first = ((p.L > SINK ? p.L : SINK) - SINK) / KV8_BLK;
  k.last = p.L1 > SINK ? (p.L1 - SINK - 1) / KV8_BLK : -1;
  k.h0 = p.H / KV8_BLK;
  k.h1 = p.H1 / KV8_BLK;
  return k;
}

__device__ __forceinline__ float* block_weights(const Kv8Append& a, size_t head) {
  return a.weights ? a.weights + head * (KV8_RING_BLOCKS + (size_t)KV8_PAGE_BLOCKS * a.cv.max_pages_per_req) : nullptr;
}

// A warp quantises one side of block `go` of (b, h) from rows Row(t).
template <int TYPE, typename Row>
__device__ __forceinline__ void quantise_block(const Kv8Append& a, int b, int h, int side, int go, int lane, Row row) {
  SideRows S;
  load_side(S, side, lane, row);
  const int pid = a.cv.page_table[(size_t)b * a.cv.max_pages_per_req + go / KV8_PAGE_BLOCKS];
  uint8_t* base = kv8_head(a.cv, pid, h);
  const int sub = go % KV8_PAGE_BLOCKS;
  quantise_side<TYPE>(S, side, base + sub * KV8_BLOCK_BYTES, (float*)(base + KV8_OFF_SCALES) + 2 * sub + side, lane);
}

// What stays in BF16: unit 0 is the sink, unit 1 + i block max(first, h1) + i of
// the window; a warp each per kv head and side.  The block that had the ring
// slots, if it leaves the window in this call, is quantised first by the same
// warp (its tokens from the ring, and from the input those it still lacked), so
// no other warp reads what this one overwrites.
template <int TYPE>
__device__ __forceinline__ void append_window(const Kv8Append& a, const AppendPlan& p, const AppendBlocks& kb, int b, int h,
                                              int side, int unit, int lane) {
  const CacheView& cv = a.cv;
  const int Hkv = cv.Hkv;
  const size_t head = (size_t)b * Hkv + h, in_row = (size_t)Hkv * D;
  const __nv_bfloat16* in = (side ? a.v : a.k) + ((size_t)b * a.T * Hkv + h) * D;  // token t at in + t Hkv D
  if (unit == 0) {
    __nv_bfloat16* sink = (side ? cv.sink_v : cv.sink_k) + head * SINK * D;
    const int end = p.L1 < SINK ? p.L1 : SINK;
    for (int t = p.L + (lane >> 4); t < end; t += 2)
      ((uint4*)(sink + (size_t)t * D))[lane & 15] = ((const uint4*)(in + (size_t)(t - p.L) * in_row))[lane & 15];
    return;
  }
  __nv_bfloat16* ring = (side ? cv.ring_v : cv.ring_k) + head * RECENT * D;
  float* wts = block_weights(a, head);
  const int k = (kb.first > kb.h1 ? kb.first : kb.h1) + unit - 1;
  const int o = k - ((k - kb.h0) & ~(KV8_RING_BLOCKS - 1));  // the block of [h0, h0 + 16) with k's ring slots
  if (o < k && o <= kb.old_last) {
    const int pos = SINK + o * KV8_BLK;
    quantise_block<TYPE>(a, b, h, side, o, lane, [&](int t) {
      const int q = pos + t;
      return q < p.L ? (const __nv_bfloat16*)(ring + (size_t)((q - SINK) & (RECENT - 1)) * D)
                     : in + (size_t)(q - p.L) * in_row;
    });
    if (wts && side == 0 && lane == 0) wts[KV8_RING_BLOCKS + o] = wts[o & (KV8_RING_BLOCKS - 1)];
    __syncwarp();  // every lane has read its rows of the block that leaves
  }
  const int p0 = SINK + k * KV8_BLK;
  const int from = p0 > p.L ? p0 : p.L, to = p0 + KV8_BLK < p.L1 ? p0 + KV8_BLK : p.L1;
  for (int t = from + (lane >> 4); t < to; t += 2)
    ((uint4*)(ring + (size_t)((t - SINK) & (RECENT - 1)) * D))[lane & 15] =
        ((const uint4*)(in + (size_t)(t - p.L) * in_row))[lane & 15];
  if (wts && side == 0 && lane == 0 && k > kb.old_last) wts[k & (KV8_RING_BLOCKS - 1)] = 0.f;
}

__device__ __forceinline__ int window_units_of(const AppendBlocks& k) {
  const int from = k.first > k.h1 ? k.first : k.h1;
  return 1 + (k.last >= from ? k.last - from + 1 : 0);
}

// Fewer than 256 tokens (so that none of them can leave the window in the call
// that brings it) and few tasks: one CTA per request, which writes the lengths
// when all its warps are done.  blockIdx.x: the request.
template <int TYPE>
__global__ void __launch_bounds__(AW * 32) append_small_kernel(Kv8Append a) {
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.x;
  const AppendPlan p = append_plan(a.cv, b, a.T);
  if (p.err) {
    if (threadIdx.x == 0) record_error(a.cv.err, p.err);
    return;
  }
  const AppendBlocks kb = append_blocks(p);
  const int tasks = window_units_of(kb) * a.cv.Hkv * 2;
  for (int w = threadIdx.x >> 5; w < tasks; w += AW)
    append_window<TYPE>(a, p, kb, b, (w >> 1) % a.cv.Hkv, w & 1, (w >> 1) / a.cv.Hkv, threadIdx.x & 31);
  __syncthreads();
  if (threadIdx.x == 0) {
    a.cv.seq_lens[b] = p.L1;
    a.cv.hist_lens[b] = p.H1;
  }
}

// Any number of tokens (blockIdx.y: the request).  The first gridDim.x - spans CTAs
// do the window; the others AP_SHARE tasks per warp of the blocks that fall out
// of the window at once: they have new tokens only and are quantised straight
// from the input, a warp per block, kv head and side.  Each warp copies its next
// rows to shared memory (cp.async) while it works on the present ones.  CTAs are
// small and many, six to an SM: SMs differ in how fast the memory serves them, and
// one even share for each SM left a fifth of the time idle.  append_lengths_kernel
// writes the lengths.
// Bound by memory: a 100K prompt of 8 kv heads (412 MB read, 205 MB written) takes
// 99 us with all launches, 6.2 TB/s; a plain kernel that reads and writes as much in
// order reaches 6.8.  16 warps an SM with three stages each: 105; shares of 12 or 16
// tasks: 103 to 106; even shares, one CTA per SM: 115.
// A request that is refused keeps its window and lengths; places behind the end
// of its history may have been written.
constexpr int PW = 4;        // warps per CTA
constexpr int AP_SHARE = 8;  // tasks per warp
constexpr int AP_DEPTH = 2;
constexpr int AP_ROW = D * 2 + 16;  // a row's place: rows start in different banks
constexpr int AP_STAGE = KV8_BLK * AP_ROW;

__device__ __forceinline__ void copy16_async(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

template <int TYPE>
__global__ void __launch_bounds__(PW * 32, 6) append_kernel(Kv8Append a, int spans) {
  extern __shared__ __align__(128) uint8_t smem[];
  pdl_wait();
  pdl_launch_dependents();  // after the wait: append_lengths_kernel looks before its own
  const CacheView& cv = a.cv;
  const int b = blockIdx.y, Hkv = cv.Hkv, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int windows = gridDim.x - spans;
  if ((int)blockIdx.x < windows) {
    const AppendPlan p = append_plan(cv, b, a.T);
    if (p.err) return;
    const AppendBlocks kb = append_blocks(p);
    const int tasks = window_units_of(kb) * Hkv * 2;
    for (int w = blockIdx.x * PW + warp; w < tasks; w += windows * PW)
      append_window<TYPE>(a, p, kb, b, (w >> 1) % Hkv, w & 1, (w >> 1) / Hkv, lane);
    return;
  }
  const AppendPlan p = append_lengths(cv, b, a.T);
  if (p.err) return;
  const AppendBlocks kb = append_blocks(p);
  const int d0 = kb.h0 > kb.old_last + 1 ? kb.h0 : kb.old_last + 1;  // blocks d0 .. h1 - 1 come from the input alone
  const size_t in_row = (size_t)Hkv * D;
  // task i of the span and warp: block d0 + (its number) / (2 Hkv), 2 head + side the rest
  const int width = 2 * Hkv;
  const long long t0 = (long long)(blockIdx.x - windows) * (PW * AP_SHARE) + warp;
  struct Task {
    int k, s;
  };
  auto forward = [&](Task& t) {
    t.k += PW / width;
    t.s += PW % width;
    if (t.s >= width) {
      t.s -= width;
      ++t.k;
    }
  };
  uint8_t* ring = smem + warp * AP_DEPTH * AP_STAGE;
  auto fetch = [&](const Task& t, int i) {
    if (i < AP_SHARE && t.k < kb.h1) {
      const __nv_bfloat16* src = (t.s & 1 ? a.v : a.k) +
                                 ((size_t)b * a.T + (SINK + t.k * KV8_BLK - p.L)) * in_row + (size_t)(t.s >> 1) * D;
      uint8_t* dst = ring + i % AP_DEPTH * AP_STAGE;
#pragma unroll
      for (int r = 0; r < KV8_BLK; r += 2) {
        const int row = r + (lane >> 4);
        copy16_async(dst + row * AP_ROW + 16 * (lane & 15), (const uint8_t*)(src + row * in_row) + 16 * (lane & 15));
      }
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");  // (an empty one past the end, so that the count holds)
  };
  Task now = {d0 + (int)(t0 / width), (int)(t0 % width)}, next = now;
#pragma unroll 1
  for (int i = 0; i < AP_DEPTH - 1; ++i, forward(next)) fetch(next, i);
#pragma unroll 1
  for (int i = 0; i < AP_SHARE && now.k < kb.h1; ++i, forward(now), forward(next)) {
    fetch(next, i + AP_DEPTH - 1);
    asm volatile("cp.async.wait_group %0;\n" ::"n"(AP_DEPTH - 1) : "memory");
    __syncwarp();
    const uint8_t* st = ring + i % AP_DEPTH * AP_STAGE;
    const int h = now.s >> 1, side = now.s & 1;
    const int pid = cv.page_table[(size_t)b * cv.max_pages_per_req + now.k / KV8_PAGE_BLOCKS];
    if (pid >= 0 && pid < cv.num_pages) {
      quantise_block<TYPE>(a, b, h, side, now.k, lane, [&](int t) { return (const __nv_bfloat16*)(st + t * AP_ROW); });
      if (side == 0 && lane == 0)
        if (float* wts = block_weights(a, (size_t)b * Hkv + h)) wts[KV8_RING_BLOCKS + now.k] = 0.f;
    }
    __syncwarp();  // every lane has read the stage
  }
}

// After append_kernel, which leaves the lengths as they are: the plan is made
// again while that still runs, past the L1 (kv8_req).  Made after the wait it was 0.5 us
// more for a chunk, 2.5 us for a prompt of 100K.
__global__ void __launch_bounds__(128) append_lengths_kernel(Kv8Append a) {
  pdl_launch_dependents();
  const AppendPlan p = append_plan(a.cv, blockIdx.x, a.T, true);
  pdl_wait();
  if (threadIdx.x != 0) return;
  if (p.err) {
    record_error(a.cv.err, p.err);
  } else {
    a.cv.seq_lens[blockIdx.x] = p.L1;
    a.cv.hist_lens[blockIdx.x] = p.H1;
  }
}

// ------------------------------------------------------------------ eviction
constexpr int EVICT_HELD = 50 * 1024;  // keys kept in shared memory (200 KB)

// Unsigned keys in the order of the floats, -0 as 0, NaN last.
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(__fadd_rn(w, 0.f));
  if (w != w) return 0xffffffffu;
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// Sum over the lower warps of the block (returned) and over all (*all) of v,
// which is the same in all lanes of a warp.  Calls alternate between two
// arrays `red`, so one barrier each is enough.
template <int ET>
__device__ __forceinline__ int warps_scan(int v, int* red, int* all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  const int n = lane < ET / 32 ? red[lane] : 0;
  *all = __reduce_add_sync(0xffffffffu, n);
  return __reduce_add_sync(0xffffffffu, lane < warp ? n : 0);
}

// The blocks of one (request, kv head) that go: the e smallest weights, the
// lower index first among equal ones.  Of the n - e that stay, those beyond
// place n - e move into the places below it that become free; both lists are
// in ascending order and equally long.
// The keys are read once into shared memory (the first `held`; a history beyond
// 800K tokens reads the others again).  The time is latency and the barriers of
// some ten short phases, each run once (fetching its code is part of it, so
// loops are hardly unrolled).  A digit is 11 bits: the weights fall apart into
// about a hundred first digits, and the second digit nearly always decides
// (eight bits took four passes of 0.7 us).  For 530 blocks it takes 4 us, for 6000
// 9 us; with a cluster of four CTAs per (request, kv head) and one histogram a whole
// eviction of 6000 blocks took 60.5 us instead of 62.1, one of 530 13.2 instead of 10.4.
template <int ET>
__global__ void __launch_bounds__(ET) evict_select_kernel(Kv8Evict a, int held) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) int hist[2048];
  __shared__ int red[2][ET / 32], found[3];
  pdl_wait();
  pdl_launch_dependents();
  constexpr int BINS = 2048 / ET;
  const CacheView& cv = a.cv;
  const int b = blockIdx.x / cv.Hkv, tid = threadIdx.x, lane = tid & 31;
  int32_t* list = a.list + (size_t)blockIdx.x * kv8_evict_stride(cv.max_pages_per_req);
  const float* w = a.weights + (size_t)blockIdx.x * (KV8_RING_BLOCKS + (size_t)KV8_PAGE_BLOCKS * cv.max_pages_per_req) +
                   KV8_RING_BLOCKS;
  const Kv8Req r = kv8_req(cv, b);
  const int n = r.H / KV8_BLK;
  // whole turns of the ring, so that the window's tokens keep their slots
  int e = r.H > a.budget ? (r.H - a.budget) / RECENT * KV8_RING_BLOCKS : 0;
  int err = r.ok ? 0 : OSCAR_ERR_STATE;
  if (e) {
    for (int i = tid; i < 2048; i += ET) hist[i] = 0;
    int bad = 0;
    for (int pg = tid; pg < (r.H + PAGE - 1) / PAGE; pg += ET) {
      const int id = cv.page_table[(size_t)b * cv.max_pages_per_req + pg];
      if (id < 0) bad |= 1;
      if (id >= cv.num_pages) bad |= 2;
    }
    const int end = n < held ? n : held;
#pragma unroll 4
    for (int i = tid; i < end; i += ET) keys[i] = order_key(w[i]);
    if (__syncthreads_or(bad)) err = __syncthreads_or(bad & 1) ? OSCAR_ERR_NO_PAGE : OSCAR_ERR_RANGE;
  }
  if (err) e = 0;
  if (tid == 0) {
    if (err) record_error(cv.err, err);
    list[1] = e * KV8_BLK;
    if (!e) list[0] = 0;
  }
  if (!e) return;
  auto key_of = [&](int i) { return i < held ? keys[i] : order_key(w[i]); };
  // the e-th smallest key, a digit at a time, until all keys that agree with it go:
  // how many of the keys that agree so far have each next digit.  A warp's keys
  // that share lane 0's digit count as one (equal weights, zeros above all, are common).
  uint32_t cut = 0;  // its bits from `shift` on
  int want = e;      // its rank among those that agree, from 1
  int agree = n, shift = 32;
  while (shift > 0 && want < agree) {
    const int bits = shift > 11 ? 11 : shift, to = shift - bits;
    const uint32_t mask = (1u << bits) - 1u;
#pragma unroll 4
    for (int i0 = tid - lane; i0 < n; i0 += ET) {
      const int i = i0 + lane;
      const uint32_t key = i < n ? key_of(i) : 0;
      const bool in = i < n && (shift == 32 || key >> shift == cut);
      const uint32_t digit = in ? key >> to & mask : ~0u;
      const uint32_t common = __shfl_sync(0xffffffffu, digit, 0);
      const uint32_t same = __ballot_sync(0xffffffffu, digit == common);
      if (in && (lane == 0 || digit != common)) atomicAdd(&hist[digit], lane == 0 ? __popc(same) : 1);
    }
    __syncthreads();
    // BINS bins a thread: how many keys stand in lower ones
    int c[BINS], own = 0;
#pragma unroll
    for (int j = 0; j < BINS; ++j) own += c[j] = hist[BINS * tid + j];
    int below = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, below, o);
      if (lane >= o) below += x;
    }
    if (lane == 31) red[0][tid >> 5] = below;
#pragma unroll
    for (int j = 0; j < BINS; ++j) hist[BINS * tid + j] = 0;
    __syncthreads();
    below += __reduce_add_sync(0xffffffffu, lane < (tid >> 5) ? red[0][lane] : 0) - own;
    if (below < want && want <= below + own) {
#pragma unroll
      for (int j = 0; j < BINS; ++j) {
        if (below < want && want <= below + c[j]) {
          found[0] = BINS * tid + j;
          found[1] = below;
          found[2] = c[j];
        }
        below += c[j];
      }
    }
    __syncthreads();
    cut = (shift == 32 ? 0u : cut << bits) | (uint32_t)found[0];
    want -= found[1];
    agree = found[2];
    shift = to;
  }
  // now a block goes if its key is below the cut (in the bits from `shift` on), or
  // agrees with it and is among the first `want` that do
  const int keep = n - e, warp = tid >> 5;
  const uint32_t lower = (1u << lane) - 1u;
  const int chunks = (n + 31) / 32, share = (chunks + ET / 32 - 1) / (ET / 32);  // 32 keys each; a warp's are in a row
  const int c0 = warp * share, c1 = min(c0 + share, chunks);
  int first = 0, all;  // agreeing keys before this warp's
  if (want < agree) {  // (when all that agree go, their order does not matter)
    int v = 0;
#pragma unroll 4
    for (int c = c0; c < c1; ++c) {
      const int i = 32 * c + lane;
      v += __popc(__ballot_sync(0xffffffffu, i < n && key_of(i) >> shift == cut));  // (shift < 32 here)
    }
    first = warps_scan<ET>(v, red[0], &all);
  }
  int32_t* holes = list + 4;
  int32_t* ends = holes + 2 * (size_t)cv.max_pages_per_req;
  int nh = 0, ne = 0;  // counts; then, in the second turn, the places to write to
#pragma unroll 1
  for (int turn = 0; turn < 2; ++turn) {
    int rank = first;
#pragma unroll 4
    for (int c = c0; c < c1; ++c) {
      const int i = 32 * c + lane;
      const uint32_t key = i < n && shift < 32 ? key_of(i) >> shift : 0u;
      const uint32_t eq = __ballot_sync(0xffffffffu, i < n && key == cut);
      const bool go = i < n && (key < cut || (key == cut && (want >= agree || rank + __popc(eq & lower) < want)));
      rank += __popc(eq);
      const bool hole = go && i < keep, end = !go && i >= keep && i < n;
      const uint32_t mh = __ballot_sync(0xffffffffu, hole), me = __ballot_sync(0xffffffffu, end);
      if (turn) {
        if (hole) holes[nh + __popc(mh & lower)] = i;
        if (end) ends[ne + __popc(me & lower)] = i;
      }
      nh += __popc(mh);
      ne += __popc(me);
    }
    if (turn == 0) {
      nh = warps_scan<ET>(nh, red[1], &all);
      if (tid == 0) list[0] = all;
      ne = warps_scan<ET>(ne, red[0], &all);
    }
  }
}

// Moves the listed blocks, a warp each, and takes the evicted tokens off the
// lengths.  Sources lie at or beyond the history's new end, targets before it.
// Bound by memory: 263 MB (32K blocks of 4104 B read and written) in 41 us,
// 0.94 of the measured HBM rate.  16 CTAs per SM: with four, one even share each,
// an eviction of 100K tokens to 20K took 4 us longer.
__global__ void __launch_bounds__(256) evict_move_kernel(Kv8Evict a) {
  pdl_launch_dependents();
  pdl_wait();
  const CacheView& cv = a.cv;
  const int seg = blockIdx.x, b = seg / cv.Hkv, h = seg % cv.Hkv;
  const int32_t* list = a.list + (size_t)seg * kv8_evict_stride(cv.max_pages_per_req);
  const int count = list[0];
  const int32_t* holes = list + 4;
  const int32_t* ends = holes + 2 * (size_t)cv.max_pages_per_req;
  const int32_t* pt = cv.page_table + (size_t)b * cv.max_pages_per_req;
  float* w = a.weights + (size_t)seg * (KV8_RING_BLOCKS + (size_t)KV8_PAGE_BLOCKS * cv.max_pages_per_req) + KV8_RING_BLOCKS;
  const int lane = threadIdx.x & 31, step = gridDim.y * 8;
  int i = blockIdx.y * 8 + (threadIdx.x >> 5);
  int to = 0, from = 0, tp = 0, fp = 0;  // the move's blocks and pages, fetched one move ahead
  auto fetch = [&](int k) {
    if (k < count) {
      to = holes[k];
      from = ends[k];
      tp = pt[to / KV8_PAGE_BLOCKS];
      fp = pt[from / KV8_PAGE_BLOCKS];
    }
  };
  fetch(i);
  for (; i < count; i += step) {
    const int t = to, f = from, ts = t % KV8_PAGE_BLOCKS, fs = f % KV8_PAGE_BLOCKS;
    uint8_t* tb = kv8_head(cv, tp, h);
    const uint8_t* fb = kv8_head(cv, fp, h);
    const uint4* src = (const uint4*)(fb + fs * KV8_BLOCK_BYTES) + lane;
    uint4* dst = (uint4*)(tb + ts * KV8_BLOCK_BYTES) + lane;
    uint4 x[KV8_BLOCK_BYTES / 512];
#pragma unroll
    for (int j = 0; j < KV8_BLOCK_BYTES / 512; ++j) x[j] = src[32 * j];
    fetch(i + step);
    float2 scales;
    float weight;
    if (lane == 0) {
      scales = ((const float2*)(fb + KV8_OFF_SCALES))[fs];
      weight = w[f];
    }
#pragma unroll
    for (int j = 0; j < KV8_BLOCK_BYTES / 512; ++j) dst[32 * j] = x[j];
    if (lane == 0) {
      ((float2*)(tb + KV8_OFF_SCALES))[ts] = scales;
      w[t] = weight;
    }
  }
  if (h == 0 && blockIdx.y == 0 && threadIdx.x == 0 && list[1]) {
    cv.seq_lens[b] -= list[1];
    cv.hist_lens[b] -= list[1];
  }
}

}  // namespace

template <int TYPE>
static cudaError_t launch_append_type(const Kv8Append& a, int B, cudaStream_t st) {
  const long long tasks = (((long long)a.T + KV8_BLK - 2) / KV8_BLK + 2) * a.cv.Hkv * 2;  // blocks a call can touch, and the sink
  // one launch while a CTA's warps have two tasks at most.  With 8 kv heads, and the
  // copy that resets the lengths (2 us): a step of 32 requests 5.8 us against 8.1 with
  // the two launches below, of one request 5.8 against 5.0 but a launch less for the
  // host; a chunk of 64 for four has up to twelve tasks a warp, 17.4 against 7.0.
  if (a.T < RECENT && tasks <= 2 * AW) return launch_pdl(append_small_kernel<TYPE>, dim3(B), dim3(AW * 32), 0, st, a);
  // at most 17 blocks and the sink of the window; 256 tokens or fewer cannot leave it at once
  const int windows = (18 * a.cv.Hkv * 2 + PW - 1) / PW;
  const long long direct = a.T <= RECENT ? 0 : (long long)(a.T / KV8_BLK) * a.cv.Hkv * 2;
  const int spans = (int)((direct + PW * AP_SHARE - 1) / (PW * AP_SHARE));
  static int limit[MAX_DEVICES];
  cudaError_t e = raise_smem_limit(append_kernel<TYPE>, limit, PW * AP_DEPTH * AP_STAGE);
  if (e == cudaSuccess)
    e = launch_pdl(append_kernel<TYPE>, dim3(windows + spans, B), dim3(PW * 32), PW * AP_DEPTH * AP_STAGE, st, a, spans);
  if (e == cudaSuccess) e = launch_pdl(append_lengths_kernel, dim3(B), dim3(128), 0, st, a);
  return e;
}

cudaError_t launch_kv8_append(const Kv8Append& a, int type, int B, cudaStream_t st, Profiler* prof) {
  prof_begin(prof, OSCAR_KERNEL_KV8_APPEND, st);
  const cudaError_t e = type == OSCAR_KV8_E4M3 ? launch_append_type<OSCAR_KV8_E4M3>(a, B, st)
                                               : launch_append_type<OSCAR_KV8_INT8>(a, B, st);
  prof_end(prof, OSCAR_KERNEL_KV8_APPEND, st);
  return e;
}

int kv8_evict_requests(int batch, int Hkv, int max_pages) {
  size_t n = KV8_SCRATCH_AIM / (kv8_evict_stride(max_pages) * 4 * Hkv);
  if (n < 1) n = 1;
  if (n > KV8_MAX_REQUESTS) n = KV8_MAX_REQUESTS;
  return (size_t)batch < n ? batch : (int)n;
}

size_t kv8_evict_scratch(int B, int Hkv, int max_pages) { return (size_t)B * Hkv * kv8_evict_stride(max_pages) * 4; }

template <int ET>
static cudaError_t launch_select(const Kv8Evict& a, int segs, cudaStream_t st) {
  int held = KV8_PAGE_BLOCKS * a.cv.max_pages_per_req;
  if (held > EVICT_HELD) held = EVICT_HELD;
  static int limit[MAX_DEVICES];
  const cudaError_t e = raise_smem_limit(evict_select_kernel<ET>, limit, held * 4);
  return e != cudaSuccess ? e : launch_pdl(evict_select_kernel<ET>, dim3(segs), dim3(ET), held * 4, st, a, held);
}

cudaError_t launch_kv8_evict(const Kv8Evict& a, int B, int num_sms, cudaStream_t st, Profiler* prof) {
  const int segs = B * a.cv.Hkv;
  const int per = (16 * num_sms + segs - 1) / segs;  // CTAs that move a (request, kv head)'s blocks
  prof_begin(prof, OSCAR_KERNEL_KV8_EVICT, st);
  // 16 warps select up to 4096 blocks' worth of pages (530 blocks: 11.1 us an eviction
  // against 11.6 with 32), 32 more (6000 blocks: 55 us against 58)
  cudaError_t e = KV8_PAGE_BLOCKS * a.cv.max_pages_per_req <= 4096 ? launch_select<512>(a, segs, st)
                                                                  : launch_select<1024>(a, segs, st);
  if (e == cudaSuccess) e = launch_pdl(evict_move_kernel, dim3(segs, per), dim3(256), 0, st, a);
  prof_end(prof, OSCAR_KERNEL_KV8_EVICT, st);
  return e;
}

}  // namespace oscar
