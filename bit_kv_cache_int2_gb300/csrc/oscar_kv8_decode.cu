// Decode attention over a cache with 8-bit history (sm_103a).
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(q k_j / sqrt(128)),
// over the sink, the history and the recent window, j one token each.  A
// history token's key is s_K c_K and its value s_V c_V, with 8-bit codes c and
// one scale per block of 16 tokens.
//
// kv8_decode_kernel splits the work evenly over its CTAs; each CTA writes one
// partial record per (request, kv head) it has a part of, and
// kv8_merge_kernel joins the records and adds up the blocks' weights.
//
// Every byte of the history is used once, 2 to 16 operations each: the bound is
// the memory.  A token takes an instruction or two per pair of codes to become
// FP16 and mma.m16n8k16 with the tokens as rows and the group's query heads as
// columns, so tensor cores are 17% and issue slots 30% busy at the memory's
// rate: tcgen05, whose smallest tile has 64 rows of one operand and 8 columns,
// would take the codes through shared or tensor memory once more for nothing.
// Measured (device time, with the merge; share of the measured 6.79 TB/s; cards differ):
// 8 x 131K tokens, 8 query heads a kv head, weights 322 to 330 us (0.99 to 0.97); 32
// requests of 8K to 32K, weights 207 to 211 us (0.95 to 0.93); one of 100K 33.0 to 33.5
// us (0.92 to 0.91); 2 x 131K with 2 kv heads 22.4 us (0.78); one of 1K 7.4 us, five
// trips to the memory and two launches.
#include "oscar_kv8.cuh"

namespace oscar {

namespace {

constexpr int KW = 8;   // warps per decode CTA
constexpr int MT = 256; // threads per merge CTA
// A partial record holds per query head: the largest logit m (base 2) and
// l = sum 2^(s - m); and M and o = sum 2^(s - M) v.  M is P_TOP below the largest
// t = s + log2 a, a the size of what the weight is multiplied with: a block's s_V,
// whose codes go up to 448 or 127, or a window token's own largest magnitude over
// 2^8.  The history's 2^(t - M) goes through fp16 on its way into the product
// with c_V; so what takes its bits is only a token that counts for more in the
// output (in the history with its block's largest value), not one with a larger
// logit alone, whatever the values' size.  fp16 has 11 bits down to 2^-14 and none below 2^-25:
// with P_TOP = 15 tokens keep all bits down to 2^-29 of the largest, and what is
// lost below 2^-40 of it is nothing to the sum of a million.
constexpr int REC_M = 0, REC_L = 1, REC_T = 2;
constexpr float P_TOP = 15.f;
// A record that says its part was not read (a wait ran out): m = 0, l = LOST_L,
// M = NaN, which make the output and lse NaN.  A sum of powers is never LOST_L.
constexpr float LOST_L = -INFINITY;

// ------------------------------------------------------------- the work list
// The work is a sequence of units, 16 KB each: for every (request, kv head) in
// order, the 32-token pieces of the BF16 regions that hold a token (bit i of
// the mask: 0, 1 the sink, 2 + r ring slots 32r .. 32r + 31), then the history
// pages.  CTA i of n takes units [floor(i W / n), floor((i + 1) W / n)).
__device__ __forceinline__ uint32_t window_units(int L, int H) {
  const int held = max(L - SINK - H, 0);
  uint32_t m = ((1u << ((held + KV8_BLK - 1) / KV8_BLK)) - 1u) << (H / KV8_BLK % KV8_RING_BLOCKS);
  m |= m >> KV8_RING_BLOCKS;         // ring blocks that hold a token, in the low 16 bits
  m = (m | m >> 1) & 0x5555u;        // ring units, every other bit
  m = (m | m >> 1) & 0x3333u;
  m = (m | m >> 2) & 0x0f0fu;
  m = (m | m >> 4) & 0x00ffu;
  return m << 2 | (L > 32 ? 3u : L > 0 ? 1u : 0u);
}

// The place of set bit number i of a unit mask.
__device__ __forceinline__ int nth_unit(uint32_t m, int i) {
  for (; i > 0; --i) m &= m - 1;
  return __ffs(m) - 1;
}

struct Segment {  // a request's share of the list, the same for each of its kv heads
  int L, H, pages, units;
  uint32_t win;
};

__device__ __forceinline__ Segment make_segment(int L, int H) {
  Segment s;
  s.L = L;
  s.H = H;
  s.win = window_units(L, H);
  s.pages = (H + PAGE - 1) / PAGE;
  s.units = s.pages + __popc(s.win);
  return s;
}

__device__ __forceinline__ Segment segment_of(const CacheView& cv, int b, bool early = false) {
  const Kv8Req r = kv8_req(cv, b, early);
  return make_segment(r.L, r.H);
}

// Shared memory: a ring of `stages` stages of a unit each, which units are copied
// into ahead of their use, the barriers and the warps' results.  A window unit
// is 32 key rows and then 32 value rows of 256 bytes, as they stand in memory:
// the fragments' loads conflict two and four times, but a unit is two copies
// (rows padded to 272 bytes took 64 copies, and 1.4 us to start them).
constexpr int WROW = D * 2;
constexpr int STAGE_BYTES = (KV8_HEAD_BYTES + 127) / 128 * 128;
static_assert(STAGE_BYTES >= 64 * WROW, "a window unit fits a stage");
constexpr int MAX_STAGES = 13;
// An SM has 228 KB: what is left of them, and without weights of the registers (173
// of the decode's threads, 80 of the merge's), lets a CTA of the merge plan beside a
// decode CTA; with weights it comes when that ends.
constexpr int SMEM_LIMIT = 215 * 1024;

// ------------------------------------------------------------------ the math
struct State {
  float o[8][4];  // o^T: row tile j, channels 16gid + 2j (o[j][hc]) and + 1 (o[j][hc + 2]), head 2tq + hc
  float m[2], l[2], M[2];
};

__device__ __forceinline__ void state_clear(State& S) {
#pragma unroll
  for (int j = 0; j < 8; ++j) S.o[j][0] = S.o[j][1] = S.o[j][2] = S.o[j][3] = 0.f;
  S.m[0] = S.m[1] = S.M[0] = S.M[1] = -INFINITY;
  S.l[0] = S.l[1] = 0.f;
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// q's fragments: word [c][j] holds channels 32c + 8tq + 2j, + 1 of head gid.
// As BF16 (the window's products), then as FP16 scaled by a power of two that
// brings the head's largest magnitude to [2^14, 2^15): exact but for channels
// more than 2^28 below the largest.
struct Query {
  uint32_t w[4][4];
  float alpha[2];  // of heads 2tq, 2tq + 1: log2(e) / sqrt(128), over the power of two once FP16
};

__device__ __forceinline__ void query_load(Query& Q, const __nv_bfloat16* q, int G, int gid, int tq) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (gid < G) x = *(const uint4*)(q + (size_t)gid * D + 32 * c + 8 * tq);
    Q.w[c][0] = x.x;
    Q.w[c][1] = x.y;
    Q.w[c][2] = x.z;
    Q.w[c][3] = x.w;
  }
  Q.alpha[0] = Q.alpha[1] = LOG2E * INV_SQRT_D;
}

__device__ __forceinline__ void query_to_fp16(Query& Q, int tq) {
  uint32_t mx = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) mx = __vmaxu2(mx, Q.w[c][j] & 0x7fff7fffu);
  mx = max(mx >> 16, mx & 0xffffu);
  mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  const int e = max((int)(mx >> 7) - 127, -100);
  const float f = pow2i(14 - e);
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = Q.w[c][j];
      const __half2 y = __floats2half2_rn(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xffff0000u) * f);
      Q.w[c][j] = *(const uint32_t*)&y;
    }
  const float al = LOG2E * INV_SQRT_D * pow2i(e - 14);
  Q.alpha[0] = __shfl_sync(0xffffffffu, al, 8 * tq);  // lane 4n holds head n
  Q.alpha[1] = __shfl_sync(0xffffffffu, al, 8 * tq + 4);
}

// Codes 0, 1 and 2, 3 of a word as FP16 pairs, exactly.
template <int TYPE>
__device__ __forceinline__ void codes_fp16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (TYPE == OSCAR_KV8_E4M3) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // c + 128 under the exponent of 1024, less 1152
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    uint32_t a = prmt(u, 0x64646464u, 0x4140), b = prmt(u, 0x64646464u, 0x4342);
    __half2 x = __hsub2(*(__half2*)&a, off), y = __hsub2(*(__half2*)&b, off);
    lo = *(uint32_t*)&x;
    hi = *(uint32_t*)&y;
  }
}

// One online-softmax step over NT tiles of 16 tokens.  s: the logits in base 2,
// -inf where there is no token (at least one token is there), rows gid and
// gid + 8, heads 2tq and 2tq + 1; lv: log2 a of the two rows.  On return p holds
// 2^(t - M) (SCALED, for codes) or 2^(s - M) (for values themselves), and sum[t][hc]
// this thread's part of the tile's sum of 2^(s - m).
template <bool SCALED, int NT>
__device__ __forceinline__ void softmax_step(State& S, const float (&s)[NT][4], const float (&lv)[NT][2],
                                             float (&p)[NT][4], float (&sum)[NT][2]) {
#pragma unroll
  for (int hc = 0; hc < 2; ++hc) {
    float ms = -INFINITY, mt = -INFINITY;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      ms = fmaxf(ms, fmaxf(s[t][hc], s[t][hc + 2]));
      mt = fmaxf(mt, fmaxf(s[t][hc] + lv[t][0], s[t][hc + 2] + lv[t][1]));
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      ms = fmaxf(ms, __shfl_xor_sync(0xffffffffu, ms, o));
      mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    }
    if (ms > S.m[hc]) {
      S.l[hc] *= ex2(S.m[hc] - ms);
      S.m[hc] = ms;
    }
    mt -= P_TOP;
    if (mt > S.M[hc]) {
      const float al = ex2(S.M[hc] - mt);
      S.M[hc] = mt;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        S.o[j][hc] *= al;
        S.o[j][hc + 2] *= al;
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      sum[t][hc] = ex2(s[t][hc] - S.m[hc]) + ex2(s[t][hc + 2] - S.m[hc]);
      S.l[hc] += sum[t][hc];
      p[t][hc] = ex2((SCALED ? s[t][hc] + lv[t][0] : s[t][hc]) - S.M[hc]);
      p[t][hc + 2] = ex2((SCALED ? s[t][hc + 2] + lv[t][1] : s[t][hc + 2]) - S.M[hc]);
    }
  }
}

// Block sums for the merge, [B Hkv][G][max_pages + 8]: of a page's four blocks
// (of a ring unit's two, after the pages), and the maximum they are relative to.
// The merge reads them a page per thread, so the pages are innermost.
struct Sums {
  float4* sum;
  float* max;
  size_t stride;  // from head to head
};

__device__ __forceinline__ Sums sums_at(const Kv8Decode& a, int seg, int rec) {
  const size_t stride = a.cv.max_pages_per_req + KV8_RING_UNITS;
  const size_t at = (size_t)seg * a.cv.G * stride + rec;
  return {(float4*)a.wsum + at, a.wmax + at, stride};
}

template <int NT>
__device__ __forceinline__ void write_sums(const State& S, float (&sum)[NT][2], const Sums& w, int G, int gid, int tq) {
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int hc = 0; hc < 2; ++hc)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sum[t][hc] += __shfl_xor_sync(0xffffffffu, sum[t][hc], o);
  const int n = 2 * tq + gid;  // lanes of gid 0 and 1 write a head each
  if (gid < 2 && n < G) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    float* x = (float*)&v;
#pragma unroll
    for (int t = 0; t < NT; ++t) x[t] = gid ? sum[t][1] : sum[t][0];
    w.sum[n * w.stride] = v;
    w.max[n * w.stride] = gid ? S.m[1] : S.m[0];
  }
}

// A page's blocks 0 .. nb - 1 (the others hold nothing and are not looked at).
// FULL: all four, with nothing between them that keeps their products in order.
template <int TYPE, bool WEIGHTS, bool FULL>
__device__ __forceinline__ void page_step(State& S, const Query& Q, const uint8_t* page, int nb, int lane, int G,
                                          const Sums& w) {
  const int gid = lane >> 2, tq = lane & 3;
  float s[4][4], lv[4][2];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    s[t][0] = s[t][1] = s[t][2] = s[t][3] = -INFINITY;
    lv[t][0] = lv[t][1] = 0.f;
    if (FULL || t < nb) {
      float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint4 k = *(const uint4*)(page + t * KV8_BLOCK_BYTES + c * 512 + lane * 16);
        uint32_t a0, a1, a2, a3;
        codes_fp16<TYPE>(k.x, a0, a1);
        codes_fp16<TYPE>(k.y, a2, a3);
        mma_f16(a, a0, a1, a2, a3, Q.w[c][0], Q.w[c][1]);
        codes_fp16<TYPE>(k.z, a0, a1);
        codes_fp16<TYPE>(k.w, a2, a3);
        mma_f16(a, a0, a1, a2, a3, Q.w[c][2], Q.w[c][3]);
      }
      const float2 sc = *(const float2*)(page + KV8_OFF_SCALES + 8 * t);
      // the append makes no scale below 2^-109; a zero (a page that nothing wrote) must not become -inf
      lv[t][0] = lv[t][1] = sc.y < 1.17549435e-38f ? -126.f : lg2(sc.y);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = a[e] * (Q.alpha[e & 1] * sc.x);
    }
  }
  float p[4][4], sum[4][2];
  softmax_step<true>(S, s, lv, p, sum);
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (FULL || t < nb) {
      const __half2 h0 = __floats2half2_rn(p[t][0], p[t][1]), h1 = __floats2half2_rn(p[t][2], p[t][3]);
      const uint32_t b0 = movmatrix_t(*(const uint32_t*)&h0), b1 = movmatrix_t(*(const uint32_t*)&h1);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint4 v = *(const uint4*)(page + t * KV8_BLOCK_BYTES + KV8_BLK * D + c * 512 + lane * 16);
        uint32_t a0, a1, a2, a3;
        codes_fp16<TYPE>(v.x, a0, a1);
        codes_fp16<TYPE>(v.y, a2, a3);
        mma_f16(S.o[2 * c], a0, a1, a2, a3, b0, b1);
        codes_fp16<TYPE>(v.z, a0, a1);
        codes_fp16<TYPE>(v.w, a2, a3);
        mma_f16(S.o[2 * c + 1], a0, a1, a2, a3, b0, b1);
      }
    }
  }
  if (WEIGHTS) write_sums<4>(S, sum, w, G, gid, tq);
}

// 32 BF16 tokens at K and V (WROW bytes from row to row), of which the first n0
// of the first 16 and the first n1 of the last 16 are there.  The others may
// hold anything: their logits become -inf and their values 0.
// The weights go into the product as two BF16 parts (16 bits together): the
// newest tokens often carry most of the weight.  A weight 2^(s - M) may be far above
// 1, where the values are small: their product is not, and BF16 takes it.
template <bool WEIGHTS>
__device__ __forceinline__ void window_step(State& S, const Query& Q, const uint8_t* K, const uint8_t* V, int n0, int n1,
                                            int lane, int G, bool sums, const Sums& w) {
  const int gid = lane >> 2, tq = lane & 3;
  // lane i: log2 of row i's largest magnitude over 2^8 (rows start at different
  // pieces, so that the banks do)
  uint32_t mx = 0;
#pragma unroll 8
  for (int j = 0; j < 16; ++j) {
    const uint4 x = *(const uint4*)(V + lane * WROW + 16 * ((lane + j) & 15));
    mx = max_abs2(max_abs2(max_abs2(max_abs2(mx, x.x), x.y), x.z), x.w);
  }
  mx = max(mx >> 16, mx & 0xffffu);
  if (mx >= 0x7f80u && (lane & 15) < (lane < 16 ? n0 : n1)) {
    // an infinity or NaN shows in its own channel: the others go by the row's finite values
    mx = 0;
#pragma unroll 1
    for (int j = 0; j < D; ++j) {
      const uint32_t x = ((const uint16_t*)(V + lane * WROW))[j] & 0x7fffu;
      if (x < 0x7f80u) mx = max(mx, x);
    }
  }
  const float row = mx >= 0x7f80u ? 0.f : lg2(fmaxf(__uint_as_float(mx << 16), KV8_TINY)) - 8.f;
  float s[2][4], lv[2][2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int n = t ? n1 : n0;
    lv[t][0] = __shfl_sync(0xffffffffu, row, 16 * t + gid);
    lv[t][1] = __shfl_sync(0xffffffffu, row, 16 * t + 8 + gid);
    float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 x = *(const uint4*)(K + (16 * t + gid) * WROW + 64 * c + 16 * tq);
      const uint4 y = *(const uint4*)(K + (16 * t + 8 + gid) * WROW + 64 * c + 16 * tq);
      mma_bf16(a, x.x, y.x, x.y, y.y, Q.w[c][0], Q.w[c][1]);
      mma_bf16(a, x.z, y.z, x.w, y.w, Q.w[c][2], Q.w[c][3]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) s[t][e] = (e < 2 ? gid : gid + 8) < n ? a[e] * Q.alpha[e & 1] : -INFINITY;
  }
  float p[2][4], sum[2][2];
  softmax_step<false>(S, s, lv, p, sum);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int n = t ? n1 : n0;
    if (n == 0) continue;
    uint32_t bh[2], bl[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const __nv_bfloat162 hi = __floats2bfloat162_rn(p[t][2 * r], p[t][2 * r + 1]);
      const float2 f = __bfloat1622float2(hi);
      const __nv_bfloat162 lo = __floats2bfloat162_rn(p[t][2 * r] - f.x, p[t][2 * r + 1] - f.y);
      bh[r] = movmatrix_t(*(const uint32_t*)&hi);
      bl[r] = movmatrix_t(*(const uint32_t*)&lo);
    }
    uint32_t v[4][8];  // rows 2tq, 2tq + 1, 8 + 2tq, 9 + 2tq, channels 16gid ..
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int row = 8 * (u >> 1) + 2 * tq + (u & 1);
      const uint4* src = (const uint4*)(V + (16 * t + row) * WROW + 32 * gid);
      const uint4 x = src[0], y = src[1];
      const bool in = row < n;
      v[u][0] = in ? x.x : 0u, v[u][1] = in ? x.y : 0u, v[u][2] = in ? x.z : 0u, v[u][3] = in ? x.w : 0u;
      v[u][4] = in ? y.x : 0u, v[u][5] = in ? y.y : 0u, v[u][6] = in ? y.z : 0u, v[u][7] = in ? y.w : 0u;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t a0 = prmt(v[0][j], v[1][j], 0x5410), a1 = prmt(v[0][j], v[1][j], 0x7632);
      const uint32_t a2 = prmt(v[2][j], v[3][j], 0x5410), a3 = prmt(v[2][j], v[3][j], 0x7632);
      mma_bf16(S.o[j], a0, a1, a2, a3, bh[0], bh[1]);
      mma_bf16(S.o[j], a0, a1, a2, a3, bl[0], bl[1]);
    }
  }
  if (WEIGHTS && sums) write_sums<2>(S, sum, w, G, gid, tq);
}

// ------------------------------------------------------------------- decode
struct DecodeSmem {
  int stages, off_bar, off_issued, off_comb, total;
};
__host__ __device__ constexpr DecodeSmem decode_smem(int G) {
  const int comb = KW * G * PART_STRIDE * 4;
  DecodeSmem s = {};
  s.stages = (SMEM_LIMIT - 256 - comb) / STAGE_BYTES;
  if (s.stages > MAX_STAGES) s.stages = MAX_STAGES;
  s.off_bar = s.stages * STAGE_BYTES;
  s.off_issued = s.off_bar + 128;
  s.off_comb = s.off_issued + 128;
  s.total = s.off_comb + comb;
  return s;
}
// eight warps take the units in turn, so more than eight stages keep all of them busy
static_assert(decode_smem(MAX_G).stages > KW, "stages at the largest group");

// Sum over the warp's lanes, and over the lanes below.
__device__ __forceinline__ uint32_t warp_scan(uint32_t v, uint32_t* all) {
  const int lane = threadIdx.x & 31;
  uint32_t upto = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  *all = __shfl_sync(0xffffffffu, upto, 31);
  return upto - v;
}

// Request b; empty beyond the batch.
__device__ __forceinline__ Segment segment_or_none(const CacheView& cv, int B, int b, bool early = false) {
  return b < B ? segment_of(cv, b, early) : make_segment(0, 0);
}

// A position in the work list.
struct Cursor {
  Segment sg;
  int b, h, i;  // unit i of (b, h)
};

// CTA i of `grid`: its first unit in c, and how many it has (0: none, c is not
// set).  A whole warp calls it; every warp finds its CTA's share by itself.  Early,
// before the wait, the lengths may change under it: then the answer is of no
// use, but every read stays in range.
// `mine`: request `lane`, as it was read.
__device__ __forceinline__ int cta_share(Cursor& c, Segment& mine, const CacheView& cv, int B, uint32_t i, uint32_t grid,
                                         bool early) {
  const int lane = threadIdx.x & 31;
  Segment own = segment_or_none(cv, B, lane, early);
  mine = own;
  uint32_t units = (uint32_t)(own.units * cv.Hkv), sum;
  uint32_t below = warp_scan(units, &sum);
  unsigned long long W = sum;
  for (int b0 = 32; b0 < B; b0 += 32)
    W += __reduce_add_sync(0xffffffffu, (uint32_t)(segment_or_none(cv, B, b0 + lane, early).units * cv.Hkv));
  const uint32_t n = W < grid ? (uint32_t)W : grid;
  if (i >= n) return 0;
  // floor(i W / n) with one division by n
  unsigned long long q;
  uint32_t r;
  if (W >> 32 == 0) {
    q = (uint32_t)W / n;
    r = (uint32_t)W - (uint32_t)q * n;
  } else {
    q = W / n;
    r = (uint32_t)(W - q * n);
  }
  const unsigned long long u0 = q * i + i * r / n;
  const int count = (int)(q * (i + 1) + (i + 1) * r / n - u0);
  unsigned long long before = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    if (b0) {
      own = segment_or_none(cv, B, b0 + lane, early);
      units = (uint32_t)(own.units * cv.Hkv);
      below = warp_scan(units, &sum);
    }
    if (u0 < before + sum) {
      const uint32_t u = (uint32_t)(u0 - before);
      const int l = __ffs(__ballot_sync(0xffffffffu, below + units > u)) - 1;
      c.b = b0 + l;
      c.sg = make_segment(__shfl_sync(0xffffffffu, own.L, l), __shfl_sync(0xffffffffu, own.H, l));
      const uint32_t v = u - __shfl_sync(0xffffffffu, below, l);
      c.h = (int)(v / (uint32_t)c.sg.units);
      c.i = (int)(v - (uint32_t)c.h * c.sg.units);
      return count;
    }
    before += sum;
  }
  return 0;
}

// Forward by n units; false at the end of the list.
__device__ __forceinline__ bool cursor_forward(Cursor& c, const CacheView& cv, int B, int n, bool early = false) {
  c.i += n;
  while (c.i >= c.sg.units) {
    c.i -= c.sg.units;
    if (++c.h == cv.Hkv) {
      c.h = 0;
      do {
        if (++c.b >= B) return false;
        c.sg = segment_of(cv, c.b, early);
      } while (c.sg.units == 0);
    }
  }
  return true;
}

// The page of the unit at c (any number for a window unit).
__device__ __forceinline__ int cursor_page(const Cursor& c, const CacheView& cv, bool early = false) {
  const int pg = c.i - __popc(c.sg.win);
  if (pg < 0) return 0;
  const int32_t* p = cv.page_table + (size_t)c.b * cv.max_pages_per_req + pg;
  return early ? __ldcg(p) : *p;
}

// A hint to bring the unit at c into the L2 (lane 0).
__device__ __forceinline__ void prefetch_unit(const Cursor& c, const CacheView& cv, int pid) {
  if (c.i < __popc(c.sg.win)) {
    const int unit = nth_unit(c.sg.win, c.i);
    const size_t seg = (size_t)c.b * cv.Hkv + c.h;
    const size_t row = unit < 2 ? seg * SINK + 32 * unit : seg * RECENT + 32 * (unit - 2);
    bulk_prefetch_l2((unit < 2 ? cv.sink_k : cv.ring_k) + row * D, 32 * WROW);
    bulk_prefetch_l2((unit < 2 ? cv.sink_v : cv.ring_v) + row * D, 32 * WROW);
  } else if (pid >= 0 && pid < cv.num_pages) {
    bulk_prefetch_l2(kv8_head(cv, pid, c.h), KV8_HEAD_BYTES);
  }
}

// A warp starts the copy of the unit at c into a stage.
__device__ __forceinline__ void issue_unit(const Cursor& c, const CacheView& cv, int pid, uint8_t* stage, uint64_t* bar,
                                           int* issued, int lane) {
  if (lane == 0) ++*issued;
  if (c.i < __popc(c.sg.win)) {
    const int unit = nth_unit(c.sg.win, c.i);
    const size_t seg = (size_t)c.b * cv.Hkv + c.h;
    const size_t row = unit < 2 ? seg * SINK + 32 * unit : seg * RECENT + 32 * (unit - 2);
    if (lane == 0) {
      mbar_expect_tx(bar, 64 * WROW);
      bulk_g2s(stage, (unit < 2 ? cv.sink_k : cv.ring_k) + row * D, 32 * WROW, bar);
      bulk_g2s(stage + 32 * WROW, (unit < 2 ? cv.sink_v : cv.ring_v) + row * D, 32 * WROW, bar);
    }
  } else if (lane == 0) {
    if (pid >= 0 && pid < cv.num_pages) {
      mbar_expect_tx(bar, KV8_HEAD_BYTES);
      bulk_g2s_hint(stage, kv8_head(cv, pid, c.h), KV8_HEAD_BYTES, bar, l2_evict_first_policy());
    } else {
      record_error(cv.err, pid < 0 ? OSCAR_ERR_NO_PAGE : OSCAR_ERR_RANGE);
      mbar_expect_tx(bar, 0);
    }
  }
}

// Waits until the copy number `use` (from 0) into a stage has arrived.  A
// barrier tells apart only odd and even phases, and the warp that waits may be
// one whole turn of the ring ahead of the copy before: it first waits until its
// own copy has been started, which is after the one before was read.
__device__ __forceinline__ bool wait_unit(uint64_t* bar, const int* issued, int use, int polls) {
  for (int it = 0; *(const volatile int*)issued <= use; ++it)
    if (it >= polls) return false;
  return mbar_wait(bar, use & 1, polls);
}

// One persistent CTA per SM.  Unit i of its range goes to warp i % 8 and
// through stage i % stages; the warp that has read a stage starts the copy
// that comes into it next, whoever will read that, so a stage needs no barrier
// that says it is free.  Each warp keeps a softmax state of its own over its
// units of a (request, kv head); they are joined when the CTA is through with
// it.
template <int TYPE, bool WEIGHTS>
__global__ void __launch_bounds__(KW * 32, 1) kv8_decode_kernel(Kv8Decode a) {
  extern __shared__ __align__(128) uint8_t smem[];
  const CacheView& cv = a.cv;
  const DecodeSmem SL = decode_smem(cv.G);
  const int NS = SL.stages;
  uint64_t* bars = (uint64_t*)(smem + SL.off_bar);
  int* issued = (int*)(smem + SL.off_issued);  // copies started into each stage; [MAX_STAGES]: a wait ran out
  float* comb = (float*)(smem + SL.off_comb);  // [warp][head] partial records
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tq = lane & 3;
  const int G = cv.G, Hkv = cv.Hkv, B = a.B;
  if (threadIdx.x <= MAX_STAGES) {
    issued[threadIdx.x] = 0;
    if (threadIdx.x < NS) mbar_init(&bars[threadIdx.x], 1);
  }
  fence_proxy_async();
  __syncthreads();
  // The CTA's share and the warp's first units are found before the wait, from
  // lengths and pages that the kernel before may still change, to have the code
  // and the data at hand (the L2 prefetch is a hint).  After it they stand if
  // every request still has the units it had (a step seldom changes them), with
  // the lengths and the page read again, together: one trip to the L2 instead of
  // two; else they are found again.
  const bool two = warp + KW < NS;  // the warp fills two stages at the start
  Cursor c, ic;                     // the CTA's first unit; the warp's next unit to copy, and its page
  int count, next = warp, pid = 0;
#pragma unroll 1
  for (bool early = true;; early = false) {
    Segment mine;
    count = cta_share(c, mine, cv, B, blockIdx.x, a.grid, early);
    ic = c;
    bool more = next < count;
    if (more) more = cursor_forward(ic, cv, B, next, early);
    if (more) pid = cursor_page(ic, cv, early);
    if (!early) break;
    if (lane == 0 && more) {
      prefetch_unit(ic, cv, pid);
      Cursor ahead = ic;
      if (two && next + KW < count && cursor_forward(ahead, cv, B, KW, true))
        prefetch_unit(ahead, cv, cursor_page(ahead, cv, true));
    }
    __syncwarp();
    pdl_wait();
    pdl_launch_dependents();  // after the wait: what the merge reads before its own wait is there
    if (B <= 32 && (next >= count || (more && ic.b == c.b))) {
      if (more) pid = cursor_page(ic, cv);
      const Segment now = segment_or_none(cv, B, lane);
      if (__all_sync(0xffffffffu, now.units == mine.units && now.win == mine.win)) {
        if (count > 0) {
          c.sg = make_segment(__shfl_sync(0xffffffffu, now.L, c.b), __shfl_sync(0xffffffffu, now.H, c.b));
          if (more) ic.sg = c.sg;
        }
        break;
      }
    }
  }
  if (count == 0) return;
  auto issue_next = [&](int stage, int step) {  // then moves on by `step` units
    if (next < count) {
      issue_unit(ic, cv, pid, smem + stage * STAGE_BYTES, &bars[stage], &issued[stage], lane);
      next += step;
      if (next < count) {
        cursor_forward(ic, cv, B, step);
        pid = cursor_page(ic, cv);
      }
    }
  };
  issue_next(warp, two ? KW : NS);
  if (two) issue_next(warp + KW, NS - KW);

  int first = 0;           // this CTA's first unit of (c.b, c.h)
  int mine = warp;         // this warp's next unit, its stage and the copies into that before it
  int stage = warp, use = 0;
  while (first < count) {
    const int lo = c.i, len = min(count - first, c.sg.units - lo);
    const int nwin = __popc(c.sg.win), seg = c.b * Hkv + c.h;
    State S;
    state_clear(S);
    Query Q;
    bool fp16 = false;
    query_load(Q, a.q + ((size_t)c.b * cv.Hq + (size_t)c.h * G) * D, G, gid, tq);
    for (; mine < first + len; mine += KW) {
      const int i = lo + mine - first;
      if (!__all_sync(0xffffffffu, wait_unit(&bars[stage], &issued[stage], use, a.wait_polls))) {
        if (lane == 0) {
          record_error(cv.err, OSCAR_ERR_TIMEOUT);
          issued[MAX_STAGES] = 1;
        }
        break;
      }
      const uint8_t* st = smem + stage * STAGE_BYTES;
      if (i < nwin) {
        const int unit = nth_unit(c.sg.win, i), r = unit - 2;
        const bool sink = unit < 2;
        const int n0 = sink ? min(max(c.sg.L - 32 * unit, 0), 16) : kv8_ring_held(c.sg.L, c.sg.H, 2 * r);
        const int n1 = sink ? min(max(c.sg.L - 32 * unit - 16, 0), 16) : kv8_ring_held(c.sg.L, c.sg.H, 2 * r + 1);
        window_step<WEIGHTS>(S, Q, st, st + 32 * WROW, n0, n1, lane, G, !sink,
                             sums_at(a, seg, cv.max_pages_per_req + max(r, 0)));
      } else {
        if (!fp16) query_to_fp16(Q, tq);
        fp16 = true;
        const int pg = i - nwin;
        const int id = cv.page_table[(size_t)c.b * cv.max_pages_per_req + pg];
        const Sums w = sums_at(a, seg, pg);
        if (id >= 0 && id < cv.num_pages) {
          const int nb = c.sg.H / KV8_BLK - pg * KV8_PAGE_BLOCKS;
          if (nb >= KV8_PAGE_BLOCKS) page_step<TYPE, WEIGHTS, true>(S, Q, st, KV8_PAGE_BLOCKS, lane, G, w);
          else page_step<TYPE, WEIGHTS, false>(S, Q, st, nb, lane, G, w);
        } else if (WEIGHTS && lane < G) {  // its tokens are left out
          w.sum[lane * w.stride] = make_float4(0.f, 0.f, 0.f, 0.f);
          w.max[lane * w.stride] = -INFINITY;
        }
      }
      __syncwarp();  // the stage has been read: the next copy may come into it
      issue_next(stage, KW);
      stage += KW;
      if (stage >= NS) {
        stage -= NS;
        ++use;
      }
    }
    // join the warps
#pragma unroll
    for (int hc = 0; hc < 2; ++hc) {
      S.l[hc] += __shfl_xor_sync(0xffffffffu, S.l[hc], 4);
      S.l[hc] += __shfl_xor_sync(0xffffffffu, S.l[hc], 8);
      S.l[hc] += __shfl_xor_sync(0xffffffffu, S.l[hc], 16);
      // the maxima pass NaN over, l does not: a warp that saw nothing else must not count as one without tokens
      if (S.l[hc] != 0.f) {
        if (S.m[hc] == -INFINITY) S.m[hc] = 0.f;
        if (S.M[hc] == -INFINITY) S.M[hc] = 0.f;
      }
      const int hd = 2 * tq + hc;
      if (hd < G) {
        float* x = comb + (warp * G + hd) * PART_STRIDE;
        if (gid == 0) {
          x[REC_M] = S.m[hc];
          x[REC_L] = S.l[hc];
          x[REC_T] = S.M[hc];
        }
#pragma unroll
        for (int j = 0; j < 8; j += 2)
          *(float4*)(x + PART_O + 16 * gid + 2 * j) = make_float4(S.o[j][hc], S.o[j][hc + 2], S.o[j + 1][hc], S.o[j + 1][hc + 2]);
      }
    }
    __syncthreads();
    float* rec = a.part + ((size_t)blockIdx.x + seg) * G * PART_STRIDE;
    const bool lost = issued[MAX_STAGES];  // a wait ran out: this part and the CTA's later ones are not read
    if (lost) {
      mine = count;
      if (threadIdx.x < G)
        *(float4*)(rec + threadIdx.x * PART_STRIDE) = make_float4(0.f, LOST_L, __uint_as_float(0x7fffffffu), 0.f);
    }
    for (int e = lost ? G * D : threadIdx.x; e < G * D; e += KW * 32) {
      const int hd = e / D, ch = e % D;
      float m = -INFINITY, M = -INFINITY;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        m = fmaxf(m, comb[(w * G + hd) * PART_STRIDE + REC_M]);
        M = fmaxf(M, comb[(w * G + hd) * PART_STRIDE + REC_T]);
      }
      float l = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const float* x = comb + (w * G + hd) * PART_STRIDE;
        if (x[REC_M] == -INFINITY) continue;
        l += x[REC_L] * ex2(x[REC_M] - m);
        o += x[PART_O + ch] * ex2(x[REC_T] - M);
      }
      float* y = rec + hd * PART_STRIDE;
      y[PART_O + ch] = o;
      if (ch == 0) {
        y[REC_M] = m;
        y[REC_L] = l;
        y[REC_T] = M;
      }
    }
    __syncthreads();
    first += len;
    if (first < count) cursor_forward(c, cv, B, len);
  }
  // a wait ran out: no CTA leaves with a copy into its memory under way
  if (issued[MAX_STAGES] && threadIdx.x < NS && issued[threadIdx.x])
    mbar_wait(&bars[threadIdx.x], (issued[threadIdx.x] - 1) & 1);
}

// -------------------------------------------------------------------- merge
// grid (B Hkv, G / heads + slices of the weights), heads = 2^log_heads: the first CTAs
// write the output of `heads` query heads each, MT / 32 / heads warps to a head; the others update
// a slice of the block weights.
// What is in the records of a (request, kv head) follows from the lengths, so
// one warp works it out while the decode kernel still runs, reading past the L1
// (kv8_req).  A second look at the lengths after the wait took 0.3 to 0.5 us more.
__global__ void __launch_bounds__(MT) kv8_merge_kernel(Kv8Decode a, int log_heads) {
  __shared__ __align__(16) float wo[MT / 32][D];
  __shared__ float scale[2][MT / 32];
  __shared__ float tot_m[MAX_G], tot_r[MAX_G];
  __shared__ int4 plan;
  const CacheView& cv = a.cv;
  const int seg = blockIdx.x, b = seg / cv.Hkv, h = seg % cv.Hkv, G = cv.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  if (warp == 0) {
    const Kv8Req r = kv8_req(cv, b, true);
    const Segment sg = make_segment(r.L, r.H);
    if (h == 0 && blockIdx.y == 0 && lane == 0 && !r.ok) record_error(cv.err, OSCAR_ERR_STATE);
    Balanced bl;
    bl.W = 0;
    bl.wch = 0;
    long long before = 0;
    for (int r0 = 0; r0 < a.B; r0 += 32) {
      const uint32_t x = (uint32_t)(segment_or_none(cv, a.B, r0 + lane, true).units * cv.Hkv);
      bl.W += __reduce_add_sync(0xffffffffu, x);
      before += __reduce_add_sync(0xffffffffu, r0 + lane < b ? x : 0u);
    }
    bl.n = (int)(bl.W < a.grid ? bl.W : a.grid);
    const long long s0 = before + (long long)h * sg.units;
    int i0 = 0, n = 0;
    if (sg.units) {
      i0 = balanced_owner(bl, s0);
      n = balanced_owner(bl, s0 + sg.units - 1) - i0 + 1;
    }
    if (lane == 0) plan = make_int4(i0, n, r.L, r.H);
  }
  __syncthreads();
  const int i0 = plan.x, n = plan.y;  // records i0 .. i0 + n - 1, one of each CTA that had a part
  const Segment sg = make_segment(plan.z, plan.w);
  pdl_wait();
  const float* recs = a.part + ((size_t)i0 + seg) * G * PART_STRIDE;
  const int heads = 1 << log_heads, outs = G >> log_heads;
  if ((int)blockIdx.y < outs) {
    const int per = (MT / 32) >> log_heads;  // warps to a head
    const int own_hd = (warp << log_heads) / (MT / 32), first = warp & (per - 1);
    const int hd = (blockIdx.y << log_heads) + own_hd;
    const float* rec = recs + hd * PART_STRIDE;
    const size_t stride = (size_t)G * PART_STRIDE;
    float4 y[4];  // the warp's first records, while the maxima are found
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = first + j * per;
      y[j] = i < n ? *(const float4*)(rec + i * stride + PART_O + 4 * lane) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float m = -INFINITY, M = -INFINITY, l = 0.f;
    for (int i = lane; i < n; i += 32) {
      const float4 x = *(const float4*)(rec + i * stride);
      const float mn = fmaxf(m, x.x);
      if (x.x != -INFINITY) l = l * ex2(m - mn) + x.y * ex2(x.x - mn);
      m = mn;
      M = fmaxf(M, x.z);
    }
    const float own = m;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    }
    if (own != -INFINITY) l *= ex2(own - m);
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const bool none = m == -INFINITY;  // no token at all: zeros and -inf
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4& x, int i) {
      const float f = ex2(rec[i * stride + REC_T] - M);
      o.x = fmaf(x.x, f, o.x);
      o.y = fmaf(x.y, f, o.y);
      o.z = fmaf(x.z, f, o.z);
      o.w = fmaf(x.w, f, o.w);
    };
    if (!none) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (first + j * per < n) add(y[j], first + j * per);
#pragma unroll 4
      for (int i = first + 4 * per; i < n; i += per) add(*(const float4*)(rec + i * stride + PART_O + 4 * lane), i);
    }
    *(float4*)&wo[warp][4 * lane] = o;
    if (lane == 0) {  // 2^(M - m) / l in two factors: values of 2^-100 with a leading logit would be lost in one
      const float f = ex2(0.5f * (M - m));
      scale[0][warp] = none ? 0.f : f;
      scale[1][warp] = none ? 0.f : f / l;
    }
    const size_t row = (size_t)b * cv.Hq + (size_t)h * G + (blockIdx.y << log_heads);
    if (a.lse && first == 0 && lane == 0) a.lse[row + own_hd] = none ? -INFINITY : (m + log2f(l)) * LN2;
    __syncthreads();
    for (int e = threadIdx.x; e < heads * (D / 2); e += MT) {
      const int w0 = e / (D / 2) * per, c = e % (D / 2);
      float x = 0.f, z = 0.f;
#pragma unroll
      for (int w = 0; w < MT / 32; ++w)
        if (w < per) {
          const float2 v = *(const float2*)&wo[w0 + w][2 * c];
          x += v.x;
          z += v.y;
        }
      ((__nv_bfloat162*)(a.out + row * D))[e] = __floats2bfloat162_rn(x * scale[0][w0] * scale[1][w0], z * scale[0][w0] * scale[1][w0]);
    }
    return;
  }
  // weights: every head's total first
  for (int hd = warp; hd < G; hd += MT / 32) {
    float m = -INFINITY, l = 0.f;
    bool lost = false;
    for (int i = lane; i < n; i += 32) {
      const float2 x = *(const float2*)(recs + ((size_t)i * G + hd) * PART_STRIDE);
      lost |= x.y == LOST_L;
      const float mn = fmaxf(m, x.x);
      if (x.x != -INFINITY) l = l * ex2(m - mn) + x.y * ex2(x.x - mn);
      m = mn;
    }
    float gm = m;
#pragma unroll
    for (int o = 16; o; o >>= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, o));
    l = m == -INFINITY ? 0.f : l * ex2(m - gm);
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    lost = __any_sync(0xffffffffu, lost);
    if (lane == 0) {
      tot_m[hd] = lost ? -INFINITY : gm;
      tot_r[hd] = 1.f / l;
    }
  }
  __syncthreads();
  if (tot_m[0] == -INFINITY) return;  // nothing was attended to, or not all of it was read
  float* w = a.weights + (size_t)seg * (KV8_RING_BLOCKS + (size_t)KV8_PAGE_BLOCKS * cv.max_pages_per_req);
  const int slice = blockIdx.y - outs, slices = gridDim.y - outs;
  auto gather = [&](int rec) {
    const Sums sums = sums_at(a, seg, rec);
    float4 y[MAX_G], x = make_float4(0.f, 0.f, 0.f, 0.f);
    float r[MAX_G];
#pragma unroll
    for (int hd = 0; hd < MAX_G; ++hd)
      if (hd < G) {
        y[hd] = sums.sum[hd * sums.stride];
        r[hd] = sums.max[hd * sums.stride];
      }
#pragma unroll
    for (int hd = 0; hd < MAX_G; ++hd)
      if (hd < G) {
        const float f = ex2(r[hd] - tot_m[hd]) * tot_r[hd];
        x.x = fmaf(y[hd].x, f, x.x);
        x.y = fmaf(y[hd].y, f, x.y);
        x.z = fmaf(y[hd].z, f, x.z);
        x.w = fmaf(y[hd].w, f, x.w);
      }
    return x;
  };
  for (int p = slice * MT + threadIdx.x; p < sg.pages; p += slices * MT) {
    const float4 x = gather(p);
    float4* dst = (float4*)(w + KV8_RING_BLOCKS) + p;
    float4 v = *dst;
    const int nb = sg.H / KV8_BLK - p * KV8_PAGE_BLOCKS;
    v.x = fmaf(v.x, a.decay, x.x);
    if (nb > 1) v.y = fmaf(v.y, a.decay, x.y);
    if (nb > 2) v.z = fmaf(v.z, a.decay, x.z);
    if (nb > 3) v.w = fmaf(v.w, a.decay, x.w);
    *dst = v;
  }
  if (slice == 0 && threadIdx.x < KV8_RING_UNITS) {
    const int r = threadIdx.x;
    const int n0 = kv8_ring_held(sg.L, sg.H, 2 * r), n1 = kv8_ring_held(sg.L, sg.H, 2 * r + 1);
    if (n0 || n1) {
      const float4 x = gather(cv.max_pages_per_req + r);
      if (n0) w[2 * r] = fmaf(w[2 * r], a.decay, x.x);
      if (n1) w[2 * r + 1] = fmaf(w[2 * r + 1], a.decay, x.y);
    }
  }
}

template <int TYPE, bool WEIGHTS>
cudaError_t launch_main(const Kv8Decode& a, cudaStream_t st) {
  const int smem = decode_smem(a.cv.G).total;
  static int limit[MAX_DEVICES];
  const cudaError_t e = raise_smem_limit(kv8_decode_kernel<TYPE, WEIGHTS>, limit, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv8_decode_kernel<TYPE, WEIGHTS>, dim3(a.grid), dim3(KW * 32), smem, st, a);
}

}  // namespace

int kv8_decode_requests(int batch, int Hkv, int G, int max_pages, bool weights) {
  size_t n = KV8_MAX_REQUESTS;
  if (weights) n = KV8_SCRATCH_AIM / ((size_t)Hkv * (max_pages + KV8_RING_UNITS) * G * 20);
  if (n < 1) n = 1;
  if (n > KV8_MAX_REQUESTS) n = KV8_MAX_REQUESTS;
  return (size_t)batch < n ? batch : (int)n;
}

Kv8Scratch kv8_decode_scratch(int B, int Hkv, int G, int max_pages, bool weights, int grid) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t recs = weights ? (size_t)B * Hkv * (max_pages + KV8_RING_UNITS) * G : 0;
  Kv8Scratch s;
  s.off_wsum = up(((size_t)grid + (size_t)B * Hkv) * G * PART_STRIDE * 4);
  s.off_wmax = s.off_wsum + up(recs * 16);
  s.total = s.off_wmax + up(recs * 4);
  return s;
}

cudaError_t launch_kv8_decode(const Kv8Decode& a, int type, cudaStream_t st, Profiler* prof) {
  prof_begin(prof, OSCAR_KERNEL_KV8_DECODE, st);
  cudaError_t e;
  if (type == OSCAR_KV8_E4M3)
    e = a.weights ? launch_main<OSCAR_KV8_E4M3, true>(a, st) : launch_main<OSCAR_KV8_E4M3, false>(a, st);
  else
    e = a.weights ? launch_main<OSCAR_KV8_INT8, true>(a, st) : launch_main<OSCAR_KV8_INT8, false>(a, st);
  prof_end(prof, OSCAR_KERNEL_KV8_DECODE, st);
  if (e != cudaSuccess) return e;
  const int segs = a.B * a.cv.Hkv;
  int slices = 0;  // a thread per page, up to 16 CTAs a (request, kv head)
  if (a.weights) {
    slices = (a.cv.max_pages_per_req + MT - 1) / MT;
    if (slices > 16) slices = 16;
  }
  // a CTA per query head while that is one wave (three CTAs an SM; the records are
  // few and their latency counts), else as many heads as it takes (32 requests, 8 kv
  // heads of 4: a merge of 13 us against 17 with a CTA per head)
  int log_heads = 0;
  while (1 << log_heads < a.cv.G && segs * (a.cv.G >> log_heads) > 3 * a.grid) ++log_heads;
  prof_begin(prof, OSCAR_KERNEL_KV8_MERGE, st);
  e = launch_pdl(kv8_merge_kernel, dim3(segs, (a.cv.G >> log_heads) + slices), dim3(MT), 0, st, a, log_heads);
  prof_end(prof, OSCAR_KERNEL_KV8_MERGE, st);
  return e;
}

}  // namespace oscar
