// Cache with 8-bit history (sm_103a): page layout, request state and the
// kernels' arguments, shared by the append, decode and eviction kernels.
//
// Layout.  A page holds 64 tokens of every kv head; one head's part is four
// blocks of 16 tokens, [K 2048 B][V 2048 B] each, then four (K scale, V scale)
// fp32 pairs.  Inside a block the bytes stand in the order in which a warp
// feeds them to mma.m16n8k16 as its A operand, 16 bytes per lane and 512-byte
// chunk, so that one conflict-free 16-byte load per lane fetches two k-steps
// (keys) or two row tiles (values).  With lane = 4 gid + tq and byte
// i = 8 s + 4 h + 2 r + l of the lane's 16 bytes in chunk c:
//   K: token 8r + gid,      channel 32c + 8tq + 4s + 2h + l
//   V: token 8h + 2tq + l,  channel 16gid + 4c + 2s + r
// Which channel stands at which k index of the product is free as long as q
// has the same order; this order lets the append kernel read whole 16-byte
// pieces of a token's row and hand every lane exactly the bytes it writes.
#pragma once

#include "oscar_internal.cuh"

namespace oscar {

constexpr int KV8_BLK = OSCAR_KV8_BLOCK;             // tokens per scale block
constexpr int KV8_BLOCK_BYTES = 2 * KV8_BLK * D;     // K then V codes of a block
constexpr int KV8_PAGE_BLOCKS = PAGE / KV8_BLK;
constexpr int KV8_OFF_SCALES = KV8_PAGE_BLOCKS * KV8_BLOCK_BYTES;
constexpr int KV8_HEAD_BYTES = KV8_OFF_SCALES + KV8_PAGE_BLOCKS * 8;
constexpr int KV8_RING_BLOCKS = RECENT / KV8_BLK;    // block weights of the window, before the history's
constexpr float KV8_TINY = 7.888609052210118e-31f;   // 2^-100: no scale is made from a smaller magnitude

// What a request holds.  A state that the append cannot have made (lengths out
// of range, a history that is not whole blocks, a window beyond 256 tokens)
// counts as an error, and the request as empty.
struct Kv8Req {
  int L, H;
  bool ok;
};

// early: read past the L1, by a kernel that looks before its wait.  Where the kernel
// before may still change the lengths (the decode after an append), they are a guess
// to be checked.  Where it does not and released this one only after its own wait (the
// merge, the lengths of an append), whatever wrote them had ended and stood in the L2
// before this kernel could start, and a line that an SM's L1 still has from before
// is passed by.
__device__ __forceinline__ Kv8Req kv8_req(const CacheView& cv, int b, bool early = false) {
  Kv8Req r;
  r.L = early ? __ldcg(cv.seq_lens + b) : cv.seq_lens[b];
  r.H = early ? __ldcg(cv.hist_lens + b) : cv.hist_lens[b];
  const int past = r.L > SINK ? r.L - SINK : 0;
  r.ok = r.L >= 0 && r.H >= 0 && r.H % KV8_BLK == 0 && r.H <= past && past - r.H <= RECENT &&
         (r.H + PAGE - 1) / PAGE <= cv.max_pages_per_req;
  if (!r.ok) r.L = r.H = 0;
  return r;
}

// Tokens held by window block q (ring slots 16q .. 16q + 15): always the
// block's first ones, because a window starts on a block boundary.
__host__ __device__ __forceinline__ int kv8_ring_held(int L, int H, int q) {
  const int held = L - SINK - H - ((KV8_BLK * q - H) & (RECENT - 1));
  return held < 0 ? 0 : held > KV8_BLK ? KV8_BLK : held;
}

__device__ __forceinline__ uint8_t* kv8_head(const CacheView& cv, int pid, int h) {
  return cv.pool + (size_t)pid * cv.page_bytes + (size_t)h * KV8_HEAD_BYTES;
}

// Larger magnitudes of two BF16 pairs; NaN if one is.
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{\n .reg .b32 t;\n abs.bf16x2 t, %2;\n max.NaN.bf16x2 %0, %1, t;\n}\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// ---------------------------------------------------------------- launchers
struct Kv8Append {
  CacheView cv;
  const __nv_bfloat16 *k, *v;  // [B][T][Hkv][128]
  float* weights;              // [B][Hkv][16 + 4 max_pages] or null
  int T;
};
cudaError_t launch_kv8_append(const Kv8Append& a, int type, int B, cudaStream_t st, Profiler* prof);

struct Kv8Decode {
  CacheView cv;
  const __nv_bfloat16* q;  // [B][Hq][128]
  __nv_bfloat16* out;      // [B][Hq][128]
  float* lse;              // [B][Hq] or null
  float* weights;          // as above or null
  float decay;
  float* part;             // scratch [grid + B Hkv][G][PART_STRIDE]: m, l, M, o (oscar_kv8_decode.cu)
  float* wsum;             // scratch [B Hkv][G][max_pages + 8][4]: sums of a page's blocks ...
  float* wmax;             // scratch [B Hkv][G][max_pages + 8]: ... relative to 2^this
  int B, grid, wait_polls;
};
constexpr int KV8_WIN_UNITS = 10;                                  // 32-token pieces of the BF16 regions
constexpr int KV8_RING_UNITS = RECENT / 32;
cudaError_t launch_kv8_decode(const Kv8Decode& a, int type, cudaStream_t st, Profiler* prof);

struct Kv8Evict {
  CacheView cv;
  float* weights;
  int32_t* list;  // scratch [B Hkv][kv8_evict_stride()]: count, history after, holes, then the blocks that fill them
  int budget;
};
__host__ __device__ __forceinline__ size_t kv8_evict_stride(int max_pages) { return 4 + 4 * (size_t)max_pages; }
cudaError_t launch_kv8_evict(const Kv8Evict& a, int B, int num_sms, cudaStream_t st, Profiler* prof);

struct Kv8Read {
  CacheView cv;
  __nv_bfloat16 *K, *V;  // [B][Hkv][n][128] or [B][n][Hkv][128]
  int first, n, order;
};
cudaError_t launch_kv8_read(const Kv8Read& a, int type, int B, cudaStream_t st, Profiler* prof);

struct Kv8Prefill {
  CacheView cv;
  const __nv_bfloat16 *q, *k, *v;  // [B][T][Hq or Hkv][128]
  __nv_bfloat16* out;              // [B][T][Hq][128]
  float* lse;                      // [B][T][Hq] or null
  int4* splits;                    // scratch [grid]: the unit that begins in a CTA's part and ends in a later one's
  float* part;                     // scratch [grid][2] records of 256·PART_STRIDE floats: o [32][256] of 4 channels,
                                   //   log2 of the sum of exponentials [256], M [256] (oscar_kv8_prefill.cu)
  int B, T, grid, wait_polls;
  // set by launch_kv8_prefill: log2 of G; units of 256 rows of a (request, kv head); M of BF16 tokens above their logits
  int lg, units;
  float room;
};
constexpr int KV8_PREFILL_MAX_GRID = 160;  // CTAs (one per SM) that the scratch has records for
struct Kv8PrefillScratch {
  size_t off_part, total;
};
cudaError_t launch_kv8_prefill(Kv8Prefill a, int type, cudaStream_t st, Profiler* prof);
Kv8PrefillScratch kv8_prefill_scratch(int grid);

// The largest number of 16 KB units a request may have: the work list counts
// 32 requests in 32 bits.
constexpr long long KV8_MAX_UNITS = 1 << 26;

// Requests that one launch takes (a longer batch is several launches on the
// stream, sharing the scratch), and the scratch of such a launch.
constexpr int KV8_MAX_REQUESTS = 1024;
constexpr int KV8_MAX_GRID = 512;  // decode CTAs (one per SM) that the scratch has records for
constexpr size_t KV8_SCRATCH_AIM = 64u << 20;
struct Kv8Scratch {
  size_t off_wsum, off_wmax, total;
};
int kv8_decode_requests(int batch, int Hkv, int G, int max_pages, bool weights);
Kv8Scratch kv8_decode_scratch(int B, int Hkv, int G, int max_pages, bool weights, int grid);
int kv8_evict_requests(int batch, int Hkv, int max_pages);
size_t kv8_evict_scratch(int B, int Hkv, int max_pages);

}  // namespace oscar
