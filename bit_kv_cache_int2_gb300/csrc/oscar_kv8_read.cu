// Reading a cache with 8-bit history back as dense BF16 (sm_103a).
//
// A warp takes the 16 tokens of one block (of the sink, the history or the
// window: all three start on multiples of 16 places), kv head and side.  A
// history block's codes are in the order of the layout (oscar_kv8.cuh): a lane
// has eight channels of two tokens per 512-byte chunk of keys, and in all four
// chunks of values 16 channels of four tokens.
#include "oscar_kv8.cuh"

namespace oscar {

namespace {

constexpr int VW = 4;  // warps per CTA

// The values of the byte pairs (0, 1) and (2, 3) of w times s, as bf16x2 words.
template <int TYPE>
__device__ __forceinline__ void decode4(uint32_t w, float s, uint32_t& lo, uint32_t& hi) {
  float f[4];
  if (TYPE == OSCAR_KV8_E4M3) {
    uint32_t h0, h1;
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(h0), "=r"(h1)
        : "r"(w));
    const float2 x = __half22float2(*(__half2*)&h0), y = __half22float2(*(__half2*)&h1);
    f[0] = x.x, f[1] = x.y, f[2] = y.x, f[3] = y.y;
  } else {
    w ^= 0x80808080u;  // code + 128 into the low bits of 2^23
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(prmt(w, 0x4b000000u, 0x7440 | i)) - 8388736.f;
  }
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(lo) : "f"(f[1] * s), "f"(f[0] * s));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(hi) : "f"(f[3] * s), "f"(f[2] * s));
}

// 32 bytes of a row, at once where the array is aligned to that.
__device__ __forceinline__ void store32(__nv_bfloat16* p, const uint32_t* w) {
  if ((uintptr_t)p & 31) {
    ((uint4*)p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    ((uint4*)p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Bound by memory, most of it written (one GB300): 100,000 tokens of 8 kv heads in 94.7 us (90.6 at
// the measured copy rate), 32 requests with 8K to 32K in 600 (582).  A block a warp, in both orders:
// its rows are whole 256-byte lines of the output.
template <int TYPE>
__global__ void __launch_bounds__(VW * 32) read_kernel(Kv8Read a) {
  pdl_wait();
  pdl_launch_dependents();
  const CacheView& cv = a.cv;
  const int b = blockIdx.y, Hkv = cv.Hkv, lane = threadIdx.x & 31;
  const Kv8Req r = kv8_req(cv, b);
  if (!r.ok) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_error(cv.err, OSCAR_ERR_STATE);
    return;
  }
  const long long task = (long long)blockIdx.x * VW + (threadIdx.x >> 5);
  const int side = (int)(task & 1), h = (int)((task >> 1) % Hkv);
  const long long blk = a.first / KV8_BLK + (task >> 1) / Hkv;
  const long long p0 = blk * KV8_BLK;  // the block's first place
  const long long end = a.first + (long long)a.n < r.L ? a.first + (long long)a.n : r.L;
  if (p0 >= end) return;
  // row of place p: dst + (p - first)·tok
  const size_t tok = a.order == OSCAR_ORDER_HEADS ? D : (size_t)Hkv * D;
  __nv_bfloat16* dst = (side ? a.V : a.K) +
                       (a.order == OSCAR_ORDER_HEADS ? ((size_t)b * Hkv + h) * a.n * D : ((size_t)b * a.n * Hkv + h) * D);
  auto row = [&](int t) { return dst + (size_t)(p0 + t - a.first) * tok; };
  const int from = a.first > p0 ? (int)(a.first - p0) : 0, to = end - p0 < KV8_BLK ? (int)(end - p0) : KV8_BLK;
  const size_t head = (size_t)b * Hkv + h;
  if (p0 < SINK || p0 >= SINK + r.H) {
    const __nv_bfloat16* src = p0 < SINK ? (side ? cv.sink_v : cv.sink_k) + (head * SINK + p0) * D
                                         : (side ? cv.ring_v : cv.ring_k) + (head * RECENT + ((p0 - SINK) & (RECENT - 1))) * D;
    for (int t = from + (lane >> 4); t < to; t += 2)
      ((uint4*)row(t))[lane & 15] = ((const uint4*)(src + (size_t)t * D))[lane & 15];
    return;
  }
  const int j = (int)(blk - SINK / KV8_BLK), sub = j % KV8_PAGE_BLOCKS;
  const int pid = cv.page_table[(size_t)b * cv.max_pages_per_req + j / KV8_PAGE_BLOCKS];
  if (pid < 0 || pid >= cv.num_pages) {
    if (lane == 0) record_error(cv.err, pid < 0 ? OSCAR_ERR_NO_PAGE : OSCAR_ERR_RANGE);
    return;
  }
  const uint8_t* base = kv8_head(cv, pid, h);
  const uint4* src = (const uint4*)(base + sub * KV8_BLOCK_BYTES + side * (KV8_BLK * D)) + lane;
  uint4 x[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) x[c] = src[32 * c];
  const float s = ((const float*)(base + KV8_OFF_SCALES))[2 * sub + side];
  const int gid = lane >> 2, tq = lane & 3;
  if (side == 0) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint4 lo, hi;  // token gid, token 8 + gid
      decode4<TYPE>(x[c].x, s, lo.x, hi.x);
      decode4<TYPE>(x[c].y, s, lo.y, hi.y);
      decode4<TYPE>(x[c].z, s, lo.z, hi.z);
      decode4<TYPE>(x[c].w, s, lo.w, hi.w);
      if (gid >= from && gid < to) ((uint4*)row(gid))[4 * c + tq] = lo;
      if (gid + 8 >= from && gid + 8 < to) ((uint4*)row(gid + 8))[4 * c + tq] = hi;
    }
  } else {
#pragma unroll
    for (int th = 0; th < 2; ++th) {
      uint32_t o[2][8];  // tokens 8th + 2tq + l
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int sp = 0; sp < 2; ++sp) {  // channels 16gid + 4c + 2sp + r: bytes (r, l) -> (l, r)
          const uint32_t w = ((const uint32_t*)&x[c])[2 * sp + th];
          decode4<TYPE>(prmt(w, 0, 0x3120), s, o[0][2 * c + sp], o[1][2 * c + sp]);
        }
#pragma unroll
      for (int l = 0; l < 2; ++l) {
        const int t = 8 * th + 2 * tq + l;
        if (t >= from && t < to) store32(row(t) + 16 * gid, o[l]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv8_read(const Kv8Read& a, int type, int B, cudaStream_t st, Profiler* prof) {
  // no request has more tokens than its sink, its pages and its window hold
  const long long most = SINK + RECENT + (long long)a.cv.max_pages_per_req * PAGE;
  const long long end = (long long)a.first + a.n < most ? (long long)a.first + a.n : most;
  const long long blocks = end > a.first ? (end - 1) / KV8_BLK - a.first / KV8_BLK + 1 : 1;
  const long long ctas = (blocks * a.cv.Hkv * 2 + VW - 1) / VW;
  prof_begin(prof, OSCAR_KERNEL_IMPORT, st);
  const cudaError_t e = type == OSCAR_KV8_E4M3
                            ? launch_pdl(read_kernel<OSCAR_KV8_E4M3>, dim3((unsigned)ctas, B), dim3(VW * 32), 0, st, a)
                            : launch_pdl(read_kernel<OSCAR_KV8_INT8>, dim3((unsigned)ctas, B), dim3(VW * 32), 0, st, a);
  prof_end(prof, OSCAR_KERNEL_IMPORT, st);
  return e;
}

}  // namespace oscar
