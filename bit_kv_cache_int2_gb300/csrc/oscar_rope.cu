// Rotary positions (sm_103a): a layer's fused projection becomes queries, keys
// and values, its query and key heads normalised (optional) and turned.
//
// Angles.  A pair's speed is a 64-bit fixed-point number of turns a position, so
// position·speed mod 2^64 is the angle in turns, exactly: whole turns fall off
// the top, whatever the position.  Its upper 32 bits as a signed fraction in
// [-1/2, 1/2) give cosine and sine to fp32's precision.
//
// Eight lanes share a head, 16 channels (eight pairs) each, so a warp has four
// heads at a time; cosines and sines are made once per token and warp.
#include "oscar_internal.cuh"
#include "oscar_rope.cuh"

namespace oscar {

namespace {

constexpr int RW = 4;      // warps per CTA
constexpr int HEADS = 4;   // heads a warp has at a time

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void unpack8(const uint4& x, float* f) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = lo_f(w[i]);
    f[2 * i + 1] = hi_f(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// Lane u of a head's eight has two groups of eight channels.  HALF: groups u and
// u + dims/16, whose channels are each other's partners, for u < dims/16; the
// groups behind dims, two by two, for the others.  INTERLEAVED: groups u and u + 8, each
// with four pairs.  A warp takes heads 4·part, 4·(part + parts), .. of its token; the
// next heads are on their way while it works on these.
// Bound by memory: what a token reads it writes.  100,003 tokens of 32/8 heads (2.46 GB in
// and out) take 378 us, 6.5 TB/s; with norms 417 to 422, as registers leave 20 warps an SM (24 with
// spills: 430; heads loaded when their turn came: 556) and a warp votes on whether one of its
// heads is out of the squares' range (7 of these).
template <int LAYOUT, bool NORM>
__global__ void __launch_bounds__(RW * 32, NORM ? 5 : 6) rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ uint64_t turn[64];
  const int lane = threadIdx.x & 31, u = lane & 7, np = a.dims >> 4;
  if (threadIdx.x < 64) turn[threadIdx.x] = a.turn[threadIdx.x];
  __syncthreads();
  const bool apart = LAYOUT == OSCAR_ROPE_HALF && u >= np;  // HALF: channels that do not turn
  const int ga = apart ? 2 * u : u;
  const int gb = apart ? 2 * u + 1 : LAYOUT == OSCAR_ROPE_HALF ? u + np : u + 8;
  // whether the groups turn; others pass as they are (x - 0·y would lose them next to an infinity)
  const bool ta = 8 * ga < a.dims, tb = 8 * gb < a.dims;
  pdl_wait();
  pdl_launch_dependents();
  uint4 wq[2], wk[2];
  if (NORM) {
    wq[0] = ((const uint4*)a.gamma_q)[ga], wq[1] = ((const uint4*)a.gamma_q)[gb];
    wk[0] = ((const uint4*)a.gamma_k)[ga], wk[1] = ((const uint4*)a.gamma_k)[gb];
  }
  const int heads = a.Hq + 2 * a.Hkv, rounds = (heads + HEADS - 1) / HEADS;
  const long long tasks = (long long)a.B * a.T * a.parts, step = (long long)gridDim.x * RW;
  for (long long task = (long long)blockIdx.x * RW + (threadIdx.x >> 5); task < tasks; task += step) {
    const long long tok = task / a.parts;
    const int part = (int)(task - tok * a.parts);
    const int b = (int)(tok / a.T), t = (int)(tok - (long long)b * a.T);
    const __nv_bfloat16* row = a.qkv + tok * a.row;
    uint4 xa, xb;
    auto load = [&](int r) {
      const int h = HEADS * r + (lane >> 3);
      xa = xb = make_uint4(0, 0, 0, 0);
      if (r < rounds && h < heads) {
        xa = ((const uint4*)(row + (size_t)h * D))[ga];
        xb = ((const uint4*)(row + (size_t)h * D))[gb];
      }
    };
    load(part);
    const uint64_t pos = (uint64_t)((long long)a.positions[b] + t);
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int p = LAYOUT == OSCAR_ROPE_HALF ? 8 * u + i : i < 4 ? 4 * ga + i : 4 * gb + i - 4;
      const int ph = (int)(uint32_t)((pos * turn[p & 63]) >> 32);
      sincospif((float)ph * 4.656612873077393e-10f, &sn[i], &cs[i]);  // 2^-31: half turns
      sn[i] *= a.size;
      cs[i] *= a.size;
    }
#pragma unroll 1
    for (int r = part; r < rounds; r += a.parts) {
      const int h = HEADS * r + (lane >> 3);
      const uint4 ya = xa, yb = xb;
      load(r + a.parts);
      __nv_bfloat16* to = h < a.Hq           ? a.q + (tok * a.Hq + h) * D
                          : h < a.Hq + a.Hkv ? a.k + (tok * a.Hkv + h - a.Hq) * D
                                             : a.v + (tok * a.Hkv + h - a.Hq - a.Hkv) * D;
      const bool in = h < heads, value = h >= a.Hq + a.Hkv;
      float f[16];
      unpack8(ya, f);
      unpack8(yb, f + 8);
      if (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(f[i], f[i], ss);
        ss += __shfl_xor_sync(0xffffffffu, ss, 1);
        ss += __shfl_xor_sync(0xffffffffu, ss, 2);
        ss += __shfl_xor_sync(0xffffffffu, ss, 4);
        float n = rsqrtf(ss * (1.f / D) + a.eps);
        // Squares that leave fp32's range: the head times the power of two that takes its largest magnitude, or the
        // root of eps where that is larger, to 1 .. 2.
        const bool rare = in && !value && !(ss + D * a.eps >= 0x1p-60f && ss < 0x1p120f);
        if (__any_sync(0xffffffffu, rare)) {
          float m = sqrtf(a.eps), sq = 0.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(f[i]));
#pragma unroll
          for (int d = 1; d < 8; d *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
          const int e = min(max((int)(__float_as_uint(m) >> 23), 1), 253);
          const float s = rare ? pow2i(127 - e) : 1.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            f[i] *= s;
            sq = fmaf(f[i], f[i], sq);
          }
#pragma unroll
          for (int d = 1; d < 8; d *= 2) sq += __shfl_xor_sync(0xffffffffu, sq, d);
          if (rare) n = rsqrtf(sq * (1.f / D) + a.eps * s * s);
        }
        const bool isq = h < a.Hq;
        float w[8];
        unpack8(isq ? wq[0] : wk[0], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= n * w[i];
        unpack8(isq ? wq[1] : wk[1], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[8 + i] *= n * w[i];
      }
      float g[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int x = LAYOUT == OSCAR_ROPE_HALF ? i : 2 * i, y = LAYOUT == OSCAR_ROPE_HALF ? i + 8 : 2 * i + 1;
        g[x] = f[x] * cs[i] - f[y] * sn[i];
        g[y] = f[y] * cs[i] + f[x] * sn[i];
      }
      if (in) {
        ((uint4*)to)[ga] = value ? ya : pack8(ta ? g : f);
        ((uint4*)to)[gb] = value ? yb : pack8(tb ? g + 8 : f + 8);
      }
    }
  }
}

template <int LAYOUT>
cudaError_t launch_layout(const RopeArgs& a, int ctas, cudaStream_t st) {
  return a.gamma_q ? launch_pdl(rope_kernel<LAYOUT, true>, dim3(ctas), dim3(RW * 32), 0, st, a)
                   : launch_pdl(rope_kernel<LAYOUT, false>, dim3(ctas), dim3(RW * 32), 0, st, a);
}

}  // namespace

cudaError_t launch_rope(RopeArgs a, int num_sms, cudaStream_t st, Profiler* prof) {
  const long long tokens = (long long)a.B * a.T, groups = (a.Hq + 2 * a.Hkv + HEADS - 1) / HEADS;
  // a token's heads over several warps while there are few tokens; no warp with a round more than others need
  long long each = tokens * groups / (32ll * num_sms);
  if (each < 1) each = 1;
  if (each > groups) each = groups;
  const long long parts = (groups + each - 1) / each;
  a.parts = (int)parts;
  long long ctas = (tokens * parts + RW - 1) / RW;
  const long long most = (a.gamma_q ? 5ll : 6ll) * num_sms;  // resident
  if (ctas > most) ctas = most;
  prof_begin(prof, OSCAR_KERNEL_PREFILL_PREP, st);
  const cudaError_t e = a.layout == OSCAR_ROPE_HALF ? launch_layout<OSCAR_ROPE_HALF>(a, (int)ctas, st)
                                                    : launch_layout<OSCAR_ROPE_INTERLEAVED>(a, (int)ctas, st);
  prof_end(prof, OSCAR_KERNEL_PREFILL_PREP, st);
  return e;
}

}  // namespace oscar
