// Chunk attention over a cache with 8-bit history (sm_103a).
//
// The plainest form: a CTA has 16 query rows (row r of a kv head: token r / G,
// query head r % G), goes over the tokens 32 at a time in fp32 and keeps each
// row's running maximum and sum.
#include "oscar_kv8.cuh"

namespace oscar {

namespace {

constexpr int QR = 16, TK = 32;

template <int TYPE>
__device__ __forceinline__ float code_value(uint8_t c) {
  if (TYPE == OSCAR_KV8_INT8) return (float)(int8_t)c;
  uint32_t h;
  asm("{\n .reg .b16 a;\n cvt.u16.u32 a, %1;\n cvt.rn.f16x2.e4m3x2 %0, a;\n}\n" : "=r"(h) : "r"((uint32_t)c));
  return __half2float(__ushort_as_half((unsigned short)h));
}

template <int TYPE>
__global__ void __launch_bounds__(128) prefill_simple_kernel(Kv8Prefill a) {
  __shared__ float Q[QR][D], K[TK][D + 1], V[TK][D], P[QR][TK];
  __shared__ float fac[QR], sum[QR];
  pdl_wait();
  pdl_launch_dependents();
  const CacheView& cv = a.cv;
  const int b = blockIdx.z, h = blockIdx.y, G = cv.G, c = threadIdx.x, Hkv = cv.Hkv, Hq = cv.Hq;
  const Kv8Req r = kv8_req(cv, b);
  if (!r.ok && threadIdx.x == 0) record_error(cv.err, OSCAR_ERR_STATE);
  const int row0 = blockIdx.x * QR, rows = a.T * G;
  const size_t head = (size_t)b * Hkv + h;
  for (int i = 0; i < QR; ++i) {
    const int rr = row0 + i;
    Q[i][c] = rr < rows ? __bfloat162float(a.q[(((size_t)b * a.T + rr / G) * Hq + h * G + rr % G) * D + c]) : 0.f;
  }
  float o[QR], m = -1e30f, l = 0.f;  // m, l: row threadIdx.x / 8
  for (int i = 0; i < QR; ++i) o[i] = 0.f;
  const int t_last = min(a.T - 1, (row0 + QR - 1) / G), n = r.L + t_last + 1;
  for (int p0 = 0; p0 < n; p0 += TK) {
    __syncthreads();
    for (int j = 0; j < TK; ++j) {
      const int p = p0 + j;
      float k = 0.f, v = 0.f;
      if (p < n && p >= r.L) {
        const size_t at = (((size_t)b * a.T + p - r.L) * Hkv + h) * D + c;
        k = __bfloat162float(a.k[at]);
        v = __bfloat162float(a.v[at]);
      } else if (p < n && (p < SINK || p >= SINK + r.H)) {
        const size_t at = p < SINK ? (head * SINK + p) * D + c : (head * RECENT + ((p - SINK) & (RECENT - 1))) * D + c;
        k = __bfloat162float((p < SINK ? cv.sink_k : cv.ring_k)[at]);
        v = __bfloat162float((p < SINK ? cv.sink_v : cv.ring_v)[at]);
      } else if (p < n) {
        const int s = p - SINK, t = s & 15, sub = (s >> 4) & 3;
        const int pid = cv.page_table[(size_t)b * cv.max_pages_per_req + s / PAGE];
        if (pid < 0 || pid >= cv.num_pages) {
          if (c == 0) record_error(cv.err, pid < 0 ? OSCAR_ERR_NO_PAGE : OSCAR_ERR_RANGE);
          k = NAN;  // marks the token as left out (below)
        } else {
          const uint8_t* base = kv8_head(cv, pid, h);
          const uint8_t* blk = base + sub * KV8_BLOCK_BYTES;
          const float2 sc = ((const float2*)(base + KV8_OFF_SCALES))[sub];
          const int kb = 512 * (c >> 5) + 16 * (4 * (t & 7) + ((c >> 3) & 3)) + 8 * ((c >> 2) & 1) + 4 * ((c >> 1) & 1) + 2 * (t >> 3) + (c & 1);
          const int vb = 512 * ((c >> 2) & 3) + 16 * (4 * (c >> 4) + ((t >> 1) & 3)) + 8 * ((c >> 1) & 1) + 4 * (t >> 3) + 2 * (c & 1) + (t & 1);
          k = code_value<TYPE>(blk[kb]) * sc.x;
          v = code_value<TYPE>(blk[2048 + vb]) * sc.y;
        }
      }
      K[j][c] = k;
      V[j][c] = v;
    }
    __syncthreads();
    const int i = threadIdx.x >> 3, t = (row0 + i) / G;
    float x[4], mx = m;
    for (int e = 0; e < 4; ++e) {
      const int j = (threadIdx.x & 7) + 8 * e, p = p0 + j;
      bool seen = p < n && p <= r.L + t;
      if (seen && p >= SINK && p < SINK + r.H) {
        const int pid = cv.page_table[(size_t)b * cv.max_pages_per_req + (p - SINK) / PAGE];
        seen = pid >= 0 && pid < cv.num_pages;
      }
      float s = 0.f;
      for (int d = 0; d < D; ++d) s = fmaf(Q[i][d], K[j][d], s);
      x[e] = seen ? s * (INV_SQRT_D * LOG2E) : -INFINITY;
      mx = fmaxf(mx, x[e]);
    }
    for (int w = 1; w < 8; w *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    float ps = 0.f;
    for (int e = 0; e < 4; ++e) {
      const float p = exp2f(x[e] - mx);
      P[i][(threadIdx.x & 7) + 8 * e] = p;
      ps += p;
    }
    for (int w = 1; w < 8; w *= 2) ps += __shfl_xor_sync(0xffffffffu, ps, w);
    if ((threadIdx.x & 7) == 0) fac[i] = exp2f(m - mx);
    l = l * exp2f(m - mx) + ps;
    m = mx;
    __syncthreads();
    for (int q = 0; q < QR; ++q) {
      float acc = o[q] * fac[q];
      for (int j = 0; j < TK; ++j) {
        const float p = P[q][j];
        acc += p == 0.f ? 0.f : p * V[j][c];  // a masked token's value does not count, whatever it is
      }
      o[q] = acc;
    }
  }
  __syncthreads();
  if ((threadIdx.x & 7) == 0) {
    sum[threadIdx.x >> 3] = l;
    fac[threadIdx.x >> 3] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
  }
  __syncthreads();
  for (int i = 0; i < QR; ++i) {
    const int rr = row0 + i;
    if (rr >= rows) break;
    const size_t at = ((size_t)b * a.T + rr / G) * Hq + h * G + rr % G;
    a.out[at * D + c] = __float2bfloat16_rn(sum[i] == 0.f ? 0.f : o[i] / sum[i]);
    if (a.lse && c == 0) a.lse[at] = fac[i];
  }
}

}  // namespace

size_t kv8_prefill_scratch() { return 256; }

cudaError_t launch_kv8_prefill(const Kv8Prefill& a, int type, cudaStream_t st, Profiler* prof) {
  const dim3 grid((unsigned)(((long long)a.T * a.cv.G + QR - 1) / QR), a.cv.Hkv, a.B);
  prof_begin(prof, OSCAR_KERNEL_PREFILL_ATTN, st);
  const cudaError_t e = type == OSCAR_KV8_E4M3 ? launch_pdl(prefill_simple_kernel<OSCAR_KV8_E4M3>, grid, dim3(128), 0, st, a)
                                               : launch_pdl(prefill_simple_kernel<OSCAR_KV8_INT8>, grid, dim3(128), 0, st, a);
  prof_end(prof, OSCAR_KERNEL_PREFILL_ATTN, st);
  return e;
}

}  // namespace oscar
