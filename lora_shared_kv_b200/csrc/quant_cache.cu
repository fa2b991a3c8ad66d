// Writing bf16 K/V rows into an 8-bit cache and reading them back.
//
//   write   scale' = need, or max(scale, need) where the block keeps older rows;
//           code = round(x / scale')
//   read    y = bf16(code * scale)
//
// Both are bound by memory: 3 bytes move per element (4 sessions x 16k x 8 heads written
// whole: floor 62 us, e4m3 82, int8 106, whose rounding still costs instructions; 16k x 8
// heads read back: floor 15 us, 20).  One CTA takes one block of
// one (session, KV head) of K or of V: 64 tokens x head_dim, at most 16 KB of
// bf16, which stays in registers between the block's maximum and its rounding,
// so every element is read once.
#include <cuda_fp16.h>

#include "common.cuh"
#include "quant_device.cuh"
#include "quant.h"

namespace lrkv {

namespace {

constexpr float kScaleMin = 7.888609052210118e-31f;  // 2^-100
constexpr uint32_t kBf16Inf = 0x7F80u;

// What a CTA works on: block `blk` (rows [lo, lo + 64)) of session s, KV head g,
// K (which = 0) or V; rows [r0, r1) of it are new tokens t0 + (r - r0).
struct Work {
  int which, s, g, blk, r0, r1, t0;
};

// False where there is nothing to do (or the session's range is refused).
__device__ __forceinline__ bool find_work(const QCacheParams& p, Work& w) {
  long long i = blockIdx.x;
  const int j = (int)(i % p.nblk);
  i /= p.nblk;
  w.which = (int)(i & 1);
  i >>= 1;
  w.g = (int)(i % p.Hkv);
  w.s = (int)(i / p.Hkv);
  const int first = p.first ? __ldg(p.first + w.s) : 0;
  const int n = p.count ? __ldg(p.count + w.s) : p.T;
  if (first < 0 || n < 0 || n > p.T || (long long)first + n > p.rows) {
    if (threadIdx.x == 0) atomicOr(p.flags, LRKV_DEVFLAG_SEQLEN);
    return false;
  }
  w.blk = first / kQBlock + j;
  const int lo = w.blk * kQBlock;
  if (n == 0 || lo >= first + n) return false;
  w.r0 = max(first - lo, 0);
  w.r1 = min(first + n - lo, kQBlock);
  w.t0 = lo + w.r0 - first;
  return true;
}

// Byte offset of the block's codes and the index of its scale; false for a bad page id.
__device__ __forceinline__ bool locate_block(const QCacheParams& p, const Work& w, long long& code, long long& sc) {
  if (p.c_table == nullptr) {
    code = w.s * p.c_ss + w.g * p.c_sh + (long long)w.blk * kQBlock * p.c_st;
    sc = w.s * p.s_ss + w.g * p.s_sh + w.blk;
    return true;
  }
  const int page = __ldg(p.c_table + w.s * p.c_pt + w.blk);
  if (page < 0 || page >= p.c_pages) {
    if (threadIdx.x == 0) atomicOr(p.flags, LRKV_DEVFLAG_PAGE);
    return false;
  }
  code = page * p.c_sp + w.g * p.c_sh;
  sc = page * p.s_sp + w.g * p.s_sh;
  return true;
}

// Element offset of token t's row on the bf16 side; -1 for a bad page id.
__device__ __forceinline__ long long x_row(const QCacheParams& p, const Work& w, int t) {
  if (p.x_table == nullptr) return w.s * p.x_ss + w.g * p.x_sh + t * p.x_st;
  const int page = __ldg(p.x_table + w.s * p.x_pt + t / kQBlock);
  if (page < 0 || page >= p.x_pages) {
    atomicOr(p.flags, LRKV_DEVFLAG_PAGE);
    return -1;
  }
  return page * p.x_sp + w.g * p.x_sh + (t % kQBlock) * p.x_st;
}

// The smallest scale that holds amax (a finite bf16 number >= 0).
template <int FMT>
__device__ __forceinline__ float scale_need(float amax) {
  float s;
  if constexpr (FMT == LRKV_Q_E4M3) {
    // amax = m 2^e with m in [1, 2), 448 = 1.75 2^8: 2^(e - 8) holds it when m <= 1.75
    const uint32_t b = __float_as_uint(amax);
    const int k = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    s = __uint_as_float((uint32_t)(max(k, -100) + 127) << 23);
  } else {
    s = __uint_as_float((__float_as_uint(__fdiv_rn(amax, 127.f)) + 0xFFFFu) & 0xFFFF0000u);
    // 127 s is exact (7 + 8 bits), so these comparisons settle which bf16 number is the smallest
    if (s * 127.f < amax) s = __uint_as_float(__float_as_uint(s) + 0x10000u);
    if (s > 0.f) {
      const float low = __uint_as_float(__float_as_uint(s) - 0x10000u);
      if (low * 127.f >= amax) s = low;
    }
  }
  return fmaxf(s, kScaleMin);
}

// Codes of eight values.  inv is 1 / scale, exact when the scale is a power of two
// (pow2); `odd`: there may be infinities or NaN among them.
template <int FMT>
__device__ __forceinline__ uint2 encode8(const float* f, float scale, float inv, bool pow2, bool odd) {
  if constexpr (FMT == LRKV_Q_E4M3) {
    uint16_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = pow2 ? f[2 * i] * inv : __fdiv_rn(f[2 * i], scale);
      const float y = pow2 ? f[2 * i + 1] * inv : __fdiv_rn(f[2 * i + 1], scale);
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r[i]) : "f"(y), "f"(x));
    }
    return make_uint2((uint32_t)r[0] | (uint32_t)r[1] << 16, (uint32_t)r[2] | (uint32_t)r[3] << 16);
  } else {
    // The nearest integer to x / scale.  Adding 1.5 2^23 rounds x inv to an integer n and
    // leaves it in the sum's low bits (with conversion instructions, a quarter of the
    // rate, the 4 x 16k write took 139 us).  n is off by at most one, and the remainder
    // x - n scale (one rounding; exact next to half a step) says so; of two equally near
    // integers the even one.  That is rarely needed: one test for the eight values.
    constexpr float kMagic = 12582912.f;
    const float half = 0.5f * scale;
    float t[8];
    bool fix = odd;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t[i] = fmaf(f[i], inv, kMagic);
      fix |= fabsf(fmaf(kMagic - t[i], scale, f[i])) >= half;
    }
    if (fix) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float rem = fmaf(kMagic - t[i], scale, f[i]);
        if (fabsf(rem) > half || (fabsf(rem) == half && (__float_as_uint(t[i]) & 1))) t[i] += copysignf(1.f, rem);
        if (odd) t[i] = f[i] != f[i] ? kMagic : kMagic + fminf(fmaxf(t[i] - kMagic, -127.f), 127.f);
      }
    }
    uint32_t n[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] = __float_as_uint(t[i]);
    return make_uint2(
        __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410),
        __byte_perm(__byte_perm(n[4], n[5], 0x0040), __byte_perm(n[6], n[7], 0x0040), 0x5410));
  }
}

__device__ __forceinline__ void bf16x8_to_f32(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// Values of four codes, as floats.
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, float* f) {
  uint32_t lo, hi;
  codes_to_half2<FMT>(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  f[code_byte<FMT>(0)] = a.x;
  f[code_byte<FMT>(1)] = a.y;
  f[code_byte<FMT>(2)] = b.x;
  f[code_byte<FMT>(3)] = b.y;
}

template <int FMT, int D, int kThreads>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QCacheParams p) {
  constexpr int CPR = D / 8;                      // 16-byte chunks of a row
  constexpr int PER = kQBlock * CPR / kThreads;   // chunks of a thread
  __shared__ uint32_t red[kThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  Work w;
  if (!find_work(p, w)) return;
  long long code, sc;
  if (!locate_block(p, w, code, sc)) return;
  float* scale_at = p.scale[w.which] + sc;
  uint8_t* out = p.c[w.which] + code;
  const uint16_t* x = p.x[w.which];
  const int row = threadIdx.x / CPR, col = (threadIdx.x % CPR) * 8;
  const float before = w.r0 > 0 ? __ldcg(scale_at) : 0.f;
  uint4 v[PER];
  uint32_t top = 0;
  bool bad_page = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int r = row + i * (kThreads / CPR);
    v[i] = make_uint4(0, 0, 0, 0);
    if (r >= w.r0 && r < w.r1) {
      const long long at = x_row(p, w, w.t0 + r - w.r0);
      if (at >= 0) v[i] = ld_stream(x + at + col);
      else bad_page = true;
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    uint32_t m = __vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu);
    m = __vmaxu2(m, __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
    top = __vmaxu2(top, m);
  }
  top = max(top & 0xFFFFu, top >> 16);
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
  // a source page out of range: the block is left as it was
  if (__syncthreads_or(bad_page)) return;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) top = max(top, red[i]);
  const bool odd = top >= kBf16Inf;
  if (odd) {  // the block holds an infinity or NaN: the largest finite magnitude
    if (threadIdx.x == 0) atomicOr(p.flags, LRKV_DEVFLAG_NONFINITE);
    top = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a = u[j] & 0x7FFFu, b = (u[j] >> 16) & 0x7FFFu;
        if (a < kBf16Inf) top = max(top, a);
        if (b < kBf16Inf) top = max(top, b);
      }
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    __syncthreads();  // every thread has read the first maxima
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) top = max(top, red[i]);
  }
  const float need = scale_need<FMT>(__uint_as_float(top << 16));
  const float scale = fmaxf(before, need);
  const bool pow2 = (__float_as_uint(scale) & 0x7FFFFFu) == 0;
  const float inv = __frcp_rn(scale);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int r = row + i * (kThreads / CPR);
    if (r < w.r0 || r >= w.r1) continue;
    float f[8];
    bf16x8_to_f32(v[i], f);
    *reinterpret_cast<uint2*>(out + (long long)r * p.c_st + col) = encode8<FMT>(f, scale, inv, pow2, odd);
  }
  if (w.r0 > 0 && scale == before) return;
  if (w.r0 > 0) {  // the scale grew: the block's older rows move to it
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int r = row + i * (kThreads / CPR);
      if (r >= w.r0) continue;
      uint2* at = reinterpret_cast<uint2*>(out + (long long)r * p.c_st + col);
      const uint2 c = *at;
      float f[8];
      decode4<FMT>(c.x, f);
      decode4<FMT>(c.y, f + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= before;
      *at = encode8<FMT>(f, scale, inv, pow2, odd);
    }
  }
  if (threadIdx.x == 0) *scale_at = scale;  // every thread's `before` was read ahead of the barrier
}

template <int FMT, int D>
__global__ void __launch_bounds__(256) dequantize_kernel(const QCacheParams p) {
  constexpr int kThreads = 256;
  constexpr int CPR = D / 16;                     // 16-code chunks of a row
  constexpr int PER = kQBlock * CPR / kThreads;
  pdl_wait();
  pdl_launch_dependents();
  Work w;
  if (!find_work(p, w)) return;
  long long code, sc;
  if (!locate_block(p, w, code, sc)) return;
  const float scale = __ldg(p.scale[w.which] + sc);
  const uint8_t* in = p.c[w.which] + code;
  uint16_t* x = p.x[w.which];
  const int row = threadIdx.x / CPR, col = (threadIdx.x % CPR) * 16;
  uint4 c[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int r = row + i * (kThreads / CPR);
    if (r >= w.r0 && r < w.r1) c[i] = ld_stream(in + (long long)r * p.c_st + col);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int r = row + i * (kThreads / CPR);
    if (r < w.r0 || r >= w.r1) continue;
    const long long at = x_row(p, w, w.t0 + r - w.r0);
    if (at < 0) continue;
    const uint32_t u[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
    uint32_t y[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[4];
      decode4<FMT>(u[j], f);
      y[2 * j] = pack_bf16x2(f[0] * scale, f[1] * scale);
      y[2 * j + 1] = pack_bf16x2(f[2] * scale, f[3] * scale);
    }
    uint4* o = reinterpret_cast<uint4*>(x + at + col);
    o[0] = make_uint4(y[0], y[1], y[2], y[3]);
    o[1] = make_uint4(y[4], y[5], y[6], y[7]);
  }
}

template <typename Kernel>
lrkv_status launch(Kernel kern, int threads, const QCacheParams& p, void* stream) {
  const long long ctas = (long long)p.S * p.Hkv * 2 * p.nblk;
  if (ctas > 0x7FFFFFFFLL) return LRKV_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(threads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? LRKV_OK : LRKV_ERR_CUDA;
}

// Threads of a writing CTA.  With many blocks, a block is 128 threads': more CTAs fit an SM and their loads and stores overlap (4 sessions x 16k x 8
// heads: 105 us int8, 82 us e4m3, against 115 and 85 with 256 threads).  With few blocks
// a block's own time counts, and 256 threads halve it (144 blocks: 3.1 us against 4.8).
template <int FMT, int D>
lrkv_status launch_quantize_fd(const QCacheParams& p, void* stream) {
  const bool few = (long long)p.S * p.Hkv * 2 * p.nblk <= 296;
  return few ? launch(quantize_kernel<FMT, D, 256>, 256, p, stream)
             : launch(quantize_kernel<FMT, D, 128>, 128, p, stream);
}

}  // namespace

lrkv_status launch_quantize(const QCacheParams& p, int D, int fmt, void* stream) {
  if (fmt == LRKV_Q_E4M3)
    return D == 128 ? launch_quantize_fd<LRKV_Q_E4M3, 128>(p, stream) : launch_quantize_fd<LRKV_Q_E4M3, 64>(p, stream);
  return D == 128 ? launch_quantize_fd<LRKV_Q_INT8, 128>(p, stream) : launch_quantize_fd<LRKV_Q_INT8, 64>(p, stream);
}

lrkv_status launch_dequantize(const QCacheParams& p, int D, int fmt, void* stream) {
  if (fmt == LRKV_Q_E4M3)
    return D == 128 ? launch(dequantize_kernel<LRKV_Q_E4M3, 128>, 256, p, stream)
                    : launch(dequantize_kernel<LRKV_Q_E4M3, 64>, 256, p, stream);
  return D == 128 ? launch(dequantize_kernel<LRKV_Q_INT8, 128>, 256, p, stream)
                  : launch(dequantize_kernel<LRKV_Q_INT8, 64>, 256, p, stream);
}

}  // namespace lrkv
