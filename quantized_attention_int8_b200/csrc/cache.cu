// Head norm and position rotation, and the paged quantized cache: its write and its read back.
//
//   norm    n_c = x_c * rsqrt(sum_c x_c^2 / d + eps) * w_c
//   rotate  pairs (a, b) of channels, angle i: y_a = n_a cos_i - n_b sin_i, y_b = n_b cos_i + n_a sin_i
//   write   per (token, kv head): y = k - k_mean, code = clamp(rint(y * (127 / amax)), +-127), ks = amax / 127;
//           code = E4M3_rne(v * (448 / amax)), vs = amax / 448
//   read    k = code * ks + k_mean, v = code * vs
//
// All of it in fp32 from the 16-bit inputs, with one rounding where a value leaves as 16 bits.  In a
// cache write with norm and rotation the key goes from fp32 straight to its INT8 code: rounding it
// to 16 bits in between would only add error.
//
// Everything here moves bytes: about ten operations per element.  A row (one head of one token) is
// owned by 8, 16 or 32 consecutive lanes, eight channels (16 bytes) to a lane, so that the sum of
// squares, the amax and the rotation's partner channels are lane shuffles inside a warp and no
// shared memory or barrier is on the path.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "sage_internal.h"

namespace sage {

// Error word of the kernels in this file, read and cleared by sage_check_status().
__device__ int g_cache_error = 0;

cudaError_t read_clear_cache_error(int* value) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_cache_error, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_cache_error, &zero, sizeof(int));
}

namespace {

constexpr int kThreads = 256;
constexpr int kBadArg = 2;  // the error word's bit for SAGE_ERR_INVALID_ARG
// Rows whose largest magnitude is below this (or zero) are stored as zeros: 127 / amax and
// 448 / amax then stay finite.
constexpr float kTinyAmax = 7.888609052210118e-31f;  // 2^-100

__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ float bits_to_f32(uint32_t h16) {
  T t;
  *reinterpret_cast<unsigned short*>(&t) = (unsigned short)h16;
  return to_f32(t);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t w = (&v.x)[e >> 1];
    x[e] = bits_to_f32<T>((e & 1) ? w >> 16 : w & 0xFFFFu);
  }
}

// Eight 16-bit channels c0..c0+7 of a row of d channels; channels past d read as zero.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const unsigned short* row, int c0, int d) {
  if (VEC) return c0 < d ? *reinterpret_cast<const uint4*>(row + c0) : make_uint4(0, 0, 0, 0);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c0 + e < d) w[e >> 1] |= (uint32_t)row[c0 + e] << (16 * (e & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The same, rounded from fp32 and stored.
template <typename T, bool VEC>
__device__ __forceinline__ void store8(unsigned short* row, int c0, int d, const float* x, const Extent& ext) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = pack2(x[2 * e], x[2 * e + 1], T());
  if (VEC) {
    if (c0 < d && SAGE_STORE_OK(ext, row + c0, 16, &g_cache_error))
      *reinterpret_cast<uint4*>(row + c0) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c0 + e < d && SAGE_STORE_OK(ext, row + c0 + e, 2, &g_cache_error))
        row[c0 + e] = (unsigned short)(w[e >> 1] >> (16 * (e & 1)));
  }
}

// Eight values c0..c0+7 of a vector of d fp32 or 16-bit values (zero past d).
__device__ __forceinline__ void load8_param(const void* src, int dtype, bool vec, int c0, int d, float (&x)[8]) {
  if (vec) {
    if (c0 >= d) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.f;
    } else if (dtype == SAGE_FP32) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(src) + c0));
      const float4 b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(src) + c0 + 4));
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const unsigned short*>(src) + c0));
      if (dtype == SAGE_FP16)
        unpack8<__half>(v, x);
      else
        unpack8<__nv_bfloat16>(v, x);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = 0.f;
    if (c0 + e < d) {
      if (dtype == SAGE_FP32) {
        x[e] = static_cast<const float*>(src)[c0 + e];
      } else {
        const uint32_t h = static_cast<const unsigned short*>(src)[c0 + e];
        x[e] = dtype == SAGE_FP16 ? bits_to_f32<__half>(h) : bits_to_f32<__nv_bfloat16>(h);
      }
    }
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// max |x| over a row.  On the bit patterns, so that a NaN or an infinity (the largest patterns)
// is never lost, as it would be in a float maximum.
template <int LPR>
__device__ __forceinline__ float row_absmax(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return __uint_as_float(m);
}

// scale and reciprocal of a row's codes: 0 and 0 for a row of (almost) zeros, NaN and 0 for one
// that holds a NaN or an infinity (it reads back as NaN).
__device__ __forceinline__ void code_scale(float amax, float top, float* scale, float* inv) {
  const bool finite = amax < __uint_as_float(0x7F800000u), keep = finite && amax >= kTinyAmax;
  *inv = keep ? __fdiv_rn(top, amax) : 0.f;
  *scale = keep ? __fdiv_rn(amax, top) : (finite ? 0.f : __uint_as_float(0x7FC00000u));
}

// The sequence of packed token t (of `total`), and that sequence's first token and token count.  The first
// probe finds it in a batch with one token each; otherwise a binary search over the offsets.  false:
// t is behind the last sequence, or (flagged) the offsets are not non-decreasing from 0 to at most total.
__device__ __forceinline__ bool find_sequence(const int32_t* cu, int B, int t, int total, int* b_out, int* first,
                                              int* count) {
  const int end = cu[B];
  if (t >= end && end <= total) return false;
  int b = min(B - 1, t);
  if (!(cu[b] <= t && t < cu[b + 1])) {
    int lo = 0, hi = B - 1;  // the last b with cu[b] <= t
    while (lo < hi) {
      const int mid = lo + ((hi - lo + 1) >> 1);
      if (cu[mid] <= t)
        lo = mid;
      else
        hi = mid - 1;
    }
    b = lo;
  }
  const int at = cu[b], next = cu[b + 1];
  if (end > total || at < 0 || at > t || next <= t || next > end || (b == 0 && at != 0)) {
    atomicOr(&g_cache_error, kBadArg);
    return false;
  }
  *b_out = b, *first = at, *count = next - at;
  return true;
}

// Page of position pos of sequence b, or -1 (flagged) where the table has none.
__device__ __forceinline__ int page_of(const PageMap& m, int b, int pos) {
  const int i = pos >> m.page_log2;
  if (pos < 0 || i >= m.max_pages) {
    atomicOr(&g_cache_error, kBadArg);
    return -1;
  }
  const int page = m.table[b * m.table_stride + i];
  if ((unsigned)page >= (unsigned)m.num_pages) {
    atomicOr(&g_cache_error, kBadArg);
    return -1;
  }
  return page;
}

enum RowKind { kQ = 0, kK = 1, kV = 2 };

// One row group (LPR lanes) takes HC heads of one kind of one token: the HC loads are issued
// first, and the cosines, the weights and the token's place are fetched once for all of them.
template <typename T, int LPR, int HC, bool VEC, bool APPEND>
__global__ void __launch_bounds__(kThreads) head_rows_kernel(HeadRowsParams p) {
  constexpr int kGroups = kThreads / LPR;
  __shared__ float partner_buf[VEC ? 1 : kGroups * LPR * 8];
  const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR, c0 = lane * 8;
  const unsigned items = (unsigned)p.items;
  unsigned item = blockIdx.x * (unsigned)kGroups + group;
  bool live = item < items;
  if (!live) item = items - 1;  // keeps the whole warp in the shuffles
  // item -> (batch, token, chunk of HC heads)
  int b = 0;
  unsigned n, chunk;
  if (p.token_fast) {
    n = item % (unsigned)p.N;
    const unsigned rest = item / (unsigned)p.N;
    chunk = rest % (unsigned)p.chunks, b = rest / (unsigned)p.chunks;
  } else {
    chunk = item % (unsigned)p.chunks;
    const unsigned rest = item / (unsigned)p.chunks;
    n = rest % (unsigned)p.N, b = rest / (unsigned)p.N;
  }
  int kind = kQ, h0 = (int)chunk * HC, heads = p.Hq;
  if ((int)chunk >= p.q_chunks) {
    kind = kK, heads = p.Hkv, h0 = ((int)chunk - p.q_chunks) * HC;
    if (APPEND && (int)chunk >= p.q_chunks + p.k_chunks) kind = kV, h0 = ((int)chunk - p.q_chunks - p.k_chunks) * HC;
  }
  const int nh = min(HC, heads - h0);
  const HeadView& in = kind == kQ ? p.q : kind == kK ? p.k : p.v;
  const unsigned short* src = static_cast<const unsigned short*>(in.ptr) + b * in.batch + n * in.token + h0 * in.head;
  uint4 raw[HC];
#pragma unroll
  for (int i = 0; i < HC; ++i)
    raw[i] = i < nh ? load8<VEC>(src + i * in.head, c0, p.d) : make_uint4(0, 0, 0, 0);

  // ---- the token's position, and its place in the cache
  int pos = 0, page = -1;
  if (APPEND) {
    int first = (int)n, seq = (int)n, count = 1;
    if (p.cu) {
      live = live && find_sequence(p.cu, p.B, (int)n, p.N, &seq, &first, &count);
    }
    if (live) {
      const int len = p.seq_lens[seq];
      pos = len - count + ((int)n - first);
      if (!p.cu && len == 0) live = false;  // a padded slot of a decode batch
    }
    if (live) {
      page = page_of(p.map, seq, pos);
      live = page >= 0;
    }
  } else if (p.cos_sin) {
    pos = p.positions ? p.positions[b * p.pos_batch + n] : (int)n;
  }
  const bool rotate = p.cos_sin != nullptr && kind != kV;
  float cs[8], sn[8];
  const int half = p.rot >> 1;
  if (rotate) {
    if (live && (unsigned)pos >= (unsigned)p.n_pos) {
      if (lane == 0) atomicOr(&g_cache_error, kBadArg);
      live = false;
    }
    const float* row = p.cos_sin + (live ? (long long)pos * p.rot : 0);
    if (VEC && !p.interleaved) {  // rot % 16 == 0: a lane's channels lie in one half
      const int i = c0 < half ? c0 : c0 - half;
      const bool in_rot = c0 < p.rot;
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const float4 a = in_rot ? __ldg(reinterpret_cast<const float4*>(row + i + e)) : make_float4(1, 1, 1, 1);
        const float4 c = in_rot ? __ldg(reinterpret_cast<const float4*>(row + half + i + e)) : make_float4(0, 0, 0, 0);
        cs[e] = a.x, cs[e + 1] = a.y, cs[e + 2] = a.z, cs[e + 3] = a.w;
        sn[e] = c.x, sn[e + 1] = c.y, sn[e + 2] = c.z, sn[e + 3] = c.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = c0 + e, i = p.interleaved ? c >> 1 : (c < half ? c : c - half);
        cs[e] = c < p.rot ? __ldg(row + i) : 1.f;
        sn[e] = c < p.rot ? __ldg(row + half + i) : 0.f;
      }
    }
  }
  float w[8];
  const void* wp = kind == kQ ? p.q_weight : p.k_weight;
  const bool norm = p.norm && kind != kV;
  if (norm && wp) load8_param(wp, p.weight_dtype, p.vec_weight, c0, p.d, w);

#pragma unroll
  for (int i = 0; i < HC; ++i) {
    if (HC > 1 && __all_sync(0xffffffffu, i >= nh)) break;
    const int h = h0 + i;
    const bool write = live && i < nh;
    float x[8];
    unpack8<T>(raw[i], x);
    if (p.norm) {  // uniform over the warp; V rows pass through unchanged
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
      const float r = rsqrtf(row_sum<LPR>(ss) * p.inv_d + p.eps);
      if (norm) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] *= r;
          if (wp) x[e] *= w[e];
        }
      }
    }
    if (p.cos_sin) {
      if (p.interleaved) {
        if (rotate)
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float a = x[e], c = x[e + 1];
            x[e] = a * cs[e] - c * sn[e], x[e + 1] = c * cs[e + 1] + a * sn[e + 1];
          }
      } else if (VEC) {
        // the partner of channel c is c + half below half and c - half above: another lane's, the
        // same element of its eight
        const int other = c0 < half ? lane + (half >> 3) : c0 < p.rot ? lane - (half >> 3) : lane;
        const float sign = c0 < half ? -1.f : 1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float y = __shfl_sync(0xffffffffu, x[e], other, LPR);
          if (rotate) x[e] = x[e] * cs[e] + sign * y * sn[e];
        }
      } else {
        float* buf = partner_buf + group * LPR * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) buf[c0 + e] = x[e];
        __syncwarp();
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = c0 + e;
          y[e] = c < half ? -buf[c + half] : c < p.rot ? buf[c - half] : 0.f;
        }
        __syncwarp();
        if (rotate)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = x[e] * cs[e] + y[e] * sn[e];
      }
    }
    if (!APPEND || kind == kQ) {
      const HeadView& o = kind == kQ ? p.q_out : p.k_out;
      unsigned short* dst =
          static_cast<unsigned short*>(const_cast<void*>(o.ptr)) + b * o.batch + n * o.token + h * o.head;
      if (write) store8<T, VEC>(dst, c0, p.d, x, kind == kQ ? p.x_q_out : p.x_k_out);
    }
    if (APPEND) {
      if (kind == kK && p.k_mean && i < nh) {
        float m[8];
        load8_param(p.k_mean + (size_t)h * p.d, SAGE_FP32, p.vec_mean, c0, p.d, m);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __fsub_rn(x[e], m[e]);
      }
      const float amax = row_absmax<LPR>(x);  // every lane of the warp takes part
      if (kind != kQ && write && c0 < p.map.dc) {
        float scale, inv;
        code_scale(amax, kind == kK ? 127.f : 448.f, &scale, &inv);
        const bool coded = inv != 0.f;
        uint32_t word[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (kind == kK) {
            uint32_t packed = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              int code = __float2int_rn(__fmul_rn(x[4 * q + e], inv));
              code = max(-127, min(127, code));
              packed |= (uint32_t)(code & 0xFF) << (8 * e);
            }
            word[q] = coded ? packed : 0u;
          } else {
            const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
                make_float2(__fmul_rn(x[4 * q], inv), __fmul_rn(x[4 * q + 1], inv)), __NV_SATFINITE, __NV_E4M3);
            const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
                make_float2(__fmul_rn(x[4 * q + 2], inv), __fmul_rn(x[4 * q + 3], inv)), __NV_SATFINITE, __NV_E4M3);
            word[q] = coded ? (uint32_t)lo | ((uint32_t)hi << 16) : 0u;
          }
        }
        const long long row = p.map.row(page, h, pos);
        uint8_t* dst = (kind == kK ? reinterpret_cast<uint8_t*>(p.map.k8) : p.map.v8) + row * p.map.dc + c0;
        if (SAGE_STORE_OK(kind == kK ? p.x_k8 : p.x_v8, dst, 8, &g_cache_error))
          *reinterpret_cast<uint2*>(dst) = make_uint2(word[0], word[1]);
        float* sdst = (kind == kK ? p.map.ks : p.map.vs) + row;
        if (lane == 0 && SAGE_STORE_OK(kind == kK ? p.x_ks : p.x_vs, sdst, 4, &g_cache_error)) *sdst = scale;
      }
    }
  }
}

// ------------------------------------------------------------------------------------------ read back
// One group of LPR lanes per (token, kv head): 16 K and 16 V codes to a lane, read as 16-byte
// vectors, written as 16-bit values.
template <typename T, int LPR, bool VEC>
__global__ void __launch_bounds__(kThreads) gather_kernel(GatherParams p) {
  constexpr int kGroups = kThreads / LPR;
  const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR, c0 = lane * 16;
  const unsigned item = blockIdx.x * (unsigned)kGroups + group;
  if (item >= (unsigned)p.items || c0 >= p.map.dc) return;
  const unsigned t = item / (unsigned)p.map.Hkv;
  const int h = (int)(item % (unsigned)p.map.Hkv);
  int seq, first, count;
  if (!find_sequence(p.cu, p.B, (int)t, p.T, &seq, &first, &count)) return;
  const int pos = (int)t - first + (p.starts ? p.starts[seq] : 0);
  const int page = page_of(p.map, seq, pos);
  if (page < 0) return;
  const long long row = p.map.row(page, h, pos);
  const uint4 kc = *reinterpret_cast<const uint4*>(p.map.k8 + row * p.map.dc + c0);
  const uint4 vc = *reinterpret_cast<const uint4*>(p.map.v8 + row * p.map.dc + c0);
  const float ks = p.map.ks[row], vs = p.map.vs[row];
  unsigned short* ko = static_cast<unsigned short*>(p.k_out) + (long long)item * p.d;
  unsigned short* vo = static_cast<unsigned short*>(p.v_out) + (long long)item * p.d;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int c = c0 + 8 * q;
    float x[8], m[8];
    if (p.k_mean) load8_param(p.k_mean + (size_t)h * p.d, SAGE_FP32, p.vec_mean, c, p.d, m);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t w = (&kc.x)[2 * q + (e >> 2)];
      x[e] = __fmul_rn((float)(int)(signed char)(w >> (8 * (e & 3))), ks);
      if (p.k_mean) x[e] = __fadd_rn(x[e], m[e]);
    }
    store8<T, VEC>(ko, c, p.d, x, p.x_k_out);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const uint32_t w = (&vc.x)[2 * q + (e >> 2)];
      const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (8 * (e & 3))), __NV_E4M3);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
      x[e] = __fmul_rn(f.x, vs), x[e + 1] = __fmul_rn(f.y, vs);
    }
    store8<T, VEC>(vo, c, p.d, x, p.x_v_out);
  }
}

template <typename T, int LPR, int HC, bool VEC>
cudaError_t launch_rows(const HeadRowsParams& p, cudaStream_t st) {
  constexpr int kGroups = kThreads / LPR;
  const unsigned grid = (unsigned)((p.items + kGroups - 1) / kGroups);
  if (p.append)
    head_rows_kernel<T, LPR, HC, VEC, true><<<grid, kThreads, 0, st>>>(p);
  else
    head_rows_kernel<T, LPR, HC, VEC, false><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int LPR>
cudaError_t launch_rows_lpr(const HeadRowsParams& p, cudaStream_t st) {
  if (!p.vec) return launch_rows<T, LPR, 1, false>(p, st);
  return p.heads_per_group == 4 ? launch_rows<T, LPR, 4, true>(p, st) : launch_rows<T, LPR, 1, true>(p, st);
}

template <typename T>
cudaError_t launch_rows_t(const HeadRowsParams& p, cudaStream_t st) {
  return p.d <= 64 ? launch_rows_lpr<T, 8>(p, st) : p.d <= 128 ? launch_rows_lpr<T, 16>(p, st)
                                                               : launch_rows_lpr<T, 32>(p, st);
}

template <typename T, int LPR>
cudaError_t launch_gather_lpr(const GatherParams& p, cudaStream_t st) {
  constexpr int kGroups = kThreads / LPR;
  const unsigned grid = (unsigned)((p.items + kGroups - 1) / kGroups);
  if (p.vec)
    gather_kernel<T, LPR, true><<<grid, kThreads, 0, st>>>(p);
  else
    gather_kernel<T, LPR, false><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_gather_t(const GatherParams& p, cudaStream_t st) {
  return p.d <= 64 ? launch_gather_lpr<T, 4>(p, st) : p.d <= 128 ? launch_gather_lpr<T, 8>(p, st)
                                                                 : launch_gather_lpr<T, 16>(p, st);
}

}  // namespace

cudaError_t launch_head_rows(const HeadRowsParams& p, int dtype, cudaStream_t st) {
  return dtype == SAGE_FP16 ? launch_rows_t<__half>(p, st) : launch_rows_t<__nv_bfloat16>(p, st);
}

cudaError_t launch_cache_gather(const GatherParams& p, int dtype, cudaStream_t st) {
  return dtype == SAGE_FP16 ? launch_gather_t<__half>(p, st) : launch_gather_t<__nv_bfloat16>(p, st);
}

}  // namespace sage
