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
// owned by 8, 16 or 32 consecutive lanes, eight channels to a lane, so that the sum of squares and
// the amax are lane shuffles and no barrier is on the path.  Where halves rotate together a lane owns
// four channels of each half, at the same place: both partners of its four pairs, and four angles
// for eight channels.
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

constexpr int kThreads = 128;
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

// Pairs of fp32 values, two to an instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
// The larger of two values, a NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// A lane's eight channels of a row, widened.
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& v, float2 (&x)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t w = (&v.x)[e];
    x[e] = make_float2(bits_to_f32<T>(w & 0xFFFFu), bits_to_f32<T>(w >> 16));
  }
}

// How a lane's eight channels lie in a row, and how they are read:
//   kScalar  c .. c + 7, element by element (any alignment, any head size)
//   kWide    c .. c + 7, 16 bytes
//   kHalves  a .. a + 3 and b .. b + 3, 8 bytes each: the same four places of the two rotated halves, or
//            (behind the rotated channels) eight in a row
enum Mode { kScalar, kWide, kHalves };

template <int MODE>
__device__ __forceinline__ uint4 load8(const unsigned short* row, int a, int b, int d) {
  if (MODE == kWide) return a < d ? *reinterpret_cast<const uint4*>(row + a) : make_uint4(0, 0, 0, 0);
  if (MODE == kHalves) {
    const uint2 x = a < d ? *reinterpret_cast<const uint2*>(row + a) : make_uint2(0, 0);
    const uint2 y = b < d ? *reinterpret_cast<const uint2*>(row + b) : make_uint2(0, 0);
    return make_uint4(x.x, x.y, y.x, y.y);
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (a + e < d) w[e >> 1] |= (uint32_t)row[a + e] << (16 * (e & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The same, rounded from fp32 and stored.
template <typename T, int MODE>
__device__ __forceinline__ void store8(unsigned short* row, int a, int b, int d, const float2 (&x)[4],
                                       const Extent& ext) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = pack2(x[e].x, x[e].y, T());
  if (MODE == kWide) {
    if (a < d && SAGE_STORE_OK(ext, row + a, 16, &g_cache_error))
      *reinterpret_cast<uint4*>(row + a) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if (MODE == kHalves) {
    if (a < d && SAGE_STORE_OK(ext, row + a, 8, &g_cache_error)) *reinterpret_cast<uint2*>(row + a) = make_uint2(w[0], w[1]);
    if (b < d && SAGE_STORE_OK(ext, row + b, 8, &g_cache_error)) *reinterpret_cast<uint2*>(row + b) = make_uint2(w[2], w[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (a + e < d && SAGE_STORE_OK(ext, row + a + e, 2, &g_cache_error))
        row[a + e] = (unsigned short)(w[e >> 1] >> (16 * (e & 1)));
  }
}

// Four values c .. c + 3 of a vector of d fp32 or 16-bit values (zero past d).
__device__ __forceinline__ void load4_param(const void* src, int dtype, bool vec, int c, int d, float* x) {
  if (vec && c < d) {
    if (dtype == SAGE_FP32) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(src) + c));
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    } else {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const unsigned short*>(src) + c));
      const uint32_t h[4] = {v.x & 0xFFFFu, v.x >> 16, v.y & 0xFFFFu, v.y >> 16};
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = dtype == SAGE_FP16 ? bits_to_f32<__half>(h[e]) : bits_to_f32<__nv_bfloat16>(h[e]);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = 0.f;
    if (c + e < d) {
      if (dtype == SAGE_FP32) {
        x[e] = static_cast<const float*>(src)[c + e];
      } else {
        const uint32_t h = static_cast<const unsigned short*>(src)[c + e];
        x[e] = dtype == SAGE_FP16 ? bits_to_f32<__half>(h) : bits_to_f32<__nv_bfloat16>(h);
      }
    }
  }
}

// Sums or maxima (NaN if any is one) over the LPR lanes of HC rows, one value per lane and row.  HC = 1: every
// lane gets its row's.  HC = 4: lane l gets row 2 (l & 1) + (l >> 1 & 1)'s, by halving the values with the first two
// exchanges: five shuffles for 16 lanes where row by row takes sixteen, and what follows from the
// sum (a root, a division) is then done once, not four times.
template <int LPR, int HC, bool MAX>
__device__ __forceinline__ float reduce_rows(const float (&v)[HC]) {
  const auto op = [](float a, float b) { return MAX ? max_nan(a, b) : a + b; };
  float r = v[0];
  int from = 1;
  if (HC == 4) {
    const bool b0 = threadIdx.x & 1, b1 = threadIdx.x & 2;
    const float u0 = op(b0 ? v[2 % HC] : v[0], __shfl_xor_sync(0xffffffffu, b0 ? v[0] : v[2 % HC], 1));
    const float u1 = op(b0 ? v[3 % HC] : v[1 % HC], __shfl_xor_sync(0xffffffffu, b0 ? v[1 % HC] : v[3 % HC], 1));
    r = op(b1 ? u1 : u0, __shfl_xor_sync(0xffffffffu, b1 ? u0 : u1, 2));
    from = 4;
  }
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1)
    if (o >= from) r = op(r, __shfl_xor_sync(0xffffffffu, r, o));
  return r;
}
// Row i's value of what reduce_rows left in the lanes, to all of them.
template <int LPR, int HC>
__device__ __forceinline__ float of_row(float v, int i) {
  return HC == 1 ? v : __shfl_sync(0xffffffffu, v, (i >> 1) | (i & 1) << 1, LPR);
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

// Four codes of a row.  INT8: the product rounded to an integer by adding 1.5 * 2^23 (ties to even, as rint),
// whose low byte is then the code; |x| inv <= 127 (1 + 2^-23), so that no code passes +-127.
__device__ __forceinline__ uint32_t code4_int8(float2 x, float2 y, float2 inv) {
  const float big = 12582912.f;  // (added one by one: a packed sum of a packed product would be fused with it)
  const float2 u = mul2(x, inv), v = mul2(y, inv);
  return __byte_perm(__byte_perm(__float_as_uint(__fadd_rn(u.x, big)), __float_as_uint(__fadd_rn(u.y, big)), 0x0040),
                     __byte_perm(__float_as_uint(__fadd_rn(v.x, big)), __float_as_uint(__fadd_rn(v.y, big)), 0x0040),
                     0x5410);
}
__device__ __forceinline__ uint32_t code4_e4m3(float2 x, float2 y, float2 inv) {
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(mul2(x, inv), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(mul2(y, inv), __NV_SATFINITE, __NV_E4M3);
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

enum RowKind { kQ = 0, kK = 1, kV = 2 };

// The rows of one kind.  An item: HC heads of one token, taken by one group of LPR lanes.  The cosines, the
// weights and the token's place are fetched once for all of them, and the heads of a group's next item
// are loaded while it works on this one: without that, 24 warps to an SM spend most of their time
// waiting for the first of a chain of loads.
template <typename T, int LPR, int HC, int MODE, bool APPEND, int KIND>
__device__ __forceinline__ void head_rows(const HeadRowsParams& p, const HeadRows& k, unsigned cta, float* partner_buf) {
  constexpr unsigned kGroups = kThreads / LPR;
  constexpr bool kCoded = APPEND && KIND != kQ;
  const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const int half = p.rot >> 1;
  int a = lane * 8, b = a + 4;
  if (MODE == kHalves) {
    if (4 * lane < half)
      a = 4 * lane, b = half + a;
    else
      a = p.rot + 8 * (lane - (half >> 2)), b = a + 4;
  }
  // This CTA's run of rounds of its groups; a group's items are kGroups apart.
  const unsigned first = (cta * k.rounds + min(cta, k.rounds_more)) * kGroups;
  const unsigned end = min(first + (k.rounds + (cta < k.rounds_more ? 1 : 0)) * kGroups, k.items);
  if (first >= end) return;
  const unsigned r0 = p.token_fast ? p.N : k.chunks, r1 = p.token_fast ? k.chunks : p.N;
  unsigned item = first + group;
  unsigned d0 = item % r0, d1 = item / r0, batch = d1 / r1;
  d1 -= batch * r1;
  const unsigned short* src;
  unsigned short* dst;
  {
    const unsigned n = p.token_fast ? d0 : d1, h = (p.token_fast ? d1 : d0) * HC;
    src = static_cast<const unsigned short*>(k.in.ptr) + batch * k.in.batch + n * k.in.token + h * k.in.head;
    dst = static_cast<unsigned short*>(const_cast<void*>(k.out.ptr)) + batch * k.out.batch + n * k.out.token + h * k.out.head;
  }
  uint4 raw[HC];
  const auto load_item = [&] {
    const int nh = item < end ? k.H - (int)(p.token_fast ? d1 : d0) * HC : 0;
#pragma unroll
    for (int i = 0; i < HC; ++i) raw[i] = i < nh ? load8<MODE>(src + i * k.in.head, a, b, p.d) : make_uint4(0, 0, 0, 0);
  };
  load_item();
  int seq = 0, seq_first = 0, seq_end = -1, seq_base = 0;  // append: the sequence last looked up, its position of token 0
  const bool weights = k.weight != nullptr;
  float2 w[4];
  if (KIND != kV && weights) {
    float f[8];
    load4_param(k.weight, p.weight_dtype, p.vec_weight, a, p.d, f);
    load4_param(k.weight, p.weight_dtype, p.vec_weight, b, p.d, f + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = make_float2(f[2 * e], f[2 * e + 1]);
  }
  const bool turn = MODE == kHalves ? a < half : a < p.rot;  // this lane's channels turn (rot 0: none does)

  // Every lane of a warp makes the same number of rounds: the shuffles need them all.
#pragma unroll 1
  for (unsigned round = first; round < end; round += kGroups) {
    uint4 cur[HC];
#pragma unroll
    for (int i = 0; i < HC; ++i) cur[i] = raw[i];
    const unsigned n = p.token_fast ? d0 : d1, cbatch = batch;
    const int h0 = (int)(p.token_fast ? d1 : d0) * HC;
    bool live = item < end;
    unsigned short* const out = dst;
    // ---- the next item's heads
    item += kGroups;
    src += k.in_step;
    if (!kCoded) dst += k.out_step;
    d0 += k.step[0], d1 += k.step[1], batch += k.step[2];
    if (d0 >= r0) {
      d0 -= r0, ++d1, src += k.in_carry[0];
      if (!kCoded) dst += k.out_carry[0];
    }
    if (d1 >= r1) {
      d1 -= r1, ++batch, src += k.in_carry[1];
      if (!kCoded) dst += k.out_carry[1];
    }
    load_item();

    // ---- this token's position, and its place in the cache
    int pos = 0, page = -1;
    if (APPEND) {
      const int t = (int)n;
      if (p.cu) {
        if (live && (t < seq_first || t >= seq_end)) {
          int count = 0;
          live = find_sequence(p.cu, p.B, t, p.N, &seq, &seq_first, &count);
          seq_end = live ? seq_first + count : -1;
          if (live) seq_base = p.seq_lens[seq] - seq_end;
        }
      } else if (live) {
        seq = t, seq_base = p.seq_lens[t] - 1 - t;
        if (seq_base == -1 - t) live = false;  // a padded slot of a decode batch
      }
      pos = seq_base + t;
      if (live) {
        page = page_of(p.map, seq, pos);
        live = page >= 0;
      }
    } else if (p.cos_sin) {
      pos = p.positions && live ? p.positions[cbatch * p.pos_batch + n] : (int)n;
    }
    if (p.cos_sin && live && (unsigned)pos >= (unsigned)p.n_pos) {
      atomicOr(&g_cache_error, kBadArg);
      live = false;
    }
    const float* angles = p.cos_sin + (live ? (long long)pos * p.rot : 0);
    float4 cs, sn;
    if (KIND != kV && MODE != kScalar && turn) {
      cs = __ldg(reinterpret_cast<const float4*>(angles + (MODE == kHalves ? a : a >> 1)));
      sn = __ldg(reinterpret_cast<const float4*>(angles + half + (MODE == kHalves ? a : a >> 1)));
    }
    const long long row0 = kCoded && live ? p.map.row(page, h0, pos) : 0;

    const bool norm = KIND != kV && p.norm;
    float r = 1.f;  // reduce_rows' layout
    if (norm) {
      float ss[HC];
#pragma unroll
      for (int i = 0; i < HC; ++i) {
        float2 x[4], q = make_float2(0.f, 0.f);
        unpack8<T>(cur[i], x);
#pragma unroll
        for (int e = 0; e < 4; ++e) q = fma2(x[e], x[e], q);
        ss[i] = q.x + q.y;
      }
      r = rsqrtf(reduce_rows<LPR, HC, false>(ss) * p.inv_d + p.eps);
    }
    float2 coded[kCoded ? HC : 1][4];
    float amax[HC];
#pragma unroll
    for (int i = 0; i < HC; ++i) {
      float2 x[4];
      unpack8<T>(cur[i], x);
      if (norm) {
        const float ri = of_row<LPR, HC>(r, i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = mul2(x[e], make_float2(ri, ri));
          if (weights) x[e] = mul2(x[e], w[e]);
        }
      }
      if (KIND != kV && MODE == kScalar) {
        if (p.cos_sin) {  // uniform; the partners through shared memory
          float* buf = partner_buf + group * LPR * 8;
#pragma unroll
          for (int e = 0; e < 4; ++e) buf[a + 2 * e] = x[e].x, buf[a + 2 * e + 1] = x[e].y;
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int c = a + e;
            if (c >= p.rot) continue;
            const bool low = p.interleaved ? !(c & 1) : c < half;
            const int i_angle = p.interleaved ? c >> 1 : low ? c : c - half;
            const float y = buf[p.interleaved ? c ^ 1 : low ? c + half : c - half];
            float& z = e & 1 ? x[e >> 1].y : x[e >> 1].x;
            z = z * __ldg(angles + i_angle) + (low ? -y : y) * __ldg(angles + half + i_angle);
          }
          __syncwarp();
        }
      } else if (KIND != kV && MODE == kHalves && turn) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 c = e ? make_float2(cs.z, cs.w) : make_float2(cs.x, cs.y);
          const float2 n = e ? make_float2(sn.z, sn.w) : make_float2(sn.x, sn.y);
          const float2 u = x[e], v = x[2 + e];
          x[e] = fma2(v, make_float2(-n.x, -n.y), mul2(u, c));
          x[2 + e] = fma2(u, n, mul2(v, c));
        }
      } else if (KIND != kV && MODE == kWide && turn) {
        const float c4[4] = {cs.x, cs.y, cs.z, cs.w}, s4[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] = fma2(make_float2(x[e].y, x[e].x), make_float2(-s4[e], s4[e]), mul2(x[e], make_float2(c4[e], c4[e])));
      }
      if (!kCoded) {
        if (live && (HC == 1 || h0 + i < k.H)) store8<T, MODE>(out + i * k.out.head, a, b, p.d, x, k.x_out);
        continue;
      }
      if (KIND == kK && p.k_mean && (HC == 1 || h0 + i < k.H)) {
        const float* mean = p.k_mean + (live ? (h0 + i) * p.d : 0);
        float m[8];
        load4_param(mean, SAGE_FP32, p.vec_mean, a, p.d, m);
        load4_param(mean, SAGE_FP32, p.vec_mean, b, p.d, m + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] = make_float2(__fsub_rn(x[e].x, m[2 * e]), __fsub_rn(x[e].y, m[2 * e + 1]));
      }
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max_nan(max_nan(top, fabsf(x[e].x)), fabsf(x[e].y)), coded[kCoded ? i : 0][e] = x[e];
      amax[i] = top;
    }
    if (!kCoded) continue;
    float scale, inv;  // reduce_rows' layout
    code_scale(reduce_rows<LPR, HC, true>(amax), KIND == kK ? 127.f : 448.f, &scale, &inv);
#pragma unroll
    for (int i = 0; i < HC; ++i) {
      const float iv = of_row<LPR, HC>(inv, i);
      const float2 inv2 = make_float2(iv, iv);
      const float2(&x)[4] = coded[kCoded ? i : 0];
      uint32_t w0 = KIND == kK ? code4_int8(x[0], x[1], inv2) : code4_e4m3(x[0], x[1], inv2);
      uint32_t w1 = KIND == kK ? code4_int8(x[2], x[3], inv2) : code4_e4m3(x[2], x[3], inv2);
      if (iv == 0.f) w0 = w1 = 0;  // also where a NaN or an infinity times 0 went into the codes
      if (live && (HC == 1 || h0 + i < k.H)) {
        const long long row = row0 + ((long long)i << p.map.page_log2);
        uint8_t* code = (KIND == kK ? reinterpret_cast<uint8_t*>(p.map.k8) : p.map.v8) + row * p.map.dc;
        const Extent& xc = KIND == kK ? p.x_k8 : p.x_v8;
        if (MODE == kHalves) {
          if (a < p.map.dc && SAGE_STORE_OK(xc, code + a, 4, &g_cache_error)) *reinterpret_cast<uint32_t*>(code + a) = w0;
          if (b < p.map.dc && SAGE_STORE_OK(xc, code + b, 4, &g_cache_error)) *reinterpret_cast<uint32_t*>(code + b) = w1;
        } else if (a < p.map.dc && SAGE_STORE_OK(xc, code + a, 8, &g_cache_error)) {
          *reinterpret_cast<uint2*>(code + a) = make_uint2(w0, w1);
        }
      }
    }
    const int my_row = HC == 1 ? 0 : 2 * (lane & 1) + (lane >> 1 & 1);
    float* sdst = (KIND == kK ? p.map.ks : p.map.vs) + row0 + ((long long)my_row << p.map.page_log2);
    if (lane < HC && live && h0 + my_row < k.H && SAGE_STORE_OK(KIND == kK ? p.x_ks : p.x_vs, sdst, 4, &g_cache_error))
      *sdst = scale;
  }
}

// Large calls: every CTA takes its share of each kind, one after the other, so that all end together
// whatever a kind's rows cost.  Small ones (`apart`): the kinds have CTAs of their own, which work at the same time.
template <typename T, int LPR, int HC, int MODE, bool APPEND>
__global__ void __launch_bounds__(kThreads, HC > 1 ? 5 : 8) head_rows_kernel(const __grid_constant__ HeadRowsParams p) {
  __shared__ float partner_buf[MODE == kScalar ? kThreads * 8 : 1];
  const unsigned cta = blockIdx.x, q = p.apart ? p.kind[kQ].ctas : 0, k = p.apart ? q + p.kind[kK].ctas : 0;
  if (!p.apart || cta < q) head_rows<T, LPR, HC, MODE, APPEND, kQ>(p, p.kind[kQ], cta, partner_buf);
  if (!p.apart || (cta >= q && cta < k)) head_rows<T, LPR, HC, MODE, APPEND, kK>(p, p.kind[kK], cta - q, partner_buf);
  if (APPEND && (!p.apart || cta >= k))
    head_rows<T, LPR, HC, MODE == kHalves ? kWide : MODE, APPEND, kV>(p, p.kind[kV], cta - k, partner_buf);
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
    float2 x[4];
    float m[8];
    if (p.k_mean) {
      load4_param(p.k_mean + (size_t)h * p.d, SAGE_FP32, p.vec_mean, c, p.d, m);
      load4_param(p.k_mean + (size_t)h * p.d, SAGE_FP32, p.vec_mean, c + 4, p.d, m + 4);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t w = (&kc.x)[2 * q + (e >> 1)] >> (16 * (e & 1));
      x[e] = mul2(make_float2((float)(int)(signed char)w, (float)(int)(signed char)(w >> 8)), make_float2(ks, ks));
      if (p.k_mean) x[e] = make_float2(__fadd_rn(x[e].x, m[2 * e]), __fadd_rn(x[e].y, m[2 * e + 1]));
    }
    store8<T, VEC ? kWide : kScalar>(ko, c, c + 4, p.d, x, p.x_k_out);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t w = (&vc.x)[2 * q + (e >> 1)] >> (16 * (e & 1));
      const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w, __NV_E4M3);
      x[e] = mul2(__half22float2(*reinterpret_cast<const __half2*>(&r)), make_float2(vs, vs));
    }
    store8<T, VEC ? kWide : kScalar>(vo, c, c + 4, p.d, x, p.x_v_out);
  }
}

template <typename T, int LPR, int HC, int MODE>
cudaError_t launch_rows(HeadRowsParams p, cudaStream_t st) {
  constexpr long long kGroups = kThreads / LPR;
  const unsigned most = 148 * (HC > 1 ? 5 : 8);  // one wave
  unsigned all = 0;
  const auto rounds_of = [&](const HeadRows& k) { return (unsigned)((k.items + kGroups - 1) / kGroups); };
  for (const HeadRows& k : p.kind) all += rounds_of(k);
  p.apart = all <= most;
  unsigned grid = 0;
  for (HeadRows& k : p.kind) {
    const unsigned rounds = rounds_of(k);
    k.ctas = p.apart ? rounds : most;
    grid = p.apart ? grid + k.ctas : most;
    if (!k.ctas) continue;
    k.rounds = rounds / k.ctas, k.rounds_more = rounds % k.ctas;
    if (!rounds) continue;
    // mixed-radix step of kGroups items, and what the addresses move by
    const long long r0 = p.token_fast ? p.N : k.chunks, r1 = p.token_fast ? k.chunks : p.N;
    k.step[0] = (unsigned)(kGroups % r0), k.step[1] = (unsigned)(kGroups / r0 % r1);
    k.step[2] = (unsigned)(kGroups / r0 / r1);
    const auto moves = [&](const HeadView& v, long long* step, long long* carry) {
      const long long s0 = p.token_fast ? v.token : v.head * HC, s1 = p.token_fast ? v.head * HC : v.token;
      *step = k.step[0] * s0 + k.step[1] * s1 + k.step[2] * v.batch;
      carry[0] = s1 - r0 * s0, carry[1] = v.batch - r1 * s1;
    };
    moves(k.in, &k.in_step, k.in_carry);
    moves(k.out, &k.out_step, k.out_carry);
  }
  if (p.append)
    head_rows_kernel<T, LPR, HC, MODE, true><<<grid, kThreads, 0, st>>>(p);
  else
    head_rows_kernel<T, LPR, HC, MODE, false><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int LPR>
cudaError_t launch_rows_lpr(const HeadRowsParams& p, cudaStream_t st) {
  if (!p.vec) return launch_rows<T, LPR, 1, kScalar>(p, st);
  if (p.cos_sin && !p.interleaved)
    return p.heads_per_group == 4 ? launch_rows<T, LPR, 4, kHalves>(p, st) : launch_rows<T, LPR, 1, kHalves>(p, st);
  return p.heads_per_group == 4 ? launch_rows<T, LPR, 4, kWide>(p, st) : launch_rows<T, LPR, 1, kWide>(p, st);
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
