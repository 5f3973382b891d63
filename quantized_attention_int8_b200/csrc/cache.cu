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
// Everything here moves bytes: about ten operations per element.  Norm and rotation of the video-DiT heads (B1
// N32768 Hq24 Hkv24 d128 bf16, 822 MB) take 133 us, 6.2 TB/s: HBM bounds them.  The write of four
// 8192-token prompts (Hq32 Hkv8 d128 fp16 with norm, rotation and k_mean, 740 MB) takes 160 us, 4.6
// TB/s: the coded rows are a third of the rows and over half of the instructions; HBM is 55% busy and 2.6 of 4
// instructions issue per cycle, with load and fixed latencies the largest stalls.  The read back of 16 prefixes (1 to 8192 tokens, Hkv8 d128, 401 MB) takes
// 75 us, 5.3 TB/s: the loads' latency, at 20 warps to an SM.  Short calls are launch latency: 4 us in a graph, 5.1 to
// 5.8 us through the package.  Heads of 40, 80 and 160 channels leave 3 of 8 lanes idle (norm and rotation of heads of 40, 80,
// 96, 128 and 160 channels, 0.34 GB each: 3.7, 3.7, 4.3, 5.3 and 3.8 TB/s).
//
// A row (one head of one token) is
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
  if (e != cudaSuccess || *value == 0) return e;  // nothing to clear: one copy less
  const int zero = 0;
  return cudaMemcpyToSymbol(g_cache_error, &zero, sizeof(int));
}

namespace {

constexpr int kThreads = 128;
constexpr int kBadArg = 2;  // the error word's bit for SAGE_ERR_INVALID_ARG
// Rows whose largest magnitude is below this (or zero) are stored as zeros: 127 / amax and
// 448 / amax then stay finite.
constexpr float kTinyAmax = 7.888609052210118e-31f;  // 2^-100

// Lets the next grid be set up (it waits for this one before it touches memory), and waits for the one before.
__device__ __forceinline__ void begin_dependent() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

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
//   kAny     as kWide, where the rotated channels are no multiple of eight: a lane's pairs are not its own, and
//            partners and angles go through shared memory, as in kScalar
enum Mode { kScalar, kWide, kHalves, kAny };

template <int MODE>
__device__ __forceinline__ uint4 load8(const unsigned short* row, int a, int b, int d) {
  if (MODE == kWide || MODE == kAny) return a < d ? *reinterpret_cast<const uint4*>(row + a) : make_uint4(0, 0, 0, 0);
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
  if (MODE == kWide || MODE == kAny) {
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

// Sums or maxima (NaN if any is one) over the LPR lanes of HC rows, one value per lane and row.  Lane l gets that of
// row_of_lane, by halving the values with the first exchanges: for four rows five shuffles of 16 lanes where
// row by row takes sixteen, and what follows from the sum (a root, a division) is done once, not four
// times.
template <int HC>
__device__ __forceinline__ int row_of_lane(int lane) {
  return HC == 1 ? 0 : HC == 2 ? (lane & 1) : 2 * (lane & 1) + (lane >> 1 & 1);
}
template <int LPR, int HC, bool MAX>
__device__ __forceinline__ float reduce_rows(const float (&v)[HC]) {
  const auto op = [](float a, float b) { return MAX ? max_nan(a, b) : a + b; };
  float r = v[0];
  int from = 1;
  if (HC == 2) {
    const bool b0 = threadIdx.x & 1;
    r = op(b0 ? v[1 % HC] : v[0], __shfl_xor_sync(0xffffffffu, b0 ? v[0] : v[1 % HC], 1));
    from = 2;
  }
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
  return HC == 1 ? v : __shfl_sync(0xffffffffu, v, HC == 2 ? i : (i >> 1) | (i & 1) << 1, LPR);
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
// t is behind the last sequence, or (flagged) it meets offsets that do not go from 0 to at most total without falling.
__device__ __forceinline__ bool find_sequence(const int32_t* cu, int B, int t, int total, int* b_out, int* first,
                                              int* count) {
  const int end = cu[B];
  if (t >= end && end >= 0 && end <= total) {
    if (cu[0] != 0) atomicOr(&g_cache_error, kBadArg);
    return false;
  }
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

// Heads that a group takes at a time.  Four; coded keys two, whose fp32 rows stay in registers from the amax to the
// codes: with four, 96 registers, spills and five CTAs to an SM, the write of four 8192-token prompts took 169
// us, with two and six CTAs 160.
__host__ __device__ constexpr int heads_at_a_time(int hc, bool append, int kind) { return append && kind == kK && hc == 4 ? 2 : hc; }

// The rows of one kind.  A group of LPR lanes takes HC heads of one token at a time, and loads the heads of its next
// round while it works on this one.  (One round to a warp, with all its loads after one another: video-DiT 211
// us.)
template <typename T, int LPR, int HC, int MODE, bool APPEND, int KIND>
__device__ __forceinline__ void head_rows(const HeadRowsParams& p, const HeadRows& k, unsigned cta, float* partner_buf,
                                          float2* turns) {
  constexpr unsigned kGroups = kThreads / LPR;
  constexpr bool kCoded = APPEND && KIND != kQ, kShared = MODE == kScalar || MODE == kAny;
  const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const int half = p.rot >> 1;
  int a = lane * 8, b = a + 4;
  if (MODE == kHalves) {
    if (4 * lane < half)
      a = 4 * lane, b = half + a;
    else
      a = p.rot + 8 * (lane - (half >> 2)), b = a + 4;
  }
  // This CTA's run of rounds.  A round: one chunk of heads of kGroups tokens, a group each; the chunks run
  // faster than the tokens, so that a group looks its token up once for all of them, and the groups'
  // rows are neighbours in every layout (and in the cache).
  const unsigned rounds = k.rounds + (cta < k.rounds_more ? 1 : 0);
  if (rounds == 0) return;
  const unsigned round0 = cta * k.rounds + min(cta, k.rounds_more);
  unsigned chunk = round0 % k.chunks, t_flat = round0 / k.chunks * kGroups + group, n, batch;
  const unsigned short* src;
  unsigned short* dst;
  const auto place_at_token = [&] {
    batch = t_flat / (unsigned)p.N, n = t_flat - batch * p.N;
    src = static_cast<const unsigned short*>(k.in.ptr) + batch * k.in.batch + n * k.in.token + chunk * k.in_chunk;
    dst = static_cast<unsigned short*>(const_cast<void*>(k.out.ptr)) + batch * k.out.batch + n * k.out.token +
          chunk * k.out_chunk;
  };
  place_at_token();
  uint4 raw[HC];
  const auto load_item = [&] {
    const int nh = t_flat < p.tokens ? k.H - (int)chunk * HC : 0;
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
  // of the token last looked up
  unsigned token = ~0u;
  bool token_ok = false;
  float4 cs, sn;
  uint8_t* codes = nullptr;
  float* scales = nullptr;
  const unsigned head_rows = 1u << p.map.page_log2, head_codes = head_rows * p.map.dc;  // of a page

  // Every lane of a warp makes the same number of rounds: the shuffles need them all.
#pragma unroll 1
  for (unsigned round = 0; round < rounds; ++round) {
    uint4 cur[HC];
#pragma unroll
    for (int i = 0; i < HC; ++i) cur[i] = raw[i];
    const unsigned cn = n, cbatch = batch, ct = t_flat;
    const int h0 = (int)chunk * HC;
    const bool there = t_flat < p.tokens;
    unsigned short* const out = dst;
    // ---- the next round's heads
    if (++chunk == k.chunks) {
      chunk = 0, t_flat += kGroups;
      if (n + kGroups < (unsigned)p.N) {
        n += kGroups, src += k.in_tokens;
        if (!kCoded) dst += k.out_tokens;
      } else {
        place_at_token();
      }
    } else {
      src += k.in_chunk;
      if (!kCoded) dst += k.out_chunk;
    }
    load_item();

    // ---- this token's position, its cosines, and its place in the cache
    if (there && ct != token) {
      token = ct, token_ok = true;
      int pos = 0, page = -1;
      if (APPEND) {
        const int t = (int)cn;
        if (p.cu) {
          if (t < seq_first || t >= seq_end) {
            int count = 0;
            token_ok = find_sequence(p.cu, p.B, t, p.N, &seq, &seq_first, &count);
            seq_end = token_ok ? seq_first + count : -1;
            if (token_ok) seq_base = p.seq_lens[seq] - seq_end;
          }
        } else {
          seq = t, seq_base = p.seq_lens[t] - 1 - t;
          if (seq_base == -1 - t) token_ok = false;  // a padded slot of a decode batch
        }
        pos = seq_base + t;
        if (token_ok) page = page_of(p.map, seq, pos), token_ok = page >= 0;
      } else if (p.cos_sin) {
        pos = p.positions ? p.positions[cbatch * p.pos_batch + cn] : (int)cn;
      }
      if (p.cos_sin && token_ok && (unsigned)pos >= (unsigned)p.n_pos) {
        atomicOr(&g_cache_error, kBadArg);
        token_ok = false;
      }
      const float* angles = p.cos_sin + (token_ok ? (long long)pos * p.rot : 0);
      if (KIND != kV && kShared) {
        if (p.cos_sin)
#pragma unroll 1
          for (int e = 0; e < 8; ++e) {  // this lane's own: no barrier
            const int c = a + e, i = p.interleaved ? c >> 1 : c < half ? c : c - half;
            if (c >= p.rot) break;
            turns[e * kThreads + threadIdx.x] = make_float2(__ldg(angles + i), __ldg(angles + half + i));
          }
      } else if (KIND != kV && turn) {
        cs = __ldg(reinterpret_cast<const float4*>(angles + (MODE == kHalves ? a : a >> 1)));
        sn = __ldg(reinterpret_cast<const float4*>(angles + half + (MODE == kHalves ? a : a >> 1)));
      }
      if (kCoded && token_ok) {
        const long long row = p.map.row(page, 0, pos);
        codes = (KIND == kK ? reinterpret_cast<uint8_t*>(p.map.k8) : p.map.v8) + row * p.map.dc;
        scales = (KIND == kK ? p.map.ks : p.map.vs) + row;
      }
    }
    const bool live = there && token_ok;

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
    float2 coded[KIND == kK && kCoded ? HC : 1][4];
    float amax[HC];
#pragma unroll
    for (int i = 0; i < HC; ++i) {
      if (KIND == kV) {  // on the bit patterns: a NaN or an infinity is the largest
        const uint32_t m = __vmaxu2(__vmaxu2(cur[i].x & 0x7FFF7FFFu, cur[i].y & 0x7FFF7FFFu),
                                    __vmaxu2(cur[i].z & 0x7FFF7FFFu, cur[i].w & 0x7FFF7FFFu));
        amax[i] = bits_to_f32<T>(max(m & 0xFFFFu, m >> 16));
        continue;
      }
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
      if (KIND != kV && kShared) {
        if (p.cos_sin) {  // uniform
          float* buf = partner_buf + group * LPR * 8;
#pragma unroll
          for (int e = 0; e < 4; ++e) *reinterpret_cast<float2*>(buf + a + 2 * e) = x[e];
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int c = a + e;
            if (c >= p.rot) continue;
            const bool low = p.interleaved ? !(c & 1) : c < half;
            const float y = buf[p.interleaved ? c ^ 1 : low ? c + half : c - half];
            const float2 turn_e = turns[e * kThreads + threadIdx.x];
            float& z = e & 1 ? x[e >> 1].y : x[e >> 1].x;
            z = z * turn_e.x + (low ? -y : y) * turn_e.y;
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
        const float* mean = p.k_mean + (there ? (h0 + i) * p.d : 0);
        float m[8];
        load4_param(mean, SAGE_FP32, p.vec_mean, a, p.d, m);
        load4_param(mean, SAGE_FP32, p.vec_mean, b, p.d, m + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] = make_float2(__fsub_rn(x[e].x, m[2 * e]), __fsub_rn(x[e].y, m[2 * e + 1]));
      }
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max_nan(max_nan(top, fabsf(x[e].x)), fabsf(x[e].y)), coded[KIND == kK && kCoded ? i : 0][e] = x[e];
      amax[i] = top;
    }
    if (!kCoded) continue;
    float scale, inv;  // reduce_rows' layout
    code_scale(reduce_rows<LPR, HC, true>(amax), KIND == kK ? 127.f : 448.f, &scale, &inv);
    const bool odd = __any_sync(0xffffffffu, inv == 0.f);  // a row of zeros, or with a NaN or an infinity: codes 0
#pragma unroll
    for (int i = 0; i < HC; ++i) {
      const float iv = of_row<LPR, HC>(inv, i);
      const float2 inv2 = make_float2(iv, iv);
      float2 vx[4];
      if (KIND == kV) unpack8<T>(cur[i], vx);
      const float2(&x)[4] = KIND == kV ? vx : coded[KIND == kK && kCoded ? i : 0];
      uint32_t w0 = KIND == kK ? code4_int8(x[0], x[1], inv2) : code4_e4m3(x[0], x[1], inv2);
      uint32_t w1 = KIND == kK ? code4_int8(x[2], x[3], inv2) : code4_e4m3(x[2], x[3], inv2);
      if (odd && iv == 0.f) w0 = w1 = 0;
      if (live && (HC == 1 || h0 + i < k.H)) {
        uint8_t* const code = codes + (unsigned long long)(unsigned)(h0 + i) * head_codes;
        [[maybe_unused]] const Extent& xc = KIND == kK ? p.x_k8 : p.x_v8;
        if (MODE == kHalves) {
          if (a < p.map.dc && SAGE_STORE_OK(xc, code + a, 4, &g_cache_error)) *reinterpret_cast<uint32_t*>(code + a) = w0;
          if (b < p.map.dc && SAGE_STORE_OK(xc, code + b, 4, &g_cache_error)) *reinterpret_cast<uint32_t*>(code + b) = w1;
        } else if (a < p.map.dc && SAGE_STORE_OK(xc, code + a, 8, &g_cache_error)) {
          *reinterpret_cast<uint2*>(code + a) = make_uint2(w0, w1);
        }
      }
    }
    const int my_row = row_of_lane<HC>(lane);
    float* sdst = scales + (unsigned long long)(unsigned)(h0 + my_row) * head_rows;
    if (lane < HC && live && h0 + my_row < k.H && SAGE_STORE_OK(KIND == kK ? p.x_ks : p.x_vs, sdst, 4, &g_cache_error))
      *sdst = scale;
  }
}

// `apart`: the kinds have CTAs of their own, which work at the same time (a decode step, a chunk of a prompt; norm and
// rotation alone, whose rows cost the same: video-DiT 138 -> 134 us).  Large cache writes: every CTA takes
// its share of each kind, one after the other, so that all end together whatever a kind's rows cost (four
// 8192-token prompts 160 us, apart 209).
template <typename T, int LPR, int HC, int MODE, bool APPEND>
__global__ void __launch_bounds__(kThreads, HC > 1 ? 6 : 8) head_rows_kernel(const __grid_constant__ HeadRowsParams p) {
  constexpr int kShared = MODE == kScalar || MODE == kAny ? kThreads * 8 : 2;
  __shared__ __align__(8) float partner_buf[kShared];
  __shared__ float2 turns[kShared];  // cosine and sine of each lane's channels
  begin_dependent();
  const unsigned cta = blockIdx.x, q = p.apart ? p.kind[kQ].ctas : 0, k = p.apart ? q + p.kind[kK].ctas : 0;
  if (!p.apart || cta < q) head_rows<T, LPR, HC, MODE, APPEND, kQ>(p, p.kind[kQ], cta, partner_buf, turns);
  if (!p.apart || (cta >= q && cta < k)) head_rows<T, LPR, heads_at_a_time(HC, APPEND, kK), MODE, APPEND, kK>(p, p.kind[kK], cta - q, partner_buf, turns);
  if (APPEND && (!p.apart || cta >= k))
    head_rows<T, LPR, HC, MODE == kScalar ? kScalar : kWide, APPEND, kV>(p, p.kind[kV], cta - k, partner_buf, turns);
}

// ------------------------------------------------------------------------------------------ read back
// The same rounds: a group of LPR lanes takes HC heads of one token, eight K and eight V codes of each to a
// lane (8-byte loads, 16-byte stores: both whole sectors), the next round's codes on their way meanwhile.
// Lanes 0 .. HC-1 hold the K scales of the HC heads, the next HC lanes the V scales.
template <typename T, int LPR, int HC, bool VEC>
__global__ void __launch_bounds__(kThreads, HC > 1 ? 5 : 8) gather_kernel(const __grid_constant__ GatherParams p) {
  constexpr unsigned kGroups = kThreads / LPR;
  begin_dependent();
  const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR, c = lane * 8;
  const unsigned rounds = p.rounds + (blockIdx.x < p.rounds_more ? 1 : 0);
  const unsigned round0 = blockIdx.x * p.rounds + min(blockIdx.x, p.rounds_more);
  unsigned chunk = round0 % p.chunks, t = round0 / p.chunks * kGroups + group;
  const int dc = p.map.dc, Hkv = p.map.Hkv;
  const unsigned head_rows = 1u << p.map.page_log2, head_codes = head_rows * dc;  // of a page
  int seq = 0, seq_first = 0, seq_end = -1, seq_base = 0;  // the sequence last looked up, and its position of token 0
  const uint8_t* kcodes = nullptr;  // of the token last looked up, head 0
  const uint8_t* vcodes = nullptr;
  const float* scales = nullptr;    // this lane's: of K or of V
  bool ok = false;
  const auto look_up = [&] {
    ok = false;
    if (t >= (unsigned)p.T) return;
    if ((int)t < seq_first || (int)t >= seq_end) {
      int count = 0;
      const bool found = find_sequence(p.cu, p.B, (int)t, p.T, &seq, &seq_first, &count);
      seq_end = found ? seq_first + count : -1;
      if (!found) return;
      seq_base = (p.starts ? p.starts[seq] : 0) - seq_first;
    }
    const int pos = seq_base + (int)t, page = page_of(p.map, seq, pos);
    if (page < 0) return;
    const long long row = p.map.row(page, 0, pos);
    kcodes = reinterpret_cast<const uint8_t*>(p.map.k8) + row * dc + c, vcodes = p.map.v8 + row * dc + c;
    scales = (lane < HC ? p.map.ks : p.map.vs) + row;
    ok = true;
  };
  look_up();
  uint2 kraw[HC], vraw[HC];
  float scale;
  const auto load_item = [&] {
    const int h0 = (int)chunk * HC;
#pragma unroll
    for (int i = 0; i < HC; ++i) {
      const bool in = ok && c < dc && (HC == 1 || h0 + i < Hkv);
      const unsigned long long at = (unsigned long long)(unsigned)(h0 + i) * head_codes;
      kraw[i] = in ? *reinterpret_cast<const uint2*>(kcodes + at) : make_uint2(0, 0);
      vraw[i] = in ? *reinterpret_cast<const uint2*>(vcodes + at) : make_uint2(0, 0);
    }
    const int h = h0 + lane % HC;
    scale = ok && lane < 2 * HC && h < Hkv ? scales[(unsigned long long)(unsigned)h * head_rows] : 0.f;
  };
  load_item();

#pragma unroll 1
  for (unsigned round = 0; round < rounds; ++round) {
    uint2 kc[HC], vc[HC];
#pragma unroll
    for (int i = 0; i < HC; ++i) kc[i] = kraw[i], vc[i] = vraw[i];
    const float sc = scale;
    const bool live = ok;
    const int h0 = (int)chunk * HC;
    const long long out = ((long long)t * Hkv + h0) * p.d;
    if (++chunk == p.chunks) chunk = 0, t += kGroups, look_up();
    load_item();
#pragma unroll
    for (int i = 0; i < HC; ++i) {
      const float ks = __shfl_sync(0xffffffffu, sc, i, LPR), vs = __shfl_sync(0xffffffffu, sc, HC + i, LPR);
      if (!live || (HC > 1 && h0 + i >= Hkv)) continue;
      float2 x[4], y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t kw = (e < 2 ? kc[i].x : kc[i].y) >> (16 * (e & 1)), vw = (e < 2 ? vc[i].x : vc[i].y) >> (16 * (e & 1));
        x[e] = mul2(make_float2((float)(int)(signed char)kw, (float)(int)(signed char)(kw >> 8)), make_float2(ks, ks));
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)vw, __NV_E4M3);
        y[e] = mul2(__half22float2(*reinterpret_cast<const __half2*>(&r)), make_float2(vs, vs));
      }
      if (p.k_mean) {
        const float* mean = p.k_mean + (h0 + i) * p.d;
        float m[8];
        load4_param(mean, SAGE_FP32, p.vec_mean, c, p.d, m);
        load4_param(mean, SAGE_FP32, p.vec_mean, c + 4, p.d, m + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = make_float2(__fadd_rn(x[e].x, m[2 * e]), __fadd_rn(x[e].y, m[2 * e + 1]));
      }
      const long long at = out + i * p.d;
      store8<T, VEC ? kWide : kScalar>(static_cast<unsigned short*>(p.k_out) + at, c, c + 4, p.d, x, p.x_k_out);
      store8<T, VEC ? kWide : kScalar>(static_cast<unsigned short*>(p.v_out) + at, c, c + 4, p.d, y, p.x_v_out);
    }
  }
}

template <typename T, int LPR, int HC, int MODE>
cudaError_t launch_rows(HeadRowsParams p, cudaStream_t st) {
  constexpr long long kGroups = kThreads / LPR;
  const unsigned most = 148 * (HC > 1 ? 6 : 8);  // one wave
  const auto rounds_of = [&](const HeadRows& k) { return (unsigned)((p.tokens + kGroups - 1) / kGroups * k.chunks); };
  const auto heads = [&](const HeadRows& k) { return heads_at_a_time(HC, p.append, (int)(&k - p.kind)); };
  unsigned all = 0;
  double cost = 0;
  // A round's time: coded keys 1.9 and values 1.1 times queries' per row.  Measured with Hq32 Hkv8 and norm, rotation and k_mean,
  // keys at 1.45, 1.9 and 2.6: 8 x 256 tokens d 128 15.6, 14.5, 14.2 us; 8 x 128 d 256 15.6, 14.6, 14.2; without k_mean
  // 8 x 512 d 64 13.9, 13.9, 14.7, 2 x 700 d 128 10.9, 10.4, 10.8.
  const double weight[3] = {1.0, p.append ? 1.9 * heads_at_a_time(HC, true, kK) / HC : 1.0, 1.1};
  for (HeadRows& k : p.kind) {
    k.chunks = (k.H + heads(k) - 1) / heads(k), all += rounds_of(k);
    cost += rounds_of(k) * weight[&k - p.kind];
  }
  p.apart = !p.append || all <= 8 * most;
  unsigned grid = 0;
  for (HeadRows& k : p.kind) {
    const unsigned rounds = rounds_of(k);
    k.ctas = all <= most ? rounds
             : p.apart   ? std::min(rounds, std::max(1u, (unsigned)(most * (rounds * weight[&k - p.kind] / cost))))
                         : most;
    grid = p.apart ? grid + k.ctas : most;
    if (!rounds) continue;
    k.rounds = rounds / k.ctas, k.rounds_more = rounds % k.ctas;
    // what the addresses move by: to the next chunk, and from the last one to the group's next token
    const auto moves = [&](const HeadView& v, long long* to_chunk, long long* to_token) {
      *to_chunk = v.head * heads(k), *to_token = kGroups * v.token - (k.chunks - 1) * *to_chunk;
    };
    moves(k.in, &k.in_chunk, &k.in_tokens);
    moves(k.out, &k.out_chunk, &k.out_tokens);
  }
  return p.append ? launch_dependent(head_rows_kernel<T, LPR, HC, MODE, true>, grid, kThreads, 0, st, p)
                  : launch_dependent(head_rows_kernel<T, LPR, HC, MODE, false>, grid, kThreads, 0, st, p);
}

template <typename T, int LPR>
cudaError_t launch_rows_lpr(const HeadRowsParams& p, cudaStream_t st) {
  if (!p.vec) return launch_rows<T, LPR, 1, kScalar>(p, st);
  if (p.cos_sin && p.rot % 8 != 0)
    return p.heads_per_group == 4 ? launch_rows<T, LPR, 4, kAny>(p, st) : launch_rows<T, LPR, 1, kAny>(p, st);
  if (p.cos_sin && !p.interleaved)
    return p.heads_per_group == 4 ? launch_rows<T, LPR, 4, kHalves>(p, st) : launch_rows<T, LPR, 1, kHalves>(p, st);
  return p.heads_per_group == 4 ? launch_rows<T, LPR, 4, kWide>(p, st) : launch_rows<T, LPR, 1, kWide>(p, st);
}

template <typename T>
cudaError_t launch_rows_t(const HeadRowsParams& p, cudaStream_t st) {
  return p.d <= 64 ? launch_rows_lpr<T, 8>(p, st) : p.d <= 128 ? launch_rows_lpr<T, 16>(p, st)
                                                               : launch_rows_lpr<T, 32>(p, st);
}

template <typename T, int LPR, int HC, bool VEC>
cudaError_t launch_gather(GatherParams p, cudaStream_t st) {
  constexpr long long kGroups = kThreads / LPR;
  p.chunks = (p.map.Hkv + HC - 1) / HC;
  const long long rounds = (p.T + kGroups - 1) / kGroups * p.chunks;
  const unsigned grid = (unsigned)std::min<long long>(rounds, 148 * (HC > 1 ? 5 : 8));  // one wave
  p.rounds = (unsigned)(rounds / grid), p.rounds_more = (unsigned)(rounds % grid);
  return launch_dependent(gather_kernel<T, LPR, HC, VEC>, grid, kThreads, 0, st, p);
}

template <typename T, int LPR>
cudaError_t launch_gather_lpr(const GatherParams& p, cudaStream_t st) {
  if (!p.vec) return launch_gather<T, LPR, 1, false>(p, st);
  return p.heads_per_group == 4 ? launch_gather<T, LPR, 4, true>(p, st) : launch_gather<T, LPR, 1, true>(p, st);
}

template <typename T>
cudaError_t launch_gather_t(const GatherParams& p, cudaStream_t st) {
  return p.d <= 64 ? launch_gather_lpr<T, 8>(p, st) : p.d <= 128 ? launch_gather_lpr<T, 16>(p, st)
                                                                 : launch_gather_lpr<T, 32>(p, st);
}

}  // namespace

cudaError_t launch_head_rows(const HeadRowsParams& p, int dtype, cudaStream_t st) {
  return dtype == SAGE_FP16 ? launch_rows_t<__half>(p, st) : launch_rows_t<__nv_bfloat16>(p, st);
}

cudaError_t launch_cache_gather(const GatherParams& p, int dtype, cudaStream_t st) {
  return dtype == SAGE_FP16 ? launch_gather_t<__half>(p, st) : launch_gather_t<__nv_bfloat16>(p, st);
}

}  // namespace sage
