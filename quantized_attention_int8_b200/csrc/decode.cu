// Attention of one new token per sequence over the paged cache (INT8 K, E4M3 V, one fp32 scale per
// token and kv head):
//
//   s_j = sm_scale * ks_j * sum_c q_c k8_jc      out_c = sum_j 2^(s_j log2 e) vs_j v8_jc / sum_j 2^(s_j log2 e)
//
// One pass over the cache with a running reference and sum per query head.  The codes are read once
// and are most of the bytes: 2 d + 8 per key and kv head against 4 d G operations (G query heads share
// a kv head), so HBM bounds it for every G that a tile holds.
//
// Keys are the M rows of both products, query heads the N columns (tiles of 8):
//   S^T = K Q^T       m16n8k16, A = 16 keys x 16 channels, codes widened exactly to the type of q
//   O^T = V^T P^T     m16n8k16, A = 16 channels x 16 keys, E4M3 widened exactly to fp16
// A handful of query rows cannot fill a 128-row tcgen05 tile, and the tensor work is a few percent of
// the time here; what counts is that no operand needs a detour through shared memory:
//   * the channels of a k16 step may be any 16, as long as K and Q agree, so a lane's 16 contiguous
//     bytes of a K row serve four steps;
//   * a lane's 16 contiguous channels of four V rows are paired by key with byte permutes, and give
//     eight A tiles;
//   * the scores' C layout becomes P^T's B layout by one 8x8 transpose (movmatrix) per 8 keys.
//
// V's scale is folded into the weights: w_j = s_j + log2(vs_j) has a running reference of its own, so
// the fp16 weights 2^(w_j - ref) keep their precision whatever the scales' spread; the sum uses s_j.
#include <cfloat>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "sage_internal.h"

namespace sage {

// Error word of the kernels in this file, read and cleared by sage_check_status().
__device__ int g_decode_error = 0;

cudaError_t read_clear_decode_error(int* value) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_decode_error, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_decode_error, &zero, sizeof(int));
}

namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kHeads = 8;       // query heads per tile (N of the products)
constexpr int kBadArg = 2;      // the error word's bit for SAGE_ERR_INVALID_ARG
constexpr float kLag = 8.f;     // the reference moves when a score passes it by 2^8: a weight stays below 2^8 in fp16

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8x8 transpose of 16-bit values spread over the warp (two per lane).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Two INT8 codes of a word (bytes 0, 1 or 2, 3) widened exactly.
// fp16: the byte as code + 128 in the low mantissa bits of 1024, less 1152.
// bf16 has 7 mantissa bits: the low seven bits in those of 128, less 128, or 256 where the sign bit is set.
template <typename T, int PAIR>
__device__ __forceinline__ uint32_t widen_int8(uint32_t word);
template <>
__device__ __forceinline__ uint32_t widen_int8<__half, 0>(uint32_t word) {
  const uint32_t h = __byte_perm(word ^ 0x80808080u, 0x64646464u, 0x4140);
  const uint32_t bias = 0x64806480u;
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&bias));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <>
__device__ __forceinline__ uint32_t widen_int8<__half, 1>(uint32_t word) {
  const uint32_t h = __byte_perm(word ^ 0x80808080u, 0x64646464u, 0x4342);
  const uint32_t bias = 0x64806480u;
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&bias));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t widen_bf16_bits(uint32_t h) {
  const uint32_t low = h & 0xFF7FFF7Fu, bias = h & 0xFF80FF80u;
  const __nv_bfloat162 r =
      __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&low), *reinterpret_cast<const __nv_bfloat162*>(&bias));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <>
__device__ __forceinline__ uint32_t widen_int8<__nv_bfloat16, 0>(uint32_t word) {
  return widen_bf16_bits(__byte_perm(word, 0x43434343u, 0x4140));
}
template <>
__device__ __forceinline__ uint32_t widen_int8<__nv_bfloat16, 1>(uint32_t word) {
  return widen_bf16_bits(__byte_perm(word, 0x43434343u, 0x4342));
}

__device__ __forceinline__ uint32_t widen_e4m3(uint32_t pair16) {
  const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)pair16, __NV_E4M3);
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ float max_over_keys(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Length of sequence b that the launch covers; a length out of range is flagged and taken as 0.
__device__ __forceinline__ int seq_len_of(const DecodeParams& p, int b, bool report) {
  const int len = p.seq_lens[b];
  if (len >= 0 && len <= p.max_len) return len;
  if (report) atomicOr(&g_decode_error, kBadArg);
  return 0;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) decode_kernel(DecodeParams p) {
  constexpr int KC = DP / 64;   // 16-byte pieces of a K row per lane
  constexpr int VB = DP / 8;    // bytes (= channels) of a V row per lane
  constexpr int VW = VB / 4;    // words of them
  constexpr bool kSplitP = sizeof(T) == 2 && std::is_same<T, __half>::value;
  __shared__ float sm_o[kWarps][kHeads][DP];
  __shared__ float sm_m[kWarps][kHeads], sm_l[kWarps][kHeads];

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x, b = blockIdx.z;
  const int hkv = blockIdx.y / p.tiles, head0 = (blockIdx.y % p.tiles) * kHeads;  // first head within the group
  const int nheads = min(kHeads, p.G - head0);
  const int len = seq_len_of(p, b, split == 0 && blockIdx.y == 0 && threadIdx.x == 0);
  const int k0 = split * p.chunk, k1 = min(len, k0 + p.chunk);
  if (k0 >= len && split > 0) return;

  // ---- Q: B operand of S^T.  Step (c, i) of the channels takes from lane t the channels
  // 64 c + 16 t + 4 i .. + 3 of head g.
  uint32_t qf[KC * 4][2];
  {
    const unsigned short* q = static_cast<const unsigned short*>(p.q.ptr) + (long long)b * p.q.batch +
                              (long long)(hkv * p.G + head0 + g) * p.q.head;
#pragma unroll
    for (int s = 0; s < KC * 4; ++s) {
      const int c = 64 * (s >> 2) + 16 * t + 4 * (s & 3);
      qf[s][0] = qf[s][1] = 0;
      if (g < nheads) {
        if (p.vec_q) {
          if (c < p.d) {
            const uint2 v = *reinterpret_cast<const uint2*>(q + c);
            qf[s][0] = v.x, qf[s][1] = v.y;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e < p.d) qf[s][e >> 1] |= (uint32_t)q[c + e] << (16 * (e & 1));
        }
      }
    }
  }

  float o[VW * 2][4];  // O^T: tile m = 2 w + hh holds channels VB g + 4 w + 2 hh, + 1 (rows g, g + 8) of heads 2t, 2t + 1
#pragma unroll
  for (int m = 0; m < VW * 2; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[m][e] = 0.f;
  float ms[2] = {-FLT_MAX, -FLT_MAX}, mw[2] = {-FLT_MAX, -FLT_MAX}, l[2] = {0.f, 0.f};

  for (int j = k0 + 16 * warp; j < k1; j += 16 * kWarps) {
    // 16 keys, all of one page (page sizes are multiples of 16)
    const int page = p.map.table[b * p.map.table_stride + (j >> p.map.page_log2)];
    if ((unsigned)page >= (unsigned)p.map.num_pages) {
      if (lane == 0) atomicOr(&g_decode_error, kBadArg);
      continue;  // its keys are left out
    }
    const long long row = p.map.row(page, hkv, j);
    const int n = min(16, k1 - j);  // rows behind the sequence are not read: they may hold anything
    uint4 kc[2][KC];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const int ch = 64 * c + 16 * t;
        kc[r][c] = make_uint4(0, 0, 0, 0);
        if (g + 8 * r < n && ch < p.map.dc)
          kc[r][c] = *reinterpret_cast<const uint4*>(p.map.k8 + (row + g + 8 * r) * p.map.dc + ch);
      }
    uint32_t vc[4][VW];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int key = 2 * t + (r & 1) + 8 * (r >> 1);
      const bool in = key < n && VB * g < p.map.dc;
      const uint8_t* src = p.map.v8 + (row + key) * p.map.dc + VB * g;
      if (VB == 8) {
        const uint2 v = in ? *reinterpret_cast<const uint2*>(src) : make_uint2(0, 0);
        vc[r][0] = v.x, vc[r][1] = v.y;
      } else {
#pragma unroll
        for (int q = 0; q < VB / 16; ++q) {
          const uint4 v = in && VB * g + 16 * q < p.map.dc ? *reinterpret_cast<const uint4*>(src + 16 * q)
                                                           : make_uint4(0, 0, 0, 0);
          vc[r][4 * q] = v.x, vc[r][4 * q + 1] = v.y, vc[r][4 * q + 2] = v.z, vc[r][4 * q + 3] = v.w;
        }
      }
    }
    float kf[2], lv[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool in = g + 8 * r < n;
      kf[r] = in ? p.map.ks[row + g + 8 * r] * p.scale_log2 : 0.f;
      lv[r] = in ? lg2(p.map.vs[row + g + 8 * r]) : 0.f;
    }

    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w0 = (&kc[0][c].x)[i], w1 = (&kc[1][c].x)[i];
        mma16816<T>(s, widen_int8<T, 0>(w0), widen_int8<T, 0>(w1), widen_int8<T, 1>(w0), widen_int8<T, 1>(w1),
                    qf[4 * c + i][0], qf[4 * c + i][1]);
      }
    float w[4];  // s, w: keys g (0, 1) and g + 8 (2, 3) of heads 2t and 2t + 1
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = e >> 1;
      const bool in = g + 8 * r < n;
      s[e] = in ? s[e] * kf[r] : -INFINITY;
      w[e] = in ? s[e] + lv[r] : -INFINITY;
    }
    bool move = false;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      move |= fmaxf(s[h], s[2 + h]) > ms[h] + kLag || fmaxf(w[h], w[2 + h]) > mw[h] + kLag;
    if (__any_sync(0xffffffffu, move)) {
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float nms = fmaxf(ms[h], max_over_keys(fmaxf(s[h], s[2 + h])));
        const float nmw = fmaxf(mw[h], max_over_keys(fmaxf(w[h], w[2 + h])));
        l[h] *= ex2(ms[h] - nms);
        f[h] = ex2(mw[h] - nmw);
        ms[h] = nms, mw[h] = nmw;
      }
#pragma unroll
      for (int m = 0; m < VW * 2; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[m][e] *= f[e & 1];
    }
    float pw[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      l[e & 1] += ex2(s[e] - ms[e & 1]);
      pw[e] = ex2(w[e] - mw[e & 1]);
    }
    // P^T as B operand: fp16.  For fp16 outputs a second fp16 term carries what the first rounds off
    // (2^-12 of a weight would be as large as the output's own rounding).
    uint32_t ph[2], pl[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const __half2 hi = __floats2half2_rn(pw[2 * r], pw[2 * r + 1]);
      ph[r] = transpose8x8(*reinterpret_cast<const uint32_t*>(&hi));
      if (kSplitP) {
        const float2 back = __half22float2(hi);
        const __half2 lo = __floats2half2_rn(pw[2 * r] - back.x, pw[2 * r + 1] - back.y);
        pl[r] = transpose8x8(*reinterpret_cast<const uint32_t*>(&lo));
      }
    }
#pragma unroll
    for (int wd = 0; wd < VW; ++wd)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const uint32_t sel = hh ? 0x7362 : 0x5140;
        const uint32_t x0 = __byte_perm(vc[0][wd], vc[1][wd], sel), x1 = __byte_perm(vc[2][wd], vc[3][wd], sel);
        const uint32_t a0 = widen_e4m3(x0 & 0xFFFFu), a1 = widen_e4m3(x0 >> 16), a2 = widen_e4m3(x1 & 0xFFFFu),
                       a3 = widen_e4m3(x1 >> 16);
        mma16816<__half>(o[2 * wd + hh], a0, a1, a2, a3, ph[0], ph[1]);
        if (kSplitP) mma16816<__half>(o[2 * wd + hh], a0, a1, a2, a3, pl[0], pl[1]);
      }
  }

  // ---- join the warps: O moves to the reference of the scores, then to the largest one
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], x);
    if (g == 0) sm_m[warp][2 * t + h] = ms[h], sm_l[warp][2 * t + h] = l[h];
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int head = 2 * t + h;
    float top = sm_m[0][head];
#pragma unroll
    for (int x = 1; x < kWarps; ++x) top = fmaxf(top, sm_m[x][head]);
    const float f = ex2(mw[h] - top);
#pragma unroll
    for (int m = 0; m < VW * 2; ++m) {
      const int c = VB * g + 2 * m;
      sm_o[warp][head][c] = o[m][h] * f;
      sm_o[warp][head][c + 1] = o[m][2 + h] * f;
    }
  }
  __syncthreads();
  const bool whole = len <= p.chunk;  // this CTA saw the whole sequence
  for (int i = threadIdx.x; i < nheads * DP; i += kThreads) {
    const int head = i / DP, c = i % DP;
    if (c >= p.d) continue;
    float top = sm_m[0][head], sum = 0.f, acc = 0.f;
#pragma unroll
    for (int x = 1; x < kWarps; ++x) top = fmaxf(top, sm_m[x][head]);
#pragma unroll
    for (int x = 0; x < kWarps; ++x) sum += sm_l[x][head] * ex2(sm_m[x][head] - top), acc += sm_o[x][head][c];
    const long long hq = (long long)b * p.Hq + hkv * p.G + head0 + head;
    if (whole) {
      T* dst = static_cast<T*>(p.out) + hq * p.d + c;
      if (SAGE_STORE_OK(p.x_out, dst, 2, &g_decode_error)) *dst = from_f32<T>(sum == 0.f ? 0.f : acc / sum);
    } else {
      const long long part = hq * p.nsplit + split;
      float* dst = p.part_o + part * p.d + c;
      if (SAGE_STORE_OK(p.x_part_o, dst, 4, &g_decode_error)) *dst = acc;
      if (c == 0) {
        float* ml = p.part_ml + part * 2;
        if (SAGE_STORE_OK(p.x_part_ml, ml, 8, &g_decode_error)) ml[0] = top, ml[1] = sum;
      }
    }
  }
}

// Joins the chunks of a sequence: out = sum_i O_i 2^(m_i - M) / sum_i l_i 2^(m_i - M).
template <typename T>
__global__ void __launch_bounds__(kThreads) decode_join_kernel(DecodeParams p) {
  const long long hq = blockIdx.x;
  const int len = seq_len_of(p, (int)(hq / p.Hq), false);
  const int n = (len + p.chunk - 1) / p.chunk;
  if (n <= 1) return;  // written by the only chunk
  const float* ml = p.part_ml + hq * p.nsplit * 2;
  const float* po = p.part_o + hq * p.nsplit * p.d;
  float top = ml[0];
  for (int i = 1; i < n; ++i) top = fmaxf(top, ml[2 * i]);
  float sum = 0.f;
  for (int i = 0; i < n; ++i) sum += ml[2 * i + 1] * ex2(ml[2 * i] - top);
  for (int c = threadIdx.x; c < p.d; c += kThreads) {
    float acc = 0.f;
    for (int i = 0; i < n; ++i) acc += po[(long long)i * p.d + c] * ex2(ml[2 * i] - top);
    T* dst = static_cast<T*>(p.out) + hq * p.d + c;
    if (SAGE_STORE_OK(p.x_out, dst, 2, &g_decode_error)) *dst = from_f32<T>(sum == 0.f ? 0.f : acc / sum);
  }
}

template <typename T>
cudaError_t launch_decode_t(const DecodeParams& p, cudaStream_t st) {
  const dim3 grid(p.nsplit, (p.Hq / p.G) * p.tiles, p.B);
  if (p.d <= 64)
    decode_kernel<T, 64><<<grid, kThreads, 0, st>>>(p);
  else if (p.d <= 128)
    decode_kernel<T, 128><<<grid, kThreads, 0, st>>>(p);
  else
    decode_kernel<T, 256><<<grid, kThreads, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.nsplit == 1) return e;
  decode_join_kernel<T><<<p.B * p.Hq, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode(const DecodeParams& p, int dtype, cudaStream_t st) {
  return dtype == SAGE_FP16 ? launch_decode_t<__half>(p, st) : launch_decode_t<__nv_bfloat16>(p, st);
}

}  // namespace sage
