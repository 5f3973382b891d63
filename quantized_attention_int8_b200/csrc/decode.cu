// Attention of one new token per sequence over the paged cache (INT8 K, E4M3 V, one fp32 scale per
// token and kv head):
//
//   s_j = sm_scale * ks_j * sum_c q_c k8_jc      out_c = sum_j 2^(s_j log2 e) vs_j v8_jc / sum_j 2^(s_j log2 e)
//
// One pass over the cache with a running reference and sum per query head.  The codes are read once
// and are most of the bytes: 2 d + 8 per key and kv head against 4 d G operations (G query heads share
// a kv head), so HBM bounds it for every G that a tile holds where the heads fill their instance (64, 128 or 256 channels):
// B32 L16384 Hq32 Hkv8 d128 bf16 (1107 MB) takes 182 us, 6.1 TB/s (fp16, with a second P term, 196 us); of that about 10 us
// are the beginning and the end.  At 64 channels the work per key is the same for half the bytes (4.3 TB/s of 0.57 GB),
// padded heads do the products of the channels that they do not have (80 and 160: 3.9 and 3.8 TB/s), and
// codes are widened once per tile (16 heads to a kv head 3.1 TB/s, 32 1.6).
//
// Keys are the M rows of both products, query heads the N columns (tiles of 8):
//   S^T = K Q^T       m16n8k16, A = 16 keys x 16 channels, codes widened exactly to fp16
//   O^T = V^T P^T     m16n8k16, A = 16 channels x 16 keys, E4M3 widened exactly to fp16
// A handful of query rows cannot fill a 128-row tcgen05 tile, and the tensor work is a sixth of the
// time here.  What counts is that the codes arrive at the rate of HBM, and get from shared memory
// into the products with few instructions:
//   * bulk copies, one elected lane to a run of rows: 2 KB of K, 512 bytes of V.  16-byte copies by the
//     lanes that use them (no bank conflicts, no barrier) reached 4.2 TB/s on B32 L16384 Hq32 Hkv8 d128, with
//     the arithmetic left out; bulk copies 6.3 TB/s;
//   * the channels of a k16 step may be any 16, as long as K and Q agree, so a lane's 16 contiguous
//     bytes of a K row serve four steps;
//   * a lane's 16 contiguous channels of four V rows are paired by key with byte permutes, and give
//     eight A tiles.  Row i of S is key 4 (i / 2) + i % 2 for i < 8 and two keys on for i + 8, so that lane t's
//     keys are the four rows 4 t ..; those groups of four are 32 bytes apart from one another's
//     banks, and the reads have no conflicts (K's have two-way ones);
//   * the scores' C layout becomes P^T's B layout by one 8x8 transpose (movmatrix) per 8 keys.
//
// V's scale is folded into the weights: w_j = s_j + log2(vs_j) has a running reference of its own, so
// that the spread of the scales takes nothing from the fp16 weights 2^(w_j - ref); the sum uses s_j, in fp32.
// What the 16 bits of the weights cost: see kLift, and the second term of fp16 outputs.
#include <atomic>
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
  if (e != cudaSuccess || *value == 0) return e;  // nothing to clear: one copy less
  const int zero = 0;
  return cudaMemcpyToSymbol(g_decode_error, &zero, sizeof(int));
}

namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kHeads = kDecodeHeads;  // query heads per tile (N of the products)
constexpr int kTimeout = 1, kBadArg = 2;  // the error word's bits for SAGE_ERR_TIMEOUT and SAGE_ERR_INVALID_ARG
// The references of the running softmax (log2 units): the sum's moves when a score passes it by kLag.  The weights
// of P V are fp16 and stand kLift above theirs (the largest seen when it moved), so that they stay below 2^15 and
// are lost (below 2^-25) only kLift + 25 powers of two under it: n such keys of a warp, whatever they hold together,
// are off by n 2^-36 of the warp's largest weight.  At 8 and 0, keys 25 powers of two below a
// dominant one vanished from O and counted in the sum.
constexpr float kLag = 4.f, kLift = 11.f;

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

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8x8 transpose of 16-bit values spread over the warp (two per lane).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Two INT8 codes of a word whose sign bits were flipped (bytes picked by `sel`), widened exactly to fp16:
// each byte, now code + 128, goes to the low mantissa bits of 1024; less 1152.
__device__ __forceinline__ uint32_t widen_int8(uint32_t flipped, uint32_t sel) {
  const uint32_t h = __byte_perm(flipped, 0x64646464u, sel), bias = 0x64806480u;
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&bias));
  return *reinterpret_cast<const uint32_t*>(&r);
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

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// Copy of `bytes` (a multiple of 16, both addresses 16-byte aligned), counted on an mbarrier.
__device__ __forceinline__ void copy_bulk(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void barrier_init(uint32_t bar) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void barrier_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Waits for the phase with this parity; gives up after about a second (never seen: the copies are
// this warp's own) and reports it.
__device__ __forceinline__ bool barrier_wait(uint32_t bar, uint32_t parity) {
  long long t0 = 0;
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(1000000)
        : "memory");
    if (ok) return true;
    if (t0 == 0) t0 = clock64();
    if (clock64() - t0 > 2000000000LL) {
      atomicOr(&g_decode_error, kTimeout);
      return false;
    }
  }
}

// One warp's ring of stages in shared memory, kTiles 16-key tiles to a stage.  A tile: 16 K rows; four groups of
// four V rows, kPad bytes apart; 16 K scales and 16 V scales.  Two or four tiles are worked on at a time where
// they fit: the chain from a score to its weight is latency, and three warps to a scheduler hide little of
// it (B32 L16384 Hq32 Hkv8: d 128 one tile 223 us, two 187; d 64 two 148 us, four 136).
template <int DP>
struct Ring {
  static constexpr int kTiles = DP == 256 ? 1 : DP == 128 ? 2 : 4;
  static constexpr int kStages = DP == 256 ? 3 : 2;
  static constexpr int kPad = 32;
  static __host__ __device__ constexpr int v_at(int dc) { return 16 * dc; }
  static __host__ __device__ constexpr int v_group(int dc) { return 4 * dc + kPad; }
  static __host__ __device__ constexpr int scales_at(int dc) { return 32 * dc + 4 * kPad; }
  static __host__ __device__ constexpr int tile_bytes(int dc) { return 32 * dc + 4 * kPad + 128; }
  static __host__ __device__ constexpr int warp_bytes(int dc) { return kStages * kTiles * tile_bytes(dc); }
  // The lanes of channels behind dc read past their rows (what they read is not used): DP bytes behind the
  // last tile.  The warps' O takes the rings' place at the end.
  static __host__ __device__ constexpr int cta_bytes(int dc) {
    return kWarps * warp_bytes(dc) + DP > kWarps * kHeads * DP * 4 ? kWarps * warp_bytes(dc) + DP
                                                                   : kWarps * kHeads * DP * 4;
  }
};

__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

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

// The work, cut into units: 2^unit_log2 keys (the launch says how many) of one (sequence, kv head, tile of heads),
// sequence by sequence, its pairs of kv head and head tile one after the other.  Every CTA takes the same
// number of units, whatever the sequences' lengths, so that a ragged batch ends everywhere at once; a
// pair that crosses CTAs is joined.  Each pair begins with `unit_extra` units without keys, for the time that a CTA
// needs to begin with it (Q, a full ring) and to write its answer: with keys alone, the CTAs of a ragged
// batch that got the shortest sequences were its last.
__device__ __forceinline__ uint32_t key_units(const DecodeParams& p, int len) {
  return len > 0 ? ((uint32_t)(len - 1) >> p.unit_log2) + 1 : 1;  // an empty sequence: one, to write its zeros
}
__device__ __forceinline__ uint32_t units_of(const DecodeParams& p, int len) { return key_units(p, len) + p.unit_extra; }

struct Place {
  uint32_t share;     // units per CTA
  uint32_t total;     // units in all
  uint32_t pair0;     // first unit of the pair at the searched unit
  int b, pair, len;   // sequence (-1: behind the last unit), pair within it, its length
};

// Finds the pair that holds unit cta * share.  All NT threads of the CTA call it.
template <int NT>
__device__ __forceinline__ Place find_place(const DecodeParams& p, uint32_t cta, bool report) {
  __shared__ uint32_t sm_sum[NT / 32];
  __shared__ Place sm_place;
  if (!p.part_o) {  // one unit to every pair: no sum over the lengths (1 us of a short call)
    Place at;
    at.total = p.B * p.pairs, at.share = (at.total + p.ctas - 1) / p.ctas, at.pair0 = cta * at.share;
    at.b = at.pair0 < at.total ? (int)(at.pair0 / p.pairs) : -1, at.pair = (int)(at.pair0 % p.pairs);
    at.len = at.b >= 0 ? seq_len_of(p, at.b, threadIdx.x == 0) : 0;
    return at;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (p.B + NT - 1) / NT, b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
  uint32_t mine = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) mine += units_of(p, seq_len_of(p, b, report));
  uint32_t before = mine;  // inclusive scan over the warp, then over the warps
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, before, x);
    if (lane >= x) before += v;
  }
  if (lane == 31) sm_sum[warp] = before;
  if (threadIdx.x == 0) sm_place.b = -1;
  __syncthreads();
  uint32_t total = 0;
#pragma unroll
  for (int x = 0; x < NT / 32; ++x) {
    if (x < warp) before += sm_sum[x];
    total += sm_sum[x];
  }
  before -= mine;
  const uint32_t all = total * p.pairs, share = (all + p.ctas - 1) / p.ctas, u = cta * share;
  if (u < all && before * p.pairs <= u && u < (before + mine) * p.pairs) {  // one thread
    int b = b0, len;
    uint32_t n;
#pragma unroll 1
    for (;; ++b, before += n) {
      len = seq_len_of(p, b, false);
      n = units_of(p, len);
      if (b + 1 == b1 || u < (before + n) * p.pairs) break;
    }
    const uint32_t pair = (u - before * p.pairs) / n;
    sm_place.b = b, sm_place.pair = (int)pair, sm_place.len = len, sm_place.pair0 = before * p.pairs + pair * n;
  }
  __syncthreads();
  Place at = sm_place;
  at.share = share, at.total = all;
  return at;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, DP == 256 ? 2 : 3) decode_kernel(DecodeParams p) {
  using R = Ring<DP>;
  constexpr int KC = DP / 64;             // 16-byte pieces of a K row per lane
  constexpr int VP = DP < 128 ? 8 : 16;   // bytes (= channels) of a V row that a lane reads at a time
  constexpr int VC = DP / 8 / VP;         // and how often, 8 VP channels apart
  constexpr int VW = VP / 4;              // words of them
  constexpr bool kSplitP = std::is_same<T, __half>::value;
  constexpr int QP = DP + 8;              // pitch of Q in shared memory
  extern __shared__ __align__(128) unsigned char smem[];  // the warps' rings; later their O, [kWarps][kHeads][DP] floats
  __shared__ float sm_m[kWarps][kHeads], sm_l[kWarps][kHeads], sm_hf[kHeads];
  __shared__ __align__(16) __half sm_q[kHeads * QP];
  __shared__ __align__(8) uint64_t sm_bar[kWarps][R::kStages];
  __shared__ int sm_dead;

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int dc = p.map.dc, tile_bytes = R::tile_bytes(dc);
  unsigned char* const ring = smem + warp * R::warp_bytes(dc);
  const uint32_t bars = smem_addr(sm_bar[warp]);
  if (threadIdx.x == 0) sm_dead = 0;
  if (lane < R::kStages) barrier_init(bars + 8 * lane);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  // The grid before may have written the cache, Q or the lengths.  Only then is the join let in, which reads the
  // lengths before it waits for this grid; it takes the SMs that this grid frees.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Place at = find_place<kThreads>(p, blockIdx.x, blockIdx.x == 0);
  if (at.b < 0) return;
  uint32_t unit = blockIdx.x * at.share, pair0 = at.pair0, parity = 0;  // parity: bit per stage
  const uint32_t unit_end = min(at.total, unit + at.share);
  int b = at.b, pair = at.pair, len = at.len;

  while (true) {  // one segment: this CTA's keys of one pair
    const uint32_t n_pair = units_of(p, len), rel = unit - pair0, n_seg = min(n_pair - rel, unit_end - unit);
    // its key units u0 .. u1 - 1 (none where only the pair's first, empty units are this CTA's)
    const uint32_t u0 = max(rel, p.unit_extra) - p.unit_extra, u1 = max(rel + n_seg, p.unit_extra) - p.unit_extra;
    if (u0 < u1) {
      const int hkv = pair / p.tiles, head0 = (pair % p.tiles) * kHeads;  // first head within the group
      const int nheads = min(kHeads, p.G - head0);
      const int k0 = (int)(u0 << p.unit_log2);
      const int k1 = rel + n_seg == n_pair ? len : (int)(u1 << p.unit_log2);

      // Q is asked for before the ring is filled, not behind its copies (B64, 1 to 1000 keys: 32.2 -> 30.2 us).
      T qx[kHeads / kWarps][DP / 32];
#pragma unroll
      for (int i = 0; i < kHeads / kWarps; ++i) {
        const int head = warp + i * kWarps;
        const T* q = static_cast<const T*>(p.q.ptr) + (long long)b * p.q.batch +
                     (long long)(hkv * p.G + head0 + head) * p.q.head;
#pragma unroll
        for (int e = 0; e < DP / 32; ++e)
          qx[i][e] = head < nheads && lane + 32 * e < p.d ? q[lane + 32 * e] : from_f32<T>(0.f);
      }

      // ---- this warp's run of 16-key tiles, each of one page (page sizes are multiples of 16)
      const int ntiles = (k1 - k0 + 15) >> 4, per_warp = (ntiles + kWarps - 1) / kWarps;
      const int tile0 = min(warp * per_warp, ntiles), n_mine = min(per_warp, ntiles - tile0);
      const int j0 = k0 + 16 * tile0, j1 = min(k1, j0 + 16 * n_mine);
      const int steps = (n_mine + R::kTiles - 1) / R::kTiles;
      // Lanes 8 x .. 8 x + 6 copy tile x of a step: its K rows, four groups of V rows, the scales of each.
      const int32_t* table = p.map.table + b * p.map.table_stride;
      const int my_tile = lane >> 3, my_part = lane & 7;
      const auto my_page = [&](int step) {
        const int i = step * R::kTiles + my_tile;
        return my_tile < R::kTiles && i < n_mine ? table[(j0 + 16 * i) >> p.map.page_log2] : -1;
      };
      int stage_in = 0, page = my_page(0);
      uint32_t there = 0;  // bit x: the tile fetched x tiles ago was copied (exists, and not on a bad page)
      const auto fetch_step = [&](int step) {
        if (step < steps) {
          const int i = step * R::kTiles + my_tile, j = j0 + 16 * i;
          const bool mine = my_tile < R::kTiles && i < n_mine, good = (unsigned)page < (unsigned)p.map.num_pages;
          if (mine && !good && my_part == 0) atomicOr(&g_decode_error, kBadArg);
          const uint32_t copied = __ballot_sync(0xffffffffu, mine && good && my_part == 0);
          const uint32_t bar = bars + 8 * stage_in;
          if (lane == 0) barrier_expect(bar, __popc(copied) * (32 * dc + 128));
          __syncwarp();
          if (mine && good && my_part < 7) {
            const long long row = p.map.row(page, hkv, j);
            uint32_t dst = smem_addr(ring) + (stage_in * R::kTiles + my_tile) * tile_bytes, bytes = 16 * dc;
            const void* src = p.map.k8 + row * dc;
            if (my_part > 4) {
              bytes = 64, src = (my_part == 5 ? p.map.ks : p.map.vs) + row, dst += R::scales_at(dc) + (my_part - 5) * 64;
            } else if (my_part > 0) {
              bytes = 4 * dc, src = p.map.v8 + (row + 4 * (my_part - 1)) * dc;
              dst += R::v_at(dc) + (my_part - 1) * R::v_group(dc);
            }
            copy_bulk(dst, src, bytes, bar);
          }
#pragma unroll
          for (int x = 0; x < R::kTiles; ++x) there = there << 1 | (copied >> (8 * x) & 1);
        } else {
          there <<= R::kTiles;
        }
        stage_in = stage_in + 1 == R::kStages ? 0 : stage_in + 1;
        page = my_page(step + 1);
      };
#pragma unroll 1
      for (int i = 0; i < R::kStages - 1; ++i) fetch_step(i);

      // ---- Q: B operand of S^T.  Step (c, i) of the channels takes from lane t the channels
      // 64 c + 16 t + 4 i .. + 3 of head g.  As fp16 whatever its type: a bf16 head is scaled by the power of two that
      // takes its largest value to 2^14 .. 2^15, which is exact down to 2^-29 of that value and rounds to
      // 2^-40 of it below (fp32 sums are off by more).
#pragma unroll
      for (int i = 0; i < kHeads / kWarps; ++i) {
        const int head = warp + i * kWarps;
        float x[DP / 32];
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < DP / 32; ++e)
          x[e] = to_f32(qx[i][e]), top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
        float up = 1.f, hf = p.scale_log2;
        if (!kSplitP) {
          top = __reduce_max_sync(0xffffffffu, top);
          const int e = min(max(127 + 14 - (int)(top >> 23), -126), 126);
          up = __uint_as_float((uint32_t)(127 + e) << 23), hf *= __uint_as_float((uint32_t)(127 - e) << 23);
        }
#pragma unroll
        for (int e = 0; e < DP / 32; ++e) sm_q[head * QP + lane + 32 * e] = __float2half_rn(x[e] * up);
        if (lane == 0) sm_hf[head] = hf;
      }
      __syncthreads();
      uint2 qf[KC * 4];
#pragma unroll
      for (int s = 0; s < KC * 4; ++s)
        qf[s] = *reinterpret_cast<const uint2*>(sm_q + g * QP + 64 * (s >> 2) + 16 * t + 4 * (s & 3));
      const float hf[2] = {sm_hf[2 * t], sm_hf[2 * t + 1]};  // score factor of heads 2t and 2t + 1

      float o[VC * VW * 2][4];  // O^T: tile (q VW + w) 2 + hh holds channels 8 VP q + VP g + 4 w + 2 hh, + 1 (rows g, g + 8) of heads 2t, 2t + 1
#pragma unroll
      for (int m = 0; m < VC * VW * 2; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[m][e] = 0.f;
      float ms[2] = {-FLT_MAX, -FLT_MAX}, mw[2] = {-FLT_MAX, -FLT_MAX}, l[2] = {0.f, 0.f};  // (mw: less kLift)

      const int krow = (4 * (g >> 1) + (g & 1));  // key of S's row g; two more for row g + 8
      const unsigned char* const k_lane = ring + krow * dc + 16 * t;
      const unsigned char* const v_lane = ring + R::v_at(dc) + t * R::v_group(dc) + VP * g;
      int stage = 0;
#pragma unroll 1
      for (int it = 0; it < steps; ++it) {
        const bool arrived = barrier_wait(bars + 8 * stage, parity >> stage & 1);
        parity ^= 1u << stage;
        if (!__all_sync(0xffffffffu, arrived)) {  // gave up: wind down, with the copies in flight given their time
          for (int x = 1; x < R::kStages - 1 && it + x < steps; ++x) barrier_wait(bars + 8 * ((stage + x) % R::kStages),
                                                                             parity >> (stage + x) % R::kStages & 1);
          sm_dead = 1;
          break;
        }
        // (past the vote: all lanes are done with the stage filled next)
        fetch_step(it + R::kStages - 1);
        const int at_stage = stage * R::kTiles * tile_bytes;
        stage = stage + 1 == R::kStages ? 0 : stage + 1;

        // Keys of each tile that count.  V rows behind them (whatever their page holds, or held before) become
        // zeros: a weight of 0 times a NaN code would be a NaN.
        int n[R::kTiles];
#pragma unroll
        for (int x = 0; x < R::kTiles; ++x) {
          n[x] = there >> (R::kStages * R::kTiles - 1 - x) & 1 ? min(16, j1 - (j0 + 16 * (it * R::kTiles + x))) : 0;
          if (n[x] < 16) {
            unsigned char* v = ring + at_stage + x * tile_bytes + R::v_at(dc);
#pragma unroll 1
            for (int r = n[x] + (lane >> 3); r < 16; r += 4)
#pragma unroll 1
              for (int c = 16 * (lane & 7); c < dc; c += 128)
                *reinterpret_cast<uint4*>(v + (r >> 2) * R::v_group(dc) + (r & 3) * dc + c) = make_uint4(0, 0, 0, 0);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before a later copy into the stage
            __syncwarp();
          }
        }

        float s[R::kTiles][4], w[R::kTiles][4];  // rows g (0, 1) and g + 8 (2, 3) of heads 2t and 2t + 1
#pragma unroll
        for (int x = 0; x < R::kTiles; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[x][e] = 0.f;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          uint4 rows[R::kTiles][2];
#pragma unroll
          for (int x = 0; x < R::kTiles; ++x)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              rows[x][r] = *reinterpret_cast<const uint4*>(k_lane + at_stage + x * tile_bytes + 2 * r * dc + 64 * c);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int x = 0; x < R::kTiles; ++x) {
              const uint32_t w0 = (&rows[x][0].x)[i] ^ 0x80808080u, w1 = (&rows[x][1].x)[i] ^ 0x80808080u;
              mma16816(s[x], widen_int8(w0, 0x4140), widen_int8(w1, 0x4140), widen_int8(w0, 0x4342),
                       widen_int8(w1, 0x4342), qf[4 * c + i].x, qf[4 * c + i].y);
            }
        }
        bool move = false;
#pragma unroll
        for (int x = 0; x < R::kTiles; ++x) {
          const float* scales = reinterpret_cast<const float*>(ring + at_stage + x * tile_bytes + R::scales_at(dc));
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int key = krow + 2 * r;
            const float kf = scales[key], lv = lg2(scales[16 + key]);
            const bool in = key < n[x];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int e = 2 * r + h;
              s[x][e] = in ? s[x][e] * hf[h] * kf : -INFINITY;
              w[x][e] = in ? s[x][e] + lv : -INFINITY;
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
            move |= fmaxf(s[x][h], s[x][2 + h]) > ms[h] + kLag || fmaxf(w[x][h], w[x][2 + h]) > mw[h] + (kLag + kLift);
        }
        if (__any_sync(0xffffffffu, move)) {
          float f[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float ts = fmaxf(s[0][h], s[0][2 + h]), tw = fmaxf(w[0][h], w[0][2 + h]);
#pragma unroll
            for (int x = 1; x < R::kTiles; ++x)
              ts = fmaxf(ts, fmaxf(s[x][h], s[x][2 + h])), tw = fmaxf(tw, fmaxf(w[x][h], w[x][2 + h]));
            const float nms = fmaxf(ms[h], max_over_keys(ts)), nmw = fmaxf(mw[h], max_over_keys(tw) - kLift);
            l[h] *= ex2(ms[h] - nms);
            f[h] = ex2(mw[h] - nmw);
            ms[h] = nms, mw[h] = nmw;
          }
#pragma unroll
          for (int m = 0; m < VC * VW * 2; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[m][e] *= f[e & 1];
        }
        // P^T as B operand: fp16, a weight off by up to 2^-11 of itself.  For bf16 outputs that is enough: an eighth of
        // their own rounding (2^-8) if all weights were off the same way.  For fp16 outputs it would be as large as
        // theirs, and a second fp16 term carries what the first rounds off (2^-22 is left).
        uint32_t ph[R::kTiles][2], pl[R::kTiles][2];
#pragma unroll
        for (int x = 0; x < R::kTiles; ++x) {
          float pw[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            l[e & 1] += ex2(s[x][e] - ms[e & 1]);
            pw[e] = ex2(w[x][e] - mw[e & 1]);
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const __half2 hi = __floats2half2_rn(pw[2 * r], pw[2 * r + 1]);
            ph[x][r] = transpose8x8(*reinterpret_cast<const uint32_t*>(&hi));
            if (kSplitP) {
              const float2 back = __half22float2(hi);
              const __half2 lo = __floats2half2_rn(pw[2 * r] - back.x, pw[2 * r + 1] - back.y);
              pl[x][r] = transpose8x8(*reinterpret_cast<const uint32_t*>(&lo));
            }
          }
        }
#pragma unroll
        for (int x = 0; x < R::kTiles; ++x)
#pragma unroll
          for (int q = 0; q < VC; ++q) {
            uint32_t vc[4][VW];  // keys 4 t .. 4 t + 3
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const unsigned char* src = v_lane + at_stage + x * tile_bytes + r * dc + 8 * VP * q;
              if (VP == 8) {
                const uint2 v = *reinterpret_cast<const uint2*>(src);
                vc[r][0] = v.x, vc[r][1] = v.y;
              } else {
                const uint4 v = *reinterpret_cast<const uint4*>(src);
                vc[r][0] = v.x, vc[r][1] = v.y, vc[r][VW - 2] = v.z, vc[r][VW - 1] = v.w;
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
                float(&om)[4] = o[(q * VW + wd) * 2 + hh];
                mma16816(om, a0, a1, a2, a3, ph[x][0], ph[x][1]);
                if (kSplitP) mma16816(om, a0, a1, a2, a3, pl[x][0], pl[x][1]);
              }
          }
      }

      // ---- join the warps: O moves to the reference of the scores, then to the largest one
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], x);
        if (g == 0) sm_m[warp][2 * t + h] = ms[h], sm_l[warp][2 * t + h] = l[h];
      }
      __syncthreads();  // and every warp is done with its ring
      float* const sm_o = reinterpret_cast<float*>(smem);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int head = 2 * t + h;
        float top = sm_m[0][head];
#pragma unroll
        for (int x = 1; x < kWarps; ++x) top = fmaxf(top, sm_m[x][head]);
        const float f = ex2(mw[h] + kLift - top), drop = 1.f / (1 << (int)kLift);  // (apart: their product may be subnormal)
#pragma unroll
        for (int q = 0; q < VC; ++q)
#pragma unroll
          for (int m = 0; m < VW * 2; ++m) {
            float* dst = sm_o + (warp * kHeads + head) * DP + 8 * VP * q + VP * g + 2 * m;
            *reinterpret_cast<float2*>(dst) = make_float2(o[q * VW * 2 + m][h] * drop * f, o[q * VW * 2 + m][2 + h] * drop * f);
          }
      }
      __syncthreads();
      const bool whole = u0 == 0 && rel + n_seg == n_pair;  // this CTA saw all of the pair's keys
      const int part = blockIdx.x * 2 + (u0 > 0 ? 0 : 1);  // a CTA's first pair may have begun before it, its last go on
#pragma unroll 1
      for (int i = threadIdx.x; i < nheads * DP; i += kThreads) {
        const int head = i / DP, c = i % DP;
        if (c >= p.d) continue;
        float top = sm_m[0][head], sum = 0.f, acc = 0.f;
#pragma unroll
        for (int x = 1; x < kWarps; ++x) top = fmaxf(top, sm_m[x][head]);
#pragma unroll
        for (int x = 0; x < kWarps; ++x)
          sum += sm_l[x][head] * ex2(sm_m[x][head] - top), acc += sm_o[(x * kHeads + head) * DP + c];
        if (whole) {
          T* dst = static_cast<T*>(p.out) + ((long long)b * p.Hq + hkv * p.G + head0 + head) * p.d + c;
          if (SAGE_STORE_OK(p.x_out, dst, 2, &g_decode_error)) *dst = from_f32<T>(sum == 0.f ? 0.f : acc / sum);
        } else {
          float* dst = p.part_o + (long long)(part * kHeads + head) * dc + c;
          if (SAGE_STORE_OK(p.x_part_o, dst, 4, &g_decode_error)) *dst = acc;
          if (c == 0) {
            float* ml = p.part_ml + (part * kHeads + head) * 2;
            if (SAGE_STORE_OK(p.x_part_ml, ml, 8, &g_decode_error)) ml[0] = top, ml[1] = sum;
          }
        }
      }
      if (sm_dead) return;
    }
    unit += n_seg, pair0 += n_pair;
    if (unit >= unit_end) return;
    if (++pair == p.pairs) pair = 0, ++b, len = seq_len_of(p, b, !p.part_o && threadIdx.x == 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();  // O is read: the rings may be filled again
  }
}

// Joins the pairs that cross CTAs: out = sum_i O_i 2^(m_i - M) / sum_i l_i 2^(m_i - M), i over the CTAs that a
// pair crosses.  CTA c of this kernel looks at the border before CTA c + 1 of the other, and takes the pair there if
// that is the first border inside it.  Launched as a programmatic dependent: it finds its pair while the
// other kernel still runs.  Warps share out the tile's heads, then the parts; a warp's loads are in
// flight eight at a time (one at a time cost 20 us for the 56 parts of a 131072-key sequence).
constexpr int kJoinWarps = 8, kJoinBatch = 8;
template <typename T, int V>  // V float4 per lane: d <= 128 V
__global__ void __launch_bounds__(kJoinWarps * 32, 3) decode_join_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int kBatch = kJoinBatch / V;
  __shared__ float4 sm_o[kJoinWarps][32 * V];
  const Place at = find_place<kJoinWarps * 32>(p, blockIdx.x + 1, false);
  // Every CTA waits, those without a border too: where none had to, this grid would end before the other, and what
  // follows it in the stream is ordered behind this grid alone.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (at.b < 0) return;
  const uint32_t u = (blockIdx.x + 1) * at.share, keys0 = at.pair0 + p.unit_extra;
  if (u <= keys0 || u - at.share > keys0) return;  // no pair's keys cross here, or they crossed an earlier border
  const int c0 = blockIdx.x, n = (int)((at.pair0 + units_of(p, at.len) - 1) / at.share) - c0 + 1;
  const int hkv = at.pair / p.tiles, head0 = (at.pair % p.tiles) * kHeads, nheads = min(kHeads, p.G - head0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, dc = p.map.dc;
  const int ways = kJoinWarps / (nheads > 4 ? 8 : nheads > 2 ? 4 : nheads);  // warps per head
  const int head = min(warp / ways, nheads - 1), way = warp % ways;
  // CTA c's part: its last pair's (1) where the pair began, its first one's (0) behind that
  const auto part = [&](int i) { return (long long)((c0 + i) * 2 + (i == 0 ? 1 : 0)) * kHeads + head; };
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  float top = -FLT_MAX, sum = 0.f;
  for (int i = lane; i < n; i += 32) top = fmaxf(top, __ldcg(ml + part(i)).x);
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  float4 acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int i0 = way; i0 < n; i0 += kBatch * ways) {
    // loads without a condition (the last part again behind the last; column 0 behind dc), so that all are in flight
    float2 x[kBatch];
    float4 o[kBatch][V];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const long long at_i = part(min(i0 + k * ways, n - 1));
      x[k] = __ldcg(ml + at_i);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = 4 * (lane + 32 * v);
        o[k][v] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at_i * dc + (c < dc ? c : 0)));
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (i0 + k * ways < n) {
        const float f = ex2(x[k].x - top);
        sum += x[k].y * f;
#pragma unroll
        for (int v = 0; v < V; ++v)
          acc[v].x += o[k][v].x * f, acc[v].y += o[k][v].y * f, acc[v].z += o[k][v].z * f, acc[v].w += o[k][v].w * f;
      }
    }
  }
  __shared__ float sm_l[kJoinWarps];
#pragma unroll
  for (int v = 0; v < V; ++v) sm_o[warp][lane + 32 * v] = acc[v];
  if (lane == 0) sm_l[warp] = sum;
  __syncthreads();
#pragma unroll 1
  for (int i = threadIdx.x; i < nheads * 128 * V; i += kJoinWarps * 32) {
    const int h = i / (128 * V), c = i % (128 * V);
    if (c >= p.d) continue;
    float num = 0.f, den = 0.f;
#pragma unroll 1
    for (int x = h * ways; x < (h + 1) * ways; ++x) num += reinterpret_cast<const float*>(sm_o[x])[c], den += sm_l[x];
    T* dst = static_cast<T*>(p.out) + ((long long)at.b * p.Hq + hkv * p.G + head0 + h) * p.d + c;
    if (SAGE_STORE_OK(p.x_out, dst, 2, &g_decode_error)) *dst = from_f32<T>(den == 0.f ? 0.f : num / den);
  }
}

template <typename T, int DP>
cudaError_t launch_decode_dp(const DecodeParams& p, cudaStream_t st) {
  const auto kernel = decode_kernel<T, DP>;
  // once per device: setting it twice does no harm
  static std::atomic<bool> ready[128];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<DP>::cta_bytes(DP));
    if (e != cudaSuccess) return e;
    ready[dev].store(true, std::memory_order_release);
  }
  return launch_dependent(kernel, p.ctas, kThreads, Ring<DP>::cta_bytes(p.map.dc), st, p);
}

template <typename T>
cudaError_t launch_decode_t(const DecodeParams& p, cudaStream_t st) {
  const cudaError_t e = p.d <= 64    ? launch_decode_dp<T, 64>(p, st)
                        : p.d <= 128 ? launch_decode_dp<T, 128>(p, st)
                                     : launch_decode_dp<T, 256>(p, st);
  if (e != cudaSuccess || !p.part_o) return e;
  return launch_dependent(p.d <= 128 ? decode_join_kernel<T, 1> : decode_join_kernel<T, 2>, p.ctas - 1, kJoinWarps * 32,
                          0, st, p);
}

}  // namespace

int decode_ctas_per_sm(int d) { return d <= 128 ? 3 : 2; }

cudaError_t launch_decode(const DecodeParams& p, int dtype, cudaStream_t st) {
  return dtype == SAGE_FP16 ? launch_decode_t<__half>(p, st) : launch_decode_t<__nv_bfloat16>(p, st);
}

}  // namespace sage
