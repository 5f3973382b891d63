// C ABI: argument checks, workspace, TMA tensor maps and launches.
// The operation and the argument contract are documented in include/sage.h.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <atomic>
#include <mutex>

#include "sage_internal.h"

using namespace sage;

namespace {

constexpr size_t kAlign = 1024;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

int padded_dim(int d) { return d <= 64 ? 64 : (d <= 128 ? 128 : 256); }

// Sizes of one call.  Dense batches: B sequences of Nq queries and Nk keys.  Packed (varlen)
// batches: B sequences of at most Nq / Nk tokens, total_q / total_k tokens in all.
struct Dims {
  int B, Hq, Hkv, Nq, Nk, d, dp, G;
  int nblk_q, nblk_k;                  // 128-token blocks of the longest query / key sequence
  long long q_head_rows, k_head_rows;  // q8 / k8 rows between heads (dense Npq / Npk; packed Tq / Tk)
  long long q_rows, k_rows;            // q8 / k8 rows in all
  bool packed;
  long long total_q, total_k;
};

long long round128(long long x) { return (x + 127) / 128 * 128; }

sage_status finish_dims(Dims* m) {
  m->dp = padded_dim(m->d);
  m->G = m->Hq / m->Hkv;
  m->nblk_q = (m->Nq + 127) / 128;
  m->nblk_k = (m->Nk + 127) / 128;
  if (m->packed) {
    // every sequence starts a fresh 128-row block: sum of round128(n_b) <= total + 127 B
    m->q_head_rows = round128(m->total_q) + 128LL * m->B;
    m->k_head_rows = round128(m->total_k) + 128LL * m->B;
    m->q_rows = m->q_head_rows * m->Hq;
    m->k_rows = m->k_head_rows * m->Hkv;
  } else {
    m->q_head_rows = round128(m->Nq);
    m->k_head_rows = round128(m->Nk);
    m->q_rows = m->q_head_rows * m->Hq * m->B;
    m->k_rows = m->k_head_rows * m->Hkv * m->B;
  }
  // TMA coordinates are 32-bit signed: rows of q8 / k8 / V^T and the byte column of V^T
  const long long v_rows = m->k_rows / m->k_head_rows * m->dp;
  if (m->q_rows >= (1LL << 31) || m->k_rows >= (1LL << 31) || v_rows >= (1LL << 31) ||
      m->k_head_rows * 2 >= (1LL << 31))
    return SAGE_ERR_INVALID_ARG;
  return SAGE_OK;
}

sage_status check_heads(int B, int Hq, int Hkv, int d) {
  if (B < 1 || Hq < 1 || Hkv < 1 || d < 1) return SAGE_ERR_INVALID_ARG;
  if (d > 256 || Hq % Hkv != 0) return SAGE_ERR_INVALID_ARG;
  if (B > 65535 || 2L * Hq > 65535 || (long)Hq + 2L * Hkv > 65535) return SAGE_ERR_INVALID_ARG;
  return SAGE_OK;
}

sage_status check_dims(int B, int Hq, int Hkv, int Nq, int Nk, int d, Dims* out) {
  sage_status s = check_heads(B, Hq, Hkv, d);
  if (s != SAGE_OK) return s;
  if (Nq < 1 || Nk < 1 || Nq > (1 << 30) || Nk > (1 << 30)) return SAGE_ERR_INVALID_ARG;
  Dims m;
  m.B = B, m.Hq = Hq, m.Hkv = Hkv, m.Nq = Nq, m.Nk = Nk, m.d = d;
  m.packed = false;
  m.total_q = (long long)B * Nq, m.total_k = (long long)B * Nk;
  if ((s = finish_dims(&m)) != SAGE_OK) return s;
  *out = m;
  return SAGE_OK;
}

sage_status check_dims_packed(int B, int Hq, int Hkv, int max_q, int max_k, long long total_q, long long total_k,
                              int d, Dims* out) {
  sage_status s = check_heads(B, Hq, Hkv, d);
  if (s != SAGE_OK) return s;
  if (max_q < 1 || max_k < 0 || total_q < 1 || total_k < 0 || max_q > (1 << 30) || max_k > (1 << 30) ||
      total_q > (1LL << 40) || total_k > (1LL << 40))
    return SAGE_ERR_INVALID_ARG;
  Dims m;
  m.B = B, m.Hq = Hq, m.Hkv = Hkv, m.Nq = max_q, m.Nk = max_k, m.d = d;
  m.packed = true;
  m.total_q = total_q, m.total_k = total_k;
  if ((s = finish_dims(&m)) != SAGE_OK) return s;
  *out = m;
  return SAGE_OK;
}

SeqMap seq_map(const Dims& m, int layout, const SeqDesc* seqs) {
  SeqMap s;
  s.seqs = m.packed ? seqs : nullptr;
  s.B = m.B, s.Hq = m.Hq, s.Hkv = m.Hkv, s.d = m.d, s.dp = m.dp;
  s.Nq = m.Nq, s.Nk = m.Nk;
  s.q_head_rows = m.q_head_rows, s.k_head_rows = m.k_head_rows;
  s.layout = m.packed ? SAGE_NHD : layout;
  return s;
}

sage_status check_dtype(int dtype) {
  if (dtype == SAGE_FP32) return SAGE_ERR_UNSUPPORTED;
  if (dtype != SAGE_FP16 && dtype != SAGE_BF16) return SAGE_ERR_INVALID_ARG;
  return SAGE_OK;
}

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}

sage_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return SAGE_OK;
  return e == cudaErrorMemoryAllocation ? SAGE_ERR_OOM : SAGE_ERR_CUDA;
}

// Host-side failure injection (sage_test_inject): a compute capability reported instead of the
// device's (0: query the device), and a number of workspace allocations to fail.
std::atomic<int> g_fake_cc{0};
std::atomic<int> g_fail_allocs{0};

sage_status check_device() {
  const int fake = g_fake_cc.load(std::memory_order_relaxed);
  if (fake) return fake == 100 ? SAGE_OK : SAGE_ERR_ARCH;
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SAGE_ERR_CUDA;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) return SAGE_ERR_CUDA;
  if (cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) return SAGE_ERR_CUDA;
  return (major == 10 && minor == 0) ? SAGE_OK : SAGE_ERR_ARCH;
}

float resolve_scale(float sm_scale, int d) {
  if (!(sm_scale > 0.f) || std::isnan(sm_scale)) return 1.0f / std::sqrt((float)d);
  return sm_scale;
}

// ---------------------------------------------------------------------------------- tensor maps
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// 2-D byte tensor: `inner` bytes per row (contiguous), `rows` rows, box {box_inner, box_rows}.
bool make_map(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint32_t box_inner, uint32_t box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {inner, rows};
  const cuuint64_t strides[1] = {inner};
  const cuuint32_t box[2] = {box_inner, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUtensorMapSwizzle swz = box_inner == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

bool pv_mode_valid(int pv_mode) {
  return pv_mode == SAGE_PV_FP32 || pv_mode == SAGE_PV_FP16_FP32 || pv_mode == SAGE_PV16_FP32 ||
         pv_mode == SAGE_PV16_FP16_FP32;
}
bool pv_mode_fp16_operands(int pv_mode) { return pv_mode == SAGE_PV16_FP32 || pv_mode == SAGE_PV16_FP16_FP32; }

// sage_opts, checked: log2 of the query tokens per Q scale, and V smoothing
struct Opts {
  int q_gran_log2 = 7;
  int smooth_v = 0;
};

sage_status parse_opts(const sage_opts* o, Opts* out) {
  Opts r;
  if (o) {
    switch (o->q_gran) {
      case 0:
      case 128: r.q_gran_log2 = 7; break;
      case 32: r.q_gran_log2 = 5; break;
      case 1: r.q_gran_log2 = 0; break;
      default: return SAGE_ERR_INVALID_ARG;
    }
    if (o->smooth_v != 0 && o->smooth_v != 1) return SAGE_ERR_INVALID_ARG;
    r.smooth_v = o->smooth_v;
  }
  *out = r;
  return SAGE_OK;
}

// Workspace memory: a stream-ordered pool per device, owned by the library, that keeps the
// memory it has handed out (release threshold = unlimited), so that repeated calls reuse
// it instead of mapping fresh device memory each time.
cudaError_t workspace_alloc(void** ptr, size_t bytes, cudaStream_t st) {
  for (int n = g_fail_allocs.load(); n > 0;)  // an injected failure, before any device call
    if (g_fail_allocs.compare_exchange_weak(n, n - 1)) return cudaErrorMemoryAllocation;
  constexpr int kMaxDevices = 128;
  static std::mutex mu;
  static cudaMemPool_t pools[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  cudaMemPool_t pool;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!pools[dev]) {
      cudaMemPoolProps props;
      memset(&props, 0, sizeof(props));
      props.allocType = cudaMemAllocationTypePinned;
      props.location.type = cudaMemLocationTypeDevice;
      props.location.id = dev;
      cudaMemPool_t p = nullptr;
      if ((e = cudaMemPoolCreate(&p, &props)) != cudaSuccess) return e;
      uint64_t keep = ~0ull;
      if ((e = cudaMemPoolSetAttribute(p, cudaMemPoolAttrReleaseThreshold, &keep)) != cudaSuccess) return e;
      pools[dev] = p;
    }
    pool = pools[dev];
  }
  return cudaMallocFromPoolAsync(ptr, bytes, pool, st);
}

// Store extents of the checked build (-DSAGE_CHECKED): each buffer's size as the header states it.
Extent extent_of(const void* ptr, size_t bytes) {
  Extent x;
  x.base = static_cast<unsigned char*>(const_cast<void*>(ptr));
  x.bytes = ptr ? bytes : 0;
  return x;
}

std::atomic<bool> g_serving{false};  // a serving kernel was launched, or captured: its error words may be set
std::atomic<long long> g_out_limit{0};  // test hook: narrows the output extent when > 0

Extent limited_extent(const void* out, size_t bytes) {
  const long long lim = g_out_limit.load();
  if (lim > 0 && (size_t)lim < bytes) bytes = (size_t)lim;
  return extent_of(out, bytes);
}

Extent out_extent(const Dims& m, const void* out) {
  return limited_extent(out, (size_t)m.total_q * m.Hq * m.d * 2);  // fp16 / bf16 output
}

struct QuantBufs {
  const SeqDesc* seqs;  // packed batches: the per-sequence table (else nullptr)
  float* vm;            // V's token mean (read only when V is smoothed)
  int8_t* q8;
  float* qs;
  int8_t* k8;
  float* ks;
  float* km;
  uint8_t* v8t;
  float* vs;
};

sage_status run_fwd(const Dims& m, const QuantBufs& qb, void* out, int dtype, int layout, int causal, float sm_scale,
                    int pv_mode, const Opts& o, cudaStream_t st) {
  CUtensorMap tq, tk, tv;
  const uint32_t ksub = m.dp >= 128 ? 128 : 64;
  const uint32_t dv = m.dp;  // V^T rows (channels) per tile: all of the padded head dim
  const bool pv16 = pv_mode_fp16_operands(pv_mode);
  const uint32_t bn = pv16 ? 64 : 128;  // keys per KV tile of the fused kernel
  const uint64_t vpitch = (uint64_t)m.k_head_rows * (pv16 ? 2 : 1);  // bytes per V^T row (one channel)
  // V^T tile box: 128 bytes of keys (128 E4M3 or 64 fp16 codes) x dv channels
  if (!make_map(&tq, qb.q8, m.dp, (uint64_t)m.q_rows, ksub, 128) ||
      !make_map(&tk, qb.k8, m.dp, (uint64_t)m.k_rows, ksub, bn) ||
      !make_map(&tv, qb.v8t, vpitch, (uint64_t)(m.k_rows / m.k_head_rows) * m.dp, 128, dv))
    return SAGE_ERR_CUDA;
  FwdParams p;
  p.qs = qb.qs, p.ks = qb.ks, p.vs = qb.vs, p.out = out;
  p.vm = o.smooth_v ? qb.vm : nullptr;
  p.q_gran_log2 = o.q_gran_log2;
  p.m = seq_map(m, layout, qb.seqs);
  p.nblk_q = m.nblk_q;
  p.G = m.G;
  p.vec_out = (m.d % 8 == 0) && aligned16(out);
  p.x_out = out_extent(m, out);
  p.scale_log2 = resolve_scale(sm_scale, m.d) * 1.4426950408889634f;
  return from_cuda(launch_fwd(tq, tk, tv, p, dtype, causal, pv_mode, st));
}

struct WsLayout {
  size_t q8, qs, k8, ks, km, v8t, vs, vm, ksum, vmax, vsum, vmin, vinv, seqs, total;
};

WsLayout ws_layout(const Dims& m, int pv_mode, const Opts& o) {
  WsLayout w;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes);
    return o;
  };
  w.q8 = take((size_t)m.q_rows * m.dp);
  w.qs = take(((size_t)m.q_rows >> o.q_gran_log2) * 4);
  w.k8 = take((size_t)m.k_rows * m.dp);
  w.ks = take((size_t)m.k_rows / 128 * 4);
  w.km = take((size_t)m.B * m.Hkv * m.dp * 4);
  w.v8t = take((size_t)m.k_rows * m.dp * (pv_mode_fp16_operands(pv_mode) ? 2 : 1));
  w.vs = take((size_t)m.B * m.Hkv * m.dp * 4);
  w.vm = take((size_t)m.B * m.Hkv * m.dp * 4);
  w.ksum = take((size_t)m.k_rows / 128 * m.dp * 4);
  w.vmax = take((size_t)m.k_rows / 128 * m.dp * 4);
  w.vsum = take(o.smooth_v ? (size_t)m.k_rows / 128 * m.dp * 4 : 0);
  w.vmin = take(o.smooth_v ? (size_t)m.k_rows / 128 * m.dp * 4 : 0);
  w.vinv = take((size_t)m.B * m.Hkv * m.dp * 4);
  w.seqs = take(m.packed ? (size_t)m.B * sizeof(SeqDesc) : 0);
  w.total = off;
  return w;
}

// Extents of every buffer the quantize kernels write, from the pointers already in p.
void set_quant_extents(QuantParams* p, const Dims& m, int pv_mode, const Opts& o) {
  const size_t per_head = (size_t)m.B * m.Hkv * m.dp * 4;
  const size_t part = (size_t)m.k_rows / 128 * m.dp * 4;
  p->x_q8 = extent_of(p->q8, (size_t)m.q_rows * m.dp);
  p->x_qs = extent_of(p->qs, ((size_t)m.q_rows >> o.q_gran_log2) * 4);
  p->x_k8 = extent_of(p->k8, (size_t)m.k_rows * m.dp);
  p->x_ks = extent_of(p->ks, (size_t)m.k_rows / 128 * 4);
  p->x_km = extent_of(p->km, per_head);
  p->x_v8t = extent_of(p->v8t, (size_t)m.k_rows * m.dp * (pv_mode_fp16_operands(pv_mode) ? 2 : 1));
  p->x_vs = extent_of(p->vs, per_head);
  p->x_vm = extent_of(p->vm, per_head);
  p->x_vinv = extent_of(p->vinv, per_head);
  p->x_ksum = extent_of(p->ksum_part, part);
  p->x_vmax = extent_of(p->vmax_part, part);
  p->x_vsum = extent_of(p->vsum_part, part);
  p->x_vmin = extent_of(p->vmin_part, part);
}

QuantParams quant_params(const Dims& m, const void* q, const void* k, const void* v, int dtype, int layout,
                         int pv_mode, const Opts& o) {
  QuantParams p;
  memset(&p, 0, sizeof(p));
  p.q = q, p.k = k, p.v = v;
  p.m = seq_map(m, layout, nullptr);  // packed batches set p.m.seqs once the table exists
  p.nblk_q = m.nblk_q, p.nblk_k = m.nblk_k;
  p.dtype = dtype;
  p.vec_q = (m.d % 8 == 0) && aligned16(q);
  p.vec_k = (m.d % 8 == 0) && aligned16(k);
  p.vec_v = (m.d % 8 == 0) && aligned16(v);
  p.vmax_code = pv_mode == SAGE_PV_FP32 ? 448.0f : 1.0f;
  p.v_fp16 = pv_mode_fp16_operands(pv_mode) ? 1 : 0;
  p.q_gran_log2 = o.q_gran_log2;
  p.smooth_v = o.smooth_v;
  return p;
}

sage_status check_common(const void* q, const void* k, const void* v, int dtype, int layout, int pv_mode) {
  if (!q || !k || !v) return SAGE_ERR_INVALID_ARG;
  sage_status s = check_dtype(dtype);
  if (s != SAGE_OK) return s;
  if (layout != SAGE_HND && layout != SAGE_NHD) return SAGE_ERR_INVALID_ARG;
  if (pv_mode == SAGE_PV16_FP16) return SAGE_ERR_UNSUPPORTED;
  if (!pv_mode_valid(pv_mode)) return SAGE_ERR_INVALID_ARG;
  return SAGE_OK;
}

// out must not overlap q, k or v (2-byte elements)
bool out_overlaps(const Dims& m, const void* q, const void* k, const void* v, const void* out) {
  const size_t qbytes = (size_t)m.total_q * m.Hq * m.d * 2, kvbytes = (size_t)m.total_k * m.Hkv * m.d * 2;
  return overlaps(out, qbytes, q, qbytes) || overlaps(out, qbytes, k, kvbytes) || overlaps(out, qbytes, v, kvbytes);
}

// Quantize pass + fused kernel on a workspace laid out by ws_layout(m, pv_mode, o); packed batches
// first build their per-sequence table from cu_q / cu_k.
sage_status attend_on(const Dims& m, unsigned char* ws, const void* q, const void* k, const void* v, void* out,
                      const int32_t* cu_q, const int32_t* cu_k, int dtype, int layout, int causal, float sm_scale,
                      int pv_mode, const Opts& o, cudaStream_t st) {
  const WsLayout w = ws_layout(m, pv_mode, o);
  SeqDesc* seqs = m.packed ? reinterpret_cast<SeqDesc*>(ws + w.seqs) : nullptr;
  if (m.packed) {
    sage_status s = from_cuda(launch_seq_plan(cu_q, cu_k, m.B, m.Nq, m.Nk, m.total_q, m.total_k, seqs, st));
    if (s != SAGE_OK) return s;
  }
  QuantParams qp = quant_params(m, q, k, v, dtype, layout, pv_mode, o);
  qp.m.seqs = seqs;
  QuantBufs qb{seqs,
               reinterpret_cast<float*>(ws + w.vm),
               reinterpret_cast<int8_t*>(ws + w.q8), reinterpret_cast<float*>(ws + w.qs),
               reinterpret_cast<int8_t*>(ws + w.k8), reinterpret_cast<float*>(ws + w.ks),
               reinterpret_cast<float*>(ws + w.km), ws + w.v8t, reinterpret_cast<float*>(ws + w.vs)};
  qp.q8 = qb.q8, qp.qs = qb.qs, qp.k8 = qb.k8, qp.ks = qb.ks, qp.km = qb.km, qp.v8t = qb.v8t, qp.vs = qb.vs;
  qp.vm = qb.vm;
  qp.ksum_part = reinterpret_cast<float*>(ws + w.ksum);
  qp.vmax_part = reinterpret_cast<float*>(ws + w.vmax);
  qp.vsum_part = reinterpret_cast<float*>(ws + w.vsum);
  qp.vmin_part = reinterpret_cast<float*>(ws + w.vmin);
  qp.vinv = reinterpret_cast<float*>(ws + w.vinv);
  set_quant_extents(&qp, m, pv_mode, o);
  sage_status s = from_cuda(launch_quantize(qp, st));
  if (s == SAGE_OK) s = run_fwd(m, qb, out, dtype, layout, causal, sm_scale, pv_mode, o, st);
  return s;
}

// The same, on a workspace taken from the library's pool and released stream-ordered.
sage_status attend_pooled(const Dims& m, const void* q, const void* k, const void* v, void* out, const int32_t* cu_q,
                          const int32_t* cu_k, int dtype, int layout, int causal, float sm_scale, int pv_mode,
                          const Opts& o, cudaStream_t st) {
  const WsLayout w = ws_layout(m, pv_mode, o);
  unsigned char* ws = nullptr;
  cudaError_t e = workspace_alloc(reinterpret_cast<void**>(&ws), w.total, st);
  if (e != cudaSuccess) return from_cuda(e);
  sage_status s = attend_on(m, ws, q, k, v, out, cu_q, cu_k, dtype, layout, causal, sm_scale, pv_mode, o, st);
  const cudaError_t ef = cudaFreeAsync(ws, st);
  if (s == SAGE_OK && ef != cudaSuccess) s = from_cuda(ef);
  return s;
}

}  // namespace

extern "C" {

size_t sage_workspace_bytes(int B, int Hq, int Hkv, int N, int d) {
  Dims m;
  if (check_dims(B, Hq, Hkv, N, N, d, &m) != SAGE_OK) return 0;
  Opts largest;
  largest.q_gran_log2 = 0, largest.smooth_v = 1;
  return ws_layout(m, SAGE_PV16_FP32, largest).total;  // the largest over the P.V modes and options
}

sage_status sage_attn_ex(const void* q, const void* k, const void* v, void* out, int B, int Hq, int Hkv, int Nq,
                         int Nk, int d, sage_dtype dtype, sage_layout layout, int is_causal, float sm_scale,
                         sage_pv_mode pv_mode, const sage_opts* opts, void* stream) {
  sage_status s = check_common(q, k, v, dtype, layout, pv_mode);
  if (s != SAGE_OK) return s;
  Opts o;
  if ((s = parse_opts(opts, &o)) != SAGE_OK) return s;
  Dims m;
  if ((s = check_dims(B, Hq, Hkv, Nq, Nk, d, &m)) != SAGE_OK) return s;
  if (!out || out_overlaps(m, q, k, v, out)) return SAGE_ERR_INVALID_ARG;
  if ((s = check_device()) != SAGE_OK) return s;
  return attend_pooled(m, q, k, v, out, nullptr, nullptr, dtype, layout, is_causal ? 1 : 0, sm_scale, pv_mode, o,
                       static_cast<cudaStream_t>(stream));
}

sage_status sage_attn(const void* q, const void* k, const void* v, void* out, int B, int Hq, int Hkv, int N, int d,
                      sage_dtype dtype, sage_layout layout, int is_causal, float sm_scale, sage_pv_mode pv_mode,
                      void* stream) {
  return sage_attn_ex(q, k, v, out, B, Hq, Hkv, N, N, d, dtype, layout, is_causal, sm_scale, pv_mode, nullptr,
                      stream);
}

sage_status sage_attn_varlen(const void* q, const void* k, const void* v, void* out, const int32_t* cu_seqlens_q,
                             const int32_t* cu_seqlens_k, int B, int max_seqlen_q, int max_seqlen_k,
                             long long total_q, long long total_k, int Hq, int Hkv, int d, sage_dtype dtype,
                             int is_causal, float sm_scale, sage_pv_mode pv_mode, const sage_opts* opts,
                             void* stream) {
  sage_status s = check_common(q, k, v, dtype, SAGE_NHD, pv_mode);
  if (s != SAGE_OK) return s;
  Opts o;
  if ((s = parse_opts(opts, &o)) != SAGE_OK) return s;
  if (!cu_seqlens_q || !cu_seqlens_k) return SAGE_ERR_INVALID_ARG;
  Dims m;
  if ((s = check_dims_packed(B, Hq, Hkv, max_seqlen_q, max_seqlen_k, total_q, total_k, d, &m)) != SAGE_OK) return s;
  if (!out || out_overlaps(m, q, k, v, out)) return SAGE_ERR_INVALID_ARG;
  if ((s = check_device()) != SAGE_OK) return s;
  return attend_pooled(m, q, k, v, out, cu_seqlens_q, cu_seqlens_k, dtype, SAGE_NHD, is_causal ? 1 : 0, sm_scale,
                       pv_mode, o, static_cast<cudaStream_t>(stream));
}

sage_status sage_quantize(const void* q, const void* k, const void* v, int B, int Hq, int Hkv, int N, int d,
                          sage_dtype dtype, sage_layout layout, sage_pv_mode pv_mode, const sage_opts* opts,
                          int8_t* q8, float* qs, int8_t* k8, float* ks, float* km, uint8_t* v8t, float* vs,
                          float* vm, void* stream) {
  sage_status s = check_common(q, k, v, dtype, layout, pv_mode);
  if (s != SAGE_OK) return s;
  Opts o;
  if ((s = parse_opts(opts, &o)) != SAGE_OK) return s;
  Dims m;
  if ((s = check_dims(B, Hq, Hkv, N, N, d, &m)) != SAGE_OK) return s;
  if (!q8 || !qs || !k8 || !ks || !km || !v8t || !vs || (o.smooth_v && !vm)) return SAGE_ERR_INVALID_ARG;
  if (!aligned16(q8) || !aligned16(k8) || !aligned16(v8t)) return SAGE_ERR_INVALID_ARG;
  if ((s = check_device()) != SAGE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t part = align_up((size_t)m.k_rows / 128 * m.dp * 4);
  const size_t vinv = align_up((size_t)m.B * m.Hkv * m.dp * 4);
  const int nparts = o.smooth_v ? 4 : 2;
  unsigned char* scratch = nullptr;
  cudaError_t e = workspace_alloc(reinterpret_cast<void**>(&scratch), nparts * part + vinv, st);
  if (e != cudaSuccess) return from_cuda(e);
  QuantParams qp = quant_params(m, q, k, v, dtype, layout, pv_mode, o);
  qp.q8 = q8, qp.qs = qs, qp.k8 = k8, qp.ks = ks, qp.km = km, qp.v8t = v8t, qp.vs = vs, qp.vm = vm;
  qp.ksum_part = reinterpret_cast<float*>(scratch);
  qp.vmax_part = reinterpret_cast<float*>(scratch + part);
  qp.vsum_part = o.smooth_v ? reinterpret_cast<float*>(scratch + 2 * part) : nullptr;
  qp.vmin_part = o.smooth_v ? reinterpret_cast<float*>(scratch + 3 * part) : nullptr;
  qp.vinv = reinterpret_cast<float*>(scratch + nparts * part);
  set_quant_extents(&qp, m, pv_mode, o);
  s = from_cuda(launch_quantize(qp, st));
  const cudaError_t ef = cudaFreeAsync(scratch, st);
  if (s == SAGE_OK && ef != cudaSuccess) s = from_cuda(ef);
  return s;
}

sage_status sage_attn_quantized(const int8_t* q8, const float* qs, const int8_t* k8, const float* ks,
                                const uint8_t* v8t, const float* vs, const float* vm, void* out, int B, int Hq,
                                int Hkv, int N, int d, sage_dtype out_dtype, sage_layout out_layout, int is_causal,
                                float sm_scale, sage_pv_mode pv_mode, const sage_opts* opts, void* stream) {
  if (!q8 || !qs || !k8 || !ks || !v8t || !vs || !out) return SAGE_ERR_INVALID_ARG;
  sage_status s = check_dtype(out_dtype);
  if (s != SAGE_OK) return s;
  if (out_layout != SAGE_HND && out_layout != SAGE_NHD) return SAGE_ERR_INVALID_ARG;
  if (pv_mode == SAGE_PV16_FP16) return SAGE_ERR_UNSUPPORTED;
  if (!pv_mode_valid(pv_mode)) return SAGE_ERR_INVALID_ARG;
  Opts o;
  if ((s = parse_opts(opts, &o)) != SAGE_OK) return s;
  if (o.smooth_v && !vm) return SAGE_ERR_INVALID_ARG;
  Dims m;
  if ((s = check_dims(B, Hq, Hkv, N, N, d, &m)) != SAGE_OK) return s;
  if (!aligned16(q8) || !aligned16(k8) || !aligned16(v8t)) return SAGE_ERR_INVALID_ARG;
  if ((s = check_device()) != SAGE_OK) return s;
  QuantBufs qb{nullptr, const_cast<float*>(vm), const_cast<int8_t*>(q8), const_cast<float*>(qs),
               const_cast<int8_t*>(k8), const_cast<float*>(ks), nullptr, const_cast<uint8_t*>(v8t),
               const_cast<float*>(vs)};
  return run_fwd(m, qb, out, out_dtype, out_layout, is_causal ? 1 : 0, sm_scale, pv_mode, o,
                 static_cast<cudaStream_t>(stream));
}

sage_status sage_qk_int32(const int8_t* q8, const int8_t* k8, int B, int Hq, int Hkv, int N, int d,
                          const int32_t* tiles, int n_tiles, int32_t* s_out, void* stream) {
  if (!q8 || !k8 || !tiles || !s_out || n_tiles < 0) return SAGE_ERR_INVALID_ARG;
  Dims m;
  sage_status s = check_dims(B, Hq, Hkv, N, N, d, &m);
  if (s != SAGE_OK) return s;
  if (!aligned16(q8) || !aligned16(k8) || !aligned16(s_out)) return SAGE_ERR_INVALID_ARG;
  if (n_tiles == 0) return SAGE_OK;
  if ((s = check_device()) != SAGE_OK) return s;
  CUtensorMap tq, tk;
  const uint32_t ksub = m.dp >= 128 ? 128 : 64;
  if (!make_map(&tq, q8, m.dp, (uint64_t)m.q_rows, ksub, 128) || !make_map(&tk, k8, m.dp, (uint64_t)m.k_rows, ksub, 128))
    return SAGE_ERR_CUDA;
  QkDumpParams p;
  p.tiles = tiles, p.n_tiles = n_tiles, p.out = s_out;
  p.B = m.B, p.Hq = m.Hq, p.Hkv = m.Hkv, p.Np = (int)m.q_head_rows, p.nblk = m.nblk_q, p.G = m.G;
  return from_cuda(launch_qk_dump(tq, tk, p, m.dp, static_cast<cudaStream_t>(stream)));
}

sage_status sage_mma_probe(int kind, int iters, double* ops, void* stream) {
  if (kind < 0 || kind > 2 || iters < 1 || iters > 1000000 || !ops) return SAGE_ERR_INVALID_ARG;
  sage_status s = check_device();
  if (s != SAGE_OK) return s;
  int dev = 0, n_sm = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SAGE_ERR_CUDA;
  if (cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n_sm <= 0)
    return SAGE_ERR_CUDA;
  const double k = kind == 2 ? 16.0 : 32.0;
  *ops = (double)n_sm * iters * 4.0 * 2.0 * 128.0 * 256.0 * k;
  return from_cuda(launch_mma_probe(kind, iters, n_sm, static_cast<cudaStream_t>(stream)));
}

sage_status sage_selftest_wait_timeout(int budget_us, void* stream) {
  if (budget_us < 1 || budget_us > 100000) return SAGE_ERR_INVALID_ARG;
  sage_status s = check_device();
  if (s != SAGE_OK) return s;
  int dev = 0, khz = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SAGE_ERR_CUDA;
  if (cudaDeviceGetAttribute(&khz, cudaDevAttrClockRate, dev) != cudaSuccess || khz <= 0) return SAGE_ERR_CUDA;
  return from_cuda(launch_wait_probe((long long)budget_us * (khz / 1000), static_cast<cudaStream_t>(stream)));
}

sage_status sage_check_status(void* stream) {
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return SAGE_ERR_CUDA;
  int flags = 0;
  int qflags = 0;
  if (read_clear_device_error(&flags) != cudaSuccess) return SAGE_ERR_CUDA;
  if (read_clear_quant_error(&qflags) != cudaSuccess) return SAGE_ERR_CUDA;
  int cflags = 0, dflags = 0;
  if (g_serving.load()) {  // (a word read is 14 us)
    if (read_clear_cache_error(&cflags) != cudaSuccess) return SAGE_ERR_CUDA;
    if (read_clear_decode_error(&dflags) != cudaSuccess) return SAGE_ERR_CUDA;
  }
  flags |= qflags | cflags | dflags;
  if (flags & 1) return SAGE_ERR_TIMEOUT;
  if (flags & SAGE_DEVERR_BOUNDS) return SAGE_ERR_BOUNDS;
  if (flags & 2) return SAGE_ERR_INVALID_ARG;
  return SAGE_OK;
}

const char* sage_status_string(sage_status s) {
  switch (s) {
    case SAGE_OK: return "ok";
    case SAGE_ERR_INVALID_ARG: return "invalid argument";
    case SAGE_ERR_UNSUPPORTED: return "unsupported (inputs must be fp16 or bf16)";
    case SAGE_ERR_ARCH: return "device is not compute capability 10.0 (B200, sm_100a)";
    case SAGE_ERR_CUDA: return "CUDA error";
    case SAGE_ERR_OOM: return "out of device memory";
    case SAGE_ERR_TIMEOUT: return "a kernel gave up on a bounded wait";
    case SAGE_ERR_BOUNDS: return "a kernel skipped a store outside its buffer (checked build)";
  }
  return "unknown status";
}

int sage_device_supported(void) { return check_device() == SAGE_OK ? 1 : 0; }

void sage_test_inject(int fake_cc, int fail_allocs) {
  g_fake_cc.store(fake_cc > 0 ? fake_cc : 0);
  g_fail_allocs.store(fail_allocs > 0 ? fail_allocs : 0);
}

void sage_test_out_limit(long long bytes) { g_out_limit.store(bytes > 0 ? bytes : 0); }

int sage_checked_build(void) {
#ifdef SAGE_CHECKED
  return 1;
#else
  return 0;
#endif
}

}  // extern "C"

// ------------------------------------------------------------------------------------------------
// Serving: head norm and rotation, the paged cache, one-token attention.
// ------------------------------------------------------------------------------------------------
namespace {

// Strides, and every view's extent along each dimension, stay below these, so that no offset passes 2^63.
constexpr long long kMaxStride = 1LL << 40, kMaxExtent = 1LL << 48;
constexpr long long kMaxItems = 1LL << 31;  // row groups of one launch (32-bit numbers)

sage_status check_strides(const long long* s, int n) {
  if (!s) return SAGE_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (s[i] < 0 || s[i] > kMaxStride) return SAGE_ERR_INVALID_ARG;
  return SAGE_OK;
}

sage_status check_norm_rope(const sage_norm_rope* nr, int d) {
  if (!nr) return SAGE_ERR_INVALID_ARG;
  if (nr->norm && !(nr->eps >= 0.f && nr->eps <= 3.4e38f)) return SAGE_ERR_INVALID_ARG;
  if (nr->norm && (nr->q_weight || nr->k_weight)) {
    if (nr->weight_dtype != SAGE_FP16 && nr->weight_dtype != SAGE_BF16 && nr->weight_dtype != SAGE_FP32)
      return SAGE_ERR_INVALID_ARG;
    const uintptr_t a = nr->weight_dtype == SAGE_FP32 ? 3 : 1;
    if (((uintptr_t)nr->q_weight & a) || ((uintptr_t)nr->k_weight & a)) return SAGE_ERR_INVALID_ARG;
  }
  if (!nr->norm && (nr->q_weight || nr->k_weight)) return SAGE_ERR_INVALID_ARG;
  if (nr->cos_sin) {
    if (nr->n_pos < 1 || nr->rot < 2 || nr->rot > d || nr->rot % 2 != 0) return SAGE_ERR_INVALID_ARG;
    if ((uintptr_t)nr->cos_sin & 3) return SAGE_ERR_INVALID_ARG;
  }
  return SAGE_OK;
}

sage_status check_cache(const sage_kv_cache* c, const int32_t* table, long long table_stride, int max_pages, int B,
                        PageMap* m) {
  if (!c || !c->k8 || !c->ks || !c->v8 || !c->vs) return SAGE_ERR_INVALID_ARG;
  if (!aligned16(c->k8) || !aligned16(c->v8) || !aligned16(c->ks) || !aligned16(c->vs) || ((uintptr_t)table & 3))
    return SAGE_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->Hkv < 1 || c->Hkv > 65535 || c->d < 1 || c->d > 256) return SAGE_ERR_INVALID_ARG;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1))) return SAGE_ERR_INVALID_ARG;
  if (max_pages < 0 || table_stride < 0 || table_stride > kMaxStride) return SAGE_ERR_INVALID_ARG;
  if (B > 0 && (!table || max_pages < 1)) return SAGE_ERR_INVALID_ARG;
  if (B > 1 && table_stride < max_pages) return SAGE_ERR_INVALID_ARG;
  m->k8 = c->k8, m->ks = c->ks, m->v8 = c->v8, m->vs = c->vs;
  m->table = table, m->table_stride = table_stride;
  m->max_pages = max_pages, m->num_pages = c->num_pages, m->Hkv = c->Hkv;
  m->dc = (c->d + 15) / 16 * 16;
  m->page_log2 = 0;
  while ((1 << m->page_log2) < c->page_size) ++m->page_log2;
  return SAGE_OK;
}

size_t cache_rows(const PageMap& m) { return ((size_t)m.num_pages * m.Hkv) << m.page_log2; }

bool overlaps_cache(const void* p, size_t n, const PageMap& m) {
  const size_t scales = cache_rows(m) * 4, codes = cache_rows(m) * m.dc;
  return overlaps(p, n, m.k8, codes) || overlaps(p, n, m.v8, codes) || overlaps(p, n, m.ks, scales) ||
         overlaps(p, n, m.vs, scales);
}

bool view_fits(const HeadView& v, long long B, long long N, long long H) {
  const auto fits = [](long long n, long long stride) { return stride == 0 || (n - 1) <= kMaxExtent / stride; };
  return fits(B, v.batch) && fits(N, v.token) && fits(H, v.head);
}

// Bytes from the first to behind the last element of (B, N, H, d) 16-bit values with these strides.
size_t view_bytes(const HeadView& v, long long B, long long N, long long H, long long d) {
  return (size_t)((B - 1) * v.batch + (N - 1) * v.token + (H - 1) * v.head + d) * 2;
}

// Whether a place can belong to both views (conservative).  They are apart where their extents are, and where they
// are slices side by side of rows S elements apart, S one of the strides: every larger stride in use a multiple of S, and what the
// others span disjoint modulo S (q and k of one fused projection).
bool views_overlap(const HeadView& a, const long long na[3], const HeadView& b, const long long nb[3], long long d) {
  const long long sa[3] = {a.batch, a.token, a.head}, sb[3] = {b.batch, b.token, b.head};
  if (!overlaps(a.ptr, view_bytes(a, na[0], na[1], na[2], d), b.ptr, view_bytes(b, nb[0], nb[1], nb[2], d))) return false;
  const long long apart = ((long long)(uintptr_t)b.ptr - (long long)(uintptr_t)a.ptr) / 2;  // (both addresses are even)
  for (const long long S : sa) {
    if (S == 0) continue;
    long long span[2] = {d, d};  // elements of the dimensions inside a row
    bool rows = true;
    for (int i = 0; i < 3; ++i) {
      const long long n[2] = {na[i], nb[i]}, s[2] = {sa[i], sb[i]};
      for (int x = 0; x < 2; ++x) {
        if (n[x] == 1) continue;
        if (s[x] < S)
          span[x] += (n[x] - 1) * s[x];
        else
          rows = rows && s[x] % S == 0;
      }
    }
    const long long at = ((apart % S) + S) % S;  // of b's first element in a's row
    if (rows && at >= span[0] && at + span[1] <= S) return false;
  }
  return true;
}

bool same_view(const HeadView& a, const HeadView& b, const long long n[3]) {
  return a.ptr == b.ptr && (n[0] == 1 || a.batch == b.batch) && (n[1] == 1 || a.token == b.token) &&
         (n[2] == 1 || a.head == b.head);
}

// Whether two elements of a view can share a place (conservative): its strides in use, in order of size, each pass over
// what the smaller ones span.
bool overlaps_itself(const HeadView& v, const long long n[3], long long d) {
  long long s[3] = {v.batch, v.token, v.head}, m[3] = {n[0], n[1], n[2]}, span = d;
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (s[j] < s[i]) std::swap(s[i], s[j]), std::swap(m[i], m[j]);
  for (int i = 0; i < 3; ++i) {
    if (m[i] == 1) continue;
    if (s[i] < span) return true;
    span += (m[i] - 1) * s[i];
  }
  return false;
}

// Outputs may be their own inputs; otherwise no output shares a place with a view that is read, another output
// or itself.  (Rows of one kind are written while others are read.)
sage_status check_apart(const HeadRowsParams& p, int batches) {
  for (const HeadRows& o : p.kind) {
    if (!o.H || !o.out.ptr) continue;
    const long long no[3] = {batches, p.N, o.H};
    if (overlaps_itself(o.out, no, p.d)) return SAGE_ERR_INVALID_ARG;
    for (const HeadRows& k : p.kind) {
      if (!k.H) continue;
      const long long nk[3] = {batches, p.N, k.H};
      if (!(&k == &o && same_view(o.out, k.in, no)) && views_overlap(o.out, no, k.in, nk, p.d)) return SAGE_ERR_INVALID_ARG;
      if (&k != &o && k.out.ptr && views_overlap(o.out, no, k.out, nk, p.d)) return SAGE_ERR_INVALID_ARG;
    }
  }
  return SAGE_OK;
}

// 16-byte vectors: the base aligned and every stride in use a multiple of eight elements.
bool vec_view(const HeadView& v, long long B, long long N, long long H) {
  return aligned16(v.ptr) && (B == 1 || v.batch % 8 == 0) && (N == 1 || v.token % 8 == 0) &&
         (H == 1 || v.head % 8 == 0);
}

// Checks the views' extents, and takes from their alignment whether rows go in vectors.
sage_status take_views(HeadRowsParams* p, int batches) {
  for (HeadRows& k : p->kind)
    for (const HeadView* v : {&k.in, &k.out}) {
      if (!k.H || !v->ptr) continue;
      if (!view_fits(*v, batches, p->N, k.H)) return SAGE_ERR_INVALID_ARG;
      p->vec = p->vec && vec_view(*v, batches, p->N, k.H);
      if (v == &k.out) k.x_out = extent_of(v->ptr, view_bytes(*v, batches, p->N, k.H, p->d));
    }
  return SAGE_OK;
}

void set_norm_rope(HeadRowsParams* p, const sage_norm_rope& nr) {
  p->norm = nr.norm ? 1 : 0, p->eps = nr.eps, p->inv_d = 1.0f / (float)p->d;
  p->kind[0].weight = nr.q_weight, p->kind[1].weight = nr.k_weight, p->weight_dtype = nr.weight_dtype;
  p->vec_weight = p->d % 8 == 0 && aligned16(nr.q_weight) && aligned16(nr.k_weight);
  p->cos_sin = nr.cos_sin, p->n_pos = nr.n_pos, p->rot = nr.cos_sin ? nr.rot : 0, p->interleaved = nr.interleaved ? 1 : 0;
  if (nr.cos_sin && nr.rot % 8 == 0) p->vec = p->vec && aligned16(nr.cos_sin);  // angles are loaded four at a time
}

// Heads of a token that a group of lanes takes at a time: four (fewer instructions per row, more loads in
// flight per thread) where `items` such groups still give every SM 2048 threads, else one (more
// threads at work on a short call: a decode step of 64 tokens).
int rows_per_group(bool vec, int d, long long items) {
  const int lanes = d <= 64 ? 8 : d <= 128 ? 16 : 32;
  return vec && items * lanes >= 148LL * 2048 ? 4 : 1;
}

sage_status shape_rows(HeadRowsParams* p, int batches) {
  const long long tokens = (long long)batches * p->N;
  if (tokens > kMaxItems) return SAGE_ERR_INVALID_ARG;
  const auto items = [&](int hc) {
    long long n = 0;
    for (const HeadRows& k : p->kind) n += (tokens + 15) * ((k.H + hc - 1) / hc);  // (whole rounds)
    return n;
  };
  p->heads_per_group = rows_per_group(p->vec, p->d, items(4));
  if (items(1) > kMaxItems) return SAGE_ERR_INVALID_ARG;
  p->tokens = (unsigned)tokens;
  return SAGE_OK;
}

}  // namespace

extern "C" {

sage_status sage_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const long long* strides,
                              const int32_t* positions, long long pos_batch_stride, int B, int N, int Hq, int Hkv,
                              int d, sage_dtype dtype, const sage_norm_rope* nr, void* stream) {
  sage_status s = check_dtype(dtype);
  if (s != SAGE_OK) return s;
  if (B < 0 || N < 0 || Hq < 1 || Hq > 65535 || d < 1 || d > 256) return SAGE_ERR_INVALID_ARG;
  if (k && (Hkv < 1 || Hkv > 65535)) return SAGE_ERR_INVALID_ARG;
  if ((s = check_strides(strides, 12)) != SAGE_OK) return s;
  if ((s = check_norm_rope(nr, d)) != SAGE_OK) return s;
  if (pos_batch_stride < 0 || pos_batch_stride > kMaxStride || ((uintptr_t)positions & 3)) return SAGE_ERR_INVALID_ARG;
  if (B == 0 || N == 0) return SAGE_OK;
  if (!q || !q_out || (k && !k_out)) return SAGE_ERR_INVALID_ARG;
  if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)q_out | (uintptr_t)k_out) & 1) return SAGE_ERR_INVALID_ARG;
  HeadRowsParams p;
  memset(&p, 0, sizeof(p));
  p.B = B, p.N = N, p.d = d, p.vec = d % 8 == 0;
  p.kind[0].in = HeadView{q, strides[0], strides[1], strides[2]}, p.kind[0].H = Hq;
  p.kind[1].in = HeadView{k, strides[3], strides[4], strides[5]}, p.kind[1].H = k ? Hkv : 0;
  p.kind[0].out = HeadView{q_out, strides[6], strides[7], strides[8]};
  p.kind[1].out = HeadView{k_out, strides[9], strides[10], strides[11]};
  if ((s = take_views(&p, B)) != SAGE_OK) return s;
  p.positions = positions, p.pos_batch = pos_batch_stride;
  set_norm_rope(&p, *nr);
  if ((s = shape_rows(&p, B)) != SAGE_OK) return s;
  if ((s = check_device()) != SAGE_OK) return s;
  if ((s = check_apart(p, B)) != SAGE_OK) return s;
  g_serving.store(true);
  return from_cuda(launch_head_rows(p, dtype, static_cast<cudaStream_t>(stream)));
}

sage_status sage_cache_append(const sage_kv_cache* cache, const void* q, const void* k, const void* v, void* q_out,
                              const long long* strides, const int32_t* page_table, long long table_stride,
                              int max_pages, const int32_t* seq_lens, const int32_t* cu_seqlens, const float* k_mean,
                              int T, int B, int Hq, sage_dtype dtype, const sage_norm_rope* nr, void* stream) {
  sage_status s = check_dtype(dtype);
  if (s != SAGE_OK) return s;
  HeadRowsParams p;
  memset(&p, 0, sizeof(p));
  if (T < 0 || B < 0 || (!cu_seqlens && T != B)) return SAGE_ERR_INVALID_ARG;
  if ((s = check_strides(strides, 8)) != SAGE_OK) return s;
  if ((s = check_cache(cache, page_table, table_stride, max_pages, B, &p.map)) != SAGE_OK) return s;
  if (q && (!nr || Hq < 1 || Hq > 65535)) return SAGE_ERR_INVALID_ARG;
  if (nr && (s = check_norm_rope(nr, cache->d)) != SAGE_OK) return s;
  if (((uintptr_t)k_mean | (uintptr_t)seq_lens | (uintptr_t)cu_seqlens) & 3) return SAGE_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return SAGE_OK;
  if (!k || !v || !seq_lens || (q && !q_out)) return SAGE_ERR_INVALID_ARG;
  if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_out) & 1) return SAGE_ERR_INVALID_ARG;
  const int d = cache->d, Hkv = cache->Hkv;
  p.B = B, p.N = T, p.d = d, p.vec = d % 8 == 0;
  p.kind[0].in = HeadView{q, 0, strides[0], strides[1]}, p.kind[0].H = q ? Hq : 0;
  p.kind[1].in = HeadView{k, 0, strides[2], strides[3]}, p.kind[1].H = Hkv;
  p.kind[2].in = HeadView{v, 0, strides[4], strides[5]}, p.kind[2].H = Hkv;
  p.kind[0].out = HeadView{q_out, 0, strides[6], strides[7]};
  if ((s = take_views(&p, 1)) != SAGE_OK) return s;
  p.append = 1, p.cu = cu_seqlens, p.seq_lens = seq_lens, p.k_mean = k_mean;
  p.vec_mean = d % 8 == 0 && aligned16(k_mean);
  if (nr) set_norm_rope(&p, *nr);
  const size_t rows = cache_rows(p.map);
  p.x_k8 = extent_of(cache->k8, rows * p.map.dc), p.x_v8 = extent_of(cache->v8, rows * p.map.dc);
  p.x_ks = extent_of(cache->ks, rows * 4), p.x_vs = extent_of(cache->vs, rows * 4);
  if ((s = shape_rows(&p, 1)) != SAGE_OK) return s;
  if ((s = check_device()) != SAGE_OK) return s;
  if ((s = check_apart(p, 1)) != SAGE_OK) return s;
  if (q && overlaps_cache(q_out, view_bytes(p.kind[0].out, 1, T, Hq, d), p.map)) return SAGE_ERR_INVALID_ARG;
  g_serving.store(true);
  return from_cuda(launch_head_rows(p, dtype, static_cast<cudaStream_t>(stream)));
}

sage_status sage_cache_gather(const sage_kv_cache* cache, const int32_t* page_table, long long table_stride,
                              int max_pages, const int32_t* cu_seqlens, const int32_t* starts, const float* k_mean,
                              void* k_out, void* v_out, int T, int B, sage_dtype dtype, void* stream) {
  sage_status s = check_dtype(dtype);
  if (s != SAGE_OK) return s;
  GatherParams p;
  memset(&p, 0, sizeof(p));
  if (T < 0 || B < 0) return SAGE_ERR_INVALID_ARG;
  if ((s = check_cache(cache, page_table, table_stride, max_pages, B, &p.map)) != SAGE_OK) return s;
  if (((uintptr_t)k_mean | (uintptr_t)starts | (uintptr_t)cu_seqlens) & 3) return SAGE_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return SAGE_OK;
  if (!cu_seqlens || !k_out || !v_out || (((uintptr_t)k_out | (uintptr_t)v_out) & 1)) return SAGE_ERR_INVALID_ARG;
  const size_t bytes = (size_t)T * cache->Hkv * cache->d * 2;
  if (overlaps(k_out, bytes, v_out, bytes) || overlaps_cache(k_out, bytes, p.map) || overlaps_cache(v_out, bytes, p.map))
    return SAGE_ERR_INVALID_ARG;
  p.cu = cu_seqlens, p.starts = starts, p.k_mean = k_mean, p.k_out = k_out, p.v_out = v_out;
  p.B = B, p.T = T, p.d = cache->d;
  const int hkv = cache->Hkv;
  if (((long long)T + 15) * hkv > kMaxItems) return SAGE_ERR_INVALID_ARG;
  p.vec = cache->d % 8 == 0 && aligned16(k_out) && aligned16(v_out);
  p.heads_per_group = rows_per_group(p.vec, p.d, (long long)T * ((hkv + 3) / 4));
  p.vec_mean = cache->d % 8 == 0 && aligned16(k_mean);
  p.x_k_out = extent_of(k_out, bytes), p.x_v_out = extent_of(v_out, bytes);
  if ((s = check_device()) != SAGE_OK) return s;
  g_serving.store(true);
  return from_cuda(launch_cache_gather(p, dtype, static_cast<cudaStream_t>(stream)));
}

sage_status sage_attn_decode(const void* q, long long q_batch_stride, long long q_head_stride,
                             const sage_kv_cache* cache, const int32_t* page_table, long long table_stride,
                             int max_pages, const int32_t* seq_lens, void* out, int B, int Hq, int max_seqlen,
                             sage_dtype dtype, float sm_scale, void* stream) {
  sage_status s = check_dtype(dtype);
  if (s != SAGE_OK) return s;
  DecodeParams p;
  memset(&p, 0, sizeof(p));
  const long long strides[2] = {q_batch_stride, q_head_stride};
  if ((s = check_strides(strides, 2)) != SAGE_OK) return s;
  if (B < 0 || B > 65535 || Hq < 1 || Hq > 65535 || max_seqlen < 0) return SAGE_ERR_INVALID_ARG;
  if ((s = check_cache(cache, page_table, table_stride, max_pages, B, &p.map)) != SAGE_OK) return s;
  if (Hq % cache->Hkv != 0) return SAGE_ERR_INVALID_ARG;
  if (B == 0) return SAGE_OK;
  if (!q || !out || !seq_lens || (((uintptr_t)q | (uintptr_t)out) & 1) || ((uintptr_t)seq_lens & 3))
    return SAGE_ERR_INVALID_ARG;
  p.q = HeadView{q, q_batch_stride, 0, q_head_stride};
  const size_t out_bytes = (size_t)B * Hq * cache->d * 2;
  if (overlaps(out, out_bytes, q, view_bytes(p.q, B, 1, Hq, cache->d)) || overlaps_cache(out, out_bytes, p.map))
    return SAGE_ERR_INVALID_ARG;
  p.out = out, p.seq_lens = seq_lens;
  p.B = B, p.Hq = Hq, p.G = Hq / cache->Hkv, p.d = cache->d;
  p.tiles = (p.G + kDecodeHeads - 1) / kDecodeHeads;
  p.pairs = cache->Hkv * p.tiles;
  const long long room = (long long)max_pages << p.map.page_log2;
  p.max_len = (int)std::min<long long>(std::min<long long>(max_seqlen, room), 1 << 30);
  p.scale_log2 = resolve_scale(sm_scale, p.d) * 1.4426950408889634f;
  p.x_out = limited_extent(out, out_bytes);
  if ((s = check_device()) != SAGE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // How the work is cut and shared out (times: Hq32, Hkv8, d128, bf16, calls in a graph).  Sequences of up to 512 keys are not
  // split at all: every pair has a CTA, and there is no join and no workspace.  One sequence: 500 keys 8.7 us, split 9.4;
  // 700 keys 9.4 split, 11.4 not; 16 sequences of 500 8.9 and 12.3, 64 of 500 20.2 and 24.7.  (With many pairs the limit
  // could be higher: 16 sequences of 1000 keys 17.8 us, not split 14.5; 64 of 1000 36.5 and 37.8.)
  // Longer ones go in units of 256 keys, a CTA to each, where those are no more than the CTAs that run at the same time (one
  // of 4000 keys: 10.3 us, in units of 64 10.9, of 512 12.3; four of 2000: 11.6, 13.0, 12.8).  Else that many CTAs
  // share units of 64 keys evenly (64 of 1 to 1000: 25.9 us, of 32 27.4, of 128 27.0).  A pair then counts for as
  // many more units as take the time that a CTA needs to begin and end with it (64 of 1 to 1000, without and with: d 64
  // 44.1 and 21.6 us, d 128 43.6 and 25.9, d 256 62.2 and 41.5; 64 of 1 to 16384: 150 and 138, 212 and 208, 401 and 387; 4 to
  // 8 units are within 9% of these).
  // All of it goes by max_seqlen, since the lengths are on the device: 16 sequences of 200 keys take 12.1 us under a bound of
  // 4096, and 6.0 not split.
  const long long most = 148LL * decode_ctas_per_sm(p.d);
  const auto units = [&] {
    const long long keys = std::max<long long>(1, ((long long)p.max_len + (1 << p.unit_log2) - 1) >> p.unit_log2);
    return (long long)B * p.pairs * (keys + p.unit_extra);
  };
  p.unit_extra = 0, p.unit_log2 = p.max_len <= 512 ? 9 : 8;
  if (p.unit_log2 == 8 && units() > most) p.unit_extra = p.d <= 64 ? 8 : p.d <= 128 ? 6 : 4, p.unit_log2 = 6;
  while (units() >= (1LL << 31) && p.unit_log2 < 30) ++p.unit_log2;
  if (p.max_len <= 1 << p.unit_log2) p.unit_extra = 0;  // one unit to every pair: nothing is shared out
  if (units() >= (1LL << 31)) return SAGE_ERR_INVALID_ARG;
  const bool split = p.max_len > 1 << p.unit_log2;  // a pair may cross CTAs
  p.ctas = (uint32_t)(split ? std::min<long long>(units(), most) : units());
  unsigned char* ws = nullptr;
  if (split) {
    const size_t parts = (size_t)p.ctas * 2 * kDecodeHeads;
    const size_t ml = align_up(parts * 8), total = ml + parts * p.map.dc * 4;
    const cudaError_t e = workspace_alloc(reinterpret_cast<void**>(&ws), total, st);
    if (e != cudaSuccess) return from_cuda(e);
    p.part_ml = reinterpret_cast<float*>(ws), p.part_o = reinterpret_cast<float*>(ws + ml);
    p.x_part_ml = extent_of(p.part_ml, parts * 8), p.x_part_o = extent_of(p.part_o, parts * p.map.dc * 4);
  }
  g_serving.store(true);
  s = from_cuda(launch_decode(p, dtype, st));
  if (ws) {
    const cudaError_t ef = cudaFreeAsync(ws, st);
    if (s == SAGE_OK && ef != cudaSuccess) s = from_cuda(ef);
  }
  return s;
}

}  // extern "C"

// ------------------------------------------------------------------------------------------------
// Allocation-free entry point: the workspace is a static device array in this library.
// ------------------------------------------------------------------------------------------------
static __device__ __align__(256) unsigned char g_noalloc_scratch[SAGE_NOALLOC_MAX_BYTES];

namespace {

// The array's device address, looked up once per device with that device current.
cudaError_t noalloc_scratch(int dev, unsigned char** out) {
  constexpr int kMaxDevices = 128;
  static std::mutex mu;
  static unsigned char* addr[kMaxDevices] = {};
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!addr[dev]) {
    void* p = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&p, g_noalloc_scratch);
    if (e != cudaSuccess) return e;
    addr[dev] = static_cast<unsigned char*>(p);
  }
  *out = addr[dev];
  return cudaSuccess;
}

}  // namespace

extern "C" sage_status sage_attn_noalloc(const void* q, const void* k, const void* v, void* out, int B, int Hq,
                                         int Hkv, int N, int d, sage_dtype dtype, sage_layout layout, int is_causal,
                                         float sm_scale, sage_pv_mode pv_mode, void* stream) {
  sage_status s = check_common(q, k, v, dtype, layout, pv_mode);
  if (s != SAGE_OK) return s;
  Dims m;
  if ((s = check_dims(B, Hq, Hkv, N, N, d, &m)) != SAGE_OK) return s;
  if (!out || out_overlaps(m, q, k, v, out)) return SAGE_ERR_INVALID_ARG;
  const Opts o;  // defaults
  const WsLayout w = ws_layout(m, pv_mode, o);
  if (w.total > (size_t)SAGE_NOALLOC_MAX_BYTES) return SAGE_ERR_INVALID_ARG;
  if ((s = check_device()) != SAGE_OK) return s;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SAGE_ERR_CUDA;
  unsigned char* ws = nullptr;
  if (noalloc_scratch(dev, &ws) != cudaSuccess) return SAGE_ERR_CUDA;
  return attend_on(m, ws, q, k, v, out, nullptr, nullptr, dtype, layout, is_causal ? 1 : 0, sm_scale, pv_mode, o,
                   static_cast<cudaStream_t>(stream));
}
