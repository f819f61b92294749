// Block quantisation of rows (a scale for each 128 elements) and of matrices (for
// each 128 x 128), and back: value = code scale, code = E4M3(x / scale), scale =
// amax / 448.
//
// One pass each. Rows: a half-warp takes a block of 128, eight elements a lane, so
// that its amax is four shuffles and its codes one 8-byte store a lane; a CTA takes
// pieces of the segments in turn (kElements of them: enough that finding the piece's
// segment costs nothing, few enough that small batches fill the GPU) and has kUnroll
// blocks of each half-warp on their way at once. 124518 x 2048 bf16: 139 us, 5.5 TB/s
// (two blocks on their way: 158 to 166), with two thirds of the issue slots busy; f32 201,
// 6.3 TB/s. Back: 125 us to bf16, 239 to f32. 8192 x 512 and 128 x 7168: 6 to 7 us, the call.
// Matrices: a CTA keeps a whole 128 x 128 in registers between its amax and its codes.
// 32 of 4096 x 4096 bf16: 271 us, 5.9 TB/s, f32 403, 6.7; bound by HBM.
#include <climits>
#include <cstring>
#include <new>

#include "ep_header.cuh"
#include "ep_launch.cuh"
#include "ep_pieces.cuh"
#include "ep_quant.cuh"
#include "ep_qlinear.cuh"
#include "ep_segments.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kHalves = kThreads / 16;
constexpr int kElements = 1 << 15;   // of a piece, at most
constexpr int kUnroll = 4;

struct QuantParams {
  LinearSegs s;
  int K, Kb;
  int64_t rows;          // of a matrix (scales of 128 rows)
  int row_blocks;        // its scale rows; 0: a scale row for each row
  int per;               // rows of a piece
  const void* x;
  uint8_t* codes;
  float* scales;
  void* out;             // dequantised
};

// The blocks of a piece that a half-warp takes, kHalves apart, without divisions: where
// rows are whole blocks (FLAT) they are one after another in memory.
template <bool FLAT>
struct Walk {
  int row, block, drow, dblock, Kb, n;
  __device__ __forceinline__ Walk(int half, int blocks) : Kb(blocks), n(half) {
    if (FLAT) return;
    row = half / Kb;
    block = half - row * Kb;
    drow = kHalves / Kb;
    dblock = kHalves - drow * Kb;
  }
  __device__ __forceinline__ void next() {
    n += kHalves;
    if (FLAT) return;
    row += drow;
    block += dblock;
    if (block >= Kb) {
      block -= Kb;
      ++row;
    }
  }
  // whether there is such a block of a piece of `all` blocks, whether this lane's part of
  // it is in, and where, counted from the piece
  __device__ __forceinline__ bool place(int all, int K, int sub, bool& in, int64_t& at) const {
    const bool there = n < all;
    if (FLAT) {
      in = there;
      at = (int64_t)n * 128 + sub * 8;
    } else {
      in = there && block * 128 + sub * 8 < K;
      at = (int64_t)row * K + block * 128 + sub * 8;
    }
    return there;
  }
};

// Every half-warp goes through the same number of steps, with blocks past the end of
// the piece left out: the shuffles are the whole warp's.
template <typename T, bool FLAT>
__global__ void __launch_bounds__(kThreads) quant_rows_kernel(QuantParams p) {
  extern __shared__ int table[];
  begin_overlapped();
  const int pieces = segment_table(p.s, p.per, table);
  const int half = threadIdx.x >> 4, sub = threadIdx.x & 15;
  for (int i = blockIdx.x; i < pieces; i += gridDim.x) {
    const Piece piece = piece_at(p.s, p.per, table, i);
    const int all = piece.rows * p.Kb;
    const T* x = static_cast<const T*>(p.x) + piece.row * p.K;
    uint8_t* codes = p.codes + piece.row * p.K;
    float* scales = p.scales + piece.row * p.Kb;
    Walk<FLAT> w(half, p.Kb);
    for (int step = 0; step < all; step += kUnroll * kHalves) {
      Raw8<T> raw[kUnroll];
      int64_t at[kUnroll];
      bool in[kUnroll], there[kUnroll];
      const int first = w.n;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u, w.next()) {
        there[u] = w.place(all, p.K, sub, in[u], at[u]);
        zero8(raw[u]);
        if (in[u]) load8<T>(x, at[u], raw[u]);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float f[8];
        floats8(raw[u], f);
        const float amax = max16(amax8(f));
        const float scale = scale_of(amax);
        const uint2 q = e4m3x8(f, block_scale(amax, scale));
        if (in[u]) *reinterpret_cast<uint2*>(codes + at[u]) = q;
        if (sub == 0 && there[u]) scales[first + u * kHalves] = scale;
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) dequant_rows_kernel(QuantParams p) {
  extern __shared__ int table[];
  begin_overlapped();
  const int pieces = segment_table(p.s, p.per, table);
  const int half = threadIdx.x >> 4, sub = threadIdx.x & 15;
  T* out = static_cast<T*>(p.out);
  for (int i = blockIdx.x; i < pieces; i += gridDim.x) {
    const Piece at = piece_at(p.s, p.per, table, i);
    const int steps = (at.rows * p.Kb + kHalves - 1) / kHalves;
    Walk<false> w(half, p.Kb);
    for (int step = 0; step < steps; step += kUnroll) {
      uint2 q[kUnroll];
      float scale[kUnroll];
      int64_t to[kUnroll];
      bool in[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u, w.next()) {
        const int col = w.block * 128 + sub * 8;
        in[u] = w.row < at.rows && col < p.K;
        const int64_t row = at.row + w.row;
        to[u] = row * p.K + col;
        q[u] = make_uint2(0, 0);
        scale[u] = 0.0f;
        if (in[u]) {
          q[u] = *reinterpret_cast<const uint2*>(p.codes + to[u]);
          int64_t scale_row = row;
          if (p.row_blocks) {
            const int64_t g = row / p.rows;
            scale_row = g * p.row_blocks + (row - g * p.rows) / 128;
          }
          scale[u] = p.scales[scale_row * p.Kb + w.block];
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float f[8];
        e4m3x8_values(q[u], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= scale[u];
        if (in[u]) store8<T>(out, to[u], f);
      }
    }
  }
}

// A CTA's 128 x 128: half-warp h has rows h, h + 16, ...
template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2) quant_tiles_kernel(QuantParams p) {
  begin_overlapped();
  __shared__ float most[kThreads / 32];
  constexpr int kRows = 128 / kHalves;
  const int half = threadIdx.x >> 4, sub = threadIdx.x & 15;
  int64_t tile = blockIdx.x;
  const int kb = (int)(tile % p.Kb);
  tile /= p.Kb;
  const int rb = (int)(tile % p.row_blocks);
  const int64_t g = tile / p.row_blocks;
  const int col = kb * 128 + sub * 8;
  const int64_t row0 = (int64_t)rb * 128 + half;
  const int64_t base = (g * p.rows + row0) * p.K + col;
  const T* x = static_cast<const T*>(p.x) + base;
  Raw8<T> raw[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    zero8(raw[i]);
    if (col < p.K && row0 + i * kHalves < p.rows) load8<T>(x, (int64_t)i * kHalves * p.K, raw[i]);
  }
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    float f[8];
    floats8(raw[i], f);
    amax = fmaxf(amax, amax8(f));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
  if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, most[w]);
  const float scale = scale_of(amax);
  const BlockScale by = block_scale(amax, scale);
  uint8_t* codes = p.codes + base;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    float f[8];
    floats8(raw[i], f);
    const uint2 q = e4m3x8(f, by);
    if (col < p.K && row0 + i * kHalves < p.rows)
      *reinterpret_cast<uint2*>(codes + (int64_t)i * kHalves * p.K) = q;
  }
  if (threadIdx.x == 0) p.scales[(g * p.row_blocks + rb) * p.Kb + kb] = scale;
}

template <typename T>
cudaError_t launch_rows(QuantParams& p, bool back, int64_t rows, int sms, cudaStream_t st) {
  // as many rows as kElements hold, fewer where that leaves SMs without a piece
  int64_t per = kElements / p.K;
  const int64_t most = rows / (2 * sms);
  if (per > most) per = most;
  p.per = per < 1 ? 1 : (int)per;
  int64_t grid = rows / p.per + p.s.G;
  if (grid > (int64_t)sms * 8) grid = (int64_t)sms * 8;
  const auto kernel = back ? dequant_rows_kernel<T> : p.K % 128 == 0 ? quant_rows_kernel<T, true> : quant_rows_kernel<T, false>;
  return launch_overlapped(kernel, dim3((unsigned)grid), kThreads, segment_bytes(p.s.G), st, p);
}

}  // namespace

cudaError_t launch_dequantize(const LinearSegs& s, const uint8_t* codes, const float* scales, int K,
                              __nv_bfloat16* out, int sms, cudaStream_t st) {
  QuantParams p;
  memset(&p, 0, sizeof(p));
  p.s = s;
  p.K = K;
  p.Kb = (K + 127) / 128;
  p.codes = const_cast<uint8_t*>(codes);
  p.scales = const_cast<float*>(scales);
  p.out = out;
  return launch_rows<__nv_bfloat16>(p, true, s.begin ? s.pool : s.dense_rows, sms, st);
}

}  // namespace ep

struct ep_quant_handle {
  ep_quant_config cfg;
  ep::Header header;
  int32_t* err;
  int sm_count;
};

namespace {

using namespace ep;

ep_status qfail(ep_status st, const char* msg) { return record_error(st, msg); }
ep_status qcuda(cudaError_t e) { return record_error(EP_ERR_CUDA, cudaGetErrorString(e)); }

ep_status plan_quant(const ep_quant_config* c) {
  if (!c) return qfail(EP_ERR_INVALID_ARG, "quant config is NULL");
  if (c->block_rows != 1 && c->block_rows != 128)
    return qfail(EP_ERR_INVALID_ARG, "block_rows must be 1 or 128");
  const bool tiles = c->block_rows == 128;
  if (c->num_groups < 1 || c->num_groups > (tiles ? 2 : 1) * EP_MAX_EXPERTS)
    return qfail(EP_ERR_INVALID_ARG, "num_groups outside [1, 1024] (matrices: 2048)");
  if (c->groups_per_base < 0)
    return qfail(EP_ERR_INVALID_ARG, "groups_per_base must be >= 0");
  if (c->features < 16 || c->features % 16 != 0 || c->features > (1 << 22))
    return qfail(EP_ERR_INVALID_ARG, "features must be a positive multiple of 16 up to 2^22");
  if (c->max_rows < 1 || c->max_rows > INT32_MAX - 1024)
    return qfail(EP_ERR_INVALID_ARG, "max_rows must be >= 1 and fit int32");
  if (c->dtype != EP_DTYPE_BF16 && c->dtype != EP_DTYPE_FP32)
    return qfail(EP_ERR_INVALID_ARG, "dtype must be BF16 or FP32");
  const int64_t rows = c->max_rows * (tiles ? c->num_groups : 1);
  if (rows > INT32_MAX - 1024 ||
      (tiles && (int64_t)c->num_groups * ((c->max_rows + 127) / 128) * ((c->features + 127) / 128) > INT32_MAX))
    return qfail(EP_ERR_INVALID_ARG, "num_groups, max_rows and features give too many rows or tiles");
  return EP_OK;
}

ep_status fill_quant(ep_quant_handle* h, const void* x, const int32_t* row_begin,
                     const int32_t* row_count, const int32_t* row_base, int64_t num_rows,
                     const void* codes, const float* scales, QuantParams* p) {
  if (!h) return qfail(EP_ERR_INVALID_ARG, "quant handle is NULL");
  const ep_quant_config& c = h->cfg;
  const bool tiles = c.block_rows == 128;
  if (!x || !codes || !scales || (uintptr_t)x % 16 != 0 || (uintptr_t)codes % 16 != 0 ||
      (uintptr_t)scales % 4 != 0)
    return qfail(EP_ERR_INVALID_ARG, "x, codes and scales must be given, 16-byte (scales 4-byte) aligned");
  if ((row_begin == nullptr) != (row_count == nullptr))
    return qfail(EP_ERR_INVALID_ARG, "give row_begin and row_count together, or neither");
  if (((uintptr_t)row_begin | (uintptr_t)row_count | (uintptr_t)row_base) % 4 != 0)
    return qfail(EP_ERR_INVALID_ARG, "row_begin, row_count or row_base is misaligned");
  if (tiles && (row_begin || row_base || num_rows != c.max_rows))
    return qfail(EP_ERR_INVALID_ARG, "blocks of 128 rows take whole matrices: no segments, num_rows = max_rows");
  if (!tiles && !row_begin && (c.num_groups != 1 || num_rows < 0 || num_rows > c.max_rows))
    return qfail(EP_ERR_INVALID_ARG,
                 "several groups need row_begin and row_count; num_rows must be in [0, max_rows]");
  if (row_base && (!row_begin || c.groups_per_base < 1))
    return qfail(EP_ERR_INVALID_ARG, "row_base needs row_begin and groups_per_base");
  memset(p, 0, sizeof(*p));
  p->s.G = tiles ? 1 : c.num_groups;
  p->s.per_base = c.groups_per_base > 0 ? c.groups_per_base : 1;
  p->s.pool = c.max_rows * (tiles ? c.num_groups : 1);
  p->s.dense_rows = tiles ? p->s.pool : num_rows;
  p->s.begin = row_begin;
  p->s.count = row_count;
  p->s.base = row_base;
  p->s.err = h->err;
  p->K = c.features;
  p->Kb = (c.features + 127) / 128;
  p->rows = c.max_rows;
  p->row_blocks = tiles ? (int)((c.max_rows + 127) / 128) : 0;
  p->codes = static_cast<uint8_t*>(const_cast<void*>(codes));
  p->scales = const_cast<float*>(scales);
  return EP_OK;
}

ep_status quant_ready(ep_quant_handle* h, cudaStream_t st) {
  if (h->sm_count == 0) {
    int dev = 0, n = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return qcuda(e);
    h->sm_count = n;
  }
  const cudaError_t e = header_ready(&h->header, st);
  return e == cudaSuccess ? EP_OK : qcuda(e);
}

}  // namespace

extern "C" size_t ep_quant_workspace_size(const ep_quant_config* cfg) {
  return plan_quant(cfg) == EP_OK ? kHeaderBytes : 0;
}

extern "C" ep_status ep_quant_create(const ep_quant_config* cfg, void* d_workspace,
                                     size_t workspace_bytes, ep_quant_handle** out_handle) {
  if (!out_handle) return qfail(EP_ERR_INVALID_ARG, "out_handle is NULL");
  *out_handle = nullptr;
  const ep_status s = plan_quant(cfg);
  if (s != EP_OK) return s;
  if (!d_workspace || (uintptr_t)d_workspace % 256 != 0)
    return qfail(EP_ERR_WORKSPACE, "quant workspace is NULL or not 256-byte aligned");
  if (workspace_bytes < kHeaderBytes) return qfail(EP_ERR_WORKSPACE, "quant workspace too small");
  ep_quant_handle* p = new (std::nothrow) ep_quant_handle{};
  if (!p) return qfail(EP_ERR_INVALID_ARG, "out of host memory");
  p->cfg = *cfg;
  p->err = static_cast<int32_t*>(d_workspace);
  open_header(&p->header, d_workspace);
  *out_handle = p;
  return EP_OK;
}

extern "C" void ep_quant_destroy(ep_quant_handle* h) { delete h; }

extern "C" ep_status ep_quantize(ep_quant_handle* h, const void* x, const int32_t* row_begin,
                                 const int32_t* row_count, const int32_t* row_base,
                                 int64_t num_rows, void* codes, float* scales, void* stream) {
  QuantParams p;
  ep_status s = fill_quant(h, x, row_begin, row_count, row_base, num_rows, codes, scales, &p);
  if (s != EP_OK) return s;
  p.x = x;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((s = quant_ready(h, st)) != EP_OK) return s;
  const bool f32 = h->cfg.dtype == EP_DTYPE_FP32;
  cudaError_t e = cudaSuccess;
  if (p.row_blocks) {
    const dim3 grid((unsigned)((int64_t)h->cfg.num_groups * p.row_blocks * p.Kb));
    e = f32 ? launch_overlapped(quant_tiles_kernel<float>, grid, kThreads, 0, st, p)
            : launch_overlapped(quant_tiles_kernel<__nv_bfloat16>, grid, kThreads, 0, st, p);
  } else {
    const int64_t rows = row_begin ? p.s.pool : num_rows;
    if (rows == 0) return EP_OK;
    e = f32 ? launch_rows<float>(p, false, rows, h->sm_count, st)
            : launch_rows<__nv_bfloat16>(p, false, rows, h->sm_count, st);
  }
  return e == cudaSuccess ? EP_OK : qcuda(e);
}

extern "C" ep_status ep_dequantize(ep_quant_handle* h, const void* codes, const float* scales,
                                   const int32_t* row_begin, const int32_t* row_count,
                                   const int32_t* row_base, int64_t num_rows, void* x,
                                   void* stream) {
  QuantParams p;
  ep_status s = fill_quant(h, x, row_begin, row_count, row_base, num_rows, codes, scales, &p);
  if (s != EP_OK) return s;
  p.out = x;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((s = quant_ready(h, st)) != EP_OK) return s;
  const int64_t rows = row_begin ? p.s.pool : p.s.dense_rows;
  if (rows == 0) return EP_OK;
  const cudaError_t e = h->cfg.dtype == EP_DTYPE_FP32
                            ? launch_rows<float>(p, true, rows, h->sm_count, st)
                            : launch_rows<__nv_bfloat16>(p, true, rows, h->sm_count, st);
  return e == cudaSuccess ? EP_OK : qcuda(e);
}

extern "C" ep_status ep_quant_sync(ep_quant_handle* h, void* stream) {
  if (!h) return qfail(EP_ERR_INVALID_ARG, "quant handle is NULL");
  uint32_t bits = 0;
  const cudaError_t e = header_report(&h->header, static_cast<cudaStream_t>(stream), &bits);
  if (e != cudaSuccess) return qcuda(e);
  if (bits & kErrSegment)
    return qfail(EP_ERR_INVALID_INDEX, "a segment reached outside the row pool and was cut, or segments overlapped so much that the "
                 "call did nothing");
  return EP_OK;
}
