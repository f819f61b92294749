// Host library of the experts' products, y = act(x W^T + b) + residual over
// the segments of a row pool (the packed layout's, one per expert, or one
// dense product), and the elementwise kernels of the backward pass. The
// products themselves are in ep_linear_mma.cu.
#include <climits>
#include <cstring>
#include <new>

#include "ep_header.cuh"
#include "ep_launch.cuh"
#include "ep_linear.cuh"

namespace ep {
namespace {

// dz = dy act'(z) and the sums of dz's columns over each block of rows: one
// pass, bound by HBM (124,518 rows, 2 x 2048 columns, SwiGLU: 2.55 GB in 398 us,
// 6.4 TB/s). A CTA takes kGradRows rows of one group, a thread VEC neighbouring
// columns of every `lanes`th row, so that a warp's access is contiguous; the
// blocks' sums go to `part` and are added in block order by bias_grad_kernel. dz is rounded to bf16 because the products read
// it as a tensor-core operand; the sums are of the unrounded values.
constexpr int kGradRows = 64;
constexpr int kGradThreads = 256;

struct GradParams {
  LinearParams p;
  __nv_bfloat16* dz;         // NULL: only the sums
  float* part;               // [row blocks][Nw] or NULL
  int64_t row_blocks;        // rows of `part`
  int lanes;                 // threads that share a column: 1, 2, 4 or 8
  float* db;                 // [G][Nw]
};

__device__ __forceinline__ int64_t blocks_of(int64_t count) {
  return (count + kGradRows - 1) / kGradRows;
}

// VEC columns from an aligned place, as f32.
template <int VEC, typename T>
__device__ __forceinline__ void load_columns(const T* at, float (&v)[VEC]) {
  if (VEC == 8 && sizeof(T) == 2) {
    const uint4 q = ld_once_v4(at);
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = (i & 1) ? bf16_hi(u[i / 2]) : bf16_lo(u[i / 2]);
  } else if (VEC == 8) {
#pragma unroll
    for (int h = 0; h < VEC / 4; ++h) {
      const uint4 q = ld_once_v4(at + h * 4);
      v[(h * 4) % VEC] = __uint_as_float(q.x);
      v[(h * 4 + 1) % VEC] = __uint_as_float(q.y);
      v[(h * 4 + 2) % VEC] = __uint_as_float(q.z);
      v[(h * 4 + 3) % VEC] = __uint_as_float(q.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = (float)at[i];
  }
}

template <int VEC>
__device__ __forceinline__ void store_dz(__nv_bfloat16* at, const float (&v)[VEC]) {
  if (VEC == 8) {
    st_v4(at, make_uint4(cvt_bf16x2(v[0], v[1 % VEC]), cvt_bf16x2(v[2 % VEC], v[3 % VEC]),
                         cvt_bf16x2(v[4 % VEC], v[5 % VEC]), cvt_bf16x2(v[6 % VEC], v[7 % VEC])));
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) at[i] = __float2bfloat16_rn(v[i]);
  }
}

// A group's block of rows, number `b` over all groups; false past the last.
struct BlockPlace {
  int64_t begin, row0, row1;
};

template <int VEC, int ACT, typename T>
__global__ void __launch_bounds__(kGradThreads) act_grad_kernel(GradParams q) {
  begin_overlapped();
  const LinearParams& p = q.p;
  __shared__ BlockPlace at;
  const bool gated = ACT == EP_ACT_SWIGLU;
  const int64_t block = blockIdx.x;
  // the group of this block: a warp adds up the groups' blocks, 32 at a time
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int64_t before = 0;
    if (lane == 0) at.row0 = at.row1 = at.begin = 0;
    __syncwarp();
    for (int g0 = 0; g0 < p.s.G && before <= block; g0 += 32) {
      int64_t begin = 0, count = 0;
      if (g0 + lane < p.s.G) segment_of(p.s, g0 + lane, begin, count);
      int64_t incl = blocks_of(count);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += v;
      }
      const int64_t mine = before + incl - blocks_of(count);
      if (block >= mine && block < before + incl) {
        at.begin = begin;
        at.row0 = (block - mine) * kGradRows;
        at.row1 = min(count, at.row0 + kGradRows);
      }
      before += __shfl_sync(kFull, incl, 31);
    }
    // segments that do not overlap leave the last block free
    if (p.s.begin && lane == 0 && block == q.row_blocks - 1 && before > block)
      atomicOr(p.s.err, kErrSegment);
  }
  __syncthreads();
  const int wide = kGradThreads / q.lanes;      // threads beside each other in a row
  const int lane_row = threadIdx.x / wide, tx = threadIdx.x - lane_row * wide;
  const int c = (blockIdx.y * wide + tx) * VEC;
  if (at.row0 >= at.row1) return;
  const bool in = c < p.N;
  float s0[VEC], s1[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) s0[i] = s1[i] = 0.0f;
  const int64_t row0 = at.row0 + lane_row;
  const T* dy = static_cast<const T*>(p.dy) + (at.begin + row0) * p.N + c;
  const __nv_bfloat16* z = p.z + (at.begin + row0) * p.Nw + c;
  __nv_bfloat16* out = q.dz + (at.begin + row0) * p.ldz + c;
#pragma unroll 4
  for (int64_t r = row0; r < (in ? at.row1 : 0); r += q.lanes) {
    float d0[VEC], d1[VEC];
    load_columns<VEC, T>(dy, d0);
    if (gated) {
      float zg[VEC], zu[VEC];
      load_columns<VEC, __nv_bfloat16>(z, zg);
      load_columns<VEC, __nv_bfloat16>(z + p.N, zu);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        // silu'(g) = s (1 + g (1 - s)), silu(g) = g s
        const float s = sigmoid_of(zg[i]);
        d1[i] = d0[i] * (zg[i] * s);
        d0[i] *= zu[i] * (s * (1.0f + zg[i] * (1.0f - s)));
      }
    } else if (ACT != EP_ACT_NONE) {
      float zv[VEC];
      load_columns<VEC, __nv_bfloat16>(z, zv);
#pragma unroll
      for (int i = 0; i < VEC; ++i) d0[i] *= slope_of(ACT, zv[i]);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      s0[i] += d0[i];
      if (gated) s1[i] += d1[i];
    }
    if (q.dz) {
      store_dz<VEC>(out, d0);
      if (gated) store_dz<VEC>(out + p.N, d1);
    }
    dy += (int64_t)q.lanes * p.N;
    z += (int64_t)q.lanes * p.Nw;
    out += (int64_t)q.lanes * p.ldz;
  }
  if (q.part && q.lanes > 1) {   // the first of the threads that share a column adds the others' sums
    __shared__ float sums[2][kGradThreads * VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      sums[0][threadIdx.x * VEC + i] = s0[i];
      if (gated) sums[1][threadIdx.x * VEC + i] = s1[i];
    }
    __syncthreads();
    if (lane_row == 0)
      for (int l = 1; l < q.lanes; ++l)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          s0[i] += sums[0][(l * wide + tx) * VEC + i];
          if (gated) s1[i] += sums[1][(l * wide + tx) * VEC + i];
        }
  }
  if (q.part && in && lane_row == 0) {
    float* part = q.part + block * p.Nw + c;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      part[i] = s0[i];
      if (gated) part[p.N + i] = s1[i];
    }
  }
}

// db_g: the sums of the group's blocks, in block order. A CTA takes 32
// columns, a warp every 8th block.
__global__ void __launch_bounds__(256) bias_grad_kernel(GradParams q) {
  begin_overlapped();
  const LinearParams& p = q.p;
  __shared__ float sum[8][32];
  __shared__ int64_t range[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const int g = blockIdx.y;
  if (warp == 0) {
    int64_t before = 0, begin, count = 0;
    for (int i = lane; i < g; i += 32) {
      segment_of(p.s, i, begin, count);
      before += blocks_of(count);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) before += __shfl_xor_sync(kFull, before, o);
    segment_of(p.s, g, begin, count);
    if (lane == 0) {
      range[0] = min(before, q.row_blocks);
      range[1] = min(before + blocks_of(count), q.row_blocks);
    }
  }
  __syncthreads();
  float s = 0.0f;
  if (c < p.Nw)
    for (int64_t b = range[0] + warp; b < range[1]; b += 8) s += q.part[b * p.Nw + c];
  sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < p.Nw) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += sum[w][lane];
    q.db[(int64_t)g * p.Nw + c] = s;
  }
}

template <int VEC, typename T>
cudaError_t grad_typed(GradParams q, cudaStream_t st) {
  // rows too short for a CTA's threads: several of them share a column
  q.lanes = 1;
  while (q.lanes < 8 && q.p.N * q.lanes * 2 <= kGradThreads * VEC) q.lanes *= 2;
  const int wide = kGradThreads / q.lanes;
  const dim3 grid((unsigned)q.row_blocks, (q.p.N + wide * VEC - 1) / (wide * VEC));
  auto kernel = act_grad_kernel<VEC, EP_ACT_NONE, T>;
  switch (q.p.act) {
    case EP_ACT_RELU: kernel = act_grad_kernel<VEC, EP_ACT_RELU, T>; break;
    case EP_ACT_SILU: kernel = act_grad_kernel<VEC, EP_ACT_SILU, T>; break;
    case EP_ACT_GELU: kernel = act_grad_kernel<VEC, EP_ACT_GELU, T>; break;
    case EP_ACT_SWIGLU: kernel = act_grad_kernel<VEC, EP_ACT_SWIGLU, T>; break;
  }
  return launch_overlapped(kernel, grid, kGradThreads, 0, st, q);
}

cudaError_t launch_act_grad(const GradParams& q, cudaStream_t st) {
  const LinearParams& p = q.p;
  // 16-byte accesses need rows and tensors on 16-byte boundaries
  const bool vec = p.N % 8 == 0 && (uintptr_t)p.dy % 16 == 0 && (uintptr_t)p.z % 16 == 0;
  if (p.y_f32) return vec ? grad_typed<8, float>(q, st) : grad_typed<1, float>(q, st);
  return vec ? grad_typed<8, __nv_bfloat16>(q, st) : grad_typed<1, __nv_bfloat16>(q, st);
}

}  // namespace
}  // namespace ep

struct ep_linear_handle {
  ep_linear_config cfg;
  uint8_t* ws;
  ep::Header header;
  int sm_count;
  int Nw;
  int64_t ldz, row_blocks;
  int32_t* err;
  unsigned int* tickets;
  float* partial;
  __nv_bfloat16* dz;
  float* part;
  size_t bytes;
};

namespace {

using namespace ep;

ep_status lfail(ep_status st, const char* msg) { return record_error(st, msg); }
ep_status lcuda(cudaError_t e) { return record_error(EP_ERR_CUDA, cudaGetErrorString(e)); }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

static_assert(kTicketOffset + kLinearMaxPairs * 2 * sizeof(unsigned int) <= kHeaderBytes, "tickets");

ep_status plan_linear(const ep_linear_config* c, ep_linear_handle* h) {
  if (!c) return lfail(EP_ERR_INVALID_ARG, "linear config is NULL");
  if (c->num_groups < 1 || c->num_groups > EP_MAX_EXPERTS)
    return lfail(EP_ERR_INVALID_ARG, "num_groups outside [1, 1024]");
  if (c->groups_per_base < 0)
    return lfail(EP_ERR_INVALID_ARG, "groups_per_base must be >= 0");
  if (c->in_features < 8 || c->in_features % 8 != 0)
    return lfail(EP_ERR_INVALID_ARG, "in_features must be a positive multiple of 8");
  if (c->out_features < 1 || c->out_features > (1 << 22) || c->in_features > (1 << 22))
    return lfail(EP_ERR_INVALID_ARG, "in_features and out_features must be in [1, 2^22]");
  if (c->max_rows < 1 || c->max_rows > INT32_MAX - 1024)
    return lfail(EP_ERR_INVALID_ARG, "max_rows must be >= 1 and fit int32");
  if (c->out_dtype != EP_DTYPE_BF16 && c->out_dtype != EP_DTYPE_FP32)
    return lfail(EP_ERR_INVALID_ARG, "out_dtype must be BF16 or FP32");
  if (c->weight_grad_dtype != EP_DTYPE_BF16 && c->weight_grad_dtype != EP_DTYPE_FP32)
    return lfail(EP_ERR_INVALID_ARG, "weight_grad_dtype must be BF16 or FP32");
  if (c->activation < EP_ACT_NONE || c->activation > EP_ACT_SWIGLU)
    return lfail(EP_ERR_INVALID_ARG, "unknown activation");
  // tiles are numbered in int32: at most one per 32 rows (and group) and 256 features
  const int64_t wide = (2 * (int64_t)c->out_features > c->in_features ? 2 * (int64_t)c->out_features
                                                                      : c->in_features) / 256 + 1;
  if ((c->max_rows / 32 + c->num_groups) * wide > INT32_MAX ||
      (int64_t)c->num_groups * wide * (c->in_features / 256 + 1) > INT32_MAX)
    return lfail(EP_ERR_INVALID_ARG, "max_rows, num_groups and features give too many tiles");
  h->cfg = *c;
  h->Nw = c->activation == EP_ACT_SWIGLU ? 2 * c->out_features : c->out_features;
  h->ldz = (h->Nw + 63) / 64 * 64;   // whole 64-element blocks
  h->row_blocks = (c->max_rows + kGradRows - 1) / kGradRows + c->num_groups;
  size_t off = kHeaderBytes;
  h->err = reinterpret_cast<int32_t*>(h->ws);
  h->tickets = reinterpret_cast<unsigned int*>(h->ws ? h->ws + kTicketOffset : nullptr);
  h->partial = reinterpret_cast<float*>(h->ws ? h->ws + off : nullptr);
  int64_t terms = c->in_features;
  if (c->backward && h->Nw > terms) terms = h->Nw;
  if (c->backward && c->max_rows > terms) terms = c->max_rows;
  off += kLinearMaxPairs * (terms > kLongTerms ? kPartBytesLong : c->backward ? kPartBytesGrad : kPartBytes);
  h->dz = nullptr;
  h->part = nullptr;
  if (c->backward) {
    h->dz = reinterpret_cast<__nv_bfloat16*>(h->ws ? h->ws + off : nullptr);
    off += up256((size_t)c->max_rows * h->ldz * 2);
    h->part = reinterpret_cast<float*>(h->ws ? h->ws + off : nullptr);
    off += up256((size_t)h->row_blocks * h->Nw * 4);
  }
  h->bytes = off;
  return EP_OK;
}

ep_status linear_ready(ep_linear_handle* h, cudaStream_t st) {
  if (h->sm_count == 0) {
    int dev = 0, n = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return lcuda(e);
    h->sm_count = n;
  }
  const cudaError_t e = header_ready(&h->header, st);
  return e == cudaSuccess ? EP_OK : lcuda(e);
}

ep_status fill_linear(const ep_linear_handle* h, const void* x, const void* w,
                      const int32_t* row_begin, const int32_t* row_count,
                      const int32_t* row_base, int64_t num_rows, LinearParams* p) {
  const ep_linear_config& c = h->cfg;
  memset(p, 0, sizeof(*p));
  if (!x || !w || (uintptr_t)x % 16 != 0 || (uintptr_t)w % 16 != 0)
    return lfail(EP_ERR_INVALID_ARG, "x and weight must be given, 16-byte aligned");
  if ((row_begin == nullptr) != (row_count == nullptr))
    return lfail(EP_ERR_INVALID_ARG, "give row_begin and row_count together, or neither");
  if (((uintptr_t)row_begin | (uintptr_t)row_count | (uintptr_t)row_base) % 4 != 0)
    return lfail(EP_ERR_INVALID_ARG, "row_begin, row_count or row_base is misaligned");
  if (!row_begin) {
    if (c.num_groups != 1)
      return lfail(EP_ERR_INVALID_ARG, "several groups need row_begin and row_count");
    if (num_rows < 0 || num_rows > c.max_rows)
      return lfail(EP_ERR_INVALID_ARG, "num_rows outside [0, max_rows]");
  }
  if (row_base && (!row_begin || c.groups_per_base < 1))
    return lfail(EP_ERR_INVALID_ARG, "row_base needs row_begin and groups_per_base");
  p->s.G = c.num_groups;
  p->s.per_base = c.groups_per_base > 0 ? c.groups_per_base : 1;
  p->s.pool = c.max_rows;
  p->s.dense_rows = num_rows;
  p->s.begin = row_begin;
  p->s.count = row_count;
  p->s.base = row_base;
  p->s.err = h->err;
  p->partial = h->partial;
  p->tickets = h->tickets;
  p->K = c.in_features;
  p->N = c.out_features;
  p->Nw = h->Nw;
  p->act = c.activation;
  p->ldz = h->ldz;
  p->x = static_cast<const __nv_bfloat16*>(x);
  p->w = static_cast<const __nv_bfloat16*>(w);
  p->y_f32 = c.out_dtype == EP_DTYPE_FP32;
  p->dw_f32 = c.weight_grad_dtype == EP_DTYPE_FP32;
  return EP_OK;
}

ep_status status_of(cudaError_t e) { return e == cudaSuccess ? EP_OK : lcuda(e); }

}  // namespace

extern "C" size_t ep_linear_workspace_size(const ep_linear_config* cfg) {
  ep_linear_handle h{};
  return plan_linear(cfg, &h) == EP_OK ? h.bytes : 0;
}

extern "C" ep_status ep_linear_create(const ep_linear_config* cfg, void* d_workspace,
                                      size_t workspace_bytes, ep_linear_handle** out_handle) {
  if (!out_handle) return lfail(EP_ERR_INVALID_ARG, "out_handle is NULL");
  *out_handle = nullptr;
  ep_linear_handle h{};
  h.ws = static_cast<uint8_t*>(d_workspace);
  const ep_status s = plan_linear(cfg, &h);
  if (s != EP_OK) return s;
  if (!d_workspace || (uintptr_t)d_workspace % 256 != 0)
    return lfail(EP_ERR_WORKSPACE, "linear workspace is NULL or not 256-byte aligned");
  if (workspace_bytes < h.bytes) return lfail(EP_ERR_WORKSPACE, "linear workspace too small");
  ep_linear_handle* p = new (std::nothrow) ep_linear_handle(h);
  if (!p) return lfail(EP_ERR_INVALID_ARG, "out of host memory");
  open_header(&p->header, d_workspace);
  *out_handle = p;
  return EP_OK;
}

extern "C" void ep_linear_destroy(ep_linear_handle* h) { delete h; }

extern "C" ep_status ep_linear_forward(ep_linear_handle* h, const void* x, const void* weight,
                                       const float* bias, const void* residual,
                                       const int32_t* row_begin, const int32_t* row_count,
                                       const int32_t* row_base, int64_t num_rows, void* y,
                                       void* preact, void* stream) {
  if (!h) return lfail(EP_ERR_INVALID_ARG, "linear handle is NULL");
  LinearParams p;
  ep_status s = fill_linear(h, x, weight, row_begin, row_count, row_base, num_rows, &p);
  if (s != EP_OK) return s;
  const size_t size = p.y_f32 ? 4 : 2;
  if (!y || (uintptr_t)y % size != 0 || (uintptr_t)residual % size != 0 ||
      (uintptr_t)preact % 2 != 0 || (uintptr_t)bias % 4 != 0)
    return lfail(EP_ERR_INVALID_ARG, "y is NULL, or an argument misaligned");
  p.bias = bias;
  p.residual = residual;
  p.y = y;
  p.z = static_cast<__nv_bfloat16*>(preact);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((s = linear_ready(h, st)) != EP_OK) return s;
  if (!row_begin && num_rows == 0) return EP_OK;
  if (few_rows_supported(p)) return status_of(launch_linear_few_rows(p, h->sm_count, st));
  return status_of(launch_linear_forward(p, h->sm_count, st));
}

extern "C" ep_status ep_linear_backward(ep_linear_handle* h, const void* dy, const void* x,
                                        const void* weight, const void* preact,
                                        const int32_t* row_begin, const int32_t* row_count,
                                        const int32_t* row_base, int64_t num_rows, void* dx,
                                        void* dweight, float* dbias, void* stream) {
  if (!h) return lfail(EP_ERR_INVALID_ARG, "linear handle is NULL");
  if (!h->cfg.backward)
    return lfail(EP_ERR_STATE, "the config did not reserve the backward pass's scratch");
  if (!dx && !dweight && !dbias)
    return lfail(EP_ERR_INVALID_ARG, "give at least one of dx, dweight and dbias");
  LinearParams p;
  ep_status s = fill_linear(h, x, weight, row_begin, row_count, row_base, num_rows, &p);
  if (s != EP_OK) return s;
  const size_t size = p.y_f32 ? 4 : 2;
  if (!dy || (uintptr_t)dy % size != 0) return lfail(EP_ERR_INVALID_ARG, "dy is NULL or misaligned");
  if (p.act != EP_ACT_NONE && (!preact || (uintptr_t)preact % 2 != 0))
    return lfail(EP_ERR_INVALID_ARG, "an activation's gradient needs preact");
  if ((uintptr_t)dx % 2 != 0 || (uintptr_t)dweight % (p.dw_f32 ? 4 : 2) != 0 ||
      (uintptr_t)dbias % 4 != 0)
    return lfail(EP_ERR_INVALID_ARG, "a gradient is misaligned");
  p.dy = dy;
  p.z = static_cast<__nv_bfloat16*>(const_cast<void*>(preact));
  p.dx = static_cast<__nv_bfloat16*>(dx);
  p.dw = dweight;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((s = linear_ready(h, st)) != EP_OK) return s;
  // without an activation dz is dy: the products read it in place where its
  // rows are whole 16-byte pieces
  const bool in_place = p.act == EP_ACT_NONE && !p.y_f32 && p.N % 8 == 0 && (uintptr_t)dy % 16 == 0;
  GradParams q;
  memset(&q, 0, sizeof(q));
  q.p = p;
  q.dz = (dx || dweight) && !in_place ? h->dz : nullptr;
  q.part = dbias ? h->part : nullptr;
  q.row_blocks = p.s.begin ? h->row_blocks : (num_rows + kGradRows - 1) / kGradRows;
  q.db = dbias;
  if ((q.dz || q.part) && q.row_blocks > 0 && (s = status_of(launch_act_grad(q, st))) != EP_OK)
    return s;
  if (dbias) {
    s = status_of(launch_overlapped(bias_grad_kernel, dim3((p.Nw + 31) / 32, p.s.G), 256, 0, st, q));
    if (s != EP_OK) return s;
  }
  p.dz = in_place ? static_cast<const __nv_bfloat16*>(dy) : h->dz;
  if (in_place) p.ldz = p.N;
  if (dx && (s = status_of(launch_linear_input_grad(p, h->sm_count, st))) != EP_OK) return s;
  return dweight ? status_of(launch_linear_weight_grad(p, h->sm_count, st)) : EP_OK;
}

extern "C" ep_status ep_linear_sync(ep_linear_handle* h, void* stream) {
  if (!h) return lfail(EP_ERR_INVALID_ARG, "linear handle is NULL");
  uint32_t bits = 0;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = header_report(&h->header, st, &bits);
  if (e != cudaSuccess) return lcuda(e);
  if (bits & kErrLinearTimeout) {
    if ((e = header_renew(&h->header, st)) != cudaSuccess) return lcuda(e);   // tickets may be left over
    return lfail(EP_ERR_TIMEOUT, "a product's bounded wait gave up; its output is not complete");
  }
  if (bits & kErrSegment)
    return lfail(EP_ERR_INVALID_INDEX,
                 "a segment reached outside the row pool and was cut, or a backward pass's overlapped");
  return EP_OK;
}
