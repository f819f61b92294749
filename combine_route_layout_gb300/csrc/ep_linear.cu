// Host library of the experts' products, y = act(x W^T + b) + residual over
// the segments of a row pool (the packed layout's, one per expert, or one
// dense product), and the elementwise kernels of the backward pass. The
// products themselves are in ep_linear_mma.cu.
#include <climits>
#include <cstring>
#include <new>

#include "ep_linear.cuh"

namespace ep {
namespace {

// dz = dy act'(z) and the sums of dz's columns over each block of rows. A CTA
// takes kGradRows rows of one group and 256 weight rows' columns, a thread a
// column; the block sums are added in block order by bias_grad_kernel. dz is
// rounded to bf16 because the products read it as a tensor-core operand; the
// sums are of the unrounded values.
constexpr int kGradRows = 64;

struct GradParams {
  LinearParams p;
  __nv_bfloat16* dz;         // NULL: only the sums
  float* part;               // [row blocks][Nw] or NULL
  float* db;                 // [G][Nw]
};

// Row blocks of the groups before each group.
__device__ int64_t blocks_of(int64_t count) { return (count + kGradRows - 1) / kGradRows; }

__global__ void __launch_bounds__(256) act_grad_kernel(GradParams q) {
  const LinearParams& p = q.p;
  const int c = blockIdx.x * 256 + threadIdx.x;
  const bool gated = p.act == EP_ACT_SWIGLU;
  int64_t seen = 0;
  for (int g = 0; g < p.s.G; ++g) {
    int64_t begin, count;
    segment_of(p.s, g, begin, count);
    const int64_t blocks = blocks_of(count);
    for (int64_t b = ((int64_t)blockIdx.y - seen % gridDim.y + gridDim.y) % gridDim.y; b < blocks;
         b += gridDim.y) {
      if (c >= p.N) continue;
      float s0 = 0.0f, s1 = 0.0f;
      const int64_t end = min(count, (b + 1) * kGradRows);
      for (int64_t r = b * kGradRows; r < end; ++r) {
        const int64_t o = (begin + r) * p.N + c;
        const float dy = p.y_f32 ? static_cast<const float*>(p.dy)[o]
                                 : __bfloat162float(static_cast<const __nv_bfloat16*>(p.dy)[o]);
        float d0 = dy, d1 = 0.0f;
        if (gated) {
          const float zg = __bfloat162float(p.z[(begin + r) * p.Nw + c]);
          const float zu = __bfloat162float(p.z[(begin + r) * p.Nw + p.N + c]);
          d0 = dy * zu * slope_of(EP_ACT_SILU, zg);
          d1 = dy * silu_of(zg);
        } else if (p.act != EP_ACT_NONE) {
          d0 = dy * slope_of(p.act, __bfloat162float(p.z[(begin + r) * p.Nw + c]));
        }
        s0 += d0;
        s1 += d1;
        if (q.dz) {
          q.dz[(begin + r) * p.ldz + c] = __float2bfloat16_rn(d0);
          if (gated) q.dz[(begin + r) * p.ldz + p.N + c] = __float2bfloat16_rn(d1);
        }
      }
      if (q.part) {
        q.part[(seen + b) * p.Nw + c] = s0;
        if (gated) q.part[(seen + b) * p.Nw + p.N + c] = s1;
      }
    }
    seen += blocks;
  }
}

__global__ void __launch_bounds__(256) bias_grad_kernel(GradParams q) {
  const LinearParams& p = q.p;
  const int c = blockIdx.x * 256 + threadIdx.x;
  const int g = blockIdx.y;
  int64_t first = 0, begin, count;
  for (int i = 0; i < g; ++i) {
    segment_of(p.s, i, begin, count);
    first += blocks_of(count);
  }
  segment_of(p.s, g, begin, count);
  if (c >= p.Nw) return;
  float s = 0.0f;
  for (int64_t b = 0; b < blocks_of(count); ++b) s += q.part[(first + b) * p.Nw + c];
  q.db[(int64_t)g * p.Nw + c] = s;
}

}  // namespace
}  // namespace ep

struct ep_linear_handle {
  ep_linear_config cfg;
  uint8_t* ws;
  bool needs_init;
  int sm_count;
  int Nw;
  int64_t ldz, row_blocks;
  int32_t* err;
  __nv_bfloat16* dz;
  float* part;
  size_t bytes;
};

namespace {

using namespace ep;

ep_status lfail(ep_status st, const char* msg) { return record_error(st, msg); }
ep_status lcuda(cudaError_t e) { return record_error(EP_ERR_CUDA, cudaGetErrorString(e)); }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

ep_status plan_linear(const ep_linear_config* c, ep_linear_handle* h) {
  if (!c) return lfail(EP_ERR_INVALID_ARG, "linear config is NULL");
  if (c->num_groups < 1 || c->num_groups > EP_MAX_EXPERTS)
    return lfail(EP_ERR_INVALID_ARG, "num_groups outside [1, 1024]");
  if (c->groups_per_base < 0)
    return lfail(EP_ERR_INVALID_ARG, "groups_per_base must be >= 0");
  if (c->in_features < 8 || c->in_features % 8 != 0)
    return lfail(EP_ERR_INVALID_ARG, "in_features must be a positive multiple of 8");
  if (c->out_features < 1 || c->out_features > (1 << 24) || c->in_features > (1 << 24))
    return lfail(EP_ERR_INVALID_ARG, "in_features and out_features must be in [1, 2^24]");
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
  h->ldz = (h->Nw + 7) / 8 * 8;
  h->row_blocks = (c->max_rows + kGradRows - 1) / kGradRows + c->num_groups;
  size_t off = 256;
  h->err = reinterpret_cast<int32_t*>(h->ws);
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

// As the router's: a captured call leaves the clearing to the next one too.
ep_status linear_ready(ep_linear_handle* h, cudaStream_t st) {
  if (h->sm_count == 0) {
    int dev = 0, n = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return lcuda(e);
    h->sm_count = n;
  }
  if (!h->needs_init) return EP_OK;
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing(st, &cap);
  if (e == cudaSuccess) e = cudaMemsetAsync(h->ws, 0, 256, st);
  if (e != cudaSuccess) return lcuda(e);
  if (cap == cudaStreamCaptureStatusNone) h->needs_init = false;
  return EP_OK;
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
  ep_linear_handle h;
  memset(&h, 0, sizeof(h));
  return plan_linear(cfg, &h) == EP_OK ? h.bytes : 0;
}

extern "C" ep_status ep_linear_create(const ep_linear_config* cfg, void* d_workspace,
                                      size_t workspace_bytes, ep_linear_handle** out_handle) {
  if (!out_handle) return lfail(EP_ERR_INVALID_ARG, "out_handle is NULL");
  *out_handle = nullptr;
  ep_linear_handle h;
  memset(&h, 0, sizeof(h));
  h.ws = static_cast<uint8_t*>(d_workspace);
  const ep_status s = plan_linear(cfg, &h);
  if (s != EP_OK) return s;
  if (!d_workspace || (uintptr_t)d_workspace % 256 != 0)
    return lfail(EP_ERR_WORKSPACE, "linear workspace is NULL or not 256-byte aligned");
  if (workspace_bytes < h.bytes) return lfail(EP_ERR_WORKSPACE, "linear workspace too small");
  ep_linear_handle* p = new (std::nothrow) ep_linear_handle(h);
  if (!p) return lfail(EP_ERR_INVALID_ARG, "out of host memory");
  p->needs_init = true;
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
  GradParams q;
  memset(&q, 0, sizeof(q));
  q.p = p;
  q.dz = dx || dweight ? h->dz : nullptr;
  q.part = dbias ? h->part : nullptr;
  q.db = dbias;
  int64_t rows = h->row_blocks < 4096 ? h->row_blocks : 4096;
  act_grad_kernel<<<dim3((p.N + 255) / 256, (unsigned)rows), 256, 0, st>>>(q);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && dbias) {
    bias_grad_kernel<<<dim3((p.Nw + 255) / 256, p.s.G), 256, 0, st>>>(q);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return lcuda(e);
  p.dz = h->dz;
  if (dx && (s = status_of(launch_linear_input_grad(p, h->sm_count, st))) != EP_OK) return s;
  return dweight ? status_of(launch_linear_weight_grad(p, h->sm_count, st)) : EP_OK;
}

extern "C" ep_status ep_linear_sync(ep_linear_handle* h, void* stream) {
  if (!h) return lfail(EP_ERR_INVALID_ARG, "linear handle is NULL");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t bits = 0;
  cudaError_t e = cudaSuccess;
  if (!h->needs_init) {
    e = cudaMemcpyAsync(&bits, h->err, sizeof(bits), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(h->err, 0, sizeof(bits), st);
  }
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return lcuda(e);
  if (bits & kErrLinearTimeout)
    return lfail(EP_ERR_TIMEOUT, "a product's bounded wait gave up; its output is not complete");
  if (bits & kErrSegment)
    return lfail(EP_ERR_INVALID_INDEX, "a segment reached outside the row pool and was cut");
  return EP_OK;
}
