// Host library of the products of block-quantised operands, and the elementwise
// kernel of their backward pass. The products themselves are in ep_qlinear_mma.cu.
#include <climits>
#include <cstring>
#include <new>
#include <type_traits>

#include "ep_header.cuh"
#include "ep_launch.cuh"
#include "ep_linear_grad.cuh"
#include "ep_pieces.cuh"
#include "ep_qlinear.cuh"
#include "ep_quant.cuh"

namespace ep {
namespace {

// dz = dy act'(z), quantised by 128 of a row for dx, rounded to bf16 for dW, and the
// sums of its columns over each block of rows: one pass. A half-warp takes 128 columns,
// eight a lane, of every `lanes`th row of a CTA's kGradRows; codes and scales are of the
// unrounded dz. Two rows are on their way ahead of the arithmetic: the sums alone of 128
// experts x 973 rows x 2 x 2048 (1.5 GB) take 305 us, 5 TB/s, 673 with one row at a time.
struct QGradParams {
  GradParams g;
  uint8_t* codes;            // [pool][ld], or NULL
  float* scales;             // [pool][Sw]
  int64_t ld;
  int Nb, Sw;
  int vec;                   // rows of dy and z are whole 16-byte pieces
};

// Eight neighbouring columns, of which `left` exist, zeros for the others: whole 16-byte
// pieces (VEC: all eight exist, or none), or one by one.
template <bool VEC, typename T>
struct Columns {
  Raw8<T> raw;
  __device__ __forceinline__ void load(const T* at, int left) {
    zero8(raw);
    if (VEC) {
      if (left >= 8) load8<T>(at, 0, raw);
    } else {
      T* to = reinterpret_cast<T*>(&raw);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) to[i] = at[i];
    }
  }
};

template <bool VEC>
__device__ __forceinline__ void store_columns(__nv_bfloat16* at, int left, const float (&v)[8]) {
  if (VEC) {
    if (left >= 8) store8<__nv_bfloat16>(at, 0, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) at[i] = __float2bfloat16_rn(v[i]);
  }
}

template <int ACT, typename T, bool VEC>
__global__ void __launch_bounds__(kGradThreads) quant_grad_kernel(QGradParams a) {
  begin_overlapped();
  const GradParams& q = a.g;
  const LinearParams& p = q.p;
  __shared__ BlockPlace at;
  __shared__ float sums[2][kGradThreads * 8];
  constexpr bool kGated = ACT == EP_ACT_SWIGLU;
  constexpr int kAhead = 2;                               // rows on their way
  const int64_t block = blockIdx.x;
  find_block(p.s, block, q.row_blocks, at);
  __syncthreads();
  if (at.row0 >= at.row1) return;
  const int half = threadIdx.x >> 4, sub = threadIdx.x & 15;
  const int wide = kGradThreads / 16 / q.lanes;           // half-warps beside each other in a row
  const int lane_row = half / wide, cb = blockIdx.y * wide + half % wide;
  const int c = cb * 128 + sub * 8;
  const bool block_in = cb < a.Nb;
  const int left = block_in ? p.N - c : 0;                // columns that exist, from this lane's on
  float s0[8], s1[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s0[i] = s1[i] = 0.0f;
  const int rows = (int)(at.row1 - at.row0);
  const int64_t row0 = at.begin + at.row0;
  struct Step {
    Columns<VEC, T> dy;
    Columns<VEC, __nv_bfloat16> z, up;
  };
  Step next[kAhead];
  const auto fetch = [&](int r, Step& t) {
    const int here = r < rows ? left : 0;
    t.dy.load(static_cast<const T*>(p.dy) + (row0 + r) * p.N + c, here);
    if (ACT != EP_ACT_NONE) t.z.load(p.z + (row0 + r) * p.Nw + c, here);
    if (kGated) t.up.load(p.z + (row0 + r) * p.Nw + p.N + c, here);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(lane_row + i * q.lanes, next[i]);
  // every half-warp goes through the same number of steps: the shuffles are the warp's
  for (int step = 0; step < rows; step += kAhead * q.lanes) {
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int r = step + n * q.lanes + lane_row;
      float d0[8], d1[8];
      floats8(next[n].dy.raw, d0);
      if (kGated) {
        float zg[8], zu[8];
        floats8(next[n].z.raw, zg);
        floats8(next[n].up.raw, zu);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // silu'(g) = s (1 + g (1 - s)), silu(g) = g s
          const float s = sigmoid_of(zg[i]);
          d1[i] = d0[i] * (zg[i] * s);
          d0[i] *= zu[i] * (s * (1.0f + zg[i] * (1.0f - s)));
        }
      } else if (ACT != EP_ACT_NONE) {
        float zv[8];
        floats8(next[n].z.raw, zv);
#pragma unroll
        for (int i = 0; i < 8; ++i) d0[i] *= slope_of(ACT, zv[i]);
      }
      fetch(r + kAhead * q.lanes, next[n]);
      // columns and rows that do not exist are zeros: zero times a finite slope
      const bool row_in = r < rows;
      const int here = row_in ? left : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s0[i] += d0[i];
        if (kGated) s1[i] += d1[i];
      }
      const int64_t row = row0 + r;
      if (q.dz) {
        __nv_bfloat16* out = q.dz + row * p.ldz + c;
        store_columns<VEC>(out, here, d0);
        if (kGated) store_columns<VEC>(out + p.N, here, d1);
      }
      if (a.codes) {
#pragma unroll
        for (int h = 0; h < (kGated ? 2 : 1); ++h) {
          const float (&v)[8] = h ? d1 : d0;
          const float amax = max16(amax8(v));
          const float scale = scale_of(amax);
          const uint2 code = e4m3x8(v, block_scale(amax, scale));
          if (row_in && block_in) {
            *reinterpret_cast<uint2*>(a.codes + row * a.ld + (int64_t)h * a.Nb * 128 + c) = code;
            if (sub == 0) a.scales[row * a.Sw + h * a.Nb + cb] = scale;
          }
        }
      }
    }
  }
  if (!q.part) return;
  if (q.lanes > 1) {   // the first of the threads that share a column adds the others' sums
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sums[0][threadIdx.x * 8 + i] = s0[i];
      if (kGated) sums[1][threadIdx.x * 8 + i] = s1[i];
    }
    __syncthreads();
    if (lane_row > 0) return;
    for (int l = 1; l < q.lanes; ++l)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s0[i] += sums[0][(l * wide * 16 + threadIdx.x) * 8 + i];
        if (kGated) s1[i] += sums[1][(l * wide * 16 + threadIdx.x) * 8 + i];
      }
  }
  float* part = q.part + block * p.Nw + c;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < left) {
      part[i] = s0[i];
      if (kGated) part[p.N + i] = s1[i];
    }
}

template <typename T>
cudaError_t launch_quant_grad(QGradParams a, cudaStream_t st) {
  const int halves = kGradThreads / 16;
  a.g.lanes = 1;       // rows too short for a CTA's threads: several of them share a column
  while (a.g.lanes < halves && a.Nb * a.g.lanes * 2 <= halves) a.g.lanes *= 2;
  const int wide = halves / a.g.lanes;
  const dim3 grid((unsigned)a.g.row_blocks, (unsigned)((a.Nb + wide - 1) / wide));
  const auto of = [&](auto vec) {
    constexpr bool VEC = decltype(vec)::value;
    switch (a.g.p.act) {
      case EP_ACT_RELU: return quant_grad_kernel<EP_ACT_RELU, T, VEC>;
      case EP_ACT_SILU: return quant_grad_kernel<EP_ACT_SILU, T, VEC>;
      case EP_ACT_GELU: return quant_grad_kernel<EP_ACT_GELU, T, VEC>;
      case EP_ACT_SWIGLU: return quant_grad_kernel<EP_ACT_SWIGLU, T, VEC>;
      default: return quant_grad_kernel<EP_ACT_NONE, T, VEC>;
    }
  };
  const auto kernel = a.vec ? of(std::true_type()) : of(std::false_type());
  return launch_overlapped(kernel, grid, kGradThreads, 0, st, a);
}

}  // namespace
}  // namespace ep

struct ep_qlinear_handle {
  ep_linear_config cfg;
  uint8_t* ws;
  ep::Header header;
  int sm_count;
  int Nw, Kb, Nb, Sw;
  int64_t ldz, row_blocks;
  int32_t* err;
  unsigned int* tickets;
  float* partial;
  __nv_bfloat16* dz;      // for dW
  __nv_bfloat16* x;       // x's values for dW
  uint8_t* dz8;           // for dx
  float* dzs;
  float* part;
  size_t bytes;
};

namespace {

using namespace ep;

ep_status qlfail(ep_status st, const char* msg) { return record_error(st, msg); }
ep_status qlcuda(cudaError_t e) { return record_error(EP_ERR_CUDA, cudaGetErrorString(e)); }
ep_status qlstatus(cudaError_t e) { return e == cudaSuccess ? EP_OK : qlcuda(e); }

static_assert(kTicketOffset + kLinearMaxPairs * 2 * sizeof(unsigned int) <= kHeaderBytes, "tickets");

// The next `bytes` of the workspace, on a 256-byte boundary.
template <typename T>
void carve(ep_qlinear_handle* h, T** at, size_t bytes) {
  *at = reinterpret_cast<T*>(h->ws ? h->ws + h->bytes : nullptr);
  h->bytes += (bytes + 255) / 256 * 256;
}

ep_status plan_qlinear(const ep_linear_config* c, ep_qlinear_handle* h) {
  const ep_status s = check_linear(c);
  if (s != EP_OK) return s;
  if (c->in_features % 16 != 0)
    return qlfail(EP_ERR_INVALID_ARG, "in_features must be a multiple of 16");
  h->cfg = *c;
  const int parts = c->activation == EP_ACT_SWIGLU ? 2 : 1;
  h->Nw = parts * c->out_features;
  h->Kb = (c->in_features + 127) / 128;
  h->Nb = (c->out_features + 127) / 128;
  h->Sw = parts * h->Nb;
  h->ldz = (h->Nw + 63) / 64 * 64;
  h->row_blocks = (c->max_rows + kGradRows - 1) / kGradRows + c->num_groups;
  h->err = reinterpret_cast<int32_t*>(h->ws);
  h->tickets = reinterpret_cast<unsigned int*>(h->ws ? h->ws + kTicketOffset : nullptr);
  h->bytes = kHeaderBytes;
  carve(h, &h->partial,
        kLinearMaxPairs * (c->backward && c->max_rows > kLongTerms ? kPartBytesLong : kPartBytesGrad));
  h->dz = h->x = nullptr;
  h->dz8 = nullptr;
  h->dzs = h->part = nullptr;
  if (c->backward) {
    const size_t rows = (size_t)c->max_rows;
    carve(h, &h->dz, rows * h->ldz * 2);
    carve(h, &h->x, rows * c->in_features * 2);
    carve(h, &h->dz8, rows * h->Sw * 128);
    carve(h, &h->dzs, rows * h->Sw * 4);
    carve(h, &h->part, (size_t)h->row_blocks * h->Nw * 4);
  }
  return EP_OK;
}

ep_status qlinear_ready(ep_qlinear_handle* h, cudaStream_t st) {
  if (h->sm_count == 0) {
    int dev = 0, n = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return qlcuda(e);
    h->sm_count = n;
  }
  return qlstatus(header_ready(&h->header, st));
}

ep_status fill_qlinear(const ep_qlinear_handle* h, const void* x, const float* x_scale,
                       const void* w, const float* w_scale, const int32_t* row_begin,
                       const int32_t* row_count, const int32_t* row_base, int64_t num_rows,
                       QLinearParams* p) {
  if (!h) return qlfail(EP_ERR_INVALID_ARG, "qlinear handle is NULL");
  const ep_linear_config& c = h->cfg;
  if (!x || !w || (uintptr_t)x % 16 != 0 || (uintptr_t)w % 16 != 0)
    return qlfail(EP_ERR_INVALID_ARG, "x and weight must be given, 16-byte aligned");
  if (!x_scale || !w_scale || ((uintptr_t)x_scale | (uintptr_t)w_scale) % 4 != 0)
    return qlfail(EP_ERR_INVALID_ARG, "x_scale and w_scale must be given, 4-byte aligned");
  if ((row_begin == nullptr) != (row_count == nullptr))
    return qlfail(EP_ERR_INVALID_ARG, "give row_begin and row_count together, or neither");
  if (((uintptr_t)row_begin | (uintptr_t)row_count | (uintptr_t)row_base) % 4 != 0)
    return qlfail(EP_ERR_INVALID_ARG, "row_begin, row_count or row_base is misaligned");
  if (!row_begin) {
    if (c.num_groups != 1)
      return qlfail(EP_ERR_INVALID_ARG, "several groups need row_begin and row_count");
    if (num_rows < 0 || num_rows > c.max_rows)
      return qlfail(EP_ERR_INVALID_ARG, "num_rows outside [0, max_rows]");
  }
  if (row_base && (!row_begin || c.groups_per_base < 1))
    return qlfail(EP_ERR_INVALID_ARG, "row_base needs row_begin and groups_per_base");
  memset(p, 0, sizeof(*p));
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
  p->Kb = h->Kb;
  p->Nb = h->Nb;
  p->Sw = h->Sw;
  p->x = static_cast<const uint8_t*>(x);
  p->xs = x_scale;
  p->w = static_cast<const uint8_t*>(w);
  p->ws = w_scale;
  p->y_f32 = c.out_dtype == EP_DTYPE_FP32;
  p->partial = h->partial;
  p->tickets = h->tickets;
  return EP_OK;
}

}  // namespace

extern "C" size_t ep_qlinear_workspace_size(const ep_linear_config* cfg) {
  ep_qlinear_handle h{};
  return plan_qlinear(cfg, &h) == EP_OK ? h.bytes : 0;
}

extern "C" ep_status ep_qlinear_create(const ep_linear_config* cfg, void* d_workspace,
                                       size_t workspace_bytes, ep_qlinear_handle** out_handle) {
  if (!out_handle) return qlfail(EP_ERR_INVALID_ARG, "out_handle is NULL");
  *out_handle = nullptr;
  ep_qlinear_handle h{};
  h.ws = static_cast<uint8_t*>(d_workspace);
  const ep_status s = plan_qlinear(cfg, &h);
  if (s != EP_OK) return s;
  if (!d_workspace || (uintptr_t)d_workspace % 256 != 0)
    return qlfail(EP_ERR_WORKSPACE, "qlinear workspace is NULL or not 256-byte aligned");
  if (workspace_bytes < h.bytes) return qlfail(EP_ERR_WORKSPACE, "qlinear workspace too small");
  ep_qlinear_handle* p = new (std::nothrow) ep_qlinear_handle(h);
  if (!p) return qlfail(EP_ERR_INVALID_ARG, "out of host memory");
  open_header(&p->header, d_workspace);
  *out_handle = p;
  return EP_OK;
}

extern "C" void ep_qlinear_destroy(ep_qlinear_handle* h) { delete h; }

extern "C" ep_status ep_qlinear_forward(ep_qlinear_handle* h, const void* x, const float* x_scale,
                                        const void* weight, const float* w_scale,
                                        const float* bias, const void* residual,
                                        const int32_t* row_begin, const int32_t* row_count,
                                        const int32_t* row_base, int64_t num_rows, void* y,
                                        void* preact, void* stream) {
  QLinearParams p;
  ep_status s = fill_qlinear(h, x, x_scale, weight, w_scale, row_begin, row_count, row_base, num_rows, &p);
  if (s != EP_OK) return s;
  const size_t size = p.y_f32 ? 4 : 2;
  if (!y || (uintptr_t)y % size != 0 || (uintptr_t)residual % size != 0 ||
      (uintptr_t)preact % 2 != 0 || (uintptr_t)bias % 4 != 0)
    return qlfail(EP_ERR_INVALID_ARG, "y is NULL, or an argument misaligned");
  p.bias = bias;
  p.residual = residual;
  p.y = y;
  p.z = static_cast<__nv_bfloat16*>(preact);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((s = qlinear_ready(h, st)) != EP_OK) return s;
  if (!row_begin && num_rows == 0) return EP_OK;
  if (few_qrows_supported(p)) return qlstatus(launch_qlinear_few_rows(p, h->sm_count, st));
  return qlstatus(launch_qlinear_forward(p, h->sm_count, st));
}

extern "C" ep_status ep_qlinear_backward(ep_qlinear_handle* h, const void* dy, const void* x,
                                         const float* x_scale, const void* weight,
                                         const float* w_scale, const void* preact,
                                         const int32_t* row_begin, const int32_t* row_count,
                                         const int32_t* row_base, int64_t num_rows, void* dx,
                                         void* dweight, float* dbias, void* stream) {
  QLinearParams p;
  ep_status s = fill_qlinear(h, x, x_scale, weight, w_scale, row_begin, row_count, row_base, num_rows, &p);
  if (s != EP_OK) return s;
  const ep_linear_config& c = h->cfg;
  if (!c.backward)
    return qlfail(EP_ERR_STATE, "the config did not reserve the backward pass's scratch");
  if (!dx && !dweight && !dbias)
    return qlfail(EP_ERR_INVALID_ARG, "give at least one of dx, dweight and dbias");
  const size_t size = p.y_f32 ? 4 : 2;
  if (!dy || (uintptr_t)dy % size != 0) return qlfail(EP_ERR_INVALID_ARG, "dy is NULL or misaligned");
  if (p.act != EP_ACT_NONE && (!preact || (uintptr_t)preact % 2 != 0))
    return qlfail(EP_ERR_INVALID_ARG, "an activation's gradient needs preact");
  const bool dw_f32 = c.weight_grad_dtype == EP_DTYPE_FP32;
  if ((uintptr_t)dx % 2 != 0 || (uintptr_t)dweight % (dw_f32 ? 4 : 2) != 0 || (uintptr_t)dbias % 4 != 0)
    return qlfail(EP_ERR_INVALID_ARG, "a gradient is misaligned");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((s = qlinear_ready(h, st)) != EP_OK) return s;
  // without an activation dz is dy: dW reads it in place where its rows are whole
  // 16-byte pieces
  const bool whole = p.N % 8 == 0 && (uintptr_t)dy % 16 == 0;
  const bool in_place = p.act == EP_ACT_NONE && !p.y_f32 && whole;
  QGradParams a;
  memset(&a, 0, sizeof(a));
  LinearParams& l = a.g.p;
  l.s = p.s;
  l.K = p.K;
  l.N = p.N;
  l.Nw = p.Nw;
  l.act = p.act;
  l.ldz = h->ldz;
  l.y_f32 = p.y_f32;
  l.dy = dy;
  l.z = static_cast<__nv_bfloat16*>(const_cast<void*>(preact));
  l.partial = h->partial;
  l.tickets = h->tickets;
  l.dw = dweight;
  l.dw_f32 = dw_f32;
  a.g.dz = dweight && !in_place ? h->dz : nullptr;
  a.g.part = dbias ? h->part : nullptr;
  a.g.row_blocks = row_begin ? h->row_blocks : (num_rows + kGradRows - 1) / kGradRows;
  a.g.db = dbias;
  a.codes = dx ? h->dz8 : nullptr;
  a.scales = h->dzs;
  a.ld = (int64_t)h->Sw * 128;
  a.Nb = h->Nb;
  a.Sw = h->Sw;
  a.vec = whole && (p.act == EP_ACT_NONE || (uintptr_t)preact % 16 == 0);
  if ((a.g.dz || a.g.part || a.codes) && a.g.row_blocks > 0) {
    s = qlstatus(p.y_f32 ? launch_quant_grad<float>(a, st) : launch_quant_grad<__nv_bfloat16>(a, st));
    if (s != EP_OK) return s;
  }
  if (dbias) {
    s = qlstatus(launch_overlapped(bias_grad_kernel, dim3((p.Nw + 31) / 32, p.s.G), 256, 0, st, a.g));
    if (s != EP_OK) return s;
  }
  if (dx && (row_begin || num_rows > 0)) {
    p.dz8 = h->dz8;
    p.dzs = h->dzs;
    p.dx = static_cast<__nv_bfloat16*>(dx);
    if ((s = qlstatus(launch_qlinear_input_grad(p, h->sm_count, st))) != EP_OK) return s;
  }
  if (!dweight) return EP_OK;
  if (row_begin || num_rows > 0) {
    s = qlstatus(launch_dequantize(p.s, p.x, p.xs, p.K, h->x, h->sm_count, st));
    if (s != EP_OK) return s;
  }
  l.x = h->x;
  l.dz = in_place ? static_cast<const __nv_bfloat16*>(dy) : h->dz;
  if (in_place) l.ldz = p.N;
  return qlstatus(launch_linear_weight_grad(l, h->sm_count, st));
}

extern "C" ep_status ep_qlinear_sync(ep_qlinear_handle* h, void* stream) {
  if (!h) return qlfail(EP_ERR_INVALID_ARG, "qlinear handle is NULL");
  uint32_t bits = 0;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = header_report(&h->header, st, &bits);
  if (e != cudaSuccess) return qlcuda(e);
  if (bits & kErrLinearTimeout) {
    if ((e = header_renew(&h->header, st)) != cudaSuccess) return qlcuda(e);   // tickets may be left over
    return qlfail(EP_ERR_TIMEOUT, "a product's bounded wait gave up; its output is not complete");
  }
  if (bits & kErrSegment)
    return qlfail(EP_ERR_INVALID_INDEX,
                  "a segment reached outside the row pool and was cut, or segments overlapped in a backward "
                  "pass, or so much that the call did nothing");
  return EP_OK;
}
