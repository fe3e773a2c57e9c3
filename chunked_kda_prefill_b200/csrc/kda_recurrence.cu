// kda_recurrence.cu -- the gated recurrence, the vector form of the KDA state:
//     a_t = exp(lb sigmoid(e^A (g_t + bias))),  h_t = a_t h_{t-1} + sigmoid(beta_t) x_t.
//
// One block walks one (sequence, head), a thread one channel, token by token.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "kda_args.h"
#include "kda_io.cuh"
#include "kda_recurrence.h"

namespace kda {
namespace {

struct RecParams {
  kda_view_t x, g, beta, dout;  // device addresses and strides
  const int32_t* plan;
  int32_t checksum;
  int32_t tnd, N, S, D, tiles, chain;
  const float* h0;
  const float* A_log;
  const float* dt_bias;
  float lower_bound;
  float* states;
  const float* dfinal;
  int32_t* status;
  void* out;      // forward: out; backward: dx
  void* dg;
  void* dbeta;
  float* final_state;  // forward
  float* dh0;
  float* part_bias;  // [B][N][D]
  float* part_A;     // [B][N][D]
  kda_view_t od, bd;  // strides of the dense outputs with and without channels
};

template <class T>
__device__ __forceinline__ const T* at(const kda_view_t& v, long long b, long long n, long long s) {
  return static_cast<const T*>(v.data) + b * v.stride_b + n * v.stride_n + s * v.stride_s;
}

template <class T>
__global__ void rec_forward_kernel(const RecParams p) {
  if (p.plan[RH_CHECKSUM] != p.checksum) {
    if (threadIdx.x == 0) *p.status = DS_PLAN;
    return;
  }
  const int32_t* rec = p.plan + kRecHeader + (blockIdx.x / p.N) * kRecRecord;
  const int n = blockIdx.x % p.N, d = threadIdx.x, R = p.plan[RH_TILE_ROWS];
  const int slot = rec[RR_SLOT], row0 = rec[RR_ROW0], len = rec[RR_LEN];
  const GateScale c = gate_scale(p.A_log[n], p.lower_bound);
  const float bias = p.dt_bias[(size_t)n * p.D + d];
  const size_t st = ((size_t)slot * p.N + n) * p.D + d;
  float h = p.h0 ? p.h0[st] : 0.f;
  T* out = static_cast<T*>(p.out) + (size_t)slot * p.od.stride_b + (size_t)n * p.od.stride_n + d;
  for (int i = 0; i < len; ++i) {
    const int s = row0 + i;
    float t;
    const float sg = gate_sigmoid(c, to_f32(at<T>(p.g, slot, n, s)[d]) + bias, &t);
    h = ex2(c.l2 * sg) * h +
        sigmoid(to_f32(*at<T>(p.beta, slot, n, s))) * to_f32(at<T>(p.x, slot, n, s)[d]);
    out[(size_t)s * p.od.stride_s] = from_f32<T>(h);
    if (p.states && (i + 1) % R == 0 && i + 1 < len)
      p.states[((size_t)(rec[RR_INDEX] + i / R) * p.N + n) * p.D + d] = h;
  }
  p.final_state[st] = h;
  if (!p.tnd)
    for (int s = len; s < p.S; ++s) out[(size_t)s * p.od.stride_s] = from_f32<T>(0.f);
}

template <class T>
__global__ void rec_backward_kernel(const RecParams p) {
  extern __shared__ float hist[];  // [R][D] states before each of a tile's tokens
  __shared__ float red[4];
  if (p.plan[RH_CHECKSUM] != p.checksum) {
    if (threadIdx.x == 0) *p.status = DS_PLAN;
    return;
  }
  const int32_t* rec = p.plan + kRecHeader + (blockIdx.x / p.N) * kRecRecord;
  const int n = blockIdx.x % p.N, d = threadIdx.x, R = p.plan[RH_TILE_ROWS];
  const int slot = rec[RR_SLOT], row0 = rec[RR_ROW0], len = rec[RR_LEN];
  const GateScale c = gate_scale(p.A_log[n], p.lower_bound);
  const float bias = p.dt_bias[(size_t)n * p.D + d];
  const size_t st = ((size_t)slot * p.N + n) * p.D + d;
  const size_t o0 = (size_t)slot * p.od.stride_b + (size_t)n * p.od.stride_n + d;
  T* dx = static_cast<T*>(p.out) + o0;
  T* dg = static_cast<T*>(p.dg) + o0;
  T* dbeta = static_cast<T*>(p.dbeta) + (size_t)slot * p.bd.stride_b + (size_t)n * p.bd.stride_n;
  float carry = p.dfinal ? p.dfinal[st] : 0.f;  // a_{t+1} lam_{t+1}, or dfinal behind the last
  float sum_bias = 0.f, sum_A = 0.f;
  for (int j = rec[RR_COUNT] - 1; j >= 0; --j) {
    const int i0 = j * R, i1 = min(len, i0 + R);
    float h = j > 0 ? p.states[((size_t)(rec[RR_INDEX] + j - 1) * p.N + n) * p.D + d]
                    : (p.h0 ? p.h0[st] : 0.f);
    for (int i = i0; i < i1; ++i) {
      hist[(i - i0) * p.D + d] = h;
      const int s = row0 + i;
      float t;
      const float sg = gate_sigmoid(c, to_f32(at<T>(p.g, slot, n, s)[d]) + bias, &t);
      h = ex2(c.l2 * sg) * h +
          sigmoid(to_f32(*at<T>(p.beta, slot, n, s))) * to_f32(at<T>(p.x, slot, n, s)[d]);
    }
    for (int i = i1 - 1; i >= i0; --i) {
      const int s = row0 + i;
      const float raw = to_f32(at<T>(p.g, slot, n, s)[d]) + bias;
      float t;
      const float sg = gate_sigmoid(c, raw, &t), a = ex2(c.l2 * sg);
      const float b = sigmoid(to_f32(*at<T>(p.beta, slot, n, s)));
      const float x = to_f32(at<T>(p.x, slot, n, s)[d]);
      const float lam = (p.dout.data ? to_f32(at<T>(p.dout, slot, n, s)[d]) : 0.f) + carry;
      carry = a * lam;
      dx[(size_t)s * p.od.stride_s] = from_f32<T>(b * lam);
      const float graw = carry * hist[(i - i0) * p.D + d] * p.lower_bound * c.ea * sg *
                         one_minus(sg, t);
      dg[(size_t)s * p.od.stride_s] = from_f32<T>(graw);
      sum_bias += graw;
      sum_A += graw * raw;
      float dot = lam * x;
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if ((d & 31) == 0) red[d >> 5] = dot;
      __syncthreads();
      if (d == 0) {
        float sum = 0.f;
        for (int w = 0; w < p.D / 32; ++w) sum += red[w];
        dbeta[(size_t)s * p.bd.stride_s] = from_f32<T>(sum * b * (1.f - b));
      }
      __syncthreads();
    }
  }
  if (p.dh0) p.dh0[st] = carry;
  p.part_bias[st] = sum_bias;
  p.part_A[st] = sum_A;
  if (!p.tnd)
    for (int s = len; s < p.S; ++s) {
      dx[(size_t)s * p.od.stride_s] = from_f32<T>(0.f);
      dg[(size_t)s * p.od.stride_s] = from_f32<T>(0.f);
      if (d == 0) dbeta[(size_t)s * p.bd.stride_s] = from_f32<T>(0.f);
    }
}

// ddt_bias and dA_log: the sequences' sums in order, in fp64
__global__ void rec_params_kernel(const float* part_bias, const float* part_A, int B, int N, int D,
                                  float* dA_log, float* ddt_bias) {
  __shared__ double red[128];
  const int n = blockIdx.x, d = threadIdx.x;
  double sb = 0, sa = 0;
  for (int b = 0; b < B; ++b) {
    sb += part_bias[((size_t)b * N + n) * D + d];
    sa += part_A[((size_t)b * N + n) * D + d];
  }
  ddt_bias[(size_t)n * D + d] = (float)sb;
  red[d] = sa;
  __syncthreads();
  if (d == 0) {
    double s = 0;
    for (int i = 0; i < D; ++i) s += red[i];
    dA_log[n] = (float)s;
  }
}

template <class T>
__global__ void rec_step_kernel(const T* x, const T* g, const T* beta, const float* h0,
                                const float* A_log, const float* dt_bias, float lower_bound, T* out,
                                float* h1, int N, int D, long long total) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= total) return;
  const long long row = i / D;
  const int n = (int)(row % N), d = (int)(i % D);
  const GateScale c = gate_scale(A_log[n], lower_bound);
  float t;
  const float sg = gate_sigmoid(c, to_f32(g[i]) + dt_bias[(size_t)n * D + d], &t);
  const float h = ex2(c.l2 * sg) * (h0 ? h0[i] : 0.f) + sigmoid(to_f32(beta[row])) * to_f32(x[i]);
  h1[i] = h;
  out[i] = from_f32<T>(h);
}

struct Sizes {
  size_t elem, x, rows, state, params;  // bytes of: an element, x dense, beta dense, a state array
};

Sizes sizes_of(const kda_recurrence_shape_t& s) {
  const size_t rows = (s.layout == KDA_LAYOUT_TND ? (size_t)s.S : (size_t)s.B * s.S) * s.N;
  const size_t e = dtype_bytes(s.dtype);
  return {e, rows * s.D * e, rows * e, (size_t)s.B * s.N * s.D * 4, (size_t)s.N * s.D * 4};
}

// What both passes check: shape, plan, views, pointers, alignment.  Fills p and the input ranges.
kda_status_t prepare(const kda_recurrence_shape_t* shape, const int32_t* plan_host,
                     const int32_t* plan_dev, size_t n_int32, const kda_view_t* x,
                     const kda_view_t* g, const kda_view_t* beta, const float* h0,
                     const float* A_log, const float* dt_bias, float lower_bound, void* workspace,
                     size_t workspace_bytes, bool backward, RecParams* p, ByteRange (&in)[9]) {
  kda_status_t st = validate_recurrence_shape(shape);
  if (st != KDA_OK) return st;
  if (!plan_host || !plan_dev || !x || !g || !beta || !A_log || !dt_bias || !workspace)
    return KDA_ERR_NULL;
  st = validate_recurrence_plan(plan_host, n_int32, shape);
  if (st != KDA_OK) return st;
  if (!(lower_bound >= -5.0f && lower_bound <= 0.0f)) return KDA_ERR_LOWER_BOUND;
  size_t need = 0;
  st = kda_recurrence_workspace_size(plan_host, n_int32, backward, &need);
  if (st != KDA_OK) return st;
  if (workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return KDA_ERR_WORKSPACE;
  for (const void* ptr : {(const void*)h0, (const void*)A_log, (const void*)dt_bias,
                          (const void*)plan_dev})
    if (!aligned16(ptr)) return KDA_ERR_ALIGN;
  const Sizes z = sizes_of(*shape);
  const int nb = shape->layout == KDA_LAYOUT_TND ? 1 : shape->B;
  p->x = *x;
  p->g = *g;
  p->beta = *beta;
  if ((st = check_view(&p->x, nb, shape->N, shape->S, shape->D, z.elem, &in[0])) != KDA_OK ||
      (st = check_view(&p->g, nb, shape->N, shape->S, shape->D, z.elem, &in[1])) != KDA_OK ||
      (st = check_view(&p->beta, nb, shape->N, shape->S, 1, z.elem, &in[2])) != KDA_OK)
    return st;
  in[3] = dense_range(h0, z.state);
  in[4] = dense_range(A_log, (size_t)shape->N * 4);
  in[5] = dense_range(dt_bias, z.params);
  in[6] = dense_range(plan_dev, n_int32 * 4);
  in[7] = dense_range(workspace, need);
  p->plan = plan_dev;
  p->checksum = plan_host[RH_CHECKSUM];
  p->tnd = shape->layout == KDA_LAYOUT_TND;
  p->N = shape->N;
  p->S = shape->S;
  p->D = shape->D;
  p->tiles = plan_host[RH_TILES];
  p->chain = plan_host[RH_CHAIN];
  p->h0 = h0;
  p->A_log = A_log;
  p->dt_bias = dt_bias;
  p->lower_bound = lower_bound;
  p->status = static_cast<int32_t*>(workspace);
  p->od = dense_view(nullptr, shape->layout, shape->N, shape->S, shape->D);
  p->bd = dense_view(nullptr, shape->layout, shape->N, shape->S, 1);
  if (p->tnd) p->od.stride_b = p->bd.stride_b = 0;
  return KDA_OK;
}

size_t states_floats(const int32_t* plan) {
  return (size_t)plan[RH_CHAIN] * plan[RH_N] * plan[RH_D];
}

// every output against every input and every other output
template <int NI, int NO>
bool any_overlap(const ByteRange (&in)[NI], const ByteRange (&out)[NO]) {
  for (int o = 0; o < NO; ++o) {
    for (const ByteRange& r : in)
      if (overlap(r, out[o])) return true;
    for (int q = 0; q < o; ++q)
      if (overlap(out[q], out[o])) return true;
  }
  return false;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status_t kda_recurrence_states_size(const int32_t* plan, size_t n, size_t* floats) {
  if (!floats) return KDA_ERR_NULL;
  const kda_status_t st = validate_recurrence_plan(plan, n, nullptr);
  if (st != KDA_OK) return st;
  *floats = states_floats(plan);
  return KDA_OK;
}

extern "C" kda_status_t kda_recurrence_workspace_size(const int32_t* plan, size_t n,
                                                      int32_t backward, size_t* bytes) {
  if (!bytes) return KDA_ERR_NULL;
  const kda_status_t st = validate_recurrence_plan(plan, n, nullptr);
  if (st != KDA_OK) return st;
  *bytes = kWsHeaderBytes;
  if (backward) *bytes += 2 * (size_t)plan[RH_B] * plan[RH_N] * plan[RH_D] * 4;
  return KDA_OK;
}

extern "C" kda_status_t kda_recurrence_forward(
    const kda_recurrence_shape_t* shape, const int32_t* plan_host, const int32_t* plan_dev,
    size_t n_int32, const kda_view_t* x, const kda_view_t* g, const kda_view_t* beta,
    const float* initial_state, const float* A_log, const float* dt_bias, float lower_bound,
    float* states, void* workspace, size_t workspace_bytes, void* out, float* final_state,
    kda_stream_t stream) {
  RecParams p{};
  ByteRange in[9];
  kda_status_t st = prepare(shape, plan_host, plan_dev, n_int32, x, g, beta, initial_state, A_log,
                            dt_bias, lower_bound, workspace, workspace_bytes, false, &p, in);
  if (st != KDA_OK) return st;
  if (!out || !final_state) return KDA_ERR_NULL;
  if (!aligned16(out) || !aligned16(final_state) || !aligned16(states)) return KDA_ERR_ALIGN;
  const Sizes z = sizes_of(*shape);
  // final_state may be initial_state itself: the tile that reads the start state does so before the
  // tile that writes the end state has its carry
  if (final_state == initial_state) in[3] = ByteRange{};
  const ByteRange outs[] = {dense_range(out, z.x), dense_range(final_state, z.state),
                            dense_range(states, states_floats(plan_host) * 4)};
  if (any_overlap(in, outs)) return KDA_ERR_ALIAS;
  if ((st = check_device()) != KDA_OK) return st;

  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  p.states = states;
  p.out = out;
  p.final_state = final_state;
  if (cudaMemsetAsync(workspace, 0, 8, s) != cudaSuccess) return KDA_ERR_CUDA;
  const unsigned grid = (unsigned)shape->B * shape->N;
  if (shape->dtype == KDA_BF16) rec_forward_kernel<__nv_bfloat16><<<grid, shape->D, 0, s>>>(p);
  else if (shape->dtype == KDA_FP16) rec_forward_kernel<__half><<<grid, shape->D, 0, s>>>(p);
  else rec_forward_kernel<float><<<grid, shape->D, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_recurrence_backward(
    const kda_recurrence_shape_t* shape, const int32_t* plan_host, const int32_t* plan_dev,
    size_t n_int32, const kda_view_t* dout, const float* dfinal_state, const kda_view_t* x,
    const kda_view_t* g, const kda_view_t* beta, const float* initial_state, const float* A_log,
    const float* dt_bias, float lower_bound, const float* states, void* workspace,
    size_t workspace_bytes, void* dx, void* dg, void* dbeta, float* dinitial_state,
    float* dA_log, float* ddt_bias, kda_stream_t stream) {
  RecParams p{};
  ByteRange in[9], r_dout;
  kda_status_t st = prepare(shape, plan_host, plan_dev, n_int32, x, g, beta, initial_state, A_log,
                            dt_bias, lower_bound, workspace, workspace_bytes, true, &p, in);
  if (st != KDA_OK) return st;
  if (!states || !dx || !dg || !dbeta || !dA_log || !ddt_bias) return KDA_ERR_NULL;
  for (const void* ptr : {(const void*)dfinal_state, (const void*)states, (const void*)dx,
                          (const void*)dg, (const void*)dinitial_state, (const void*)dA_log,
                          (const void*)ddt_bias})
    if (!aligned16(ptr)) return KDA_ERR_ALIGN;
  const Sizes z = sizes_of(*shape);
  if (reinterpret_cast<uintptr_t>(dbeta) % z.elem) return KDA_ERR_ALIGN;
  if (dout && dout->data) {
    p.dout = *dout;
    st = check_view(&p.dout, p.tnd ? 1 : shape->B, shape->N, shape->S, shape->D, z.elem, &r_dout);
    if (st != KDA_OK) return st;
  }
  in[8] = dense_range(states, states_floats(plan_host) * 4);
  const ByteRange outs[] = {dense_range(dx, z.x), dense_range(dg, z.x), dense_range(dbeta, z.rows),
                            dense_range(dinitial_state, z.state),
                            dense_range(dA_log, (size_t)shape->N * 4),
                            dense_range(ddt_bias, z.params)};
  const ByteRange grads[] = {r_dout, dense_range(dfinal_state, z.state)};
  if (any_overlap(in, outs) || any_overlap(grads, outs)) return KDA_ERR_ALIAS;
  if ((st = check_device()) != KDA_OK) return st;

  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  p.states = const_cast<float*>(states);
  p.dfinal = dfinal_state;
  p.out = dx;
  p.dg = dg;
  p.dbeta = dbeta;
  p.dh0 = dinitial_state;
  p.part_bias = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kWsHeaderBytes);
  p.part_A = p.part_bias + (size_t)shape->B * shape->N * shape->D;
  if (cudaMemsetAsync(workspace, 0, 8, s) != cudaSuccess) return KDA_ERR_CUDA;
  const unsigned grid = (unsigned)shape->B * shape->N;
  const size_t smem = (size_t)kRecTileElems * 4;
  if (shape->dtype == KDA_BF16) rec_backward_kernel<__nv_bfloat16><<<grid, shape->D, smem, s>>>(p);
  else if (shape->dtype == KDA_FP16) rec_backward_kernel<__half><<<grid, shape->D, smem, s>>>(p);
  else rec_backward_kernel<float><<<grid, shape->D, smem, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
  rec_params_kernel<<<shape->N, shape->D, 0, s>>>(p.part_bias, p.part_A, shape->B, shape->N,
                                                  shape->D, dA_log, ddt_bias);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_recurrence_step(int32_t B, int32_t N, int32_t D, int32_t dtype,
                                            const void* x, const void* g, const void* beta,
                                            const float* state_in, const float* A_log,
                                            const float* dt_bias, float lower_bound, void* out,
                                            float* state_out, kda_stream_t stream) {
  // a step is the recurrence's shape with one token per sequence
  const kda_recurrence_shape_t shape = {KDA_LAYOUT_BSND, B, N, 1, D, dtype};
  kda_status_t st = validate_recurrence_shape(&shape);
  if (st != KDA_OK) return st;
  if (!x || !g || !beta || !A_log || !dt_bias || !out || !state_out) return KDA_ERR_NULL;
  if (!(lower_bound >= -5.0f && lower_bound <= 0.0f)) return KDA_ERR_LOWER_BOUND;
  for (const void* ptr : {x, g, (const void*)state_in, (const void*)A_log, (const void*)dt_bias,
                          (const void*)out, (const void*)state_out})
    if (!aligned16(ptr)) return KDA_ERR_ALIGN;
  const Sizes z = sizes_of(shape);
  if (reinterpret_cast<uintptr_t>(beta) % z.elem) return KDA_ERR_ALIGN;
  const ByteRange in[] = {dense_range(x, z.x), dense_range(g, z.x), dense_range(beta, z.rows),
                          dense_range(A_log, (size_t)N * 4), dense_range(dt_bias, z.params),
                          state_in == state_out ? ByteRange{} : dense_range(state_in, z.state)};
  const ByteRange outs[] = {dense_range(out, z.x), dense_range(state_out, z.state)};
  if (any_overlap(in, outs)) return KDA_ERR_ALIAS;
  if ((st = check_device()) != KDA_OK) return st;

  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const long long total = (long long)B * N * D;
  const long long blocks = (total + 255) / 256;
  if (blocks > INT_MAX) return KDA_ERR_SHAPE;
  auto launch = [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    rec_step_kernel<T><<<(unsigned)blocks, 256, 0, s>>>(
        static_cast<const T*>(x), static_cast<const T*>(g), static_cast<const T*>(beta), state_in,
        A_log, dt_bias, lower_bound, static_cast<T*>(out), state_out, N, D, total);
  };
  if (dtype == KDA_BF16) launch((__nv_bfloat16*)nullptr);
  else if (dtype == KDA_FP16) launch((__half*)nullptr);
  else launch((float*)nullptr);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
