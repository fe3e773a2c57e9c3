// kda_qk.cu -- RMS norm of query and key heads with a learned weight and the rotation by position,
// in one pass over the data, and its backward pass.
//
// Per row (token, head): r = 1/sqrt(mean(x^2) + eps), n = x r w; the pair i of the first
// rotary_dim channels turns by position * inv_freq[i].  A rotation's gradient is the rotation by
// the opposite angles, so with dn = R^T dy and xh = x r the backward pass is
//     dx = r (dn w - xh mean(dn w xh)),    dw = sum over rows of dn xh.
//
// D/8 lanes hold a row, 8 channels each: one 16-byte access per lane and row (two for fp32), the
// row's sums and the exchange of half-split pairs by shuffles.  Such a group of lanes keeps its
// token and walks the token's heads, so a token's cosines and sines are formed once, in registers.
// Both passes are bound by HBM: 4 bytes a value forward (16-bit), 6 backward.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "kda_args.h"
#include "kda_internal.h"
#include "kda_io.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
// Blocks of the backward pass at most; each leaves one partial sum of the weights' gradients.
constexpr int kMaxBlocks = 592;
// Blocks wanted before heads stop being split over blocks (about two for each SM).
constexpr int kWantBlocks = 296;

struct QkSide {
  kda_view_t x, dy;  // dy: backward only
  const float* w;    // null: ones
  void* out;         // forward: the output; backward: dx
  kda_view_t od;     // strides of out (dense)
  int heads;
};

struct QkParams {
  QkSide side[2];  // queries, keys
  const int32_t* positions;
  const float* inv_freq;
  long long tokens;
  int S;
  int turned8;     // rotary_dim / 16: chunks of 8 channels in one half of the turned channels
  int heads_per;   // heads of one block (grid.y splits the Nq + Nk heads)
  float eps;
  float* part;     // backward: [blocks][2][D] partial weight gradients
};

// 8 consecutive channels as they lie in memory
template <class T>
struct Vec8 {
  Vec4<T> lo, hi;
};
// plain loads: a row may be turned in place
template <class T>
__device__ __forceinline__ Vec8<T> ld8(const T* p) {
  Vec8<T> v;
  if constexpr (sizeof(T) == 2) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    v.lo.w = make_uint2(w.x, w.y);
    v.hi.w = make_uint2(w.z, w.w);
  } else {
    v.lo.w = *reinterpret_cast<const float4*>(p);
    v.hi.w = *reinterpret_cast<const float4*>(p + 4);
  }
  return v;
}
template <class T>
__device__ __forceinline__ void widen8(const Vec8<T>& v, float (&x)[8]) {
  float a[4], b[4];
  widen(v.lo, a);
  widen(v.hi, b);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = a[e];
    x[4 + e] = b[e];
  }
}
template <class T>
__device__ __forceinline__ void st8(T* p, const float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    const float a[4] = {x[0], x[1], x[2], x[3]}, b[4] = {x[4], x[5], x[6], x[7]};
    uint4 w;
    st4(reinterpret_cast<T*>(&w.x), a);
    st4(reinterpret_cast<T*>(&w.z), b);
    *reinterpret_cast<uint4*>(p) = w;
  } else {
    const float a[4] = {x[0], x[1], x[2], x[3]}, b[4] = {x[4], x[5], x[6], x[7]};
    st4(p, a);
    st4(p + 4, b);
  }
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Cosine and signed sine of this lane's channels at a position: out = own * cs + partner * sn.
// Channels that do not turn get 1 and 0.
template <bool INTER>
__device__ __forceinline__ void angles(const QkParams& p, int chunk, int pos, float (&cs)[8],
                                       float (&sn)[8]) {
  constexpr double kInv2Pi = 0.15915494309189533577;
  constexpr int kPairs = INTER ? 4 : 8;
  const bool second = !INTER && chunk >= p.turned8;
  const int first = INTER ? chunk * 4 : (second ? chunk - p.turned8 : chunk) * 8;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cs[e] = 1.f;
    sn[e] = 0.f;
  }
  if (chunk >= 2 * p.turned8) return;
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    // whole turns drop out in fp64: the product is off by at most 2^-53 of up to 2^31 radians
    double turns = (double)pos * ((double)__ldg(p.inv_freq + first + i) * kInv2Pi);
    turns -= rint(turns);
    float s, c;
    sincospif(2.f * (float)turns, &s, &c);
    if (INTER) {
      cs[2 * i] = cs[2 * i + 1] = c;
      sn[2 * i] = -s;
      sn[2 * i + 1] = s;
    } else {
      cs[i] = c;
      sn[i] = second ? s : -s;
    }
  }
}

// own * cs + DIR * partner * sn: the rotation (DIR = 1) or its transpose (-1)
template <bool INTER, int DIR>
__device__ __forceinline__ void turn(float (&v)[8], const float (&cs)[8], const float (&sn)[8],
                                     int partner_lane) {
  float o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    o[e] = INTER ? v[e ^ 1] : __shfl_sync(0xffffffffu, v[e], partner_lane);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = fmaf(v[e], cs[e], (DIR > 0 ? o[e] : -o[e]) * sn[e]);
}

template <int D>
struct Place {
  static constexpr int kLanes = D / 8;
  static constexpr int kGroups = kThreads / kLanes;
  int chunk, group, partner;
  __device__ explicit Place(int turned8) {
    chunk = threadIdx.x % kLanes;
    group = threadIdx.x / kLanes;
    const int other = chunk < turned8 ? chunk + turned8
                                      : (chunk < 2 * turned8 ? chunk - turned8 : chunk);
    partner = (threadIdx.x & 31) - chunk + other;
  }
};

// this lane's 8 weights of a side
template <int D>
__device__ __forceinline__ void load_weight(const QkSide& a, int chunk, float (&w)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = a.w ? __ldg(a.w + chunk * 8 + e) : 1.f;
}

// the heads [lo, hi) of a side that a block of this grid.y works on
__device__ __forceinline__ void head_range(const QkParams& p, int side, int* lo, int* hi) {
  const int before = side ? p.side[0].heads : 0, n = p.side[side].heads;
  *lo = max(0, (int)blockIdx.y * p.heads_per - before);
  *hi = min(n, ((int)blockIdx.y + 1) * p.heads_per - before);
}

template <class T, int D, bool INTER>
__global__ void __launch_bounds__(kThreads) qk_forward_kernel(const QkParams p) {
  using P = Place<D>;
  constexpr int U = sizeof(T) == 2 ? 4 : 2;  // rows requested before the first is used
  const P me(p.turned8);
  const long long tk = (long long)blockIdx.x * P::kGroups + me.group;
  const bool mine = tk < p.tokens;
  const long long b = mine ? tk / p.S : 0;
  const int s = (int)(mine ? tk - b * p.S : 0);
  const int pos = !mine ? -1 : (p.positions ? __ldg(p.positions + tk) : s);
  const bool live = pos >= 0;
  float cs[8], sn[8];
  angles<INTER>(p, me.chunk, live ? pos : 0, cs, sn);
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const QkSide& a = p.side[side];
    int h, end;
    head_range(p, side, &h, &end);
    float w[8];
    if (h < end) load_weight<D>(a, me.chunk, w);
    const T* src = static_cast<const T*>(a.x.data) + b * a.x.stride_b + s * a.x.stride_s +
                   me.chunk * 8;
    T* dst = static_cast<T*>(a.out) + b * a.od.stride_b + s * a.od.stride_s + me.chunk * 8;
    for (; h < end; h += U) {
      Vec8<T> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        raw[u] = Vec8<T>{};
        if (live && h + u < end) raw[u] = ld8(src + (h + u) * a.x.stride_n);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h + u >= end) break;
        float x[8];
        widen8(raw[u], x);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
        const float r = rsqrtf(group_sum<P::kLanes>(ss) * (1.f / D) + p.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * r * w[e];
        turn<INTER, 1>(x, cs, sn, me.partner);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = live ? x[e] : 0.f;
        if (mine) st8(dst + (h + u) * a.od.stride_n, x);
      }
    }
  }
}

template <class T, int D, bool INTER>
__global__ void __launch_bounds__(kThreads) qk_backward_kernel(const QkParams p) {
  using P = Place<D>;
  constexpr int U = 2;
  __shared__ float red[P::kGroups][D];
  const P me(p.turned8);
  float dw[2][8] = {};
  // the loop's bounds are the block's, so that a warp's lanes stay together for the shuffles
  for (long long t0 = (long long)blockIdx.x * P::kGroups; t0 < p.tokens;
       t0 += (long long)gridDim.x * P::kGroups) {
    const long long tk = t0 + me.group;
    const bool mine = tk < p.tokens;
    const long long b = mine ? tk / p.S : 0;
    const int s = (int)(mine ? tk - b * p.S : 0);
    const int pos = !mine ? -1 : (p.positions ? __ldg(p.positions + tk) : s);
    const bool live = pos >= 0;
    float cs[8], sn[8];
    angles<INTER>(p, me.chunk, live ? pos : 0, cs, sn);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const QkSide& a = p.side[side];
      int h, end;
      head_range(p, side, &h, &end);
      float w[8];
      if (h < end) load_weight<D>(a, me.chunk, w);
      const T* xs = static_cast<const T*>(a.x.data) + b * a.x.stride_b + s * a.x.stride_s +
                    me.chunk * 8;
      const T* ys = static_cast<const T*>(a.dy.data) + b * a.dy.stride_b + s * a.dy.stride_s +
                    me.chunk * 8;
      T* dst = static_cast<T*>(a.out) + b * a.od.stride_b + s * a.od.stride_s + me.chunk * 8;
      for (; h < end; h += U) {
        Vec8<T> rx[U], ry[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          rx[u] = ry[u] = Vec8<T>{};
          if (live && h + u < end) {
            rx[u] = ld8(xs + (h + u) * a.x.stride_n);
            ry[u] = ld8(ys + (h + u) * a.dy.stride_n);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (h + u >= end) break;
          float x[8], dn[8];
          widen8(rx[u], x);
          widen8(ry[u], dn);
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
          const float norm = rsqrtf(group_sum<P::kLanes>(ss) * (1.f / D) + p.eps);
          const float r = live ? norm : 0.f;  // eps may be 0
          turn<INTER, -1>(dn, cs, sn, me.partner);
          float dot = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] *= r;
            dn[e] = live ? dn[e] : 0.f;
            dw[side][e] = fmaf(dn[e], x[e], dw[side][e]);
            dn[e] *= w[e];
            dot = fmaf(dn[e], x[e], dot);
          }
          dot = group_sum<P::kLanes>(dot) * (1.f / D);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = live ? r * (dn[e] - x[e] * dot) : 0.f;
          if (mine) st8(dst + (h + u) * a.od.stride_n, x);
        }
      }
    }
  }
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) red[me.group][me.chunk * 8 + e] = dw[side][e];
    __syncthreads();
    if (threadIdx.x < D) {
      float sum = 0.f;
#pragma unroll
      for (int g = 0; g < P::kGroups; ++g) sum += red[g][threadIdx.x];
      const size_t block = (size_t)blockIdx.y * gridDim.x + blockIdx.x;
      p.part[(block * 2 + side) * D + threadIdx.x] = sum;
    }
  }
}

// The blocks' partial sums in a fixed order, in fp64: 8 threads for a channel, then those 8.
template <int D>
__global__ void qk_weights_kernel(const float* part, int blocks, float* dwq, float* dwk) {
  __shared__ double red[8][32];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int d = blockIdx.x * 32 + lane, side = blockIdx.y;
  float* dw = side ? dwk : dwq;
  if (!dw) return;
  double sum = 0;
  for (int i = row; i < blocks; i += 8) sum += part[((size_t)i * 2 + side) * D + d];
  red[row][lane] = sum;
  __syncthreads();
  if (row == 0) {
    for (int i = 1; i < 8; ++i) sum += red[i][lane];
    dw[d] = (float)sum;
  }
}

kda_status_t validate(const kda_qk_shape_t* s) {
  if (!s) return KDA_ERR_NULL;
  if (s->layout < KDA_LAYOUT_BNSD || s->layout > KDA_LAYOUT_TND) return KDA_ERR_LAYOUT;
  if (s->D != 128 && s->D != 64) return KDA_ERR_DIM;
  if (s->rotary_dim < 0 || s->rotary_dim > s->D || s->rotary_dim % 16) return KDA_ERR_DIM;
  if (s->dtype < KDA_BF16 || s->dtype > KDA_FP32) return KDA_ERR_DTYPE;
  if (s->Nq < 1 || s->Nk < 1) return KDA_ERR_HEADS;
  if ((s->layout != KDA_LAYOUT_TND && s->B < 1) || s->S < 1) return KDA_ERR_SHAPE;
  if (s->interleaved != 0 && s->interleaved != 1) return KDA_ERR_SHAPE;
  if (!std::isfinite(s->eps) || s->eps < 0.f) return KDA_ERR_SHAPE;
  const long long tokens = (s->layout == KDA_LAYOUT_TND ? 1LL : s->B) * s->S;
  const long long heads = (long long)s->Nq + s->Nk;
  if (heads > 65535 || tokens > (1LL << 34) || tokens * heads > (1LL << 46) / s->D)
    return KDA_ERR_SHAPE;
  return KDA_OK;
}

int batches(const kda_qk_shape_t& s) { return s.layout == KDA_LAYOUT_TND ? 1 : s.B; }

// Checks and fills what both passes share: `in` gets the ranges of positions, inv_freq and the
// weights, x_range those of q and k.
kda_status_t prepare(const kda_qk_shape_t* s, const kda_view_t* q, const kda_view_t* k,
                     const int32_t* positions, const float* inv_freq, const float* qw,
                     const float* kw, void* out_q, void* out_k, QkParams* p, ByteRange (&x_range)[2],
                     ByteRange (&in)[4], ByteRange (&out)[2]) {
  kda_status_t st = validate(s);
  if (st != KDA_OK) return st;
  if (!q || !k || !out_q || !out_k || (s->rotary_dim > 0 && !inv_freq)) return KDA_ERR_NULL;
  const size_t e = dtype_bytes(s->dtype);
  const int nb = batches(*s);
  p->tokens = (long long)nb * s->S;
  p->S = s->S;
  p->turned8 = s->rotary_dim / 16;
  p->eps = s->eps;
  p->positions = positions;
  p->inv_freq = inv_freq;
  const kda_view_t* x[] = {q, k};
  const float* w[] = {qw, kw};
  void* o[] = {out_q, out_k};
  const int heads[] = {s->Nq, s->Nk};
  for (int i = 0; i < 2; ++i) {
    QkSide& a = p->side[i];
    a.heads = heads[i];
    a.x = *x[i];
    a.w = w[i];
    a.out = o[i];
    a.od = dense_view(nullptr, s->layout, heads[i], s->S, s->D);
    if (nb <= 1) a.od.stride_b = 0;
    st = check_view(&a.x, nb, heads[i], s->S, s->D, e, &x_range[i]);
    if (st != KDA_OK) return st;
    if (!aligned16(o[i]) || (reinterpret_cast<uintptr_t>(w[i]) & 3u)) return KDA_ERR_ALIGN;
    out[i] = dense_range(o[i], (size_t)p->tokens * heads[i] * s->D * e);
    in[i] = dense_range(w[i], (size_t)s->D * 4);
  }
  if ((reinterpret_cast<uintptr_t>(positions) & 3u) || (reinterpret_cast<uintptr_t>(inv_freq) & 3u))
    return KDA_ERR_ALIGN;
  in[2] = dense_range(positions, (size_t)p->tokens * 4);
  in[3] = dense_range(inv_freq, (size_t)s->rotary_dim * 2);
  return KDA_OK;
}

// Whether a view is exactly the dense tensor `out`: the one overlap that is allowed, since every
// lane reads its channels of a row before it writes them.
bool same_tensor(const kda_view_t& v, const QkSide& a, int nb, int S) {
  return v.data == a.out && (nb <= 1 || v.stride_b == a.od.stride_b) &&
         (a.heads <= 1 || v.stride_n == a.od.stride_n) && (S <= 1 || v.stride_s == a.od.stride_s);
}

// Heads of one block: all of a token's, unless that leaves SMs without a block.
int heads_per_block(const QkParams& p, long long token_blocks) {
  const int heads = p.side[0].heads + p.side[1].heads;
  const long long split = std::min<long long>(heads, (kWantBlocks + token_blocks - 1) / token_blocks);
  return (int)((heads + split - 1) / split);
}

template <template <class, int, bool> class K, class... A>
void dispatch(const kda_qk_shape_t& s, A&&... a) {
  auto with_type = [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    if (s.D == 128) s.interleaved ? K<T, 128, true>::run(a...) : K<T, 128, false>::run(a...);
    else s.interleaved ? K<T, 64, true>::run(a...) : K<T, 64, false>::run(a...);
  };
  if (s.dtype == KDA_BF16) with_type((__nv_bfloat16*)nullptr);
  else if (s.dtype == KDA_FP16) with_type((__half*)nullptr);
  else with_type((float*)nullptr);
}

template <class T, int D, bool INTER>
struct Forward {
  static void run(dim3 grid, const QkParams& p, cudaStream_t s) {
    qk_forward_kernel<T, D, INTER><<<grid, kThreads, 0, s>>>(p);
  }
};
template <class T, int D, bool INTER>
struct Backward {
  static void run(dim3 grid, const QkParams& p, cudaStream_t s) {
    qk_backward_kernel<T, D, INTER><<<grid, kThreads, 0, s>>>(p);
  }
};

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status_t kda_qk_norm_rope(const kda_qk_shape_t* shape, const kda_view_t* q,
                                         const kda_view_t* k, const int32_t* positions,
                                         const float* inv_freq, const float* q_weight,
                                         const float* k_weight, void* q_out, void* k_out,
                                         kda_stream_t stream) {
  QkParams p{};
  ByteRange x[2], in[4], out[2];
  kda_status_t st = prepare(shape, q, k, positions, inv_freq, q_weight, k_weight, q_out, k_out, &p,
                            x, in, out);
  if (st != KDA_OK) return st;
  const int nb = batches(*shape);
  for (int i = 0; i < 2; ++i) {
    for (const ByteRange& r : in)
      if (overlap(r, out[i])) return KDA_ERR_ALIAS;
    for (int j = 0; j < 2; ++j)
      if (overlap(x[j], out[i]) && !(i == j && same_tensor(p.side[i].x, p.side[i], nb, shape->S)))
        return KDA_ERR_ALIAS;
  }
  if (overlap(out[0], out[1])) return KDA_ERR_ALIAS;
  if ((st = check_device()) != KDA_OK) return st;
  const int groups = kThreads / (shape->D / 8);
  const long long blocks = (p.tokens + groups - 1) / groups;
  if (blocks > INT_MAX) return KDA_ERR_SHAPE;
  p.heads_per = heads_per_block(p, blocks);
  const int heads = shape->Nq + shape->Nk;
  const dim3 grid((unsigned)blocks, (unsigned)((heads + p.heads_per - 1) / p.heads_per));
  dispatch<Forward>(*shape, grid, p, reinterpret_cast<cudaStream_t>(stream));
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_qk_norm_rope_workspace_size(const kda_qk_shape_t* shape,
                                                        size_t* bytes) {
  if (!bytes) return KDA_ERR_NULL;
  const kda_status_t st = validate(shape);
  if (st != KDA_OK) return st;
  *bytes = (size_t)kMaxBlocks * 2 * shape->D * 4;
  return KDA_OK;
}

extern "C" kda_status_t kda_qk_norm_rope_backward(
    const kda_qk_shape_t* shape, const kda_view_t* dq_out, const kda_view_t* dk_out,
    const kda_view_t* q, const kda_view_t* k, const int32_t* positions, const float* inv_freq,
    const float* q_weight, const float* k_weight, void* workspace, size_t workspace_bytes,
    void* dq, void* dk, float* dq_weight, float* dk_weight, kda_stream_t stream) {
  QkParams p{};
  ByteRange x[2], in[4], out[2], dy[2];
  kda_status_t st = prepare(shape, q, k, positions, inv_freq, q_weight, k_weight, dq, dk, &p, x, in,
                            out);
  if (st != KDA_OK) return st;
  if (!dq_out || !dk_out || !workspace) return KDA_ERR_NULL;
  size_t need = 0;
  kda_qk_norm_rope_workspace_size(shape, &need);
  if (workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return KDA_ERR_WORKSPACE;
  const size_t e = dtype_bytes(shape->dtype);
  const int nb = batches(*shape);
  const kda_view_t* d[] = {dq_out, dk_out};
  for (int i = 0; i < 2; ++i) {
    p.side[i].dy = *d[i];
    st = check_view(&p.side[i].dy, nb, p.side[i].heads, shape->S, shape->D, e, &dy[i]);
    if (st != KDA_OK) return st;
  }
  if ((reinterpret_cast<uintptr_t>(dq_weight) & 3u) || (reinterpret_cast<uintptr_t>(dk_weight) & 3u))
    return KDA_ERR_ALIGN;
  const size_t wb = (size_t)shape->D * 4;
  const ByteRange outs[] = {out[0], out[1], dense_range(dq_weight, wb), dense_range(dk_weight, wb),
                            dense_range(workspace, need)};
  const ByteRange ins[] = {x[0], x[1], in[0], in[1], in[2], in[3]};
  for (int i = 0; i < 5; ++i) {
    for (const ByteRange& r : ins)
      if (overlap(r, outs[i])) return KDA_ERR_ALIAS;
    for (int j = 0; j < 2; ++j)
      if (overlap(dy[j], outs[i]) &&
          !(i == j && same_tensor(p.side[j].dy, p.side[j], nb, shape->S)))
        return KDA_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[j], outs[i])) return KDA_ERR_ALIAS;
  }
  if ((st = check_device()) != KDA_OK) return st;
  const int groups = kThreads / (shape->D / 8);
  const int heads = shape->Nq + shape->Nk;
  const long long want = std::min<long long>((p.tokens + groups - 1) / groups, kMaxBlocks);
  p.heads_per = heads_per_block(p, want);
  const int splits = (heads + p.heads_per - 1) / p.heads_per;
  const int across = (int)std::min<long long>(want, std::max(1, kMaxBlocks / splits));
  p.part = static_cast<float*>(workspace);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  dispatch<Backward>(*shape, dim3((unsigned)across, (unsigned)splits), p, s);
  if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
  if (dq_weight || dk_weight) {
    const dim3 grid(shape->D / 32, 2);
    if (shape->D == 128) qk_weights_kernel<128><<<grid, 256, 0, s>>>(p.part, across * splits, dq_weight, dk_weight);
    else qk_weights_kernel<64><<<grid, 256, 0, s>>>(p.part, across * splits, dq_weight, dk_weight);
  }
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
