// kda_qk.cu -- RMS norm of query and key heads with a learned weight and the rotation by position,
// in one pass over the data, and its backward pass.
//
// Per row (token, head): r = 1/sqrt(mean(x^2) + eps), n = x r w; the pair i of the first
// rotary_dim channels turns by position * inv_freq[i].  A rotation's gradient is the rotation by
// the opposite angles, so with dn = R^T dy and xh = x r the backward pass is
//     dx = r (dn w - xh mean(dn w xh)),    dw = sum over rows of dn xh.
//
// D/8 lanes hold a row, 8 channels each, chosen so that both channels of a pair lie in one lane: 4
// channels of either half of the turned ones, or 8 in a row.  Such a group of lanes keeps its token
// and walks the token's heads, so a token's cosines and sines are formed once, in registers.  The
// rows of the next steps are on their way to shared memory meanwhile (without them in registers more
// blocks fit a multiprocessor), and only the sums over a row cross lanes.
// Both passes are bound by HBM: 4 bytes a value forward (16-bit), 6 backward.  Forward 4x32x16384
// bf16, 64 heads a token, 344 us: 6.24 TB/s of the 6.47 that a copy reaches; backward of 65536 tokens
// with 40 heads 324 us, 6.2 TB/s.  The weights' gradients are fp32 sums over a block's rows, fp64 from
// there on.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "kda_args.h"
#include "kda_internal.h"
#include "kda_io.cuh"
#include "kda_once.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
// Multiprocessors that the grids are made for.  In the backward pass each block leaves one partial sum
// of the weights' gradients.
constexpr int kSpread = 148;

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
  int turned;      // rotary_dim
  int heads_per;   // heads of one block (grid.y splits the Nq + Nk heads)
  float eps;
  float* part;     // backward: [blocks][2][D] partial weight gradients
};

// Rows of a step (so that their sums over lanes overlap), blocks on a multiprocessor, and the steps
// whose copies a warp has under way or at work.  More of either is slower, and fewer: 4x32x16384
// forward takes 344 us with 3 steps, 371 with 4 and 428 with 2; three blocks took 397, one block 488.
template <class T>
constexpr int kRows = sizeof(T) == 2 ? 2 : 1;
constexpr int kResident = 2;
constexpr int kStages = 3;

template <class T, int D, bool BACKWARD>
constexpr int kQkSmem = kStages * (BACKWARD ? 2 : 1) * kRows<T> * kThreads * 8 * (int)sizeof(T);

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A lane's 8 channels: 4 from `a` on and 4 from `b` on.
using F = Pairs<2>;
struct Eight {
  F a, b;
};
__device__ __forceinline__ Eight operator*(Eight x, Eight y) { return {x.a * y.a, x.b * y.b}; }
__device__ __forceinline__ Eight operator*(Eight x, float y) { return {x.a * y, x.b * y}; }
__device__ __forceinline__ Eight fma(Eight x, Eight y, Eight z) {
  return {fma(x.a, y.a, z.a), fma(x.b, y.b, z.b)};
}
__device__ __forceinline__ float dot(Eight x, Eight y) { return sum(fma(x.a, y.a, x.b * y.b)); }

// A lane's place: its row's group, its part of the row's copy, its channels, and whether they turn.
template <int D, bool INTER>
struct Place {
  static constexpr int kLanes = D / 8;
  static constexpr int kGroups = kThreads / kLanes;
  int lane, group, a, b;
  bool turns;
  __device__ explicit Place(int turned) {
    lane = threadIdx.x % kLanes;
    group = threadIdx.x / kLanes;
    turns = lane * 8 < turned;
    a = lane * 8;
    b = a + 4;
    if (!INTER && turns) {
      a = lane * 4;
      b = turned / 2 + lane * 4;
    }
  }
  template <class T>
  __device__ Eight read(const T* row) const {
    return {load<2>(row + a), load<2>(row + b)};
  }
  template <class T>
  __device__ void write(T* row, const Eight& v) const {
    store(row + a, v.a);
    store(row + b, v.b);
  }
};

// Cosines and sines of the lane's 4 pairs at a position; a lane whose channels do not turn gets ones
// and zeros.
struct Angles {
  F c, s;
};
template <class P>
__device__ __forceinline__ double turn_rate(const QkParams& p, const P& me, int i) {
  constexpr double kInv2Pi = 0.15915494309189533577;
  return me.turns ? (double)__ldg(p.inv_freq + me.lane * 4 + i) * kInv2Pi : 0.0;
}
template <class P>
__device__ __forceinline__ Angles angles(const P& me, const double (&rate)[4], int pos) {
  Angles r{splat<2>(1.f), splat<2>(0.f)};
  if (!me.turns) return r;
  float c[4], s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // whole turns drop out in fp64: the product is off by at most 2^-53 of up to 2^31 radians
    double turns = (double)pos * rate[i];
    turns -= rint(turns);
    sincospif(2.f * (float)turns, &s[i], &c[i]);
  }
  r.c.v[0] = make_float2(c[0], c[1]);
  r.c.v[1] = make_float2(c[2], c[3]);
  r.s.v[0] = make_float2(s[0], s[1]);
  r.s.v[1] = make_float2(s[2], s[3]);
  return r;
}

// The rotation, or its transpose (the angles negated).
template <bool INTER, bool BACK>
__device__ __forceinline__ Eight turn(Eight v, const Angles& t) {
  const F s = BACK ? t.s * -1.f : t.s;
  if constexpr (!INTER) {
    const F n = s * -1.f;
    return {fma(v.a, t.c, v.b * n), fma(v.b, t.c, v.a * s)};
  } else {
    // pairs (2i, 2i + 1): those of v.a take the first two angles
    auto two = [](float2 x, float c, float sn) {
      return make_float2(fmaf(x.x, c, -x.y * sn), fmaf(x.y, c, x.x * sn));
    };
    Eight r;
    r.a.v[0] = two(v.a.v[0], t.c.v[0].x, s.v[0].x);
    r.a.v[1] = two(v.a.v[1], t.c.v[0].y, s.v[0].y);
    r.b.v[0] = two(v.b.v[0], t.c.v[1].x, s.v[1].x);
    r.b.v[1] = two(v.b.v[1], t.c.v[1].y, s.v[1].y);
    return r;
  }
}

// this lane's 8 weights of a side
template <class P>
__device__ __forceinline__ Eight load_weight(const QkSide& a, const P& me) {
  Eight w{splat<2>(1.f), splat<2>(1.f)};
  if (!a.w) return w;
  auto four = [](const float* f) {  // of any address
    F r;
    r.v[0] = make_float2(__ldg(f), __ldg(f + 1));
    r.v[1] = make_float2(__ldg(f + 2), __ldg(f + 3));
    return r;
  };
  return {four(a.w + me.a), four(a.w + me.b)};
}

// the heads [lo, hi) of a side that a block of this grid.y works on
__device__ __forceinline__ void head_range(const QkParams& p, int side, int* lo, int* hi) {
  const int before = side ? p.side[0].heads : 0, n = p.side[side].heads;
  *lo = max(0, (int)blockIdx.y * p.heads_per - before);
  *hi = min(n, ((int)blockIdx.y + 1) * p.heads_per - before);
}

// A token of a group: its slot and its place there.
struct Token {
  long long b;
  int s;
  bool mine;
  __device__ Token(const QkParams& p, long long t) {
    mine = t < p.tokens;
    if (!mine) t = 0;
    b = p.tokens <= UINT32_MAX ? (uint32_t)t / (uint32_t)p.S : t / p.S;
    s = (int)(t - b * p.S);
  }
};
// Its position where positions are given; it is asked for a token ahead, so that nothing waits for it.
__device__ __forceinline__ int given_position(const QkParams& p, long long t) {
  return p.positions && t < p.tokens ? __ldg(p.positions + t) : 0;
}

// The copies that run ahead: a warp's way through its groups' tokens, sides and heads, kRows heads of
// one side a step.  The bounds are the block's, so that a warp's lanes stay together.
template <class T, int D, bool INTER, bool BACKWARD>
struct Ahead {
  using P = Place<D, INTER>;
  static constexpr int U = kRows<T>, kTensors = BACKWARD ? 2 : 1;
  static constexpr int kRowBytes = D * (int)sizeof(T), kCopies = (int)sizeof(T) / 2;
  long long t0;
  int side, h, end, next_pos, s;
  long long b;  // the token's slot, s its place there
  bool done, live;
  const char *x, *y;

  __device__ void enter(const QkParams& p, const P& me) {
    const QkSide& a = p.side[side];
    head_range(p, side, &h, &end);
    x = static_cast<const char*>(a.x.data) +
        (b * a.x.stride_b + s * a.x.stride_s + h * a.x.stride_n) * (long long)sizeof(T) +
        me.lane * 16;
    if (BACKWARD)
      y = static_cast<const char*>(a.dy.data) +
          (b * a.dy.stride_b + s * a.dy.stride_s + h * a.dy.stride_n) * (long long)sizeof(T) +
          me.lane * 16;
  }
  // at a token: its first side with heads
  __device__ void arrive(const QkParams& p, const P& me) {
    done = t0 >= p.tokens;
    if (done) return;
    const Token t(p, t0 + me.group);
    b = t.b;
    s = t.s;
    live = t.mine && next_pos >= 0;
    next_pos = given_position(p, t0 + me.group + (long long)gridDim.x * P::kGroups);
    side = 0;
    enter(p, me);
    if (h >= end) {
      side = 1;
      enter(p, me);
    }
  }
  __device__ void begin(const QkParams& p, const P& me) {
    x = y = nullptr;
    t0 = (long long)blockIdx.x * P::kGroups;
    next_pos = given_position(p, t0 + me.group);
    arrive(p, me);
  }
  // Starts the copies of a step; rows of padding become zeros.
  __device__ void issue(const QkParams& p, const P& me, uint32_t stage) {
    if (!done) {
      const QkSide& a = p.side[side];
      uint32_t to = stage + me.group * kRowBytes + me.lane * 16;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int bytes = live && h + u < end ? 16 : 0;
#pragma unroll
        for (int c = 0; c < kCopies; ++c) {
          copy16(to + c * 16 * P::kLanes, x + c * 16 * P::kLanes, bytes);
          if (BACKWARD)
            copy16(to + kThreads * 16 * kCopies + c * 16 * P::kLanes, y + c * 16 * P::kLanes, bytes);
        }
        to += kTensors * kThreads * 16 * kCopies;
        x += a.x.stride_n * (long long)sizeof(T);
        if (BACKWARD) y += a.dy.stride_n * (long long)sizeof(T);
      }
      h += U;
      if (h >= end && side == 0) {
        side = 1;
        enter(p, me);
      }
      if (h >= end) {
        t0 += (long long)gridDim.x * P::kGroups;
        arrive(p, me);
      }
    }
    copies_issued();
  }
  // 16 bytes, or zeros where `bytes` is 0
  __device__ static void copy16(uint32_t to, const char* from, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes)
                 : "memory");
  }
};

template <class T, int D, bool INTER, bool BACKWARD>
__global__ void __launch_bounds__(kThreads, kResident)
    qk_kernel(const __grid_constant__ QkParams p) {
  using P = Place<D, INTER>;
  constexpr int U = kRows<T>, kTensors = BACKWARD ? 2 : 1;
  constexpr int kTensor = kThreads * 8, kStage = U * kTensors * kTensor;  // elements
  extern __shared__ __align__(16) uint8_t smem[];
  T* const ring = reinterpret_cast<T*>(smem);  // [kStages][U][kTensors][kGroups][D]
  const P me(p.turned);
  Ahead<T, D, INTER, BACKWARD> ahead;
  ahead.begin(p, me);
  for (int i = 0; i < kStages - 1; ++i) ahead.issue(p, me, smem_u32(ring + i * kStage));
  launch_dependents();
  // The forward pass keeps both sides' weights and the frequencies in registers; the backward pass has
  // none left, and reads them again for every token.
  Eight dw[2], weights[2];
  double rate[4];  // turns for a position
  if (!BACKWARD) {
    for (int i = 0; i < 2; ++i) weights[i] = load_weight(p.side[i], me);
    for (int i = 0; i < 4; ++i) rate[i] = turn_rate(p, me, i);
  }
  if (BACKWARD)
    for (int i = 0; i < 2; ++i) dw[i] = {splat<2>(0.f), splat<2>(0.f)};
  int stage = 0, free = kStages - 1, next_pos = given_position(p, (long long)blockIdx.x * P::kGroups + me.group);
  for (long long t0 = (long long)blockIdx.x * P::kGroups; t0 < p.tokens;
       t0 += (long long)gridDim.x * P::kGroups) {
    const Token t(p, t0 + me.group);
    const int pos = p.positions ? next_pos : t.s;
    next_pos = given_position(p, t0 + me.group + (long long)gridDim.x * P::kGroups);
    const bool live = t.mine && pos >= 0;
    if (BACKWARD)
      for (int i = 0; i < 4; ++i) rate[i] = turn_rate(p, me, i);
    const Angles turns = angles(me, rate, live ? pos : 0);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const QkSide& a = p.side[side];
      int h, end;
      head_range(p, side, &h, &end);
      if (h >= end) continue;
      const Eight w = BACKWARD ? load_weight(a, me) : weights[side];
      T* to = static_cast<T*>(a.out) + t.b * a.od.stride_b + t.s * a.od.stride_s +
              h * a.od.stride_n;
      for (; h < end; h += U) {
        copies_arrived<kStages - 2>();
        ahead.issue(p, me, smem_u32(ring + free * kStage));
        free = free + 1 == kStages ? 0 : free + 1;
        const T* row = ring + stage * kStage + me.group * D;
        stage = stage + 1 == kStages ? 0 : stage + 1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          Eight x = me.read(row);
          const float norm = rsqrtf(group_sum<P::kLanes>(dot(x, x)) * (1.f / D) + p.eps);
          if constexpr (!BACKWARD) {
            x = turn<INTER, false>(x * norm * w, turns);
          } else {
            const float r = live && h + u < end ? norm : 0.f;  // eps may be 0
            Eight dn = turn<INTER, true>(me.read(row + kTensor), turns);
            x = x * r;
            dw[side] = fma(dn, x, dw[side]);
            dn = dn * w;
            const float m = group_sum<P::kLanes>(dot(dn, x)) * (-1.f / D);
            const F m2 = splat<2>(m);
            x = Eight{fma(x.a, m2, dn.a), fma(x.b, m2, dn.b)} * r;
          }
          if (!live) x = {splat<2>(0.f), splat<2>(0.f)};
          if (t.mine && h + u < end) me.write(to, x);
          to += a.od.stride_n;
          row += kTensors * kTensor;
        }
      }
    }
  }
  if constexpr (BACKWARD) {
    float* const red = reinterpret_cast<float*>(smem);  // [kGroups][D]
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      __syncthreads();
      me.write(red + me.group * D, dw[side]);
      __syncthreads();
      if (threadIdx.x < D) {
        float sum = 0.f;
#pragma unroll
        for (int g = 0; g < P::kGroups; ++g) sum += red[g * D + threadIdx.x];
        const size_t block = (size_t)blockIdx.y * gridDim.x + blockIdx.x;
        p.part[(block * 2 + side) * D + threadIdx.x] = sum;
      }
    }
  }
}

// The blocks' partial sums in a fixed order, in fp64: 128 threads for a channel, then a warp.
constexpr int kSumChannels = 8;
template <int D>
__global__ void __launch_bounds__(1024) qk_weights_kernel(const float* part, int blocks, float* dwq,
                                                          float* dwk) {
  constexpr int kRows = 1024 / kSumChannels;
  __shared__ double red[kSumChannels][kRows];
  const int c = threadIdx.x % kSumChannels, row = threadIdx.x / kSumChannels, side = blockIdx.y;
  float* const dw = side ? dwk : dwq;
  if (!dw) return;
  wait_dependencies();
  double sum = 0;
#pragma unroll 4
  for (int i = row; i < blocks; i += kRows)
    sum += part[((size_t)i * 2 + side) * D + blockIdx.x * kSumChannels + c];
  red[c][row] = sum;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp >= kSumChannels) return;
  sum = 0;
#pragma unroll
  for (int i = lane; i < kRows; i += 32) sum += red[warp][i];
  sum = warp_sum(sum);
  if (lane == 0) dw[blockIdx.x * kSumChannels + warp] = (float)sum;
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
  p->turned = s->rotary_dim;
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

// Launches a pass; blocks that share a token's heads lie along y.
template <class T, int D, bool INTER, bool BACKWARD>
struct Pass {
  static void run(dim3 grid, const QkParams& p, cudaStream_t s, cudaError_t* e) {
    static PerDevice once;
    constexpr int kSmem = kQkSmem<T, D, BACKWARD>;
    const auto kernel = qk_kernel<T, D, INTER, BACKWARD>;
    int dev = 0, unused;
    *e = cudaGetDevice(&dev);
    if (*e != cudaSuccess) return;
    *e = once_per_device(once, dev, &unused, [&](int, int*) {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    });
    if (*e != cudaSuccess) return;
    kernel<<<grid, kThreads, kSmem, s>>>(p);
    *e = cudaGetLastError();
  }
};
template <class T, int D, bool INTER>
using Forward = Pass<T, D, INTER, false>;
template <class T, int D, bool INTER>
using Backward = Pass<T, D, INTER, true>;

// The grid: blocks over tokens and, where that takes less time, over the heads of a token.  A block's
// turn over its groups' tokens costs its steps over the heads and about four more to begin with
// (positions, angles, the first copies).
dim3 grid_of(const kda_qk_shape_t& s, int most, QkParams* p) {
  const int groups = kThreads / (s.D / 8), heads = s.Nq + s.Nk, rows = s.dtype == KDA_FP32 ? 1 : 2;
  const long long blocks = (p->tokens + groups - 1) / groups;
  long long least = LLONG_MAX;
  dim3 grid;
  for (int want = 1; want <= std::min(heads, most); ++want) {
    const int per = (heads + want - 1) / want, splits = (heads + per - 1) / per;
    const long long across = std::min<long long>(blocks, most / splits);
    const long long cost = (blocks + across - 1) / across * (4 + (per + rows - 1) / rows);
    if (cost < least) {
      least = cost;
      grid = dim3((unsigned)across, (unsigned)splits);
      p->heads_per = per;
    }
  }
  return grid;
}

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
  const dim3 grid = grid_of(*shape, kSpread * kResident, &p);
  cudaError_t e = cudaSuccess;
  dispatch<Forward>(*shape, grid, p, reinterpret_cast<cudaStream_t>(stream), &e);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_qk_norm_rope_workspace_size(const kda_qk_shape_t* shape,
                                                        size_t* bytes) {
  if (!bytes) return KDA_ERR_NULL;
  const kda_status_t st = validate(shape);
  if (st != KDA_OK) return st;
  *bytes = (size_t)kSpread * kResident * 2 * shape->D * 4;
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
  const dim3 grid = grid_of(*shape, kSpread * kResident, &p);
  p.part = static_cast<float*>(workspace);
  const cudaStream_t stm = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t err = cudaSuccess;
  dispatch<Backward>(*shape, grid, p, stm, &err);
  if (err != cudaSuccess) return KDA_ERR_CUDA;
  if (dq_weight || dk_weight)
    err = launch_early(shape->D == 128 ? qk_weights_kernel<128> : qk_weights_kernel<64>,
                       dim3(shape->D / kSumChannels, 2), 1024, 0, stm, p.part, (int)(grid.x * grid.y),
                       dq_weight, dk_weight);
  return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
