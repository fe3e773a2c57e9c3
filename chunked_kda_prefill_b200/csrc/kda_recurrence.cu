// kda_recurrence.cu -- the gated recurrence, the vector form of the KDA state:
//     a_t = exp(lb sigmoid(e^A (g_t + bias))),  h_t = a_t h_{t-1} + sigmoid(beta_t) x_t.
//
// A run of tokens maps its start state to its end state by h -> A h + H, with A the product of its
// decays, and such maps compose.  So a sequence is cut into tiles that blocks work on at the same
// time: a block reads its tile once, forms the tile's map, gets the state before the tile from the
// tiles before it, and writes the tile's outputs (the backward pass the same from the other end).
// Both passes are bound by HBM: 6 bytes a value forward (16-bit), 10 backward.
//
// The state before a tile.  A block publishes its tile's map as soon as it has it and the state
// behind the tile once it knows that; each with a flag.  It looks back over the flags for the
// nearest tile whose end state is known, and applies the maps in between in order.  Whichever way
// a state is reached, it is the same sequence of multiply-adds on the same values, so results do
// not depend on timing.  Blocks take their tiles from a counter, in the plan's order, so a tile's
// predecessors are always with blocks that already run: the waits end.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "kda_args.h"
#include "kda_io.cuh"
#include "kda_once.h"
#include "kda_recurrence.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 8;  // tokens of a thread, 4 channels each

// A tile's place in the chain of its sequence: 0 nothing yet, then the tile's map, then the state
// that leaves it.
enum Flag : int32_t { FLAG_NONE = 0, FLAG_MAP = 1, FLAG_STATE = 2 };

struct RecParams {
  kda_view_t x, g, beta, dout;  // device addresses and strides
  const int32_t* plan;
  int32_t checksum;
  int32_t N, chain;
  int32_t chained;   // some sequence has more than one tile
  const float* h0;
  const float* A_log;
  const float* dt_bias;
  float lower_bound;
  const float* dfinal;
  int32_t* status;   // [0] the status word, [1] the tile counter
  int32_t* flags;    // [chain][N]
  float* map_a;      // [chain][N][D] products of decays
  float* map_h;      // [chain][N][D] end states from zero
  float* ends;       // [chain][N][D] states that leave the tiles
  const float* states;  // backward: the forward pass's ends
  void* out;         // forward: out; backward: dx
  void* dg;
  void* dbeta;
  float* final_state;
  float* dh0;
  float* part_bias;  // [chain][N][D]
  float* part_A;     // [chain][N]
  kda_view_t od, bd; // strides of the dense outputs with and without channels
};

template <class T>
__device__ __forceinline__ const T* at(const kda_view_t& v, long long b, long long n, long long s) {
  return static_cast<const T*>(v.data) + b * v.stride_b + n * v.stride_n + s * v.stride_s;
}

__device__ __forceinline__ int32_t ld_acquire(const int32_t* p) {
  int32_t v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(int32_t* p, int32_t v) {
  asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// A work item: a tile's record and a head.
struct Item {
  int slot, row0, valid, store, index, tile, count, n;
};

// The block's item, or false when the plan on the device is not the host's.  Forward, counter value
// i is item i; backward, the tiles with tokens are taken from the last to the first.
template <bool BACKWARD>
__device__ __forceinline__ bool take_item(const RecParams& p, int* shared, Item* it) {
  if (p.plan[RH_CHECKSUM] != p.checksum) {
    if (threadIdx.x == 0) *p.status = DS_PLAN;
    return false;
  }
  int id = blockIdx.x;
  if (p.chained) {
    if (threadIdx.x == 0) *shared = atomicAdd(p.status + 1, 1);
    __syncthreads();
    id = *shared;
  }
  int k = id / p.N;
  it->n = id - k * p.N;
  if (BACKWARD && k < p.chain) k = p.chain - 1 - k;
  const int4* r = reinterpret_cast<const int4*>(p.plan + kRecHeader + (size_t)k * kRecRecord);
  const int4 u = __ldg(r), v = __ldg(r + 1);
  it->slot = u.x;
  it->row0 = u.y;
  it->valid = u.z;
  it->store = u.w;
  it->index = v.x;
  it->tile = v.y;
  it->count = v.z;
  return true;
}

// One warp publishes 4 channels a lane of one or two arrays, then the flag.
__device__ __forceinline__ void publish(int32_t* flag, int32_t value, bool mine, float* to_a,
                                        const float (&a)[4], float* to_b, const float (&b)[4]) {
  if (mine) {
    *reinterpret_cast<float4*>(to_a) = make_float4(a[0], a[1], a[2], a[3]);
    if (to_b) *reinterpret_cast<float4*>(to_b) = make_float4(b[0], b[1], b[2], b[3]);
  }
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    __threadfence();
    st_release(flag, value);
  }
}

__device__ __forceinline__ void ld_shared_by_blocks(const float* p, float (&v)[4]) {
  const float4 w = __ldcg(reinterpret_cast<const float4*>(p));
  v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
}

// The state that enters a tile, for one warp: 4 channels a lane at `chan`.  `before` tiles precede
// it in the chain's direction, at index + step, index + 2 step, ...; the first one of a chain
// publishes its end state without looking.  Publishes the tile's own map first if it has to wait.
// A wait that gives up records DS_TIMEOUT and returns NaN.
template <int D>
__device__ void look_back(const RecParams& p, const Item& it, int step, int before, bool mine,
                          int chan, bool successor, const float (&ta)[4], const float (&th)[4],
                          float (&c)[4]) {
  const int lane = threadIdx.x & 31;
  const size_t own = (size_t)it.index * p.N + it.n;
  const long long stride = (long long)step * p.N;
  bool published = !successor;
  int base = 0, found = -1;
  for (int tries = 0; found < 0; ++tries) {
    const int back = base + lane;  // 0 is the direct predecessor
    const int32_t f =
        back < before ? ld_acquire(p.flags + (long long)own + (back + 1) * stride) : FLAG_NONE;
    const unsigned state = __ballot_sync(0xffffffffu, f == FLAG_STATE);
    const unsigned some = __ballot_sync(0xffffffffu, f != FLAG_NONE);
    const int first = __ffs(state) - 1;
    if (first >= 0 && (~some & ((1u << first) - 1u)) == 0) {
      found = base + first;
      break;
    }
    if (!published) {
      publish(p.flags + own, FLAG_MAP, mine, p.map_a + own * D + chan, ta, p.map_h + own * D + chan,
              th);
      published = true;
    }
    if (some == 0xffffffffu) base += 32;  // only maps so far: look further back
    if ((tries & 1023) == 1023 &&
        (tries > (1 << 21) || *reinterpret_cast<volatile int32_t*>(p.status) != DS_OK)) {
      if (lane == 0) atomicCAS(p.status, DS_OK, DS_TIMEOUT);
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] = __int_as_float(0x7fc00000);
      return;
    }
  }
  __syncwarp();
  ld_shared_by_blocks(p.ends + (own + (found + 1) * stride) * D + chan, c);
  for (int i = found - 1; i >= 0; --i) {
    float a[4], h[4];
    ld_shared_by_blocks(p.map_a + (own + (i + 1) * stride) * D + chan, a);
    ld_shared_by_blocks(p.map_h + (own + (i + 1) * stride) * D + chan, h);
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = fmaf(a[e], c[e], h[e]);
  }
}

// Which 4 channels and 8 tokens of a tile a thread has.
template <int D>
struct Place {
  static constexpr int kLanes = D / 4;
  static constexpr int kGroups = kThreads / kLanes;
  static constexpr int kTile = kGroups * kRows;
  static_assert(kTile == rec_tile_rows(D), "a tile is the block's threads by their tokens");
  int chan, group;
  __device__ Place() : chan((threadIdx.x % kLanes) * 4), group(threadIdx.x / kLanes) {}
};

// sigmoid of the write logits of the tile's tokens, into shared memory
template <class T, int D>
__device__ __forceinline__ void load_beta(const RecParams& p, const Item& it, float* sb) {
  for (int r = threadIdx.x; r < Place<D>::kTile; r += kThreads)
    sb[r] = r < it.valid ? sigmoid(to_f32(*at<T>(p.beta, it.slot, it.n, it.row0 + r))) : 0.f;
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads, 2) rec_forward_kernel(const RecParams p) {
  using P = Place<D>;
  __shared__ int ticket;
  __shared__ float sb[P::kTile];
  __shared__ __align__(16) float sa[P::kGroups][D], sh[P::kGroups][D], carry[D];
  Item it;
  if (!take_item<false>(p, &ticket, &it)) return;
  const P me;
  const int r0 = me.group * kRows;
  T* out = static_cast<T*>(p.out) + (long long)it.slot * p.od.stride_b +
           (long long)it.n * p.od.stride_n + (long long)it.row0 * p.od.stride_s + me.chan;
  if (it.valid == 0) {  // padding
    const float z[4] = {};
    for (int i = 0; i < kRows; ++i)
      if (r0 + i < it.store) st4(out + (long long)(r0 + i) * p.od.stride_s, z);
    return;
  }
  const T* xs = at<T>(p.x, it.slot, it.n, it.row0) + me.chan;
  const T* gs = at<T>(p.g, it.slot, it.n, it.row0) + me.chan;
  Vec4<T> rx[kRows], rg[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    rx[i] = rg[i] = Vec4<T>{};
    if (r0 + i < it.valid) {
      rg[i] = ld4(gs + (long long)(r0 + i) * p.g.stride_s);
      rx[i] = ld4(xs + (long long)(r0 + i) * p.x.stride_s);
    }
  }
  load_beta<T, D>(p, it, sb);
  const GateScale gc = gate_scale(__ldg(p.A_log + it.n), p.lower_bound);
  float bias[4];
  ld_shared_by_blocks(p.dt_bias + (size_t)it.n * D + me.chan, bias);
  __syncthreads();

  // the thread's own run of tokens: decays, writes and the map
  float a[kRows][4], u[kRows][4], pa[4], ph[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    pa[e] = 1.f;
    ph[e] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    float g[4];
    widen(rg[i], g);
    widen(rx[i], u[i]);
    const float b = sb[r0 + i];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float t;
      a[i][e] = r0 + i < it.valid ? ex2(gc.l2 * gate_sigmoid(gc, g[e] + bias[e], &t)) : 1.f;
      u[i][e] *= b;
      pa[e] *= a[i][e];
      ph[e] = fmaf(a[i][e], ph[e], u[i][e]);
    }
  }
  st4(&sa[me.group][me.chan], pa);
  st4(&sh[me.group][me.chan], ph);
  __syncthreads();
  // the map of the tokens before the thread's own
  float qa[4], qh[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    qa[e] = 1.f;
    qh[e] = 0.f;
  }
  for (int k = 0; k < me.group; ++k) {
    const float4 ka = *reinterpret_cast<const float4*>(&sa[k][me.chan]);
    const float4 kh = *reinterpret_cast<const float4*>(&sh[k][me.chan]);
    qa[0] *= ka.x; qa[1] *= ka.y; qa[2] *= ka.z; qa[3] *= ka.w;
    qh[0] = fmaf(ka.x, qh[0], kh.x);
    qh[1] = fmaf(ka.y, qh[1], kh.y);
    qh[2] = fmaf(ka.z, qh[2], kh.z);
    qh[3] = fmaf(ka.w, qh[3], kh.w);
  }
  const size_t st = ((size_t)it.slot * p.N + it.n) * D + me.chan;
  const size_t own = (size_t)it.index * p.N + it.n;
  if (threadIdx.x >= kThreads - 32) {  // the warp that has the last tokens
    const bool mine = me.group == P::kGroups - 1;
    const bool successor = it.tile + 1 < it.count;
    float ta[4], th[4], c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ta[e] = qa[e] * pa[e];
      th[e] = fmaf(pa[e], qh[e], ph[e]);
    }
    if (it.tile > 0) {
      look_back<D>(p, it, -1, it.tile, mine, me.chan, successor, ta, th, c);
    } else if (p.h0) {
      const float4 w = *reinterpret_cast<const float4*>(p.h0 + st);
      c[0] = w.x; c[1] = w.y; c[2] = w.z; c[3] = w.w;
    }
    float end[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) end[e] = fmaf(ta[e], c[e], th[e]);
    if (successor) publish(p.flags + own, FLAG_STATE, mine, p.ends + own * D + me.chan, end, nullptr, end);
    if (mine) {
      st4(&carry[me.chan], c);
      if (!successor) st4(p.final_state + st, end);
    }
  }
  __syncthreads();
  float h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = fmaf(qa[e], carry[me.chan + e], qh[e]);
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = fmaf(a[i][e], h[e], u[i][e]);
    T* dst = out + (long long)(r0 + i) * p.od.stride_s;
    if (r0 + i < it.valid) {
      st4(dst, h);
    } else if (r0 + i < it.store) {
      const float z[4] = {};
      st4(dst, z);
    }
  }
}

// 4 channels from global to the thread's own place in shared memory, or zeros there
template <class T>
__device__ __forceinline__ void copy_async(T* to, const T* from, bool real) {
  const uint32_t dst = (uint32_t)__cvta_generic_to_shared(to);
  const int n = real ? (int)sizeof(T) * 4 : 0;
  if constexpr (sizeof(T) == 2)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(from), "r"(n));
  else
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(from), "r"(n));
}

template <class T>
__device__ __forceinline__ void ld_own(const T* p, float (&x)[4]) {
  Vec4<T> v;
  v.w = *reinterpret_cast<const decltype(v.w)*>(p);
  widen(v, x);
}

// Sums of 8 values over the LANES lanes of a group, by halving the values as the distance halves:
// lane i of every LANES / 8 ends with the sum of value i * 8 / LANES.
template <int LANES>
__device__ __forceinline__ float group_sum8(float (&v)[8], int lane) {
  int n = 8, o = LANES / 2;
#pragma unroll
  for (; n > 1; n /= 2, o /= 2) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= n / 2) break;
      const float keep = upper ? v[i + n / 2] : v[i], give = upper ? v[i] : v[i + n / 2];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
#pragma unroll
  for (; o > 0; o /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads, 2) rec_backward_kernel(const RecParams p) {
  using P = Place<D>;
  extern __shared__ __align__(16) unsigned char raw_smem[];
  T* const sg = reinterpret_cast<T*>(raw_smem);  // g, x, dout of the tile, [kTile][D] each
  T* const sx = sg + kRecTileElems;
  T* const sd = sx + kRecTileElems;
  __shared__ int ticket;
  __shared__ float sb[P::kTile], sum_a[kThreads / 32];
  __shared__ __align__(16) float sa[P::kGroups][D], sh[P::kGroups][D], sc[P::kGroups][D], carry[D];
  Item it;
  if (!take_item<true>(p, &ticket, &it)) return;
  const P me;
  const int r0 = me.group * kRows;
  const long long o0 = (long long)it.slot * p.od.stride_b + (long long)it.n * p.od.stride_n +
                       (long long)it.row0 * p.od.stride_s + me.chan;
  T* dx = static_cast<T*>(p.out) + o0;
  T* dg = static_cast<T*>(p.dg) + o0;
  T* dbeta = static_cast<T*>(p.dbeta) + (long long)it.slot * p.bd.stride_b +
             (long long)it.n * p.bd.stride_n + (long long)it.row0 * p.bd.stride_s;
  const float zeros[4] = {};
  // padding rows, of a tile without tokens or behind the last one
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = r0 + i;
    if (r >= it.valid && r < it.store) {
      st4(dx + (long long)r * p.od.stride_s, zeros);
      st4(dg + (long long)r * p.od.stride_s, zeros);
      if (me.chan == 0) dbeta[(long long)r * p.bd.stride_s] = from_f32<T>(0.f);
    }
  }
  if (it.valid == 0) return;

  const T* xs = at<T>(p.x, it.slot, it.n, it.row0) + me.chan;
  const T* gs = at<T>(p.g, it.slot, it.n, it.row0) + me.chan;
  const T* ds = p.dout.data ? at<T>(p.dout, it.slot, it.n, it.row0) + me.chan : xs;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = r0 + i, s = r * D + me.chan;
    const bool real = r < it.valid;
    copy_async(sg + s, real ? gs + (long long)r * p.g.stride_s : gs, real);
    copy_async(sx + s, real ? xs + (long long)r * p.x.stride_s : xs, real);
    copy_async(sd + s, real ? ds + (long long)r * p.dout.stride_s : ds, real && p.dout.data);
  }
  load_beta<T, D>(p, it, sb);
  const GateScale gc = gate_scale(__ldg(p.A_log + it.n), p.lower_bound);
  const size_t st = ((size_t)it.slot * p.N + it.n) * D + me.chan;
  const size_t own = (size_t)it.index * p.N + it.n;
  float bias[4], h[4] = {};
  ld_shared_by_blocks(p.dt_bias + (size_t)it.n * D + me.chan, bias);
  if (it.tile > 0) ld_shared_by_blocks(p.states + (own - p.N) * D + me.chan, h);
  else if (p.h0) ld_shared_by_blocks(p.h0 + st, h);
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();

  // decays, and the maps of the thread's tokens: of the state forwards, of a_t lam_t backwards
  float a[kRows][4], w[kRows][4], pa[4], ph[4], pc[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    pa[e] = 1.f;
    ph[e] = pc[e] = 0.f;
  }
  const float slope = p.lower_bound * gc.ea;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int s = (r0 + i) * D + me.chan;
    float g[4], x[4], d[4];
    ld_own(sg + s, g);
    ld_own(sx + s, x);
    ld_own(sd + s, d);
    const float b = sb[r0 + i];
    const bool real = r0 + i < it.valid;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float t;
      const float sig = gate_sigmoid(gc, g[e] + bias[e], &t);
      a[i][e] = real ? ex2(gc.l2 * sig) : 1.f;
      w[i][e] = real ? slope * sig * one_minus(sig, t) * a[i][e] : 0.f;
      pa[e] *= a[i][e];
      ph[e] = fmaf(a[i][e], ph[e], b * x[e]);
      pc[e] = fmaf(pa[e], d[e], pc[e]);
    }
  }
  st4(&sa[me.group][me.chan], pa);
  st4(&sh[me.group][me.chan], ph);
  st4(&sc[me.group][me.chan], pc);
  __syncthreads();
  // the warp with the first tokens gets what comes from behind the tile
  if (threadIdx.x < 32) {
    const bool mine = me.group == 0, last = it.tile + 1 == it.count;
    float ta[4], tc[4], c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ta[e] = 1.f;
      tc[e] = 0.f;
    }
    for (int k = P::kGroups - 1; k >= 0; --k)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float ka = sa[k][me.chan + e];
        ta[e] *= ka;
        tc[e] = fmaf(ka, tc[e], sc[k][me.chan + e]);
      }
    if (!last) look_back<D>(p, it, 1, it.count - 1 - it.tile, mine, me.chan, it.tile > 0, ta, tc, c);
    else if (p.dfinal) ld_shared_by_blocks(p.dfinal + st, c);
    float end[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) end[e] = fmaf(ta[e], c[e], tc[e]);
    if (it.tile > 0) publish(p.flags + own, FLAG_STATE, mine, p.ends + own * D + me.chan, end, nullptr, end);
    if (mine) {
      st4(&carry[me.chan], c);
      if (it.tile == 0 && p.dh0) st4(p.dh0 + st, end);
    }
  }
  // the state before each token, into w: dg = lam w
  for (int k = 0; k < me.group; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = fmaf(sa[k][me.chan + e], h[e], sh[k][me.chan + e]);
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    float x[4];
    ld_own(sx + (r0 + i) * D + me.chan, x);
    const float b = sb[r0 + i];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[i][e] *= h[e];
      h[e] = fmaf(a[i][e], h[e], b * x[e]);
    }
  }
  __syncthreads();
  float c[4], dot[kRows], sum_b[4] = {}, sum_raw = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] = carry[me.chan + e];
  for (int k = P::kGroups - 1; k > me.group; --k)
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = fmaf(sa[k][me.chan + e], c[e], sc[k][me.chan + e]);
#pragma unroll
  for (int i = kRows - 1; i >= 0; --i) {
    const int r = r0 + i, s = r * D + me.chan;
    float g[4], x[4], d[4], lam[4], dgr[4];
    ld_own(sg + s, g);
    ld_own(sx + s, x);
    ld_own(sd + s, d);
    const float b = sb[r];
    dot[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lam[e] = d[e] + c[e];
      c[e] = a[i][e] * lam[e];
      dot[i] = fmaf(lam[e], x[e], dot[i]);
      dgr[e] = lam[e] * w[i][e];
      lam[e] *= b;
      sum_b[e] += dgr[e];
      sum_raw = fmaf(dgr[e], g[e] + bias[e], sum_raw);
    }
    if (r < it.valid) {
      st4(dx + (long long)r * p.od.stride_s, lam);
      st4(dg + (long long)r * p.od.stride_s, dgr);
    }
  }
  // dbeta: the sum over the token's channels
  {
    constexpr int kEach = P::kLanes / 8;  // lanes that end with the same token
    const int lane = threadIdx.x % P::kLanes;
    const float sum = group_sum8<P::kLanes>(dot, lane);
    const int r = r0 + lane / kEach;
    if (lane % kEach == 0 && r < it.valid) {
      const float b = sb[r];
      dbeta[(long long)r * p.bd.stride_s] = from_f32<T>(sum * b * (1.f - b));
    }
  }
  // the tile's part of the parameters' gradients
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum_raw += __shfl_xor_sync(0xffffffffu, sum_raw, o);
  if ((threadIdx.x & 31) == 0) sum_a[threadIdx.x >> 5] = sum_raw;
  __syncthreads();  // sh is free: its last reads are before the previous barrier
  st4(&sh[me.group][me.chan], sum_b);
  __syncthreads();
  if (threadIdx.x < D) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < P::kGroups; ++k) sum += sh[k][threadIdx.x];
    p.part_bias[own * D + threadIdx.x] = sum;
  } else if (threadIdx.x == D) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) sum += sum_a[k];
    p.part_A[own] = sum;
  }
}

// ddt_bias and dA_log: the tiles' parts in a fixed order, in fp64.  A block has 32 channels of a
// head (the first one of a head its dA_log too), 32 threads a channel.
template <int D>
__global__ void __launch_bounds__(1024) rec_params_kernel(const float* part_bias,
                                                          const float* part_A, int chain, int N,
                                                          float* dA_log, float* ddt_bias) {
  __shared__ double red[32][33];
  constexpr int kBlocks = D / 32;
  const int n = blockIdx.x / kBlocks, d = (blockIdx.x % kBlocks) * 32 + (threadIdx.x & 31);
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  double sum = 0;
#pragma unroll 4
  for (int k = row; k < chain; k += 32) sum += part_bias[((size_t)k * N + n) * D + d];
  red[row][lane] = sum;
  __syncthreads();
  if (row == 0) {
    for (int k = 1; k < 32; ++k) sum += red[k][lane];
    ddt_bias[(size_t)n * D + d] = (float)sum;
  }
  if (blockIdx.x % kBlocks != 0) return;
  __syncthreads();
  sum = 0;
  for (int k = threadIdx.x; k < chain; k += 1024) sum += part_A[(size_t)k * N + n];
  red[row][lane] = sum;
  __syncthreads();
  if (row == 0) {
    sum = 0;
    for (int k = 0; k < 32; ++k) sum += red[k][lane];
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_down_sync(0xffffffffu, sum, o);
    if (lane == 0) dA_log[n] = (float)sum;
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

int slots(const kda_recurrence_shape_t& s) { return s.layout == KDA_LAYOUT_TND ? 1 : s.B; }

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
  const int nb = slots(*shape);
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
  p->N = shape->N;
  p->chain = plan_host[RH_CHAIN];
  p->chained = plan_host[RH_MAX_TILES] > 1;
  p->h0 = h0;
  p->A_log = A_log;
  p->dt_bias = dt_bias;
  p->lower_bound = lower_bound;
  p->status = static_cast<int32_t*>(workspace);
  p->od = dense_view(nullptr, shape->layout, shape->N, shape->S, shape->D);
  p->bd = dense_view(nullptr, shape->layout, shape->N, shape->S, 1);
  if (nb == 1) p->od.stride_b = p->bd.stride_b = 0;
  return KDA_OK;
}

size_t states_floats(const int32_t* plan) {
  return (size_t)plan[RH_CHAIN] * plan[RH_N] * plan[RH_D];
}

// The workspace after its header: the flags, and the tiles' maps and end states of a chained plan;
// then the parameters' partial gradients of a backward pass.
struct Scratch {
  size_t flags, map_a, map_h, ends, part_bias, part_A, total;
  Scratch(const int32_t* plan, bool backward) {
    const size_t items = (size_t)plan[RH_CHAIN] * plan[RH_N];
    const bool chained = plan[RH_MAX_TILES] > 1;
    size_t off = kWsHeaderBytes;
    auto take = [&off](size_t bytes) {
      const size_t here = off;
      off += (bytes + 255) / 256 * 256;
      return here;
    };
    flags = take(chained ? items * 4 : 0);
    map_a = take(chained ? states_floats(plan) * 4 : 0);
    map_h = take(chained ? states_floats(plan) * 4 : 0);
    ends = take(chained ? states_floats(plan) * 4 : 0);
    part_bias = take(backward ? states_floats(plan) * 4 : 0);
    part_A = take(backward ? items * 4 : 0);
    total = off;
  }
  void place(void* workspace, RecParams* p) const {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p->flags = reinterpret_cast<int32_t*>(ws + flags);
    p->map_a = reinterpret_cast<float*>(ws + map_a);
    p->map_h = reinterpret_cast<float*>(ws + map_h);
    p->ends = reinterpret_cast<float*>(ws + ends);
    p->part_bias = reinterpret_cast<float*>(ws + part_bias);
    p->part_A = reinterpret_cast<float*>(ws + part_A);
  }
};

template <class T, int D>
cudaError_t launch_forward(const RecParams& p, unsigned grid, cudaStream_t s) {
  rec_forward_kernel<T, D><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <class T, int D>
cudaError_t launch_backward(const RecParams& p, unsigned grid, cudaStream_t s) {
  static PerDevice ready;
  constexpr int kSmem = 3 * kRecTileElems * (int)sizeof(T);
  int dev = 0, unused = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess)
    e = once_per_device(ready, dev, &unused, [](int, int*) {
      return cudaFuncSetAttribute(rec_backward_kernel<T, D>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    });
  if (e != cudaSuccess) return e;
  rec_backward_kernel<T, D><<<grid, kThreads, kSmem, s>>>(p);
  return cudaGetLastError();
}

template <class F>
cudaError_t dispatch(const kda_recurrence_shape_t& s, F&& f) {
  auto with_type = [&](auto* tag) {
    return s.D == 128 ? f(tag, std::integral_constant<int, 128>())
                      : f(tag, std::integral_constant<int, 64>());
  };
  if (s.dtype == KDA_BF16) return with_type((__nv_bfloat16*)nullptr);
  if (s.dtype == KDA_FP16) return with_type((__half*)nullptr);
  return with_type((float*)nullptr);
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
  *bytes = Scratch(plan, backward != 0).total;
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
  const Scratch scratch(plan_host, false);
  scratch.place(workspace, &p);
  if (states) p.ends = states;
  p.out = out;
  p.final_state = final_state;
  // the status word, the tile counter and the flags start at zero
  if (cudaMemsetAsync(workspace, 0, scratch.map_a, s) != cudaSuccess) return KDA_ERR_CUDA;
  const unsigned grid = (unsigned)plan_host[RH_TILES] * shape->N;
  const cudaError_t e = dispatch(*shape, [&](auto* tag, auto d) {
    return launch_forward<std::remove_pointer_t<decltype(tag)>, decltype(d)::value>(p, grid, s);
  });
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
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
    st = check_view(&p.dout, slots(*shape), shape->N, shape->S, shape->D, z.elem, &r_dout);
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
  const Scratch scratch(plan_host, true);
  scratch.place(workspace, &p);
  p.states = states;
  p.dfinal = dfinal_state;
  p.out = dx;
  p.dg = dg;
  p.dbeta = dbeta;
  p.dh0 = dinitial_state;
  if (cudaMemsetAsync(workspace, 0, scratch.map_a, s) != cudaSuccess) return KDA_ERR_CUDA;
  const unsigned grid = (unsigned)plan_host[RH_TILES] * shape->N;
  const cudaError_t e = dispatch(*shape, [&](auto* tag, auto d) {
    constexpr int D = decltype(d)::value;
    const cudaError_t err =
        launch_backward<std::remove_pointer_t<decltype(tag)>, D>(p, grid, s);
    if (err != cudaSuccess) return err;
    rec_params_kernel<D><<<(unsigned)shape->N * (D / 32), 1024, 0, s>>>(
        p.part_bias, p.part_A, p.chain, p.N, dA_log, ddt_bias);
    return cudaGetLastError();
  });
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
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
