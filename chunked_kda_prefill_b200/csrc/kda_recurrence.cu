// kda_recurrence.cu -- the gated recurrence, the vector form of the KDA state:
//     a_t = exp(lb sigmoid(e^A (g_t + bias))),  h_t = a_t h_{t-1} + sigmoid(beta_t) x_t.
//
// A run of tokens maps its start state to its end state by h -> A h + H, with A the product of its
// decays, and such maps compose.  A cluster of 1 to 8 blocks walks one (sequence, head) from its
// start (the backward pass from its end), a tile of 8192 values per block and step; a thread has 8
// tokens of 4 channels.  In a step every thread forms its tokens' map, the block composes its
// threads' maps and the cluster its blocks', through shared memory, and with the state before its
// tokens a thread runs through them once more from registers and writes.  The data is read once.
// Which block does what is fixed by the plan and the launch, so the same call gives the same bits.
//
// Both passes are bound by HBM: 6 bytes a value forward (16-bit), 10 backward.
#include <cuda_runtime.h>

#include <algorithm>
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

struct RecParams {
  kda_view_t x, g, beta, dout;  // device addresses and strides
  const int32_t* plan;
  int32_t checksum;
  int32_t N, units;
  int32_t slot_rows;  // rows that a slot's outputs have, padding included; 0 for packed rows
  int32_t cluster;
  const float* h0;
  const float* A_log;
  const float* dt_bias;
  float lower_bound;
  const float* dfinal;
  int32_t* status;
  float* states;  // [tiles][N][D] the states before the tiles: forward writes, backward reads
  void* out;      // forward: out; backward: dx
  void* dg;
  void* dbeta;
  float* final_state;
  float* dh0;
  float* part_bias;   // [B][cluster][N][D]
  float* part_A;      // [B][cluster][N]
  kda_view_t od, bd;  // strides of the dense outputs with and without channels
};

template <class T>
__device__ __forceinline__ const T* at(const kda_view_t& v, long long b, long long n, long long s) {
  return static_cast<const T*>(v.data) + b * v.stride_b + n * v.stride_n + s * v.stride_s;
}

// Which 4 channels and 8 tokens of a tile a thread has.
template <int D>
struct Place {
  static constexpr int kLanes = D / 4;
  static constexpr int kGroups = kThreads / kLanes;
  static constexpr int kTile = kGroups * kRows;
  static_assert(kTile == rec_tile_rows(D), "a tile is the block's threads by their tokens");
  int chan, group, r0;
  __device__ Place()
      : chan((threadIdx.x % kLanes) * 4), group(threadIdx.x / kLanes), r0(group * kRows) {}
};

// One (sequence, head) of the walk.
struct Unit {
  int slot, start, len, base;  // the plan's record
  int n, steps;
  int place;  // of the sequence in the plan
};

// A block's walk: units in rounds over the clusters, every other round in reverse, so that with the
// plan's order (longest first) no cluster gets the longer unit of every round.  The record of the
// unit after the current one is requested a unit ahead.
struct Walk {
  Unit u;
  int step, round;
  int4 ahead;

  __device__ static int index(const RecParams& p, int round) {
    const int clusters = gridDim.x / p.cluster, q = blockIdx.x / p.cluster;
    const long long i = (long long)round * clusters + (round & 1 ? clusters - 1 - q : q);
    return i < p.units ? (int)i : -1;
  }
  __device__ static int4 record(const RecParams& p, int round) {
    const int i = index(p, round);
    const int4* rec = reinterpret_cast<const int4*>(p.plan + kRecHeader);
    return i < 0 ? make_int4(0, 0, 0, 0) : __ldg(rec + i / p.N);
  }
  template <int R>
  __device__ void enter(const RecParams& p) {
    const int i = index(p, round);
    u.slot = ahead.x;
    u.start = ahead.y;
    u.len = ahead.z;
    u.base = ahead.w;
    u.place = i < 0 ? -1 : i / p.N;
    u.n = i < 0 ? -1 : i - u.place * p.N;
    const int rows = p.slot_rows ? p.slot_rows : u.len;
    u.steps = ((rows - 1) / R) / p.cluster + 1;
    step = 0;
    ahead = record(p, round + 1);
  }
  template <int R>
  __device__ void begin(const RecParams& p) {
    round = 0;
    ahead = record(p, 0);
    enter<R>(p);
  }
  template <int R>
  __device__ void next(const RecParams& p) {
    if (++step < u.steps) return;
    ++round;
    enter<R>(p);
  }
  __device__ bool done() const { return u.n < 0; }
};

// A block's tile in a step: its first row within the sequence, its rows with tokens, and whether any
// block of the cluster has such rows.
struct Tile {
  int row, valid, index;
  bool work;
};
template <int R, bool BACKWARD>
__device__ __forceinline__ Tile tile_of(const RecParams& p, const Walk& w, int rank) {
  Tile t;
  const int first = (BACKWARD ? w.u.steps - 1 - w.step : w.step) * p.cluster;
  t.index = first + rank;
  // the cluster's last tiles may lie behind the slot, and behind 32 bits
  t.row = (int)min((long long)t.index * R, (long long)INT_MAX);
  t.valid = max(0, min(R, w.u.len - t.row));
  t.work = (long long)first * R < w.u.len;
  return t;
}

// Whether the plan on the device is the host's; block 0 leaves the status.
__device__ __forceinline__ bool same_plan(const RecParams& p) {
  const bool same = p.plan[RH_CHECKSUM] == p.checksum;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = same ? DS_OK : DS_PLAN;
  return same;
}

// ---- clusters ----
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 4 floats at this block's shared address `p` in the block of another rank
__device__ __forceinline__ F4 ld_rank(const float* p, int rank) {
  uint32_t addr = (uint32_t)__cvta_generic_to_shared(p), far;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(addr), "r"(rank));
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(far)
               : "memory");
  return f4(v);
}

// ---- loads ----
// 4 channels from global to the thread's own place in shared memory
template <class T>
__device__ __forceinline__ void copy_async(T* to, const T* from) {
  const uint32_t dst = (uint32_t)__cvta_generic_to_shared(to);
  if constexpr (sizeof(T) == 2)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(from));
  else
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(from));
}
template <class T>
__device__ __forceinline__ F4 own4(const T* p) {
  Vec4<T> v;
  v.w = *reinterpret_cast<const decltype(v.w)*>(p);
  float x[4];
  widen(v, x);
  return f4(x);
}

// Starts the loads of the thread's tokens of one tensor; every thread reads only what it copied
// itself.  Behind the last token the channels are zeros, or -inf where they are gates: sigmoid and
// write are then zero and the decay one, so those rows change no map.
template <class T, int D>
__device__ __forceinline__ void request(T* to, const kda_view_t& v, const Unit& u, const Tile& t,
                                        const Place<D>& me, bool gate) {
  const T* from = at<T>(v, u.slot, u.n, (long long)u.start + t.row + me.r0) + me.chan;
  T* dst = to + me.r0 * D + me.chan;
  const int mine = t.valid - me.r0;
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    if (k < mine) {
      copy_async(dst + k * D, from);
      from += v.stride_s;
    } else {
      st4(dst + k * D, splat(gate ? -INFINITY : 0.f));
    }
  }
}
// The write logits of a tile, one a thread.
template <class T>
__device__ __forceinline__ float request_beta(const RecParams& p, const Unit& u, const Tile& t) {
  const int r = threadIdx.x;
  return r < t.valid ? to_f32(*at<T>(p.beta, u.slot, u.n, (long long)u.start + t.row + r)) : 0.f;
}

// Two stages of shared memory for the tile at work and the next one; fp32 tiles have one, so that
// two blocks still fit an SM.
template <class T>
constexpr int kStages = sizeof(T) == 2 ? 2 : 1;

template <class T, int D>
constexpr int forward_smem() {
  return kStages<T> * 2 * kRecTileElems * (int)sizeof(T);
}
template <class T, int D>
constexpr int backward_smem() {
  return kStages<T> * 3 * kRecTileElems * (int)sizeof(T);
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads, 2) rec_forward_kernel(const RecParams p) {
  using P = Place<D>;
  constexpr int R = P::kTile;
  extern __shared__ __align__(16) unsigned char raw_smem[];
  T* const stage = reinterpret_cast<T*>(raw_smem);  // [kStages][g, x][R][D]
  __shared__ float sb[2][R];
  __shared__ __align__(16) float sa[2][P::kGroups][D], sh[2][P::kGroups][D];
  __shared__ __align__(16) float map_a[2][D], map_h[2][D], carry_in[D], carry_out[D];
  if (!same_plan(p)) return;
  const P me;
  const int rank = blockIdx.x % p.cluster;
  Walk now, next;
  now.begin<R>(p);
  next = now;
  F4 h0_next = splat(0.f);
  float beta = 0.f;
  // the loads of `next`'s tile, and its start state where a unit begins
  auto start = [&](int i) {
    if (!next.done()) {
      const Tile t = tile_of<R, false>(p, next, rank);
      T* to = stage + (i % kStages<T>) * 2 * kRecTileElems;
      if (t.work) {
        request(to, p.g, next.u, t, me, true);
        request(to + kRecTileElems, p.x, next.u, t, me, false);
      }
      beta = request_beta<T>(p, next.u, t);
      if (next.step == 0) {
        h0_next = splat(0.f);
        if (p.h0)
          h0_next = f4(*reinterpret_cast<const float4*>(
              p.h0 + ((size_t)next.u.slot * p.N + next.u.n) * D + me.chan));
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  start(0);
  if (threadIdx.x < R) sb[0][threadIdx.x] = sigmoid(beta);
  __syncthreads();
  F4 carry = splat(0.f);
  for (int i = 0; !now.done(); ++i) {
    const int buf = i & 1;
    const Tile t = tile_of<R, false>(p, now, rank);
    if (now.step == 0) carry = h0_next;
    next.next<R>(p);
    if (kStages<T> == 2) start(i + 1);
    const T* const tg = stage + (i % kStages<T>) * 2 * kRecTileElems + me.r0 * D + me.chan;
    const T* const tx = tg + kRecTileElems;
    const GateScale gc = gate_scale(__ldg(p.A_log + now.u.n), p.lower_bound);
    const F4 bias =
        f4(__ldg(reinterpret_cast<const float4*>(p.dt_bias + (size_t)now.u.n * D + me.chan)));
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages<T> - 1) : "memory");

    // the thread's own tokens: decays, writes and the map
    F4 a[kRows], u[kRows], pa = splat(1.f), ph = splat(0.f);
    if (t.work) {
      const F4 nz = splat(gc.nz), l2 = splat(gc.l2), one = splat(1.f);
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const F4 e = each((own4(tg + k * D) + bias) * nz, ex2);
        a[k] = each(each(e + one, rcp) * l2, ex2);
        u[k] = own4(tx + k * D) * splat(sb[buf][me.r0 + k]);
        pa = pa * a[k];
        ph = fma4(a[k], ph, u[k]);
      }
      sts4(&sa[buf][me.group][me.chan], pa);
      sts4(&sh[buf][me.group][me.chan], ph);
    }
    if (kStages<T> == 1) start(i + 1);
    if (threadIdx.x < R) sb[buf ^ 1][threadIdx.x] = sigmoid(beta);
    __syncthreads();
    F4 h = carry;
    if (t.work) {
      if (p.cluster == 1) {
        for (int k = 0; k < P::kGroups; ++k) {
          if (k == me.group) h = carry;
          carry = fma4(lds4(&sa[buf][k][me.chan]), carry, lds4(&sh[buf][k][me.chan]));
        }
      } else {
        // the block's map, for the other ranks; the map before the thread's own tokens meanwhile
        if (threadIdx.x < P::kLanes) {
          F4 ta = splat(1.f), th = splat(0.f);
          for (int k = 0; k < P::kGroups; ++k) {
            const F4 ka = lds4(&sa[buf][k][me.chan]);
            ta = ta * ka;
            th = fma4(ka, th, lds4(&sh[buf][k][me.chan]));
          }
          sts4(&map_a[buf][me.chan], ta);
          sts4(&map_h[buf][me.chan], th);
        }
        cluster_arrive();
        F4 qa = splat(1.f), qh = splat(0.f);
        for (int k = 0; k < me.group; ++k) {
          const F4 ka = lds4(&sa[buf][k][me.chan]);
          qa = qa * ka;
          qh = fma4(ka, qh, lds4(&sh[buf][k][me.chan]));
        }
        cluster_wait();
        if (threadIdx.x < P::kLanes) {
          for (int r = 0; r < p.cluster; ++r) {
            if (r == rank) sts4(&carry_in[me.chan], carry);
            carry = fma4(ld_rank(&map_a[buf][me.chan], r), carry, ld_rank(&map_h[buf][me.chan], r));
          }
          sts4(&carry_out[me.chan], carry);
        }
        __syncthreads();
        h = lds4(&carry_in[me.chan]);
        carry = lds4(&carry_out[me.chan]);
        if (me.group == 0 && p.states && t.valid > 0)
          sts4(p.states + ((size_t)(now.u.base + t.index) * p.N + now.u.n) * D + me.chan, h);
        h = fma4(qa, h, qh);
      }
    }
    if (p.cluster == 1 && me.group == 0 && p.states && t.valid > 0)
      sts4(p.states + ((size_t)(now.u.base + t.index) * p.N + now.u.n) * D + me.chan, h);
    // the outputs, and zeros behind the last token
    {
      const int rows = p.slot_rows ? min(R, p.slot_rows - t.row) : t.valid;
      T* out = static_cast<T*>(p.out) + (long long)now.u.slot * p.od.stride_b +
               (long long)now.u.n * p.od.stride_n +
               ((long long)now.u.start + t.row + me.r0) * p.od.stride_s + me.chan;
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        if (t.work) h = fma4(a[k], h, u[k]);
        if (me.r0 + k < rows) st4(out, me.r0 + k < t.valid ? h : splat(0.f));
        out += p.od.stride_s;
      }
    }
    if (rank == 0 && me.group == 0 && now.step + 1 == now.u.steps)
      sts4(p.final_state + ((size_t)now.u.slot * p.N + now.u.n) * D + me.chan, carry);
    now = next;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (p.cluster > 1) {  // no block leaves while another reads its map
    cluster_arrive();
    cluster_wait();
  }
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
  constexpr int R = P::kTile;
  extern __shared__ __align__(16) unsigned char raw_smem[];
  T* const stage = reinterpret_cast<T*>(raw_smem);  // [kStages][g, x, dout][R][D]
  __shared__ float sb[2][R], sum_a[kThreads / 32];
  __shared__ __align__(16) float sa[P::kGroups][D], sh[P::kGroups][D], sc[P::kGroups][D];
  __shared__ __align__(16) float map_a[D], map_c[D], carry_in[D], carry_out[D];
  if (!same_plan(p)) return;
  const P me;
  const int rank = blockIdx.x % p.cluster;
  Walk now, next;
  now.begin<R>(p);
  next = now;
  F4 c_next = splat(0.f), h_next = splat(0.f);
  float beta = 0.f;
  auto start = [&](int i) {
    if (!next.done()) {
      const Tile t = tile_of<R, true>(p, next, rank);
      T* to = stage + (i % kStages<T>) * 3 * kRecTileElems;
      if (t.work) {
        request(to, p.g, next.u, t, me, true);
        request(to + kRecTileElems, p.x, next.u, t, me, false);
        if (p.dout.data) {
          request(to + 2 * kRecTileElems, p.dout, next.u, t, me, false);
        } else {
#pragma unroll
          for (int k = 0; k < kRows; ++k)
            st4(to + 2 * kRecTileElems + (me.r0 + k) * D + me.chan, splat(0.f));
        }
      }
      beta = request_beta<T>(p, next.u, t);
      h_next = splat(0.f);
      if (t.valid > 0)
        h_next = f4(__ldg(reinterpret_cast<const float4*>(
            p.states + ((size_t)(next.u.base + t.index) * p.N + next.u.n) * D + me.chan)));
      if (next.step == 0) {
        c_next = splat(0.f);
        if (p.dfinal)
          c_next = f4(__ldg(reinterpret_cast<const float4*>(
              p.dfinal + ((size_t)next.u.slot * p.N + next.u.n) * D + me.chan)));
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  start(0);
  if (threadIdx.x < R) sb[0][threadIdx.x] = sigmoid(beta);
  __syncthreads();
  F4 carry = splat(0.f), sum_b = splat(0.f), sum_raw = splat(0.f);
  for (int i = 0; !now.done(); ++i) {
    const Tile t = tile_of<R, true>(p, now, rank);
    const float* const b = sb[i & 1] + me.r0;
    if (now.step == 0) {
      carry = c_next;
      sum_b = sum_raw = splat(0.f);
    }
    F4 h = h_next;
    next.next<R>(p);
    if (kStages<T> == 2) start(i + 1);
    const T* const tg = stage + (i % kStages<T>) * 3 * kRecTileElems + me.r0 * D + me.chan;
    const T* const tx = tg + kRecTileElems;
    const T* const td = tx + kRecTileElems;
    const GateScale gc = gate_scale(__ldg(p.A_log + now.u.n), p.lower_bound);
    const F4 bias =
        f4(__ldg(reinterpret_cast<const float4*>(p.dt_bias + (size_t)now.u.n * D + me.chan)));
    const long long row = p.od.stride_s;
    const long long first = (long long)now.u.start + t.row + me.r0;
    const long long o0 = (long long)now.u.slot * p.od.stride_b + (long long)now.u.n * p.od.stride_n +
                         first * row + me.chan;
    T* const dx = static_cast<T*>(p.out) + o0;
    T* const dg = static_cast<T*>(p.dg) + o0;
    T* const dbeta = static_cast<T*>(p.dbeta) + (long long)now.u.slot * p.bd.stride_b +
                     (long long)now.u.n * p.bd.stride_n + first * p.bd.stride_s;
    const int rows = p.slot_rows ? min(R, p.slot_rows - t.row) : t.valid;
    if (t.valid < rows) {  // zeros behind the last token
      for (int k = 0; k < kRows; ++k)
        if (me.r0 + k >= t.valid && me.r0 + k < rows) {
          st4(dx + k * row, splat(0.f));
          st4(dg + k * row, splat(0.f));
          if (me.chan == 0) dbeta[k * p.bd.stride_s] = from_f32<T>(0.f);
        }
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages<T> - 1) : "memory");

    // decays, and the maps of the thread's tokens: of the state forwards, of a_t lam_t backwards
    F4 a[kRows], w[kRows];
    if (t.work) {
      F4 pa = splat(1.f), ph = splat(0.f), pc = splat(0.f);
      const F4 nz = splat(gc.nz), l2 = splat(gc.l2), one = splat(1.f);
      const F4 slope = splat(p.lower_bound * gc.ea);
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        // e is kept finite: 1 - sigmoid is e sigmoid, without cancellation, and where the sigmoid
        // is zero so is their product
        const F4 e = each((own4(tg + k * D) + bias) * nz, [](float z) { return fminf(ex2(z), 3e38f); });
        const F4 sig = each(e + one, rcp);
        a[k] = each(sig * l2, ex2);
        w[k] = sig * (e * sig) * (slope * a[k]);
        pa = pa * a[k];
        ph = fma4(a[k], ph, own4(tx + k * D) * splat(b[k]));
        pc = fma4(pa, own4(td + k * D), pc);
      }
      sts4(&sa[me.group][me.chan], pa);
      sts4(&sh[me.group][me.chan], ph);
      sts4(&sc[me.group][me.chan], pc);
    }
    if (kStages<T> == 2 && threadIdx.x < R) sb[~i & 1][threadIdx.x] = sigmoid(beta);
    __syncthreads();
    float dot[kRows];
    if (t.work) {
      if (p.cluster > 1) {
        if (threadIdx.x < P::kLanes) {
          F4 ta = splat(1.f), tc = splat(0.f);
          for (int k = P::kGroups - 1; k >= 0; --k) {
            const F4 ka = lds4(&sa[k][me.chan]);
            ta = ta * ka;
            tc = fma4(ka, tc, lds4(&sc[k][me.chan]));
          }
          sts4(&map_a[me.chan], ta);
          sts4(&map_c[me.chan], tc);
        }
        cluster_arrive();
      }
      // the state before each token, into w: dg = lam w
      for (int k = 0; k < me.group; ++k) h = fma4(lds4(&sa[k][me.chan]), h, lds4(&sh[k][me.chan]));
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        w[k] = w[k] * h;
        h = fma4(a[k], h, own4(tx + k * D) * splat(b[k]));
      }
      // a_t lam_t of what follows the thread's tokens
      F4 c = carry;
      if (p.cluster > 1) {
        cluster_wait();
        if (threadIdx.x < P::kLanes) {
          for (int r = p.cluster - 1; r >= 0; --r) {
            if (r == rank) sts4(&carry_in[me.chan], carry);
            carry = fma4(ld_rank(&map_a[me.chan], r), carry, ld_rank(&map_c[me.chan], r));
          }
          sts4(&carry_out[me.chan], carry);
        }
        cluster_arrive();  // the maps have been read
        __syncthreads();
        c = lds4(&carry_in[me.chan]);
        carry = lds4(&carry_out[me.chan]);
        for (int k = P::kGroups - 1; k > me.group; --k)
          c = fma4(lds4(&sa[k][me.chan]), c, lds4(&sc[k][me.chan]));
        cluster_wait();
      } else {
        for (int k = P::kGroups - 1; k >= 0; --k) {
          if (k == me.group) c = carry;
          carry = fma4(lds4(&sa[k][me.chan]), carry, lds4(&sc[k][me.chan]));
        }
      }
      F4 here_b = splat(0.f), here_raw = splat(0.f);
#pragma unroll
      for (int k = kRows - 1; k >= 0; --k) {
        dot[k] = 0.f;
        if (me.r0 + k < t.valid) {
          const F4 lam = own4(td + k * D) + c;
          c = a[k] * lam;
          const F4 dgk = lam * w[k], lx = lam * own4(tx + k * D);
          dot[k] = (lx.lo.x + lx.lo.y) + (lx.hi.x + lx.hi.y);
          st4(dx + k * row, lam * splat(b[k]));
          st4(dg + k * row, dgk);
          here_b = here_b + dgk;
          here_raw = fma4(dgk, own4(tg + k * D) + bias, here_raw);
        }
      }
      sum_b = sum_b + here_b;
      sum_raw = sum_raw + here_raw;
      // dbeta: the sum over the token's channels
      constexpr int kEach = P::kLanes / kRows;  // lanes that end with the same token
      const int lane = threadIdx.x % P::kLanes, k = lane / kEach;
      const float sum = group_sum8<P::kLanes>(dot, lane);
      if (lane % kEach == 0 && me.r0 + k < t.valid)
        dbeta[k * p.bd.stride_s] = from_f32<T>(sum * b[k] * (1.f - b[k]));
    }
    if (kStages<T> == 1) {
      start(i + 1);
      if (threadIdx.x < R) sb[~i & 1][threadIdx.x] = sigmoid(beta);
    }
    __syncthreads();  // the maps are read, and of one stage the next logits written
    if (now.step + 1 == now.u.steps) {
      if (p.dh0 && rank == 0 && me.group == 0)
        sts4(p.dh0 + ((size_t)now.u.slot * p.N + now.u.n) * D + me.chan, carry);
      // the unit's part of the parameters' gradients
      float raw = (sum_raw.lo.x + sum_raw.lo.y) + (sum_raw.hi.x + sum_raw.hi.y);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) raw += __shfl_xor_sync(0xffffffffu, raw, o);
      if ((threadIdx.x & 31) == 0) sum_a[threadIdx.x >> 5] = raw;
      sts4(&sh[me.group][me.chan], sum_b);
      __syncthreads();
      const size_t part = ((size_t)now.u.place * p.cluster + rank) * p.N + now.u.n;
      if (threadIdx.x < D) {
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < P::kGroups; ++k) sum += sh[k][threadIdx.x];
        p.part_bias[part * D + threadIdx.x] = sum;
      } else if (threadIdx.x == D) {
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k) sum += sum_a[k];
        p.part_A[part] = sum;
      }
      __syncthreads();
    }
    now = next;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (p.cluster > 1) {
    cluster_arrive();
    cluster_wait();
  }
}

// ddt_bias and dA_log: the units' parts in a fixed order, in fp64.  A block has 32 channels of a
// head (the first one of a head its dA_log too), 32 threads a channel.
template <int D>
__global__ void __launch_bounds__(1024) rec_params_kernel(const float* part_bias,
                                                          const float* part_A, int parts, int N,
                                                          float* dA_log, float* ddt_bias) {
  __shared__ double red[32][33];
  constexpr int kBlocks = D / 32;
  const int n = blockIdx.x / kBlocks, d = (blockIdx.x % kBlocks) * 32 + (threadIdx.x & 31);
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  double sum = 0;
#pragma unroll 4
  for (int k = row; k < parts; k += 32) sum += part_bias[((size_t)k * N + n) * D + d];
  red[row][lane] = sum;
  __syncthreads();
  if (row == 0) {
    for (int k = 1; k < 32; ++k) sum += red[k][lane];
    ddt_bias[(size_t)n * D + d] = (float)sum;
  }
  if (blockIdx.x % kBlocks != 0) return;
  __syncthreads();
  sum = 0;
  for (int k = threadIdx.x; k < parts; k += 1024) sum += part_A[(size_t)k * N + n];
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
  p->units = shape->B * shape->N;
  p->slot_rows = shape->layout == KDA_LAYOUT_TND ? 0 : shape->S;
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

// The workspace after its header: the parameters' partial gradients of a backward pass, one of each
// block of a cluster at the most.
struct Scratch {
  size_t part_A, total;
  Scratch(const int32_t* plan, bool backward) {
    const size_t heads = (size_t)plan[RH_B] * (1 << (kRecClusters - 1)) * plan[RH_N];
    part_A = kWsHeaderBytes + heads * plan[RH_D] * 4;
    total = backward ? part_A + heads * 4 : kWsHeaderBytes;
  }
};

// What a kernel's launches need to know of a device: the blocks that it holds at a time, as clusters
// of each size.
struct Resident {
  PerDevice of[kRecClusters];
};

void configure(int smem, int cluster, unsigned blocks, cudaStream_t s, cudaLaunchConfig_t* cfg,
               cudaLaunchAttribute* attr) {
  *cfg = cudaLaunchConfig_t{};
  cfg->gridDim = dim3(blocks);
  cfg->blockDim = dim3(kThreads);
  cfg->dynamicSmemBytes = (size_t)smem;
  cfg->stream = s;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = (unsigned)cluster;
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 1;
}

// Clusters of 2^c blocks that the current device holds at a time.
template <class K>
cudaError_t resident_clusters(K kernel, Resident& r, int smem, int c, int* clusters) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  return once_per_device(r.of[c], dev, clusters, [&](int, int* n) {
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr;
    configure(smem, 1 << c, 1u << c, nullptr, &cfg, &attr);
    err = cudaOccupancyMaxActiveClusters(n, kernel, &cfg);
    return err == cudaSuccess && *n < 1 ? cudaErrorLaunchOutOfResources : err;
  });
}

// Launches a pass on clusters of the size that takes the fewest steps one after another: those of
// the longest unit, or, where that is more, of all units over the clusters that run at a time.  The
// exchange between blocks makes a step of a cluster longer by about a third.
template <class K>
cudaError_t launch(K kernel, Resident& r, int smem, RecParams& p, const int32_t* plan,
                   cudaStream_t s) {
  int best = 0, best_clusters = 0;
  double least = 0;
  for (int c = 0; c < kRecClusters; ++c) {
    int clusters = 0;
    const cudaError_t e = resident_clusters(kernel, r, smem, c, &clusters);
    if (e != cudaSuccess) return e;
    const double all = (double)plan[RH_STEPS + c] * p.N / std::min(clusters, p.units);
    const double one = (double)((plan[RH_MAX_TILES] + (1 << c) - 1) >> c);
    const double cost = std::max(all, one) * (c == 0 ? 3 : 4);
    if (c == 0 || cost < least) {
      least = cost;
      best = c;
      best_clusters = clusters;
    }
  }
  p.cluster = 1 << best;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  configure(smem, p.cluster, (unsigned)std::min(best_clusters, p.units) * p.cluster, s, &cfg, &attr);
  return cudaLaunchKernelEx(&cfg, kernel, (const RecParams)p);
}

template <class T, int D>
cudaError_t launch_forward(RecParams& p, const int32_t* plan, cudaStream_t s) {
  static Resident resident;
  return launch(rec_forward_kernel<T, D>, resident, forward_smem<T, D>(), p, plan, s);
}

template <class T, int D>
cudaError_t launch_backward(RecParams& p, const int32_t* plan, cudaStream_t s) {
  static Resident resident;
  return launch(rec_backward_kernel<T, D>, resident, backward_smem<T, D>(), p, plan, s);
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
  // final_state may be initial_state itself: a unit's blocks have read its start state before the
  // barrier of its first step, and its end state is written after that of its last
  if (final_state == initial_state) in[3] = ByteRange{};
  const ByteRange outs[] = {dense_range(out, z.x), dense_range(final_state, z.state),
                            dense_range(states, states_floats(plan_host) * 4)};
  if (any_overlap(in, outs)) return KDA_ERR_ALIAS;
  if ((st = check_device()) != KDA_OK) return st;

  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  p.states = states;
  p.out = out;
  p.final_state = final_state;
  const cudaError_t e = dispatch(*shape, [&](auto* tag, auto d) {
    return launch_forward<std::remove_pointer_t<decltype(tag)>, decltype(d)::value>(p, plan_host, s);
  });
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_recurrence_backward(
    const kda_recurrence_shape_t* shape, const int32_t* plan_host, const int32_t* plan_dev,
    size_t n_int32, const kda_view_t* dout, const float* dfinal_state, const kda_view_t* x,
    const kda_view_t* g, const kda_view_t* beta, const float* A_log, const float* dt_bias,
    float lower_bound, const float* states, void* workspace, size_t workspace_bytes, void* dx,
    void* dg, void* dbeta, float* dinitial_state, float* dA_log, float* ddt_bias,
    kda_stream_t stream) {
  RecParams p{};
  ByteRange in[9], r_dout;
  kda_status_t st = prepare(shape, plan_host, plan_dev, n_int32, x, g, beta, nullptr, A_log,
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
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  p.part_bias = reinterpret_cast<float*>(ws + kWsHeaderBytes);
  p.part_A = reinterpret_cast<float*>(ws + scratch.part_A);
  p.states = const_cast<float*>(states);
  p.dfinal = dfinal_state;
  p.out = dx;
  p.dg = dg;
  p.dbeta = dbeta;
  p.dh0 = dinitial_state;
  const cudaError_t e = dispatch(*shape, [&](auto* tag, auto d) {
    constexpr int D = decltype(d)::value;
    using T = std::remove_pointer_t<decltype(tag)>;
    const cudaError_t err = launch_backward<T, D>(p, plan_host, s);
    if (err != cudaSuccess) return err;
    rec_params_kernel<D><<<(unsigned)shape->N * (D / 32), 1024, 0, s>>>(
        p.part_bias, p.part_A, shape->B * p.cluster, p.N, dA_log, ddt_bias);
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
