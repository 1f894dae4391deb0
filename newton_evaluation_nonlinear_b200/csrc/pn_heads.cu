// pn_heads.cu -- rotary positions and per-head norms of queries and keys.
//
//   rotation   (a, b) -> m (a cos w - b sin w, b cos w + a sin w), w = p f_i,
//              for the pairs i of a head vector at position p;
//   norm       y_j = x_j w_j r, r = 1 / sqrt(mean(x^2) + eps), then the rotation.
// Gradients: of the rotation, the inverse rotation (times m again); of the norm,
// with t the gradient rotated back, n = x r and u = t w:
//   dx = r (u - n mean(u n)),   dw = sum over rows of t n.
//
// All of it is bound by memory: each vector is read once and written once.  A
// head vector is cut into units of two VE-element pieces, the two that hold a
// rotation's pairs (piece u of the first half and of the second; the interleaved
// layout's pairs lie inside a piece, so there any two do, and they are taken so that a
// group reads whole lines at once), so that every pair sits in one thread;
// a group of lanes (the next power of two) takes one vector.  Angles depend on
// (token, pair) alone, so a group takes several heads of one token with the same
// sines.  What it takes to fill the memory is bytes in flight, and registers hold
// too few of them next to sines, weights and sums: each thread copies its pieces of
// the next vectors to slots of its own in shared memory (cp.async), several vectors
// ahead, over the borders of tokens too, and needs no barrier to read them.
// Measured in replayed graphs, bfloat16 of width 128: rotation of half of the head, 65536 rows x 20 heads,
// interleaved, 107 us, 6.2 TB/s, 0.95 of the measured copy rate (183 us with the pieces loaded to
// registers); norm and rotation of 16384 x 40 heads 63 us, 5.3 TB/s, 0.82 (143 us); its gradient
// 110 us, 4.6 TB/s, 0.70 (272 us): what is left there is not the memory but chains of the sums over a group's lanes, the
// sines and shared-memory reads, at four warps a scheduler.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <memory>

#include "pn_seq.cuh"

namespace pn {

pn_status seq_fail(pn_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_thread_error(buf);
  return st;
}

pn_status seq_device(const void* p, const char* name, int* dev) {
  if (!p) return seq_fail(PN_ERR_INVALID, "%s is NULL", name);
  cudaPointerAttributes at;
  const cudaError_t e = cudaPointerGetAttributes(&at, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return seq_fail(PN_ERR_INVALID, "%s is not a CUDA pointer (%s)", name, cudaGetErrorString(e));
  }
  if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged)
    return seq_fail(PN_ERR_INVALID, "%s is not device memory", name);
  if (*dev < 0) *dev = at.device;
  else if (at.type == cudaMemoryTypeDevice && at.device != *dev)
    return seq_fail(PN_ERR_INVALID, "%s is on device %d, the first array on device %d", name, at.device, *dev);
  return PN_OK;
}

pn_status seq_output(const pn_heads* y, const char* name, long long B, long long T, int H, int dim) {
  if ((B > 1 && y->batch_stride < dim) || (T > 1 && y->token_stride < dim) || (H > 1 && y->head_stride < dim))
    return seq_fail(PN_ERR_INVALID, "%s has overlapping rows", name);
  return PN_OK;
}

pn_status seq_apart(const void* y, const char* name, const void* x, const char* other) {
  if (y == x) return seq_fail(PN_ERR_INVALID, "%s is the memory of %s", name, other);
  return PN_OK;
}

namespace {

struct HeadsArgs {
  int tokens;            // T of one batch entry
  long long rows;        // B * T
  int heads[2];          // query and key heads
  int blocks[2];         // blocks of hb heads per token
  int hb[2];
  int dim, rot;
  int half_units;        // units that hold rotated pairs of the half layout (0: interleaved)
  int units;
  int interleaved;
  float sign;            // +1, or -1 for the inverse rotation
  float m;
  float eps;
  float inv_dim;
  int items_fit;         // the list's numbers fit 31 bits
  int w_f32;             // weights are float32 (else the tensors' type)
  const long long* positions;
  const void* w[2];
  const void* x[2];      // inputs of the norm (or of the rotation)
  const void* g[2];      // gradient: of the outputs
  void* y[2];
  long long xs[2][3], gs[2][3], ys[2][3];   // batch, token, head strides in elements
  float* partial;        // gradient: [grid][dim] partial sums of the weights' gradients
  int grid_q;            // gradient: CTAs that take queries (the rest takes keys)
  unsigned long long turn[kMaxRotPairs];
};

constexpr int kHeadThreads = 256;

constexpr int ahead(bool grad) { return grad ? 3 : 5; }   // slots: vectors on their way, and the one at hand

template <int BYTES> __device__ __forceinline__ void copy_async(void* dst, const void* src) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(BYTES) : "memory");
}

// One (token, block of heads) of a group's list.
struct HeadsItem {
  int kind, h0, h1;
  long long b, t;
  __device__ __forceinline__ void at(const HeadsArgs& A, long long it, int kind0, int per_token, bool grad) {
    // (32-bit divisions where they reach: 64-bit ones take a hundred instructions)
    int blk;
    if (A.items_fit) {
      const unsigned r = (unsigned)it / (unsigned)per_token;
      blk = (int)((unsigned)it - r * (unsigned)per_token);
      const unsigned bb = r / (unsigned)A.tokens;
      b = bb;
      t = r - bb * (unsigned)A.tokens;
    } else {
      const long long row = it / per_token;
      blk = (int)(it - row * per_token);
      b = row / A.tokens;
      t = row - b * A.tokens;
    }
    kind = kind0;
    if (!grad && blk >= A.blocks[0]) {
      kind = 1;
      blk -= A.blocks[0];
    }
    h0 = blk * A.hb[kind];
    h1 = min(A.heads[kind], h0 + A.hb[kind]);
  }
};

// NU units per lane (1 for VE >= 4, where 32 lanes hold the widest vector)
template <typename T, int VE, int NU, bool NORM, bool GRAD>
__global__ void __launch_bounds__(kHeadThreads, VE < 4 ? 1 : GRAD ? 2 : 3) heads_kernel(const __grid_constant__ HeadsArgs A, int group) {
  constexpr bool kAsync = VE >= 4;            // (single elements are read straight)
  constexpr int kSlots = kAsync ? ahead(GRAD) : 1;
  constexpr int kPieces = GRAD ? 4 : 2;       // of one vector, or of it and its gradient
  using Piece = typename RawVec<VE * (int)sizeof(T)>::type;
  __shared__ unsigned long long s_turn[kMaxRotPairs];
  __shared__ __align__(16) float s_w[NORM ? 512 : 4];   // both weights
  extern __shared__ __align__(16) unsigned char s_heads[];
  Piece* slots = reinterpret_cast<Piece*>(s_heads) + threadIdx.x;   // piece p of slot s at (s * kPieces + p) * kHeadThreads
  float* s_dw = reinterpret_cast<float*>(s_heads);                  // GRAD, at the end: [kHeadThreads / group][dim]
  const int pairs = A.rot >> 1;
  for (int i = threadIdx.x; i < pairs; i += kHeadThreads) s_turn[i] = A.turn[i];
  if constexpr (NORM) {
    for (int i = threadIdx.x; i < 2 * A.dim; i += kHeadThreads) {
      const int kind = i >= A.dim, j = i - kind * A.dim;
      s_w[i] = A.w_f32 ? ((const float*)A.w[kind])[j] : to_f<T>(((const T*)A.w[kind])[j]);
    }
  }
  __syncthreads();

  const int lane = threadIdx.x & (group - 1);
  const int per_cta = kHeadThreads / group;
  const int sub = threadIdx.x / group;
  const unsigned mask = group == 32 ? 0xffffffffu : ((1u << group) - 1u) << ((threadIdx.x & 31) & ~(group - 1));

  // the pieces of this lane's units: element offsets, and whether they exist
  int c0[NU], c1[NU];
  bool on0[NU], on1[NU];
#pragma unroll
  for (int n = 0; n < NU; ++n) {
    const int u = lane + n * group;
    if (u < A.half_units) {
      c0[n] = u * VE;
      c1[n] = c0[n] + A.half_units * VE;
    } else if (VE == 1) {   // (an interleaved pair)
      c0[n] = 2 * u;
      c1[n] = c0[n] + 1;
    } else {                // whole lines to a load, as above
      c0[n] = (A.half_units + u) * VE;
      c1[n] = c0[n] + (A.units - A.half_units) * VE;
    }
    on0[n] = u < A.units && c0[n] < A.dim;
    on1[n] = u < A.units && c1[n] < A.dim;
  }

  // items: (token, block of hb heads); the gradient's CTAs take queries only or keys only
  const int kind0 = GRAD ? ((int)blockIdx.x >= A.grid_q ? 1 : 0) : 0;
  const int per_token = GRAD ? A.blocks[kind0] : A.blocks[0] + A.blocks[1];
  const long long items = A.rows * per_token;
  const long long first = (long long)(GRAD && kind0 ? blockIdx.x - A.grid_q : blockIdx.x) * per_cta + sub;
  const long long stride = (long long)(GRAD ? (kind0 ? gridDim.x - A.grid_q : A.grid_q) : gridDim.x) * per_cta;

  float dw[GRAD ? 2 * NU : 1][VE] = {};

  // the vectors on their way
  HeadsItem next;
  long long next_it = first;
  int next_h = 0;
  const T *next_x = nullptr, *next_g = nullptr;
  auto open = [&]() {
    next.at(A, next_it, kind0, per_token, GRAD);
    next_h = next.h0;
    next_x = (const T*)A.x[next.kind] + next.b * A.xs[next.kind][0] + next.t * A.xs[next.kind][1] + next_h * A.xs[next.kind][2];
    if constexpr (GRAD) next_g = (const T*)A.g[next.kind] + next.b * A.gs[next.kind][0] + next.t * A.gs[next.kind][1] + next_h * A.gs[next.kind][2];
  };
  auto fetch = [&](int slot) {
    if constexpr (kAsync) {
      if (next_it < items) {
        Piece* to = slots + slot * (kPieces * kHeadThreads);
        if (on0[0]) copy_async<sizeof(Piece)>(to, next_x + c0[0]);
        if (on1[0]) copy_async<sizeof(Piece)>(to + kHeadThreads, next_x + c1[0]);
        next_x += A.xs[next.kind][2];
        if constexpr (GRAD) {
          if (on0[0]) copy_async<sizeof(Piece)>(to + 2 * kHeadThreads, next_g + c0[0]);
          if (on1[0]) copy_async<sizeof(Piece)>(to + 3 * kHeadThreads, next_g + c1[0]);
          next_g += A.gs[next.kind][2];
        }
        if (++next_h == next.h1) {
          next_it += stride;
          if (next_it < items) open();
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
  int slot = 0;
  if constexpr (kAsync) {
    for (int i = 0; i < kSlots * kPieces; ++i) slots[i * kHeadThreads] = Piece{};   // pieces that do not exist stay zero
    if (next_it < items) open();
    for (int i = 0; i < kSlots - 1; ++i) fetch(i);
  }

  auto position_of = [&](long long it) {
    if (!pairs || it >= items) return 0LL;
    return A.positions[A.items_fit ? (long long)((unsigned)it / (unsigned)per_token) : it / per_token];
  };
  long long next_pos = position_of(first);   // (a load ahead, or each item would begin with a wait for it)
  for (long long it = first; it < items; it += stride) {
    HeadsItem cur;
    cur.at(A, it, kind0, per_token, GRAD);
    const int kind = cur.kind;
    const long long pos = next_pos;
    next_pos = position_of(it + stride);

    float cs[NU][VE], sn[NU][VE];   // of the pairs this lane holds
    if (pairs) {
#pragma unroll
      for (int n = 0; n < NU; ++n) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          // half layout: pair c0 + e.  interleaved: VE / 2 pairs in each piece (VE = 1: one pair in both)
          int p;
          if (!A.interleaved) p = c0[n] + e;
          else if (VE == 1) p = c0[n] >> 1;
          else p = (e < VE / 2) ? (c0[n] >> 1) + e : (c1[n] >> 1) + e - VE / 2;
          const bool live = A.interleaved ? p < pairs : (lane + n * group) < A.half_units;
          cs[n][e] = 1.0f;
          sn[n][e] = 0.0f;
          if (live && on0[n]) {
            turn_cos_sin<sizeof(T) == 2 && !GRAD>(s_turn[p], pos, A.m, cs[n][e], sn[n][e]);
            sn[n][e] *= A.sign;
          }
        }
      }
    }
    const float* wk = s_w + kind * A.dim;   // (registers are short: the weights stay in shared memory)
    auto weights = [&](int n, int i, float (&w)[VE]) {
      const int c = i ? c1[n] : c0[n];
      const bool on = i ? on1[n] : on0[n];
#pragma unroll
      for (int e = 0; e < VE; ++e) w[e] = 0.0f;
      if constexpr (VE >= 4) {
        if (on) {
#pragma unroll
          for (int e = 0; e < VE; e += 4) {
            const float4 f = *reinterpret_cast<const float4*>(wk + c + e);
            w[e] = f.x;
            w[e + 1] = f.y;
            w[e + 2] = f.z;
            w[e + 3] = f.w;
          }
        }
      } else if (on) {
        w[0] = wk[c];
      }
    };
    T* yp = (T*)A.y[kind] + cur.b * A.ys[kind][0] + cur.t * A.ys[kind][1] + cur.h0 * A.ys[kind][2];

    // v (two pieces of each unit) turned by sign * angle.  What does not rotate is not touched: times 1 and 0, a NaN or an
    // infinity would reach the element beside it.  (Behind a norm, whose sum such a value reaches anyway, it is multiplied: the
    // branches cost 3 % there, 62.6 and 64.8 us at 16384 x 40 bfloat16 heads of 128, and 1 % of a rotation alone.)
    auto rotate = [&](float (&v)[2 * NU][VE]) {
      if (!pairs) return;
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        const int u = lane + n * group;
        if (!A.interleaved || VE == 1) {
          if (!NORM && u >= (A.interleaved ? pairs : A.half_units)) continue;
          float p[VE], q[VE];
          mul_vec<VE>(v[2 * n + 1], sn[n], p);
          mul_vec<VE>(v[2 * n], sn[n], q);
#pragma unroll
          for (int e = 0; e < VE; ++e) v[2 * n][e] = fmaf(v[2 * n][e], cs[n][e], -p[e]);
          fma_vec<VE>(v[2 * n + 1], cs[n], q, v[2 * n + 1]);
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int live = pairs - ((j ? c1[n] : c0[n]) >> 1);   // pairs of this piece that rotate
#pragma unroll
            for (int e = 0; e < VE / 2; ++e) {
              if (!NORM && e >= live) continue;
              const float c = cs[n][e + j * (VE / 2)], s = sn[n][e + j * (VE / 2)];
              const float a = v[2 * n + j][2 * e], q = v[2 * n + j][2 * e + 1];
              v[2 * n + j][2 * e] = a * c - q * s;
              v[2 * n + j][2 * e + 1] = q * c + a * s;
            }
          }
        }
      }
    };
    auto sum_group = [&](float v) {
      for (int o = group >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
      return v;
    };
    // vector h of x (which = 0) or of the gradient (1)
    auto load = [&](int h, int which, float (&v)[2 * NU][VE]) {
      if constexpr (kAsync) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          VecOf<T, VE> u;
          u.raw = slots[(slot * kPieces + 2 * which + i) * kHeadThreads];
          u.widen(v[i]);
        }
      } else {
        const long long* st = which ? A.gs[kind] : A.xs[kind];
        const T* p = (const T*)(which ? A.g[kind] : A.x[kind]) + cur.b * st[0] + cur.t * st[1] + h * st[2];
#pragma unroll
        for (int n = 0; n < NU; ++n) {
#pragma unroll
          for (int e = 0; e < VE; ++e) v[2 * n][e] = v[2 * n + 1][e] = 0.0f;
          if (on0[n]) ld_vec<T, VE>(p + c0[n], v[2 * n]);
          if (on1[n]) ld_vec<T, VE>(p + c1[n], v[2 * n + 1]);
        }
      }
    };

    for (int h = cur.h0; h < cur.h1; ++h) {
      if constexpr (kAsync) {
        fetch(slot ? slot - 1 : kSlots - 1);   // the slot read last
        asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
      }
      float x[2 * NU][VE];
      load(h, 0, x);
      float r = 1.0f;
      if constexpr (NORM) {
        unsigned long long s2 = 0;
#pragma unroll
        for (int i = 0; i < 2 * NU; ++i) dot_vec<VE>(x[i], x[i], s2);
        float s0, s1;
        unpack2(s2, s0, s1);
        r = rsqrtf(fmaf(sum_group(s0 + s1), A.inv_dim, A.eps));
      }
      if constexpr (GRAD) {
        float g[2 * NU][VE];
        load(h, 1, g);
        rotate(g);
        unsigned long long u2 = 0;
#pragma unroll
        for (int i = 0; i < 2 * NU; ++i) {
          scale_vec<VE>(r, x[i]);                       // n
          fma_vec<VE>(g[i], x[i], dw[i], dw[i]);
          float w[VE];
          weights(i >> 1, i & 1, w);
          mul_vec<VE>(g[i], w, g[i]);                   // u
          dot_vec<VE>(g[i], x[i], u2);
        }
        float u0, u1;
        unpack2(u2, u0, u1);
        const float un = -sum_group(u0 + u1) * A.inv_dim;
        float m[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) m[e] = un;
#pragma unroll
        for (int i = 0; i < 2 * NU; ++i) {
          fma_vec<VE>(x[i], m, g[i], x[i]);
          scale_vec<VE>(r, x[i]);
        }
      } else {
        if constexpr (NORM) {
#pragma unroll
          for (int i = 0; i < 2 * NU; ++i) {
            scale_vec<VE>(r, x[i]);
            float w[VE];
            weights(i >> 1, i & 1, w);
            mul_vec<VE>(x[i], w, x[i]);
          }
        }
        rotate(x);
      }
      T* o = yp;
      yp += A.ys[kind][2];
      if constexpr (kAsync) slot = slot + 1 == kSlots ? 0 : slot + 1;
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        if (on0[n]) st_vec<T, VE>(o + c0[n], x[2 * n]);
        if (on1[n]) st_vec<T, VE>(o + c1[n], x[2 * n + 1]);
      }
    }
  }

  if constexpr (GRAD) {
    // this CTA's sums, in the order of its groups
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NU; ++n)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        if (on0[n]) s_dw[sub * A.dim + c0[n] + e] = dw[2 * n][e];
        if (on1[n]) s_dw[sub * A.dim + c1[n] + e] = dw[2 * n + 1][e];
      }
    __syncthreads();
    for (int j = threadIdx.x; j < A.dim; j += kHeadThreads) {
      float s = 0.0f;
      for (int i = 0; i < per_cta; ++i) s += s_dw[i * A.dim + j];
      A.partial[(long long)blockIdx.x * A.dim + j] = s;
    }
  }
}

// dw[kind][j] = sum of the partial sums of that kind's CTAs, in one fixed order
__global__ void __launch_bounds__(256) dw_reduce_kernel(const float* __restrict__ partial, int grid_q, int grid, int dim,
                                                        float* dwq, float* dwk) {
  __shared__ float s[8][33];
  const int kind = blockIdx.y;
  const int lo = kind ? grid_q : 0, hi = kind ? grid : grid_q;
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + c;
  float v = 0.0f;
  if (j < dim)
    for (int i = lo + g; i < hi; i += 8) v += partial[(long long)i * dim + j];
  s[g][c] = v;
  __syncthreads();
  if (g == 0 && j < dim) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += s[i][c];
    (kind ? dwk : dwq)[j] = v;
  }
}

pn_status check_heads(const pn_heads* h, const char* name) {
  if (!h) return seq_fail(PN_ERR_INVALID, "%s is NULL", name);
  if (h->batch_stride < 0 || h->token_stride < 0 || h->head_stride < 0)
    return seq_fail(PN_ERR_INVALID, "%s has a negative stride", name);
  return PN_OK;
}

bool aligned_to(const pn_heads* h, size_t es, int ve) {
  const size_t bytes = es * ve;
  return ((uintptr_t)h->data % bytes) == 0 && h->batch_stride % ve == 0 && h->token_stride % ve == 0 &&
         h->head_stride % ve == 0;
}

constexpr int kGradCtasPerSm = 2;   // as many as run at once: each starts and sums once (4: 131 us in place of 116 at 16384 x 40 heads of 128)

// CTAs of the gradient: queries first, then keys, in the ratio of their heads
void grad_grid(long long rows, int Hq, int Hk, int* gq, int* gk) {
  const int total = 148 * kGradCtasPerSm;
  long long q = std::max(1LL, (long long)total * Hq / (Hq + Hk));
  long long k = std::max(1LL, (long long)total - q);
  q = std::min(q, (rows * Hq + 7) / 8);   // no more CTAs than groups of vectors
  k = std::min(k, (rows * Hk + 7) / 8);
  *gq = (int)std::max(1LL, q);
  *gk = (int)std::max(1LL, k);
}

template <typename T, int VE, int NU, bool NORM, bool GRAD>
cudaError_t launch_heads(const HeadsArgs& A, int grid, int group, size_t smem, cudaStream_t st) {
  if (smem > 40 * 1024) {   // (48 KB with what the kernel has of its own)
    const cudaError_t e = cudaFuncSetAttribute(heads_kernel<T, VE, NU, NORM, GRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  heads_kernel<T, VE, NU, NORM, GRAD><<<grid, kHeadThreads, smem, st>>>(A, group);
  return cudaGetLastError();
}

template <typename T, int VE, int NU>
cudaError_t launch_kind(const HeadsArgs& A, bool norm, bool grad, int grid, int group, size_t smem, cudaStream_t st) {
  if (grad) return launch_heads<T, VE, NU, true, true>(A, grid, group, smem, st);
  if (norm) return launch_heads<T, VE, NU, true, false>(A, grid, group, smem, st);
  return launch_heads<T, VE, NU, false, false>(A, grid, group, smem, st);
}

template <typename T>
cudaError_t launch_type(const HeadsArgs& A, int ve, bool norm, bool grad, int grid, int group, size_t smem, cudaStream_t st) {
  if constexpr (sizeof(T) == 2) {
    if (ve == 8) return launch_kind<T, 8, 1>(A, norm, grad, grid, group, smem, st);
  }
  if (ve == 4) return launch_kind<T, 4, 1>(A, norm, grad, grid, group, smem, st);
  return launch_kind<T, 1, 4>(A, norm, grad, grid, group, smem, st);
}

// One pass over q and k: `g` (the gradients of the outputs) makes it the norm's gradient.
pn_status run_heads(const pn_rotary_plan* r, int dtype, int B, int T, int Hq, int Hk, int dim, const pn_heads* q,
                    const pn_heads* k, const pn_heads* gq, const pn_heads* gk, const long long* positions, float sign,
                    const void* wq, const void* wk, int w_dtype, float eps, const pn_heads* yq, const pn_heads* yk,
                    float* dwq, float* dwk, void* ws, size_t ws_bytes, cudaStream_t st) {
  const bool norm = wq != nullptr, grad = gq != nullptr;
  if (dtype != PN_F32 && dtype != PN_BF16 && dtype != PN_F16) return seq_fail(PN_ERR_INVALID, "unknown dtype %d", dtype);
  if (B < 0 || T < 0 || Hq < 1 || Hk < 1) return seq_fail(PN_ERR_INVALID, "bad shape B=%d T=%d Hq=%d Hk=%d", B, T, Hq, Hk);
  if (dim < 2 || dim > 256 || (dim & 1)) return seq_fail(PN_ERR_INVALID, "dim=%d: an even number up to 256", dim);
  if (r && 2 * r->pairs > dim) return seq_fail(PN_ERR_INVALID, "rot_dim=%d exceeds dim=%d", 2 * r->pairs, dim);
  const pn_heads* every[] = {q, k, yq, yk, gq, gk};
  const char* names[] = {"q", "k", "q_out", "k_out", "dq_out", "dk_out"};
  for (int i = 0; i < (grad ? 6 : 4); ++i)
    if (pn_status e = check_heads(every[i], names[i])) return e;
  if (norm) {
    if (!wk) return seq_fail(PN_ERR_INVALID, "wk is NULL");
    if (w_dtype != PN_F32 && w_dtype != dtype) return seq_fail(PN_ERR_INVALID, "weights: float32 or the tensors' type");
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return seq_fail(PN_ERR_INVALID, "eps must be finite and >= 0");
  }
  if (grad && (!dwq || !dwk)) return seq_fail(PN_ERR_INVALID, "dwq or dwk is NULL");
  const long long rows = (long long)B * T;
  int dev = -1;
  if (rows > 0) {
    for (int i = 0; i < (grad ? 6 : 4); ++i)
      if (pn_status e = seq_device(every[i]->data, names[i], &dev)) return e;
    if (r)
      if (pn_status e = seq_device(positions, "positions", &dev)) return e;
  }
  if (norm && (rows > 0 || grad)) {
    if (pn_status e = seq_device(wq, "wq", &dev)) return e;
    if (pn_status e = seq_device(wk, "wk", &dev)) return e;
  }
  if (grad) {
    if (pn_status e = seq_device(dwq, "dwq", &dev)) return e;
    if (pn_status e = seq_device(dwk, "dwk", &dev)) return e;
  }
  for (int i = 0; i < (grad ? 6 : 4) && rows > 0; ++i)
    if ((uintptr_t)every[i]->data % dtype_size(dtype)) return seq_fail(PN_ERR_INVALID, "%s is misaligned", names[i]);
  for (int o = 2; o < 4 && rows > 0; ++o) {   // an output may be the input or the gradient that it takes the place of, no other array
    const int H = o == 2 ? Hq : Hk;
    if (pn_status e = seq_output(every[o], names[o], B, T, H, dim)) return e;
    for (int i = 0; i < (grad ? 6 : 4); ++i) {
      if (i == o) continue;
      const bool in_place = (i & 1) == (o & 1) && (B == 1 || every[i]->batch_stride == every[o]->batch_stride) &&
                            (T == 1 || every[i]->token_stride == every[o]->token_stride) &&
                            (H == 1 || every[i]->head_stride == every[o]->head_stride);
      if (in_place) continue;
      if (pn_status e = seq_apart(every[o]->data, names[o], every[i]->data, names[i])) return e;
    }
  }
  if (rows == 0 && !grad) return PN_OK;
  SeqDeviceGuard dg(dev);
  if (rows == 0) {
    cudaError_t e = cudaMemsetAsync(dwq, 0, dim * sizeof(float), st);
    if (e == cudaSuccess) e = cudaMemsetAsync(dwk, 0, dim * sizeof(float), st);
    if (e != cudaSuccess) return seq_fail(PN_ERR_CUDA, "clearing the weights' gradients failed: %s", cudaGetErrorString(e));
    return PN_OK;
  }

  HeadsArgs A = {};
  A.tokens = T;
  A.rows = rows;
  A.heads[0] = Hq;
  A.heads[1] = Hk;
  A.dim = dim;
  A.rot = r ? 2 * r->pairs : 0;
  A.interleaved = r ? r->interleaved : 0;
  A.sign = sign;
  A.m = r ? r->factor : 1.0f;
  A.eps = eps;
  A.inv_dim = 1.0f / (float)dim;
  A.items_fit = rows * (Hq + Hk) < (1LL << 30);
  A.w_f32 = w_dtype == PN_F32;
  A.positions = positions;
  A.w[0] = wq;
  A.w[1] = wk;
  if (r) std::copy(r->turn, r->turn + r->pairs, A.turn);
  auto put = [](const pn_heads* h, long long (&s)[3]) {
    s[0] = h->batch_stride;
    s[1] = h->token_stride;
    s[2] = h->head_stride;
  };
  A.x[0] = q->data;
  A.x[1] = k->data;
  put(q, A.xs[0]);
  put(k, A.xs[1]);
  A.y[0] = yq->data;
  A.y[1] = yk->data;
  put(yq, A.ys[0]);
  put(yk, A.ys[1]);
  if (grad) {
    A.g[0] = gq->data;
    A.g[1] = gk->data;
    put(gq, A.gs[0]);
    put(gk, A.gs[1]);
  }

  // the widest piece that the addresses, the strides and the halves of the rotation allow
  const size_t es = dtype_size(dtype);
  auto fits = [&](int ve) {
    if (dim % ve) return false;
    if (r && !r->interleaved && r->pairs % ve) return false;
    for (int i = 0; i < (grad ? 6 : 4); ++i)
      if (!aligned_to(every[i], es, ve)) return false;
    return true;
  };
  const int ve = (es == 2 && fits(8)) ? 8 : fits(4) ? 4 : 1;
  A.half_units = (r && !r->interleaved) ? r->pairs / ve : 0;
  const int rest = dim / ve - 2 * A.half_units;   // pieces behind the rotated halves
  A.units = A.half_units + (rest + 1) / 2;
  int group = 1;
  while (group < 32 && group < A.units) group <<= 1;

  // heads per group: as many as keep the card's threads busy (the sines are shared among them)
  const int per_cta = kHeadThreads / group;
  const long long vectors = rows * (Hq + Hk);
  int hb = 1;
  while (hb < 8 && vectors / (2 * hb) >= 148LL * 4 * per_cta) hb <<= 1;
  for (int i = 0; i < 2; ++i) {   // in blocks of nearly one size (12 heads: 6 and 6, not 8 and 4)
    A.blocks[i] = (A.heads[i] + hb - 1) / hb;
    A.hb[i] = (A.heads[i] + A.blocks[i] - 1) / A.blocks[i];
  }

  int grid;
  size_t smem = 0;
  if (grad) {
    int gk_ = 0;
    grad_grid(rows, Hq, Hk, &A.grid_q, &gk_);
    grid = A.grid_q + gk_;
    const size_t need = (size_t)grid * dim * sizeof(float);
    if (ws_bytes < need) return seq_fail(PN_ERR_INVALID, "workspace of %zu bytes, %zu needed", ws_bytes, need);
    if (pn_status e = seq_device(ws, "workspace", &dev)) return e;
    if ((uintptr_t)ws & 15u) return seq_fail(PN_ERR_INVALID, "workspace must be 16-byte aligned");
    A.partial = (float*)ws;
  } else {
    const long long items = rows * (A.blocks[0] + A.blocks[1]);
    // Where instructions bound it (the norm of 16-bit vectors; groups with idle lanes), as many CTAs as run at once, each with a
    // long list, else more and shorter ones, which even out the SMs' shares of the memory: 3 against 16 on an SM, norm of 16384 x
    // 40 bfloat16 heads of 128 63 and 73 us, rotation of 6135 x 24 float32 heads of 80 21 and 23; rotation of 65536 x 20 bfloat16
    // heads of 128 128 and 107, norm of 16384 x 20 float32 heads of 128 67 and 61.
    const bool busy = ve > 1 && ((norm && es == 2) || A.units < group);
    grid = (int)std::min<long long>((items + per_cta - 1) / per_cta, 148LL * (busy ? 3 : 16));
  }
  // the slots; the gradient's sums lie in the same memory
  smem = ve == 1 ? 0 : (size_t)ahead(grad) * (grad ? 4 : 2) * kHeadThreads * ve * es;
  if (grad) smem = std::max(smem, (size_t)per_cta * dim * sizeof(float));
  cudaError_t e = dtype == PN_F32    ? launch_type<float>(A, ve, norm, grad, grid, group, smem, st)
                  : dtype == PN_BF16 ? launch_type<__nv_bfloat16>(A, ve, norm, grad, grid, group, smem, st)
                                     : launch_type<__half>(A, ve, norm, grad, grid, group, smem, st);
  if (e == cudaSuccess && grad) {
    dw_reduce_kernel<<<dim3((dim + 31) / 32, 2), 256, 0, st>>>(A.partial, A.grid_q, grid, dim, dwq, dwk);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return seq_fail(PN_ERR_CUDA, "launch failed: %s", cudaGetErrorString(e));
  return PN_OK;
}

}  // namespace
}  // namespace pn

using namespace pn;

extern "C" {

pn_status pn_rotary_create(pn_rotary* out, const pn_rotary_desc* d) {
  if (!out) return seq_fail(PN_ERR_INVALID, "out is NULL");
  *out = nullptr;
  if (!d) return seq_fail(PN_ERR_INVALID, "desc is NULL");
  if (d->rot_dim < 2 || d->rot_dim > 2 * kMaxRotPairs || (d->rot_dim & 1))
    return seq_fail(PN_ERR_INVALID, "rot_dim=%d: an even number from 2 to %d", d->rot_dim, 2 * kMaxRotPairs);
  if (d->layout != PN_ROT_HALF && d->layout != PN_ROT_INTERLEAVED)
    return seq_fail(PN_ERR_INVALID, "unknown layout %d", d->layout);
  if (d->scaling < PN_ROT_PLAIN || d->scaling > PN_ROT_YARN) return seq_fail(PN_ERR_INVALID, "unknown scaling %d", d->scaling);
  if (!(d->base > 1.0) || !std::isfinite(d->base)) return seq_fail(PN_ERR_INVALID, "base must be finite and > 1");
  const bool scaled = d->scaling != PN_ROT_PLAIN;
  if (scaled && (!(d->factor >= 1.0) || !std::isfinite(d->factor)))
    return seq_fail(PN_ERR_INVALID, "factor must be finite and >= 1");
  if (d->scaling == PN_ROT_NTK && d->rot_dim < 4) return seq_fail(PN_ERR_INVALID, "ntk scaling needs rot_dim >= 4");
  if (d->scaling == PN_ROT_YARN &&
      (d->original_length < 1 || !(d->beta_slow >= 0.0) || !(d->beta_fast > d->beta_slow) || !std::isfinite(d->beta_fast)))
    return seq_fail(PN_ERR_INVALID, "yarn needs original_length >= 1 and beta_fast > beta_slow >= 0");
  if (!(d->attention_scale >= 0.0) || !std::isfinite((float)d->attention_scale) ||
      (d->attention_scale > 0.0 && (float)d->attention_scale == 0.0f))
    return seq_fail(PN_ERR_INVALID, "attention_scale must be finite and >= 0, as a float32 too");
  pn_rotary_plan* p = new (std::nothrow) pn_rotary_plan();
  if (!p) return seq_fail(PN_ERR_NOMEM, "out of host memory");
  p->pairs = d->rot_dim / 2;
  p->interleaved = d->layout == PN_ROT_INTERLEAVED;
  const long double two_pi = 6.283185307179586476925286766559005768L;
  const long double s = scaled ? (long double)d->factor : 1.0L;
  long double base = d->base;
  if (d->scaling == PN_ROT_NTK) base *= powl(s, (long double)d->rot_dim / (d->rot_dim - 2));
  // base^(-2i/rot_dim) as a product of two powers, i in eights and the rest: off by 2.5 units of 2^-64 at most, which with
  // the turn's own rounding (2 pi 2^-65) stays below 2^-61, and a plan of 64 pairs takes 9 us (24 with a power for each)
  long double fine[8];
  for (int i = 0; i < 8; ++i) fine[i] = powl(base, -2.0L * i / d->rot_dim);
  long double coarse = 1.0L;
  for (int i = 0; i < p->pairs; ++i) {
    if (i % 8 == 0) coarse = powl(base, -2.0L * i / d->rot_dim);
    long double f = coarse * fine[i % 8];
    if (d->scaling == PN_ROT_LINEAR) f /= s;
    if (d->scaling == PN_ROT_YARN) {
      const long double turns = (long double)d->original_length * f / two_pi;
      const long double keep =
          std::min(1.0L, std::max(0.0L, (turns - (long double)d->beta_slow) / ((long double)d->beta_fast - d->beta_slow)));
      f *= keep + (1.0L - keep) / s;
    }
    const long double frac = fmodl(f / two_pi, 1.0L);   // f <= 1
    p->turn[i] = (unsigned long long)roundl(frac * 18446744073709551616.0L);
  }
  p->factor = d->attention_scale > 0.0 ? (float)d->attention_scale
              : d->scaling == PN_ROT_YARN ? (float)(0.1L * logl(s) + 1.0L) : 1.0f;
  *out = p;
  return PN_OK;
}

void pn_rotary_destroy(pn_rotary r) { delete r; }

pn_status pn_rotary_apply(pn_rotary r, int dtype, int B, int T, int Hq, int Hk, int dim, const pn_heads* q,
                          const pn_heads* k, const long long* positions, int inverse, const pn_heads* q_out,
                          const pn_heads* k_out, void* cuda_stream) {
  if (!r) return seq_fail(PN_ERR_INVALID, "rotary is NULL");
  if (inverse != 0 && inverse != 1) return seq_fail(PN_ERR_INVALID, "inverse must be 0 or 1");
  return run_heads(r, dtype, B, T, Hq, Hk, dim, q, k, nullptr, nullptr, positions, inverse ? -1.0f : 1.0f, nullptr, nullptr,
                   0, 0.0f, q_out, k_out, nullptr, nullptr, nullptr, 0, (cudaStream_t)cuda_stream);
}

pn_status pn_norm_rotary_apply(pn_rotary r, int dtype, int B, int T, int Hq, int Hk, int dim, const pn_heads* q,
                               const pn_heads* k, const long long* positions, const void* wq, const void* wk, int w_dtype,
                               float eps, const pn_heads* q_out, const pn_heads* k_out, void* cuda_stream) {
  if (!wq || !wk) return seq_fail(PN_ERR_INVALID, "wq or wk is NULL");
  return run_heads(r, dtype, B, T, Hq, Hk, dim, q, k, nullptr, nullptr, positions, 1.0f, wq, wk, w_dtype, eps, q_out, k_out,
                   nullptr, nullptr, nullptr, 0, (cudaStream_t)cuda_stream);
}

size_t pn_norm_rotary_workspace(int B, int T, int Hq, int Hk, int dim) {
  if (B < 0 || T < 0 || Hq < 1 || Hk < 1 || dim < 2 || dim > 256) return 0;
  int gq, gk;
  grad_grid((long long)B * T, Hq, Hk, &gq, &gk);
  return (size_t)(gq + gk) * dim * sizeof(float);
}

pn_status pn_norm_rotary_backward(pn_rotary r, int dtype, int B, int T, int Hq, int Hk, int dim, const pn_heads* dq_out,
                                  const pn_heads* dk_out, const pn_heads* q, const pn_heads* k, const long long* positions,
                                  const void* wq, const void* wk, int w_dtype, float eps, const pn_heads* dq,
                                  const pn_heads* dk, float* dwq, float* dwk, void* workspace, size_t workspace_bytes,
                                  void* cuda_stream) {
  if (!wq || !wk) return seq_fail(PN_ERR_INVALID, "wq or wk is NULL");
  if (!dq_out || !dk_out) return seq_fail(PN_ERR_INVALID, "dq_out or dk_out is NULL");
  return run_heads(r, dtype, B, T, Hq, Hk, dim, q, k, dq_out, dk_out, positions, -1.0f, wq, wk, w_dtype, eps, dq, dk, dwq,
                   dwk, workspace, workspace_bytes, (cudaStream_t)cuda_stream);
}

}  // extern "C"
