// pn_linattn.cuh -- linear attention with a decay for each head: the parameter
// block of one pass over the rows, and the FP32 kernels.
//
//   S_t = e^{g_h} S_{t-1} + alpha b_t c_t^T,   out_t = beta a_t S_t
//
// is evaluated by chunks of C rows.  With S what leaves the chunk before,
//   out_i = beta [ e^{g(i+1)} a_i S + alpha sum_{j<=i} e^{g(i-j)} (a_i . b_j) c_j ],
//   S'    = e^{gC} S + alpha sum_j e^{g(C-1-j)} b_j c_j^T.
// Forward: (a, b, c) = (q, k, v).  Gradients are the same pass over other
// operands, two of them against time (row index counted from the end, and the
// state that enters is the gradient of the last state, which the last row
// still sees undecayed):
//   dq: (do, v, k) in time, S transposed;   dk: (v, do, q) and dv: (k, q, do) against time.
#pragma once

#include "pn_seq.cuh"

constexpr int kMaxLinHeads = 256;

struct pn_linattn_s {
  int H, Hkv, dk, dv, dtype;
  float scale;
  float log2_decay[kMaxLinHeads];
};

namespace pn {

struct LinOperand {
  const void* p;
  long long bs, ts, hs;   // batch, token, head strides in elements
  int per;                // consecutive heads that share one of the operand's
};

struct LinPass {
  LinOperand a, b, c;
  void* out;
  long long out_bs, out_ts, out_hs;
  int out_f32;             // out is float32 (partial gradients of shared heads)
  int out_map;             // whole chunks of out are stored by TMA
  int vec;                 // every row of the four arrays is aligned to four elements
  int da, dc;              // widths: a and b, c and out
  int H, n_seq;
  long long T;             // rows of a sequence (no cu), or of the whole buffer
  const int* cu;           // [n_seq + 1] row offsets, or NULL
  int reverse;             // against time
  float alpha, beta;
  // entering and leaving states of a sequence and head: element (i of da, j of dc) at
  // (seq * H + h) * da * dc + i * s_row + j * s_col
  const float* s_in;
  float* s_out;
  int s_row, s_col;
  // segments: a sequence is cut into nseg parts that run side by side; seg_state
  // [n_seq * H][nseg][da][dc]: slot p holds what part p - 1 leaves, then what
  // enters part p
  int nseg;
  float* seg_state;
};

struct LinDecay {
  float log2[kMaxLinHeads];
};

// The rows of sequence s.  Offsets come from the device: whatever they say,
// rows stay inside the buffer.
__device__ __forceinline__ void lin_rows(const LinPass& P, int s, long long& start, int& len) {
  if (P.cu) {
    long long lo = P.cu[s], hi = P.cu[s + 1];
    lo = lo < 0 ? 0 : lo > P.T ? P.T : lo;
    hi = hi < lo ? lo : hi > P.T ? P.T : hi;
    start = lo;
    len = (int)(hi - lo);
  } else {
    start = 0;
    len = (int)P.T;
  }
}

// Rows of each of nseg parts of len rows, in whole chunks of C.
__device__ __forceinline__ int lin_seg_len(int len, int nseg, int C) {
  const int per = (len + nseg - 1) / nseg;
  return (per + C - 1) / C * C;
}

// exp2(n * l), n >= 0: one for n = 0 whatever l
__device__ __forceinline__ float lin_pow(float l, int n) { return n <= 0 ? 1.0f : exp2f(l * (float)n); }

// four neighbours, at once where the arrays allow (vec)
template <typename T> __device__ __forceinline__ void lin_load4(const T* p, int vec, float (&v)[4]) {
  if (vec) {
    ld_vec<T, 4>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = to_f<T>(p[i]);
  }
}
template <typename T> __device__ __forceinline__ void lin_store4(T* p, int vec, const float (&v)[4]) {
  if (vec) {
    st_vec<T, 4>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = from_f<T>(v[i]);
  }
}

constexpr int kLinThreads = 256;
constexpr int kLinDC = 64;     // columns of c one CTA takes

template <int C, int DA>
struct LinFmaCfg {
  static constexpr int PA = DA + 4;        // row strides, a multiple of 4 floats
  static constexpr int PC = C + 4;
  static constexpr int PV = kLinDC + 4;
  static constexpr int OFF_AT = 0;                     // a^T [DA][PC]
  static constexpr int OFF_BT = OFF_AT + DA * PC;      // b^T [DA][PC]
  static constexpr int OFF_BW = OFF_BT + DA * PC;      // b, decayed to the chunk's end [C][PA]
  static constexpr int OFF_C = OFF_BW + C * PA;        // c [C][PV]
  static constexpr int OFF_PT = OFF_C + C * PV;        // masked, decayed products, transposed [C][PC]
  static constexpr int OFF_S = OFF_PT + C * PC;        // S [DA][PV]
  static constexpr int OFF_L = OFF_S + DA * PV;        // powers [C + 1]
  static constexpr int FLOATS = OFF_L + C + 4;
  static constexpr int SMEM_BYTES = FLOATS * 4;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

// One CTA: one (sequence, head, part, 64 columns of c), its chunks in turn; the
// four products of a chunk by 16 x 16 threads with 4 x 4 values each (2 x 4 where a
// chunk has 32 rows), both operands read as four neighbours at once.  Bound by the
// FP32 units and by shared memory, three wavefronts for sixteen FMA.  STATE_ONLY
// leaves out the outputs: what the part adds to the state, from zero.
template <typename T, int C, int DA, bool STATE_ONLY>
__global__ void __launch_bounds__(kLinThreads) lin_fma_kernel(const __grid_constant__ LinPass P,
                                                              const __grid_constant__ LinDecay G) {
  using K = LinFmaCfg<C, DA>;
  extern __shared__ __align__(16) float smem_lin[];
  float* sAT = smem_lin + K::OFF_AT;
  float* sBT = smem_lin + K::OFF_BT;
  float* sBW = smem_lin + K::OFF_BW;
  float* sC = smem_lin + K::OFF_C;
  float* sPT = smem_lin + K::OFF_PT;
  float* sS = smem_lin + K::OFF_S;
  float* sL = smem_lin + K::OFF_L;

  const int tid = threadIdx.x;
  const int tx = tid & 15, ty = tid >> 4;
  const int dc0 = blockIdx.x * kLinDC;
  const int seg = blockIdx.y;
  const int sh = blockIdx.z;
  const int h = sh % P.H, s = sh / P.H;
  const float l2 = G.log2[h];
  const int da = P.da, dc = P.dc;

  long long start;
  int len;
  lin_rows(P, s, start, len);
  const int seg_len = lin_seg_len(len, P.nseg, C);
  const long long lo64 = (long long)seg * seg_len;
  const int lo = (int)(lo64 < len ? lo64 : len);
  const int hi = (len - lo < seg_len) ? len : lo + seg_len;
  const bool owns_end = (hi == len) && (lo < len || seg == 0);   // the part that holds the last row
  if (STATE_ONLY && (lo >= hi || hi == len)) return;   // nothing reads what the last part leaves
  if (!STATE_ONLY && lo >= hi && !owns_end) return;

  const T* ap = (const T*)P.a.p + (P.cu ? 0 : s * P.a.bs) + (long long)(h / P.a.per) * P.a.hs;
  const T* bp = (const T*)P.b.p + (P.cu ? 0 : s * P.b.bs) + (long long)(h / P.b.per) * P.b.hs;
  const T* cp = (const T*)P.c.p + (P.cu ? 0 : s * P.c.bs) + (long long)(h / P.c.per) * P.c.hs;

  // what enters: the caller's state, or what the parts before left (STATE_ONLY: nothing)
  const long long mat = (long long)sh * da * dc;
  const bool from_user = !STATE_ONLY && seg == 0;
  for (int e = tid; e < DA * kLinDC; e += kLinThreads) {
    const int i = e / kLinDC, j = e % kLinDC;
    float v = 0.0f;
    if (!STATE_ONLY && i < da && dc0 + j < dc) {
      if (P.nseg > 1) v = P.seg_state[((long long)sh * P.nseg + seg) * da * dc + (long long)i * dc + dc0 + j];
      else if (P.s_in) v = P.s_in[mat + (long long)i * P.s_row + (long long)(dc0 + j) * P.s_col];
    }
    sS[i * K::PV + j] = v;
  }
  for (int n = tid; n <= C; n += kLinThreads) sL[n] = lin_pow(l2, n);
  __syncthreads();

  int e0 = (from_user && P.reverse) ? 1 : 0;   // the state that enters against time is not decayed by its first row
  for (int r0 = lo; r0 < hi; r0 += C) {
    const int n = hi - r0 < C ? hi - r0 : C;   // rows of this chunk
    auto row_of = [&](int i) { return start + (P.reverse ? len - 1 - (r0 + i) : r0 + i); };
    // a^T and b^T, b towards the chunk's end, and c: four columns of a row to a thread, eight rows and four such
    // neighbours to a warp (whole sectors of memory, and no more than two rows of a bank when written transposed)
    for (int e = tid; e < C * DA / 4; e += kLinThreads) {
      const int i = (e & 7) + 8 * (e / (2 * DA)), d = 4 * ((e >> 3) % (DA / 4));
      float av[4] = {}, bv[4] = {};
      if (i < n && d < da) {
        const long long r = row_of(i);
        if (!STATE_ONLY) lin_load4<T>(ap + r * P.a.ts + d, P.vec, av);
        lin_load4<T>(bp + r * P.b.ts + d, P.vec, bv);
      }
      const float f = i < n ? P.alpha * sL[n - 1 - i] : 0.0f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (!STATE_ONLY) {
          sAT[(d + x) * K::PC + i] = av[x];
          sBT[(d + x) * K::PC + i] = bv[x];
        }
        bv[x] *= f;
      }
      *reinterpret_cast<float4*>(sBW + i * K::PA + d) = make_float4(bv[0], bv[1], bv[2], bv[3]);
    }
    for (int e = tid; e < C * kLinDC / 4; e += kLinThreads) {
      const int i = e / (kLinDC / 4), j = 4 * (e % (kLinDC / 4));
      float v[4] = {};
      if (i < n && dc0 + j < dc) lin_load4<T>(cp + row_of(i) * P.c.ts + dc0 + j, P.vec, v);
      *reinterpret_cast<float4*>(sC + i * K::PV + j) = make_float4(v[0], v[1], v[2], v[3]);
    }
    __syncthreads();

    constexpr int RM = C / 16;   // rows of a thread's values (4 or 2)
    auto rows4 = [](const float* p, float (&x)[RM]) {
      if constexpr (RM == 4) {
        const float4 f = *reinterpret_cast<const float4*>(p);
        x[0] = f.x;
        x[1] = f.y;
        x[2] = f.z;
        x[3] = f.w;
      } else {
        const float2 f = *reinterpret_cast<const float2*>(p);
        x[0] = f.x;
        x[1] = f.y;
      }
    };
    if (!STATE_ONLY) {
      // products of rows i = ty RM .. and j = tx RM ..
      float acc[RM][RM] = {};
#pragma unroll 4
      for (int d = 0; d < da; ++d) {
        float x[RM], y[RM];
        rows4(sAT + d * K::PC + ty * RM, x);
        rows4(sBT + d * K::PC + tx * RM, y);
#pragma unroll
        for (int u = 0; u < RM; ++u)
#pragma unroll
          for (int w = 0; w < RM; ++w) acc[u][w] = fmaf(x[u], y[w], acc[u][w]);
      }
#pragma unroll
      for (int w = 0; w < RM; ++w) {
        const int j = tx * RM + w;
        float p[RM];
#pragma unroll
        for (int u = 0; u < RM; ++u) {
          const int i = ty * RM + u;
          p[u] = (j <= i && i < n) ? acc[u][w] * (P.alpha * sL[i - j]) : 0.0f;
        }
        if constexpr (RM == 4) *reinterpret_cast<float4*>(sPT + j * K::PC + ty * RM) = make_float4(p[0], p[1], p[2], p[3]);
        else *reinterpret_cast<float2*>(sPT + j * K::PC + ty * RM) = make_float2(p[0], p[1]);
      }
      __syncthreads();
      float o[RM][4] = {};
      auto product = [&](const float* xs, const float* ys, int k) {   // x [k][rows] times y [k][columns]
#pragma unroll 4
        for (int d = 0; d < k; ++d) {
          float x[RM];
          rows4(xs + d * K::PC + ty * RM, x);
          const float4 y = *reinterpret_cast<const float4*>(ys + d * K::PV + tx * 4);
#pragma unroll
          for (int u = 0; u < RM; ++u) {
            o[u][0] = fmaf(x[u], y.x, o[u][0]);
            o[u][1] = fmaf(x[u], y.y, o[u][1]);
            o[u][2] = fmaf(x[u], y.z, o[u][2]);
            o[u][3] = fmaf(x[u], y.w, o[u][3]);
          }
        }
      };
      product(sAT, sS, da);
#pragma unroll
      for (int u = 0; u < RM; ++u) {
        const float f = sL[max(ty * RM + u + 1 - e0, 0)];
#pragma unroll
        for (int w = 0; w < 4; ++w) o[u][w] *= f;
      }
      // (a warp's last row is (ty | 1) RM + RM - 1: no row of it takes a later one)
      product(sPT, sC, min(n, (ty | 1) * RM + RM));
#pragma unroll
      for (int u = 0; u < RM; ++u) {
        const int i = ty * RM + u;
        if (i < n) {
          const long long at = (P.cu ? 0 : s * P.out_bs) + row_of(i) * P.out_ts + (long long)h * P.out_hs + dc0 + tx * 4;
          float v[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) v[w] = P.beta * o[u][w];
          if (dc0 + tx * 4 < dc) {
            if (P.out_f32) lin_store4<float>((float*)P.out + at, P.vec, v);
            else lin_store4<T>((T*)P.out + at, P.vec, v);
          }
        }
      }
      __syncthreads();   // S is read; it changes below
    }
    // S: thread (ty, tx) takes rows 4 ty .. of every 64, and columns tx * 4 ..
    const float f = sL[n - e0];
    for (int d = 4 * ty; d < da; d += 64) {
      float4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        v[u] = *reinterpret_cast<const float4*>(sS + (d + u) * K::PV + tx * 4);
        v[u].x *= f;
        v[u].y *= f;
        v[u].z *= f;
        v[u].w *= f;
      }
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const float4 x4 = *reinterpret_cast<const float4*>(sBW + j * K::PA + d);
        const float4 y = *reinterpret_cast<const float4*>(sC + j * K::PV + tx * 4);
        const float x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          v[u].x = fmaf(x[u], y.x, v[u].x);
          v[u].y = fmaf(x[u], y.y, v[u].y);
          v[u].z = fmaf(x[u], y.z, v[u].z);
          v[u].w = fmaf(x[u], y.w, v[u].w);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) *reinterpret_cast<float4*>(sS + (d + u) * K::PV + tx * 4) = v[u];
    }
    __syncthreads();
    e0 = 0;
  }

  if (STATE_ONLY) {
    float* dst = P.seg_state + ((long long)sh * P.nseg + seg + 1) * da * dc;
    for (int e = tid; e < da * kLinDC; e += kLinThreads) {
      const int i = e / kLinDC, j = e % kLinDC;
      if (dc0 + j < dc) dst[(long long)i * dc + dc0 + j] = sS[i * K::PV + j];
    }
  } else if (P.s_out && owns_end) {
    // against time the first state's gradient still decays by the first row
    const float f = (P.reverse && len > 0) ? sL[1] : 1.0f;
    for (int e = tid; e < da * kLinDC; e += kLinThreads) {
      const int i = e / kLinDC, j = e % kLinDC;
      if (dc0 + j < dc) P.s_out[mat + (long long)i * P.s_row + (long long)(dc0 + j) * P.s_col] = f * sS[i * K::PV + j];
    }
  }
}

// What each part left becomes what enters the next: slot p holds what part
// p - 1 left and receives E_p = e^{g rows_(p-1)} E_(p-1) + left_(p-1), E_0 the
// caller's state, in order of the parts.  `chunked`: parts are whole chunks of C in
// the order of the rows even against time, so that the first part then has the short
// chunk; else they are rows in the order they are taken.
__global__ void __launch_bounds__(256) lin_combine_kernel(const __grid_constant__ LinPass P,
                                                          const __grid_constant__ LinDecay G, int C, int chunked) {
  const int sh = blockIdx.y;
  const int h = sh % P.H, s = sh / P.H;
  const int e = blockIdx.x * 256 + threadIdx.x;
  const int size = P.da * P.dc;
  if (e >= size) return;
  long long start;
  int len;
  lin_rows(P, s, start, len);
  const int nch = (len + C - 1) / C;
  const int seg_len = chunked ? (nch + P.nseg - 1) / P.nseg * C : lin_seg_len(len, P.nseg, C);
  const int first = seg_len - (chunked && P.reverse ? nch * C - len : 0);   // rows of part 0, where others follow it
  const int i = e / P.dc, j = e % P.dc;
  float v = P.s_in ? P.s_in[(long long)sh * size + (long long)i * P.s_row + (long long)j * P.s_col] : 0.0f;
  float* at = P.seg_state + (long long)sh * P.nseg * size + e;
  at[0] = v;   // the parts read it here: the last one may overwrite the caller's state meanwhile
  const float f = lin_pow(G.log2[h], seg_len);
  float f_in = lin_pow(G.log2[h], first - (P.reverse ? 1 : 0));
  for (int p = 1; p < P.nseg && (long long)p * seg_len < (chunked ? (long long)nch * C : (long long)len); ++p) {
    v = fmaf(f_in, v, at[(long long)p * size]);
    at[(long long)p * size] = v;
    f_in = f;
  }
}

// dst = sum of the partial gradients [rows][H][d] of each group of heads, in the
// order of the heads; rows of no sequence are left as they are.
template <typename T>
__global__ void __launch_bounds__(256) lin_group_sum_kernel(const float* __restrict__ part, long long rows, int H, int G,
                                                            int d, T* dst, long long bs, long long ts, long long hs,
                                                            long long tokens, const int* cu, int n_seq) {
  const int K = H / G;
  const long long n = rows * K * d;
  long long lo = 0, hi = rows;
  if (cu) {
    lo = cu[0];
    hi = cu[n_seq];
  }
  for (long long e = (long long)blockIdx.x * 256 + threadIdx.x; e < n; e += (long long)gridDim.x * 256) {
    const int j = (int)(e % d);
    const long long rk = e / d;
    const int k = (int)(rk % K);
    const long long r = rk / K;
    if (r < lo || r >= hi) continue;
    const float* p = part + (r * H + (long long)k * G) * d + j;
    float v = 0.0f;
    for (int g = 0; g < G; ++g) v += p[(long long)g * d];
    const long long b = r / tokens, t = r - b * tokens;
    dst[b * bs + t * ts + k * hs + j] = from_f<T>(v);
  }
}

struct LinStep {
  LinOperand q, k, v;      // ts unused: one row per batch entry
  void* o;
  long long o_bs, o_hs;
  int H, dk, dv;
  float scale;
  float* states;           // [n_slots][H][dk][dv]
  long long n_slots;
  const long long* slots;  // [rows], or NULL: row b at slot b
  const long long* positions;
  const void* wq;
  const void* wk;
  int w_f32;
  float eps;
  int pairs, interleaved;  // rotation (pairs = 0: none)
  float m;
  unsigned long long turn[kMaxRotPairs];
};

constexpr int kStepThreads = 256;

// One token of a sequence and head: S <- e^g S + k v^T, o = scale q S.  Bound by
// the state's one read and one write.  A CTA takes CX * 4 columns of one state;
// a thread four columns of every RG-th row, so that a warp reads whole lines.
// Norm and rotation of q and k, where asked for, are done by two warps while
// the state's first rows are on their way.
template <typename T, int CX>
__global__ void __launch_bounds__(kStepThreads) lin_step_kernel(const __grid_constant__ LinStep P,
                                                                const __grid_constant__ LinDecay G) {
  constexpr int RG = kStepThreads / CX;   // row groups
  constexpr int U = CX == 32 ? 8 : 4;     // rows in flight per thread
  __shared__ float s_q[256], s_k[256];
  __shared__ float s_red[8][CX * 4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.z, h = blockIdx.y;
  const int cx = tid % CX, rg = tid / CX;
  const int col = (blockIdx.x * CX + cx) * 4;
  const bool on = col < P.dv;
  const long long slot = P.slots ? P.slots[b] : b;
  if (slot < 0 || slot >= P.n_slots) return;   // padding: the whole CTA leaves
  float* S = P.states + (slot * P.H + h) * (long long)P.dk * P.dv + col;

  float4 s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = rg + u * RG;
    s[u] = (on && r < P.dk) ? *reinterpret_cast<const float4*>(S + (long long)r * P.dv) : make_float4(0, 0, 0, 0);
  }
  // of rows that name one slot the first is computed, the others are padding
  int twice = 0;
  if (P.slots)
    for (int i = tid; i < b; i += kStepThreads) twice |= (P.slots[i] == slot);
  if (warp < 2) {
    const T* x = warp ? (const T*)P.k.p + b * P.k.bs + (h / P.k.per) * P.k.hs : (const T*)P.q.p + b * P.q.bs + (long long)h * P.q.hs;
    float* dst = warp ? s_k : s_q;
    float v[8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = lane + 32 * i;
      v[i] = d < P.dk ? to_f<T>(x[d]) : 0.0f;
      ss = fmaf(v[i], v[i], ss);
    }
    const void* w = warp ? P.wk : P.wq;
    if (w) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = rsqrtf(ss / (float)P.dk + P.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int d = lane + 32 * i;
        if (d < P.dk) v[i] *= r * (P.w_f32 ? ((const float*)w)[d] : to_f<T>(((const T*)w)[d]));
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) dst[lane + 32 * i] = v[i];
    __syncwarp();
    if (P.pairs) {
      const long long pos = P.positions[b];
      for (int p = lane; p < P.pairs; p += 32) {
        float c, sn;
        turn_cos_sin<false>(P.turn[p], pos, P.m, c, sn);
        const int i0 = P.interleaved ? 2 * p : p, i1 = P.interleaved ? 2 * p + 1 : p + P.pairs;
        const float x0 = dst[i0], x1 = dst[i1];
        dst[i0] = x0 * c - x1 * sn;
        dst[i1] = x1 * c + x0 * sn;
      }
    }
  }
  const float decay = exp2f(G.log2[h]);
  float4 v = make_float4(0, 0, 0, 0), acc = make_float4(0, 0, 0, 0);
  if (on) {
    float t[4];
    const T* vp = (const T*)P.v.p + b * P.v.bs + (h / P.v.per) * P.v.hs + col;
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = to_f<T>(vp[i]);
    v = make_float4(t[0], t[1], t[2], t[3]);
  }
  if (__syncthreads_or(twice)) return;
  for (int r0 = rg; r0 < P.dk; r0 += U * RG) {
    if (r0 != rg) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * RG;
        if (on && r < P.dk) s[u] = *reinterpret_cast<const float4*>(S + (long long)r * P.dv);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RG;
      if (on && r < P.dk) {
        const float kk = s_k[r], qq = s_q[r];
        s[u].x = fmaf(decay, s[u].x, kk * v.x);
        s[u].y = fmaf(decay, s[u].y, kk * v.y);
        s[u].z = fmaf(decay, s[u].z, kk * v.z);
        s[u].w = fmaf(decay, s[u].w, kk * v.w);
        *reinterpret_cast<float4*>(S + (long long)r * P.dv) = s[u];
        acc.x = fmaf(qq, s[u].x, acc.x);
        acc.y = fmaf(qq, s[u].y, acc.y);
        acc.z = fmaf(qq, s[u].z, acc.z);
        acc.w = fmaf(qq, s[u].w, acc.w);
      }
    }
  }
  // rows of one warp, then of the eight warps
#pragma unroll
  for (int o = CX; o < 32; o <<= 1) {
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
  }
  if (lane < CX) *reinterpret_cast<float4*>(&s_red[warp][cx * 4]) = acc;
  __syncthreads();
  if (tid < CX * 4) {
    const int j = blockIdx.x * CX * 4 + tid;
    float o = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) o += s_red[w][tid];
    if (j < P.dv) ((T*)P.o)[b * P.o_bs + (long long)h * P.o_hs + j] = from_f<T>(P.scale * o);
  }
}

}  // namespace pn
