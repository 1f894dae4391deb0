// pn_linattn.cuh -- linear attention with a decay for each head: the parameter
// block of one pass over the rows, and the kernels for any type and width.
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
  unsigned wait_ns;    // limit of each device wait
  int stall;           // test hook: from this chunk of each part on none is loaded (-1: all are)
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
  unsigned wait_ns;        // limit of a device wait
  int stall;               // test hook: from this chunk of each part on none is loaded (-1: all are)
  int by_length;           // sequences are taken longest first
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

// The rows lo .. hi - 1 of sequence s of a buffer of T rows.  Offsets come from the device: whatever they say,
// rows stay inside the buffer.
__device__ __forceinline__ void lin_span(const int* cu, long long T, int s, long long& lo, long long& hi) {
  lo = cu[s];
  hi = cu[s + 1];
  lo = lo < 0 ? 0 : lo > T ? T : lo;
  hi = hi < lo ? lo : hi > T ? T : hi;
}
__device__ __forceinline__ void lin_rows(const LinPass& P, int s, long long& start, int& len) {
  if (P.cu) {
    long long hi;
    lin_span(P.cu, P.T, s, start, hi);
    len = (int)(hi - start);
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

constexpr int kLinDC = 64;     // columns of c one CTA takes

template <typename T, int C, int DA>
struct LinMmaCfg {
  // Row strides in floats.  Fragments read rows (lane >> 2) and columns (lane & 3) of an A operand, and the other way round
  // of a B operand: strides of 12 and 8 banks keep both free of conflicts.
  static constexpr int PA = DA + 12;
  static constexpr int PV = kLinDC + 8;
  static constexpr int PP = C + 4;
  static constexpr int OFF_A = 0;                      // a [C][PA]
  static constexpr int OFF_B = OFF_A + C * PA;         // b [C][PA]
  static constexpr int OFF_C = OFF_B + C * PA;         // c [C][PV]
  static constexpr int OFF_W = OFF_C + C * PV;         // c, decayed to the chunk's end [C][PV]
  static constexpr int OFF_P = OFF_W + C * PV;         // masked, decayed products [C][PP]
  static constexpr int OFF_S = OFF_P + C * PP;         // S [DA][PV]
  static constexpr int OFF_L = OFF_S + DA * PV;        // powers [C + 1]
  static constexpr int SMEM_BYTES = (OFF_L + C + 4) * 4;
  static constexpr int CTAS = SMEM_BYTES <= 112 * 1024 ? 2 : 1;   // on an SM
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
  // Sixteen warps where one CTA has the SM and operands need no splitting (4 x 16 heads x 4096 float16 rows of width 128
  // 844 -> 742 us; float32, with more to do for each fragment that a warp reads, would lose, 906 -> 944).
  // warps: RT x CG over P's and the outputs' rows (16 each) and columns; MW x SG over S's
  static constexpr int NT = CTAS == 1 && sizeof(T) == 2 ? 512 : 256, NW = NT / 32;
  static constexpr int RT = C / 16, CG = NW / RT;
  static constexpr int NP = C / 8 > CG ? C / 8 / CG : 1, NO = kLinDC / 8 / CG;
  static_assert(C * DA / 4 % (4 * NT) == 0, "whole groups of loads");
  static constexpr int MT = DA / 16, MW = MT < 8 ? MT : 8, SG = NW / MW, MS = MT / MW, NS = kLinDC / 8 / SG;
};

// D += A B, 16 x 8 x 8 in TF32.  Lane (g, t) = (lane >> 2, lane & 3) holds rows g, g + 8 and columns t, t + 4 of A, rows
// t, t + 4 and column g of B, rows g, g + 8 and columns 2t, 2t + 1 of D.
__device__ __forceinline__ void lin_mma(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// An operand's fragment as the TF32 value nearest to it and, where TF32 does not hold it (SPLIT), what is left.
template <int N, bool SPLIT>
struct LinFrag {
  uint32_t hi[N], lo[SPLIT ? N : 1];
  __device__ __forceinline__ void set(int i, float x) {
    if constexpr (SPLIT) {
      uint32_t r;
      asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
      hi[i] = r;
      lo[i] = __float_as_uint(x - __uint_as_float(r));
    } else {
      hi[i] = __float_as_uint(x);
    }
  }
};
// D = A B, the same with nothing to add to
__device__ __forceinline__ void lin_mma0(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.0f));
}
// Their products: lo hi + hi lo + hi hi (22 bits of each factor), a pass over all N tiles at a time, so that a tile's sum is
// not waited for by its next term.  The tensor cores truncate what they add: eight terms are summed there, the small ones
// first, and the eights in float32 (float32 outputs of 1500 rows, width 64, are 2.0e-7 off in the mean square so, and were
// 1.1e-6 off with the accumulators left there; 2 to 5 % of the time).
template <int N, bool SA, bool SB>
__device__ __forceinline__ void lin_mma_split(float (&d)[N][4], const LinFrag<4, SA>& a, const LinFrag<2, SB> (&b)[N], int n) {
  float u[N][4];
  if constexpr (SA) {
#pragma unroll
    for (int y = 0; y < N; ++y)
      if (y < n) lin_mma0(u[y], a.lo, b[y].hi);
  }
  if constexpr (SB) {
#pragma unroll
    for (int y = 0; y < N; ++y)
      if (y < n) {
        if constexpr (SA) lin_mma(u[y], a.hi, b[y].lo);
        else lin_mma0(u[y], a.hi, b[y].lo);
      }
  }
#pragma unroll
  for (int y = 0; y < N; ++y)
    if (y < n) {
      if constexpr (SA || SB) lin_mma(u[y], a.hi, b[y].hi);
      else lin_mma0(u[y], a.hi, b[y].hi);
    }
#pragma unroll
  for (int y = 0; y < N; ++y)
    if (y < n)
#pragma unroll
      for (int e = 0; e < 4; ++e) d[y][e] += u[y][e];
}

// One CTA: one (sequence, head, part, 64 columns of c), its chunks in turn; the
// four products of a chunk by all warps on the TF32 tensor cores (mma.sync), in
// split form: 16-bit operands are TF32 values as they are, everything else takes two.
// S is summed in float32 registers (the tensor cores truncate) and copied to
// shared memory for the outputs.  What it is for is float32, which the tcgen05 kernel
// does not take: 4 x 16 heads x 4096 rows of width 64 took 616 us by FP32 FMA with
// 4 x 4 values a thread, which shared memory bounds, and take 328 to 338 us so.
// STATE_ONLY leaves out the outputs: what the part adds to the state, from zero.
template <typename T, int C, int DA, bool STATE_ONLY>
__global__ void __launch_bounds__(LinMmaCfg<T, C, DA>::NT, LinMmaCfg<T, C, DA>::CTAS) lin_mma_kernel(const __grid_constant__ LinPass P,
                                                                                     const __grid_constant__ LinDecay G) {
  using K = LinMmaCfg<T, C, DA>;
  constexpr bool X = sizeof(T) == 4;   // inputs are split
  extern __shared__ __align__(16) float smem_lin[];
  float* sA = smem_lin + K::OFF_A;
  float* sB = smem_lin + K::OFF_B;
  float* sC = smem_lin + K::OFF_C;
  float* sW = smem_lin + K::OFF_W;
  float* sP = smem_lin + K::OFF_P;
  float* sS = smem_lin + K::OFF_S;
  float* sL = smem_lin + K::OFF_L;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
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

  // this warp's part of S: rows 16 (sm + 8 x) + g (+ 8), columns 8 (sn0 + y) + 2 t (+ 1)
  const int sm = warp % K::MW, sn0 = warp / K::MW * K::NS;
  auto s_row = [&](int x, int e) { return 16 * (sm + 8 * x) + g + (e & 2) * 4; };
  auto s_col = [&](int y, int e) { return 8 * (sn0 + y) + 2 * t + (e & 1); };
  float S[K::MS][K::NS][4];
  // what enters: the caller's state, or what the parts before left (STATE_ONLY: nothing)
  const long long mat = (long long)sh * da * dc;
  const bool from_user = !STATE_ONLY && seg == 0;
#pragma unroll
  for (int x = 0; x < K::MS; ++x)
#pragma unroll
    for (int y = 0; y < K::NS; ++y)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = s_row(x, e), j = dc0 + s_col(y, e);
        float v = 0.0f;
        if (!STATE_ONLY && i < da && j < dc) {
          if (P.nseg > 1) v = P.seg_state[((long long)sh * P.nseg + seg) * da * dc + (long long)i * dc + j];
          else if (P.s_in) v = P.s_in[mat + (long long)i * P.s_row + (long long)j * P.s_col];
        }
        S[x][y][e] = v;
      }
  auto publish = [&]() {   // S to shared memory
#pragma unroll
    for (int x = 0; x < K::MS; ++x)
#pragma unroll
      for (int y = 0; y < K::NS; ++y) {
        *reinterpret_cast<float2*>(sS + s_row(x, 0) * K::PV + s_col(y, 0)) = make_float2(S[x][y][0], S[x][y][1]);
        *reinterpret_cast<float2*>(sS + s_row(x, 2) * K::PV + s_col(y, 0)) = make_float2(S[x][y][2], S[x][y][3]);
      }
  };
  if (!STATE_ONLY) publish();
  for (int n = tid; n <= C; n += K::NT) sL[n] = lin_pow(l2, n);
  __syncthreads();

  const int wr = warp % K::RT, wc = warp / K::RT;
  int e0 = (from_user && P.reverse) ? 1 : 0;   // the state that enters against time is not decayed by its first row
  for (int r0 = lo; r0 < hi; r0 += C) {
    const int n = hi - r0 < C ? hi - r0 : C;   // rows of this chunk
    auto row_of = [&](int i) { return start + (P.reverse ? len - 1 - (r0 + i) : r0 + i); };
    // several loads in flight before their values are needed: a thread's 4 x 4 values of a and b at a time, then c's
    constexpr int kC = C * kLinDC / 4 / K::NT;
    float cv[kC][4];
#pragma unroll
    for (int x = 0; x < kC; ++x) {
      const int e = tid + x * K::NT, i = e / (kLinDC / 4), j = 4 * (e % (kLinDC / 4));
#pragma unroll
      for (int y = 0; y < 4; ++y) cv[x][y] = 0.0f;
      if (i < n && dc0 + j < dc) lin_load4<T>(cp + row_of(i) * P.c.ts + dc0 + j, P.vec, cv[x]);
    }
#pragma unroll 1
    for (int first = tid; first < C * DA / 4; first += 4 * K::NT) {
      float av[4][4], bv[4][4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int e = first + x * K::NT, i = e / (DA / 4), d = 4 * (e % (DA / 4));
#pragma unroll
        for (int y = 0; y < 4; ++y) av[x][y] = bv[x][y] = 0.0f;
        if (i < n && d < da) {
          const long long r = row_of(i);
          if (!STATE_ONLY) lin_load4<T>(ap + r * P.a.ts + d, P.vec, av[x]);
          lin_load4<T>(bp + r * P.b.ts + d, P.vec, bv[x]);
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int e = first + x * K::NT, i = e / (DA / 4), d = 4 * (e % (DA / 4));
        if (!STATE_ONLY) *reinterpret_cast<float4*>(sA + i * K::PA + d) = make_float4(av[x][0], av[x][1], av[x][2], av[x][3]);
        *reinterpret_cast<float4*>(sB + i * K::PA + d) = make_float4(bv[x][0], bv[x][1], bv[x][2], bv[x][3]);
      }
    }
#pragma unroll
    for (int x = 0; x < kC; ++x) {
      const int e = tid + x * K::NT, i = e / (kLinDC / 4), j = 4 * (e % (kLinDC / 4));
      const float (&v)[4] = cv[x];
      if (!STATE_ONLY) *reinterpret_cast<float4*>(sC + i * K::PV + j) = make_float4(v[0], v[1], v[2], v[3]);
      const float f = i < n ? P.alpha * sL[n - 1 - i] : 0.0f;
      *reinterpret_cast<float4*>(sW + i * K::PV + j) = make_float4(f * v[0], f * v[1], f * v[2], f * v[3]);
    }
    // The next chunk's rows on their way to L2 meanwhile, a line of 128 bytes to a thread: one CTA an SM, as at widths above
    // 64, has little else in flight (4 x 16 heads x 4096 float16 rows of width 128 960 -> 829 us; float32 892 -> 877, of
    // width 64 326 -> 320; only a few long heads of width 256 lose, 156 -> 160).
    if (r0 + C < hi) {
      const int m = min(C, hi - r0 - C);
      constexpr int kA = (DA * (int)sizeof(T) + 127) / 128, kV = kLinDC * (int)sizeof(T) / 128;
      for (int e = tid; e < m * (2 * kA + kV); e += K::NT) {
        const int i = C + e % m, l = e / m;   // row from r0 on, line: a's, b's, c's
        const int at = 128 / (int)sizeof(T) * (l < kA ? l : l < 2 * kA ? l - kA : l - 2 * kA);
        const long long r = row_of(i);
        const T* p = l < kA ? ap + r * P.a.ts : l < 2 * kA ? bp + r * P.b.ts : cp + r * P.c.ts + dc0;
        if (at < (l < 2 * kA ? da : dc - dc0) && !(STATE_ONLY && l < kA)) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + at));
      }
    }
    __syncthreads();

    if (!STATE_ONLY) {
      // products of rows 16 wr .. with rows 8 (wc NP + y) .., up to the diagonal
      float acc[K::NP][4] = {};
      const int tiles = min(K::NP, 2 * wr + 2 - wc * K::NP);   // column tiles that this row tile takes
#pragma unroll 2
      for (int k = 0; k < (tiles > 0 ? da : 0); k += 8) {
        LinFrag<4, X> a;
        const float* pa = sA + (16 * wr + g) * K::PA + k + t;
        a.set(0, pa[0]);
        a.set(1, pa[8 * K::PA]);
        a.set(2, pa[4]);
        a.set(3, pa[8 * K::PA + 4]);
        LinFrag<2, X> b[K::NP];
#pragma unroll
        for (int y = 0; y < K::NP; ++y) {
          const float* pb = sB + (8 * (wc * K::NP + y) + g) * K::PA + k + t;
          b[y].set(0, pb[0]);
          b[y].set(1, pb[4]);
        }
        lin_mma_split<K::NP, X, X>(acc, a, b, tiles);
      }
#pragma unroll
      for (int y = 0; y < K::NP; ++y) {
        if (y >= tiles) break;
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const int i = 16 * wr + g + e * 4, j = 8 * (wc * K::NP + y) + 2 * t;
          float p[2];
#pragma unroll
          for (int u = 0; u < 2; ++u)
            p[u] = (j + u <= i && i < n) ? acc[y][e + u] * (P.alpha * sL[i - j - u]) : 0.0f;
          *reinterpret_cast<float2*>(sP + i * K::PP + j) = make_float2(p[0], p[1]);
        }
      }
      __syncthreads();
      // outputs of rows 16 wr .., columns 8 (wc NO + y) ..: the state's share, then the chunk's
      float o[K::NO][4] = {};
      auto product = [&](const float* x, int px, const float* z, int k1, auto split_x, auto split_z) {
        constexpr bool SX = decltype(split_x)::value, SZ = decltype(split_z)::value;
#pragma unroll 2
        for (int k = 0; k < k1; k += 8) {
          LinFrag<4, SX> a;
          const float* pa = x + (16 * wr + g) * px + k + t;
          a.set(0, pa[0]);
          a.set(1, pa[8 * px]);
          a.set(2, pa[4]);
          a.set(3, pa[8 * px + 4]);
          LinFrag<2, SZ> b[K::NO];
#pragma unroll
          for (int y = 0; y < K::NO; ++y) {
            const float* pb = z + (k + t) * K::PV + 8 * (wc * K::NO + y) + g;
            b[y].set(0, pb[0]);
            b[y].set(1, pb[4 * K::PV]);
          }
          lin_mma_split<K::NO, SX, SZ>(o, a, b, K::NO);
        }
      };
      using Yes = std::integral_constant<bool, true>;
      using In = std::integral_constant<bool, X>;
      product(sA, K::PA, sS, da, In{}, Yes{});
      const float f0 = sL[max(16 * wr + g + 1 - e0, 0)], f1 = sL[max(16 * wr + g + 9 - e0, 0)];
#pragma unroll
      for (int y = 0; y < K::NO; ++y) {
        o[y][0] *= f0;
        o[y][1] *= f0;
        o[y][2] *= f1;
        o[y][3] *= f1;
      }
      product(sP, K::PP, sC, min(n, 16 * wr + 16), Yes{}, In{});
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int i = 16 * wr + g + e * 4;
        if (i >= n) continue;
        const long long at = (P.cu ? 0 : s * P.out_bs) + row_of(i) * P.out_ts + (long long)h * P.out_hs + dc0;
#pragma unroll
        for (int y = 0; y < K::NO; ++y) {
          const int j = 8 * (wc * K::NO + y) + 2 * t;
          if (dc0 + j >= dc) continue;
          const float v[2] = {P.beta * o[y][e], P.beta * o[y][e + 1]};
          if (P.out_f32) {
            float* p = (float*)P.out + at + j;
            if (P.vec) st_vec<float, 2>(p, v);
            else p[0] = v[0], p[1] = v[1];
          } else {
            T* p = (T*)P.out + at + j;
            if (P.vec) st_vec<T, 2>(p, v);
            else p[0] = from_f<T>(v[0]), p[1] = from_f<T>(v[1]);
          }
        }
      }
    }
    // S = e^{g n} S + b^T c'
    const float f = sL[n - e0];
#pragma unroll
    for (int x = 0; x < K::MS; ++x) {
      float u[K::NS][4] = {};
#pragma unroll 2
      for (int k = 0; k < n; k += 8) {
        LinFrag<4, X> a;
        const float* pa = sB + (k + t) * K::PA + 16 * (sm + 8 * x) + g;
        a.set(0, pa[0]);
        a.set(1, pa[8]);
        a.set(2, pa[4 * K::PA]);
        a.set(3, pa[4 * K::PA + 8]);
        LinFrag<2, true> b[K::NS];
#pragma unroll
        for (int y = 0; y < K::NS; ++y) {
          const float* pb = sW + (k + t) * K::PV + 8 * (sn0 + y) + g;
          b[y].set(0, pb[0]);
          b[y].set(1, pb[4 * K::PV]);
        }
        lin_mma_split<K::NS, X, true>(u, a, b, K::NS);
      }
#pragma unroll
      for (int y = 0; y < K::NS; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[x][y][e] = fmaf(f, S[x][y][e], u[y][e]);
    }
    __syncthreads();   // everything of this chunk is read
    if (!STATE_ONLY) publish();
    e0 = 0;
  }

  float* dst = nullptr;
  long long di = 0, dj = 0;
  float f = 1.0f;
  if (STATE_ONLY) {
    dst = P.seg_state + ((long long)sh * P.nseg + seg + 1) * da * dc;
    di = dc;
    dj = 1;
  } else if (P.s_out && owns_end) {
    dst = P.s_out + mat;
    di = P.s_row;
    dj = P.s_col;
    if (P.reverse && len > 0) f = sL[1];   // against time the first state's gradient still decays by the first row
  }
  if (dst) {
#pragma unroll
    for (int x = 0; x < K::MS; ++x)
#pragma unroll
      for (int y = 0; y < K::NS; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = s_row(x, e), j = dc0 + s_col(y, e);
          if (i < da && j < dc) dst[(long long)i * di + (long long)j * dj] = f * S[x][y][e];
        }
  }
}

// What each part left becomes what enters the next: slot p holds what part
// p - 1 left and receives E_p = e^{g rows_(p-1)} E_(p-1) + left_(p-1), E_0 the
// caller's state, in order of the parts.  `chunked`: parts are whole chunks of C in
// the order of the rows even against time, so that the first part then has the short
// chunk; else they are rows in the order they are taken.
__global__ void __launch_bounds__(128) lin_combine_kernel(const __grid_constant__ LinPass P,
                                                          const __grid_constant__ LinDecay G, int C, int chunked) {
  constexpr int kFlight = 8;   // parts read at once
  const int sh = blockIdx.y;
  const int h = sh % P.H, s = sh / P.H;
  const int e = 4 * (blockIdx.x * 128 + threadIdx.x);   // four neighbours of a state (widths are multiples of 8)
  const int size = P.da * P.dc;
  if (e >= size) return;
  long long start;
  int len;
  lin_rows(P, s, start, len);
  const int nch = (len + C - 1) / C;
  const int seg_len = chunked ? (nch + P.nseg - 1) / P.nseg * C : lin_seg_len(len, P.nseg, C);
  const int first = seg_len - (chunked && P.reverse ? nch * C - len : 0);   // rows of part 0, where others follow it
  const int rows = chunked ? nch * C : len;
  const int parts = seg_len > 0 ? min(P.nseg, (rows + seg_len - 1) / seg_len) : 1;   // with rows
  const int i = e / P.dc, j = e % P.dc;
  float v[4] = {};
  if (P.s_in) {
    const float* in = P.s_in + (long long)sh * size + (long long)i * P.s_row + (long long)j * P.s_col;
#pragma unroll
    for (int x = 0; x < 4; ++x) v[x] = in[(long long)x * P.s_col];
  }
  float4* at = reinterpret_cast<float4*>(P.seg_state + (long long)sh * P.nseg * size + e);
  const long long step = size / 4;
  at[0] = make_float4(v[0], v[1], v[2], v[3]);   // the parts read it here: the last one may overwrite the caller's state meanwhile
  const float f = lin_pow(G.log2[h], seg_len);
  float f_in = lin_pow(G.log2[h], first - (P.reverse ? 1 : 0));
  for (int p0 = 1; p0 < parts; p0 += kFlight) {
    float4 left[kFlight];
#pragma unroll
    for (int p = 0; p < kFlight; ++p)
      if (p0 + p < parts) left[p] = at[(p0 + p) * step];
#pragma unroll
    for (int p = 0; p < kFlight; ++p) {
      if (p0 + p >= parts) break;
      v[0] = fmaf(f_in, v[0], left[p].x);
      v[1] = fmaf(f_in, v[1], left[p].y);
      v[2] = fmaf(f_in, v[2], left[p].z);
      v[3] = fmaf(f_in, v[3], left[p].w);
      at[(p0 + p) * step] = make_float4(v[0], v[1], v[2], v[3]);
      f_in = f;
    }
  }
}

// dst = sum of the partial gradients [rows][H][d] of each group of heads, in the
// order of the heads, four neighbours to a thread; rows of no sequence are left as
// they are: with offsets, a CTA takes rows of the sequence blockIdx.y, as the passes
// that wrote them did.  A block takes whole rows of K heads.
template <typename T>
__global__ void __launch_bounds__(256) lin_group_sum_kernel(const float* __restrict__ part, long long rows, int H, int G,
                                                            int d, T* dst, long long bs, long long ts, long long hs,
                                                            long long tokens, const int* cu, int vec) {
  const int K = H / G, quads = K * d / 4;
  long long lo = 0, hi = rows;
  if (cu) lin_span(cu, rows, blockIdx.y, lo, hi);
  for (long long r = lo + blockIdx.x; r < hi; r += gridDim.x) {
    const long long b = r / tokens, t = r - b * tokens;
    T* out = dst + b * bs + t * ts;
    for (int e = threadIdx.x; e < quads; e += 256) {
      const int k = 4 * e / d, j = 4 * e - k * d;
      const float4* p = reinterpret_cast<const float4*>(part + (r * H + (long long)k * G) * d + j);
      float v[4] = {};
#pragma unroll 4
      for (int g = 0; g < G; ++g) {
        const float4 x = p[(long long)g * (d / 4)];
        v[0] += x.x;
        v[1] += x.y;
        v[2] += x.z;
        v[3] += x.w;
      }
      lin_store4<T>(out + k * hs + j, vec, v);
    }
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
// the state's first rows are on their way.  192 rows x 32 heads of 128 x 128: 133 us, 6.1 TB/s,
// 0.92 of the measured copy rate.
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
  // Of rows that name one slot the first is computed, the others are padding.  (Each row looks through those before it: 3 % of
  // 192 rows' time, 10 % of 4096's; at 65535 rows of one head it is what counts.)
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
