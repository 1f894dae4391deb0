// pn_linattn_tc.cuh -- linear attention over whole sequences on the tensor cores
// (tcgen05), for bfloat16 operands of widths a, b up to 128 (float16 would need a scale for every row of P and of S:
// neither stays within its range; wider ones do not fit TMEM and shared memory beside three chunks in flight).
//
// One pass of pn_linattn.cuh by chunks of C = 64 rows.  One CTA owns one
// (sequence, head, part) and takes its chunks in turn; the state S^T (dc x da,
// float32) never leaves the SM: it sits in the registers of eight warps.  Per chunk, all from operands
// that TMA brought in 128-byte swizzled rows:
//   P    = a b^T                          64 x 64     (masked, weighted, rounded: P~)
//   O1^T = S~^T a^T                       dc x 64     (S~: S rounded to the operands' type)
//   O2^T = c^T P~^T                       dc x 64
//   U^T  = c'^T b                         dc x da     (c'_j = e^{g(n-1-j)} c_j)
//   out_i = beta (e^{g(i+1)} O1_i + O2_i),   S = e^{gn} S + U.
// O1 and O2 share one accumulator: with x_i = i + 1 the rows seen at row i and r = 32,
//   out_i = beta e^{g(x_i - r)} [ (e^{gr} S) a_i + sum_j e^{g(r - x_j)} P_ij c_j ],
// so P~ takes the weight e^{g(r - x_j)}, the state is kept times e^{gr}, and one factor a row is left
// for the end.  It is the same sum times a power of e^g that is at most 2^40 either way where
// |g| <= 1.25 ln 2 (e^g >= 0.42); heads that forget faster keep two accumulators.
// The outputs are formed transposed, so that a TMEM lane is a column of c: a warp
// writes 32 neighbouring outputs of a row, and the state's rows stay in their lanes.
// No operand is rounded for the decay alone.  P~ and S~ are rounded once each to the
// operands' type: with u its half step, two relative errors of u on disjoint shares of
// an output that is itself rounded by u.  The state, which accumulates over the whole
// sequence and is returned in float32, takes c' in three pieces (c' = hi + mid + lo, 24
// bits), so that its products are float32 products, and is summed in float32 registers:
// accumulated by the tensor cores over many chunks it lost four bits to their truncation.
//
// Why this shape: a row and head of 128-wide bf16 operands is 1 KB of traffic, 64 rows take
// an SM 2850 clocks at the card's bandwidth, and the products of a chunk (six of up to
// 128 x 128 x 64) 1600 clocks of its tensor cores; what must not add up is the work
// between them.  So it is spread over warps that meet at mbarriers only:
//   warp 0       TMA loads, NS chunks ahead
//   warps 1-3    issue the products: U; the outputs'; P
//   warps 4-7    P -> P~
//   warps 8-11   the outputs
//   warps 12-19  S: the sum, in registers, and S~ (four warps for each half of its columns)
//   warps 20-27  c' of the chunk
// The chain from chunk to chunk is U and its sum; S~ and O1 hang off it.  At dc = 128 the pieces
// of c' lie in TMEM, transposed on their way by ldmatrix: an operand less for shared memory to
// feed (two such operands of a 128 x 128 x 16 step are its whole bandwidth), and room for a third
// chunk in flight.  At dc = 64 they lie in shared memory.
//
// What bounds the rest is instructions and the waits between the roles, which share four schedulers:
// accumulators are read in the 16 x 256-bit fragments, in which every lane holds values whatever M is and
// two neighbours sit in one thread, and go to shared memory by stmatrix, transposed for the outputs.
// Loops of several hundred instructions are rolled (unrolled, five roles overran the instruction
// cache: 3.7 stalls for each instruction issued; 2.1 rolled).
// Measured, 4 x 37 heads x 4096 rows (one CTA on every SM): width 128 129 us, 4.8 TB/s of the arrays'
// bytes, 0.73 of the measured copy rate, 0.58 instructions a scheduler and clock, tensor cores
// busy half of the time; width 64 69 to 77 us from process to process, 4.0 to 4.5 TB/s.
#pragma once

#include <type_traits>

#include "pn_wide_gemm.cuh"
#include "pn_linattn.cuh"

namespace pn {

// Waits that gave up on this device, ever (see pn_linattn_check): never cleared, so that nobody's report is taken by another.
__device__ unsigned lin_gave_up;

constexpr unsigned kLinWaitNs = 2000000000u;   // the limit where the handle sets none, and of the closing waits

// A try that the hardware may keep asleep for up to 20 us.
__device__ __forceinline__ bool lin_try(uint64_t* bar, unsigned parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity), "r"(20000)
      : "memory");
  return ok != 0;
}
// Bounded wait; gives up when the CTA has been told to, or after P.wait_ns.
__device__ __forceinline__ bool lin_wait(uint64_t* bar, unsigned parity, volatile int* abort, const LinPass& P) {
  if (lin_try(bar, parity)) return true;
  const unsigned t0 = (unsigned)globaltimer();
  while (true) {
    if (lin_try(bar, parity)) return true;
    if (*abort) return false;
    if ((unsigned)globaltimer() - t0 > P.wait_ns) {
      atomicAdd(&lin_gave_up, 1u);
      *abort = 1;
      return false;
    }
  }
}
// Waits for what the CTA has in flight before it ends.
__device__ __forceinline__ void lin_drain(uint64_t* bar, unsigned parity) {
  if (!mbar_drain(bar, parity, kLinWaitNs)) atomicAdd(&lin_gave_up, 1u);
}

// Instruction descriptor for kind::f16: D fp32, A and B of one 16-bit type (0: f16, 1: bf16),
// A MN-major at bit 15, B MN-major at bit 16, N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t umma_idesc_16(int type, int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((uint32_t)type << 7) | ((uint32_t)type << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void umma_16(uint32_t dtmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(dtmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The same with A in TMEM: row i in lane i, two 16-bit elements of K to a column.
__device__ __forceinline__ void umma_16_ts(uint32_t dtmem, uint32_t atmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(dtmem),
      "r"(atmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 4-D TMA tensor load of one box at (column, head, row, batch), counted on bar; the column is a multiple of 64.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar))
      : "memory");
}

// 4 N registers of 16 TMEM lanes x 8 N columns: of every 8 columns a thread gets columns 2 (lane & 3), + 1 of row
// lane >> 2, then of row (lane >> 2) + 8.
__device__ __forceinline__ void tmem_frag16(uint32_t a, float (&x)[16]) {
  __syncwarp();
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a)
      : "memory");
#pragma unroll
  for (int j = 0; j < 16; ++j) x[j] = __uint_as_float(r[j]);
}
// Waits for this warp's TMEM loads; the values they loaded pass through it.
__device__ __forceinline__ void tmem_wait16(float (&x)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7]), "+f"(x[8]),
                 "+f"(x[9]), "+f"(x[10]), "+f"(x[11]), "+f"(x[12]), "+f"(x[13]), "+f"(x[14]), "+f"(x[15])
               :
               : "memory");
}

// Four 8 x 8 matrices of 16-bit elements to shared memory; lane l gives the address of row l & 7 of matrix l >> 3.
__device__ __forceinline__ void stmatrix4(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(smem_addr(p)), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void stmatrix4_t(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(smem_addr(p)), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

// Four 8 x 8 matrices of 16-bit elements from shared memory, each transposed.
__device__ __forceinline__ void ldmatrix4_t(const void* p, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_addr(p))
               : "memory");
}
// 16 TMEM lanes x 8 columns: of every 4 columns a thread gives column lane & 3 of row lane >> 2, then of row + 8.
__device__ __forceinline__ void tmem_st_frag4(uint32_t a, const uint32_t (&r)[4]) {
  __syncwarp();
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

// Copies f times DH x DC values of a state between global memory g (strides gd, gc; one of them is 1; nd x nc values are
// there, the others count as zero) and shared memory x, [c][DH] with d moved by 8 (c & 3) places; 128 threads.  A function of
// its own: it runs once, and inlined it lay between the loops, which an instruction cache holds with little to spare (the
// same loops took 72 or 87 us at 4 x 37 heads x 4096 rows of width 64, by what lay between them).
template <int DC, int DH, bool OUT>
__device__ __noinline__ void lin_carry(float* x, const float* g, long long gd, long long gc, float f, int nd, int nc, int tw) {
  constexpr int kEach = DC * DH / 512, kBatch = kEach < 8 ? kEach : 8;   // groups of four of a thread; on their way at once
  const bool along_c = gc == 1;   // four of c (times 8 of d to a warp), or four of d
#pragma unroll 1
  for (int i0 = tw; i0 < 128 * kEach; i0 += 128 * kBatch) {
    float4 v[kBatch];
    auto place = [&](int u, int& c, int& d) {
      const int i = i0 + 128 * u;
      c = along_c ? 4 * ((i & 3) + 4 * (i / (4 * DH))) : i / (DH / 4);
      d = along_c ? (i >> 2) % DH : 4 * (i % (DH / 4));
      return c < nc && d < nd;
    };
    auto memory = [&](int c, int d) { return reinterpret_cast<float4*>(const_cast<float*>(g) + d * gd + c * gc); };
    auto stage = [&](float4& y, int c, int d, bool store) {
      if (along_c) {
        float* z[4] = {x + c * DH + d, x + (c + 1) * DH + (d ^ 8), x + (c + 2) * DH + (d ^ 16), x + (c + 3) * DH + (d ^ 24)};
        if (store) *z[0] = y.x, *z[1] = y.y, *z[2] = y.z, *z[3] = y.w;
        else y = make_float4(*z[0], *z[1], *z[2], *z[3]);
      } else {
        float4* z = reinterpret_cast<float4*>(x + c * DH + (d ^ (8 * (c & 3))));
        if (store) *z = y;
        else y = *z;
      }
    };
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      int c, d;
      const bool on = place(u, c, d);
      v[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (OUT) stage(v[u], c, d, false);
      else if (on) v[u] = *memory(c, d);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      int c, d;
      const bool on = place(u, c, d);
      v[u] = make_float4(f * v[u].x, f * v[u].y, f * v[u].z, f * v[u].w);
      if (!OUT) stage(v[u], c, d, true);
      else if (on) *memory(c, d) = v[u];
    }
  }
}

// The n staged rows of outputs (boxes of 64 columns, 128-byte swizzled) to global memory, 16 bytes a thread where `wide`;
// nc columns are there; 128 threads.  Short chunks and outputs that TMA cannot store.
template <typename T, int DC>
__device__ __noinline__ void lin_rows_out(T* out, const unsigned char* stage, long long ts, int n, int nc, bool wide, int t) {
#pragma unroll 1
  for (int e = t; e < 64 * DC / 8; e += 128) {
    const int r = e / (DC / 8), ch = e % (DC / 8);
    if (r >= n || 8 * ch >= nc) continue;
    const uint4 v = *reinterpret_cast<const uint4*>(stage + (ch >> 3) * (64 * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
    T* o = out + r * ts + 8 * ch;
    if (wide) {
      *reinterpret_cast<uint4*>(o) = v;
    } else {
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
      unsigned short* o16 = reinterpret_cast<unsigned short*>(o);
#pragma unroll
      for (int i = 0; i < 8; ++i) o16[i] = (unsigned short)(u[i >> 1] >> (16 * (i & 1)));
    }
  }
}

template <int N> __device__ __forceinline__ void regs_take() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_give() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

template <typename T> struct Tc16;
template <> struct Tc16<__nv_bfloat16> {
  static constexpr int kType = 1;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {   // two elements, the first in the low half
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
  // both elements of v, weighted, in three pieces of 8 bits by truncation: their sum is the float32 product
  static __device__ __forceinline__ void pieces(unsigned long long w, uint32_t v, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    const unsigned long long minus = pack2(-1.0f, -1.0f);
    auto cut = [&](unsigned long long& x) {   // the top 16 bits of both, which x loses
      float a, b;
      unpack2(x, a, b);
      const uint32_t top = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
      x = fma2(pack2(__uint_as_float(__float_as_uint(a) & 0xffff0000u), __uint_as_float(__float_as_uint(b) & 0xffff0000u)), minus, x);
      return top;
    };
    unsigned long long x = mul2(w, pack2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)));
    hi = cut(x);
    mid = cut(x);
    float a, b;
    unpack2(x, a, b);
    lo = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
  }
};

// One lane of the warp, the same in every call; unlike a comparison of the lane it leaves the compiler a
// uniform branch (products are issued every 28-54 clocks by this one, every 48-61 by `lane == 0`).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  __syncwarp();
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// 4-D TMA tensor store of one box; elements outside the array are not written.
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, int c0, int c1, int c2, int c3, const void* src) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(map), "r"(c0), "r"(c1),
               "r"(c2), "r"(c3), "r"(smem_addr(src))
               : "memory");
}

struct LinMaps {
  CUtensorMap a, b, c, o;
};

constexpr int kLinSorted = 512;   // up to this many sequences can be taken by length

// The sequence with `s` others before it by length in chunks, equal ones in their order; n <= kLinSorted of them.  Every CTA asks:
// one warp finds the s-th largest key, a bit at a time (each of n threads ranking one against all took a CTA 30 us at 512
// sequences).  All threads call it.
template <int NT>
__device__ __forceinline__ int lin_by_length(const int* cu, long long T, int n, int s) {
  __shared__ unsigned s_key[kLinSorted];
  __shared__ int s_seq;
  for (int i = threadIdx.x; i < kLinSorted; i += NT) {
    unsigned key = 0;
    if (i < n) {
      long long lo, hi;
      lin_span(cu, T, i, lo, hi);
      const long long chunks = (hi - lo + 63) / 64;
      key = (unsigned)(chunks < (1 << 22) - 1 ? chunks : (1 << 22) - 1) << 10 | (unsigned)(1023 - i);
    }
    s_key[i] = key;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    unsigned key[kLinSorted / 32], top = 0;
#pragma unroll
    for (int x = 0; x < kLinSorted / 32; ++x) {
      key[x] = s_key[threadIdx.x + 32 * x];
      top = max(top, key[x]);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    unsigned found = 0;   // the largest value that more than s keys reach
#pragma unroll 1
    for (unsigned bit = 1u << (31 - __clz(top)); bit; bit >>= 1) {
      int reach = key[0] >= (found | bit);
      if (n > 32) {
#pragma unroll
        for (int x = 1; x < kLinSorted / 32; ++x) reach += key[x] >= (found | bit);
      }
      if (__reduce_add_sync(0xffffffffu, reach) > s) found |= bit;
    }
    if (threadIdx.x == 0) s_seq = 1023 - (int)(found & 1023u);
  }
  __syncthreads();
  return s_seq;
}

template <int DA, int DC>
struct LinTcCfg {
  static constexpr int C = 64;
  static constexpr int NT = 896;
  static constexpr int SUB = C * 128;                      // one box: 64 rows of 64 elements
  static constexpr int A_BYTES = C * DA * 2, C_BYTES = C * DC * 2;
  static constexpr int STAGE = 2 * A_BYTES + C_BYTES;      // a, b, c
  static constexpr int SB_BYTES = DC * DA * 2;             // S~^T
  static constexpr int P_BYTES = C * C * 2;                // P~
  static constexpr int NP = 3;                             // pieces of c'
  static constexpr int O_BYTES = C * DC * 2;               // outputs on their way, twice where there is room
  static constexpr int NOUT = DA == 128 && DC == 128 ? 1 : 2;
  static constexpr bool TS = DC == 128;                    // the pieces lie in TMEM
  static constexpr int CP_BYTES = TS ? 0 : 2 * NP * C_BYTES;   // (twice, as in TMEM)
  static constexpr int FIXED = SB_BYTES + 2 * P_BYTES + CP_BYTES + NOUT * O_BYTES;
  static constexpr int NSTAGE = (220 * 1024 - FIXED) / STAGE < 4 ? (220 * 1024 - FIXED) / STAGE : 4;
  static constexpr int OFF_SB = NSTAGE * STAGE;
  static constexpr int OFF_P = OFF_SB + SB_BYTES;
  static constexpr int OFF_CP = OFF_P + 2 * P_BYTES;
  static constexpr int OFF_O = OFF_CP + CP_BYTES;
  static constexpr int SMEM_BYTES = OFF_O + NOUT * O_BYTES + 1024;   // + alignment slack
  static constexpr int COL_U = 0, COL_P = DA, COL_O = DA + 64;   // outputs twice: two chunks', or O1 and O2 of one
  static constexpr int COL_CP = DA + 192;                  // twice 32 columns a piece
  static constexpr int TCOLS = 512;
  static_assert(COL_CP + (TS ? 2 * 32 * NP : 0) <= TCOLS, "TMEM columns");
  static_assert(NSTAGE >= 2, "two stages at least");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

enum { kLinOut, kLinOutF32, kLinStateOnly };   // what a pass writes: outputs of type T, float32 ones, states only

template <typename T, int DA, int DC, int WHAT>
__global__ void __launch_bounds__(896, 1) lin_tc_kernel(const __grid_constant__ LinMaps maps, const __grid_constant__ LinPass P,
                                                        const __grid_constant__ LinDecay G) {
  using K = LinTcCfg<DA, DC>;
  using X = Tc16<T>;
  constexpr int C = K::C, NS = K::NSTAGE, R = C / 2;
  constexpr bool STATE_ONLY = WHAT == kLinStateOnly;
  extern __shared__ __align__(1024) unsigned char smem_lt[];
  unsigned char* base = smem_lt + ((1024u - (smem_addr(smem_lt) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t bar_full[NS], bar_empty[NS], bar_pacc, bar_p[2], bar_s, bar_u, bar_ur, bar_o1, bar_cp[2], bar_cpf[2], bar_zero, bar_init, bar_oacc[2], bar_o[2], bar_done[3];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ int s_loaded;
  __shared__ __align__(16) float s_out[2][C];   // the factor of row i's outputs (two: of O1): the first chunk, the others
  __shared__ float s_w[C];                      // the weight of column j of P (two: at |i - j|)
  __shared__ __align__(16) float s_c[C];        // the weights of c', from the far end of a whole chunk

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // CTAs start in the order of their numbers, each for the whole of its part: the longest sequences first, so that no long
  // one starts late, where that can matter (the rule is the caller's)
  const int h = blockIdx.y % P.H;
  int s = blockIdx.y / P.H;
  if (P.by_length) s = lin_by_length<K::NT>(P.cu, P.T, P.n_seq, s);
  const int sh = s * P.H + h;
  const int dc0 = blockIdx.x * DC;
  const int part = blockIdx.z;
  const float l2 = G.log2[h];

  long long start;
  int len;
  lin_rows(P, s, start, len);
  const int nch = (len + C - 1) / C;                       // chunks of the sequence, in the order of the rows
  const int cps = (nch + P.nseg - 1) / P.nseg;             // chunks of a part, in the order they are taken
  const int m0 = part * cps < nch ? part * cps : nch, m1 = m0 + cps < nch ? m0 + cps : nch;
  const int M = m1 - m0;
  const bool owns_end = m1 == nch && (M > 0 || part == 0);
  if (STATE_ONLY ? (M == 0 || m1 == nch) : (M == 0 && !owns_end)) return;
  const int tail = len - (nch - 1) * C;                    // rows of the last chunk (in row order)
  auto chunk_of = [&](int m) { return P.reverse ? nch - 1 - (m0 + m) : m0 + m; };
  auto rows_of = [&](int m) { return chunk_of(m) == nch - 1 ? tail : C; };
  // against time the state that enters the last row is not decayed by it
  const int e0 = (!STATE_ONLY && P.reverse && part == 0) ? 1 : 0;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&bar_full[i], 1u);
      mbar_init(&bar_empty[i], STATE_ONLY ? 1u : 3u);
    }
    mbar_init(&bar_pacc, 1u);
    mbar_init(&bar_s, 8u);
    mbar_init(&bar_u, 1u);
    mbar_init(&bar_ur, 8u);
    mbar_init(&bar_init, 8u);
    mbar_init(&bar_zero, 8u);   // c is zero behind the last row (once, for the one short chunk there may be)
    mbar_init(&bar_o1, 1u);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_cp[i], 8u);
      mbar_init(&bar_cpf[i], 1u);
      mbar_init(&bar_oacc[i], 1u);
      mbar_init(&bar_o[i], 4u);
      mbar_init(&bar_p[i], 4u);
    }
    for (int i = 0; i < 3; ++i) mbar_init(&bar_done[i], 1u);
    mbar_init_fence();
    s_abort = 0;
    s_loaded = 0;
  }
  const bool two = !STATE_ONLY && !(l2 >= -1.25f);            // O1 and O2 apart
  const float frame = STATE_ONLY || two ? 1.0f : exp2f(l2 * R);   // the state is kept times this
  if (tid < 2 * C) {
    const int which = tid / C, i = tid % C;
    int n = P.reverse ? C - i : i + 1;
    if (two && P.reverse && which == 0) n = (M > 0 ? rows_of(0) : C) - i - e0;
    s_out[which][i] = P.beta * (two ? lin_pow(l2, n) : exp2f(l2 * (float)(n - R)));
  } else if (tid < 3 * C) {
    const int n = tid - 2 * C;
    s_w[n] = P.alpha * (two ? P.beta * lin_pow(l2, n) : exp2f(l2 * (float)(R - (P.reverse ? C - n : n + 1))));
    s_c[P.reverse ? n : C - 1 - n] = P.alpha * frame * lin_pow(l2, n);
  }
  if (warp == 0) tmem_alloc(&s_tmem, (uint32_t)K::TCOLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  unsigned char* sb = base + K::OFF_SB;
  auto sA = [&](int st) { return base + st * K::STAGE; };
  auto sB = [&](int st) { return base + st * K::STAGE + K::A_BYTES; };
  auto sC = [&](int st) { return base + st * K::STAGE + 2 * K::A_BYTES; };

  // registers: 896 threads start with 72 each; what some give others take (40 + 72 + 72 + 2 * 104 + 2 * 56 = 7 * 72)
  if (warp < 4) {
    regs_give<40>();
    if (warp == 0) {
      // ------------------------------- loads -------------------------------
      if (lane == 0) {
        const int bz = P.cu ? 0 : s;
        const int loads = (int)min((unsigned)M, (unsigned)P.stall);   // (all; a test may leave out the rest, and the waits for them run out)
        for (int m = 0; m < loads; ++m) {
          const int st = m % NS;
          if (m == 1 && !lin_wait(&bar_init, 0u, &s_abort, P)) break;   // the state came in by way of the other stages
          if (m >= NS && !lin_wait(&bar_empty[st], (unsigned)(m / NS - 1) & 1u, &s_abort, P)) break;
          const int row = (int)start + chunk_of(m) * C;
          mbar_arrive_expect_tx(&bar_full[st], (unsigned)(STATE_ONLY ? K::STAGE - K::A_BYTES : K::STAGE));
#pragma unroll
          for (int i = 0; i < DA / 64; ++i) {
            tma_load_4d(sB(st) + i * K::SUB, &maps.b, i * 64, h / P.b.per, row, bz, &bar_full[st]);
            if (!STATE_ONLY) tma_load_4d(sA(st) + i * K::SUB, &maps.a, i * 64, h / P.a.per, row, bz, &bar_full[st]);
          }
#pragma unroll
          for (int i = 0; i < DC / 64; ++i)
            tma_load_4d(sC(st) + i * K::SUB, &maps.c, dc0 + i * 64, h / P.c.per, row, bz, &bar_full[st]);
          s_loaded = m + 1;
        }
      }
      __syncwarp();
    } else {
      // ------------------------------ products -----------------------------
      constexpr uint32_t id_p = umma_idesc_16(X::kType, C, C, false, false);
      constexpr uint32_t id_o1 = umma_idesc_16(X::kType, DC, C, false, false);
      constexpr uint32_t id_o2 = umma_idesc_16(X::kType, DC, C, true, false);
      constexpr uint32_t id_u = umma_idesc_16(X::kType, DC, DA, true, true), id_u_ts = umma_idesc_16(X::kType, DC, DA, false, true);
      // K-major: 8 rows of 128 bytes 1024 apart, 16 elements of K 32 bytes along the row.
      // MN-major: 64 elements along the row, the next 64 a box on; 8 rows of K 1024 apart.
      auto kmaj = [&](const void* p) { return umma_smem_desc(smem_addr(p), 16, 1024, 2); };
      auto mnmaj = [&](const void* p) { return umma_smem_desc(smem_addr(p), K::SUB, 1024, 2); };
      const uint64_t d_sb = kmaj(sb);
      // product of K = 16 steps; an operand advances by a step of its kind: 32 bytes along a K-major row (the next box
      // after 64 elements), 16 rows of an MN-major one
      auto product = [&](uint32_t d, uint64_t x, auto x_box, uint64_t y, auto y_box, auto steps, uint32_t id, bool add) {
        constexpr int xb = decltype(x_box)::value, yb = decltype(y_box)::value, ks = decltype(steps)::value;
#pragma unroll
        for (int k = 0; k < ks; ++k)
          umma_16(d, x + (uint64_t)((xb ? (k & 3) * 32 + (k >> 2) * xb : k * 2048) >> 4),
                  y + (uint64_t)((yb ? (k & 3) * 32 + (k >> 2) * yb : k * 2048) >> 4), id, (k || add) ? 1u : 0u);
      };
      using Box = std::integral_constant<int, K::SUB>;
      using SBox = std::integral_constant<int, DC * 128>;
      using Mn = std::integral_constant<int, 0>;
      using DSteps = std::integral_constant<int, DA / 16>;
      using CSteps = std::integral_constant<int, C / 16>;
      bool ok = true;
      for (int m = 0; m < M && ok && warp == 1; ++m) {
        const int st = m % NS;
        // what the chunk adds to the state, once what the chunk before added is read
        if (!(ok = lin_wait(&bar_cp[m & 1], (unsigned)(m >> 1) & 1u, &s_abort, P))) break;
        if (m > 0 && !(ok = lin_wait(&bar_ur, (unsigned)(m - 1) & 1u, &s_abort, P))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t db = mnmaj(sB(st));
#pragma unroll
          for (int p = 0; p < K::NP; ++p) {
            if constexpr (K::TS) {
#pragma unroll
              for (int k = 0; k < C / 16; ++k)
                umma_16_ts(tmem + K::COL_U, tmem + K::COL_CP + 32 * K::NP * (m & 1) + 32 * p + 8 * k, db + (uint64_t)(k * 2048 >> 4),
                           id_u_ts, (p || k) ? 1u : 0u);
            } else {
              product(tmem + K::COL_U, mnmaj(base + K::OFF_CP + (K::NP * (m & 1) + p) * K::C_BYTES), Mn{}, db, Mn{}, CSteps{}, id_u, p > 0);
            }
          }
          umma_commit(&bar_u);
          umma_commit(&bar_cpf[m & 1]);
          umma_commit(&bar_empty[st]);
        }
        __syncwarp();
      }
      // the outputs: the state's share and the chunk's own, once what their columns held is read
      for (int m = 0; m < M && ok && warp == 2 && !STATE_ONLY; ++m) {
        const int st = m % NS, before = two ? m - 1 : m - 2;
        if (!(ok = lin_wait(&bar_p[m & 1], (unsigned)(m >> 1) & 1u, &s_abort, P))) break;
        if (before >= 0 && !(ok = lin_wait(&bar_o[before & 1], (unsigned)(before >> 1) & 1u, &s_abort, P))) break;
        if (rows_of(m) < C && !(ok = lin_wait(&bar_zero, 0u, &s_abort, P))) break;
        if (!(ok = lin_wait(&bar_s, (unsigned)m & 1u, &s_abort, P))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t o1 = tmem + K::COL_O + (two ? 0 : 64 * (m & 1)), o2 = tmem + K::COL_O + (two ? 64 : 64 * (m & 1));
          product(o1, d_sb, SBox{}, kmaj(sA(st)), Box{}, DSteps{}, id_o1, false);
          umma_commit(&bar_o1);
          product(o2, mnmaj(sC(st)), Mn{}, kmaj(base + K::OFF_P + (m & 1) * K::P_BYTES), Box{}, CSteps{}, id_o2, !two);
          umma_commit(&bar_oacc[m & 1]);
          umma_commit(&bar_empty[st]);
        }
        __syncwarp();
      }
      // P, once the chunk before's is read
      for (int m = 0; m < M && ok && warp == 3 && !STATE_ONLY; ++m) {
        const int st = m % NS;
        if (!(ok = lin_wait(&bar_full[st], (unsigned)(m / NS) & 1u, &s_abort, P))) break;
        if (m > 0 && !(ok = lin_wait(&bar_p[(m - 1) & 1], (unsigned)((m - 1) >> 1) & 1u, &s_abort, P))) break;
        tc_fence_after();
        if (elect_one()) {
          product(tmem + K::COL_P, kmaj(sA(st)), Box{}, kmaj(sB(st)), Box{}, DSteps{}, id_p, false);
          umma_commit(&bar_pacc);
          umma_commit(&bar_empty[st]);
        }
        __syncwarp();
      }
    }
  } else if (warp < 8) {
    if (!STATE_ONLY) {
      // --------------------------------- P~ --------------------------------
      const int w = warp & 3;
      const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16);
      const int fr = lane >> 2, fc = 2 * (lane & 3);   // this thread's row and column of an 8 x 8 fragment
      const int mr = lane & 7, mi = lane >> 3;         // the row and matrix it addresses
      // rows 16 w .. of P (an M = 64 accumulator takes lanes 0-15 of each quarter); the weights on this side of the
      // diagonal, zero on the other
      float wt[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const int i = 16 * w + fr + (e & 2) * 4, jj = (e >> 2) * 8 + fc + (e & 1);
        const int n = P.reverse ? jj - i : i - jj;
        wt[e] = n >= 0 ? s_w[two ? (n >= 0 ? n : 0) : jj] : 0.0f;
      }
      const int pi = 16 * w + mr + (mi & 1) * 8;       // row of P~ addressed; matrices: rows, rows + 8, next 8 columns
      for (int m = 0; m < M; ++m) {
        if (m > 1 && !lin_wait(&bar_oacc[m & 1], (unsigned)((m >> 1) - 1) & 1u, &s_abort, P)) break;   // P~ two chunks ago is used
        if (!lin_wait(&bar_pacc, (unsigned)m & 1u, &s_abort, P)) break;
        tc_fence_after();
        const int n = rows_of(m);
        unsigned char* dst = base + K::OFF_P + (m & 1) * K::P_BYTES + pi * 128;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float v[16];
          tmem_frag16(lanes + (uint32_t)(K::COL_P + 32 * q), v);
          tmem_wait16(v);
#pragma unroll
          for (int e = 0; e < 16; e += 2)
            unpack2(mul2(pack2(wt[16 * q + e], wt[16 * q + e + 1]), pack2(v[e], v[e + 1])), v[e], v[e + 1]);
          if (n < C) {   // rows behind the last one hold anything
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 32 * q + (e >> 2) * 8 + fc + (e & 1) < n ? v[e] : 0.0f;
          }
#pragma unroll
          for (int k = 0; k < 4; k += 2)
            stmatrix4(dst + (((4 * q + k + (mi >> 1)) ^ mr) << 4), X::pack(v[4 * k], v[4 * k + 1]), X::pack(v[4 * k + 2], v[4 * k + 3]),
                      X::pack(v[4 * k + 4], v[4 * k + 5]), X::pack(v[4 * k + 6], v[4 * k + 7]));
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_p[m & 1]);
      }
    }
  } else if (warp < 12) {
    if (!STATE_ONLY) {
      // ------------------------------ the outputs --------------------------
      const int w = warp & 3, t = tid - 256;
      const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16);
      const int fr = lane >> 2, fc = 2 * (lane & 3), mr = lane & 7, mi = lane >> 3;
      const long long at = (P.cu ? 0 : s * P.out_bs) + (long long)h * P.out_hs + dc0;
      const bool wide = P.out_map || (((uintptr_t)P.out | (uintptr_t)(2 * P.out_bs) | (uintptr_t)(2 * P.out_ts) | (uintptr_t)(2 * P.out_hs)) & 15u) == 0;
      for (int m = 0; m < M; ++m) {
        unsigned char* stage = base + K::OFF_O + (K::NOUT == 2 ? (m & 1) * K::O_BYTES : 0);
        const bool ok = lin_wait(&bar_oacc[m & 1], (unsigned)(m >> 1) & 1u, &s_abort, P);
        if (t == 0) {   // the copy that last read this memory is done with it
          if (K::NOUT == 2) bulk_wait_read_but1();
          else bulk_wait_read();
        }
        if (!named_barrier_and(1, 128, ok)) break;   // one decision; and the staged outputs before these are gone
        tc_fence_after();
        const int n = rows_of(m);
        const float* f = s_out[m == 0 ? 0 : 1] + fc;
        T* out = (T*)P.out + at + (start + (long long)chunk_of(m) * C) * P.out_ts;
#pragma unroll 2
        for (int q = 0; q < DC / 32; ++q) {   // 16 columns of c and 32 rows at a time
          const int g = DC == 128 ? q >> 1 : 0, r0 = 32 * (DC == 128 ? q & 1 : q);
          const uint32_t a = lanes + ((uint32_t)(16 * g) << 16) + (uint32_t)(K::COL_O + r0);
          float x[16];
          tmem_frag16(two ? a : a + (uint32_t)(64 * (m & 1)), x);
          tmem_wait16(x);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const unsigned long long ff = *reinterpret_cast<const unsigned long long*>(f + r0 + 8 * k);
#pragma unroll
            for (int e = 4 * k; e < 4 * k + 4; e += 2) unpack2(mul2(ff, pack2(x[e], x[e + 1])), x[e], x[e + 1]);
          }
          if (two) {
            float y[16];
            tmem_frag16(a + 64u, y);
            tmem_wait16(y);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] += y[e];
          }
          const int c0 = DC == 128 ? 32 * w + 16 * g : 16 * w;   // first column of c
          if constexpr (WHAT == kLinOutF32) {
            float* o = (float*)P.out + at + (start + (long long)chunk_of(m) * C + r0 + fc) * P.out_ts + c0 + fr;
            const int left = n - r0 - fc;   // rows from this thread's first on
            const bool on0 = dc0 + c0 + fr < P.dc, on1 = dc0 + c0 + fr + 8 < P.dc;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float* oe = e ? o + P.out_ts : o;
                if (8 * k + e < left) {
                  if (on0) oe[0] = x[4 * k + e];
                  if (on1) oe[8] = x[4 * k + e + 2];
                }
              }
              o += 8 * P.out_ts;
            }
          } else {
            // transposed: row r0 + 8 (k + (mi >> 1)) + mr, 8 columns from c0 + 8 (mi & 1)
            unsigned char* to = stage + (c0 >> 6) * K::SUB;
            const int ch = ((c0 & 63) >> 3) + (mi & 1);
#pragma unroll
            for (int k = 0; k < 4; k += 2)
              stmatrix4_t(to + (r0 + 8 * (k + (mi >> 1)) + mr) * 128 + ((ch ^ mr) << 4), X::pack(x[4 * k], x[4 * k + 1]),
                          X::pack(x[4 * k + 2], x[4 * k + 3]), X::pack(x[4 * k + 4], x[4 * k + 5]), X::pack(x[4 * k + 6], x[4 * k + 7]));
          }
        }
        tc_fence_before();   // the accumulators are read
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_o[m & 1]);
        if (WHAT == kLinOut && n == C && P.out_map) {
          fence_async_smem();
          named_barrier(1, 128);
          if (t == 0) {
#pragma unroll
            for (int x = 0; x < DC / 64; ++x)
              if (dc0 + 64 * x < P.dc) tma_store_4d(&maps.o, dc0 + 64 * x, h, (int)start + chunk_of(m) * C, P.cu ? 0 : s, stage + x * K::SUB);
            bulk_commit();
          }
        } else if (WHAT == kLinOut) {
          named_barrier(1, 128);
          lin_rows_out<T, DC>(out, stage, P.out_ts, n, P.dc - dc0, wide, t);
        }
      }
      if (t == 0) bulk_wait_all();
    }
  } else if (warp < 20) {
    regs_take<104>();
    // ------------------------------- the state ---------------------------
    constexpr int NB = DC / 64;        // 16-lane groups of a warp: 16 columns of c each
    constexpr int NQ = DA / 64;        // 32-column blocks of this warp's half
    const int w = warp & 3;
    const int half = warp < 16 ? 0 : DA / 2;
    const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16);
    const int fr = lane >> 2, fc = 2 * (lane & 3), mr = lane & 7, mi = lane >> 3;
    const long long size = (long long)P.da * P.dc;
    const float* src = nullptr;   // what enters: (d, j) at src[d * sd + j * sj]
    float* dst = nullptr;         // what leaves
    long long sd = 0, sj = 0, dd = 0, dj = 0;
    float f_out = 1.0f;
    if (!STATE_ONLY && P.nseg > 1) {
      src = P.seg_state + ((long long)sh * P.nseg + part) * size;
      sd = P.dc;
      sj = 1;
    } else if (!STATE_ONLY && P.s_in) {
      src = P.s_in + sh * size;
      sd = P.s_row;
      sj = P.s_col;
    }
    if (STATE_ONLY) {
      dst = P.seg_state + ((long long)sh * P.nseg + part + 1) * size;
      dd = P.dc;
      dj = 1;
    } else if (P.s_out && owns_end) {
      dst = P.s_out + sh * size;
      dd = P.s_row;
      dj = P.s_col;
      if (P.reverse && len > 0) f_out = lin_pow(l2, 1);   // against time the first state's gradient still decays by the first row
    }
    // States go in and out by way of stages that hold no chunk then (the second and third before they do; those of the two
    // chunks before the last), four neighbours at a time in the order they lie in memory: as fragments, straight, they were
    // 64 loads of single values in code that runs once, which took 18 us.  Each half of the columns has a stage of its own,
    // [c][DH] with d moved by 8 (c & 3) places, so that a fragment's pairs lie in different banks.
    constexpr int DH = DA / 2;
    static_assert(NS >= 3 && DC * DH * 4 <= K::STAGE, "a stage holds half of a state");
    const int hi_half = half ? 1 : 0, tw = (warp & 3) * 32 + lane;
    auto stage_of = [&](int i) { return reinterpret_cast<float*>(base + i * K::STAGE); };
    auto carry = [&](auto out, float* x, const float* g, long long gd, long long gc, float f) {
      lin_carry<DC, DH, decltype(out)::value>(x, g + half * gd + dc0 * gc, gd, gc, f, P.da - half, P.dc - dc0, tw);
    };
    // pair (e, e + 1) of block (b, q): row c, column 32 q + 8 (e >> 2) + fc of the half
    auto pair_at = [&](float* x, int b, int q, int e) {
      const int c = (DC == 128 ? 32 * w + 16 * b : 16 * w) + fr + (e & 2) * 4;
      return reinterpret_cast<float2*>(x + c * DH + 32 * q + ((8 * (e >> 2)) ^ (8 * (fr & 3))) + fc);
    };
    // Against time the first chunk's rows (a short chunk, or the last row undecayed) see the state this much earlier than
    // those of a whole one, for which the row factors and P~ are made: it enters that much larger, and decays as over a
    // whole chunk.  (No rows, no frame: the state of an empty sequence passes as it is.)
    const int early = P.reverse && !two && M > 0 && !STATE_ONLY ? C - rows_of(0) + e0 : 0;
    const float lead = M > 0 ? frame * exp2f(-l2 * (float)early) : 1.0f;
    float S[NB][NQ][16] = {};
    if (src) {
      float* x = stage_of(1 + hi_half);
      carry(std::false_type{}, x, src, sd, sj, lead);
      named_barrier(2 + hi_half, 128);   // (nothing waited for yet: every warp comes here)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float2 v = *pair_at(x, b, q, e);
            S[b][q][e] = v.x;
            S[b][q][e + 1] = v.y;
          }
      fence_async_smem();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar_init);
    if (!two && M > 0) f_out *= exp2f(-l2 * R);
    if (STATE_ONLY) f_out = 1.0f;
    const float f_full = lin_pow(l2, C);
    bool ok = true;
    for (int m = 0; m <= M; ++m) {
      if (m > 0) {
        if (!(ok = lin_wait(&bar_u, (unsigned)(m - 1) & 1u, &s_abort, P))) break;
        tc_fence_after();
        const int n = rows_of(m - 1) - (m == 1 ? e0 - early : 0);
        const float f = n == C ? f_full : lin_pow(l2, n);
        const unsigned long long ff = pack2(f, f);
        auto add = [&](float (&v)[16], const float (&u)[16]) {
#pragma unroll
          for (int e = 0; e < 16; e += 2) unpack2(fma2(ff, pack2(v[e], v[e + 1]), pack2(u[e], u[e + 1])), v[e], v[e + 1]);
        };
        auto where = [&](int b, int q) { return lanes + ((uint32_t)(16 * b) << 16) + (uint32_t)(K::COL_U + half + 32 * q); };
        constexpr int NX = NB * NQ;
#pragma unroll
        for (int x = 0; x < NX; x += 2) {   // two blocks in flight
          float u[16], u2[16];
          tmem_frag16(where(x / NQ, x % NQ), u);
          if (x + 1 < NX) tmem_frag16(where((x + 1) / NQ, (x + 1) % NQ), u2);
          tmem_wait16(u);
          add(S[x / NQ][x % NQ], u);
          if (x + 1 < NX) {
            tmem_wait16(u2);
            add(S[(x + 1) / NQ][(x + 1) % NQ], u2);
          }
        }
        tc_fence_before();   // U is read
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_ur);
        // O1 of the chunk before has read S~
        if (!STATE_ONLY && !(ok = lin_wait(&bar_o1, (unsigned)(m - 1) & 1u, &s_abort, P))) break;
      }
      if (m == M) break;
      if (!STATE_ONLY) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int row = (DC == 128 ? 32 * w + 16 * b : 16 * w) + mr + (mi & 1) * 8;
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            const int d0 = half + 32 * q;
            unsigned char* to = sb + (d0 >> 6) * (DC * 128) + row * 128;
            const float (&v)[16] = S[b][q];
#pragma unroll
            for (int k = 0; k < 4; k += 2)
              stmatrix4(to + (((((d0 & 63) >> 3) + k + (mi >> 1)) ^ mr) << 4), X::pack(v[4 * k], v[4 * k + 1]),
                        X::pack(v[4 * k + 2], v[4 * k + 3]), X::pack(v[4 * k + 4], v[4 * k + 5]), X::pack(v[4 * k + 6], v[4 * k + 7]));
          }
        }
        fence_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_s);
    }
    if (dst) {   // (the same in every thread)
      float* x = stage_of(M == 0 ? 1 + hi_half : (M + hi_half) % NS);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
          for (int e = 0; e < 16; e += 2)
            if (ok) *pair_at(x, b, q, e) = make_float2(S[b][q][e], S[b][q][e + 1]);
      if (named_barrier_and(2 + hi_half, 128, ok)) carry(std::true_type{}, x, dst, dd, dj, f_out);
    }
  } else {
    regs_give<56>();
    // -------------------------------- c' ---------------------------------
    const int t = tid - 640;
    // transposed (TS): 16 columns of c, in TMEM lanes of their own, and all 64 rows; this thread's rows of a fragment are
    // 8 k + 2 (lane & 3), + 1.  Else rows (t >> 3) + 32 k of every 64 columns, 16 bytes at (t & 7).
    const int w = warp & 3, g = (warp - 20) >> 2, mr = lane & 7, mi = lane >> 3;
    const int c0 = 32 * w + 16 * g;
    const uint32_t to_tmem = tmem + ((uint32_t)c0 << 16) + (uint32_t)K::COL_CP;
    const int from = (c0 >> 6) * K::SUB + (8 * (mi >> 1) + mr) * 128 + (((((c0 & 63) >> 3) + (mi & 1)) ^ mr) << 4);
    for (int m = 0; m < M; ++m) {
      const int st = m % NS, n = rows_of(m);
      if (!lin_wait(&bar_full[st], (unsigned)(m / NS) & 1u, &s_abort, P)) break;
      unsigned char* src = sC(st);
      if (n < C) {
        // Rows behind the last one hold anything: zero b and c there (the products that may be reading b
        // meanwhile are masked in those rows, and so are the pieces below).
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          if ((t >> 3) + 32 * k >= n) {
            const uint4 z = make_uint4(0, 0, 0, 0);
            for (int x = 0; x < DC / 64; ++x) *reinterpret_cast<uint4*>(src + x * K::SUB + (t + 256 * k) * 16) = z;
            for (int x = 0; x < DA / 64; ++x) *reinterpret_cast<uint4*>(sB(st) + x * K::SUB + (t + 256 * k) * 16) = z;
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_zero);
      }
      if (m > 1 && !lin_wait(&bar_cpf[m & 1], (unsigned)((m >> 1) - 1) & 1u, &s_abort, P)) break;   // the pieces two chunks ago are used
      if constexpr (K::TS) {
        __syncwarp();
#pragma unroll 1
        for (int jb = 0; jb < 4; ++jb) {   // 16 rows
          uint32_t v[4], o[3][4];
          ldmatrix4_t(src + from + 16 * jb * 128, v);
          const int r0 = 16 * jb + 2 * (lane & 3);
#pragma unroll
          for (int k = 0; k < 2; ++k) {   // 8 rows
            const int r = r0 + 8 * k;
            unsigned long long wt = *reinterpret_cast<const unsigned long long*>(s_c + r);
            if (n < C) {
              const int d = P.reverse ? 0 : C - n;
              wt = pack2(r < n ? s_c[r + d] : 0.0f, r + 1 < n ? s_c[r + 1 + d] : 0.0f);
              const uint32_t keep = (r < n ? 0xffffu : 0u) | (r + 1 < n ? 0xffff0000u : 0u);
              v[2 * k] &= keep;
              v[2 * k + 1] &= keep;
            }
#pragma unroll
            for (int i = 2 * k; i < 2 * k + 2; ++i) X::pieces(wt, v[i], o[0][i], o[1][i], o[2][i]);
          }
#pragma unroll
          for (int p = 0; p < 3; ++p) tmem_st_frag4(to_tmem + (uint32_t)(32 * K::NP * (m & 1) + 32 * p + 8 * jb), o[p]);
        }
        tmem_st_wait();
        tc_fence_before();
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int r = (t >> 3) + 32 * k;
          const float wk = r < n ? s_c[P.reverse ? r : r + C - n] : 0.0f;
#pragma unroll
          for (int x = 0; x < DC / 64; ++x) {
            const uint4 c = *reinterpret_cast<const uint4*>(src + x * K::SUB + (t + 256 * k) * 16);
            const uint32_t cu[4] = {c.x, c.y, c.z, c.w};
            uint32_t o[3][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) X::pieces(pack2(wk, wk), cu[i], o[0][i], o[1][i], o[2][i]);
            unsigned char* to = base + K::OFF_CP + K::NP * (m & 1) * K::C_BYTES + x * K::SUB + (t + 256 * k) * 16;
#pragma unroll
            for (int p = 0; p < 3; ++p)
              *reinterpret_cast<uint4*>(to + p * K::C_BYTES) = make_uint4(o[p][0], o[p][1], o[p][2], o[p][3]);
          }
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_cp[m & 1]);
    }
  }

  // every copy and product of this CTA ends before it gives up TMEM and shared memory
  __syncwarp();
  if (warp == 0 && lane == 0) {
    const int n = s_loaded;
    for (int m = n > NS ? n - NS : 0; m < n; ++m) lin_drain(&bar_full[m % NS], (unsigned)(m / NS) & 1u);
  }
  if (warp >= 1 && warp <= 3) {
    if (elect_one()) umma_commit(&bar_done[warp - 1]);
    lin_drain(&bar_done[warp - 1], 0u);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, (uint32_t)K::TCOLS);
}

}  // namespace pn
