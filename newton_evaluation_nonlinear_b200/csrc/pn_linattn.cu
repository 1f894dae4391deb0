// pn_linattn.cu -- entry points of linear attention with a decay for each head.
#include <algorithm>
#include <cmath>
#include <memory>
#include <mutex>
#include <vector>

#include "pn_linattn_tc.cuh"

namespace pn {
CUresult encode_tensor_map(CUtensorMap* m, CUtensorMapDataType type, unsigned rank, const void* base, const cuuint64_t* dims,
                           const cuuint64_t* strides, const cuuint32_t* box);   // pn_api.cu
namespace {

pn_status check_op(const pn_heads* x, const char* name, size_t es, int* dev, bool empty) {
  if (!x) return seq_fail(PN_ERR_INVALID, "%s is NULL", name);
  if (x->batch_stride < 0 || x->token_stride < 0 || x->head_stride < 0)
    return seq_fail(PN_ERR_INVALID, "%s has a negative stride", name);
  if (empty) return PN_OK;
  if (pn_status e = seq_device(x->data, name, dev)) return e;
  if ((uintptr_t)x->data % es) return seq_fail(PN_ERR_INVALID, "%s is misaligned", name);
  return PN_OK;
}

pn_status check_f32(const void* p, const char* name, int* dev) {
  if (!p) return PN_OK;
  if (pn_status e = seq_device(p, name, dev)) return e;
  if ((uintptr_t)p & 15u) return seq_fail(PN_ERR_INVALID, "%s must be 16-byte aligned", name);
  return PN_OK;
}

LinOperand operand(const pn_heads* x, int per) {
  return LinOperand{x->data, x->batch_stride, x->token_stride, x->head_stride, per};
}

// Rows of one chunk of the kernels for any type and width.
int mma_chunk(int da) { return da <= 128 ? 64 : 32; }

// Parts a sequence is cut into there: as many as fit the card beside each other (two CTAs on an SM up to width 64).  A part's
// state alone takes a third of its outputs' time, so parts of one chunk pay where SMs are idle (float32, 8 heads of width 64,
// 512 rows: 20 us, 54 in parts of four); where a second CTA on an SM is all there is to win, which is little, parts have four chunks.
int mma_parts(const pn_linattn_s* h, int n_seq, long long max_len, int da, int dc) {
  const long long ctas = std::max(1LL, (long long)n_seq * h->H * ((dc + kLinDC - 1) / kLinDC));
  const long long want = 148 * (da <= 64 ? 2 : 1) / ctas;
  return (int)std::max(1LL, std::min(want, max_len / (mma_chunk(da) * (2 * ctas <= 148 ? 1 : 4))));
}

// Whether the tensor-core kernel is for a pass of that many rows (of all sequences) and widths da.  Its rounding of the weights
// between rows to bfloat16 is one relative error for a whole row, 2^-8 at most: of many rows it averages out (outputs are 1.42
// times as far off as by their own rounding), of a few it is the outputs' error (up to 2.0 times below 64 rows and heads, 1.53 from
// there on, in thousands of drawn calls).  The other kernel then takes 7.5 to 8.4 us in place of 6.8 at width 64, 11 to 12 in place of 8.6 at 128.
bool tc_takes(const pn_linattn_s* h, long long rows, int da) {
  return h->dtype == PN_BF16 && da <= 128 && rows > 0 && rows * h->H >= 64;
}

// Columns of c that one CTA of the tensor-core kernel takes: 64 where 128 leave SMs idle (a and b are then read twice, out of
// L2, which costs less than a second part).
int tc_columns(const pn_linattn_s* h, int n_seq, int dc) {
  return dc <= 64 || (long long)n_seq * h->H * ((dc + 63) / 64) <= 148 ? 64 : 128;
}

// Parts for the tensor-core kernel: a CTA fills its SM, so as many as fit the card beside each other, of four chunks at least.
// A part's state alone takes three quarters of its outputs' time, and the two launches more take that of 10 chunks or so, so p
// parts of n chunks pay from n (1 - 1.75 / p) = 10 on (32 heads of width 128, 1024 rows: 25 us whole, 34 in two parts; 2 heads
// of width 64, 2048 rows: 19 us in eight parts, 24 in four).
int tc_parts(const pn_linattn_s* h, int n_seq, long long max_len, int dc) {
  const int w = tc_columns(h, n_seq, dc);
  const long long ctas = std::max(1LL, (long long)n_seq * h->H * ((dc + w - 1) / w));
  const long long n = (max_len + 63) / 64, p = std::min(148 / ctas, max_len / (4 * 64));
  return p > 1 && 4 * n * p - 7 * n >= 40 * p ? (int)p : 1;
}

// Whether a ragged batch takes its longest sequences first: where the longest one is a quarter or more of what an SM takes of
// all rows (w columns of c to a CTA), so that it must not start last.  With more and shorter ones the order is all the same, and
// finding it costs every CTA a microsecond.  Heads of width 128: 16 sequences of 300 to 3800 rows x 32 heads 217 us, 240 in the
// given order; 64 of 10 to 1000 rows 325 and 305; 512 of 10 to 200 rows 1377 and 1204.
bool tc_by_length(const pn_linattn_s* h, const LinPass& P, long long max_len, int w) {
  return P.cu && P.n_seq > 1 && P.n_seq <= kLinSorted && max_len * 4 * 148 >= P.T * h->H * ((P.dc + w - 1) / w);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

size_t seg_bytes(const pn_linattn_s* h, int n_seq, long long max_len) {
  // the largest of what either kernel takes in either direction (which one runs goes by the arrays' alignment)
  int p = 1;
  for (int t = 0; t < 2; ++t) {
    const int da = t ? h->dv : h->dk, dc = t ? h->dk : h->dv;
    p = std::max(p, std::max(mma_parts(h, n_seq, max_len, da, dc), tc_parts(h, n_seq, max_len, dc)));
  }
  return p > 1 ? align256((size_t)n_seq * h->H * p * h->dk * h->dv * sizeof(float)) : 0;
}

template <typename T, int C, int DA>
cudaError_t launch_mma(const LinPass& P, const LinDecay& G, cudaStream_t st) {
  using K = LinMmaCfg<T, C, DA>;
  const dim3 grid((P.dc + kLinDC - 1) / kLinDC, P.nseg, P.n_seq * P.H);
  cudaError_t e;
  if (P.nseg > 1) {
    if ((e = cudaFuncSetAttribute(lin_mma_kernel<T, C, DA, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  K::SMEM_BYTES)) != cudaSuccess)
      return e;
    lin_mma_kernel<T, C, DA, true><<<dim3(grid.x, P.nseg - 1, grid.z), K::NT, K::SMEM_BYTES, st>>>(P, G);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    lin_combine_kernel<<<dim3((P.da * P.dc + 511) / 512, P.n_seq * P.H), 128, 0, st>>>(P, G, C, 0);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if ((e = cudaFuncSetAttribute(lin_mma_kernel<T, C, DA, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                K::SMEM_BYTES)) != cudaSuccess)
    return e;
  lin_mma_kernel<T, C, DA, false><<<grid, K::NT, K::SMEM_BYTES, st>>>(P, G);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_pass(const LinPass& P, const LinDecay& G, cudaStream_t st) {
  if (P.da <= 64) return launch_mma<T, 64, 64>(P, G, st);
  if (P.da <= 128) return launch_mma<T, 64, 128>(P, G, st);
  return launch_mma<T, 32, 256>(P, G, st);
}

// The tensor map of one operand: boxes of 64 rows x 64 columns of one head, 128-byte swizzled.
// False where TMA cannot read it (alignment, strides).
bool encode_operand(CUtensorMap* m, const LinOperand& x, int width, int heads, long long T, int batch) {
  if ((uintptr_t)x.p & 15u) return false;
  const cuuint64_t row = ((cuuint64_t)width * 2 + 15) / 16 * 16;
  cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)batch};
  const long long es[3] = {x.hs, x.ts, x.bs};
  cuuint64_t strides[3];
  for (int i = 0; i < 3; ++i) {
    const bool one = dims[i + 1] == 1;   // a stride that is never taken
    if (!one && (es[i] <= 0 || es[i] % 8 || es[i] * 2 >= (1LL << 40))) return false;
    strides[i] = one ? row : (cuuint64_t)es[i] * 2;
  }
  const cuuint32_t box[4] = {64, 1, 64, 1};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, x.p, dims, strides, box) == CUDA_SUCCESS;
}

template <typename T, int DA, int DC, int WHAT>
cudaError_t launch_tc_kernel(const LinMaps& maps, const LinPass& P, const LinDecay& G, unsigned parts, cudaStream_t st) {
  using K = LinTcCfg<DA, DC>;
  const cudaError_t e = cudaFuncSetAttribute(lin_tc_kernel<T, DA, DC, WHAT>, cudaFuncAttributeMaxDynamicSharedMemorySize, K::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  lin_tc_kernel<T, DA, DC, WHAT><<<dim3((P.dc + DC - 1) / DC, P.n_seq * P.H, parts), K::NT, K::SMEM_BYTES, st>>>(maps, P, G);
  return cudaGetLastError();
}

template <typename T, int DA, int DC>
cudaError_t launch_tc(const LinMaps& maps, const LinPass& P, const LinDecay& G, cudaStream_t st) {
  if (P.nseg > 1) {
    cudaError_t e = launch_tc_kernel<T, DA, DC, kLinStateOnly>(maps, P, G, P.nseg - 1, st);
    if (e != cudaSuccess) return e;
    lin_combine_kernel<<<dim3((P.da * P.dc + 511) / 512, P.n_seq * P.H), 128, 0, st>>>(P, G, LinTcCfg<DA, DC>::C, 1);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return P.out_f32 ? launch_tc_kernel<T, DA, DC, kLinOutF32>(maps, P, G, P.nseg, st)
                   : launch_tc_kernel<T, DA, DC, kLinOut>(maps, P, G, P.nseg, st);
}

// The tensor-core kernel, where it can take the pass; false where the other one has to.
bool try_tc(const pn_linattn_s* h, LinPass& P, const LinDecay& G, long long max_len, cudaStream_t st, cudaError_t* e) {
  if (!tc_takes(h, P.cu ? P.T : P.n_seq * P.T, P.da)) return false;
  LinMaps maps;
  const int batch = P.cu ? 1 : P.n_seq;
  if (!encode_operand(&maps.a, P.a, P.da, P.H / P.a.per, P.T, batch) ||
      !encode_operand(&maps.b, P.b, P.da, P.H / P.b.per, P.T, batch) ||
      !encode_operand(&maps.c, P.c, P.dc, P.H / P.c.per, P.T, batch))
    return false;
  P.out_map = !P.out_f32 && encode_operand(&maps.o, LinOperand{P.out, P.out_bs, P.out_ts, P.out_hs, 1}, P.dc, P.H, P.T, batch);
  P.nseg = tc_parts(h, P.n_seq, max_len, P.dc);
  using T = __nv_bfloat16;
  const bool narrow = tc_columns(h, P.n_seq, P.dc) == 64;
  P.wait_ns = h->wait_ns;
  P.stall = h->stall;
  P.by_length = tc_by_length(h, P, max_len, narrow ? 64 : 128);
  if (P.da <= 64) *e = narrow ? launch_tc<T, 64, 64>(maps, P, G, st) : launch_tc<T, 64, 128>(maps, P, G, st);
  else *e = narrow ? launch_tc<T, 128, 64>(maps, P, G, st) : launch_tc<T, 128, 128>(maps, P, G, st);
  return true;
}

// One pass over every sequence and head.
cudaError_t run_pass(const pn_linattn_s* h, LinPass P, int n_seq, long long max_len, void* seg, cudaStream_t st) {
  LinDecay G;
  std::copy(h->log2_decay, h->log2_decay + h->H, G.log2);
  P.H = h->H;
  P.n_seq = n_seq;
  P.seg_state = (float*)seg;
  cudaError_t e;
  if (try_tc(h, P, G, max_len, st, &e)) return e;
  P.nseg = mma_parts(h, n_seq, max_len, P.da, P.dc);
  auto aligned = [](const void* p, long long bs, long long ts, long long hs, size_t es) {
    return (uintptr_t)p % (4 * es) == 0 && bs % 4 == 0 && ts % 4 == 0 && hs % 4 == 0;
  };
  const size_t es = dtype_size(h->dtype);
  P.vec = aligned(P.out, P.out_bs, P.out_ts, P.out_hs, P.out_f32 ? 4 : es);
  for (const LinOperand* x : {&P.a, &P.b, &P.c}) P.vec = P.vec && aligned(x->p, x->bs, x->ts, x->hs, es);
  switch (h->dtype) {
    case PN_F32: return launch_pass<float>(P, G, st);
    case PN_BF16: return launch_pass<__nv_bfloat16>(P, G, st);
    default: return launch_pass<__half>(P, G, st);
  }
}

template <typename T>
cudaError_t group_sum(const float* part, long long rows, int H, int G, int d, const pn_heads* dst, long long tokens,
                      const int* cu, int n_seq, cudaStream_t st) {
  // (sequences differ in length: more and shorter shares than CTAs that run at once)
  const dim3 grid((unsigned)std::min<long long>(rows, cu ? (148LL * 64 + n_seq - 1) / n_seq : 148LL * 16), cu ? n_seq : 1);
  const bool vec = (uintptr_t)dst->data % (4 * sizeof(T)) == 0 && dst->batch_stride % 4 == 0 && dst->token_stride % 4 == 0 &&
                   dst->head_stride % 4 == 0;
  lin_group_sum_kernel<T><<<grid, 256, 0, st>>>(part, rows, H, G, d, (T*)dst->data, dst->batch_stride, dst->token_stride,
                                               dst->head_stride, tokens, cu, vec);
  return cudaGetLastError();
}

struct Shape {
  long long rows;      // of the buffers
  long long tokens;    // rows of a batch entry (ragged: all rows)
  long long max_len;
};

pn_status check_shape(const pn_linattn_s* h, int n_seq, long long T, const int* cu, long long max_len, Shape* s) {
  if (!h) return seq_fail(PN_ERR_INVALID, "handle is NULL");
  if (n_seq < 0 || T < 0) return seq_fail(PN_ERR_INVALID, "bad shape n_seq=%d T=%lld", n_seq, T);
  if (T > 0x7fffff00LL) return seq_fail(PN_ERR_INVALID, "T=%lld: at most 2^31 - 256 rows", T);
  if ((long long)n_seq * h->H > 65535) return seq_fail(PN_ERR_INVALID, "n_seq * heads = %lld: at most 65535", (long long)n_seq * h->H);
  if (max_len < 0) return seq_fail(PN_ERR_INVALID, "max_len must be >= 0");
  s->rows = cu ? T : n_seq * T;
  s->tokens = T;
  s->max_len = cu ? (max_len > 0 ? std::min(max_len, T) : T) : T;
  return PN_OK;
}

}  // namespace
}  // namespace pn

using namespace pn;

extern "C" {

pn_status pn_linattn_create(pn_linattn* out, int H, int Hkv, int dk, int dv, int dtype, const float* log_decay, float scale) {
  if (!out) return seq_fail(PN_ERR_INVALID, "out is NULL");
  *out = nullptr;
  if (H < 1 || H > kMaxLinHeads) return seq_fail(PN_ERR_INVALID, "H=%d: from 1 to %d", H, kMaxLinHeads);
  if (Hkv < 1 || H % Hkv) return seq_fail(PN_ERR_INVALID, "Hkv=%d does not divide H=%d", Hkv, H);
  for (int d : {dk, dv})
    if (d < 8 || d > 256 || d % 8) return seq_fail(PN_ERR_INVALID, "dk=%d dv=%d: multiples of 8 from 8 to 256", dk, dv);
  if (dtype != PN_F32 && dtype != PN_BF16 && dtype != PN_F16) return seq_fail(PN_ERR_INVALID, "unknown dtype %d", dtype);
  if (!log_decay) return seq_fail(PN_ERR_INVALID, "log_decay is NULL");
  if (!std::isfinite(scale)) return seq_fail(PN_ERR_INVALID, "scale must be finite");
  for (int i = 0; i < H; ++i)
    if (!std::isfinite(log_decay[i]) || log_decay[i] > 0.0f)
      return seq_fail(PN_ERR_INVALID, "log_decay[%d]=%g: finite and <= 0", i, (double)log_decay[i]);
  pn_linattn_s* h = new (std::nothrow) pn_linattn_s();
  if (!h) return seq_fail(PN_ERR_NOMEM, "out of host memory");
  h->H = H;
  h->Hkv = Hkv;
  h->dk = dk;
  h->dv = dv;
  h->dtype = dtype;
  h->scale = scale;
  h->wait_ns = kLinWaitNs;
  h->stall = -1;
  // (2^-1e30 is zero as well, and its multiples by zero are zero: an infinite exponent's are not)
  for (int i = 0; i < H; ++i) h->log2_decay[i] = (float)std::max((double)log_decay[i] * 1.4426950408889634074, -1e30);
  *out = h;
  return PN_OK;
}

void pn_linattn_destroy(pn_linattn h) { delete h; }

size_t pn_linattn_workspace(pn_linattn h, int backward, int n_seq, long long T, int ragged, long long max_len) {
  if (!h || n_seq < 1 || T < 1) return 0;
  const long long len = ragged && max_len > 0 ? std::min(max_len, T) : T;
  size_t n = seg_bytes(h, n_seq, len);
  if (backward && h->H > h->Hkv)
    n += align256((size_t)(ragged ? T : n_seq * T) * h->H * std::max(h->dk, h->dv) * sizeof(float));
  return n;
}

pn_status pn_linattn_split(pn_linattn h, int pass, int n_seq, long long T, int ragged, long long max_len, int* columns, int* parts) {
  if (!h || !columns || !parts) return seq_fail(PN_ERR_INVALID, "handle, columns or parts is NULL");
  if (pass < 0 || pass > 3) return seq_fail(PN_ERR_INVALID, "pass=%d: from 0 to 3", pass);
  Shape s;
  static const int some = 0;
  if (pn_status e = check_shape(h, n_seq, T, ragged ? &some : nullptr, max_len, &s)) return e;
  const int da = pass == 0 || pass == 3 ? h->dk : h->dv, dc = pass == 0 || pass == 3 ? h->dv : h->dk;
  const bool tc = tc_takes(h, s.rows, da);
  *columns = tc ? tc_columns(h, n_seq, dc) : 0;
  *parts = tc ? tc_parts(h, n_seq, s.max_len, dc) : mma_parts(h, n_seq, s.max_len, da, dc);
  return PN_OK;
}

pn_status pn_linattn_forward(pn_linattn h, int n_seq, long long T, const int* cu_seqlens, long long max_len,
                             const pn_heads* q, const pn_heads* k, const pn_heads* v, const float* initial_state,
                             const pn_heads* o, float* final_state, void* workspace, size_t workspace_bytes,
                             void* cuda_stream) {
  Shape s;
  if (pn_status e = check_shape(h, n_seq, T, cu_seqlens, max_len, &s)) return e;
  int dev = -1;
  const size_t es = dtype_size(h->dtype);
  const bool empty = s.rows == 0;
  const pn_heads* ops[] = {q, k, v, o};
  const char* names[] = {"q", "k", "v", "o"};
  for (int i = 0; i < 4; ++i)
    if (pn_status e = check_op(ops[i], names[i], es, &dev, empty)) return e;
  if (pn_status e = check_f32(initial_state, "initial_state", &dev)) return e;
  if (pn_status e = check_f32(final_state, "final_state", &dev)) return e;
  if (cu_seqlens)
    if (pn_status e = seq_device(cu_seqlens, "cu_seqlens", &dev)) return e;
  if (!empty) {
    if (pn_status e = seq_output(o, "o", cu_seqlens ? 1 : n_seq, T, h->H, h->dv)) return e;
    for (int i = 0; i < 3; ++i)
      if (pn_status e = seq_apart(o->data, "o", ops[i]->data, names[i])) return e;
  }
  if (n_seq == 0 || (empty && !final_state)) return PN_OK;
  const size_t need = pn_linattn_workspace(h, 0, n_seq, T, cu_seqlens != nullptr, max_len);
  if (workspace_bytes < need) return seq_fail(PN_ERR_INVALID, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (need)
    if (pn_status e = check_f32(workspace, "workspace", &dev)) return e;
  if (need && !workspace) return seq_fail(PN_ERR_INVALID, "workspace is NULL");
  SeqDeviceGuard dg(dev);
  const int G = h->H / h->Hkv;
  LinPass P = {};
  P.a = operand(q, 1);
  P.b = operand(k, G);
  P.c = operand(v, G);
  P.out = o->data;
  P.out_bs = o->batch_stride;
  P.out_ts = o->token_stride;
  P.out_hs = o->head_stride;
  P.da = h->dk;
  P.dc = h->dv;
  P.T = T;
  P.cu = cu_seqlens;
  P.alpha = 1.0f;
  P.beta = h->scale;
  P.s_in = initial_state;
  P.s_out = final_state;
  P.s_row = h->dv;
  P.s_col = 1;
  const cudaError_t e = run_pass(h, P, n_seq, s.max_len, workspace, (cudaStream_t)cuda_stream);
  if (e != cudaSuccess) return seq_fail(PN_ERR_CUDA, "launch failed: %s", cudaGetErrorString(e));
  return PN_OK;
}

pn_status pn_linattn_backward(pn_linattn h, int n_seq, long long T, const int* cu_seqlens, long long max_len,
                              const pn_heads* d_o, const pn_heads* q, const pn_heads* k, const pn_heads* v,
                              const float* initial_state, const float* d_final_state, const pn_heads* dq,
                              const pn_heads* dk, const pn_heads* dv, float* d_initial_state, void* workspace,
                              size_t workspace_bytes, void* cuda_stream) {
  Shape s;
  if (pn_status e = check_shape(h, n_seq, T, cu_seqlens, max_len, &s)) return e;
  int dev = -1;
  const size_t es = dtype_size(h->dtype);
  const bool empty = s.rows == 0;
  const pn_heads* ops[] = {d_o, q, k, v, dq, dk, dv};
  const char* names[] = {"d_o", "q", "k", "v", "dq", "dk", "dv"};
  for (int i = 0; i < 7; ++i)
    if (pn_status e = check_op(ops[i], names[i], es, &dev, empty)) return e;
  if (pn_status e = check_f32(initial_state, "initial_state", &dev)) return e;
  if (pn_status e = check_f32(d_final_state, "d_final_state", &dev)) return e;
  if (pn_status e = check_f32(d_initial_state, "d_initial_state", &dev)) return e;
  if (cu_seqlens)
    if (pn_status e = seq_device(cu_seqlens, "cu_seqlens", &dev)) return e;
  for (int o = 4; o < 7 && !empty; ++o) {
    if (pn_status e = seq_output(ops[o], names[o], cu_seqlens ? 1 : n_seq, T, o == 4 ? h->H : h->Hkv, o == 6 ? h->dv : h->dk)) return e;
    for (int i = 0; i < o; ++i)
      if (pn_status e = seq_apart(ops[o]->data, names[o], ops[i]->data, names[i])) return e;
  }
  if (n_seq == 0 || (empty && !d_initial_state)) return PN_OK;
  const size_t need = pn_linattn_workspace(h, 1, n_seq, T, cu_seqlens != nullptr, max_len);
  if (workspace_bytes < need) return seq_fail(PN_ERR_INVALID, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (need)
    if (pn_status e = check_f32(workspace, "workspace", &dev)) return e;
  if (need && !workspace) return seq_fail(PN_ERR_INVALID, "workspace is NULL");
  SeqDeviceGuard dg(dev);
  cudaStream_t st = (cudaStream_t)cuda_stream;
  const int G = h->H / h->Hkv;
  float* part = G > 1 ? (float*)((char*)workspace + seg_bytes(h, n_seq, s.max_len)) : nullptr;
  cudaError_t e = cudaSuccess;

  LinPass P = {};
  P.T = T;
  P.cu = cu_seqlens;
  if (!empty) {
    // dq_t = scale S_t do_t
    P.a = operand(d_o, 1);
    P.b = operand(v, G);
    P.c = operand(k, G);
    P.out = dq->data;
    P.out_bs = dq->batch_stride;
    P.out_ts = dq->token_stride;
    P.out_hs = dq->head_stride;
    P.da = h->dv;
    P.dc = h->dk;
    P.alpha = 1.0f;
    P.beta = h->scale;
    P.s_in = initial_state;
    P.s_row = 1;
    P.s_col = h->dv;
    e = run_pass(h, P, n_seq, s.max_len, workspace, st);
  }
  // against time, G_t = scale q_t do_t^T + e^g G_{t+1}: dk_t = G_t v_t, dv_t = G_t^T k_t, dS_0 = e^g G_1
  P.reverse = 1;
  P.alpha = h->scale;
  P.beta = 1.0f;
  P.s_in = d_final_state;
  P.out_f32 = G > 1;
  for (int which = 0; which < 2 && e == cudaSuccess; ++which) {
    const pn_heads* dst = which ? dv : dk;
    const int d = which ? h->dv : h->dk;
    if (which == 0 && empty) continue;
    P.a = operand(which ? k : v, G);
    P.b = which ? operand(q, 1) : operand(d_o, 1);
    P.c = which ? operand(d_o, 1) : operand(q, 1);
    P.da = which ? h->dk : h->dv;
    P.dc = which ? h->dv : h->dk;
    P.s_row = which ? h->dv : 1;
    P.s_col = which ? 1 : h->dv;
    P.s_out = which ? d_initial_state : nullptr;
    P.out = G > 1 ? part : dst->data;
    P.out_bs = G > 1 ? T * h->H * d : dst->batch_stride;
    P.out_ts = G > 1 ? (long long)h->H * d : dst->token_stride;
    P.out_hs = G > 1 ? d : dst->head_stride;
    e = run_pass(h, P, n_seq, s.max_len, workspace, st);
    if (G > 1 && e == cudaSuccess && !empty) {
      e = h->dtype == PN_F32    ? group_sum<float>(part, s.rows, h->H, G, d, dst, T, cu_seqlens, n_seq, st)
          : h->dtype == PN_BF16 ? group_sum<__nv_bfloat16>(part, s.rows, h->H, G, d, dst, T, cu_seqlens, n_seq, st)
                                : group_sum<__half>(part, s.rows, h->H, G, d, dst, T, cu_seqlens, n_seq, st);
    }
  }
  if (e != cudaSuccess) return seq_fail(PN_ERR_CUDA, "launch failed: %s", cudaGetErrorString(e));
  return PN_OK;
}

pn_status pn_linattn_debug_waits(pn_linattn h, long long timeout_ns, int stall_chunk) {
  if (!h) return seq_fail(PN_ERR_INVALID, "handle is NULL");
  if (timeout_ns < 1000 || timeout_ns > 4000000000LL) return seq_fail(PN_ERR_INVALID, "timeout: from 1000 to 4e9 ns");
  if (stall_chunk < -1) return seq_fail(PN_ERR_INVALID, "stall_chunk must be >= -1");
  h->wait_ns = (unsigned)timeout_ns;
  h->stall = stall_chunk;
  return PN_OK;
}

pn_status pn_linattn_check(void* cuda_stream) {
  // what each stream has been told of so far
  struct Told {
    int dev;
    void* stream;
    unsigned count;
  };
  static std::mutex lock;
  static std::vector<Told> told;
  cudaStream_t st = (cudaStream_t)cuda_stream;
  unsigned count = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbolAsync(&count, lin_gave_up, sizeof count, 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return seq_fail(PN_ERR_CUDA, "reading the device's count of waits failed: %s", cudaGetErrorString(e));
  unsigned before = 0;
  try {
    std::lock_guard<std::mutex> g(lock);
    auto it = std::find_if(told.begin(), told.end(), [&](const Told& t) { return t.dev == dev && t.stream == cuda_stream; });
    if (it == told.end()) it = told.insert(told.end(), Told{dev, cuda_stream, 0u});
    before = it->count;
    // (a check of this stream in another thread may have read a later count)
    if ((int)(count - before) > 0) it->count = count;
  } catch (...) {
    return seq_fail(PN_ERR_NOMEM, "out of host memory");
  }
  if ((int)(count - before) > 0)
    return seq_fail(PN_ERR_TIMEOUT, "a device wait of linear attention gave up: results since the last check are invalid");
  return PN_OK;
}

pn_status pn_linattn_step(pn_linattn h, int rows, const pn_heads* q, const pn_heads* k, const pn_heads* v, const pn_heads* o,
                          float* states, long long n_slots, const long long* slots, pn_rotary r, const long long* positions,
                          const void* wq, const void* wk, int w_dtype, float eps, void* cuda_stream) {
  if (!h) return seq_fail(PN_ERR_INVALID, "handle is NULL");
  if (rows < 0 || rows > 65535) return seq_fail(PN_ERR_INVALID, "rows=%d: from 0 to 65535", rows);
  if (n_slots < 0) return seq_fail(PN_ERR_INVALID, "n_slots must be >= 0");
  if (!slots && rows > n_slots) return seq_fail(PN_ERR_INVALID, "rows=%d exceeds n_slots=%lld", rows, n_slots);
  if ((wq == nullptr) != (wk == nullptr)) return seq_fail(PN_ERR_INVALID, "wq and wk come together");
  if (wq && w_dtype != PN_F32 && w_dtype != h->dtype) return seq_fail(PN_ERR_INVALID, "weights: float32 or the tensors' type");
  if (wq && (!(eps >= 0.0f) || !std::isfinite(eps))) return seq_fail(PN_ERR_INVALID, "eps must be finite and >= 0");
  if (r && 2 * r->pairs > h->dk) return seq_fail(PN_ERR_INVALID, "rot_dim=%d exceeds dk=%d", 2 * r->pairs, h->dk);
  int dev = -1;
  const size_t es = dtype_size(h->dtype);
  const pn_heads* ops[] = {q, k, v, o};
  const char* names[] = {"q", "k", "v", "o"};
  for (int i = 0; i < 4; ++i)
    if (pn_status e = check_op(ops[i], names[i], es, &dev, rows == 0)) return e;
  if (rows == 0 || n_slots == 0) return PN_OK;
  if (!states) return seq_fail(PN_ERR_INVALID, "states is NULL");
  if (pn_status e = check_f32(states, "states", &dev)) return e;
  if (slots)
    if (pn_status e = seq_device(slots, "slots", &dev)) return e;
  if (r)
    if (pn_status e = seq_device(positions, "positions", &dev)) return e;
  if (wq) {
    if (pn_status e = seq_device(wq, "wq", &dev)) return e;
    if (pn_status e = seq_device(wk, "wk", &dev)) return e;
  }
  if (pn_status e = seq_output(o, "o", rows, 1, h->H, h->dv)) return e;
  for (int i = 0; i < 3; ++i)
    if (pn_status e = seq_apart(o->data, "o", ops[i]->data, names[i])) return e;
  if (pn_status e = seq_apart(o->data, "o", states, "states")) return e;
  SeqDeviceGuard dg(dev);
  const int G = h->H / h->Hkv;
  LinStep P = {};
  P.q = operand(q, 1);
  P.k = operand(k, G);
  P.v = operand(v, G);
  P.o = o->data;
  P.o_bs = o->batch_stride;
  P.o_hs = o->head_stride;
  P.H = h->H;
  P.dk = h->dk;
  P.dv = h->dv;
  P.scale = h->scale;
  P.states = states;
  P.n_slots = n_slots;
  P.slots = slots;
  P.positions = positions;
  P.wq = wq;
  P.wk = wk;
  P.w_f32 = w_dtype == PN_F32;
  P.eps = eps;
  if (r) {
    P.pairs = r->pairs;
    P.interleaved = r->interleaved;
    P.m = r->factor;
    std::copy(r->turn, r->turn + r->pairs, P.turn);
  }
  LinDecay D;
  std::copy(h->log2_decay, h->log2_decay + h->H, D.log2);
  cudaStream_t st = (cudaStream_t)cuda_stream;
  // narrow columns (32) while that many CTAs fit the card at once, else 128 columns
  const bool narrow = (long long)rows * h->H * ((h->dv + 31) / 32) <= 148 * 4;
  const int w = narrow ? 32 : 128;
  const dim3 grid((h->dv + w - 1) / w, h->H, rows);
  auto go = [&](auto tag) {
    using T = decltype(tag);
    if (narrow) lin_step_kernel<T, 8><<<grid, kStepThreads, 0, st>>>(P, D);
    else lin_step_kernel<T, 32><<<grid, kStepThreads, 0, st>>>(P, D);
    return cudaGetLastError();
  };
  const cudaError_t e = h->dtype == PN_F32 ? go(float{}) : h->dtype == PN_BF16 ? go(__nv_bfloat16{}) : go(__half{});
  if (e != cudaSuccess) return seq_fail(PN_ERR_CUDA, "launch failed: %s", cudaGetErrorString(e));
  return PN_OK;
}

}  // extern "C"
