// C ABI of the TwELL FFN library: argument validation, then launches on the caller's stream.
// Declarations, layouts and error contract: include/twell.h.
#include <string.h>

#include <algorithm>
#include <mutex>
#include <new>

#include "../../include/twell.h"
#include "launch.h"

using namespace tw;

// Device scratch of twell_ffn_bwd_noalloc, for callers that cannot allocate: one copy per GPU
// (at its own address on each), held for the life of the process. In host code `scratch`
// names a host-side stand-in, not device memory: only the address hipGetSymbolAddress returns
// for the current device may be handed to kernels.
static __device__ __align__(256) char scratch[TWELL_NOALLOC_SCRATCH_BYTES];

namespace {

constexpr int kMaxDevices = 64;
std::mutex scratch_mu;
void *scratch_ptr[kMaxDevices];

// The current device's address of `scratch` (looked up once per device), or NULL on error.
void *scratch_on_current_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(scratch_mu);
  if (!scratch_ptr[dev]) {
    void *p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return nullptr;
    scratch_ptr[dev] = p;
  }
  return scratch_ptr[dev];
}

}  // namespace

namespace {

inline bool al16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline bool al4(const void *p) { return ((uintptr_t)p & 3u) == 0; }
inline bool dtype_ok(int32_t t) { return t == TWELL_F32 || t == TWELL_BF16; }
inline hipStream_t S(void *s) { return (hipStream_t)s; }
inline int hip_status(hipError_t e) { return e == hipSuccess ? TWELL_OK : TWELL_ERR_HIP; }

#define TW_TRY(expr)                               \
  do {                                             \
    hipError_t e_ = (expr);                        \
    if (e_ != hipSuccess) return TWELL_ERR_HIP;    \
  } while (0)

// A TwELL whose single tile spans the row: the compact row-ELL of the hybrid format.
inline bool is_row_ell(const twell_matrix_t *m) { return m->tile_w == m->cols && m->tile_w != 64 && m->tile_w != 128; }

// Shape and pointer checks of a TwELL struct used as output (writable) or input. row_ell:
// the consumer also takes the row-ELL form (tile_w == cols, 1 <= slots <= cols <= 16384).
int check_matrix(const twell_matrix_t *m, bool need_ovf_bits, bool need_rows = false, bool row_ell = false) {
  if (!m) return TWELL_ERR_ARG;
  if (!dtype_ok(m->val_dtype)) return TWELL_ERR_ARG;
  if (m->rows < 0 || m->cols <= 0 || m->ovf_cap < 0) return TWELL_ERR_SHAPE;
  if (row_ell && is_row_ell(m)) {
    if (m->cols > 16384) return TWELL_ERR_UNSUPPORTED;
    if (m->slots < 1 || m->slots > m->cols) return TWELL_ERR_SHAPE;
  } else {
    if (m->tile_w != 64 && m->tile_w != 128) return TWELL_ERR_UNSUPPORTED;
    if (m->cols % m->tile_w) return TWELL_ERR_SHAPE;
    if (m->slots < 1 || m->slots > m->tile_w || m->slots > 64) return TWELL_ERR_SHAPE;
  }
  if (!m->ovf_n) return TWELL_ERR_ARG;
  if (m->rows > 0) {
    if (!m->counts || !m->col_idx || !m->vals || !m->ovf_slot) return TWELL_ERR_ARG;
    if (need_ovf_bits && !m->ovf_bits) return TWELL_ERR_ARG;
    if (need_rows && (!m->row_nnz || !m->row_list)) return TWELL_ERR_ARG;
  }
  if (m->ovf_cap > 0 && (!m->ovf_rows || !m->ovf_dense)) return TWELL_ERR_ARG;
  if (!al4(m->counts) || !al4(m->col_idx) || !al4(m->vals) || !al4(m->ovf_n) || !al4(m->ovf_rows) ||
      !al4(m->ovf_slot) || !al4(m->ovf_bits) || !al16(m->ovf_dense) || !al4(m->row_nnz) || !al16(m->row_list))
    return TWELL_ERR_ALIGN;
  return TWELL_OK;
}

size_t list_bytes(int32_t rows, int32_t cols, int32_t tile_w, int32_t slots) {
  return (size_t)rows * (size_t)(cols / tile_w) * (size_t)slots * 8;
}

TwellOut out_of(const twell_matrix_t *m) {
  TwellOut o;
  o.counts = m->counts;
  o.col_idx = m->col_idx;
  o.vals = m->vals;
  o.ovf_bits = m->ovf_bits;
  o.dec_part = nullptr;
  o.dec_ticket = nullptr;
  o.dec_bytes = 0;
  if (m->row_list && m->rows <= kDecodeMaxT) {
    char *ws = (char *)m->row_list + align256(list_bytes(m->rows, m->cols, m->tile_w, m->slots));
    o.dec_part = (float *)ws;
    o.dec_ticket = (uint64_t *)(ws + dec_tiles(m->cols) * 2 * kDecHalfBytes);
    o.dec_bytes = dec_tiles(m->cols) * 2 * kDecHalfBytes;
  }
  o.n_t = m->cols / m->tile_w;
  o.S = m->slots;
  o.words = (m->rows + 31) / 32;
  o.val_bf16 = m->val_dtype == TWELL_BF16;
  return o;
}

TwellFinish finish_of(twell_matrix_t *m, bool complete) {
  TwellFinish f;
  f.complete = complete;
  f.row_nnz = m->row_nnz;
  f.row_list = (uint2 *)m->row_list;
  f.ovf_n = m->ovf_n;
  f.ovf_rows = m->ovf_rows;
  f.ovf_slot = m->ovf_slot;
  f.ovf_dense = m->ovf_dense;
  f.cap = m->ovf_cap;
  return f;
}

TwellIn in_of(const twell_matrix_t *m) {
  TwellIn h;
  h.counts = m->counts;
  h.col_idx = m->col_idx;
  h.vals = m->vals;
  h.ovf_slot = m->ovf_slot;
  h.ovf_dense = m->ovf_dense;
  h.ovf_n = m->ovf_n;
  h.ovf_rows = m->ovf_rows;
  h.cap = m->ovf_cap;
  h.row_nnz = m->row_nnz;
  h.row_list = (uint2 *)m->row_list;
  h.rows = m->rows;
  h.cols = m->cols;
  h.n_t = m->cols / m->tile_w;
  h.S = m->slots;
  h.W = m->tile_w;
  h.val_bf16 = m->val_dtype == TWELL_BF16;
  return h;
}

}  // namespace

extern "C" {

int twell_abi_version(void) { return TWELL_ABI_VERSION; }

const char *twell_status_str(int status) {
  switch (status) {
    case TWELL_OK: return "TWELL_OK";
    case TWELL_ERR_ARG: return "TWELL_ERR_ARG: null pointer or invalid enum/struct field";
    case TWELL_ERR_SHAPE: return "TWELL_ERR_SHAPE: invalid or inconsistent sizes";
    case TWELL_ERR_ALIGN: return "TWELL_ERR_ALIGN: misaligned pointer or d_model % 8 != 0";
    case TWELL_ERR_WORKSPACE: return "TWELL_ERR_WORKSPACE: workspace too small";
    case TWELL_ERR_OVF_CAPACITY: return "TWELL_ERR_OVF_CAPACITY: more overflow rows than ovf_cap";
    case TWELL_ERR_HIP: return "TWELL_ERR_HIP: HIP runtime or launch failure";
    case TWELL_ERR_UNSUPPORTED: return "TWELL_ERR_UNSUPPORTED: valid request not implemented";
    default: return "TWELL_UNKNOWN_STATUS";
  }
}

size_t twell_ovf_bits_words(int32_t rows, int32_t cols, int32_t tile_w) {
  if (rows < 0 || cols <= 0 || tile_w <= 0) return 0;
  return (size_t)(cols / tile_w) * (size_t)((rows + 31) / 32);
}

size_t twell_row_list_bytes(int32_t rows, int32_t cols, int32_t tile_w, int32_t slots) {
  if (rows < 0 || cols <= 0 || tile_w <= 0 || slots <= 0) return 0;
  const size_t lists = list_bytes(rows, cols, tile_w, slots);
  return rows <= kDecodeMaxT ? align256(lists) + dec_ws_bytes(cols) : lists;
}

int twell_pack(const void *h, int32_t h_dtype, twell_matrix_t *out, void *stream) {
  if (!h || !out) return TWELL_ERR_ARG;
  if (!dtype_ok(h_dtype)) return TWELL_ERR_ARG;
  int st = check_matrix(out, true);
  if (st) return st;
  if (h_dtype == TWELL_F32 && out->val_dtype == TWELL_BF16) return TWELL_ERR_UNSUPPORTED;
  if (!al16(h)) return TWELL_ERR_ALIGN;
  const int R = out->rows, C = out->cols;
  if (R == 0) return hip_status(launch_set_int(out->ovf_n, 0, S(stream)));
  const TwellOut o = out_of(out);
  TW_TRY(launch_pack(h, h_dtype == TWELL_BF16, R, C, o, out->tile_w, S(stream)));
  TW_TRY(launch_ovf_scan(out->ovf_bits, o.n_t, o.words, R, out->ovf_cap, out->ovf_n, out->ovf_rows,
                         out->ovf_slot, S(stream)));
  TW_TRY(launch_ovf_copy(h, h_dtype == TWELL_BF16, R, C, out->ovf_n, out->ovf_rows, out->ovf_cap,
                         out->ovf_dense, out->val_dtype == TWELL_BF16, S(stream)));
  return TWELL_OK;
}

static int check_ffn_args(const void *x, const void *w1t, const void *w2, int32_t in_dtype, int32_t T,
                          int32_t d, int32_t f) {
  if (!w1t || (T > 0 && !x)) return TWELL_ERR_ARG;
  if (!dtype_ok(in_dtype)) return TWELL_ERR_ARG;
  if (T < 0 || d <= 0 || f <= 0) return TWELL_ERR_SHAPE;
  if (d % 8) return TWELL_ERR_ALIGN;
  if (!al16(x) || !al16(w1t) || (w2 && !al16(w2))) return TWELL_ERR_ALIGN;
  // the GEMM addresses each operand with 32-bit byte offsets
  const size_t es = in_dtype == TWELL_BF16 ? 2 : 4;
  if ((size_t)T * d * es >= ((size_t)1 << 31) || (size_t)f * d * es >= ((size_t)1 << 31)) return TWELL_ERR_UNSUPPORTED;
  return TWELL_OK;
}

static int check_up_args(const void *x, const void *w1t, const float *b1, int32_t in_dtype, int32_t T,
                         int32_t d_model, int32_t d_ff, const twell_matrix_t *h) {
  if (!b1 || !h) return TWELL_ERR_ARG;
  int st = check_ffn_args(x, w1t, nullptr, in_dtype, T, d_model, d_ff);
  if (st) return st;
  st = check_matrix(h, true);
  if (st) return st;
  if (h->rows != T || h->cols != d_ff) return TWELL_ERR_SHAPE;
  if (T > 0 && T <= kDecodeMaxT && !h->row_list) return TWELL_ERR_ARG;   // decode workspace
  if (!al4(b1)) return TWELL_ERR_ALIGN;
  return TWELL_OK;
}

// complete: let the GEMM stage also build the lists, the overflow scan and the backup rows
// where it can do that itself (one or two tokens; see gemm_completes)
static int up_gemm(const void *x, const void *w1t, const float *b1, int32_t in_dtype, int32_t T, int32_t d_model,
                   int32_t d_ff, twell_matrix_t *h, hipStream_t s, bool complete = false) {
  if (T == 0) return TWELL_OK;
  TW_TRY(launch_up_twell(in_dtype == TWELL_BF16, x, w1t, b1, T, d_ff, d_model, out_of(h), finish_of(h, complete),
                         h->tile_w, s));
  return TWELL_OK;
}

// true if up_gemm(..., complete = true) completes the matrix (lists, overflow scan, backup
// rows): then up_finish has nothing left to do
static bool gemm_completes(int32_t in_dtype, int32_t T, int32_t d_model, twell_matrix_t *h) {
  return T > 0 && up_twell_completes(in_dtype == TWELL_BF16, T, d_model, finish_of(h, true));
}

static int up_finish(const void *x, const void *w1t, const float *b1, int32_t in_dtype, int32_t T,
                     int32_t d_model, int32_t d_ff, twell_matrix_t *h, hipStream_t s) {
  if (T == 0) return hip_status(launch_set_int(h->ovf_n, 0, s));
  const TwellOut o = out_of(h);
  const hipError_t fe = launch_finish_dec(in_dtype == TWELL_BF16, in_of(h), h->ovf_bits, o.words, h->ovf_n,
                                          h->ovf_rows, h->ovf_slot, x, w1t, b1, d_model, h->ovf_dense, s);
  if (fe == hipSuccess) return TWELL_OK;
  if (fe != hipErrorNotSupported) return hip_status(fe);
  TW_TRY(launch_lists_scan(in_of(h), h->ovf_bits, o.words, h->ovf_n, h->ovf_rows, h->ovf_slot, s));
  if (h->ovf_cap > 0) {
    const int M = h->ovf_cap < T ? h->ovf_cap : T;
    TW_TRY(launch_up_dense(in_dtype == TWELL_BF16, x, w1t, b1, M, d_ff, d_model, T, h->ovf_rows, h->ovf_n,
                           h->ovf_dense, h->val_dtype == TWELL_BF16, 1, s));
  }
  return TWELL_OK;
}

int twell_up_gemm(const void *x, const void *w1t, const float *b1, int32_t in_dtype, int32_t T,
                  int32_t d_model, int32_t d_ff, twell_matrix_t *h, void *stream) {
  int st = check_up_args(x, w1t, b1, in_dtype, T, d_model, d_ff, h);
  if (st) return st;
  return up_gemm(x, w1t, b1, in_dtype, T, d_model, d_ff, h, S(stream));
}

int twell_up_finish(const void *x, const void *w1t, const float *b1, int32_t in_dtype, int32_t T,
                    int32_t d_model, int32_t d_ff, twell_matrix_t *h, void *stream) {
  int st = check_up_args(x, w1t, b1, in_dtype, T, d_model, d_ff, h);
  if (st) return st;
  st = check_matrix(h, true, true);
  if (st) return st;
  return up_finish(x, w1t, b1, in_dtype, T, d_model, d_ff, h, S(stream));
}

int twell_ffn_fwd(const void *x, const void *w1t, const float *b1, const void *w2, int32_t in_dtype,
                  int32_t T, int32_t d_model, int32_t d_ff, twell_matrix_t *h, void *y, int32_t y_dtype,
                  void *stream) {
  if (!w2 || (T > 0 && !y)) return TWELL_ERR_ARG;
  if (!dtype_ok(y_dtype)) return TWELL_ERR_ARG;
  int st = check_up_args(x, w1t, b1, in_dtype, T, d_model, d_ff, h);
  if (st) return st;
  st = check_matrix(h, true, true);
  if (st) return st;
  if (!al16(w2) || !al16(y)) return TWELL_ERR_ALIGN;
  hipStream_t s = S(stream);
  if (T > 0 && in_dtype == TWELL_BF16 && up_stream_ok(1, T, d_model)) {
    // up to 16 tokens: the W1 stream, then the TwELL, the overflow scan and y in one launch
    const TwellOut o = out_of(h);
    TW_TRY(launch_up_stream(x, w1t, T, d_ff, d_model, o, s));
    TW_TRY(launch_dec_fused_down(b1, T, d_ff, o, finish_of(h, true), w2, d_model, y, y_dtype == TWELL_BF16, h->tile_w,
                                 s));
    return TWELL_OK;
  }
  st = up_gemm(x, w1t, b1, in_dtype, T, d_model, d_ff, h, s, true);
  if (st) return st;
  if (!gemm_completes(in_dtype, T, d_model, h)) st = up_finish(x, w1t, b1, in_dtype, T, d_model, d_ff, h, s);
  if (st || T == 0) return st;
  TW_TRY(launch_twell_down(in_of(h), w2, in_dtype == TWELL_BF16, d_model, y, y_dtype == TWELL_BF16, false, s));
  return TWELL_OK;
}

static int down_args(const twell_matrix_t *h, const void *w2, int32_t w_dtype, int32_t d_model, const void *y,
                     int32_t y_dtype, bool row_ell = false) {
  if (!h || !w2 || !y) return TWELL_ERR_ARG;
  if (!dtype_ok(w_dtype) || !dtype_ok(y_dtype)) return TWELL_ERR_ARG;
  int st = check_matrix(h, false, true, row_ell);
  if (st) return st;
  if (d_model <= 0) return TWELL_ERR_SHAPE;
  if (d_model % 8) return TWELL_ERR_ALIGN;
  if (!al16(w2) || !al16(y)) return TWELL_ERR_ALIGN;
  // the gathers address W2 rows (and y) with 32-bit byte offsets
  const size_t wb = w_dtype == TWELL_BF16 ? 2 : 4, yb = y_dtype == TWELL_BF16 ? 2 : 4;
  if ((size_t)h->cols * d_model * wb >= ((size_t)1 << 31) || (size_t)h->rows * d_model * yb >= ((size_t)1 << 31))
    return TWELL_ERR_UNSUPPORTED;
  return TWELL_OK;
}

int twell_fwd_down(const twell_matrix_t *h, const void *w2, int32_t w_dtype, int32_t d_model, void *y,
                   int32_t y_dtype, void *stream) {
  int st = down_args(h, w2, w_dtype, d_model, y, y_dtype);
  if (st) return st;
  if (h->rows == 0) return TWELL_OK;
  TW_TRY(launch_twell_down(in_of(h), w2, w_dtype == TWELL_BF16, d_model, y, y_dtype == TWELL_BF16, false,
                           S(stream)));
  return TWELL_OK;
}

int twell_down(const twell_matrix_t *h, const void *w2, int32_t w_dtype, int32_t d_model, void *y,
               int32_t y_dtype, void *stream) {
  int st = down_args(h, w2, w_dtype, d_model, y, y_dtype, true);
  if (st) return st;
  if (h->rows == 0) return TWELL_OK;
  TW_TRY(launch_twell_down(in_of(h), w2, w_dtype == TWELL_BF16, d_model, y, y_dtype == TWELL_BF16, true,
                           S(stream)));
  return TWELL_OK;
}

size_t twell_gate_up_workspace_bytes(int32_t T, int32_t d_model, int32_t d_ff, int32_t in_dtype,
                                     const twell_matrix_t *h) {
  if (!h || T < 0 || d_model <= 0 || d_ff <= 0 || h->tile_w <= 0 || h->slots <= 0) return 0;
  if (!dtype_ok(in_dtype)) return 0;
  return gate_up_workspace_bytes(T, d_model, d_ff / h->tile_w, h->slots, in_dtype == TWELL_BF16);
}

// The workspace the up products need for this h (checked before anything is enqueued).
static int gate_ws_check(const twell_matrix_t *h, int32_t in_dtype, int32_t d_model, const void *ws,
                         size_t ws_bytes) {
  const size_t need = gate_up_workspace_bytes(h->rows, d_model, h->cols / h->tile_w, h->slots, in_dtype == TWELL_BF16);
  if (need == 0) return TWELL_OK;
  if (!ws || ws_bytes < need) return TWELL_ERR_WORKSPACE;
  if (!al16(ws)) return TWELL_ERR_ALIGN;
  return TWELL_OK;
}

int twell_gate_up(twell_matrix_t *h, const void *x, const void *w_up_t, int32_t in_dtype, int32_t T,
                  int32_t d_model, int32_t d_ff, void *workspace, size_t workspace_bytes, void *stream) {
  if (!h) return TWELL_ERR_ARG;
  int st = check_ffn_args(x, w_up_t, nullptr, in_dtype, T, d_model, d_ff);
  if (st) return st;
  st = check_matrix(h, false, true);
  if (st) return st;
  if (h->rows != T || h->cols != d_ff) return TWELL_ERR_SHAPE;
  st = gate_ws_check(h, in_dtype, d_model, workspace, workspace_bytes);
  if (st) return st;
  if (T == 0) return TWELL_OK;
  TW_TRY(launch_gate_up(in_of(h), x, w_up_t, in_dtype == TWELL_BF16, d_model, (float *)workspace, S(stream)));
  return TWELL_OK;
}

int twell_gated_ffn_fwd(const void *x, const void *w_gate_t, const float *b_gate, const void *w_up_t,
                        const void *w2, int32_t in_dtype, int32_t T, int32_t d_model, int32_t d_ff,
                        twell_matrix_t *h, void *y, int32_t y_dtype, void *workspace, size_t workspace_bytes,
                        void *stream) {
  if (!w2 || !w_up_t || (T > 0 && !y)) return TWELL_ERR_ARG;
  if (!dtype_ok(y_dtype)) return TWELL_ERR_ARG;
  int st = check_up_args(x, w_gate_t, b_gate, in_dtype, T, d_model, d_ff, h);
  if (st) return st;
  st = check_matrix(h, true, true);
  if (st) return st;
  if (!al16(w2) || !al16(y) || !al16(w_up_t)) return TWELL_ERR_ALIGN;
  st = gate_ws_check(h, in_dtype, d_model, workspace, workspace_bytes);
  if (st) return st;
  hipStream_t s = S(stream);
  st = up_gemm(x, w_gate_t, b_gate, in_dtype, T, d_model, d_ff, h, s, true);
  if (st) return st;
  if (!gemm_completes(in_dtype, T, d_model, h)) st = up_finish(x, w_gate_t, b_gate, in_dtype, T, d_model, d_ff, h, s);
  if (st || T == 0) return st;
  TW_TRY(launch_gate_up(in_of(h), x, w_up_t, in_dtype == TWELL_BF16, d_model, (float *)workspace, s));
  TW_TRY(launch_twell_down(in_of(h), w2, in_dtype == TWELL_BF16, d_model, y, y_dtype == TWELL_BF16, false, s));
  return TWELL_OK;
}

int twell_gated_ffn_infer(const void *x, const void *w_gate_t, const float *b_gate, const void *w_up_t,
                          const void *w2, int32_t in_dtype, int32_t T, int32_t d_model, int32_t d_ff,
                          twell_matrix_t *h, void *y, int32_t y_dtype, void *stream) {
  if (!w2 || !w_up_t || (T > 0 && !y)) return TWELL_ERR_ARG;
  if (!dtype_ok(y_dtype)) return TWELL_ERR_ARG;
  int st = check_up_args(x, w_gate_t, b_gate, in_dtype, T, d_model, d_ff, h);
  if (st) return st;
  st = check_matrix(h, true, true);
  if (st) return st;
  if (!al16(w2) || !al16(y) || !al16(w_up_t)) return TWELL_ERR_ALIGN;
  if (T > kDecodeMaxT || d_ff / h->tile_w > 256) return TWELL_ERR_UNSUPPORTED;
  if (T == 0) return TWELL_OK;
  hipStream_t s = S(stream);
  st = up_gemm(x, w_gate_t, b_gate, in_dtype, T, d_model, d_ff, h, s);
  if (st) return st;
  const TwellOut o = out_of(h);           // o.dec_part: the dense scratch rows [T][d_ff] fp32
  TW_TRY(launch_gated_fused(in_of(h), x, w_gate_t, b_gate, w_up_t, w2, in_dtype == TWELL_BF16, d_model, y,
                            y_dtype == TWELL_BF16, o.dec_part, s));
  return TWELL_OK;
}

int ffn_up_relu_dense(const void *x, const void *w1t, const float *b1, int32_t in_dtype, int32_t T,
                      int32_t d_model, int32_t d_ff, void *h, int32_t h_dtype, void *stream) {
  if (!b1 || (T > 0 && !h)) return TWELL_ERR_ARG;
  if (!dtype_ok(h_dtype)) return TWELL_ERR_ARG;
  int st = check_ffn_args(x, w1t, nullptr, in_dtype, T, d_model, d_ff);
  if (st) return st;
  if (!al16(h) || !al4(b1)) return TWELL_ERR_ALIGN;
  if (T == 0) return TWELL_OK;
  TW_TRY(launch_up_dense(in_dtype == TWELL_BF16, x, w1t, b1, T, d_ff, d_model, T, nullptr, nullptr, h,
                         h_dtype == TWELL_BF16, 1, S(stream)));
  return TWELL_OK;
}

size_t twell_ffn_bwd_workspace_bytes(int32_t T, int32_t d_model, int32_t d_ff, int32_t in_dtype,
                                     const twell_matrix_t *h) {
  if (!h || T < 0 || d_model <= 0 || d_ff <= 0 || h->tile_w <= 0 || h->slots <= 0 || h->ovf_cap < 0) return 0;
  if (!dtype_ok(in_dtype)) return 0;
  const size_t nz = bwd_entry_capacity(T, d_ff, d_ff / h->tile_w, h->slots, h->ovf_cap);
  return bwd_workspace_bytes(T, d_model, d_ff, nz, in_dtype == TWELL_BF16);
}

size_t twell_ffn_bwd_workspace_bytes_nnz(int32_t T, int32_t d_model, int32_t d_ff, int32_t in_dtype,
                                         const twell_matrix_t *h, int64_t nnz) {
  if (!h || T < 0 || d_model <= 0 || d_ff <= 0 || h->tile_w <= 0 || h->slots <= 0 || h->ovf_cap < 0 || nnz < 0)
    return 0;
  if (!dtype_ok(in_dtype)) return 0;
  const size_t cap = bwd_entry_capacity(T, d_ff, d_ff / h->tile_w, h->slots, h->ovf_cap);
  return bwd_workspace_bytes(T, d_model, d_ff, (size_t)nnz < cap ? (size_t)nnz : cap, in_dtype == TWELL_BF16);
}

int twell_ffn_bwd(const void *x, const void *w1t, const void *w2, int32_t in_dtype, int32_t T,
                  int32_t d_model, int32_t d_ff, const twell_matrix_t *h, const void *dy, float l1_coef,
                  float *dx, float *dw1t, float *dw2, float *db1, void *workspace, size_t workspace_bytes,
                  void *stream) {
  if (!h || !w2 || !dw1t || !dw2 || !workspace) return TWELL_ERR_ARG;
  if (T > 0 && (!dy || !dx)) return TWELL_ERR_ARG;
  int st = check_ffn_args(x, w1t, w2, in_dtype, T, d_model, d_ff);
  if (st) return st;
  st = check_matrix(h, false, false, true);
  if (st) return st;
  if (h->rows != T || h->cols != d_ff) return TWELL_ERR_SHAPE;
  if (!al16(dy) || !al16(dx) || !al16(dw1t) || !al16(dw2) || !al4(db1) || !al16(workspace)) return TWELL_ERR_ALIGN;
  // unit masks of a 32-token block live in LDS (4 bytes per unit)
  if (d_ff > 16384) return TWELL_ERR_UNSUPPORTED;
  // the workspace holds `nz` entries (all of h's capacity if it is that large); whether the
  // call's actual entries fit is checked on the device
  const size_t cap = bwd_entry_capacity(T, d_ff, d_ff / h->tile_w, h->slots, h->ovf_cap);
  const size_t nz = bwd_fit_entries(T, d_model, d_ff, workspace_bytes, cap, in_dtype == TWELL_BF16);
  if (nz == SIZE_MAX) return TWELL_ERR_WORKSPACE;
  BwdArgs a;
  a.nz = nz;
  a.h = in_of(h);
  a.x = x; a.w1t = w1t; a.w2 = w2; a.dy = dy;
  a.l1 = l1_coef;
  a.dx = dx; a.dw1t = dw1t; a.dw2 = dw2; a.db1 = db1;
  a.ws = workspace;
  a.d = d_model;
  a.bf16 = in_dtype == TWELL_BF16;
  a.cap = h->ovf_cap;
  TW_TRY(launch_bwd(a, S(stream)));
  return TWELL_OK;
}

int twell_ffn_bwd_noalloc(const void *x, const void *w1t, const void *w2, int32_t in_dtype, int32_t T,
                          int32_t d_model, int32_t d_ff, const twell_matrix_t *h, const void *dy, float l1_coef,
                          float *dx, float *dw1t, float *dw2, float *db1, void *stream) {
  if (!h) return TWELL_ERR_ARG;
  // the size check comes first, so that a problem beyond the fixed scratch is refused before
  // any device lookup
  if (T >= 0 && d_model > 0 && d_ff > 0 && dtype_ok(in_dtype) && h->tile_w > 0 && h->slots > 0 && h->ovf_cap >= 0 &&
      twell_ffn_bwd_workspace_bytes(T, d_model, d_ff, in_dtype, h) > (size_t)TWELL_NOALLOC_SCRATCH_BYTES)
    return TWELL_ERR_WORKSPACE;
  void *ws = scratch_on_current_device();
  if (!ws) return TWELL_ERR_HIP;
  return twell_ffn_bwd(x, w1t, w2, in_dtype, T, d_model, d_ff, h, dy, l1_coef, dx, dw1t, dw2, db1, ws,
                       (size_t)TWELL_NOALLOC_SCRATCH_BYTES, stream);
}

int nm_prune(const void *h, int32_t dtype, int32_t T, int32_t d_ff, int32_t n, int32_t m, void *vals,
             uint8_t *idx, void *stream) {
  if ((T > 0 && (!h || !vals || !idx))) return TWELL_ERR_ARG;
  if (!dtype_ok(dtype)) return TWELL_ERR_ARG;
  if (T < 0 || d_ff <= 0) return TWELL_ERR_SHAPE;
  if (!((n == 2 && m == 4) || (n == 4 && m == 8) || (n == 8 && m == 16) || (n == 16 && m == 32)))
    return TWELL_ERR_SHAPE;
  if (d_ff % m) return TWELL_ERR_SHAPE;
  if (!al16(h) || !al16(vals) || !al16(idx)) return TWELL_ERR_ALIGN;
  TW_TRY(launch_nm_prune(h, dtype == TWELL_BF16, T, d_ff, n, m, vals, idx, S(stream)));
  return TWELL_OK;
}

int ffn_up_relu_nm(const void *x, const void *w1t, const float *b1, int32_t in_dtype, int32_t T, int32_t d_model,
                   int32_t d_ff, int32_t n, int32_t m, void *vals, uint8_t *idx, void *stream) {
  if (!b1 || (T > 0 && (!vals || !idx))) return TWELL_ERR_ARG;
  int st = check_ffn_args(x, w1t, nullptr, in_dtype, T, d_model, d_ff);
  if (st) return st;
  if (!((n == 2 && m == 4) || (n == 4 && m == 8) || (n == 8 && m == 16) || (n == 16 && m == 32)))
    return TWELL_ERR_SHAPE;
  if (d_ff % m) return TWELL_ERR_SHAPE;
  if (!al4(b1) || !al16(vals) || !al16(idx)) return TWELL_ERR_ALIGN;
  if (T == 0) return TWELL_OK;
  TW_TRY(launch_up_nm(in_dtype == TWELL_BF16, x, w1t, b1, T, d_ff, d_model, n, m, vals, idx, S(stream)));
  return TWELL_OK;
}

int nm_ffn_down(const void *vals, const uint8_t *idx, int32_t dtype, int32_t T, int32_t d_ff, int32_t n,
                int32_t m, const void *w2, int32_t d_model, void *y, int32_t y_dtype, void *stream) {
  if (!w2 || (T > 0 && (!vals || !idx || !y))) return TWELL_ERR_ARG;
  if (!dtype_ok(dtype) || !dtype_ok(y_dtype)) return TWELL_ERR_ARG;
  if (T < 0 || d_ff <= 0 || d_model <= 0) return TWELL_ERR_SHAPE;
  if (!((n == 8 && m == 16) || (n == 16 && m == 32))) {
    if ((n == 2 && m == 4) || (n == 4 && m == 8)) return TWELL_ERR_UNSUPPORTED;
    return TWELL_ERR_SHAPE;
  }
  if (dtype != TWELL_BF16) return TWELL_ERR_UNSUPPORTED;
  if (d_ff % 32 || d_model % 8) return TWELL_ERR_SHAPE;
  if (!al16(vals) || !al16(idx) || !al16(w2) || !al16(y)) return TWELL_ERR_ALIGN;
  if ((size_t)d_model * d_ff * 2 >= ((size_t)1 << 31) || d_ff >= (1 << 23)) return TWELL_ERR_UNSUPPORTED;
  TW_TRY(launch_nm_down(vals, idx, T, d_ff, n, m, w2, d_model, y, y_dtype == TWELL_BF16, S(stream)));
  return TWELL_OK;
}

int twell_row_max_histogram(const twell_matrix_t *h, int32_t *hist, void *stream) {
  if (!hist) return TWELL_ERR_ARG;
  int st = check_matrix(h, false, false, true);
  if (st) return st;
  if (!al4(hist)) return TWELL_ERR_ALIGN;
  TW_TRY(launch_rowmax_hist(h->counts, h->rows, h->cols / h->tile_w, h->tile_w, hist, S(stream)));
  return TWELL_OK;
}

size_t twell_stash_bytes(int32_t rows, int32_t cols, int32_t tile_w, int32_t slots, int32_t n_ovf,
                         int32_t val_dtype) {
  if (rows < 0 || cols <= 0 || tile_w <= 0 || cols % tile_w || slots <= 0 || n_ovf < 0 || !dtype_ok(val_dtype))
    return 0;
  const size_t vb = val_dtype == TWELL_BF16 ? 2 : 4;
  const size_t cells = (size_t)rows * (size_t)(cols / tile_w);
  return cells * 4 + cells * (size_t)slots * (4 + vb) + (size_t)rows * 4 + (size_t)n_ovf * (4 + (size_t)cols * vb);
}

int twell_choose_slots(const int32_t *hist, int32_t tile_w, int32_t rows, int32_t cols, int32_t ovf_cap,
                       int32_t val_dtype, size_t *stash_bytes) {
  if (!hist || !dtype_ok(val_dtype)) return TWELL_ERR_ARG;
  if ((tile_w != 64 && tile_w != 128) || rows < 0 || cols <= 0 || cols % tile_w || ovf_cap < 0)
    return TWELL_ERR_SHAPE;
  int best = TWELL_ERR_OVF_CAPACITY;
  size_t best_bytes = 0;
  const int smax = tile_w < 64 ? tile_w : 64;
  for (int S = 1; S <= smax; ++S) {
    long long n_ovf = 0;
    for (int m = S + 1; m <= tile_w; ++m) n_ovf += hist[m];
    if (n_ovf > ovf_cap) continue;
    const size_t b = twell_stash_bytes(rows, cols, tile_w, S, (int32_t)n_ovf, val_dtype);
    if (best < 0 || b < best_bytes) {
      best = S;
      best_bytes = b;
    }
  }
  if (stash_bytes) *stash_bytes = best > 0 ? best_bytes : 0;
  return best;
}

int twell_row_nnz_histogram(const twell_matrix_t *h, int32_t *hist, int32_t nbins, void *stream) {
  if (!hist) return TWELL_ERR_ARG;
  int st = check_matrix(h, false, false, true);
  if (st) return st;
  if (nbins < 2) return TWELL_ERR_SHAPE;
  if (!al4(hist)) return TWELL_ERR_ALIGN;
  TW_TRY(launch_row_nnz_hist(h->counts, h->rows, h->cols / h->tile_w, nbins, hist, S(stream)));
  return TWELL_OK;
}

int twell_choose_row_ell_width(const int32_t *hist, int32_t nbins, int32_t rows, int32_t cols, int32_t ovf_cap,
                               int32_t val_dtype, size_t *stash_bytes) {
  if (!hist || !dtype_ok(val_dtype)) return TWELL_ERR_ARG;
  if (nbins < 3 || rows < 0 || cols <= 0 || ovf_cap < 0) return TWELL_ERR_SHAPE;
  // rows with more than N entries overflow; the last bin holds every row of nbins - 1 or more
  int best = TWELL_ERR_OVF_CAPACITY;
  size_t best_bytes = 0;
  long long above = 0;
  for (int m = 0; m < nbins; ++m) above += hist[m];
  const int nmax = nbins - 2 < cols ? nbins - 2 : cols;
  for (int N = 0; N <= nmax; ++N) {
    above -= hist[N];                          // rows with more than N entries
    if (N < 1 || above > ovf_cap) continue;
    const size_t b = twell_stash_bytes(rows, cols, cols, N, (int32_t)above, val_dtype);
    if (best < 0 || b < best_bytes) {
      best = N;
      best_bytes = b;
    }
  }
  if (stash_bytes) *stash_bytes = best > 0 ? best_bytes : 0;
  return best;
}

int twell_to_row_ell(const twell_matrix_t *src, twell_matrix_t *dst, void *stream) {
  int st = check_matrix(src, false);
  if (st) return st;
  st = check_matrix(dst, true, false, true);
  if (st) return st;
  if (dst->rows != src->rows || dst->cols != src->cols || dst->tile_w != dst->cols) return TWELL_ERR_SHAPE;
  if (src->val_dtype == TWELL_F32 && dst->val_dtype == TWELL_BF16) return TWELL_ERR_UNSUPPORTED;
  if (dst->cols > 16384) return TWELL_ERR_UNSUPPORTED;
  TW_TRY(launch_to_row_ell(in_of(src), out_of(dst), dst->slots, dst->ovf_cap, dst->ovf_n, dst->ovf_rows, dst->ovf_slot,
                           dst->ovf_dense, S(stream)));
  return TWELL_OK;
}

// A row stride: at least d, and whole 16-byte units, so that every row starts aligned.
static bool ld_ok(int64_t ld, int32_t d) { return ld >= d && ld % 8 == 0; }

int layer_norm_fwd(const void *x, int64_t ldx, const void *residual, int64_t ldr, const float *w, const float *b,
                   int32_t x_dtype, int32_t T, int32_t d, float eps, void *y, int32_t y_dtype, void *s, float *mean,
                   float *rstd, void *stream) {
  if (!w || (T > 0 && (!x || !y)) || (T > 0 && residual && !s)) return TWELL_ERR_ARG;
  if (!dtype_ok(x_dtype) || !dtype_ok(y_dtype) || !(eps >= 0.f)) return TWELL_ERR_ARG;
  if (T < 0 || d <= 0) return TWELL_ERR_SHAPE;
  if (d % 8) return TWELL_ERR_ALIGN;
  if (T > 1 && (ldx < d || (residual && ldr < d))) return TWELL_ERR_SHAPE;
  if (T > 1 && (!ld_ok(ldx, d) || (residual && !ld_ok(ldr, d)))) return TWELL_ERR_ALIGN;
  if (!al16(x) || !al16(residual) || !al16(w) || !al16(b) || !al16(y) || !al16(s) || !al4(mean) || !al4(rstd))
    return TWELL_ERR_ALIGN;
  if (d > kNormMaxD) return TWELL_ERR_UNSUPPORTED;
  if (T == 0) return TWELL_OK;
  NormFwd a;
  a.x = x; a.res = residual; a.ldx = ldx; a.ldr = ldr;
  a.w = w; a.b = b;
  a.rows = T; a.d = d; a.eps = eps;
  a.x_bf16 = x_dtype == TWELL_BF16; a.y_bf16 = y_dtype == TWELL_BF16;
  a.y = y; a.s = s; a.mean = mean; a.rstd = rstd;
  TW_TRY(launch_norm_fwd(a, S(stream)));
  return TWELL_OK;
}

size_t layer_norm_bwd_workspace_bytes(int32_t T, int32_t d) {
  if (T <= 0 || d <= 0) return 0;
  const int p = norm_bwd_strips(T, d);
  return p > 1 ? (size_t)p * 2 * d * sizeof(float) : 0;
}

int layer_norm_bwd(const void *dy, int64_t lddy, int32_t dy_dtype, const void *s, int64_t lds, int32_t x_dtype,
                   const float *w, const float *mean, const float *rstd, const void *dres, int64_t lddr, int32_t T,
                   int32_t d, void *dx, int32_t dx_dtype, float *dw, float *db, void *workspace,
                   size_t workspace_bytes, void *stream) {
  if (!w || !dw || (T > 0 && (!dy || !s || !mean || !rstd || !dx))) return TWELL_ERR_ARG;
  if (!dtype_ok(x_dtype) || !dtype_ok(dy_dtype) || !dtype_ok(dx_dtype)) return TWELL_ERR_ARG;
  if (T < 0 || d <= 0) return TWELL_ERR_SHAPE;
  if (d % 8) return TWELL_ERR_ALIGN;
  if (T > 1 && (lddy < d || lds < d || (dres && lddr < d))) return TWELL_ERR_SHAPE;
  if (T > 1 && (!ld_ok(lddy, d) || !ld_ok(lds, d) || (dres && !ld_ok(lddr, d)))) return TWELL_ERR_ALIGN;
  if (!al16(dy) || !al16(s) || !al16(w) || !al16(dres) || !al16(dx) || !al16(dw) || !al16(db) || !al4(mean) ||
      !al4(rstd))
    return TWELL_ERR_ALIGN;
  if (d > kNormMaxD) return TWELL_ERR_UNSUPPORTED;
  const size_t need = layer_norm_bwd_workspace_bytes(T, d);
  if (need && (!workspace || workspace_bytes < need)) return TWELL_ERR_WORKSPACE;
  if (need && !al16(workspace)) return TWELL_ERR_ALIGN;
  if (T == 0) {                             // no rows: the sums over them are zero
    TW_TRY(launch_zero_i32((int32_t *)dw, d, S(stream)));
    if (db) TW_TRY(launch_zero_i32((int32_t *)db, d, S(stream)));
    return TWELL_OK;
  }
  NormBwd a;
  a.dy = dy; a.s = s; a.dres = dres; a.lddy = lddy; a.lds = lds; a.lddr = lddr;
  a.w = w; a.mean = mean; a.rstd = rstd;
  a.rows = T; a.d = d;
  a.x_bf16 = x_dtype == TWELL_BF16; a.dy_bf16 = dy_dtype == TWELL_BF16; a.dx_bf16 = dx_dtype == TWELL_BF16;
  a.dx = dx; a.dw = dw; a.db = db; a.part = (float *)workspace;
  TW_TRY(launch_norm_bwd(a, S(stream)));
  return TWELL_OK;
}

// the tiles of w and of the kept exponentials are addressed with 32-bit byte offsets
static constexpr int kXentMaxV = 1 << 21, kXentMaxT = 1 << 24, kXentMaxD = 1 << 16;

static int xent_shape(int32_t T, int32_t d, int32_t V) {
  if (T < 0 || d <= 0 || V <= 0) return TWELL_ERR_SHAPE;
  if (d % 8) return TWELL_ERR_ALIGN;
  if (T > kXentMaxT || d > kXentMaxD || V > kXentMaxV) return TWELL_ERR_UNSUPPORTED;
  return TWELL_OK;
}

size_t linear_xent_workspace_bytes(int32_t T, int32_t d, int32_t V, int32_t dtype, int32_t want_grad) {
  if (T <= 0 || !dtype_ok(dtype) || xent_shape(T, d, V) != TWELL_OK) return 0;
  return xent_workspace_bytes(T, d, V, dtype == TWELL_BF16, want_grad != 0);
}

static int xent_check(const XentArgs &a, int32_t dtype, bool grad, size_t workspace_bytes) {
  if (!a.w || (a.T > 0 && (!a.x || !a.y || !a.loss || !a.lse))) return TWELL_ERR_ARG;
  if (grad && (!a.dw || (a.T > 0 && (!a.dx || !a.dloss)))) return TWELL_ERR_ARG;
  if (!dtype_ok(dtype)) return TWELL_ERR_ARG;
  const int st = xent_shape(a.T, a.d, a.V);
  if (st) return st;
  if (a.T > 1 && a.ldx < a.d) return TWELL_ERR_SHAPE;
  if (a.T > 1 && !ld_ok(a.ldx, a.d)) return TWELL_ERR_ALIGN;
  if (!al16(a.x) || !al16(a.w) || !al16(a.dx) || !al16(a.dw) || ((uintptr_t)a.y & 7u) || !al4(a.loss) || !al4(a.lse) ||
      !al4(a.dloss))
    return TWELL_ERR_ALIGN;
  if (a.T == 0) return TWELL_OK;
  if (!a.ws || workspace_bytes < xent_workspace_bytes(a.T, a.d, a.V, a.bf16, grad)) return TWELL_ERR_WORKSPACE;
  if (!al16(a.ws)) return TWELL_ERR_ALIGN;
  return TWELL_OK;
}

static XentArgs xent_args(const void *x, int64_t ldx, const void *w, const int64_t *targets, int32_t dtype, int32_t T,
                          int32_t d, int32_t V, float *loss, float *lse, void *workspace) {
  XentArgs a = {};
  a.x = x; a.w = w; a.ldx = ldx; a.y = targets;
  a.T = T; a.d = d; a.V = V; a.bf16 = dtype == TWELL_BF16;
  a.loss = loss; a.lse = lse;
  a.ws = workspace;
  return a;
}

int linear_xent_fwd(const void *x, int64_t ldx, const void *w, const int64_t *targets, int32_t dtype, int32_t T,
                    int32_t d, int32_t V, float *loss, float *lse, void *workspace, size_t workspace_bytes,
                    void *stream) {
  const XentArgs a = xent_args(x, ldx, w, targets, dtype, T, d, V, loss, lse, workspace);
  const int st = xent_check(a, dtype, false, workspace_bytes);
  if (st || T == 0) return st;
  TW_TRY(launch_xent(a, S(stream)));
  return TWELL_OK;
}

int linear_xent_fwd_bwd(const void *x, int64_t ldx, const void *w, const int64_t *targets, const float *dloss,
                        int32_t dtype, int32_t T, int32_t d, int32_t V, float *loss, float *lse, void *dx, void *dw,
                        void *workspace, size_t workspace_bytes, void *stream) {
  XentArgs a = xent_args(x, ldx, w, targets, dtype, T, d, V, loss, lse, workspace);
  a.dloss = dloss; a.dx = dx; a.dw = dw;
  const int st = xent_check(a, dtype, true, workspace_bytes);
  if (st) return st;
  TW_TRY(launch_xent(a, S(stream)));
  return TWELL_OK;
}

size_t grad_norm_workspace_bytes(int32_t n) { return n > 0 ? grad_workspace_bytes(n) : 0; }

// Whether every output lies apart from all other outputs and from all gradients but its own, which it
// may replace: the scaling's workgroups run in no order, so an element that two of them write, or one
// writes and another reads, would come out scaled once or twice. n log n on the host (1000 tensors
// in no order: 12 us; 41: 0.3).
static int grad_outs_apart(const void *const *grads, void *const *outs, const int64_t *sizes, const int32_t *dtypes,
                           const int32_t *out_dtypes, int32_t n) {
  struct Span {
    uintptr_t at, end;
  } few[64], *span = n <= 64 ? few : new (std::nothrow) Span[n];
  if (!span) return TWELL_ERR_HIP;          // no host memory
  int m = 0;
  for (int i = 0; i < n; ++i) {
    if (sizes[i] == 0) continue;
    const uintptr_t at = (uintptr_t)outs[i];
    span[m++] = {at, at + (uintptr_t)sizes[i] * (out_dtypes[i] == TWELL_BF16 ? 2 : 4)};
  }
  std::sort(span, span + m, [](const Span &a, const Span &b) { return a.at < b.at; });
  bool ok = true;
  for (int k = 1; k < m; ++k) ok = ok && span[k - 1].end <= span[k].at;
  // the outputs are apart, so of those that begin before a gradient's end the last reaches furthest
  for (int i = 0; ok && i < n; ++i) {
    if (sizes[i] == 0 || outs[i] == grads[i]) continue;
    const uintptr_t at = (uintptr_t)grads[i], end = at + (uintptr_t)sizes[i] * (dtypes[i] == TWELL_BF16 ? 2 : 4);
    const Span *s = std::lower_bound(span, span + m, end, [](const Span &a, uintptr_t e) { return a.at < e; });
    ok = s == span || s[-1].end <= at;
  }
  if (span != few) delete[] span;
  return ok ? TWELL_OK : TWELL_ERR_ARG;
}

// Shared checks of grad_norm and grad_clip (outs == NULL: the norm only).
static int grad_run(const void *const *grads, void *const *outs, const int64_t *sizes, const int32_t *dtypes,
                    const int32_t *out_dtypes, int32_t n, float max_norm, float *norm, void *workspace,
                    size_t workspace_bytes, hipStream_t s) {
  if (n < 0) return TWELL_ERR_SHAPE;
  if (!norm || (n > 0 && (!grads || !sizes || !dtypes))) return TWELL_ERR_ARG;
  if (!al4(norm)) return TWELL_ERR_ALIGN;
  int64_t total = 0;
  for (int i = 0; i < n; ++i) {
    if (sizes[i] < 0) return TWELL_ERR_SHAPE;
    if (!dtype_ok(dtypes[i]) || (out_dtypes && !dtype_ok(out_dtypes[i]))) return TWELL_ERR_ARG;
    if (sizes[i] == 0) continue;
    if (!grads[i] || (outs && !outs[i])) return TWELL_ERR_ARG;
    if (outs && outs[i] == grads[i] && out_dtypes[i] != dtypes[i]) return TWELL_ERR_ARG;
    if ((uintptr_t)grads[i] % (dtypes[i] == TWELL_BF16 ? 2 : 4)) return TWELL_ERR_ALIGN;
    if (outs && (uintptr_t)outs[i] % (out_dtypes[i] == TWELL_BF16 ? 2 : 4)) return TWELL_ERR_ALIGN;
    // chunks of the whole set are counted in 32 bits
    if (sizes[i] > ((int64_t)1 << 40) || (total += sizes[i]) > ((int64_t)1 << 40)) return TWELL_ERR_UNSUPPORTED;
  }
  if (outs) {
    const int st = grad_outs_apart(grads, outs, sizes, dtypes, out_dtypes, n);
    if (st) return st;
  }
  if (n > 0 && (!workspace || workspace_bytes < grad_workspace_bytes(n))) return TWELL_ERR_WORKSPACE;
  if (n > 0 && !al16(workspace)) return TWELL_ERR_ALIGN;
  GradArgs a;
  a.g = grads; a.out = outs; a.len = sizes; a.dtype = dtypes; a.out_dtype = out_dtypes;
  a.n = n; a.max_norm = max_norm; a.norm = norm; a.part = (double *)workspace;
  return hip_status(launch_grad(a, s));
}

int grad_norm(const void *const *grads, const int64_t *sizes, const int32_t *dtypes, int32_t n, float *norm,
              void *workspace, size_t workspace_bytes, void *stream) {
  return grad_run(grads, nullptr, sizes, dtypes, nullptr, n, 0.f, norm, workspace, workspace_bytes, S(stream));
}

int grad_clip(const void *const *grads, void *const *outs, const int64_t *sizes, const int32_t *dtypes,
              const int32_t *out_dtypes, int32_t n, float max_norm, float *norm, void *workspace,
              size_t workspace_bytes, void *stream) {
  if (!(max_norm >= 0.f) || (n > 0 && (!outs || !out_dtypes))) return TWELL_ERR_ARG;
  return grad_run(grads, outs, sizes, dtypes, out_dtypes, n, max_norm, norm, workspace, workspace_bytes, S(stream));
}

// ------------------------------------------------------------------------------ dense layers

static bool act_ok(int32_t act) { return act >= TWELL_ACT_NONE && act <= TWELL_ACT_GELU_TANH; }
static bool layout_ok(int32_t l) { return l == TWELL_W_NK || l == TWELL_W_KN; }

// rows of a tile are addressed with 32-bit byte offsets
static constexpr int kDenseMaxT = 1 << 24, kDenseMaxD = 1 << 20, kDenseMaxLd = 1 << 21;

static int dense_shape(int32_t T, int32_t a, int32_t b) {
  if (T < 0 || a <= 0 || b <= 0) return TWELL_ERR_SHAPE;
  if (a % 8 || b % 8) return TWELL_ERR_ALIGN;
  if (T > kDenseMaxT || a > kDenseMaxD || b > kDenseMaxD) return TWELL_ERR_UNSUPPORTED;
  return TWELL_OK;
}

// The stride of an operand's T rows of d (p NULL: not used).
static int dense_ld(const void *p, int64_t ld, int32_t T, int32_t d) {
  if (!p || T <= 1) return TWELL_OK;
  if (ld < d) return TWELL_ERR_SHAPE;
  if (ld % 8) return TWELL_ERR_ALIGN;
  return ld > kDenseMaxLd ? TWELL_ERR_UNSUPPORTED : TWELL_OK;
}

static int dense_ws(const void *ws, size_t bytes, size_t need) {
  if (need && (!ws || bytes < need)) return TWELL_ERR_WORKSPACE;
  return need && !al16(ws) ? TWELL_ERR_ALIGN : TWELL_OK;
}

size_t linear_fwd_workspace_bytes(int32_t T, int32_t d_in, int32_t d_out, int32_t dtype, int32_t w_layout) {
  if (T <= 0 || !dtype_ok(dtype) || !layout_ok(w_layout) || dense_shape(T, d_in, d_out) != TWELL_OK) return 0;
  return linear_fwd_workspace(T, d_in, d_out, dtype == TWELL_BF16, w_layout == TWELL_W_KN);
}

int linear_fwd(const void *x, int64_t ldx, const void *w, int32_t w_layout, const float *bias, const void *residual,
               int64_t ldr, int32_t dtype, int32_t T, int32_t d_in, int32_t d_out, int32_t act, void *y, int32_t y_dtype,
               void *pre, void *workspace, size_t workspace_bytes, void *stream) {
  if (!w || (T > 0 && (!x || !y))) return TWELL_ERR_ARG;
  if (!dtype_ok(dtype) || !dtype_ok(y_dtype) || !act_ok(act) || !layout_ok(w_layout)) return TWELL_ERR_ARG;
  int st = dense_shape(T, d_in, d_out);
  if (st || (st = dense_ld(x, ldx, T, d_in)) || (st = dense_ld(residual, ldr, T, d_out))) return st;
  if (!al16(x) || !al16(w) || !al16(bias) || !al16(residual) || !al16(y) || !al16(pre)) return TWELL_ERR_ALIGN;
  if (T == 0) return TWELL_OK;
  st = dense_ws(workspace, workspace_bytes, linear_fwd_workspace_bytes(T, d_in, d_out, dtype, w_layout));
  if (st) return st;
  LinearArgs a = {};
  a.x = x; a.w = w; a.res = residual; a.bias = bias;
  a.ldx = T > 1 ? ldx : d_in; a.ldr = T > 1 ? ldr : d_out;
  a.T = T; a.K = d_in; a.N = d_out;
  a.bf16 = dtype == TWELL_BF16; a.y_bf16 = y_dtype == TWELL_BF16; a.kn = w_layout == TWELL_W_KN; a.act = act;
  a.y = y; a.pre = pre; a.ws = workspace;
  TW_TRY(launch_linear_fwd(a, S(stream)));
  return TWELL_OK;
}

size_t linear_bwd_workspace_bytes(int32_t T, int32_t d_in, int32_t d_out, int32_t dtype, int32_t w_layout, int32_t act,
                                  int32_t want_dx, int32_t want_dw, int32_t want_db) {
  if (T <= 0 || !dtype_ok(dtype) || !layout_ok(w_layout) || !act_ok(act) || dense_shape(T, d_in, d_out) != TWELL_OK) return 0;
  return linear_bwd_workspace(T, d_in, d_out, dtype == TWELL_BF16, w_layout == TWELL_W_KN, act, want_dx != 0, want_dw != 0,
                              want_db != 0);
}

int linear_bwd(const void *dy, int64_t lddy, const void *x, int64_t ldx, const void *w, int32_t w_layout, const void *pre,
               int32_t dtype, int32_t T, int32_t d_in, int32_t d_out, int32_t act, void *dx, void *dw, float *db,
               void *workspace, size_t workspace_bytes, void *stream) {
  if (!dtype_ok(dtype) || !act_ok(act) || !layout_ok(w_layout)) return TWELL_ERR_ARG;
  if (T > 0 && (dx || dw || db) && (!dy || (act != TWELL_ACT_NONE && !pre))) return TWELL_ERR_ARG;
  if (T > 0 && ((dx && !w) || (dw && !x))) return TWELL_ERR_ARG;
  int st = dense_shape(T, d_in, d_out);
  if (st || (st = dense_ld(dy, lddy, T, d_out)) || (st = dense_ld(dw ? x : nullptr, ldx, T, d_in))) return st;
  if (!dx && !dw && !db) return TWELL_OK;
  if (!al16(dy) || (dw && !al16(x)) || (dx && !al16(w)) || (act != TWELL_ACT_NONE && !al16(pre)) || !al16(dx) || !al16(dw) ||
      !al16(db))
    return TWELL_ERR_ALIGN;
  if (T > 0) {
    st = dense_ws(workspace, workspace_bytes,
                  linear_bwd_workspace_bytes(T, d_in, d_out, dtype, w_layout, act, dx != nullptr, dw != nullptr, db != nullptr));
    if (st) return st;
  }
  LinearBackArgs a = {};
  a.dy = dy; a.x = x; a.w = w; a.pre = pre;
  a.lddy = T > 1 ? lddy : d_out; a.ldx = T > 1 ? ldx : d_in;
  a.T = T; a.K = d_in; a.N = d_out;
  a.bf16 = dtype == TWELL_BF16; a.kn = w_layout == TWELL_W_KN; a.act = act;
  a.dx = dx; a.dw = dw; a.db = db; a.ws = workspace;
  TW_TRY(launch_linear_bwd(a, S(stream)));
  return TWELL_OK;
}

size_t ffn_gated_dense_fwd_workspace_bytes(int32_t T, int32_t d_model, int32_t d_ff, int32_t dtype) {
  if (T <= 0 || !dtype_ok(dtype) || dense_shape(T, d_model, d_ff) != TWELL_OK) return 0;
  return gated_fwd_workspace(T, d_model, d_ff, dtype == TWELL_BF16);
}

int ffn_gated_dense_fwd(const void *x, int64_t ldx, const void *wg, const void *wu, const void *w2, const float *bg,
                        const float *bu, const void *residual, int64_t ldr, int32_t dtype, int32_t T, int32_t d_model,
                        int32_t d_ff, int32_t act, void *y, int32_t y_dtype, void *g, void *u, void *workspace,
                        size_t workspace_bytes, void *stream) {
  if (!wg || !wu || !w2 || (T > 0 && (!x || !y)) || (g == nullptr) != (u == nullptr)) return TWELL_ERR_ARG;
  if (!dtype_ok(dtype) || !dtype_ok(y_dtype) || !act_ok(act)) return TWELL_ERR_ARG;
  int st = dense_shape(T, d_model, d_ff);
  if (st || (st = dense_ld(x, ldx, T, d_model)) || (st = dense_ld(residual, ldr, T, d_model))) return st;
  if (!al16(x) || !al16(wg) || !al16(wu) || !al16(w2) || !al16(bg) || !al16(bu) || !al16(residual) || !al16(y) || !al16(g) ||
      !al16(u))
    return TWELL_ERR_ALIGN;
  if (T == 0) return TWELL_OK;
  st = dense_ws(workspace, workspace_bytes, ffn_gated_dense_fwd_workspace_bytes(T, d_model, d_ff, dtype));
  if (st) return st;
  GatedArgs a = {};
  a.x = x; a.wg = wg; a.wu = wu; a.w2 = w2; a.res = residual; a.bg = bg; a.bu = bu;
  a.ldx = T > 1 ? ldx : d_model; a.ldr = T > 1 ? ldr : d_model;
  a.T = T; a.d = d_model; a.f = d_ff;
  a.bf16 = dtype == TWELL_BF16; a.y_bf16 = y_dtype == TWELL_BF16; a.act = act;
  a.y = y; a.g = g; a.u = u; a.ws = workspace;
  TW_TRY(launch_gated_fwd(a, S(stream)));
  return TWELL_OK;
}

size_t ffn_gated_dense_bwd_workspace_bytes(int32_t T, int32_t d_model, int32_t d_ff, int32_t dtype, int32_t want_bias) {
  if (T <= 0 || !dtype_ok(dtype) || dense_shape(T, d_model, d_ff) != TWELL_OK) return 0;
  return gated_bwd_workspace(T, d_model, d_ff, dtype == TWELL_BF16, want_bias != 0);
}

int ffn_gated_dense_bwd(const void *dy, int64_t lddy, const void *x, int64_t ldx, const void *wg, const void *wu,
                        const void *w2, const void *g, const void *u, int32_t dtype, int32_t T, int32_t d_model,
                        int32_t d_ff, int32_t act, void *dx, void *dwg, void *dwu, void *dw2, float *dbg, float *dbu,
                        void *workspace, size_t workspace_bytes, void *stream) {
  if (!wg || !wu || !w2 || !dwg || !dwu || !dw2 || (T > 0 && (!dy || !x || !g || !u || !dx))) return TWELL_ERR_ARG;
  if (!dtype_ok(dtype) || !act_ok(act)) return TWELL_ERR_ARG;
  int st = dense_shape(T, d_model, d_ff);
  if (st || (st = dense_ld(dy, lddy, T, d_model)) || (st = dense_ld(x, ldx, T, d_model))) return st;
  if (!al16(dy) || !al16(x) || !al16(wg) || !al16(wu) || !al16(w2) || !al16(g) || !al16(u) || !al16(dx) || !al16(dwg) ||
      !al16(dwu) || !al16(dw2) || !al16(dbg) || !al16(dbu))
    return TWELL_ERR_ALIGN;
  if (T > 0) {
    st = dense_ws(workspace, workspace_bytes, ffn_gated_dense_bwd_workspace_bytes(T, d_model, d_ff, dtype, dbg || dbu));
    if (st) return st;
  }
  GatedBackArgs a = {};
  a.dy = dy; a.x = x; a.wg = wg; a.wu = wu; a.w2 = w2; a.g = g; a.u = u;
  a.lddy = T > 1 ? lddy : d_model; a.ldx = T > 1 ? ldx : d_model;
  a.T = T; a.d = d_model; a.f = d_ff; a.bf16 = dtype == TWELL_BF16; a.act = act;
  a.dx = dx; a.dwg = dwg; a.dwu = dwu; a.dw2 = dw2; a.dbg = dbg; a.dbu = dbu; a.ws = workspace;
  TW_TRY(launch_gated_bwd(a, S(stream)));
  return TWELL_OK;
}

// ------------------------------------------------------------------------------------- AdamW

namespace {
struct Span {
  uintptr_t at, end;
};
// Host memory for up to 256 spans without the heap, which a step of 40 tensors stays below.
struct Spans {
  Span few[256], *p = few;
  int n = 0;
  explicit Spans(size_t most) {
    if (most > 256) p = new (std::nothrow) Span[most];
  }
  ~Spans() {
    if (p != few) delete[] p;
  }
  void add(const void *q, int64_t bytes) {
    if (q && bytes > 0) p[n++] = {(uintptr_t)q, (uintptr_t)q + (uintptr_t)bytes};
  }
  void sort() {
    std::sort(p, p + n, [](const Span &a, const Span &b) { return a.at < b.at; });
  }
  bool apart() const {
    for (int k = 1; k < n; ++k)
      if (p[k - 1].end > p[k].at) return false;
    return true;
  }
  // no span reaches into [q, q + bytes) (sorted and apart)
  bool clear_of(const void *q, int64_t bytes) const {
    if (!q || bytes <= 0) return true;
    const uintptr_t at = (uintptr_t)q, end = at + (uintptr_t)bytes;
    const Span *s = std::lower_bound(p, p + n, end, [](const Span &a, uintptr_t e) { return a.at < e; });
    return s == p || s[-1].end <= at;
  }
};
}  // namespace

static int64_t bytes_of(int64_t n, int32_t dtype) { return n * (dtype == TWELL_BF16 ? 2 : 4); }
static bool aligned(const void *p, int32_t dtype) { return (uintptr_t)p % (dtype == TWELL_BF16 ? 2 : 4) == 0; }
static int64_t adamw_blocks(int64_t n) { return (n + TWELL_ADAMW_BLOCK - 1) / TWELL_ADAMW_BLOCK; }
static_assert(TWELL_ADAMW_BLOCK == kAdamBlock, "block");

int adamw_step(void *const *params, const void *const *grads, void *const *m, void *const *v, float *const *m_scales,
               float *const *v_scales, void *const *copies, const int64_t *sizes, const int32_t *dtypes,
               const int32_t *grad_dtypes, const double *weight_decay, int32_t n, int32_t state_bits, double lr,
               const float *lr_dev, double beta1, double beta2, double eps, int64_t step, const int64_t *step_dev,
               const float *norm, float max_norm, void *stream) {
  if (n < 0) return TWELL_ERR_SHAPE;
  if (state_bits != 8 && state_bits != 32) return TWELL_ERR_ARG;
  const bool eight = state_bits == 8;
  if (n > 0 && (!params || !grads || !m || !v || !sizes || !dtypes || !grad_dtypes || !weight_decay)) return TWELL_ERR_ARG;
  if (n > 0 && eight && (!m_scales || !v_scales)) return TWELL_ERR_ARG;
  if (!lr_dev && !(lr >= 0.0 && lr <= 1e30)) return TWELL_ERR_ARG;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0)) return TWELL_ERR_ARG;
  if (!(eps >= 1.17549435e-38 && eps <= 1e30)) return TWELL_ERR_ARG;        // not zero in fp32
  if (!step_dev && step < 1) return TWELL_ERR_ARG;
  if (norm && !(max_norm >= 0.f)) return TWELL_ERR_ARG;
  if (!al4(lr_dev) || !al4(norm) || ((uintptr_t)step_dev & 7u)) return TWELL_ERR_ALIGN;
  int64_t total = 0;
  for (int i = 0; i < n; ++i) {
    if (sizes[i] < 0) return TWELL_ERR_SHAPE;
    if (!dtype_ok(dtypes[i]) || !dtype_ok(grad_dtypes[i])) return TWELL_ERR_ARG;
    if (!(weight_decay[i] >= 0.0 && weight_decay[i] <= 1e30)) return TWELL_ERR_ARG;
    if (sizes[i] == 0) continue;
    if (!params[i] || !grads[i] || !m[i] || !v[i] || (eight && (!m_scales[i] || !v_scales[i]))) return TWELL_ERR_ARG;
    if (copies && copies[i] && dtypes[i] != TWELL_F32) return TWELL_ERR_ARG;
    if (!aligned(params[i], dtypes[i]) || !aligned(grads[i], grad_dtypes[i])) return TWELL_ERR_ALIGN;
    if (copies && !aligned(copies[i], TWELL_BF16)) return TWELL_ERR_ALIGN;
    if (eight ? !al4(m_scales[i]) || !al4(v_scales[i]) : !al4(m[i]) || !al4(v[i])) return TWELL_ERR_ALIGN;
    // chunks of the whole set are counted in 32 bits
    if (sizes[i] > ((int64_t)1 << 40) || (total += sizes[i]) > ((int64_t)1 << 40)) return TWELL_ERR_UNSUPPORTED;
  }
  // workgroups run in no order: an element that two of them write, or one writes and another reads, would
  // come out either way
  Spans out((size_t)n * 6);
  if (!out.p) return TWELL_ERR_HIP;         // no host memory
  for (int i = 0; i < n; ++i) {
    if (sizes[i] == 0) continue;
    const int64_t state = eight ? sizes[i] : sizes[i] * 4, scales = adamw_blocks(sizes[i]) * 4;
    out.add(params[i], bytes_of(sizes[i], dtypes[i]));
    out.add(m[i], state);
    out.add(v[i], state);
    if (copies) out.add(copies[i], sizes[i] * 2);
    if (eight) {
      out.add(m_scales[i], scales);
      out.add(v_scales[i], scales);
    }
  }
  out.sort();
  bool ok = out.apart() && out.clear_of(norm, 4) && out.clear_of(lr_dev, 4) && out.clear_of(step_dev, 8);
  for (int i = 0; ok && i < n; ++i) ok = out.clear_of(grads[i], bytes_of(sizes[i], grad_dtypes[i]));
  if (!ok) return TWELL_ERR_ARG;
  AdamArgs a = {};
  a.p = params; a.g = grads; a.m = m; a.v = v; a.copy = copies; a.ms = m_scales; a.vs = v_scales;
  a.len = sizes; a.p_dtype = dtypes; a.g_dtype = grad_dtypes; a.decay = weight_decay;
  a.n = n; a.eight = eight;
  a.lr = lr; a.beta1 = beta1; a.beta2 = beta2; a.eps = eps; a.step = step;
  a.lr_dev = lr_dev; a.step_dev = step_dev; a.norm = norm; a.max_norm = max_norm;
  TW_TRY(launch_adamw(a, S(stream)));
  return TWELL_OK;
}

int adamw8_values(const void *const *codes, const float *const *scales, const int32_t *second, const int64_t *sizes,
                  int32_t n, void *const *outs, int32_t out_dtype, void *stream) {
  if (n < 0) return TWELL_ERR_SHAPE;
  if (!dtype_ok(out_dtype) || (n > 0 && (!codes || !scales || !second || !sizes || !outs))) return TWELL_ERR_ARG;
  int64_t total = 0;
  for (int i = 0; i < n; ++i) {
    if (sizes[i] < 0) return TWELL_ERR_SHAPE;
    if (sizes[i] == 0) continue;
    if (!codes[i] || !scales[i] || !outs[i]) return TWELL_ERR_ARG;
    if (!al4(scales[i]) || !aligned(outs[i], out_dtype)) return TWELL_ERR_ALIGN;
    if (sizes[i] > ((int64_t)1 << 40) || (total += sizes[i]) > ((int64_t)1 << 40)) return TWELL_ERR_UNSUPPORTED;
  }
  Spans out((size_t)n);
  if (!out.p) return TWELL_ERR_HIP;
  for (int i = 0; i < n; ++i)
    if (sizes[i]) out.add(outs[i], bytes_of(sizes[i], out_dtype));
  out.sort();
  bool ok = out.apart();
  for (int i = 0; ok && i < n; ++i)
    ok = sizes[i] == 0 || (out.clear_of(codes[i], sizes[i]) && out.clear_of(scales[i], adamw_blocks(sizes[i]) * 4));
  if (!ok) return TWELL_ERR_ARG;
  AdamValuesArgs a = {};
  a.codes = codes; a.scales = scales; a.second = second; a.len = sizes; a.n = n;
  a.out = outs; a.out_bf16 = out_dtype == TWELL_BF16;
  TW_TRY(launch_adamw8_values(a, S(stream)));
  return TWELL_OK;
}

int twell_sync_status(const twell_matrix_t *h, void *stream) {
  if (!h || !h->ovf_n) return TWELL_ERR_ARG;
  if (hipStreamSynchronize(S(stream)) != hipSuccess) return TWELL_ERR_HIP;
  int32_t n = 0;
  if (hipMemcpy(&n, h->ovf_n, sizeof(n), hipMemcpyDeviceToHost) != hipSuccess) return TWELL_ERR_HIP;
  return n > h->ovf_cap ? TWELL_ERR_OVF_CAPACITY : TWELL_OK;
}

}  // extern "C"
