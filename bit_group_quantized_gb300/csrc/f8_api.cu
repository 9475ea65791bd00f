// f8_api.cu — the e4m3 entry points of the C ABI (include/bgq.h): argument
// checks, then the launches of f8_quant.cu and f8_product.cu.
#include <math.h>

#include "f8.h"
#include "kernels.h"
#include "overlap.h"

using namespace bgq;

namespace {

constexpr int kMaxCols = 65536, kMaxRows = (1 << 24) - 1, kMaxOut = 1 << 20;

inline bool al(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline cudaStream_t st(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? BGQ_OK : BGQ_ERR_CUDA; }

// An e4m3 matrix with scales for `block_rows` rows each (0: either).
int check_f8(const bgq_f8matrix* m, int block_rows) {
  if (!m || !m->q || !m->scale || !al(m->q, 16) || !al(m->scale, 4)) return BGQ_ERR_INVALID_ARG;
  if (m->rows < 0 || m->cols < 16 || m->cols % 16) return BGQ_ERR_INVALID_ARG;
  if (m->block_rows != 1 && m->block_rows != kF8Block) return BGQ_ERR_INVALID_ARG;
  if (block_rows && m->block_rows != block_rows) return BGQ_ERR_INVALID_ARG;
  if (m->cols > kMaxCols || m->rows > kMaxRows) return BGQ_ERR_UNSUPPORTED;
  if (m->q_stride < m->cols || m->q_stride % 16 || m->scale_stride % 4 || m->scale_stride < (f8_blocks(m->cols) + 3) / 4 * 4)
    return BGQ_ERR_INVALID_ARG;
  if (m->q_stride >= (int64_t)1 << 36 || m->scale_stride >= (int64_t)1 << 36) return BGQ_ERR_UNSUPPORTED;
  return BGQ_OK;
}

int check_product(const bgq_f8matrix* W, const bgq_f8matrix* x) {
  int r = check_f8(W, kF8Block);
  if (r || (r = check_f8(x, 1))) return r;
  if (W->rows < 1 || W->cols != x->cols) return BGQ_ERR_INVALID_ARG;
  if (W->rows > kMaxOut) return BGQ_ERR_UNSUPPORTED;
  return BGQ_OK;
}

int check_out(const void* y, int64_t stride, int64_t width) {
  if (!al(y, 16)) return BGQ_ERR_INVALID_ARG;
  if (y && (stride < width || stride % 8)) return BGQ_ERR_INVALID_ARG;
  if (y && stride >= (int64_t)1 << 36) return BGQ_ERR_UNSUPPORTED;
  return BGQ_OK;
}

// What a call reads and writes of a matrix, and of `size` bytes a value elsewhere.
Rows codes(const bgq_f8matrix& m) { return {m.q, m.rows, m.cols, m.q_stride}; }
Rows scales(const bgq_f8matrix& m) {
  return {m.scale, ((int64_t)m.rows + m.block_rows - 1) / m.block_rows, f8_blocks(m.cols), m.scale_stride};
}
Rows values(const void* p, int64_t rows, int64_t width, int64_t stride, int size) { return {p, rows, width * size, stride * size}; }

constexpr size_t kWsBytes = sizeof(Ctrl);

F8Prod product(const bgq_f8matrix* W, const bgq_f8matrix* up, const bgq_f8matrix* x, uint16_t* y, float* yf,
               int64_t y_stride, void* ws) {
  F8Prod p = {};
  const bgq_f8matrix* both[2] = {W, up ? up : W};
  for (int i = 0; i < 2; ++i) {
    p.w[i] = both[i]->q;
    p.ws[i] = both[i]->scale;
    p.w_stride[i] = both[i]->q_stride;
    p.ws_stride[i] = both[i]->scale_stride;
  }
  p.x = x->q;
  p.xs = x->scale;
  p.x_stride = x->q_stride;
  p.xs_stride = x->scale_stride;
  p.M = x->rows;
  p.N = W->rows;
  p.K = x->cols;
  p.y = y;
  p.yf = yf;
  p.y_stride = y_stride;
  p.ctrl = static_cast<Ctrl*>(ws);
  return p;
}

}  // namespace

extern "C" {

int32_t bgq_f8_quantise(const uint16_t* x, int64_t x_stride, const bgq_f8matrix* m, void* stream) {
  const int r = check_f8(m, 0);
  if (r) return r;
  if (!x || !al(x, 16) || x_stride < m->cols || x_stride % 8) return BGQ_ERR_INVALID_ARG;
  if (x_stride >= (int64_t)1 << 36) return BGQ_ERR_UNSUPPORTED;
  if (m->rows == 0) return BGQ_OK;
  if (overlap({codes(*m), scales(*m)}, {values(x, m->rows, m->cols, x_stride, 2)})) return BGQ_ERR_INVALID_ARG;
  return cuda_status(launch_f8_quantise(x, x_stride, *m, st(stream)));
}

int32_t bgq_rmsnorm_f8(float* h, const void* delta, int32_t delta_f32, const uint16_t* rho, int32_t batch, int32_t d,
                       float eps, const bgq_f8matrix* m, uint16_t* a, void* stream) {
  const int r = check_f8(m, 1);
  if (r) return r;
  if (!h || !al(h, 16) || !al(delta, 16) || !al(rho, 16) || !al(a, 16)) return BGQ_ERR_INVALID_ARG;
  if (batch != m->rows || d != m->cols || !(eps >= 0.f)) return BGQ_ERR_INVALID_ARG;
  if (batch == 0) return BGQ_OK;
  if (overlap({values(h, batch, d, d, 4), codes(*m), scales(*m), values(a, batch, d, d, 2)},
              {values(delta, batch, d, d, delta_f32 ? 4 : 2), values(rho, 1, d, d, 2)}))
    return BGQ_ERR_INVALID_ARG;
  return cuda_status(launch_rmsnorm_f8(h, delta, delta_f32 != 0, rho, eps, *m, a, st(stream)));
}

size_t bgq_f8_gemm_workspace_bytes(const bgq_f8matrix* W, const bgq_f8matrix* x) {
  return check_product(W, x) ? 0 : kWsBytes;
}

int32_t bgq_f8_gemm(const bgq_f8matrix* W, const bgq_f8matrix* x, uint16_t* y, float* y_f32, int64_t y_stride,
                    void* ws, size_t ws_bytes, void* stream) {
  int r = check_product(W, x);
  if (r || (r = check_out(y, y_stride, W->rows)) || (r = check_out(y_f32, y_stride, W->rows))) return r;
  if (!y && !y_f32) return BGQ_ERR_INVALID_ARG;
  if (!ws || !al(ws, 256) || ws_bytes < kWsBytes) return BGQ_ERR_WORKSPACE;
  if (x->rows == 0) return BGQ_OK;
  if (overlap({values(y, x->rows, W->rows, y_stride, 2), values(y_f32, x->rows, W->rows, y_stride, 4)},
              {codes(*x), scales(*x), codes(*W), scales(*W)}))
    return BGQ_ERR_INVALID_ARG;
  return cuda_status(launch_f8_product(product(W, nullptr, x, y, y_f32, y_stride, ws), false, st(stream)));
}

int32_t bgq_f8_swiglu(const bgq_f8matrix* gate, const bgq_f8matrix* up, const bgq_f8matrix* x, const bgq_f8matrix* h,
                      uint16_t* y, int64_t y_stride, void* ws, size_t ws_bytes, void* stream) {
  int r = check_product(gate, x);
  if (r || (r = check_product(up, x)) || (r = check_out(y, y_stride, gate->rows))) return r;
  if (gate->rows != up->rows || gate->rows % 16 || (!h && !y)) return BGQ_ERR_INVALID_ARG;
  if (h && (r = check_f8(h, 1))) return r;
  if (h && (h->rows != x->rows || h->cols != gate->rows)) return BGQ_ERR_INVALID_ARG;
  if (!ws || !al(ws, 256) || ws_bytes < kWsBytes) return BGQ_ERR_WORKSPACE;
  if (x->rows == 0) return BGQ_OK;
  const Rows none = {};
  if (overlap({values(y, x->rows, gate->rows, y_stride, 2), h ? codes(*h) : none, h ? scales(*h) : none},
              {codes(*x), scales(*x), codes(*gate), scales(*gate), codes(*up), scales(*up)}))
    return BGQ_ERR_INVALID_ARG;
  F8Prod p = product(gate, up, x, y, nullptr, y_stride, ws);
  if (h) {
    p.h = h->q;
    p.hs = h->scale;
    p.h_stride = h->q_stride;
    p.hs_stride = h->scale_stride;
  }
  return cuda_status(launch_f8_product(p, true, st(stream)));
}

}  // extern "C"
