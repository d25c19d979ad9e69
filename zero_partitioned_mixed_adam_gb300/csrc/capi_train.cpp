// capi_train.cpp -- the extern "C" entry points of a training step around the ZeRO step
// (linear maps, the gradient norm, AdamW over a list of tensors, embedding, cross
// entropy, block norms): argument checks, scalars, dispatch.
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "capi_common.hpp"
#include "train_ops.cuh"
#include "zeroadam.h"

namespace zeroadam {
namespace {

bool misaligned(const void* p, uintptr_t k) {
  return (reinterpret_cast<uintptr_t>(p) & (k - 1)) != 0;
}

// A row-major matrix's place in memory; base NULL: none.
struct Matrix {
  const void* base;
  int64_t rows, cols, ld;
  int esize;
};

bool empty(const Matrix& m) { return m.base == nullptr || m.rows < 1 || m.cols < 1; }

Range span(const Matrix& m) {
  return bytes_of(m.base, 0, (m.rows - 1) * m.ld + m.cols, m.esize);
}

// Whether two matrices share an element.  Matrices of one pitch may lie side by
// side in a wider one (the q, k and v columns of a joint projection): then their
// spans overlap but no element does.
bool share(const Matrix& a, const Matrix& b) {
  if (empty(a) || empty(b) || !overlap(span(a), span(b))) return false;
  if (a.ld * a.esize == b.ld * b.esize) {
    const int64_t pitch = a.ld * a.esize;
    const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.base) -
                                           reinterpret_cast<uintptr_t>(a.base));
    const int64_t off = ((d % pitch) + pitch) % pitch;  // b's first column, from a's
    if (off >= a.cols * a.esize && off + b.cols * b.esize <= pitch) return false;
  }
  return true;
}

constexpr int64_t kMostSide = INT32_MAX;
constexpr int64_t kMostElements = INT64_MAX / 16;

int check_shape(const zero_linear_t* s) {
  if (s == nullptr) return ZERO_E_NULLPTR;
  if (s->rows < 0 || s->in < 1 || s->out < 1 || s->rows >= kMostSide || s->in >= kMostSide ||
      s->out >= kMostSide)
    return ZERO_E_SHAPE;
  return ZERO_OK;
}

int check_matrix(const Matrix& m) {
  if (m.base == nullptr) return ZERO_OK;
  if (m.ld < m.cols || (m.rows > 0 && m.ld > kMostElements / m.rows)) return ZERO_E_SHAPE;
  return misaligned(m.base, static_cast<uintptr_t>(m.esize)) ? ZERO_E_ALIGN : ZERO_OK;
}

// Whether the kernel can read a matrix, or a bias, where it lies (ZERO_LINEAR_ALIGNED).
bool in_place(const Matrix& m) {
  return m.base == nullptr || (!misaligned(m.base, 16) && (m.rows <= 1 || m.ld % 8 == 0));
}

bool known_act(int32_t act) { return act >= ZERO_ACT_NONE && act <= ZERO_ACT_SILU; }

int check_workspace(const void* p, int64_t have, int64_t need) {
  if (need == 0) return ZERO_OK;
  return p == nullptr || misaligned(p, 16) || have < need ? ZERO_E_WORKSPACE : ZERO_OK;
}

int check_step_scalars(double lr, double beta1, double beta2, double eps, int64_t t) {
  if (!std::isfinite(lr) || !std::isfinite(eps) || !std::isfinite(beta1) ||
      !std::isfinite(beta2) || lr < 0.0 || eps < 0.0 || beta1 < 0.0 || beta1 >= 1.0 ||
      beta2 < 0.0 || beta2 >= 1.0)
    return ZERO_E_HPARAM;
  return t < 1 ? ZERO_E_STEP : ZERO_OK;
}

constexpr int64_t kMostNumel = int64_t{1} << 40;

int check_sides(int64_t rows, int64_t width, int64_t vocab) {
  if (rows < 0 || width < 1 || vocab < 1 || rows >= kMostSide || width >= kMostSide ||
      vocab >= kMostSide)
    return ZERO_E_SHAPE;
  return ZERO_OK;
}

// A list of ids, as a row.
Matrix ids_row(const void* ids, int64_t rows, int32_t flags) {
  return Matrix{ids, 1, rows, rows, (flags & ZERO_IDS_I32) ? 4 : 8};
}

int check_embedding(const zero_embedding_t* s, const Matrix& from, const Matrix& ids, const Matrix& to,
                    double scale) {
  if (!std::isfinite(scale) || std::fabs(scale) > FLT_MAX) return ZERO_E_HPARAM;
  for (const Matrix* m : {&from, &ids, &to}) {
    const int rc = check_matrix(*m);
    if (rc != ZERO_OK) return rc;
  }
  return share(to, from) || share(to, ids) ? ZERO_E_ALIAS : ZERO_OK;
}

// A matrix of the block norms, whose kernels count a row's bytes in 32 bits.
int check_rows(const Matrix& m) {
  return m.base != nullptr && m.ld > kMostSide ? ZERO_E_SHAPE : check_matrix(m);
}

bool norm_kind(int32_t kind) { return kind == ZERO_NORM_RMS || kind == ZERO_NORM_LAYER; }

// What the two directions of the block norms share.
int check_block_norm(const zero_block_norm_t* s) {
  if (s == nullptr) return ZERO_E_NULLPTR;
  if (s->rows < 0 || s->rows >= kMostSide || s->width < 1 || s->width > ZERO_MAX_NORM_WIDTH)
    return ZERO_E_SHAPE;
  return ZERO_OK;
}
int check_block_norm_inputs(const zero_block_norm_t& s, const void* h, const void* post_weight,
                            const void* post_bias, const void* gate, const void* bias) {
  if (!norm_kind(s.kind) || (s.post != ZERO_NORM_NONE && !norm_kind(s.post))) return ZERO_E_LAYOUT;
  if (h == nullptr && s.rows > 0 && (s.post != ZERO_NORM_NONE || gate != nullptr)) return ZERO_E_LAYOUT;
  if (s.post == ZERO_NORM_NONE && post_weight != nullptr) return ZERO_E_LAYOUT;
  if (s.post != ZERO_NORM_LAYER && post_bias != nullptr) return ZERO_E_LAYOUT;
  if (s.kind != ZERO_NORM_LAYER && bias != nullptr) return ZERO_E_LAYOUT;
  if (!std::isfinite(s.alpha) || std::fabs(s.alpha) > FLT_MAX || !std::isfinite(s.eps) || s.eps < 0.0 ||
      s.eps > FLT_MAX)
    return ZERO_E_HPARAM;
  return ZERO_OK;
}

}  // namespace
}  // namespace zeroadam

using namespace zeroadam;

extern "C" {

int64_t zero_linear_workspace(const zero_linear_t* shape, int32_t flags) {
  const int rc = check_shape(shape);
  if (rc != ZERO_OK) return rc;
  if ((flags & ~(ZERO_LINEAR_BACKWARD | ZERO_LINEAR_ALIGNED | ZERO_LINEAR_PLAIN)) != 0)
    return ZERO_E_LAYOUT;
  return linear_workspace(*shape, flags);
}

int zero_linear_forward(const zero_linear_t* shape, const void* x, const void* w,
                        const void* bias, int32_t act, const void* residual, void* pre, void* y,
                        void* workspace, int64_t workspace_bytes, void* stream) {
  Trace trace("zero_linear_forward");
  int rc = check_shape(shape);
  if (rc != ZERO_OK) return rc;
  if (w == nullptr || (shape->rows > 0 && (x == nullptr || y == nullptr))) return ZERO_E_NULLPTR;
  if (!known_act(act)) return ZERO_E_LAYOUT;
  const zero_linear_t& s = *shape;
  const Matrix mx{x, s.rows, s.in, s.ldx, 2}, mw{w, s.out, s.in, s.ldw, 2},
      mb{bias, 1, s.out, s.out, 2}, mr{residual, s.rows, s.out, s.ldr, 2},
      mp{pre, s.rows, s.out, s.ldp, 2}, my{y, s.rows, s.out, s.ldy, 2};
  for (const Matrix* m : {&mx, &mw, &mb, &mr, &mp, &my})
    if ((rc = check_matrix(*m)) != ZERO_OK) return rc;
  for (const Matrix* m : {&mx, &mw, &mb})
    if (share(my, *m) || share(mp, *m)) return ZERO_E_ALIAS;
  if (share(my, mp) || share(mp, mr)) return ZERO_E_ALIAS;
  if (!(residual == y && s.ldr == s.ldy) && share(my, mr)) return ZERO_E_ALIAS;
  const int64_t need = linear_workspace(
      s, in_place(mx) && in_place(mw) && in_place(mb) ? ZERO_LINEAR_ALIGNED : 0);
  if ((rc = check_workspace(workspace, workspace_bytes, need)) != ZERO_OK) return rc;
  const Matrix ms{need > 0 ? workspace : nullptr, 1, need, need, 1};
  for (const Matrix* m : {&mx, &mw, &mb, &mr, &mp, &my})
    if (share(ms, *m)) return ZERO_E_ALIAS;
  if (s.rows == 0) return ZERO_OK;
  LinearForwardLaunch L;
  L.s = s;
  L.x = static_cast<const uint16_t*>(x);
  L.w = static_cast<const uint16_t*>(w);
  L.bias = static_cast<const uint16_t*>(bias);
  L.residual = static_cast<const uint16_t*>(residual);
  L.act = act;
  L.pre = static_cast<uint16_t*>(pre);
  L.y = static_cast<uint16_t*>(y);
  L.workspace = workspace;
  L.stream = static_cast<cudaStream_t>(stream);
  L.withhold = withhold_copies();
  return launch_status(launch_linear_forward(L));
}

int zero_linear_backward(const zero_linear_t* shape, const void* dy, const void* x, const void* w,
                         int32_t act, const void* pre, int32_t act_in, const void* pre_in,
                         void* dx, void* dw, void* dbias, int32_t flags, void* workspace,
                         int64_t workspace_bytes, void* stream) {
  Trace trace("zero_linear_backward");
  int rc = check_shape(shape);
  if (rc != ZERO_OK) return rc;
  if (!known_act(act) || !known_act(act_in)) return ZERO_E_LAYOUT;
  if ((flags & ~(ZERO_GRAD_F32 | ZERO_GRAD_ACCUMULATE)) != 0) return ZERO_E_LAYOUT;
  if (dx != nullptr && w == nullptr) return ZERO_E_NULLPTR;
  if (shape->rows > 0 &&
      (dy == nullptr || (dw != nullptr && x == nullptr) ||
       (act != ZERO_ACT_NONE && pre == nullptr) ||
       (dx != nullptr && act_in != ZERO_ACT_NONE && pre_in == nullptr)))
    return ZERO_E_NULLPTR;
  const zero_linear_t& s = *shape;
  const int gsize = (flags & ZERO_GRAD_F32) ? 4 : 2;
  const Matrix mdy{dy, s.rows, s.out, s.ldy, 2}, mx{dw != nullptr ? x : nullptr, s.rows, s.in, s.ldx, 2},
      mw{dx != nullptr ? w : nullptr, s.out, s.in, s.ldw, 2},
      mp{act != ZERO_ACT_NONE ? pre : nullptr, s.rows, s.out, s.ldp, 2},
      mi{dx != nullptr && act_in != ZERO_ACT_NONE ? pre_in : nullptr, s.rows, s.in, s.ldpi, 2},
      mdx{dx, s.rows, s.in, s.lddx, 2}, mdw{dw, s.out, s.in, s.lddw, gsize},
      mdb{dbias, 1, s.out, s.out, gsize};
  for (const Matrix* m : {&mdy, &mx, &mw, &mp, &mi, &mdx, &mdw, &mdb})
    if ((rc = check_matrix(*m)) != ZERO_OK) return rc;
  for (const Matrix* o : {&mdx, &mdw, &mdb})
    for (const Matrix* m : {&mdy, &mx, &mw, &mp, &mi})
      if (share(*o, *m)) return ZERO_E_ALIAS;
  if (share(mdx, mdw) || share(mdx, mdb) || share(mdw, mdb)) return ZERO_E_ALIAS;
  const int64_t need = linear_workspace(
      s, ZERO_LINEAR_BACKWARD | (act == ZERO_ACT_NONE ? ZERO_LINEAR_PLAIN : 0) |
             (in_place(mdy) && in_place(mx) && in_place(mw) ? ZERO_LINEAR_ALIGNED : 0));
  if ((rc = check_workspace(workspace, workspace_bytes, need)) != ZERO_OK) return rc;
  const Matrix ms{need > 0 ? workspace : nullptr, 1, need, need, 1};
  for (const Matrix* m : {&mdy, &mx, &mw, &mp, &mi, &mdx, &mdw, &mdb})
    if (share(ms, *m)) return ZERO_E_ALIAS;
  LinearBackwardLaunch L{};
  L.s = s;
  L.dy = static_cast<const uint16_t*>(dy);
  L.x = static_cast<const uint16_t*>(x);
  L.w = static_cast<const uint16_t*>(w);
  L.pre = static_cast<const uint16_t*>(pre);
  L.pre_in = static_cast<const uint16_t*>(pre_in);
  L.act = act;
  L.act_in = act_in;
  L.dx = static_cast<uint16_t*>(dx);
  L.dw = dw;
  L.dbias = dbias;
  L.grad_f32 = (flags & ZERO_GRAD_F32) ? 1 : 0;
  L.accumulate = (flags & ZERO_GRAD_ACCUMULATE) ? 1 : 0;
  L.workspace = workspace;
  L.stream = static_cast<cudaStream_t>(stream);
  L.withhold = withhold_copies();
  return launch_status(launch_linear_backward(L));
}

int64_t zero_grad_norm_workspace(void) { return kNormWorkspace; }

int zero_grad_norm(int32_t ntensors, const void* const* grads, const int64_t* numels,
                   int32_t flags, double max_norm, float* out, void* workspace,
                   int64_t workspace_bytes, void* stream) {
  Trace trace("zero_grad_norm");
  if (ntensors < 0 || ntensors > ZERO_MAX_LIST) return ZERO_E_SHAPE;
  if ((flags & ~ZERO_GRAD_F32) != 0) return ZERO_E_LAYOUT;
  if (!std::isfinite(max_norm) || max_norm < 0.0) return ZERO_E_HPARAM;
  if (out == nullptr || (ntensors > 0 && (grads == nullptr || numels == nullptr)))
    return ZERO_E_NULLPTR;
  const int gsize = (flags & ZERO_GRAD_F32) ? 4 : 2;
  if (misaligned(out, 4)) return ZERO_E_ALIGN;
  const int rc = check_workspace(workspace, workspace_bytes, kNormWorkspace);
  if (rc != ZERO_OK) return rc;
  const Range ro = bytes_of(out, 0, 2, 4), rw = bytes_of(workspace, 0, kNormWorkspace, 1);
  if (overlap(ro, rw)) return ZERO_E_ALIAS;
  for (int32_t i = 0; i < ntensors; ++i) {
    if (numels[i] < 0 || numels[i] > kMostNumel) return ZERO_E_SHAPE;
    if (numels[i] == 0) continue;
    if (grads[i] == nullptr) return ZERO_E_NULLPTR;
    if (misaligned(grads[i], static_cast<uintptr_t>(gsize))) return ZERO_E_ALIGN;
    const Range g = bytes_of(grads[i], 0, numels[i], gsize);
    if (overlap(g, ro) || overlap(g, rw)) return ZERO_E_ALIAS;
  }
  NormLaunch L;
  L.ntensors = ntensors;
  L.grads = grads;
  L.numels = numels;
  L.grad_f32 = gsize == 4;
  L.max_norm = static_cast<float>(max_norm);
  L.out = out;
  L.workspace = workspace;
  L.stream = static_cast<cudaStream_t>(stream);
  return launch_status(launch_grad_norm(L));
}

int zero_adamw_step(int32_t ntensors, const zero_adamw_tensor_t* tensors, int32_t flags,
                    double lr, double beta1, double beta2, double eps, int64_t t,
                    const float* grad_scale, uint32_t seed, void* stream) {
  Trace trace("zero_adamw_step");
  if (ntensors < 0 || ntensors > ZERO_MAX_LIST) return ZERO_E_SHAPE;
  if ((flags & ~(ZERO_GRAD_F32 | ZERO_STATE_8BIT)) != 0) return ZERO_E_LAYOUT;
  const int rc = check_step_scalars(lr, beta1, beta2, eps, t);
  if (rc != ZERO_OK) return rc;
  if (ntensors > 0 && tensors == nullptr) return ZERO_E_NULLPTR;
  if (misaligned(grad_scale, 4)) return ZERO_E_ALIGN;
  const bool eight = (flags & ZERO_STATE_8BIT) != 0;
  const int gsize = (flags & ZERO_GRAD_F32) ? 4 : 2, ssize = eight ? 1 : 4;
  for (int32_t i = 0; i < ntensors; ++i) {
    const zero_adamw_tensor_t& x = tensors[i];
    if (x.numel < 0 || x.numel > kMostNumel) return ZERO_E_SHAPE;
    if (!std::isfinite(x.weight_decay) || x.weight_decay < 0.0) return ZERO_E_HPARAM;
    if (x.numel == 0) continue;
    if (x.grad == nullptr || x.master == nullptr || x.m == nullptr || x.v == nullptr ||
        (eight && (x.m_scale == nullptr || x.v_scale == nullptr)))
      return ZERO_E_NULLPTR;
    if (misaligned(x.grad, gsize) || misaligned(x.master, 4) || misaligned(x.param_bf16, 2) ||
        misaligned(x.m, ssize) || misaligned(x.v, ssize) ||
        (eight && (misaligned(x.m_scale, 4) || misaligned(x.v_scale, 4))))
      return ZERO_E_ALIGN;
    const int64_t blocks = eight ? (x.numel + ZERO_MOMENT_BLOCK - 1) / ZERO_MOMENT_BLOCK : 0;
    const Range r[8] = {bytes_of(x.grad, 0, x.numel, gsize), bytes_of(x.master, 0, x.numel, 4),
                        bytes_of(x.m, 0, x.numel, ssize), bytes_of(x.v, 0, x.numel, ssize),
                        bytes_of(x.param_bf16, 0, x.param_bf16 != nullptr ? x.numel : 0, 2),
                        bytes_of(x.m_scale, 0, blocks, 4), bytes_of(x.v_scale, 0, blocks, 4),
                        bytes_of(grad_scale, 0, grad_scale != nullptr ? 1 : 0, 4)};
    for (int a = 0; a < 8; ++a)
      for (int b = a + 1; b < 8; ++b)
        if (nonempty(r[a]) && nonempty(r[b]) && overlap(r[a], r[b]) && !(a == 0 && b == 7))
          return ZERO_E_ALIAS;
  }
  AdamwLaunch L;
  L.ntensors = ntensors;
  L.tensors = tensors;
  L.grad_f32 = gsize == 4;
  L.eight = eight;
  L.lr = lr;
  L.s.b1 = static_cast<float>(beta1);
  L.s.omb1 = static_cast<float>(1.0 - beta1);
  L.s.b2 = static_cast<float>(beta2);
  L.s.omb2 = static_cast<float>(1.0 - beta2);
  const double td = static_cast<double>(t);
  L.s.size = static_cast<float>(lr / (1.0 - std::pow(beta1, td)));
  L.s.inv_root = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(beta2, td)));
  L.s.eps = static_cast<float>(eps);
  L.grad_scale = grad_scale;
  L.seed = seed;
  L.stream = static_cast<cudaStream_t>(stream);
  return launch_status(launch_adamw(L));
}

int zero_adamw_state_f32(int32_t ntensors, const zero_adamw_tensor_t* tensors,
                         float* const* m_out, float* const* v_out, void* stream) {
  Trace trace("zero_adamw_state_f32");
  if (ntensors < 0 || ntensors > ZERO_MAX_LIST) return ZERO_E_SHAPE;
  if (ntensors > 0 && tensors == nullptr) return ZERO_E_NULLPTR;
  for (int32_t i = 0; i < ntensors; ++i) {
    const zero_adamw_tensor_t& x = tensors[i];
    if (x.numel < 0 || x.numel > kMostNumel) return ZERO_E_SHAPE;
    if (x.numel == 0) continue;
    const int64_t blocks = (x.numel + ZERO_MOMENT_BLOCK - 1) / ZERO_MOMENT_BLOCK;
    const Range in[4] = {bytes_of(x.m, 0, x.numel, 1), bytes_of(x.v, 0, x.numel, 1),
                         bytes_of(x.m_scale, 0, blocks, 4), bytes_of(x.v_scale, 0, blocks, 4)};
    Range out[2] = {{0, 0}, {0, 0}};
    for (int k = 0; k < 2; ++k) {
      float* const* o = k == 0 ? m_out : v_out;
      if (o == nullptr) continue;
      const void *codes = k == 0 ? x.m : x.v, *scale = k == 0 ? x.m_scale : x.v_scale;
      if (o[i] == nullptr || codes == nullptr || scale == nullptr) return ZERO_E_NULLPTR;
      if (misaligned(o[i], 4) || misaligned(scale, 4)) return ZERO_E_ALIGN;
      out[k] = bytes_of(o[i], 0, x.numel, 4);
      for (const Range& r : in)
        if (overlap(out[k], r)) return ZERO_E_ALIAS;
    }
    if (nonempty(out[0]) && nonempty(out[1]) && overlap(out[0], out[1])) return ZERO_E_ALIAS;
  }
  MomentsLaunch L;
  L.ntensors = ntensors;
  L.tensors = tensors;
  L.m_out = m_out;
  L.v_out = v_out;
  L.stream = static_cast<cudaStream_t>(stream);
  return launch_status(launch_adamw_moments(L));
}

int zero_embedding_forward(const zero_embedding_t* shape, const void* table, const void* ids,
                           int32_t flags, double scale, void* y, void* stream) {
  Trace trace("zero_embedding_forward");
  if (shape == nullptr) return ZERO_E_NULLPTR;
  const zero_embedding_t& s = *shape;
  int rc = check_sides(s.rows, s.width, s.vocab);
  if (rc != ZERO_OK) return rc;
  if ((flags & ~ZERO_IDS_I32) != 0) return ZERO_E_LAYOUT;
  if (table == nullptr || (s.rows > 0 && (ids == nullptr || y == nullptr))) return ZERO_E_NULLPTR;
  const Matrix mt{table, s.vocab, s.width, s.ldt, 2}, my{y, s.rows, s.width, s.ldy, 2};
  if ((rc = check_embedding(shape, mt, ids_row(ids, s.rows, flags), my, scale)) != ZERO_OK) return rc;
  if (s.rows == 0) return ZERO_OK;
  EmbeddingLaunch L{};
  L.s = s;
  L.from = static_cast<const uint16_t*>(table);
  L.ids = ids;
  L.ids_i32 = (flags & ZERO_IDS_I32) ? 1 : 0;
  L.scale = static_cast<float>(scale);
  L.to = y;
  L.stream = static_cast<cudaStream_t>(stream);
  return launch_status(launch_embedding_forward(L));
}

int zero_embedding_backward(const zero_embedding_t* shape, const void* dy, const void* ids,
                            int32_t flags, double scale, int64_t padding, void* dtable,
                            void* stream) {
  Trace trace("zero_embedding_backward");
  if (shape == nullptr) return ZERO_E_NULLPTR;
  const zero_embedding_t& s = *shape;
  int rc = check_sides(s.rows, s.width, s.vocab);
  if (rc != ZERO_OK) return rc;
  if ((flags & ~(ZERO_IDS_I32 | ZERO_GRAD_F32 | ZERO_GRAD_ACCUMULATE)) != 0) return ZERO_E_LAYOUT;
  if (dtable == nullptr || (s.rows > 0 && (ids == nullptr || dy == nullptr))) return ZERO_E_NULLPTR;
  const Matrix md{dy, s.rows, s.width, s.ldy, 2},
      mt{dtable, s.vocab, s.width, s.ldt, (flags & ZERO_GRAD_F32) ? 4 : 2};
  if ((rc = check_embedding(shape, md, ids_row(ids, s.rows, flags), mt, scale)) != ZERO_OK) return rc;
  if (s.rows == 0 && (flags & ZERO_GRAD_ACCUMULATE) != 0) return ZERO_OK;
  EmbeddingLaunch L{};
  L.s = s;
  L.from = static_cast<const uint16_t*>(dy);
  L.ids = ids;
  L.ids_i32 = (flags & ZERO_IDS_I32) ? 1 : 0;
  L.scale = static_cast<float>(scale);
  L.padding = padding;
  L.to = dtable;
  L.grad_f32 = (flags & ZERO_GRAD_F32) ? 1 : 0;
  L.accumulate = (flags & ZERO_GRAD_ACCUMULATE) ? 1 : 0;
  L.stream = static_cast<cudaStream_t>(stream);
  return launch_status(launch_embedding_backward(L));
}

int64_t zero_linear_cross_entropy_workspace(const zero_cross_entropy_t* shape, int32_t flags) {
  if (shape == nullptr) return ZERO_E_NULLPTR;
  const int rc = check_sides(shape->rows, shape->width, shape->vocab);
  if (rc != ZERO_OK) return rc;
  if ((flags & ~(ZERO_LINEAR_BACKWARD | ZERO_LINEAR_ALIGNED | ZERO_GRAD_F32)) != 0) return ZERO_E_LAYOUT;
  // (as the call refuses them with their pitches, so that no size below wraps)
  for (const int64_t n : {shape->rows, shape->vocab})
    if (n > 0 && shape->width > kMostElements / n) return ZERO_E_SHAPE;
  return cross_entropy_workspace(*shape, flags);
}

int zero_linear_cross_entropy(const zero_cross_entropy_t* shape, const void* x, const void* w,
                              const void* targets, int64_t ignore_index, const float* scale,
                              float* losses, float* total, void* dx, void* dw, int32_t flags,
                              void* workspace, int64_t workspace_bytes, void* stream) {
  Trace trace("zero_linear_cross_entropy");
  if (shape == nullptr) return ZERO_E_NULLPTR;
  const zero_cross_entropy_t& s = *shape;
  int rc = check_sides(s.rows, s.width, s.vocab);
  if (rc != ZERO_OK) return rc;
  if ((flags & ~(ZERO_IDS_I32 | ZERO_GRAD_F32 | ZERO_GRAD_ACCUMULATE)) != 0) return ZERO_E_LAYOUT;
  if (w == nullptr || (s.rows > 0 && (x == nullptr || targets == nullptr))) return ZERO_E_NULLPTR;
  const int gsize = (flags & ZERO_GRAD_F32) ? 4 : 2;
  const Matrix mx{x, s.rows, s.width, s.ldx, 2}, mw{w, s.vocab, s.width, s.ldw, 2},
      mt = ids_row(targets, s.rows, flags), ms{scale, 1, s.rows, s.rows, 4},
      ml{losses, 1, s.rows, s.rows, 4}, mo{total, 1, 1, 1, 4}, mdx{dx, s.rows, s.width, s.lddx, 2},
      mdw{dw, s.vocab, s.width, s.lddw, gsize};
  for (const Matrix* m : {&mx, &mw, &mt, &ms, &ml, &mo, &mdx, &mdw})
    if ((rc = check_matrix(*m)) != ZERO_OK) return rc;
  const Matrix* const in[] = {&mx, &mw, &mt, &ms};
  const Matrix* const out[] = {&ml, &mo, &mdx, &mdw};
  for (int i = 0; i < 4; ++i) {
    for (const Matrix* m : in)
      if (share(*out[i], *m)) return ZERO_E_ALIAS;
    for (int j = 0; j < i; ++j)
      if (share(*out[i], *out[j])) return ZERO_E_ALIAS;
  }
  const int64_t need = cross_entropy_workspace(
      s, (dx != nullptr || dw != nullptr ? ZERO_LINEAR_BACKWARD : 0) | (in_place(mw) ? ZERO_LINEAR_ALIGNED : 0) |
             (flags & ZERO_GRAD_F32));
  if ((rc = check_workspace(workspace, workspace_bytes, need)) != ZERO_OK) return rc;
  const Matrix mws{workspace, 1, need, need, 1};
  for (int i = 0; i < 4; ++i)
    if (share(mws, *in[i]) || share(mws, *out[i])) return ZERO_E_ALIAS;
  CrossEntropyLaunch L{};
  L.s = s;
  L.x = static_cast<const uint16_t*>(x);
  L.w = static_cast<const uint16_t*>(w);
  L.targets = targets;
  L.ids_i32 = (flags & ZERO_IDS_I32) ? 1 : 0;
  L.ignore = ignore_index;
  L.scale = scale;
  L.losses = losses;
  L.total = total;
  L.dx = static_cast<uint16_t*>(dx);
  L.dw = dw;
  L.grad_f32 = (flags & ZERO_GRAD_F32) ? 1 : 0;
  L.accumulate = (flags & ZERO_GRAD_ACCUMULATE) ? 1 : 0;
  L.workspace = workspace;
  L.stream = static_cast<cudaStream_t>(stream);
  L.withhold = withhold_copies();
  return launch_status(launch_cross_entropy(L));
}

int64_t zero_block_norm_workspace(const zero_block_norm_t* shape) {
  const int rc = check_block_norm(shape);
  return rc != ZERO_OK ? rc : block_norm_workspace(*shape);
}

int zero_block_norm_forward(const zero_block_norm_t* shape, const void* r, const void* h,
                            const void* post_weight, const void* post_bias, const void* gate,
                            const void* weight, const void* bias, void* s, void* y, void* stream) {
  Trace trace("zero_block_norm_forward");
  int rc = check_block_norm(shape);
  if (rc != ZERO_OK) return rc;
  const zero_block_norm_t& z = *shape;
  if ((rc = check_block_norm_inputs(z, h, post_weight, post_bias, gate, bias)) != ZERO_OK) return rc;
  if (z.rows > 0 && (r == nullptr || y == nullptr)) return ZERO_E_NULLPTR;
  const bool one = z.ldg == 0;  // gate for all rows
  const int64_t rows = z.rows, d = z.width;
  const Matrix mr{r, rows, d, z.ldr, 2}, mh{h, rows, d, z.ldh, 2}, ms{s, rows, d, z.lds, 2},
      my{y, rows, d, z.ldy, 2}, mg{gate, one ? 1 : rows, d, one ? d : z.ldg, 2}, mpw{post_weight, 1, d, d, 2},
      mpb{post_bias, 1, d, d, 2}, mw{weight, 1, d, d, 2}, mb{bias, 1, d, d, 2};
  for (const Matrix* m : {&mr, &mh, &ms, &my, &mg, &mpw, &mpb, &mw, &mb})
    if ((rc = check_rows(*m)) != ZERO_OK) return rc;
  for (const Matrix* m : {&mh, &mg, &mpw, &mpb, &mw, &mb})
    if (share(ms, *m) || share(my, *m)) return ZERO_E_ALIAS;
  if (share(my, mr) || share(my, ms) || (!(s == r && z.lds == z.ldr) && share(ms, mr))) return ZERO_E_ALIAS;
  if (rows == 0) return ZERO_OK;
  BlockNormLaunch L{};
  L.s = z;
  L.r = static_cast<const uint16_t*>(r);
  L.h = static_cast<const uint16_t*>(h);
  L.post_weight = static_cast<const uint16_t*>(post_weight);
  L.post_bias = static_cast<const uint16_t*>(post_bias);
  L.gate = static_cast<const uint16_t*>(gate);
  L.weight = static_cast<const uint16_t*>(weight);
  L.bias = static_cast<const uint16_t*>(bias);
  L.s_out = static_cast<uint16_t*>(s);
  L.y = static_cast<uint16_t*>(y);
  L.stream = static_cast<cudaStream_t>(stream);
  return launch_status(launch_block_norm_forward(L));
}

int zero_block_norm_backward(const zero_block_norm_t* shape, const void* dy, const void* ds,
                             const void* s, const void* h, const void* post_weight,
                             const void* post_bias, const void* gate, const void* weight,
                             void* dr, void* dh, void* dgate, void* dpost_weight,
                             void* dpost_bias, void* dweight, void* dbias, int32_t flags,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  Trace trace("zero_block_norm_backward");
  int rc = check_block_norm(shape);
  if (rc != ZERO_OK) return rc;
  const zero_block_norm_t& z = *shape;
  if ((rc = check_block_norm_inputs(z, h, post_weight, post_bias, gate, nullptr)) != ZERO_OK) return rc;
  if ((flags & ~(ZERO_GRAD_F32 | ZERO_GRAD_ACCUMULATE)) != 0) return ZERO_E_LAYOUT;
  if ((z.rows > 0 && h == nullptr && dh != nullptr) || (gate == nullptr && dgate != nullptr) ||
      (z.post == ZERO_NORM_NONE && dpost_weight != nullptr) ||
      (z.post != ZERO_NORM_LAYER && dpost_bias != nullptr) ||
      (z.kind != ZERO_NORM_LAYER && dbias != nullptr))
    return ZERO_E_LAYOUT;
  if (z.rows > 0 && (dy == nullptr || s == nullptr)) return ZERO_E_NULLPTR;
  const bool one = z.ldg == 0;
  const int gsize = (flags & ZERO_GRAD_F32) ? 4 : 2;
  const int64_t rows = z.rows, d = z.width;
  const Matrix mdy{dy, rows, d, z.lddy, 2}, mds{ds, rows, d, z.ldds, 2}, ms{s, rows, d, z.lds, 2},
      mh{h, rows, d, z.ldh, 2}, mg{gate, one ? 1 : rows, d, one ? d : z.ldg, 2}, mpw{post_weight, 1, d, d, 2},
      mpb{post_bias, 1, d, d, 2}, mw{weight, 1, d, d, 2}, mdr{dr, rows, d, z.lddr, 2}, mdh{dh, rows, d, z.lddh, 2},
      mdg{dgate, one ? 1 : rows, d, one ? d : z.lddg, one ? gsize : 2}, mdpw{dpost_weight, 1, d, d, gsize},
      mdpb{dpost_bias, 1, d, d, gsize}, mdw{dweight, 1, d, d, gsize}, mdb{dbias, 1, d, d, gsize};
  const Matrix* const in[] = {&mdy, &mds, &ms, &mh, &mg, &mpw, &mpb, &mw};
  const Matrix* const out[] = {&mdr, &mdh, &mdg, &mdpw, &mdpb, &mdw, &mdb};
  for (const Matrix* m : in)
    if ((rc = check_rows(*m)) != ZERO_OK) return rc;
  for (const Matrix* m : out)
    if ((rc = check_rows(*m)) != ZERO_OK) return rc;
  for (const Matrix* o : out) {
    for (const Matrix* m : in)
      if (!(o == &mdr && m == &mds && dr == ds && z.lddr == z.ldds) && share(*o, *m)) return ZERO_E_ALIAS;
    for (const Matrix* other : out) {
      if (other == o) break;
      if (share(*o, *other)) return ZERO_E_ALIAS;
    }
  }
  const int64_t need = block_norm_workspace(z);
  if ((rc = check_workspace(workspace, workspace_bytes, need)) != ZERO_OK) return rc;
  const Matrix mws{need > 0 ? workspace : nullptr, 1, need, need, 1};
  for (const Matrix* m : in)
    if (share(mws, *m)) return ZERO_E_ALIAS;
  for (const Matrix* m : out)
    if (share(mws, *m)) return ZERO_E_ALIAS;
  BlockNormLaunch L{};
  L.s = z;
  L.dy = static_cast<const uint16_t*>(dy);
  L.ds = static_cast<const uint16_t*>(ds);
  L.sum = static_cast<const uint16_t*>(s);
  L.h = static_cast<const uint16_t*>(h);
  L.post_weight = static_cast<const uint16_t*>(post_weight);
  L.post_bias = static_cast<const uint16_t*>(post_bias);
  L.gate = static_cast<const uint16_t*>(gate);
  L.weight = static_cast<const uint16_t*>(weight);
  L.dr = static_cast<uint16_t*>(dr);
  L.dh = static_cast<uint16_t*>(dh);
  L.dgate = dgate;
  L.dpost_weight = dpost_weight;
  L.dpost_bias = dpost_bias;
  L.dweight = dweight;
  L.dbias = dbias;
  L.grad_f32 = (flags & ZERO_GRAD_F32) ? 1 : 0;
  L.accumulate = (flags & ZERO_GRAD_ACCUMULATE) ? 1 : 0;
  L.workspace = workspace;
  L.stream = static_cast<cudaStream_t>(stream);
  return launch_status(launch_block_norm_backward(L));
}

}  // extern "C"
