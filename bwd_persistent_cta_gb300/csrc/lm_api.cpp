// lm_api.cpp - the C ABI of the gated delta rule and the block norm: descriptor
// and argument checks, buffer sizes and the launch sequence of each call.
#include <cuda_runtime.h>

#include <cmath>
#include <new>

#include "api_util.h"
#include "delta.h"
#include "delta_tc.h"
#include "norm.h"
#include "rnn.h"
#include "rnn_debug.h"

using namespace rnn;

struct rnn_delta_s {
  rnn_delta_desc_t desc;
  float scale;
  int device, num_sms, bf16;
  int tc;                      // the tensor-core kernels run whole sequences
  size_t es;
  int* d_len;
  int has_len;
  CallOrder order;             // of the calls that read d_len or use scratch
  unsigned int* status;        // device word
  uint64_t launches;
  // byte offsets.  Forward workspace (tensor cores): the tiles of prep; a
  // training forward keeps all of them but th in the reserve
  size_t w_k16, w_q16, w_th, w_p, w_sc, workspace_bytes;
  // reserve: states before each chunk and e (with their scales), and those tiles
  size_t r_s0, r_e, r_s0s, r_es, r_k16, r_q16, r_tb, r_p, r_sc, reserve_bytes;
  // backward workspace: state gradients after each chunk and y, with scales
  size_t b_ds1, b_y, b_ds1s, b_ys, b_dos, bwd_workspace_bytes;
};

struct rnn_norm_s {
  rnn_norm_desc_t desc;
  int device, num_sms, bf16;
  CallOrder order;             // of the calls that use the workspace
  uint64_t launches;
};

namespace {

rnn_status_t check_delta(const rnn_delta_desc_t* d) {
  if (!d) return RNN_BAD_PARAM;
  if (d->batch < 1 || d->seq_len < 1 || d->heads_k < 1 || d->heads_v < 1) return RNN_BAD_PARAM;
  if (d->heads_v % d->heads_k) return RNN_BAD_PARAM;
  if (d->dim_k < 8 || d->dim_k > 256 || d->dim_k % 8 || d->dim_v < 8 || d->dim_v > 256 || d->dim_v % 8)
    return RNN_BAD_PARAM;
  if (d->dtype != RNN_F32 && d->dtype != RNN_BF16) return RNN_BAD_PARAM;
  if (!flag(d->batch_first) || !std::isfinite(d->scale)) return RNN_BAD_PARAM;
  const long long rows = static_cast<long long>(d->seq_len) * d->batch;
  if (rows > (1LL << 30)) return RNN_BAD_PARAM;
  // CTAs of the largest grid: one per chunk or slice of 16 value columns of a head
  const long long nc = (d->seq_len + kSimtChunk - 1) / kSimtChunk;
  const long long per = nc > 16 ? nc : 16;
  if (per * d->batch > (1LL << 31) - 1 || per * d->batch * d->heads_v > (1LL << 31) - 1) return RNN_BAD_PARAM;
  return RNN_OK;
}

rnn_status_t check_norm(const rnn_norm_desc_t* d) {
  if (!d) return RNN_BAD_PARAM;
  if (d->rows < 1 || d->groups < 1 || static_cast<long long>(d->rows) * d->groups > (1LL << 30)) return RNN_BAD_PARAM;
  if (d->cols < 8 || d->cols > 8192 || d->cols % 8) return RNN_BAD_PARAM;
  if (d->dtype != RNN_F32 && d->dtype != RNN_BF16) return RNN_BAD_PARAM;
  if (!flag(d->norm_in) || !flag(d->residual) || !flag(d->norm_out)) return RNN_BAD_PARAM;
  if (d->gate < RNN_GATE_NONE || d->gate > RNN_GATE_SIGMOID) return RNN_BAD_PARAM;
  if (!(d->eps > 0.f) || !std::isfinite(d->eps)) return RNN_BAD_PARAM;
  return RNN_OK;
}

// From this many tokens on sequences run by chunks: where heads are many or
// gradients follow (128 x 128, chunks and recurrence, kernels alone: 8 sequences x
// 16 heads, 12 tokens 24 and 21 us, 16 tokens 25 and 26, training 56 and 124; 32 x
// 32, 12 tokens 107 and 128, training 280 and 639).  A few heads' inference would
// be faster token by token up to 48 tokens (4 heads, 16 tokens: 18 and 8.5 us) but
// for the training forward, 45 and 99 with its backward, which shares the layout.
constexpr int kTcMinTokens = 16;

void delta_layout(rnn_delta_s* h) {
  const rnn_delta_desc_t& d = h->desc;
  const size_t bh = static_cast<size_t>(d.batch) * d.heads_v;
  Bump w, r, b;
  if (!h->tc) {
    const size_t nc = (d.seq_len + kSimtChunk - 1) / kSimtChunk;
    const size_t states = bh * nc * d.dim_v * d.dim_k * 4, vectors = bh * d.seq_len * d.dim_v * 4;
    h->r_s0 = r.take(states);
    h->r_e = r.take(vectors);
    h->b_ds1 = b.take(states);
    h->b_y = b.take(vectors);
  } else {
    const size_t nc = (d.seq_len + kTc - 1) / kTc;
    const size_t vc = bh * nc, kc = static_cast<size_t>(d.batch) * d.heads_k * nc;
    const size_t keys = kc * kTc * d.dim_k * 2, tile = vc * kTri, sc = vc * kSc * 4;
    const size_t states = vc * d.dim_v * d.dim_k * 2, vectors = vc * kTc * d.dim_v * 2, scales = vc * (d.dim_v / 16) * 4;
    h->w_th = w.take(tile);
    h->w_k16 = w.take(keys);
    h->w_q16 = w.take(keys);
    h->w_p = w.take(tile);
    h->w_sc = w.take(sc);
    h->r_k16 = r.take(keys);
    h->r_q16 = r.take(keys);
    h->r_tb = r.take(tile);
    h->r_p = r.take(tile);
    h->r_sc = r.take(sc);
    h->r_s0 = r.take(states);
    h->r_s0s = r.take(scales);
    h->r_e = r.take(vectors);
    h->r_es = r.take(scales);
    h->b_ds1 = b.take(states);
    h->b_ds1s = b.take(scales);
    h->b_y = b.take(vectors);
    h->b_ys = b.take(scales);
    h->b_dos = b.take(scales);
  }
  h->workspace_bytes = w.off;
  h->reserve_bytes = r.off;
  h->bwd_workspace_bytes = b.off;
}

rnn_status_t delta_args(const rnn_delta_s* h, const rnn_delta_in_t* in, DeltaArgs* a) {
  const rnn_delta_desc_t& d = h->desc;
  if (!in || !in->q || !in->k || !in->v || !in->g || !in->beta) return RNN_BAD_PARAM;
  if (!aligned16(in->q) || !aligned16(in->k) || !aligned16(in->v)) return RNN_BAD_PARAM;
  if (reinterpret_cast<uintptr_t>(in->g) % h->es || reinterpret_cast<uintptr_t>(in->beta) % h->es)
    return RNN_BAD_PARAM;
  const int64_t unit = 16 / h->es, qk = static_cast<int64_t>(d.heads_k) * d.dim_k,
                vd = static_cast<int64_t>(d.heads_v) * d.dim_v;
  if (!row_ok(in->q_row, qk, unit, &a->q_row) || !row_ok(in->k_row, qk, unit, &a->k_row) ||
      !row_ok(in->v_row, vd, unit, &a->v_row) || !row_ok(in->g_row, d.heads_v, 1, &a->g_row) ||
      !row_ok(in->beta_row, d.heads_v, 1, &a->beta_row))
    return RNN_BAD_PARAM;
  a->B = d.batch; a->T = d.seq_len; a->Hk = d.heads_k; a->Hv = d.heads_v; a->Dk = d.dim_k; a->Dv = d.dim_v;
  a->bfirst = d.batch_first;
  a->scale = h->scale;
  a->len = h->has_len ? h->d_len : nullptr;
  a->q = in->q; a->k = in->k; a->v = in->v; a->g = in->g; a->beta = in->beta;
  return RNN_OK;
}

DeltaTcBufs tc_bufs(const rnn_delta_s* h, void* workspace, const void* reserve) {
  DeltaTcBufs w{};
  w.th = workspace ? at<void>(workspace, h->w_th) : nullptr;
  if (!reserve) {
    w.k16 = at<void>(workspace, h->w_k16);
    w.q16 = at<void>(workspace, h->w_q16);
    w.p = at<void>(workspace, h->w_p);
    w.sc = at<float>(workspace, h->w_sc);
    return w;
  }
  w.k16 = at<void>(reserve, h->r_k16);
  w.q16 = at<void>(reserve, h->r_q16);
  w.tb = at<void>(reserve, h->r_tb);
  w.p = at<void>(reserve, h->r_p);
  w.sc = at<float>(reserve, h->r_sc);
  w.s0 = at<void>(reserve, h->r_s0);
  w.s0_scale = at<float>(reserve, h->r_s0s);
  w.e = at<void>(reserve, h->r_e);
  w.e_scale = at<float>(reserve, h->r_es);
  return w;
}

rnn_status_t norm_args(const rnn_norm_s* h, const rnn_norm_in_t* in, NormArgs* a) {
  const rnn_norm_desc_t& d = h->desc;
  *a = NormArgs{};
  a->rows = d.rows; a->groups = d.groups; a->cols = d.cols;
  a->norm_in = d.norm_in; a->gate = d.gate; a->residual = d.residual; a->norm_out = d.norm_out;
  a->eps = d.eps;
  a->num_sms = h->num_sms;
  if (!in) return RNN_OK;      // sizes only
  if (!in->y || (d.gate != RNN_GATE_NONE && !in->z) || (d.residual && !in->x)) return RNN_BAD_PARAM;
  const int64_t unit = h->bf16 ? 8 : 4, dense = static_cast<int64_t>(d.groups) * d.cols;
  if (!row_ok(in->y_row, dense, unit, &a->y_row) || !row_ok(in->z_row, dense, unit, &a->z_row) ||
      !row_ok(in->x_row, dense, unit, &a->x_row))
    return RNN_BAD_PARAM;
  a->y = in->y;
  a->z = d.gate != RNN_GATE_NONE ? in->z : nullptr;
  a->x = d.residual ? in->x : nullptr;
  a->w_in = d.norm_in ? in->w_in : nullptr;
  a->scale = d.residual ? in->scale : nullptr;
  a->w_out = d.norm_out ? in->w_out : nullptr;
  for (const void* p : {a->y, a->z, a->x, a->w_in, a->scale, a->w_out})
    if (!aligned16(p)) return RNN_BAD_PARAM;
  return RNN_OK;
}

}  // namespace

extern "C" {

rnn_status_t rnn_delta_create(const rnn_delta_desc_t* desc, rnn_delta_t* out) {
  if (!out) return RNN_BAD_PARAM;
  *out = nullptr;
  rnn_status_t rc = check_delta(desc);
  if (rc != RNN_OK) return rc;
  int dev = 0, sms = 0;
  rc = pick_device(&dev, &sms);
  if (rc != RNN_OK) return rc;
  rnn_delta_s* h = new (std::nothrow) rnn_delta_s();
  if (!h) return RNN_INTERNAL;
  h->desc = *desc;
  h->scale = desc->scale != 0.f ? desc->scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(desc->dim_k)));
  h->device = dev;
  h->num_sms = sms;
  h->bf16 = desc->dtype == RNN_BF16;
  h->es = h->bf16 ? 2 : 4;
  h->d_len = nullptr;
  h->has_len = 0;
  h->launches = 0;
  h->tc = desc->seq_len >= kTcMinTokens && delta_tc_supported(desc->dim_k, desc->dim_v, h->bf16);
  if (h->tc && delta_tc_init(desc->dim_k)) {
    delete h;
    return RNN_CUDA_ERROR;
  }
  if (cudaMalloc(&h->status, sizeof(unsigned int)) != cudaSuccess) {
    delete h;
    return RNN_CUDA_ERROR;
  }
  if (cudaMemset(h->status, 0, sizeof(unsigned int)) != cudaSuccess || h->order.create() != RNN_OK) {
    cudaFree(h->status);
    delete h;
    return RNN_CUDA_ERROR;
  }
  delta_layout(h);
  *out = h;
  return RNN_OK;
}

rnn_status_t rnn_delta_destroy(rnn_delta_t h) {
  if (!h) return RNN_OK;
  DeviceGuard dg(h->device);
  if (h->d_len) cudaFree(h->d_len);
  cudaFree(h->status);
  h->order.destroy();
  delete h;
  return RNN_OK;
}

rnn_status_t rnn_delta_get_sizes(rnn_delta_t h, size_t* ws, size_t* bws, size_t* rs) {
  if (!h) return RNN_BAD_PARAM;
  if (ws) *ws = h->workspace_bytes;
  if (bws) *bws = h->bwd_workspace_bytes;
  if (rs) *rs = h->reserve_bytes;
  return RNN_OK;
}

rnn_status_t rnn_delta_set_seq_lengths(rnn_delta_t h, const int* lengths) {
  if (!h) return RNN_BAD_PARAM;
  DeviceGuard dg(h->device);
  if (!dg.ok) return RNN_CUDA_ERROR;
  return set_lengths(h->order, lengths, h->desc.batch, h->desc.seq_len, &h->d_len, &h->has_len);
}

rnn_status_t rnn_delta_forward(rnn_delta_t h, const rnn_delta_in_t* in, const float* s0, void* o, float* sT,
                               void* workspace, void* reserve, void* stream) {
  if (!h || !o || !aligned16(o) || !aligned16(s0) || !aligned16(sT)) return RNN_BAD_PARAM;
  DeltaRecurArgs r{};
  const rnn_status_t rc = delta_args(h, in, &r.a);
  if (rc != RNN_OK) return rc;
  if ((h->workspace_bytes && !workspace) || !aligned16(workspace) || !aligned16(reserve)) return RNN_BAD_WORKSPACE;
  DeviceGuard dg(h->device);
  if (!dg.ok) return RNN_CUDA_ERROR;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Ordered call(h->order, h->has_len || h->tc || reserve, s);
  if (call.rc != RNN_OK) return call.rc;
  if (h->tc) {
    DeltaTcArgs t{};
    t.a = r.a;
    t.w = tc_bufs(h, workspace, reserve);
    t.s_in = s0;
    t.s_out = sT;
    t.o = o;
    t.status = h->status;
    t.train = reserve != nullptr;
    t.num_sms = h->num_sms;
    int n = 0;
    const int e = launch_delta_tc_forward(t, s, &n);
    h->launches += n;
    return call.done(e);
  }
  r.s_in = s0;
  r.s_out = sT;
  r.num_slots = -1;
  r.num_sms = h->num_sms;
  r.o = o;
  r.ckpt = reserve ? at<float>(reserve, h->r_s0) : nullptr;
  r.e = reserve ? at<float>(reserve, h->r_e) : nullptr;
  const int e = launch_delta_recur(r, h->bf16, s);
  if (!e) ++h->launches;
  return call.done(e);
}

rnn_status_t rnn_delta_backward(rnn_delta_t h, const rnn_delta_in_t* in, const void* do_, const float* dsT, void* dq,
                                void* dk, void* dv, void* dg, void* dbeta, float* ds0, void* workspace,
                                const void* reserve, void* stream) {
  if (!h || !do_ || !dq || !dk || !dv || !dg || !dbeta) return RNN_BAD_PARAM;
  for (const void* p : {do_, static_cast<const void*>(dsT), static_cast<const void*>(dq), static_cast<const void*>(dk),
                        static_cast<const void*>(dv), static_cast<const void*>(dg), static_cast<const void*>(dbeta),
                        static_cast<const void*>(ds0)})
    if (!aligned16(p)) return RNN_BAD_PARAM;
  DeltaArgs a{};
  const rnn_status_t rc = delta_args(h, in, &a);
  if (rc != RNN_OK) return rc;
  if (!workspace || !reserve || !aligned16(workspace) || !aligned16(reserve)) return RNN_BAD_WORKSPACE;
  DeviceGuard guard(h->device);
  if (!guard.ok) return RNN_CUDA_ERROR;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Ordered call(h->order, true, s);
  if (call.rc != RNN_OK) return call.rc;
  if (h->tc) {
    DeltaTcBwdArgs t{};
    t.a = a;
    t.w = tc_bufs(h, nullptr, reserve);
    t.dout = do_;
    t.dsT = dsT;
    t.ds0 = ds0;
    t.ds1 = at<void>(workspace, h->b_ds1);
    t.ds1_scale = at<float>(workspace, h->b_ds1s);
    t.y = at<void>(workspace, h->b_y);
    t.y_scale = at<float>(workspace, h->b_ys);
    t.do_scale = at<float>(workspace, h->b_dos);
    t.status = h->status;
    t.dq = dq; t.dk = dk; t.dv = dv; t.dg = dg; t.dbeta = dbeta;
    t.num_sms = h->num_sms;
    int n = 0;
    const int e = launch_delta_tc_backward(t, s, &n);
    h->launches += n;
    return call.done(e);
  }
  DeltaRecurBwdArgs b{};
  b.a = a;
  b.dout = do_;
  b.dsT = dsT;
  b.ds0 = ds0;
  b.ckpt = at<float>(workspace, h->b_ds1);
  b.y = at<float>(workspace, h->b_y);
  b.num_sms = h->num_sms;
  int e = launch_delta_recur_bwd(b, h->bf16, s);
  if (e) return call.done(e);
  ++h->launches;
  DeltaChunkBwdArgs c{};
  c.a = a;
  c.dout = do_;
  c.s0 = at<float>(reserve, h->r_s0);
  c.ds1 = b.ckpt;
  c.e = at<float>(reserve, h->r_e);
  c.y = b.y;
  c.dq = dq; c.dk = dk; c.dv = dv; c.dg = dg; c.dbeta = dbeta;
  e = launch_delta_chunk_bwd(c, h->bf16, s);
  if (!e) ++h->launches;
  return call.done(e);
}

rnn_status_t rnn_delta_step(rnn_delta_t h, const rnn_delta_in_t* in, float* state, int num_slots, const int* slots,
                            void* o, void* stream) {
  if (!h || !state || !o || num_slots < 0 || !aligned16(state) || !aligned16(o)) return RNN_BAD_PARAM;
  if (reinterpret_cast<uintptr_t>(slots) & 3) return RNN_BAD_PARAM;
  DeltaRecurArgs r{};
  const rnn_status_t rc = delta_args(h, in, &r.a);
  if (rc != RNN_OK) return rc;
  DeviceGuard dg(h->device);
  if (!dg.ok) return RNN_CUDA_ERROR;
  r.s_in = state;
  r.s_out = state;
  r.slots = slots;
  r.num_slots = num_slots;
  r.status = h->status;
  r.num_sms = h->num_sms;
  r.o = o;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Ordered call(h->order, h->has_len, s);
  if (call.rc != RNN_OK) return call.rc;
  const int e = launch_delta_recur(r, h->bf16, s);
  if (!e) ++h->launches;
  return call.done(e);
}

rnn_status_t rnn_delta_sync_status(rnn_delta_t h, void* stream) {
  if (!h) return RNN_BAD_PARAM;
  DeviceGuard dg(h->device);
  if (!dg.ok) return RNN_CUDA_ERROR;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned int v = 0;
  if (cudaMemcpyAsync(&v, h->status, sizeof v, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return RNN_CUDA_ERROR;
  if (v && (cudaMemsetAsync(h->status, 0, sizeof v, s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess))
    return RNN_CUDA_ERROR;
  return static_cast<rnn_status_t>(v);
}

uint64_t rnn_delta_launch_count(rnn_delta_t h) { return h ? h->launches : 0; }

rnn_status_t rnn_norm_create(const rnn_norm_desc_t* desc, rnn_norm_t* out) {
  if (!out) return RNN_BAD_PARAM;
  *out = nullptr;
  rnn_status_t rc = check_norm(desc);
  if (rc != RNN_OK) return rc;
  int dev = 0, sms = 0;
  rc = pick_device(&dev, &sms);
  if (rc != RNN_OK) return rc;
  rnn_norm_s* h = new (std::nothrow) rnn_norm_s();
  if (!h) return RNN_INTERNAL;
  h->desc = *desc;
  h->device = dev;
  h->num_sms = sms;
  h->bf16 = desc->dtype == RNN_BF16;
  h->launches = 0;
  if (h->order.create() != RNN_OK) {
    delete h;
    return RNN_CUDA_ERROR;
  }
  *out = h;
  return RNN_OK;
}

rnn_status_t rnn_norm_destroy(rnn_norm_t h) {
  if (!h) return RNN_OK;
  DeviceGuard dg(h->device);
  h->order.destroy();
  delete h;
  return RNN_OK;
}

rnn_status_t rnn_norm_get_sizes(rnn_norm_t h, size_t* ws) {
  if (!h) return RNN_BAD_PARAM;
  NormArgs a;
  norm_args(h, nullptr, &a);
  if (ws) *ws = norm_workspace_bytes(a);
  return RNN_OK;
}

rnn_status_t rnn_norm_forward(rnn_norm_t h, const rnn_norm_in_t* in, void* x_out, void* n_out, void* stream) {
  if (!h || !in || !x_out || !aligned16(x_out) || !aligned16(n_out)) return RNN_BAD_PARAM;
  if ((h->desc.norm_out != 0) != (n_out != nullptr)) return RNN_BAD_PARAM;
  NormArgs a;
  const rnn_status_t rc = norm_args(h, in, &a);
  if (rc != RNN_OK) return rc;
  DeviceGuard dg(h->device);
  if (!dg.ok) return RNN_CUDA_ERROR;
  a.x_out = x_out;
  a.n_out = n_out;
  const int e = launch_norm_forward(a, h->bf16, static_cast<cudaStream_t>(stream));
  if (!e) ++h->launches;
  return static_cast<rnn_status_t>(e);
}

rnn_status_t rnn_norm_backward(rnn_norm_t h, const rnn_norm_in_t* in, const void* dx_out, const void* dn_out, void* dy,
                               void* dz, void* dx, float* dw_in, float* dscale, float* dw_out, void* workspace,
                               void* stream) {
  if (!h || !in || (!dx_out && !dn_out)) return RNN_BAD_PARAM;
  const rnn_norm_desc_t& d = h->desc;
  // a gradient of something the descriptor leaves out has no value
  if ((dn_out && !d.norm_out) || (dz && d.gate == RNN_GATE_NONE) || (dx && !d.residual) || (dw_in && !d.norm_in) ||
      (dscale && !d.residual) || (dw_out && !d.norm_out))
    return RNN_BAD_PARAM;
  for (const void* p : {dx_out, dn_out, static_cast<const void*>(dy), static_cast<const void*>(dz),
                        static_cast<const void*>(dx), static_cast<const void*>(dw_in),
                        static_cast<const void*>(dscale), static_cast<const void*>(dw_out)})
    if (!aligned16(p)) return RNN_BAD_PARAM;
  NormArgs a;
  const rnn_status_t rc = norm_args(h, in, &a);
  if (rc != RNN_OK) return rc;
  const bool weights = dw_in || dscale || dw_out;
  if ((weights && !workspace) || !aligned16(workspace)) return RNN_BAD_WORKSPACE;
  DeviceGuard dg(h->device);
  if (!dg.ok) return RNN_CUDA_ERROR;
  a.dx_out = dx_out; a.dn_out = dn_out;
  a.dy = dy; a.dz = dz; a.dx = dx;
  a.dw_in = dw_in; a.dscale = dscale; a.dw_out = dw_out;
  a.partial = weights ? static_cast<float*>(workspace) : nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Ordered call(h->order, weights, s);
  if (call.rc != RNN_OK) return call.rc;
  int n = 0;
  const int e = launch_norm_backward(a, h->bf16, s, &n);
  h->launches += n;
  return call.done(e);
}

uint64_t rnn_norm_launch_count(rnn_norm_t h) { return h ? h->launches : 0; }

int rnn_debug_step_drain(int turn, int turns, int* out) {
  if (!out || turn < 0 || turn >= turns) return 0;
  int n = 0;
  for (int t = turn; t <= step_last_fill(turn, turns); ++t, ++n) {
    out[2 * n] = step_fill(t).stage;
    out[2 * n + 1] = static_cast<int>(step_fill(t).parity);
  }
  return n;
}

}  // extern "C"
