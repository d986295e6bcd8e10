// ssm_api.cpp - the C ABI of the selective scan, the causal convolution and gradient
// clipping: descriptor and argument checks, buffer sizes and the launches of each call.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <utility>
#include <vector>

#include "api_util.h"
#include "clip.h"
#include "conv.h"
#include "rnn.h"
#include "scan.h"

using namespace rnn;

using Ranges = std::vector<std::pair<uintptr_t, uintptr_t>>;

struct rnn_scan_s {
  rnn_scan_desc_t desc;
  int device, num_sms, bf16;
  size_t es;
  int* d_len;
  int has_len;
  CallOrder order;             // of the calls that read d_len or use scratch
  uint64_t launches;
  size_t workspace_bytes, bwd_workspace_bytes, reserve_bytes;
};

struct rnn_conv_s {
  rnn_conv_desc_t desc;
  int device, num_sms, bf16;
  int* d_len;
  int has_len;
  CallOrder order;
  uint64_t launches;
};

struct rnn_clip_s {
  int num, device, num_sms;
  int64_t* d_start;            // [num + 1], then dtypes [num]
  int* d_dtype;
  std::vector<int64_t> start;
  std::vector<int> dtype;
  Ranges inplace, apart, reads;        // scratch of a call's checks
  CallOrder order;
  uint64_t launches;
};

namespace {

rnn_status_t check_sequences(int batch, int seq_len, int channels) {
  if (batch < 1 || seq_len < 1 || channels < 8 || channels > 65536 || channels % 8) return RNN_BAD_PARAM;
  const long long rows = static_cast<long long>(seq_len) * batch;
  if (rows > (1LL << 30) || rows * channels > (1LL << 43)) return RNN_BAD_PARAM;      // grids stay below 2^31 CTAs
  // CTAs of the largest grid: one for each 8 channels of a sequence
  return static_cast<long long>(batch) * (channels / 8) <= (1LL << 31) - 1 ? RNN_OK : RNN_BAD_PARAM;
}

rnn_status_t check_scan(const rnn_scan_desc_t* d) {
  if (!d || check_sequences(d->batch, d->seq_len, d->channels) != RNN_OK) return RNN_BAD_PARAM;
  if (d->states < 8 || d->states > 64 || d->states % 8) return RNN_BAD_PARAM;
  if (d->groups < 1 || d->groups > d->channels / 8 || d->channels % (8 * d->groups)) return RNN_BAD_PARAM;
  if (d->dtype != RNN_F32 && d->dtype != RNN_BF16) return RNN_BAD_PARAM;
  return flag(d->batch_first) && flag(d->softplus) ? RNN_OK : RNN_BAD_PARAM;
}

rnn_status_t check_conv(const rnn_conv_desc_t* d) {
  if (!d || check_sequences(d->batch, d->seq_len, d->channels) != RNN_OK) return RNN_BAD_PARAM;
  if (d->width < 2 || d->width > 4) return RNN_BAD_PARAM;
  if (d->dtype != RNN_F32 && d->dtype != RNN_BF16) return RNN_BAD_PARAM;
  if (d->act != RNN_GATE_NONE && d->act != RNN_GATE_SILU) return RNN_BAD_PARAM;
  return flag(d->batch_first) ? RNN_OK : RNN_BAD_PARAM;
}

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

ScanArgs scan_shape(const rnn_scan_s* h) {
  const rnn_scan_desc_t& d = h->desc;
  ScanArgs a{};
  a.B = d.batch; a.T = d.seq_len; a.D = d.channels; a.N = d.states; a.G = d.groups;
  a.bfirst = d.batch_first;
  a.softplus = d.softplus;
  a.len = h->has_len ? h->d_len : nullptr;
  a.num_sms = h->num_sms;
  return a;
}

rnn_status_t scan_args(const rnn_scan_s* h, const rnn_scan_in_t* in, ScanArgs* a) {
  if (!in || !in->x || !in->dt || !in->B || !in->C || !in->A) return RNN_BAD_PARAM;
  for (const void* p : {in->x, in->dt, in->z, in->A, in->D, in->dt_bias})
    if (!aligned16(p)) return RNN_BAD_PARAM;
  if (!aligned(in->B, h->es) || !aligned(in->C, h->es)) return RNN_BAD_PARAM;
  *a = scan_shape(h);
  const int64_t unit = 16 / h->es, rows = static_cast<int64_t>(a->G) * a->N;
  if (!row_ok(in->x_row, a->D, unit, &a->x_row) || !row_ok(in->dt_row, a->D, unit, &a->dt_row) ||
      !row_ok(in->z_row, a->D, unit, &a->z_row) || !row_ok(in->B_row, rows, 1, &a->B_row) ||
      !row_ok(in->C_row, rows, 1, &a->C_row))
    return RNN_BAD_PARAM;
  a->x = in->x; a->dt = in->dt; a->z = in->z; a->Bm = in->B; a->Cm = in->C;
  a->A = static_cast<const float*>(in->A);
  a->skip = static_cast<const float*>(in->D);
  a->bias = static_cast<const float*>(in->dt_bias);
  return RNN_OK;
}

ConvArgs conv_shape(const rnn_conv_s* h) {
  const rnn_conv_desc_t& d = h->desc;
  ConvArgs a{};
  a.B = d.batch; a.T = d.seq_len; a.D = d.channels; a.W = d.width;
  a.bfirst = d.batch_first;
  a.silu = d.act == RNN_GATE_SILU;
  a.len = h->has_len ? h->d_len : nullptr;
  a.num_sms = h->num_sms;
  return a;
}

rnn_status_t conv_args(const rnn_conv_s* h, const rnn_conv_in_t* in, ConvArgs* a) {
  if (!in || !in->x || !in->w) return RNN_BAD_PARAM;
  for (const void* p : {in->x, in->w, in->bias})
    if (!aligned16(p)) return RNN_BAD_PARAM;
  *a = conv_shape(h);
  if (!row_ok(in->x_row, a->D, h->bf16 ? 8 : 4, &a->x_row)) return RNN_BAD_PARAM;
  a->x = in->x; a->w = in->w; a->bias = in->bias;
  return RNN_OK;
}

// Whether dense memory shares any with the rows (of ``row`` bytes, every ``hop`` bytes) of a
// sequence's input; the gaps of a packed projection are not part of it.
bool over_rows(const void* to, int64_t bytes, const void* from, int64_t row, int64_t hop, int64_t rows) {
  const int64_t at = static_cast<int64_t>(reinterpret_cast<uintptr_t>(to)) - static_cast<int64_t>(reinterpret_cast<uintptr_t>(from));
  if (at < 0) return at + bytes > 0;
  const int64_t r = at / hop, in = at - r * hop;
  return r < rows && (in < row || (in + bytes > hop && r + 1 < rows));
}
// An output of a whole sequence over x, of which threads read tokens that are others' to write.
bool over_x(const rnn_conv_s* h, const ConvArgs& a, const void* out) {
  const int64_t es = h->bf16 ? 2 : 4, rows = static_cast<int64_t>(a.B) * a.T;
  return over_rows(out, rows * a.D * es, a.x, a.D * es, a.x_row * es, rows);
}
bool over_dense(const rnn_conv_s* h, const ConvArgs& a, const void* out, const void* in) {
  const int64_t bytes = static_cast<int64_t>(a.B) * a.T * a.D * (h->bf16 ? 2 : 4);
  return over_rows(out, bytes, in, bytes, bytes, 1);
}

// A new handle of type H with its device and call order; null after a failure.
template <typename H>
rnn_status_t make(H** out) {
  int dev = 0, sms = 0;
  const rnn_status_t rc = pick_device(&dev, &sms);
  if (rc != RNN_OK) return rc;
  H* h = new (std::nothrow) H();
  if (!h) return RNN_INTERNAL;
  h->device = dev;
  h->num_sms = sms;
  if (h->order.create() != RNN_OK) {
    delete h;
    return RNN_CUDA_ERROR;
  }
  *out = h;
  return RNN_OK;
}

void add(Ranges& r, const void* p, uint64_t bytes) {                        // within its capacity
  r.emplace_back(reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes);
}
// Sorts them; whether no two overlap.
bool disjoint(Ranges& r) {
  if (!std::is_sorted(r.begin(), r.end())) std::sort(r.begin(), r.end());
  for (size_t i = 1; i < r.size(); ++i)
    if (r[i].first < r[i - 1].second) return false;
  return true;
}
// Whether any of ``w``, sorted and disjoint, overlaps any of ``r``, sorted.
bool meet(const Ranges& w, const Ranges& r) {
  size_t j = 0;                              // the first that ends behind the other's beginning
  for (const auto& x : r) {
    while (j < w.size() && w[j].second <= x.first) ++j;
    if (j < w.size() && w[j].first < x.second) return true;
  }
  return false;
}
// What a call writes is written once (a tensor listed twice would be scaled once or twice, as
// it happens), and an output other than its own gradient lies apart from all that is read, the
// norm from everything.  False where it is not so.  A gradient scaled in place may share memory
// with others whose outputs lie elsewhere: ``split``, those go first.
bool memory_ok(rnn_clip_t h, const void* const* grads, void* const* out, const float* norm, int* split) {
  auto &w = h->inplace, &a = h->apart, &r = h->reads;
  w.clear();
  a.clear();
  r.clear();
  for (int i = 0; i < h->num; ++i) {
    const uint64_t bytes = static_cast<uint64_t>(h->start[i + 1] - h->start[i]) * (h->dtype[i] == RNN_F32 ? 4 : 2);
    if (!bytes) continue;
    if (!out || out[i] == grads[i]) {
      add(w, grads[i], bytes);
    } else {
      add(a, out[i], bytes);
      add(r, grads[i], bytes);
    }
  }
  const uintptr_t n = reinterpret_cast<uintptr_t>(norm);
  for (const Ranges* v : {&w, &a, &r})
    for (const auto& x : *v)
      if (n < x.second && n + sizeof(float) > x.first) return false;
  if (!disjoint(w) || !disjoint(a)) return false;
  disjoint(r);                               // gradients that are only read may overlap
  if (meet(w, a) || meet(a, r)) return false;
  *split = meet(w, r);
  return true;
}

rnn_status_t clip_call(rnn_clip_t h, const void* const* grads, void* const* out, float max_norm, float eps, float* norm,
                       void* workspace, void* stream, int scale) {
  if (!h || !grads || !norm || !aligned(norm, 4)) return RNN_BAD_PARAM;
  if (!(max_norm >= 0.f) || !(eps >= 0.f) || !std::isfinite(max_norm) || !std::isfinite(eps)) return RNN_BAD_PARAM;
  for (int i = 0; i < h->num; ++i) {
    if (h->start[i + 1] == h->start[i]) continue;
    const size_t es = h->dtype[i] == RNN_F32 ? 4 : 2;
    if (!grads[i] || !aligned(grads[i], es)) return RNN_BAD_PARAM;
    if (out && (!out[i] || !aligned(out[i], es))) return RNN_BAD_PARAM;
  }
  int split = 0;
  if (scale && !memory_ok(h, grads, out, norm, &split)) return RNN_BAD_PARAM;
  if (!workspace || !aligned16(workspace)) return RNN_BAD_WORKSPACE;
  DeviceGuard dg(h->device);
  if (!dg.ok) return RNN_CUDA_ERROR;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Ordered call(h->order, true, s);
  if (call.rc != RNN_OK) return call.rc;
  ClipArgs c{};
  c.num = h->num;
  c.start = h->d_start;
  c.dtype = h->d_dtype;
  c.host_start = h->start.data();
  c.grads = grads;
  c.out = out;
  c.max_norm = max_norm;
  c.eps = eps;
  c.norm = norm;
  c.partial = static_cast<double*>(workspace);
  c.scale = scale;
  c.split = split;
  c.num_sms = h->num_sms;
  int n = 0;
  const int e = launch_clip(c, s, &n);
  h->launches += n;
  return call.done(e);
}

}  // namespace

extern "C" {

rnn_status_t rnn_scan_create(const rnn_scan_desc_t* desc, rnn_scan_t* out) {
  if (!out) return RNN_BAD_PARAM;
  *out = nullptr;
  rnn_status_t rc = check_scan(desc);
  if (rc != RNN_OK) return rc;
  rnn_scan_s* h = nullptr;
  rc = make(&h);
  if (rc != RNN_OK) return rc;
  h->desc = *desc;
  h->bf16 = desc->dtype == RNN_BF16;
  h->es = h->bf16 ? 2 : 4;
  const ScanArgs a = scan_shape(h);
  h->workspace_bytes = scan_split_forward(a, h->bf16).bytes;
  h->bwd_workspace_bytes = scan_bwd_layout(a).bytes;
  h->reserve_bytes = scan_reserve(a).bytes;
  *out = h;
  return RNN_OK;
}

rnn_status_t rnn_scan_destroy(rnn_scan_t h) {
  if (!h) return RNN_OK;
  DeviceGuard dg(h->device);
  if (h->d_len) cudaFree(h->d_len);
  h->order.destroy();
  delete h;
  return RNN_OK;
}

rnn_status_t rnn_scan_get_sizes(rnn_scan_t h, size_t* ws, size_t* bws, size_t* rs) {
  if (!h) return RNN_BAD_PARAM;
  if (ws) *ws = h->workspace_bytes;
  if (bws) *bws = h->bwd_workspace_bytes;
  if (rs) *rs = h->reserve_bytes;
  return RNN_OK;
}

rnn_status_t rnn_scan_set_seq_lengths(rnn_scan_t h, const int* lengths) {
  if (!h) return RNN_BAD_PARAM;
  DeviceGuard dg(h->device);
  if (!dg.ok) return RNN_CUDA_ERROR;
  return set_lengths(h->order, lengths, h->desc.batch, h->desc.seq_len, &h->d_len, &h->has_len);
}

rnn_status_t rnn_scan_forward(rnn_scan_t h, const rnn_scan_in_t* in, const float* h0, void* y, float* hT,
                              void* workspace, void* reserve, void* stream) {
  if (!h || !y || !aligned16(y) || !aligned16(h0) || !aligned16(hT)) return RNN_BAD_PARAM;
  ScanFwdArgs f{};
  const rnn_status_t rc = scan_args(h, in, &f.a);
  if (rc != RNN_OK) return rc;
  if ((h->workspace_bytes && !workspace) || !aligned16(workspace) || !aligned16(reserve)) return RNN_BAD_WORKSPACE;
  DeviceGuard dg(h->device);
  if (!dg.ok) return RNN_CUDA_ERROR;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Ordered call(h->order, h->has_len || h->workspace_bytes || reserve, s);
  if (call.rc != RNN_OK) return call.rc;
  f.h0 = h0;
  f.hT = hT;
  f.y = y;
  if (reserve) {
    f.kept = at<float>(reserve, scan_reserve(f.a).kept);
    f.ungated = f.a.z ? at<float>(reserve, scan_reserve(f.a).ungated) : nullptr;
  }
  int n = 0;
  const int e = launch_scan_forward(f, workspace, h->bf16, s, &n);
  h->launches += n;
  return call.done(e);
}

rnn_status_t rnn_scan_backward(rnn_scan_t h, const rnn_scan_in_t* in, const void* dy, const float* dhT,
                               const rnn_scan_grad_t* grad, void* workspace, const void* reserve, void* stream) {
  if (!h || !dy || !grad || !aligned16(dy) || !aligned16(dhT)) return RNN_BAD_PARAM;
  ScanBwdArgs b{};
  const rnn_status_t rc = scan_args(h, in, &b.a);
  if (rc != RNN_OK) return rc;
  for (const void* p : {grad->dx, grad->ddt, grad->dz, grad->dB, grad->dC, grad->dA, grad->dD, grad->ddt_bias, grad->dh0})
    if (!aligned16(p)) return RNN_BAD_PARAM;
  // a gradient of something that is not there has no value
  if ((grad->dz && !in->z) || (grad->dD && !in->D) || (grad->ddt_bias && !in->dt_bias)) return RNN_BAD_PARAM;
  if (!workspace || !reserve || !aligned16(workspace) || !aligned16(reserve)) return RNN_BAD_WORKSPACE;
  DeviceGuard dg(h->device);
  if (!dg.ok) return RNN_CUDA_ERROR;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Ordered call(h->order, true, s);
  if (call.rc != RNN_OK) return call.rc;
  b.dy = dy;
  b.dhT = dhT;
  b.kept = at<float>(reserve, scan_reserve(b.a).kept);
  b.ungated = at<float>(reserve, scan_reserve(b.a).ungated);
  b.grad = *grad;
  b.work = static_cast<char*>(workspace);
  int n = 0;
  const int e = launch_scan_backward(b, h->bf16, s, &n);
  h->launches += n;
  return call.done(e);
}

rnn_status_t rnn_scan_step(rnn_scan_t h, const rnn_scan_in_t* in, float* state, int num_slots, const int* slots, void* y,
                           void* stream) {
  if (!h || !state || !y || num_slots < 0 || !aligned16(state) || !aligned16(y) || !aligned(slots, 4)) return RNN_BAD_PARAM;
  ScanStepArgs p{};
  const rnn_status_t rc = scan_args(h, in, &p.a);
  if (rc != RNN_OK) return rc;
  DeviceGuard dg(h->device);
  if (!dg.ok) return RNN_CUDA_ERROR;
  p.state = state;
  p.slots = slots;
  p.num_slots = num_slots;
  p.y = y;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Ordered call(h->order, h->has_len, s);
  if (call.rc != RNN_OK) return call.rc;
  const int e = launch_scan_step(p, h->bf16, s);
  if (!e) ++h->launches;
  return call.done(e);
}

uint64_t rnn_scan_launch_count(rnn_scan_t h) { return h ? h->launches : 0; }

rnn_status_t rnn_conv_create(const rnn_conv_desc_t* desc, rnn_conv_t* out) {
  if (!out) return RNN_BAD_PARAM;
  *out = nullptr;
  rnn_status_t rc = check_conv(desc);
  if (rc != RNN_OK) return rc;
  rnn_conv_s* h = nullptr;
  rc = make(&h);
  if (rc != RNN_OK) return rc;
  h->desc = *desc;
  h->bf16 = desc->dtype == RNN_BF16;
  *out = h;
  return RNN_OK;
}

rnn_status_t rnn_conv_destroy(rnn_conv_t h) {
  if (!h) return RNN_OK;
  DeviceGuard dg(h->device);
  if (h->d_len) cudaFree(h->d_len);
  h->order.destroy();
  delete h;
  return RNN_OK;
}

rnn_status_t rnn_conv_get_sizes(rnn_conv_t h, size_t* bws) {
  if (!h) return RNN_BAD_PARAM;
  if (bws) *bws = conv_workspace_bytes(conv_shape(h));
  return RNN_OK;
}

rnn_status_t rnn_conv_set_seq_lengths(rnn_conv_t h, const int* lengths) {
  if (!h) return RNN_BAD_PARAM;
  DeviceGuard dg(h->device);
  if (!dg.ok) return RNN_CUDA_ERROR;
  return set_lengths(h->order, lengths, h->desc.batch, h->desc.seq_len, &h->d_len, &h->has_len);
}

rnn_status_t rnn_conv_forward(rnn_conv_t h, const rnn_conv_in_t* in, const void* s0, void* y, void* sT, void* stream) {
  if (!h || !y || !aligned16(y) || !aligned16(s0) || !aligned16(sT)) return RNN_BAD_PARAM;
  ConvFwdArgs f{};
  const rnn_status_t rc = conv_args(h, in, &f.a);
  if (rc != RNN_OK) return rc;
  if (over_x(h, f.a, y)) return RNN_BAD_PARAM;
  DeviceGuard dg(h->device);
  if (!dg.ok) return RNN_CUDA_ERROR;
  f.s0 = s0;
  f.y = y;
  f.sT = sT;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Ordered call(h->order, h->has_len, s);
  if (call.rc != RNN_OK) return call.rc;
  const int e = launch_conv_forward(f, h->bf16, s);
  if (!e) ++h->launches;
  return call.done(e);
}

rnn_status_t rnn_conv_backward(rnn_conv_t h, const rnn_conv_in_t* in, const void* s0, const void* dy, const void* dsT,
                               void* dx, float* dw, float* dbias, void* ds0, void* workspace, void* stream) {
  if (!h || !dy) return RNN_BAD_PARAM;
  for (const void* p : {s0, dy, dsT, static_cast<const void*>(dx), static_cast<const void*>(dw),
                        static_cast<const void*>(dbias), static_cast<const void*>(ds0)})
    if (!aligned16(p)) return RNN_BAD_PARAM;
  ConvBwdArgs b{};
  const rnn_status_t rc = conv_args(h, in, &b.a);
  if (rc != RNN_OK) return rc;
  if (dbias && !in->bias) return RNN_BAD_PARAM;
  if (dx && (over_x(h, b.a, dx) || over_dense(h, b.a, dx, dy))) return RNN_BAD_PARAM;
  const bool weights = dw || dbias;
  if ((weights && !workspace) || !aligned16(workspace)) return RNN_BAD_WORKSPACE;
  DeviceGuard dg(h->device);
  if (!dg.ok) return RNN_CUDA_ERROR;
  b.s0 = s0; b.dy = dy; b.dsT = dsT;
  b.dx = dx; b.ds0 = ds0;
  b.dw = dw; b.dbias = dbias;
  b.partial = weights ? static_cast<float*>(workspace) : nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Ordered call(h->order, h->has_len || weights, s);
  if (call.rc != RNN_OK) return call.rc;
  int n = 0;
  const int e = launch_conv_backward(b, h->bf16, s, &n);
  h->launches += n;
  return call.done(e);
}

rnn_status_t rnn_conv_step(rnn_conv_t h, const rnn_conv_in_t* in, void* state, int num_slots, const int* slots, void* y,
                           void* stream) {
  if (!h || !state || !y || num_slots < 0 || !aligned16(state) || !aligned16(y) || !aligned(slots, 4)) return RNN_BAD_PARAM;
  ConvStepArgs p{};
  const rnn_status_t rc = conv_args(h, in, &p.a);
  if (rc != RNN_OK) return rc;
  DeviceGuard dg(h->device);
  if (!dg.ok) return RNN_CUDA_ERROR;
  p.state = state;
  p.slots = slots;
  p.num_slots = num_slots;
  p.y = y;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Ordered call(h->order, h->has_len, s);
  if (call.rc != RNN_OK) return call.rc;
  const int e = launch_conv_step(p, h->bf16, s);
  if (!e) ++h->launches;
  return call.done(e);
}

uint64_t rnn_conv_launch_count(rnn_conv_t h) { return h ? h->launches : 0; }

rnn_status_t rnn_clip_create(int num, const int64_t* counts, const int* dtypes, rnn_clip_t* out) {
  if (!out) return RNN_BAD_PARAM;
  *out = nullptr;
  if (num < 1 || num > 65536 || !counts || !dtypes) return RNN_BAD_PARAM;
  int64_t all = 0;
  for (int i = 0; i < num; ++i) {
    if (counts[i] < 0 || counts[i] > (int64_t{1} << 40) || (dtypes[i] != RNN_F32 && dtypes[i] != RNN_BF16)) return RNN_BAD_PARAM;
    all += counts[i];
    if (all > (int64_t{1} << 42)) return RNN_BAD_PARAM;
  }
  rnn_clip_s* h = nullptr;
  rnn_status_t rc = make(&h);
  if (rc != RNN_OK) return rc;
  try {
    h->dtype.assign(dtypes, dtypes + num);
    h->inplace.reserve(num);
    h->apart.reserve(num);
    h->reads.reserve(num);
    h->start.assign(1, 0);
    h->start.reserve(num + 1);
    for (int i = 0; i < num; ++i) h->start.push_back(h->start[i] + counts[i]);
  } catch (const std::bad_alloc&) {
    h->order.destroy();
    delete h;
    return RNN_INTERNAL;
  }
  h->num = num;
  // the table is on the device before the handle is handed out: calls on any stream read it
  const size_t starts = sizeof(int64_t) * (num + 1), types = sizeof(int) * num;
  if (cudaMalloc(&h->d_start, starts + types) != cudaSuccess) h->d_start = nullptr;
  h->d_dtype = reinterpret_cast<int*>(reinterpret_cast<char*>(h->d_start) + starts);
  if (!h->d_start || cudaMemcpy(h->d_start, h->start.data(), starts, cudaMemcpyHostToDevice) != cudaSuccess ||
      cudaMemcpy(h->d_dtype, h->dtype.data(), types, cudaMemcpyHostToDevice) != cudaSuccess ||
      cudaStreamSynchronize(cudaStreamLegacy) != cudaSuccess) {
    rnn_clip_destroy(h);
    return RNN_CUDA_ERROR;
  }
  *out = h;
  return RNN_OK;
}

rnn_status_t rnn_clip_destroy(rnn_clip_t h) {
  if (!h) return RNN_OK;
  DeviceGuard dg(h->device);
  if (h->d_start) cudaFree(h->d_start);
  h->order.destroy();
  delete h;
  return RNN_OK;
}

rnn_status_t rnn_clip_get_sizes(rnn_clip_t h, size_t* ws) {
  if (!h) return RNN_BAD_PARAM;
  if (ws) *ws = clip_workspace_bytes(h->num, h->num_sms);
  return RNN_OK;
}

rnn_status_t rnn_clip_scale(rnn_clip_t h, const void* const* grads, void* const* out, float max_norm, float eps, float* norm,
                            void* workspace, void* stream) {
  return clip_call(h, grads, out, max_norm, eps, norm, workspace, stream, 1);
}

rnn_status_t rnn_clip_norm(rnn_clip_t h, const void* const* grads, float* norm, void* workspace, void* stream) {
  return clip_call(h, grads, nullptr, 0.f, 0.f, norm, workspace, stream, 0);
}

uint64_t rnn_clip_launch_count(rnn_clip_t h) { return h ? h->launches : 0; }

}  // extern "C"
