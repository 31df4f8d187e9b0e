// Host side of the trainer's attention (include/leyline_train.h): argument checks,
// the layout of the workspace and the launches of its kernels.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/leyline_train.h"
#include "host_common.h"
#include "kvs_internal.h"
#include "pool_internal.h"
#include "train_internal.h"

using namespace ll;

namespace {

constexpr int64_t kMaxStride = int64_t{1} << 40;
// Shares of tiles of keys that the workspace has room for, where they may be cut at all,
// and shares of one tile at most.
constexpr int64_t kTrainParts = 2048, kTrainShares = 16;

ll_status check_sizes(const kvs_attend_desc* d) {
  if (d->n < 0) return fail(LL_EINVAL, "n must not be negative");
  if (d->n_pad < 1 || d->n_pad >= (int64_t{1} << 31) - 1) return fail(LL_EINVAL, "n_pad must be in [1, 2^31 - 2]");
  if (d->kv_heads < 1 || d->heads < 1 || d->heads % d->kv_heads)
    return fail(LL_EINVAL, "heads must be a positive multiple of kv_heads");
  if (d->key_dim < 8 || d->key_dim > 256 || d->key_dim % 8 || d->value_dim < 8 || d->value_dim > 256 || d->value_dim % 8)
    return fail(LL_EINVAL, "key_dim and value_dim must be multiples of 8 in [8, 256]");
  const int64_t rows = int64_t{d->n} * d->heads, blocks = ceil_div(d->n_pad, kTrainBlock), most = int64_t{1} << 23;
  if (rows >= most || rows * blocks >= most)
    return fail(LL_EUNSUPPORTED, "n * heads * ceil(n_pad / 64) must stay below 2^23");
  return LL_OK;
}

// Rows of a tensor may not overlap where they are written: some order of the axes
// has each one's stride outside the ones below it.
bool rows_apart(const kvs_heads& x, int64_t n, int64_t tokens, int64_t heads, int64_t width) {
  int64_t size[3] = {n, tokens, heads}, stride[3] = {x.rollout_stride, x.token_stride, x.head_stride};
  int64_t span = width;   // values that the axes so far cover
  for (int done = 0; done < 3; ++done) {
    int best = -1;
    for (int i = 0; i < 3; ++i)
      if (size[i] > 1 && (best < 0 || stride[i] < stride[best])) best = i;
    if (best < 0) break;
    if (stride[best] < span) return false;
    span += stride[best] * (size[best] - 1);
    size[best] = 1;
  }
  return true;
}

ll_status check_heads(const kvs_heads& x, const kvs_attend_desc* d, int64_t heads, int64_t width, bool written, const char* name) {
  if (!x.data) return fail(LL_EINVAL, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(x.data) & 15) return fail(LL_EINVAL, "%s is not 16-byte aligned", name);
  const int64_t size[3] = {d->n, d->n_pad, heads}, stride[3] = {x.rollout_stride, x.token_stride, x.head_stride};
  for (int i = 0; i < 3; ++i)
    if (size[i] > 1 && ((stride[i] & 7) || stride[i] < 0 || stride[i] > kMaxStride))
      return fail(LL_EINVAL, "%s: strides must be multiples of 8 values in [0, 2^40]", name);
  if (written && !rows_apart(x, d->n, d->n_pad, heads, width)) return fail(LL_EINVAL, "%s: rows overlap", name);
  return LL_OK;
}

Heads view(const kvs_heads& x, const kvs_attend_desc* d, int64_t heads) {
  // a stride that no second index uses says nothing
  return Heads{static_cast<uint16_t*>(x.data), d->n > 1 ? x.rollout_stride : 0, d->n_pad > 1 ? x.token_stride : 0,
               heads > 1 ? x.head_stride : 0};
}

// The workspace's parts; returns its size.
int64_t lay_out(TrainLaunch* a, bool backward, char* at) {
  int64_t size = 0;
  auto take = [&](int64_t bytes) {
    char* p = at + size;
    size = static_cast<int64_t>(align_up(static_cast<size_t>(size + bytes), 256));
    return p;
  };
  const int64_t nb = int64_t{a->n} * a->blocks;
  a->keys = reinterpret_cast<KeyBlock*>(take(nb * static_cast<int64_t>(sizeof(KeyBlock))));
  const int64_t listed = int64_t{a->n} * a->list_keys();
  a->list = reinterpret_cast<KeyEntry*>(take(listed * static_cast<int64_t>(sizeof(KeyEntry))));
  a->list_blocks = reinterpret_cast<KeyBlock*>(take(listed / kTrainBlock * static_cast<int64_t>(sizeof(KeyBlock))));
  a->list_count = reinterpret_cast<int32_t*>(take(int64_t{a->n} * a->epochs * 4));
  a->odd_v = reinterpret_cast<uint32_t*>(take(nb * a->kv_heads * 4));
  if (backward) {
    a->order = reinterpret_cast<int32_t*>(take(int64_t{a->n} * a->n_pad * 4));
    a->seen_keys = reinterpret_cast<int32_t*>(take(int64_t{a->n} * 4));
    a->work = reinterpret_cast<int64_t*>(take(int64_t{a->n} * 8));
    a->odd_k = reinterpret_cast<uint32_t*>(take(nb * a->kv_heads * 4));
    a->odd_q = reinterpret_cast<uint32_t*>(take(nb * a->heads * 4));
    a->odd_do = reinterpret_cast<uint32_t*>(take(nb * a->heads * 4));
    a->delta = reinterpret_cast<float*>(take(int64_t{a->n} * a->heads * a->n_pad * 4));
    a->ref = reinterpret_cast<float*>(take(int64_t{a->n} * a->heads * a->n_pad * 4));
    const int64_t units = int64_t{a->n} * a->kv_heads * ceil_div(a->n_pad, kTrainTile);
    const HeadShape w = head_shape(a->dk, a->dv);
    a->used = reinterpret_cast<int32_t*>(take(units * 4));
    // (as much room for the longest n_pad as for any shorter one, though long ones are not cut)
    a->parts = reinterpret_cast<float*>(take(std::min(units * kTrainShares, kTrainParts) * kTrainTile * (w.dk + w.dv) * 4));
  }
  return size;
}

TrainLaunch sizes(const kvs_attend_desc* d) {
  TrainLaunch a{};
  a.n = d->n;
  a.heads = d->heads;
  a.kv_heads = d->kv_heads;
  a.group = d->heads / d->kv_heads;
  a.n_pad = static_cast<int32_t>(d->n_pad);
  a.blocks = static_cast<int32_t>(ceil_div(d->n_pad, kTrainBlock));
  a.epoch = static_cast<int32_t>(ceil_div(ceil_div(d->n_pad, kTrainEpochs), kTrainTile) * kTrainTile);
  a.epochs = static_cast<int32_t>(ceil_div(d->n_pad, a.epoch));
  a.dk = d->key_dim;
  a.dv = d->value_dim;
  // A tile of keys that many queries see takes long: with few tiles the longest may be
  // cut (see share_blocks), as far as there is room for the shares' sums.
  const int64_t units = std::max<int64_t>(1, int64_t{a.n} * a.kv_heads * ceil_div(a.n_pad, kTrainTile));
  a.shares = static_cast<int32_t>(std::clamp<int64_t>(kTrainParts / units, 1, kTrainShares));
  return a;
}

ll_status fill(const kvs_attend_desc* d, bool backward, TrainLaunch* a) {
  ll_status rc = check_sizes(d);
  if (rc) return rc;
  if ((rc = check_scale(d->scale, d->cap))) return rc;
  *a = sizes(d);
  if (d->n == 0) return LL_OK;
  if (!d->death || (reinterpret_cast<uintptr_t>(d->death) & 3)) return fail(LL_EINVAL, "death is NULL or not 4-byte aligned");
  if ((rc = check_heads(d->q, d, d->heads, d->key_dim, false, "q"))) return rc;
  if ((rc = check_heads(d->k, d, d->kv_heads, d->key_dim, false, "k"))) return rc;
  if ((rc = check_heads(d->v, d, d->kv_heads, d->value_dim, false, "v"))) return rc;
  if ((rc = check_heads(d->out, d, d->heads, d->value_dim, !backward, "out"))) return rc;
  if (!d->lse || (reinterpret_cast<uintptr_t>(d->lse) & 3)) return fail(LL_EINVAL, "lse is NULL or not 4-byte aligned");
  if (!d->workspace || (reinterpret_cast<uintptr_t>(d->workspace) & 15))
    return fail(LL_EINVAL, "the workspace is NULL or not 16-byte aligned");
  const int64_t need = lay_out(a, backward, static_cast<char*>(d->workspace));
  if (d->workspace_bytes < need)
    return fail(LL_EINVAL, "a workspace of %lld bytes, but %lld are needed", (long long)d->workspace_bytes, (long long)need);
  a->scale = d->scale;
  a->cap = d->cap;
  a->death = d->death;
  a->q = view(d->q, d, d->heads);
  a->k = view(d->k, d, d->kv_heads);
  a->v = view(d->v, d, d->kv_heads);
  a->out = view(d->out, d, d->heads);
  a->lse = d->lse;
  return LL_OK;
}

ll_status run(kvs_ctx* c, const TrainLaunch& a, hipError_t (*launch)(const TrainLaunch&, hipStream_t), const char* what, void* stream) {
  if (a.n == 0) return LL_OK;
  DeviceGuard g(kvs_device(c));
  if (!g.ok()) return fail(LL_EDEVICE, "hipSetDevice(%d) failed", kvs_device(c));
  hipError_t e = launch(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(LL_EDEVICE, "%s: %s", what, hipGetErrorString(e));
  return LL_OK;
}

}  // namespace

extern "C" {

ll_status kvs_attend_workspace(const kvs_attend_desc* d, int32_t backward, int64_t* bytes) {
  if (!d || !bytes) return fail(LL_EINVAL, "NULL argument");
  if (backward != 0 && backward != 1) return fail(LL_EINVAL, "backward must be 0 or 1");
  if (ll_status rc = check_sizes(d)) return rc;
  TrainLaunch a = sizes(d);
  *bytes = lay_out(&a, backward != 0, nullptr);
  return LL_OK;
}

ll_status kvs_attend(kvs_ctx* c, const kvs_attend_desc* d, void* stream) {
  if (!c) return fail(LL_EINVAL, "context is NULL");
  if (!d) return fail(LL_EINVAL, "NULL argument");
  TrainLaunch a;
  if (ll_status rc = fill(d, false, &a)) return rc;
  return run(c, a, launch_train, "train_kernel launch", stream);
}

ll_status kvs_attend_backward(kvs_ctx* c, const kvs_attend_backward_desc* d, void* stream) {
  if (!c) return fail(LL_EINVAL, "context is NULL");
  if (!d) return fail(LL_EINVAL, "NULL argument");
  TrainLaunch a;
  ll_status rc = fill(&d->f, true, &a);
  if (rc) return rc;
  if (a.n == 0) return LL_OK;
  const kvs_attend_desc* f = &d->f;
  if ((rc = check_heads(d->dout, f, f->heads, f->value_dim, false, "dout"))) return rc;
  if ((rc = check_heads(d->dq, f, f->heads, f->key_dim, true, "dq"))) return rc;
  if ((rc = check_heads(d->dk, f, f->kv_heads, f->key_dim, true, "dk"))) return rc;
  if ((rc = check_heads(d->dv, f, f->kv_heads, f->value_dim, true, "dv"))) return rc;
  a.dout = view(d->dout, f, f->heads);
  a.dq = view(d->dq, f, f->heads);
  a.dk_ = view(d->dk, f, f->kv_heads);
  a.dv_ = view(d->dv, f, f->kv_heads);
  return run(c, a, launch_train_back, "train_back_kernel launch", stream);
}

}  // extern "C"
