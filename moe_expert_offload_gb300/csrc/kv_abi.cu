// C ABI entry points of the 4-bit key/value cache (declared in include/moe.h):
// argument checks on the host, then kernel launches on the caller's stream.
#include "kv_common.cuh"

namespace {

using moe::set_error;
using moe::set_ok;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int cuda_fail(cudaError_t e, const char* where) {
  return set_error(MOE_ECUDA, "%s: %s", where, cudaGetErrorString(e));
}

// the cache's shape alone
int check_shape(const moe_kv* kv) {
  if (!kv) return set_error(MOE_EINVAL, "kv is NULL");
  if (kv->num_blocks < 1) return set_error(MOE_EINVAL, "num_blocks must be >= 1");
  if (kv->block_tokens != 16 && kv->block_tokens != 32 && kv->block_tokens != 64 &&
      kv->block_tokens != 128)
    return set_error(MOE_EINVAL, "block_tokens must be 16, 32, 64 or 128");
  if (kv->kv_heads < 1 || kv->kv_heads > MOE_KV_MAX_HEADS)
    return set_error(MOE_EINVAL, "kv_heads must be in 1..%d", MOE_KV_MAX_HEADS);
  if (kv->head_dim != 64 && kv->head_dim != 128 && kv->head_dim != 256)
    return set_error(MOE_EUNSUPPORTED, "head_dim must be 64, 128 or 256");
  if ((int64_t)kv->num_blocks * kv->block_tokens > 0x7fffffff)
    return set_error(MOE_EUNSUPPORTED, "num_blocks * block_tokens exceeds 2^31 - 1 slots");
  return MOE_OK;
}

// and its tables
int check_tables(const moe_kv* kv) {
  const int rc = check_shape(kv);
  if (rc) return rc;
  if (kv->max_rows < 1 || kv->max_blocks < 1)
    return set_error(MOE_EINVAL, "max_rows and max_blocks must be >= 1");
  if ((int64_t)kv->max_blocks * kv->block_tokens > 0x7fffffff)
    return set_error(MOE_EUNSUPPORTED, "max_blocks * block_tokens exceeds 2^31 - 1 positions");
  if (!kv->block_table || !kv->seq_len || !kv->free_list || !kv->free_count)
    return set_error(MOE_EINVAL, "kv table pointer is NULL");
  return MOE_OK;
}

int check_pool(const moe_kv* kv) {
  if (!kv->pool) return set_error(MOE_EINVAL, "kv pool is NULL");
  if (!aligned(kv->pool, 128)) return set_error(MOE_EINVAL, "kv pool must be 128-byte aligned");
  return MOE_OK;
}

int check_batch(const moe_kv_batch* b) {
  if (!b) return set_error(MOE_EINVAL, "batch is NULL");
  if (b->max_tokens < 1 || b->max_rows < 1)
    return set_error(MOE_EINVAL, "batch max_tokens and max_rows must be >= 1");
  if (!b->q_start || !b->kv_len || !b->slot || !b->pos || !b->err)
    return set_error(MOE_EINVAL, "batch buffer pointer is NULL");
  return MOE_OK;
}

int check_rows(const moe_kv* kv, const moe_kv_batch* b, int32_t rows) {
  if (rows < 1) return set_error(MOE_EINVAL, "rows must be >= 1");
  if (rows > kv->max_rows || rows > b->max_rows)
    return set_error(MOE_ECAPACITY, "rows = %d exceeds the cache's %d or the batch's %d", rows,
                     kv->max_rows, b->max_rows);
  return MOE_OK;
}

int check_tokens(const moe_kv_batch* b, int32_t T) {
  if (T < 0) return set_error(MOE_EINVAL, "T must be >= 0");
  if (T > b->max_tokens)
    return set_error(MOE_ECAPACITY, "T = %d exceeds the batch's %d tokens", T, b->max_tokens);
  return MOE_OK;
}

int check_tree(const moe_kv_tree* t) {
  if (t->max_new < 1 || t->max_new > MOE_KV_MAX_TREE)
    return set_error(MOE_EINVAL, "tree max_new must be in 1..%d", MOE_KV_MAX_TREE);
  if (!t->parent) return set_error(MOE_EINVAL, "tree parent is NULL");
  return MOE_OK;
}

// a view and its tree's visibility of T tokens
int check_view(const moe_kv_view* v, int32_t T) {
  if (!v) return set_error(MOE_EINVAL, "view is NULL");
  if (v->window < 0) return set_error(MOE_EINVAL, "window must be >= 0");
  if (v->sinks < 0) return set_error(MOE_EINVAL, "sinks must be >= 0");
  if (!v->tree) return MOE_OK;
  const int rc = check_tree(v->tree);
  if (rc) return rc;
  if (!v->tree->seen) return set_error(MOE_EINVAL, "tree seen is NULL");
  if ((int64_t)T * moe_kv_tree_words(v->tree->max_new) > 0x7fffffff)
    return set_error(MOE_EUNSUPPORTED, "T * moe_kv_tree_words exceeds 2^31 - 1");
  return MOE_OK;
}

int check_batch_rows(const moe_kv_batch* b, int32_t rows) {
  if (rows < 1) return set_error(MOE_EINVAL, "rows must be >= 1");
  if (rows > b->max_rows)
    return set_error(MOE_ECAPACITY, "rows = %d exceeds the batch's %d", rows, b->max_rows);
  return MOE_OK;
}

int check_strided(const char* what, const void* p, int64_t token_stride, int64_t head_stride) {
  if (!p) return set_error(MOE_EINVAL, "%s is NULL", what);
  if (!aligned(p, 16) || token_stride % 8 || head_stride % 8 || token_stride < 0 ||
      head_stride < 0)
    return set_error(MOE_EINVAL, "%s must be 16-byte aligned, its strides >= 0 and multiples of 8",
                     what);
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_kv_block_bytes(const moe_kv* kv) {
  if (check_shape(kv) != MOE_OK) return 0;
  return (size_t)kv->kv_heads * (kv->block_tokens / moe::kv::kTile) *
         moe::kv::tile_bytes(kv->head_dim);
}

int moe_kv_reset(const moe_kv* kv, moe_stream_t stream) {
  const int rc = check_tables(kv);
  if (rc) return rc;
  const cudaError_t e = moe::kv::launch_reset(*kv, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kv reset launch");
  return set_ok();
}

int moe_kv_plan(const moe_kv* kv, const int32_t* new_len, int32_t rows, const moe_kv_batch* batch,
                moe_stream_t stream) {
  int rc = check_tables(kv);
  if (!rc) rc = check_batch(batch);
  if (!rc) rc = check_rows(kv, batch, rows);
  if (rc) return rc;
  if (!new_len) return set_error(MOE_EINVAL, "moe_kv_plan: new_len is NULL");
  moe::kv::PlanArgs a;
  a.kv = *kv;
  a.batch = *batch;
  a.new_len = new_len;
  a.rows = rows;
  const cudaError_t e = moe::kv::launch_plan(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kv plan launch");
  return set_ok();
}

int moe_qkv_store(const moe_kv* kv, const moe_kv_batch* batch, const moe_rope* rope,
                  const moe_qkv* proj, int32_t T, const int32_t* positions, void* q_out,
                  moe_stream_t stream) {
  int rc = check_shape(kv);
  if (!rc) rc = check_pool(kv);
  if (!rc) rc = check_batch(batch);
  if (!rc) rc = check_tokens(batch, T);
  if (rc) return rc;
  if (T == 0) return set_ok();
  if (!proj) return set_error(MOE_EINVAL, "proj is NULL");
  if (proj->q_heads < 1 || proj->q_heads > MOE_KV_MAX_HEADS)
    return set_error(MOE_EINVAL, "q_heads must be in 1..%d", MOE_KV_MAX_HEADS);
  if (!(proj->eps >= 0.0f)) return set_error(MOE_EINVAL, "eps must be >= 0");
  if ((rc = check_strided("q", proj->q, proj->q_token_stride, proj->q_head_stride))) return rc;
  if ((rc = check_strided("k", proj->k, proj->k_token_stride, proj->k_head_stride))) return rc;
  if ((rc = check_strided("v", proj->v, proj->v_token_stride, proj->v_head_stride))) return rc;
  if (!aligned(proj->q_norm, 16) || !aligned(proj->k_norm, 16))
    return set_error(MOE_EINVAL, "q_norm and k_norm must be 16-byte aligned");
  if (!q_out || !aligned(q_out, 16))
    return set_error(MOE_EINVAL, "q_out is NULL or not 16-byte aligned");
  moe::kv::StoreArgs a = {};
  if (rope && rope->rotary_dim != 0) {
    if (rope->rotary_dim < 0 || rope->rotary_dim % 16 || rope->rotary_dim > kv->head_dim)
      return set_error(MOE_EINVAL, "rotary_dim must be a multiple of 16 up to head_dim");
    if (!rope->table || !aligned(rope->table, 16))
      return set_error(MOE_EINVAL, "rope table is NULL or not 16-byte aligned");
    if (rope->max_pos < 1) return set_error(MOE_EINVAL, "max_pos must be >= 1");
    if (rope->adjacent != 0 && rope->adjacent != 1)
      return set_error(MOE_EINVAL, "adjacent must be 0 or 1");
    if (rope->axes < 1 || rope->axes > MOE_ROPE_MAX_AXES)
      return set_error(MOE_EINVAL, "axes must be in 1..%d", MOE_ROPE_MAX_AXES);
    if (rope->axes > 1 && !positions)
      return set_error(MOE_EINVAL, "several axes need positions [axes][T]");
    for (int i = 0; i < rope->rotary_dim / 2; ++i)
      if (rope->pair_axis[i] >= rope->axes)
        return set_error(MOE_EINVAL, "pair_axis[%d] = %d is not below axes = %d", i,
                         (int)rope->pair_axis[i], rope->axes);
    a.rope = *rope;
  }
  a.kv = *kv;
  a.proj = *proj;
  a.slot = batch->slot;
  a.positions = positions ? positions : batch->pos;
  a.err = batch->err;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.T = T;
  const cudaError_t e = moe::kv::launch_store(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "qkv store launch");
  return set_ok();
}

int moe_kv_load(const moe_kv* kv, const int32_t* slots, int32_t T, void* k, void* v, int32_t* err,
                moe_stream_t stream) {
  int rc = check_shape(kv);
  if (!rc) rc = check_pool(kv);
  if (rc) return rc;
  if (T < 0) return set_error(MOE_EINVAL, "T must be >= 0");
  if (T == 0) return set_ok();
  if (!slots || !k || !v) return set_error(MOE_EINVAL, "moe_kv_load: NULL argument");
  if (!aligned(k, 16) || !aligned(v, 16))
    return set_error(MOE_EINVAL, "moe_kv_load: k and v must be 16-byte aligned");
  moe::kv::LoadArgs a;
  a.kv = *kv;
  a.slot = slots;
  a.k = static_cast<uint16_t*>(k);
  a.v = static_cast<uint16_t*>(v);
  a.err = err;
  a.T = T;
  const cudaError_t e = moe::kv::launch_load(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kv load launch");
  return set_ok();
}

static int check_heads(const moe_kv* kv, int32_t heads, int32_t max_new) {
  if (heads < 1 || heads > MOE_KV_MAX_HEADS || heads % kv->kv_heads)
    return set_error(MOE_EINVAL, "heads must be a multiple of kv_heads up to %d",
                     MOE_KV_MAX_HEADS);
  if (heads / kv->kv_heads > MOE_KV_MAX_GROUP)
    return set_error(MOE_EUNSUPPORTED, "more than %d query heads on a kv head", MOE_KV_MAX_GROUP);
  if (max_new < 1) return set_error(MOE_EINVAL, "max_new must be >= 1");
  return MOE_OK;
}

size_t moe_kv_attention_workspace_bytes(const moe_kv* kv, int32_t rows, int32_t T, int32_t heads,
                                        int32_t max_new) {
  if (check_shape(kv) != MOE_OK || check_heads(kv, heads, max_new) != MOE_OK) return 0;
  if (rows < 1 || T < 0) {
    set_error(MOE_EINVAL, "rows must be >= 1 and T >= 0");
    return 0;
  }
  return moe::kv::attn_workspace_bytes(*kv, heads, max_new, true);
}

static int attention(const moe_kv* kv, const moe_kv_batch* batch, const moe_kv_view* view,
                     int32_t rows, const void* q, int32_t T, int32_t heads, int32_t max_new,
                     float scale, void* workspace, size_t workspace_bytes, void* out,
                     moe_stream_t stream) {
  int rc = check_tables(kv);
  if (!rc) rc = check_pool(kv);
  if (!rc) rc = check_batch(batch);
  if (!rc) rc = check_rows(kv, batch, rows);
  if (!rc) rc = check_tokens(batch, T);
  if (!rc) rc = check_heads(kv, heads, max_new);
  if (!rc && view) rc = check_view(view, T);
  if (rc) return rc;
  if (T == 0) return set_ok();
  if (!q || !out || !workspace) return set_error(MOE_EINVAL, "moe_kv_attention: NULL argument");
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 256))
    return set_error(MOE_EINVAL, "q and out (16 B) and workspace (256 B) alignment");
  if (!(scale > 0.0f) || scale > 3.0e38f)
    return set_error(MOE_EINVAL, "scale must be finite and > 0");
  const size_t need = moe::kv::attn_workspace_bytes(*kv, heads, max_new, view != nullptr);
  if (workspace_bytes < need)
    return set_error(MOE_ECAPACITY, "workspace %zu < %zu bytes", workspace_bytes, need);
  moe::kv::AttnArgs a = {};
  a.kv = *kv;
  a.batch = *batch;
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.ws = workspace;
  a.rows = rows;
  a.T = T;
  a.heads = heads;
  a.max_new = max_new;
  a.scale = scale;
  if (view) {
    a.window = view->window;
    a.sinks = view->window ? view->sinks : 0;
    if (view->tree) {
      a.tree = view->tree->seen;
      a.tree_max = view->tree->max_new;
      a.words = moe_kv_tree_words(a.tree_max);
    }
  }
  const cudaError_t e = moe::kv::launch_attention(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kv attention launch");
  return set_ok();
}

int moe_kv_attention(const moe_kv* kv, const moe_kv_batch* batch, int32_t rows, const void* q,
                     int32_t T, int32_t heads, int32_t max_new, float scale, void* workspace,
                     size_t workspace_bytes, void* out, moe_stream_t stream) {
  return attention(kv, batch, nullptr, rows, q, T, heads, max_new, scale, workspace,
                   workspace_bytes, out, stream);
}

int moe_kv_attention_view(const moe_kv* kv, const moe_kv_batch* batch, const moe_kv_view* view,
                          int32_t rows, const void* q, int32_t T, int32_t heads, int32_t max_new,
                          float scale, void* workspace, size_t workspace_bytes, void* out,
                          moe_stream_t stream) {
  if (!view) return set_error(MOE_EINVAL, "view is NULL");
  return attention(kv, batch, view, rows, q, T, heads, max_new, scale, workspace, workspace_bytes,
                   out, stream);
}

int32_t moe_kv_tree_words(int32_t max_new) {
  return max_new < 1 || max_new > MOE_KV_MAX_TREE ? 0 : 1 + (max_new + 31) / 32;
}

int moe_kv_tree_plan(const moe_kv_batch* batch, const moe_kv_view* view, int32_t rows, int32_t T,
                     moe_stream_t stream) {
  int rc = check_batch(batch);
  if (!rc) rc = check_batch_rows(batch, rows);
  if (!rc) rc = check_tokens(batch, T);
  if (!rc) rc = check_view(view, T);
  if (rc) return rc;
  if (!view->tree) return set_error(MOE_EINVAL, "moe_kv_tree_plan: the view has no tree");
  if (T == 0) return set_ok();
  moe::kv::TreePlanArgs a;
  a.batch = *batch;
  a.parent = view->tree->parent;
  a.seen = view->tree->seen;
  a.rows = rows;
  a.T = T;
  a.max_new = view->tree->max_new;
  a.words = moe_kv_tree_words(a.max_new);
  a.window = view->window;
  a.sinks = view->sinks;
  const cudaError_t e = moe::kv::launch_tree_plan(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kv tree plan launch");
  return set_ok();
}

int moe_kv_tree_accept(const moe_kv_batch* batch, const moe_kv_tree* tree, int32_t rows, int32_t T,
                       const int32_t* token, const int32_t* next, int32_t* path, int32_t* kept,
                       int32_t* drop, int32_t* last, moe_stream_t stream) {
  int rc = check_batch(batch);
  if (!rc) rc = check_batch_rows(batch, rows);
  if (!rc) rc = check_tokens(batch, T);
  if (!rc) rc = tree ? check_tree(tree) : set_error(MOE_EINVAL, "tree is NULL");
  if (rc) return rc;
  if (!kept || !drop || !last || (T && (!token || !next || !path)))
    return set_error(MOE_EINVAL, "moe_kv_tree_accept: NULL argument");
  moe::kv::TreeAcceptArgs a;
  a.batch = *batch;
  a.parent = tree->parent;
  a.token = token;
  a.next = next;
  a.path = path;
  a.kept = kept;
  a.drop = drop;
  a.last = last;
  a.rows = rows;
  a.T = T;
  a.max_new = tree->max_new;
  const cudaError_t e = moe::kv::launch_tree_accept(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "kv tree accept launch");
  return set_ok();
}

int moe_kv_tree_keep(const moe_kv* kv, int32_t layers, const moe_kv_batch* batch, int32_t rows,
                     int32_t T, const int32_t* path, const int32_t* kept, moe_stream_t stream) {
  if (layers < 1) return set_error(MOE_EINVAL, "layers must be >= 1");
  for (int l = 0; l < (kv ? layers : 1); ++l) {
    int rc = check_shape(kv ? kv + l : nullptr);
    if (!rc) rc = check_pool(kv + l);
    if (rc) return rc;
    if (kv[l].num_blocks != kv->num_blocks || kv[l].block_tokens != kv->block_tokens ||
        kv[l].kv_heads != kv->kv_heads || kv[l].head_dim != kv->head_dim)
      return set_error(MOE_EINVAL, "layer %d's pool has another shape than the first one's", l);
  }
  int rc = check_batch(batch);
  if (!rc) rc = check_batch_rows(batch, rows);
  if (!rc) rc = check_tokens(batch, T);
  if (rc) return rc;
  if (T == 0) return set_ok();
  if (!path || !kept) return set_error(MOE_EINVAL, "moe_kv_tree_keep: NULL argument");
  moe::kv::TreeKeepArgs a;
  a.batch = *batch;
  a.path = path;
  a.kept = kept;
  a.rows = rows;
  a.T = T;
  a.num_blocks = kv->num_blocks;
  a.block_tokens = kv->block_tokens;
  a.kv_heads = kv->kv_heads;
  for (int at = 0; at < layers; at += a.layers) {
    a.layers = layers - at < moe::kv::kKeepLayers ? layers - at : moe::kv::kKeepLayers;
    for (int l = 0; l < a.layers; ++l) a.pool[l] = static_cast<uint8_t*>(kv[at + l].pool);
    const cudaError_t e = moe::kv::launch_tree_keep(a, kv->head_dim, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "kv tree keep launch");
  }
  return set_ok();
}

}  // extern "C"
