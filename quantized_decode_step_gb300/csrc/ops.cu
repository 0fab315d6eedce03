// The pieces of a decoding loop outside the built-in step: session extension, one layer's cache write, read-back
// and attention over a context's pool, and sampling.
#include "engine.h"

namespace mag {

// The rows of a call: session sids[i]'s newest ntok[i] tokens, sessions without any left out. Errors leave `r`
// unspecified.
static mag_status op_rows(mag_ctx* c, const char* what, int32_t layer, int32_t n, const int32_t* sids,
                          const int32_t* ntok, KvRows& r) {
  r = KvRows{};
  if (n < 1 || n > MAG_MAX_BATCH)
    return fail(c, MAG_ERR_INVALID_ARG, "%s: %d sessions not in 1..%d", what, n, MAG_MAX_BATCH);
  if (!sids || !ntok) return fail(c, MAG_ERR_INVALID_ARG, "%s: null session or token list", what);
  if (layer < 0 || layer >= c->L) return fail(c, MAG_ERR_INVALID_ARG, "%s: bad layer %d", what, layer);
  int64_t rows = 0;
  for (int i = 0; i < n; ++i) {
    const int sid = sids[i];
    if (sid < 0 || sid >= (int)c->sessions.size() || !c->sessions[sid].open)
      return fail(c, MAG_ERR_INVALID_ARG, "%s: session %d is not open", what, sid);
    for (int j = 0; j < i; ++j)
      if (sids[j] == sid) return fail(c, MAG_ERR_INVALID_ARG, "%s: session %d appears twice", what, sid);
    const Session& s = c->sessions[sid];
    if (ntok[i] < 0 || ntok[i] > s.len)
      return fail(c, MAG_ERR_INVALID_ARG, "%s: %d tokens of session %d, which holds %d", what, ntok[i], sid, s.len);
    if (ntok[i] == 0) continue;
    if (rows + ntok[i] > (1 << 24)) return fail(c, MAG_ERR_INVALID_ARG, "%s: more than 2^24 tokens", what);
    r.seg[r.n_seg++] = KvSeg{(int32_t)rows, ntok[i], s.len - ntok[i], sid};
    rows += ntok[i];
  }
  r.n_rows = (int32_t)rows;
  return MAG_OK;
}

// fp16 rows of `width` values: 16-byte aligned, a row stride that is a multiple of 8 values and holds a row.
static mag_status op_buffer(mag_ctx* c, const char* what, const char* name, const void* p, int64_t ld, int64_t width) {
  if (!p) return fail(c, MAG_ERR_INVALID_ARG, "%s: %s is null", what, name);
  if (reinterpret_cast<uintptr_t>(p) & 15) return fail(c, MAG_ERR_INVALID_ARG, "%s: %s is not 16-byte aligned", what, name);
  if (ld < width || ld % 8)
    return fail(c, MAG_ERR_INVALID_ARG, "%s: %s has row stride %lld, not a multiple of 8 of at least %lld", what, name,
                (long long)ld, (long long)width);
  return MAG_OK;
}

static mag_status op_device(mag_ctx* c, const char* what) {
  int dev = -1;
  CUDA_TRY(c, cudaGetDevice(&dev));
  if (dev != c->device)
    return fail(c, MAG_ERR_INVALID_ARG, "%s: make the context's device %d current (not %d)", what, c->device, dev);
  return MAG_OK;
}

// Work that a graph must not hold: it would be done at the capture and not again, or read host memory at a replay.
static mag_status op_not_captured(mag_ctx* c, const char* what, const char* why) {
  cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
  CUDA_TRY(c, cudaStreamIsCapturing(c->stream, &st));
  if (st != cudaStreamCaptureStatusNone) return fail(c, MAG_ERR_INVALID_ARG, "%s: the stream is being captured; %s", what, why);
  return MAG_OK;
}

// Blocks of a read: the pool blocks that each session's tokens touch.
static int read_blocks(const KvRows& r, int32_t* blk0) {
  int n = 0;
  for (int i = 0; i < r.n_seg; ++i) {
    blk0[i] = n;
    n += ((r.seg[i].pos0 + r.seg[i].n_tok - 1) >> 4) - (r.seg[i].pos0 >> 4) + 1;
  }
  return n;
}

// The workspace of split attention tiles, made by the first call that needs it.
static mag_status attend_workspace(mag_ctx* c) {
  if (c->at_part) return MAG_OK;
  const mag_status cap = op_not_captured(c, "attend", "make one call before the capture, which makes the workspace");
  if (cap != MAG_OK) return cap;
  const size_t part = kAttendPartFloats * 4, ml = kAttendMlFloats * 4, cnt = kAttendArrivals * 4;
  cudaError_t e;
  float *p = nullptr, *m = nullptr;
  uint32_t* n = nullptr;
  if ((e = dev_malloc(&p, part)) != cudaSuccess || (e = dev_malloc(&m, ml)) != cudaSuccess ||
      (e = dev_malloc(&n, cnt)) != cudaSuccess) {
    cudaFree(p);
    cudaFree(m);
    return fail(c, MAG_ERR_OOM, "attend: workspace: %s", cudaGetErrorString(e));
  }
  if ((e = cudaMemsetAsync(n, 0, cnt, c->stream)) != cudaSuccess) {
    cudaFree(p);
    cudaFree(m);
    cudaFree(n);
    return fail(c, MAG_ERR_CUDA, "attend: workspace: %s", cudaGetErrorString(e));
  }
  c->at_part = p;
  c->at_ml = m;
  c->at_arrivals = n;
  c->other_bytes += part + ml + cnt;
  return MAG_OK;
}

// Which kernel a session goes to, by its packed rows (tokens times query heads per KV head). Up to kFewRows, one
// tile of the register kernel, that one (us, register and streaming; 32 heads over 8 KV heads of 128): 16 rows on
// 20,000 keys, one session FP16 24 and 27, INT8 22 and 32, INT4 24 and 28; 16 sessions 217 and 237, 169 and 297,
// 171 and 228. Up to kStreamRows, one tile of the streaming kernel, that one: 20 rows, one session 29 and 27, 28
// and 32, 30 and 28; 16 sessions 421 and 238, 323 and 296, 324 and 228; of 2,000 keys 59 and 38, 46 and 40, 49 and
// 33 (one INT8 session, and one or four short ones, are faster in registers, by a tenth). So a fifth draft token
// costs 16 INT8 sessions 169 -> 296, and two register tiles would cost them more. Others to the two-tile one
// (streaming and two-tile: 256 rows on 20,000 keys 41 and 32, 49 and 40, 42 and 38; on 800 keys 12 and 15, 14 and
// 17, 13 and 17; 2,048 rows on 800 26 and 26, 31 and 31, 27 and 31; 8,192 on 2,000 166 and 108, 240 and 141, 211
// and 137). The kernels of one call run one after another.
constexpr int kFewRows = 16, kStreamRows = 128;
constexpr float kLog2e = 1.44269504088896340736f;

static mag_status run_attend(mag_ctx* c, int32_t layer, const KvRows& rows, const void* q, int64_t ldq, void* out, int64_t ldo,
                      int32_t window, float scale) {
  AttendArgs a = {};
  a.q = (const __half*)q;
  a.ldq = ldq;
  a.o = (__half*)out;
  a.ldo = ldo;
  a.n_heads = c->Hq;
  a.n_kv_heads = c->Hkv;
  a.group = c->G;
  a.layer = layer;
  a.window = window;
  a.scale_log2 = scale * kLog2e;
  a.pool = pool_geom(c);
  a.err = c->d_err;
  a.wait_limit = c->wait_limit;
  const mag_status ws = attend_workspace(c);
  if (ws != MAG_OK) return ws;
  a.part = c->at_part;
  a.part_ml = c->at_ml;
  a.arrivals = c->at_arrivals;
  const Launch L{c->stream, false, nullptr};
  for (int kind = 0; kind < 3; ++kind) {
    int64_t most = 0;
    a.n_seg = 0;
    for (int i = 0; i < rows.n_seg; ++i) {
      const KvSeg& s = rows.seg[i];
      const int64_t n = (int64_t)s.n_tok * c->G;
      if ((n <= kFewRows ? 0 : (n <= kStreamRows ? 1 : 2)) != kind) continue;
      a.seg[a.n_seg++] = AttendSeg{s.row0, s.n_tok, s.pos0, s.sess, 0, 0};
      most = std::max(most, n);
    }
    if (!a.n_seg) continue;
    CUDA_TRY(c, kind == 0 ? launch_attend_few(L, a, c->n_sm, most <= 8 ? 8 : 16)
                          : (kind == 1 ? launch_attend_stream(L, a, c->n_sm) : launch_attend_tc(L, a, c->n_sm)));
  }
  return MAG_OK;
}

}  // namespace mag

extern "C" {

mag_status mag_session_extend(mag_ctx* c, int32_t n, const int32_t* sids, const int32_t* ntok) {
  if (!c) return MAG_ERR_INVALID_ARG;
  if (n < 1 || n > MAG_MAX_BATCH)
    return fail(c, MAG_ERR_INVALID_ARG, "session_extend: %d sessions not in 1..%d", n, MAG_MAX_BATCH);
  if (!sids || !ntok) return fail(c, MAG_ERR_INVALID_ARG, "session_extend: null session or token list");
  int64_t need = 0;
  for (int i = 0; i < n; ++i) {
    const int sid = sids[i];
    if (sid < 0 || sid >= (int)c->sessions.size() || !c->sessions[sid].open)
      return fail(c, MAG_ERR_INVALID_ARG, "session_extend: session %d is not open", sid);
    for (int j = 0; j < i; ++j)
      if (sids[j] == sid) return fail(c, MAG_ERR_INVALID_ARG, "session_extend: session %d appears twice", sid);
    const Session& s = c->sessions[sid];
    if (ntok[i] < 0) return fail(c, MAG_ERR_INVALID_ARG, "session_extend: %d tokens", ntok[i]);
    if ((int64_t)s.len + ntok[i] > c->cfg.max_context)
      return fail(c, MAG_ERR_CONTEXT_FULL, "session_extend: %d + %d tokens exceed max_context %d", s.len, ntok[i],
                  c->cfg.max_context);
    need += (s.len + ntok[i] + 15) / 16 - (s.len + 15) / 16;
  }
  const mag_status dv = op_device(c, "session_extend");
  if (dv != MAG_OK) return dv;
  const mag_status cap = op_not_captured(c, "session_extend", "a replay would not extend the sessions");
  if (cap != MAG_OK) return cap;
  const mag_status st = reserve_blocks(c, "session_extend", need);
  if (st != MAG_OK) return st;
  for (int i = 0; i < n; ++i) {
    Session& s = c->sessions[sids[i]];
    const int nb_old = (s.len + 15) / 16, nb_new = (s.len + ntok[i] + 15) / 16;
    for (int b = nb_old; b < nb_new; ++b) s.table.push_back(c->kv.pop());
    if (nb_new > nb_old)
      CUDA_TRY(c, cudaMemcpyAsync(c->d_tables + (size_t)sids[i] * c->table_stride + nb_old, s.table.data() + nb_old,
                                  (size_t)(nb_new - nb_old) * 4, cudaMemcpyHostToDevice, c->stream));
    s.len += ntok[i];
  }
  return MAG_OK;
}

mag_status mag_kv_write(mag_ctx* c, int32_t layer, int32_t n, const int32_t* sids, const int32_t* ntok, const void* k,
                        const void* v, int64_t ld) {
  if (!c) return MAG_ERR_INVALID_ARG;
  KvWriteArgs a = {};
  mag_status st = op_rows(c, "kv_write", layer, n, sids, ntok, a.rows);
  if (st != MAG_OK || a.rows.n_rows == 0) return st;
  if ((st = op_buffer(c, "kv_write", "k", k, ld, (int64_t)c->Hkv * c->d)) != MAG_OK) return st;
  if ((st = op_buffer(c, "kv_write", "v", v, ld, (int64_t)c->Hkv * c->d)) != MAG_OK) return st;
  if ((st = op_device(c, "kv_write")) != MAG_OK) return st;
  a.k = (const __half*)k;
  a.v = (const __half*)v;
  a.ld = ld;
  a.layer = layer;
  a.pool = pool_geom(c);
  a.err = c->d_err;
  CUDA_TRY(c, launch_kv_write(Launch{c->stream, false, nullptr}, a));
  return MAG_OK;
}

mag_status mag_kv_read(mag_ctx* c, int32_t layer, int32_t n, const int32_t* sids, const int32_t* ntok, void* k, void* v,
                       int64_t ld) {
  if (!c) return MAG_ERR_INVALID_ARG;
  KvReadArgs a = {};
  mag_status st = op_rows(c, "kv_read", layer, n, sids, ntok, a.rows);
  if (st != MAG_OK || a.rows.n_rows == 0) return st;
  if ((st = op_buffer(c, "kv_read", "k", k, ld, (int64_t)c->Hkv * c->d)) != MAG_OK) return st;
  if ((st = op_buffer(c, "kv_read", "v", v, ld, (int64_t)c->Hkv * c->d)) != MAG_OK) return st;
  if ((st = op_device(c, "kv_read")) != MAG_OK) return st;
  a.k = (__half*)k;
  a.v = (__half*)v;
  a.ld = ld;
  a.layer = layer;
  a.n_blocks = read_blocks(a.rows, a.blk0);
  a.pool = pool_geom(c);
  a.err = c->d_err;
  CUDA_TRY(c, launch_kv_read(Launch{c->stream, false, nullptr}, a, 1));
  return MAG_OK;
}

mag_status mag_kv_export(mag_ctx* c, int32_t sid, int32_t first, int32_t n, void* k, void* v) {
  if (!c) return MAG_ERR_INVALID_ARG;
  if (sid < 0 || sid >= (int)c->sessions.size() || !c->sessions[sid].open)
    return fail(c, MAG_ERR_INVALID_ARG, "kv_export: session %d is not open", sid);
  const int len = c->sessions[sid].len;
  if (first < 0 || n < 0 || (int64_t)first + n > len)
    return fail(c, MAG_ERR_INVALID_ARG, "kv_export: tokens %d .. + %d of a session that holds %d", first, n, len);
  if (n == 0) return MAG_OK;
  const int64_t ld = (int64_t)c->Hkv * c->d;
  mag_status st = op_buffer(c, "kv_export", "k", k, ld, ld);
  if (st == MAG_OK) st = op_buffer(c, "kv_export", "v", v, ld, ld);
  if (st == MAG_OK) st = op_device(c, "kv_export");
  if (st != MAG_OK) return st;
  KvReadArgs a = {};
  a.rows.n_seg = 1;
  a.rows.n_rows = n;
  a.rows.seg[0] = KvSeg{0, n, first, sid};
  a.k = (__half*)k;
  a.v = (__half*)v;
  a.ld = ld;
  a.layer_stride = n * ld;
  a.n_blocks = read_blocks(a.rows, a.blk0);
  a.pool = pool_geom(c);
  a.err = c->d_err;
  CUDA_TRY(c, launch_kv_read(Launch{c->stream, false, nullptr}, a, c->L));
  return MAG_OK;
}

mag_status mag_attend(mag_ctx* c, int32_t layer, int32_t n, const int32_t* sids, const int32_t* ntok, const void* q,
                      int64_t ldq, void* out, int64_t ldo, int32_t window, float scale) {
  if (!c) return MAG_ERR_INVALID_ARG;
  KvRows rows;
  mag_status st = op_rows(c, "attend", layer, n, sids, ntok, rows);
  if (st != MAG_OK) return st;
  if (window < 0) return fail(c, MAG_ERR_INVALID_ARG, "attend: window %d", window);
  if (!std::isfinite(scale * kLog2e))
    return fail(c, MAG_ERR_INVALID_ARG, "attend: the scale, or its log2(e)-fold, is not finite");
  if (rows.n_rows == 0) return MAG_OK;
  if ((st = op_buffer(c, "attend", "q", q, ldq, (int64_t)c->Hq * c->d)) != MAG_OK) return st;
  if ((st = op_buffer(c, "attend", "out", out, ldo, (int64_t)c->Hq * c->d)) != MAG_OK) return st;
  if ((st = op_device(c, "attend")) != MAG_OK) return st;
  return run_attend(c, layer, rows, q, ldq, out, ldo, window, scale);
}

mag_status mag_sample(const void* logits, int32_t type, int32_t rows, int32_t vocab, int64_t ld,
                      const mag_sample_params* p, const float* uniform, int32_t* token, float* prob, void* stream) {
  if (rows < 0 || vocab < 1 || ld < vocab || (type != MAG_LOGITS_F16 && type != MAG_LOGITS_F32))
    return MAG_ERR_INVALID_ARG;
  const bool f32 = type == MAG_LOGITS_F32;
  if (vocab > sample_max_vocab(f32)) return MAG_ERR_UNSUPPORTED;
  if (rows == 0) return MAG_OK;
  const uintptr_t at = reinterpret_cast<uintptr_t>(logits);
  if (!logits || !uniform || !token || at % (f32 ? 4 : 2)) return MAG_ERR_INVALID_ARG;
  const void* words[] = {uniform, token, prob, p ? p->temperature : nullptr, p ? (const void*)p->top_k : nullptr,
                         p ? p->top_p : nullptr, p ? p->min_p : nullptr, p ? (const void*)p->allowed : nullptr};
  for (const void* w : words)
    if (reinterpret_cast<uintptr_t>(w) % 4) return MAG_ERR_INVALID_ARG;
  SampleArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.rows = rows;
  a.vocab = vocab;
  a.f32 = f32;
  if (p) {
    a.temperature = p->temperature;
    a.top_k = p->top_k;
    a.top_p = p->top_p;
    a.min_p = p->min_p;
    a.allowed = p->allowed;
  }
  a.uniform = uniform;
  a.token = token;
  a.prob = prob;
  return launch_sample((cudaStream_t)stream, a) == cudaSuccess ? MAG_OK : MAG_ERR_CUDA;
}

}  // extern "C"
