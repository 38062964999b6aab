// The selective scan's entry points (atlas_scan.h).  The work is the decay
// attention's, with gates (decay_common.cuh; atlas_decay.cu and its kernels).
#include "../../include/atlas_scan.h"

#include <math.h>

#include <new>

#include "decay_tc.cuh"

using namespace layer;

struct atlas_scan_handle : HandleBase {
  atlas_scan_config cfg;
  int path = -1;
  // its part that the decay attention has as well
  atlas_decay_config common() const {
    return atlas_decay_config{cfg.H, cfg.d_k, cfg.d_v, cfg.share, cfg.qkv_dtype, cfg.y_dtype, cfg.qkv_layout, cfg.y_layout, cfg.scale};
  }
};

static thread_local std::string g_create_err;

extern "C" int atlas_scan_create(const atlas_scan_config* cfg, atlas_scan_handle** out) {
  if (!out || !cfg) {
    g_create_err = "cfg and out must be non-NULL";
    if (out) *out = nullptr;
    return ATLAS_ERR_INVALID_ARG;
  }
  *out = nullptr;
  const atlas_scan_config& c = *cfg;
  auto bad = [&](int code, const char* why) {
    g_create_err = why;
    return code;
  };
  if (c.H < 1 || c.d_k < 1 || c.d_v < 1) return bad(ATLAS_ERR_INVALID_ARG, "H, d_k, d_v must be >= 1");
  if (c.share < 1 || c.H % c.share) return bad(ATLAS_ERR_INVALID_ARG, "share must divide H");
  if (c.gates != ATLAS_GATES_MEMORY && c.gates != ATLAS_GATES_STEP)
    return bad(ATLAS_ERR_INVALID_ARG, "gates must be ATLAS_GATES_MEMORY or ATLAS_GATES_STEP");
  if (!dtype_ok(c.qkv_dtype) || !dtype_ok(c.y_dtype))
    return bad(ATLAS_ERR_INVALID_ARG, "qkv_dtype and y_dtype must be ATLAS_F32 or ATLAS_BF16");
  auto layout_ok = [](int l) { return l == ATLAS_LAYOUT_HEADS || l == ATLAS_LAYOUT_TOKENS; };
  if (!layout_ok(c.qkv_layout) || !layout_ok(c.y_layout))
    return bad(ATLAS_ERR_INVALID_ARG, "qkv_layout and y_layout must be ATLAS_LAYOUT_HEADS or ATLAS_LAYOUT_TOKENS");
  if (!isfinite(c.scale)) return bad(ATLAS_ERR_INVALID_ARG, "scale must be finite");
  if (c.d_k > 256 || c.d_v > 1024) return bad(ATLAS_ERR_UNSUPPORTED, "d_k > 256 or d_v > 1024 is not supported");
  if (c.H > 65535) return bad(ATLAS_ERR_UNSUPPORTED, "H > 65535 is not supported");
  auto* h = new (std::nothrow) atlas_scan_handle();
  if (!h) return bad(ATLAS_ERR_OOM, "out of host memory");
  h->cfg = c;
  *out = h;
  return ATLAS_OK;
}

extern "C" size_t atlas_scan_workspace_bytes(const atlas_scan_handle* h, int B, int T) {
  return h ? decay::workspace_bytes(h->common(), B, T, true) : 0;
}

extern "C" int atlas_scan_forward(atlas_scan_handle* h, const atlas_scan_io* io, void* stream) {
  if (!h) return ATLAS_ERR_INVALID_ARG;
  if (!io) return h->fail(ATLAS_ERR_INVALID_ARG, "io must be non-NULL");
  const atlas_scan_config& c = h->cfg;
  if (io->B < 1 || io->T < 1) return h->fail(ATLAS_ERR_INVALID_ARG, "B and T must be >= 1");
  if (!io->q || !io->k || !io->v || !io->step || !io->y)
    return h->fail(ATLAS_ERR_INVALID_ARG, "q, k, v, step, y must be non-NULL");
  const bool memory = c.gates == ATLAS_GATES_MEMORY, tokens = c.qkv_layout == ATLAS_LAYOUT_TOKENS;
  if (memory ? !io->alpha || io->A || io->dt_bias : io->alpha || !io->A)
    return h->fail(ATLAS_ERR_INVALID_ARG, "ATLAS_GATES_MEMORY takes alpha, ATLAS_GATES_STEP A and dt_bias");
  const long long Hq = c.H / c.share, qk = Hq * c.d_k, vw = (long long)c.H * c.d_v;
  if ((io->ld_qk || io->ld_v || io->ld_gates) &&
      (!tokens || (io->ld_qk && io->ld_qk < qk) || (io->ld_v && io->ld_v < vw) || (io->ld_gates && io->ld_gates < c.H)))
    return h->fail(ATLAS_ERR_INVALID_ARG,
                   "ld_qk, ld_v and ld_gates are of ATLAS_LAYOUT_TOKENS, and at least a token's values");
  if (io->T > decay::kMostTokens) return h->fail(ATLAS_ERR_UNSUPPORTED, "T > 2^30 is not supported");
  const size_t rows = (size_t)io->B * io->T, es = dtype_size(c.qkv_dtype);
  const size_t ld_qk = io->ld_qk ? io->ld_qk : qk, ld_v = io->ld_v ? io->ld_v : vw, ld_g = io->ld_gates ? io->ld_gates : c.H;
  if ((double)rows * (double)(ld_qk > ld_v ? ld_qk : ld_v) > 1e17) return h->fail(ATLAS_ERR_UNSUPPORTED, "B * T rows are too large");
  const size_t yb = rows * vw * dtype_size(c.y_dtype), qb = ((rows - 1) * ld_qk + qk) * es, vb = ((rows - 1) * ld_v + vw) * es,
               gb = ((rows - 1) * ld_g + c.H) * 4, sb = (size_t)io->B * c.H * c.d_k * c.d_v * 4, hb = (size_t)c.H * 4;
  auto clash = [&](const void* p, size_t n, bool own_state) {
    return overlap(p, n, io->q, qb) || overlap(p, n, io->k, qb) || overlap(p, n, io->v, vb) || overlap(p, n, io->step, gb) ||
           overlap(p, n, io->alpha, gb) || overlap(p, n, io->A, hb) || overlap(p, n, io->dt_bias, hb) || overlap(p, n, io->D, hb) ||
           (!own_state && overlap(p, n, io->S0, sb));
  };
  if (clash(io->y, yb, false)) return h->fail(ATLAS_ERR_INVALID_ARG, "y must not overlap an input");
  if (clash(io->S_out, sb, io->S_out == io->S0) || overlap(io->S_out, sb, io->y, yb))
    return h->fail(ATLAS_ERR_INVALID_ARG, "S_out may be S0 itself, else it must not overlap another tensor");
  atlas_decay_io common{};
  common.B = io->B, common.T = io->T, common.q = io->q, common.k = io->k, common.v = io->v, common.lens = io->lens;
  common.S0 = io->S0, common.y = io->y, common.S_out = io->S_out;
  decay::Selective x{};
  x.gates.step = io->step, x.gates.alpha = io->alpha, x.gates.A = io->A, x.gates.dt_bias = io->dt_bias;
  x.gates.b = tokens ? (size_t)io->T * ld_g : (size_t)c.H * io->T;
  x.gates.h = tokens ? 1 : (size_t)io->T;
  x.gates.t = tokens ? ld_g : 1;
  x.D = io->D;
  // (dense rows are the decay attention's case)
  x.ld_qk = io->ld_qk == qk && io->ld_v == vw ? 0 : io->ld_qk;
  x.ld_v = io->ld_qk == qk && io->ld_v == vw ? 0 : io->ld_v;
  return decay::run(h, h->common(), common, &x, (cudaStream_t)stream, &h->path);
}

extern "C" int atlas_scan_status(atlas_scan_handle* h) { return h ? h->read_status() : ATLAS_ERR_INVALID_ARG; }
extern "C" int atlas_scan_last_path(const atlas_scan_handle* h) { return h ? h->path : -1; }
extern "C" const char* atlas_scan_last_error(const atlas_scan_handle* h) {
  return h ? h->err.c_str() : g_create_err.c_str();
}
extern "C" void atlas_scan_destroy(atlas_scan_handle* h) { delete h; }
