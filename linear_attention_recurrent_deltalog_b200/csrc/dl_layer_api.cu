// dl_layer_api.cu -- C ABI of the operators around the recurrent step
// (declared in deltalog.h): argument checks on the host, then the launch.

#include <cuda_runtime.h>

#include <cstdint>

#include "deltalog.h"
#include "dl_layer.cuh"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool dtype_ok(int t) { return t == DL_F32 || t == DL_BF16; }
size_t elem(int t) { return t == DL_BF16 ? 2 : (t == DL_F32 ? 4 : 1); }

// Rows of a batch or tile behind the last one still have int32 numbers: the
// largest step is a convolution's tile of 128 rows at most.
constexpr int32_t kMaxRows = 0x7fffffff - 1023;

// starts[0..n]: non-decreasing, 0 .. kMaxRows.
int check_starts(int32_t n, const int32_t* starts) {
  if (n < 0 || starts == nullptr) return DL_ERR_ARG;
  if (starts[0] < 0) return DL_ERR_ARG;
  for (int32_t s = 0; s < n; ++s)
    if (starts[s + 1] < starts[s]) return DL_ERR_ARG;
  if (starts[n] > kMaxRows) return DL_ERR_ARG;
  return DL_OK;
}

// Without rows (every sequence empty) x and y may be null.
int check_conv(const dl_conv_config* c, bool rows, const void* x, int64_t ldx, const float* w,
               const float* bias, const void* h0, const void* h1, const void* y, int64_t ldy) {
  if (c == nullptr || c->C < 1 || c->W < 1 || !dtype_ok(c->in_dtype)) return DL_ERR_ARG;
  if ((c->flags & ~int32_t(DL_CONV_SILU)) != 0) return DL_ERR_ARG;
  if (c->W < 2 || c->W > 4) return DL_ERR_UNSUPPORTED;
  if (!w || (rows && (!x || !y || x == y))) return DL_ERR_ARG;
  if (ldx < c->C || ldy < c->C) return DL_ERR_ARG;
  if (h1 != nullptr && (h1 == x || h1 == y)) return DL_ERR_ARG;
  const size_t e = elem(c->in_dtype);
  if (!aligned(x, e) || !aligned(y, e) || !aligned(w, 4) || !aligned(bias, 4) || !aligned(h0, e) ||
      !aligned(h1, e))
    return DL_ERR_ALIGN;
  return DL_OK;
}

// Whether four channels at a time can be read and written: rows, states and
// C in units of four elements, taps and bias 16-byte aligned.
bool conv_wide(const dl_conv_config& c, const dl::ConvParams& p) {
  const size_t a = 4 * elem(c.in_dtype);
  return aligned(p.x, a) && aligned(p.y, a) && aligned(p.h0, a) && aligned(p.h1, a) &&
         aligned(p.w, 16) && aligned(p.bias, 16) && p.ldx % 4 == 0 && p.ldy % 4 == 0 && c.C % 4 == 0;
}

dl::ConvParams conv_params(const dl_conv_config& c, const void* x, int64_t ldx, const float* w,
                           const float* bias, const void* h0, void* h1, void* y, int64_t ldy) {
  dl::ConvParams p{};
  p.x = x;
  p.w = w;
  p.bias = bias;
  p.h0 = h0;
  p.h1 = h1;
  p.y = y;
  p.ldx = ldx;
  p.ldy = ldy;
  p.C = c.C;
  p.silu = (c.flags & DL_CONV_SILU) ? 1 : 0;
  return p;
}

int check_ssm(const dl_ssm_config* c) {
  if (c == nullptr || c->H < 1 || c->G < 1 || c->H % c->G != 0 || !dtype_ok(c->in_dtype))
    return DL_ERR_ARG;
  if (c->d_k < 1 || c->d_v < 1 || (c->flags & ~int32_t(DL_SSM_SOFTPLUS)) != 0) return DL_ERR_ARG;
  if ((c->d_k != 64 && c->d_k != 128) || (c->d_v != 64 && c->d_v != 128)) return DL_ERR_UNSUPPORTED;
  if (int64_t(c->H) * c->d_v > 0x7fffffff || int64_t(c->G) * c->d_k > 0x7fffffff) return DL_ERR_ARG;
  return DL_OK;
}

// Without rows (every sequence empty) their buffers may be null.
int check_ssm_io(const dl_ssm_config& c, bool rows, const dl_ssm_io* io) {
  if (io == nullptr || !io->a) return DL_ERR_ARG;
  if (rows) {
    if (!io->q || !io->k || !io->v || !io->dt || !io->o) return DL_ERR_ARG;
    if (io->o == io->q || io->o == io->k || io->o == io->v) return DL_ERR_ARG;
  }
  const int64_t nk = int64_t(c.G) * c.d_k, nv = int64_t(c.H) * c.d_v;
  if (io->ldq < nk || io->ldk < nk || io->ldv < nv || io->ldo < nv || io->lddt < c.H)
    return DL_ERR_ARG;
  const int64_t per16 = 16 / int64_t(elem(c.in_dtype));
  if (io->ldq % per16 || io->ldk % per16 || io->ldv % per16 || io->ldo % per16) return DL_ERR_ALIGN;
  if (!aligned(io->q, 16) || !aligned(io->k, 16) || !aligned(io->v, 16) || !aligned(io->o, 16))
    return DL_ERR_ALIGN;
  if (!aligned(io->dt, 4) || !aligned(io->a, 4) || !aligned(io->d, 4) || !aligned(io->dt_bias, 4))
    return DL_ERR_ALIGN;
  return DL_OK;
}

dl::SsmParams ssm_params(const dl_ssm_config& c, const dl_ssm_io& io, const float* S0, float* S1) {
  dl::SsmParams p{};
  p.q = io.q;
  p.k = io.k;
  p.v = io.v;
  p.dt = io.dt;
  p.a = io.a;
  p.d = io.d;
  p.bias = io.dt_bias;
  p.S0 = S0;
  p.S1 = S1;
  p.o = io.o;
  p.ldq = io.ldq;
  p.ldk = io.ldk;
  p.ldv = io.ldv;
  p.lddt = io.lddt;
  p.ldo = io.ldo;
  p.H = c.H;
  p.G = c.G;
  p.softplus = (c.flags & DL_SSM_SOFTPLUS) ? 1 : 0;
  return p;
}

// SMs the plan of a prompt call reckons with.  Without a device (sizes asked
// for on the host alone) a B200's.
int plan_sms() {
  const int n = dl::sm_count();
  return n > 0 ? n : 148;
}

dl::SsmPlan ssm_plan(const dl_ssm_config& c, int32_t n, const int32_t* starts) {
  if (c.in_dtype == DL_BF16 && starts[n] > starts[0])
    return dl::plan_ssm(c.H, c.G, c.d_k, c.d_v, n, starts, plan_sms());
  return dl::plan_ssm_scan(c.H, c.d_k, c.d_v, n, starts, plan_sms());
}

int status(cudaError_t e) { return e == cudaSuccess ? DL_OK : DL_ERR_CUDA; }

}  // namespace

extern "C" {

int dl_conv_prompt(const dl_conv_config* cfg, int32_t n, const int32_t* starts, const void* x,
                   int64_t ldx, const float* w, const float* bias, const void* h0, void* h1,
                   void* y, int64_t ldy, void* stream) {
  int rc = check_starts(n, starts);
  if (rc != DL_OK) return rc;
  rc = check_conv(cfg, starts[n] > starts[0], x, ldx, w, bias, h0, h1, y, ldy);
  if (rc != DL_OK) return rc;
  if (n == 0) return DL_OK;
  const dl::ConvParams p = conv_params(*cfg, x, ldx, w, bias, h0, h1, y, ldy);
  return status(dl::launch_conv_prompt(p, n, starts, cfg->W, cfg->in_dtype == DL_BF16,
                                       conv_wide(*cfg, p), static_cast<cudaStream_t>(stream)));
}

int dl_conv_step(const dl_conv_config* cfg, int32_t B, const void* x, int64_t ldx, const float* w,
                 const float* bias, void* h, void* y, int64_t ldy, void* stream) {
  const int rc = check_conv(cfg, B > 0, x, ldx, w, bias, h, h, y, ldy);
  if (rc != DL_OK) return rc;
  if (B < 0 || B > kMaxRows || (B > 0 && h == nullptr)) return DL_ERR_ARG;
  if (B == 0) return DL_OK;
  const dl::ConvParams p = conv_params(*cfg, x, ldx, w, bias, h, h, y, ldy);
  return status(dl::launch_conv_step(p, B, cfg->W, cfg->in_dtype == DL_BF16, conv_wide(*cfg, p),
                                     static_cast<cudaStream_t>(stream)));
}

int dl_ssm_bytes(const dl_ssm_config* cfg, int32_t n, const int32_t* starts, size_t* bytes) {
  int rc = check_ssm(cfg);
  if (rc != DL_OK) return rc;
  if (bytes == nullptr) return DL_ERR_ARG;
  rc = check_starts(n, starts);
  if (rc != DL_OK) return rc;
  *bytes = ssm_plan(*cfg, n, starts).bytes;
  return DL_OK;
}

int dl_ssm_prompt(const dl_ssm_config* cfg, int32_t n, const int32_t* starts, const dl_ssm_io* io,
                  const float* S0, float* S1, void* workspace, size_t workspace_bytes,
                  void* stream) {
  int rc = check_ssm(cfg);
  if (rc != DL_OK) return rc;
  rc = check_starts(n, starts);
  if (rc != DL_OK) return rc;
  const bool rows = starts[n] > starts[0];
  rc = check_ssm_io(*cfg, rows, io);
  if (rc != DL_OK) return rc;
  if (!aligned(S0, 16) || !aligned(S1, 16)) return DL_ERR_ALIGN;
  if (int64_t(n) * cfg->H > 0x7fffffff) return DL_ERR_ARG;
  const dl::SsmPlan plan = ssm_plan(*cfg, n, starts);
  if (plan.bytes > 0 && (workspace == nullptr || workspace_bytes < plan.bytes)) return DL_ERR_ARG;
  if (!aligned(workspace, 256)) return DL_ERR_ALIGN;
  if (n == 0) return DL_OK;
  dl::SsmParams p = ssm_params(*cfg, *io, S0, S1);
  if (cfg->in_dtype == DL_BF16 && rows) {
    p.err = dl::shared_err_word();
    if (p.err == nullptr) return DL_ERR_CUDA;
    return status(dl::launch_ssm_chunked(p, n, starts, cfg->d_k, cfg->d_v, plan, workspace,
                                         static_cast<cudaStream_t>(stream)));
  }
  return status(dl::launch_ssm_scan(p, n, starts, cfg->d_k, cfg->d_v, plan, workspace,
                                    static_cast<cudaStream_t>(stream)));
}

int dl_ssm_step(const dl_ssm_config* cfg, int32_t B, const dl_ssm_io* io, float* S, void* stream) {
  int rc = check_ssm(cfg);
  if (rc != DL_OK) return rc;
  rc = check_ssm_io(*cfg, B > 0, io);
  if (rc != DL_OK) return rc;
  if (B < 0 || (B > 0 && S == nullptr) || int64_t(B) * cfg->H > 0x7fffffff) return DL_ERR_ARG;
  if (!aligned(S, 16)) return DL_ERR_ALIGN;
  if (B == 0) return DL_OK;
  const dl::SsmParams p = ssm_params(*cfg, *io, S, S);
  return status(dl::launch_ssm_step(p, B, cfg->d_k, cfg->d_v, cfg->in_dtype == DL_BF16,
                                    static_cast<cudaStream_t>(stream)));
}

int dl_norm(const dl_norm_config* cfg, int64_t rows, const void* x, int64_t ldx, const void* res,
            int64_t ldr, const float* w, void* res_out, int64_t ldro, void* out, int64_t ldo,
            float* scales, void* stream) {
  if (cfg == nullptr || cfg->D < 1 || !dtype_ok(cfg->in_dtype)) return DL_ERR_ARG;
  const bool q = cfg->out_dtype == DL_E4M3;
  if (!q && !dtype_ok(cfg->out_dtype)) return DL_ERR_ARG;
  if (cfg->block != 0 && !(q && cfg->block == 128)) return DL_ERR_ARG;
  if (!(cfg->eps >= 0.f)) return DL_ERR_ARG;
  if (cfg->D > 16384) return DL_ERR_UNSUPPORTED;
  if (rows == 0) return DL_OK;
  if (rows < 0 || !x || !w || !out || (q && scales == nullptr)) return DL_ERR_ARG;
  if (ldx < cfg->D || ldo < cfg->D || (res && ldr < cfg->D) || (res_out && ldro < cfg->D))
    return DL_ERR_ARG;
  if (out == x || out == res || out == res_out) return DL_ERR_ARG;
  // in place only row by row
  if ((res_out && res_out == x && ldro != ldx) || (res_out && res_out == res && ldro != ldr))
    return DL_ERR_ARG;
  const size_t e = elem(cfg->in_dtype), eo = elem(cfg->out_dtype);
  if (!aligned(x, e) || !aligned(res, e) || !aligned(res_out, e) || !aligned(w, 4) ||
      !aligned(out, eo) || !aligned(scales, 4))
    return DL_ERR_ALIGN;
  dl::NormParams p{};
  p.x = x;
  p.res = res;
  p.w = w;
  p.res_out = res_out;
  p.out = out;
  p.scales = q ? scales : nullptr;
  p.rows = rows;
  p.ldx = ldx;
  p.ldr = ldr;
  p.ldro = ldro;
  p.ldo = ldo;
  p.D = cfg->D;
  p.block = cfg->block;
  p.eps = cfg->eps;
  // 8 channels at a time: 16-byte rows of x, res and res_out (32 bytes of
  // fp32), and 8, 16 or 32 bytes of the output
  const size_t ao = q ? 8 : 16;
  const bool vec = cfg->D % 8 == 0 && aligned(x, 16) && aligned(res, 16) && aligned(res_out, 16) &&
                   aligned(w, 16) && aligned(out, ao) && (size_t(ldx) * e) % 16 == 0 &&
                   (!res || (size_t(ldr) * e) % 16 == 0) &&
                   (!res_out || (size_t(ldro) * e) % 16 == 0) && (size_t(ldo) * eo) % ao == 0;
  return status(dl::launch_norm(p, cfg->in_dtype == DL_BF16,
                                q ? dl::kOutE4M3 : (cfg->out_dtype == DL_BF16 ? dl::kOutBF16 : dl::kOutF32),
                                vec, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
