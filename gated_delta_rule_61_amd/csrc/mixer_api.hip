// C ABI of the operators around the scans (causal convolution and its
// gradients, norm of the heads and its gradients, selective state-space scan and
// step, the delta rule's step with one gate per key channel, 8-bit state cache): argument validation (host
// only, before any HIP call) and the launch of each.

#include <stdint.h>

#include "gdn61.h"
#include "gdn_launch.h"
#include "mixer_launch.h"

namespace gdn {
namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

int known_dtype(int dtype) {
  if (dtype != GDN_DTYPE_F32 && dtype != GDN_DTYPE_BF16)
    return fail(GDN_ERR_INVALID_ARGUMENT, "unknown dtype code %d", dtype);
  return GDN_OK;
}

// sequences of a call and the number of its tokens
int check_seqs(const int64_t* cu, int num_seqs, int B, int T, int& N) {
  if (B < 0 || T < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "sizes must be positive (B, T >= 0): B=%d T=%d", B, T);
  if ((long long)B * T >= (1LL << 25))
    return fail(GDN_ERR_UNSUPPORTED, "B*T too large (got %lld tokens)", (long long)B * T);
  N = B;
  if (cu) {
    if (B != 1) return fail(GDN_ERR_INVALID_ARGUMENT, "cu_seqlens requires B == 1 (got B=%d)", B);
    if (num_seqs < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "num_seqs must be >= 0 (got %d)", num_seqs);
    N = num_seqs;
  }
  return GDN_OK;
}

// Strides of a row operand: not negative, and multiples of `unit` elements
// where the kernels read 16-byte vectors (rows that are not visited have none).
int check_rows(const char* name, const Rows& r, int B, int T, int unit) {
  const long long lim = 1LL << 40;
  const bool tok = T > 1, bat = B > 1;
  if ((tok && (r.token < 0 || r.token >= lim)) || (bat && (r.batch < 0 || r.batch >= lim)))
    return fail(GDN_ERR_INVALID_ARGUMENT, "%s: strides must lie in [0, 2^40) (got %lld, %lld)", name, r.batch,
                    r.token);
  if ((tok && r.token % unit) || (bat && r.batch % unit))
    return fail(GDN_ERR_UNSUPPORTED, "%s: strides must be multiples of %d elements (got %lld, %lld)", name, unit,
                    r.batch, r.token);
  if (unit > 1 && !aligned16(r.p))
    return fail(GDN_ERR_INVALID_ARGUMENT, "%s must be 16-byte aligned", name);
  return GDN_OK;
}

int check_conv(ConvArgs& a, int width0, int width1, int width2, int dtype) {
  if (int st = known_dtype(dtype)) return st;
  a.bf16 = dtype == GDN_DTYPE_BF16;
  if (a.D <= 0) return fail(GDN_ERR_INVALID_ARGUMENT, "D must be positive (got %d)", a.D);
  if (a.W < 2 || a.W > 4) return fail(GDN_ERR_UNSUPPORTED, "the convolution takes W = 2..4 taps (got %d)", a.W);
  if (width0 <= 0 || width1 < 0 || width2 < 0 || (width1 == 0 && width2 > 0) ||
      (long long)width0 + width1 + width2 != a.D)
    return fail(GDN_ERR_INVALID_ARGUMENT, "section widths %d, %d, %d must add up to D = %d", width0, width1, width2,
                    a.D);
  if (width0 % 8 || width1 % 8 || width2 % 8)
    return fail(GDN_ERR_UNSUPPORTED, "section widths must be multiples of 8 (got %d, %d, %d)", width0, width1,
                    width2);
  a.end[0] = width0;
  a.end[1] = width0 + width1;
  a.end[2] = a.D;
  if (a.silu != 0 && a.silu != 1) return fail(GDN_ERR_INVALID_ARGUMENT, "silu must be 0 or 1 (got %d)", a.silu);
  if (a.norm_sections < 0 || a.norm_sections > 3)
    return fail(GDN_ERR_INVALID_ARGUMENT, "norm_sections must be 0..3 (got %d)", a.norm_sections);
  if (a.norm_sections > 0) {
    if (a.norm_dim != 64 && a.norm_dim != 128)
      return fail(GDN_ERR_UNSUPPORTED, "norm_dim must be 64 or 128 (got %d)", a.norm_dim);
    const int widths[3] = {width0, width1, width2};
    for (int i = 0; i < a.norm_sections; ++i)
      if (widths[i] % a.norm_dim)
        return fail(GDN_ERR_INVALID_ARGUMENT, "norm_dim (%d) must divide the width of section %d (%d)", a.norm_dim,
                        i, widths[i]);
    if (!(a.eps >= 0.f)) return fail(GDN_ERR_INVALID_ARGUMENT, "norm_eps must be >= 0");
  }
  if (a.pool < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "pool must be >= 0 (got %d)", a.pool);
  return GDN_OK;
}

// pointers of a convolution that has work to do
int check_conv_ptrs(const ConvArgs& a, bool tokens) {
  if (!a.weight || (tokens && !a.x.p)) return fail(GDN_ERR_INVALID_ARGUMENT, "x and weight are required");
  for (int i = 0; i < 3; ++i) {
    const bool used = i == 0 || a.end[i] > a.end[i - 1];
    if (used && tokens && !a.out[i]) return fail(GDN_ERR_INVALID_ARGUMENT, "out%d is required", i);
  }
  const void* ptrs[] = {a.weight, a.bias, a.state, a.out[0], a.out[1], a.out[2]};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return fail(GDN_ERR_INVALID_ARGUMENT, "tensor pointers must be 16-byte aligned");
  return GDN_OK;
}

int check_ssm(SsmArgs& a, int dtype) {
  if (int st = known_dtype(dtype)) return st;
  a.bf16 = dtype == GDN_DTYPE_BF16;
  if (a.Hk <= 0 || a.HV <= 0 || a.K <= 0 || a.V <= 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "sizes must be positive: Hk=%d HV=%d K=%d V=%d", a.Hk, a.HV, a.K, a.V);
  if (a.HV % a.Hk != 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "HV (%d) must be a multiple of Hk (%d)", a.HV, a.Hk);
  if ((a.K != 64 && a.K != 128) || (a.V != 64 && a.V != 128))
    return fail(GDN_ERR_UNSUPPORTED, "supported head dims are K, V in {64, 128} (got K=%d V=%d)", a.K, a.V);
  if (a.softplus != 0 && a.softplus != 1)
    return fail(GDN_ERR_INVALID_ARGUMENT, "dt_softplus must be 0 or 1 (got %d)", a.softplus);
  return GDN_OK;
}

int check_ssm_rows(const SsmArgs& a) {
  if (!a.x.p || !a.dt.p || !a.B.p || !a.C.p || !a.A_log || !a.y)
    return fail(GDN_ERR_INVALID_ARGUMENT, "x, dt, Bm, Cm, A_log and y are required");
  const int unit = a.bf16 ? 8 : 4;
  if (int st = check_rows("x", a.x, a.nb, a.T, unit)) return st;
  if (int st = check_rows("dt", a.dt, a.nb, a.T, 1)) return st;
  if (int st = check_rows("Bm", a.B, a.nb, a.T, unit)) return st;
  if (int st = check_rows("Cm", a.C, a.nb, a.T, unit)) return st;
  if (a.z.p)
    if (int st = check_rows("z", a.z, a.nb, a.T, unit)) return st;
  if (!aligned16(a.y)) return fail(GDN_ERR_INVALID_ARGUMENT, "y must be 16-byte aligned");
  // rows of a chunk are addressed with 32-bit byte offsets
  for (const Rows* r : {&a.x, &a.dt, &a.B, &a.C, &a.z})
    if (a.T > 1 && r->p && r->token >= (1 << 23))
      return fail(GDN_ERR_UNSUPPORTED, "token strides must stay below 2^23 elements");
  if ((long long)a.HV * a.V >= (1 << 23)) return fail(GDN_ERR_UNSUPPORTED, "HV * V must stay below 2^23");
  return GDN_OK;
}

int check_norm(GroupNormArgs& a, int weight_dtype, int dtype) {
  if (int st = known_dtype(dtype)) return st;
  a.bf16 = dtype == GDN_DTYPE_BF16;
  if (a.B < 0 || a.T < 0 || a.G <= 0 || a.d <= 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "sizes must be positive (B, T >= 0): B=%d T=%d G=%d d=%d", a.B, a.T, a.G,
                a.d);
  if ((long long)a.B * a.T >= (1LL << 25))
    return fail(GDN_ERR_UNSUPPORTED, "B*T too large (got %lld tokens)", (long long)a.B * a.T);
  if (a.d % 8 || a.d > 8192)
    return fail(GDN_ERR_UNSUPPORTED, "groups take a multiple of 8 channels up to 8192 (got %d)", a.d);
  if ((long long)a.G * a.d >= (1 << 23)) return fail(GDN_ERR_UNSUPPORTED, "G * d must stay below 2^23");
  if (a.act < 0 || a.act > 2) return fail(GDN_ERR_INVALID_ARGUMENT, "unknown activation code %d", a.act);
  if (a.rms != 0 && a.rms != 1) return fail(GDN_ERR_INVALID_ARGUMENT, "rms must be 0 or 1 (got %d)", a.rms);
  if (a.shared != 0 && a.shared != 1)
    return fail(GDN_ERR_INVALID_ARGUMENT, "weight_shared must be 0 or 1 (got %d)", a.shared);
  if (!(a.eps >= 0.f)) return fail(GDN_ERR_INVALID_ARGUMENT, "eps must be >= 0");
  if (weight_dtype != GDN_DTYPE_F32 && weight_dtype != GDN_DTYPE_BF16)
    return fail(GDN_ERR_INVALID_ARGUMENT, "unknown weight dtype code %d", weight_dtype);
  a.w_bf16 = weight_dtype == GDN_DTYPE_BF16;
  const void* ptrs[] = {a.weight, a.bias, a.y, a.dx, a.dz, a.dweight, a.dbias};
  for (const void* p : ptrs)
    if (!aligned16(p)) return fail(GDN_ERR_INVALID_ARGUMENT, "tensor pointers must be 16-byte aligned");
  return GDN_OK;
}

int check_workspace(const void* workspace, size_t have, size_t need) {
  if (need == 0) return GDN_OK;
  if (!workspace || have < need)
    return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need, workspace ? have : (size_t)0);
  if (((uintptr_t)workspace & 255u) != 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "workspace must be 256-byte aligned");
  return GDN_OK;
}

// A launch has fewer than 2^32 threads.
bool too_many(long long groups, int threads) { return groups >= (1LL << 32) / threads; }

int done(hipError_t e) {
  if (e != hipSuccess) return fail(GDN_ERR_LAUNCH, "HIP launch failed: %s", hipGetErrorString(e));
  return ok();
}

template <typename F>
int timed(int stage, void* stream, F&& launch) {
  prof_begin(stage, (hipStream_t)stream);
  const hipError_t e = launch((hipStream_t)stream);
  prof_end(stage, (hipStream_t)stream);
  return done(e);
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_conv_fwd(const void* x, long long x_batch, long long x_token, const void* weight, const void* bias,
                 int silu, void* out0, void* out1, void* out2, int width0, int width1, int width2,
                 int norm_dim, int norm_sections, float norm_eps, void* state, const int32_t* state_indices,
                 const int32_t* has_state, int pool, const int64_t* cu_seqlens, int num_seqs, int B, int T, int D,
                 int W, int dtype, void* stream) {
  ConvArgs a{};
  a.x = {x, x_batch, x_token};
  a.weight = weight; a.bias = bias; a.silu = silu;
  a.out[0] = out0; a.out[1] = out1; a.out[2] = out2;
  a.norm_dim = norm_dim; a.norm_sections = norm_sections; a.eps = norm_eps;
  a.state = state; a.idx = state_indices; a.has = has_state; a.pool = state ? pool : 0;
  a.cu = cu_seqlens; a.B = B; a.T = T; a.D = D; a.W = W;
  if (int st = check_seqs(cu_seqlens, num_seqs, B, T, a.N)) return st;
  if (int st = check_conv(a, width0, width1, width2, dtype)) return st;
  if (has_state && !state) return fail(GDN_ERR_INVALID_ARGUMENT, "has_state needs a state");
  if (state && !state_indices && pool < a.N)
    return fail(GDN_ERR_INVALID_ARGUMENT, "identity slots need pool >= N (pool=%d N=%d)", pool, a.N);
  const bool tokens = (long long)B * T > 0;
  if (a.N == 0 || (!tokens && !state)) return ok();
  if (int st = check_conv_ptrs(a, tokens)) return st;
  if (int st = check_rows("x", a.x, B, T, 8)) return st;
  if (too_many(((long long)B * T / 16 + 4096) * (D / 512 + 1), 64))   // runs of 16 tokens, or 4096 shorter ones
    return fail(GDN_ERR_UNSUPPORTED, "too many tokens x channels for one launch");
  return timed(GDN_STAGE_CONV, stream, [&](hipStream_t s) { return launch_conv_fwd(a, s); });
}

int gdn_conv_step(const void* x, long long x_batch, long long x_token, const void* weight, const void* bias,
                  int silu, void* out0, void* out1, void* out2, int width0, int width1, int width2,
                  void* state, const int32_t* state_indices, int pool, int B, int T, int D, int W, int dtype,
                  void* stream) {
  ConvArgs a{};
  a.x = {x, x_batch, x_token};
  a.weight = weight; a.bias = bias; a.silu = silu;
  a.out[0] = out0; a.out[1] = out1; a.out[2] = out2;
  a.state = state; a.idx = state_indices; a.pool = pool;
  a.B = B; a.T = T; a.D = D; a.W = W;
  if (B < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "B must be >= 0 (got %d)", B);
  if (T < 1 || T > 4) return fail(GDN_ERR_INVALID_ARGUMENT, "a step takes T = 1..4 tokens (got T=%d)", T);
  if (int st = check_seqs(nullptr, 0, B, T, a.N)) return st;
  if (int st = check_conv(a, width0, width1, width2, dtype)) return st;
  if (!state_indices && pool < B)
    return fail(GDN_ERR_INVALID_ARGUMENT, "identity slots need pool >= B (pool=%d B=%d)", pool, B);
  if (B == 0) return ok();
  if (!state) return fail(GDN_ERR_INVALID_ARGUMENT, "state is required");
  if (int st = check_conv_ptrs(a, true)) return st;
  if (int st = check_rows("x", a.x, B, T, 8)) return st;
  if (too_many((long long)B * (D / 512 + 1), 64))
    return fail(GDN_ERR_UNSUPPORTED, "too many rows x channels for one launch");
  return timed(GDN_STAGE_CONV, stream, [&](hipStream_t s) { return launch_conv_step(a, s); });
}

size_t gdn_conv_bwd_workspace_bytes(int B, int T, int D, int W) {
  if (B < 0 || T < 0 || D <= 0 || D % 8 || W < 2 || W > 4) return 0;
  ConvBwdArgs a{};
  a.B = B; a.T = T; a.D = D; a.W = W;
  a.dweight = &a;   // any: the size is the same for one of the sums and for both
  return conv_bwd_bytes(a);
}

int gdn_conv_bwd(const void* dout0, const void* dout1, const void* dout2, int width0, int width1, int width2,
                 const void* x, long long x_batch, long long x_token, const void* weight, const void* bias, int silu,
                 int norm_dim, int norm_sections, float norm_eps, const int64_t* cu_seqlens, int num_seqs, int B,
                 int T, int D, int W, int dtype, void* dx, void* dweight, void* dbias, void* workspace,
                 size_t workspace_bytes, void* stream) {
  const int zero_rows = dtype & GDN_ROWS_ZERO;
  dtype &= ~GDN_ROWS_ZERO;
  // the checks of the forward convolution, dout in the place of its outputs
  ConvArgs f{};
  f.x = {x, x_batch, x_token};
  f.weight = weight; f.bias = bias; f.silu = silu;
  f.out[0] = const_cast<void*>(dout0); f.out[1] = const_cast<void*>(dout1); f.out[2] = const_cast<void*>(dout2);
  f.norm_dim = norm_dim; f.norm_sections = norm_sections; f.eps = norm_eps;
  f.B = B; f.T = T; f.D = D; f.W = W;
  if (int st = check_seqs(cu_seqlens, num_seqs, B, T, f.N)) return st;
  if (int st = check_conv(f, width0, width1, width2, dtype)) return st;
  const bool tokens = (long long)B * T > 0;
  if (!tokens && !dweight && !dbias) return ok();
  if (int st = check_conv_ptrs(f, tokens)) return st;
  if (tokens && !dx) return fail(GDN_ERR_INVALID_ARGUMENT, "dx is required");
  if (!aligned16(dx) || !aligned16(dweight) || !aligned16(dbias))
    return fail(GDN_ERR_INVALID_ARGUMENT, "tensor pointers must be 16-byte aligned");
  if (int st = check_rows("x", f.x, B, T, 8)) return st;
  if (too_many(((long long)B * T / 8 + 2048) * (D / 512 + 1), 64))   // runs of 8 tokens, or 2048 shorter ones
    return fail(GDN_ERR_UNSUPPORTED, "too many tokens x channels for one launch");
  ConvBwdArgs a{};
  a.x = f.x; a.weight = weight; a.bias = bias;
  a.dout[0] = dout0; a.dout[1] = dout1; a.dout[2] = dout2;
  a.end[0] = f.end[0]; a.end[1] = f.end[1]; a.end[2] = f.end[2];
  a.norm_dim = norm_dim; a.norm_sections = norm_sections; a.eps = norm_eps; a.silu = silu;
  a.dx = dx; a.dweight = dweight; a.dbias = dbias;
  a.cu = cu_seqlens; a.zero_rows = zero_rows; a.N = f.N; a.B = B; a.T = T; a.D = D; a.W = W; a.bf16 = f.bf16;
  if (int st = check_workspace(workspace, workspace_bytes, conv_bwd_bytes(a))) return st;
  a.partial = (float*)workspace;
  return timed(GDN_STAGE_CONV_BWD, stream, [&](hipStream_t s) { return launch_conv_bwd(a, s); });
}

int gdn_group_norm_fwd(const void* x, long long x_batch, long long x_token, const void* weight, const void* bias,
                       int weight_dtype, int weight_shared, const void* z, long long z_batch, long long z_token,
                       int activation, int rms, float eps, int B, int T, int G, int d, int dtype, void* y,
                       void* stream) {
  GroupNormArgs a{};
  a.x = {x, x_batch, x_token}; a.z = {z, z_batch, z_token};
  a.weight = weight; a.bias = bias; a.shared = weight_shared; a.y = y;
  a.act = activation; a.rms = rms; a.eps = eps; a.B = B; a.T = T; a.G = G; a.d = d;
  if (int st = check_norm(a, weight_dtype, dtype)) return st;
  if ((long long)B * T == 0) return ok();
  if (!x || !y) return fail(GDN_ERR_INVALID_ARGUMENT, "x and y are required");
  const int unit = a.bf16 ? 8 : 4;
  if (int st = check_rows("x", a.x, B, T, unit)) return st;
  if (z)
    if (int st = check_rows("z", a.z, B, T, unit)) return st;
  return timed(GDN_STAGE_NORM, stream, [&](hipStream_t s) { return launch_group_norm_fwd(a, s); });
}

size_t gdn_group_norm_bwd_workspace_bytes(int B, int T, int G, int d, int weight_shared) {
  if (B < 0 || T < 0 || G <= 0 || d <= 0 || d % 8 || d > 8192 || (long long)G * d >= (1 << 23) ||
      (long long)B * T >= (1LL << 25))
    return 0;
  GroupNormArgs a{};
  a.B = B; a.T = T; a.G = G; a.d = d; a.shared = weight_shared;
  a.dweight = &a;   // any: the size is the same for one of the sums and for both
  return group_norm_bwd_bytes(a);
}

int gdn_group_norm_bwd(const void* dout, long long dout_batch, long long dout_token, const void* x, long long x_batch,
                       long long x_token, const void* weight, const void* bias, int weight_dtype, int weight_shared,
                       const void* z, long long z_batch, long long z_token, int activation, int rms, float eps, int B,
                       int T, int G, int d, int dtype, void* dx, void* dz, void* dweight, void* dbias, void* workspace,
                       size_t workspace_bytes, void* stream) {
  GroupNormArgs a{};
  a.dout = {dout, dout_batch, dout_token}; a.x = {x, x_batch, x_token}; a.z = {z, z_batch, z_token};
  a.weight = weight; a.bias = bias; a.shared = weight_shared;
  a.dx = dx; a.dz = dz; a.dweight = dweight; a.dbias = dbias;
  a.act = activation; a.rms = rms; a.eps = eps; a.B = B; a.T = T; a.G = G; a.d = d;
  if (int st = check_norm(a, weight_dtype, dtype)) return st;
  const bool tokens = (long long)B * T > 0;
  if (!tokens && !dweight && !dbias) return ok();
  if (tokens) {
    if (!dout || !x || !dx || (z && !dz))
      return fail(GDN_ERR_INVALID_ARGUMENT, "dout, x and dx are required, and dz with z");
    const int unit = a.bf16 ? 8 : 4;
    if (int st = check_rows("dout", a.dout, B, T, unit)) return st;
    if (int st = check_rows("x", a.x, B, T, unit)) return st;
    if (z)
      if (int st = check_rows("z", a.z, B, T, unit)) return st;
  }
  if (int st = check_workspace(workspace, workspace_bytes, group_norm_bwd_bytes(a))) return st;
  a.partial = (float*)workspace;
  return timed(GDN_STAGE_NORM, stream, [&](hipStream_t s) { return launch_group_norm_bwd(a, s); });
}

int kda_decode(const void* q, const void* k, const void* v, const void* a, const void* b, const float* A_log,
               const float* dt_bias, void* state, int state_dtype, const int32_t* state_indices, void* o, int B, int T,
               int H, int HV, int K, int V, int pool, float scale, float softplus_beta, float softplus_threshold,
               int use_qk_l2norm, float eps, int dtype, void* stream) {
  if (int st = known_dtype(dtype)) return st;
  if (state_dtype != GDN_DTYPE_F32 && state_dtype != GDN_DTYPE_BF16)
    return fail(GDN_ERR_INVALID_ARGUMENT, "unknown state dtype code %d", state_dtype);
  if (B < 0 || H <= 0 || HV <= 0 || K <= 0 || V <= 0 || pool < 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "sizes must be positive: B=%d H=%d HV=%d K=%d V=%d pool=%d", B, H, HV, K, V,
                pool);
  if (T < 1 || T > 4) return fail(GDN_ERR_INVALID_ARGUMENT, "a step takes T = 1..4 tokens (got T=%d)", T);
  if (HV % H != 0) return fail(GDN_ERR_INVALID_ARGUMENT, "HV (%d) must be a multiple of H (%d)", HV, H);
  if ((K != 64 && K != 128) || (V != 64 && V != 128))
    return fail(GDN_ERR_UNSUPPORTED, "supported head dims are K, V in {64, 128} (got K=%d V=%d)", K, V);
  if (!state_indices && pool < B)
    return fail(GDN_ERR_INVALID_ARGUMENT, "identity slots need pool >= B (pool=%d B=%d)", pool, B);
  if (!(softplus_beta > 0.f)) return fail(GDN_ERR_INVALID_ARGUMENT, "softplus_beta must be > 0");
  if (!(eps >= 0.f)) return fail(GDN_ERR_INVALID_ARGUMENT, "eps must be >= 0");
  if (B == 0) return ok();
  if (!q || !k || !v || !a || !b || !A_log || !dt_bias || !state || !o)
    return fail(GDN_ERR_INVALID_ARGUMENT, "q, k, v, a, b, A_log, dt_bias, state and o are required");
  const void* ptrs[] = {q, k, v, state, o};
  for (const void* p : ptrs)
    if (!aligned16(p)) return fail(GDN_ERR_INVALID_ARGUMENT, "q, k, v, state and o must be 16-byte aligned");
  if ((long long)pool * HV * V * K >= (1LL << 40)) return fail(GDN_ERR_UNSUPPORTED, "state pool too large");
  if (too_many((long long)B * HV, 256))
    return fail(GDN_ERR_UNSUPPORTED, "too many batch rows x heads for one launch (B=%d HV=%d)", B, HV);
  KdaStepArgs s{};
  s.q = q; s.k = k; s.v = v; s.a = a; s.b = b; s.A_log = A_log; s.dt_bias = dt_bias;
  s.state = state; s.state_bf16 = state_dtype == GDN_DTYPE_BF16; s.idx = state_indices; s.pool = pool; s.o = o;
  s.B = B; s.T = T; s.H = H; s.HV = HV; s.K = K; s.V = V;
  s.scale = scale; s.sp_beta = softplus_beta; s.sp_thr = softplus_cut(softplus_threshold); s.eps = eps;
  s.use_norm = use_qk_l2norm != 0; s.bf16 = dtype == GDN_DTYPE_BF16;
  return timed(GDN_STAGE_DECODE, stream, [&](hipStream_t st) { return launch_kda_decode(s, st); });
}

size_t ssm_chunk_fwd_workspace_bytes(int B, int T, int Hk, int HV, int K, int V, int num_seqs, int varlen,
                                     int dtype) {
  if (B < 0 || T < 0 || Hk <= 0 || HV <= 0 || HV % Hk || K <= 0 || V <= 0 || num_seqs < 0) return 0;
  if (dtype != GDN_DTYPE_F32 && dtype != GDN_DTYPE_BF16) return 0;
  const int N = varlen ? num_seqs : B;
  if (N == 0 || too_many((long long)N * HV, 256)) return 0;
  return ssm_plan(B, T, Hk, HV, K, V, N, varlen != 0, dtype == GDN_DTYPE_BF16).bytes;
}

int ssm_chunk_fwd(const void* x, long long x_batch, long long x_token, const void* dt, long long dt_batch,
                  long long dt_token, const void* Bm, long long B_batch, long long B_token, const void* Cm,
                  long long C_batch, long long C_token, const void* z, long long z_batch, long long z_token,
                  const float* A_log, const float* dt_bias, const float* D, int dt_softplus, const float* h0,
                  float* ht, const int64_t* cu_seqlens, int num_seqs, int B, int T, int Hk, int HV, int K, int V,
                  int chunk_size, int dtype, void* y, void* workspace, size_t workspace_bytes, void* stream) {
  SsmArgs a{};
  a.x = {x, x_batch, x_token}; a.dt = {dt, dt_batch, dt_token};
  a.B = {Bm, B_batch, B_token}; a.C = {Cm, C_batch, C_token}; a.z = {z, z_batch, z_token};
  a.A_log = A_log; a.dt_bias = dt_bias; a.D = D; a.softplus = dt_softplus;
  a.h0 = h0; a.ht = ht; a.cu = cu_seqlens; a.y = y;
  a.nb = B; a.T = T; a.Hk = Hk; a.HV = HV; a.K = K; a.V = V;
  if (int st = check_seqs(cu_seqlens, num_seqs, B, T, a.N)) return st;
  if (int st = check_ssm(a, dtype)) return st;
  if (chunk_size != 64) return fail(GDN_ERR_UNSUPPORTED, "chunk_size must be 64 (got %d)", chunk_size);
  if (a.N == 0) return ok();
  const bool tokens = (long long)B * T > 0;
  if (!tokens && !ht) return ok();
  if (tokens) {
    if (int st = check_ssm_rows(a)) return st;
  } else if (!A_log) {
    return fail(GDN_ERR_INVALID_ARGUMENT, "A_log is required");
  }
  if (!aligned16(h0) || !aligned16(ht))
    return fail(GDN_ERR_INVALID_ARGUMENT, "h0 and ht must be 16-byte aligned");
  // one launch has a work-group per (segment, head), at most one segment per 64 tokens
  // and one more for each sequence
  if (too_many(((long long)B * T / 64 + a.N + 8) * HV, 256))
    return fail(GDN_ERR_UNSUPPORTED, "too many sequences x heads for one launch (N=%d HV=%d)", a.N, HV);
  const SsmPlan p = ssm_plan(B, T, Hk, HV, K, V, a.N, cu_seqlens != nullptr, a.bf16 != 0);
  if (p.bytes > 0) {
    if (!workspace || workspace_bytes < p.bytes)
      return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", p.bytes,
                      workspace ? workspace_bytes : (size_t)0);
    if (((uintptr_t)workspace & 255u) != 0)
      return fail(GDN_ERR_INVALID_ARGUMENT, "workspace must be 256-byte aligned");
  }
  a.workspace = workspace;
  return timed(GDN_STAGE_SSM_SCAN, stream, [&](hipStream_t s) { return launch_ssm_fwd(a, s); });
}

int ssm_step(const void* x, long long x_batch, long long x_token, const void* dt, long long dt_batch,
             long long dt_token, const void* Bm, long long B_batch, long long B_token, const void* Cm,
             long long C_batch, long long C_token, const void* z, long long z_batch, long long z_token,
             const float* A_log, const float* dt_bias, const float* D, int dt_softplus, void* state,
             int state_dtype, const int32_t* state_indices, int pool, int B, int T, int Hk, int HV, int K, int V,
             int dtype, void* y, void* stream) {
  SsmArgs a{};
  a.x = {x, x_batch, x_token}; a.dt = {dt, dt_batch, dt_token};
  a.B = {Bm, B_batch, B_token}; a.C = {Cm, C_batch, C_token}; a.z = {z, z_batch, z_token};
  a.A_log = A_log; a.dt_bias = dt_bias; a.D = D; a.softplus = dt_softplus;
  a.state = state; a.idx = state_indices; a.pool = pool; a.y = y;
  a.nb = B; a.T = T; a.Hk = Hk; a.HV = HV; a.K = K; a.V = V;
  if (B < 0 || pool < 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "sizes must be positive (B, pool >= 0): B=%d pool=%d", B, pool);
  if (T < 1 || T > 4) return fail(GDN_ERR_INVALID_ARGUMENT, "a step takes T = 1..4 tokens (got T=%d)", T);
  if (int st = check_ssm(a, dtype)) return st;
  if (state_dtype != GDN_DTYPE_F32 && state_dtype != GDN_DTYPE_BF16)
    return fail(GDN_ERR_INVALID_ARGUMENT, "unknown state dtype code %d", state_dtype);
  a.state_bf16 = state_dtype == GDN_DTYPE_BF16;
  if (!state_indices && pool < B)
    return fail(GDN_ERR_INVALID_ARGUMENT, "identity slots need pool >= B (pool=%d B=%d)", pool, B);
  if (B == 0) return ok();
  if (!state) return fail(GDN_ERR_INVALID_ARGUMENT, "state is required");
  if (int st = check_ssm_rows(a)) return st;
  if (!aligned16(state)) return fail(GDN_ERR_INVALID_ARGUMENT, "state must be 16-byte aligned");
  if ((long long)pool * HV * V * K >= (1LL << 40)) return fail(GDN_ERR_UNSUPPORTED, "state pool too large");
  if (too_many((long long)B * HV, 256))
    return fail(GDN_ERR_UNSUPPORTED, "too many batch rows x heads for one launch (B=%d HV=%d)", B, HV);
  return timed(GDN_STAGE_SSM_STEP, stream, [&](hipStream_t s) { return launch_ssm_step(a, s); });
}

static int state_q8(bool store, void* wide, int state_dtype, int entries, void* q8, int q8_format, float* scales,
                    int pool, const int32_t* src_indices, const int32_t* dst_indices, int N, int HV, int K, int V,
                    void* stream) {
  if (N < 0 || HV <= 0 || K <= 0 || V <= 0 || pool < 0 || entries < 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "sizes must be positive: N=%d HV=%d K=%d V=%d pool=%d entries=%d", N, HV,
                    K, V, pool, entries);
  if (K != 64 && K != 128) return fail(GDN_ERR_UNSUPPORTED, "K must be 64 or 128 (got %d)", K);
  if (state_dtype != GDN_DTYPE_F32 && state_dtype != GDN_DTYPE_BF16)
    return fail(GDN_ERR_INVALID_ARGUMENT, "unknown state dtype code %d", state_dtype);
  if (q8_format != GDN_Q8_INT8 && q8_format != GDN_Q8_E4M3)
    return fail(GDN_ERR_INVALID_ARGUMENT, "unknown 8-bit format code %d", q8_format);
  const int from = store ? entries : pool, to = store ? pool : entries;
  if (!src_indices && from < N)
    return fail(GDN_ERR_INVALID_ARGUMENT, "identity sources need %d entries (got %d)", N, from);
  if (!dst_indices && to < N)
    return fail(GDN_ERR_INVALID_ARGUMENT, "identity targets need %d entries (got %d)", N, to);
  const long long most = N > pool ? (N > entries ? N : entries) : (pool > entries ? pool : entries);
  if (most * HV * V * K >= (1LL << 40)) return fail(GDN_ERR_UNSUPPORTED, "state arrays too large");
  if (N == 0) return ok();
  if (!wide || !q8 || !scales) return fail(GDN_ERR_INVALID_ARGUMENT, "the states, q8 and scales are required");
  if (!aligned16(wide) || !aligned16(q8) || !aligned16(scales))
    return fail(GDN_ERR_INVALID_ARGUMENT, "tensor pointers must be 16-byte aligned");
  if (too_many((long long)N * HV * V / (2048 / K) + 1, 256))   // K / 8 threads a row
    return fail(GDN_ERR_UNSUPPORTED, "too many state rows for one launch");
  StateQ8Args a{};
  a.wide = wide; a.wide_bf16 = state_dtype == GDN_DTYPE_BF16; a.wide_n = entries;
  a.q8 = q8; a.scales = scales; a.pool = pool; a.e4m3 = q8_format == GDN_Q8_E4M3;
  a.src_idx = src_indices; a.dst_idx = dst_indices; a.N = N; a.HV = HV; a.K = K; a.V = V;
  return timed(GDN_STAGE_STATE_Q8, stream, [&](hipStream_t s) {
    return store ? launch_state_store_q8(a, s) : launch_state_load_q8(a, s);
  });
}

int gdn_state_store_q8(const void* src, int state_dtype, int entries, const int32_t* src_indices, void* q8,
                       int q8_format, float* scales, int pool, const int32_t* dst_indices, int N, int HV, int K,
                       int V, void* stream) {
  return state_q8(true, const_cast<void*>(src), state_dtype, entries, q8, q8_format, scales, pool, src_indices,
                  dst_indices, N, HV, K, V, stream);
}

int gdn_state_load_q8(const void* q8, int q8_format, const float* scales, int pool, const int32_t* src_indices,
                      void* dst, int state_dtype, int entries, const int32_t* dst_indices, int N, int HV, int K, int V,
                      void* stream) {
  return state_q8(false, dst, state_dtype, entries, const_cast<void*>(q8), q8_format, const_cast<float*>(scales), pool,
                  src_indices, dst_indices, N, HV, K, V, stream);
}

}  // extern "C"
