// Host-side launch arguments of the operators around the scans: the short
// causal convolution, the selective state-space scan and step, and the 8-bit
// state cache (internal to the library).  Arguments have been validated by the
// C-ABI layer (mixer_api.hip) before these run.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

// Records the detail message of the calling thread's last failing call and
// returns `status`; ok() clears it.  (gdn_api.hip)
int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int ok();

// A [B, T, ...] operand whose rows need not be packed: row t of batch b starts
// `batch * b + token * t` elements behind `p`.
struct Rows {
  const void* p;
  long long batch, token;
};

struct ConvArgs {
  Rows x;                       // [B, T, D]
  const void* weight;           // [D, W]
  const void* bias;             // [D] or nullptr
  void* state;                  // [pool, W - 1, D] or nullptr
  const int32_t* idx;           // [N] slot of each sequence, or nullptr (slot n)
  const int32_t* has;           // [N] or nullptr (prompts: every sequence starts from zeros)
  const int64_t* cu;            // [N + 1] or nullptr (dense)
  void* out[3];                 // packed [B, T, width] each; unused sections nullptr
  int end[3];                   // channel ends of the sections
  int norm_dim, norm_sections;  // 0 = no norm
  float eps;
  int silu;
  int N, B, T, D, W, pool;
  int bf16;
};
hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t s);
hipError_t launch_conv_step(const ConvArgs& a, hipStream_t s);

struct SsmArgs {
  Rows x, dt, B, C, z;          // [B, T, HV, V], [B, T, HV], [B, T, Hk, K] x 2, [B, T, HV, V] (z.p may be nullptr)
  const float *A_log, *dt_bias, *D;   // [HV]; the last two may be nullptr
  int softplus;
  // prompts
  const float* h0;              // [N, HV, V, K] or nullptr
  float* ht;                    // [N, HV, V, K] or nullptr
  const int64_t* cu;            // [N + 1] or nullptr
  void* workspace;              // segment states and log-decays; nullptr when one segment a sequence is enough
  // single tokens
  void* state;                  // [pool, HV, V, K]
  int state_bf16;
  const int32_t* idx;
  int pool;
  void* y;                      // [B, T, HV, V]
  int N, nb, T, Hk, HV, K, V;   // nb: batch rows
  int bf16;
};
// How a prompt call is cut: every sequence into segments of `seg` tokens (a
// multiple of 64), at most `slots` segments in all, `nh` heads a work-group.  At most
// `joins` sequences have more than one segment, together at most `states`, whose
// states the workspace holds.
struct SsmPlan {
  int nh, seg, slots, joins, states;
  bool split;                   // whether a sequence can have more than one segment
  size_t decay_off, table_off, bytes;   // workspace: states, log2-decays, the table of split sequences
};
SsmPlan ssm_plan(int nb, int T, int Hk, int HV, int K, int V, int N, bool varlen, bool bf16);
hipError_t launch_ssm_fwd(const SsmArgs& a, hipStream_t s);
hipError_t launch_ssm_step(const SsmArgs& a, hipStream_t s);

struct StateQ8Args {
  void* wide;                   // [wide_n, HV, V, K] fp32 or bf16: the source of a store, the target of a load
  int wide_bf16;
  int wide_n;
  void* q8;                     // [pool, HV, V, K] codes
  float* scales;                // [pool, HV, V]
  int pool;
  int e4m3;                     // 1 = e4m3 codes, 0 = int8
  const int32_t *src_idx, *dst_idx;   // [N] or nullptr (the identity)
  int N, HV, K, V;
};
hipError_t launch_state_store_q8(const StateQ8Args& a, hipStream_t s);
hipError_t launch_state_load_q8(const StateQ8Args& a, hipStream_t s);

}  // namespace gdn
