// attn_packed.h -- launch interface of the packed-sequence kernels (attn_packed.cu), used by
// api_packed.cu.
#pragma once
#include "attn_kernels.h"

namespace sdpa {

struct PackedPlanParams {
  const int* cu_q;   // [B + 1]
  const int* cu_kv;  // [B + 1] (cu_q where queries and keys share their offsets)
  int B, T_q, T_kv;
  int causal, window;
  int* clean_q;   // [B + 1] scratch
  int* clean_kv;  // [B + 1] scratch
  PackedCounts* counts;
  PackedTile* tiles_fwd;  // the lists that are wanted, else null
  PackedTile* tiles_kv;
  PackedTile* tiles_q;
};

int launch_packed_plan(const PackedPlanParams& p, cudaStream_t stream);
int launch_attn_fwd_packed(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           const FwdParams& p, cudaStream_t stream);
int launch_packed_preprocess(int d_qk, int d_v, const BwdParams& p, cudaStream_t stream);
// After launch_bwd_q_packed with p.ds_rowsum set.
int launch_packed_doffset(const BwdParams& p, cudaStream_t stream);
int launch_packed_kv_combine(int d_qk, int d_v, const BwdParams& p, cudaStream_t stream);
// dK, dV: 128-row Q / dO boxes (d_qk = d_v = d), or 64-row ones (192, 128).
int launch_bwd_kv_wide_packed(int d, const CUtensorMap& tq128, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& tdo128, const BwdParams& p, cudaStream_t stream);
int launch_bwd_kv_packed_mla(const CUtensorMap& tq64, const CUtensorMap& tk, const CUtensorMap& tv,
                             const CUtensorMap& tdo64, const BwdParams& p, cudaStream_t stream);
// early: launched right behind the kv kernel, in whose tail it is set up.
int launch_bwd_q_packed(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                        const CUtensorMap& tdo, const BwdParams& p, bool early, cudaStream_t stream);

}  // namespace sdpa
