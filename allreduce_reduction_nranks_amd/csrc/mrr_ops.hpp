// mrr_ops.hpp -- argument blocks and launchers of the operators that follow
// the rank sum in a training step: layer norm and sharded cross entropy.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "mrr.h"

namespace mrr {

// ---- layer norm of a rank sum -------------------------------------------------
struct NormFwdArgs {
  const void* in[MRR_MAX_RANKS];
  const void* residual;  // may be null
  const void* weight;    // may be null: 1
  const void* bias;      // may be null: 0
  void* sum;             // may be null
  void* out;
  float* mean;           // may be null
  float* rstd;           // may be null
  uint64_t rows, ld_in, ld_out;
  uint32_t cols;
  int nranks;
  float eps;
  int wf32;              // weight and bias are f32 (otherwise the data type)
  int in_place;          // sum is one of the inputs or the residual
};

struct NormBwdArgs {
  const void* dout;
  const void* sum;
  const void* weight;     // may be null: 1
  const float* mean;
  const float* rstd;
  const void* dresidual;  // may be null
  void* dsum;             // may be null
  void* dweight;          // may be null
  void* dbias;            // may be null
  float* partial;         // [groups][2][cols]: dweight and dbias of a group of rows
  uint64_t rows, ld_in, ld_out;
  uint32_t cols;
  uint32_t groups;
  int wf32;
};

// Groups of rows whose weight gradients are summed apart, for a call of this shape.
uint32_t norm_bwd_groups(uint64_t rows, uint32_t cols);
hipError_t launch_norm_fwd(const NormFwdArgs& a, int t, hipStream_t stream);
hipError_t launch_norm_bwd(NormBwdArgs a, int t, hipStream_t stream);

// ---- cross entropy over a sharded vocabulary ---------------------------------------
// The shards' rows, each shard padded to whole tiles of 256 rows.
struct XentVocab {
  const void* w[MRR_MAX_RANKS];
  uint32_t first_tile[MRR_MAX_RANKS + 1];
  uint32_t rows[MRR_MAX_RANKS];
  uint32_t first_row[MRR_MAX_RANKS];  // of the whole vocabulary
  int n;
};

// A counted token of a backward call.
struct XentToken {
  float lse, dl;
  int32_t target, pad;
};

// What the kernels of a backward call leave for each other.
struct XentScalars {
  uint32_t count;    // counted tokens
  float unscale_dz;  // f16: 1 / the scale of dz
};

struct XentArgs {
  XentVocab v;
  const XentScalars* scalars;
  const uint8_t* laid;  // weights of the piece laid out, null: read where they are
  const uint8_t* h;     // hidden states laid out, [tpad][kpad]
  uint64_t laid_plane, h_plane, dz_plane;
  uint32_t ldw, ldh, lddz;      // bytes between rows
  const void* hidden;           // the caller's, rows ld_h elements apart; the shards' ld_w
  uint64_t ld_h, ld_w;
  uint32_t tokens, tpad, cols, kpad;
  uint32_t tile0, ntiles;       // the piece
  uint32_t sub0, sub;           // tiles of the piece that a launch takes: from sub0 on, sub of them
  // forward
  float2* part;                 // max and sum of exponentials: logits_k [parts][tokens], few_k [tokens][parts]
  float* zt;                    // [tokens]: the target's logit
  const int64_t* targets;
  int64_t ignore;
  uint64_t part0;               // logits_k: pairs of the launches before
  uint32_t parts;               // few_k: pairs of a token
  // backward
  uint8_t* dz;                  // [tpad][piece]
  const XentToken* token;
  const int32_t* place;
  const int32_t* idx;
  uint32_t lo;                  // row of dz that holds what token 0's lost in rounding; 0: none do
  float* residue;               // [tpad]: lo 0: what rounding took from the target's dz
  uint32_t* hits;               // counted tokens by their target's tile
  uint32_t* hits_first;         // [tiles + 1]: a tile's first
  float* sum;                   // [splits][tpad][kpad]
  uint32_t splits, add;
  void* dhidden;
  void* dw[MRR_MAX_RANKS];
  uint64_t ld_dh, ld_dw;
};

struct XentJoinArgs {
  const float2* part;
  const float* zt;
  const int64_t* targets;
  int64_t ignore, vocab;
  float* loss;
  float* lse;
  uint64_t part_stride, token_stride;
  uint32_t parts, tokens;
};

// A call as the C ABI received it.
struct XentCall {
  const void* hidden;
  const void* const* weights;
  const size_t* rows;
  int nranks;
  const int64_t* targets;
  int64_t ignore;
  float* loss;         // forward
  float* lse_out;      // forward
  const float* lse;    // backward
  const float* dloss;  // backward
  size_t dloss_stride;
  void* dhidden;
  void* const* dweights;
  uint32_t tokens, cols;
  size_t ld_hidden, ld_weight;
  void* workspace;
};

// Tiles, pieces and the workspace's parts (byte offsets) of a call.
struct XentPlan {
  uint32_t tpad, kpad, tiles, piece, splits, dh_tile;
  uint64_t h_plane, laid_plane, dz_plane;
  uint64_t h, laid, dz, sum, token, idx, place, residue, hits, hits_first, scalars, part, zt;
  uint64_t bytes_in_place, bytes;  // weights (and a forward's hidden states) read where they are, and laid out
};

XentPlan xent_plan(uint32_t tokens, uint32_t cols, const size_t* rows, int nranks, int t, bool backward);

// How a call reads its operands.
struct XentWays {
  bool direct, hidden_direct;  // weights, hidden states where they are
  uint32_t groups;             // few_k's 16-token groups, 0: tiles
  uint64_t bytes;              // of the workspace
};
XentWays xent_ways(const XentCall& c, const XentPlan& p, int t, bool backward);
// Workspace of a call of these sizes: of any operands, or (in_place) of such as are read where they are.
uint64_t xent_bytes(uint32_t tokens, uint32_t cols, const size_t* rows, int nranks, int t, bool backward, bool in_place);
hipError_t launch_xent_fwd(const XentCall& c, int t, hipStream_t stream);
hipError_t launch_xent_bwd(const XentCall& c, int t, hipStream_t stream);

}  // namespace mrr
