// host_checks.hpp -- host-only rules of libmoe: the limits the kernels are
// built for, buffer sizes and launch geometry, and the argument checks of
// every entry point.  Plain C++17 with no HIP dependency, so that it can be
// compiled and exercised on its own (for instance under address and
// undefined-behaviour sanitizers); the kernels' launchers include it for the
// same sizes.  Return codes and the meaning of each argument: include/moe.h.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

// ---- limits the kernels are written for ------------------------------------
constexpr int kMaxExperts = 1024;     // expert scans hold 4 (LDS plan) or 2 experts a thread
constexpr int kMaxTopK = 64;          // one slot per lane of a wave64
constexpr int kPlanThreads = 512;     // plan kernels: 8 waves per block
constexpr int kPlanTilePairs = 2048;  // count tile of the plan kernels (whole tokens)
constexpr int kPlanSubPairs = kPlanThreads;  // assign block: one 64-pair chunk per wave
constexpr int kSmallPairs = 2048;     // plan-and-dispatch in one launch: pairs it plans
constexpr int kTileHist = 2048;       // tiled plan-and-dispatch: histogram entries it reads
constexpr int kMapThreads = 256;      // routing-map conversion block
constexpr int kMapLaneExperts = 16;   // map bytes per lane

// ---- sizes -------------------------------------------------------------------

// Rows of the packed buffer: N*k + E*(A-1), or E*cap with a fixed capacity.
inline int64_t max_rows(const moe_problem &p) {
  if (p.expert_capacity > 0) return static_cast<int64_t>(p.n_experts) * p.expert_capacity;
  return p.n_tokens * p.top_k + static_cast<int64_t>(p.n_experts) * (p.pad_multiple - 1);
}

int64_t payload_row_bytes(const moe_problem &p);  // of a valid problem
int64_t scale_row_bytes(const moe_problem &p);

// How the (token, k) pairs are split into tiles for the plan kernels.
struct PlanGeom {
  int64_t npairs;      // N * k
  int tile_tokens;     // whole tokens per tile (at most kPlanTilePairs pairs)
  int64_t tile_pairs;  // tile_tokens * k
  int ntiles;          // ceil(N / tile_tokens), >= 1
  int subs;            // sub-tiles of kPlanSubPairs pairs per count tile (assign blocks)
  bool single;         // one count tile: no separate counting kernel
  int key_bits;        // bits needed for an expert id (ceil(log2 E))
};
PlanGeom plan_geometry(const moe_problem &p);
// ntiles * (E + 1) int32 (tile histograms, then each tile's fault bits),
// rounded up to 256 bytes; 0 for a single-tile plan
size_t plan_workspace_bytes(const moe_problem &p);

// How moe_plan_and_dispatch runs a problem: one launch (at most kSmallPairs
// pairs), tiled (the counting kernel, then one launch that finishes the plan
// and dispatches; at most kTileHist histogram entries), or the plan's
// kernels then the dispatch.  A fixed expert capacity takes the same modes
// (each expert's first cap pairs kept, the rest dropped by the launch that
// places them).
enum class PlanDispatchMode { kOneLaunch, kTiled, kSeparate };
PlanDispatchMode plan_dispatch_mode(const moe_problem &p);
// In one-launch mode without padding (A = 1) or capacity, a pair's packed row is the
// count of valid pairs ahead of it in (expert, pair index) order, which a
// workgroup can count for its own pairs with ballots and one barrier, while
// workgroup 0 writes the plan arrays (the dispatch launcher also bounds the
// ballots a wave makes); otherwise every workgroup builds the plan in LDS.
bool one_launch_direct(const moe_problem &p);

// Workspace of the exchange plan: [EP][E+1] offsets and [EP][N*k] packed_src
// of the per-rank plans, then EP copies of the single-rank plan workspace.
struct ExchangeLayout {
  size_t offsets, packed_src, plan_ws, total;
  size_t plan_ws_bytes;  // per rank
};
moe_problem exchange_rank_problem(const moe_problem &p);  // one rank's own plan
ExchangeLayout exchange_layout(const moe_problem &p);

// Routing-map conversion: lanes per token (ceil(E/16) rounded up to a power
// of two), blocks, and workspace (one flag word per block, 256-byte rounded).
int map_lanes_per_token(int n_experts);
int map_blocks(const moe_problem &p);
size_t map_workspace_bytes(const moe_problem &p);

// ceil(cf * N * k / E) in double precision, or a negative error code
int64_t expert_capacity(int64_t n_tokens, int32_t top_k, int32_t n_experts, double cf);

// Rows of the packed buffer that can hold a token: N*k, or what the fixed
// capacity leaves of it.
inline int64_t expert_row_bound(const moe_problem &p) {
  const int64_t pairs = p.n_tokens * p.top_k, rows = max_rows(p);
  return pairs < rows ? pairs : rows;
}

// Parts that the rows of an expert are split into for its weights' gradient
// [E][n][k]: more than one where 64 x 64 tiles of it would leave most compute units
// without work and the rows are many.  At most kDwWorkgroups workgroups.  (us a call,
// parts against whole, by the rows of an expert:
//   rows                          1024           2048           8192
//   1 expert, 128 x 128       11.9 / 10.0    11.8 / 15.1    13.8 / 51.1
//   2 experts, 512 x 256      13.1 / 11.0    16.7 / 15.4    22.6 / 49.8
//   8 experts, 256 x 256      15.7 / 10.2    16.7 / 15.8    31.1 / 53.1
//   4 experts, 512 x 512      16.9 / 12.1    21.0 / 16.0    52.4 / 54.8 (two parts)
// The launch that joins the parts costs 2 to 5 us, which the split
// earns back somewhere between 2000 and 8000 rows, and before in the smallest dw.)
constexpr int kDwTile = 64, kDwWorkgroups = 512, kDwMostParts = 16, kDwPartRows = 256;
int dw_parts(const moe_problem &p, int64_t n, int64_t k);

// Workspace of the experts' backward passes: column sums of dz over 16-row
// chunks of each expert (at most rows / 16 + E of them, up to 2 * out_dim
// columns), for dbias; then the parts of dw, fp32.
constexpr int kBiasChunkRows = 16;
// The launch that computes dz (of a layer's out_dim columns): one workgroup for
// every such chunk, of any routing, and kGradCols columns, in whole rounds of the 8 XCDs.
constexpr int kGradCols = 512, kGradThreads = 256;
int64_t expert_grad_workgroups(const moe_problem &p, int64_t out_dim);
size_t expert_bias_bytes(const moe_problem &p, const moe_expert_op &op);
size_t expert_workspace_bytes(const moe_problem &p, const moe_expert_op &op);

// ---- argument checks: MOE_OK or the code the entry point returns -----------
namespace host {

int check_problem(const moe_problem *p);
int check_exchange(const moe_problem *p);

int check_plan_args(const moe_problem *p, const int32_t *topk_ids, const moe_plan *plan,
                    const void *workspace);
// moe_plan_and_dispatch and its halves: the plan's arguments and the dispatch's
int check_plan_and_dispatch_args(const moe_problem *p, const int32_t *topk_ids, const moe_plan *plan,
                                 const uint16_t *hidden, const float *topk_weights,
                                 const float *input_scale, const void *payload, const void *scales,
                                 const void *workspace);
int check_dispatch_args(const moe_problem *p, const moe_plan *plan, const uint16_t *hidden,
                        const void *payload, const void *scales);
int check_dispatch_scaled_args(const moe_problem *p, const moe_plan *plan, const uint16_t *hidden,
                               const float *input_scale, const void *payload, const void *scales);
int check_dispatch_gated_args(const moe_problem *p, const moe_plan *plan, const uint16_t *hidden,
                              const float *topk_weights, const void *payload, const void *scales);
int check_combine_args(const moe_problem *p, const moe_plan *plan, const uint16_t *expert_out,
                       const float *topk_weights, const uint16_t *out);

int check_exchange_plan_args(const moe_problem *p, const int32_t *topk_ids, const moe_exchange *x,
                             const void *workspace);
int check_exchange_dispatch_args(const moe_problem *p, const moe_exchange *x, const uint16_t *hidden,
                                 const void *payload, const void *scales);
int check_exchange_dispatch_scaled_args(const moe_problem *p, const moe_exchange *x,
                                        const uint16_t *hidden, const float *input_scale,
                                        const void *payload, const void *scales);
int check_exchange_dispatch_gated_args(const moe_problem *p, const moe_exchange *x,
                                       const uint16_t *hidden, const float *topk_weights,
                                       const void *payload, const void *scales);
int check_exchange_combine_args(const moe_problem *p, const moe_exchange *x, const uint16_t *expert_out,
                                const float *topk_weights, const uint16_t *out);

int check_map_args(const moe_problem *p, const uint8_t *routing_map, const float *probs,
                   const int32_t *topk_ids, const float *topk_weights, const uint32_t *status,
                   const void *workspace);

int check_combine_backward_args(const moe_problem *p, const moe_plan *plan, const uint16_t *expert_out,
                                const float *topk_weights, const uint16_t *dout, const uint16_t *dy,
                                const float *dweights);

int check_expert_op(const moe_problem *p, const moe_expert_op *op);
// residual: the linear layer only
int check_expert_forward_args(const moe_problem *p, const moe_plan *plan, const moe_expert_op *op,
                              const void *x, const float *x_scales, const void *w, const float *w_scales,
                              const float *bias, const uint16_t *residual, const uint16_t *y,
                              const uint16_t *preact);
int check_expert_backward_args(const moe_problem *p, const moe_plan *plan, const moe_expert_op *op,
                               bool glu, const uint16_t *dy, const uint16_t *preact, const uint16_t *x,
                               const uint16_t *w, const uint16_t *dz, const uint16_t *dx,
                               const uint16_t *dw, const float *dbias, const void *workspace);

const char *error_text(int code);

}  // namespace host
}  // namespace moe
