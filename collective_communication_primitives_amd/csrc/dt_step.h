// dt_step.h -- kernel argument blocks and launchers of the model-step
// operators whose mathematics crosses the ranks: layer norm (norm.hip),
// expert routing and the experts' token exchange (moe.hip), the loss over a
// sharded vocabulary (loss.hip).  step_api.cpp checks, plans and enqueues.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dt.h"
#include "dt_launch.h"

namespace dt {

// Records this thread's last error message (api.cpp) and hands `st` back.
dt_status report_error(dt_status st, const char* message);

// Rows of all ranks in rank order: rank r holds rows [start[r], start[r + 1]).
// Entries past the last rank repeat the total, so a search needs no bound.
struct RowTable {
    uint32_t start[kMaxRanksHost + 1];
};

// ------------------------------------------------------------ layer norm --
struct NormArgs {
    const void* x[kMaxRanksHost];
    const void* weight[kMaxRanksHost];
    const void* bias[kMaxRanksHost];   // all NULL: no bias
    void* y[kMaxRanksHost];
    float* mean[kMaxRanksHost];        // all NULL: the statistics are not stored
    float* rstd[kMaxRanksHost];
    RowTable rows;
    uint32_t cols;
    float eps;
    int nranks;
};
struct NormBackArgs {
    const void* dy[kMaxRanksHost];
    const void* x[kMaxRanksHost];
    const void* weight[kMaxRanksHost];
    const float* mean[kMaxRanksHost];
    const float* rstd[kMaxRanksHost];
    void* dx[kMaxRanksHost];
    void* dweight[kMaxRanksHost];
    void* dbias[kMaxRanksHost];        // all NULL: no bias
    float* partial;                    // [strips][2][cols]
    RowTable rows;
    uint32_t cols;
    uint32_t strips;
    int nranks;
};
hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t s);
uint32_t norm_strips(uint32_t rows, uint32_t cols);
hipError_t launch_norm_backward(const NormBackArgs& a, int dtype, hipStream_t s);

// --------------------------------------------------------------- routing --
struct RouteArgs {
    const void* logits[kMaxRanksHost];
    int32_t* experts[kMaxRanksHost];
    float* weights[kMaxRanksHost];
    const float* bias;
    RowTable rows;
    uint32_t nexperts, topk, groups, topk_groups;
    int sigmoid, renormalize;
    float scale;
};
struct RouteBackArgs {
    const void* logits[kMaxRanksHost];
    const int32_t* experts[kMaxRanksHost];
    const float* dweights[kMaxRanksHost];
    void* dlogits[kMaxRanksHost];
    RowTable rows;
    uint32_t nexperts, topk;
    int sigmoid, renormalize;
    float scale;
};
hipError_t launch_route(const RouteArgs& a, int nranks, int dtype, hipStream_t s);
hipError_t launch_route_backward(const RouteBackArgs& a, int nranks, int dtype, hipStream_t s);

// -------------------------------------------------------------- exchange --
// A slot is one (rank, token, choice); slots are numbered in that order.
constexpr uint32_t kPlanSlots = 1024;  // slots per workgroup of the plan (2048 took 10 us longer for 131072 slots)
constexpr uint32_t kFewSlots = 4096;   // up to here plan and copy are one launch
struct PlanArgs {
    const int32_t* experts[kMaxRanksHost];
    int32_t* positions[kMaxRanksHost];
    int32_t* offsets[kMaxRanksHost];
    uint32_t capacity[kMaxRanksHost];
    RowTable rows;
    uint32_t* counts;                  // [plan workgroups + 1][nexperts]
    uint32_t nexperts, topk, per_rank;
    int nranks;
};
// Row traffic between tokens (rank r's rows) and the experts' rows (rank q's
// buffer): dispatch, combine and combine's backward pass.
struct ExchangeRowsArgs {
    const void* tokens_in[kMaxRanksHost];   // dispatch: x; combine's backward: dout
    void* tokens_out[kMaxRanksHost];        // combine: out
    const void* rows_in[kMaxRanksHost];     // combine and its backward: y
    void* rows_out[kMaxRanksHost];          // dispatch: recv; combine's backward: dy
    const int32_t* experts[kMaxRanksHost];
    const int32_t* positions[kMaxRanksHost];
    const float* weights[kMaxRanksHost];    // all NULL: ones
    float* dweights[kMaxRanksHost];
    uint32_t capacity[kMaxRanksHost];
    RowTable rows;
    uint32_t cols, nexperts, topk, per_rank;
    int nranks;
};
inline uint32_t plan_blocks(uint64_t slots) { return uint32_t((slots + kPlanSlots - 1) / kPlanSlots); }
hipError_t launch_dispatch(const PlanArgs& p, const ExchangeRowsArgs& a, int esize, hipStream_t s);
hipError_t launch_combine(const ExchangeRowsArgs& a, int dtype, hipStream_t s);
hipError_t launch_combine_backward(const ExchangeRowsArgs& a, int dtype, hipStream_t s);

// ------------------------------------------------------- vocabulary loss --
// Everything of one call; the launchers cut it into tiles and pieces.  Of the
// inputs that are Replicate, rank 0's copy is read.
struct LossArgs {
    const void* hidden;                     // [tokens, cols]
    const void* weight[kMaxRanksHost];      // [vocab rows of rank r, cols]
    const int64_t* targets;
    const float* lse_in;                    // backward
    const float* dloss;
    float* loss[kMaxRanksHost];             // forward
    float* lse[kMaxRanksHost];
    void* dhidden[kMaxRanksHost];
    void* dweight[kMaxRanksHost];
    RowTable vocab;                         // vocabulary rows of the ranks
    uint32_t tokens, cols;
    uint32_t piece;                         // backward: vocabulary rows per piece
    int64_t ignore_index;
    char* workspace;
    int nranks;
};
constexpr uint32_t kLossPiece = 16384;      // vocabulary rows per piece at least, unless the caller says otherwise
constexpr uint32_t kMaxLossPiece = 1 << 20; // 256 rows of d stay within the 31 bits of a buffer resource's offsets
uint32_t loss_piece(const RowTable& vocab, int nranks, uint64_t tokens, uint64_t cols, int dtype, uint64_t asked);
uint64_t loss_workspace(const RowTable& vocab, int nranks, uint64_t tokens, uint64_t cols, int dtype);
uint64_t loss_backward_workspace(int nranks, uint64_t tokens, uint64_t cols, uint32_t piece, int dtype);
hipError_t launch_loss(const LossArgs& a, int dtype, hipStream_t s);
hipError_t launch_loss_backward(const LossArgs& a, int dtype, hipStream_t s);

}  // namespace dt
