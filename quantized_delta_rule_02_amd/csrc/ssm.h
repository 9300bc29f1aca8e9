// Launchers of the selective state space scan (ssm.hip, ssm_bwd.hip), called by the C ABI (mix_api.cpp).
#pragma once
#include "runs.h"

namespace sq {

struct SsmParams {
    Runs runs;                       // segments; forward without segments: not used by the scan kernel
    int32_t dtype, channels, d_state, n_groups, group_channels, softplus;
    Rows u, dt, b, c, z, y;          // z.p NULL: no gate
    const float* a;                  // [channels][d_state]
    const float* d;                  // [channels] or NULL
    const float* dt_bias;            // [channels] or NULL
    const float* s0;                 // [n_seq][channels][d_state] or NULL
    float* s1;
    // workspace, per segment
    float* hseg;                     // [slot][channels][d_state] state after the segment from zero, then the state before it; the gradients'
                                     // main kernel, its last reader, leaves the segment's sum of da there
    float* kseg;                     // backward: the same of the state's gradient, in the other direction
    float* dsum;                     // [slot][channels] sum of the steps
    // State before a segment's tiles of 8 tokens but the first, from zero, and the sum of the steps up to there: of the tile that starts at
    // token t in row t / 8.  Such a tile starts 8 tokens or more behind its sequence's start, so no two of them share a row.
    float* htile;                    // backward: [(n_tokens + 7) / 8][channels][d_state]
    float* dtile;                    // [(n_tokens + 7) / 8][channels]
    // backward
    Rows dy, du, ddt, db, dc, dz;
    const float* ds1;
    float* ds0;
    float* da;
    float* dd;
    float* ddt_bias;
    float* dd_part;                  // [slot][2][channels]: of dd and ddt_bias
    float* bc_part;                  // [block of channels][n_tokens][2][d_state]
    // one token of each request
    const int32_t* slots;
    int64_t n_slots, batch;
    float* state;                    // [n_slots][channels][d_state]
};

constexpr int kSsmWaves = 4;         // of a workgroup
constexpr int kSsmTile = 8;          // tokens whose decays a lane of the gradients' main kernel holds in registers
// Channels of a workgroup: a lane holds four states of one channel.
inline int ssm_block_channels(int d_state) { return kSsmWaves * 256 / d_state; }
// Workgroups' blocks of channels; none holds channels of two groups.
inline int64_t ssm_blocks(int channels, int n_groups, int d_state) {
    const int per = ssm_block_channels(d_state), g = channels / n_groups;
    return int64_t(n_groups) * ((g + per - 1) / per);
}
// log2 of a segment's tokens; -1: the forward scan goes without segments
int ssm_segment_log(int64_t n_tokens, int64_t n_seq, int64_t blocks, bool backward);

// workgroups' blocks of channels in the gradients' main kernel
int64_t ssm_grad_blocks(int channels, int n_groups, int d_state);

hipError_t launch_ssm_join(const SsmParams& p, int directions, hipStream_t s);     // 2: the gradients' direction too
hipError_t launch_ssm(const SsmParams& p, bool vec, hipStream_t s);
hipError_t launch_ssm_bwd(const SsmParams& p, bool vec, hipStream_t s);
hipError_t launch_ssm_step(const SsmParams& p, bool vec, hipStream_t s);

}  // namespace sq
