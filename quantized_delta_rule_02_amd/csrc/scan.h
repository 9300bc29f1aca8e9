// Launchers of the gated delta scan (scan_prep.hip, scan.hip, scan_bwd.hip), called by the C ABI (ops_api.cpp).
//
// Workspace of a call, per chunk slot and head (chunks of 32 tokens, counted from each sequence's start):
// chunk c of sequence b has the slot (start_b >> 5) + b + c.  Slots of different chunks differ, because
// ceil(len / 32) <= ((start + len) >> 5) - (start >> 5) + 1, and all lie below (n_tokens >> 5) + n_seq.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sq {

constexpr int kChunk = 32;
// One 32 x 32 matrix as MFMA A operands: 2 row tiles x 3 bfloat16 planes x 64 lanes x 8 elements.
constexpr int kMatShorts = 2 * 3 * 64 * 8;

struct ScanRows {
    void* p;
    int64_t stride;                  // elements between tokens
};

struct ScanParams {
    int32_t form, dtype, n_heads, n_heads_k, dk, dv, n_seq;
    int64_t n_tokens, n_slots;
    int64_t short_len;               // sequences of at most this length are not the chunked scan's (-1: all are)
    int32_t n_long;                  // at most so many are the chunked scan's
    const int32_t* seq_start;        // [n_seq + 1], or NULL: one sequence of n_tokens
    ScanRows q, k, v, y;
    const float* gate;               // [n_tokens][H] or [n_tokens][H][dk]
    const float* beta;               // [n_tokens][H]
    const float* s0;                 // [n_seq][H][dk][dv] or NULL
    float* s1;                       // or NULL
    // workspace
    uint16_t* mat_f;                 // [slot][H][2] diag(beta) That, That = (I + A diag(beta))^-1, and P; backward: [slot][H] That
    float* mat_gb;                   // [slot][H][2][32] products of the gates up to and after each token (GDN)
    // backward
    uint16_t* mat_r;                 // [slot][H][2] T^T, T = (I + diag(beta) A)^-1, and P^T
    float* mat_ap;                   // [slot][H][2][32][32] A and P in float32 (GDN)
    // in blocks of 16 value columns
    float* e;                        // [slot][H][dv / 16][32][16]
    float* du;                       // [slot][H][dv / 16][32][16]
    float* st;                       // [slot][H][dv / 16][dk][16] state before each chunk
    float* gt;                       // [slot][H][dv / 16][dk][16] gradient of the state after each chunk
    ScanRows dy, dq, dkk, dvv;
    const float* ds1;
    float* ds0;
    float* dgate;
    float* dbeta;
};

inline int64_t scan_slots(int64_t n_tokens, int n_seq) { return (n_tokens / kChunk) + n_seq; }

// prep: the chunks' small matrices; scan: forward with outputs, or for the backward pass the forward scan that keeps the
// states and e, beside the reverse scan of the state's gradient; grad: the gradients, all chunks at once.
hipError_t launch_scan_prep(const ScanParams& p, bool backward, hipStream_t s);
hipError_t launch_scan(const ScanParams& p, bool backward, hipStream_t s);
hipError_t launch_scan_grad(const ScanParams& p, hipStream_t s);
// The sequences of at most short_len tokens, token by token (d_k of 64 and more; outputs and final states), and with prep, in
// the same launch, the preparation of the others.
hipError_t launch_scan_short(const ScanParams& p, bool prep, hipStream_t s);

}  // namespace sq
