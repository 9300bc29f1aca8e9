// Packed sequences cut into runs of 2^log tokens, counted from each sequence's start: run c of sequence b has the slot
// (start_b >> log) + b + c.  Slots of different runs differ, because ceil(len / R) <= ((start + len) / R) - (start / R) + 1, every
// sequence has at least one (also an empty one), and all lie below (n_tokens >> log) + n_seq.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sq {

struct Rows {
    void* p;
    int64_t stride;                  // elements between tokens
};

struct Runs {
    const int32_t* seq_start;        // [n_seq + 1], or NULL: one sequence of n_tokens
    int64_t n_tokens;
    int32_t n_seq, log;
};

inline int64_t run_slots(int64_t n_tokens, int64_t n_seq, int log) { return (n_tokens >> log) + n_seq; }

struct Span {
    int64_t start, len;
};
// Sequence b, with offsets outside the packed arrays pulled inside (nothing beyond them is read or written).
__device__ __forceinline__ Span span_of(const Runs& r, int b) {
    if (!r.seq_start) return Span{0, r.n_tokens};
    int64_t s = r.seq_start[b], e = r.seq_start[b + 1];
    s = s < 0 ? 0 : s > r.n_tokens ? r.n_tokens : s;
    e = e < s ? s : e > r.n_tokens ? r.n_tokens : e;
    return Span{s, e - s};
}
__device__ __forceinline__ int64_t run_slot0(const Runs& r, const Span& q, int b) { return (q.start >> r.log) + b; }

struct RunAt {
    int seq, n;                      // the sequence, and how many tokens the run has (0: the slot is no run's, or an empty sequence's)
    bool first, last;                // of its sequence (an empty sequence's slot is both)
    int64_t tok0, start, len;        // the run's first token, the sequence
};
// Of the sequences whose first slot is not above the slot the run is the last one's: a search by 64 lanes at a time (one round
// for 64 sequences, two for 4096), since a round is a load's latency.  Called by whole waves; the result is the same in all lanes.
__device__ __forceinline__ RunAt run_of_slot(const Runs& r, int64_t slot) {
    int lo = 0, n = r.n_seq;                         // it is one of the n from lo
    while (n > 1) {
        const int step = (n + 63) / 64, at = ((int)threadIdx.x & 63) * step;
        const bool below = at < n && run_slot0(r, span_of(r, lo + at), lo + at) <= slot;
        const int last = 63 - __builtin_clzll(__ballot(below) | 1);
        lo += last * step;
        n = n - last * step < step ? n - last * step : step;
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    Span q = span_of(r, lo);
    const int64_t c0 = (slot - run_slot0(r, q, lo)) << r.log;
    const int64_t left = q.len - c0, most = int64_t(1) << r.log;
    const int len = __builtin_amdgcn_readfirstlane((int)q.len);
    q.start = __builtin_amdgcn_readfirstlane((int)q.start);
    const int rem = __builtin_amdgcn_readfirstlane((int)(c0 < 0 || left <= 0 ? 0 : left < most ? left : most));
    const int c = __builtin_amdgcn_readfirstlane((int)c0);
    return RunAt{lo, rem, c == 0, rem > 0 ? c + rem == len : c == 0, q.start + c, q.start, len};
}

}  // namespace sq
