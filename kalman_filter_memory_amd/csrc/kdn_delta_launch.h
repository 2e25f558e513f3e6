// kdn_delta_launch.h -- arguments and launchers that the gated delta rule's forward and
// backward passes share (host side, internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/kdn.h"

namespace kdn {
namespace delta {

// workgroups of a launch stay below 2^32 with four slices of a head, and below the
// 2^32 threads of a grid with 512 each
constexpr int64_t kMaxStates = (1 << 20) - 1;
constexpr int32_t kMaxTokens = 1 << 30;

struct ForwardArgs {
    const void *q, *k, *v, *g, *beta;
    const int32_t* cu;  // packed sequences' first rows [B + 1], or null
    const float* S0;
    void* o;
    float* S_T;
    void *keep_E, *keep_S;  // for the backward pass
    int B, H, Hk, T, dv;
    int group;  // chunks per kept state (and a multiple of which a segment holds)
    // segments of every sequence (see Segments); maps: this launch forms their maps
    int segs;
    float *starts, *maps;
    float scale;
    bool gate_bf16;
};

// What the backward pass keeps between its kernels: chunks per kept state, and places
// for states (per head of values).
inline int kept_chunks(int dtype) { return dtype == KDN_BF16 ? 2 : 1; }
inline size_t kept_slots(const int32_t* cu, int B, int T, int group) {
    const int per = 32 * group;
    return cu != nullptr ? size_t(T / per) + B + 1 : size_t(B) * ((T + per - 1) / per);
}

// Few heads over long sequences leave most of the CUs idle, so their chunks are cut into
// `count` segments: a segment's tokens map the state in front of them affinely, S -> M S +
// N (S [d_k, d_v]; N from the zero state, M from the unit matrix with v = 0), all maps but
// the last segment's are formed at once, composed in order, and every segment then runs
// from its own state.
struct Segments {
    int count;
    size_t starts, maps, total;  // bytes: states in front of each segment, M of 1 .. count - 2
};
Segments segments_of(const kdn_delta_desc* d, bool packed, int group);
// The states in front of all segments, in a.starts, from a.S0; sets a.segs and the pointers
hipError_t launch_segments(ForwardArgs& a, const Segments& s, void* ws, int dtype, int dk, hipStream_t st);

// states[g + 1] += M_g states[g] for g = 1 .. segs - 2, or, backward, states[g - 1] +=
// M_g^T states[g] for g = segs - 2 .. 1 (a state of all heads each)
hipError_t launch_compose(int heads, int dv, int dk, int segs, const float* maps, float* states, bool backward, hipStream_t st);

kdn_status check(const kdn_delta_desc* d, bool one_token);
hipError_t launch_forward(const ForwardArgs& a, int dtype, int dk, bool keep, hipStream_t st);
hipError_t launch_states(size_t n, const float* in, float* out, hipStream_t st);

}  // namespace delta
}  // namespace kdn
