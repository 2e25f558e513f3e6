// kdn_gated.hip -- the gated linear recurrence h_t = a_t h_{t-1} + x_t, each
// channel on its own, over [B, H, T, d]; its backward; one step of it.
//
// The token maps h -> a h + x compose associatively, like the Moebius maps of
// the precision recurrence:  (A2, X2) after (A1, X1) is (A2 A1, A2 X1 + X2).
//
// Backward: with m_t = a_t (dh_t + m_{t+1}) and m behind the last token the
// gradient of h_T,
//   dx_t = dh_t + m_{t+1},   da_t = dx_t h_{t-1},   dh_0 = m_1,
// the same kind of recurrence, run from the last token to the first.
//
// Both are bound by HBM: the inputs are read once, the outputs written once.
// A workgroup holds a tile of TG x L tokens and LANES x 8 channels in registers:
// thread (tg, lane) has L consecutive tokens of 8 channels, packed as they were
// loaded.  It folds them into one map, the TG maps of a channel are folded in
// LDS, and once the tile's incoming state is known each thread replays its
// tokens from its own start.
//
// Many (sequence, channel block) pairs: a workgroup walks along its sequence and
// the state stays with it.  Few: a workgroup per tile (CHAIN), and the state
// travels between them through the workspace.  A tile publishes its map as soon
// as it has it, and 16 tiles form a group: a tile folds the maps of its group
// before it, in order, and applies them to the state at the group's start, which
// the last tile of the group before publishes; so the chain is T / (16 tile)
// steps long.  The walk folds its tiles in the same groups, so the bracketing is fixed by
// T, d and the types: a sequence gives the same bits alone and in any batch.  A workgroup
// takes its tile from a counter, in an order in which a tile
// comes after everything it waits for: whoever holds an earlier tile is already
// running and waits for earlier tiles only, so every wait ends.
// The rule: the walk where it has two tiles at most, where the pairs are 1024 or more, four
// to a CU, and where they leave few of the 256 CUs idle in their last round: a tile is
// 200 KB, 10 us of a CU's share of the memory's time, and the chain's clearing and waits
// cost 6 us, 0.6 of that, so the walk is ahead up to 160 idle CU tiles.  (us, with walk and
// chain: 256 x 300 x 128 bfloat16 14.6, 21.3, x 4000 142, 144, the backward in float32 564,
// 627; 215 x 335 x 128 float32 28.4, 34.5; 16 x 200 x 128 float32 backward, two tiles, 10.1,
// 13.6; but 406 pairs of 826 tokens in float32 123, 106, 64 x 1000 x 128 bfloat16 24.3,
// 16.5.)  B1 H16 T65536 d128 bfloat16, a chain, runs at 5.2 TB/s in 154 us with its 5.5 us
// of clearing; the backward of B8 H16 T4096 takes 188 us, 5.0 TB/s.  16 x 16384 x 128, a
// chain: float32 94.5 us (4.3 TB/s), x bfloat16 and a float32 67 (4.0), x float32 and a
// bfloat16 78 (4.3); the backward 146 (4.6; as a chain 256 and 16 registers, one wave per
// SIMD, where the walk's 240 leave two), 106 and 119 (5.1).  Few channels wait for the
// chain: 500000 x 32 bfloat16 39 us (2.4 TB/s), 31 groups one after the other; a block of
// channels that is not full leaves lanes idle: 9 x 6521 x 200 bfloat16, 72 of 128 channels
// in the second block, 26 us (2.7 TB/s).
// A published word is one atomic access whose value cannot be the mark "not yet
// there" (all bits set), so it needs no flag and no fence.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kdn.h"
#include "kdn_quant.h"

namespace {

using kdn::bf16_t;

constexpr int kThreads = 256;
// tiles per group of the chain (8: 500000 tokens of 32 channels bfloat16 take 55 us and
// 100 backward, against 41 and 75; 32: 39 and 69, but B1 H16 T65536 d128 144 -> 177)
constexpr int kGroup = 16;
constexpr int kMaxGroups = (1 << 24) - 1;  // a grid holds fewer than 2^32 threads
constexpr uint32_t kNotYet = 0xffffffffu;
constexpr uint32_t kNaN = 0x7fc00000u;

// 8 channels as loaded: 4 or 8 words
template <typename E> struct Vec8 {
    kdn::u32x4 u[sizeof(E) / 2];
    // (non-temporal: nothing is read twice.  B1 H16 T65536 d128 bfloat16 159 -> 141 us,
    // the backward of B8 H16 T4096 d128 204 -> 190 us; non-temporal stores take the
    // backward to 289 us)
    __device__ __forceinline__ void load(const E* p) {
#pragma unroll
        for (int i = 0; i < int(sizeof(E) / 2); ++i)
            u[i] = __builtin_nontemporal_load(reinterpret_cast<const kdn::u32x4*>(p) + i);
    }
    __device__ __forceinline__ void fill(float x) {
        const uint32_t b = __float_as_uint(x);
        const uint32_t w = sizeof(E) == 4 ? b : (b & 0xffff0000u) | (b >> 16);
#pragma unroll
        for (int i = 0; i < int(sizeof(E) / 2); ++i) u[i] = kdn::u32x4{w, w, w, w};
    }
    // makes the compiler unpack the words anew behind this point, instead of
    // keeping the floats of the first use (twice the registers in bfloat16)
    __device__ __forceinline__ void fresh() {
#pragma unroll
        for (int i = 0; i < int(sizeof(E) / 2); ++i) asm volatile("" : "+v"(u[i]));
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(E) == 4) return __uint_as_float(u[i / 4][i % 4]);
        const uint32_t w = u[0][i / 2];
        return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    }
};

__device__ __forceinline__ void publish(uint64_t* p, float A, float X) {
    uint32_t a = __float_as_uint(A);
    if (a == kNotYet) a = kNaN;
    __hip_atomic_store(p, (uint64_t(a) << 32) | __float_as_uint(X), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish(uint32_t* p, float h) {
    uint32_t b = __float_as_uint(h);
    if (b == kNotYet) b = kNaN;
    __hip_atomic_store(p, b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename W> __device__ __forceinline__ W peek(const W* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

struct Chain {
    uint64_t* agg;    // [sequence][tile][d]: the tile's map (A, X)
    uint32_t* start;  // [sequence][group][d]: the state at the group's start
    uint32_t* ticket;
};

struct ScanArgs {
    int seqs, T, d, nt, nblk;  // nt tiles along T, nblk channel blocks
    const void *a, *x, *h;  // forward: a, x; backward: a, dh (as x), h
    const float* first;     // the state that enters: h0, or the gradient of h_T; may be NULL
    const float* h0;        // backward: h before the first token; may be NULL
    void* out;              // h
    float *dx, *da;
    float* last;            // the state that leaves: h_T, or dh0; may be NULL
    Chain chain;
};

// The state that enters tile j > 0 of a chain, for one channel.
__device__ __forceinline__ float chain_wait(const Chain& c, size_t seq, int nt, int ng, int d, int j,
                                            int ch) {
    const int g = j / kGroup, j0 = g * kGroup;
    float A = 1.f, X = 0.f;
    const uint64_t* p = c.agg + (seq * nt + j0) * d + ch;
    uint64_t w[kGroup - 1];
#pragma unroll
    for (int i = 0; i < kGroup - 1; ++i) w[i] = j0 + i < j ? peek(p + size_t(i) * d) : 0;
#pragma unroll
    for (int i = 0; i < kGroup - 1; ++i) {
        if (j0 + i < j) {
            while (w[i] == ~uint64_t(0)) {
                __builtin_amdgcn_s_sleep(1);
                w[i] = peek(p + size_t(i) * d);
            }
            const float At = __uint_as_float(uint32_t(w[i] >> 32));
            X = fmaf(At, X, __uint_as_float(uint32_t(w[i])));
            A *= At;
        }
    }
    const uint32_t* s = c.start + (seq * ng + g) * d + ch;
    uint32_t b = peek(s);
    while (b == kNotYet) {
        __builtin_amdgcn_s_sleep(1);
        b = peek(s);
    }
    const float h = __uint_as_float(b);
    return j == j0 ? h : fmaf(A, h, X);
}

template <typename Ex, typename Ea, int LANES, int L, bool BWD, bool CHAIN>
__global__ __launch_bounds__(kThreads) void gated_kernel(ScanArgs p) {
    constexpr int TG = kThreads / LANES, CB = LANES * 8, TT = TG * L;
    __shared__ __attribute__((aligned(16))) float mA[TG][CB], mX[TG][CB];
    __shared__ float hin[CB];
    __shared__ uint32_t my_ticket;
    const int tid = threadIdx.x, lane = tid % LANES, tg = tid / LANES;
    const Ea* pa = static_cast<const Ea*>(p.a);
    const Ex* px = static_cast<const Ex*>(p.x);
    const Ex* ph = static_cast<const Ex*>(p.h);
    uint32_t id = blockIdx.x;
    int j0 = 0, j1 = p.nt;
    if constexpr (CHAIN) {
        if (tid == 0)
            my_ticket = __hip_atomic_fetch_add(p.chain.ticket, 1u, __ATOMIC_RELAXED,
                                               __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        const uint32_t n = uint32_t(p.seqs) * p.nblk, k = my_ticket;
        j0 = int(k / n);
        j1 = j0 + 1;
        id = k - uint32_t(j0) * n;
    }
    const size_t seq = id / uint32_t(p.nblk);
    const int c0 = int(id % uint32_t(p.nblk)) * CB, c = c0 + 8 * lane;
    const bool in = c < p.d;
    const int ng = (p.nt + kGroup - 1) / kGroup;
    // the thread that carries channel c0 + tid between tiles
    const bool carrier = tid < CB && c0 + tid < p.d;
    float state = 0.f;  // enters the tile
    // walk: the state at the start of its group of tiles, and the map of the group so far
    float start = 0.f, gA = 1.f, gX = 0.f;
    if (carrier && j0 == 0) {
        if (p.first != nullptr) start = p.first[seq * p.d + c0 + tid];
        state = start;
        // read by tile 0 alone and passed on from there, so that the state that
        // leaves may be written over it
        if constexpr (CHAIN) publish(p.chain.start + seq * ng * p.d + c0 + tid, start);
    }

    for (int j = j0; j < j1; ++j) {
        const int tile = BWD ? p.nt - 1 - j : j;
        const int t0 = tile * TT + tg * L;  // (T + TT fits: T <= 2^30)
        const size_t base = (seq * p.T + t0) * p.d + c;
        Vec8<Ea> a[L];
        Vec8<Ex> x[L], h[BWD ? L : 1];
#pragma unroll
        for (int l = 0; l < L; ++l) {
            if (in && t0 + l < p.T) {
                a[l].load(pa + base + size_t(l) * p.d);
                x[l].load(px + base + size_t(l) * p.d);
                if constexpr (BWD) {
                    // the state before the token (token 0 has h0 instead, below)
                    if (t0 + l > 0) h[l].load(ph + base + size_t(l) * p.d - p.d);
                    else h[l].fill(0.f);
                }
            } else {  // a token that changes nothing
                a[l].fill(1.f);
                x[l].fill(0.f);
                if constexpr (BWD) h[l].fill(0.f);
            }
        }
        // this thread's map
        float A[8], X[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            A[i] = 1.f;
            X[i] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < L; ++k) {
            const int l = BWD ? L - 1 - k : k;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float al = a[l].get(i);
                X[i] = BWD ? al * (x[l].get(i) + X[i]) : fmaf(al, X[i], x[l].get(i));
                A[i] *= al;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            *reinterpret_cast<kdn::floatx4*>(&mA[tg][8 * lane + i]) =
                kdn::floatx4{A[i], A[i + 1], A[i + 2], A[i + 3]};
            *reinterpret_cast<kdn::floatx4*>(&mX[tg][8 * lane + i]) =
                kdn::floatx4{X[i], X[i + 1], X[i + 2], X[i + 3]};
        }
#pragma unroll
        for (int l = 0; l < L; ++l) {
            a[l].fresh();
            x[l].fresh();
        }
        __syncthreads();
        // the maps of a channel, folded in order; each leaves what lies before it
        if (tid < CB) {
            float PA = 1.f, PX = 0.f;
#pragma unroll 8
            for (int k = 0; k < TG; ++k) {
                const int g = BWD ? TG - 1 - k : k;
                const float At = mA[g][tid], Xt = mX[g][tid];
                mA[g][tid] = PA;
                mX[g][tid] = PX;
                PX = fmaf(At, PX, Xt);
                PA *= At;
            }
            if (carrier) {
                if constexpr (CHAIN) {
                    const int ch = c0 + tid;
                    publish(p.chain.agg + (seq * p.nt + j) * p.d + ch, PA, PX);
                    if (j > 0) state = chain_wait(p.chain, seq, p.nt, ng, p.d, j, ch);
                    if (j % kGroup == kGroup - 1 && j + 1 < p.nt)
                        publish(p.chain.start + (seq * ng + j / kGroup + 1) * p.d + ch,
                                fmaf(PA, state, PX));
                } else {
                    // as chain_wait folds them
                    state = j % kGroup == 0 ? start : fmaf(gA, start, gX);
                    gX = fmaf(PA, gX, PX);
                    gA *= PA;
                    if (j % kGroup == kGroup - 1) {
                        start = fmaf(PA, state, PX);
                        gA = 1.f;
                        gX = 0.f;
                    }
                }
                hin[tid] = state;
            }
        }
        __syncthreads();
        if (in) {
            float m[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                m[i] = fmaf(mA[tg][8 * lane + i], hin[8 * lane + i], mX[tg][8 * lane + i]);
#pragma unroll
            for (int k = 0; k < L; ++k) {
                const int l = BWD ? L - 1 - k : k;
                const size_t o = base + size_t(l) * p.d;
                if constexpr (!BWD) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) m[i] = fmaf(a[l].get(i), m[i], x[l].get(i));
                    if (t0 + l < p.T) kdn::store8<Ex>(static_cast<Ex*>(p.out) + o, m);
                } else {
                    float g[8], da[8];
                    float before[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) before[i] = h[l].get(i);
                    if (t0 + l == 0 && p.h0 != nullptr)
                        kdn::load_vec<float, 8>(p.h0 + seq * p.d + c, before);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        g[i] = x[l].get(i) + m[i];
                        da[i] = g[i] * before[i];
                        m[i] = a[l].get(i) * g[i];
                    }
                    if (t0 + l < p.T) {
                        kdn::store8<float>(p.dx + o, g);
                        kdn::store8<float>(p.da + o, da);
                    }
                }
            }
            // the state that leaves, as the thread of the last token has it (tokens
            // behind T leave m as it is): h_T is h of that token, bit for bit
            const int t_last = BWD ? 0 : p.T - 1;
            if (p.last != nullptr && t0 <= t_last && t_last < t0 + L)
                kdn::store8<float>(p.last + seq * p.d + c, m);
        }
        if constexpr (!CHAIN) __syncthreads();  // the maps are free for the next tile
    }
}

// marks every word of the chain "not yet there" and sets the counter to 0 (its
// word is the last one).  A kernel and not a memset: the call may be captured
// into a graph, whose replays have to clear it again.
__global__ __launch_bounds__(kThreads) void chain_clear_kernel(uint32_t* ws, size_t words) {
    const size_t n4 = words / 4;
    const size_t step = size_t(gridDim.x) * kThreads;
    for (size_t i = size_t(blockIdx.x) * kThreads + threadIdx.x; i < n4; i += step)
        reinterpret_cast<kdn::u32x4*>(ws)[i] =
            kdn::u32x4{kNotYet, kNotYet, kNotYet, i == n4 - 1 ? 0u : kNotYet};
}

// no tokens: the state passes through
__global__ __launch_bounds__(kThreads) void state_copy_kernel(size_t n, const float* in, float* out) {
    const size_t i = size_t(blockIdx.x) * kThreads + threadIdx.x;
    if (i < n) out[i] = in != nullptr ? in[i] : 0.f;
}

// one token in place, 8 channels per thread: 256 x 16 x 128 takes 2.5 us, a launch and
// one round of loads
template <typename Ex, typename Ea>
__global__ __launch_bounds__(kThreads) void gated_step_kernel(
    uint32_t n, uint32_t per_seq, int n_slots, const int32_t* __restrict__ slot,
    const Ex* __restrict__ x, const Ea* __restrict__ a, float* __restrict__ h, Ex* __restrict__ o) {
    const uint32_t v = blockIdx.x * kThreads + threadIdx.x;
    if (v >= n) return;
    const uint32_t seq = v / per_seq, r = v - seq * per_seq;
    size_t at = v;
    if (slot != nullptr) {
        const int s = slot[seq];
        if (s < 0 || s >= n_slots) return;
        at = size_t(s) * per_seq + r;
    }
    float xv[8], av[8], hv[8];
    kdn::load_vec<Ex, 8>(x + size_t(v) * 8, xv);
    kdn::load_vec<Ea, 8>(a + size_t(v) * 8, av);
    kdn::load_vec<float, 8>(h + at * 8, hv);
#pragma unroll
    for (int i = 0; i < 8; ++i) hv[i] = fmaf(av[i], hv[i], xv[i]);
    kdn::store8<float>(h + at * 8, hv);
    kdn::store8<Ex>(o + size_t(v) * 8, hv);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool type_ok(int t) { return t == KDN_F32 || t == KDN_BF16; }

// Lanes across the channels of a tile (8 channels each): the whole head where it
// fits, so that little of the tile is idle.
int lanes_of(int d) { return d <= 32 ? 4 : d <= 64 ? 8 : 16; }

// Tokens per thread: what two (backward: three) packed inputs leave room for.
constexpr int strip(bool f32, bool bwd) { return f32 || bwd ? 8 : 16; }

struct Plan {
    int seqs, lanes, L, tile, nt, nblk;
    bool chain;
    size_t start, total;  // byte offsets in the workspace; total 16 without a chain
};

Plan plan_of(const kdn_scan_desc* s, bool bwd) {
    Plan p{};
    p.seqs = s->B * s->H;
    p.lanes = lanes_of(s->d);
    p.L = strip(s->dtype == KDN_F32 || s->gate_dtype == KDN_F32, bwd);
    p.tile = kThreads / p.lanes * p.L;
    p.nt = int((int64_t(s->T) + p.tile - 1) / p.tile);
    p.nblk = (s->d + 8 * p.lanes - 1) / (8 * p.lanes);
    const int64_t pairs = int64_t(p.seqs) * p.nblk, idle = (256 - pairs % 256) % 256;
    p.chain = p.nt > 2 && pairs < 1024 && p.nt * idle > 160;
    p.total = 16;
    if (p.chain) {
        const size_t ng = (p.nt + kGroup - 1) / kGroup;
        p.start = size_t(p.seqs) * p.nt * s->d * 8;
        p.total = p.start + size_t(p.seqs) * ng * s->d * 4 + 16;  // (d is a multiple of 8)
    }
    return p;
}

kdn_status check_scan(const kdn_scan_desc* s) {
    if (!s) return KDN_ERR_NULL;
    if (s->B < 0 || s->H < 0 || s->T < 0 || s->d < 0) return KDN_ERR_SHAPE;
    if (!type_ok(s->dtype) || !type_ok(s->gate_dtype)) return KDN_ERR_UNSUPPORTED;
    if (s->d == 0 || s->d % 8 != 0 || s->d > (1 << 20) || s->T > (1 << 30)) return KDN_ERR_UNSUPPORTED;
    if (int64_t(s->B) * s->H > kMaxGroups) return KDN_ERR_UNSUPPORTED;
    return KDN_OK;
}

kdn_status check_grid(const kdn_scan_desc* s, const Plan& p) {
    const int64_t groups = int64_t(p.seqs) * p.nblk * (p.chain ? p.nt : 1);
    return groups > kMaxGroups ? KDN_ERR_UNSUPPORTED : KDN_OK;
}

template <typename Ex, typename Ea, int LANES, int L, bool BWD>
void launch_chain(const ScanArgs& a, bool chain, hipStream_t st) {
    const unsigned n = unsigned(a.seqs) * unsigned(a.nblk);
    if (chain) gated_kernel<Ex, Ea, LANES, L, BWD, true><<<n * unsigned(a.nt), kThreads, 0, st>>>(a);
    else gated_kernel<Ex, Ea, LANES, L, BWD, false><<<n, kThreads, 0, st>>>(a);
}

template <typename Ex, typename Ea, bool BWD>
void launch_lanes(const ScanArgs& a, const Plan& p, hipStream_t st) {
    constexpr int L = strip(sizeof(Ex) == 4 || sizeof(Ea) == 4, BWD);
    if (p.lanes == 4) launch_chain<Ex, Ea, 4, L, BWD>(a, p.chain, st);
    else if (p.lanes == 8) launch_chain<Ex, Ea, 8, L, BWD>(a, p.chain, st);
    else launch_chain<Ex, Ea, 16, L, BWD>(a, p.chain, st);
}

template <bool BWD>
kdn_status launch_scan(const kdn_scan_desc* s, ScanArgs a, const Plan& p, void* ws, hipStream_t st) {
    a.seqs = p.seqs;
    a.T = s->T;
    a.d = s->d;
    a.nt = p.nt;
    a.nblk = p.nblk;
    if (p.chain) {
        char* w = static_cast<char*>(ws);
        a.chain = Chain{reinterpret_cast<uint64_t*>(w), reinterpret_cast<uint32_t*>(w + p.start),
                        reinterpret_cast<uint32_t*>(w + p.total - 4)};
        const size_t words = p.total / 4;
        const unsigned g = unsigned(std::min<size_t>((words / 4 + kThreads - 1) / kThreads, 2048));
        chain_clear_kernel<<<g, kThreads, 0, st>>>(static_cast<uint32_t*>(ws), words);
        if (hipGetLastError() != hipSuccess) return KDN_ERR_HIP;
    }
    const bool xf = s->dtype == KDN_F32, af = s->gate_dtype == KDN_F32;
    if (xf && af) launch_lanes<float, float, BWD>(a, p, st);
    else if (xf) launch_lanes<float, bf16_t, BWD>(a, p, st);
    else if (af) launch_lanes<bf16_t, float, BWD>(a, p, st);
    else launch_lanes<bf16_t, bf16_t, BWD>(a, p, st);
    return hipGetLastError() == hipSuccess ? KDN_OK : KDN_ERR_HIP;
}

kdn_status pass_through(const kdn_scan_desc* s, const float* in, float* out, hipStream_t st) {
    const size_t n = size_t(s->B) * s->H * s->d;
    if (out == nullptr || out == in) return KDN_OK;
    if (n > size_t(kMaxGroups) * kThreads) return KDN_ERR_UNSUPPORTED;
    state_copy_kernel<<<unsigned((n + kThreads - 1) / kThreads), kThreads, 0, st>>>(n, in, out);
    return hipGetLastError() == hipSuccess ? KDN_OK : KDN_ERR_HIP;
}

size_t scan_ws(const kdn_scan_desc* s, bool bwd) {
    if (check_scan(s) != KDN_OK) return 0;
    const Plan p = plan_of(s, bwd);
    return check_grid(s, p) == KDN_OK ? p.total : 0;
}

}  // namespace

extern "C" {

size_t kdn_gated_scan_workspace_bytes(const kdn_scan_desc* s) { return scan_ws(s, false); }
size_t kdn_gated_scan_backward_workspace_bytes(const kdn_scan_desc* s) { return scan_ws(s, true); }

kdn_status kdn_gated_scan(const kdn_scan_desc* s, const void* x, const void* a, const float* h0,
                          void* h, float* h_T, void* ws, size_t ws_bytes, void* stream) {
    kdn_status st = check_scan(s);
    if (st != KDN_OK) return st;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    const Plan p = plan_of(s, false);
    if ((st = check_grid(s, p)) != KDN_OK) return st;
    if (p.seqs == 0) return KDN_OK;
    for (const void* q : {x, a, (const void*)h0, (const void*)h, (const void*)h_T, (const void*)ws})
        if (!aligned16(q)) return KDN_ERR_ALIGN;
    if (s->T == 0) return pass_through(s, h0, h_T, hs);
    if (!x || !a || !h || (p.chain && !ws)) return KDN_ERR_NULL;
    if (p.chain && ws_bytes < p.total) return KDN_ERR_WORKSPACE;
    ScanArgs g{};
    g.a = a;
    g.x = x;
    g.first = h0;
    g.out = h;
    g.last = h_T;
    return launch_scan<false>(s, g, p, ws, hs);
}

kdn_status kdn_gated_scan_backward(const kdn_scan_desc* s, const void* a, const void* h,
                                   const float* h0, const void* dh, const float* dh_T, float* dx,
                                   float* da, float* dh0, void* ws, size_t ws_bytes, void* stream) {
    kdn_status st = check_scan(s);
    if (st != KDN_OK) return st;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    const Plan p = plan_of(s, true);
    if ((st = check_grid(s, p)) != KDN_OK) return st;
    if (p.seqs == 0) return KDN_OK;
    for (const void* q : {a, h, (const void*)h0, dh, (const void*)dh_T, (const void*)dx,
                          (const void*)da, (const void*)dh0, (const void*)ws})
        if (!aligned16(q)) return KDN_ERR_ALIGN;
    if (s->T == 0) return pass_through(s, dh_T, dh0, hs);
    if (!a || !h || !dh || !dx || !da || (p.chain && !ws)) return KDN_ERR_NULL;
    if (p.chain && ws_bytes < p.total) return KDN_ERR_WORKSPACE;
    ScanArgs g{};
    g.a = a;
    g.x = dh;
    g.h = h;
    g.h0 = h0;
    g.first = dh_T;
    g.dx = dx;
    g.da = da;
    g.last = dh0;
    return launch_scan<true>(s, g, p, ws, hs);
}

kdn_status kdn_gated_scan_step(const kdn_scan_desc* s, const void* x, const void* a, float* h,
                               const int32_t* slot, int32_t n_slots, void* o, void* stream) {
    const kdn_status st = check_scan(s);
    if (st != KDN_OK) return st;
    if (n_slots < 0) return KDN_ERR_SHAPE;
    const int64_t vecs = int64_t(s->B) * s->H * (s->d / 8);
    if (vecs > int64_t(kMaxGroups) * kThreads) return KDN_ERR_UNSUPPORTED;
    if (vecs == 0) return KDN_OK;
    if (!x || !a || !h || !o) return KDN_ERR_NULL;
    for (const void* q : {x, a, (const void*)h, (const void*)o})
        if (!aligned16(q)) return KDN_ERR_ALIGN;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    const unsigned grid = unsigned((vecs + kThreads - 1) / kThreads);
    const uint32_t n = uint32_t(vecs), per = uint32_t(s->H) * uint32_t(s->d / 8);
    auto go = [&](auto ex, auto ea) {
        using Ex = decltype(ex);
        using Ea = decltype(ea);
        gated_step_kernel<Ex, Ea><<<grid, kThreads, 0, hs>>>(
            n, per, n_slots, slot, static_cast<const Ex*>(x), static_cast<const Ea*>(a), h,
            static_cast<Ex*>(o));
    };
    const bool xf = s->dtype == KDN_F32, af = s->gate_dtype == KDN_F32;
    if (xf && af) go(float{}, float{});
    else if (xf) go(float{}, bf16_t{});
    else if (af) go(bf16_t{}, float{});
    else go(bf16_t{}, bf16_t{});
    return hipGetLastError() == hipSuccess ? KDN_OK : KDN_ERR_HIP;
}

}  // extern "C"
