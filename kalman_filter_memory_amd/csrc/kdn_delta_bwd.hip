// kdn_delta_bwd.hip -- gradients of the gated delta rule.
//
// For <dO, o> + <dS_T, S_T>, per chunk (kdn_delta.h), with D the gradient of the state
// behind it, S the state before it, U = beta E, P = scale tril(Q K^T Gamma):
//   X  = T^T ((gamma_C / gamma) K D + P^T dO),   T = (I + diag(beta) L)^-1
//   dV = beta X,  dbeta = rows of X . E
//   D <- gamma_C D + Q^T (scale gamma dO) - K^T (gamma dV)
//   dP = scale dO U^T Gamma (lower triangle), M = -dV U^T Gamma (strictly lower)
//   dQ = scale gamma dO S + dP K
//   dK = dP^T Q + M K + M^T K + (gamma_C / gamma) U D - gamma dV S
// and of the decays: token t's scales every path that crosses it,
//   dg_t = gamma_C <D, S> + sum_{t' >= t} A_t' + sum_{s < t} B_s + sum_{s < t <= t'} W_t's,
//   A_t = gamma_t (scale q_t S dO_t - k_t S dV_t),  B_s = (gamma_C / gamma_s) k_s D u_s,
//   W = dP (Q K^T) + M (K K^T) element by element,
// the last by sums over W's rows and columns: both see the same numbers, so a rounding of
// W_t's reaches the tokens between s and t' alone.
// Three kernels: the forward recurrence, which keeps E and states; the backward one
// (dV, dbeta, and D), over the chunks in reverse; and the rest, chunks in parallel.
#include "kdn_delta.h"
#include "kdn_delta_launch.h"

namespace kdn {
namespace delta {
namespace {

struct BackwardArgs {
    const void *q, *k, *g, *beta, *dO;
    const int32_t* cu;
    const float* dS_T;
    void *dq, *dk, *dv_out, *dg, *dbeta;
    float* dS0;
    const void *E, *S;  // kept by the forward recurrence
    void* D;            // gradients of the kept states' successors
    float* part;        // dbeta, a row for each 16 columns of d_v
    size_t rows;        // tokens of all heads of values
    int B, H, Hk, T, dv;
    int group;
    float scale;
    bool gate_bf16;
};

// ------------------------------------------------------------------ backward recurrence
template <typename E, int DK, int W> struct ReverseLds {
    using Cf = Cfg<E, DK, W>;
    bf16_t k[2][Cf::NP * C * DK], q[2][Cf::NP * C * DK];
    bf16_t d[2][Cf::NP * C * Cf::LDO];
    bf16_t t[2][3 * C * C], p[2][3 * C * C];
    float a[C * kLdA];
    float tmp[32 * kLdT];
    float gam[2][C], rest[2][C], beta[2][C];
    LogSum G[2][C];
    float gb[C];
};

template <typename E, int DK, int W>
__global__ __launch_bounds__((Cfg<E, DK, W>::kThreads)) void delta_reverse_kernel(BackwardArgs a) {
    using Cf = Cfg<E, DK, W>;
    constexpr int NP = Cf::NP, KT = Cf::KT, KS = Cf::KS, HT = 64 * Cf::NH;
    __shared__ __align__(16) ReverseLds<E, DK, W> L;

    const unsigned slices = unsigned(a.dv) / Cf::COLS;
    const unsigned id = xcd_order(blockIdx.x, gridDim.x);
    const int slice = int(id % slices), h = int(id / slices % unsigned(a.H)), b = int(id / slices / unsigned(a.H));
    const Seq sq = sequence(a.cu, b, h, a.H, a.Hk, a.T);
    const int nc = (sq.len + C - 1) / C;
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int col0 = slice * Cf::COLS;
    const size_t state = (size_t(b) * a.H + h) * size_t(a.dv) * DK;

    for (unsigned i = threadIdx.x; i < 2 * 3 * C * C / 8; i += Cf::kThreads)
        reinterpret_cast<u32x4*>(L.t)[i] = reinterpret_cast<u32x4*>(L.p)[i] = u32x4{0, 0, 0, 0};
    sync_lds();

    if (wave >= W) {
        const int ht = threadIdx.x - 64 * W, hw = wave - W;
        const E* q = static_cast<const E*>(a.q) + sq.rq * DK;
        const E* k = static_cast<const E*>(a.k) + sq.rq * DK;
        const E* dO = static_cast<const E*>(a.dO) + sq.rv * a.dv + col0;
        Stage<E, DK, HT> sk, sq_;
        Stage<E, Cf::COLS, HT> sd;
        float g = 0.f, be = 0.f;
        // chunk c of the sequence goes through buffer c & 1
        auto load = [&](int c) {
            const int t0 = c * C, rows = sq.len - t0;
            sk.load(k + size_t(t0) * DK, DK, rows, ht);
            sq_.load(q + size_t(t0) * DK, DK, rows, ht);
            sd.load(dO + size_t(t0) * a.dv, a.dv, rows, ht);
        };
        auto gates = [&](int c) {
            const int t = c * C + (lane & 31);
            g = t < sq.len ? load_gate(a.g, sq.rv + t, a.gate_bf16) : 0.f;
            be = t < sq.len ? load_gate(a.beta, sq.rv + t, a.gate_bf16) : 0.f;
        };
        auto put = [&](int c) {
            const int s = c & 1;
            auto rows_into = [&](bf16_t* x) {
                return [x](const Raw8<E>& r, int row, int p) {
                    const auto y = planes_of<E>(r);
#pragma unroll
                    for (int n = 0; n < NP; ++n)
                        *reinterpret_cast<bf16x8*>(x + n * C * DK + Cf::Tile::at(row, p)) = y.p[n];
                };
            };
            sk.each(ht, rows_into(L.k[s]));
            sq_.each(ht, rows_into(L.q[s]));
            sd.each(ht, [&](const Raw8<E>& r, int row, int p) {
                const auto y = planes_of<E>(r);
#pragma unroll
                for (int n = 0; n < NP; ++n)
                    *reinterpret_cast<bf16x8*>(L.d[s] + (n * C + row) * Cf::LDO + 8 * p) = y.p[n];
            });
        };
        auto prepare = [&](int c) {
            const int s = c & 1;
            const LogSum G = log_sums<C>(g, lane);
            if (hw == 0) {
                if (lane < C) {
                    L.G[0][lane] = G;
                    L.gb[lane] = be;
                }
                wave_lds_fence();
                system_of<Cf, true>(L.k[s], L.G[0], L.gb, L.a, lane);
                wave_lds_fence();
                invert<true>(L.a, L.tmp, L.t[s], lane);
            } else if (hw == 1) {
                const LogSum last = {lane_value(G.hi, 31), lane_value(G.lo, 31)};
                if (lane < C) {
                    L.G[1][lane] = G;
                    L.gam[s][lane] = decay_of(G);
                    L.rest[s][lane] = decay_between(last, G);
                    L.beta[s][lane] = be;
                }
                wave_lds_fence();
                readout_of<Cf, true, 3>(L.q[s], L.k[s], L.G[1], a.scale, C, L.p[s], lane);
            }
        };
        int c = nc - 1;
        if (nc > 0) {
            load(c);
            gates(c);
            put(c);
            if (nc > 1) load(c - 1);
        }
        sync_lds();
        if (nc > 0) prepare(c);
        if (nc > 1) {
            gates(c - 1);
            put(c - 1);
        }
        sync_lds();
        for (; c >= 0; --c) {
            if (c > 1) load(c - 2);
            if (c > 0) {
                prepare(c - 1);
                if (c > 1) gates(c - 2);
            }
            sync_lds();
            if (c > 1) put(c - 2);
            sync_lds();
        }
        return;
    }

    const int g = lane >> 4, m = lane & 15, col = col0 + 16 * wave + m;
    floatx4 st[KT];
    if (a.dS_T != nullptr) {
        load_state<KS>(st, a.dS_T + state, col, lane);
    } else {
#pragma unroll
        for (int i = 0; i < KT; ++i) st[i] = floatx4{0.f, 0.f, 0.f, 0.f};
    }
    const size_t groups = group_slot(a.cu, b, sq.start, a.group * C, (a.T + a.group * C - 1) / (a.group * C));
    const E* Ep = static_cast<const E*>(a.E) + sq.rv * a.dv + col;
    E* dV = static_cast<E*>(a.dv_out) + sq.rv * a.dv + col;
    float* part = a.part + size_t(col0 / 16 + wave) * a.rows + sq.rv;
    sync_lds();
    sync_lds();
    for (int c = nc - 1; c >= 0; --c) {
        const int s = c & 1, rows = sq.len - c * C;
        const size_t row0 = size_t(c) * C + 8 * g;
        if (c == nc - 1 || (c + 1) % a.group == 0)
            keep_state<E, KS>(st, static_cast<E*>(a.D) + ((groups + c / a.group) * a.H + h) * size_t(a.dv) * DK, col0 + 16 * wave, lane);
        float ev[8];  // E of this lane's tokens, 8 g + 0..7
#pragma unroll
        for (int e = 0; e < 8; ++e) ev[e] = 8 * g + e < rows ? to_f<E>(Ep[(row0 + e) * a.dv]) : 0.f;
        floatx4 kd[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int j = 0; j < KS; ++j) {
            const Planes<3> sp = state_planes<KT>(st, j);
#pragma unroll
            for (int x = 0; x < 2; ++x) kd[x] = product<2>(row_frag<Cf>(L.k[s], x, j, lane), sp, kd[x]);
        }
        Planes<NP> dp;  // dO, tokens along the contraction
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const bf16_t* x = L.d[s] + (n * C + 8 * g + (m >> 2)) * Cf::LDO + 16 * wave + 4 * (lane & 3);
            const short4x lo = read_tr16(x), hi = read_tr16(x + 4 * Cf::LDO);
            const short8x v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            dp.p[n] = __builtin_bit_cast(bf16x8, v);
        }
        float f[8], be[8], gam[8];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int t = 8 * g + 4 * x;
            const floatx4 rs = *reinterpret_cast<const floatx4*>(&L.rest[s][t]);
            const floatx4 bt = *reinterpret_cast<const floatx4*>(&L.beta[s][t]);
            const floatx4 gm = *reinterpret_cast<const floatx4*>(&L.gam[s][t]);
            floatx4 u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                u[e] = rs[e] * kd[x][e];
                be[4 * x + e] = bt[e];
                gam[4 * x + e] = gm[e];
            }
            u = product<2>(square_frag<3>(L.p[s], x, lane), dp, u);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[4 * x + e] = u[e];
        }
        const Planes<3> up = split8<3>(f);
        float y[8], z[8], db[8];
        float dof[8];
        join8<NP>(dp, dof);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const floatx4 xx = product<2>(square_frag<3>(L.t[s], x, lane), up, floatx4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 4 * x + e;
                const float w = be[i] * xx[e];
                db[i] = xx[e] * ev[i];
                if (8 * g + i < rows) dV[(row0 + i) * a.dv] = from_f<E>(w);
                y[i] = -gam[i] * w;
                z[i] = a.scale * gam[i] * dof[i];
            }
        }
        const Planes<3> yp = split8<3>(y), zp = split8<3>(z);
        const float last = L.gam[s][C - 1];
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            floatx4 w = {last * st[i][0], last * st[i][1], last * st[i][2], last * st[i][3]};
            w = product<2>(col_frag<Cf>(L.k[s], i / 2, i % 2, lane), yp, w);
            st[i] = product<2>(col_frag<Cf>(L.q[s], i / 2, i % 2, lane), zp, w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            db[i] = group_sum<16>(db[i]);
            if (m == i && 8 * g + i < rows) part[row0 + i] = db[i];
        }
        sync_lds();
        sync_lds();
    }
    if (a.dS0 != nullptr) store_state<KS>(st, a.dS0 + state, col, lane);
}

// ---------------------------------------------------------------------- bfloat16 inputs
// The backward recurrence with the chunks prepared ahead, as the forward one has them
// (kdn_delta.hip).  Interval i is at chunk nc - 1 - i; helper 3 copies the rows of interval
// i + 3 and sums the decays of i + 3, helper 2 forms P of i + 1, helpers 0 and 1 form the
// system of i + 2 and invert that of i + 1.
template <int DK, int DV> struct ReverseAheadLds {
    static constexpr int W = DV == 32 ? 2 : 4, COLS = 16 * W;
    bf16_t k[4][C * DK], q[4][C * DK];
    bf16_t d[4][C * COLS], e[4][C * COLS];  // dO, E
    bf16_t t[2][3 * C * C], p[2][3 * C * C];
    float a[2][C * kLdA];
    float tmp[2][32 * kLdT];
    // gam[.][31] is the whole chunk's decay; zg = scale gam, 0 behind the last token
    float gam[4][C], rest[4][C], beta[4][C], zg[4][C];
    LogSum G[4][C];
};

template <int DK, int DV>
__global__ __launch_bounds__(64 * (ReverseAheadLds<DK, DV>::W + 4)) void delta_reverse_ahead_kernel(BackwardArgs a) {
    using Lds = ReverseAheadLds<DK, DV>;
    constexpr int W = Lds::W, COLS = Lds::COLS;
    using Cf = Cfg<bf16_t, DK, W>;
    constexpr int KT = Cf::KT, KS = Cf::KS;
    __shared__ __align__(16) Lds L;

    constexpr unsigned slices = DV / COLS;
    const unsigned id = xcd_order(blockIdx.x, gridDim.x);
    const int slice = int(id % slices), h = int(id / slices % unsigned(a.H)), b = int(id / slices / unsigned(a.H));
    const Seq sq = sequence(a.cu, b, h, a.H, a.Hk, a.T);
    const int nc = (sq.len + C - 1) / C;
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int col0 = slice * COLS;
    const size_t state = (size_t(b) * a.H + h) * size_t(DV) * DK;

    for (unsigned i = threadIdx.x; i < 2 * 3 * C * C / 8; i += 64 * (W + 4))
        reinterpret_cast<u32x4*>(L.t)[i] = reinterpret_cast<u32x4*>(L.p)[i] = u32x4{0, 0, 0, 0};

    if (wave >= W) {
        const int hw = wave - W;
        if (hw == 3) {
            const bf16_t* q = static_cast<const bf16_t*>(a.q) + sq.rq * DK;
            const bf16_t* k = static_cast<const bf16_t*>(a.k) + sq.rq * DK;
            const bf16_t* d = static_cast<const bf16_t*>(a.dO) + sq.rv * DV + col0;
            const bf16_t* e = static_cast<const bf16_t*>(a.E) + sq.rv * DV + col0;
            const uint32_t lk = lds_address(L.k), lq = lds_address(L.q), ld = lds_address(L.d), le = lds_address(L.e);
            float g = 0.f, be = 0.f;
            auto gates = [&](int i) {
                const int t = (nc - 1 - i) * C + (lane & 31);
                g = t < sq.len ? load_gate(a.g, sq.rv + t, a.gate_bf16) : 0.f;
                be = t < sq.len ? load_gate(a.beta, sq.rv + t, a.gate_bf16) : 0.f;
            };
            auto copy = [&](int i) {
                const int c = nc - 1 - i, s = i & 3, rows = sq.len - c * C;
                copy_rows<DK, false>(k + size_t(c) * (C * DK), DK, rows, lk + s * (C * DK * 2), lane);
                copy_rows<DK, false>(q + size_t(c) * (C * DK), DK, rows, lq + s * (C * DK * 2), lane);
                copy_rows<COLS, true>(d + size_t(c) * (C * DV), DV, rows, ld + s * (C * COLS * 2), lane);
                copy_rows<COLS, true>(e + size_t(c) * (C * DV), DV, rows, le + s * (C * COLS * 2), lane);
            };
            auto sums = [&](int i) {
                const int s = i & 3;
                const LogSum G = log_sums<C>(g, lane);
                const LogSum last = {lane_value(G.hi, 31), lane_value(G.lo, 31)};
                if (lane < C) {
                    const float gm = decay_of(G);
                    L.G[s][lane] = G;
                    L.gam[s][lane] = gm;
                    L.rest[s][lane] = decay_between(last, G);
                    L.beta[s][lane] = be;
                    L.zg[s][lane] = (nc - 1 - i) * C + lane < sq.len ? a.scale * gm : 0.f;
                }
            };
            if (nc > 0) {
                gates(0);
                copy(0);
                sums(0);
                gates(1 < nc ? 1 : 0);
            }
            copies_done<0>();
            sync_lds();
            for (int i = -2; i < nc; ++i) {
                if (i + 3 < nc) {
                    sums(i + 3);
                    if (i + 4 < nc) gates(i + 4);
                    copy(i + 3);
                }
                copies_done<0>();
                sync_lds();
            }
        } else if (hw == 2) {
            sync_lds();
            for (int i = -2; i < nc; ++i) {
                const int n = i + 1;
                if (i >= -1 && n < nc)
                    readout_of<Cf, true, 3>(L.q[n & 3], L.k[n & 3], L.G[n & 3], a.scale, sq.len - (nc - 1 - n) * C,
                                            L.p[n & 1], lane);
                sync_lds();
            }
        } else {
            sync_lds();
            for (int i = -2; i < nc; ++i) {
                const int n = i + 2;
                if ((i & 1) == hw) {
                    if (n < nc) system_of<Cf, true>(L.k[n & 3], L.G[n & 3], L.beta[n & 3], L.a[hw], lane);
                } else if (i >= -1 && i + 1 < nc) {
                    invert<true>(L.a[hw], L.tmp[hw], L.t[(i + 1) & 1], lane);
                }
                sync_lds();
            }
        }
        return;
    }

    const int g = lane >> 4, m = lane & 15, col = col0 + 16 * wave + m;
    floatx4 st[KT];
    if (a.dS_T != nullptr) {
        load_state<KS>(st, a.dS_T + state, col, lane);
    } else {
#pragma unroll
        for (int i = 0; i < KT; ++i) st[i] = floatx4{0.f, 0.f, 0.f, 0.f};
    }
    const size_t groups = group_slot(a.cu, b, sq.start, a.group * C, (a.T + a.group * C - 1) / (a.group * C));
    bf16_t* dV = static_cast<bf16_t*>(a.dv_out) + sq.rv * DV + col0 + 16 * wave + 4 * g;
    float* part = a.part + size_t(col0 / 16 + wave) * a.rows + sq.rv;
    bf16x8 plus[2], minus[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        plus[x] = unit(lane, x);
        minus[x] = minus_unit(lane, x);
    }
    // what is left of a chunk when the state has gone on: rows of dV, and dbeta's part
    Planes<1> dv_left;
    float db[8];
    auto results = [&](int c, int rows) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
            if (rows >= C || paired_row(lane, x) < rows)
                put4(dV + (size_t(c) * C + paired_row(lane, x)) * DV, turned(dv_left, plus[x]));
        // sums over the 16 columns; lane m < 8 of a group takes token 8 g + m
#pragma unroll
        for (int i = 0; i < 8; ++i) db[i] = group_sum<16>(db[i]);
        float v = (m & 1) ? db[1] : db[0];
        v = (m & 6) == 2 ? ((m & 1) ? db[3] : db[2]) : v;
        v = (m & 6) == 4 ? ((m & 1) ? db[5] : db[4]) : v;
        v = (m & 6) == 6 ? ((m & 1) ? db[7] : db[6]) : v;
        if (m < 8 && 8 * g + m < rows) part[size_t(c) * C + 8 * g + m] = v;
    };
    sync_lds();
    sync_lds();
    sync_lds();
    Planes<1> kf[2][KS];
    auto fetch = [&](int s) {
#pragma unroll
        for (int j = 0; j < KS; ++j)
#pragma unroll
            for (int x = 0; x < 2; ++x) kf[x][j] = row_frag<Cf>(L.k[s], x, j, lane);
    };
    if (nc > 0) fetch(0);
    for (int i = 0; i < nc; ++i) {
        const int c = nc - 1 - i, s = i & 3;
        if (i == 0 || (c + 1) % a.group == 0)
            keep_state<bf16_t, KS>(st, static_cast<bf16_t*>(a.D) + ((groups + c / a.group) * a.H + h) * size_t(DV) * DK,
                                   col0 + 16 * wave, lane);
        const float last = L.gam[s][C - 1];
        Planes<1> dp;  // dO, tokens along the contraction
        {
            short4x w[2];
#pragma unroll
            for (int x = 0; x < 2; ++x)
                w[x] = read_tr16(L.d[s] + value_at<COLS>(8 * g + 4 * x + (m >> 2), 2 * wave + ((lane & 3) >> 1)) + 4 * (lane & 1));
            const short8x v = {w[0][0], w[0][1], w[0][2], w[0][3], w[1][0], w[1][1], w[1][2], w[1][3]};
            dp.p[0] = __builtin_bit_cast(bf16x8, v);
        }
        Planes<3> pf[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) pf[x] = square_frag<3>(L.p[i & 1], x, lane);
        float z[8];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const floatx4 w = *reinterpret_cast<const floatx4*>(&L.zg[s][8 * g + 4 * x]);
#pragma unroll
            for (int e = 0; e < 4; ++e) z[4 * x + e] = w[e];
        }
        // planes of D, K D, P^T dO
        floatx4 kd[2], pd[2], r1[KT];
        bf16x8 sp[KS];
#pragma unroll
        for (int x = 0; x < 2; ++x) kd[x] = pd[x] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < KS; ++j) {
            sp[j] = pack8(st[2 * j], st[2 * j + 1]);
#pragma unroll
            for (int x = 0; x < 2; ++x) r1[2 * j + x] = Mma<bf16_t>::mma(minus[x], sp[j], st[2 * j + x]);
#pragma unroll
            for (int x = 0; x < 2; ++x) kd[x] = Mma<bf16_t>::mma(kf[x][j].p[0], sp[j], kd[x]);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) pd[x] = product<2>(pf[x], dp, pd[x]);
        if (i > 0) results(c + 1, i == 1 ? sq.len - (nc - 1) * C : C);
#pragma unroll
        for (int j = 0; j < KS; ++j) {
            sp[j] = pack8(r1[2 * j], r1[2 * j + 1]);
#pragma unroll
            for (int x = 0; x < 2; ++x) r1[2 * j + x] = Mma<bf16_t>::mma(minus[x], sp[j], r1[2 * j + x]);
#pragma unroll
            for (int x = 0; x < 2; ++x) kd[x] = Mma<bf16_t>::mma(kf[x][j].p[0], sp[j], kd[x]);
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) st[2 * j + x][e] *= last;
        }
#pragma unroll
        for (int j = 0; j < KS; ++j) {
            const bf16x8 p2 = pack8(r1[2 * j], r1[2 * j + 1]);
#pragma unroll
            for (int x = 0; x < 2; ++x) kd[x] = Mma<bf16_t>::mma(kf[x][j].p[0], p2, kd[x]);
        }
        // D <- gamma_C D + Q^T (scale gamma dO), beside the way to X
        {
            float f[8];
            join8<1>(dp, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] *= f[e];
        }
        const Planes<3> zp = split8<3>(z);
        Planes<3> tf[2];
        float rest[8], be[8], gam[8], ev[8], f[8];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int t = 8 * g + 4 * x;
            tf[x] = square_frag<3>(L.t[i & 1], x, lane);
            const floatx4 rs = *reinterpret_cast<const floatx4*>(&L.rest[s][t]);
            const floatx4 bt = *reinterpret_cast<const floatx4*>(&L.beta[s][t]);
            const floatx4 gm = *reinterpret_cast<const floatx4*>(&L.gam[s][t]);
            const short4x w = read_tr16(L.e[s] + value_at<COLS>(t + (m >> 2), 2 * wave + ((lane & 3) >> 1)) + 4 * (lane & 1));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                rest[4 * x + e] = rs[e];
                be[4 * x + e] = bt[e];
                gam[4 * x + e] = gm[e];
                ev[4 * x + e] = bf2f(static_cast<bf16_t>(w[e]));
                f[4 * x + e] = fmaf(rest[4 * x + e], kd[x][e], pd[x][e]);
            }
        }
#pragma unroll
        for (int j = 0; j < KT; ++j) st[j] = product<2>(col_frag<Cf>(L.q[s], j / 2, j % 2, lane), zp, st[j]);
        // X = T^T dU
        const Planes<3> up = split8<3>(f);
        floatx4 xx[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) xx[x] = product<2>(tf[x], up, floatx4{0.f, 0.f, 0.f, 0.f});
        // D <- D - K^T (gamma dV)
        floatx4 w[2];
        float y[8];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int n = 4 * x + e;
                w[x][e] = be[n] * xx[x][e];
                y[n] = -gam[n] * w[x][e];
                db[n] = xx[x][e] * ev[n];
            }
        dv_left.p[0] = pack8(w[0], w[1]);
        const Planes<3> yp = split8<3>(y);
#pragma unroll
        for (int n = 0; n < 3; ++n)
#pragma unroll
            for (int j = 0; j < KT; ++j)
                st[j] = Mma<bf16_t>::mma(col_frag<Cf>(L.k[s], j / 2, j % 2, lane).p[0], yp.p[n], st[j]);
        if (i + 1 < nc) fetch((i + 1) & 3);
        sync_lds();
    }
    if (nc > 0) results(0, nc == 1 ? sq.len : C);
    if (a.dS0 != nullptr) store_state<KS>(st, a.dS0 + state, col, lane);
}

// -------------------------------------------------------------------------- gradients
// A workgroup takes one group of tokens of one head of queries and keys, and the heads of
// values that share it one after the other.  A wave holds 16 key dimensions of dQ and dK
// (in the order of paired_row) for all tokens of the group.
template <typename E, int DK, int DV> struct GradCfg {
    static constexpr int NP = sizeof(E) == 2 ? 1 : 3;
    static constexpr int G = sizeof(E) == 2 ? 64 : 32;  // tokens of a group
    static constexpr int NW = DK / 16, kThreads = 64 * NW;
    static constexpr int NJ = G / 32, NN = DV / 32;  // steps over the tokens, over d_v
    using KRow = Rows<DK>;
    using VRow = Rows<DV>;
    using MRow = Rows<G>;
};
template <typename E, int DK, int DV> struct GradLds {
    using Cf = GradCfg<E, DK, DV>;
    bf16_t q[Cf::NP * Cf::G * DK], k[Cf::NP * Cf::G * DK];
    bf16_t o[Cf::NP * Cf::G * DV], u[Cf::NP * Cf::G * DV], v[Cf::NP * Cf::G * DV];  // dO, U, dV
    bf16_t p[Cf::NP * Cf::G * Cf::G], m[Cf::NP * Cf::G * Cf::G];                    // dP and M, [s][t]
    LogSum sum[Cf::G];
    float gam[Cf::G], rest[Cf::G];
    float red[Cf::NW][Cf::G], ds[Cf::NW];
    float wr[Cf::G / 8][Cf::G], wc[Cf::G / 8][Cf::G];  // W's row and column sums by blocks, of dP's part and of M's
};

template <typename Row, int NP, int G, int D>
__device__ __forceinline__ Planes<NP> rows_at(const bf16_t* x, int row, int piece) {
    Planes<NP> r;
#pragma unroll
    for (int n = 0; n < NP; ++n) r.p[n] = Row::row(x + n * G * D, row, piece);
    return r;
}
template <typename Row, int NP, int G, int D>
__device__ __forceinline__ Planes<NP> cols_at(const bf16_t* x, int t0, int j, int h, int lane) {
    Planes<NP> r;
#pragma unroll
    for (int n = 0; n < NP; ++n) r.p[n] = Row::col(x + n * G * D, t0, j, h, lane);
    return r;
}

template <typename E, int DK, int DV>
__global__ __launch_bounds__((GradCfg<E, DK, DV>::kThreads)) void delta_grad_kernel(BackwardArgs a) {
    using Cf = GradCfg<E, DK, DV>;
    constexpr int NP = Cf::NP, G = Cf::G, NW = Cf::NW, NJ = Cf::NJ, NN = Cf::NN, LIM = NP - 1;
    __shared__ __align__(16) GradLds<E, DK, DV> L;
    const int lane = threadIdx.x & 63, wave = wave_id(), tid = threadIdx.x;
    const int g = lane >> 4, m = lane & 15;
    const int groups_T = (a.T + G - 1) / G;
    const unsigned id = xcd_order(blockIdx.x, gridDim.x);
    const int hk = int(id % unsigned(a.Hk)), slot = int(id / unsigned(a.Hk));
    // the sequence and its group
    int b = 0, gr = 0;
    if (a.cu == nullptr) {
        b = slot / groups_T;
        gr = slot - b * groups_T;
    } else {
        int lo = 0, hi = a.B - 1;  // the last sequence whose places begin at slot or before
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (min(max(a.cu[mid], 0), a.T) / G + mid <= slot) lo = mid;
            else hi = mid - 1;
        }
        b = lo;
        gr = slot - (min(max(a.cu[b], 0), a.T) / G + b);
    }
    const int r = a.H / a.Hk;
    const Seq s0 = sequence(a.cu, b, hk * r, a.H, a.Hk, a.T);
    const int t0 = gr * G, rows = s0.len - t0;
    if (gr < 0 || rows <= 0) return;
    const size_t rq = s0.rq + t0;
    const size_t place = group_slot(a.cu, b, s0.start, G, groups_T) + gr;

    // Q and K; zeros where dP and M are never written
    const E* qp = static_cast<const E*>(a.q) + rq * DK;
    const E* kp = static_cast<const E*>(a.k) + rq * DK;
    for (int e = tid; e < G * DK / 8; e += Cf::kThreads) {
        const int row = e / (DK / 8), p = e % (DK / 8);
        const auto x = planes_of<E>(load_raw8<E>(qp + size_t(row) * DK + 8 * p, row < rows));
        const auto y = planes_of<E>(load_raw8<E>(kp + size_t(row) * DK + 8 * p, row < rows));
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            *reinterpret_cast<bf16x8*>(L.q + n * G * DK + Cf::KRow::at(row, p)) = x.p[n];
            *reinterpret_cast<bf16x8*>(L.k + n * G * DK + Cf::KRow::at(row, p)) = y.p[n];
        }
    }
    for (int e = tid; e < NP * G * G / 8; e += Cf::kThreads)
        reinterpret_cast<u32x4*>(L.p)[e] = reinterpret_cast<u32x4*>(L.m)[e] = u32x4{0, 0, 0, 0};

    const int wj = wave >> 1, wh = wave & 1;  // this wave's key dimensions: 32 wj + paired_row(., wh)
    floatx4 dq[2 * NJ], dk[2 * NJ];
#pragma unroll
    for (int x = 0; x < 2 * NJ; ++x) dq[x] = dk[x] = floatx4{0.f, 0.f, 0.f, 0.f};

    for (int hv = 0; hv < r; ++hv) {
        const int h = hk * r + hv;
        const size_t rv = sequence(a.cu, b, h, a.H, a.Hk, a.T).rv + t0;
        const E* Sp = static_cast<const E*>(a.S) + (place * a.H + h) * size_t(DV) * DK;
        const E* Dp = static_cast<const E*>(a.D) + (place * a.H + h) * size_t(DV) * DK;
        __syncthreads();  // the tiles of the head before are done with
        if (wave == 0) {
            const bool in = lane < rows && lane < G;
            const LogSum x = log_sums<G>(in ? load_gate(a.g, rv + lane, a.gate_bf16) : 0.f, lane);
            const LogSum last = {lane_value(x.hi, G - 1), lane_value(x.lo, G - 1)};
            if (lane < G) {
                L.sum[lane] = x;
                L.gam[lane] = decay_of(x);
                L.rest[lane] = decay_between(last, x);
            }
        }
        constexpr int kPer = DV / 8;
        for (int e = tid; e < G * kPer; e += Cf::kThreads) {
            const int row = e / kPer, p = e % kPer;
            const size_t at = (rv + row) * DV + 8 * p;
            const bool ok = row < rows;
            const auto xo = planes_of<E>(load_raw8<E>(static_cast<const E*>(a.dO) + at, ok));
            const auto xv = planes_of<E>(load_raw8<E>(static_cast<const E*>(a.dv_out) + at, ok));
            const auto ee = planes_of<E>(load_raw8<E>(static_cast<const E*>(a.E) + at, ok));
            const float bt = ok ? load_gate(a.beta, rv + row, a.gate_bf16) : 0.f;
            float f[8];
            join8<NP>(ee, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= bt;
            const Planes<NP> xu = split8<NP>(f);
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                const int at2 = n * G * DV + Cf::VRow::at(row, p);
                *reinterpret_cast<bf16x8*>(L.o + at2) = xo.p[n];
                *reinterpret_cast<bf16x8*>(L.v + at2) = xv.p[n];
                *reinterpret_cast<bf16x8*>(L.u + at2) = xu.p[n];
            }
        }
        __syncthreads();
        // dP and M, blocks of 16 x 16 on and below the diagonal, dealt to the waves
        constexpr int NB = G / 16, NBLK = NB * (NB + 1) / 2, KSTEPS = DK / 32;
        for (int x = wave; x < 2 * NBLK; x += NW) {
            const bool is_p = x < NBLK;
            int y = is_p ? x : x - NBLK, bt = 0;
            while (y > bt) y -= ++bt;
            const int bs = y;
            floatx4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < NN; ++j)
                acc = product<LIM>(rows_at<typename Cf::VRow, NP, G, DV>(is_p ? L.o : L.v, 16 * bt + m, 4 * j + g),
                                   rows_at<typename Cf::VRow, NP, G, DV>(L.u, 16 * bs + m, 4 * j + g), acc);
            floatx4 qk = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < KSTEPS; ++j)
                qk = product<LIM>(rows_at<typename Cf::KRow, NP, G, DK>(is_p ? L.q : L.k, 16 * bt + m, 4 * j + g),
                                  rows_at<typename Cf::KRow, NP, G, DK>(L.k, 16 * bs + m, 4 * j + g), qk);
            const int s = 16 * bs + m, t = 16 * bt + 4 * g;  // (tokens behind the last have zeros in dO, dV and U)
            float f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool keep = is_p ? s <= t + e : s < t + e;
                f[e] = keep ? (is_p ? a.scale : -1.f) * acc[e] * decay_between(L.sum[t + e], L.sum[s]) : 0.f;
            }
            float col = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float w = f[e] * qk[e];
                col += w;
                const float row = group_sum<16>(w);
                if (m == e) L.wr[(is_p ? 0 : NB) + bs][t + e] = row;
            }
            col += __shfl_xor(col, 16, 64);
            col += __shfl_xor(col, 32, 64);
            if (g == 0) L.wc[(is_p ? 0 : NB) + bt][s] = col;
            uint2 w[NP];
            split4<NP>(f, w);
#pragma unroll
            for (int n = 0; n < NP; ++n)
                *reinterpret_cast<uint2*>((is_p ? L.p : L.m) + n * G * G + Cf::MRow::at(s, t >> 3) + (t & 7)) = w[n];
        }
        // dO S, dV S and U D
        floatx4 os[2 * NJ], vs[2 * NJ], ud[2 * NJ];
#pragma unroll
        for (int x = 0; x < 2 * NJ; ++x) os[x] = vs[x] = ud[x] = floatx4{0.f, 0.f, 0.f, 0.f};
        float along = 0.f;  // <D, S>
#pragma unroll
        for (int j = 0; j < NN; ++j) {
            const size_t at = size_t(j * (DK / 16) + wave) * 512 + lane * 8;
            const Planes<NP> sf = planes_of<E>(load_raw8<E>(Sp + at, true)), df = planes_of<E>(load_raw8<E>(Dp + at, true));
            float x8[8], y8[8];
            join8<NP>(sf, x8);
            join8<NP>(df, y8);
#pragma unroll
            for (int i = 0; i < 8; ++i) along = fmaf(x8[i], y8[i], along);
#pragma unroll
            for (int x = 0; x < 2 * NJ; ++x) {
                const int row = 32 * (x >> 1) + paired_row(lane, x & 1), pc = 4 * j + g;
                os[x] = product<LIM>(rows_at<typename Cf::VRow, NP, G, DV>(L.o, row, pc), sf, os[x]);
                vs[x] = product<LIM>(rows_at<typename Cf::VRow, NP, G, DV>(L.v, row, pc), sf, vs[x]);
                ud[x] = product<LIM>(rows_at<typename Cf::VRow, NP, G, DV>(L.u, row, pc), df, ud[x]);
            }
        }
        along *= L.gam[G - 1];
        __syncthreads();  // dP and M are there
        float qsum[8 * NJ];
#pragma unroll
        for (int jt = 0; jt < NJ; ++jt) {
            float qv[8], kv[8];
            join8<NP>(cols_at<typename Cf::KRow, NP, G, DK>(L.q, 32 * jt, wj, wh, lane), qv);
            join8<NP>(cols_at<typename Cf::KRow, NP, G, DK>(L.k, 32 * jt, wj, wh, lane), kv);
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int x = 2 * jt + hh;
                floatx4 aq, ak = dk[x];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 32 * jt + 8 * g + 4 * hh + e;
                    const float gm = L.gam[t], rs = L.rest[t];
                    aq[e] = a.scale * gm * os[x][e];
                    ak[e] += rs * ud[x][e] - gm * vs[x][e];
                    const float into = kv[4 * hh + e] * rs * ud[x][e];
                    along += into;
                    qsum[8 * jt + 4 * hh + e] = gm * (a.scale * qv[4 * hh + e] * os[x][e] - kv[4 * hh + e] * vs[x][e]) - into;
                }
#pragma unroll
                for (int js = 0; js < NJ; ++js) {
                    const Planes<NP> kf = cols_at<typename Cf::KRow, NP, G, DK>(L.k, 32 * js, wj, wh, lane);
                    if (js <= jt) {  // rows t, contraction over s
                        aq = product<LIM>(cols_at<typename Cf::MRow, NP, G, G>(L.p, 32 * js, jt, hh, lane), kf, aq);
                        ak = product<LIM>(cols_at<typename Cf::MRow, NP, G, G>(L.m, 32 * js, jt, hh, lane), kf, ak);
                    }
                    if (js >= jt) {  // rows s, contraction over t
                        const int row = 32 * jt + paired_row(lane, hh);
                        const Planes<NP> qf = cols_at<typename Cf::KRow, NP, G, DK>(L.q, 32 * js, wj, wh, lane);
                        ak = product<LIM>(rows_at<typename Cf::MRow, NP, G, G>(L.p, row, 4 * js + g), qf, ak);
                        ak = product<LIM>(rows_at<typename Cf::MRow, NP, G, G>(L.m, row, 4 * js + g), kf, ak);
                    }
                }
                dk[x] = ak;
#pragma unroll
                for (int e = 0; e < 4; ++e) dq[x][e] += aq[e];
            }
        }
#pragma unroll
        for (int i = 0; i < 8 * NJ; ++i) {
            const float s = group_sum<16>(qsum[i]);
            if (m == (i & 15)) L.red[wave][32 * (i >> 3) + 8 * g + (i & 7)] = s;
        }
        along = wave_sum(along);
        if (lane == 0) L.ds[wave] = along;
        __syncthreads();
        if (wave == 0) {
            float x = 0.f, ds = 0.f;
            if (lane < G) {
#pragma unroll
                for (int w = 0; w < NW; ++w) x += L.red[w][lane];
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    if (i <= lane / 16) x += L.wr[i][lane] + L.wr[NB + i][lane];
                    if (i >= lane / 16) x -= L.wc[i][lane] + L.wc[NB + i][lane];
                }
            }
#pragma unroll
            for (int w = 0; w < NW; ++w) ds += L.ds[w];
            // sums over the tokens from this one to the group's last
#pragma unroll
            for (int d = 1; d < G; d <<= 1) {
                const float y = __shfl_down(x, d, 64);
                x += lane + d < G ? y : 0.f;
            }
            if (lane < G && lane < rows) {
                float db = 0.f;
                for (int i = 0; i < DV / 16; ++i) db += a.part[size_t(i) * a.rows + rv + lane];
                static_cast<E*>(a.dg)[rv + lane] = from_f<E>(x + ds);
                static_cast<E*>(a.dbeta)[rv + lane] = from_f<E>(db);
            }
        }
    }
    const int d = 32 * wj + paired_row(lane, wh);
    E* dqp = static_cast<E*>(a.dq) + rq * DK + d;
    E* dkp = static_cast<E*>(a.dk) + rq * DK + d;
#pragma unroll
    for (int x = 0; x < 2 * NJ; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int t = 32 * (x >> 1) + 8 * g + 4 * (x & 1) + e;
            if (t < rows) {
                dqp[size_t(t) * DK] = from_f<E>(dq[x][e]);
                dkp[size_t(t) * DK] = from_f<E>(dk[x][e]);
            }
        }
}

// ---------------------------------------------------------------------------- launches
template <typename E, int DK, int DV> void backward_d(const BackwardArgs& a, size_t slots, hipStream_t st) {
    constexpr int W = DV == 32 ? 2 : 4;
    const unsigned n = unsigned(a.B) * unsigned(a.H) * unsigned(DV / (16 * W));
    if constexpr (sizeof(E) == 2) delta_reverse_ahead_kernel<DK, DV><<<n, 64 * (W + 4), 0, st>>>(a);
    else delta_reverse_kernel<E, DK, W><<<n, Cfg<E, DK, W>::kThreads, 0, st>>>(a);
    delta_grad_kernel<E, DK, DV><<<unsigned(slots * a.Hk), GradCfg<E, DK, DV>::kThreads, 0, st>>>(a);
}
template <typename E, int DK> void backward_k(const BackwardArgs& a, size_t slots, hipStream_t st) {
    if (a.dv == 32) backward_d<E, DK, 32>(a, slots, st);
    else if (a.dv == 64) backward_d<E, DK, 64>(a, slots, st);
    else backward_d<E, DK, 128>(a, slots, st);
}
template <typename E> void backward_e(const BackwardArgs& a, int dk, size_t slots, hipStream_t st) {
    if (dk == 32) backward_k<E, 32>(a, slots, st);
    else if (dk == 64) backward_k<E, 64>(a, slots, st);
    else backward_k<E, 128>(a, slots, st);
}

struct Layout {
    size_t E, S, D, part, total;
    size_t rows, slots;
};
Layout layout_of(const kdn_delta_desc* d, bool packed) {
    Layout l{};
    const size_t e = d->dtype == KDN_BF16 ? 2 : 4;
    const int32_t any = 0;
    l.rows = size_t(packed ? 1 : d->B) * d->H * d->T;
    l.slots = kept_slots(packed ? &any : nullptr, d->B, d->T, kept_chunks(d->dtype));
    auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
    l.S = up(l.rows * d->d_v * e);
    l.D = l.S + up(l.slots * d->H * d->d_v * d->d_k * e);
    l.part = l.D + up(l.slots * d->H * d->d_v * d->d_k * e);
    l.total = l.part + up(l.rows * (d->d_v / 16) * 4) + 16;
    return l;
}

// the gradient kernel's workgroups stay within a launch
kdn_status check_backward(const kdn_delta_desc* d, bool packed) {
    const kdn_status c = check(d, false);
    if (c != KDN_OK) return c;
    return layout_of(d, packed).slots * size_t(d->Hk) >= (size_t(1) << 23) ? KDN_ERR_UNSUPPORTED : KDN_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace delta
}  // namespace kdn

extern "C" {

size_t kdn_gated_delta_backward_workspace_bytes(const kdn_delta_desc* d, int32_t packed) {
    using namespace kdn::delta;
    return check_backward(d, packed != 0) == KDN_OK ? layout_of(d, packed != 0).total : 0;
}

kdn_status kdn_gated_delta_backward(const kdn_delta_desc* d, const int32_t* cu_seqlens, const void* q, const void* k,
                                    const void* v, const void* g, const void* beta, const float* S0, const void* dO,
                                    const float* dS_T, void* dq, void* dk, void* dv, void* dg, void* dbeta, float* dS0,
                                    void* ws, size_t ws_bytes, void* stream) {
    using namespace kdn::delta;
    const bool packed = cu_seqlens != nullptr;
    const kdn_status c = check_backward(d, packed);
    if (c != KDN_OK) return c;
    if (d->B == 0 || d->H == 0) return KDN_OK;
    for (const void* p : {q, k, v, (const void*)S0, dO, (const void*)dS_T, (const void*)dq, (const void*)dk,
                          (const void*)dv, (const void*)dS0, (const void*)ws})
        if (!aligned16(p)) return KDN_ERR_ALIGN;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (d->T == 0)
        return launch_states(size_t(d->B) * d->H * d->d_k * d->d_v, dS_T, dS0, st) == hipSuccess ? KDN_OK : KDN_ERR_HIP;
    if (!q || !k || !v || !g || !beta || !dO || !dq || !dk || !dv || !dg || !dbeta || !ws) return KDN_ERR_NULL;
    const Layout l = layout_of(d, packed);
    if (ws_bytes < l.total) return KDN_ERR_WORKSPACE;
    char* w = static_cast<char*>(ws);

    ForwardArgs f{};
    f.q = q;
    f.k = k;
    f.v = v;
    f.g = g;
    f.beta = beta;
    f.cu = cu_seqlens;
    f.S0 = S0;
    f.keep_E = w;
    f.keep_S = w + l.S;
    f.B = d->B;
    f.H = d->H;
    f.Hk = d->Hk;
    f.T = d->T;
    f.dv = d->d_v;
    f.group = kept_chunks(d->dtype);
    f.scale = d->scale;
    f.gate_bf16 = d->gate_dtype == KDN_BF16;
    if (launch_forward(f, d->dtype, d->d_k, true, st) != hipSuccess) return KDN_ERR_HIP;

    BackwardArgs a{};
    a.q = q;
    a.k = k;
    a.g = g;
    a.beta = beta;
    a.dO = dO;
    a.cu = cu_seqlens;
    a.dS_T = dS_T;
    a.dq = dq;
    a.dk = dk;
    a.dv_out = dv;
    a.dg = dg;
    a.dbeta = dbeta;
    a.dS0 = dS0;
    a.E = w;
    a.S = w + l.S;
    a.D = w + l.D;
    a.part = reinterpret_cast<float*>(w + l.part);
    a.rows = l.rows;
    a.B = d->B;
    a.H = d->H;
    a.Hk = d->Hk;
    a.T = d->T;
    a.dv = d->d_v;
    a.group = f.group;
    a.scale = d->scale;
    a.gate_bf16 = f.gate_bf16;
    if (d->dtype == KDN_BF16) backward_e<kdn::bf16_t>(a, d->d_k, l.slots, st);
    else backward_e<float>(a, d->d_k, l.slots, st);
    return hipGetLastError() == hipSuccess ? KDN_OK : KDN_ERR_HIP;
}

}  // extern "C"
