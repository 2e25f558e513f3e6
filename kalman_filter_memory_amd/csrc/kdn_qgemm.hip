// kdn_qgemm.hip -- matrix product of 8-bit operands with a scale for each block
// of 128:
//   C[m][n] = sum_kb sA[m][kb] sB[n / 128][kb] sum_{k in block kb} A[m][k] B[n][k]
// A [M][K] and B [N][K] are e4m3 with k contiguous (activations and a weight in a
// linear layer's layout), C is float32 or bfloat16.
//
// One v_mfma_f32_16x16x128_f8f6f4 is exactly one block deep, so a tile's product
// with a block comes out of one instruction whole, in float32, and one multiply-add
// per element brings it, scaled, to the accumulator.  The matrix instruction takes
// 32 cycles of its unit, the four multiply-adds 16 of the vector unit, side by side.
// Its own scale operands are powers of two and are not used.
//
// The 8-bit instructions add 8 products at a time aligned to the largest of them
// and drop what lies more than 2^14 below it (448 x 448 and a product of 4: the 4 is
// gone; the groups of 8 are then added in float32).  Each group loses at most 7 2^-14 of
// its largest product; on random operands a product of any depth is 1.5e-5 off, 2-norm
// over 2-norm.  Operands widened to bfloat16 in registers (exactly) and multiplied by the
// bfloat16 instruction, at half the rate, have float32's sums (1e-8).  A float32 C is
// computed that way, and a bfloat16 C of few rows, where the weights' way from memory sets
// the pace (1 x 6192 x 2048 4.3 us against 4.2, 16 x 2048 x 2048 4.2 against 4.1).  A
// bfloat16 C of more rows takes the 8-bit instruction: 1.5e-5 is 1 % of its rounding, and
// what a group loses, 7 2^-14 of its largest product, is a hundredth of what rounding
// that product's operands to e4m3, by up to 2^-4 each, may have cost before (us, widened
// and in 8 bits: 64 x 6192 x 2048 7.4, 6.1; 1024 x 6192 x 2048 30.7, 20.2; 32768 x 6192 x
// 2048 752, 423; 8192^3 912, 450).
//
// B is the instruction's first operand: a lane then holds consecutive columns n of
// one row m of C.  Which weight row stands in which row of the instruction is free,
// and is chosen so that a lane has 16 bytes of C in one piece (column_of).  The order of k inside a block is free as
// well (both operands only have to agree): lane group g takes bytes 16 g .. + 15 and
// 64 + 16 g .. + 15 of the 128.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "kdn.h"
#include "kdn_quant.h"

namespace {

using kdn::bf16_t;
using kdn::floatx4;
using kdn::u32x4;
typedef int v8i __attribute__((ext_vector_type(8)));

constexpr int kKB = kdn::kQuantBlock;  // bytes of k per block

// what a lane reads in place of anything outside A or B
__device__ __attribute__((aligned(16))) const uint8_t kZeros[16] = {0};

struct GemmArgs {
    int M, N, K, kb;  // kb blocks along K
    const uint8_t *A, *B;
    const float *sA, *sB;
    void* C;
    int ldc;
    int wide;  // rows of C start 16-byte aligned
    int mt, nt;
};

// a lane's 32 bytes of a row of one block
struct Raw {
    u32x4 lo, hi;
};
// the same as the instruction takes them (WIDE: in bfloat16), and the product of 16 rows
// by 16 rows
template <bool WIDE> struct Block;
template <> struct Block<false> {
    v8i x;
    __device__ __forceinline__ void set(const Raw& r) {
        x = v8i{int(r.lo[0]), int(r.lo[1]), int(r.lo[2]), int(r.lo[3]),
                int(r.hi[0]), int(r.hi[1]), int(r.hi[2]), int(r.hi[3])};
    }
    static __device__ __forceinline__ floatx4 mul(const Block& a, const Block& b) {
        const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.x, b.x, zero, 0, 0, 0, 0, 0, 0);
    }
};
template <> struct Block<true> {
    kdn::bf16x8 x[4];
    __device__ __forceinline__ void set(const Raw& r) {
        typedef __bf16 pair __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const unsigned u = w < 4 ? r.lo[w & 3] : r.hi[w & 3];
            const pair p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u, 1.f, false);
            const pair q = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u, 1.f, true);
            x[w / 2][4 * (w & 1)] = p[0];
            x[w / 2][4 * (w & 1) + 1] = p[1];
            x[w / 2][4 * (w & 1) + 2] = q[0];
            x[w / 2][4 * (w & 1) + 3] = q[1];
        }
    }
    static __device__ __forceinline__ floatx4 mul(const Block& a, const Block& b) {
        floatx4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.x[i], b.x[i], c, 0, 0, 0);
        return c;
    }
};

// The column, within a wave's 16 TN, that row r of the j-th instruction's B stands for:
// a lane's four elements of one instruction (float32) or two (bfloat16) are 16 bytes
// of C, and the lane groups r / 4 = 0..3 follow each other.
template <typename Eo> __device__ __forceinline__ int column_of(int j, int r) {
    return sizeof(Eo) == 2 ? 32 * (j / 2) + 8 * (r / 4) + 4 * (j & 1) + (r & 3) : 16 * j + r;
}

// 16 (4) bytes per lane from base + off straight into LDS: lane l's land at lds +
// 16 l (4 l).  As inline assembly because the compiler, which cannot see that the
// buffers of a tile take turns, would wait for the copy before the next LDS read; the
// waits are step_wait's.  (No register is loaded; m0 needs the one wait state before
// it is used.)
__device__ __forceinline__ void copy16_to_lds(const void* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(off), "s"(base), "s"(lds)
                 : "memory");
}
__device__ __forceinline__ void copy4_to_lds(const void* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
                 :
                 : "v"(off), "s"(base), "s"(lds)
                 : "memory");
}
// this wave's LDS accesses are done, and its copies but the last N; every wave is here
template <int N> __device__ __forceinline__ void step_wait() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

// Tiles of BM x BN, WM x WN waves, one block of k per step, S steps of operands in
// LDS.  Both operands and A's scales are copied straight there (8 rows of 128 bytes
// per wave and instruction); a row's eight 16-byte pieces are stored in an order that
// depends on the row (the lane that writes a place chooses what it loads), so that the
// 16 rows a fragment reads at one k lie in different banks.  Rows behind the last one
// of A or B are copies of it, whose products are not stored; pieces behind K are
// zeros.
// The one barrier of a step stands before the products of its last rows of fragments:
// by then everybody has read the step's operands, whose buffer is filled anew, and
// has its part of the next step's, whose first fragments are read while those
// products run.
// Measured (bfloat16 results): 8192^3 429 us, 2.6 PFLOP/s; 32768 x 6192 x 2048 408 to 424 us,
// 2.0 PFLOP/s, the matrix unit busy 51 % of its cycles at 2.0 GHz: a step takes 1.56 us, and
// a tile 6 us besides, its first loads and its C, with nothing beside them, since one
// workgroup fills a CU.  Float32 results: 760 and 881 us.  Timing copies without
// the copies into LDS, or without the fragments' reads, take 379 and 298 us where the
// whole took 490 (8192^3): both ways through LDS bound it, and the multiply-adds.
//
// KS groups of such waves share the steps (group i takes blocks i, i + KS, ...), each
// with its own buffers, and their sums meet at the end, the first group's first: a
// small tile leaves a SIMD one wave, whose instructions (in float32 the conversions),
// not the matrix unit, set the pace.
template <int BM, int BN, int WM, int WN, int S, int KS, typename Eo>
__global__ __launch_bounds__(64 * WM * WN * KS, 2) void qgemm_kernel(GemmArgs p) {
    using Op = Block<sizeof(Eo) == 4>;
    constexpr int W = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int PIECES = (BM + BN) / 8, PW = PIECES / W, PA = BM / 8 / W;
    constexpr int SK = 8;  // steps of scales per copy: a cache line is asked for once for eight
    constexpr int SW = BM / 8 / W;  // such copies of 8 rows per wave
    static_assert(S - 1 < SK && BM / 8 % W == 0 && BN / 8 % W == 0 && BN / WN <= kKB && TM % 2 == 0, "tile");
    __shared__ __attribute__((aligned(16))) uint8_t tiles[KS][S][(BM + BN) * kKB];
    __shared__ float scales[KS][2][BM][SK], scales_b[KS][2][W][64];  // (of 64, SK count)
    const int lane = threadIdx.x & 63, wave = kdn::wave_id() % W, grp = kdn::wave_id() / W;
    auto& tile = tiles[grp];
    auto& scale = scales[grp];
    auto& scale_b = scales_b[grp];
    const int wm = wave % WM, wn = wave / WM;
    // each XCD (workgroups are handed to the eight in turn) takes a run of tiles, and
    // walks it in strips of 6 tiles of m, so that its 32 CUs work on about 6 x 5 tiles at
    // a time and read the least through its L2 (us in strips of 4, 6, 8, 16 tiles: 32768 x
    // 6192 x 2048 425, 410, 430, 473; 8192^3 430, 433, 430, 441; 16384 x 4096 x 4096 228,
    // 229, 228, 236; 4096 x 16384 x 2048 131, 130, 131, 132; 32768 x 2048 x 2048 131, 131,
    // 132, 132)
    constexpr int STRIP = 6;
    const int total = p.mt * p.nt;
    int t = blockIdx.x;
    {
        const int per = total / 8, more = total % 8, x = t % 8, i = t / 8;
        t = x * per + (x < more ? x : more) + i;
    }
    const int strip = t / (STRIP * p.nt), in_strip = t - strip * STRIP * p.nt;
    const int width = p.mt - STRIP * strip < STRIP ? p.mt - STRIP * strip : STRIP;
    const int m0 = (STRIP * strip + in_strip % width) * BM, n0 = (in_strip / width) * BN;

    // where a row's piece c is stored: at c ^ key.  The 64 banks of LDS hold two rows of
    // 128 bytes, so 16 rows at one k use each bank once if the rows of either parity
    // have eight different keys.
    auto key_a = [](int r) { return (r >> 1) & 7; };
    auto key_b = [](int r) {
        return sizeof(Eo) == 2 ? ((r >> 3) & 3) * 2 + ((r >> 1) & 1) : (r >> 1) & 7;
    };
    // piece = wave + W i: rows 8 piece .. + 7 of A's tile (i < PA), then of B's
    const int row8 = lane >> 3, place = lane & 7;
    auto piece_row = [&](int i) { return 8 * (wave + W * (i < PA ? i : i - PA)) + row8; };
    auto piece_k = [&](int i) {
        const int r = piece_row(i);
        return 16 * (place ^ (i < PA ? key_a(r) : key_b(r)));
    };
    uint32_t off[PW];
#pragma unroll
    for (int i = 0; i < PW; ++i) {
        const int r = piece_row(i), last = (i < PA ? p.M - m0 : p.N - n0) - 1;
        off[i] = uint32_t(r < last ? r : last) * uint32_t(p.K) + uint32_t(piece_k(i));
    }
    const uint8_t* a0 = p.A + size_t(m0) * p.K;
    const uint8_t* b0 = p.B + size_t(n0) * p.K;
    const float* s0 = p.sA + size_t(m0) * p.kb;
    const int nb = (n0 + wn * 16 * TN) / kKB, nbs = (p.N + kKB - 1) / kKB;
    const float* sb = p.sB + size_t(nb < nbs ? nb : nbs - 1) * p.kb;
    const uint32_t lds0 = uint32_t(uintptr_t((__attribute__((address_space(3))) uint8_t*)&tile[0][0]));
    const uint32_t ldss = uint32_t(uintptr_t((__attribute__((address_space(3))) float*)&scale[0][0][0]));
    const uint32_t ldsb = uint32_t(uintptr_t((__attribute__((address_space(3))) float*)&scale_b[0][wave][0]));
    const int full = p.K / kKB;  // whole blocks; p.kb is one more with a partial one
    const int steps = (p.kb + KS - 1) / KS;
    auto block_of = [&](int step) { return step * KS + grp; };
    auto piece_at = [&](int k, int i) {  // byte of LDS
        return k % S * (BM + BN) * kKB + 8 * (wave + W * i) * kKB;
    };
    auto load_piece = [&](int k, int i) {  // of a whole block
        copy16_to_lds((i < PA ? a0 : b0) + size_t(block_of(k)) * kKB, off[i],
                      lds0 + uint32_t(piece_at(k, i)));
    };
    auto load = [&](int k) {
        const int kb = block_of(k);
#pragma unroll
        for (int i = 0; i < PW; ++i) {
            if (kb < full || kb * kKB + piece_k(i) < p.K) load_piece(k, i);
            else *reinterpret_cast<u32x4*>(&tile[0][0] + piece_at(k, i) + 16 * lane) = u32x4{0, 0, 0, 0};
        }
    };
    // the scales of steps k .. k + SK - 1 (k a multiple of SK; behind K: the last one's)
    auto load_scales = [&](int k) {
        const int buf = k / SK & 1, kb = block_of(k + lane % SK), col = kb < p.kb ? kb : p.kb - 1;
#pragma unroll
        for (int i = 0; i < SW; ++i) {
            const int r = 8 * (wave + W * i), row = r + lane / SK, last = p.M - m0 - 1;
            const int from = (row < last ? row : last) * p.kb + col;
            copy4_to_lds(s0, uint32_t(from) * 4u, ldss + (buf * BM + r) * SK * 4);
        }
        copy4_to_lds(sb, uint32_t(col) * 4u, ldsb + buf * W * 64 * 4);
    };

    floatx4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

    const int r16 = lane & 15, g = lane >> 4;
    const int ra = wm * 16 * TM + r16, ka = key_a(ra);
    const int rb = wn * 16 * TN + column_of<Eo>(0, r16);
    const int kbkey = key_b(rb);  // (the same for all j)
    const int a_lo = ra * kKB + 16 * (g ^ ka), a_hi = ra * kKB + 16 * ((g + 4) ^ ka);
    const int b_lo = (BM + rb) * kKB + 16 * (g ^ kbkey), b_hi = (BM + rb) * kKB + 16 * ((g + 4) ^ kbkey);
    constexpr int DIST = TM % 4 == 0 ? 2 : 1, NA = 2 * DIST;  // rows of A read ahead
    Raw fa[NA], fb[TN];
    float s[NA], sbk = 0.f;
    auto read_a = [&](int k, int i) {
        const int buf = k % S;
        fa[i % NA].lo = *reinterpret_cast<const u32x4*>(&tile[buf][a_lo + 16 * i * kKB]);
        fa[i % NA].hi = *reinterpret_cast<const u32x4*>(&tile[buf][a_hi + 16 * i * kKB]);
        s[i % NA] = scale[k / SK & 1][ra + 16 * i][k % SK];
    };
    auto read_b = [&](int buf, int j) {
        fb[j].lo = *reinterpret_cast<const u32x4*>(&tile[buf][b_lo + column_of<Eo>(j, 0) * kKB]);
        fb[j].hi = *reinterpret_cast<const u32x4*>(&tile[buf][b_hi + column_of<Eo>(j, 0) * kKB]);
    };
    if (p.kb > 0) {
        load_scales(0);
#pragma unroll
        for (int k = 0; k < S; ++k)
            if (k < steps) load(k);
        if (full >= (S + 1) * KS) step_wait<(S - 1) * PW>();
        else step_wait<0>();
#pragma unroll
        for (int i = 0; i < DIST; ++i) read_a(0, i);
#pragma unroll
        for (int j = 0; j < TN; ++j) read_b(0, j);
        sbk = scale_b[0][wave][0];
    }
    // One step.  In the steps before the last S there is nothing to ask for: LAST is
    // false.  The order is the source's (sched_barrier): the copies go out one by one
    // between the products, and a product's multiply-adds follow DELAY products later,
    // when it is there.
    auto step = [&](int k, auto last) {
        constexpr bool LAST = decltype(last)::value;
        constexpr int DELAY = TN > 2 ? 2 : 1;
        constexpr int X0 = (TM - DIST) * TN;  // the barrier
        constexpr int PER = (PW + DIST * TN - 1) / (DIST * TN);  // copies per product behind it
        const int nbuf = (k + 1) % S;
        const bool live = KS == 1 || block_of(k) < p.kb;  // (else zeros, whatever their scale)
        Op xb[TN], xa;
        floatx4 part[DELAY + 1];
        float sc[2], sb_next = 0.f;
#pragma unroll
        for (int j = 0; j < TN; ++j) xb[j].set(fb[j]);
#pragma unroll
        for (int x = 0; x < TM * TN + DELAY; ++x) {
            const int i = x / TN, j = x % TN;
            if (x < TM * TN) {
                if (x == X0) {
                    // (what is added up by now is, and does not move behind the branches,
                    // where its products would take registers)
#pragma unroll
                    for (int y = 0; y < x - DELAY; ++y) asm volatile("" : "+v"(acc[y / TN][y % TN]));
                    // the copies of the steps behind the next one stay under way; the
                    // last steps wait for all
                    if constexpr (LAST) step_wait<0>();
                    else step_wait<(S - 2) * PW>();
                    if (k % SK == 0 && k + SK < steps) load_scales(k + SK);
                }
                if (j == 0) {
                    xa.set(fa[i % NA]);
                    sc[i & 1] = live ? s[i % NA] * sbk : 0.f;
                }
                part[x % (DELAY + 1)] = Op::mul(xb[j], xa);
                // (in the last step this reads what an earlier one left, unused)
                if (i == TM - 1) read_b(nbuf, j);
                if (j == 0) read_a(i + DIST < TM ? k : k + 1, (i + DIST) % TM);
                if (x == TM * TN - 1) sb_next = scale_b[(k + 1) / SK & 1][wave][(k + 1) % SK];
                if constexpr (!LAST) {
                    if (x >= X0)
#pragma unroll
                        for (int c = 0; c < PER; ++c)
                            if ((x - X0) * PER + c < PW) load_piece(k + S, (x - X0) * PER + c);
                } else if (x == X0) {
                    if (k + S < steps) load(k + S);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if (x >= DELAY) {
                const int y = x - DELAY, iy = y / TN, jy = y % TN;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[iy][jy][e] = fmaf(part[y % (DELAY + 1)][e], sc[iy & 1], acc[iy][jy][e]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        sbk = sb_next;
    };
    int k = 0;
    for (; (k + S + 1) * KS <= full; ++k) step(k, std::false_type{});
    for (; k < steps; ++k) step(k, std::true_type{});
    if constexpr (KS > 1) {
        static_assert((KS - 1) * BM * BN * 4 <= int(sizeof(tiles)), "the groups' sums fit the operands' place");
        floatx4* sums = reinterpret_cast<floatx4*>(&tiles[0][0][0]);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TM * TN; ++i)
            if (grp > 0) sums[((grp - 1) * TM * TN * W + i * W + wave) * 64 + lane] = acc[i / TN][i % TN];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TM * TN; ++i)
            if (grp == 0)
#pragma unroll
                for (int o = 0; o < KS - 1; ++o)
                    acc[i / TN][i % TN] += sums[(o * TM * TN * W + i * W + wave) * 64 + lane];
    }
    // C goes through LDS, rounded, so that a wave writes whole rows of the tile: written
    // from the fragments, 64 bytes of 16 rows at a time, rows that do not start on a
    // cache line cost twice the write requests (32768 x 6144 x 2048 into rows of 6192:
    // 453 against 397 us for rows of 6208).  Pieces of a row are stored in an order that
    // depends on the row, as above.
    constexpr int V = 16 / int(sizeof(Eo)), CR = BN / V;  // columns, and pieces of a row
    static_assert(BM * CR * 16 <= int(sizeof(tiles)) && CR >= 4, "C fits the operands' place");
    auto key_c = [](int r) { return CR >= 16 ? r & 15 : CR >= 8 ? (r >> 1) & 7 : (r >> 2) & 3; };
    u32x4* out = reinterpret_cast<u32x4*>(&tiles[0][0][0]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int r = ra + 16 * i;
#pragma unroll
        for (int v = 0; v < 4 * TN / V; ++v) {
            u32x4 u;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if constexpr (sizeof(Eo) == 2) {
                    const floatx4& t = acc[i][2 * v + w / 2];
                    u[w] = kdn::pack_bf16(t[2 * (w & 1)], t[2 * (w & 1) + 1]);
                } else {
                    u[w] = __float_as_uint(acc[i][v][w]);
                }
            }
            if (grp == 0) out[r * CR + ((wn * 16 * TN / V + 4 * v + g) ^ key_c(r))] = u;
        }
    }
    __syncthreads();
    constexpr int NT = 64 * W * KS;
    if (p.wide) {
#pragma unroll 4
        for (int o = threadIdx.x; o < BM * CR; o += NT) {
            const int r = o / CR, c = o % CR, m = m0 + r, n = n0 + c * V;
            const u32x4 u = out[r * CR + (c ^ key_c(r))];
            if (m < p.M && n < p.N) {
                Eo* row = static_cast<Eo*>(p.C) + size_t(m) * p.ldc;
                if (n + V <= p.N) {
                    *reinterpret_cast<u32x4*>(row + n) = u;
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (n + e < p.N) {
                            if constexpr (sizeof(Eo) == 2) row[n + e] = bf16_t(u[e / 2] >> (16 * (e & 1)));
                            else row[n + e] = __uint_as_float(u[e]);
                        }
                }
            }
        }
    } else {
        // Rows that start anywhere: the pieces are those of memory, aligned there, each
        // from two neighbours of the tile's, and what is left at the row's two ends is
        // written in elements.  8192 x 4097 x 1024 bfloat16 86 us with the tile's own
        // pieces, written in elements, 55 so; 25230 x 3861 x 64 float32 151 and 90.
        const int end = p.N - n0 < BN ? p.N - n0 : BN;
        // the first column of row m that is aligned
        auto first = [&](int m) { return int((0u - uint32_t(m) * uint32_t(p.ldc)) & (V - 1)); };
#pragma unroll 2
        for (int o = threadIdx.x; o < BM * CR; o += NT) {
            const int r = o / CR, c = o % CR, m = m0 + r, off = first(m), n = c * V + off;
            const u32x4 lo = out[r * CR + (c ^ key_c(r))];
            const u32x4 hi = out[r * CR + ((c + 1 < CR ? c + 1 : c) ^ key_c(r))];
            const int words = off * int(sizeof(Eo)) / 4;
            const bool two = words & 2, one = words & 1, half = sizeof(Eo) == 2 && (off & 1);
            // (by value: a choice between two elements of an array would be one of their
            // addresses, and the array in memory)
            auto pick = [](bool x, uint32_t a, uint32_t b) { return x ? a : b; };
            uint32_t w[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = pick(two, w[i + 2], w[i]);
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = pick(one, w[i + 1], w[i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pick(half, (w[i] >> 16) | (w[i + 1] << 16), w[i]);
            if (m < p.M && n + V <= end)
                *reinterpret_cast<u32x4*>(static_cast<Eo*>(p.C) + size_t(m) * p.ldc + n0 + n) =
                    u32x4{w[0], w[1], w[2], w[3]};
        }
        const Eo* el = reinterpret_cast<const Eo*>(out);
        for (int o = threadIdx.x; o < BM * 2 * V; o += NT) {
            const int r = o / (2 * V), e = o % (2 * V), m = m0 + r, off = first(m);
            const int tail = off + (end > off ? (end - off) / V * V : 0);
            const int c = e < V ? e : tail + e - V;
            if (m < p.M && c < (e < V && off < end ? off : end))
                static_cast<Eo*>(p.C)[size_t(m) * p.ldc + n0 + c] =
                    el[(r * CR + ((c / V) ^ key_c(r))) * V + c % V];
        }
    }
}

// Few rows of A (up to 16 TM, TM 1 or 2): the weights are what has to be read, once, and every
// workgroup has to have its share of them in flight at once.  A workgroup takes 16
// columns and all of K, its W waves the blocks w, w + W, ...; fragments go from
// memory straight into registers, and the waves' sums meet in LDS in their order.
// 1 x 6192 x 2048: 4.4 us (2.9 TB/s); 1 x 8192 x 8192: 12.6 us (5.3 TB/s); 16 x 2048 x 2048:
// 4.4 us.  A wave waits for the loads of each of its blocks, two of them one after the
// other at K 2048: latency bounds the short ones, memory the long ones.
template <int TM, int W, typename Eo>
__global__ __launch_bounds__(64 * W) void qgemm_few_kernel(GemmArgs p) {
    using Op = Block<true>;
    __shared__ float sum[W][TM][16][17];
    const int tid = threadIdx.x, lane = tid & 63, wave = kdn::wave_id();
    const int r16 = lane & 15, g = lane >> 4, n0 = blockIdx.x * 16;
    const int n = n0 + r16 < p.N ? n0 + r16 : p.N - 1;
    const uint8_t* b = p.B + size_t(n) * p.K;
    const float* sb = p.sB + size_t(n0 / kKB) * p.kb;
    const uint8_t* a[TM];
    const float* sa[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int m = 16 * i + r16 < p.M ? 16 * i + r16 : p.M - 1;
        a[i] = p.A + size_t(m) * p.K;
        sa[i] = p.sA + size_t(m) * p.kb;
    }
    const u32x4* zeros = reinterpret_cast<const u32x4*>(kZeros);
    floatx4 acc[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) acc[i] = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int kb = wave; kb < p.kb; kb += W) {
        const int k0 = kb * kKB + 16 * g, k1 = k0 + 64;
        const bool in0 = k0 < p.K, in1 = k1 < p.K;
        Op fb, fa;
        fb.set(Raw{*(in0 ? reinterpret_cast<const u32x4*>(b + k0) : zeros),
               *(in1 ? reinterpret_cast<const u32x4*>(b + k1) : zeros)});
        const float sbk = sb[kb];
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            fa.set(Raw{*(in0 ? reinterpret_cast<const u32x4*>(a[i] + k0) : zeros),
                   *(in1 ? reinterpret_cast<const u32x4*>(a[i] + k1) : zeros)});
            const float s = sa[i][kb] * sbk;
            const floatx4 part = Op::mul(fb, fa);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(part[e], s, acc[i][e]);
        }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[wave][i][r16][4 * g + e] = acc[i][e];
    __syncthreads();
    for (int o = tid; o < TM * 256; o += 64 * W) {
        const int m = o / 16, c = o % 16;
        float x = sum[0][m / 16][m % 16][c];
#pragma unroll
        for (int w = 1; w < W; ++w) x += sum[w][m / 16][m % 16][c];
        if (m < p.M && n0 + c < p.N)
            static_cast<Eo*>(p.C)[size_t(m) * p.ldc + n0 + c] = kdn::from_f<Eo>(x);
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

kdn_status check_gemm(const kdn_gemm_desc* d) {
    if (!d) return KDN_ERR_NULL;
    if (d->M < 0 || d->N < 0 || d->K < 0 || d->ldc < d->N) return KDN_ERR_SHAPE;
    if (d->dtype != KDN_F32 && d->dtype != KDN_BF16) return KDN_ERR_UNSUPPORTED;
    if (d->K % 16 != 0) return KDN_ERR_UNSUPPORTED;  // rows of A and B start 16-byte aligned
    // 32-bit tile and row arithmetic (a tile's rows of A start 255 K apart at most); a
    // grid holds fewer than 2^32 threads, 512 per 16 columns with few rows
    if (d->M > (1 << 26) || d->N > (1 << 26) || d->ldc > (1 << 26) || d->K > (1 << 23))
        return KDN_ERR_UNSUPPORTED;
    if (((int64_t(d->M) + 63) / 64) * ((int64_t(d->N) + 63) / 64) >= (1 << 22))
        return KDN_ERR_UNSUPPORTED;
    return KDN_OK;
}

template <int BM, int BN, int WM, int WN, int S, int KS, typename Eo> void launch_tiles(GemmArgs a, hipStream_t st) {
    a.mt = (a.M + BM - 1) / BM;
    a.nt = (a.N + BN - 1) / BN;
    qgemm_kernel<BM, BN, WM, WN, S, KS, Eo>
        <<<unsigned(a.mt) * unsigned(a.nt), 64 * WM * WN * KS, 0, st>>>(a);
}

template <typename Eo> void launch_gemm(const GemmArgs& a, hipStream_t st) {
    const unsigned cols = unsigned((a.N + 15) / 16);
    // Few rows, and no more than one workgroup per CU (bfloat16): 16 x 2048 x 2048 takes 4.4
    // us against 5.3 in tiles of 32 x 32, 16 x 4096 x 8192 11.5 against 13.0, but 16 x 6192 x
    // 2048 6.6 against 5.3 and 16 x 8192 x 8192 20.5 against 15.5, for every workgroup reads
    // every row of A.  Up to four rows are ahead anywhere (4 x 8192 x 8192 14.8 against 15.4,
    // 1 row 12.8 against 15.8), 17 to 32 with a short K (24 x 1000 x 1024 3.7 against 4.4; 32
    // x 2048 x 2048 5.7 against 5.1).
    if (a.M <= 4 || (a.M <= 16 && cols <= 256)) {
        qgemm_few_kernel<1, 8, Eo><<<cols, 512, 0, st>>>(a);
    } else if (a.M <= 32 && cols <= 256 && a.kb <= 8) {
        qgemm_few_kernel<2, 8, Eo><<<cols, 512, 0, st>>>(a);
    } else {
        // The larger the tile, the less is read per product, as long as the tiles fill
        // the 256 CUs.  Tiles of 128 x 128 run two to a CU and end one by one; a round of
        // 256 tiles of 256 x 256, one to a CU, takes as long as 712 of them (us, bfloat16,
        // K 2048): 4096 x 6192 (400 large tiles, two rounds) 57.5 in large ones against
        // 63.1, 3000 x 6192 (300, two rounds) 66.0 against 53.4.  Against 64 x 64: 512 x
        // 6192 is 196 tiles of 128 x 128 and takes 13.4 in them against 15.7, 1024 x 2048
        // is 128 and takes 11.8 against 9.9.  (Widened operands leave no registers for
        // the largest tile.)
        // With fewer tiles than fill the GPU groups of waves share K, if it is long enough:
        // two groups per 64 x 64 tile while all tiles run at once, two to a CU (509 x 2048 x
        // 2064 8.8 -> 8.2, float32 11.8 -> 10.3; but 384 x 6192 x 2048, 582 tiles, 12.5 ->
        // 15.5, and 100 x 1000 x 128 3.1 -> 3.8); one to a CU with four steps in LDS, or in
        // float32 with four groups, where K is longer (256 x 4096 x 8192 24.5 -> 18.5, x 4096
        // in float32 14.5 -> 14.1; 509 x 2048 x 2064 8.2 -> 8.4); four groups per 32 x 32 tile
        // while those run at once, two to a CU (64 x 6192 x 2048 6.7 -> 5.9, 128 x 2048 x
        // 8192 16.8 -> 9.8, 430 x 270 x 4576 in float32 16.1 -> 9.0; 256 x 4096 x 2048, 1024
        // such tiles, 7.1 -> 10.6).
        const int64_t tiny = int64_t((a.M + 31) / 32) * ((a.N + 31) / 32);
        const int64_t few = int64_t((a.M + 63) / 64) * ((a.N + 63) / 64);
        const int64_t big = int64_t((a.M + 255) / 256) * ((a.N + 255) / 256);
        const int64_t mid = int64_t((a.M + 127) / 128) * ((a.N + 127) / 128);
        if (sizeof(Eo) == 2 && (big + 255) / 256 * 712 <= mid)
            launch_tiles<256, 256, 2, 4, 2, 1, bf16_t>(a, st);
        else if (mid >= 192)
            launch_tiles<128, 128, 2, 2, 2, 1, Eo>(a, st);
        else if (a.kb >= 8 && tiny <= 512)
            launch_tiles<32, 32, 1, 1, 2, 4, Eo>(a, st);
        else if (a.kb >= 32 && few <= 256)
            launch_tiles<64, 64, 2, 2, sizeof(Eo) == 2 ? 4 : 2, sizeof(Eo) == 2 ? 2 : 4, Eo>(a, st);
        else if (a.kb >= 8 && few <= 512)
            launch_tiles<64, 64, 2, 2, 2, 2, Eo>(a, st);
        else
            launch_tiles<64, 64, 2, 2, 2, 1, Eo>(a, st);
    }
}

}  // namespace

extern "C" {

kdn_status kdn_quant_gemm(const kdn_gemm_desc* d, const void* A, const float* sA, const void* B,
                          const float* sB, void* C, void* stream) {
    const kdn_status st = check_gemm(d);
    if (st != KDN_OK) return st;
    if (d->M == 0 || d->N == 0) return KDN_OK;
    if (!C || (d->K > 0 && (!A || !sA || !B || !sB))) return KDN_ERR_NULL;
    if (!aligned16(A) || !aligned16(B) || !aligned16(C)) return KDN_ERR_ALIGN;
    GemmArgs a{};
    a.M = d->M;
    a.N = d->N;
    a.K = d->K;
    a.kb = (d->K + kKB - 1) / kKB;
    a.A = static_cast<const uint8_t*>(A);
    a.B = static_cast<const uint8_t*>(B);
    a.sA = sA;
    a.sB = sB;
    a.C = C;
    a.ldc = d->ldc;
    a.wide = (size_t(d->ldc) * (d->dtype == KDN_BF16 ? 2 : 4)) % 16 == 0;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    if (d->dtype == KDN_BF16) launch_gemm<bf16_t>(a, hs);
    else launch_gemm<float>(a, hs);
    return hipGetLastError() == hipSuccess ? KDN_OK : KDN_ERR_HIP;
}

}  // extern "C"
