// block_gemm.hip -- grouped FP8 e4m3 x e4m3 products with one scale per block
// of 128 (include/moe_block8.h), on gfx950's v_mfma_f32_32x32x64_f8f6f4.
//
// One kernel body computes out[p][q] = sum_k P[p][k] Q[q][k] over tiles of
// BP x BQ outputs:
//   product  P = the pool's rows, Q = the weights of the row's expert;
//            fp32 scales per (row, 128 k) and per (128 q, 128 k)
//   wgrad    P = the gradient's columns, Q = the input's columns, k = the
//            rows of one group; UE8M0 scales per (column, 128 k)
//
// Mathematics of the scales.  A K step is one block of 128, so its scales are
// constant along it.  product: two MFMAs per 32 x 32 tile sum the block's
// codes from zero (the exact range of e4m3 products fits float32), then
// acc += (sp * sq) * part in float32 FMAs; with Q as the MFMA's row operand
// and P as its column operand a lane holds one pool row, so sp * sq is one
// value per lane, tile column and step.  wgrad: the power-of-two scales go
// into the MFMA itself and the sum stays in its accumulator.
//
// Layout.  P and Q tiles of one K step go straight from global memory to LDS
// (128-byte rows; 16-byte chunks XOR-swizzled through the load's source
// address so that each 16 lanes of a ds_read_b128 meet distinct banks).  The
// MFMA's row r of column tile j is LDS row (r / 4) * 4J + 4j + r % 4 of the
// wave's Q rows, so that a lane ends up with 4J adjacent outputs of a row.
// The k order inside a 64-wide MFMA is the same permutation for both operands.
#include "../../include/moe_block8.h"
#include "moe_device.hpp"
#include "moe_host.hpp"

namespace moe {
namespace {

constexpr int kBK = 128;
constexpr int kMaxGroups = 1024;
constexpr int kProduct = 0, kWgrad = 1;

typedef __attribute__((address_space(3))) void lds_void_t;
__device__ __forceinline__ uint32_t lds_addr(const void* p) { return (uint32_t)(uintptr_t)(const lds_void_t*)p; }

// Direct global -> LDS loads: lane l's 16 (4) bytes land at LDS address
// m0 + 16 l (4 l).  Inline asm, so that the compiler neither reorders LDS
// reads around them nor waits for them; M0 is set in the same statement and
// nothing else in this file may use it (a test reads the assembly).
__device__ __forceinline__ const void* uniform_ptr(const void* p) {
    const uint64_t v = (uint64_t)(uintptr_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (const void*)(uintptr_t)(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ void dma_x4(uint32_t lds, const void* sbase, uint32_t voff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(
                     __builtin_amdgcn_readfirstlane(lds)),
                 "v"(voff), "s"(uniform_ptr(sbase))
                 : "memory");
}
__device__ __forceinline__ void dma_x1(uint32_t lds, const void* sbase, uint32_t voff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(
                     __builtin_amdgcn_readfirstlane(lds)),
                 "v"(voff), "s"(uniform_ptr(sbase))
                 : "memory");
}
// All of this wave's loads but the newest N have landed and its LDS reads are
// done; then the workgroup meets.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

__device__ __forceinline__ int clamp_int(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

struct BlockArgs {
    const uint8_t* p;
    const uint8_t* q;
    const void* ps;
    const void* qs;
    const int32_t* offsets;
    uint16_t* out;
    int64_t R;   // rows of the pool
    int64_t ld;  // bytes of a row of p and q
    int N, K, E;
    int wide;    // rows of out start on 16-byte boundaries
};

// Rows [lo, lo + n) of group e, inside 0..R whatever the offsets hold.
__device__ __forceinline__ void group_rows(const BlockArgs& g, int e, int& lo, int& n) {
    if (!g.offsets) {
        lo = 0;
        n = (int)g.R;
        return;
    }
    lo = clamp_int(g.offsets[e], 0, (int)g.R);
    n = clamp_int(g.offsets[e + 1], lo, (int)g.R) - lo;
}

// One output tile: operand bases (uniform), valid rows and columns, K steps.
struct Tile {
    const uint8_t* p;
    const uint8_t* q;
    const uint8_t* ps;
    const uint8_t* qs;
    uint16_t* out;
    int rows, cols, nk;
};

template <int MODE_, int WQ_, int WP_, int J_, int TT_, int STAGES_, int GROUP_, int PER_CU_>
struct Cfg {
    static constexpr int MODE = MODE_, WQ = WQ_, WP = WP_, J = J_, TT = TT_, STAGES = STAGES_, GROUP = GROUP_,
                         PER_CU = PER_CU_;
    static constexpr int BQ = 32 * J * WQ, BP = 32 * TT * WP, WAVES = WQ * WP, THREADS = 64 * WAVES;
    static constexpr int PP = BP * 8 / THREADS, QP = BQ * 8 / THREADS;  // 16-byte loads per thread and step
    static constexpr int ROWS = THREADS / 8;                            // LDS rows one pass fills
    static constexpr int LOADS = PP + QP + (MODE == kProduct ? 1 : 0);  // per wave and step
    static constexpr int QOFF = BP * kBK, SOFF = (BP + BQ) * kBK;
    static constexpr int STAGE = SOFF + (MODE == kProduct ? BP * 4 + 256 : 0);
    static_assert(BP / 64 < WAVES || MODE == kWgrad, "a wave for the Q scales");
    static_assert(ROWS % 16 == 0 && ROWS % (16 * J) == 0, "a thread's chunk does not depend on the pass");
};

// Swizzle keys of LDS rows: 16-byte chunk c of row r lies at chunk c ^ key(r).
__device__ __forceinline__ int p_key(int r) { return (r >> 1) & 7; }
template <int J>
__device__ __forceinline__ int q_key(int r) {
    return ((r / (4 * J)) & 3) << 1 | ((r >> 1) & 1);
}

template <class C>
struct Worker {
    static constexpr int MODE = C::MODE;
    const BlockArgs& g;
    uint8_t* lds;
    const int* pre;  // product: m-tiles before expert e; wgrad: K steps before group e
    int tid, lane, wave, wq, wp;
    int nq, np;  // tiles along q; along p (wgrad)

    __device__ __forceinline__ Worker(const BlockArgs& g_, uint8_t* l, const int* t) : g(g_), lds(l), pre(t) {
        tid = threadIdx.x;
        lane = tid & 63;
        wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        wq = wave % C::WQ;
        wp = wave / C::WQ;
        nq = ((MODE == kProduct ? g.N : g.K) + C::BQ - 1) / C::BQ;
        np = (g.N + C::BP - 1) / C::BP;
    }
    __device__ __forceinline__ int64_t tiles() const {
        return MODE == kProduct ? (int64_t)pre[g.E] * nq : (int64_t)g.E * np * nq;
    }

    // Tile idx of the order: GROUP p-tiles by all q-tiles, p fastest.
    __device__ __forceinline__ Tile at(int64_t idx) const {
        const int64_t mt = MODE == kProduct ? (int64_t)pre[g.E] : (int64_t)g.E * np;
        const int64_t grp = idx / ((int64_t)C::GROUP * nq), in = idx % ((int64_t)C::GROUP * nq);
        const int64_t left = mt - grp * C::GROUP;
        const int gm = left < C::GROUP ? (int)left : C::GROUP;
        const int64_t m = grp * C::GROUP + in % gm;
        const int qt = __builtin_amdgcn_readfirstlane((int)(in / gm));
        Tile t;
        if (MODE == kProduct) {
            int lo = 0, hi = g.E;  // the expert of m-tile m: pre[lo] <= m < pre[lo + 1]
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (pre[mid] <= (int)m) lo = mid;
                else hi = mid;
            }
            const int e = __builtin_amdgcn_readfirstlane(lo);
            int first, n;
            group_rows(g, e, first, n);
            const int r0 = ((int)m - pre[e]) * C::BP;
            const int64_t row = (int64_t)first + r0;
            const int q0 = qt * C::BQ, kb = g.K / kBK, nb = (g.N + 127) / 128;
            t.rows = n - r0 < C::BP ? n - r0 : C::BP;
            t.cols = g.N - q0 < C::BQ ? g.N - q0 : C::BQ;
            t.nk = kb;
            t.p = g.p + row * g.ld;
            t.q = g.q + ((int64_t)e * g.N + q0) * g.ld;
            t.ps = (const uint8_t*)((const float*)g.ps + row);
            t.qs = (const uint8_t*)((const float*)g.qs + ((int64_t)e * nb + q0 / 128) * kb);
            t.out = g.out + row * g.N + q0;
        } else {
            const int e = __builtin_amdgcn_readfirstlane((int)(m / np)), p0 = (int)(m % np) * C::BP, q0 = qt * C::BQ;
            const int most = (int)(g.ld / kBK), k0 = clamp_int(pre[e], 0, most);
            t.rows = g.N - p0 < C::BP ? g.N - p0 : C::BP;
            t.cols = g.K - q0 < C::BQ ? g.K - q0 : C::BQ;
            t.nk = clamp_int(pre[e + 1], k0, most) - k0;
            t.p = g.p + p0 * g.ld + (int64_t)k0 * kBK;
            t.q = g.q + q0 * g.ld + (int64_t)k0 * kBK;
            t.ps = (const uint8_t*)g.ps + (int64_t)k0 * g.N + p0;
            t.qs = (const uint8_t*)g.qs + (int64_t)k0 * g.K + q0;
            t.out = g.out + ((int64_t)e * g.N + p0) * g.K + q0;
        }
        t.rows = __builtin_amdgcn_readfirstlane(t.rows);
        t.cols = __builtin_amdgcn_readfirstlane(t.cols);
        t.nk = __builtin_amdgcn_readfirstlane(t.nk);
        t.p = (const uint8_t*)uniform_ptr(t.p);
        t.q = (const uint8_t*)uniform_ptr(t.q);
        t.ps = (const uint8_t*)uniform_ptr(t.ps);
        t.qs = (const uint8_t*)uniform_ptr(t.qs);
        t.out = (uint16_t*)uniform_ptr(t.out);
        return t;
    }
};

// The load side: walks the workgroup's K steps STAGES - 1 ahead of the sums.
template <class C>
struct Loader {
    Tile t;
    int k;
    int64_t idx, end, step;
    bool live;
    uint32_t po[C::PP], qo[C::QP], so;        // byte offsets from the tile's bases
    int sp_at[C::TT], sq_at[C::J];            // wgrad: this lane's scale rows
    uint32_t sp[C::TT], sq[C::J];             // wgrad: scales of the step issued last

    __device__ __forceinline__ void open(const Worker<C>& w) {
        live = false;
        while (idx < end) {
            t = w.at(idx);
            idx += step;
            if (t.nk > 0) {
                live = true;
                break;
            }
        }
        if (!live) return;
        k = 0;
        const int r = w.tid >> 3;
        const uint32_t ld = (uint32_t)w.g.ld;
        const int pc = (w.tid & 7) ^ p_key(r), qc = (w.tid & 7) ^ q_key<C::J>(r);
#pragma unroll
        for (int i = 0; i < C::PP; ++i) po[i] = (uint32_t)min(r + i * C::ROWS, t.rows - 1) * ld + 16 * pc;
#pragma unroll
        for (int i = 0; i < C::QP; ++i) qo[i] = (uint32_t)min(r + i * C::ROWS, t.cols - 1) * ld + 16 * qc;
        if (C::MODE == kProduct) {
            // waves below BP / 64: 64 row scales each; the others: the scales of the tile's q blocks
            const int kb = w.g.K / kBK, qb = min(w.lane % ((C::BQ + 127) / 128), (t.cols - 1) / 128);
            so = w.wave < C::BP / 64 ? 4u * (uint32_t)min(w.wave * 64 + w.lane, t.rows - 1) : 4u * (uint32_t)(qb * kb);
        } else {
            const int c = w.lane & 31;
#pragma unroll
            for (int i = 0; i < C::TT; ++i) sp_at[i] = min((w.wp * C::TT + i) * 32 + c, t.rows - 1);
#pragma unroll
            for (int j = 0; j < C::J; ++j)
                sq_at[j] = min(w.wq * 32 * C::J + (c >> 2) * 4 * C::J + 4 * j + (c & 3), t.cols - 1);
        }
    }

    // Issue the loads of the next step into `stage` and move on.
    __device__ __forceinline__ void issue(const Worker<C>& w, int stage) {
        if (C::MODE == kWgrad) {
            const uint8_t* a = t.ps + (int64_t)k * w.g.N;
            const uint8_t* b = t.qs + (int64_t)k * w.g.K;
#pragma unroll
            for (int i = 0; i < C::TT; ++i) sp[i] = a[sp_at[i]];
#pragma unroll
            for (int j = 0; j < C::J; ++j) sq[j] = b[sq_at[j]];
        }
        const uint32_t at = lds_addr(w.lds) + (uint32_t)(stage * C::STAGE) + (uint32_t)w.wave * 1024u;
        const uint8_t* pb = t.p + (int64_t)k * kBK;
        const uint8_t* qb = t.q + (int64_t)k * kBK;
#pragma unroll
        for (int i = 0; i < C::PP; ++i) dma_x4(at + i * C::THREADS * 16, pb, po[i]);
#pragma unroll
        for (int i = 0; i < C::QP; ++i) dma_x4(at + C::QOFF + i * C::THREADS * 16, qb, qo[i]);
        if (C::MODE == kProduct) {
            const uint32_t s = lds_addr(w.lds) + (uint32_t)(stage * C::STAGE + C::SOFF);
            const bool rows = w.wave < C::BP / 64;
            const uint8_t* base = rows ? t.ps + 4 * (int64_t)k * w.g.R : t.qs + 4 * (int64_t)k;
            dma_x1(s + (rows ? (uint32_t)w.wave * 256u : C::BP * 4u), base, so);
        }
        if (++k == t.nk) open(w);
    }
};

template <class C>
__global__ __launch_bounds__(C::THREADS, C::WAVES * C::PER_CU / 4) void k_block(BlockArgs g) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[C::STAGES * C::STAGE];
    __shared__ int pre[kMaxGroups + 1];
    __shared__ int wave_sum[C::WAVES];
    Worker<C> w(g, lds, pre);
    const int lane = w.lane;

    {  // pre: exclusive prefix sums over the groups
        constexpr int kPer = kMaxGroups / C::THREADS;
        constexpr int kUnit = C::MODE == kProduct ? C::BP : kBK;
        int n[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = w.tid * kPer + i;
            int lo = 0, rows = 0;
            if (e < g.E) group_rows(g, e, lo, rows);
            n[i] = (rows + kUnit - 1) / kUnit;
            sum += n[i];
        }
        int before = sum;
        for (int d = 1; d < kWave; d <<= 1) {
            const int up = __shfl_up(before, d);
            before += lane >= d ? up : 0;
        }
        if (lane == kWave - 1) wave_sum[w.wave] = before;
        __syncthreads();
        before -= sum;
        for (int v = 0; v < w.wave; ++v) before += wave_sum[v];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = w.tid * kPer + i;
            if (e <= g.E) pre[e] = before;
            before += n[i];
        }
        if (w.tid == C::THREADS - 1 && g.E == kMaxGroups) pre[kMaxGroups] = before;
        __syncthreads();
    }

    // XCD x (workgroups go round-robin over the 8) takes the x-th contiguous
    // eighth of the tile order, so that its L2 sees neighbouring tiles.
    const int64_t total = w.tiles();
    const int xcd = blockIdx.x & 7;
    const int64_t step = gridDim.x / 8, end = total * (xcd + 1) / 8;
    int64_t idx = total * xcd / 8 + (blockIdx.x >> 3);
    if (idx >= end) return;

    Loader<C> ld;
    ld.idx = idx;
    ld.end = end;
    ld.step = step;
    ld.open(w);
    int ahead = 0;   // stages issued and not yet used
    int stage = 0;   // next stage to use
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s)
        if (ld.live) {
            ld.issue(w, s);
            ++ahead;
        }

    // LDS read offsets: the four 16-byte chunks of this lane's half
    const int c = lane & 31, h = lane >> 5;
    const int prow = w.wp * 32 * C::TT + c;
    const int qrow = w.wq * 32 * C::J + (c >> 2) * 4 * C::J + (c & 3);
    uint32_t pr[4], qr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        pr[i] = prow * kBK + (((2 * i + h) ^ p_key(prow)) << 4);
        qr[i] = C::QOFF + qrow * kBK + (((2 * i + h) ^ q_key<C::J>(qrow)) << 4);
    }

    for (; idx < end; idx += step) {
        const Tile t = w.at(idx);
        v16f acc[C::J][C::TT];
#pragma unroll
        for (int j = 0; j < C::J; ++j)
#pragma unroll
            for (int i = 0; i < C::TT; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.f;
        // waves whose rows are all past the tile's end only load and meet
        const bool mine = w.wp * 32 * C::TT < t.rows;

        for (int k = 0; k < t.nk; ++k) {
            if (C::STAGES > 2 && ahead == C::STAGES - 1) wait_and_meet<C::LOADS*(C::STAGES - 2)>();
            else wait_and_meet<0>();
            uint32_t sp[C::TT], sq[C::J];
            if (C::MODE == kWgrad) {
                // taken over before the next loads go out, so that the wait for
                // them is the one above
#pragma unroll
                for (int i = 0; i < C::TT; ++i) {
                    sp[i] = ld.sp[i];
                    asm volatile("" : "+v"(sp[i]));
                }
#pragma unroll
                for (int j = 0; j < C::J; ++j) {
                    sq[j] = ld.sq[j];
                    asm volatile("" : "+v"(sq[j]));
                }
            }
            if (ld.live) {
                ld.issue(w, stage == 0 ? C::STAGES - 1 : stage - 1);
                ++ahead;
            }
            const uint8_t* b = lds + stage * C::STAGE;
            if (mine) {
                v8i pf[C::TT][2];
#pragma unroll
                for (int i = 0; i < C::TT; ++i)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const v4i x = *reinterpret_cast<const v4i*>(b + pr[2 * s] + i * 32 * kBK);
                        const v4i y = *reinterpret_cast<const v4i*>(b + pr[2 * s + 1] + i * 32 * kBK);
                        pf[i][s] = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
                    }
                float sc[C::TT];
                if (C::MODE == kProduct) {
                    const float* s = reinterpret_cast<const float*>(b + C::SOFF);
                    const float q = s[C::BP + w.wq * 32 * C::J / 128];
#pragma unroll
                    for (int i = 0; i < C::TT; ++i) sc[i] = s[prow + 32 * i] * q;
                }
#pragma unroll
                for (int j = 0; j < C::J; ++j) {
                    v8i qf[2];
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const v4i x = *reinterpret_cast<const v4i*>(b + qr[2 * s] + 4 * j * kBK);
                        const v4i y = *reinterpret_cast<const v4i*>(b + qr[2 * s + 1] + 4 * j * kBK);
                        qf[s] = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
                    }
#pragma unroll
                    for (int i = 0; i < C::TT; ++i) {
                        if (C::MODE == kProduct) {
                            v16f part = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
                            part = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(qf[0], pf[i][0], part, 0, 0, 0, 0, 0, 0);
                            part = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(qf[1], pf[i][1], part, 0, 0, 0, 0, 0, 0);
#pragma unroll
                            for (int r = 0; r < 16; ++r) acc[j][i][r] += part[r] * sc[i];
                        } else {
#pragma unroll
                            for (int s = 0; s < 2; ++s)
                                acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                    qf[s], pf[i][s], acc[j][i], 0, 0, 0, (int)sq[j], 0, (int)sp[i]);
                        }
                    }
                }
            }
            stage = stage + 1 == C::STAGES ? 0 : stage + 1;
            --ahead;
        }

        // lane: row prow + 32 i of the tile; register 4a + b of tile j is
        // output (2a + h) * 4J + 4j + b of the wave's 32 J
        if (mine) {
            const int64_t ldo = C::MODE == kProduct ? g.N : g.K;
#pragma unroll
            for (int i = 0; i < C::TT; ++i) {
                if (prow + 32 * i >= t.rows) continue;
                uint16_t* o = t.out + (prow + 32 * i) * ldo;
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const int q = w.wq * 32 * C::J + (2 * a + h) * 4 * C::J;
                    if (C::J % 2 == 0 && g.wide) {
#pragma unroll
                        for (int j = 0; j + 1 < C::J; j += 2) {
                            const uint4 v = make_uint4(pack_bf16x2(acc[j][i][4 * a], acc[j][i][4 * a + 1]),
                                                       pack_bf16x2(acc[j][i][4 * a + 2], acc[j][i][4 * a + 3]),
                                                       pack_bf16x2(acc[j + 1][i][4 * a], acc[j + 1][i][4 * a + 1]),
                                                       pack_bf16x2(acc[j + 1][i][4 * a + 2], acc[j + 1][i][4 * a + 3]));
                            if (q + 4 * j < t.cols) *reinterpret_cast<uint4*>(o + q + 4 * j) = v;
                        }
                    } else if (g.wide) {
#pragma unroll
                        for (int j = 0; j < C::J; ++j) {
                            const uint2 v = make_uint2(pack_bf16x2(acc[j][i][4 * a], acc[j][i][4 * a + 1]),
                                                       pack_bf16x2(acc[j][i][4 * a + 2], acc[j][i][4 * a + 3]));
                            if (q + 4 * j < t.cols) *reinterpret_cast<uint2*>(o + q + 4 * j) = v;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < C::J; ++j)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                if (q + 4 * j + x < t.cols)
                                    o[q + 4 * j + x] = (uint16_t)pack_bf16x2(acc[j][i][4 * a + x], 0.f);
                    }
                }
            }
        }
    }
}

// ---- host -----------------------------------------------------------------------
typedef Cfg<kProduct, 2, 4, 4, 2, 2, 4, 1> BigProduct;  // 256 x 256, 8 waves of 64 x 128
typedef Cfg<kProduct, 4, 1, 1, 2, 3, 1, 2> SmallProduct;  // 64 rows x 128, 4 waves of 64 x 32
typedef Cfg<kWgrad, 2, 4, 4, 2, 2, 4, 1> BigWgrad;

template <class C>
void launch(const BlockArgs& g, int64_t p_tiles, int q, hipStream_t stream) {
    const int64_t most = p_tiles * ((q + C::BQ - 1) / C::BQ);
    const int64_t fill = (int64_t)(device_cus() / 8 * 8) * C::PER_CU;
    const int64_t grid = most < fill ? (most + 7) / 8 * 8 : fill;
    hipLaunchKernelGGL(k_block<C>, dim3((unsigned)grid), dim3(C::THREADS), 0, stream, g);
}

bool block_shape_ok(const moe_block_shape_t* s) {
    return s->R <= (int64_t(1) << 28) && s->N <= (1 << 20) && s->K <= (1 << 20) && s->E <= kMaxGroups;
}
bool block_shape_valid(const moe_block_shape_t* s, const int32_t* offsets) {
    return s && s->R >= 0 && s->N >= 1 && s->K >= 1 && s->E >= 1 && (offsets || s->E == 1);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_block_gemm(const moe_block_shape_t* s, const uint8_t* a, const float* a_scales, const uint8_t* w,
                   const float* w_scales, const int32_t* offsets, void* out, moe_stream_t stream) {
    if (!block_shape_valid(s, offsets)) return MOE_ERR_INVALID_ARG;
    if (!block_shape_ok(s) || s->K % kBK) return MOE_ERR_UNSUPPORTED;
    if (s->R == 0) return MOE_OK;
    if (!a || !a_scales || !w || !w_scales || !out) return MOE_ERR_INVALID_ARG;
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(a_scales, 4) || !aligned(w_scales, 4) ||
        !aligned(offsets, 4) || !aligned(out, 2))
        return MOE_ERR_INVALID_ARG;
    if (!device_ok()) return MOE_ERR_DEVICE;
    BlockArgs g = {a, w, a_scales, w_scales, offsets, static_cast<uint16_t*>(out), s->R, s->K, s->N, s->K, s->E,
                   s->N % 8 == 0 && aligned(out, 16)};
    const int64_t used = s->E < s->R ? s->E : s->R;
    // At most 64 rows a group on average: the weights' stream bounds it, and
    // 64-row tiles waste the least of the matrix cores.
    if (s->R <= 64 * (int64_t)s->E)
        launch<SmallProduct>(g, s->R / SmallProduct::BP + used, s->N, stream);
    else
        launch<BigProduct>(g, s->R / BigProduct::BP + used, s->N, stream);
    return launch_status();
}

int moe_block_gemm_wgrad(const moe_block_shape_t* s, const uint8_t* gr, const uint8_t* g_scales, const uint8_t* x,
                         const uint8_t* x_scales, const int32_t* offsets, void* out, moe_stream_t stream) {
    if (!block_shape_valid(s, offsets)) return MOE_ERR_INVALID_ARG;
    if (!block_shape_ok(s) || s->R > (int64_t(1) << 23)) return MOE_ERR_UNSUPPORTED;
    if (!out || (s->R > 0 && (!gr || !g_scales || !x || !x_scales))) return MOE_ERR_INVALID_ARG;
    if (!aligned(gr, 16) || !aligned(x, 16) || !aligned(offsets, 4) || !aligned(out, 2)) return MOE_ERR_INVALID_ARG;
    if (!device_ok()) return MOE_ERR_DEVICE;
    BlockArgs g = {gr, x, g_scales, x_scales, offsets, static_cast<uint16_t*>(out), s->R, moe_padded_rows(s->R, s->E),
                   s->N, s->K, s->E, s->K % 8 == 0 && aligned(out, 16)};
    launch<BigWgrad>(g, (int64_t)s->E * ((s->N + BigWgrad::BP - 1) / BigWgrad::BP), s->K, stream);
    return launch_status();
}

}  // extern "C"
