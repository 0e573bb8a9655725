// Backward of the selective state space scan.
//
// With ds = dy silu(z) (the gradient of the sum over n plus the skip), and dh
// the gradient of the state after token t, walked backwards:
//   dC_n = sum_c ds h_n,   dh_n += ds C_n,   dB_n = sum_c dh_n u,  u = delta x,
//   du = sum_n dh_n B_n,   dh'_n = a_n dh_n (the gradient of the state before t),
//   m_n = dh'_n h_n(t - 1),   ddelta = sum_n A_n m_n + du x,
//   dA_log_n = A_n sum_t delta m_n,   dx = du delta + D ds,   dD = sum ds x,
//   ddt = ddelta s(dt + bias),   dz = dy (sum_n C_n h_n + D x) silu'(z).
//
// The states before each token come from the forward's checkpoints (every 8
// packed tokens).  A block of 8 tokens is run forward once, keeping the state
// before every second token in shared memory; then its pieces of two tokens are
// taken from the last to the first: forward again, with the decays a and the
// products a h in registers, then backward, where m = dh a h.  Longer pieces need
// registers (two warps a scheduler instead of three: 3.1 against 2.9 ms on 32768
// tokens of 4096 channels), longer blocks shared memory.
//
// Work split.  A channel's states lie on K lanes with four each, and a lane
// holds four channels as two pairs, so a warp works on 128 / K channels and a
// lane on 16 states a token.  delta, u and ds of a pair are read as one operand
// of the two-wide instructions; B and C lie in shared memory twice each for the
// same reason.  The sums over channels (dB, dC) are taken over the lane's own
// channels first, then by halving exchanges over the lanes K apart, over the
// block's four warps through shared memory, and over the channel tiles through
// one partial each, added by a second kernel.  The sums over a channel's states
// (y, du, ddelta) go by halving exchanges over its K lanes, which leave each lane
// with one of its four channels: that lane writes the channel's outputs.  All
// orders of summation are fixed.
//
// x, dt, dy and z of the next block come by asynchronous copies while this one
// is worked on, its checkpoint from the last piece on; every warp stages its own
// channels, one channel a lane, so that the warps meet only at the sums of dB
// and dC, once a block.
//
// Parallelism over tokens as in the forward: segments of equal length; a first
// launch runs each segment's part of the sequence that came in from the segment
// before, backwards from zero (or from dh_final where the sequence ends in it),
// and the segments behind a block's own are folded by the block or by a launch.
//
// What bounds it: issue slots, 526 a token of 32 channels (114 two-wide operations
// that hold the FMA pipe for two cycles, 32 of the special function unit, 62 loads,
// stores and exchanges), of which 62 % are used with the three warps a scheduler
// that 168 registers allow.  32768 tokens of 4096 channels: 2.82 ms; in fp32, whose
// 80 KB of shared memory a block leave room for two blocks, 3.38.  As many states in
// wider channels: 2048 of 32 3.04 ms, 1024 of 64 3.11.
#include "chunk_common.cuh"
#include "ssm_scan.cuh"

namespace gdn {
namespace {

constexpr int BT = kCkpt;  // tokens per block
constexpr int Q = 2;       // tokens per piece
constexpr int NS = 4;      // states per lane and channel
constexpr int P = 2;       // channel pairs per lane
constexpr int NC = 2 * P;  // channels per lane
constexpr int NW = 4;      // warps per block
constexpr int OCC = 3;     // blocks per SM: 168 registers a thread (fp32 up to 16 states: two, by shared memory)
constexpr int NT = 32 * NW;
static_assert(Q == 2 && kShifts % (BT / 2) == 0, "pieces are pairs of shifted decays");
constexpr float kLn2 = 0.6931471805599453f;

struct ScanBwdParams {
    const void* dy; int64_t lddy;
    const void* x; int64_t ldx;
    const void* dt; int64_t lddt;
    const void* z; int64_t ldz;
    const void* B; int64_t ldb;
    const void* C; int64_t ldc;
    const float* A_log; const float* D; const float* dt_bias; const float* h0; const float* ckpt; const float* dhf;
    const int32_t* cu;
    int num_seqs, T, ch, N, per, tiles;
    bool vec;  // states in pieces of four: N is a multiple of it and the caller's arrays are 16-byte aligned
    void* dx; void* ddt; void* dz; float* dh0;
    int seg, S;
    float* G; float* sd;   // [S, ch, N], [S, ch]: the segments' own start gradients and sums of delta
    float* bc;             // [groups * tiles, T, 2, N]: partial dB, dC
    float* par;            // [S, ch N + 2 ch]: partial dA_log, dD, ddt_bias
};

template <typename E, int K>
struct BShape {
    static constexpr int WC = NC * 32 / K;  // channels per warp
    static constexpr int CH = NW * WC;      // channels per block
    static constexpr int NP = NS * K;       // padded states
    // a warp's floats: delta, u, ds, slope, q1, x [BT][WC] each; the block's checkpoint and the states before its
    // other pieces [BT / Q][NC][32] float4
    static constexpr int AR = BT * WC;
    static constexpr int WARP = 6 * AR + BT / Q * NC * 32 * 4;
    static constexpr size_t raw_bytes = sizeof(E) * 4 * BT * CH;  // x, dt, dy, z as they come
    // B and C of two blocks, every value twice, [2][BT][4 NP]; the warps' dB and dC [NW][BT][2 NP]
    static constexpr size_t smem = 4 * (size_t)(NW * WARP + 2 * BT * 4 * NP + NW * BT * 2 * NP) + raw_bytes;
};

// Sums over a channel's K adjacent lanes of the lane's four channels; lane k ends
// with the sum of channel k % 4.
template <int K>
__device__ __forceinline__ float sum_states(float v0, float v1, float v2, float v3, int k) {
#pragma unroll
    for (int m = 4; m < K; m <<= 1) {
        v0 += __shfl_xor_sync(0xffffffffu, v0, m);
        v1 += __shfl_xor_sync(0xffffffffu, v1, m);
        v2 += __shfl_xor_sync(0xffffffffu, v2, m);
        v3 += __shfl_xor_sync(0xffffffffu, v3, m);
    }
    const bool b0 = k & 1, b1 = k & 2;
    const float s0 = b0 ? v0 : v1, s1 = b0 ? v2 : v3;
    float a = b0 ? v1 : v0, b = b0 ? v3 : v2;
    a += __shfl_xor_sync(0xffffffffu, s0, 1);
    b += __shfl_xor_sync(0xffffffffu, s1, 1);
    const float s2 = b1 ? a : b, c = b1 ? b : a;
    return c + __shfl_xor_sync(0xffffffffu, s2, 2);
}

// Sums over the warp's lanes K apart of eight values (two tokens x four states).
// Halves the values while lanes are left: the lane ends with kLeft8 of them, the
// first of index `first`.
template <int K>
constexpr int kLeft8 = K / 4;
template <int K>
__device__ __forceinline__ void sum_channels8(float (&v)[8], int lane, int& first) {
    first = 0;
    int cnt = 8;
#pragma unroll
    for (int m = K; m < 32; m <<= 1) {
        const bool up = lane & m;
        cnt >>= 1;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < cnt) {
                const float snd = up ? v[i] : v[i + cnt], kp = up ? v[i + cnt] : v[i];
                v[i] = kp + __shfl_xor_sync(0xffffffffu, snd, m);
            }
        if (up) first += cnt;
    }
}

// the lane's channels, in pairs
__device__ __forceinline__ void lds_pairs(F2 (&f)[P], const float* p) {
    f2_load2(p, f[0], f[1]);
}
// four values that lie there twice each
__device__ __forceinline__ void lds_dup(F2 (&f)[4], const float* p) {
    f2_load2(p, f[0], f[1]);
    f2_load2(p + 4, f[2], f[3]);
}

template <typename E, int K>
__global__ void __launch_bounds__(NT, OCC) scan_bwd_kernel(const ScanBwdParams p) {
    using Sh = BShape<E, K>;
    constexpr int WC = Sh::WC, CH = Sh::CH, NP = Sh::NP, AR = Sh::AR;
    constexpr int TPS = 32 / WC;  // tokens that a warp stages at a time, a channel a lane
    constexpr int VEC = 16 / sizeof(E), VR = WC / VEC;  // 16-byte vectors a row
    static_assert(K >= 4 && K <= 16 && NC == 4, "a lane's four channels spread over four lanes at least");
    extern __shared__ float4 smem4[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = lane % K, cg = lane / K;
    float* wb = reinterpret_cast<float*>(smem4) + warp * Sh::WARP;
    float *dl = wb, *uu = wb + AR, *dsv = wb + 2 * AR, *slope = wb + 3 * AR, *q1 = wb + 4 * AR, *xx = wb + 5 * AR;
    float4* hs = reinterpret_cast<float4*>(wb + 6 * AR);                       // [BT / Q][NC][32]
    float* bcs = reinterpret_cast<float*>(smem4) + NW * Sh::WARP;              // [2][BT][4 NP]
    float* slab = bcs + 2 * BT * 4 * NP;                                       // [NW][BT][2 NP]
    E* raw = reinterpret_cast<E*>(slab + NW * BT * 2 * NP) + warp * 4 * BT * WC;  // [x, dt, dy, z][BT][WC]
    const int grp = blockIdx.x / p.tiles, cend = (grp + 1) * p.per;
    const int wc0 = grp * p.per + (blockIdx.x % p.tiles) * CH + warp * WC;  // the warp's first channel
    const int c4 = wc0 + cg * NC;                                          // the lane's first channel
    const int s = blockIdx.y, t0 = s * p.seg, te = min(p.T, t0 + p.seg);

    // two channels side by side: delta, u and ds of both are one operand as they are read
    F2 A2[P][NS], dh[P][NS], h[P][NS], dA[P][NS];
    const bool vec = p.vec;
    auto load_state = [&](F2 (&f)[P][NS], const float* src, int64_t row) {  // src [rows, ch, N] or null
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = c4 + 2 * i;
            const bool in0 = src && c < cend, in1 = src && c + 1 < cend;
            const float* g = src + (row * p.ch + c) * p.N + k * NS;
            if (vec) {
                const bool ok = k * NS < p.N;
                const float4 z4 = make_float4(0.f, 0.f, 0.f, 0.f);
                const float4 v0 = ok && in0 ? __ldg(reinterpret_cast<const float4*>(g)) : z4;
                const float4 v1 = ok && in1 ? __ldg(reinterpret_cast<const float4*>(g + p.N)) : z4;
                f[i][0] = f2(v0.x, v1.x);
                f[i][1] = f2(v0.y, v1.y);
                f[i][2] = f2(v0.z, v1.z);
                f[i][3] = f2(v0.w, v1.w);
            } else {
#pragma unroll
                for (int n = 0; n < NS; ++n) {
                    const bool ok = k * NS + n < p.N;
                    f[i][n] = f2(ok && in0 ? __ldg(g + n) : 0.f, ok && in1 ? __ldg(g + p.N + n) : 0.f);
                }
            }
        }
    };
    auto store_state = [&](float* dst, int64_t row, const F2 (&f)[P][NS]) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = c4 + 2 * i;
            float* g = dst + (row * p.ch + c) * p.N + k * NS;
#pragma unroll
            for (int n = 0; n < NS; ++n)
                if (k * NS + n < p.N) {
                    if (c < cend) g[n] = f[i][n].x();
                    if (c + 1 < cend) g[p.N + n] = f[i][n].y();
                }
        }
    };
    auto scale_state = [&](F2 (&f)[P][NS], float v) {
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int n = 0; n < NS; ++n) f[i][n] = f2_mul(f[i][n], f2_dup(v));
    };
    auto pass_empty = [&](int m) {  // an empty sequence's final state is its initial one
        if (!p.dh0) return;
        F2 f[P][NS];
        load_state(f, p.dhf, m);
        store_state(p.dh0, m, f);
    };
    load_state(A2, p.A_log, 0);
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            const bool ok = k * NS + n < p.N;
            const int c = c4 + 2 * i;
            A2[i][n] = f2(ok && c < cend ? -expf(A2[i][n].x()) * kLog2e : 0.f,
                          ok && c + 1 < cend ? -expf(A2[i][n].y()) * kLog2e : 0.f);
            dh[i][n] = h[i][n] = dA[i][n] = f2_dup(0.f);
        }
    // the gradient of the state behind the segment's last token
    if (p.T > 0) {
        const int n = seq_of(p.cu, p.num_seqs, te - 1);
        const int end = __ldg(p.cu + n + 1);
        if (end <= te) {
            load_state(dh, p.dhf, n);
        } else {
            const int je = p.S > kFoldSegments ? s + 1 : (min(end, p.T) - 1) / p.seg;  // folded: the next row is all
            load_state(dh, p.G, je);
            for (int j = je - 1; j > s; --j) {
                F2 g[P][NS];
                load_state(g, p.G, j);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const int c = c4 + 2 * i;
                    const float* sd = p.sd + (int64_t)j * p.ch + c;
                    const F2 d = f2(c < cend ? __ldg(sd) : 0.f, c + 1 < cend ? __ldg(sd + 1) : 0.f);
#pragma unroll
                    for (int q = 0; q < NS; ++q) dh[i][q] = f2_fma(f2_exp2(f2_mul(d, A2[i][q])), dh[i][q], g[i][q]);
                }
            }
        }
        if (te == p.T)
            for (int m = n + 1; m < p.num_seqs; ++m) pass_empty(m);
    } else {
        for (int m = 0; m < p.num_seqs; ++m) pass_empty(m);
    }

    // the channel that this lane stages and the one whose outputs it writes
    const int sch = lane % WC, och = cg * NC + (k & 3);
    const bool writer = k < 4 && wc0 + och < cend;
    const float sbias = p.dt_bias && wc0 + sch < cend ? __ldg(p.dt_bias + wc0 + sch) : 0.f;
    const float Do = p.D && wc0 + och < cend ? __ldg(p.D + wc0 + och) : 0.f;
    float aD = 0.f, aT = 0.f, bD = 0.f, bT = 0.f;  // a block's sums b, added to the segment's: fewer terms in a row

    int cks = 0;  // the checkpoint that is in place
    auto copy = [&](int tb) {
#pragma unroll
        for (int it = lane; it < BT * VR; it += 32) {
            const int r = it / VR, v = it % VR;
            const bool ok = tb + r < te && wc0 + v * VEC < cend;
            const int64_t t = ok ? tb + r : t0;
            const int cv = ok ? wc0 + v * VEC : grp * p.per;
            E* d = raw + r * WC + v * VEC;
            const int bytes = ok ? 16 : 0;
            cp_async16(d, static_cast<const E*>(p.x) + t * p.ldx + cv, bytes);
            cp_async16(d + BT * WC, static_cast<const E*>(p.dt) + t * p.lddt + cv, bytes);
            cp_async16(d + 2 * BT * WC, static_cast<const E*>(p.dy) + t * p.lddy + cv, bytes);
            if (p.z) cp_async16(d + 3 * BT * WC, static_cast<const E*>(p.z) + t * p.ldz + cv, bytes);
        }
        cp_async_commit();
    };
    // the checkpoint before a block: each lane copies its own channels' states and reads them back
    const int ckq = c4 + NC <= cend ? NC : (c4 < cend ? cend - c4 : 0);  // its channels that exist
    auto fetch_state = [&](int tb) {
        if (vec) {
            const float* g = p.ckpt + ((int64_t)(tb / BT) * p.ch + (ckq ? c4 : 0)) * p.N;
            const bool ok = k * NS < p.N;
#pragma unroll
            for (int i = 0; i < NC; ++i)
                cp_async16(hs + i * 32 + lane, g + (i < ckq ? (int64_t)i * p.N : 0) + (ok ? k * NS : 0), ok && i < ckq ? 16 : 0);
        }
        cp_async_commit();
        cks = tb / BT;
    };
    auto block_state = [&]() {
        if (!vec) return load_state(h, p.ckpt, cks);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float4 v0 = hs[2 * i * 32 + lane], v1 = hs[(2 * i + 1) * 32 + lane];
            h[i][0] = f2(v0.x, v1.x);
            h[i][1] = f2(v0.y, v1.y);
            h[i][2] = f2(v0.z, v1.z);
            h[i][3] = f2(v0.w, v1.w);
        }
    };
    constexpr int PER = BT * 2 * NP / NT;
    E bc[PER];
    auto fetch_bc = [&](int tb) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int it = tid + i * NT, r = it / (2 * NP), j = it % (2 * NP), n = j % NP;
            const int64_t t = min(tb + r, te - 1);
            const E* q = (j < NP ? static_cast<const E*>(p.B) + t * p.ldb : static_cast<const E*>(p.C) + t * p.ldc) +
                         (int64_t)grp * p.N;
            bc[i] = n < p.N ? load_now(q + n) : Elem<E>::from_f(0.f);
        }
    };
    auto put_bc = [&](int b) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const float v = Elem<E>::to_f(bc[i]);
            reinterpret_cast<float2*>(bcs)[b * BT * 2 * NP + tid + i * NT] = make_float2(v, v);
        }
    };

    // a sequence starts at row r of the block: its initial state, scaled to where in a pair that is
    auto start_state = [&](int r, int tb, float up) {
        load_state(h, p.h0, seq_of(p.cu, p.num_seqs, tb + r));
        scale_state(h, up);
    };
    // the outputs of the lane's channel at row r of the block, from its sums over the states
    // (up, down: 2^s and 2^-s in the first rows of pairs)
    auto outputs = [&](int r, int tb, float dus, float dds, float y, float up, float down) {
        const int i = r * WC + och;
        if (writer && tb + r < te) {
            const int64_t off = (int64_t)(tb + r) * p.ch + wc0 + och;
            dus *= up;
            y *= down;
            const float g = dsv[i] * up, xv = xx[i];
            const float gd = fmaf(kLn2, dds, dus * xv) * slope[i];
            static_cast<E*>(p.dx)[off] = Elem<E>::from_f(fmaf(dus, dl[i], Do * g));
            static_cast<E*>(p.ddt)[off] = Elem<E>::from_f(gd);
            if (p.z) static_cast<E*>(p.dz)[off] = Elem<E>::from_f(fmaf(Do, xv, y) * q1[i]);
            bD = fmaf(g, xv, bD);
            bT += gd;
        }
    };

    const int nblk = (te - t0 + BT - 1) / BT;
    if (nblk > 0) {
        copy(t0 + (nblk - 1) * BT);
        fetch_state(t0 + (nblk - 1) * BT);
        fetch_bc(t0 + (nblk - 1) * BT);
        put_bc(0);
        __syncthreads();
    }
    int buf = 0;
    // the sequence that the walk is in, and its start
    int sq = nblk > 0 ? seq_of(p.cu, p.num_seqs, te - 1) : 0;
    int cur = nblk > 0 ? min(__ldg(p.cu + sq), te - 1) : -1;
    for (int b = nblk - 1; b >= 0; --b, buf ^= 1) {
        const int tb = t0 + b * BT;
        uint32_t starts = 0;  // which of the block's tokens start a sequence
        while (cur >= tb) {
            if (cur < te) starts |= 1u << (cur - tb);
            do --sq;
            while (sq >= 0 && __ldg(p.cu + sq) == cur);
            cur = sq >= 0 ? min(__ldg(p.cu + sq), cur - 1) : -1;
        }
        const int shift0 = tb / BT % (kShifts / (BT / 2)) * (BT / 2);  // the block's pairs' first shift
        cp_async_wait_all();
        __syncwarp();
        constexpr int SG = BT / TPS < 4 ? 2 : 4;  // a lane's tokens staged together
#pragma unroll
        for (int g0 = 0; g0 < BT; g0 += SG * TPS) {
            F2 vp[SG / 2], dp[SG / 2], et[SG / 2];  // v = dt + bias, delta, e^-|v|
#pragma unroll
            for (int m = 0; m < SG; m += 2) {
                const int i = (g0 + m * TPS) * WC + lane;
                vp[m / 2] = f2(Elem<E>::to_f(raw[BT * WC + i]) + sbias, Elem<E>::to_f(raw[BT * WC + i + 32]) + sbias);
                dp[m / 2] = vp[m / 2];
            }
            f2_softplus(dp, et);
#pragma unroll
            for (int m = 0; m < SG; ++m) {
                const int i = (g0 + m * TPS) * WC + lane, row = g0 + m * TPS + lane / WC;  // token row, channel sch
                const bool ok = tb + row < te;
                auto of = [&](const F2 (&f)[SG / 2]) { return m & 1 ? f[m / 2].y() : f[m / 2].x(); };
                const float xv = Elem<E>::to_f(raw[i]), gy = Elem<E>::to_f(raw[2 * BT * WC + i]), d = of(dp);
                float g = gy, qv = 0.f;
                if (p.z) {
                    const float zv = Elem<E>::to_f(raw[3 * BT * WC + i]), sg = sigmoid_fast(zv);
                    g = gy * (zv * sg);
                    qv = gy * sg * fmaf(zv, 1.f - sg, 1.f);
                }
                // the first rows of pairs, between whose tokens the state is 2^s times its value: u and ds to match
                const int pr = shift0 + row / 2;
                const float up = row & 1 ? 1.f : kShiftUp[pr], down = row & 1 ? 1.f : kShiftDown[pr];
                dl[i] = ok ? d : 0.f;
                uu[i] = ok ? d * xv * up : 0.f;
                dsv[i] = ok ? g * down : 0.f;
                const float v = of(vp), t = of(et);
                slope[i] = v > 20.f ? 1.f : (v < 0.f ? t : 1.f) * rcp_fast(1.f + t);  // the logistic function of v
                q1[i] = qv;
                xx[i] = xv;
            }
        }
        __syncwarp();
        if (b > 0) {
            copy(tb - BT);
            fetch_bc(tb - BT);
        }
        block_state();
        const float* bcb = bcs + buf * BT * 4 * NP + 2 * k * NS;
        const int co = cg * NC;
        // forward: the state before every piece
#pragma unroll 1
        for (int q = 0; q < BT / Q - 1; ++q) {
            const bool any = starts >> (q * Q) & (1u << Q) - 1;
            const float sh = kShift[shift0 + q], up = kShiftUp[shift0 + q];
#pragma unroll
            for (int e = 0; e < Q; ++e) {
                const int r = q * Q + e;
                if (any)
                    if (starts >> r & 1) start_state(r, tb, e ? up : 1.f);
                const F2 bi = f2_dup((e ? -sh : sh) + kDecayBias);
                F2 d[P], u[P], bb[NS];
                lds_pairs(d, dl + r * WC + co);
                lds_pairs(u, uu + r * WC + co);
                lds_dup(bb, bcb + r * 4 * NP);
#pragma unroll
                for (int i = 0; i < P; ++i)
#pragma unroll
                    for (int n = 0; n < NS; ++n) h[i][n] = f2_fma(u[i], bb[n], f2_mul(f2_decay(d[i], A2[i][n], bi), h[i][n]));
            }
#pragma unroll
            for (int i = 0; i < NC; ++i)
                f2_store2(hs + ((q + 1) * NC + i) * 32 + lane, h[i >> 1][(i & 1) * 2], h[i >> 1][(i & 1) * 2 + 1]);
        }
        // the pieces, last to first
#pragma unroll 1
        for (int q = BT / Q - 1; q >= 0; --q) {
            const bool any = starts >> (q * Q) & (1u << Q) - 1;
            const float sh = kShift[shift0 + q], up = kShiftUp[shift0 + q], down = kShiftDown[shift0 + q];
            F2 a[Q][P][NS], w[Q][P][NS];
            float ys[Q];
            if (q) {
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    f2_load2(reinterpret_cast<const float*>(hs + (q * NC + i) * 32 + lane), h[i >> 1][(i & 1) * 2],
                             h[i >> 1][(i & 1) * 2 + 1]);
            } else {
                block_state();
                if (b > 0) fetch_state(tb - BT);  // the slot is free, and the piece's work lies before the next block
            }
            float* sl = slab + warp * BT * 2 * NP + k * NS;
#pragma unroll
            for (int e2 = 0; e2 < Q; e2 += 2) {
                float v8[8];
                F2 yv[2][P];
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    const int e = e2 + o, r = q * Q + e;
                    if (any)
                        if (starts >> r & 1) start_state(r, tb, e ? up : 1.f);
                    const F2 bi = f2_dup((e ? -sh : sh) + kDecayBias);
                    F2 d[P], u[P], g[P], bb[NS], cc[NS], t[NS];
                    lds_pairs(d, dl + r * WC + co);
                    lds_pairs(u, uu + r * WC + co);
                    lds_pairs(g, dsv + r * WC + co);
                    lds_dup(bb, bcb + r * 4 * NP);
                    lds_dup(cc, bcb + r * 4 * NP + 2 * NP);
#pragma unroll
                    for (int i = 0; i < P; ++i)
#pragma unroll
                        for (int n = 0; n < NS; ++n) {
                            a[e][i][n] = f2_decay(d[i], A2[i][n], bi);
                            w[e][i][n] = f2_mul(a[e][i][n], h[i][n]);
                            h[i][n] = f2_fma(u[i], bb[n], w[e][i][n]);
                            t[n] = i ? f2_fma(g[i], h[i][n], t[n]) : f2_mul(g[i], h[i][n]);
                            yv[o][i] = n ? f2_fma(h[i][n], cc[n], yv[o][i]) : f2_mul(h[i][n], cc[n]);
                        }
#pragma unroll
                    for (int n = 0; n < NS; ++n) v8[4 * o + n] = f2_sum(t[n]);
                    ys[e] = sum_states<K>(yv[o][0].x(), yv[o][0].y(), yv[o][1].x(), yv[o][1].y(), k);
                }
                int first;
                sum_channels8<K>(v8, lane, first);
#pragma unroll
                for (int j = 0; j < kLeft8<K>; ++j)
                    sl[(q * Q + e2 + ((first + j) >> 2)) * 2 * NP + NP + ((first + j) & 3)] = v8[j];
            }
#pragma unroll
            for (int e2 = Q - 2; e2 >= 0; e2 -= 2) {
                float v8[8];
                F2 du[2][P], dd[2][P];
#pragma unroll
                for (int o = 1; o >= 0; --o) {
                    const int e = e2 + o, r = q * Q + e, t = tb + r;
                    F2 d[P], u[P], g[P], bb[NS], cc[NS], tt[NS];
                    lds_pairs(d, dl + r * WC + co);
                    lds_pairs(u, uu + r * WC + co);
                    lds_pairs(g, dsv + r * WC + co);
                    lds_dup(bb, bcb + r * 4 * NP);
                    lds_dup(cc, bcb + r * 4 * NP + 2 * NP);
#pragma unroll
                    for (int i = 0; i < P; ++i)
#pragma unroll
                        for (int n = 0; n < NS; ++n) {
                            dh[i][n] = f2_fma(g[i], cc[n], dh[i][n]);
                            tt[n] = i ? f2_fma(u[i], dh[i][n], tt[n]) : f2_mul(u[i], dh[i][n]);
                            du[o][i] = n ? f2_fma(dh[i][n], bb[n], du[o][i]) : f2_mul(dh[i][n], bb[n]);
                            const F2 m = f2_mul(dh[i][n], w[e][i][n]);
                            dA[i][n] = f2_fma(d[i], m, dA[i][n]);
                            dd[o][i] = n ? f2_fma(m, A2[i][n], dd[o][i]) : f2_mul(m, A2[i][n]);
                            dh[i][n] = f2_mul(dh[i][n], a[e][i][n]);
                        }
#pragma unroll
                    for (int n = 0; n < NS; ++n) v8[4 * o + n] = f2_sum(tt[n]);
                    if (any && (starts >> r & 1)) {  // the token starts a sequence: dh is the gradient of its h0
                        const int n = seq_of(p.cu, p.num_seqs, t);
                        if (e) scale_state(dh, up);
                        if (p.dh0) store_state(p.dh0, n, dh);
                        int m = n - 1;
                        while (m >= 0 && __ldg(p.cu + m) == t) pass_empty(m--);
                        load_state(dh, m >= 0 ? p.dhf : nullptr, m >= 0 ? m : 0);
                        if (e) scale_state(dh, down);
                    }
                    outputs(r, tb, sum_states<K>(du[o][0].x(), du[o][0].y(), du[o][1].x(), du[o][1].y(), k),
                            sum_states<K>(dd[o][0].x(), dd[o][0].y(), dd[o][1].x(), dd[o][1].y(), k), ys[e], e ? 1.f : up,
                            e ? 1.f : down);
                }
                int first;
                sum_channels8<K>(v8, lane, first);
#pragma unroll
                for (int j = 0; j < kLeft8<K>; ++j)
                    sl[(q * Q + e2 + ((first + j) >> 2)) * 2 * NP + ((first + j) & 3)] = v8[j];
            }
        }
        if (b > 0) put_bc(buf ^ 1);  // last read a block ago
        __syncthreads();
        // dB, dC of the block over its warps
        for (int it = tid; it < BT * 2 * NP; it += NT) {
            const int r = it / (2 * NP), j = it % (2 * NP), n = j % NP, which = j / NP;
            float sum = 0.f;
#pragma unroll
            for (int v = 0; v < NW; ++v) sum += slab[v * BT * 2 * NP + it];
            if (tb + r < te && n < p.N) p.bc[(((int64_t)blockIdx.x * p.T + tb + r) * 2 + which) * p.N + n] = sum;
        }
        __syncthreads();  // the slabs are read
        aD += bD;
        aT += bT;
        bD = bT = 0.f;
    }
    // the parameters' partial gradients of this segment
    float* pg = p.par + (int64_t)s * p.ch * (p.N + 2);
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int n = 0; n < NS; ++n) dA[i][n] = f2_mul(f2_mul(dA[i][n], A2[i][n]), f2_dup(kLn2));
    store_state(pg, 0, dA);
    if (writer) {
        pg[(int64_t)p.ch * p.N + wc0 + och] = aD;
        pg[(int64_t)p.ch * p.N + p.ch + wc0 + och] = aT;
    }
}

// dB, dC [T, groups, N] from the channel tiles' partials, in tile order
template <typename E>
__global__ void __launch_bounds__(256) scan_bc_kernel(const float* bc, int T, int groups, int tiles, int N, E* dB,
                                                      E* dC) {
    const int64_t per = (int64_t)T * 2 * N;  // one tile's partials
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= per * groups) return;
    const int g = (int)(i / per);
    const int64_t j = i - g * per;
    const float* src = bc + (int64_t)g * tiles * per + j;
    float s = 0.f;
    for (int k = 0; k < tiles; ++k) s += src[k * per];
    const int64_t t = j / (2 * N);
    const int rem = (int)(j - t * 2 * N), n = rem % N;
    E* out = rem < N ? dB : dC;
    out[(t * groups + g) * N + n] = Elem<E>::from_f(s);
}

int lanes_of(int N) { return N <= 16 ? 4 : (N <= 32 ? 8 : 16); }
int block_channels(int N) { return NW * NC * 32 / lanes_of(N); }

constexpr int64_t kMostSegments = 32768;  // a byte each in the fold's shared memory

// Segments: two waves of resident blocks (one wave leaves the launch before, whose
// blocks cover more channels, too few blocks to fill the SMs), of whole pairs of
// token blocks (71 tokens of 3584 channels: 54 us for both passes, 94 with segments of 64);
// more where they would be longer than kLongestSum.
// Returns the most segments that a call of up to T tokens has.
int segments(int T, int ch, int N, int groups, int& tiles, int& seg, int& S) {
    const int per = ch / groups, cb = block_channels(N);
    tiles = (per + cb - 1) / cb;
    const int64_t waves = (int64_t)device_sm_count() * OCC * 2 / ((int64_t)groups * tiles);
    const int64_t least = 2 * BT, most = (T + least - 1) / least;
    int64_t want = blocks_for_sum(T, waves > 1 ? waves : 1);
    if (want > most) want = most;
    if (want > kMostSegments) want = kMostSegments;
    if (want < 1) want = 1;
    seg = (int)(((T + want - 1) / want + 2 * BT - 1) / (2 * BT) * (2 * BT));
    if (seg < least) seg = least;
    S = (T + seg - 1) / seg;
    if (S < 1) S = 1;
    return (int)want;
}

struct Layout {
    size_t G, sd, bc, par, total;
};
Layout layout(int T, int ch, int N, int groups) {
    int tiles, seg, S;
    const int most = segments(T, ch, N, groups, tiles, seg, S);
    auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
    Layout L{};
    size_t o = 0;
    L.G = o; o += up(sizeof(float) * (size_t)most * ch * N);
    L.sd = o; o += up(sizeof(float) * (size_t)most * ch);
    L.bc = o; o += up(sizeof(float) * (size_t)groups * tiles * T * 2 * N);
    L.par = o; o += up(sizeof(float) * (size_t)most * ch * (N + 2));
    L.total = o;
    return L;
}

}  // namespace

gdn_status set_smem_attr(const void* func, size_t bytes);

namespace {

template <typename E, int K>
gdn_status run_bwd(const ScanBwdParams& p, int groups, cudaStream_t s) {
    using Sh = BShape<E, K>;
    const gdn_status st = set_smem_attr((const void*)scan_bwd_kernel<E, K>, Sh::smem);
    if (st != GDN_OK) return st;
    scan_bwd_kernel<E, K><<<dim3(groups * p.tiles, p.S), NT, Sh::smem, s>>>(p);
    return check_launch("scan_bwd_kernel");
}

template <typename E>
gdn_status dispatch_bwd(const ScanBwdParams& p, int groups, void* dB, void* dC, cudaStream_t s) {
    gdn_status st;
    switch (lanes_of(p.N)) {
        case 4: st = run_bwd<E, 4>(p, groups, s); break;
        case 8: st = run_bwd<E, 8>(p, groups, s); break;
        default: st = run_bwd<E, 16>(p, groups, s); break;
    }
    if (st != GDN_OK || p.T == 0) return st;
    const int64_t n = (int64_t)p.T * 2 * p.N * groups;
    scan_bc_kernel<E><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(p.bc, p.T, groups, p.tiles, p.N, static_cast<E*>(dB),
                                                                  static_cast<E*>(dC));
    return check_launch("scan_bc_kernel");
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_ssm_scan_bwd_workspace_size(int32_t T, int32_t channels, int32_t d_state, int32_t groups) {
    if (T < 0 || T > kMaxTokens || channels < 1 || groups < 1 || channels % groups || (channels / groups) % 8 ||
        d_state < 1 || d_state > 64)
        return 0;
    return layout(T, channels, d_state, groups).total;
}

gdn_status gdn_ssm_scan_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* dt, int64_t lddt,
                            const void* z, int64_t ldz, const void* B, int64_t ldb, const void* C, int64_t ldc,
                            gdn_dtype dtype, const float* A_log, const float* D, const float* dt_bias, const float* h0,
                            const float* ckpt, const float* dh_final, const int32_t* cu_seqlens, int32_t num_seqs,
                            int32_t T, int32_t channels, int32_t d_state, int32_t groups, void* dx, void* ddt, void* dz,
                            void* dB, void* dC, float* dA_log, float* dD, float* ddt_bias, float* dh0, void* workspace,
                            size_t workspace_bytes, void* stream) {
    gdn_status st = check_scan_shape(dtype, T, channels, d_state, groups);
    if (st != GDN_OK) return st;
    if (num_seqs < 1 || !cu_seqlens) return fail(GDN_ERR_INVALID_ARG, "num_seqs=%d or cu_seqlens is NULL", num_seqs);
    if (!A_log || !dA_log) return fail(GDN_ERR_INVALID_ARG, "A_log or dA_log is NULL");
    if (T > 0) {
        if ((st = check_scan_inputs(x, ldx, dt, lddt, z, ldz, B, ldb, C, ldc, A_log, channels, d_state, groups)) != GDN_OK)
            return st;
        if ((st = check_scan_row(dy, lddy, channels, "dy")) != GDN_OK) return st;
        if (!ckpt) return fail(GDN_ERR_INVALID_ARG, "ckpt is NULL");
        if (!dx || !ddt || !dB || !dC || (z && !dz)) return fail(GDN_ERR_INVALID_ARG, "a gradient output is NULL");
        if (!al16(dx) || !al16(ddt) || !al16(dz))
            return fail(GDN_ERR_INVALID_ARG, "dx, ddt and dz must be 16-byte aligned");
    }
    if (!al16(ckpt)) return fail(GDN_ERR_INVALID_ARG, "ckpt must be 16-byte aligned");
    if (dh_final && dh_final == dh0) return fail(GDN_ERR_INVALID_ARG, "dh0 must not be dh_final");
    const Layout L = layout(T, channels, d_state, groups);
    if (!workspace || workspace_bytes < L.total)
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes < required %zu", workspace ? workspace_bytes : 0,
                    L.total);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(GDN_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    char* ws = static_cast<char*>(workspace);
    ScanBwdParams p{};
    p.dy = dy; p.lddy = lddy; p.x = x; p.ldx = ldx; p.dt = dt; p.lddt = lddt; p.z = z; p.ldz = ldz; p.B = B; p.ldb = ldb;
    p.C = C; p.ldc = ldc; p.A_log = A_log; p.D = D; p.dt_bias = dt_bias; p.h0 = h0; p.ckpt = ckpt; p.dhf = dh_final;
    p.cu = cu_seqlens; p.num_seqs = num_seqs; p.T = T; p.ch = channels; p.N = d_state; p.per = channels / groups;
    p.dx = dx; p.ddt = ddt; p.dz = dz; p.dh0 = dh0;
    p.vec = d_state % 4 == 0 && al16(A_log) && al16(h0) && al16(dh_final);
    segments(T, channels, d_state, groups, p.tiles, p.seg, p.S);
    p.G = reinterpret_cast<float*>(ws + L.G);
    p.sd = reinterpret_cast<float*>(ws + L.sd);
    p.bc = reinterpret_cast<float*>(ws + L.bc);
    p.par = reinterpret_cast<float*>(ws + L.par);
    cudaStream_t s = (cudaStream_t)stream;
    if (T > 0) {
        ScanParams g{};
        g.x = dy; g.ldx = lddy; g.dt = dt; g.lddt = lddt; g.z = z; g.ldz = ldz; g.B = C; g.ldb = ldc; g.C = C; g.ldc = ldc;
        g.A_log = A_log; g.dt_bias = dt_bias; g.h0 = dh_final; g.cu = cu_seqlens; g.num_seqs = num_seqs; g.T = T;
        g.ch = channels; g.N = d_state; g.per = channels / groups; g.seg = p.seg; g.S = p.S; g.H = p.G; g.sd = p.sd;
        if ((st = launch_scan_start_grad(g, dtype, groups, s)) != GDN_OK) return st;
    }
    st = dtype == GDN_BF16 ? dispatch_bwd<__nv_bfloat16>(p, groups, dB, dC, s) : dispatch_bwd<float>(p, groups, dB, dC, s);
    if (st != GDN_OK) return st;
    const int64_t nA = (int64_t)channels * d_state;
    return launch_column_sum(p.par, p.S, nA + 2 * (int64_t)channels, nA, nA + channels, dA_log, dD, ddt_bias, s);
}

}  // extern "C"
