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
// The states before each token come from the forward's checkpoints (every 64
// packed tokens): a block of 64 tokens is run forward once, keeping the state
// at every eighth token in shared memory, then its eight-token pieces are
// taken from the last to the first: forward again with the eight states and
// decays in registers, then backward.  A channel's states are spread over K
// lanes with four each; the sums over a channel's lanes (y, du, ddelta) and the
// sums over channels (dB, dC) are halving exchanges within the warp, the latter
// go on over the block's warps through shared memory and over the blocks
// through one partial per channel tile, added by a second kernel.  All orders
// of summation are fixed.
//
// Parallelism over tokens as in the forward: segments of equal length; a first
// launch runs each segment's part of the sequence that came in from the segment
// before, backwards from zero (or from dh_final where the sequence ends in it),
// and a block of the main launch folds the segments behind its own.
#include "ssm_common.cuh"

namespace gdn {

gdn_status check_scan_shape(gdn_dtype dtype, int rows, int ch, int N, int groups);
gdn_status check_scan_row(const void* p, int64_t ld, int64_t least, const char* name);
gdn_status check_scan_inputs(const void* x, int64_t ldx, const void* dt, int64_t lddt, const void* z, int64_t ldz,
                             const void* B, int64_t ldb, const void* C, int64_t ldc, const float* A_log, int ch,
                             int N, int groups);

namespace {

constexpr int BT = 64;   // tokens per block (the checkpoints' spacing)
constexpr int Q = 8;     // tokens per piece
constexpr int NS = 4;    // states per lane
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
    void* dx; void* ddt; void* dz; float* dh0;
    int seg, S;
    float* G; float* sd;   // [S, ch, N], [S, ch]: the segments' own start gradients and sums of delta
    float* bc;             // [groups * tiles, T, 2, N]: partial dB, dC
    float* par;            // [S, ch N + 2 ch]: partial dA_log, dD, ddt_bias
};

template <int K>
struct BShape {
    static constexpr int CH = K <= 4 ? 64 : 256 / K;  // channels per block
    static constexpr int NT = CH * K;
    static constexpr int NW = NT / 32;
    static constexpr int CPW = 32 / K;
    static constexpr int NP = NS * K;
    static constexpr int VR = CH / 8;                 // 16-byte vectors (of bf16) per row
    // floats: delta, u, ds [BT][CH]; B, C [BT][NP]; states [BT / Q][NS][NT]; slabs [2][NW][Q][2 NP]
    static constexpr size_t words = 3 * BT * CH + 2 * BT * NP + BT / Q * NS * NT + 2 * NW * Q * 2 * NP;
    static constexpr size_t smem = 4 * words + 16;
    static constexpr size_t smem_summary = 4 * (2 * BT * CH + BT * NP) + 16;
};

// Sum over a channel's K adjacent lanes of four tokens' values; lane k (its two
// low bits) ends with token (k & 1) * 2 + (k >> 1 & 1) in v[0] (K >= 4), with
// tokens 2 k, 2 k + 1 in v[0], v[1] (K = 2).
template <int K>
__device__ __forceinline__ void sum_lanes4(float (&v)[4], int k) {
    if constexpr (K == 1) return;
    if constexpr (K > 4) {
#pragma unroll
        for (int m = 4; m < K; m <<= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
    }
    const bool b0 = k & 1;
    const float s0 = b0 ? v[0] : v[2], s1 = b0 ? v[1] : v[3];
    float k0 = b0 ? v[2] : v[0], k1 = b0 ? v[3] : v[1];
    k0 += __shfl_xor_sync(0xffffffffu, s0, 1);
    k1 += __shfl_xor_sync(0xffffffffu, s1, 1);
    if (K == 2) {
        v[0] = k0;
        v[1] = k1;
        return;
    }
    const bool b1 = k & 2;
    const float snd = b1 ? k0 : k1, kp = b1 ? k1 : k0;
    v[0] = kp + __shfl_xor_sync(0xffffffffu, snd, 2);
}
// which tokens of four the lane holds afterwards, and whether it is the one to store them
template <int K>
__device__ __forceinline__ void put_lanes4(float* row0, int64_t stride, const float (&v)[4], int k) {
    if (K == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) row0[i * stride] = v[i];
    } else if (K == 2) {
        row0[(2 * k) * stride] = v[0];
        row0[(2 * k + 1) * stride] = v[1];
    } else if (k < 4) {
        row0[((k & 1) * 2 + (k >> 1)) * stride] = v[0];
    }
}

// Sum of eight values (two tokens x four states) over the warp's channels
// (lanes K apart).  Halves the values while lanes are left, so the lane ends with
// 8 / min(8, CPW) of them, the first of index `first`; lanes whose channel bits
// beyond those are set hold copies.
template <int K>
__device__ __forceinline__ void sum_channels8(float (&v)[8], int lane, int& first, bool& keep) {
    first = 0;
    keep = true;
    int cnt = 8;
#pragma unroll
    for (int m = K; m < 32; m <<= 1) {
        const bool up = lane & m;
        if (cnt > 1) {
            cnt >>= 1;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < cnt) {
                    const float snd = up ? v[i] : v[i + cnt], kp = up ? v[i + cnt] : v[i];
                    v[i] = kp + __shfl_xor_sync(0xffffffffu, snd, m);
                }
            if (up) first += cnt;
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
            if (up) keep = false;
        }
    }
}
template <int K>
constexpr int kLeft8 = 32 / K >= 8 ? 1 : 8 * K / 32;

template <typename E, int K, bool SUMMARY>
__global__ void __launch_bounds__(BShape<K>::NT) scan_bwd_kernel(const ScanBwdParams p) {
    using Sh = BShape<K>;
    constexpr int CH = Sh::CH, NT = Sh::NT, NP = Sh::NP, CPW = Sh::CPW, VR = Sh::VR, NW = Sh::NW;
    extern __shared__ float4 smem4[];
    uint32_t* mask = reinterpret_cast<uint32_t*>(smem4);   // which of the block's tokens start a sequence
    float* dl = reinterpret_cast<float*>(smem4 + 1);       // [BT][CH] delta, then ddelta's sum over n
    float* ds = dl + BT * CH;                              // ds, then the sum C h
    float* Cs = ds + BT * CH;                              // [BT][NP]
    float* uu = Cs + BT * NP;                              // u, then du
    float* Bs = uu + BT * CH;
    float* hs = Bs + BT * NP;                              // [BT / Q][NS][NT]
    float* slab = hs + BT / Q * NS * NT;                   // [2][NW][Q][2 NP]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = lane % K;
    const int grp = blockIdx.x / p.tiles;
    const int cbase = grp * p.per + (blockIdx.x % p.tiles) * CH, cend = (grp + 1) * p.per;
    const int s = SUMMARY ? blockIdx.y + 1 : blockIdx.y;
    const int t0 = s * p.seg, te = min(p.T, t0 + p.seg);
    const int cl = warp * CPW + lane / K, c = cbase + cl;
    const bool cin = c < cend;
    float A2[NS], dh[NS], h[NS], dA[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        const int st = k * NS + n;
        A2[n] = cin && st < p.N ? -expf(__ldg(p.A_log + (int64_t)c * p.N + st)) * kLog2e : 0.f;
        dh[n] = h[n] = dA[n] = 0.f;
    }
    auto load_state = [&](float (&f)[NS], const float* src, int64_t row) {
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            const int st = k * NS + n;
            f[n] = src && cin && st < p.N ? __ldg(src + (row * p.ch + c) * p.N + st) : 0.f;
        }
    };
    auto store_state = [&](float* dst, int64_t row, const float (&f)[NS]) {
        if (!cin) return;
#pragma unroll
        for (int n = 0; n < NS; ++n)
            if (k * NS + n < p.N) dst[(row * p.ch + c) * p.N + k * NS + n] = f[n];
    };
    auto pass_empty = [&](int m) {  // an empty sequence's final state is its initial one
        if (!p.dh0) return;
        float f[NS];
        load_state(f, p.dhf, m);
        store_state(p.dh0, m, f);
    };
    // row vectors of the block: fixed columns per thread
    const int vcol = tid % VR, vrow = tid / VR;
    const int cv = cbase + 8 * vcol;
    const bool vin = cv < cend;
    float bias[8], Dv[8], aD[8], aT[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        bias[i] = vin && p.dt_bias ? __ldg(p.dt_bias + cv + i) : 0.f;
        Dv[i] = vin && p.D ? __ldg(p.D + cv + i) : 0.f;
        aD[i] = aT[i] = 0.f;
    }

    int first_t = t0;  // SUMMARY: the first token to take
    int last_t = te;   // one past the last
    float dsum = 0.f;
    if (SUMMARY) {
        const int n = seq_of(p.cu, p.num_seqs, t0);
        if (__ldg(p.cu + n) >= t0) return;  // nothing came in
        const int end = __ldg(p.cu + n + 1);
        if (end <= te) {
            last_t = max(end, t0);
            load_state(dh, p.dhf, n);
        }
    } else if (p.T > 0) {
        const int n = seq_of(p.cu, p.num_seqs, te - 1);
        const int end = __ldg(p.cu + n + 1);
        if (end <= te) {
            load_state(dh, p.dhf, n);
        } else {
            const int je = (min(end, p.T) - 1) / p.seg;
            for (int j = je; j > s; --j) {
                const float d = j < je && cin ? __ldg(p.sd + (int64_t)j * p.ch + c) : 0.f;
                float g[NS];
                load_state(g, p.G, j);
#pragma unroll
                for (int q = 0; q < NS; ++q) dh[q] = j == je ? g[q] : fmaf(exp2_fast(d * A2[q]), dh[q], g[q]);
            }
        }
        if (te == p.T)
            for (int m = n + 1; m < p.num_seqs; ++m) pass_empty(m);
    } else {
        for (int m = 0; m < p.num_seqs; ++m) pass_empty(m);
    }

    const int nblk = (last_t - t0 + BT - 1) / BT;
    int done = -1;  // token of the block whose sums wait in shared memory
    for (int b = nblk - 1; b >= -1; --b) {
        const int tb = t0 + b * BT;
        // the finished block's outputs, then the next block's inputs, row by row
        for (int r = vrow; r < BT; r += NT / VR) {
            const int i0 = r * CH + 8 * vcol;
            if (!SUMMARY && done >= 0 && vin && done + r < te) {
                const int64_t t = done + r;
                float xv[8], raw[8], gy[8], o[8], o2[8];
                load8(static_cast<const E*>(p.x) + t * p.ldx + cv, xv);
                load8(static_cast<const E*>(p.dt) + t * p.lddt + cv, raw);
                load8(static_cast<const E*>(p.dy) + t * p.lddy + cv, gy);
                float sil[8];
                if (p.z) {
                    float zv[8];
                    load8(static_cast<const E*>(p.z) + t * p.ldz + cv, zv);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float sg = sigmoid_fast(zv[i]);
                        sil[i] = zv[i] * sg;
                        o[i] = gy[i] * fmaf(Dv[i], xv[i], ds[i0 + i]) * sg * fmaf(zv[i], 1.f - sg, 1.f);
                    }
                    store8(static_cast<E*>(p.dz) + t * p.ch + cv, o);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) sil[i] = 1.f;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float v = raw[i] + bias[i], g = gy[i] * sil[i], du = uu[i0 + i];
                    const float delta = softplus_f(v);
                    o[i] = fmaf(du, delta, Dv[i] * g);
                    o2[i] = fmaf(kLn2, dl[i0 + i], du * xv[i]) * (v > 20.f ? 1.f : sigmoid_fast(v));
                    aD[i] = fmaf(g, xv[i], aD[i]);
                    aT[i] += o2[i];
                }
                store8(static_cast<E*>(p.dx) + t * p.ch + cv, o);
                store8(static_cast<E*>(p.ddt) + t * p.ch + cv, o2);
            }
            if (b >= 0) {
                const int64_t t = tb + r;
                float a[8], u[8], g[8];
                if (vin && t >= first_t && t < last_t) {
                    load8(static_cast<const E*>(p.dt) + t * p.lddt + cv, a);
#pragma unroll
                    for (int i = 0; i < 8; ++i) a[i] = softplus_f(a[i] + bias[i]);
                    load8(static_cast<const E*>(p.dy) + t * p.lddy + cv, g);
                    if (p.z) {
                        float zv[8];
                        load8(static_cast<const E*>(p.z) + t * p.ldz + cv, zv);
#pragma unroll
                        for (int i = 0; i < 8; ++i) g[i] *= silu_fast(zv[i]);
                    }
                    if (!SUMMARY) {
                        load8(static_cast<const E*>(p.x) + t * p.ldx + cv, u);
#pragma unroll
                        for (int i = 0; i < 8; ++i) u[i] *= a[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) a[i] = u[i] = g[i] = 0.f;
                }
                store8(dl + i0, a);
                store8(ds + i0, g);
                if (!SUMMARY) store8(uu + i0, u);
            }
        }
        if (b < 0) break;
        for (int it = tid; it < BT * NP; it += NT) {
            const int r = it / NP, n = it - r * NP;
            const int64_t t = tb + r;
            const bool in = t < last_t && n < p.N;
            const int64_t off = (int64_t)grp * p.N + n;
            Cs[it] = in ? Elem<E>::load(static_cast<const E*>(p.C) + t * p.ldc + off) : 0.f;
            if (!SUMMARY) Bs[it] = in ? Elem<E>::load(static_cast<const E*>(p.B) + t * p.ldb + off) : 0.f;
        }
        if (!SUMMARY && tid < BT) {
            const int t = tb + tid;
            const bool st = t < te && __ldg(p.cu + seq_of(p.cu, p.num_seqs, t)) == t;
            const uint32_t m = __ballot_sync(0xffffffffu, st);
            if (lane == 0) mask[warp] = m;
        }
        __syncthreads();
        if (SUMMARY) {
#pragma unroll 4
            for (int r = BT - 1; r >= 0; --r) {
                const float d = dl[r * CH + cl], g = ds[r * CH + cl];
                const float4 cv4 = *reinterpret_cast<const float4*>(Cs + r * NP + k * NS);
                const float cc[4] = {cv4.x, cv4.y, cv4.z, cv4.w};
#pragma unroll
                for (int n = 0; n < NS; ++n) dh[n] = fmaf(g, cc[n], dh[n]) * decay_fast(d, A2[n]);
                dsum += d;
            }
            __syncthreads();
            continue;
        }
        const uint64_t starts = (uint64_t)mask[0] | (uint64_t)mask[1] << 32;
        // forward over the block: the state before every piece
        load_state(h, p.ckpt, tb / BT);
        for (int q = 0; q < BT / Q; ++q) {
#pragma unroll
            for (int n = 0; n < NS; ++n) hs[(q * NS + n) * NT + tid] = h[n];
            if (q == BT / Q - 1) break;
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const int r = q * Q + i;
                if (starts >> r & 1) load_state(h, p.h0, seq_of(p.cu, p.num_seqs, tb + r));
                const float d = dl[r * CH + cl], u = uu[r * CH + cl];
                const float4 b4 = *reinterpret_cast<const float4*>(Bs + r * NP + k * NS);
                const float bb[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                for (int n = 0; n < NS; ++n) h[n] = fmaf(decay_fast(d, A2[n]), h[n], u * bb[n]);
            }
        }
        // the pieces, last to first
        for (int q = BT / Q - 1; q >= 0; --q) {
            float* sl = slab + ((q & 1) * NW + warp) * Q * 2 * NP;
            float a[Q][NS], hb[Q][NS], ys[2][4];
#pragma unroll
            for (int n = 0; n < NS; ++n) h[n] = hs[(q * NS + n) * NT + tid];
#pragma unroll
            for (int i2 = 0; i2 < Q; i2 += 2) {
                float v8[8];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = i2 + e, r = q * Q + i;
                    if (starts >> r & 1) load_state(h, p.h0, seq_of(p.cu, p.num_seqs, tb + r));
                    const float d = dl[r * CH + cl], u = uu[r * CH + cl], g = ds[r * CH + cl];
                    const float4 b4 = *reinterpret_cast<const float4*>(Bs + r * NP + k * NS);
                    const float4 c4 = *reinterpret_cast<const float4*>(Cs + r * NP + k * NS);
                    const float bb[4] = {b4.x, b4.y, b4.z, b4.w}, cc[4] = {c4.x, c4.y, c4.z, c4.w};
                    float acc = 0.f;
#pragma unroll
                    for (int n = 0; n < NS; ++n) {
                        a[i][n] = decay_fast(d, A2[n]);
                        hb[i][n] = h[n];
                        h[n] = fmaf(a[i][n], h[n], u * bb[n]);
                        acc = fmaf(h[n], cc[n], acc);
                        v8[4 * e + n] = cin ? g * h[n] : 0.f;
                    }
                    ys[i >> 2][i & 3] = acc;
                }
                int first;
                bool keep;
                sum_channels8<K>(v8, lane, first, keep);
                if (keep)
#pragma unroll
                    for (int j = 0; j < kLeft8<K>; ++j) {
                        const int idx = first + j;
                        sl[(i2 + (idx >> 2)) * 2 * NP + NP + k * NS + (idx & 3)] = v8[j];
                    }
            }
            sum_lanes4<K>(ys[0], k);
            sum_lanes4<K>(ys[1], k);
            float du4[4], dd4[4];
#pragma unroll
            for (int i2 = Q - 2; i2 >= 0; i2 -= 2) {
                float v8[8];
#pragma unroll
                for (int e = 1; e >= 0; --e) {
                    const int i = i2 + e, r = q * Q + i;
                    const float d = dl[r * CH + cl], u = uu[r * CH + cl], g = ds[r * CH + cl];
                    const float4 b4 = *reinterpret_cast<const float4*>(Bs + r * NP + k * NS);
                    const float4 c4 = *reinterpret_cast<const float4*>(Cs + r * NP + k * NS);
                    const float bb[4] = {b4.x, b4.y, b4.z, b4.w}, cc[4] = {c4.x, c4.y, c4.z, c4.w};
                    float du = 0.f, dd = 0.f;
#pragma unroll
                    for (int n = 0; n < NS; ++n) {
                        dh[n] = fmaf(g, cc[n], dh[n]);
                        v8[4 * e + n] = cin ? dh[n] * u : 0.f;
                        du = fmaf(dh[n], bb[n], du);
                        dh[n] *= a[i][n];
                        const float m = dh[n] * hb[i][n];
                        dd = fmaf(A2[n], m, dd);
                        dA[n] = fmaf(d, m, dA[n]);
                    }
                    du4[i & 3] = du;
                    dd4[i & 3] = dd;
                    if (starts >> r & 1) {  // the token starts a sequence: dh is the gradient of its h0
                        const int t = tb + r, n = seq_of(p.cu, p.num_seqs, t);
                        if (p.dh0) store_state(p.dh0, n, dh);
                        int m = n - 1;
                        while (m >= 0 && __ldg(p.cu + m) == t) pass_empty(m--);
                        load_state(dh, m >= 0 ? p.dhf : nullptr, m >= 0 ? m : 0);
                    }
                }
                int first;
                bool keep;
                sum_channels8<K>(v8, lane, first, keep);
                if (keep)
#pragma unroll
                    for (int j = 0; j < kLeft8<K>; ++j) {
                        const int idx = first + j;
                        sl[(i2 + (idx >> 2)) * 2 * NP + k * NS + (idx & 3)] = v8[j];
                    }
                if ((i2 & 2) == 0) {  // four tokens are done: their inputs are dead, their sums take the place
                    sum_lanes4<K>(du4, k);
                    sum_lanes4<K>(dd4, k);
                    const int r = q * Q + i2;
                    put_lanes4<K>(uu + r * CH + cl, CH, du4, k);
                    put_lanes4<K>(dl + r * CH + cl, CH, dd4, k);
                    put_lanes4<K>(ds + r * CH + cl, CH, ys[i2 >> 2], k);
                }
            }
            __syncthreads();
            // dB, dC of the piece over the block's warps
            for (int it = tid; it < Q * 2 * NP; it += NT) {
                const int i = it / (2 * NP), j = it - i * 2 * NP, n = j % NP, which = j / NP;
                const int64_t t = tb + q * Q + i;
                if (t < te && n < p.N) {
                    const float* sp = slab + (q & 1) * NW * Q * 2 * NP + it;
                    float sum = 0.f;
#pragma unroll
                    for (int w = 0; w < NW; ++w) sum += sp[w * Q * 2 * NP];
                    p.bc[(((int64_t)blockIdx.x * p.T + t) * 2 + which) * p.N + n] = sum;
                }
            }
        }
        done = tb;
    }
    if (SUMMARY) {
        store_state(p.G, s, dh);
        if (k == 0 && cin) p.sd[(int64_t)s * p.ch + c] = dsum;
        return;
    }
    // the parameters' partial gradients of this segment
    float* par = p.par + (int64_t)s * p.ch * (p.N + 2);
    if (cin)
#pragma unroll
        for (int n = 0; n < NS; ++n)
            if (k * NS + n < p.N) par[(int64_t)c * p.N + k * NS + n] = dA[n] * A2[n] * kLn2;
    __syncthreads();
    float* red = dl;  // [2][NT / VR][CH]: the tiles are dead
    constexpr int RR = NT / VR;
    static_assert(2 * RR * CH <= 2 * BT * CH + BT * NP, "the partial sums lie in the tiles' place");
    store8(red + vrow * CH + 8 * vcol, aD);
    store8(red + (RR + vrow) * CH + 8 * vcol, aT);
    __syncthreads();
    for (int i = tid; i < 2 * CH; i += NT) {
        const int cc = i % CH;
        const float* src = i < CH ? red : red + RR * CH;
        float sum = 0.f;
        for (int r = 0; r < RR; ++r) sum += src[r * CH + cc];
        if (cbase + cc < cend) par[(int64_t)p.ch * p.N + (i < CH ? 0 : p.ch) + cbase + cc] = sum;
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

int lanes_of(int N) {
    int K = 1;
    while (4 * K < N) K <<= 1;
    return K;
}
int block_channels(int N) {
    const int K = lanes_of(N);
    return K <= 4 ? 64 : 256 / K;
}

// Segments: enough blocks for two resident ones an SM, 64 tokens or more.
void segments(int T, int ch, int N, int groups, int& tiles, int& seg, int& S) {
    const int per = ch / groups, cb = block_channels(N);
    tiles = (per + cb - 1) / cb;
    int64_t want = (int64_t)device_sm_count() * 2 / ((int64_t)groups * tiles);
    const int64_t most = (T + 63) / 64;
    if (want > most) want = most;
    if (want < 1) want = 1;
    seg = (int)(((T + want - 1) / want + 63) / 64 * 64);
    if (seg < 64) seg = 64;
    S = (T + seg - 1) / seg;
    if (S < 1) S = 1;
}

struct Layout {
    size_t G, sd, bc, par, total;
};
Layout layout(int T, int ch, int N, int groups) {
    int tiles, seg, S;
    segments(T, ch, N, groups, tiles, seg, S);
    auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
    Layout L{};
    size_t o = 0;
    L.G = o; o += up(sizeof(float) * (size_t)S * ch * N);
    L.sd = o; o += up(sizeof(float) * (size_t)S * ch);
    L.bc = o; o += up(sizeof(float) * (size_t)groups * tiles * T * 2 * N);
    L.par = o; o += up(sizeof(float) * (size_t)S * ch * (N + 2));
    L.total = o;
    return L;
}

}  // namespace

gdn_status set_smem_attr(const void* func, size_t bytes);

namespace {

template <typename E, int K>
gdn_status run_bwd(const ScanBwdParams& p, int groups, cudaStream_t s) {
    using Sh = BShape<K>;
    gdn_status st = set_smem_attr((const void*)scan_bwd_kernel<E, K, false>, Sh::smem);
    if (st != GDN_OK) return st;
    if ((st = set_smem_attr((const void*)scan_bwd_kernel<E, K, true>, Sh::smem_summary)) != GDN_OK) return st;
    dim3 grid(groups * p.tiles, p.S);
    if (p.S > 1) {
        dim3 g1(grid.x, p.S - 1);
        scan_bwd_kernel<E, K, true><<<g1, Sh::NT, Sh::smem_summary, s>>>(p);
        if ((st = check_launch("scan_bwd_kernel (start gradients)")) != GDN_OK) return st;
    }
    scan_bwd_kernel<E, K, false><<<grid, Sh::NT, Sh::smem, s>>>(p);
    return check_launch("scan_bwd_kernel");
}

template <typename E>
gdn_status dispatch_bwd(const ScanBwdParams& p, int groups, void* dB, void* dC, cudaStream_t s) {
    gdn_status st;
    switch (lanes_of(p.N)) {
        case 1: st = run_bwd<E, 1>(p, groups, s); break;
        case 2: st = run_bwd<E, 2>(p, groups, s); break;
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
    if (T < 0 || channels < 1 || groups < 1 || channels % groups || (channels / groups) % 8 || d_state < 1 ||
        d_state > 64)
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
    segments(T, channels, d_state, groups, p.tiles, p.seg, p.S);
    p.G = reinterpret_cast<float*>(ws + L.G);
    p.sd = reinterpret_cast<float*>(ws + L.sd);
    p.bc = reinterpret_cast<float*>(ws + L.bc);
    p.par = reinterpret_cast<float*>(ws + L.par);
    cudaStream_t s = (cudaStream_t)stream;
    st = dtype == GDN_BF16 ? dispatch_bwd<__nv_bfloat16>(p, groups, dB, dC, s) : dispatch_bwd<float>(p, groups, dB, dC, s);
    if (st != GDN_OK) return st;
    const int64_t nA = (int64_t)channels * d_state;
    return launch_column_sum(p.par, p.S, nA + 2 * (int64_t)channels, nA, nA + channels, dA_log, dD, ddt_bias, s);
}

}  // extern "C"
