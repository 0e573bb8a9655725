// Selective state space scan: the forward over packed prompts and the
// single-token step.
//
// Per channel with N diagonal states (fp32 throughout):
//   delta = softplus(dt + dt_bias), a_n = 2^(delta A2_n), A2 = -exp(A_log) log2 e,
//   h_n <- a_n h_n + (delta x) B_n,   y = (sum_n C_n h_n + D x) silu(z).
//
// Work split.  A lane holds up to 16 states of one channel in registers, so that
// for N <= 16 a warp is 32 channels side by side and nothing crosses lanes: the
// lane reads its channel's x, dt and z, forms delta, runs the recurrence and
// stores y.  Above 16 states K = 2 or 4 adjacent lanes share a channel and add
// their sums by exchanges.  x, dt and z come by 16-byte asynchronous copies into
// a ring of three tiles of TT tokens in shared memory, so that two tiles are
// under way without holding registers; B and C, which all channels of a group
// read, are laid beside them as fp32 and come back as broadcasts.
//
// What bounds it: issue slots and the FMA pipe.  A token of 32 channels takes 108
// slots (70 in the launch that keeps end states only): 37 two-wide operations, which
// hold the FMA pipe for two cycles each, 19 of the special function unit (16 decays; 4
// cycles each), 13 loads and stores, and the rest of delta, u and the SiLU.  63 % of
// the slots are used with the four warps a scheduler that 128 registers allow (fp32:
// the ring leaves room for two blocks an SM with 9 to 16 states, three below).  Pairs
// of states, and of tokens in delta and the SiLU, go through the two-wide fp32
// instructions, without which the slots would be 37 more.  32768 tokens of 4096
// channels in prompts of 512 to 8192: 0.90 ms, of which the first launch 0.34 and the
// main one 0.55; two channels a lane were no faster.  In fp32 1.05 ms (0.37 and 0.66).
// As many states in wider ones: 2048 channels of 32 states 1.03 ms, 1024 of 64 1.63.
//
// Parallelism over tokens.  The packed tokens are cut into S segments of equal
// length, whatever the sequences' lengths.  A first launch runs each segment's
// part of the sequence that goes on into the next segment from a zero state (or
// from h0 where the sequence starts in it), keeping only the end state H and
// the sum of delta; from the first token of a segment that continues a
// sequence, the state is the fold  h <- 2^(A2 sum delta_j) h + H_j  over the
// segments before it.  Up to kFoldSegments segments each block of the main launch
// folds for its own channels; above, a launch between the two does, one thread a
// channel and state.
#include "chunk_common.cuh"
#include "ssm_scan.cuh"

namespace gdn {

gdn_status set_smem_attr(const void* func, size_t bytes);

namespace {

constexpr int TT = 16;     // tokens per tile
constexpr int UN = 8;      // tokens handled together (pairs of them, see kShift)
static_assert(kCkpt % UN == 0 && TT % kCkpt == 0, "checkpoints fall on the groups' starts");
constexpr int NST = 3;     // tiles of x, dt and z in flight or in use
constexpr int NTH = 128;   // threads per block

template <typename E, int K, int NS, int MODE>
__global__ void __launch_bounds__(NTH, 4) scan_kernel(const ScanParams p) {
    constexpr bool LAST = MODE != SCAN_FULL;  // a state and the sum of delta only: no y, no C
    constexpr bool REV = MODE == SCAN_START_GRAD;
    constexpr int NP = K * NS, CH = NTH / K, NB = LAST ? NP : 2 * NP;  // B, or B and C, per token
    constexpr int PER = (TT * NB + NTH - 1) / NTH;                    // elements of a tile each thread stages
    constexpr int NA = MODE == SCAN_END ? 2 : 3;                      // arrays in the ring
    extern __shared__ float4 smem4[];
    const int tid = threadIdx.x, k = tid % K, cl = tid / K;
    const int grp = blockIdx.x / p.tiles;
    const int cend = (grp + 1) * p.per;
    const int c = grp * p.per + (blockIdx.x % p.tiles) * CH + cl;
    const bool in = c < cend;
    const int cc = in ? c : cend - 1;  // a channel to read for lanes without one
    const int s = REV ? blockIdx.y + 1 : blockIdx.y;
    int t0 = s * p.seg, te = min(p.T, t0 + p.seg);
    E* yp = static_cast<E*>(p.y) + cc;
    const bool gate = MODE != SCAN_END && p.z;
    const float bias = p.dt_bias ? __ldg(p.dt_bias + cc) : 0.f, Dc = p.D ? __ldg(p.D + cc) : 0.f;
    // the ring: [NST][x, dt, z][TT][CH]
    E* ring = reinterpret_cast<E*>(smem4);
    float* bcs = reinterpret_cast<float*>(ring + NST * NA * TT * CH);  // [2][TT][NB]
    constexpr int VEC = 16 / sizeof(E), VR = CH / VEC;  // 16-byte vectors a row
    const int c0 = grp * p.per + (blockIdx.x % p.tiles) * CH;
    // row j of the walk is token t0 + j, or te - 1 - j backwards
    int len = te - t0;
    auto tok = [&](int j) { return (int64_t)(REV ? te - 1 - j : t0 + j); };
    auto copy = [&](int jb, int st) {
        if (jb < len) {
#pragma unroll
            for (int it = tid; it < TT * VR; it += NTH) {
                const int r = it / VR, v = it - r * VR;
                const bool ok = jb + r < len && c0 + v * VEC < cend;
                const int64_t t = ok ? tok(jb + r) : t0;
                const int cv = ok ? c0 + v * VEC : c0;
                E* d = ring + (st * NA * TT + r) * CH + v * VEC;
                const int bytes = ok ? 16 : 0;
                cp_async16(d, static_cast<const E*>(p.x) + t * p.ldx + cv, bytes);
                cp_async16(d + TT * CH, static_cast<const E*>(p.dt) + t * p.lddt + cv, bytes);
                if (gate) cp_async16(d + 2 * TT * CH, static_cast<const E*>(p.z) + t * p.ldz + cv, bytes);
            }
        }
        cp_async_commit();
    };
    E bc[PER];
    const int64_t goff = (int64_t)grp * p.N;
    auto fetch_bc = [&](int jb) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int it = tid + i * NTH, r = it / NB, j = it % NB, n = j % NP;
            const int64_t t = tok(min(jb + r, len - 1));
            const E* q = (j < NP ? static_cast<const E*>(p.B) + t * p.ldb : static_cast<const E*>(p.C) + t * p.ldc) + goff;
            bc[i] = it < TT * NB && n < p.N ? load_now(q + n) : Elem<E>::from_f(0.f);
        }
    };
    auto put_bc = [&](int b) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int it = tid + i * NTH;
            if (it < TT * NB) bcs[b * TT * NB + it] = Elem<E>::to_f(bc[i]);
        }
    };
    // the first tiles' copies start here, before the loads that the state's start needs; a launch for the segments'
    // ends learns there where it begins
    auto first_tiles = [&]() {
        fetch_bc(0);
#pragma unroll
        for (int i = 0; i < NST - 1; ++i) copy(i * TT, i);
    };
    if (!LAST && p.T > 0) first_tiles();
    F2 A2[NS / 2], h[NS / 2];
#pragma unroll
    for (int q = 0; q < NS / 2; ++q) {
        const int st = k * NS + 2 * q;
        const float* g = p.A_log + (int64_t)cc * p.N + st;
        A2[q] = f2(st < p.N ? -expf(__ldg(g)) * kLog2e : 0.f, st + 1 < p.N ? -expf(__ldg(g + 1)) * kLog2e : 0.f);
        h[q] = f2_dup(0.f);
    }
    const bool vec = p.N % 4 == 0;
    auto load_state = [&](const float* src, int64_t row) {  // src [rows, ch, N] or null
        const float* g = src + (row * p.ch + cc) * p.N + k * NS;
#pragma unroll
        for (int q = 0; q < NS / 2; ++q) {
            const int st = k * NS + 2 * q;
            h[q] = f2(src && st < p.N ? __ldg(g + 2 * q) : 0.f, src && st + 1 < p.N ? __ldg(g + 2 * q + 1) : 0.f);
        }
    };
    auto store_state = [&](float* dst, int64_t row) {
        float* g = dst + (row * p.ch + cc) * p.N + k * NS;
        if (!in) return;
#pragma unroll
        for (int q = 0; q < NS / 2; q += 2) {
            const int st = k * NS + 2 * q;
            if (vec) {
                if (st < p.N) f2_store2(g + 2 * q, h[q], h[q + 1]);
            } else {
                if (st < p.N) g[2 * q] = h[q].x();
                if (st + 1 < p.N) g[2 * q + 1] = h[q].y();
                if (st + 2 < p.N) g[2 * q + 2] = h[q + 1].x();
                if (st + 3 < p.N) g[2 * q + 3] = h[q + 1].y();
            }
        }
    };
    // the sequence at the first token, and the state there
    int next = 0x7fffffff;  // first token of the next sequence
    // sum of delta: a tile's, and all before it with what its additions lost, since an exponent made of thousands of
    // terms added one by one would be off by a few of its last digits
    float dsum = 0.f, dall = 0.f, dlost = 0.f;
    if (REV) {
        const int n = seq_of(p.cu, p.num_seqs, t0);
        if (__ldg(p.cu + n) >= t0) return;  // nothing came in
        const int end = __ldg(p.cu + n + 1);
        if (end <= te) {
            te = max(end, t0 + 1);
            load_state(p.h0, n);
        }
    } else if (LAST) {
        const int n = seq_of(p.cu, p.num_seqs, te - 1);
        if (__ldg(p.cu + n + 1) <= te) return;  // nothing goes on into the next segment
        const int start = __ldg(p.cu + n);
        if (start >= t0) {
            t0 = min(start, te - 1);
            load_state(p.h0, n);
        }
    } else {
        if (p.T == 0) {  // every sequence is empty
            if (p.h_final)
                for (int m = 0; m < p.num_seqs; ++m) {
                    load_state(p.h0, m);
                    store_state(p.h_final, m);
                }
            return;
        }
        const int n = seq_of(p.cu, p.num_seqs, t0);
        const int start = __ldg(p.cu + n);
        next = __ldg(p.cu + n + 1);
        if (start >= t0) {
            if (p.h_final)  // empty sequences that end where this segment starts
                for (int m = n - 1; m >= 0 && __ldg(p.cu + m) == t0; --m) {
                    load_state(p.h0, m);
                    store_state(p.h_final, m);
                }
            load_state(p.h0, n);
        } else if (p.folded) {
            load_state(p.H, s - 1);
        } else {
            const int j0 = max(start, 0) / p.seg;
            load_state(p.H, j0);
            for (int j = j0 + 1; j < s; ++j) {
                const int64_t row = (int64_t)j * p.ch + cc;
                const F2 d = f2_dup(__ldg(p.sd + row));
                const float* Hj = p.H + row * p.N + k * NS;
#pragma unroll
                for (int q = 0; q < NS / 2; ++q) {
                    const F2 add = f2(k * NS + 2 * q < p.N ? __ldg(Hj + 2 * q) : 0.f,
                                      k * NS + 2 * q + 1 < p.N ? __ldg(Hj + 2 * q + 1) : 0.f);
                    h[q] = f2_fma(f2_exp2(f2_mul(d, A2[q])), h[q], add);  // one exponential for the whole segment
                }
            }
        }
    }

    // one token: state and y; shift: of its decays; u and the sum that makes y come scaled to what the state is
    auto token = [&](const float* row, float dlt, float u, float xv, float sil, float shift, float down, E* yo) {
        const F2 d = f2_dup(dlt), uu = f2_dup(u), bi = f2_dup(shift);
        F2 acc[2];
#pragma unroll
        for (int q = 0; q < NS / 2; q += 2) {
            F2 b0, b1;
            f2_load2(row + 2 * q, b0, b1);
            if (REV) {
                h[q] = f2_mul(f2_decay(d, A2[q], bi), f2_fma(uu, b0, h[q]));
                h[q + 1] = f2_mul(f2_decay(d, A2[q + 1], bi), f2_fma(uu, b1, h[q + 1]));
            } else {
                h[q] = f2_fma(f2_decay(d, A2[q], bi), h[q], f2_mul(uu, b0));
                h[q + 1] = f2_fma(f2_decay(d, A2[q + 1], bi), h[q + 1], f2_mul(uu, b1));
            }
            if (!LAST) {
                F2 c0, c1;
                f2_load2(row + NP + 2 * q, c0, c1);
                acc[0] = q ? f2_fma(h[q], c0, acc[0]) : f2_mul(h[q], c0);
                acc[1] = q ? f2_fma(h[q + 1], c1, acc[1]) : f2_mul(h[q + 1], c1);
            }
        }
        if (LAST) {
            dsum += dlt;
        } else {
            float o = f2_sum(acc[0]) + f2_sum(acc[1]);
#pragma unroll
            for (int m = 1; m < K; m <<= 1) o += __shfl_xor_sync(0xffffffffu, o, m);
            o = fmaf(o, down, Dc * xv);
            if (gate) o *= sil;
            if (in && k == 0) *yo = Elem<E>::from_f(o);
        }
    };
    if (LAST) {
        len = te - t0;
        first_tiles();
    }
    put_bc(0);
    int buf = 0, st = 0;
    for (int jb = 0; jb < len; jb += TT, buf ^= 1, st = st == NST - 1 ? 0 : st + 1) {
        cp_async_wait<NST - 2>();
        __syncthreads();  // this tile's copies are in; the last tile's readers are done
        copy(jb + (NST - 1) * TT, st == 0 ? NST - 1 : st - 1);
        const bool more = jb + TT < len;
        if (more) fetch_bc(jb + TT);
        const E* xs = ring + st * NA * TT * CH + cl;
#pragma unroll  // whole tiles: the shifts are then operands of instructions (eight tokens together too: 1029 -> 890 us)
        for (int r0 = 0; r0 < TT; r0 += UN) {
            const int jg = jb + r0, tg = t0 + jg;  // tg: the first of the group's tokens (forwards)
            if (jg >= len) break;
            if (!LAST && p.ckpt && tg % kCkpt == 0) store_state(p.ckpt, tg / kCkpt);
            const float* row = bcs + (buf * TT + r0) * NB + k * NS;
            const E* xg = xs + r0 * CH;
            E* yo = yp + (int64_t)tg * p.ldy;
            if (jg + UN <= len && next >= tg + UN) {
                float dl[UN], sil[UN];
                F2 dp[UN / 2], et[UN / 2];
#pragma unroll
                for (int u = 0; u < UN; u += 2)
                    dp[u / 2] = f2(Elem<E>::to_f(xg[(TT + u) * CH]) + bias, Elem<E>::to_f(xg[(TT + u + 1) * CH]) + bias);
                f2_softplus(dp, et);
#pragma unroll
                for (int u = 0; u < UN; ++u) dl[u] = u & 1 ? dp[u / 2].y() : dp[u / 2].x();
#pragma unroll
                for (int u = 0; u < UN; u += 2) {
                    F2 g = f2_dup(1.f);
                    if (gate) g = f2_silu(f2(Elem<E>::to_f(xg[(2 * TT + u) * CH]), Elem<E>::to_f(xg[(2 * TT + u + 1) * CH])));
                    sil[u] = g.x();
                    sil[u + 1] = g.y();
                }
#pragma unroll
                for (int u = 0; u < UN; ++u) {
                    // pairs: the state is 2^s times its value behind the first token (kShift)
                    const int pr = (r0 + u) / 2 % kShifts;
                    const float xv = Elem<E>::to_f(xg[u * CH]);
                    float ut = (REV ? sil[u] : dl[u]) * xv;
                    if ((u & 1) == (REV ? 1 : 0)) ut *= kShiftUp[pr];  // backwards it enters before the decay
                    token(row + u * NB, dl[u], ut, xv, sil[u], (u & 1 ? -kShift[pr] : kShift[pr]) + kDecayBias,
                          u & 1 ? 1.f : kShiftDown[pr], yo + u * p.ldy);
                }
            } else {  // a sequence's end or the segment's is near: one by one
#pragma unroll 1
                for (int u = 0; u < UN && jg + u < len; ++u) {
                    if (!LAST && tg + u == next) {
                        const int n = seq_of(p.cu, p.num_seqs, next);
                        int m = n - 1;  // the sequence that ended: empty ones may lie between
                        while (m >= 0 && __ldg(p.cu + m) == next) --m;
                        if (p.h_final) {
                            if (m >= 0) store_state(p.h_final, m);
                            for (int e = m + 1; e < n; ++e) {
                                load_state(p.h0, e);
                                store_state(p.h_final, e);
                            }
                        }
                        load_state(p.h0, n);
                        next = __ldg(p.cu + n + 1);
                    }
                    const float xv = Elem<E>::to_f(xg[u * CH]);
                    const float d = softplus_f(Elem<E>::to_f(xg[(TT + u) * CH]) + bias);
                    const float sl = gate ? silu_fast(Elem<E>::to_f(xg[(2 * TT + u) * CH])) : 1.f;
                    token(row + u * NB, d, (REV ? sl : d) * xv, xv, sl, kDecayBias, 1.f, yo + u * p.ldy);
                }
            }
        }
        if (more) put_bc(buf ^ 1);
        if (LAST) {
            const float t = __fadd_rn(dall, dsum);
            dlost = __fadd_rn(dlost, __fadd_rn(dsum, -__fadd_rn(t, -dall)));
            dall = t;
            dsum = 0.f;
        }
    }
    cp_async_wait<0>();
    if (LAST) {
        store_state(p.H, s);
        if (k == 0 && in) p.sd[(int64_t)s * p.ch + c] = dall + dlost;
    } else if (p.h_final && next <= te) {  // the sequence ends with the segment
        const int m = seq_of(p.cu, p.num_seqs, te - 1);
        store_state(p.h_final, m);
        if (te == p.T)  // empty sequences behind the last token
            for (int e = m + 1; e < p.num_seqs; ++e) {
                load_state(p.h0, e);
                store_state(p.h_final, e);
            }
    }
}

// The fold of the segments' own ends (REV: start gradients) into the states at the
// segments' starts (the gradients behind their ends), in place: row s - 1 becomes
// the state at segment s's start (row s + 1 the gradient behind segment s), for
// segments in the middle of a sequence.  One thread per channel and state.
constexpr int FTH = 256;
template <bool REV>
__global__ void __launch_bounds__(FTH) scan_fold_kernel(const ScanParams p) {
    extern __shared__ unsigned char kind[];  // [S]: 0 no fold ends here, 1 the row as it is, 2 folded with the one before
    for (int s = threadIdx.x; s < p.S; s += FTH) {
        int kd = 0;
        if (!REV && s > 0) {
            const int t0 = s * p.seg, start = max(__ldg(p.cu + seq_of(p.cu, p.num_seqs, t0)), 0);
            if (start < t0) kd = start / p.seg == s - 1 ? 1 : 2;
        } else if (REV && s < p.S - 1) {
            const int te = (s + 1) * p.seg, end = min(__ldg(p.cu + seq_of(p.cu, p.num_seqs, te - 1) + 1), p.T);
            if (end > te) kd = (end - 1) / p.seg == s + 1 ? 1 : 2;
        }
        kind[s] = kd;
    }
    __syncthreads();
    const int64_t i = (int64_t)blockIdx.x * FTH + threadIdx.x;
    if (i >= (int64_t)p.ch * p.N) return;
    const float A2 = -expf(__ldg(p.A_log + i)) * kLog2e;
    const int c = (int)(i / p.N);
    float v = 0.f;
    constexpr int U = 16;  // rows loaded at a time: the walk is bound by their latency
    for (int b = 1; b < p.S; b += U) {
        float Hr[U], d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int q = min(b + u, p.S - 1), row = REV ? p.S - q : q - 1;
            Hr[u] = p.H[(int64_t)row * p.ch * p.N + i];
            d[u] = p.sd[(int64_t)row * p.ch + c];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int q = b + u, row = REV ? p.S - q : q - 1;
            if (q >= p.S) break;
            const int kd = kind[REV ? p.S - 1 - q : q];
            if (kd == 0) continue;
            v = kd == 1 ? Hr[u] : fmaf(exp2_fast(d[u] * A2), v, Hr[u]);
            if (kd == 2) p.H[(int64_t)row * p.ch * p.N + i] = v;
        }
    }
}

constexpr int STG = 4;     // requests whose states are in flight or in use (step)

// One token per request.  Bound by the states, read and written once (for a few
// requests by the launch).  As in the prompt's kernel a lane holds up to 16 states
// of one channel (four lanes a channel and four states, which reads states
// directly, took 272 instructions for 8 channels and was bound by them at 70 us
// for 256 requests of 4096 channels); a warp's channels are one contiguous piece
// of a slot, which comes by 16-byte asynchronous copies into the warp's ring and
// goes back from there, both in full lines.  A warp takes the requests gridDim.y
// apart, three of them under way.  FULL: N is all of a lane's states and the warp's
// channels exist, so that the copies' counts are known.
template <typename E, int K, int NS, bool FULL>
__global__ void __launch_bounds__(NTH, 4) scan_step_kernel(const ScanParams p, int batch, float* states, int num_slots,
                                                           const int32_t* src, const int32_t* dst) {
    constexpr int NP = K * NS, NBC = (2 * NP + 31) / 32;  // padded states; values of B and C per lane
    constexpr int WC = 32 / K;  // channels per warp
    extern __shared__ float4 smem4[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = lane % K, G = gridDim.y;
    const int grp = blockIdx.x / p.tiles, cend = (grp + 1) * p.per;
    const int c0 = grp * p.per + (blockIdx.x % p.tiles) * (NTH / K) + warp * WC;  // the warp's first channel
    if (c0 >= cend) return;
    const int c = c0 + lane / K;
    const bool in = c < cend, vec = FULL || p.N % 4 == 0;
    const int cc = in ? c : c0, N = FULL ? NP : p.N;
    const int tile = WC * N, chunks = FULL ? WC * NP / 4 : min(WC, cend - c0) * N / 4;  // floats; 16-byte pieces that exist
    float* ring = reinterpret_cast<float*>(smem4) + warp * (STG * tile + 4 * NP);
    float* bcs = ring + STG * tile;  // [2][B, C][NP]
    F2 A2[NS / 2];
#pragma unroll
    for (int q = 0; q < NS / 2; ++q) {
        const int st = k * NS + 2 * q;
        const float* g = p.A_log + (int64_t)cc * p.N + st;
        A2[q] = f2(st < p.N ? -expf(__ldg(g)) * kLog2e : 0.f, st + 1 < p.N ? -expf(__ldg(g + 1)) * kLog2e : 0.f);
    }
    const float bias = p.dt_bias ? __ldg(p.dt_bias + cc) : 0.f, Dc = p.D ? __ldg(p.D + cc) : 0.f;
    // four-state pieces of 16 lie 64 bytes apart between lanes: their order within a channel turns with the lane,
    // so that eight lanes' reads meet all banks
    constexpr bool TURN = FULL && NS == 16 && K == 1;
    const int turn = TURN ? lane >> 1 & 3 : 0;
    // the slots that request r reads (-1: none) and writes (-1: a padded row)
    auto slots = [&](int r, int& from, int& to) {
        from = to = -1;
        if (r < batch) {
            from = src ? __ldg(src + r) : r;
            to = dst ? __ldg(dst + r) : r;
            if (to >= num_slots) to = -1;
            if (from >= num_slots || to < 0) from = -1;
        }
    };
    auto piece = [&](int t) {  // where 16-byte piece t of the tile lies
        return TURN ? (t & ~3) | ((t & 3) ^ (t >> 3 & 3)) : t;
    };
    auto copy = [&](int from, int stage) {
        const float* g = states + ((int64_t)(from < 0 ? 0 : from) * p.ch + c0) * p.N;
        float* d = ring + stage * tile;
        if constexpr (FULL && WC * NP / 4 % 32 == 0) {
#pragma unroll
            for (int i = 0; i < WC * NP / 128; ++i)
                cp_async16(d + 4 * piece(lane + 32 * i), g + 4 * (lane + 32 * i), from < 0 ? 0 : 16);
        } else {
            for (int t = lane; t < chunks; t += 32) cp_async16(d + 4 * piece(t), g + 4 * t, from < 0 ? 0 : 16);
        }
        cp_async_commit();
    };
    struct Row {
        E x, dt, z, bc[NBC];
    };
    auto fetch = [&](int r, Row& w) {
        w.x = __ldg(static_cast<const E*>(p.x) + (int64_t)r * p.ldx + cc);
        w.dt = __ldg(static_cast<const E*>(p.dt) + (int64_t)r * p.lddt + cc);
        if (p.z) w.z = __ldg(static_cast<const E*>(p.z) + (int64_t)r * p.ldz + cc);
#pragma unroll
        for (int i = 0; i < NBC; ++i) {
            const int j = lane + 32 * i, n = j % NP;
            const E* q = j < NP ? static_cast<const E*>(p.B) + (int64_t)r * p.ldb : static_cast<const E*>(p.C) + (int64_t)r * p.ldc;
            w.bc[i] = j < 2 * NP && n < N ? __ldg(q + (int64_t)grp * N + n) : Elem<E>::from_f(0.f);
        }
    };
    int from[STG], to[STG];  // of this request and the next ones
#pragma unroll
    for (int i = 0; i < STG; ++i) slots(blockIdx.y + i * G, from[i], to[i]);
#pragma unroll
    for (int i = 0; i < STG - 1; ++i) copy(from[i], i);
    Row cur, nxt;
    int stage = 0, par = 0;
    fetch(blockIdx.y, cur);
    for (int r = blockIdx.y; r < batch; r += G, par ^= 1) {
        copy(from[STG - 1], stage == 0 ? STG - 1 : stage - 1);
        if (r + G < batch) fetch(r + G, nxt);
        const int out = to[0];
#pragma unroll
        for (int i = 0; i < STG - 1; ++i) {
            from[i] = from[i + 1];
            to[i] = to[i + 1];
        }
        slots(r + STG * G, from[STG - 1], to[STG - 1]);
        float* bcw = bcs + par * 2 * NP;
#pragma unroll
        for (int i = 0; i < NBC; ++i)
            if (lane + 32 * i < 2 * NP) bcw[lane + 32 * i] = Elem<E>::to_f(cur.bc[i]);
        const float xv = Elem<E>::to_f(cur.x), dlt = softplus_f(Elem<E>::to_f(cur.dt) + bias);
        const F2 d = f2_dup(dlt), u = f2_dup(dlt * xv), bi = f2_dup(kDecayBias);
        F2 acc = f2_dup(0.f);
        cp_async_wait<STG - 1>();
        __syncwarp();
        float* own = ring + stage * tile + (lane / K) * N + k * NS;
#pragma unroll
        for (int q = 0; q < NS / 4; ++q) {
            const int left = N - (k * NS + 4 * q);
            float* g = own + 4 * (q ^ turn);
            F2 h0, h1, b0, b1, d0, d1;
            if (vec) {
                if (left > 0) f2_load2(g, h0, h1);
                else h0 = h1 = f2_dup(0.f);
            } else {
                h0 = f2(left > 0 ? g[0] : 0.f, left > 1 ? g[1] : 0.f);
                h1 = f2(left > 2 ? g[2] : 0.f, left > 3 ? g[3] : 0.f);
            }
            f2_load2(bcw + k * NS + 4 * q, b0, b1);
            f2_load2(bcw + NP + k * NS + 4 * q, d0, d1);
            h0 = f2_fma(f2_decay(d, A2[2 * q], bi), h0, f2_mul(u, b0));
            h1 = f2_fma(f2_decay(d, A2[2 * q + 1], bi), h1, f2_mul(u, b1));
            acc = f2_fma(h0, d0, acc);
            acc = f2_fma(h1, d1, acc);
            if (vec) {
                if (left > 0) f2_store2(g, h0, h1);
            } else {
                if (left > 0) g[0] = h0.x();
                if (left > 1) g[1] = h0.y();
                if (left > 2) g[2] = h1.x();
                if (left > 3) g[3] = h1.y();
            }
        }
        float o = f2_sum(acc);
#pragma unroll
        for (int off = 1; off < K; off <<= 1) o += __shfl_xor_sync(0xffffffffu, o, off);
        if (in && k == 0) {
            o = fmaf(Dc, xv, o);
            if (p.z) o *= silu_fast(Elem<E>::to_f(cur.z));
            static_cast<E*>(p.y)[(int64_t)r * p.ldy + c] = Elem<E>::from_f(out < 0 ? 0.f : o);
        }
        __syncwarp();
        if (out >= 0) {
            float4* g = reinterpret_cast<float4*>(states + ((int64_t)out * p.ch + c0) * p.N);
            const float* sm = ring + stage * tile;
            if constexpr (FULL && WC * NP / 4 % 32 == 0) {
#pragma unroll
                for (int i = 0; i < WC * NP / 128; ++i)
                    g[lane + 32 * i] = *reinterpret_cast<const float4*>(sm + 4 * piece(lane + 32 * i));
            } else {
                for (int t = lane; t < chunks; t += 32) g[t] = *reinterpret_cast<const float4*>(sm + 4 * piece(t));
            }
        }
        __syncwarp();  // the stage is read before it is copied into again
        cur = nxt;
        stage = stage == STG - 1 ? 0 : stage + 1;
    }
    cp_async_wait<0>();
}

// ---- host ----------------------------------------------------------------------

int channels_per_block(int N) { return N <= 16 ? NTH : (N <= 32 ? NTH / 2 : NTH / 4); }

// Segments of a call: one wave of four resident blocks an SM (of the outputs' launch in
// fp32 fewer fit, so that there it is two waves or one and a half), two where that
// leaves segments of 512 tokens or more (the last blocks' idle time halves: 2.05 ->
// 1.99 ms on 131072 tokens of 2048 channels); whole tiles, on whose starts the
// checkpoints fall, down to one: few tokens are a walk, and a shorter one costs only
// a fold (207 tokens of 88 channels: 19 us, 27 with segments of 64).  Returns the most
// segments that a call of up to T tokens has, which the workspace is for.
int segments(int T, int ch, int N, int groups, int& seg, int& S) {
    const int per = ch / groups, cb = channels_per_block(N);
    const int64_t blocks = (int64_t)groups * ((per + cb - 1) / cb);
    int64_t want = (int64_t)device_sm_count() * 4 / blocks;
    if (T >= 2 * want * 512) want *= 2;
    if (want < 1) want = 1;
    const int64_t least = TT, most = (T + least - 1) / least;
    if (want > most) want = most;
    if (want < 1) want = 1;
    seg = (int)(((T + want - 1) / want + TT - 1) / TT * TT);
    if (seg < least) seg = least;
    S = (T + seg - 1) / seg;
    if (S < 1) S = 1;
    return (int)want;
}

constexpr size_t kSmemPlain = 48 << 10;  // dynamic shared memory that needs no attribute

template <typename E, int K, int NS, int MODE>
constexpr size_t scan_smem() {
    return sizeof(E) * NST * (MODE == SCAN_END ? 2 : 3) * TT * (NTH / K) +
           sizeof(float) * 2 * TT * K * NS * (MODE == SCAN_FULL ? 2 : 1);
}

template <typename E, int K, int NS, int MODE>
gdn_status run_mode(const ScanParams& p, dim3 grid, cudaStream_t s) {
    constexpr size_t smem = scan_smem<E, K, NS, MODE>();
    if (smem > kSmemPlain) {
        const gdn_status st = set_smem_attr((const void*)scan_kernel<E, K, NS, MODE>, smem);
        if (st != GDN_OK) return st;
    }
    scan_kernel<E, K, NS, MODE><<<grid, NTH, smem, s>>>(p);
    return check_launch("scan_kernel");
}

template <bool REV>
gdn_status run_fold(const ScanParams& p, cudaStream_t s) {
    const int64_t n = (int64_t)p.ch * p.N;
    scan_fold_kernel<REV><<<(unsigned)((n + FTH - 1) / FTH), FTH, p.S, s>>>(p);
    return check_launch("scan_fold_kernel");
}

template <typename E, int K, int NS>
gdn_status run_scan(ScanParams p, int groups, bool grad, cudaStream_t s) {
    p.tiles = (p.per + NTH / K - 1) / (NTH / K);
    const dim3 all(groups * p.tiles, p.S), joints(groups * p.tiles, p.S - 1);
    gdn_status st;
    if (grad) {
        if (p.S == 1) return GDN_OK;
        if ((st = run_mode<E, K, NS, SCAN_START_GRAD>(p, joints, s)) != GDN_OK) return st;
        return p.S > kFoldSegments ? run_fold<true>(p, s) : GDN_OK;
    }
    if (p.S > 1) {
        if ((st = run_mode<E, K, NS, SCAN_END>(p, joints, s)) != GDN_OK) return st;
        p.folded = p.S > kFoldSegments;
        if (p.folded && (st = run_fold<false>(p, s)) != GDN_OK) return st;
    }
    return run_mode<E, K, NS, SCAN_FULL>(p, all, s);
}

template <typename E>
gdn_status dispatch_scan(const ScanParams& p, int groups, bool grad, cudaStream_t s) {
    if (p.N <= 4) return run_scan<E, 1, 4>(p, groups, grad, s);
    if (p.N <= 8) return run_scan<E, 1, 8>(p, groups, grad, s);
    if (p.N <= 16) return run_scan<E, 1, 16>(p, groups, grad, s);
    if (p.N <= 32) return run_scan<E, 2, 16>(p, groups, grad, s);
    return run_scan<E, 4, 16>(p, groups, grad, s);
}

template <typename E, int K, int NS>
gdn_status run_step_k(ScanParams p, int groups, int batch, float* states, int num_slots, const int32_t* src,
                      const int32_t* dst, cudaStream_t s) {
    const size_t smem = sizeof(float) * (STG * (NTH / K) * p.N + NTH / 32 * 4 * K * NS);  // 36 KB at most
    p.tiles = (p.per + NTH / K - 1) / (NTH / K);
    const int nx = groups * p.tiles, most = (device_sm_count() * 4 + nx - 1) / nx;
    const dim3 grid(nx, batch < most ? batch : most);
    if (p.N == K * NS && p.per % (32 / K) == 0)
        scan_step_kernel<E, K, NS, true><<<grid, NTH, smem, s>>>(p, batch, states, num_slots, src, dst);
    else
        scan_step_kernel<E, K, NS, false><<<grid, NTH, smem, s>>>(p, batch, states, num_slots, src, dst);
    return check_launch("scan_step_kernel");
}

template <typename E>
gdn_status run_step(const ScanParams& p, int groups, int batch, float* states, int num_slots, const int32_t* src,
                    const int32_t* dst, cudaStream_t s) {
    if (p.N <= 4) return run_step_k<E, 1, 4>(p, groups, batch, states, num_slots, src, dst, s);
    if (p.N <= 8) return run_step_k<E, 1, 8>(p, groups, batch, states, num_slots, src, dst, s);
    if (p.N <= 16) {
        // few warps a scheduler: the latency of a lane's 16 states counts, and four lanes a channel take a quarter of
        // them each.  With all 16 that pays below three warps of one lane a channel (4096 channels in us, four lanes
        // against one: 2 requests 2.3, 2.9; 8 3.5, 3.8; 12 4.4, 4.6; 16 5.1, 5.3; 20 5.6, 5.6; 8192 channels: 3 requests
        // 3.5, 3.5; 6 5.0, 4.6); with fewer, whose pieces are not the copies' whole rows, below one (12 states, 4096
        // channels: 2 requests 2.7, 2.9; 4 2.9, 3.0; 6 4.3, 3.3; 12 6.1, 3.9)
        if ((int64_t)batch * p.ch <= (int64_t)device_sm_count() * 4 * 32 * (p.N == 16 ? 3 : 1))
            return run_step_k<E, 4, 4>(p, groups, batch, states, num_slots, src, dst, s);
        return run_step_k<E, 1, 16>(p, groups, batch, states, num_slots, src, dst, s);
    }
    if (p.N <= 32) return run_step_k<E, 2, 16>(p, groups, batch, states, num_slots, src, dst, s);
    return run_step_k<E, 4, 16>(p, groups, batch, states, num_slots, src, dst, s);
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

gdn_status launch_scan_start_grad(const ScanParams& p, gdn_dtype dtype, int groups, cudaStream_t s) {
    return dtype == GDN_BF16 ? dispatch_scan<__nv_bfloat16>(p, groups, true, s) : dispatch_scan<float>(p, groups, true, s);
}

gdn_status check_scan_shape(gdn_dtype dtype, int rows, int ch, int N, int groups) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return fail(GDN_ERR_DTYPE, "unknown dtype %d", (int)dtype);
    if (rows < 0 || ch < 1 || groups < 1)
        return fail(GDN_ERR_INVALID_ARG, "rows=%d channels=%d groups=%d", rows, ch, groups);
    if (rows > kMaxTokens) return fail(GDN_ERR_UNSUPPORTED_SHAPE, "%d tokens, more than %d", rows, kMaxTokens);
    if (ch % groups != 0 || (ch / groups) % 8 != 0)
        return fail(GDN_ERR_UNSUPPORTED_SHAPE, "channels=%d per group of %d must be a multiple of 8", ch, groups);
    if (N < 1 || N > 64) return fail(GDN_ERR_UNSUPPORTED_SHAPE, "d_state=%d not in 1..64", N);
    return GDN_OK;
}
gdn_status check_scan_row(const void* p, int64_t ld, int64_t least, const char* name) {
    if (!p || !al16(p)) return fail(GDN_ERR_INVALID_ARG, "%s must be 16-byte aligned and not NULL", name);
    if (ld < least || ld % 8 != 0)
        return fail(GDN_ERR_INVALID_ARG, "row stride of %s (%lld) must be >= %lld and a multiple of 8", name,
                    (long long)ld, (long long)least);
    return GDN_OK;
}
gdn_status check_scan_inputs(const void* x, int64_t ldx, const void* dt, int64_t lddt, const void* z, int64_t ldz,
                             const void* B, int64_t ldb, const void* C, int64_t ldc, const float* A_log, int ch,
                             int N, int groups) {
    gdn_status st;
    if ((st = check_scan_row(x, ldx, ch, "x")) != GDN_OK) return st;
    if ((st = check_scan_row(dt, lddt, ch, "dt")) != GDN_OK) return st;
    if (z && (st = check_scan_row(z, ldz, ch, "z")) != GDN_OK) return st;
    if (!B || !C || !A_log) return fail(GDN_ERR_INVALID_ARG, "B, C or A_log is NULL");
    if (ldb < (int64_t)groups * N || ldc < (int64_t)groups * N)
        return fail(GDN_ERR_INVALID_ARG, "row strides of B and C must be >= groups * d_state");
    return GDN_OK;
}

}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_ssm_scan_ckpt_floats(int32_t T, int32_t channels, int32_t d_state) {
    if (T < 0 || T > kMaxTokens || channels < 1 || d_state < 1) return 0;
    return (size_t)((T + kCkpt - 1) / kCkpt) * channels * d_state;
}

size_t gdn_ssm_scan_workspace_size(int32_t T, int32_t channels, int32_t d_state, int32_t groups) {
    if (T < 0 || T > kMaxTokens || channels < 1 || groups < 1 || channels % groups || (channels / groups) % 8 ||
        d_state < 1 || d_state > 64)
        return 0;
    int seg, S;
    const int most = segments(T, channels, d_state, groups, seg, S);
    return (sizeof(float) * (size_t)most * channels * (d_state + 1) + 255) & ~size_t(255);
}

gdn_status gdn_ssm_scan_fwd(const void* x, int64_t ldx, const void* dt, int64_t lddt, const void* z, int64_t ldz,
                            const void* B, int64_t ldb, const void* C, int64_t ldc, gdn_dtype dtype,
                            const float* A_log, const float* D, const float* dt_bias, const float* h0,
                            const int32_t* cu_seqlens, int32_t num_seqs, int32_t T, int32_t channels, int32_t d_state,
                            int32_t groups, void* y, int64_t ldy, float* h_final, float* ckpt, void* workspace,
                            size_t workspace_bytes, void* stream) {
    gdn_status st = check_scan_shape(dtype, T, channels, d_state, groups);
    if (st != GDN_OK) return st;
    if (num_seqs < 1 || !cu_seqlens) return fail(GDN_ERR_INVALID_ARG, "num_seqs=%d or cu_seqlens is NULL", num_seqs);
    if (T > 0) {
        if ((st = check_scan_inputs(x, ldx, dt, lddt, z, ldz, B, ldb, C, ldc, A_log, channels, d_state, groups)) != GDN_OK)
            return st;
        if ((st = check_scan_row(y, ldy, channels, "y")) != GDN_OK) return st;
    }
    if (!A_log) return fail(GDN_ERR_INVALID_ARG, "A_log is NULL");
    if (!al16(h_final) || !al16(ckpt)) return fail(GDN_ERR_INVALID_ARG, "h_final and ckpt must be 16-byte aligned");
    if (h0 && h0 == h_final) return fail(GDN_ERR_INVALID_ARG, "h_final must not be h0");
    const size_t need = gdn_ssm_scan_workspace_size(T, channels, d_state, groups);
    if (!workspace || workspace_bytes < need)
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes < required %zu", workspace ? workspace_bytes : 0, need);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(GDN_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    ScanParams p{};
    p.x = x; p.ldx = ldx; p.dt = dt; p.lddt = lddt; p.z = z; p.ldz = ldz; p.B = B; p.ldb = ldb; p.C = C; p.ldc = ldc;
    p.A_log = A_log; p.D = D; p.dt_bias = dt_bias; p.h0 = h0; p.cu = cu_seqlens; p.num_seqs = num_seqs; p.T = T;
    p.ch = channels; p.N = d_state; p.per = channels / groups; p.y = y; p.ldy = ldy; p.h_final = h_final; p.ckpt = ckpt;
    segments(T, channels, d_state, groups, p.seg, p.S);
    p.H = static_cast<float*>(workspace);
    p.sd = p.H + (size_t)p.S * channels * d_state;
    cudaStream_t s = (cudaStream_t)stream;
    return dtype == GDN_BF16 ? dispatch_scan<__nv_bfloat16>(p, groups, false, s)
                             : dispatch_scan<float>(p, groups, false, s);
}

gdn_status gdn_ssm_scan_step(const void* x, int64_t ldx, const void* dt, int64_t lddt, const void* z, int64_t ldz,
                             const void* B, int64_t ldb, const void* C, int64_t ldc, gdn_dtype dtype,
                             const float* A_log, const float* D, const float* dt_bias, int32_t batch, int32_t channels,
                             int32_t d_state, int32_t groups, float* states, int32_t num_slots, const int32_t* src,
                             const int32_t* dst, void* y, int64_t ldy, void* stream) {
    gdn_status st = check_scan_shape(dtype, batch, channels, d_state, groups);
    if (st != GDN_OK) return st;
    if (batch > 65535) return fail(GDN_ERR_UNSUPPORTED_SHAPE, "batch=%d above 65535", batch);
    if (num_slots < 0) return fail(GDN_ERR_INVALID_ARG, "num_slots=%d", num_slots);
    if ((!src || !dst) && num_slots < batch)
        return fail(GDN_ERR_INVALID_ARG, "num_slots=%d < batch=%d without slot numbers", num_slots, batch);
    if (batch == 0) return GDN_OK;
    if ((st = check_scan_inputs(x, ldx, dt, lddt, z, ldz, B, ldb, C, ldc, A_log, channels, d_state, groups)) != GDN_OK)
        return st;
    if ((st = check_scan_row(y, ldy, channels, "y")) != GDN_OK) return st;
    if (!states || !al16(states)) return fail(GDN_ERR_INVALID_ARG, "states must be 16-byte aligned and not NULL");
    ScanParams p{};
    p.x = x; p.ldx = ldx; p.dt = dt; p.lddt = lddt; p.z = z; p.ldz = ldz; p.B = B; p.ldb = ldb; p.C = C; p.ldc = ldc;
    p.A_log = A_log; p.D = D; p.dt_bias = dt_bias; p.ch = channels; p.N = d_state; p.per = channels / groups; p.y = y;
    p.ldy = ldy;
    cudaStream_t s = (cudaStream_t)stream;
    return dtype == GDN_BF16 ? run_step<__nv_bfloat16>(p, groups, batch, states, num_slots, src, dst, s)
                             : run_step<float>(p, groups, batch, states, num_slots, src, dst, s);
}

}  // extern "C"
