// Selective state space scan: the forward over packed prompts and the
// single-token step.
//
// Per channel with N diagonal states (fp32 throughout):
//   delta = softplus(dt + dt_bias), a_n = 2^(delta A2_n), A2 = -exp(A_log) log2 e,
//   h_n <- a_n h_n + (delta x) B_n,   y = (sum_n C_n h_n + D x) silu(z).
//
// Work split.  K lanes share a channel, each with NS states in registers; a
// thread may hold NC channels, so that one read of B and C from shared memory
// serves NC of them.  A block walks down a range of packed tokens in tiles of
// TT: its threads first turn the tile's x, dt into (delta, delta x) in shared
// memory, 16 bytes of a row at a time, then run the recurrence, leaving the
// sums over n in place, and last apply skip and gate and store, again by rows.
//
// Parallelism over tokens.  The packed tokens are cut into S segments of equal
// length, whatever the sequences' lengths.  A first launch runs each segment's
// part of the sequence that goes on into the next segment from a zero state (or
// from h0 where the sequence starts in it), keeping only the end state H and
// the sum of delta; from the first token of a segment that continues a
// sequence, the state is the fold  h <- 2^(A2 sum delta_j) h + H_j  over the
// segments before it, which each block does for its own channels.
#include "ssm_common.cuh"

namespace gdn {
namespace {

constexpr int TT = 32;     // tokens per tile
constexpr int NTH = 128;   // threads per block

struct ScanParams {
    const void* x; int64_t ldx;
    const void* dt; int64_t lddt;
    const void* z; int64_t ldz;
    const void* B; int64_t ldb;
    const void* C; int64_t ldc;
    const float* A_log; const float* D; const float* dt_bias; const float* h0;
    const int32_t* cu;
    int num_seqs, T, ch, N, per;     // per = channels per group
    int tiles;                       // channel tiles per group
    void* y; int64_t ldy;
    float* h_final; float* ckpt;
    int seg, S;                      // tokens per segment, segments
    float* H; float* sd;             // [S, ch, N], [S, ch]
};

// Sum over the K lanes of a channel (adjacent lanes), four tokens at a time:
// the exchange halves the values, so that each lane ends with the tokens of its
// own index.  K = 4: lane k holds token (k & 1) * 2 + (k >> 1).
template <int K>
__device__ __forceinline__ void lane_sums(float (&v)[4], int k) {
    if (K == 1) return;
    const bool b0 = k & 1;
    float s0 = b0 ? v[0] : v[2], s1 = b0 ? v[1] : v[3];
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

template <int K, int NS, int NC>
struct Shape {
    static constexpr int CPW = 32 / K;                 // channels side by side in a warp
    static constexpr int CH = NTH / 32 * CPW * NC;     // channels per block
    static constexpr int NP = K * NS;                  // padded states
    static constexpr size_t smem = sizeof(float2) * TT * CH + sizeof(float) * 2 * TT * NP;
};

// LAST: the segment's end state only (no y, no C).
template <typename E, int K, int NS, int NC, bool LAST>
__global__ void __launch_bounds__(NTH) scan_kernel(const ScanParams p) {
    using Sh = Shape<K, NS, NC>;
    constexpr int CH = Sh::CH, NP = Sh::NP, CPW = Sh::CPW;
    extern __shared__ float4 smem4[];
    float2* du = reinterpret_cast<float2*>(smem4);       // [TT][CH]
    float* Bs = reinterpret_cast<float*>(du + TT * CH);  // [TT][NP]
    float* Cs = Bs + TT * NP;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int grp = blockIdx.x / p.tiles;
    const int cbase = grp * p.per + (blockIdx.x % p.tiles) * CH;  // first channel
    const int cend = (grp + 1) * p.per;                           // end of the group's channels
    const int nv = min(CH, cend - cbase) >> 3;                    // vectors of eight channels
    const int s = blockIdx.y;
    int t0 = s * p.seg;
    const int te = min(p.T, t0 + p.seg);
    const int k = lane % K;
    int cl[NC];  // channel within the block
    float A2[NC][NS], h[NC][NS];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        cl[i] = (i * (NTH / 32) + warp) * CPW + lane / K;
        const int c = cbase + cl[i];
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            const int st = k * NS + n;
            A2[i][n] = c < cend && st < p.N ? -expf(__ldg(p.A_log + (int64_t)c * p.N + st)) * kLog2e : 0.f;
            h[i][n] = 0.f;
        }
    }
    auto load_state = [&](const float* src, int64_t row) {  // src [rows, ch, N] or null
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = cbase + cl[i];
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                const int st = k * NS + n;
                h[i][n] = src && c < cend && st < p.N ? __ldg(src + (row * p.ch + c) * p.N + st) : 0.f;
            }
        }
    };
    auto store_state = [&](float* dst, int64_t row) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = cbase + cl[i];
            if (c < cend) {
                float* q = dst + (row * p.ch + c) * p.N + k * NS;
                if (NS % 4 == 0 && p.N % 4 == 0) {
#pragma unroll
                    for (int n = 0; n < NS; n += 4)
                        if (k * NS + n < p.N)
                            *reinterpret_cast<float4*>(q + n) = make_float4(h[i][n], h[i][n + 1], h[i][n + 2], h[i][n + 3]);
                } else {
#pragma unroll
                    for (int n = 0; n < NS; ++n)
                        if (k * NS + n < p.N) q[n] = h[i][n];
                }
            }
        }
    };
    // the sequence at the first token, and the state there
    int next;  // first token of the next sequence
    float dsum[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) dsum[i] = 0.f;
    if (LAST) {
        const int n = seq_of(p.cu, p.num_seqs, te - 1);
        if (__ldg(p.cu + n + 1) <= te) return;  // nothing goes on into the next segment
        const int start = __ldg(p.cu + n);
        if (start >= t0) {
            t0 = min(start, te - 1);
            load_state(p.h0, n);
        }
        next = p.T;
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
        } else {
            for (int j = max(start, 0) / p.seg; j < s; ++j) {
                const bool first = max(start, 0) / p.seg == j;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    const int c = cbase + cl[i];
                    if (c < cend) {
                        const int64_t row = (int64_t)j * p.ch + c;
                        const float d = first ? 0.f : __ldg(p.sd + row);
#pragma unroll
                        for (int q = 0; q < NS; ++q) {
                            const int st = k * NS + q;
                            const float Hj = st < p.N ? __ldg(p.H + row * p.N + st) : 0.f;
                            h[i][q] = first ? Hj : fmaf(exp2_fast(d * A2[i][q]), h[i][q], Hj);
                        }
                    }
                }
            }
        }
    }

    for (int tb = t0 - (LAST ? t0 % TT : 0); tb < te; tb += TT) {
        // (delta, delta x) of the tile; rows outside [t0, te) leave the state alone
        for (int it = tid; it < TT * nv; it += NTH) {
            const int r = it / nv, v = it - r * nv, t = tb + r;
            float2* out = du + r * CH + 8 * v;
            if (t >= t0 && t < te) {
                float xv[8], dv[8];
                load8(static_cast<const E*>(p.x) + (int64_t)t * p.ldx + cbase + 8 * v, xv);
                load8(static_cast<const E*>(p.dt) + (int64_t)t * p.lddt + cbase + 8 * v, dv);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float dl = softplus_f(dv[i] + (p.dt_bias ? __ldg(p.dt_bias + cbase + 8 * v + i) : 0.f));
                    out[i] = make_float2(dl, dl * xv[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) out[i] = make_float2(0.f, 0.f);
            }
        }
        for (int it = tid; it < TT * NP; it += NTH) {
            const int r = it / NP, n = it - r * NP, t = tb + r;
            const bool in = t >= t0 && t < te && n < p.N;
            const int64_t off = (int64_t)grp * p.N + n;
            Bs[it] = in ? Elem<E>::load(static_cast<const E*>(p.B) + t * p.ldb + off) : 0.f;
            if (!LAST) Cs[it] = in ? Elem<E>::load(static_cast<const E*>(p.C) + t * p.ldc + off) : 0.f;
        }
        __syncthreads();
        if (!LAST && p.ckpt && (tb & 63) == 0) store_state(p.ckpt, tb >> 6);
#pragma unroll 1
        for (int r0 = 0; r0 < TT; r0 += 4) {
            float ys[NC][4];
            const bool plain = LAST || next >= tb + r0 + 4 || next >= te;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int r = r0 + u;
                if (!LAST && !plain && tb + r == next && next < te) {  // a sequence ends and another starts
                    const int n = seq_of(p.cu, p.num_seqs, next);
                    int m = n - 1;  // the sequence that ended: empty ones may lie between
                    while (m >= 0 && __ldg(p.cu + m) == next) --m;
                    if (p.h_final) {
                        if (m >= 0) store_state(p.h_final, m);
                        for (int e = max(m, 0) + 1; e < n; ++e) {
                            load_state(p.h0, e);
                            store_state(p.h_final, e);
                        }
                    }
                    load_state(p.h0, n);
                    next = __ldg(p.cu + n + 1);
                }
                float Bv[NS], Cv[NS];
#pragma unroll
                for (int n = 0; n < NS; n += 4) {
                    const float4 b = *reinterpret_cast<const float4*>(Bs + r * NP + k * NS + n);
                    Bv[n] = b.x; Bv[n + 1] = b.y; Bv[n + 2] = b.z; Bv[n + 3] = b.w;
                    if (!LAST) {
                        const float4 c = *reinterpret_cast<const float4*>(Cs + r * NP + k * NS + n);
                        Cv[n] = c.x; Cv[n + 1] = c.y; Cv[n + 2] = c.z; Cv[n + 3] = c.w;
                    }
                }
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    const float2 d = du[r * CH + cl[i]];
                    float acc = 0.f;
#pragma unroll
                    for (int n = 0; n < NS; ++n) {
                        h[i][n] = fmaf(exp2_fast(d.x * A2[i][n]), h[i][n], d.y * Bv[n]);
                        if (!LAST) acc = fmaf(h[i][n], Cv[n], acc);
                    }
                    if (LAST) dsum[i] += d.x;
                    else ys[i][u] = acc;
                }
            }
            if (!LAST) {
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    lane_sums<K>(ys[i], k);
                    if (K == 1) {
#pragma unroll
                        for (int u = 0; u < 4; ++u) du[(r0 + u) * CH + cl[i]].x = ys[i][u];
                    } else if (K == 2) {
                        du[(r0 + 2 * k) * CH + cl[i]].x = ys[i][0];
                        du[(r0 + 2 * k + 1) * CH + cl[i]].x = ys[i][1];
                    } else {
                        du[(r0 + (k & 1) * 2 + (k >> 1)) * CH + cl[i]].x = ys[i][0];
                    }
                }
            }
        }
        __syncthreads();
        if (!LAST) {
            for (int it = tid; it < TT * nv; it += NTH) {
                const int r = it / nv, v = it - r * nv, t = tb + r;
                if (t >= te) continue;
                float o[8], f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = du[r * CH + 8 * v + i].x;
                if (p.D) {
                    load8(static_cast<const E*>(p.x) + (int64_t)t * p.ldx + cbase + 8 * v, f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = fmaf(__ldg(p.D + cbase + 8 * v + i), f[i], o[i]);
                }
                if (p.z) {
                    load8(static_cast<const E*>(p.z) + (int64_t)t * p.ldz + cbase + 8 * v, f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] *= silu_fast(f[i]);
                }
                store8(static_cast<E*>(p.y) + (int64_t)t * p.ldy + cbase + 8 * v, o);
            }
            __syncthreads();
        }
    }
    if (LAST) {
        store_state(p.H, s);
        if (k == 0)
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (cbase + cl[i] < cend) p.sd[(int64_t)s * p.ch + cbase + cl[i]] = dsum[i];
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

// One token per request.  Bound by the states, read and written once (for a few
// requests by the launch): one thread per channel and four states, K lanes a channel.
template <typename E, int K>
__global__ void __launch_bounds__(256) scan_step_kernel(const ScanParams p, float* states, int num_slots,
                                                        const int32_t* src, const int32_t* dst) {
    const int r = blockIdx.y, lane_k = threadIdx.x % K;
    const int c = (blockIdx.x * 256 + threadIdx.x) / K;
    int from = src ? __ldg(src + r) : r;
    const int to = dst ? __ldg(dst + r) : r;
    if (from >= num_slots) from = -1;
    const bool pad = to < 0 || to >= num_slots;
    const bool in = c < p.ch;
    float acc = 0.f, xv = 0.f;
    if (in && !pad) {
        xv = Elem<E>::load(static_cast<const E*>(p.x) + (int64_t)r * p.ldx + c);
        const float dl = softplus_f(Elem<E>::load(static_cast<const E*>(p.dt) + (int64_t)r * p.lddt + c) +
                                    (p.dt_bias ? __ldg(p.dt_bias + c) : 0.f));
        const float u = dl * xv;
        const int grp = c / p.per;
        const E* B = static_cast<const E*>(p.B) + (int64_t)r * p.ldb + (int64_t)grp * p.N;
        const E* C = static_cast<const E*>(p.C) + (int64_t)r * p.ldc + (int64_t)grp * p.N;
        for (int n0 = 4 * lane_k; n0 < p.N; n0 += 4 * K) {
            float h[4] = {0.f, 0.f, 0.f, 0.f}, a[4];
            const int64_t off = (int64_t)c * p.N + n0;
            const float* in_p = states + (int64_t)from * p.ch * p.N + off;
            float* out_p = states + (int64_t)to * p.ch * p.N + off;
            if (p.N % 4 == 0) {
                if (from >= 0) {
                    const float4 v = *reinterpret_cast<const float4*>(in_p);
                    h[0] = v.x; h[1] = v.y; h[2] = v.z; h[3] = v.w;
                }
                const float4 v = __ldg(reinterpret_cast<const float4*>(p.A_log + off));
                a[0] = v.x; a[1] = v.y; a[2] = v.z; a[3] = v.w;
            } else {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const bool ok = n0 + n < p.N;
                    if (ok && from >= 0) h[n] = in_p[n];
                    a[n] = ok ? __ldg(p.A_log + off + n) : 0.f;
                }
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                if (n0 + n < p.N) {
                    h[n] = fmaf(exp2_fast(-expf(a[n]) * kLog2e * dl), h[n], u * Elem<E>::load(B + n0 + n));
                    acc = fmaf(h[n], Elem<E>::load(C + n0 + n), acc);
                }
            }
            if (p.N % 4 == 0) *reinterpret_cast<float4*>(out_p) = make_float4(h[0], h[1], h[2], h[3]);
            else
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    if (n0 + n < p.N) out_p[n] = h[n];
        }
    }
#pragma unroll
    for (int off = 1; off < K; off <<= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (in && lane_k == 0) {
        if (p.D) acc = fmaf(__ldg(p.D + c), xv, acc);
        if (p.z && !pad) acc *= silu_fast(Elem<E>::load(static_cast<const E*>(p.z) + (int64_t)r * p.ldz + c));
        static_cast<E*>(p.y)[(int64_t)r * p.ldy + c] = Elem<E>::from_f(pad ? 0.f : acc);
    }
}

// ---- host ----------------------------------------------------------------------

int lanes_of(int N) { return N <= 4 ? 1 : (N <= 8 ? 2 : 4); }
int channels_per_block(int N) {
    const int K = lanes_of(N), NC = 1;
    return NTH / 32 * (32 / K) * NC;
}

// Segments of a call: enough blocks for four resident ones an SM, of 64 tokens
// or more; multiples of 64 so that the backward's state checkpoints fall on
// segment starts.
void segments(int T, int ch, int N, int groups, int& seg, int& S) {
    const int per = ch / groups, cb = channels_per_block(N);
    const int64_t blocks = (int64_t)groups * ((per + cb - 1) / cb);
    int64_t want = (int64_t)device_sm_count() * 4 / blocks;
    if (want < 1) want = 1;
    const int64_t most = (T + 63) / 64;
    if (want > most) want = most;
    if (want < 1) want = 1;
    seg = (int)(((T + want - 1) / want + 63) / 64 * 64);
    if (seg < 64) seg = 64;
    S = (T + seg - 1) / seg;
    if (S < 1) S = 1;
}

template <typename E, int K, int NS, int NC>
gdn_status run_scan(ScanParams p, int groups, cudaStream_t s) {
    using Sh = Shape<K, NS, NC>;
    p.tiles = (p.per + Sh::CH - 1) / Sh::CH;
    dim3 grid(groups * p.tiles, p.S);
    if (p.S > 1) {
        dim3 g1(grid.x, p.S - 1);
        scan_kernel<E, K, NS, NC, true><<<g1, NTH, Sh::smem, s>>>(p);
        const gdn_status st = check_launch("scan_kernel (end states)");
        if (st != GDN_OK) return st;
    }
    scan_kernel<E, K, NS, NC, false><<<grid, NTH, Sh::smem, s>>>(p);
    return check_launch("scan_kernel");
}

template <typename E>
gdn_status dispatch_scan(const ScanParams& p, int groups, cudaStream_t s) {
    if (p.N <= 4) return run_scan<E, 1, 4, 1>(p, groups, s);
    if (p.N <= 8) return run_scan<E, 2, 4, 1>(p, groups, s);
    if (p.N <= 16) return run_scan<E, 4, 4, 1>(p, groups, s);
    if (p.N <= 32) return run_scan<E, 4, 8, 1>(p, groups, s);
    return run_scan<E, 4, 16, 1>(p, groups, s);
}

template <typename E>
gdn_status run_step(const ScanParams& p, int batch, float* states, int num_slots, const int32_t* src,
                    const int32_t* dst, cudaStream_t s) {
    const int K = lanes_of(p.N);
    const dim3 grid((unsigned)(((int64_t)p.ch * K + 255) / 256), batch);
    if (K == 1) scan_step_kernel<E, 1><<<grid, 256, 0, s>>>(p, states, num_slots, src, dst);
    else if (K == 2) scan_step_kernel<E, 2><<<grid, 256, 0, s>>>(p, states, num_slots, src, dst);
    else scan_step_kernel<E, 4><<<grid, 256, 0, s>>>(p, states, num_slots, src, dst);
    return check_launch("scan_step_kernel");
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

gdn_status check_scan_shape(gdn_dtype dtype, int rows, int ch, int N, int groups) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return fail(GDN_ERR_DTYPE, "unknown dtype %d", (int)dtype);
    if (rows < 0 || ch < 1 || groups < 1)
        return fail(GDN_ERR_INVALID_ARG, "rows=%d channels=%d groups=%d", rows, ch, groups);
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
    if (T < 0 || channels < 1 || d_state < 1) return 0;
    return (size_t)((T + 63) / 64) * channels * d_state;
}

size_t gdn_ssm_scan_workspace_size(int32_t T, int32_t channels, int32_t d_state, int32_t groups) {
    if (T < 0 || channels < 1 || groups < 1 || channels % groups || (channels / groups) % 8 || d_state < 1 ||
        d_state > 64)
        return 0;
    int seg, S;
    segments(T, channels, d_state, groups, seg, S);
    return (sizeof(float) * (size_t)S * channels * (d_state + 1) + 255) & ~size_t(255);
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
    return dtype == GDN_BF16 ? dispatch_scan<__nv_bfloat16>(p, groups, s) : dispatch_scan<float>(p, groups, s);
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
    if (!states || !al16(states) || !al16(A_log))
        return fail(GDN_ERR_INVALID_ARG, "states and A_log must be 16-byte aligned and states not NULL");
    ScanParams p{};
    p.x = x; p.ldx = ldx; p.dt = dt; p.lddt = lddt; p.z = z; p.ldz = ldz; p.B = B; p.ldb = ldb; p.C = C; p.ldc = ldc;
    p.A_log = A_log; p.D = D; p.dt_bias = dt_bias; p.ch = channels; p.N = d_state; p.per = channels / groups; p.y = y;
    p.ldy = ldy;
    cudaStream_t s = (cudaStream_t)stream;
    return dtype == GDN_BF16 ? run_step<__nv_bfloat16>(p, batch, states, num_slots, src, dst, s)
                             : run_step<float>(p, batch, states, num_slots, src, dst, s);
}

}  // extern "C"
