// Softmax cross entropy over a vocabulary for few tokens: the formulas of vocab_loss.cu.
//
// What bounds it: the weights, read once for the loss; read twice and their gradient
// written once for the gradients.  The tensor cores' tiles hold 128 tokens, and what they
// read has to be bf16 or fp16 at whole 16 bytes, other weights two passes more; here each weight
// goes through the fp32 units once for every token.
//
//   logits  a warp takes R rows of w after R rows, a lane's 16 bytes (or less, as the
//           alignment allows) of each, the next ones on their way, against up to 8 tokens'
//           h in shared memory: R rows share what is read there.  The R x TT sums over lanes
//           are halved step by step, 31 exchanges for 32 sums, and end one a lane, which
//           keeps its running maximum and sum of exponentials, or writes P.
//   grads   a thread has C columns of all tokens' h and dh and walks rows of w:
//           dh += P w, dw = P h.  Chunks of rows leave dh in parts, joined in their order by
//           a launch behind, so that equal calls give equal bits.
//
// Sums are fp32 and P is not rounded.
#include "vocab_few.cuh"

namespace gdn {

gdn_status set_smem_attr(const void* func, size_t bytes);

namespace {

// ---- elements ----------------------------------------------------------------

template <int BYTES> struct Word;
template <> struct Word<2> { using type = unsigned short; };
template <> struct Word<4> { using type = unsigned; };
template <> struct Word<8> { using type = uint2; };
template <> struct Word<16> { using type = uint4; };

// N consecutive elements in one access
template <typename E, int N>
struct Piece {
    using raw = typename Word<N * sizeof(E)>::type;
    static __device__ __forceinline__ raw zero() {
        raw r;
        unsigned char* b = reinterpret_cast<unsigned char*>(&r);
#pragma unroll
        for (int i = 0; i < (int)sizeof(raw); ++i) b[i] = 0;
        return r;
    }
    static __device__ __forceinline__ void to_f(const raw& r, float (&f)[N]) {
        if constexpr (sizeof(E) == 4) {
            const float* x = reinterpret_cast<const float*>(&r);
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = x[i];
        } else if constexpr (N == 1) {
            f[0] = __uint_as_float((unsigned)r << 16);
        } else {
            const unsigned* x = reinterpret_cast<const unsigned*>(&r);
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                f[2 * i] = __uint_as_float(x[i] << 16);
                f[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
            }
        }
    }
    static __device__ __forceinline__ raw from_f(const float (&f)[N]) {
        raw r;
        if constexpr (sizeof(E) == 4) {
            float* x = reinterpret_cast<float*>(&r);
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = f[i];
        } else if constexpr (N == 1) {
            const __nv_bfloat16 b = __float2bfloat16_rn(f[0]);
            r = *reinterpret_cast<const raw*>(&b);
        } else {
            unsigned* x = reinterpret_cast<unsigned*>(&r);
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                x[i] = *reinterpret_cast<const unsigned*>(&b);
            }
        }
        return r;
    }
};

// a token's target, -1 where it is left out, V where it is that or more
__device__ __forceinline__ int target_at(const FewArgs& a, int t) {
    if (!a.wide) {
        const int v = __ldg(static_cast<const int*>(a.targets) + t);
        return v < 0 ? -1 : min(v, a.V);
    }
    const long long v = __ldg(static_cast<const long long*>(a.targets) + t);
    return v < 0 ? -1 : v > a.V ? a.V : (int)v;
}

// ---- logits ------------------------------------------------------------------

constexpr int LT = 512, LW = LT / 32;  // threads and warps of a block
constexpr int kGroup = 8;              // the most tokens of a block

// accesses of a lane to a row in one step: 16 bytes together, or four
template <typename E, int VEC>
__host__ __device__ constexpr int pieces() {
    return 16 / (VEC * (int)sizeof(E)) < 4 ? 16 / (VEC * (int)sizeof(E)) : 4;
}
// columns of a token's h in shared memory: whole steps of 32 lanes
__host__ __device__ constexpr int padded(int W, int step) { return (W + step - 1) / step * step; }

// where column c is kept, so that lanes' 16-byte reads do not meet in a bank: for eight columns
// a lane the first four of all lanes, then the second four
template <int VEC>
__device__ __forceinline__ int place(int c) {
    return VEC == 8 ? (c & ~255) + ((c >> 2) & 1) * 128 + ((c >> 3) & 31) * 4 + (c & 3) : c;
}
// up to four columns of a lane: those from `at` on
template <int Q>
__device__ __forceinline__ void read_h(const float* at, int lane, float (&f)[Q]) {
    if constexpr (Q == 4) {
        const float4 x = *reinterpret_cast<const float4*>(at + lane * 4);
        f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
    } else if constexpr (Q == 2) {
        const float2 x = *reinterpret_cast<const float2*>(at + lane * 2);
        f[0] = x.x; f[1] = x.y;
    } else {
        f[0] = at[lane];
    }
}

// Sums over the warp of N values a lane: value i in the lanes i << (5 - log2 N) and behind
template <int N, int O>
__device__ __forceinline__ float warp_sums(float (&v)[N], int lane) {
    if constexpr (O == 0) {
        return v[0];
    } else if constexpr (N > 1) {
        const bool up = lane & O;
        float u[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float keep = up ? v[i + N / 2] : v[i], give = up ? v[i] : v[i + N / 2];
            u[i] = keep + __shfl_xor_sync(0xffffffffu, give, O);
        }
        return warp_sums<N / 2, O / 2>(u, lane);
    } else {
        float u[1] = {v[0] + __shfl_xor_sync(0xffffffffu, v[0], O)};
        return warp_sums<1, O / 2>(u, lane);
    }
}

__host__ __device__ constexpr int log2_of(int n) { return n == 1 ? 0 : 1 + log2_of(n / 2); }

__host__ __device__ constexpr int rows_of(int tt) { return tt == 1 ? 8 : 4; }  // of a warp, with tt tokens

struct LogitArgs {
    FewArgs a;
    int groups;                          // of TT tokens
    float2* stat; float* at;             // the loss
    const float* dloss; const float* lse; float* P;  // the gradients
    const float* loss;                   // for P at the targets, or null: by lse
};

template <typename E, int TT, int VEC>
__global__ void __launch_bounds__(LT, 1) few_logits_kernel(const LogitArgs p) {
    constexpr int R = rows_of(TT);
    constexpr int N = R * TT, SH = 5 - log2_of(N);
    using X = Piece<E, VEC>;
    using raw = typename X::raw;
    extern __shared__ __align__(16) float hs[];  // [TT][Wp]
    __shared__ float2 part[LW][TT];
    __shared__ int target[TT];          // of the block's tokens
    __shared__ float lse[TT], g[TT], hot[TT];  // (registers are for the sums); hot: P at the target
    const FewArgs& a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int blk = blockIdx.x / p.groups, blks = gridDim.x / p.groups;
    constexpr int S = pieces<E, VEC>(), STEP = 32 * VEC * S;
    const int t0 = (blockIdx.x - blk * p.groups) * TT, Wp = padded(a.W, STEP), steps = Wp / STEP;
    for (int t = 0; t < TT; ++t) {
        const E* h = static_cast<const E*>(a.h) + (int64_t)(t0 + t) * a.ldh;
        for (int c = tid; c < Wp; c += LT) hs[t * Wp + place<VEC>(c)] = t0 + t < a.T && c < a.W ? Elem<E>::load(h + c) : 0.f;
    }
    // this lane's sum: of row r and token t of the warp's
    const int r = (lane >> SH) / TT, t = t0 + (lane >> SH) % TT;
    const bool one = (lane & ((1 << SH) - 1)) == 0 && t < a.T;  // the only lane that writes it
    float m = -INFINITY, sum = 0.f;
    if (tid < TT) {
        const bool real = t0 + tid < a.T;
        const int v = real ? target_at(a, t0 + tid) : -1;
        target[tid] = v;
        if (p.P && real) {
            lse[tid] = __ldg(p.lse + t0 + tid);
            g[tid] = v < 0 ? 0.f : v >= a.V ? NAN : __ldg(p.dloss + t0 + tid) * a.scale;
            // p - 1 from the loss, -log p: the rounded lse would not tell p from 1
            if (p.loss) hot[tid] = g[tid] * expm1f(-__ldg(p.loss + t0 + tid));
        }
    }
    __syncthreads();
    const int64_t sets = (a.V + R - 1) / R;
    raw next[R][S];
    auto load = [&](const E* row, int c) {
#pragma unroll
        for (int z = 0; z < S; ++z)
#pragma unroll
            for (int i = 0; i < R; ++i)
                next[i][z] = lane * VEC + c + z * 32 * VEC < a.W
                                 ? __ldg(reinterpret_cast<const raw*>(row + c + z * 32 * VEC + i * a.ldw))
                                 : X::zero();
    };
    // the first of a set's rows (the last set: rows of the one before again, which are not counted
    // twice), this lane's columns
    auto rows = [&](int64_t q) {
        return static_cast<const E*>(a.w) + (int64_t)min((int)q * R, a.V - R) * a.ldw + lane * VEC;
    };
    int64_t q = (int64_t)warp * blks + blk;
    const E* row = rows(q);
    if (q < sets) load(row, 0);
    for (; q < sets; q += (int64_t)LW * blks) {
        const int64_t after = q + (int64_t)LW * blks;
        const E* const row_after = rows(after < sets ? after : q);
        float acc[N];
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = 0.f;
#pragma unroll 1
        for (int k = 0; k < steps; ++k) {
            raw now[R][S];
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int z = 0; z < S; ++z) now[i][z] = next[i][z];
            if (k + 1 < steps) load(row, (k + 1) * STEP);
            else if (after < sets) load(row_after, 0);
            constexpr int Q = VEC == 8 ? 4 : VEC;  // columns at a time
#pragma unroll
            for (int z = 0; z < S * (VEC / Q); ++z) {
                float f[R][Q];
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    if constexpr (VEC == 8) {
                        const uint4 r = now[i][0];
                        Piece<E, Q>::to_f(z ? make_uint2(r.z, r.w) : make_uint2(r.x, r.y), f[i]);
                    } else {
                        X::to_f(now[i][z], f[i]);
                    }
                }
#pragma unroll
                for (int j = 0; j < TT; ++j) {
                    float x[Q];
                    read_h<Q>(hs + j * Wp + k * STEP + z * Q * 32, lane, x);
#pragma unroll
                    for (int i = 0; i < R; ++i)
#pragma unroll
                        for (int e = 0; e < Q; ++e) acc[i * TT + j] = fmaf(f[i][e], x[e], acc[i * TT + j]);
                }
            }
        }
        const float x = __fmul_rn(warp_sums<N, 16>(acc, lane), a.scale);
        row = row_after;
        const int v = min((int)q * R, a.V - R) + r, j = t - t0;
        if (v < (int)q * R) continue;
        if (p.P) {
            // (g of 0: a token that is left out, whatever its h holds)
            if (one) {
                float P = 0.f;
                if (g[j] != 0.f) {
                    P = g[j] * exp2_fast((x - lse[j]) * kLog2e);
                    if (v == target[j]) P = p.loss ? hot[j] : P - g[j];
                }
                p.P[(int64_t)v * a.T + t] = P;
            }
        } else {
            if (v == target[j]) {  // goes its own way (lse_join_kernel)
                if (one) p.at[t] = x;
                continue;
            }
            const float top = fmaxf(m, x), ref = top == -INFINITY ? 0.f : top;
            sum = sum * exp2_fast((m - ref) * kLog2e) + exp2_fast((x - ref) * kLog2e);
            m = top;
        }
    }
    if (p.P) return;
    // the rows of the warp, then its block's warps
#pragma unroll
    for (int o = TT << SH; o < 32; o <<= 1) {
        const float mo = __shfl_xor_sync(0xffffffffu, m, o), so = __shfl_xor_sync(0xffffffffu, sum, o);
        const float top = fmaxf(m, mo), ref = top == -INFINITY ? 0.f : top;
        sum = sum * exp2_fast((m - ref) * kLog2e) + so * exp2_fast((mo - ref) * kLog2e);
        m = top;
    }
    if (r == 0 && (lane & ((1 << SH) - 1)) == 0) part[warp][t - t0] = make_float2(m, sum);
    __syncthreads();
    if (tid >= TT || t0 + tid >= a.T) return;
    m = -INFINITY;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < LW; ++i) {
        const float2 v = part[i][tid];
        const float top = fmaxf(m, v.x), ref = top == -INFINITY ? 0.f : top;
        sum = sum * exp2_fast((m - ref) * kLog2e) + v.y * exp2_fast((v.x - ref) * kLog2e);
        m = top;
    }
    p.stat[(int64_t)blk * a.T + t0 + tid] = make_float2(m, sum);
}

// ---- gradients ---------------------------------------------------------------

constexpr int GT = 128;     // threads of a block
constexpr int ROWS = 256;   // the most rows whose P is staged together

// rows of a thread that are loaded together, beside the last ones' sums: 64 bytes, or eight
template <typename E, int C>
__host__ __device__ constexpr int rows_ahead() {
    return C * sizeof(E) == 16 ? 4 : 8;
}

// Sums of two tokens in one register pair: half the instructions
template <int TT> struct Tokens {
    static constexpr int N = 2;
    using type = F2;
    static __device__ __forceinline__ F2 make(float x, float y) { return f2(x, y); }
    static __device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) { return f2_fma(a, b, c); }
    static __device__ __forceinline__ float sum(F2 a) { return f2_sum(a); }
    static __device__ __forceinline__ float of(F2 a, int odd) { return odd ? a.y() : a.x(); }
};
template <> struct Tokens<1> {
    static constexpr int N = 1;
    using type = float;
    static __device__ __forceinline__ float make(float x, float) { return x; }
    static __device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
    static __device__ __forceinline__ float sum(float a) { return a; }
    static __device__ __forceinline__ float of(float a, int) { return a; }
};
// blocks of an SM: all run at the same time
__host__ __device__ constexpr int resident(int TT) { return TT == 1 ? 6 : TT == 4 ? 4 : 3; }

struct GradArgs {
    FewArgs a;
    const float* dloss; const float* P;
    float* parts;      // [gridDim.y][T][W]
    void* dw; int64_t lddw;
    int lanes;         // log2 of the threads along a row; the others take other rows
    int rows;          // of a chunk
};

template <typename E, int TT, int C>
__global__ void __launch_bounds__(GT, resident(TT)) few_grads_kernel(const GradArgs p) {
    using X = Piece<E, C>;
    using raw = typename X::raw;
    constexpr int GU = rows_ahead<E, C>();
    using A = Tokens<TT>;
    constexpr int TP = TT / A::N;
    using V = typename A::type;
    __shared__ __align__(16) float Ps[ROWS][TT];
    __shared__ float fold[GT][C];
    const FewArgs& a = p.a;
    const int tid = threadIdx.x, wide = 1 << p.lanes, x = tid & (wide - 1), y = tid >> p.lanes, ny = GT >> p.lanes;
    const int col = (blockIdx.x * wide + x) * C;
    const bool real = col < a.W;
    V h[TP][C], dh[TP][C];
    auto of_h = [&](int t, int j) {
        // (a token without a gradient counts as zeros, whatever it holds)
        const bool live = real && t < a.T && target_at(a, t) >= 0 && __ldg(p.dloss + t) != 0.f;
        return live ? Elem<E>::load(static_cast<const E*>(a.h) + t * a.ldh + col + j) : 0.f;
    };
#pragma unroll
    for (int t = 0; t < TP; ++t)
#pragma unroll
        for (int j = 0; j < C; ++j) {
            h[t][j] = A::make(of_h(A::N * t, j), A::N > 1 ? of_h(A::N * t + 1, j) : 0.f);
            dh[t][j] = A::make(0.f, 0.f);
        }
    const int v0 = blockIdx.y * p.rows, v1 = min(a.V, v0 + p.rows);
    const int batch = GU * ny, tile = max(batch, 64);
    const E* w = static_cast<const E*>(a.w) + col;
    E* dw = static_cast<E*>(p.dw) + col;
    raw next[GU];
    auto load = [&](int v) {
#pragma unroll
        for (int u = 0; u < GU; ++u)
            if (real && v + u * ny < v1) next[u] = __ldg(reinterpret_cast<const raw*>(w + (v + u * ny) * a.ldw));
    };
    load(v0 + y);
    for (int b = v0; b < v1; b += tile) {
        const int n = min(tile, v1 - b);
        __syncthreads();
        for (int i = tid; i < n * TT; i += GT) {
            const int v = i / TT, t = i % TT;
            Ps[v][t] = t < a.T ? __ldg(p.P + (int64_t)(b + v) * a.T + t) : 0.f;
        }
        __syncthreads();
        for (int i0 = y; i0 < n; i0 += batch) {
            raw now[GU];
#pragma unroll
            for (int u = 0; u < GU; ++u) now[u] = next[u];
            load(b + i0 + batch);
#pragma unroll
            for (int u = 0; u < GU; ++u) {
                const int i = i0 + u * ny;
                if (i >= n || !real) break;
                float f[C];
                V d[C];
                X::to_f(now[u], f);
#pragma unroll
                for (int j = 0; j < C; ++j) d[j] = A::make(0.f, 0.f);
#pragma unroll
                for (int t = 0; t < TP; ++t) {
                    const V P = *reinterpret_cast<const V*>(&Ps[i][A::N * t]);
#pragma unroll
                    for (int j = 0; j < C; ++j) {
                        dh[t][j] = A::fma(P, A::make(f[j], f[j]), dh[t][j]);
                        d[j] = A::fma(P, h[t][j], d[j]);
                    }
                }
#pragma unroll
                for (int j = 0; j < C; ++j) f[j] = A::sum(d[j]);
                *reinterpret_cast<raw*>(dw + (b + i) * p.lddw) = X::from_f(f);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        if (t >= a.T) break;
        float s[C];
#pragma unroll
        for (int j = 0; j < C; ++j) s[j] = A::of(dh[t / A::N][j], t & 1);
        if (ny > 1) {  // the same columns of other threads
            __syncthreads();
#pragma unroll
            for (int j = 0; j < C; ++j) fold[tid][j] = s[j];
            __syncthreads();
            if (y) continue;
            for (int i = 1; i < ny; ++i)
#pragma unroll
                for (int j = 0; j < C; ++j) s[j] += fold[(i << p.lanes) + x][j];
        }
        float* o = p.parts + ((int64_t)blockIdx.y * a.T + t) * a.W + col;
        if (real) {
#pragma unroll
            for (int j = 0; j < C; ++j) o[j] = s[j];
        }
    }
}

// dh of a token's 32 columns from its parts, in 32 runs
template <typename E>
__global__ void __launch_bounds__(1024) few_join_kernel(const float* __restrict__ parts, int n, int T, int W,
                                                        E* __restrict__ dh, int64_t lddh) {
    __shared__ float sum[32][33];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5, t = blockIdx.y, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < W) {
#pragma unroll 8
        for (int i = g; i < n; i += 32) s += __ldg(parts + ((int64_t)i * T + t) * W + c);
    }
    sum[g][lane] = s;
    __syncthreads();
    // a warp a column
    s = sum[lane][g];
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int col = blockIdx.x * 32 + g;
    if (lane == 0 && col < W) dh[t * lddh + col] = Elem<E>::from_f(s);
}

// ---- host --------------------------------------------------------------------

int up(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// The most tokens of these kernels: of fp32, of bf16 rows that the tensor cores' copies read in place,
// of other bf16 rows.  Loss and gradients in us, here and by the tensor cores:
//   fp32  32000 x 2048   1 token  48 + 136, 239 + 440;  8  62 + 169, 196 + 367;  16  89 + 240, 155 + 324;
//                        32 tokens  167 + 505, 189 + 363
//   bf16  64000 x 2048   1 token  49 + 138, 64 + 175;  4  55 + 159, 58 + 175;  8  72 + 214, 59 + 173
//         35215 x 832    1 token  18 + 40, 21 + 63;  4  22 + 56, 21 + 63;  8  29 + 78, 20 + 59
//         64000 x 2046   4 tokens  55 + 201, 160 + 329;  8  72 + 261, 158 + 327;  16  135 + 449, 158 + 327
constexpr int kFewF32 = 16, kFewBf16 = 4, kFewBf16Odd = 8;
constexpr int kLeastRows = 64;  // of w: fewer would leave most warps without any
constexpr size_t kSmem = 200 << 10;  // of h
constexpr int kMaxParts = 608;

// elements of an access of w's (and dw's) rows: as many as width, strides and addresses allow
int access(int most, size_t e, int W, const void* x, int64_t ldx, const void* y, int64_t ldy) {
    int n = most;
    while (n > 1 && (W % n || ldx % n || ldy % n || (reinterpret_cast<uintptr_t>(x) & (n * e - 1)) ||
                     (reinterpret_cast<uintptr_t>(y) & (n * e - 1))))
        n /= 2;
    return n;
}

int tokens_of(int T) { return T == 1 ? 1 : T <= 4 ? 4 : kGroup; }  // of a block of the logits

template <typename E, int TT, int VEC>
gdn_status launch_logits(LogitArgs p, cudaStream_t s) {
    const void* fn = (const void*)few_logits_kernel<E, TT, VEC>;
    const size_t smem = sizeof(float) * TT * (size_t)padded(p.a.W, 32 * VEC * pieces<E, VEC>());
    gdn_status st = set_smem_attr(fn, kSmem);
    if (st != GDN_OK) return st;
    p.groups = up(p.a.T, TT);
    few_logits_kernel<E, TT, VEC><<<(unsigned)(few_blocks(p.a.T, p.a.V) * p.groups), LT, smem, s>>>(p);
    return check_launch("few_logits_kernel");
}
template <typename E, int VEC>
gdn_status logits_tokens(const LogitArgs& p, cudaStream_t s) {
    const int tt = tokens_of(p.a.T);
    if (tt == 1) return launch_logits<E, 1, VEC>(p, s);
    if constexpr (VEC < 8)  // (rows of eights: up to four tokens)
        if (tt == 8) return launch_logits<E, 8, VEC>(p, s);
    return launch_logits<E, 4, VEC>(p, s);
}
gdn_status run_logits(const LogitArgs& p, cudaStream_t s) {
    const FewArgs& a = p.a;
    if (a.dtype == GDN_F32) {
        const int n = access(4, 4, a.W, a.w, a.ldw, a.w, a.ldw);
        return n == 4 ? logits_tokens<float, 4>(p, s)
                      : n == 2 ? logits_tokens<float, 2>(p, s) : logits_tokens<float, 1>(p, s);
    }
    const int n = access(8, 2, a.W, a.w, a.ldw, a.w, a.ldw);
    return n == 8 ? logits_tokens<__nv_bfloat16, 8>(p, s)
                  : n >= 2 ? logits_tokens<__nv_bfloat16, 2>(p, s) : logits_tokens<__nv_bfloat16, 1>(p, s);
}

// blocks of rows and of columns of the gradients
int grad_slabs(int W, int C, int& lanes) {
    lanes = 7;
    while (lanes > 2 && (C << (lanes - 1)) >= W) --lanes;
    return up(W, C << lanes);
}
int grad_chunks(int V, int slabs, int per_sm) {
    int n = device_sm_count() * per_sm / slabs;
    if (n > kMaxParts) n = kMaxParts;
    if (n > up(V, 64)) n = up(V, 64);
    return n < 1 ? 1 : n;
}

template <typename E, int TT, int C>
gdn_status launch_grads(GradArgs p, void* dh, int64_t lddh, cudaStream_t s) {
    const int slabs = grad_slabs(p.a.W, C, p.lanes);
    p.rows = up(p.a.V, grad_chunks(p.a.V, slabs, resident(TT)));
    const int chunks = up(p.a.V, p.rows);
    few_grads_kernel<E, TT, C><<<dim3(slabs, chunks), GT, 0, s>>>(p);
    gdn_status st = check_launch("few_grads_kernel");
    if (st != GDN_OK) return st;
    few_join_kernel<E><<<dim3(up(p.a.W, 32), p.a.T), 1024, 0, s>>>(p.parts, chunks, p.a.T, p.a.W, static_cast<E*>(dh), lddh);
    return check_launch("few_join_kernel");
}
int grad_tokens(int T) { return T == 1 ? 1 : T <= 4 ? 4 : T <= 8 ? 8 : 16; }
// columns of a thread: what 32 registers each hold of h and dh
constexpr int columns(int tt, int e) {
    const int n = tt == 1 ? 8 : tt <= 8 ? 4 : 2;
    return n < 16 / e ? n : 16 / e;
}

template <typename E, int TT>
gdn_status grads_tokens(const GradArgs& p, int n, void* dh, int64_t lddh, cudaStream_t s) {
    constexpr int C = columns(TT, sizeof(E));
    if (n >= C) return launch_grads<E, TT, C>(p, dh, lddh, s);
    if constexpr (sizeof(E) == 2)
        if (n >= 2) return launch_grads<E, TT, 2>(p, dh, lddh, s);
    return launch_grads<E, TT, 1>(p, dh, lddh, s);
}
template <typename E>
gdn_status run_grads(const GradArgs& p, int n, void* dh, int64_t lddh, cudaStream_t s) {
    const int tt = grad_tokens(p.a.T);
    if (tt == 1) return grads_tokens<E, 1>(p, n, dh, lddh, s);
    if (tt == 4) return grads_tokens<E, 4>(p, n, dh, lddh, s);
    if constexpr (sizeof(E) == 4)
        if (tt == 16) return grads_tokens<E, 16>(p, n, dh, lddh, s);
    return grads_tokens<E, 8>(p, n, dh, lddh, s);
}

}  // namespace

bool few_takes(int T, int V, int W, gdn_dtype dtype) {
    return V >= kLeastRows && T <= (dtype == GDN_F32 ? kFewF32 : W % 8 ? kFewBf16Odd : kFewBf16) &&
           sizeof(float) * tokens_of(T) * (size_t)padded(W, 256) <= kSmem;
}

int few_blocks(int T, int V) {
    const int groups = up(T, tokens_of(T));
    const int most = device_sm_count() / groups, sets = up(V, rows_of(tokens_of(T)));
    return most < sets ? (most < 1 ? 1 : most) : sets;
}

gdn_status few_logits(const FewArgs& a, float2* stat, float* at, cudaStream_t s) {
    LogitArgs p{};
    p.a = a;
    p.stat = stat;
    p.at = at;
    return run_logits(p, s);
}

int few_parts(int T, int V, int W, gdn_dtype dtype) {
    const int tt = grad_tokens(T);
    int lanes;
    return grad_chunks(V, grad_slabs(W, columns(tt, dtype == GDN_F32 ? 4 : 2), lanes), resident(tt));
}

gdn_status few_grads(const FewArgs& a, const float* dloss, const float* loss, const float* lse, float* P, float* parts,
                     void* dh, int64_t lddh, void* dw, int64_t lddw, cudaStream_t s) {
    LogitArgs l{};
    l.a = a;
    l.dloss = dloss;
    l.loss = loss;
    l.lse = lse;
    l.P = P;
    gdn_status st = run_logits(l, s);
    if (st != GDN_OK) return st;
    GradArgs p{};
    p.a = a;
    p.dloss = dloss;
    p.P = P;
    p.parts = parts;
    p.dw = dw;
    p.lddw = lddw;
    const int n = access(a.dtype == GDN_F32 ? 4 : 8, a.dtype == GDN_F32 ? 4 : 2, a.W, a.w, a.ldw, dw, lddw);
    return a.dtype == GDN_F32 ? run_grads<float>(p, n, dh, lddh, s) : run_grads<__nv_bfloat16>(p, n, dh, lddh, s);
}

}  // namespace gdn
