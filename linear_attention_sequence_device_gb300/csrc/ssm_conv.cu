// The selective scan layer's short convolution over packed sequences, each with
// its own state: forward, gradient, single-token form and the C entry points.
//
// Forward: pre[t] = b + sum_j w[j] x'[t - K + 1 + j], y = pre s(pre), s the
// logistic function.  Backward, with ds[t] = dy s (1 + pre (1 - s)):
//   dx'[t] = sum_j w[j] ds[t + K - 1 - j] within the sequence,
//   dw[j] = sum_t ds[t] x'[t - K + 1 + j],  db = sum_t ds[t];
// the gradients of the K - 1 rows before a sequence's start are its state's,
// and dstate_out adds to the last K - 1 rows.
#include "chunk_common.cuh"
#include "ssm_common.cuh"

namespace gdn {

gdn_status set_smem_attr(const void* func, size_t bytes);

namespace {

constexpr int NT = 128;
constexpr int CV = 4;   // channels per thread of the backward
constexpr int RB = 4;   // rows per batch

// four channels as they come, and as two pairs
template <typename T> struct Raw4;
template <> struct Raw4<__nv_bfloat16> {
    uint2 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint2*>(p)); }
    __device__ __forceinline__ void take(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void unpack(F2 (&f)[2]) const {
        f[0] = f2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u));
        f[1] = f2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const F2 (&f)[2]) {
        uint2 r;
        __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&r);
        h[0] = __floats2bfloat162_rn(f[0].x(), f[0].y());
        h[1] = __floats2bfloat162_rn(f[1].x(), f[1].y());
        *reinterpret_cast<uint2*>(p) = r;
    }
};
template <> struct Raw4<float> {
    ulonglong2 v;
    __device__ __forceinline__ void load(const float* p) { v = __ldg(reinterpret_cast<const ulonglong2*>(p)); }
    __device__ __forceinline__ void take(const float* p) { v = *reinterpret_cast<const ulonglong2*>(p); }
    __device__ __forceinline__ void unpack(F2 (&f)[2]) const { f[0].b = v.x; f[1].b = v.y; }
    static __device__ __forceinline__ void store(float* p, const F2 (&f)[2]) { f2_store2(p, f[0], f[1]); }
};

struct ConvParams {
    const void* x; int64_t ldx;
    const void* w; const void* b;
    int T, C;
    const int32_t* cu; int num_seqs;
    const void* state; void* state_out;
    void* y; int64_t ldy;
    int rows;  // rows per strip, a multiple of RB
};

// weights of N channels from c0 on, as pairs of channels
template <typename T, int K, int N>
__device__ __forceinline__ void load_weights(const void* w, const void* b, int c0, F2 (&wv)[K][N / 2], F2 (&bv)[N / 2]) {
    const T *wp = static_cast<const T*>(w) + (int64_t)c0 * K, *bp = static_cast<const T*>(b) + c0;
#pragma unroll
    for (int h = 0; h < N / 2; ++h) {
#pragma unroll
        for (int j = 0; j < K; ++j)
            wv[j][h] = f2(Elem<T>::to_f(wp[2 * h * K + j]), Elem<T>::to_f(wp[(2 * h + 1) * K + j]));
        bv[h] = b ? f2(Elem<T>::to_f(bp[2 * h]), Elem<T>::to_f(bp[2 * h + 1])) : f2_dup(0.f);
    }
}

// Forward.  HBM-bound: x in, y out, each once.  A thread owns eight channels of a
// strip of rows and walks down it with a window of the last K - 1 inputs; rows come
// by asynchronous copies into a ring of kStages batches of RB rows that it fills and
// reads alone.  A batch that no sequence starts in, all but a few, runs without a
// check, which also lets the window stay where it is instead of moving up row by
// row.  A block's threads cover 1024 channels, so that of 2112 channels the third
// block has 8 threads at work and holds a slot all the same (fp32, 30038 rows: 138 us
// for 75 us of bytes; 4096 channels, 32768 rows: 245 for 159).  The SiLU is a / (1 + e^-a) for both types, so that a bf16 result is off by
// its own rounding only; in pairs that is 3 issue slots an element.
template <typename T>
constexpr int kStages = sizeof(T) == 4 ? 3 : 4;  // four blocks' rings fit an SM (fp32, 30038 x 2112: 172 us with 4)
template <typename T, int K>
__global__ void __launch_bounds__(NT, 4) conv_fwd_kernel(const ConvParams p) {
    constexpr int NST = kStages<T>;
    constexpr int H = K > 1 ? K - 1 : 1, VEC = sizeof(T) * 8 / 16;
    const int c0 = (blockIdx.x * NT + threadIdx.x) * 8;
    if (c0 >= p.C) return;
    const int nseq = p.num_seqs, tid = threadIdx.x;
    const int32_t* cu = p.cu;
    const T* x = static_cast<const T*>(p.x) + c0;
    T* y = static_cast<T*>(p.y) + c0;
    F2 win[H][4];
    auto load_state = [&](int seq) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            if (p.state) f2_load8(static_cast<const T*>(p.state) + ((int64_t)seq * (K - 1) + j) * p.C + c0, win[j]);
            else
#pragma unroll
                for (int i = 0; i < 4; ++i) win[j][i] = f2_dup(0.f);
        }
    };
    auto store_state = [&](int seq) {  // exact: the window holds the values as loaded
        if (p.state_out)
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
                f2_store8(static_cast<T*>(p.state_out) + ((int64_t)seq * (K - 1) + j) * p.C + c0, win[j]);
    };
    auto pass_empty = [&](int seq) {  // its final state is its initial one
        load_state(seq);
        store_state(seq);
    };
    if (p.T == 0) {
        if (blockIdx.y == 0)
            for (int m = 0; m < nseq; ++m) pass_empty(m);
        return;
    }
    const int lt0 = blockIdx.y * p.rows, lt1 = min(p.T, lt0 + p.rows);
    if (lt0 >= p.T) return;
    int seg = seq_of(cu, nseq, lt0);
    const int start = __ldg(cu + seg);
    int next = __ldg(cu + seg + 1);
    if (start == lt0)  // empty sequences that end where this strip starts
        for (int m = seg - 1; m >= 0 && __ldg(cu + m) == lt0; --m) pass_empty(m);

    extern __shared__ uint4 ring[];  // [NST][RB][VEC][NT]
    const int nb = (lt1 - lt0 + RB - 1) / RB;
    auto issue = [&](int b) {
        if (b < nb) {
            uint4* st = ring + (size_t)(b % NST) * RB * VEC * NT + tid;
#pragma unroll
            for (int u = 0; u < RB; ++u) {
                const int t = lt0 + RB * b + u;
                const T* src = x + (int64_t)min(t, lt1 - 1) * p.ldx;
#pragma unroll
                for (int v = 0; v < VEC; ++v)
                    cp_async16(st + (u * VEC + v) * NT, reinterpret_cast<const uint4*>(src) + v, t < lt1 ? 16 : 0);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int b = 0; b < NST - 1; ++b) issue(b);

    F2 w[K][4], b[4];
    load_weights<T, K, 8>(p.w, p.b, c0, w, b);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const int row = lt0 - (K - 1) + j, m = K - 1 - (start - row);  // m: its row of the state
        if (row >= start && row >= 0) f2_load8(x + (int64_t)row * p.ldx, win[j]);
        else if (p.state && m >= 0 && m < K - 1)
            f2_load8(static_cast<const T*>(p.state) + ((int64_t)seg * (K - 1) + m) * p.C + c0, win[j]);
        else
#pragma unroll
            for (int i = 0; i < 4; ++i) win[j][i] = f2_dup(0.f);
    }
    for (int bt = 0; bt < nb; ++bt) {
        issue(bt + NST - 1);
        cp_async_wait<NST - 1>();
        const uint4* st = ring + (size_t)(bt % NST) * RB * VEC * NT + tid;
        const int tb = lt0 + RB * bt;
        auto row = [&](int u) {
            uint4 raw[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) raw[v] = st[(u * VEC + v) * NT];
            F2 cur[4], out[4];
            f2_load8(reinterpret_cast<const T*>(raw), cur);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                F2 a = b[i];
#pragma unroll
                for (int j = 0; j < K - 1; ++j) a = f2_fma(w[j][i], win[j][i], a);
                out[i] = f2_silu(f2_fma(w[K - 1][i], cur[i], a));
#pragma unroll
                for (int j = 0; j + 1 < K - 1; ++j) win[j][i] = win[j + 1][i];
                if (K > 1) win[H - 1][i] = cur[i];
            }
            f2_store8(y + (int64_t)(tb + u) * p.ldy, out);
        };
        if (tb + RB <= lt1 && next >= tb + RB) {
#pragma unroll
            for (int u = 0; u < RB; ++u) row(u);
        } else {
#pragma unroll 1
            for (int u = 0; u < RB && tb + u < lt1; ++u) {
                while (tb + u == next) {  // a sequence ends and the next one starts
                    store_state(seg);
                    if (++seg >= nseq) {
                        next = p.T;  // malformed cu
                    } else {
                        load_state(seg);
                        next = __ldg(cu + seg + 1);
                    }
                }
                row(u);
            }
        }
    }
    cp_async_wait<0>();
    if (next == lt1 && seg < nseq) {  // the sequence ends with the strip
        store_state(seg);
        if (lt1 == p.T)  // empty sequences behind the last token
            for (int m = seg + 1; m < nseq; ++m) pass_empty(m);
    }
}

// four channels' copy, 8 or 16 bytes
__device__ __forceinline__ void copy4(__nv_bfloat16* dst, const __nv_bfloat16* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src));
}
__device__ __forceinline__ void copy4(float* dst, const float* src) { cp_async16(dst, src, 16); }

struct ConvBwdParams {
    const void* dy; int64_t lddy;
    const void* x; int64_t ldx;
    const void* w; const void* b;
    int T, C;
    const int32_t* cu; int num_seqs;
    const void* state; const float* dso;
    void* dx; int64_t lddx;
    float* dstate;
    float* part;  // [strips, C K + C]
    int rows;     // rows per strip
};

// HBM-bound: x and dy in, dx out, each once.  A thread owns four channels of a
// strip of rows and walks down it with a window of the last K - 1 inputs and of
// the K - 1 rows whose dx is not complete yet.  A strip runs K - 1 rows past
// its end (within the sequence) for the dx of its own last rows; those rows'
// dw and db belong to the next strip.  Groups of four rows that touch no sequence's
// end and no strip's edge, all but a few, run without a check.  Channels go in
// pairs through the two-wide instructions: single ones took 44 issue slots an
// element, which bounded it at 290 us for 65536 x 2048.  x and dy come through a ring
// as in the forward.
constexpr int NSTAGE = 4;
template <typename T, int K>
__global__ void __launch_bounds__(NT, 4) conv_bwd_kernel(const ConvBwdParams p) {
    constexpr int H = K > 1 ? K - 1 : 1;
    const int c0 = (blockIdx.x * NT + threadIdx.x) * CV;
    if (c0 >= p.C) return;
    const int nseq = p.num_seqs;
    const int32_t* cu = p.cu;
    const T* x = static_cast<const T*>(p.x) + c0;
    const T* dy = static_cast<const T*>(p.dy) + c0;
    T* dx = static_cast<T*>(p.dx) + c0;

    auto end_grad = [&](int seq, int j, F2 (&f)[2]) {  // dstate_out row j
        if (p.dso) {
            Raw4<float> r;
            r.load(p.dso + ((int64_t)seq * (K - 1) + j) * p.C + c0);
            r.unpack(f);
        } else {
            f[0] = f[1] = f2_dup(0.f);
        }
    };
    auto put_state = [&](int seq, int j, const F2 (&f)[2]) {
        if (p.dstate) Raw4<float>::store(p.dstate + ((int64_t)seq * (K - 1) + j) * p.C + c0, f);
    };
    auto pass_empty = [&](int seq) {  // its final state is its initial one
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            F2 f[2];
            end_grad(seq, j, f);
            put_state(seq, j, f);
        }
    };

    F2 w[K][2], b[2], dw[K][2], db[2];
    const F2 zero = f2_dup(0.f), one = f2_dup(1.f), neg = f2_dup(-1.f);
    load_weights<T, K, 4>(p.w, p.b, c0, w, b);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < K; ++j) dw[j][h] = zero;
        db[h] = zero;
    }
    const int lt0 = blockIdx.y * p.rows, lt1 = min(p.T, lt0 + p.rows);
    if (p.T == 0) {
        if (blockIdx.y == 0)
            for (int m = 0; m < nseq; ++m) pass_empty(m);
    } else if (lt0 < p.T) {
        int seg = seq_of(cu, nseq, lt0);
        int start = __ldg(cu + seg), next = __ldg(cu + seg + 1);
        if (start == lt0)  // empty sequences that end where this strip starts
            for (int m = seg - 1; m >= 0 && __ldg(cu + m) == lt0; --m) pass_empty(m);
        F2 win[H][2], acc[H][2];
        auto load_state = [&](int j, F2 (&f)[2]) {
            if (p.state) {
                Raw4<T> r;
                r.load(static_cast<const T*>(p.state) + ((int64_t)seg * (K - 1) + j) * p.C + c0);
                r.unpack(f);
            } else {
                f[0] = f[1] = zero;
            }
        };
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const int row = lt0 - (K - 1) + j, m = K - 1 - (start - row);
            acc[j][0] = acc[j][1] = zero;
            if (row >= start && row >= 0) {
                Raw4<T> r;
                r.load(x + (int64_t)row * p.ldx);
                r.unpack(win[j]);
            } else if (m >= 0 && m < K - 1) {
                load_state(m, win[j]);
            } else {
                win[j][0] = win[j][1] = zero;
            }
        }
        auto emit = [&](int row, const F2 (&f)[2]) {
            if (row >= start) {
                if (row >= lt0 && row < lt1) Raw4<T>::store(dx + (int64_t)row * p.lddx, f);
            } else if (start >= lt0) {
                const int m = K - 1 - (start - row);
                if (m >= 0 && m < K - 1) put_state(seg, m, f);
            }
        };
        // one row: ds, the sums, and the dx that it completes (of the row K - 1 before it)
        auto step = [&](const Raw4<T>& rx, const Raw4<T>& ry, bool own, F2 (&first)[2]) {
            F2 xv[2], g[2];
            rx.unpack(xv);
            ry.unpack(g);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                F2 pre = b[h];
#pragma unroll
                for (int j = 0; j < K - 1; ++j) pre = f2_fma(w[j][h], win[j][h], pre);
                pre = f2_fma(w[K - 1][h], xv[h], pre);
                const F2 sg = f2_sigmoid(pre);
                const F2 ds = f2_mul(f2_mul(g[h], sg), f2_fma(pre, f2_fma(sg, neg, one), one));
                if (own) {
#pragma unroll
                    for (int j = 0; j < K - 1; ++j) dw[j][h] = f2_fma(ds, win[j][h], dw[j][h]);
                    dw[K - 1][h] = f2_fma(ds, xv[h], dw[K - 1][h]);
                    db[h] = f2_add(db[h], ds);
                }
                first[h] = K > 1 ? f2_fma(w[0][h], ds, acc[0][h]) : f2_mul(w[0][h], ds);
#pragma unroll
                for (int j = 0; j + 1 < K - 1; ++j) {
                    acc[j][h] = f2_fma(w[j + 1][h], ds, acc[j + 1][h]);
                    win[j][h] = win[j + 1][h];
                }
                if (K > 1) {
                    acc[H - 1][h] = f2_mul(w[K - 1][h], ds);
                    win[H - 1][h] = xv[h];
                }
            }
        };
        const int tend = min(p.T, lt1 + K - 1), nb = (tend - lt0 + RB - 1) / RB;
        extern __shared__ uint4 ring[];  // [NSTAGE][RB][x, dy][NT][CV] elements
        auto slot = [&](int b, int u, int a) {
            return reinterpret_cast<T*>(ring) + (((b % NSTAGE * RB + u) * 2 + a) * NT + threadIdx.x) * CV;
        };
        auto issue = [&](int b) {
            if (b < nb)
#pragma unroll
                for (int u = 0; u < RB; ++u) {
                    const int r = min(lt0 + RB * b + u, tend - 1);
                    copy4(slot(b, u, 0), x + (int64_t)r * p.ldx);
                    copy4(slot(b, u, 1), dy + (int64_t)r * p.lddy);
                }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < NSTAGE - 1; ++i) issue(i);
        bool done = false;
        for (int bt = 0; bt < nb && !done; ++bt) {
            const int tb = lt0 + RB * bt;
            issue(bt + NSTAGE - 1);
            cp_async_wait<NSTAGE - 1>();
            Raw4<T> cx[RB], cy[RB];
#pragma unroll
            for (int u = 0; u < RB; ++u) {
                cx[u].take(slot(bt, u, 0));
                cy[u].take(slot(bt, u, 1));
            }
            if (tb + RB <= lt1 && next > tb + RB && tb - (K - 1) >= max(start, lt0)) {
                T* out = dx + (int64_t)(tb - (K - 1)) * p.lddx;
#pragma unroll
                for (int u = 0; u < RB; ++u) {
                    F2 first[2];
                    step(cx[u], cy[u], true, first);
                    Raw4<T>::store(out + u * p.lddx, first);
                }
                continue;
            }
#pragma unroll
            for (int u = 0; u < RB; ++u) {
                const int t = tb + u;
                if (t == next && !done) {  // a new sequence
                    if (t >= lt1) done = true;
                    else {
                        while (seg + 1 < nseq) {
                            ++seg;
                            next = __ldg(cu + seg + 1);
                            if (next != t) break;
                            pass_empty(seg);
                        }
                        start = t;
#pragma unroll
                        for (int j = 0; j < K - 1; ++j) {
                            load_state(j, win[j]);
                            acc[j][0] = acc[j][1] = zero;
                        }
                    }
                }
                if (done || t >= tend) continue;
                F2 first[2];
                step(cx[u], cy[u], t < lt1, first);
                emit(t - (K - 1), first);
                if (t + 1 == next) {  // the sequence ends: its last rows are complete
#pragma unroll
                    for (int j = 0; j < K - 1; ++j) {
                        F2 f[2];
                        end_grad(seg, j, f);
                        f[0] = f2_add(f[0], acc[j][0]);
                        f[1] = f2_add(f[1], acc[j][1]);
                        emit(t - (K - 1) + 1 + j, f);
                    }
                }
            }
        }
        cp_async_wait<0>();
        if (lt1 == p.T && next == p.T)
            for (int m = seg + 1; m < nseq; ++m) pass_empty(m);
    }
    float* part = p.part + (int64_t)blockIdx.y * p.C * (K + 1);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < K; ++j) {
            part[(int64_t)(c0 + 2 * h) * K + j] = dw[j][h].x();
            part[(int64_t)(c0 + 2 * h + 1) * K + j] = dw[j][h].y();
        }
    Raw4<float>::store(part + (int64_t)p.C * K + c0, db);
}

// One token per request: read K - 1 state rows, write K - 1 (shifted) and y.
// Bound by those bytes (or, for a few requests, by the launch): a thread holds the
// weights of eight channels and takes the requests gridDim.y apart, the next one's
// rows on their way while it works on one (256 requests of 8192 channels in bf16,
// states in L2: 5.8 us, 7.7 without).
template <typename T>
constexpr int kStepBlocks = sizeof(T) == 4 ? 3 : 4;  // resident on an SM
template <typename T, int K>
__global__ void __launch_bounds__(NT, kStepBlocks<T>) conv_step_kernel(const T* x, int64_t ldx, int batch, int C, const T* w,
                                                       const T* bias, T* states, int num_slots, const int32_t* src,
                                                       const int32_t* dst, T* y, int64_t ldy) {
    const int c0 = (blockIdx.x * NT + threadIdx.x) * 8;
    if (c0 >= C) return;
    float wv[8 * K], b[8];
    const T* wp = w + (int64_t)c0 * K;
    if ((reinterpret_cast<uintptr_t>(w) & 15u) == 0) {
#pragma unroll
        for (int j = 0; j < K; ++j) load8(wp + 8 * j, *reinterpret_cast<float(*)[8]>(wv + 8 * j));
    } else {
#pragma unroll
        for (int i = 0; i < 8 * K; ++i) wv[i] = Elem<T>::to_f(wp[i]);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) b[c] = bias ? Elem<T>::to_f(bias[c0 + c]) : 0.f;
    constexpr int VEC = sizeof(T) * 8 / 16;
    struct Raw {
        uint4 v[K][VEC];  // the state's rows and x, as they lie in memory
        int from, to;     // slots read (-1: none) and written (-1: a padded row)
    };
    auto fetch = [&](int r, Raw& w) {
        w.from = w.to = -1;
        if (r >= batch) return;
        w.to = dst ? __ldg(dst + r) : r;
        w.from = src ? __ldg(src + r) : r;
        if (w.to >= num_slots) w.to = -1;
        if (w.to < 0) return;
        if (w.from >= num_slots) w.from = -1;
        const T* in = states + (int64_t)w.from * (K - 1) * C + c0;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
                w.v[j][v] = w.from >= 0 ? reinterpret_cast<const uint4*>(in + (int64_t)j * C)[v] : make_uint4(0, 0, 0, 0);
            w.v[K - 1][v] = __ldg(reinterpret_cast<const uint4*>(x + (int64_t)r * ldx + c0) + v);
        }
    };
    Raw cur, nxt;
    fetch(blockIdx.y, cur);
    for (int r = blockIdx.y; r < batch; r += gridDim.y) {
        fetch(r + gridDim.y, nxt);
        T* yr = y + (int64_t)r * ldy + c0;
        float f[8];
        if (cur.to < 0) {
#pragma unroll
            for (int c = 0; c < 8; ++c) f[c] = 0.f;
        } else {
            T* out = states + (int64_t)cur.to * (K - 1) * C + c0;
#pragma unroll
            for (int j = 1; j < K; ++j)
#pragma unroll
                for (int v = 0; v < VEC; ++v) reinterpret_cast<uint4*>(out + (int64_t)(j - 1) * C)[v] = cur.v[j][v];
#pragma unroll
            for (int c = 0; c < 8; ++c) f[c] = b[c];
#pragma unroll
            for (int j = 0; j < K; ++j) {
                float row[8];
                load8_rw(reinterpret_cast<const T*>(cur.v[j]), row);
#pragma unroll
                for (int c = 0; c < 8; ++c) f[c] = fmaf(wv[c * K + j], row[c], f[c]);
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) f[c] = silu_fast(f[c]);
        }
        store8(yr, f);
        cur = nxt;
    }
}

// Strips of the backward: one wave of four resident blocks an SM, of 16 rows at least
// (104 rows: 13 us, 23 with 64), whole waves of kLongestSum rows at most.
int bwd_strips(int T, int C) {
    const int nx = (C / CV + NT - 1) / NT, wave = device_sm_count() * 4 / nx, most = T / 16;
    int64_t n = blocks_for_sum(T, wave > 1 ? wave : 1);
    if (n > most) n = most;
    if (n > 65535) n = 65535;
    return n < 1 ? 1 : (int)n;
}

template <typename T, int K>
gdn_status run_fwd_k(ConvParams p, cudaStream_t s) {
    constexpr size_t smem = (size_t)kStages<T> * RB * sizeof(T) * 8 * NT;
    static_assert(smem <= (48 << 10), "dynamic shared memory that needs no attribute");
    // Strips: one wave of four blocks an SM, of 8 rows at least: the K - 1 rows before a strip
    // are read twice, but a strip's rows follow one another (104 rows: 23 us at 64, 9 at 8).
    const int nx = (p.C / 8 + NT - 1) / NT;
    int n = device_sm_count() * 4 / nx;
    if (n > p.T / 8) n = p.T / 8;
    if (n > 65535) n = 65535;
    if (n < 1) n = 1;
    p.rows = p.T > 0 ? ((p.T + n - 1) / n + RB - 1) / RB * RB : RB;
    const int strips = p.T > 0 ? (p.T + p.rows - 1) / p.rows : 1;
    conv_fwd_kernel<T, K><<<dim3(nx, strips), NT, smem, s>>>(p);
    return check_launch("conv_fwd_kernel");
}
template <typename T>
gdn_status run_fwd(const ConvParams& p, int K, cudaStream_t s) {
    switch (K) {
        case 1: return run_fwd_k<T, 1>(p, s);
        case 2: return run_fwd_k<T, 2>(p, s);
        case 3: return run_fwd_k<T, 3>(p, s);
        default: return run_fwd_k<T, 4>(p, s);
    }
}

template <typename T, int K>
gdn_status run_bwd_k(const ConvBwdParams& p, dim3 grid, cudaStream_t s) {
    constexpr size_t smem = (size_t)NSTAGE * RB * 2 * NT * CV * sizeof(T);
    if (smem > (48 << 10)) {
        const gdn_status st = set_smem_attr((const void*)conv_bwd_kernel<T, K>, smem);
        if (st != GDN_OK) return st;
    }
    conv_bwd_kernel<T, K><<<grid, NT, smem, s>>>(p);
    return check_launch("conv_bwd_kernel");
}
template <typename T>
gdn_status run_bwd(ConvBwdParams p, int K, cudaStream_t s) {
    const int strips = bwd_strips(p.T, p.C);
    p.rows = p.T > 0 ? (p.T + strips - 1) / strips : 1;
    const dim3 grid((p.C / CV + NT - 1) / NT, strips);
    switch (K) {
        case 1: return run_bwd_k<T, 1>(p, grid, s);
        case 2: return run_bwd_k<T, 2>(p, grid, s);
        case 3: return run_bwd_k<T, 3>(p, grid, s);
        default: return run_bwd_k<T, 4>(p, grid, s);
    }
}

template <typename T>
gdn_status run_step(const void* x, int64_t ldx, int batch, int C, const void* w, const void* bias, int K, void* states,
                    int num_slots, const int32_t* src, const int32_t* dst, void* y, int64_t ldy, cudaStream_t s) {
    const int nx = (C / 8 + NT - 1) / NT, most = (device_sm_count() * kStepBlocks<T> + nx - 1) / nx;  // one wave
    const dim3 grid(nx, batch < most ? batch : most);
    const T *xt = static_cast<const T*>(x), *wt = static_cast<const T*>(w), *bt = static_cast<const T*>(bias);
    T *st = static_cast<T*>(states), *yt = static_cast<T*>(y);
    switch (K) {
        case 1: conv_step_kernel<T, 1><<<grid, NT, 0, s>>>(xt, ldx, batch, C, wt, bt, st, num_slots, src, dst, yt, ldy); break;
        case 2: conv_step_kernel<T, 2><<<grid, NT, 0, s>>>(xt, ldx, batch, C, wt, bt, st, num_slots, src, dst, yt, ldy); break;
        case 3: conv_step_kernel<T, 3><<<grid, NT, 0, s>>>(xt, ldx, batch, C, wt, bt, st, num_slots, src, dst, yt, ldy); break;
        default: conv_step_kernel<T, 4><<<grid, NT, 0, s>>>(xt, ldx, batch, C, wt, bt, st, num_slots, src, dst, yt, ldy); break;
    }
    return check_launch("conv_step_kernel");
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

gdn_status check_conv(gdn_dtype dtype, int rows, int channels, const void* w, int conv_k) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return fail(GDN_ERR_DTYPE, "unknown dtype %d", (int)dtype);
    if (rows < 0 || channels < 1) return fail(GDN_ERR_INVALID_ARG, "rows=%d channels=%d", rows, channels);
    if (rows > kMaxTokens) return fail(GDN_ERR_UNSUPPORTED_SHAPE, "%d tokens, more than %d", rows, kMaxTokens);
    if (channels % 8 != 0) return fail(GDN_ERR_UNSUPPORTED_SHAPE, "channels=%d not a multiple of 8", channels);
    if (conv_k < 1 || conv_k > 4) return fail(GDN_ERR_UNSUPPORTED_SHAPE, "conv_k=%d not in 1..4", conv_k);
    if (!w) return fail(GDN_ERR_INVALID_ARG, "w is NULL");
    return GDN_OK;
}

gdn_status check_rows(const void* p, int64_t ld, int64_t least, const char* name) {
    if (!p || !al16(p)) return fail(GDN_ERR_INVALID_ARG, "%s must be 16-byte aligned and not NULL", name);
    if (ld < least || ld % 8 != 0)
        return fail(GDN_ERR_INVALID_ARG, "row stride of %s (%lld) must be >= %lld and a multiple of 8", name,
                    (long long)ld, (long long)least);
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_ssm_conv_fwd(const void* x, int64_t ldx, gdn_dtype dtype, int32_t T, int32_t channels, const void* w,
                            const void* bias, int32_t conv_k, const int32_t* cu_seqlens, int32_t num_seqs,
                            const void* state, void* state_out, void* y, int64_t ldy, void* stream) {
    gdn_status st = check_conv(dtype, T, channels, w, conv_k);
    if (st != GDN_OK) return st;
    if (num_seqs < 1 || !cu_seqlens) return fail(GDN_ERR_INVALID_ARG, "num_seqs=%d or cu_seqlens is NULL", num_seqs);
    if (!al16(state) || !al16(state_out))
        return fail(GDN_ERR_INVALID_ARG, "state and state_out must be 16-byte aligned");
    if (state && state == state_out) return fail(GDN_ERR_INVALID_ARG, "state_out must not be state");
    if (T > 0) {
        if ((st = check_rows(x, ldx, channels, "x")) != GDN_OK) return st;
        if ((st = check_rows(y, ldy, channels, "y")) != GDN_OK) return st;
        if (x == y) return fail(GDN_ERR_INVALID_ARG, "y must not be x");
    }
    ConvParams p{x, ldx, w, bias, T, channels, cu_seqlens, num_seqs, state, state_out, y, ldy, 0};
    cudaStream_t s = (cudaStream_t)stream;
    return dtype == GDN_BF16 ? run_fwd<__nv_bfloat16>(p, conv_k, s) : run_fwd<float>(p, conv_k, s);
}

size_t gdn_ssm_conv_bwd_workspace_size(int32_t T, int32_t channels, int32_t conv_k) {
    if (T < 0 || T > kMaxTokens || channels < 1 || channels % 8 != 0 || conv_k < 1 || conv_k > 4) return 0;
    return (sizeof(float) * (size_t)channels * (conv_k + 1) * bwd_strips(T, channels) + 255) & ~size_t(255);
}

gdn_status gdn_ssm_conv_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, gdn_dtype dtype, int32_t T,
                            int32_t channels, const void* w, const void* bias, int32_t conv_k,
                            const int32_t* cu_seqlens, int32_t num_seqs, const void* state, const float* dstate_out,
                            void* dx, int64_t lddx, float* dw, float* dbias, float* dstate, void* workspace,
                            size_t workspace_bytes, void* stream) {
    gdn_status st = check_conv(dtype, T, channels, w, conv_k);
    if (st != GDN_OK) return st;
    if (num_seqs < 1 || !cu_seqlens) return fail(GDN_ERR_INVALID_ARG, "num_seqs=%d or cu_seqlens is NULL", num_seqs);
    if (!al16(state) || !al16(dstate_out) || !al16(dstate))
        return fail(GDN_ERR_INVALID_ARG, "state, dstate_out and dstate must be 16-byte aligned");
    if (!dw) return fail(GDN_ERR_INVALID_ARG, "dw is NULL");
    if (T > 0) {
        if ((st = check_rows(dy, lddy, channels, "dy")) != GDN_OK) return st;
        if ((st = check_rows(x, ldx, channels, "x")) != GDN_OK) return st;
        if ((st = check_rows(dx, lddx, channels, "dx")) != GDN_OK) return st;
    }
    const size_t need = gdn_ssm_conv_bwd_workspace_size(T, channels, conv_k);
    if (!workspace || workspace_bytes < need)
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes < required %zu", workspace ? workspace_bytes : 0, need);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(GDN_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (T > 0 && (dx == x || dx == dy)) return fail(GDN_ERR_INVALID_ARG, "dx must not be x or dy");
    ConvBwdParams p{dy, lddy, x, ldx, w, bias, T, channels, cu_seqlens, num_seqs, state, dstate_out, dx, lddx, dstate,
                    static_cast<float*>(workspace), 0};
    cudaStream_t s = (cudaStream_t)stream;
    st = dtype == GDN_BF16 ? run_bwd<__nv_bfloat16>(p, conv_k, s) : run_bwd<float>(p, conv_k, s);
    if (st != GDN_OK) return st;
    const int64_t nw = (int64_t)channels * conv_k, all = nw + channels;
    return launch_column_sum(p.part, bwd_strips(T, channels), all, nw, all, dw, dbias, nullptr, s);
}

gdn_status gdn_ssm_conv_step(const void* x, int64_t ldx, gdn_dtype dtype, int32_t batch, int32_t channels,
                             const void* w, const void* bias, int32_t conv_k, void* states, int32_t num_slots,
                             const int32_t* src, const int32_t* dst, void* y, int64_t ldy, void* stream) {
    gdn_status st = check_conv(dtype, batch, channels, w, conv_k);
    if (st != GDN_OK) return st;
    if (batch > 65535) return fail(GDN_ERR_UNSUPPORTED_SHAPE, "batch=%d above 65535", batch);
    if (num_slots < 0) return fail(GDN_ERR_INVALID_ARG, "num_slots=%d", num_slots);
    if ((!src || !dst) && num_slots < batch)
        return fail(GDN_ERR_INVALID_ARG, "num_slots=%d < batch=%d without slot numbers", num_slots, batch);
    if (batch == 0) return GDN_OK;
    if ((st = check_rows(x, ldx, channels, "x")) != GDN_OK) return st;
    if ((st = check_rows(y, ldy, channels, "y")) != GDN_OK) return st;
    if (conv_k > 1 && (!states || !al16(states)))
        return fail(GDN_ERR_INVALID_ARG, "states must be 16-byte aligned and not NULL");
    cudaStream_t s = (cudaStream_t)stream;
    return dtype == GDN_BF16
               ? run_step<__nv_bfloat16>(x, ldx, batch, channels, w, bias, conv_k, states, num_slots, src, dst, y, ldy, s)
               : run_step<float>(x, ldx, batch, channels, w, bias, conv_k, states, num_slots, src, dst, y, ldy, s);
}

}  // extern "C"
