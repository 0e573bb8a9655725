// Block norm: post norm, gate, residual scale, residual add and pre norm in
// one pass over the rows, and its gradient.
//
//   p = w_post o / rms(o),  b = scale sigmoid(gate) p,  r' = r + b,
//   y = w_pre r' / rms(r')
// Backward at the stored r', with r^ = r' / rms(r'), o^ = o / rms(o):
//   dr   = dr' + (w_pre dy - r^ mean(w_pre dy r^)) / rms(r')   (= the residual's gradient)
//   dp   = dr scale sigmoid(gate),  dgate = dr scale p sg (1 - sg),  dscale = sum dr sg p
//   do   = (w_post dp - o^ mean(w_post dp o^)) / rms(o)
//   dw_pre = sum dy r^,  dw_post = sum dp o^
// The mean in do needs dr, which needs the mean of the pre norm: its sum is taken
// apart into three that do not, so that a row has one reduction:
//   sum_i q_i dr_i = sum q dr' + (sum q w_pre dy - mean(w_pre dy r^) sum q r^) / rms(r'),
//   q = w_post scale sg o^.
//
// HBM-bound: each array is read or written once.  A block works on one row at a
// time, in vectors of eight columns.  The forward's threads read all that they need
// of a row, one to four vectors, before the first reduction, and keep it in
// registers; several blocks share an SM and cover each other's reductions (32768
// rows of 4096 with a gate: 237 us in bf16, 5.7 TB/s; 301 with an fp32 residual
// stream, 6.2 TB/s).  A ring of rows in shared memory gained nothing there: two
// blocks an SM wait for their reductions (330 and 460 us).
// The blocks of the backward are persistent, so that its column sums stay in
// registers over all of a block's rows and leave as one partial row per block,
// summed in block order by a second kernel; its rows come by asynchronous copies
// into a ring in shared memory that every thread fills and reads alone, once before
// and once behind the reduction (32768 rows of 4096 in bf16: 374 us, 5.7 TB/s; 512
// threads of 128 registers fill an SM, so that little covers a reduction).  Up to two
// vectors a thread the weights stay in registers: read twice a row they cost half as
// much again (8192 rows of 5120: 280 us, 164 kept).
// Rows of which a block's share of shared memory holds fewer than two are read where
// they are used: fp32 of 264 to 4096 columns and above 5120, bf16 above 10240, bf16
// with an fp32 stream above 7168.
#include "chunk_common.cuh"
#include "ssm_common.cuh"

#include <type_traits>

namespace gdn {

gdn_status set_smem_attr(const void* func, size_t bytes);

namespace {

struct NormParams {
    const void* o; int64_t ldo;
    const void* gate; int64_t ldg;
    const void* res;  // fwd: the residual stream; bwd: the stored res_out
    const void* w_post; const void* w_pre; const float* scale;
    float eps;
    int T, W;
    void* res_out; void* y;                                 // fwd
    const void* dy; const void* dres_out;                   // bwd
    void* d_o; void* dgate; void* dres; float* part;
};

// A sum over the block, in one order for all threads: lane w of every warp takes
// warp w's sum, then the lanes are added.  Callers alternate the scratch [32], so
// that one barrier a call is enough.
__device__ __forceinline__ float block_sum(float v, float* scratch) {
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    const int nw = blockDim.x >> 5, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (nw == 1) return v;
    if (lane == 0) scratch[w] = v;
    __syncthreads();
    v = lane < nw ? scratch[lane] : 0.f;
#pragma unroll
    for (int off = 8; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return __shfl_sync(0xffffffffu, v, 0);
}

// Eight sums over the block's at most 16 warps, likewise.  Halving exchanges leave
// each lane with the value of its three low bits (seven exchanges instead of the
// forty that whole sums of eight values would take); scratch [16][8].
__device__ __forceinline__ void block_sum8(float (&v)[8], float* scratch) {
    const int nw = blockDim.x >> 5, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 1, cnt = 4; m < 8; m <<= 1, cnt >>= 1) {
        const bool up = lane & m;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < cnt) {
                const float snd = up ? v[2 * i] : v[2 * i + 1], kp = up ? v[2 * i + 1] : v[2 * i];
                v[i] = kp + __shfl_xor_sync(0xffffffffu, snd, m);
            }
    }
    float t = v[0];
    t += __shfl_xor_sync(0xffffffffu, t, 8);
    t += __shfl_xor_sync(0xffffffffu, t, 16);
    if (nw > 1) {
        if (lane < 8) scratch[w * 8 + lane] = t;
        __syncthreads();
        t = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int u = 4 * i + (lane >> 3);
            if (u < nw) t += scratch[u * 8 + (lane & 7)];
        }
        t += __shfl_xor_sync(0xffffffffu, t, 8);
        t += __shfl_xor_sync(0xffffffffu, t, 16);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __shfl_sync(0xffffffffu, t, i);
}

constexpr int kMaxThreads = 512;

// Eight elements as they lie in memory.
template <typename X>
struct Raw8 {
    uint4 v[8 * sizeof(X) / 16];
    __device__ __forceinline__ void load(const X* p) {
#pragma unroll
        for (int i = 0; i < (int)(8 * sizeof(X) / 16); ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void get(F2 (&f)[4]) const { f2_load8(reinterpret_cast<const X*>(v), f); }
};

template <typename E, typename R, int VPT>
__global__ void __launch_bounds__(kMaxThreads, VPT == 1 || (sizeof(E) == 4 && VPT == 2) ? 2 : 1)
    norm_fwd_kernel(const NormParams p) {
    __shared__ float red[2][32];
    const int nv = p.W >> 3, nt = blockDim.x, tid = threadIdx.x;
    const float inv = 1.f / (float)p.W;
    const E* wpost = static_cast<const E*>(p.w_post);
    const E* wpre = static_cast<const E*>(p.w_pre);
    constexpr bool EARLY = sizeof(E) == 2;  // the gate's row with the others; fp32 needs the registers
    int par = 0;
    for (int row = blockIdx.x; row < p.T; row += gridDim.x) {
        const E* o = static_cast<const E*>(p.o) + (int64_t)row * p.ldo;
        const E* g = p.gate ? static_cast<const E*>(p.gate) + (int64_t)row * p.ldg : nullptr;
        const R* res = static_cast<const R*>(p.res) + (int64_t)row * p.W;
        R* ro = static_cast<R*>(p.res_out) + (int64_t)row * p.W;
        E* y = static_cast<E*>(p.y) + (int64_t)row * p.W;
        Raw8<E> oraw[VPT], graw[VPT];
        Raw8<R> rraw[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * nt;
            if (v < nv) {
                oraw[j].load(o + 8 * v);
                rraw[j].load(res + 8 * v);
                if (EARLY && g) graw[j].load(g + 8 * v);
            }
        }
        F2 R1 = f2_dup(1.f);
        if (wpost) {
            F2 ss = f2_dup(0.f);
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (tid + j * nt < nv) {
                    F2 t[4];
                    oraw[j].get(t);
#pragma unroll
                    for (int i = 0; i < 4; ++i) ss = f2_fma(t[i], t[i], ss);
                }
            R1 = f2_dup(1.f / sqrtf(block_sum(f2_sum(ss), red[par]) * inv + p.eps));
            par ^= 1;
        }
        F2 r[VPT][4], sr = f2_dup(0.f);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * nt;
            if (v < nv) {
                F2 b[4], t[4];
                oraw[j].get(b);
                if (wpost) {
                    f2_load8(wpost + 8 * v, t);
#pragma unroll
                    for (int i = 0; i < 4; ++i) b[i] = f2_mul(b[i], f2_mul(R1, t[i]));
                }
                if (g) {
                    if (!EARLY) graw[j].load(g + 8 * v);
                    graw[j].get(t);
#pragma unroll
                    for (int i = 0; i < 4; ++i) b[i] = f2_mul(b[i], f2_sigmoid(t[i]));
                }
                rraw[j].get(r[j]);
                if (p.scale) {
                    f2_load8(p.scale + 8 * v, t);
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[j][i] = f2_fma(b[i], t[i], r[j][i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[j][i] = f2_add(r[j][i], b[i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) sr = f2_fma(r[j][i], r[j][i], sr);
                f2_store8(ro + 8 * v, r[j]);
            }
        }
        const F2 R2 = f2_dup(1.f / sqrtf(block_sum(f2_sum(sr), red[par]) * inv + p.eps));
        par ^= 1;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * nt;
            if (v < nv) {
                F2 w[4];
                f2_load8(wpre + 8 * v, w);
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = f2_mul(f2_mul(r[j][i], R2), w[i]);
                f2_store8(y + 8 * v, w);
            }
        }
    }
}

// What the backward reads of a row: res_out, dres_out (R), dy, o, gate (E).
template <typename E, typename R, int VPT>
constexpr size_t row_bytes(int threads) {
    return (size_t)threads * VPT * (2 * 8 * sizeof(R) + 3 * 8 * sizeof(E));
}
constexpr size_t kRingBytes = 200 << 10;  // of an SM's shared memory, for the rings of its blocks
constexpr int kMaxStages = 4;

// RING: rows come through the ring of `stages` rows; else (rows too wide for two
// of them) they are read where they are used.
template <typename E, typename R, int VPT, bool RING>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_kernel(const NormParams p, int stages) {
    extern __shared__ uint4 ring[];
    __shared__ float red[2][16 * 8];
    constexpr int VE = 8 * sizeof(E) / 16, VRS = 8 * sizeof(R) / 16;  // 16-byte pieces of eight elements
    const int nv = p.W >> 3, nt = blockDim.x, tid = threadIdx.x;
    const float inv = 1.f / (float)p.W;
    const E* wpost = static_cast<const E*>(p.w_post);
    const E* wpre = static_cast<const E*>(p.w_pre);
    const R* res = static_cast<const R*>(p.res);
    const R* dro = static_cast<const R*>(p.dres_out);
    const E* dy = static_cast<const E*>(p.dy);
    const E* o = static_cast<const E*>(p.o);
    const E* gate = static_cast<const E*>(p.gate);
    constexpr int PIECES = VPT * (2 * VRS + 3 * VE);
    auto piece = [&](int st, int q) { return ring + ((size_t)st * PIECES + q) * nt + tid; };
    auto copy8 = [&](int st, int q, const void* src, int pieces) {
        for (int i = 0; i < pieces; ++i) cp_async16(piece(st, q + i), static_cast<const uint4*>(src) + i, 16);
    };
    auto fetch = [&](int64_t row, int st) {
        if (row < p.T)
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = tid + j * nt, q = j * (2 * VRS + 3 * VE);
                if (v < nv) {
                    copy8(st, q, res + row * p.W + 8 * v, VRS);
                    if (dro) copy8(st, q + VRS, dro + row * p.W + 8 * v, VRS);
                    copy8(st, q + 2 * VRS, dy + row * p.W + 8 * v, VE);
                    copy8(st, q + 2 * VRS + VE, o + row * p.ldo + 8 * v, VE);
                    if (gate) copy8(st, q + 2 * VRS + 2 * VE, gate + row * p.ldg + 8 * v, VE);
                }
            }
        cp_async_commit();
    };
    auto take = [&](auto* src, int st, int q, F2 (&f)[4]) {
        using X = typename std::remove_const<typename std::remove_pointer<decltype(src)>::type>::type;
        if constexpr (RING) {
            uint4 raw[8 * sizeof(X) / 16];
#pragma unroll
            for (int i = 0; i < (int)(8 * sizeof(X) / 16); ++i) raw[i] = *piece(st, q + i);
            f2_load8(reinterpret_cast<const X*>(raw), f);
        } else {
            f2_load8(src, f);
        }
    };
    // w_pre and f = w_post scale of vector v (1 where missing)
    auto weights = [&](int v, F2 (&w)[4], F2 (&f)[4]) {
        f2_load8(wpre + 8 * v, w);
        if (wpost) f2_load8(wpost + 8 * v, f);
        if (p.scale) {
            F2 t[4];
            f2_load8(p.scale + 8 * v, t);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = wpost ? f2_mul(f[i], t[i]) : t[i];
        } else if (!wpost) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = f2_dup(1.f);
        }
    };
    constexpr bool KEEP = VPT == 1;   // a row's vector stays in registers; else it is read twice
    constexpr bool KEEPW = VPT <= 2;  // so do the weights
    F2 kw[KEEPW ? VPT : 1][4], kf[KEEPW ? VPT : 1][4], kr[5][4];
    if (KEEPW)
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (tid + j * nt < nv) weights(tid + j * nt, kw[j], kf[j]);
    // sums over the rows: dy r^, and dr sg o^, of which dw_post and dscale are multiples by column
    F2 a_pre[VPT][4], a_br[VPT][4];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) a_pre[j][i] = a_br[j][i] = f2_dup(0.f);
    int st = 0, par = 0;
    if (RING)
        for (int i = 0; i < stages - 1; ++i) fetch((int64_t)blockIdx.x + (int64_t)i * gridDim.x, i);
    for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x, par ^= 1) {
        const int64_t base = row * p.W;
        if (RING) {
            fetch(row + (int64_t)(stages - 1) * gridDim.x, st == 0 ? stages - 1 : st - 1);
            if (stages == 4) cp_async_wait<3>();
            else if (stages == 3) cp_async_wait<2>();
            else cp_async_wait<1>();
        }
        // x: res_out, dres_out, dy, o, sigmoid(gate)
        auto row_vec = [&](int j, F2 (&x)[5][4]) {
            const int q = j * (2 * VRS + 3 * VE), v = tid + j * nt;
            take(res + base + 8 * v, st, q, x[0]);
            if (dro) take(dro + base + 8 * v, st, q + VRS, x[1]);
            else
#pragma unroll
                for (int i = 0; i < 4; ++i) x[1][i] = f2_dup(0.f);
            take(dy + base + 8 * v, st, q + 2 * VRS, x[2]);
            take(o + row * p.ldo + 8 * v, st, q + 2 * VRS + VE, x[3]);
            if (gate) {
                take(gate + row * p.ldg + 8 * v, st, q + 2 * VRS + 2 * VE, x[4]);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[4][i] = f2_sigmoid(x[4][i]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) x[4][i] = f2_dup(1.f);
            }
        };
        // sums: r'^2, w_pre dy r', o^2, and of q = f sg o: q dr', q w_pre dy, q r' (the last four used with
        // w_post; without it r1 is 1 and m1 is 0, without a gate sg is 1: choices cost more here than products)
        F2 s6[6];
#pragma unroll
        for (int i = 0; i < 6; ++i) s6[i] = f2_dup(0.f);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (tid + j * nt < nv) {
                F2 x[5][4], w[4], f[4];
                row_vec(j, x);
                if constexpr (!KEEPW) weights(tid + j * nt, w, f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const F2 wd = f2_mul(KEEPW ? kw[KEEPW ? j : 0][i] : w[i], x[2][i]);
                    s6[0] = f2_fma(x[0][i], x[0][i], s6[0]);
                    s6[1] = f2_fma(wd, x[0][i], s6[1]);
                    const F2 qv = f2_mul(f2_mul(KEEPW ? kf[KEEPW ? j : 0][i] : f[i], x[3][i]), x[4][i]);
                    s6[2] = f2_fma(x[3][i], x[3][i], s6[2]);
                    s6[3] = f2_fma(qv, x[1][i], s6[3]);
                    s6[4] = f2_fma(qv, wd, s6[4]);
                    s6[5] = f2_fma(qv, x[0][i], s6[5]);
                }
                if constexpr (KEEP)
#pragma unroll
                    for (int a = 0; a < 5; ++a)
#pragma unroll
                        for (int i = 0; i < 4; ++i) kr[a][i] = x[a][i];
            }
        }
        float s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = i < 6 ? f2_sum(s6[i]) : 0.f;
        block_sum8(s, red[par]);
        const float r2 = 1.f / sqrtf(s[0] * inv + p.eps);
        const float r1 = wpost ? 1.f / sqrtf(s[2] * inv + p.eps) : 1.f;
        const float m2 = s[1] * r2 * inv;                                            // mean(w_pre dy r^)
        const float m1 = wpost ? r1 * inv * (s[3] + r2 * (s[4] - m2 * r2 * s[5])) : 0.f;  // mean(w_post dp o^)
        const F2 R2 = f2_dup(r2), R1 = f2_dup(r1), M2 = f2_dup(-m2), M1 = f2_dup(-m1), one = f2_dup(1.f), neg = f2_dup(-1.f);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * nt;
            if (v < nv) {
                F2 x[5][4], w[4], f[4], t[4], dp[4], dr[4];
                if constexpr (KEEP) {
#pragma unroll
                    for (int a = 0; a < 5; ++a)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[a][i] = kr[a][i];
                } else {
                    row_vec(j, x);
                    if constexpr (!KEEPW) weights(v, w, f);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const F2 rh = f2_mul(x[0][i], R2), wi = KEEPW ? kw[KEEPW ? j : 0][i] : w[i], fi = KEEPW ? kf[KEEPW ? j : 0][i] : f[i];
                    a_pre[j][i] = f2_fma(x[2][i], rh, a_pre[j][i]);
                    dr[i] = f2_fma(R2, f2_fma(wi, x[2][i], f2_mul(rh, M2)), x[1][i]);
                    const F2 oh = f2_mul(x[3][i], R1), dg = f2_mul(dr[i], x[4][i]);
                    a_br[j][i] = f2_fma(dg, oh, a_br[j][i]);
                    const F2 df = f2_mul(dg, fi);
                    t[i] = f2_mul(f2_mul(df, oh), f2_fma(x[4][i], neg, one));
                    dp[i] = f2_mul(R1, f2_fma(oh, M1, df));
                }
                f2_store8(static_cast<R*>(p.dres) + base + 8 * v, dr);
                if (gate) f2_store8(static_cast<E*>(p.dgate) + base + 8 * v, t);
                f2_store8(static_cast<E*>(p.d_o) + base + 8 * v, dp);
            }
        }
        st = st == stages - 1 ? 0 : st + 1;
    }
    if (RING) cp_async_wait<0>();
    float* part = p.part + (int64_t)blockIdx.x * 3 * p.W;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = tid + j * nt;
        if (v < nv) {
            f2_store8(part + 8 * v, a_pre[j]);
            F2 c[4], d[4];
            if (p.scale) {
                f2_load8(p.scale + 8 * v, c);
                if (wpost) f2_load8(wpost + 8 * v, d);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[i] = p.scale ? f2_mul(a_br[j][i], c[i]) : a_br[j][i];                // dw_post
                d[i] = p.scale && wpost ? f2_mul(a_br[j][i], d[i]) : a_br[j][i];       // dscale
            }
            f2_store8(part + p.W + 8 * v, c);
            f2_store8(part + 2 * (int64_t)p.W + 8 * v, d);
        }
    }
}

}  // namespace

// out[c] = sum over rows b of part[b * stride + c], in row order within each of
// eight interleaved chains (a fixed order); null outputs are skipped.
__global__ void __launch_bounds__(256) column_sum_kernel(const float* part, int rows, int64_t stride, int64_t n0, int64_t n1,
                                                         float* out0, float* out1, float* out2) {
    __shared__ float sm[8][33];
    const int64_t c = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    const int lane_row = threadIdx.x >> 5;
    float s = 0.f;
    if (c < stride)
        for (int b = lane_row; b < rows; b += 8) s += part[(int64_t)b * stride + c];
    sm[lane_row][threadIdx.x & 31] = s;
    __syncthreads();
    if (lane_row == 0 && c < stride) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t += sm[k][threadIdx.x];
        float* out = c < n0 ? out0 : (c < n1 ? out1 : out2);
        const int64_t i = c < n0 ? c : (c < n1 ? c - n0 : c - n1);
        if (out) out[i] = t;
    }
}

gdn_status launch_column_sum(const float* part, int rows, int64_t stride, int64_t n0, int64_t n1, float* out0, float* out1,
                             float* out2, cudaStream_t s) {
    column_sum_kernel<<<(unsigned)((stride + 31) / 32), 256, 0, s>>>(part, rows, stride, n0, n1, out0, out1, out2);
    return check_launch("column_sum_kernel");
}

namespace {

// threads of a row's block and vectors per thread
void norm_shape(int W, int& threads, int& vpt) {
    const int nv = W / 8;
    vpt = nv <= kMaxThreads ? 1 : (nv <= 2 * kMaxThreads ? 2 : 4);
    threads = ((nv + vpt - 1) / vpt + 31) / 32 * 32;
}

// Of the backward: two vectors where the types are the same, and bf16 rows wider
// than 2048 (bf16, 16384 rows of 2560: 129 us, 161 with one; 32768 of 4096: 374 and
// 381; 32768 of 1024: 103 and 96; fp32, 8192 of 4096: 212 and 280), one where the
// stream is fp32 beside bf16 (32768 of 4096: 633 us, 693 with two).
void bwd_shape(int W, bool mixed, bool f32, int& threads, int& vpt) {
    norm_shape(W, threads, vpt);
    const int nv = W / 8;
    if (vpt == 1 && !mixed && nv > (f32 ? 32 : 256)) {
        vpt = 2;
        threads = ((nv + 1) / 2 + 31) / 32 * 32;
    }
}
// 128 registers a thread: 512 threads fill an SM
constexpr int bwd_per_sm(int threads) { return threads >= 512 ? 1 : 512 / threads; }
int bwd_blocks(int T, int threads) {
    const int n = device_sm_count() * bwd_per_sm(threads);
    return T < n ? (T > 0 ? T : 1) : (int)blocks_for_sum(T, n);
}

// Rows that a block's ring holds; below two there is none.
template <typename E, typename R, int VPT>
constexpr int ring_stages(int threads) {
    const int n = (int)(kRingBytes / bwd_per_sm(threads) / row_bytes<E, R, VPT>(threads));
    return n < kMaxStages ? n : kMaxStages;
}
// whether blocks of some size have a ring (or none)
template <typename E, typename R, int VPT>
constexpr bool some_block(bool ring) {
    for (int threads = 32; threads <= kMaxThreads; threads += 32)
        if ((ring_stages<E, R, VPT>(threads) >= 2) == ring) return true;
    return false;
}

template <typename E, typename R, int VPT>
gdn_status run_bwd(const NormParams& p, int threads, cudaStream_t s) {
    const int grid = bwd_blocks(p.T, threads), stages = ring_stages<E, R, VPT>(threads);
    if constexpr (some_block<E, R, VPT>(false)) {
        if (stages < 2) {
            norm_bwd_kernel<E, R, VPT, false><<<grid, threads, 0, s>>>(p, 1);
            return check_launch("norm_bwd_kernel");
        }
    }
    if constexpr (some_block<E, R, VPT>(true)) {
        const gdn_status st = set_smem_attr((const void*)norm_bwd_kernel<E, R, VPT, true>, kRingBytes);
        if (st != GDN_OK) return st;
        norm_bwd_kernel<E, R, VPT, true><<<grid, threads, stages * row_bytes<E, R, VPT>(threads), s>>>(p, stages);
    }
    return check_launch("norm_bwd_kernel");
}

template <typename E, typename R>
gdn_status run_norm(const NormParams& p, bool bwd, cudaStream_t s) {
    int threads, vpt;
    norm_shape(p.W, threads, vpt);
    if (!bwd) {
        // Wide threads when there are more rows than two waves of blocks: the
        // reductions, roots and addresses are per thread and row (32768 rows of 4096
        // bf16: 237 us with four vectors, 333 with two, 303 with one; fp32 rows, 8192 of
        // 2560: 78 with two, 85 with one, 106 with four).  Few rows are a matter of
        // latency: one vector (64 rows: 3.5 us).
        const int sms = device_sm_count(), nv = p.W / 8, most = sizeof(E) == 4 ? 2 : 4;
        if (p.T > 2 * sms) {
            while (vpt < most && nv > 32 * vpt) vpt *= 2;
            threads = ((nv + vpt - 1) / vpt + 31) / 32 * 32;
        }
        const int per = 2048 / threads;
        const int64_t cap = (int64_t)sms * (per > 32 ? 32 : per);
        const int grid = (int)(p.T < cap ? p.T : cap);
        if (vpt == 1) norm_fwd_kernel<E, R, 1><<<grid, threads, 0, s>>>(p);
        else if (vpt == 2) norm_fwd_kernel<E, R, 2><<<grid, threads, 0, s>>>(p);
        else norm_fwd_kernel<E, R, 4><<<grid, threads, 0, s>>>(p);
        return check_launch("norm_fwd_kernel");
    }
    bwd_shape(p.W, sizeof(E) != sizeof(R), sizeof(E) == 4, threads, vpt);
    if (vpt == 1) return run_bwd<E, R, 1>(p, threads, s);
    if (vpt == 2) return run_bwd<E, R, 2>(p, threads, s);
    return run_bwd<E, R, 4>(p, threads, s);
}

gdn_status dispatch_norm(const NormParams& p, bool bwd, gdn_dtype dt, gdn_dtype rdt, cudaStream_t s) {
    if (dt == GDN_F32) return run_norm<float, float>(p, bwd, s);
    if (rdt == GDN_F32) return run_norm<__nv_bfloat16, float>(p, bwd, s);
    return run_norm<__nv_bfloat16, __nv_bfloat16>(p, bwd, s);
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

gdn_status check_norm(gdn_dtype dt, gdn_dtype rdt, int T, int W, const void* o, int64_t ldo, const void* gate,
                      int64_t ldg, const void* w_post, const void* w_pre, const float* scale, float eps) {
    if (dt != GDN_F32 && dt != GDN_BF16) return fail(GDN_ERR_DTYPE, "unknown dtype %d", (int)dt);
    if (rdt != GDN_F32 && rdt != dt) return fail(GDN_ERR_DTYPE, "res_dtype %d must be fp32 or the dtype", (int)rdt);
    if (T < 0 || W < 1) return fail(GDN_ERR_INVALID_ARG, "T=%d width=%d", T, W);
    if (T > kMaxTokens) return fail(GDN_ERR_UNSUPPORTED_SHAPE, "%d tokens, more than %d", T, kMaxTokens);
    if (W % 8 != 0 || W > 16384)
        return fail(GDN_ERR_UNSUPPORTED_SHAPE, "width=%d must be a multiple of 8 up to 16384", W);
    if (!(eps >= 0.f)) return fail(GDN_ERR_INVALID_ARG, "eps must not be negative");
    if (!w_pre) return fail(GDN_ERR_INVALID_ARG, "w_pre is NULL");
    if (!al16(w_post) || !al16(w_pre) || !al16(scale))
        return fail(GDN_ERR_INVALID_ARG, "w_post, w_pre and scale must be 16-byte aligned");
    if (T == 0) return GDN_OK;
    if (!o || !al16(o) || ldo < W || ldo % 8 != 0)
        return fail(GDN_ERR_INVALID_ARG, "o must be 16-byte aligned with a row stride >= width that is a multiple of 8");
    if (gate && (!al16(gate) || ldg < W || ldg % 8 != 0))
        return fail(GDN_ERR_INVALID_ARG,
                    "gate must be 16-byte aligned with a row stride >= width that is a multiple of 8");
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_block_norm_fwd(const void* o, int64_t ldo, const void* gate, int64_t ldgate, gdn_dtype dtype,
                              const void* res, gdn_dtype res_dtype, const void* w_post, const void* w_pre,
                              const float* scale, float eps, int32_t T, int32_t width, void* res_out, void* y,
                              void* stream) {
    gdn_status st = check_norm(dtype, res_dtype, T, width, o, ldo, gate, ldgate, w_post, w_pre, scale, eps);
    if (st != GDN_OK) return st;
    if (T == 0) return GDN_OK;
    if (!res || !res_out || !y || !al16(res) || !al16(res_out) || !al16(y))
        return fail(GDN_ERR_INVALID_ARG, "res, res_out and y must be 16-byte aligned and not NULL");
    NormParams p{};
    p.o = o; p.ldo = ldo; p.gate = gate; p.ldg = ldgate; p.res = res; p.w_post = w_post; p.w_pre = w_pre;
    p.scale = scale; p.eps = eps; p.T = T; p.W = width; p.res_out = res_out; p.y = y;
    return dispatch_norm(p, false, dtype, res_dtype, (cudaStream_t)stream);
}

size_t gdn_block_norm_bwd_workspace_size(int32_t T, int32_t width) {
    if (T < 0 || T > kMaxTokens || width < 1 || width % 8 != 0 || width > 16384) return 0;
    int blocks = 0;
    for (int i = 0; i < 3; ++i) {  // whatever the types
        int threads, vpt;
        bwd_shape(width, i == 2, i == 1, threads, vpt);
        blocks = max(blocks, bwd_blocks(T, threads));
    }
    return (sizeof(float) * 3 * (size_t)width * blocks + 255) & ~size_t(255);
}

gdn_status gdn_block_norm_bwd(const void* dy, const void* dres_out, const void* o, int64_t ldo, const void* gate,
                              int64_t ldgate, gdn_dtype dtype, const void* res_out, gdn_dtype res_dtype,
                              const void* w_post, const void* w_pre, const float* scale, float eps, int32_t T,
                              int32_t width, void* d_o, void* dgate, void* dres, float* dw_pre, float* dw_post,
                              float* dscale, void* workspace, size_t workspace_bytes, void* stream) {
    gdn_status st = check_norm(dtype, res_dtype, T, width, o, ldo, gate, ldgate, w_post, w_pre, scale, eps);
    if (st != GDN_OK) return st;
    if (!dw_pre || (w_post && !dw_post) || (scale && !dscale))
        return fail(GDN_ERR_INVALID_ARG, "dw_pre, dw_post or dscale is NULL");
    const size_t need = gdn_block_norm_bwd_workspace_size(T, width);
    if (!workspace || workspace_bytes < need)
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes < required %zu", workspace ? workspace_bytes : 0, need);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(GDN_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (T > 0) {
        if (!dy || !res_out || !d_o || !dres || (gate && !dgate))
            return fail(GDN_ERR_INVALID_ARG, "dy, res_out, d_o, dres or dgate is NULL");
        if (!al16(dy) || !al16(dres_out) || !al16(res_out) || !al16(d_o) || !al16(dgate) || !al16(dres))
            return fail(GDN_ERR_INVALID_ARG, "dy, dres_out, res_out, d_o, dgate and dres must be 16-byte aligned");
    }
    NormParams p{};
    p.o = o; p.ldo = ldo; p.gate = gate; p.ldg = ldgate; p.res = res_out; p.w_post = w_post; p.w_pre = w_pre;
    p.scale = scale; p.eps = eps; p.T = T; p.W = width; p.dy = dy; p.dres_out = dres_out; p.d_o = d_o;
    p.dgate = dgate; p.dres = dres; p.part = static_cast<float*>(workspace);
    cudaStream_t s = (cudaStream_t)stream;
    if ((st = dispatch_norm(p, true, dtype, res_dtype, s)) != GDN_OK) return st;  // T == 0: zero partial sums
    int threads, vpt;
    bwd_shape(width, res_dtype != dtype, dtype == GDN_F32, threads, vpt);
    return launch_column_sum(p.part, bwd_blocks(T, threads), 3 * (int64_t)width, width, 2 * width, dw_pre,
                             w_post ? dw_post : nullptr, scale ? dscale : nullptr, s);
}

}  // extern "C"
