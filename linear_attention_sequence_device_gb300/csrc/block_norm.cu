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
// HBM-bound: each array is read or written once.  A block works on one row at a
// time, eight columns per thread and vector, and keeps the row in registers
// between the two reductions; the blocks are persistent, so that the backward's
// column sums stay in registers over all of a block's rows and leave as one
// partial row per block, summed in block order by a second kernel.
#include "ssm_common.cuh"

namespace gdn {
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

// Sums over the block; the scratch alternates so that one barrier a call is enough.
template <int NV>
__device__ __forceinline__ void block_sum(float (&v)[NV], float* scratch) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int off = 16; off; off >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    const int nw = blockDim.x >> 5, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < NV; ++i) scratch[w * NV + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float s = 0.f;
        for (int k = 0; k < nw; ++k) s += scratch[k * NV + i];
        v[i] = s;
    }
}

constexpr int kMaxThreads = 512;

template <typename E, typename R, int VPT>
__global__ void __launch_bounds__(kMaxThreads) norm_fwd_kernel(const NormParams p) {
    __shared__ float red[2][kMaxThreads / 32];
    const int nv = p.W >> 3;
    const float inv = 1.f / (float)p.W;
    const E* wpost = static_cast<const E*>(p.w_post);
    const E* wpre = static_cast<const E*>(p.w_pre);
    for (int row = blockIdx.x; row < p.T; row += gridDim.x) {
        const E* o = static_cast<const E*>(p.o) + (int64_t)row * p.ldo;
        const E* g = p.gate ? static_cast<const E*>(p.gate) + (int64_t)row * p.ldg : nullptr;
        const R* r = static_cast<const R*>(p.res) + (int64_t)row * p.W;
        float b[VPT][8], rv[VPT][8];
        float ss[1] = {0.f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = threadIdx.x + j * blockDim.x;
            if (v < nv) {
                load8(o + 8 * v, b[j]);
                load8_rw(r + 8 * v, rv[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) ss[0] = fmaf(b[j][i], b[j][i], ss[0]);
            }
        }
        float r1 = 1.f;
        if (wpost) {
            block_sum<1>(ss, red[0]);
            r1 = 1.f / sqrtf(ss[0] * inv + p.eps);
        }
        float sr[1] = {0.f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = threadIdx.x + j * blockDim.x;
            if (v < nv) {
                float t[8];
                if (wpost) {
                    load8(wpost + 8 * v, t);
#pragma unroll
                    for (int i = 0; i < 8; ++i) b[j][i] *= r1 * t[i];
                }
                if (g) {
                    load8(g + 8 * v, t);
#pragma unroll
                    for (int i = 0; i < 8; ++i) b[j][i] *= sigmoid_fast(t[i]);
                }
                if (p.scale) {
                    load8(p.scale + 8 * v, t);
#pragma unroll
                    for (int i = 0; i < 8; ++i) b[j][i] *= t[i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    rv[j][i] += b[j][i];
                    sr[0] = fmaf(rv[j][i], rv[j][i], sr[0]);
                }
                store8(static_cast<R*>(p.res_out) + (int64_t)row * p.W + 8 * v, rv[j]);
            }
        }
        block_sum<1>(sr, red[1]);
        const float r2 = 1.f / sqrtf(sr[0] * inv + p.eps);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = threadIdx.x + j * blockDim.x;
            if (v < nv) {
                float t[8];
                load8(wpre + 8 * v, t);
#pragma unroll
                for (int i = 0; i < 8; ++i) t[i] *= rv[j][i] * r2;
                store8(static_cast<E*>(p.y) + (int64_t)row * p.W + 8 * v, t);
            }
        }
        if (!wpost) __syncthreads();  // red[1] is read before the next row writes it
    }
}

template <typename E, typename R, int VPT>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_kernel(const NormParams p) {
    __shared__ float red[2][3 * kMaxThreads / 32];
    const int nv = p.W >> 3;
    const float inv = 1.f / (float)p.W;
    const E* wpost = static_cast<const E*>(p.w_post);
    const E* wpre = static_cast<const E*>(p.w_pre);
    float a_pre[VPT][8], a_post[VPT][8], a_sc[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) a_pre[j][i] = a_post[j][i] = a_sc[j][i] = 0.f;
    for (int row = blockIdx.x; row < p.T; row += gridDim.x) {
        const int64_t base = (int64_t)row * p.W;
        const E* o = static_cast<const E*>(p.o) + (int64_t)row * p.ldo;
        const E* g = p.gate ? static_cast<const E*>(p.gate) + (int64_t)row * p.ldg : nullptr;
        float ov[VPT][8], rv[VPT][8], gy[VPT][8];
        float s3[3] = {0.f, 0.f, 0.f};  // sum r'^2, sum w_pre dy r', sum o^2
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = threadIdx.x + j * blockDim.x;
            if (v < nv) {
                float w[8];
                load8(static_cast<const R*>(p.res) + base + 8 * v, rv[j]);
                load8(static_cast<const E*>(p.dy) + base + 8 * v, gy[j]);
                load8(o + 8 * v, ov[j]);
                load8(wpre + 8 * v, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s3[0] = fmaf(rv[j][i], rv[j][i], s3[0]);
                    s3[1] = fmaf(w[i] * gy[j][i], rv[j][i], s3[1]);
                    s3[2] = fmaf(ov[j][i], ov[j][i], s3[2]);
                }
            }
        }
        block_sum<3>(s3, red[0]);
        const float r2 = 1.f / sqrtf(s3[0] * inv + p.eps);
        const float r1 = 1.f / sqrtf(s3[2] * inv + p.eps);
        const float m2 = s3[1] * r2 * inv;  // mean(w_pre dy r^)
        float s1[1] = {0.f};
        float dp[VPT][8];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = threadIdx.x + j * blockDim.x;
            if (v < nv) {
                float w[8], dr[8], sg[8], pv[8], t[8];
                load8(wpre + 8 * v, w);
                if (p.dres_out) load8_rw(static_cast<const R*>(p.dres_out) + base + 8 * v, dr);
                else
#pragma unroll
                    for (int i = 0; i < 8; ++i) dr[i] = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float rh = rv[j][i] * r2;
                    a_pre[j][i] = fmaf(gy[j][i], rh, a_pre[j][i]);
                    dr[i] += r2 * (w[i] * gy[j][i] - rh * m2);
                }
                store8(static_cast<R*>(p.dres) + base + 8 * v, dr);
                if (g) {
                    load8(g + 8 * v, t);
#pragma unroll
                    for (int i = 0; i < 8; ++i) sg[i] = sigmoid_fast(t[i]);
                }
                if (wpost) load8(wpost + 8 * v, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) pv[i] = wpost ? ov[j][i] * r1 * w[i] : ov[j][i];
                if (p.scale) {
                    load8(p.scale + 8 * v, t);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        a_sc[j][i] = fmaf(g ? dr[i] * sg[i] : dr[i], pv[i], a_sc[j][i]);
                        dr[i] *= t[i];
                    }
                }
                if (g) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) t[i] = dr[i] * pv[i] * sg[i] * (1.f - sg[i]);
                    store8(static_cast<E*>(p.dgate) + base + 8 * v, t);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dp[j][i] = g ? dr[i] * sg[i] : dr[i];
                    if (wpost) {
                        const float oh = ov[j][i] * r1;
                        a_post[j][i] = fmaf(dp[j][i], oh, a_post[j][i]);
                        dp[j][i] *= w[i];
                        s1[0] = fmaf(dp[j][i], oh, s1[0]);
                        ov[j][i] = oh;
                    }
                }
            }
        }
        block_sum<1>(s1, red[1]);
        const float m1 = s1[0] * inv;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = threadIdx.x + j * blockDim.x;
            if (v < nv) {
                if (wpost)
#pragma unroll
                    for (int i = 0; i < 8; ++i) dp[j][i] = r1 * (dp[j][i] - ov[j][i] * m1);
                store8(static_cast<E*>(p.d_o) + base + 8 * v, dp[j]);
            }
        }
    }
    float* part = p.part + (int64_t)blockIdx.x * 3 * p.W;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = threadIdx.x + j * blockDim.x;
        if (v < nv) {
            store8(part + 8 * v, a_pre[j]);
            store8(part + p.W + 8 * v, a_post[j]);
            store8(part + 2 * (int64_t)p.W + 8 * v, a_sc[j]);
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

int bwd_blocks(int T, int W) {
    int threads, vpt;
    norm_shape(W, threads, vpt);
    const int per = threads >= 512 ? 1 : 512 / threads;  // 128 registers a thread: 512 threads fill an SM
    const int n = device_sm_count() * (per > 8 ? 8 : per);
    return T < n ? (T > 0 ? T : 1) : n;
}

template <typename E, typename R>
gdn_status run_norm(const NormParams& p, bool bwd, cudaStream_t s) {
    int threads, vpt;
    norm_shape(p.W, threads, vpt);
    if (!bwd) {
        const int per = 2048 / threads;
        const int64_t most = (int64_t)device_sm_count() * (per > 16 ? 16 : per);
        const int grid = (int)(p.T < most ? p.T : most);
        if (vpt == 1) norm_fwd_kernel<E, R, 1><<<grid, threads, 0, s>>>(p);
        else if (vpt == 2) norm_fwd_kernel<E, R, 2><<<grid, threads, 0, s>>>(p);
        else norm_fwd_kernel<E, R, 4><<<grid, threads, 0, s>>>(p);
        return check_launch("norm_fwd_kernel");
    }
    const int grid = bwd_blocks(p.T, p.W);
    if (vpt == 1) norm_bwd_kernel<E, R, 1><<<grid, threads, 0, s>>>(p);
    else if (vpt == 2) norm_bwd_kernel<E, R, 2><<<grid, threads, 0, s>>>(p);
    else norm_bwd_kernel<E, R, 4><<<grid, threads, 0, s>>>(p);
    return check_launch("norm_bwd_kernel");
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
    if (T < 0 || width < 1 || width % 8 != 0 || width > 16384) return 0;
    return (sizeof(float) * 3 * (size_t)width * bwd_blocks(T, width) + 255) & ~size_t(255);
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
    return launch_column_sum(p.part, bwd_blocks(T, width), 3 * (int64_t)width, width, 2 * width, dw_pre,
                             w_post ? dw_post : nullptr, scale ? dscale : nullptr, s);
}

}  // extern "C"
