// The gated delta rule for one token of each request, over a cache of states:
//
//   S' = e^g S,  u = v - S'^T k,  S <- S' + beta k u^T,  o = S^T (scale q)
//      = S'^T (scale q) + beta scale (k.q) u
//
// so both column sums, S'^T k and S'^T q, come from one sweep over the state, which is
// read once and written once.  q and k are read as they come, or divided by their
// norms; the gates come ready or from the raw projections; the gated RMS norm of the
// layer's output is taken from the sums in fp32, before anything is rounded.
//
// What bounds it: 8 dk dv bytes of state a head.  A block holds a whole head in
// registers, 32 values a thread as eight 16-byte pieces of eight rows, all of whose
// loads are in flight before the first sum; a warp covers whole lines of 1024 / dv rows.  The
// sums over rows end in shared memory (two barriers); every warp forms the norms and
// k.q by itself, which takes no barrier.
#include "ssm_common.cuh"
#include "tc_util.cuh"

namespace gdn {

extern __device__ int g_gdn_timeouts;
gdn_status set_smem_attr(const void* func, size_t bytes);

namespace {

// States of a call from which on the heads go through a ring: it keeps the loads of the
// next heads on their way, and costs 2.3 us more to start.  In us, blocks of their own
// against the ring: 32 heads of 128 x 128, 4 requests 5.2, 7.4; 8 10.1, 11.8; 16 (33 MB)
// 19.6, 19.3; 32 34.0, 30.3; 128 122, 94.5; 128 x 64, 16 requests 9.6, 10.2; 32 (33 MB)
// 18.2, 16.9; 64 x 64, 8 heads, 128 requests (17 MB) 8.5, 12.8.
constexpr int64_t kRingBytes = 28 << 20;

struct StepParams {
    const void* q; const void* k; const void* v;  // head h of request b at + b * ld + h * d
    int64_t ldq, ldk, ldv;
    const void* g;      // fp32 [batch, Hv], or with A_log the raw projection a
    const void* beta;   // [batch, Hv], or with A_log the raw projection b
    int64_t ldg, ldb;
    const float* A_log; const float* dt_bias;
    const void* z; int64_t ldz;  // gated norm of the output, or null
    const void* norm_w;
    float eps, scale;
    int l2norm;
    float* states;
    const int32_t* src; const int32_t* dst;
    int num_slots, Hk, Hv, group;
    void* o;
};

// g and beta of a request's head, ready or from the raw projections
template <typename E>
__device__ __forceinline__ void gates(const StepParams& p, int b, int hv, float& g, float& beta) {
    beta = Elem<E>::load(static_cast<const E*>(p.beta) + (int64_t)b * p.ldb + hv);
    if (p.A_log) {
        const float x = Elem<E>::load(static_cast<const E*>(p.g) + (int64_t)b * p.ldg + hv) + __ldg(p.dt_bias + hv);
        g = -expf(__ldg(p.A_log + hv)) * (x > 20.f ? x : log1pf(expf(x)));
        beta = 1.f / (1.f + expf(-beta));
    } else {
        g = __ldg(static_cast<const float*>(p.g) + (int64_t)b * p.ldg + hv);
    }
}

template <typename E, int DK, int DV>
__global__ void __launch_bounds__(DK * DV / 32) rule_step_kernel(const StepParams p) {
    constexpr int NT = DK * DV / 32, NW = NT / 32;
    constexpr int LPR = DV / 4;      // lanes of a row
    constexpr int RPW = 32 / LPR;    // rows of a warp's one load
    constexpr int KP = DK / 32;      // elements of q and k a lane
    __shared__ float part[NW][2][DV];
    __shared__ float sums[2][DV];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.x / p.Hv, hv = blockIdx.x % p.Hv, hk = hv / p.group;
    int slot = p.src ? __ldg(p.src + b) : b;
    const int to = p.dst ? __ldg(p.dst + b) : b;
    E* const out = static_cast<E*>(p.o) + ((int64_t)b * p.Hv + hv) * DV;
    if (to < 0 || to >= p.num_slots) {  // a padded row
        for (int c = tid; c < DV; c += NT) out[c] = Elem<E>::from_f(0.f);
        return;
    }
    const int row0 = warp * (8 * RPW) + lane / LPR, col = (lane % LPR) * 4;
    const int64_t head = (int64_t)DK * DV;
    float4 S[8];
    if (slot >= 0 && slot < p.num_slots) {
        const float* s = p.states + ((int64_t)slot * p.Hv + hv) * head + (int64_t)row0 * DV + col;
#pragma unroll
        for (int i = 0; i < 8; ++i) S[i] = __ldcs(reinterpret_cast<const float4*>(s + i * RPW * DV));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const E* q = static_cast<const E*>(p.q) + (int64_t)b * p.ldq + hk * DK;
    const E* k = static_cast<const E*>(p.k) + (int64_t)b * p.ldk + hk * DK;
    const E* v = static_cast<const E*>(p.v) + (int64_t)b * p.ldv + hv * DV + col;
    float kr[8], qr[8], vc[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        kr[i] = Elem<E>::load(k + row0 + i * RPW);
        qr[i] = Elem<E>::load(q + row0 + i * RPW);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) vc[j] = Elem<E>::load(v + j);
    float qq = 0.f, kk = 0.f, kq = 0.f;
#pragma unroll
    for (int j = 0; j < KP; ++j) {
        const float a = Elem<E>::load(q + lane + 32 * j), c = Elem<E>::load(k + lane + 32 * j);
        qq = fmaf(a, a, qq);
        kk = fmaf(c, c, kk);
        kq = fmaf(a, c, kq);
    }
    float g, beta;
    gates<E>(p, b, hv, g, beta);
    const float decay = expf(g);
#pragma unroll
    for (int m = 16; m; m >>= 1) {
        qq += __shfl_xor_sync(0xffffffffu, qq, m);
        kk += __shfl_xor_sync(0xffffffffu, kk, m);
        kq += __shfl_xor_sync(0xffffffffu, kq, m);
    }
    const float nk = p.l2norm ? rsqrtf(kk + 1e-6f) : 1.f;
    const float nq = p.scale * (p.l2norm ? rsqrtf(qq + 1e-6f) : 1.f);
    float sk[4] = {0.f, 0.f, 0.f, 0.f}, sq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float s[4] = {S[i].x, S[i].y, S[i].z, S[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sk[j] = fmaf(s[j], kr[i], sk[j]);
            sq[j] = fmaf(s[j], qr[i], sq[j]);
        }
    }
#pragma unroll
    for (int m = LPR; m < 32; m <<= 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sk[j] += __shfl_xor_sync(0xffffffffu, sk[j], m);
            sq[j] += __shfl_xor_sync(0xffffffffu, sq[j], m);
        }
    if (lane < LPR) {
        *reinterpret_cast<float4*>(&part[warp][0][col]) = make_float4(sk[0], sk[1], sk[2], sk[3]);
        *reinterpret_cast<float4*>(&part[warp][1][col]) = make_float4(sq[0], sq[1], sq[2], sq[3]);
    }
    __syncthreads();
    for (int c = tid; c < 2 * DV; c += NT) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) t += (&part[w][0][0])[c];
        (&sums[0][0])[c] = t;
    }
    __syncthreads();
    const float dk_ = decay * nk;
    float bu[4];  // beta |k|^-1 u
#pragma unroll
    for (int j = 0; j < 4; ++j) bu[j] = beta * nk * (vc[j] - dk_ * sums[0][col + j]);
    float* d = p.states + ((int64_t)to * p.Hv + hv) * head + (int64_t)row0 * DV + col;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float4 r;
        r.x = fmaf(kr[i], bu[0], decay * S[i].x);
        r.y = fmaf(kr[i], bu[1], decay * S[i].y);
        r.z = fmaf(kr[i], bu[2], decay * S[i].z);
        r.w = fmaf(kr[i], bu[3], decay * S[i].w);
        __stcs(reinterpret_cast<float4*>(d + i * RPW * DV), r);
    }
    if (warp == 0) {
        float o[4], ss = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            o[j] = nq * fmaf(kq, bu[j], decay * sums[1][col + j]);
            ss = fmaf(o[j], o[j], ss);
        }
        if (p.z) {
#pragma unroll
            for (int m = LPR / 2; m; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
            const float r = 1.f / sqrtf(ss * (1.f / DV) + p.eps);
            const E* z = static_cast<const E*>(p.z) + (int64_t)b * p.ldz + (int64_t)hv * DV + col;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float zz = Elem<E>::load(z + j);
                o[j] *= r * Elem<E>::load(static_cast<const E*>(p.norm_w) + col + j) * (zz / (1.f + expf(-zz)));
            }
        }
        if (lane < LPR) {
#pragma unroll
            for (int j = 0; j < 4; ++j) out[col + j] = Elem<E>::from_f(o[j]);
        }
    }
}

// ---- many heads: a ring of them in shared memory ------------------------------

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* mbar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     tc::smem_addr(dst)),
                 "l"(src), "r"(bytes), "r"(tc::smem_addr(mbar))
                 : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(tc::smem_addr(src)),
                 "r"(bytes)
                 : "memory");
}

constexpr int RING = 3;
constexpr uint64_t kWaitNs = 4000000000ull;

// Waits for a phase, up to kWaitNs or until another role gave up
__device__ __forceinline__ bool ring_wait(uint64_t* mbar, uint32_t parity, const volatile int* bad) {
    if (tc::mbar_wait(mbar, parity, 64)) return true;
    uint64_t t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    while (!tc::mbar_wait(mbar, parity, 64)) {
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if (*bad || t - t0 > kWaitNs) return false;
    }
    return true;
}

// What a head's rule needs beside its state, formed a stage ahead
template <int DK, int DV>
struct alignas(16) Head {
    float k[DK], q[DK];          // as they come
    float v[DV];
    float zw[DV];                // norm_w silu(z)
    float decay, bk, nk, nq, kq;  // e^g, beta / |k|, 1 / |k|, scale / |q|, k.q
    int state;                   // has a state to start from
    int at;                      // the head's number; -1: there is none any more
};
template <int DK, int DV>
struct Ring {
    alignas(128) float S[RING][DK * DV];
    Head<DK, DV> head[RING];
    alignas(16) float part[DK * DV / 1024][2][DV];
    alignas(16) float sums[2][DV];
    uint64_t full[RING], done[RING], empty[RING];
    int bad;
};

// The heads of a CTA, blockIdx.x + j gridDim.x, without those of padded rows; a warp looks
// at 32 at a time.
struct Heads {
    int base, to, slot;  // of this lane's head
    unsigned live, padded;
    __device__ __forceinline__ void look(const StepParams& p, int heads) {
        const int64_t i = base + (int64_t)(threadIdx.x & 31) * gridDim.x;
        to = slot = -1;
        if (i < heads) {
            const int b = (int)i / p.Hv;
            to = p.dst ? __ldg(p.dst + b) : b;
            slot = p.src ? __ldg(p.src + b) : b;
            if (to >= p.num_slots) to = -1;
            if (slot >= p.num_slots) slot = -1;
        }
        live = __ballot_sync(0xffffffffu, to >= 0);
        padded = __ballot_sync(0xffffffffu, i < heads && to < 0);
    }
    // the next head's number, -1 behind the last; its slots
    __device__ __forceinline__ int next(const StepParams& p, int heads, int& to_, int& slot_) {
        while (live == 0) {
            const int64_t b = base + 32ll * gridDim.x;
            if (b >= heads) return -1;
            base = (int)b;
            look(p, heads);
        }
        const int l = __ffs(live) - 1;
        live &= live - 1;
        to_ = __shfl_sync(0xffffffffu, to, l);
        slot_ = __shfl_sync(0xffffffffu, slot, l);
        return base + l * gridDim.x;
    }
};

// One CTA walks heads, which go through a ring in shared memory: a warp loads their states,
// by bulk copies, RING warps form what else the rule needs (in fp32, with norms and gates;
// a chain of loads of several heads' time, which is why they are several), NT threads do
// a head at a time, and a warp sends the states back.
template <typename E, int DK, int DV>
__global__ void __launch_bounds__(DK * DV / 32 + 32 * (RING + 2)) rule_ring_kernel(const StepParams p, int heads) {
    constexpr int NT = DK * DV / 32, NW = NT / 32;
    constexpr int LPR = DV / 4, RPW = 32 / LPR;
    constexpr uint32_t BYTES = DK * DV * 4;
    extern __shared__ unsigned char raw[];
    Ring<DK, DV>& sm = *reinterpret_cast<Ring<DK, DV>*>(raw + ((128 - (tc::smem_addr(raw) & 127)) & 127));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < RING; ++s) {
            tc::mbar_init(&sm.full[s], 2);
            tc::mbar_init(&sm.done[s], NW);
            tc::mbar_init(&sm.empty[s], 1);
        }
        sm.bad = 0;
    }
    __syncthreads();
    if (warp >= NW) {
        Heads list;
        list.base = blockIdx.x;
        list.look(p, heads);
        int to, slot;
        if (warp == NW) {
            // ---- states in ----
            for (int n = 0;; ++n) {
                const int i = list.next(p, heads, to, slot), s = n % RING;
                if (n >= RING && !__all_sync(0xffffffffu, ring_wait(&sm.empty[s], (n / RING - 1) & 1, &sm.bad))) {
                    sm.bad = 1;
                    break;
                }
                __syncwarp();
                if (lane == 0) {
                    if (i >= 0 && slot >= 0) {
                        tc::mbar_expect_tx(&sm.full[s], BYTES);
                        bulk_load(sm.S[s], p.states + ((int64_t)slot * p.Hv + i % p.Hv) * (DK * DV), BYTES, &sm.full[s]);
                    } else {
                        tc::mbar_arrive(&sm.full[s]);
                    }
                }
                if (i < 0) break;
            }
        } else if (warp <= NW + RING) {
            // ---- what else the heads of stage s need, read before the stage is free ----
            const int s = warp - NW - 1;
            Head<DK, DV>& h = sm.head[s];
            for (int n = 0;; ++n) {
                const int i = list.next(p, heads, to, slot);
                if (n % RING != s) {
                    if (i < 0) break;
                    continue;
                }
                float qr[DK / 32], kr[DK / 32], vr[DV / 32], zw[DV / 32], g = 0.f, beta = 0.f;
                float qq = 0.f, kk = 0.f, kq = 0.f;
                if (i >= 0) {
                    const int b = i / p.Hv, hv = i % p.Hv, hk = hv / p.group;
                    const E* q = static_cast<const E*>(p.q) + (int64_t)b * p.ldq + hk * DK;
                    const E* k = static_cast<const E*>(p.k) + (int64_t)b * p.ldk + hk * DK;
                    const E* v = static_cast<const E*>(p.v) + (int64_t)b * p.ldv + hv * DV;
#pragma unroll
                    for (int j = 0; j < DK / 32; ++j) {
                        qr[j] = Elem<E>::load(q + lane + 32 * j);
                        kr[j] = Elem<E>::load(k + lane + 32 * j);
                    }
#pragma unroll
                    for (int j = 0; j < DV / 32; ++j) {
                        vr[j] = Elem<E>::load(v + lane + 32 * j);
                        zw[j] = 1.f;
                        if (p.z) {
                            const E* z = static_cast<const E*>(p.z) + (int64_t)b * p.ldz + (int64_t)hv * DV;
                            const float x = Elem<E>::load(z + lane + 32 * j);
                            zw[j] = Elem<E>::load(static_cast<const E*>(p.norm_w) + lane + 32 * j) * (x / (1.f + expf(-x)));
                        }
                    }
                    gates<E>(p, b, hv, g, beta);
#pragma unroll
                    for (int j = 0; j < DK / 32; ++j) {
                        qq = fmaf(qr[j], qr[j], qq);
                        kk = fmaf(kr[j], kr[j], kk);
                        kq = fmaf(qr[j], kr[j], kq);
                    }
#pragma unroll
                    for (int m = 16; m; m >>= 1) {
                        qq += __shfl_xor_sync(0xffffffffu, qq, m);
                        kk += __shfl_xor_sync(0xffffffffu, kk, m);
                        kq += __shfl_xor_sync(0xffffffffu, kq, m);
                    }
                }
                if (n >= RING && !__all_sync(0xffffffffu, ring_wait(&sm.empty[s], (n / RING - 1) & 1, &sm.bad))) {
                    sm.bad = 1;
                    break;
                }
                __syncwarp();
                if (i >= 0) {
#pragma unroll
                    for (int j = 0; j < DK / 32; ++j) {
                        h.q[lane + 32 * j] = qr[j];
                        h.k[lane + 32 * j] = kr[j];
                    }
#pragma unroll
                    for (int j = 0; j < DV / 32; ++j) {
                        h.v[lane + 32 * j] = vr[j];
                        h.zw[lane + 32 * j] = zw[j];
                    }
                }
                if (lane == 0) {
                    const float nk = p.l2norm ? rsqrtf(kk + 1e-6f) : 1.f;
                    h.decay = expf(g);
                    h.nk = nk;
                    h.bk = beta * nk;
                    h.nq = p.scale * (p.l2norm ? rsqrtf(qq + 1e-6f) : 1.f);
                    h.kq = kq;
                    h.state = slot >= 0;
                    h.at = i;
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sm.full[s]);
                if (i < 0) break;
            }
        } else {
            // ---- states out, zeros for padded rows ----
            for (int n = 0;; ++n) {
                const int i = list.next(p, heads, to, slot), s = n % RING;
                if (i < 0) break;
                if (!__all_sync(0xffffffffu, ring_wait(&sm.done[s], (n / RING) & 1, &sm.bad))) {
                    sm.bad = 1;
                    break;
                }
                __syncwarp();
                if (lane == 0) {
                    bulk_store(p.states + ((int64_t)to * p.Hv + i % p.Hv) * (DK * DV), sm.S[s], BYTES);
                    tc::bulk_commit();
                    tc::bulk_wait_read();
                    tc::mbar_arrive(&sm.empty[s]);
                }
            }
            if (sm.bad && lane == 0) {  // a wait ran out: the copies in flight get a millisecond
                atomicAdd(&g_gdn_timeouts, 1);
                for (int i = 0; i < 1000; ++i) __nanosleep(1000);
            }
            __syncwarp();
            for (int64_t i0 = blockIdx.x; i0 < heads; i0 += 32ll * gridDim.x) {
                list.base = (int)i0;
                list.look(p, heads);
                for (unsigned m = list.padded; m; m &= m - 1) {
                    E* const out = static_cast<E*>(p.o) + (i0 + (int64_t)(__ffs(m) - 1) * gridDim.x) * DV;
#pragma unroll
                    for (int j = 0; j < DV / 32; ++j) out[lane + 32 * j] = Elem<E>::from_f(0.f);
                }
            }
        }
        return;
    }
    // ---- the heads ----
    const int row0 = warp * (8 * RPW) + lane / LPR, col = (lane % LPR) * 4;
    for (int n = 0;; ++n) {
        const int s = n % RING;
        if (!tc::bar_and(1, NT, ring_wait(&sm.full[s], (n / RING) & 1, &sm.bad))) {
            sm.bad = 1;
            break;
        }
        if (sm.head[s].at < 0) break;
        E* const out = static_cast<E*>(p.o) + (int64_t)sm.head[s].at * DV;
        const Head<DK, DV>& h = sm.head[s];
        float* const tile = sm.S[s] + row0 * DV + col;
        const bool has = h.state != 0;
        float4 S[8];
        float sk[4] = {0.f, 0.f, 0.f, 0.f}, sq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 8; ++r)
            S[r] = has ? *reinterpret_cast<const float4*>(tile + r * RPW * DV) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const float k = h.k[row0 + r * RPW], q = h.q[row0 + r * RPW];
            const float t[4] = {S[r].x, S[r].y, S[r].z, S[r].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sk[j] = fmaf(t[j], k, sk[j]);
                sq[j] = fmaf(t[j], q, sq[j]);
            }
        }
#pragma unroll
        for (int m = LPR; m < 32; m <<= 1)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sk[j] += __shfl_xor_sync(0xffffffffu, sk[j], m);
                sq[j] += __shfl_xor_sync(0xffffffffu, sq[j], m);
            }
        if (lane < LPR) {
            *reinterpret_cast<float4*>(&sm.part[warp][0][col]) = make_float4(sk[0], sk[1], sk[2], sk[3]);
            *reinterpret_cast<float4*>(&sm.part[warp][1][col]) = make_float4(sq[0], sq[1], sq[2], sq[3]);
        }
        tc::bar_sync(1, NT);
        for (int c = tid; c < 2 * DV; c += NT) {
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) t += (&sm.part[w][0][0])[c];
            (&sm.sums[0][0])[c] = t;
        }
        tc::bar_sync(1, NT);
        const float decay = h.decay, dk_ = decay * h.nk, bk = h.bk;
        float bu[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) bu[j] = bk * (h.v[col + j] - dk_ * sm.sums[0][col + j]);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const float k = h.k[row0 + r * RPW];
            float4 t;
            t.x = fmaf(k, bu[0], decay * S[r].x);
            t.y = fmaf(k, bu[1], decay * S[r].y);
            t.z = fmaf(k, bu[2], decay * S[r].z);
            t.w = fmaf(k, bu[3], decay * S[r].w);
            *reinterpret_cast<float4*>(tile + r * RPW * DV) = t;
        }
        if (warp == NW - 1) {
            float o[4], zw[4], ss = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                o[j] = h.nq * fmaf(h.kq, bu[j], decay * sm.sums[1][col + j]);
                zw[j] = h.zw[col + j];
                ss = fmaf(o[j], o[j], ss);
            }
            if (p.z) {
#pragma unroll
                for (int m = LPR / 2; m; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
                const float r = 1.f / sqrtf(ss * (1.f / DV) + p.eps);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] *= r * zw[j];
            }
            if (lane < LPR) {
#pragma unroll
                for (int j = 0; j < 4; ++j) out[col + j] = Elem<E>::from_f(o[j]);
            }
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.done[s]);
    }
}

// ---- host ----------------------------------------------------------------------

template <typename E, int DK, int DV>
gdn_status run_kernel(const StepParams& p, int heads, cudaStream_t s) {
    constexpr int NT = DK * DV / 32;
    constexpr size_t smem = sizeof(Ring<DK, DV>) + 128;
    if ((int64_t)heads * (DK * DV * 4) >= kRingBytes) {
        const void* fn = (const void*)rule_ring_kernel<E, DK, DV>;
        gdn_status st = set_smem_attr(fn, smem);
        if (st != GDN_OK) return st;
        // CTAs of an SM: by shared memory (a kilobyte of each is the system's) and threads
        int per = (int)((228 << 10) / (smem + 1024));
        if (per > 2048 / (NT + 32 * (RING + 2))) per = 2048 / (NT + 32 * (RING + 2));
        if (per > 16) per = 16;
        const int most = per * device_sm_count();
        rule_ring_kernel<E, DK, DV><<<heads < most ? heads : most, NT + 32 * (RING + 2), smem, s>>>(p, heads);
        return check_launch("rule_ring_kernel");
    }
    rule_step_kernel<E, DK, DV><<<heads, NT, 0, s>>>(p);
    return check_launch("rule_step_kernel");
}

template <typename E, int DK>
gdn_status run_dv(const StepParams& p, int dv, int heads, cudaStream_t s) {
    if (dv == 32) return run_kernel<E, DK, 32>(p, heads, s);
    if (dv == 64) return run_kernel<E, DK, 64>(p, heads, s);
    return run_kernel<E, DK, 128>(p, heads, s);
}

template <typename E>
gdn_status run_step(const StepParams& p, int batch, int dk, int dv, cudaStream_t s) {
    const int heads = batch * p.Hv;
    if (dk == 32) return run_dv<E, 32>(p, dv, heads, s);
    if (dk == 64) return run_dv<E, 64>(p, dv, heads, s);
    return run_dv<E, 128>(p, dv, heads, s);
}

bool head_size(int d) { return d == 32 || d == 64 || d == 128; }

gdn_status check_step(gdn_dtype dtype, int batch, int Hk, int Hv, int dk, int dv, const float* states, int num_slots,
                      const int32_t* src, const int32_t* dst) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return fail(GDN_ERR_DTYPE, "unknown dtype %d", (int)dtype);
    if (batch < 0 || Hk < 1 || Hv < 1 || num_slots < 0)
        return fail(GDN_ERR_INVALID_ARG, "batch=%d Hk=%d Hv=%d num_slots=%d", batch, Hk, Hv, num_slots);
    if (!head_size(dk) || !head_size(dv))
        return fail(GDN_ERR_UNSUPPORTED_SHAPE, "dk=%d, dv=%d must be 32, 64 or 128", dk, dv);
    if (Hv % Hk != 0) return fail(GDN_ERR_UNSUPPORTED_SHAPE, "Hv=%d must be a multiple of Hk=%d", Hv, Hk);
    if ((int64_t)batch * Hv > 0x7fffffff)
        return fail(GDN_ERR_UNSUPPORTED_SHAPE, "batch * Hv = %lld above 2^31 - 1", (long long)batch * Hv);
    if ((int64_t)Hv * 128 > 0x7fffffff) return fail(GDN_ERR_UNSUPPORTED_SHAPE, "Hv=%d", Hv);
    if ((!src || !dst) && num_slots < batch)
        return fail(GDN_ERR_INVALID_ARG, "num_slots=%d < batch=%d without slot numbers", num_slots, batch);
    if (batch > 0 && (!states || (reinterpret_cast<uintptr_t>(states) & 15u)))
        return fail(GDN_ERR_INVALID_ARG, "states must be 16-byte aligned and not NULL");
    return GDN_OK;
}

gdn_status check_ld(const void* p, int64_t ld, int64_t least, const char* name) {
    if (!p) return fail(GDN_ERR_INVALID_ARG, "%s is NULL", name);
    if (ld < least)
        return fail(GDN_ERR_INVALID_ARG, "row stride of %s (%lld) must be >= %lld", name, (long long)ld, (long long)least);
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_chunk_step(const void* q, const void* k, const void* v, int64_t ldq, int64_t ldk, int64_t ldv,
                          gdn_dtype dtype, const float* g, const void* beta, int32_t batch, int32_t Hk, int32_t Hv,
                          int32_t dk, int32_t dv, float scale, uint32_t flags, float* states, int32_t num_slots,
                          const int32_t* src, const int32_t* dst, void* o, void* stream) {
    gdn_status st = check_step(dtype, batch, Hk, Hv, dk, dv, states, num_slots, src, dst);
    if (st != GDN_OK) return st;
    if (flags & ~(uint32_t)GDN_QK_L2NORM) return fail(GDN_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
    if (batch == 0) return GDN_OK;
    if ((st = check_ld(q, ldq, (int64_t)Hk * dk, "q")) != GDN_OK) return st;
    if ((st = check_ld(k, ldk, (int64_t)Hk * dk, "k")) != GDN_OK) return st;
    if ((st = check_ld(v, ldv, (int64_t)Hv * dv, "v")) != GDN_OK) return st;
    if (!g || !beta || !o) return fail(GDN_ERR_INVALID_ARG, "g, beta or o is NULL");
    StepParams p{};
    p.q = q; p.k = k; p.v = v; p.ldq = ldq; p.ldk = ldk; p.ldv = ldv; p.g = g; p.beta = beta; p.ldg = p.ldb = Hv;
    p.scale = scale; p.l2norm = (flags & GDN_QK_L2NORM) != 0; p.states = states; p.src = src; p.dst = dst;
    p.num_slots = num_slots; p.Hk = Hk; p.Hv = Hv; p.group = Hv / Hk; p.o = o;
    return dtype == GDN_BF16 ? run_step<__nv_bfloat16>(p, batch, dk, dv, (cudaStream_t)stream)
                             : run_step<float>(p, batch, dk, dv, (cudaStream_t)stream);
}

gdn_status gdn_layer_step(const void* x, int64_t ldx, const void* a, int64_t lda, const void* b, int64_t ldb,
                          gdn_dtype dtype, const float* A_log, const float* dt_bias, const void* z, int64_t ldz,
                          const void* norm_w, float norm_eps, int32_t batch, int32_t Hk, int32_t Hv, int32_t dk,
                          int32_t dv, float scale, float* states, int32_t num_slots, const int32_t* src,
                          const int32_t* dst, void* y, void* stream) {
    gdn_status st = check_step(dtype, batch, Hk, Hv, dk, dv, states, num_slots, src, dst);
    if (st != GDN_OK) return st;
    if (batch == 0) return GDN_OK;
    const int64_t nk = (int64_t)Hk * dk;
    if ((st = check_ld(x, ldx, 2 * nk + (int64_t)Hv * dv, "x")) != GDN_OK) return st;
    if ((st = check_ld(a, lda, Hv, "a")) != GDN_OK) return st;
    if ((st = check_ld(b, ldb, Hv, "b")) != GDN_OK) return st;
    if (z && (st = check_ld(z, ldz, (int64_t)Hv * dv, "z")) != GDN_OK) return st;
    if (z && !norm_w) return fail(GDN_ERR_INVALID_ARG, "z needs norm_w");
    if (!A_log || !dt_bias || !y) return fail(GDN_ERR_INVALID_ARG, "A_log, dt_bias or y is NULL");
    const size_t e = dtype == GDN_BF16 ? 2 : 4;
    StepParams p{};
    p.q = x; p.k = static_cast<const char*>(x) + e * nk; p.v = static_cast<const char*>(x) + e * 2 * nk;
    p.ldq = p.ldk = p.ldv = ldx; p.g = a; p.ldg = lda; p.beta = b; p.ldb = ldb; p.A_log = A_log; p.dt_bias = dt_bias;
    p.z = z; p.ldz = ldz; p.norm_w = norm_w; p.eps = norm_eps; p.scale = scale; p.l2norm = 1; p.states = states;
    p.src = src; p.dst = dst; p.num_slots = num_slots; p.Hk = Hk; p.Hv = Hv; p.group = Hv / Hk; p.o = y;
    return dtype == GDN_BF16 ? run_step<__nv_bfloat16>(p, batch, dk, dv, (cudaStream_t)stream)
                             : run_step<float>(p, batch, dk, dv, (cudaStream_t)stream);
}

}  // extern "C"
