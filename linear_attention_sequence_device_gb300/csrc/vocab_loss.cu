// Softmax cross entropy over a vocabulary, straight from hidden states and output
// weights, and its gradients; the logits never exist as an array.
//
//   x_tv = scale h_t . w_v        lse_t = log sum_v e^x_tv       loss_t = lse_t - x_{t, target_t}
//   P_tv = scale dloss_t (e^{x_tv - lse_t} - [v = target_t])
//   dh = P w                      dw = P^T h
//
// Four matrix products, one forward and three backward (the logits again, dh, dw), all
// by one kernel on the tensor cores; what bounds them is those.  Forward: a tile's
// epilogue keeps a maximum and a sum of exponentials a row, without the target's, which a
// small launch joins.  Backward, a piece of the vocabulary after the other: a launch writes the
// piece's P in bf16 (another, where the loss is given, P at the targets: 2.5 us), one more forms
// both gradients' products from it.
//
// Numerics.  Products of bf16 inputs are exact and added in fp32; maxima, sums, lse and
// P are fp32.  P is rounded to bf16 for the products behind it, relative to its own
// size, which puts dh and dw off by as much as their own rounding; what that takes from the
// entry at the target, often the largest of its row, is given back in fp32: to dh for every
// token, to dw for the tokens that have a target of their own (dh off by 1.66e-3 of itself
// in norm, its own rounding, and dw by 2.0e-3, 2.3e-3 where most tokens share their targets; 2.5e-3
// both without; P in two parts would take both gradients' products twice).  fp32 inputs, and P for them, are taken as the
// sum of two fp16 parts (22 bits) after a scaling by powers of two that brings the
// largest to 2^14, and three of their four products are formed (of bf16, three parts
// and six products would take it, twice the time).  The scalings: h by its row, w by one
// for all, P by its row's dloss; in dw's product h by the inverse of the latter.  A value
// of 2^-16 of the largest under the same scaling keeps all 22 bits, smaller ones are off
// by up to 2^-39 of the largest (P: 2^-15 and 2^-38 of its dloss, whose largest comes to 2^13).
//
// The product kernel: a pair of CTAs (cta_group::2) forms a 256 x 256 tile, 128 rows of
// each operand a CTA, from a ring of stages of 64 along K by TMA; accumulators in tensor
// memory, two of them, so that the epilogue's sixteen warps run beside the next tile.  One
// CTA an SM walks tiles by its number.
//
// Up to 128 tokens a pair's second CTA would multiply rows of nothing: then each CTA forms
// 128 x 256 tiles by itself (76 tokens of 64000 x 2048 in bf16, loss and gradients: 62 + 202 us by
// pairs, 52 + 174 so).  Calls of few tokens go to vocab_few.cu.
#include <cuda.h>
#include <cuda_fp16.h>

#include "ssm_common.cuh"
#include "tc_util.cuh"
#include "vocab_few.cuh"

namespace gdn {

extern __device__ int g_gdn_timeouts;
gdn_status set_smem_attr(const void* func, size_t bytes);

namespace {

// ---- tensor maps -------------------------------------------------------------

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<EncodeFn>(ptr);
    }();
    return fn;
}

// [parts][rows][cols] bf16 with row stride ld, parts `apart` rows from each other, boxes of
// 64 (or 32) columns and box_rows rows, swizzled over a box's row; what lies outside reads as
// zero and is not written
gdn_status make_map_rows(CUtensorMap* m, const void* base, int64_t ld, int64_t cols, int64_t rows, int64_t apart,
                         int parts, int box_rows, int box_cols = 64) {
    EncodeFn fn = encode_fn();
    if (!fn) return fail(GDN_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)parts};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)ld * 2 * (cuuint64_t)apart};
    const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1}, es[3] = {1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE,
                          box_cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(GDN_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return GDN_OK;
}

gdn_status make_map3(CUtensorMap* m, const void* base, int64_t ld, int64_t cols, int64_t rows, int parts, int box_rows) {
    return make_map_rows(m, base, ld, cols, rows, rows, parts, box_rows);
}

// ---- device: pairs of CTAs ---------------------------------------------------

__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address of this CTA's shared variable in the pair's first CTA
__device__ __forceinline__ uint32_t in_leader(uint32_t addr) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
template <bool ALONE>
__device__ __forceinline__ void arrive(uint32_t addr) {
    if (ALONE) asm volatile("mbarrier.arrive.shared.b64 _, [%0];" ::"r"(addr) : "memory");
    else arrive_cluster(addr);
}
// one box into this CTA's shared memory; its bytes are counted on a barrier of either CTA
__device__ __forceinline__ void load_box(uint32_t dst, const void* map, int x, int y, int z, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(mbar)
        : "memory");
}
// the same without a pair
__device__ __forceinline__ void load_box_alone(uint32_t dst, const void* map, int x, int y, int z, uint64_t* mbar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(tc::smem_addr(mbar))
        : "memory");
}
__device__ __forceinline__ void store_box(const void* map, int x, int y, int z, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// arrives on the barrier at this offset in both CTAs when the products so far are done
__device__ __forceinline__ void commit_pair(uint64_t* mbar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            tc::smem_addr(mbar)),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

constexpr uint64_t kWaitNs = 4000000000ull;

// Waits for a phase, up to kWaitNs or until another role gave up; sets *abort when it
// runs out itself.
__device__ __forceinline__ bool wait_for(uint64_t* mbar, uint32_t parity, volatile int* abort) {
    if (tc::mbar_wait(mbar, parity, 64)) return true;
    const uint64_t t0 = now_ns();
    while (!tc::mbar_wait(mbar, parity, 64)) {
        if (*abort) return false;
        if (now_ns() - t0 > kWaitNs) {
            if (!atomicExch(const_cast<int*>(abort), 1)) atomicAdd(&g_gdn_timeouts, 1);
            return false;
        }
    }
    return true;
}

// ---- the product kernel ------------------------------------------------------

constexpr int BM = 256, BN = 256, BK = 64;      // a pair's tile
constexpr int kNarrow = 128;                    // columns of a tile of the logits where tiles are few
constexpr int HALF = 128;                       // rows of an operand a CTA; a tile's without a pair
constexpr int OPB = HALF * BK * 2;              // bytes of as many rows of a stage
constexpr int GT = 576;                         // threads: a warp of loads, one of products, 16 of epilogue
constexpr int SC = 32;                          // columns of a staged piece of a result
constexpr int OUTB = HALF * SC * 2;             // its bytes; each quarter of the columns has two

enum Kind { K_LSE = 0, K_P = 1, K_GRAD = 2 };

// Up to as many tokens as a CTA has rows (ALONE) each CTA forms 128 x 256 tiles of its own, from all of B.
constexpr int kAloneTokens = 128;

// rows of B of a CTA, bytes of a stage
template <bool ALONE, int TN>
__host__ __device__ constexpr int b_rows() {
    return ALONE ? TN : TN / 2;
}
template <bool ALONE, int TN>
__host__ __device__ constexpr int stage_bytes() {
    return OPB + b_rows<ALONE, TN>() * BK * 2;
}
// Stages of the ring: 144 to 192 KB; results leave through shared memory but for the logits'
// maxima and sums
template <int KIND, bool ALONE, int TN>
__host__ __device__ constexpr int stages() {
    return (KIND == K_LSE ? 192 * 1024 : 160 * 1024) / stage_bytes<ALONE, TN>();
}
template <int KIND>
__host__ __device__ constexpr int staged_bytes() {
    return KIND == K_LSE ? 2 * 3 * HALF * 8 : 4 * 2 * OUTB;
}
struct Ctl {
    uint64_t full[8], empty[8], done[2], free_[2];
    uint32_t tmem;
    int abort;
};
template <int KIND, bool ALONE, int TN>
constexpr size_t smem_bytes() {
    return 1024 + (size_t)stages<KIND, ALONE, TN>() * stage_bytes<ALONE, TN>() + staged_bytes<KIND>() + sizeof(Ctl);
}
static_assert(stages<K_LSE, false, kNarrow>() == 8 && smem_bytes<K_LSE, false, kNarrow>() <= 227 * 1024 &&
                  smem_bytes<K_GRAD, false, BN>() <= 227 * 1024,
              "barriers, shared memory of a CTA");

struct Maps {
    CUtensorMap a, b;    // logits: h, w.  Gradients of h: P, w
    CUtensorMap a2, b2;  // gradients of w: P, h
    CUtensorMap out;     // P, or dw in bf16
};

struct GemmParams {
    int mt, nt, group;    // tiles (logits; gradients of h), rows of tiles walked together
    int kb;               // K steps
    int chunk;            // of which so many are added up at a time
    int splits, kper;     // gradients of h: K cut into splits of kper steps
    int mt2, nt2, kb2;    // gradients of w
    int more, early;      // pairs with a dh tile more than the others; rounds of dw tiles that those run alone
    int f32;              // operands are two parts of fp32 values
    int T, V, W;          // V: columns of this launch's logits (the piece's, from v0 on)
    int v0, vocab;
    float scale;
    const void* targets; int wide;
    float2* stat;         // K_LSE: [nt][T] maximum and sum of a tile's row, without the target
    float* at;            // K_LSE: [T] the target's logit
    const float* lse; const float* dloss;  // K_P
    const int* he; const int* pa;          // fp32: exponents of the scalings of h's rows, of P's
    const int* we;                         // K_LSE in fp32: of w's rows
    const unsigned* most;                  // and what the others are taken from: largest |w|, exponent of |h| 2^-pa
    float* lo;            // [T] what P's entry at the target lost when it was rounded
    const int* only;      // [vocab] the one token with this target; below 0: none or several
    const __nv_bfloat16* h; int64_t ldh;   // gradients of w: the rows behind `only`
    float* acc; int ldacc; int add;        // gradients of h: [splits][T][ldacc] fp32; add to what is there
    void* dw; int64_t lddw; int dw_store;  // dw_store: by TMA through `out`
};

// a token's target: -1 where it is left out, vocab where it is that or more
__device__ __forceinline__ int target_of(const GemmParams& p, int t) {
    if (!p.wide) {
        const int v = __ldg(static_cast<const int*>(p.targets) + t);
        return v < 0 ? -1 : min(v, p.vocab);
    }
    const long long v = __ldg(static_cast<const long long*>(p.targets) + t);
    return v < 0 ? -1 : v > p.vocab ? p.vocab : (int)v;
}

struct Unit {
    int m, n, k0, k1, split;
    bool second;  // a gradient of w
};

// Unit i of a pair of CTAs (or of one alone), false behind its last.  Logits: tile pair + i pairs.  Gradients:
// dh's tiles the same way, then dw's, of which the pairs that have a tile of dh less run
// `early` more, so that all end together (round robin over both kinds left the last fifth
// of a short call's time to a few pairs).
template <int KIND>
__device__ __forceinline__ bool unit(const GemmParams& p, int pair, int pairs, int i, Unit& r) {
    r.second = false;
    r.split = 0;
    r.k0 = 0;
    r.k1 = p.kb;
    const int n1 = p.mt * p.nt * (KIND == K_GRAD ? p.splits : 1);
    const int u = pair + i * pairs;
    if (KIND != K_GRAD) {
        if (u >= n1) return false;
        // `group` rows of tiles, column after column: the tiles that run together share
        // few operands
        const int per = p.group * p.nt, g = u / per, first = g * p.group;
        const int rows = min(p.group, p.mt - first), in = u - g * per;
        r.m = first + in % rows;
        r.n = in / rows;
        return true;
    }
    if (u < n1) {
        const int tiles = p.mt * p.nt;
        r.split = u / tiles;
        const int in = u - r.split * tiles;
        r.m = in / p.nt;
        r.n = in % p.nt;
        r.k0 = r.split * p.kper;
        r.k1 = min(p.kb, r.k0 + p.kper);
        return true;
    }
    const bool fewer = pair >= p.more;  // pairs 0 .. more - 1 have one tile of dh more
    int j = i - n1 / pairs - (fewer ? 0 : 1), v;
    if (fewer && j < p.early) {
        v = j * (pairs - p.more) + pair - p.more;
    } else {
        if (fewer) j -= p.early;
        v = p.early * (pairs - p.more) + j * pairs + pair;
    }
    if (v >= p.mt2 * p.nt2) return false;
    r.second = true;
    r.m = v / p.nt2;
    r.n = v % p.nt2;
    r.k1 = p.kb2;
    return true;
}

// part of a and of b of product c: high and low, low and high, high and high
__device__ __forceinline__ int part_a(int c) { return c == 1; }
__device__ __forceinline__ int part_b(int c) { return c == 0; }

// 2^k, -126 <= k <= 127
__device__ __forceinline__ float pow2(int k) { return __int_as_float((k + 127) << 23); }
// the exponent k, -126 to 126, that brings m to [2^to, 2^(to + 1)); 0 where m is zero or not finite
__device__ __forceinline__ int exponent_for(float m, int to) {
    if (!(m > 0.f) || !isfinite(m)) return 0;
    const int k = to + 127 - (__float_as_int(m) >> 23);
    return k < -126 ? -126 : k > 126 ? 126 : k;
}

// floor(log2 m) of a positive finite m
__device__ __forceinline__ int log2_floor(float m) {
    const int b = __float_as_int(m);
    return b >> 23 ? (b >> 23) - 127 : -118 - __clz(b);
}
// most[1], the largest log2_floor(|h_t|) - pa[t] of the tokens that count, plus kMostBias (0: none), as a
// whole number: |h_t| 2^-pa[t] itself may lie below fp32's range.  The exponent that brings it to
// [2^14, 2^15); beyond 2^250 dw is zero or infinite.
constexpr int kMostBias = 1024;
__device__ __forceinline__ int exponent_of_h(unsigned most) {
    return most ? max(-250, min(250, 14 + kMostBias - (int)most)) : 0;
}

// K steps that are added up in tensor memory; CH = 0: all.  The tensor cores cut their
// sums towards zero, step after step: 2^-24 of a sum each, always to the same side.
// Where that counts, chunks are added up in registers, rounded: for logits of bf16 (the loss
// of 4096 tokens, 50021 columns and a width of 2048 off by 1.6e-6 of itself without chunks,
// 0.4e-6 with eight steps each; 531 us without, 541 with 16, 560 with 8), and for all of
// fp32, whose small products come first in a chunk, while the sum is small.  The
// gradients' logits are added up as the loss's are, of bf16 bit for bit (of fp32 w has its rows'
// scalings there and one for all here): where a token is nearly certain and the loss is not
// given, P at its target is a small difference from 1, which errors that lse does not
// share would drown (5 tokens with 1 - p of 1e-4: dh off by 3.7e-2 of itself).
// The gradients' products of bf16 are added up in one chain of up to kMostSteps steps, 16384 tokens
// or words; longer ones (LONG) in chunks of kChunkGrad (one chain over 2^20 tokens or 2^16 words: 1.5e-3 and
// 6e-4 too small).  Chunks for all: 130 x 32000 x 2048 124 us instead of 118, 1000 x 32000 x 2048
// 267 instead of 261; 8192 x 131072 x 2048, where words come in 32768, 8.16 ms instead of 8.09.  Up
// to 128 tokens have no chunks (local memory), and their words at most 16 splits of kMostSteps.
template <int KIND, bool F32, bool LONG>
__host__ __device__ constexpr bool chunked() {
    return F32 || KIND != K_GRAD || LONG;
}
constexpr int kChunkF32 = 4;   // the most steps of a chunk
constexpr int kChunkBf16 = 12;
constexpr int kChunkGrad = 64;
constexpr int kMostSteps = 256;
// and of the logits of up to kFewTokens tokens: the loss of one token may be a small difference of
// large logits, which no other token's outweighs (single tokens: losses off by up to 3.8e-6
// of themselves with twelve steps, 1.2e-6 with two, before those had kernels of their own; 130 tokens of 32000 x 2048, both
// directions: 149 us with twelve, 156 with four, 169 with two)
constexpr int kChunkFew = 2, kFewTokens = 64;

// v = x, or x -= g, where column o is i, for every i of a row in registers.  Written out:
// the compiler makes an array in local memory of a chain of choices.
__device__ __forceinline__ void take_at(float& v, float x, int o, int i) {
    asm volatile("{\n .reg .pred p;\n setp.eq.s32 p, %2, %3;\n @p mov.f32 %0, %1;\n}\n" : "+f"(v) : "f"(x), "r"(o), "r"(i));
}
__device__ __forceinline__ void sub_at(float& x, float g, int o, int i) {
    asm volatile("{\n .reg .pred p;\n setp.eq.s32 p, %2, %3;\n @p sub.f32 %0, %0, %1;\n}\n" : "+f"(x) : "f"(g), "r"(o), "r"(i));
}

// A warp's 32 rows and the 32 columns behind j of its quarter, staged at `mine`, to dh's sums
// or dw, a row at a time.  (What they need is found again: the sums leave few registers.)
template <int KIND, bool F32, bool ALONE>
__device__ __forceinline__ void store_rows(const GemmParams& p, int pair, int pairs, int u, uint32_t rank, uint32_t mine,
                                           int j) {
    int t;
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(t));
    asm volatile("" : "+r"(u));
    Unit w;
    unit<KIND>(p, pair, pairs, u, w);
    constexpr int EW = BN / 4;  // columns of an epilogue warp
    const int l = t & 31, row = w.m * (ALONE ? HALF : BM) + (int)rank * HALF + ((t >> 5) & 3) * 32;
    const int col = w.n * BN + ((t >> 5) - 2) / 4 * EW + j + l;
    const int n = min(32, (w.second ? p.V : p.T) - row);
    if (col >= (w.second ? p.W : p.ldacc)) return;
    auto value = [&](int i) {
        float v;
        asm volatile("ld.shared.f32 %0, [%1];"
                     : "=f"(v)
                     : "r"(mine + i * 128 + (((l >> 2) ^ (i & 7)) << 4) + (l & 3) * 4)
                     : "memory");
        return v;
    };
    if (F32 || !w.second) {
        float* q = (w.second ? static_cast<float*>(p.dw) + row * p.lddw
                             : p.acc + ((int64_t)w.split * p.T + row) * p.ldacc) + col;
        const int64_t ld = w.second ? p.lddw : p.ldacc;
        const bool add = !w.second && p.add;
#pragma unroll 4
        for (int i = 0; i < n; ++i, q += ld) *q = value(i) + (add ? *q : 0.f);
    } else {
        __nv_bfloat16* q = static_cast<__nv_bfloat16*>(p.dw) + row * p.lddw + col;
#pragma unroll 4
        for (int i = 0; i < n; ++i, q += p.lddw) *q = __float2bfloat16_rn(value(i));
    }
}

template <int KIND, bool F32, bool ALONE, int TN, bool LONG>
__global__ void __cluster_dims__(ALONE ? 1 : 2, 1, 1) __launch_bounds__(GT, 1)
    vocab_gemm_kernel(const GemmParams p, const __grid_constant__ Maps maps) {
    constexpr bool CH = chunked<KIND, F32, LONG>();
    const int ch = p.chunk;
    constexpr int NP = F32 ? 3 : 1;  // products of parts
    constexpr int STAGES = stages<KIND, ALONE, TN>(), STAGE = stage_bytes<ALONE, TN>(), TM = ALONE ? HALF : BM;
    constexpr int HB = b_rows<ALONE, TN>();
    constexpr int EW = TN / 4;  // columns of an epilogue warp: a quarter of the tile's
    extern __shared__ unsigned char raw[];
    unsigned char* base = raw + ((1024 - (tc::smem_addr(raw) & 1023)) & 1023);
    const uint32_t ring = tc::smem_addr(base);
    unsigned char* staged = base + STAGES * STAGE;
    Ctl& c = *reinterpret_cast<Ctl*>(staged + staged_bytes<KIND>());
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = ALONE ? 0u : cta_rank();
    const int pair = ALONE ? blockIdx.x : blockIdx.x >> 1, pairs = ALONE ? gridDim.x : gridDim.x >> 1;
    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            tc::mbar_init(&c.full[s], 1);
            tc::mbar_init(&c.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&c.done[b], 1);
            tc::mbar_init(&c.free_[b], ALONE ? 16 : 32);  // a warp of the epilogue (of either CTA) each
        }
        c.abort = 0;
    }
    if (ALONE) {
        if (warp == 0) tc::tmem_alloc(&c.tmem, 512);
    } else if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc::smem_addr(&c.tmem)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc::fence_before();
    __syncthreads();
    if (!ALONE) cluster_sync();
    tc::fence_after();
    const uint32_t tmem = c.tmem;
    Unit w;

    if (warp == 0 && lane == 0) {
        // ---- loads ----
        int s = 0, phase = 0;
        int64_t issued = 0;
        bool ok = true;
        for (int i = 0; ok && unit<KIND>(p, pair, pairs, i, w); ++i) {
            const int row_a = w.m * TM + (int)rank * HALF, row_b = w.n * TN + (int)rank * HB;
            for (int k0 = w.k0; k0 < w.k1 && ok; k0 += CH ? ch : w.k1 - w.k0) {
                const int k1 = CH ? min(w.k1, k0 + ch) : w.k1;
                for (int q = 0; q < NP && ok; ++q)
                    for (int k = k0; k < k1; ++k) {
                        if (issued >= STAGES && !wait_for(&c.empty[s], phase ^ 1, &c.abort)) {
                            ok = false;
                            break;
                        }
                        if (rank == 0) tc::mbar_expect_tx(&c.full[s], (ALONE ? 1 : 2) * STAGE);
                        const uint32_t bar = ALONE ? 0u : in_leader(tc::smem_addr(&c.full[s]));
                        const uint32_t da = ring + s * STAGE, db = da + OPB;
                        const int za = F32 ? part_a(q) : 0, zb = F32 ? part_b(q) : 0;
                        auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y, int z) {
                            if (ALONE) load_box_alone(dst, map, x, y, z, &c.full[s]);
                            else load_box(dst, map, x, y, z, bar);
                        };
                        constexpr int BH = HB > HALF ? 2 : 1;  // copies of B
                        if (KIND != K_GRAD) {
                            load(da, &maps.a, k * BK, row_a, za);
#pragma unroll
                            for (int i = 0; i < BH; ++i) load(db + i * OPB, &maps.b, k * BK, row_b + i * HALF, zb);
                        } else if (!w.second) {  // P [t][v], K = v; w [v][column]
                            load(da, &maps.a, k * BK, row_a, za);
#pragma unroll
                            for (int i = 0; i < 2 * BH; ++i) load(db + i * (OPB / 2), &maps.b, row_b + i * 64, k * BK, zb);
                        } else {  // P [t][v], K = t; h [t][column]
                            load(da, &maps.a2, row_a, k * BK, za);
                            load(da + OPB / 2, &maps.a2, row_a + 64, k * BK, za);
#pragma unroll
                            for (int i = 0; i < 2 * BH; ++i) load(db + i * (OPB / 2), &maps.b2, row_b + i * 64, k * BK, zb);
                        }
                        ++issued;
                        if (++s == STAGES) {
                            s = 0;
                            phase ^= 1;
                        }
                    }
            }
        }
        // every stage's products are done, and with them the loads and the arrivals here
        if (ok) {
            const int left = issued < STAGES ? (int)issued : STAGES;
            int ls = s, lp = phase;
            for (int i = 0; i < left && ok; ++i) {
                if (issued < STAGES) {  // stages 0 .. issued - 1, first use
                    ok = wait_for(&c.empty[i], 0, &c.abort);
                } else {
                    ok = wait_for(&c.empty[ls], lp ^ 1, &c.abort);
                    if (++ls == STAGES) {
                        ls = 0;
                        lp ^= 1;
                    }
                }
            }
        }
        if (!ok) {  // gave up: let the copies in flight land
            const uint64_t t0 = now_ns();
            while (now_ns() - t0 < 1000000ull) __nanosleep(1000);
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ---- products ----
        int s = 0, phase = 0, it = 0;
        bool ok = true;
        for (int i = 0; ok && unit<KIND>(p, pair, pairs, i, w); ++i) {
            const bool a_mn = KIND == K_GRAD && w.second, b_mn = KIND == K_GRAD;
            // (bits 7 and 10: operands of bf16 instead of fp16)
            const uint32_t id = (tc::idesc_bf16(TM, TN, false, b_mn, false) | (a_mn ? 1u << 15 : 0u)) &
                                (F32 ? ~(1u << 7 | 1u << 10) : ~0u);
            int k0 = w.k0;
            do {
                const int k1 = CH ? min(w.k1, k0 + ch) : w.k1;
                const int buf = it & 1;
                if (it >= 2 && !wait_for(&c.free_[buf], ((it >> 1) & 1) ^ 1, &c.abort)) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                const uint32_t d = tmem + (uint32_t)buf * TN;
                uint32_t acc = 0;
                const int steps = (k1 - k0) * NP;
                for (int k = 0; k < steps; ++k) {
                    if (!wait_for(&c.full[s], phase, &c.abort)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after();
                    const uint32_t ra = ring + s * STAGE, rb = ra + OPB;
                    const uint64_t da = tc::desc(ra, a_mn ? OPB / 2 : 16, 1024);
                    const uint64_t db = tc::desc(rb, b_mn ? OPB / 2 : 16, 1024);
                    const uint64_t sa = a_mn ? 128 : 2, sb = b_mn ? 128 : 2;
#pragma unroll
                    for (int j = 0; j < BK / 16; ++j) {
                        if (ALONE) tc::mma(d, da + sa * j, db + sb * j, id, acc);
                        else mma_pair(d, da + sa * j, db + sb * j, id, acc);
                        acc = 1;
                    }
                    if (ALONE) tc::commit(&c.empty[s]);
                    else commit_pair(&c.empty[s]);
                    if (++s == STAGES) {
                        s = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                if (ALONE) tc::commit(&c.done[buf]);
                else commit_pair(&c.done[buf]);
                ++it;
                k0 = k1;
            } while (k0 < w.k1);
        }
    } else if (warp >= 2) {
        // ---- epilogue: this thread's row, a quarter of the columns ----
        // its lanes of tensor memory and columns
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)((warp - 2) >> 2) * EW;
        // K_LSE: the other quarters' maximum and sum of a row, of this tile and the last
        float2* part = reinterpret_cast<float2*>(staged);
        int it = 0, tile = 0;
        bool ok = true;
        // gradients of bf16: the one token with this thread's row of w as its target, looked up a tile
        // ahead (dw of 130 tokens: a tile's loads take as long as its products)
        constexpr bool ONLY = KIND == K_GRAD && !F32;
        auto only_of = [&](int u) {
            Unit x;
            if (!unit<KIND>(p, pair, pairs, u, x) || !x.second) return -1;
            const int r = x.m * TM + (int)rank * HALF + (warp & 3) * 32 + lane;
            return r < p.V ? __ldg(p.only + p.v0 + r) : -1;
        };
        int only = ONLY ? only_of(0) : -1;
        for (int u = 0; unit<KIND>(p, pair, pairs, u, w); ++u) {
            const int only_next = ONLY ? only_of(u + 1) : -1;
            float acc[CH ? EW : 1];
#pragma unroll
            for (int i = 0; i < (CH ? EW : 1); ++i) acc[i] = 0.f;
            uint32_t d = 0;
            uint32_t release = 0;
            for (int left = CH ? (w.k1 - w.k0 + ch - 1) / ch : 1; left > 0; --left) {
                const int buf = it & 1;
                // A wait that gives up ends no loop here: the warps' barriers stay matched, and what is
                // left of the tiles goes by without waiting, with whatever the accumulators hold.
                if (ok) ok = wait_for(&c.done[buf], (it >> 1) & 1, &c.abort);
                __syncwarp();
                tc::fence_after();
                d = lanes + (uint32_t)buf * TN;
                release = ALONE ? tc::smem_addr(&c.free_[buf]) : in_leader(tc::smem_addr(&c.free_[buf]));
                if constexpr (CH) {
#pragma unroll
                    for (int j = 0; j < EW; j += 8) {
                        float x[8];
                        tc::ld8(d + j, x);
#pragma unroll
                        for (int i = 0; i < 8; ++i) acc[j + i] += x[i];
                    }
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) arrive<ALONE>(release);
                }
                ++it;
            }
            // (found again: the sums above leave few registers)
            int t = tid;
            if (CH) {
                asm volatile("" : "+r"(u));
                unit<KIND>(p, pair, pairs, u, w);
                asm volatile("mov.u32 %0, %%tid.x;" : "=r"(t));
            }
            const int quad = (t >> 5) & 3, quarter = ((t >> 5) - 2) >> 2, row = quad * 32 + (t & 31);
            const bool lead = quad == 0 && (t & 31) == 0;  // of the quarter: its stores
            const uint32_t stage = ring + STAGES * STAGE + (KIND == K_LSE ? 0 : quarter * 2 * OUTB);
            const int r0 = ALONE && KIND != K_GRAD ? 0 : w.m * TM + (int)rank * HALF, r = r0 + row;
            const int c0 = w.n * TN + quarter * EW;
            // logits and sums of fp32 inputs are 2^(exponents of the scalings) times too large (dh's
            // by w's after this)
            float f = p.scale, f2 = 1.f;
            if (F32) {
                if (KIND == K_LSE) {
                    // half of h's before w's, half behind: alone it may pass fp32's range where w's brings it back
                    f = r < p.T ? pow2(-__ldg(p.he + r) / 2) * p.scale : 0.f;
                } else if (KIND == K_P) {
                    // (beyond the range of one factor the logits are below 2^-80, or infinite)
                    const int k = -exponent_for(__uint_as_float(__ldg(p.most)), 14) - (r < p.T ? __ldg(p.he + r) : 0);
                    f = pow2(max(-126, min(127, k))) * p.scale;
                } else if (!w.second) {
                    f = r < p.T ? pow2(-__ldg(p.pa + r)) : 0.f;
                } else {
                    const int k = exponent_of_h(__ldg(p.most + 1));  // up to 250: in two factors
                    f = pow2(-k / 2);
                    f2 = pow2(-k - -k / 2);
                }
            }
            if (KIND == K_LSE) {
                const bool real = r < p.T;
                const int left = p.V - c0;
                const int o = real ? target_of(p, r) - c0 : -1;
                float top = -INFINITY, sum = 0.f;
                if constexpr (CH) {
#pragma unroll
                    for (int i = 0; i < EW; i += 4) {
                        int4 e = make_int4(0, 0, 0, 0);
                        if (F32) e = __ldg(reinterpret_cast<const int4*>(p.we + c0 + i));
                        const int es[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[i + j] = F32 ? acc[i + j] * f * pow2(-es[j]) : acc[i + j] * f;
                    }
                    if (F32) {  // (read again: a register less)
                        int k = 0;
                        if (real) asm volatile("ld.global.s32 %0, [%1];" : "=r"(k) : "l"(p.he + r));
                        f = pow2(-k - -k / 2);
                    }
#pragma unroll
                    for (int i = 0; i < EW; ++i) {
                        if (F32) acc[i] *= f;
                        if (i >= left) acc[i] = -INFINITY;
                    }
                    // the target's logit goes its own way (lse_join_kernel)
                    if (o >= 0 && o < EW) {
                        float v = 0.f;
#pragma unroll
                        for (int i = 0; i < EW; ++i) {
                            take_at(v, acc[i], o, i);
                            take_at(acc[i], -INFINITY, o, i);
                        }
                        p.at[r] = v;
                    }
#pragma unroll
                    for (int i = 0; i < EW; ++i) top = fmaxf(top, acc[i]);
                    const float ref = top == -INFINITY ? 0.f : top;
                    float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < EW; ++i) s4[i & 3] += exp2_fast((acc[i] - ref) * kLog2e);
                    sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
                }
                part = reinterpret_cast<float2*>(staged) + (tile++ & 1) * 3 * HALF;
                if (quarter) part[(quarter - 1) * HALF + row] = make_float2(top, sum);
                tc::bar_sync(1, 512);
                if (!quarter && real) {
#pragma unroll
                    for (int i = 0; i < 3; ++i) {
                        const float2 v = part[i * HALF + row];
                        const float m = fmaxf(top, v.x), ref = m == -INFINITY ? 0.f : m;
                        sum = sum * exp2_fast((top - ref) * kLog2e) + v.y * exp2_fast((v.x - ref) * kLog2e);
                        top = m;
                    }
                    p.stat[(int64_t)w.n * p.T + r] = make_float2(top, sum);
                }
            } else if (KIND == K_P || (!F32 && w.second && p.dw_store)) {
                float lse = 0.f, g = 0.f;
                int tgt = -1;  // the target's column of this piece
                if (KIND == K_P && r < p.T) {
                    tgt = target_of(p, r);
                    lse = __ldg(p.lse + r);
                    g = tgt < 0 ? 0.f : tgt >= p.vocab ? NAN : __ldg(p.dloss + r) * p.scale;
                    tgt = tgt < 0 ? -1 : tgt - p.v0;
                    if (F32) g *= pow2(__ldg(p.pa + r));
                }
                const bool live = KIND != K_P || g != 0.f;
                float lo = 0.f;
                const __nv_bfloat16* hrow = nullptr;
                if (ONLY && only >= 0) {
                    lo = __ldg(p.lo + only);
                    hrow = p.h + only * p.ldh;
                }
                constexpr int PARTS = KIND == K_P && F32 ? 2 : 1;
                const int out_cols = KIND == K_P ? p.V : p.W, out_rows = KIND == K_P ? p.T : p.V;
                // the copies of the last tile have read their pieces
                if (PARTS == 1) {
                    if (lead) tc::bulk_wait_read();
                    tc::bar_sync(2 + quarter, 128);
                }
#pragma unroll
                for (int j = 0; j < EW; j += SC) {
                    float x[SC];
                    if constexpr (CH) {
#pragma unroll
                        for (int i = 0; i < SC; ++i) {
                            x[i] = acc[j + i];
                            asm volatile("" : "+f"(x[i]));  // (one piece at a time: registers)
                        }
                    } else {
                        __syncwarp();  // (behind branches of single lanes: the load is the whole warp's)
                        tc::ld32(d + j, x);
                        if (j == EW - SC) {  // the tile is read
                            tc::fence_before();
                            __syncwarp();
                            if (lane == 0) arrive<ALONE>(release);
                        }
                    }
                    if (KIND == K_P) {
#pragma unroll
                        for (int i = 0; i < SC; ++i) x[i] = live ? g * exp2_fast((__fmul_rn(x[i], f) - lse) * kLog2e) : 0.f;
                        const int o = tgt < 0 ? -1 : tgt - (c0 + j);
                        if (o >= 0 && o < SC) {
                            float at = 0.f;
#pragma unroll
                            for (int i = 0; i < SC; ++i) {
                                sub_at(x[i], live ? g : 0.f, o, i);
                                if (!F32) take_at(at, x[i], o, i);
                            }
                            if (!F32) p.lo[r] = at - __bfloat162float(__float2bfloat16_rn(at));
                        }
                    } else if (hrow) {
#pragma unroll
                        for (int i = 0; i < SC; i += 8) {
                            if (c0 + j + i >= p.W) break;  // (rows of whole 16-byte pieces)
                            float f[8];
                            load8(hrow + c0 + j + i, f);
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[i + e] = fmaf(lo, f[e], x[i + e]);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < PARTS; ++q) {
                        const uint32_t to = stage + ((j / SC * PARTS + q) & 1) * OUTB;
                        if (PARTS > 1) {  // one piece may still be on its way, the other one
                            if (lead) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                            tc::bar_sync(2 + quarter, 128);
                        }
#pragma unroll
                        for (int h = 0; h < SC / 8; ++h) {
                            uint4 o4;
                            uint32_t* o32 = reinterpret_cast<uint32_t*>(&o4);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int e = h * 8 + i * 2;
                                if (PARTS > 1) {
                                    const __half2 b = __floats2half2_rn(x[e], x[e + 1]);
                                    o32[i] = *reinterpret_cast<const uint32_t*>(&b);
                                    x[e] -= __low2float(b);
                                    x[e + 1] -= __high2float(b);
                                } else {
                                    o32[i] = tc::pack_bf16x2(x[e], x[e + 1]);
                                }
                            }
                            // rows of 64 bytes under the 64-byte swizzle
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                             to + row * 64 + ((h ^ ((row >> 1) & 3)) << 4)),
                                         "r"(o4.x), "r"(o4.y), "r"(o4.z), "r"(o4.w)
                                         : "memory");
                        }
                        if (PARTS > 1) {
                            tc::fence_async_smem();
                            tc::bar_sync(2 + quarter, 128);
                            if (lead) {
                                // (a group is closed with or without a copy: the wait above counts them)
                                if (c0 + j < out_cols && r0 < out_rows) store_box(&maps.out, c0 + j, r0, q, to);
                                tc::bulk_commit();
                            }
                        }
                    }
                }
                if (PARTS == 1) {
                    tc::fence_async_smem();
                    tc::bar_sync(2 + quarter, 128);
                    if (lead && r0 < out_rows) {
                        for (int j = 0; j < EW; j += SC)
                            if (c0 + j < out_cols) store_box(&maps.out, c0 + j, r0, 0, stage + j / SC * OUTB);
                        tc::bulk_commit();
                    }
                }
            } else {
                // fp32 results, or bf16 ones that TMA cannot store: through 4 KB of the warp's own, so that
                // a warp stores a row's 32 columns at a time (dw of 32003 x 1001 in fp32, row by row of a
                // thread: 390 us of both gradients' products instead of 247)
                float lo = 0.f;
                const __nv_bfloat16* hrow = nullptr;
                if (ONLY && only >= 0) {
                    lo = __ldg(p.lo + only);
                    hrow = p.h + only * p.ldh;
                }
                const int tl = t & 31;
                const uint32_t mine = stage + quad * 4096;
#pragma unroll
                for (int j = 0; j < EW; j += 32) {
                    float x[CH ? 1 : 32];
                    if constexpr (!CH) {
                        __syncwarp();  // (behind branches of single lanes: the load is the whole warp's)
                        tc::ld32(d + j, x);
                        if (j == EW - 32) {
                            tc::fence_before();
                            __syncwarp();
                            if (lane == 0) arrive<ALONE>(release);
                        }
                    }
                    const int col = c0 + j;
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        float y[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if constexpr (CH) {
                                y[e] = acc[j + i + e];
                                asm volatile("" : "+f"(y[e]));  // (a few at a time: registers)
                            } else {
                                y[e] = x[i + e];
                            }
                            if (F32) y[e] = y[e] * f * f2;
                            if (!F32 && hrow && col + i + e < p.W) y[e] = fmaf(lo, __bfloat162float(hrow[col + i + e]), y[e]);
                        }
                        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(mine + tl * 128 + (((i >> 2) ^ (tl & 7)) << 4)),
                                     "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3])
                                     : "memory");
                    }
                    __syncwarp();
                    store_rows<KIND, F32, ALONE>(p, pair, pairs, u, rank, mine, j);
                }
            }
            only = only_next;
        }
        if ((warp & 3) == 0 && lane == 0) tc::bulk_wait();  // the threads that stored
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (!ALONE) cluster_sync();
    tc::fence_after();
    if (ALONE) {
        if (warp == 0) tc::tmem_dealloc(tmem, 512);
    } else if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ---- small kernels -----------------------------------------------------------

__device__ __forceinline__ int64_t raw_target(const void* targets, int wide, int64_t r) {
    return wide ? __ldg(static_cast<const long long*>(targets) + r) : __ldg(static_cast<const int*>(targets) + r);
}

// bf16 [rows][W] -> [rows][ld]: the tokens' h, then w (V = 0: h alone).  For the gradients
// (targets): tokens that are left out, or whose dloss is zero, are rows of zeros (0 times an
// infinity there would reach every weight's gradient), and `only` gets the token of every
// target that has just one.  Columns of W and beyond are written as zeros.
__global__ void __launch_bounds__(256) pack_kernel(const __nv_bfloat16* __restrict__ h, int64_t ldh, int T,
                                                   const __nv_bfloat16* __restrict__ w, int64_t ldw, int V, int W, int ld,
                                                   const void* targets, int wide, const float* dloss, int vocab, int* only,
                                                   __nv_bfloat16* __restrict__ out_h, __nv_bfloat16* __restrict__ out_w) {
    const int nv = ld / 8;
    const int64_t n = ((int64_t)T + V) * nv;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        int64_t r = i / nv;
        const int c = (int)(i - r * nv) * 8;
        bool real = true;
        const bool of_w = r >= T;
        if (of_w) {
            r -= T;
        } else if (targets) {
            const int64_t tgt = raw_target(targets, wide, r);
            real = tgt >= 0 && __ldg(dloss + r) != 0.f;
            // the one token with a target; a second one makes it -2, whatever their order
            if (c == 0 && real && tgt < vocab && atomicCAS(only + tgt, -1, (int)r) != -1) only[tgt] = -2;
        }
        const __nv_bfloat16* s = (of_w ? w + r * ldw : h + r * ldh) + c;
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = real && c + j < W ? __bfloat162float(s[j]) : 0.f;
        store8((of_w ? out_w : out_h) + r * ld + c, f);
    }
}

// The scalings of fp32 inputs of the gradients: a warp a row of h, then of w.  most[0]: the
// largest |w|; most[1]: of the largest |h_t| 2^-pa[t] over the tokens that count (exponent_of_h).
__global__ void __launch_bounds__(256) scale_kernel(const float* __restrict__ h, int64_t ldh, int T,
                                                    const float* __restrict__ w, int64_t ldw, int V, int W,
                                                    const void* targets, int wide, const float* dloss, float scale,
                                                    int* he, int* pa, unsigned* most) {
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * 8;
    float wm = 0.f;
    int hm = 0;
    const bool dense = ldw == W && (reinterpret_cast<uintptr_t>(w) & 15u) == 0;
    if (dense) {  // w as one array (rows of 1001: 20 us, 31 by rows)
        const int64_t n = (int64_t)V * W, n4 = n / 4;
        const float4* w4 = reinterpret_cast<const float4*>(w);
#pragma unroll 8
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (int64_t)gridDim.x * 256) {
            const float4 v = __ldg(w4 + i);
            // (a NaN is left out)
            wm = fmaxf(wm, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
        }
        if (blockIdx.x == 0 && threadIdx.x < n - 4 * n4) wm = fmaxf(wm, fabsf(__ldg(w + 4 * n4 + threadIdx.x)));
    }
    for (int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); r < (int64_t)T + (dense ? 0 : V); r += step) {
        const float* x = r < T ? h + r * ldh : w + (r - T) * ldw;
        float m = 0.f;
#pragma unroll 8
        for (int c = lane; c < W; c += 32) {
            const float a = fabsf(__ldg(x + c));
            m = a > m ? a : m;  // (a NaN is left out)
        }
        if (r >= T) {
            wm = fmaxf(wm, m);
            continue;
        }
#pragma unroll
        for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
        if (lane == 0) {
            he[r] = exponent_for(m, 14);
            const bool real = raw_target(targets, wide, r) >= 0;
            const int a = real ? exponent_for(fabsf(__ldg(dloss + r) * scale), 13) : 0;
            pa[r] = a;
            if (real && __ldg(dloss + r) != 0.f && m > 0.f && isfinite(m)) hm = max(hm, log2_floor(m) - a + kMostBias);
        }
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, k));
    // (bits of numbers that are not negative are ordered as they are)
    if (lane == 0 && wm > 0.f) atomicMax(most, __float_as_uint(wm));
    if (lane == 0 && hm > 0) atomicMax(most + 1, (unsigned)hm);
}

// For the loss alone both are scaled by their rows, which takes one pass over w: a warp
// finds a row's exponent and splits it, the second time out of the caches (scoring 513 x
// 32000 x 1024: 171 us with a pass for w's largest value before, 150 so).
__global__ void __launch_bounds__(256) split_rows_kernel(const float* __restrict__ h, int64_t ldh, int T,
                                                         const float* __restrict__ w, int64_t ldw, int V, int W, int ld,
                                                         int* __restrict__ he, int* __restrict__ we,
                                                         __half* __restrict__ out_h, __half* __restrict__ out_w) {
    const int lane = threadIdx.x & 31;
    const int64_t n = (int64_t)V + T;
    for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < n; i += (int64_t)gridDim.x * 8) {
        const bool of_w = i < V;
        const int64_t r = of_w ? i : i - V, low = of_w ? V : T;  // the second parts' first row
        const float* s = of_w ? w + r * ldw : h + r * ldh;
        __half* out = (of_w ? out_w : out_h) + r * ld;
        float m = 0.f;
#pragma unroll 8
        for (int c = lane; c < W; c += 32) m = fmaxf(m, fabsf(__ldg(s + c)));  // (a NaN is left out)
#pragma unroll
        for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
        const int k = exponent_for(m, 14);
        if (lane == 0) (of_w ? we : he)[r] = k;
        const float k1 = pow2(k);
#pragma unroll 4
        for (int c = 2 * lane; c < ld; c += 64) {
            const float a = c < W ? __ldg(s + c) * k1 : 0.f, b = c + 1 < W ? __ldg(s + c + 1) * k1 : 0.f;
            const __half2 v = __floats2half2_rn(a, b);
            const float va = __low2float(v), vb = __high2float(v);
            *reinterpret_cast<__half2*>(out + c) = v;
            *reinterpret_cast<__half2*>(out + low * ld + c) =
                __floats2half2_rn(isfinite(va) ? a - va : 0.f, isfinite(vb) ? b - vb : 0.f);
        }
    }
}

// fp32 [rows][W] -> two fp16 parts [2][rows][ld] of its scaled values, in one launch: w by
// most[0]'s exponent; h for the logits by its rows' own, he; h for dw by most[1]'s less the
// row's pa, zeros where a token does not count.
__global__ void __launch_bounds__(256) split_kernel(const float* __restrict__ h, int64_t ldh, int T,
                                                    const float* __restrict__ w, int64_t ldw, int V, int W, int ld,
                                                    const int* he, const int* pa, const unsigned* most,
                                                    const void* targets, int wide, const float* dloss,
                                                    __half* __restrict__ out_h, __half* __restrict__ out_hw,
                                                    __half* __restrict__ out_w) {
    const int nv = ld / 8;
    const int64_t n = ((int64_t)V + 2 * (int64_t)T) * nv;
    const int all = exponent_for(__uint_as_float(__ldg(most)), 14), all_h = exponent_of_h(__ldg(most + 1));
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        int64_t r = i / nv, rows = V;
        const int c = (int)(i - r * nv) * 8;
        int k = all;
        bool real = true;
        const float* s = w + r * ldw + c;
        __half* out = out_w;
        if (r >= V) {
            r -= V;
            rows = T;
            const bool of_dw = r >= T;
            if (of_dw) r -= T;
            s = h + r * ldh + c;
            out = of_dw ? out_hw : out_h;
            k = of_dw ? max(-250, min(250, all_h - __ldg(pa + r))) : __ldg(he + r);
            if (of_dw) real = raw_target(targets, wide, r) >= 0 && __ldg(dloss + r) != 0.f;
        }
        // (up to 2^250: in two steps)
        const float k1 = pow2(k / 2), k2 = pow2(k - k / 2);
        uint4 hi, lo;
        __half2* h2 = reinterpret_cast<__half2*>(&hi);
        __half2* l2 = reinterpret_cast<__half2*>(&lo);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float a = real && c + j < W ? s[j] * k1 * k2 : 0.f, b = real && c + j + 1 < W ? s[j + 1] * k1 * k2 : 0.f;
            const __half2 v = __floats2half2_rn(a, b);
            const float va = __low2float(v), vb = __high2float(v);
            h2[j / 2] = v;
            l2[j / 2] = __floats2half2_rn(isfinite(va) ? a - va : 0.f, isfinite(vb) ? b - vb : 0.f);
        }
        *reinterpret_cast<uint4*>(out + r * ld + c) = hi;
        *reinterpret_cast<uint4*>(out + (rows + r) * ld + c) = lo;
    }
}

// lse and loss of 32 rows from the tiles' maxima and sums, which are those of all words but
// the target, and the target's logit: eight threads a row
__global__ void __launch_bounds__(256) lse_join_kernel(const float2* __restrict__ stat, int nt, int T, int V,
                                                       const float* __restrict__ at, const void* targets, int wide,
                                                       float* __restrict__ loss, float* __restrict__ lse) {
    __shared__ float2 part[8][32];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int r = blockIdx.x * 32 + lane;
    float m = -INFINITY, s = 0.f;
    if (r < T) {
#pragma unroll 4
        for (int n = g; n < nt; n += 8) {
            const float2 v = __ldg(stat + (int64_t)n * T + r);
            const float t = fmaxf(m, v.x), ref = t == -INFINITY ? 0.f : t;
            s = s * exp2_fast((m - ref) * kLog2e) + v.y * exp2_fast((v.x - ref) * kLog2e);
            m = t;
        }
    }
    part[g][lane] = make_float2(m, s);
    __syncthreads();
    if (g || r >= T) return;
    for (int i = 1; i < 8; ++i) {
        const float2 v = part[i][lane];
        const float t = fmaxf(m, v.x), ref = t == -INFINITY ? 0.f : t;
        s = s * exp2_fast((m - ref) * kLog2e) + v.y * exp2_fast((v.x - ref) * kLog2e);
        m = t;
    }
    const int64_t tgt = raw_target(targets, wide, r);
    if (tgt < 0 || tgt >= V) {  // nothing was left out of the sums
        lse[r] = m + logf(s);
        loss[r] = tgt < 0 ? 0.f : NAN;
        return;
    }
    // loss = log(1 + s e^(m - x)), x the target's logit: with the target's own term, 1, in s,
    // a loss of 1e-5 would be good to 2^-24 of that 1, and not of itself
    const float x = __ldg(at + r), d = m - x;
    if (d <= 0.f) {
        const float l = x == INFINITY ? NAN : log1pf(s * expf(d));
        loss[r] = l;
        lse[r] = x + l;
    } else {
        const float l = logf(s + expf(-d));
        loss[r] = d + l;
        lse[r] = m + l;
    }
}

// P at the targets of this piece, dloss scale (softmax - 1), from the loss, -log softmax, instead of
// lse: beside a rounded lse a softmax near 1 cannot be told from it.  (Not by the kernel that
// forms the rest of P: its fp32 form has no register left.)
// pa: the scalings of P in fp32, which is in two parts then.
__global__ void __launch_bounds__(256) hot_kernel(const float* __restrict__ dloss, const float* __restrict__ loss,
                                                  const void* targets, int wide, float scale, int T, int v0, int cols,
                                                  const int* pa, void* P, int64_t ldp, float* lo) {
    for (int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x; r < T; r += (int64_t)gridDim.x * 256) {
        const int64_t tgt = raw_target(targets, wide, r);
        if (tgt < v0 || tgt - v0 >= cols) continue;
        const int64_t c = tgt - v0;
        float g = __ldg(dloss + r) * scale;
        if (pa) g *= pow2(__ldg(pa + r));
        const float x = g != 0.f ? g * expm1f(-__ldg(loss + r)) : 0.f;  // (no gradient, whatever the loss)
        if (pa) {
            __half* o = static_cast<__half*>(P) + r * ldp + c;
            const __half hi = __float2half_rn(x);
            o[0] = hi;
            o[(int64_t)T * ldp] = __float2half_rn(x - __half2float(hi));
        } else {
            const __nv_bfloat16 b = __float2bfloat16_rn(x);
            static_cast<__nv_bfloat16*>(P)[r * ldp + c] = b;
            lo[r] = x - __bfloat162float(b);
        }
    }
}

// dh from the splits' sums, eight columns a thread; for bf16 with what P's rounding took
// at the target (lo)
template <typename E>
__global__ void __launch_bounds__(256) dh_kernel(const float* __restrict__ acc, int splits, int T, int W, int ldacc,
                                                 const float* __restrict__ lo, const void* targets, int wide, int vocab,
                                                 const E* __restrict__ w, int64_t ldw, const unsigned* most,
                                                 E* __restrict__ dh, int64_t lddh, int vec) {
    const int nv = ldacc / 8;
    const float f32 = sizeof(E) == 4 ? pow2(-exponent_for(__uint_as_float(__ldg(most)), 14)) : 1.f;  // w's scaling
    const int64_t n = (int64_t)T * nv;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = (n >> 31) ? i / nv : (int64_t)((unsigned)i / (unsigned)nv);
        const int c = (int)(i - r * nv) * 8;
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
        for (int s = 0; s < splits; ++s) {
            float x[8];
            load8(acc + (s * (int64_t)T + r) * ldacc + c, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] += x[j];
        }
        if (sizeof(E) == 2) {
            const int64_t tgt =
                wide ? __ldg(static_cast<const long long*>(targets) + r) : __ldg(static_cast<const int*>(targets) + r);
            if (tgt >= 0 && tgt < vocab) {
                const float l = __ldg(lo + r);
                float x[8];
                if (vec) load8(w + tgt * ldw + c, x);
                else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = c + j < W ? Elem<E>::to_f(w[tgt * ldw + c + j]) : 0.f;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = fmaf(l, x[j], f[j]);
            }
        }
        if (sizeof(E) == 4) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= f32;
        }
        E* o = dh + r * lddh + c;
        if (vec) store8(o, f);
        else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < W) o[j] = Elem<E>::from_f(f[j]);
        }
    }
}

// ---- host --------------------------------------------------------------------

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }
int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
int round8(int W) { return (W + 7) / 8 * 8; }

// An operand that the tensor maps read as it is: bf16 with rows of whole 16-byte pieces
bool direct(gdn_dtype dt, int W) { return dt == GDN_BF16 && W % 8 == 0; }

bool alone(int T) { return T <= kAloneTokens; }

// Columns of a piece of the vocabulary: P of up to half a gigabyte (more only where 1024
// columns take more), whole tiles; up to 128 tokens in bf16 as many as 16 splits of dh's K take
constexpr size_t kPieceBytes = size_t(512) << 20;
int piece_cols(int T, int V, gdn_dtype dt) {
    int64_t c = (int64_t)(kPieceBytes / ((size_t)(dt == GDN_F32 ? 4 : 2) * (size_t)T)) / BN * BN;
    if (c < 1024) c = 1024;
    if (dt == GDN_BF16 && alone(T) && c > 16 * kMostSteps * BK) c = 16 * kMostSteps * BK;
    const int64_t all = div_up(V, BN) * BN;
    return (int)(c < all ? c : all);
}
int rows_of_tile(int T) { return alone(T) ? HALF : BM; }

// Columns of a tile of the logits: half of them where whole tiles would leave half of the GPU idle
// (66 x 5310 x 3498 in fp32, loss and gradients: 111 + 186 us in whole tiles, 95 + 158 so; 49 x 1738 x
// 1786 in bf16: 24 + 42, 22 + 40)
int tile_cols(int T, int V) {
    const int64_t tiles = div_up(T, rows_of_tile(T)) * div_up(V, kNarrow);
    return tiles <= device_sm_count() / (alone(T) ? 1 : 2) ? kNarrow : BN;
}
// rows of w of a copy
int copy_rows(int T, int cols) { return alone(T) ? HALF : cols / 2; }

// K of dh's product cut into as many splits as leave its tiles no more than the pairs of
// CTAs; splits of 16 steps at least, of up to 128 tokens in bf16 kMostSteps at most
int dh_splits(int T, int W, int cols, gdn_dtype dt) {
    const int64_t tiles = div_up(T, rows_of_tile(T)) * div_up(W, BN), kb = div_up(cols, BK);
    int64_t s = device_sm_count() / (alone(T) ? 1 : 2) / tiles;
    if (s > kb / 16) s = kb / 16;
    if (s > 16) s = 16;
    if (s < 1) s = 1;
    if (dt == GDN_BF16 && alone(T) && s < div_up(kb, kMostSteps)) s = div_up(kb, kMostSteps);
    return (int)div_up(kb, div_up(kb, s));  // none is left without steps
}

// What the workspace holds of a call of T tokens is never less than of a call of fewer, so that one
// for the longest serves all: of the sizes that fall with T, the most up to T.
// Sums of dh's splits, in rows: the GPU's pairs (or CTAs) shared among tiles of 256 (128) tokens
int64_t most_sums(int64_t T, int W, int V, gdn_dtype dt) {
    const int64_t nw = div_up(W, BN), kb = div_up(V, BN) * (BN / BK), most = kb / 16 < 16 ? kb / 16 : 16;
    auto rows = [&](int64_t ctas, int64_t tiles, int64_t t) {
        const int64_t s = ctas / (tiles * nw) < most ? ctas / (tiles * nw) : most;
        return (s < 1 ? 1 : s) * t;
    };
    const int64_t few = T < kAloneTokens ? T : kAloneTokens;
    int64_t n = rows(device_sm_count(), 1, few);
    if (dt == GDN_BF16) {
        const int64_t s = div_up(kb, kMostSteps) < 16 ? div_up(kb, kMostSteps) : 16;
        if (s * few > n) n = s * few;
    }
    if (T > kAloneTokens)
        for (int64_t m = 1; m <= div_up(T, BM); ++m) {
            const int64_t pairs = device_sm_count() / 2, x = rows(pairs, m, T < m * BM ? T : m * BM);
            if (x > n) n = x;
            if (m * nw >= pairs) break;  // one split from here on: T rows
        }
    return n > T ? n : T;
}
// Elements of a piece's P
int64_t most_p(int64_t T, int V, gdn_dtype dt) {
    const int64_t all = T * (div_up(V, BN) * BN), bytes = dt == GDN_F32 ? 4 : 2;
    const int64_t piece = (int64_t)kPieceBytes / bytes > T * 1024 ? (int64_t)kPieceBytes / bytes : T * 1024;
    return all < piece ? all : piece;
}
// Maxima and sums of the logits' tiles: the narrow ones' of as many tokens as have them
int64_t most_stats(int64_t T, int V) {
    const int64_t nn = div_up(V, kNarrow), rows = device_sm_count() / 2 / nn * BM;
    int64_t t = rows < T ? rows : T;
    if (nn <= device_sm_count()) {
        const int64_t alone = T < kAloneTokens ? T : kAloneTokens;
        if (alone > t) t = alone;
    }
    const int64_t wide = div_up(V, BN) * T;
    return nn * t > wide ? nn * t : wide;
}

struct Plan {
    size_t h, hw, w, stat, at, p, acc, lo, only, he, pa, we, most, total;
    int piece, splits, ldacc;
    bool few;
};
Plan plan(int T, int V, int W, gdn_dtype dt, bool grad) {
    Plan l{};
    size_t o = 0;
    const int parts = dt == GDN_F32 ? 2 : 1;
    const int64_t ld = round8(W);
    const int64_t t = T > 0 ? T : 1;
    // few tokens: the sizes fall where another kernel takes them, behind these numbers
    size_t few = 0;
    for (int n : {1, 4, 8, 16, (int)t}) {
        if (n > t || !few_takes(n, V, W, dt)) continue;
        const size_t stat = up256(sizeof(float2) * (size_t)few_blocks(n, V) * n), p = up256(sizeof(float) * (size_t)V * n);
        const size_t all = grad ? p + up256(sizeof(float) * (size_t)few_parts(n, V, W, dt) * n * W) : stat + up256(sizeof(float) * n);
        if (all > few) few = all;
        if (n == t) {
            l.few = true;
            l.acc = p;  // behind P, which begins the workspace
            l.at = stat;
        }
    }
    if (l.few) {
        l.total = few;
        return l;
    }
    if (grad || !direct(dt, W)) {
        l.h = o;
        o += up256((size_t)parts * t * ld * 2);
    }
    if (!direct(dt, W)) {
        l.w = o;
        o += up256((size_t)parts * V * ld * 2);
    }
    if (dt == GDN_F32) {
        l.he = o;
        o += up256(sizeof(int) * t);
        if (!grad) {
            l.we = o;
            o += up256(sizeof(int) * (size_t)div_up(V, BN) * BN);
        } else {
            l.most = o;
            o += 256;
            l.pa = o;
            o += up256(sizeof(int) * t);
            l.hw = o;
            o += up256((size_t)parts * t * ld * 2);
        }
    }
    if (!grad) {
        l.stat = o;
        o += up256(sizeof(float2) * (size_t)most_stats(t, V));
        l.at = o;
        o += up256(sizeof(float) * t);
    } else {
        l.piece = piece_cols((int)t, V, dt);
        l.splits = dh_splits((int)t, W, l.piece, dt);
        l.ldacc = (int)ld;
        l.p = o;
        o += up256((size_t)parts * most_p(t, V, dt) * 2);
        l.acc = o;
        o += up256(sizeof(float) * (size_t)most_sums(t, W, V, dt) * ld);
        l.lo = o;
        o += up256(sizeof(float) * t);
        l.only = o;
        o += up256(sizeof(int) * (size_t)V);
    }
    l.total = o > few ? o : few;
    return l;
}

// Pairs of CTAs that run at the same time, a CTA an SM; asked once per device
int pair_count(const void* fn, size_t smem) {
    constexpr int kMaxDev = 64;
    static int known[kMaxDev] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return device_sm_count() / 2;
    if (known[dev]) return known[dev];
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(device_sm_count() / 2 * 2);
    cfg.blockDim = dim3(GT);
    cfg.dynamicSmemBytes = smem;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = device_sm_count() / 2;
    }
    known[dev] = n;
    return n;
}

// The rounds of dw tiles that the pairs with one dh tile less run alone: the count that makes
// the longest pair's time least.  Times in K steps; a tile of few steps takes its epilogue's.
void balance(GemmParams& p, int64_t n1, int64_t n2, int pairs) {
    constexpr int64_t kEpilogue = 8;
    const int64_t c1 = (p.kper > kEpilogue ? p.kper : kEpilogue), c2 = (p.kb2 > kEpilogue ? p.kb2 : kEpilogue);
    const int64_t more = n1 % pairs, rest = pairs - more;
    p.more = (int)more;
    p.early = 0;
    if (more == 0) return;
    int64_t best = -1;
    const int64_t most = c1 / c2 + 2 < div_up(n2, rest) ? c1 / c2 + 2 : div_up(n2, rest);
    for (int64_t e = 0; e <= most; ++e) {
        const int64_t left = n2 - e * rest, b = left > 0 ? div_up(left, pairs) : 0;  // rounds of all pairs
        const int64_t t = b * c2 + (c1 > e * c2 ? c1 : e * c2);
        if (best < 0 || t < best) {
            best = t;
            p.early = (int)e;
        }
    }
}

template <int KIND, bool F32, bool ALONE, int TN, bool LONG = false>
gdn_status launch_gemm_t(GemmParams p, const Maps& m, cudaStream_t s) {
    if constexpr (KIND == K_GRAD && !F32 && !ALONE && !LONG)
        if (p.kper > kMostSteps || p.kb2 > kMostSteps) return launch_gemm_t<KIND, F32, ALONE, TN, true>(p, m, s);
    const void* fn = (const void*)vocab_gemm_kernel<KIND, F32, ALONE, TN, LONG>;
    constexpr size_t smem = smem_bytes<KIND, ALONE, TN>();
    gdn_status st = set_smem_attr(fn, smem);
    if (st != GDN_OK) return st;
    const int64_t n1 = (int64_t)p.mt * p.nt * (KIND == K_GRAD ? p.splits : 1), n2 = (int64_t)p.mt2 * p.nt2;
    if (n1 + n2 > 0x7fffffff / 2) return fail(GDN_ERR_UNSUPPORTED_SHAPE, "%lld tiles", (long long)(n1 + n2));
    int pairs = ALONE ? device_sm_count() : pair_count(fn, smem);
    if (n1 + n2 < pairs) pairs = (int)(n1 + n2);
    const int steps =
        KIND != K_GRAD && p.T <= kFewTokens ? kChunkFew : F32 ? kChunkF32 : KIND == K_GRAD ? kChunkGrad : kChunkBf16;
    p.chunk = KIND == K_GRAD ? steps : (int)div_up(p.kb, div_up(p.kb, steps));
    if (KIND == K_GRAD) balance(p, n1, n2, pairs);
    vocab_gemm_kernel<KIND, F32, ALONE, TN, LONG><<<(ALONE ? 1 : 2) * (unsigned)pairs, GT, smem, s>>>(p, m);
    return check_launch("vocab_gemm_kernel");
}
template <int KIND, bool F32>
gdn_status launch_gemm_f(const GemmParams& p, const Maps& m, int cols, cudaStream_t s) {
    if constexpr (KIND != K_GRAD)
        if (cols == kNarrow)
            return alone(p.T) ? launch_gemm_t<KIND, F32, true, kNarrow>(p, m, s) : launch_gemm_t<KIND, F32, false, kNarrow>(p, m, s);
    return alone(p.T) ? launch_gemm_t<KIND, F32, true, BN>(p, m, s) : launch_gemm_t<KIND, F32, false, BN>(p, m, s);
}
// cols: a tile's columns
template <int KIND>
gdn_status launch_gemm(const GemmParams& p, const Maps& m, int cols, cudaStream_t s) {
    return p.f32 ? launch_gemm_f<KIND, true>(p, m, cols, s) : launch_gemm_f<KIND, false>(p, m, cols, s);
}

unsigned grid_for(int64_t n) {
    const int64_t b = div_up(n, 256), most = (int64_t)device_sm_count() * 16;
    return (unsigned)(b < 1 ? 1 : b < most ? b : most);
}

gdn_status pack(const void* h, int64_t ldh, int T, const void* w, int64_t ldw, int V, int W, const void* targets, int wide,
                const float* dloss, int vocab, int* only, void* out_h, void* out_w, cudaStream_t s) {
    const int ld = round8(W);
    pack_kernel<<<grid_for(((int64_t)T + V) * (ld / 8)), 256, 0, s>>>(
        static_cast<const __nv_bfloat16*>(h), ldh, T, static_cast<const __nv_bfloat16*>(w), ldw, V, W, ld, targets, wide,
        dloss, vocab, only, static_cast<__nv_bfloat16*>(out_h), static_cast<__nv_bfloat16*>(out_w));
    return check_launch("pack_kernel");
}
// fp32 inputs of the gradients: their scalings, then their parts into the workspace
gdn_status split(const void* h, int64_t ldh, int T, const void* w, int64_t ldw, int V, int W, const void* targets, int wide,
                 const float* dloss, float scale, const Plan& l, char* ws, cudaStream_t s) {
    const int ld = round8(W);
    int* he = reinterpret_cast<int*>(ws + l.he);
    int* pa = reinterpret_cast<int*>(ws + l.pa);
    unsigned* most = reinterpret_cast<unsigned*>(ws + l.most);
    const float *hf = static_cast<const float*>(h), *wf = static_cast<const float*>(w);
    if (cudaMemsetAsync(most, 0, 2 * sizeof(unsigned), s) != cudaSuccess) return check_launch("memset");
    const int64_t blocks = div_up((int64_t)T + V, 8), wave = (int64_t)device_sm_count() * 8;
    scale_kernel<<<(unsigned)(blocks < wave ? blocks : wave), 256, 0, s>>>(hf, ldh, T, wf, ldw, V, W, targets, wide, dloss,
                                                                           scale, he, pa, most);
    split_kernel<<<grid_for(((int64_t)V + 2 * (int64_t)T) * (ld / 8)), 256, 0, s>>>(
        hf, ldh, T, wf, ldw, V, W, ld, he, pa, most, targets, wide, dloss, reinterpret_cast<__half*>(ws + l.h),
        reinterpret_cast<__half*>(ws + l.hw), reinterpret_cast<__half*>(ws + l.w));
    return check_launch("split_kernel");
}

// What a product reads: the array itself, or its packed copy
struct Operand {
    const void* base;
    int64_t ld;
};

// Rows of tiles that are walked together: their rows of h stay in L2 (32 MB of 129)
int group_rows(int mt, int W, int parts) {
    int64_t g = (int64_t(32) << 20) / ((int64_t)BM * W * 2 * parts);
    if (g > 16) g = 16;
    if (g < 1) g = 1;
    return (int)(g < mt ? g : mt);
}

gdn_status check_loss(gdn_dtype dtype, int32_t index_bits, int T, int V, int W, const void* h, int64_t ldh,
                      const void* w, int64_t ldw, const void* targets, float scale) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return fail(GDN_ERR_DTYPE, "unknown dtype %d", (int)dtype);
    if (index_bits != 32 && index_bits != 64) return fail(GDN_ERR_DTYPE, "targets of %d bits", index_bits);
    if (T < 0 || V < 1 || W < 1) return fail(GDN_ERR_INVALID_ARG, "T=%d vocab=%d width=%d", T, V, W);
    if (T > (1 << 28) || V > (1 << 28) || W > (1 << 20))
        return fail(GDN_ERR_UNSUPPORTED_SHAPE, "T=%d or vocab=%d above 2^28, or width=%d above 2^20", T, V, W);
    if (!w || (T > 0 && (!h || !targets))) return fail(GDN_ERR_INVALID_ARG, "h, w or targets is NULL");
    if ((T > 0 && ldh < W) || ldw < W) return fail(GDN_ERR_INVALID_ARG, "row strides of h and w must be >= width=%d", W);
    if (direct(dtype, W) && ((T > 0 && ((reinterpret_cast<uintptr_t>(h) & 15u) || ldh % 8)) ||
                             (reinterpret_cast<uintptr_t>(w) & 15u) || ldw % 8))
        return fail(GDN_ERR_INVALID_ARG, "h and w must be 16-byte aligned with row strides that are multiples of 8");
    if (ldh > (int64_t(1) << 36) || ldw > (int64_t(1) << 36)) return fail(GDN_ERR_UNSUPPORTED_SHAPE, "row strides");
    if (!(scale - scale == 0.f)) return fail(GDN_ERR_INVALID_ARG, "scale is not finite");
    return GDN_OK;
}
gdn_status check_ws(const void* ws, size_t have, size_t need) {
    if (!ws || have < need)
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes < required %zu", ws ? have : 0, need);
    if (reinterpret_cast<uintptr_t>(ws) & 255u) return fail(GDN_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    return GDN_OK;
}
bool loss_sizes_ok(int T, int V, int W, gdn_dtype dt) {
    return T >= 0 && V >= 1 && W >= 1 && T <= (1 << 28) && V <= (1 << 28) && W <= (1 << 20) &&
           (dt == GDN_F32 || dt == GDN_BF16);
}

// loss: the forward's, or null: then P at the targets is what lse says
gdn_status loss_bwd(const float* dloss, const void* h, int64_t ldh, const void* w, int64_t ldw, gdn_dtype dtype,
                    const void* targets, int32_t index_bits, const float* loss, const float* lse, int32_t T, int32_t vocab,
                    int32_t width, float scale, void* dh, int64_t lddh, void* dw, int64_t lddw, void* workspace,
                    size_t workspace_bytes, void* stream) {
    gdn_status st = check_loss(dtype, index_bits, T, vocab, width, h, ldh, w, ldw, targets, scale);
    if (st != GDN_OK) return st;
    const Plan l = plan(T, vocab, width, dtype, true);
    if ((st = check_ws(workspace, workspace_bytes, l.total)) != GDN_OK) return st;
    if (!dw || lddw < width) return fail(GDN_ERR_INVALID_ARG, "dw is NULL or its row stride < width=%d", width);
    cudaStream_t s = (cudaStream_t)stream;
    const size_t e = dtype == GDN_F32 ? 4 : 2;
    if (T == 0) {
        if (cudaMemset2DAsync(dw, e * lddw, 0, e * width, vocab, s) != cudaSuccess) return check_launch("memset");
        return GDN_OK;
    }
    if (!dloss || !lse || !dh || lddh < width)
        return fail(GDN_ERR_INVALID_ARG, "dloss, lse or dh is NULL, or dh's row stride < width=%d", width);
    char* ws = static_cast<char*>(workspace);
    const int wide = index_bits == 64, parts = dtype == GDN_F32 ? 2 : 1;
    if (l.few)
        return few_grads({h, ldh, w, ldw, dtype, targets, wide, T, vocab, width, scale}, dloss, loss, lse,
                         reinterpret_cast<float*>(ws + l.p), reinterpret_cast<float*>(ws + l.acc), dh, lddh, dw, lddw, s);
    const int ldp = round8(width);
    int* only = nullptr;
    Operand H{ws + l.h, ldp}, Hw{ws + (dtype == GDN_F32 ? l.hw : l.h), ldp}, Wt{w, ldw};
    if (!direct(dtype, width)) Wt = {ws + l.w, ldp};
    if (dtype == GDN_F32) {
        if ((st = split(h, ldh, T, w, ldw, vocab, width, targets, wide, dloss, scale, l, ws, s)) != GDN_OK) return st;
    } else {
        only = reinterpret_cast<int*>(ws + l.only);
        if (cudaMemsetAsync(only, 0xff, sizeof(int) * (size_t)vocab, s) != cudaSuccess) return check_launch("memset");
        if ((st = pack(h, ldh, T, w, ldw, direct(dtype, width) ? 0 : vocab, width, targets, wide, dloss, vocab, only,
                       ws + l.h, ws + l.w, s)) != GDN_OK)
            return st;
    }
    const bool store = dtype == GDN_BF16 && (reinterpret_cast<uintptr_t>(dw) & 15u) == 0 && lddw % 8 == 0;
    GemmParams p{};
    p.mt = (int)div_up(T, rows_of_tile(T));
    p.group = group_rows(p.mt, width, parts);
    p.f32 = parts == 2;
    p.T = T; p.W = width; p.vocab = vocab; p.scale = scale;
    p.targets = targets; p.wide = wide; p.lse = lse; p.dloss = dloss;
    p.lo = reinterpret_cast<float*>(ws + l.lo);
    p.only = only;
    p.he = reinterpret_cast<int*>(ws + l.he);
    p.pa = reinterpret_cast<int*>(ws + l.pa);
    p.most = reinterpret_cast<unsigned*>(ws + l.most);
    p.h = reinterpret_cast<const __nv_bfloat16*>(ws + l.h); p.ldh = ldp;
    for (int v0 = 0; v0 < vocab; v0 += l.piece) {
        const int cols = vocab - v0 < l.piece ? vocab - v0 : l.piece;
        // the piece's rows of w, whose parts lie a whole vocabulary apart
        Maps m{};
        const char* wp = static_cast<const char*>(Wt.base) + 2 * (int64_t)v0 * Wt.ld;
        const void* P = ws + l.p;
        p.v0 = v0;
        p.V = cols;
        // the piece's P
        if ((st = make_map3(&m.a, H.base, H.ld, width, T, parts, HALF)) != GDN_OK) return st;
        const int tn = tile_cols(T, cols);
        if ((st = make_map_rows(&m.b, wp, Wt.ld, width, cols, vocab, parts, copy_rows(T, tn))) != GDN_OK) return st;
        if ((st = make_map_rows(&m.out, P, l.piece, cols, T, T, parts, HALF, SC)) != GDN_OK) return st;
        p.nt = (int)div_up(cols, tn);
        p.kb = (int)div_up(width, BK);
        p.splits = 1;
        p.mt2 = p.nt2 = 0;
        if ((st = launch_gemm<K_P>(p, m, tn, s)) != GDN_OK) return st;
        if (loss) {
            hot_kernel<<<grid_for(T), 256, 0, s>>>(dloss, loss, targets, wide, scale, T, v0, cols,
                                                   dtype == GDN_F32 ? p.pa : nullptr, ws + l.p, l.piece, p.lo);
            if ((st = check_launch("hot_kernel")) != GDN_OK) return st;
        }
        // both gradients' products
        if ((st = make_map3(&m.a, P, l.piece, cols, T, parts, HALF)) != GDN_OK) return st;
        if ((st = make_map_rows(&m.b, wp, Wt.ld, width, cols, vocab, parts, 64)) != GDN_OK) return st;
        if ((st = make_map3(&m.a2, P, l.piece, cols, T, parts, 64)) != GDN_OK) return st;
        if ((st = make_map3(&m.b2, Hw.base, Hw.ld, width, T, parts, 64)) != GDN_OK) return st;
        char* dwp = static_cast<char*>(dw) + e * (int64_t)v0 * lddw;
        if (store && (st = make_map_rows(&m.out, dwp, lddw, width, cols, cols, 1, HALF, SC)) != GDN_OK) return st;
        p.nt = (int)div_up(width, BN);
        p.kb = (int)div_up(cols, BK);
        // (the last piece may be done with fewer splits than there are sums)
        p.kper = (int)div_up(p.kb, l.splits);
        p.splits = (int)div_up(p.kb, p.kper);
        p.mt2 = (int)div_up(cols, rows_of_tile(T));
        p.nt2 = p.nt;
        p.kb2 = (int)div_up(T, BK);
        p.acc = reinterpret_cast<float*>(ws + l.acc);
        p.ldacc = l.ldacc;
        p.add = v0 > 0;
        p.dw = dwp; p.lddw = lddw; p.dw_store = store;
        if ((st = launch_gemm<K_GRAD>(p, m, BN, s)) != GDN_OK) return st;
    }
    const unsigned g = grid_for((int64_t)T * (l.ldacc / 8));
    // 16-byte accesses of dh and, in bf16, of w
    const int vec = width % 8 == 0 && (reinterpret_cast<uintptr_t>(dh) & 15u) == 0 && lddh % 8 == 0;
    if (dtype == GDN_F32)
        dh_kernel<float><<<g, 256, 0, s>>>(p.acc, l.splits, T, width, l.ldacc, nullptr, targets, wide, vocab,
                                           static_cast<const float*>(w), ldw, p.most, static_cast<float*>(dh), lddh, vec);
    else
        dh_kernel<__nv_bfloat16><<<g, 256, 0, s>>>(p.acc, l.splits, T, width, l.ldacc, p.lo, targets, wide, vocab,
                                                   static_cast<const __nv_bfloat16*>(w), ldw, nullptr,
                                                   static_cast<__nv_bfloat16*>(dh), lddh, vec);
    return check_launch("dh_kernel");
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_vocab_loss_fwd_workspace_size(int32_t T, int32_t vocab, int32_t width, gdn_dtype dtype) {
    return loss_sizes_ok(T, vocab, width, dtype) ? plan(T, vocab, width, dtype, false).total : 0;
}
size_t gdn_vocab_loss_bwd_workspace_size(int32_t T, int32_t vocab, int32_t width, gdn_dtype dtype) {
    return loss_sizes_ok(T, vocab, width, dtype) ? plan(T, vocab, width, dtype, true).total : 0;
}

gdn_status gdn_vocab_loss_fwd(const void* h, int64_t ldh, const void* w, int64_t ldw, gdn_dtype dtype,
                              const void* targets, int32_t index_bits, int32_t T, int32_t vocab, int32_t width,
                              float scale, float* loss, float* lse, void* workspace, size_t workspace_bytes,
                              void* stream) {
    gdn_status st = check_loss(dtype, index_bits, T, vocab, width, h, ldh, w, ldw, targets, scale);
    if (st != GDN_OK) return st;
    const Plan l = plan(T, vocab, width, dtype, false);
    if ((st = check_ws(workspace, workspace_bytes, l.total)) != GDN_OK) return st;
    if (T == 0) return GDN_OK;
    if (!loss || !lse) return fail(GDN_ERR_INVALID_ARG, "loss or lse is NULL");
    cudaStream_t s = (cudaStream_t)stream;
    char* ws = static_cast<char*>(workspace);
    const int wide = index_bits == 64, parts = dtype == GDN_F32 ? 2 : 1;
    if (l.few) {
        float2* stat = reinterpret_cast<float2*>(ws + l.stat);
        float* at = reinterpret_cast<float*>(ws + l.at);
        if ((st = few_logits({h, ldh, w, ldw, dtype, targets, wide, T, vocab, width, scale}, stat, at, s)) != GDN_OK)
            return st;
        lse_join_kernel<<<(unsigned)div_up(T, 32), 256, 0, s>>>(stat, few_blocks(T, vocab), T, vocab, at, targets, wide,
                                                                loss, lse);
        return check_launch("lse_join_kernel");
    }
    Operand H{h, ldh}, Wt{w, ldw};
    if (!direct(dtype, width)) {
        H = {ws + l.h, round8(width)};
        Wt = {ws + l.w, round8(width)};
        if (dtype == GDN_F32) {
            const int ld = round8(width);
            const int64_t wave = (int64_t)device_sm_count() * 8, n = div_up((int64_t)T + vocab, 8);
            split_rows_kernel<<<(unsigned)(n < wave ? n : wave), 256, 0, s>>>(
                static_cast<const float*>(h), ldh, T, static_cast<const float*>(w), ldw, vocab, width, ld,
                reinterpret_cast<int*>(ws + l.he), reinterpret_cast<int*>(ws + l.we), reinterpret_cast<__half*>(ws + l.h),
                reinterpret_cast<__half*>(ws + l.w));
            st = check_launch("split_rows_kernel");
        } else {
            st = pack(h, ldh, T, w, ldw, vocab, width, nullptr, 0, nullptr, 0, nullptr, ws + l.h, ws + l.w, s);
        }
        if (st != GDN_OK) return st;
    }
    Maps m{};
    if ((st = make_map3(&m.a, H.base, H.ld, width, T, parts, HALF)) != GDN_OK) return st;
    const int tn = tile_cols(T, vocab);
    if ((st = make_map3(&m.b, Wt.base, Wt.ld, width, vocab, parts, copy_rows(T, tn))) != GDN_OK) return st;
    GemmParams p{};
    p.mt = (int)div_up(T, rows_of_tile(T));
    p.nt = (int)div_up(vocab, tn);
    p.group = group_rows(p.mt, width, parts);
    p.kb = (int)div_up(width, BK);
    p.f32 = parts == 2;
    p.T = T; p.V = p.vocab = vocab; p.W = width; p.scale = scale;
    p.targets = targets; p.wide = wide;
    p.he = reinterpret_cast<int*>(ws + l.he);
    p.we = reinterpret_cast<int*>(ws + l.we);
    p.stat = reinterpret_cast<float2*>(ws + l.stat);
    p.at = reinterpret_cast<float*>(ws + l.at);
    if ((st = launch_gemm<K_LSE>(p, m, tn, s)) != GDN_OK) return st;
    lse_join_kernel<<<(unsigned)div_up(T, 32), 256, 0, s>>>(p.stat, p.nt, T, vocab, p.at, targets, wide, loss, lse);
    return check_launch("lse_join_kernel");
}

gdn_status gdn_vocab_loss_bwd(const float* dloss, const void* h, int64_t ldh, const void* w, int64_t ldw,
                              gdn_dtype dtype, const void* targets, int32_t index_bits, const float* lse, int32_t T,
                              int32_t vocab, int32_t width, float scale, void* dh, int64_t lddh, void* dw, int64_t lddw,
                              void* workspace, size_t workspace_bytes, void* stream) {
    return loss_bwd(dloss, h, ldh, w, ldw, dtype, targets, index_bits, nullptr, lse, T, vocab, width, scale, dh, lddh, dw,
                    lddw, workspace, workspace_bytes, stream);
}

gdn_status gdn_vocab_loss_bwd_from_loss(const float* dloss, const void* h, int64_t ldh, const void* w, int64_t ldw,
                                        gdn_dtype dtype, const void* targets, int32_t index_bits, const float* loss,
                                        const float* lse, int32_t T, int32_t vocab, int32_t width, float scale, void* dh,
                                        int64_t lddh, void* dw, int64_t lddw, void* workspace, size_t workspace_bytes,
                                        void* stream) {
    if (T > 0 && !loss) return fail(GDN_ERR_INVALID_ARG, "loss is NULL");
    return loss_bwd(dloss, h, ldh, w, ldw, dtype, targets, index_bits, loss, lse, T, vocab, width, scale, dh, lddh, dw,
                    lddw, workspace, workspace_bytes, stream);
}

}  // extern "C"
