// Embedding lookup with a scale, and its gradient by sorted tokens.
//
//   y_t = scale table[token_t]           dtable[v] = scale sum_{t : token_t = v} dy_t
//
// A token outside [0, vocab) is a padded one: a row of zeros, and no gradient.
//
// The lookup is a copy of rows; what bounds it is DRAM.
//
// The gradient sorts the tokens' positions by token (a stable radix sort, so that a
// token's rows are added in their order and equal calls give equal bits), walks the
// sorted rows in pieces of `piece` rows, and fills the rows of tokens that do not occur
// with zeros.  A piece adds up the rows of one token after the other in registers, its
// loads ahead; a token whose rows go on into the next piece and end there is its too.
// Longer ones are left in parts, which go to the workspace in fp32 and are added, in the
// pieces' order, by a second launch, so that a token that fills a twentieth of a batch
// costs no more than the others.  What bounds it: dy read once, the table's gradient
// written once.
#include "ssm_common.cuh"

namespace gdn {
namespace {

// ---- vectors ---------------------------------------------------------------

// VEC consecutive elements: 8 (bf16) or 4 (fp32) in 16-byte accesses, or one
template <typename E, int VEC> struct Vec;
template <> struct Vec<__nv_bfloat16, 8> {
    using raw = uint4;
    static __device__ __forceinline__ void to_f(const uint4& r, float (&f)[8]) {
        const unsigned w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 from_f(const float (&f)[8]) {
        uint4 r;
        __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&r);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        return r;
    }
    static __device__ __forceinline__ void store(uint4* p, const uint4& r) { __stcs(p, r); }
};
template <> struct Vec<float, 4> {
    using raw = float4;
    static __device__ __forceinline__ void to_f(const float4& r, float (&f)[4]) {
        f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w;
    }
    static __device__ __forceinline__ float4 from_f(const float (&f)[4]) { return make_float4(f[0], f[1], f[2], f[3]); }
    static __device__ __forceinline__ void store(float4* p, const float4& r) { __stcs(p, r); }
};
template <> struct Vec<__nv_bfloat16, 1> {
    using raw = __nv_bfloat16;
    static __device__ __forceinline__ void to_f(raw r, float (&f)[1]) { f[0] = __bfloat162float(r); }
    static __device__ __forceinline__ raw from_f(const float (&f)[1]) { return __float2bfloat16_rn(f[0]); }
    static __device__ __forceinline__ void store(raw* p, raw r) { *p = r; }
};
template <> struct Vec<float, 1> {
    using raw = float;
    static __device__ __forceinline__ void to_f(raw r, float (&f)[1]) { f[0] = r; }
    static __device__ __forceinline__ raw from_f(const float (&f)[1]) { return f[0]; }
    static __device__ __forceinline__ void store(raw* p, raw r) { __stcs(p, r); }
};

template <typename I>
__device__ __forceinline__ int token_of(const I* tokens, int64_t t, int vocab) {
    const I v = __ldg(tokens + t);
    return v < 0 || v >= (I)vocab ? -1 : (int)v;
}

// ---- lookup ----------------------------------------------------------------

constexpr int FT = 256;  // threads of a block
constexpr int FU = 8;    // accesses of a lane, loaded together

// A warp copies a piece of 32 FU vectors of one row, pieces of a row next to each other.
// The results are written past the cache, which is for the table's frequent rows.
template <typename E, int VEC, typename I>
__global__ void __launch_bounds__(FT) embed_fwd_kernel(const I* __restrict__ tokens, const E* __restrict__ table,
                                                       int64_t ldt, int vocab, int T, int nv, int pieces, float scale,
                                                       E* __restrict__ y, int64_t ldy) {
    using V = Vec<E, VEC>;
    using R = typename V::raw;
    const unsigned at = blockIdx.x * (FT / 32) + (threadIdx.x >> 5);
    const unsigned t = at / (unsigned)pieces, piece = at - t * (unsigned)pieces;
    if (t >= (unsigned)T) return;
    const int first = (int)piece * (32 * FU) + (threadIdx.x & 31);
    const int v = token_of(tokens, t, vocab);
    R* const out = reinterpret_cast<R*>(y + t * ldy);
    if (v < 0) {
        float f[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] = 0.f;
#pragma unroll
        for (int u = 0; u < FU; ++u)
            if (first + 32 * u < nv) V::store(out + first + 32 * u, V::from_f(f));
        return;
    }
    const R* const row = reinterpret_cast<const R*>(table + v * ldt);
    R r[FU];
#pragma unroll
    for (int u = 0; u < FU; ++u)
        if (first + 32 * u < nv) r[u] = __ldg(row + first + 32 * u);
#pragma unroll
    for (int u = 0; u < FU; ++u) {
        if (first + 32 * u >= nv) continue;
        float f[VEC];
        V::to_f(r[u], f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] *= scale;
        V::store(out + first + 32 * u, V::from_f(f));
    }
}

// ---- rows of zeros ---------------------------------------------------------

constexpr int kMaxPiece = 256;  // rows of a piece
constexpr int kMaxZero = 64;    // rows filled by a block

// zeros, in 16-byte accesses but for the ends, by NT threads of which this is number i0
template <typename E, int NT>
__device__ __forceinline__ void fill_zero(E* p, int64_t n, int i0) {
    constexpr int N = 16 / sizeof(E);
    int64_t head = (16 - (int64_t)(reinterpret_cast<uintptr_t>(p) & 15u)) % 16 / (int)sizeof(E);
    if (head > n) head = n;
    for (int64_t i = i0; i < head; i += NT) p[i] = Elem<E>::from_f(0.f);
    p += head;
    n -= head;
    uint4* q = reinterpret_cast<uint4*>(p);
    for (int64_t i = i0; i < n / N; i += NT) __stcs(q + i, make_uint4(0u, 0u, 0u, 0u));
    for (int64_t i = n / N * N + i0; i < n; i += NT) p[i] = Elem<E>::from_f(0.f);
}
// The rows [v0, v1) that do not occur.  Rows of up to a kilobyte a warp each (the gradient of 56666
// tokens in 24322 rows of 127: 114 us by the whole block, 68 so); wider ones by all
// threads, those without a gap between them as one.
template <typename E, int NT, typename F>
__device__ __forceinline__ void fill_rows(E* out, int64_t ldo, int W, int v0, int v1, F occurs) {
    if (W * (int)sizeof(E) <= 1024) {
        for (int v = v0 + (int)threadIdx.x / 32; v < v1; v += NT / 32)
            if (!occurs(v)) fill_zero<E, 32>(out + v * ldo, W, threadIdx.x & 31);
        return;
    }
    for (int v = v0; v < v1;) {
        if (occurs(v)) {
            ++v;
            continue;
        }
        int w = v + 1;
        if (ldo == W)
            while (w < v1 && !occurs(w)) ++w;
        fill_zero<E, NT>(out + v * ldo, (int64_t)(w - v) * W, threadIdx.x);
        v = w;
    }
}

// ---- sort ------------------------------------------------------------------

// Keys are the tokens, `vocab` for a padded one, which ends up behind the others.  A pass
// sorts by up to 9 bits, low ones first: the blocks' counts of digits, then the
// places.  Block b takes the rows [b per, (b + 1) per) of the order so far.
constexpr int SW = 8;               // warps of a block
constexpr int ST = SW * 32;
constexpr int SI = 4;               // rows of a lane in one step
constexpr int STILE = ST * SI;      // rows of a step
constexpr int kBits = 9, kBins = 1 << kBits;
constexpr int kMaxSortBlocks = 128;

struct SortArgs {
    const void* tokens;    // the first pass's input
    const int* key_in; const int* pos_in;
    int* key_out; int* pos_out;
    int* count;            // [blocks][kBins] counts of this pass
    int T, vocab, per, shift, blocks;
    // beside it, rows [v0, v1) of the gradient that no token has are filled with zeros, zrows a
    // block; hit: a byte a token, 1 where it occurs
    unsigned char* hit;
    int v0, v1, zrows, W;
    int64_t ldo;
    void* out;
};

template <typename I>
__device__ __forceinline__ int sort_key(const SortArgs& a, int i) {
    if (a.key_in) return a.key_in[i];
    const int v = token_of(static_cast<const I*>(a.tokens), i, a.vocab);
    return v < 0 ? a.vocab : v;
}

template <typename I>
__global__ void __launch_bounds__(ST) sort_count_kernel(const SortArgs a) {
    __shared__ int hist[kBins];
    for (int i = threadIdx.x; i < kBins; i += ST) hist[i] = 0;
    __syncthreads();
    const int lo = blockIdx.x * a.per, hi = min(a.T, lo + a.per);
    for (int i = lo + threadIdx.x; i < hi; i += ST) {
        const int key = sort_key<I>(a, i);
        atomicAdd(&hist[(key >> a.shift) & (kBins - 1)], 1);
        if (a.hit && key < a.vocab) a.hit[key] = 1;  // (asking first whether it is set: 155 -> 185 us of the whole)
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += ST) a.count[blockIdx.x * kBins + i] = hist[i];
}

// Sum of v over the threads below, for one value a thread; all ST threads
__device__ __forceinline__ int exclusive_sum(int v, int* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, m);
        if (lane >= m) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int w = 0; w < SW; ++w) before += w < warp ? warp_sums[w] : 0;
    __syncthreads();
    return before + x - v;
}

template <typename I, typename E>
__global__ void __launch_bounds__(ST) sort_place_kernel(const SortArgs a) {
    if ((int)blockIdx.x >= a.blocks) {
        __shared__ unsigned char hit[kMaxZero];
        const int v0 = a.v0 + ((int)blockIdx.x - a.blocks) * a.zrows, v1 = min(a.v1, v0 + a.zrows);
        for (int v = v0 + threadIdx.x; v < v1; v += ST) hit[v - v0] = a.hit[v];
        __syncthreads();
        fill_rows<E, ST>(static_cast<E*>(a.out), a.ldo, a.W, v0, v1, [&](int v) { return hit[v - v0] != 0; });
        return;
    }
    __shared__ int base[kBins];       // where this block's next row of a digit goes
    __shared__ int wc[SW][kBins];     // a warp's rows of a digit in this step, then where they begin
    __shared__ int warp_sums[SW];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // rows of smaller digits anywhere, and of the same digit in the blocks before
    {
        int all[kBins / ST], mine[kBins / ST], sum = 0;
#pragma unroll
        for (int j = 0; j < kBins / ST; ++j) {
            const int d = tid * (kBins / ST) + j;
            all[j] = mine[j] = 0;
#pragma unroll 16
            for (int b = 0; b < a.blocks; ++b) {
                const int c = __ldg(a.count + b * kBins + d);
                all[j] += c;
                mine[j] += b < (int)blockIdx.x ? c : 0;
            }
            sum += all[j];
        }
        int at = exclusive_sum(sum, warp_sums);
#pragma unroll
        for (int j = 0; j < kBins / ST; ++j) {
            base[tid * (kBins / ST) + j] = at + mine[j];
            at += all[j];
        }
    }
    const int lo = blockIdx.x * a.per, hi = min(a.T, lo + a.per);
    for (int t0 = lo; t0 < hi; t0 += STILE) {
        for (int i = lane; i < kBins; i += 32) wc[warp][i] = 0;
        __syncwarp();
        int key[SI], pos[SI], rank[SI];
#pragma unroll
        for (int j = 0; j < SI; ++j) {
            const int i = t0 + warp * (32 * SI) + j * 32 + lane;
            key[j] = i < hi ? sort_key<I>(a, i) : -1;
            pos[j] = i < hi ? (a.pos_in ? a.pos_in[i] : i) : 0;
        }
#pragma unroll
        for (int j = 0; j < SI; ++j) {
            const int d = key[j] < 0 ? kBins : (key[j] >> a.shift) & (kBins - 1);
            const unsigned same = __match_any_sync(0xffffffffu, d);
            const int before = d < kBins ? wc[warp][d] : 0;
            rank[j] = before + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (d < kBins && lane == __ffs(same) - 1) wc[warp][d] = before + __popc(same);
            __syncwarp();
        }
        __syncthreads();
        for (int d = tid; d < kBins; d += ST) {  // where each warp's rows of digit d begin
            int at = base[d];
#pragma unroll
            for (int w = 0; w < SW; ++w) {
                const int c = wc[w][d];
                wc[w][d] = at;
                at += c;
            }
            base[d] = at;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < SI; ++j)
            if (key[j] >= 0) {
                const int to = wc[warp][(key[j] >> a.shift) & (kBins - 1)] + rank[j];
                a.key_out[to] = key[j];
                a.pos_out[to] = pos[j];
            }
        __syncwarp();  // a warp clears only its own counts
    }
}

// Up to SMALL rows: every pass in one block, keys and positions in shared memory
constexpr int SMALL_I = 16, SMALL = ST * SMALL_I;

template <typename I>
__global__ void __launch_bounds__(ST) sort_small_kernel(const SortArgs a, int bits) {
    __shared__ int wc[SW][kBins];
    __shared__ int key_s[SMALL];
    __shared__ unsigned short pos_s[SMALL];
    __shared__ int warp_sums[SW];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // a warp has the rows [warp per, (warp + 1) per) of the order so far, 32 after 32
    const int rounds = (a.T + ST - 1) / ST, first = warp * rounds * 32 + lane;
    for (int i = tid; i < a.T; i += ST) {
        key_s[i] = sort_key<I>(a, i);
        pos_s[i] = (unsigned short)i;
    }
    __syncthreads();
    for (int shift = 0; shift < bits; shift += kBits) {
        int key[SMALL_I], pos[SMALL_I], rank[SMALL_I];
        for (int i = lane; i < kBins; i += 32) wc[warp][i] = 0;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < SMALL_I; ++j) {
            if (j >= rounds) break;
            const int i = first + j * 32;
            key[j] = i < a.T ? key_s[i] : -1;
            pos[j] = i < a.T ? pos_s[i] : 0;
            const int d = key[j] < 0 ? kBins : (key[j] >> shift) & (kBins - 1);
            const unsigned same = __match_any_sync(0xffffffffu, d);
            const int before = d < kBins ? wc[warp][d] : 0;
            rank[j] = before + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (d < kBins && lane == __ffs(same) - 1) wc[warp][d] = before + __popc(same);
            __syncwarp();
        }
        __syncthreads();
        {
            int total[kBins / ST], sum = 0;
#pragma unroll
            for (int j = 0; j < kBins / ST; ++j) {
                const int d = tid * (kBins / ST) + j;
                total[j] = 0;
#pragma unroll
                for (int w = 0; w < SW; ++w) total[j] += wc[w][d];
                sum += total[j];
            }
            int at = exclusive_sum(sum, warp_sums);
#pragma unroll
            for (int j = 0; j < kBins / ST; ++j) {
                const int d = tid * (kBins / ST) + j;
                int next = at;
#pragma unroll
                for (int w = 0; w < SW; ++w) {
                    const int c = wc[w][d];
                    wc[w][d] = next;
                    next += c;
                }
                at += total[j];
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < SMALL_I; ++j)
            if (j < rounds && key[j] >= 0) {
                const int to = wc[warp][(key[j] >> shift) & (kBins - 1)] + rank[j];
                key_s[to] = key[j];
                pos_s[to] = (unsigned short)pos[j];
            }
        __syncthreads();
    }
    for (int i = tid; i < a.T; i += ST) {
        a.key_out[i] = key_s[i];
        a.pos_out[i] = pos_s[i];
    }
}

// ---- sums of sorted rows ---------------------------------------------------

constexpr int PT = 128;       // threads of a block; each has U vectors of a row, PT vectors apart
struct SumArgs {
    const int* key; const int* pos;
    int T, vocab, W, piece, pieces, zrows;
    int64_t lddy, ldo;
    const void* dy;
    float scale;
    void* out;
    int into;           // add to what is there
    float* part;        // [pieces][2][W]: a piece's first token's part, its last one's
};

// first i in [0, T) with key[i] >= v, T if there is none; a whole warp, 32 places a step
__device__ __forceinline__ int first_at(const int* key, int T, int v) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = T;  // the answer lies in [lo, lo + n]
    while (n > 0) {
        const int step = n / 33 + 1;  // n + 1 answers in 33 runs; lane l looks at lo + (l + 1) step - 1
        const int i = lo + (lane + 1) * step - 1;
        const bool below = i < lo + n && __ldg(key + i) < v;
        const int c = __popc(__ballot_sync(0xffffffffu, below));  // the first c places are below v
        const int end = lo + n;
        lo += c * step;
        n = min(step - 1, end - lo);
    }
    return lo;
}

// one vector of columns of row v
template <typename E, int VEC>
__device__ __forceinline__ void put(const SumArgs& a, int v, int c, const float (&acc)[VEC]) {
    using V = Vec<E, VEC>;
    typename V::raw* o = reinterpret_cast<typename V::raw*>(static_cast<E*>(a.out) + v * a.ldo + c);
    float f[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = acc[j] * a.scale;
    if (a.into) {
        float old[VEC];
        V::to_f(*o, old);
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] += old[j];
    }
    V::store(o, V::from_f(f));
}

template <int VEC>
__device__ __forceinline__ void put_part(float* w, const float (&acc)[VEC]) {
    if constexpr (VEC == 1) {
        *w = acc[0];
    } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 4)
            *reinterpret_cast<float4*>(w + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
    }
}
template <int VEC>
__device__ __forceinline__ void add_part(const float* w, float (&acc)[VEC]) {
    if constexpr (VEC == 1) {
        acc[0] += *w;
    } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 4) {
            const float4 x = *reinterpret_cast<const float4*>(w + j);
            acc[j] += x.x; acc[j + 1] += x.y; acc[j + 2] += x.z; acc[j + 3] += x.w;
        }
    }
}

// Whether the token v, whose rows go on over the start r of a piece, is added up by the
// piece that it begins in: it begins in the one before r and ends in the one behind.
// Longer ones are left in parts.
__device__ __forceinline__ bool one_piece_has(const SumArgs& a, int v, int r) {
    return (r - a.piece - 1 < 0 || __ldg(a.key + r - a.piece - 1) != v) &&
           (r + a.piece >= a.T || __ldg(a.key + r + a.piece) != v);
}

// Blocks [0, pieces ny) add up the rows of a piece's tokens, PT * U vectors of columns
// each; the others fill the rows of tokens that do not occur, zrows each.
template <typename E, int VEC, int U>
__global__ void __launch_bounds__(PT) embed_sum_kernel(const SumArgs a, int ny) {
    using V = Vec<E, VEC>;
    using R = typename V::raw;
    if ((int)blockIdx.x >= a.pieces * ny) {
        __shared__ unsigned hit[kMaxZero / 32];
        __shared__ int range[2];
        const int v0 = ((int)blockIdx.x - a.pieces * ny) * a.zrows, v1 = min(a.vocab, v0 + a.zrows);
        if (threadIdx.x < kMaxZero / 32) hit[threadIdx.x] = 0;
        if (threadIdx.x < 64) {
            const int i = first_at(a.key, a.T, threadIdx.x < 32 ? v0 : v1);
            if ((threadIdx.x & 31) == 0) range[threadIdx.x >> 5] = i;
        }
        __syncthreads();
        const int lo = range[0], hi = range[1];
        // a token's rows lie together: only its first one counts
        for (int i = lo + threadIdx.x; i < hi; i += PT) {
            const int v = __ldg(a.key + i);
            if (i == lo || __ldg(a.key + i - 1) != v) atomicOr(&hit[(v - v0) >> 5], 1u << ((v - v0) & 31));
        }
        __syncthreads();
        fill_rows<E, PT>(static_cast<E*>(a.out), a.ldo, a.W, v0, v1,
                         [&](int v) { return (hit[(v - v0) >> 5] >> ((v - v0) & 31) & 1u) != 0; });
        return;
    }
    const int piece = blockIdx.x / ny, c0 = ((blockIdx.x - piece * ny) * U * PT + threadIdx.x) * VEC;  // vector u: + u PT VEC
    __shared__ int key[2 * kMaxPiece + 1];  // with the rows of the next piece, where the last token may end
    __shared__ int pos[2 * kMaxPiece];
    __shared__ int ends[2];
    const int r0 = piece * a.piece, r1 = min(a.T, r0 + a.piece), rmax = min(a.T, r1 + a.piece);
    for (int i = threadIdx.x; i <= rmax - r0; i += PT) {
        key[i] = r0 + i < rmax ? __ldg(a.key + r0 + i) : -1;
        if (r0 + i < rmax) pos[i] = __ldg(a.pos + r0 + i);
    }
    if (threadIdx.x == 0) {
        const int v = __ldg(a.key + r0);
        // 0: a token begins here; 1: the piece before has the first one; 2: it is left in parts
        ends[0] = r0 == 0 || __ldg(a.key + r0 - 1) != v ? 0 : one_piece_has(a, v, r0) ? 1 : 2;
    } else if (threadIdx.x == 32) {
        const int v = __ldg(a.key + r1 - 1);
        ends[1] = r1 == a.T || __ldg(a.key + r1) != v ? 0 : one_piece_has(a, v, r1) ? 1 : 2;
    }
    __syncthreads();
    if (c0 >= a.W) return;
    int i0 = 0, n = r1 - r0;
    if (ends[0] == 1) {
        const int v = key[0];
        while (i0 < n && key[i0] == v) ++i0;
        if (i0 == n) return;
    }
    if (ends[1] == 1) {
        const int v = key[n - 1];
        while (key[n] == v) ++n;
    }
    const E* dy = static_cast<const E*>(a.dy) + c0;
    constexpr int AHEAD = 8;
    R row[AHEAD][U];
    auto load = [&](int slot, int i) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (U == 1 || c0 + u * PT * VEC < a.W)
                row[slot][u] = __ldg(reinterpret_cast<const R*>(dy + pos[i] * a.lddy + u * PT * VEC));
    };
#pragma unroll
    for (int s = 0; s < AHEAD; ++s)
        if (i0 + s < n && key[i0 + s] < a.vocab) load(s, i0 + s);
    float acc[U][VEC];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[u][j] = 0.f;
    bool whole = ends[0] != 2;  // all rows of the token are added up here
    for (; i0 < n; i0 += AHEAD) {
#pragma unroll
        for (int s = 0; s < AHEAD; ++s) {
            const int i = i0 + s;
            if (i >= n) break;
            const int v = key[i];
            if (v >= a.vocab) return;  // padded tokens are behind all others
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[VEC];
                V::to_f(row[s][u], f);
#pragma unroll
                for (int j = 0; j < VEC; ++j) acc[u][j] += f[j];
            }
            const int nx = i + AHEAD;
            if (nx < n && key[nx] < a.vocab) load(s, nx);
            const bool last = key[i + 1] != v;
            if (last || i == n - 1) {
                // its sum, or its part in this piece: the first one's, or the last one's that goes on
                float* const part = a.part + ((int64_t)piece * 2 + (last ? 0 : 1)) * a.W + c0;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (U == 1 || c0 + u * PT * VEC < a.W) {
                        if (last && whole) put<E, VEC>(a, v, c0 + u * PT * VEC, acc[u]);
                        else put_part<VEC>(part + u * PT * VEC, acc[u]);
                    }
#pragma unroll
                    for (int j = 0; j < VEC; ++j) acc[u][j] = 0.f;
                }
                whole = true;
            }
        }
    }
}

// Adds up the tokens that are left in parts: the one that begins in piece b, if it goes on
// over more than the next piece, is the sum of the last parts of piece b and of the pieces
// that it fills and the first part of the one that it ends in (where it fills that too, it
// ends there all the same).  A block looks at every gridDim.x-th piece, 32 at a time: few
// have such a token.  JG groups of threads take a run of the parts each; their sums are
// added in the runs' order.
constexpr int JG = 4;

template <typename E, int VEC>
__global__ void __launch_bounds__(PT * JG, 2) embed_join_kernel(const SumArgs a) {
    __shared__ float sum[JG - 1][PT][VEC];
    __shared__ unsigned found;
    const int x = threadIdx.x % PT, g = threadIdx.x / PT;
    const int c = (blockIdx.y * PT + x) * VEC;
    for (int64_t b0 = blockIdx.x; b0 < a.pieces - 1; b0 += 32ll * gridDim.x) {
        if (threadIdx.x < 32) {
            const int64_t b = b0 + (int64_t)threadIdx.x * gridDim.x;
            bool parts = false;
            if (b < a.pieces - 1) {
                const int r = (int)(b + 1) * a.piece, v = __ldg(a.key + r);  // the next piece's start
                parts = v < a.vocab && __ldg(a.key + r - 1) == v && !one_piece_has(a, v, r) &&
                        (b == 0 || __ldg(a.key + r - a.piece - 1) != v);
            }
            const unsigned m = __ballot_sync(0xffffffffu, parts);
            if (threadIdx.x == 0) found = m;
        }
        __syncthreads();
        for (unsigned m = found; m; m &= m - 1) {
            const int b = (int)(b0 + (int64_t)(__ffs(m) - 1) * gridDim.x);
            const int v = __ldg(a.key + (b + 1) * a.piece);
            const int end = first_at(a.key, a.T, v + 1);  // behind the token's last row
            const int pe = (end - 1) / a.piece;           // the piece that it ends in
            const int n = pe - b + 1, per = (n + JG - 1) / JG;  // parts, of a group
            float acc[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) acc[j] = 0.f;
            if (c < a.W) {
                const int i1 = min(n, (g + 1) * per);
#pragma unroll 4
                for (int i = g * per; i < i1; ++i)
                    add_part<VEC>(a.part + ((int64_t)(b + i) * 2 + (i < n - 1 ? 1 : 0)) * a.W + c, acc);
            }
            if (g) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) sum[g - 1][x][j] = acc[j];
            }
            __syncthreads();
            if (!g && c < a.W) {
#pragma unroll
                for (int k = 0; k < JG - 1; ++k)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) acc[j] += sum[k][x][j];
                put<E, VEC>(a, v, c, acc);
            }
            __syncthreads();
        }
        __syncthreads();
    }
}

// ---- host ------------------------------------------------------------------

int sort_blocks(int64_t T) {
    const int64_t n = (T + STILE - 1) / STILE;
    return (int)(n < 1 ? 1 : n > kMaxSortBlocks ? kMaxSortBlocks : n);
}
// Rows of a piece: enough pieces for the GPU, and few parts of a token that fills many
constexpr int kPieces = 2048;
int piece_rows(int64_t T) {
    int p = 16;
    while (p < kMaxPiece && T / p > kPieces) p *= 2;
    return p;
}
size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

struct Layout {
    size_t key[2], pos[2], count, part, hit, total;
};
Layout layout(int64_t T, int W, int vocab) {
    Layout l{};
    size_t at = 0;
    const size_t row = round256(4 * (size_t)T);
    for (int i = 0; i < 2; ++i) {
        l.key[i] = at; at += row;
        l.pos[i] = at; at += row;
    }
    l.count = at; at += round256(sizeof(int) * (size_t)kMaxSortBlocks * kBins);
    // the most pieces of any call of up to T rows
    int64_t pieces = (T + 15) / 16;
    if (pieces > kPieces + 1) pieces = kPieces + 1;
    if (pieces < T / kMaxPiece + 1) pieces = T / kMaxPiece + 1;
    l.part = at; at += round256(sizeof(float) * 2 * (size_t)pieces * W);
    l.hit = at; at += round256((size_t)vocab);
    l.total = at;
    return l;
}

// Sorts, and for more than SMALL tokens fills the rows that do not occur: a share beside
// each pass, whose few blocks leave the GPU to it (65536 tokens into 131072 rows of 2048:
// 183 us with the filling beside the sums, 155 so).
template <typename I, typename E>
gdn_status sort_tokens(const void* tokens, const SumArgs& sum, char* ws, const Layout& l, int& which, bool& filled,
                       cudaStream_t s) {
    const int T = sum.T, vocab = sum.vocab;
    int bits = 1;
    while (bits < 31 && ((int64_t)1 << bits) <= vocab) ++bits;  // keys up to vocab
    SortArgs a{};
    a.tokens = tokens;
    a.T = T;
    a.vocab = vocab;
    filled = false;
    which = 0;
    if (T <= SMALL) {
        a.key_out = reinterpret_cast<int*>(ws + l.key[0]);
        a.pos_out = reinterpret_cast<int*>(ws + l.pos[0]);
        sort_small_kernel<I><<<1, ST, 0, s>>>(a, bits);
        return check_launch("sort_small_kernel");
    }
    a.blocks = sort_blocks(T);
    a.per = (T + a.blocks - 1) / a.blocks;
    a.count = reinterpret_cast<int*>(ws + l.count);
    const int passes = (bits + kBits - 1) / kBits;
    if (!sum.into) {
        filled = true;
        a.hit = reinterpret_cast<unsigned char*>(ws + l.hit);
        a.zrows = sum.zrows; a.W = sum.W; a.ldo = sum.ldo; a.out = sum.out;
        if (cudaMemsetAsync(a.hit, 0, vocab, s) != cudaSuccess) return check_launch("memset");
    }
    for (int p = 0; p < passes; ++p) {
        a.shift = p * kBits;
        a.key_out = reinterpret_cast<int*>(ws + l.key[which]);
        a.pos_out = reinterpret_cast<int*>(ws + l.pos[which]);
        sort_count_kernel<I><<<a.blocks, ST, 0, s>>>(a);
        int fill = 0;
        if (filled) {
            a.v0 = (int)((int64_t)vocab * p / passes);
            a.v1 = (int)((int64_t)vocab * (p + 1) / passes);
            fill = (a.v1 - a.v0 + a.zrows - 1) / a.zrows;
        }
        sort_place_kernel<I, E><<<a.blocks + fill, ST, 0, s>>>(a);
        a.key_in = a.key_out;
        a.pos_in = a.pos_out;
        which ^= 1;
    }
    which ^= 1;
    return check_launch("sort kernels");
}

template <typename E, int VEC>
gdn_status run_sum(const SumArgs& a, bool filled, cudaStream_t s) {
    // single elements: eight of a thread, or the blocks would be small
    constexpr int U = VEC == 1 ? 8 : 1;
    const unsigned ny = (unsigned)((a.W + PT * VEC * U - 1) / (PT * VEC * U));
    const int64_t blocks = (int64_t)a.pieces * ny + (a.into || filled ? 0 : (a.vocab + a.zrows - 1) / a.zrows);
    if (blocks > 0x7fffffff) return fail(GDN_ERR_UNSUPPORTED_SHAPE, "T=%d rows of %d elements", a.T, a.W);
    if (blocks > 0) {
        embed_sum_kernel<E, VEC, U><<<(unsigned)blocks, PT, 0, s>>>(a, (int)ny);
        gdn_status st = check_launch("embed_sum_kernel");
        if (st != GDN_OK) return st;
    }
    if (a.pieces > 1) {
        const int most = 2 * device_sm_count();
        embed_join_kernel<E, VEC><<<dim3(a.pieces - 1 < most ? a.pieces - 1 : most, (a.W + PT * VEC - 1) / (PT * VEC)),
                                    PT * JG, 0, s>>>(a);
        return check_launch("embed_join_kernel");
    }
    return GDN_OK;
}

bool al(const void* p, int64_t ld, size_t e) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * (int64_t)e) % 16 == 0;
}

template <typename E, int VEC, typename I>
gdn_status run_fwd_i(const void* tokens, const void* table, int64_t ldt, int vocab, int T, int W, float scale, void* y,
                     int64_t ldy, cudaStream_t s) {
    const int nv = W / VEC, pieces = (nv + 32 * FU - 1) / (32 * FU);
    const int64_t warps = (int64_t)T * pieces;
    if (warps > 0xfffffff0ll) return fail(GDN_ERR_UNSUPPORTED_SHAPE, "T=%d rows of %d elements", T, W);
    embed_fwd_kernel<E, VEC, I><<<(unsigned)((warps + FT / 32 - 1) / (FT / 32)), FT, 0, s>>>(
        static_cast<const I*>(tokens), static_cast<const E*>(table), ldt, vocab, T, nv, pieces, scale,
        static_cast<E*>(y), ldy);
    return check_launch("embed_fwd_kernel");
}
template <typename E, int VEC>
gdn_status run_fwd(int wide, const void* tokens, const void* table, int64_t ldt, int vocab, int T, int W, float scale,
                   void* y, int64_t ldy, cudaStream_t s) {
    return wide ? run_fwd_i<E, VEC, int64_t>(tokens, table, ldt, vocab, T, W, scale, y, ldy, s)
                : run_fwd_i<E, VEC, int32_t>(tokens, table, ldt, vocab, T, W, scale, y, ldy, s);
}

gdn_status check_embed(gdn_dtype dtype, int32_t index_bits, int T, int W, int vocab, const void* tokens) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return fail(GDN_ERR_DTYPE, "unknown dtype %d", (int)dtype);
    if (index_bits != 32 && index_bits != 64) return fail(GDN_ERR_DTYPE, "tokens of %d bits", index_bits);
    if (T < 0 || W < 1 || vocab < 0) return fail(GDN_ERR_INVALID_ARG, "T=%d width=%d vocab=%d", T, W, vocab);
    if (T > kMaxTokens) return fail(GDN_ERR_UNSUPPORTED_SHAPE, "%d tokens, more than %d", T, kMaxTokens);
    if (W > (1 << 20)) return fail(GDN_ERR_UNSUPPORTED_SHAPE, "width=%d above 2^20", W);
    if (vocab > (1 << 30)) return fail(GDN_ERR_UNSUPPORTED_SHAPE, "vocab=%d above 2^30", vocab);
    if (T > 0 && !tokens) return fail(GDN_ERR_INVALID_ARG, "tokens is NULL");
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_embed_fwd(const void* tokens, int32_t index_bits, const void* table, int64_t ldt, gdn_dtype dtype,
                         int32_t vocab, int32_t T, int32_t width, float scale, void* y, int64_t ldy, void* stream) {
    gdn_status st = check_embed(dtype, index_bits, T, width, vocab, tokens);
    if (st != GDN_OK) return st;
    if (T == 0) return GDN_OK;
    if (!y || (vocab > 0 && !table)) return fail(GDN_ERR_INVALID_ARG, "table or y is NULL");
    if (ldt < width || ldy < width)
        return fail(GDN_ERR_INVALID_ARG, "row strides of table and y must be >= width=%d", width);
    cudaStream_t s = (cudaStream_t)stream;
    const int w64 = index_bits == 64;
    if (dtype == GDN_BF16)
        return width % 8 == 0 && al(table, ldt, 2) && al(y, ldy, 2)
                   ? run_fwd<__nv_bfloat16, 8>(w64, tokens, table, ldt, vocab, T, width, scale, y, ldy, s)
                   : run_fwd<__nv_bfloat16, 1>(w64, tokens, table, ldt, vocab, T, width, scale, y, ldy, s);
    return width % 4 == 0 && al(table, ldt, 4) && al(y, ldy, 4)
               ? run_fwd<float, 4>(w64, tokens, table, ldt, vocab, T, width, scale, y, ldy, s)
               : run_fwd<float, 1>(w64, tokens, table, ldt, vocab, T, width, scale, y, ldy, s);
}

size_t gdn_embed_bwd_workspace_size(int32_t T, int32_t vocab, int32_t width) {
    if (T < 0 || T > kMaxTokens || width < 1 || width > (1 << 20) || vocab < 0 || vocab > (1 << 30)) return 0;
    return layout(T, width, vocab).total;
}

gdn_status gdn_embed_bwd(const void* dy, int64_t lddy, gdn_dtype dtype, const void* tokens, int32_t index_bits,
                         int32_t vocab, int32_t T, int32_t width, float scale, int32_t accumulate, void* dtable,
                         int64_t ldd, void* workspace, size_t workspace_bytes, void* stream) {
    gdn_status st = check_embed(dtype, index_bits, T, width, vocab, tokens);
    if (st != GDN_OK) return st;
    if (vocab == 0) return GDN_OK;
    if (!dtable || (T > 0 && !dy)) return fail(GDN_ERR_INVALID_ARG, "dy or dtable is NULL");
    if (ldd < width || (T > 0 && lddy < width))
        return fail(GDN_ERR_INVALID_ARG, "row strides of dy and dtable must be >= width=%d", width);
    const Layout l = layout(T, width, vocab);
    if (!workspace || workspace_bytes < l.total)
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes < required %zu", workspace ? workspace_bytes : 0, l.total);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(GDN_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    cudaStream_t s = (cudaStream_t)stream;
    char* ws = static_cast<char*>(workspace);
    SumArgs a{};
    a.T = T; a.vocab = vocab; a.W = width; a.piece = piece_rows(T);
    a.pieces = (T + a.piece - 1) / a.piece;
    // rows of up to 64 KB together
    const int64_t zrows = (64 << 10) / ((int64_t)width * (dtype == GDN_BF16 ? 2 : 4));
    a.zrows = (int)(zrows < 1 ? 1 : zrows > kMaxZero ? kMaxZero : zrows);
    a.dy = dy; a.lddy = lddy; a.ldo = ldd; a.scale = scale; a.out = dtable; a.into = accumulate != 0;
    a.part = reinterpret_cast<float*>(ws + l.part);
    int which = 0;
    bool filled = false;
    if (T > 0) {
        const bool wide = index_bits == 64;
        if (dtype == GDN_BF16)
            st = wide ? sort_tokens<int64_t, __nv_bfloat16>(tokens, a, ws, l, which, filled, s)
                      : sort_tokens<int32_t, __nv_bfloat16>(tokens, a, ws, l, which, filled, s);
        else
            st = wide ? sort_tokens<int64_t, float>(tokens, a, ws, l, which, filled, s)
                      : sort_tokens<int32_t, float>(tokens, a, ws, l, which, filled, s);
        if (st != GDN_OK) return st;
    }
    a.key = reinterpret_cast<int*>(ws + l.key[which]);
    a.pos = reinterpret_cast<int*>(ws + l.pos[which]);
    if (dtype == GDN_BF16)
        return width % 8 == 0 && al(dy, lddy, 2) && al(dtable, ldd, 2) ? run_sum<__nv_bfloat16, 8>(a, filled, s)
                                                                       : run_sum<__nv_bfloat16, 1>(a, filled, s);
    return width % 4 == 0 && al(dy, lddy, 4) && al(dtable, ldd, 4) ? run_sum<float, 4>(a, filled, s)
                                                                   : run_sum<float, 1>(a, filled, s);
}

}  // extern "C"
