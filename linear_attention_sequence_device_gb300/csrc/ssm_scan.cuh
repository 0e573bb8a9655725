// What the scan's forward and backward share on the host side and at launch.
#pragma once

#include "ssm_common.cuh"

namespace gdn {

constexpr int kCkpt = 8;  // tokens between the forward's checkpoints for the backward

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
    float* h_final; float* ckpt;     // ckpt [ceil(T / kCkpt), ch, N]
    int seg, S;                      // tokens per segment, segments
    float* H; float* sd;             // [S, ch, N], [S, ch]
    bool folded;                     // H's row s - 1 holds the state at segment s's start already
};

// Which part of a segment a scan_kernel launch runs: the outputs; only the end
// state of its part of the sequence that goes on behind it; or, walking the
// tokens backwards, only the gradient that its part of the sequence that came in
// sends to the state before it (x, B and h0 are then dy, C and dh_final).
enum ScanMode : int { SCAN_FULL = 0, SCAN_END = 1, SCAN_START_GRAD = 2 };

// Segments above which the rows of H are folded once by a launch of their own
// instead of by every block for its own channels.
constexpr int kFoldSegments = 4;
gdn_status launch_scan_start_grad(const ScanParams& p, gdn_dtype dtype, int groups, cudaStream_t s);

// argument checks (ssm_scan.cu)
gdn_status check_scan_shape(gdn_dtype dtype, int rows, int ch, int N, int groups);
gdn_status check_scan_row(const void* p, int64_t ld, int64_t least, const char* name);
gdn_status check_scan_inputs(const void* x, int64_t ldx, const void* dt, int64_t lddt, const void* z, int64_t ldz,
                             const void* B, int64_t ldb, const void* C, int64_t ldc, const float* A_log, int ch,
                             int N, int groups);

}  // namespace gdn
