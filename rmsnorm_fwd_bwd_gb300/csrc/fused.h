// fused.h -- host-side interface between the entry points of
// include/rmsnorm_fused.h (fused_api.cu) and their kernels (add.cu, quant.cu,
// rope.cu). Internal: not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/rmsnorm.h"

namespace rmsnorm {

// Most rope sets (query heads, key heads) of one call.
constexpr int kRopeMaxSets = 2;
// Threads of a block that holds one row, at most; of one that holds several.
constexpr int kFusedMaxThreads = 512;
// The forwards' blocks for the widest rows off 16 bytes.
constexpr int kFusedWideThreads = 1024;
constexpr int kFusedGroupThreads = 128;

// How a kernel's rows lie. kRowsAligned: every row on a 16-byte boundary and of whole
// octets (blocks of 8 columns, octet.cuh). kRowsOnePhase: the rows of all its tensors
// (but for gamma) start at one offset from a 16-byte boundary, as dense tensors of any
// width do: octets start on the boundaries, and only a row's two ends are masked.
// kRowsAny: anything.
enum RowMode : int { kRowsAny = 0, kRowsAligned = 1, kRowsOnePhase = 2 };

// Residual addition (with dropout), norm and, in quant.cu, 8-bit output.
struct AddArgs {
    const void* x;
    const void* res;                // may be null: nothing is added
    const void* gamma;
    void* h;                        // may be null: not written
    void* y;                        // quant: the e4m3 codes
    float* rstd;                    // forward output, may be null; backward input
    const void* dy;                 // backward
    const void* dh;                 // backward, may be null: zero
    void* dx;                       // backward output, may be null
    void* dres;                     // backward output, may be null
    float* ws;                      // backward: dgamma partials [units][ldws]
    float* scales;                  // quant
    int64_t ldx, ldres, ldh, ldy, lddy, lddh, lddx, lddres, ldws, ldscales;
    int64_t M;
    int N;
    float eps;
    float inv_n;                    // quant: 1 / N
    float one;                      // 1 with the offset variant (g = 1 + gamma), else 0
    const unsigned long long* rng;  // dropout: {seed, offset} in device memory
    unsigned long long* rng_used;   // forward: a copy of them, may be null
    uint32_t threshold;             // dropout: 0 for none
    float scale;
    int group;                      // quant: columns per scale, 0 for the row
    int group_shift;                // log2 of a group's octets
    int pow2;                       // quant: scales rounded up to a power of two
    int stages;                     // ring: rows staged
    uint32_t slot;                  // bytes of a row's place in a stage
    int same_phase;                 // outputs at one offset from a 16-byte boundary
    uint32_t* err;                  // device error word
};

// A launch shape. lanes: lanes per row (0: a block per row, -1: a wide block).
struct AddPlan {
    int dtype = 0;
    int mode = kRowsAny;
    int lanes = 0;
    int octets = 1;  // per thread
    int threads = 0;
    int64_t blocks = 0;
    size_t smem = 0;
    bool drop = false;
    bool ring = false;  // add_bwd.cu's ring
    int stages = 0;
    uint32_t slot = 0;
};

const void* add_fwd_kernel(const AddPlan& p);
const void* add_bwd_kernel(const AddPlan& p);
const void* quant_kernel(const AddPlan& p);

// One tensor of heads [T, heads, D] and its weight.
struct RopeSet {
    const void* x;
    const void* gamma;   // may be null: no norm
    const void* dy;      // backward
    void* y;             // forward: output; backward: dx
    int64_t x_token, x_head, dy_token, dy_head, y_token, y_head;  // strides in elements
    int heads;
};

struct RopeArgs {
    RopeSet set[kRopeMaxSets];
    int nsets;
    int heads;                 // of all sets
    const int64_t* pos;        // [T]
    const double* inv_freq;    // [R / 2]
    int64_t T;
    int D, R;
    int interleaved;
    int chunk;                 // heads that a group of lanes takes of a token
    int nchunk;                // chunks per token
    int chunks0;               // of them of the first set (octet kernels)
    float mscale;
    float eps;
    float one;
    float* ws;                 // backward: partials of dgamma, a plane of [units][ldws] per set
    int64_t ldws;
    int64_t units;
};

// How a head row is taken: entry by entry, or in 16-byte octets with neighbours paired,
// whole octets of the halves paired, or the partners through shared memory.
enum RopeRows { kRopeEntries = 0, kRopeNeighbours, kRopeHalves, kRopeSwap };

struct RopePlan {
    int dtype = 0;
    RopeRows rows = kRopeEntries;
    int lanes = 0;             // per head row
    int pairs = 0;             // per lane, elsewhere
    int threads = 0;
    int64_t blocks = 0;
    size_t smem = 0;
};

// Most heads that a group of lanes takes at a time in the forward: their loads are in
// flight together (128 bytes a lane).
constexpr int rope_fwd_batch(int dtype) { return dtype == 0 ? 2 : 4; }

// Most heads for which a group computes a token's cosines and sines once, but for the forward
// of whole octets.
constexpr int kRopeRun = 8;

const void* rope_kernel(const RopePlan& p, bool bwd);
// How head rows are taken, and the lanes (and pairs of each) that take one; wide: they start on
// 16-byte boundaries.
void rope_lanes(int64_t D, int64_t R, int interleaved, bool wide, RopePlan& p);

// Checks that the entry points of heads share. Strides of [T, heads, D] heads; of an output,
// whose rows must not overlap (tokens outside heads, or heads outside tokens); the numbers.
bool strides_ok(int64_t token, int64_t head, int64_t heads, int64_t T, int64_t D);
bool output_strides_ok(int64_t token, int64_t head, int64_t heads, int64_t T, int64_t D);
// Heads [T, heads, D] in memory: where the first starts, and strides in elements.
struct HeadsAt {
    const void* p;
    int64_t token, head, heads;
};
// Whether no two head rows of p and q (elements of `s` bytes) share a byte. Heads that lie between one
// another are told apart by their distance within what the strides are multiples of; where that does
// not show it, false.
bool heads_apart(const HeadsAt& p, const HeadsAt& q, int64_t T, int64_t D, int64_t s);
// Whether p is q: the same first row and strides.
bool heads_same(const HeadsAt& p, const HeadsAt& q, int64_t T);
rmsnorm_status check_rope(int nsets, int64_t T, int64_t D, int64_t R, int interleaved, float mscale, float eps,
                          rmsnorm_dtype dtype, int offset);

// SMs of the current device, whose number goes to dev; 0 on failure.
int current_sms(int& dev);
// Allow the kernel the device's whole shared memory.
bool allow_shared_memory(const void* k, int dev);
// Blocks of `threads` that an SM holds; 0 on failure. Sets the attribute above where needed.
int resident_blocks(const void* k, int dev, int threads, size_t smem);

}  // namespace rmsnorm
