// z1_ops_internal.h -- what the host code of the operators (z1_ops_api.hip)
// and their kernels (z1_muon.hip, z1_embed.hip, z1_loss.hip) share.  Not
// installed.
#pragma once

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "z1_muon_tile.h"
#include "z1_ops.h"

namespace z1 {
namespace ops {

typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef float float16v __attribute__((ext_vector_type(16)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint2v __attribute__((ext_vector_type(2)));

constexpr int kWaveLanes = 64;

// bf16 <-> fp32, to nearest even, NaN kept (quiet).
__device__ __forceinline__ float bf16_to_f32(uint16_t h)
{
    return __uint_as_float((uint32_t)h << 16);
}
__device__ __forceinline__ uint16_t f32_to_bf16(float x)
{
    return __builtin_bit_cast(uint16_t, (__bf16)x);
}

// Element types of the operators' tensors: storage, and conversion from and
// to fp32 (to nearest even).
struct F32 {
    typedef float store;
    static __device__ __forceinline__ float up(store x) { return x; }
    static __device__ __forceinline__ store down(float x) { return x; }
};
struct BF16 {
    typedef uint16_t store;
    static __device__ __forceinline__ float up(store x) { return bf16_to_f32(x); }
    static __device__ __forceinline__ store down(float x) { return f32_to_bf16(x); }
};
struct F16 {
    typedef _Float16 store;
    static __device__ __forceinline__ float up(store x) { return (float)x; }
    static __device__ __forceinline__ store down(float x) { return (_Float16)x; }
};

// 16 bytes of storage of type T, and what they hold.
template <typename T>
struct Pack16 {
    static constexpr int N = 16 / (int)sizeof(typename T::store);
    union {
        uint4v raw;
        typename T::store e[N];
    };
};

// --------------------------------------------------------------------------
// Muon
// --------------------------------------------------------------------------

// One matrix of a z1_muon.  X is the matrix with the smaller side first:
// U itself, or its transpose where flip is set.  m x n are X's sides, mp x np
// the same padded to whole tiles; the padding of every buffer holds zeros.
struct MuonMat {
    const void *grad;
    float *mom;
    float *master;
    uint16_t *weight;
    uint16_t *ortho;
    int32_t rows, cols;     // of the caller's matrix
    int32_t m, n, mp, np;
    int32_t flip;
    int32_t vec;            // 1: grad and momentum are 16-byte aligned
    int32_t vec4;           // 1: so are the rows of master, weight and ortho (8 bytes for bf16)
    int64_t part0, n_part;  // its norm partials
    // operands, panel-major (see panel_at)
    _Float16 *X;            // mp rows, np deep: the operand copy of X
    _Float16 *Y[2];         // np rows, mp deep: of X^T, one being read and one written
    _Float16 *A, *B;        // mp rows, mp deep
    _Float16 *L;            // what the operand copy of X leaves of it (see carry_at)
    // wide products: what each operand leaves of its value, laid out as it, and
    // X itself in fp32, laid out as L (which they do without)
    _Float16 *Xl, *Yl[2], *Al, *Bl;
    float *F;
    double lr_scale, wd_scale;
};

struct MuonTile {
    int32_t mat, ti, tj;
    int32_t part;   // X X^T: the tile's number, or splits times it plus the piece's
};

// A piece of one matrix for the elementwise pass.
struct MuonChunk {
    int64_t start;
    int32_t mat, count;
};

struct MuonTables {
    const MuonMat *mats;
    const MuonChunk *chunks;   // elementwise pass; chunk q writes partial q
    const MuonTile *cast;      // kCastTile square tiles of the padded X
    // the tiles of the products X X^T and A A (ti >= tj) and B X, and their side
    const MuonTile *tiles[3];
    int64_t n_chunks, n_cast, n_tiles[3];
    int32_t tile[3];           // 64, 128 or 256
    // X X^T of few tiles and much depth: every tile in `splits` pieces of it
    const MuonTile *pieces;    // [n_tiles[0] * splits]
    float *parts;              // [n_tiles[0] * splits][64 * 64]
    int32_t splits;            // 1: not split
    int64_t n_part_most;       // partials of the matrix that has most
    double *partials;          // [n_chunks]
    double *inv;               // [n]  1 / (|U|_F + eps)
    int32_t n;                 // matrices of the tiled path: mats[0 .. n - 1]
    int32_t n_small;           // those one workgroup takes whole: the n_small after them
    int32_t grad_bf16;
    int32_t wide;              // products of 22-bit operands
    float a, b, c;
    double eps;
};

struct MuonUpdate {
    double lr, wd;             // of the step
    float mu;
    int32_t nesterov;
    double clip;               // <= 0: no clipping
    const double *d_S;
    int32_t step;              // 1: z1_muon_step, 0: z1_muon_orthogonalize
};

// Element (row, k) of an fp16 operand with `rows` rows: panels of 32 along k,
// each [rows][32], so that a tile's share of a panel is one contiguous piece.
__host__ __device__ __forceinline__ int64_t panel_at(int64_t rows, int64_t row, int64_t k)
{
    return ((k >> 5) * rows + row) * 32 + (k & 31);
}

// Element (i, j) of X's remainder (np columns): blocks of 32 x 32 in the order
// in which the matrix instruction's lanes hold them, 4 elements a lane.
__host__ __device__ __forceinline__ int64_t carry_at(int64_t np, int64_t i, int64_t j)
{
    const int64_t block = (i >> 5) * (np >> 5) + (j >> 5);
    return block * 1024 + ((i & 31) >> 3) * 256 + (((i >> 2) & 1) * 32 + (j & 31)) * 4 + (i & 3);
}

constexpr int kCastTile = 64;
constexpr int kMuonChunk = 8192;

hipError_t launch_muon(const MuonTables &t, const MuonUpdate &u, int ns_steps, hipStream_t s);

// --------------------------------------------------------------------------
// Embedding
// --------------------------------------------------------------------------

struct EmbedShape {
    int64_t n, vocab, dim;     // ids, rows, row length
    const void *ids;
    int32_t id32;              // ids are int32
    float scale;
};

constexpr int kSortBlock = 1024;   // ids one workgroup of the radix sort handles
constexpr int kSortSmall = 8192;   // ids one workgroup sorts alone

// Where z1_embed_grad's workspace holds what; offsets in bytes.
struct EmbedWork {
    int64_t keys[2], perm[2], hist, parts, bytes;
    int64_t n_blocks;          // of the radix sort
    int64_t chunk, n_chunks;   // sorted positions per chunk of the sums
};

EmbedWork embed_work(int64_t n, int64_t vocab, int64_t dim);

hipError_t launch_lookup(int32_t dtype, const EmbedShape &e, const void *w, int64_t ld_w, void *out,
                         int64_t ld_out, hipStream_t s);
hipError_t launch_embed_grad(int32_t dtype, const EmbedShape &e, const void *dout, int64_t ld,
                             float *dw, bool accumulate, void *work, hipStream_t s);

// --------------------------------------------------------------------------
// Losses
// --------------------------------------------------------------------------

// z1_logits as the kernels take it, and where the gradient goes.
struct Rows {
    int64_t n, vocab, ld, ld_d;
    const void *x;
    const void *y;          // targets
    void *d;                // dlogits or null
    int32_t y32;            // targets are int32
    int32_t d_vec;          // a row of d sits at its x row's place mod 16 bytes
};

struct PolicyScalars {
    float lo, hi, kl, scale;   // 1 - clip_low, 1 + clip_high
};

struct PolicyPtrs {
    const float *old_logp, *ref_logp, *adv, *w;
    float *token_loss, *logp;
};

hipError_t launch_logprob(int32_t dtype, const Rows &r, float *logp, float *lse, hipStream_t s);
hipError_t launch_logprob_grad(int32_t dtype, const Rows &r, const float *lse, const float *dlogp,
                               hipStream_t s);
hipError_t launch_policy(int32_t dtype, const Rows &r, const PolicyPtrs &p, const PolicyScalars &k,
                         float *loss, double scale, hipStream_t s);
hipError_t launch_preference(const z1_preference_args &a, hipStream_t s);

}  // namespace ops
}  // namespace z1
