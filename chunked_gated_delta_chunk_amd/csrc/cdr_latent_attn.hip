// Latent attention in the expanded form: prefill and training.
//
//     s_ij = scale (qn_i . kn_j + qr_i . kr_j)     qn, kn: 128 dimensions a head, qr, kr: 64, kr one
//     o_i  = sum_j p_ij v_j,  p = softmax(s)        for all heads; v: 128; causal, the last row of a
//     lse_i = log sum_j exp s_ij                    sequence sees all its keys
//
// and with delta_i = do_i . o_i, ds_ij = p_ij (do_i . v_j - delta_i):
//
//     dv_j = sum_i p_ij do_i,   dq_i = scale sum_j ds_ij k_j,   dk_j = scale sum_i ds_ij q_i,
//     dkr_j = the rope part of dk_j summed over the heads.
//
// All products run on 32x32x16 MFMA with fp32 accumulators; p and ds enter the next product as bf16
// (8 bits of each weight, the same as the outputs carry).  What bounds them is the matrix rate, so the
// layout is chosen to feed it:
//  - A wave owns 32 rows (keys in the dk/dv kernel) whose operands stay in registers; the tiles of
//    the other side stream through LDS two deep, by copies that need no registers.
//  - Products are taken transposed where that puts the owned index in the lane (S^T = K Q^T): the
//    softmax statistics are then a lane's own, and the result's registers are, in the order
//    8 (i / 4) + 4 (lane / 32) + i % 4, directly the right operand of the next product.  No weights
//    pass through LDS.  The other operand of that product comes through the transposing read.
//  - 16-byte pieces of a tile row are stored at piece ^ f(row), with f one to one on 16 rows: both the
//    row reads and the transposing reads then use all banks.
//
// The backward computes the scores twice, once for dq (rows in the lanes) and once for dk and dv
// (keys in the lanes), rather than adding dq's parts by atomics, whose order would change the
// result; dkr's parts are written a head each and added in order.
#include "chunk_dr.h"
#include "cdr_latent.h"

namespace cdr {

namespace {

constexpr int AN = 128;       // nope dimensions
constexpr int AV = 128;       // value dimensions
constexpr int AQ = AN + LR;   // a query's
constexpr int A_ROWS = 128;   // rows (or keys) of a workgroup
constexpr int A_CUS = 256;
constexpr int A_TILE = 64;    // rows of a streamed tile
constexpr int A_LDS = 2 * A_TILE * (256 + 128 + 256);   // two tiles of 320 dimensions

struct LatentAttnArgs {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* kr;
    const uint16_t* v;
    const int32_t* cuq;
    const int32_t* cuk;
    const uint16_t* d_o;
    float* delta;       // written by the dq kernel
    uint16_t* o;        // forward: o; dq kernel: dq
    float* lse;
    uint16_t* dk;
    uint16_t* dv;
    float* dkr;         // [H][Tk total][64]
    int64_t qt, qh, kt, kh, rt, vt, vh;   // strides, elements
    int T, Tk, H, N, slots, total_k;
    int ranked;         // blocks by weight rather than by slot
    int fill;           // rows (keys) that no sequence holds are written too
    float scale, scale2;
};

struct Seq {
    int64_t q0, k0;    // first row and key
    int lq, lk;
};

// an offset at an index that the whole wave shares, through the scalar cache
__device__ __forceinline__ int offset_at(const int32_t* cu, int i) {
    typedef const int32_t __attribute__((address_space(4))) cint32;
    return ((const cint32*)cu)[i];
}

__device__ __forceinline__ Seq attn_seq(const LatentAttnArgs& a, int n) {
    Seq s;
    if (a.cuq) {
        const int qb = min(max(offset_at(a.cuq, n), 0), a.T), kb = min(max(offset_at(a.cuk, n), 0), a.Tk);
        s.q0 = qb, s.k0 = kb;
        s.lq = min(max(offset_at(a.cuq, n + 1), qb), a.T) - qb;
        s.lk = min(max(offset_at(a.cuk, n + 1), kb), a.Tk) - kb;
    } else {
        s.q0 = (int64_t)n * a.T, s.k0 = (int64_t)n * a.Tk;
        s.lq = a.T, s.lk = a.Tk;
    }
    return s;
}

// Sequence and block of a slot: as in the chunk map, sequence n owns the slots from
// cu[n] / ROWS + n on (packed), or n * ceil(T / ROWS) on.  False for an unused slot.
template <int ROWS>
__device__ __forceinline__ bool attn_slot(const LatentAttnArgs& a, const int32_t* cu, int T, int slot, int& n, int& block) {
    if (cu == nullptr) {
        const int per = (T + ROWS - 1) / ROWS;
        n = slot / per;
        block = slot - n * per;
        return true;
    }
    int lo = 0, hi = a.N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (min(max(offset_at(cu, mid), 0), T) / ROWS + mid <= slot) lo = mid; else hi = mid - 1;
    }
    n = lo;
    const int b = min(max(offset_at(cu, n), 0), T);
    block = slot - (b / ROWS + n);
    return block >= 0 && block * ROWS < min(max(offset_at(cu, n + 1), b), T) - b;
}

// The same with the heaviest blocks first, `rank` counting them: of up to 64 packed sequences, all last blocks
// of the longest, then those a block shorter and so on.  With few blocks for each CU the device otherwise ends
// with a long sequence's heavy blocks alone.
template <int ROWS>
__device__ __forceinline__ bool attn_ranked(const LatentAttnArgs& a, const int32_t* cu, int T, int rank, int& n, int& block) {
    const int lane = threadIdx.x & 63;
    int blocks = 0;
    if (lane < a.N) {
        const int b = min(max(cu[lane], 0), T);
        blocks = (min(max(cu[lane + 1], b), T) - b + ROWS - 1) / ROWS;
    }
    int most = blocks;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) most = max(most, __shfl_xor(most, m, 64));
    most = __builtin_amdgcn_readfirstlane(most);
    for (int b = most - 1; b >= 0; --b) {
        uint64_t with = __ballot(blocks > b);
        const int count = __popcll(with);
        if (rank < count) {
            for (; rank > 0; --rank) with &= with - 1;
            n = __builtin_ctzll(with);
            block = b;
            return true;
        }
        rank -= count;
    }
    return false;
}

// The block of rows of a workgroup: heaviest first.
template <int ROWS>
__device__ __forceinline__ bool attn_block(const LatentAttnArgs& a, int i, int& n, int& block) {
    if (a.ranked) return attn_ranked<ROWS>(a, a.cuq, a.T, i, n, block);
    return attn_slot<ROWS>(a, a.cuq, a.T, a.slots - 1 - i, n, block);
}

// Copies rows `first` .. + 63 (clipped to `last`) of an array with 256-byte or 128-byte rows to LDS:
// this wave's share of NW.  base: row 0; stride: bytes between rows.
template <int NW>
__device__ __forceinline__ void copy256(const void* base, int64_t first, int64_t last, uint32_t stride, uint32_t lds, int w,
                                        int lane) {
    const char* b = static_cast<const char*>(base) + first * stride;
    const int top = (int)min(last - first, (int64_t)63);
#pragma unroll
    for (int i = 0; i < 16 / NW; ++i) {
        const int row = 4 * (w + NW * i) + (lane >> 4);
        const uint32_t off = __umul24(min(row, top), stride) + (((lane & 15) ^ f16(row)) * 16);
        dma16(b, off, lds + 1024 * (w + NW * i));
    }
}
template <int NW>
__device__ __forceinline__ void copy128(const void* base, int64_t first, int64_t last, uint32_t stride, uint32_t lds, int w,
                                        int lane) {
    const char* b = static_cast<const char*>(base) + first * stride;
    const int top = (int)min(last - first, (int64_t)63);
#pragma unroll
    for (int i = 0; i < 8 / NW; ++i) {
        const int row = 8 * (w + NW * i) + (lane >> 3);
        const uint32_t off = __umul24(min(row, top), stride) + (((lane & 7) ^ f8(row)) * 16);
        dma16(b, off, lds + 1024 * (w + NW * i));
    }
}

// Where a lane reads in a tile.  The exclusive or with f16 or f8 leaves a step's or column tile's part of the
// offset free, so each read is a base, one exclusive or with a constant and a fixed step; `again` keeps
// the compiler from holding every one of them in a register over the loop.
struct Reads {
    int r256, r128, c256[2], c128[2];
    __device__ __forceinline__ explicit Reads(int lane) {
        const int r = lane & 31, i = lane & 15, piece = 2 * ((lane >> 4) & 1) + ((i >> 1) & 1);
        r256 = r * 256 + (((lane >> 5) ^ f16(r)) * 16);
        r128 = r * 128 + (((lane >> 5) ^ f8(r)) * 16);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int row = 8 * g + 4 * (lane >> 5) + (i >> 2);
            c256[g] = row * 256 + ((piece ^ f16(row)) * 16) + (i & 1) * 8;
            c128[g] = row * 128 + ((piece ^ f8(row)) * 16) + (i & 1) * 8;
        }
    }
    __device__ __forceinline__ Reads again() const {
        Reads x = *this;
        x.r256 = fresh(r256), x.r128 = fresh(r128);
        x.c256[0] = fresh(c256[0]), x.c256[1] = fresh(c256[1]);
        x.c128[0] = fresh(c128[0]), x.c128[1] = fresh(c128[1]);
        return x;
    }
    // left operand of 16 contracted dimensions (step s): rows 32 t + (lane & 31) of a tile
    __device__ __forceinline__ bf16x8 row256(const char* tile, int t, int s) const {
        return lds16(tile + t * 32 * 256 + (r256 ^ (32 * s)));
    }
    __device__ __forceinline__ bf16x8 row128(const char* tile, int t, int s) const {
        return lds16(tile + t * 32 * 128 + (r128 ^ (32 * s)));
    }
    // left operand of 16 contracted rows (step s: rows 16 s ..) for columns 32 c + (lane & 31) of a tile, the
    // rows in the order 8 (i / 4) + 4 (lane / 32) + i % 4 of a result's registers
    __device__ __forceinline__ bf16x8 col256(const char* tile, int s, int c) const {
        const char* p = tile + s * 16 * 256;
        return join8(lds_tr(p + (c256[0] ^ (64 * c))), lds_tr(p + (c256[1] ^ (64 * c))));
    }
    __device__ __forceinline__ bf16x8 col128(const char* tile, int s, int c) const {
        const char* p = tile + s * 16 * 128;
        return join8(lds_tr(p + (c128[0] ^ (64 * c))), lds_tr(p + (c128[1] ^ (64 * c))));
    }
};

// four neighbouring columns of a transposed result as bf16
__device__ __forceinline__ void put4(uint16_t* p, const f32x16& x, int g, float f) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf2(x[4 * g] * f, x[4 * g + 1] * f), pack_bf2(x[4 * g + 2] * f, x[4 * g + 3] * f));
}

// What the forward and the dq kernel share: a workgroup's 128 rows, streamed keys and values.
struct Tiles {
    uint32_t kn, kr, v;   // LDS offsets of buffer 0
};

template <int NW>
__device__ __forceinline__ void load_keys(const LatentAttnArgs& a, const Seq& s, int h, int tile, int buf, const Tiles& at,
                                          int w, int lane) {
    const int64_t first = (int64_t)tile * A_TILE, last = s.lk - 1;
    copy256<NW>(a.k + s.k0 * a.kt + h * a.kh, first, last, (uint32_t)a.kt * 2, at.kn + buf * A_TILE * 256, w, lane);
    copy128<NW>(a.kr + s.k0 * a.rt, first, last, (uint32_t)a.rt * 2, at.kr + buf * A_TILE * 128, w, lane);
    copy256<NW>(a.v + s.k0 * a.vt + h * a.vh, first, last, (uint32_t)a.vt * 2, at.v + buf * A_TILE * 256, w, lane);
}

// o and lse of a block of 128 rows: two workgroups a CU, so that one's products cover the other's softmax; a
// wave is preferred during its products, so that the two stay apart.
//
// A row's running maximum m is raised by a larger score only where that key's weight is over a sixteenth of the
// sum so far, or over 2^8: o is otherwise rescaled in most tiles, some row or other having met a slightly larger
// score.  Weights over 1 are as exact in bf16 and their sums in fp32; but the largest weight is 1 and exact where m
// is its score, and so it stays for every key that carries a sixteenth of its row or more.
//
// 8192 tokens, 16 heads: 340 us, 1.01 PFLOP/s, the matrix unit 55 % busy; the softmax's arithmetic, which both
// workgroups of a SIMD share, and the waits at its ends bound the rest.  The two go together, and pay in that range
// of lengths: 8192 tokens 341 us with both, 364 without the preference, 371 with o rescaled at every new maximum, 363
// with neither; 5 packed sequences of 8168 tokens 111, 111, 113 and 110; 2048 tokens 54.4, 52.2, 54.7 and 52.4; 32768
// tokens 5.15, 5.23, 5.09 and 5.06 ms.
__global__ __launch_bounds__(256, 2) void latent_fwd_kernel(LatentAttnArgs a) {
    __shared__ __align__(256) char lds[A_LDS];
    char* kn = lds;
    char* kr = kn + 2 * A_TILE * 256;
    char* vt = kr + 2 * A_TILE * 128;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (a.fill) {
        fill_unheld(reinterpret_cast<uint4*>(a.o), a.H * (AV / 8), make_uint4(0, 0, 0, 0), a.cuq, a.N, a.T, blockIdx.x, gridDim.x);
        fill_unheld(a.lse, a.H, -INFINITY, a.cuq, a.N, a.T, blockIdx.x, gridDim.x);
    }
    const int h = blockIdx.x % a.H;
    int n, block;
    if (!attn_block<A_ROWS>(a, blockIdx.x / a.H, n, block)) return;
    const Seq s = attn_seq(a, n);
    const Tiles at = {lds_offset(kn), lds_offset(kr), lds_offset(vt)};
    const Reads reads(lane);

    // this lane's row, and the keys it sees
    const int row = block * A_ROWS + 32 * w + (lane & 31);
    const int use = min(row, s.lq - 1);
    const int lim = min(s.lk, s.lk - s.lq + use + 1);
    const int lim_first = min(s.lk, s.lk - s.lq + min(block * A_ROWS + 32 * w, s.lq - 1) + 1);
    const int lim_last = min(s.lk, s.lk - s.lq + min(block * A_ROWS + 32 * w + 31, s.lq - 1) + 1);
    const int keys = min(s.lk, s.lk - s.lq + min(block * A_ROWS + A_ROWS - 1, s.lq - 1) + 1);
    const int tiles = keys > 0 ? (keys + A_TILE - 1) / A_TILE : 0;

    bf16x8 qf[12];
    {
        const uint16_t* q = a.q + (s.q0 + use) * a.qt + h * a.qh + 8 * (lane >> 5);
#pragma unroll
        for (int k = 0; k < 12; ++k) qf[k] = *reinterpret_cast<const bf16x8*>(q + 16 * k);
    }
    f32x16 o[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = zero16();
    float m = -INFINITY, l = 0.f;

    if (tiles > 0) load_keys<4>(a, s, h, 0, 0, at, w, lane);
    for (int j = 0; j < tiles; ++j) {
        const int buf = j & 1;
        dma_wait();
        __syncthreads();
        if (j + 1 < tiles) load_keys<4>(a, s, h, j + 1, buf ^ 1, at, w, lane);
        if (j * A_TILE >= lim_last) continue;   // all of this wave's rows end before this tile
        const Reads x = reads.again();
        const char* tn = kn + buf * A_TILE * 256;
        const char* tr = kr + buf * A_TILE * 128;
        const char* tv = vt + buf * A_TILE * 256;
        // a score over this raises m; worked out here, where the products cover it
        const float bound = m + fminf(fmaxf(lg2((l + __shfl_xor(l, 32, 64)) * (1.f / 16.f)), 0.f), 8.f);
        f32x16 sc[2] = {zero16(), zero16()};
        bf16x8 f[2][2][2];
        auto read_keys = [&](int batch) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int k = 2 * batch + i;
                    f[batch & 1][i][t] = k < 8 ? x.row256(tn, t, k) : x.row128(tr, t, k - 8);
                }
        };
        __builtin_amdgcn_s_setprio(1);
        read_keys(0);
#pragma unroll
        for (int batch = 0; batch < 6; ++batch) {
            if (batch < 5) read_keys(batch + 1);
            keep_order();
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int t = 0; t < 2; ++t) sc[t] = mma(f[batch & 1][i][t], qf[2 * batch + i], sc[t]);
            keep_order();
        }
        __builtin_amdgcn_s_setprio(0);
        if ((j + 1) * A_TILE > lim_first) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (j * A_TILE + 32 * t + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3) >= lim) sc[t][i] = -INFINITY;
        }
        float top = -INFINITY;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, sc[t][i]);
        top = fmaxf(top, __shfl_xor(top, 32, 64)) * a.scale2;
        const float now = top > bound ? top : m;
        const float ref = now == -INFINITY ? 0.f : now;
        const float alpha = ex2(m - ref);
        m = now;
        float sum = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                sc[t][i] = ex2(sc[t][i] * a.scale2 - ref);
                sum += sc[t][i];
            }
        l = l * alpha + sum;
        if (__builtin_expect(!__all(alpha == 1.f), 0)) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[c][i] *= alpha;
        }
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const bf16x8 p = operand(sc[t], u);
#pragma unroll
                for (int c = 0; c < 4; ++c) o[c] = mma(x.col256(tv, 2 * t + u, c), p, o[c]);
            }
        __builtin_amdgcn_s_setprio(0);
    }
    l += __shfl_xor(l, 32, 64);
    if (row >= s.lq) return;
    const float inv = l > 0.f ? 1.f / l : l;   // a row without keys gives zeros, NaN stays NaN
    const size_t out = (size_t)(s.q0 + row) * a.H + h;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int g = 0; g < 4; ++g) put4(a.o + out * AV + 32 * c + 8 * g + 4 * (lane >> 5), o[c], g, inv);
    if (lane < 32) a.lse[out] = l == 0.f ? -INFINITY : LN2 * (m + lg2(l));
}

// dq of a block of 32 NW rows, and delta on the way.  A wave holds 48 registers of q and 96 of sums; do, 32 more,
// stays in LDS (`mine`), without which the loop spilled and each spill's reload waited for the copies under way.
//
// delta is do . o from the forward's o, but for rows that see at most 128 keys it is summed from the weights.
// There ds is a difference of two numbers of one size (a row of one key has ds = 0), o is large and its rounding
// to bf16 would be a tenth of the error of dq and dk; behind many keys that share a row o is an average and its
// rounding counts little.  Where one key carries such a row it counts: the error of dq and dk, of which 1.7e-3 is
// their own rounding, is 2.4e-3 with largest weights of 0.03 on average (2048 keys), 2.8e-3 with 0.29, 5.0e-3 with
// 0.77 and 6.6e-3 with 0.92.
//
// Blocks of 256 rows, two waves a SIMD; of 128 where the 256-row ones are fewer than two a CU (512), and a block's
// own time is what counts.  Forward and gradients, us, with 128 and 256 rows: one sequence of 8192 tokens, 16 heads
// (528 blocks of 256) 1717 and 1540, 8 heads (264) 924 and 976; 4 packed ones of 8192 tokens, 16 heads (576) 643 and
// 589, 8 heads (288) 384 and 407; 2048 tokens, 64 heads (576) 547 and 499, 16 heads (144) 228 and 246; 1001 tokens of 7
// sequences, 8 heads (80) 58 and 65; but 40 sequences of 8168 tokens, 8 heads (568) 158 and 163.  8192 tokens, 16 heads:
// 503 us, the matrix unit 55 % busy, 1.09 PFLOP/s with the scores that it computes again.
template <int ROWS>
__global__ __launch_bounds__(2 * ROWS, ROWS == 256 ? 2 : 1) void latent_dq_kernel(LatentAttnArgs a, const uint16_t* o) {
    constexpr int NW = ROWS / 32;
    __shared__ __align__(256) char lds[A_LDS + ROWS * 256];
    if (a.fill)
        fill_unheld(reinterpret_cast<uint4*>(a.o), a.H * (AQ / 8), make_uint4(0, 0, 0, 0), a.cuq, a.N, a.T, blockIdx.x, gridDim.x);
    const int h = blockIdx.x % a.H;
    int n, block;
    if (!attn_block<ROWS>(a, blockIdx.x / a.H, n, block)) return;
    const Seq s = attn_seq(a, n);
    char* kn = lds;
    char* kr = kn + 2 * A_TILE * 256;
    char* vt = kr + 2 * A_TILE * 128;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Tiles at = {lds_offset(kn), lds_offset(kr), lds_offset(vt)};
    const Reads reads(lane);
    const int row = block * ROWS + 32 * w + (lane & 31);
    const int use = min(row, s.lq - 1);
    const int lim = min(s.lk, s.lk - s.lq + use + 1);
    const int lim_first = min(s.lk, s.lk - s.lq + min(block * ROWS + 32 * w, s.lq - 1) + 1);
    const int lim_last = min(s.lk, s.lk - s.lq + min(block * ROWS + 32 * w + 31, s.lq - 1) + 1);
    const int keys = min(s.lk, s.lk - s.lq + min(block * ROWS + ROWS - 1, s.lq - 1) + 1);
    const int tiles = keys > 0 ? (keys + A_TILE - 1) / A_TILE : 0;

    const size_t in = (size_t)(s.q0 + use) * a.H + h;
    bf16x8 qf[12];
    char* mine = lds + A_LDS + w * 32 * 256;
    float delta = 0.f;
    {
        uint4 of[8];
        const uint16_t* at_o = o + in * AV + 8 * (lane >> 5);
#pragma unroll
        for (int k = 0; k < 8; ++k) of[k] = *reinterpret_cast<const uint4*>(at_o + 16 * k);
        const uint16_t* q = a.q + (s.q0 + use) * a.qt + h * a.qh + 8 * (lane >> 5);
#pragma unroll
        for (int k = 0; k < 12; ++k) qf[k] = *reinterpret_cast<const bf16x8*>(q + 16 * k);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 4), at_row = min(block * ROWS + 32 * w + r, s.lq - 1);
            dma16(a.d_o + ((size_t)(s.q0 + at_row) * a.H + h) * AV + ((lane & 15) ^ f16(r)) * 8, lds_offset(mine) + 1024 * i);
        }
        if (tiles > 0) load_keys<NW>(a, s, h, 0, 0, at, w, lane);
        dma_wait();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float x[8], y[8];
            unpack8(of[k], x);
            unpack8(__builtin_bit_cast(uint4, reads.row256(mine, 0, k)), y);
#pragma unroll
            for (int e = 0; e < 8; ++e) delta += x[e] * y[e];
        }
        delta += __shfl_xor(delta, 32, 64);
    }
    float lse = a.lse[in] * LOG2E;
    if (lse == -INFINITY) lse = INFINITY;   // a row without keys: all its weights are zero

    // s, then do . v, of this lane's row and the 32 keys of half t of tile j, and the weights
    auto scores = [&](const Reads& x, int j, int t, float (&p)[16], f32x16& dp) {
        const int buf = j & 1;
        const char* tn = kn + buf * A_TILE * 256;
        const char* tr = kr + buf * A_TILE * 128;
        const char* tv = vt + buf * A_TILE * 256;
        const Reads again = reads.again();   // do's own reads: not kept from one half to the next
        f32x16 sc = zero16();
        dp = zero16();
        // the two sums in turn: of products of one sum each waits for the one before (8192 tokens, 16 heads: 7 us)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            dp = mma(x.row256(tv, t, k), again.row256(mine, 0, k), dp);
            sc = mma(x.row256(tn, t, k), qf[k], sc);
            if (k & 1) sc = mma(x.row128(tr, t, k >> 1), qf[8 + (k >> 1)], sc);
        }
        const bool cut = j * A_TILE + 32 * t + 32 > lim_first;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            p[i] = ex2(sc[i] * a.scale2 - lse);
            if (cut && j * A_TILE + 32 * t + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3) >= lim) p[i] = 0.f;
        }
    };

    const bool early = s.lk - s.lq + block * ROWS + 1 <= 2 * A_TILE;   // the block's first row at least
    if (early) {   // leaves both tiles in LDS
        float sum = 0.f;
        for (int j = 0; j < min(tiles, 2); ++j) {
            dma_wait();
            __syncthreads();
            if (j == 0 && tiles > 1) load_keys<NW>(a, s, h, 1, 1, at, w, lane);
            const Reads x = reads.again();
#pragma unroll 1
            for (int t = 0; t < 2; ++t) {
                if (j * A_TILE + 32 * t >= lim_last) break;
                float p[16];
                f32x16 dp;
                scores(x, j, t, p, dp);
#pragma unroll
                for (int i = 0; i < 16; ++i) sum += p[i] * dp[i];
            }
        }
        sum += __shfl_xor(sum, 32, 64);
        if (lim <= 2 * A_TILE) delta = sum;
    }
    if (row < s.lq && lane < 32) a.delta[in] = delta;

    f32x16 dq[6];
#pragma unroll
    for (int c = 0; c < 6; ++c) dq[c] = zero16();
    for (int j = 0; j < tiles; ++j) {
        const int buf = j & 1;
        dma_wait();
        __syncthreads();
        if (j + 1 < tiles && !(early && j == 0)) load_keys<NW>(a, s, h, j + 1, buf ^ 1, at, w, lane);
        const Reads x = reads.again();
        const char* tn = kn + buf * A_TILE * 256;
        const char* tr = kr + buf * A_TILE * 128;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (j * A_TILE + 32 * t >= lim_last) break;
            float p[16];
            f32x16 dp;
            scores(x, j, t, p, dp);
#pragma unroll
            for (int i = 0; i < 16; ++i) dp[i] = p[i] * (dp[i] - delta);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const bf16x8 d = operand(dp, u);
#pragma unroll
                for (int c = 0; c < 4; ++c) dq[c] = mma(x.col256(tn, 2 * t + u, c), d, dq[c]);
#pragma unroll
                for (int c = 0; c < 2; ++c) dq[4 + c] = mma(x.col128(tr, 2 * t + u, c), d, dq[4 + c]);
            }
        }
    }
    if (row >= s.lq) return;
    const size_t out = (size_t)(s.q0 + row) * a.H + h;
#pragma unroll
    for (int c = 0; c < 6; ++c)
#pragma unroll
        for (int g = 0; g < 4; ++g) put4(a.o + out * AQ + 32 * c + 8 * g + 4 * (lane >> 5), dq[c], g, a.scale);
}

// dk and dv of a block of 128 keys, and the head's part of dkr: one wave a SIMD, whose 512 registers hold v and
// the 10 blocks of sums; the softmax of one half tile runs between the products of the other.  8192 tokens, 16
// heads: 692 us, 0.99 PFLOP/s, the matrix unit 47 % busy: with one wave a SIMD, waits for LDS reads are not covered.
__global__ __launch_bounds__(256, 1) void latent_dkv_kernel(LatentAttnArgs a) {
    __shared__ __align__(256) char lds[A_LDS];
    __shared__ __align__(256) char own[A_ROWS * (256 + 128)];   // this block's keys, 32 a wave: operands like v's,
                                                               // for which the registers do not reach
    __shared__ __align__(16) float stat[2][2][A_TILE];   // lse (base 2) and delta of a tile's rows
    char* qn = lds;
    char* qr = qn + 2 * A_TILE * 256;
    char* td = qr + 2 * A_TILE * 128;
    const uint32_t qn0 = lds_offset(qn), qr0 = lds_offset(qr), td0 = lds_offset(td);
    if (a.fill) {
        const uint4 zero = make_uint4(0, 0, 0, 0);
        fill_unheld(reinterpret_cast<uint4*>(a.dk), a.H * (AN / 8), zero, a.cuk, a.N, a.Tk, blockIdx.x, gridDim.x);
        fill_unheld(reinterpret_cast<uint4*>(a.dv), a.H * (AV / 8), zero, a.cuk, a.N, a.Tk, blockIdx.x, gridDim.x);
    }
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = blockIdx.x % a.H;
    int n, block;
    if (!attn_slot<A_ROWS>(a, a.cuk, a.Tk, blockIdx.x / a.H, n, block)) return;
    const Seq s = attn_seq(a, n);
    const Reads reads(lane);
    const int key = block * A_ROWS + 32 * w + (lane & 31);
    const int use = min(key, s.lk - 1);
    const int shift = s.lk - s.lq;                          // row i sees keys up to i + shift
    const int first_row = max(0, block * A_ROWS - shift);   // the first row that sees a key of this block
    const int j0 = first_row / A_TILE, tiles = (s.lq + A_TILE - 1) / A_TILE;

    const char* kn = own + w * 32 * 256;
    const char* kr = own + A_ROWS * 256 + w * 32 * 128;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + (lane >> 4), at = min(block * A_ROWS + 32 * w + r, s.lk - 1);
        dma16(a.k + (s.k0 + at) * a.kt + h * a.kh + ((lane & 15) ^ f16(r)) * 8, lds_offset(kn) + 1024 * i);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 3), at = min(block * A_ROWS + 32 * w + r, s.lk - 1);
        dma16(a.kr + (s.k0 + at) * a.rt + ((lane & 7) ^ f8(r)) * 8, lds_offset(kr) + 1024 * i);
    }
    bf16x8 vf[8];
    {
        const uint16_t* v = a.v + (s.k0 + use) * a.vt + h * a.vh + 8 * (lane >> 5);
#pragma unroll
        for (int i = 0; i < 8; ++i) vf[i] = *reinterpret_cast<const bf16x8*>(v + 16 * i);
    }
    f32x16 dk[6], dv[4];
#pragma unroll
    for (int c = 0; c < 6; ++c) dk[c] = zero16();
#pragma unroll
    for (int c = 0; c < 4; ++c) dv[c] = zero16();

    auto load_rows = [&](int tile, int buf) {
        const int64_t first = (int64_t)tile * A_TILE, last = s.lq - 1;
        const uint16_t* q = a.q + s.q0 * a.qt + h * a.qh;
        copy256<4>(q, first, last, (uint32_t)a.qt * 2, qn0 + buf * A_TILE * 256, w, lane);
        copy128<4>(q + AN, first, last, (uint32_t)a.qt * 2, qr0 + buf * A_TILE * 128, w, lane);
        copy256<4>(a.d_o + ((size_t)s.q0 * a.H + h) * AV, first, last, (uint32_t)a.H * AV * 2, td0 + buf * A_TILE * 256, w, lane);
    };
    // wave 0: lse, so that a row behind the end or without keys has weights of zero; wave 1: delta.  Loaded a
    // tile before it is put into LDS: a value needed at once would be waited for behind the copies.
    auto load_stat = [&](int tile) {
        if (w >= 2) return 0.f;
        const int64_t r = (int64_t)tile * A_TILE + lane;
        const size_t at = (size_t)(s.q0 + min(r, (int64_t)s.lq - 1)) * a.H + h;
        return w == 0 ? (r < s.lq ? a.lse[at] : INFINITY) : a.delta[at];
    };
    auto put_stat = [&](float x, int buf) {
        if (w < 2) stat[buf][w][lane] = w == 0 ? (x == -INFINITY ? INFINITY : x * LOG2E) : x;
    };

    float ahead = 0.f;
    if (j0 < tiles) {
        put_stat(load_stat(j0), 0);
        ahead = load_stat(j0 + 1);   // a tile behind the end reads the last row, and is not used
        load_rows(j0, 0);
    }
    // a tile's begin: it has arrived, the next one is sent for
    auto arrive = [&](int j, int buf) {
        dma_wait();
        __syncthreads();
        if (j + 1 < tiles) {
            put_stat(ahead, buf ^ 1);
            ahead = load_stat(j + 2);
            load_rows(j + 1, buf ^ 1);
        }
    };
    // Two loops, the tiles whose rows do not all see this wave's keys (they come first) and the others: as
    // branches of one loop, the sums were copied between registers at every turn.  The waves leave the
    // first at different tiles; each tile has one barrier in either.
    int j = j0;
    for (; j < tiles && j * A_TILE + shift < block * A_ROWS + 32 * w + 31; ++j) {
        const int buf = (j - j0) & 1;
        arrive(j, buf);
        const Reads x = reads.again();
        const char* tn = qn + buf * A_TILE * 256;
        const char* tr = qr + buf * A_TILE * 128;
        const char* to = td + buf * A_TILE * 256;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int r0 = j * A_TILE + 32 * t;
            if (r0 + 31 + shift < block * A_ROWS + 32 * w) continue;   // no row here sees these keys
            f32x16 sc = zero16(), dp = zero16();
            // scores and do v^T side by side, two steps' rows read ahead
            bf16x8 f[2][2], g[2][2], kf[2][2];
            auto read_rows = [&](int batch) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int k = 2 * batch + i;
                    f[batch & 1][i] = k < 8 ? x.row256(tn, t, k) : x.row128(tr, t, k - 8);
                    kf[batch & 1][i] = k < 8 ? x.row256(kn, 0, k) : x.row128(kr, 0, k - 8);
                    if (k < 8) g[batch & 1][i] = x.row256(to, t, k);
                }
            };
            read_rows(0);
#pragma unroll
            for (int batch = 0; batch < 6; ++batch) {
                if (batch < 5) read_rows(batch + 1);
                keep_order();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int k = 2 * batch + i;
                    sc = mma(f[batch & 1][i], kf[batch & 1][i], sc);
                    if (k < 8) dp = mma(g[batch & 1][i], vf[k], dp);
                }
                keep_order();
            }
            // a key behind the sequence's end is computed like its last and not stored
            const bool cut = r0 + shift < block * A_ROWS + 32 * w + 31;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 ls = *reinterpret_cast<const f32x4*>(&stat[buf][0][32 * t + 8 * g + 4 * (lane >> 5)]);
                const f32x4 de = *reinterpret_cast<const f32x4*>(&stat[buf][1][32 * t + 8 * g + 4 * (lane >> 5)]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 4 * g + e;
                    float p = ex2(sc[i] * a.scale2 - ls[e]);
                    if (cut && r0 + 8 * g + 4 * (lane >> 5) + e + shift < key) p = 0.f;
                    sc[i] = p;
                    dp[i] = p * (dp[i] - de[e]);
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const bf16x8 p = operand(sc, u), d = operand(dp, u);
#pragma unroll
                for (int c = 0; c < 4; ++c) dv[c] = mma(x.col256(to, 2 * t + u, c), p, dv[c]);
#pragma unroll
                for (int c = 0; c < 4; ++c) dk[c] = mma(x.col256(tn, 2 * t + u, c), d, dk[c]);
#pragma unroll
                for (int c = 0; c < 2; ++c) dk[4 + c] = mma(x.col128(tr, 2 * t + u, c), d, dk[4 + c]);
            }
        }
    }
    for (; j < tiles; ++j) {
        const int buf = (j - j0) & 1;
        arrive(j, buf);
        const Reads x = reads.again();
        const char* tn = qn + buf * A_TILE * 256;
        const char* tr = qr + buf * A_TILE * 128;
        const char* to = td + buf * A_TILE * 256;
        // Every row sees every key.  A wave issues in order, and it is alone on its SIMD: what it computes besides
        // the products is put between them, one element's weight behind each, so that it costs no time of its own.
        f32x16 sc[2] = {zero16(), zero16()}, dp[2] = {zero16(), zero16()};
        f32x4 ls[2], de[2];   // of four rows, and the next four's
        auto read_stat = [&](int t, int g) {
            ls[g & 1] = *reinterpret_cast<const f32x4*>(&stat[buf][0][32 * t + 8 * g + 4 * (lane >> 5)]);
            de[g & 1] = *reinterpret_cast<const f32x4*>(&stat[buf][1][32 * t + 8 * g + 4 * (lane >> 5)]);
        };
        auto weight = [&](int t, int i) {
            if ((i & 3) == 0 && i < 12) read_stat(t, (i >> 2) + 1);
            const float p = ex2(sc[t][i] * a.scale2 - ls[(i >> 2) & 1][i & 3]);
            sc[t][i] = p;
            dp[t][i] = p * (dp[t][i] - de[(i >> 2) & 1][i & 3]);
        };
        bf16x8 f[3], g[3], kf[3];   // rows and keys of three steps: two ahead
        auto read_rows = [&](int t, int k) {
            f[k % 3] = k < 8 ? x.row256(tn, t, k) : x.row128(tr, t, k - 8);
            kf[k % 3] = k < 8 ? x.row256(kn, 0, k) : x.row128(kr, 0, k - 8);
            if (k < 8) g[k % 3] = x.row256(to, t, k);
        };
        read_stat(0, 0);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            read_rows(t, 0);
            read_rows(t, 1);
            keep_order();
#pragma unroll
            for (int k = 0; k < 12; ++k) {
                if (k < 10) read_rows(t, k + 2);
                sc[t] = mma(f[k % 3], kf[k % 3], sc[t]);
                // the twenty products carry sixteen weights: k and k + 1 where there are two products
                const int i = k < 4 ? 2 * k : k + 4;
                if (t == 1) weight(0, i);
                keep_order();
                if (k < 8) {
                    dp[t] = mma(g[k % 3], vf[k], dp[t]);
                    if (t == 1 && k < 4) weight(0, i + 1);
                    keep_order();
                }
            }
        }
        bf16x8 c[4];   // column operands: three ahead
        auto read_columns = [&](int y) {   // dv's four column tiles and dk's six, of each 16 rows
            const int at = y / 10, z = y % 10;
            c[y % 4] = z < 4 ? x.col256(to, at, z) : z < 8 ? x.col256(tn, at, z - 4) : x.col128(tr, at, z - 8);
        };
        read_stat(1, 0);
        bf16x8 p[2], d[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) p[u] = operand(sc[0], u), d[u] = operand(dp[0], u);
        read_columns(0);
        read_columns(1);
        read_columns(2);
        keep_order();
#pragma unroll
        for (int y = 0; y < 40; ++y) {
            const int u = (y / 10) & 1, z = y % 10;
            if (y < 37) read_columns(y + 3);
            if (z < 4) dv[z] = mma(c[y % 4], p[u], dv[z]);
            else dk[z - 4] = mma(c[y % 4], d[u], dk[z - 4]);
            if (y < 16) weight(1, y);
            keep_order();
            if (y == 19)
#pragma unroll
                for (int v = 0; v < 2; ++v) p[v] = operand(sc[1], v), d[v] = operand(dp[1], v);
        }
    }
    dma_wait();   // where no row sees these keys, their copies are still under way
    if (key >= s.lk) return;
    const size_t out = (size_t)(s.k0 + key) * a.H + h;
    const int c4 = 4 * (lane >> 5);
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            put4(a.dv + out * AV + 32 * c + 8 * g + c4, dv[c], g, 1.f);
            put4(a.dk + out * AN + 32 * c + 8 * g + c4, dk[c], g, a.scale);
        }
    float* r = a.dkr + ((size_t)h * a.total_k + s.k0 + key) * LR;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const f32x16& x = dk[4 + c];
            *reinterpret_cast<float4*>(r + 32 * c + 8 * g + c4) =
                make_float4(x[4 * g] * a.scale, x[4 * g + 1] * a.scale, x[4 * g + 2] * a.scale, x[4 * g + 3] * a.scale);
        }
}

// dkr: the heads' parts added in order, 4 dimensions a thread.  8192 tokens, 16 heads: 7.8 us, 34 MB, mostly from
// the Infinity Cache.
__global__ __launch_bounds__(256) void latent_dkr_kernel(const float* part, uint16_t* dkr, const int32_t* cuk, int N, int total,
                                                         int H, int fill) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t first = cuk ? min(max(cuk[0], 0), total) : 0, end = cuk ? min(max(cuk[N], 0), total) : total;
    const bool held = i >= first * (LR / 4) && i < end * (LR / 4);   // only such keys have parts
    if (!held && (!fill || i >= (int64_t)total * (LR / 4))) return;
    f32x4 t = {0.f, 0.f, 0.f, 0.f};
    for (int h = 0; h < (held ? H : 0); ++h) t += *reinterpret_cast<const f32x4*>(part + ((size_t)h * total) * LR + 4 * i);
    *reinterpret_cast<uint2*>(dkr + 4 * i) = make_uint2(pack_bf2(t[0], t[1]), pack_bf2(t[2], t[3]));
}

int64_t total_q(const cdr_latent_attn_problem* p) { return p->varlen ? p->T : (int64_t)p->N * p->T; }
int64_t total_k(const cdr_latent_attn_problem* p) { return p->varlen ? p->Tk : (int64_t)p->N * p->Tk; }

int64_t attn_slots(int64_t T, const cdr_latent_attn_problem* p, int rows = A_ROWS) {
    return p->varlen ? T / rows + p->N : p->N * ((T + rows - 1) / rows);
}

// Slots of a launch over rows, and whether its blocks are taken by weight: of 2 to `most` packed sequences with at
// most six blocks of 128 rows a CU.  Ragged batches of 16 heads, time by weight over time by slot, forward and dq:
//
//     sequences        2             5             8             16            32            48            64
//     4000 tokens   1.00  0.93    0.92  0.90    0.93  0.91    0.87  0.94    1.09  0.90    1.09  0.97    1.15  0.97
//     8168          0.97  0.98    0.87  0.86    0.80  0.88    0.88  0.93    0.99  0.88    1.00  0.99    1.04  0.90
//     12000         0.96  0.93    0.89  0.99    0.90  0.97    0.92  0.92    1.01  0.88    1.02  0.91    1.08  0.94
//     16000         1.01  1.03    1.00  1.07    0.92  0.96    0.97  0.98                                1.08  1.01
//     16000, 32 heads  1.03 1.05  1.02  1.05    1.02  1.05    1.04  1.05                                1.16  1.03
//
// (8168 tokens of 5 sequences: 119 and 104 us, 197 and 170.)  Finding a block costs steps in the number of blocks a
// sequence has, and in short forwards of many sequences that shows: they stop at 32, dq at 64.  dk and dv go by slot:
// by weight they took longer in 35 of 40 such batches, 7 % in the middle and 29 % at most.
void set_order(LatentAttnArgs& a, const cdr_latent_attn_problem* p, int rows, int most) {
    a.slots = (int)attn_slots(p->T, p, rows);
    a.ranked = p->varlen && p->N >= 2 && p->N <= most && attn_slots(p->T, p) * p->H <= 6 * A_CUS;
}

bool ok_stride(int64_t s) { return s >= 0 && (s & 7) == 0 && s < (1 << 23); }
bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

LatentAttnArgs attn_args(const cdr_latent_attn_problem* p, const void* q, const void* k, const void* kr, const void* v,
                         const int32_t* cuq, const int32_t* cuk) {
    LatentAttnArgs a = {};
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.kr = static_cast<const uint16_t*>(kr);
    a.v = static_cast<const uint16_t*>(v);
    a.cuq = p->varlen ? cuq : nullptr;
    a.cuk = p->varlen ? cuk : nullptr;
    a.qt = p->q_stride[0], a.qh = p->q_stride[1];
    a.kt = p->k_stride[0], a.kh = p->k_stride[1];
    a.rt = p->k_rope_stride;
    a.vt = p->v_stride[0], a.vh = p->v_stride[1];
    a.T = p->T, a.Tk = p->Tk, a.H = p->H, a.N = p->N;
    a.total_k = (int)total_k(p);
    a.fill = p->varlen == CDR_VARLEN_FILL;
    a.scale = p->scale;
    a.scale2 = p->scale * LOG2E;
    return a;
}

size_t up16(size_t x) { return (x + 15) / 16 * 16; }

}  // namespace

}  // namespace cdr

extern "C" {

cdr_status cdr_latent_attn_check(const cdr_latent_attn_problem* p) {
    if (p == nullptr) return CDR_ERR_NULL_ARG;
    if (p->N <= 0 || p->T < 0 || p->Tk < 0 || p->H <= 0) return CDR_ERR_BAD_SHAPE;
    if (!(p->scale > 0.f) || p->scale > 3.0e38f) return CDR_ERR_BAD_SHAPE;
    if (p->H > (1 << 15)) return CDR_ERR_UNSUPPORTED;
    const int64_t tq = cdr::total_q(p), tk = cdr::total_k(p);
    if (tq * p->H > INT32_MAX || tk * p->H > INT32_MAX) return CDR_ERR_BAD_SHAPE;
    if (cdr::attn_slots(p->T, p) * p->H > INT32_MAX || cdr::attn_slots(p->Tk, p) * p->H > INT32_MAX) return CDR_ERR_BAD_SHAPE;
    for (int i = 0; i < 2; ++i)
        if (!cdr::ok_stride(p->q_stride[i]) || !cdr::ok_stride(p->k_stride[i]) || !cdr::ok_stride(p->v_stride[i]))
            return CDR_ERR_UNSUPPORTED;
    if (!cdr::ok_stride(p->k_rope_stride)) return CDR_ERR_UNSUPPORTED;
    return CDR_OK;
}

cdr_status cdr_latent_attn_fwd(const cdr_latent_attn_problem* p, const void* q, const void* k_nope, const void* k_rope,
                               const void* v, const int32_t* cu_seqlens, const int32_t* cu_seqlens_k, void* o, float* lse,
                               void* stream) {
    const cdr_status st = cdr_latent_attn_check(p);
    if (st != CDR_OK) return st;
    if (cdr::total_q(p) == 0) return CDR_OK;
    if (!q || !o || !lse || (p->varlen && (!cu_seqlens || !cu_seqlens_k))) return CDR_ERR_NULL_ARG;
    if (cdr::total_k(p) > 0 && (!k_nope || !k_rope || !v)) return CDR_ERR_NULL_ARG;
    if (!cdr::aligned16(q) || !cdr::aligned16(k_nope) || !cdr::aligned16(k_rope) || !cdr::aligned16(v) || !cdr::aligned16(o))
        return CDR_ERR_UNSUPPORTED;
    cdr::LatentAttnArgs a = cdr::attn_args(p, q, k_nope, k_rope, v, cu_seqlens, cu_seqlens_k);
    a.o = static_cast<uint16_t*>(o);
    a.lse = lse;
    cdr::set_order(a, p, cdr::A_ROWS, 32);
    hipLaunchKernelGGL(cdr::latent_fwd_kernel, dim3((unsigned)(a.slots * (int64_t)a.H)), dim3(256), 0,
                       static_cast<hipStream_t>(stream), a);
    return hipGetLastError() == hipSuccess ? CDR_OK : CDR_ERR_HIP;
}

size_t cdr_latent_attn_bwd_workspace_bytes(const cdr_latent_attn_problem* p) {
    if (cdr_latent_attn_check(p) != CDR_OK) return 0;
    return cdr::up16((size_t)cdr::total_q(p) * p->H * sizeof(float)) + (size_t)cdr::total_k(p) * p->H * cdr::LR * sizeof(float);
}

cdr_status cdr_latent_attn_bwd(const cdr_latent_attn_problem* p, const void* q, const void* k_nope, const void* k_rope,
                               const void* v, const int32_t* cu_seqlens, const int32_t* cu_seqlens_k, const void* o,
                               const float* lse, const void* d_o, void* dq, void* dk_nope, void* dk_rope, void* dv,
                               void* workspace, size_t workspace_bytes, void* stream) {
    const cdr_status st = cdr_latent_attn_check(p);
    if (st != CDR_OK) return st;
    const int64_t tq = cdr::total_q(p), tk = cdr::total_k(p);
    if (p->varlen && (!cu_seqlens || !cu_seqlens_k)) return CDR_ERR_NULL_ARG;
    if (tq > 0 && (!q || !o || !lse || !d_o || !dq)) return CDR_ERR_NULL_ARG;
    if (tk > 0 && (!k_nope || !k_rope || !v || !dk_nope || !dk_rope || !dv)) return CDR_ERR_NULL_ARG;
    const void* all[] = {q, k_nope, k_rope, v, o, d_o, dq, dk_nope, dk_rope, dv};
    for (const void* x : all)
        if (!cdr::aligned16(x)) return CDR_ERR_UNSUPPORTED;
    const size_t need = cdr_latent_attn_bwd_workspace_bytes(p);
    if (need > 0 && (!workspace || !cdr::aligned16(workspace) || workspace_bytes < need)) return CDR_ERR_WORKSPACE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    cdr::LatentAttnArgs a = cdr::attn_args(p, q, k_nope, k_rope, v, cu_seqlens, cu_seqlens_k);
    a.delta = static_cast<float*>(workspace);
    a.dkr = reinterpret_cast<float*>(static_cast<char*>(workspace) + cdr::up16((size_t)tq * p->H * sizeof(float)));
    a.lse = const_cast<float*>(lse);
    a.d_o = static_cast<const uint16_t*>(d_o);
    a.o = static_cast<uint16_t*>(dq);
    a.dk = static_cast<uint16_t*>(dk_nope);
    a.dv = static_cast<uint16_t*>(dv);
    if (tq > 0) {
        const uint16_t* fo = static_cast<const uint16_t*>(o);
        const bool large = cdr::attn_slots(p->T, p, 256) * p->H >= 2 * cdr::A_CUS;
        cdr::set_order(a, p, large ? 256 : 128, 64);
        const dim3 grid((unsigned)(a.slots * (int64_t)a.H));
        if (large) hipLaunchKernelGGL((cdr::latent_dq_kernel<256>), grid, dim3(512), 0, s, a, fo);
        else hipLaunchKernelGGL((cdr::latent_dq_kernel<128>), grid, dim3(256), 0, s, a, fo);
        if (hipGetLastError() != hipSuccess) return CDR_ERR_HIP;
    }
    if (tk > 0) {
        hipLaunchKernelGGL(cdr::latent_dkv_kernel, dim3((unsigned)(cdr::attn_slots(p->Tk, p) * p->H)), dim3(256), 0, s, a);
        if (hipGetLastError() != hipSuccess) return CDR_ERR_HIP;
        hipLaunchKernelGGL(cdr::latent_dkr_kernel, dim3((unsigned)((tk * (cdr::LR / 4) + 255) / 256)), dim3(256), 0, s, a.dkr,
                           static_cast<uint16_t*>(dk_rope), a.cuk, p->N, (int)tk, p->H, a.fill);
        if (hipGetLastError() != hipSuccess) return CDR_ERR_HIP;
    }
    return CDR_OK;
}

}  // extern "C"
