// Latent attention in the absorbed form, over a paged cache: the decode path.
//
// A cached key is one row of 576 bf16 shared by all heads: 512 latent dimensions c, which are also
// its value, and 64 rope dimensions r.  For a new token's head, with its key limit (causal among the
// new tokens),
//
//     s_j = scale (q_c . c_j + q_r . r_j),   o = sum_j softmax(s)_j c_j,   lse = log sum_j exp s_j.
//
// All heads (and new tokens) of a sequence read the same keys, so they are the rows of one matrix
// product: 2 (576 + 512) flops a key and row against 1152 bytes a key.  With 16 rows the cache's
// bytes bound it, with 128 the matrix rate is as near.
//
// A workgroup of four waves (eight for M > 16) takes M = 16, 32 or 64 rows and walks over tiles of
// 64 keys.
//  - A tile (72 KiB) goes to LDS once, two deep, by 16-byte copies that need no registers; a key's
//    latent row is one wave's copy, so its page is looked up in scalar registers.  16-byte pieces
//    are stored at position p ^ f16w(key), which spreads both reads below over the banks.
//  - Scores: a wave takes 16 or 32 keys against 16 rows, whose q stays in registers as the right
//    operand, so the result S^T has a row of q in each lane and the running maximum is a lane's own
//    value after two shuffles and one exchange between the waves.
//  - Values: a wave takes its share of the 512 columns, O^T += V^T P^T, V^T through the transposing
//    read; P^T goes through LDS in the operand's order.  So the tile is read from LDS once or twice
//    a product and not once for every 16 rows, which would be the bound.
//
// Work is cut evenly over the device whatever the lengths: the tiles of all (sequence, row block)
// units are numbered and each workgroup takes an equal run of them.  Where a sequence has several row
// blocks, a team of neighbouring workgroups takes them side by side, one block each, so that they
// read the same keys at the same time through one L2.  A unit that one workgroup covers is written
// directly; a unit cut between workgroups leaves partial sums (fp32, with their maximum and sum) that
// a second kernel joins in order.  The cut depends on the lengths and sizes alone, so the same inputs
// give the same bits.
//
// Measured, inputs changing from call to call: 256 sequences of up to 8192 keys, 16 heads, 225 us, 5.4 TB/s of cache,
// which HBM bounds; 64 sequences of 4 tokens and 64 heads, up to 4096 keys, 142 us, of which the copies to LDS alone
// (four row blocks read each key, 10 TB/s) take 74; 8192 keys of one sequence, 16 heads, 13.6 us and 7.3 for the join,
// all latency.
#include "chunk_dr.h"
#include "cdr_latent.h"

namespace cdr {

namespace {

constexpr int DEC_GRID = 256;        // workgroups; LDS holds one on a CU
constexpr int DEC_KEYS = 64;         // keys of a tile
// Most row blocks that are taken side by side.  64 sequences of 512 rows, up to 4096 keys, with 1, 2, 4, 8 and 16: 308,
// 266, 259, 254 and 254 us; of 256 rows (four blocks) 168, 148, 147; 256 sequences of 2048 rows with 8 and 16: 1924, 1838.
constexpr int DEC_TEAM = 8;
// Keys of a sequence at most: pages are looked up two tiles ahead, up to key len + 190, which stays in int.
constexpr int64_t DEC_MAX_LEN = (int64_t)INT32_MAX - 255;

struct LatentDecodeArgs {
    const uint16_t* qc;
    const uint16_t* qr;
    const uint16_t* cache;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* cu;
    uint16_t* o;
    float* lse;
    float* part;       // [2 grid][M][512] partial sums
    float2* part_ml;   // [2 grid][M] their maximum (base 2) and sum
    int4* rec;         // [grid] (n, row block, parts) of the unit cut at this workgroup's end
    int64_t qct, qch, qrt, qrh;
    int N, T, H, cols, num_pages, shift;
    int fill;          // rows that no sequence holds are written too
    int team;          // workgroups that take the row blocks of one sequence side by side
    float scale2;      // scale * log2(e)
};

struct SeqInfo {
    int bos, tokens, len;    // first new token, new tokens, keys that the table has room for
    int total;               // seq_lens, from which the rows' limits count
};

__device__ __forceinline__ SeqInfo dec_seq(const LatentDecodeArgs& a, int n) {
    SeqInfo s;
    if (a.cu) {
        s.bos = min(max(a.cu[n], 0), a.T);
        s.tokens = min(max(a.cu[n + 1], s.bos), a.T) - s.bos;
    } else {
        s.bos = n * a.T;
        s.tokens = a.T;
    }
    const int64_t room = (int64_t)a.cols << a.shift;
    s.total = max(a.lens[n], 0);
    s.len = (int)min((int64_t)s.total, min(room, DEC_MAX_LEN));
    return s;
}

// key tiles of a sequence, at least one so that rows without keys are written too
__device__ __forceinline__ int dec_tiles(const SeqInfo& s) { return max((s.len + DEC_KEYS - 1) / DEC_KEYS, 1); }

template <int M>
__device__ __forceinline__ int dec_blocks(const LatentDecodeArgs& a, const SeqInfo& s) {
    return (int)(((int64_t)s.tokens * a.H + M - 1) / M);
}
// units of a sequence: its row blocks in teams
template <int M>
__device__ __forceinline__ int dec_units(const LatentDecodeArgs& a, const SeqInfo& s) {
    return (dec_blocks<M>(a, s) + a.team - 1) / a.team;
}

// The page of key `key` of sequence n, -1 behind its end; and that key's cache row, -1 where there is
// none.  Apart, so that a page is loaded two tiles before its row is worked out.
__device__ __forceinline__ int dec_page(const LatentDecodeArgs& a, int n, int len, int key) {
    return key < len ? a.table[(size_t)n * a.cols + (key >> a.shift)] : -1;
}
__device__ __forceinline__ int dec_row(const LatentDecodeArgs& a, int page, int key) {
    if (page < 0 || page >= a.num_pages) return -1;
    return (page << a.shift) + (key & ((1 << a.shift) - 1));
}

// This workgroup's run of tiles: [begin, end) of all units' tiles, the sequence n in which it begins
// and the number unit0 of that sequence's first tile.  False where there is nothing to do.
struct Run {
    int64_t begin, end, share, unit0;
    int n, team, member;
};

template <int M, int THREADS>
__device__ __forceinline__ bool dec_run(const LatentDecodeArgs& a, int wg, Run& run) {
    constexpr int NW = THREADS / 64;
    __shared__ int64_t scan[NW];
    __shared__ int64_t found[2];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    auto tiles_of = [&](int n) {
        if (n >= a.N) return (int64_t)0;
        const SeqInfo s = dec_seq(a, n);
        return (int64_t)dec_units<M>(a, s) * dec_tiles(s);
    };
    const int64_t first = tiles_of(tid);
    int64_t total = first;
    for (int n = tid + THREADS; n < a.N; n += THREADS) total += tiles_of(n);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) total += __shfl_xor(total, m, 64);
    if (lane == 0) scan[w] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) total += scan[i];
    __syncthreads();
    const int teams = DEC_GRID / a.team;
    run.team = wg / a.team, run.member = wg - run.team * a.team;
    run.share = (total + teams - 1) / teams;
    run.begin = run.team * run.share, run.end = min(total, run.begin + run.share);
    if (tid == 0) a.rec[wg] = make_int4(-1, 0, 0, 0);
    if (run.begin >= run.end || run.team >= teams) return false;
    int64_t before = 0;
    for (int base = 0; base < a.N; base += THREADS) {
        const int64_t own = base == 0 ? first : tiles_of(base + tid);
        int64_t sum = own;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const int64_t x = __shfl_up(sum, m, 64);
            if (lane >= m) sum += x;
        }
        if (lane == 63) scan[w] = sum;
        __syncthreads();
        int64_t lo = before + sum - own, chunk = 0;
        for (int i = 0; i < NW; ++i) {
            if (i < w) lo += scan[i];
            chunk += scan[i];
        }
        if (run.begin >= lo && run.begin < lo + own) {
            found[0] = base + tid;
            found[1] = lo;
        }
        before += chunk;
        __syncthreads();
        if (before > run.begin) break;
    }
    run.n = __builtin_amdgcn_readfirstlane((int)found[0]);
    run.unit0 = found[1];
    return true;
}

// The next unit of a run at tile `pos`: false where there is none for this workgroup there, with pos
// and the sequence moved on.
struct Unit {
    SeqInfo s;
    int tiles, t0, t1, rb;
    int64_t rows;
};

template <int M>
__device__ __forceinline__ bool dec_unit(const LatentDecodeArgs& a, Run& run, int64_t& pos, Unit& u) {
    u.s = dec_seq(a, run.n);
    u.tiles = dec_tiles(u.s);
    const int64_t all = (int64_t)dec_units<M>(a, u.s) * u.tiles;
    if (pos >= run.unit0 + all) {
        run.unit0 += all;
        ++run.n;
        return false;
    }
    const int unit = (int)((pos - run.unit0) / u.tiles);
    u.t0 = (int)((pos - run.unit0) - (int64_t)unit * u.tiles);
    u.t1 = (int)min((int64_t)u.tiles, u.t0 + (run.end - pos));
    u.rb = unit * a.team + run.member;
    u.rows = (int64_t)u.s.tokens * a.H;
    if (u.rb >= dec_blocks<M>(a, u.s)) {   // the last team of a sequence may be short
        pos += u.t1 - u.t0;
        return false;
    }
    return true;
}

// This wave's share of a tile to LDS (kc, kr: offsets of the buffer; zeros: its start, for rows that are
// not there).  row: this lane's cache row, of key `lane` of the tile.
template <int NW>
__device__ __forceinline__ void dec_load(const LatentDecodeArgs& a, uint32_t kc, uint32_t kr, char* zeros, int row, int w,
                                         int lane) {
    constexpr int KPW = DEC_KEYS / NW;   // keys that a wave copies
    const int lane16 = fresh(lane * 16);
    if (a.shift >= 4 && __ballot(row >= 0) == ~0ull) {
        // Pages of 16 keys or more and a whole tile: the wave's keys are neighbours in one page, one address
        // for all.  (With an address a key, looked up and multiplied out in scalar registers, the 64 x 4 token,
        // 64 head batch took 7 us more.)
        const uint16_t* base = a.cache + (size_t)__builtin_amdgcn_readlane(row, KPW * w) * LROW;
#pragma unroll
        for (int i = 0; i < KPW; ++i)
            dma16(base, (lane16 ^ (f16w(KPW * w + i) * 16)) + i * (LROW * 2), kc + (KPW * w + i) * (LC * 2));
#pragma unroll
        for (int i = 0; i < KPW / 8; ++i) {
            const int k = 8 * i + (lane >> 3);
            dma16(base, k * (LROW * 2) + LC * 2 + (((lane & 7) ^ (((KPW * w + k) >> 1) & 7)) * 16), kr + (KPW * w + 8 * i) * (LR * 2));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < KPW; ++i) {
        const int key = KPW * w + i;
        const int from = __builtin_amdgcn_readlane(row, key);
        if (from >= 0) {
            dma16(a.cache + (size_t)from * LROW, lane16 ^ (f16w(key) * 16), kc + key * (LC * 2));
        } else {
            *reinterpret_cast<uint4*>(zeros + key * (LC * 2) + lane16) = make_uint4(0, 0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < KPW / 8; ++i) {
        const int key = KPW * w + 8 * i + (lane >> 3);
        const int at = max(__shfl(row, key, 64), 0);   // scores of absent keys are replaced
        dma16(a.cache + (size_t)at * LROW + LC + (((lane & 7) ^ ((key >> 1) & 7)) * 8), kr + (KPW * w + 8 * i) * (LR * 2));
    }
}

// workgroups go round the 8 XCDs: numbered so that neighbours, which read the same sequence, share an L2
__device__ __forceinline__ int dec_wg() { return (blockIdx.x & 7) * (DEC_GRID / 8) + (blockIdx.x >> 3); }

template <int MT, int NW, int KG>
__global__ __launch_bounds__(64 * NW, 1) void latent_decode_kernel(LatentDecodeArgs a) {
    constexpr int M = 16 * MT;
    constexpr int KT = 4 / KG;                 // scores: key groups KG, 16-key tiles of a wave,
    constexpr int RH = NW / KG, MQ = MT / RH;  // row parts, row tiles of a wave
    constexpr int CT = 32 / NW;                // 16-column tiles of a wave in the values' product
    __shared__ __align__(256) char kc[2][DEC_KEYS * LC * 2];
    __shared__ __align__(256) char kr[2][DEC_KEYS * LR * 2];
    __shared__ __align__(16) char pf[MT * 2 * 1024];   // P^T in operand order
    __shared__ float mx[KG][M];
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int kg = w % KG, rh = w / KG;        // the wave's keys and row part in the scores
    const int wg = dec_wg();
    if (a.fill) {
        fill_unheld(reinterpret_cast<uint4*>(a.o), (int64_t)a.H * (LC / 8), make_uint4(0, 0, 0, 0), a.cu, a.N, a.T, wg, DEC_GRID);
        if (a.lse) fill_unheld(a.lse, a.H, -INFINITY, a.cu, a.N, a.T, wg, DEC_GRID);
    }
    Run run;
    if (!dec_run<M, 64 * NW>(a, wg, run)) return;
    int64_t pos = run.begin;

    const uint32_t kc0 = lds_offset(kc), kr0 = lds_offset(kr);
    // where this lane reads in a tile: key 16 KT kg + r, pieces 4 k + q (the exclusive or leaves bits 4
    // and up of the piece alone, so four bases and fixed steps serve all k), the rope pieces, and for
    // the transposed reads key 4 q + r / 4, the 8 bytes 4 (r & 3) .. of each column tile
    int k_at[4], r_at[2], v_at[CT];
#pragma unroll
    for (int k = 0; k < 4; ++k) k_at[k] = (16 * KT * kg + r) * (LC * 2) + ((4 * k + q) ^ f16w(r)) * 16;
#pragma unroll
    for (int k = 0; k < 2; ++k) r_at[k] = (16 * KT * kg + r) * (LR * 2) + ((4 * k + q) ^ ((r >> 1) & 7)) * 16;
#pragma unroll
    for (int c = 0; c < CT; ++c)
        v_at[c] = (4 * q + (r >> 2)) * (LC * 2) + ((2 * (CT * w + c) + ((r >> 1) & 1)) ^ f16w(4 * q + (r >> 2))) * 16 +
                  (r & 1) * 8;
    while (pos < run.end) {
        Unit u;
        if (!dec_unit<M>(a, run, pos, u)) continue;
        const SeqInfo s = u.s;
        const int n = run.n, t0 = u.t0, t1 = u.t1, tiles = u.tiles, rb = u.rb;
        const int64_t rows = u.rows;

        // ---- q of this block's rows, and each row's key limit
        bf16x8 qf[MQ][18];
        int lim[MQ];
#pragma unroll
        for (int mt = 0; mt < MQ; ++mt) {
            int64_t row = (int64_t)rb * M + 16 * (rh * MQ + mt) + r;
            if (row >= rows) row = 0;
            const int tok = (int)(row / a.H), h = (int)(row - (int64_t)tok * a.H);
            lim[mt] = s.total - s.tokens + tok + 1;   // (keys from len on are not there)
            const uint16_t* c = a.qc + (s.bos + tok) * a.qct + h * a.qch;
            const uint16_t* p = a.qr + (s.bos + tok) * a.qrt + h * a.qrh;
#pragma unroll
            for (int k = 0; k < 16; ++k) qf[mt][k] = *reinterpret_cast<const bf16x8*>(c + 32 * k + 8 * q);
#pragma unroll
            for (int k = 0; k < 2; ++k) qf[mt][16 + k] = *reinterpret_cast<const bf16x8*>(p + 32 * k + 8 * q);
        }
        f32x4 o[MT][CT];
        float m[MT], l[MQ];
#pragma unroll
        for (int mt = 0; mt < MQ; ++mt) l[mt] = 0.f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            m[mt] = -INFINITY;
#pragma unroll
            for (int c = 0; c < CT; ++c) o[mt][c] = f32x4{0.f, 0.f, 0.f, 0.f};
        }

        auto load_tile = [&](int buf, int row) {
            dec_load<NW>(a, kc0 + buf * (DEC_KEYS * LC * 2), kr0 + buf * (DEC_KEYS * LR * 2), kc[buf], row, w, lane);
        };

        const int page0 = dec_page(a, n, s.len, 64 * t0 + lane);
        int page = dec_page(a, n, s.len, 64 * (t0 + 1) + lane);   // of the next tile
        dma_wait();        // q and the pages are there
        __syncthreads();   // the previous block's reads of LDS have ended
        int row = dec_row(a, page0, 64 * t0 + lane);
        load_tile(0, row);
        for (int j = t0; j < t1; ++j) {
            const int buf = (j - t0) & 1;
            const uint64_t there = __ballot(row >= 0);
            dma_wait();
            __syncthreads();
            row = dec_row(a, page, 64 * (j + 1) + lane);
            page = dec_page(a, n, s.len, 64 * (j + 2) + lane);
            if (j + 1 < t1) load_tile(buf ^ 1, row);

            // ---- S^T of this wave's keys and row part
            f32x4 sc[KT][MQ];
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int mt = 0; mt < MQ; ++mt) sc[kt][mt] = f32x4{0.f, 0.f, 0.f, 0.f};
            const char* kw = kc[buf];
            const char* rw = kr[buf];
            // a few of the eighteen steps at a time, the next few's keys read ahead
            constexpr int STEPS = KT == 2 ? 2 : 3;
            bf16x8 f[2][STEPS][KT];
            auto read_keys = [&](int batch) {
#pragma unroll
                for (int i = 0; i < STEPS; ++i)
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt) {
                        const int k = STEPS * batch + i;
                        f[batch & 1][i][kt] = k < 16 ? lds16(kw + k_at[k & 3] + (k >> 2) * 256 + kt * 16 * (LC * 2))
                                                     : lds16(rw + r_at[k - 16] + kt * 16 * (LR * 2));
                    }
            };
            read_keys(0);
#pragma unroll
            for (int batch = 0; batch < 18 / STEPS; ++batch) {
                if (batch < 18 / STEPS - 1) read_keys(batch + 1);
                keep_order();
#pragma unroll
                for (int i = 0; i < STEPS; ++i)
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                        for (int mt = 0; mt < MQ; ++mt)
                            sc[kt][mt] = mfma32(f[batch & 1][i][kt], qf[mt][STEPS * batch + i], sc[kt][mt]);
                keep_order();
            }
            const bool whole = there == ~0ull && 64 * j + 63 <= s.total - s.tokens;
#pragma unroll
            for (int mt = 0; mt < MQ; ++mt) {
                float t = -INFINITY;
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float v = sc[kt][mt][i] * a.scale2;
                        if (!whole) {
                            const int key = 16 * (KT * kg + kt) + 4 * q + i;
                            if (64 * j + key >= lim[mt] || !((there >> key) & 1)) v = -INFINITY;
                        }
                        sc[kt][mt][i] = v;
                        t = fmaxf(t, v);
                    }
                t = fmaxf(t, __shfl_xor(t, 16, 64));
                t = fmaxf(t, __shfl_xor(t, 32, 64));
                if (q == 0) mx[kg][16 * (rh * MQ + mt) + r] = t;
            }
            lds_barrier();
            // ---- the new maximum of every row, and this wave's weights
            bool same = true;
            float alpha[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float now = m[mt];
#pragma unroll
                for (int g = 0; g < KG; ++g) now = fmaxf(now, mx[g][16 * mt + r]);
                alpha[mt] = ex2(m[mt] - (now == -INFINITY ? 0.f : now));
                same = same && alpha[mt] == 1.f;
                m[mt] = now;
            }
#pragma unroll
            for (int mt = 0; mt < MQ; ++mt) {
                float now = m[mt], al = alpha[mt];
#pragma unroll
                for (int h = 1; h < RH; ++h)
                    if (rh == h) now = m[h * MQ + mt], al = alpha[h * MQ + mt];
                const float ref = now == -INFINITY ? 0.f : now;
                float sum = 0.f;
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[e] = ex2(sc[kt][mt][e] - ref);
                        sum += p[e];
                    }
                    const int tile = KT * kg + kt;
                    *reinterpret_cast<uint2*>(&pf[((rh * MQ + mt) * 2 + (tile >> 1)) * 1024 + lane * 16 + (tile & 1) * 8]) =
                        make_uint2(pack_bf2(p[0], p[1]), pack_bf2(p[2], p[3]));
                }
                l[mt] = l[mt] * al + sum;
            }
            if (!__all(same)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int c = 0; c < CT; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[mt][c][e] *= alpha[mt];
            }
            // ---- O^T of this wave's columns: the columns of the first 32 keys are read ahead of the
            // barrier, those of the others during the first's products
            bf16x8 v[2][CT], p[MT];
            auto read_columns = [&](int t) {
                const char* at = kc[buf] + t * 32 * (LC * 2);
#pragma unroll
                for (int c = 0; c < CT; ++c) v[t][c] = join8(lds_tr(at + v_at[c]), lds_tr(at + 16 * (LC * 2) + v_at[c]));
            };
            auto read_weights = [&](int t) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) p[mt] = lds16(&pf[(mt * 2 + t) * 1024 + lane * 16]);
            };
            read_columns(0);
            lds_barrier();
            read_weights(0);
            read_columns(1);
            keep_order();
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) o[mt][c] = mfma32(v[t][c], p[mt], o[mt][c]);
                if (t == 0) {
                    read_weights(1);
                    keep_order();
                }
            }
        }
        // ---- the row sums of all waves, then the output
        __syncthreads();
#pragma unroll
        for (int mt = 0; mt < MQ; ++mt) {
            float t = l[mt];
            t += __shfl_xor(t, 16, 64);
            t += __shfl_xor(t, 32, 64);
            if (q == 0) mx[kg][16 * (rh * MQ + mt) + r] = t;
        }
        __syncthreads();
        const bool direct = t0 == 0 && t1 == tiles;
        const int slot = 2 * wg + (t0 == 0 ? 1 : 0);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int i = 16 * mt + r;
            float sum = mx[0][i];
#pragma unroll
            for (int g = 1; g < KG; ++g) sum += mx[g][i];
            const int64_t grow = (int64_t)rb * M + i;
            if (grow >= rows) continue;
            if (direct) {
                const float inv = sum > 0.f ? 1.f / sum : sum;   // a row without keys gives zeros, NaN stays NaN
                const size_t out = (size_t)s.bos * a.H + grow;
#pragma unroll
                for (int c = 0; c < CT; ++c)
                    *reinterpret_cast<uint2*>(a.o + out * LC + 16 * (CT * w + c) + 4 * q) =
                        make_uint2(pack_bf2(o[mt][c][0] * inv, o[mt][c][1] * inv),
                                   pack_bf2(o[mt][c][2] * inv, o[mt][c][3] * inv));
                if (a.lse && w == 0 && q == 0) a.lse[out] = sum == 0.f ? -INFINITY : LN2 * (m[mt] + lg2(sum));
            } else {
                float* part = a.part + ((size_t)slot * M + i) * LC + 16 * CT * w + 4 * q;
#pragma unroll
                for (int c = 0; c < CT; ++c) *reinterpret_cast<f32x4*>(part + 16 * c) = o[mt][c];
                if (w == 0 && q == 0) a.part_ml[(size_t)slot * M + i] = make_float2(m[mt], sum);
            }
        }
        if (t0 == 0 && t1 < tiles && tid == 0)
            a.rec[wg] = make_int4(n, rb, (int)((pos + tiles - 1) / run.share) - run.team + 1, 0);
        pos += t1 - t0;
    }
}

// Joins the partial sums of units that were cut.  Workgroup (wg, i) serves the unit that began in
// workgroup wg's run.  A unit of many parts (one long sequence over the whole device) takes a workgroup
// for each row, whose eight waves take every eighth part; one of few parts a wave for each row, and
// every eighth workgroup for eight rows.  (A workgroup a row for two parts each took 26 us for 256 units of
// 64 rows, a wave a row 13 us.  The eight waves together take 5.5 to 7 us for 16 rows of 128 parts.)
constexpr int JOIN_WAVES = 8;

struct Joined {
    float acc[8];   // columns 8 lane ..
    float m, l;
};

__device__ __forceinline__ Joined join_parts(const LatentDecodeArgs& a, int wg, int row, int M, int parts, int first, int step,
                                             int lane) {
    Joined x;
    x.m = -INFINITY, x.l = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) x.acc[e] = 0.f;
#pragma unroll 4
    for (int k = first; k < parts; k += step) {
        const size_t slot = k == 0 ? 2 * wg + 1 : 2 * (size_t)(wg + k * a.team);
        const float2 pm = a.part_ml[slot * M + row];
        const f32x4* p = reinterpret_cast<const f32x4*>(a.part + (slot * M + row) * LC) + 2 * lane;
        const f32x4 u = p[0], v = p[1];
        const float now = fmaxf(x.m, pm.x);
        const float ref = now == -INFINITY ? 0.f : now;
        const float fa = ex2(x.m - ref), fb = ex2(pm.x - ref);
        x.m = now;
        x.l = x.l * fa + pm.y * fb;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x.acc[e] = x.acc[e] * fa + u[e] * fb;
            x.acc[4 + e] = x.acc[4 + e] * fa + v[e] * fb;
        }
    }
    return x;
}

template <int MT>
__global__ __launch_bounds__(64 * JOIN_WAVES) void latent_join_kernel(LatentDecodeArgs a) {
    constexpr int M = 16 * MT;
    const int wg = blockIdx.x / M, i = blockIdx.x % M;
    const int4 rec = a.rec[wg];
    const int parts = rec.z;
    // (the working ones of a unit differ from unit to unit: workgroups go round the 8 XCDs)
    if (rec.x < 0 || (parts <= JOIN_WAVES && i % JOIN_WAVES != wg % JOIN_WAVES)) return;
    const SeqInfo s = dec_seq(a, rec.x);
    const int64_t rows = (int64_t)s.tokens * a.H - (int64_t)rec.y * M;   // of this block
    const size_t out0 = (size_t)s.bos * a.H + (size_t)rec.y * M;
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if (parts <= JOIN_WAVES) {
        const int row = i - i % JOIN_WAVES + w;
        if (row >= rows) return;
        const Joined x = join_parts(a, wg, row, M, parts, 0, 1, lane);
        const float inv = x.l > 0.f ? 1.f / x.l : x.l;
        uint4 v;
        v.x = pack_bf2(x.acc[0] * inv, x.acc[1] * inv), v.y = pack_bf2(x.acc[2] * inv, x.acc[3] * inv);
        v.z = pack_bf2(x.acc[4] * inv, x.acc[5] * inv), v.w = pack_bf2(x.acc[6] * inv, x.acc[7] * inv);
        *reinterpret_cast<uint4*>(a.o + (out0 + row) * LC + 8 * lane) = v;
        if (a.lse && lane == 0) a.lse[out0 + row] = x.l == 0.f ? -INFINITY : LN2 * (x.m + lg2(x.l));
        return;
    }
    if (i >= rows) return;
    __shared__ float sums[JOIN_WAVES][LC];
    __shared__ float ml[JOIN_WAVES][2];
    const Joined x = join_parts(a, wg, i, M, parts, w, JOIN_WAVES, lane);
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[w][8 * lane + e] = x.acc[e];
    if (lane == 0) ml[w][0] = x.m, ml[w][1] = x.l;
    __syncthreads();
    float top = -INFINITY, sum = 0.f, v = 0.f;
#pragma unroll
    for (int k = 0; k < JOIN_WAVES; ++k) top = fmaxf(top, ml[k][0]);
    const float ref = top == -INFINITY ? 0.f : top;
    const int c = threadIdx.x;
#pragma unroll
    for (int k = 0; k < JOIN_WAVES; ++k) {
        const float f = ex2(ml[k][0] - ref);
        sum += ml[k][1] * f;
        v += sums[k][c] * f;
    }
    const float inv = sum > 0.f ? 1.f / sum : sum;
    a.o[(out0 + i) * LC + c] = f2bf(v * inv);
    if (a.lse && c == 0) a.lse[out0 + i] = sum == 0.f ? -INFINITY : LN2 * (top + lg2(sum));
}

// One wave a token: 64 16-byte pieces of the latent and 8 of the rope part into the cache row that
// its slot names.  256 tokens take 4.7 us, latency.
__global__ __launch_bounds__(256) void latent_write_kernel(const uint16_t* c, const uint16_t* r, int64_t cs, int64_t rs,
                                                           uint16_t* cache, const int32_t* slots, int T,
                                                           int64_t num_slots) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= T) return;
    const int slot = slots[t];
    if (slot < 0 || slot >= num_slots) return;
    uint16_t* to = cache + (size_t)slot * LROW;
    const uint4 v = *reinterpret_cast<const uint4*>(c + t * cs + 8 * lane);
    *reinterpret_cast<uint4*>(to + 8 * lane) = v;
    if (lane < LR / 8)
        *reinterpret_cast<uint4*>(to + LC + 8 * lane) = *reinterpret_cast<const uint4*>(r + t * rs + 8 * lane);
}

// Rows of a block: the fewest of 16, 32 and 64 that hold the rows of a sequence (of an average one in a packed
// batch, whose T counts spare tokens too); more rows would be computed for nothing, fewer would read the keys again.
// Decode and join, us, with blocks of 16, 32 and 64:
//
//     rows a sequence                     16             32             64             128             256
//     64 sequences, to 4096 keys      52  54  60     61  60  65     93  73  75     147 112  96     277 179 149
//     256 sequences, to 2048 keys     92  97 106    120 112 117    192 140 142     352 221 183     642 402 303
//     8 sequences, to 8192 keys       31  33  37     33  39  41     40  42  48      56  49  53      88  66  64
//     1 sequence, 16384 keys          27  28  30     26  32  33     29  33  37      35  36  41      51  44  47
//
// (Few sequences would take blocks of half the size or less up to 64 rows, where the device is not full.)
int dec_m(const cdr_latent_decode_problem* p) {
    const int64_t tokens = p->varlen ? ((int64_t)p->T + p->N - 1) / p->N : p->T;
    const int64_t rows = tokens * p->H;
    return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

template <int MT>
hipError_t launch_latent_decode(const LatentDecodeArgs& a, hipStream_t s) {
    if constexpr (MT == 1) hipLaunchKernelGGL((latent_decode_kernel<1, 4, 4>), dim3(DEC_GRID), dim3(256), 0, s, a);
    else if constexpr (MT == 2) hipLaunchKernelGGL((latent_decode_kernel<2, 8, 4>), dim3(DEC_GRID), dim3(512), 0, s, a);
    else hipLaunchKernelGGL((latent_decode_kernel<4, 8, 2>), dim3(DEC_GRID), dim3(512), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((latent_join_kernel<MT>), dim3(DEC_GRID * 16 * MT), dim3(64 * JOIN_WAVES), 0, s, a);
    return hipGetLastError();
}

bool mult8(int64_t x) { return (x & 7) == 0; }
bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace

}  // namespace cdr

extern "C" {

cdr_status cdr_latent_decode_check(const cdr_latent_decode_problem* p) {
    if (p == nullptr) return CDR_ERR_NULL_ARG;
    if (p->N <= 0 || p->T < 0 || p->H <= 0 || p->num_pages <= 0 || p->page_size <= 0 || p->table_cols <= 0)
        return CDR_ERR_BAD_SHAPE;
    if (p->page_size & (p->page_size - 1)) return CDR_ERR_UNSUPPORTED;
    if ((int64_t)p->num_pages * p->page_size > INT32_MAX) return CDR_ERR_BAD_SHAPE;
    if ((p->varlen ? 1 : (int64_t)p->N) * p->T * p->H > INT32_MAX) return CDR_ERR_BAD_SHAPE;
    for (int i = 0; i < 2; ++i)
        if (!cdr::mult8(p->qc_stride[i]) || !cdr::mult8(p->qr_stride[i])) return CDR_ERR_UNSUPPORTED;
    return CDR_OK;
}

size_t cdr_latent_decode_workspace_bytes(const cdr_latent_decode_problem* p) {
    if (cdr_latent_decode_check(p) != CDR_OK) return 0;
    const size_t rows = 2 * (size_t)cdr::DEC_GRID * cdr::dec_m(p);
    return rows * (cdr::LC * sizeof(float) + sizeof(float2)) + cdr::DEC_GRID * sizeof(int4);
}

cdr_status cdr_latent_decode_fwd(const cdr_latent_decode_problem* p, const void* q_latent, const void* q_rope,
                                 const void* cache, const int32_t* block_table, const int32_t* seq_lens,
                                 const int32_t* cu_seqlens, void* o, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    const cdr_status st = cdr_latent_decode_check(p);
    if (st != CDR_OK) return st;
    if (p->T == 0) return CDR_OK;
    if (!q_latent || !q_rope || !cache || !block_table || !seq_lens || !o || (p->varlen && !cu_seqlens))
        return CDR_ERR_NULL_ARG;
    if (!cdr::aligned16(q_latent) || !cdr::aligned16(q_rope) || !cdr::aligned16(cache) || !cdr::aligned16(o))
        return CDR_ERR_UNSUPPORTED;
    if (!workspace || !cdr::aligned16(workspace) || workspace_bytes < cdr_latent_decode_workspace_bytes(p))
        return CDR_ERR_WORKSPACE;
    cdr::LatentDecodeArgs a;
    a.qc = static_cast<const uint16_t*>(q_latent);
    a.qr = static_cast<const uint16_t*>(q_rope);
    a.cache = static_cast<const uint16_t*>(cache);
    a.table = block_table;
    a.lens = seq_lens;
    a.cu = p->varlen ? cu_seqlens : nullptr;
    a.o = static_cast<uint16_t*>(o);
    a.lse = lse;
    const int m = cdr::dec_m(p);
    const size_t rows = 2 * (size_t)cdr::DEC_GRID * m;
    a.part = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part + rows * cdr::LC);
    a.rec = reinterpret_cast<int4*>(a.part_ml + rows);
    a.qct = p->qc_stride[0], a.qch = p->qc_stride[1];
    a.qrt = p->qr_stride[0], a.qrh = p->qr_stride[1];
    a.N = p->N, a.T = p->T, a.H = p->H;
    a.fill = p->varlen == CDR_VARLEN_FILL;
    a.cols = p->table_cols;
    a.num_pages = p->num_pages;
    a.shift = __builtin_ctz((unsigned)p->page_size);
    a.scale2 = p->scale * cdr::LOG2E;
    // Packed batches have row blocks of no common number: each is a unit of its own, and a sequence's blocks read its
    // keys one after the other (64 sequences of 256 rows, up to 4096 keys: 149 us as a batch, 171 us packed).
    const int64_t blocks = ((int64_t)p->T * p->H + m - 1) / m;
    a.team = p->varlen ? 1 : (int)(blocks < cdr::DEC_TEAM ? blocks : cdr::DEC_TEAM);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = m == 16   ? cdr::launch_latent_decode<1>(a, s)
                         : m == 32 ? cdr::launch_latent_decode<2>(a, s)
                                   : cdr::launch_latent_decode<4>(a, s);
    return e == hipSuccess ? CDR_OK : CDR_ERR_HIP;
}

cdr_status cdr_latent_cache_write(int32_t T, int32_t num_pages, int32_t page_size, const void* c, const void* k_rope,
                                  int64_t c_stride, int64_t k_rope_stride, void* cache, const int32_t* slot_map,
                                  void* stream) {
    if (T < 0 || num_pages <= 0 || page_size <= 0) return CDR_ERR_BAD_SHAPE;
    if (!cdr::mult8(c_stride) || !cdr::mult8(k_rope_stride)) return CDR_ERR_UNSUPPORTED;
    if (T == 0) return CDR_OK;
    if (!c || !k_rope || !cache || !slot_map) return CDR_ERR_NULL_ARG;
    if (!cdr::aligned16(c) || !cdr::aligned16(k_rope) || !cdr::aligned16(cache)) return CDR_ERR_UNSUPPORTED;
    hipLaunchKernelGGL(cdr::latent_write_kernel, dim3((unsigned)(((int64_t)T + 3) / 4)), dim3(256), 0,
                       static_cast<hipStream_t>(stream), static_cast<const uint16_t*>(c),
                       static_cast<const uint16_t*>(k_rope), c_stride, k_rope_stride, static_cast<uint16_t*>(cache),
                       slot_map, T, (int64_t)num_pages * page_size);
    return hipGetLastError() == hipSuccess ? CDR_OK : CDR_ERR_HIP;
}

}  // extern "C"
