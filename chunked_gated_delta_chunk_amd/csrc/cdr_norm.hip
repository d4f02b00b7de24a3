// The block boundary: norm after a token mixer, its gate, the residual, the norm before the next block.
//
//     n = y rstd(y) w            (no weight: n = y)         rstd(x) = 1 / sqrt(mean x^2 + eps)
//     r = x + alpha s a(z) n     (each factor optional)     a(z) = sigmoid(z) or z sigmoid(z)
//     h = r rstd(r) w2           (optional)
//
// and its gradients, with d = dL/dr in total, c(x, p) = p - x^ mean(p x^), x^ = x rstd(x):
//
//     d   = dr + rstd(r) c(r, dh w2)       dw2 = sum_rows dh r^
//     dx  = d                              ds  = sum_rows alpha d a n
//     dz  = alpha d s n a'(z)              dw  = sum_rows alpha d s a y^
//     dy  = rstd(y) c(y, alpha d s a w)    (no weight: dy = alpha d s a)
//
// Both are bound by HBM: every input is read once and every output written once.  A row belongs to
// G threads (16, 64, 256 or 512, the fewest that hold it with eight elements each, sixteen beyond
// 4096) and stays in their registers between the row sums, so the second norm and the backward's
// three reductions cost no second read.  (65536 x 128 with every part, 16, 64 and 256 threads a row:
// forward 15, 38 and 129 us, with gradients 53, 142 and 543; 16384 x 512, 64 and 256: 15.5 and 36, 55 and
// 151; 8192 x 2048, 256 and 512: 32 and 46, the gradients alone 71 and 128; 4096 x 4096, 512 threads with 8
// elements each, 256 with 16 and 512 with 16: 35, 31 and 57, the gradients alone 90, 97 and 239.)  Beyond 4096
// columns the backward's arrays do not all fit the registers: 92 to 180 of a lane's values wait in scratch
// memory, and 2048 x 8192 take 177 us (1.5 TB/s) where 4096 x 4096 take 90 (3.0); forward 44 and 36.
// 8192 x 2048 with an fp32 residual takes 48 us forward, 4.9 TB/s; with gradients, all bf16, 105
// us, 4.2 TB/s, where the backward's three row sums are waited for.  Groups walk over rows with a fixed
// stride, so the weights are loaded once and the backward's column sums stay in registers until the end,
// where each workgroup writes one partial row; a second kernel adds the partial rows in a fixed order (no
// atomics: the same inputs give the same bits).  Everything is computed in fp32; outputs are
// rounded once.  h is the norm of the fp32 r, not of the rounded one.
#include "chunk_dr.h"
#include "cdr_common.h"
#include <type_traits>

namespace cdr {

namespace {

constexpr int NORM_MAX_D = 8192;
constexpr int NORM_PARTS = 512;   // workgroups of the backward, and partial rows of its column sums

struct NormArgs {
    const void* y;
    const void* z;
    const void* x;
    const float* w;
    const float* s;
    const float* w2;
    const void* dr;
    const void* dh;
    void* r;    // forward: out; backward: dx
    void* h;    // forward: next_out; backward: dy
    void* dz;
    float* part;   // [NORM_PARTS, 3, D]: dw, ds, dw2
    int rows, D, inner;
    int64_t yo, yi, zo, zi, xo, xi;   // strides of row (o, i) = o * outer + i * inner
    int act;
    float alpha, eps, inv_d;
};

template <typename T>
struct Elem;
template <>
struct Elem<uint16_t> {
    static __device__ __forceinline__ float get(uint16_t v) { return bf2f(v); }
    static __device__ __forceinline__ uint16_t put(float v) { return f2bf(v); }
};
template <>
struct Elem<float> {
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float v) { return v; }
};

// Elements of a row that a thread holds: with VEC 8, eight neighbours at (c * G + lane) * 8; with
// VEC 1, every G-th one (rows whose width or alignment does not allow 16-byte accesses).
template <int G, int E, int VEC>
struct Row {
    static __device__ __forceinline__ int at(int lane, int e) {
        return VEC == 8 ? ((e >> 3) * G + lane) * 8 + (e & 7) : e * G + lane;
    }
    // A thread's elements as loaded.  All of a row's operands are loaded before the first is
    // unpacked: unpacked one by one inside the bounds check, each waited for the one before (the
    // backward at 8192 x 2048 took 95 us, now 66).
    template <typename T>
    struct Raw {
        static constexpr int N = VEC == 8 ? (sizeof(T) == 2 ? E / 8 : E / 4) : E;
        typedef typename std::conditional<VEC == 8, uint4, T>::type Unit;
        Unit v[N];
        __device__ __forceinline__ void load(const T* p, int lane, int D) {
            if constexpr (VEC == 8) {
                constexpr int PER = sizeof(T) == 2 ? 1 : 2;   // 16-byte units of eight elements
#pragma unroll
                for (int c = 0; c < E / 8; ++c) {
                    const int i = (c * G + lane) * 8;
#pragma unroll
                    for (int u = 0; u < PER; ++u)
                        v[PER * c + u] = i < D ? reinterpret_cast<const uint4*>(p + i)[u] : make_uint4(0, 0, 0, 0);
                }
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int i = e * G + lane;
                    v[e] = i < D ? p[i] : T(0);
                }
            }
        }
        __device__ __forceinline__ void get(float (&f)[E]) const {
            if constexpr (VEC == 8 && sizeof(T) == 2) {
#pragma unroll
                for (int c = 0; c < N; ++c) unpack8(v[c], f + 8 * c);
            } else if constexpr (VEC == 8) {
#pragma unroll
                for (int c = 0; c < N; ++c) {
                    f[4 * c] = __uint_as_float(v[c].x), f[4 * c + 1] = __uint_as_float(v[c].y);
                    f[4 * c + 2] = __uint_as_float(v[c].z), f[4 * c + 3] = __uint_as_float(v[c].w);
                }
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) f[e] = Elem<T>::get(v[e]);
            }
        }
    };
    static __device__ __forceinline__ void load(const float* p, int lane, int D, float (&f)[E]) {
        Raw<float> r;
        r.load(p, lane, D);
        r.get(f);
    }
    template <typename T>
    static __device__ __forceinline__ void store(T* p, int lane, int D, const float (&f)[E]) {
        if constexpr (VEC == 8) {
#pragma unroll
            for (int c = 0; c < E / 8; ++c) {
                const int i = (c * G + lane) * 8;
                if (i >= D) continue;
                if constexpr (sizeof(T) == 2) {
                    const uint4 v = make_uint4(pack_bf2(f[8 * c], f[8 * c + 1]), pack_bf2(f[8 * c + 2], f[8 * c + 3]),
                                               pack_bf2(f[8 * c + 4], f[8 * c + 5]), pack_bf2(f[8 * c + 6], f[8 * c + 7]));
                    *reinterpret_cast<uint4*>(p + i) = v;
                } else {
                    *reinterpret_cast<float4*>(p + i) = make_float4(f[8 * c], f[8 * c + 1], f[8 * c + 2], f[8 * c + 3]);
                    *reinterpret_cast<float4*>(p + i + 4) =
                        make_float4(f[8 * c + 4], f[8 * c + 5], f[8 * c + 6], f[8 * c + 7]);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int i = e * G + lane;
                if (i < D) p[i] = Elem<T>::put(f[e]);
            }
        }
    }
};

// Sums of N values over the G threads of a row, the same in every one of them.  Groups wider than a
// wave exchange through `red` ([2][N * 16]); `turn` alternates its halves, so that one barrier a
// call is enough.
template <int G, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* red, int& turn) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int m = 1; m < (G < 64 ? G : 64); m <<= 1) v[n] += __shfl_xor(v[n], m, 64);
    if constexpr (G > 64) {
        float* buf = red + (turn & 1) * 2 * 16;
        turn ^= 1;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) buf[n * 16 + (threadIdx.x >> 6)] = v[n];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < G / 64; ++i) t += buf[n * 16 + i];
            v[n] = t;
        }
    }
}

__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + ex(-z)); }

template <typename TA>
__device__ __forceinline__ const TA* row_at(const void* base, int row, int inner, int64_t so, int64_t si) {
    const int o = row / inner;
    return static_cast<const TA*>(base) + o * so + (row - o * inner) * si;
}

template <typename TA, typename TR, int G, int E, int VEC>
__global__ __launch_bounds__(G > 256 ? G : 256) void norm_fwd_kernel(NormArgs a) {
    constexpr int WG = G > 256 ? G : 256, RPW = WG / G;
    using R = Row<G, E, VEC>;
    __shared__ float red[64];
    int turn = 0;
    const int lane = threadIdx.x % G;
    const int D = a.D;
    float w[E], s[E], w2[E];
    if (a.w) R::load(a.w, lane, D, w);
    if (a.s) R::load(a.s, lane, D, s);
    if (a.w2) R::load(a.w2, lane, D, w2);
    // Every thread of a workgroup takes the same number of turns (row_sums holds a barrier); rows
    // past the end are computed from row 0 and not stored.
    for (int64_t base = (int64_t)blockIdx.x * RPW; base < a.rows; base += (int64_t)gridDim.x * RPW) {
        const int64_t at = base + threadIdx.x / G;
        const bool live = at < a.rows;
        const int row = live ? (int)at : 0;
        float n[E], z[E], x[E];
        typename R::template Raw<TA> ly, lz;
        typename R::template Raw<TR> lx;
        ly.load(row_at<TA>(a.y, row, a.inner, a.yo, a.yi), lane, D);
        if (a.z) lz.load(row_at<TA>(a.z, row, a.inner, a.zo, a.zi), lane, D);
        if (a.x) lx.load(row_at<TR>(a.x, row, a.inner, a.xo, a.xi), lane, D);
        ly.get(n);
        if (a.z) lz.get(z);
        if (a.x) lx.get(x);
        float k = a.alpha;
        if (a.w) {
            float q[1] = {0.f};
#pragma unroll
            for (int e = 0; e < E; ++e) q[0] += n[e] * n[e];
            row_sums<G, 1>(q, red, turn);
            k *= rsqrtf(q[0] * a.inv_d + a.eps);
#pragma unroll
            for (int e = 0; e < E; ++e) n[e] *= k * w[e];
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) n[e] *= k;
        }
        if (a.s)
#pragma unroll
            for (int e = 0; e < E; ++e) n[e] *= s[e];
        if (a.z) {
            if (a.act == CDR_ACT_SILU) {
#pragma unroll
                for (int e = 0; e < E; ++e) n[e] *= z[e] * sigmoid(z[e]);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) n[e] *= sigmoid(z[e]);
            }
        }
        if (a.x)
#pragma unroll
            for (int e = 0; e < E; ++e) n[e] += x[e];
        if (live) R::store(static_cast<TR*>(a.r) + (size_t)row * D, lane, D, n);
        if (a.w2) {
            float q[1] = {0.f};
#pragma unroll
            for (int e = 0; e < E; ++e) q[0] += n[e] * n[e];
            row_sums<G, 1>(q, red, turn);
            const float rr = rsqrtf(q[0] * a.inv_d + a.eps);
#pragma unroll
            for (int e = 0; e < E; ++e) n[e] *= rr * w2[e];
            if (live) R::store(static_cast<TA*>(a.h) + (size_t)row * D, lane, D, n);
        }
    }
}

template <typename TA, typename TR, int G, int E, int VEC>
__global__ __launch_bounds__(G > 256 ? G : 256) void norm_bwd_kernel(NormArgs a) {
    constexpr int WG = G > 256 ? G : 256, RPW = WG / G;
    using R = Row<G, E, VEC>;
    __shared__ float red[64];
    int turn = 0;
    const int lane = threadIdx.x % G;
    const int D = a.D;
    float w[E], s[E], w2[E];
    if (a.w) R::load(a.w, lane, D, w);
    if (a.s) R::load(a.s, lane, D, s);
    if (a.w2) R::load(a.w2, lane, D, w2);
    const bool silu = a.z && a.act == CDR_ACT_SILU;
    float cw[E], cs[E], cw2[E];   // column sums of the rows that this thread's group takes
#pragma unroll
    for (int e = 0; e < E; ++e) cw[e] = cs[e] = cw2[e] = 0.f;
    for (int64_t base = (int64_t)blockIdx.x * RPW; base < a.rows; base += (int64_t)gridDim.x * RPW) {
        const int64_t at = base + threadIdx.x / G;
        const bool live = at < a.rows;
        const int row = live ? (int)at : 0;
        float y[E], z[E], x[E], d[E], dh[E];
        typename R::template Raw<TA> ly, lz, lh;
        typename R::template Raw<TR> lx, ld;
        ly.load(row_at<TA>(a.y, row, a.inner, a.yo, a.yi), lane, D);
        if (a.z) lz.load(row_at<TA>(a.z, row, a.inner, a.zo, a.zi), lane, D);
        if (a.x && a.w2) lx.load(row_at<TR>(a.x, row, a.inner, a.xo, a.xi), lane, D);
        if (a.dr) ld.load(static_cast<const TR*>(a.dr) + (size_t)row * D, lane, D);
        if (a.w2) lh.load(static_cast<const TA*>(a.dh) + (size_t)row * D, lane, D);
        ly.get(y);
        if (a.z) lz.get(z);
        if (a.x && a.w2) lx.get(x);
        if (a.dr) ld.get(d);
        if (a.w2) lh.get(dh);
#pragma unroll
        for (int e = 0; e < E; ++e) {   // rows past the end have no gradients
            d[e] = a.dr && live ? d[e] : 0.f;
            dh[e] = a.w2 && live ? dh[e] : 0.f;
        }
        float ry = 1.f;
        if (a.w) {
            float q[1] = {0.f};
#pragma unroll
            for (int e = 0; e < E; ++e) q[0] += y[e] * y[e];
            row_sums<G, 1>(q, red, turn);
            ry = rsqrtf(q[0] * a.inv_d + a.eps);
        }
        // y^ from here on, and the gate's sigmoid
        float sg[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            y[e] *= ry;
            sg[e] = a.z ? sigmoid(z[e]) : 1.f;
        }
        if (a.w2) {
            // r again, then d += rstd(r) c(r, dh w2)
            float r[E];
            float q[2] = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float t = a.alpha * y[e] * sg[e];
                if (a.w) t *= w[e];
                if (a.s) t *= s[e];
                if (silu) t *= z[e];
                if (a.x) t += x[e];
                r[e] = t;
                q[0] += t * t;
                q[1] += t * dh[e] * w2[e];
            }
            row_sums<G, 2>(q, red, turn);
            const float rr = rsqrtf(q[0] * a.inv_d + a.eps);
            const float m = q[1] * rr * a.inv_d;   // mean of dh w2 r^
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float hat = r[e] * rr;
                cw2[e] += dh[e] * hat;
                d[e] += rr * (dh[e] * w2[e] - hat * m);
            }
        }
        if (a.r && live) R::store(static_cast<TR*>(a.r) + (size_t)row * D, lane, D, d);
        // p = d alpha s a, the gradient of n; z becomes dz
        float q[1] = {0.f};
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float g = silu ? z[e] * sg[e] : sg[e];
            const float slope = sg[e] * (silu ? 1.f + z[e] * (1.f - sg[e]) : 1.f - sg[e]);
            const float n = a.w ? y[e] * w[e] : y[e];
            const float da = a.alpha * d[e];
            if (a.s) cs[e] += da * g * n;
            const float ds = a.s ? da * s[e] : da;
            if (a.z) z[e] = ds * n * slope;
            float p = ds * g;
            if (a.w) {
                cw[e] += p * y[e];
                p *= w[e];
                q[0] += p * y[e];
            }
            d[e] = p;
        }
        if (a.dz && live) R::store(static_cast<TA*>(a.dz) + (size_t)row * D, lane, D, z);
        if (a.w) {
            row_sums<G, 1>(q, red, turn);
            const float m = q[0] * a.inv_d;
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] = ry * (d[e] - y[e] * m);
        }
        if (live) R::store(static_cast<TA*>(a.h) + (size_t)row * D, lane, D, d);
    }
    // one partial row a workgroup, the groups of a workgroup added in their order
    if constexpr (RPW == 1) {
        float* p = a.part + (size_t)blockIdx.x * 3 * D;
        if (a.w) R::store(p, lane, D, cw);
        if (a.s) R::store(p + D, lane, D, cs);
        if (a.w2) R::store(p + 2 * (size_t)D, lane, D, cw2);
    } else {
        __shared__ float cols[RPW][G * E];
        float* p = a.part + (size_t)blockIdx.x * 3 * D;
        const int g = threadIdx.x / G;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const bool wanted = k == 0 ? a.w != nullptr : k == 1 ? a.s != nullptr : a.w2 != nullptr;
            if (!wanted) continue;
            __syncthreads();
#pragma unroll
            for (int e = 0; e < E; ++e) cols[g][R::at(lane, e)] = k == 0 ? cw[e] : k == 1 ? cs[e] : cw2[e];
            __syncthreads();
            for (int i = threadIdx.x; i < D; i += WG) {
                float t = 0.f;
#pragma unroll
                for (int j = 0; j < RPW; ++j) t += cols[j][i];
                p[(size_t)k * D + i] = t;
            }
        }
    }
}

// Column sums of the partial rows: 64 columns a workgroup, sixteen threads a column that each add every
// sixteenth partial row, their sums added in order.  blockIdx.y names the vector.  (With four threads
// a column the chain of dependent loads took 38 us at 2048 columns, as long as the data's own pass.)
__global__ __launch_bounds__(1024) void norm_cols_kernel(const float* part, int parts, int D, float* dw, float* ds,
                                                         float* dw2) {
    float* out = blockIdx.y == 0 ? dw : blockIdx.y == 1 ? ds : dw2;
    if (out == nullptr) return;
    __shared__ float sums[16][64];
    const int c = blockIdx.x * 64 + (threadIdx.x & 63), k = threadIdx.x >> 6;
    float t = 0.f;
    if (c < D)
#pragma unroll 8
        for (int i = k; i < parts; i += 16) t += part[((size_t)i * 3 + blockIdx.y) * D + c];
    sums[k][threadIdx.x & 63] = t;
    __syncthreads();
    if (k == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < 16; ++i) t += sums[i][c & 63];
        out[c] = t;
    }
}

int64_t bwd_parts(const cdr_block_norm_problem* p) {
    const int g = p->D <= 128 ? 16 : p->D <= 512 ? 64 : 256;   // rows a workgroup takes at once: 256 / g
    const int64_t groups = ((int64_t)p->rows + 256 / g - 1) / (256 / g);
    return groups < NORM_PARTS ? groups : NORM_PARTS;
}

template <typename TA, typename TR, int G, int E, int VEC>
void launch_one(bool bwd, const NormArgs& a, int64_t parts, hipStream_t s) {
    constexpr int WG = G > 256 ? G : 256, RPW = WG / G;
    if (bwd) {
        hipLaunchKernelGGL((norm_bwd_kernel<TA, TR, G, E, VEC>), dim3((unsigned)parts), dim3(WG), 0, s, a);
    } else {
        const int64_t groups = ((int64_t)a.rows + RPW - 1) / RPW;
        hipLaunchKernelGGL((norm_fwd_kernel<TA, TR, G, E, VEC>), dim3((unsigned)(groups < 2048 ? groups : 2048)),
                           dim3(WG), 0, s, a);
    }
}

template <typename TA, typename TR, int VEC>
void launch_width(bool bwd, const NormArgs& a, int64_t parts, hipStream_t s) {
    if (a.D <= 128) launch_one<TA, TR, 16, 8, VEC>(bwd, a, parts, s);
    else if (a.D <= 512) launch_one<TA, TR, 64, 8, VEC>(bwd, a, parts, s);
    else if (a.D <= 2048) launch_one<TA, TR, 256, 8, VEC>(bwd, a, parts, s);
    else if (a.D <= 4096) launch_one<TA, TR, 512, 8, VEC>(bwd, a, parts, s);
    else launch_one<TA, TR, 512, 16, VEC>(bwd, a, parts, s);
}

template <typename TA, typename TR>
void launch_vec(bool bwd, const NormArgs& a, int64_t parts, bool vec, hipStream_t s) {
    if (vec) launch_width<TA, TR, 8>(bwd, a, parts, s);
    else launch_width<TA, TR, 1>(bwd, a, parts, s);
}

bool has_out_res(const cdr_block_norm_problem* p) { return p->has_residual != 0; }

NormArgs norm_args(const cdr_block_norm_problem* p) {
    NormArgs a = {};
    a.rows = p->rows;
    a.D = p->D;
    a.inner = p->inner > 0 ? p->inner : 1;
    a.yo = p->y_stride[0], a.yi = p->y_stride[1];
    a.zo = p->gate_stride[0], a.zi = p->gate_stride[1];
    a.xo = p->residual_stride[0], a.xi = p->residual_stride[1];
    a.act = p->gate_act;
    a.alpha = p->alpha;
    a.eps = p->eps;
    a.inv_d = 1.f / (float)p->D;
    return a;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

void launch_norm(bool bwd, const cdr_block_norm_problem* p, const NormArgs& a, int64_t parts, hipStream_t s) {
    // 16-byte accesses: every row of every operand starts at a multiple of 16 bytes
    const int64_t odd = (a.yo | a.yi | (a.z ? a.zo | a.zi : 0) | (a.x ? a.xo | a.xi : 0)) & 7;
    const bool vec = p->D % 8 == 0 && odd == 0 && aligned16(a.y) && aligned16(a.z) && aligned16(a.x) && aligned16(a.w) &&
                     aligned16(a.s) && aligned16(a.w2) && aligned16(a.dr) && aligned16(a.dh) && aligned16(a.r) &&
                     aligned16(a.h) && aligned16(a.dz) && aligned16(a.part);
    const bool ab = p->dtype == CDR_BF16;
    const bool rb = has_out_res(p) ? p->res_dtype == CDR_BF16 : ab;
    if (ab && rb) launch_vec<uint16_t, uint16_t>(bwd, a, parts, vec, s);
    else if (ab) launch_vec<uint16_t, float>(bwd, a, parts, vec, s);
    else if (rb) launch_vec<float, uint16_t>(bwd, a, parts, vec, s);
    else launch_vec<float, float>(bwd, a, parts, vec, s);
}

}  // namespace

}  // namespace cdr

extern "C" {

cdr_status cdr_block_norm_check(const cdr_block_norm_problem* p) {
    if (p == nullptr) return CDR_ERR_NULL_ARG;
    if (p->rows < 0 || p->D <= 0 || p->inner < 0) return CDR_ERR_BAD_SHAPE;
    if (p->inner > 1 && p->rows % p->inner != 0) return CDR_ERR_BAD_SHAPE;
    if (p->D > cdr::NORM_MAX_D) return CDR_ERR_UNSUPPORTED;
    if (p->dtype != CDR_BF16 && p->dtype != CDR_F32) return CDR_ERR_UNSUPPORTED;
    if (p->has_residual && p->res_dtype != CDR_BF16 && p->res_dtype != CDR_F32) return CDR_ERR_UNSUPPORTED;
    if (p->gate_act != CDR_ACT_NONE && p->gate_act != CDR_ACT_SIGMOID && p->gate_act != CDR_ACT_SILU)
        return CDR_ERR_UNSUPPORTED;
    if (!(p->eps >= 0.f)) return CDR_ERR_BAD_SHAPE;
    return CDR_OK;
}

cdr_status cdr_block_norm_fwd(const cdr_block_norm_problem* p, const void* y, const void* gate, const void* residual,
                              const float* weight, const float* res_scale, const float* next_weight, void* out,
                              void* next_out, void* stream) {
    const cdr_status st = cdr_block_norm_check(p);
    if (st != CDR_OK) return st;
    if (p->rows == 0) return CDR_OK;
    if (!y || !out) return CDR_ERR_NULL_ARG;
    if ((p->gate_act != CDR_ACT_NONE && !gate) || (p->has_residual && !residual) || (p->has_weight && !weight) ||
        (p->has_scale && !res_scale) || (p->has_next && (!next_weight || !next_out)))
        return CDR_ERR_NULL_ARG;
    cdr::NormArgs a = cdr::norm_args(p);
    a.y = y;
    a.z = p->gate_act != CDR_ACT_NONE ? gate : nullptr;
    a.x = p->has_residual ? residual : nullptr;
    a.w = p->has_weight ? weight : nullptr;
    a.s = p->has_scale ? res_scale : nullptr;
    a.w2 = p->has_next ? next_weight : nullptr;
    a.r = out;
    a.h = p->has_next ? next_out : nullptr;
    cdr::launch_norm(false, p, a, 0, static_cast<hipStream_t>(stream));
    return hipGetLastError() == hipSuccess ? CDR_OK : CDR_ERR_HIP;
}

size_t cdr_block_norm_bwd_workspace_bytes(const cdr_block_norm_problem* p) {
    if (cdr_block_norm_check(p) != CDR_OK) return 0;
    return (size_t)cdr::bwd_parts(p) * 3 * (size_t)p->D * sizeof(float);
}

cdr_status cdr_block_norm_bwd(const cdr_block_norm_problem* p, const void* y, const void* gate, const void* residual,
                              const float* weight, const float* res_scale, const float* next_weight, const void* d_out,
                              const void* d_next, void* dy, void* dgate, void* dresidual, float* dweight,
                              float* dres_scale, float* dnext_weight, void* workspace, size_t workspace_bytes,
                              void* stream) {
    const cdr_status st = cdr_block_norm_check(p);
    if (st != CDR_OK) return st;
    if ((p->has_weight && (!weight || !dweight)) || (p->has_scale && (!res_scale || !dres_scale)) ||
        (p->has_next && (!next_weight || !dnext_weight)))
        return CDR_ERR_NULL_ARG;
    if (p->rows > 0 && (!y || !dy || (p->gate_act != CDR_ACT_NONE && (!gate || !dgate)) ||
                        (p->has_residual && (!residual || !dresidual)) || (p->has_next && !d_next) ||
                        (!p->has_next && !d_out)))
        return CDR_ERR_NULL_ARG;
    const size_t need = cdr_block_norm_bwd_workspace_bytes(p);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return CDR_ERR_WORKSPACE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t parts = cdr::bwd_parts(p);
    float* part = static_cast<float*>(workspace);
    if (p->rows > 0) {
        cdr::NormArgs a = cdr::norm_args(p);
        a.y = y;
        a.z = p->gate_act != CDR_ACT_NONE ? gate : nullptr;
        a.x = p->has_residual ? residual : nullptr;
        a.w = p->has_weight ? weight : nullptr;
        a.s = p->has_scale ? res_scale : nullptr;
        a.w2 = p->has_next ? next_weight : nullptr;
        a.dr = d_out;
        a.dh = p->has_next ? d_next : nullptr;
        a.r = p->has_residual ? dresidual : nullptr;
        a.h = dy;
        a.dz = p->gate_act != CDR_ACT_NONE ? dgate : nullptr;
        a.part = part;
        cdr::launch_norm(true, p, a, parts, s);
        if (hipGetLastError() != hipSuccess) return CDR_ERR_HIP;
    }
    if (p->has_weight || p->has_scale || p->has_next) {
        hipLaunchKernelGGL(cdr::norm_cols_kernel, dim3((unsigned)((p->D + 63) / 64), 3), dim3(1024), 0, s, part, (int)parts,
                           p->D, p->has_weight ? dweight : nullptr, p->has_scale ? dres_scale : nullptr,
                           p->has_next ? dnext_weight : nullptr);
        if (hipGetLastError() != hipSuccess) return CDR_ERR_HIP;
    }
    return CDR_OK;
}

}  // extern "C"
