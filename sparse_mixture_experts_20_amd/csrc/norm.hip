// Layer norm of token rows and its backward, the norm a pre-norm block puts in
// front of the router:
//
//   h = x + r (rounded to the rows' type and kept; without r: h = x)
//   mean = sum h / d,  var = sum (h - mean)^2 / d,  rstd = 1 / sqrt(var + eps)
//   y = (h - mean) rstd w + b
//   backward: g = dy w, xh = (h - mean) rstd,
//   dx = rstd (g - sum g / d - xh (sum g xh) / d) + dres,
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Both are bound by HBM: a row is read once into registers, reduced there
// (mean first, then the centred squares, so a large mean costs no precision)
// and written from there. A group of TPR threads (a wave, or a workgroup for
// wide rows) holds one row, NV vectors of VEC elements per thread, and walks
// rows b, b + gridDim, ..., the weights staying in its registers and the next
// row's loads issued before the current row is reduced. All sums are fp32.
// The backward's column sums stay in registers over a group's rows; each
// workgroup writes one partial row of dw and db and a second kernel adds the
// partials in order, so the result does not depend on timing.
//
// Measured (8192 x 7168 bf16 with a residual, 470 MB each way): forward 90 us,
// backward 94 + 5 us, 5.2 and 5.0 TB/s, the rate of a large copy on this card
// (5.1). One row of 4096: 3.2 us on the GPU, launch and two reductions.
#include "common.hpp"

namespace moe {
namespace {

// VEC elements of a row: 8 bf16 or 4 fp32 in 16 bytes, or one fp32 (rows whose
// width or base is not a multiple of 16 bytes).
template <typename T, int VEC>
struct Row;
template <>
struct Row<unsigned short, 8> {
    typedef u32x4 Raw;
    static __device__ __forceinline__ void unpack(const Raw &r, float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(r[i] << 16);
            v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ Raw pack(const float (&v)[8]) {
        return Raw{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                   pack_bf16x2(v[6], v[7])};
    }
};
template <>
struct Row<float, 4> {
    typedef f32x4 Raw;
    static __device__ __forceinline__ void unpack(const Raw &r, float (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = r[i];
    }
    static __device__ __forceinline__ Raw pack(const float (&v)[4]) {
        return Raw{v[0], v[1], v[2], v[3]};
    }
};
template <>
struct Row<float, 1> {
    typedef float Raw;
    static __device__ __forceinline__ void unpack(const Raw &r, float (&v)[1]) { v[0] = r; }
    static __device__ __forceinline__ Raw pack(const float (&v)[1]) { return v[0]; }
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        v += __shfl_xor(v, o);
    return v;
}

// Sum over the TPR threads of a row. red: one float per wave; the caller
// alternates buffers, so that one barrier per sum is enough (a buffer is
// written again only after a later sum's barrier, which every reader of the
// first has passed).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *red) {
    v = wave_sum(v);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0)
            red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w)
            v += red[w];
    }
    return v;
}

// Whether a row's loads are issued a row ahead: 16 waves of 16 elements a
// thread have no registers for it (they would spill).
template <int TPR, int ELEMS>
constexpr bool kLoadAhead = TPR < 1024 || ELEMS < 16;

template <typename T, int VEC, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void layer_norm_kernel(
    const T *x, const T *res, const float *__restrict__ w, const float *__restrict__ b, float eps,
    int64_t N, int d, T *h, T *out, float *__restrict__ mean_out, float *__restrict__ rstd_out) {
    typedef Row<T, VEC> R;
    typedef typename R::Raw Raw;
    constexpr int GROUPS = TPR < 256 ? 256 / TPR : 1;
    __shared__ float red[2][TPR / 64];
    const int lt = threadIdx.x % TPR;
    const int nvec = d / VEC;
    const float inv_d = 1.0f / (float)d;
    auto weights = [&](const float *p, int j, float (&o)[VEC]) {
        const int vi = j * TPR + lt;
        if constexpr (VEC >= 4) {
#pragma unroll
            for (int q = 0; q < VEC / 4; ++q) {
                const f32x4 t = vi < nvec
                                    ? *reinterpret_cast<const f32x4 *>(p + (int64_t)vi * VEC + 4 * q)
                                    : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[4 * q + i] = t[i];
            }
        } else {
            o[0] = vi < nvec ? p[vi] : 0.f;
        }
    };
    // rows of up to 1024 threads leave too few registers per lane to keep them
    constexpr bool KEEP = TPR < 1024 && NV * VEC <= 16;
    float wk[KEEP ? NV : 1][VEC], bk[KEEP ? NV : 1][VEC];
    if constexpr (KEEP) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            weights(w, j, wk[j]);
            if (b)
                weights(b, j, bk[j]);
        }
    }
    auto load = [&](const T *p, int64_t row, Raw (&o)[NV]) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int vi = j * TPR + lt;
            o[j] = Raw{};
            if (vi < nvec)
                o[j] = *reinterpret_cast<const Raw *>(p + row * d + (int64_t)vi * VEC);
        }
    };
    const int64_t step = (int64_t)gridDim.x * GROUPS;
    int64_t row = (int64_t)blockIdx.x * GROUPS + threadIdx.x / TPR;
    constexpr bool AHEAD = kLoadAhead<TPR, NV * VEC>;
    Raw xr[NV], rr[NV];
    auto fetch = [&](int64_t r) {
        load(x, r, xr);
        if (res)
            load(res, r, rr);
    };
    if (AHEAD && row < N)
        fetch(row);
    for (; row < N; row += step) {
        if constexpr (!AHEAD)
            fetch(row);
        float v[NV][VEC];
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            R::unpack(xr[j], v[j]);
            if (res) {
                float rv[VEC];
                R::unpack(rr[j], rv);
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    v[j][i] += rv[i];
                // the stream is kept in the rows' type, and it is what is
                // kept that is normalised: the backward sees the same values
                const Raw hp = R::pack(v[j]);
                const int vi = j * TPR + lt;
                if (vi < nvec)
                    *reinterpret_cast<Raw *>(h + row * d + (int64_t)vi * VEC) = hp;
                R::unpack(hp, v[j]);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                s += v[j][i];
        }
        if (AHEAD && row + step < N)
            fetch(row + step);
        const float mean = row_sum<TPR>(s, red[0]) * inv_d;
        float q = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool in = j * TPR + lt < nvec;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                v[j][i] -= mean;
                q += in ? v[j][i] * v[j][i] : 0.f;
            }
        }
        const float rstd = 1.0f / sqrtf(row_sum<TPR>(q, red[1]) * inv_d + eps);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int vi = j * TPR + lt;
            float wv[VEC], bv[VEC];
            if constexpr (!KEEP) {
                weights(w, j, wv);
                if (b)
                    weights(b, j, bv);
            }
            if (vi < nvec) {
                float y[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float wi = KEEP ? wk[KEEP ? j : 0][i] : wv[i];
                    y[i] = v[j][i] * rstd * wi;
                    if (b)
                        y[i] += KEEP ? bk[KEEP ? j : 0][i] : bv[i];
                }
                *reinterpret_cast<Raw *>(out + row * d + (int64_t)vi * VEC) = R::pack(y);
            }
        }
        if (lt == 0) {
            if (mean_out)
                mean_out[row] = mean;
            if (rstd_out)
                rstd_out[row] = rstd;
        }
    }
}

// dx of every row, and per workgroup one partial row of dw and of db
// (part [gridDim.x][2][d]; the waves of a workgroup that hold rows of their
// own are added in wave order through LDS).
template <typename T, int VEC, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void layer_norm_backward_kernel(
    const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ mean_in,
    const float *__restrict__ rstd_in, const T *dout, const T *dres, int64_t N, int d, T *dx,
    float *__restrict__ part) {
    typedef Row<T, VEC> R;
    typedef typename R::Raw Raw;
    constexpr int GROUPS = TPR < 256 ? 256 / TPR : 1;
    __shared__ float red[2][2][TPR / 64];
    __shared__ float cols[GROUPS > 1 ? GROUPS * 2 * TPR * VEC : 1];
    const int lt = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int nvec = d / VEC;
    const float inv_d = 1.0f / (float)d;
    float aw[NV][VEC], ab[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            aw[j][i] = ab[j][i] = 0.f;
    auto weight = [&](int j, float (&o)[VEC]) {
        const int vi = j * TPR + lt;
        if constexpr (VEC >= 4) {
#pragma unroll
            for (int q = 0; q < VEC / 4; ++q) {
                const f32x4 t = vi < nvec
                                    ? *reinterpret_cast<const f32x4 *>(w + (int64_t)vi * VEC + 4 * q)
                                    : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[4 * q + i] = t[i];
            }
        } else {
            o[0] = vi < nvec ? w[vi] : 0.f;
        }
    };
    auto load = [&](const T *p, int64_t row, Raw (&o)[NV]) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int vi = j * TPR + lt;
            o[j] = Raw{};
            if (vi < nvec)
                o[j] = *reinterpret_cast<const Raw *>(p + row * d + (int64_t)vi * VEC);
        }
    };
    const int64_t step = (int64_t)gridDim.x * GROUPS;
    int64_t row = (int64_t)blockIdx.x * GROUPS + grp;
    int parity = 0;
    Raw xr[NV], gr[NV], rr[NV];
    float mean = 0.f, rstd = 0.f;
    constexpr bool AHEAD = kLoadAhead<TPR, NV * VEC>;
    auto fetch = [&](int64_t r) {
        load(x, r, xr);
        load(dout, r, gr);
        if (AHEAD && dres)
            load(dres, r, rr);
        mean = mean_in[r];
        rstd = rstd_in[r];
    };
    if (AHEAD && row < N)
        fetch(row);
    for (; row < N; row += step) {
        if constexpr (!AHEAD)
            fetch(row);
        // xh and g = dy w; the column sums of this row are added at once
        float xh[NV][VEC], g[NV][VEC];
        Raw rc[NV];
        float s1 = 0.f, s2 = 0.f;
        const float rs = rstd;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool in = j * TPR + lt < nvec;
            float wv[VEC];
            weight(j, wv);
            R::unpack(xr[j], xh[j]);
            R::unpack(gr[j], g[j]);
            if constexpr (AHEAD)
                rc[j] = rr[j];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                xh[j][i] = in ? (xh[j][i] - mean) * rs : 0.f;
                aw[j][i] = fmaf(g[j][i], xh[j][i], aw[j][i]);
                ab[j][i] += g[j][i];
                g[j][i] *= wv[i];
                s1 += g[j][i];
                s2 = fmaf(g[j][i], xh[j][i], s2);
            }
        }
        if (AHEAD && row + step < N)
            fetch(row + step);
        s1 = wave_sum(s1);
        s2 = wave_sum(s2);
        if constexpr (TPR > 64) {
            if ((threadIdx.x & 63) == 0) {
                red[parity][0][threadIdx.x >> 6] = s1;
                red[parity][1][threadIdx.x >> 6] = s2;
            }
            __syncthreads();
            s1 = s2 = 0.f;
#pragma unroll
            for (int q = 0; q < TPR / 64; ++q) {
                s1 += red[parity][0][q];
                s2 += red[parity][1][q];
            }
            parity ^= 1;
        }
        const float m1 = s1 * inv_d, m2 = s2 * inv_d;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int vi = j * TPR + lt;
            if (vi < nvec) {
                float o[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    o[i] = rs * (g[j][i] - m1 - xh[j][i] * m2);
                if (dres) {
                    float rv[VEC];
                    if constexpr (!AHEAD)
                        rc[j] = *reinterpret_cast<const Raw *>(dres + row * d + (int64_t)vi * VEC);
                    R::unpack(rc[j], rv);
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        o[i] += rv[i];
                }
                *reinterpret_cast<Raw *>(dx + row * d + (int64_t)vi * VEC) = R::pack(o);
            }
        }
    }
    float *pw = part + (int64_t)blockIdx.x * 2 * d;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int vi = j * TPR + lt;
        if constexpr (GROUPS > 1) {
            // [group][2][TPR * VEC]: this vector's columns of every group
            __syncthreads();
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                cols[(grp * 2 + 0) * TPR * VEC + i * TPR + lt] = aw[j][i];
                cols[(grp * 2 + 1) * TPR * VEC + i * TPR + lt] = ab[j][i];
            }
            __syncthreads();
            for (int c = threadIdx.x; c < 2 * TPR * VEC; c += 256) {
                float s = 0.f;
#pragma unroll
                for (int q = 0; q < GROUPS; ++q)
                    s += cols[q * 2 * TPR * VEC + c];
                const int which = c / (TPR * VEC), i = c % (TPR * VEC) / TPR, l = c % TPR;
                const int v = j * TPR + l;
                if (v < nvec)
                    pw[(int64_t)which * d + (int64_t)v * VEC + i] = s;
            }
        } else if (vi < nvec) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                pw[(int64_t)vi * VEC + i] = aw[j][i];
                pw[d + (int64_t)vi * VEC + i] = ab[j][i];
            }
        }
    }
}

// a[c] and, from column d on, b[c] = sum over P partial rows of ld, each of
// kSumGroups interleaved sets in order and then the sets in order: a chain of
// P / 16 loads (the latency of a chain of P / 4 was most of this kernel's time).
// 64 columns per workgroup.
constexpr int kSumGroups = 16;
__global__ __launch_bounds__(kSumGroups * 64) void column_sums_kernel(
    const float *__restrict__ part, int P, int ld, int d, float *__restrict__ a,
    float *__restrict__ b) {
    __shared__ float red[kSumGroups][64];
    const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    const float *p = part + (int64_t)blockIdx.y * d + c;
    float s = 0.f;
    if (c < d) {
#pragma unroll 8
        for (int r = q; r < P; r += kSumGroups)
            s += p[(int64_t)r * ld];
    }
    red[q][lane] = s;
    __syncthreads();
    if (q == 0 && c < d) {
        float t = red[0][lane];
#pragma unroll
        for (int g = 1; g < kSumGroups; ++g)
            t += red[g][lane];
        (blockIdx.y == 0 ? a : b)[c] = t;
    }
}

// Workgroups of the backward (rows of the partial sums): about one round of
// the 256 CUs. More hide more latency but write and add more partial rows
// (8192x7168 bf16: 97 us at 256, 113 at 512, 136 at 1024).
constexpr int kNormBackwardMax = 512;
constexpr int backward_groups(int threads) { return threads >= 512 ? 256 : kNormBackwardMax; }

// Calls f(<T, VEC, TPR, NV> tag) for the variant that holds a row of d
// elements: waves for narrow rows, a workgroup for wide ones.
template <typename T, int VEC, int TPR, int NV>
struct NormCfg {
    typedef T type;
    static constexpr int vec = VEC, tpr = TPR, nv = NV;
};
template <bool BACKWARD, typename F>
hipError_t with_norm(bool bf16, bool vec, int d, F f) {
    if (bf16) {
        typedef unsigned short u16;
        if (d <= 512) return f(NormCfg<u16, 8, 64, 1>{});
        if (d <= 1024) return f(NormCfg<u16, 8, 64, 2>{});
        // (the backward's column sums take registers: more threads per row;
        // 4096x4096: 34.7 against 37.8 us, the forward 15.8 against 17.4)
        if (BACKWARD && d <= 2048) return f(NormCfg<u16, 8, 256, 1>{});
        if (d <= 4096) return f(NormCfg<u16, 8, BACKWARD ? 512 : 256, BACKWARD ? 1 : 2>{});
        if (d <= 8192) return f(NormCfg<u16, 8, 512, 2>{});
        return f(NormCfg<u16, 8, 1024, 2>{});
    }
    if (vec) {
        if (d <= 512) return f(NormCfg<float, 4, 64, 2>{});
        if (d <= 2048) return f(NormCfg<float, 4, 256, 2>{});
        if (d <= 4096) return f(NormCfg<float, 4, 512, 2>{});
        if (d <= 8192) return f(NormCfg<float, 4, 1024, 2>{});
        return f(NormCfg<float, 4, 1024, 4>{});
    }
    if (d <= 256) return f(NormCfg<float, 1, 64, 4>{});
    if (d <= 1024) return f(NormCfg<float, 1, 256, 4>{});
    if (d <= 4096) return f(NormCfg<float, 1, 1024, 4>{});
    return f(NormCfg<float, 1, 1024, 16>{});
}

}  // namespace

size_t layer_norm_backward_bytes(int64_t N, int64_t d) {
    const int64_t P = N < kNormBackwardMax ? N : kNormBackwardMax;
    return (size_t)(P * 2 * d) * sizeof(float);
}

hipError_t launch_layer_norm(bool bf16, bool vec, const void *x, const void *res, const float *w,
                             const float *b, float eps, int64_t N, int64_t d, void *h, void *out,
                             float *mean, float *rstd, hipStream_t s) {
    return with_norm<false>(bf16, vec, (int)d, [&](auto c) {
        typedef decltype(c) C;
        typedef typename C::type T;
        constexpr int groups = C::tpr < 256 ? 256 / C::tpr : 1;
        const int64_t blocks = (N + groups - 1) / groups;
        // a grid of 2048 threads per CU (256 CUs) walks the rows
        const int64_t most = 2048 * 256 / (C::tpr < 256 ? 256 : C::tpr);
        hipLaunchKernelGGL((layer_norm_kernel<T, C::vec, C::tpr, C::nv>),
                           dim3((unsigned)(blocks < most ? blocks : most)),
                           dim3(C::tpr < 256 ? 256 : C::tpr), 0, s, static_cast<const T *>(x),
                           static_cast<const T *>(res), w, b, eps, N, (int)d,
                           static_cast<T *>(h), static_cast<T *>(out), mean, rstd);
        return hipGetLastError();
    });
}

hipError_t launch_layer_norm_backward(bool bf16, bool vec, const void *x, const float *w,
                                      const float *mean, const float *rstd, const void *dout,
                                      const void *dres, int64_t N, int64_t d, void *dx, float *dw,
                                      float *db, float *part, hipStream_t s) {
    int P = 0;
    hipError_t err = with_norm<true>(bf16, vec, (int)d, [&](auto c) {
        typedef decltype(c) C;
        typedef typename C::type T;
        constexpr int groups = C::tpr < 256 ? 256 / C::tpr : 1;
        const int64_t blocks = (N + groups - 1) / groups;
        const int64_t most = backward_groups(C::tpr);
        P = (int)(blocks < most ? blocks : most);
        hipLaunchKernelGGL((layer_norm_backward_kernel<T, C::vec, C::tpr, C::nv>),
                           dim3((unsigned)P), dim3(C::tpr < 256 ? 256 : C::tpr), 0, s,
                           static_cast<const T *>(x), w, mean, rstd, static_cast<const T *>(dout),
                           static_cast<const T *>(dres), N, (int)d, static_cast<T *>(dx), part);
        return hipGetLastError();
    });
    if (err != hipSuccess)
        return err;
    return launch_column_sums(part, P, 2 * d, d, dw, db, s);
}

hipError_t launch_column_sums(const float *part, int P, int64_t ld, int64_t d, float *a, float *b,
                              hipStream_t s) {
    // a launch has fewer than 2^32 threads: wider sums (the bias gradient of 2^28
    // neurons) go in several
    constexpr int64_t most = (int64_t)1 << 27;
    if (d > most) {
        for (int64_t c = 0; c < d; c += most)
            for (float *o : {a, b}) {
                if (!o)
                    continue;
                const hipError_t err =
                    launch_column_sums(part + (o == b ? d : 0) + c, P, ld,
                                       d - c < most ? d - c : most, o + c, nullptr, s);
                if (err != hipSuccess)
                    return err;
            }
        return hipSuccess;
    }
    hipLaunchKernelGGL(column_sums_kernel, dim3((unsigned)((d + 63) / 64), b ? 2u : 1u),
                       dim3(kSumGroups * 64), 0, s, part, P, (int)ld, (int)d, a, b);
    return hipGetLastError();
}

}  // namespace moe
