// rope.cu -- rotary positions: one tensor of heads, or q and k of a step with
// k and v written to their pages.
//
// The pair i of a head (elements i and i + rot/2 in the half layout, 2i and
// 2i + 1 in the interleaved one) of a token at position p turns by p f_i:
//   (a, b) -> m (a cos - b sin, b cos + a sin);   inverse: sin -> -sin,
// which is the transpose of the rotation, hence its gradient.
//
// The angle is reduced exactly: f_i / (2 pi), a product of two words, becomes a
// fraction of a turn in 64-bit fixed point, and p times it modulo 2^64 is the
// fraction of the turn whatever p is (error p 2^-64 turns; with the product in one
// fp64 word 3.5e-8 turns at p = 2^31).  Its top 32 bits (rounded) are kept, within
// 2^-32 turns in all; the top two of them (rounded) pick the quarter; the rest, at
// most an eighth of a turn, loses nothing that fp32 holds.  bf16 outputs take the
// hardware sine and cosine there (absolute error 2^-21, far below the 2^-9 of the
// rounding); fp32 ones sincospif.
//
// Bound by memory: one read and one write of every element.  A thread keeps
// one unit of every head (two 16-byte vectors that hold whole pairs), so the
// sines of a token are formed once per unit and used for all the heads of its
// slice; neighbouring threads read neighbouring vectors, four heads of them in
// flight (8191 tokens of 32 + 2 x 8 heads appended: 38 us, 81% of the measured
// copy rate; one head in flight 46, eight 56, which need too many registers).
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "launch.h"

namespace asmk {
namespace rope {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // heads in flight per thread

struct View {
    void *p;
    long long st, sh;  // token and head strides, in elements
};

struct Args {
    View x, y;            // q (or the only tensor) and its output
    View k, v;            // append only
    void *kp, *vp;        // append only: [n_pages][Hk][S][d]
    const int *pos, *slot;
    const double *freq;   // [rot / 2]
    int T, H, Hk, d, rot, shift;
    long long n_slots;
    int same;             // y is x: elements beyond rot need no copy
    float ms, sgn;        // factor on cos and sin, -1 for the inverse
};

// fraction of a turn per position, modulo 1, in units of 2^-64
__device__ __forceinline__ unsigned long long turns(double f) {
    constexpr double c0 = 0x1.45f306dc9c883p-3, c1 = -0x1.6b01ec5417056p-57;  // 1 / (2 pi) in two words
    double t = f * c0, e = fma(f, c0, -t) + f * c1;
    t -= rint(t);
    e -= rint(e);
    const unsigned long long hi = t >= 0.5 ? 0x8000000000000000ull
                                           : (unsigned long long)__double2ll_rn(t * 18446744073709551616.0);
    return hi + (unsigned long long)__double2ll_rn(e * 18446744073709551616.0);
}

template <bool FAST>
__device__ __forceinline__ void cos_sin(unsigned long long turn, int p, float ms, float sgn, float &c, float &s) {
    const unsigned f = (unsigned)((turn * (unsigned long long)(long long)p + 0x80000000ull) >> 32);
    const unsigned quarter = (f + 0x20000000u) >> 30;
    const float r = (float)(int)(f - (quarter << 30));  // within an eighth of a turn, units 2^-32
    float sn, cs;
    if (FAST) {
        const float ang = r * 1.4629180792671596e-9f;  // 2 pi / 2^32
        sn = __sinf(ang);
        cs = __cosf(ang);
    } else {
        sincospif(r * 4.6566128730773926e-10f, &sn, &cs);  // 2^-31
    }
    const bool odd = quarter & 1u;
    const float a = odd ? sn : cs, b = odd ? cs : sn;
    c = ((quarter + 1u) & 2u) ? -a * ms : a * ms;
    s = (quarter & 2u) ? -b * (ms * sgn) : b * (ms * sgn);
}

template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    __device__ static void unpack(const uint4 &v, float (&x)[4]) {
        x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    }
    __device__ static uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static void unpack(const uint4 &v, float (&x)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ static uint4 pack(const float (&x)[8]) {
        return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    }
};

// PAIRS: interleaved layout.  A block covers slices x units threads of one
// token at a time; slice s takes heads s, s + S, ...
template <typename T, bool PAIRS, bool APPEND>
__global__ void __launch_bounds__(kThreads)
rope_vec_kernel(const Args a, int units, int slices) {
    constexpr int N = Vec<T>::N;
    const int per_tok = units * slices, toks = kThreads / per_tok;
    const int tid = threadIdx.x;
    if (tid >= toks * per_tok) return;
    const int u = tid % units, s = (tid / units) % slices, tb = tid / per_tok;
    const int ru = a.rot / (2 * N);  // rotated units
    const bool turn = u < ru;
    // the unit's two vectors: element offsets within a head
    const int o0 = turn ? u * N : a.rot + (u - ru) * N;
    const int o1 = turn ? a.rot / 2 + u * N : a.rot + (units - ru) * N + (u - ru) * N;
    unsigned long long w[N];
    if (turn) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            // half: pair o0 + i; interleaved: N/2 pairs of each vector
            const int pair = PAIRS ? (i < N / 2 ? o0 / 2 + i : o1 / 2 + i - N / 2) : o0 + i;
            w[i] = turns(a.freq[pair]);
        }
    }
    for (long long t = (long long)blockIdx.x * toks + tb; t < a.T; t += (long long)gridDim.x * toks) {
        float c[N], sn[N];
        if (turn) {
            const int p = a.pos[t];
#pragma unroll
            for (int i = 0; i < N; ++i) cos_sin<sizeof(T) == 2>(w[i], p, a.ms, a.sgn, c[i], sn[i]);
        }
        auto rotate = [&](uint4 &v0, uint4 &v1) {
            float x[N], y[N], p[N], q[N];
            Vec<T>::unpack(v0, x);
            Vec<T>::unpack(v1, y);
            if (PAIRS) {
#pragma unroll
                for (int i = 0; i < N / 2; ++i) {
                    p[2 * i] = x[2 * i] * c[i] - x[2 * i + 1] * sn[i];
                    p[2 * i + 1] = x[2 * i + 1] * c[i] + x[2 * i] * sn[i];
                    q[2 * i] = y[2 * i] * c[N / 2 + i] - y[2 * i + 1] * sn[N / 2 + i];
                    q[2 * i + 1] = y[2 * i + 1] * c[N / 2 + i] + y[2 * i] * sn[N / 2 + i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    p[i] = x[i] * c[i] - y[i] * sn[i];
                    q[i] = y[i] * c[i] + x[i] * sn[i];
                }
            }
            v0 = Vec<T>::pack(p);
            v1 = Vec<T>::pack(q);
        };
        if (turn || !a.same) {
            const T *x = static_cast<const T *>(a.x.p) + t * a.x.st;
            T *y = static_cast<T *>(a.y.p) + t * a.y.st;
            // kBatch heads' vectors are read before any is written: x and y may be the
            // same, so the compiler would not read ahead of a store
            for (int h0 = s; h0 < a.H; h0 += kBatch * slices) {
                uint4 v[kBatch][2];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int h = h0 + i * slices;
                    if (h >= a.H) break;
                    v[i][0] = *reinterpret_cast<const uint4 *>(x + h * a.x.sh + o0);
                    v[i][1] = *reinterpret_cast<const uint4 *>(x + h * a.x.sh + o1);
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int h = h0 + i * slices;
                    if (h >= a.H) break;
                    if (turn) rotate(v[i][0], v[i][1]);
                    *reinterpret_cast<uint4 *>(y + h * a.y.sh + o0) = v[i][0];
                    *reinterpret_cast<uint4 *>(y + h * a.y.sh + o1) = v[i][1];
                }
            }
        }
        if (APPEND) {
            const long long slot = a.slot[t];
            if (slot >= 0 && slot < a.n_slots) {
                const long long page = slot >> a.shift, off = slot & ((1 << a.shift) - 1);
                const T *k = static_cast<const T *>(a.k.p) + t * a.k.st, *v = static_cast<const T *>(a.v.p) + t * a.v.st;
                for (int h = s; h < a.Hk; h += slices) {
                    const long long dst = (((page * a.Hk + h) << a.shift) + off) * a.d;
                    T *kd = static_cast<T *>(a.kp) + dst, *vd = static_cast<T *>(a.vp) + dst;
                    uint4 v0 = *reinterpret_cast<const uint4 *>(k + h * a.k.sh + o0);
                    uint4 v1 = *reinterpret_cast<const uint4 *>(k + h * a.k.sh + o1);
                    const uint4 w0 = *reinterpret_cast<const uint4 *>(v + h * a.v.sh + o0);
                    const uint4 w1 = *reinterpret_cast<const uint4 *>(v + h * a.v.sh + o1);
                    if (turn) rotate(v0, v1);
                    *reinterpret_cast<uint4 *>(kd + o0) = v0;
                    *reinterpret_cast<uint4 *>(kd + o1) = v1;
                    *reinterpret_cast<uint4 *>(vd + o0) = w0;
                    *reinterpret_cast<uint4 *>(vd + o1) = w1;
                }
            }
        }
    }
}

// Element by element: rotated parts that are no whole number of vectors, and
// rows that are not 16-byte aligned.  One thread per (token, element pair);
// e < rot / 2 turns pair e, the others copy element rot / 2 + e.
template <typename T, bool PAIRS, bool APPEND>
__global__ void __launch_bounds__(kThreads)
rope_any_kernel(const Args a) {
    const int per = a.d - a.rot / 2;
    const long long n = (long long)a.T * per;
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kThreads) {
        const long long t = i / per;
        const int e = (int)(i - t * per);
        const bool turn = e < a.rot / 2;
        const int o0 = turn ? (PAIRS ? 2 * e : e) : a.rot / 2 + e, o1 = PAIRS ? 2 * e + 1 : a.rot / 2 + e;
        float c = 1.f, s = 0.f;
        if (turn) cos_sin<sizeof(T) == 2>(turns(a.freq[e]), a.pos[t], a.ms, a.sgn, c, s);
        auto move = [&](const T *x, T *y) {
            if (!turn) {
                y[o0] = x[o0];
                return;
            }
            const float p = Elem<T>::to_f(x[o0]), q = Elem<T>::to_f(x[o1]);
            y[o0] = Elem<T>::from_f(p * c - q * s);
            y[o1] = Elem<T>::from_f(q * c + p * s);
        };
        const T *x = static_cast<const T *>(a.x.p) + t * a.x.st;
        T *y = static_cast<T *>(a.y.p) + t * a.y.st;
        if (turn || !a.same)
            for (int h = 0; h < a.H; ++h) move(x + h * a.x.sh, y + h * a.y.sh);
        if (APPEND) {
            const long long slot = a.slot[t];
            if (slot >= 0 && slot < a.n_slots) {
                const long long page = slot >> a.shift, off = slot & ((1 << a.shift) - 1);
                for (int h = 0; h < a.Hk; ++h) {
                    const long long dst = (((page * a.Hk + h) << a.shift) + off) * a.d;
                    move(static_cast<const T *>(a.k.p) + t * a.k.st + h * a.k.sh, static_cast<T *>(a.kp) + dst);
                    const T *v = static_cast<const T *>(a.v.p) + t * a.v.st + h * a.v.sh;
                    T *vd = static_cast<T *>(a.vp) + dst;
                    vd[o0] = v[o0];
                    if (turn) vd[o1] = v[o1];
                }
            }
        }
    }
}

template <typename T, bool PAIRS, bool APPEND>
cudaError_t launch(const Args &a, int num_sms, cudaStream_t st) {
    constexpr int N = Vec<T>::N;
    auto vec_ok = [](const View &v) {
        return reinterpret_cast<uintptr_t>(v.p) % 16 == 0 && v.st % N == 0 && v.sh % N == 0;
    };
    const bool vec = a.rot % (2 * N) == 0 && vec_ok(a.x) && vec_ok(a.y) && (!APPEND || (vec_ok(a.k) && vec_ok(a.v)));
    if (!vec) {
        const long long n = (long long)a.T * (a.d - a.rot / 2);
        const long long blocks = (n + kThreads - 1) / kThreads;
        rope_any_kernel<T, PAIRS, APPEND><<<(unsigned)(blocks < 16LL * num_sms ? blocks : 16LL * num_sms), kThreads, 0,
                                            st>>>(a);
        return cudaGetLastError();
    }
    const int units = a.d / (2 * N);
    // Slices per token: one warp's worth, twice as many while that leaves fewer than 128
    // threads per SM (each slice forms the sines again).  Queries of 32 heads, bf16, one
    // warp's worth against the rule: 64 tokens 4.4 us against 3.2, 512 4.7 against 4.0, 1024
    // 4.9 either way; a bound of 2048 threads 6.2 and 10.1 for 512 and 1024.
    int slices = 32 / units;
    while (slices > 1 && slices > a.H) slices /= 2;
    while ((long long)a.T * slices * units < 128LL * num_sms && 2 * slices * units <= kThreads && slices < a.H)
        slices *= 2;
    const int toks = kThreads / (units * slices);
    const long long blocks = ((long long)a.T + toks - 1) / toks;
    const long long most = 8LL * num_sms;  // resident blocks: the turns are formed once per thread
    rope_vec_kernel<T, PAIRS, APPEND><<<(unsigned)(blocks < most ? blocks : most), kThreads, 0, st>>>(a, units, slices);
    return cudaGetLastError();
}

template <bool APPEND>
cudaError_t launch_t(const Args &a, int layout, asm_dtype dt, int num_sms, cudaStream_t st) {
    if (dt == ASM_BF16)
        return layout == ASM_ROPE_PAIRS ? launch<__nv_bfloat16, true, APPEND>(a, num_sms, st)
                                        : launch<__nv_bfloat16, false, APPEND>(a, num_sms, st);
    return layout == ASM_ROPE_PAIRS ? launch<float, true, APPEND>(a, num_sms, st)
                                    : launch<float, false, APPEND>(a, num_sms, st);
}

// Angles per position.  BASE raises the base so that the slowest pair turns
// factor times slower and the fastest as before; BANDS and YARN leave fast
// pairs, slow the others down by factor, and blend between (BANDS linearly in
// the turns made over the trained length, YARN linearly in the pair's index).
__global__ void freqs_kernel(double *freq, int rot, double theta, int scaling, double factor, double lo, double hi,
                             double ctx) {
    constexpr double kTwoPi = 6.283185307179586;
    for (int i = threadIdx.x; i < rot / 2; i += blockDim.x) {
        double base = theta;
        if (scaling == ASM_ROPE_SCALE_BASE) base = theta * pow(factor, (double)rot / (rot > 2 ? rot - 2 : 1));
        double f = pow(base, -2.0 * i / rot);
        if (scaling == ASM_ROPE_SCALE_LINEAR) {
            f /= factor;
        } else if (scaling == ASM_ROPE_SCALE_BANDS) {
            const double w = fmin(1.0, fmax(0.0, (ctx * f / kTwoPi - lo) / (hi - lo)));
            f = (1.0 - w) * f / factor + w * f;
        } else if (scaling == ASM_ROPE_SCALE_YARN) {
            // index of the pair that makes a given number of turns over the trained length
            const double l2 = 2.0 * log(theta);
            double a = floor(rot * log(ctx / (hi * kTwoPi)) / l2), b = ceil(rot * log(ctx / (lo * kTwoPi)) / l2);
            a = fmax(a, 0.0);
            b = fmin(b, rot - 1.0);
            const double ramp = fmin(1.0, fmax(0.0, (i - a) / fmax(b - a, 0.001)));
            f = f / factor * ramp + f * (1.0 - ramp);
        }
        freq[i] = f;
    }
}

}  // namespace rope
}  // namespace asmk

cudaError_t asm_rope_freqs_launch(double *freq, int rot, double theta, int scaling, double factor, double lo,
                                  double hi, double ctx, cudaStream_t st) {
    asmk::rope::freqs_kernel<<<1, 64, 0, st>>>(freq, rot, theta, scaling, factor, lo, hi, ctx);
    return cudaGetLastError();
}

cudaError_t asm_rope_launch(const void *x, int64_t x_st, int64_t x_sh, int T, int H, int d, asm_dtype dt,
                            const int32_t *pos, const double *freq, int rot, int layout, float mscale, int inverse,
                            void *y, int64_t y_st, int64_t y_sh, int num_sms, cudaStream_t st) {
    asmk::rope::Args a{};
    a.x = {const_cast<void *>(x), x_st, x_sh};
    a.y = {y, y_st, y_sh};
    a.pos = pos; a.freq = freq;
    a.T = T; a.H = H; a.d = d; a.rot = rot;
    a.same = x == y;
    a.ms = mscale; a.sgn = inverse ? -1.f : 1.f;
    return asmk::rope::launch_t<false>(a, layout, dt, num_sms, st);
}

cudaError_t asm_rope_append_launch(const void *q, int64_t q_st, int64_t q_sh, const void *k, int64_t k_st,
                                   int64_t k_sh, const void *v, int64_t v_st, int64_t v_sh, int T, int Hq, int Hkv,
                                   int d, asm_dtype dt, const int32_t *pos, const int32_t *slot, const double *freq,
                                   int rot, int layout, float mscale, void *q_out, int64_t o_st, int64_t o_sh,
                                   void *k_pages, void *v_pages, int n_pages, int page_size, int num_sms,
                                   cudaStream_t st) {
    asmk::rope::Args a{};
    a.x = {const_cast<void *>(q), q_st, q_sh};
    a.y = {q_out, o_st, o_sh};
    a.k = {const_cast<void *>(k), k_st, k_sh};
    a.v = {const_cast<void *>(v), v_st, v_sh};
    a.kp = k_pages; a.vp = v_pages;
    a.pos = pos; a.slot = slot; a.freq = freq;
    a.T = T; a.H = Hq; a.Hk = Hkv; a.d = d; a.rot = rot;
    while ((1 << a.shift) < page_size) ++a.shift;
    a.n_slots = (long long)n_pages * page_size;
    a.same = q == q_out;
    a.ms = mscale; a.sgn = 1.f;
    return asmk::rope::launch_t<true>(a, layout, dt, num_sms, st);
}
