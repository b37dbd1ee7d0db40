// rmsnorm_gate_residual: the norm after a block, its gate and residual scale, and the norm
// before the next block, one pass over each row.
//
// A row stays in registers from its one read to its one write: y is squared and summed,
// u and h' are formed in place, h' is squared and summed, z is formed.  Bound by memory
// for many rows (two reads, two writes) and by latency for a few: one load round, two
// reductions, one store round.
//   rows of up to 256 values : one warp per row, no shared memory
//   longer rows              : one CTA per row, 8 values a thread in 32 registers, so that
//                              2048 threads of an SM have their loads in flight; above 8192
//                              values 32 a thread, h being read after the first reduction
// VEC: 16-byte accesses of eight consecutive values (n a multiple of 8, everything 16-byte
// aligned); otherwise the same loop takes single values, a warp's neighbours side by side.
// Measured and not kept (8191 x 2048 bfloat16, 23.6 us as it is, 5.6 TB/s): two rows to a CTA
// 32.7 us, 16 values a thread 25.4 us (fp32 58.5 against 45.5 us), a CTA that walks over rows
// with the next one's loads in flight 35.9 us, each for want of registers; a warp for rows of
// 512 and 1024 (21.4 and 36.8 against 19.0 and 23.8 us for 16384 of them).
#include "kv8.cuh"

namespace qg {
namespace norm {

struct NormParams {
    const void* y;
    const void* h;
    const void* gate;
    const void* w_post;
    const void* w_pre;
    void* h_out;
    void* z;
    long long y_stride, h_stride, gate_stride, h_out_stride, z_stride;
    int rows, n;
    float eps, w_offset, res_scale, inv_n;
};

template <bool VEC, typename T>
__device__ __forceinline__ void load_chunk(const T* row, int first, int step, int n, float (&x)[8]) {
    if constexpr (VEC && sizeof(T) == 4) {
        // spelled out: as pairs of registers the compiler takes them in four 8-byte loads (58 against
        // 46 us for 8191 x 2048 in fp32)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(x[4 * i]), "=f"(x[4 * i + 1]), "=f"(x[4 * i + 2]), "=f"(x[4 * i + 3])
                         : "l"(row + first + 4 * i)
                         : "memory");
    } else if constexpr (VEC) {
        kv8::load8(row + first, x);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = first + e * step < n ? kv8::to_float(row[first + e * step]) : 0.0f;
    }
}
template <bool VEC, typename T>
__device__ __forceinline__ void store_chunk(T* row, int first, int step, int n, const float (&x)[8]) {
    if constexpr (VEC) {
        kv8::store8(row + first, x);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (first + e * step < n) kv8::from_float(x[e], row[first + e * step]);
    }
}

// the sum of v over the row's threads (a warp, or the CTA), in a fixed order
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = warp_sum(v);
    if constexpr (WARP) {
        return v;
    } else {
        const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        return warp_sum(lane < warps ? red[lane] : 0.0f);
    }
}

// IT chunks of eight values per thread, held as pairs (packed fp32 arithmetic: at 8191 x 2048
// the scalar form issued 42 instructions a value and kept the issue slots 80 % busy)
template <typename T, typename R, bool VEC, int IT, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : 1024, WARP ? 16 : IT == 1 && VEC ? 2 : 1) norm_kernel(const NormParams p) {
    __shared__ float red[2][32];
    pdl_wait();
    pdl_launch_dependents();
    const int threads = WARP ? 32 : blockDim.x, tid = WARP ? threadIdx.x & 31 : threadIdx.x;
    const long long row = WARP ? (long long)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= p.rows) return;
    const int n = p.n;
    const T* gate = reinterpret_cast<const T*>(p.gate);
    const T* wpost = reinterpret_cast<const T*>(p.w_post);
    const T* wpre = reinterpret_cast<const T*>(p.w_pre);
    const R* h = reinterpret_cast<const R*>(p.h) + row * p.h_stride;
    using Pair = unsigned long long;
    using kv8::add2;
    using kv8::fma2;
    using kv8::mul2;
    using kv8::pair;

    // chunk i: eight values from place(i), `step` apart; n / 8 whole chunks where VEC
    const int step = VEC ? 1 : threads;
    auto place = [&](int i) { return VEC ? (i * threads + tid) * 8 : i * threads * 8 + tid; };
    auto load = [&](const auto* from, int at, Pair (&x)[4]) {
        float v[8];
        load_chunk<VEC>(from, at, step, n, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = pair(v[2 * e], v[2 * e + 1]);
    };
    auto store = [&](auto* to, int at, const Pair (&x)[4]) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = kv8::unpair(x[e]);
            v[2 * e] = f.x, v[2 * e + 1] = f.y;
        }
        store_chunk<VEC>(to, at, step, n, v);
    };
    auto both = [](Pair s) {
        const float2 f = kv8::unpair(s);
        return f.x + f.y;
    };

    Pair a[IT][4], hv[IT][4];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int at = place(i);
#pragma unroll
        for (int e = 0; e < 4; ++e) a[i][e] = 0ull;
        if (at < n && p.y) load(reinterpret_cast<const T*>(p.y) + row * p.y_stride, at, a[i]);
        if (IT == 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) hv[i][e] = 0ull;
            if (at < n) load(h, at, hv[i]);
        }
    }
    float r = 1.0f;
    if (wpost) {
        Pair s = 0ull;
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s = fma2(a[i][e], a[i][e], s);
        r = rsqrtf(fmaf(row_sum<WARP>(both(s), red[0]), p.inv_n, p.eps));
    }
    Pair s = 0ull;
    {
        const Pair r2 = pair(r, r), off = pair(r * p.w_offset, r * p.w_offset), scale = pair(p.res_scale, p.res_scale);
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int at = place(i);
            if (at >= n) continue;
            Pair c[4];
            if (IT > 1) load(h, at, hv[i]);
            if (wpost) {
                load(wpost, at, c);
#pragma unroll
                for (int e = 0; e < 4; ++e) a[i][e] = mul2(a[i][e], fma2(c[e], r2, off));
            }
            if (gate) {
                load(gate + row * p.gate_stride, at, c);
#pragma unroll
                for (int e = 0; e < 4; ++e) a[i][e] = mul2(a[i][e], c[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[i][e] = mul2(add2(hv[i][e], a[i][e]), scale);  // h'
                s = fma2(a[i][e], a[i][e], s);
            }
            if (p.h_out) store(reinterpret_cast<R*>(p.h_out) + row * p.h_out_stride, at, a[i]);
        }
    }
    if (!wpre) return;
    r = rsqrtf(fmaf(row_sum<WARP>(both(s), red[1]), p.inv_n, p.eps));
    const Pair r2 = pair(r, r), off = pair(r * p.w_offset, r * p.w_offset);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int at = place(i);
        if (at >= n) continue;
        Pair c[4];
        load(wpre, at, c);
#pragma unroll
        for (int e = 0; e < 4; ++e) a[i][e] = mul2(a[i][e], fma2(c[e], r2, off));
        store(reinterpret_cast<T*>(p.z) + row * p.z_stride, at, a[i]);
    }
}

template <typename T, typename R, bool VEC>
static int launch_rows(const NormParams& p, const LaunchCtx& lc) {
    if (p.n <= 256) return launch_kernel(norm_kernel<T, R, VEC, 1, true>, dim3((unsigned)((p.rows + 3) / 4)), dim3(128), 0, lc, p);
    const int it = p.n > 8192 ? 4 : 1;
    const dim3 grid((unsigned)p.rows), block((unsigned)(((p.n + 8 * it - 1) / (8 * it) + 31) & ~31));
    return it == 4 ? launch_kernel(norm_kernel<T, R, VEC, 4, false>, grid, block, 0, lc, p)
                   : launch_kernel(norm_kernel<T, R, VEC, 1, false>, grid, block, 0, lc, p);
}

template <typename T, typename R>
static int launch_types(const NormParams& p, const LaunchCtx& lc) {
    auto rows16 = [](const void* q, long long stride, size_t size) {
        return !q || (((reinterpret_cast<uintptr_t>(q) | (uintptr_t)(stride * (long long)size)) & 15u) == 0);
    };
    const size_t t = sizeof(T), r = sizeof(R);
    const bool vec = p.n % 8 == 0 && rows16(p.y, p.y_stride, t) && rows16(p.h, p.h_stride, r) &&
                     rows16(p.gate, p.gate_stride, t) && rows16(p.w_post, 0, t) && rows16(p.w_pre, 0, t) &&
                     rows16(p.h_out, p.h_out_stride, r) && rows16(p.z, p.z_stride, t);
    return vec ? launch_rows<T, R, true>(p, lc) : launch_rows<T, R, false>(p, lc);
}

}  // namespace norm

int launch_norm(const qg_norm_args& a, const LaunchCtx& lc) {
    using namespace norm;
    const NormParams p = {a.y,        a.h,        a.gate,        a.w_post,       a.w_pre,    a.h_out, a.z,   a.y_stride,
                          a.h_stride, a.gate_stride, a.h_out_stride, a.z_stride, a.rows,  a.n,   a.eps, a.w_offset,
                          a.res_scale, 1.0f / (float)a.n};
    const bool f32_res = a.res_dtype == QG_DTYPE_F32;
    switch (a.dtype) {
        case QG_DTYPE_F32:
            return launch_types<float, float>(p, lc);
        case QG_DTYPE_F16:
            return f32_res ? launch_types<__half, float>(p, lc) : launch_types<__half, __half>(p, lc);
        default:
            return f32_res ? launch_types<__nv_bfloat16, float>(p, lc) : launch_types<__nv_bfloat16, __nv_bfloat16>(p, lc);
    }
}

}  // namespace qg
