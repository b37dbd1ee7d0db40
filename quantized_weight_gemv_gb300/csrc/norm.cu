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
// Two rows to a CTA (twice the loads in flight, half the threads) was slower: 32.7 against
// 26.8 us for 8191 x 2048 in bfloat16; so was a warp for rows of 512 and 1024 (21.4 and 36.8
// against 19.1 and 25.9 us for 16384 of them), and a CTA that walks over rows with the next
// one's loads in flight (35.9 us at 8191 x 2048: 40 registers do not hold both rows).
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
    float eps, w_offset, res_scale;
};

template <bool VEC, typename T>
__device__ __forceinline__ void load_chunk(const T* row, int first, int step, int n, float (&x)[8]) {
    if constexpr (VEC) {
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

// IT chunks of eight values per thread
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

    // chunk i: eight values from place(i), `step` apart; n / 8 whole chunks where VEC
    const int step = VEC ? 1 : threads;
    auto place = [&](int i) { return VEC ? (i * threads + tid) * 8 : i * threads * 8 + tid; };

    float a[IT][8], hv[IT][8];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int at = place(i);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[i][e] = 0.0f;
        if (at < n && p.y) load_chunk<VEC>(reinterpret_cast<const T*>(p.y) + row * p.y_stride, at, step, n, a[i]);
        if (IT == 1) {
#pragma unroll
            for (int e = 0; e < 8; ++e) hv[i][e] = 0.0f;
            if (at < n) load_chunk<VEC>(h, at, step, n, hv[i]);
        }
    }
    float r = 1.0f;
    if (wpost) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(a[i][e], a[i][e], s);
        r = rsqrtf(row_sum<WARP>(s, red[0]) / (float)n + p.eps);
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int at = place(i);
        if (at >= n) continue;
        float c[8];
        if (IT > 1) load_chunk<VEC>(h, at, step, n, hv[i]);
        if (wpost) {
            load_chunk<VEC>(wpost, at, step, n, c);
#pragma unroll
            for (int e = 0; e < 8; ++e) a[i][e] = a[i][e] * r * (c[e] + p.w_offset);
        }
        if (gate) {
            load_chunk<VEC>(gate + row * p.gate_stride, at, step, n, c);
#pragma unroll
            for (int e = 0; e < 8; ++e) a[i][e] *= c[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            a[i][e] = (hv[i][e] + a[i][e]) * p.res_scale;  // h'
            s = fmaf(a[i][e], a[i][e], s);
        }
        if (p.h_out) store_chunk<VEC>(reinterpret_cast<R*>(p.h_out) + row * p.h_out_stride, at, step, n, a[i]);
    }
    if (!wpre) return;
    r = rsqrtf(row_sum<WARP>(s, red[1]) / (float)n + p.eps);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int at = place(i);
        if (at >= n) continue;
        float c[8];
        load_chunk<VEC>(wpre, at, step, n, c);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[i][e] = a[i][e] * r * (c[e] + p.w_offset);
        store_chunk<VEC>(reinterpret_cast<T*>(p.z) + row * p.z_stride, at, step, n, a[i]);
    }
}

template <typename T, typename R, bool VEC>
static int launch_rows(const NormParams& p, const LaunchCtx& lc) {
    if (p.n <= 256) return launch_kernel(norm_kernel<T, R, VEC, 1, true>, dim3((unsigned)((p.rows + 3) / 4)), dim3(128), 0, lc, p);
    const int per = p.n <= 8192 ? 8 : 32;
    const dim3 grid((unsigned)p.rows), block((unsigned)(((p.n + per - 1) / per + 31) & ~31));
    return per == 8 ? launch_kernel(norm_kernel<T, R, VEC, 1, false>, grid, block, 0, lc, p)
                    : launch_kernel(norm_kernel<T, R, VEC, 4, false>, grid, block, 0, lc, p);
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
                          a.res_scale};
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
