// rms_norm.hip — the norm in front of the vocabulary projection (forward with
// the residual's addition, bf16 and / or e4m3 output; backward) and the block
// quantiser.
//
// Mathematics. r = bf16(x + residual); rstd = (mean r^2 + eps)^(-1/2);
// y_j = r_j rstd (o + w_j). A block of 128 columns of y has the scale s =
// max|y| / 448 and q_j = e4m3(y_j / s). Backward, with g_j = dy_j (o + w_j) and
// h_j = r_j rstd: dx_j = rstd (g_j - h_j mean(g h)) + dres_j, dw_j = sum_n dy h.
//
// All of it is bound by memory: a few operations per value of 2 to 14 bytes.
// So a row is read once into registers (packed bf16, 16 bytes per lane and
// load), reduced, and written from there. A row belongs to one workgroup, or to
// one or two waves of it where it is short, so that narrow rows fill the
// lanes too; sums are fp32: per lane over its columns, then an xor-butterfly
// over the wave, then the waves in order.
#include "decode_kernels.h"
#include "host_util.h"

namespace lmhead {

namespace {

__device__ __forceinline__ float bf_lo(uint32_t p) { return __builtin_bit_cast(float, p << 16); }
__device__ __forceinline__ float bf_hi(uint32_t p) { return __builtin_bit_cast(float, p & 0xffff0000u); }

struct F8 {
    float v[8];
};

__device__ __forceinline__ F8 unpack8(const uint4& p) {
    F8 f;
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f.v[2 * i] = bf_lo(w[i]);
        f.v[2 * i + 1] = bf_hi(w[i]);
    }
    return f;
}
__device__ __forceinline__ uint4 pack8(const F8& f) {
    return make_uint4(pack_bf16x2(f.v[0], f.v[1]), pack_bf16x2(f.v[2], f.v[3]), pack_bf16x2(f.v[4], f.v[5]),
                      pack_bf16x2(f.v[6], f.v[7]));
}

// Quotients by one scale, rounded as one fp32 division each: a product with 1 / s
// alone is off by an e4m3 step where the quotient is a tie (153 over 204 / 448 is
// 336, between 320 and 352). Two steps of x inv with the remainder x - q s, which
// one fma gives exactly, reach the rounded quotient when inv is 1 / s rounded to
// nearest and nothing underflows: q s of a q that does not round to 0 holds all
// its bits from s = 2^-90 up. Other scales (a block near the smallest normal number,
// or with an infinity) divide. Norm of 8192 x 4096 to e4m3: 36.7 us so, 36.0 with the
// product alone, 40 to 42 with eight divisions.
struct Quotient {
    float s, inv;
    bool two_steps;
    __device__ __forceinline__ explicit Quotient(float scale)
        : s(scale), inv(1.0f / scale), two_steps(scale >= 0x1p-90f && scale <= 0x1p120f) {}
    __device__ __forceinline__ float step(float x, float q) const {
        return __builtin_fmaf(__builtin_fmaf(-q, s, x), inv, q);
    }
    __device__ __forceinline__ F8 operator()(const F8& f) const {
        F8 q;
        if (two_steps) {
#pragma unroll
            for (int i = 0; i < 8; ++i) q.v[i] = step(f.v[i], step(f.v[i], f.v[i] * inv));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) q.v[i] = f.v[i] / s;
        }
        return q;
    }
};

// e4m3 of eight values over their block's scale
__device__ __forceinline__ uint2 pack_e4m3(const F8& f, const Quotient& over) {
    const F8 q = over(f);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(q.v[4 * i], q.v[4 * i + 1], 0, false);
        v = __builtin_amdgcn_cvt_pk_fp8_f32(q.v[4 * i + 2], q.v[4 * i + 3], v, true);
        w[i] = (uint32_t)v;
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ F8 load_weight8(const void* w, int f32, int i) {
    if (f32) {
        const float4 a = reinterpret_cast<const float4*>(w)[2 * i], b = reinterpret_cast<const float4*>(w)[2 * i + 1];
        return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
    }
    return unpack8(reinterpret_cast<const uint4*>(w)[i]);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
    return v;
}
// over the 16 lanes that hold one block of 128 columns
__device__ __forceinline__ float block_max16(float v) {
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
    return v;
}

// Sum over the WAVES waves of a row; red: one float per wave of the
// workgroup, two sets used in turn so that one barrier per sum is enough.
template <int WAVES>
__device__ __forceinline__ float row_sum(float v, float* red, int wave, int& turn) {
    v = wave_sum(v);
    if (WAVES == 1) return v;
    float* r = red + turn * 16;
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) r[wave] = v;
    __syncthreads();
    const int w0 = wave / WAVES * WAVES;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) s += r[w0 + i];
    return s;
}

constexpr int rows_per_group(int waves) { return waves < 4 ? 4 / waves : 1; }
constexpr int group_threads(int waves) { return 64 * waves * rows_per_group(waves); }

template <int WAVES, int VPT>
__global__ __launch_bounds__(group_threads(WAVES)) void rms_norm_kernel(NormArgs a) {
    constexpr int ROWS = rows_per_group(WAVES), LANES = 64 * WAVES;
    __shared__ float red[32];
    const int wave = threadIdx.x >> 6, slot = wave / WAVES, t = threadIdx.x - slot * LANES;
    const int nv = a.hidden >> 3;
    int turn = 0;
    // every wave of a workgroup makes the same number of trips (barriers inside)
    for (int64_t row0 = (int64_t)blockIdx.x * ROWS; row0 < a.n; row0 += (int64_t)gridDim.x * ROWS) {
        const int64_t row = row0 + slot;
        const bool live = row < a.n;
        const int64_t base = (live ? row : a.n - 1) * nv;   // in vectors of 8
        uint4 r[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = t + j * LANES;
            r[j] = make_uint4(0u, 0u, 0u, 0u);
            if (i < nv) r[j] = reinterpret_cast<const uint4*>(a.x)[base + i];
        }
        if (a.residual != nullptr) {
            uint4 e[VPT];
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = t + j * LANES;
                e[j] = make_uint4(0u, 0u, 0u, 0u);
                if (i < nv) e[j] = reinterpret_cast<const uint4*>(a.residual)[base + i];
            }
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                F8 f = unpack8(r[j]);
                const F8 g = unpack8(e[j]);
#pragma unroll
                for (int c = 0; c < 8; ++c) f.v[c] += g.v[c];
                r[j] = pack8(f);
            }
        }
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const F8 f = unpack8(r[j]);
#pragma unroll
            for (int c = 0; c < 8; ++c) ss = __builtin_fmaf(f.v[c], f.v[c], ss);
        }
        ss = row_sum<WAVES>(ss, red, wave, turn);
        const float rstd = 1.0f / sqrtf(ss / (float)a.hidden + a.eps);
        if (live && t == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = t + j * LANES;
            const bool in = i < nv && live;
            if (in && a.residual_out != nullptr) reinterpret_cast<uint4*>(a.residual_out)[base + i] = r[j];
            if (a.y == nullptr && a.q == nullptr) continue;
            F8 f = unpack8(r[j]);
            const F8 w = load_weight8(a.weight, a.weight_f32, i < nv ? i : 0);
#pragma unroll
            for (int c = 0; c < 8; ++c) f.v[c] = f.v[c] * rstd * (a.offset + w.v[c]);
            if (in && a.y != nullptr) reinterpret_cast<uint4*>(a.y)[base + i] = pack8(f);
            if (a.q != nullptr) {
                float m = 0.0f;
#pragma unroll
                for (int c = 0; c < 8; ++c) m = fmaxf(m, fabsf(f.v[c]));
                const float s = block_scale(block_max16(m));
                const uint2 q = pack_e4m3(f, Quotient(s));
                if (in) {
                    reinterpret_cast<uint2*>(a.q)[base + i] = q;
                    if ((i & 15) == 0) a.scale[(base + i) >> 4] = s;
                }
            }
        }
    }
}

template <int WAVES, int VPT>
__global__ __launch_bounds__(group_threads(WAVES)) void rms_norm_bwd_kernel(NormBwdArgs a) {
    constexpr int ROWS = rows_per_group(WAVES), LANES = 64 * WAVES;
    __shared__ float red[32];
    __shared__ __attribute__((aligned(16))) float join[ROWS > 1 ? (ROWS - 1) * LANES * VPT * 8 : 4];
    const int wave = threadIdx.x >> 6, slot = wave / WAVES, t = threadIdx.x - slot * LANES;
    const int nv = a.hidden >> 3;
    const float inv_h = 1.0f / (float)a.hidden;
    F8 dw[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int c = 0; c < 8; ++c) dw[j].v[c] = 0.0f;
    // The next row's operands are loaded while this one is reduced and written:
    // with two workgroups to a compute unit the loads of one row alone do not
    // cover the memory's latency (16,384 x 4096: 149 us without, 108 us with;
    // 768 or 1024 workgroups: 116 and 121 us). Rows over 16 waves have no registers for it.
    constexpr bool AHEAD = WAVES < 16, KEEP = AHEAD;
    struct Operands {
        uint4 dy[VPT], r[VPT], e[AHEAD ? VPT : 1];
        float rstd;
    };
    const bool want_e = a.dx != nullptr && a.dresidual != nullptr;
    auto load = [&](Operands& o, int64_t row0) {
        const int64_t row = row0 + slot;
        const int64_t base = (row < a.n ? row : a.n - 1) * nv;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = t + j * LANES;
            o.dy[j] = o.r[j] = make_uint4(0u, 0u, 0u, 0u);
            if (AHEAD) o.e[AHEAD ? j : 0] = make_uint4(0u, 0u, 0u, 0u);
            if (i < nv && row < a.n) {
                o.dy[j] = reinterpret_cast<const uint4*>(a.dy)[base + i];
                o.r[j] = reinterpret_cast<const uint4*>(a.r)[base + i];
                if (AHEAD && want_e) o.e[AHEAD ? j : 0] = reinterpret_cast<const uint4*>(a.dresidual)[base + i];
            }
        }
        o.rstd = a.rstd[row < a.n ? row : a.n - 1];
    };
    // o + w of the lane's columns: kept where the registers allow it
    F8 wk[KEEP ? VPT : 1];
    auto weights = [&](int j) {
        const int i = t + j * LANES;
        F8 w = load_weight8(a.weight, a.weight_f32, i < nv ? i : 0);
#pragma unroll
        for (int c = 0; c < 8; ++c) w.v[c] += a.offset;
        return w;
    };
    if (KEEP)
#pragma unroll
        for (int j = 0; j < VPT; ++j) wk[j] = weights(j);
    int turn = 0;
    Operands cur, nxt;
    const int64_t stride = (int64_t)a.groups * ROWS;
    int64_t row0 = (int64_t)blockIdx.x * ROWS;
    if (AHEAD && row0 < a.n) load(cur, row0);
    for (; row0 < a.n; row0 += stride) {
        const int64_t row = row0 + slot;
        const bool live = row < a.n;
        const int64_t base = (live ? row : a.n - 1) * nv;
        if (!AHEAD) load(cur, row0);
        else if (row0 + stride < a.n) load(nxt, row0 + stride);
        const float rstd = cur.rstd;
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const F8 d = unpack8(cur.dy[j]), x = unpack8(cur.r[j]), w = KEEP ? wk[j] : weights(j);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float h = x.v[c] * rstd;
                dot = __builtin_fmaf(d.v[c] * w.v[c], h, dot);
                dw[j].v[c] = __builtin_fmaf(d.v[c], h, dw[j].v[c]);
            }
        }
        if (a.dx != nullptr) {
            const float mean = row_sum<WAVES>(dot, red, wave, turn) * inv_h;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = t + j * LANES;
                if (i >= nv || !live) continue;
                const F8 d = unpack8(cur.dy[j]), x = unpack8(cur.r[j]), w = KEEP ? wk[j] : weights(j);
                F8 o;
#pragma unroll
                for (int c = 0; c < 8; ++c) o.v[c] = rstd * (d.v[c] * w.v[c] - x.v[c] * rstd * mean);
                if (want_e) {
                    const F8 e = unpack8(AHEAD ? cur.e[AHEAD ? j : 0] : reinterpret_cast<const uint4*>(a.dresidual)[base + i]);
#pragma unroll
                    for (int c = 0; c < 8; ++c) o.v[c] += e.v[c];
                }
                reinterpret_cast<uint4*>(a.dx)[base + i] = pack8(o);
            }
        }
        if (AHEAD) cur = nxt;
    }
    if (a.partial == nullptr) return;
    // the row slots' sums in order, then one row of partials per workgroup
    if (ROWS > 1) {
        if (slot > 0)
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int c = 0; c < 8; ++c) join[((slot - 1) * VPT * 8 + j * 8 + c) * LANES + t] = dw[j].v[c];
        __syncthreads();
        if (slot > 0) return;
#pragma unroll
        for (int q = 0; q < ROWS - 1; ++q)
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int c = 0; c < 8; ++c) dw[j].v[c] += join[(q * VPT * 8 + j * 8 + c) * LANES + t];
    }
    float4* out = reinterpret_cast<float4*>(a.partial + (int64_t)blockIdx.x * a.hidden);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = t + j * LANES;
        if (i >= nv) continue;
        out[2 * i] = make_float4(dw[j].v[0], dw[j].v[1], dw[j].v[2], dw[j].v[3]);
        out[2 * i + 1] = make_float4(dw[j].v[4], dw[j].v[5], dw[j].v[6], dw[j].v[7]);
    }
}

// dweight = the groups' partials, 16 interleaved sums per column joined in
// order. One workgroup per 64 columns.
__global__ __launch_bounds__(1024) void dweight_kernel(const float* partial, int groups, int hidden, void* out,
                                                       int f32) {
    __shared__ float s[16][64];
    const int c = threadIdx.x & 63, k = threadIdx.x >> 6;
    const int col = blockIdx.x * 64 + c;   // hidden is a multiple of 64
    float v = 0.0f;
#pragma unroll 8
    for (int g = k; g < groups; g += 16) v += partial[(int64_t)g * hidden + col];
    s[k][c] = v;
    __syncthreads();
    if (k != 0) return;
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) d += s[i][c];
    if (f32)
        reinterpret_cast<float*>(out)[col] = d;
    else
        reinterpret_cast<__bf16*>(out)[col] = (__bf16)d;
}

// One scale per row and 128 columns: 16 lanes hold a block.
__global__ __launch_bounds__(256) void quantize_rows_kernel(const uint4* x, int64_t vectors, uint2* q,
                                                            float* scale) {
    // vectors is a multiple of 16, so the 16 lanes of a block stay together
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < vectors; i += (int64_t)gridDim.x * 256) {
        const F8 f = unpack8(x[i]);
        float m = 0.0f;
#pragma unroll
        for (int c = 0; c < 8; ++c) m = fmaxf(m, fabsf(f.v[c]));
        const float s = block_scale(block_max16(m));
        q[i] = pack_e4m3(f, Quotient(s));
        if ((i & 15) == 0) scale[i >> 4] = s;
    }
}

// One scale per 128 x 128 block, one workgroup per block: 16 lanes take a
// row's 256 bytes, 16 rows at a time, all eight loads in flight; the block
// stays in registers between its maximum and its rounding.
__global__ __launch_bounds__(256) void quantize_blocks_kernel(const bf16_bits* x, int64_t rows, int cols, uint8_t* q,
                                                              float* scale) {
    __shared__ float red[4];
    const int nb = cols / kQBlock;
    const int64_t br = blockIdx.x / nb;
    const int bc = (int)(blockIdx.x - br * nb);
    const int r0 = threadIdx.x >> 4, v = threadIdx.x & 15;
    uint4 d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t row = br * 128 + r0 + 16 * j;
        d[j] = make_uint4(0u, 0u, 0u, 0u);
        if (row < rows) d[j] = *reinterpret_cast<const uint4*>(x + row * cols + bc * kQBlock + v * 8);
    }
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const F8 f = unpack8(d[j]);
#pragma unroll
        for (int c = 0; c < 8; ++c) m = fmaxf(m, fabsf(f.v[c]));
    }
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) m = fmaxf(m, __shfl_xor(m, k));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    const float s = block_scale(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const Quotient over(s);
    if (threadIdx.x == 0) scale[blockIdx.x] = s;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t row = br * 128 + r0 + 16 * j;
        if (row < rows)
            *reinterpret_cast<uint2*>(q + row * cols + bc * kQBlock + v * 8) = pack_e4m3(unpack8(d[j]), over);
    }
}

constexpr int kMaxGrid = 1 << 20;

template <int WAVES, int VPT>
void norm_fwd(const NormArgs& a, hipStream_t s) {
    rms_norm_kernel<WAVES, VPT>
        <<<grid_1d(a.n, rows_per_group(WAVES), kMaxGrid), group_threads(WAVES), 0, s>>>(a);
}
template <int WAVES, int VPT>
void norm_bwd(NormBwdArgs a, hipStream_t s) {
    a.groups = grid_1d(a.n, rows_per_group(WAVES), kNormMaxGroups);
    rms_norm_bwd_kernel<WAVES, VPT><<<a.groups, group_threads(WAVES), 0, s>>>(a);
}

}  // namespace

// Waves per row and vectors per lane by the row's width: two vectors of 8 in
// flight per lane while the row fits 8 waves, more of both above.
void launch_rms_norm(const NormArgs& a, hipStream_t s) {
    if (a.hidden <= 512) norm_fwd<1, 1>(a, s);
    else if (a.hidden <= 1024) norm_fwd<1, 2>(a, s);
    else if (a.hidden <= 2048) norm_fwd<2, 2>(a, s);
    else if (a.hidden <= 4096) norm_fwd<4, 2>(a, s);
    else if (a.hidden <= 8192) norm_fwd<8, 2>(a, s);
    else if (a.hidden <= 16384) norm_fwd<16, 2>(a, s);
    else if (a.hidden <= 32768) norm_fwd<16, 4>(a, s);
    else norm_fwd<16, 8>(a, s);
}

// Groups of the backward at these sizes: min(ceil(n / rows per group), 512).
void launch_rms_norm_bwd(const NormBwdArgs& a, void* dweight, hipStream_t s) {
    int rows = 1;
    if (a.hidden <= 512) norm_bwd<1, 1>(a, s), rows = rows_per_group(1);
    else if (a.hidden <= 1024) norm_bwd<1, 2>(a, s), rows = rows_per_group(1);
    else if (a.hidden <= 2048) norm_bwd<2, 2>(a, s), rows = rows_per_group(2);
    else if (a.hidden <= 4096) norm_bwd<4, 2>(a, s);
    else if (a.hidden <= 8192) norm_bwd<8, 2>(a, s);
    else if (a.hidden <= 16384) norm_bwd<16, 2>(a, s);
    else if (a.hidden <= 32768) norm_bwd<16, 4>(a, s);
    else norm_bwd<16, 8>(a, s);
    if (dweight != nullptr)
        dweight_kernel<<<a.hidden / 64, 1024, 0, s>>>(a.partial, grid_1d(a.n, rows, kNormMaxGroups), a.hidden,
                                                      dweight, a.weight_f32);
}

void launch_quantize(const bf16_bits* x, int64_t rows, int cols, int block_rows, uint8_t* q, float* scale,
                     hipStream_t s) {
    if (block_rows == 1) {
        const int64_t vectors = rows * cols / 8;
        quantize_rows_kernel<<<grid_1d(vectors, 256, 1 << 14), 256, 0, s>>>((const uint4*)x, vectors, (uint2*)q,
                                                                            scale);
    } else {
        quantize_blocks_kernel<<<(unsigned)(cdiv(rows, 128) * (cols / kQBlock)), 256, 0, s>>>(x, rows, cols, q,
                                                                                              scale);
    }
}

}  // namespace lmhead
