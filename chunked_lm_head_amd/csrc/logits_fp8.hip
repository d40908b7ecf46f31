// logits_fp8.hip — logits from e4m3 rows and an e4m3 vocabulary matrix with a
// scale per block of 128 columns (rows) or 128 x 128 (W):
//   out[i, v] = sum_b sa[i, b] sw[v / 128, b] sum_{j in b} a[i, j] w[v, j].
//
// Precision. The 8-bit matrix instructions align each 8 consecutive products
// to the largest of them and cut the others off 13 bits below its power of two
// (measured; products further down vanish), which leaves a block's sum up to
// 8 * 2^-13 of each eight's largest product off, 1.5e-5 in the 2-norm. A bf16
// output, rounded to 2^-9, takes them; an fp32 output does not: there the e4m3
// values are widened to bf16 (exact: 4 significant bits) and multiplied by
// v_mfma_f32_16x16x32_bf16, whose products and sums keep fp32 precision. A
// block's sum is added to the fp32 accumulator after the two scales.
//
// Few rows (up to kStreamRows): the W stream from memory decides (Hd bytes per
// vocabulary row and pass). Waves read W fragments straight into registers,
// and the four waves of a workgroup take a quarter of the columns each, so a
// workgroup is small enough to spread evenly over the chip and nothing is
// staged or waited for inside the loop; their sums are joined in wave order
// through LDS. More rows: the matrix instructions decide, on 256-row tiles.
#include "decode_kernels.h"
#include "host_util.h"

namespace lmhead {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// four e4m3 values to bf16 (gfx950's packed conversion, scale 1)
__device__ __forceinline__ void widen4(uint32_t v, bf16x8& f, int at) {
    const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false);
    const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true);
    f[at] = lo[0], f[at + 1] = lo[1], f[at + 2] = hi[0], f[at + 3] = hi[1];
}

// A 16 x 128 operand block: lane l holds row l % 16, bytes 16 (l / 16) .. + 16
// of each 64-byte half. Both operands use the same order of k, so the sum over
// k does not depend on it, and a lane's two 16-byte loads sit in lines that
// the four lanes of its row read whole.
struct Frag {
    u32x4 lo, hi;
    // the 16 x 32 bf16 fragment of quarter s
    __device__ __forceinline__ bf16x8 part(int s) const {
        const uint32_t w[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        bf16x8 f;
        widen4(w[2 * s], f, 0);
        widen4(w[2 * s + 1], f, 4);
        return f;
    }
    __device__ __forceinline__ i32x8 all() const {
        return __builtin_bit_cast(i32x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};
struct Wide {
    bf16x8 p[4];
    __device__ __forceinline__ Wide(const Frag& f) {
#pragma unroll
        for (int s = 0; s < 4; ++s) p[s] = f.part(s);
    }
};

__device__ __forceinline__ floatx4 block_sum(const Wide& a, const Wide& b) {
    floatx4 z = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < 4; ++s) z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[s], b.p[s], z, 0, 0, 0);
    return z;
}
__device__ __forceinline__ floatx4 block_sum(const i32x8& a, const i32x8& b) {
    const floatx4 z = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, z, 0, 0, 0, 0, 0, 0);
}

// ------------------------------------------------------------- few rows

constexpr int kStreamRows = 128;
constexpr int kStreamWaves = 4;

__device__ __forceinline__ void store_out(const LogitsArgs& a, int64_t at, float v) {
    if (a.out_f32)
        reinterpret_cast<float*>(a.out)[at] = v;
    else
        reinterpret_cast<__bf16*>(a.out)[at] = (__bf16)v;
}

// One workgroup: VT * 16 vocabulary rows x all (NT * 16) input rows.
template <int VT, int NT>
__global__ __launch_bounds__(64 * kStreamWaves) void logits_stream_kernel(LogitsArgs a) {
    constexpr int kV = 16 * VT, kN = 16 * NT, kPitch = kV + 4;
    __shared__ __attribute__((aligned(16))) float part[kStreamWaves][kN][kPitch];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int64_t v0 = (int64_t)blockIdx.x * kV;
    const int nb = a.hidden / kQBlock;
    const int b0 = nb * wave / kStreamWaves, b1 = nb * (wave + 1) / kStreamWaves;
    const uint8_t* w[VT];
    const uint8_t* x[NT];
    const float* sa[NT];
#pragma unroll
    for (int i = 0; i < VT; ++i) {
        const int64_t r = v0 + 16 * i + c;
        w[i] = a.w + (r < a.vocab ? r : a.vocab - 1) * a.hidden + 16 * g;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int64_t r = 16 * j + c;
        const int64_t rc = r < a.n ? r : a.n - 1;
        x[j] = a.a + rc * a.hidden + 16 * g;
        sa[j] = a.a_scale + rc * nb;
    }
    const float* sw = a.w_scale + (v0 / kQBlock) * nb;   // kV divides 128: one block of rows
    floatx4 acc[VT][NT];
#pragma unroll
    for (int i = 0; i < VT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    Frag fw[VT];
    auto load_w = [&](Frag (&f)[VT], int b) {
#pragma unroll
        for (int i = 0; i < VT; ++i) {
            f[i].lo = *reinterpret_cast<const u32x4*>(w[i] + b * kQBlock);
            f[i].hi = *reinterpret_cast<const u32x4*>(w[i] + b * kQBlock + 64);
        }
    };
    if (b0 < b1) load_w(fw, b0);
    for (int b = b0; b < b1; ++b) {
        Frag nw[VT];
        load_w(nw, b + 1 < b1 ? b + 1 : b);
        const float s0 = sw[b];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            Frag fx;
            fx.lo = *reinterpret_cast<const u32x4*>(x[j] + b * kQBlock);
            fx.hi = *reinterpret_cast<const u32x4*>(x[j] + b * kQBlock + 64);
            const float s = sa[j][b] * s0;
            const Wide wx(fx);
#pragma unroll
            for (int i = 0; i < VT; ++i) {
                const floatx4 z = block_sum(Wide(fw[i]), wx);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(z[e], s, acc[i][j][e]);
            }
        }
#pragma unroll
        for (int i = 0; i < VT; ++i) fw[i] = nw[i];
    }
    // lane: vocabulary rows 16 i + 4 g .. + 4 of input row 16 j + c
#pragma unroll
    for (int i = 0; i < VT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            *reinterpret_cast<floatx4*>(&part[wave][16 * j + c][16 * i + 4 * g]) = acc[i][j];
    __syncthreads();
    const int rows = a.n < kN ? (int)a.n : kN;
    for (int q = threadIdx.x; q < rows * kV; q += 64 * kStreamWaves) {
        const int r = q / kV, v = q % kV;
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < kStreamWaves; ++k) s += part[k][r][v];
        if (v0 + v < a.vocab) store_out(a, r * a.ld + v0 + v, s);
    }
}

template <int VT, int NT>
void stream(const LogitsArgs& a, hipStream_t s) {
    logits_stream_kernel<VT, NT><<<(unsigned)cdiv(a.vocab, 16 * VT), 64 * kStreamWaves, 0, s>>>(a);
}

// ------------------------------------------------------------- many rows

// The rows packed for the tile kernel: 16-row x 128-column blocks of 2 KB in
// fragment order (the lanes' low 16 bytes, then their high ones), block (i /
// 16, b) at ((i / 16) nb + b) * 2 KB, rows up to n_pad zero; and the scales
// transposed, [nb][n_pad].
__global__ __launch_bounds__(256) void pack_rows_kernel(const uint8_t* a, const float* a_scale, int64_t n,
                                                        int64_t n_pad, int hidden, uint8_t* out, float* scale_t) {
    const int nb = hidden / kQBlock;
    const int64_t pieces = n_pad * hidden / 16, scales = n_pad * nb;
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < pieces; q += step) {
        const int64_t blk = q >> 7;
        const int l = (int)(q & 63), half = (int)(q >> 6) & 1;
        const int64_t row = blk / nb * 16 + (l & 15);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (row < n)
            v = *reinterpret_cast<const uint4*>(a + row * hidden + blk % nb * kQBlock + 64 * half + 16 * (l >> 4));
        reinterpret_cast<uint4*>(out)[q] = v;
    }
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < scales; q += step) {
        const int64_t b = q / n_pad, row = q - b * n_pad;
        scale_t[q] = row < n ? a_scale[row * nb + b] : 0.0f;
    }
}

constexpr int kTileRows = 256;       // input rows of a tile
constexpr int kTileThreads = 512;    // eight waves: 2 along the vocabulary, 4 along the rows
constexpr int kStages = 4;

struct TileArgs {
    LogitsArgs p;
    const uint8_t* rows;    // packed (pack_rows_kernel)
    const float* scale_t;
    int64_t n_pad, tiles_n, tiles_v;
};

// One workgroup: 256 input rows x 32 VI vocabulary rows (2 VI fragments of 16).
// W goes through LDS: one 128-column step of the tile is rows of 128 bytes,
// 16-byte chunk q of row r at q ^ ((r >> 1) & 7) (conflict-free fragment
// reads), written by LDS-direct buffer loads, four steps in a ring. The rows'
// fragments come straight from the packed copy into registers, a step ahead.
// In a step a wave issues the next step's row fragments first and then the W
// loads of step b + 3: waiting for the former at the next step's start leaves
// only the latter in flight, so W of step b + 1 has landed for every wave that
// has begun step b, and one barrier per step is enough.
template <bool EXACT, int VI>
__global__ __launch_bounds__(kTileThreads, 1) void logits_tile_kernel(TileArgs t) {
    constexpr int kV = 32 * VI, kStage = kV * 128, kLoads = kStage / (kTileThreads * 16);
    __shared__ __attribute__((aligned(16))) char smem[kStages * kStage];
    const LogitsArgs& a = t.p;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wv = wave & 1, wn = wave >> 1;
    const int c = lane & 15, g = lane >> 4;
    int64_t tn, tv;
    map_tile(blockIdx.x, t.tiles_n, t.tiles_v, tn, tv);
    const int64_t v0 = tv * kV;
    const int nb = a.hidden / kQBlock;
    const int64_t vrows = a.vocab - v0 < kV ? a.vocab - v0 : kV;
    // W rows past the vocabulary read as zero (buffer range)
    const __amdgpu_buffer_rsrc_t rw =
        __builtin_amdgcn_make_buffer_rsrc((void*)(a.w + v0 * a.hidden), 0, (int)(vrows * a.hidden), 0x00020000);
    // load u of a wave: LDS rows 8 (kLoads w + u) .. + 8 in lane order; row r + 8 has swizzle(r) ^ 4
    const int lr = wave * 8 * kLoads + (lane >> 3);
    const int lq = (lane & 7) ^ swizzle(lr);
    const uint32_t vw[2] = {(uint32_t)(lr * a.hidden + lq * 16), (uint32_t)(lr * a.hidden + (lq ^ 4) * 16)};
    auto load_w = [&](int b) {
        const int bc = b < nb ? b : nb - 1;
        char* stage = smem + (b & (kStages - 1)) * kStage;
#pragma unroll
        for (int u = 0; u < kLoads; ++u)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void_t*)(stage + (wave * kLoads + u) * 1024), 16, vw[u & 1],
                                                     (uint32_t)(u * 8 * a.hidden + bc * kQBlock), 0, 0);
    };
    const int64_t i0 = tn * kTileRows + wn * 64;
    const uint8_t* rows = t.rows + (i0 / 16) * nb * 2048 + lane * 16;
    const float* sat = t.scale_t + i0 + c;
    // a wave's rows of W share a scale block; where they lie past the vocabulary they are
    // zero, and the tile's first block stands in
    const int64_t vw0 = v0 + wv * 16 * VI;
    const float* sw = a.w_scale + (vw0 < a.vocab ? vw0 : v0) / kQBlock * nb;
    struct Step {
        Frag f[4];
        float s[4], s0;
    };
    auto load_rows = [&](int b, Step& n) {
        const int bc = b < nb ? b : nb - 1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint8_t* p = rows + ((int64_t)j * nb + bc) * 2048;
            n.f[j].lo = *reinterpret_cast<const u32x4*>(p);
            n.f[j].hi = *reinterpret_cast<const u32x4*>(p + 1024);
            n.s[j] = sat[(int64_t)bc * t.n_pad + 16 * j];
        }
        n.s0 = sw[bc];
    };
    floatx4 acc[VI][4];
#pragma unroll
    for (int i = 0; i < VI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    // One step: the W fragment of group i + 1 is read, and group i - 1's sums
    // are scaled and added, between the matrix instructions of group i.
    auto step = [&](int b, Step& cur, Step& nxt) {
        load_rows(b + 1, nxt);
        load_w(b + 3);
        __builtin_amdgcn_sched_barrier(0);
        const char* stage = smem + (b & (kStages - 1)) * kStage + wv * 16 * VI * 128;
        auto w_frag = [&](int i) {
            const int r = 16 * i + c;
            Frag f;
            f.lo = *reinterpret_cast<const u32x4*>(stage + r * 128 + ((g ^ swizzle(r)) << 4));
            f.hi = *reinterpret_cast<const u32x4*>(stage + r * 128 + (((4 + g) ^ swizzle(r)) << 4));
            return f;
        };
        float s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = cur.s[j] * cur.s0;
        floatx4 z[2][4];
        auto add = [&](int i, int j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(z[i & 1][j][e], s[j], acc[i][j][e]);
        };
        Frag fw = w_frag(0);
        if constexpr (EXACT) {
            const Wide wx[4] = {Wide(cur.f[0]), Wide(cur.f[1]), Wide(cur.f[2]), Wide(cur.f[3])};
#pragma unroll
            for (int i = 0; i < VI; ++i) {
                const Wide ww(fw);
                if (i + 1 < VI) fw = w_frag(i + 1);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (q == 0) z[i & 1][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
                        z[i & 1][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ww.p[q], wx[j].p[q], z[i & 1][j], 0, 0, 0);
                    }
                    if (i > 0) add(i - 1, q);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        } else {
            const i32x8 wx[4] = {cur.f[0].all(), cur.f[1].all(), cur.f[2].all(), cur.f[3].all()};
#pragma unroll
            for (int i = 0; i < VI; ++i) {
                const i32x8 ww = fw.all();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    z[i & 1][j] = block_sum(ww, wx[j]);
                    if (j == 0 && i + 1 < VI) fw = w_frag(i + 1);
                    if (i > 0) add(i - 1, j);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) add(VI - 1, j);
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    Step s0, s1;
    load_w(0);
    load_w(1);
    load_rows(0, s0);
    load_w(2);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    int b = 0;
    for (; b + 1 < nb; b += 2) {
        step(b, s0, s1);
        step(b + 1, s1, s0);
    }
    if (b < nb) step(b, s0, s1);
    // every LDS-direct load (the clamped ones past the last step included) lands before the end
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    // four consecutive logits of a row per lane: one store where rows keep that aligned
    const bool whole = (a.ld & 3) == 0;
#pragma unroll
    for (int i = 0; i < VI; ++i) {
        const int64_t v = v0 + wv * 16 * VI + 16 * i + 4 * g;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t row = i0 + 16 * j + c;
            if (row >= a.n) continue;
            const int64_t at = row * a.ld + v;
            if (whole && v + 4 <= a.vocab) {
                if (EXACT)
                    *reinterpret_cast<floatx4*>(reinterpret_cast<float*>(a.out) + at) = acc[i][j];
                else
                    *reinterpret_cast<uint2*>(reinterpret_cast<bf16_bits*>(a.out) + at) =
                        make_uint2(pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3]));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (v + e < a.vocab) {
                        if (EXACT)
                            reinterpret_cast<float*>(a.out)[at + e] = acc[i][j][e];
                        else
                            reinterpret_cast<__bf16*>(a.out)[at + e] = (__bf16)acc[i][j][e];
                    }
            }
        }
    }
}

}  // namespace

size_t logits_workspace(int64_t n, int hidden) {
    if (n <= kStreamRows) return 256;
    const int64_t n_pad = round_up(n, kTileRows);
    return (size_t)(n_pad * hidden + round_up(4 * n_pad * (hidden / kQBlock), 256));
}

void launch_logits(const LogitsArgs& a, void* workspace, hipStream_t s) {
    if (a.n <= 16) return stream<2, 1>(a, s);
    if (a.n <= 32) return stream<4, 2>(a, s);
    if (a.n <= 64) return stream<4, 4>(a, s);
    if (a.n <= kStreamRows) return stream<2, 8>(a, s);
    TileArgs t;
    t.p = a;
    t.n_pad = round_up(a.n, kTileRows);
    uint8_t* rows = (uint8_t*)workspace;
    float* scale_t = (float*)(rows + t.n_pad * a.hidden);
    t.rows = rows;
    t.scale_t = scale_t;
    pack_rows_kernel<<<grid_1d(t.n_pad * a.hidden / 16, 256, 8192), 256, 0, s>>>(a.a, a.a_scale, a.n, t.n_pad, a.hidden,
                                                                                rows, scale_t);
    t.tiles_n = t.n_pad / kTileRows;
    if (a.out_f32) {
        t.tiles_v = cdiv(a.vocab, 128);
        logits_tile_kernel<true, 4><<<(unsigned)(t.tiles_n * t.tiles_v), kTileThreads, 0, s>>>(t);
    } else {
        t.tiles_v = cdiv(a.vocab, 256);
        logits_tile_kernel<false, 8><<<(unsigned)(t.tiles_n * t.tiles_v), kTileThreads, 0, s>>>(t);
    }
}

}  // namespace lmhead
