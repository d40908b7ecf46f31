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
// vocabulary row and pass). Every wave takes a share of the vocabulary with an
// LDS ring of its own and no barrier. More rows: the matrix instructions
// decide, on 256-row tiles (or the same stream over sets of 64 rows where the
// tiles would be few).
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
    __device__ __forceinline__ void set(const Frag& f) {
#pragma unroll
        for (int s = 0; s < 4; ++s) p[s] = f.part(s);
    }
};

__device__ __forceinline__ floatx4 block_sum(const i32x8& a, const i32x8& b) {
    const floatx4 z = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, z, 0, 0, 0, 0, 0, 0);
}

// ------------------------------------------------------------- few rows

constexpr int kStreamRows = 64;

// Four consecutive logits of a row per lane, `count` of them (<= 0: none)
// inside the vocabulary: one store where the pitch and the buffer keep them aligned.
__device__ __forceinline__ void store4(const LogitsArgs& a, int64_t row, int64_t v, int count, const floatx4& x) {
    if (row >= a.n || count <= 0) return;
    const int64_t at = row * a.ld + v;
    if (count >= 4 && a.quads) {
        if (a.out_f32)
            *reinterpret_cast<floatx4*>(reinterpret_cast<float*>(a.out) + at) = x;
        else
            *reinterpret_cast<uint2*>(reinterpret_cast<bf16_bits*>(a.out) + at) =
                make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < count) {
            if (a.out_f32)
                reinterpret_cast<float*>(a.out)[at + e] = x[e];
            else
                reinterpret_cast<__bf16*>(a.out)[at + e] = (__bf16)x[e];
        }
}

// The rows packed: 16-row x 128-column blocks of 2 KB in fragment order (the
// lanes' low 16 bytes, then their high ones), block (i / 16, b) at ((i / 16) nb
// + b) * 2 KB, rows up to n_pad zero; and the scales transposed, [nb][n_pad],
// row 64 t + 16 j + c at 64 t + 4 c + j when n_pad is a multiple of 64 (a
// lane's four rows side by side), else in order.
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
        const int64_t b = q / n_pad, at = q - b * n_pad;
        const int64_t row = n_pad % 64 == 0 ? at / 64 * 64 + (at & 3) * 16 + (at >> 2 & 15) : at;
        scale_t[q] = row < n ? a_scale[row * nb + b] : 0.0f;
    }
}

// Every wave takes its share of the vocabulary's 16-row groups, kStreamWaves of
// them over the whole chip at once (eight per compute unit, all resident), VT
// groups at a time over all columns and all (NT * 16) input rows: the shares
// differ by one group at most, there is no last round that leaves units idle,
// nothing to join, and the waves of a unit read the same rows' fragments at
// about the same time. A wave's part of W goes through two steps of LDS of its
// own: LDS-direct loads of whole 128-byte lines (a fragment loaded straight
// from row-major W takes 16 bytes of 16 lines per 16 lanes), 16-byte chunk q of
// row r at q ^ ((r >> 1) & 7) for conflict-free fragment reads. Only the wave's
// own counters order it: no barrier. The input rows' fragments come from
// the packed copy (PACKED), or from the rows themselves while they are at
// most 16.
constexpr int kStreamWaves = 2048;   // 256 compute units x 8
constexpr int kStreamGroup = 8;      // waves per workgroup

template <int VT, int NT, bool PACKED>
__global__ __launch_bounds__(64 * kStreamGroup) void logits_stream_kernel(LogitsArgs a, const uint8_t* packed,
                                                                         const float* scale_t, int n_pad, int waves) {
    constexpr int kStage = 16 * VT * 128;
    __shared__ __attribute__((aligned(16))) char smem[kStreamGroup * 2 * kStage];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int nb = a.hidden / kQBlock;
    // Step k of a workgroup is column block (k + rot) mod nb. All waves read
    // 128 bytes of many rows at a time; were they all at the same columns, the
    // addresses would agree in their low bits and meet in a few memory
    // channels (one row: 127 us so, 107 us rotated).
    const int rot = (int)blockIdx.x % nb;
    auto block_of = [&](int k) { return k + rot < nb ? k + rot : k + rot - nb; };
    const int64_t groups = (a.vocab + 15) / 16;
    const int id = (int)blockIdx.x * kStreamGroup + wave;
    const int64_t first = groups * id / waves, last = groups * (id + 1) / waves;
    const int set = blockIdx.y;   // of 64 rows
    char* const ring = smem + wave * 2 * kStage;
    // load u: rows 8 u .. + 8 in lane order; row r + 8 has swizzle(r) ^ 4
    const int lr = lane >> 3, lq = (lane & 7) ^ swizzle(lr);
    const uint32_t vw[2] = {(uint32_t)(lr * a.hidden + lq * 16), (uint32_t)(lr * a.hidden + (lq ^ 4) * 16)};
    const uint8_t* x[NT];
    const float* sa[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        if (PACKED) {
            x[j] = packed + (int64_t)(4 * set + j) * nb * 2048 + lane * 16;
            sa[j] = scale_t + 64 * set + (n_pad % 64 == 0 ? 4 * c + j : 16 * j + c);
        } else {
            const int64_t r = 16 * j + c < a.n ? 16 * j + c : a.n - 1;
            x[j] = a.a + r * a.hidden + 16 * g;
            sa[j] = a.a_scale + r * nb;
        }
    }
    for (int64_t g0 = first; g0 < last; g0 += VT) {
        const int64_t v0 = 16 * g0;
        const int64_t left = (last * 16 < a.vocab ? last * 16 : a.vocab) - v0;
        const int vrows = left < 16 * VT ? (int)left : 16 * VT;
        // rows past the wave's share read as zero (buffer range)
        auto load_w = [&](int i, int b) {   // group i of step b; past the last step an empty range: nothing is read
            const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
                (void*)(a.w + v0 * a.hidden), 0, b < nb ? vrows * a.hidden : 0, 0x00020000);
            char* stage = ring + (b & 1) * kStage;
#pragma unroll
            for (int u = 2 * i; u < 2 * i + 2; ++u)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void_t*)(stage + u * 1024), 16, vw[u & 1],
                                                         (uint32_t)(u * 8 * a.hidden + block_of(b) * kQBlock), 0, 0);
        };
        // a group of 16 rows lies in one scale block; a group past the share has rows of zeros
        const float* sw[VT];
#pragma unroll
        for (int i = 0; i < VT; ++i) sw[i] = a.w_scale + (16 * i < vrows ? v0 + 16 * i : v0) / kQBlock * nb;
        Frag fx[NT];
        float sx[NT], sv[VT];
        auto load_x = [&](int k) {
            const int b = block_of(k);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint8_t* p = x[j] + (int64_t)b * (PACKED ? 2048 : kQBlock);
                fx[j].lo = *reinterpret_cast<const u32x4*>(p);
                fx[j].hi = *reinterpret_cast<const u32x4*>(p + (PACKED ? 1024 : 64));
                sx[j] = sa[j][PACKED ? b * n_pad : b];
            }
#pragma unroll
            for (int i = 0; i < VT; ++i) sv[i] = sw[i][b];
        };
        floatx4 acc[VT][NT];
#pragma unroll
        for (int i = 0; i < VT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < VT; ++i) load_w(i, 0);
        load_x(0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < VT; ++i) load_w(i, 1);
        for (int b = 0; b < nb; ++b) {
            // all but the next step's W, issued last, has landed
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * VT) : "memory");
            __builtin_amdgcn_sched_barrier(0);
            Wide wx[NT];
            float s[NT], t[VT];
#pragma unroll
            for (int j = 0; j < NT; ++j) wx[j].set(fx[j]), s[j] = sx[j];
#pragma unroll
            for (int i = 0; i < VT; ++i) t[i] = sv[i];
            __builtin_amdgcn_sched_barrier(0);
            load_x(b + 1 < nb ? b + 1 : b);
            __builtin_amdgcn_sched_barrier(0);
            const char* stage = ring + (b & 1) * kStage;
#pragma unroll
            for (int i = 0; i < VT; ++i) {
                const int r = 16 * i + c;
                Frag f;
                f.lo = *reinterpret_cast<const u32x4*>(stage + r * 128 + ((g ^ swizzle(r)) << 4));
                f.hi = *reinterpret_cast<const u32x4*>(stage + r * 128 + (((4 + g) ^ swizzle(r)) << 4));
                // the fragment is in registers: its slot takes the step after next
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                load_w(i, b + 2);
                __builtin_amdgcn_sched_barrier(0);
                Wide ww;
                ww.set(f);
                floatx4 z[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) z[j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        z[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ww.p[q], wx[j].p[q], z[j], 0, 0, 0);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const float m = s[j] * t[i];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(z[j][e], m, acc[i][j][e]);
                }
            }
        }
        // the empty loads too have landed before the slots are used again
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
        for (int i = 0; i < VT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                store4(a, 64 * set + 16 * j + c, v0 + 16 * i + 4 * g, 16 * i + 4 * g < vrows ? vrows - 16 * i - 4 * g : 0, acc[i][j]);
    }
}

// Waves for each of the sets of 64 rows: an equal part of the chip's, whole workgroups.
int64_t stream_waves(int64_t sets) {
    const int64_t w = kStreamWaves / sets / kStreamGroup * kStreamGroup;
    return w > kStreamGroup ? w : kStreamGroup;
}

template <int VT, int NT, bool PACKED>
void stream(const LogitsArgs& a, const uint8_t* packed, const float* scale_t, int64_t n_pad, int sets, hipStream_t s) {
    const int waves = (int)stream_waves(sets);
    logits_stream_kernel<VT, NT, PACKED>
        <<<dim3(waves / kStreamGroup, sets), 64 * kStreamGroup, 0, s>>>(a, packed, scale_t, (int)n_pad, waves);
}

// Groups of 16 rows at a time: the wave's whole share where it is at most five
// (more would not fit the LDS or the registers), else a divisor-like part of it.
template <int NT, bool PACKED>
void stream_by_share(const LogitsArgs& a, const uint8_t* packed, const float* scale_t, int64_t n_pad, int sets,
                     hipStream_t s) {
    const int64_t share = cdiv(cdiv(a.vocab, 16), stream_waves(sets));
    const int64_t vt = cdiv(share, cdiv(share, 5));
    if (vt <= 1) return stream<1, NT, PACKED>(a, packed, scale_t, n_pad, sets, s);
    if (vt == 2) return stream<2, NT, PACKED>(a, packed, scale_t, n_pad, sets, s);
    if (vt == 3) return stream<3, NT, PACKED>(a, packed, scale_t, n_pad, sets, s);
    if (vt == 4) return stream<4, NT, PACKED>(a, packed, scale_t, n_pad, sets, s);
    return stream<5, NT, PACKED>(a, packed, scale_t, n_pad, sets, s);
}

// ------------------------------------------------------------- many rows

constexpr int kTileThreads = 512;    // eight waves: VW along the vocabulary, 8 / VW along the rows
constexpr int kStages = 4;

struct TileArgs {
    LogitsArgs p;
    const uint8_t* rows;    // packed (pack_rows_kernel)
    const float* scale_t;
    int64_t n_pad, tiles_n, tiles_v;
};

// One workgroup: 64 * 8 / VW input rows x 16 VI VW vocabulary rows; a wave has
// 64 x 16 VI of them.
// W goes through LDS: one 128-column step of the tile is rows of 128 bytes,
// 16-byte chunk q of row r at q ^ ((r >> 1) & 7) (conflict-free fragment
// reads), written by LDS-direct buffer loads, four steps in a ring. The rows'
// fragments come straight from the packed copy into registers, a step ahead.
// In a step a wave issues the next step's row fragments and scales first and
// then the W loads of step b + 3: waiting for the former at the next step's start leaves
// only the latter in flight, so W of step b + 1 has landed for every wave that
// has begun step b, and one barrier per step is enough.
template <bool EXACT, int VI, int VW, bool LINES>
__global__ __launch_bounds__(kTileThreads, 1) void logits_tile_kernel(TileArgs t) {
    static_assert(VI == 8 || VI == 4, "a step's loads are spread over eight (half) groups");
    constexpr int kV = 16 * VI * VW, kRows = 64 * (8 / VW), kStage = kV * 128, kLoads = kStage / (kTileThreads * 16);
    constexpr int kOut = 8 * 64 * 16 * VI * (EXACT ? 4 : 2);   // the results on their way out
    __shared__ __attribute__((aligned(16))) char smem[kStages * kStage > kOut ? kStages * kStage : kOut];
    const LogitsArgs& a = t.p;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wv = wave % VW, wn = wave / VW;
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
    // step k is column block (k + rot) mod nb, an eighth of the way on from one eighth of
    // the vocabulary to the next: the XCDs are at different ones (map_tile), so fewer waves
    // meet at the same columns of memory (256 rows: 233 us without, 215 us with), and every
    // row of the batch sums a logit in the same order
    const int rot = (int)(tv * 8 / t.tiles_v) * nb / 8;
    auto block_of = [&](int k) {
        const int kc = (k < nb ? k : nb - 1) + rot;
        return kc < nb ? kc : kc - nb;
    };
    auto load_w = [&](int b, int half) {
        const int bc = block_of(b);
        char* stage = smem + (b & (kStages - 1)) * kStage;
#pragma unroll
        for (int u = half * (kLoads / 2); u < (half + 1) * (kLoads / 2); ++u)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void_t*)(stage + (wave * kLoads + u) * 1024), 16, vw[u & 1],
                                                     (uint32_t)(u * 8 * a.hidden + bc * kQBlock), 0, 0);
    };
    const int64_t i0 = tn * kRows + wn * 64;
    const uint8_t* rows = t.rows + (i0 / 16) * nb * 2048 + lane * 16;
    const float* sat = t.scale_t + i0 + 4 * c;
    // a wave's rows of W share a scale block; where they lie past the vocabulary they are
    // zero, and the tile's first block stands in
    const int64_t vw0 = v0 + wv * 16 * VI;
    const float* sw = a.w_scale + (vw0 < a.vocab ? vw0 : v0) / kQBlock * nb;
    struct Step {
        Frag f[4];
        floatx4 s;
        float s0;
    };
    auto load_row = [&](int b, Step& n, int j) {
        const uint8_t* p = rows + ((int64_t)j * nb + block_of(b)) * 2048;
        n.f[j].lo = *reinterpret_cast<const u32x4*>(p);
        n.f[j].hi = *reinterpret_cast<const u32x4*>(p + 1024);
    };
    auto load_scales = [&](int b, Step& n) {
        const int bc = block_of(b);
        n.s = *reinterpret_cast<const floatx4*>(sat + (int64_t)bc * t.n_pad);
        n.s0 = sw[bc];
    };
    floatx4 acc[VI][4];
#pragma unroll
    for (int i = 0; i < VI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    // One step: the W fragment of group i + 1 is read, and group i - 1's sums
    // are scaled and added, between the matrix instructions of group i. The
    // step's loads are spread over its groups too, the row fragments in the
    // first half, the scales, then W: issued together at the start they filled
    // the load queue and every wave stood before its first matrix instruction.
    auto step = [&](int b, Step& cur, Step& nxt) {
        auto issue = [&](int i) {   // after group i of 8 (VI = 8) or half group of 4
            if (i < 4) load_row(b + 1, nxt, i);
            if (i == 4) load_scales(b + 1, nxt);
            if (i == 5) load_w(b + 3, 0);
            if (i == 6) load_w(b + 3, 1);
        };
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
        __builtin_amdgcn_sched_barrier(0);
        floatx4 z[2][4];
        auto add = [&](int i, int j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(z[i & 1][j][e], s[j], acc[i][j][e]);
        };
        Frag fw = w_frag(0);
        if constexpr (EXACT) {
            Wide wx[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) wx[j].set(cur.f[j]);
#pragma unroll
            for (int i = 0; i < VI; ++i) {
                Wide ww;
                ww.set(fw);
                if (i + 1 < VI) fw = w_frag(i + 1);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (q == 0) z[i & 1][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
                        z[i & 1][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ww.p[q], wx[j].p[q], z[i & 1][j], 0, 0, 0);
                    }
                    if (i > 0) add(i - 1, q);
                    if (q & 1) issue(2 * i + (q >> 1));
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
                    if (VI == 8 && j == 2) issue(i);
                    if (VI == 4 && (j & 1)) issue(2 * i + (j >> 1));
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
#pragma unroll
    for (int k = 0; k < 2; ++k) load_w(k, 0), load_w(k, 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) load_row(0, s0, j);
    load_scales(0, s0);
    __builtin_amdgcn_sched_barrier(0);
    load_w(2, 0), load_w(2, 1);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    int b = 0;
    for (; b + 1 < nb; b += 2) {
        step(b, s0, s1);
        step(b + 1, s1, s0);
    }
    if (b < nb) step(b, s0, s1);
    // every LDS-direct load (the clamped ones past the last step included) has landed
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    // Through LDS, a part of it per wave: rows of 16 VI logits, 16-byte piece q
    // of row r at q ^ (r mod pieces), then whole rows of 128 or 256 bytes to
    // memory, past the L2 that W and the rows live in. Stored from the
    // fragments, a row's 32 bytes at a time, the results took 165 of 1262 us
    // (2048 rows, bf16); this way 1178 us in all, 1165 us with the
    // non-temporal hint (256 rows: 202, 187, 177 us).
    __syncthreads();
    constexpr int kSize = EXACT ? 4 : 2, kPitch = 16 * VI * kSize, kPieces = kPitch / 16;
    char* const part = smem + wave * 64 * kPitch;
    auto place = [&](int r, int at) { return part + r * kPitch + (((at >> 4) ^ (r & (kPieces - 1))) << 4) + (at & 15); };
#pragma unroll
    for (int i = 0; i < VI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            char* p = place(16 * j + c, (16 * i + 4 * g) * kSize);
            if (EXACT)
                *reinterpret_cast<floatx4*>(p) = acc[i][j];
            else
                *reinterpret_cast<uint2*>(p) =
                    make_uint2(pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3]));
        }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    // the tile's place made again: kept through the loop it cost registers that the loop needs
    int bid = blockIdx.x;
    asm volatile("" : "+s"(bid));
    map_tile(bid, t.tiles_n, t.tiles_v, tn, tv);
    const int64_t i1 = tn * kRows + wn * 64, v1 = tv * kV + wv * 16 * VI;
    const int left = a.vocab - v1 < 16 * VI ? (int)(a.vocab - v1) : 16 * VI;   // logits of a row inside the vocabulary
    char* const out = reinterpret_cast<char*>(a.out) + (i1 * a.ld + v1) * kSize;
    const int rows_left = a.n - i1 < 64 ? (int)(a.n - i1) : 64;
    if constexpr (LINES) {
        const int q = lane % kPieces, e0 = q * (16 / kSize);
#pragma unroll 4
        for (int r = lane / kPieces; r < rows_left; r += 64 / kPieces) {
            const u32x4 x = *reinterpret_cast<const u32x4*>(place(r, 16 * q));
            char* to = out + r * a.ld * kSize + 16 * q;
            if (e0 + 16 / kSize <= left) {
                __builtin_nontemporal_store(x, reinterpret_cast<u32x4*>(to));
            } else {
                for (int e = 0; e < 16 / kSize && e0 + e < left; ++e) {
                    if (EXACT)
                        reinterpret_cast<uint32_t*>(to)[e] = x[e];
                    else
                        reinterpret_cast<uint16_t*>(to)[e] = (uint16_t)(x[e >> 1] >> (16 * (e & 1)));
                }
            }
        }
        return;
    }
    // Rows that start at any element: four bytes a lane, bf16 pairs from the
    // row's first aligned one on (151,935 columns, 2048 rows: 1260 us; element by
    // element 1426 us).
    constexpr int kLanes = EXACT ? 16 * VI : 8 * VI;
    const int l = lane % kLanes;
#pragma unroll 4
    for (int r = lane / kLanes; r < rows_left; r += 64 / kLanes) {
        char* to = out + r * a.ld * kSize;
        if (EXACT) {
            if (l < left) reinterpret_cast<uint32_t*>(to)[l] = *reinterpret_cast<const uint32_t*>(place(r, 4 * l));
        } else {
            const int odd = (int)(reinterpret_cast<uintptr_t>(to) >> 1) & 1, e = 2 * l + odd;
            const uint32_t lo = *reinterpret_cast<const uint16_t*>(place(r, 2 * e));
            const uint32_t hi = *reinterpret_cast<const uint16_t*>(place(r, 2 * (e + 1 < 16 * VI ? e + 1 : e)));
            if (e + 1 < left)
                *reinterpret_cast<uint32_t*>(to + 2 * e) = lo | hi << 16;
            else if (e < left)
                reinterpret_cast<uint16_t*>(to)[e] = (uint16_t)lo;
            if (odd && l == 0 && left > 0)
                reinterpret_cast<uint16_t*>(to)[0] = *reinterpret_cast<const uint16_t*>(place(r, 0));
        }
    }
}

}  // namespace

// Rows of a matrix tile. With an fp32 output, tiles of 128 rows x 256 columns and
// of 256 x 128 take the same time per row, so 128 wherever 256 would leave the
// last half tile empty. A bf16 output's larger 256 x 256 tile reads less per
// product and loses to 128 only when one tile holds all rows. us at 151,936 x
// 4096, 128 and 256 rows a tile:
//   rows    70        128       200       256       300       400       512       1024        1100        2048
//   fp32    185, 289  203, 291  326, 326  343, 340  459, 579  616, 601  657, 637  1251, 1219  1407, 1467  2422, 2423
//   bf16    160, 193  170, 197  245, 198  242, 198  318, 296  429, 305  432, 317   808, 602    927, 700   1548, 1138
int64_t tile_rows(int64_t n, int out_f32) {
    if (out_f32) return cdiv(n, 128) % 2 ? 128 : 256;
    return n <= 128 ? 128 : 256;
}

// rows padded for the packed copy: none up to 16
int64_t packed_rows(int64_t n, int out_f32) {
    return n <= 16 ? 0 : round_up(n, n <= kStreamRows ? 16 : tile_rows(n, out_f32));
}

size_t logits_workspace(int64_t n, int hidden, int out_f32) {
    const int64_t n_pad = packed_rows(n, out_f32);
    return (size_t)(n_pad * hidden + round_up(4 * n_pad * (hidden / kQBlock) + 1, 256));
}

// More rows than kStreamRows against so few columns that tiles leave most of the
// chip idle: the stream kernel over sets of 64 rows, while a wave has one group
// of 16 columns (two for an fp32 output, whose tile takes longer; half the waves
// at most one where a bf16 tile of 128 rows, the quickest, is the other way).
// us at hidden 5120, stream and tiles:
//                        70 rows   130 rows   300 rows   700 rows   2048 rows
//   1000 columns, fp32    26, 67     26, 66     29, 69     34, 70      55, 74
//   1000, bf16            26, 41     26, 53     29, 55     34, 57      54, 61
//   4000, fp32            34, 68     31, 67     39, 70     63, 71
//   4000, bf16            33, 41     31, 54     38, 56     60, 57 (two groups)
//   16000, fp32           50, 69     60, 69     86, 75 (three groups)
//   16000, bf16           48, 42     58, 54     84, 55 (three)
bool few_groups(int64_t n, int64_t vocab, int out_f32) {
    const int64_t sets = cdiv(n, kStreamRows), groups = cdiv(vocab, 16);
    if (sets > kStreamWaves / kStreamGroup) return false;
    if (!out_f32 && n <= 128 && sets * groups > kStreamWaves / 2) return false;
    return cdiv(groups, stream_waves(sets)) <= (out_f32 ? 2 : 1);
}

template <bool EXACT, int VI, int VW>
void tiles(TileArgs t, hipStream_t s) {
    t.tiles_n = t.n_pad / (64 * (8 / VW));
    t.tiles_v = cdiv(t.p.vocab, 16 * VI * VW);
    const unsigned grid = (unsigned)(t.tiles_n * t.tiles_v);
    if (t.p.lines)
        logits_tile_kernel<EXACT, VI, VW, true><<<grid, kTileThreads, 0, s>>>(t);
    else
        logits_tile_kernel<EXACT, VI, VW, false><<<grid, kTileThreads, 0, s>>>(t);
}

void launch_logits(const LogitsArgs& a, void* workspace, hipStream_t s) {
    if (a.n <= 16) return stream_by_share<1, false>(a, nullptr, nullptr, 0, 1, s);
    TileArgs t;
    t.p = a;
    t.n_pad = packed_rows(a.n, a.out_f32);
    uint8_t* rows = (uint8_t*)workspace;
    float* scale_t = (float*)(rows + t.n_pad * a.hidden);
    t.rows = rows;
    t.scale_t = scale_t;
    pack_rows_kernel<<<grid_1d(t.n_pad * a.hidden / 16, 256, 8192), 256, 0, s>>>(a.a, a.a_scale, a.n, t.n_pad, a.hidden,
                                                                                rows, scale_t);
    if (a.n <= 32) return stream_by_share<2, true>(a, rows, scale_t, t.n_pad, 1, s);
    if (a.n <= 48) return stream_by_share<3, true>(a, rows, scale_t, t.n_pad, 1, s);
    if (a.n <= kStreamRows) return stream_by_share<4, true>(a, rows, scale_t, t.n_pad, 1, s);
    if (few_groups(a.n, a.vocab, a.out_f32))
        return stream_by_share<4, true>(a, rows, scale_t, t.n_pad, (int)cdiv(a.n, kStreamRows), s);
    const bool narrow = tile_rows(a.n, a.out_f32) == 128;
    if (a.out_f32) return narrow ? tiles<true, 4, 4>(t, s) : tiles<true, 4, 2>(t, s);
    return narrow ? tiles<false, 4, 4>(t, s) : tiles<false, 8, 2>(t, s);
}

}  // namespace lmhead
