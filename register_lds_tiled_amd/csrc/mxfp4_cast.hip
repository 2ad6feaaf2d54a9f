// mxfp4_cast.hip -- quantising a matrix to MXFP4 along its rows, its columns
// or both, and reading MXFP4 back.
//
// For a block x_0 .. x_31 with largest magnitude t:
//     s = max(floor(log2 t) - 2, -127),  q_i = E2M1(x_i 2^-s)
// to nearest, ties to even, saturating at 6 (the specification's rule: 2 is
// the exponent of E2M1's largest value).  The magnitudes' bit patterns order
// as the magnitudes do, NaN and infinities above all others, so t is an
// integer maximum; as a float's bits, t's exponent field less 2 is the scale
// byte, and a field of 255 (NaN or infinity in the block) is itself the byte
// of a NaN block.  v_cvt_scalef32_pk_fp4_* then divides by 2^s, rounds and
// saturates exactly so.
//
// Everything here is bound by memory: two or four bytes read and about half a
// byte written per element and direction.  At 8192 x 8192 bf16: along rows 31 us
// (5.4 TB/s of what it reads and writes), both ways 55 (3.7), reading back 21.5
// (7.9: the codes come from the last-level cache); 16384 x 8192 f32 114 and 98
// (5.4 and 6.2).  A copy of 2 GB reaches 4.9.
#include "mxfp4.h"

namespace sgemm {
namespace {

typedef unsigned short mx_us2 __attribute__((ext_vector_type(2)));

// f(v, the value of lane ^ MASK) for every lane, f symmetric: by the data
// paths between lanes of a quad and of a row of 16, and by exchanging rows.
template <int MASK, class F>
__device__ __forceinline__ unsigned with_lane_xor(unsigned v, F&& f) {
    if constexpr (MASK == 1 || MASK == 2) {
        constexpr int quad = MASK == 1 ? 0xB1 : 0x4E;   // quad_perm [1,0,3,2] / [2,3,0,1]
        return f(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, quad, 0xF, 0xF, true));
    } else if constexpr (MASK == 8) {
        return f(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, true));   // row_ror:8
    } else if constexpr (MASK == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return f(r[0], r[1]);
    } else {
        static_assert(MASK == 32, "lane exchanges that are used");
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return f(r[0], r[1]);
    }
}
__device__ __forceinline__ unsigned max_of(unsigned a, unsigned b) { return max(a, b); }
// The largest over a quad of lanes.
__device__ __forceinline__ unsigned quad_max(unsigned v) {
    return with_lane_xor<2>(with_lane_xor<1>(v, max_of), max_of);
}

// N bytes from an address of any alignment: the memory unit takes wide accesses
// at every byte address.
template <int N>
__device__ __forceinline__ void unaligned_copy(void* to, const void* from) {
    __builtin_memcpy(reinterpret_cast<unsigned char*>(to), reinterpret_cast<const unsigned char*>(from), N);
}

// Eight consecutive elements in a lane's registers, by type: loads (guarded:
// the first n elements exist, the others are 0), the magnitudes' maximum as
// float bits, and conversion of pairs.
template <MxType T>
struct Eight;

template <>
struct Eight<MxType::f32> {
    static constexpr int SIZE = 4;
    unsigned w[8];
    __device__ __forceinline__ void load(const void* base, long long at, int n) {
        const unsigned* p = static_cast<const unsigned*>(base) + at;
        if (n >= 8) {
            unaligned_copy<32>(w, p);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = i < n ? p[i] : 0u;
        }
    }
    // Running maxima of magnitudes, one per column (COLS) or over all eight.
    struct Max {
        unsigned m[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
        __device__ __forceinline__ void take(const Eight& x) {
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] = max(m[i], x.w[i] & 0x7FFFFFFFu);
        }
        template <int MASK>
        __device__ __forceinline__ void across() {
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] = with_lane_xor<MASK>(m[i], max_of);
        }
        __device__ __forceinline__ unsigned bits(int i) const { return m[i]; }
    };
    // The largest magnitude of the eight, in a form that maxima of several
    // lanes are taken in, and that form's float bits.
    __device__ __forceinline__ unsigned top() const {
        unsigned m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
        return m;
    }
    static __device__ __forceinline__ unsigned top_bits(unsigned m) { return m; }
    // Codes of the eight, the first in the lowest four bits.
    __device__ __forceinline__ unsigned codes(float s) const {
        unsigned q = 0u;
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f(0), f(1), s, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f(2), f(3), s, 1);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f(4), f(5), s, 2);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f(6), f(7), s, 3);
    }
    // Codes of element i of four rows, the first row's in the lowest bits.
    static __device__ __forceinline__ unsigned column(const Eight (&x)[4], int i, float s) {
        unsigned q = 0u;
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[0].f(i), x[1].f(i), s, 0);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[2].f(i), x[3].f(i), s, 1);
    }
    __device__ __forceinline__ float f(int i) const { return __uint_as_float(w[i]); }
};

// bf16 and f16: pairs in a register; magnitudes compare as 15-bit integers.
template <MxType T>
struct Eight {
    static constexpr int SIZE = 2;
    unsigned w[4];
    __device__ __forceinline__ void load(const void* base, long long at, int n) {
        const unsigned short* p = static_cast<const unsigned short*>(base) + at;
        if (n >= 8) {
            unaligned_copy<16>(w, p);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = (2 * i < n ? (unsigned)p[2 * i] : 0u) |
                       (2 * i + 1 < n ? (unsigned)p[2 * i + 1] : 0u) << 16;
        }
    }
    static __device__ __forceinline__ unsigned pk_max(unsigned a, unsigned b) {
        return __builtin_bit_cast(unsigned, __builtin_elementwise_max(__builtin_bit_cast(mx_us2, a),
                                                                      __builtin_bit_cast(mx_us2, b)));
    }
    static __device__ __forceinline__ unsigned float_bits(unsigned h) {
        if constexpr (T == MxType::bf16) return h << 16;
        else return __float_as_uint((float)__builtin_bit_cast(mx_h2, h)[0]);
    }
    struct Max {
        unsigned m[4] = {0u, 0u, 0u, 0u};
        __device__ __forceinline__ void take(const Eight& x) {
#pragma unroll
            for (int i = 0; i < 4; ++i) m[i] = pk_max(m[i], x.w[i] & 0x7FFF7FFFu);
        }
        template <int MASK>
        __device__ __forceinline__ void across() {
#pragma unroll
            for (int i = 0; i < 4; ++i) m[i] = with_lane_xor<MASK>(m[i], pk_max);
        }
        __device__ __forceinline__ unsigned bits(int i) const {
            return float_bits(i & 1 ? m[i / 2] >> 16 : m[i / 2] & 0xFFFFu);
        }
    };
    __device__ __forceinline__ unsigned top() const {
        const unsigned m = pk_max(pk_max(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                  pk_max(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
        return max(m & 0xFFFFu, m >> 16);
    }
    static __device__ __forceinline__ unsigned top_bits(unsigned m) { return float_bits(m); }
    template <int SEL>
    static __device__ __forceinline__ unsigned pair(unsigned q, unsigned v, float s) {
        if constexpr (T == MxType::bf16)
            return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(mx_bf2, v), s, SEL);
        else
            return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(mx_h2, v), s, SEL);
    }
    __device__ __forceinline__ unsigned codes(float s) const {
        unsigned q = 0u;
        static_for<4>([&](auto i) { q = pair<i>(q, w[i], s); });
        return q;
    }
    static __device__ __forceinline__ unsigned column(const Eight (&x)[4], int i, float s) {
        const unsigned sel = i & 1 ? 0x07060302u : 0x05040100u;   // high or low halves of two rows
        const unsigned q = pair<0>(0u, __builtin_amdgcn_perm(x[1].w[i / 2], x[0].w[i / 2], sel), s);
        return pair<1>(q, __builtin_amdgcn_perm(x[3].w[i / 2], x[2].w[i / 2], sel), s);
    }
};

// Scale byte from the float bits of a block's largest magnitude.
__device__ __forceinline__ unsigned scale_byte(unsigned bits) {
    const unsigned e = bits >> 23;
    return e == 255u ? 255u : max(e, 2u) - 2u;
}

// Store of the first n (1 .. 4) bytes of q.
__device__ __forceinline__ void store_bytes(unsigned char* p, unsigned q, int n) {
    if (n >= 4) {
        __builtin_memcpy(p, &q, 4);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = (unsigned char)(q >> (8 * i));
    }
}

constexpr int kCastItems = 4;   // items a wave has in flight

// How R rows of C elements, E to a lane and a block's lanes together, are
// divided: log2 of the lanes a row gets, segments of that many lanes in a row,
// items (a segment of one row group) and workgroups of four waves that take
// `at_a_time` items each.
struct Items {
    int lpr;
    unsigned segs, grid;
    long long items;
};
Items items_of(int R, int C, int E, int at_a_time) {
    const long long units = ((long long)C + 31) / 32 * (32 / E);
    Items it;
    it.lpr = E == 8 ? 2 : 3;
    while (it.lpr < 6 && (1 << it.lpr) < units) ++it.lpr;
    it.segs = (unsigned)((units + (1 << it.lpr) - 1) >> it.lpr);
    it.items = it.segs * (((long long)R + (64 >> it.lpr) - 1) / (64 >> it.lpr));
    const long long want = (it.items + 4 * at_a_time - 1) / (4 * at_a_time);
    it.grid = (unsigned)(want < (1 << 20) ? want : (1 << 20));
    return it;
}

// Quantising along rows.  A lane holds 8 consecutive elements, four lanes a
// block, a wave's lanes one row's segment of 8 << LPR elements or, where rows
// are short, several rows' (lpr: log2 of lanes per row).  Items (segments of
// row groups) are numbered along the rows; a wave takes four neighbours at a
// time and loads them all before it converts the first.
template <MxType T>
__global__ __launch_bounds__(256) void mx_quantize_rows_kernel(MxQuantArgs p, int lpr, unsigned segs,
                                                               long long items) {
    const int lane = threadIdx.x & 63;
    const int rows_per = 64 >> lpr;
    const int sub = lane >> lpr, unit = lane & ((1 << lpr) - 1);
    const long long wave = (long long)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const long long waves = (long long)gridDim.x * 4;
    for (long long first = wave * kCastItems; first < items; first += waves * kCastItems) {
        Eight<T> x[kCastItems];
        long long row[kCastItems];
        int col[kCastItems];
#pragma unroll
        for (int u = 0; u < kCastItems; ++u) {
            const unsigned long long item = first + u;
            const unsigned long long group =
                items <= 0xFFFFFFFFll ? (unsigned)item / segs : item / segs;
            const unsigned seg = (unsigned)(item - group * segs);
            row[u] = (long long)group * rows_per + sub;
            // (a segment's start stays below C, so an int holds it; in the
            // last segment lanes past the row's end could pass 2^31)
            const long long c = ((long long)seg << lpr) * 8 + unit * 8;
            const bool in = first + u < items && row[u] < p.R && c < p.C;
            col[u] = in ? (int)c : -1;
            x[u].load(p.X, in ? row[u] * p.ldx + c : 0, in ? min(p.C - (int)c, 8) : 0);
        }
#pragma unroll
        for (int u = 0; u < kCastItems; ++u) {
            const unsigned m = quad_max(x[u].top());
            const unsigned byte = scale_byte(Eight<T>::top_bits(m));
            const unsigned q = x[u].codes(mx_scale(byte));
            if (col[u] < 0) continue;
            store_bytes(p.Q + row[u] * p.ldq + col[u] / 2, q, (min(p.C - col[u], 8) + 1) / 2);
            if ((lane & 3) == 0) p.S[row[u] * p.lds + col[u] / 32] = (unsigned char)byte;
        }
    }
}

// Quantising along columns, and along rows too where ROWS, in one pass.  A
// workgroup owns a piece of kTileR x 128; each wave takes 32 rows of it (one
// block of every column), 64 columns at a time: lane l holds rows 4 (l / 8) .. + 3,
// columns 8 (l % 8) .. + 7.  A row's blocks are quads of lanes; a column's
// block is the lanes of equal l % 8.  Codes and scales are gathered in LDS and
// leave as whole segments of rows and columns.
constexpr int kTileC = 128;

template <MxType T, bool ROWS, int kTileR>
__global__ __launch_bounds__(2 * kTileR) void mx_quantize_both_kernel(MxQuantArgs p, int tiles_m, int tiles_n) {
    constexpr int kTileWaves = kTileR / 32, NT = 64 * kTileWaves;
    constexpr int kTilePitch = kTileR / 2 + 4;   // LDS bytes of a column's codes: odd in words
    constexpr int kRowPitch = kTileC / 2 + 4;    // of a row's
    __shared__ __attribute__((aligned(16))) unsigned char qt[kTileC * kTilePitch];
    __shared__ __attribute__((aligned(16))) unsigned char st[kTileC * kTileWaves];
    __shared__ __attribute__((aligned(16))) unsigned char qr[ROWS ? kTileR * kRowPitch : 4];
    __shared__ __attribute__((aligned(16))) unsigned char sr[ROWS ? kTileR * (kTileC / 32) : 4];
    int tm, tn;
    tile_coords(blockIdx.x, tiles_m, tiles_n, 8, p.xcds, tm, tn);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int rg = lane >> 3, cg = lane & 7;
    const long long r0 = (long long)tm * kTileR, c0 = (long long)tn * kTileC;
    const long long r = r0 + wave * 32 + rg * 4;
#pragma unroll
    for (int half = 0; half < kTileC / 64; ++half) {
        const long long c = c0 + half * 64 + cg * 8;
        const int n = (int)max(0ll, min((long long)p.C - c, 8ll));
        Eight<T> x[4];
        typename Eight<T>::Max cols;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = r + i < p.R && n > 0;
            x[i].load(p.X, in ? (r + i) * p.ldx + c : 0, in ? n : 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) cols.take(x[i]);
        if constexpr (ROWS) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const unsigned m = quad_max(x[i].top());
                const unsigned byte = scale_byte(Eight<T>::top_bits(m));
                const unsigned q = x[i].codes(mx_scale(byte));
                const int row = wave * 32 + rg * 4 + i;
                *reinterpret_cast<unsigned*>(&qr[row * kRowPitch + half * 32 + cg * 4]) = q;
                if ((lane & 3) == 0) sr[row * (kTileC / 32) + half * 2 + (cg >> 2)] = (unsigned char)byte;
            }
        }
        cols.template across<8>();
        cols.template across<16>();
        cols.template across<32>();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const unsigned byte = scale_byte(cols.bits(i));
            const unsigned q = Eight<T>::column(x, i, mx_scale(byte));
            const int col = half * 64 + cg * 8 + i;
            *reinterpret_cast<unsigned short*>(&qt[col * kTilePitch + wave * 16 + rg * 2]) = (unsigned short)q;
            if (rg == i) st[col * kTileWaves + wave] = (unsigned char)byte;
        }
    }
    __syncthreads();
    // A run of codes (16-byte pieces, PER of them to a line of `pitch` bytes in
    // LDS) or scales (PER bytes a line) of the lines that exist.
    auto store_codes = [&](const unsigned char* from, int pitch, auto PER, int lines, int n, unsigned char* to,
                           long long ld) {
        for (int id = threadIdx.x; id < lines * PER; id += NT) {
            const int line = id / PER, at = id % PER * 16;
            const unsigned* w = reinterpret_cast<const unsigned*>(from + line * pitch + at);
            unsigned char* out = to + line * ld + at;
            if (at + 16 <= n) {
                const uint4 v = make_uint4(w[0], w[1], w[2], w[3]);
                __builtin_memcpy(out, &v, 16);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (at + 4 * j < n) store_bytes(out + 4 * j, w[j], min(n - at - 4 * j, 4));
            }
        }
    };
    auto store_scales = [&](const unsigned char* from, auto PER, int lines, int n, unsigned char* to, long long ld) {
        for (int line = threadIdx.x; line < lines; line += NT) {
            unsigned char* out = to + line * ld;
            const unsigned char* in = from + line * PER;
            if (n == PER) {
                __builtin_memcpy(out, in, PER);      // any alignment
            } else {
                for (int i = 0; i < n; ++i) out[i] = in[i];
            }
        }
    };
    const int rows = (int)min((long long)p.R - r0, (long long)kTileR);
    const int ncols = (int)min((long long)p.C - c0, (long long)kTileC);
    store_codes(qt, kTilePitch, std::integral_constant<int, kTileR / 32>{}, ncols, (rows + 1) / 2,
                p.QT + c0 * p.ldqt + r0 / 2, p.ldqt);
    store_scales(st, std::integral_constant<int, kTileWaves>{}, ncols, (rows + 31) / 32, p.ST + c0 * p.ldst + r0 / 32,
                 p.ldst);
    if constexpr (ROWS) {
        store_codes(qr, kRowPitch, std::integral_constant<int, kTileC / 32>{}, rows, (ncols + 1) / 2,
                    p.Q + r0 * p.ldq + c0 / 2, p.ldq);
        store_scales(sr, std::integral_constant<int, kTileC / 32>{}, rows, (ncols + 31) / 32,
                     p.S + r0 * p.lds + c0 / 32, p.lds);
    }
}

template <MxType T, int ROWS>
hipError_t launch_both(const MxQuantArgs& a, hipStream_t s) {
    const int tm = (int)(((long long)a.R + ROWS - 1) / ROWS), tn = (int)(((long long)a.C + kTileC - 1) / kTileC);
    if (a.Q != nullptr)
        mx_quantize_both_kernel<T, true, ROWS><<<(unsigned)(tm * tn), 2 * ROWS, 0, s>>>(a, tm, tn);
    else
        mx_quantize_both_kernel<T, false, ROWS><<<(unsigned)(tm * tn), 2 * ROWS, 0, s>>>(a, tm, tn);
    return hipGetLastError();
}

template <MxType T>
hipError_t quantize_t(const MxQuantArgs& a, hipStream_t s) {
    if (a.QT != nullptr) {
        // 256 rows at a time where there are more than 128 and that leaves two
        // workgroups to a CU (and the launch holds their 512 threads each): the
        // transposed codes leave in longer runs.  us both ways, 256 and 128 rows
        // at a time, bf16: 8192^2 55.5 57.2, 16384 x 4096 55.1 62.6, 256 x 65536
        // 14.1 14.4, 160 x 262144 36.2 45.5, but 384 x 65536 24.5 22.0; f32:
        // 8192^2 83.6 82.7, 1024 x 32768 39.5 42.0.  Of at most 128 rows half
        // the waves and more would have none: 128 x 65536 10.8 8.5, 1 x 10^6 83
        // 46.  128 rows at a time always fit: the argument checks see to it.
        const long long tall = ((long long)a.R + 255) / 256 * (((long long)a.C + kTileC - 1) / kTileC);
        return a.R > 128 && tall >= 2 * a.cus && tall * 512 <= 0xFFFFFFFFll ? launch_both<T, 256>(a, s)
                                                                            : launch_both<T, 128>(a, s);
    }
    const Items it = items_of(a.R, a.C, 8, kCastItems);
    mx_quantize_rows_kernel<T><<<it.grid, 256, 0, s>>>(a, it.lpr, it.segs, it.items);
    return hipGetLastError();
}

// Reading back: a lane takes 16 bytes of output -- 4 floats or 8 16-bit values
// -- so that a wave's stores are whole kilobytes; lanes and items as in the
// row quantiser.
// VEC: rows of Y start 16-byte aligned.
template <MxType T, bool VEC>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(MxDequantArgs p, int lpr, unsigned segs,
                                                            long long items) {
    constexpr int E = T == MxType::f32 ? 4 : 8, ITEMS = 32 / E;
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
    const int lane = threadIdx.x & 63;
    const int rows_per = 64 >> lpr;
    const int sub = lane >> lpr, unit = lane & ((1 << lpr) - 1);
    const long long wave = (long long)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const long long waves = (long long)gridDim.x * 4;
    for (long long first = wave * ITEMS; first < items; first += waves * ITEMS) {
        unsigned q[ITEMS], byte[ITEMS];
        long long row[ITEMS];
        int col[ITEMS];
#pragma unroll
        for (int u = 0; u < ITEMS; ++u) {
            const unsigned long long item = first + u;
            const unsigned long long group =
                items <= 0xFFFFFFFFll ? (unsigned)item / segs : item / segs;
            const unsigned seg = (unsigned)(item - group * segs);
            row[u] = (long long)group * rows_per + sub;
            const long long c = (((long long)seg << lpr) + unit) * E;
            const bool in = first + u < items && row[u] < p.R && c < p.C;
            col[u] = in ? (int)c : -1;
            q[u] = 0u;
            byte[u] = 0u;
            if (!in) continue;
            const unsigned char* src = p.Q + row[u] * p.ldq + c / 2;
            if (p.C - c >= E) {
                __builtin_memcpy(&q[u], src, E / 2);
            } else {
                const int n = (min(p.C - (int)c, E) + 1) / 2;
#pragma unroll
                for (int i = 0; i < E / 2; ++i)
                    if (i < n) q[u] |= (unsigned)src[i] << (8 * i);
            }
            byte[u] = p.S[row[u] * p.lds + c / 32];
        }
#pragma unroll
        for (int u = 0; u < ITEMS; ++u) {
            if (col[u] < 0) continue;
            const float s = mx_scale(byte[u]);
            const int n = min(p.C - col[u], E);
            unsigned v[E];
            static_for<E / 2>([&](auto i) {
                const mx_f2 t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], s, i);
                v[2 * i] = __float_as_uint(t.x);
                v[2 * i + 1] = __float_as_uint(t.y);
            });
            const long long at = row[u] * p.ldy + col[u];
            if constexpr (T == MxType::f32) {
                unsigned* y = static_cast<unsigned*>(p.Y) + at;
                if (VEC && n == E) {
                    __builtin_nontemporal_store(u32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<u32x4*>(y));
                } else if (n == E) {
                    unaligned_copy<16>(y, v);
                } else {
#pragma unroll
                    for (int i = 0; i < E; ++i)
                        if (i < n) y[i] = v[i];
                }
            } else {
                // bf16: every value is one of bf16's own, its float's upper
                // half (two significant bits; a NaN stays one).  f16: rounded
                // from the exact float.
                unsigned h[E];
#pragma unroll
                for (int i = 0; i < E; ++i)
                    h[i] = T == MxType::bf16 ? v[i] >> 16
                                             : __builtin_bit_cast(unsigned short, (_Float16)__uint_as_float(v[i]));
                unsigned short* y = static_cast<unsigned short*>(p.Y) + at;
                const u32x4 o = {h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
                if (VEC && n == E) {
                    __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(y));
                } else if (n == E) {
                    unaligned_copy<16>(y, &o);
                } else {
#pragma unroll
                    for (int i = 0; i < E; ++i)
                        if (i < n) y[i] = (unsigned short)h[i];
                }
            }
        }
    }
}

template <MxType T>
hipError_t dequantize_v(const MxDequantArgs& a, hipStream_t s) {
    constexpr int E = T == MxType::f32 ? 4 : 8, ITEMS = 32 / E;
    const Items it = items_of(a.R, a.C, E, ITEMS);
    const bool vec = mx_aligned(a.Y, a.ldy * Eight<T>::SIZE, 16);
    if (vec)
        mx_dequantize_kernel<T, true><<<it.grid, 256, 0, s>>>(a, it.lpr, it.segs, it.items);
    else
        mx_dequantize_kernel<T, false><<<it.grid, 256, 0, s>>>(a, it.lpr, it.segs, it.items);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantArgs& a, MxType t, hipStream_t s) {
    switch (t) {
        case MxType::f32: return quantize_t<MxType::f32>(a, s);
        case MxType::bf16: return quantize_t<MxType::bf16>(a, s);
        default: return quantize_t<MxType::f16>(a, s);
    }
}

hipError_t launch_mx_dequantize(const MxDequantArgs& a, MxType t, hipStream_t s) {
    switch (t) {
        case MxType::f32: return dequantize_v<MxType::f32>(a, s);
        case MxType::bf16: return dequantize_v<MxType::bf16>(a, s);
        default: return dequantize_v<MxType::f16>(a, s);
    }
}

}  // namespace sgemm
