// mxfp4_rows.hip -- C = A.B^T for few rows of A (a token, or a batch of them, in
// decoding: at most 16, or 64 where C is narrow, see mx_few_rows) and MXFP4 B:
// B is streamed once, A is MXFP4 or 16-bit.
//
// Bound by memory: half a byte of codes and 1/32 of scales per element of B,
// and the latency of asking for them.  A workgroup owns 16 NT columns of C
// (rows of B) and its NW waves take the spans of 512 k in turn, each with the
// next span's operands on their way while it multiplies one, so nearly all of
// B is in flight at once; the waves' parts are added in LDS at the end, in
// wave order.
//
// B goes straight to registers as the matrix instructions want it, row l % 16
// in lane l, and lane group g = l / 16 takes the blocks 4g .. 4g + 3 of a span,
// one in each of four steps: its scales are four neighbouring bytes.  Such a
// load touches a line per lane, which the address unit takes one at a time: a
// quarter of its rate, still above what HBM delivers.  A read the same way
// costs as much per 16 rows again (16-bit A four times that), in every
// workgroup: 64 rows x 8192 x 8192 took 28 us (MXFP4) and 44 (16-bit).  So A
// is read along its rows and turned in a piece of LDS of the wave's own,
// without barriers.  (Turning B through LDS too, in stages that the workgroup
// shares, keeps too little in flight: one token x 8192 x 8192 12 to 17 us
// against 9.6.)  Where B has many rows and A is 16-bit, several waves share A.
//
// A's piece: 16 MT rows of 16 chunks of 16 bytes; MXFP4: a span, chunk 4g + s
// for step s; 16-bit: a step, chunk 4g + t with the step's t-th eight elements
// of group g's block.  Chunk 4g + x of row r lies at (4x + g) ^ (r & 15): of
// the sixteen lanes that LDS serves at a time (0-3, 12-15, 20-23, 24-27, and so
// on) eight are rows 0-3 and 12-15 of one group and eight rows 4-11 of the
// next, whose g differs in bit 0, so all sixteen places differ.
#include "mxfp4.h"

namespace sgemm {
namespace {

// Order between the LDS accesses of one wave's lanes: LDS serves a wave's
// instructions in order, so only the compiler has to keep them.
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// SHARED: the waves, four of them, take columns of their own and walk k
// together; each brings the piece of A of one of a span's four steps, two spans
// in LDS in turn.
template <MxType A, MxType OUT, int MT, int NT, int NW, bool SHARED>
__global__ __launch_bounds__(64 * NW, MT * NT == 1 ? 4 : NW == 8 ? 2 : 1) void mx_rows_kernel(MxGemmArgs p) {
    constexpr bool MX = A == MxType::mxfp4;
    static_assert(!SHARED || (NW == 4 && !MX), "a wave to each of a span's steps");
    constexpr int PIECE = 16 * MT * 16;                  // chunks of a wave's piece of A
    constexpr int PART = MT * NT * 64;                   // and of its results
    constexpr int MINE = PIECE > PART ? PIECE : PART;
    __shared__ __attribute__((aligned(16))) uint4 lds[SHARED ? 2 * NW * PIECE : NW * MINE];
    __shared__ __attribute__((aligned(16))) uint4 lds_sa[MX ? NW * 16 * MT : 1];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, g = lane >> 4;
    uint4* as = lds + wave * (SHARED ? PIECE : MINE);
    uint4* const ss = lds_sa + (MX ? wave * 16 * MT : 0);
    const long long first = ((long long)blockIdx.x * (SHARED ? NW : 1) + (SHARED ? wave : 0)) * (16 * NT);
    const long long n0 = SHARED ? min(first, (long long)p.N - 1) : first;
    const long long ks = ((long long)p.K + 31) / 32;
    const int nlast = (int)min((long long)p.N - 1 - n0, 16ll * NT - 1);   // rows past B's last read it again
    // Addresses: a wave-uniform base and a 32-bit offset of the lane's own.
    const unsigned char* const B = p.B + n0 * p.ldb;
    const unsigned char* const SB = p.SB + n0 * p.ldsb;
    unsigned ob[NT], os[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const unsigned r = (unsigned)min(16 * j + li, nlast);
        ob[j] = r * (unsigned)p.ldb + 64 * g;
        os[j] = r * (unsigned)p.ldsb + 4 * g;
    }
    struct Span {
        uint4 b[NT][4];
        unsigned s[NT];
    };
    auto load_b = [&](Span& t, long long k0) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int h = 0; h < 4; ++h) __builtin_memcpy(&t.b[j][h], B + k0 / 2 + 16 * h + ob[j], 16);
            __builtin_memcpy(&t.s[j], SB + k0 / 32 + os[j], 4);
        }
    };
    // A's piece: instruction u, lane l: row 4u + l / 16, chunk l % 16.  Rows
    // past M are not loaded; what LDS holds for them reaches only outputs that
    // do not exist.
    struct Piece {
        uint4 a[4 * MT], s;
    };
    const unsigned chunk = MX ? 16 * li : 256 * (li >> 2) + 16 * (li & 3);
    const unsigned oa = (unsigned)g * (unsigned)p.lda + chunk;
    auto load_a = [&](Piece& t, long long k0, int s) __attribute__((always_inline)) {
        const unsigned char* const base = p.A + (MX ? k0 / 2 : 2 * k0 + 64 * s);
#pragma unroll
        for (int u = 0; u < 4 * MT; ++u)
            if (4 * u + g < p.M) __builtin_memcpy(&t.a[u], base + 4 * u * p.lda + oa, 16);
        if constexpr (MX)
            if (lane < p.M) __builtin_memcpy(&t.s, p.SA + k0 / 32 + (unsigned)lane * (unsigned)p.ldsa, 16);
    };
    // The same for the span that K ends in.
    auto load_b_end = [&](Span& t, long long k0) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int h = 0; h < 4; ++h)
                t.b[j][h] = mx_codes16(B + (ob[j] - 64 * g), k0 / 2 + 64 * g + 16 * h, p.K);
            unsigned w[1];
            mx_scales<4>(SB + (os[j] - 4 * g), k0 / 32 + 4 * g, ks, w);
            t.s[j] = w[0];
        }
    };
    auto load_a_end = [&](Piece& t, long long k0, int s) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < 4 * MT; ++u)
            if (4 * u + g < p.M) {
                const unsigned char* const row = p.A + 4 * u * p.lda + (unsigned)g * (unsigned)p.lda;
                if constexpr (MX)
                    t.a[u] = mx_codes16(row, k0 / 2 + chunk, p.K);
                else
                    t.a[u] = mx_bytes16(row, 2 * k0 + 64 * s + chunk, 2ll * p.K);
            }
        if constexpr (MX)
            if (lane < p.M) t.s = mx_bytes16(p.SA + (unsigned)lane * (unsigned)p.ldsa, k0 / 32, ks);
    };
    auto place_a = [&](const Piece& t) __attribute__((always_inline)) {
        wave_order();
#pragma unroll
        for (int u = 0; u < 4 * MT; ++u) {
            const int r = 4 * u + g;
            if (r < p.M) {
                const int at = r * 16 + ((((li & 3) << 2) | (li >> 2)) ^ (r & 15));
                lds_poison_f4(&as[at]);
                as[at] = t.a[u];
            }
        }
        if constexpr (MX)
            if (lane < p.M) ss[lane] = t.s;
        wave_order();
    };
    mx_f4 acc[MT][NT] = {};
    // Step h of a span: lane group g has block 4g + h.
    auto multiply_mx = [&](const Span& t) __attribute__((always_inline)) {
        unsigned sa[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) sa[i] = reinterpret_cast<const unsigned*>(ss + 16 * i + li)[g];
        static_for<4>([&](auto h) {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const uint4 a = as[(16 * i + li) * 16 + ((4 * h + g) ^ li)];
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[i][j] = mfma_mx<h>(t.b[j][h], t.s[j], a, sa[i], acc[i][j]);
            }
        });
    };
    auto multiply_16 = [&](const Span& t, auto h) __attribute__((always_inline)) {
        unsigned byte[NT];
        bool in_range = true, ok = true;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            byte[j] = t.s[j] >> (8 * h) & 255u;
            ok = ok && f16_holds(byte[j]);
        }
        if constexpr (A == MxType::f16) in_range = __all(ok);
        auto steps = [&](auto split) __attribute__((always_inline)) {
            static_for<4>([&](auto x) {
                uint4 v[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint4 q = t.b[j][h];
                    v[j] = decode8<A, split>(x == 0 ? q.x : x == 1 ? q.y : x == 2 ? q.z : q.w, mx_scale(byte[j]));
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    mfma_row<A, split, NT>(v, as[(16 * i + li) * 16 + ((4 * x + g) ^ li)], acc[i]);
            });
        };
        if (in_range)
            steps(std::false_type{});
        else
            steps(std::true_type{});
    };
    const int spans = p.K / 512;      // whole ones
    if constexpr (SHARED) {
        const int all = (int)(((long long)p.K + 511) / 512);
        Span cur, next;
        Piece a;
        // The span's pieces are there for all waves once the last barrier is
        // passed; the next span's go to the other half meanwhile.
        auto fetch = [&](Span& t, int i) __attribute__((always_inline)) {
            if (i < spans) {
                load_b(t, 512ll * i);
                load_a(a, 512ll * i, wave);
            } else {
                load_b_end(t, 512ll * i);
                load_a_end(a, 512ll * i, wave);
            }
        };
        auto half = [&](int i) { return lds + (i & 1) * (NW * PIECE); };
        if (all > 0) {
            fetch(cur, 0);
            as = half(0) + wave * PIECE;
            place_a(a);
        }
        __syncthreads();
        for (int i = 0; i < all; ++i) {
            if (i + 1 < all) fetch(next, i + 1);
            static_for<4>([&](auto h) {
                as = half(i) + h * PIECE;
                multiply_16(cur, h);
            });
            if (i + 1 < all) {
                as = half(i + 1) + wave * PIECE;
                place_a(a);
            }
            cur = next;
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) store4<OUT>(p, 16 * i + li, first + 16 * j + 4 * g, acc[i][j]);
        return;
    }
    Span cur, next;
    Piece a;
    if (wave < spans) {
        load_b(cur, 512ll * wave);
        load_a(a, 512ll * wave, 0);
    }
    for (int i = wave; i < spans; i += NW) {
        const long long k0 = 512ll * i, k1 = 512ll * (i + NW);
        const bool more = i + NW < spans;
        if (more) load_b(next, k1);
        if constexpr (MX) {
            place_a(a);
            if (more) load_a(a, k1, 0);
            multiply_mx(cur);
        } else {
            static_for<4>([&](auto h) {
                place_a(a);
                if constexpr (h < 3)
                    load_a(a, k0, h + 1);
                else if (more)
                    load_a(a, k1, 0);
                multiply_16(cur, h);
            });
        }
        cur = next;
    }
    if (spans % NW == wave && 512ll * spans < p.K) {
        const long long k0 = 512ll * spans;
        load_b_end(cur, k0);
        if constexpr (MX) {
            load_a_end(a, k0, 0);
            place_a(a);
            multiply_mx(cur);
        } else {
            static_for<4>([&](auto h) {
                load_a_end(a, k0, h);
                place_a(a);
                multiply_16(cur, h);
            });
        }
    }
    __syncthreads();
    mx_f4* const part = reinterpret_cast<mx_f4*>(lds);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) part[wave * MINE + (i * NT + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int t = wave; t < MT * NT; t += NW) {
        mx_f4 v = part[t * 64 + lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) v += part[w * MINE + t * 64 + lane];
        store4<OUT>(p, 16 * (t / NT) + li, n0 + 16 * (t % NT) + 4 * g, v);
    }
}

template <MxType A, MxType OUT, int MT, int NT, int NW, bool SHARED = false>
hipError_t launch_cfg(const MxGemmArgs& a, hipStream_t s) {
    constexpr int columns = 16 * NT * (SHARED ? NW : 1);
    const unsigned grid = (unsigned)(((long long)a.N + columns - 1) / columns);
    mx_rows_kernel<A, OUT, MT, NT, NW, SHARED><<<grid, 64 * NW, 0, s>>>(a);
    return hipGetLastError();
}

template <MxType A, MxType OUT, int MT>
hipError_t launch_mt(const MxGemmArgs& a, hipStream_t s) {
    // More columns to a workgroup read A less often, fewer leave more
    // workgroups.  us at K = 8192, N = 65536 and 8192 (binary16 A: 65536 and, of
    // 16 rows, 8192):
    //                           MXFP4 A            bfloat16 A          binary16 A
    //                      one row    16 rows   one row   16 rows    one   16 rows
    //   16 columns, 8 waves  60 11.0   79 12.5   73 12.3  119 17.9    72   121 18.2
    //   32 columns, 8 waves  60 10.9   74 12.1   73 12.7  106 16.2    77   108 16.6
    //   32 columns, 4 waves  60 12.7   71 14.8   68 15.0   98 20.4    72   102 20.9
    //   64 columns, 4 waves  57 15.0   64 17.3   67 19.7   83 24.4    83   120 28.2
    //   4 x 32, A shared                         75 45.5   84 47.5    74    82 49.0
    // (N = K = 1024: 16 columns 2.7, 32 columns 3.0.)
    // One row of 16-bit A takes 256 threads to 32 columns while a launch holds
    // them (N to 2^29 - 32), past that the shared form's 128.
    if constexpr (MT == 1) {   // (more than 16 rows come here only where N < 64 CUs)
        if (a.N >= 128 * a.cus) {
            if constexpr (A == MxType::mxfp4)
                return launch_cfg<A, OUT, 1, 4, 4>(a, s);
            else
                return a.M == 1 && a.N <= (1 << 29) - 32 ? launch_cfg<A, OUT, 1, 2, 4>(a, s)
                                                         : launch_cfg<A, OUT, 1, 2, 4, true>(a, s);
        }
    }
    if (a.N >= 32 * a.cus && a.M > 1) return launch_cfg<A, OUT, MT, MT == 4 && A == MxType::f16 ? 1 : 2, 8>(a, s);
    return launch_cfg<A, OUT, MT, 1, 8>(a, s);
}

template <MxType A, MxType OUT>
hipError_t launch_a(const MxGemmArgs& a, hipStream_t s) {
    if (a.M <= 16) return launch_mt<A, OUT, 1>(a, s);
    if (a.M <= 32) return launch_mt<A, OUT, 2>(a, s);
    return launch_mt<A, OUT, 4>(a, s);
}

}  // namespace

hipError_t launch_mx_rows(const MxGemmArgs& a, MxType a_type, MxType out, hipStream_t s) {
    if (a_type == MxType::bf16) return launch_a<MxType::bf16, MxType::f32>(a, s);
    if (a_type == MxType::f16) return launch_a<MxType::f16, MxType::f32>(a, s);
    return out == MxType::f32 ? launch_a<MxType::mxfp4, MxType::f32>(a, s)
                              : launch_a<MxType::mxfp4, MxType::bf16>(a, s);
}

}  // namespace sgemm
