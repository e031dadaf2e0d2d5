// Rotary positions on the way from a product's output to where attention reads: queries and
// keys out of place or in place, keys into a paged cache with their values beside them.
// Pair i < r/2 of a head's first r elements -- (i, i + r/2) or (2i, 2i + 1) -- turns by
// theta = p f_i and is scaled by c; the other elements pass through:
//     a' = c (a cos theta - b sin theta),   b' = c (b cos theta + a sin theta)
//
// The angle.  f_i / 2 pi, the turns that a position adds, is kept as a fraction of 2^64, so the
// angle modulo a turn is the low 64 bits of one integer product: exact but for the fraction's
// own rounding, |p| 2^-63 turns at most.  No table of positions is built,
// read or outgrown (at 131072 positions of 64 frequencies one would fill half the L2).  The nearest quarter turn is
// split off, the rest taken to 2^-55 turn and 24 bits, and its sine and cosine, |x| <= pi/4, are their Taylor
// polynomials to x^9 and x^10, whose next terms are below 1.8e-9 and 1.2e-10.
//
// Work.  A unit is two vectors of a head: those at i and i + r/2, or interleaved pairs' vectors j and
// j + half of them (side by side, each lane would touch half of every 32 bytes: 36 us against 28 for
// 8192 tokens of 40 heads); of the part that passes through likewise.  An angle is formed once for
// many heads.  Each element is read and written once.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "foak_ce.h"
#include "internal.h"
#include "launch_once.h"
#include "rotary.h"

namespace foak {

namespace {

constexpr int kThreads = 256;

// W elements of ES bytes in one access.
template <int ES, int W>
struct Piece {
    static constexpr int kBytes = ES * W;
    uint32_t w[kBytes >= 4 ? kBytes / 4 : 1];

    __device__ __forceinline__ void load(const char* p) {
        if constexpr (kBytes == 16) {
            const uint4 v = ld_global_v4(p);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else if constexpr (kBytes == 8) {
            asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p) : "memory");
        } else if constexpr (kBytes == 4) {
            asm volatile("ld.global.b32 %0, [%1];" : "=r"(w[0]) : "l"(p) : "memory");
        } else {
            asm volatile("ld.global.u16 %0, [%1];" : "=r"(w[0]) : "l"(p) : "memory");
        }
    }
    __device__ __forceinline__ void load_shared(const char* p) {
        if constexpr (kBytes == 16) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else if constexpr (kBytes == 8) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x; w[1] = v.y;
        } else if constexpr (kBytes == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            w[0] = *reinterpret_cast<const unsigned short*>(p);
        }
    }
    __device__ __forceinline__ void store(char* p) const {
        if constexpr (kBytes == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
        else *reinterpret_cast<unsigned short*>(p) = static_cast<unsigned short>(w[0]);
    }
    __device__ __forceinline__ void get(float (&f)[W]) const {
        if constexpr (ES == 4) {
#pragma unroll
            for (int k = 0; k < W; ++k) f[k] = __uint_as_float(w[k]);
        } else if constexpr (W == 1) {
            f[0] = bf16_lo(w[0]);
        } else {
#pragma unroll
            for (int k = 0; k < W / 2; ++k) {
                f[2 * k] = bf16_lo(w[k]);
                f[2 * k + 1] = bf16_hi(w[k]);
            }
        }
    }
    // rounded to nearest even, the one rounding of the output
    __device__ __forceinline__ void set(const float (&f)[W]) {
        if constexpr (ES == 4) {
#pragma unroll
            for (int k = 0; k < W; ++k) w[k] = __float_as_uint(f[k]);
        } else if constexpr (W == 1) {
            w[0] = pack_bf16x2(f[0], 0.f);
        } else {
#pragma unroll
            for (int k = 0; k < W / 2; ++k) w[k] = pack_bf16x2(f[2 * k], f[2 * k + 1]);
        }
    }
};

// c times cosine and sine of `turn` 2^-64 turns.  What is left of the nearest quarter turn is taken to 2^-55 turn, and to
// 24 bits where it is larger: the upper word as a float, less 1, and 1.f with the lower word's first 23 bits behind it,
// whose sum is exact where the upper word is 0 or -1.  (Of the upper word alone, 2^-32 turn, the sine of a slow pair near
// position 0 would be off by half a percent; a 64-bit conversion instead: 3001 fp32 tokens 11.1 us against 9.9.)
__device__ __forceinline__ void turn_cos_sin(uint64_t turn, float c, float sign, float& co, float& si) {
    const uint32_t hi = static_cast<uint32_t>(turn >> 32), lo = static_cast<uint32_t>(turn);
    const uint32_t quarter = (hi + 0x20000000u) & 0xc0000000u;
    const int32_t below = static_cast<int32_t>(hi - quarter - 1u);  // [-2^29 - 1, 2^29): an eighth of a turn
    const float rest = static_cast<float>(below) + __uint_as_float(0x3f800000u | lo >> 9);
    const float x = rest * 1.4629180792671596e-9f;  // 2 pi / 2^32
    const float z = x * x;
    float s = fmaf(z, 2.7557319223985893e-6f, -1.9841269841269841e-4f);
    s = fmaf(z, s, 8.3333333333333333e-3f);
    s = fmaf(z, s, -1.6666666666666667e-1f);
    s = fmaf(x * z, s, x);
    float k = fmaf(z, -2.7557319223985888e-7f, 2.4801587301587302e-5f);
    k = fmaf(z, k, -1.3888888888888889e-3f);
    k = fmaf(z, k, 4.1666666666666667e-2f);
    k = fmaf(z, k, -0.5f);
    k = fmaf(z, k, 1.f);
    const bool odd = quarter & 0x40000000u;
    co = __uint_as_float(__float_as_uint(c * (odd ? s : k)) ^ ((quarter + 0x40000000u) & 0x80000000u));
    si = __uint_as_float(__float_as_uint(c * sign * (odd ? k : s)) ^ (quarter & 0x80000000u));
}

// Where a unit's vectors lie in its head, and whose angles they take.
struct Unit {
    int at0, at1;      // elements
    int freq0, freq1;  // of the first pair of each vector (half layout and single elements: of both); -1: passes through
    bool two;          // the second vector is there
};

// Units of a head that turn: pairs of vectors in the half layout (or of single elements); of interleaved vectors
// the j-th with the j-th of the second half, so that neighbouring units lie side by side.
template <int W, bool INTERLEAVED>
__host__ __device__ __forceinline__ int turning_of(int r) {
    return INTERLEAVED && W > 1 ? (r / W + 1) / 2 : r / 2 / W;
}

template <int W, bool INTERLEAVED>
__host__ __device__ __forceinline__ int units_of(int d, int r) {
    return turning_of<W, INTERLEAVED>(r) + ((d - r) / W + 1) / 2;
}

template <int W, bool INTERLEAVED>
__device__ __forceinline__ Unit unit_of(int j, int d, int r) {
    const int turning = turning_of<W, INTERLEAVED>(r);
    Unit u;
    if (j < turning) {
        if constexpr (!INTERLEAVED) {
            u.at0 = j * W;
            u.at1 = r / 2 + j * W;
            u.freq0 = u.freq1 = j * W;
        } else if constexpr (W == 1) {
            u.at0 = 2 * j;
            u.at1 = 2 * j + 1;
            u.freq0 = u.freq1 = j;
        } else {
            u.at0 = j * W;
            u.at1 = (j + turning) * W;
            u.freq0 = u.at0 / 2;
            u.freq1 = u.at1 / 2;
        }
        u.two = u.at1 < r;
        return u;
    }
    j -= turning;
    u.at0 = r + j * W;
    u.at1 = u.at0 + ((d - r) / W + 1) / 2 * W;
    u.freq0 = u.freq1 = -1;
    u.two = u.at1 < d;
    return u;
}

// Division of numbers below 2^31 by one that a launch keeps: multiplied by 2^(31 + b) / d, rounded up,
// where d <= 2^b; the product's excess stays below 1 / d of the quotient's unit.
struct Divisor {
    unsigned d, mul, shift;
};

Divisor divisor(unsigned d) {
    Divisor v = {d, 0, 0};
    if (d == 1) return v;
    unsigned b = 1;
    while ((1ull << b) < d) ++b;
    v.mul = static_cast<unsigned>((1ull << (31 + b)) / d + 1);
    v.shift = b - 1;
    return v;
}

__device__ __forceinline__ unsigned quotient(unsigned n, const Divisor& v) {
    return v.d == 1 ? n : __umulhi(n, v.mul) >> v.shift;
}

// The rotation of a unit's two vectors by W cosines and sines.
template <int W, bool INTERLEAVED>
__device__ __forceinline__ void rotate(float (&x)[W], float (&y)[W], const float (&co)[W], const float (&si)[W]) {
    if constexpr (INTERLEAVED && W > 1) {
#pragma unroll
        for (int k = 0; k < W / 2; ++k) {
            const float a = x[2 * k], b = x[2 * k + 1], c = y[2 * k], d = y[2 * k + 1];
            x[2 * k] = fmaf(a, co[k], -b * si[k]);
            x[2 * k + 1] = fmaf(b, co[k], a * si[k]);
            y[2 * k] = fmaf(c, co[W / 2 + k], -d * si[W / 2 + k]);
            y[2 * k + 1] = fmaf(d, co[W / 2 + k], c * si[W / 2 + k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const float a = x[k], b = y[k];
            x[k] = fmaf(a, co[k], -b * si[k]);
            y[k] = fmaf(b, co[k], a * si[k]);
        }
    }
}

// The items of a token are the units of its heads: those of move 0, then of 1 and 2, heads by heads,
// units fastest.
struct Items {
    Divisor per_token;
    Divisor units[3];
    unsigned end[2];  // of a token's items of move 0, and of 1
    unsigned count;   // of the launch
    int64_t t0;       // the first token
};

// Jobs of warps: a token's are runs of the items of move 0, then of 1 and 2.
struct Jobs {
    Divisor per_token;
    Divisor units[3];
    unsigned end[3];    // of a token's jobs of each move
    unsigned share[3];  // items of a job, a multiple of 32
    unsigned items[3];  // of a token
    unsigned count;     // of the launch
    int turning;        // units of a head that turn
    int freqs;          // r / 2
    int table_bytes;    // of a warp's shared memory
    int warp_bytes;
    int64_t t0;         // the first token
};

struct Item {
    unsigned m, h;  // move, head
    int j;          // unit of the head
    Unit u;
};

template <int W, bool INTERLEAVED>
__device__ __forceinline__ Item item_of(unsigned at, const RotaryArgs& a, const Items& it) {
    Item x;
    x.m = at >= it.end[1] ? 2 : at >= it.end[0] ? 1 : 0;
    at -= x.m == 2 ? it.end[1] : x.m == 1 ? it.end[0] : 0;
    x.h = quotient(at, it.units[x.m]);
    x.j = static_cast<int>(at - x.h * it.units[x.m].d);
    x.u = unit_of<W, INTERLEAVED>(x.j, a.move[x.m].d, a.move[x.m].r);
    return x;
}

// a / b of numbers that are not negative, by the 32-bit division where both fit (they nearly always do).
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
    if (static_cast<uint64_t>(a | b) >> 32) return a / b;
    return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}

// Where token t of a move goes, in elements; -1: nowhere.
__device__ __forceinline__ int64_t place_of(const RotaryArgs& a, const HeadMove& mv, int64_t t) {
    if (!a.slots) return t * mv.dst_t;
    const int64_t slot = a.slots[t];
    if (static_cast<uint64_t>(slot) >= static_cast<uint64_t>(a.capacity)) {  // padding, or past the cache
        if (slot >= 0 && a.err) atomicOr(reinterpret_cast<unsigned*>(a.err), FOAK_ERRBIT_PAGE_RANGE);
        return -1;
    }
    if (!mv.paged) return t * mv.dst_t;
    const int64_t page = divide(slot, a.page_size);
    return page * mv.dst_page + (slot - page * a.page_size) * mv.dst_t;
}

constexpr int kWarpCtas = 5;
constexpr int kMaxShare = 4;  // items of a lane (8192 tokens of 40 heads: 27.1 us; two 31, six 28)

// One piece from global to shared memory, completed by this thread's wait_group (a hardware wait, no spin), or
// at once where a piece is smaller than the asynchronous copy's four bytes.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const char* src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
    else if constexpr (BYTES >= 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
    else *static_cast<unsigned short*>(dst) = *reinterpret_cast<const unsigned short*>(src);
}

// A warp's job is a run of the items of a token's move.  The loads of all of them go out at once, to the warp's
// part of shared memory, each lane its own; behind them the warp forms the token's cosines and sines, once for
// all heads of the job, beside: for W > 1 vectors of (two cosines, two sines), those of one unit `turning`
// vectors apart, so that neighbouring units read neighbouring 16 bytes; for W = 1 a cosine and a sine a
// unit.  A lane keeps its unit from round to round where the units of a head divide 32.
//
// Bound by memory latency (it is the bytes in flight that count, and shared memory holds more of them than
// registers would) and by the issue slots.  8192 tokens of 32 + 8 heads x 128 bf16: 27.1 us, 6.2 TB/s (a copy of as
// many bytes 26.2); with jobs over all moves' items 27.9 (290 instructions a round, now 251), with the loads in
// registers, two rounds ahead, 32.0; each item's angles by its own thread 41.5, by CTAs with a table a CTA 36.2.
template <int ES, int W, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, kWarpCtas)
    rotary_warp_kernel(const __grid_constant__ RotaryArgs a, const __grid_constant__ Jobs jb) {
    griddep_launch_dependents();  // programmatic dependent launch: no global access before the wait
    griddep_wait();
    constexpr int kBytes = ES * W;
    using Vec = Piece<ES, W>;
    extern __shared__ float4 shared[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned job = blockIdx.x * (kThreads / 32) + warp;
    if (job >= jb.count) return;
    const unsigned token = quotient(job, jb.per_token);
    const int64_t t = jb.t0 + token;
    unsigned run = job - token * jb.per_token.d;
    const int m = run >= jb.end[1] ? 2 : run >= jb.end[0] ? 1 : 0;
    run -= m == 2 ? jb.end[1] : m == 1 ? jb.end[0] : 0;
    const HeadMove& mv = a.move[m];
    const unsigned begin = run * jb.share[m], end = min(begin + jb.share[m], jb.items[m]), units = jb.units[m].d;
    const bool steady = 32 % units == 0;  // a lane's unit is the same in every round
    const unsigned h_first = quotient(begin + lane, jb.units[m]);
    const int j_first = static_cast<int>(begin + lane - h_first * units);
    const Unit u_first = unit_of<W, INTERLEAVED>(j_first, mv.d, mv.r);
    char* mine = reinterpret_cast<char*>(shared) + warp * jb.warp_bytes;
    float* cs = reinterpret_cast<float*>(mine);
    char* const data = mine + jb.table_bytes + lane * kBytes;  // [round][two vectors][lanes]
    // body(unit, its number, head, the lane's place in `data`) for each of the lane's items
    auto rounds = [&](auto&& body) {
        Unit u = u_first;
        int j = j_first;
        unsigned h = h_first;
        char* at = data;
        for (unsigned i = begin + lane; i < end; i += 32, at += 64 * kBytes) {
            body(u, j, h, at);
            if (steady) h += 32 / units;
            else {
                h = quotient(i + 32, jb.units[m]);
                j = static_cast<int>(i + 32 - h * units);
                u = unit_of<W, INTERLEAVED>(j, mv.d, mv.r);
            }
        }
    };
    const char* src = mv.src + t * mv.src_t * ES;
    const int64_t src_h = mv.src_h * ES, dst_h = mv.dst_h * ES;
    rounds([&](const Unit& u, int, unsigned h, char* at) {
        const char* from = src + h * src_h;
        copy_async<kBytes>(at, from + u.at0 * ES);
        if (u.two) copy_async<kBytes>(at + 32 * kBytes, from + u.at1 * ES);
    });
    asm volatile("cp.async.commit_group;" ::: "memory");
    const int64_t place = place_of(a, mv, t);
    if (mv.r) {
        const uint64_t pos = static_cast<uint64_t>(a.positions[t]);
#pragma unroll 1
        for (int f = lane; f < jb.freqs; f += 32) {
            // frequency f is number k of unit i
            int i = f / W, k = f % W;
            if constexpr (INTERLEAVED && W > 1) {
                i = f / (W / 2);
                k = f % (W / 2);
                if (i >= jb.turning) {
                    i -= jb.turning;
                    k += W / 2;
                }
            }
            float co, si;
            turn_cos_sin(pos * a.turns[f], a.factor, a.sign, co, si);
            float* c = cs + (W == 1 ? 2 * i : (k / 2 * jb.turning + i) * 4 + k % 2);
            c[0] = co;
            c[W == 1 ? 1 : 2] = si;
        }
        __syncwarp();
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (place < 0) return;
    char* dst = mv.dst + place * ES;
    rounds([&](const Unit& u, int j, unsigned h, char* at) {
        Vec v, w;
        v.load_shared(at);
        if (u.two) w.load_shared(at + 32 * kBytes);
        else w = v;
        if (u.freq0 >= 0) {
            float e[W], f[W], co[W], si[W];
            if constexpr (W == 1) {
                const float2 c = *reinterpret_cast<const float2*>(cs + 2 * j);
                co[0] = c.x;
                si[0] = c.y;
            } else {
                const float4* table = reinterpret_cast<const float4*>(cs) + j;
#pragma unroll
                for (int k = 0; k < W / 2; ++k) {
                    const float4 c = table[k * jb.turning];
                    co[2 * k] = c.x;
                    co[2 * k + 1] = c.y;
                    si[2 * k] = c.z;
                    si[2 * k + 1] = c.w;
                }
            }
            v.get(e);
            w.get(f);
            rotate<W, INTERLEAVED>(e, f, co, si);
            v.set(e);
            w.set(f);
        }
        char* to = dst + h * dst_h;
        v.store(to + u.at0 * ES);
        if (u.two) w.store(to + u.at1 * ES);
    });
}

// The same without shared memory, an item a thread with its own angles: calls too small to fill the GPU, whose
// latency this shortens (a token of 32 + 8 heads 1.9 us against 2.6), and heads whose table does not fit.
// At most 32 registers, 40 for eight angles (3001 fp32 tokens, four angles: 9.9 us, unbounded 10.7; 300 bf16 tokens of
// 56 heads x 96, eight: 3.9, unbounded 4.0, with 32 registers 4.0; 512 of 40 x 128 4.3, unbounded 4.3, 32 registers 5.8).
template <int ES, int W, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, W == 8 ? 6 : 8)
    rotary_kernel(const __grid_constant__ RotaryArgs a, const __grid_constant__ Items it) {
    griddep_launch_dependents();  // programmatic dependent launch: no global access before the wait
    griddep_wait();
    const unsigned item = blockIdx.x * kThreads + threadIdx.x;
    if (item >= it.count) return;
    const unsigned token = quotient(item, it.per_token);
    const Item x = item_of<W, INTERLEAVED>(item - token * it.per_token.d, a, it);
    const HeadMove& mv = a.move[x.m];
    const int64_t t = it.t0 + token, to = place_of(a, mv, t);
    if (to < 0) return;
    const char* src = mv.src + (t * mv.src_t + x.h * mv.src_h) * ES;
    Piece<ES, W> v[2];
    v[0].load(src + x.u.at0 * ES);
    if (x.u.two) v[1].load(src + x.u.at1 * ES);
    else v[1] = v[0];
    if (x.u.freq0 >= 0) {
        float co[W], si[W], p[W], q[W];
        const uint64_t pos = static_cast<uint64_t>(a.positions[t]);
#pragma unroll
        for (int k = 0; k < W; ++k) {
            int f = x.u.freq0 + k;
            if (INTERLEAVED && W > 1 && k >= W / 2) f = x.u.two ? x.u.freq1 + k - W / 2 : x.u.freq0;
            turn_cos_sin(pos * a.turns[f], a.factor, a.sign, co[k], si[k]);
        }
        v[0].get(p);
        v[1].get(q);
        rotate<W, INTERLEAVED>(p, q, co, si);
        v[0].set(p);
        v[1].set(q);
    }
    char* dst = mv.dst + (to + x.h * mv.dst_h) * ES;
    v[0].store(dst + x.u.at0 * ES);
    if (x.u.two) v[1].store(dst + x.u.at1 * ES);
}

constexpr int kTableSmem = 200 * 1024;

template <int ES, int W, bool INTERLEAVED>
cudaError_t launch_heads(const RotaryArgs& a, cudaStream_t s) {
    Items it = {};
    Jobs jb = {};
    unsigned items = 0, rounds = 0, jobs = 0, most = 0;
    for (int m = 0; m < 3; ++m) {
        const HeadMove& mv = a.move[m];
        it.units[m] = divisor(1);
        if (mv.src) {
            it.units[m] = divisor(static_cast<unsigned>(units_of<W, INTERLEAVED>(mv.d, mv.r)));
            jb.items[m] = it.units[m].d * static_cast<unsigned>(mv.H);
            items += jb.items[m];
            const unsigned n = (jb.items[m] + 31) / 32, parts = (n + kMaxShare - 1) / kMaxShare;
            jb.share[m] = (n + parts - 1) / parts * 32;
            jobs += (jb.items[m] + jb.share[m] - 1) / jb.share[m];
            rounds += n;
            most = std::max(most, jb.share[m]);
            if (mv.r) {
                jb.freqs = mv.r / 2;
                jb.turning = turning_of<W, INTERLEAVED>(mv.r);
            }
        }
        if (m < 2) it.end[m] = items;
        jb.end[m] = jobs;
        jb.units[m] = it.units[m];
    }
    it.per_token = divisor(items);
    jb.per_token = divisor(jobs);
    jb.table_bytes = static_cast<int>((static_cast<int64_t>(jb.turning) * W * 8 + 15) / 16 * 16);
    jb.warp_bytes = jb.table_bytes + static_cast<int>(most) * (2 * ES * W);
    const size_t smem = static_cast<size_t>(jb.warp_bytes) * (kThreads / 32);
    // Warps with a table once the rounds fill the GPU several times over, a few times more where an item has four
    // angles or fewer of its own (32 + 8 heads x 128 bf16: 1024 tokens, 10240 rounds, 7.5 us against 6.5 by items, 2048
    // 9.3 against 12.0; 8 + 2 heads x 96 fp32: 4096 tokens, 16384 rounds, 8.7 against 6.5, 8192 12.9 against 13.2)
    const int64_t enough = static_cast<int64_t>(device_sm_count()) * (W == 8 ? 96 : 256);
    const bool by_warps = smem <= kTableSmem && a.T * rounds >= enough;
    if (by_warps) {
        static SmemOnce limit;
        const cudaError_t e = limit.allow(rotary_warp_kernel<ES, W, INTERLEAVED>, kTableSmem);
        if (e != cudaSuccess) return e;
    }
    const unsigned each = by_warps ? jobs : items, per_cta = by_warps ? kThreads / 32 : kThreads;
    const int64_t step = std::max<int64_t>(1, static_cast<int64_t>((1u << 30) / each));  // a launch's count below 2^31
    for (int64_t t0 = 0; t0 < a.T; t0 += step) {
        it.t0 = jb.t0 = t0;
        it.count = jb.count = static_cast<unsigned>(std::min(a.T - t0, step)) * each;
        const dim3 grid((it.count + per_cta - 1) / per_cta), block(kThreads);
        const cudaError_t e = by_warps ? launch_dependent(rotary_warp_kernel<ES, W, INTERLEAVED>, grid, block, smem, s, a, jb)
                                       : launch_dependent(rotary_kernel<ES, W, INTERLEAVED>, grid, block, 0, s, a, it);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <int ES, int W>
cudaError_t launch_width(const RotaryArgs& a, cudaStream_t s) {
    return a.interleaved ? launch_heads<ES, W, true>(a, s) : launch_heads<ES, W, false>(a, s);
}

// The widest access that every vector of every head allows.
int width_of(int es, const RotaryArgs& a) {
    int w = 16 / es;
    auto fits = [&](int64_t elements) {
        while (elements % w) w /= 2;
    };
    for (const HeadMove& mv : a.move) {
        if (!mv.src) continue;
        while (reinterpret_cast<uintptr_t>(mv.src) % (w * es) || reinterpret_cast<uintptr_t>(mv.dst) % (w * es)) w /= 2;
        fits(mv.src_t);
        fits(mv.src_h);
        fits(mv.dst_t);
        fits(mv.dst_h);
        fits(mv.dst_page);
        fits(mv.d);
        fits(a.interleaved ? mv.r : mv.r / 2);
        fits(mv.r);
    }
    return w;
}

// Slots and positions of a step's tokens, a thread a token: the token's sequence is the last one that starts at
// or before it, found by bisection, in shared memory where the starts fit (256 sequences of one token: 8
// dependent loads of an L2 latency each otherwise).
constexpr int kSlotStarts = 4096;
__global__ void __launch_bounds__(kThreads)
    kv_slots_kernel(const int32_t* __restrict__ page_table, int64_t ld_table, int64_t max_pages,
                    const int32_t* __restrict__ cache_lens, const int32_t* __restrict__ seq_starts, int64_t B, int64_t T,
                    int64_t page_size, int64_t num_pages, int64_t* __restrict__ slots, int64_t* __restrict__ positions,
                    int32_t* err) {
    griddep_launch_dependents();  // programmatic dependent launch: no global access before the wait
    griddep_wait();
    __shared__ int32_t kept[kSlotStarts];
    const int32_t* starts = seq_starts;
    if (B < kSlotStarts) {
        for (int i = threadIdx.x; i <= B; i += kThreads) kept[i] = seq_starts[i];
        __syncthreads();
        starts = kept;
    }
    const int64_t t = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    if (t >= T) return;
    int64_t lo = 0, hi = B + 1;  // starts before lo are <= t, those from hi on are not
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (starts[mid] <= t) lo = mid + 1;
        else hi = mid;
    }
    int64_t slot = -1, pos = 0;
    if (lo > 0 && lo <= B) {  // behind no start, or before the first: padding
        const int64_t b = lo - 1, len = cache_lens[b];
        pos = len + (t - starts[b]);
        int64_t id = -1, page = 0;
        if (len >= 0) {
            page = divide(pos, page_size);
            if (page < max_pages) id = page_table[b * ld_table + page];
        }
        if (id >= 0 && id < num_pages) slot = id * page_size + (pos - page * page_size);
        else {
            pos = 0;
            if (err) atomicOr(reinterpret_cast<unsigned*>(err), FOAK_ERRBIT_PAGE_RANGE);
        }
    }
    slots[t] = slot;
    positions[t] = pos;
}

}  // namespace

void rotary_inv_freq(double base, int64_t r, int scaling, double factor, double low, double high, double original,
                     double* inv_freq) {
    const double two_pi = 6.283185307179586476925;
    if (scaling == FOAK_ROTARY_NTK) base *= std::pow(factor, static_cast<double>(r) / static_cast<double>(r - 2));
    // the index at which a frequency makes n turns over the original context
    auto index_of = [&](double n) { return r * std::log(original / (n * two_pi)) / (2.0 * std::log(base)); };
    double first = 0.0, last = 0.0;
    if (scaling == FOAK_ROTARY_RAMP) {
        first = std::max(std::floor(index_of(high)), 0.0);
        last = std::min(std::ceil(index_of(low)), static_cast<double>(r - 1));
        if (!(last > first)) last = first + 0.001;
    }
    for (int64_t i = 0; i < r / 2; ++i) {
        const double f = std::pow(base, -2.0 * static_cast<double>(i) / static_cast<double>(r));
        double stretch = 0.0;  // the share that the factor divides
        if (scaling == FOAK_ROTARY_LINEAR) stretch = 1.0;
        if (scaling == FOAK_ROTARY_BANDS) stretch = (high - original * f / two_pi) / (high - low);
        if (scaling == FOAK_ROTARY_RAMP) stretch = (static_cast<double>(i) - first) / (last - first);
        stretch = std::min(std::max(stretch, 0.0), 1.0);
        inv_freq[i] = f * (1.0 - stretch) + f * stretch / factor;
    }
}

// The quotient by 2 pi as two numbers, the second from the first one's remainder, with 2 pi as two numbers as well.
uint64_t rotary_turns(double inv_freq) {
    constexpr double kTwoPi = 6.283185307179586, kTwoPiRest = 2.4492935982947064e-16;
    const auto fraction = [](double turns) {  // times 2^64, cut off; of the absolute value, whose fraction is exact
        const double size = std::fabs(turns);
        const uint64_t scaled = static_cast<uint64_t>(std::ldexp(size - std::floor(size), 64));
        return turns < 0.0 ? 0 - scaled : scaled;
    };
    const double turns = inv_freq / kTwoPi;
    const double rest = std::fma(-turns, kTwoPiRest, std::fma(-turns, kTwoPi, inv_freq));
    return fraction(turns) + fraction(rest / kTwoPi);
}

cudaError_t launch_rotary(int es, const RotaryArgs& a, cudaStream_t s) {
    if (a.T == 0 || (!a.move[0].src && !a.move[1].src && !a.move[2].src)) return cudaSuccess;
    const int w = width_of(es, a);
    if (es == 2) {
        if (w == 8) return launch_width<2, 8>(a, s);
        if (w == 4) return launch_width<2, 4>(a, s);
        return w == 2 ? launch_width<2, 2>(a, s) : launch_width<2, 1>(a, s);
    }
    if (w == 4) return launch_width<4, 4>(a, s);
    return w == 2 ? launch_width<4, 2>(a, s) : launch_width<4, 1>(a, s);
}

cudaError_t launch_kv_slots(const int32_t* page_table, int64_t ld_table, int64_t max_pages, const int32_t* cache_lens,
                            const int32_t* seq_starts, int64_t B, int64_t T, int64_t page_size, int64_t num_pages,
                            int64_t* slots, int64_t* positions, int32_t* err, cudaStream_t s) {
    if (T == 0) return cudaSuccess;
    const int64_t grid = (T + kThreads - 1) / kThreads;
    return launch_dependent(kv_slots_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, page_table, ld_table,
                            max_pages, cache_lens, seq_starts, B, T, page_size, num_pages, slots, positions, err);
}

}  // namespace foak
