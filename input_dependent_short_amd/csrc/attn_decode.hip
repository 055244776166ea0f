// attn_decode.hip -- attention of one new token per sequence over a paged
// key-value cache, for gfx950:
//   o[s, a] = sum_{t < len_s} p_t v_t,  p = softmax(scale * <q[s, a], k_t>),
// k_t, v_t the rows of query head a's key head, at page pages[s, t / page].
//
// The cache is read once and little is computed on it, so bytes in flight
// decide.  A block takes one (sequence, key head, chunk of the length) and up
// to 16 query heads of the group (one side of the 16 x 16 matrix
// instructions); its waves take tiles of kTok tokens in turn, each wave on its
// own, without barriers: a tile's K and V rows go straight from memory into
// the wave's own LDS stages, one tile ahead of the one being worked on, with
// the page numbers looked up one tile earlier still.  Places past the length
// (and channels past the head's own) are read from a 16-byte zero instead, so
// what the page holds there never enters.  Scores are formed transposed
// (S^T = K Q^T), so that the probabilities are the right operand of
// O^T = V^T P^T without moving between lanes.
// The waves' results are joined in LDS; when the length is cut into several
// chunks each writes its maximum, sum and unscaled fp32 row to the workspace
// and a second launch joins them.
#include <algorithm>

#include "attn_common.h"

namespace dsc {
namespace {

constexpr int kDecWaves = 2;

template <class E>
constexpr int kTok = sizeof(typename E::store_t) == 2 ? 32 : 16;  // tokens per wave tile

__device__ const uint4 kZeroChunk = {0, 0, 0, 0};

struct DecodeParams {
    const void *q, *k, *v;
    const int32_t *pages, *lens;
    void *o;
    float *part;  // (S, Hq, nsplit, hd + 2) fp32: row, maximum (base 2), sum
    int64_t S, qs, num_pages, max_pages;
    int32_t Hq, Hkv, G, hd, page, page_shift, nsplit, chunk, qtiles;
    float c2;
};

template <class E>
struct Mma16;
template <>
struct Mma16<BF16> {
    using frag = bf16x8;
    static constexpr int KC = 32;
    __device__ __forceinline__ static floatx4 mul(frag a, frag b, floatx4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Mma16<F32> {
    using frag = floatx4;
    static constexpr int KC = 16;
    __device__ __forceinline__ static floatx4 mul(frag a, frag b, floatx4 c) {
#pragma unroll
        for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], c, 0, 0, 0);
        return c;
    }
};

// Largest over the four 16-lane groups, in every lane.
__device__ __forceinline__ float groups_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float groups_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

template <class E, int HDC>
__global__ __launch_bounds__(64 * kDecWaves, 1) void attn_decode_kernel(DecodeParams p) {
    using T = Tile<E, HDC>;
    using M = Mma16<E>;
    using S = typename E::store_t;
    using frag = typename M::frag;
    constexpr int TN = kTok<E>, NS = TN / 16, KF = HDC / M::KC, DT = HDC / 16, NW = kDecWaves;
    constexpr int TB = TN * T::RB;               // bytes of a K (or V) tile
    constexpr int INST = TB / 1024, RPI = 1024 / T::RB;  // load instructions per tile, rows per instruction
    __shared__ __align__(16) unsigned char k0s[NW][TB], v0s[NW][TB], k1s[NW][TB], v1s[NW][TB];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, grp = lane >> 4;
    int64_t b = blockIdx.x;
    const int split = (int)(b % p.nsplit);
    b /= p.nsplit;
    const int qt = (int)(b % p.qtiles);
    b /= p.qtiles;
    const int kvh = (int)(b % p.Hkv);
    const int64_t seq = b / p.Hkv;
    const int64_t cap = p.max_pages * p.page;
    int len = p.lens[seq];
    bool bad = len < 0 || len > cap;
    if (bad) len = 0;
    const int t_lo = split * p.chunk, t_hi = (int)min((int64_t)len, (int64_t)t_lo + p.chunk);
    if (split > 0 && t_lo >= len) return;  // the join reads the chunks that the length reaches

    // queries: column col is head qt*16 + col of the group
    const int a = qt * 16 + col;
    const bool live = a < p.G;
    const int64_t head = (int64_t)kvh * p.G + a;
    frag qf[KF];
#pragma unroll
    for (int kc = 0; kc < KF; ++kc) {
        const int d = T::VEC * (4 * kc + grp);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live && d < p.hd) v = *reinterpret_cast<const uint4 *>(static_cast<const S *>(p.q) + seq * p.qs + head * p.hd + d);
        qf[kc] = __builtin_bit_cast(frag, v);
    }

    const int32_t *pages = p.pages + seq * p.max_pages;
    // Page number of this lane's token of the tile at t0 (tokens past the end
    // repeat the last one's: the load is never skipped, so that the loads in
    // flight can be counted).
    auto page_of = [&](int t) __attribute__((always_inline)) {
        return p.page_shift >= 0 ? (uint32_t)t >> p.page_shift : (uint32_t)t / (uint32_t)p.page;
    };
    const int t_last = max(t_hi - 1, 0);
    auto lookup = [&](int t0) __attribute__((always_inline)) -> int32_t {
        return pages[page_of(min(t0 + (lane & (TN - 1)), t_last))];
    };
    // K and V rows of the tile at t0, whose lanes looked up pg.  A page number
    // outside the pool spoils the result.
    auto issue = [&](int t0, int32_t pg, unsigned char *ks, unsigned char *vs) __attribute__((always_inline)) {
        const int t = t0 + (lane & (TN - 1));
        const bool in_pool = pg >= 0 && pg < p.num_pages;
        bad |= t < t_hi && !in_pool;
        const int64_t slot = t < t_hi && in_pool
                                 ? ((int64_t)pg * p.Hkv + kvh) * p.page + (t - (int)page_of(t) * p.page)
                                 : -1;
#pragma unroll
        for (int i = 0; i < INST; ++i) {
            const int row = i * RPI + lane / T::NCH, c = (lane % T::NCH) ^ T::swz(row);
            const int64_t r = __shfl(slot, row);
            const bool in = r >= 0 && c * T::VEC < p.hd;
            const int64_t off = r * p.hd + c * T::VEC;
            const void *kp = in ? (const void *)(static_cast<const S *>(p.k) + off) : (const void *)&kZeroChunk;
            const void *vp = in ? (const void *)(static_cast<const S *>(p.v) + off) : (const void *)&kZeroChunk;
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)kp,
                                             (attn_lds_void *)(ks + 1024 * i), 16, 0, 0);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)vp,
                                             (attn_lds_void *)(vs + 1024 * i), 16, 0, 0);
        }
    };

    floatx4 acc[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[d] = floatx4{0.f, 0.f, 0.f, 0.f};
    float mx = -INFINITY, sum = 0.f;

    auto compute = [&](int t0, const unsigned char *ks, const unsigned char *vs) __attribute__((always_inline)) {
        floatx4 s[NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            s[j] = floatx4{0.f, 0.f, 0.f, 0.f};
            const int r = 16 * j + col;
#pragma unroll
            for (int kc = 0; kc < KF; ++kc)
                s[j] = M::mul(*reinterpret_cast<const frag *>(ks + r * T::RB + 16 * ((4 * kc + grp) ^ T::swz(r))),
                              qf[kc], s[j]);
        }
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (t0 + 16 * j + 4 * grp + i >= t_hi) s[j][i] = -INFINITY;
                top = fmaxf(top, s[j][i]);
            }
        top = groups_max(top);
        const float nm = fmaxf(mx, top), safe = nm == -INFINITY ? 0.f : nm;
        const float al = __builtin_amdgcn_exp2f((mx - safe) * p.c2);
        mx = nm;
        sum *= al;
#pragma unroll
        for (int d = 0; d < DT; ++d) acc[d] *= al;
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[j][i] = __builtin_amdgcn_exp2f((s[j][i] - safe) * p.c2);
                sum += s[j][i];
            }
        frag pf;
        if constexpr (sizeof(S) == 2)
            pf = __builtin_bit_cast(frag, make_uint4(pack_bf16x2(s[0][0], s[0][1]), pack_bf16x2(s[0][2], s[0][3]),
                                                     pack_bf16x2(s[1][0], s[1][1]), pack_bf16x2(s[1][2], s[1][3])));
        else
            pf = s[0];
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            frag vf;
            if constexpr (sizeof(S) == 2) {
                // a 16-lane group reads a 4 x 16 block (rows 4 grp + 0..3), lane i its 8-byte piece i, and gets column i
                const int r = 4 * grp + (col >> 2), c = 2 * d + ((col >> 1) & 1);
                const shortx4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (attn_lds_s4 *)(vs + r * T::RB + 16 * (c ^ T::swz(r)) + 8 * (col & 1)));
                const shortx4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (attn_lds_s4 *)(vs + (r + 16) * T::RB + 16 * (c ^ T::swz(r + 16)) + 8 * (col & 1)));
                vf = __builtin_bit_cast(frag, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
            } else {
                const int ch = 16 * d + col;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 4 * grp + i;
                    vf[i] = *reinterpret_cast<const float *>(vs + r * T::RB + 16 * ((ch >> 2) ^ T::swz(r)) + 4 * (ch & 3));
                }
            }
            acc[d] = M::mul(vf, pf, acc[d]);
        }
    };

    // Tile i of the wave: tokens t_lo + (i*NW + wave)*TN.  While it is worked
    // on, the loads of tile i+1 (2*INST instructions) and, behind them, of the
    // page numbers of tile i+3 are in flight.
    constexpr int STEP = NW * TN;
    const int tw = t_lo + wave * TN;
    const int32_t pg0 = lookup(tw);
    int32_t pg1 = lookup(tw + STEP), pg2 = 0;
    issue(tw, pg0, k0s[wave], v0s[wave]);
    pg2 = lookup(tw + 2 * STEP);
    auto step = [&](int t0, int32_t &pg, unsigned char *ks, unsigned char *vs, unsigned char *kn,
                    unsigned char *vn) __attribute__((always_inline)) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the stage refilled below has been read
        issue(t0 + STEP, pg, kn, vn);
        pg = lookup(t0 + 3 * STEP);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * INST + 1) : "memory");
        compute(t0, ks, vs);
    };
    for (int t0 = tw; t0 < t_hi; t0 += 2 * STEP) {
        step(t0, pg1, k0s[wave], v0s[wave], k1s[wave], v1s[wave]);
        if (t0 + STEP < t_hi) step(t0 + STEP, pg2, k1s[wave], v1s[wave], k0s[wave], v0s[wave]);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    sum = groups_sum(sum);
    if (__any(bad)) sum = __builtin_nanf("");

    // Join of the two waves over the stages: rows (HDC, 16) of each, then (2, 16) maximum and sum.
    static_assert(NW == 2 && NW * TB >= 16 * HDC * 4, "the join takes two waves whose rows fit a stage array each");
    __syncthreads();
    float *r0 = reinterpret_cast<float *>(&k0s[0][0]), *r1 = reinterpret_cast<float *>(&v0s[0][0]);
    float *st = reinterpret_cast<float *>(&k1s[0][0]);
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ch = 16 * d + 4 * grp + i;
            (wave == 0 ? r0 : r1)[ch * 16 + col] = acc[d][i];
        }
    if (grp == 0) {
        st[(wave * 16 + col) * 2] = mx;
        st[(wave * 16 + col) * 2 + 1] = sum;
    }
    __syncthreads();
    for (int e = tid; e < 16 * p.hd; e += 64 * NW) {
        const int c = e / p.hd, d = e - c * p.hd;
        if (qt * 16 + c >= p.G) break;
        const float m0 = st[c * 2], m1 = st[(16 + c) * 2];
        const float m = fmaxf(m0, m1), safe = m == -INFINITY ? 0.f : m;
        const float w0 = __builtin_amdgcn_exp2f((m0 - safe) * p.c2), w1 = __builtin_amdgcn_exp2f((m1 - safe) * p.c2);
        const float l = st[c * 2 + 1] * w0 + st[(16 + c) * 2 + 1] * w1;
        const float r = r0[d * 16 + c] * w0 + r1[d * 16 + c] * w1;
        const int64_t hq = (int64_t)kvh * p.G + qt * 16 + c;
        if (p.nsplit == 1) {
            const float out = r * (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l));
            S *dst = static_cast<S *>(p.o) + (seq * p.Hq + hq) * p.hd + d;
            if constexpr (sizeof(S) == 4) *dst = out;
            else *dst = to_bf16(out);
        } else {
            float *dst = p.part + ((seq * p.Hq + hq) * p.nsplit + split) * (p.hd + 2);
            dst[d] = r;
            if (d == 0) {
                dst[p.hd] = m * p.c2;
                dst[p.hd + 1] = l;
            }
        }
    }
}

// Chunks of one (sequence, query head) joined; one wave each.
template <class E>
__global__ __launch_bounds__(64) void attn_decode_join(DecodeParams p) {
    using S = typename E::store_t;
    const int64_t row = blockIdx.x;
    const int64_t seq = row / p.Hq, cap = p.max_pages * p.page;
    int len = p.lens[seq];
    if (len < 0 || len > cap) len = 0;
    const int n = len > 0 ? (len + p.chunk - 1) / p.chunk : 1;
    const float *src = p.part + row * p.nsplit * (p.hd + 2);
    const int lane = threadIdx.x;
    float m = -INFINITY;
    for (int i = lane; i < n; i += 64) m = fmaxf(m, src[(int64_t)i * (p.hd + 2) + p.hd]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    const float safe = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    for (int i = 0; i < n; ++i) {
        const float *r = src + (int64_t)i * (p.hd + 2);
        l += r[p.hd + 1] * __builtin_amdgcn_exp2f(r[p.hd] - safe);
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    for (int d = lane; d < p.hd; d += 64) {
        float a = 0.f;
        for (int i = 0; i < n; ++i) {
            const float *r = src + (int64_t)i * (p.hd + 2);
            a = __builtin_fmaf(r[d], __builtin_amdgcn_exp2f(r[p.hd] - safe), a);
        }
        S *dst = static_cast<S *>(p.o) + row * p.hd + d;
        if constexpr (sizeof(S) == 4) *dst = a * inv;
        else *dst = to_bf16(a * inv);
    }
}

// Tokens per block and blocks per row: chunks of a multiple of kUnit tokens,
// as long as about kTarget blocks remain over the longest length the page
// table can hold.
constexpr int64_t kUnit = 128, kTarget = 2048;
void plan(int64_t S, int32_t Hq, int32_t Hkv, int32_t page, int64_t max_pages, int32_t &chunk, int32_t &nsplit,
          int32_t &qtiles) {
    const int32_t G = Hq / Hkv;
    qtiles = (G + 15) / 16;
    const int64_t cap = std::max<int64_t>(1, page * max_pages), rows = std::max<int64_t>(1, S * Hkv * qtiles);
    const int64_t per = std::max<int64_t>(1, kTarget / rows);  // chunks per row
    const int64_t c = ((cap + per - 1) / per + kUnit - 1) / kUnit * kUnit;
    chunk = (int32_t)std::min<int64_t>(c, (int64_t)1 << 30);
    nsplit = (int32_t)((cap + chunk - 1) / chunk);
}

template <class E>
void run(DecodeParams &p, hipStream_t s) {
    const dim3 grid((unsigned)(p.S * p.Hkv * p.qtiles * p.nsplit)), block(64 * kDecWaves);
    if (p.hd <= 64) hipLaunchKernelGGL((attn_decode_kernel<E, 64>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((attn_decode_kernel<E, 128>), grid, block, 0, s, p);
    if (p.nsplit > 1) hipLaunchKernelGGL((attn_decode_join<E>), dim3((unsigned)(p.S * p.Hq)), dim3(64), 0, s, p);
}

}  // namespace

size_t attn_decode_workspace(int64_t S, int32_t Hq, int32_t Hkv, int32_t hd, int32_t page, int64_t max_pages) {
    int32_t chunk, nsplit, qtiles;
    plan(S, Hq, Hkv, page, max_pages, chunk, nsplit, qtiles);
    return nsplit > 1 ? sizeof(float) * (size_t)S * Hq * nsplit * (hd + 2) : 0;
}

hipError_t attn_decode(const AttnDecodeProblem &a, hipStream_t s) {
    DecodeParams p{a.q, a.c.k, a.c.v, a.c.pages, a.lens, a.o, static_cast<float *>(a.ws), a.S, a.qs, a.c.num_pages,
                   a.c.max_pages, a.Hq, a.c.Hkv, a.Hq / a.c.Hkv, a.c.hd, a.c.page, -1, 1, 1, 1, a.scale * kLog2e};
    plan(a.S, a.Hq, a.c.Hkv, a.c.page, a.c.max_pages, p.chunk, p.nsplit, p.qtiles);
    if ((a.c.page & (a.c.page - 1)) == 0) p.page_shift = __builtin_ctz((unsigned)a.c.page);
    if (a.dtype == Dtype::BF16) run<BF16>(p, s);
    else run<F32>(p, s);
    return hipGetLastError();
}

}  // namespace dsc
