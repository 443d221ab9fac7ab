// Which nodes of a tree of drafted tokens are kept, from given random numbers,
// so that the tokens that come out are distributed as the target's: a walk from
// the root. At a node with target probabilities p and draft probabilities q
// its children are tried in index order, with r = p and z = 1 at first: child x
// is kept if u z q(x) < r(x), and the walk goes on there; one that is not leaves
// r <- max(r - z q, 0), z <- sum r. Where no child is kept, the next token is
// drawn from r. Drafts that were chosen, not drawn, have q = 1 at the child
// itself: r loses that token, z its weight.
//
// After m rejections r = max(p - c q, 0) with c the sum of the z's so far: max
// (max(p - a q, 0) - b q, 0) = max(p - (a + b) q, 0). So nothing is written
// between rejections, and each takes one pass over a row of p and of q.
//
// Sums are held in fp64: which token is drawn, and whether one is kept, is
// decided next to a border, and a token of probability 2^-17 among 10^5 others
// would fall to the wrong side of fp32 sums.
//
// One workgroup a sequence. What every node's test needs of p and q is fetched
// at once; the walk is then the same code on the same values in every wave.
#include "int8.hpp"

namespace ptq {
namespace {

constexpr int NT = 1024, NW = NT / 64;
constexpr int NODES = TREE_NODES;

struct VerifyArgs {
    const void* P; int64_t ldp;
    const void* Q; int64_t ldq;
    int vocab;
    Drafts d;
    int32_t* path; int32_t* counts; int32_t* next;
};

// 16 bytes of a row that need not be aligned (vocabularies of odd sizes)
template <typename T>
struct Chunk {
    static constexpr int N = 16 / sizeof(T);
    T x[N];
    // the first `left` elements, zeros past them
    __device__ __forceinline__ void load(const T* p, int64_t left) {
        if (left >= N) {
            __builtin_memcpy(x, p, 16);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) x[k] = k < left ? p[k] : (T)0;
        }
    }
    __device__ __forceinline__ float at(int k) const { return load_as_float(x, k); }
};

__device__ __forceinline__ double sum_wave(double x) {
#pragma unroll
    for (int o = 32; o > 0; o /= 2) x += __shfl_xor(x, o, 64);
    return x;
}

// What is left of p: r = max(p - c q, 0), or p without the tokens ex[0 .. nex)
template <typename T, bool DRAWN>
struct Rest {
    const T* p; const T* q;
    double c;
    const int* ex;
    int nex;

    __device__ __forceinline__ double weight(float pv, float qv) const {
        double w = (double)pv;
        if constexpr (DRAWN) w -= c * (double)qv;
        return w < 0 ? 0. : w;      // a NaN stays one
    }
    __device__ __forceinline__ double one(int64_t k) const {
        for (int j = 0; j < nex; ++j)
            if (ex[j] == k) return 0.;
        return weight(load_as_float(p, k), DRAWN ? load_as_float(q, k) : 0.f);
    }
};

// Sums of the 16 shares of the vocabulary, one a wave, into seg; the whole sum comes back.
template <typename T, bool DRAWN>
__device__ double sum_rest(const Rest<T, DRAWN>& r, int vocab, int share, double (&seg)[NW]) {
    constexpr int N = Chunk<T>::N, STEP = 64 * N, U = 4;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t lo = (int64_t)wave * share, hi = std::min<int64_t>(lo + share, vocab);
    double s[U] = {};
    for (int64_t k0 = lo; k0 < hi; k0 += STEP * U) {
        Chunk<T> p[U], q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = k0 + u * STEP + lane * N;
            p[u].load(r.p + k, hi - k);
            if constexpr (DRAWN) q[u].load(r.q + k, hi - k);
        }
        for (int j = 0; j < r.nex; ++j) {
            const int64_t at = r.ex[j] - k0 - lane * N;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < N; ++k)
                    if (at == u * STEP + k) p[u].x[k] = 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < N; ++k) s[u] += r.weight(p[u].at(k), DRAWN ? q[u].at(k) : 0.f);
    }
    const double mine = sum_wave((s[0] + s[1]) + (s[2] + s[3]));
    __syncthreads();      // seg of the sum before has been read
    if (lane == 0) seg[wave] = mine;
    __syncthreads();
    double total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) total += seg[w];
    return total;
}

// First token whose running sum exceeds goal; the last one with a weight where rounding leaves none.
template <typename T, bool DRAWN>
__device__ int draw_rest(const Rest<T, DRAWN>& r, int vocab, int share, const double (&seg)[NW], double goal,
                         double (&part)[NW], int& found) {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    double before = 0;
    int at = -1, last = 0;
    for (int w = 0; w < NW; ++w) {
        if (seg[w] > 0) last = w;
        if (at < 0) {
            if (before + seg[w] > goal) at = w;
            else before += seg[w];
        }
    }
    if (at < 0) {
        at = last;
        before -= seg[last];
    }
    // the share again, each thread its own stretch
    const int64_t lo = (int64_t)at * share, hi = std::min<int64_t>(lo + share, vocab);
    const int64_t each = cdiv(hi - lo, NT), k0 = std::min(lo + t * each, hi), k1 = std::min(k0 + each, hi);
    double sum = 0;
    for (int64_t k = k0; k < k1; ++k) sum += r.one(k);
    double upto = sum;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
        const double x = __shfl_up(upto, o, 64);
        if (lane >= o) upto += x;
    }
    if (lane == 63) part[wave] = upto;
    if (t == 0) found = NT;
    __syncthreads();
    for (int w = 0; w < wave; ++w) before += part[w];
    const uint64_t over = __ballot(before + upto > goal && sum > 0), some = __ballot(sum > 0);
    if (lane == 0 && over) atomicMin(&found, 64 * wave + __builtin_ctzll(over));
    __syncthreads();
    if (found == NT) {      // none: the last with a weight
        __syncthreads();
        if (t == 0) found = -1;
        __syncthreads();
        if (lane == 0 && some) atomicMax(&found, 64 * wave + 63 - __builtin_clzll(some));
        __syncthreads();
    }
    const int who = found;
    __syncthreads();
    if (t == who) {
        double run = before + (upto - sum);
        int token = -1;
        for (int64_t k = k0; k < k1; ++k) {
            const double w = r.one(k);
            run += w;
            if (w > 0) token = (int)k;
            if (w > 0 && run > goal) break;
        }
        found = token;
    }
    __syncthreads();
    return found;
}

template <typename T, bool DRAWN>
__global__ __launch_bounds__(NT) void verify_kernel(VerifyArgs a) {
    __shared__ int par[NODES], tok[NODES], line[NODES], ex[NODES];
    __shared__ float pu[NODES], pp[NODES], qq[NODES];
    __shared__ double seg[NW], part[NW];
    __shared__ int found;
    const int t = threadIdx.x, lane = t & 63, b = blockIdx.x;
    auto clamp = [&](int o) { return std::min<int64_t>(std::max(o, 0), a.d.rows); };
    const int64_t off = clamp(a.d.offsets[b]), rows = clamp(a.d.offsets[b + 1]) - off;
    if (rows <= 0 || rows > NODES) {
        for (int64_t i = t; i < rows; i += NT) a.path[off + i] = -1;
        if (t == 0) {
            a.counts[b] = 0;
            a.next[b] = -1;
        }
        return;
    }
    const int n = (int)rows, words = (n + 63) / 64;
    const T* P = (const T*)a.P + off * a.ldp;
    const T* Q = DRAWN ? (const T*)a.Q + off * a.ldq : nullptr;
    for (int i = t; i < n; i += NT) {
        const int p = a.d.parents[off + i], x = a.d.tokens[off + i];
        const bool ok = i > 0 && p >= 0 && p < i && (unsigned)x < (unsigned)a.vocab;      // others are passed over
        par[i] = ok ? p : -1;
        tok[i] = x;
        pu[i] = a.d.u[off + i];
        pp[i] = ok ? load_as_float(P + p * a.ldp, x) : 0.f;
        if constexpr (DRAWN) qq[i] = ok ? load_as_float(Q + p * a.ldq, x) : 0.f;
    }
    __syncthreads();

    // shares of whole chunks of a wave
    const int step = 64 * Chunk<T>::N;
    const int share = (int)std::min<int64_t>(cdiv(cdiv((int64_t)a.vocab, NW), step) * step, INT32_MAX);
    Rest<T, DRAWN> r{P, Q, 0., ex, 0};
    double z = 1., total = -1.;      // total: sum of what is left, -1 before it is known
    int cur = 0, count = 1;
    if (t == 0) line[0] = 0;
    for (bool moved = true; moved;) {
        moved = false;
        for (int w = cur / 64; w < words && !moved; ++w) {
            const int mine = 64 * w + lane;
            const bool child = mine < n && par[mine] == cur;
            uint64_t mask = __ballot(child);
            while (mask && !moved) {
                const int i = 64 * w + __builtin_ctzll(mask);
                mask &= mask - 1;
                double left;
                if constexpr (DRAWN) {
                    left = r.weight(pp[i], qq[i]);
                } else {
                    left = r.weight(pp[i], 0.f);
                    for (int j = cur + 1; j < i; ++j)      // the same token has been tried
                        if (par[j] == cur && tok[j] == tok[i]) left = 0.;
                }
                const double q = DRAWN ? (double)qq[i] : 1.;
                if ((double)pu[i] * z * q < left) {
                    cur = i;
                    if (t == 0) line[count] = i;
                    ++count;
                    r.p = P + (int64_t)cur * a.ldp;
                    if constexpr (DRAWN) r.q = Q + (int64_t)cur * a.ldq;
                    r.c = 0.;
                    z = 1.;
                    total = -1.;
                    moved = true;
                } else if constexpr (DRAWN) {
                    r.c += z;
                    z = total = sum_rest(r, a.vocab, share, seg);
                } else {
                    z -= left;
                }
            }
        }
    }
    if constexpr (!DRAWN) {      // the children that were tried
        for (int w = cur / 64; w < words; ++w) {
            const int mine = 64 * w + lane;
            const bool child = mine < n && par[mine] == cur;
            const uint64_t mask = __ballot(child);
            if (child && t < 64) ex[r.nex + __builtin_popcountll(mask & ((1ull << lane) - 1))] = tok[mine];
            r.nex += __builtin_popcountll(mask);
        }
        __syncthreads();
    }
    if (total == -1.) total = sum_rest(r, a.vocab, share, seg);
    if (total == 0.) {      // nothing is left: p itself
        r.c = 0.;
        r.nex = 0;
        total = sum_rest(r, a.vocab, share, seg);
    }
    int token = -1;
    if (total > 0. && total < INFINITY) token = draw_rest(r, a.vocab, share, seg, (double)a.d.r[b] * total, part, found);
    __syncthreads();
    for (int i = t; i < n; i += NT) a.path[off + i] = i < count ? line[i] : -1;
    if (t == 0) {
        a.counts[b] = count;
        a.next[b] = token;
    }
}

template <typename T>
int launch(const VerifyArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)a.d.batch);
    if (a.Q)
        hipLaunchKernelGGL((verify_kernel<T, true>), grid, dim3(NT), 0, st, a);
    else
        hipLaunchKernelGGL((verify_kernel<T, false>), grid, dim3(NT), 0, st, a);
    PTQ_LAUNCH_CHECK();
    return PTQ_OK;
}

}  // namespace

int launch_verify_drafts(const void* P, int64_t ldp, const void* Q, int64_t ldq, int dtype, int64_t vocab,
                         const Drafts& d, int32_t* path, int32_t* counts, int32_t* next, hipStream_t st) {
    if (d.batch == 0) return PTQ_OK;
    const VerifyArgs a{P, ldp, Q, ldq, (int)vocab, d, path, counts, next};
    return dtype == PTQ_F32 ? launch<float>(a, st) : launch<uint16_t>(a, st);
}

}  // namespace ptq
