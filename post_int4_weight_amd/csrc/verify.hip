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
// One workgroup a sequence walks. What every node's test needs of p and q is
// fetched at once; the walk is then the same code on the same values in every
// wave. What bounds it: for small vocabularies the chain of loads (offsets, nodes,
// their probabilities, the rows: 9.6 us for one sequence and 32000 tokens), for
// large ones what one CU can load, 9 us for two rows of 128256 in fp32 (108 GB/s).
// So there other workgroups help with the sums, see Help: 48 trees over 128256
// tokens, fp32: 28 us, 43 without.
#include "int8.hpp"

namespace ptq {
namespace {

constexpr int NT = 1024, NW = NT / 64;
constexpr int NODES = TREE_NODES;
constexpr int MAX_SHARES = VERIFY_SHARES;
static_assert(MAX_SHARES * NW <= 64, "sums of a wave's segments: one a lane");

// How the workgroups of a sequence share a sum. Its walker posts a job (the row,
// and what is taken from it) under a new number and every workgroup, the walker
// too, claims shares of it until none is left; the walker then waits for the
// shares that were claimed. So it waits for workgroups alone that are running and
// wait for nothing themselves, and needs no other: a helper that never runs, or
// runs late, or has given up (POLLS looks without a new job) claims nothing.
// Shares are summed in their order, whoever took them.
//
// Everything here is read and written by relaxed atomics of the device, which pass
// the caches by. Acquiring and releasing would empty the L2 at every look: 207 us
// where it takes 71 (48 sequences by four).
struct Help {
    unsigned long long ticket;     // number of the job << 32 | shares claimed
    int node, without;             // the job: the row, whether tried tokens are left out, and c
    double c;
    double seg[MAX_SHARES * NW];   // sums, or NOT_YET
};
constexpr unsigned long long NOT_YET = 0x7ff4deadbeef0001ull;      // a NaN that no sum is: it signals
constexpr unsigned OVER = 0xffffffffu;      // number after the last job
constexpr int POLLS = 256;                  // at about 1 us each

template <typename V>
__device__ __forceinline__ V peek(const V* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
template <typename V>
__device__ __forceinline__ void put(V* p, V x) { __hip_atomic_store(p, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
// what this wave has put is there for all
__device__ __forceinline__ void wait_put() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}
__device__ __forceinline__ unsigned long long claim_share(Help* h) {
    return __hip_atomic_fetch_add(&h->ticket, 1ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

struct VerifyArgs {
    const void* P; int64_t ldp;
    const void* Q; int64_t ldq;
    int vocab;
    Drafts d;
    int32_t* path; int32_t* counts; int32_t* next;
    int shares;          // workgroups of a sequence
    Help* help;          // of each sequence, with more than one
};

// 16 bytes of a row that need not be aligned (vocabularies of odd sizes)
template <typename T>
struct Chunk {
    static constexpr int N = 16 / sizeof(T);
    T x[N];
    __device__ __forceinline__ void load(const T* p) { __builtin_memcpy(x, p, 16); }
    // the first `left` elements, zeros past them
    __device__ __forceinline__ void load(const T* p, int64_t left) {
#pragma unroll
        for (int k = 0; k < N; ++k) x[k] = k < left ? p[k] : (T)0;
    }
    __device__ __forceinline__ float at(int k) const { return load_as_float(x, k); }
};

// x of the lane that a DPP control names, 0 where there is none or the row is not in ROWS
template <int CONTROL, int ROWS>
__device__ __forceinline__ double from_lane(double x) {
    const long long v = __double_as_longlong(x);
    const int lo = __builtin_amdgcn_update_dpp(0, (int)v, CONTROL, ROWS, 0xf, false);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(v >> 32), CONTROL, ROWS, 0xf, false);
    return __longlong_as_double((long long)hi << 32 | (unsigned)lo);
}
// Sums of the lanes up to each: within rows of 16, then over the rows before. (By shuffles through LDS the kernel's five
// sums and scans took 2 us of one sequence's 11.)
__device__ __forceinline__ double scan_wave(double x) {
    x += from_lane<0x111, 0xf>(x);      // row_shr 1, 2, 4, 8
    x += from_lane<0x112, 0xf>(x);
    x += from_lane<0x114, 0xf>(x);
    x += from_lane<0x118, 0xf>(x);
    x += from_lane<0x142, 0xa>(x);      // row_bcast 15: into the second and the fourth row
    x += from_lane<0x143, 0xc>(x);      // row_bcast 31: into the upper two
    return x;
}
// x of one lane for all
__device__ __forceinline__ double of_lane(double x, int lane) {
    const long long v = __double_as_longlong(x);
    const int lo = __builtin_amdgcn_readlane((int)v, lane), hi = __builtin_amdgcn_readlane((int)(v >> 32), lane);
    return __longlong_as_double((long long)hi << 32 | (unsigned)lo);
}
__device__ __forceinline__ double sum_wave(double x) { return of_lane(scan_wave(x), 63); }

// What is left of p: r = max(p - c q, 0), or p without the tokens ex[0 .. nex)
template <typename T, bool DRAWN>
struct Rest {
    const T* p; const T* q;
    double c;
    const int* ex;
    int nex;

    static __device__ __forceinline__ double weight(float pv, float qv, double c) {
        const double w = (double)pv - c * (double)qv;
        return w < 0 ? 0. : w;      // a NaN stays one
    }
    // weights of the 8 tokens from k on; zeros from `end` on
    __device__ __forceinline__ void eight(int64_t k, int64_t end, double (&w)[8]) const {
        float pv[8], qv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            pv[e] = k + e < end ? load_as_float(p, k + e) : 0.f;
            qv[e] = DRAWN && c != 0. && k + e < end ? load_as_float(q, k + e) : 0.f;
        }
        for (int j = 0; j < nex; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (ex[j] == k + e) pv[e] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = weight(pv[e], qv[e], c);
    }
};

// This wave's sum of the weights of tokens lo .. hi; q counts where COVERED
template <typename T, bool COVERED, typename R>
__device__ __forceinline__ double sum_part(const R& r, int64_t lo, int64_t hi) {
    constexpr int N = Chunk<T>::N, STEP = 64 * N, U = 4;
    const int lane = threadIdx.x & 63;
    double s[U] = {};
    // leaves out the tried tokens among the wave's `count` chunks
    auto leave = [&](Chunk<T>* p, int count, int64_t at) __attribute__((always_inline)) {
        const int64_t first = at - lane * N;
        for (int j = 0; j < r.nex; j += 64) {
            const int mine = j + lane < r.nex ? r.ex[j + lane] : -1;      // each once: one in 64 lanes takes 64 rounds below
            uint64_t mask = __ballot(mine >= first && mine < first + count * STEP);
            while (mask) {
                const int64_t k = __builtin_amdgcn_readlane(mine, __builtin_ctzll(mask)) - at;
                mask &= mask - 1;
#pragma unroll
                for (int u = 0; u < count; ++u)
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        if (k == u * STEP + e) p[u].x[e] = 0;
            }
        }
    };
    auto add = [&](const Chunk<T>& p, const Chunk<T>& q, double& to) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < N; ++k) to += R::weight(p.at(k), COVERED ? q.at(k) : 0.f, COVERED ? r.c : 0.);
    };
    int64_t k0 = lo + lane * N;
    for (; k0 - lane * N + STEP * U <= hi; k0 += STEP * U) {
        Chunk<T> p[U], q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            p[u].load(r.p + k0 + u * STEP);
            if constexpr (COVERED) q[u].load(r.q + k0 + u * STEP);
        }
        leave(p, U, k0);
#pragma unroll
        for (int u = 0; u < U; ++u) add(p[u], q[u], s[u]);
    }
    for (; k0 - lane * N < hi; k0 += STEP) {
        Chunk<T> p, q;
        if (k0 + N <= hi) {
            p.load(r.p + k0);
            if constexpr (COVERED) q.load(r.q + k0);
        } else {
            p.load(r.p + k0, hi - k0);
            if constexpr (COVERED) q.load(r.q + k0, hi - k0);
        }
        leave(&p, 1, k0);
        add(p, q, s[0]);
    }
    return sum_wave((s[0] + s[1]) + (s[2] + s[3]));
}

// Segment `i` of the vocabulary: a wave's part of a share
struct Segments {
    int vocab, each, count;
    __device__ __forceinline__ int64_t from(int i) const { return std::min<int64_t>((int64_t)i * each, vocab); }
};

// Sums a wave's segment of a share, for the walker to add up
template <typename T, bool DRAWN>
__device__ __forceinline__ void sum_share(const Rest<T, DRAWN>& r, const Segments& g, Help* h, int share, double* seg) {
    const int lane = threadIdx.x & 63, i = share * NW + (threadIdx.x >> 6);
    // a row that nothing is taken from yet is read alone
    const double sum = DRAWN && r.c != 0. ? sum_part<T, DRAWN>(r, g.from(i), g.from(i + 1))
                                          : sum_part<T, false>(r, g.from(i), g.from(i + 1));
    if (lane != 0) return;
    if (h) {
        put(&h->seg[i], sum);
    } else {
        seg[i] = sum;
    }
}

// Sums of all segments, into seg; the whole sum comes back.
template <typename T, bool DRAWN>
__device__ double sum_rest(const Rest<T, DRAWN>& r, const Segments& g, double (&seg)[MAX_SHARES * NW], Help* h,
                           unsigned& job, int node, int& claim) {
    const int t = threadIdx.x;
    __syncthreads();      // seg of the sum before has been read
    if (h) {
        ++job;
        if (t < g.count) put((unsigned long long*)&h->seg[t], NOT_YET);
        if (t == 0) {
            put(&h->node, node);
            put(&h->c, r.c);
            put(&h->without, (int)(r.nex > 0));
        }
        wait_put();
        __syncthreads();
        if (t == 0) put(&h->ticket, (unsigned long long)job << 32 | 1);
    }
    for (int share = 0; share < g.count / NW;) {
        sum_share(r, g, h, share, seg);
        if (!h) break;
        __syncthreads();      // claim has been read
        if (t == 0) claim = (int)(unsigned)claim_share(h);
        __syncthreads();
        share = claim;
    }
    if (h && t < g.count) {
        unsigned long long x;
        while ((x = peek((const unsigned long long*)&h->seg[t])) == NOT_YET) __builtin_amdgcn_s_sleep(1);
        seg[t] = __longlong_as_double((long long)x);
    }
    __syncthreads();
    const int lane = t & 63;
    return sum_wave(lane < g.count ? seg[lane] : 0.);
}

// First token whose running sum exceeds goal; the last one with a weight where rounding leaves none.
template <typename T, bool DRAWN>
__device__ int draw_rest(const Rest<T, DRAWN>& r, const Segments& g, const double (&seg)[MAX_SHARES * NW], double goal,
                         double (&part)[NW], int& found) {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const double mine = lane < g.count ? seg[lane] : 0., to = scan_wave(mine);
    const uint64_t past = __ballot(mine > 0 && to > goal), any = __ballot(mine > 0);
    const int at = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(any | 1);
    double before = of_lane(to - mine, at);
    // the segment again, each thread its own stretch
    const int64_t lo = g.from(at), hi = g.from(at + 1);
    const int64_t each = cdiv(hi - lo, NT), k0 = std::min(lo + t * each, hi), k1 = std::min(k0 + each, hi);
    double sum = 0, w[8];
    for (int64_t k = k0; k < k1; k += 8) {
        r.eight(k, k1, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += w[e];
    }
    const double upto = scan_wave(sum);
    if (lane == 63) part[wave] = upto;
    if (t == 0) found = NT;
    __syncthreads();
    before += sum_wave(lane < wave ? part[lane] : 0.);
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
        for (int64_t k = k0; k < k1 && (token < 0 || run <= goal); k += 8) {
            r.eight(k, k1, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (!(w[e] > 0) || (token >= 0 && run > goal)) continue;
                run += w[e];
                token = (int)k + e;
            }
        }
        found = token;
    }
    __syncthreads();
    return found;
}

// Tokens of the children of `node` (DRAWN = false: they have been tried)
__device__ __forceinline__ int tried_tokens(const int* par, const int* tok, int n, int node, int* ex) {
    const int lane = threadIdx.x & 63;
    int count = 0;
    for (int w = node / 64; w < (n + 63) / 64; ++w) {
        const int i = 64 * w + lane;
        const bool child = i < n && par[i] == node;
        const uint64_t mask = __ballot(child);
        if (child && threadIdx.x < 64) ex[count + __builtin_popcountll(mask & ((1ull << lane) - 1))] = tok[i];
        count += __builtin_popcountll(mask);
    }
    __syncthreads();
    return count;
}

template <typename T, bool DRAWN>
__global__ __launch_bounds__(NT) void verify_kernel(VerifyArgs a) {
    __shared__ int par[NODES], tok[NODES], line[NODES], ex[NODES];
    __shared__ float pu[NODES], pp[NODES], qq[NODES];
    __shared__ double seg[MAX_SHARES * NW], part[NW];
    __shared__ int found, claim;
    __shared__ unsigned number;
    // walkers come first
    const int t = threadIdx.x, lane = t & 63, batch = (int)a.d.batch, b = (int)(blockIdx.x % (unsigned)batch);
    const bool walker = blockIdx.x < (unsigned)batch;
    Help* const h = a.shares > 1 ? a.help + b : nullptr;
    auto over = [&] {
        if (h && t == 0) put(&h->ticket, (unsigned long long)OVER << 32);
    };
    auto clamp = [&](int o) { return std::min<int64_t>(std::max(o, 0), a.d.rows); };
    const int64_t off = clamp(a.d.offsets[b]), rows = clamp(a.d.offsets[b + 1]) - off;
    if (rows <= 0 || rows > NODES) {
        if (!walker) return;
        over();
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
        if (!walker) continue;
        pu[i] = a.d.u[off + i];
        pp[i] = ok ? load_as_float(P + p * a.ldp, x) : 0.f;
        if constexpr (DRAWN) qq[i] = ok ? load_as_float(Q + p * a.ldq, x) : 0.f;
    }
    __syncthreads();

    // segments of whole steps of a wave
    const int step = 64 * Chunk<T>::N, count_seg = a.shares * NW;
    const Segments g{a.vocab, (int)std::min<int64_t>(cdiv(cdiv((int64_t)a.vocab, count_seg), step) * step, INT32_MAX), count_seg};
    Rest<T, DRAWN> r{P, Q, 0., ex, 0};
    if (!walker) {
        unsigned seen = 0;
        for (bool look = true;;) {
            if (t == 0) {
                int polls = 0;
                if (look)
                    while (polls < POLLS && (unsigned)(peek(&h->ticket) >> 32) == seen) {
                        ++polls;
                        __builtin_amdgcn_s_sleep(8);
                    }
                number = OVER;
                if (polls < POLLS) {
                    const unsigned long long x = claim_share(h);
                    number = (unsigned)(x >> 32);
                    claim = (int)(unsigned)x;
                }
            }
            __syncthreads();
            if (number == OVER) return;
            seen = number;
            look = claim >= a.shares;
            if (!look) {      // the job stays as it is while a share of it is being summed
                const int node = std::min(std::max(peek(&h->node), 0), n - 1);
                r.p = P + (int64_t)node * a.ldp;
                if constexpr (DRAWN) r.q = Q + (int64_t)node * a.ldq;
                r.c = peek(&h->c);
                r.nex = 0;
                if constexpr (!DRAWN)
                    if (peek(&h->without)) r.nex = tried_tokens(par, tok, n, node, ex);
                sum_share(r, g, h, claim, seg);
            }
            __syncthreads();      // number and claim have been read
        }
    }
    double z = 1., total = -1.;      // total: sum of what is left, -1 before it is known
    int cur = 0, count = 1;
    unsigned job = 0;
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
                    left = r.c != 0. ? r.weight(pp[i], qq[i], r.c) : r.weight(pp[i], 0.f, 0.);
                } else {
                    left = r.weight(pp[i], 0.f, 0.);
                    for (int v = cur / 64; v <= w; ++v) {      // the same token has been tried
                        const int j = 64 * v + lane;
                        if (__any(j < i && par[j] == cur && tok[j] == tok[i])) left = 0.;
                    }
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
                    z = total = sum_rest(r, g, seg, h, job, cur, claim);
                } else {
                    z -= left;
                }
            }
        }
    }
    if constexpr (!DRAWN) r.nex = tried_tokens(par, tok, n, cur, ex);
    for (bool whole = false; total <= 0. && !whole;) {
        if (total == 0.) {      // nothing is left: p itself
            r.c = 0.;
            r.nex = 0;
            whole = true;
        }
        total = sum_rest(r, g, seg, h, job, cur, claim);
    }
    over();
    int token = -1;
    if (total > 0. && total < INFINITY) token = draw_rest(r, g, seg, (double)a.d.r[b] * total, part, found);
    __syncthreads();
    for (int i = t; i < n; i += NT) a.path[off + i] = i < count ? line[i] : -1;
    if (t == 0) {
        a.counts[b] = count;
        a.next[b] = token;
    }
}

__global__ void clear_help_kernel(Help* h, int batch) {
    const int b = blockIdx.x * 64 + threadIdx.x;
    if (b < batch) h[b].ticket = 0;
}

template <typename T>
int launch(const VerifyArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)(a.d.batch * a.shares));
    if (a.Q)
        hipLaunchKernelGGL((verify_kernel<T, true>), grid, dim3(NT), 0, st, a);
    else
        hipLaunchKernelGGL((verify_kernel<T, false>), grid, dim3(NT), 0, st, a);
    PTQ_LAUNCH_CHECK();
    return PTQ_OK;
}

}  // namespace

// Workgroups of a sequence. Four, or as many as the CUs allow: 48 sequences of 6
// nodes, 128256 tokens, fp32, 3 children not kept: 73 us by one, 59 by two, 51 by
// four, 53 by five; 128 sequences 71 and 69 by two. Clearing what they share and
// meeting cost more than that below about 10^5 tokens. 48 sequences, one child not
// kept, by one and by four: 65536 tokens 15 and 17 us, 80000 16 and 17, 100003 20
// and 17, 128256 27 and 19, 152064 28 and 21; by two, 128 sequences: 25 and 27,
// 33 and 31, 35 and 34 of the last three. Chosen drafts, which need one pass: 13
// and 17 at 100003, 17 and 16 at 128256.
int verify_drafts_shares(int64_t batch, int64_t vocab) {
    if (vocab < 98304 || batch < 1) return 1;
    return (int)std::max<int64_t>(1, std::min<int64_t>(MAX_SHARES, 256 / batch));
}

size_t verify_drafts_help_bytes(int64_t batch, int shares) { return shares > 1 ? (size_t)batch * sizeof(Help) : 0; }

int launch_verify_drafts(const void* P, int64_t ldp, const void* Q, int64_t ldq, int dtype, int64_t vocab,
                         const Drafts& d, int shares, int32_t* path, int32_t* counts, int32_t* next, void* workspace,
                         hipStream_t st) {
    if (d.batch == 0) return PTQ_OK;
    const VerifyArgs a{P, ldp, Q, ldq, (int)vocab, d, path, counts, next, shares, (Help*)workspace};
    if (shares > 1) {
        hipLaunchKernelGGL(clear_help_kernel, dim3((unsigned)cdiv(d.batch, 64)), dim3(64), 0, st, a.help, (int)d.batch);
        PTQ_LAUNCH_CHECK();
    }
    return dtype == PTQ_F32 ? launch<float>(a, st) : launch<uint16_t>(a, st);
}

}  // namespace ptq
