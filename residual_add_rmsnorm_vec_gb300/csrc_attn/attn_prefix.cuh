// Attention of a group's queries over the tokens that the group shares: the parts
// that attn_attend.cuh's kernels add to each sequence's own tokens.
//
//   s_j = scale q . k_j,  l = sum exp(s_j - m),  O = sum exp(s_j - m) v_j
//
// A row is one column of the group (sequence x query token x head of a key head).
// All of a group's rows meet the same keys and values, so the products are matrix
// products: 4 D flops for each pair of a row and a token against 2 D + 1/2 bytes a
// token.  From about 150 rows on the tensor cores bound it, below that DRAM.
//
// Measured (this launch alone), 32 / 8 heads x 128: 64 sequences x 8192 shared tokens 24 us, of which 7 are a
// block's start (TMEM, barriers, plan, queries, first pages); 256 x 16384 85 us, 808 TFLOP/s
// (0.42 of the library's matrix product).  A step of 64 tokens and 256 rows takes 2000 cycles.
// What bounds it there: a product of 128 rows and 16 of the inner dimension takes 65
// cycles with 64 columns as with 128, for its A operand comes from shared memory, so S = Q
// K^T runs at half its rate, and shared memory carries the codes, their widened copies and
// Q beside it.  Steps of 128 tokens, whose scores fill TMEM once, took 104 us: products and
// softmax in turn.
//
// A block holds R tiles of 128 rows (R = 2 where a group has more than 128 rows)
// and walks over its share of the line of all steps, 64 tokens of an item (group x key
// head x R tiles) each.  Its warps have fixed parts:
//
//   plan     one warp: pages, scales, what a step is (32 blocks of 16 tokens at a time,
//            so that their loads' latencies are met once), some steps ahead of the rest
//   K, V     four warps each: asynchronous copies of the codes into slots, from there
//            widened to fp16 into the swizzled stages of the B operands
//   MMA      two threads: one issues S = Q K^T, a step ahead, the other O += P V
//   softmax  four warps to a row tile, a thread to a row: scores from TMEM, weights
//            back into TMEM as the second product's A operand, in fp16
//
// * S has two buffers (the weights go over the scores that they are made of), so the
//   products of the next scores do not wait for this step's softmax.
// * Widening 16-bit copies into shared memory pays here, other than in attn_attend.cuh:
//   256 rows use each copy.
// * A value's scale is 2^e times a significand in [1, 2).  The significand multiplies
//   the weight before that is rounded to fp16 (the one rounding of the weight: half a
//   step, 2^-11), 2^e the codes: code * 2^(7 + e - E) is exact in fp16 for e in
//   [E - 22, E].  E is the block's reference; a block of tokens outside its window makes
//   a step of its own, for which what was summed so far is added to the part in memory
//   and E set anew.  Scales that lie 2^22 apart are rare, so that path is small.
// * A row's reference m follows its maximum only when that has grown by more than
//   2^kSlack; then the row's sum is multiplied in TMEM by the softmax warp itself, behind
//   the product before.  Weights are lifted by kLift: a lifted weight times a significand
//   stays below 2^15 + 2^12, and fp16's subnormals end 2^-34 below the reference.
// * Parts go to the workspace in the order of the line: nothing depends on timing.
// * Every wait gives up after a second (or the limit that a test sets): the block then
//   stops, waits for its products and copies in flight, gives TMEM back, and bit 0 of the
//   status word is set.
// * Code is kept small (loops over a tile's pieces are rolled): most calls run a few
//   steps a block, and each instruction that runs once is fetched from L2 first.
#pragma once

#include "attn_common.cuh"

namespace rmsattn {
namespace prefix {

using rmsn::F2;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -3.402823466e38f;  // the reference before any token is seen
constexpr float kSlack = 5.f;
constexpr int kLiftLog = 9;
constexpr float kLift = 512.f;
constexpr float kWide = 4194304.f;  // 2^22: up to it, a product's rounding error is 2^-3 at most

// flags of a step
constexpr uint32_t kFirst = 1u, kLast = 2u, kFlush = 4u, kEnd = 8u, kTwo = 16u;

template <int D_, int R_>
struct Shape {
    static constexpr int D = D_, R = R_;
    static constexpr int TOK = 64, BLK = TOK / kBlock;
    static constexpr int PARTS = D / 64;      // 64-dim parts of 128-byte lines
    static constexpr int M = 8;               // slots of the steps' words
    static constexpr int kTile = TOK * D * 2; // a stage of K or V; there are two of each
    static constexpr int kQ = 128 * D * 2;
    static constexpr int kRaw = kTile;        // codes of a step of K and V
    static constexpr int N = D == 256 ? 1 : 4;  // slots of codes
    static constexpr int kSmem = R * kQ + 4 * kTile + N * kRaw + 1024;
    static constexpr int kWarps = 4 * R + 12;  // softmax; K; V; products, plan and an idle one
    // four warps to a role: registers move between them at the begin (of the 480 or 512
    // that four threads have, one of each role)
    static constexpr int kRegsS = R == 2 ? 136 : 200, kRegsW = R == 2 ? 64 : 96, kRegsM = R == 2 ? 80 : 104;
    static constexpr int kCols = 512;         // of TMEM: S at 64 (2 x + buffer), O behind
    static constexpr int kO = 256;
    static constexpr int ITERS = TOK / 8 * PARTS / 4;  // 16-byte pieces of a thread, K or V
};

// What the plan says of a step.
struct Step {
    int64_t off[4];    // the blocks' codes, in bytes from the cache's begin; -1: none
    float ks[4];       // K scales
    float vm[4];       // significands of the V scales, lifted
    uint32_t f[4];     // 2^(7 + e - E), packed fp16
    uint32_t mask;     // blocks of this step
    uint32_t flags;
    int32_t e;         // E
};

// ---------------------------------------------------------------- instructions

__device__ __forceinline__ uint32_t smem_of(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float exp2a(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Shared-memory operand: rows of 128 bytes, 128-byte swizzle, eight rows to 1024
// bytes; `lead`: bytes between 64-element parts of an operand whose rows are the
// product's inner dimension.  The low word has the place; the high one is the same
// for all.
__device__ __forceinline__ uint32_t operand(uint32_t addr, uint32_t lead) {
    return (addr & 0x3FFFF) >> 4 | (lead >> 4) << 16;
}
constexpr uint32_t kOperandHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
// fp16 operands, fp32 sums, 128 rows, n columns; `inner`: B's rows are the inner dimension.
__host__ __device__ constexpr uint32_t product(int n, bool inner) {
    return 1u << 4 | (inner ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24;
}
// The k-th of a chain of products; the first one of a chain sets the sums, with FRESH.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, int k) {
    if (k == 0)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, 0, 0;\n\tmov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(kOperandHigh), "r"(idesc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.eq.b32 p, 0, 0;\n\tmov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(kOperandHigh), "r"(idesc)
            : "memory");
}
template <bool FRESH>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, int k) {
    if (FRESH && k == 0)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, 0, 0;\n\tmov.b64 db, {%2, %3};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(kOperandHigh), "r"(idesc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.eq.b32 p, 0, 0;\n\tmov.b64 db, {%2, %3};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(kOperandHigh), "r"(idesc)
            : "memory");
}
// 32 columns of the warp's 32 rows, on their way: the registers hold them behind
// tmem_loaded(), which names them so that nothing reads them before.
__device__ __forceinline__ void tmem_begin(float* v, uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tmem_begin16(float* v, uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tmem_named(float* v) {  // 16 registers
    asm volatile(""
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                   "+f"(v[15])
                 :
                 : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_loaded(float (&v)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; i += 16) tmem_named(v + i);
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------- the block

struct Bars {
    uint64_t step[8], step_free[8], k_full[2], v_full[2], s_full[2][2], p_full[2][2], pv[2], q_full[2], last[2];
    uint32_t tmem, stop;
};

// All of a warp's lanes wait together, for `limit` cycles at most; false: the block stops.
__device__ __forceinline__ bool wait(const uint64_t* bar, int phase, uint32_t* stop, long long limit) {
    const uint32_t b = smem_of(bar);
    bool ok = rmsn::mbar_try_wait(b, phase & 1);
    if (!__all_sync(0xFFFFFFFFu, ok)) {
        const long long t0 = clock64();
        while (!__all_sync(0xFFFFFFFFu, ok)) {
            if (!ok) ok = rmsn::mbar_try_wait(b, phase & 1);
            const bool out = *reinterpret_cast<volatile uint32_t*>(stop) != 0 || clock64() - t0 > limit;
            if (__any_sync(0xFFFFFFFFu, out && !ok)) {
                *reinterpret_cast<volatile uint32_t*>(stop) = 1;
                return false;
            }
        }
    }
    return true;
}
// The same for one thread.
__device__ __forceinline__ bool wait_alone(const uint64_t* bar, int phase, uint32_t* stop, long long limit) {
    const uint32_t b = smem_of(bar);
    if (rmsn::mbar_try_wait(b, phase & 1)) return true;
    const long long t0 = clock64();
    while (!rmsn::mbar_try_wait(b, phase & 1)) {
        if (*reinterpret_cast<volatile uint32_t*>(stop) != 0 || clock64() - t0 > limit) {
            *reinterpret_cast<volatile uint32_t*>(stop) = 1;
            return false;
        }
    }
    return true;
}

// A block's piece of an item: `steps` of its steps from `step0` on.
struct Piece {
    int hk, tile, step0, steps;
    PrefixGroup g;
};

// The pieces of a share, in the line's order.
struct Walk {
    int at, stop, g;
    __device__ __forceinline__ void begin(const PrefixArgs& a) {
        const int4 line = __ldcg(reinterpret_cast<const int4*>(a.line));  // total, chunk
        const int64_t from = (int64_t)blockIdx.x * line.y, to = from + line.y;
        at = (int)(from < line.x ? from : line.x);
        stop = (int)(to < line.x ? to : line.x);
        g = 0;
        if (at < stop) {  // the last group that begins at `at` or before; groups without steps begin where the next does
            int hi = a.n_groups;
            while (hi - g > 1) {
                const int mid = (g + hi) >> 1;
                if (__ldcg(&a.groups[mid].first) <= at) g = mid;
                else hi = mid;
            }
        }
    }
    __device__ __forceinline__ bool next(const PrefixArgs& a, Piece* p) {
        if (at >= stop) return false;
        for (;;) {
            const int4* from = reinterpret_cast<const int4*>(a.groups + g);
            const int4 u = __ldcg(from), v = __ldcg(from + 1);
            p->g = PrefixGroup{u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
            if (p->g.ns > 0 && at < p->g.first + p->g.ns * p->g.tiles * a.c.H) break;
            ++g;
        }
        const int item = (at - p->g.first) / p->g.ns;
        p->step0 = (at - p->g.first) - item * p->g.ns;
        const int left = p->g.ns - p->step0;
        p->steps = stop - at < left ? stop - at : left;
        p->hk = item / p->g.tiles;
        p->tile = item - p->hk * p->g.tiles;
        at += p->steps;
        return true;
    }
};

// A softmax warp's way through its share, in shared memory (its registers hold
// scores): lane 0 goes on, all read.
struct Way {
    Walk walk;
    Piece p;
    bool more;
    __device__ __forceinline__ void begin(const PrefixArgs& a, int lane) {
        if (lane == 0) {
            walk.begin(a);
            more = walk.next(a, &p);
        }
        __syncwarp();
    }
    __device__ __forceinline__ void next_piece(const PrefixArgs& a, int lane) {
        __syncwarp();
        if (lane == 0) more = walk.next(a, &p);
        __syncwarp();
    }
};

// The warp that plans the steps, 8 tiles of 4 blocks at a time: lane 4 i + b has block
// b of tile i.
template <class C>
__device__ __forceinline__ void plan(const PrefixArgs& a, Bars* bars, Step* steps) {
    const int lane = threadIdx.x & 31;
    Walk walk;
    Piece p;
    walk.begin(a);
    int n = 0;  // steps so far
    while (walk.next(a, &p)) {
        const bool two = C::R == 2 && (p.g.s1 - p.g.s0) * a.n * a.group - p.tile * (128 * C::R) > 128;
        const int32_t* row = a.table + p.g.seq * a.table_stride;
        bool begin = true;
        int E = 0;  // the piece's reference
        // the lane's block of the tiles from t0 on
        auto at = [&](int t0) { return (p.step0 + t0) * C::TOK + lane * kBlock; };
        auto in = [&](int t0) { return t0 + (lane >> 2) < p.steps && at(t0) < p.g.shared; };
        auto slot_of = [&](int j) { return (int)(((uint64_t)(uint32_t)(j >> 4) * a.page_rcp) >> 37); };
        int32_t ahead = in(0) ? __ldcg(row + slot_of(at(0))) : 0;
        for (int t0 = 0; t0 < p.steps; t0 += 8) {
            const int j = at(t0), slot = slot_of(j);
            const bool there = in(t0);
            const int32_t entry = ahead;
            // (on their way while these tiles are planned: 256 x 16384 165.4 us, not 166.8)
            ahead = in(t0 + 8) ? __ldcg(row + slot_of(at(t0 + 8))) : 0;
            const bool have = there && (uint32_t)entry < (uint32_t)a.c.n_pages;
            if (there && !have) atomicOr(a.status, kBadPage);
            // (a block that is not there reads page 0's scale, and is left out)
            const int64_t page = have ? entry : 0;
            const int64_t block = have ? (int64_t)p.hk * (a.c.page >> 4) + ((j - slot * a.c.page) >> 4) : 0;
            float ks = __ldcg(a.c.ks + page * a.c.scale_stride + block), vs = __ldcg(a.c.vs + page * a.c.scale_stride + block);
            if (!have) ks = vs = 0.f;
            const int64_t off = page * a.c.page_stride + block * (kBlock * C::D);
            const uint32_t valid = __ballot_sync(0xFFFFFFFFu, have);
            // the lane's value scale: 2^e vm, vm in [1, 2); 0 fits any reference
            uint32_t bits = __float_as_uint(vs) & 0x7FFFFFFFu;
            int e = -127;
            if (bits != 0 && bits < 0x00800000u) {  // below fp32's normal range
                bits = __float_as_uint(__uint_as_float(bits) * 16777216.f);
                e -= 24;
            }
            const bool zero = bits == 0;
            e += (int)(bits >> 23);
            const float vm = (zero ? 1.f : __uint_as_float((bits & 0x007FFFFFu) | 0x3F800000u)) * kLift;
            const int tiles = p.steps - t0 < 8 ? p.steps - t0 : 8;
            for (int i = 0; i < tiles; ++i) {
                uint32_t rem = valid & (15u << (4 * i));
                const bool last = t0 + i == p.steps - 1;
                do {
                    uint32_t flags = (begin ? kFirst : 0u) | (two ? kTwo : 0u);
                    auto fitting = [&]() {
                        return __ballot_sync(0xFFFFFFFFu, zero || (e <= E && e >= E - 22)) & rem;
                    };
                    uint32_t mask = fitting();
                    if (begin || (rem != 0 && mask == 0)) {
                        const int top = __reduce_max_sync(0xFFFFFFFFu, !zero && (rem >> lane & 1) ? e : -1000);
                        if (!begin) flags |= kFlush;
                        E = top == -1000 ? 0 : top + 3;
                        mask = fitting();
                    }
                    rem &= ~mask;
                    if (rem == 0 && last) flags |= kLast;
                    begin = false;
                    Step* w = steps + n % C::M;
                    if (n >= C::M && !wait(&bars->step_free[n % C::M], n / C::M - 1, &bars->stop, a.wait_cycles)) return;
                    if (lane >> 2 == i) {
                        const int b = lane & 3, k7 = 7 + e - E;
                        const bool on = mask >> lane & 1;
                        uint32_t f = zero || !on ? 0u : (k7 >= -14 ? (uint32_t)(k7 + 15) << 10 : 0x200u);
                        w->off[b] = have ? off : -1;
                        w->ks[b] = ks;
                        w->vm[b] = vm;
                        w->f[b] = f | f << 16;
                        if (b == 0) {
                            w->mask = mask >> (4 * i);
                            w->flags = flags;
                            w->e = E;
                        }
                    }
                    __syncwarp();
                    if (lane == 0) arrive(smem_of(&bars->step[n % C::M]));
                    ++n;
                } while (rem != 0);
            }
        }
    }
    // one more step's word: there are none left
    if (n >= C::M && !wait(&bars->step_free[n % C::M], n / C::M - 1, &bars->stop, a.wait_cycles)) return;
    if (lane == 0) {
        steps[n % C::M].flags = kEnd;
        arrive(smem_of(&bars->step[n % C::M]));
    }
}

// The four warps that fill the stages of K (V = false) or V.  A lane's pieces are 16
// codes of eight tokens' 64 dims, which it copies and widens itself, so that nobody else
// waits for its copies (a bulk copy's operands move to uniform registers lane by lane:
// 16 of them took 2000 cycles).  A quarter warp has two tokens whose numbers differ in
// bit 0, four chunks each, of different parts where a token has several: it meets all
// banks once, reading the codes and storing the halves.
template <class C, bool V>
__device__ __forceinline__ void widen(const PrefixArgs& a, unsigned char* stages, unsigned char* raw, Bars* bars,
                                      const Step* steps, int wp) {
    constexpr int D = C::D, N = C::N, kSlot = C::kRaw / 2;
    const int lane = threadIdx.x & 31;
    const int r8 = (lane >> 3) * 2 + ((lane >> 2) & 1), c4 = lane & 3, odd = C::PARTS > 1 ? r8 & 1 : 0;
    const int mine = r8 * D + odd * 64 + c4 * 16;
    const uint32_t stages_s = smem_of(stages), raw_s = smem_of(raw);
    const uint8_t* codes = V ? a.c.v : a.c.k;
    // unit u: tokens 8 (u / PARTS) on, part u % PARTS of them (^ odd)
    auto place = [&](int u) { return u / C::PARTS * (8 * D) + ((u % C::PARTS ^ odd) - odd) * 64 + mine; };
    bool ok = true, more = true;
    int fetched = 0;
    auto fetch = [&]() {  // the next step's codes into its slot
        if (more) {
            if (!(ok = wait(&bars->step[fetched % C::M], fetched / C::M, &bars->stop, a.wait_cycles))) return;
            const Step* w = steps + fetched % C::M;
            more = !(w->flags & kEnd);
            if (more) {
                const uint32_t dst = raw_s + fetched % N * kSlot;
#pragma unroll
                for (int i = 0; i < C::ITERS; ++i) {
                    const int u = i * 4 + wp, b = u / C::PARTS >> 1, at = place(u);
                    const int64_t off = w->off[b];
                    const int64_t from = (off < 0 ? 0 : off) + (at - b * (kBlock * D));
                    const int bytes = off < 0 ? 0 : 16;  // (0: zeros)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + at), "l"(codes + from),
                                 "r"(bytes)
                                 : "memory");
                }
                ++fetched;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int i = 0; i < N && ok; ++i) fetch();
    for (int n = 0; ok && n < fetched; ++n) {
        const Step* w = steps + n % C::M;
        const int st = n & 1;
        asm volatile("cp.async.wait_group %0;" ::"n"(N - 1) : "memory");
        // K's stage is free behind the scores of step n - 2, V's behind its sums
        if (n >= 2 && !(ok = wait(V ? &bars->pv[st] : &bars->s_full[C::R - 1][st], n / 2 - 1, &bars->stop, a.wait_cycles))) break;
        const uint32_t dst = stages_s + st * C::kTile, src = raw_s + n % N * kSlot;
#pragma unroll
        for (int i = 0; i < C::ITERS; ++i) {
            const int u = i * 4 + wp, tg = u / C::PARTS, h = u % C::PARTS ^ odd, r = tg * 8 + r8;
            uint32_t x[4], y[8];
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                         : "r"(src + place(u))
                         : "memory");
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                y[2 * k] = e4m3x2_to_f16x2(x[k]);
                y[2 * k + 1] = e4m3x2_to_f16x2(x[k] >> 16);
            }
            if constexpr (V) {
                const uint32_t f = w->f[tg >> 1];
#pragma unroll
                for (int k = 0; k < 8; ++k) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(y[k]) : "r"(f));
                if (!(w->mask >> (tg >> 1) & 1)) {  // not of this step (a NaN code times 0 is not 0)
#pragma unroll
                    for (int k = 0; k < 8; ++k) y[k] = 0u;
                }
            }
            const uint32_t line = dst + h * (C::TOK * 128) + r * 128;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(line + (((2 * c4 + k) ^ (r & 7)) << 4)),
                             "r"(y[4 * k]), "r"(y[4 * k + 1]), "r"(y[4 * k + 2]), "r"(y[4 * k + 3])
                             : "memory");
        }
        fence_async();
        __syncwarp();
        if (lane == 0) {
            arrive(smem_of(V ? &bars->v_full[st] : &bars->k_full[st]));
            arrive(smem_of(&bars->step_free[n % C::M]));
        }
        fetch();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // no copy outlives the block
}

// The two threads that issue the products, one the scores and one the sums.  The tensor
// cores take a product in 65 cycles and have about four of them queued; a wait costs 100
// cycles, a commit 60: with one thread, 1000 of a step's 3100 cycles were such gaps.
// Operands' places are worked out for each product (kept, they fill the registers).
template <class C, int X, bool FRESH>
__device__ __forceinline__ void product_pv(uint32_t v_op, int st) {
    v_op += st * (C::kTile >> 4);
#pragma unroll
    for (int k = 0; k < C::TOK / 16; ++k)
        mma_ts<FRESH>(C::kO + X * C::D, (2 * X + st) * 64 + k * 8, v_op + (k * 2048 >> 4), product(C::D, true), k);
}
template <class C, int X>
__device__ __forceinline__ void product_qk(uint32_t q_op, uint32_t k_op, int st) {
    k_op += st * (C::kTile >> 4);
#pragma unroll
    for (int k = 0; k < C::D / 16; ++k)
        mma_ss((2 * X + st) * 64, q_op + ((X * C::kQ + (k / 4) * (128 * 128) + (k % 4) * 32) >> 4),
               k_op + (((k / 4) * (C::TOK * 128) + (k % 4) * 32) >> 4), product(C::TOK, false), k);
}

// Nothing of the thread's is in flight when it leaves (the default limit, whatever the call's is).
__device__ __forceinline__ void settle(uint64_t* bar) {
    commit(smem_of(bar));
    const long long t0 = clock64();
    while (!rmsn::mbar_try_wait(smem_of(bar), 0) && clock64() - t0 < kWaitCycles) {
    }
}

template <class C>
__device__ __forceinline__ void scores(const PrefixArgs& a, unsigned char* smem, Bars* bars, const Step* steps) {
    uint32_t q_op = operand(smem_of(smem), 16), k_op = operand(smem_of(smem) + C::R * C::kQ, 16);
    uint32_t* stop = &bars->stop;
    int turn[2] = {0, 0};
    for (int n = 0;; ++n) {
        const int st = n & 1;
        asm volatile("" : "+r"(q_op), "+r"(k_op));
        if (!wait_alone(&bars->step[n % C::M], n / C::M, stop, a.wait_cycles)) break;
        const uint32_t flags = steps[n % C::M].flags;
        if (flags & kEnd) break;
        // the scores' place is free behind the sums of step n - 2
        if (n >= 2 && !wait_alone(&bars->pv[st], n / 2 - 1, stop, a.wait_cycles)) break;
        if (!wait_alone(&bars->k_full[st], n >> 1, stop, a.wait_cycles)) break;
        if (flags & kFirst) {
            if (!wait_alone(&bars->q_full[0], turn[0]++, stop, a.wait_cycles)) break;
            if (C::R == 2 && (flags & kTwo) && !wait_alone(&bars->q_full[1], turn[1]++, stop, a.wait_cycles)) break;
        }
        tc_after();
        product_qk<C, 0>(q_op, k_op, st);
        commit(smem_of(&bars->s_full[0][st]));
        if constexpr (C::R == 2) {  // (a row tile without rows keeps step with the other)
            if (flags & kTwo) product_qk<C, 1>(q_op, k_op, st);
            commit(smem_of(&bars->s_full[1][st]));
        }
    }
    settle(&bars->last[0]);
}

template <class C>
__device__ __forceinline__ void sums(const PrefixArgs& a, unsigned char* smem, Bars* bars, const Step* steps) {
    uint32_t v_op = operand(smem_of(smem) + C::R * C::kQ + 2 * C::kTile, C::TOK * 128);
    uint32_t* stop = &bars->stop;
    for (int n = 0;; ++n) {
        const int st = n & 1;
        asm volatile("" : "+r"(v_op));
        if (!wait_alone(&bars->step[n % C::M], n / C::M, stop, a.wait_cycles)) break;
        const uint32_t flags = steps[n % C::M].flags;
        if (flags & kEnd) break;
        arrive(smem_of(&bars->step_free[n % C::M]));
        const bool fresh = flags & (kFirst | kFlush);
        if (!wait_alone(&bars->v_full[st], n >> 1, stop, a.wait_cycles) || !wait_alone(&bars->p_full[0][st], n >> 1, stop, a.wait_cycles)) break;
        tc_after();
        if (fresh) product_pv<C, 0, true>(v_op, st);
        else product_pv<C, 0, false>(v_op, st);
        if constexpr (C::R == 2) {
            if (!wait_alone(&bars->p_full[1][st], n >> 1, stop, a.wait_cycles)) break;
            tc_after();
            if (flags & kTwo) {
                if (fresh) product_pv<C, 1, true>(v_op, st);
                else product_pv<C, 1, false>(v_op, st);
            }
        }
        commit(smem_of(&bars->pv[st]));
    }
    settle(&bars->last[1]);
}

// The four warps of row tile x.
template <class T, class C>
__device__ __forceinline__ void soften(const PrefixArgs& a, unsigned char* smem, Bars* bars, const Step* steps,
                                       Way* way, int x) {
    constexpr int D = C::D, ROWS = 128 * C::R;
    const int wp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, r = wp * 32 + lane;
    const uint32_t lanes = (uint32_t)(wp * 32) << 16;
    const uint32_t o_at = lanes + C::kO + x * D;
    unsigned char* q_rows = smem + x * C::kQ;
    way->begin(a, lane);
    int n = 0;  // steps of the block so far
    float q_scale = 0.f, q_next = 0.f;
    int valid = 0, valid_next = 0;  // rows of this tile
    // The piece's queries, scaled to fp16 by a power of two as in attn_attend.cuh: copied
    // as they are (a warp its own rows), and rounded in place, a thread a row.
    auto load_q = [&]() {
        const Piece& p = way->p;
        const int first = p.tile * ROWS + x * 128, cols = (p.g.s1 - p.g.s0) * a.n * a.group - first;
        valid_next = cols < 0 ? 0 : cols;
        if (valid_next == 0) return;  // (x == 1 alone: the products leave it out)
        // 16-byte chunk c of row i, swizzled
        auto chunk = [&](int i, int c) {
            return smem_of(q_rows) + (c >> 3) * (128 * 128) + i * 128 + (((c & 7) ^ (i & 7)) << 4);
        };
        constexpr int CH = D / 8;
#pragma unroll 4
        for (int k = 0; k < CH; ++k) {
            const int e = k * 32 + lane, i = wp * 32 + e / CH, c = e % CH;
            const bool on = i < valid_next;  // (rows of nothing: zeros, scores of 0)
            const int cc = on ? first + i : first, token = cc / a.group;
            const uint16_t* src = static_cast<const uint16_t*>(a.q) + ((int64_t)p.g.s0 * a.n + token) * a.q_stride +
                                  (int64_t)(p.hk * a.group + cc - token * a.group) * D + c * 8;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(chunk(i, c)), "l"(src), "r"(on ? 16 : 0)
                         : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        float m = 0.f;
#pragma unroll 2
        for (int c = 0; c < CH; ++c) {
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(chunk(r, c))
                         : "memory");
#pragma unroll
            for (int k = 0; k < 4; ++k)  // (a maximum leaves NaN out; its products find it)
                m = rmsn::absmax3(m, rmsn::lo2<T>(w[k]), rmsn::hi2<T>(w[k]));
        }
        int e = (int)(__float_as_uint(m) >> 23) - 127 - 7;
        e = e < -126 ? -126 : (e > 126 ? 126 : e);
        const float down =
            m > 3.402823466e38f ? __uint_as_float(0x7FFFFFFFu) : copysignf(pow2(-e), a.scale);
        q_next = pow2(e) * (fabsf(a.scale) * kLog2e);
#pragma unroll 2
        for (int c = 0; c < CH; ++c) {
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(chunk(r, c))
                         : "memory");
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = rmsn::pack_f16x2(rmsn::lo2<T>(w[k]) * down, rmsn::hi2<T>(w[k]) * down);
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(chunk(r, c)), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                         "r"(w[3])
                         : "memory");
        }
        fence_async();
        __syncwarp();
        if (lane == 0) arrive(smem_of(&bars->q_full[x]));
    };
    if (way->more) load_q();
    while (way->more) {
        q_scale = q_next;
        valid = valid_next;
        const bool busy = wp * 32 < valid;  // the warp has rows
        const uint32_t eight = blockIdx.x * (ROWS / 8) + x * 16 + (r >> 3) +
                               prefix_eight(way->p.g, a.n * a.group, way->p.hk, way->p.tile, ROWS);
        float* part = a.parts + (int64_t)eight * (8 * (D + 2)) + (r & 7) * 8;
        float ref = kNone, l = 0.f;
        float part_ref = 0.f;
        bool has_part = false;
        int E = 0;
        // what O holds goes to the part, in units of the reference
        auto drain = [&]() {
            const int up = E - 7 - kLiftLog, half = up >> 1;  // 2^up in two steps: it may lie outside fp32's range
            const float f0 = pow2(half), f1 = pow2(up - half);
            const float keep = has_part ? exp2a(part_ref - ref) : 0.f;
#pragma unroll 1
            for (int d = 0; d < D; d += 32) {
                float o[32];
                tmem_begin(o, o_at + d);
                tmem_loaded(o);
                if (r < valid) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {  // 32 bytes: a whole sector
                        float* y = part + (d / 8 + i / 8) * 64;
                        uint32_t u[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            o[i + k] *= f0;
                            o[i + k] *= f1;
                        }
                        if (has_part) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) o[i + k] += y[k] * keep;
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k) u[k] = __float_as_uint(o[i + k]);
                        rmsn::st_stream32(y, u);
                    }
                }
            }
            has_part = true;
            part_ref = ref;
        };
        uint32_t flags = 0;
        if (valid > 0 || x == 0) {
            do {
                const Step* w = steps + n % C::M;
                const uint32_t s_at = lanes + (2 * x + (n & 1)) * 64;
                if (!wait(&bars->step[n % C::M], n / C::M, &bars->stop, a.wait_cycles)) return;
                if (!wait(&bars->s_full[x][n & 1], n >> 1, &bars->stop, a.wait_cycles)) return;
                tc_after();
                flags = w->flags;
                if (busy) {
                    const uint32_t mask = w->mask;
                    if (flags & kFlush) {
                        if (!wait(&bars->pv[(n - 1) & 1], (n - 1) >> 1, &bars->stop, a.wait_cycles)) return;
                        tc_after();
                        drain();
                    }
                    E = w->e;
                    // a row's scores stay in its thread's registers
                    float s[C::TOK], kc[C::BLK];
#pragma unroll
                    for (int c = 0; c < C::TOK; c += 32) tmem_begin(s + c, s_at + c);
#pragma unroll
                    for (int b = 0; b < C::BLK; ++b) kc[b] = w->ks[b] * q_scale;  // not negative
                    tmem_loaded(s);
                    float top = -INFINITY;
#pragma unroll
                    for (int b = 0; b < C::BLK; ++b) {
                        float m0 = s[16 * b], m1 = s[16 * b + 1];
#pragma unroll
                        for (int i = 2; i < 16; i += 4) {
                            m0 = max3(m0, s[16 * b + i], s[16 * b + i + 1]);
                            if (i + 3 < 16) m1 = max3(m1, s[16 * b + i + 2], s[16 * b + i + 3]);
                        }
                        const float m = __fmul_rn(fmaxf(m0, m1), kc[b]);
                        if (mask >> b & 1) top = fmaxf(top, m);
                    }
                    if (__any_sync(0xFFFFFFFFu, top > ref + kSlack)) {
                        const float to = fmaxf(ref, top), keep = exp2a(ref - to);
                        ref = to;
                        l *= keep;
                        if (!(flags & (kFirst | kFlush))) {
                            if (!wait(&bars->pv[(n - 1) & 1], (n - 1) >> 1, &bars->stop, a.wait_cycles)) return;
                            tc_after();
#pragma unroll 1
                            for (int d = 0; d < D; d += 16) {
                                float o[16];
                                tmem_begin16(o, o_at + d);
                                tmem_loaded(o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] *= keep;
                                tmem_store16(o_at + d, reinterpret_cast<const uint32_t(&)[16]>(o));
                            }
                            tmem_stored();
                        }
                    }
                    // the weights
                    F2 sum[2] = {rmsn::f2(0.f, 0.f), rmsn::f2(0.f, 0.f)};
                    if (__any_sync(0xFFFFFFFFu, fabsf(ref) > kWide && ref != kNone)) {
                        // from the rounded products, as the reference was taken
#pragma unroll
                        for (int j = 0; j < C::TOK; ++j) s[j] = __fmul_rn(s[j], kc[j / 16]);
#pragma unroll
                        for (int b = 0; b < C::BLK; ++b) kc[b] = 1.f;
                    }
                    const F2 less = rmsn::f2(-ref, -ref);
#pragma unroll
                    for (int j = 0; j < C::TOK; j += 2) {
                        const F2 k2 = rmsn::f2(kc[j / 16], kc[j / 16]);
                        float lo, hi;
                        rmsn::f2split(rmsn::fma2(rmsn::f2(s[j], s[j + 1]), k2, less), lo, hi);
                        s[j] = exp2a(lo);
                        s[j + 1] = exp2a(hi);
                    }
                    if (mask != (1u << C::BLK) - 1) {
#pragma unroll
                        for (int j = 0; j < C::TOK; ++j)
                            if (!(mask >> (j / 16) & 1)) s[j] = 0.f;
                    }
#pragma unroll
                    for (int c = 0; c < C::TOK; c += 32) {
                        uint32_t y[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int j = c + 2 * i;
                            const F2 pp = rmsn::f2(s[j], s[j + 1]);
                            const float vm = w->vm[j / 16];
                            float lo, hi;
                            sum[i & 1] = rmsn::add2(sum[i & 1], pp);
                            rmsn::f2split(rmsn::mul2(pp, rmsn::f2(vm, vm)), lo, hi);
                            y[i] = rmsn::pack_f16x2(lo, hi);
                        }
                        tmem_store16(s_at + c / 2, y);
                    }
                    float lo, hi;
                    rmsn::f2split(rmsn::add2(sum[0], sum[1]), lo, hi);
                    l += lo + hi;
                    tmem_stored();
                }
                tc_before();
                __syncwarp();
                if (lane == 0) {
                    arrive(smem_of(&bars->p_full[x][n & 1]));
                    arrive(smem_of(&bars->step_free[n % C::M]));
                }
                ++n;
            } while (!(flags & kLast));
        } else {  // the other row tile's steps
            do {
                if (!wait(&bars->step[n % C::M], n / C::M, &bars->stop, a.wait_cycles)) return;
                if (!wait(&bars->s_full[x][n & 1], n >> 1, &bars->stop, a.wait_cycles)) return;
                flags = steps[n % C::M].flags;
                __syncwarp();
                if (lane == 0) {
                    arrive(smem_of(&bars->p_full[x][n & 1]));
                    arrive(smem_of(&bars->step_free[n % C::M]));
                }
                ++n;
            } while (!(flags & kLast));
        }
        // the next piece's queries while the last product runs: its scores are through
        way->next_piece(a, lane);
        if (way->more) load_q();
        if (valid > 0 || x == 0) {
            if (!wait(&bars->pv[(n - 1) & 1], (n - 1) >> 1, &bars->stop, a.wait_cycles)) return;
            tc_after();
            if (busy) {
                drain();
                if (r < valid)
                    *reinterpret_cast<float2*>(part + D * 8 - (r & 7) * 6) = make_float2(ref, l);
            }
        }
    }
}

template <class T, class C>
__global__ void __launch_bounds__(C::kWarps * 32, 1) prefix_kernel(const PrefixArgs a) {
    extern __shared__ unsigned char raw[];
    __shared__ Bars bars;
    __shared__ Step steps[C::M];
    __shared__ Way ways[4 * C::R];
    unsigned char* smem = raw + ((1024 - (smem_of(raw) & 1023)) & 1023);
    const int wp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::M; ++i) {
            rmsn::mbar_init(smem_of(&bars.step[i]), 1);
            rmsn::mbar_init(smem_of(&bars.step_free[i]), 4 * C::R + 9);
        }
        for (int i = 0; i < 2; ++i) {
            rmsn::mbar_init(smem_of(&bars.k_full[i]), 4);
            rmsn::mbar_init(smem_of(&bars.v_full[i]), 4);
            rmsn::mbar_init(smem_of(&bars.pv[i]), 1);
            rmsn::mbar_init(smem_of(&bars.q_full[i]), 4);
            for (int k = 0; k < 2; ++k) {
                rmsn::mbar_init(smem_of(&bars.s_full[i][k]), 1);
                rmsn::mbar_init(smem_of(&bars.p_full[i][k]), 4);
            }
        }
        rmsn::mbar_init(smem_of(&bars.last[0]), 1);
        rmsn::mbar_init(smem_of(&bars.last[1]), 1);
        bars.stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (wp == 4 * C::R + 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_of(&bars.tmem)),
                     "n"(C::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    // (all of TMEM is the block's, so it begins at 0, and places in it are constants)
    if (threadIdx.x == 0 && bars.tmem != 0) bars.stop = 1;
    // The plan's launch, and with it all that the stream wrote before this call, is over and
    // its results are in L2: the launch between, whose programmatic dependent this is, has
    // waited for it in each of its blocks before it let this one begin.  This one does not
    // wait itself before its end, so whatever it reads goes past L1 (plan, table entries,
    // scales by __ldcg, codes and queries by cp.async.cg).
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    unsigned char* stages = smem + C::R * C::kQ;
    unsigned char* codes = stages + 4 * C::kTile;
    if (wp < 4 * C::R) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsS));
        soften<T, C>(a, smem, &bars, steps, &ways[wp], wp >> 2);
    } else if (wp < 4 * C::R + 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsW));
        if (wp < 4 * C::R + 4) widen<C, false>(a, stages, codes, &bars, steps, wp & 3);
        else widen<C, true>(a, stages + 2 * C::kTile, codes + C::N * C::kRaw / 2, &bars, steps, wp & 3);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsM));
        if (threadIdx.x == (4 * C::R + 8) * 32) scores<C>(a, smem, &bars, steps);
        else if (threadIdx.x == (4 * C::R + 9) * 32) sums<C>(a, smem, &bars, steps);
        else if (wp == 4 * C::R + 10) plan<C>(a, &bars, steps);
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (wp == 4 * C::R + 8)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(bars.tmem), "n"(C::kCols) : "memory");
    if (threadIdx.x == 0 && bars.stop) atomicOr(a.status, kWaitRanOut);
    // what waits for this launch has then waited for the one between, too
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <class C>
PrefixEntry entry(int dt) {
    return PrefixEntry{dt, C::D, C::R, C::TOK, C::kWarps * 32, C::kSmem,
                       dt == 1 ? (const void*)&prefix_kernel<BF16, C> : (const void*)&prefix_kernel<F16, C>};
}

}  // namespace prefix
}  // namespace rmsattn
