// Attention with a shared prefix: which sequences share how much, and the line of
// the shared parts' steps (PrefixGroup).  One block; a warp to a group.  A sequence
// shares a prefix if each of its queries sees all of it.
//
// What bounds it: latency, 3 to 4 us with the launch (lengths, then the groups' places).  It
// stands before both parts, which wait for nothing else.
#include "attn_common.cuh"

namespace rmsattn {

namespace {

constexpr int kThreads = 512;

__global__ void __launch_bounds__(kThreads) prefix_plan(const PrefixArgs a) {
    __shared__ int64_t sums[2][kThreads / 32];
    __shared__ int4 sizes[kThreads];  // tiles, steps and sequences of the first groups
    rmsn::pdl_wait(a.pdl);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const PrefixSeq alone = {0, 0};
    // borders that are out of order, or of other sequences: nobody shares
    bool bad = false;
    if (a.cu) {
        for (int g = threadIdx.x; g < a.n_groups; g += kThreads)
            bad = bad || a.cu[g] < 0 || a.cu[g + 1] < a.cu[g] || a.cu[g + 1] > a.B;
    }
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0) atomicOr(a.status, kBadPage);
    // sequences of no group (the groups lie one behind the other)
    const bool none = bad || a.n_groups == 0;
    const int64_t from = none ? a.B : (a.cu ? a.cu[0] : 0), to = none ? a.B : (a.cu ? a.cu[a.n_groups] : a.B);
    for (int64_t b = threadIdx.x; b < a.B; b += kThreads)
        if (b < from || b >= to) a.seqs[b] = alone;
    const int64_t room = a.table_width * a.c.page;
    for (int g = wp; g < a.n_groups; g += kThreads / 32) {
        PrefixGroup G = {0, 0, 0, -1, 0, 0, 0, 0};
        if (!bad) {
            G.s0 = a.cu ? a.cu[g] : 0;
            G.s1 = a.cu ? a.cu[g + 1] : (int32_t)a.B;
            // whole blocks; the rest is each sequence's own
            int32_t shared = a.shared[g];
            if (shared > room) shared = (int32_t)room;
            shared = shared < 0 ? 0 : shared & ~(kBlock - 1);
            int count = 0;
            constexpr int U = 8;  // lengths of a lane on their way at once
            for (int b0 = G.s0; b0 < G.s1; b0 += 32 * U) {
                uint32_t on = 0;
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int b = b0 + 32 * k + lane;
                    const bool in = b < G.s1;
                    const int32_t len = a.lengths[in ? b : G.s0];
                    on |= (uint32_t)(in && shared > 0 && len - (int64_t)a.n + 1 >= shared) << k;
                }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const uint32_t who = __ballot_sync(0xFFFFFFFFu, on >> k & 1);
                    if (G.seq < 0 && who) G.seq = b0 + 32 * k + __ffs(who) - 1;
                    count += __popc(who);
                    const int b = b0 + 32 * k + lane;
                    if (b < G.s1) a.seqs[b] = on >> k & 1 ? PrefixSeq{shared, g} : alone;
                }
            }
            if (count > 1) {
                G.shared = shared;
                G.ns = (shared + a.tok - 1) / a.tok;
                G.tiles = (int)(((int64_t)(G.s1 - G.s0) * a.n * a.group + a.rows - 1) / a.rows);
            } else if (count == 1) {  // nobody to share with
                __syncwarp();
                if (lane == 0) a.seqs[G.seq] = alone;
            }
        }
        __syncwarp();
        if (lane == 0) {
            a.groups[g] = G;
            if (g < kThreads) sizes[g] = make_int4(G.tiles, G.ns, G.s0, G.s1);
        }
    }
    __syncthreads();
    // the groups' places on the line, and those of their parts' rows, in eights
    int64_t steps = 0, rows = 0;
    for (int g0 = 0; g0 < a.n_groups; g0 += kThreads) {
        const int g = g0 + threadIdx.x;
        int64_t ro = 0, st = 0;
        if (g < a.n_groups) {
            int4 n;
            if (g < kThreads) n = sizes[g];
            else n = make_int4(a.groups[g].tiles, a.groups[g].ns, a.groups[g].s0, a.groups[g].s1);
            if (n.x > 0) ro = (int64_t)prefix_eights((uint32_t)(n.w - n.z) * a.n * a.group) * a.c.H;
            st = (int64_t)n.x * a.c.H * n.y;
        }
        int64_t r1 = ro, s1 = st;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xFFFFFFFFu, r1, o), v = __shfl_up_sync(0xFFFFFFFFu, s1, o);
            if (lane >= o) {
                r1 += u;
                s1 += v;
            }
        }
        if (lane == 31) {
            sums[0][wp] = r1;
            sums[1][wp] = s1;
        }
        __syncthreads();
        int64_t r0 = rows + r1 - ro, s0 = steps + s1 - st;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < wp) {
                r0 += sums[0][w];
                s0 += sums[1][w];
            }
            rows += sums[0][w];
            steps += sums[1][w];
        }
        __syncthreads();
        if (g < a.n_groups) {
            a.groups[g].first = (int32_t)s0;
            a.groups[g].row0 = (int32_t)r0;
        }
    }
    if (threadIdx.x == 0) {
        int64_t chunk = (steps + a.shares - 1) / a.shares;
        if (chunk < 1) chunk = 1;
        *a.line = PrefixLine{(int32_t)steps, (int32_t)chunk, {0, 0}};
    }
}

}  // namespace

const void* prefix_plan_kernel() { return (const void*)&prefix_plan; }

}  // namespace rmsattn
