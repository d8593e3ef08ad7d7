// The root-mean-square norm's geometry: how many threads share a row, and what
// each of them holds.
#include "rms_norm.h"

namespace ct {

namespace {

constexpr int kMaxTpr = 512;

int pow2_at_least(int64_t n) {
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

// What a thread of a row may hold, and at what price.
struct Choice {
    const int *vectors;        // numbers of vectors, ascending, 0 at their end
    int least, most;           // lanes that a row has at least, if it has as many vectors; threads at most
                               // (of more than kRmsFewElements: 512)
    double (*cost)(int);       // of a number of elements
    double whole;              // factor where every thread has all of them
    int threads;               // of a block whose rows have fewer
};

// How many lanes or warps share a row of n vectors of V elements: the choice
// that leaves the fewest places empty, weighed by its cost.
void spread(RmsGeom &g, int64_t n, int V, const Choice &c) {
    double best = 0.0;
    g.K = 0;
    g.lanes_log2 = 5;
    g.warps = kMaxTpr / 32;
    for (const int *of = c.vectors; *of; ++of) {
        const int K = *of;
        int64_t lanes = (n + K - 1) / K, warps = 1;
        if (lanes < 32) {
            lanes = pow2_at_least(lanes);
            const int64_t all = n < c.least ? pow2_at_least(n) : c.least;
            if (lanes < all) lanes = all;
        } else {
            warps = (lanes + 31) / 32;
            lanes = 32;
        }
        if (V == 1 && K > 1 && lanes < 32) continue;     // the kernels know these as whole warps
        if (lanes * warps > (K * V <= kRmsFewElements ? c.most : kMaxTpr)) continue;
        double now = (double)(lanes * warps * K) / (double)n * c.cost(K * V);
        if (lanes == 32 && warps * 32 * K == n) now *= c.whole;
        if (g.K == 0 || now < best) {
            best = now;
            g.K = K;
            g.warps = (int)warps;
            for (g.lanes_log2 = 0; 1 << g.lanes_log2 < lanes;) ++g.lanes_log2;
        }
    }
    const int tpr = (1 << g.lanes_log2) * g.warps;
    g.rpb = tpr < c.threads ? c.threads / tpr : 1;
    g.threads = g.rpb * tpr;
}

// Numbers of vectors a thread that some row's lowest cost is: the kernels have
// no others.
const int kDirect16[] = {1, 2, 3, 8, 0}, kDirect32[] = {1, 2, 3, 4, 0};
const int kRing16[] = {1, 2, 3, 4, 8, 0}, kRing32[] = {1, 4, 0};
const int kBack16[] = {1, 2, 4, 0}, kBack32[] = {1, 2, 3, 4, 8, 0};
const int kSingle[] = {1, 2, 4, 8, 16, 0}, kBackSingle[] = {1, 2, 4, 8, 16, 32, 0};

// Costs, from what part of the floor each way reached with the others' places
// as full.  16 elements a thread are best where nothing else decides (e4m3 of
// 1024 channels 94 %; 8: 81, 24: 65).  768 channels: 24 in one warp 94 %, 8 in
// three 77, 16 in two, one of them half empty, 66; without codes 97, 94, 83.
double cost_codes(int e) { return e < 8 ? 1.4 : e < 12 ? 1.1 : e <= 16 ? 1.0 : e <= 24 ? 1.08 : e <= 32 ? 1.2 : 1.4; }
double cost_plain(int e) { return e < 8 ? 1.4 : e < 12 ? 1.1 : e <= 16 ? 1.0 : e <= 24 ? 1.03 : e <= 32 ? 1.2 : 1.4; }
// The ring of 16-bit elements: eight of them keep little in flight (1280 channels
// 61 %, 16 with a sixth of the places empty 72).
double cost_ring(int e) { return e < 12 ? 1.45 : e <= 16 ? 1.0 : e <= 24 ? 1.03 : e <= 32 ? 1.2 : 1.4; }
// fp32 elements: 16 or as many as there are (320 channels 87 %, 12: 81).
double cost_ring32(int e) { return e < 12 ? 1.5 : e < 16 ? 1.4 : e == 16 ? 1.0 : 1.6; }
// Rows that start inside a vector: the masks weigh less on more of them (1001
// channels: 24 elements 81 %, 16: 73).
double cost_shift(int e) { return e < 12 ? 1.5 : e <= 16 ? 1.1 : e <= 24 ? 1.0 : 1.05; }
// Backward: bf16 of 768 channels 16 elements in two warps, one half empty, 79 %,
// 24 in one 63, 8 in three 61; fp32, 12 in two 102, 16 in two 93.
double cost_back(int e) { return e < 8 ? 1.5 : e < 12 ? 1.4 : e <= 16 ? 1.0 : e <= 24 ? 1.6 : 1.3; }
// Single elements: eight of them a thread.
double cost_single(int e) { return e < 2 ? 2.5 : e < 4 ? 1.6 : e < 8 ? 1.2 : e < 16 ? 1.0 : e < 32 ? 1.15 : 1.6; }

// Rows after which a row starts in its vector where it did before.
int64_t period(int64_t C, int V) {
    int64_t d = V;
    while (C % d != 0) d /= 2;
    return V / d;
}

}  // namespace

RmsGeom rms_forward_geom(const RmsArgs &a, bool aligned) {
    RmsGeom g = {};
    const int V = a.dtype == CT_F32 ? 4 : 8;
    const bool codes = a.scale != nullptr, blocks = codes && a.block != 0 && a.block < a.C;
    // Rows of no whole number of vectors, by vectors all the same: 16-bit elements,
    // from 32 channels on (bf16 with a residual, of the floor and of that of single
    // elements: 100 channels 59 and 48 %, 1001 82 and 67, 8191 77 and 36; e4m3 54
    // and 29, 65 and 33, 51 and 23).  fp32 single elements are nearer (255 channels
    // 102 %, this 70).
    g.shift = aligned && V == 8 && a.C % V != 0 && a.C >= 32 && !blocks;
    g.vec = aligned && (a.C % V == 0 || g.shift);
    // Blocks that stay for many rows.  With one tensor to read they keep more bytes
    // in flight (bf16 of 8192 channels 77 % of the floor, 68 without; 16384 87 and
    // 49; 320 64 and 56); with a residual (190 us, 157 without, for [32768,4096])
    // and for codes (34 %, 41 without) they do not, nor with fp32 elements (83 %,
    // 98 without) but in short rows (64 channels 87 and 65), nor where 16-bit rows
    // of at most 256 threads fill them with 16 elements each, which takes but 32
    // registers (1024 channels 83 %, 87 without; 4096 80 and 82).
    bool stays = g.shift || (!a.residual && !codes && (V == 8 || a.C < 128));
    if (g.vec) {
        // Eight neighbours at least read 128 bytes together; a block's channels lie
        // in one warp.  Blocks of 128 threads: e4m3 of 1536 channels 93 %, of 256
        // threads 76.
        const Choice direct = {V == 8 ? kDirect16 : kDirect32, blocks && a.block / V > 8 ? a.block / V : 8, 1024,
                               codes ? cost_codes : cost_plain, 0.87, 128};
        Choice ring = direct;
        ring.vectors = V == 8 ? kRing16 : kRing32;
        ring.cost = g.shift ? cost_shift : V == 8 ? cost_ring : cost_ring32;
        ring.whole = 1.0;
        ring.most = kMaxTpr;
        // a row that starts inside a vector has one vector more
        const int64_t n = g.shift ? (a.C + 2 * V - 2) / V : a.C / V;
        if (!g.shift) {
            spread(g, n, V, direct);
            if (stays && V == 8 && g.K == 2 && g.threads <= 256 && n == (int64_t)64 * g.warps && g.lanes_log2 == 5 &&
                a.weight && a.rows % g.rpb == 0)
                stays = false;
        }
        if (stays) spread(g, n, V, ring);
        if (g.shift && (g.K == 0 || g.K > 4)) g.vec = g.shift = false;
    }
    if (!g.vec) {
        // a block of 64 or 128 single channels lies in two or four vectors of a warp
        const int skip = !blocks ? 0 : a.block == 128 ? 2 : a.block == 64 ? 1 : 0;
        spread(g, a.C, 1, {kSingle + skip, 32, 1024, cost_single, 1.0, 256});
    }
    g.blocks = ceil_div(a.rows, (int64_t)g.rpb);
    if (g.blocks > 0x7FFFFFFF) g.blocks = 0x7FFFFFFF;
    if (g.vec && g.K > 0 && g.K <= 4 && stays) {
        // as many as are resident
        const int64_t bytes = (int64_t)rms_forward_stages(g.K) * (a.residual ? 2 : 1) * g.K * g.threads * 16 + 2048;
        int64_t resident = 228 * 1024 / bytes;
        // 64 registers a thread, or up to 128
        const bool many = g.K * V > kRmsFewElements || (g.shift && codes && g.K > 1);
        const int64_t most = (many ? 512 : 1024) / g.threads;
        if (resident > most) resident = most;
        if (resident < 1) resident = 1;
        if (g.shift || g.blocks >= 296 * resident) g.ring = 148 * resident;
        if (g.shift) {
            const int64_t P = period(a.C, V);
            g.ring = g.ring / P * P;
            if (g.ring > g.blocks) g.ring = g.blocks;      // a round at most: every slot has one row
        }
    }
    return g;
}

// dweight's partial sums.  Rows in registers: one of each block, all resident
// at once.  Rows that are walked: enough for a round of blocks of 256 columns.
int64_t rms_parts(int64_t rows, int64_t C) {
    const int64_t most = C <= 16384 ? 148 * 4 : 148 * 8 * 256 / C;
    const int64_t n = C <= 16384 ? rows : ceil_div(rows, (int64_t)32);
    const int64_t parts = n < most ? n : most;
    return parts < 1 ? 1 : parts;
}

RmsGeom rms_backward_geom(const RmsArgs &a, bool aligned) {
    RmsGeom g = {};
    const int V = a.dtype == CT_F32 ? 4 : 8;
    g.vec = aligned && a.C % V == 0;
    // blocks of 256 threads (1536 channels 78 %, of 128: 56)
    if (g.vec) spread(g, a.C / V, V, {V == 8 ? kBack16 : kBack32, 8, kMaxTpr, cost_back, 1.0, 256});
    else spread(g, a.C, 1, {kBackSingle, 32, kMaxTpr, cost_single, 1.0, 256});
    const int64_t rounds = ceil_div(a.rows, (int64_t)g.rpb);
    // one round of resident blocks, as the ring lets them be
    int64_t parts = rms_parts(a.rows, a.C);
    if (g.vec && g.K > 0) {
        const int64_t ring = (int64_t)rms_stages(g.K) * (a.dsum ? 3 : 2) * g.K * g.threads * 16 + 2048;
        int64_t resident = (228 * 1024) / ring;
        // the registers of 512 threads; with more than 16 elements, of one block
        if (resident > 512 / g.threads) resident = 512 / g.threads;
        if (resident > (g.K * V > kRmsFewElements ? 1 : 2)) resident = g.K * V > kRmsFewElements ? 1 : 2;
        if (resident < 1) resident = 1;
        if (parts > 148 * resident) parts = 148 * resident;
    }
    g.blocks = rounds < parts ? rounds : parts;
    if (g.blocks < 1) g.blocks = 1;
    return g;
}

namespace {

bool all_aligned(const RmsArgs &a) {
    const uintptr_t p = (uintptr_t)a.x | (uintptr_t)a.residual | (uintptr_t)a.weight | (uintptr_t)a.sum |
                        (uintptr_t)a.dy | (uintptr_t)a.dsum | (uintptr_t)a.dx;
    // codes: a vector's worth of them is half as long as a vector, or a quarter
    return (p & 15) == 0 && ((uintptr_t)a.y & (a.scale ? 7 : 15)) == 0;
}

}  // namespace

ct_status rms_forward(const RmsArgs &a, cudaStream_t st) {
    const RmsGeom g = rms_forward_geom(a, all_aligned(a));
    if (a.dtype == CT_F32) return rms_forward_f32(a, g, st);
    if (a.dtype == CT_F16) return rms_forward_f16(a, g, st);
    return rms_forward_bf16(a, g, st);
}

ct_status rms_backward(const RmsArgs &a, cudaStream_t st) {
    const RmsGeom g = rms_backward_geom(a, all_aligned(a));
    if (a.dtype == CT_F32) return rms_backward_f32(a, g, st);
    if (a.dtype == CT_F16) return rms_backward_f16(a, g, st);
    return rms_backward_bf16(a, g, st);
}

}  // namespace ct
