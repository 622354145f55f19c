// C-ABI entry points of the token embedding and of the log probabilities (include/txl.h):
// argument validation, work division, workspace layout, launches.
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "txl.h"
#include "vocab.h"

namespace {

using txl::GemmParams;

bool on(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int status_of(cudaError_t e) { return e == cudaSuccess ? TXL_OK : TXL_ERR_CUDA; }
cudaStream_t stream_of(void *s) { return static_cast<cudaStream_t>(s); }
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
long long up64(long long x) { return (x + 63) / 64 * 64; }
long long up128(long long x) { return (x + 127) / 128 * 128; }
int elem(int dtype) { return dtype == TXL_BF16 ? 2 : 4; }

constexpr int kMaxRows = 1 << 28;   // rows, tokens
constexpr int kMaxVocab = 1 << 28;
constexpr int kMaxWidth = 1 << 16;

int check_type(int dtype)
{
    return dtype == TXL_F32 || dtype == TXL_BF16 ? TXL_OK : TXL_ERR_INVALID_ARG;
}

int check_ids(const void *ids, int index_type)
{
    if (index_type != TXL_I32 && index_type != TXL_I64) return TXL_ERR_INVALID_ARG;
    return on(ids, (size_t)index_type) ? TXL_OK : TXL_ERR_MISALIGNED;
}

// A [rows][d] operand whose rows are stride elements apart.
int check_rows(const void *p, long long stride, int rows, int d, int dtype)
{
    if (stride < 1) return TXL_ERR_INVALID_ARG;
    if (stride < d && rows > 1) return TXL_ERR_SHAPE;
    if (!on(p, 16) || (stride * elem(dtype)) % 16 != 0) return TXL_ERR_MISALIGNED;
    return stride > (1LL << 36) ? TXL_ERR_UNSUPPORTED : TXL_OK;
}

// d a multiple of `unit`.
int check_sizes(int n, int V, int d, int unit)
{
    if (n < 0 || V < 1 || d < 1) return TXL_ERR_INVALID_ARG;
    if (d % unit != 0 || n > kMaxRows || V > kMaxVocab || d > kMaxWidth) return TXL_ERR_UNSUPPORTED;
    return TXL_OK;
}

// 16 bytes of elements of this type, or of the narrower of two.
int unit_of(int dtype, int other = TXL_F32)
{
    return dtype == TXL_BF16 || other == TXL_BF16 ? 8 : 4;
}

// A range of memory; what is written must overlap nothing else.
struct Range {
    const void *p;
    size_t bytes;
};

Range rows_range(const void *p, long long stride, int rows, int d, int dtype)
{
    return {p, rows < 1 ? 0 : ((size_t)(rows - 1) * stride + d) * elem(dtype)};
}

// Whether one of the first n_out ranges (outputs) overlaps any other.
bool overlap(std::initializer_list<Range> r, int n_out)
{
    const Range *a = r.begin();
    for (int i = 0; i < n_out; ++i)
        for (int j = i + 1; j < (int)r.size(); ++j) {
            const uintptr_t x = reinterpret_cast<uintptr_t>(a[i].p), y = reinterpret_cast<uintptr_t>(a[j].p);
            if (x && y && a[i].bytes && a[j].bytes && x < y + a[j].bytes && y < x + a[i].bytes) return true;
        }
    return false;
}

// ---------------------------------------------------------------------------
// work division of the log probabilities
// ---------------------------------------------------------------------------

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// Row stride of rows in the workspace: whole lines of 128 bytes of bf16, so that a tile's 128-byte
// rows do not straddle two (G of 333 x 5003 from fp32 rows of 520: 28.8 us with terms of stride 520, 24.3
// so).
int line_ld(int d) { return (int)up64(d); }

// Tiles of a product of `rows` x `cols`: 256 rows (a pair of blocks'), 128 or 256 columns, and parts
// of its longer dimension where there are fewer tiles than pairs.
struct Shape {
    int bn, mb, nb, parts;
};

// What an item adds besides its steps, in cycles: its epilogue runs beside the next item's steps,
// but its accumulator's first use and its stores do not quite.
constexpr double kItemCost = 1500.0;

// Steps of a part of a product whose result is fp32, at most: the accumulators' cut additions are made good
// on average only, and a longer chain leaves more of them.  fp32 dh of 2048 x 32000 x 512, relative to its norm, in
// parts of 500 steps 9.5e-6, of 125 6.7e-6, of 63 1.6e-6, of 32 1.3e-6 (the whole gradient 673, 682, 689
// and 701 us; fp32 library products 4.5e-6).  Where nothing is cut (one term among zeros) the mean itself is the
// error: 4.1e-6 of the value with 64 steps, 8.2e-6 where G is a pair; a word of 20000 rows in one part 4.0e-5.
constexpr int kMaxChain = 64;

// The launch that sums parts, in cycles.
constexpr double kSumLaunch = 4500.0;

// A cold step's latency, in cycles: over the ring's six stages, or four with two terms each, it is the least
// that a step takes (29 x 56301 x 224, dh by 16 pairs with four stages: 760 cycles a step).
constexpr double kColdStep = 3000.0;

// Cycles of one 64-wide step of `terms` (GemmParams): the MMAs' (one product, 256 columns: 512) or the
// copies' at some 58 bytes a cycle and SM (602 cycles a step in the statistics of 2048 x 131072).
double step_cycles(int bn, int terms, int a_rows = 128)
{
    const int products = terms == 3 ? 6 : terms, a = terms, b = terms == 3 ? 3 : 1;
    return std::max({2.0 * bn * products, (128.0 * a_rows * a + 64.0 * bn * b) / 58.0,
                     kColdStep / (terms == 2 ? 4 : 6)});
}

// Rows of A's boxes.
int box_rows(long long rows) { return rows < 128 ? (int)(rows + 7) / 8 * 8 : 128; }

// Whether tiles of bn columns are a choice: 256 only past 128 columns, and not with three terms, whose
// two accumulators take the room (nor would they gain: their steps are bound by the MMAs).
bool columns_fit(int bn, long long cols, int terms) { return bn == 128 || (cols > 128 && terms < 3); }

// `steps`: 64-wide steps of a tile; parts: up to `most` ranges of a row block's tiles (0: an item
// a tile).
Shape choose_shape(long long rows, long long cols, int steps, int terms, int most)
{
    const int pairs = txl::device_sm_count() / 2;
    Shape best{};
    double least = 0.0;
    for (const int bn : {256, 128}) {
        if (!columns_fit(bn, cols, terms)) continue;
        Shape s{bn, ceil_div(rows, 256), ceil_div(cols, bn), 1};
        const int n = std::max(1, std::min(most, s.nb));
        for (; s.parts <= n; ++s.parts) {
            const long long items = (long long)s.mb * (most ? s.parts : s.nb);
            const double waves = (double)((items + pairs - 1) / pairs);
            const double work = (double)steps * (most ? ceil_div(s.nb, s.parts) : 1);
            const double cost = waves * (work * step_cycles(bn, terms) + kItemCost);
            if (best.mb == 0 || cost < least) {
                best = s;
                least = cost;
            }
        }
    }
    return best;
}

double item_cycles(int steps, int bn, int terms, int a_rows = 128)
{
    return (double)steps * step_cycles(bn, terms, a_rows) + kItemCost;
}

// Two products share a launch: the items of the first over the pairs in turn, then those of the
// second, of which the pairs that have one less of the first begin with `early`.  The cycles of the
// longest pair, and the best `early`.  (Without it the gradient of 2048 x 32000 x 1024 has pairs of 474
// steps where the mean is 421; with it 442.)
struct Turns {
    int early;
    double cycles;
};

Turns take_turns(long long n0, double c0, long long n1, double c1)
{
    const long long pairs = std::min<long long>(n0 + n1, txl::device_sm_count() / 2);
    const long long more = n0 % pairs, fewer = pairs - more, k = n0 / pairs;
    // (an item of the first is worth about c0 / c1 of the second)
    const long long about = more ? (long long)(c0 / c1) : 0, most = more ? std::min(n1 / fewer, about + 1) : 0;
    Turns best{0, 0.0};
    for (long long e = std::max(0LL, std::min(most, about - 1)); e <= most; ++e) {
        const long long rest = n1 - e * fewer, f = rest / pairs, x = rest % pairs;
        const double a = more ? (double)(k + 1) * c0 + (double)(f + (x > 0)) * c1 : 0.0,
                     b = (double)k * c0 + (double)(e + f + (x > more)) * c1, cycles = std::max(a, b);
        if (best.cycles == 0.0 || cycles < best.cycles) best = {(int)e, cycles};
    }
    return best;
}

// The tiles and parts of two products that share a launch.
struct Two {
    Shape a, b;
    double cycles;
};

constexpr int kParts[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 15, 16, 19, 25, 32, 38, 50, 64, 76};
constexpr int kPartChoices = sizeof kParts / sizeof kParts[0];

// The first of kParts from place k on that is more than `parts`, or 0.
int next_parts(int parts, int &k)
{
    while (k < kPartChoices && kParts[k] <= parts) ++k;
    return k < kPartChoices ? kParts[k] : 0;
}

// (f32: whether the results are)
Two choose_two(const long long (&rows)[2], long long cols, const int (&steps)[2], const int (&terms)[2],
               const bool (&f32)[2], int planes)
{
    const int pairs = txl::device_sm_count() / 2;
    struct Option {
        Shape s;
        long long items;
        double cost, extra;  // cycles of an item, and of the parts' writes and reads (3.6 kB a cycle)
    };
    Option o[2][2 * kPartChoices];  // (`least` and those of kParts above it: no more than kParts has)
    int n[2] = {};
    for (int i = 0; i < 2; ++i)
        for (const int bn : {256, 128}) {
            if (!columns_fit(bn, cols, terms[i])) continue;
            const int least = f32[i] ? ceil_div(steps[i], kMaxChain) : 1;
            for (int k = 0, parts = least; parts > 0; parts = next_parts(parts, k)) {
                const int mb = ceil_div(rows[i], 256), nb = ceil_div(cols, bn);
                // (the fewest that are allowed are always a choice; beyond them four items a pair are as even
                // as it needs)
                if (parts > least && (parts > steps[i] || (long long)mb * nb * parts > 4 * pairs)) break;
                Option &x = o[i][n[i]++];
                x.s = {bn, mb, nb, parts};
                x.items = (long long)x.s.mb * x.s.nb * parts;
                x.cost = item_cycles(ceil_div(steps[i], parts), bn, terms[i],
                                     i == 0 && planes == 2 ? box_rows(rows[0]) : 128);
                const int written = parts * (i ? 1 : planes);  // (planes: parts of dh that one of them leaves)
                x.extra = written > 1 ? written * 2.0 * rows[i] * cols * 4 / 3600.0 : 0.0;
            }
        }
    Two best{};
    double least = 0.0;
    for (int i = 0; i < n[0]; ++i)
        for (int j = 0; j < n[1]; ++j) {
            const Option &x = o[0][i], &y = o[1][j];
            const double cost = take_turns(x.items, x.cost, y.items, y.cost).cycles + x.extra + y.extra +
                                (x.s.parts * planes > 1 || y.s.parts > 1 ? kSumLaunch : 0.0);
            if (best.a.mb == 0 || cost < least) {
                best = {x.s, y.s, cost};
                least = cost;
            }
        }
    return best;
}

struct StatsPlan {
    bool few;                     // the vocabulary in the tiles' rows
    bool full;                    // ... and the logits written
    int mb, nb, bn, splits, list;
    size_t h_planes, w_planes, stats, val, id, keys, logits, target_z, total;  // offsets
};

StatsPlan plan_stats(int N, int V, int d, int dtype, int top)
{
    StatsPlan s{};
    // Up to kFewRows states the vocabulary takes the tiles' rows: the table is read at DRAM's rate, and
    // alternatives need no lists (4 of them, 32000 x 1024 in bf16: 64, 128, 256 states 21.2, 24.2, 35.8 us;
    // with the states in the tiles' rows 60 each).  Without alternatives the other way is no slower where
    // the vocabulary leaves SMs without a tile: 5003 x 256, 64, 96, 160, 256 states 7.0, 8.4, 12.0, 13.9 us
    // and 8.2, 8.1, 8.5, 8.5; but 131072 x 512, 160 and 256 states 43 and 53, and 61; 32000 x 1024 23.4 and
    // 25.7, and 24.7.  In fp32 (5003 x 520) from 129 states on: 29.7 us and 28.4, 200 states 39.8 and 29.0.
    const bool idle = ceil_div(V, 128) < txl::device_sm_count();
    s.few = N <= txl::kFewRows && !(top == 0 && idle && N > (dtype == TXL_F32 ? 128 : 64));
    if (s.few) {
        s.mb = 1;
        s.bn = std::max(16, ceil_div(N, 16) * 16);
        s.nb = ceil_div(V, 128);
        // The logits of up to d / 16 states are an eighth of the table's bytes at most; with them the
        // merge forms a quarter of the exact products (one state, 32000 x 1024, eight alternatives:
        // 4.8 us less).
        s.full = top > 0 && (long long)N * 16 <= d && N <= 64;
        s.splits = std::min(s.nb, std::min(txl::device_sm_count(), txl::kMaxStatSplits));
    } else {
        const Shape c = choose_shape(N, V, ceil_div(d, 64), dtype == TXL_F32 ? 3 : 1, txl::kMaxRowSplits);
        s.mb = c.mb;
        s.bn = c.bn;
        s.nb = c.nb;
        s.splits = c.parts;
    }
    s.list = txl::list_length(top);
    size_t o = 0;
    const size_t row = (size_t)line_ld(d) * 2 * txl::kMaxPieces;
    s.h_planes = o;
    if (dtype == TXL_F32) o = up256(o + N * row);
    s.w_planes = o;
    if (dtype == TXL_F32) o = up256(o + V * row);
    s.stats = o;
    o = up256(o + (size_t)(s.few ? 1 : 2) * s.splits * N * sizeof(float4));
    const size_t lists = s.few ? 0 : (size_t)2 * s.splits * s.list * N * 4;
    s.val = o;
    o = up256(o + lists);
    s.id = o;
    o = up256(o + lists);
    s.keys = o;
    if (s.few && top > 0) o = up256(o + (size_t)N * s.nb * 32 * 4);
    s.logits = o;
    if (s.full) o = up256(o + (size_t)N * s.nb * 128 * 4);
    s.target_z = o;
    s.total = s.few ? up256(o + (size_t)N * 4) : o;
    return s;
}

constexpr int kPairRows = 128;
constexpr size_t kGradBytes = (size_t)1 << 30;  // of G in the workspace: vocabulary chunks beyond

struct GradPlan {
    int chunk, chunks;            // vocabulary rows at a time
    int pieces, pieces_h;         // terms of G, and those that dh takes
    int stacked;                  // GemmParams, of dh
    Shape g, h, w;                // tiles of G, of dh, and of a chunk's dW
    int parts_h;                  // of a chunk's dh
    long long g_ld, g_plane;
    size_t live, target_logp, w_planes, g_at, part_h, part_w, total;
};

GradPlan make_grad_plan(int N, int V, int d, int dtype, int grad_dtype)
{
    GradPlan g{};
    // Terms of G.  One bf16 value for bf16 gradients: its rounding is as large as the result's own, and
    // averages over the rows.  Few rows do not average, and their products are bound by the table's
    // bytes: up to 128 rows (about where two terms' MMAs take as long as reading and writing the
    // table) G is a pair.
    const bool few = N <= kPairRows;
    g.pieces_h = dtype == TXL_F32 ? 3 : few ? 2 : 1;
    g.pieces = dtype == TXL_F32 ? 3 : few || grad_dtype == TXL_F32 ? 2 : 1;
    const long long most = (long long)(kGradBytes / ((size_t)g.pieces * 2 * std::max(N, 1)));
    g.chunk = V;
    if (V > std::max(64LL, most)) g.chunk = (int)std::max(64LL, most / 64 * 64);
    g.chunks = ceil_div(V, g.chunk);
    if (g.chunks > 1) g.chunk = (int)up64(ceil_div(V, g.chunks));
    g.chunks = ceil_div(V, g.chunk);
    g.g_ld = up128(g.chunk);
    g.g_plane = g.g_ld * N;
    g.g = choose_shape(N, g.chunk, ceil_div(d, 64), dtype == TXL_F32 ? 3 : 1, 0);
    const int kb_h = ceil_div(g.chunk, 64), kb_w = ceil_div(N, 64);
    const bool f32[2] = {dtype == TXL_F32, grad_dtype == TXL_F32};
    // (G a pair: its terms in the two blocks of a pair, which leaves parts to sum, or both in each)
    Two two = choose_two({(long long)N, (long long)g.chunk}, d, {kb_h, kb_w}, {g.pieces_h, g.pieces}, f32, 1);
    if (g.pieces_h == 2) {
        const Two apart = choose_two({(long long)N, (long long)g.chunk}, d, {kb_h, 2 * kb_w}, {1, 1}, f32, 2);
        g.stacked = apart.cycles < two.cycles;
        if (g.stacked) two = apart;
    }
    g.h = two.a;
    g.w = two.b;
    g.parts_h = g.h.parts * (g.stacked ? 2 : 1);
    size_t o = 0;
    const size_t row = (size_t)line_ld(d) * 2 * txl::kMaxPieces;
    g.live = o;
    o = up256(o + (dtype == TXL_F32 ? N * row : (size_t)N * line_ld(d) * 2));
    g.target_logp = o;
    o = up256(o + (size_t)N * 4);
    g.w_planes = o;
    if (dtype == TXL_F32) o = up256(o + V * row);
    g.g_at = o;
    o = up256(o + (size_t)g.pieces * g.g_plane * 2);
    // (past one chunk: what the chunks so far have summed, then a chunk's parts.  Parts of all chunks would
    // be N rows for each of N V / 2^29 chunks)
    g.part_h = o;
    if (g.parts_h > 1 || g.chunks > 1) o = up256(o + (size_t)(g.parts_h + (g.chunks > 1)) * N * d * 4);
    g.part_w = o;
    if (g.w.parts > 1) o = up256(o + (size_t)g.w.parts * g.chunk * d * 4);
    g.total = o;
    return g;
}

// A training loop asks for one plan again and again: the thread's last one is kept (its sizes, that
// is; choosing takes some microseconds).
GradPlan plan_grad(int N, int V, int d, int dtype, int grad_dtype)
{
    struct Last {
        int key[6] = {};
        GradPlan plan;
    };
    static thread_local Last last;
    const int key[6] = {N, V, d, dtype, grad_dtype, txl::device_sm_count()};
    if (!std::equal(key, key + 6, last.key)) {
        last.plan = make_grad_plan(N, V, d, dtype, grad_dtype);
        std::copy(key, key + 6, last.key);
    }
    return last.plan;
}

// (a lone row may come with any stride: its own width then)
long long own_ld(long long ld, int rows, int d) { return rows > 1 ? ld : d; }

// The bf16 terms of a [rows][d] operand: itself, or its planes in the workspace.
struct Operand {
    const void *p;
    long long ld;
    int planes;
    long long plane;
};

Operand operand(const void *p, long long ld, const char *planes, int rows, int d, int dtype)
{
    if (dtype == TXL_BF16) return {p, own_ld(ld, rows, d), 1, own_ld(ld, rows, d)};  // (one plane: its stride is of no meaning)
    return {planes, line_ld(d), txl::kMaxPieces, (long long)rows * line_ld(d)};
}

txl::SplitRows split_of(const void *x, long long ld, int rows, int d, char *planes)
{
    return {static_cast<const float *>(x), ld, rows, d, line_ld(d), reinterpret_cast<__nv_bfloat16 *>(planes)};
}

bool map_of(CUtensorMap *map, const Operand &o, int rows, int d, unsigned box_rows)
{
    return txl::make_map_planes(map, o.p, d, rows, o.ld, o.planes, o.plane, box_rows);
}

// A product's parts, or the result, for its tiles' stores.
bool map_out(CUtensorMap *map, const GemmParams &p, char *base)
{
    const long long plane = (long long)p.M * p.N;
    const int parts = p.part ? p.splits * (p.stacked ? 2 : 1) : 1;
    return p.part || !p.out_bf16
               ? txl::make_map_planes_f32(map, base, p.N, p.M, p.N, parts, plane, 32)
               : txl::make_map_planes(map, base, p.N, p.M, p.N, 1, plane, 32);
}

} // namespace

extern "C" {

int txl_embed_fwd(const void *tokens, int index_type, const void *emb, long long emb_stride,
                  void *out, int n, int V, int d, float scale, int dtype, void *stream)
{
    int rc;
    if ((rc = check_type(dtype)) != TXL_OK || (rc = check_sizes(n, V, d, 1)) != TXL_OK) return rc;
    if ((rc = check_ids(tokens, index_type)) != TXL_OK) return rc;
    if (!emb || (n > 0 && (!tokens || !out)) || !std::isfinite(scale) || emb_stride < 1) return TXL_ERR_INVALID_ARG;
    if (emb_stride < d && V > 1) return TXL_ERR_SHAPE;
    if (emb_stride > (1LL << 36)) return TXL_ERR_UNSUPPORTED;
    if (!on(emb, (size_t)elem(dtype)) || !on(out, (size_t)elem(dtype))) return TXL_ERR_MISALIGNED;
    if (overlap({{out, (size_t)n * d * elem(dtype)}, {tokens, (size_t)n * index_type},
                 rows_range(emb, emb_stride, V, d, dtype)}, 1))
        return TXL_ERR_INVALID_ARG;
    if (n == 0) return TXL_OK;
    if ((long long)n * d / 1024 > 0x7ffffff0LL) return TXL_ERR_UNSUPPORTED;
    txl::EmbedParams p{};
    p.status = txl::device_status_word();
    if (!p.status) return TXL_ERR_CUDA;
    p.tokens = tokens;
    p.index_bytes = index_type;
    p.emb = emb;
    p.emb_ld = emb_stride;
    p.out = out;
    p.n = n;
    p.V = V;
    p.d = d;
    p.scale = scale;
    return status_of(txl::launch_embed_fwd(p, dtype == TXL_BF16, stream_of(stream)));
}

size_t txl_embed_bwd_workspace_size(int n, int V, int d)
{
    if (check_sizes(n, V, d, unit_of(TXL_F32)) != TXL_OK) return 0;
    return n == 0 ? 0 : txl::embed_bwd_workspace_bytes(n, d);
}

int txl_embed_bwd(const void *tokens, int index_type, const void *dout, long long dout_stride,
                  void *demb, int n, int V, int d, float scale, int dtype, int grad_dtype,
                  int accumulate, void *workspace, size_t workspace_bytes, void *stream)
{
    int rc;
    if ((rc = check_type(dtype)) != TXL_OK || (rc = check_type(grad_dtype)) != TXL_OK) return rc;
    if ((rc = check_sizes(n, V, d, unit_of(dtype, grad_dtype))) != TXL_OK) return rc;
    if ((rc = check_ids(tokens, index_type)) != TXL_OK) return rc;
    if (!demb || (n > 0 && (!tokens || !dout)) || !std::isfinite(scale)) return TXL_ERR_INVALID_ARG;
    if (accumulate && grad_dtype != TXL_F32) return TXL_ERR_UNSUPPORTED;
    if (n > 0 && (rc = check_rows(dout, dout_stride, n, d, dtype)) != TXL_OK) return rc;
    if (!on(demb, 16)) return TXL_ERR_MISALIGNED;
    if (overlap({{demb, (size_t)V * d * elem(grad_dtype)}, {workspace, n > 0 ? workspace_bytes : 0},
                 {tokens, (size_t)n * index_type}, rows_range(dout, dout_stride, n, d, dtype)}, 2))
        return TXL_ERR_INVALID_ARG;
    cudaStream_t s = stream_of(stream);
    if (n == 0)
        return accumulate ? TXL_OK
                          : status_of(cudaMemsetAsync(demb, 0, (size_t)V * d * elem(grad_dtype), s));
    if (!workspace || workspace_bytes < txl::embed_bwd_workspace_bytes(n, d)) return TXL_ERR_WORKSPACE;
    if (!on(workspace, 256)) return TXL_ERR_MISALIGNED;
    txl::EmbedBwdParams p{};
    p.status = txl::device_status_word();
    if (!p.status) return TXL_ERR_CUDA;
    p.tokens = tokens;
    p.index_bytes = index_type;
    p.dout = dout;
    p.dout_ld = dout_stride;
    p.demb = demb;
    p.n = n;
    p.V = V;
    p.d = d;
    p.scale = scale;
    p.accumulate = accumulate != 0;
    return status_of(txl::launch_embed_bwd(p, dtype == TXL_BF16, grad_dtype == TXL_BF16, workspace, s));
}

size_t txl_logprob_fwd_workspace_size(int N, int V, int d, int top, int dtype)
{
    if (check_sizes(N, V, d, 8) != TXL_OK || check_type(dtype) != TXL_OK || top < 0 || top > txl::kMaxTop)
        return 0;
    return N == 0 ? 0 : plan_stats(N, V, d, dtype, top).total;
}

int txl_logprob_fwd(const void *h, long long h_stride, const void *w, long long w_stride,
                    const void *targets, int index_type, float *logp, float *lse, float *entropy,
                    float *top_logp, int *top_ids, int N, int V, int d, int top, float scale,
                    int dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    int rc;
    if ((rc = check_type(dtype)) != TXL_OK || (rc = check_sizes(N, V, d, 8)) != TXL_OK) return rc;
    if ((rc = check_ids(targets, index_type)) != TXL_OK) return rc;
    if (top < 0 || !w || (N > 0 && !h) || !std::isfinite(scale)) return TXL_ERR_INVALID_ARG;
    if (top > txl::kMaxTop) return TXL_ERR_UNSUPPORTED;
    if (N > 0 && top > 0 && (!top_logp || !top_ids)) return TXL_ERR_INVALID_ARG;
    if (N > 0 && !logp && !lse && !entropy && top == 0) return TXL_ERR_INVALID_ARG;
    if (N > 0 && (rc = check_rows(h, h_stride, N, d, dtype)) != TXL_OK) return rc;
    if ((rc = check_rows(w, w_stride, V, d, dtype)) != TXL_OK) return rc;
    for (const void *p : {(const void *)logp, (const void *)lse, (const void *)entropy,
                          (const void *)top_logp, (const void *)top_ids})
        if (!on(p, 4)) return TXL_ERR_MISALIGNED;
    const size_t row4 = (size_t)N * 4;
    if (overlap({{logp, row4}, {lse, row4}, {entropy, row4}, {top_logp, row4 * top}, {top_ids, row4 * top},
                 {workspace, N > 0 ? workspace_bytes : 0}, {targets, (size_t)N * index_type},
                 rows_range(h, h_stride, N, d, dtype), rows_range(w, w_stride, V, d, dtype)}, 6))
        return TXL_ERR_INVALID_ARG;
    if (N == 0) return TXL_OK;
    const StatsPlan s = plan_stats(N, V, d, dtype, top);
    if (!workspace || workspace_bytes < s.total) return TXL_ERR_WORKSPACE;
    if (!on(workspace, 256)) return TXL_ERR_MISALIGNED;
    cudaStream_t st = stream_of(stream);
    char *ws = static_cast<char *>(workspace);
    unsigned int *status = txl::device_status_word();
    if (!status) return TXL_ERR_CUDA;

    if (dtype == TXL_F32 &&
        txl::launch_split_f32(split_of(h, h_stride, N, d, ws + s.h_planes),
                              split_of(w, w_stride, V, d, ws + s.w_planes), st) != cudaSuccess)
        return TXL_ERR_CUDA;
    const Operand oh = operand(h, h_stride, ws + s.h_planes, N, d, dtype);
    const Operand ow = operand(w, w_stride, ws + s.w_planes, V, d, dtype);
    txl::GemmLaunch l{};
    if (!map_of(&l.maps[0].a, oh, N, d, s.few ? (unsigned)s.bn : 128u) ||
        !map_of(&l.maps[0].b, ow, V, d, s.few ? 128u : (unsigned)s.bn / 2))
        return TXL_ERR_CUDA;
    GemmParams &p = l.p[0];
    p.M = N;
    p.N = V;
    p.V = V;
    p.mb = s.mb;
    p.nb = s.nb;
    p.bn = s.bn;
    p.kb = ceil_div(d, 64);
    p.splits = s.splits;
    p.n_items = s.mb * s.splits;
    p.terms = oh.planes;
    p.a_rows = 128;
    p.status = status;
    p.wait_ns = txl::wait_limit_ns();
    p.targets = targets;
    p.index_bytes = index_type;
    p.scale = scale;
    p.stats = reinterpret_cast<float4 *>(ws + s.stats);
    p.list_val = reinterpret_cast<float *>(ws + s.val);
    p.list_id = reinterpret_cast<int *>(ws + s.id);
    p.group_key = top > 0 ? reinterpret_cast<unsigned *>(ws + s.keys) : nullptr;
    p.logits = s.full ? reinterpret_cast<float *>(ws + s.logits) : nullptr;
    p.target_z = reinterpret_cast<float *>(ws + s.target_z);
    if ((s.few ? txl::launch_logprob_few(l.maps[0].b, l.maps[0].a, p, st)
               : txl::launch_logprob_stats(l, s.list, st)) != cudaSuccess)
        return TXL_ERR_CUDA;

    txl::MergeParams m{};
    m.stats = p.stats;
    m.list_val = p.list_val;
    m.list_id = p.list_id;
    m.group_key = p.group_key;
    m.logits = p.logits;
    m.target_z = p.target_z;
    m.nb = s.nb;
    m.splits = s.few ? s.splits : 2 * s.splits;
    m.N = N;
    m.V = V;
    m.d = d;
    m.top = top;
    m.list = s.list;
    m.h = h;
    m.w = w;
    m.h_ld = h_stride;
    m.w_ld = w_stride;
    m.targets = targets;
    m.index_bytes = index_type;
    m.scale = scale;
    const double c = (double)scale * 1.4426950408889634;
    m.c_hi = (float)c;
    m.c_lo = (float)(c - (double)m.c_hi);
    m.logp = logp;
    m.lse = lse;
    m.entropy = entropy;
    m.top_logp = top_logp;
    m.top_ids = top_ids;
    m.status = status;
    return status_of(s.few ? txl::launch_logprob_few_merge(m, dtype == TXL_BF16, st)
                           : txl::launch_logprob_merge(m, dtype == TXL_BF16, st));
}

size_t txl_logprob_bwd_workspace_size(int N, int V, int d, int dtype, int grad_dtype)
{
    if (check_sizes(N, V, d, 8) != TXL_OK || check_type(dtype) != TXL_OK || check_type(grad_dtype) != TXL_OK)
        return 0;
    return N == 0 ? 0 : plan_grad(N, V, d, dtype, grad_dtype).total;
}

int txl_logprob_bwd(const void *h, long long h_stride, const void *w, long long w_stride,
                    const void *targets, int index_type, const float *lse, const float *entropy,
                    const float *dlogp, const float *dentropy, void *dh, void *dw, int N, int V,
                    int d, float scale, int dtype, int grad_dtype, void *workspace,
                    size_t workspace_bytes, void *stream)
{
    int rc;
    if ((rc = check_type(dtype)) != TXL_OK || (rc = check_type(grad_dtype)) != TXL_OK) return rc;
    if ((rc = check_sizes(N, V, d, 8)) != TXL_OK) return rc;
    if ((rc = check_ids(targets, index_type)) != TXL_OK) return rc;
    if (!w || (!dh && !dw) || (N > 0 && (!h || !lse)) || !std::isfinite(scale)) return TXL_ERR_INVALID_ARG;
    if ((targets == nullptr) != (dlogp == nullptr)) return TXL_ERR_INVALID_ARG;
    if (N > 0 && ((!dlogp && !dentropy) || (dentropy && !entropy))) return TXL_ERR_INVALID_ARG;
    if (dtype == TXL_F32 && grad_dtype != TXL_F32) return TXL_ERR_UNSUPPORTED;
    if (N > 0 && (rc = check_rows(h, h_stride, N, d, dtype)) != TXL_OK) return rc;
    if ((rc = check_rows(w, w_stride, V, d, dtype)) != TXL_OK) return rc;
    if (!on(dh, 16) || !on(dw, 16)) return TXL_ERR_MISALIGNED;
    for (const void *p : {(const void *)lse, (const void *)entropy, (const void *)dlogp, (const void *)dentropy})
        if (!on(p, 4)) return TXL_ERR_MISALIGNED;
    const size_t row4 = (size_t)N * 4;
    if (overlap({{dh, (size_t)N * d * elem(dtype)}, {dw, (size_t)V * d * elem(grad_dtype)},
                 {workspace, N > 0 ? workspace_bytes : 0}, {targets, (size_t)N * index_type},
                 rows_range(h, h_stride, N, d, dtype), rows_range(w, w_stride, V, d, dtype), {lse, row4},
                 {entropy, row4}, {dlogp, row4}, {dentropy, row4}}, 3))
        return TXL_ERR_INVALID_ARG;
    cudaStream_t st = stream_of(stream);
    if (N == 0)
        return dw ? status_of(cudaMemsetAsync(dw, 0, (size_t)V * d * elem(grad_dtype), st)) : TXL_OK;
    const GradPlan g = plan_grad(N, V, d, dtype, grad_dtype);
    if (!workspace || workspace_bytes < g.total) return TXL_ERR_WORKSPACE;
    if (!on(workspace, 256)) return TXL_ERR_MISALIGNED;
    char *ws = static_cast<char *>(workspace);
    unsigned int *status = txl::device_status_word();
    if (!status) return TXL_ERR_CUDA;

    // h without the rows that have no part, and the targets' log probabilities; fp32: both
    // operands' terms
    txl::GradRowsParams l{};
    l.h = h;
    l.w = w;
    l.out = reinterpret_cast<__nv_bfloat16 *>(ws + g.live);
    l.out_ld = line_ld(d);
    l.target_logp = reinterpret_cast<float *>(ws + g.target_logp);
    l.h_ld = h_stride;
    l.w_ld = w_stride;
    l.N = N;
    l.V = V;
    l.d = d;
    l.index_bytes = index_type;
    l.targets = targets;
    l.lse = lse;
    l.dentropy = dentropy;
    l.scale = scale;
    l.status = status;
    if (dtype == TXL_F32) l.table = split_of(w, w_stride, V, d, ws + g.w_planes);
    if (txl::launch_grad_rows(l, dtype == TXL_BF16, st) != cudaSuccess) return TXL_ERR_CUDA;
    const int h_terms = dtype == TXL_F32 ? txl::kMaxPieces : 1;
    const Operand oh = {ws + g.live, line_ld(d), h_terms, (long long)N * line_ld(d)};
    const Operand ow = operand(w, w_stride, ws + g.w_planes, V, d, dtype);

    GemmParams base{};
    base.status = status;
    base.wait_ns = txl::wait_limit_ns();
    base.V = V;
    base.scale = scale;
    base.targets = targets;
    base.index_bytes = index_type;
    base.lse = lse;
    base.entropy = entropy;
    base.target_logp = l.target_logp;
    base.dlogp = dlogp;
    base.dentropy = dentropy;
    base.g_pieces = g.pieces;
    txl::GemmLaunch grad{}, prod{};
    const unsigned rows_box = (unsigned)box_rows(N);
    if (!map_of(&grad.maps[0].a, oh, N, d, rows_box) ||
        !map_of(&grad.maps[0].b, ow, V, d, (unsigned)g.g.bn / 2) ||
        !map_of(&prod.maps[0].b, ow, V, d, 64) || !map_of(&prod.maps[1].b, oh, N, d, 64))
        return TXL_ERR_CUDA;
    const Operand og = {ws + g.g_at, g.g_ld, g.pieces, g.g_plane};
    for (int c = 0; c < g.chunks; ++c) {
        const int v0 = c * g.chunk, cols = std::min(g.chunk, V - v0);
        // G of the chunk
        GemmParams &p = grad.p[0];
        p = base;
        p.M = N;
        p.N = cols;
        p.mb = g.g.mb;
        p.bn = g.g.bn;
        p.nb = ceil_div(cols, p.bn);
        p.kb = ceil_div(d, 64);
        p.splits = 1;
        p.n_items = p.mb * p.nb;
        p.b_row0 = v0;
        p.terms = oh.planes;
        p.a_rows = box_rows(N);
        if (!map_of(&grad.maps[0].out, og, N, cols, 32) || !map_of(&prod.maps[0].a, og, N, cols, g.stacked ? rows_box : 128))
            return TXL_ERR_CUDA;
        if (txl::launch_logprob_grad(grad, st) != cudaSuccess) return TXL_ERR_CUDA;
        prod.p[0] = prod.p[1] = base;
        txl::PartsSum sums[2] = {};
        if (dh) {
            GemmParams &q = prod.p[0];
            q.M = N;
            q.N = d;
            q.mb = g.h.mb;
            q.nb = g.h.nb;
            q.bn = g.h.bn;
            q.kb = ceil_div(cols, 64);
            q.splits = g.h.parts;
            q.n_items = q.mb * q.nb * q.splits;
            q.b_row0 = v0;
            q.part = g.parts_h > 1 || g.chunks > 1;
            q.out_bf16 = dtype == TXL_BF16;
            q.stacked = g.stacked;
            q.terms = q.stacked ? 1 : g.pieces_h;
            q.a_rows = q.stacked ? box_rows(N) : 128;
            float *so_far = reinterpret_cast<float *>(ws + g.part_h);
            float *parts = so_far + (g.chunks > 1 ? (long long)N * d : 0);
            if (!map_out(&prod.maps[0].out, q, q.part ? reinterpret_cast<char *>(parts) : (char *)dh))
                return TXL_ERR_CUDA;
            // the chunks' sums in their order, the last one's to dh
            const bool last = c + 1 == g.chunks;
            if (q.part)
                sums[0] = {c > 0 ? so_far : parts, last ? dh : so_far, (long long)N * d, g.parts_h + (c > 0),
                           last && dtype == TXL_BF16};
        }
        if (dw) {
            char *rows = static_cast<char *>(dw) + (size_t)v0 * d * elem(grad_dtype);
            GemmParams &q = prod.p[1];
            q.M = cols;
            q.N = d;
            q.mb = ceil_div(cols, 256);
            q.nb = g.w.nb;
            q.bn = g.w.bn;
            q.kb = ceil_div(N, 64);
            q.splits = g.w.parts;
            q.n_items = q.mb * q.nb * q.splits;
            q.part = g.w.parts > 1;
            q.out_bf16 = grad_dtype == TXL_BF16;
            q.twice = g.stacked;
            q.terms = g.stacked ? 1 : g.pieces;
            q.a_rows = 128;
            if (!map_of(&prod.maps[1].a, og, N, cols, 64) ||
                !map_out(&prod.maps[1].out, q, q.part ? ws + g.part_w : rows))
                return TXL_ERR_CUDA;
            if (q.part)
                sums[1] = {reinterpret_cast<float *>(ws + g.part_w), rows, (long long)cols * d, g.w.parts,
                           grad_dtype == TXL_BF16};
        }
        const GemmParams &q0 = prod.p[0], &q1 = prod.p[1];
        prod.early = 0;
        if (dh && dw)
            prod.early = take_turns(q0.n_items, item_cycles(ceil_div(q0.kb, q0.splits), q0.bn, q0.terms, q0.a_rows), q1.n_items,
                                    item_cycles(ceil_div(q1.kb << q1.twice, q1.splits), q1.bn, q1.terms)).early;
        if (txl::launch_products(prod, st) != cudaSuccess) return TXL_ERR_CUDA;
        if (txl::launch_sum_parts(sums, st) != cudaSuccess) return TXL_ERR_CUDA;
    }
    return TXL_OK;
}

} // extern "C"
