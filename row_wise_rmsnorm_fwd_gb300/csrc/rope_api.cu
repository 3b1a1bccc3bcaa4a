// rope_api.cu -- C ABI of rotary positions with head norms (include/rmsnorm_rope.h):
// the frequencies, validation, kernel choice and launch.  Shares the library's per-device
// state (device.h) and status conventions with the other entry points.
#include "rmsnorm_rope.h"
#include "checks.h"
#include "device.h"
#include "rope_launch.h"

#include <cfloat>
#include <cmath>
#include <cstring>

namespace rmsnorm {
namespace {

// ---------------------------------------------------------------- frequencies --

// Numbers as sums of two long doubles, the second at most half a last place of the first: one
// long double (64 bits here or 113, by machine) rounds a frequency before its last of 64 bits
// behind the point is known.  Sums and products are off by a few 2^-2p of themselves, p bits.
static_assert(LDBL_MANT_DIG >= 64, "two of them have 128 bits");

struct Two {
    long double hi, lo;
};

Two normal(long double a, long double b) {          // |a| >= |b|
    const long double s = a + b;
    return {s, b - (s - a)};
}

Two operator+(Two a, Two b) {
    const long double s = a.hi + b.hi, t = s - a.hi;
    return normal(s, (a.hi - (s - t)) + (b.hi - t) + (a.lo + b.lo));
}

Two operator-(Two a) { return {-a.hi, -a.lo}; }

Two operator*(Two a, Two b) {
    const long double p = a.hi * b.hi;
    return normal(p, fmal(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}

Two two(long double v) { return {v, 0.0L}; }

Two operator/(Two a, Two b) {                       // a quotient, and that of what it leaves
    const long double q = a.hi / b.hi;
    return normal(q, (a + -(two(q) * b)).hi / b.hi);
}

// 2 pi to 163 bits, 32 or 35 at a time.
Two two_pi() {
    return (((two(0x6.487ED511p0L) + two(0x0B4611A6p-64L)) + two(0x2633145Cp-96L)) + two(0x06E0E689p-128L)) +
           two(0x48127044p-160L);
}

Two power(Two v, int n) {
    Two r = two(1.0L);
    for (; n > 0; n >>= 1, v = v * v)
        if (n & 1) r = r * v;
    return r;
}

// The n-th root of v >= 1: one step of Newton's method, which doubles powl's bits.
Two root(double v, int n) {
    const Two y = two(powl(v, 1.0L / n)), below = power(y, n - 1);
    return y + -((below * y + two(-static_cast<long double>(v))) / (two(n) * below));
}

// The nearest multiple of 2^-64 to v >= 0, in those units modulo 2^64.
uint64_t turns_of(Two v) {
    const long double part = (v.hi - floorl(v.hi)) * 0x1p64L, whole = floorl(part);
    long double rest = roundl((part - whole) + (v.lo - roundl(v.lo)) * 0x1p64L);
    if (rest >= 0x1p63L) rest -= 0x1p64L;
    return static_cast<uint64_t>(whole) + static_cast<uint64_t>(static_cast<int64_t>(rest));
}

bool positive(double v) { return std::isfinite(v) && v > 0.0; }

rmsnorm_status_t freqs_of(const rmsnorm_rope_rule_t* r, uint64_t* freqs, float* mscale) {
    if (!r || !freqs || !mscale) return RMSNORM_ERR_INVALID_ARG;
    if (r->rot_dim < 2 || r->rot_dim % 2 || r->rot_dim > kRopeMaxDim || !std::isfinite(r->base) ||
        !(r->base > 1.0) || r->scaling < RMSNORM_ROPE_NONE || r->scaling > RMSNORM_ROPE_BANDS)
        return RMSNORM_ERR_INVALID_ARG;
    const bool turns = r->scaling == RMSNORM_ROPE_RAMP || r->scaling == RMSNORM_ROPE_BANDS;
    if (r->scaling != RMSNORM_ROPE_NONE && !(std::isfinite(r->factor) && r->factor >= 1.0))
        return RMSNORM_ERR_INVALID_ARG;
    if (turns && !(positive(r->low) && positive(r->high) && r->low < r->high && r->original_len >= 1))
        return RMSNORM_ERR_INVALID_ARG;
    if (r->scaling == RMSNORM_ROPE_BASE && r->rot_dim < 4) return RMSNORM_ERR_INVALID_ARG;
    const int half = r->rot_dim / 2;
    if (r->divisors) {
        for (int i = 0; i < half; ++i)
            if (!positive(r->divisors[i])) return RMSNORM_ERR_INVALID_ARG;
    }
    const Two one = two(1.0L), circle = two_pi();
    long double first = 0.0L, last = 0.0L;
    if (r->scaling == RMSNORM_ROPE_RAMP) {
        // the pair that makes t turns: len * base^(-2i / dim) / (2 pi) = t
        const long double len = r->original_len, log_base = logl(r->base);
        auto pair = [&](long double t) { return half * logl(len / (t * circle.hi)) / log_base; };
        first = fmaxl(floorl(pair(r->high)), 0.0L);
        last = fminl(ceill(pair(r->low)), r->rot_dim - 1.0L);
    }
    // each frequency from the one before it, down by base^(1 / half); with a raised base, base *
    // factor^(half / (half - 1)), by factor^(1 / (half - 1)) more
    Two step = root(r->base, half);
    if (r->scaling == RMSNORM_ROPE_BASE) step = step * root(r->factor, half - 1);
    step = one / step;
    const bool part = r->scaling != RMSNORM_ROPE_NONE && r->scaling != RMSNORM_ROPE_BASE;
    const Two divided = part ? one / two(r->factor) : one;
    const Two low = two(-static_cast<long double>(r->low)), len = two(r->original_len);
    const Two per_turn = turns ? one / (two(r->high) + low) : one;
    const Two per_pair = one / two(fmaxl(last - first, 0.001L));
    Two plain = one / circle;                                   // turns per position, not scaled
    for (int i = 0; i < half; ++i, plain = plain * step) {
        Two f = plain;
        if (part) {
            Two kept = two(0.0L);
            if (r->scaling == RMSNORM_ROPE_RAMP) kept = one + -(two(i - first) * per_pair);
            if (r->scaling == RMSNORM_ROPE_BANDS) kept = (len * f + low) * per_turn;
            if (kept.hi <= 0.0L) f = f * divided;
            else if (kept.hi < 1.0L) f = f * (kept + (one + -kept) * divided);
        }
        if (r->divisors) f = f / two(r->divisors[i]);
        freqs[i] = turns_of(f);
    }
    *mscale = r->scaling == RMSNORM_ROPE_RAMP
                  ? static_cast<float>(0.1L * logl(r->factor) + 1.0L) : 1.0f;
    return RMSNORM_OK;
}

// ---------------------------------------------------------------------- checks --

constexpr int64_t kMaxItems = 1ll << 40;
constexpr int64_t kAngleRounds = 2;     // rounds of heads that a token's angles cost

struct RopeCall {
    int dtype = 0;
    int sz = 0;
    int64_t batch = 0;
    RopeParams p;
    int32_t path = RMSNORM_PATH_AUTO;
    DeviceView dv;
};

// A view with its sizes: dims batch, token, head; the innermost is head_dim elements.
struct Box {
    uintptr_t p;
    int64_t n[3], stride[3];
    int64_t dim;
    int64_t extent;            // elements from its first to behind its last
};

// false: strides out of range.
bool box_of(const void* p, const int64_t (&stride)[3], int64_t batch, int64_t seq, int64_t heads,
            int64_t dim, Box* b) {
    b->p = reinterpret_cast<uintptr_t>(p);
    const int64_t n[3] = {batch, seq, heads};
    b->dim = dim;
    b->extent = dim;
    for (int k = 0; k < 3; ++k) {
        b->n[k] = n[k];
        b->stride[k] = stride[k];
        int64_t far;
        if (stride[k] < 0 || __builtin_mul_overflow(n[k] - 1, stride[k], &far) ||
            __builtin_add_overflow(b->extent, far, &b->extent) || b->extent > (INT64_MAX >> 4))
            return false;
    }
    return true;
}

// Whether no two elements of the view share an address: from the smallest stride on, each
// is at least as large as all that lies within it.
bool distinct(const Box& b) {
    bool done[3] = {b.n[0] == 1, b.n[1] == 1, b.n[2] == 1};
    int64_t within = b.dim;
    for (;;) {
        int k = -1;
        for (int i = 0; i < 3; ++i)
            if (!done[i] && (k < 0 || b.stride[i] < b.stride[k])) k = i;
        if (k < 0) return true;
        if (b.stride[k] < within) return false;
        within += (b.n[k] - 1) * b.stride[k];
        done[k] = true;
    }
}

bool same_place(const Box& a, const Box& b) {
    if (a.p != b.p) return false;
    for (int k = 0; k < 3; ++k)
        if (a.n[k] != b.n[k] || (a.n[k] > 1 && a.stride[k] != b.stride[k])) return false;
    return true;
}

// Extent of a view modulo m: strides that are multiples of m do not count.  -1: it does not
// fit within m.
int64_t extent_modulo(const Box& b, int64_t m) {
    int64_t e = b.dim;
    for (int k = 0; k < 3; ++k)
        if (b.n[k] > 1 && b.stride[k] % m) e += (b.n[k] - 1) * b.stride[k];
    return e <= m ? e : -1;
}

// Whether two views are shown to share no address: their address ranges are apart, or,
// modulo some stride, the ranges that they take are (two groups of heads side by side
// in each token of one array, say).
bool apart(const Box& a, const Box& b, int sz) {
    if (!a.p || !b.p) return true;
    if (a.p + static_cast<uint64_t>(a.extent) * sz <= b.p || b.p + static_cast<uint64_t>(b.extent) * sz <= a.p)
        return true;
    for (int k = 0; k < 3; ++k) {
        const int64_t m = a.stride[k];
        if (a.n[k] == 1 || m <= 0) continue;
        const int64_t ea = extent_modulo(a, m), eb = extent_modulo(b, m);
        if (ea < 0 || eb < 0) continue;
        const int64_t d = static_cast<int64_t>(b.p / sz) - static_cast<int64_t>(a.p / sz);
        const int64_t at = (d % m + m) % m;
        if (at >= ea && at + eb <= m) return true;
    }
    return false;
}

bool apart(const Box& a, const Span& s, int sz) {
    return !overlaps(Span{a.p, static_cast<uint64_t>(a.extent) * sz}, s);
}

RopeView view_of(const void* p, const int64_t (&stride)[3]) {
    return RopeView{const_cast<void*>(p), stride[0], stride[1], stride[2]};
}

rmsnorm_status_t check_options(const rmsnorm_options_t* opt, RopeCall* c) {
    if (!opt) return RMSNORM_OK;
    const rmsnorm_options_t& o = *opt;
    if (o.cluster || o.threads || o.grid || o.vec_bytes || o.chunk_bytes || o.stages || o.weights ||
        o.reserved || o.epilogue || o.fault_inject)
        return RMSNORM_ERR_INVALID_ARG;
    if (o.path != RMSNORM_PATH_AUTO && o.path != RMSNORM_PATH_TWOPASS) return RMSNORM_ERR_INVALID_ARG;
    c->path = o.path;
    return RMSNORM_OK;
}

// Sizes, the rule and the views.  back: dy is turned, x is read with the norm only.
rmsnorm_status_t check_call(int32_t dtype, const rmsnorm_rope_heads_t* q, const rmsnorm_rope_heads_t* k,
                            int64_t batch, int64_t seq, int64_t dim, const rmsnorm_rope_t* r, bool back,
                            const void* workspace, uint64_t workspace_bytes,
                            const rmsnorm_options_t* opt, RopeCall* c) {
    if (dtype != RMSNORM_DTYPE_F32 && dtype != RMSNORM_DTYPE_BF16) return RMSNORM_ERR_INVALID_ARG;
    if (!q || !r || batch < 0 || seq < 0 || dim < 2 || dim > kRopeMaxDim) return RMSNORM_ERR_INVALID_ARG;
    std::memset(&c->p, 0, sizeof(c->p));
    c->dtype = dtype;
    c->sz = dtype == RMSNORM_DTYPE_F32 ? 4 : 2;
    c->batch = batch;
    RopeParams& p = c->p;
    if (r->rot_dim < 2 || r->rot_dim % 2 || r->rot_dim > dim || r->norm < 0 || r->norm > 1 ||
        r->interleaved < 0 || r->interleaved > 1 || !std::isfinite(r->mscale) || !std::isfinite(r->eps) ||
        r->eps < 0.f || !r->freqs || !aligned(r->freqs, 8))
        return RMSNORM_ERR_INVALID_ARG;
    if (r->positions && ((r->position_bytes != 4 && r->position_bytes != 8) || r->n_positions < 1 ||
                         r->n_positions > (INT64_MAX >> 4) ||
                         !aligned(r->positions, static_cast<uintptr_t>(r->position_bytes))))
        return RMSNORM_ERR_INVALID_ARG;
    const int64_t heads_q = q->heads, heads_k = k ? k->heads : 0;
    if (heads_q < 1 || heads_q > INT32_MAX / 2 || (k && heads_k < 1) || heads_k > INT32_MAX / 2)
        return RMSNORM_ERR_INVALID_ARG;
    int64_t items;
    if (__builtin_mul_overflow(batch, seq, &items) || __builtin_mul_overflow(items, heads_q + heads_k, &items) ||
        items > kMaxItems)
        return RMSNORM_ERR_INVALID_ARG;
    const rmsnorm_status_t st = check_options(opt, c);
    if (st != RMSNORM_OK) return st;
    p.tokens = batch * seq;
    p.seq = seq;
    p.freqs = r->freqs;
    p.positions = r->positions;
    p.n_positions = r->n_positions;
    p.start = r->start;
    p.wide = r->position_bytes == 8;
    p.dim = static_cast<int32_t>(dim);
    p.rot = r->rot_dim;
    p.norm = r->norm;
    p.inv_dim = 1.0f / static_cast<float>(dim);
    p.eps = r->eps;
    p.mscale = r->mscale;
    const uintptr_t sz = static_cast<uintptr_t>(c->sz);
    const int64_t b1 = batch > 0 ? batch : 1, s1 = seq > 0 ? seq : 1;
    const uint64_t row = static_cast<uint64_t>(dim) * sz;
    Box in[4], out[2];                          // x of q and k, dy of q and k
    std::memset(in, 0, sizeof(in));
    std::memset(out, 0, sizeof(out));
    Span small[7] = {span(r->freqs, static_cast<uint64_t>(r->rot_dim) * 4),
                     r->positions ? span(r->positions, static_cast<uint64_t>(r->n_positions) * r->position_bytes)
                                  : Span{0, 0},
                     {0, 0}, {0, 0}, {0, 0}, {0, 0}, span(workspace, workspace_bytes)};
    const rmsnorm_rope_heads_t* both[2] = {q, k};
    for (int i = 0; i < 2; ++i) {
        const rmsnorm_rope_heads_t* t = both[i];
        if (!t) continue;
        const bool with_x = !back || r->norm;
        if (!t->out || (with_x && !t->x) || (back && !t->dy)) return RMSNORM_ERR_INVALID_ARG;
        if (t->dw && !(back && r->norm)) return RMSNORM_ERR_INVALID_ARG;
        if (!aligned(t->out, sz) || (with_x && !aligned(t->x, sz)) || (back && !aligned(t->dy, sz)) ||
            !aligned(t->w, sz) || !aligned(t->dw, 4))
            return RMSNORM_ERR_INVALID_ARG;
        if ((with_x && !box_of(t->x, t->x_stride, b1, s1, t->heads, dim, &in[i])) ||
            (back && !box_of(t->dy, t->dy_stride, b1, s1, t->heads, dim, &in[2 + i])) ||
            !box_of(t->out, t->out_stride, b1, s1, t->heads, dim, &out[i]) || !distinct(out[i]))
            return RMSNORM_ERR_INVALID_ARG;
        if (r->norm) small[2 + i] = span(t->w, row);
        small[4 + i] = span(t->dw, static_cast<uint64_t>(dim) * 4);
        RopeHeads& h = p.t[i];
        if (with_x) h.x = view_of(t->x, t->x_stride);
        if (back) h.dy = view_of(t->dy, t->dy_stride);
        h.out = view_of(t->out, t->out_stride);
        h.w = r->norm ? t->w : nullptr;
        h.dw = t->dw;
        h.heads = static_cast<int32_t>(t->heads);
    }
    if (p.tokens == 0) return RMSNORM_OK;        // nothing is read or written but dw
    for (int i = 0; i < 2; ++i) {
        if (!out[i].p) continue;
        for (int j = 0; j < 4; ++j)
            if (!(j % 2 == i && same_place(out[i], in[j])) && !apart(out[i], in[j], c->sz))
                return RMSNORM_ERR_INVALID_ARG;
        for (const Span& s : small)
            if (!apart(out[i], s, c->sz)) return RMSNORM_ERR_INVALID_ARG;
    }
    if (!apart(out[0], out[1], c->sz)) return RMSNORM_ERR_INVALID_ARG;
    for (int i = 4; i < 7; ++i) {                // dw and the workspace against what is read
        if (clashes(small[i], small, i, 0)) return RMSNORM_ERR_INVALID_ARG;
        for (const Box& b : in)
            if (b.p && !apart(b, small[i], c->sz)) return RMSNORM_ERR_INVALID_ARG;
    }
    return RMSNORM_OK;
}

rmsnorm_status_t launch(const RopeCall& c, RopeFn fn, const LaunchShape& s, cudaStream_t stream) {
    return note(launch_ex(fn, s, stream, c.p)) == cudaSuccess ? RMSNORM_OK : RMSNORM_ERR_CUDA;
}

// CTAs of the any kernel, and of the vector kernel, at most: what a workspace has parts for.
int64_t any_ctas(const DeviceView& dv, int64_t items) {
    const int64_t ctas = div_up(items, kRopeAnyWarps), most = 8ll * dv.sms;
    return ctas < most ? ctas : most;
}
constexpr int64_t kVecCtasPerSm = 8;

rmsnorm_status_t launch_any(RopeCall* c, bool interleaved, bool back, cudaStream_t stream) {
    RopeParams& p = c->p;
    const int ctas = static_cast<int>(any_ctas(c->dv, p.tokens * (p.t[0].heads + p.t[1].heads)));
    p.part_stride = 2 * p.dim;
    p.part_at[1] = p.dim;
    p.part_n[0] = p.part_n[1] = ctas;
    const LaunchShape s{ctas, 32 * kRopeAnyWarps, 1, 0};
    return launch(*c, rope_any_ptr(c->dtype, interleaved, back), s, stream);
}

// Widest vector that the views, the head and its turned part (whole units) allow.
int vec_bytes(const RopeCall& c, bool back) {
    const RopeParams& p = c.p;
    const uint64_t sz = static_cast<uint64_t>(c.sz);
    uint64_t bits = static_cast<uint64_t>(p.dim | (p.rot / 2)) * sz;
    for (const RopeHeads& t : p.t) {
        bits |= reinterpret_cast<uintptr_t>(t.w);
        const RopeView* views[] = {&t.x, &t.out, &t.dy};
        for (int i = 0; i < (back ? 3 : 2); ++i) {
            bits |= reinterpret_cast<uintptr_t>(views[i]->p);
            // a dim of one element has a stride that is not used
            if (c.batch > 1) bits |= static_cast<uint64_t>(views[i]->batch) * sz;
            if (p.seq > 1) bits |= static_cast<uint64_t>(views[i]->token) * sz;
            if (t.heads > 1) bits |= static_cast<uint64_t>(views[i]->head) * sz;
        }
    }
    int v = 16;
    while (v > c.sz && bits % v) v >>= 1;
    return v;
}

int pow2_ceil(int v) {
    int p = 1;
    while (p < v) p <<= 1;
    return p;
}

// Heads in vectors; *done stays false where a head has more than 32 units.
rmsnorm_status_t launch_vec(RopeCall* c, bool interleaved, int kind, bool* done, cudaStream_t stream) {
    RopeParams& p = c->p;
    const int vb = vec_bytes(*c, kind != kRopeTurn);
    const int epv = vb / c->sz;
    p.units = static_cast<int32_t>(div_up(p.dim / epv, 2));
    if (p.units > 32) return RMSNORM_OK;
    p.lanes = pow2_ceil(p.units);
    const int whole = p.lanes == p.units && p.dim / epv == 2 * p.units ? p.lanes : 0;
    RopeFn fn;
    if (c->dtype == RMSNORM_DTYPE_F32)
        fn = kind == kRopeTurn ? rope_vec_f32_turn(vb, interleaved, whole)
             : kind == kRopeTurnBack ? rope_vec_f32_back(vb, interleaved, whole)
                                     : rope_vec_f32_grad(vb, interleaved, whole);
    else
        fn = kind == kRopeTurn ? rope_vec_bf16_turn(vb, interleaved, whole)
             : kind == kRopeTurnBack ? rope_vec_bf16_back(vb, interleaved, whole)
                                     : rope_vec_bf16_grad(vb, interleaved, whole);
    int occ = 0;
    if (cached_occupancy(c->dv.dev, c->dv.smem_optin, reinterpret_cast<KernelFn>(fn), 32 * kRopeVecWarps, 0,
                         1, &occ) != cudaSuccess)
        return RMSNORM_ERR_CUDA;
    const int64_t most = c->dv.sms * (occ < kVecCtasPerSm ? occ : kVecCtasPerSm);
    // A token's heads are shared by as many warps as it takes to have a warp for each of
    // the GPU's warp slots, of one round of heads at least; fewer heads than a warp has lane
    // groups leave groups for other tokens.
    const int groups = 32 / p.lanes;
    int64_t want[2] = {0, 0}, cost[2] = {0, 0};
    for (int i = 0; i < 2; ++i) {
        p.split[i] = p.share[i] = 1;
        if (!p.t[i].heads) continue;
        const int64_t share = pow2_ceil(p.t[i].heads < groups ? p.t[i].heads : groups);
        const int64_t places = div_up(p.tokens, groups / share);
        const int64_t rounds = div_up(p.t[i].heads, share);
        int64_t split = div_up(most * kRopeVecWarps, places);
        if (split > rounds) split = rounds;
        p.split[i] = static_cast<int32_t>(split);
        p.share[i] = static_cast<int32_t>(share);
        want[i] = div_up(places * split, kRopeVecWarps);
        // what a token's heads cost, and its angles
        cost[i] = (rounds + kAngleRounds) * share;
    }
    int64_t q = want[0], k = want[1];
    if (q + k > most) {           // shares of what they cost
        q = most * cost[0] / (cost[0] + cost[1]);
        if (q < 1) q = 1;
        if (q > want[0]) q = want[0];
        k = most - q;
        if (k > want[1]) {
            k = want[1];
            q = most - k < want[0] ? most - k : want[0];
        }
        if (want[1] && k < 1) {
            k = 1;
            q = most - 1;
        }
    }
    p.q_ctas = static_cast<int32_t>(q);
    p.part_stride = p.dim;
    p.part_at[1] = q * p.dim;
    p.part_n[0] = static_cast<int32_t>(q);
    p.part_n[1] = static_cast<int32_t>(k);
    *done = true;
    const LaunchShape s{static_cast<int>(q + k), 32 * kRopeVecWarps, 1, 0};
    return launch(*c, fn, s, stream);
}

rmsnorm_status_t launch_rope(RopeCall* c, bool interleaved, int kind, cudaStream_t stream) {
    if (c->path != RMSNORM_PATH_TWOPASS) {
        bool done = false;
        const rmsnorm_status_t st = launch_vec(c, interleaved, kind, &done, stream);
        if (st != RMSNORM_OK || done) return st;
    }
    return launch_any(c, interleaved, kind != kRopeTurn, stream);
}

rmsnorm_status_t fwd_run(int32_t dtype, const rmsnorm_rope_heads_t* q, const rmsnorm_rope_heads_t* k,
                         int64_t batch, int64_t seq, int64_t dim, const rmsnorm_rope_t* r,
                         const rmsnorm_options_t* opt, cudaStream_t stream) {
    RopeCall c;
    const rmsnorm_status_t st = check_call(dtype, q, k, batch, seq, dim, r, false, nullptr, 0, opt, &c);
    if (st != RMSNORM_OK || c.p.tokens == 0) return st;
    if (current_device(&c.dv) != cudaSuccess) return RMSNORM_ERR_CUDA;
    return launch_rope(&c, r->interleaved != 0, kRopeTurn, stream);
}

rmsnorm_status_t bwd_workspace(int32_t dtype, int64_t batch, int64_t seq, int64_t heads, int64_t dim,
                               size_t* bytes) {
    if ((dtype != RMSNORM_DTYPE_F32 && dtype != RMSNORM_DTYPE_BF16) || !bytes || batch < 0 || seq < 0 ||
        heads < 1 || dim < 2 || dim > kRopeMaxDim)
        return RMSNORM_ERR_INVALID_ARG;
    int64_t items;
    if (__builtin_mul_overflow(batch, seq, &items) || __builtin_mul_overflow(items, heads, &items) ||
        items > kMaxItems)
        return RMSNORM_ERR_INVALID_ARG;
    *bytes = 0;
    if (items == 0) return RMSNORM_OK;
    DeviceView dv;
    if (current_device(&dv) != cudaSuccess) return RMSNORM_ERR_CUDA;
    // the any kernel has rows for q and k in each part, the vector kernel one
    const int64_t any = 2 * any_ctas(dv, items), vec = kVecCtasPerSm * dv.sms;
    *bytes = static_cast<size_t>(any > vec ? any : vec) * dim * 4;
    return RMSNORM_OK;
}

rmsnorm_status_t bwd_run(int32_t dtype, const rmsnorm_rope_heads_t* q, const rmsnorm_rope_heads_t* k,
                         int64_t batch, int64_t seq, int64_t dim, const rmsnorm_rope_t* r,
                         void* workspace, size_t workspace_bytes, const rmsnorm_options_t* opt,
                         cudaStream_t stream) {
    RopeCall c;
    rmsnorm_status_t st = check_call(dtype, q, k, batch, seq, dim, r, true, workspace, workspace_bytes,
                                     opt, &c);
    if (st != RMSNORM_OK) return st;
    if (!aligned(workspace, 16)) return RMSNORM_ERR_INVALID_ARG;
    const bool sums = c.p.t[0].dw || c.p.t[1].dw;
    if (c.p.tokens == 0) {
        for (const RopeHeads& t : c.p.t)
            if (t.dw && note(cudaMemsetAsync(t.dw, 0, static_cast<size_t>(dim) * 4, stream)) != cudaSuccess)
                return RMSNORM_ERR_CUDA;
        return RMSNORM_OK;
    }
    if (sums && !workspace) return RMSNORM_ERR_INVALID_ARG;
    if (current_device(&c.dv) != cudaSuccess) return RMSNORM_ERR_CUDA;
    if (sums) {
        size_t need = 0;
        st = bwd_workspace(dtype, batch, seq, c.p.t[0].heads + c.p.t[1].heads, dim, &need);
        if (st != RMSNORM_OK) return st;
        if (workspace_bytes < need) return RMSNORM_ERR_INVALID_ARG;
        c.p.part = static_cast<float*>(workspace);
    }
    st = launch_rope(&c, r->interleaved != 0, r->norm ? kRopeGrad : kRopeTurnBack, stream);
    if (st != RMSNORM_OK || !sums) return st;
    LaunchShape s{static_cast<int>(div_up(dim, 32)), kRopeReduceThreads, 1, 0};
    s.grid_y = 2;
    return launch(c, rope_reduce_ptr(), s, stream);
}

}  // namespace
}  // namespace rmsnorm

using namespace rmsnorm;

extern "C" {

rmsnorm_status_t rmsnorm_rope_freqs(const rmsnorm_rope_rule_t* rule, uint64_t* freqs, float* mscale) {
    return freqs_of(rule, freqs, mscale);
}

rmsnorm_status_t rmsnorm_rope_fwd_f32(const rmsnorm_rope_heads_t* q, const rmsnorm_rope_heads_t* k,
                                      int64_t batch, int64_t seq, int64_t head_dim,
                                      const rmsnorm_rope_t* rope, rmsnorm_stream_t stream) {
    return fwd_run(RMSNORM_DTYPE_F32, q, k, batch, seq, head_dim, rope, nullptr,
                   reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t rmsnorm_rope_fwd_bf16(const rmsnorm_rope_heads_t* q, const rmsnorm_rope_heads_t* k,
                                       int64_t batch, int64_t seq, int64_t head_dim,
                                       const rmsnorm_rope_t* rope, rmsnorm_stream_t stream) {
    return fwd_run(RMSNORM_DTYPE_BF16, q, k, batch, seq, head_dim, rope, nullptr,
                   reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t rmsnorm_rope_fwd_ex(int32_t dtype, const rmsnorm_rope_heads_t* q,
                                     const rmsnorm_rope_heads_t* k, int64_t batch, int64_t seq,
                                     int64_t head_dim, const rmsnorm_rope_t* rope,
                                     const rmsnorm_options_t* opt, rmsnorm_stream_t stream) {
    return fwd_run(dtype, q, k, batch, seq, head_dim, rope, opt, reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t rmsnorm_rope_bwd_workspace(int32_t dtype, int64_t batch, int64_t seq, int64_t heads,
                                            int64_t head_dim, size_t* bytes) {
    return bwd_workspace(dtype, batch, seq, heads, head_dim, bytes);
}

rmsnorm_status_t rmsnorm_rope_bwd_f32(const rmsnorm_rope_heads_t* q, const rmsnorm_rope_heads_t* k,
                                      int64_t batch, int64_t seq, int64_t head_dim,
                                      const rmsnorm_rope_t* rope, void* workspace,
                                      size_t workspace_bytes, rmsnorm_stream_t stream) {
    return bwd_run(RMSNORM_DTYPE_F32, q, k, batch, seq, head_dim, rope, workspace, workspace_bytes,
                   nullptr, reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t rmsnorm_rope_bwd_bf16(const rmsnorm_rope_heads_t* q, const rmsnorm_rope_heads_t* k,
                                       int64_t batch, int64_t seq, int64_t head_dim,
                                       const rmsnorm_rope_t* rope, void* workspace,
                                       size_t workspace_bytes, rmsnorm_stream_t stream) {
    return bwd_run(RMSNORM_DTYPE_BF16, q, k, batch, seq, head_dim, rope, workspace, workspace_bytes,
                   nullptr, reinterpret_cast<cudaStream_t>(stream));
}

rmsnorm_status_t rmsnorm_rope_bwd_ex(int32_t dtype, const rmsnorm_rope_heads_t* q,
                                     const rmsnorm_rope_heads_t* k, int64_t batch, int64_t seq,
                                     int64_t head_dim, const rmsnorm_rope_t* rope, void* workspace,
                                     size_t workspace_bytes, const rmsnorm_options_t* opt,
                                     rmsnorm_stream_t stream) {
    return bwd_run(dtype, q, k, batch, seq, head_dim, rope, workspace, workspace_bytes, opt,
                   reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
