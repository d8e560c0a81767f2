// distill_kernels.hip -- distillation from a teacher's top logits over rows of
// logits, forward and backward.
#include "token_loss_device.h"

namespace zero {
namespace {

using namespace dev;

// What a row's teacher record comes to, as one wave leaves it in LDS.  Entry k
// is lane k % 64's.  The teacher's probabilities are binary64: 1 - sum q would
// lose the rest's digits in binary32.
struct Teacher {
    double q[ZERO_MAX_TOP];
    double token_q[ZERO_MAX_TOP];   // the token's probability over all entries that name it
    double total, rest;             // sum of q and rest; the other tokens' probability
    double cross;                   // sum of q (ln q - scale (logit - listed_max))
    int index[ZERO_MAX_TOP];        // the token; -1: no token of the vocabulary
    int lead[ZERO_MAX_TOP];         // the token where this is the first entry that names it, else -1
    float value[ZERO_MAX_TOP];
    float logit[ZERO_MAX_TOP];      // the student's
    float listed_max, listed_sum;   // of the listed tokens, each once
    float max, log2z;               // of the row: largest logit, binary logarithm of the sum
    int bad;                        // an entry outside the vocabulary or with a NaN value
};

// The backward pass's share of it.
struct Listed {
    double q[ZERO_MAX_TOP];
    int index[ZERO_MAX_TOP];
    float logit[ZERO_MAX_TOP];
    bool twice;
};

// Orders a wave's LDS writes before its lanes' later reads.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
__device__ __forceinline__ int wave_count(int x)
{
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        x += __shfl_xor(x, o, kWave);
    return x;
}

// exp(x) in binary64, to about 1e-11: 2^n times the 16th power of a Taylor sum
// of exp(z), |z| <= ln2 / 32 (the first term left out is below 2e-13).  Few
// constants: the library's takes more registers than a wave that holds a row can
// spare.
__device__ __forceinline__ double exp64(double x)
{
    const double y = x * 1.4426950408889634074;
    if (!(y > -1000.0))
        return x != x ? x : 0.0;
    const double n = __builtin_rint(y), z = (y - n) * (0.69314718055994530942 / 16);
    double p = 1.0 + z * (1.0 + z * (1.0 / 2 + z * (1.0 / 6 + z * (1.0 / 24 + z * (1.0 / 120)))));
#pragma unroll
    for (int i = 0; i < 4; ++i)
        p = p * p;
    return __builtin_ldexp(p, (int)fmin(n, 2000.0));
}
// ln(x), x > 0: binary32's, then one Newton step (the error is squared).
__device__ __forceinline__ double log64(double x)
{
    const double l = (double)log2f((float)x) * 0.69314718055994530942;
    return l + (x * exp64(-l) - 1.0);
}

// Below this the rest's probability is the rounding of the listed ones: binary32
// log probabilities v put at most |v| 2^-24 into each exp(v), and sum q |v| is
// an entropy, below 16 nats for any vocabulary here.
constexpr double kLeastRest = 0x1p-20;

// True where a record is padding: no entry, and no NaN value (whole waves).  Most
// records name a token first.
__device__ __forceinline__ bool is_padding(const int32_t *index, const float *value, int K)
{
    if (ld_uniform(index) >= 0)
        return false;
    bool some = false;
#pragma nounroll
    for (int k = threadIdx.x & (kWave - 1); k < K; k += kWave) {
        const float v = value[k];
        some = some || index[k] >= 0 || v != v;
    }
    return !__any(some);
}

// The teacher's total and the other tokens' probability from the sum over its
// entries (relative to their largest value where it is normalised).
__device__ __forceinline__ void teacher_total(double sum, bool renorm, double &total, double &rest)
{
    rest = renorm ? 0.0 : 1.0 - sum;
    if (rest < kLeastRest)
        rest = 0.0;
    total = !renorm ? sum + rest : sum != sum ? sum : sum == 0.0 ? 0.0 : 1.0;
}

// Distinct tokens of the vocabulary that a record names (one whole wave).
__device__ __forceinline__ int tokens_named(const int32_t *index, int K, int vocab, int lane)
{
    int named = 0;
    for (int k = lane; k < K; k += kWave) {
        const int id = index[k];
        bool lead = id >= 0 && id < vocab;
        for (int o = 0; o < k && lead; ++o)
            lead = index[o] != id;
        named += lead;
    }
    return wave_count(named);
}

// Clears a 16-byte aligned bitmap of `words` words (of a multiple of 4) and sets
// the bits id + base in [0, end) of a record's tokens (one whole wave).  True
// where one of them was set already: a token is named twice.
__device__ __forceinline__ bool mark_listed(unsigned *bits, int words, const int32_t *index, int K,
                                            int base, int end, int vocab, int lane)
{
    for (int i = lane; i < (words + 3) / 4; i += kWave)
        reinterpret_cast<u32x4 *>(bits)[i] = u32x4{0, 0, 0, 0};
    wave_sync();
    bool twice = false;
    for (int k = lane; k < K; k += kWave) {
        const int id = index[k], at = id + base;
        if (id >= 0 && id < vocab && at >= 0 && at < end) {
            const unsigned was = atomicOr(&bits[at >> 5], 1u << (at & 31));
            twice = twice || (was >> (at & 31) & 1);
        }
    }
    return __any(twice);
}

// Reads a row's record and the listed tokens' logits (one whole wave calls it).
// `twice`: some token is named by several entries.  Loops over a lane's entries are
// kept rolled and the entries in LDS: the wave may hold a row in its registers
// meanwhile.
template <typename T>
__device__ __forceinline__ void read_teacher(Teacher &te, const int32_t *index, const float *value,
                                             int K, int mode, const T *logits, int vocab,
                                             const Scale &sc, float scale, bool twice, int lane)
{
    const bool renorm = mode == ZERO_DISTILL_RENORM;
    bool bad = false;
    float top = kLowest, lm = -kInf;
#pragma nounroll
    for (int k = lane; k < K; k += kWave) {
        int id = index[k];
        const float val = value[k];
        bad = bad || id >= vocab || val != val;
        id = id < 0 || id >= vocab ? -1 : id;
        const float l = id >= 0 ? grad_at<T>(logits, id) : -kInf;
        te.index[k] = te.lead[k] = id;
        te.value[k] = id >= 0 ? val : -kInf;
        te.logit[k] = l;
        if (id >= 0)
            top = __builtin_fmaxf(top, val);
        lm = __builtin_fmaxf(lm, l);
    }
    bad = __any(bad);
    lm = wave_max(lm);
    // q: exp of the given value, or the softmax over the entries
    top = renorm ? wave_max(top) : 0.0f;
    double sum = 0.0;
#pragma nounroll
    for (int k = lane; k < K; k += kWave) {
        const double q = exp64((double)te.value[k] - (double)top);
        te.q[k] = q;
        sum += q;
    }
    sum = wave_sum(sum);
    double total, rest;
    teacher_total(sum, renorm, total, rest);
    const double ln = renorm ? log64(sum) + (double)top : 0.0;
    // entries that name the same token: the first of them stands for it.  The
    // student's share of the listed tokens and the loss's sum over the entries.
    wave_sync();
    const double part = renorm ? sum == 0.0 ? 0.0 : 1.0 / sum : 1.0;   // 0: no finite value
    const float ref = __builtin_fmaxf(lm, kLowest), r = ref * sc.c;
    int named = 0;
    float ls = 0.0f;
    double cross = 0.0;
#pragma nounroll
    for (int k = lane; k < K; k += kWave) {
        const int id = te.index[k];
        const double q = te.q[k] * part;
        double token_q = q;
        bool lead = id >= 0;
        if (lead && twice) {
            token_q = 0.0;
            for (int o = 0; o < K; ++o)
                if (te.index[o] == id) {
                    token_q += te.q[o] * part;
                    lead = lead && o >= k;
                }
            if (!lead)
                te.lead[k] = -1;
        }
        te.token_q[k] = token_q;
        named += lead;
        const float l = te.logit[k];
        if (lead)
            ls += pow2(rel(l, ref, r, sc));
        if (q != 0.0)   // NaN too
            cross += q * ((double)te.value[k] - ln - ((double)l - (double)ref) * (double)scale);
    }
    named = wave_count(named);
    ls = wave_add(ls);
    cross = wave_sum(cross);
    if (named == vocab && rest != 0.0) {   // no token is left for the rest
        total -= rest;
        rest = 0.0;
    }
    if (lane == 0) {
        te.total = total;
        te.rest = rest;
        te.cross = cross;
        te.listed_max = ref;
        te.listed_sum = ls;
        te.bad = bad;
    }
}

// The whole row's sum: the tail's (tokens not listed) and the listed tokens'.
__device__ __forceinline__ Total whole_row(const Total &tail, float listed_max, float listed_sum,
                                           const Scale &k)
{
    Total t{__builtin_fmaxf(tail.empty() ? kLowest : tail.m, listed_sum == 0.0f ? kLowest : listed_max),
            0.0f, 0.0f};
    if (!tail.empty())
        add_total(t, tail, k);
    if (listed_sum != 0.0f)
        add_total(t, Total{listed_max, listed_sum, 0.0f}, k);
    return t;
}

// The row's loss and statistics from the total over the tokens that are not
// listed (one lane, where the record is read).
__device__ __forceinline__ void finish_distill(Teacher &te, const Total &tail, const LossRows &in,
                                               float *loss, float *stats, int64_t row)
{
    const Scale k(in.c);
    const Total t = whole_row(tail, te.listed_max, te.listed_sum, k);
    const float log2z = log2f(t.s), ln = ln_sum(t, k);
    te.max = t.m;
    te.log2z = log2z;
    if (loss) {
        const double rest = te.rest;
        double v;
        if (t.empty()) {
            v = te.total == 0.0 ? 0.0 : te.total * (double)kInf;
        } else {
            // ln p of an entry = scale (logit - listed_max) - (scale (max - listed_max) + ln)
            v = te.cross;
            if (te.total - rest != 0.0)
                v += (te.total - rest) * (((double)t.m - (double)te.listed_max) * (double)in.scale + (double)ln);
            if (rest > 0.0) {
                const float lp = kLn2 * (log2f(tail.s) + shift_of(tail.m, t.m, k) - log2z);
                v += rest * ((double)(kLn2 * log2f((float)rest)) - (double)(tail.empty() ? -kInf : lp));
            }
        }
        // a NaN in the row reaches v only through entries with a probability
        loss[row] = te.bad || t.s != t.s ? __builtin_nanf("") : (float)v;
    }
    if (stats) {
        stats[4 * row] = t.empty() ? -kInf : t.m;
        stats[4 * row + 1] = t.empty() ? -kInf : ln;
        stats[4 * row + 2] = tail.empty() ? -kInf : tail.m;
        stats[4 * row + 3] = tail.empty() ? -kInf : ln_sum(tail, k);
    }
}
__device__ __forceinline__ void pad_distill(float *loss, float *stats, int64_t row)
{
    if (threadIdx.x == 0) {
        if (loss)
            loss[row] = 0.0f;
        if (stats)
            stats[4 * row] = stats[4 * row + 1] = stats[4 * row + 2] = stats[4 * row + 3] = 0.0f;
    }
}

// A listed token's gradient, entry k's: m the row's largest logit, off what
// log2 p is below t.
__device__ __forceinline__ float listed_grad(const Teacher &te, int k, float m, float off, double w,
                                             const Scale &sc)
{
    const float p = pow2(rel(te.logit[k], m, m * sc.c, sc) - off);
    return (float)(w * (te.total * (double)p - te.token_q[k]));
}

// Words of a segment's bitmap: one bit per element of its chunks, whose first
// and last may stick out of it.
constexpr int kBitWords = (int)(kLossMaxSegment / 32) + 8;

// One workgroup per segment of a row: the sum over its tokens that the teacher
// does not list, which a bitmap in LDS leaves out (subtracting the listed ones
// from the whole sum would lose the rest's digits where little is left).  A wide
// workgroup (few rows, each whole: latency counts) leaves the record to its last
// wave, beside the others' sums, and has its first chunks on their way before it
// looks at anything else: 3 x 50257 fp32 8.2 us; 2048 x 128256 bf16, 64 listed, 93 us,
// 5.6 TB/s.
template <typename T, int NT>
__global__ __launch_bounds__(NT) void distill_kernel(DistillArgs a, int64_t row0, int segs, int cps)
{
    constexpr bool kApart = NT == kWide;
    constexpr int U = kApart ? 8 : 4, W = Row<T>::W, NS = kApart ? NT - kWave : NT;
    __shared__ Total tot[NT / kWave];
    __shared__ Teacher te;
    __shared__ alignas(16) unsigned bits[kBitWords];
    const int64_t row_i = row0 + blockIdx.x / segs;
    const int seg = blockIdx.x % segs, tid = threadIdx.x, K = a.top_k, lane = tid & (kWave - 1);
    const int32_t *index = a.top_index + row_i * K;
    const float *value = a.top_value + row_i * K;
    const T *p = static_cast<const T *>(a.in.logits) + row_i * a.in.stride;
    const Row<T> row(p, a.in.vocab);
    const int k0 = min(seg * cps, row.chunks), k1 = min(k0 + cps, row.chunks);
    const Sweep<T> sweep(row, k0, k1);
    const int n = sweep.n;
    const bool teaches = tid / kWave == (kApart ? NS / kWave : 0);
    Chunk<T> ch[U];
    auto fetch = [&](int b) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            ch[u] = sweep.read(b + NS * u);
    };
    if (kApart && !teaches)
        fetch(0);
    if (is_padding(index, value, K)) {
        if (segs == 1)
            pad_distill(a.loss, a.stats, row_i);
        return;
    }
    const Scale sc(a.in.c);
    bool twice = false;
    auto read = [&] {
        read_teacher(te, index, value, K, a.mode, row.p, a.in.vocab, sc, a.in.scale, twice, lane);
    };
    if (teaches) {
        twice = mark_listed(bits, ((k1 - k0) * W + 31) / 32, index, K, row.phase - k0 * W,
                            (k1 - k0) * W, a.in.vocab, lane);
        if (!kApart && segs == 1)
            read();
    }
    __syncthreads();
    Sum q;
    if (kApart && teaches) {
        if (segs == 1)
            read();
    } else {
        if (!kApart)
            fetch(0);
        for (int b = 0; b < n;) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int first = b + NS * u;
                if (first >= n)
                    break;
                sweep.trim(ch[u], first, NS);
                float x[W];
                ch[u].widen(x);
                const int at = (min(max(first + tid, sweep.skip), n) + sweep.from - k0) * W;
                const unsigned listed = bits[at >> 5] >> (at & 31) & ((1u << W) - 1);
                if (listed) {
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        x[i] = listed >> i & 1 ? -kInf : x[i];
                }
                q.add<W, false>(x, sc);
            }
            b += NS * U;
            if (b < n)
                fetch(b);
        }
    }
    const int e = tid < 2 * W ? row.edge(tid, k0, k1) : -1;
    if (e >= 0) {
        const int at = e + row.phase - k0 * W;
        const float x[1] = {bits[at >> 5] >> (at & 31) & 1 ? -kInf : row.at(e)};
        q.add<1, false>(x, sc);
    }
    const Total t = block_total<false, NT / kWave>(q, sc, tot);
    if (segs > 1) {
        if (tid == 0)
            a.parts[row_i * segs + seg] = LossPart{t.m, t.s, 0.0f, 0.0f};
    } else if (tid == 0) {
        finish_distill(te, t, a.in, a.loss, a.stats, row_i);
    }
}

template <typename T>
__global__ __launch_bounds__(kNT) void distill_join_kernel(DistillArgs a, int64_t row0, int segs)
{
    __shared__ Total tot[kNW];
    __shared__ Teacher te;
    const int64_t r = row0 + blockIdx.x;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), K = a.top_k;
    const int32_t *index = a.top_index + r * K;
    const float *value = a.top_value + r * K;
    if (is_padding(index, value, K)) {
        pad_distill(a.loss, a.stats, r);
        return;
    }
    const Scale sc(a.in.c);
    if (tid < kWave)
        read_teacher(te, index, value, K, a.mode, static_cast<const T *>(a.in.logits) + r * a.in.stride,
                     a.in.vocab, sc, a.in.scale, true, lane);   // no bitmap of the row: look for them
    const Total t = join_parts(a.parts + r * segs, segs, sc, tot);
    if (tid == 0)
        finish_distill(te, t, a.in, a.loss, a.stats, r);
}

// d_logits_j = w (Q p_j - q_j) for a listed token and w (Q p_rest - q_rest)
// p_j / p_rest for the others (w = scale d_loss, Q the teacher's total), where
// p_j / p_rest is the softmax over the tokens that are not listed.  Every
// element is written in the second form first, then the listed ones again.
//
// One workgroup per kNT U chunks of a row, U to a thread, so that neighbouring
// workgroups sweep the memory in order.  Each wave adds up the record's
// probabilities for itself; a workgroup that holds no listed token needs nothing
// more of the record and no barrier.  (The first of sixteen waves adding them up
// for all, one chunk to a thread: 330 us for 2048 rows of 128256 bf16 and 64
// listed, where this takes 184: the other waves wait for its reads and products.)
// 2048 x 128256 bf16: 32 listed 179 us, 5.9 TB/s, 64 listed 184, 256 listed 230.
template <typename T, int U>
__global__ __launch_bounds__(kNT) void distill_grad_kernel(DistillGradArgs a, int64_t row0, int segs)
{
    constexpr int W = Row<T>::W;
    __shared__ Listed li;
    __shared__ alignas(16) unsigned bits[kNT * U * W / 32];
    const int64_t r = row0 + blockIdx.x / segs;
    const int k0 = (int)(blockIdx.x % segs) * (kNT * U);
    const int tid = threadIdx.x, lane = tid & (kWave - 1), K = a.top_k;
    T *out = static_cast<T *>(a.d_logits) + r * a.d_stride;
    const Row<T> row(static_cast<const T *>(a.in.logits) + r * a.in.stride, a.in.vocab);
    const int32_t *index = a.top_index + r * K;
    const float *value = a.top_value + r * K;
    const RowPart<T, kNT, U> seg(row, k0);   // on its way while the record is read
    const float dl = ld_uniform(a.d_loss + r);
    const float m = ld_uniform(a.stats + 4 * r), ln = ld_uniform(a.stats + 4 * r + 1);
    const float tm = ld_uniform(a.stats + 4 * r + 2), tln = ld_uniform(a.stats + 4 * r + 3);
    const bool renorm = a.mode == ZERO_DISTILL_RENORM;
    const int first = k0 * W - row.phase, last = first + kNT * U * W;   // the workgroup's elements
    bool some = false, bad = false, here = false;
    float top = kLowest;
    for (int k = lane; k < K; k += kWave) {
        const int id = index[k];
        const float v = value[k];
        some = some || id >= 0 || v != v;
        bad = bad || id >= a.in.vocab || v != v;
        here = here || (id >= 0 && id < a.in.vocab && id >= first && id < last);
        if (id >= 0 && id < a.in.vocab)
            top = __builtin_fmaxf(top, v);
    }
    some = __any(some);
    bad = __any(bad);
    here = __any(here);
    const bool zero = !some || dl == 0.0f;
    if (zero || bad || m == -kInf) {
        fill_row(row, out, k0, k0 + kNT * U, bad && !zero ? __builtin_nanf("") : 0.0f);
        return;
    }
    top = renorm ? wave_max(top) : 0.0f;
    double sum = 0.0;
    for (int k = lane; k < K; k += kWave) {
        const int id = index[k];   // below vocab: the row is not bad
        const double q = id >= 0 ? exp64((double)value[k] - (double)top) : 0.0;
        sum += q;
        if (here && tid < kWave) {   // the first wave leaves the record for the listed tokens
            li.index[k] = id;
            li.q[k] = q;
            // an entry of padding is no element, also where the row's first chunk
            // starts before the row (first < 0)
            li.logit[k] = id >= 0 && id >= first && id < last ? row.at(id) : 0.0f;
        }
    }
    sum = wave_sum(sum);
    if (here && tid < kWave)
        li.twice = mark_listed(bits, kNT * U * W / 32, index, K, -first, last - first, a.in.vocab, lane);
    double total, rest;
    teacher_total(sum, renorm, total, rest);
    // where the record may name the whole vocabulary, no token may be left for the
    // rest (the statistics say whether one has a probability, not whether it is there)
    if (K >= a.in.vocab && rest != 0.0 && tokens_named(index, K, a.in.vocab, lane) == a.in.vocab) {
        total -= rest;
        rest = 0.0;
    }
    const double w = (double)dl * (double)a.in.scale;
    const Scale k(a.in.c);
    // ln p_rest, then log2 of the tail's softmax = t - off
    const float ref = tm * k.c, off = residue(tm, k) + tln * kLog2E;
    const float rest_ln = (float)(((double)tm - (double)m) * (double)a.in.scale + ((double)tln - (double)ln));
    const float coef = (float)(w * (total * (double)pow2(rest_ln * kLog2E) - rest)) * pow2(-off);
    if (here)   // in place: the listed logits are read before any is overwritten
        __syncthreads();
    if (tm == -kInf)   // all others are masked: NaN where a listed logit is NaN or +inf
        fill_row(row, out, k0, k0 + kNT * U, ln != ln ? __builtin_nanf("") : 0.0f);
    else if (__builtin_fabsf(tm) > k.big)
        seg.map(row, out, [&](float x) { return coef * pow2((x - tm) * k.c); });
    else
        seg.map(row, out, [&](float x) { return coef * pow2(__builtin_fmaf(x, k.c, -ref)); });
    if (!here)
        return;
    __syncthreads();
    // the listed tokens of this workgroup, each by its first entry
    const bool look = li.twice;
    const double part = renorm ? sum == 0.0 ? 0.0 : 1.0 / sum : 1.0;
    const float whole_off = residue(m, k) + ln * kLog2E;
    for (int i = tid; i < K; i += kNT) {
        const int id = li.index[i];
        if (id < first || id >= last || id < 0 || id >= a.in.vocab)
            continue;
        double q = li.q[i];
        bool lead = true;
        if (look) {
            q = 0.0;
            for (int o = 0; o < K; ++o)
                if (li.index[o] == id) {
                    q += li.q[o];
                    lead = lead && o >= i;
                }
        }
        const float p = pow2(rel(li.logit[i], m, m * k.c, k) - whole_off);
        if (lead)
            store_one(out + id, (float)(w * (total * (double)p - q * part)));
    }
}

constexpr int kHeld = 17;   // chunks a thread holds: 960 threads hold 128256 bf16

// Forward and backward of whole rows, at most kHeld NS chunks each, by NS threads
// and one more wave, which reads the next row's record while the others sum the
// row, and writes the listed tokens' gradients while they sum the next one:
// what takes its time there are a few dependent reads, which would hold up a
// wave that also has its share of the row.  Records and bitmaps have two places.
// 4096 x 128256 bf16, 64 listed: 399 us, 5.3 TB/s (497 us with the record in the
// hands of a wave that also sums); 511 x 50257 27 us.  A copy kernel that only holds
// such rows, 1024 and 512 threads to a row, takes 361 and 22.
template <typename T, int NS, bool SAME>
__global__ __launch_bounds__(NS + kWave) __attribute__((amdgpu_waves_per_eu(4)))
void distill_row_kernel(DistillArgs a, DistillGradArgs b)
{
    typedef HeldRow<T, NS, kHeld, SAME> Held;
    constexpr int W = Row<T>::W, N = Held::G * W;
    constexpr int kWords = (((NS * kHeld + 1) * W + 31) / 32 + 3) / 4 * 4;
    __shared__ Total tot[2][NS / kWave];
    __shared__ Teacher teacher[2];
    __shared__ alignas(16) unsigned bitmap[2][kWords];   // the row's listed tokens
    __shared__ alignas(16) unsigned dirty[2][NS];        // a thread's chunks that hold one
    __shared__ u32x4 park[NS * parked(NS) + 1];
    __shared__ unsigned written;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), K = a.top_k;
    const bool sums = __builtin_amdgcn_readfirstlane(tid / kWave) < NS / kWave;
    const Scale k(a.in.c);
    auto out_at = [&](int64_t r) { return static_cast<T *>(b.d_logits) + r * b.d_stride; };
    auto row_at = [&](int64_t r) {
        return Row<T>(static_cast<const T *>(a.in.logits) + r * a.in.stride, a.in.vocab);
    };
    auto skip_padding = [&](int64_t r) {
        while (r < a.in.rows && is_padding(a.top_index + r * K, a.top_value + r * K, K)) {
            const Row<T> row = row_at(r);
            pad_distill(a.loss, a.stats, r);
            if (sums)
                fill_row<T, NS>(row, out_at(r), 0, row.chunks, 0.0f);
            r += gridDim.x;
        }
        return r;
    };
    auto mark_record = [&](int64_t r, const Row<T> &row, int set) {
        const int32_t *index = a.top_index + r * K;
        const bool twice = mark_listed(bitmap[set], (row.chunks * W + 31) / 32, index, K, row.phase,
                                       row.chunks * W, a.in.vocab, lane);
        for (int i = lane; i < NS / 4; i += kWave)
            reinterpret_cast<u32x4 *>(dirty[set])[i] = u32x4{0, 0, 0, 0};
        wave_sync();
        for (int i = lane; i < K; i += kWave) {
            const int id = index[i], c = (id + row.phase) / W;
            if (id >= 0 && id < a.in.vocab && c >= row.full_lo && c < row.full_hi)
                atomicOr(&dirty[set][c % NS], 1u << c / NS);
        }
        return twice;
    };
    auto read_record = [&](int64_t r, const Row<T> &row, int set, bool twice) {
        read_teacher(teacher[set], a.top_index + r * K, a.top_value + r * K, K, a.mode, row.p, a.in.vocab,
                     k, a.in.scale, twice, lane);
    };
    // What both halves need of a row once its sum is known (barrier, then this).
    auto outcome = [&](int64_t r, const Teacher &te, const Total &t, float &dl, bool &fill) {
        dl = ld_uniform(b.d_loss + r);
        fill = dl == 0.0f || te.bad || (t.empty() && te.listed_sum == 0.0f);
    };
    int64_t r = skip_padding(blockIdx.x);
    if (r >= a.in.rows)
        return;
    // Two loops with the same barriers, one before the first row and one when a row
    // is summed.  The waves that hold a row count in `written` when its gradients
    // are on their way; only the other wave waits for that, so each of them can go
    // on to sum the next row by itself.
    if (!sums) {
        if (lane == 0)
            written = 0;
        const bool twice = mark_record(r, row_at(r), 0);
        __syncthreads();
        read_record(r, row_at(r), 0, twice);   // beside the first row's sums
        unsigned all = 0;
        for (int turn = 0;; turn ^= 1) {
            Teacher &te = teacher[turn];
            const int64_t rn = skip_padding(r + gridDim.x);
            if (rn < a.in.rows)
                read_record(rn, row_at(rn), turn ^ 1, mark_record(rn, row_at(rn), turn ^ 1));
            __syncthreads();
            const Total t = add_waves<false, NS / kWave>(tot[turn], k);
            float dl;
            bool fill;
            outcome(r, te, t, dl, fill);
            if (lane == 0)
                finish_distill(te, t, a.in, a.loss, a.stats, r);
            all += NS / kWave;
            while (__hip_atomic_load(&written, __ATOMIC_ACQUIRE, __HIP_MEMORY_SCOPE_WORKGROUP) != all)
                __builtin_amdgcn_s_sleep(1);
            if (!fill) {
                const double w = (double)dl * (double)a.in.scale;
                T *out = out_at(r);
                for (int i = lane; i < K; i += kWave)
                    if (te.lead[i] >= 0)
                        store_one(out + te.lead[i], listed_grad(te, i, te.max, te.log2z, w, k));
            }
            if (rn >= a.in.rows)
                return;
            r = rn;
        }
    }
    Held held;
    held.park = park;
    held.read(row_at(r));
    held.take(row_at(r));
    __syncthreads();
    for (int turn = 0;; turn ^= 1) {
        const Teacher &te = teacher[turn];
        const unsigned *bits = bitmap[turn];
        const int64_t rn = skip_padding(r + gridDim.x);
        const Row<T> next = rn < a.in.rows ? row_at(rn) : Row<T>();
        const unsigned mine = dirty[turn][tid];
        Sum q;
        held.each_group([&](int i, float (&x)[N]) {
#pragma unroll
            for (int j = 0; j < N / W; ++j)
                if (mine >> (i + j) & 1) {
                    int t = tid;
                    asm volatile("" : "+v"(t));   // or the places of all chunks would be kept over all rows
                    const int at = (t + NS * (i + j)) * W;
                    const unsigned listed = bits[at >> 5] >> (at & 31);
#pragma unroll
                    for (int w = 0; w < W; ++w)
                        x[j * W + w] = listed >> w & 1 ? -kInf : x[j * W + w];
                }
            q.template add<N, false>(x, k);
        });
        if (held.e >= 0) {
            const int at = held.e + held.row.phase;
            const float x[1] = {bits[at >> 5] >> (at & 31) & 1 ? -kInf : held.edge};
            q.template add<1, false>(x, k);
        }
        const Total own = wave_total<false>(q, k);
        if (lane == 0)
            tot[turn][tid / kWave] = own;
        __syncthreads();
        const Total t = add_waves<false, NS / kWave>(tot[turn], k);
        T *out = out_at(r);
        float dl;
        bool fill;
        outcome(r, te, t, dl, fill);
        const bool big = __builtin_fabsf(t.m) > k.big;
        // the rest's share of the whole sum, then the coefficient of 2^t
        const double w = (double)dl * (double)a.in.scale;
        const Total whole = whole_row(t, te.listed_max, te.listed_sum, k);
        const float share = t.s * pow2(shift_of(t.m, whole.m, k)) / whole.s;
        const float coef = (float)(w * (te.total * (double)share - te.rest)) / t.s;
        const float m = t.m, ref = m * k.c;
        if (fill || t.empty())   // NaN too where a listed logit is NaN or +inf and all others are masked
            fill_row<T, NS>(held.row, out, 0, held.row.chunks,
                            dl != 0.0f && (te.bad || whole.s != whole.s) ? __builtin_nanf("") : 0.0f);
        else if (big)   // rare: from memory, so that the held row's code is not there twice
            for (int k0 = 0; k0 < held.row.chunks; k0 += NS)
                RowPart<T, NS, 1>(held.row, k0).map(held.row, out,
                                                    [&](float x) { return coef * pow2((x - m) * k.c); });
        held.map(out, !fill && !t.empty() && !big, next,
                 [&](float x) { return coef * pow2(__builtin_fmaf(x, k.c, -ref)); });
        if (lane == 0)
            __hip_atomic_fetch_add(&written, 1u, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_WORKGROUP);
        held.take(next);
        if (rn >= a.in.rows)
            return;
        r = rn;
    }
}

// -- launches ---------------------------------------------------------------------------------

template <typename T>
int launch_distill_of(const DistillArgs &a, int segs, hipStream_t st)
{
    const int cps = chunks_per<T>(a.in.vocab, segs);
    if (segs == 1 && wide_rows(a.in)) {
        hipLaunchKernelGGL((distill_kernel<T, kWide>), dim3((unsigned)a.in.rows), dim3(kWide), 0, st, a,
                           (int64_t)0, 1, cps);
        return hipGetLastError();
    }
    if (int e = each_launch(a.in.rows, segs, [&](int64_t r, unsigned n) {
            hipLaunchKernelGGL((distill_kernel<T, kNT>), dim3(n * (unsigned)segs), dim3(kNT), 0, st, a, r,
                               segs, cps);
        }))
        return e;
    if (segs == 1)
        return hipSuccess;
    return each_launch(a.in.rows, 1, [&](int64_t r, unsigned n) {
        hipLaunchKernelGGL((distill_join_kernel<T>), dim3(n), dim3(kNT), 0, st, a, r, segs);
    });
}

// Threads that hold a row in registers; 0: the row is too long for 960.
template <typename T>
int held_threads(int vocab)
{
    const int most = chunks_per<T>(vocab, 1);
    return most <= 64 * kHeld ? 64 : most <= 192 * kHeld ? 192 : most <= 448 * kHeld ? 448
         : most <= 960 * kHeld ? 960 : 0;
}

template <typename T, int NS>
int launch_distill_row_ns(const DistillArgs &a, const DistillGradArgs &b, hipStream_t st)
{
    const dim3 grid(held_grid(a.in.rows, NS + kWave)), block(NS + kWave);
    if (same_phase(a.in, b.d_logits, b.d_stride))
        hipLaunchKernelGGL((distill_row_kernel<T, NS, true>), grid, block, 0, st, a, b);
    else
        hipLaunchKernelGGL((distill_row_kernel<T, NS, false>), grid, block, 0, st, a, b);
    return hipGetLastError();
}
template <typename T>
int launch_distill_row(const DistillArgs &a, const DistillGradArgs &b, hipStream_t st)
{
    const int threads = held_threads<T>(a.in.vocab);
    return threads == 64  ? launch_distill_row_ns<T, 64>(a, b, st)
         : threads == 192 ? launch_distill_row_ns<T, 192>(a, b, st)
         : threads == 448 ? launch_distill_row_ns<T, 448>(a, b, st)
                          : launch_distill_row_ns<T, 960>(a, b, st);
}

}  // namespace

int launch_distill(const DistillArgs &a, int32_t segs, void *stream)
{
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return a.in.dtype == ZERO_BF16 ? launch_distill_of<uint16_t>(a, segs, st)
                                   : launch_distill_of<float>(a, segs, st);
}

int launch_distill_grad(const DistillGradArgs &a, void *stream)
{
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    const bool bf = a.in.dtype == ZERO_BF16;
    const int chunks = bf ? chunks_per<uint16_t>(a.in.vocab, 1) : chunks_per<float>(a.in.vocab, 1);
    auto launch = [&](auto u) {
        constexpr int U = decltype(u)::value;
        const int segs = (chunks + kNT * U - 1) / (kNT * U);
        return each_launch(a.in.rows, segs, [&](int64_t r, unsigned n) {
            const dim3 grid(n * (unsigned)segs), block(kNT);
            if (bf)
                hipLaunchKernelGGL((distill_grad_kernel<uint16_t, U>), grid, block, 0, st, a, r, segs);
            else
                hipLaunchKernelGGL((distill_grad_kernel<float, U>), grid, block, 0, st, a, r, segs);
        });
    };
    // Fewer workgroups add up long records (2048 rows of 128256 bf16, U = 4 and 8:
    // 186 and 195 us at 64 listed, one to a lane; 213 and 202 at 128; 286 and 230
    // at 256).
    return a.top_k <= kWave ? launch(std::integral_constant<int, 4>())
                            : launch(std::integral_constant<int, 8>());
}

bool distill_row_held(const LossRows &in)
{
    return (in.dtype == ZERO_BF16 ? held_threads<uint16_t>(in.vocab) : held_threads<float>(in.vocab)) > 0;
}

int launch_distill_fused(const DistillArgs &a, const DistillGradArgs &b, void *stream)
{
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return a.in.dtype == ZERO_BF16 ? launch_distill_row<uint16_t>(a, b, st)
                                   : launch_distill_row<float>(a, b, st);
}

}  // namespace zero
